"""GPU: stq_attn_prompt, causal softmax attention over packed prompts, against
numpy in fp64."""
import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


class _Attn:
    def __init__(self, lens, heads, kv_heads, kind="bf16", prefix=0, seed=0, spread=1.0, pad=0):
        rng = np.random.default_rng(seed)
        self.lq = list(lens)
        self.lk = [max(0, m + p) for m, p in zip(lens, prefix if isinstance(prefix, list) else [prefix] * len(lens))]
        self.heads, self.kv, self.dt = heads, kv_heads, TYPES[kind]
        self.qs, self.ks = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (self.lq, self.lk))
        tq, tk = sum(self.lq) + pad, sum(self.lk) + pad
        self.q = _cuda(rng.standard_normal((tq, heads, 128)) * spread).to(self.dt)
        self.k = _cuda(rng.standard_normal((tk, kv_heads, 128)) * spread).to(self.dt)
        self.v = _cuda(rng.standard_normal((tk, kv_heads, 128))).to(self.dt)
        self.q_start, self.k_start = _cuda(self.qs), _cuda(self.ks)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **more):
        y = torch.full(self.q.shape, 55.0, dtype=self.dt, device="cuda")
        stq.stq_attn_prompt(self.q_start, self.k_start, self.q, self.k, self.v, y, err=self.err, **more)
        torch.cuda.synchronize()
        return y

    def check(self, y, scale=128 ** -0.5):
        """A weight is rounded to the type (half a step of itself) and y once more; a score's fp32 sum of 128 exact
        products is off by less than 2^-17 of their sizes, a weight by twice a score's error; exp2 and the weights' sum
        by 2^-20."""
        f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        y, q, k, v = f(y), f(self.q), f(self.k), f(self.v)
        half = torch.finfo(self.dt).eps / 2
        g = self.heads // self.kv
        assert int(self.err[0]) == 0
        for i, (m, n) in enumerate(zip(self.lq, self.lk)):
            if m == 0:
                continue
            for h in range(self.heads):
                qq = q[self.qs[i]:self.qs[i + 1], h]
                kk, vv = (t[self.ks[i]:self.ks[i + 1], h // g] for t in (k, v))
                seen = np.arange(n)[None] <= np.arange(m)[:, None] + n - m
                x = np.where(seen, qq @ kk.T * scale, -np.inf)
                top = x.max(1, keepdims=True, initial=-np.inf)
                p = np.exp(x - np.where(np.isfinite(top), top, 0))
                s = p.sum(1, keepdims=True)
                p = p / np.where(s == 0, 1, s)
                want = p @ vv
                size = np.where(seen, np.abs(qq) @ np.abs(kk).T, 0).max(1, keepdims=True, initial=0) * abs(scale)
                tol = (half + 2 * size * 2.0 ** -17 + 2.0 ** -20) * (p @ np.abs(vv)) + 1.01 * half * np.abs(want) + 2.0 ** -24
                got = y[self.qs[i]:self.qs[i + 1], h]
                bad = ~(np.abs(got - want) <= tol)
                assert not bad.any(), (i, h, m, n, np.argwhere(bad)[:3], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 2), (3, 1), (12, 2), (16, 1)])
def test_prompts(kind, heads, kv_heads):
    """Group sizes that fill a tile's rows by 1, 2, 4 and 16 heads; lengths around tiles; empty and one-token prompts."""
    a = _Attn([1, 0, 63, 64, 65, 127, 130, 300, 2], heads, kv_heads, kind, seed=heads)
    a.check(a.run())


@pytest.mark.parametrize("lens, prefix", [([1], 0), ([700], 0), ([5, 40, 300], [1000, 128, 77]), ([130, 64, 1, 200], [-100, -64, 0, -1]),
                                          ([1] * 70, 0), ([1, 1, 1], [0, 127, 128]), ([256, 257], [256, 255])])
@pytest.mark.parametrize("heads, kv_heads", [(2, 2), (8, 1)])
def test_pieces(lens, prefix, heads, kv_heads):
    """Pieces behind earlier keys, and more queries than keys: rows that see none are zero."""
    a = _Attn(lens, heads, kv_heads, prefix=prefix, seed=len(lens))
    a.check(a.run())


def test_many_short_prompts():
    """Far more sequences than a warp looks at once, some of them empty."""
    s = _Attn([(7 * i) % 5 for i in range(1500)], 4, 2)
    s.check(s.run())


def test_one_long_prompt():
    a = _Attn([2300], 2, 1, seed=3)
    a.check(a.run())


@pytest.mark.parametrize("spread, scale", [(0.02, None), (4.0, None), (1.0, 1.5), (1.0, -0.2), (1.0, 0.0)])
def test_sharp_and_flat_weights(spread, scale):
    """Weights from all alike to one alone, rising maxima along the keys, scales of either sign and of zero."""
    a = _Attn([400, 129], 4, 2, "fp16" if spread < 1 else "bf16", seed=4, spread=spread)
    ramp = torch.linspace(0.1, 3.0, a.k.shape[0], device="cuda")[:, None, None]
    a.k = (a.k.float() * ramp).to(a.dt)
    a.check(a.run(scale=scale), 128 ** -0.5 if scale is None else scale)


def test_strided_parts_of_one_projection():
    a = _Attn([77, 200, 3], 8, 2, seed=5)
    want = a.run()
    fused = torch.empty(280, 12, 128, dtype=a.dt, device="cuda")
    fused[:, :8], fused[:, 8:10], fused[:, 10:] = a.q, a.k, a.v
    a.q, a.k, a.v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    assert torch.equal(a.run(), want)
    # heads outermost
    a.q, a.k, a.v = (t.permute(1, 0, 2).contiguous().permute(1, 0, 2) for t in (a.q, a.k, a.v))
    assert torch.equal(a.run(), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_and_padding_are_not_seen(bad):
    """Rows behind the last sequence hold infinities, and so does a sequence between the others: nobody else notices."""
    lens = [100, 60, 200]
    a = _Attn(lens, 4, 2, seed=6, pad=150)
    m = sum(lens)
    for t in (a.q, a.k, a.v):
        t[m:] = bad
    y = a.run()
    a.check(y)
    assert bool((y[m:] == 55).all())
    a.k[100:160] = bad
    a.v[100:160] = bad
    z = a.run()
    assert torch.equal(z[:100], y[:100]) and torch.equal(z[160:m], y[160:m])


def test_bad_ranges_are_skipped_and_reported():
    a = _Attn([50, 60, 70], 4, 2, seed=7, pad=5)
    y = a.run()
    a.k_start = _cuda(np.array([0, 50, 40, 110], np.int32))
    z = a.run()
    assert int(a.err[0]) == stq.STQ_ERR_INDEX
    assert torch.equal(z[:50], y[:50]) and bool((z[50:110] == 55).all())
    a.err.zero_()
    a.k_start, a.q_start = _cuda(a.ks), _cuda(np.array([0, 50, 110, 10 ** 6], np.int32))
    z = a.run()
    assert int(a.err[0]) == stq.STQ_ERR_INDEX
    assert torch.equal(z[:110], y[:110]) and bool((z[110:] == 55).all())


def test_repeats_graphs_and_streams():
    a = _Attn([333, 20, 128], 8, 2, seed=8)
    y = a.run()
    assert torch.equal(y, a.run())
    out = torch.zeros_like(y)
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        stq.stq_attn_prompt(a.q_start, a.k_start, a.q, a.k, a.v, out)
    b = _Attn([200, 153, 128], 8, 2, seed=9)
    for name in ("q", "k", "v", "q_start", "k_start"):
        getattr(a, name).copy_(getattr(b, name))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    b.check(out)
    out.zero_()
    torch.cuda.synchronize()
    stq.stq_attn_prompt(a.q_start, a.k_start, a.q, a.k, a.v, out, stream=stream)
    stream.synchronize()
    b.check(out)


def test_nothing_to_do_and_refusals():
    before = stq.stq_launch_count()
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    stq.stq_attn_prompt(one, one, e, e[:, :2], e[:, :2], e.clone())
    s = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    q, k = (torch.zeros(8, h, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2))

    def refused(error, status=None, q=q, k=k, v=k, y=q, q_start=s, k_start=s, **more):
        with pytest.raises(error) as info:
            stq.stq_attn_prompt(q_start, k_start, q, k, v, y, **more)
        if status is not None:
            assert info.value.status == status

    refused(TypeError, k=k.half())
    refused(TypeError, y=q.float())
    refused(ValueError, v=k[:7])
    refused(ValueError, y=q[:7])
    refused(ValueError, k_start=one)
    refused(ValueError, q=q.mT.contiguous().mT)
    refused(ValueError, q_start=s.cpu())
    refused(stq.StqError, stq.STQ_ERR_UNSUPPORTED, q=q.float(), k=k.float(), v=k.float(), y=q.float())
    refused(stq.StqError, stq.STQ_ERR_UNSUPPORTED, k=k[:, :1].expand(-1, 2, -1))
    refused(stq.StqError, stq.STQ_ERR_ARG, q=q[:, :3], y=q[:, :3].contiguous())
    refused(stq.StqError, stq.STQ_ERR_ARG, scale=float("inf"))
    refused(stq.StqError, stq.STQ_ERR_ARG, v=torch.zeros(8, 2, 132, dtype=torch.bfloat16, device="cuda")[..., 1:129])
    assert stq.stq_launch_count() == before
