"""GPU: the 4-bit cache (append, read) and attention of single tokens over it,
against plain numpy implementations (the codes bit for bit, attention in fp64)."""
import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _quantized(x):
    """The values 4-bit codes stand for: x fp32 [..., 128], a binary16 scale per 32 values."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], 4, 32)
    s = (np.abs(g).max(-1, keepdims=True) / np.float32(7)).astype(np.float16).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s > 0, np.rint(g / s), 0)
    return (np.clip(z, -7, 7) * s).astype(np.float32).reshape(x.shape)


class _Sequences:
    """Sequences of the given lengths in a cache, their pages in a shuffled order."""

    def __init__(self, lens, heads, kv_heads, kind="bf16", seed=0, spread=1.0, size=1.0, extra_pages=1):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv_heads, self.dt = list(lens), heads, kv_heads, TYPES[kind]
        n, pages = len(lens), [(m + 63) // 64 for m in lens]
        self.max_pages = max(max(pages), 1) + extra_pages
        order = rng.permutation(sum(pages) + 3)
        self.table = np.full((n, self.max_pages), -7, np.int32)  # entries that no length reaches are never read
        self.slots, at = [], 0
        for i, p in enumerate(pages):
            self.table[i, :p] = order[at:at + p]
            at += p
            t = np.arange(lens[i])
            self.slots.append(self.table[i][t // 64].astype(np.int64) * 64 + t % 64)
        tokens = sum(lens)
        k = rng.standard_normal((tokens, kv_heads, 128)) * spread
        v = rng.standard_normal((tokens, kv_heads, 128)) * size
        k[..., 5] *= 5
        self.k, self.v = _cuda(k).to(self.dt), _cuda(v).to(self.dt)
        self.q = _cuda(rng.standard_normal((n, heads, 128)) * spread).to(self.dt)
        self.cache = stq.stq_cache_create(sum(pages) + 3, kv_heads)
        self.slot = _cuda(np.concatenate(self.slots) if tokens else np.zeros(0, np.int64))
        self.page_table, self.seq_len = _cuda(self.table), _cuda(np.array(lens, np.int32))

    def append(self):
        stq.stq_cache_append(self.cache, self.slot, self.k, self.v)

    def attend(self, **more):
        y = torch.full((len(self.lens), self.heads, 128), float("nan"), dtype=self.dt, device="cuda")
        stq.stq_attn_decode(self.cache, self.page_table, self.seq_len, self.q, y, **more)
        stq.stq_cache_check(self.cache)
        return y

    def check(self, y, scale=128 ** -0.5):
        """Against fp64 attention over the quantized values.  A weight is rounded to binary16, and so is its product with
        its value's scale (2^-11 each); a score's error delta changes a weight by at most 2 delta of itself; y is rounded
        once; q in binary16 after scaling is exact for 16-bit types and rounded by 2^-11 for fp32.  Weights are held as
        2^15 w / (w_max up) at most and 2^11 at least, with up at most twice the largest value scale or 1, so where they or
        their products are subnormal each of the two roundings is off by up to half of 2^-24: w_max up 2^-36 (1 + s), times
        |z| <= 7 each."""
        got = y.float().cpu().numpy().astype(np.float64)
        k, v = (_quantized(x.float().cpu().numpy()).astype(np.float64) for x in (self.k, self.v))
        q = self.q.float().cpu().numpy().astype(np.float64)
        g, at = self.heads // self.kv_heads, 0
        half_step = torch.finfo(self.dt).eps / 2
        for i, m in enumerate(self.lens):
            if m == 0:
                assert np.all(got[i] == 0)
                continue
            for h in range(self.heads):
                kk, vv = k[at:at + m, h // g], v[at:at + m, h // g]
                x = kk @ q[i, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                ref = p @ vv
                size = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
                delta = size * (2.0 ** -11 if self.dt == torch.float32 else 2.0 ** -19)
                s_max = np.abs(vv).max() / 7 * 1.01
                small = 2.0 ** -36 * p.max() * max(1.0, 2 * s_max) * (1 + s_max) * 7 * m
                tol = small + (2.0 ** -10 + 2 * delta + 2.0 ** -18) * (p @ np.abs(vv)) + 1.01 * half_step * np.abs(ref) + 1e-30
                bad = np.abs(got[i, h] - ref) > tol + (2.0 ** -25 if self.dt == torch.float16 else 0)
                assert not bad.any(), (i, h, m, np.abs(got[i, h] - ref)[bad][:4], tol[bad][:4])
            at += m


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads", [1, 3])
def test_append_and_read_are_the_quantizer(kind, heads):
    """Codes and scales bit for bit, at sizes from subnormal to large, tokens in any order, padded rows skipped."""
    rng = np.random.default_rng(3)
    n = 333
    x = rng.standard_normal((2, n, heads, 128)) * np.exp(rng.uniform(-12, 6, (2, n, heads, 1)))
    x[0, 5] = 0.0
    x[1, 7, 0, 32:64] = 1e-9  # a group whose scale underflows is zero
    k, v = (_cuda(a).to(TYPES[kind]) for a in x)
    cache = stq.stq_cache_create(9, heads)
    slot = rng.permutation(9 * 64)[:n].astype(np.int64)
    slot[[3, 100]] = -1
    stq.stq_cache_append(cache, _cuda(slot), k, v)
    stq.stq_cache_check(cache)
    out = [torch.full((n, heads, 128), 7.0, device="cuda") for _ in range(2)]
    stq.stq_cache_read(cache, _cuda(slot), *out)
    stq.stq_cache_check(cache)
    for got, a in zip(out, (k, v)):
        want = _quantized(a.float().cpu().numpy())
        want[slot < 0] = 7.0
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_append_one_token_of_a_pair_leaves_the_other():
    """Value words hold two tokens: each append changes its own alone, alone or both in a call."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, 2, 2, 128)).astype(np.float32)
    cache = stq.stq_cache_create(1, 2)
    slots = [torch.tensor(s, dtype=torch.int64, device="cuda") for s in ([10, 11], [11], [10], [11, 10])]
    held = {}
    for s, a in zip(slots, x):
        m = len(s)
        stq.stq_cache_append(cache, s, _cuda(a[:m]), _cuda(-a[:m]))
        for j, at in enumerate(s.tolist()):
            held[at] = a[j]
        out = [torch.empty(2, 2, 128, device="cuda") for _ in range(2)]
        stq.stq_cache_read(cache, slots[0], *out)
        want = _quantized(np.stack([held[10], held[11]]))
        np.testing.assert_array_equal(out[0].cpu().numpy(), want)
        np.testing.assert_array_equal(out[1].cpu().numpy(), -want)


def test_append_reports_what_it_cannot_hold():
    cache = stq.stq_cache_create(2, 2)
    k = torch.ones(4, 2, 128, device="cuda")
    v = k.clone()
    k[0, 1, 40], v[1, 0, 3], k[2, 0, 127] = float("nan"), float("inf"), 1e9  # the last one's scale overflows binary16
    slot = torch.tensor([0, 1, 2, 3], dtype=torch.int64, device="cuda")
    stq.stq_cache_append(cache, slot, k, v)
    assert stq.stq_cache_check(cache, raise_on_error=False) == stq.STQ_ERR_NONFINITE
    assert stq.stq_cache_check(cache, raise_on_error=False) == stq.STQ_OK
    out = [torch.empty(4, 2, 128, device="cuda") for _ in range(2)]
    stq.stq_cache_read(cache, slot, *out)
    want_k, want_v = np.ones((4, 2, 128), np.float32), np.ones((4, 2, 128), np.float32)
    want_k[0, 1, 32:64] = want_v[1, 0, :32] = want_k[2, 0, 96:] = 0
    # ones: s = half(1 / 7), z = 7
    one = _quantized(np.ones((1, 128), np.float32))[0, 0]
    np.testing.assert_array_equal(out[0].cpu().numpy(), want_k * one)
    np.testing.assert_array_equal(out[1].cpu().numpy(), want_v * one)
    stq.stq_cache_append(cache, torch.tensor([0, 128, -5, 1], dtype=torch.int64, device="cuda"), v * 0, v * 0)
    assert stq.stq_cache_check(cache, raise_on_error=False) == stq.STQ_ERR_INDEX


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 2), (6, 2), (9, 1), (32, 2), (40, 2), (14, 2)])
def test_attend(kind, heads, kv_heads):
    """Group sizes on both sides of a block of 8 and of 16; lengths around pages and of zero."""
    s = _Sequences([0, 1, 63, 64, 65, 200, 1000], heads, kv_heads, kind, seed=heads)
    s.append()
    s.check(s.attend())


@pytest.mark.parametrize("lens", [[1], [100], [5000, 0, 0, 3], [30000], [70] * 150, [64 * 31, 64 * 33 + 1, 2]])
def test_attend_shares(lens):
    """One long sequence over all CTAs, many short ones to a CTA, empty ones between."""
    s = _Sequences(lens, 8, 2, "bf16", seed=len(lens))
    s.append()
    y = s.attend()
    s.check(y)
    assert torch.equal(y, s.attend())


@pytest.mark.parametrize("spread, size", [(1e-3, 1.0), (6.0, 1.0), (1.0, 2000.0), (1.0, 1e-4), (3.0, 3e4)])
def test_attend_sizes(spread, size):
    """Sharp and flat weights; values from near binary16's subnormals to near its end."""
    s = _Sequences([700, 3, 129], 8, 2, "fp32", spread=spread, size=size)
    s.append()
    s.check(s.attend())


def test_attend_many_sequences():
    """More sequences than warps look at once, and more segments than shares."""
    s = _Sequences([(37 * i) % 131 for i in range(900)], 4, 2, "bf16", seed=21)
    s.append()
    s.check(s.attend())


def test_attend_values_of_mixed_sizes():
    """Tokens and groups whose values differ by orders: each dim to its own group's size."""
    s = _Sequences([900, 65], 8, 2, "bf16", seed=5)
    f = torch.ones(965, 1, 128, device="cuda")
    f[..., 32:64] = 1e-3
    f[300:310, :, 96:] = 300.0
    s.v = (s.v.float() * f).to(s.dt)
    s.append()
    s.check(s.attend())


def test_attend_scale_and_strided_query():
    s = _Sequences([321, 40], 6, 2, "bf16", seed=6)
    s.append()
    torch.manual_seed(6)
    wide = torch.randn(2, 3, 6, 128, device="cuda").to(torch.bfloat16)
    s.q = wide[:, 1]
    s.check(s.attend(scale=0.3), scale=0.3)
    s.q = wide[:, 2].expand(2, 6, 128)[:1].expand(2, 6, 128)  # one row for both sequences
    s.check(s.attend(scale=-0.05), scale=-0.05)


def test_attend_skips_and_reports_bad_lengths_and_pages():
    s = _Sequences([100, 300, 50, 10], 4, 2, seed=7)
    s.append()
    good = s.attend()
    s.seq_len = _cuda(np.array([100, -1, 50, 64 * s.max_pages + 1], np.int32))
    y = torch.full_like(good, 9.0)
    stq.stq_attn_decode(s.cache, s.page_table, s.seq_len, s.q, y)
    assert stq.stq_cache_check(s.cache, raise_on_error=False) == stq.STQ_ERR_INDEX
    assert torch.all(y[1] == 9) and torch.all(y[3] == 9)
    assert torch.equal(y[0], good[0]) and torch.equal(y[2], good[2])
    # a page outside the cache: its tokens are not seen
    s = _Sequences([128, 64], 4, 2, seed=8)
    s.append()
    s.page_table[0, 0] = s.cache.num_pages
    s.page_table[1, 0] = -1
    y = torch.full((2, 4, 128), 9.0, dtype=s.dt, device="cuda")
    stq.stq_attn_decode(s.cache, s.page_table, s.seq_len, s.q, y)
    assert stq.stq_cache_check(s.cache, raise_on_error=False) == stq.STQ_ERR_INDEX
    assert torch.all(y[1] == 0)
    s.page_table[0, 0] = s.page_table[0, 1]
    s.seq_len = _cuda(np.array([64, 0], np.int32))
    assert torch.equal(y[0], s.attend()[0])


def test_attend_does_not_see_what_lies_behind_the_last_token():
    """Pages that end inside: stale tokens of other sizes behind a sequence's end change nothing."""
    s = _Sequences([70, 1, 127], 8, 2, "fp16", seed=9)
    s.append()
    y = s.attend()
    stale = np.concatenate([s.table[i, -(-m // 64) - 1].astype(np.int64) * 64 + np.arange(m % 64, 64) for i, m in enumerate(s.lens)])
    big = torch.randn(len(stale), 2, 128, device="cuda") * 1e4
    stq.stq_cache_append(s.cache, _cuda(stale), big, big)
    s.check(s.attend())
    del y


def test_append_and_attend_in_a_graph_on_another_stream():
    """Captured once and replayed with other lengths and tokens; a second graph with its own workspace."""
    s = _Sequences([90, 64, 200], 8, 2, seed=10)
    s.append()
    s.attend()
    work = [torch.empty(stq.stq_attn_decode_workspace(s.cache, 3, 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    y = [torch.zeros(3, 8, 128, dtype=s.dt, device="cuda") for _ in range(2)]
    stream, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for j in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            stq.stq_cache_append(s.cache, s.slot, s.k, s.v)
            stq.stq_attn_decode(s.cache, s.page_table, s.seq_len, s.q, y[j], workspace=work[j])
        graphs.append(g)
    rng = np.random.default_rng(11)
    s.k.copy_(_cuda(rng.standard_normal(s.k.shape)).to(s.dt))
    s.q.copy_(_cuda(rng.standard_normal(s.q.shape)).to(s.dt))
    torch.cuda.synchronize()
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    s.check(y[0])
    assert torch.equal(y[0], y[1])
    # a stream handed over as an argument, with the workspace made for it
    with torch.cuda.stream(stream):
        z = torch.zeros_like(y[0])
    stq.stq_attn_decode(s.cache, s.page_table, s.seq_len, s.q, z, stream=stream)
    stream.synchronize()
    assert torch.equal(z, y[0])


def test_no_sequences_and_no_tokens():
    cache = stq.stq_cache_create(1, 2)
    e = torch.empty(0, 2, 128, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    before = stq.stq_launch_count()
    stq.stq_cache_append(cache, none, e, e)
    stq.stq_cache_read(cache, none, e, e.clone())
    stq.stq_attn_decode(cache, torch.empty(0, 3, dtype=torch.int32, device="cuda"), none.int(), torch.empty(0, 4, 128, device="cuda"),
                        torch.empty(0, 4, 128, device="cuda"))
    assert stq.stq_launch_count() == before
    # a table without columns: every length is zero
    y = torch.full((2, 4, 128), 3.0, device="cuda")
    stq.stq_attn_decode(cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                        torch.randn(2, 4, 128, device="cuda"), y)
    stq.stq_cache_check(cache)
    assert torch.all(y == 0)


def test_refusals():
    cache = stq.stq_cache_create(2, 2)
    k = torch.zeros(4, 2, 128, device="cuda")
    slot = torch.zeros(4, dtype=torch.int64, device="cuda")
    table, lens = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    before = stq.stq_launch_count()
    with pytest.raises(TypeError):
        stq.stq_cache_append(cache, slot, k, k.half())
    with pytest.raises(TypeError):
        stq.stq_cache_append(cache, slot.int(), k, k)
    with pytest.raises(ValueError):
        stq.stq_cache_append(cache, slot, k, k[:, :1])
    with pytest.raises(ValueError):
        stq.stq_cache_append(cache, slot, k.mT.contiguous().mT, k)
    with pytest.raises(ValueError):
        stq.stq_cache_append(cache, slot, k.cpu(), k)
    with pytest.raises(TypeError):
        stq.stq_cache_append(cache, slot, k.double(), k.double())
    q = torch.zeros(4, 4, 128, device="cuda")
    for bad in (torch.zeros(4, 3, 128, device="cuda"),                         # heads no multiple of the cache's
                torch.zeros(4 * 4 * 130, device="cuda").view(4, 4, 130)[..., 1:129],  # rows off 16 bytes
                torch.zeros(4 * 4 * 130, device="cuda").view(4, 4, 130)[..., :128]):
        with pytest.raises(stq.StqError) as e:
            stq.stq_attn_decode(cache, table, lens, bad, torch.zeros_like(bad, memory_format=torch.contiguous_format))
        assert e.value.status == stq.STQ_ERR_ARG
    with pytest.raises(stq.StqError) as e:
        stq.stq_attn_decode(cache, table, lens, q, q.clone(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == stq.STQ_ERR_ARG
    with pytest.raises(stq.StqError) as e:
        stq.stq_attn_decode(cache, table, lens, q, q.clone(), scale=float("nan"))
    assert e.value.status == stq.STQ_ERR_ARG
    with pytest.raises(stq.StqError) as e:
        stq.stq_cache_create(1, 1, head_dim=64)
    assert e.value.status == stq.STQ_ERR_UNSUPPORTED
    assert stq.stq_launch_count() == before
