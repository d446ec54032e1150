"""GPU: stq_prompt_step, the gated delta rule over whole prompts, against the
recurrence in fp64 on the CPU."""
import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def recurrence(q, k, v, beta, alpha, X):
    """One prompt: q, k, v [T, H, 128], beta, alpha [T, H], X [H, 128, 128] -> (y, X_T, size), all fp64.  In chunks of 64
    tokens y_t = R_t X_0^T q_t + sum_i R_ti (q_t . k_i) u_i with the products R of the decays; size[t] is the sum of the
    sizes of these terms, which may cancel (one key for all tokens)."""
    X = X.copy()
    y, size = np.zeros_like(q), np.zeros_like(q)
    for t in range(len(q)):
        if t % 64 == 0:
            start, r0, r, us = np.abs(X), np.ones(q.shape[1]), np.zeros((0, q.shape[1])), np.zeros((0, *q.shape[1:]))
        X = alpha[t][:, None, None] * X
        u = beta[t][:, None] * (v[t] - np.einsum("hi,hij->hj", k[t], X))
        X = X + k[t][:, :, None] * u[:, None, :]
        y[t] = np.einsum("hi,hij->hj", q[t], X)
        r0, r = r0 * np.abs(alpha[t]), np.concatenate([r * np.abs(alpha[t]), np.ones((1, q.shape[1]))])
        us = np.concatenate([us, np.abs(u)[None]])
        p = r * np.abs(np.einsum("hi,thi->th", q[t], k[t - t % 64:t + 1]))
        size[t] = r0[:, None] * np.einsum("hi,hij->hj", np.abs(q[t]), start) + np.einsum("th,thj->hj", p, us)
    return y, X, size


class _Prompts:
    def __init__(self, lens, heads, kind, seed=0, alpha=(0.9, 0.999), bits=6, fresh=None, state=True, pad=0, slots=2):
        rng = np.random.default_rng(seed)
        self.lens, self.n, self.H, self.dt = list(lens), len(lens), heads, TYPES[kind]
        self.total = sum(lens) + pad
        shape = (self.total, heads, 128)
        q, k, v = (rng.standard_normal(shape) for _ in range(3))
        q /= np.linalg.norm(q, axis=-1, keepdims=True)
        k /= np.linalg.norm(k, axis=-1, keepdims=True)
        self.q, self.k, self.v = (_cuda(a).to(self.dt) for a in (q, k, v))
        self.beta = _cuda(rng.uniform(0, 1, shape[:2]).astype(np.float32))
        self.alpha = _cuda(rng.uniform(*alpha, shape[:2]).astype(np.float32))
        self.starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.seq_start = _cuda(self.starts)
        self.bits = np.full(heads, bits, np.uint8) if np.isscalar(bits) else bits
        self.pool = self.new_pool(slots)
        self.req = _cuda(rng.permutation(self.n).astype(np.int32))
        self.slot = _cuda(rng.integers(0, slots, self.n).astype(np.int32))
        self.fresh_np = np.ones(self.n, np.int32) if fresh is None else np.asarray(fresh, np.int32)
        self.fresh = None if fresh is not None and not np.any(fresh) else _cuda(self.fresh_np)
        self.S0 = np.zeros((self.n, heads, 128, 128))
        if state:
            S = _cuda(rng.standard_normal((self.n, heads, 128, 128)).astype(np.float32))
            stq.stq_quantize_state(self.pool, self.req, self.slot, S)
            out = torch.empty_like(S)
            stq.stq_dequantize_state(self.pool, self.req, self.slot, out)
            self.S0 = np.where(self.fresh_np[:, None, None, None] != 0, 0.0, _f64(out))

    def new_pool(self, slots=2):
        return stq.stq_pool_create(stq.STQ_GDN, self.n, slots, self.H, self.bits)

    def run(self, pool=None, **more):
        self.y = torch.full((self.total, self.H, 128), 77.0, dtype=self.dt, device="cuda")
        self.state = torch.full((self.n, self.H, 128, 128), float("nan"), device="cuda")
        stq.stq_prompt_step(pool or self.pool, self.req, self.slot, self.seq_start, self.q, self.k, self.v, self.beta, self.alpha,
                            self.y, self.state, fresh=self.fresh, **more)
        return self.y, self.state

    def check(self):
        """fp32: 1e-5 of the head's largest value, the tolerance of the decode step.  A 16-bit y is rounded once (half a
        step of itself) and the two factors of every product of its chunk's form to 11 bits: 2 times 2^-11 of every term."""
        half = torch.finfo(self.dt).eps / 2
        y, state = _f64(self.y), _f64(self.state)
        for e, m in enumerate(self.lens):
            a, b = self.starts[e], self.starts[e + 1]
            ins = [_f64(t[a:b]) for t in (self.q, self.k, self.v, self.beta, self.alpha)]
            want, X, size = recurrence(*ins, self.S0[e])
            if m > 0 or self.fresh_np[e]:
                top = np.abs(X).max((1, 2), keepdims=True)
                err = np.abs(state[e] - X) / np.where(top > 0, top, 1)
                assert err.max() <= 1e-5, (e, m, err.max())
            if m > 0:
                tol = 1e-5 * np.abs(want).max((0, 2), keepdims=True)
                if self.dt != torch.float32:
                    tol = tol + 1.01 * half * np.abs(want) + 2.0 ** -10 * size + 2.0 ** -25
                bad = np.abs(y[a:b] - want) > tol
                assert not bad.any(), (e, m, np.abs(y[a:b] - want)[bad][:4], want[bad][:4])

    def pages(self, pool, e):
        return stq.stq_export_slot(pool, int(self.req[e]), int(self.slot[e]))


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 400]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads", [3, 12, 24])
def test_prompts(kind, heads):
    """Few and many heads; lengths around chunks; half of the entries start from their pages."""
    s = _Prompts(LENS, heads, kind, seed=heads, fresh=[i % 2 for i in range(len(LENS))])
    s.run()
    stq.stq_pool_check(s.pool)
    s.check()


@pytest.mark.parametrize("bits", [4, 8, 16, 32, "mixed"])
def test_pages_are_the_quantized_states(bits):
    """What the pool holds afterwards is stq_quantize_state of the returned states, byte for byte; an empty prompt
    leaves its page alone, or zero when fresh."""
    lens = [5, 0, 70, 0]
    ub = np.array([6, 16, 4], np.uint8) if bits == "mixed" else np.full(3, bits, np.uint8)
    s = _Prompts(lens, 3, "bf16", seed=1, bits=ub, fresh=[1, 1, 0, 0])
    before = s.pages(s.pool, 3)
    y, state = s.run()
    stq.stq_pool_check(s.pool)
    s.check()
    twin = s.new_pool()
    state[3] = 0
    stq.stq_quantize_state(twin, s.req, s.slot, state)
    for e in range(3):
        assert np.array_equal(s.pages(s.pool, e), s.pages(twin, e)), e
    assert np.array_equal(s.pages(s.pool, 3), before)
    assert not state[1].any()


@pytest.mark.parametrize("heads, kind", [(2, "fp32"), (2, "bf16"), (40, "fp32"), (40, "fp16")])
def test_pieces_and_decode_steps_continue_a_prompt(heads, kind):
    """A pool of fp32 states: a prompt in two pieces, and a prompt with its last tokens decoded one by one, end where
    the whole prompt does."""
    lens = [100, 37, 150, 64, 90, 71, 33]
    whole = _Prompts(lens, heads, kind, seed=2, bits=32, state=False)
    y, state = (t.clone() for t in whole.run())
    whole.check()
    cut = [60, 36, 64, 1, 77, 8, 32]
    part = _Prompts(lens, heads, kind, seed=2, bits=32, state=False)
    ya = torch.zeros_like(y)
    where = [np.concatenate([np.arange(a, a + c) for a, c in zip(part.starts, cut)]),
             np.concatenate([np.arange(a + c, b) for a, c, b in zip(part.starts, cut, part.starts[1:])])]
    full = {n: getattr(part, n) for n in ("q", "k", "v", "beta", "alpha")}
    for step, rows in enumerate(where):
        idx = _cuda(rows.astype(np.int64))
        for name, t in full.items():
            setattr(part, name, t[idx])
        sizes = cut if step == 0 else [m - c for m, c in zip(lens, cut)]
        part.total, part.seq_start = len(rows), _cuda(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))
        part.fresh = _cuda(np.full(part.n, 1 - step, np.int32))
        yp, sp = part.run()
        ya[idx] = yp
    scale = state.abs().amax((2, 3), keepdim=True)
    assert float(((sp - state).abs() / scale).max()) <= 2e-5
    half = torch.finfo(whole.dt).eps / 2
    tol = 2e-5 * float(y.float().abs().max()) + (0 if kind == "fp32" else 2.1 * half * y.float().abs() + 2.0 ** -10 * 4)
    assert bool(((ya.float() - y.float()).abs() <= tol).all())
    # the last three tokens of every prompt by decode steps
    short = _Prompts(lens, heads, kind, seed=2, bits=32, state=False)
    rows = np.concatenate([np.arange(a, b - 3) for a, b in zip(short.starts, short.starts[1:])])
    idx = _cuda(rows.astype(np.int64))
    for name, t in full.items():
        setattr(short, name, t[idx])
    short.total, short.seq_start = len(rows), _cuda(np.concatenate([[0], np.cumsum([m - 3 for m in lens])]).astype(np.int32))
    short.run()
    for j in (3, 2, 1):
        at = _cuda((whole.starts[1:] - j).astype(np.int64))
        args = [full[n][at].float().contiguous() for n in ("q", "k", "v", "beta", "alpha")]
        yd = torch.empty(short.n, heads, 128, device="cuda")
        stq.stq_decode_step(short.pool, short.req, short.slot, *args, yd)
        want = y[at].float()
        tol = 2e-5 * float(want.abs().max()) + (0 if kind == "fp32" else 1.1 * half * want.abs() + 2.0 ** -10 * 4)
        assert bool(((yd - want).abs() <= tol).all()), j
    stq.stq_pool_check(short.pool)
    last = torch.empty_like(state)
    stq.stq_dequantize_state(short.pool, short.req, short.slot, last)
    assert float(((last - state).abs() / scale).max()) <= 2e-5


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [2, 64])
def test_decays_and_gates_at_their_ends(kind, heads):
    """Decays of 0, 1e-30, 1 and below 0, gates of 0, 1 and 2, and one key for all tokens."""
    lens = [200, 130, 64, 190]
    s = _Prompts(lens, heads, kind, seed=3, fresh=[0, 1, 0, 1])
    a, b = s.alpha, s.beta
    a[5] = 0.0
    a[70:75] = 1e-30
    a[100:164] = 1.0
    b[120:130] = 0.0
    b[130:140] = 2.0
    a[160:170] = -0.7
    s.k[200:330] = s.k[200]
    b[200:330] = 1.0
    a[330:394] = 0.05
    s.run()
    stq.stq_pool_check(s.pool)
    s.check()


def test_full_gate_stores_the_value():
    """b = 1 and a unit key: X_T^T k_T = v_T."""
    s = _Prompts([33, 64, 129], 4, "fp32", seed=4)
    s.beta[:] = 1.0
    _, state = s.run()
    for e in range(3):
        t = s.starts[e + 1] - 1
        got = torch.einsum("hij,hi->hj", state[e].double(), s.k[t].double())
        assert float((got - s.v[t].double()).abs().max()) <= 1e-5 * float(s.v[t].abs().max())


@pytest.mark.parametrize("heads", [3, 30])
def test_strided_rows_and_rows_of_no_prompt(heads):
    """q, k, v as parts of one projection; rows behind the last prompt and between prompts hold NaN and are left alone."""
    lens = [70, 9, 64, 1, 20, 30, 41, 50, 3]
    s = _Prompts(lens, heads, "bf16", seed=5, pad=40)
    s.run()
    want_y, want = s.y.clone(), s.state.clone()
    fused = torch.full((s.total, 3, heads, 128), float("nan"), dtype=s.dt, device="cuda")
    m = sum(lens)
    for i, t in enumerate((s.q, s.k, s.v)):
        fused[:m, i] = t[:m]
    s.q, s.k, s.v = fused.unbind(1)
    s.beta[m:] = float("nan")
    s.alpha[m:] = float("nan")
    y, state = s.run()
    stq.stq_pool_check(s.pool)
    assert torch.equal(y[:m], want_y[:m]) and torch.equal(state, want)
    assert bool((y[m:] == 77).all())
    # one head's rows for all heads (a stride of zero)
    s.q = fused[:, 0, :1].expand(-1, heads, -1)
    s.run()
    s.check()


def test_bad_ranges_and_entries_are_skipped_and_reported():
    s = _Prompts([20, 30, 40, 10, 5], 3, "bf16", seed=6, fresh=[0] * 5, pad=3)
    s.run()
    good_y, good = s.y.clone(), s.state.clone()
    # twin with one range running backwards, one behind the end, one request out of range
    t = _Prompts([20, 30, 40, 10, 5], 3, "bf16", seed=6, fresh=[0] * 5, pad=3)
    t.seq_start = _cuda(np.array([0, 20, 50, 45, 45 + 10, 10 ** 6], np.int32))
    before = [t.pages(t.pool, e) for e in range(5)]
    t.run()
    assert stq.stq_pool_check(t.pool, raise_on_error=False) == stq.STQ_ERR_INDEX
    assert torch.equal(t.state[:2], good[:2]) and torch.equal(t.y[:45], good_y[:45])
    assert np.array_equal(t.pages(t.pool, 2), before[2]) and np.array_equal(t.pages(t.pool, 4), before[4])
    assert bool((t.y[55:] == 77).all())
    u = _Prompts([20, 30, 40, 10, 5], 3, "bf16", seed=6, fresh=[0] * 5, pad=3)
    r = int(u.req[1])
    u.req[1] = 99
    u.run()
    assert stq.stq_pool_check(u.pool, raise_on_error=False) == stq.STQ_ERR_INDEX
    assert bool((u.y[20:50] == 77).all())
    assert torch.equal(u.y[:20], good_y[:20]) and torch.equal(u.y[50:105], good_y[50:105])
    u.req[1] = r
    assert np.array_equal(u.pages(u.pool, 1), before[1])


def test_non_finite_input_is_reported_and_stays_in_its_head():
    s = _Prompts([70, 40], 3, "bf16", seed=7)
    s.run()
    want_y, want = s.y.clone(), s.state.clone()
    s.v[30, 1, 5] = float("nan")
    y, state = s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_NONFINITE
    for h in (0, 2):
        assert torch.equal(y[:, h], want_y[:, h]) and torch.equal(state[:, h], want[:, h])
    assert torch.equal(y[70:], want_y[70:]) and torch.equal(state[1], want[1])


@pytest.mark.parametrize("heads", [2, 20])
def test_graph_and_streams(heads):
    """Captured once, replayed on new tokens and lengths; then on a stream handed over as an argument."""
    lens = [70, 65, 10, 128]
    s = _Prompts(lens, heads, "bf16", seed=8, fresh=[1, 0, 1, 0], bits=32)
    s.run()
    y, state = torch.zeros_like(s.y), torch.zeros_like(s.state)
    work = torch.empty(stq.stq_prompt_workspace(s.pool, s.n, s.total), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=stream):
        stq.stq_prompt_step(s.pool, s.req, s.slot, s.seq_start, s.q, s.k, s.v, s.beta, s.alpha, y, state, fresh=s.fresh, workspace=work)
    other = _Prompts([60, 100, 1, 112], heads, "bf16", seed=9, fresh=[1, 0, 1, 0], bits=32)
    for name in ("q", "k", "v", "beta", "alpha", "seq_start"):
        getattr(s, name).copy_(getattr(other, name))
    S = _cuda(other.S0.astype(np.float32))
    stq.stq_quantize_state(s.pool, s.req, s.slot, S)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    stq.stq_pool_check(s.pool)
    other.y, other.state = y, state
    other.check()
    stq.stq_quantize_state(s.pool, s.req, s.slot, S)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        y2, state2 = torch.zeros_like(y), torch.zeros_like(state)
    stq.stq_prompt_step(s.pool, s.req, s.slot, s.seq_start, s.q, s.k, s.v, s.beta, s.alpha, y2, state2, fresh=s.fresh, stream=stream)
    stream.synchronize()
    assert torch.equal(y, y2) and torch.equal(state, state2)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [2, 70])
@pytest.mark.parametrize("lens", [[1], [3, 0, 20], [39]])
def test_few_tokens_of_16_bits(kind, heads, lens):
    """So few that no chunk is worth while; rows as parts of one projection, and behind them rows of NaN."""
    s = _Prompts(lens, heads, kind, seed=12, fresh=[0] * len(lens))
    m = sum(lens)
    fused = torch.full((m + 1, 3, heads, 128), float("nan"), dtype=s.dt, device="cuda")
    for i, t in enumerate((s.q, s.k, s.v)):
        fused[:m, i] = t
    s.q, s.k, s.v = fused[:m].unbind(1)
    s.run()
    stq.stq_pool_check(s.pool)
    s.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_many_prompts(kind):
    """More entries than the walk ranks by their length, from none to two chunks of tokens."""
    s = _Prompts([(29 * i) % 97 for i in range(200)], 1, kind, seed=15, fresh=[i % 3 == 0 for i in range(200)])
    s.run()
    stq.stq_pool_check(s.pool)
    s.check()


def test_two_calls_at_once():
    """Two pools on two streams, in turn, each with its own workspace: as alone."""
    calls = [_Prompts([300, 64, 7], 20, "bf16", seed=13), _Prompts([90, 250, 128, 1], 16, "fp16", seed=14)]
    want = [tuple(t.clone() for t in s.run()) for s in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    work = [torch.empty(stq.stq_prompt_workspace(s.pool, s.n, s.total), dtype=torch.uint8, device="cuda") for s in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream, w in zip(calls, streams, work):
            with torch.cuda.stream(stream):
                s.run(workspace=w)
    torch.cuda.synchronize()
    for s, (y, state) in zip(calls, want):
        stq.stq_pool_check(s.pool)
        assert torch.equal(s.y, y) and torch.equal(s.state, state)


def test_after_a_split_step_and_with_debug_checks(monkeypatch):
    """A pending write-back is waited for; a (request, slot) named twice is reported when debug checks are on."""
    monkeypatch.setenv("STQ_DEBUG_CHECKS", "1")
    s = _Prompts([12, 9], 4, "fp32", seed=10, fresh=[0, 0])
    twin = _Prompts([12, 9], 4, "fp32", seed=10, fresh=[0, 0])
    side = torch.cuda.Stream()
    args = [torch.randn(2, 4, 128, device="cuda") * 0.1 for _ in range(3)] + [torch.rand(2, 4, device="cuda") for _ in range(2)]
    y, u = torch.empty(2, 4, 128, device="cuda"), torch.empty(2, 4, 128, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    stq.stq_decode_step_split(s.pool, s.req, s.slot, *args, y, u, None, side)
    s.run()
    stq.stq_decode_step(twin.pool, twin.req, twin.slot, *args, y)
    twin.run()
    assert torch.equal(s.y, twin.y) and torch.equal(s.state, twin.state)
    stq.stq_pool_check(s.pool)
    s.req[1], s.slot[1] = s.req[0], s.slot[0]
    s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_INDEX


def test_nothing_to_do_and_refusals():
    s = _Prompts([4, 5], 2, "bf16", seed=11)
    before = stq.stq_launch_count()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(0, 2, device="cuda")
    stq.stq_prompt_step(s.pool, none, none, torch.zeros(1, dtype=torch.int32, device="cuda"), e, e, e, b, b, e.clone(),
                        torch.empty(0, 2, 128, 128, device="cuda"))
    args = [s.pool, s.req, s.slot, s.seq_start, s.q, s.k, s.v, s.beta, s.alpha, s.q.clone(), torch.empty(2, 2, 128, 128, device="cuda")]

    def refused(error, status=None, **change):
        names = ["pool", "req", "slot", "seq_start", "q", "k", "v", "beta", "alpha", "y", "state"]
        with pytest.raises(error) as info:
            stq.stq_prompt_step(*[change.get(n, a) for n, a in zip(names, args)],
                                **{k: w for k, w in change.items() if k not in names})
        if status is not None:
            assert info.value.status == status

    refused(TypeError, k=s.k.half())
    refused(TypeError, q=s.q.double())
    refused(TypeError, y=s.q.float())
    refused(TypeError, alpha=s.alpha.bfloat16())
    refused(ValueError, beta=s.beta[:5])
    refused(ValueError, seq_start=s.seq_start[:2])
    refused(ValueError, v=s.v.mT.contiguous().mT)
    refused(ValueError, state=torch.empty(2, 2, 128, 64, device="cuda"))
    refused(ValueError, k=s.k.cpu())
    odd = torch.zeros(9, 2, 132, dtype=torch.bfloat16, device="cuda")[..., 3:131]
    refused(stq.StqError, stq.STQ_ERR_ARG, k=odd)
    refused(stq.StqError, stq.STQ_ERR_ARG, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    kda = stq.stq_pool_create(stq.STQ_KDA, 2, 2, 2, np.full(256, 6, np.uint8))
    refused(stq.StqError, stq.STQ_ERR_UNSUPPORTED, pool=kda)
    assert stq.stq_launch_count() == before
