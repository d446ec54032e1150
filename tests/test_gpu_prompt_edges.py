"""GPU: stq_prompt_step at its edges."""
import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq
from test_gpu_prompt import _Prompts, _cuda, _f64, recurrence

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp16", "fp32"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_nan_in_q_is_in_its_row_of_y(kind):
    s = _Prompts([200, 70], 3, kind, seed=51)
    want_y, want = (t.clone() for t in s.run())
    s.q[70, 1, 5] = float("nan")
    y, state = s.run()
    assert bool(y[70, 1].isnan().all())
    assert torch.equal(state, want)
    y[70, 1] = want_y[70, 1]
    assert torch.equal(y, want_y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [0, 70, 199])
def test_a_nan_in_v_is_in_its_column_from_there_on(kind, t):
    s = _Prompts([200, 70], 3, kind, seed=52)
    want_y, want = (x.clone() for x in s.run())
    s.v[t, 1, 5] = float("nan")
    y, state = s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_NONFINITE
    assert bool(y[t:200, 1, 5].isnan().all()) and bool(state[0, 1, :, 5].isnan().all())
    # other columns, heads and prompts, and chunks of 64 that ended before
    rest = torch.ones(270, 3, 128, dtype=torch.bool, device="cuda")
    rest[t - t % 64:200, 1, 5] = False
    assert torch.equal(y[rest], want_y[rest])
    rest = torch.ones_like(state, dtype=torch.bool)
    rest[0, 1, :, 5] = False
    assert torch.equal(state[rest], want[rest])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", ["k", "beta", "alpha"])
def test_a_nan_in_k_and_the_gates_is_in_y_from_there_on(kind, name):
    s = _Prompts([200, 70], 3, kind, seed=53)
    want_y, want = (x.clone() for x in s.run())
    x = getattr(s, name)
    if name == "k":
        x[70, 1, 5] = float("nan")
    else:
        x[70, 1] = float("nan")
    y, state = s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_NONFINITE
    assert bool(y[70:200, 1].isnan().all()) and bool(state[0, 1].isnan().all())
    assert torch.equal(y[:64], want_y[:64]) and torch.equal(y[200:], want_y[200:]) and torch.equal(state[1], want[1])
    for h in (0, 2):
        assert torch.equal(y[:, h], want_y[:, h]) and torch.equal(state[:, h], want[:, h])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_state_that_is_no_number_is_in_its_column(kind, bad):
    """A page of an fp32 pool that an earlier call spoilt."""
    s = _Prompts([200], 2, kind, seed=54, bits=32, fresh=[0])
    S = _cuda(s.S0.astype(np.float32))
    S[0, 1, 7, 5] = bad
    stq.stq_quantize_state(s.pool, s.req, s.slot, S)
    stq.stq_pool_check(s.pool, raise_on_error=False)
    y, state = s.run()
    assert not bool(y[:, 1, 5].isfinite().any())
    keep = torch.arange(128, device="cuda") != 5
    assert bool(y[:, 0].isfinite().all()) and bool(y[:, 1, keep].isfinite().all())


@pytest.mark.parametrize("kind", KINDS)
def test_ranges_in_any_order(kind):
    """A range that runs backwards is empty, so that the ones around it may lie in any order."""
    s = _Prompts([64, 0, 128], 3, kind, seed=55)
    s.starts = np.array([128, 192, 0, 128], np.int32)
    s.seq_start = _cuda(s.starts)
    s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_INDEX
    s.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_many_ranges_in_any_order(kind):
    """Every second range runs backwards, over more entries than the walk ranks: the blocks of rows come last to first."""
    m, n = 70, 150
    s = _Prompts([m if e % 2 == 0 else 0 for e in range(2 * n - 1)], 1, kind, seed=58, bits=32, fresh=[e % 3 == 0 for e in range(2 * n - 1)])
    s.starts = np.array([(n - 1 - e // 2 + e % 2) * m for e in range(2 * n)], np.int32)
    s.seq_start = _cuda(s.starts)
    s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_INDEX
    s.check()


def test_fp32_rows_need_no_workspace():
    s = _Prompts([2000, 96], 8, "fp32", seed=57, state=False)
    y, state = (t.clone() for t in s.run())
    torch.cuda.synchronize()
    y2, state2 = torch.zeros_like(y), torch.zeros_like(state)
    args = (s.pool, s.req, s.slot, s.seq_start, s.q, s.k, s.v, s.beta, s.alpha, y2, state2)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    stq.stq_prompt_step(*args, fresh=s.fresh)
    assert torch.cuda.max_memory_allocated() - before < 1 << 16
    assert torch.equal(y2, y) and torch.equal(state2, state)
    stq.stq_prompt_step(*args, fresh=s.fresh, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert torch.equal(y2, y) and torch.equal(state2, state)


@pytest.mark.parametrize("flags", [stq.STQ_SCALE_F16, stq.STQ_FIT_COLUMNS, stq.STQ_FIT_COLUMNS | stq.STQ_SCALE_F16])
@pytest.mark.parametrize("kind, lens", [("bf16", [5, 0, 70, 130, 0]), ("fp32", [5, 0, 70, 1, 0]), ("fp16", [3, 0, 1, 9, 0])])
def test_pools_of_other_formats(flags, kind, lens):
    """binary16 scales and fitted columns, 16-bit pivot heads among them: pages are read before and quantized after as the
    calls of their own do it, byte for byte."""
    class P(_Prompts):
        def new_pool(self, slots=2):
            return stq.stq_pool_create(stq.STQ_GDN, self.n, slots, self.H, self.bits, flags=flags)

    s = P(lens, 4, kind, seed=56, bits=np.array([6, 16, 4, 8], np.uint8), fresh=[0, 1, 0, 1, 0])
    before = s.pages(s.pool, 4)
    y, state = s.run()
    stq.stq_pool_check(s.pool)
    s.check()
    twin = s.new_pool()
    state[4] = 0
    stq.stq_quantize_state(twin, s.req, s.slot, state)
    for e in range(4):
        assert np.array_equal(s.pages(s.pool, e), s.pages(twin, e)), e
    assert np.array_equal(s.pages(s.pool, 4), before)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("lens, launches", [([1] * 100, 3), ([2] * 70 + [0] * 9, 3), ([1] * 100 + [300], 4), ([64], 4), ([63], 3)])
def test_entries_of_few_tokens_each(kind, lens, launches):
    """A step of single tokens takes no chunks however many entries it has (unpack, advance, quantize: three launches; a
    fourth prepares chunks), and with a prompt beside them all are as right."""
    s = _Prompts(lens, 2, kind, seed=59, fresh=[e % 2 for e in range(len(lens))])
    before = stq.stq_launch_count()
    s.run()
    assert stq.stq_launch_count() - before == launches
    stq.stq_pool_check(s.pool)
    s.check()


@pytest.mark.parametrize("lens", [[64, 64, 33, 1, 50], [64] * 12])
@pytest.mark.parametrize("heads", [2, 16])
def test_fp16_rows_are_rounded_once(heads, lens):
    """Prompts of one chunk from the zero state: y = P U, P and U two terms each (2^-20 of every product is left, and the
    recurrence's 1e-5), is off by half a step of itself; one term each would add two more roundings of that size."""
    s = _Prompts(lens, heads, "fp16", seed=60, state=False)
    s.run()
    y = _f64(s.y)
    for e, m in enumerate(s.lens):
        a, b = s.starts[e], s.starts[e + 1]
        want, _, size = recurrence(*(_f64(t[a:b]) for t in (s.q, s.k, s.v, s.beta, s.alpha)), s.S0[e])
        tol = 1e-5 * np.abs(want).max((0, 2), keepdims=True) + 1.001 * 2.0 ** -11 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -25
        bad = ~(np.abs(y[a:b] - want) <= tol)
        assert not bad.any(), (e, m, np.abs(y[a:b] - want)[bad][:4], tol[bad][:4])
