"""GPU: attention of single tokens over the 4-bit cache at its edges."""
import ctypes as C

import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq
from test_gpu_cache import _Sequences, _cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LENS = [70, 1, 127, 9, 1000]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads, kv_heads", [(8, 2), (16, 1)])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-30, -1e-45])
def test_scales_that_leave_no_score_give_the_mean(kind, heads, kv_heads, scale):
    """Every length but the last ends inside a page: what lies behind has no weight, however small the scores are."""
    s = _Sequences(LENS, heads, kv_heads, kind, seed=31)
    s.append()
    y = s.attend(scale=scale)
    assert bool(y.isfinite().all())
    s.check(y, scale=scale)


@pytest.mark.parametrize("scale", [None, 1e-12])
@pytest.mark.parametrize("lens", [LENS, [9]])
def test_queries_of_zeros_and_near_them(lens, scale):
    s = _Sequences(lens, 8, 2, "fp32", seed=32)
    s.append()
    s.q[0] = 0.0
    s.q[-1, 0] = 1e-37
    y = s.attend(scale=scale)
    assert bool(y.isfinite().all())
    s.check(y, 128 ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("lens", [[70, 1, 127], [17, 33], [5], [64 * 40 + 2] * 3])
@pytest.mark.parametrize("size", [0.02, 1.0])
def test_recycled_pages_give_the_bits_of_new_ones(lens, size):
    """Tokens behind a sequence's end, left by another sequence with values near the top of binary16."""
    s = _Sequences(lens, 8, 2, "bf16", seed=33, size=size)
    s.append()
    y = s.attend()
    assert bool(y.isfinite().all())
    s.check(y)
    stale = np.concatenate([s.table[i, -(-m // 64) - 1].astype(np.int64) * 64 + np.arange(m % 64, 64) for i, m in enumerate(s.lens)])
    big = torch.randn(len(stale), 2, 128, device="cuda") * 1e5
    stq.stq_cache_append(s.cache, _cuda(stale), big, big)
    stq.stq_cache_check(s.cache, raise_on_error=False)  # (groups above binary16's range are reported, and zero)
    assert torch.equal(s.attend(), y)


@pytest.mark.parametrize("pages", [2 ** 25, 2 ** 31 - 1, -1])
def test_tables_too_wide_for_a_length_are_refused(pages):
    """Lengths up to 64 max_pages are counted in 31 bits."""
    cache = stq.stq_cache_create(1, 2)
    q, y = (torch.zeros(1, 4, 128, device="cuda") for _ in range(2))
    small, work = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.empty(stq.stq_attn_decode_workspace(cache, 1, 4), dtype=torch.uint8, device="cuda")
    before = stq.stq_launch_count()
    rows = stq._Rows(q.data_ptr(), 0, 128)
    st = stq.load().stq_attn_decode(cache.handle, small.data_ptr(), pages, small.data_ptr(), 1, 4, stq.STQ_F32, C.byref(rows), 0.1,
                                    y.data_ptr(), work.data_ptr(), work.numel(), 0)
    assert st == stq.STQ_ERR_ARG and "max_pages" in stq.stq_last_error()
    assert stq.stq_launch_count() == before
