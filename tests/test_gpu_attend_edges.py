"""GPU: attention of single tokens over the 4-bit cache at its edges."""
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
