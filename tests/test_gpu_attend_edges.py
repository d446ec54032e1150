"""GPU: attention of single tokens over the 4-bit cache at its edges."""
import ctypes as C

import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq
from test_gpu_cache import _Sequences, _cuda, _quantized

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


class _Fp32(_Sequences):
    def check_fp32(self, y, scale=128 ** -0.5):
        """fp32 rows: q, the weights and their products with the scales are two binary16 terms each (2^-22 of them is left);
        a score's sum of 128 products is off by less than 2^-19 of their sizes, a weight by twice a score's error; exp2, the
        sums and the join by 2^-18 together; terms that are subnormal by half of 2^-24, as _Sequences.check has it."""
        got = y.cpu().numpy().astype(np.float64)
        k, v = (_quantized(x.cpu().numpy()).astype(np.float64) for x in (self.k, self.v))
        q = self.q.cpu().numpy().astype(np.float64)
        g, at = self.heads // self.kv_heads, 0
        for i, m in enumerate(self.lens):
            for h in range(self.heads):
                kk, vv = k[at:at + m, h // g], v[at:at + m, h // g]
                x = kk @ q[i, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                ref = p @ vv
                delta = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale) * (2.0 ** -19 + 2.0 ** -21)
                s_max = np.abs(vv).max() / 7 * 1.01
                small = 2.0 ** -36 * p.max() * max(1.0, 2 * s_max) * (1 + s_max) * 7 * m
                tol = small + (2.0 ** -18 + 2 * delta + 2.0 ** -20) * (p @ np.abs(vv)) + 2.0 ** -24 * np.abs(ref)
                bad = ~(np.abs(got[i, h] - ref) <= tol)
                assert not bad.any(), (i, h, m, np.abs(got[i, h] - ref)[bad][:4], tol[bad][:4])
            at += m


@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 2), (9, 1), (32, 2), (40, 2)])
@pytest.mark.parametrize("spread", [0.3, 1.0, 3.0])
def test_fp32_rows_keep_fp32(heads, kv_heads, spread):
    s = _Fp32([1, 63, 64, 65, 200, 1000], heads, kv_heads, "fp32", seed=34, spread=spread)
    s.append()
    y = s.attend()
    s.check_fp32(y)
    assert torch.equal(y, s.attend())


@pytest.mark.parametrize("lens", [[30000], [70] * 150])
def test_fp32_rows_over_many_shares(lens):
    s = _Fp32(lens, 8, 2, "fp32", seed=35)
    s.append()
    s.check_fp32(s.attend())


class _Fp16(_Sequences):
    def check_fp16(self, y):
        """As fp32 rows, but for y, which is rounded once (half a step, and half of the smallest)."""
        got = y.float().cpu().numpy().astype(np.float64)
        k, v = (_quantized(x.float().cpu().numpy()).astype(np.float64) for x in (self.k, self.v))
        q = self.q.float().cpu().numpy().astype(np.float64)
        g, at = self.heads // self.kv_heads, 0
        for i, m in enumerate(self.lens):
            for h in range(self.heads):
                kk, vv = k[at:at + m, h // g], v[at:at + m, h // g]
                x = kk @ q[i, h] * 128 ** -0.5
                p = np.exp(x - x.max())
                p /= p.sum()
                ref = p @ vv
                delta = (np.abs(kk) @ np.abs(q[i, h])).max() * 128 ** -0.5 * 2.0 ** -19
                s_max = np.abs(vv).max() / 7 * 1.01
                small = 2.0 ** -36 * p.max() * max(1.0, 2 * s_max) * (1 + s_max) * 7 * m
                tol = small + (2.0 ** -18 + 2 * delta + 2.0 ** -20) * (p @ np.abs(vv)) + 1.001 * 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
                bad = ~(np.abs(got[i, h] - ref) <= tol)
                assert not bad.any(), (i, h, m, np.abs(got[i, h] - ref)[bad][:4], tol[bad][:4])
            at += m


@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 2), (9, 1), (32, 2), (40, 2)])
@pytest.mark.parametrize("lens", [[1, 63, 64, 65, 200, 1000], [9], [20000]])
def test_fp16_rows_are_rounded_once(heads, kv_heads, lens):
    """No error beside the output's own rounding, which one binary16 value for a weight would double."""
    s = _Fp16(lens, heads, kv_heads, "fp16", seed=36)
    s.append()
    y = s.attend()
    s.check_fp16(y)
    assert torch.equal(y, s.attend())


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
