"""GPU: stq_attn_prompt where one key outweighs a long tail."""
import numpy as np
import pytest

from test_gpu_attn_prompt import _Attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("at", [0, 1500, 2999])
@pytest.mark.parametrize("score", [12.0, 19.0])
def test_a_tail_far_below_one_key_keeps_its_values(kind, at, score):
    """One key `score` above all others and with values of zero: y is what the others give, e^-score of theirs each.
    A weight is held as 2^7 w / w_max at least in fp16, so where it is subnormal there it is off by half of 2^-24:
    2^-32 w_max a key, times |v|."""
    a = _Attn([3], 4, 2, kind, prefix=2999, seed=41)
    n = a.lk[0]
    a.q.zero_()
    a.k.zero_()
    a.q[..., 0] = 8.0
    a.k[at, :, 0] = score * 128 ** 0.5 / 8.0
    a.v.abs_()
    a.v[at] = 0.0
    y = a.run().float().cpu().numpy().astype(np.float64)
    k0 = float(a.k[at, 0, 0])
    v = a.v.float().cpu().numpy().astype(np.float64)
    half = torch.finfo(a.dt).eps / 2
    for j in range(3):
        seen = n - 2 + j
        w = np.full(seen, np.exp(-8.0 * k0 * 128 ** -0.5) if at < seen else 1.0)
        if at < seen:
            w[at] = 1.0
        w /= w.sum()
        for h in range(4):
            vv = v[:seen, h // 2]
            want = w @ vv
            small = 2.0 ** -32 * w.max() * vv.sum(0) if kind == "fp16" else 0.0
            tol = small + (half + 2 * score * 2.0 ** -17 + 2.0 ** -20) * want + 1.01 * half * want + 2.0 ** -24
            assert np.all(np.abs(y[j, h] - want) <= tol), (j, h, np.abs(y[j, h] - want).max(), want.max(), np.min(tol))
