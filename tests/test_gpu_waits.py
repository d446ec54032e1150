"""GPU: the bounded waits of prompts in chunks, prompt attention and cache
attention end in an error status.

STQ_FAULT=timeout makes one wait run out on purpose: the limit drops to 2 ms and
the first stage of the launch expects 16 bytes that no copy delivers (every copy
lands; no fault, trap or hang is involved).  What the stalled CTA did not have to
do is as without it, and the same objects work on."""
import time

import pytest

from quantized_linear_attention_decode_b200 import stq
from test_gpu_attn_prompt import _Attn
from test_gpu_cache import _Sequences
from test_gpu_prompt import _Prompts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _stalled(monkeypatch, call):
    monkeypatch.setenv("STQ_FAULT", "timeout")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    out = call()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    monkeypatch.delenv("STQ_FAULT")
    assert took < 0.5, f"the stalled call took {took:.3f} s"
    return out


@pytest.mark.parametrize("lens", [[64], [100, 330, 64, 7]])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_prompt_step(kind, lens, monkeypatch):
    s = _Prompts(lens, 3, kind, seed=61, bits=32, slots=1)
    y, state = (t.clone() for t in s.run())
    stq.stq_pool_check(s.pool)
    bad_y, bad = _stalled(monkeypatch, s.run)
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_ERR_TIMEOUT
    assert "timed out" in stq.stq_last_error()
    longest = max(range(len(lens)), key=lambda e: lens[e])  # its head 0 is the first CTA's
    a, b = s.starts[longest], s.starts[longest + 1]
    bad_y[a:b, 0], bad[longest, 0] = y[a:b, 0], state[longest, 0]
    assert torch.equal(bad_y, y) and torch.equal(bad, state)
    again_y, again = s.run()
    assert stq.stq_pool_check(s.pool, raise_on_error=False) == stq.STQ_OK
    assert torch.equal(again_y, y) and torch.equal(again, state)


@pytest.mark.parametrize("lens, prefix", [([40], 0), ([300, 200], 0), ([20, 64], 900)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_attn_prompt(kind, lens, prefix, monkeypatch):
    a = _Attn(lens, 4, 2, kind, prefix=prefix, seed=62)
    y = a.run()
    a.check(y)
    bad = _stalled(monkeypatch, a.run)
    assert int(a.err[0]) == stq.STQ_ERR_TIMEOUT
    # the first CTA has the last 128 tokens or fewer of the first sequence, counted from a multiple of 128, for heads 0 and 1
    first = (lens[0] - 1) // 128 * 128
    bad[first:lens[0], :2] = y[first:lens[0], :2]
    assert torch.equal(bad, y)
    a.err.zero_()
    a.check(a.run())


@pytest.mark.parametrize("kind, heads", [("bf16", 8), ("fp16", 24), ("fp32", 8)])
@pytest.mark.parametrize("lens", [[9], [70, 1, 0, 500], [1000] * 40])
def test_attn_decode(kind, heads, lens, monkeypatch):
    s = _Sequences(lens, heads, 2, kind, seed=63)
    s.append()
    y = s.attend()
    s.check(y)
    bad = torch.full_like(y, 3.0)
    _stalled(monkeypatch, lambda: stq.stq_attn_decode(s.cache, s.page_table, s.seq_len, s.q, bad))
    assert stq.stq_cache_check(s.cache, raise_on_error=False) == stq.STQ_ERR_TIMEOUT
    assert "timed out" in stq.stq_last_error()
    # the first warp's share begins with the first sequence and key head; it has no more than 1 / 1000 of all
    bad[0, :heads // 2] = y[0, :heads // 2]
    assert torch.equal(bad, y)
    assert torch.equal(s.attend(), y)
