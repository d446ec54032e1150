"""Host-side checks of the prompt and cache entry points that need no GPU: what
they refuse, and with which status, before they touch a device."""
import ctypes as C

import pytest

from quantized_linear_attention_decode_b200 import stq

ROW = 1 << 20  # an address that no refused call follows


def _rows(address=ROW, token=1024, head=128):
    return C.byref(stq._Rows(address, token, head))


def _attn(**change):
    a = dict(q_start=ROW, k_start=ROW, n=1, heads=8, kv=2, tq=4, tk=4, dtype=stq.STQ_BF16, q=_rows(), k=_rows(), v=_rows(),
             scale=0.1, y=ROW, err=None, stream=None)
    a |= change
    return stq.load().stq_attn_prompt(*a.values())


@pytest.mark.parametrize("status, change", [
    ("STQ_ERR_ARG", dict(n=-1)),
    ("STQ_ERR_ARG", dict(tq=-1)),
    ("STQ_ERR_ARG", dict(tk=-1)),
    ("STQ_ERR_ARG", dict(heads=0)),
    ("STQ_ERR_ARG", dict(kv=0)),
    ("STQ_ERR_ARG", dict(heads=7)),
    ("STQ_ERR_ARG", dict(dtype=3)),
    ("STQ_ERR_UNSUPPORTED", dict(dtype=2)),
    ("STQ_ERR_ARG", dict(scale=float("nan"))),
    ("STQ_ERR_ARG", dict(scale=float("inf"))),
    ("STQ_ERR_ARG", dict(q_start=None)),
    ("STQ_ERR_ARG", dict(k_start=None)),
    ("STQ_ERR_ARG", dict(q=None)),
    ("STQ_ERR_ARG", dict(k=_rows(None))),
    ("STQ_ERR_ARG", dict(v=_rows(ROW + 2))),
    ("STQ_ERR_ARG", dict(q=_rows(token=1025))),
    ("STQ_ERR_ARG", dict(k=_rows(head=129))),
    ("STQ_ERR_UNSUPPORTED", dict(v=_rows(token=-1024))),
    ("STQ_ERR_UNSUPPORTED", dict(q=_rows(head=0))),
    ("STQ_ERR_ARG", dict(y=None)),
    ("STQ_ERR_ARG", dict(y=ROW + 8)),
])
def test_attn_prompt_refuses(status, change):
    assert stq.STATUS[_attn(**change)] == status
    assert stq.load().stq_last_error()


def test_attn_prompt_of_nothing_and_launch_failure(monkeypatch):
    assert _attn(n=0, q_start=None, k_start=None) == 0
    assert _attn(tq=0, y=None) == 0
    monkeypatch.setenv("STQ_FAULT", "launch")
    assert stq.STATUS[_attn()] == "STQ_ERR_CUDA"


@pytest.mark.parametrize("status, pages, heads, dim", [
    ("STQ_ERR_ARG", 0, 2, 128),
    ("STQ_ERR_ARG", -1, 2, 128),
    ("STQ_ERR_ARG", 4, 0, 128),
    ("STQ_ERR_UNSUPPORTED", 4, 2, 64),
    ("STQ_ERR_ARG", 2 ** 31 - 1, 2 ** 31 - 1, 128),
])
def test_cache_create_refuses(status, pages, heads, dim):
    h = C.c_void_p()
    assert stq.STATUS[stq.load().stq_cache_create(pages, heads, dim, C.byref(h))] == status
    assert not h.value


def test_cache_create_out_of_memory(monkeypatch):
    monkeypatch.setenv("STQ_FAULT", "alloc")
    with pytest.raises(stq.StqError) as e:
        stq.stq_cache_create(4, 2)
    assert e.value.status == stq.STQ_ERR_OOM


def test_null_handles():
    L, a = stq.load(), C.c_size_t()
    bad = {v: k for k, v in stq.STATUS.items()}["STQ_ERR_ARG"]
    assert L.stq_cache_create(4, 2, 128, None) == bad
    assert L.stq_cache_destroy(None) == 0
    assert L.stq_cache_bytes(None, C.byref(a)) == bad
    assert L.stq_cache_append(None, None, 0, 0, _rows(), _rows(), None) == bad
    assert L.stq_cache_read(None, None, 0, None, None, None) == bad
    assert L.stq_cache_check(None, None) == bad
    assert L.stq_attn_decode_workspace(None, 1, 1, C.byref(a)) == bad
    assert L.stq_attn_decode(None, None, 0, None, 0, 1, 0, _rows(), 1.0, None, None, 0, None) == bad
    assert L.stq_prompt_workspace(None, 1, 1, C.byref(a)) == bad
    assert L.stq_prompt_step(None, None, None, 0, None, 0, None, 0, _rows(), _rows(), _rows(), None, None, None, None, None, 0,
                             None) == bad


def test_bindings_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, s = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        stq.stq_attn_prompt(s, s, x, x, x, x)
    with pytest.raises(ValueError):
        stq.stq_attn_prompt(s, s, x[0], x, x, x)


def test_pool_device_refuses():
    a = C.c_int32()
    assert stq.STATUS[stq.load().stq_pool_device(None, C.byref(a))] == "STQ_ERR_ARG"
