"""GPU: prompts through a linear-attention and a softmax-attention layer, then
decode steps of both as one captured graph, as a hybrid stack runs them."""
import numpy as np
import pytest

from quantized_linear_attention_decode_b200 import stq
from test_gpu_attn_prompt import _Attn
from test_gpu_cache import _Sequences
from test_gpu_prompt import _Prompts, recurrence

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

STEPS = 4


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("lens", [[70, 1, 0, 130, 62], [3]])
def test_prompts_then_decode_steps(kind, lens):
    n, H, heads, kv = len(lens), 4, 8, 2
    rng = np.random.default_rng(5)
    stream = torch.cuda.Stream()
    linear, attn = _Prompts(lens, H, kind, seed=3), _Attn(lens, heads, kv, kind, seed=4)
    dt = linear.dt
    # pages of each sequence in any order, with room for the steps
    pages = [(m + STEPS + 63) // 64 for m in lens]
    order, table = rng.permutation(sum(pages)), np.zeros((n, max(pages)), np.int32)
    for i, p in enumerate(pages):
        table[i, :p], order = order[:p], order[p:]
    slot_of = lambda i, t: int(table[i, t // 64]) * 64 + t % 64  # noqa: E731
    cache = stq.stq_cache_create(sum(pages), kv)
    slots = torch.tensor([slot_of(i, t) for i, m in enumerate(lens) for t in range(m)], dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        linear.run()
        y = torch.empty_like(attn.q)
        stq.stq_attn_prompt(attn.q_start, attn.k_start, attn.q, attn.k, attn.v, y, err=attn.err)
        stq.stq_cache_append(cache, slots, attn.k, attn.v)
    torch.cuda.synchronize()
    linear.check()
    attn.check(y)

    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    q, k, v, yl = (new(n, H, 128) for _ in range(4))
    beta, alpha = new(n, H), new(n, H)
    qa, ya, ka, va = new(n, heads, 128, dtype=dt), new(n, heads, 128, dtype=dt), new(n, kv, 128, dtype=dt), new(n, kv, 128, dtype=dt)
    slot, seq_len = new(n, dtype=torch.int64), new(n, dtype=torch.int32)
    page_table = torch.from_numpy(table).cuda()
    work = new(stq.stq_attn_decode_workspace(cache, n, heads), dtype=torch.uint8)

    def step():
        stq.stq_decode_step(linear.pool, linear.req, linear.slot, q, k, v, beta, alpha, yl)
        stq.stq_cache_append(cache, slot, ka, va)
        stq.stq_attn_decode(cache, page_table, seq_len, qa, ya, workspace=work)

    # all token slots negative and all lengths zero: the step that is run before the capture leaves the cache alone
    slot.fill_(-1)
    seq_len.zero_()
    for t in (q, k, v, beta, qa, ka, va):
        t.zero_()
    alpha.fill_(1)
    saved = [stq.stq_export_slot(linear.pool, int(r), int(s)) for r, s in zip(linear.req, linear.slot)]
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    assert bool((ya == 0).all())
    for r, s, page in zip(linear.req, linear.slot, saved):
        stq.stq_import_slot(linear.pool, int(r), int(s), page)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()

    ks, vs = ([list(_part) for _part in (t[a:b] for a, b in zip(attn.ks, attn.ks[1:]))] for t in (attn.k, attn.v))
    S = new(n, H, 128, 128)
    for at in range(STEPS):
        stq.stq_dequantize_state(linear.pool, linear.req, linear.slot, S)
        before = _f64(S)
        for t, unit in ((q, True), (k, True), (v, False), (qa, False), (ka, False), (va, False)):
            x = rng.standard_normal(t.shape)
            t.copy_(torch.from_numpy(x / np.linalg.norm(x, axis=-1, keepdims=True) if unit else x))
        beta.copy_(torch.from_numpy(rng.uniform(0, 1, beta.shape)))
        alpha.copy_(torch.from_numpy(rng.uniform(0.9, 0.999, alpha.shape)))
        slot.copy_(torch.tensor([slot_of(i, m + at) for i, m in enumerate(lens)], dtype=torch.int64))
        seq_len.copy_(torch.tensor([m + at + 1 for m in lens], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        stq.stq_pool_check(linear.pool)
        stq.stq_cache_check(cache)
        # the decode step: 1e-5 of the head's largest value
        for i in range(n):
            want, _, _ = recurrence(*(_f64(t[i:i + 1]) for t in (q, k, v, beta, alpha)), before[i])
            assert np.all(np.abs(_f64(yl[i:i + 1]) - want) <= 1e-5 * np.abs(want).max(-1, keepdims=True)), (at, i)
        # attention over the prompt's tokens and the steps' so far
        for i in range(n):
            ks[i].append(ka[i].clone())
            vs[i].append(va[i].clone())
        seen = object.__new__(_Sequences)
        seen.lens, seen.heads, seen.kv_heads, seen.dt, seen.q = [len(x) for x in ks], heads, kv, dt, qa
        seen.k, seen.v = (torch.stack([t for x in part for t in x]) for part in (ks, vs))
        seen.check(ya)
