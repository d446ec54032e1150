"""What the prompt and cache operators are measured on: cases, their plain forms, and their definitions in 64 bits.

Three operators, 128 values a head throughout:

  linear  stq_prompt_step: the gated delta rule over whole prompts.  For every head of every prompt,
              X_t = a_t X_{t-1} + b_t k_t (v_t - a_t X_{t-1}^T k_t)^T,   y_t = X_t^T q_t,   X_0 = 0,
          with one decay a_t a head and token.  Outputs: y, and the states after the last tokens in fp32.
          (The call also quantizes those states into the pool's pages, as stq_quantize_state does; the
          codes follow from the states that are returned here.)
  prompt  stq_attn_prompt: causal softmax attention over packed prompts with grouped heads; a prompt's
          queries are its last ones, so that a piece of a prompt can follow keys that are there already.
  cache   stq_cache_append and stq_attn_decode: keys and values held in 4 bits, in pages of 64 tokens.
          Each group of 32 values of a head has a binary16 scale s = half(max|x| / 7) and codes
          z = clip(rint(x / s), -7, 7).  A pass appends each prompt's new tokens and attends from its last.
          Outputs: y, and the values that the cache now holds for the new tokens (stq_cache_read).
"""
import math
import random

import torch

own = False

D, CHUNK, PAGE, GROUP = 128, 64, 64, 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # one short prompt on a few heads: what a single user's first question costs, all latency
        {"name": "linear one short", "kind": "linear", "type": "bf16", "n": 1, "longest": 37, "ragged": False, "heads": 4, "fused": False},
        # a serving step that admits a batch of prompts of mixed lengths; q, k and v are parts of one projection
        {"name": "linear ragged batch", "kind": "linear", "type": "bf16", "n": 24, "longest": 1500, "ragged": True, "heads": 32, "fused": True},
        # two long documents: few chains of many tokens
        {"name": "linear two long", "kind": "linear", "type": "fp16", "n": 2, "longest": 8192, "ragged": False, "heads": 32, "fused": False},
        # fp32 inputs, as the decode step takes them
        {"name": "linear fp32", "kind": "linear", "type": "fp32", "n": 6, "longest": 700, "ragged": True, "heads": 16, "fused": False},
        # three short prompts, the first of one token
        {"name": "prompt three short", "kind": "prompt", "type": "bf16", "n": 3, "longest": 61, "ragged": True, "heads": 8, "kv_heads": 2, "prefix": 0, "fused": False},
        # a serving step that admits a batch of prompts of mixed lengths
        {"name": "prompt ragged batch", "kind": "prompt", "type": "bf16", "n": 24, "longest": 2000, "ragged": True, "heads": 32, "kv_heads": 8, "prefix": 0, "fused": True},
        # one long document
        {"name": "prompt one long", "kind": "prompt", "type": "bf16", "n": 1, "longest": 8192, "ragged": False, "heads": 32, "kv_heads": 8, "prefix": 0, "fused": False},
        # pieces of long prompts behind keys that earlier pieces left; three query heads to a key head
        {"name": "prompt pieces", "kind": "prompt", "type": "fp16", "n": 4, "longest": 501, "ragged": False, "heads": 12, "kv_heads": 4, "prefix": 4100, "fused": False},
        # one sequence early in its answer
        {"name": "cache one short", "kind": "cache", "type": "bf16", "n": 1, "longest": 100, "ragged": False, "heads": 8, "kv_heads": 2, "new": 1},
        # a full serving batch at mixed lengths
        {"name": "cache ragged batch", "kind": "cache", "type": "bf16", "n": 64, "longest": 8192, "ragged": True, "heads": 32, "kv_heads": 8, "new": 1},
        # two very long sequences: few rows, a long axis
        {"name": "cache two long", "kind": "cache", "type": "fp16", "n": 2, "longest": 131071, "ragged": False, "heads": 16, "kv_heads": 2, "new": 1},
        # whole prompts put into the cache, and the first token after them
        {"name": "cache filled", "kind": "cache", "type": "bf16", "n": 8, "longest": 2049, "ragged": True, "heads": 32, "kv_heads": 8, "new": 2049},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "prompt", "cache"])
    c = {"kind": kind, "type": rng.choice(["bf16", "fp16"]), "ragged": rng.random() < 0.6}
    while True:
        n = c["n"] = _log(rng, 1, 64)
        if kind == "linear":
            c["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            c |= {"longest": _log(rng, 1, 8192), "heads": rng.randint(1, 48), "fused": rng.random() < 0.5}
            if n * c["longest"] * c["heads"] <= 24 * 1500 * 32 // (4 if c["type"] == "fp32" else 1):
                return c
        elif kind == "prompt":
            kv = rng.choice([1, 2, 4, 8])
            c |= {"longest": _log(rng, 1, 8192), "kv_heads": kv, "heads": kv * rng.choice([1, 2, 3, 4, 5, 8]),
                  "prefix": 0 if rng.random() < 0.6 else _log(rng, 1, 8000), "fused": False}
            c["fused"] = c["prefix"] == 0 and rng.random() < 0.5
            if n * c["longest"] * (c["longest"] + 2 * c["prefix"]) * c["heads"] <= 8192 * 8192 * 32 and n * (c["longest"] + c["prefix"]) <= 65536:
                return c
        else:
            kv = rng.choice([1, 2, 4, 8])
            c |= {"longest": _log(rng, 1, 131071), "kv_heads": kv, "heads": kv * rng.choice([1, 2, 3, 4, 7, 8, 16])}
            c["new"] = 1 if rng.random() < 0.7 else _log(rng, 1, 2048)
            if n * c["longest"] * kv <= 64 * 8192 * 8:
                return c


def _lengths(case):
    """Tokens of each sequence: all `longest`, or spread evenly below it with the longest and one of one token among them."""
    n, most = case["n"], case["longest"]
    if not case["ragged"]:
        return [most] * n
    rng = random.Random("%(n)d %(longest)d" % case)
    lens = [rng.randint(1, most) for _ in range(n)]
    lens[0] = 1
    lens[-1] = most
    return lens


def _starts(lens):
    return [0] + [sum(lens[:i + 1]) for i in range(len(lens))]


def _int(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["type"]]
    lens = _lengths(case)
    n, H = case["n"], case["heads"]
    s = {"case": case, "lens": lens, "dt": dt}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["kind"] == "linear":
        total = sum(lens)
        # one array [tokens][q, k, v][heads][128], or three; unit keys and queries, decays near one
        x = normal(total, 3, H, D)
        x[:, :2] /= x[:, :2].norm(dim=-1, keepdim=True)
        x = x.to(dt)
        s["q"], s["k"], s["v"] = (x[:, i] if case["fused"] else x[:, i].contiguous() for i in range(3))
        s["beta"] = torch.rand(total, H, generator=g, device=DEV)
        s["alpha"] = 0.9 + 0.099 * torch.rand(total, H, generator=g, device=DEV)
        s["start"] = _int(_starts(lens))
        s["y"] = torch.zeros(total, H, D, dtype=dt, device=DEV)
        s["state"] = torch.zeros(n, H, D, D, device=DEV)
        if own:
            import numpy as np

            from quantized_linear_attention_decode_b200 import stq
            # a program keeps its pool, the index lists of the batch and the workspace
            s["pool"] = stq.stq_pool_create(stq.STQ_GDN, n, 1, H, np.full(H, 6, np.uint8))
            s["req"], s["slot"], s["fresh"] = _int(list(range(n))), _int([0] * n), _int([1] * n)
            s["work"] = torch.empty(stq.stq_prompt_workspace(s["pool"], n, total), dtype=torch.uint8, device=DEV)
        return s
    Hk = case["kv_heads"]
    if case["kind"] == "prompt":
        tq, tk = sum(lens), sum(lens) + n * case["prefix"]
        if case["fused"]:  # one array [tokens][query heads, key heads, value heads][128]
            x = normal(tq, H + 2 * Hk, D).to(dt)
            s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        else:
            s["q"], s["k"], s["v"] = normal(tq, H, D).to(dt), normal(tk, Hk, D).to(dt), normal(tk, Hk, D).to(dt)
        s["q_start"], s["k_start"] = _int(_starts(lens)), _int(_starts([m + case["prefix"] for m in lens]))
        s["y"] = torch.zeros(tq, H, D, dtype=dt, device=DEV)
        return s
    x = _cache_inputs(case, seed)
    s |= {name: x[name] for name in ("table", "len", "q")}
    s["slot"], s["k"], s["v"] = (x[name][x["fresh"]] for name in ("slot", "k", "v"))
    s["y"] = torch.zeros(n, H, D, dtype=dt, device=DEV)
    s["k_held"], s["v_held"] = (torch.zeros(len(s["slot"]), Hk, D, device=DEV) for _ in range(2))
    old = [x[name][~x["fresh"]] for name in ("slot", "k", "v")]
    if own:
        from quantized_linear_attention_decode_b200 import stq
        s["cache"] = stq.stq_cache_create(x["num_pages"], Hk)
        stq.stq_cache_append(s["cache"], *old)
        s["work"] = torch.empty(stq.stq_attn_decode_workspace(s["cache"], n, H), dtype=torch.uint8, device=DEV)
    else:
        shape = (x["num_pages"], PAGE, Hk)
        s["held"] = [(torch.zeros(*shape, D // 2, dtype=torch.uint8, device=DEV),
                      torch.zeros(*shape, D // GROUP, dtype=torch.float16, device=DEV)) for _ in range(2)]
        for held, y in zip(s["held"], old[1:]):
            _put(held, old[0], y)
    return s


def _cache_inputs(case, seed):
    """All tokens of all sequences in order, and where the cache has them: every sequence's pages lie scattered over it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, lens, n = TYPES[case["type"]], _lengths(case), case["n"]
    pages = [(m + PAGE - 1) // PAGE for m in lens]
    order = random.Random(seed).sample(range(sum(pages) + 3), sum(pages))
    table = torch.zeros(n, max(pages), dtype=torch.int32)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = torch.tensor(order[at:at + p], dtype=torch.int32)
        at += p
    table, ln = table.to(DEV), _int(lens)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), ln.long())
    pos = torch.arange(sum(lens), device=DEV) - _int(_starts(lens)[:-1]).long()[seq]
    k, v = (torch.randn(sum(lens), case["kv_heads"], D, generator=g, device=DEV) for _ in range(2))
    k[..., 5] *= 6.0  # keys have channels of larger size
    k[..., 77] *= 4.0
    return {"table": table, "len": ln, "num_pages": sum(pages) + 3, "slot": table.long()[seq, pos // PAGE] * PAGE + pos % PAGE,
            "fresh": pos >= (ln.long()[seq] - case["new"]).clamp(min=0), "k": k.to(dt), "v": v.to(dt),
            "q": torch.randn(n, case["heads"], D, generator=g, device=DEV).to(dt)}


# ---------------------------------------------------------------- plain forms


def _put(held, slot, x):
    """Quantizes x [tokens][heads][128] into the token slots of a plain cache: two codes to a byte, offset by 8."""
    codes, scales = held
    x = x.float().unflatten(-1, (D // GROUP, GROUP))
    a = x.abs().amax(-1)
    s = (a / torch.full_like(a, 7.0)).half()
    sf = s.float()[..., None]
    z = torch.where(sf > 0, torch.round(x / sf), torch.zeros_like(x)).clamp(-7, 7).flatten(-2)
    u = (z + 8).to(torch.uint8)
    codes.view(-1, *codes.shape[2:])[slot] = u[..., 0::2] | (u[..., 1::2] << 4)
    scales.view(-1, *scales.shape[2:])[slot] = s


def _value(codes, scales):
    """fp32 [...][heads][128] of the codes and scales of a plain cache."""
    z = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    x = z.unflatten(-1, (D // GROUP, GROUP)) * scales.float()[..., None]
    return x.flatten(-2)


def _softmax(x):
    """Along the last axis; a row of -inf alone gives zeros."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t == 0, torch.ones_like(t), t)


def _plain_cache(s):
    case = s["case"]
    n, H, Hk = case["n"], case["heads"], case["kv_heads"]
    _put(s["held"][0], s["slot"], s["k"])
    _put(s["held"][1], s["slot"], s["v"])
    k, v = (_value(h[0][s["table"].long()], h[1][s["table"].long()]).flatten(1, 2) for h in s["held"])
    q = s["q"].float().view(n, Hk, H // Hk, D)
    x = q @ k.permute(0, 2, 3, 1) / math.sqrt(D)
    live = torch.arange(k.shape[1], device=DEV) < s["len"][:, None]
    x = torch.where(live[:, None, None], x, -math.inf)
    y = (_softmax(x) @ v.permute(0, 2, 1, 3)).reshape(n, H, D).to(s["dt"])
    return [y] + [_value(h[0].flatten(0, 1)[s["slot"]], h[1].flatten(0, 1)[s["slot"]]) for h in s["held"]]


def _plain_prompt(s):
    case = s["case"]
    Hk, G, pre = case["kv_heads"], case["heads"] // case["kv_heads"], case["prefix"]
    out, q0, k0 = [], 0, 0
    for m in s["lens"]:
        q = s["q"][q0:q0 + m].float().unflatten(1, (Hk, G)).permute(1, 2, 0, 3)
        k, v = (s[name][k0:k0 + m + pre].float().permute(1, 0, 2)[:, None] for name in ("k", "v"))
        x = q @ k.mT / math.sqrt(D)
        seen = torch.arange(m + pre, device=DEV) <= torch.arange(m, device=DEV)[:, None] + pre
        y = _softmax(torch.where(seen, x, -math.inf)) @ v
        out.append(y.permute(2, 0, 1, 3).flatten(1, 2))
        q0, k0 = q0 + m, k0 + m + pre
    return torch.cat(out).to(s["dt"])


def _plain_linear(s):
    """In chunks of 64 tokens.  With u_t = b_t (v_t - a_t X_{t-1}^T k_t) and R_ti the product of the decays behind i up to t,
    (I + A) U = diag(b) (V - diag(R_t0) K X_0), A_ti = b_t R_ti k_t.k_i for i < t, and the chunk's outputs and next state are
    products with U.  A is nilpotent, so its inverse is a product of six factors."""
    n, H = s["case"]["n"], s["case"]["heads"]
    lens = torch.tensor(s["lens"], device=DEV)
    chunks = (max(s["lens"]) + CHUNK - 1) // CHUNK
    at = torch.arange(chunks * CHUNK, device=DEV)
    live = at < lens[:, None]
    token = (s["start"][:-1].long()[:, None] + torch.where(live, at, 0)).view(n, chunks, CHUNK)
    live = live.view(n, 1, chunks, CHUNK)
    q, k, v = (s[x][token].float().permute(0, 3, 1, 2, 4) * live[..., None] for x in ("q", "k", "v"))
    b = s["beta"][token].permute(0, 3, 1, 2) * live
    lg = torch.where(live, s["alpha"][token].permute(0, 3, 1, 2).double().log(), 0.0).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=DEV).tril()
    R = torch.exp((lg[..., :, None] - lg[..., None, :]).tril()).float() * low
    first = torch.exp(lg).float()[..., None]
    A = b[..., None] * R.tril(-1) * (k @ k.mT)
    inv = torch.eye(CHUNK, device=DEV) - A
    for _ in range(5):
        A = A @ A
        inv = inv + inv @ A
    P = R * (q @ k.mT)
    last = R[..., -1, :, None] * k
    X, ys = torch.zeros(n, H, D, D, device=DEV), []
    for c in range(chunks):
        u = inv[:, :, c] @ (b[:, :, c, :, None] * (v[:, :, c] - first[:, :, c] * (k[:, :, c] @ X)))
        ys.append(first[:, :, c] * (q[:, :, c] @ X) + P[:, :, c] @ u)
        X = first[:, :, c, -1:] * X + last[:, :, c].mT @ u
    y = torch.stack(ys, 2).permute(0, 2, 3, 1, 4).flatten(1, 2)
    return [y[live.view(n, -1)].to(s["dt"]), X]


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"linear": _plain_linear, "prompt": _plain_prompt, "cache": _plain_cache}[kind](s)
    from quantized_linear_attention_decode_b200 import stq
    if kind == "linear":
        stq.stq_prompt_step(s["pool"], s["req"], s["slot"], s["start"], s["q"], s["k"], s["v"], s["beta"], s["alpha"], s["y"], s["state"],
                            fresh=s["fresh"], workspace=s["work"])
        return [s["y"], s["state"]]
    if kind == "prompt":
        stq.stq_attn_prompt(s["q_start"], s["k_start"], s["q"], s["k"], s["v"], s["y"])
        return s["y"]
    stq.stq_cache_append(s["cache"], s["slot"], s["k"], s["v"])
    stq.stq_attn_decode(s["cache"], s["table"], s["len"], s["q"], s["y"], workspace=s["work"])
    stq.stq_cache_read(s["cache"], s["slot"], s["k_held"], s["v_held"])
    return [s["y"], s["k_held"], s["v_held"]]


def work(case):
    lens = _lengths(case)
    H, size = case["heads"], 4 if case["type"] == "fp32" else 2
    if case["kind"] == "linear":
        # q, k, v, y, beta, alpha of every token and head, and each state once; three products of the state with a vector
        t = sum(lens) * H
        return {"bytes": t * (4 * D * size + 8) + len(lens) * H * D * D * 4, "flops": t * 6 * D * D}
    Hk = case["kv_heads"]
    if case["kind"] == "prompt":
        pairs = sum(m * case["prefix"] + m * (m + 1) // 2 for m in lens)
        return {"bytes": (2 * sum(lens) * H + 2 * sum(m + case["prefix"] for m in lens) * Hk) * D * size, "flops": 4 * D * H * pairs}
    # a token of a key head takes 2 x 64 bytes of codes and 2 x 8 of scales; new tokens are read in full, written packed, and given back in fp32
    new = sum(min(m, case["new"]) for m in lens)
    return {"bytes": sum(lens) * Hk * 144 + new * Hk * (2 * D * size + 144 + 2 * D * 4) + 2 * len(lens) * H * D * size, "flops": 4 * D * H * sum(lens)}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    lens, H = _lengths(case), case["heads"]
    if case["kind"] == "cache":
        c = _cache_inputs(case, seed)
    else:
        s = prepare(case, seed)
    if case["kind"] == "linear":
        # token by token: sequences of one length or longer advance together
        start = s["start"].tolist()
        order = sorted(range(len(lens)), key=lambda i: -lens[i])
        X = torch.zeros(len(lens), H, D, D, dtype=torch.float64, device=DEV)
        y = torch.zeros(sum(lens), H, D, dtype=torch.float64, device=DEV)
        first = torch.tensor([start[i] for i in order], device=DEV)
        sizes = [lens[i] for i in order]
        act = len(order)
        for t in range(max(lens)):
            while sizes[act - 1] <= t:
                act -= 1
            at = first[:act] + t
            a, b = s["alpha"][at].double()[..., None, None], s["beta"][at].double()[..., None, None]
            k, v, q = (s[x][at].double()[..., None, :] for x in ("k", "v", "q"))
            S = X[:act] * a
            S = S + b * k.mT @ (v - k @ S)
            X[:act] = S
            y[at] = (q @ S)[..., 0, :]
        back = torch.empty(len(order), dtype=torch.long)
        back[torch.tensor(order)] = torch.arange(len(order))
        return [y, X[back.to(DEV)]]
    G, out = H // case["kv_heads"], []
    if case["kind"] == "prompt":
        qs, ks = s["q_start"].tolist(), s["k_start"].tolist()
        for i, m in enumerate(lens):
            y = torch.empty(m, H, D, dtype=torch.float64, device=DEV)
            for h in range(H):
                k, v = (s[x][ks[i]:ks[i + 1], h // G].double() for x in ("k", "v"))
                x = torch.einsum("td,sd->ts", s["q"][qs[i]:qs[i + 1], h].double(), k) * D ** -0.5
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu(ks[i + 1] - ks[i] - m + 1), -math.inf)
                w = (x - x.max(-1, keepdim=True).values).exp_()
                y[:, h] = torch.einsum("ts,sd->td", w, v) / w.sum(-1, keepdim=True)
            out.append(y)
        return torch.cat(out)
    i0, new = 0, []
    for i, m in enumerate(lens):
        kv = []
        for name in ("k", "v"):
            x = c[name][i0:i0 + m].double().reshape(m, case["kv_heads"], D // GROUP, GROUP)
            step = (x.abs().max(-1, keepdim=True).values / 7).half().double()
            z = torch.nan_to_num(x / step).round().clamp(-7, 7)
            kv.append((z * step).reshape(m, case["kv_heads"], D))
        new.append([x[-case["new"]:] for x in kv])
        kv = [x.repeat_interleave(G, 1) for x in kv]
        x = torch.einsum("hd,shd->hs", c["q"][i].double(), kv[0]) * D ** -0.5
        w = (x - x.max(-1, keepdim=True).values).exp_()
        out.append(torch.einsum("hs,shd->hd", w, kv[1]) / w.sum(-1, keepdim=True))
        i0 += m
    return [torch.stack(out)] + [torch.cat(x) for x in zip(*new)]
