"""Measured cases of the operators that take whole prompts and batches of
requests around the BitLinear products:

  rope       qk_norm_rope: RMS norm of every query and key head (optional),
             rotation by the token's position, keys and values written to
             their cache rows
  attention  attention_prefill: causal attention of packed sequences, grouped
             heads, queries at the end of their sequence's keys
  adapter    adapter_add: low-rank adapters of many requests added to the
             output of a shared projection

`run` computes an operator in plain torch where `own` is false, and through the
package's entry points where it is true.  `exact` gives the same results from
the definitions in 64 bits.
"""
import math
import random

import torch

own = False

HEAD_DIM = 128
EPS = 1e-5
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ the cases

def listed():
    """The head layout 20 / 5 x 128, hidden 2560, feed-forward 6912 and caches
    of 4096 rows are those of the package's 2.4B-shaped decoder; the others are
    generic."""
    return [
        # one prompt that fills two caches' worth of positions: the largest product
        {"name": "prompt 8192", "op": "attention", "heads": 20, "kv_heads": 5, "batch": 1, "q_lo": 8192, "q_hi": 8192,
         "past_lo": 0, "past_hi": 0, "lens_seed": 0, "layout": "packed", "gap": 0},
        # prompts of different lengths waiting together, packed without padding
        {"name": "prompts packed", "op": "attention", "heads": 20, "kv_heads": 5, "batch": 12, "q_lo": 1, "q_hi": 1301,
         "past_lo": 0, "past_hi": 0, "lens_seed": 3, "layout": "packed", "gap": 5},
        # a short prompt on its own: the time to the first token is latency
        {"name": "prompt 37", "op": "attention", "heads": 20, "kv_heads": 5, "batch": 1, "q_lo": 37, "q_hi": 37,
         "past_lo": 0, "past_hi": 0, "lens_seed": 0, "layout": "packed", "gap": 0},
        # the next piece of a long prompt, against the decoder's own cache
        {"name": "chunk on a cache", "op": "attention", "heads": 20, "kv_heads": 5, "batch": 1, "q_lo": 509, "q_hi": 509,
         "past_lo": 3500, "past_hi": 3500, "lens_seed": 0, "layout": "cache", "gap": 87},
        # one new token for each of many running requests
        {"name": "tokens of 64 requests", "op": "attention", "heads": 20, "kv_heads": 5, "batch": 64, "q_lo": 1, "q_hi": 1,
         "past_lo": 0, "past_hi": 4095, "lens_seed": 7, "layout": "packed", "gap": 0},
        # one token at the end of a long history: all of the GPU for few rows
        {"name": "token after 30000", "op": "attention", "heads": 16, "kv_heads": 2, "batch": 1, "q_lo": 1, "q_hi": 1,
         "past_lo": 30011, "past_hi": 30011, "lens_seed": 0, "layout": "cache", "gap": 2756},
        # a long prompt's queries and keys, one fused projection's output
        {"name": "rope 8192", "op": "rope", "heads": 20, "kv_heads": 5, "tokens": 8192, "rows": 8192, "past": 0,
         "norm": True, "halves": False, "f32": False, "skip": 0.0},
        # prompts of odd lengths on projections kept in fp32, no norm
        {"name": "rope 1283 f32", "op": "rope", "heads": 20, "kv_heads": 5, "tokens": 1283, "rows": 4096, "past": 700,
         "norm": False, "halves": True, "f32": True, "skip": 0.02},
        # one new token for each of 48 requests, some of them padding
        {"name": "rope 48", "op": "rope", "heads": 16, "kv_heads": 2, "tokens": 48, "rows": 4096, "past": 1000,
         "norm": True, "halves": False, "f32": False, "skip": 0.05},
        # packed prompts of 6 requests, each with its adapter, on the gate projection
        {"name": "adapters of prompts", "op": "adapter", "tokens": 4093, "K": 2560, "N": 6912, "rank": 16, "adapters": 6,
         "runs": True, "none": 0.1, "f32": False},
        # tokens of 32 running requests, nearly every one with an adapter of its own
        {"name": "adapters of 32 tokens", "op": "adapter", "tokens": 32, "K": 2560, "N": 2560, "rank": 16, "adapters": 24,
         "runs": False, "none": 0.1, "f32": False},
        # one token with one adapter, on the down projection in fp32
        {"name": "adapter of a token", "op": "adapter", "tokens": 1, "K": 6912, "N": 2560, "rank": 64, "adapters": 4,
         "runs": False, "none": 0.0, "f32": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "adapter"])
    heads, kv = rng.choice([(20, 5), (20, 5), (16, 2), (8, 8), (6, 2), (7, 1)])
    if op == "rope":
        T = _spread(rng, 1, 8192)
        rows = T + rng.randrange(0, 2000)
        return {"op": op, "heads": heads, "kv_heads": kv, "tokens": T, "rows": rows, "past": rng.randrange(0, 3000),
                "norm": rng.random() < 0.6, "halves": rng.random() < 0.4, "f32": rng.random() < 0.3,
                "skip": rng.choice([0.0, 0.03, 0.3])}
    if op == "adapter":
        K, N = rng.choice([(2560, 2560), (2560, 640), (2560, 6912), (6912, 2560), (704, 1001), (256, 333)])
        T = _spread(rng, 1, 4096)
        return {"op": op, "tokens": T, "K": K, "N": N, "rank": rng.choice([8, 16, 16, 24, 32, 64]),
                "adapters": rng.randrange(1, 17), "runs": rng.random() < 0.6, "none": rng.choice([0.0, 0.1, 0.5]),
                "f32": rng.random() < 0.3}
    kind = rng.choice(["prompts", "prompts", "chunk", "tokens"])
    case = {"op": op, "heads": heads, "kv_heads": kv, "lens_seed": rng.randrange(1 << 20), "layout": "packed",
            "gap": rng.choice([0, 0, 3, 64])}
    if kind == "prompts":
        batch = rng.randrange(1, 13)
        hi = _spread(rng, 1, 4800 // batch)
        return {**case, "batch": batch, "q_lo": rng.randrange(1, hi + 1), "q_hi": hi, "past_lo": 0, "past_hi": 0}
    if kind == "chunk":
        nq, past = _spread(rng, 2, 1500), _spread(rng, 1, 8000)
        return {**case, "batch": 1, "q_lo": nq, "q_hi": nq, "past_lo": past, "past_hi": past, "layout": "cache"}
    batch = _spread(rng, 1, 96)
    hi = _spread(rng, 1, 4095)
    return {**case, "batch": batch, "q_lo": 1, "q_hi": rng.choice([1, 1, 4]), "past_lo": rng.randrange(0, hi + 1),
            "past_hi": hi}


def _lens(case):
    """Query and key lengths of the sequences: a request's keys are its past
    and its new tokens."""
    r = random.Random(case["lens_seed"])
    nq = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    nk = [n + r.randint(case["past_lo"], case["past_hi"]) for n in nq]
    return nq, nk


def work(case):
    D = HEAD_DIM
    if case["op"] == "attention":
        nq, nk = _lens(case)
        H, Hkv = case["heads"], case["kv_heads"]
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))
        return {"bytes": 2.0 * D * (2 * H * sum(nq) + 2 * Hkv * sum(nk)), "flops": 4.0 * D * H * pairs}
    if case["op"] == "rope":
        T, n = case["tokens"], (case["heads"] + 2 * case["kv_heads"]) * D
        b = T * n * ((4 if case["f32"] else 2) + 2) + min(T, case["rows"]) * D * 4
        return {"bytes": float(b), "flops": 8.0 * T * n}
    T, K, N, r = case["tokens"], case["K"], case["N"], case["rank"]
    used = min(case["adapters"], T)
    b = T * K * 2 + 2 * T * N * (4 if case["f32"] else 2) + used * r * (K + N) * 2
    return {"bytes": float(b), "flops": 2.0 * T * r * (K + N)}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    return {"attention": _prepare_attention, "rope": _prepare_rope, "adapter": _prepare_adapter}[case["op"]](case, seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _prepare_attention(case, seed):
    g, D = _gen(seed), HEAD_DIM
    H, Hkv = case["heads"], case["kv_heads"]
    nq, nk = _lens(case)
    Tq, Tk = sum(nq), sum(nk)
    q = _randn(g, Tq, H, D).to(torch.bfloat16)
    rows = Tk + case["gap"]      # rows behind the last key belong to nobody
    if case["layout"] == "cache":
        k = (1.5 * _randn(g, Hkv, rows, D)).to(torch.bfloat16).transpose(0, 1)
        v = _randn(g, Hkv, rows, D).to(torch.bfloat16).transpose(0, 1)
    else:
        kv = _randn(g, rows, 2 * Hkv, D)
        kv[:, :Hkv] *= 1.5
        kv = kv.to(torch.bfloat16)
        k, v = kv[:, :Hkv], kv[:, Hkv:]
    return {"case": case, "q": q, "k": k, "v": v, "cu_q": _cu(nq), "cu_k": _cu(nk), "out": torch.empty_like(q)}


def _prepare_rope(case, seed):
    g, D = _gen(seed), HEAD_DIM
    T, H, Hkv, R = case["tokens"], case["heads"], case["kv_heads"], case["rows"]
    dt = torch.float32 if case["f32"] else torch.bfloat16
    qkv = (_randn(g, T, H + 2 * Hkv, D) * (0.5 + torch.rand(T, 1, 1, generator=g, device="cuda"))).to(dt)
    P = T + case["past"]
    inv = ROPE_BASE ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    ang = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * inv
    table = torch.stack([ang.cos(), ang.sin()], -1).to(torch.float32)
    positions = (torch.arange(T, device="cuda") + case["past"]).to(torch.int32)
    slots = torch.randperm(R, generator=g, device="cuda")[:T]
    if T > 256:                  # a prompt's rows lie one behind the other
        slots = torch.arange(T, device="cuda") + int(seed) % (R - T + 1)
    if case["skip"]:             # padding of the batch: no cache row
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["skip"], -1, slots)
    cache = torch.zeros(2, Hkv, R, D, dtype=torch.bfloat16, device="cuda")
    gains = [(1 + 0.1 * _randn(g, D)).to(torch.bfloat16) if case["norm"] else None for _ in range(2)]
    return {"case": case, "q": qkv[:, :H], "k": qkv[:, H:H + Hkv], "v": qkv[:, H + Hkv:], "table": table,
            "positions": positions, "slots": slots.to(torch.int32), "q_gain": gains[0], "k_gain": gains[1],
            "q_out": torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"),
            "cache_k": cache[0].transpose(0, 1), "cache_v": cache[1].transpose(0, 1)}


def _prepare_adapter(case, seed):
    g = _gen(seed)
    T, K, N, r, n = (case[f] for f in ("tokens", "K", "N", "rank", "adapters"))
    x = _randn(g, T, K).to(torch.bfloat16)
    y = _randn(g, T, N).to(torch.float32 if case["f32"] else torch.bfloat16)
    down = (_randn(g, n, r, K) * K ** -0.5).to(torch.bfloat16)
    up = (_randn(g, n, N, r) * r ** -0.5).to(torch.bfloat16)
    if case["runs"]:             # each request's tokens lie together
        cuts = torch.randint(0, T + 1, (n,), generator=g, device="cuda").sort().values
        index = torch.bucketize(torch.arange(T, device="cuda"), cuts, right=True) % n
    else:
        index = torch.randint(0, n, (T,), generator=g, device="cuda")
    if case["none"]:             # requests without an adapter
        out = torch.rand(n if case["runs"] else T, generator=g, device="cuda") < case["none"]
        index = torch.where(out[index] if case["runs"] else out, -1, index)
    scale = 0.5 + torch.rand(n, generator=g, device="cuda")
    return {"case": case, "x": x, "y": y, "down": down, "up": up, "index": index.to(torch.int32), "scale": scale,
            "out": torch.empty_like(y)}


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import bit_ternary_weight_b200 as bl
        if op == "attention":
            return bl.attention_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["out"])
        if op == "rope":
            return bl.qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["table"], q_gain=s["q_gain"],
                                   k_gain=s["k_gain"], eps=EPS, halves=s["case"]["halves"], slots=s["slots"],
                                   q_out=s["q_out"], k_out=s["cache_k"], v_out=s["cache_v"])
        return bl.adapter_add(s["y"], s["x"], s["down"], s["up"], s["index"], scale=s["scale"], out=s["out"])
    return {"attention": _plain_attention, "rope": _plain_rope, "adapter": _plain_adapter}[op](s)


def _plain_attention(s):
    """softmax(scale q k^T) v over the keys each query sees, all sequences in
    one masked product."""
    q, k, v, D = s["q"].float(), s["k"].float(), s["v"].float(), HEAD_DIM
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    Tq, H = q.shape[:2]
    rows, Hkv = k.shape[:2]
    G = H // Hkv
    tq, tk = torch.arange(Tq, device=q.device), torch.arange(rows, device=q.device)
    bq = torch.bucketize(tq, cu_q[1:], right=True)
    # query i of a sequence sees its keys up to i + nk - nq
    last = cu_k[bq + 1] - (cu_q[bq + 1] - tq)
    seen = (tk >= cu_k[bq][:, None]) & (tk <= last[:, None])
    q = q.view(Tq, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * Tq, D)
    score = (q @ k.permute(1, 2, 0)).view(Hkv, G, Tq, rows).mul_(D ** -0.5)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(Hkv, G * Tq, rows) @ v.transpose(0, 1)
    out = out.view(Hkv, G, Tq, D) / torch.where(total == 0, 1.0, total)
    return out.permute(2, 0, 1, 3).reshape(Tq, H, D).to(torch.bfloat16)


def _rotate(x, cs, halves):
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]
    if halves:
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * n, a * n + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)


def _plain_rope(s):
    q, k, halves = s["q"].float(), s["k"].float(), s["case"]["halves"]
    cs = s["table"][s["positions"].long()]
    if s["q_gain"] is not None:
        q = q * (q.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["q_gain"].float()
        k = k * (k.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["k_gain"].float()
    s["q_out"].copy_(_rotate(q, cs, halves))
    keep = s["slots"] >= 0
    to = s["slots"][keep].long()
    s["cache_k"][to] = _rotate(k, cs, halves).to(torch.bfloat16)[keep]
    s["cache_v"][to] = s["v"].to(torch.bfloat16)[keep]
    return s["q_out"], s["cache_k"], s["cache_v"]


def _plain_adapter(s):
    x, y, down, up = s["x"].float(), s["y"].float(), s["down"].float(), s["up"].float()
    n, r, K = down.shape
    which = s["index"][:, None] == torch.arange(n, device=x.device)
    u = (x @ down.view(n * r, K).t()).view(-1, n, r) * (which * s["scale"])[..., None]
    return (y + u.view(-1, n * r) @ up.transpose(1, 2).reshape(n * r, -1)).to(s["y"].dtype)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "rope": _exact_rope, "adapter": _exact_adapter}[case["op"]](s)


def _exact_attention(s):
    nq, nk = _lens(s["case"])
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    group = q.shape[1] // k.shape[1]
    a = b = 0
    for m, n in zip(nq, nk):
        future = torch.ones(m, n, dtype=torch.bool, device=q.device).triu(n - m + 1)
        for h in range(q.shape[1]):
            score = q[a:a + m, h].double() @ k[b:b + n, h // group].double().t() / math.sqrt(HEAD_DIM)
            out[a:a + m, h] = score.masked_fill(future, -math.inf).softmax(-1) @ v[b:b + n, h // group].double()
        a, b = a + m, b + n
    return out


def _exact_rope(s):
    table = s["table"].double()[s["positions"].long()]
    turn = torch.complex(table[..., 0], table[..., 1])[:, None]

    def head(x, gain):
        x = x.double()
        if gain is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD_DIM + EPS) * gain.double()
        if s["case"]["halves"]:
            z = torch.complex(x[..., :HEAD_DIM // 2].contiguous(), x[..., HEAD_DIM // 2:].contiguous()) * turn
            return torch.cat([z.real, z.imag], -1)
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2)) * turn).flatten(-2)

    k, caches = head(s["k"], s["k_gain"]), []
    for x in (k, s["v"].double()):
        cache = torch.zeros(s["cache_k"].shape, dtype=torch.float64, device=x.device)
        for t, row in enumerate(s["slots"].tolist()):
            if row >= 0:
                cache[row] = x[t]
        caches.append(cache)
    return head(s["q"], s["q_gain"]), caches[0], caches[1]


def _exact_adapter(s):
    out = s["y"].double()
    for a in range(s["down"].shape[0]):
        at = (s["index"] == a).nonzero().flatten()
        out[at] += s["scale"][a].double() * (s["x"][at].double() @ s["down"][a].double().t() @ s["up"][a].double().t())
    return out
