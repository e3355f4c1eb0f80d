"""The operators of a serving step over a paged key/value cache, as measured cases.

Four operators, used in this order by every decoder block of a step over many requests:

  plan    block tables, slots and positions of the step's tokens from the requests' lengths
  norm    residual addition + BitNetRMSNorm + per-token absmax int8 codes
  rope    rotary embedding of q and k, k and v appended to their slots of the paged cache
  attn    causal grouped-query attention of each request's new tokens over its pages

`own` chooses between the plain forms (elementary torch operations) and the framework's calls.
"""
import math
import random

import torch

own = False

D = 128  # head size
EPS = 1e-6


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one request decoding one token: the smallest step, where only latency counts (2B4T heads)
        {"name": "plan_one", "op": "plan", "B": 1, "new_max": 1, "ctx_max": 700, "ragged": False, "page": 16, "lens": 1},
        # a full decode batch: one new token each, some of them opening a page
        {"name": "plan_decode_256", "op": "plan", "B": 256, "new_max": 1, "ctx_max": 8192, "ragged": True, "page": 16, "lens": 2},
        # prompts arriving together: many new pages and tokens
        {"name": "plan_prompts_96", "op": "plan", "B": 96, "new_max": 700, "ctx_max": 1000, "ragged": True, "page": 32, "lens": 3},
        # one token between two blocks of the 2B4T model
        {"name": "norm_one", "op": "norm", "T": 1, "K": 2560, "x": "bf16", "res": "bf16"},
        # a decode batch of a 5120-wide model that keeps its residual stream in fp32
        {"name": "norm_batch", "op": "norm", "T": 333, "K": 5120, "x": "bf16", "res": "f32"},
        # a prefill step of an 8192-wide model
        {"name": "norm_prefill", "op": "norm", "T": 8192, "K": 8192, "x": "bf16", "res": "bf16"},
        # one token's heads (2B4T)
        {"name": "rope_one", "op": "rope", "B": 1, "new_max": 1, "ctx_max": 700, "ragged": False, "page": 16, "Hq": 20, "Hkv": 5, "x": "bf16", "theta": 10000.0, "lens": 4},
        # the tokens of a prefill step at the 70B shape
        {"name": "rope_prefill", "op": "rope", "B": 5, "new_max": 2048, "ctx_max": 8192, "ragged": True, "page": 64, "Hq": 64, "Hkv": 8, "x": "bf16", "theta": 500000.0, "lens": 5},
        # one request decoding at a short context (2B4T heads)
        {"name": "attn_decode_one", "op": "attn", "B": 1, "new_max": 1, "ctx_max": 700, "ragged": False, "page": 16, "Hq": 20, "Hkv": 5, "lens": 6},
        # a decode batch at the 70B shape, contexts from a few tokens to 8192
        {"name": "attn_decode_64", "op": "attn", "B": 64, "new_max": 1, "ctx_max": 8192, "ragged": True, "page": 64, "Hq": 64, "Hkv": 8, "lens": 7},
        # one prompt's chunk behind a cached prefix (2B4T heads)
        {"name": "attn_chunk_500", "op": "attn", "B": 1, "new_max": 500, "ctx_max": 4096, "ragged": False, "page": 16, "Hq": 20, "Hkv": 5, "lens": 8},
        # chunks of several prompts in one step at the 70B shape, ragged in both lengths
        {"name": "attn_chunks_4", "op": "attn", "B": 4, "new_max": 2048, "ctx_max": 8192, "ragged": True, "page": 32, "Hq": 64, "Hkv": 8, "lens": 9},
    ]


HEADS = [(20, 5), (64, 8), (8, 8), (40, 8), (32, 8), (16, 1), (12, 4)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "norm", "norm", "rope", "attn", "attn", "attn"])
    lens = rng.randrange(1 << 20)
    if op == "norm":
        K = rng.choice([128 * _log(rng, 1, 64), 8 * _log(rng, 1, 1024), _log(rng, 1, 8192)])
        T = min(_log(rng, 1, 8192), max(1, (1 << 25) // K))
        return {"op": op, "T": T, "K": K, "x": rng.choice(["bf16", "f32"]), "res": rng.choice(["bf16", "f32"])}
    page = rng.choice([16, 32, 64, 128])
    Hq, Hkv = rng.choice(HEADS)
    B = _log(rng, 1, 256 if op == "plan" else 64)
    new_max = rng.choice([1, _log(rng, 1, 2048)])
    ctx_max = _log(rng, 1, 8192)
    c = {"op": op, "B": B, "new_max": new_max, "ctx_max": ctx_max, "ragged": rng.random() < 0.7, "page": page, "lens": lens}
    if op == "plan":
        c["new_max"] = min(new_max, max(1, 65536 // B))
    elif op == "rope":
        c["B"] = max(1, min(B, 8192 // new_max))
        c |= {"Hq": Hq, "Hkv": Hkv, "x": rng.choice(["bf16", "f32"]), "theta": rng.choice([10000.0, 500000.0])}
    else:
        rows = (new_max + ctx_max) * max(new_max * Hq / 64, Hkv)  # products of scores, rows of the cache
        c["B"] = max(1, min(B, int(4 * 2048 * 8192 / rows)))
        c |= {"Hq": Hq, "Hkv": Hkv}
    return c


def lengths(case):
    """The requests' new and cached token counts: they belong to the case, not to the seed."""
    B, r = case["B"], random.Random(case["lens"])
    if not case["ragged"]:
        return [case["new_max"]] * B, [case["ctx_max"]] * B
    new = [max(1, int(case["new_max"] * r.random() + 1)) for _ in range(B)]
    ctx = [int((case["ctx_max"] + 1) * r.random()) for _ in range(B)]
    new[r.randrange(B)] = case["new_max"]
    ctx[r.randrange(B)] = case["ctx_max"]
    return [min(n, case["new_max"]) for n in new], [min(c, case["ctx_max"]) for c in ctx]


def _pages(n, page):
    return (n + page - 1) // page


# ------------------------------------------------------------------------------- inputs

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    if case["op"] == "norm":
        # a residual stream of a few units with some large channels, a sublayer's output, gains near one
        T, K = case["T"], case["K"]
        res = randn(T, K) * 2.0
        wide = torch.randperm(K, generator=g, device=dev)[: max(1, K // 100)]
        res[:, wide] *= 10.0
        return {"op": "norm", "x": randn(T, K, dtype=DTYPE[case["x"]]), "res": res.to(DTYPE[case["res"]]), "gain": 1.0 + 0.1 * randn(K)}

    new, ctx = lengths(case)
    B, P, T = case["B"], case["page"], sum(new)
    width = max(_pages(n + c, P) for n, c in zip(new, ctx))
    used = sum(_pages(n + c, P) for n, c in zip(new, ctx))
    pool = used + used // 8 + 2
    pages = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    new_t, ctx_t = (torch.tensor(v, dtype=torch.int32, device=dev) for v in (new, ctx))

    if case["op"] == "plan":
        old = [_pages(c, P) for c in ctx]
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        have = torch.arange(width, device=dev)[None, :] < torch.tensor(old, device=dev)[:, None]
        table[have] = pages[: sum(old)]
        free = pages.roll(-sum(old))  # the free pages first, then entries that are not free
        n_free = torch.tensor([pool - sum(old)], dtype=torch.int32, device=dev)
        return {"op": "plan", "new": new_t, "ctx": ctx_t, "table": table, "free": free, "n_free": n_free, "page": P, "T": T}

    # the plan of such a step, already made
    kv = new_t + ctx_t
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), torch.cumsum(new_t, 0).to(torch.int32)])
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    have = torch.arange(width, device=dev)[None, :] < ((kv + P - 1) // P)[:, None]
    table[have] = pages[:used]
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        t = torch.arange(T, device=dev)
        s = torch.searchsorted(cu[1:].long(), t, right=True)
        pos = ctx_t[s].long() + t - cu[s].long()
        slots = table[s, pos // P].long() * P + pos % P
        dt = DTYPE[case["x"]]
        return {"op": "rope", "q": randn(T, Hq, D, dtype=dt), "k": randn(T, Hkv, D, dtype=dt), "v": randn(T, Hkv, D, dtype=dt),
                "pos": pos.to(torch.int32), "slots": slots.to(torch.int32), "theta": case["theta"],
                "kp": randn(pool, Hkv, P, D, dtype=torch.bfloat16), "vp": randn(pool, Hkv, P, D, dtype=torch.bfloat16)}
    # scores of a few units, values with a mean of their own in each dimension
    q = (1.5 * randn(T, Hq, D)).to(torch.bfloat16)
    vp = randn(pool, Hkv, P, D) + randn(1, Hkv, 1, D)
    return {"op": "attn", "q": q, "kp": randn(pool, Hkv, P, D, dtype=torch.bfloat16), "vp": vp.to(torch.bfloat16),
            "table": table, "cu": cu, "kv": kv, "new_max": max(new)}


# ------------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[state["op"]](state)


def _own(s):
    import ternary_bitlinear_quantized_b200 as tb
    if s["op"] == "plan":
        cu, kv, pos, slots, n_free = tb.paged_plan(s["new"], s["ctx"], s["table"], s["free"], s["n_free"], s["page"], s["T"])
        return {"cu": cu, "kv": kv, "pos": pos, "slots": slots, "n_free": n_free, "table": s["table"]}
    if s["op"] == "norm":
        res, q, sx, sum_q = tb.add_rmsnorm_quant_act(s["x"], s["res"], s["gain"], EPS)
        return {"res": res, "q": q, "s": sx, "sum": sum_q}
    if s["op"] == "rope":
        q = tb.rope_paged_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["theta"], s["kp"], s["vp"])
        return {"q": q, "kp": s["kp"], "vp": s["vp"]}
    return tb.attention_paged(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["kv"], s["new_max"])


def _plain_plan(s):
    new, ctx, P, T = s["new"].long(), s["ctx"].long(), s["page"], s["T"]
    dev = new.device
    kv = new + ctx
    old = (ctx + P - 1) // P
    need = (kv + P - 1) // P - old
    start = torch.cumsum(need, 0) - need
    n_free = s["n_free"].long()
    # a request's j-th new page is the free list's entry n_free - 1 - (start + j)
    col = torch.arange(s["table"].shape[1], device=dev)[None, :]
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    at = (n_free - 1 - (start[:, None] + col - old[:, None])).clamp(0, s["free"].shape[0] - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[r] + t - cu[r]
    slots = s["table"][r, pos // P].long() * P + pos % P
    i32 = torch.int32
    return {"cu": cu.to(i32), "kv": kv.to(i32), "pos": pos.to(i32), "slots": slots.to(i32), "n_free": (n_free - need.sum()).to(i32), "table": s["table"]}


def _plain_norm(s):
    # The codes are whole numbers (they enter an integer product) and lie next to rounding borders:
    # every step is one fp32 operation, with the mean of the squares summed in 64 bits and rounded once.
    res = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    h = res.float()
    ms = h.double().square().mean(-1, keepdim=True).float()
    inv = 1.0 / torch.sqrt(ms + EPS)
    y = (h * inv) * s["gain"]
    top = y.abs().amax(-1, keepdim=True).clamp_min(1e-5)
    sx = torch.full_like(top, 127.0) / top  # one division: 127.0 / top would be two roundings
    q = torch.round(y * sx).clamp(-128, 127)
    return {"res": res, "q": q.to(torch.int8), "s": sx[:, 0], "sum": q.to(torch.int32).sum(-1, dtype=torch.int32)}


def _plain_rope(s):
    half = D // 2
    i = torch.arange(half, device=s["q"].device, dtype=torch.float64)
    a = s["pos"].double()[:, None] * s["theta"] ** (-2.0 * i / D)
    c, sn = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]

    def turn(x):
        x1, x2 = x[..., :half].float(), x[..., half:].float()
        return torch.cat([x1 * c - x2 * sn, x2 * c + x1 * sn], -1).to(torch.bfloat16)

    P = s["kp"].shape[2]
    page, row = s["slots"].long() // P, s["slots"].long() % P
    s["kp"][page, :, row] = turn(s["k"])
    s["vp"][page, :, row] = s["v"].to(torch.bfloat16)
    return {"q": turn(s["q"]), "kp": s["kp"], "vp": s["vp"]}


def _plain_attn(s):
    q, kp, vp, table, cu, kv, N = s["q"], s["kp"], s["vp"], s["table"], s["cu"].long(), s["kv"].long(), s["new_max"]
    (T, Hq, _), (pool, Hkv, P, _) = q.shape, kp.shape
    B, W = table.shape
    G, dev = Hq // Hkv, q.device
    # each request's pages in a row, and its new tokens padded to the longest
    at = table.long().clamp_min(0)
    K = kp[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * P, D).float()
    V = vp[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * P, D).float()
    n = torch.arange(N, device=dev)
    new = cu[1:] - cu[:-1]
    there = n[None, :] < new[:, None]  # [B, N]
    src = (cu[:-1, None] + n[None, :]).clamp_max(T - 1)
    Q = q[src].reshape(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D).float()
    S = (Q @ K.transpose(-1, -2)).view(B, Hkv, G, N, W * P).mul_(1.0 / math.sqrt(D))
    last = (kv - new)[:, None] + n[None, :]  # the last position that a token sees
    far = torch.arange(W * P, device=dev)[None, None, :] > last[:, :, None]
    S.masked_fill_(far[:, None, None], -math.inf)
    S.sub_(S.amax(-1, keepdim=True)).exp_()
    total = S.sum(-1, keepdim=True)
    # rows behind a request's length hold anything: they count for nothing
    V = torch.where((torch.arange(W * P, device=dev)[None, :] < kv[:, None])[:, None, :, None], V, 0.0)
    O = (S.view(B, Hkv, G * N, W * P) @ V).view(B, Hkv, G, N, D).div_(total)
    return O.permute(0, 3, 1, 2, 4)[there].reshape(T, Hq, D).to(torch.bfloat16)


# ------------------------------------------------------------------------------- the work

def work(case):
    if case["op"] == "norm":
        T, K, bx, br = case["T"], case["K"], 2 if case["x"] == "bf16" else 4, 2 if case["res"] == "bf16" else 4
        return {"bytes": T * K * (bx + 2 * br + 1) + 4 * K + 8 * T, "flops": 8 * T * K}
    new, ctx = lengths(case)
    B, P, T = case["B"], case["page"], sum(new)
    fresh = sum(_pages(n + c, P) - _pages(c, P) for n, c in zip(new, ctx))
    if case["op"] == "plan":
        # lengths, free entries, one table entry a token in; lengths, new entries, positions and slots out
        return {"bytes": 4 * (4 * B + 2 + 2 * fresh + T + 2 * T), "flops": 6 * T + 8 * B}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        bx = 2 if case["x"] == "bf16" else 4
        return {"bytes": T * D * (Hq + 2 * Hkv) * (bx + 2) + 8 * T, "flops": 3 * T * D * (Hq + Hkv)}
    rows = sum(n + c for n, c in zip(new, ctx))
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    table = sum(_pages(n + c, P) for n, c in zip(new, ctx))
    return {"bytes": rows * Hkv * D * 4 + 4 * T * Hq * D + 4 * table + 8 * B, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "norm":
        total = s["x"].double() + s["res"].double()
        # the norm is taken of the stored stream, in its type; the codes are whole numbers
        h = total.to(s["res"].dtype).double()
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + EPS) * s["gain"].double()
        return {"res": total, "q": None, "s": 127.0 / y.abs().max(-1).values.clamp_min(1e-5), "sum": None}
    if case["op"] == "rope":
        freq = torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=s["q"].device), -torch.arange(0, D, 2, device=s["q"].device).double() / D)
        e = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device), torch.outer(s["pos"].double(), freq))

        def turn(x):
            z = torch.complex(x[..., : D // 2].double(), x[..., D // 2:].double()) * e[:, None]
            return torch.cat([z.real, z.imag], -1)

        kp, vp = (s[c].double().transpose(1, 2).reshape(-1, case["Hkv"], D) for c in ("kp", "vp"))
        kp[s["slots"].long()], vp[s["slots"].long()] = turn(s["k"]), s["v"].double()
        back = lambda c: c.view(-1, case["page"], case["Hkv"], D).transpose(1, 2).contiguous()  # noqa: E731
        return {"q": turn(s["q"]), "kp": back(kp), "vp": back(vp)}
    new, ctx = lengths(case)
    G, out, t0 = case["Hq"] // case["Hkv"], [], 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][b, : _pages(n + c, case["page"])].long()
        o = torch.empty(n, case["Hq"], D, dtype=torch.float64, device=s["q"].device)
        sees = torch.ones(n, n + c, dtype=torch.bool, device=s["q"].device).tril(c)
        for h in range(case["Hkv"]):
            K, V = (s[x][pages, h].reshape(-1, D)[: n + c].double() for x in ("kp", "vp"))
            Q = s["q"][t0: t0 + n, h * G: (h + 1) * G].double()
            w = torch.einsum("tgd,ld->tgl", Q, K) / math.sqrt(D)
            w = torch.softmax(w.masked_fill(~sees[:, None], -math.inf), -1)
            o[:, h * G: (h + 1) * G] = torch.einsum("tgl,ld->tgd", w, V)
        out.append(o)
        t0 += n
    return torch.cat(out)
