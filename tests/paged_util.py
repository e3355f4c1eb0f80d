"""Plain forms of the paged serving step for its tests: loops over requests and tokens, 64 bits."""
from __future__ import annotations

import math

import torch

D = 128


def pages_of(n: int, P: int) -> int:
    return (n + P - 1) // P


def plan_ref(new, ctx, table, free, n_free, P, T):
    """Token by token: (cu, kv, positions, slots, n_free_out, table), lists; for valid lengths."""
    table, cu, kv, pos, slots, left = [list(r) for r in table], [0], [], [], [], n_free
    for i, (n, c) in enumerate(zip(new, ctx)):
        for j in range(pages_of(c, P), pages_of(c + n, P)):
            left -= 1
            table[i][j] = free[left] if left >= 0 else -1
        for t in range(n):
            page = table[i][(c + t) // P]
            pos.append(c + t)
            slots.append(page * P + (c + t) % P if page >= 0 else -1)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = T - len(pos)
    return cu, kv, pos + [0] * pad, slots + [-1] * pad, left, table


class Batch:
    """Requests with their pages in random places of a pool; what no request sees holds NaN."""

    def __init__(self, new, kv, Hq, Hkv, P, seed=0, pad=0, spare=3, device="cuda", nan=True, width_extra=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kvl, self.P, self.Hq, self.Hkv = list(new), list(kv), P, Hq, Hkv
        B, n = len(new), [pages_of(k, P) for k in kv]
        pool = sum(n) + spare
        order = torch.randperm(pool, generator=g)
        self.width = max(n + [1]) + width_extra
        table = torch.full((B, self.width), 0x7FFFFFFF if nan else 0, dtype=torch.int32)  # unused entries: no page
        T = sum(new) + pad
        self.q = (1.5 * torch.randn(T, Hq, D, generator=g)).bfloat16().to(device)
        kp, vp = torch.randn(pool, Hkv, P, D, generator=g), torch.randn(pool, Hkv, P, D, generator=g) + 0.5
        fill = float("nan") if nan else 0.0
        o, seen = 0, torch.zeros(pool, P, dtype=torch.bool)
        for i in range(B):
            table[i, : n[i]] = order[o: o + n[i]].int()
            for j in range(n[i]):
                seen[order[o + j], : min(P, kv[i] - j * P)] = True
            o += n[i]
        kp.masked_fill_(~seen[:, None, :, None], fill)
        vp.masked_fill_(~seen[:, None, :, None], fill)
        self.kp, self.vp = kp.bfloat16().to(device), vp.bfloat16().to(device)
        self.table = table.to(device)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv = torch.tensor(self.kvl, dtype=torch.int32, device=device)
        self.max_new = max(list(new) + [0])


def attention_ref(b: Batch):
    """(out, bound without the output's rounding and the probabilities' one, sum of weights times |v|), all fp64
    [T, Hq, 128]; rows behind the last request are NaN.

    The bound counts, relative to sum w |v| of the element (A):
      scores     8 tensor instructions of 16 products each, every one off by at most 2^-22 of what it has
                 summed in absolute value, s_abs = sum |q k| / sqrt(128): 8 * 2^-22 * s_abs, two more fp32 roundings
                 of the score (2^-23 |s|), entering numerator and denominator: twice
      exp        2^-22 relative by its documented error, twice; and the subtraction before it, 2^-24 |s|
      sums       kv / 16 accumulation steps at 2^-22 each, and joins (64 at most here) at 2^-22
    """
    G = b.Hq // b.Hkv
    out = torch.full((b.q.shape[0], b.Hq, D), float("nan"), dtype=torch.float64, device=b.q.device)
    bound, absum = torch.zeros_like(out), torch.zeros_like(out)
    t0 = 0
    for i, (n, kv) in enumerate(zip(b.new, b.kvl)):
        pages = b.table[i, : pages_of(kv, b.P)].long()
        for h in range(b.Hkv):
            K = b.kp[pages, h].reshape(-1, D)[:kv].double()
            V = b.vp[pages, h].reshape(-1, D)[:kv].double()
            for t in range(0, n, 64):
                rows = torch.arange(t, min(t + 64, n), device=b.q.device)
                Q = b.q[t0 + rows, h * G: (h + 1) * G].double()
                s = torch.einsum("tgd,ld->tgl", Q, K) / math.sqrt(D)
                sees = torch.arange(kv, device=b.q.device)[None, :] <= (kv - n + rows)[:, None]
                s = s.masked_fill(~sees[:, None], -math.inf)
                w = torch.softmax(s, -1) if kv else s
                w = torch.nan_to_num(w, nan=0.0)  # a row that sees nothing: zeros
                o = torch.einsum("tgl,ld->tgd", w, V)
                A = torch.einsum("tgl,ld->tgd", w, V.abs())
                s_abs = torch.einsum("tgd,ld->tgl", Q.abs(), K.abs()).amax(-1, keepdim=True) / math.sqrt(D) if kv else 0.0
                rel = 2 * (8 * 2.0 ** -22 * s_abs + 2.0 ** -22 * s_abs + 2.0 ** -22) + (kv / 16 + 64) * 2.0 ** -22
                out[t0 + rows, h * G: (h + 1) * G] = o
                bound[t0 + rows, h * G: (h + 1) * G] = A * rel
                absum[t0 + rows, h * G: (h + 1) * G] = A
        t0 += n
    return out, bound, absum


def weight_step(b: Batch) -> float:
    """Half a step of the weights in the second product, as the call's documentation has it: two bf16 (2^-8 of 2^-8)
    up to 32 query rows per request and key/value head, one bf16 above."""
    return 2.0 ** -16 if b.max_new * (b.Hq // b.Hkv) <= 32 else 2.0 ** -8


def check_attention(b: Batch, got: torch.Tensor, p_round: float = 2.0 ** -8, skip=()):
    """`skip`: requests that are not looked at.  `p_round`: rounding of a probability before the second product (a bf16's half step; 2^-16 where it enters
    as the sum of two bf16).  Rows behind the last request are not looked at."""
    ref, bound, A = attention_ref(b)
    T = sum(b.new)
    tol = bound + A * p_round
    if got.dtype == torch.bfloat16:
        tol = tol + (ref.abs() + tol) * 2.0 ** -8
    err = (got.double() - ref).abs()[:T]
    bad = ~(err <= tol[:T])
    for i in skip:
        bad[sum(b.new[:i]): sum(b.new[: i + 1])] = False
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / tol[:T].clamp_min(1e-300)).max())} of the bound"
