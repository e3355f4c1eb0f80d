"""The paged serving step on the GPU: plan, residual add + norm + codes, rotary embedding + append and
attention against plain 64-bit forms, at the lengths, pages and masks where they can go wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ternary_bitlinear_quantized_b200 as tb
from oracle import bitnet_oracle as O
from tests.paged_util import D, Batch, attention_ref, check_attention, pages_of, plan_ref, weight_step
from tests.parity_util import act_to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------- plan

def _plan_inputs(new, ctx, P, extra_free=5, width_extra=2, seed=0):
    g = torch.Generator().manual_seed(seed)
    old = [pages_of(c, P) for c in ctx]
    need = sum(pages_of(n + c, P) for n, c in zip(new, ctx)) - sum(old)
    width = max([pages_of(n + c, P) for n, c in zip(new, ctx)] + [1]) + width_extra
    ids = torch.randperm(sum(old) + need + extra_free, generator=g).tolist()
    table, o = [], 0
    for k in old:
        table.append(ids[o: o + k] + [-7] * (width - k))
        o += k
    return table, ids[o:], width


def _run_plan(new, ctx, table, free, n_free, P, T, tail=3):
    tab = torch.tensor(table, **I32).reshape(len(new), -1)
    fr = torch.tensor(list(free) + [-99] * tail, **I32)
    out = tb.paged_plan(torch.tensor(new, **I32), torch.tensor(ctx, **I32), tab, fr, torch.tensor([n_free], **I32), P, T)
    torch.cuda.synchronize()
    return [o.tolist() for o in out], tab.tolist()


@pytest.mark.parametrize("B,P,new_max,ctx_max,pad", [(1, 16, 1, 700, 0), (1, 16, 1, 0, 0), (3, 32, 40, 100, 7), (7, 64, 1, 64, 0),
                                                     (256, 16, 1, 3000, 0), (257, 128, 3, 500, 1000), (1000, 16, 20, 40, 1),
                                                     (4096, 256, 2, 300, 0), (2, 16, 5000, 33, 0)])
def test_plan(B, P, new_max, ctx_max, pad):
    r = np.random.RandomState(B + P)
    new, ctx = r.randint(0, new_max + 1, B).tolist(), r.randint(0, ctx_max + 1, B).tolist()
    new[0], ctx[-1] = new_max, ctx_max // P * P  # a context that ends with its page
    table, free, _ = _plan_inputs(new, ctx, P)
    T = sum(new) + pad
    (cu, kv, pos, slots, left), tab = _run_plan(new, ctx, table, free, len(free), P, T)
    want = plan_ref(new, ctx, table, free, len(free), P, T)
    assert (cu, kv, pos, slots, left[0], tab) == want
    assert tb.device_status() == 0


def test_plan_outputs_are_tensors_of_their_own():
    """Parts of one allocation: ordinary tensors for torch, alive as long as any of them is."""
    new, ctx = torch.tensor([3, 1], **I32), torch.tensor([0, 16], **I32)
    table = torch.tensor([[-1, -1], [4, -1]], **I32)
    free, n = torch.arange(4, **I32), torch.tensor([4], **I32)
    cu, kv, pos, slots, left = tb.paged_plan(new, ctx, table, free, n, 16, 5)
    assert [tuple(t.shape) for t in (cu, kv, pos, slots, left)] == [(3,), (2,), (5,), (5,), (1,)]
    assert all(t.is_contiguous() and t.dtype == torch.int32 for t in (cu, kv, pos, slots, left))
    n.copy_(left)
    ctx.copy_(kv)
    del cu, kv, left
    junk = [torch.full((64,), -5, **I32) for _ in range(20)]
    assert pos.tolist() == [0, 1, 2, 16, 0] and (slots + 1).tolist() == [49, 50, 51, 33, 0] and pos.clone().sum() == 19
    assert n.item() == 2 and ctx.tolist() == [3, 17] and len(junk) == 20
    res, q, s, sq = tb.add_rmsnorm_quant_act(torch.ones(3, 64, device=DEV), torch.ones(3, 64, device=DEV), None)
    assert s.data_ptr() % 16 == 0 and sq.data_ptr() % 16 == 0 and s.dtype == torch.float32 and sq.dtype == torch.int32
    s.mul_(2)
    assert sq.tolist() == [64 * 127] * 3 and s.tolist() == [127.0] * 3


def test_plan_takes_the_top_of_the_list_only():
    new, ctx, P = [17, 0, 1], [0, 5, 16], 16
    table, free, _ = _plan_inputs(new, ctx, P, extra_free=9)
    (_, _, _, _, left), tab = _run_plan(new, ctx, table, free, len(free), P, 18)
    assert left == [len(free) - 3]
    assert tab[0][:2] == [free[-1], free[-2]] and tab[2][1] == free[-3] and tab[1][1] == -7


def test_plan_without_enough_pages():
    new, ctx, P = [20, 20, 20], [0, 0, 0], 16
    table, free, _ = _plan_inputs(new, ctx, P)
    want = plan_ref(new, ctx, table, free, 3, P, 60)
    (cu, kv, pos, slots, left), tab = _run_plan(new, ctx, table, free, 3, P, 60)
    assert (cu, kv, pos, slots, left[0], tab) == want and left[0] == -3
    assert tb.device_status() == 0


def test_plan_of_no_requests_and_no_tokens():
    none = torch.empty(0, **I32)
    out = tb.paged_plan(none, none, torch.empty(0, 2, **I32), torch.tensor([4], **I32), torch.tensor([1], **I32), 16, 3)
    cu, kv, pos, slots, left = [o.tolist() for o in out]
    assert cu == [0] and kv == [] and pos == [0, 0, 0] and slots == [-1, -1, -1] and left == [1]
    (cu, kv, pos, slots, left), _ = _run_plan([0], [5], [[3, -7]], [4], 1, 16, 0)
    assert cu == [0, 0] and kv == [5] and left == [1] and tb.device_status() == 0


def test_plan_flags_lengths_out_of_range():
    P = 16
    # request 1 exceeds its row of the table, request 2 has a negative length: neither gets pages
    new, ctx = [3, 40, -2, 4], [10, 10, 5, 16]
    table = [[0, -7, -7], [1, -7, -7], [2, -7, -7], [3, -7, -7]]
    (cu, kv, pos, slots, left), tab = _run_plan(new, ctx, table, [9, 8, 7], 3, P, 47)
    assert cu == [0, 3, 43, 43, 47] and kv == [13, 10, 5, 20] and left == [2]
    assert slots[:3] == [10, 11, 12] and slots[3:43] == [-1] * 40 and slots[43:] == [7 * 16 + i for i in range(4)]
    assert tab == [[0, -7, -7], [1, -7, -7], [2, -7, -7], [3, 7, -7]]
    assert tb.device_status() == 8
    # more new tokens than the step has room for
    (cu, _, pos, slots, _), _ = _run_plan([5, 5], [0, 0], [[-7], [-7]], [9, 8, 7], 3, P, 6)
    assert cu == [0, 5, 6] and pos == [0, 1, 2, 3, 4, 0] and tb.device_status() == 8
    # a count of free pages outside the list, page ids whose slots would pass 32 bits
    (_, _, _, slots, left), _ = _run_plan([1], [0], [[-7]], [5], 99, P, 1)
    assert slots == [-1] and left == [-1] and tb.device_status() == 8
    (_, _, _, slots, _), _ = _run_plan([1], [0], [[-7]], [1 << 28], 1, P, 1, tail=0)
    assert slots == [-1] and tb.device_status() == 8
    assert tb.device_status() == 0


# ------------------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (2, 57), (5, 128), (1, 2560), (300, 640), (7, 5120), (4, 8192), (3, 8200),
                                 (2, 12289), (2, 49152), (257, 2048),
                                 (3, 12288), (300, 1023), (300, 1025), (600, 3001), (2, 8191), (300, 8185), (300, 8186), (3, 16377), (3, 16378), (2, 16384), (9, 249), (9, 250)])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
def test_add_rmsnorm_quant_act(T, K, xt, rt):
    g = torch.Generator().manual_seed(T * 100 + K)
    x, r = torch.randn(T, K, generator=g).to(xt), (3 * torch.randn(T, K, generator=g)).to(rt)
    gain = 1.0 + 0.1 * torch.randn(K, generator=g)
    for gn in (gain, None):
        res, q, s, sq = tb.add_rmsnorm_quant_act(x.to(DEV), r.to(DEV), None if gn is None else gn.to(DEV), 1e-6)
        torch.cuda.synchronize()
        want = (x.float() + r.float()).to(rt)
        assert torch.equal(res.cpu(), want)
        oq, os_, osq = O.rmsnorm_quant_act(act_to_np(want), None if gn is None else gn.numpy(), 1e-6)
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_) and np.array_equal(sq.cpu().numpy(), osq)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [12224, 12288, 12296])
def test_rmsnorm_quant_act_rows_of_48_kb(K, dt):
    """A row of 48 KB in shared memory, beside the kernel's own few bytes."""
    x = torch.randn(3, K, generator=torch.Generator().manual_seed(K)).to(dt)
    q, s, sq = tb.rmsnorm_quant_act(x.to(DEV), None)
    oq, os_, osq = O.rmsnorm_quant_act(act_to_np(x), None, 1e-6)
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_) and np.array_equal(sq.cpu().numpy(), osq)


def test_add_rmsnorm_quant_act_in_place_and_zero_rows():
    x = torch.randn(9, 640, device=DEV).bfloat16()
    r = torch.randn(9, 640, device=DEV).bfloat16()
    x[4], r[4] = 0, 0
    want = (x.float() + r.float()).bfloat16()
    fresh = tb.add_rmsnorm_quant_act(x, r, None)
    got = tb.add_rmsnorm_quant_act(x, r, None, residual_out=r)
    assert got[0].data_ptr() == r.data_ptr() and torch.equal(r, want)
    for a, b in zip(fresh, got):
        assert torch.equal(a, b)
    assert not got[1][4].any() and got[3][4] == 0
    assert tb.add_rmsnorm_quant_act(x[:0], r[:0], None)[0].shape == (0, 640)


@pytest.mark.parametrize("K", [640, 2047, 5120, 8200])
def test_add_rmsnorm_quant_act_non_finite(K):
    """Rows with NaN and infinities, large sums, an infinite or NaN gain and eps = 0 on a zero row: what rmsnorm_quant_act
    gives for the same stream."""
    g = torch.Generator().manual_seed(K)
    x = torch.zeros(9, K)
    r = torch.randn(9, K, generator=g)
    r[0, 3], r[1, 5], r[2, 7] = float("nan"), float("inf"), -float("inf")
    r[3, 1], r[3, 2] = float("inf"), -float("inf")
    r[4] = 3e38
    r[5] = 0
    gain = 1.0 + 0.1 * torch.randn(K, generator=g)
    odd = gain.clone()
    odd[2], odd[4] = float("inf"), float("nan")
    for gn, eps in ((gain, 1e-6), (odd, 1e-6), (gain, 0.0), (None, 1e-6)):
        gd = None if gn is None else gn.to(DEV)
        res, *got = tb.add_rmsnorm_quant_act(x.to(DEV), r.to(DEV), gd, eps)
        assert torch.equal(torch.nan_to_num(res), torch.nan_to_num(r.to(DEV)))
        for a, b in zip(got, tb.rmsnorm_quant_act(res, gd, eps)):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


# ------------------------------------------------------------------------------------------- rope

@pytest.mark.parametrize("T,Hq,Hkv,P,theta", [(1, 20, 5, 16, 10000.0), (4, 64, 8, 32, 500000.0), (5, 8, 8, 256, 10000.0),
                                              (37, 12, 4, 64, 10000.0), (130, 16, 1, 128, 500000.0),
                                              (1701, 20, 5, 32, 10000.0)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rope_paged_append(T, Hq, Hkv, P, theta, dt):
    g = torch.Generator().manual_seed(T)
    n_pages = pages_of(2 * T, P) + 1
    q, k, v = (torch.randn(T, h, D, generator=g).to(dt) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(n_pages * P, generator=g)[:T].int()
    pos = torch.randint(0, 70000, (T,), generator=g).int()
    pos[0] = 0
    if T > 2:
        slots[1], pos[2] = -1, 1 << 30  # a padded token; a position far out
    kc, vc = (torch.randn(n_pages, Hkv, P, D, generator=g).bfloat16() for _ in range(2))
    kp, vp = kc.to(DEV), vc.to(DEV)
    q_rot = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
    tb.rope_paged_append(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), theta, kp, vp, q_rot=q_rot)
    torch.cuda.synchronize()
    i = torch.arange(D // 2, dtype=torch.float64)
    a = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64) ** (-2.0 * i / D)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]

    def turn(x):
        x1, x2 = x[..., :64].double(), x[..., 64:].double()
        # beside the bf16's half step: sine and cosine off by an ulp or two and the angle's own rounding to fp32
        # (half a turn's 2^-24), and by 2^-53 of the turns counted, on this side and the other; three fp32 roundings
        size = (x1.abs() + x2.abs()) * (10 * 2.0 ** -24 + 4 * 2.0 ** -53 * a.abs()[:, None])
        return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1), torch.cat([size, size], -1)

    live = slots >= 0
    want, size = turn(q)
    got = q_rot.cpu().double()
    assert ((got - want).abs() <= 2.0 ** -8 * (want.abs() + size) + size)[live].all()
    assert (got[~live] == 77.0).all()
    want, size = turn(k)
    wk, wv = kc.double(), vc.clone()
    tol = torch.zeros_like(wk)
    for t in range(T):
        if slots[t] >= 0:
            p, r = int(slots[t]) // P, int(slots[t]) % P
            wk[p, :, r], tol[p, :, r] = want[t], 2.0 ** -8 * (want[t].abs() + size[t]) + size[t]
            wv[p, :, r] = v[t].bfloat16()
    assert ((kp.cpu().double() - wk).abs() <= tol).all()
    assert torch.equal(vp.cpu(), wv)
    assert tb.device_status() == 0


def test_rope_paged_append_skips_slots_out_of_range():
    q, k, v = (torch.randn(3, h, D, device=DEV) for h in (4, 2, 2))
    kp, vp = torch.zeros(2, 2, 16, D, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 16, D, dtype=torch.bfloat16, device=DEV)
    q_rot = torch.zeros(3, 4, D, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([32, 5, 0x7FFFFFFF], **I32)
    tb.rope_paged_append(q, k, v, torch.arange(3, **I32), slots, 1e4, kp, vp, q_rot=q_rot)
    assert tb.device_status() == 8 and tb.device_status() == 0
    assert torch.equal(vp[0, :, 5], v[1].bfloat16()) and int((vp != 0).any(-1).sum()) == 2 and int((kp != 0).any(-1).sum()) == 2
    assert not q_rot[0].any() and q_rot[1].any() and not q_rot[2].any()


# ------------------------------------------------------------------------------------------- attention

def _attend(b, out_dtype=torch.bfloat16, **kw):
    out = torch.full((b.q.shape[0], b.Hq, D), 77.0, dtype=out_dtype, device=DEV)
    got = tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, out=out, **kw)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    assert (got[sum(b.new):] == 77.0).all()  # rows behind the last request
    return got


# (new, kv, Hq, Hkv, P)
FEW = [
    ([1], [1], 20, 5, 16),
    ([1], [701], 20, 5, 16),
    ([1, 1, 1], [64, 65, 63], 64, 8, 64),
    ([1] * 9, [0, 1, 15, 16, 17, 127, 128, 129, 1000], 16, 1, 128),
    ([1, 0, 1, 0], [5, 77, 300, 0], 8, 8, 32),
    ([2, 4, 1], [2, 2, 90], 12, 4, 16),        # fewer rows than tokens: the first tokens see nothing
    ([3], [1000], 40, 8, 256),
    ([1] * 70, [(37 * i) % 400 for i in range(70)], 32, 8, 16),
    ([1] * 300, [(61 * i) % 90 for i in range(300)], 4, 2, 16),
    ([1], [5], 33, 1, 16),                     # more query heads per key/value head than a tile has rows
]


@pytest.mark.parametrize("case", FEW, ids=range(len(FEW)))
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attention_few_rows(case, out_dtype):
    new, kv, Hq, Hkv, P = case
    b = Batch(new, kv, Hq, Hkv, P, seed=len(new), pad=2)
    # 33 rows of one token (the last case) take the kernel for many rows, whose weights are one bf16: by the definition
    # o = sum w v / sum w, a half step of 2^-8 on each w moves o by at most 2^-8 sum w |v| / sum w
    check_attention(b, _attend(b, out_dtype), p_round=weight_step(b))
    assert tb.device_status() == 0


CHUNKS = [
    ([128], [128], 16, 1, 16),
    ([129], [129], 8, 8, 64),
    ([500], [4596], 20, 5, 16),
    ([257], [300], 64, 8, 32),
    ([31, 1, 200, 0, 77], [31, 900, 777, 40, 1077], 12, 4, 128),
    ([300, 5], [100, 3], 16, 4, 16),           # most tokens see nothing
    ([64, 64], [64, 2000], 40, 8, 256),
    ([700], [1400], 4, 4, 16),
    ([90], [90], 33, 1, 32),
    ([260, 1, 1], [513, 512, 1], 64, 8, 64),
    ([150], [0], 8, 2, 16),
]


@pytest.mark.parametrize("case", CHUNKS, ids=range(len(CHUNKS)))
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attention_chunks(case, out_dtype):
    new, kv, Hq, Hkv, P = case
    b = Batch(new, kv, Hq, Hkv, P, seed=sum(new), pad=3)
    got = _attend(b, out_dtype)
    check_attention(b, got)
    assert torch.equal(got, _attend(b, out_dtype))  # equal calls, equal bits
    assert tb.device_status() == 0


def test_attention_long_context():
    b = Batch([1, 2], [70001, 33000], 16, 2, 64, seed=3)
    check_attention(b, _attend(b, torch.float32), p_round=2.0 ** -16)
    b = Batch([130], [20000], 8, 2, 16, seed=4)
    check_attention(b, _attend(b, torch.float32))


@pytest.mark.parametrize("new", [1, 100])
def test_attention_far_pages(new):
    """Pages whose elements start behind 2^31."""
    Hq, Hkv, P, kv = 8, 8, 256, 700
    n_pages = (1 << 31) // (Hkv * P * D) + 6
    b = Batch([new], [kv], Hq, Hkv, P, spare=0, nan=False, width_extra=0)
    kp = torch.empty(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.empty(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    far = torch.tensor([[n_pages - 1, 2, n_pages - 3]], **I32)
    kp[far[0].long()], vp[far[0].long()] = b.kp[b.table[0].long()], b.vp[b.table[0].long()]
    near = _attend(b)
    b.kp, b.vp, b.table = kp, vp, far
    assert torch.equal(near, _attend(b))


@pytest.mark.parametrize("new", [1, 100])
def test_attention_flags_bad_pages_and_lengths(new):
    b = Batch([new] * 3, [400, 500, 600], 8, 2, 16, seed=1)
    good = _attend(b)
    for bad in (-1, b.kp.shape[0], 0x7FFFFFFF, -0x80000000):
        c = Batch([new] * 3, [400, 500, 600], 8, 2, 16, seed=1)
        c.table[1, 7] = bad
        got = _attend(c)
        assert tb.device_status() == 8
        assert torch.equal(got[:new], good[:new]) and torch.equal(got[2 * new:], good[2 * new:])
    # lengths that do not fit: the request is skipped, the others are answered.  Not bit for bit: the cuts lie at
    # equal shares of the batch's work, which is less without the skipped request, so sums are joined at other
    # places; what holds of any cut is the bound of check_attention.
    c = Batch([new] * 3, [400, 500, 600], 8, 2, 16, seed=1)
    for kv in (-5, c.width * 16 + 1, 0x7FFFFFFF):
        c.kv[1] = kv
        got = _attend(c)
        assert tb.device_status() == 8 and (got[new: 2 * new] == 77.0).all()
        check_attention(c, got, skip=(1,))
    c.kv[1] = 500
    for cu in ([0, new, 2 * new, 3 * new + 1], [0, new, 2 * new, new], [-1, new, 2 * new, 3 * new]):
        c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        got = _attend(c)
        assert tb.device_status() == 8
        check_attention(c, got, skip=(0, 2))
    c.cu.copy_(torch.tensor([0, new, 2 * new, 3 * new], dtype=torch.int32))
    c.max_new = new - 1 if new > 1 else 1
    if new > 1:
        assert (_attend(c) == 77.0).all() and tb.device_status() == 8
    assert tb.device_status() == 0


def test_attention_captured_and_replayed_on_new_lengths():
    """One graph of a step's plan, append and attention, replayed as the requests grow by a token each."""
    Hq, Hkv, P, B, theta = 8, 2, 16, 5, 1e4
    ctx0 = [0, 15, 16, 200, 31]
    n_pages, width = 60, 20
    g = torch.Generator().manual_seed(0)
    ctx = torch.tensor(ctx0, **I32)
    new = torch.ones(B, **I32)
    free = torch.randperm(n_pages, generator=g).int().to(DEV)
    table = torch.full((B, width), -1, **I32)
    n_free = torch.tensor([n_pages], **I32)
    kp = torch.full((n_pages, Hkv, P, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    # the requests' prompts go through the same calls
    T0 = sum(ctx0)
    hk, hv = torch.randn(T0, Hkv, D, device=DEV).bfloat16(), torch.randn(T0, Hkv, D, device=DEV).bfloat16()
    _, _, pos, slots, left = tb.paged_plan(ctx, torch.zeros_like(ctx), table, free, n_free, P, T0)
    tb.rope_paged_append(torch.zeros(T0, Hq, D, device=DEV).bfloat16(), hk, hv, pos, slots, theta, kp, vp)
    n_free.copy_(left)
    q, k, v = (torch.zeros(B, h, D, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv))
    out = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(tb.attention_paged_workspace_bytes(Hq, Hkv, 1), dtype=torch.uint8, device=DEV)
    kept = {}

    def step():
        cu, kv, pos, slots, left = tb.paged_plan(new, ctx, table, free, n_free, P, B)
        q_rot = tb.rope_paged_append(q, k, v, pos, slots, theta, kp, vp)
        tb.attention_paged(q_rot, kp, vp, table, cu, kv, 1, out=out, ws=ws)
        n_free.copy_(left)
        ctx.copy_(kv)
        kept.update(q_rot=q_rot, cu=cu, kv=kv)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n in range(40):
        for x, h in ((q, Hq), (k, Hkv), (v, Hkv)):
            x.copy_(torch.randn(B, h, D, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        b = Batch([1] * B, [c + n + 1 for c in ctx0], Hq, Hkv, P)
        b.q, b.kp, b.vp, b.table = kept["q_rot"], kp, vp, table
        assert kept["kv"].tolist() == b.kvl
        check_attention(b, out, p_round=2.0 ** -16)
    used = sum(pages_of(c + 40, P) for c in ctx0)
    assert int(n_free) == n_pages - used and tb.device_status() == 0


def test_attention_on_other_streams_with_workspaces_of_their_own():
    bs = [Batch([1] * 8, [50 * i + 1 for i in range(8)], 16, 4, 16, seed=1), Batch([200, 3], [900, 40], 16, 4, 32, seed=2)]
    alone = [_attend(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(10):
        outs = []
        for b, s in zip(bs, streams):
            s.wait_stream(torch.cuda.current_stream())
            ws = torch.empty(tb.attention_paged_workspace_bytes(16, 4, b.max_new), dtype=torch.uint8, device=DEV)
            outs.append((tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, ws=ws, stream=s), ws))
        torch.cuda.synchronize()
        for (o, _), a, b in zip(outs, alone, bs):
            assert torch.equal(o, a)


def test_attention_chunks_captured_and_replayed_on_new_lengths():
    """A graph of the kernel for many rows, replayed on lengths it was not captured with: one request, ragged ones, none,
    and a request whose lengths do not fit."""
    Hq, Hkv, P = 12, 4, 32
    b = Batch([150, 33, 1, 90], [150, 600, 40, 2000], Hq, Hkv, P, seed=11, pad=5)
    out = torch.zeros(b.q.shape, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(tb.attention_paged_workspace_bytes(Hq, Hkv, 280), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, 280, out=out, ws=ws)
    for new, kv in (([150, 33, 1, 90], [150, 600, 40, 2000]), ([0, 274, 0, 0], [150, 600, 40, 0]), ([1, 1, 1, 1], [2, 599, 33, 1999]),
                    ([0, 0, 0, 0], [150, 600, 40, 2000]), ([60, 100, 14, 100], [3, 601, 14, 1000])):
        c = Batch([150, 33, 1, 90], [150, 600, 40, 2000], Hq, Hkv, P, seed=11, pad=5)
        c.new, c.kvl = new, kv
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        b.kv.copy_(torch.tensor(kv, dtype=torch.int32))
        c.cu, c.kv = b.cu, b.kv
        if kv[1] == 601:  # one more row than the request's pages hold: a page id out of range, seen as zeros
            b.kv[1], c.kvl[1] = b.width * P + 1, 600
        out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        bad = kv[1] == 600 and int(b.kv[1]) != 600
        assert tb.device_status() == (8 if bad else 0)
        check_attention(c, out, skip=(1,) if bad else ())
        assert (out[sum(new):] == 77.0).all()
        if bad:
            assert (out[60:160] == 77.0).all()


@pytest.mark.parametrize("new,kv,Hq,Hkv,P", [([3], [70], 200, 1, 16), ([2, 1], [300, 9], 1024, 4, 32), ([1], [140], 1024, 1, 64),
                                             ([40], [50], 129, 1, 16)])
def test_attention_of_more_query_heads_than_a_block(new, kv, Hq, Hkv, P):
    b = Batch(new, kv, Hq, Hkv, P, seed=Hq)
    check_attention(b, _attend(b, torch.float32))
    assert tb.device_status() == 0


@pytest.mark.parametrize("new", [1, 130])
def test_attention_of_pages_that_requests_share(new):
    """A prefix held once: two requests name the same pages."""
    b = Batch([new, new], [640, 640], 8, 2, 64, seed=5, nan=False)
    b.table[1, :8] = b.table[0, :8]
    check_attention(b, _attend(b, torch.float32), p_round=weight_step(b))


def test_attention_on_growing_maxima():
    """Scores that grow along the cache by more than 2^8 in weight, so that the running maximum moves again and again."""
    for new in (1, 70):
        b = Batch([new], [900], 8, 2, 32, seed=6, nan=False)
        pages = b.table[0, : pages_of(900, 32)].long()
        ramp = torch.arange(pages.numel() * 32, device=DEV).view(-1, 1, 32, 1) / 8.0
        b.kp[pages] = (torch.sign(b.q[0, 0]) * ramp / D ** 0.5).bfloat16().expand(-1, 2, -1, -1)
        b.q = (0.1 * b.q + torch.sign(b.q[0, 0])).bfloat16()
        check_attention(b, _attend(b, torch.float32), p_round=weight_step(b))


def test_attention_wait_limit():
    """Waits cut to one cycle: the kernel for many rows gives up, says so, and the next call is right."""
    b = Batch([200, 3], [500, 90], 8, 2, 16, seed=8)
    try:
        tb.debug_set_wait_limit(1)
        tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new)
        torch.cuda.synchronize()
        assert tb.device_status() == 7
    finally:
        tb.debug_set_wait_limit(0)
    for _ in range(2):
        check_attention(b, _attend(b))
        assert tb.device_status() == 0


def test_calls_on_a_given_stream():
    """Outputs and workspaces that a call allocates belong to the stream it is given."""
    b = Batch([200, 3], [900, 40], 16, 4, 32, seed=2)
    x = torch.randn(600, 2560, device=DEV).bfloat16()
    want, norm = _attend(b), tb.add_rmsnorm_quant_act(x, x, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, stream=s) for _ in range(4)]
        got = tb.add_rmsnorm_quant_act(x, x, None, stream=s)
        junk = [torch.full((1 << 22,), 1.0, device=DEV) for _ in range(4)]  # on the current stream, meanwhile
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs) and all(torch.equal(p, q) for p, q in zip(got, norm))
        del junk


def test_attention_decode_agrees_with_the_contiguous_cache():
    """One request whose pages lie in order is the contiguous cache of attention_decode."""
    T, Hq, Hkv, P, kv = 3, 20, 5, 64, 830
    b = Batch([T], [kv], Hq, Hkv, P, nan=False)
    pages = b.table[0, : pages_of(kv, P)].long()
    kc, vc = (x[pages].transpose(0, 1).reshape(Hkv, -1, D).contiguous() for x in (b.kp, b.vp))
    want = tb.attention_decode(b.q.float(), kc, vc, kv - T, torch.float32)
    got = _attend(b, torch.float32)
    _, bound, A = attention_ref(b)
    assert ((got.double() - want.double()).abs() <= 2 * bound + A * 2.0 ** -15).all()


# ------------------------------------------------------------------------------------------- refusals

def _refused(status, fn, *args, **kw):
    """ValueError for what the binding checks, BitnetError with its status for what the library does."""
    with pytest.raises(ValueError if status is None else tb.BitnetError) as e:
        fn(*args, **kw)
    if status is not None:
        assert e.value.status == status


def test_refusals_of_the_binding():
    b = Batch([2, 1], [20, 33], 4, 2, 16)
    att = (b.q, b.kp, b.vp, b.table, b.cu, b.kv, 2)

    def swap(i, x):
        return (*att[:i], x, *att[i + 1:])

    _refused(None, tb.attention_paged, *swap(0, b.q.float()))
    _refused(None, tb.attention_paged, *swap(0, b.q.transpose(0, 1)))
    _refused(None, tb.attention_paged, *swap(0, b.q[0]))
    _refused(None, tb.attention_paged, *swap(1, b.kp[:, :1].contiguous()))
    _refused(None, tb.attention_paged, *swap(2, b.vp.float()))
    _refused(None, tb.attention_paged, *swap(3, b.table.long()))
    _refused(None, tb.attention_paged, *swap(3, b.table[:, ::2]))
    _refused(None, tb.attention_paged, *swap(4, b.cu[:-1]))
    _refused(None, tb.attention_paged, *swap(5, b.kv.cpu()))
    _refused(None, tb.attention_paged, *att, out_dtype=torch.float16)
    _refused(None, tb.attention_paged, *att, out=torch.empty(1, 4, D, device=DEV))
    _refused(2, tb.attention_paged, *swap(6, -1))
    _refused(5, tb.attention_paged, *att, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    _refused(3, tb.attention_paged, *att, ws=torch.empty(1 << 26, dtype=torch.uint8, device=DEV)[1:])
    k, v, pos, slots = b.q[:, :2].contiguous(), b.q[:, 2:].contiguous(), torch.zeros(3, **I32), torch.arange(3, **I32)
    rope = (b.q, k, v, pos, slots, 1e4, b.kp.clone(), b.vp.clone())
    _refused(None, tb.rope_paged_append, b.q, k.float(), *rope[2:])
    _refused(None, tb.rope_paged_append, b.q, k, v[:2], *rope[3:])
    _refused(None, tb.rope_paged_append, *rope[:3], pos[:2], *rope[4:])
    _refused(None, tb.rope_paged_append, *rope, q_rot=torch.empty(3, 4, D, device=DEV))
    _refused(2, tb.rope_paged_append, *rope[:5], 0.0, *rope[6:])
    _refused(2, tb.rope_paged_append, *rope[:6], b.kp[:, :, :8].contiguous(), b.vp[:, :, :8].contiguous())
    new, ctx, free, n = torch.ones(2, **I32), torch.zeros(2, **I32), torch.arange(4, **I32), torch.tensor([4], **I32)
    plan = (new, ctx, torch.full((2, 2), -1, **I32), free, n, 16, 2)
    outs = [torch.empty(s, **I32) for s in (3, 2, 2, 2, 1)]
    _refused(None, tb.paged_plan, *plan, out=(*outs[:4], n))
    _refused(None, tb.paged_plan, *plan, out=(outs[0], ctx, *outs[2:]))
    _refused(None, tb.paged_plan, *plan, out=(outs[0], outs[1], outs[2][:1], *outs[3:]))
    _refused(None, tb.paged_plan, new[:1], *plan[1:])
    _refused(2, tb.paged_plan, *plan[:5], 24, 2)
    _refused(2, tb.paged_plan, *plan[:6], -1)
    x = torch.ones(2, 64, device=DEV)
    _refused(None, tb.add_rmsnorm_quant_act, x, x.half(), None)
    _refused(None, tb.add_rmsnorm_quant_act, x, x[:1], None)
    _refused(None, tb.add_rmsnorm_quant_act, x, x.t().contiguous().t(), None)
    _refused(None, tb.add_rmsnorm_quant_act, x, x, x[0, :32])
    _refused(None, tb.add_rmsnorm_quant_act, x, x, None, residual_out=x.bfloat16())
    _refused(2, tb.add_rmsnorm_quant_act, x[:, :0].contiguous(), x[:, :0].contiguous(), None)
    y = torch.ones(129, device=DEV)[1:].view(2, 64)
    _refused(3, tb.add_rmsnorm_quant_act, y, x, None)
    assert tb.device_status() == 0
    check_attention(b, tb.attention_paged(*att), p_round=weight_step(b))


# ------------------------------------------------------------------------------------------- a block together

@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [40, 0, 333]), ([70, 1, 19, 0], [5, 400, 0, 64])])
def test_decoder_block_over_the_paged_cache(new, ctx):
    """residual + norm + codes -> q/k/v -> rotary + append -> attention -> o -> residual + norm + codes -> gate/up,
    as a serving step calls them, against the single steps' plain forms on the same codes."""
    H, Hq, Hkv, P, I, theta = 512, 4, 2, 16, 640, 1e4
    g = torch.Generator().manual_seed(7)
    T, B = sum(new), len(new)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)
    W = {n: tb.pack_i2s(0.02 * rnd(*s)) for n, s in dict(q=(Hq * D, H), k=(Hkv * D, H), v=(Hkv * D, H), o=(H, Hq * D),
                                                       gate=(I, H), up=(I, H), down=(H, I)).items()}
    g1, g2, gs = (1 + 0.1 * rnd(n) for n in (H, H, Hq * D))
    stream, sub = rnd(T, H).bfloat16(), rnd(T, H).bfloat16()
    n_pages = sum(pages_of(n + c, P) for n, c in zip(new, ctx)) + 2
    width = max(pages_of(n + c, P) for n, c in zip(new, ctx))
    kp, vp = rnd(n_pages, Hkv, P, D).bfloat16(), rnd(n_pages, Hkv, P, D).bfloat16()
    free, table = torch.randperm(n_pages, generator=g).int().to(DEV), torch.full((B, width), -1, **I32)
    ctx_t, zero = torch.tensor(ctx, **I32), torch.zeros(B, **I32)
    n_free = torch.tensor([n_pages], **I32)
    n_free = tb.paged_plan(ctx_t, zero, table, free, n_free, P, sum(ctx))[4]  # the cached tokens' pages

    res, qx, sx, sumx = tb.add_rmsnorm_quant_act(sub, stream, g1)
    q, k, v = tb.bitlinear_group(qx, sx, sumx, [W["q"], W["k"], W["v"]], [Hq * D, Hkv * D, Hkv * D])
    cu, kv, pos, slots, _ = tb.paged_plan(torch.tensor(new, **I32), ctx_t, table, free, n_free, P, T)
    q_rot = tb.rope_paged_append(q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D), pos, slots, theta, kp, vp)
    att = tb.attention_paged(q_rot, kp, vp, table, cu, kv, max(new))
    qa, sa, suma = tb.rmsnorm_quant_act(att.view(T, Hq * D), gs)
    o = tb.bitlinear(qa, sa, suma, W["o"], H)
    res2, qf, sf, sumf = tb.add_rmsnorm_quant_act(o, res, g2)
    h = tb.bitlinear_gate_up_act(qf, sf, sumf, W["gate"], W["up"], I)
    torch.cuda.synchronize()
    assert tb.device_status() == 0

    assert torch.equal(res, (sub.float() + stream.float()).bfloat16())
    assert torch.equal(res2, (o.float() + res.float()).bfloat16())
    b = Batch(new, [n + c for n, c in zip(new, ctx)], Hq, Hkv, P)
    b.q, b.kp, b.vp, b.table = q_rot, kp, vp, table
    check_attention(b, att)
    # the appended rows are the new tokens' keys and values, at their request's places
    t = 0
    for i, (n, c) in enumerate(zip(new, ctx)):
        for j in range(n):
            page, row = int(table[i, (c + j) // P]), (c + j) % P
            assert torch.equal(vp[page, :, row], v.view(T, Hkv, D)[t + j])
            x = k.view(T, Hkv, D)[t + j: t + j + 1].cpu().float().numpy()
            want = torch.from_numpy(O.apply_rope(x, np.array([c + j]), theta))[0]
            size = (want[:, :64] ** 2 + want[:, 64:] ** 2).sqrt().repeat(1, 2)
            assert ((kp[page, :, row].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6 * size).all()
        t += n
    q2, s2, sq2 = tb.rmsnorm_quant_act(res2, g2)
    assert torch.equal(q2, qf) and torch.equal(s2, sf) and torch.equal(sq2, sumf)
    assert torch.isfinite(h).all()
