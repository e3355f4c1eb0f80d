"""The paged serving step without a GPU: what its entry points refuse, before any CUDA call, and the plain forms
that its GPU tests compare with, against other ways to compute the same."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import ternary_bitlinear_quantized_b200 as tb
from oracle import bitnet_oracle as O
from ternary_bitlinear_quantized_b200 import build as tbuild
from tests.paged_util import D, Batch, attention_ref, pages_of, plan_ref

P16, ODD = ctypes.c_void_p(16), ctypes.c_void_p(18)  # never dereferenced: every call fails its checks first


@pytest.fixture(scope="module")
def L():
    tbuild.build()
    return tb.lib()


def _call(fn, args, **change):
    a = dict(args)
    a.update(change)
    return fn(*a.values())


def test_add_norm_refusals(L):
    f = L.bitnet_add_rmsnorm_quant_act
    a = dict(x=P16, xt=0, r=P16, rt=0, gain=None, eps=1e-6, T=1, K=128, ro=P16, q=P16, s=P16, sq=P16, st=None)
    assert _call(f, a, xt=2) == 4 and _call(f, a, rt=-1) == 4
    assert _call(f, a, K=0) == 2 and _call(f, a, K=49153) == 2 and _call(f, a, T=-1) == 2 and _call(f, a, T=1 << 31) == 2
    for n in ("x", "r", "ro", "q", "s", "sq"):
        assert _call(f, a, **{n: None}) == 1 and _call(f, a, **{n: ODD}) == 3
    assert _call(f, a, gain=ODD) == 3
    assert _call(f, a, T=0, x=None) == 0


def test_plan_refusals(L):
    f = L.bitnet_paged_plan
    a = dict(new=P16, ctx=P16, B=2, P=16, tab=P16, width=4, free=P16, n_list=8, n_free=P16, T=3, cu=P16, kv=P16, pos=P16,
             slots=P16, out=P16, st=None)
    assert _call(f, a, B=-1) == 2 and _call(f, a, B=4097) == 2 and _call(f, a, T=-1) == 2 and _call(f, a, T=(1 << 22) + 1) == 2
    for P in (0, 8, 24, 512, -16):
        assert _call(f, a, P=P) == 2
    assert _call(f, a, width=0) == 2 and _call(f, a, width=1 << 27) == 2 and _call(f, a, n_list=-1) == 2
    for n in ("new", "ctx", "tab", "free", "n_free", "cu", "kv", "pos", "slots", "out"):
        assert _call(f, a, **{n: None}) == 1 and _call(f, a, **{n: ODD}) == 3


def test_rope_refusals(L):
    f = L.bitnet_rope_paged_append
    a = dict(q=P16, k=P16, v=P16, xt=0, T=1, Hq=4, Hkv=2, d=128, pos=P16, slots=P16, theta=1e4, qr=P16, kp=P16, vp=P16, n=3,
             P=16, st=None)
    assert _call(f, a, xt=5) == 4
    for c in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=1026), dict(d=64), dict(P=48), dict(n=0), dict(n=1 << 27),
              dict(theta=0.0), dict(theta=float("nan"))):
        assert _call(f, a, **c) == 2, c
    for n in ("q", "k", "v", "pos", "slots", "qr", "kp", "vp"):
        assert _call(f, a, **{n: None}) == 1 and _call(f, a, **{n: ODD}) == 3
    assert _call(f, a, T=0, q=None) == 0


def test_attention_refusals(L):
    f = L.bitnet_attention_paged
    a = dict(q=P16, kp=P16, vp=P16, tab=P16, cu=P16, kv=P16, T=1, B=1, Hq=4, Hkv=2, d=128, n=3, P=16, width=4, max_new=1, out=P16,
             ot=0, ws=P16, ws_bytes=1 << 40, st=None)
    assert _call(f, a, ot=3) == 4
    for c in (dict(T=-1), dict(B=-1), dict(B=4097), dict(Hq=0), dict(Hq=5), dict(Hq=1026), dict(d=64), dict(n=0), dict(P=8),
              dict(n=1 << 27), dict(width=0), dict(width=1 << 27), dict(max_new=-1)):
        assert _call(f, a, **c) == 2, c
    for n in ("q", "kp", "vp", "tab", "cu", "kv", "out"):
        assert _call(f, a, **{n: None}) == 1 and _call(f, a, **{n: ODD}) == 3
    assert _call(f, a, ws=None) == 5 and _call(f, a, ws_bytes=64) == 5 and _call(f, a, ws=ODD) == 3
    for c in (dict(T=0), dict(B=0), dict(max_new=0)):
        assert _call(f, a, q=None, **c) == 0
    assert L.bitnet_attention_paged_workspace_bytes(5, 2, 1) == 0 and L.bitnet_attention_paged_workspace_bytes(4, 2, -1) == 0
    # the most rows there are take the workspace of the kernel for many rows, as 33 of one head do
    assert L.bitnet_attention_paged_workspace_bytes(4, 2, 1 << 62) == L.bitnet_attention_paged_workspace_bytes(1, 1, 33)
    assert L.bitnet_attention_paged_workspace_bytes(1, 1, 33) > L.bitnet_attention_paged_workspace_bytes(1, 1, 32) > 0
    assert L.bitnet_status_string(8) != b"unknown status"


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        tb.add_rmsnorm_quant_act(x, x, None)
    with pytest.raises(ValueError):
        tb.paged_plan(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1], 16, 2)
    with pytest.raises(ValueError):
        tb.rope_paged_append(torch.zeros(1, 2, D), torch.zeros(1, 1, D), torch.zeros(1, 1, D), i[:1], i[:1], 1e4,
                             torch.zeros(1, 1, 16, D), torch.zeros(1, 1, 16, D))
    with pytest.raises(ValueError):
        tb.attention_paged(torch.zeros(1, 2, D), torch.zeros(1, 1, 16, D), torch.zeros(1, 1, 16, D), i.view(1, 2), i, i[:1], 1)


def test_plain_plan():
    cu, kv, pos, slots, left, table = plan_ref([3, 0, 17], [15, 4, 0], [[7, 0], [5, 0], [0, 0]], [1, 2, 3, 4], 4, 16, 22)
    assert cu == [0, 3, 3, 20] and kv == [18, 4, 17] and left == 1
    assert table == [[7, 4], [5, 0], [3, 2]]
    assert pos[:3] == [15, 16, 17] and slots[:3] == [7 * 16 + 15, 64, 65] and slots[3:20] == [48 + i for i in range(16)] + [32]
    assert pos[20:] == [0, 0] and slots[20:] == [-1, -1]


def test_plain_attention_is_the_oracles():
    b = Batch([3, 1], [20, 33], 4, 2, 16, device="cpu")
    out, bound, A = attention_ref(b)
    t0 = 0
    for i, (n, kv) in enumerate(zip(b.new, b.kvl)):
        rows = b.table[i, : pages_of(kv, 16)].long()
        K, V = (x[rows].transpose(0, 1).reshape(2, -1, D)[:, :kv].transpose(0, 1).float().numpy() for x in (b.kp, b.vp))
        want = O.attention(b.q[t0: t0 + n].float().numpy(), K, V, range(kv - n, kv))
        assert abs(out[t0: t0 + n].numpy() - want).max() < 1e-12
        t0 += n
    assert (out.abs() <= A * (1 + 1e-12)).all() and (bound > 0).all() and not math.isnan(float(out.sum()))


def test_plain_attention_of_a_row_that_sees_nothing():
    b = Batch([3], [1], 2, 1, 16, device="cpu")
    out, _, _ = attention_ref(b)
    assert not out[:2].any() and torch.equal(out[2], b.vp[b.table[0, 0], 0, 0].double().expand(2, D))
