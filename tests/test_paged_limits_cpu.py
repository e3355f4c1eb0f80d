"""Edges of the paged serving step that need no GPU: sizes whose products pass 64 bits, angles that the rotary call
does not take, the polynomial exponential of the attention of chunks, and what the built binding was built for."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import ternary_bitlinear_quantized_b200 as tb
from ternary_bitlinear_quantized_b200 import build as tbuild

P16 = ctypes.c_void_p(16)  # never dereferenced: every call fails its checks first
ROPE = dict(q=P16, k=P16, v=P16, xt=0, T=1, Hq=4, Hkv=2, d=128, pos=P16, slots=P16, theta=1e4, qr=P16, kp=P16, vp=P16, n=3,
            P=16, st=None)
PLAN = dict(new=P16, ctx=P16, B=2, P=16, tab=P16, width=4, free=P16, n_list=8, n_free=P16, T=3, cu=P16, kv=P16, pos=P16,
            slots=P16, out=P16, st=None)
ATTENTION = dict(q=P16, kp=P16, vp=P16, tab=P16, cu=P16, kv=P16, T=1, B=1, Hq=4, Hkv=2, d=128, n=3, P=16, width=4, max_new=1,
                 out=P16, ot=0, ws=P16, ws_bytes=1 << 40, st=None)


@pytest.fixture(scope="module")
def L():
    tbuild.build()
    return tb.lib()


def _call(fn, args, **change):
    return fn(*dict(args, **change).values())


@pytest.mark.parametrize("theta", [0.999, 1e-6, 1e-300, -1.0, float("inf"), float("nan")])
def test_rope_refuses_angles_that_outgrow_the_positions(L, theta):
    """Below theta = 1 the pairs turn by more than their position, and the fp64 reduction to one turn loses its accuracy."""
    assert _call(L.bitnet_rope_paged_append, ROPE, theta=theta) == 2
    assert _call(L.bitnet_rope_paged_append, ROPE, theta=1.0, q=None) == 1  # 1 itself passes that check: the next one answers


@pytest.mark.parametrize("extra", [0, 5, 1])
@pytest.mark.parametrize("P", [16, 256])
def test_sizes_whose_products_pass_64_bits_are_refused(L, P, extra):
    """n_pages page_size and width page_size of 2^64 and little more, which are little numbers in 64 bits."""
    big = (1 << 64) // P // 2 * 2 + extra
    for n in (big, big // 2, big // 16, (1 << 31) // P + extra):
        n = min(n, (1 << 63) - 1)
        assert _call(L.bitnet_rope_paged_append, ROPE, P=P, n=n) == 2
        assert _call(L.bitnet_attention_paged, ATTENTION, P=P, n=n) == 2
        assert _call(L.bitnet_attention_paged, ATTENTION, P=P, width=n) == 2
        assert _call(L.bitnet_paged_plan, PLAN, P=P, width=n) == 2
    # the largest there are pass that check: the next one answers
    n = 0x7FFFFFFF // P
    assert _call(L.bitnet_rope_paged_append, ROPE, P=P, n=n, q=None) == 1
    assert _call(L.bitnet_attention_paged, ATTENTION, P=P, n=n, width=(1 << 30) // P, q=None) == 1
    assert _call(L.bitnet_paged_plan, PLAN, P=P, width=(1 << 30) // P, cu=None) == 1


def test_the_binding_is_built_again_for_another_torch_or_python(L, monkeypatch):
    """A binary for another ABI is neither kept by the build nor loaded."""
    assert tbuild.binding_fits() and tb._load_serving().built_for == tbuild.built_for()
    runs = []
    monkeypatch.setattr(tbuild, "_run", lambda out, srcs, cmd, verbose, force: runs.append((out, cmd, force)))
    tbuild.build()
    assert not any(force for _, _, force in runs) and tbuild.BINDING not in [out for out, _, _ in runs]
    monkeypatch.setattr(tbuild.torch, "__version__", tbuild.torch.__version__ + ".1")
    assert not tbuild.binding_fits()
    runs.clear()
    tbuild.build()
    out, cmd, force = runs[-1]
    assert out == tbuild.BINDING and force and any(tbuild.built_for() in c for c in cmd)
    monkeypatch.setattr(tb, "_native", None)
    with pytest.raises(ImportError, match="build it with"):
        tb._load_serving()


def _exp2_pair(z):
    """exp2_pair of attn_chunk.cuh: the same fp32 steps.  fma: the exact product and sum in fp64, rounded once to fp32 but
    for double rounding (fp64 holds the product of two fp32 exactly; a tie that fp64 makes of a sum is off by 2^-53 of it)."""
    f32 = np.float32
    fma = lambda a, b, c: (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(f32)  # noqa: E731
    z = np.maximum(z.astype(f32), f32(-127))
    t = (z + f32(12582912.0)).astype(f32)
    n = (t + f32(-12582912.0)).astype(f32)
    f = (z - n).astype(f32)  # exact: n is the integer next to z
    p = np.full_like(z, f32(0.001326472032815218))
    for c in (0.009671512991189957, 0.05550733581185341, 0.24022242426872253, 0.6931470036506653, 1.0):
        p = fma(p, f, f32(c))
    return (p.view(np.uint32) + (t.view(np.uint32) << np.uint32(23))).view(f32)


def test_polynomial_exponential():
    """Its documented error: 2^-23.1 by the coefficients, 2^-22.4 as evaluated in fp32; powers of two exact; weights of scores
    far below the maximum, and of masked ones, zero or below the smallest normal number."""
    f = np.linspace(-0.5, 0.5, 400001)
    c = np.float32([0.001326472032815218, 0.009671512991189957, 0.05550733581185341, 0.24022242426872253, 0.6931470036506653, 1.0])
    assert np.abs(np.polyval(c.astype(np.float64), f) / 2.0 ** f - 1).max() <= 2.0 ** -23.1
    rng = np.random.default_rng(0)
    z = np.concatenate([np.linspace(-125.4, 8.0, 1500001), rng.uniform(-1, 1, 500000), np.arange(-125, 9) + 0.5,
                        np.arange(-125, 9) - 0.5]).astype(np.float32)
    assert np.abs(_exp2_pair(z).astype(np.float64) / 2.0 ** z.astype(np.float64) - 1).max() <= 2.0 ** -22.4
    whole = np.arange(-126, 9).astype(np.float32)
    assert np.array_equal(_exp2_pair(whole).astype(np.float64), 2.0 ** whole.astype(np.float64))
    low = _exp2_pair(np.concatenate([np.float32([-np.inf, -1e30, -127.0]), np.linspace(-200, -126.6, 1000).astype(np.float32)]))
    assert not low[:3].any() and (low >= 0).all() and (low < 2.0 ** -126).all()
