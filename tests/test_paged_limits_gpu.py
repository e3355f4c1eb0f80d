"""Edges of the paged serving step on the GPU."""
from __future__ import annotations

import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

import ternary_bitlinear_quantized_b200 as tb
from tests.paged_util import D, Batch, check_attention, weight_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


STAND_IN = """
#include <time.h>
static volatile int inside_, go_;
int inside(void) { return inside_; }
void go(void) { go_ = 1; }
static int wait_for_go(void) {  /* two seconds at most: 6 is BITNET_ERR_CUDA */
  int ms, ok;
  inside_ = 1;
  for (ms = 0; ms < 2000 && !go_; ++ms) {
    struct timespec t = {0, 1000000};
    nanosleep(&t, 0);
  }
  ok = go_;
  inside_ = go_ = 0;
  return ok ? 0 : 6;
}
int bitnet_add_rmsnorm_quant_act() { return wait_for_go(); }
int bitnet_paged_plan() { return wait_for_go(); }
int bitnet_rope_paged_append() { return wait_for_go(); }
unsigned long bitnet_attention_paged_workspace_bytes() { return 64; }
int bitnet_attention_paged() { return wait_for_go(); }
"""


def test_other_threads_run_during_a_call(tmp_path):
    """A launch can wait for room in the stream's queue, which other threads (or a host callback in that stream) may have to
    make.  Stand-ins for the library's calls, which launch nothing, return once another Python thread has let them."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    (tmp_path / "stand_in.c").write_text(STAND_IN)
    lib = str(tmp_path / "stand_in.so")
    subprocess.run([cc, "-shared", "-fPIC", "-O1", "-std=gnu89", "-o", lib, str(tmp_path / "stand_in.c")], check=True, capture_output=True)
    stand_in = ctypes.CDLL(lib)
    b = Batch([1, 1], [20, 33], 4, 2, 16)
    x, i, k = torch.ones(2, 64, device=DEV), torch.ones(2, **I32), b.q[:, :2].contiguous()
    calls = [lambda: tb.add_rmsnorm_quant_act(x, x, None),
             lambda: tb.paged_plan(i, i, b.table, torch.arange(4, **I32), torch.ones(1, **I32), 16, 2),
             lambda: tb.rope_paged_append(b.q, k, k, i, i, 1e4, b.kp, b.vp),
             lambda: tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, 1)]
    native = tb._load_serving()

    def let_go(done):
        while not done.is_set():
            if stand_in.inside():
                stand_in.go()
            time.sleep(0.001)

    done = threading.Event()
    other = threading.Thread(target=let_go, args=(done,), daemon=True)
    native.bind(stand_in._handle, tb.BitnetError)
    try:
        other.start()
        for call in calls:
            call()
    finally:
        done.set()
        other.join()
        native.bind(tb.lib()._handle, tb.BitnetError)
    check_attention(b, calls[3](), p_round=weight_step(b))


def _refused(fn, *args, **kw):
    with pytest.raises(ValueError, match="overlap"):
        fn(*args, **kw)


def test_plan_refuses_outputs_that_overlap():
    B, T, W = 4, 6, 3
    pool = torch.zeros(200, **I32)
    new, ctx, table = pool[0:B], pool[B:2 * B], pool[20:20 + B * W].view(B, W)
    free, n_free = pool[40:60], pool[60:61]
    new.fill_(1)
    free.copy_(torch.arange(20))
    n_free.fill_(20)
    sizes = (B + 1, B, T, T, 1)
    own = lambda: [torch.empty(s, **I32) for s in sizes]  # noqa: E731
    plan = lambda out: tb.paged_plan(new, ctx, table, free, n_free, 16, T, out=tuple(out))  # noqa: E731
    for k, n in enumerate(sizes):
        for at in {0, B - 1, 2 * B - 1, 19, 20 + B * W - 1, 40 - n + 1, 59, 61 - n}:  # each reaches into an input or the table
            out = own()
            out[k] = pool[max(0, at): max(0, at) + n]
            touches = any(max(0, at) < e and s < max(0, at) + n for s, e in ((0, 2 * B), (20, 20 + B * W), (40, 61)))
            if touches:
                _refused(plan, out)
    for j in range(5):  # one output inside another
        for k in range(5):
            if j != k:
                out = own()
                both = torch.empty(sizes[j] + sizes[k], **I32)
                out[j], out[k] = both[: sizes[j]], both[sizes[j] - 1: sizes[j] - 1 + sizes[k]]
                _refused(plan, out)
    _refused(tb.paged_plan, new, ctx, pool[2: 2 + B * W].view(B, W), free, n_free, 16, T)  # the table is written too
    _refused(tb.paged_plan, new, ctx, table, pool[31:51], n_free, 16, T)
    # side by side is fine
    buf, at, out = torch.empty(sum(sizes), **I32), 0, []
    for s in sizes:
        out.append(buf[at: at + s])
        at += s
    cu, kv, pos, slots, left = plan(out)
    assert cu.tolist() == [0, 1, 2, 3, 4] and kv.tolist() == [1] * 4 and left.tolist() == [16] and tb.device_status() == 0
    assert slots.tolist() == [19 * 16, 18 * 16, 17 * 16, 16 * 16, -1, -1] and pos.tolist() == [0] * 6


def test_norm_refuses_outputs_that_overlap():
    T, K = 6, 64
    x, r = torch.randn(T, K, device=DEV), torch.randn(T, K, device=DEV)
    want = tb.add_rmsnorm_quant_act(x, r, None)
    _refused(tb.add_rmsnorm_quant_act, x, r, None, residual_out=x)
    both = torch.cat([r, r])
    _refused(tb.add_rmsnorm_quant_act, x, both[:T], None, residual_out=both[1: T + 1])
    _refused(tb.add_rmsnorm_quant_act, r, r, None, residual_out=r)
    q, s, sq = torch.empty(T, K, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV), torch.empty(T, **I32)
    _refused(tb.add_rmsnorm_quant_act, x, r, None, out=(x.view(torch.int8).flatten()[: T * K].view(T, K), s, sq))
    _refused(tb.add_rmsnorm_quant_act, x, r, None, out=(q, s, s.view(torch.int32)))
    gain = torch.ones(K, device=DEV)
    _refused(tb.add_rmsnorm_quant_act, x, r, gain, out=(q, gain[:T], sq))
    got = tb.add_rmsnorm_quant_act(x, r, None, residual_out=r, out=(q, s, sq))  # in place
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rope_refuses_outputs_that_overlap():
    T, Hq, Hkv, P = 3, 4, 2, 16
    q, k, v = (torch.randn(T, h, D, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv))
    kv = torch.zeros(2, 2, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    pos, slots = torch.arange(T, **I32), torch.arange(T, **I32)
    call = lambda q_rot=None, kp=kv[0], vp=kv[1], k=k: tb.rope_paged_append(q, k, v, pos, slots, 1e4, kp, vp, q_rot=q_rot)  # noqa: E731
    want = call()
    _refused(call, q)
    _refused(call, kp=kv[1])
    _refused(call, kv[0].flatten()[: T * Hq * D].view(T, Hq, D))
    _refused(call, k=kv[1].flatten()[: T * Hkv * D].view(T, Hkv, D))
    assert torch.equal(call(torch.empty_like(q)), want)


@pytest.mark.parametrize("new", [1, 70])
def test_attention_refuses_outputs_that_overlap_but_for_q_itself(new):
    b = Batch([new, new], [600, 650], 8, 2, 16, seed=new, pad=1)
    args = (b.kp, b.vp, b.table, b.cu, b.kv, b.max_new)
    want = tb.attention_paged(b.q, *args)
    ws = torch.empty(tb.attention_paged_workspace_bytes(8, 2, new), dtype=torch.uint8, device=DEV)
    n = b.q.numel()
    _refused(tb.attention_paged, b.q, *args, out=b.kp.flatten()[:n].view_as(b.q))
    _refused(tb.attention_paged, b.q, *args, out=ws[: 2 * n].view(torch.bfloat16).view_as(b.q), ws=ws)
    _refused(tb.attention_paged, b.q, *args, ws=b.vp.view(torch.uint8).flatten())
    shifted = torch.cat([b.q, b.q])
    _refused(tb.attention_paged, shifted[: len(b.q)], *args, out=shifted[1: 1 + len(b.q)])
    check_attention(b, want, p_round=weight_step(b))
    for _ in range(5):
        q = b.q.clone()
        got = tb.attention_paged(q, *args, out=q, ws=ws)
        assert got.data_ptr() == q.data_ptr() and torch.equal(got[: 2 * new], want[: 2 * new]) and torch.equal(got[2 * new:], b.q[2 * new:])


def test_a_max_new_of_zero_is_too_small_for_requests_with_tokens():
    """As with any max_new that a request exceeds: the request is skipped and flagged."""
    b = Batch([1, 0, 1], [40, 7, 90], 8, 2, 16)
    out = torch.full(b.q.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, 0, out=out)
    assert tb.device_status() == 8 and (out == 77.0).all()
    b.cu.zero_()  # no request has tokens: nothing to flag
    tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, 0, out=out)
    assert tb.device_status() == 0 and (out == 77.0).all()


# The kernel for many rows gives each request 32, 16, .. 1 of its 384 threads (up to 12, 24, .. 384 requests), and takes more
# requests in rounds: a chunk or two among many requests of one token or none, at the start, in the middle and at the end.
@pytest.mark.parametrize("B", [12, 13, 25, 60, 97, 200, 384, 385, 800, 1300])
@pytest.mark.parametrize("at", ["start", "middle", "end", "both"])
def test_chunks_among_many_requests(B, at):
    new, kv = [0 if i % 5 == 2 else 1 for i in range(B)], [(37 * i) % 150 + 1 for i in range(B)]
    for i, n, k in {"start": [(0, 70, 200)], "middle": [(B // 2, 45, 45), (B // 2 + 1, 33, 20)], "end": [(B - 1, 100, 390)],
                    "both": [(0, 40, 41), (B - 1, 64, 700)]}[at]:
        new[i], kv[i] = n, k
    b = Batch(new, kv, 8, 2, 16, seed=B, pad=2)
    out = torch.full(b.q.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, out=out)
    assert tb.device_status() == 0 and (out[sum(new):] == 77.0).all()
    check_attention(b, out)
    assert torch.equal(out[: sum(new)], tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new)[: sum(new)])


@pytest.mark.parametrize("B", [385, 2000])
def test_many_requests_some_of_which_do_not_fit(B):
    new, kv = [1] * B, [(61 * i) % 90 + 1 for i in range(B)]
    new[B // 2], kv[B // 2] = 50, 60
    b = Batch(new, kv, 4, 2, 16, seed=1)
    skip = (0, 7, B // 2 + 1, B - 1)
    for i in skip:
        b.kv[i] = b.width * 16 + 1
    out = torch.full(b.q.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, out=out)
    assert tb.device_status() == 8
    check_attention(b, out, skip=skip)
    for i in skip:
        assert (out[sum(new[:i]): sum(new[: i + 1])] == 77.0).all()
