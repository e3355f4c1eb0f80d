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
from tests.paged_util import Batch, check_attention, weight_step

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
