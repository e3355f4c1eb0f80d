"""The weights of the paged attention's second product: fp32 outputs keep them as the sum of two bf16 in both kernels, so a
request's fp32 result is as precise beside a prompt's chunk as it is alone.

Scores here are exact: q and k hold small whole numbers, whose products and sums fp32 holds without rounding in any order.
What is left, relative to A = sum w |v| / sum w of an element (w: the weights, L: visible rows):
  weights    two bf16: half a step of half a step, 2^-16
  exp        2^-22 by its documented error and 2^-22.5 by the polynomial, in numerator and denominator: 2 * 2^-22
  exponents  the scaled score and the scaled maximum, a rounding of 2^-24 of |s| each, s <= S, and the fused step's own; in
             numerator and denominator: 2 * 3 * 2^-24 * S
  products   2 ceil(L / 16) instructions of 16 products, each cut to no less than 23 bits of the largest number in it, the
             accumulator among them: 17 * 2^-23 each
  sums       L additions of the denominator at most, 2^-24 each; joins and the division: 2^-21
"""
from __future__ import annotations

import math

import pytest
import torch

import ternary_bitlinear_quantized_b200 as tb
from tests.paged_util import D, Batch, attention_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _exact_scores(new, kv, Hq, Hkv, P, seed):
    b = Batch(new, kv, Hq, Hkv, P, seed=seed)
    g = torch.Generator().manual_seed(seed)
    b.q = torch.randint(-2, 3, b.q.shape, generator=g).bfloat16().to(DEV)
    whole = torch.randint(-1, 2, b.kp.shape, generator=g).bfloat16().to(DEV)
    b.kp = torch.where(torch.isnan(b.kp), b.kp, whole)  # what no request sees stays NaN
    return b


def _tolerance(b):
    _, _, A = attention_ref(b)
    L = max(b.kvl)
    S = 2 * D / math.sqrt(D)
    rel = 2.0 ** -16 + 2 * 2.0 ** -22 + 6 * 2.0 ** -24 * S + 2 * -(-L // 16) * 17 * 2.0 ** -23 + L * 2.0 ** -24 + 2.0 ** -21
    return A * rel


def _check(b, got, rows):
    ref, _, _ = attention_ref(b)
    err, tol = (got.double() - ref).abs()[rows], _tolerance(b)[rows]
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-300)).max())} of the tolerance"


def _attend(b, out_dtype=torch.float32):
    return tb.attention_paged(b.q, b.kp, b.vp, b.table, b.cu, b.kv, b.max_new, out_dtype)


@pytest.mark.parametrize("new,kv,Hq,Hkv,P", [
    ([40], [40], 2, 2, 16),                  # a prompt behind nothing, one query head a key/value head
    ([60], [64], 8, 2, 64),
    ([33, 1, 20], [33, 30, 60], 12, 4, 16),
    ([5, 1, 1], [5, 12, 1], 40, 4, 32),      # 10 heads a key/value head: 50 rows
    ([2], [3], 33, 1, 16),
    ([130, 7], [200, 190], 4, 4, 128),       # several units, tiles that several CTAs share
    ([64] * 20, [64 + i for i in range(20)], 8, 1, 16),
])
def test_fp32_outputs_of_many_rows_keep_the_weights(new, kv, Hq, Hkv, P):
    b = _exact_scores(new, kv, Hq, Hkv, P, seed=sum(new))
    assert b.max_new * (Hq // Hkv) > 32
    got = _attend(b)
    _check(b, got, slice(0, sum(new)))
    assert torch.equal(got, _attend(b)) and tb.device_status() == 0


def test_a_single_token_is_as_precise_beside_a_chunk_as_alone():
    Hq, Hkv, P = 8, 2, 16
    alone = _exact_scores([1, 1, 1], [9, 40, 64], Hq, Hkv, P, seed=1)
    _check(alone, _attend(alone), slice(0, 3))
    mixed = _exact_scores([1, 1, 1, 90], [9, 40, 64, 100], Hq, Hkv, P, seed=1)
    _check(mixed, _attend(mixed), slice(0, 3))


def test_bf16_outputs_are_within_their_own_half_step():
    """bf16 outputs of many rows: one bf16 a weight, half a step of 2^-8 each, beside the output's own half step."""
    b = _exact_scores([60], [64], 8, 2, 16, seed=3)
    ref, _, A = attention_ref(b)
    tol = _tolerance(b) + A * 2.0 ** -8
    assert bool(((_attend(b, torch.bfloat16).double() - ref).abs() <= tol + (ref.abs() + tol) * 2.0 ** -8).all())
