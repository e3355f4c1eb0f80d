// The paged key/value cache of a serving step over many requests: which pages and rows the
// step's tokens go to (k_paged_plan), and the rotary embedding with the append to those rows
// (k_rope_paged).  The cache is k_pages / v_pages, bf16 [pages][Hkv][page_size][128]; slot s
// names row s % page_size of page s / page_size, in every key/value head.  The attention that
// reads the cache is in attn_paged.cuh.
//
// Lengths, tables, slots and page ids live on the device, so no step waits for the host; what
// the host cannot check the kernels do: an index out of range is skipped and the device status
// word set to BITNET_ERR_INDEX.
#pragma once
#include "common.cuh"
#include "quant.cuh"

namespace bitnet {

constexpr int PG_D = 128;               // head size

BN_DEV void flag_index_error() { atomicExch(&g_device_status, (int)BITNET_ERR_INDEX); }

// Inclusive prefix sums over the block of two numbers per thread, and the block's sums.
// `scratch`: 64 long longs of shared memory, not read or written otherwise.
BN_DEV void block_scan_incl2(long long (&v)[2], long long* scratch, long long (&total)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long u = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += u;
    }
  if (lane == 31) {
    scratch[2 * warp] = v[0];
    scratch[2 * warp + 1] = v[1];
  }
  __syncthreads();
  total[0] = total[1] = 0;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long s = scratch[2 * w + k];
      if (w < warp) v[k] += s;
      total[k] += s;
    }
}

// Largest i in [0, n) with a[i] <= x, for ascending a with a[0] <= x.
BN_DEV int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ the step's plan
// need_i = ceil((ctx_i + new_i) / P) - ceil(ctx_i / P) pages are taken from the top of the free
// list, request by request: with start_i the sum of the needs before i, page j of request i is
// free[n_free - 1 - start_i - j].  Token t of the step belongs to the request i with
// cu_i <= t < cu_{i+1}; its position is ctx_i + t - cu_i and its slot table[i][pos / P] P + pos % P.
//
// Bound by latency (a few dependent loads and two scans; the largest steps write two ints a
// token).  So it is one launch: every CTA makes both prefix sums for itself (B lengths are a few
// KB from L2) and then writes its share of the tokens and of the new table entries; a token's new
// page is read from the free list directly, not from the table entry that another CTA may be
// writing.
constexpr int PLAN_THREADS = 256;
constexpr int PLAN_TOKENS = 256;  // tokens per CTA: 36371 tokens of 96 requests 3.9 us, with 1024 per CTA 6.4 us
__global__ void __launch_bounds__(PLAN_THREADS) k_paged_plan(const int* __restrict__ new_lens, const int* __restrict__ ctx_lens,
                                                             int B, int log2P, int* table, int width,
                                                             const int* __restrict__ free_pages, int n_list,
                                                             const int* __restrict__ n_free, int T, int* __restrict__ cu_out,
                                                             int* __restrict__ kv_out, int* __restrict__ pos_out,
                                                             int* __restrict__ slot_out, int* __restrict__ n_free_out) {
  extern __shared__ int plan_sm[];  // two sums of B + 1 requests: 32 KB for BITNET_MAX_REQUESTS
  __shared__ long long scratch[64];
  int* cu = plan_sm;            // [B + 1] tokens before request i
  int* start = plan_sm + B + 1; // [B + 1] new pages before request i
  pdl_launch_dependents();
  pdl_wait();
  const int P = 1 << log2P;
  const long long cap = (long long)width * P;
  bool bad = false;
  int nf = __ldg(n_free);
  if (nf < 0 || nf > n_list) {
    bad = true;
    nf = 0;
  }
  // A request's lengths; one that does not fit its row of the table keeps its place among the
  // tokens, but gets no pages and no slots.
  auto judge = [&](int& n, int& c, bool& fits) {
    fits = true;
    if (n < 0 || c < 0 || c + (long long)n > cap) {
      bad = true;
      fits = false;
      n = max(n, 0);
      c = (int)min((long long)max(c, 0), cap);
    }
    if (n > T) {  // keeps the sums in range
      bad = true;
      n = T;
    }
  };
  // slot of row r of a page; ids below 0 stand for no page, others must keep the slot an int32
  auto slot_of = [&](int page, int r) {
    if (page > (0x7FFFFFFF - r) >> log2P) {
      bad = true;
      return -1;
    }
    return page < 0 ? -1 : (page << log2P) + r;
  };
  // q consecutive requests a thread
  const int q = (B + PLAN_THREADS - 1) / PLAN_THREADS, i0 = min(B, (int)threadIdx.x * q), i1 = min(B, i0 + q);
  auto pages = [&](int n, int c, bool fits) { return fits ? ((c + n + P - 1) >> log2P) - ((c + P - 1) >> log2P) : 0; };
  for (int i = threadIdx.x; i < B; i += PLAN_THREADS) {  // the lengths, in the places of the sums
    cu[i] = __ldg(new_lens + i);
    start[i] = __ldg(ctx_lens + i);
  }
  __syncthreads();
  long long sum[2] = {0, 0}, total[2];  // tokens, new pages
  for (int i = i0; i < i1; ++i) {
    int n = cu[i], c = start[i];
    bool fits;
    judge(n, c, fits);
    sum[0] += n;
    sum[1] += pages(n, c, fits);
  }
  long long at0 = sum[0], at1 = sum[1];
  block_scan_incl2(sum, scratch, total);
  at0 = sum[0] - at0;
  at1 = sum[1] - at1;
  for (int i = i0; i < i1; ++i) {
    int n = cu[i], c = start[i];
    bool fits;
    judge(n, c, fits);
    cu[i] = (int)min(at0, (long long)T);
    start[i] = (int)at1;
    if (blockIdx.x == 0) kv_out[i] = fits ? c + n : c;
    at0 += n;
    at1 += pages(n, c, fits);
  }
  long long tok = total[0];
  const long long pg = total[1];  // at most (T / 16 + 1) B < 2^31
  if (tok > T) {
    bad = true;
    tok = T;
  }
  if (threadIdx.x == 0) {
    cu[B] = (int)tok;
    start[B] = (int)pg;
    if (blockIdx.x == 0) n_free_out[0] = nf - (int)pg;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= B; i += PLAN_THREADS) cu_out[i] = cu[i];
  // new table entries, over the whole grid
  const int nthreads = gridDim.x * PLAN_THREADS, gid = blockIdx.x * PLAN_THREADS + threadIdx.x;
  for (int e = gid; e < (int)pg; e += nthreads) {
    const int i = last_not_above(start, B, e);
    const int c = __ldg(ctx_lens + i);
    const int at = nf - 1 - e;
    table[(long long)i * width + ((c + P - 1) >> log2P) + (e - start[i])] = at >= 0 ? __ldg(free_pages + at) : -1;
  }
  // tokens
  const int t1 = min(T, (int)(blockIdx.x + 1) * PLAN_TOKENS);
  for (int t = blockIdx.x * PLAN_TOKENS + threadIdx.x; t < t1; t += PLAN_THREADS) {
    int pos = 0, slot = -1;
    if (t < (int)tok) {
      const int i = last_not_above(cu, B, t);
      int n = __ldg(new_lens + i), c = __ldg(ctx_lens + i);
      bool fits;
      judge(n, c, fits);
      pos = c + t - cu[i];
      if (fits) {
        const int pi = pos >> log2P, old = (c + P - 1) >> log2P;
        int page;
        if (pi < old) {
          page = table[(long long)i * width + pi];
        } else {
          const int at = nf - 1 - start[i] - (pi - old);
          page = at >= 0 ? __ldg(free_pages + at) : -1;
        }
        slot = slot_of(page, pos & (P - 1));
      }
    }
    pos_out[t] = pos;
    slot_out[t] = slot;
  }
  if (bad) flag_index_error();
}

// ------------------------------------------------------------------ rotary embedding + append
// The pair (x_i, x_{i+64}) of q and k turns by a = p theta^(-2i/128).  The host passes
// g_i = theta^(-2i/128) / (2 pi) in fp64, so a is p g_i turns: its whole turns are dropped in
// fp64 (p g_i - rint(p g_i) is exact) and sine and cosine of pi times the rest, |rest| <= 1,
// taken in fp32.  theta >= 1, so |p g_i| <= |p| / (2 pi) < 2^29, and the fp64 product is off by at most
// 2^-23 turns there (g_i's rounding and its own, 2^-53 of it each) and by 2^-37 at positions below 2^16.
// The rotation is fp32, one rounding an operation; q_rot and the cache are bf16 (nearest even).
//
// Bound by HBM: each value is read and written once.  A CTA takes TOKENS tokens: their 64
// angles each are made once and shared by all heads (a sine and cosine per head would cost more
// than the copy), then every thread moves 8 + 8 values of one head for all the tokens at once, 2 TOKENS
// 16-byte loads in flight.  8400 tokens of 64 + 8 + 8 heads: 57.5 us (6.0 TB/s) with two tokens and 128 threads
// a CTA, 58.5 with four (cosines read one by one: 60.7), 62 us one token after the other.  With few
// tokens each has a CTA of 256 threads: 64 tokens 3.5 us, of 128 threads 4.1, four tokens per CTA 7.2.
constexpr int ROPE_TOKENS = 2;
BN_HOST_DEV constexpr int rope_threads(int tokens) { return tokens == 1 ? 256 : 128; }
struct RopeTurns {
  double g[PG_D / 2];
};
template <typename TIn, int TOKENS>
__global__ void __launch_bounds__(rope_threads(TOKENS)) k_rope_paged(const TIn* __restrict__ q, const TIn* __restrict__ k,
                                                             const TIn* __restrict__ v, const int* __restrict__ positions,
                                                             const int* __restrict__ slots, int T, int Hq, int Hkv, int log2P,
                                                             long long n_slots, const __grid_constant__ RopeTurns turns,
                                                             __nv_bfloat16* __restrict__ q_rot,
                                                             __nv_bfloat16* __restrict__ k_pages,
                                                             __nv_bfloat16* __restrict__ v_pages) {
  constexpr int HALF = PG_D / 2, THREADS = rope_threads(TOKENS);
  __shared__ __align__(16) float s_cos[TOKENS][HALF], s_sin[TOKENS][HALF];
  __shared__ int s_slot[TOKENS];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * TOKENS;
#pragma unroll
  for (int a0 = 0; a0 < TOKENS * HALF; a0 += THREADS) {
    const int tt = (a0 + threadIdx.x) / HALF, i = threadIdx.x % HALF, t = t0 + tt;
    const int slot = tt < TOKENS && t < T ? __ldg(slots + t) : -1;
    if (i == 0 && tt < TOKENS) {
      s_slot[tt] = slot < n_slots ? slot : -1;
      if (slot >= n_slots) flag_index_error();
    }
    if (slot >= 0) {
      const double a = __dmul_rn((double)__ldg(positions + t), turns.g[i]);
      const float r = __double2float_rn(__dsub_rn(a, rint(a)));
      sincospif(__fmul_rn(2.0f, r), &s_sin[tt][i], &s_cos[tt][i]);
    }
  }
  __syncthreads();
  auto pack = [](float a, float b) {
    const __nv_bfloat162 w = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&w);
  };
  const int units = (Hq + 2 * Hkv) * 8;  // (head, 8-value chunk of its lower half with the chunk 64 above)
  for (int u = threadIdx.x; u < units; u += THREADS) {
    const int hh = u >> 3, c = (u & 7) * 8;
    const bool is_q = hh < Hq, is_v = hh >= Hq + Hkv;
    const int h = is_q ? hh : hh - Hq - (is_v ? Hkv : 0), heads = is_q ? Hq : Hkv;
    const TIn* src = (is_q ? q : (is_v ? v : k)) + ((long long)t0 * heads + h) * PG_D + c;
    Raw8<TIn> lo[TOKENS], hi[TOKENS];
#pragma unroll
    for (int tt = 0; tt < TOKENS; ++tt)
      if (s_slot[tt] >= 0) {
        lo[tt].load(src + tt * heads * PG_D);
        hi[tt].load(src + tt * heads * PG_D + HALF);
      }
#pragma unroll
    for (int tt = 0; tt < TOKENS; ++tt) {
      const int slot = s_slot[tt];
      if (slot < 0) continue;
      float a[8], b[8];
      lo[tt].get(a);
      hi[tt].get(b);
      if (!is_v) {
        float cs[8], sn[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          *reinterpret_cast<float4*>(cs + j) = *reinterpret_cast<const float4*>(&s_cos[tt][c + j]);
          *reinterpret_cast<float4*>(sn + j) = *reinterpret_cast<const float4*>(&s_sin[tt][c + j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float co = cs[j], si = sn[j], x1 = a[j], x2 = b[j];
          a[j] = __fsub_rn(__fmul_rn(x1, co), __fmul_rn(x2, si));
          b[j] = __fadd_rn(__fmul_rn(x2, co), __fmul_rn(x1, si));
        }
      }
      __nv_bfloat16* dst = is_q ? q_rot + ((long long)(t0 + tt) * Hq + h) * PG_D + c
                                : (is_v ? v_pages : k_pages) + (((long long)(slot >> log2P) * Hkv + h << log2P) + (slot & ((1 << log2P) - 1))) * PG_D + c;
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack(a[0], a[1]), pack(a[2], a[3]), pack(a[4], a[5]), pack(a[6], a[7]));
      *reinterpret_cast<uint4*>(dst + HALF) = make_uint4(pack(b[0], b[1]), pack(b[2], b[3]), pack(b[4], b[5]), pack(b[6], b[7]));
    }
  }
}

}  // namespace bitnet
