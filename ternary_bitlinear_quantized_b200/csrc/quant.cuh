// K-quant: fused BitNetRMSNorm + per-token absmax + int8 quantisation.
//
// "Add optional RMSNorm support to BitNet quantization (config + layers)": BitLinear
// applies BitNetRMSNorm (eps 1e-6 by default) to the activations before they are
// quantised; with use_rms_norm off (gain == nullptr) the activations go straight to
// the absmax quantiser.  "More BitNet-like IQ1_S quantizations": the activations of
// BitNet b1.58 are 8-bit.
//
// One CTA per token.  The row is staged once in shared memory as fp32; the three
// reductions (max|x|, the fixed-point sum of x^2, max|y|) and the sum of q are exact,
// so the result is independent of the thread count and of the order of summation.
//
// With a residual type TRes (bitnet_add_rmsnorm_quant_act) the kernels first add the residual
// stream: r' = TRes(x + r), one fp32 addition and one rounding, is written to r_out and is what
// the norm reads, so the codes are those of the plain kernels run on r'.  The row is in registers
// or shared memory anyway, so the stream is read and written once and r' is not read again.
// Every value is read before its own r_out is written, by the same thread: r_out may be r_in.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace bitnet {

template <typename TIn>
struct RowLoader;

template <>
struct RowLoader<__nv_bfloat16> {
  static constexpr int V = 8;  // elements per 16-byte vector
  BN_DEV static void load(const __nv_bfloat16* p, float* o) {
    uint4 v = *reinterpret_cast<const uint4*>(p);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  BN_DEV static float load1(const __nv_bfloat16* p) { return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p)); }
};

template <>
struct RowLoader<float> {
  static constexpr int V = 8;
  BN_DEV static void load(const float* p, float* o) {
    float4 a = *reinterpret_cast<const float4*>(p);
    float4 b = *reinterpret_cast<const float4*>(p + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
  BN_DEV static float load1(const float* p) { return *p; }
};

// Eight values as they lie in memory.  The loads of a row's pieces are issued before the first one is
// used: between them stand stores to r_out, which may be r_in, so the compiler keeps their order.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  BN_DEV void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  BN_DEV void get(float (&o)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4)
        o[i] = __uint_as_float(u[i]);
      else
        o[i] = __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
    }
  }
};
// v[0..8) = the stored residual TRes(x + r), also written to r_out.
template <typename TIn, typename TRes>
BN_DEV void add_residual8(float (&v)[8], const Raw8<TIn>& x, const Raw8<TRes>& res, TRes* r_out) {
  float r[8];
  x.get(v);
  res.get(r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], r[i]);
  if constexpr (std::is_same<TRes, float>::value) {
    reinterpret_cast<float4*>(r_out)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(r_out)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4*>(r_out) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// Stores v as a residual; the value as stored.
BN_DEV float store_residual1(float v, float* out) {
  *out = v;
  return v;
}
BN_DEV float store_residual1(float v, __nv_bfloat16* out) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  *out = b;
  return __bfloat162float(b);
}

// Quantise one staged row xs[0..K) in place of nothing: writes q, s_x, sum_q of the row.
// `vec` says whether K % 8 == 0 and the row pointers are 16-byte aligned.
BN_DEV void quantise_staged_row(float* xs, int K, const float* gain, float eps, int8_t* qrow,
                                float* s_out, int32_t* sum_out, bool vec, void* red_scratch,
                                float amax_x) {
  float* redf = reinterpret_cast<float*>(red_scratch);
  long long* redl = reinterpret_cast<long long*>(red_scratch);
  int* redi = reinterpret_cast<int*>(red_scratch);
  const int tid = threadIdx.x, nt = blockDim.x;

  float a;
  if (gain != nullptr) {
    float ms = 0.0f;
    if (amax_x > 0.0f) {
      const double M = __dmul_rn((double)amax_x, (double)amax_x);
      const int e = fixed_point_exponent(M, K);
      const double p2e = pow2_f64(e);
      long long part = 0;
      if (K >= kFixedSmallMinN)
        for (int k = tid; k < K; k += nt) part += fixed_sq_term_t<true>(xs[k], p2e);
      else
        for (int k = tid; k < K; k += nt) part += fixed_sq_term(xs[k], p2e);
      const long long S = block_reduce(part, redl, AddOpLL());
      ms = fixed_point_mean(S, e, K);
    }
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, eps)));
    float am = 0.0f;
    for (int k = tid; k < K; k += nt) {
      const float y = __fmul_rn(__fmul_rn(xs[k], inv), __ldg(gain + k));
      xs[k] = y;
      am = fmaxf(am, fabsf(y));
    }
    a = block_reduce(am, redf, MaxOp());
  } else {
    a = amax_x;  // y = x
  }
  const float s = __fdiv_rn(127.0f, fmaxf(a, 1e-5f));
  int sum = 0;
  if (vec) {
    for (int k = tid * 8; k < K; k += nt * 8) {
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t packed = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          int v = quant_code(__fmul_rn(xs[k + 4 * h + j], s));
          sum += v;
          packed |= (uint32_t)(v & 0xFF) << (8 * j);
        }
        w[h] = packed;
      }
      *reinterpret_cast<uint2*>(qrow + k) = make_uint2(w[0], w[1]);
    }
  } else {
    for (int k = tid; k < K; k += nt) {
      int v = quant_code(__fmul_rn(xs[k], s));
      sum += v;
      qrow[k] = (int8_t)v;
    }
  }
  sum = block_reduce(sum, redi, AddOpI());
  if (tid == 0) {
    *s_out = s;
    *sum_out = sum;
  }
}

// Stage row `x` [K] into xs as fp32 (with a residual type: the stored sum); returns max|x| over the block.
template <typename TIn, typename TRes = void>
BN_DEV float stage_row(const TIn* x, int K, float* xs, bool vec, void* red_scratch, const TRes* r_in = nullptr,
                       TRes* r_out = nullptr) {
  const int tid = threadIdx.x, nt = blockDim.x;
  float am = 0.0f;
  if (vec) {
    for (int k = tid * 8; k < K; k += nt * 8) {
      float v[8];
      if constexpr (std::is_void<TRes>::value) {
        RowLoader<TIn>::load(x + k, v);
      } else {
        Raw8<TIn> rx;
        Raw8<TRes> rr;
        rx.load(x + k);
        rr.load(r_in + k);
        add_residual8(v, rx, rr, r_out + k);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xs[k + j] = v[j];
        am = fmaxf(am, fabsf(v[j]));
      }
    }
  } else {
    if constexpr (std::is_void<TRes>::value) {
      for (int k = tid; k < K; k += nt) {
        const float v = RowLoader<TIn>::load1(x + k);
        xs[k] = v;
        am = fmaxf(am, fabsf(v));
      }
    } else {
      for (int k0 = tid; k0 < K; k0 += 8 * nt) {  // eight loads in flight, see Raw8
        float v[8], r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = k0 + i * nt;
          v[i] = k < K ? RowLoader<TIn>::load1(x + k) : 0.0f;
          r[i] = k < K ? RowLoader<TRes>::load1(r_in + k) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = k0 + i * nt;
          if (k < K) {
            xs[k] = v[i] = store_residual1(__fadd_rn(v[i], r[i]), r_out + k);
            am = fmaxf(am, fabsf(v[i]));
          }
        }
      }
    }
  }
  return block_reduce(am, reinterpret_cast<float*>(red_scratch), MaxOp());
}

template <typename TIn, typename TRes = void>
__global__ void __launch_bounds__(1024) k_rmsnorm_quant(const TIn* __restrict__ x, const float* __restrict__ gain,
                                                        float eps, int K, int8_t* __restrict__ q,
                                                        float* __restrict__ s_x, int32_t* __restrict__ sum_q,
                                                        int vec, const TRes* r_in, TRes* r_out) {
  extern __shared__ float xs[];
  __shared__ long long red[32];
  const long long t = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  float amax;
  if constexpr (std::is_void<TRes>::value)
    amax = stage_row<TIn>(x + t * K, K, xs, vec != 0, red);
  else
    amax = stage_row<TIn, TRes>(x + t * K, K, xs, vec != 0, red, r_in + t * K, r_out + t * K);
  quantise_staged_row(xs, K, gain, eps, q + t * K, s_x + t, sum_q + t, vec != 0, red, amax);
}

// Long fp32 rows (the FFN's h at prefill): one CTA per SM, persistent over rows blockIdx.x,
// blockIdx.x + gridDim.x, ...; two row buffers in shared memory, the next row fetched with a
// set of bulk copies (completing on the buffer's mbarrier) while the current one is reduced,
// so the row reads stream at the HBM rate instead of waiting behind each row's reduction
// chain.  Thread i owns the four elements 4 (i + QL_THREADS j) .. + 3 of every group j, read
// from shared memory with 16-byte loads; its gain values stay in registers for all rows
// (reading them from L2 per row put a memory round trip behind every element of the y pass).
// The y pass writes y over the row; the q pass writes four codes per 4-byte store.  The
// reductions use one barrier each and are the row's only barriers.  The arithmetic is
// quantise_staged_row's.  K % 4 == 0, K <= 4 QL_THREADS QL_MAXV, rows 16-byte aligned,
// 2 K floats of shared memory.
constexpr int QL_THREADS = 1024;
constexpr int QL_MAXV = 7;  // K <= 28672
constexpr int QL_PARTS = 8;  // bulk copies per row
__global__ void __launch_bounds__(QL_THREADS, 1) k_rmsnorm_quant_long(const float* __restrict__ x,
                                                                     const float* __restrict__ gain, float eps,
                                                                     int T, int K, int8_t* __restrict__ q,
                                                                     float* __restrict__ s_x,
                                                                     int32_t* __restrict__ sum_q) {
  extern __shared__ __align__(16) float ql_buf[];  // [2][K]
  __shared__ long long red[2][32];  // the two scratch areas of the reductions, used in turn
  int ra = 0;
  __shared__ __align__(8) unsigned long long ql_bar[2];  // one per row buffer: its bulk copy landed
  volatile __shared__ int ql_abort;
  const int tid = threadIdx.x;
  const int K4 = K >> 2;
  float4 gr[QL_MAXV];
#pragma unroll
  for (int j = 0; j < QL_MAXV; ++j) {
    const int k4 = tid + QL_THREADS * j;
    gr[j] = (gain != nullptr && k4 < K4) ? __ldg(reinterpret_cast<const float4*>(gain) + k4)
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  if (tid == 0) {
    mbar_init(smem_addr(&ql_bar[0]), 1);
    mbar_init(smem_addr(&ql_bar[1]), 1);
    ql_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  // A row is fetched by thread 0 as QL_PARTS bulk copies (several in flight stream faster than
  // one long copy), all completing on the buffer's barrier.
  const uint32_t row_bytes = (uint32_t)K * 4u;
  const uint32_t part = (row_bytes + 16u * QL_PARTS - 1u) / (16u * QL_PARTS) * 16u;  // multiple of 16
  auto fetch = [&](long long row, int b) {
    const uint32_t bar = smem_addr(&ql_bar[b]), dst = smem_addr(ql_buf + b * K);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(x + row * K);
    mbar_arrive_expect_tx(bar, row_bytes);
    for (uint32_t o = 0; o < row_bytes; o += part) bulk_g2s(dst + o, src + o, min(part, row_bytes - o), bar);
  };
  long long row = blockIdx.x;
  int issued = 0;
  if (tid == 0 && row < T) {
    fetch(row, 0);
    issued = 1;
  }
  for (int it = 0; row < T; ++it, row += gridDim.x) {
    const int b = it & 1;
    float4* cur = reinterpret_cast<float4*>(ql_buf + b * K);
    const long long next = row + gridDim.x;
    if (tid == 0 && next < T) {  // the other buffer was released by the last barrier of it - 1
      fetch(next, b ^ 1);
      ++issued;
    }
    // A wait that gives up is seen by every thread after the first reduction's barrier (the
    // max pass before it may read an incomplete row; its result is not used).
    if (!mbar_wait_bounded(smem_addr(&ql_bar[b]), (uint32_t)((it >> 1) & 1))) ql_abort = 1;
    float am = 0.0f;
#pragma unroll
    for (int j = 0; j < QL_MAXV; ++j) {
      const int k4 = tid + QL_THREADS * j;
      if (k4 < K4) {
        const float4 v = cur[k4];
        am = fmaxf(am, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
      }
    }
    am = block_reduce_alt(am, reinterpret_cast<float*>(red[ra++ & 1]), MaxOp());
    if (ql_abort) break;
    float a = am, inv = 1.0f;
    if (gain != nullptr) {
      float ms = 0.0f;
      if (am > 0.0f) {
        const int e = fixed_point_exponent(__dmul_rn((double)am, (double)am), K);
        const double p2e = pow2_f64(e);
        long long part = 0;
        if (K >= kFixedSmallMinN) {
          // Each term rint(v^2 2^e) < 2^51 as the bits of the fp64 sum 1.5 * 2^52 + v^2 2^e:
          // v (v 2^e) is exact (a power-of-two scaling, or below 2^-1022 where the term is 0
          // either way), so one fused multiply-add rounds exactly once, like the rounding add
          // of fixed_sq_term_t.  The bits are summed as they are (mod 2^64) and the offset of
          // every term taken off once.
          unsigned long long bits = 0ull;
          int n = 0;
#pragma unroll
          for (int j = 0; j < QL_MAXV; ++j) {
            const int k4 = tid + QL_THREADS * j;
            if (k4 < K4) {
              const float4 v = cur[k4];
              const double d0 = (double)v.x, d1 = (double)v.y, d2 = (double)v.z, d3 = (double)v.w;
              constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52
              bits += (unsigned long long)__double_as_longlong(__fma_rn(d0, __dmul_rn(d0, p2e), kRound)) +
                      (unsigned long long)__double_as_longlong(__fma_rn(d1, __dmul_rn(d1, p2e), kRound)) +
                      (unsigned long long)__double_as_longlong(__fma_rn(d2, __dmul_rn(d2, p2e), kRound)) +
                      (unsigned long long)__double_as_longlong(__fma_rn(d3, __dmul_rn(d3, p2e), kRound));
              n += 4;
            }
          }
          part = (long long)(bits - (unsigned long long)n * 0x4338000000000000ull);
        } else {
#pragma unroll
          for (int j = 0; j < QL_MAXV; ++j) {
            const int k4 = tid + QL_THREADS * j;
            if (k4 < K4) {
              const float4 v = cur[k4];
              part += fixed_sq_term(v.x, p2e) + fixed_sq_term(v.y, p2e) + fixed_sq_term(v.z, p2e) +
                      fixed_sq_term(v.w, p2e);
            }
          }
        }
        ms = fixed_point_mean(block_reduce_alt(part, red[ra++ & 1], AddOpLL()), e, K);
      }
      inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, eps)));
      float ay = 0.0f;
#pragma unroll
      for (int j = 0; j < QL_MAXV; ++j) {
        const int k4 = tid + QL_THREADS * j;
        if (k4 < K4) {
          float4 v = cur[k4];
          v.x = __fmul_rn(__fmul_rn(v.x, inv), gr[j].x);
          v.y = __fmul_rn(__fmul_rn(v.y, inv), gr[j].y);
          v.z = __fmul_rn(__fmul_rn(v.z, inv), gr[j].z);
          v.w = __fmul_rn(__fmul_rn(v.w, inv), gr[j].w);
          ay = fmaxf(ay, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
          cur[k4] = v;  // y, read by the q pass
        }
      }
      fence_proxy_async_smem();  // this thread's y writes ordered before the buffer's next bulk copy
      a = block_reduce_alt(ay, reinterpret_cast<float*>(red[ra++ & 1]), MaxOp());
    }
    const float s = __fdiv_rn(127.0f, fmaxf(a, 1e-5f));
    // quant_code's steps with its offset kept: the fp32 bits of clamp(p) + 1.5 * 2^23 are
    // 0x4B400000 + code, so their low byte is the code's byte; the bits are summed as they are
    // (mod 2^32) and the offset of every element taken off once.
    uint32_t cbits = 0u;
    int n = 0;
    uint32_t* qrow = reinterpret_cast<uint32_t*>(q + row * K);
#pragma unroll
    for (int j = 0; j < QL_MAXV; ++j) {
      const int k4 = tid + QL_THREADS * j;
      if (k4 < K4) {
        const float4 y = cur[k4];
        const float p[4] = {__fmul_rn(y.x, s), __fmul_rn(y.y, s), __fmul_rn(y.z, s), __fmul_rn(y.w, s)};
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = p[i] == p[i] ? fminf(fmaxf(p[i], -128.0f), 127.0f) : 0.0f;  // NaN: code 0
          b[i] = __float_as_uint(__fadd_rn(c, 12582912.0f));
        }
        cbits += (b[0] + b[1]) + (b[2] + b[3]);
        n += 4;
        qrow[k4] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      }
    }
    const int sum = block_reduce_alt((int)(cbits - (uint32_t)n * 0x4B400000u), reinterpret_cast<int*>(red[ra++ & 1]),
                                     AddOpI());
    if (tid == 0) {
      s_x[row] = s;
      sum_q[row] = sum;
    }
    // The buffer is refilled by the fetch of iteration it + 1, issued after the barrier of the
    // reduction above, which every thread reaches after its last read of the buffer.
  }
  // After a wait gave up, the copies still in flight land (fixed limit) before the CTA exits.
  if (tid == 0 && ql_abort)
    for (int k = (issued > 2 ? issued - 2 : 0); k < issued; ++k) mbar_drain(smem_addr(&ql_bar[k & 1]), (uint32_t)((k >> 1) & 1));
}

// The same arithmetic with W warps per row (W = 1, 2 or 4) and 8 / W rows per 256-thread
// CTA, for rows of K <= 2048 W values (K a multiple of 8, 16-byte aligned rows).  Lane l of
// the row's warp `rank` holds elements 8 (l + 32 (rank + W j)) .. +7, j < 8, in registers, so
// the row is read once; the reductions are warp shuffles, joined across the W warps by one
// named barrier each (two scratch halves used in turn).  Many rows are in flight per SM,
// which hides the latency of the loads and of the reduction chain.
constexpr int QW_THREADS = 256;
constexpr int QW_GROUPS = 8;

template <int W, typename T, typename Op>
BN_DEV T qw_reduce(T v, T* slots, int& flip, int bar_id, int rank, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (W == 1) return v;
  T* b = slots + flip * W;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0) b[rank] = v;
  named_sync(bar_id, 32 * W);
  T r = b[0];
#pragma unroll
  for (int i = 1; i < W; ++i) r = op(r, b[i]);
  return r;
}

template <typename TIn, int W>
__global__ void __launch_bounds__(QW_THREADS) k_rmsnorm_quant_warps(const TIn* __restrict__ x,
                                                                   const float* __restrict__ gain, float eps, int T,
                                                                   int K, int8_t* __restrict__ q,
                                                                   float* __restrict__ s_x, int32_t* __restrict__ sum_q) {
  constexpr int ROWS = QW_THREADS / 32 / W;
  __shared__ float redf[ROWS][2 * W];
  __shared__ long long redl[ROWS][2 * W];
  __shared__ int redi[ROWS][2 * W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = warp / W, rank = warp - rr * W;
  const long long t = (long long)blockIdx.x * ROWS + rr;
  pdl_launch_dependents();
  pdl_wait();
  if (t >= T) return;  // every warp of the row leaves together
  const int bar = 1 + rr;
  int ff = 0, fl = 0, fi = 0;
  const TIn* xr = x + t * K;
  float v[QW_GROUPS][8];
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < QW_GROUPS; ++j) {
    const int k = 8 * (lane + 32 * (rank + W * j));
    if (k < K) {
      RowLoader<TIn>::load(xr + k, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[j][i]));
  }
  am = qw_reduce<W>(am, &redf[rr][0], ff, bar, rank, MaxOp());
  float a = am;
  if (gain != nullptr) {
    float ms = 0.0f;
    if (am > 0.0f) {
      const double M = __dmul_rn((double)am, (double)am);
      const int e = fixed_point_exponent(M, K);
      const double p2e = pow2_f64(e);
      long long part = 0;
      if (K >= kFixedSmallMinN) {
#pragma unroll
        for (int j = 0; j < QW_GROUPS; ++j)
          if (8 * (lane + 32 * (rank + W * j)) < K) {
#pragma unroll
            for (int i = 0; i < 8; ++i) part += fixed_sq_term_t<true>(v[j][i], p2e);
          }
      } else {
#pragma unroll
        for (int j = 0; j < QW_GROUPS; ++j)
          if (8 * (lane + 32 * (rank + W * j)) < K) {
#pragma unroll
            for (int i = 0; i < 8; ++i) part += fixed_sq_term(v[j][i], p2e);
          }
      }
      ms = fixed_point_mean(qw_reduce<W>(part, &redl[rr][0], fl, bar, rank, AddOpLL()), e, K);
    }
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, eps)));
    float ay = 0.0f;
#pragma unroll
    for (int j = 0; j < QW_GROUPS; ++j) {
      const int k = 8 * (lane + 32 * (rank + W * j));
      if (k < K) {
        const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain + k));
        const float4 g1 = __ldg(reinterpret_cast<const float4*>(gain + k + 4));
        const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][i] = __fmul_rn(__fmul_rn(v[j][i], inv), g[i]);
          ay = fmaxf(ay, fabsf(v[j][i]));
        }
      }
    }
    a = qw_reduce<W>(ay, &redf[rr][0], ff, bar, rank, MaxOp());
  }
  const float s = __fdiv_rn(127.0f, fmaxf(a, 1e-5f));
  int sum = 0;
  int8_t* qr = q + t * K;
#pragma unroll
  for (int j = 0; j < QW_GROUPS; ++j) {
    const int k = 8 * (lane + 32 * (rank + W * j));
    if (k < K) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int qv = quant_code(__fmul_rn(v[j][i], s));
        sum += qv;
        w[i >> 2] |= (uint32_t)(qv & 0xFF) << (8 * (i & 3));
      }
      *reinterpret_cast<uint2*>(qr + k) = make_uint2(w[0], w[1]);
    }
  }
  sum = qw_reduce<W>(sum, &redi[rr][0], fi, bar, rank, AddOpI());
  if (rank == 0 && lane == 0) {
    s_x[t] = s;
    sum_q[t] = sum;
  }
}

// Residual addition + norm + codes (see the top of the file) for rows of up to 1024 W values: W warps
// per row, 32 values a thread in registers, eight consecutive ones at a time.  ALIGNED: K is a
// multiple of 8.  Otherwise the groups of eight are those of the whole tensor, on which its 16-byte
// boundaries lie: a row begins `off` values into its first group and takes K + off <= 1024 W places; its
// first and last group, where not whole, are read and written value by value.
//
// Bound by HBM if enough loads are in flight: all of a thread's loads stand before its first store
// (r_out may be r_in, so the compiler keeps their order), and 32 values a thread leave room for 24 or 32
// warps an SM.  Then the instructions count: the terms of the sum are one fused multiply-add each with
// the rounding offset taken off once, codes and their sum come from the bits of the rounding addition
// (as in k_rmsnorm_quant_long), and additions and products are done two at a time.
// T = K = 8192, bf16: 150 us with 64 values a thread and one load, add and store after the other,
// 94 us with the loads first and 32 values, 82 us with fewer instructions, 80.4 us (5.8 TB/s) with the
// warp-wide reduction instruction (K = 12288: 75 instead of 89 us).  These are repeated calls over the same
// buffers, part of whose writes stay in L2; over inputs of several seeds in turn 81 to 90 us (5.2 to 5.8 TB/s).
// Values behind the row are 0: their terms and codes are those of 0 and cancel with the offsets.
// Pairs of fp32 in one 64-bit register, one instruction for both.
BN_DEV uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BN_DEV void halves(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
BN_DEV uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BN_DEV uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Reductions over the W warps of a row by the warp-wide reduction instruction (of 32-bit integers:
// non-negative floats order like their bits; 64-bit sums go in three pieces that 32 lanes cannot
// overflow), first over the lanes, then over the warps' results, one per lane.
struct RowMax {
  typedef uint32_t T;
  BN_DEV static T warp(T v) { return __reduce_max_sync(0xffffffffu, v); }
};
struct RowSum {
  typedef int T;
  BN_DEV static T warp(T v) { return __reduce_add_sync(0xffffffffu, v); }
};
struct RowSum64 {  // of numbers from 0 to 2^63 - 1 whose sum is too
  typedef unsigned long long T;
  BN_DEV static T warp(T v) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0xFFFFFFu), b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 24) & 0xFFFFFFu);
    return a + ((T)b << 24) + ((T)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 48)) << 48);
  }
};
template <int W, typename Op>
BN_DEV typename Op::T row_reduce(typename Op::T v, typename Op::T* slots, int& flip, int bar_id, int rank) {
  v = Op::warp(v);
  if (W == 1) return v;
  typename Op::T* b = slots + flip * W;
  flip ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0) b[rank] = v;
  named_sync(bar_id, 32 * W);
  return Op::warp(lane < W ? b[lane] : 0);
}
BN_HOST_DEV constexpr int qw_threads(int W) { return W > 8 ? 32 * W : QW_THREADS; }
template <typename TIn, typename TRes, int W, bool ALIGNED>
__global__ void __launch_bounds__(qw_threads(W), W > 8 ? 2 : (ALIGNED && sizeof(TIn) + sizeof(TRes) < 8 ? 4 : 3)) k_add_rmsnorm_quant(const TIn* __restrict__ x, const float* __restrict__ gain, float eps,
                                                                  int T, int K, int8_t* __restrict__ q, float* __restrict__ s_x,
                                                                  int32_t* __restrict__ sum_q, const TRes* r_in, TRes* r_out) {
  constexpr int ROWS = qw_threads(W) / 32 / W, N = 32;
  __shared__ uint32_t redf[ROWS][2 * W];
  __shared__ unsigned long long redl[ROWS][2 * W];
  __shared__ int redi[ROWS][2 * W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = warp / W, rank = warp - rr * W;
  const long long t = (long long)blockIdx.x * ROWS + rr;
  pdl_launch_dependents();
  pdl_wait();
  if (t >= T) return;  // every warp of the row leaves together
  const int bar = 1 + rr;
  int ff = 0, fl = 0, fi = 0;
  const int off = ALIGNED ? 0 : (int)((t * K) & 7);
  auto at = [&](int j) { return 8 * (lane + 32 * (rank + W * j)) - off; };  // first value of this thread's group j
  auto whole = [&](int j) { return ALIGNED ? at(j) < K : at(j) >= 0 && at(j) + 8 <= K; };
  auto has = [&](int j, int i) { return (unsigned)(at(j) + i) < (unsigned)K; };
  auto any = [&](int j) { return 256 * (rank + W * j) - off < K; };  // whether the warp has any of them
  uint64_t v[N / 2];
  {
    Raw8<TIn> rx[N / 8];
    Raw8<TRes> rr8[N / 8];
#pragma unroll
    for (int j = 0; j < N / 8; ++j)
      if (whole(j)) {
        rx[j].load(x + t * K + at(j));
        rr8[j].load(r_in + t * K + at(j));
      }
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
      float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (whole(j)) {
        add_residual8(o, rx[j], rr8[j], r_out + t * K + at(j));
      } else if (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const long long at1 = t * K + at(j) + i;
          if (has(j, i)) o[i] = store_residual1(__fadd_rn(RowLoader<TIn>::load1(x + at1), RowLoader<TRes>::load1(r_in + at1)), r_out + at1);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = pair(o[2 * i], o[2 * i + 1]);
    }
  }
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float lo, hi;
    halves(v[i], lo, hi);
    am = fmaxf(fmaxf(am, fabsf(lo)), fabsf(hi));
  }
  am = __uint_as_float(row_reduce<W, RowMax>(__float_as_uint(am), &redf[rr][0], ff, bar, rank));
  float a = am;
  uint64_t seen = 0ull;  // sums of this thread's y: finite only if every one of them is
  if (gain != nullptr) {
    float ms = 0.0f;
    if (am > 0.0f) {
      const int e = fixed_point_exponent(__dmul_rn((double)am, (double)am), K);
      const double p2e = pow2_f64(e);
      unsigned long long bits = 0ull;
#pragma unroll
      for (int j = 0; j < N / 8; ++j) {
        if (!any(j)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          halves(v[4 * j + i], lo, hi);
          if (K >= kFixedSmallMinN) {
            const double d0 = (double)lo, d1 = (double)hi;
            bits += (unsigned long long)__double_as_longlong(__fma_rn(d0, __dmul_rn(d0, p2e), 6755399441055744.0)) +
                    (unsigned long long)__double_as_longlong(__fma_rn(d1, __dmul_rn(d1, p2e), 6755399441055744.0));
          } else {
            bits += (unsigned long long)(fixed_sq_term(lo, p2e) + fixed_sq_term(hi, p2e));
          }
        }
        if (K >= kFixedSmallMinN) bits -= 8 * 0x4338000000000000ull;
      }
      ms = fixed_point_mean((long long)row_reduce<W, RowSum64>(bits, &redl[rr][0], fl, bar, rank), e, K);
    }
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, eps)));
    const uint64_t inv2 = pair(inv, inv);
    float ay = 0.0f;
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
      if (!any(j)) continue;
      uint64_t g[4];
      if constexpr (ALIGNED) {
        const ulonglong2* p = reinterpret_cast<const ulonglong2*>(gain + (at(j) < K ? at(j) : 0));
        const ulonglong2 g0 = __ldg(p), g1 = __ldg(p + 1);
        g[0] = g0.x, g[1] = g0.y, g[2] = g1.x, g[3] = g1.y;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[i] = pair(__ldg(gain + (has(j, 2 * i) ? at(j) + 2 * i : 0)), __ldg(gain + (has(j, 2 * i + 1) ? at(j) + 2 * i + 1 : 0)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t& y = v[4 * j + i];
        y = mul_pair(mul_pair(y, inv2), g[i]);
        seen = add_pair(seen, y);
        float lo, hi;
        halves(y, lo, hi);
        ay = fmaxf(fmaxf(ay, fabsf(lo)), fabsf(hi));
      }
    }
    a = __uint_as_float(row_reduce<W, RowMax>(__float_as_uint(ay), &redf[rr][0], ff, bar, rank));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) seen = add_pair(seen, v[i]);
  }
  // |y| <= a for every number y, so |y s| rounds to at most 127 and needs no clamp; what does need it
  // is a NaN or an infinity, which the sum shows.
  const float s = __fdiv_rn(127.0f, fmaxf(a, 1e-5f));
  const uint64_t s2 = pair(s, s), round2 = pair(12582912.0f, 12582912.0f);
  float slo, shi;
  halves(seen, slo, shi);
  const bool finite = fabsf(__fadd_rn(slo, shi)) < INFINITY;
  uint32_t cbits = 0;
  int8_t* qr = q + t * K;
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    if (!any(j)) continue;
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint64_t p = mul_pair(v[4 * j + i], s2);
      float lo, hi;
      if (!finite) {
        halves(p, lo, hi);
        p = pair(lo == lo ? fminf(fmaxf(lo, -128.0f), 127.0f) : 0.0f, hi == hi ? fminf(fmaxf(hi, -128.0f), 127.0f) : 0.0f);
      }
      halves(add_pair(p, round2), lo, hi);
      b[2 * i] = __float_as_uint(lo);
      b[2 * i + 1] = __float_as_uint(hi);
      cbits += b[2 * i] + b[2 * i + 1];
    }
    cbits -= 8 * 0x4B400000u;
    if (whole(j)) {
      *reinterpret_cast<uint2*>(qr + at(j)) =
          make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                     __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    } else if (!ALIGNED) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(j, i)) qr[at(j) + i] = (int8_t)b[i];
    }
  }
  const int sum = row_reduce<W, RowSum>((int)cbits, &redi[rr][0], fi, bar, rank);
  if (rank == 0 && lane == 0) {
    s_x[t] = s;
    sum_q[t] = sum;
  }
}

}  // namespace bitnet
