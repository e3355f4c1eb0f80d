// The paged attention of attn_paged.cuh for requests with many query rows (chunks of a prompt), on
// the 5th-generation tensor cores.  Tiles of 256 query rows, units of 128 cache rows, the same line
// of units with equal shares, one CTA per SM:
//   warps 0-3, 4-7  softmax of the tile's rows 0-127 and 128-255, one thread per row: scores from
//                   tensor memory, maximum, weights (bf16) back to tensor memory; the output at the end
//   warp 8          tcgen05.mma: S = Q K^T (both operands in shared memory), O += P V (P in tensor memory)
//   warp 9          TMA loads of K and V, page by page, into a ring of 32 KB slots
//   warp 10         TMA loads of the next tile's Q
// The two halves take turns: while one half's softmax runs, the tensor core does the other's
// products.  Tensor memory (512 columns): S of each half 128 columns, of which P takes the first 64
// once the scores are in registers; O of each half 128 columns.
//
// The running maximum of a row moves only when the scores outgrow it by 2^8: until then the weights
// are at most 2^8, which fp32 sums and bf16's exponent hold without loss, and O needs no rescaling.
// The weights are rounded to bf16 for the second product (the tensor core's operand type; half a
// step is 2^-8 of each weight); the row sum adds the unrounded weights in fp32.
//
// Pages that no row sees and page ids out of range are loaded as zeros (a page coordinate beyond
// the tensor: the copy fills zeros).  Rows at and behind kv in the last page may hold anything: their
// scores are masked, their V rows are overwritten with zeros in shared memory.
#pragma once
#include <cuda.h>

#include "attn_paged.cuh"
#include "common.cuh"
#include "gemm_tc.cuh"

namespace bitnet {

// A block of at most 128 query rows is TB tokens of GB query heads, row = token * GB + head, so that
// one box of q holds it: GB = min(G, 128), TB = 128 / GB; NB = ceil(G / 128) blocks cover a token's
// heads.  A tile is two consecutive blocks of a request and key/value head.
struct ChunkTiles {
  static constexpr int M = 256, U = 128;
  BN_DEV static int blocks(const PagedArgs& a, int n) { return (n + a.TB - 1) / a.TB * a.NB; }
  BN_DEV static int tiles(const PagedArgs& a, int n) { return (blocks(a, n) + 1) >> 1; }
  BN_DEV static int visible(const PagedArgs& a, int n, int kv, int j) {
    const int b = 2 * j + 1, group = a.NB == 1 ? b : b / a.NB;
    return max(0, kv - n + min(n, (group + 1) * a.TB));
  }
};
// A row of a tile: its token and head (of the G), and whether the request has it.
struct ChunkRow {
  int t, g;
  bool there;
};
BN_DEV ChunkRow chunk_row(const PagedArgs& a, int n, int tile, int row) {
  const int b = 2 * tile + (row >> 7), i = row & 127, ti = i / a.GB;
  ChunkRow r;
  r.t = (a.NB == 1 ? b : b / a.NB) * a.TB + ti;
  r.g = (a.NB == 1 ? 0 : (b % a.NB) * 128) + i - ti * a.GB;
  r.there = ti < a.TB && r.t < n && r.g < a.G;
  return r;
}

constexpr int PC_M = ChunkTiles::M;
constexpr int PC_U = ChunkTiles::U;
constexpr int PC_THREADS = 384;
constexpr int PC_MMA_WARP = 8, PC_KV_WARP = 9, PC_Q_WARP = 10;
constexpr int PC_SLOTS = 5;
constexpr int PC_EARLY = 96;  // weights that the second product starts with, while the others are computed
constexpr uint32_t PC_TILE_BYTES = 128 * 256;  // 128 rows of 128 bf16: two 64-column halves of 128-byte rows, swizzled
constexpr int PC_SMEM = (2 + PC_SLOTS) * PC_TILE_BYTES + 1024;
constexpr int PC_PART = PC_M * (PG_D + 2);     // floats of a partial tile: values [32][256 rows][4], maxima, sums
constexpr float PC_GROW = 8.0f / PG_SCALE_LOG2;

struct alignas(64) PagedMaps {
  CUtensorMap k, v;  // bf16 [n_pages][Hkv][P][128], box {64, min(P, 128), 1, 1}, 128-byte swizzle
  CUtensorMap q;     // bf16 [T][Hkv][G][128], box {64, GB, 1, TB}, the same
};

// bf16 x bf16 -> fp32, M = N = 128; `mn_b`: B is stored with its N index contiguous
BN_DEV constexpr uint32_t pc_idesc(bool mn_b) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((mn_b ? 1u : 0u) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}
// Descriptor of a V tile as B operand (d contiguous): 64-column halves 16384 bytes apart, groups of
// eight cache rows 1024 bytes apart.
BN_DEV uint64_t pc_desc_v(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
BN_DEV void umma_bf16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
BN_DEV void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
BN_DEV void tma_load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
BN_DEV void tmem_ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
BN_DEV void tmem_ld16f(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
BN_DEV void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
BN_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 at a time: one instruction each.
BN_DEV uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BN_DEV void unpack_f32x2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
BN_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
BN_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// One lane of a converged warp.  Unlike lane == 0 this tells the compiler that a single thread
// follows, which lets it keep the operands of tcgen05.mma in uniform registers.
BN_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P1;\n\telect.sync _|P1, 0xffffffff;\n\tselp.b32 %0, 1, 0, P1;\n\t}" : "=r"(p));
  return p != 0;
}

// The whole warp waits; false if any lane's wait ran out.
BN_DEV bool warp_wait(uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity)); }

__global__ void __launch_bounds__(PC_THREADS, 1) k_attn_paged_chunk(const __grid_constant__ PagedMaps maps, const PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long s_bars[2 * PC_SLOTS + 9];
  __shared__ long long s_walk[4], s_red[32];
  volatile __shared__ int s_abort;
  __shared__ int s_issued, s_q_issued;  // ring slots and tiles of Q that were loaded (for the drain after an abort)
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, ring = base + 2 * PC_TILE_BYTES;
  const uint32_t bars = smem_addr(s_bars);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (PC_SLOTS + s); };
  const uint32_t bar0 = bars + 8u * 2 * PC_SLOTS;
  const uint32_t q_full = bar0, q_empty = bar0 + 8, mma_done = bar0 + 16;
  auto s_full = [&](int w) { return bar0 + 24u + 8u * w; };
  auto p_full = [&](int w, int part) { return bar0 + 40u + 8u * (2 * w + part); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < PC_SLOTS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w, 0), 4);
      mbar_init(p_full(w, 1), 4);
    }
    s_abort = 0;
    s_issued = 0;
    s_q_issued = 0;
    fence_mbar_init();
  }
  if (warp == PC_MMA_WARP) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_launch_dependents();
  pdl_wait();
  PagedWalk<ChunkTiles> w;
  w.begin(a, gridDim.x, s_walk, s_red);
  if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);

  // The launch gives every thread at most 168 registers (65536 / 384); the softmax warps, which hold a
  // row of scores, take 208: 8 * 32 * 208 + 4 * 32 * 80 <= 384 * 168 holds for the whole block.
  if (warp < 8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");

  if (warp < 8) {
    // ------------------------------------------------------------ softmax, one row per thread
    const int half = warp >> 2, row = half * 128 + (warp & 3) * 32 + lane;
    const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t_lane + half * 128, tO = tmem + t_lane + 256 + half * 128;
    uint32_t ph = 0;
    bool ok = true;
    while (w.left > 0 && ok) {
      const int nu = w.units(a), cnt = (int)min(w.left, (long long)(nu - w.unit));
      if (2 * w.tile + half < ChunkTiles::blocks(a, w.n)) {
        const ChunkRow r = chunk_row(a, w.n, w.tile, row);
        const int lim = r.there ? max(0, w.kv - w.n + r.t + 1) : 0x7FFFFFFF;  // rows of the cache that this row sees
        float m = -INFINITY, l = 0.0f;  // running maximum of the raw scores (may trail by 2^8), sum
        for (int it = 0; it < cnt; ++it) {
          ok = warp_wait(s_full(half), ph) && !s_abort;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ph ^= 1u;
          tc_fence_after();
          float s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
          tmem_wait_ld();
          const int col0 = (w.unit + it) * PC_U;
          if (__any_sync(0xffffffffu, lim < col0 + PC_U)) {
            const int rel = lim - col0;
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = c < rel ? s[c] : -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 128; c += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = c + 4 + k < 128 ? fmaxf(fmaxf(mx[k], s[c + k]), s[c + 4 + k]) : fmaxf(mx[k], s[c + k]);
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool grow = mt > __fadd_rn(m, PC_GROW);  // from -inf: at the first score
          if (__any_sync(0xffffffffu, grow)) {
            float alpha = 1.0f;
            if (grow) {
              alpha = exp2_approx(__fmul_rn(__fsub_rn(m, mt), PG_SCALE_LOG2));
              m = mt;
              l = __fmul_rn(l, alpha);
            }
            if (it > 0) {  // this row's O: every product so far has ended, S(it) was behind them
#pragma unroll 1
              for (int c = 0; c < 128; c += 16) {
                float o[16];
                tmem_ld16f(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __fmul_rn(o[k], alpha);
                tmem_st16(tO + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          const float mu = m == -INFINITY ? 0.0f : -__fmul_rn(m, PG_SCALE_LOG2);
          const uint64_t sc2 = pack_f32x2(PG_SCALE_LOG2, PG_SCALE_LOG2), mu2 = pack_f32x2(mu, mu);
          uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float x, y;
              unpack_f32x2(fma_f32x2(pack_f32x2(s[c + k], s[c + k + 1]), sc2, mu2), x, y);
              x = exp2_approx(x);
              y = exp2_approx(y);
              sum2[(k >> 1) & 1] = add_f32x2(sum2[(k >> 1) & 1], pack_f32x2(x, y));
              p[k >> 1] = pack_bf16(x, y);
            }
            tmem_st16(tS + (c >> 1), p);
            if (c >= PC_EARLY - 32) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && (c == PC_EARLY - 32 || c == 96)) mbar_arrive(p_full(half, c == 96));
            }
          }
          float x, y;
          unpack_f32x2(add_f32x2(sum2[0], sum2[1]), x, y);
          l = __fadd_rn(l, __fadd_rn(x, y));
        }
        if (!ok) break;
        ok = warp_wait(s_full(half), ph) && !s_abort;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ph ^= 1u;
        tc_fence_after();
        if (cnt == nu) {
          const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);  // NaN stays
          const long long off = ((long long)(w.t0 + r.t) * a.Hq + w.head * a.G + r.g) * PG_D;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
            if (!r.there) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = l == 0.0f ? 0.0f : __fmul_rn(o[k], inv);
            if (a.out_dtype == BITNET_BF16) {
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + off + c);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                    pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + off + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        } else {
          float* part = a.part + ((long long)blockIdx.x * 2 + (w.unit > 0 ? 0 : 1)) * PC_PART;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<float4*>(part)[(c / 4 + k) * PC_M + row] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          part[PC_M * PG_D + row] = m;
          part[PC_M * PG_D + PC_M + row] = l;
        }
      }
      if (threadIdx.x == 0 && w.unit > 0 && w.unit + cnt == nu)
        a.desc[blockIdx.x] = make_int4((int)((w.pos - w.unit) / w.per), w.seq, w.head, w.tile);
      w.advance(a, cnt, nu);
    }
    if (!ok) s_abort = 1;
  } else if (warp == PC_MMA_WARP) {
    // ------------------------------------------------------------ products
    int slot = 0;
    uint32_t ph_s = 0, ph_q = 0, ph_p[2] = {0, 0};
    bool ok = true;
    auto next_slot = [&]() {
      if (++slot == PC_SLOTS) {
        slot = 0;
        ph_s ^= 1u;
      }
    };
    auto scores = [&](int h, uint32_t k_addr) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        umma_bf16_ss(tmem + h * 128, umma_desc_sw128(sQ + h * PC_TILE_BYTES + off), umma_desc_sw128(k_addr + off), pc_idesc(false),
                     kk > 0);
      }
    };
    auto values = [&](int h, uint32_t v_addr, bool first, int k0, int k1) {
#pragma unroll
      for (int kk = k0; kk < k1; ++kk)
        umma_bf16_ts(tmem + 256 + h * 128, tmem + h * 128 + kk * 8, pc_desc_v(v_addr + kk * 2048), pc_idesc(true),
                     (first && kk == 0) ? 0u : 1u);
    };
    while (w.left > 0 && ok && !s_abort) {
      const int nu = w.units(a), cnt = (int)min(w.left, (long long)(nu - w.unit));
      const int nh = 2 * w.tile + 1 < ChunkTiles::blocks(a, w.n) ? 2 : 1;
      ok = warp_wait(q_full, ph_q) && warp_wait(full(slot), ph_s);
      if (!ok) break;
      ph_q ^= 1u;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t k = ring + slot * PC_TILE_BYTES;
        for (int h = 0; h < nh; ++h) {
          scores(h, k);
          if (h == nh - 1) {
            umma_commit(empty(slot));
            if (cnt == 1) umma_commit(q_empty);
          }
          umma_commit(s_full(h));
        }
      }
      __syncwarp();
      next_slot();
      for (int it = 0; it < cnt && ok; ++it) {
        const int vs = slot;
        const uint32_t v = ring + vs * PC_TILE_BYTES;
        ok = warp_wait(full(vs), ph_s);
        if (!ok) break;
        next_slot();
        // rows behind kv in the request's last page
        const int row0 = (w.unit + it) * PC_U, tail = w.kv - row0;
        if (tail > 0 && tail < PC_U && (tail & (a.P - 1))) {
          const int end = min(PC_U, (tail + a.P - 1) & ~(a.P - 1));
          for (int i = tail * 16 + lane; i < end * 16; i += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(v + ((i >> 3) & 1) * 16384 + (i >> 4) * 128 + (i & 7) * 16), "r"(0)
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
        }
        for (int h = 0; h < nh; ++h) {
          if (h == 0 && it + 1 < cnt) ok = warp_wait(full(slot), ph_s);
          ok = ok && warp_wait(p_full(h, 0), ph_p[h]);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) values(h, v, it == 0, 0, PC_EARLY / 16);
          __syncwarp();
          ok = warp_wait(p_full(h, 1), ph_p[h]);
          if (!ok) break;
          ph_p[h] ^= 1u;
          tc_fence_after();
          if (elect_one()) {
            values(h, v, false, PC_EARLY / 16, 8);
            if (it + 1 < cnt) scores(h, ring + slot * PC_TILE_BYTES);
            if (h == nh - 1) {
              umma_commit(empty(vs));
              if (it + 1 < cnt) umma_commit(empty(slot));
              if (it + 2 == cnt) umma_commit(q_empty);
            }
            umma_commit(s_full(h));
          }
          __syncwarp();
        }
        if (it + 1 < cnt) next_slot();
      }
      w.advance(a, cnt, nu);
    }
    if (!ok) s_abort = 1;
  } else if (warp == PC_KV_WARP) {
    // ------------------------------------------------------------ K and V
    const int log2b = min(a.log2P, 7), npg = 1 << (7 - log2b);  // rows of a copy, copies per unit and 64-column half
    int slot = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    while (w.left > 0 && ok && !s_abort) {
      const int nu = w.units(a), cnt = (int)min(w.left, (long long)(nu - w.unit));
      const int vis = ChunkTiles::visible(a, w.n, w.kv, w.tile);
      const int* trow = a.table + (long long)w.seq * a.width;
      // this lane's page of a unit: its id, or n_pages (zeros) where there is none to see
      auto page_of = [&](int u) {
        const int row = u * PC_U + (lane << log2b);
        if (lane >= npg || row >= vis) return a.n_pages;
        const int id = __ldg(trow + (row >> a.log2P));
        if (id >= 0 && id < a.n_pages) return id;
        flag_index_error();
        return a.n_pages;
      };
      int page = page_of(w.unit);
      for (int it = 0; it < cnt && ok; ++it) {
        const int row = (w.unit + it) * PC_U + (lane << log2b);
        const int cur = page;
        if (it + 1 < cnt) page = page_of(w.unit + it + 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = warp_wait(empty(slot), ph);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full(slot), PC_TILE_BYTES);
          __syncwarp();
          if (lane < npg) {
            const uint32_t dst = ring + slot * PC_TILE_BYTES + (lane << log2b) * 128;
            const void* map = kv ? &maps.v : &maps.k;
            tma_load_4d(dst, map, 0, row & (a.P - 1), w.head, cur, full(slot));
            tma_load_4d(dst + 16384, map, 64, row & (a.P - 1), w.head, cur, full(slot));
          }
          ++issued;
          if (++slot == PC_SLOTS) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      w.advance(a, cnt, nu);
    }
    if (!ok) s_abort = 1;
    if (lane == 0) s_issued = issued;
  } else if (warp == PC_Q_WARP) {
    // ------------------------------------------------------------ Q
    uint32_t ph = 1;
    bool ok = true;
    while (w.left > 0 && ok && !s_abort) {
      const int nu = w.units(a), cnt = (int)min(w.left, (long long)(nu - w.unit));
      ok = warp_wait(q_empty, ph);
      if (!ok) break;
      ph ^= 1u;
      if (lane == 0) {
        const int nh = 2 * w.tile + 1 < ChunkTiles::blocks(a, w.n) ? 2 : 1;
        mbar_arrive_expect_tx(q_full, nh * a.TB * a.GB * PG_D * 2);
        for (int h = 0; h < nh; ++h) {
          const ChunkRow r = chunk_row(a, w.n, w.tile, h * 128);
          const uint32_t dst = sQ + h * PC_TILE_BYTES;
          tma_load_4d(dst, &maps.q, 0, r.g, w.head, w.t0 + r.t, q_full);
          tma_load_4d(dst + 16384, &maps.q, 64, r.g, w.head, w.t0 + r.t, q_full);
        }
        ++s_q_issued;
      }
      __syncwarp();
      w.advance(a, cnt, nu);
    }
    if (!ok) s_abort = 1;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (s_abort) {
    // every issued product ends and every issued copy lands before tensor memory is released
    if (warp == PC_MMA_WARP && lane == 0) {
      umma_commit(mma_done);
      mbar_drain(mma_done, 0);
    }
    if (warp == PC_Q_WARP && lane == 0 && s_q_issued > 0) mbar_drain(q_full, (uint32_t)((s_q_issued - 1) & 1));
    if (warp == PC_KV_WARP && lane == 0)
      for (int k = max(0, s_issued - PC_SLOTS); k < s_issued; ++k) mbar_drain(full(k % PC_SLOTS), (uint32_t)((k / PC_SLOTS) & 1));
  }
  __syncthreads();
  if (warp == PC_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the tile that CTA c finished (blockIdx.x), as k_attn_paged_few_join does.
// Thread: a row and 16 of its dimensions (blockIdx.y).
__global__ void __launch_bounds__(PC_M) k_attn_paged_chunk_join(const PagedArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x;
  const int4 d = a.desc[c];
  if (d.x < 0) return;
  int t0, n, kv;
  paged_request(a, d.y, t0, n, kv);
  const int row = threadIdx.x, g0 = blockIdx.y * 4;
  const ChunkRow r = chunk_row(a, n, d.w, row);
  if (!r.there) return;
  auto part = [&](int i) { return a.part + ((long long)i * 2 + (i == d.x ? 1 : 0)) * PC_PART; };
  float m = -INFINITY;
  for (int i = d.x; i <= c; ++i) m = fmaxf(m, part(i)[PC_M * PG_D + row]);
  const float mu = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, o[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.0f;
  for (int i = d.x; i <= c; ++i) {
    const float* p = part(i);
    const float f = exp2_approx(__fmul_rn(__fsub_rn(p[PC_M * PG_D + row], mu), PG_SCALE_LOG2));
    l = __fmaf_rn(p[PC_M * PG_D + PC_M + row], f, l);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = reinterpret_cast<const float4*>(p)[(g0 + k) * PC_M + row];
      o[4 * k] = __fmaf_rn(x.x, f, o[4 * k]);
      o[4 * k + 1] = __fmaf_rn(x.y, f, o[4 * k + 1]);
      o[4 * k + 2] = __fmaf_rn(x.z, f, o[4 * k + 2]);
      o[4 * k + 3] = __fmaf_rn(x.w, f, o[4 * k + 3]);
    }
  }
  const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);
  const long long off = ((long long)(t0 + r.t) * a.Hq + d.z * a.G + r.g) * PG_D + g0 * 4;
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = __fmul_rn(o[k], inv);
  if (a.out_dtype == BITNET_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + off);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      dst[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                          pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
  } else {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + off);
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
  }
}

}  // namespace bitnet
