// The paged attention of attn_paged.cuh for requests with many query rows (chunks of a prompt), on
// the 5th-generation tensor cores.  Tiles of 256 query rows, units of 128 cache rows, the same line
// of units with equal shares, one CTA per SM:
//   warps 0-3, 4-7  softmax of the tile's rows 0-127 and 128-255, one thread per row: scores from
//                   tensor memory, maximum, weights (bf16) back to tensor memory; the output at the end
//   warps 8, 9      one thread each, for the rows 0-127 and 128-255: tcgen05.mma S = Q K^T (both
//                   operands in shared memory) and O += P V (P in tensor memory)
//   warp 10         TMA loads of K, page by page, into a ring of two 32 KB slots
//   warp 11         TMA loads of Q, and of V into another ring
// A unit is done in two steps of 64 cache rows.  Tensor memory (512 columns): each half has S of both
// steps (64 columns each, of which P takes the first 32, or all, once the scores are in registers) and O
// (128).  So the scores of the next step are there while the softmax works on this one's, and a
// half waits for neither the other half nor its own products.
//
// What bounds it: a unit of a full tile takes about 3300 cycles; the products alone take 2484 (S with
// N = 64 costs 48 cycles per instruction instead of 32, because Q is read from shared memory twice
// as often; with N = 128 and one buffer the softmax waited for its own products, 3700 cycles), the
// exponentials 1536 of each scheduler.  In long runs the SM clock falls to 1.5 GHz at 1000 W, and
// power is what counts.  Four chunks at the 70B shape (783 GFLOP): 667 us, 1170 TFLOP/s; 787 us, 1000
// TFLOP/s without a pause between calls.
//
// The running maximum of a row moves only when the scores outgrow it by 2^8: until then the weights
// are at most 2^8, which fp32 sums and bf16's exponent hold without loss, and O needs no rescaling.
// The weights enter the second product as bf16, the tensor core's operand type; the row sum adds the
// unrounded weights in fp32.  For bf16 outputs one bf16 a weight: half a step is 2^-8 of each, which the
// output's own half step outweighs (four chunks at the 70B shape, error against 64 bits 0.00168 where
// unrounded weights give 0.00167).  For fp32 outputs (SPLIT) two: the weight rounded and what that left
// over, 2^-16, in the columns that the scores leave free, and a second product over the same V: the four
// chunks 857-900 us instead of 711-772 with one bf16, a 500-token chunk of 20/5 heads 42.5 instead of 37.2.
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
  // FIXED: a tile's start, output and last waits; four chunks at the 70B shape 708 us with 1, 668 with 2, 672
  // with 3, 677 with 4
  static constexpr int M = 256, U = 128, FIXED = 2;
  BN_DEV static int blocks(const PagedArgs& a, int n) { return div_small(n + a.TB - 1, a.by_TB) * a.NB; }
  BN_DEV static int tiles(int blocks) { return (blocks + 1) >> 1; }
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
  const int b = 2 * tile + (row >> 7), i = row & 127, ti = div_small(i, a.by_GB);
  ChunkRow r;
  r.t = (a.NB == 1 ? b : b / a.NB) * a.TB + ti;
  r.g = (a.NB == 1 ? 0 : (b % a.NB) * 128) + i - ti * a.GB;
  r.there = ti < a.TB && r.t < n && r.g < a.G;
  return r;
}

constexpr int PC_M = ChunkTiles::M;
constexpr int PC_U = ChunkTiles::U;
constexpr int PC_THREADS = 384;
constexpr int PC_MMA_WARP = 8, PC_LOAD_WARP = 10;  // two warps each
constexpr int PC_KSLOTS = 2, PC_VSLOTS = 2;
constexpr uint32_t PC_TILE_BYTES = 128 * 256;  // 128 rows of 128 bf16: two 64-column halves of 128-byte rows, swizzled
constexpr int PC_SMEM = (3 + PC_KSLOTS + PC_VSLOTS) * PC_TILE_BYTES + 1024;  // Q, K, V, 4 KB per softmax warp
constexpr int PC_PART = PC_M * (PG_D + 2);     // floats of a partial tile: values [32][256 rows][4], maxima, sums
constexpr float PC_GROW = 8.0f / PG_SCALE_LOG2;

struct alignas(64) PagedMaps {
  CUtensorMap k, v;  // bf16 [n_pages][Hkv][P][128], box {64, min(P, 128), 1, 1}, 128-byte swizzle
  CUtensorMap q;     // bf16 [T][Hkv][G][128], box {64, GB, 1, TB}, the same
};

// bf16 x bf16 -> fp32, M = 128; `mn_b`: B is stored with its N index contiguous
BN_DEV constexpr uint32_t pc_idesc(int n, bool mn_b) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((mn_b ? 1u : 0u) << 16) | (((uint32_t)n >> 3) << 17) | ((128u >> 4) << 24);
}
// The upper words of the operands' descriptors (128-byte swizzle, eight-row groups 1024 bytes
// apart); the lower word is the address / 16, with the distance of the 64-column halves (16384 bytes)
// above it for V, whose d index is contiguous.
constexpr uint32_t PC_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t PC_DESC_K = 1u << 16, PC_DESC_V = (16384u >> 4) << 16;
// One tcgen05.mma.  The descriptors are put together inside the statement from a base and a constant
// OFF (bytes / 16): as 64-bit operands the compiler keeps all of a loop's in registers, and spills them.
template <uint32_t A_OFF, uint32_t B_OFF>
BN_DEV void umma_bf16_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %3, 0;\n\tadd.u32 x, %1, %4;\n\tadd.u32 y, %2, %5;\n\t"
      "mov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %7, p;\n\t}"
      ::"r"(d_tmem), "r"(a), "r"(b), "r"(accumulate), "n"(A_OFF), "n"(B_OFF), "r"(PC_DESC_HI), "r"(pc_idesc(64, false))
      : "memory");
}
template <uint32_t B_OFF>
BN_DEV void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 y;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %3, 0;\n\tadd.u32 y, %2, %4;\n\tmov.b64 db, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %6, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "r"(b), "r"(accumulate), "n"(B_OFF), "r"(PC_DESC_HI), "r"(pc_idesc(128, true))
      : "memory");
}
BN_DEV void prefetch_map(const void* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
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
BN_DEV void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
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

// 2^z for two values without the exponential unit: z = n + f with n the nearest integer (from the low
// bits of z + 1.5 2^23), 2^f on [-1/2, 1/2] as a polynomial of degree 5 through 1 at 0 (its
// coefficients fitted here; largest relative error 2^-23.1, with the fp32 steps 2^-22.4), n added to the exponent.
// Values below -127 and -inf give exactly 0.  Every fourth pair of weights goes this way: at 16
// exponentials per cycle and SM they bound the softmax.  Four prompts' chunks at the 70B shape, calls
// without a pause: 757 us with a quarter of the pairs moved, 778 with an eighth, 792 with none; with
// three eighths (measured earlier) 5 % more than with a quarter, for want of issue slots.
BN_DEV void exp2_pair(uint64_t z, float& x, float& y) {
  unpack_f32x2(z, x, y);
  z = pack_f32x2(fmaxf(x, -127.0f), fmaxf(y, -127.0f));
  const uint64_t t = add_f32x2(z, pack_f32x2(12582912.0f, 12582912.0f));
  const uint64_t n = add_f32x2(t, pack_f32x2(-12582912.0f, -12582912.0f));
  const uint64_t f = fma_f32x2(n, pack_f32x2(-1.0f, -1.0f), z);
  uint64_t p = pack_f32x2(0.001326472032815218f, 0.001326472032815218f);
  p = fma_f32x2(p, f, pack_f32x2(0.009671512991189957f, 0.009671512991189957f));
  p = fma_f32x2(p, f, pack_f32x2(0.05550733581185341f, 0.05550733581185341f));
  p = fma_f32x2(p, f, pack_f32x2(0.24022242426872253f, 0.24022242426872253f));
  p = fma_f32x2(p, f, pack_f32x2(0.6931470036506653f, 0.6931470036506653f));
  p = fma_f32x2(p, f, pack_f32x2(1.0f, 1.0f));
  float tx, ty;
  unpack_f32x2(t, tx, ty);
  unpack_f32x2(p, x, y);
  x = __uint_as_float(__float_as_uint(x) + (__float_as_uint(tx) << 23));
  y = __uint_as_float(__float_as_uint(y) + (__float_as_uint(ty) << 23));
}
// One lane of a converged warp.  Unlike lane == 0 this tells the compiler that a single thread
// follows, which lets it keep the operands of tcgen05.mma in uniform registers.
BN_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P1;\n\telect.sync _|P1, 0xffffffff;\n\tselp.b32 %0, 1, 0, P1;\n\t}" : "=r"(p));
  return p != 0;
}

// The whole warp waits for a barrier that is most often ready; false (for all lanes) if a lane's
// wait ran out or another warp gave up.
BN_DEV bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity) && !*abort);
}

// Step B (cache rows 64 B .. 64 B + 63) of a unit for half h: S = Q K^T into columns 128 h + 64 B of
// tensor memory (all 512 columns are allocated, so they begin at address 0), O (+)= P V into 256 + 128 h.
template <int B, int KK = 0>
BN_DEV void pc_scores(int h, uint32_t q, uint32_t k) {
  constexpr uint32_t off = (KK >> 2) * 1024 + (KK & 3) * 2;
  umma_bf16_ss<off, off + B * 512>(h * 128 + B * 64, q, k, KK > 0);
  if constexpr (KK < 7) pc_scores<B, KK + 1>(h, q, k);
}
// SPLIT: the second bf16 of the weights in the 32 columns behind the first.
template <bool SPLIT, int B, int KK = 0>
BN_DEV void pc_values(int h, uint32_t v, bool first) {
  umma_bf16_ts<(B * 4 + KK) * 128>(256 + h * 128, h * 128 + B * 64 + KK * 8, v, !first);
  if constexpr (SPLIT) umma_bf16_ts<(B * 4 + KK) * 128>(256 + h * 128, h * 128 + B * 64 + 32 + KK * 8, v, 1);
  if constexpr (KK < 3) pc_values<SPLIT, B, KK + 1>(h, v, false);
}
// First row of unit u behind kv if it lies inside a page of that unit (whose rows from there on may
// hold anything), else 0.
BN_DEV int pc_tail(const PagedArgs& a, int kv, int u) {
  const int tail = kv - u * PC_U;
  return tail > 0 && tail < PC_U && (tail & (a.P - 1)) ? tail : 0;
}

// SPLIT: fp32 outputs; otherwise bf16 ones.
template <bool SPLIT>
__global__ void __launch_bounds__(PC_THREADS, 1) k_attn_paged_chunk(const __grid_constant__ PagedMaps maps, const PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long s_bars[2 * PC_KSLOTS + 3 * PC_VSLOTS + 11];
  __shared__ PagedWalkShared s_walk;
  volatile __shared__ int s_abort;
  __shared__ int s_issued[2], s_q_issued;  // tiles of K and V, and of Q, that were loaded (for the drain after an abort)
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sK = base + 2 * PC_TILE_BYTES, sV = sK + PC_KSLOTS * PC_TILE_BYTES;
  const uint32_t bars = smem_addr(s_bars);
  auto k_full = [&](int s) { return bars + 8u * s; };
  auto k_empty = [&](int s) { return bars + 8u * (PC_KSLOTS + s); };
  auto v_full = [&](int s) { return bars + 8u * (2 * PC_KSLOTS + s); };
  auto v_empty = [&](int s) { return bars + 8u * (2 * PC_KSLOTS + PC_VSLOTS + s); };
  auto v_fixed = [&](int s) { return bars + 8u * (2 * PC_KSLOTS + 2 * PC_VSLOTS + s); };
  const uint32_t bar0 = bars + 8u * (2 * PC_KSLOTS + 3 * PC_VSLOTS);
  const uint32_t q_full = bar0, q_empty = bar0 + 8, mma_done = bar0 + 16;
  auto s_full = [&](int h, int step) { return bar0 + 24u + 8u * (2 * h + step); };
  auto p_full = [&](int h, int step) { return bar0 + 56u + 8u * (2 * h + step); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < PC_KSLOTS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 2);
    }
    for (int s = 0; s < PC_VSLOTS; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 2);
      mbar_init(v_fixed(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(mma_done, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full(i >> 1, i & 1), 1);
      mbar_init(p_full(i >> 1, i & 1), 4);
    }
    s_abort = 0;
    s_issued[0] = s_issued[1] = s_q_issued = 0;
    fence_mbar_init();
  }
  if (warp >= PC_LOAD_WARP && lane == 0) {
    prefetch_map(warp == PC_LOAD_WARP ? &maps.k : &maps.v);
    if (warp != PC_LOAD_WARP) prefetch_map(&maps.q);
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
  w.begin<PC_THREADS>(a, gridDim.x, &s_walk);
  if (threadIdx.x == 0) a.desc[blockIdx.x].first = -1;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax, one row per thread
    const int half = warp >> 2, row = half * 128 + (warp & 3) * 32 + lane;
    const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t_lane + half * 128, tO = tmem + t_lane + 256 + half * 128;
    uint32_t ph = 0;  // parities of s_full, a bit per step
    bool ok = true;
    while (ok && w.take(a)) {
      const int cnt = w.cnt;
      if (2 * w.tile + half < w.blocks) {
        const ChunkRow r = chunk_row(a, w.n, w.tile, row);
        const int lim = r.there ? max(0, w.kv - w.n + r.t + 1) : 0x7FFFFFFF;  // rows of the cache that this row sees
        const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
        float m = -INFINITY, l = 0.0f;  // running maximum of the raw scores (may trail by 2^8), sum
        for (int it = 0; it < cnt && ok; ++it) {
#pragma unroll 1  // one copy of the code: the loops of all roles have to fit the instruction cache
          for (int b = 0; b < 2; ++b) {
            ok = warp_wait(s_full(half, b), (ph >> b) & 1u, &s_abort);
            if (!ok) break;
            ph ^= 1u << b;
            tc_fence_after();
            float s[64];
            tmem_ld32(tS + 64 * b, s);
            tmem_ld32(tS + 64 * b + 32, s + 32);
            tmem_wait_ld();
            const int col0 = (w.unit + it) * PC_U + 64 * b;
            if (lim_warp < col0 + 64) {
              const int rel = lim - col0;
#pragma unroll
              for (int c = 0; c < 64; ++c) s[c] = c < rel ? s[c] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 60; c += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[c + k]), s[c + 4 + k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[60 + k]);
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grow = mt > __fadd_rn(m, PC_GROW);  // from -inf: at the first score
            if (__any_sync(0xffffffffu, grow)) {
              float alpha = 1.0f;
              if (grow) {
                alpha = exp2_approx(__fmul_rn(__fsub_rn(m, mt), PG_SCALE_LOG2));
                m = mt;
                l = __fmul_rn(l, alpha);
              }
              if (it + b > 0) {  // this row's O, once the product of the step before has ended
                ok = warp_wait(s_full(half, b ^ 1), (ph >> (b ^ 1)) & 1u, &s_abort);
                if (!ok) break;
                tc_fence_after();
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
            for (int c = 0; c < 64; c += 32) {
              uint32_t p[16], left[SPLIT ? 16 : 1];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float x, y;
                const uint64_t z = fma_f32x2(pack_f32x2(s[c + k], s[c + k + 1]), sc2, mu2);
                if ((k & 6) == 6) exp2_pair(z, x, y);
                else {
                  unpack_f32x2(z, x, y);
                  x = exp2_approx(x);
                  y = exp2_approx(y);
                }
                sum2[(k >> 1) & 1] = add_f32x2(sum2[(k >> 1) & 1], pack_f32x2(x, y));
                const uint32_t w = pack_bf16(x, y);
                p[k >> 1] = w;
                if constexpr (SPLIT) left[k >> 1] = pack_bf16(__fsub_rn(x, __uint_as_float(w << 16)), __fsub_rn(y, __uint_as_float(w & 0xFFFF0000u)));
              }
              tmem_st16(tS + 64 * b + (c >> 1), p);
              if constexpr (SPLIT) tmem_st16(tS + 64 * b + 32 + (c >> 1), left);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(half, b));
            float x, y;
            unpack_f32x2(add_f32x2(sum2[0], sum2[1]), x, y);
            l = __fadd_rn(l, __fadd_rn(x, y));
          }
        }
        if (!ok) break;
        ok = warp_wait(s_full(half, 0), ph & 1u, &s_abort) && warp_wait(s_full(half, 1), (ph >> 1) & 1u, &s_abort);
        if (!ok) break;
        ph ^= 3u;
        tc_fence_after();
        if (cnt == w.nu) {
          // By way of shared memory, so that a warp writes whole 128-byte lines: 32 rows of 128 bytes
          // (64 bf16 or 32 fp32 columns), their 16-byte chunks permuted by the row.
          const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);  // NaN stays
          constexpr bool bf = !SPLIT;
          const long long off = r.there ? ((long long)(w.t0 + r.t) * a.Hq + w.head * a.G + r.g) * (bf ? PG_D * 2 : PG_D * 4) : -1;
          const uint32_t stage = sV + PC_VSLOTS * PC_TILE_BYTES + warp * 4096;
          long long to[8];  // of the rows whose chunk lane & 7 this lane writes
#pragma unroll
          for (int i = 0; i < 8; ++i) to[i] = __shfl_sync(0xffffffffu, off, i * 4 + (lane >> 3));
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            float o[16];
            tmem_ld16f(tO + 16 * g, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __fmul_rn(o[k], inv);
            if (bf) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                sts128(stage + lane * 128 + ((((g & 3) * 2 + k) ^ (lane & 7)) << 4), pack_bf16(o[8 * k], o[8 * k + 1]),
                       pack_bf16(o[8 * k + 2], o[8 * k + 3]), pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
              if ((g & 3) != 3) continue;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                sts128(stage + lane * 128 + ((((g & 1) * 4 + k) ^ (lane & 7)) << 4), __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                       __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
              if ((g & 1) == 0) continue;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3), ch = lane & 7;
              const uint4 x = lds128(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
              if (to[i] >= 0) *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + to[i] + (bf ? g >> 2 : g >> 1) * 128 + ch * 16) = x;
            }
            __syncwarp();
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
      if (threadIdx.x == 0 && w.unit > 0 && w.unit + cnt == w.nu)
        a.desc[blockIdx.x] = w.ended();
    }
    if (!ok) s_abort = 1;
  } else if (warp < PC_LOAD_WARP) {
    // ------------------------------------------------------------ products
    // A thread per half: one for both would spend longer issuing (each wait and commit takes it about
    // 120 cycles) than the tensor core computing.  A half without rows passes its slots on.
    if (elect_one()) {
      const int h = warp - PC_MMA_WARP;
      const uint32_t q = (sQ + h * PC_TILE_BYTES) >> 4 | PC_DESC_K;
      int ks = 0, vs = 0;
      uint32_t ph_k = 0, ph_v = 0, ph_q = 0, ph_p = 0, ph_f = 0;  // ph_p: per step of a unit, ph_f: per slot
      bool ok = true;
      while (ok && !s_abort && w.take(a)) {
        const int cnt = w.cnt;
        const bool rows = 2 * w.tile + h < w.blocks;
        auto release = [&](uint32_t bar) {
          if (rows) umma_commit(bar);
          else mbar_arrive(bar);
        };
        // One loop for the first scores (it = -1) and the rest: what runs once per tile would have left
        // the instruction cache, which costs about 1000 cycles a miss.
        for (int it = -1; it < cnt; ++it) {
          const bool have = it >= 0, more = it + 1 < cnt;
          if (have) {
            ok = mbar_wait_bounded(v_full(vs), ph_v);
            if (ok && pc_tail(a, w.kv, w.unit + it) > 0) {
              ok = mbar_wait_bounded(v_fixed(vs), (ph_f >> vs) & 1u);
              ph_f ^= 1u << vs;
            }
          } else {
            ok = mbar_wait_bounded(q_full, ph_q);
            ph_q ^= 1u;
          }
          if (more) ok = ok && mbar_wait_bounded(k_full(ks), ph_k);
          if (!ok) break;
          if (rows) {
            const uint32_t v = (sV + vs * PC_TILE_BYTES) >> 4 | PC_DESC_V, k = (sK + ks * PC_TILE_BYTES) >> 4 | PC_DESC_K;
            if (have) ok = mbar_wait_bounded(p_full(h, 0), ph_p);
            if (!ok) break;
            tc_fence_after();
            if (have) pc_values<SPLIT, 0>(h, v, it == 0);
            if (more) pc_scores<0>(h, q, k);
            umma_commit(s_full(h, 0));
            if (have) {
              ok = mbar_wait_bounded(p_full(h, 1), ph_p);
              if (!ok) break;
              ph_p ^= 1u;
              tc_fence_after();
              pc_values<SPLIT, 1>(h, v, false);
            }
            if (more) pc_scores<1>(h, q, k);
          }
          if (more) {
            release(k_empty(ks));
            if (++ks == PC_KSLOTS) {
              ks = 0;
              ph_k ^= 1u;
            }
          }
          if (it + 2 == cnt) release(q_empty);
          if (have) {
            release(v_empty(vs));
            if (++vs == PC_VSLOTS) {
              vs = 0;
              ph_v ^= 1u;
            }
          }
          if (rows) umma_commit(s_full(h, 1));
        }
      }
      if (!ok) s_abort = 1;
      umma_commit(mma_done);  // every product ends before tensor memory is released, also after an abort
      mbar_drain(mma_done, 0);
    }
  } else {
    // ------------------------------------------------------------ K (warp 10), Q and V (warp 11)
    const bool is_v = warp != PC_LOAD_WARP;
    const void* map = is_v ? &maps.v : &maps.k;
    const uint32_t buf = is_v ? sV : sK;
    const int slots = is_v ? PC_VSLOTS : PC_KSLOTS;
    const int log2b = min(a.log2P, 7), npg = 1 << (7 - log2b);  // rows of a copy, copies per unit and 64-column half
    int slot = 0, issued = 0, q_issued = 0;
    uint32_t ph = 1, ph_q = 1;
    bool ok = true;
    while (ok && !s_abort && w.take(a)) {
      const int cnt = w.cnt;
      const int vis = ChunkTiles::visible(a, w.n, w.kv, w.tile);
      const int* trow = a.table + (long long)w.seq * a.width;
      // this lane's entry of the table for a unit (-1 where no row sees it)
      auto entry = [&](int u) {
        const int row = u * PC_U + (lane << log2b);
        return lane < npg && row < vis ? __ldg(trow + (row >> a.log2P)) : -1;
      };
      int ahead = entry(w.unit);
      for (int it = 0; it < cnt; ++it) {
        const int row0 = (w.unit + it) * PC_U;
        int page = ahead;
        if (page < 0 || page >= a.n_pages) {  // zeros; an error where a row would see the page
          if (lane < npg && row0 + (lane << log2b) < vis) flag_index_error();
          page = a.n_pages;
        }
        if (it + 1 < cnt) ahead = entry(w.unit + it + 1);
        if (is_v && it == 0) {  // Q, which is needed before the first V
          ok = warp_wait(q_empty, ph_q, &s_abort);
          if (!ok) break;
          ph_q ^= 1u;
          if (elect_one()) {
            const int nh = 2 * w.tile + 1 < w.blocks ? 2 : 1;
            mbar_arrive_expect_tx(q_full, nh * a.TB * a.GB * PG_D * 2);
            for (int h = 0; h < nh; ++h) {
              const ChunkRow r = chunk_row(a, w.n, w.tile, h * 128);
              const uint32_t dst = sQ + h * PC_TILE_BYTES;
              tma_load_4d(dst, &maps.q, 0, r.g, w.head, w.t0 + r.t, q_full);
              tma_load_4d(dst + 16384, &maps.q, 64, r.g, w.head, w.t0 + r.t, q_full);
            }
          }
          __syncwarp();
          ++q_issued;
        }
        const uint32_t bar_full = is_v ? v_full(slot) : k_full(slot);
        ok = warp_wait(is_v ? v_empty(slot) : k_empty(slot), ph, &s_abort);
        if (!ok) break;
        const uint32_t dst = buf + slot * PC_TILE_BYTES;
        int id[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) id[p] = __shfl_sync(0xffffffffu, page, p);
        if (elect_one()) {
          mbar_arrive_expect_tx(bar_full, PC_TILE_BYTES);
#pragma unroll
          for (int p = 0; p < 8; ++p)
            if (p < npg) {
              const int at = p << log2b;
              tma_load_4d(dst + at * 128, map, 0, (row0 + at) & (a.P - 1), w.head, id[p], bar_full);
              tma_load_4d(dst + at * 128 + 16384, map, 64, (row0 + at) & (a.P - 1), w.head, id[p], bar_full);
            }
        }
        __syncwarp();
        ++issued;
        if (is_v) {
          // rows behind kv in the request's last page become zeros once the copy has landed
          const int tail = pc_tail(a, w.kv, w.unit + it);
          if (tail > 0) {
            ok = warp_wait(bar_full, ph ^ 1u, &s_abort);
            if (!ok) break;
            const int end = min(PC_U, (tail + a.P - 1) & ~(a.P - 1));
            for (int i = tail * 16 + lane; i < end * 16; i += 32)
              sts128(dst + ((i >> 3) & 1) * 16384 + (i >> 4) * 128 + (i & 7) * 16, 0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_fixed(slot));
          }
        }
        if (++slot == slots) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok) s_abort = 1;
    if (lane == 0) {
      s_issued[is_v] = issued;
      if (is_v) s_q_issued = q_issued;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (s_abort) {
    // every issued copy lands before the block ends
    if (warp >= PC_LOAD_WARP && lane == 0) {
      const bool is_v = warp != PC_LOAD_WARP;
      const int slots = is_v ? PC_VSLOTS : PC_KSLOTS, n = s_issued[is_v];
      for (int i = max(0, n - slots); i < n; ++i)
        mbar_drain(is_v ? v_full(i % slots) : k_full(i % slots), (uint32_t)((i / slots) & 1));
      if (is_v && s_q_issued > 0) mbar_drain(q_full, (uint32_t)((s_q_issued - 1) & 1));
    }
  }
  __syncthreads();
  if (warp == PC_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Thread: a row and PC_JOIN_V4 float4 of its dimensions (blockIdx.y); most tiles have two parts.  Four
// chunks at the 70B shape (39 MB of parts): 10.7 us, with four parts of two float4 at a time 12.9 us.
constexpr int PC_JOIN_V4 = 4;
__global__ void __launch_bounds__(PC_M) k_attn_paged_chunk_join(const PagedArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const PagedTile d = a.desc[blockIdx.x];
  if (d.first < 0) return;
  const int row = threadIdx.x, g0 = blockIdx.y * PC_JOIN_V4;
  const ChunkRow r = chunk_row(a, d.n, d.tile, row);
  if (!r.there) return;
  float o[4 * PC_JOIN_V4], m, l;
  join_parts<PC_JOIN_V4, 2>(a.part, PC_PART, PC_M * PG_D, PC_M, row, d.first, d.first, 1, blockIdx.x, PG_SCALE_LOG2,
                [&](int k) { return ((g0 + k) * PC_M + row) * 4; }, o, m, l);
  divide_row(o, l);
  store_row<PC_JOIN_V4>(a.out, a.out_dtype, ((long long)(d.t0 + r.t) * a.Hq + d.head * a.G + r.g) * PG_D + g0 * 4, o);
}

}  // namespace bitnet
