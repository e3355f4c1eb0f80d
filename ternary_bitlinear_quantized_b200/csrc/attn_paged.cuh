// Causal grouped-query attention of each request's new tokens over its pages of the cache:
//   out[t, h] = sum_l w_l v_l,  w = softmax over l of (q[t, h] . k_l) / sqrt(128),
// l running over the request's rows 0 .. kv - new + t' (t' = the token's place among the
// request's new tokens), query head h reading key/value head h / G, G = Hq / Hkv.  A row that
// sees nothing is zero.
//
// Work is cut the same way for every size.  The query rows r = t' G + g of one request and one
// key/value head (all of them read the same keys) form tiles of M rows; a tile's visible cache
// rows form units of U rows.  All units of all tiles, in the order request, head, tile, unit, make
// one line, and every CTA takes an equal stretch of it (a tile counts for a fixed number of units more
// than it has, for its start and output).  So a long cache with one
// query row, a ragged batch and a causal triangle are all spread evenly without the host knowing a
// length.  A tile that lies in one CTA's share is written straight to the output; of the others
// each CTA keeps (running maximum, sum, weighted values) in the workspace, at most two per CTA
// (the tile that its share begins in and the one that it ends in), and a second launch joins
// them in the order of the units.  The cut depends on the lengths and the GPU alone, so results
// repeat bit for bit.
#pragma once
#include "common.cuh"
#include "gemv.cuh"
#include "paged.cuh"

namespace bitnet {

// A tile whose units lie in several CTAs: `first` is the one it begins in, -1 for no tile.
struct alignas(16) PagedTile {
  int first, t0, n, head, tile, pad[3];
};

struct PagedArgs {
  const __nv_bfloat16* q;        // [T][Hq][128]
  const __nv_bfloat16* k_pages;  // [n_pages][Hkv][P][128]
  const __nv_bfloat16* v_pages;
  const int* table;              // [B][width]
  const int* cu;                 // [B + 1]
  const int* kv;                 // [B]
  void* out;                     // [T][Hq][128]
  PagedTile* desc;               // [C] the tile that a CTA ended and another one began
  float* part;                   // [C][2] partial tiles
  int T, B, Hq, Hkv, G, P, log2P, width, n_pages, max_new, out_dtype;
  uint64_t by_G, by_TB, by_GB;   // ceil(2^32 / divisor), for div_small
  int TB, GB, NB;                // chunk kernel: a block of query rows is TB tokens x GB heads, NB blocks cover the G heads
};

constexpr float PG_SCALE_LOG2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)

BN_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x / d for x >= 0, x d < 2^32, m = ceil(2^32 / d): m d - 2^32 < d, so x m / 2^32 exceeds x / d by less
// than x / 2^32 < 1 / d.
BN_DEV int div_small(int x, uint64_t m) { return (int)(((uint64_t)(uint32_t)x * m) >> 32); }
// a / b for non-negative numbers, most often of 32 bits (a 64-bit division takes several times as long).
BN_DEV long long div_nonneg(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Request i's new tokens and cache rows; false for lengths that do not fit the call.
BN_DEV bool paged_request(const PagedArgs& a, int i, int& t0, int& n, int& kv) {
  t0 = __ldg(a.cu + i);
  const int t1 = __ldg(a.cu + i + 1);
  kv = __ldg(a.kv + i);
  n = t1 - t0;
  return t0 >= 0 && t1 >= t0 && t1 <= a.T && n <= a.max_new && kv >= 0 && kv <= (long long)a.width * a.P;
}

// How a kernel cuts a request's query rows (of one key/value head) into blocks and those into tiles,
// and how many cache rows the last row of tile j sees (0 where it sees none).  FIXED: what a tile
// costs beside its units, in units.
struct FewTiles {  // 16 consecutive rows
  static constexpr int M = 16, U = 64, FIXED = 1;
  BN_DEV static int blocks(const PagedArgs& a, int n) { return (n * a.G + M - 1) / M; }
  BN_DEV static int tiles(int blocks) { return blocks; }
  BN_DEV static int visible(const PagedArgs& a, int n, int kv, int j) {
    const int last = min((j + 1) * M, n * a.G) - 1;
    return max(0, kv - n + div_small(last, a.by_G) + 1);
  }
};
template <typename Tiles>
BN_DEV int tile_units(const PagedArgs& a, int n, int kv, int j) {
  return max(1, (Tiles::visible(a, n, kv, j) + Tiles::U - 1) / Tiles::U);
}

// A CTA's place on the line of units.
struct PagedWalkShared {
  long long warp_sum[32];
  int seq, t0, n, kv, head, tile, at;
};
template <typename Tiles>
struct PagedWalk {
  int seq, t0, n, kv;  // request
  int head, tile, blocks;
  int unit, cnt, nu;   // this piece of the tile: cnt of its nu units, from `unit` on
  int at;              // its place in the tile, the FIXED cost included
  int took;            // its length there
  long long pos, left; // the place of the piece on the line, and what is left of the CTA's share from there on
  long long per;       // the share of every CTA

  // Goes on to the next piece of the CTA's share; false at its end.  A piece that lies within its
  // tile's fixed cost has no units and is passed over.
  BN_DEV bool take(const PagedArgs& a) {
    for (;;) {
      left -= took;
      if (left <= 0) return false;
      pos += took;
      at += took;
      if (at >= nu + Tiles::FIXED) {
        at = 0;
        if (++tile >= Tiles::tiles(blocks)) {
          tile = 0;
          if (++head >= a.Hkv) {
            head = 0;
            do {  // something is left, so a request with tokens follows
              if (++seq >= a.B) {  // unless the lengths changed meanwhile
                left = 0;
                return false;
              }
            } while (!paged_request(a, seq, t0, n, kv) || n == 0);
            blocks = Tiles::blocks(a, n);
          }
        }
        nu = tile_units<Tiles>(a, n, kv, tile);
      }
      took = (int)min(left, (long long)(nu + Tiles::FIXED - at));
      unit = max(0, at - Tiles::FIXED);
      cnt = at + took - Tiles::FIXED - unit;
      if (cnt > 0) return true;
    }
  }
  // The descriptor of this tile, which began in another CTA's share.
  BN_DEV PagedTile ended() const { return {(int)div_nonneg(pos - at + Tiles::FIXED, per), t0, n, head, tile}; }

  // Block-wide: finds the CTA's share.  Up to THREADS requests are taken at once, S threads of one
  // warp (a power of two) per request, each with q consecutive tiles of one head; prefix sums over
  // the threads give the place of each request (times Hkv) and of each thread's tiles in a head.
  template <int THREADS>
  BN_DEV void begin(const PagedArgs& a, int C, PagedWalkShared* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int logS = 0;
    while (logS < 5 && (a.B << (logS + 1)) <= THREADS) ++logS;
    const int S = 1 << logS, sub = threadIdx.x & (S - 1), per_round = THREADS >> logS;
    bool bad = false;
    int rt0, rn, rkv, j0, j1;  // this thread's request and tiles of the last round
    auto mine_of = [&](int i) {
      rt0 = rn = rkv = j0 = j1 = 0;
      if (i >= a.B) return 0ll;
      if (!paged_request(a, i, rt0, rn, rkv)) {  // lengths that do not fit: no units
        bad = true;
        rn = 0;
        return 0ll;
      }
      const int k = Tiles::tiles(Tiles::blocks(a, rn)), q = (k + S - 1) >> logS;
      j0 = min(k, sub * q);
      j1 = min(k, j0 + q);
      long long w = 0;
      for (int j = j0; j < j1; ++j) w += tile_units<Tiles>(a, rn, rkv, j) + Tiles::FIXED;
      return w;
    };
    // inclusive prefix sum over the block and its total
    auto scan = [&](long long v, long long& all) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) sm->warp_sum[warp] = v;
      __syncthreads();
      all = 0;
#pragma unroll
      for (int k = 0; k < THREADS / 32; ++k) {
        const long long x = sm->warp_sum[k];
        if (k < warp) v += x;
        all += x;
      }
      return v;
    };
    long long total = 0, incl = 0, mine = 0, last_round = 0;
    const int rounds = (a.B + per_round - 1) / per_round;
    for (int r = 0; r < rounds; ++r) {
      if (r > 0) __syncthreads();  // the sums of the round before have been read
      mine = mine_of(r * per_round + (threadIdx.x >> logS));
      incl = total + scan(mine, last_round);
      total += last_round;
    }
    if (bad && blockIdx.x == 0) flag_index_error();
    per = div_nonneg(total * a.Hkv + C - 1, C);
    pos = (long long)blockIdx.x * per;
    left = max(0ll, min(per, total * a.Hkv - pos));
    took = 0;
    if (left == 0) return;
    long long before = total - last_round;
    int round = rounds - 1;
    while (pos < before * a.Hkv) {  // from the last round, whose sums are at hand, downwards
      --round;
      __syncthreads();
      mine = mine_of(round * per_round + (threadIdx.x >> logS));
      long long all;
      incl = scan(mine, all);
      before -= all;
      incl += before;
    }
    // the threads of the request that pos lies in, and of them the one whose tiles it lies in
    const long long start = incl - mine;
    const long long pr0 = __shfl_sync(0xffffffffu, start, lane & ~(S - 1)), pr1 = __shfl_sync(0xffffffffu, incl, lane | (S - 1));
    if (pr0 * a.Hkv <= pos && pos < pr1 * a.Hkv) {
      const long long w = pr1 - pr0, off = pos - pr0 * a.Hkv, hd = div_nonneg(off, w), target = pr0 + off - hd * w;
      if (target >= start && target < incl) {
        long long rem = target - start;
        int j = j0;
        for (;; ++j) {
          const int u = tile_units<Tiles>(a, rn, rkv, j) + Tiles::FIXED;
          if (rem < u) break;
          rem -= u;
        }
        sm->seq = round * per_round + (threadIdx.x >> logS);
        sm->t0 = rt0;
        sm->n = rn;
        sm->kv = rkv;
        sm->head = (int)hd;
        sm->tile = j;
        sm->at = (int)rem;
      }
    }
    __syncthreads();
    seq = sm->seq;
    t0 = sm->t0;
    n = sm->n;
    kv = sm->kv;
    head = sm->head;
    tile = sm->tile;
    at = sm->at;
    blocks = Tiles::blocks(a, n);
    nu = tile_units<Tiles>(a, n, kv, tile);
  }
};

// ------------------------------------------------------------------ few rows: mma.sync
// Requests with few query rows (single tokens, short drafts) are bound by the read of their cache
// rows.  A CTA of four warps takes tiles of 16 query rows and units of 64 cache rows; each warp
// works through its own 16 cache rows of every unit with its own running maximum, sum and
// weighted values, so the warps never wait for one another inside a tile; they are joined at
// the tile's end.  Each warp copies its rows (4 KB of keys, 4 KB of values, inside one page
// because page sizes are multiples of 16) through a ring of PD_STAGES stages of its own with
// cp.async, two stages ahead; two CTAs fit an SM, so 128 KB are in flight per SM.  Rows of 256
// bytes are stored with their 16-byte chunks permuted by the row (chunk ^ row % 8), which keeps
// the ldmatrix reads free of bank conflicts; rows behind the visible ones are filled with
// zeros, so what the cache holds there (NaN included) is never used.
// Products are m16n8k16 bf16 with fp32 sums; the probabilities enter the second product as the
// sum of two bf16 (p rounded, and what that left over), so their rounding is 2^-16 of p; the
// extra instruction is free beside the read.  64 requests of one token behind up to 8192 rows at the 70B
// shape (1.06 GB of cache): 175 us, 6.07 TB/s.
constexpr int PD_M = FewTiles::M;
constexpr int PD_U = FewTiles::U;
constexpr int PD_WARPS = 4;
constexpr int PD_THREADS = 32 * PD_WARPS;
constexpr int PD_STAGES = 3;
constexpr int PD_STAGE_BYTES = 2 * 16 * 256;
constexpr int PD_RING = PD_WARPS * PD_STAGES * PD_STAGE_BYTES;
static_assert((64 + 4) * 32 * 4 <= PD_STAGES * PD_STAGE_BYTES, "a warp's fragments fit its drained ring at the join");
constexpr int PD_PART = PD_M * (PG_D + 2);      // floats of a partial tile: values, maxima, sums

BN_DEV void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
BN_DEV void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
BN_DEV void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared, or 16 zero bytes where !valid (src is not read then).
BN_DEV void cp_async16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
template <int N>
BN_DEV void cp_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

BN_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&w);
}

__global__ void __launch_bounds__(PD_THREADS, 2) k_attn_paged_few(const PagedArgs a) {
  extern __shared__ __align__(128) uint8_t pd_sm[];
  __shared__ PagedWalkShared s_walk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  PagedWalk<FewTiles> w;
  w.begin<PD_THREADS>(a, gridDim.x, &s_walk);
  if (threadIdx.x == 0) a.desc[blockIdx.x].first = -1;
  const uint32_t ring = smem_addr(pd_sm) + warp * PD_STAGES * PD_STAGE_BYTES;
  const int g = lane >> 2, tq = lane & 3;
  const long long page_elems = (long long)a.Hkv * a.P * PG_D;

  while (w.take(a)) {
    const int nu = w.nu, cnt = w.cnt;
    const int R = w.n * a.G, r0 = w.tile * PD_M;
    const int vis = FewTiles::visible(a, w.n, w.kv, w.tile);
    // this thread's two query rows (g and g + 8 of the tile): what they see, and their q fragments
    int lim[2];
    uint32_t qf[8][4];
    long long qoff[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + g + 8 * e;
      const bool there = r < R;
      const int t = there ? div_small(r, a.by_G) : 0, hg = there ? r - t * a.G : 0;
      lim[e] = there ? max(0, w.kv - w.n + t + 1) : 0;
      qoff[e] = there ? ((long long)(w.t0 + t) * a.Hq + w.head * a.G + hg) * PG_D : -1;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + qoff[e] + ks * 16 + 2 * tq);
        qf[ks][e] = there ? __ldg(src) : 0u;
        qf[ks][e + 2] = there ? __ldg(src + 4) : 0u;
      }
    }
    float O[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    // page ids, 32 units at a time: lane i holds the page of unit ids0 + i (this warp's rows)
    const int* trow = a.table + (long long)w.seq * a.width;
    int ids = -1, ids0 = w.unit - 32;
    auto load = [&](int u, int stage) {
      if (u >= ids0 + 32) {
        ids0 = u;
        const long long row = (long long)(u + lane) * PD_U + warp * 16;
        ids = -1;
        if (row < vis) {
          ids = __ldg(trow + (row >> a.log2P));
          if (ids < 0 || ids >= a.n_pages) {
            ids = -1;
            flag_index_error();
          }
        }
      }
      const int page = __shfl_sync(0xffffffffu, ids, u - ids0);
      const int row0 = u * PD_U + warp * 16;
      const long long base = (long long)max(page, 0) * page_elems + ((long long)w.head * a.P + (row0 & (a.P - 1))) * PG_D;
      const uint32_t dst = ring + stage * PD_STAGE_BYTES;
      const int ch = lane & 15;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + (lane >> 4);
        const bool ok = page >= 0 && row0 + row < vis;
        const long long off = base + row * PG_D + ch * 8;
        const uint32_t d = dst + row * 256 + ((ch ^ (row & 7)) << 4);
        cp_async16_or_zero(d, a.k_pages + (ok ? off : 0), ok);
        cp_async16_or_zero(d + 4096, a.v_pages + (ok ? off : 0), ok);
      }
    };
#pragma unroll
    for (int s = 0; s < PD_STAGES - 1; ++s) {
      if (s < cnt) load(w.unit + s, s);
      cp_async_commit();
    }
    int st = 0;
    for (int it = 0; it < cnt; ++it) {
      cp_async_wait_group<PD_STAGES - 2>();
      __syncwarp();
      if (it + PD_STAGES - 1 < cnt) load(w.unit + it + PD_STAGES - 1, st == 0 ? PD_STAGES - 1 : st - 1);
      cp_async_commit();
      const uint32_t kb = ring + st * PD_STAGE_BYTES, vb = kb + 4096;
      float S[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      {
        const int row = (lane & 7) + ((lane >> 4) << 3), c1 = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t b[4];
          ldmatrix_x4(b, kb + row * 256 + (((2 * ks + c1) ^ (row & 7)) << 4));
          mma_bf16(S[0], qf[ks], b[0], b[1]);
          mma_bf16(S[1], qf[ks], b[2], b[3]);
        }
      }
      const int col0 = (w.unit + it) * PD_U + warp * 16 + 2 * tq;
      uint32_t ph[4], pl[4];
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = col0 + (i >> 1) * 8 + (i & 1);
          x[i] = col < lim[e] ? __fmul_rn(S[i >> 1][2 * e + (i & 1)], PG_SCALE_LOG2) : -INFINITY;
        }
        float mt = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        const float mn = fmaxf(m[e], mt);
        const float mu = mn == -INFINITY ? 0.0f : mn;  // a row that has seen nothing yet: all weights 0
        alpha[e] = exp2_approx(__fsub_rn(m[e], mu));
        m[e] = mn;
        float p[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = exp2_approx(__fsub_rn(x[i], mu));
          hi[i] = __bfloat162float(__float2bfloat16_rn(p[i]));
        }
        l[e] = __fmaf_rn(l[e], alpha[e], __fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])));
        ph[e] = pack_bf16(hi[0], hi[1]);
        ph[e + 2] = pack_bf16(hi[2], hi[3]);
        pl[e] = pack_bf16(__fsub_rn(p[0], hi[0]), __fsub_rn(p[1], hi[1]));
        pl[e + 2] = pack_bf16(__fsub_rn(p[2], hi[2]), __fsub_rn(p[3], hi[3]));
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          O[i][0] = __fmul_rn(O[i][0], alpha[0]);
          O[i][1] = __fmul_rn(O[i][1], alpha[0]);
          O[i][2] = __fmul_rn(O[i][2], alpha[1]);
          O[i][3] = __fmul_rn(O[i][3], alpha[1]);
        }
      }
      {
        const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c1 = lane >> 4;
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) {
          uint32_t b[4];
          ldmatrix_x4_trans(b, vb + row * 256 + (((2 * dt + c1) ^ (row & 7)) << 4));
          mma_bf16(O[2 * dt], ph, b[0], b[1]);
          mma_bf16(O[2 * dt + 1], ph, b[2], b[3]);
          mma_bf16(O[2 * dt], pl, b[0], b[1]);
          mma_bf16(O[2 * dt + 1], pl, b[2], b[3]);
        }
      }
      if (++st == PD_STAGES) st = 0;
    }
    cp_async_wait_all();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] = __fadd_rn(l[e], __shfl_xor_sync(0xffffffffu, l[e], 1));
      l[e] = __fadd_rn(l[e], __shfl_xor_sync(0xffffffffu, l[e], 2));
    }
    // Join the four warps: each leaves its values in its ring (drained), then each adds up a quarter of
    // the columns, blocks 4 warp .. 4 warp + 3 of eight.
    {
      float* buf = reinterpret_cast<float*>(pd_sm + warp * PD_STAGES * PD_STAGE_BYTES) + lane;
#pragma unroll
      for (int i = 0; i < 64; ++i) buf[i * 32] = O[i >> 2][i & 3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        buf[(64 + e) * 32] = m[e];
        buf[(66 + e) * 32] = l[e];
      }
    }
    __syncthreads();
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.0f;
    {
      const float* buf = reinterpret_cast<const float*>(pd_sm) + lane;
      constexpr int STRIDE = PD_STAGES * PD_STAGE_BYTES / 4;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mv[PD_WARPS];
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) mv[v] = buf[v * STRIDE + (64 + e) * 32];
        m[e] = fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3]));
        const float mu = m[e] == -INFINITY ? 0.0f : m[e];
        l[e] = 0.0f;
#pragma unroll
        for (int v = 0; v < PD_WARPS; ++v) {
          const float f = exp2_approx(__fsub_rn(mv[v], mu));
          l[e] = __fmaf_rn(buf[v * STRIDE + (66 + e) * 32], f, l[e]);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (((i >> 1) & 1) == e) o[i] = __fmaf_rn(buf[v * STRIDE + (16 * warp + i) * 32], f, o[i]);
        }
      }
    }
    if (cnt == nu) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (qoff[e] < 0) continue;
        const float inv = l[e] > 0.0f ? __fdiv_rn(1.0f, l[e]) : (l[e] == 0.0f ? 0.0f : l[e]);  // NaN stays
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __fmul_rn(o[4 * i + 2 * e], inv), y = __fmul_rn(o[4 * i + 2 * e + 1], inv);
          const long long off = qoff[e] + (4 * warp + i) * 8 + 2 * tq;
          if (a.out_dtype == BITNET_BF16)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) + off) = pack_bf16(x, y);
          else
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + off) = make_float2(x, y);
        }
      }
    } else {
      float* part = a.part + ((long long)blockIdx.x * 2 + (w.unit > 0 ? 0 : 1)) * PD_PART;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float2*>(part + (g + 8 * e) * PG_D + (4 * warp + i) * 8 + 2 * tq) = make_float2(o[4 * i + 2 * e], o[4 * i + 2 * e + 1]);
        if (tq == 0 && warp == 0) {
          part[PD_M * PG_D + g + 8 * e] = m[e];
          part[PD_M * PG_D + PD_M + g + 8 * e] = l[e];
        }
      }
      if (threadIdx.x == 0 && w.unit > 0 && w.unit + cnt == nu) a.desc[blockIdx.x] = w.ended();
    }
    __syncthreads();  // the rings are filled again for the next tile
  }
}

// Joins the parts of the tile that CTA blockIdx.x ended: part 1 of the CTA that the tile began in, and
// part 0 of every later one.  Each thread adds up V4 float4 of one row over the parts first,
// first + step, ... BATCH at a time so that their loads are in flight together; `at(part, k)` is the
// place of the row's k-th one.
template <int V4, int BATCH, typename At>
BN_DEV void join_parts(const float* parts, int stride, int stats, int rows, int row, int tile_first, int first, int step, int last,
                       float scale_log2, At at, float (&o)[4 * V4], float& m, float& l) {
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int k = 0; k < 4 * V4; ++k) o[k] = 0.0f;
  for (int i0 = first; i0 <= last; i0 += BATCH * step) {
    float pm[BATCH], pl[BATCH], mn = m;
    float4 x[BATCH][V4];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u * step;
      pm[u] = -INFINITY;  // weight 0 behind the last part
      pl[u] = 0.0f;
#pragma unroll
      for (int k = 0; k < V4; ++k) x[u][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i <= last) {
        const float* p = parts + ((long long)i * 2 + (i == tile_first ? 1 : 0)) * stride;
        pm[u] = p[stats + row];
        pl[u] = p[stats + rows + row];
#pragma unroll
        for (int k = 0; k < V4; ++k) x[u][k] = *reinterpret_cast<const float4*>(p + at(k));
      }
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) mn = fmaxf(mn, pm[u]);
    const float mu = mn == -INFINITY ? 0.0f : mn;
    const float old = exp2_approx(__fmul_rn(__fsub_rn(m, mu), scale_log2));
    m = mn;
    l = __fmul_rn(l, old);
#pragma unroll
    for (int k = 0; k < 4 * V4; ++k) o[k] = __fmul_rn(o[k], old);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float f = exp2_approx(__fmul_rn(__fsub_rn(pm[u], mu), scale_log2));
      l = __fmaf_rn(pl[u], f, l);
#pragma unroll
      for (int k = 0; k < V4; ++k) {
        o[4 * k] = __fmaf_rn(x[u][k].x, f, o[4 * k]);
        o[4 * k + 1] = __fmaf_rn(x[u][k].y, f, o[4 * k + 1]);
        o[4 * k + 2] = __fmaf_rn(x[u][k].z, f, o[4 * k + 2]);
        o[4 * k + 3] = __fmaf_rn(x[u][k].w, f, o[4 * k + 3]);
      }
    }
  }
}
// o / l, zero for a row that sees nothing.
template <int N>
BN_DEV void divide_row(float (&o)[N], float l) {
  const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);  // NaN stays
#pragma unroll
  for (int k = 0; k < N; ++k) o[k] = __fmul_rn(o[k], inv);
}
template <int V4>
BN_DEV void store_row(void* out, int out_dtype, long long off, const float (&o)[4 * V4]) {
  if (out_dtype == BITNET_BF16) {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(out) + off;
    if constexpr (V4 % 2 == 0) {
#pragma unroll
      for (int k = 0; k < V4; k += 2)
        reinterpret_cast<uint4*>(dst)[k / 2] = make_uint4(pack_bf16(o[4 * k], o[4 * k + 1]), pack_bf16(o[4 * k + 2], o[4 * k + 3]),
                                                          pack_bf16(o[4 * k + 4], o[4 * k + 5]), pack_bf16(o[4 * k + 6], o[4 * k + 7]));
    } else {
#pragma unroll
      for (int k = 0; k < V4; ++k)
        reinterpret_cast<uint2*>(dst)[k] = make_uint2(pack_bf16(o[4 * k], o[4 * k + 1]), pack_bf16(o[4 * k + 2], o[4 * k + 3]));
    }
  } else {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + off);
#pragma unroll
    for (int k = 0; k < V4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
  }
}

// A long cache with few rows leaves many parts to a tile, and their loads' latency is what counts:
// a block takes PJ_ROWS rows, and PJ_GROUPS threads share the parts of four dimensions of a row, each
// with four in flight.
constexpr int PJ_ROWS = 8, PJ_GROUPS = 2;
__global__ void __launch_bounds__(PJ_ROWS * 32 * PJ_GROUPS) k_attn_paged_few_join(const PagedArgs a) {
  __shared__ float4 s_o[PJ_GROUPS - 1][PJ_ROWS][32];
  __shared__ float s_m[PJ_GROUPS - 1][PJ_ROWS], s_l[PJ_GROUPS - 1][PJ_ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const PagedTile d = a.desc[blockIdx.x];
  if (d.first < 0) return;
  const int lane = threadIdx.x & 31, rr = (threadIdx.x >> 5) & (PJ_ROWS - 1), group = threadIdx.x / (32 * PJ_ROWS);
  const int row = blockIdx.y * PJ_ROWS + rr, r = d.tile * PD_M + row;
  if (d.tile * PD_M + blockIdx.y * PJ_ROWS >= d.n * a.G) return;
  float o[4], m, l;
  join_parts<1, 4>(a.part, PD_PART, PD_M * PG_D, PD_M, row, d.first, d.first + group, PJ_GROUPS, blockIdx.x, 1.0f,
                [&](int) { return row * PG_D + lane * 4; }, o, m, l);
  if (group > 0) {
    s_o[group - 1][rr][lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) {
      s_m[group - 1][rr] = m;
      s_l[group - 1][rr] = l;
    }
  }
  __syncthreads();
  if (group > 0 || r >= d.n * a.G) return;
  float mn = m;
#pragma unroll
  for (int g = 0; g < PJ_GROUPS - 1; ++g) mn = fmaxf(mn, s_m[g][rr]);
  const float mu = mn == -INFINITY ? 0.0f : mn;
  const float f0 = exp2_approx(__fsub_rn(m, mu));
  l = __fmul_rn(l, f0);
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = __fmul_rn(o[k], f0);
#pragma unroll
  for (int g = 0; g < PJ_GROUPS - 1; ++g) {
    const float f = exp2_approx(__fsub_rn(s_m[g][rr], mu));
    const float4 x = s_o[g][rr][lane];
    l = __fmaf_rn(s_l[g][rr], f, l);
    o[0] = __fmaf_rn(x.x, f, o[0]);
    o[1] = __fmaf_rn(x.y, f, o[1]);
    o[2] = __fmaf_rn(x.z, f, o[2]);
    o[3] = __fmaf_rn(x.w, f, o[3]);
  }
  divide_row(o, l);
  const int t = div_small(r, a.by_G);
  store_row<1>(a.out, a.out_dtype, ((long long)(d.t0 + t) * a.Hq + d.head * a.G + (r - t * a.G)) * PG_D + lane * 4, o);
}

}  // namespace bitnet
