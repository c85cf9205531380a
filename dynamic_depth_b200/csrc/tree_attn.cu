// Attention of draft trees (and single tokens) over a paged cache.
//
// The rows of one request that share a key head (nodes x query heads of the
// group, node major) are one matrix of queries; its keys are the request's
// context and its own nodes, read from the pages by TMA in tiles of KT
// positions.  Work is cut into units of one key tile of one (request, key
// head, block of BM query rows); the units, in that order, are dealt in equal
// contiguous ranges to two persistent CTAs per SM, so ragged lengths and few
// long requests fill the machine alike, and one CTA streams while the other is
// between row blocks.  A CTA whose range covers all tiles of
// a row block writes the result; a block cut by range boundaries leaves
// (max, sum, output) pieces in the workspace - at most two per CTA, whatever
// the problem - and a second, small kernel joins them in order.  No atomics:
// results do not depend on timing.
//
// Every row block of a request runs all of the request's tiles, also where no
// masks are given and its rows see only a part of the nodes: blocks of prompt
// positions are right but far from their floor (2 x 4,000 rows from an empty
// cache, 32 heads over 8, width 128: 1,180 us, floor 161; 8 x 128 rows behind
// 4,000 positions: 128 us, floor 42).
//
// Inside a CTA (flash attention, one pass over the keys with a running maximum
// and sum per row): a producer warp loads tiles into a ring of stages; four
// warps multiply, split over the block's 16-row parts and, where those are
// fewer than four, over parts of the tile's keys.  Every warp keeps its own
// running state over the keys it sees; the states of a row block meet once per
// block, in shared memory, where each warp joins and writes a share of the
// columns.  A page's part of a tile, keys and values of one
// head, is one four-dimensional TMA box: with one box per 64 columns of keys or
// values, pages of 16 positions streamed at 4.4 TB/s where pages of 64 reached
// 5.6.
//
// Bound by the cache's bytes: a position of a key head is 4 * hd bytes for
// 4 * hd * BM multiply-adds.  64 single tokens x 32 heads over 8 key heads, 4,000
// positions of width 128: 172 us, 6.1 TB/s (93 % of a copy), pages of 16 or 64;
// 512 such requests of 500 positions: 195 us, 5.4 TB/s (323 us with one CTA of
// eight multiplying warps an SM).
#include "tree_attn.h"

#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "host_util.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace tl {

// Driver entry point of the tensor-map encoder and 2D maps of row-major arrays (runtime.cu).
int encode_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                  uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw);
int encode_map_4d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, const uint64_t (&dims)[4],
                  const uint64_t (&strides)[3], const uint32_t (&box)[4], CUtensorMapSwizzle sw);

namespace tree {

constexpr int kWarps = 4;                     // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kLn2 = 0.6931471805599453f;
// Limits that keep positions, rows of a key head and mask bits, each rounded up to a tile, within 31 bits.
constexpr int64_t kMaxLen = (int64_t(1) << 31) - 4096, kMaxRows = int64_t(1) << 30;
constexpr int kMaxR = 1 << 20, kMaxWords = 1 << 20;

// How far, in powers of two, the reference of a row lies below the largest score
// seen: probabilities enter the second product up to 2^kLift times larger, and
// the sum and the natural-log result follow the same reference.  fp16 loses
// probabilities below 2^-14 of its 1 digit by digit, and all below 2^-25, while
// the sum keeps them: relative to the maximum itself, 6,000 keys at 2^-24.3 of
// the largest came out 3.6 % off.  At 2^7 what is lost is below 2^-32 of the
// largest, and the tensor-core kernel's probabilities (up to 2^8 past the
// reference) end at 2^15, inside fp16.  bf16 has fp32's range.
template <bool BF>
constexpr float kLift = BF ? 0.f : 7.f;

template <int HD>
struct Cfg {
  static constexpr int KT = HD == 128 ? 64 : 128;   // key positions per tile
  static constexpr int COLS = HD < 64 ? HD : 64;    // columns of a TMA box (one swizzled row)
  static constexpr int CT = HD / COLS;
  static constexpr int ROWB = COLS * 2;             // bytes of a box row
  static constexpr int STAGE = 2 * KT * HD * 2;     // K and V of a tile
  static constexpr int STAGES = HD == 32 ? 4 : 2;
  static constexpr int SLOT = (HD / 2 + 4) * 32;    // floats of one warp's state: output, 2 maxima, 2 sums
  static constexpr int MERGE = kWarps * SLOT * 4;
  static constexpr int SMEM = 1024 + STAGES * STAGE + MERGE + 256;
  static_assert(SMEM + 1024 <= 113 * 1024, "two CTAs per SM");
};

struct Req {
  int32_t row0, n, ctx, len, tiles, blocks;  // blocks: row blocks of a key head
  bool bad;
};

// A CTA's range of units, and where its first unit lies; kept in the workspace
// for the joining kernel.
struct Range {
  int64_t u0, u1;   // units of this CTA
  int64_t ua, ub;   // units of the row block that holds u0
  int64_t total;    // units in all
  int32_t r, hk, blk;
  // the CTAs with pieces of the row block that u0 cuts, first to last (between them some may have no units, where
  // there are fewer units than CTAs); -1: u0 cuts none, or it is not the block's first cut
  int32_t cut_first, cut_last;
  Req q;
};
// What the joining kernel needs beyond the range itself; thread 0 notes it when the CTA's work is done.
__device__ __forceinline__ void note_cut(const TreeAttnArgs& a, const Range& me) {
  Range* out = reinterpret_cast<Range*>(a.ws) + blockIdx.x;
  const uint64_t U = me.total, G = gridDim.x;
  auto owner = [&](uint64_t u) { return (int)(((u + 1) * G - 1) / U); };  // the CTA whose range holds u
  int first = -1, last = -1;
  if (me.u0 < me.u1 && me.u0 > me.ua) {
    const int p = owner(me.ua);
    if (owner(me.u0 - 1) == p) {
      first = p;
      last = owner(me.ub - 1);
    }
  }
  out->cut_first = first;
  out->cut_last = last;
}

// A piece of a row block in the workspace: (maximum, sum) of each row, then the
// output as [hd / 4][BM] groups of four values, so that neighbouring rows are
// neighbours in memory.  Two per CTA: 0 for a block that began in an earlier
// range, 1 for one that goes on in the next.
template <int HD, int BM>
struct Piece {
  float2 ml[BM];
  float4 o[HD / 4][BM];
};
template <int HD, int BM>
__device__ __forceinline__ Piece<HD, BM>* piece_of(const TreeAttnArgs& a, int ctas, int cta, int slot) {
  const size_t head = ((size_t)ctas * sizeof(Range) + 255) / 256 * 256;
  return reinterpret_cast<Piece<HD, BM>*>(a.ws + head) + (size_t)cta * 2 + slot;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <int KT, int BM>
__device__ __forceinline__ Req request(const TreeAttnArgs& a, int r) {
  Req q;
  const int c0 = a.cu[r], c1 = a.cu[r + 1], ctx = a.ctx[r];
  const int64_t cap = min((int64_t)a.max_pages << a.page_shift, kMaxLen);
  q.bad = c0 < 0 || c1 < c0 || c1 > a.n_rows || c1 - c0 > a.max_nodes || ctx < 0 ||
          (int64_t)ctx + a.node0 + (c1 - c0) > cap;
  q.row0 = c0;
  q.n = q.bad ? 0 : c1 - c0;
  q.ctx = ctx;
  q.len = ctx + a.node0 + q.n;
  q.tiles = q.len > 0 ? (q.len + KT - 1) / KT : 1;
  q.blocks = (int)(((int64_t)q.n * (a.H / a.Hk) + BM - 1) / BM);
  return q;
}

// The n lowest bits.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// Bits of the 32 positions from p0 on that a row sees.
__device__ __forceinline__ uint32_t row_sees(const TreeAttnArgs& a, const Req& q, int64_t row, int node, int p0) {
  const int j0 = p0 - q.ctx;  // node index of the first position
  uint32_t v = low_bits(-j0);      // the context
  if (j0 > -32) {
    if (a.masks) {
      const uint32_t* w = a.masks + row * a.words;
      auto word = [&](int i) { return i >= 0 && i < a.words ? __ldg(w + i) : 0u; };
      v |= j0 >= 0 ? __funnelshift_r(word(j0 >> 5), word((j0 >> 5) + 1), j0 & 31) : word(0) << -j0;
    } else {
      v |= low_bits(node + a.node0 + 1 - j0) & ~low_bits(-j0);
    }
  }
  return v & low_bits(q.len - p0);
}

// A stretch of one row block's key tiles within a CTA's range.
struct Seg {
  Req q;
  int32_t r, hk, blk, t0, t1;
};

// The stretches of a CTA's range, one after another.
template <int KT, int BM>
struct Walk {
  int64_t u, u1;  // units given out, and the range's end
  Seg s;          // the last one given out; t1 < 0: the first is still to come
  __device__ __forceinline__ explicit Walk(const Range& g)
      : u(g.u0), u1(g.u1), s{g.q, g.r, g.hk, g.blk, (int32_t)(g.u0 - g.ua), -1} {}
  __device__ __forceinline__ bool next(const TreeAttnArgs& a) {
    if (u >= u1) return false;
    if (s.t1 >= 0) {
      s.t0 = 0;
      if (++s.blk == s.q.blocks) {
        s.blk = 0;
        if (++s.hk == a.Hk) {
          s.hk = 0;
          do {
            if (s.r + 1 >= a.R) return false;  // only if the lengths changed during the call
            s.q = request<KT, BM>(a, ++s.r);
          } while (s.q.blocks == 0);
        }
      }
    }
    s.t1 = (int)min((int64_t)s.q.tiles, s.t0 + (u1 - u));
    u += s.t1 - s.t0;
    return true;
  }
};

// Block-wide: this CTA's range (valid after a __syncthreads).  Up to blockDim.x
// requests are read once; more take a second pass over the lengths.
template <int KT, int BM>
__device__ __forceinline__ void find_range(const TreeAttnArgs& a, Range* sh, long long* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long all = 0, u0 = 0, u1 = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long run = 0;
    for (int r0 = 0; r0 < a.R; r0 += blockDim.x) {
      const int r = r0 + threadIdx.x;
      long long x = 0;
      Req q;
      if (r < a.R) {
        q = request<KT, BM>(a, r);
        x = (long long)q.tiles * q.blocks * a.Hk;
        if (pass == 0 && q.bad && blockIdx.x == 0 && a.status) atomicOr(a.status, TL_BAD_LENGTH);
      }
      const long long mine = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
      }
      __syncthreads();
      if (lane == 31) wsum[warp] = x;
      __syncthreads();
      long long pre = run + x - mine;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w < warp) pre += wsum[w];
        run += wsum[w];
      }
      if (a.R <= (int)blockDim.x) {
        all = run;
        u0 = all * blockIdx.x / gridDim.x;
        u1 = all * (blockIdx.x + 1) / gridDim.x;
      }
      if ((pass == 1 || a.R <= (int)blockDim.x) && u0 < u1 && mine > 0 && u0 >= pre && u0 < pre + mine) {
        const int64_t item = (u0 - pre) / q.tiles;
        const int hk = (int)(item / q.blocks);
        *sh = Range{u0, u1, pre + item * q.tiles, pre + (item + 1) * q.tiles, all, r, hk,
                    (int)(item - (int64_t)hk * q.blocks), -1, -1, q};
        reinterpret_cast<Range*>(a.ws)[blockIdx.x] = *sh;
      }
    }
    if (a.R <= (int)blockDim.x) break;
    all = run;
    u0 = all * blockIdx.x / gridDim.x;
    u1 = all * (blockIdx.x + 1) / gridDim.x;
  }
  if (threadIdx.x == 0 && u0 >= u1) {  // nothing to do
    sh->u0 = sh->u1 = u0;
    reinterpret_cast<Range*>(a.ws)[blockIdx.x].u0 = u0;
    reinterpret_cast<Range*>(a.ws)[blockIdx.x].u1 = u0;
  }
}

// The producer warp: the tiles of the CTA's range into the ring, a box per page
// (or part of one) with the keys and values of its positions: [K, V][column
// tiles][positions][64 columns].
template <class C, int KT, int BM>
__device__ __forceinline__ void produce(const TreeAttnArgs& a, const CUtensorMap& kvmap, Walk<KT, BM> walk,
                                        uint8_t* ring, uint64_t* full, uint64_t* empty, volatile uint32_t* info,
                                        volatile int32_t* abort_flag) {
  const int lane = threadIdx.x & 31;
  const int P = 1 << a.page_shift, PR = P < KT ? P : KT, boxes = KT / PR, box_bytes = C::STAGE / boxes;
  const Seg& s = walk.s;
  int k = 0;
  bool ok = true;
  while (ok && walk.next(a)) {
    const int32_t* table = a.table + (int64_t)s.r * a.max_pages;
    auto page_of = [&](int t) {
      const int pos = t * KT + lane * PR;
      return lane < boxes && pos < s.q.len ? __ldg(table + (pos >> a.page_shift)) : -1;
    };
    int page = page_of(s.t0);
    for (int t = s.t0; t < s.t1; ++t, ++k) {
      const int next_page = t + 1 < s.t1 ? page_of(t + 1) : -1;
      const int st = k % C::STAGES, round = k / C::STAGES;
      if (round > 0 && !mbar_wait_warp(smem_u32(&empty[st]), (round - 1) & 1, abort_flag)) { ok = false; break; }
      const int pos = t * KT + lane * PR;
      const bool want = lane < boxes && pos < s.q.len;
      const bool good = want && page >= 0 && page < a.n_pages;
      if (want && !good && a.status) atomicOr(a.status, TL_BAD_PAGE);
      const uint32_t in = __ballot_sync(0xffffffffu, good);
      const uint32_t bar = smem_u32(&full[st]);
      if (lane == 0) {
        info[st] = in;
        mbar_expect_tx(bar, __popc(in) * box_bytes);
      }
      __syncwarp();
      if (good) {
        const int64_t y = (((int64_t)page * 2 * a.Hk + s.hk) << a.page_shift) + (pos & (P - 1));
        tma_load_4d(smem_u32(ring + st * C::STAGE) + lane * box_bytes, &kvmap, 0, (int)y, 0, 0, bar);
      }
      __syncwarp();
      page = next_page;
    }
  }
  if (!ok && lane == 0) {  // let the copies in flight land
    volatile int32_t never = 0;
    for (int i = k > C::STAGES ? k - C::STAGES : 0; i < k; ++i)
      mbar_wait(smem_u32(&full[i % C::STAGES]), (i / C::STAGES) & 1, &never);
  }
}

}  // namespace tree
}  // namespace tl

#include "tree_attn_tc.cuh"

namespace tl {
namespace tree {

template <int HD, int WM, bool BF>
__global__ void __launch_bounds__(kThreads, 2)
tree_attn_kernel(const __grid_constant__ CUtensorMap kvmap, const TreeAttnArgs a) {
  using C = Cfg<HD>;
  constexpr int KT = C::KT, BM = 16 * WM, WN = 4 / WM, KW = KT / WN, NT = KW / 8;
  extern __shared__ __align__(1024) uint8_t smem_ta[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_ta) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(ring + C::STAGES * C::STAGE);
  uint64_t* full = reinterpret_cast<uint64_t*>(merge + kWarps * C::SLOT);
  uint64_t* empty = full + C::STAGES;
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(empty + C::STAGES);  // [STAGES] boxes that landed
  __shared__ int32_t abort_s;
  __shared__ Range range_s;
  __shared__ long long wsum[kWarps + 1];
  volatile int32_t* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 4);
    }
    abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_launch_dependents();
  __syncthreads();
  find_range<KT, BM>(a, &range_s, wsum);
  __syncthreads();
  if (range_s.u0 < range_s.u1) {
    Walk<KT, BM> walk(range_s);
    const Seg& s = walk.s;
    const int64_t u_first = walk.u;
    const int P = 1 << a.page_shift;
    const int PR = P < KT ? P : KT, boxes = KT / PR;  // positions per box, boxes per tile
    const uint32_t all_boxes = (1u << boxes) - 1u;
    int k = 0;  // tiles of this CTA so far
    if (warp == kWarps) {
      produce<C, KT, BM>(a, kvmap, walk, ring, full, empty, info, abort_flag);
    } else {
      // ----------------------------------------------------------- consumers
      const int wm = warp % WM, wn = warp / WM;
      // a 16-byte chunk of a tile row: the row's box, the head's K or V in it, the row, the chunk swizzled by the row
      const int pshift = 31 - __clz(PR), box_bytes = C::STAGE / boxes, col_bytes = PR * C::ROWB;
      auto row_at = [&](int y) { return (y >> pshift) * box_bytes + (y & (PR - 1)) * C::ROWB; };
      auto chunk_at = [&](int y, int c) {  // c static or not; K (V: + CT column tiles)
        const int sw = C::ROWB == 128 ? (y & 7) : ((y >> 1) & 3);
        return row_at(y) + (c / (C::COLS / 8)) * col_bytes + (((c % (C::COLS / 8)) ^ sw) << 4);
      };
      const int G = a.H / a.Hk;
      const int r0 = lane >> 2, c0 = (lane & 3) * 2;  // the thread's rows r0, r0 + 8; columns c0, c0 + 1 of each 8
      // the lane's rows of the 16-key steps that it addresses for ldmatrix, and its swizzled column bits
      uint32_t k_row[NT / 2], v_row[NT / 2];
      const int sw = C::ROWB == 128 ? (lane & 7) : ((lane & 7) >> 1);
      const uint32_t k_col = (((lane >> 3) & 1) ^ sw) << 4, v_col = (((lane >> 4) & 1) ^ sw) << 4;
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        k_row[j] = row_at(wn * KW + j * 16 + (lane & 7) + ((lane >> 4) & 1) * 8);
        v_row[j] = row_at(wn * KW + j * 16 + (lane & 7) + ((lane >> 3) & 1) * 8);
      }
      bool ok = true;
      while (walk.next(a)) {
        const Req& q = s.q;
        const int rows = q.n * G;
        int rho[2], node[2];
        const uint8_t* qp[2];
        int64_t row[2];
        int head[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rho[i] = s.blk * BM + wm * 16 + r0 + 8 * i;
          const bool in = rho[i] < rows;
          node[i] = in ? rho[i] / G : -1;
          head[i] = s.hk * G + (in ? rho[i] - node[i] * G : 0);
          row[i] = q.row0 + (in ? node[i] : 0);
          qp[i] = static_cast<const uint8_t*>(a.q) + (row[i] * a.q_stride + (int64_t)head[i] * HD) * 2;
        }
        uint32_t qf[HD / 16][4];
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = e & 1, col = kk * 16 + c0 + (e >> 1) * 8;
            // (no read-only load: the output may take the queries' place, row block by row block)
            qf[kk][e] = node[i] >= 0 ? *reinterpret_cast<const uint32_t*>(qp[i] + col * 2) : 0u;
          }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float O[HD / 8][4];
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[i][e] = 0.f;

        for (int t = s.t0; t < s.t1; ++t, ++k) {
          const int st = k % C::STAGES;
          if (ok) ok = mbar_wait_warp(smem_u32(&full[st]), (k / C::STAGES) & 1, abort_flag);
          if (!ok) continue;
          uint8_t* sk = ring + st * C::STAGE;
          uint8_t* sv = sk + C::CT * col_bytes;
          const uint32_t ka = smem_u32(sk), va = smem_u32(sv);
          const uint32_t landed = info[st];
          const int key0 = t * KT + wn * KW;  // first position of this warp's part
          // -------------------------------------------------- S = Q K^T
          float S[NT][4];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
              uint32_t b[4];
              ldsm4(ka + k_row[j] + (kk * 2 / (C::COLS / 8)) * col_bytes + ((kk * 2 % (C::COLS / 8) * 16) ^ k_col), b);
              mma16816<BF>(S[2 * j], qf[kk], b[0], b[1]);
              mma16816<BF>(S[2 * j + 1], qf[kk], b[2], b[3]);
            }
          // -------------------------------------------------- what each row sees
          const bool mask = landed != all_boxes || key0 + KW > q.ctx;
          bool odd_v = false;  // values of the tree hold NaN or infinity
          // Values of positions that nobody sees may be anything, and 0 * NaN is not 0: they leave the matrix product as
          // zeros, by masks of the lane's two keys of each 8 (64 ragged single tokens: 123 us then,
          // 135 with zeros written to the tile).
          uint32_t vm[NT / 2][2];
          if (mask) {
            constexpr uint32_t X = BF ? 0x7f80u : 0x7c00u;
            uint32_t tm[NT / 2][2];  // the tree's among them
            uint32_t see[2], there = 0, tree = 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              // Of 32 positions, those that the rows see, that there are, and the tree's, as words: tested one by one
              // they made a block's last tile cost as much as two (64 ragged single tokens 123 us, 116 so).
              if (i % 4 == 0) {
                const int p0 = key0 + i * 8;
#pragma unroll
                for (int e = 0; e < 2; ++e) see[e] = row_sees(a, q, row[e], node[e], p0);
                there = low_bits(q.len - p0);
                tree = there & ~low_bits(q.ctx - p0);
              }
              const int at = i % 4 * 8 + c0;
              const uint32_t box = landed >> ((wn * KW + i * 8) >> pshift) & 1u ? 3u : 0u;
              const uint32_t v = there >> at & box, w = tree >> at & box;
              vm[i / 2][i & 1] = (v & 1u) * 0xffffu | (v >> 1) * 0xffff0000u;
              tm[i / 2][i & 1] = (w & 1u) * 0xffffu | (w >> 1) * 0xffff0000u;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!(see[e >> 1] >> at & box & (e & 1 ? 2u : 1u))) S[i][e] = -INFINITY;
            }
            if ((q.len > q.ctx + 1 || a.masks) && key0 + KW > q.ctx) {
#pragma unroll
              for (int j = 0; j < NT / 2; ++j)
#pragma unroll
                for (int d = 0; d < HD / 16; ++d) {
                  uint32_t b[4];
                  ldsm4t(va + v_row[j] + (d * 2 / (C::COLS / 8)) * col_bytes + ((d * 2 % (C::COLS / 8) * 16) ^ v_col), b);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t w = b[e] & tm[j][e & 1];
                    odd_v |= (w & X) == X || (w >> 16 & X) == X;
                  }
                }
              odd_v = __any_sync(0xffffffffu, odd_v);
            }
          }
          // -------------------------------------------------- running maximum and sum
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mx[0] = fmaxf(mx[0], fmaxf(S[i][0], S[i][1]));
            mx[1] = fmaxf(mx[1], fmaxf(S[i][2], S[i][3]));
          }
          float mb[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            const float mn = fmaxf(m[i], mx[i] * a.scale_log2 - kLift<BF>);
            mb[i] = mn == -INFINITY ? 0.f : mn;
            const float corr = ex2(m[i] - mb[i]);  // 0 from -inf
            l[i] *= corr;
            if (mn != m[i]) {
#pragma unroll
              for (int d = 0; d < HD / 8; ++d) { O[d][2 * i] *= corr; O[d][2 * i + 1] *= corr; }
            }
            m[i] = mn;
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              S[i][e] = ex2(fmaf(S[i][e], a.scale_log2, -mb[e >> 1]));
              l[e >> 1] += S[i][e];
            }
          // -------------------------------------------------- O += P V
          // one rounding of each probability to the values' type (the matrix instruction takes one type)
          auto pv = [&](auto masked) {
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
              const uint32_t p[4] = {pack2<BF>(S[2 * j][0], S[2 * j][1]), pack2<BF>(S[2 * j][2], S[2 * j][3]),
                                     pack2<BF>(S[2 * j + 1][0], S[2 * j + 1][1]),
                                     pack2<BF>(S[2 * j + 1][2], S[2 * j + 1][3])};
#pragma unroll
              for (int d = 0; d < HD / 16; ++d) {
                uint32_t b[4];
                ldsm4t(va + v_row[j] + (d * 2 / (C::COLS / 8)) * col_bytes + ((d * 2 % (C::COLS / 8) * 16) ^ v_col), b);
                if constexpr (masked.value) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) b[e] &= vm[j][e & 1];
                }
                mma16816<BF>(O[2 * d], p, b[0], b[1]);
                mma16816<BF>(O[2 * d + 1], p, b[2], b[3]);
              }
            }
          };
          if (!mask) {
            pv(std::false_type{});
          } else if (!odd_v) {
            pv(std::true_type{});
          } else {
            // a value that some row does not see is not finite: products by hand, where the row sees the key
            float pl[NT * 4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) pl[i * 4 + e] = S[i][e];
#pragma unroll 1
            for (int y = 0; y < KW; ++y) {
              const int src = (lane & ~3) | ((y & 7) >> 1), e = y & 1;
              const float p0 = __shfl_sync(0xffffffffu, pl[(y >> 3) * 4 + e], src);
              const float p1 = __shfl_sync(0xffffffffu, pl[(y >> 3) * 4 + 2 + e], src);
#pragma unroll
              for (int d = 0; d < HD / 8; ++d) {
                const float2 v = unpack2<BF>(*reinterpret_cast<const uint32_t*>(
                    sv + chunk_at(wn * KW + y, d) + c0 * 2));
                if (p0 != 0.f) { O[d][0] = fmaf(p0, v.x, O[d][0]); O[d][1] = fmaf(p0, v.y, O[d][1]); }
                if (p1 != 0.f) { O[d][2] = fmaf(p1, v.x, O[d][2]); O[d][3] = fmaf(p1, v.y, O[d][3]); }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
        }

        // ---------------------------------------- the states of a row block meet
        // The WN warps of 16 rows put their states down; each then joins its share of the columns and writes it.
        constexpr int ND = HD / 8 / WN;  // groups of 8 columns of a warp's share
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        float X[ND][4];
        if constexpr (WN == 1) {
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[d][e] = O[d][e];
        } else {
          float* b = merge + warp * C::SLOT + lane;
#pragma unroll
          for (int d = 0; d < HD / 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) b[(d * 4 + e) * 32] = O[d][e];
          b[(HD / 2) * 32] = m[0];
          b[(HD / 2 + 1) * 32] = m[1];
          b[(HD / 2 + 2) * 32] = l[0];
          b[(HD / 2 + 3) * 32] = l[1];
          asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
          float f[WN][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mn = -INFINITY, ln = 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
              f[w][i] = merge[(wm + w * WM) * C::SLOT + (HD / 2 + i) * 32 + lane];
              mn = fmaxf(mn, f[w][i]);
            }
            const float z = mn == -INFINITY ? 0.f : mn;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
              f[w][i] = ex2(f[w][i] - z);  // a state that saw nothing adds nothing
              ln = fmaf(merge[(wm + w * WM) * C::SLOT + (HD / 2 + 2 + i) * 32 + lane], f[w][i], ln);
            }
            m[i] = mn;
            l[i] = ln;
          }
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = 0.f;
#pragma unroll
              for (int w = 0; w < WN; ++w)
                x = fmaf(merge[(wm + w * WM) * C::SLOT + ((wn * ND + d) * 4 + e) * 32 + lane], f[w][e >> 1], x);
              X[d][e] = x;
            }
          asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // read before the next block's states
        }
        if (ok) {
          const bool whole = s.t0 == 0 && s.t1 == q.tiles;
          const int col0 = wn * ND * 8 + c0;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (node[i] < 0) continue;
              const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
              const int64_t o = row[i] * a.out_stride + (int64_t)head[i] * HD + col0;
#pragma unroll
              for (int d = 0; d < ND; ++d) {
                const float x = X[d][2 * i] * inv, y = X[d][2 * i + 1] * inv;
                if (a.out_f32)
                  *reinterpret_cast<float2*>(static_cast<float*>(a.out) + o + d * 8) = make_float2(x, y);
                else
                  *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o + d * 8) = pack2<BF>(x, y);
                if (a.out16) {
                  act16_put(a.out16, row[i], a.H * HD, head[i] * HD + d * 8 + col0, x, a.split16);
                  act16_put(a.out16, row[i], a.H * HD, head[i] * HD + d * 8 + col0 + 1, y, a.split16);
                }
              }
              if (a.lse && wn == 0 && (lane & 3) == 0)
                a.lse[row[i] * a.H + head[i]] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
            }
          } else {
            // slot 0: the CTA's first stretch, when it does not begin the row block; slot 1: the last
            const int64_t begin = walk.u - (s.t1 - s.t0);
            auto* w = piece_of<HD, BM>(a, gridDim.x, blockIdx.x, begin == u_first && s.t0 > 0 ? 0 : 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int y = wm * 16 + r0 + 8 * i;
              if (wn == 0 && (lane & 3) == 0) w->ml[y] = make_float2(m[i], l[i]);
#pragma unroll
              for (int d = 0; d < ND; ++d)
                reinterpret_cast<float2*>(&w->o[(wn * ND + d) * 2 + c0 / 4][y])[c0 / 2 & 1] =
                    make_float2(X[d][2 * i], X[d][2 * i + 1]);
            }
          }
        }
      }
    }
  }
  if (threadIdx.x == 0) note_cut(a, range_s);
  __syncthreads();
  if (threadIdx.x == 0 && abort_s && a.status) atomicOr(a.status, TL_TIMED_OUT);
}

// Joins the pieces of the row blocks that the CTAs' ranges cut: CTA b looks at
// the cut at the start of range b, and acts if it is the first of its block.  A
// lane a row, four output columns at a time; the rows and the halves of the
// columns are dealt over blockIdx.y.  Short chains of loads are what counts:
// the range, then maxima and sums and the first outputs together.
template <int HD, int BM, bool BF>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeAttnArgs a) {
  constexpr int RW = BM < 32 ? BM : 32, CW = 32 / RW;  // rows of a warp, column groups it takes at once
  constexpr int N = 4;                                 // pieces at a time
  pdl_wait();
  const Range* ranges = reinterpret_cast<const Range*>(a.ws);
  const int G = gridDim.x, b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p = ranges[b].cut_first, e = ranges[b].cut_last;
  if (p < 0) return;
  const Range me = ranges[b];
  const bool dense = me.total >= G;  // every CTA has units
  const int grp = a.H / a.Hk;
  const int y = (blockIdx.y >> 1) * RW + lane % RW, rho = me.blk * BM + y;
  if (rho >= me.q.n * grp) return;
  const int node = rho / grp, head = me.hk * grp + rho - node * grp;
  const int64_t row = me.q.row0 + node;
  auto holds = [&](int c) { return c <= e && (dense || ranges[c].u0 < ranges[c].u1); };
  float2 ml[N];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      ml[i] = holds(c0 + i) ? piece_of<HD, BM>(a, G, c0 + i, c0 + i == p)->ml[y] : make_float2(-INFINITY, 0.f);
  };
  float m = -INFINITY, l = 0.f;
  for (int c = p; c <= e; c += N) {
    load(c);
    float mn = m;
#pragma unroll
    for (int i = 0; i < N; ++i) mn = fmaxf(mn, ml[i].x);
    const float z = mn == -INFINITY ? 0.f : mn;
    l *= ex2(m - z);
#pragma unroll
    for (int i = 0; i < N; ++i) l += ml[i].y * ex2(ml[i].x - z);
    m = mn;
  }
  const float z = m == -INFINITY ? 0.f : m, inv = l > 0.f || l != l ? 1.f / l : 0.f;
  constexpr int half = HD / 8;  // column groups of a half
  for (int c = (blockIdx.y & 1) * half + warp * CW + lane / RW; c < ((int)(blockIdx.y & 1) + 1) * half; c += 8 * CW) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = p; c0 <= e; c0 += N) {
      if (e - p >= N) load(c0);
      float4 v[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = holds(c0 + i) ? piece_of<HD, BM>(a, G, c0 + i, c0 + i == p)->o[c][y] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float f = ex2(ml[i].x - z);
        o.x += f * v[i].x;
        o.y += f * v[i].y;
        o.z += f * v[i].z;
        o.w += f * v[i].w;
      }
    }
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    const int64_t at = row * a.out_stride + (int64_t)head * HD + c * 4;
    if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(pack2<BF>(o.x, o.y), pack2<BF>(o.z, o.w));
    if (a.out16) {
      const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) act16_put(a.out16, row, a.H * HD, head * HD + c * 4 + i, v[i], a.split16);
    }
  }
  if (a.lse && blockIdx.y % 2 == 0 && warp == 0 && lane < RW)
    a.lse[row * a.H + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Rows of a block: the smallest that holds a request's rows of a key head.  More than 32 rows of widths 64 and 128
// take the tensor-core kernel's 128.  That kernel's tiles are 64 columns (one 128-byte swizzled row) wide, so width 32
// stays on the warp-level instructions, in blocks of 64 rows: 16 requests x 32 nodes x 4 heads over 8 key heads, 4,000
// positions, take 58 us (5.6 times the time of their bytes), no less than width 64 on the tensor cores (57 us, 2.8
// times).
static int block_rows(int hd, int64_t rows_per_head) {
  if (rows_per_head <= 16) return 16;
  if (rows_per_head <= 32) return 32;
  return hd >= 64 ? 128 : 64;
}

template <int HD, int KT, int BM, bool BF, class K>
static int launch(K kern, int ctas, int threads, int smem, const TreeAttnArgs& a, const tl_kv_pool& p,
                  cudaStream_t s) {
  constexpr uint32_t cols = HD < 64 ? HD : 64;
  constexpr CUtensorMapSwizzle sw = cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const CUtensorMapDataType dt = BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap map;
  const uint64_t rows = (uint64_t)p.n_pages * 2 * p.n_kv_heads * p.page_tokens;
  const uint32_t pr = p.page_tokens < KT ? p.page_tokens : KT;
  if (BM == 128) {  // boxes of 64 columns: the layout that the tensor core reads has positions next to one another
    TL_TRY(encode_map_2d(&map, dt, p.dev_pool, HD, rows, HD * 2, cols, pr, sw));
  } else {          // columns, positions, column tiles, K and V
    TL_TRY(encode_map_4d(&map, dt, p.dev_pool, {cols, rows, HD / cols, 2},
                         {HD * 2, cols * 2, (uint64_t)p.n_kv_heads * p.page_tokens * HD * 2}, {cols, pr, HD / cols, 2},
                         sw));
  }
  static std::atomic<uint64_t> set{0};  // per kernel: one bit per device
  int dev = 0;
  TL_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(set >> dev & 1)) {
    TL_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (dev < 64) set |= 1ull << dev;
  }
  kern<<<ctas, threads, smem, s>>>(map, a);
  TL_CUDA(cudaGetLastError());
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(ctas, 2 * (BM < 32 ? 1 : BM / 32));
  lc.blockDim = dim3(256);
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  TL_CUDA(cudaLaunchKernelEx(&lc, tree_join_kernel<HD, BM, BF>, a));
  return check_cuda(cudaGetLastError());
}

template <int HD, bool BF>
static int run(const TreeAttnArgs& a, const tl_kv_pool& p, int n_sms, cudaStream_t s) {
  using C = Cfg<HD>;
  switch (block_rows(HD, (int64_t)a.max_nodes * (a.H / a.Hk))) {
    case 16: return launch<HD, C::KT, 16, BF>(tree_attn_kernel<HD, 1, BF>, 2 * n_sms, kThreads, C::SMEM, a, p, s);
    case 32: return launch<HD, C::KT, 32, BF>(tree_attn_kernel<HD, 2, BF>, 2 * n_sms, kThreads, C::SMEM, a, p, s);
    default:
      if constexpr (HD == 32)
        return launch<HD, C::KT, 64, BF>(tree_attn_kernel<HD, 4, BF>, 2 * n_sms, kThreads, C::SMEM, a, p, s);
      else
        return launch<HD, TcCfg<HD>::KT, 128, BF>(tree_attn_tc_kernel<HD, BF>, 2 * n_sms, TcCfg<HD>::THREADS,
                                                  TcCfg<HD>::SMEM, a, p, s);
  }
}

static int sm_count(int* n) {
  int dev = 0;
  TL_CUDA(cudaGetDevice(&dev));
  TL_CUDA(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev));
  return TL_OK;
}

}  // namespace tree

size_t tree_attn_workspace(int hd, int64_t rows_per_head, int n_sms) {
  const int rows = tree::block_rows(hd, rows_per_head);
  const size_t ctas = 2 * (size_t)n_sms;
  return (ctas * sizeof(tree::Range) + 255) / 256 * 256 + ctas * 2 * rows * (hd + 2) * 4;
}

int tree_attn_run(TreeAttnArgs a, const tl_kv_pool& p, cudaStream_t s, int64_t* launches) {
  int n_sms = 0;
  TL_TRY(tree::sm_count(&n_sms));
  if (a.max_sms && n_sms > a.max_sms) n_sms = a.max_sms;
  a.Hk = p.n_kv_heads;
  a.n_pages = p.n_pages;
  a.page_shift = 0;
  while ((1 << a.page_shift) < p.page_tokens) ++a.page_shift;
  if (launches) *launches += 2;
  const bool bf = p.dtype == TL_BF16;
  switch (p.head_dim) {
    case 32: return bf ? tree::run<32, true>(a, p, n_sms, s) : tree::run<32, false>(a, p, n_sms, s);
    case 64: return bf ? tree::run<64, true>(a, p, n_sms, s) : tree::run<64, false>(a, p, n_sms, s);
    default: return bf ? tree::run<128, true>(a, p, n_sms, s) : tree::run<128, false>(a, p, n_sms, s);
  }
}

}  // namespace tl

using namespace tl;

extern "C" int tl_tree_attention_workspace(int32_t head_dim, int32_t n_heads, int32_t n_kv_heads, int32_t max_nodes,
                                           size_t* out_bytes) {
  if (!out_bytes || (head_dim != 32 && head_dim != 64 && head_dim != 128) || n_heads < 1 || n_kv_heads < 1 ||
      n_heads % n_kv_heads || max_nodes < 1)
    return TL_EINVAL;
  int n_sms = 0;
  TL_TRY(tree::sm_count(&n_sms));
  *out_bytes = tree_attn_workspace(head_dim, (int64_t)max_nodes * (n_heads / n_kv_heads), n_sms);
  return TL_OK;
}

extern "C" int tl_tree_attention(const void* dev_q, int64_t q_stride, const tl_kv_pool* pool,
                                 const int32_t* dev_block_table, int32_t max_pages, const int32_t* dev_ctx,
                                 const int32_t* dev_cu, int32_t R, int32_t n_rows, int32_t n_heads, int32_t max_nodes,
                                 const uint32_t* dev_masks, int32_t mask_words, float scale, void* dev_out,
                                 int32_t out_dtype, int64_t out_stride, float* dev_lse, void* dev_workspace,
                                 size_t workspace_bytes, int32_t* dev_status, void* cuda_stream) {
  if (!kv_pool_ok(pool)) return TL_EINVAL;
  const int64_t width = (int64_t)n_heads * pool->head_dim;
  const int os = out_dtype == TL_F32 ? 4 : 2;
  if (n_heads < 1 || n_heads % pool->n_kv_heads || R < 0 || R > tree::kMaxR || n_rows < 0 || max_pages < 1 ||
      max_nodes < 1 ||
      (out_dtype != TL_F32 && out_dtype != pool->dtype) || (n_rows > 1 && (q_stride < width || out_stride < width)) ||
      (q_stride * 2) % 16 || (out_stride * os) % 16 || (mask_words > 0 ? !dev_masks && n_rows > 0 : dev_masks != nullptr) || mask_words < 0 ||
      mask_words > tree::kMaxWords ||
      (dev_masks && max_nodes > 32 * (int64_t)mask_words) || !(scale >= 0.f) || scale > 1e38f ||
      (int64_t)max_nodes * (n_heads / pool->n_kv_heads) > tree::kMaxRows)
    return TL_EINVAL;
  if (R == 0 || n_rows == 0) return TL_OK;
  if (!dev_q || !dev_block_table || !dev_ctx || !dev_cu || !dev_out || !dev_workspace) return TL_EINVAL;
  if (((uintptr_t)dev_q & 15) || ((uintptr_t)dev_out & 15) || ((uintptr_t)dev_block_table & 3) ||
      ((uintptr_t)dev_ctx & 3) || ((uintptr_t)dev_cu & 3) || ((uintptr_t)dev_masks & 3) || ((uintptr_t)dev_lse & 3) ||
      ((uintptr_t)dev_workspace & 255) || ((uintptr_t)dev_status & 3))
    return TL_EINVAL;
  // The output may be the queries' own place: a row block is written by the one CTA that read its queries, or by the
  // joining kernel.  Any other overlap lets one block's output overwrite another's queries; rows that only interleave
  // share nothing.
  const int64_t rows1 = n_rows - 1, qb = q_stride * 2, ob = out_stride * os, qw = width * 2, ow = width * os;
  const bool same = dev_q == dev_out && os == 2 && (rows1 == 0 || qb == ob);
  if (!same && share_bytes({dev_q, (size_t)(rows1 * qb + qw)}, {dev_out, (size_t)(rows1 * ob + ow)})) {
    if (rows1 == 0 || qb != ob) return TL_EINVAL;
    const int64_t d = (int64_t)((intptr_t)dev_out - (intptr_t)dev_q) % qb, at = d < 0 ? d + qb : d;
    if (at < qw || at + ow > qb) return TL_EINVAL;
  }
  size_t need = 0;
  TL_TRY(tl_tree_attention_workspace(pool->head_dim, n_heads, pool->n_kv_heads, max_nodes, &need));
  if (workspace_bytes < need) return TL_ENOMEM;
  if (scale == 0.f) scale = 1.f / sqrtf((float)pool->head_dim);
  TreeAttnArgs a{};
  a.q = dev_q;
  a.q_stride = q_stride;
  a.table = dev_block_table;
  a.max_pages = max_pages;
  a.ctx = dev_ctx;
  a.cu = dev_cu;
  a.R = R;
  a.n_rows = n_rows;
  a.H = n_heads;
  a.max_nodes = max_nodes;
  a.masks = dev_masks;
  a.words = mask_words;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.out = dev_out;
  a.out_f32 = out_dtype == TL_F32;
  a.out_stride = out_stride;
  a.lse = dev_lse;
  a.ws = static_cast<char*>(dev_workspace);
  a.status = dev_status;
  return tree_attn_run(a, *pool, (cudaStream_t)cuda_stream);
}
