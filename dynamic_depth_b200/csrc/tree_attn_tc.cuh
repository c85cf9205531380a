// Tree attention on the 5th-generation tensor cores (tcgen05 + TMEM), for row
// blocks of more rows than the warp-level matrix instructions keep up with.
// Same units, ranges, pieces and page handling as tree_attn_kernel.
//
// One CTA per SM; a row block is 128 query rows (one TMEM lane, one thread
// each), a tile 128 key positions:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, into one of two
//                  TMEM buffers, so the next tile's product runs under this
//                  tile's softmax
//   P = exp2(S-m)  one thread a row; 16-bit P replaces S in its TMEM buffer
//   O += P V       tcgen05.mma with P as the TMEM operand A and V (rows of
//                  keys) as the N-major operand B, accumulating in TMEM
// The reference m of a row moves only when a tile's maximum passes it by more
// than 2^8 (P then stays below 256, far inside fp16 and bf16, and sums are
// fp32), so O is rescaled in TMEM a few times per row block instead of once
// per tile.
//
// Warp 0: TMA producer; warp 1: MMA issuer; warp 2: TMEM; warps 4-7: rows.
// Bound by the cache's bytes up to 128 rows: 128 positions of width 128 are
// 64 KB (about 2,800 cycles of one SM's share of HBM) against 16 MMAs of
// 128 x 128 x 16 and 128 exponentials a thread.
#pragma once

#include "ptx.cuh"

namespace tl {
namespace tree {

template <int HD>
struct TcCfg {
  static constexpr int KT = 128, BM = 128;
  static constexpr int CT = HD / 64;               // 64-wide column tiles
  static constexpr int TILE = KT * 128;            // bytes of one: [128 positions x 64] 16 bit
  static constexpr int STAGE = 2 * CT * TILE;      // K tiles, then V tiles
  static constexpr int STAGES = HD == 128 ? 3 : 6;
  static constexpr int Q_BYTES = BM * HD * 2;
  static constexpr int SMEM = 1024 + Q_BYTES + STAGES * STAGE + 256;
  static constexpr int TMEM_COLS = 512;            // S / P twice 128, O HD
  static_assert(SMEM <= 227 * 1024, "tile ring does not fit");
  // a second CTA on the SM would wait for TMEM that the first holds: the ring leaves no room for one
  static_assert(SMEM > 114 * 1024, "one CTA per SM");
};

__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {  // 128-byte swizzle
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | (2ull << 61);
}
// D fp32; A, B fp16 or bf16; A K-major, B K-major or N-major; M = 128.
__device__ __forceinline__ constexpr uint32_t tc_idesc(bool bf, int N, int b_mn) {
  return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive columns of the thread's lane (tc_wait_ld before the values are used).
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Whether any of the 128 row threads says so (all of them call it).
__device__ __forceinline__ bool rows_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Bits of the 32 positions from p0 on that a row sees.
__device__ __forceinline__ uint32_t row_sees(const TreeAttnArgs& a, const Req& q, int64_t row, int node, int p0,
                                             uint32_t landed, int PR, int tile_off) {
  auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
  const int j0 = p0 - q.ctx;  // node index of the first position
  uint32_t v = low(-j0);      // the context
  if (j0 > -32 && node >= 0) {
    if (a.masks) {
      const uint32_t* w = a.masks + row * a.words;
      auto word = [&](int i) { return i >= 0 && i < a.words ? __ldg(w + i) : 0u; };
      v |= j0 >= 0 ? __funnelshift_r(word(j0 >> 5), word((j0 >> 5) + 1), j0 & 31) : word(0) << -j0;
    } else {
      v |= low(node + 1 - j0) & ~low(-j0);
    }
  }
  const uint32_t lo = landed >> (tile_off / PR) & 1u, hi = landed >> ((tile_off + 16) / PR) & 1u;
  return v & low(q.len - p0) & ((lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u));
}

template <int HD, bool BF>
__global__ void __launch_bounds__(256, 1)
tree_attn_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const TreeAttnArgs a) {
  using C = TcCfg<HD>;
  constexpr int KT = C::KT, BM = C::BM, ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_tt[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_tt) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = sQ + C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ST * C::STAGE);
  uint64_t* empty = full + ST;
  uint64_t* s_full = empty + ST;   // [2] S of a tile in TMEM
  uint64_t* p_full = s_full + 2;   // [2] P of a tile in TMEM, V clean
  uint64_t* o_full = p_full + 2;   // [2] P V of a tile added
  uint64_t* q_full = o_full + 2;   // Q of a row block in shared memory
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(q_full + 1);  // [ST] boxes that landed
  __shared__ int32_t abort_s;
  __shared__ uint32_t tmem_s;
  __shared__ int64_t total_s;
  __shared__ Start start_s;
  __shared__ long long wsum[8];
  volatile int32_t* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&p_full[b]), 4);
      mbar_init(smem_u32(&o_full[b]), 1);
    }
    mbar_init(smem_u32(q_full), 4);
    abort_s = 0;
    start_s = Start{0, 0, 0, 0};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)),
                 "r"((uint32_t)C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  tc_before();
  __syncthreads();
  tc_after();
  find_range<KT, BM>(a, &total_s, &start_s, wsum);
  __syncthreads();
  const uint32_t tmem = tmem_s;
  const int64_t total = total_s;
  Walk<KT, BM> walk;
  walk.u = total * blockIdx.x / gridDim.x;
  walk.u1 = total * (blockIdx.x + 1) / gridDim.x;
  const int64_t u_first = walk.u;
  if (threadIdx.x == 0) {
    Start st = start_s;
    st.total = total;
    reinterpret_cast<Start*>(a.ws)[blockIdx.x] = st;
  }
  if (walk.u < walk.u1 && warp != 2 && warp != 3) {
    walk.base = start_s.base;
    walk.r = start_s.r;
    walk.q = request<KT, BM>(a, walk.r);
    const int P = 1 << a.page_shift;
    const int PR = P < KT ? P : KT, boxes = KT / PR;
    const uint32_t all_boxes = (1u << boxes) - 1u;
    Seg s;
    int k = 0;  // tiles of this CTA so far
    if (warp == 0) {
      produce<C, KT, BM>(a, kvmap, walk, ring, full, empty, info, abort_flag);
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t id_s = tc_idesc(BF, KT, 0), id_o = tc_idesc(BF, HD, 1);
      bool ok = true;
      auto issue_s = [&](int kk) {
        const int st = kk % ST;
        if (!mbar_wait_warp(smem_u32(&full[st]), (kk / ST) & 1, abort_flag)) return false;
        tc_after();
        const uint8_t* kt = ring + st * C::STAGE;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
            tc_mma_ss(tmem + (kk & 1) * KT, tc_desc(smem_u32(sQ + (i / 4) * (BM * 128)) + (i % 4) * 32, 16, 1024),
                      tc_desc(smem_u32(kt + (i / 4) * C::TILE) + (i % 4) * 32, 16, 1024), id_s, i > 0);
          tc_commit(smem_u32(&s_full[kk & 1]));
        }
        __syncwarp();
        return true;
      };
      for (int seg = 0; ok && walk.next(a, s); ++seg) {
        if (!(ok = mbar_wait_warp(smem_u32(q_full), seg & 1, abort_flag))) break;
        tc_after();
        if (!(ok = issue_s(k))) break;
        for (int t = s.t0; t < s.t1; ++t, ++k) {
          if (t + 1 < s.t1 && !(ok = issue_s(k + 1))) break;
          if (!(ok = mbar_wait_warp(smem_u32(&p_full[k & 1]), (k >> 1) & 1, abort_flag))) break;
          tc_after();
          const int st = k % ST;
          const uint8_t* vt = ring + st * C::STAGE + C::CT * C::TILE;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < KT / 16; ++i)
              // V: rows of keys, 64 values of N per 128-byte row; 8-key groups 1024 B apart, the next 64 of N one
              // column tile further
              tc_mma_ts(tmem + 2 * KT, tmem + (k & 1) * KT + i * 8, tc_desc(smem_u32(vt) + i * 16 * 128, C::TILE, 1024),
                        id_o, t > s.t0 || i > 0);
            tc_commit(smem_u32(&o_full[k & 1]));
            tc_commit(smem_u32(&empty[st]));
          }
          __syncwarp();
        }
      }
    } else {
      // ------------------------------------------------------------------ rows
      const int t_row = threadIdx.x - 128;
      const uint32_t tl = tmem + ((uint32_t)((warp - 4) * 32) << 16);  // the warp's TMEM lanes
      const int G = a.H / a.Hk;
      bool ok = true;  // once a wait ran out: no more waits or TMEM, but every barrier of the rows is still met
      while (walk.next(a, s)) {
        const Req& q = s.q;
        const int rho = s.blk * BM + t_row;
        const bool valid = rho < q.n * G;
        const int node = valid ? rho / G : -1, head = s.hk * G + (valid ? rho - node * G : 0);
        const int64_t row = q.row0 + (valid ? node : 0);
        const bool active = __any_sync(0xffffffffu, valid);
        if (ok) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row * a.q_stride +
                                                            (int64_t)head * HD);
#pragma unroll
          for (int c = 0; c < HD / 8; ++c) {
            const uint4 v = valid ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(sQ + (c / 8) * (BM * 128) + t_row * 128 + (((c % 8) ^ (t_row & 7)) << 4)) = v;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(q_full));
        }
        float m = -INFINITY, l = 0.f;
        for (int t = s.t0; t < s.t1; ++t, ++k) {
          const int buf = k & 1, st = k % ST;
          const bool nodes_here = (t + 1) * KT > q.ctx;
          ok = ok && mbar_wait_warp(smem_u32(&s_full[buf]), (k >> 1) & 1, abort_flag) &&
               mbar_wait_warp(smem_u32(&full[st]), (k / ST) & 1, abort_flag);
          if (!ok) {
            if (nodes_here && rows_any(false)) asm volatile("bar.sync 1, 128;" ::: "memory");
            continue;
          }
          tc_after();
          const uint32_t landed = info[st];
          const bool mask = landed != all_boxes || nodes_here;
          float sv[KT];
          if (active) {
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) tc_ld32(tl + buf * KT + 32 * c, sv + 32 * c);
            tc_wait_ld();
            if (mask) {
#pragma unroll
              for (int c = 0; c < KT / 32; ++c) {
                const uint32_t v = valid ? row_sees(a, q, row, node, t * KT + 32 * c, landed, PR, 32 * c) : 0u;
#pragma unroll
                for (int i = 0; i < 32; ++i) sv[32 * c + i] = v >> i & 1u ? sv[32 * c + i] : -INFINITY;
              }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < KT; i += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], fmaxf(sv[i + e], sv[i + 4 + e]));
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            // the row's reference: the first tile's maximum, and a new one only past 2^8 times it
            const bool move = mt > (t == s.t0 ? m : m + 8.f);
            const float mn = move ? mt : m, z = mn == -INFINITY ? 0.f : mn;
            if (t > s.t0 && __any_sync(0xffffffffu, move)) {
              const float corr = move ? ex2(m - z) : 1.f;
              ok = mbar_wait_warp(smem_u32(&o_full[buf ^ 1]), ((k - 1) >> 1) & 1, abort_flag);
              tc_after();
#pragma unroll
              for (int c = 0; c < HD / 32; ++c) {
                float o[32];
                tc_ld32(tl + 2 * KT + 32 * c, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= corr;
                tc_st32(tl + 2 * KT + 32 * c, reinterpret_cast<const uint32_t*>(o));
              }
              l *= corr;
            }
            m = mn;
            F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
            const F2 sc = f2(a.scale_log2, a.scale_log2), mz = f2(-z, -z);
            uint32_t pk[KT / 2];
#pragma unroll
            for (int i = 0; i < KT; i += 2) {
              float x, y;
              f2_out(fma2(f2(sv[i], sv[i + 1]), sc, mz), x, y);
              x = ex2(x);
              y = ex2(y);
              sv[i] = x;
              sv[i + 1] = y;
              sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], f2(x, y));
              // one rounding of each probability to the values' type (the matrix instruction takes one type)
              pk[i / 2] = pack2<BF>(x, y);
            }
            float s0, s1;
            f2_out(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            tc_st32(tl + buf * KT, pk);
            tc_st32(tl + buf * KT + 32, pk + 32);
            tc_wait_st();
          }
          bool odd = false;
          if (mask) {
            // Values of positions that nobody sees may be anything, and 0 * NaN is not 0.  Thread y looks after
            // position y of the tile.
            const int pos = t * KT + t_row;
            uint8_t* vt = ring + st * C::STAGE + C::CT * C::TILE;
            bool mine = false;
            auto chunk = [&](int y, int c) {
              return reinterpret_cast<uint4*>(vt + (c / 8) * C::TILE + y * 128 + (((c % 8) ^ (y & 7)) << 4));
            };
            constexpr uint32_t X = BF ? 0x7f80u : 0x7c00u;
            if (pos >= q.len || !(landed >> (t_row / PR) & 1u)) {
#pragma unroll
              for (int c = 0; c < HD / 8; ++c) *chunk(t_row, c) = make_uint4(0, 0, 0, 0);
            } else if (pos >= q.ctx && (q.n > 1 || a.masks)) {
#pragma unroll
              for (int c = 0; c < HD / 8; ++c) {
                const uint4 w = *chunk(t_row, c);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) mine |= (u[e] & X) == X || (u[e] >> 16 & X) == X;
              }
            }
            if (nodes_here) {  // have all rows agree on whether a value is not finite
              odd = rows_any(mine);
              if (odd) {
                // the values that are not finite enter by hand, where the row sees the position, and as 0 in P V
                float add[HD], pl[KT];
#pragma unroll
                for (int d = 0; d < HD; ++d) add[d] = 0.f;
#pragma unroll
                for (int i = 0; i < KT; ++i) pl[i] = active ? sv[i] : 0.f;
#pragma unroll 1
                for (int y = 0; y < KT; ++y)
#pragma unroll 1
                  for (int c = 0; c < HD / 8; ++c) {
                    const uint4 w = *chunk(y, c);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                      const uint32_t b = u[e >> 1] >> (16 * (e & 1)) & 0xffffu;
                      const float2 v = unpack2<BF>(b);
                      if ((b & X) == X && pl[y] != 0.f) add[c * 8 + e] += pl[y] * v.x;
                    }
                  }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (mine)
#pragma unroll 1
                  for (int c = 0; c < HD / 8; ++c) {
                    uint32_t* u = reinterpret_cast<uint32_t*>(chunk(t_row, c));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      if ((u[e] & X) == X) u[e] &= 0xffff0000u;
                      if ((u[e] >> 16 & X) == X) u[e] &= 0xffffu;
                    }
                  }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
                ok = ok && mbar_wait_warp(smem_u32(&o_full[buf]), (k >> 1) & 1, abort_flag);
                tc_after();
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                  float o[32];
                  tc_ld32(tl + 2 * KT + 32 * c, o);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] += add[32 * c + i];
                  tc_st32(tl + 2 * KT + 32 * c, reinterpret_cast<const uint32_t*>(o));
                }
                tc_wait_st();
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // zeros before P V reads them
          }
          if (!odd) {
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
          }
        }
        // ------------------------------------------------ the row block's end
        ok = ok && mbar_wait_warp(smem_u32(&o_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort_flag);
        if (!ok) continue;
        tc_after();
        const bool whole = s.t0 == 0 && s.t1 == q.tiles;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        float* ws = reinterpret_cast<float*>(a.ws + gridDim.x * sizeof(Start)) +
                    ((int64_t)blockIdx.x * 2 + (walk.u - (s.t1 - s.t0) == u_first && s.t0 > 0 ? 0 : 1)) * BM * (HD + 2) +
                    t_row * (HD + 2);
        if (active) {
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            float o[32];
            tc_ld32(tl + 2 * KT + 32 * c, o);
            tc_wait_ld();
            if (!valid) continue;
            if (whole) {
              const int64_t at = row * a.out_stride + (int64_t)head * HD + 32 * c;
              if (a.out_f32) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + i) =
                      make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
              } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + i) =
                      make_uint4(pack2<BF>(o[i] * inv, o[i + 1] * inv), pack2<BF>(o[i + 2] * inv, o[i + 3] * inv),
                                 pack2<BF>(o[i + 4] * inv, o[i + 5] * inv), pack2<BF>(o[i + 6] * inv, o[i + 7] * inv));
              }
              if (a.out16)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  act16_put(a.out16, row, a.H * HD, head * HD + 32 * c + i, o[i] * inv, a.split16);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                *reinterpret_cast<float2*>(ws + 2 + 32 * c + i) = make_float2(o[i], o[i + 1]);
            }
          }
          if (valid && whole && a.lse) a.lse[row * a.H + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          if (valid && !whole) *reinterpret_cast<float2*>(ws) = make_float2(m, l);
        }
        tc_before();
      }
    }
  }
  tc_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_s && a.status) atomicOr(a.status, TL_TIMED_OUT);
  if (warp == 2) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::TMEM_COLS)
                 : "memory");
  }
}

}  // namespace tree
}  // namespace tl
