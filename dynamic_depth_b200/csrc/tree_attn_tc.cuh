// Tree attention on the 5th-generation tensor cores (tcgen05 + TMEM), for row
// blocks of more rows than the warp-level matrix instructions keep up with.
// Same units, ranges, pieces and page handling as tree_attn_kernel.
//
// A row block is 128 query rows (one TMEM lane and one thread each), a tile 64
// key positions:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, into one of two
//                  or three TMEM buffers
//   P = exp2(S-m)  one thread a row; 16-bit P replaces S in its TMEM columns
//   O += P V       tcgen05.mma with P as the TMEM operand A and V (rows of
//                  keys) as the N-major operand B, accumulating in TMEM
// The reference m of a row (kLift below a maximum) moves only when a tile's
// maximum passes the last one by more than 2^8 (P then stays below 2^15 in fp16
// and 2^8 in bf16, and sums are fp32), so O is rescaled in TMEM a few times per
// row block instead of once per tile (a published technique for this chip).
//
// Two CTAs an SM, each with half of shared memory and TMEM: one streams while
// the other is between row blocks (the next queries, the output: about a tenth
// of a CTA's time in the case below).
// 64 requests x 32 nodes x 4 heads on 4,000 positions of width 128 take 229 us
// (4.8 TB/s, 590 TFLOP/s); one CTA an SM with 128-position tiles took 252, two
// threads a row with three S buffers 259, two groups of rows on alternate tiles
// 374.
//
// Warp 0 loads K, warp 2 loads V (each its own ring), warp 1 issues Q K^T, warp
// 3 issues P V, so no one of them waits for another's turn; warps 4-7: rows.
// A plain tile takes a CTA 1,520 + 1,550 cycles (wait + work) with two CTAs an SM,
// so 1,535 a tile and SM; its 32 KB are about 1,370 of an SM's share of HBM, its
// 12 matrix instructions of about 110 cycles each (whatever their size up to
// N = 128) 1,350, its exponentials 512.  The steady loop is within 12 % of memory.
// Of the 87 us of 16 requests x 32 nodes x 4 heads on up to 8,190 positions it is
// about 50; the rest is the starts of row blocks (6,270 cycles each: queries, first
// tiles), their ends (3,640), tiles with nodes (5,900), the range search, and
// 13 us of joining.
#pragma once

#include "ptx.cuh"

namespace tl {
namespace tree {

template <int HD>
struct TcCfg {
  static constexpr int KT = 64, BM = 128;
  static constexpr int CT = HD / 64;               // 64-wide column tiles
  static constexpr int TILE = KT * 128;            // bytes of one: [64 positions x 64] 16 bit
  static constexpr int STAGE = CT * TILE;          // K or V of a tile
  static constexpr int STAGES = HD == 128 ? 2 : 4; // of K, and of V
  static constexpr int Q_BYTES = BM * HD * 2;
  static constexpr int SB = HD == 128 ? 2 : 3;     // S buffers
  static constexpr int TMEM_COLS = 256;            // S / P two or three times 64, O HD
  static constexpr int THREADS = 256;
  static constexpr int SMEM = 1024 + Q_BYTES + 2 * STAGES * STAGE + 512;
  // two CTAs share an SM (and its 512 columns of TMEM), never three
  static_assert(SMEM <= 113 * 1024 && SMEM > 76 * 1024, "two CTAs per SM");
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

// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Barrier 1: the 128 row threads.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Whether any row thread says so (all of them call it).
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

// Tiles whose boxes are remembered: K runs at most STAGES tiles ahead of S, and S at most three ahead of the rows.
constexpr int kInfo = 16;

// A producer warp: K or V of the tiles of the CTA's range into its ring, a box
// per page (or part of one).
template <class C>
__device__ __forceinline__ void produce_half(const TreeAttnArgs& a, const CUtensorMap& kvmap, Walk<C::KT, C::BM> walk,
                                             bool values, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                             volatile uint32_t* info, volatile int32_t* abort_flag) {
  constexpr int KT = C::KT;
  const int lane = threadIdx.x & 31;
  const int P = 1 << a.page_shift, PR = P < KT ? P : KT, boxes = KT / PR;
  const Seg& s = walk.s;
  int k = 0;
  bool ok = true;
  while (ok && walk.next(a)) {
    const int32_t* table = a.table + (int64_t)s.r * a.max_pages;
    const int64_t head = (int64_t)s.hk + (values ? a.Hk : 0);
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
        if (!values) info[k % kInfo] = in;
        mbar_expect_tx(bar, __popc(in) * C::CT * PR * 128);
      }
      __syncwarp();
      if (good) {
        const int64_t y = (((int64_t)page * 2 * a.Hk + head) << a.page_shift) + (pos & (P - 1));
        const uint32_t dst = smem_u32(ring + st * C::STAGE) + lane * PR * 128;
#pragma unroll
        for (int ct = 0; ct < C::CT; ++ct) tma_load_2d(dst + ct * C::TILE, &kvmap, ct * 64, (int)y, bar);
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

// Sums p * v of the values of 64 positions that are not finite, over the positions with a probability.
template <int HD, bool BF>
__device__ __noinline__ void add_odd(const float* p, const uint8_t* vt, float* add) {
  constexpr uint32_t X = BF ? 0x7f80u : 0x7c00u;
  for (int d = 0; d < HD; ++d) add[d] = 0.f;
  for (int y = 0; y < 64; ++y) {
    if (p[y] == 0.f) continue;
    for (int d = 0; d < HD; ++d) {
      const int r = y, c = d / 8;
      const uint32_t b = *reinterpret_cast<const uint16_t*>(vt + (c / 8) * TcCfg<HD>::TILE + r * 128 +
                                                            (((c % 8) ^ (r & 7)) << 4) + (d % 8) * 2);
      if ((b & X) == X) add[d] += p[y] * unpack2<BF>(b).x;
    }
  }
}
// Adds HD values to the thread's row of O.
template <int HD>
__device__ __noinline__ void add_to_o(uint32_t to, const float* add) {
  for (int c = 0; c < HD; c += 32) {
    float o[32];
    tc_ld32(to + c, o);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] += add[c + i];
    tc_st32(to + c, reinterpret_cast<const uint32_t*>(o));
  }
  tc_wait_st();
}

// Scales the thread's row of O.
template <int HD>
__device__ __noinline__ void scale_o(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < HD; c += 32) {
    float o[32];
    tc_ld32(to + c, o);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= f;
    tc_st32(to + c, reinterpret_cast<const uint32_t*>(o));
  }
  tc_wait_st();
}

template <int HD, bool BF>
__global__ void __launch_bounds__(TcCfg<HD>::THREADS, 2)
tree_attn_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const TreeAttnArgs a) {
  using C = TcCfg<HD>;
  constexpr int KT = C::KT, BM = C::BM, ST = C::STAGES, SB = C::SB;
  extern __shared__ __align__(1024) uint8_t smem_tt[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_tt) + 1023) & ~uintptr_t(1023));
  uint8_t* ring_k = sQ + C::Q_BYTES;
  uint8_t* ring_v = ring_k + ST * C::STAGE;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(ring_v + ST * C::STAGE);
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* s_full = v_empty + ST;  // [SB] S of a tile in TMEM
  uint64_t* p_full = s_full + SB;   // [SB] P of a tile in TMEM, V clean
  uint64_t* o_full = p_full + SB;   // [SB] P V of a tile added
  uint64_t* q_full = o_full + SB;   // Q of a row block in shared memory
  Range& range_s = *reinterpret_cast<Range*>(q_full + 1);
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(&range_s + 1);  // [kInfo] boxes in the pool
  uint32_t& tmem_s = *const_cast<uint32_t*>(info + kInfo);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(&tmem_s + 1);
  long long* wsum = reinterpret_cast<long long*>(sQ);  // before any Q
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int b = 0; b < SB; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&p_full[b]), 4);
      mbar_init(smem_u32(&o_full[b]), 1);
    }
    mbar_init(smem_u32(q_full), 4);
    *abort_flag = 0;
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
  find_range<KT, BM>(a, &range_s, wsum);
  __syncthreads();
  const uint32_t tmem = tmem_s;
  Walk<KT, BM> walk(range_s);  // nothing where u0 == u1
  const int64_t u_first = walk.u;
  const Seg& s = walk.s;
  int k = 0;  // tiles of this CTA so far
  if (warp < 4) {
    if (warp == 0 || warp == 2) {
      produce_half<C>(a, kvmap, walk, warp == 2, warp == 0 ? ring_k : ring_v, warp == 0 ? k_full : v_full,
                      warp == 0 ? k_empty : v_empty, info, abort_flag);
    } else if (warp == 1) {
      // ------------------------------------------------------------- S = Q K^T
      constexpr uint32_t idesc = tc_idesc(BF, KT, 0);
      bool ok = true;
      for (int seg = 0; ok && walk.next(a); ++seg) {
        if (!(ok = mbar_wait_warp(smem_u32(q_full), seg & 1, abort_flag))) break;
        for (int t = s.t0; t < s.t1; ++t, ++k) {
          const int st = k % ST, buf = k % SB;
          // P of tile k - SB has been read from this buffer
          ok = (k < SB || mbar_wait_warp(smem_u32(&o_full[buf]), (k / SB - 1) & 1, abort_flag)) &&
               mbar_wait_warp(smem_u32(&k_full[st]), (k / ST) & 1, abort_flag);
          if (!ok) break;
          tc_after();
          const uint8_t* kt = ring_k + st * C::STAGE;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < HD / 16; ++i)
              tc_mma_ss(tmem + buf * KT, tc_desc(smem_u32(sQ + (i / 4) * (BM * 128)) + (i % 4) * 32, 16, 1024),
                        tc_desc(smem_u32(kt + (i / 4) * C::TILE) + (i % 4) * 32, 16, 1024), idesc, i > 0);
            tc_commit(smem_u32(&s_full[buf]));
            tc_commit(smem_u32(&k_empty[st]));
          }
          __syncwarp();
        }
      }
    } else {
      // --------------------------------------------------------------- O += P V
      constexpr uint32_t idesc = tc_idesc(BF, HD, 1);
      bool ok = true;
      while (ok && walk.next(a)) {
        for (int t = s.t0; t < s.t1; ++t, ++k) {
          const int st = k % ST, buf = k % SB;
          ok = mbar_wait_warp(smem_u32(&v_full[st]), (k / ST) & 1, abort_flag) &&
               mbar_wait_warp(smem_u32(&p_full[buf]), (k / SB) & 1, abort_flag);
          if (!ok) break;
          tc_after();
          const uint8_t* vt = ring_v + st * C::STAGE;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < KT / 16; ++i)
              // V: rows of keys, 64 values of N per 128-byte row; 8-key groups 1024 B apart, the next 64 of N one
              // column tile further
              tc_mma_ts(tmem + SB * KT, tmem + buf * KT + i * 8,
                        tc_desc(smem_u32(vt) + i * 16 * 128, C::TILE, 1024), idesc, t > s.t0 || i > 0);
            tc_commit(smem_u32(&o_full[buf]));
            tc_commit(smem_u32(&v_empty[st]));
          }
          __syncwarp();
        }
      }
    }
  } else {
    {
      // ------------------------------------------------------------------ rows
      const int t_row = threadIdx.x - 128;
      const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // the warp's TMEM lanes
      const uint32_t to = tl + SB * KT;
      const int G = a.H / a.Hk;
      const int PR = min(1 << a.page_shift, KT), pshift = 31 - __clz(PR);
      const uint32_t all_boxes = (1u << (KT >> pshift)) - 1u;
      bool ok = true;  // once a wait ran out: no more waits or TMEM, but every barrier of the rows is still met
      while (walk.next(a)) {
        const int ctx = s.q.ctx, len = s.q.len;
        const int rho = s.blk * BM + t_row;
        const bool valid = rho < s.q.n * G;
        const int node = valid ? rho / G : -1, head = s.hk * G + (valid ? rho - node * G : 0);
        const int64_t row = s.q.row0 + (valid ? node : 0);
        const bool active = __any_sync(0xffffffffu, valid);
        if (ok) {
          // the warp's 32 rows, neighbouring lanes at neighbouring 16 bytes, all on their way at once (a thread that
          // loads its own row spreads each load over 32 lines; 16 lanes x 32 nodes: 88.6 us, 94.5 so, with the walk's
          // divisions)
          constexpr int CH = HD / 8, RI = 32 / CH;  // 16-byte chunks of a row, rows of an access
          const int64_t from = valid ? row * a.q_stride + (int64_t)head * HD : -1;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int y = i * RI + lane / CH, c = lane % CH;
            const int64_t o = __shfl_sync(0xffffffffu, from, y);
            cp_async16(smem_u32(sQ) + (c / 8) * (BM * 128) + ((warp & 3) * 32 + y) * 128 + (((c % 8) ^ (y & 7)) << 4),
                       static_cast<const uint16_t*>(a.q) + (o < 0 ? 0 : o + c * 8), o >= 0);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(q_full));
        }
        float m = -INFINITY, l = 0.f;
        for (int t = s.t0; t < s.t1; ++t, ++k) {
          const int st = k % ST, buf = k % SB;
          const bool nodes_here = (t + 1) * KT > ctx;
          uint32_t see[2] = {0u, 0u};
          if (nodes_here && valid) {  // on their way while the product runs
            see[0] = row_sees(a, s.q, row, node, t * KT);
            see[1] = row_sees(a, s.q, row, node, t * KT + 32);
          }
          ok = ok && mbar_wait_warp(smem_u32(&s_full[buf]), (k / SB) & 1, abort_flag);
          const uint32_t landed = ok ? info[k % kInfo] : 0u;
          const bool mask = landed != all_boxes || nodes_here;
          if (ok && mask) ok = mbar_wait_warp(smem_u32(&v_full[st]), (k / ST) & 1, abort_flag);
          if (!ok) {
            if (nodes_here && rows_any(false)) rows_sync();
            continue;
          }
          tc_after();
          const uint32_t ts = tl + buf * KT;
          uint8_t* vt = ring_v + st * C::STAGE;
          float sv[KT];
          if (active) {
            tc_ld32(ts, sv);
            tc_ld32(ts + 32, sv + 32);
            tc_wait_ld();
            if (mask) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t lo = landed >> (32 * c >> pshift) & 1u, hi = landed >> (32 * c + 16 >> pshift) & 1u;
                const uint32_t v = (nodes_here ? see[c] : 0xffffffffu) & ((lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u));
#pragma unroll
                for (int i = 0; i < 32; ++i) sv[32 * c + i] = v >> i & 1u ? sv[32 * c + i] : -INFINITY;
              }
            }
            float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
            for (int i = 4; i < KT; i += 4)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], sv[i + e]);
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2 - kLift<BF>;
            // the row's reference, from the first tile's maximum, and a new one only past 2^8 times it
            const bool move = mt > (t == s.t0 ? m : m + 8.f);
            const float mn = move ? mt : m, z = mn == -INFINITY ? 0.f : mn;
            if (t > s.t0 && __any_sync(0xffffffffu, move)) {
              const float corr = move ? ex2(m - z) : 1.f;
              ok = mbar_wait_warp(smem_u32(&o_full[(k - 1) % SB]), ((k - 1) / SB) & 1, abort_flag);
              tc_after();
              scale_o<HD>(to, corr);
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
              sv[i] = ex2(x);
              sv[i + 1] = ex2(y);
              sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], f2(sv[i], sv[i + 1]));
              // one rounding of each probability to the values' type (the matrix instruction takes one type)
              pk[i / 2] = pack2<BF>(sv[i], sv[i + 1]);
            }
            tc_st32(ts, pk);
            float s0, s1;
            f2_out(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            tc_wait_st();
          }
          bool odd = false;
          if (mask) {
            // Values of positions that nobody sees may be anything, and 0 * NaN is not 0.  Two threads look after a
            // position of the tile.
            constexpr uint32_t X = BF ? 0x7f80u : 0x7c00u;
            const int y = t_row & 63, pos = t * KT + y, c0 = (t_row >> 6) * (HD / 16);
            auto chunk = [&](int c) {  // 8 of its values
              return reinterpret_cast<uint4*>(vt + (c / 8) * C::TILE + y * 128 + (((c % 8) ^ (y & 7)) << 4));
            };
            bool mine = false;
            if (pos >= len || !(landed >> (y >> pshift) & 1u)) {
#pragma unroll
              for (int c = 0; c < HD / 16; ++c) *chunk(c0 + c) = make_uint4(0, 0, 0, 0);
            } else if (pos >= ctx && (len > ctx + 1 || a.masks)) {
#pragma unroll
              for (int c = 0; c < HD / 16; ++c) {
                const uint4 w = *chunk(c0 + c);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) mine |= (u[e] & X) == X || (u[e] >> 16 & X) == X;
              }
            }
            if (nodes_here) odd = rows_any(mine);
            if (odd) {
              // the values that are not finite enter by hand, where the row sees the position, and as 0 in P V
              float add[HD], pl[KT];
#pragma unroll
              for (int i = 0; i < KT; ++i) pl[i] = active ? sv[i] : 0.f;
              add_odd<HD, BF>(pl, vt, add);
              rows_sync();
              if (mine) {
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                  uint32_t* u = reinterpret_cast<uint32_t*>(chunk(c0 + c));
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if ((u[e] & X) == X) u[e] &= 0xffff0000u;
                    if ((u[e] >> 16 & X) == X) u[e] &= 0xffffu;
                  }
                }
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              tc_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
              ok = ok && mbar_wait_warp(smem_u32(&o_full[buf]), (k / SB) & 1, abort_flag);
              tc_after();
              add_to_o<HD>(to, add);
            }
          }
          if (!odd) {
            if (mask) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // zeros before P V reads them
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
          }
        }
        // ---------------------------------------------- the row block's end
        ok = ok && mbar_wait_warp(smem_u32(&o_full[(k - 1) % SB]), ((k - 1) / SB) & 1, abort_flag);
        tc_after();
        if (active && ok) {
          const bool whole = s.t0 == 0 && s.t1 == s.q.tiles;
          const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
          auto* w = piece_of<HD, BM>(a, gridDim.x, blockIdx.x, walk.u - (s.t1 - s.t0) == u_first && s.t0 > 0 ? 0 : 1);
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {
            float o[32];
            tc_ld32(to + c0, o);
            tc_wait_ld();
            if (!valid) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= inv;
            if (whole) {
              const int64_t at = row * a.out_stride + (int64_t)head * HD + c0;
              if (a.out_f32) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + i) =
                      make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + i) =
                      make_uint4(pack2<BF>(o[i], o[i + 1]), pack2<BF>(o[i + 2], o[i + 3]),
                                 pack2<BF>(o[i + 4], o[i + 5]), pack2<BF>(o[i + 6], o[i + 7]));
              }
              if (a.out16)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  act16_put(a.out16, row, a.H * HD, head * HD + c0 + i, o[i], a.split16);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                w->o[(c0 + i) / 4][t_row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
          if (valid) {
            if (whole && a.lse) a.lse[row * a.H + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            if (!whole) w->ml[t_row] = make_float2(m, l);
          }
        }
        tc_before();
      }
    }
  }
  if (threadIdx.x == 0) note_cut(a, range_s);
  tc_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag && a.status) atomicOr(a.status, TL_TIMED_OUT);
  if (warp == 2) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::TMEM_COLS)
                 : "memory");
  }
}

}  // namespace tree
}  // namespace tl
