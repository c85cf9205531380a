// Log probabilities, rank, entropy and best alternatives of rows of logits.
//
//   lse = m + ln S,  S = sum exp(x - m),  T = sum (x - m) exp(x - m)
//   logprob_t = (x_t - m) - ln S,  entropy = ln S - T / S
//
// One pass over the row.  A row is cut into chunks of 256 consecutive
// elements; a warp takes a chunk at a time, 8 elements a lane, and keeps a
// running maximum (uniform in the warp) with S and T rescaled when it rises.
// The chunk maxima that this needs anyway are kept in shared memory.  A bound
// on the n-th largest element comes from the threads' own maxima; only chunks
// whose maxima reach it are read again (they are in L2), and the elements that
// reach it, some tens, are ordered.  Where masks or equal logits let too many
// through, the exact form: the n first elements in the order (value
// descending, id ascending) lie in the n chunks whose maxima come first in
// (maximum descending, chunk ascending), since each chunk before an element's
// own holds an element before it.
//
// Few rows: a cluster of up to 8 CTAs shares a row and its first CTA merges the
// partial sums and lists over distributed shared memory, with no scratch in
// global memory.  Chunks and candidates enter their lists in shared memory in
// any order (atomic counters) and are then put into a total order, and the sums
// are joined in a fixed one, so results do not depend on timing.
//
// S and T are held and joined in fp32: a lane adds vocab / (256 * CTAs) terms or
// so (vocab / 32, 512 at most, where a warp takes a row), then lanes, warps and
// CTAs meet in trees, and the logarithm is fp32.  That leaves a relative error
// of a few 2^-24 for ordinary rows and vocab / 256 times 2^-24 at worst, which
// is a lane's own sum: joining the lanes in fp64 would not lower it.
// Bound by issue as much as by memory: 1000 rows of 131,072 bf16 logits with
// n = 20 take 60 us (4.4 TB/s), without the best 20 53 us (5.0 TB/s); the
// difference is the end of each row.
#include <cooperative_groups.h>

#include "common.cuh"
#include "host_util.h"
#include "packed.cuh"

namespace tl {
namespace logprobs {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 256;      // elements a warp reads at a time: 8 a lane
constexpr int kMaxTop = 64;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kCand = 2048;      // candidates ordered in shared memory; more take the extraction loop
constexpr int kList = 256;       // chunks that reach the bound; more take the exact search
constexpr int kWarpCand = 256;   // candidates of a row that one warp handles
constexpr int kWarpTop = 56;     // most best tokens of such a row (see launch)
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const void* x;
  int64_t rows, stride;
  int32_t V, n_top;
  const int32_t* targets;
  float* logprob;
  int32_t* rank;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_lp;
  int32_t n_chunks;  // chunks per CTA, at most
};

// Total order of values as unsigned integers: -inf lowest, +inf high, NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t sort_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <class T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two packed elements as floats, and the operations on packed words.
template <class T>
struct Word {};
template <>
struct Word<float> {
  static constexpr uint32_t kNegInf = 0xff800000u;
  static constexpr float kPlain = 1e30f;  // below this, x - m is finite for finite x, and lowest - m an exponential of 0
};
template <>
struct Word<__half> {
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static constexpr float kPlain = 3e4f;
  typedef __half2 V2;
  static __device__ __forceinline__ V2 lowest() { return __halves2half2(__ushort_as_half(0xfbff), __ushort_as_half(0xfbff)); }
  static __device__ __forceinline__ V2 both(float x) { return __float2half2_rn(x); }
  static __device__ __forceinline__ float2 two(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static constexpr float kPlain = 1e30f;
  typedef __nv_bfloat162 V2;
  static __device__ __forceinline__ V2 lowest() {
    return __halves2bfloat162(__ushort_as_bfloat16(0xff7f), __ushort_as_bfloat16(0xff7f));
  }
  static __device__ __forceinline__ V2 both(float x) { return __float2bfloat162_rn(x); }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// A lane's 8 elements of a chunk, as they lie in memory.
template <class T>
struct Raw {
  static constexpr int W = 8 * sizeof(T) / 16;
  uint4 w[W];
};

// Positions are counted from the 16-byte boundary at or before the row (`lead`
// elements before it), so whole words are aligned; a word that holds the row's
// first or last elements is read by element.  Elements outside the row are
// -inf.  Lane l holds, of each word w of its 8 elements, positions
// base + w * 32 * E + l * E + (0 .. E-1).
template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* row, int lead, int V, int pos0, int lane) {
  constexpr int E = 16 / sizeof(T);  // elements of a word
  Raw<T> r;
#pragma unroll
  for (int w = 0; w < Raw<T>::W; ++w) {
    const int p = pos0 + (w * 32 + lane) * E - lead;  // element index of the word's first
    if (p >= 0 && p + E <= V) {
      r.w[w] = __ldg(reinterpret_cast<const uint4*>(row + p));
    } else {
      r.w[w] = make_uint4(Word<T>::kNegInf, Word<T>::kNegInf, Word<T>::kNegInf, Word<T>::kNegInf);
      T* e = reinterpret_cast<T*>(&r.w[w]);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (p + i >= 0 && p + i < V) e[i] = row[p + i];
    }
  }
  return r;
}
// U chunks from chunk c on: one test for all of them, except at the row's ends.
template <class T, int U>
__device__ __forceinline__ void load_group(Raw<T> (&r)[U], const T* row, int lead, int V, int c, int lane) {
  const int first = c * kChunk - lead;
  if (first >= 0 && first + U * kChunk <= V) {
    const uint4* p = reinterpret_cast<const uint4*>(row + first) + lane;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int w = 0; w < Raw<T>::W; ++w) r[u].w[w] = __ldg(p + (u * Raw<T>::W + w) * 32);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_raw<T>(row, lead, V, (c + u) * kChunk, lane);
  }
}
template <class T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&f)[8]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r.w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(u[i]);
    } else {
      const float2 v = Word<T>::two(u[i >> 1]);
      f[i] = i & 1 ? v.y : v.x;
    }
  }
}
// -inf to the lowest number, whose exponential is 0 and 0 times which is not NaN.
template <class T>
__device__ __forceinline__ void raise_lowest(Raw<T>& r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r.w);
#pragma unroll
  for (int i = 0; i < 4 * Raw<T>::W; ++i) {
    if constexpr (sizeof(T) == 4) {
      u[i] = __float_as_uint(fmaxf(__uint_as_float(u[i]), -3.4e38f));
    } else {
      const auto v = __hmax2(*reinterpret_cast<const typename Word<T>::V2*>(&u[i]), Word<T>::lowest());
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}
// How many of the lane's elements of U chunks are above x (EQ: at x or above).
template <class T, int U, bool EQ>
__device__ __forceinline__ int count_group(const Raw<T> (&r)[U], float x) {
  if constexpr (sizeof(T) == 4) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(r[u].w);
#pragma unroll
      for (int i = 0; i < 8; ++i) n += EQ ? __uint_as_float(w[i]) >= x : __uint_as_float(w[i]) > x;
    }
    return n;
  } else {
    typedef typename Word<T>::V2 V2;
    const V2 xx = Word<T>::both(x);
    V2 s = Word<T>::both(0.f);  // counts up to 16, exact
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const V2* v = reinterpret_cast<const V2*>(r[u].w);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = __hadd2(s, EQ ? __hge2(v[i], xx) : __hgt2(v[i], xx));
    }
    const float2 f = Word<T>::two(*reinterpret_cast<const uint32_t*>(&s));
    return (int)(f.x + f.y);
  }
}
// Largest of the 8, NaN if one is.
template <class T>
__device__ __forceinline__ float max8(const Raw<T>& r) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r.w);
  if constexpr (sizeof(T) == 4) {
    float m = __uint_as_float(u[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, __uint_as_float(u[i]));
    return m;
  } else {
    const float2 v = Word<T>::two(Word<T>::max2(Word<T>::max2(u[0], u[1]), Word<T>::max2(u[2], u[3])));
    return max_nan(v.x, v.y);
  }
}
template <class T>
__device__ __forceinline__ void load8(const T* row, int lead, int V, int pos0, int lane, float (&f)[8]) {
  unpack<T>(load_raw<T>(row, lead, V, pos0, lane), f);
}
template <class T>
__device__ __forceinline__ int elem_index(int pos0, int lead, int lane, int i) {
  constexpr int E = 16 / sizeof(T);
  return pos0 + ((i / E) * 32 + lane) * E + i % E - lead;
}

// Largest over the warp, NaN if one is.
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A part of a row: maximum, sums relative to it, tokens before the target.
struct Part {
  float m, S, T;
  int32_t before;
  int32_t nan;
};

// The lanes' parts, joined.
__device__ __forceinline__ Part merge_parts(const Part& q) {
  Part p;
  p.nan = __any_sync(0xffffffffu, q.nan);
  p.m = warp_max(q.m);
  const float d = p.m - q.m, k = q.m > -INFINITY ? expf(-d) : 0.f;
  p.S = warp_sum(k * q.S);
  p.T = warp_sum(k > 0.f ? k * (q.T - d * q.S) : 0.f);  // (d * S may be infinite where k is 0)
  p.before = __reduce_add_sync(0xffffffffu, q.before);
  return p;
}

// One pass of a warp over chunks cb, cb + step, ... below c1 of a row, U at a
// time (64 bytes a lane) with the next U on their way meanwhile; lead_fn(chunk,
// maximum) hears of every chunk.  mine: the lane's largest element of the even
// and of the odd chunks of its groups.
template <class T, int U, class F>
__device__ __forceinline__ Part stream_chunks(const T* row, int lead, int V, int t, float xt, bool has_t, int cb, int c1,
                                              int step, int lane, float (&mine)[2], F lead_fn) {
  float m = -INFINITY;
  F2 S2 = f2(0.f, 0.f), T2 = f2(0.f, 0.f);
  int before = 0;
  bool nan = false;
  mine[0] = mine[1] = -INFINITY;
  const F2 log2e = f2(kLog2e, kLog2e);
  Raw<T> next[U];
  load_group<T, U>(next, row, lead, V, cb, lane);
  for (; cb < c1; cb += step) {
    Raw<T> cur[U];
    float cm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = next[u];
    if (cb + step < c1) load_group<T, U>(next, row, lead, V, cb + step, lane);
    float top_m = -INFINITY;  // NaN if one is
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float lm = max8<T>(cur[u]);
      mine[u & 1] = max_nan(mine[u & 1], lm);
      cm[u] = warp_max_nan(lm);
      lead_fn(cb + u, cm[u]);
      top_m = u == 0 ? cm[0] : max_nan(top_m, cm[u]);
    }
    if (!(top_m <= m)) {
      nan |= top_m != top_m;
      // (from -inf, or so far that nothing is left of the sums, the difference itself must not enter them)
      const float d = top_m - m, k = m == -INFINITY ? 0.f : ex2(-d * kLog2e);
      const F2 kk = f2(k, k), dd = k == 0.f ? f2(0.f, 0.f) : f2(-d, -d);
      T2 = mul2(kk, fma2(dd, S2, T2));
      S2 = mul2(kk, S2);
      m = fmaxf(m, top_m);  // past a NaN the sums mean nothing
    }
    if (has_t && top_m >= xt) {  // only chunks whose maximum reaches the target's logit hold tokens before it
      const int lo = cb * kChunk - lead;
      if (lo > t) {
        before += count_group<T, U, false>(cur, xt);
      } else if (lo >= 0 && lo + U * kChunk <= t) {
        before += count_group<T, U, true>(cur, xt);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[8];
          unpack<T>(cur[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int id = elem_index<T>((cb + u) * kChunk, lead, lane, i);
            before += f[i] > xt || (f[i] == xt && id >= 0 && id < t);
          }
        }
      }
    }
    if (fabsf(m) <= Word<T>::kPlain) {
      const F2 mm = f2(-m, -m);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raise_lowest<T>(cur[u]);
        float f[8];
        unpack<T>(cur[u], f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const F2 z = add2(f2(f[i], f[i + 1]), mm);
          float y0, y1;
          f2_out(mul2(z, log2e), y0, y1);
          const F2 e = f2(ex2(y0), ex2(y1));
          S2 = add2(S2, e);
          T2 = fma2(e, z, T2);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[8], s = 0.f, t1 = 0.f;
        unpack<T>(cur[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = fmaxf(f[i] - m, -1000.f);  // also for -inf - -inf
          const float e = ex2(z * kLog2e);
          s += e;
          t1 = fmaf(e, z, t1);
        }
        S2 = add2(S2, f2(s, 0.f));
        T2 = add2(T2, f2(t1, 0.f));
      }
    }
  }
  float s0, s1, t0, t1;
  f2_out(S2, s0, s1);
  f2_out(T2, t0, t1);
  Part p;
  p.m = m;
  p.S = warp_sum(s0 + s1);
  p.T = warp_sum(t0 + t1);
  p.before = __reduce_add_sync(0xffffffffu, before);
  p.nan = nan;
  return p;
}

// The n-th largest of 32 (n <= 20) or 64 group maxima, two a lane: a bound with n elements at or above it.  Fewer
// groups are ordered sooner, but the nearer n is to their number, the more elements reach the bound.  32 against 64
// groups at n = 20: 62.4 / 63.8 us for 1000 x 131072 bf16, 10.1 / 10.7 for one row of 50,257, but 57 / 53 for 4000 x
// 16000 (a warp a row); at n = 24 65.1 / 65.2, 10.5 / 10.7 and 63 / 57; at n = 32 90 / 68, 12.9 / 11.5 and 817 / 64.
__device__ __forceinline__ uint32_t nth_bound(uint32_t g0, uint32_t g1, int n, int lane) {
  if (n <= 20) {
    const uint32_t g = max(g0, g1);
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t o = __shfl_sync(0xffffffffu, g, j);
      rank += o > g || (o == g && j < lane);
    }
    return __reduce_max_sync(0xffffffffu, rank == n - 1 ? g : 0u);
  }
  int r0 = 0, r1 = 0;
#pragma unroll 4
  for (int j = 0; j < 32; ++j) {
    const uint32_t a0 = __shfl_sync(0xffffffffu, g0, j), a1 = __shfl_sync(0xffffffffu, g1, j);
    r0 += (a0 > g0 || (a0 == g0 && j < lane)) + (a1 > g0);
    r1 += (a0 >= g1) + (a1 > g1 || (a1 == g1 && j < lane));
  }
  return __reduce_max_sync(0xffffffffu, max(r0 == n - 1 ? g0 : 0u, r1 == n - 1 ? g1 : 0u));
}

// Adds the lane's elements that reach b, a number above -inf (NaN reaches it,
// the -inf outside the row does not), to the candidates: (key, ~id), in any
// order.  Most lanes hold none; the others take them one by one.
template <class T>
__device__ __forceinline__ void add_reaching(const Raw<T>& raw, int pos0, int lead, int lane, float b,
                                             unsigned long long* cand, int cap, int* n_cand) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(raw.w);
  uint32_t in = 0;  // bit e: element e
  if constexpr (sizeof(T) == 4) {
    bool below = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) below &= __uint_as_float(u[i]) < b;
    if (below) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) in |= (uint32_t)!(__uint_as_float(u[i]) < b) << i;
  } else {
    typedef typename Word<T>::V2 V2;
    const V2 bb = Word<T>::both(b);
    const V2* v = reinterpret_cast<const V2*>(u);
    const uint32_t l0 = __hlt2_mask(v[0], bb), l1 = __hlt2_mask(v[1], bb), l2 = __hlt2_mask(v[2], bb),
                   l3 = __hlt2_mask(v[3], bb);
    if ((l0 & l1 & l2 & l3) == ~0u) return;
    // one bit of each half word, side by side
    in = (~l0 & 0x00020001u) | (~l1 & 0x00080004u) | (~l2 & 0x00200010u) | (~l3 & 0x00800040u);
    in = (in | in >> 16) & 0xffu;
  }
  int at = atomicAdd(n_cand, __popc(in));
  do {
    const int e = __ffs(in) - 1;
    in &= in - 1;
    float x;
    if constexpr (sizeof(T) == 4) {
      uint32_t w = u[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) w = e == i ? u[i] : w;
      x = __uint_as_float(w);
    } else {
      const uint32_t w = e < 4 ? (e < 2 ? u[0] : u[1]) : (e < 6 ? u[2] : u[3]);
      const float2 f = Word<T>::two(w);
      x = e & 1 ? f.y : f.x;
    }
    if (at < cap)
      cand[at] = (unsigned long long)sort_key(x) << 32 | (0xffffffffu - (uint32_t)elem_index<T>(pos0, lead, lane, e));
    ++at;
  } while (in);
}

// Adds the chunk's elements above key `tk`, and of those equal to it the first
// `ties` (which it lowers), to the candidates: (key, ~id), in any order.
template <class T>
__device__ __forceinline__ void add_candidates(const Raw<T>& raw, int pos0, int lead, int V, int lane, uint32_t tk,
                                               int* ties, unsigned long long* cand, int cap, int* n_cand) {
  constexpr int E = 16 / sizeof(T);
  uint32_t in = 0, eq = 0;
  float f[8];
  unpack<T>(raw, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int id = elem_index<T>(pos0, lead, lane, e);
    const uint32_t k = sort_key(f[e]);
    const bool real = id >= 0 && id < V;
    in |= (uint32_t)(real && k > tk) << e;
    eq |= (uint32_t)(real && k == tk) << e;
  }
  if (__any_sync(0xffffffffu, eq)) {
    int left = *ties;
#pragma unroll
    for (int w = 0; w < 8 / E; ++w) {  // by id: word after word, lane after lane
      uint32_t mine = eq >> (w * E) & ((1u << E) - 1u);
      const int n = __popc(mine);
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      for (int keep = left - (x - n); mine && keep > 0; --keep) {
        in |= (mine & -mine) << (w * E);
        mine &= mine - 1;
      }
      left -= __shfl_sync(0xffffffffu, x, 31);
    }
    *ties = max(left, 0);
  }
  if (in) {
    int at = atomicAdd(n_cand, __popc(in));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (in >> e & 1u) {
        const uint32_t id = (uint32_t)elem_index<T>(pos0, lead, lane, e);
        if (at < cap) cand[at] = (unsigned long long)sort_key(f[e]) << 32 | (0xffffffffu - id);
        ++at;
      }
  }
  __syncwarp();
}

// The outputs of one row from its joined part.
struct RowOut {
  float m, lnS, xt;
  bool bad, none;
  __device__ __forceinline__ RowOut(const Part& p) {
    m = p.m;
    bad = p.nan || p.m == INFINITY;
    none = p.m == -INFINITY;
    lnS = none || bad ? 0.f : logf(p.S);
  }
  __device__ __forceinline__ float lp(float x) const {
    return bad ? __uint_as_float(0x7fc00000u) : (x == -INFINITY ? -INFINITY : (x - m) - lnS);
  }
  __device__ __forceinline__ void write(const Args& a, int64_t r, const Part& p, int t, bool has_t, float xt) const {
    const float qnan = __uint_as_float(0x7fc00000u);
    if (a.logprob) a.logprob[r] = has_t ? lp(xt) : (t == -1 ? 0.f : qnan);
    if (a.rank) a.rank[r] = has_t && !p.nan ? p.before : -1;
    if (a.entropy) a.entropy[r] = bad ? qnan : (none ? 0.f : lnS - p.T / p.S);
    if (a.lse) a.lse[r] = bad ? qnan : (none ? -INFINITY : m + lnS);
  }
  __device__ __forceinline__ void write_top(const Args& a, int64_t r, int i, unsigned long long k) const {
    if (a.top_ids) a.top_ids[r * a.n_top + i] = (int32_t)(0xffffffffu - (uint32_t)k);
    if (a.top_lp) a.top_lp[r * a.n_top + i] = lp(key_value((uint32_t)(k >> 32)));
  }
};

// A CTA, or a cluster of CTAs, a row.  CTAs an SM: four of fp32 rows (500 x
// 131072: 51 us, against 65 with three), three of 16-bit rows, whose unpacking
// takes more registers (1000 x 131072, n 20: 62 us, against 68 with four).
template <class T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 3) logprobs_kernel(Args a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t leaders[];  // [n_chunks] chunk maxima; their sort keys from an exact search on
  __shared__ Part part, wpart[kWarps];
  __shared__ unsigned long long top[kMaxTop];               // this CTA's first n keys, in order
  __shared__ unsigned long long cand[kCand];
  __shared__ int32_t sel[kMaxTop], list[kList];
  __shared__ uint32_t tmax[2][kThreads];
  __shared__ int32_t n_cand, n_sel, n_keys, n_list;
  __shared__ uint32_t thr_key;
  __shared__ unsigned long long best_w[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = cluster.num_blocks(), cr = cluster.block_rank();
  const int64_t r = blockIdx.x / cs;
  const int V = a.V, n_top = a.n_top;
  const T* row = reinterpret_cast<const T*>(a.x) + r * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int all_chunks = (V + lead + kChunk - 1) / kChunk;
  // whole groups of U chunks per CTA; those past the row's end read as -inf
  constexpr int U = 4 / Raw<T>::W;
  const int per = ((all_chunks + cs - 1) / cs + U - 1) / U * U;
  const int c0 = min(all_chunks, per * cr), c1 = min(all_chunks, c0 + per), nc = c1 - c0;
  const int t = a.targets ? a.targets[r] : -1;
  const bool has_t = t >= 0 && t < V;
  const float xt = has_t ? to_f<T>(row[t]) : 0.f;
  float mine[2];
  if (threadIdx.x == 0) n_cand = n_list = 0;
  {
    const Part p = stream_chunks<T, U>(row, lead, V, t, xt, has_t, c0 + warp * U, c1, kWarps * U, lane, mine,
                                       [&](int c, float cm) { if (lane == 0) leaders[c - c0] = __float_as_uint(cm); });
    if (lane == 0) wpart[warp] = p;
  }
  tmax[0][threadIdx.x] = sort_key(mine[0]);
  tmax[1][threadIdx.x] = sort_key(mine[1]);
  __syncthreads();
  if (warp == kWarps - 1) {  // lane w takes warp w's part
    const Part p = merge_parts(lane < kWarps ? wpart[lane] : Part{-INFINITY, 0.f, 0.f, 0, 0});
    if (lane == 0) part = p;
  }

  // ------------------------------------- the first n_top keys of this CTA's part
  if (n_top > 0) {
    // every warp finds the bound from the threads' maxima and lists its share of the chunks that reach it
    uint32_t g0 = 0, g1 = 0;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
      g0 = max(g0, tmax[0][j * 32 + lane]);
      g1 = max(g1, tmax[1][j * 32 + lane]);
    }
    const uint32_t bound = nth_bound(g0, g1, n_top, lane);
    const float b = key_value(bound);
    const bool plain = b > -INFINITY;  // else masked rows, or NaN: the exact form
    for (int i = 0; plain && i < nc; i += kThreads) {
      const int c = i + lane * kWarps + warp;
      if (c < nc && sort_key(__uint_as_float(leaders[c])) >= bound) {
        const int at = atomicAdd(&n_list, 1);
        if (at < kList) list[at] = c;
      }
    }
    __syncthreads();
    const int nl = n_list;
    if (nl <= kList) {  // four chunks of a warp at a time, loaded together
      for (int i = warp * 4; i < nl; i += kWarps * 4) {
        Raw<T> raw[4];
        int c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          c[u] = i + u < nl ? list[i + u] : -1;
          if (c[u] >= 0) raw[u] = load_raw<T>(row, lead, V, (c0 + c[u]) * kChunk, lane);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c[u] >= 0) add_reaching<T>(raw[u], (c0 + c[u]) * kChunk, lead, lane, b, cand, kCand, &n_cand);
      }
    }
    __syncthreads();
    int ns = 0;
    if (!plain || nl > kList || n_cand > kCand) {
      // Many at the bound (masked or constant rows) or few chunks holding all the best: the n_top first chunks
      // exactly, in the order of their maxima; of elements equal to the last one's, n_top of a chunk at most.
      __syncthreads();
      if (threadIdx.x == 0) n_cand = 0;
      if (warp == 0) {  // lane l owns chunks l, l + 32, ...
        int taken = 0;
        const int want = min(n_top, nc);
        uint32_t bk = 0;
        int bc = 0x7fffffff;
        for (int c = lane; c < nc; c += 32) leaders[c] = sort_key(__uint_as_float(leaders[c]));
        auto rescan = [&]() {
          bk = 0;
          bc = 0x7fffffff;
          for (int c = lane; c < nc; c += 32) {
            const uint32_t k = leaders[c];
            if (k > bk) { bk = k; bc = c; }  // key 0 marks a chunk taken (no value has it)
          }
        };
        rescan();
        for (; taken < want; ++taken) {
          const uint32_t k = __reduce_max_sync(0xffffffffu, bk);
          const int c = (int)__reduce_min_sync(0xffffffffu, bk == k ? (unsigned)bc : 0x7fffffffu);
          if (lane == 0) { sel[taken] = c; thr_key = k; }
          if ((c & 31) == lane) { leaders[c] = 0; rescan(); }
        }
        if (lane == 0) {
          n_sel = want;
          if (want < n_top) thr_key = 0;
        }
      }
      __syncthreads();
      ns = n_sel;
      const uint32_t tk = thr_key;
      for (int i = warp; i < ns; i += kWarps) {
        int ties = n_top;
        add_candidates<T>(load_raw<T>(row, lead, V, (c0 + sel[i]) * kChunk, lane), (c0 + sel[i]) * kChunk, lead, V, lane,
                          tk, &ties, cand, kCand, &n_cand);
      }
    }
    __syncthreads();
    const int n = n_cand, out = min(n_top, n);
    if (n <= kCand) {
      // few: rank of each = keys above it
      if (n <= 256) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const unsigned long long k = cand[i];
          int rank = 0;
#pragma unroll 4
          for (int j = 0; j < n; ++j) rank += cand[j] > k;
          if (rank < out) top[rank] = k;
        }
      } else {  // bitonic, descending
        int p2 = 512;
        while (p2 < n) p2 <<= 1;
        for (int i = n + threadIdx.x; i < p2; i += kThreads) cand[i] = 0;
        __syncthreads();
        for (int k = 2; k <= p2; k <<= 1)
          for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < p2; i += kThreads) {
              const int x = i ^ j;
              if (x > i) {
                const unsigned long long u = cand[i], v = cand[x];
                if ((u < v) == ((i & k) == 0)) { cand[i] = v; cand[x] = u; }
              }
            }
            __syncthreads();
          }
        for (int i = threadIdx.x; i < out; i += kThreads) top[i] = cand[i];
      }
    } else {
      // many ascending values: extract one after another
      unsigned long long last = ~0ull;
      for (int o = 0; o < out; ++o) {
        unsigned long long best = 0;
        for (int i = warp; i < ns; i += kWarps) {
          float f[8];
          const int pos0 = (c0 + sel[i]) * kChunk;
          load8<T>(row, lead, V, pos0, lane, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int id = elem_index<T>(pos0, lead, lane, e);
            const unsigned long long k = (unsigned long long)sort_key(f[e]) << 32 | (0xffffffffu - (uint32_t)id);
            if (id >= 0 && id < V && k < last && k > best) best = k;
          }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, s);
          best = k > best ? k : best;
        }
        if (lane == 0) best_w[warp] = best;
        __syncthreads();
        best = best_w[0];
        for (int w = 1; w < kWarps; ++w) best = best_w[w] > best ? best_w[w] : best;
        if (threadIdx.x == 0) top[o] = best;
        last = best;
        __syncthreads();
      }
    }
    if (threadIdx.x == 0) n_keys = out;
  }

  // ------------------------------------------------- merge over the cluster
  if (cs > 1) {
    cluster.sync();
    Part all{};
    if (cr == 0) {
      // the lists, one behind the other: the rank of a key is the keys above it in every list
      if (n_top > 0) {
        for (int i = threadIdx.x; i < cs * n_top; i += kThreads) {
          const int b = i / n_top, j = i % n_top;
          cand[i] = j < *cluster.map_shared_rank(&n_keys, b) ? cluster.map_shared_rank(top, b)[j] : 0ull;
        }
      }
      all = merge_parts(lane < cs ? *cluster.map_shared_rank(&part, lane) : Part{-INFINITY, 0.f, 0.f, 0, 0});
    }
    cluster.sync();  // the other CTAs are done
    if (cr != 0) return;
    const RowOut o(all);
    if (threadIdx.x == 0) o.write(a, r, all, t, has_t, xt);
    for (int i = threadIdx.x; i < cs * n_top; i += kThreads) {
      const unsigned long long k = cand[i];
      if (k == 0ull) continue;
      int rank = 0;
      for (int b = 0; b < cs; ++b) {
        int lo = 0, hi = n_top;  // keys of list b above k
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (cand[b * n_top + mid] > k) lo = mid + 1; else hi = mid;
        }
        rank += lo;
      }
      if (rank < n_top) o.write_top(a, r, rank, k);
    }
    return;
  }
  __syncthreads();
  const Part p = part;
  const RowOut o(p);
  if (threadIdx.x == 0) o.write(a, r, p, t, has_t, xt);
  for (int i = threadIdx.x; i < n_top; i += kThreads) o.write_top(a, r, i, top[i]);
}

// A warp a row, for many rows of up to 64 chunks and n <= 56: everything stays in the warp,
// with no barrier.  4000 rows of 8000 bf16 logits, n 20: 37 us, against 60 us
// with a CTA a row, whose end (several barriers a row) outweighs the row.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_warp_kernel(Args a) {
  __shared__ unsigned long long cand_s[kWarps][kWarpCand];
  __shared__ int32_t n_cand_s[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (r >= a.rows) return;
  const int V = a.V, n_top = a.n_top;
  const T* row = reinterpret_cast<const T*>(a.x) + r * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int nc = (V + lead + kChunk - 1) / kChunk;
  constexpr int U = 4 / Raw<T>::W;
  const int t = a.targets ? a.targets[r] : -1;
  const bool has_t = t >= 0 && t < V;
  const float xt = has_t ? to_f<T>(row[t]) : 0.f;
  unsigned long long* cand = cand_s[warp];
  int* n_cand = &n_cand_s[warp];
  if (lane == 0) *n_cand = 0;
  float mine[2], lead_max[2] = {-INFINITY, -INFINITY};  // lane l: the maxima of chunks l and l + 32
  const Part p = stream_chunks<T, U>(row, lead, V, t, xt, has_t, 0, nc, U, lane, mine, [&](int c, float cm) {
    lead_max[0] = c == lane ? cm : lead_max[0];
    lead_max[1] = c == lane + 32 ? cm : lead_max[1];
  });
  const RowOut o(p);
  if (lane == 0) o.write(a, r, p, t, has_t, xt);
  if (n_top == 0) return;
  const uint32_t bound = nth_bound(sort_key(mine[0]), sort_key(mine[1]), n_top, lane);
  const uint32_t reach[2] = {
      __ballot_sync(0xffffffffu, lane < nc && sort_key(lead_max[0]) >= bound),
      __ballot_sync(0xffffffffu, lane + 32 < nc && sort_key(lead_max[1]) >= bound)};
  // four chunks at a time, loaded together
  auto each = [&](auto fn) {
    uint64_t left = (uint64_t)reach[1] << 32 | reach[0];
    while (left) {
      Raw<T> raw[4];
      int c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        c[u] = left ? __ffsll((long long)left) - 1 : -1;
        left &= left - 1;
        if (c[u] >= 0) raw[u] = load_raw<T>(row, lead, V, c[u] * kChunk, lane);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c[u] >= 0) fn(raw[u], c[u] * kChunk);
    }
    __syncwarp();
  };
  const float b = key_value(bound);
  const bool plain = b > -INFINITY;
  if (plain) each([&](const Raw<T>& w, int pos0) { add_reaching<T>(w, pos0, lead, lane, b, cand, kWarpCand, n_cand); });
  if (!plain || *n_cand > kWarpCand) {
    // masked or constant rows: chunks in the order of ids, so no more than n_top equals of the bound are among the first
    __syncwarp();
    if (lane == 0) *n_cand = 0;
    __syncwarp();
    int ties = n_top;
    each([&](const Raw<T>& w, int pos0) {
      add_candidates<T>(w, pos0, lead, V, lane, bound, &ties, cand, kWarpCand, n_cand);
    });
  }
  const int n = *n_cand;
  if (n <= kWarpCand) {
    for (int i = lane; i < n; i += 32) {
      const unsigned long long k = cand[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += cand[j] > k;
      if (rank < n_top) o.write_top(a, r, rank, k);
    }
  } else {  // many above the bound (ascending values, say): extract one after another, a pass over the row each
    unsigned long long last = ~0ull;
    for (int i = 0; i < n_top; ++i) {
      unsigned long long best = 0;
      for (int c = 0; c < nc; ++c) {
        if (!(reach[c >> 5] >> (c & 31) & 1u)) continue;
        float f[8];
        load8<T>(row, lead, V, c * kChunk, lane, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int id = elem_index<T>(c * kChunk, lead, lane, e);
          const unsigned long long k = (unsigned long long)sort_key(f[e]) << 32 | (0xffffffffu - (uint32_t)id);
          if (id >= 0 && id < V && k < last && k > best) best = k;
        }
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, s);
        best = k > best ? k : best;
      }
      last = best;
      if (lane == 0) o.write_top(a, r, i, best);
    }
  }
}

template <class T>
static int launch(Args a, cudaStream_t s) {
  int dev = 0, sms = 0;
  TL_CUDA(cudaGetDevice(&dev));
  TL_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  // Many short rows: a warp a row, unless so many of the best are wanted that ordinary rows hold more than kWarpCand
  // candidates (the bound is the n-th of 64 maxima: at n = 64 some 300 elements reach the lowest of them) and would be
  // read once per token wanted.  4000 x 8000 bf16, a warp against a CTA a row: n 20 38 / 65 us, n 56 70 / 96, n 60
  // 605 / 110, n 64 2,991 / 186; 4000 x 16000: n 56 97 / 120, n 58 589 / 124; 1300 x 3001 fp32: n 56 31 / 30.
  const bool by_warp = a.V + 8 <= 64 * kChunk && a.rows >= 8 * sms && a.n_top <= kWarpTop;
  // CTAs of a row: as many as fill the SMs at most once (a second wave of them costs more than the first saves:
  // 128 x 131072 bf16 took 16 us with 2 CTAs a row and 31 us with 8), each with 2 groups of chunks a warp or more
  int cs = 1;
  while (cs < kMaxCluster && a.rows * cs * 2 <= 3 * sms && a.V >= 2 * cs * kWarps * kChunk) cs *= 2;
  const int chunks = (a.V + 8 + kChunk - 1) / kChunk;
  a.n_chunks = (chunks + cs - 1) / cs + 4;  // rounded up to groups of 4 at most
  const int64_t most = 0x7fffffff / kMaxCluster;  // rows of one launch
  for (int64_t r0 = 0; r0 < a.rows; r0 += most) {
    Args b = a;
    b.rows = a.rows - r0 < most ? a.rows - r0 : most;
    b.x = static_cast<const T*>(a.x) + r0 * a.stride;
    if (b.targets) b.targets += r0;
    if (b.logprob) b.logprob += r0;
    if (b.rank) b.rank += r0;
    if (b.entropy) b.entropy += r0;
    if (b.lse) b.lse += r0;
    if (b.top_ids) b.top_ids += r0 * a.n_top;
    if (b.top_lp) b.top_lp += r0 * a.n_top;
    if (by_warp) {
      const int wpc = kWarps;
      logprobs_warp_kernel<T><<<(unsigned)((b.rows + wpc - 1) / wpc), wpc * 32, 0, s>>>(b);
      TL_CUDA(cudaGetLastError());
      continue;
    }
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(b.rows * cs));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = (size_t)a.n_chunks * 4;
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    TL_CUDA(cudaLaunchKernelEx(&lc, logprobs_kernel<T>, b));
  }
  return check_cuda(cudaGetLastError());
}

}  // namespace logprobs
}  // namespace tl

using namespace tl;

extern "C" int tl_token_logprobs(const void* dev_logits, int32_t dtype, int64_t rows, int32_t vocab,
                                 int64_t row_stride, const int32_t* dev_targets, int32_t n_top, float* dev_logprob,
                                 int32_t* dev_rank, float* dev_entropy, float* dev_lse, int32_t* dev_top_ids,
                                 float* dev_top_logprobs, void* cuda_stream) {
  namespace lp = logprobs;
  if (dtype != TL_F32 && dtype != TL_F16 && dtype != TL_BF16) return TL_EINVAL;
  const int es = dtype == TL_F32 ? 4 : 2;
  if (rows < 0 || vocab < 1 || vocab > lp::kMaxVocab || n_top < 0 || n_top > lp::kMaxTop || n_top > vocab ||
      (rows > 1 && row_stride < vocab))
    return TL_EINVAL;
  if ((dev_logprob || dev_rank) && !dev_targets) return TL_EINVAL;
  if ((dev_top_ids || dev_top_logprobs) && n_top == 0) return TL_EINVAL;
  if (((uintptr_t)dev_logits & (es - 1)) || ((uintptr_t)dev_targets & 3) || ((uintptr_t)dev_logprob & 3) ||
      ((uintptr_t)dev_rank & 3) || ((uintptr_t)dev_entropy & 3) || ((uintptr_t)dev_lse & 3) ||
      ((uintptr_t)dev_top_ids & 3) || ((uintptr_t)dev_top_logprobs & 3))
    return TL_EINVAL;
  if (rows == 0) return TL_OK;
  if (!dev_logits) return TL_EINVAL;
  const lp::Args a{dev_logits, rows, row_stride, vocab, dev_top_ids || dev_top_logprobs ? n_top : 0, dev_targets,
                   dev_logprob, dev_rank, dev_entropy, dev_lse, dev_top_ids, dev_top_logprobs, 0};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  switch (dtype) {
    case TL_F32: return lp::launch<float>(a, s);
    case TL_F16: return lp::launch<__half>(a, s);
    default: return lp::launch<__nv_bfloat16>(a, s);
  }
}
