// Log probabilities, rank, entropy and best alternatives of rows of logits.
//
//   lse = m + ln S,  S = sum exp(x - m),  T = sum (x - m) exp(x - m)
//   logprob_t = (x_t - m) - ln S,  entropy = ln S - T / S
//
// One pass over the row.  A row is cut into chunks of 256 consecutive
// elements; a warp takes a chunk at a time, 8 elements a lane, and keeps a
// running maximum (uniform in the warp) with S and T rescaled when it rises.
// The chunk maxima that this needs anyway are kept in shared memory: the n
// first elements in the order (value descending, id ascending) lie in the n
// chunks whose maxima come first in (maximum descending, chunk ascending),
// since each chunk before an element's own holds an element before it.  So only
// those n chunks are read again (they are in L2), filtered by the n-th chunk
// maximum, and the few that pass are ordered.
//
// Few rows: a cluster of up to 8 CTAs shares a row and its first CTA merges the
// partial sums and lists over distributed shared memory, with no scratch in
// global memory and no atomics, so results do not depend on timing.
//
// Per lane S and T are fp32 sums of vocab / (256 * CTAs) terms or so; they are
// merged, and the logarithm taken, in fp64.
#include <cooperative_groups.h>

#include "common.cuh"
#include "host_util.h"

namespace tl {
namespace logprobs {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 256;      // elements a warp reads at a time: 8 a lane
constexpr int kMaxTop = 64;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kCand = 2048;      // candidates ordered in shared memory; more take the extraction loop
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
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <class T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Elements of one 16-byte word.
template <class T>
__device__ __forceinline__ void unpack(const uint4& w, float* f) {
  const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) f[i] = to_f<T>(e[i]);
}

// The lane's 8 elements of a chunk.  Positions are counted from the 16-byte
// boundary at or before the row (`lead` elements before it), so whole words
// are aligned; a word that holds the row's first or last elements is read by
// element.  Elements outside the row are -inf.  Lane l holds, of each word w
// of its 8 elements, positions base + w * 32 * E + l * E + (0 .. E-1).
template <class T>
__device__ __forceinline__ void load8(const T* row, int lead, int V, int64_t pos0, int lane, float* f) {
  constexpr int E = 16 / sizeof(T);  // elements of a word
#pragma unroll
  for (int w = 0; w < 8 / E; ++w) {
    const int64_t p = pos0 + (w * 32 + lane) * E - lead;  // element index of the word's first
    if (p >= 0 && p + E <= V) {
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(row + p)), f + w * E);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[w * E + e] = (p + e >= 0 && p + e < V) ? to_f<T>(row[p + e]) : -INFINITY;
    }
  }
}
template <class T>
__device__ __forceinline__ int elem_index(int64_t pos0, int lead, int lane, int i) {
  constexpr int E = 16 / sizeof(T);
  return (int)(pos0 + ((i / E) * 32 + lane) * E + i % E - lead);
}

struct Part {  // a CTA's share of a row
  double S, T;
  float m;
  int32_t before;
  int32_t n_keys;
  int32_t nan;
};

template <class T>
__global__ void __launch_bounds__(kThreads, 4) kernel(Args a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t leaders[];  // [n_chunks] sort keys of the chunk maxima
  __shared__ Part part;
  __shared__ double wS[kWarps], wT[kWarps];
  __shared__ float wm[kWarps];
  __shared__ int32_t wcnt[kWarps];
  __shared__ unsigned long long top[kMaxTop];               // this CTA's first n keys, in order
  __shared__ unsigned long long cand[kCand];
  __shared__ int32_t sel[kMaxTop];
  __shared__ int32_t n_cand, n_sel, thr_chunk;
  __shared__ uint32_t thr_key;
  __shared__ unsigned long long best_w[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = cluster.num_blocks(), cr = cluster.block_rank();
  const int64_t r = blockIdx.x / cs;
  const int V = a.V, n_top = a.n_top;
  const T* row = reinterpret_cast<const T*>(a.x) + r * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int all_chunks = (V + lead + kChunk - 1) / kChunk;
  const int per = (all_chunks + cs - 1) / cs;
  const int c0 = min(all_chunks, per * cr), c1 = min(all_chunks, c0 + per), nc = c1 - c0;
  const int t = a.targets ? a.targets[r] : -1;
  const bool has_t = t >= 0 && t < V;
  const float xt = has_t ? to_f<T>(row[t]) : 0.f;

  // ------------------------------------------------------------ one pass
  float m = -INFINITY, S = 0.f, U = 0.f;
  int before = 0;
  bool nan = false;
  for (int c = c0 + warp; c < c1; c += kWarps) {
    float f[8];
    const int64_t pos0 = (int64_t)c * kChunk;
    load8<T>(row, lead, V, pos0, lane, f);
    float mx = f[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = max_nan(mx, f[i]);
    const uint32_t key = __reduce_max_sync(0xffffffffu, sort_key(mx));
    if (lane == 0) leaders[c - c0] = key;
    nan |= key == 0xffffffffu;
    const float cm = key_value(key);
    if (cm > m) {
      const float d = cm - m, s = m == -INFINITY ? 0.f : ex2(-d * kLog2e);
      U = m == -INFINITY ? 0.f : s * (U - d * S);
      S *= s;
      m = cm;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = fmaxf(f[i] - m, -1000.f);  // -inf (and -inf - -inf) to a value whose exponential is 0
      const float e = ex2(z * kLog2e);
      S += e;
      U = fmaf(e, z, U);
    }
    if (has_t) {
      const int lo = (int)(pos0 - lead), hi = lo + kChunk;
      if (hi <= t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) before += f[i] >= xt && (lo >= 0 || elem_index<T>(pos0, lead, lane, i) >= 0);
      } else if (lo > t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) before += f[i] > xt;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int id = elem_index<T>(pos0, lead, lane, i);
          before += f[i] > xt || (f[i] == xt && id >= 0 && id < t);
        }
      }
    }
  }
  {
    const double s = warp_sum_d((double)S), u = warp_sum_d((double)U);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) { wS[warp] = s; wT[warp] = u; wm[warp] = nan ? __uint_as_float(0x7fc00000u) : m; wcnt[warp] = before; }
  }
  if (threadIdx.x == 0) n_cand = 0;
  __syncthreads();
  if (threadIdx.x == 0) {
    Part p{0.0, 0.0, -INFINITY, 0, 0, 0};
    for (int w = 0; w < kWarps; ++w) { p.nan |= wm[w] != wm[w]; p.m = fmaxf(p.m, wm[w]); p.before += wcnt[w]; }
    for (int w = 0; w < kWarps; ++w) {
      if (!(wm[w] > -INFINITY)) continue;
      const double d = (double)p.m - (double)wm[w], s = exp(-d);
      p.S += s * wS[w];
      p.T += s * (wT[w] - d * wS[w]);
    }
    part = p;
  }

  // ------------------------------------- the first n_top keys of this CTA's part
  if (n_top > 0) {
    if (warp == 0) {
      // the n_top first chunks, in order: lane l owns chunks l, l + 32, ...
      int taken = 0;
      const int want = min(n_top, nc);
      uint32_t bk = 0;
      int bc = 0x7fffffff;
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
        if (lane == 0) { sel[taken] = c; thr_key = k; thr_chunk = c; }
        if ((c & 31) == lane) { leaders[c] = 0; rescan(); }
      }
      if (lane == 0) {
        n_sel = want;
        if (want < n_top) { thr_key = 0; thr_chunk = 0x7fffffff; }
      }
    }
    __syncthreads();
    // elements at or before the last selected chunk's maximum
    const uint32_t tk = thr_key;
    const int tc = thr_chunk, ns = n_sel;
    for (int i = warp; i < ns; i += kWarps) {
      const int c = sel[i];
      float f[8];
      const int64_t pos0 = (int64_t)(c0 + c) * kChunk;
      load8<T>(row, lead, V, pos0, lane, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int id = elem_index<T>(pos0, lead, lane, e);
        const uint32_t k = sort_key(f[e]);
        const bool in = id >= 0 && id < V && (k > tk || (k == tk && c <= tc));
        const unsigned bal = __ballot_sync(0xffffffffu, in);
        int at = 0;
        if (lane == 0 && bal) at = atomicAdd(&n_cand, __popc(bal));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(bal & ((1u << lane) - 1u));
        if (in && at < kCand) cand[at] = (unsigned long long)k << 32 | (0xffffffffu - (uint32_t)id);
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
      // many equal or ascending values: extract one after another
      unsigned long long last = ~0ull;
      for (int o = 0; o < out; ++o) {
        unsigned long long best = 0;
        for (int i = warp; i < ns; i += kWarps) {
          float f[8];
          const int64_t pos0 = (int64_t)(c0 + sel[i]) * kChunk;
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
    __syncthreads();
    if (threadIdx.x == 0) part.n_keys = out;
  }

  // ------------------------------------------------- merge over the cluster
  if (cs > 1) {
    cluster.sync();
    if (cr == 0) {
      // the lists, one behind the other: the rank of a key is the keys above it in every list
      if (n_top > 0) {
        for (int i = threadIdx.x; i < cs * n_top; i += kThreads) {
          const int b = i / n_top, j = i % n_top;
          const Part* pb = cluster.map_shared_rank(&part, b);
          cand[i] = j < pb->n_keys ? cluster.map_shared_rank(top, b)[j] : 0ull;
        }
        __syncthreads();
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
          if (rank < n_top) top[rank] = k;
        }
      }
      if (threadIdx.x == 0) {
        Part p{0.0, 0.0, -INFINITY, 0, 0, 0};
        for (int b = 0; b < cs; ++b) {
          const Part q = *cluster.map_shared_rank(&part, b);
          p.nan |= q.nan;
          p.m = fmaxf(p.m, q.m);
          p.before += q.before;
        }
        for (int b = 0; b < cs; ++b) {
          const Part q = *cluster.map_shared_rank(&part, b);
          if (!(q.m > -INFINITY)) continue;
          const double d = (double)p.m - (double)q.m, s = exp(-d);
          p.S += s * q.S;
          p.T += s * (q.T - d * q.S);
        }
        part = p;
      }
    }
    cluster.sync();
  } else {
    __syncthreads();
  }
  if (cr != 0) return;

  // ------------------------------------------------------------- outputs
  const Part p = part;
  const bool bad = p.nan || p.m == INFINITY, none = p.m == -INFINITY;
  const float qnan = __uint_as_float(0x7fc00000u);
  const double lnS = none || bad ? 0.0 : log(p.S);
  auto lp = [&](float x) { return bad ? qnan : (x == -INFINITY ? -INFINITY : (float)((double)x - (double)p.m - lnS)); };
  if (threadIdx.x == 0) {
    if (a.logprob) a.logprob[r] = has_t ? lp(xt) : (t == -1 ? 0.f : qnan);
    if (a.rank) a.rank[r] = has_t && !p.nan ? p.before : -1;
    if (a.entropy) a.entropy[r] = bad ? qnan : (none ? 0.f : (float)(lnS - p.T / p.S));
    if (a.lse) a.lse[r] = bad ? qnan : (none ? -INFINITY : (float)((double)p.m + lnS));
  }
  for (int i = threadIdx.x; i < n_top; i += kThreads) {
    const unsigned long long k = top[i];
    if (a.top_ids) a.top_ids[r * n_top + i] = (int32_t)(0xffffffffu - (uint32_t)k);
    if (a.top_lp) a.top_lp[r * n_top + i] = lp(key_value((uint32_t)(k >> 32)));
  }
}

template <class T>
static int launch(Args a, cudaStream_t s) {
  int dev = 0, sms = 0;
  TL_CUDA(cudaGetDevice(&dev));
  TL_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  // CTAs of a row: enough for four on every SM, each with 8 chunks or more
  int cs = 1;
  while (cs < kMaxCluster && a.rows * cs < 4 * sms && a.V >= 2 * cs * kWarps * kChunk) cs *= 2;
  const int chunks = (a.V + 8 + kChunk - 1) / kChunk;
  a.n_chunks = (chunks + cs - 1) / cs;
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
    TL_CUDA(cudaLaunchKernelEx(&lc, kernel<T>, b));
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
