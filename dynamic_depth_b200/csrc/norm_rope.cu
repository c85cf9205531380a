// Per-head RMSNorm of queries and keys, rotation, and the append to a paged
// cache, in one pass over the projection's rows (tl_norm_rope_append).
//
// A thread owns 8 elements of a head's first half and the 8 they rotate with in
// the second half, so the rotation needs no exchange and a head's sum of
// squares is one shuffle reduction over head_dim / 16 neighbouring lanes.  All
// global accesses are 16-byte words: every element is read once and written
// once, in the order of the projection row, so the pass is bound by memory:
// 8,190 fp32 rows of 48 heads x 128 take 50.6 us, 6.05 TB/s (92 % of a copy).
// Small CTAs turn over sooner: 256 threads a CTA took 53.7 us, and 59.3 with
// the position looked at before the row's loads were on their way.
#include "common.cuh"
#include "host_util.h"
#include "tree_attn.h"

namespace tl {
namespace norm_rope {

constexpr int kThreads = 128;

struct Args {
  const void* x;
  int64_t rows, stride;
  int32_t H, Hk;
  const float *gq, *gk;
  float eps;
  const float2* table;
  int32_t length;
  const int32_t* pos;
  const int64_t* slots;
  void* pool;
  int64_t n_slots;
  int32_t shift;
  void* q;
  int32_t* status;
  // a context's lane: slots count positions of one cache slot of the lane, whose pages are map[0 .. map_pages)
  const int32_t* map;
  int32_t map_pages;
};

template <class T>
struct Pair2 {};
template <>
struct Pair2<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
};
template <>
struct Pair2<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Pair2<T>::unpack(u[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  uint4 w;
  w.x = Pair2<T>::pack(f[0], f[1]);
  w.y = Pair2<T>::pack(f[2], f[3]);
  w.z = Pair2<T>::pack(f[4], f[5]);
  w.w = Pair2<T>::pack(f[6], f[7]);
  *reinterpret_cast<uint4*>(p) = w;
}

template <class TI, class TC, int HD>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(Args a) {
  constexpr int LT = HD / 16;  // lanes of a head
  const int heads = a.H + 2 * a.Hk;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LT;
  const int part = threadIdx.x % LT;
  const int64_t row = unit / heads;
  const int h = (int)(unit - row * heads);
  if (row >= a.rows) return;  // a head's lanes leave together
  const bool is_q = h < a.H, is_v = h >= a.H + a.Hk;
  // every load that does not wait for another is on its way before the first is looked at
  const int pos = __ldg(a.pos + row);
  int64_t slot = is_q ? 0 : __ldg(reinterpret_cast<const long long*>(a.slots) + row);
  const TI* src = static_cast<const TI*>(a.x) + row * a.stride + h * HD + part * 8;
  float lo[8], hi[8];
  load8<TI>(src, lo);
  load8<TI>(src + HD / 2, hi);
  if (pos < 0 || pos >= a.length) {
    if (part == 0 && a.status) atomicOr(a.status, TL_BAD_POSITION);
    return;
  }
  if (!is_v) {
    const float* g = is_q ? a.gq : a.gk;
    if (g) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
      const unsigned group = LT == 32 ? 0xffffffffu : ((1u << LT) - 1u) << ((threadIdx.x & 31) / LT * LT);
#pragma unroll
      for (int o = LT / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float inv = rsqrtf(ss * (1.f / HD) + a.eps);
      float g0[8], g1[8];
      load8<float>(g + part * 8, g0);
      load8<float>(g + HD / 2 + part * 8, g1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] *= inv * g0[i];
        hi[i] *= inv * g1[i];
      }
    }
    const float4* cs = reinterpret_cast<const float4*>(a.table + (int64_t)pos * (HD / 2) + part * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = __ldg(cs + i);
      const float x0 = lo[2 * i], y0 = hi[2 * i], x1 = lo[2 * i + 1], y1 = hi[2 * i + 1];
      lo[2 * i] = x0 * c.x - y0 * c.y;
      hi[2 * i] = y0 * c.x + x0 * c.y;
      lo[2 * i + 1] = x1 * c.z - y1 * c.w;
      hi[2 * i + 1] = y1 * c.z + x1 * c.w;
    }
  }
  TC* dst;
  if (is_q) {
    dst = static_cast<TC*>(a.q) + (row * a.H + h) * HD;
  } else {
    if (a.map && slot >= 0) {
      const int64_t i = slot >> a.shift;
      const int page = i < a.map_pages ? a.map[i] : -1;
      slot = page < 0 ? -2 : ((int64_t)page << a.shift) + (slot & ((1 << a.shift) - 1));
    }
    if (slot < 0 || slot >= a.n_slots) {
      if (slot != -1 && part == 0 && a.status) atomicOr(a.status, TL_BAD_SLOT);
      return;
    }
    const int64_t page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
    const int kh = h - a.H;  // a page: [key heads | value heads], as in the row
    dst = static_cast<TC*>(a.pool) + (((page * 2 * a.Hk + kh) << a.shift) + off) * HD;
  }
  store8<TC>(dst + part * 8, lo);
  store8<TC>(dst + HD / 2 + part * 8, hi);
}

__global__ void table_kernel(float2* t, int length, int half, double base) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)length * half) return;
  const int p = (int)(i / half), k = (int)(i % half);
  double s, c;
  sincos((double)p * pow(base, -2.0 * k / (2.0 * half)), &s, &c);
  t[i] = make_float2((float)c, (float)s);
}

template <class TI, class TC>
static int launch(const Args& a, int hd, cudaStream_t s) {
  const int64_t threads = a.rows * (a.H + 2 * a.Hk) * (hd / 16);
  const int64_t grid = (threads + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return TL_EINVAL;
  switch (hd) {
    case 32: norm_rope_kernel<TI, TC, 32><<<(unsigned)grid, kThreads, 0, s>>>(a); break;
    case 64: norm_rope_kernel<TI, TC, 64><<<(unsigned)grid, kThreads, 0, s>>>(a); break;
    default: norm_rope_kernel<TI, TC, 128><<<(unsigned)grid, kThreads, 0, s>>>(a); break;
  }
  return check_cuda(cudaGetLastError());
}
template <class TC>
static int launch_in(const Args& a, int dtype, int hd, cudaStream_t s) {
  switch (dtype) {
    case TL_F32: return launch<float, TC>(a, hd, s);
    case TL_F16: return launch<__half, TC>(a, hd, s);
    default: return launch<__nv_bfloat16, TC>(a, hd, s);
  }
}

}  // namespace norm_rope

int norm_rope_lane(const float* qkv, int64_t rows, int32_t n_heads, const float2* table, int32_t length,
                   const int32_t* positions, const int64_t* slots, const tl_kv_pool& pool, const int32_t* map,
                   int32_t map_pages, __half* q_out, int32_t* status, cudaStream_t s) {
  norm_rope::Args a{qkv, rows, 3 * (int64_t)n_heads * pool.head_dim, n_heads, n_heads, nullptr, nullptr, 0.f, table,
                    length, positions, slots, pool.dev_pool, pool.n_pages * pool.page_tokens, 0, q_out, status, map,
                    map_pages};
  while ((1 << a.shift) < pool.page_tokens) ++a.shift;
  return norm_rope::launch<float, __half>(a, pool.head_dim, s);
}

// The pool of the serving operators: sizes, alignment, and rows within a tensor map's 32-bit coordinates.
bool kv_pool_ok(const tl_kv_pool* p) {
  if (!p || !p->dev_pool || ((uintptr_t)p->dev_pool & 15) || p->n_pages < 1 || p->n_kv_heads < 1) return false;
  if (p->dtype != TL_F16 && p->dtype != TL_BF16) return false;
  if (p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128) return false;
  if (p->page_tokens < 16 || p->page_tokens > 1024 || (p->page_tokens & (p->page_tokens - 1))) return false;
  const int64_t per = 2 * (int64_t)p->n_kv_heads * p->page_tokens;
  return p->n_pages <= 0x7fffffff / per;
}

}  // namespace tl

using namespace tl;

extern "C" int tl_rope_table(float* dev_table, int32_t length, int32_t head_dim, double base, void* cuda_stream) {
  if (!dev_table || ((uintptr_t)dev_table & 15) || length < 1 || head_dim < 2 || head_dim > 1024 || head_dim % 2 ||
      !(base > 0.0))
    return TL_EINVAL;
  const int64_t n = (int64_t)length * (head_dim / 2);
  if ((n + 255) / 256 > 0x7fffffff) return TL_EINVAL;
  norm_rope::table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, (cudaStream_t)cuda_stream>>>(
      reinterpret_cast<float2*>(dev_table), length, head_dim / 2, base);
  return check_cuda(cudaGetLastError());
}

extern "C" int tl_norm_rope_append(const void* dev_qkv, int32_t dtype, int64_t rows, int64_t row_stride,
                                   int32_t n_heads, const float* dev_q_gain, const float* dev_k_gain, float eps,
                                   const float* dev_table, int32_t length, const int32_t* dev_positions,
                                   const int64_t* dev_slots, const tl_kv_pool* pool, void* dev_q_out,
                                   int32_t* dev_status, void* cuda_stream) {
  if (!kv_pool_ok(pool)) return TL_EINVAL;
  if (dtype != TL_F32 && dtype != TL_F16 && dtype != TL_BF16) return TL_EINVAL;
  const int es = dtype == TL_F32 ? 4 : 2;
  const int64_t width = ((int64_t)n_heads + 2 * pool->n_kv_heads) * pool->head_dim;
  if (rows < 0 || rows > (int64_t(1) << 40) || n_heads < 1 || n_heads % pool->n_kv_heads || (rows > 1 && row_stride < width) ||
      (row_stride * es) % 16 || length < 1 || (dev_q_gain == nullptr) != (dev_k_gain == nullptr) || !(eps >= 0.f))
    return TL_EINVAL;
  if (rows == 0) return TL_OK;
  if (!dev_qkv || !dev_table || !dev_positions || !dev_slots || !dev_q_out) return TL_EINVAL;
  if (((uintptr_t)dev_qkv & 15) || ((uintptr_t)dev_q_gain & 15) || ((uintptr_t)dev_k_gain & 15) ||
      ((uintptr_t)dev_table & 15) || ((uintptr_t)dev_positions & 3) || ((uintptr_t)dev_slots & 7) ||
      ((uintptr_t)dev_q_out & 15) || ((uintptr_t)dev_status & 3))
    return TL_EINVAL;
  norm_rope::Args a{dev_qkv, rows, row_stride, n_heads, pool->n_kv_heads, dev_q_gain, dev_k_gain, eps,
                    reinterpret_cast<const float2*>(dev_table), length, dev_positions, dev_slots, pool->dev_pool,
                    pool->n_pages * pool->page_tokens, 0, dev_q_out, dev_status, nullptr, 0};
  while ((1 << a.shift) < pool->page_tokens) ++a.shift;
  cudaStream_t s = (cudaStream_t)cuda_stream;
  return pool->dtype == TL_F16 ? norm_rope::launch_in<__half>(a, dtype, pool->head_dim, s)
                               : norm_rope::launch_in<__nv_bfloat16>(a, dtype, pool->head_dim, s);
}
