// Pages, slots, positions and tree masks of a batch's new tokens, from the
// request lengths (tl_plan_batch).
//
// One launch.  Every CTA scans all request lengths (prefix sums of new tokens
// and of pages needed) into shared memory, so no CTA waits for another; what
// the scan needs is read only, and everything written is a different array or
// entry (the block table grows only past the entries that any CTA reads).  The
// CTAs then share the rows (one thread a row, its request found by binary
// search) and the requests (one warp each for the new table entries).
// Latency bound at serving sizes: the scan is R * 8 bytes from L2.  64 single
// tokens take 3.3 us, trees of up to 64 nodes for 200 requests 6.6 us (a node's
// mask is a walk up its parents, a cached load a step).
#include "common.cuh"
#include "host_util.h"

namespace tl {
namespace plan {

constexpr int kThreads = 256;
constexpr int kMaxR = 8192;
constexpr int kMaxWords = 8;
constexpr int kMaxFresh = 1 << 24;
constexpr int kMaxRows = 1 << 30;      // row indices are int, with room for a grid's stride behind them
constexpr int kMaxTreeRows = 1 << 20;  // a node's thread walks up all its ancestors
enum : int32_t { BAD_PARENT = TL_BAD_PARENT, BAD_LENGTH = TL_BAD_LENGTH };

struct Args {
  const int32_t *cached, *fresh;
  int32_t R, shift, max_pages;
  int32_t* table;
  const int32_t* free_pages;
  int32_t n_free;
  const int32_t* free_head;
  const int32_t* parents;
  int32_t n_rows, words;
  int32_t *cu, *lens, *granted, *free_head_out;
  int64_t* slots;
  int32_t* positions;
  uint32_t* masks;
  int32_t* status;
  int32_t pad;  // rows behind the batch: 1 written as rows of no token, 0 left as they are
};

struct Req {
  int32_t c, f;    // tokens held, new tokens (0 for bad lengths)
  int32_t held, need;
  bool ok;         // lengths valid and within the table row
  bool bad;
};

__device__ __forceinline__ Req request(const Args& a, int r) {
  Req q;
  const int c = a.cached[r], f = a.fresh[r], P = 1 << a.shift;
  q.bad = c < 0 || f < 0 || f > kMaxFresh || c > 0x7fffffff - kMaxFresh - P;
  q.c = q.bad ? 0 : c;
  q.f = q.bad ? 0 : f;
  q.held = (q.c + P - 1) >> a.shift;
  const int want = (q.c + q.f + P - 1) >> a.shift;
  const bool fits = want <= a.max_pages;
  q.need = fits && !q.bad ? want - q.held : 0;
  q.ok = fits && !q.bad;
  q.bad |= !fits;
  return q;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(Args a) {
  extern __shared__ int32_t sh[];
  int32_t* cu = sh;                // [R + 1]
  int32_t* off = sh + a.R + 1;     // [R] pages taken before the request; -1: refused
  __shared__ long long wsum[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long head = a.free_head[0];
  const bool head_ok = head >= 0 && head <= a.n_free;
  const long long avail = head_ok ? a.n_free - head : 0;
  long long rows = 0, pages = 0;
  long long taken_here = 0;  // pages granted (thread-local)
  int bad_any = head_ok ? 0 : BAD_LENGTH;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    Req q{0, 0, 0, 0, false, false};
    if (r < a.R) q = request(a, r);
    long long x = q.f, y = q.need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) { x += u; y += v; }
    }
    if (lane == 31) { wsum[0][warp] = x; wsum[1][warp] = y; }
    __syncthreads();
    long long bx = rows, by = pages;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) { bx += wsum[0][w]; by += wsum[1][w]; }
      rows += wsum[0][w];
      pages += wsum[1][w];
    }
    __syncthreads();
    if (r < a.R) {
      const long long first = bx + x - q.f, upto = by + y;  // rows before it; pages needed through it
      cu[r] = (int)min(first, 0x7fffffffll);
      const bool granted = q.ok && (q.need == 0 || upto <= avail);
      off[r] = granted ? (int)(upto - q.need) : -1;
      if (granted) taken_here += q.need;
      if (q.bad) bad_any |= BAD_LENGTH;
      if (blockIdx.x == 0) {
        a.cu[r] = cu[r];
        a.granted[r] = granted;
        a.lens[r] = granted ? q.c + q.f : a.cached[r];
      }
    }
  }
  const int total = (int)min(rows, 0x7fffffffll);
  if (threadIdx.x == 0) cu[a.R] = total;
  if (blockIdx.x == 0) {
    long long s = taken_here;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) wsum[0][warp] = s;
    if (total > a.n_rows) bad_any |= BAD_LENGTH;
    if (a.status && bad_any) atomicOr(a.status, bad_any);
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    long long s = 0;
    for (int w = 0; w < kThreads / 32; ++w) s += wsum[0][w];
    a.cu[a.R] = total;
    a.free_head_out[0] = (int)(head + s);
  }
  // the new entries of the block table: a warp a request
  for (int r = blockIdx.x * (kThreads / 32) + warp; r < a.R; r += gridDim.x * (kThreads / 32)) {
    if (off[r] < 0) continue;
    const Req q = request(a, r);
    for (int i = lane; i < q.need; i += 32)
      a.table[(int64_t)r * a.max_pages + q.held + i] = a.free_pages[head + off[r] + i];
  }
  // the rows
  int bad = 0;
  const int n = min(total, a.n_rows), upto = a.pad ? a.n_rows : n;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < upto; i += gridDim.x * kThreads) {
    if (i >= n) {
      a.slots[i] = -1;
      a.positions[i] = 0;
      for (int w = 0; a.masks && w < a.words; ++w) a.masks[(int64_t)i * a.words + w] = 0u;
      continue;
    }
    int lo = 0, hi = a.R;  // the last request with cu <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= i) lo = mid; else hi = mid;
    }
    const int r = lo, j = i - cu[r], nodes = cu[r + 1] - cu[r];
    const Req q = request(a, r);
    const int pos = q.c + j;
    int64_t slot = -1;
    if (off[r] >= 0) {
      const int pi = pos >> a.shift;
      const int page = pi < q.held ? a.table[(int64_t)r * a.max_pages + pi]
                                   : a.free_pages[head + off[r] + pi - q.held];
      if (page >= 0) slot = ((int64_t)page << a.shift) + (pos & ((1 << a.shift) - 1));
    }
    a.slots[i] = slot;
    int depth = j;
    if (a.parents) {
      uint32_t m[kMaxWords];
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w) m[w] = 0;
      depth = -1;
      for (int x = j; x >= 0;) {
        ++depth;
#pragma unroll
        for (int w = 0; w < kMaxWords; ++w)
          if (x >> 5 == w) m[w] |= 1u << (x & 31);
        const int p = a.parents[cu[r] + x];
        if (p < -1 || p >= x) { bad |= BAD_PARENT; break; }
        x = p;
      }
      if (a.masks) {
#pragma unroll
        for (int w = 0; w < kMaxWords; ++w)
          if (w < a.words) a.masks[(int64_t)i * a.words + w] = j < 32 * a.words ? m[w] : 0u;
      }
    } else if (a.masks) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        if (w < a.words) {
          const int k = j - 32 * w;  // bits 0 .. k of the word
          a.masks[(int64_t)i * a.words + w] =
              j >= 32 * a.words || k < 0 ? 0u : (k >= 31 ? 0xffffffffu : (2u << k) - 1u);
        }
    }
    a.positions[i] = q.c + depth;
    if (a.masks && nodes > 32 * a.words) bad |= BAD_LENGTH;
  }
  if (a.status && bad) atomicOr(a.status, bad);
}

static int plan_batch(bool pad, const int32_t* dev_cached, const int32_t* dev_fresh, int32_t R, int32_t page_tokens,
                      int32_t* dev_block_table, int32_t max_pages, const int32_t* dev_free_pages, int32_t n_free,
                      const int32_t* dev_free_head, const int32_t* dev_parents, int32_t n_rows, int32_t mask_words,
                      int32_t* dev_cu, int32_t* dev_lens, int32_t* dev_granted, int32_t* dev_free_head_out,
                      int64_t* dev_slots, int32_t* dev_positions, uint32_t* dev_masks, int32_t* dev_status,
                      void* cuda_stream) {
  if (R < 1 || R > plan::kMaxR || page_tokens < 1 || page_tokens > 4096 || (page_tokens & (page_tokens - 1)) ||
      max_pages < 1 || n_free < 0 || n_rows < 0 || n_rows > (dev_parents ? plan::kMaxTreeRows : plan::kMaxRows) ||
      mask_words < 0 || mask_words > plan::kMaxWords ||
      (mask_words > 0 ? !dev_masks && n_rows > 0 : dev_masks != nullptr))
    return TL_EINVAL;
  const void* need[] = {dev_cached, dev_fresh, dev_block_table, dev_free_head, dev_cu, dev_lens, dev_granted,
                        dev_free_head_out};
  for (const void* p : need)
    if (!p || ((uintptr_t)p & 3)) return TL_EINVAL;
  if ((n_free > 0 && !dev_free_pages) || (n_rows > 0 && (!dev_slots || !dev_positions))) return TL_EINVAL;
  if (((uintptr_t)dev_free_pages & 3) || ((uintptr_t)dev_slots & 7) || ((uintptr_t)dev_positions & 3) ||
      ((uintptr_t)dev_masks & 3) || ((uintptr_t)dev_parents & 3) || ((uintptr_t)dev_status & 3))
    return TL_EINVAL;
  // the CTAs read the inputs while others write: an output shares no byte with an input or another output
  const size_t nr = (size_t)n_rows, nR = (size_t)R;
  const Buf ins[] = {{dev_cached, 4 * nR}, {dev_fresh, 4 * nR}, {dev_free_pages, 4 * (size_t)n_free},
                     {dev_free_head, 4}, {dev_parents, 4 * nr}};
  const Buf outs[] = {{dev_block_table, 4 * nR * max_pages}, {dev_cu, 4 * nR + 4}, {dev_lens, 4 * nR},
                      {dev_granted, 4 * nR}, {dev_free_head_out, 4}, {dev_slots, 8 * nr}, {dev_positions, 4 * nr},
                      {dev_masks, 4 * nr * mask_words}, {dev_status, 4}};
  for (const Buf& o : outs) {
    for (const Buf& i : ins)
      if (share_bytes(o, i)) return TL_EINVAL;
    for (const Buf* q = &o + 1; q < outs + sizeof(outs) / sizeof(outs[0]); ++q)
      if (share_bytes(o, *q)) return TL_EINVAL;
  }
  plan::Args a{dev_cached, dev_fresh, R, 0, max_pages, dev_block_table, dev_free_pages, n_free, dev_free_head,
               dev_parents, n_rows, mask_words, dev_cu, dev_lens, dev_granted, dev_free_head_out, dev_slots,
               dev_positions, dev_masks, dev_status, pad};
  while ((1 << a.shift) < page_tokens) ++a.shift;
  const size_t smem = (size_t)(2 * R + 1) * 4;  // at most 64 KB
  if (smem > 46 * 1024)
    TL_CUDA(cudaFuncSetAttribute(plan::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  const int64_t by_rows = ((int64_t)n_rows + plan::kThreads - 1) / plan::kThreads;
  const int64_t by_req = ((int64_t)R + plan::kThreads / 32 - 1) / (plan::kThreads / 32);
  const int64_t grid = by_rows > by_req ? by_rows : by_req;
  plan::plan_kernel<<<(unsigned)(grid < 592 ? grid : 592), plan::kThreads, smem, (cudaStream_t)cuda_stream>>>(a);
  return check_cuda(cudaGetLastError());
}

}  // namespace plan
}  // namespace tl

extern "C" int tl_plan_batch(const int32_t* dev_cached, const int32_t* dev_fresh, int32_t R, int32_t page_tokens,
                             int32_t* dev_block_table, int32_t max_pages, const int32_t* dev_free_pages,
                             int32_t n_free, const int32_t* dev_free_head, const int32_t* dev_parents, int32_t n_rows,
                             int32_t mask_words, int32_t* dev_cu, int32_t* dev_lens, int32_t* dev_granted,
                             int32_t* dev_free_head_out, int64_t* dev_slots, int32_t* dev_positions,
                             uint32_t* dev_masks, int32_t* dev_status, void* cuda_stream) {
  return tl::plan::plan_batch(false, dev_cached, dev_fresh, R, page_tokens, dev_block_table, max_pages, dev_free_pages,
                              n_free, dev_free_head, dev_parents, n_rows, mask_words, dev_cu, dev_lens, dev_granted,
                              dev_free_head_out, dev_slots, dev_positions, dev_masks, dev_status, cuda_stream);
}

extern "C" int tl_plan_batch_padded(const int32_t* dev_cached, const int32_t* dev_fresh, int32_t R,
                                    int32_t page_tokens, int32_t* dev_block_table, int32_t max_pages,
                                    const int32_t* dev_free_pages, int32_t n_free, const int32_t* dev_free_head,
                                    const int32_t* dev_parents, int32_t n_rows, int32_t mask_words, int32_t* dev_cu,
                                    int32_t* dev_lens, int32_t* dev_granted, int32_t* dev_free_head_out,
                                    int64_t* dev_slots, int32_t* dev_positions, uint32_t* dev_masks,
                                    int32_t* dev_status, void* cuda_stream) {
  return tl::plan::plan_batch(true, dev_cached, dev_fresh, R, page_tokens, dev_block_table, max_pages, dev_free_pages,
                              n_free, dev_free_head, dev_parents, n_rows, mask_words, dev_cu, dev_lens, dev_granted,
                              dev_free_head_out, dev_slots, dev_positions, dev_masks, dev_status, cuda_stream);
}
