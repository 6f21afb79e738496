// Writing to a paged key-value cache and evicting from it.
//
// Both move whole (token, head) rows of d elements, so what bounds them is the
// bytes moved; the eviction first finds, per (request, key-value head), which
// positions stay: a selection by radix over the weights.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/onela.h"
#include "cache.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

__device__ __forceinline__ void flag(int32_t *status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------- write
// A thread per unit of V bytes of one (token, head) row: rows are contiguous on both
// sides, V is the widest unit (16, 8, 4 or 2 bytes) that every row start allows.
template <typename U>
__global__ void __launch_bounds__(256) cache_write(CacheWriteParams p) {
  const int per_row = p.row_bytes / (int)sizeof(U);           // units in one (token, head) row
  const int64_t per_tok = (int64_t)per_row * p.Hkv;
  const int64_t total = per_tok * p.n * p.B;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t tok = i / per_tok;
  const int in = (int)(i - tok * per_tok), h = in / per_row, c = in - h * per_row;
  const int b = (int)(tok / p.n), j = (int)(tok - (int64_t)b * p.n);
  if (p.counts && j >= p.counts[b]) {
    if (in == 0 && j == 0 && p.counts[b] < 0) flag(p.status, ONELA_STATUS_LENGTH);
    return;
  }
  const bool lead = in == 0;
  if (p.counts && j == 0 && lead && p.counts[b] > p.n) flag(p.status, ONELA_STATUS_LENGTH);
  const int64_t pos = (int64_t)p.start[b] + j;
  if (pos < 0 || pos >= (int64_t)p.page * p.row_pages) {
    if (lead) flag(p.status, ONELA_STATUS_LENGTH);
    return;
  }
  const int pg = p.table[(int64_t)b * p.row_pages + pos / p.page];
  if (pg < 0 || pg >= p.pages) {
    if (lead) flag(p.status, ONELA_STATUS_PAGE);
    return;
  }
  const int64_t dst = (((int64_t)pg * p.Hkv + h) * p.page + pos % p.page) * per_row + c;
  const U kk = *(reinterpret_cast<const U *>(static_cast<const uint8_t *>(p.k) + tok * p.k_stride) + in);
  const U vv = *(reinterpret_cast<const U *>(static_cast<const uint8_t *>(p.v) + tok * p.v_stride) + in);
  reinterpret_cast<U *>(p.k_pool)[dst] = kk;
  reinterpret_cast<U *>(p.v_pool)[dst] = vv;
}

// ------------------------------------------------------------------- evict
__device__ __forceinline__ uint32_t orderable(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN: below everything
  if (u == 0x80000000u) u = 0u;                     // -0 equals +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSel = 1024;   // threads of the selection
constexpr int kBins = 2048;  // 11 bits at a time: 11 + 11 + 10

struct EvictSel {
  uint32_t hist[kBins];
  uint32_t warp[kSel / 32];
  uint32_t prefix, want, run;
  int done;
};

// Block-wide exclusive sum of x; the total in `total`.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *warp_sums, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const uint32_t before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
  return before + incl - x;
}

// One CTA per (request, head): the positions that stay, in order, to kept.
// The threshold is the want-th largest key of the positions before the recent
// ones; keys above it stay, and the first keys equal to it until want is met.
__global__ void __launch_bounds__(kSel) evict_select(CacheEvictParams p) {
  __shared__ EvictSel sm;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rh = blockIdx.x, r = rh / p.Hkv, h = rh % p.Hkv;
  const int64_t cap = (int64_t)p.page * p.row_pages;
  const int given = p.lengths[r];
  const int len = given < 0 ? 0 : (given > cap ? (int)cap : given);
  const int n = min(len, p.keep), rec = min(p.recent, n), free_len = len - rec, want = n - rec;
  const float *mass = p.mass + (int64_t)rh * cap;
  int32_t *kept = p.kept + (int64_t)rh * p.keep;
  if (h == 0 && tid == 0) {
    p.dst_lengths[r] = n;
    if (given != len) flag(p.status, ONELA_STATUS_LENGTH);
  }
  ptx::pdl_launch_dependents();
  if (tid == 0) {
    sm.prefix = 0;
    sm.want = (uint32_t)want;
    sm.done = want == free_len || want == 0;
  }
  __syncthreads();
  const bool all = want == free_len;
  uint32_t mask = 0;
  int shift = 21, bits = 11;
  for (int pass = 0; pass < 3 && !sm.done; ++pass) {
    for (int e = tid; e < kBins; e += kSel) sm.hist[e] = 0;
    __syncthreads();
    const uint32_t prefix = sm.prefix, digit = (1u << bits) - 1u;
    for (int e = tid; e < free_len; e += kSel) {
      const uint32_t key = orderable(mass[e]);
      if ((key & mask) == prefix) atomicAdd(&sm.hist[(key >> shift) & digit], 1u);
    }
    __syncthreads();
    // From the top bin down: thread t takes bins nb - 1 - 2t and nb - 2 - 2t.
    const int nb = 1 << bits;
    const int b0 = nb - 1 - 2 * tid;
    const uint32_t c0 = b0 >= 0 ? sm.hist[b0] : 0, c1 = b0 >= 1 ? sm.hist[b0 - 1] : 0;
    uint32_t total;
    const uint32_t above = block_scan(c0 + c1, sm.warp, total);
    const uint32_t w = sm.want;
    __syncthreads();
    if (above < w && w <= above + c0 + c1) {  // exactly one thread
      const bool second = w > above + c0;
      sm.prefix = prefix | ((uint32_t)(second ? b0 - 1 : b0) << shift);
      sm.want = w - above - (second ? c0 : 0);
    }
    __syncthreads();
    mask |= digit << shift;
    const int next = pass == 0 ? 11 : 10;
    shift -= next;
    bits = next;
  }
  // Two running counts over the positions: keys above the threshold, and keys
  // equal to it (of which the first `ties` stay).
  const uint32_t thr = sm.prefix, ties = sm.want;
  uint32_t above_run = 0, eq_run = 0;
  for (int e0 = 0; e0 < free_len && want > 0; e0 += kSel) {
    const int e = e0 + tid;
    const uint32_t key = e < free_len ? orderable(mass[e]) : 0u;
    const uint32_t gt = e < free_len && (all || key > thr), eq = e < free_len && !all && key == thr;
    uint32_t total;
    const uint32_t pre = block_scan(gt | (eq << 16), sm.warp, total);
    const uint32_t g = above_run + (pre & 0xffffu), q = eq_run + (pre >> 16);
    if (gt || (eq && q < ties)) kept[g + min(q, ties)] = e;
    above_run += total & 0xffffu;
    eq_run += total >> 16;
  }
  for (int e = tid; e < rec; e += kSel) kept[want + e] = free_len + e;
  for (int e = n + tid; e < p.keep; e += kSel) kept[e] = -1;
  (void)lane;
}

// Copies the kept tokens: a thread per unit of V bytes of a kept (token, head) row.
template <typename U>
__global__ void __launch_bounds__(256) evict_copy(CacheEvictParams p) {
  ptx::pdl_wait();
  const int per_row = p.row_bytes / (int)sizeof(U);
  const int64_t per_rh = (int64_t)per_row * p.keep;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= per_rh * p.R * p.Hkv) return;
  const int rh = (int)(i / per_rh);
  const int64_t in = i - rh * per_rh;
  const int j = (int)(in / per_row), c = (int)(in - (int64_t)j * per_row);
  const int r = rh / p.Hkv, h = rh % p.Hkv;
  const int pos = p.kept[(int64_t)rh * p.keep + j];
  if (pos < 0) return;
  const int64_t cap = (int64_t)p.page * p.row_pages;
  if (c == 0) p.dst_mass[(int64_t)rh * p.page * p.dst_row_pages + j] = p.mass[rh * cap + pos];
  const int dp = p.dst_table[(int64_t)r * p.dst_row_pages + j / p.page];
  const int sp = p.table[(int64_t)r * p.row_pages + pos / p.page];
  if (dp < 0 || dp >= p.dst_pages || sp < 0 || sp >= p.pages) {
    if (c == 0) flag(p.status, ONELA_STATUS_PAGE);
    if (dp < 0 || dp >= p.dst_pages) return;
  }
  U kk = {}, vv = {};
  if (sp >= 0 && sp < p.pages) {
    const int64_t src = (((int64_t)sp * p.Hkv + h) * p.page + pos % p.page) * per_row + c;
    kk = reinterpret_cast<const U *>(p.k_pool)[src];
    vv = reinterpret_cast<const U *>(p.v_pool)[src];
  }
  const int64_t dst = (((int64_t)dp * p.Hkv + h) * p.page + j % p.page) * per_row + c;
  reinterpret_cast<U *>(p.dst_k)[dst] = kk;
  reinterpret_cast<U *>(p.dst_v)[dst] = vv;
}

// The widest unit of 16, 8, 4 or 2 bytes that divides x.
int unit_of(uint64_t x) { return x % 16 == 0 ? 16 : (x % 8 == 0 ? 8 : (x % 4 == 0 ? 4 : 2)); }
template <typename P>
uint64_t addr(const P *p) {
  return reinterpret_cast<uintptr_t>(p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams &p, cudaStream_t s) {
  const uint64_t all = addr(p.k) | addr(p.v) | addr(p.k_pool) | addr(p.v_pool) | (uint64_t)p.row_bytes |
                       (uint64_t)p.k_stride | (uint64_t)p.v_stride;
  const int u = unit_of(all);
  const int64_t units = (int64_t)p.row_bytes / u * p.Hkv * p.n * p.B;
  const int64_t grid = (units + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (u == 16) cache_write<uint4><<<(unsigned)grid, 256, 0, s>>>(p);
  else if (u == 8) cache_write<uint2><<<(unsigned)grid, 256, 0, s>>>(p);
  else if (u == 4) cache_write<uint32_t><<<(unsigned)grid, 256, 0, s>>>(p);
  else cache_write<uint16_t><<<(unsigned)grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s) {
  evict_select<<<(unsigned)(p.R * p.Hkv), kSel, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const uint64_t all = addr(p.dst_k) | addr(p.dst_v) | addr(p.k_pool) | addr(p.v_pool) | (uint64_t)p.row_bytes;
  const int u = unit_of(all);
  const int64_t units = (int64_t)p.row_bytes / u * p.keep * p.R * p.Hkv;
  const int64_t grid = (units + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (u == 16) return cudaLaunchKernelEx(&cfg, evict_copy<uint4>, p);
  if (u == 8) return cudaLaunchKernelEx(&cfg, evict_copy<uint2>, p);
  if (u == 4) return cudaLaunchKernelEx(&cfg, evict_copy<uint32_t>, p);
  return cudaLaunchKernelEx(&cfg, evict_copy<uint16_t>, p);
}

}  // namespace onela
