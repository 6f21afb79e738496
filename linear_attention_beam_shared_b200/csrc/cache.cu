// Writing to a paged key-value cache and evicting from it.
//
// Both move whole (token, head) rows of d elements, so what bounds them is the
// bytes moved; the eviction first finds, per (request, key-value head), which
// positions stay: a selection by radix over the weights.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/onela.h"
#include "cache.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace cg = cooperative_groups;

namespace onela {
namespace {

__device__ __forceinline__ void flag(int32_t *status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------- write
// A CTA moves 512 units of K and of V, two of each per thread, all four loads
// under way at once.  A unit is the widest of 16, 8, 4 and 2 bytes that every
// row start allows; (token, head) rows are contiguous on both sides.
template <typename U>
__global__ void __launch_bounds__(256) cache_write(CacheWriteParams p) {
  const int per_row = p.row_bytes / (int)sizeof(U);  // units of a (token, head) row
  const int per_tok = per_row * p.Hkv;
  const int64_t i0 = (int64_t)blockIdx.x * 512, tok0 = i0 / per_tok;
  const int skip = (int)(i0 - tok0 * per_tok);
  U kk[2], vv[2];
  int64_t dst[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    dst[e] = -1;
    const int o = skip + e * 256 + (int)threadIdx.x, t = o / per_tok, in = o - t * per_tok;
    const int64_t tok = tok0 + t;
    if (tok >= (int64_t)p.B * p.n) continue;
    const int b = (int)((uint32_t)tok / (uint32_t)p.n), j = (int)tok - b * p.n;  // B * n fits 31 bits
    const bool lead = in == 0;
    if (p.counts) {
      const int given = p.counts[b];
      if (lead && j == 0 && (given < 0 || given > p.n)) flag(p.status, ONELA_STATUS_LENGTH);
      if (j >= given) continue;
    }
    const int64_t pos = (int64_t)p.start[b] + j;
    if (pos < 0 || pos >= (int64_t)p.page * p.row_pages) {
      if (lead) flag(p.status, ONELA_STATUS_LENGTH);
      continue;
    }
    const int q = (int)pos / p.page;  // rows hold at most 2^30 positions
    const int pg = p.table[(int64_t)b * p.row_pages + q];
    if (pg < 0 || pg >= p.pages) {
      if (lead) flag(p.status, ONELA_STATUS_PAGE);
      continue;
    }
    const int h = in / per_row;
    dst[e] = (((int64_t)pg * p.Hkv + h) * p.page + ((int)pos - q * p.page)) * per_row + (in - h * per_row);
    kk[e] = *(reinterpret_cast<const U *>(static_cast<const uint8_t *>(p.k) + tok * p.k_stride) + in);
    vv[e] = *(reinterpret_cast<const U *>(static_cast<const uint8_t *>(p.v) + tok * p.v_stride) + in);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (dst[e] >= 0) {
      reinterpret_cast<U *>(p.k_pool)[dst[e]] = kk[e];
      reinterpret_cast<U *>(p.v_pool)[dst[e]] = vv[e];
    }
}

// ------------------------------------------------------------------- evict
__device__ __forceinline__ uint32_t orderable(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN: below everything
  if (u == 0x80000000u) u = 0u;                     // -0 equals +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSel = 1024;        // threads of the selection
constexpr int kSelWarps = kSel / 32;
constexpr int kBins = 2048;       // 11 bits at a time: 11 + 11 + 10
constexpr int kSelKeys = 16384;   // keys of its stretch that a CTA keeps in shared memory (64 KB: two CTAs per SM)

struct EvictSel {
  uint32_t hist[3][kBins];  // by pass
  uint32_t warp[kSelWarps];
  uint32_t above[kSelWarps], equal[kSelWarps];  // by warp: keys above the threshold, keys equal to it
  uint32_t totals[2];       // of the CTA, read by the cluster
  uint32_t prefix, want;
};

// Block-wide exclusive sum of x.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *warp_sums) {
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
  const uint32_t before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  return (warp ? before : 0) + incl - x;
}

// One cluster per (request, head): the positions that stay, in order, to kept.
// The threshold is the want-th largest key of the positions before the recent
// ones; keys above it stay, and the first keys equal to it until want is met.
// Every CTA of the cluster takes one stretch of the positions: three passes
// over its keys build histograms of the digits that still match, the cluster's
// histograms are added through distributed shared memory, and every CTA finds
// the same digit.  Then each warp counts and writes a run of positions of its
// own, so that no barrier sits inside the loops.
__global__ void __launch_bounds__(kSel, 2) evict_select(CacheEvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ EvictSel sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int csize = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rh = blockIdx.x / csize, r = rh / p.Hkv, h = rh % p.Hkv;
  const int64_t cap = (int64_t)p.page * p.row_pages;
  const int given = p.lengths[r];
  const int len = given < 0 ? 0 : (given > cap ? (int)cap : given);
  const int n = min(len, p.keep), rec = min(p.recent, n), free_len = len - rec, want = n - rec;
  const float *mass = p.mass + (int64_t)rh * cap;
  int32_t *kept = p.kept + (int64_t)rh * p.keep;
  if (h == 0 && rank == 0 && tid == 0) {
    p.dst_lengths[r] = n;
    if (given != len) flag(p.status, ONELA_STATUS_LENGTH);
  }
  ptx::pdl_launch_dependents();
  for (int e = rank * kSel + tid; e < rec; e += csize * kSel) kept[want + e] = free_len + e;
  for (int e = n + rank * kSel + tid; e < p.keep; e += csize * kSel) kept[e] = -1;
  if (want == free_len) {  // all of them stay
    for (int e = rank * kSel + tid; e < want; e += csize * kSel) kept[e] = e;
    return;
  }
  if (want == 0) return;

  const int seg = ((free_len + csize - 1) / csize + kSel - 1) / kSel * kSel;
  const int s0 = min(free_len, rank * seg), sn = min(free_len, s0 + seg) - s0;
  const float *mine = mass + s0;
  const int in_smem = min(sn, kSelKeys);
  auto key_at = [&](int e) { return e < in_smem ? keys[e] : orderable(mine[e]); };
  for (int e = tid; e < 3 * kBins; e += kSel) sm.hist[0][e] = 0;
  if (tid == 0) {
    sm.prefix = 0;
    sm.want = (uint32_t)want;
  }
  __syncthreads();
  uint32_t mask = 0;
  int shift = 21, bits = 11;
  for (int pass = 0; pass < 3; ++pass) {
    const uint32_t prefix = sm.prefix, digit = (1u << bits) - 1u;
    uint32_t *hist = sm.hist[pass];
    auto count = [&](uint32_t key) {
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1u);
    };
    int e = tid;
    for (; e + 7 * kSel < sn; e += 8 * kSel) {
      uint32_t key[8];
      if (pass == 0) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = mine[e + i * kSel];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          key[i] = orderable(f[i]);
          if (e + i * kSel < in_smem) keys[e + i * kSel] = key[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) key[i] = key_at(e + i * kSel);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) count(key[i]);
    }
    for (; e < sn; e += kSel) {
      const uint32_t key = pass == 0 ? orderable(mine[e]) : key_at(e);
      if (pass == 0 && e < in_smem) keys[e] = key;
      count(key);
    }
    if (csize > 1) cluster.sync();
    else __syncthreads();
    // From the top bin down: thread t takes bins nb - 1 - 2t and nb - 2 - 2t of all CTAs.
    const int b0 = (1 << bits) - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
    if (b0 >= 1)
      for (int c = 0; c < csize; ++c) {
        const uint32_t *other = csize > 1 ? cluster.map_shared_rank(hist, c) : hist;
        c0 += other[b0];
        c1 += other[b0 - 1];
      }
    const uint32_t above = block_scan(c0 + c1, sm.warp);
    const uint32_t w = sm.want;
    __syncthreads();
    if (above < w && w <= above + c0 + c1) {  // exactly one thread
      const bool second = w > above + c0;
      sm.prefix = prefix | ((uint32_t)(second ? b0 - 1 : b0) << shift);
      sm.want = w - above - (second ? c0 : 0);
    }
    __syncthreads();
    mask |= digit << shift;
    bits = pass == 0 ? 11 : 10;
    shift -= bits;
  }
  const uint32_t thr = sm.prefix, ties = sm.want;
  // Each warp has a run of positions; its keys above and equal, then those of
  // the warps and CTAs before it.
  const int run = ((sn + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(sn, warp * run), w1 = min(sn, w0 + run);
  uint32_t g = 0, q = 0;
  for (int e = w0 + lane; e < w1; e += 32) {
    const uint32_t key = key_at(e);
    g += key > thr;
    q += key == thr;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    g += __shfl_xor_sync(0xffffffffu, g, o);
    q += __shfl_xor_sync(0xffffffffu, q, o);
  }
  if (lane == 0) {
    sm.above[warp] = g;
    sm.equal[warp] = q;
  }
  __syncthreads();
  uint32_t gb = sm.above[lane], qb = sm.equal[lane];
  const uint32_t g_all = __reduce_add_sync(0xffffffffu, gb), q_all = __reduce_add_sync(0xffffffffu, qb);
  gb = __reduce_add_sync(0xffffffffu, lane < warp ? gb : 0);
  qb = __reduce_add_sync(0xffffffffu, lane < warp ? qb : 0);
  if (csize > 1) {
    if (tid == 0) {
      sm.totals[0] = g_all;
      sm.totals[1] = q_all;
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const uint32_t *other = cluster.map_shared_rank(sm.totals, c);
      gb += other[0];
      qb += other[1];
    }
  }
  for (int e0 = w0; e0 < w1; e0 += 32) {
    const int e = e0 + lane;
    const uint32_t key = e < w1 ? key_at(e) : 0u;
    const bool is_g = e < w1 && key > thr, is_q = e < w1 && key == thr;
    const uint32_t mg = __ballot_sync(0xffffffffu, is_g), mq = __ballot_sync(0xffffffffu, is_q), below = (1u << lane) - 1u;
    const uint32_t gi = gb + __popc(mg & below), qi = qb + __popc(mq & below);
    if (is_g || (is_q && qi < ties)) kept[gi + min(qi, ties)] = s0 + e;
    gb += __popc(mg);
    qb += __popc(mq);
  }
  if (csize > 1) cluster.sync();  // the others have read this CTA's totals
}

// Copies the kept tokens.  A warp takes 8 kept positions of a (request, head):
// their places are looked up by 8 lanes, then the rows of K and of V move in
// 16-byte units with 8 loads under way per lane.  kLog: log2 of the
// units in a row.
template <int kLog>
__global__ void __launch_bounds__(256) evict_copy_rows(CacheEvictParams p) {
  ptx::pdl_wait();
  const int lane = threadIdx.x & 31;
  const int groups = (p.keep + 7) / 8;
  const int64_t wid = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (wid >= (int64_t)groups * p.R * p.Hkv) return;
  const int rh = (int)(wid / groups), j0 = (int)(wid - (int64_t)rh * groups) * 8;
  const int r = rh / p.Hkv, h = rh % p.Hkv;
  int64_t src = -1, dst = -1;  // first unit of this lane's row
  if (lane < 8 && j0 + lane < p.keep) {
    const int j = j0 + lane, pos = p.kept[(int64_t)rh * p.keep + j];
    if (pos >= 0) {
      const int64_t cap = (int64_t)p.page * p.row_pages;
      p.dst_mass[(int64_t)rh * p.page * p.dst_row_pages + j] = p.mass[rh * cap + pos];
      const int dp = p.dst_table[(int64_t)r * p.dst_row_pages + j / p.page];
      const int sp = p.table[(int64_t)r * p.row_pages + pos / p.page];
      const bool dok = dp >= 0 && dp < p.dst_pages, sok = sp >= 0 && sp < p.pages;
      if (!dok || !sok) flag(p.status, ONELA_STATUS_PAGE);
      if (dok) dst = (((int64_t)dp * p.Hkv + h) * p.page + j % p.page) << kLog;
      if (sok) src = (((int64_t)sp * p.Hkv + h) * p.page + pos % p.page) << kLog;
    }
  }
  constexpr int kSteps = (8 << kLog) / 32;             // of K, and of V
  constexpr int kBatch = kSteps < 4 ? kSteps : 4;      // of each at once
  const uint4 *ks = static_cast<const uint4 *>(p.k_pool), *vs = static_cast<const uint4 *>(p.v_pool);
  uint4 *kd = static_cast<uint4 *>(p.dst_k), *vd = static_cast<uint4 *>(p.dst_v);
#pragma unroll
  for (int e0 = 0; e0 < kSteps; e0 += kBatch) {
    uint4 kk[kBatch], vv[kBatch];
    int64_t to[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int at = (e0 + e) * 32 + lane, row = at >> kLog, c = at & ((1 << kLog) - 1);
      const int64_t s = __shfl_sync(0xffffffffu, src, row), d = __shfl_sync(0xffffffffu, dst, row);
      to[e] = d < 0 ? -1 : d + c;
      kk[e] = vv[e] = make_uint4(0, 0, 0, 0);
      if (s >= 0 && d >= 0) {
        kk[e] = __ldcs(ks + s + c);
        vv[e] = __ldcs(vs + s + c);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (to[e] >= 0) {
        kd[to[e]] = kk[e];
        vd[to[e]] = vv[e];
      }
  }
}

// The same for rows of any length: a thread per unit of a kept (token, head) row.
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

template <typename F>
cudaError_t launch_after(F *f, int64_t grid, const CacheEvictParams &p, cudaStream_t s) {
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
  return cudaLaunchKernelEx(&cfg, f, p);
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
  const int64_t grid = (units + 511) / 512;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (u == 16) cache_write<uint4><<<(unsigned)grid, 256, 0, s>>>(p);
  else if (u == 8) cache_write<uint2><<<(unsigned)grid, 256, 0, s>>>(p);
  else if (u == 4) cache_write<uint32_t><<<(unsigned)grid, 256, 0, s>>>(p);
  else cache_write<uint16_t><<<(unsigned)grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s) {
  // CTAs per (request, head): as many as keep the row's keys in shared memory, up to 8.
  const int64_t cap = (int64_t)p.page * p.row_pages;
  int csize = 1;
  while (csize < 8 && (int64_t)csize * kSelKeys < cap) csize *= 2;
  const int64_t per = std::min<int64_t>(kSelKeys, (cap + csize - 1) / csize + kSel);
  const int64_t sel_grid = (int64_t)p.R * p.Hkv * csize;
  if (sel_grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit((const void *)evict_select, kSelKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sel_grid);
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = (size_t)per * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select, p);
  if (e != cudaSuccess) return e;
  const uint64_t all = addr(p.dst_k) | addr(p.dst_v) | addr(p.k_pool) | addr(p.v_pool) | (uint64_t)p.row_bytes;
  const int u = unit_of(all), per_row = p.row_bytes / u;
  const int64_t rows = (int64_t)p.R * p.Hkv;
  if (u == 16 && per_row >= 4 && per_row <= 64 && (per_row & (per_row - 1)) == 0) {
    const int64_t grid = (rows * ((p.keep + 7) / 8) + 7) / 8;
    if (per_row == 4) return launch_after(evict_copy_rows<2>, grid, p, s);
    if (per_row == 8) return launch_after(evict_copy_rows<3>, grid, p, s);
    if (per_row == 16) return launch_after(evict_copy_rows<4>, grid, p, s);
    if (per_row == 32) return launch_after(evict_copy_rows<5>, grid, p, s);
    return launch_after(evict_copy_rows<6>, grid, p, s);
  }
  const int64_t grid = (rows * per_row * p.keep + 255) / 256;
  if (u == 16) return launch_after(evict_copy<uint4>, grid, p, s);
  if (u == 8) return launch_after(evict_copy<uint2>, grid, p, s);
  if (u == 4) return launch_after(evict_copy<uint32_t>, grid, p, s);
  return launch_after(evict_copy<uint16_t>, grid, p, s);
}

}  // namespace onela
