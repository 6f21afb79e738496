// Writing to a paged key-value cache and evicting from it.
//
// Both move whole (token, head) rows of d elements, so what bounds them is the
// bytes moved: 8 prompts of 5120 tokens x 8 heads of 128 are written in 52.7 us
// (97 % of the measured copy rate), and 524288 kept rows of 128 copied in 87
// (95 %).  The eviction first finds, per (request, key-value head), which
// positions stay: a selection by radix over the weights.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/onela.h"
#include "attention.h"
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
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
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

constexpr int kCand = 2048;       // positions in the threshold's first bin that a CTA lists

struct EvictSel {
  alignas(16) uint32_t hist[3][kBins];  // by digit
  uint32_t warp[kSelWarps];
  uint32_t above[kSelWarps], equal[kSelWarps];  // by warp: keys above the threshold, keys equal to it
  uint32_t totals[2];    // of the CTA, read by the cluster
  uint32_t found[3][2];  // by digit: the threshold's digits so far, and how many of its bin are wanted
  uint32_t ncand;
  int cand[kCand];
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
// Every CTA of the cluster takes one stretch of the positions and every warp
// a run of that.  The threshold is found digit by digit (11, 11 and 10 bits)
// from histograms of the keys that match so far, the cluster's added up through distributed
// shared memory, so that every CTA finds the same digit.
//
// 64 rows of 65500 positions take 27 us, two stretches of 16384 on an SM: a
// sixth each for the first digit's histogram, that digit, the list, the other
// two digits, the counts and the positions, most of them ended by a barrier of the
// cluster.  All keys are looked at three times only: when they are loaded (first
// digit), once to list the keys of the threshold's first bin (few, unless
// weights are nearly equal: then every key is looked at again) and count those
// above it, and to write the positions.  Positions past the row have key 0,
// the lowest (NaN's): they come last among equals, so want never reaches them.
// kBig: stretches beyond shared memory are read from the weights each time.
template <bool kBig>
__global__ void __launch_bounds__(kSel, 2) evict_select(CacheEvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ EvictSel sm;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int csize = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rh = blockIdx.x / csize, r = rh / p.Hkv, h = rh % p.Hkv;
  const int64_t cap = (int64_t)p.page * p.row_pages;
  const int given = p.lengths[r];
  const int len = given < 0 ? 0 : (given > cap ? (int)cap : given);
  const int n = min(len, p.keep), rec = min(p.recent, n), free_len = len - rec, want = n - rec;
  int32_t *kept = p.kept + (int64_t)rh * p.keep;
  if (h == 0 && rank == 0 && tid == 0) {
    p.dst_lengths[r] = n;
    if (given != len) flag(p.status, ONELA_STATUS_LENGTH);
  }
  for (int e = rank * kSel + tid; e < rec; e += csize * kSel) kept[want + e] = free_len + e;
  for (int e = n + rank * kSel + tid; e < p.keep; e += csize * kSel) kept[e] = -1;
  if (want == free_len) {  // all of them stay
    for (int e = rank * kSel + tid; e < want; e += csize * kSel) kept[e] = e;
    return;
  }
  if (want == 0) return;

  // Stretches of 32 runs of a multiple of 128: only the row's last one has positions that are not there.
  const int seg = ((free_len + csize - 1) / csize + 4095) / 4096 * 4096;
  const int s0 = min(free_len, rank * seg), sn = min(free_len, s0 + seg) - s0;
  const int run = ((sn + kSelWarps - 1) / kSelWarps + 127) / 128 * 128;  // positions of a warp
  const float *mine = p.mass + (int64_t)rh * cap + s0;
  const bool wide = (reinterpret_cast<uintptr_t>(mine) & 15) == 0;
  // Keys e .. e + 3 of the stretch, e a multiple of 4.
  auto fresh4 = [&](int e, uint32_t (&k)[4]) {
    if (wide && e + 4 <= sn) {
      const float4 v = *reinterpret_cast<const float4 *>(mine + e);
      k[0] = orderable(v.x);
      k[1] = orderable(v.y);
      k[2] = orderable(v.z);
      k[3] = orderable(v.w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = e + i < sn ? orderable(mine[e + i]) : 0u;
    }
  };
  auto keys4 = [&](int e, uint32_t (&k)[4]) {
    if constexpr (kBig) {
      fresh4(e, k);
    } else {
      const uint4 v = *reinterpret_cast<const uint4 *>(keys + e);
      k[0] = v.x;
      k[1] = v.y;
      k[2] = v.z;
      k[3] = v.w;
    }
  };
  auto sync = [&] {
    if (csize > 1) cluster.sync();
    else __syncthreads();
  };
  uint32_t prefix = 0, left = (uint32_t)want;
  // The digit of the threshold at `shift`, from the cluster's histograms: from
  // the top bin down, thread t takes bins nb - 1 - 2t and nb - 2 - 2t.
  auto find = [&](int pass, int shift, int nb) {
    const int b1 = nb - 2 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
    if (b1 >= 0) {
#pragma unroll 4
      for (int c = 0; c < csize; ++c) {
        const uint2 v = *reinterpret_cast<const uint2 *>(
            csize > 1 ? cluster.map_shared_rank(&sm.hist[pass][b1], c) : &sm.hist[pass][b1]);
        c0 += v.y;
        c1 += v.x;
      }
    }
    const uint32_t above = block_scan(c0 + c1, sm.warp);
    if (above < left && left <= above + c0 + c1) {  // exactly one thread
      const bool second = left > above + c0;
      sm.found[pass][0] = prefix | ((uint32_t)(second ? b1 : b1 + 1) << shift);
      sm.found[pass][1] = left - above - (second ? c0 : 0);
    }
    __syncthreads();
    prefix = sm.found[pass][0];
    left = sm.found[pass][1];
  };
  for (int e = tid; e < 3 * kBins / 4; e += kSel) reinterpret_cast<uint4 *>(sm.hist)[e] = make_uint4(0, 0, 0, 0);
  if (tid == 0) sm.ncand = 0;
  __syncthreads();
  const int w0 = warp * run + 4 * lane, w1 = (warp + 1) * run;  // this lane's keys: w0, w0 + 128, ... four each
#pragma unroll 4
  for (int e = w0; e < w1; e += 128) {
    uint32_t k[4];
    fresh4(e, k);
    if (!kBig) *reinterpret_cast<uint4 *>(keys + e) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) atomicAdd(&sm.hist[0][k[i] >> 21], 1u);
  }
  sync();
  find(0, 21, 2048);
  uint32_t g = 0, q = 0;
#pragma unroll 1
  for (int e = w0; e < w1; e += 128) {
    uint32_t k[4];
    keys4(e, k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t d = k[i] >> 21;
      g += d > prefix >> 21;
      if (d == prefix >> 21) {
        atomicAdd(&sm.hist[1][(k[i] >> 10) & 2047u], 1u);
        const uint32_t at = atomicAdd(&sm.ncand, 1u);
        if (at < kCand) sm.cand[at] = e + i;
      }
    }
  }
  sync();
  const uint32_t ncand = sm.ncand;
  const bool listed = ncand <= kCand;
  auto key_of = [&](int e) { return kBig ? orderable(mine[e]) : keys[e]; };  // of a listed position
  find(1, 10, 2048);
  if (listed) {
    for (uint32_t c = tid; c < ncand; c += kSel) {
      const int e = sm.cand[c];
      const uint32_t key = e < sn ? key_of(e) : 0u;
      if (((key ^ prefix) >> 10) == 0) atomicAdd(&sm.hist[2][key & 1023u], 1u);
    }
  } else {
#pragma unroll 1
    for (int e = w0; e < w1; e += 128) {
      uint32_t k[4];
      keys4(e, k);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (((k[i] ^ prefix) >> 10) == 0) atomicAdd(&sm.hist[2][k[i] & 1023u], 1u);
    }
  }
  sync();
  find(2, 0, 1024);
  const uint32_t thr = prefix, ties = left;
  // Keys above and equal, by warp; then those of the warps and CTAs before.
  if (!listed) {
    g = 0;
#pragma unroll 1
    for (int e = w0; e < w1; e += 128) {
      uint32_t k[4];
      keys4(e, k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g += k[i] > thr;
        q += k[i] == thr;
      }
    }
  }
  g = __reduce_add_sync(0xffffffffu, g);
  q = __reduce_add_sync(0xffffffffu, q);
  if (lane == 0) {
    sm.above[warp] = g;
    sm.equal[warp] = q;
  }
  __syncthreads();
  if (listed) {
    for (uint32_t c = tid; c < ncand; c += kSel) {
      const int e = sm.cand[c];
      const uint32_t key = e < sn ? key_of(e) : 0u;
      if (key > thr) atomicAdd(&sm.above[e / run], 1u);
      if (key == thr) atomicAdd(&sm.equal[e / run], 1u);
    }
    __syncthreads();
  }
  uint32_t gb = sm.above[lane], qb = sm.equal[lane];
  if (csize > 1) {
    const uint32_t g_all = __reduce_add_sync(0xffffffffu, gb), q_all = __reduce_add_sync(0xffffffffu, qb);
    if (tid == 0) {
      sm.totals[0] = g_all;
      sm.totals[1] = q_all;
    }
  }
  gb = __reduce_add_sync(0xffffffffu, lane < warp ? gb : 0);
  qb = __reduce_add_sync(0xffffffffu, lane < warp ? qb : 0);
  if (csize > 1) {
    cluster.sync();
    const uint32_t *other = cluster.map_shared_rank(sm.totals, lane < rank ? lane : rank);
    gb += __reduce_add_sync(0xffffffffu, lane < rank ? other[0] : 0);
    qb += __reduce_add_sync(0xffffffffu, lane < rank ? other[1] : 0);
  }
#pragma unroll 1
  for (int e = w0; e < w1; e += 128) {
    uint32_t k[4], mine2 = 0;  // above in the low half, equal in the high half
    keys4(e, k);
#pragma unroll
    for (int i = 0; i < 4; ++i) mine2 += (k[i] > thr ? 1u : 0u) + (k[i] == thr ? 0x10000u : 0u);
    if (__any_sync(0xffffffffu, mine2)) {
      uint32_t incl = mine2;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const uint32_t before = incl - mine2, all2 = __shfl_sync(0xffffffffu, incl, 31);
      if (mine2) {
        uint32_t gi = gb + (before & 0xffffu), qi = qb + (before >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k[i] > thr) kept[gi++ + min(qi, ties)] = s0 + e + i;
          else if (k[i] == thr) {
            if (qi < ties) kept[gi + qi] = s0 + e + i;
            ++qi;
          }
        }
      }
      gb += all2 & 0xffffu;
      qb += all2 >> 16;
    }
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
  ptx::pdl_launch_dependents();
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
  ptx::pdl_launch_dependents();
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

template <typename F, typename P>
cudaError_t launch_pdl(F *f, int64_t grid, const P &p, cudaStream_t s) {
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_kernel(f, (unsigned)grid, 256, 0, true, s, p);
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
  if (u == 16) return launch_pdl(cache_write<uint4>, grid, p, s);
  if (u == 8) return launch_pdl(cache_write<uint2>, grid, p, s);
  if (u == 4) return launch_pdl(cache_write<uint32_t>, grid, p, s);
  return launch_pdl(cache_write<uint16_t>, grid, p, s);
}

cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s) {
  // CTAs per (request, head): as many as keep the row's keys in shared memory, up to 8.
  const int64_t cap = (int64_t)p.page * p.row_pages;
  int csize = 1;
  while (csize < 8 && (int64_t)csize * kSelKeys < cap) csize *= 2;
  const int64_t stretch = ((cap + csize - 1) / csize + 4095) / 4096 * 4096;
  const bool big = stretch > kSelKeys;
  const int64_t sel_grid = (int64_t)p.R * p.Hkv * csize;
  if (sel_grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit((const void *)evict_select<false>, kSelKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sel_grid);
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = big ? 0 : (size_t)stretch * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, big ? evict_select<true> : evict_select<false>, p);
  if (e != cudaSuccess) return e;
  const uint64_t all = addr(p.dst_k) | addr(p.dst_v) | addr(p.k_pool) | addr(p.v_pool) | (uint64_t)p.row_bytes;
  const int u = unit_of(all), per_row = p.row_bytes / u;
  const int64_t rows = (int64_t)p.R * p.Hkv;
  if (u == 16 && per_row >= 4 && per_row <= 64 && (per_row & (per_row - 1)) == 0) {
    const int64_t grid = (rows * ((p.keep + 7) / 8) + 7) / 8;
    if (per_row == 4) return launch_pdl(evict_copy_rows<2>, grid, p, s);
    if (per_row == 8) return launch_pdl(evict_copy_rows<3>, grid, p, s);
    if (per_row == 16) return launch_pdl(evict_copy_rows<4>, grid, p, s);
    if (per_row == 32) return launch_pdl(evict_copy_rows<5>, grid, p, s);
    return launch_pdl(evict_copy_rows<6>, grid, p, s);
  }
  const int64_t grid = (rows * per_row * p.keep + 255) / 256;
  if (u == 16) return launch_pdl(evict_copy<uint4>, grid, p, s);
  if (u == 8) return launch_pdl(evict_copy<uint2>, grid, p, s);
  if (u == 4) return launch_pdl(evict_copy<uint32_t>, grid, p, s);
  return launch_pdl(evict_copy<uint16_t>, grid, p, s);
}

}  // namespace onela
