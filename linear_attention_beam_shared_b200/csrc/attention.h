// Internal declarations of the attention over a paged key-value cache: the
// parameters every kernel takes, the division of the prompts into units of
// work, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

namespace onela {

constexpr int kAttnSMs = 148;         // multiprocessors the units are spread over
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One call.  A (request, key-value head) has M = W * G query rows, row m
// being head m % G of the group of beam m / G.  Scores and their maxima are kept
// as the products q.k come out; a weight is exp2((score - maximum) * scale *
// log2(e)).  The difference comes first: equal scores are equal to the maximum
// exactly, however large they are, and the rounded argument is off by a part of
// the difference, not of the score.
struct AttnParams {
  int R, W, Hq, Hkv, d, G, M;
  int page, pages, row_pages;
  int cap;  // positions a prompt row holds: row_pages * page
  int bpage, bpages, brow_pages;
  int64_t q_stride;
  float scale_log2;  // scale * log2(e)
  const void *q, *k, *v;
  const int32_t *table, *lengths;
  const void *bk, *bv;
  const int32_t *btable, *blengths;
  const float *mass;
  float *mass_out;
  void *o;
  float *lse;
  int32_t *status;
  // Division of the prompts (plan_* below) into tiles of `tile` tokens, over
  // `parts` CTAs for every (key-value head, row tile).
  int tile, parts;
  int rows, row_tiles;  // query rows per CTA, and CTAs for the M rows
  int per_slot;         // results per slot (two where two warp groups share the rows)
  int direct;           // a CTA per request and no beam segment: the split kernel writes o itself
  // Scratch: per (slot, key-value head, row) the unnormalised output and
  // (maximum, sum); for the mass norm [R][Hkv][M], a row's (maximum, 1 / sum),
  // +inf and 0 where it has nothing to attend to (not its lse: next to a large
  // maximum the logarithm of the sum would lose its bits, and weights with it),
  // and scores [R][Hkv][M][cap].
  float *part_o;
  float2 *part_ml;
  float2 *norm;
  float *scores;
  // Of the tensor-core kernel's waits between its warps: the bound of each, and
  // (tests) the barriers that expect one arrival more than will come.
  unsigned long long wait_ns;
  int stall;  // 0 or kStall*
};
enum {
  kStallEmpty = 1, kStallFull, kStallScores, kStallWeights, kStallOutputs,       // attn_wide
  kStallMassEmpty, kStallMassFull, kStallMassScores, kStallMassRead, kStallEnd  // attn_mass_wide
};

__device__ __forceinline__ int prompt_len(const AttnParams &p, int r) {
  const int n = p.lengths[r];
  return n < 0 ? 0 : (n > p.cap ? p.cap : n);
}

// The prompts, cut into tiles, are laid end to end: T tiles in all, and part
// c of n takes tiles floor(c T / n) .. floor((c + 1) T / n) - 1 of them.  So
// every CTA has the same work to within a tile, whatever the lengths of a
// batch; a part may end inside one request and begin inside another.  What
// part c finds for request r goes to slot c + r: walking along the tiles
// either c or r grows by one at each border, so a slot has one writer, and a
// request's slots are consecutive.  Every CTA derives the division from the
// lengths itself (they live on the device and the host never waits for them),
// which costs one pass over R integers.
struct PlanSmem {
  long long tot[32];
  int r;
  long long base;
};

__device__ __forceinline__ int tiles_of(const AttnParams &p, int r) { return (prompt_len(p, r) + p.tile - 1) / p.tile; }

// Block-wide: the tiles of all requests, and of those before this thread's
// stretch of requests [r0, r1).
template <int kThreads>
__device__ __forceinline__ long long plan_scan(const AttnParams &p, PlanSmem &sm, int &r0, int &r1, long long &before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const int seg = (p.R + kThreads - 1) / kThreads;
  r0 = min(p.R, tid * seg);
  r1 = min(p.R, r0 + seg);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += tiles_of(p, r);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sm.tot[warp] = incl;
  __syncthreads();
  long long total = 0;
  before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.tot[w];
    total += sm.tot[w];
  }
  return total;
}

// Part `c`: walks its pieces.  next() gives the next request and its token
// range [lo, hi); false at the end.  Every thread holds the same values.
struct PlanWalk {
  long long at, end, base;  // tiles: the next one, the part's end, the request's first
  int r, lo, hi, slot;
  template <int kThreads>
  __device__ __forceinline__ void begin(const AttnParams &p, PlanSmem &sm, int c) {
    if (p.direct) {  // part c is request c
      r = c - 1;
      at = 0;
      end = 1;
      base = 0;
      return;
    }
    slot = c;
    if (p.R <= 32) {
      // Each warp for itself: lane = request, no barrier.
      const int lane = threadIdx.x & 31, mine = lane < p.R ? tiles_of(p, lane) : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const long long total = __shfl_sync(0xffffffffu, incl, 31);
      if (!share(c, total, p.parts)) return;
      // The first request that ends behind the part's first tile.
      r = __ffs(__ballot_sync(0xffffffffu, incl > at)) - 1;
      base = __shfl_sync(0xffffffffu, incl - mine, r);
      slot += --r;
      return;
    }
    int r0, r1;
    long long before;
    const long long total = plan_scan<kThreads>(p, sm, r0, r1, before);
    if (!share(c, total, p.parts)) return;
    for (int q = r0; q < r1; ++q) {
      const int t = tiles_of(p, q);
      if (at >= before && at < before + t) {  // exactly one thread and request
        sm.r = q;
        sm.base = before;
      }
      before += t;
    }
    __syncthreads();
    r = sm.r - 1;
    base = sm.base;
    slot += r;
  }
  // Part c's tiles; false if there are none.
  __device__ __forceinline__ bool share(int c, long long total, int parts) {
    const long long n = total < parts ? total : parts;
    at = end = 0;
    if (c >= n) return false;
    if (total < (1LL << 18)) {  // 32-bit division is several times shorter; at most 4736 parts
      at = (uint32_t)c * (uint32_t)total / (uint32_t)n;
      end = ((uint32_t)c + 1u) * (uint32_t)total / (uint32_t)n;
    } else {
      at = c * total / n;
      end = (c + 1) * total / n;
    }
    return true;
  }
  __device__ __forceinline__ bool next(const AttnParams &p) {
    if (at >= end) return false;
    if (p.direct) {
      ++r;
      at = end;
      lo = 0;
      hi = prompt_len(p, r);
      return true;
    }
    for (;;) {
      ++r;
      ++slot;
      const int len = prompt_len(p, r), t = (len + p.tile - 1) / p.tile;
      if (at < base + t) {
        const long long stop = end < base + t ? end : base + t;
        lo = (int)(at - base) * p.tile;
        hi = min(len, (int)(stop - base) * p.tile);
        at = stop;
        base += t;
        return true;
      }
      base += t;
    }
  }
};

// The slots of request r, whose t tiles start at `first`: tile x lies in part
// ((x + 1) n - 1) / total.
__device__ __forceinline__ void slots_of(long long first, int t, long long total, int parts, int r, int &off, int &pieces) {
  if (t == 0) {
    off = pieces = 0;
    return;
  }
  const long long n = total < parts ? total : parts;
  long long c0, c1;
  if (total < (1LL << 18)) {
    c0 = ((uint32_t)(first + 1) * (uint32_t)n - 1u) / (uint32_t)total;
    c1 = ((uint32_t)(first + t) * (uint32_t)n - 1u) / (uint32_t)total;
  } else {
    c0 = ((first + 1) * n - 1) / total;
    c1 = ((first + t) * n - 1) / total;
  }
  off = (int)c0 + r;
  pieces = (int)(c1 - c0) + 1;
}

// Request r: its first slot and how many it has.
template <int kThreads>
__device__ __forceinline__ void plan_row(const AttnParams &p, PlanSmem &sm, int r, int &off, int &pieces) {
  if (p.R <= 32) {
    const int lane = threadIdx.x & 31, mine = lane < p.R ? tiles_of(p, lane) : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int t = __shfl_sync(0xffffffffu, mine, r);
    slots_of(__shfl_sync(0xffffffffu, incl, r) - t, t, __shfl_sync(0xffffffffu, incl, 31), p.parts, r, off, pieces);
    return;
  }
  int r0, r1;
  long long before;
  const long long total = plan_scan<kThreads>(p, sm, r0, r1, before);
  if (r >= r0 && r < r1) {
    for (int q = r0; q < r; ++q) before += tiles_of(p, q);
    sm.base = before;
  }
  __syncthreads();
  slots_of(sm.base, tiles_of(p, r), total, p.parts, r, off, pieces);
}

// Partial results of row m of (slot, head).
__device__ __forceinline__ int64_t part_row(const AttnParams &p, int slot, int h, int m) {
  return ((int64_t)slot * p.Hkv + h) * p.M + m;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// exp2((a - b) * scale), b >= a: 0 for a = -inf, even where b is -inf too (nothing
// seen yet); NaN stays NaN.
__device__ __forceinline__ float exp2_sub(float a, float b, float scale) {
  return a == -CUDART_INF_F ? 0.f : exp2f((a - b) * scale);
}

// 2^x by the special-function unit (2 ulp); results below 2^-126 become 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The smaller of two; NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
constexpr float kSlack = 8.f;  // growth of a row's maximum, in log2, before the tensor-core kernels rescale its output

constexpr int32_t kStatusPage = 1, kStatusLength = 2;  // ONELA_STATUS_*
__device__ __forceinline__ void set_status(int32_t *status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// Kernels of a call, chosen on the host.
enum AttnKind { kAttnSimt = 0, kAttnNarrow = 1, kAttnWide = 2 };
cudaError_t launch_attn_narrow(const AttnParams &p, cudaStream_t s);  // attention_narrow.cu
int attn_narrow_ctas(int d);                                           // CTAs of it per SM
cudaError_t launch_attn_wide(const AttnParams &p, cudaStream_t s);    // attention_wide.cu
cudaError_t launch_attn_mass_wide(const AttnParams &p, cudaStream_t s);

// pdl: the kernel may be launched while the one before it in the stream still
// runs (programmatic dependent launch).  Every kernel launched so waits for
// that one before it touches anything the stream's earlier work may write, and
// lets its own successor start only after that wait; so when a kernel runs,
// all but its immediate predecessor are complete.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*f)(P...), unsigned grid, unsigned threads, size_t smem, bool pdl, cudaStream_t s, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, a...);
}

}  // namespace onela
