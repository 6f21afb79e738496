// Internal declarations of the attention over a paged key-value cache: the
// parameters every kernel takes, the division of the prompts into units of
// work, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace onela {

constexpr int kAttnSMs = 148;         // multiprocessors the units are spread over
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One call.  A (request, key-value head) has M = W * G query rows, row m
// being head m % G of the group of beam m / G.  Scores are kept times log2(e)
// so that the softmax is taken with exp2.
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
  // Division of the prompts (plan_* below): pieces are multiples of `tile`
  // tokens, at least min_chunk (but for a request's last), and there are at
  // most `units` of them.
  int tile, min_chunk, target, units;
  int rows, row_tiles;  // query rows per CTA, and CTAs for the M rows
  int direct;           // one piece per request and no beam segment: the split kernel writes o itself
  // Scratch: per (unit, key-value head, row) the unnormalised output and
  // (maximum, sum); lse2 [R][Hkv][M] and scores [R][Hkv][M][cap] for the mass.
  float *part_o;
  float2 *part_ml;
  float *lse2;
  float *scores;
};

__device__ __forceinline__ int prompt_len(const AttnParams &p, int r) {
  const int n = p.lengths[r];
  return n < 0 ? 0 : (n > p.cap ? p.cap : n);
}

// The prompts are cut into pieces of about the same size whatever their
// lengths, so that a batch of very different lengths keeps every SM busy:
// with T tokens in all and `target` pieces wanted, a piece has about T /
// target tokens, a request of n tokens ceil(n / that) pieces.  Every CTA
// derives the division from the lengths itself (they live on the device and
// the host never waits for them), which costs one pass over R integers.
struct PlanSmem {
  long long tot[32];
  int cnt[32];
  int r, c, pieces, off;
};

// Block-wide: fills sm.cnt with the warps' piece counts; returns the tokens
// per piece, and in `before` / `mine` the pieces of the requests before this
// thread's stretch of requests and in it.
template <int kThreads>
__device__ __forceinline__ int plan_scan(const AttnParams &p, PlanSmem &sm, int &before, int &mine) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const int seg = (p.R + kThreads - 1) / kThreads;
  const int r0 = min(p.R, tid * seg), r1 = min(p.R, r0 + seg);
  long long t = 0;
  for (int r = r0; r < r1; ++r) t += prompt_len(p, r);
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) sm.tot[warp] = t;
  if (tid == 0) sm.r = -1;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sm.tot[w];
  long long want = (total + p.target - 1) / p.target;
  if (want < p.min_chunk) want = p.min_chunk;
  if (want > p.cap) want = p.cap;
  const int chunk = (int)((want + p.tile - 1) / p.tile) * p.tile;
  int c = 0;
  for (int r = r0; r < r1; ++r) c += (prompt_len(p, r) + chunk - 1) / chunk;
  mine = c;
  int incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sm.cnt[warp] = incl;
  __syncthreads();
  before = incl - c;
  for (int w = 0; w < warp; ++w) before += sm.cnt[w];
  return chunk;
}

// Piece `u`: its request and token range [lo, hi); false past the last piece.
template <int kThreads>
__device__ __forceinline__ bool plan_unit(const AttnParams &p, PlanSmem &sm, int u, int &r, int &lo, int &hi) {
  int before, mine;
  const int chunk = plan_scan<kThreads>(p, sm, before, mine);
  if (u >= before && u < before + mine) {
    const int seg = (p.R + kThreads - 1) / kThreads;
    int at = before, q = threadIdx.x * seg;
    for (;; ++q) {
      const int n = (prompt_len(p, q) + chunk - 1) / chunk;
      if (u < at + n) {
        sm.r = q;
        sm.c = u - at;
        sm.pieces = n;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  r = sm.r;
  if (r < 0) return false;
  const int len = prompt_len(p, r);
  const int per = ((len + sm.pieces - 1) / sm.pieces + p.tile - 1) / p.tile * p.tile;
  lo = sm.c * per;
  hi = min(len, lo + per);
  return true;
}

// Request r: its first piece and how many it has.
template <int kThreads>
__device__ __forceinline__ void plan_row(const AttnParams &p, PlanSmem &sm, int r, int &off, int &pieces) {
  int before, mine;
  const int chunk = plan_scan<kThreads>(p, sm, before, mine);
  const int seg = (p.R + kThreads - 1) / kThreads;
  if (r / seg == (int)threadIdx.x) {
    int at = before;
    for (int q = threadIdx.x * seg; q < r; ++q) at += (prompt_len(p, q) + chunk - 1) / chunk;
    sm.off = at;
    sm.pieces = (prompt_len(p, r) + chunk - 1) / chunk;
  }
  __syncthreads();
  off = sm.off;
  pieces = sm.pieces;
}

// Partial results of row m of (unit, head).
__device__ __forceinline__ int64_t part_row(const AttnParams &p, int unit, int h, int m) {
  return ((int64_t)unit * p.Hkv + h) * p.M + m;
}

constexpr int32_t kStatusPage = 1, kStatusLength = 2;  // ONELA_STATUS_*
__device__ __forceinline__ void set_status(int32_t *status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

}  // namespace onela
