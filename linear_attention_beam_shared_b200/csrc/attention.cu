// Attention of new tokens over a paged key-value cache: the general kernel,
// the kernel that joins the pieces of a prompt and adds the beams' own
// tokens, and the attention weight each cached token drew.
//
// A softmax over a long row is taken in pieces: a piece keeps its maximum m,
// its sum l = sum exp2(s - m) and o = sum exp2(s - m) v, and pieces join by
//     m* = max m_i,  l* = sum l_i exp2(m_i - m*),  o* = sum o_i exp2(m_i - m*),
// which is the softmax of the whole row exactly (in real arithmetic).  All of
// it is held in fp32.
#include "attention.h"

#include <algorithm>

#include "../../include/onela.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_f(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int kThreads = 128;
constexpr int kToks = 32;  // tokens per step

// N consecutive elements as floats.
template <int N, bool kVec>
__device__ __forceinline__ void ldn(const float *p, float (&v)[N]) {
  if constexpr (kVec && N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(p + i);
      v[i] = a.x;
      v[i + 1] = a.y;
      v[i + 2] = a.z;
      v[i + 3] = a.w;
    }
  } else if constexpr (kVec && N == 2) {
    const float2 a = *reinterpret_cast<const float2 *>(p);
    v[0] = a.x;
    v[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}
template <int N, bool kVec>
__device__ __forceinline__ void ldn(const __nv_bfloat16 *p, float (&v)[N]) {
  static_assert(kVec && N % 2 == 0, "pairs");
  uint32_t u[N / 2];
  if constexpr (N == 8) *reinterpret_cast<uint4 *>(u) = *reinterpret_cast<const uint4 *>(p);
  else if constexpr (N == 4) *reinterpret_cast<uint2 *>(u) = *reinterpret_cast<const uint2 *>(p);
  else u[0] = *reinterpret_cast<const uint32_t *>(p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// 4-byte asynchronous copy global -> shared; src_bytes = 0 writes zeros without reading src.
__device__ __forceinline__ void cp_async4_zfill(void *dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(src_bytes)
               : "memory");
}

// Shared memory of the general kernel: q as fp32, then stages of raw K and V
// rows.  K rows are an odd number of 16-byte chunks apart, so that 32 lanes
// reading the same chunk of 32 rows meet no bank twice.
struct SimtLayout {
  int rows, dp, k_stride, v_stride, stage, stages;  // q rows, floats of one; bytes of a K row, a V row, a stage
  __host__ __device__ SimtLayout(int d, int es, int rows) {
    const int row = (d * es + 15) & ~15;
    this->rows = rows;
    dp = row / es;
    k_stride = row / 16 % 2 ? row : row + 16;
    v_stride = row;
    stage = kToks * (k_stride + v_stride);
    stages = row <= 256 ? 3 : 2;
  }
  __host__ __device__ int bytes() const { return rows * dp * 4 + stages * stage; }
  // CTAs that fit an SM by shared memory, at most 4 (by registers).
  int per_sm() const { return std::min(4, std::max(1, 225 * 1024 / (bytes() + 3 * 1024))); }
};

// The general kernel: any d, fp32 or bf16.  A CTA takes one part of the
// prompts, one key-value head and kRows (8, or 4 where there are no more)
// query rows.  Steps of 32 tokens pass through a ring of stages filled by
// asynchronous copies of kUnit bytes: 16, or 4 where rows are no multiple of 16
// bytes or not on such boundaries; bf16 rows of odd d by plain loads (kUnit =
// 2).  Per step each warp forms one or two rows' scores (lane = token: a K
// chunk from shared memory serves both rows, 8 FMAs for 3 loads), takes their
// softmax by shuffles, and each thread adds to one or two columns of the
// outputs (one V element for all rows).  Up to four rows the latency of the steps
// and their two block barriers bounds it, well before reading the cache would (32
// requests x 16 / 4 heads on 5120 tokens, fp32: d = 64 112 us, 128 172 us = 3.9 TB/s,
// 256, one CTA an SM, 424 us; bf16: d = 96 136 us, 37 by plain loads 252 us), the
// FMAs beyond: rows past 8 read K and V again (1 request of 256 beams, 16 / 4 heads
// of 128, 5120 tokens: 839 us in fp32, 748 in bf16).
template <typename T, int kUnit, int kRows>
__global__ void __launch_bounds__(kThreads, 4) attn_simt(AttnParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ PlanSmem plan;
  __shared__ __align__(16) float ps[kToks][kRows];
  __shared__ __align__(16) float corr[kRows];
  __shared__ __align__(4) uint8_t there[4][4];  // by stage and warp: which of its 8 tokens are there
  const SimtLayout L(p.d, sizeof(T), kRows);
  constexpr int kOwn = kRows / 4;  // rows whose scores a warp forms
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *qs = smem;
  uint8_t *ring = reinterpret_cast<uint8_t *>(smem + kRows * L.dp);

  const int rt = blockIdx.x % p.row_tiles, uh = blockIdx.x / p.row_tiles;
  const int h = uh % p.Hkv;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  PlanWalk walk;
  walk.begin<kThreads>(p, plan, uh / p.Hkv);

  const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
  const int m0 = rt * kRows;
  const int c0 = tid, c1 = tid + kThreads;
  while (walk.next(p)) {
    const int r = walk.r, lo = walk.lo, hi = walk.hi, n = (hi - lo + kToks - 1) / kToks;
    __syncthreads();  // the previous piece's shared memory is read
    if (p.direct && h == 0 && rt == 0 && tid == 0 && p.lengths[r] != hi) set_status(p.status, kStatusLength);
    // The page and the place on it of this lane's token of step i (lanes 0 ..
    // 7: the warp's 8 tokens).  The entry is looked at a step later, so that
    // no warp waits for the table.
    int pg = 0, place = 0;
    auto look = [&](int i) {
      const int pos = lo + i * kToks + warp * 8 + lane;
      if (lane < 8 && pos < hi) {
        const int at = pos / p.page;
        pg = p.table[(int64_t)r * p.row_pages + at];
        place = pos - at * p.page;
      }
    };
    auto fill = [&](int i) {
      if (i < n) {
        int64_t row = -1;  // element offset of the token's row; -1 if it is not there
        if (lane < 8 && lo + i * kToks + warp * 8 + lane < hi) {
          if (pg >= 0 && pg < p.pages) row = (((int64_t)pg * p.Hkv + h) * p.page + place) * p.d;
          else set_status(p.status, kStatusPage);
        }
        const int st = i % L.stages;
        uint8_t *kd = ring + st * L.stage, *vd = kd + kToks * L.k_stride;
        const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0) there[st][warp] = (uint8_t)bits;
#pragma unroll 4
        for (int t = 0; t < 8; ++t) {
          const int64_t at = __shfl_sync(0xffffffffu, row, t);
          uint8_t *kr = kd + (warp * 8 + t) * L.k_stride, *vr = vd + (warp * 8 + t) * L.v_stride;
          if constexpr (kUnit == 16) {
            for (int c = lane * 16; c < p.d * (int)sizeof(T); c += 512) {
              ptx::cp_async16(kr + c, reinterpret_cast<const uint8_t *>(k + (at < 0 ? 0 : at)) + c, at < 0 ? 0 : 16);
              ptx::cp_async16(vr + c, reinterpret_cast<const uint8_t *>(v + (at < 0 ? 0 : at)) + c, at < 0 ? 0 : 16);
            }
          } else if constexpr (kUnit == 4) {
            for (int c = lane * 4; c < L.dp * (int)sizeof(T); c += 128) {
              const bool in = at >= 0 && c < p.d * (int)sizeof(T);
              const int64_t from = in ? at * (int)sizeof(T) + c : 0;
              cp_async4_zfill(kr + c, reinterpret_cast<const uint8_t *>(k) + from, in ? 4 : 0);
              cp_async4_zfill(vr + c, reinterpret_cast<const uint8_t *>(v) + from, in ? 4 : 0);
            }
          } else {
            for (int c = lane; c < L.dp; c += 32) {
              const bool in = at >= 0 && c < p.d;
              reinterpret_cast<T *>(kr)[c] = in ? k[at + c] : T(0.f);
              reinterpret_cast<T *>(vr)[c] = in ? v[at + c] : T(0.f);
            }
          }
        }
      }
      ptx::cp_async_commit();
    };
    look(0);
    for (int i = 0; i < L.stages - 1; ++i) {
      fill(i);
      look(i + 1);
    }
    for (int i = warp; i < kRows; i += 4) {
      const int m = m0 + i;
      const int w = m / p.G, hq = h * p.G + m % p.G;
      for (int c = lane; c < L.dp; c += 32)
        qs[i * L.dp + c] =
            (m < p.M && c < p.d) ? to_f(q[((int64_t)r * p.W + w) * p.q_stride + (int64_t)hq * p.d + c]) : 0.f;
    }

    float acc0[kRows], acc1[kRows], mx[kOwn], sum[kOwn];
#pragma unroll
    for (int i = 0; i < kRows; ++i) acc0[i] = acc1[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      mx[i] = -CUDART_INF_F;
      sum[i] = 0.f;
    }

    for (int i = 0; i < n; ++i) {
      if (L.stages == 3) ptx::cp_async_wait_group1();
      else ptx::cp_async_wait_all();
      __syncthreads();  // step i is there for every warp, step i - 1 read by all
      fill(i + L.stages - 1);
      look(i + L.stages);
      const int st = i % L.stages;
      const uint8_t *ks = ring + st * L.stage, *vs = ks + kToks * L.k_stride;
      const uint32_t live = *reinterpret_cast<const uint32_t *>(there[st]);
      float s[kOwn];
#pragma unroll
      for (int e = 0; e < kOwn; ++e) s[e] = 0.f;
      {
        const uint8_t *kr = ks + lane * L.k_stride;
        const float *qa = qs + kOwn * warp * L.dp;
        constexpr int kE = 16 / sizeof(T);
#pragma unroll 4
        for (int c = 0; c < L.dp; c += kE) {
          float x[kE];
          ldn<kE, true>(reinterpret_cast<const T *>(kr) + c, x);
#pragma unroll
          for (int e = 0; e < kE; e += 4) {
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
              const float4 a = *reinterpret_cast<const float4 *>(qa + o * L.dp + c + e);
              s[o] += x[e] * a.x + x[e + 1] * a.y + x[e + 2] * a.z + x[e + 3] * a.w;
            }
          }
        }
      }
      const int pos = lo + i * kToks + lane;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        const int m = m0 + kOwn * warp + e;
        const float x = (live >> lane) & 1 ? s[e] : -CUDART_INF_F;
        if (p.scores && m < p.M && pos < hi) p.scores[(((int64_t)r * p.Hkv + h) * p.M + m) * p.cap + pos] = x;
        const float mnew = fmaxf(mx[e], warp_max(x));
        const float w = exp2_sub(x, mnew, p.scale_log2), f = exp2_sub(mx[e], mnew, p.scale_log2);
        sum[e] = sum[e] * f + warp_sum(w);
        mx[e] = mnew;
        ps[lane][kOwn * warp + e] = w;
        if (lane == 0) corr[kOwn * warp + e] = f;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        acc0[e] *= corr[e];
        acc1[e] *= corr[e];
      }
      const int nt = min(kToks, hi - lo - i * kToks);
      if (c0 < p.d) {
        const T *vc = reinterpret_cast<const T *>(vs) + c0;
        const int step = L.v_stride / (int)sizeof(T);
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
          float w[kRows];
          ldn<kRows, true>(ps[t], w);
          const float x0 = to_f(vc[t * step]);
#pragma unroll
          for (int e = 0; e < kRows; ++e) acc0[e] += w[e] * x0;
          if (c1 < p.d) {
            const float x1 = to_f(vc[t * step + kThreads]);
#pragma unroll
            for (int e = 0; e < kRows; ++e) acc1[e] += w[e] * x1;
          }
        }
      }
    }
    ptx::cp_async_wait_all();
    __syncthreads();
    if (p.direct) {
      // Sums by row through shared memory (each warp holds its own).
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          corr[kOwn * warp + i] = sum[i];
          ps[0][kOwn * warp + i] = mx[i];
        }
      }
      __syncthreads();
      T *o = static_cast<T *>(p.o);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = m0 + i;
        if (m >= p.M) continue;
        const int64_t orow = ((int64_t)r * p.W + m / p.G) * p.Hq + h * p.G + m % p.G;
        const float inv = corr[i] == 0.f ? 0.f : 1.f / corr[i];
        if (c0 < p.d) store_f(o + orow * p.d + c0, acc0[i] * inv);
        if (c1 < p.d) store_f(o + orow * p.d + c1, acc1[i] * inv);
        if (tid == 0 && p.lse) p.lse[orow] = corr[i] == 0.f ? -CUDART_INF_F : (ps[0][i] * p.scale_log2 + log2f(corr[i])) * kLn2;
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int m = m0 + i;
      if (m >= p.M) continue;
      float *po = p.part_o + part_row(p, walk.slot, h, m) * p.d;
      if (c0 < p.d) po[c0] = acc0[i];
      if (c1 < p.d) po[c1] = acc1[i];
    }
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int m = m0 + kOwn * warp + i;
        if (m < p.M) p.part_ml[part_row(p, walk.slot, h, m)] = make_float2(mx[i], sum[i]);
      }
    }
  }
}

// A row of d over a group of lanes, as loaded and as floats: with kD (64, 128
// or 256) known, 8 consecutive columns for each of kD / 8 lanes; kD = -1: the
// same over a whole warp for any multiple of 8; kD = 0: columns lane + 32 i of
// the whole warp for any d and alignment.
template <typename T, int kD>
struct Cols {
  static constexpr int kLanes = kD > 0 ? kD / 8 : 32;
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *row, int gl, int d) {
    if (kD < 0 && gl * 8 >= d) {
      zero();
      return;
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(row + gl * 8)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
          v[4 * i + e] = __uint_as_float(w[e]);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T *row, int gl, int d, const float (&v)[8]) {
    if (kD < 0 && gl * 8 >= d) return;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(row + gl * 8) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
      reinterpret_cast<float4 *>(row + gl * 8)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4 *>(row + gl * 8)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};
template <typename T>
struct Cols<T, 0> {
  static constexpr int kLanes = 32;
  float f[8];
  __device__ __forceinline__ void load(const T *row, int gl, int d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = gl + 32 * i < d ? to_f(row[gl + 32 * i]) : 0.f;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i];
  }
  static __device__ __forceinline__ void store(T *row, int gl, int d, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (gl + 32 * i < d) store_f(row + gl + 32 * i, v[i]);
  }
};

// Joins a row's pieces and the beam's own tokens.  A query row takes a group
// of lanes (8, 16 or 32 for d = 64, 128, 256: 16 bytes of bf16 a lane), and a
// group of lanes takes kGr rows of one beam and key-value head, so that their
// K and V are read once (kGr = 4 or 2 where that leaves 12 warps for every SM:
// with 8192 rows of 256 and 7 beam tokens one row each makes three waves of
// CTAs, and the whole call 45.5 instead of 43.7 us).  kWpr warps share those rows: 1 when there are rows enough to fill
// the SMs, 8 when a few rows have many pieces (64 rows of 18 pieces: half the
// time).  The beams' own tokens are few (a decode horizon) and differ from
// beam to beam, so their scores are formed here, four tokens at a time.
template <typename T, int kD, int kWpr, int kGr>
__global__ void __launch_bounds__(kWpr == 1 ? 128 : kWpr * 32, kWpr == 1 ? (kGr == 1 ? 5 : kGr == 2 ? 4 : 3) : 2)
    attn_join(const __grid_constant__ AttnParams p) {
  using C = Cols<T, kD>;
  constexpr int kBlock = kWpr == 1 ? 128 : kWpr * 32, kL = C::kLanes;
  constexpr int kRpw = 32 / kL, kSetsPer = kRpw * (kWpr == 1 ? 4 : 1);  // sets of kGr rows, of a warp and of a CTA
  static_assert(kWpr == 1 || kGr == 1, "warps share single rows");
  __shared__ PlanSmem plan;
  __shared__ float2 wml[kWpr][kRpw];
  __shared__ float wacc[kWpr == 1 ? 1 : kWpr][kWpr == 1 ? 1 : 256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane % kL, grp = lane / kL;
  const int part = kWpr == 1 ? 0 : warp;
  const int sets = p.W * p.Hq / kGr, blocks = (sets + kSetsPer - 1) / kSetsPer;
  const int r = blockIdx.x / blocks;
  const int want = (blockIdx.x % blocks) * kSetsPer + (kWpr == 1 ? warp * kRpw : 0) + grp;
  const int row = min(want, sets - 1) * kGr;  // the first of the set
  int off, pieces;
  plan_row<kBlock>(p, plan, r, off, pieces);
  off *= p.per_slot;
  pieces *= p.per_slot;
  if (blockIdx.x % blocks == 0 && threadIdx.x == 0 && p.lengths[r] != prompt_len(p, r)) set_status(p.status, kStatusLength);
  const int w = row / p.Hq, hq = row % p.Hq, h = hq / p.G, m = w * p.G + hq % p.G;
  auto group_sum = [](float x) {
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };

  float acc[kGr][8], mx[kGr], sum[kGr];
#pragma unroll
  for (int g = 0; g < kGr; ++g) {
    mx[g] = -CUDART_INF_F;
    sum[g] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[g][i] = 0.f;
  }
  // The beam's own tokens first: nothing of them comes from the split kernel,
  // which may still be running.
  if (p.bk) {
    const T *bk = static_cast<const T *>(p.bk), *bv = static_cast<const T *>(p.bv);
    C qr[kGr];
#pragma unroll
    for (int g = 0; g < kGr; ++g)
      qr[g].load(static_cast<const T *>(p.q) + ((int64_t)r * p.W + w) * p.q_stride + (int64_t)(hq + g) * p.d, gl, p.d);
    const int bcap = p.brow_pages * p.bpage, given = p.blengths[(int64_t)r * p.W + w];
    const int n = given < 0 ? 0 : (given > bcap ? bcap : given), most = __reduce_max_sync(0xffffffffu, n);
    if (n != given && gl == 0) set_status(p.status, kStatusLength);
    const int32_t *tab = p.btable + ((int64_t)r * p.W + w) * p.brow_pages;
    // The table's entries kL tokens at a time, one per lane, as element
    // offsets of the rows (-1: not there); then K and V rows four at a time.
    for (int tb = 0; tb < most; tb += kL) {
      int64_t where = -1;
      if (tb + gl < n) {
        const int at = (tb + gl) / p.bpage, pg = tab[at];
        if (pg >= 0 && pg < p.bpages) where = (((int64_t)pg * p.Hkv + h) * p.bpage + (tb + gl - at * p.bpage)) * p.d;
        else set_status(p.status, kStatusPage);
      }
      const int nb = min(kL, most - tb);
      for (int t0 = 4 * part; t0 < nb; t0 += 4 * kWpr) {
        C kk[4], vv[4];
        uint32_t there = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t at = __shfl_sync(0xffffffffu, where, t0 + j, kL);
          if (at >= 0) {
            kk[j].load(bk + at, gl, p.d);
            vv[j].load(bv + at, gl, p.d);
            there |= 1u << j;
          } else {
            kk[j].zero();
            vv[j].zero();
          }
        }
#pragma unroll
        for (int g = 0; g < kGr; ++g) {
          float s[4], qv[8], x[8];
          qr[g].get(qv);
          float top = mx[g];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            kk[j].get(x);
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) t += qv[i] * x[i];
            t = group_sum(t);
            s[j] = (there >> j) & 1 ? t : -CUDART_INF_F;
            top = fmaxf(top, s[j]);
          }
          const float f = exp2_sub(mx[g], top, p.scale_log2);
          mx[g] = top;
          sum[g] *= f;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[g][i] *= f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = exp2_sub(s[j], top, p.scale_log2);
            vv[j].get(x);
            sum[g] += e;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g][i] += e * x[i];
          }
        }
      }
    }
  }
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  for (int c0 = 0; c0 < pieces; c0 += kL * kWpr) {
    // One piece's (maximum, sum) per lane, then the outputs weighted by them.
    const int mine = c0 + gl * kWpr + part;
    float2 ml[kGr];
#pragma unroll
    for (int g = 0; g < kGr; ++g) {
      ml[g] = make_float2(-CUDART_INF_F, 0.f);
      if (mine < pieces) ml[g] = p.part_ml[part_row(p, off + mine, h, m + g)];
    }
    float e[kGr];
#pragma unroll
    for (int g = 0; g < kGr; ++g) {
      float mnew = ml[g].x;
#pragma unroll
      for (int o = kL / 2; o; o >>= 1) mnew = fmaxf(mnew, __shfl_xor_sync(0xffffffffu, mnew, o));
      mnew = fmaxf(mx[g], mnew);
      const float f = exp2_sub(mx[g], mnew, p.scale_log2);
      e[g] = exp2_sub(ml[g].x, mnew, p.scale_log2);
      sum[g] = sum[g] * f + group_sum(ml[g].y * e[g]);
      mx[g] = mnew;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[g][i] *= f;
    }
    const int n = (min(kL * kWpr, pieces - c0) - part + kWpr - 1) / kWpr;
#pragma unroll(4 / kGr)
    for (int j = 0; j < n; ++j) {
      Cols<float, kD> x[kGr];
#pragma unroll
      for (int g = 0; g < kGr; ++g) x[g].load(p.part_o + part_row(p, off + c0 + j * kWpr + part, h, m + g) * p.d, gl, p.d);
#pragma unroll
      for (int g = 0; g < kGr; ++g) {
        const float ej = __shfl_sync(0xffffffffu, e[g], j, kL);
        float y[8];
        x[g].get(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[g][i] += ej * y[i];
      }
    }
  }
  if constexpr (kWpr > 1) {
    // Warps' results through shared memory, joined by the first.
    if (gl == 0) wml[warp][grp] = make_float2(mx[0], sum[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) wacc[warp][lane + 32 * i] = acc[0][i];
    __syncthreads();
    if (warp != 0) return;
    float top = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < kWpr; ++j) top = fmaxf(top, wml[j][grp].x);
    sum[0] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] = 0.f;
#pragma unroll
    for (int j = 0; j < kWpr; ++j) {
      const float f = exp2_sub(wml[j][grp].x, top, p.scale_log2);
      sum[0] += wml[j][grp].y * f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[0][i] += wacc[j][lane + 32 * i] * f;
    }
    mx[0] = top;
  }
  if (want >= sets) return;
#pragma unroll
  for (int g = 0; g < kGr; ++g) {
    const float inv = sum[g] == 0.f ? 0.f : 1.f / sum[g];
    const int64_t orow = ((int64_t)r * p.W + w) * p.Hq + hq + g;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[g][i] *= inv;
    C::store(static_cast<T *>(p.o) + orow * p.d, gl, p.d, acc[g]);
    if (gl == 0) {
      if (p.lse) p.lse[orow] = sum[g] == 0.f ? -CUDART_INF_F : (mx[g] * p.scale_log2 + log2f(sum[g])) * kLn2;
      if (p.norm) p.norm[((int64_t)r * p.Hkv + h) * p.M + m + g] = make_float2(sum[g] == 0.f ? CUDART_INF_F : mx[g], inv);
    }
  }
}

// The weight each prompt position drew, from the scores the split kernel
// stored: sum exp2(s - max) / sum over the M rows.  A thread takes four positions
// (kP; one where rows are no multiple of 4) and, for few rows, all of these;
// for many the CTA's four warps take every fourth row each of the same positions
// (kSplit = 4), joined through shared memory in a fixed order.
template <int kP, int kSplit>
__global__ void __launch_bounds__(kThreads) attn_mass(const __grid_constant__ AttnParams p) {
  constexpr int kAcross = kThreads / kSplit;  // threads side by side
  __shared__ float part[kSplit][kAcross * kP];
  const int lane = threadIdx.x % kAcross, warp = threadIdx.x / kAcross;
  const int chunks = (p.cap + kAcross * kP - 1) / (kAcross * kP);
  const int first = (int)(blockIdx.x % chunks) * kAcross * kP, pos = first + lane * kP;
  const int rh = blockIdx.x / chunks, r = rh / p.Hkv;
  const int len = prompt_len(p, r);
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (first >= len) return;
  const float2 *norm = p.norm + (int64_t)rh * p.M;
  const float *sc = p.scores + (int64_t)rh * p.M * p.cap + pos;
  float t[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) t[i] = 0.f;
  if (pos < len) {
#pragma unroll 8
    for (int m = warp; m < p.M; m += kSplit) {
      float x[kP];
      ldn<kP, true>(sc + (int64_t)m * p.cap, x);
      const float2 l = norm[m];
#pragma unroll
      for (int i = 0; i < kP; ++i) t[i] += exp2_sub(x[i], l.x, p.scale_log2) * l.y;
    }
  }
  if constexpr (kSplit > 1) {
#pragma unroll
    for (int i = 0; i < kP; ++i) part[warp][lane + kAcross * i] = t[i];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kSplit; ++w)
#pragma unroll
      for (int i = 0; i < kP; ++i) t[i] += part[w][lane + kAcross * i];
  }
  if (pos >= len) return;
  const int64_t at = (int64_t)rh * p.cap + pos;
  if (kP == 4 && pos + 4 <= len) {
    float4 o = make_float4(t[0], t[1], t[2], t[kP - 1]);
    if (p.mass) {
      const float4 a = *reinterpret_cast<const float4 *>(p.mass + at);
      o = make_float4(o.x + a.x, o.y + a.y, o.z + a.z, o.w + a.w);
    }
    *reinterpret_cast<float4 *>(p.mass_out + at) = o;
  } else {
#pragma unroll
    for (int i = 0; i < kP; ++i)
      if (pos + i < len) p.mass_out[at + i] = p.mass ? p.mass[at + i] + t[i] : t[i];
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The tensor-core kernels take bf16 with d in {64, 128, 256}; the pools' and
// q's rows must lie on 16-byte boundaries, o on 4 (pointers not yet known:
// assumed).
bool tc_fits(const onela_attention_config &c, const AttnParams &p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.q);
  return c.dtype == ONELA_BF16 && (c.d == 64 || c.d == 128 || c.d == 256) && c.q_stride % 8 == 0 && (at & 15) == 0 &&
         (reinterpret_cast<uintptr_t>(p.o) & 3) == 0;
}

AttnKind choose(const onela_attention_config &c, const AttnParams &p) {
  if (c.kernel == ONELA_KERNEL_SIMT || !tc_fits(c, p)) return kAttnSimt;
  return p.M <= 16 ? kAttnNarrow : kAttnWide;
}

// Chooses the division and lays out the scratch; the bytes needed.
size_t plan_call(const onela_attention_config &c, bool want_mass, AttnParams &p, uint8_t *scratch, AttnKind &used) {
  p.R = c.R;
  p.W = c.W;
  p.Hq = c.H_q;
  p.Hkv = c.H_kv;
  p.d = c.d;
  p.G = c.H_q / c.H_kv;
  p.M = p.W * p.G;
  p.page = c.page;
  p.pages = c.pages;
  p.row_pages = c.row_pages;
  p.cap = c.page * c.row_pages;
  p.bpage = c.beam_page;
  p.bpages = c.beam_pages;
  p.brow_pages = c.beam_row_pages;
  p.q_stride = c.q_stride;
  p.scale_log2 = c.scale * kLog2e;
  const AttnKind kind = choose(c, p);
  p.rows = p.M <= 4 ? 4 : 8;
  int ctas = SimtLayout(c.d, c.dtype == ONELA_BF16 ? 2 : 4, p.rows).per_sm() * kAttnSMs;  // that run at once
  p.tile = kToks;
  p.per_slot = 1;
  if (kind == kAttnNarrow) {
    p.rows = 16;
    p.tile = 64;
    ctas = attn_narrow_ctas(c.d) * kAttnSMs;
  } else if (kind == kAttnWide) {
    p.rows = c.d < 256 && p.M > 128 ? 256 : 128;
    p.tile = 64;
    p.per_slot = c.d < 256 && p.M <= 128 ? 2 : 1;
    ctas = kAttnSMs;
  }
  p.row_tiles = (p.M + p.rows - 1) / p.rows;
  // Parts per (head, row tile).  n parts take ceil(groups n / ctas) waves of
  // T / n tiles and, for each, about as long as 4 tiles to start and finish;
  // T is at most `most`.  The cheapest n, up to 8 waves: of the n with the same
  // waves the largest is the cheapest.
  const long long groups = (long long)p.Hkv * p.row_tiles;
  const long long most = (long long)p.R * ((p.cap + p.tile - 1) / p.tile);
  auto cost = [&](long long n) { return (double)((groups * n + ctas - 1) / ctas) * ((double)most / n + 4.0); };
  double best = cost(1);
  p.parts = 1;
  for (long long waves = 1; waves <= 8; ++waves) {
    const long long n = std::min(most, waves * ctas / groups);
    if (n > 1 && cost(n) < best) {
      best = cost(n);
      p.parts = (int)n;
    }
  }
  p.direct = kind != kAttnWide && p.cap <= 256 && c.beam_row_pages == 0 && !want_mass;
  if (p.direct) p.parts = p.R;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *q = scratch + at;
    at += align256(bytes);
    return q;
  };
  if (!p.direct) {
    const size_t rows = (size_t)(p.parts + p.R) * p.per_slot * p.Hkv * p.M;
    p.part_o = reinterpret_cast<float *>(take(rows * p.d * 4));
    p.part_ml = reinterpret_cast<float2 *>(take(rows * 8));
  }
  if (want_mass) {
    p.norm = reinterpret_cast<float2 *>(take((size_t)p.R * p.Hkv * p.M * 8));
    if (kind != kAttnWide) p.scores = reinterpret_cast<float *>(take((size_t)p.R * p.Hkv * p.M * p.cap * 4));
  }
  used = kind;
  return at;
}

template <typename T, int kRows>
cudaError_t run_simt(const AttnParams &p, cudaStream_t s) {
  const size_t smem = (size_t)SimtLayout(p.d, sizeof(T), kRows).bytes();
  const uint64_t at = (uint64_t)p.d * sizeof(T) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v);
  auto f = at % 16 == 0 ? attn_simt<T, 16, kRows> : attn_simt<T, 4, kRows>;
  if constexpr (sizeof(T) == 2)
    if (at % 4) f = attn_simt<T, 2, kRows>;
  const cudaError_t e = ensure_smem_limit((const void *)f, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(f, (unsigned)((long long)p.parts * p.Hkv * p.row_tiles), kThreads, smem, true, s, p);
}

template <typename T, int kD>
cudaError_t run_join_d(const AttnParams &p, cudaStream_t s) {
  constexpr int kRpw = 32 / Cols<T, kD>::kLanes;  // rows a warp joins
  const long long rows = (long long)p.W * p.Hq;
  auto grid = [&](int per) { return (unsigned)(p.R * ((rows + per - 1) / per)); };
  // Eight warps for a warp's rows while that is at most about one wave of warps.
  if (p.R * rows <= 8LL * kRpw * kAttnSMs)
    return launch_kernel(attn_join<T, kD, 8, 1>, grid(kRpw), 256, 0, true, s, p);
  if constexpr (kD != 0) {
    const long long most = p.R * rows / (12LL * kRpw * kAttnSMs);  // rows a set, 12 warps left for every SM
    if (p.G % 4 == 0 && most >= 4) return launch_kernel(attn_join<T, kD, 1, 4>, grid(16 * kRpw), 128, 0, true, s, p);
    if (p.G % 2 == 0 && most >= 2) return launch_kernel(attn_join<T, kD, 1, 2>, grid(8 * kRpw), 128, 0, true, s, p);
  }
  return launch_kernel(attn_join<T, kD, 1, 1>, grid(4 * kRpw), 128, 0, true, s, p);
}

template <typename T>
cudaError_t run_join(const AttnParams &p, cudaStream_t s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.bk) |
                       reinterpret_cast<uintptr_t>(p.bv) | reinterpret_cast<uintptr_t>(p.o);
  if ((at & 15) == 0 && p.q_stride * sizeof(T) % 16 == 0) {
    if (p.d == 64) return run_join_d<T, 64>(p, s);
    if (p.d == 128) return run_join_d<T, 128>(p, s);
    if (p.d == 256) return run_join_d<T, 256>(p, s);
    if (p.d % 8 == 0) return run_join_d<T, -1>(p, s);
  }
  return run_join_d<T, 0>(p, s);
}

template <typename T>
cudaError_t run(const AttnParams &p, AttnKind kind, cudaStream_t s) {
  cudaError_t e;
  if (kind == kAttnNarrow) {
    e = launch_attn_narrow(p, s);
  } else if (kind == kAttnWide) {
    e = launch_attn_wide(p, s);
  } else {
    e = p.rows == 4 ? run_simt<T, 4>(p, s) : run_simt<T, 8>(p, s);
  }
  if (e != cudaSuccess || p.direct) return e;

  e = run_join<T>(p, s);
  if (e != cudaSuccess || !p.mass_out) return e;
  if (kind == kAttnWide) return launch_attn_mass_wide(p, s);
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.mass) | reinterpret_cast<uintptr_t>(p.mass_out);
  const int per = p.cap % 4 == 0 && (at & 15) == 0 ? 4 : 1;
  const bool split = p.M > 16;
  const int span = (split ? 32 : kThreads) * per;
  const unsigned grid = (unsigned)((long long)p.R * p.Hkv * ((p.cap + span - 1) / span));
  auto f = per == 4 ? (split ? attn_mass<4, 4> : attn_mass<4, 1>) : (split ? attn_mass<1, 4> : attn_mass<1, 1>);
  return launch_kernel(f, grid, kThreads, 0, true, s, p);
}

}  // namespace

bool attention_tc_supports(const onela_attention_config &c, const AttnParams &p) { return tc_fits(c, p); }

size_t attention_scratch_bytes(const onela_attention_config &c, bool want_mass, const AttnParams &given) {
  AttnParams p = given;
  AttnKind kind;
  return plan_call(c, want_mass, p, nullptr, kind);
}

cudaError_t launch_attention(const onela_attention_config &c, AttnParams &p, void *scratch, cudaStream_t s) {
  AttnKind kind;
  plan_call(c, p.mass_out != nullptr, p, static_cast<uint8_t *>(scratch), kind);
  return c.dtype == ONELA_BF16 ? run<__nv_bfloat16>(p, kind, s) : run<float>(p, kind, s);
}

}  // namespace onela
