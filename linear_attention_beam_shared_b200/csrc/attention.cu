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

#include <math_constants.h>

#include "../../include/onela.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_f(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

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
// exp2(a - b) for a maximum b that may be -inf (nothing seen yet): 0 then.
__device__ __forceinline__ float exp2_sub(float a, float b) { return b == -CUDART_INF_F ? 0.f : exp2f(a - b); }

constexpr int kThreads = 128;
constexpr int kRows = 8;   // query rows per CTA
constexpr int kToks = 32;  // tokens per step

// The general kernel: any d, fp32 or bf16.  A CTA takes one piece of a prompt,
// one key-value head and 8 query rows; per step of 32 tokens K and V rows go
// through shared memory as fp32, each warp forms two rows' scores (lane =
// token), and each thread keeps one or two columns of the 8 outputs.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) attn_simt(AttnParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ PlanSmem plan;
  __shared__ float ps[kToks][kRows];
  __shared__ float corr[kRows];
  __shared__ int ok[kToks];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int dp = (p.d + 3) & ~3, dk = dp + 4;
  float *qs = smem, *ks = qs + kRows * dp, *vs = ks + kToks * dk;

  const int rt = blockIdx.x % p.row_tiles, uh = blockIdx.x / p.row_tiles;
  const int h = uh % p.Hkv, u = uh / p.Hkv;
  ptx::pdl_launch_dependents();
  int r, lo, hi;
  if (p.direct) {  // one piece per request, an empty one included: its rows are written here
    r = u;
    lo = 0;
    hi = prompt_len(p, r);
  } else if (!plan_unit<kThreads>(p, plan, u, r, lo, hi)) {
    return;
  }
  if (h == 0 && rt == 0 && lo == 0 && tid == 0 && p.lengths[r] != prompt_len(p, r)) set_status(p.status, kStatusLength);

  const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
  const int m0 = rt * kRows;
  for (int i = warp; i < kRows; i += 4) {
    const int m = m0 + i;
    const int w = m / p.G, hq = h * p.G + m % p.G;
    for (int c = lane; c < dp; c += 32)
      qs[i * dp + c] = (m < p.M && c < p.d) ? to_f(q[((int64_t)r * p.W + w) * p.q_stride + (int64_t)hq * p.d + c]) : 0.f;
  }
  // Columns past d of the key rows stay zero.
  for (int i = tid; i < kToks; i += kThreads)
    for (int c = p.d; c < dp; ++c) ks[i * dk + c] = 0.f;

  float acc0[kRows], acc1[kRows], mx[2], sum[2];
#pragma unroll
  for (int i = 0; i < kRows; ++i) acc0[i] = acc1[i] = 0.f;
  mx[0] = mx[1] = -CUDART_INF_F;
  sum[0] = sum[1] = 0.f;
  const int c0 = tid, c1 = tid + kThreads;

  for (int t0 = lo; t0 < hi; t0 += kToks) {
    __syncthreads();  // the previous step's K, V and ps are read
    for (int i = warp; i < kToks; i += 4) {
      const int pos = t0 + i;
      int64_t row = -1;
      if (pos < hi) {
        const int pg = p.table[(int64_t)r * p.row_pages + pos / p.page];
        if (pg >= 0 && pg < p.pages) {
          row = (((int64_t)pg * p.Hkv + h) * p.page + pos % p.page) * p.d;
        } else if (lane == 0) {
          set_status(p.status, kStatusPage);
        }
      }
      if (lane == 0) ok[i] = row >= 0;
      if constexpr (kVec) {
        constexpr int kE = 16 / sizeof(T);
        for (int c = lane * kE; c < p.d; c += 32 * kE) {
          union { uint4 u; T e[kE]; } a, b;
          a.u = b.u = make_uint4(0, 0, 0, 0);
          if (row >= 0) {
            a.u = *reinterpret_cast<const uint4 *>(k + row + c);
            b.u = *reinterpret_cast<const uint4 *>(v + row + c);
          }
#pragma unroll
          for (int e = 0; e < kE; e += 4) {
            *reinterpret_cast<float4 *>(&ks[i * dk + c + e]) =
                make_float4(to_f(a.e[e]), to_f(a.e[e + 1]), to_f(a.e[e + 2]), to_f(a.e[e + 3]));
            *reinterpret_cast<float4 *>(&vs[i * dp + c + e]) =
                make_float4(to_f(b.e[e]), to_f(b.e[e + 1]), to_f(b.e[e + 2]), to_f(b.e[e + 3]));
          }
        }
      } else {
        for (int c = lane; c < p.d; c += 32) {
          ks[i * dk + c] = row >= 0 ? to_f(k[row + c]) : 0.f;
          vs[i * dp + c] = row >= 0 ? to_f(v[row + c]) : 0.f;
        }
      }
    }
    __syncthreads();
    float s[2] = {0.f, 0.f};
    {
      const float *kr = ks + lane * dk, *qa = qs + (2 * warp) * dp, *qb = qa + dp;
      for (int c = 0; c < dp; c += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(kr + c);
        const float4 a = *reinterpret_cast<const float4 *>(qa + c), b = *reinterpret_cast<const float4 *>(qb + c);
        s[0] += x.x * a.x + x.y * a.y + x.z * a.z + x.w * a.w;
        s[1] += x.x * b.x + x.y * b.y + x.z * b.z + x.w * b.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + 2 * warp + i;
      const float x = ok[lane] ? s[i] * p.scale_log2 : -CUDART_INF_F;
      if (p.scores && m < p.M && t0 + lane < hi)
        p.scores[(((int64_t)r * p.Hkv + h) * p.M + m) * p.cap + t0 + lane] = x;
      const float mnew = fmaxf(mx[i], warp_max(x));
      const float e = exp2_sub(x, mnew), f = exp2_sub(mx[i], mnew);
      sum[i] = sum[i] * f + warp_sum(e);
      mx[i] = mnew;
      ps[lane][2 * warp + i] = e;
      if (lane == 0) corr[2 * warp + i] = f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      acc0[i] *= corr[i];
      acc1[i] *= corr[i];
    }
    const int n = min(kToks, hi - t0);
    if (c0 < p.d) {
      for (int t = 0; t < n; ++t) {
        const float4 a = *reinterpret_cast<const float4 *>(&ps[t][0]), b = *reinterpret_cast<const float4 *>(&ps[t][4]);
        const float e[kRows] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const float x0 = vs[t * dp + c0];
#pragma unroll
        for (int i = 0; i < kRows; ++i) acc0[i] += e[i] * x0;
        if (c1 < p.d) {
          const float x1 = vs[t * dp + c1];
#pragma unroll
          for (int i = 0; i < kRows; ++i) acc1[i] += e[i] * x1;
        }
      }
    }
  }
  __syncthreads();
  if (p.direct) {
    // Sums by row through shared memory (each warp holds two rows').
    if (lane == 0) {
      corr[2 * warp] = sum[0];
      corr[2 * warp + 1] = sum[1];
      ps[0][2 * warp] = mx[0];
      ps[0][2 * warp + 1] = mx[1];
    }
    __syncthreads();
    T *o = static_cast<T *>(p.o);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int m = m0 + i;
      if (m >= p.M) continue;
      const int64_t row = ((int64_t)r * p.W + m / p.G) * p.Hq + h * p.G + m % p.G;
      const float inv = corr[i] == 0.f ? 0.f : 1.f / corr[i];
      if (c0 < p.d) store_f(o + row * p.d + c0, acc0[i] * inv);
      if (c1 < p.d) store_f(o + row * p.d + c1, acc1[i] * inv);
      if (tid == 0 && p.lse) p.lse[row] = corr[i] == 0.f ? -CUDART_INF_F : (ps[0][i] + log2f(corr[i])) * kLn2;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int m = m0 + i;
    if (m >= p.M) continue;
    float *po = p.part_o + part_row(p, u, h, m) * p.d;
    if (c0 < p.d) po[c0] = acc0[i];
    if (c1 < p.d) po[c1] = acc1[i];
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + 2 * warp + i;
      if (m < p.M) p.part_ml[part_row(p, u, h, m)] = make_float2(mx[i], sum[i]);
    }
  }
}

// Joins a row's pieces and the beam's own tokens: a warp per query row, lane
// = column of d (c = lane + 32 i).  The beams' own tokens are few (a decode
// horizon), so their scores are formed here, one token at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_join(AttnParams p) {
  __shared__ PlanSmem plan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = p.W * p.Hq, groups = (rows + 3) / 4;
  const int r = blockIdx.x / groups, row = (blockIdx.x % groups) * 4 + warp;
  int off, pieces;
  plan_row<kThreads>(p, plan, r, off, pieces);
  if (row == 0 && lane == 0 && p.lengths[r] != prompt_len(p, r)) set_status(p.status, kStatusLength);
  ptx::pdl_wait();
  if (row >= rows) return;
  const int w = row / p.Hq, hq = row % p.Hq, h = hq / p.G, m = w * p.G + hq % p.G;

  float acc[8], mx = -CUDART_INF_F, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int c0 = 0; c0 < pieces; c0 += 32) {
    // One piece's (maximum, sum) per lane, then the outputs weighted by them.
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (c0 + lane < pieces) ml = p.part_ml[part_row(p, off + c0 + lane, h, m)];
    const float mnew = fmaxf(mx, warp_max(ml.x));
    const float f = exp2_sub(mx, mnew), e = exp2_sub(ml.x, mnew);
    sum = sum * f + warp_sum(ml.y * e);
    mx = mnew;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= f;
    const int n = min(32, pieces - c0);
    for (int j = 0; j < n; ++j) {
      const float ej = __shfl_sync(0xffffffffu, e, j);
      const float *po = p.part_o + part_row(p, off + c0 + j, h, m) * p.d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        if (c < p.d) acc[i] += ej * po[c];
      }
    }
  }
  if (p.bk) {
    const T *q = static_cast<const T *>(p.q) + ((int64_t)r * p.W + w) * p.q_stride + (int64_t)hq * p.d;
    const T *bk = static_cast<const T *>(p.bk), *bv = static_cast<const T *>(p.bv);
    float qv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) qv[i] = lane + 32 * i < p.d ? to_f(q[lane + 32 * i]) : 0.f;
    const int bcap = p.brow_pages * p.bpage, given = p.blengths[(int64_t)r * p.W + w];
    const int n = given < 0 ? 0 : (given > bcap ? bcap : given);
    if (n != given && lane == 0) set_status(p.status, kStatusLength);
    const int32_t *tab = p.btable + ((int64_t)r * p.W + w) * p.brow_pages;
    for (int t = 0; t < n; ++t) {
      const int pg = tab[t / p.bpage];
      if (pg < 0 || pg >= p.bpages) {
        if (lane == 0) set_status(p.status, kStatusPage);
        continue;
      }
      const int64_t at = (((int64_t)pg * p.Hkv + h) * p.bpage + t % p.bpage) * p.d;
      float s = 0.f, vv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        vv[i] = 0.f;
        if (c < p.d) {
          s += qv[i] * to_f(bk[at + c]);
          vv[i] = to_f(bv[at + c]);
        }
      }
      s = warp_sum(s) * p.scale_log2;
      const float mnew = fmaxf(mx, s), f = exp2_sub(mx, mnew), e = exp2_sub(s, mnew);
      sum = sum * f + e;
      mx = mnew;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = acc[i] * f + e * vv[i];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t orow = ((int64_t)r * p.W + w) * p.Hq + hq;
  T *o = static_cast<T *>(p.o) + orow * p.d;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < p.d) store_f(o + lane + 32 * i, acc[i] * inv);
  if (lane == 0) {
    const float l2 = sum == 0.f ? -CUDART_INF_F : mx + log2f(sum);
    if (p.lse) p.lse[orow] = l2 * kLn2;
    if (p.lse2) p.lse2[((int64_t)r * p.Hkv + h) * p.M + m] = l2;
  }
}

// The weight each prompt position drew, from the scores the split kernel
// stored: a thread per position adds exp2(s - lse2) over the M rows in order.
__global__ void __launch_bounds__(kThreads) attn_mass(AttnParams p) {
  const int chunks = (p.cap + kThreads - 1) / kThreads;
  const int pos = (blockIdx.x % chunks) * kThreads + threadIdx.x;
  const int rh = blockIdx.x / chunks, r = rh / p.Hkv;
  ptx::pdl_wait();
  if (pos >= prompt_len(p, r)) return;
  const float *l2 = p.lse2 + (int64_t)rh * p.M, *sc = p.scores + (int64_t)rh * p.M * p.cap + pos;
  float t = 0.f;
  for (int m = 0; m < p.M; ++m) t += exp2_sub(sc[(int64_t)m * p.cap], l2[m]);
  const int64_t at = (int64_t)rh * p.cap + pos;
  p.mass_out[at] = p.mass ? p.mass[at] + t : t;
}

template <typename F, typename... A>
cudaError_t launch(F *f, unsigned grid, unsigned threads, size_t smem, bool pdl, cudaStream_t s, A... a) {
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

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Chooses the division and lays out the scratch; the bytes needed.
size_t plan_call(const onela_attention_config &c, bool want_mass, AttnParams &p, uint8_t *scratch) {
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
  p.rows = kRows;
  p.row_tiles = (p.M + kRows - 1) / kRows;
  p.tile = kToks;
  p.min_chunk = 128;
  // About four CTAs for every SM, fewer and longer pieces where the heads
  // and rows alone give as many.
  const long long groups = (long long)p.Hkv * p.row_tiles;
  const long long slots = 4 * kAttnSMs;
  long long target = (slots + groups - 1) / groups;
  const long long most = (long long)p.R * ((p.cap + p.min_chunk - 1) / p.min_chunk);
  if (target > most) target = most;
  p.target = (int)target;
  const long long by_len = most;
  p.units = (int)(target + p.R < by_len ? target + p.R : by_len);
  p.direct = p.cap <= p.min_chunk && c.beam_row_pages == 0 && !want_mass;
  if (p.direct) p.units = p.R;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *q = scratch + at;
    at += align256(bytes);
    return q;
  };
  if (!p.direct) {
    const size_t rows = (size_t)p.units * p.Hkv * p.M;
    p.part_o = reinterpret_cast<float *>(take(rows * p.d * 4));
    p.part_ml = reinterpret_cast<float2 *>(take(rows * 8));
  }
  if (want_mass) {
    p.lse2 = reinterpret_cast<float *>(take((size_t)p.R * p.Hkv * p.M * 4));
    p.scores = reinterpret_cast<float *>(take((size_t)p.R * p.Hkv * p.M * p.cap * 4));
  }
  return at;
}

template <typename T>
cudaError_t run(const AttnParams &p, bool vec, cudaStream_t s) {
  const int dp = (p.d + 3) & ~3;
  const size_t smem = (size_t)(kRows * dp + kToks * (dp + 4) + kToks * dp) * 4;
  auto f = vec ? attn_simt<T, true> : attn_simt<T, false>;
  cudaError_t e = ensure_smem_limit((const void *)f, smem);
  if (e != cudaSuccess) return e;
  e = launch(f, (unsigned)((long long)p.units * p.Hkv * p.row_tiles), kThreads, smem, false, s, p);
  if (e != cudaSuccess || p.direct) return e;
  e = launch(attn_join<T>, (unsigned)((long long)p.R * ((p.W * p.Hq + 3) / 4)), kThreads, 0, true, s, p);
  if (e != cudaSuccess || !p.mass_out) return e;
  return launch(attn_mass, (unsigned)((long long)p.R * p.Hkv * ((p.cap + kThreads - 1) / kThreads)), kThreads, 0, true,
                s, p);
}

}  // namespace

bool attention_tc_supports(const onela_attention_config &, const AttnParams &) { return false; }

size_t attention_scratch_bytes(const onela_attention_config &c, bool want_mass) {
  AttnParams p = {};
  return plan_call(c, want_mass, p, nullptr);
}

cudaError_t launch_attention(const onela_attention_config &c, AttnParams &p, void *scratch, cudaStream_t s) {
  plan_call(c, p.mass_out != nullptr, p, static_cast<uint8_t *>(scratch));
  const int es = c.dtype == ONELA_BF16 ? 2 : 4;
  const bool vec = (c.d * es) % 16 == 0 && ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 15) == 0;
  return c.dtype == ONELA_BF16 ? run<__nv_bfloat16>(p, vec, s) : run<float>(p, vec, s);
}

}  // namespace onela
