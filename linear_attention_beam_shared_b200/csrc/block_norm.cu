// The norms around a block, fused with its gate and residual scale:
//     u  = y * rsqrt(mean_group(y^2) + eps) * w_post * act(gate)
//     x' = x + alpha * scale * u,   n' = x' * rsqrt(mean(x'^2) + eps) * w_pre.
//
// Every input is read once and every output written once, so the bytes bound
// it: a row's values stay in registers (fp32) from the first load to the last
// store, across the two reductions.
#include "block_norm.h"

#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "../../include/onela.h"
#include "attention.h"
#include "f32x2.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

constexpr int kSMs = 148;

__device__ __forceinline__ float ld(const void *p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st(void *p, int64_t i, float x, int bf16) {
  if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<float *>(p)[i] = x;
}

// Eight consecutive elements, 16-byte aligned, as they lie in memory and as floats.
template <bool kBf>
struct Vec;
template <>
struct Vec<true> {
  uint4 u;
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i));
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, const F2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = un(v[e]);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(f.y), "f"(f.x));
    }
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    a = __ldcs(q);
    b = __ldcs(q + 1);
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
    v[0] = f2(a.x, a.y);
    v[1] = f2(a.z, a.w);
    v[2] = f2(b.x, b.y);
    v[3] = f2(b.z, b.w);
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, const F2 (&v)[4]) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    const float2 c = un(v[0]), d = un(v[1]), e = un(v[2]), f = un(v[3]);
    q[0] = make_float4(c.x, c.y, d.x, d.y);
    q[1] = make_float4(e.x, e.y, f.x, f.y);
  }
};
__device__ __forceinline__ void weights8(const float *p, F2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = f2(a.x, a.y);
  v[1] = f2(a.z, a.w);
  v[2] = f2(b.x, b.y);
  v[3] = f2(b.z, b.w);
}

// 1 / (1 + exp(-z)) by the special-function unit: exp2 within 2 ulp, the
// reciprocal within 1 (an IEEE division takes three times the instructions,
// and at D = 4096 in bf16 the instructions are as long as the loads).
__device__ __forceinline__ float sigmoid(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ F2 sigmoid2(F2 z) {
  const float2 t = un(z * f2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = un(f2(e.x, e.y) + f2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
  return f2(e.x, e.y);
}
__device__ __forceinline__ float act(float z, int kind) {
  return kind == ONELA_ACT_SILU ? z * sigmoid(z) : sigmoid(z);
}

// Block-wide sum; every thread gets it.  red holds two sets of one float per
// warp, used in turn (n counts the sums): the one barrier of a sum keeps the
// next-but-one from writing over it.
__device__ __forceinline__ float block_sum(float x, float (&red)[2][32], int &n) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  float *r = red[n++ & 1];
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; w += 4) {
    const float4 q = *reinterpret_cast<const float4 *>(r + w);  // past the last warp: zeros
    s += (q.x + q.y) + (q.z + q.w);
  }
  return s;
}

// A CTA takes rows blockIdx.x, + gridDim.x, ..., kV vectors of 8 channels per
// thread (vector e of thread t holds channels 8 (t + e * threads) ..).  With
// more rows than CTAs at once the weights stay in shared memory (w_post,
// alpha and scale as one factor), for they are as many bytes as a row in fp32, and
// the next row is loaded before this one is reduced, so that loads are always
// under way.  kLoop = false: a row per CTA, weights from global memory (few rows:
// latency is what counts, and nothing would be reused).
// kAll: y, gate, x, w_post over the whole row, w_pre and x_out are all there
// (the sandwich norm in full), so that nothing is asked at run time.
template <bool kYBf, bool kBf, int kV, bool kLoop, bool kAll = false, int kMaxThreads = 512>
__global__ void __launch_bounds__(kMaxThreads, kV == 4 || (kV == 2 && !kLoop) ? 1 : 2) block_norm_vec(const __grid_constant__ BlockNormParams p) {
  // kLoop: [D] factor of u, [D] w_pre; then, for group norms that do not fit a warp, [D / 8] sums.
  extern __shared__ __align__(16) float sm[];
  __shared__ __align__(16) float red[2][32];
  int sums = 0;
  const int tid = threadIdx.x, nt = blockDim.x, nv = p.D / 8, gv = p.group / 8;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (tid < 64) red[tid >> 5][tid & 31] = 0.f;
  const bool has_y = kAll || p.y, has_g = kAll || p.gate, has_x = kAll || p.x, has_post = kAll || p.w_post;
  const bool has_pre = kAll || p.w_pre, has_out = kAll || p.x_out, whole = kAll || p.group == p.D;
  float *fac = sm, *wpre = sm + p.D, *gsum = kLoop ? sm + 2 * p.D : sm;
  const bool in_warp = gv <= 32 && (gv & (gv - 1)) == 0;  // a group is an aligned power of two of lanes
  auto factor = [&](int c, F2 (&w)[4]) {                  // of u at vector c: w_post * alpha * scale
    if (has_post) {
      weights8(p.w_post + (8 * c) % p.group, w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f2(1.f, 1.f);
    }
    F2 z[4];
    const F2 al = f2(p.alpha, p.alpha);
    if (p.scale) weights8(p.scale + 8 * c, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * (p.scale ? al * z[i] : al);
  };
  if (kLoop) {
    for (int c = tid; c < nv; c += nt) {
      F2 w[4];
      factor(c, w);
      Vec<false>::store(fac, 8 * c, w);
      if (has_pre) {
        weights8(p.w_pre + 8 * c, w);
        Vec<false>::store(wpre, 8 * c, w);
      }
    }
  }
  __syncthreads();
  Vec<kYBf> y[kV];
  Vec<kBf> x[kV], g[kV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      const int c = tid + e * nt;
      if (c < nv) {
        if (has_y) y[e].load(p.y, row * p.y_stride + 8 * c);
        if (has_g) g[e].load(p.gate, row * p.gate_stride + 8 * c);
        if (has_x) x[e].load(p.x, row * p.x_stride + 8 * c);
      }
    }
  };
  int64_t row = blockIdx.x;
  fetch(row);
  for (;;) {
    F2 v[kV][4];  // y, then x'
    float inv[kV];
    if (has_y) {
      float sq[kV], s = 0.f;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        sq[e] = 0.f;
        if (tid + e * nt < nv) {
          y[e].get(v[e]);
          F2 t = v[e][0] * v[e][0];
#pragma unroll
          for (int i = 1; i < 4; ++i) t = fma2(v[e][i], v[e][i], t);
          const float2 f = un(t);
          sq[e] = f.x + f.y;
        }
        s += sq[e];
        inv[e] = 1.f;
      }
      if (has_post) {
        if (whole) {
          const float t = rsqrtf(block_sum(s, red, sums) / (float)p.D + p.eps);
#pragma unroll
          for (int e = 0; e < kV; ++e) inv[e] = t;
        } else if (in_warp) {
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            float t = sq[e];
            for (int o = gv >> 1; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            inv[e] = rsqrtf(t / (float)p.group + p.eps);
          }
        } else {
          __syncthreads();  // the last row's sums are read
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (tid + e * nt < nv) gsum[tid + e * nt] = sq[e];
          __syncthreads();
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const int c = tid + e * nt;
            float t = 0.f;
            if (c < nv)
              for (int j = c / gv * gv; j < c / gv * gv + gv; ++j) t += gsum[j];
            inv[e] = rsqrtf(t / (float)p.group + p.eps);
          }
        }
      }
    }
    F2 s2 = f2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      const int c = tid + e * nt;
      if (c >= nv) continue;
      F2 z[4];
      if (has_y) {
        F2 w[4];
        if (kLoop) weights8(fac + 8 * c, w);
        else factor(c, w);
        const F2 iv = f2(inv[e], inv[e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[e][i] = v[e][i] * (iv * w[i]);
        if (has_g) {
          g[e].get(z);
          // z sigmoid(z) before the product with v: v z may overflow where the gate is shut.
          if (p.act == ONELA_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[e][i] = v[e][i] * (z[i] * sigmoid2(z[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[e][i] = v[e][i] * sigmoid2(z[i]);
          }
        }
        if (has_x) {
          x[e].get(z);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[e][i] = v[e][i] + z[i];
        }
      } else {
        x[e].get(v[e]);
      }
      if (has_out) Vec<kBf>::store(p.x_out, row * p.D + 8 * c, v[e]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = fma2(v[e][i], v[e][i], s2);
    }
    const int64_t next = row + gridDim.x;
    if (kLoop && next < p.N) fetch(next);
    if (has_pre) {
      const float2 f = un(s2);
      const float t = rsqrtf(block_sum(f.x + f.y, red, sums) / (float)p.D + p.eps);
      const F2 tv = f2(t, t);
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const int c = tid + e * nt;
        if (c >= nv) continue;
        F2 w[4];
        weights8(kLoop ? wpre + 8 * c : p.w_pre + 8 * c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i] * (v[e][i] * tv);
        Vec<kBf>::store(p.n_out, row * p.D + 8 * c, w);
      }
    }
    if (!kLoop || next >= p.N) return;
    row = next;
  }
}

// Any D, group, stride and alignment: one CTA per row, its values in shared
// memory, element by element.
__global__ void __launch_bounds__(256) block_norm_any(BlockNormParams p) {
  extern __shared__ float buf[];  // [D] the row
  __shared__ __align__(16) float red[2][32];
  int sums = 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (tid < 64) red[tid >> 5][tid & 31] = 0.f;
  __syncthreads();
  float inv = 1.f;  // of the one group over the whole row; smaller groups are scaled in place
  if (p.y) {
    for (int c = tid; c < p.D; c += 256) buf[c] = ld(p.y, row * p.y_stride + c, p.y_bf16);
    __syncthreads();
    if (p.w_post) {
      const int groups = p.D / p.group;
      if (groups == 1) {
        float s = 0.f;
        for (int c = tid; c < p.D; c += 256) s += buf[c] * buf[c];
        s = block_sum(s, red, sums);
        inv = rsqrtf(s / (float)p.D + p.eps);
      } else {
        for (int g = warp; g < groups; g += 8) {
          float s = 0.f;
          for (int c = lane; c < p.group; c += 32) s += buf[g * p.group + c] * buf[g * p.group + c];
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const float t = rsqrtf(s / (float)p.group + p.eps);
          for (int c = lane; c < p.group; c += 32) buf[g * p.group + c] *= t;
        }
        __syncthreads();
      }
    }
  }
  float s = 0.f;
  for (int c = tid; c < p.D; c += 256) {
    float t = p.x ? ld(p.x, row * p.x_stride + c, p.bf16) : 0.f;
    if (p.y) {
      float u = buf[c];
      if (p.w_post) u = u * inv * p.w_post[c % p.group];
      if (p.gate) u *= act(ld(p.gate, row * p.gate_stride + c, p.bf16), p.act);
      u *= p.alpha;
      if (p.scale) u *= p.scale[c];
      t += u;
    }
    if (p.x_out) st(p.x_out, row * p.D + c, t, p.bf16);
    buf[c] = t;
    s += t * t;
  }
  if (p.w_pre) {
    const float t = rsqrtf(block_sum(s, red, sums) / (float)p.D + p.eps);
    for (int c = tid; c < p.D; c += 256) st(p.n_out, row * p.D + c, buf[c] * t * p.w_pre[c], p.bf16);
  }
}

template <bool kYBf, bool kBf, int kV, int kMaxThreads = 512>
cudaError_t run_vec(const BlockNormParams &p, int threads, cudaStream_t s) {
  const int gv = p.group / 8;
  const bool sums = p.y && p.w_post && p.group != p.D && !(gv <= 32 && (gv & (gv - 1)) == 0);
  const size_t gs = sums ? (size_t)p.D / 8 * 4 : 0;
  return launch_kernel(block_norm_vec<kYBf, kBf, kV, false, false, kMaxThreads>, (unsigned)p.N, threads, gs, true, s, p);
}

// Rows looping over CTAs; false if there are too few rows for the CTAs that run at once.
template <bool kYBf, bool kBf, int kV>
bool run_loop(const BlockNormParams &p, int threads, cudaStream_t s, cudaError_t &e) {
  const int gv = p.group / 8;
  const bool sums = p.y && p.w_post && p.group != p.D && !(gv <= 32 && (gv & (gv - 1)) == 0);
  const size_t smem = (size_t)p.D * 8 + (sums ? (size_t)p.D / 8 * 4 : 0);
  const int per_sm = std::max(1, std::min(std::min(1024 / threads, 32), (int)(200 * 1024 / (smem + 1024))));
  const int64_t ctas = (int64_t)kSMs * per_sm;
  if (p.N < 4 * ctas) return false;
  const bool all = p.y && p.gate && p.x && p.w_post && p.group == p.D && p.w_pre && p.x_out;
  auto f = all ? block_norm_vec<kYBf, kBf, kV, true, true> : block_norm_vec<kYBf, kBf, kV, true, false>;
  e = ensure_smem_limit((const void *)f, smem);
  if (e == cudaSuccess) e = launch_kernel(f, (unsigned)ctas, threads, smem, true, s, p);
  return true;
}

template <bool kYBf, bool kBf>
cudaError_t run_types(const BlockNormParams &p, cudaStream_t s) {
  const int nv = p.D / 8;
  auto threads = [nv](int per) { return ((nv + per - 1) / per + 31) / 32 * 32; };
  cudaError_t e;
  // Looping, two vectors a thread from 256 vectors on: fewer warps to wait for
  // at a sum (20480 rows of 4096 in bf16: 174 us with one, 158 with two).  fp32 rows
  // in flight take twice the registers: one vector up to 512.
  if (nv <= (kYBf && kBf ? 256 : 512) ? run_loop<kYBf, kBf, 1>(p, threads(1), s, e) : nv <= 1024 && run_loop<kYBf, kBf, 2>(p, threads(2), s, e))
    return e;
  if (nv <= 512) return run_vec<kYBf, kBf, 1>(p, threads(1), s);
  if (nv <= 1024) return run_vec<kYBf, kBf, 2>(p, threads(2), s);
  if (nv <= 2048) return run_vec<kYBf, kBf, 4>(p, threads(4), s);
  return run_vec<kYBf, kBf, 4, 1024>(p, threads(4), s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t s) {
  auto addr = [](const void *q) { return (uint64_t) reinterpret_cast<uintptr_t>(q); };
  const uint64_t ptrs = addr(p.y) | addr(p.gate) | addr(p.x) | addr(p.w_post) | addr(p.scale) | addr(p.w_pre) |
                        addr(p.x_out) | addr(p.n_out);
  const uint64_t strides = (p.y ? (uint64_t)p.y_stride : 0) | (p.gate ? (uint64_t)p.gate_stride : 0) |
                           (p.x ? (uint64_t)p.x_stride : 0);
  const bool vec = p.D % 8 == 0 && p.group % 8 == 0 && (ptrs & 15) == 0 && strides % 8 == 0;
  if (vec) {
    if (p.y_bf16) return p.bf16 ? run_types<true, true>(p, s) : run_types<true, false>(p, s);
    return p.bf16 ? run_types<false, true>(p, s) : run_types<false, false>(p, s);
  }
  const size_t smem = (size_t)p.D * 4;
  cudaError_t e = ensure_smem_limit((const void *)block_norm_any, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(block_norm_any, (unsigned)p.N, 256, smem, true, s, p);
}

}  // namespace onela
