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

#include "../../include/onela.h"
#include "internal.h"

namespace onela {
namespace {

__device__ __forceinline__ float ld(const void *p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st(void *p, int64_t i, float x, int bf16) {
  if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<float *>(p)[i] = x;
}

// Eight consecutive elements as floats; 16-byte aligned rows.
__device__ __forceinline__ void ld8(const void *p, int64_t i, int bf16, float (&v)[8]) {
  if (bf16) {
    union { uint4 u; __nv_bfloat162 h[4]; } a;
    a.u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(a.h[e]);
      v[2 * e] = f.x;
      v[2 * e + 1] = f.y;
    }
  } else {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
__device__ __forceinline__ void st8(void *p, int64_t i, int bf16, const float (&v)[8]) {
  if (bf16) {
    union { uint4 u; __nv_bfloat162 h[4]; } a;
#pragma unroll
    for (int e = 0; e < 4; ++e) a.h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = a.u;
  } else {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float act(float z, int kind) {
  const float s = 1.f / (1.f + __expf(-z));
  return kind == ONELA_ACT_SILU ? z * s : (kind == ONELA_ACT_SIGMOID ? s : z);
}

// Block-wide sum; every thread gets it.  red holds one float per warp.
__device__ __forceinline__ float block_sum(float x, float *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One CTA per row, kV vectors of 8 channels per thread (vector e of thread t
// holds channels 8 (t + e * threads) ..).
template <int kV>
__global__ void __launch_bounds__(1024) block_norm_vec(BlockNormParams p) {
  extern __shared__ float gsum[];  // per vector, its sum of squares (group norms)
  __shared__ float red[32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t row = blockIdx.x;
  const int nv = p.D / 8;
  float v[kV][8], xr[kV][8], gt[kV][8];
#pragma unroll
  for (int e = 0; e < kV; ++e) {
    const int c = tid + e * nt;
    if (c < nv) {
      if (p.y) ld8(p.y, row * p.y_stride + 8 * c, p.y_bf16, v[e]);
      if (p.x) ld8(p.x, row * p.x_stride + 8 * c, p.bf16, xr[e]);
      if (p.gate) ld8(p.gate, row * p.gate_stride + 8 * c, p.bf16, gt[e]);
    }
  }
  if (p.y) {
    float sq[kV];
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      sq[e] = 0.f;
      if (tid + e * nt < nv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[e] += v[e][i] * v[e][i];
      }
      s += sq[e];
    }
    float inv[kV];
    if (p.w_post) {
      if (p.group == p.D) {
        const float t = rsqrtf(block_sum(s, red) / (float)p.D + p.eps);
#pragma unroll
        for (int e = 0; e < kV; ++e) inv[e] = t;
      } else {
        const int gv = p.group / 8;
#pragma unroll
        for (int e = 0; e < kV; ++e)
          if (tid + e * nt < nv) gsum[tid + e * nt] = sq[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          const int c = tid + e * nt;
          float t = 0.f;
          if (c < nv) {
            const int g0 = c / gv * gv;
            for (int j = 0; j < gv; ++j) t += gsum[g0 + j];
          }
          inv[e] = rsqrtf(t / (float)p.group + p.eps);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      const int c = tid + e * nt;
      if (c >= nv) continue;
      float wp[8], sc[8];
      if (p.w_post) ld8(p.w_post, 8 * c % p.group, 0, wp);
      if (p.scale) ld8(p.scale, 8 * c, 0, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u = v[e][i];
        if (p.w_post) u = u * inv[e] * wp[i];
        if (p.gate) u *= act(gt[e][i], p.act);
        u *= p.alpha;
        if (p.scale) u *= sc[i];
        v[e][i] = p.x ? xr[e][i] + u : u;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kV; ++e)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[e][i] = xr[e][i];
  }
  if (p.x_out) {
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (tid + e * nt < nv) st8(p.x_out, row * p.D + 8 * (tid + e * nt), p.bf16, v[e]);
  }
  if (p.w_pre) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (tid + e * nt < nv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[e][i] * v[e][i];
      }
    const float t = rsqrtf(block_sum(s, red) / (float)p.D + p.eps);
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      const int c = tid + e * nt;
      if (c >= nv) continue;
      float w[8];
      ld8(p.w_pre, 8 * c, 0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= v[e][i] * t;
      st8(p.n_out, row * p.D + 8 * c, p.bf16, w);
    }
  }
}

// Any D, group, stride and alignment: one CTA per row, its values in shared
// memory, element by element.
__global__ void __launch_bounds__(256) block_norm_any(BlockNormParams p) {
  extern __shared__ float buf[];  // [D] the row, then [D / group] the groups' factors
  __shared__ float red[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  float *inv = buf + p.D;
  if (p.y) {
    for (int c = tid; c < p.D; c += 256) buf[c] = ld(p.y, row * p.y_stride + c, p.y_bf16);
    __syncthreads();
    if (p.w_post) {
      const int groups = p.D / p.group;
      if (groups == 1) {
        float s = 0.f;
        for (int c = tid; c < p.D; c += 256) s += buf[c] * buf[c];
        s = block_sum(s, red);
        if (tid == 0) inv[0] = rsqrtf(s / (float)p.D + p.eps);
      } else {
        for (int g = warp; g < groups; g += 8) {
          float s = 0.f;
          for (int c = lane; c < p.group; c += 32) s += buf[g * p.group + c] * buf[g * p.group + c];
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) inv[g] = rsqrtf(s / (float)p.group + p.eps);
        }
      }
      __syncthreads();
    }
  }
  float s = 0.f;
  for (int c = tid; c < p.D; c += 256) {
    float t = p.x ? ld(p.x, row * p.x_stride + c, p.bf16) : 0.f;
    if (p.y) {
      float u = buf[c];
      if (p.w_post) u = u * inv[c / p.group] * p.w_post[c % p.group];
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
    const float t = rsqrtf(block_sum(s, red) / (float)p.D + p.eps);
    for (int c = tid; c < p.D; c += 256) st(p.n_out, row * p.D + c, buf[c] * t * p.w_pre[c], p.bf16);
  }
}

template <int kV>
cudaError_t run_vec(const BlockNormParams &p, int threads, cudaStream_t s) {
  const size_t smem = p.y && p.w_post && p.group != p.D ? (size_t)p.D / 8 * 4 : 0;
  block_norm_vec<kV><<<(unsigned)p.N, threads, smem, s>>>(p);
  return cudaGetLastError();
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
    const int nv = p.D / 8;
    auto threads = [nv](int per) { return ((nv + per - 1) / per + 31) / 32 * 32; };
    if (nv <= 512) return run_vec<1>(p, threads(1), s);
    if (nv <= 1024) return run_vec<2>(p, threads(2), s);
    return run_vec<4>(p, threads(4), s);
  }
  const size_t smem = (size_t)(p.D + p.D / p.group) * 4;
  cudaError_t e = ensure_smem_limit((const void *)block_norm_any, smem);
  if (e != cudaSuccess) return e;
  block_norm_any<<<(unsigned)p.N, 256, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace onela
