// Attention over a paged cache for few query rows per key-value head (W * G
// <= 16, the single-token decode of grouped heads): bf16, d in {64, 128, 256}.
//
// Every cached K and V row is used by at most 16 query rows, 4 d * 16
// operations for 4 d bytes, so what bounds it is reading the cache; the work
// is kept in the shadow of the loads.  The 16 rows are one m16 tile of the
// warp-wide matrix instruction (a tcgen05 tile of 128 rows would be 7/8 empty): S = Q
// K^T from shared memory by ldmatrix, the softmax on the accumulators in
// registers, O += P V with P straight from those registers.  Four warps each
// run a ring of 16-token tiles filled by 16-byte asynchronous copies, on their
// own (no block barrier inside a piece), and join through shared memory at
// the end of a piece.
//
// P enters the second product as two bf16 terms (p = hi + lo, 16 bits of p):
// the tensor cores have the time, and the weights then lose nothing that
// shows next to the rounding of o.  The sum of weights is the sum of the
// unrounded p.
#include "attention.h"

#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

constexpr int kWarps = 4, kThreads = 128, kTok = 16;

template <int D>
struct Cfg {
  static constexpr int kRow = D * 2;                 // bytes of a K or V row
  static constexpr int kTile = kTok * kRow;          // one warp's K (or V) tile
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kSmem = kWarps * kStages * 2 * kTile;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) attn_narrow(AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanSmem plan;
  __shared__ float2 wml[kWarps][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv;
  ptx::pdl_launch_dependents();
  PlanWalk walk;
  walk.begin<kThreads>(p, plan, blockIdx.x / p.Hkv);

  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
  const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
  uint8_t *ring = smem + warp * (C::kStages * 2 * C::kTile);
  const uint32_t ring_u32 = ptx::smem_u32(ring);
  const int g = lane >> 2, t4 = lane & 3;

  while (walk.next(p)) {
    const int r = walk.r, lo = walk.lo, hi = walk.hi;
    if (p.direct && h == 0 && tid == 0 && p.lengths[r] != hi) set_status(p.status, kStatusLength);
    const int32_t *tab = p.table + (int64_t)r * p.row_pages;
    // This warp's tiles start at lo + 16 (warp + 4 i).
    const int first = lo + warp * kTok;
    const int n = first < hi ? (hi - first + 63) / 64 : 0;

    // The (token, head) row of this lane's token of tile i, as a byte offset; -1 if it has none.
    auto row_of = [&](int i) -> int64_t {
      const int pos = first + 64 * i + (lane & 15);
      if (i >= n || pos >= hi) return -1;
      const int pg = tab[pos / p.page];
      if (pg < 0 || pg >= p.pages) {
        set_status(p.status, kStatusPage);
        return -1;
      }
      return (((int64_t)pg * p.Hkv + h) * p.page + pos % p.page) * C::kRow;
    };
    // Copies of tile i into its stage: zeros for tokens that are not there.
    auto issue = [&](int i, int64_t row) {
      if (i < n) {
        constexpr int kPer = C::kRow / 16;  // 16-byte chunks of a row
        uint8_t *kd = ring + (i % C::kStages) * 2 * C::kTile, *vd = kd + C::kTile;
#pragma unroll
        for (int e = 0; e < kTok * kPer / 32; ++e) {
          const int at = e * 32 + lane, tok = at / kPer, ch = at % kPer;
          const int64_t off = __shfl_sync(0xffffffffu, row, tok);
          const uint32_t to = tok * C::kRow + ((ch ^ (tok & 7)) << 4);
          const int64_t src = (off < 0 ? 0 : off) + ch * 16;
          ptx::cp_async16(kd + to, kp + src, off < 0 ? 0 : 16);
          ptx::cp_async16(vd + to, vp + src, off < 0 ? 0 : 16);
        }
      }
      ptx::cp_async_commit();
    };

    uint32_t live[C::kStages];  // by stage: the tokens that are there
    int64_t row = row_of(0);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      live[i] = __ballot_sync(0xffffffffu, row >= 0);
      issue(i, row);
      row = row_of(i + 1);
    }
    live[C::kStages - 1] = 0;

    // Q as the A operand, rows past M zero.
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = g + (e & 1) * 8, c = ks * 16 + t4 * 2 + (e >> 1) * 8;
        qf[ks][e] = 0;
        if (m < p.M) {
          const int w = m / p.G, hq = h * p.G + m % p.G;
          qf[ks][e] = *reinterpret_cast<const uint32_t *>(q + ((int64_t)r * p.W + w) * p.q_stride + (int64_t)hq * D + c);
        }
      }

    float acc[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float mx[2] = {-CUDART_INF_F, -CUDART_INF_F}, sum[2] = {0.f, 0.f};

    for (int i0 = 0; i0 < n; i0 += C::kStages) {
#pragma unroll
      for (int st = 0; st < C::kStages; ++st) {
        const int i = i0 + st;
        if (i >= n) break;
        cp_wait<C::kStages - 2>();
        __syncwarp();
        const uint32_t k_u32 = ring_u32 + st * 2 * C::kTile, v_u32 = k_u32 + C::kTile;
        const uint32_t here = live[st];
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
          const int tok = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
          const uint32_t base = k_u32 + tok * C::kRow;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldsm4(b, base + (((ks * 2 + half) ^ (tok & 7)) << 4));
            mma16816(s[0], qf[ks], b[0], b[1]);
            mma16816(s[1], qf[ks], b[2], b[3]);
          }
        }
        // Columns of this thread: tokens 8 j + 2 t4 + {0, 1}; rows g and g + 8.
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 8 * j + 2 * t4 + (e & 1);
            s[j][e] = (here >> tok) & 1 ? s[j][e] * p.scale_log2 : -CUDART_INF_F;
            top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
          }
        if (p.scores) {
          const int pos = first + 64 * i;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = g + (e >> 1) * 8, at = pos + 8 * j + 2 * t4 + (e & 1);
              if (m < p.M && at < hi) p.scores[(((int64_t)r * p.Hkv + h) * p.M + m) * p.cap + at] = s[j][e];
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        }
        if (__any_sync(0xffffffffu, top[0] > mx[0] || top[1] > mx[1])) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mnew = fmaxf(mx[e], top[e]);
            f[e] = exp2_sub(mx[e], mnew);
            mx[e] = mnew;
            sum[e] *= f[e];
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            acc[j][0] *= f[0];
            acc[j][1] *= f[0];
            acc[j][2] *= f[1];
            acc[j][3] *= f[1];
          }
        }
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = exp2_sub(s[j][2 * e], mx[e]), b = exp2_sub(s[j][2 * e + 1], mx[e]);
            sum[e] += a + b;
            const uint32_t hi2 = pack(a, b);
            ph[2 * j + e] = hi2;
            pl[2 * j + e] = pack(a - __uint_as_float(hi2 << 16), b - __uint_as_float(hi2 & 0xffff0000u));
          }
        {
          const int tok = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
          const uint32_t base = v_u32 + tok * C::kRow;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldsm4_t(b, base + (((j * 2 + half) ^ (tok & 7)) << 4));
            mma16816(acc[2 * j], ph, b[0], b[1]);
            mma16816(acc[2 * j + 1], ph, b[2], b[3]);
            mma16816(acc[2 * j], pl, b[0], b[1]);
            mma16816(acc[2 * j + 1], pl, b[2], b[3]);
          }
        }
        __syncwarp();  // the stage filled next was read in the previous round
        // Stage (st + kStages - 1) % kStages, read in the previous round, takes tile i + kStages - 1.
        live[(st + C::kStages - 1) % C::kStages] = __ballot_sync(0xffffffffu, row >= 0);
        issue(i + C::kStages - 1, row);
        row = row_of(i + C::kStages);
      }
    }
    cp_wait<0>();

    // Join the four warps: outputs and (maximum, sum) through shared memory.
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      if (t4 == 0) wml[warp][g + 8 * e] = make_float2(mx[e], sum[e]);
    }
    __syncthreads();  // every warp is done with its ring
    float *buf = reinterpret_cast<float *>(smem) + warp * 16 * D;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (g + 8 * e < p.M)
          *reinterpret_cast<float2 *>(buf + (g + 8 * e) * D + 8 * j + 2 * t4) = make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
    __syncthreads();
    for (int at = tid; at < p.M * (D / 4); at += kThreads) {
      const int m = at / (D / 4), c = at % (D / 4) * 4;
      float2 ml[kWarps];
      float top = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = wml[w][m];
        top = fmaxf(top, ml[w].x);
      }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_sub(ml[w].x, top);
        const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (w * 16 + m) * D + c);
        l += ml[w].y * f;
        o.x += x.x * f;
        o.y += x.y * f;
        o.z += x.z * f;
        o.w += x.w * f;
      }
      if (p.direct) {
        const int64_t orow = ((int64_t)r * p.W + m / p.G) * p.Hq + h * p.G + m % p.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat162 *out = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.o) + orow * D + c);
        out[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        out[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        if (c == 0 && p.lse) p.lse[orow] = l == 0.f ? -CUDART_INF_F : (top + log2f(l)) * kLn2;
      } else {
        const int64_t pr = part_row(p, walk.slot, h, m);
        *reinterpret_cast<float4 *>(p.part_o + pr * D + c) = o;
        if (c == 0) p.part_ml[pr] = make_float2(top, l);
      }
    }
    __syncthreads();  // the ring is free for the next piece
  }
}

template <int D>
cudaError_t run(const AttnParams &p, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit((const void *)attn_narrow<D>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_narrow<D>, (unsigned)(p.parts * p.Hkv), kThreads, Cfg<D>::kSmem, false, s, p);
}

}  // namespace

cudaError_t launch_attn_narrow(const AttnParams &p, cudaStream_t s) {
  if (p.d == 64) return run<64>(p, s);
  return p.d == 128 ? run<128>(p, s) : run<256>(p, s);
}

}  // namespace onela
