// Attention over a paged cache for few query rows per key-value head (W * G
// <= 16, the single-token decode of grouped heads): bf16, d in {64, 128, 256}.
//
// Every cached K and V row is used by at most 16 query rows, 4 d * 16
// operations for 4 d bytes, so what bounds it is reading the cache; the work
// has to stay in the shadow of the loads.  A tcgen05 tile of 128 rows would be
// 7/8 empty; here the tokens are the long side of the warp-wide matrix
// instruction (m16n8k16) and the query rows its 8 columns (one or two of them, kNT):
//     S^T = K Q^T   (16 tokens x 8 rows, K by ldmatrix),
//     O^T += V^T P^T (16 columns of d x 8 rows, V by transposing ldmatrix),
// P^T from the accumulators of S^T by an in-register 8 x 8 transpose.  (With the
// rows as the 16-row side half of every product was padding: 583
// instructions a tile of 16 tokens, 47 instead of 36 us for 32 ragged requests
// of up to 5120 tokens.)  Four warps each run
// a ring of 16-token tiles filled by 16-byte asynchronous copies, on their
// own (no block barrier inside a piece), and join through shared memory at
// the end of a piece.
//
// P enters the second product as two bf16 terms (p = hi + lo, 16 bits of p):
// the tensor cores have the time, and the weights then lose nothing that
// shows next to the rounding of o.  The sum of weights is the sum of the
// unrounded p.  The maximum that weights are taken against moves only when
// the row's maximum grew by more than 2^8 (kSlack).
#include "attention.h"

#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

constexpr int kWarps = 4, kThreads = 128, kTok = 16;

template <int D>
struct Cfg {
  static constexpr int kRow = D * 2;         // bytes of a K or V row
  static constexpr int kTile = kTok * kRow;  // one warp's K (or V) tile
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 2 : 3;
  static constexpr int kSmem = kWarps * kStages * 2 * kTile;
  static constexpr int kCtas = D == 256 ? 1 : 3;  // per SM
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
// The 8 x 8 matrix of 16-bit elements that a warp holds (row lane / 4, columns 2 (lane % 4) + {0, 1}), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

template <int D, int kNT>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas) attn_narrow(const __grid_constant__ AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanSmem plan;
  __shared__ float2 wml[kWarps][8 * kNT];
  __shared__ uint32_t live[kWarps][C::kStages];  // by warp and stage: the tile's tokens that are there
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  PlanWalk walk;
  walk.begin<kThreads>(p, plan, blockIdx.x / p.Hkv);

  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
  const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
  uint8_t *ring = smem + warp * (C::kStages * 2 * C::kTile);
  const uint32_t ring_u32 = ptx::smem_u32(ring);
  const int g = lane >> 2, t4 = lane & 3;
  const bool one_page = (p.page & 15) == 0;  // a tile lies on one page
  constexpr int kPer = C::kRow / 16;         // 16-byte chunks of a row

  while (walk.next(p)) {
    const int r = walk.r, lo = walk.lo, hi = walk.hi;
    if (p.direct && h == 0 && tid == 0 && p.lengths[r] != hi) set_status(p.status, kStatusLength);
    const int32_t *tab = p.table + (int64_t)r * p.row_pages;
    // This warp's tiles start at lo + 16 (warp + 4 i).
    const int first = lo + warp * kTok;
    const int n = first < hi ? (hi - first + 63) / 64 : 0;

    // The page and the place on it of this lane's token of tile i, or of the
    // tile's first when it lies on one page.  The entry is looked at a tile
    // later, so that no warp waits for the table.
    int pg = 0, place = 0;
    auto look = [&](int i) {
      const int pos = first + 64 * i + (one_page ? 0 : lane & 15);
      if (i < n && pos < hi) {
        const int at = pos / p.page;
        pg = tab[at];
        place = pos - at * p.page;
      }
    };
    // Copies of tile i into stage st: zeros for tokens that are not there.
    auto issue = [&](int i, int st) {
      if (i < n) {
        // Byte offset of the (token, head) row in the pools, -1 if it is not there.
        int64_t row = -1;
        if (first + 64 * i + (one_page ? 0 : lane & 15) < hi) {
          if (pg >= 0 && pg < p.pages) row = (((int64_t)pg * p.Hkv + h) * p.page + place) * C::kRow;
          else set_status(p.status, kStatusPage);
        }
        uint8_t *kd = ring + st * 2 * C::kTile, *vd = kd + C::kTile;
        const int left = hi - (first + 64 * i);
        if (one_page) {
          const int cnt = row < 0 ? 0 : left;
          const int64_t src = row < 0 ? 0 : row + lane * 16;
          if (lane == 0) live[warp][st] = cnt >= 16 ? 0xffffu : (1u << cnt) - 1u;
#pragma unroll
          for (int e = 0; e < kTok * kPer / 32; ++e) {
            const int at = e * 32 + lane, tok = at / kPer, ch = at % kPer;
            const uint32_t to = tok * C::kRow + ((ch ^ (tok & 7)) << 4);
            const bool in = tok < cnt;
            const int64_t from = in ? src + e * 512 : 0;
            ptx::cp_async16(kd + to, kp + from, in ? 16 : 0);
            ptx::cp_async16(vd + to, vp + from, in ? 16 : 0);
          }
        } else {
          const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
          if (lane == 0) live[warp][st] = bits;
#pragma unroll 2
          for (int e = 0; e < kTok * kPer / 32; ++e) {
            const int at = e * 32 + lane, tok = at / kPer, ch = at % kPer;
            const int64_t off = __shfl_sync(0xffffffffu, row, tok);
            const uint32_t to = tok * C::kRow + ((ch ^ (tok & 7)) << 4);
            const int64_t src = off < 0 ? 0 : off + ch * 16;
            ptx::cp_async16(kd + to, kp + src, off < 0 ? 0 : 16);
            ptx::cp_async16(vd + to, vp + src, off < 0 ? 0 : 16);
          }
        }
      }
      ptx::cp_async_commit();
    };

    look(0);
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) {
      issue(i, i);
      look(i + 1);
    }

    // Q^T as the B operand (column = query row g + 8 nt), rows past M zero.
    uint32_t qf[kNT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int m = g + 8 * nt;
      const __nv_bfloat16 *src = q;
      if (m < p.M) src += ((int64_t)r * p.W + m / p.G) * p.q_stride + (int64_t)(h * p.G + m % p.G) * D + t4 * 2;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[nt][ks][e] = m < p.M ? *reinterpret_cast<const uint32_t *>(src + ks * 16 + e * 8) : 0;
    }

    // O^T: rows of d (16 j + g, + 8), columns = query rows 8 nt + 2 t4 + {0, 1}.
    float acc[kNT][D / 16][4];
    float mref[kNT][2], sum[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.f;
      mref[nt][0] = mref[nt][1] = -CUDART_INF_F;
      sum[nt][0] = sum[nt][1] = 0.f;
    }

    int st = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      {  // The stage read in the last round takes tile i + kStages - 1.
        const int fs = st == 0 ? C::kStages - 1 : st - 1;
        issue(i + C::kStages - 1, fs);
        look(i + C::kStages);
      }
      const uint32_t k_u32 = ring_u32 + st * 2 * C::kTile, v_u32 = k_u32 + C::kTile;
      const uint32_t here = live[warp][st];
      st = st + 1 == C::kStages ? 0 : st + 1;
      // S^T: tokens g, g + 8; query rows 8 nt + 2 t4 + {0, 1}.
      float s[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      {
        const int tok = lane & 15, half = lane >> 4;
        const uint32_t base = k_u32 + tok * C::kRow;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t a[4];
          ldsm4(a, base + (((ks * 2 + half) ^ (tok & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma16816(s[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
        }
      }
      if (here != 0xffffu) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((here >> (g + 8 * (e >> 1))) & 1)) s[nt][e] = -CUDART_INF_F;
      }
      if (p.scores) {
        const int at = first + 64 * i + g;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 8 * nt + 2 * t4 + (e & 1), pos = at + 8 * (e >> 1);
            if (m < p.M && pos < hi)
              p.scores[(((int64_t)r * p.Hkv + h) * p.M + m) * p.cap + pos] = s[nt][e];
          }
      }
      // The rows' maxima over the tile, of all lanes with the same t4.
      float top[kNT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
          top[nt][e] = t;
          grow = grow || (t - mref[nt][e]) * p.scale_log2 > kSlack;  // from -inf: always, unless there is nothing yet
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mnew = fmaxf(mref[nt][e], top[nt][e]), f = exp2_sub(mref[nt][e], mnew, p.scale_log2);
            mref[nt][e] = mnew;
            sum[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[nt][j][e] *= f;
              acc[nt][j][e + 2] *= f;
            }
          }
      }
      // P^T as the B operand, in two terms.
      uint32_t ph[kNT][2], pl[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const float o0 = mref[nt][0] == -CUDART_INF_F ? 0.f : mref[nt][0];
        const float o1 = mref[nt][1] == -CUDART_INF_F ? 0.f : mref[nt][1];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float a = ex2((s[nt][2 * t] - o0) * p.scale_log2), b = ex2((s[nt][2 * t + 1] - o1) * p.scale_log2);
          sum[nt][0] += a;
          sum[nt][1] += b;
          const uint32_t hi2 = pack_bf16(a, b);
          ph[nt][t] = transpose8(hi2);
          pl[nt][t] = transpose8(pack_bf16(a - __uint_as_float(hi2 << 16), b - __uint_as_float(hi2 & 0xffff0000u)));
        }
      }
      {
        const int tok = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
        const uint32_t base = v_u32 + tok * C::kRow;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t a[4];
          ldsm4_t(a, base + (((j * 2 + half) ^ (tok & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma16816(acc[nt][j], a, ph[nt][0], ph[nt][1]);
            mma16816(acc[nt][j], a, pl[nt][0], pl[nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
    }
    cp_wait<0>();

    // Join the four warps: outputs and (maximum, sum) through shared memory.
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = sum[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (g == 0) wml[warp][8 * nt + 2 * t4 + e] = make_float2(mref[nt][e], t);
      }
    __syncthreads();  // every warp is done with its ring
    // [warp][row][D + 4]: 4 floats of padding keep the columns of a fragment on different banks.
    constexpr int kLd = D + 4;
    float *all = reinterpret_cast<float *>(smem), *buf = all + warp * (8 * kNT * kLd);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) buf[(8 * nt + 2 * t4 + (e & 1)) * kLd + 16 * j + g + 8 * (e >> 1)] = acc[nt][j][e];
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
        const float f = exp2_sub(ml[w].x, top, p.scale_log2);
        const float4 x = *reinterpret_cast<const float4 *>(all + (w * 8 * kNT + m) * kLd + c);
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
        if (c == 0 && p.lse) p.lse[orow] = l == 0.f ? -CUDART_INF_F : (top * p.scale_log2 + log2f(l)) * kLn2;
      } else {
        const int64_t pr = part_row(p, walk.slot, h, m);
        *reinterpret_cast<float4 *>(p.part_o + pr * D + c) = o;
        if (c == 0) p.part_ml[pr] = make_float2(top, l);
      }
    }
    __syncthreads();  // the ring is free for the next piece
  }
}

template <int D, int kNT>
cudaError_t run(const AttnParams &p, cudaStream_t s) {
  static_assert(kWarps * 8 * kNT * (D + 4) * 4 <= Cfg<D>::kSmem, "the warps' outputs go through the ring");
  const cudaError_t e = ensure_smem_limit((const void *)attn_narrow<D, kNT>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_narrow<D, kNT>, (unsigned)(p.parts * p.Hkv), kThreads, Cfg<D>::kSmem, true, s, p);
}

}  // namespace

int attn_narrow_ctas(int d) { return d == 64 ? Cfg<64>::kCtas : d == 128 ? Cfg<128>::kCtas : Cfg<256>::kCtas; }

cudaError_t launch_attn_narrow(const AttnParams &p, cudaStream_t s) {
  if (p.d == 64) return p.M <= 8 ? run<64, 1>(p, s) : run<64, 2>(p, s);
  if (p.d == 128) return p.M <= 8 ? run<128, 1>(p, s) : run<128, 2>(p, s);
  return p.M <= 8 ? run<256, 1>(p, s) : run<256, 2>(p, s);
}

}  // namespace onela
