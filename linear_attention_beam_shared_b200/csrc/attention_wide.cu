// Attention over a paged cache for many query rows per key-value head: the
// beams of a request share its prompt, so W * G rows (1024 for 256 beams of
// 4 grouped heads) read the same K and V.  bf16, d in {64, 128, 256}.
//
// At 128 rows per tile a K and V row is used 128 times for every read, so the
// matrix products (4 d operations per row and token) and the exponentials (one per
// row and token, 16 a clock on an SM) bound it: at d = 128 both take about 512
// clocks for 128 rows x 64 tokens.  Both products run on tcgen05: S = Q K^T
// with both operands in shared memory, O += P V with P in tensor memory, where the
// softmax warps write it over the scores they read, and V as it lies in the
// cache (token rows, an MN-major B operand).  O stays in tensor memory.
//
// Two groups of four softmax warps (thread = row) work on two score buffers, so that one group's exponentials
// overlap the other's products.  The groups take the two
// halves of 256 rows (kSub = 2, K and V read once for both) or, with at most
// 128 rows, every other token tile of the same rows (kSub = 1), each with its own O
// and its own result slot.  At d = 256 O fills half of the tensor memory,
// so one group works through both score buffers.
//
// The running maximum that weights are taken against moves only when a row's
// maximum grew by more than 2^8 (scores in log2 units): weights then stay
// below 2^8, exact in range for bf16 and fp32 alike, and O is rescaled rarely.
// P is rounded to bf16 (2^-8 relative per weight at most, of the size of the
// rounding of o itself); its sum is that of the unrounded weights, in fp32.
//
// Four warps gather the K and V rows with 16-byte asynchronous copies through
// the page table into a ring of two K and two V tiles, zeros for tokens
// that are not there; one thread issues the products.  Every wait is bounded:
// one that runs out sets ONELA_STATUS_TIMEOUT and the results become NaN.
#include "attention.h"

#include "../../include/onela.h"
#include "internal.h"
#include "sm100_ptx.h"

namespace onela {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;  // bound of every wait
constexpr float kSlack = 8.f;                // growth of the maximum, in log2, before O is rescaled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;  // scores behind the outputs in tensor memory

template <int D, int kSub>
struct Cfg {
  static constexpr int TT = D == 256 ? 64 : 128;      // tokens per tile
  static constexpr int kGroups = D == 256 ? 1 : 2;    // softmax groups
  static constexpr int kSoft = kGroups * 128;
  static constexpr int kThreads = kSoft + 128 + 32;
  static constexpr int kQ = 128 * D * 2;              // bytes of 128 Q rows
  static constexpr int kTile = TT * D * 2;            // bytes of a K or V tile
  static constexpr int oK = kSub * kQ, oV = oK + 2 * kTile, oEnd = oV + 2 * kTile;
  // Above half of an SM's shared memory, so that one CTA has the SM (and its
  // tensor memory) for itself.
  static constexpr int kSmem = oEnd + 1024 < 120 * 1024 ? 120 * 1024 : oEnd + 1024;
};

struct Shared {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t s[2], p[2], pv[2];
  uint64_t q, done;
  uint32_t tmem;
  uint32_t mask[4][4];  // by K tile (ring of 4): the tokens that are there
  PlanSmem plan;
};

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Wait unless a wait of this thread has run out before.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &dead) {
  if (!dead && !ptx::mbar_wait(bar, parity, kWaitNs)) dead = true;
}
// The same by a whole warp, which goes on together.
__device__ __forceinline__ void wait_warp(uint64_t *bar, uint32_t parity, bool &dead) {
  wait(bar, parity, dead);
  __syncwarp();
}

template <int D, int kSub>
__global__ void __launch_bounds__(Cfg<D, kSub>::kThreads, 1) attn_wide(AttnParams p) {
  using C = Cfg<D, kSub>;
  constexpr int TT = C::TT, G = C::kGroups;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = ptx::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rt = blockIdx.x % p.row_tiles, ch = blockIdx.x / p.row_tiles;
  const int h = ch % p.Hkv, part = ch / p.Hkv;
  const int m0 = rt * (128 * kSub);

  constexpr int kMmaWarp = C::kSoft / 32 + 4;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh.kfull[i], 4);
      ptx::mbar_init(&sh.vfull[i], 4);
      ptx::mbar_init(&sh.kempty[i], 1);
      ptx::mbar_init(&sh.vempty[i], 1);
      ptx::mbar_init(&sh.s[i], 1);
      ptx::mbar_init(&sh.p[i], 128);
      ptx::mbar_init(&sh.pv[i], 1);
    }
    ptx::mbar_init(&sh.q, C::kSoft);
    ptx::mbar_init(&sh.done, 1);
    ptx::mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::pdl_launch_dependents();
  PlanWalk walk;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  walk.begin<C::kThreads>(p, sh.plan, part);
  const uint32_t tmem = sh.tmem;
  bool dead = false;

  if (warp < C::kSoft / 32) {
    // ------------------------------------------------------------- softmax
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;  // thread = query row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int m = m0 + (kSub == 2 ? grp * 128 : 0) + row;
    uint32_t ns[2] = {0, 0};  // jobs done on each score buffer
    uint32_t tile0 = 0;       // K tiles of earlier pieces (the mask ring runs on)
    while (walk.next(p)) {
      const int r = walk.r;
      const int nt = (walk.hi - walk.lo + TT - 1) / TT, nj = nt * kSub;
      // Every product of the last piece is done (each group waited for its
      // own): Q may be replaced.
      ptx::bar_sync(1, C::kSoft);
      if (kSub == 2 || grp == 0) {
        uint8_t *qd = smem + (kSub == 2 ? grp * C::kQ : 0);
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q);
        if (m < p.M) src += ((int64_t)r * p.W + m / p.G) * p.q_stride + (int64_t)(h * p.G + m % p.G) * D;
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (m < p.M) x = __ldg(reinterpret_cast<const uint4 *>(src) + c);
          *reinterpret_cast<uint4 *>(qd + (c >> 3) * 16384 + ptx::swz128(row, c & 7)) = x;
        }
      }
      ptx::fence_proxy_async();
      ptx::mbar_arrive(&sh.q);

      float mref = -CUDART_INF_F, sum = 0.f;
      bool any = false;  // this group has a product in O
      const uint32_t o_t = tmem + lanes + (G == 2 ? grp * 128 : 0);
      for (int j = G == 2 ? grp : 0; j < nj; j += G) {
        const int b = j & 1, tile = kSub == 2 ? j >> 1 : j;
        const uint32_t s_t = tmem + lanes + kSCol + b * TT;
        wait_warp(&sh.s[b], ns[b] & 1, dead);
        ++ns[b];
        ptx::tc_fence_after();
        uint32_t msk[TT / 32];
        bool full = true;
#pragma unroll
        for (int e = 0; e < TT / 32; ++e) {
          msk[e] = TT == 128 ? sh.mask[(tile0 + tile) & 3][e]
                             : sh.mask[(tile0 + tile) & 3][2 * e] | (sh.mask[(tile0 + tile) & 3][2 * e + 1] << 16);
          full = full && msk[e] == 0xffffffffu;
        }
        // Pass 1: the row's maximum over the tile.
        float top = -CUDART_INF_F;
#pragma unroll
        for (int e = 0; e < TT / 32; ++e) {
          float x[32];
          ptx::tmem_ld32(s_t + e * 32, x);
          ptx::tmem_ld_wait();
          if (full) {
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, x[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, (msk[e] >> i) & 1 ? x[i] : -CUDART_INF_F);
          }
        }
        top *= p.scale_log2;
        // Move the reference when the maximum outgrew it (or on the first tile).
        const bool grow = top > mref + kSlack || (mref == -CUDART_INF_F && top > mref);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? exp2_sub(mref, top) : 1.f;
          if (any) {
            // The last product into O must be done: at d = 256 it is that of
            // the other score buffer; otherwise the scores' own order says so.
            if (G == 1) wait_warp(&sh.pv[b ^ 1], (ns[b ^ 1] - 1) & 1, dead);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              float x[16];
              uint32_t y[16];
              ptx::tmem_ld16(o_t + e * 16, x);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * f);
              ptx::tmem_st<16>(o_t + e * 16, y);
            }
          }
          if (grow) {
            sum *= f;
            mref = top;
          }
        }
        any = true;
        // Pass 2: the weights, over the scores' own columns.
        const float off = mref == -CUDART_INF_F ? 0.f : mref;
        float part_sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < TT / 32; ++e) {
          float x[32];
          uint32_t y[16];
          ptx::tmem_ld32(s_t + e * 32, x);
          ptx::tmem_ld_wait();
          if (full) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = exp2f(fmaf(x[i], p.scale_log2, -off));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (msk[e] >> i) & 1 ? exp2f(fmaf(x[i], p.scale_log2, -off)) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            part_sum[i & 3] += x[2 * i] + x[2 * i + 1];
            y[i] = pack(x[2 * i], x[2 * i + 1]);
          }
          ptx::tmem_st<16>(s_t + e * 16, y);
        }
        sum += (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sh.p[b]);
      }
      tile0 += nt;
      // The outputs, unnormalised, and (maximum, sum) to the piece's slot.
      const int slot = G == 2 && kSub == 1 ? 2 * walk.slot + grp : walk.slot;
      const int64_t pr = part_row(p, slot, h, m);
      if (any) {
        const int bl = G == 2 ? grp : (nj - 1) & 1;  // score buffer of the group's last job
        wait_warp(&sh.pv[bl], (ns[bl] - 1) & 1, dead);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int e = 0; e < D / 32; ++e) {
          float x[32];
          ptx::tmem_ld32(o_t + e * 32, x);
          ptx::tmem_ld_wait();
          if (m < p.M) {
            float4 *out = reinterpret_cast<float4 *>(p.part_o + pr * D + e * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
        ptx::tc_fence_before();
      } else if (m < p.M) {
        float4 *out = reinterpret_cast<float4 *>(p.part_o + pr * D);
        for (int i = 0; i < D / 4; ++i) out[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (m < p.M) p.part_ml[pr] = dead ? make_float2(0.f, CUDART_NAN_F) : make_float2(mref, sum);
    }
  } else if (warp < kMmaWarp) {
    // -------------------------------------------------------------- loads
    const int lw = warp - C::kSoft / 32;
    constexpr int kTokW = TT / 4;                // tokens of a tile this warp copies
    constexpr int kPer = D * 2 / 16;             // 16-byte chunks of a row
    const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
    uint32_t it = 0, told = 0;  // items (K and V tiles in turn) issued, and reported full
    auto full_bar = [&](uint32_t i) { return (i & 1) ? &sh.vfull[(i >> 1) & 1] : &sh.kfull[(i >> 1) & 1]; };
    // Copies that have landed become visible to the tensor cores' reads.
    auto tell = [&](uint32_t upto) {
      if (told < upto) {
        ptx::fence_proxy_async();
        __syncwarp();
        for (; told < upto; ++told)
          if (lane == 0) ptx::mbar_arrive(full_bar(told));
      }
    };
    while (walk.next(p)) {
      const int32_t *tab = p.table + (int64_t)walk.r * p.row_pages;
      const int nt = (walk.hi - walk.lo + TT - 1) / TT;
      auto row_of = [&](int t) -> int64_t {
        const int pos = walk.lo + t * TT + lw * kTokW + lane;
        if (lane >= kTokW || pos >= walk.hi) return -1;
        const int pg = tab[pos / p.page];
        if (pg < 0 || pg >= p.pages) {
          set_status(p.status, kStatusPage);
          return -1;
        }
        return (((int64_t)pg * p.Hkv + h) * p.page + pos % p.page) * (D * 2);
      };
      int64_t next_row = row_of(0);
      for (int t = 0; t < nt; ++t) {
        const int64_t row = next_row;
        const uint32_t here = __ballot_sync(0xffffffffu, row >= 0);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t st = (it >> 1) & 1, n = it >> 2;  // stage, and its uses before
          uint64_t *empty = kv ? &sh.vempty[st] : &sh.kempty[st];
          if (n > 0 && !dead && !__all_sync(0xffffffffu, ptx::mbar_try_wait(empty, (n - 1) & 1))) {
            // Nothing to issue yet: hand over all that is under way first.
            cp_wait<0>();
            tell(it);
            wait(empty, (n - 1) & 1, dead);
            dead = __any_sync(0xffffffffu, dead);  // the warp stays together
          }
          if (kv == 0 && lane == 0) sh.mask[(it >> 1) & 3][lw] = here;
          uint8_t *dst = smem + (kv ? C::oV : C::oK) + st * C::kTile;
          const uint8_t *src = kv ? vp : kp;
#pragma unroll 8
          for (int e = 0; e < kTokW * kPer / 32; ++e) {
            const int at = e * 32 + lane, tk = at / kPer, c = at % kPer;
            const int64_t off = __shfl_sync(0xffffffffu, row, tk);
            ptx::cp_async16(dst + (c >> 3) * (TT * 128) + ptx::swz128(lw * kTokW + tk, c & 7),
                            src + (off < 0 ? 0 : off) + c * 16, off < 0 ? 0 : 16);
          }
          ptx::cp_async_commit();
          if (kv == 0) next_row = t + 1 < nt ? row_of(t + 1) : -1;
          if (it >= 2) {
            cp_wait<2>();
            tell(it - 1);
          }
        }
      }
    }
    cp_wait<0>();
    tell(it);
  } else if (lane == 0) {
    // ----------------------------------------------------------- products
    constexpr uint32_t id_s = ptx::idesc_bf16_f32(128, TT);
    constexpr uint32_t id_o = ptx::idesc_bf16_f32(128, D) | ptx::kIdescBMnMajor;
    uint32_t nq = 0, kt = 0, vt = 0, np[2] = {0, 0}, npv[2] = {0, 0};
    bool work = false;
    while (walk.next(p)) {
      const int nt = (walk.hi - walk.lo + TT - 1) / TT, nj = nt * kSub;
      work = true;
      wait(&sh.q, nq++ & 1, dead);
      auto scores = [&](int j) {
        const int b = j & 1;
        const bool first = kSub == 1 || b == 0, last = kSub == 1 || b == 1;
        const uint32_t st = kt & 1;
        if (first) wait(&sh.kfull[st], (kt >> 1) & 1, dead);
        // P of this buffer's last job is read once its product is done.
        if (npv[b] > 0) wait(&sh.pv[b], (npv[b] - 1) & 1, dead);
        ptx::tc_fence_after();
        if (!dead) {
          const uint32_t qa = base + (kSub == 2 ? b * C::kQ : 0), ka = base + C::oK + st * C::kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_bf16(tmem + kSCol + b * TT, ptx::desc_k128(qa + (kk >> 2) * 16384 + (kk & 3) * 32),
                          ptx::desc_k128(ka + (kk >> 2) * (TT * 128) + (kk & 3) * 32), id_s, kk > 0);
          ptx::mma_commit(&sh.s[b]);
          if (last) ptx::mma_commit(&sh.kempty[st]);
        }
        if (last) ++kt;
      };
      scores(0);
      if (nj > 1) scores(1);
      for (int j = 0; j < nj; ++j) {
        const int b = j & 1;
        const bool first = kSub == 1 || b == 0, last = kSub == 1 || b == 1;
        const uint32_t st = vt & 1;
        if (first) wait(&sh.vfull[st], (vt >> 1) & 1, dead);
        wait(&sh.p[b], np[b]++ & 1, dead);
        ptx::tc_fence_after();
        if (!dead) {
          const uint32_t va = base + C::oV + st * C::kTile;
          const uint32_t acc = G == 2 ? j >= 2 : j >= 1;
#pragma unroll
          for (int kk = 0; kk < TT / 16; ++kk)
            ptx::mma_bf16_ts(tmem + (G == 2 ? b * 128 : 0), tmem + kSCol + b * TT + kk * 8,
                             ptx::desc_mn128(va + kk * 2048, TT * 128), id_o, acc || kk > 0);
          ptx::mma_commit(&sh.pv[b]);
          if (last) ptx::mma_commit(&sh.vempty[st]);
        }
        ++npv[b];
        if (last) ++vt;
        if (j + 2 < nj) scores(j + 2);
      }
    }
    if (work) {
      ptx::mma_commit(&sh.done);
      if (!ptx::mbar_wait(&sh.done, 0, kWaitNs)) dead = true;
    }
  }
  if (dead) set_status(p.status, ONELA_STATUS_TIMEOUT);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int kSub>
cudaError_t run(const AttnParams &p, cudaStream_t s) {
  using C = Cfg<D, kSub>;
  const cudaError_t e = ensure_smem_limit((const void *)attn_wide<D, kSub>, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_wide<D, kSub>, (unsigned)((long long)p.parts * p.Hkv * p.row_tiles), C::kThreads, C::kSmem,
                       false, s, p);
}

}  // namespace

cudaError_t launch_attn_wide(const AttnParams &p, cudaStream_t s) {
  const bool two = p.rows == 256;
  if (p.d == 64) return two ? run<64, 2>(p, s) : run<64, 1>(p, s);
  if (p.d == 128) return two ? run<128, 2>(p, s) : run<128, 1>(p, s);
  return run<256, 1>(p, s);
}

}  // namespace onela
