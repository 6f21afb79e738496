// Attention over a paged cache for many query rows per key-value head: the
// beams of a request share its prompt, so W * G rows (1024 for 256 beams of
// 4 grouped heads) read the same K and V.  bf16, d in {64, 128, 256}.
//
// At 128 rows per tile a K and V row is used 128 times for every read, so the
// matrix products (4 d operations per row and token) and the exponentials
// (one per row and token, 16 a clock on an SM) bound it: at d = 128 both take
// about 512 clocks for 128 rows x 64 tokens.  Both products run on tcgen05: S
// = Q K^T with both operands in shared memory, O += P V with P in tensor
// memory, where the softmax warps write it over the scores they read, and V
// as it lies in the cache (token rows, an MN-major B operand).  O stays in
// tensor memory.
//
// Two groups of four softmax warps (thread = row) each own an O and two score
// buffers of 64 tokens: while a group takes the exponentials of one buffer, the
// tensor cores fill its other one and work for the other group.  (With one
// buffer of 128 tokens a group, each group's products waited for its
// exponentials and these for its products.)  The groups take the two halves of
// 256 rows (kSub = 2, K and V read once for both) or, with at
// most 128 rows, every other token tile of the same rows (kSub = 1), each with
// its own result slot.  At d = 256 O fills half of the tensor memory, so there
// is one group.
//
// The running maximum that weights are taken against moves only when a row's
// maximum grew by more than 2^8 (scores in log2 units): weights then stay
// below 2^8, exact in range for bf16 and fp32 alike, and O is rescaled rarely.
// P is rounded to bf16 (2^-8 relative per weight at most, of the size of the
// rounding of o itself); its sum is that of the unrounded weights, in fp32.
//
// 256 beams of 16 / 4 heads of 128 take 23 us on 5120 tokens (7 of their own
// each), two thirds of it start, partial outputs and their join, and 86 us on
// 40960 (994 TFLOP/s; 1150 in steady state, where the scores' products, held by
// shared memory at N = 64, take twice the outputs' time).
//
// Four warps bring in the K and V rows, a quarter of a tile each, through the
// page table into rings of K and V tiles: by TMA boxes of 16 or 8 tokens
// where all of a warp's tokens are there and pages are multiples of 8 tokens,
// otherwise by 16-byte asynchronous copies, zeros for tokens that are not
// there.  (Those alone held the SM to 18 bytes a clock.)  Every wait is bounded: one that runs out sets
// ONELA_STATUS_TIMEOUT and the results become NaN.
#include "attention.h"

#include "../../include/onela.h"
#include "copy_reports.h"
#include "f32x2.h"
#include "internal.h"
#include "sm100_ptx.h"
#include "tc_common.h"

namespace onela {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;  // scores behind the outputs in tensor memory
constexpr int TT = 64;           // tokens per tile

template <int D, int kSub>
struct Cfg {
  static constexpr int G = D == 256 ? 1 : 2;  // softmax groups
  static constexpr int kSoft = G * 128;
  static constexpr int kThreads = kSoft + 128 + 64;
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kQ = 128 * D * 2;    // bytes of 128 Q rows
  static constexpr int kTile = TT * D * 2;  // bytes of a K or V tile
  static constexpr int oK = kSub * kQ, oV = oK + kStages * kTile, oOut = oV + kStages * kTile;
  // 32 rows x 32 columns of O for each softmax warp, on their way out: over
  // the group's own Q rows (kSub = 2), else in a place of its own, for the other group may still read Q.
  static constexpr int oEnd = oOut + (kSub == 2 ? 0 : kSoft / 32 * 4096);
  // Above half of an SM's shared memory, so that one CTA has the SM (and its
  // tensor memory) for itself.
  static constexpr int kSmem = oEnd + 1024 < 120 * 1024 ? 120 * 1024 : oEnd + 1024;
};

struct Shared {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t s[4], p[4], pv[4];  // by group and score buffer
  uint64_t q, done[2];
  uint32_t tmem;
  uint32_t mask[8][4];  // by tile (ring of 8) and load warp: the 16 tokens that are there
  PlanSmem plan;
};

// K and V pools as {64 elements, 1, tokens of a page, (page, head)}; q as {64
// elements, the G heads of a group, 64 / G tokens, request}: 64 query rows.
struct Maps {
  CUtensorMap k, v, q;
  int box;    // tokens per box of K and V: 16, 8, or 0 (pages not a multiple of 8: no boxes)
  int q_box;  // q comes in boxes (G divides 64)
};

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Wait of a whole warp, which goes on together and alike: `dead` is the same in
// all its lanes (a barrier may complete between two lanes' last looks at it).
// No wait once one has run out.  A warp whose wait ran out hands nothing on from
// then: it issues no copy and no product and arrives on no barrier of the
// others, whose own waits then run out too before they take anything unfinished.
__device__ __forceinline__ void wait_warp(const AttnParams &p, uint64_t *bar, uint32_t parity, bool &dead) {
  if (!dead && !ptx::mbar_wait(bar, parity, p.wait_ns)) dead = true;
  dead = __any_sync(0xffffffffu, dead);
}

template <int D, int kSub>
__global__ void __launch_bounds__(Cfg<D, kSub>::kThreads, 1) attn_wide(const __grid_constant__ AttnParams p,
                                                                       const __grid_constant__ Maps maps) {
  using C = Cfg<D, kSub>;
  constexpr int G = C::G, NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = ptx::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rt = blockIdx.x % p.row_tiles, ch = blockIdx.x / p.row_tiles;
  const int h = ch % p.Hkv, part = ch / p.Hkv;
  const int m0 = rt * (128 * kSub);

  constexpr int kMmaWarp = C::kSoft / 32 + 4;
  if (tid == 0) {
    // stall (tests): an arrival that never comes.
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&sh.kfull[i], 4 + (p.stall == kStallFull));
      ptx::mbar_init(&sh.vfull[i], 4 + (p.stall == kStallFull));
      ptx::mbar_init(&sh.kempty[i], 1 + (p.stall == kStallEmpty));
      ptx::mbar_init(&sh.vempty[i], 1 + (p.stall == kStallEmpty));
      ptx::mbar_init(&sh.s[i], 1 + (p.stall == kStallScores));
      ptx::mbar_init(&sh.p[i], 128 + (p.stall == kStallWeights));
      ptx::mbar_init(&sh.pv[i], 1 + (p.stall == kStallOutputs));
    }
    ptx::mbar_init(&sh.q, C::kSoft);
    ptx::mbar_init(&sh.done[0], 1);
    ptx::mbar_init(&sh.done[1], 1);
    ptx::mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  if (tid == 32 && maps.box) {
    ptx::prefetch_tmap(&maps.k);
    ptx::prefetch_tmap(&maps.v);
  }
  if (tid == 64 && maps.q_box) ptx::prefetch_tmap(&maps.q);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  PlanWalk walk;
  walk.begin<C::kThreads>(p, sh.plan, part);
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  bool dead = false;

  if (warp < C::kSoft / 32) {
    // ------------------------------------------------------------- softmax
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;  // thread = query row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int m1 = m0 + (kSub == 2 ? grp * 128 : 0), m = m1 + row;
    const uint32_t o_t = tmem + lanes + (G == 2 ? grp * 128 : 0);
    uint32_t c = 0;      // jobs of this group so far: buffer c & 1, use c >> 1 of it
    uint32_t tile0 = 0;  // tiles of earlier pieces (the mask ring runs on)
    while (walk.next(p)) {
      const int r = walk.r;
      const int nt = (walk.hi - walk.lo + TT - 1) / TT;
      // Every product of the last piece is done (each group waited for its
      // own): Q may be replaced.
      ptx::bar_sync(1, C::kSoft);
      if (kSub == 2 || grp == 0) {
        // By boxes of 64 rows, or a warp brings its 32 rows, 32 16-byte chunks at a time.
        uint8_t *qd = smem + (kSub == 2 ? grp * C::kQ : 0);
        if (maps.q_box) {
          if (warp == 4 * grp && lane == 0 && !dead) {
            ptx::fence_proxy_async();  // the rows that went out through this memory were written by plain stores
            ptx::mbar_expect_tx(&sh.q, C::kQ);
#pragma unroll
            for (int a = 0; a < 2 * (D / 64); ++a)
              ptx::tma_load_4d(qd + (a >> 1) * 16384 + (a & 1) * 8192, &maps.q, (a >> 1) * 64, h * p.G,
                               (m1 + (a & 1) * 64) / p.G, r, &sh.q);
          }
        } else {
          constexpr int kPer = D / 8;
          const int64_t mine =
              m < p.M ? ((int64_t)r * p.W + m / p.G) * p.q_stride + (int64_t)(h * p.G + m % p.G) * D : -1;
#pragma unroll 4
          for (int e = 0; e < kPer; ++e) {
            const int rl = (e * 32 + lane) / kPer, cc = (e * 32 + lane) % kPer, rw = (warp & 3) * 32 + rl;
            const int64_t at = __shfl_sync(0xffffffffu, mine, rl);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (at >= 0) x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + at) + cc);
            *reinterpret_cast<uint4 *>(qd + (cc >> 3) * 16384 + ptx::swz128(rw, cc & 7)) = x;
          }
        }
      }
      ptx::fence_proxy_async();
      if (!dead) ptx::mbar_arrive(&sh.q);

      float mref = -CUDART_INF_F, sum = 0.f;
      bool any = false;  // this group has a product in O
      constexpr int kStep = kSub == 1 ? G : 1;
      for (int t = kSub == 1 ? grp : 0; t < nt; t += kStep, ++c) {
        const int b = grp * 2 + (c & 1);
        const uint32_t s_t = tmem + lanes + kSCol + b * TT;
        wait_warp(p, &sh.s[b], (c >> 1) & 1, dead);
        ptx::tc_fence_after();
        float x[2][32];
        ptx::tmem_ld32(s_t, x[0]);
        ptx::tmem_ld32(s_t + 32, x[1]);
        const uint32_t *mk = sh.mask[(tile0 + t) & 7];
        const uint32_t msk[2] = {mk[0] | (mk[1] << 16), mk[2] | (mk[3] << 16)};
        ptx::tmem_ld_wait();
        if ((msk[0] & msk[1]) != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 32; ++i) x[e][i] = (msk[e] >> i) & 1 ? x[e][i] : -CUDART_INF_F;
        }
        float t4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int i = 0; i < 64; ++i) t4[i & 3] = fmaxf(t4[i & 3], x[i >> 5][i & 31]);
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        // Move the reference when the maximum outgrew it (from -inf: always,
        // unless there is nothing yet).
        const bool grow = (top - mref) * p.scale_log2 > kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? exp2_sub(mref, top, p.scale_log2) : 1.f;
          if (any) {
            // The group's last product into O must be done.
            wait_warp(p, &sh.pv[b ^ 1], ((c - 1) >> 1) & 1, dead);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              float z[16];
              uint32_t y[16];
              ptx::tmem_ld16(o_t + e * 16, z);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(z[i] * f);
              ptx::tmem_st<16>(o_t + e * 16, y);
            }
          }
          if (grow) {
            sum *= f;
            mref = top;
          }
        }
        any = true;
        // The weights, over the scores' own columns.
        const float off = mref == -CUDART_INF_F ? 0.f : -mref;
        const F2 off2 = f2(off, off), sc2 = f2(p.scale_log2, p.scale_log2);
        F2 s4[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 w = un((f2(x[e >> 1][(e & 1) * 16 + 2 * i], x[e >> 1][(e & 1) * 16 + 2 * i + 1]) + off2) * sc2);
            const float a = ex2(w.x), bb = ex2(w.y);
            s4[i & 3] = s4[i & 3] + f2(a, bb);
            y[i] = pack_bf16(a, bb);
          }
          ptx::tmem_st<8>(s_t + e * 8, y);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        if (!dead) ptx::mbar_arrive(&sh.p[b]);
        const float2 sw = un((s4[0] + s4[1]) + (s4[2] + s4[3]));
        sum += sw.x + sw.y;
      }
      tile0 += nt;
      // The outputs, unnormalised, and (maximum, sum) to the piece's slot.
      const int slot = G == 2 && kSub == 1 ? 2 * walk.slot + grp : walk.slot;
      const int64_t pr = part_row(p, slot, h, m);
      if (any) {
        wait_warp(p, &sh.pv[grp * 2 + ((c - 1) & 1)], ((c - 1) >> 1) & 1, dead);
        ptx::tc_fence_after();
      }
      // Rows go out 128 bytes at a time: 32 columns of the warp's 32 rows through shared memory.
      uint8_t *stage = smem + (kSub == 2 ? grp * C::kQ + (warp & 3) * 4096 : C::oOut + warp * 4096);
#pragma unroll 1
      for (int e = 0; e < D / 32; ++e) {
        float z[32];
        if (any) {
          ptx::tmem_ld32(o_t + e * 32, z);
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4 *>(stage + ptx::swz128(lane, i)) =
              make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
        __syncwarp();
        float *out = p.part_o + (pr - lane) * D + e * 32;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rl = i * 4 + (lane >> 3);
          if (m - lane + rl < p.M)
            *reinterpret_cast<float4 *>(out + (int64_t)rl * D + (lane & 7) * 4) =
                *reinterpret_cast<const float4 *>(stage + ptx::swz128(rl, lane & 7));
        }
        __syncwarp();
      }
      if (any) ptx::tc_fence_before();
      if (m < p.M) p.part_ml[pr] = dead ? make_float2(0.f, CUDART_NAN_F) : make_float2(mref, sum);
    }
  } else if (warp < kMmaWarp) {
    // -------------------------------------------------------------- loads
    const int lw = warp - C::kSoft / 32;
    constexpr int kTokW = TT / 4;     // tokens of a tile this warp brings
    constexpr int kPer = D * 2 / 16;  // 16-byte chunks of a row
    const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
    const bool one_page = p.page % 16 == 0;
    uint32_t it = 0;             // items (K and V tiles in turn) issued
    CopyReports rep;             // which of them this warp has to report full
    auto full_bar = [&](uint32_t i) { return (i & 1) ? &sh.vfull[(i >> 1) % NS] : &sh.kfull[(i >> 1) % NS]; };
    // Asynchronous copies that have landed become visible to the tensor cores' reads.
    auto tell = [&](uint32_t upto) {
      if (!rep.due(upto)) return;
      ptx::fence_proxy_async();
      __syncwarp();
      rep.landed(upto, [&](uint32_t i) {
        if (lane == 0) ptx::mbar_arrive(full_bar(i));
      });
    };
    while (!dead && walk.next(p)) {
      const int32_t *tab = p.table + (int64_t)walk.r * p.row_pages;
      const int nt = (walk.hi - walk.lo + TT - 1) / TT;
      // Where this warp's 16 tokens of a tile are: page * Hkv + head (-1: not
      // there) and place on the page, by lane.  Pages of a multiple of 16
      // tokens hold them together: one entry for a tile, and the entries of 32
      // tiles in one load.  Otherwise each lane looks its token's entry up a tile ahead.
      int ph = -1, place = 0;
      auto entry = [&](int pos) {
        ph = -1;
        if (pos < walk.hi) {
          const int at = pos / p.page, pg = tab[at];
          place = pos - at * p.page;
          if (pg >= 0 && pg < p.pages) ph = pg * p.Hkv + h;
          else set_status(p.status, kStatusPage);
        }
      };
      const int first = walk.lo + lw * kTokW;
      if (!one_page) entry(lane < kTokW ? first + lane : walk.hi);
      for (int t = 0; t < nt && !dead; ++t) {
        int cph = ph, cplace = place;
        if (one_page) {
          if (t % 32 == 0) entry(first + (t + lane) * TT);
          cph = __shfl_sync(0xffffffffu, ph, t % 32);
          cplace = __shfl_sync(0xffffffffu, place, t % 32) + lane;
          if (lane >= kTokW || first + t * TT + lane >= walk.hi) cph = -1;
        } else {
          entry(lane < kTokW ? first + (t + 1) * TT + lane : walk.hi);
        }
        const uint32_t here = __ballot_sync(0xffffffffu, cph >= 0);
        const bool boxes = maps.box && here == (1u << kTokW) - 1u;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t st = (it >> 1) % NS, n = (it >> 1) / NS;  // stage, and its uses before
          uint64_t *empty = kv ? &sh.vempty[st] : &sh.kempty[st];
          if (n > 0 && !dead && !__all_sync(0xffffffffu, ptx::mbar_try_wait(empty, (n - 1) & 1))) {
            // Nothing to issue yet: hand over all that is under way first.
            if (rep.pend) {
              cp_wait<0>();
              tell(it);
            }
            wait_warp(p, empty, (n - 1) & 1, dead);
          }
          if (dead) break;
          if (kv == 0 && lane == 0) sh.mask[(it >> 1) & 7][lw] = here;
          uint8_t *dst = smem + (kv ? C::oV : C::oK) + st * C::kTile;
          if (boxes) {
            const int ph8 = __shfl_sync(0xffffffffu, cph, 8), pl8 = __shfl_sync(0xffffffffu, cplace, 8);
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(full_bar(it), kTokW * D * 2);
              const CUtensorMap *tm = kv ? &maps.v : &maps.k;
#pragma unroll
              for (int a = 0; a < D / 64; ++a) {
                uint8_t *to = dst + a * (TT * 128) + lw * (kTokW * 128);
                ptx::tma_load_4d(to, tm, a * 64, 0, cplace, cph, full_bar(it));
                if (maps.box == 8) ptx::tma_load_4d(to + 8 * 128, tm, a * 64, 0, pl8, ph8, full_bar(it));
              }
            }
          } else {
            const uint8_t *src = kv ? vp : kp;
#pragma unroll 4
            for (int e = 0; e < kTokW * kPer / 32; ++e) {
              const int at = e * 32 + lane, tk = at / kPer, cc = at % kPer;
              const int sph = __shfl_sync(0xffffffffu, cph, tk), spl = __shfl_sync(0xffffffffu, cplace, tk);
              const int64_t off = sph < 0 ? 0 : ((int64_t)sph * p.page + spl) * (D * 2) + cc * 16;
              ptx::cp_async16(dst + (cc >> 3) * (TT * 128) + ptx::swz128(lw * kTokW + tk, cc & 7), src + off,
                              sph < 0 ? 0 : 16);
            }
            rep.mark(it);
          }
          ptx::cp_async_commit();
          if (rep.pend && it >= 2) {
            cp_wait<2>();
            tell(it - 1);
          }
        }
      }
    }
    cp_wait<0>();
    tell(it);
    // Boxes of a piece that was given up may still be on their way: no CTA
    // ends before its copies have landed (they have, too, once a wait has run out).
    for (uint32_t i = it < 2 * NS ? 0 : it - 2 * NS; i < it; ++i) {
      const uint32_t turn = (i >> 1) / NS;
      if (!ptx::mbar_wait(full_bar(i), turn & 1, p.wait_ns)) {
        dead = true;
        break;
      }
    }
  } else {
    // ----------------------------------------------------------- products
    // One warp issues the scores and one the outputs, so that the waits of
    // one lie under the products of the other; barriers order them.  The
    // whole warp walks along and waits and one elected lane issues: that way every
    // descriptor is a warp-uniform value (with the loop itself in one lane's
    // branch an instruction took about 100 clocks to issue).
    const bool is_s = warp == kMmaWarp;
    constexpr uint32_t id_s = ptx::idesc_bf16_f32(128, TT);
    constexpr uint32_t id_o = ptx::idesc_bf16_f32(128, D) | ptx::kIdescBMnMajor;
    const uint64_t qd = ptx::desc_k128(base), kd = ptx::desc_k128(base + C::oK);
    const uint64_t vd = ptx::desc_mn128(base + C::oV, TT * 128);
    uint32_t nq = 0, tiles = 0;   // Q tiles, K or V tiles used
    uint32_t c[2] = {0, 0};       // jobs of each group so far
    while (walk.next(p)) {
      const int nt = __shfl_sync(0xffffffffu, (walk.hi - walk.lo + TT - 1) / TT, 0);
      // Jobs in the order of issue: job j of the piece is group j % G's, tile
      // j (kSub = 1) or j / 2 (kSub = 2).
      const int nj = nt * kSub;
      if (is_s) wait_warp(p, &sh.q, nq & 1, dead);
      ++nq;
      for (int j0 = 0; j0 < nj; j0 += G) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (j0 + g >= nj) break;
          const uint32_t cg = c[g]++;
          const int b = g * 2 + (cg & 1);
          const bool first = kSub == 1 || g == 0, last = kSub == 1 || g == 1;
          const uint32_t st = tiles % NS, turn = tiles / NS;
          if (last) ++tiles;
          if (is_s) {
            if (first) wait_warp(p, &sh.kfull[st], turn & 1, dead);
            // The weights that were in this buffer have been used.
            if (cg >= 2) wait_warp(p, &sh.pv[b], ((cg >> 1) - 1) & 1, dead);
            ptx::tc_fence_after();
            const uint64_t qa = qd + (kSub == 2 ? g * (C::kQ >> 4) : 0), ka = kd + st * (C::kTile >> 4);
            const uint32_t to = tmem + kSCol + b * TT;
            if (!dead && ptx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                ptx::mma_bf16(to, qa + ((kk >> 2) * 16384 + (kk & 3) * 32) / 16,
                              ka + ((kk >> 2) * (TT * 128) + (kk & 3) * 32) / 16, id_s, kk > 0);
              ptx::mma_commit(&sh.s[b]);
              if (last) ptx::mma_commit(&sh.kempty[st]);
            }
          } else {
            if (first) wait_warp(p, &sh.vfull[st], turn & 1, dead);
            wait_warp(p, &sh.p[b], (cg >> 1) & 1, dead);
            ptx::tc_fence_after();
            const uint64_t va = vd + st * (C::kTile >> 4);
            const uint32_t to = tmem + (G == 2 ? g * 128 : 0), from = tmem + kSCol + b * TT;
            if (!dead && ptx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < TT / 16; ++kk)
                ptx::mma_bf16_ts(to, from + kk * 8, va + kk * (2048 / 16), id_o, j0 > 0 || kk > 0);
              ptx::mma_commit(&sh.pv[b]);
              if (last) ptx::mma_commit(&sh.vempty[st]);
            }
          }
          __syncwarp();
        }
      }
    }
    if (nq > 0) {
      if (ptx::elect_one()) ptx::mma_commit(&sh.done[is_s]);
      if (!ptx::mbar_wait(&sh.done[is_s], 0, p.wait_ns)) dead = true;
      if (is_s && !ptx::mbar_wait(&sh.q, (nq - 1) & 1, p.wait_ns)) dead = true;  // Q's boxes have landed
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

// ---------------------------------------------------------------------------
// The weight each prompt position drew, once every row's (maximum, 1 / sum) is known: the
// scores again, this time transposed, S^T = K Q^T, so that a thread owns a
// token and adds exp2(s - max) / sum over the rows in order (no atomics, one writer
// per position).  Recomputing costs half of the attention's products; keeping
// the scores would cost 4 bytes a row and token, more than K and V themselves
// from 64 rows on at d = 64.  One CTA per (request, head, 128 tokens): K is an operand
// held in shared memory, tiles of 64 rows of Q pass through a ring, two groups
// of four warps take them in turn; two CTAs per SM for d <= 128.
template <int D>
struct MassCfg {
  static constexpr int kStages = 4;
  static constexpr int kK = 128 * D * 2, kTile = 64 * D * 2;
  static constexpr int kThreads = 256 + 128 + 32;
  static constexpr int kSmem = kK + kStages * kTile + 1024;
};

struct MassShared {
  uint64_t k, full[4], empty[4], s[4], sfree[4], done;
  uint32_t tmem;
  alignas(16) float neg[4][64], inv[4][64];  // of the rows, by Q stage: -maximum, 1 / sum
  float sums[128];
};

template <int D>
__global__ void __launch_bounds__(MassCfg<D>::kThreads, D == 256 ? 1 : 2) attn_mass_wide(const __grid_constant__ AttnParams p,
                                                                                            const __grid_constant__ Maps maps) {
  using C = MassCfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MassShared sh;
  uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = ptx::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int chunks = (p.cap + 127) / 128;
  const int t0 = (int)(blockIdx.x % chunks) * 128, rh = blockIdx.x / chunks, r = rh / p.Hkv, h = rh % p.Hkv;
  const int len = prompt_len(p, r);
  if (t0 >= len) {
    ptx::pdl_wait();  // a launch is never over before the one it depends on
    return;
  }
  const int nt = (p.M + 63) / 64;  // tiles of Q rows

  if (tid == 0) {
    ptx::mbar_init(&sh.k, 128);
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&sh.full[i], 128 + (p.stall == kStallMassFull));
      // By the threads that took the stage's tile: its product is done by then.
      ptx::mbar_init(&sh.empty[i], 128 + (p.stall == kStallMassEmpty));
      ptx::mbar_init(&sh.s[i], 1 + (p.stall == kStallMassScores));
      ptx::mbar_init(&sh.sfree[i], 128 + (p.stall == kStallMassRead));
    }
    ptx::mbar_init(&sh.done, 1);
    ptx::mbar_fence_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(&sh.tmem, 256);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  bool dead = false;

  if (warp < 8) {
    // ----------------------------------------------------- thread = token
    const int grp = warp >> 2, tok = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    float sum = 0.f;
    uint32_t c = 0;
    for (int t = grp; t < nt; t += 2, ++c) {
      const int b = grp * 2 + (c & 1), st = t % NS;
      wait_warp(p, &sh.s[b], (c >> 1) & 1, dead);
      ptx::tc_fence_after();
      F2 a[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
      const F2 sc2 = f2(p.scale_log2, p.scale_log2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[32];
        ptx::tmem_ld32(tmem + lanes + b * 64 + e * 32, x);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 m = *reinterpret_cast<const float4 *>(&sh.neg[st][e * 32 + i]);
          const float4 l = *reinterpret_cast<const float4 *>(&sh.inv[st][e * 32 + i]);
          const float2 w0 = un((f2(x[i], x[i + 1]) + f2(m.x, m.y)) * sc2);
          const float2 w1 = un((f2(x[i + 2], x[i + 3]) + f2(m.z, m.w)) * sc2);
          // The maximum is a reference, which scores pass by up to kSlack; the bound
          // is for scores so large that their last bits, which may come out another
          // way in this product, are many powers of two.
          constexpr float kTop = 2.f * kSlack;
          a[0] = fma2(f2(ex2(min_nan(w0.x, kTop)), ex2(min_nan(w0.y, kTop))), f2(l.x, l.y), a[0]);
          a[1] = fma2(f2(ex2(min_nan(w1.x, kTop)), ex2(min_nan(w1.y, kTop))), f2(l.z, l.w), a[1]);
        }
      }
      const float2 at2 = un(a[0] + a[1]);
      sum += at2.x + at2.y;
      ptx::tc_fence_before();
      if (!dead) {
        ptx::mbar_arrive(&sh.sfree[b]);
        ptx::mbar_arrive(&sh.empty[st]);
      }
    }
    if (grp == 1) sh.sums[tok] = dead ? CUDART_NAN_F : sum;
    ptx::bar_sync(1, 256);
    if (grp == 0 && t0 + tok < len) {
      const int64_t at = (int64_t)rh * p.cap + t0 + tok;
      // A position on a bad page (its zeros gave scores of 0) draws nothing.
      const int pg = p.table[(int64_t)r * p.row_pages + (t0 + tok) / p.page];
      const float drawn = dead ? CUDART_NAN_F : (pg >= 0 && pg < p.pages ? sum + sh.sums[tok] : 0.f);
      p.mass_out[at] = p.mass ? p.mass[at] + drawn : drawn;
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- loads
    const int lw = warp - 8, lt = tid - 256;
    constexpr int kPer = D * 2 / 16;
    {
      // K rows of this warp's 32 tokens, zeros for those that are not there.
      const int pos = t0 + lw * 32 + lane;
      int64_t mine = -1;
      if (pos < len) {
        const int pg = p.table[(int64_t)r * p.row_pages + pos / p.page];
        if (pg >= 0 && pg < p.pages) mine = (((int64_t)pg * p.Hkv + h) * p.page + pos % p.page) * (D * 2);
      }
      if (maps.box && __all_sync(0xffffffffu, mine >= 0)) {
        // Boxes of 16 or 8 tokens; this warp's share of the bytes is expected by its first lane.
        if (lane == 0) ptx::mbar_expect_tx(&sh.k, 32 * D * 2);
        __syncwarp();
        if (lane % maps.box == 0) {
          const int ph = (int)(mine / (D * 2) / p.page), pl = (int)(mine / (D * 2) % p.page);
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
            ptx::tma_load_4d(smem + a * 16384 + (lw * 32 + lane) * 128, &maps.k, a * 64, 0, pl, ph, &sh.k);
        }
        __syncwarp();
      } else {
#pragma unroll 4
        for (int e = 0; e < kPer; ++e) {
          const int rl = (e * 32 + lane) / kPer, cc = (e * 32 + lane) % kPer;
          const int64_t at = __shfl_sync(0xffffffffu, mine, rl);
          ptx::cp_async16(smem + (cc >> 3) * 16384 + ptx::swz128(lw * 32 + rl, cc & 7),
                          static_cast<const uint8_t *>(p.k) + (at < 0 ? 0 : at + cc * 16), at < 0 ? 0 : 16);
        }
      }
      ptx::cp_async_commit();
    }
    auto tell = [&](int t) {  // tile t has landed
      ptx::fence_proxy_async();
      ptx::mbar_arrive(&sh.full[t % NS]);
    };
    int issued = 0;  // tiles; all of them, unless a wait ran out
    for (int t = 0; t < nt; ++t) {
      const int st = t % NS;
      if (t >= NS) wait_warp(p, &sh.empty[st], (t / NS - 1) & 1, dead);
      if (dead) break;
      issued = t + 1;
      uint8_t *dst = smem + C::kK + st * C::kTile;
      const int m = t * 64 + lw * 16 + lane;  // lanes 0 .. 15: this warp's rows
      const int64_t mine = lane < 16 && m < p.M
                               ? (((int64_t)r * p.W + m / p.G) * p.q_stride + (int64_t)(h * p.G + m % p.G) * D) * 2
                               : -1;
      if (maps.q_box) {
        if (lt == 0) {
          ptx::mbar_expect_tx(&sh.full[st], C::kTile);
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
            ptx::tma_load_4d(dst + a * 8192, &maps.q, a * 64, h * p.G, t * 64 / p.G, r, &sh.full[st]);
        }
      } else
#pragma unroll 4
      for (int e = 0; e < kPer / 2; ++e) {
        const int rl = (e * 32 + lane) / kPer, cc = (e * 32 + lane) % kPer;
        const int64_t at = __shfl_sync(0xffffffffu, mine, rl);
        ptx::cp_async16(dst + (cc >> 3) * 8192 + ptx::swz128(lw * 16 + rl, cc & 7),
                        static_cast<const uint8_t *>(p.q) + (at < 0 ? 0 : at + cc * 16), at < 0 ? 0 : 16);
      }
      ptx::cp_async_commit();
      if (t == 0) ptx::pdl_wait();  // the rows' norms are the join's
      if (lt < 64) {
        // A row that is not there adds exp2(-inf) = 0, as one that attends to nothing.
        const int mm = t * 64 + lt;
        const float2 l = mm < p.M ? p.norm[(int64_t)rh * p.M + mm] : make_float2(CUDART_INF_F, 0.f);
        sh.neg[st][lt] = -l.x;
        sh.inv[st][lt] = l.y;
      }
      if (t == 0) {
        cp_wait<1>();
        ptx::fence_proxy_async();
        ptx::mbar_arrive(&sh.k);
      }
      if (t >= 1) {
        cp_wait<1>();
        tell(t - 1);
      }
    }
    cp_wait<0>();
    tell(issued - 1);
    // No CTA ends before its boxes have landed.
    if (!ptx::mbar_wait(&sh.k, 0, p.wait_ns)) dead = true;
    for (int t = max(0, issued - NS); t < issued; ++t)
      if (!ptx::mbar_wait(&sh.full[t % NS], (t / NS) & 1, p.wait_ns)) {
        dead = true;
        break;
      }
  } else {
    // ----------------------------------------------------------- products
    constexpr uint32_t id = ptx::idesc_bf16_f32(128, 64);
    const uint64_t kd = ptx::desc_k128(base), qd = ptx::desc_k128(base + C::kK);
    wait_warp(p, &sh.k, 0, dead);
    for (int t = 0; t < nt; ++t) {
      const int g = t & 1, n = t >> 1, b = g * 2 + (n & 1), st = t % NS;
      wait_warp(p, &sh.full[st], (t / NS) & 1, dead);
      if (n >= 2) wait_warp(p, &sh.sfree[b], ((n >> 1) - 1) & 1, dead);
      ptx::tc_fence_after();
      const uint64_t qa = qd + st * (C::kTile >> 4);
      if (!dead && ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ptx::mma_bf16(tmem + b * 64, kd + ((kk >> 2) * 16384 + (kk & 3) * 32) / 16,
                        qa + ((kk >> 2) * 8192 + (kk & 3) * 32) / 16, id, kk > 0);
        ptx::mma_commit(&sh.s[b]);
      }
      __syncwarp();
    }
    if (ptx::elect_one()) ptx::mma_commit(&sh.done);
    if (!ptx::mbar_wait(&sh.done, 0, p.wait_ns)) dead = true;
  }
  if (dead) set_status(p.status, ONELA_STATUS_TIMEOUT);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
}

// The tensor maps of a call; boxes are left out where a shape rules them out.
Maps make_maps(const AttnParams &p) {
  Maps maps = {};
  maps.box = p.page % 16 == 0 ? 16 : (p.page % 8 == 0 ? 8 : 0);
  // Coordinates are 32-bit: the entry point refuses pages * H_kv from 2^31 on.
  if (maps.box && (!encode_rows(&maps.k, p.k, p.d, 1, p.page, p.pages * p.Hkv, maps.box) ||
                   !encode_rows(&maps.v, p.v, p.d, 1, p.page, p.pages * p.Hkv, maps.box)))
    maps.box = 0;
  maps.q_box = 64 % p.G == 0 && encode_heads(&maps.q, p.q, p.d, p.Hq, p.W, p.R, p.q_stride, p.G, 64 / p.G);
  return maps;
}

template <int D, int kSub>
cudaError_t run(const AttnParams &p, cudaStream_t s) {
  using C = Cfg<D, kSub>;
  const cudaError_t e = ensure_smem_limit((const void *)attn_wide<D, kSub>, C::kSmem);
  if (e != cudaSuccess) return e;
  const Maps maps = make_maps(p);
  return launch_kernel(attn_wide<D, kSub>, (unsigned)((long long)p.parts * p.Hkv * p.row_tiles), C::kThreads, C::kSmem,
                       true, s, p, maps);
}

}  // namespace

cudaError_t launch_attn_wide(const AttnParams &p, cudaStream_t s) {
  const bool two = p.rows == 256;
  if (p.d == 64) return two ? run<64, 2>(p, s) : run<64, 1>(p, s);
  if (p.d == 128) return two ? run<128, 2>(p, s) : run<128, 1>(p, s);
  return run<256, 1>(p, s);
}

template <int D>
static cudaError_t run_mass(const AttnParams &p, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit((const void *)attn_mass_wide<D>, MassCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_mass_wide<D>, (unsigned)((long long)p.R * p.Hkv * ((p.cap + 127) / 128)),
                       MassCfg<D>::kThreads, MassCfg<D>::kSmem, true, s, p, make_maps(p));
}

cudaError_t launch_attn_mass_wide(const AttnParams &p, cudaStream_t s) {
  if (p.d == 64) return run_mass<64>(p, s);
  return p.d == 128 ? run_mass<128>(p, s) : run_mass<256>(p, s);
}

}  // namespace onela
