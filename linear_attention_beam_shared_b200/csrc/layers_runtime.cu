// Entry points of the operators around a GDN layer (include/onela.h): checks
// of the arguments on the host, then the launches.  Nothing is kept between
// calls but their number and the wait policy, and nothing is allocated.
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/onela.h"
#include "attention.h"
#include "block_norm.h"
#include "cache.h"
#include "internal.h"

namespace onela {
// `p`: the call's pointers, or none of them (taken to be aligned).
size_t attention_scratch_bytes(const onela_attention_config &c, bool want_mass, const AttnParams &p);
bool attention_tc_supports(const onela_attention_config &c, const AttnParams &p);
cudaError_t launch_attention(const onela_attention_config &c, AttnParams &p, void *scratch, cudaStream_t s);
}  // namespace onela

namespace {

std::atomic<uint64_t> g_calls{0};
std::atomic<uint64_t> g_wait_ns{2000000000};  // onela_set_attention_wait_policy
std::atomic<int> g_stall{0};

bool valid_dtype(int d) { return d == ONELA_F32 || d == ONELA_BF16; }
size_t esize(int d) { return d == ONELA_BF16 ? 2 : 4; }
bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Device memory a call reads or writes; empty where the pointer is null.
struct Span {
  uintptr_t at, bytes;
  Span(const void *p, size_t n) : at(reinterpret_cast<uintptr_t>(p)), bytes(p ? n : 0) {}
  bool overlaps(const Span &o) const { return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes; }
};
// Is any of `a` over any of `b`?
template <size_t N, size_t M>
bool overlap(const Span (&a)[N], const Span (&b)[M]) {
  for (const Span &x : a)
    for (const Span &y : b)
      if (x.overlaps(y)) return true;
  return false;
}

// Switch to the call's device for its duration.
struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      cudaGetLastError();
      return;
    }
    ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
    if (!ok) cudaGetLastError();
  }
  ~DeviceGuard() {
    if (ok && prev >= 0) cudaSetDevice(prev);
  }
};

// Launches on `device`; a failed CUDA call, or an exception of the host's own
// (no memory), becomes ONELA_ERR_CUDA.
template <typename F>
int on_device(int device, F f) {
  try {
    DeviceGuard g(device);
    if (!g.ok) return ONELA_ERR_CUDA;
    g_calls.fetch_add(1, std::memory_order_relaxed);  // calls on one stream are ordered by their caller
    if (f() != cudaSuccess) {
      cudaGetLastError();
      return ONELA_ERR_CUDA;
    }
    return ONELA_OK;
  } catch (...) {
    return ONELA_ERR_CUDA;
  }
}

// A pool's geometry: positions a row holds stay below 2^30 so that position
// arithmetic fits 32 bits (element offsets are 64-bit).
bool valid_rows(int page, int pages, int row_pages) {
  return page >= 1 && pages >= 1 && row_pages >= 1 && (long long)page * row_pages <= (1LL << 30);
}

bool valid_attention(const onela_attention_config &c) {
  if (c.R < 1 || c.R > 65535 || c.W < 1 || c.H_q < 1 || c.H_kv < 1 || c.H_kv > 65535 || c.H_q % c.H_kv != 0 || c.d < 1 ||
      c.d > 256 || !valid_dtype(c.dtype) || c.kernel < ONELA_KERNEL_AUTO || c.kernel > ONELA_KERNEL_TC ||
      !valid_rows(c.page, c.pages, c.row_pages) || c.device < 0 || !(c.scale > 0.f) || c.scale > 2.0e38f ||
      (long long)c.pages * c.H_kv > 0x7fffffffLL)
    return false;
  if ((long long)c.W * (c.H_q / c.H_kv) > 65536 || c.q_stride < (int64_t)c.H_q * c.d) return false;
  const bool none = c.beam_page == 0 && c.beam_pages == 0 && c.beam_row_pages == 0;
  if (!none && !valid_rows(c.beam_page, c.beam_pages, c.beam_row_pages)) return false;
  // Grids: at most one CTA per (request, token, head) row, per (request, head,
  // 32 positions), and per (piece, head, 4 rows).
  const long long rows = (long long)c.R * c.W * c.H_q;
  const long long pos = (long long)c.R * c.H_kv * (((long long)c.page * c.row_pages + 31) / 32);
  return rows <= 0x0fffffffLL && pos <= 0x7fffffffLL;
}

bool valid_evict(const onela_cache_evict_config &c) {
  return c.R >= 1 && c.R <= 65535 && c.H_kv >= 1 && c.H_kv <= 65535 && (long long)c.R * c.H_kv <= 0x7fffffffLL &&
         c.d >= 1 && c.d <= 256 && valid_dtype(c.dtype) && valid_rows(c.page, c.pages, c.row_pages) &&
         valid_rows(c.page, c.dst_pages, c.dst_row_pages) && c.keep >= 1 && c.recent >= 0 && c.recent <= c.keep &&
         (long long)c.dst_row_pages * c.page >= c.keep && c.device >= 0;
}

}  // namespace

uint64_t onela::operator_calls() { return g_calls.load(std::memory_order_relaxed); }

extern "C" {

size_t onela_paged_attention_scratch_bytes(const onela_attention_config *cfg, int32_t want_mass) {
  if (!cfg || !valid_attention(*cfg)) return 0;
  return onela::attention_scratch_bytes(*cfg, want_mass != 0, onela::AttnParams{});
}

int onela_paged_attention(const onela_attention_config *cfg, const void *q, const void *k_pool, const void *v_pool,
                          const int32_t *table, const int32_t *lengths, const void *beam_k, const void *beam_v,
                          const int32_t *beam_table, const int32_t *beam_lengths, const float *mass, float *mass_out,
                          void *o, float *lse, void *scratch, size_t scratch_bytes, int32_t *status,
                          onela_stream stream) {
  if (!cfg || !q || !k_pool || !v_pool || !table || !lengths || !o) return ONELA_ERR_ARG;
  const onela_attention_config c = *cfg;
  if (!valid_attention(c)) return ONELA_ERR_ARG;
  const bool beams = c.beam_row_pages > 0;
  if (beams ? (!beam_k || !beam_v || !beam_table || !beam_lengths)
            : (beam_k || beam_v || beam_table || beam_lengths))
    return ONELA_ERR_ARG;
  if ((mass && !mass_out) || o == q) return ONELA_ERR_ARG;
  const size_t es = esize(c.dtype);
  for (const void *x : {q, k_pool, v_pool, beam_k, beam_v, (const void *)o})
    if (!aligned(x, es)) return ONELA_ERR_ARG;
  for (const void *x : {(const void *)table, (const void *)lengths, (const void *)beam_table, (const void *)beam_lengths,
                        (const void *)mass, (const void *)mass_out, (const void *)lse, (const void *)status})
    if (!aligned(x, 4)) return ONELA_ERR_ARG;
  onela::AttnParams p = {};
  p.q = q;
  p.k = k_pool;
  p.v = v_pool;
  p.table = table;
  p.lengths = lengths;
  p.bk = beam_k;
  p.bv = beam_v;
  p.btable = beam_table;
  p.blengths = beam_lengths;
  p.mass = mass;
  p.mass_out = mass_out;
  p.o = o;
  p.lse = lse;
  p.status = status;
  p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  p.stall = g_stall.load(std::memory_order_relaxed);
  if (c.kernel == ONELA_KERNEL_TC && !onela::attention_tc_supports(c, p)) return ONELA_ERR_UNSUPPORTED;
  const size_t need = onela::attention_scratch_bytes(c, mass_out != nullptr, p);
  if (need > 0 && (!scratch || !aligned(scratch, 256))) return ONELA_ERR_ARG;
  if (scratch_bytes < need) return ONELA_ERR_SCRATCH;
  // Every warp derives its work from the lengths and the tables, and they have
  // to find the same: nothing that is written may lie over them.
  const size_t rows = (size_t)c.R * c.W * c.H_q, cells = (size_t)c.R * c.H_kv * c.page * c.row_pages;
  const Span out[] = {{o, rows * c.d * es}, {lse, rows * 4}, {mass_out, cells * 4}, {scratch, need}, {status, 4}};
  const Span plan[] = {{lengths, (size_t)c.R * 4},
                       {table, (size_t)c.R * c.row_pages * 4},
                       {beam_lengths, (size_t)c.R * c.W * 4},
                       {beam_table, (size_t)c.R * c.W * c.beam_row_pages * 4}};
  if (overlap(out, plan)) return ONELA_ERR_ARG;
  return on_device(c.device,
                   [&] { return onela::launch_attention(c, p, scratch, static_cast<cudaStream_t>(stream)); });
}

int onela_set_attention_wait_policy(uint64_t limit_ns, int32_t stall) {
  if (limit_ns < 1000000ull || limit_ns > 10000000000ull || stall < 0 || stall >= onela::kStallEnd)
    return ONELA_ERR_ARG;
  g_wait_ns.store(limit_ns, std::memory_order_relaxed);
  g_stall.store(stall, std::memory_order_relaxed);
  return ONELA_OK;
}

int onela_cache_write(const onela_cache_write_config *cfg, const void *k, const void *v, void *k_pool, void *v_pool,
                      const int32_t *table, const int32_t *start, const int32_t *counts, int32_t *status,
                      onela_stream stream) {
  if (!cfg || !k || !v || !k_pool || !v_pool || !table || !start || k_pool == v_pool) return ONELA_ERR_ARG;
  const onela_cache_write_config c = *cfg;
  const int64_t row = (int64_t)c.H_kv * c.d;
  if (c.B < 1 || c.n < 1 || c.H_kv < 1 || c.H_kv > 65535 || c.d < 1 || c.d > 256 || !valid_dtype(c.dtype) ||
      !valid_rows(c.page, c.pages, c.row_pages) || c.device < 0 || c.k_stride < row || c.v_stride < row ||
      (long long)c.B * c.n > 0x7fffffffLL)
    return ONELA_ERR_ARG;
  const size_t es = esize(c.dtype);
  for (const void *x : {k, v, (const void *)k_pool, (const void *)v_pool})
    if (!aligned(x, es)) return ONELA_ERR_ARG;
  for (const int32_t *x : {table, start, counts, (const int32_t *)status})
    if (!aligned(x, 4)) return ONELA_ERR_ARG;
  onela::CacheWriteParams p = {};
  p.B = c.B;
  p.n = c.n;
  p.Hkv = c.H_kv;
  p.row_bytes = (int)(c.d * es);
  p.page = c.page;
  p.pages = c.pages;
  p.row_pages = c.row_pages;
  p.k_stride = c.k_stride * (int64_t)es;
  p.v_stride = c.v_stride * (int64_t)es;
  p.k = k;
  p.v = v;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.table = table;
  p.start = start;
  p.counts = counts;
  p.status = status;
  return on_device(c.device, [&] { return onela::launch_cache_write(p, static_cast<cudaStream_t>(stream)); });
}

size_t onela_cache_evict_scratch_bytes(const onela_cache_evict_config *cfg) {
  if (!cfg || !valid_evict(*cfg)) return 0;
  return ((size_t)cfg->R * cfg->H_kv * cfg->keep * 4 + 255) & ~(size_t)255;
}

int onela_cache_evict(const onela_cache_evict_config *cfg, const void *k_pool, const void *v_pool,
                      const int32_t *table, const int32_t *lengths, const float *mass, void *dst_k, void *dst_v,
                      const int32_t *dst_table, int32_t *dst_lengths, float *dst_mass, int32_t *kept, void *scratch,
                      size_t scratch_bytes, int32_t *status, onela_stream stream) {
  if (!cfg || !k_pool || !v_pool || !table || !lengths || !mass || !dst_k || !dst_v || !dst_table || !dst_lengths ||
      !dst_mass || (!kept && !scratch))
    return ONELA_ERR_ARG;
  const onela_cache_evict_config c = *cfg;
  if (!valid_evict(c)) return ONELA_ERR_ARG;
  // Lengths and weights are read by every head while they are written.
  if (dst_lengths == lengths || dst_mass == mass || dst_k == dst_v) return ONELA_ERR_ARG;
  const size_t es = esize(c.dtype);
  for (const void *x : {k_pool, v_pool, (const void *)dst_k, (const void *)dst_v})
    if (!aligned(x, es)) return ONELA_ERR_ARG;
  for (const void *x : {(const void *)table, (const void *)lengths, (const void *)mass, (const void *)dst_table,
                        (const void *)dst_lengths, (const void *)dst_mass, (const void *)kept, (const void *)status})
    if (!aligned(x, 4)) return ONELA_ERR_ARG;
  if (!kept) {
    if (!aligned(scratch, 256)) return ONELA_ERR_ARG;
    if (scratch_bytes < onela_cache_evict_scratch_bytes(&c)) return ONELA_ERR_SCRATCH;
  }
  // The CTAs of a cluster have to find the same lengths and weights each time
  // they look, and the copy the positions that were found: nothing that is
  // written may lie over them.
  const size_t heads = (size_t)c.R * c.H_kv, slot = (size_t)c.H_kv * c.page * c.d * es;
  const Span found[] = {{kept ? kept : scratch, heads * c.keep * 4}};
  const Span out[] = {{dst_lengths, (size_t)c.R * 4},
                      {dst_mass, heads * c.page * c.dst_row_pages * 4},
                      {dst_k, (size_t)c.dst_pages * slot},
                      {dst_v, (size_t)c.dst_pages * slot},
                      {status, 4}};
  const Span plan[] = {{lengths, (size_t)c.R * 4},
                       {mass, heads * c.page * c.row_pages * 4},
                       {table, (size_t)c.R * c.row_pages * 4},
                       {dst_table, (size_t)c.R * c.dst_row_pages * 4}};
  if (overlap(out, plan) || overlap(found, plan) || overlap(found, out)) return ONELA_ERR_ARG;
  onela::CacheEvictParams p = {};
  p.R = c.R;
  p.Hkv = c.H_kv;
  p.row_bytes = (int)(c.d * es);
  p.page = c.page;
  p.pages = c.pages;
  p.row_pages = c.row_pages;
  p.dst_pages = c.dst_pages;
  p.dst_row_pages = c.dst_row_pages;
  p.keep = c.keep;
  p.recent = c.recent;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.dst_k = dst_k;
  p.dst_v = dst_v;
  p.table = table;
  p.lengths = lengths;
  p.dst_table = dst_table;
  p.dst_lengths = dst_lengths;
  p.kept = kept ? kept : static_cast<int32_t *>(scratch);
  p.mass = mass;
  p.dst_mass = dst_mass;
  p.status = status;
  return on_device(c.device, [&] { return onela::launch_cache_evict(p, static_cast<cudaStream_t>(stream)); });
}

int onela_block_norm(const onela_block_norm_config *cfg, const void *y, const void *gate, const void *x,
                     const float *w_post, const float *scale, const float *w_pre, void *x_out, void *n_out,
                     onela_stream stream) {
  if (!cfg) return ONELA_ERR_ARG;
  const onela_block_norm_config c = *cfg;
  if (c.N < 0 || c.N > 0x7fffffffLL || c.D < 1 || c.D > 32768 || c.group < 1 || c.D % c.group != 0 ||
      !valid_dtype(c.y_dtype) || !valid_dtype(c.dtype) || c.device < 0 || c.act < ONELA_ACT_NONE ||
      c.act > ONELA_ACT_SILU || !(c.eps >= 0.f))
    return ONELA_ERR_ARG;
  if (c.N == 0) return ONELA_OK;  // empty tensors have no address
  if ((!y && !x) || (!y && (gate || w_post || scale)) || (!x_out && !n_out) || (x_out && x_out == n_out) || ((n_out != nullptr) != (w_pre != nullptr)))
    return ONELA_ERR_ARG;
  if ((gate != nullptr) != (c.act != ONELA_ACT_NONE)) return ONELA_ERR_ARG;
  if ((y && c.y_stride < c.D) || (gate && c.gate_stride < c.D) || (x && c.x_stride < c.D)) return ONELA_ERR_ARG;
  // x_out over x keeps every row in its place only when x's rows are dense.
  if (x_out && x_out == x && c.x_stride != c.D) return ONELA_ERR_ARG;
  if (!aligned(y, esize(c.y_dtype))) return ONELA_ERR_ARG;
  for (const void *q : {gate, x, (const void *)x_out, (const void *)n_out})
    if (!aligned(q, esize(c.dtype))) return ONELA_ERR_ARG;
  for (const float *q : {w_post, scale, w_pre})
    if (!aligned(q, 4)) return ONELA_ERR_ARG;
  onela::BlockNormParams p = {};
  p.N = c.N;
  p.y_stride = c.y_stride;
  p.gate_stride = c.gate_stride;
  p.x_stride = c.x_stride;
  p.D = c.D;
  p.group = c.group;
  p.y_bf16 = c.y_dtype == ONELA_BF16;
  p.bf16 = c.dtype == ONELA_BF16;
  p.act = c.act;
  p.alpha = c.alpha;
  p.eps = c.eps;
  p.y = y;
  p.gate = gate;
  p.x = x;
  p.w_post = w_post;
  p.scale = scale;
  p.w_pre = w_pre;
  p.x_out = x_out;
  p.n_out = n_out;
  return on_device(c.device, [&] { return onela::launch_block_norm(p, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
