// C ABI of the 8-bit block-scaled cache and of the page pool: argument checks, workspaces and
// launches.  The declarations and their contracts are in include/tq.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kv8_launch.h"
#include "pages.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int64_t kMaxTokens = 1ll << 30;
constexpr int64_t kMaxRecords = (1ll << 31) - 1;     // row index of a tensor map

tq_status check_kv8(const tq_kv8& c) {
  if (!c.codes || !c.scales) return fail(TQ_ERR_INVALID_ARG, "codes or scales is NULL");
  if (!aligned16(c.codes) || !aligned16(c.scales)) return fail(TQ_ERR_ALIGNMENT, "codes or scales not 16-byte aligned");
  return TQ_OK;
}

// The cache's record map; recs: records of each side.
tq_status map_of(const tq_pages* pages, int B, int Hkv, int64_t Nmax, Kv8Map& m, int64_t& recs) {
  m.Hkv = Hkv;
  if (pages) {
    tq_status s = check_pages(pages);
    if (s != TQ_OK) return s;
    m.table = pages->block_table;
    m.page = pages->page_size;
    m.max_pages = pages->max_pages;
    m.num_pages = pages->num_pages;
    m.cap = static_cast<int64_t>(pages->max_pages) * pages->page_size;
  } else {
    if (Nmax < kKv8Block || Nmax % kKv8Block || Nmax > kMaxTokens)
      return fail(TQ_ERR_INVALID_ARG, "Nmax must be a multiple of %d in %d..2^30 (got %lld)", kKv8Block, kKv8Block,
                  static_cast<long long>(Nmax));
    m.table = nullptr;
    m.page = Nmax;
    m.max_pages = 1;
    m.num_pages = B;
    m.cap = Nmax;
  }
  if (m.num_pages > kMaxRecords / m.page / Hkv)
    return fail(TQ_ERR_UNSUPPORTED, "a side of the cache holds 2^31 records or more");
  recs = m.num_pages * Hkv * m.page;
  return TQ_OK;
}

tq_status check_common(int dtype, int B, int Hkv, int d) {
  if (dtype < TQ_F32 || dtype > TQ_F16) return fail(TQ_ERR_INVALID_ARG, "unknown dtype");
  if (B < 1 || Hkv < 1 || B > (1 << 24) || Hkv > (1 << 16)) return fail(TQ_ERR_INVALID_ARG, "B and Hkv must be >= 1");
  if (d != 64 && d != 128) return fail(TQ_ERR_UNSUPPORTED, "the 8-bit cache takes d = 64 or 128 (got %d)", d);
  return TQ_OK;
}

// Strides of [B][H][T][d] rows (NULL: contiguous), and the bytes that they span.
tq_status strides_of(const tq_strides* in, int dtype, int B, int H, int T, int d, tq_strides& out, size_t& bytes) {
  if (in) out = *in;
  else out = {static_cast<int64_t>(H) * T * d, static_cast<int64_t>(T) * d, d};
  const int64_t unit = dtype == TQ_F32 ? 4 : 8;
  if (out.b < 0 || out.h < 0 || out.t < 0) return fail(TQ_ERR_INVALID_ARG, "strides must be >= 0");
  if ((B > 1 && out.b % unit) || (H > 1 && out.h % unit) || (T > 1 && out.t % unit))
    return fail(TQ_ERR_ALIGNMENT, "strides must keep rows 16-byte aligned");
  int64_t last = d;
  const int64_t steps[3] = {B - 1ll, H - 1ll, T - 1ll}, by[3] = {out.b, out.h, out.t};
  for (int i = 0; i < 3; ++i) {
    if (steps[i] && by[i] > ((1ll << 60) - last) / steps[i]) return fail(TQ_ERR_INVALID_ARG, "strides too large");
    last += steps[i] * by[i];
  }
  bytes = static_cast<size_t>(last) * dtype_size(dtype);
  return TQ_OK;
}

void kv8_ranges(const tq_kv8& c, int64_t recs, int d, Range out[2]) {
  out[0] = {c.codes, static_cast<size_t>(recs) * d};
  out[1] = {c.scales, static_cast<size_t>(recs) / kKv8Block * 4};
}

struct Append {
  const void* k_new;
  const void* v_new;
  const tq_strides* k_strides;
  const tq_strides* v_strides;
  const int32_t* new_lens;
  int T;
};

// Checks an append into the cache and fills its launch; ranges: the new rows.
tq_status prepare_append(const Append& a, int dtype, int B, int Hkv, int d, const int32_t* kv_lens, const Kv8Map& m,
                         int64_t recs, const tq_pages* pages, const tq_kv8& kc, const tq_kv8& vc, Kv8AppendParams& p,
                         Range rows[2]) {
  if (a.T < 1 || a.T > kMaxTokens) return fail(TQ_ERR_INVALID_ARG, "T must be >= 1");
  if (!a.k_new || !a.v_new) return fail(TQ_ERR_INVALID_ARG, "k_new or v_new is NULL");
  if (!aligned16(a.k_new) || !aligned16(a.v_new)) return fail(TQ_ERR_ALIGNMENT, "k_new or v_new not 16-byte aligned");
  if (a.new_lens && !aligned16(a.new_lens)) return fail(TQ_ERR_ALIGNMENT, "new_lens not 16-byte aligned");
  tq_strides st[2];
  size_t bytes[2];
  tq_status s;
  if ((s = strides_of(a.k_strides, dtype, B, Hkv, a.T, d, st[0], bytes[0])) != TQ_OK) return s;
  if ((s = strides_of(a.v_strides, dtype, B, Hkv, a.T, d, st[1], bytes[1])) != TQ_OK) return s;
  rows[0] = {a.k_new, bytes[0]};
  rows[1] = {a.v_new, bytes[1]};
  Range outs[4], ins[5] = {rows[0], rows[1], {kv_lens, static_cast<size_t>(B) * 4},
                           {a.new_lens, a.new_lens ? static_cast<size_t>(B) * 4 : 0},
                           {pages ? pages->block_table : nullptr, static_cast<size_t>(B) * m.max_pages * 4}};
  kv8_ranges(kc, recs, d, outs);
  kv8_ranges(vc, recs, d, outs + 2);
  if ((s = check_no_alias(outs, 4, ins, 5)) != TQ_OK) return s;
  p = {};
  p.x[0] = a.k_new;
  p.x[1] = a.v_new;
  for (int i = 0; i < 2; ++i) {
    p.stride_b[i] = st[i].b;
    p.stride_h[i] = st[i].h;
    p.stride_t[i] = st[i].t;
  }
  p.dtype = dtype;
  p.B = B;
  p.T = a.T;
  p.blocks = (a.T + kKv8Block - 1) / kKv8Block + (a.T > 1 ? 1 : 0);
  p.kv_lens = kv_lens;
  p.new_lens = a.new_lens;
  p.codes[0] = kc.codes;
  p.codes[1] = vc.codes;
  p.scales[0] = kc.scales;
  p.scales[1] = vc.scales;
  p.map = m;
  p.status = device_status_ptr();
  if (2ll * B * Hkv * p.blocks > (1ll << 31)) return fail(TQ_ERR_UNSUPPORTED, "more than 2^31 blocks in one append");
  return TQ_OK;
}

// ---- attention
struct AttnPlan {
  bool prefill;        // the tensor-memory kernel
  bool team;           // else a CTA's warps share its runs, or each has its own
  int64_t VB;          // virtual sequences: row groups of a sequence
  int RG, grid, max_vb, run_cost;
  size_t off_lse, off_plan, bytes;
};

size_t up16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// 16-bit queries with more than 16 rows a key head take the tensor-memory kernel: it works on 256
// rows for what the other spends on 16 (d = 128, eight sequences of 32768 tokens: 20 rows 217 us
// against 279, 128 rows 220 against 1051; one of 1000 tokens: 20 rows 20 against 17, 64 rows 21
// against 26).  fp32 queries always take the other.
AttnPlan plan_attn(int dtype, int B, int Hkv, int G, int T, int d, int64_t cap) {
  AttnPlan P{};
  const int64_t R = static_cast<int64_t>(T) * G;
  P.prefill = dtype != TQ_F32 && R > kKv8DecodeRows;
  const int rows = P.prefill ? kKv8PrefillRows : kKv8DecodeRows, tile = P.prefill ? 128 : kv8_decode_tile(d);
  P.RG = static_cast<int>((R + rows - 1) / rows);
  P.VB = static_cast<int64_t>(B) * P.RG;
  // the tiles of a launch are counted in 32 bits
  P.max_vb = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(P.prefill ? kKv8PrefillMaxVB : kKv8DecodeMaxVB,
                                                                     (1ll << 30) / (cap / tile + 2))));
  const int sms = sm_count();
  const int64_t pairs = std::min<int64_t>(P.VB, P.max_vb) * Hkv, tiles = pairs * (cap / tile + 2);
  const int warps = kv8_decode_warps(R, dtype == TQ_F32);
  // Decode: where the (sequence, key head) pairs are as many as the SMs, each warp takes its own, which
  // needs no joining in the CTA (2048 pairs of up to 512 tokens: 46 us against 130; 192 of up to 8192,
  // d = 64: 40 against 45); else a CTA's warps share one, so that fewer partial results are left to join
  // (64 pairs of 4096 tokens: 26 us against 31).
  P.team = !P.prefill && pairs < sms;
  const int64_t least = P.team ? 8 : 1;
  P.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, (tiles + least - 1) / least)));
  const int64_t parts = P.prefill || P.team ? P.grid : static_cast<int64_t>(P.grid) * warps;
  // What a key head's run costs beside its tiles, in tiles: for a CTA q and the joining of the warps, for
  // a warp q.  Where a part gets few tiles the cut would be the cost's, not the tiles'.
  P.run_cost = static_cast<int>(P.team ? std::clamp<int64_t>((tiles / parts - 16) / 2, 0, 32)
                                       : std::clamp<int64_t>((tiles / parts - 2) / 2, 0, 2));
  P.off_lse = static_cast<size_t>(2) * parts * rows * d * 4;
  P.off_plan = P.off_lse + up16(static_cast<size_t>(2) * parts * rows * 4);
  P.bytes = P.off_plan + static_cast<size_t>(parts) * 16;
  return P;
}

struct AttnCall {
  const void* q;
  const tq_strides* q_strides;
  int dtype, B, Hq, Hkv, T, d;
  const int32_t* q_pos;
  const int32_t* kv_lens;
  const tq_scoring* scoring;
  const tq_pages* pages;
  int64_t Nmax;
  tq_kv8 kc, vc;
  void* out;
  float* lse;
  void* ws;
  size_t ws_bytes;
  cudaStream_t stream;
  const Append* append;
};

tq_status check_attn_shape(int dtype, int B, int Hq, int Hkv, int T, int d) {
  tq_status s = check_common(dtype, B, Hkv, d);
  if (s != TQ_OK) return s;
  if (Hq < 1 || Hq % Hkv) return fail(TQ_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (T < 1 || static_cast<int64_t>(T) * (Hq / Hkv) > (1 << 24)) return fail(TQ_ERR_INVALID_ARG, "T out of range");
  if (static_cast<int64_t>(B) * Hq * T > (1ll << 31)) return fail(TQ_ERR_INVALID_ARG, "too many query rows");
  return TQ_OK;
}

tq_status run_attn(const AttnCall& c) {
  tq_status s = check_attn_shape(c.dtype, c.B, c.Hq, c.Hkv, c.T, c.d);
  if (s != TQ_OK) return s;
  if (!c.q || !c.kv_lens || !c.out) return fail(TQ_ERR_INVALID_ARG, "NULL q, kv_lens or out");
  if (!aligned16(c.q) || !aligned16(c.kv_lens) || !aligned16(c.out) || !aligned16(c.lse) || !aligned16(c.q_pos))
    return fail(TQ_ERR_ALIGNMENT, "q, q_pos, kv_lens, out or lse not 16-byte aligned");
  Kv8Map m{};
  int64_t recs = 0;
  if ((s = map_of(c.pages, c.B, c.Hkv, c.Nmax, m, recs)) != TQ_OK) return s;
  if ((s = check_kv8(c.kc)) != TQ_OK || (s = check_kv8(c.vc)) != TQ_OK) return s;
  tq_scoring sc{};
  sc.scale = 1.f / std::sqrt(static_cast<float>(c.d));
  if (c.scoring) sc = *c.scoring;
  if (!std::isfinite(sc.scale)) return fail(TQ_ERR_INVALID_ARG, "scale must be finite");
  if (sc.softcap != 0.f && !(sc.softcap >= 1e-30f && sc.softcap <= 1e30f))
    return fail(TQ_ERR_INVALID_ARG, "softcap must be 0 or in 1e-30..1e30");
  if (sc.window < 0) return fail(TQ_ERR_INVALID_ARG, "window must be >= 0");
  if (!aligned16(sc.slopes) || !aligned16(sc.first) || !aligned16(sc.prefix))
    return fail(TQ_ERR_ALIGNMENT, "slopes, first or prefix not 16-byte aligned");
  tq_strides qs;
  size_t q_bytes;
  if ((s = strides_of(c.q_strides, c.dtype, c.B, c.Hq, c.T, c.d, qs, q_bytes)) != TQ_OK) return s;

  const int G = c.Hq / c.Hkv;
  const AttnPlan P = plan_attn(c.dtype, c.B, c.Hkv, G, c.T, c.d, m.cap);
  // a sequence's tiles over all key heads are counted in 32 bits
  if ((m.cap / 32 + 32) * c.Hkv > INT32_MAX) return fail(TQ_ERR_UNSUPPORTED, "Hkv times the tokens a sequence can hold is too large");
  if (!c.ws || c.ws_bytes < P.bytes) return fail(TQ_ERR_WORKSPACE, "workspace needs %zu bytes", P.bytes);
  if (!aligned16(c.ws)) return fail(TQ_ERR_ALIGNMENT, "workspace not 16-byte aligned");

  const size_t rows = static_cast<size_t>(c.B) * c.Hq * c.T, bt = static_cast<size_t>(c.B) * c.T * 4;
  Range outs[3] = {{c.out, rows * c.d * dtype_size(c.dtype)}, {c.lse, c.lse ? rows * 4 : 0}, {c.ws, P.bytes}};
  Range ins[12];
  kv8_ranges(c.kc, recs, c.d, ins);
  kv8_ranges(c.vc, recs, c.d, ins + 2);
  ins[4] = {c.q, q_bytes};
  ins[5] = {c.kv_lens, static_cast<size_t>(c.B) * 4};
  ins[6] = {m.table, static_cast<size_t>(c.B) * m.max_pages * 4};
  ins[7] = {c.q_pos, bt};
  ins[8] = {sc.first, bt};
  ins[9] = {sc.prefix, static_cast<size_t>(c.B) * 4};
  ins[10] = {sc.slopes, static_cast<size_t>(c.Hq) * 4};
  if ((s = check_no_alias(outs, 3, ins, 11)) != TQ_OK) return s;

  Kv8AppendParams ap{};
  if (c.append) {
    Range fresh[2];
    if ((s = prepare_append(*c.append, c.dtype, c.B, c.Hkv, c.d, c.kv_lens, m, recs, c.pages, c.kc, c.vc, ap, fresh)) != TQ_OK)
      return s;
    ap.empty_ok = true;
    Range caches[4];
    kv8_ranges(c.kc, recs, c.d, caches);
    kv8_ranges(c.vc, recs, c.d, caches + 2);
    // the cache is written here, so it must not share memory with what the attention reads
    Range reads[5] = {ins[4], ins[7], ins[8], ins[9], ins[10]};
    if ((s = check_no_alias(outs, 3, fresh, 2)) != TQ_OK || (s = check_no_alias(caches, 4, reads, 5)) != TQ_OK) return s;
  }
  CUtensorMap kmap, vmap;
  if (!P.prefill) {
    if ((s = byte_rows_map(&kmap, c.kc.codes, recs, c.d, kKv8Block)) != TQ_OK) return s;
    if ((s = byte_rows_map(&vmap, c.vc.codes, recs, c.d, kKv8Block)) != TQ_OK) return s;
  }
  cudaError_t e = cudaSuccess;
  if (c.append && (e = launch_kv8_append(ap, c.d, c.stream)) != cudaSuccess) return cuda_fail(e, "append launch");

  char* ws = static_cast<char*>(c.ws);
  Kv8AttnParams p{};
  p.q = c.q;
  p.q_stride_b = qs.b;
  p.q_stride_h = qs.h;
  p.q_stride_t = qs.t;
  p.dtype = c.dtype;
  p.Hq = c.Hq;
  p.G = G;
  p.T = c.T;
  p.RG = P.RG;
  p.kscales = c.kc.scales;
  p.vscales = c.vc.scales;
  p.sc.kv_lens = c.kv_lens;
  p.sc.q_pos = c.q_pos;
  p.sc.first = sc.first;
  p.sc.prefix = sc.prefix;
  p.sc.slopes = sc.slopes;
  p.sc.window = sc.window;
  p.sc.scale_log2 = sc.scale * kLog2E;
  p.sc.cap = sc.softcap;
  p.map = m;
  p.out = c.out;
  p.lse = c.lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + P.off_lse);
  p.plan = reinterpret_cast<int*>(ws + P.off_plan);
  p.status = device_status_ptr();
  p.wait_limit = wait_limit();
  p.appended = c.append != nullptr;
  p.run_cost = P.run_cost;
  for (int64_t v = 0; v < P.VB; v += P.max_vb) {
    p.v0 = static_cast<int>(v);
    p.VB = static_cast<int>(std::min<int64_t>(P.max_vb, P.VB - v));
    e = P.prefill ? launch_kv8_prefill(c.kc.codes, c.vc.codes, p, c.d, P.grid, c.stream)
                  : launch_kv8_decode(kmap, vmap, p, c.d, P.team, P.grid, c.stream);
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  }
  return TQ_OK;
}

// ---- page pool
struct PagesPlan {
  size_t off_prefix, off_marks, off_bad, off_from, off_to, bytes;
  int chunks;
};

PagesPlan plan_pages(const tq_page_pool* pool, int64_t n) {
  PagesPlan P{};
  P.chunks = static_cast<int>((pool->num_pages + kPageChunk - 1) / kPageChunk);
  const size_t pairs = static_cast<size_t>(std::max<int64_t>(n, pool->num_pages / 2 + 1)) * 4;
  P.off_prefix = up16(static_cast<size_t>(P.chunks) * 4);
  P.off_marks = P.off_prefix + up16(static_cast<size_t>(n + 1) * 4);
  P.off_bad = P.off_marks + up16(static_cast<size_t>((pool->rows + 31) / 32) * 8);
  P.off_from = P.off_bad + up16(static_cast<size_t>(kCheckBlocks) * 4);
  P.off_to = P.off_from + up16(pairs);
  P.bytes = P.off_to + up16(pairs);
  return P;
}

tq_status check_pool(const tq_page_pool* pool) {
  if (!pool || !pool->block_table || !pool->refs) return fail(TQ_ERR_INVALID_ARG, "pool, block_table or refs is NULL");
  if (!aligned16(pool->block_table) || !aligned16(pool->refs))
    return fail(TQ_ERR_ALIGNMENT, "block_table or refs not 16-byte aligned");
  if (pool->rows < 1 || pool->max_pages < 1 || pool->num_pages < 1 || pool->num_pages > (1ll << 30))
    return fail(TQ_ERR_INVALID_ARG, "rows, max_pages and num_pages must be >= 1 (num_pages at most 2^30)");
  if (pool->page_size < 1 || static_cast<int64_t>(pool->max_pages) * pool->page_size > kMaxTokens)
    return fail(TQ_ERR_INVALID_ARG, "page_size out of range");
  const Range outs[2] = {{pool->block_table, static_cast<size_t>(pool->rows) * pool->max_pages * 4},
                         {pool->refs, static_cast<size_t>(pool->num_pages) * 4}};
  return check_no_alias(outs, 2, nullptr, 0);
}

tq_status check_arrays(const tq_pool_array* arrays, int n, int64_t num_pages, PoolCopy& copy, Range* ranges) {
  if (n < 0 || n > TQ_MAX_POOL_ARRAYS || (n > 0 && !arrays))
    return fail(TQ_ERR_INVALID_ARG, "arrays: 0..%d are taken", TQ_MAX_POOL_ARRAYS);
  copy = {};
  copy.n = n;
  for (int i = 0; i < n; ++i) {
    if (!arrays[i].data) return fail(TQ_ERR_INVALID_ARG, "array %d is NULL", i);
    if (!aligned16(arrays[i].data)) return fail(TQ_ERR_ALIGNMENT, "array %d not 16-byte aligned", i);
    const int64_t pb = arrays[i].page_bytes;
    if (pb < 4 || pb % 4 || pb > (1ll << 34)) return fail(TQ_ERR_INVALID_ARG, "page_bytes must be a positive multiple of 4");
    copy.data[i] = static_cast<char*>(arrays[i].data);
    copy.page_bytes[i] = pb;
    copy.slice0[i + 1] = copy.slice0[i] + static_cast<int>((pb + kCopySlice - 1) / kCopySlice);
    ranges[i] = {arrays[i].data, static_cast<size_t>(pb) * num_pages};
  }
  return TQ_OK;
}

tq_status check_list(const int32_t* v, int n, const char* name) {
  if (!v) return fail(TQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(v)) return fail(TQ_ERR_ALIGNMENT, "%s not 16-byte aligned", name);
  (void)n;
  return TQ_OK;
}

tq_status pool_scratch(const tq_page_pool* pool, int64_t n, void* ws, size_t ws_bytes, PagesParams& p, Range& range) {
  const PagesPlan P = plan_pages(pool, n);
  if (!ws || ws_bytes < P.bytes) return fail(TQ_ERR_WORKSPACE, "workspace needs %zu bytes", P.bytes);
  if (!aligned16(ws)) return fail(TQ_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  char* w = static_cast<char*>(ws);
  p.chunks = P.chunks;
  p.chunk_free = reinterpret_cast<int32_t*>(w);
  p.prefix = reinterpret_cast<int32_t*>(w + P.off_prefix);
  p.marks = reinterpret_cast<uint32_t*>(w + P.off_marks);
  p.bad = reinterpret_cast<int32_t*>(w + P.off_bad);
  p.from = reinterpret_cast<int32_t*>(w + P.off_from);
  p.to = reinterpret_cast<int32_t*>(w + P.off_to);
  range = {ws, P.bytes};
  return TQ_OK;
}

Range list_range(const int32_t* v, int64_t n) { return {v, v ? static_cast<size_t>(n) * 4 : 0}; }

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_kv8_append(const void* k_new, const void* v_new, int32_t dtype, const tq_strides* k_strides,
                        const tq_strides* v_strides, int32_t B, int32_t Hkv, int32_t T, int32_t d,
                        const int32_t* kv_lens, const int32_t* new_lens, const tq_pages* pages, int64_t Nmax,
                        tq_kv8 kcache, tq_kv8 vcache, tq_stream stream) {
  tq_status s = check_common(dtype, B, Hkv, d);
  if (s != TQ_OK) return s;
  if (!kv_lens) return fail(TQ_ERR_INVALID_ARG, "kv_lens is NULL");
  if (!aligned16(kv_lens)) return fail(TQ_ERR_ALIGNMENT, "kv_lens not 16-byte aligned");
  Kv8Map m{};
  int64_t recs = 0;
  if ((s = map_of(pages, B, Hkv, Nmax, m, recs)) != TQ_OK) return s;
  if ((s = check_kv8(kcache)) != TQ_OK || (s = check_kv8(vcache)) != TQ_OK) return s;
  const Append a{k_new, v_new, k_strides, v_strides, new_lens, T};
  Kv8AppendParams p;
  Range rows[2];
  if ((s = prepare_append(a, dtype, B, Hkv, d, kv_lens, m, recs, pages, kcache, vcache, p, rows)) != TQ_OK) return s;
  const cudaError_t e = launch_kv8_append(p, d, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "append launch");
}

tq_status tq_kv8_attn_workspace(int32_t dtype, int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t d, int64_t Nmax,
                                size_t* bytes) {
  tq_status s = check_attn_shape(dtype, B, Hq, Hkv, T, d);
  if (s != TQ_OK) return s;
  if (!bytes || Nmax < 1 || Nmax > kMaxTokens) return fail(TQ_ERR_INVALID_ARG, "bad workspace query");
  *bytes = plan_attn(dtype, B, Hkv, Hq / Hkv, T, d, Nmax).bytes;
  return TQ_OK;
}

tq_status tq_kv8_decode_attn(const void* q, const tq_strides* q_strides, int32_t dtype, int32_t B, int32_t Hq,
                             int32_t Hkv, int32_t d, const int32_t* kv_lens, const tq_scoring* scoring,
                             const tq_pages* pages, int64_t Nmax, const void* k_new, const void* v_new,
                             const tq_strides* k_strides, const tq_strides* v_strides, tq_kv8 kcache, tq_kv8 vcache,
                             void* out, float* lse, void* workspace, size_t ws_bytes, tq_stream stream) {
  if ((k_new == nullptr) != (v_new == nullptr)) return fail(TQ_ERR_INVALID_ARG, "k_new and v_new go together");
  const Append a{k_new, v_new, k_strides, v_strides, nullptr, 1};
  const AttnCall c{q, q_strides, dtype, B, Hq, Hkv, 1, d, nullptr, kv_lens, scoring, pages, Nmax, kcache, vcache, out, lse,
                   workspace, ws_bytes, reinterpret_cast<cudaStream_t>(stream), k_new ? &a : nullptr};
  return run_attn(c);
}

tq_status tq_kv8_prefill_attn(const void* q, const tq_strides* q_strides, int32_t dtype, int32_t B, int32_t Hq,
                              int32_t Hkv, int32_t T, int32_t d, const int32_t* q_pos, const int32_t* kv_lens,
                              const tq_scoring* scoring, const tq_pages* pages, int64_t Nmax, tq_kv8 kcache,
                              tq_kv8 vcache, void* out, float* lse, void* workspace, size_t ws_bytes, tq_stream stream) {
  if (!q_pos) return fail(TQ_ERR_INVALID_ARG, "q_pos is NULL");
  const AttnCall c{q, q_strides, dtype, B, Hq, Hkv, T, d, q_pos, kv_lens, scoring, pages, Nmax, kcache, vcache, out, lse,
                   workspace, ws_bytes, reinterpret_cast<cudaStream_t>(stream), nullptr};
  return run_attn(c);
}

tq_status tq_pages_workspace(const tq_page_pool* pool, int32_t n, size_t* bytes) {
  tq_status s = check_pool(pool);
  if (s != TQ_OK) return s;
  if (!bytes || n < 0) return fail(TQ_ERR_INVALID_ARG, "bad workspace query");
  *bytes = plan_pages(pool, n).bytes;
  return TQ_OK;
}

tq_status tq_pages_free(const tq_page_pool* pool, const int32_t* rows, const int32_t* lens, int32_t n, tq_stream stream) {
  tq_status s = check_pool(pool);
  if (s != TQ_OK) return s;
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "n must be >= 0");
  if (n == 0) return TQ_OK;
  if ((s = check_list(rows, n, "rows")) != TQ_OK || (s = check_list(lens, n, "lens")) != TQ_OK) return s;
  const Range outs[2] = {{pool->block_table, static_cast<size_t>(pool->rows) * pool->max_pages * 4},
                         {pool->refs, static_cast<size_t>(pool->num_pages) * 4}};
  const Range ins[2] = {list_range(rows, n), list_range(lens, n)};
  if ((s = check_no_alias(outs, 2, ins, 2)) != TQ_OK) return s;
  PagesParams p{};
  p.pool = *pool;
  p.rows = rows;
  p.lens = lens;
  p.n = n;
  p.status = device_status_ptr();
  const cudaError_t e = launch_pages_free(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "pages_free launch");
}

tq_status tq_pages_reserve(const tq_page_pool* pool, const int32_t* rows, const int32_t* old_lens,
                           const int32_t* new_lens, int32_t n, int32_t* shortfall, void* workspace, size_t ws_bytes,
                           tq_stream stream) {
  tq_status s = check_pool(pool);
  if (s != TQ_OK) return s;
  if (n < 1) return fail(TQ_ERR_INVALID_ARG, "n must be >= 1");
  if ((s = check_list(rows, n, "rows")) != TQ_OK || (s = check_list(old_lens, n, "old_lens")) != TQ_OK ||
      (s = check_list(new_lens, n, "new_lens")) != TQ_OK || (s = check_list(shortfall, 1, "shortfall")) != TQ_OK)
    return s;
  PagesParams p{};
  Range outs[4] = {{pool->block_table, static_cast<size_t>(pool->rows) * pool->max_pages * 4},
                   {pool->refs, static_cast<size_t>(pool->num_pages) * 4}, {shortfall, 4}, {}};
  if ((s = pool_scratch(pool, n, workspace, ws_bytes, p, outs[3])) != TQ_OK) return s;
  const Range ins[3] = {list_range(rows, n), list_range(old_lens, n), list_range(new_lens, n)};
  if ((s = check_no_alias(outs, 4, ins, 3)) != TQ_OK) return s;
  p.pool = *pool;
  p.rows = rows;
  p.old_lens = old_lens;
  p.lens = new_lens;
  p.n = n;
  p.shortfall = shortfall;
  p.status = device_status_ptr();
  const cudaError_t e = launch_pages_reserve(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "pages_reserve launch");
}

tq_status tq_pages_fork(const tq_page_pool* pool, const tq_pool_array* arrays, int32_t n_arrays, const int32_t* src,
                        const int32_t* dst, const int32_t* lens, int32_t n, int32_t* shortfall, void* workspace,
                        size_t ws_bytes, tq_stream stream) {
  tq_status s = check_pool(pool);
  if (s != TQ_OK) return s;
  if (n < 1) return fail(TQ_ERR_INVALID_ARG, "n must be >= 1");
  if ((s = check_list(src, n, "src")) != TQ_OK || (s = check_list(dst, n, "dst")) != TQ_OK ||
      (s = check_list(lens, n, "lens")) != TQ_OK || (s = check_list(shortfall, 1, "shortfall")) != TQ_OK)
    return s;
  PagesParams p{};
  Range outs[4 + TQ_MAX_POOL_ARRAYS] = {{pool->block_table, static_cast<size_t>(pool->rows) * pool->max_pages * 4},
                                        {pool->refs, static_cast<size_t>(pool->num_pages) * 4}, {shortfall, 4}, {}};
  if ((s = pool_scratch(pool, n, workspace, ws_bytes, p, outs[3])) != TQ_OK) return s;
  if ((s = check_arrays(arrays, n_arrays, pool->num_pages, p.copy, outs + 4)) != TQ_OK) return s;
  const Range ins[3] = {list_range(src, n), list_range(dst, n), list_range(lens, n)};
  if ((s = check_no_alias(outs, 4 + n_arrays, ins, 3)) != TQ_OK) return s;
  p.pool = *pool;
  p.src = src;
  p.rows = dst;
  p.lens = lens;
  p.n = n;
  p.shortfall = shortfall;
  p.status = device_status_ptr();
  const cudaError_t e = launch_pages_fork(p, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "pages_fork launch");
}

tq_status tq_pages_compact(const tq_page_pool* pool, const tq_pool_array* arrays, int32_t n_arrays, int32_t* page_map,
                           int32_t* live, void* workspace, size_t ws_bytes, tq_stream stream) {
  tq_status s = check_pool(pool);
  if (s != TQ_OK) return s;
  if ((s = check_list(page_map, 1, "page_map")) != TQ_OK || (s = check_list(live, 1, "live")) != TQ_OK) return s;
  PagesParams p{};
  Range outs[5 + TQ_MAX_POOL_ARRAYS] = {{pool->block_table, static_cast<size_t>(pool->rows) * pool->max_pages * 4},
                                        {pool->refs, static_cast<size_t>(pool->num_pages) * 4},
                                        {page_map, static_cast<size_t>(pool->num_pages) * 4}, {live, 4}, {}};
  if ((s = pool_scratch(pool, 0, workspace, ws_bytes, p, outs[4])) != TQ_OK) return s;
  if ((s = check_arrays(arrays, n_arrays, pool->num_pages, p.copy, outs + 5)) != TQ_OK) return s;
  if ((s = check_no_alias(outs, 5 + n_arrays, nullptr, 0)) != TQ_OK) return s;
  p.pool = *pool;
  p.page_map = page_map;
  p.live = live;
  p.status = device_status_ptr();
  const cudaError_t e = launch_pages_compact(p, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "pages_compact launch");
}

tq_status tq_pages_copy(const tq_pool_array* arrays, int32_t n_arrays, int64_t num_pages, const int32_t* src,
                        const int32_t* dst, int32_t n, tq_stream stream) {
  if (n < 0 || num_pages < 1 || num_pages > (1ll << 30)) return fail(TQ_ERR_INVALID_ARG, "n or num_pages out of range");
  PagesParams p{};
  Range outs[TQ_MAX_POOL_ARRAYS];
  tq_status s = check_arrays(arrays, n_arrays, num_pages, p.copy, outs);
  if (s != TQ_OK) return s;
  if (n == 0 || n_arrays == 0) return TQ_OK;
  if ((s = check_list(src, n, "src")) != TQ_OK || (s = check_list(dst, n, "dst")) != TQ_OK) return s;
  const Range ins[2] = {list_range(src, n), list_range(dst, n)};
  if ((s = check_no_alias(outs, n_arrays, ins, 2)) != TQ_OK) return s;
  p.pool.num_pages = num_pages;
  p.src = src;
  p.rows = dst;
  p.n = n;
  p.status = device_status_ptr();
  const cudaError_t e = launch_pages_copy(p, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "pages_copy launch");
}

}  // extern "C"
