// Host side of the decode-step entry points of include/nexus.h (nx_qk_norm_rope,
// nx_paged_*): argument validation, workspace carving and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged.hpp"

using namespace nx;

namespace {

constexpr int64_t kMaxCacheRows = int64_t(1) << 24;
// What a head's table may hold: the attention sums 64 heads' blocks in 32 bits.
constexpr int64_t kMaxHeadRows = int64_t(1) << 29;
constexpr int64_t kMaxGrid = int64_t(1) << 23;   // workgroups of up to 512 threads: 2^32 threads
constexpr int64_t kCUs = 256;
// Workgroups per CU that an attention call is cut into.  16-row tiles: one
// where that leaves four pieces a head (it reads at the memory's rate already,
// with fewer pieces to merge: 8 heads of 32768 rows 19.8 us, two 21.4), else
// two (128 uneven heads: 66 us, one 74).  32-row tiles: two (registers).
constexpr int64_t kPiecesPerHead = 4;
// Fewest blocks of a full piece: one per wavefront (8 heads of 6810 rows: 12.4 us,
// with eight blocks 13.6).
constexpr int64_t kMinShare = 4;
// Heads of up to kWholeTokens rows are taken whole by a workgroup each (8 heads of
// 819 rows: 8.9 us, in shares 9.2; of 1536: 11.5 and 9.6), of up to kWholeMany
// rows where they nearly fill one round of workgroups (128 heads of 2560 rows:
// 18.5 and 23.0, of 3200: 28.7 and 26.2; 256 of 2560: 34.7 and 36.6; but 64 of
// 2048: 15.0 and 14.2, 384 of 2048: 46.0 and 42.6).  From kRounds heads on the
// rounds of workgroups even out by themselves, and every workgroup's search
// through the heads for its piece costs more: whole up to kWholeRounds rows (1024
// heads of 256 to 4096 rows: 115 and 133, of 512 to 16384: 411 and 469, 4096 of
// 1024: 202 and 355; 512 of 512 to 16384: 231 and 210), with 32-row tiles up to a
// quarter (32 query rows, 512 to 4096 rows: 141 and 172; 128, 512 to 8192: 686 and 569).
constexpr int64_t kWholeTokens = 1024, kWholeMany = 2560, kManyHeads = 96;
constexpr int64_t kWholeRounds = 16384, kRounds = 1024;
// Codes of more than this many bytes are read and written past the caches (a
// quarter of the 256 MB cache: other layers' calls lie between two uses of the
// same bytes).  Attention over 268 MB: 51.1 us, cached 56.9, 134 MB: 30.5 and
// 34.7, 67 MB: 21.0 and 19.9.  An append that writes 106 MB: 79 us, cached 81.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

int32_t elem_size(int32_t dtype) { return dtype == NX_BF16 ? 2 : 4; }
bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Of the 32-bit arrays: tables, counts, starts, positions, scales.
bool words(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

struct Range {
  uintptr_t lo, hi;
};
Range bytes_at(const void* p, int64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(n)};
}
// (An array of no bytes meets nothing, wherever it lies.)
bool overlap(Range a, Range b) { return std::max(a.lo, b.lo) < std::min(a.hi, b.hi); }

// A set of rows as the calls address it.
struct RowSet {
  const nx_rows* r;
  int64_t n, heads, d, esz;
  int64_t extent() const { return (heads > 1 ? (heads - 1) * r->head_stride : 0) + d; }   // of one row's heads
  Range range() const {
    return bytes_at(r->p, n ? ((n > 1 ? (n - 1) * r->row_stride : 0) + extent()) * esz : 0);
  }
};

// Exact for two sets that share a row stride which holds a whole row of each
// (slices of one fused projection); otherwise by address range.
bool overlap(const RowSet& a, const RowSet& b) {
  if (!overlap(a.range(), b.range())) return false;
  const int64_t rs = a.r->row_stride;
  if (a.n > 1 && rs == b.r->row_stride && a.extent() <= rs && b.extent() <= rs) {
    const int64_t diff = int64_t(reinterpret_cast<uintptr_t>(b.r->p) - reinterpret_cast<uintptr_t>(a.r->p));
    const int64_t at = ((diff / a.esz) % rs + rs) % rs;
    return !(at >= a.extent() && at + b.extent() <= rs);
  }
  return true;
}
// Strides between rows or heads of which there is one only may be anything.
bool same_rows(const RowSet& a, const RowSet& b) {
  return a.r->p == b.r->p && (a.n <= 1 || a.r->row_stride == b.r->row_stride) &&
         (a.heads == 1 || a.r->head_stride == b.r->head_stride);
}

nx_status check_rows(const RowSet& s, bool output) {
  if (s.r == nullptr || (s.r->p == nullptr && s.n > 0)) return NX_EINVAL;
  const int64_t row = s.n > 1 ? s.r->row_stride : 0, head = s.heads > 1 ? s.r->head_stride : 0;
  if (row < 0 || head < 0) return NX_EINVAL;
  if (!aligned(s.r->p) || row * s.esz % 16 || head * s.esz % 16) return NX_EUNSUPPORTED;
  if (output) {   // rows of an output must not share memory
    const bool by_row = (s.heads == 1 || s.r->head_stride >= s.d) && (s.n <= 1 || s.r->row_stride >= s.extent());
    const bool by_head = (s.n <= 1 || s.r->row_stride >= s.d) &&
                         (s.heads == 1 || s.r->head_stride >= (s.n - 1) * s.r->row_stride + s.d);
    if (!by_row && !by_head) return NX_EINVAL;
  }
  return NX_OK;
}

nx_status check_rope(const nx_rope* r, int32_t head_dim) {
  if (r == nullptr) return NX_OK;
  if (r->cos_sin == nullptr || r->n_pos < 1 || r->rot_dim < 0 || r->rot_dim > head_dim) return NX_EINVAL;
  if (r->style != NX_ROPE_HALF && r->style != NX_ROPE_PAIRS) return NX_EINVAL;
  if (r->rot_dim % 16 || !aligned(r->cos_sin) || !words(r->positions)) return NX_EUNSUPPORTED;
  return NX_OK;
}

// Whether an output meets the rotation's arrays.
bool meets(const Range& out, const nx_rope* r, int64_t n_rows) {
  return r != nullptr && (overlap(out, bytes_at(r->cos_sin, int64_t(r->n_pos) * r->rot_dim * 4)) ||
                          overlap(out, bytes_at(r->positions, r->positions != nullptr ? n_rows * 4 : 0)));
}

nx_status check_shape(const nx_paged* c) {
  if (c == nullptr) return NX_EINVAL;
  if (c->n_seqs < 1 || c->n_kv_heads < 1 || c->n_q_heads < c->n_kv_heads || c->n_q_heads % c->n_kv_heads)
    return NX_EINVAL;
  if (c->n_pages < 1 || c->max_pages < 1 || c->page_blocks < 1) return NX_EINVAL;
  if (c->dtype != NX_BF16 && c->dtype != NX_F32) return NX_EUNSUPPORTED;
  if (c->format != NX_CACHE_E4M3 && c->format != NX_CACHE_I8) return NX_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return NX_EUNSUPPORTED;
  if (c->page_blocks > 1024 || (c->page_blocks & (c->page_blocks - 1))) return NX_EUNSUPPORTED;
  if (c->n_q_heads / c->n_kv_heads > 256) return NX_EUNSUPPORTED;
  if (int64_t(c->n_seqs) * c->n_kv_heads > 65535) return NX_EUNSUPPORTED;     // grid y
  if (int64_t(c->n_pages) * c->page_blocks > INT32_MAX) return NX_EUNSUPPORTED;
  if (int64_t(c->max_pages) * c->page_blocks * kBlock > kMaxHeadRows) return NX_EUNSUPPORTED;
  return NX_OK;
}

struct CacheRanges {
  Range r[6];   // codes, scales, tails
};
CacheRanges cache_ranges(const nx_paged* c) {
  const int64_t blocks = int64_t(c->n_pages) * c->page_blocks;
  const int64_t units = int64_t(c->n_seqs) * c->n_kv_heads;
  const int64_t codes = blocks * kBlock * c->head_dim;
  const int64_t tail = units * kBlock * c->head_dim * elem_size(c->dtype);
  return {{bytes_at(c->k_codes, codes), bytes_at(c->v_codes, codes), bytes_at(c->k_scale, blocks * 4),
           bytes_at(c->v_scale, blocks * 4), bytes_at(c->k_tail, tail), bytes_at(c->v_tail, tail)}};
}

nx_status check_cache(const nx_paged* c) {
  nx_status st = check_shape(c);
  if (st != NX_OK) return st;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail || !c->table ||
      !c->lens)
    return NX_EINVAL;
  if (!aligned(c->k_codes) || !aligned(c->v_codes) || !aligned(c->k_tail) || !aligned(c->v_tail))
    return NX_EUNSUPPORTED;
  if (!words(c->k_scale) || !words(c->v_scale) || !words(c->table) || !words(c->lens) || !aligned(c->workspace))
    return NX_EUNSUPPORTED;
  if (c->workspace == nullptr || c->workspace_bytes < 256) return NX_EWORKSPACE;
  return NX_OK;
}

PagedArgs base_args(const nx_paged* c) {
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = *c;
  a.group = c->n_q_heads / c->n_kv_heads;
  while ((1 << a.page_shift) < c->page_blocks) ++a.page_shift;
  a.status = static_cast<uint32_t*>(c->workspace);
  return a;
}

// How an attention call is cut: query-row tiles and pieces of about equal size.
// Heads in several pieces have at most 2 n_wg pieces together.
struct Cut {
  int64_t tile, n_rt, n_wg;
  int64_t bytes;         // of codes, at max_tokens rows a head
  bool whole;            // a workgroup per head and row tile
};
nx_status make_cut(const nx_paged* c, int64_t max_tokens, int64_t max_q, Cut* out) {
  if (max_tokens < 0 || max_q < 1) return NX_EINVAL;
  const int64_t rows = max_q * (c->n_q_heads / c->n_kv_heads);
  if (max_tokens > kMaxCacheRows || rows > (int64_t(1) << 20)) return NX_EUNSUPPORTED;
  const int64_t tile = paged_tile_rows(rows);
  const int64_t n_rt = (rows + tile - 1) / tile;
  const int64_t units = int64_t(c->n_seqs) * c->n_kv_heads;
  // One round of workgroups fills the chip; no more than there are smallest
  // pieces.
  const int64_t blocks = units * std::max<int64_t>(1, (max_tokens + kBlock - 1) / kBlock);
  const int64_t per_cu = tile == 16 && units * kPiecesPerHead <= kCUs ? 1 : 2;
  const int64_t most = std::max<int64_t>(8, kCUs * per_cu / n_rt);
  const int64_t n_wg = std::min(most, (blocks + kMinShare - 1) / kMinShare);
  if ((n_wg + units + 16) * n_rt >= kMaxGrid) return NX_EUNSUPPORTED;
  const int64_t whole = units >= kRounds ? (tile == 16 ? kWholeRounds : kWholeRounds / 4)
                        : units >= kManyHeads && units <= kCUs ? kWholeMany : kWholeTokens;
  *out = {tile, n_rt, (n_wg + 7) / 8 * 8, blocks * kBlock * 2 * c->head_dim, max_tokens <= whole};
  return NX_OK;
}
// Workspace: status word, the heads' pieces, partials.
size_t pieces_bytes(const nx_paged* c) { return align256(size_t(c->n_seqs) * c->n_kv_heads * sizeof(int2)); }
size_t part_ml_bytes(const Cut& k) { return align256(size_t(2 * k.n_wg * k.n_rt * k.tile) * 2 * sizeof(float)); }
size_t cut_bytes(const nx_paged* c, const Cut& k) {
  return 256 + pieces_bytes(c) + part_ml_bytes(k) + size_t(2 * k.n_wg * k.n_rt * k.tile) * c->head_dim * sizeof(float);
}
// The most that calls of up to max_tokens rows and max_q queries take.  The rounding
// of n_wg and the change of tile size make a call's bytes rise and fall with its
// query rows, so every count is asked for, up to the 2 kCUs / 8 row tiles past
// which n_wg is the constant 8 and bytes only rise.  (They never fall as
// max_tokens rises.)
size_t most_bytes(const nx_paged* c, int64_t max_tokens, int64_t max_q) {
  Cut k;
  if (make_cut(c, max_tokens, max_q, &k) != NX_OK) return 0;
  size_t most = cut_bytes(c, k);
  const int64_t rows = 2 * kCUs / 8 * 32, group = c->n_q_heads / c->n_kv_heads;
  for (int64_t q = std::min(max_q, rows / group + 1); q > 0; --q)
    if (make_cut(c, max_tokens, q, &k) == NX_OK) most = std::max(most, cut_bytes(c, k));
  return most;
}

}  // namespace

extern "C" {

size_t nx_paged_workspace_bytes(const nx_paged* cache, int32_t max_tokens, int32_t max_q) {
  return check_shape(cache) == NX_OK ? most_bytes(cache, max_tokens, max_q) : 0;
}

nx_status nx_qk_norm_rope(const nx_desc* desc, const nx_rope* rope, int32_t n_rows, const nx_rows* q,
                          const nx_rows* out_q, const void* q_weight, const nx_rows* k,
                          const nx_rows* out_k, const void* k_weight, float eps) {
  if (desc == nullptr || n_rows < 0) return NX_EINVAL;
  if (desc->n_kv_heads < 1 || desc->n_q_heads < 1) return NX_EINVAL;
  if (desc->dtype != NX_BF16 && desc->dtype != NX_F32) return NX_EUNSUPPORTED;
  if (desc->head_dim != 64 && desc->head_dim != 128) return NX_EUNSUPPORTED;
  if (!std::isfinite(eps) || eps < 0.f) return NX_EINVAL;
  if ((k == nullptr) != (out_k == nullptr) || (k == nullptr && k_weight != nullptr)) return NX_EINVAL;
  nx_status st = check_rope(rope, desc->head_dim);
  if (st != NX_OK) return st;
  const int64_t esz = elem_size(desc->dtype), d = desc->head_dim;
  const RowSet sq{q, n_rows, desc->n_q_heads, d, esz}, soq{out_q, n_rows, desc->n_q_heads, d, esz};
  const RowSet sk{k, n_rows, desc->n_kv_heads, d, esz}, sok{out_k, n_rows, desc->n_kv_heads, d, esz};
  if ((st = check_rows(sq, false)) != NX_OK || (st = check_rows(soq, true)) != NX_OK) return st;
  if (!same_rows(sq, soq) && overlap(sq, soq)) return NX_EALIAS;
  if (k != nullptr) {
    if ((st = check_rows(sk, false)) != NX_OK || (st = check_rows(sok, true)) != NX_OK) return st;
    if (!same_rows(sk, sok) && overlap(sk, sok)) return NX_EALIAS;
    if (overlap(soq, sk) || overlap(soq, sok) || overlap(sok, sq)) return NX_EALIAS;
  }
  if (!aligned(q_weight) || !aligned(k_weight) || !aligned(desc->workspace)) return NX_EUNSUPPORTED;
  const Range status = bytes_at(desc->workspace, 256);
  if (overlap(status, sq.range()) || (k != nullptr && overlap(status, sk.range())) || meets(status, rope, n_rows) ||
      overlap(status, bytes_at(q_weight, q_weight != nullptr ? d * esz : 0)) ||
      overlap(status, bytes_at(k_weight, k_weight != nullptr ? d * esz : 0)))
    return NX_EALIAS;
  for (const RowSet* o : {&soq, &sok}) {
    if (o == &sok && k == nullptr) break;
    const Range r = o->range();
    if (meets(r, rope, n_rows) || overlap(r, bytes_at(q_weight, q_weight != nullptr ? d * esz : 0)) ||
        overlap(r, bytes_at(k_weight, k_weight != nullptr ? d * esz : 0)) ||
        overlap(r, status))
      return NX_EALIAS;
  }
  if (desc->workspace == nullptr || desc->workspace_bytes < 256) return NX_EWORKSPACE;
  if (n_rows == 0) return NX_OK;
  if (int64_t(n_rows) * (int64_t(desc->n_q_heads) + desc->n_kv_heads) / (4096 / d) >= kMaxGrid - 1)
    return NX_EUNSUPPORTED;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  if (rope != nullptr) a.rope = *rope;
  a.in[0] = *q;
  a.out[0] = *out_q;
  a.weight[0] = q_weight;
  a.heads[0] = desc->n_q_heads;
  if (k != nullptr) {
    a.in[1] = *k;
    a.out[1] = *out_k;
    a.weight[1] = k_weight;
    a.heads[1] = desc->n_kv_heads;
  }
  a.n_rows = n_rows;
  a.head_dim = desc->head_dim;
  a.dtype = desc->dtype;
  a.eps = eps;
  a.status = static_cast<uint32_t*>(desc->workspace);
  hipStream_t s = static_cast<hipStream_t>(desc->stream);
  if (launch_norm_rope(a, s) != hipSuccess) return NX_EHIP;
  return debug_status(a.status, s, "qk_norm_rope");
}

nx_status nx_paged_append(const nx_paged* cache, const nx_rope* rope, const nx_rows* k, const nx_rows* v,
                          int32_t n_rows, const int32_t* new_start, const int32_t* head_new,
                          int32_t max_new, int32_t* lens_out) {
  nx_status st = check_cache(cache);
  if (st != NX_OK) return st;
  if (n_rows < 0 || max_new < 0 || max_new > kMaxCacheRows) return NX_EINVAL;
  if (!words(new_start) || !words(head_new) || !words(lens_out)) return NX_EUNSUPPORTED;
  if ((int64_t(max_new) / kBlock + 8) * cache->n_kv_heads >= kMaxGrid) return NX_EUNSUPPORTED;
  if (new_start == nullptr && int64_t(cache->n_seqs) * max_new > n_rows) return NX_EINVAL;
  if ((st = check_rope(rope, cache->head_dim)) != NX_OK) return st;
  const int64_t esz = elem_size(cache->dtype), d = cache->head_dim;
  const RowSet sk{k, n_rows, cache->n_kv_heads, d, esz}, sv{v, n_rows, cache->n_kv_heads, d, esz};
  if ((st = check_rows(sk, false)) != NX_OK || (st = check_rows(sv, false)) != NX_OK) return st;
  // A block's 32 rows are addressed by 32-bit offsets.
  if (n_rows > 1 && std::max(k->row_stride, v->row_stride) * esz >= (int64_t(1) << 31) / kBlock - 4096) return NX_EUNSUPPORTED;
  const CacheRanges cr = cache_ranges(cache);
  const int64_t units = int64_t(cache->n_seqs) * cache->n_kv_heads;
  const Range lens = bytes_at(cache->lens, units * 4);
  const Range lout = bytes_at(lens_out != nullptr ? lens_out : cache->lens, units * 4);
  // lens_out is written while some workgroups still read the counts and starts.
  const Range ins[] = {sk.range(), sv.range(), bytes_at(cache->table, units * cache->max_pages * 4),
                       bytes_at(head_new, head_new != nullptr ? units * 4 : 0),
                       bytes_at(new_start, new_start != nullptr ? (int64_t(cache->n_seqs) + 1) * 4 : 0),
                       bytes_at(cache->workspace, 256)};
  const Range& status = ins[5];
  for (int i = 0; i < 5; ++i)
    if (overlap(status, ins[i])) return NX_EALIAS;
  if (meets(status, rope, n_rows)) return NX_EALIAS;
  for (int i = 0; i < 6; ++i) {
    for (int j = i + 1; j < 6; ++j)
      if (overlap(cr.r[i], cr.r[j])) return NX_EALIAS;
    for (const Range& x : ins)
      if (overlap(cr.r[i], x)) return NX_EALIAS;
    if (overlap(cr.r[i], lens) || overlap(cr.r[i], lout) || meets(cr.r[i], rope, n_rows)) return NX_EALIAS;
  }
  for (const Range& x : ins)
    if (overlap(lout, x)) return NX_EALIAS;
  if (meets(lout, rope, n_rows) || (lout.lo != lens.lo && overlap(lout, lens))) return NX_EALIAS;
  PagedArgs a = base_args(cache);
  if (rope != nullptr) a.rope = *rope;
  a.k = *k;
  a.v = *v;
  a.n_rows = n_rows;
  a.max_new = max_new;
  a.start = new_start;
  a.head_new = head_new;
  a.lens_out = lens_out != nullptr ? lens_out : cache->lens;
  a.stream_nt = int64_t(n_rows) * cache->n_kv_heads * 2 * d > kStreamBytes;
  hipStream_t s = static_cast<hipStream_t>(cache->stream);
  if (launch_paged_append(a, s) != hipSuccess) return NX_EHIP;
  return debug_status(a.status, s, "paged_append");
}

nx_status nx_paged_attn(const nx_paged* cache, const nx_rows* q, const nx_rows* out, int32_t n_rows,
                        const int32_t* q_start, int32_t max_tokens, int32_t max_q, float scale,
                        float* out_lse) {
  nx_status st = check_cache(cache);
  if (st != NX_OK) return st;
  if (n_rows < 0 || !std::isfinite(scale) || scale < 0.f) return NX_EINVAL;
  if (!words(q_start) || !words(out_lse)) return NX_EUNSUPPORTED;
  if (q_start == nullptr && n_rows > 0 && int64_t(cache->n_seqs) * max_q > n_rows) return NX_EINVAL;
  Cut cut;
  if ((st = make_cut(cache, max_tokens, max_q, &cut)) != NX_OK) return st;
  const int64_t esz = elem_size(cache->dtype), d = cache->head_dim;
  const RowSet sq{q, n_rows, cache->n_q_heads, d, esz}, so{out, n_rows, cache->n_q_heads, d, esz};
  if ((st = check_rows(sq, false)) != NX_OK || (st = check_rows(so, true)) != NX_OK) return st;
  if (overlap(sq, so)) return NX_EALIAS;
  const CacheRanges cr = cache_ranges(cache);
  const Range lse = bytes_at(out_lse, out_lse != nullptr ? int64_t(n_rows) * cache->n_q_heads * 4 : 0);
  const int64_t units = int64_t(cache->n_seqs) * cache->n_kv_heads;
  // (A workspace that is too small is refused below, not taken to reach into what follows it.)
  const Range ro = so.range(), ins[] = {
      bytes_at(cache->table, units * cache->max_pages * 4), bytes_at(cache->lens, units * 4),
      bytes_at(q_start, q_start != nullptr ? (int64_t(cache->n_seqs) + 1) * 4 : 0),
      bytes_at(cache->workspace, int64_t(std::min(cache->workspace_bytes, cut_bytes(cache, cut))))};
  for (int i = 0; i < 3; ++i)
    if (overlap(ins[3], ins[i])) return NX_EALIAS;
  if (overlap(ins[3], sq.range())) return NX_EALIAS;
  for (const Range& x : cr.r)
    if (overlap(ins[3], x)) return NX_EALIAS;
  for (const Range& x : cr.r)
    if (overlap(ro, x) || overlap(lse, x)) return NX_EALIAS;
  for (const Range& x : ins)
    if (overlap(ro, x) || overlap(lse, x)) return NX_EALIAS;
  if (overlap(lse, sq.range()) || overlap(lse, ro)) return NX_EALIAS;
  if (cache->workspace_bytes < cut_bytes(cache, cut)) return NX_EWORKSPACE;
  if (n_rows == 0) return NX_OK;
  PagedArgs a = base_args(cache);
  a.q = *q;
  a.out = *out;
  a.n_rows = n_rows;
  a.start = q_start;
  a.max_q = max_q;
  a.n_rt = int32_t(cut.n_rt);
  a.n_wg = int32_t(cut.n_wg);
  a.min_share = int32_t(kMinShare);
  a.whole = cut.whole;
  a.stream_nt = cut.n_rt == 1 && cut.bytes > kStreamBytes;
  a.scale_log2 = float((scale > 0.f ? double(scale) : 1.0 / std::sqrt(double(d))) * 1.4426950408889634);
  a.lse = out_lse;
  char* ws = static_cast<char*>(cache->workspace) + 256;
  a.pieces = reinterpret_cast<int2*>(ws);
  ws += pieces_bytes(cache);
  a.part_ml = reinterpret_cast<float*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + part_ml_bytes(cut));
  hipStream_t s = static_cast<hipStream_t>(cache->stream);
  if (launch_paged_attn(a, s) != hipSuccess) return NX_EHIP;
  return debug_status(a.status, s, "paged_attn");
}

nx_status nx_paged_gather(const nx_paged* cache, int32_t max_tokens, void* out_k, void* out_v,
                          int64_t out_seq_stride, int64_t out_head_stride) {
  nx_status st = check_cache(cache);
  if (st != NX_OK) return st;
  if (max_tokens < 0 || max_tokens > kMaxCacheRows || out_k == nullptr || out_v == nullptr) return NX_EINVAL;
  const int64_t d = cache->head_dim, esz = elem_size(cache->dtype), hk = cache->n_kv_heads;
  const int64_t rows = int64_t(max_tokens) * d;
  if (hk == 1) out_head_stride = rows;   // (strides of one head or sequence may be anything)
  if (cache->n_seqs == 1) out_seq_stride = (hk - 1) * out_head_stride + rows;
  if (out_head_stride < rows || out_seq_stride < (hk - 1) * out_head_stride + rows) return NX_EINVAL;
  if (!aligned(out_k) || !aligned(out_v) || out_seq_stride * esz % 16 || out_head_stride * esz % 16)
    return NX_EUNSUPPORTED;
  const int64_t n = rows > 0 ? ((cache->n_seqs - 1) * out_seq_stride + (hk - 1) * out_head_stride + rows) * esz : 0;
  const Range ok = bytes_at(out_k, n), ov = bytes_at(out_v, n);
  const CacheRanges cr = cache_ranges(cache);
  if (overlap(ok, ov)) return NX_EALIAS;
  for (const Range& x : cr.r)
    if (overlap(ok, x) || overlap(ov, x)) return NX_EALIAS;
  const int64_t units = int64_t(cache->n_seqs) * hk;
  const Range status = bytes_at(cache->workspace, 256);
  for (const Range& x : {bytes_at(cache->table, units * cache->max_pages * 4), bytes_at(cache->lens, units * 4)})
    if (overlap(ok, x) || overlap(ov, x) || overlap(status, x)) return NX_EALIAS;
  for (const Range& x : cr.r)
    if (overlap(status, x)) return NX_EALIAS;
  if (overlap(ok, status) || overlap(ov, status)) return NX_EALIAS;
  if (max_tokens == 0) return NX_OK;
  PagedArgs a = base_args(cache);
  a.max_tokens = max_tokens;
  a.out_k = out_k;
  a.out_v = out_v;
  a.out_seq_stride = out_seq_stride;
  a.out_head_stride = out_head_stride;
  hipStream_t s = static_cast<hipStream_t>(cache->stream);
  if (launch_paged_gather(a, s) != hipSuccess) return NX_EHIP;
  return debug_status(a.status, s, "paged_gather");
}

}  // extern "C"
