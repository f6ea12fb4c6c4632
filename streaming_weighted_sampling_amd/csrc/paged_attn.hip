// Attention over the paged 8-bit cache.
//
//   o_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = exp(scale q_r . k_t - m_r)
//
// One pass over the cached rows with a running reference m_r and sum per query
// row.  The call's blocks, all (sequence, KV head)s together, are cut into
// pieces of about equal size, one per workgroup, whatever the heads' lengths:
// a head of n blocks gives ceil(n / share) pieces, share = all blocks over the
// number of workgroups wanted.  The wavefronts split a piece and merge through
// LDS.  A head in one piece is written at once, otherwise its pieces leave
// partials (base, sum, o) that a second small kernel merges in head order.
// (Merging by the last workgroup to arrive at a counter instead cost 4 us in
// the counter's atomics alone at 54 pieces a head, all arriving at once; cuts
// that run on from one head into the next cost a workgroup a second start.)
//
// Bounds.  One query: the codes' read (16 heads of 131077 rows in groups of 8, 537 MB:
// 88 us, 6.1 TB/s of the 6.2 that this access pattern reaches; 128 heads of 4096 to
// 16384 rows, 339 MB: 64 us, 5.3 TB/s).  8 heads of 819 rows: 9 us, latency: launch,
// table, codes, products and the wavefronts' merge one after another.  64 queries
// of 8 heads in groups of 8 over 32768 rows: 88 us, 780 TFLOP/s; a SIMD's two wavefronts
// (registers) alternate matrix and exponential work without overlapping
// them fully (MFMA 30 % busy, VALU 50 %).
//
// Matrix form, per block of 32 rows: S^T = K Q^T and O^T += V^T P^T with
// 16x16x32 f16 MFMAs.  8-bit codes are exact in f16, so the codes are the
// operands and the block scales stay outside: K's scale multiplies the logits
// in fp32, V's scale multiplies p.  Both contractions are permuted so that no
// value crosses lanes: row 4 g + i of K tile u stands for token 8 g + 4 u + i,
// which leaves lane (g, c) of S^T with the logits of tokens 8 g .. 8 g + 7 of
// query row c -- just the k-slice its P^T operand needs -- and V is stored
// with 8 tokens of one element side by side.
//
// Roundings.  q enters as f16 after a power-of-two scaling of its row (largest
// magnitude in [2^13, 2^14)): bf16 elements are exact down to 2^-20 of the
// row's largest and off by at most 2^-38 of it below, fp32 rows use a second f16
// term for the remainder (22 bits).
// p enters as f16 (relative 2^-11, against the bf16 result's 2^-8), or as two
// f16 terms for fp32 rows, with its block's V scale over the wavefront's reference
// scale in it.  f16's smallest step bounds how far below the largest p a product
// with a large |v| may still count, so where a wavefront's V scales lie far apart
// (kNear) what f16 leaves of a small p enters too, scaled up, in further products.
// Sums, references and accumulators are fp32.
#include "paged.hpp"

namespace nx {
namespace {

constexpr float kNoBase = 1e30f;     // base of a row that has seen nothing
constexpr float kNoScale = -200.f;   // log2 of V's reference before the first block
// p is held times 2^7 at its row's reference and may grow by 2^7 (times V's
// scale ratio, at most 2) before the reference moves: f16 values stay below 2^16.
constexpr float kHead = 7.f;
// A wavefront keeps p in f16 while the scales of the V blocks that it has met lie
// within 2^kNear of the first one's, so within w = 2 kNear of each other: half of
// f16's smallest step is 2^-25, the sum of p at least 2^7, so o is exact to
// n 2^(w - 32) of the weighted mean of each block's largest |v| (n cached rows).
// (Normally distributed values: within 2^1.)
template <bool kF32> constexpr float kNear = kF32 ? 4.f : 7.f;
// Where they do not, what f16 left of the p below kBelow (at most 2^-25) is scaled
// by kStep, o with it, and enters as f16 again, kRounds times: up by 2^72 in all and
// exact to 2^-97 then, where the largest p of a block of the least ratio is 2^-73.
// (From kBelow on p is exact to 2^-11, its two terms to 2^-22.)  o stays below 2^48
// (2^15 times a code times 2^24 rows), scaled up below 2^120.
// Rare, so made small and not fast (scales alternating by 2^20: 16 heads of 131077
// rows 93 -> 141 us, 64 queries of 8 heads in groups of 8 over 32768 rows 94 -> 255).
template <bool kF32> struct Rest {
  static constexpr int kRounds = kF32 ? 4 : 3;
  static constexpr float kBelow = kF32 ? 0x1p-3f : 0x1p-14f, kStep = kF32 ? 0x1p18f : 0x1p24f;
};
// V's scale ratio counts as at least 2^kLeast, which is 2^-80 of the head's
// largest |v|.  A block of scale 0 has its p held 2^40 lower, at most 2^-26: less
// than half of f16's smallest step, so whatever its codes are they add nothing.
constexpr float kLeast = -80.f, kLeastZero = -40.f;

template <int kFmt>
__device__ inline h8_t codes_f16(uint32_t lo, uint32_t hi) {
  union { h2_t h[4]; h8_t v; } r;
  if constexpr (kFmt == NX_CACHE_E4M3) {
    r.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(lo), 1.0f, false);
    r.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(lo), 1.0f, true);
    r.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(hi), 1.0f, false);
    r.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(hi), 1.0f, true);
  } else {
    // c + 128 as the low mantissa byte of 1024 (f16 0x6400), then minus 1152: exact.
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    const h2_t off = {_Float16(1152.f), _Float16(1152.f)};
    r.h[0] = __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)) - off;
    r.h[1] = __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)) - off;
    r.h[2] = __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)) - off;
    r.h[3] = __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)) - off;
  }
  return r.v;
}

// One (sequence, KV head) as the kernel sees it.
struct Job {
  int n_q, rows;       // queries of the sequence, query rows (queries * group)
  int64_t q0;          // first row in q / out
  int len, n_blk;      // cached rows; its weight in the line of blocks: blocks
                       // (the tail counts as one), at least 1; 0 without queries
  bool ok;
};
__device__ inline Job make_job(const PagedArgs& a, int unit) {
  Job j;
  j.n_q = seq_rows(a, unit / a.c.n_kv_heads, a.max_q, &j.q0);
  j.len = a.c.lens[unit];
  j.ok = j.n_q >= 0 && j.len >= 0 &&
         int64_t(j.len) <= (int64_t(a.c.max_pages) << a.page_shift) * kBlock;
  j.rows = j.ok ? j.n_q * a.group : 0;
  if (!j.ok) j.len = 0;
  j.n_blk = j.rows > 0 ? max(1, (j.len + kBlock - 1) / kBlock) : 0;
  return j;
}

// Sum over the lanes below and including this one (row shifts within 16 lanes,
// then row broadcasts: VALU only).
__device__ inline int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);   // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);   // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);   // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // row_bcast:15 to rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // row_bcast:31 to rows 2 and 3
  return x;
}

// One workgroup's piece: blocks [b0, b1) of a head.
struct Piece {
  int unit, b0, b1;    // unit < 0: no piece
  int nth, of;         // which of the head's pieces
  int slot;            // partial of the head's first piece (heads in several pieces only)
};

// Every wavefront works the cut out for itself (no barrier; the same in all
// workgroups).  The share is the smallest that cuts the heads into at most
// n_wg pieces: one more would be a second round on some CU, and a second
// round of a piece costs as much as the first (16 heads of about 4096 blocks
// on 256 CUs: 137 us with 265 pieces, 93 with 256).
constexpr int kHeadRegs = 4;   // heads whose weights stay in registers, times 64
__device__ inline Piece find_piece(const PagedArgs& a, int wg, int units, int lane) {
  auto weight = [&](int unit) {
    if (unit >= units) return 0;
    const Job j = make_job(a, unit);
    if (!j.ok && wg == 0) paged_status(a.status, kStatusBadItem);
    return j.n_blk;
  };
  int w[kHeadRegs];
  int64_t total = 0;
#pragma unroll
  for (int x = 0; x < kHeadRegs; ++x) {
    w[x] = 0;
    if (64 * x < units) {
      w[x] = weight(64 * x + lane);
      total += __builtin_amdgcn_readlane(wave_scan(w[x]), 63);
    }
  }
  for (int u0 = 64 * kHeadRegs; u0 < units; u0 += 64)
    total += __builtin_amdgcn_readlane(wave_scan(weight(u0 + lane)), 63);
  Piece p{-1, 0, 0, 0, 0, 0};
  if (total > INT32_MAX) {   // more blocks than a pool can hold many times over
    if (wg == 0) paged_status(a.status, kStatusBadItem);
    return p;
  }
  int share = max(a.min_share, int((uint32_t(total) + uint32_t(a.n_wg) - 1) / uint32_t(a.n_wg)));
  if (units <= 64 * kHeadRegs && 2 * units <= a.n_wg) {
    // Between total / n_wg and total / (n_wg - units), to within 1/32.
    int lo = share, hi = max(share, int((uint32_t(total) + uint32_t(a.n_wg - units) - 1) / uint32_t(a.n_wg - units)));
    while (true) {
      int n = 0;
#pragma unroll
      for (int x = 0; x < kHeadRegs; ++x)
        if (64 * x < units) n += __builtin_amdgcn_readlane(wave_scan((w[x] + share - 1) / share), 63);
      if (n <= a.n_wg) hi = share;
      else lo = share + 1;
      if (lo >= hi || (hi - lo) * 32 <= hi) break;
      share = (lo + hi) / 2;
    }
    share = hi;
  }
  for (int u0 = 0, at = 0, slot = 0; u0 < units; u0 += 64) {
    int mine = 0;
    if (u0 >= 64 * kHeadRegs) {
      mine = weight(u0 + lane);
    } else {
#pragma unroll
      for (int x = 0; x < kHeadRegs; ++x)
        if (u0 == 64 * x) mine = w[x];
    }
    const int n = (mine + share - 1) / share, parts = n > 1 ? n : 0;
    const int n_incl = wave_scan(n), parts_incl = wave_scan(parts);
    const uint64_t hit = __ballot(at + n_incl - n <= wg && wg < at + n_incl);
    if (hit != 0) {
      const int i = __builtin_ctzll(hit);
      const int blocks = __builtin_amdgcn_readlane(mine, i);
      p.unit = u0 + i;
      p.of = __builtin_amdgcn_readlane(n, i);
      p.nth = wg - (at + __builtin_amdgcn_readlane(n_incl - n, i));
      p.slot = slot + __builtin_amdgcn_readlane(parts_incl - parts, i);
      p.b0 = int(int64_t(blocks) * p.nth / p.of);
      p.b1 = int(int64_t(blocks) * (p.nth + 1) / p.of);
      return p;
    }
    at += __builtin_amdgcn_readlane(n_incl, 63);
    slot += __builtin_amdgcn_readlane(parts_incl, 63);
  }
  return p;
}

// Accumulators of a wavefront: query row c of tile rt in lanes (., c).
template <int D, int RT>
struct State {
  f32x4_t o[RT][D / 16];   // in units of vref
  float base[RT];          // p = 2^(logit + base), logits in log2 units
  float l[RT];             // sum of p over this lane's tokens
  float vref, lvref;       // V's reference scale (wave-uniform) and its log2
};

__device__ inline float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
__device__ inline float lane_of(float x, int i) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
}

// The exponents z of one block's p from its products s (-infinity: hidden),
// with the block's V scale vs over the reference in them; moves references.
// t[rt] > 0: factor to log2 units; lvs: log2(vs).  Returns the power that the sum
// of p takes out again (log2 of the ratio is good to 2^-18, the sum sees the same
// value).
template <int D, int RT>
__device__ inline float exponents(State<D, RT>& st, const f32x4_t (&s)[RT][2], const float (&t)[RT], float vs,
                                  float lvs, float (&z)[RT][8]) {
  float shift = fmaxf(lvs - st.lvref, vs > 0.f ? kLeast : kLeastZero);
  float top = -__builtin_inff();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float b = st.base[rt] + shift;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      z[rt][e] = __builtin_fmaf(s[rt][e / 4][e % 4], t[rt], b);
      top = fmaxf(top, z[rt][e]);
    }
  }
  if (__any(top > 2.f * kHead + shift) || shift > 1.f) {   // (p itself, without the ratio)
    // Rare: a row's reference moves to its largest logit so far, or V's
    // reference scale to this block's; what is accumulated follows.
    float f = 1.f;
    if (shift > 1.f) {
      f = uniform(st.vref / vs);
      st.vref = vs;
      st.lvref = lvs;
      shift = 0.f;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = kHead - st.base[rt];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, s[rt][e / 4][e % 4] * t[rt]);
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float base = kHead - mx;
      const float alpha = __builtin_amdgcn_exp2f(base - st.base[rt]);
      st.base[rt] = base;
      st.l[rt] *= alpha;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) st.o[rt][n] *= alpha * f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        z[rt][e] = __builtin_fmaf(s[rt][e / 4][e % 4], t[rt], base + shift);
    }
  }
  return __builtin_amdgcn_exp2f(-shift);
}

// z becomes p, the sums take it up.
template <int D, int RT>
__device__ inline void exponentiate(State<D, RT>& st, float back, float (&z)[RT][8]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[rt][e] = __builtin_amdgcn_exp2f(z[rt][e]);
    const float sum = ((z[rt][0] + z[rt][1]) + (z[rt][2] + z[rt][3])) +
                      ((z[rt][4] + z[rt][5]) + (z[rt][6] + z[rt][7]));
    st.l[rt] = __builtin_fmaf(sum, back, st.l[rt]);
  }
}

// Bytes from the array's start to query row r of a sequence's KV head h (row r is query
// r / group, head r % group of the group).
template <bool kF32>
__device__ inline int64_t row_offset(const PagedArgs& a, const nx_rows& rows, const Job& job, int h, int r) {
  const int i = r / a.group, gh = r - i * a.group;
  return ((job.q0 + i) * rows.row_stride + (int64_t(h) * a.group + gh) * rows.head_stride) *
         Elem<kF32>::kBytes;
}

__device__ inline void write_lse(const PagedArgs& a, const Job& job, int h, int r, float l, float base) {
  const int i = r / a.group, gh = r - i * a.group;
  a.lse[(job.q0 + i) * a.c.n_q_heads + h * a.group + gh] =
      l == 0.f ? -__builtin_inff() : 0.69314718056f * (log2f(l) - base);
}

// 16 RT query rows a workgroup.  kWhole: workgroup (u, row tile) takes head u
// whole, for calls of short heads, which then need neither the search for the
// piece nor the merge launch.
template <int D, bool kF32, int kFmt, int RT, bool kNT, bool kWhole, int kWaves>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_kernel(PagedArgs a) {
  using E = Elem<kF32>;
  constexpr int kC = D / 32;          // 32-element chunks of a row
  constexpr int NP = kF32 ? 2 : 1;    // f16 terms of q and p
  constexpr int kRows = RT * 16;
  constexpr int kKL = D / 64 * 2, kVL = D / 32;   // 16-byte loads of a block
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = a.c.n_seqs * a.c.n_kv_heads;
  const int slot_mask = (1 << a.page_shift) - 1;
  __shared__ float sb[kWaves][kRows], sl[kWaves][kRows];
  __shared__ f32x4_t so[kWaves][RT * (D / 16)][64];

  // The row tiles of one piece sit on one XCD (ids eight apart) and near in
  // time, so that they share its L2.
  const int per8 = 8 * a.n_rt;
  const int wg = !kWhole ? int(blockIdx.x) / per8 * 8 + int(blockIdx.x) % 8 : 0;
  const int rt0 = !kWhole ? int(blockIdx.x) % per8 / 8 : int(blockIdx.x) % a.n_rt;
  const int row0 = rt0 * kRows;
  Piece piece;
  if constexpr (kWhole) piece = Piece{int(blockIdx.x) / a.n_rt, 0, 0, 0, 1, 0};
  else piece = find_piece(a, wg, units, threadIdx.x & 63);
  if (piece.unit < 0) return;
  const int unit = piece.unit;
  const Job job = make_job(a, unit);
  if constexpr (kWhole) {
    if (!job.ok && rt0 == 0 && threadIdx.x == 0) paged_status(a.status, kStatusBadItem);
    piece.b1 = job.n_blk;
  }
  if (row0 >= job.rows) return;
  const int h = unit % a.c.n_kv_heads, b0 = piece.b0, b1 = piece.b1;
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;

  State<D, RT> st;
  st.vref = 0.f;
  st.lvref = kNoScale;
  // Row r sees tokens up to seen[rt]; blocks past all_see need the test.
  int seen[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    st.base[rt] = kNoBase;
    st.l[rt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) st.o[rt][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    seen[rt] = job.len - job.n_q + (row0 + rt * 16 + c16) / a.group;
  }
  const int all_see = job.len - job.n_q;
  const int full = job.len / kBlock;
  const int per = (b1 - b0 + kWaves - 1) / kWaves;
  const int w0 = b0 + wave * per, w1 = min(w0 + per, b1), wf = min(w1, full);
  // Lane j looks up block x0 + j of up to 64 blocks.
  int slot_l, n8;
  float ks_l, vs_l;
  auto look_up = [&](int x0) {
    n8 = min(wf - x0, 64);
    slot_l = 0;
    ks_l = vs_l = 0.f;
    if (lane < n8) {
      const int b = x0 + lane;
      int page = a.c.table[int64_t(unit) * a.c.max_pages + (b >> a.page_shift)];
      if (page < 0 || page >= a.c.n_pages) {
        paged_status(a.status, kStatusBadItem);
        page = 0;
      }
      slot_l = (page << a.page_shift) + (b & slot_mask);
      ks_l = a.c.k_scale[slot_l];
      vs_l = a.c.v_scale[slot_l];
    }
  };
  // A block's K is fetched while the block before is settled, its V while
  // its own logits form: each register is refilled as soon as it is used.
  uint4 kr[kKL], vr[kVL];
  auto codes = [&](const void* base, int i) {
    const int64_t at = int64_t(__builtin_amdgcn_readlane(slot_l, i)) * (kBlock * D);
    return Buf(static_cast<const char*>(base) + at, kBlock * D);
  };
  auto load_k = [&](int i) {
    const Buf kb = codes(a.c.k_codes, i);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        kr[u * (D / 64) + x] =
            kb.ld16<kNT ? kNonTemporal : 0>(((c16 / 4) * 8 + c16 % 4) * D + 16 * g + u * 4 * D + 64 * x);
  };
  auto load_v = [&](int i) {
    const Buf vb = codes(a.c.v_codes, i);
#pragma unroll
    for (int n = 0; n < kVL; ++n) vr[n] = vb.ld16<kNT ? kNonTemporal : 0>((g * D + 2 * c16) * 8 + 256 * n);
  };
  // V's first scale (log2), and whether another lies further from it than kNear.
  float lv_first = kNoScale;
  bool far_apart = false;
  // fp32 rows in two tiles leave no registers for p until its rest is known to be
  // needed: it waits in this wavefront's part of so.
  constexpr bool kParked = kF32 && RT == 2;
  auto park = [&](const float (&x)[RT][8]) {
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i)
      so[wave][i][lane] = f32x4_t{x[i / 2][i % 2 * 4], x[i / 2][i % 2 * 4 + 1], x[i / 2][i % 2 * 4 + 2], x[i / 2][i % 2 * 4 + 3]};
  };
  auto fetch = [&](float (&x)[RT][8]) {
#pragma unroll
    for (int i = 0; i < 8 * RT; ++i) x[i / 8][i % 8] = so[wave][i / 4][lane][i % 4];
  };
  auto to_f16 = [](const float (&x)[RT][8], h8_t (&y)[RT][NP]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const _Float16 hi = _Float16(x[rt][e]);
        y[rt][0][e] = hi;
        if constexpr (kF32) y[rt][NP - 1][e] = _Float16(x[rt][e] - float(hi));
      }
  };
  // The first block is on its way while q is prepared.
  if (w0 < wf) {
    look_up(w0);
    load_k(0);
    load_v(0);
  }

  // ---- q: f16 operand terms and the factor of the logits per row ----
  h8_t q[RT][kC][NP];
  float qmul[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = row0 + rt * 16 + c16;
    const char* src = static_cast<const char*>(a.q.p) + row_offset<kF32>(a, a.q, job, h, min(r, job.rows - 1));
    float x[kC][8];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      E::load8(src + (64 * (c / 2) + 16 * g + 8 * (c % 2)) * E::kBytes, x[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (r >= job.rows) x[c][e] = 0.f;
        top = fmaxf(top, fabsf(x[c][e]));
      }
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int ex = top > 0.f ? int(__builtin_bit_cast(uint32_t, top) >> 23) - 127 : 0;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = ldexpf(x[c][e], 13 - ex);
        const _Float16 hi = _Float16(s);
        q[rt][c][0][e] = hi;
        if constexpr (kF32) q[rt][c][NP - 1][e] = _Float16(s - float(hi));
      }
    qmul[rt] = ldexpf(a.scale_log2, ex - 13);
  }

  for (int x0 = w0; x0 < wf; x0 += 64) {
    if (x0 > w0) {
      look_up(x0);
      load_k(0);
      load_v(0);
    }
    const float lvs_l = vs_l > 0.f ? log2f(vs_l) : kNoScale * 4.f;
    // Lanes without a block have scale 0.
    const uint64_t live = __ballot(vs_l > 0.f);
    if (lv_first == kNoScale && live != 0) lv_first = lane_of(lvs_l, __builtin_ctzll(live));
    if (__any(vs_l > 0.f && fabsf(lvs_l - lv_first) > kNear<kF32>)) far_apart = true;
    f32x4_t s[RT][2];
    auto products = [&] {   // s = K q^T of the block in kr
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint4 w = kr[u * (D / 64) + c / 2];
          const h8_t k8 = c % 2 ? codes_f16<kFmt>(w.z, w.w) : codes_f16<kFmt>(w.x, w.y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int np = 0; np < NP; ++np)
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, q[rt][c][np], s[rt][u], 0, 0, 0);
        }
    };
    for (int i = 0; i < n8; ++i) {
      products();
      if (i + 1 < n8) load_k(i + 1);
      const float ks = lane_of(ks_l, i), vs = lane_of(vs_l, i), lvs = lane_of(lvs_l, i);
      float t[RT], z[RT][8];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) t[rt] = fmaxf(ks * qmul[rt], 0x1p-126f);   // > 0: hidden stays -infinity
      const int t0 = (x0 + i) * kBlock;
      if (t0 + kBlock - 1 > all_see) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (t0 + 8 * g + e > seen[rt]) s[rt][e / 4][e % 4] = -__builtin_inff();
      }
      const float back = exponents<D, RT>(st, s, t, vs, lvs, z);
      exponentiate<D, RT>(st, back, z);
      if constexpr (kParked) park(z);
      h8_t pp[RT][NP];
      to_f16(z, pp);
#pragma unroll
      for (int n = 0; n < kVL; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const h8_t v8 = u ? codes_f16<kFmt>(vr[n].z, vr[n].w) : codes_f16<kFmt>(vr[n].x, vr[n].y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int np = 0; np < NP; ++np)
              st.o[rt][2 * n + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, pp[rt][np],
                                                                         st.o[rt][2 * n + u], 0, 0, 0);
        }
      if (__builtin_expect(far_apart && vs > 0.f, 0)) {
#pragma unroll 1
        for (int round = 0; round < Rest<kF32>::kRounds; ++round) {
          if constexpr (kParked) fetch(z);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[rt][e] = fabsf(z[rt][e]) < Rest<kF32>::kBelow ? z[rt][e] : 0.f;
          h8_t pr[RT][NP];
          to_f16(z, pr);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              z[rt][e] -= float(pr[rt][0][e]);
              if constexpr (kF32) z[rt][e] -= float(pr[rt][NP - 1][e]);
              z[rt][e] *= Rest<kF32>::kStep;
            }
          if constexpr (kParked) park(z);
          to_f16(z, pr);
#pragma unroll
          for (int n = 0; n < kVL; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              // Converted anew, a few at a time: there are no registers to keep them in.
              __builtin_amdgcn_sched_barrier(0);
              uint32_t lo = u ? vr[n].z : vr[n].x, hi = u ? vr[n].w : vr[n].y;
              asm volatile("" : "+v"(lo), "+v"(hi));
              const h8_t v8 = codes_f16<kFmt>(lo, hi);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                st.o[rt][2 * n + u] *= Rest<kF32>::kStep;
#pragma unroll
                for (int np = 0; np < NP; ++np)
                  st.o[rt][2 * n + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, pr[rt][np],
                                                                             st.o[rt][2 * n + u], 0, 0, 0);
              }
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int n = 0; n < D / 16; ++n) st.o[rt][n] *= 0x1p-72f;
      }
      if (i + 1 < n8) load_v(i + 1);
    }
  }
  if (w0 <= full && full < w1 && full * kBlock < job.len) {
    // The tail: up to 31 rows in the call's own type.  bf16 rows use bf16
    // MFMAs (q as it is, p in two terms), fp32 rows fp32 MFMAs.
    const int nt = job.len - full * kBlock;
    const int64_t tail_at = int64_t(unit) * kBlock * D * E::kBytes;
    const Buf kt(static_cast<const char*>(a.c.k_tail) + tail_at, kBlock * D * E::kBytes);
    const Buf vt(static_cast<const char*>(a.c.v_tail) + tail_at, kBlock * D * E::kBytes);
    const int k_at = ((c16 / 4) * 8 + c16 % 4) * D * E::kBytes;
    const int v_at = (g * D + 2 * c16) * 8 * E::kBytes;
    f32x4_t s[RT][2];
    float t[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      s[rt][0] = s[rt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      t[rt] = fmaxf(a.scale_log2, 0x1p-126f);
      const int r = row0 + rt * 16 + c16;   // rows past the last repeat it; they are not written
      const char* src = static_cast<const char*>(a.q.p) + row_offset<kF32>(a, a.q, job, h, min(r, job.rows - 1));
      if constexpr (!kF32) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const int d = 64 * (c / 2) + 16 * g + 8 * (c % 2);
          const uint4 qw = *reinterpret_cast<const uint4*>(src + d * 2);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 kw = kt.ld16(k_at + u * 4 * D * 2 + d * 2);
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, kw), __builtin_bit_cast(bf16x8_t, qw), s[rt][u], 0, 0, 0);
          }
        }
      } else {
        for (int c = 0; c < D / 16; ++c) {
          const int d = 16 * c + 4 * g;
          const float4 qw = *reinterpret_cast<const float4*>(src + d * 4);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float4 kw = __builtin_bit_cast(float4, kt.ld16(k_at + u * 4 * D * 4 + d * 4));
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.x, qw.x, s[rt][u], 0, 0, 0);
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.y, qw.y, s[rt][u], 0, 0, 0);
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.z, qw.z, s[rt][u], 0, 0, 0);
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.w, qw.w, s[rt][u], 0, 0, 0);
          }
        }
      }
      // Rows past the tail's count may hold anything.
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * g + e >= nt || full * kBlock + 8 * g + e > seen[rt]) s[rt][e / 4][e % 4] = -__builtin_inff();
    }
    float p[RT][8];
    exponentiate<D, RT>(st, exponents<D, RT>(st, s, t, 1.f, 0.f, p), p);
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // Zeros where no row is: whatever lies there must not meet p = 0.
        float v[8];
        const int at = v_at + (32 * n + u) * 8 * E::kBytes;
        E::unpack8(vt.ld16(at), kF32 ? vt.ld16(at + 16) : uint4{}, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 8 * g + e < nt ? v[e] : 0.f;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if constexpr (!kF32) {
            bf16x8_t v8, hi, lo;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = p[rt][e];
              v8[e] = __bf16(v[e]);
              hi[e] = __bf16(x);
              lo[e] = __bf16(x - float(hi[e]));
            }
            st.o[rt][2 * n + u] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, hi, st.o[rt][2 * n + u], 0, 0, 0);
            st.o[rt][2 * n + u] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, lo, st.o[rt][2 * n + u], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st.o[rt][2 * n + u] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  v[e], p[rt][e], st.o[rt][2 * n + u], 0, 0, 0);
          }
        }
      }
  }

  // ---- merge the wavefronts ----
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    st.l[rt] += __shfl_xor(st.l[rt], 16, 64);
    st.l[rt] += __shfl_xor(st.l[rt], 32, 64);
    if (g == 0) {
      sb[wave][rt * 16 + c16] = st.base[rt];
      sl[wave][rt * 16 + c16] = st.l[rt];
    }
  }
  __syncthreads();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + c16;
    float bmin = sb[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) bmin = fminf(bmin, sb[w][r]);
    const float f = exp2f(bmin - st.base[rt]) * st.vref;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) st.o[rt][n] *= f;
  }
  // Each wavefront leaves its o in LDS and sums its part of the columns.
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < D / 16; ++n) so[wave][rt * (D / 16) + n][lane] = st.o[rt][n];
  __syncthreads();

  // ---- the result, or a partial ----
  constexpr int kParts = RT * (D / 32);      // (row tile, 32 columns) pairs
#pragma unroll
  for (int k = 0; k < (kParts + kWaves - 1) / kWaves; ++k) {
    const int part = k * kWaves + wave;
    if (kParts % kWaves != 0 && part >= kParts) break;
    const int rt = part / (D / 32), n = part % (D / 32);
    float x[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t o = so[0][2 * part + u][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) o += so[w][2 * part + u][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * e + u] = o[e];
    }
    const int r = row0 + rt * 16 + c16;
    if (r >= job.rows) continue;
    const int rr = rt * 16 + c16;
    float bmin = sb[0][rr];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) bmin = fminf(bmin, sb[w][rr]);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) l += sl[w][rr] * exp2f(bmin - sb[w][rr]);
    if (piece.of == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
      E::store8(static_cast<char*>(a.out.p) + row_offset<kF32>(a, a.out, job, h, r) +
                    (32 * n + 8 * g) * E::kBytes, x);
      if (a.lse != nullptr && g == 0 && n == 0) write_lse(a, job, h, r, l, bmin);
    } else {
      const int64_t pr = (int64_t(piece.slot + piece.nth) * a.n_rt + rt0) * kRows + rr;
      Elem<true>::store8(a.part_o + pr * D + 32 * n + 8 * g, x);
      if (g == 0 && n == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * pr) = make_float2(bmin, l);
    }
  }
  // The head's first piece says where its pieces are, in the first row
  // tile's name (the cut is the same for all).
  if (!kWhole && piece.nth == 0 && rt0 == 0 && threadIdx.x == 0)
    a.pieces[unit] = make_int2(piece.of > 1 ? piece.of : 0, piece.slot);
}

// Merges the pieces of one query row of one head, in order: D / 4 lanes a
// piece, the workgroup's 256 / (D / 4) lane groups take every so manyth piece.
// 4 to 5 us, launch and one read latency (512 rows a head in 8 heads: 6).
template <int D, bool kF32>
__global__ __launch_bounds__(256) void attn_merge_kernel(PagedArgs a, int tile) {
  using E = Elem<kF32>;
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  const int unit = blockIdx.y, r = blockIdx.x, tid = threadIdx.x;
  const int2 pieces = a.pieces[unit];   // (count, slot of the first); not written without queries
  const Job job = make_job(a, unit);
  if (r >= job.rows || pieces.x == 0) return;
  // (Not a cut of this call: it had too many blocks and wrote none.)
  if (pieces.x < 0 || pieces.y < 0 || int64_t(pieces.x) + pieces.y > 2 * int64_t(a.n_wg)) return;
  const int grp = tid / kLanes, col = 4 * (tid % kLanes);
  const int rt = r / tile;
  auto row_of = [&](int i) { return (int64_t(pieces.y + i) * a.n_rt + rt) * tile + (r - rt * tile); };
  float base = kNoBase, l = 0.f;
  f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 4;
  for (int i0 = grp; i0 < pieces.x; i0 += kGroups * kAhead) {
    float2 ml[kAhead];
    f32x4_t x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t pr = row_of(min(i0 + i * kGroups, pieces.x - 1));
      ml[i] = *reinterpret_cast<const float2*>(a.part_ml + 2 * pr);
      x[i] = *reinterpret_cast<const f32x4_t*>(a.part_o + pr * D + col);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i * kGroups >= pieces.x) break;
      const float b = fminf(base, ml[i].x);
      const float f = exp2f(b - base), fi = exp2f(b - ml[i].x);
      base = b;
      l = l * f + ml[i].y * fi;
      o = o * f + x[i] * fi;
    }
  }
  __shared__ float sb[kGroups], sl[kGroups];
  __shared__ f32x4_t so[kGroups][kLanes];
  if (tid % kLanes == 0) {
    sb[grp] = base;
    sl[grp] = l;
  }
  so[grp][tid % kLanes] = o;
  __syncthreads();
  if (grp != 0) return;
  float bmin = sb[0];
#pragma unroll
  for (int k = 1; k < kGroups; ++k) bmin = fminf(bmin, sb[k]);
  l = 0.f;
  o = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float f = exp2f(bmin - sb[k]);
    l += sl[k] * f;
    o += so[k][tid % kLanes] * f;
  }
  const int h = unit % a.c.n_kv_heads;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* dst = static_cast<char*>(a.out.p) + row_offset<kF32>(a, a.out, job, h, r) + col * E::kBytes;
  E::store2(dst, o[0] * inv, o[1] * inv);
  E::store2(dst + 2 * E::kBytes, o[2] * inv, o[3] * inv);
  if (a.lse != nullptr && tid == 0) write_lse(a, job, h, r, l, bmin);
}

template <int D, bool kF32, int kFmt>
hipError_t launch(const PagedArgs& a, hipStream_t s) {
  const int units = a.c.n_seqs * a.c.n_kv_heads;
  const int tile = paged_tile_rows(int64_t(a.max_q) * a.group);
  if (a.whole) {
    const dim3 grid(uint32_t(units) * a.n_rt);
    if (tile == 16)
      hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 1, false, true, 8>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 2, false, true, 4>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  // At most n_wg pieces of a full share and one shorter one per head.
  const dim3 grid(uint32_t((a.n_wg + units + 7) / 8 * 8) * a.n_rt);
  if (tile == 16 && a.stream_nt)
    hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 1, true, false, 4>), grid, dim3(256), 0, s, a);
  else if (tile == 16)
    hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 1, false, false, 4>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 2, false, false, 4>), grid, dim3(256), 0, s, a);
  hipLaunchKernelGGL((attn_merge_kernel<D, kF32>), dim3(uint32_t(a.max_q) * a.group, units), dim3(256), 0, s, a,
                     tile);
  return hipGetLastError();
}

}  // namespace

int paged_tile_rows(int64_t rows) { return rows <= 16 ? 16 : 32; }

hipError_t launch_paged_attn(const PagedArgs& a, hipStream_t s) {
  const bool f32 = a.c.dtype == NX_F32, i8 = a.c.format == NX_CACHE_I8;
  if (a.c.head_dim == 128) {
    if (f32) return i8 ? launch<128, true, 1>(a, s) : launch<128, true, 0>(a, s);
    return i8 ? launch<128, false, 1>(a, s) : launch<128, false, 0>(a, s);
  }
  if (f32) return i8 ? launch<64, true, 1>(a, s) : launch<64, true, 0>(a, s);
  return i8 ? launch<64, false, 1>(a, s) : launch<64, false, 0>(a, s);
}

}  // namespace nx
