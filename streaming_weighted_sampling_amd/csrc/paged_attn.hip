// Attention over the paged 8-bit cache.
//
//   o_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = exp(scale q_r . k_t - m_r)
//
// One pass over the cached rows with a running reference m_r and sum per query
// row.  Work is split over (sequence, KV head) x query-row tile x chunk of
// blocks; four wavefronts of a workgroup take the blocks of a chunk, merge
// through LDS, and write either the result or a partial (m, sum, o) that
// attn_combine merges.
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
// row's largest and off by at most 2^-38 of it below, fp32 rows use a second f16 term for the remainder (22 bits).
// p enters as f16 (relative 2^-11, against the bf16 result's 2^-8), or as two
// f16 terms for fp32 rows.  Sums, references and accumulators are fp32.
#include "paged.hpp"

namespace nx {
namespace {

constexpr float kNoMax = -1e30f;   // reference of a row that has seen nothing
// p is held times 2^7 and may exceed its reference by 2^7, V's scale ratio is at
// most 2: f16 values stay below 2^15.
constexpr float kHead = 7.f;
// Smallest V scale ratio that multiplies p: p keeps 11 bits down to 2^-9 there.
constexpr float kApart = 0x1p-12f;

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

// What a workgroup works on.
struct Job {
  int unit, rt, split;
  int n_q, rows;       // queries of the sequence, query rows (queries * group)
  int64_t q0;          // first row in q / out
  int len, n_blk;      // cached rows; blocks, the tail counted as one
  bool ok;
};
__device__ inline Job make_job(const PagedArgs& a, int unit, int rt, int split) {
  Job j;
  j.unit = unit;
  j.rt = rt;
  j.split = split;
  const int s = unit / a.c.n_kv_heads;
  j.n_q = seq_rows(a, s, a.max_q, &j.q0);
  j.len = a.c.lens[unit];
  j.ok = j.n_q >= 0 && j.len >= 0 &&
         int64_t(j.len) <= (int64_t(a.c.max_pages) << a.page_shift) * kBlock;
  j.rows = j.ok ? j.n_q * a.group : 0;
  if (!j.ok) j.len = 0;
  j.n_blk = (j.len + kBlock - 1) / kBlock;
  return j;
}

template <int D, int RT>
struct State {
  f32x4_t o[RT][D / 16];
  float m[RT], l[RT];
  float vref;
};

// Folds the logits z[rt][0..7] (log2 units, already minus m - kHead) of one
// block into the state: p = 2^z, scaled by vs / vref for the V product.
// `y(rt, e)` recomputes a masked logit when a reference has to move.
template <int D, int RT, typename Y>
__device__ inline void settle(State<D, RT>& st, float (&z)[RT][8], float vs, float& ratio, Y&& y) {
  float top = z[0][0];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, z[rt][e]);
  if (__any(top > 2.f * kHead) || vs > 2.f * st.vref) {
    // Rare: a row's reference moves to its largest logit so far, or V's
    // reference scale to this block's; what is accumulated follows.
    float f = 1.f;
    if (vs > 2.f * st.vref) {
      f = st.vref / vs;
      st.vref = vs;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = st.m[rt];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, y(rt, e));
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float alpha = exp2f(st.m[rt] - mx);
      st.m[rt] = mx;
      st.l[rt] *= alpha;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) st.o[rt][n] *= alpha * f;
#pragma unroll
      for (int e = 0; e < 8; ++e) z[rt][e] = y(rt, e) - (mx - kHead);
    }
  }
  ratio = st.vref > 0x1p-120f ? vs / st.vref : 0.f;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      z[rt][e] = __builtin_amdgcn_exp2f(z[rt][e]);
      st.l[rt] += z[rt][e];
    }
}

template <int D, bool kF32, int kFmt, int RT>
__global__ __launch_bounds__(256) void attn_kernel(PagedArgs a) {
  using E = Elem<kF32>;
  constexpr int kC = D / 32;          // 32-element chunks of a row
  constexpr int NP = kF32 ? 2 : 1;    // f16 terms of q and p
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % a.n_splits, rt0 = blockIdx.x / a.n_splits;
  const Job job = make_job(a, blockIdx.y, rt0, split);
  if (!job.ok) {
    if (blockIdx.x == 0 && tid == 0) paged_status(a.status, kStatusBadItem);
    return;
  }
  const int row0 = rt0 * RT * 16;
  if (row0 >= job.rows) return;
  if (split > 0 && split * a.chunk >= job.n_blk) return;
  const int h = job.unit % a.c.n_kv_heads;

  // ---- q: f16 operand terms and the factor of the logits per row ----
  h8_t q[RT][kC][NP];
  float qmul[RT];
  auto q_row = [&](int rt) -> const char* {
    const int r = row0 + rt * 16 + c16;
    if (r >= job.rows) return nullptr;
    const int i = r / a.group, gh = r - i * a.group;
    return static_cast<const char*>(a.q.p) +
           ((job.q0 + i) * a.q.row_stride + (int64_t(h) * a.group + gh) * a.q.head_stride) * E::kBytes;
  };
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const char* p = q_row(rt);
    float x[kC][8];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (p != nullptr) {
        E::load8(p + (64 * (c / 2) + 16 * g + 8 * (c % 2)) * E::kBytes, x[c]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[c][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[c][e]));
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

  State<D, RT> st;
  st.vref = 0.f;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    st.m[rt] = kNoMax;
    st.l[rt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) st.o[rt][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  // Row r sees tokens up to seen[rt]; tokens from first_hidden on need the test.
  int seen[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    seen[rt] = job.len - job.n_q + (row0 + rt * 16 + c16) / a.group;
  const int all_see = job.len - job.n_q;

  const int full = job.len / kBlock;
  const int slot_mask = (1 << a.page_shift) - 1;
  const int64_t trow = int64_t(job.unit) * a.c.max_pages;
  for (int c0 = split * a.chunk; c0 < job.n_blk; c0 += a.n_splits * a.chunk) {
    const int c1 = min(c0 + a.chunk, job.n_blk);
    const int per = (c1 - c0 + 3) / 4;
    const int w0 = c0 + wave * per, w1 = min(w0 + per, c1);
    const int n8 = min(w1, full) - w0;   // whole blocks of this wavefront, at most 64
    // Lane j looks up block w0 + j.
    int slot_l = 0;
    float ks_l = 0.f, vs_l = 0.f;
    if (lane < n8) {
      const int b = w0 + lane;
      int page = a.c.table[trow + (b >> a.page_shift)];
      if (page < 0 || page >= a.c.n_pages) {
        paged_status(a.status, kStatusBadItem);
        page = 0;
      }
      slot_l = (page << a.page_shift) + (b & slot_mask);
      ks_l = a.c.k_scale[slot_l];
      vs_l = a.c.v_scale[slot_l];
    }
    constexpr int kKL = D / 64 * 2, kVL = D / 32;   // 16-byte loads of a block
    uint4 kr[kKL], vr[kVL];
    auto load = [&](int i) {
      const int64_t base = int64_t(__builtin_amdgcn_readlane(slot_l, i)) * kBlock * D;
      const Buf kb(static_cast<const char*>(a.c.k_codes) + base, kBlock * D);
      const Buf vb(static_cast<const char*>(a.c.v_codes) + base, kBlock * D);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          kr[u * (D / 64) + x] =
              kb.ld16(((c16 / 4) * 8 + u * 4 + c16 % 4) * D + 64 * x + 16 * g);
#pragma unroll
      for (int n = 0; n < kVL; ++n) vr[n] = vb.ld16((g * D + 32 * n + 2 * c16) * 8);
    };
    if (n8 > 0) load(0);
    for (int i = 0; i < n8; ++i) {
      uint4 kc[kKL], vc[kVL];
#pragma unroll
      for (int x = 0; x < kKL; ++x) kc[x] = kr[x];
#pragma unroll
      for (int x = 0; x < kVL; ++x) vc[x] = vr[x];
      if (i + 1 < n8) load(i + 1);
      const float ks = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ks_l), i));
      const float vs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vs_l), i));
      f32x4_t s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint4 w = kc[u * (D / 64) + c / 2];
          const h8_t k8 = c % 2 ? codes_f16<kFmt>(w.z, w.w) : codes_f16<kFmt>(w.x, w.y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int np = 0; np < NP; ++np)
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, q[rt][c][np], s[rt][u], 0, 0, 0);
        }
      const int t0 = (w0 + i) * kBlock;
      const bool hide = t0 + kBlock - 1 > all_see;
      float z[RT][8];
      auto logit = [&](int rt, int e) {
        const float y = s[rt][e / 4][e % 4] * (ks * qmul[rt]);
        return hide && t0 + 8 * g + e > seen[rt] ? -__builtin_inff() : y;
      };
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 8; ++e) z[rt][e] = logit(rt, e) - (st.m[rt] - kHead);
      float ratio;
      settle<D, RT>(st, z, vs, ratio, logit);
      // A block whose V scale is far below the reference would push p out of
      // f16's range: its product is formed apart and scaled in fp32.
      const bool apart = ratio < kApart;
      const float pscale = apart ? 1.f : ratio;
      h8_t pp[RT][NP];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = z[rt][e] * pscale;
          const _Float16 hi = _Float16(x);
          pp[rt][0][e] = hi;
          if constexpr (kF32) pp[rt][NP - 1][e] = _Float16(x - float(hi));
        }
#pragma unroll
      for (int n = 0; n < kVL; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const h8_t v8 = u ? codes_f16<kFmt>(vc[n].z, vc[n].w) : codes_f16<kFmt>(vc[n].x, vc[n].y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            f32x4_t& o = st.o[rt][2 * n + u];
            if (apart) {
              f32x4_t x = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int np = 0; np < NP; ++np)
                x = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, pp[rt][np], x, 0, 0, 0);
              o += x * ratio;
            } else {
#pragma unroll
              for (int np = 0; np < NP; ++np)
                o = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, pp[rt][np], o, 0, 0, 0);
            }
          }
        }
    }
    if (w0 <= full && full < w1) {
      // The tail: up to 31 rows in the call's own type.  bf16 rows use bf16
      // MFMAs (q as it is, p in two terms), fp32 rows fp32 MFMAs.
      const int nt = job.len - full * kBlock;
      const char* kt = static_cast<const char*>(a.c.k_tail) + int64_t(job.unit) * kBlock * D * E::kBytes;
      const char* vt = static_cast<const char*>(a.c.v_tail) + int64_t(job.unit) * kBlock * D * E::kBytes;
      f32x4_t s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      // (K rows past the tail's count give logits that are masked.)
      if constexpr (!kF32) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const char* p = q_row(rt);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int d = 64 * (c / 2) + 16 * g + 8 * (c % 2);
            uint4 qw = make_uint4(0, 0, 0, 0);
            if (p != nullptr) qw = *reinterpret_cast<const uint4*>(p + d * 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int t = (c16 / 4) * 8 + u * 4 + c16 % 4;
              const uint4 kw = *reinterpret_cast<const uint4*>(kt + (t * D + d) * 2);
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kw),
                                                               __builtin_bit_cast(bf16x8_t, qw), s[rt][u],
                                                               0, 0, 0);
            }
          }
        }
      } else {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const char* p = q_row(rt);
          for (int c = 0; c < D / 16; ++c) {
            const int d = 16 * c + 4 * g;
            float4 qw = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p != nullptr) qw = *reinterpret_cast<const float4*>(p + d * 4);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int t = (c16 / 4) * 8 + u * 4 + c16 % 4;
              const float4 kw = *reinterpret_cast<const float4*>(kt + (t * D + d) * 4);
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.x, qw.x, s[rt][u], 0, 0, 0);
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.y, qw.y, s[rt][u], 0, 0, 0);
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.z, qw.z, s[rt][u], 0, 0, 0);
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kw.w, qw.w, s[rt][u], 0, 0, 0);
            }
          }
        }
      }
      float z[RT][8];
      auto logit = [&](int rt, int e) {
        const int t = 8 * g + e;
        return t >= nt || full * kBlock + t > seen[rt] ? -__builtin_inff()
                                                      : s[rt][e / 4][e % 4] * a.scale_log2;
      };
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 8; ++e) z[rt][e] = logit(rt, e) - (st.m[rt] - kHead);
      float ratio;
      settle<D, RT>(st, z, 1.f, ratio, logit);
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // Rows past the count may hold anything: zeros go into the product.
          float v[8];
          E::load8(vt + (g * D + 32 * n + 2 * c16 + u) * 8 * E::kBytes, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 8 * g + e < nt ? v[e] : 0.f;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if constexpr (!kF32) {
              bf16x8_t v8, hi, lo;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x = z[rt][e] * ratio;
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
                    v[e], z[rt][e] * ratio, st.o[rt][2 * n + u], 0, 0, 0);
            }
          }
        }
    }
  }

  // ---- merge the four wavefronts ----
  constexpr int kRows = RT * 16;
  __shared__ float sm[4][kRows], sl[4][kRows];
  __shared__ f32x4_t so[2][RT * (D / 16)][64];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    st.l[rt] += __shfl_xor(st.l[rt], 16, 64);
    st.l[rt] += __shfl_xor(st.l[rt], 32, 64);
    if (g == 0) {
      sm[wave][rt * 16 + c16] = st.m[rt];
      sl[wave][rt * 16 + c16] = st.l[rt];
    }
  }
  __syncthreads();
  float mx[RT], lsum[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + c16;
    mx[rt] = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
    lsum[rt] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) lsum[rt] += sl[w][r] * exp2f(sm[w][r] - mx[rt]);
    const float f = exp2f(st.m[rt] - mx[rt]) * st.vref;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) st.o[rt][n] *= f;
  }
  auto put = [&](int at) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int n = 0; n < D / 16; ++n) so[at][rt * (D / 16) + n][lane] = st.o[rt][n];
  };
  auto add = [&](int at) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int n = 0; n < D / 16; ++n) st.o[rt][n] += so[at][rt * (D / 16) + n][lane];
  };
  if (wave >= 2) put(wave - 2);
  __syncthreads();
  if (wave < 2) add(wave);
  __syncthreads();
  if (wave == 1) put(0);
  __syncthreads();
  if (wave != 0) return;
  add(0);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = row0 + rt * 16 + c16;
    if (r >= job.rows) continue;
    if (a.n_splits == 1) {
      const int i = r / a.group, gh = r - i * a.group;
      const float inv = lsum[rt] == 0.f ? 0.f : 1.f / lsum[rt];
      char* dst = static_cast<char*>(a.out.p) +
                  ((job.q0 + i) * a.out.row_stride + (int64_t(h) * a.group + gh) * a.out.head_stride) *
                      E::kBytes;
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = st.o[rt][2 * n][e] * inv;
          x[2 * e + 1] = st.o[rt][2 * n + 1][e] * inv;
        }
        E::store8(dst + (32 * n + 8 * g) * E::kBytes, x);
      }
      if (a.lse != nullptr && g == 0)
        a.lse[(job.q0 + i) * a.c.n_q_heads + h * a.group + gh] =
            lsum[rt] == 0.f ? -__builtin_inff() : 0.69314718056f * (mx[rt] - kHead + log2f(lsum[rt]));
    } else {
      const int64_t pr =
          ((int64_t(job.unit) * a.n_rt + rt0) * a.n_splits + split) * kRows + rt * 16 + c16;
      float* dst = a.part_o + pr * D;
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = st.o[rt][2 * n][e];
          x[2 * e + 1] = st.o[rt][2 * n + 1][e];
        }
        Elem<true>::store8(dst + 32 * n + 8 * g, x);
      }
      if (g == 0) {
        a.part_ml[2 * pr] = mx[rt];
        a.part_ml[2 * pr + 1] = lsum[rt];
      }
    }
  }
}

// Merges the splits of one query row: a workgroup per (row, unit), each
// wavefront a quarter of the splits, D / 2 lanes two elements each.
template <int D, bool kF32>
__global__ __launch_bounds__(256) void attn_combine_kernel(PagedArgs a, int tile) {
  using E = Elem<kF32>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Job job = make_job(a, blockIdx.y, 0, 0);
  const int r = blockIdx.x;
  if (!job.ok || r >= job.rows) return;
  const int n = max(1, min(a.n_splits, (job.n_blk + a.chunk - 1) / a.chunk));
  const int rt0 = r / tile;
  const int64_t p0 = (int64_t(job.unit) * a.n_rt + rt0) * a.n_splits * tile + (r - rt0 * tile);
  float mx = kNoMax;
  for (int s = lane; s < n; s += 64) mx = fmaxf(mx, a.part_ml[2 * (p0 + int64_t(s) * tile)]);
  mx = fmaxf(half_max(mx), __shfl_xor(half_max(mx), 32, 64));
  float l = 0.f, x = 0.f, y = 0.f;
  for (int s = wave; s < n; s += 4) {
    const int64_t p = p0 + int64_t(s) * tile;
    const float f = exp2f(a.part_ml[2 * p] - mx);
    l += a.part_ml[2 * p + 1] * f;
    if (lane < D / 2) {
      const float2 o = *reinterpret_cast<const float2*>(a.part_o + p * D + 2 * lane);
      x += o.x * f;
      y += o.y * f;
    }
  }
  __shared__ float red[3][4][64];
  red[0][wave][lane] = l;
  red[1][wave][lane] = x;
  red[2][wave][lane] = y;
  __syncthreads();
  if (wave != 0) return;
  l = (red[0][0][lane] + red[0][1][lane]) + (red[0][2][lane] + red[0][3][lane]);
  x = (red[1][0][lane] + red[1][1][lane]) + (red[1][2][lane] + red[1][3][lane]);
  y = (red[2][0][lane] + red[2][1][lane]) + (red[2][2][lane] + red[2][3][lane]);
  const int i = r / a.group, gh = r - i * a.group, h = job.unit % a.c.n_kv_heads;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (lane < D / 2)
    E::store2(static_cast<char*>(a.out.p) +
                  ((job.q0 + i) * a.out.row_stride + (int64_t(h) * a.group + gh) * a.out.head_stride +
                   2 * lane) * E::kBytes,
              x * inv, y * inv);
  if (a.lse != nullptr && lane == 0)
    a.lse[(job.q0 + i) * a.c.n_q_heads + h * a.group + gh] =
        l == 0.f ? -__builtin_inff() : 0.69314718056f * (mx - kHead + log2f(l));
}

template <int D, bool kF32, int kFmt>
hipError_t launch(const PagedArgs& a, hipStream_t s) {
  const int units = a.c.n_seqs * a.c.n_kv_heads;
  const dim3 grid(uint32_t(a.n_splits * a.n_rt), units);
  const int tile = paged_tile_rows(int64_t(a.max_q) * a.group, a.c.dtype);
  if (tile == 16) hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 1>), grid, dim3(256), 0, s, a);
  else if (tile == 32) hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 2>), grid, dim3(256), 0, s, a);
  else if constexpr (!kF32) hipLaunchKernelGGL((attn_kernel<D, kF32, kFmt, 4>), grid, dim3(256), 0, s, a);
  if (a.n_splits > 1)
    hipLaunchKernelGGL((attn_combine_kernel<D, kF32>), dim3(uint32_t(a.max_q) * a.group, units),
                       dim3(256), 0, s, a, tile);
  return hipGetLastError();
}

}  // namespace

int paged_tile_rows(int64_t rows, int dtype) {
  return rows <= 16 ? 16 : rows <= 32 || dtype == NX_F32 ? 32 : 64;
}

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
