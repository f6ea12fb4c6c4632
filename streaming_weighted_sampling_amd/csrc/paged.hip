// The decode step around the attention: norm and rotation of query and key
// heads, appending rows to the paged 8-bit cache, and reading it back.
#include <type_traits>

#include "paged.hpp"

namespace nx {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// The 16 elements of one row that one thread holds, as two runs of 8, chosen
// so that a rotation pair never crosses threads: threads j < rot / 16 hold
// elements 8 j .. and rot / 2 + 8 j .. (pairs (i, i + rot / 2) face each other;
// pairs (2 i, 2 i + 1) lie inside each run), the others 16 j .. and 16 j + 8 ..
struct Runs {
  int d0, d1;
  bool rot;
};
__device__ inline Runs runs_of(int j, int rot_dim) {
  const bool rot = 16 * j < rot_dim;
  return {rot ? 8 * j : 16 * j, rot ? rot_dim / 2 + 8 * j : 16 * j + 8, rot};
}

// Table row of call row `row`; a position outside the table is noted and reads row 0.
__device__ inline const float* table_row(const nx_rope& r, int64_t row, bool& off_table) {
  int64_t p = r.positions != nullptr ? int64_t(r.positions[row]) : row;
  if (p < 0 || p >= r.n_pos) {
    off_table = true;
    p = 0;
  }
  return r.cos_sin + p * r.rot_dim;
}

__device__ inline void ld4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// Rotates a thread's runs; T = float, or double where the result is compared
// with rounding borders.
template <typename T>
__device__ inline void rotate_runs(float (&x)[8], float (&y)[8], const float* cs, int j, int rot_dim,
                                   int style) {
  const int half = rot_dim / 2;
  float c[8], s[8];
  if (style == NX_ROPE_HALF) {
    ld4(cs + 8 * j, c); ld4(cs + 8 * j + 4, c + 4);
    ld4(cs + half + 8 * j, s); ld4(cs + half + 8 * j + 4, s + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T a = x[i], b = y[i], cc = c[i], ss = s[i];
      x[i] = float(a * cc - b * ss);
      y[i] = float(b * cc + a * ss);
    }
  } else {
    // Pairs 4 j .. 4 j + 3 in the first run, half / 2 + 4 j .. in the second.
    ld4(cs + 4 * j, c); ld4(cs + half / 2 + 4 * j, c + 4);
    ld4(cs + half + 4 * j, s); ld4(cs + half + half / 2 + 4 * j, s + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float* e = i < 4 ? x + 2 * i : y + 2 * (i - 4);
      const T a = e[0], b = e[1], cc = c[i], ss = s[i];
      e[0] = float(a * cc - b * ss);
      e[1] = float(b * cc + a * ss);
    }
  }
}

// ---- norm and rotation ----
// One thread holds 16 elements of a head, head_dim / 16 threads a head; the
// square sum is reduced over them.  Memory bound: every element is read and
// written once, in 16-byte accesses (8192 rows of 64 + 8 bf16 heads of 128,
// 304 MB: 59.6 us, 5.1 TB/s, the rate of a large copy).  16 rows of 32 + 8 heads
// take 3.4 us, most of it launch and one read's latency.
template <int D, bool kF32>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormArgs a) {
  using E = Elem<kF32>;
  constexpr int kLanes = D / 16;
  const int heads = a.heads[0] + a.heads[1];
  const int64_t idx = int64_t(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes;
  const int64_t row = idx / heads;
  if (row >= a.n_rows) return;
  int h = int(idx - row * heads);
  const int side = h >= a.heads[0];
  h -= side ? a.heads[0] : 0;
  const nx_rows in = side ? a.in[1] : a.in[0], out = side ? a.out[1] : a.out[0];
  const void* weight = side ? a.weight[1] : a.weight[0];
  const Runs r = runs_of(j, a.rope.rot_dim);
  const char* src = static_cast<const char*>(in.p) + (row * in.row_stride + h * in.head_stride) * E::kBytes;
  float x[8], y[8];
  E::load8(src + r.d0 * E::kBytes, x);
  E::load8(src + r.d1 * E::kBytes, y);
  if (weight != nullptr) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * x[i] + y[i] * y[i];
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) s += __shfl_xor(s, m, 64);
    const float f = 1.0f / sqrtf(s * (1.0f / D) + a.eps);
    float w[8];
    E::load8(static_cast<const char*>(weight) + r.d0 * E::kBytes, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * w[i];
    E::load8(static_cast<const char*>(weight) + r.d1 * E::kBytes, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * f * w[i];
  }
  bool off_table = false;
  if (r.rot) rotate_runs<float>(x, y, table_row(a.rope, row, off_table), j, a.rope.rot_dim, a.rope.style);
  char* dst = static_cast<char*>(out.p) + (row * out.row_stride + h * out.head_stride) * E::kBytes;
  E::store8(dst + r.d0 * E::kBytes, x);
  E::store8(dst + r.d1 * E::kBytes, y);
  if (off_table) paged_status(a.status, kStatusBadItem);
}

// ---- append ----

// What a (sequence, head)'s append does: rows [row0, row0 + n) go to [len, len + n).
struct Span {
  int64_t row0;
  int len, n;
  bool ok;
};
__device__ inline Span append_span(const PagedArgs& a, int unit) {
  const int s = unit / a.c.n_kv_heads;
  Span p;
  p.n = seq_rows(a, s, a.max_new, &p.row0);
  p.len = a.c.lens[unit];
  p.ok = p.n >= 0 && p.len >= 0;
  if (a.head_new != nullptr) {
    const int hn = a.head_new[unit];
    p.ok = p.ok && hn >= 0 && hn <= p.n;
    p.n = hn;
  }
  p.ok = p.ok && int64_t(p.len) + p.n <= (int64_t(a.c.max_pages) << a.page_shift) * kBlock;
  return p;
}

__global__ __launch_bounds__(256) void bump_kernel(PagedArgs a, int units) {
  const int u = blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const Span p = append_span(a, u);
  if (p.ok) a.lens_out[u] = p.len + p.n;
}

// A non-finite element is stored as 0 and reported.
__device__ inline float finite_or_zero(float x, bool& bad) {
  const bool f = __builtin_isfinite(x);
  bad |= !f;
  return f ? x : 0.f;
}

// Largest magnitude of a thread's elements, as bits.
__device__ inline uint32_t top_bits(const float (&x)[8], const float (&y)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    m = max(m, max(__builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu, __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu));
  return m;
}

// The wavefront's maximum, in every lane (row shifts, row broadcasts, lane 63).
__device__ inline uint32_t wave_top(uint32_t v) {
  auto step = [&](int x) { v = max(v, uint32_t(x)); };
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false));
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// 4 values -> 4 codes, round to nearest even.  |x| exceeds the largest code by
// fp32 roundings at most, so neither conversion overflows.
template <int kFmt>
__device__ inline uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (kFmt == NX_CACHE_E4M3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
  } else {
    // Adding 1.5 * 2^23 rounds to an integer, whose two's complement is then in
    // the low bits; v_perm collects the low bytes.
    constexpr float kRound = 12582912.f;
    const uint32_t ab = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b + kRound),
                                              __builtin_bit_cast(uint32_t, a + kRound), 0x0C0C0400u);
    const uint32_t cd = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, d + kRound),
                                              __builtin_bit_cast(uint32_t, c + kRound), 0x0C0C0400u);
    return ab | (cd << 16);
  }
}

// The product is rounded by itself, as the definition has it: fused with the
// rounding addition it would move ties.
template <int kFmt>
__device__ inline u32x2_t codes8(const float (&x)[8], float inv) {
#pragma clang fp contract(off)
  return {codes4<kFmt>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
          codes4<kFmt>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
}

// Scale and inverse of a block whose largest magnitude is `top`.
template <int kFmt>
__device__ inline void block_scale(float top, float& scale, float& inv) {
  constexpr float kTop = kFmt == NX_CACHE_E4M3 ? 448.f : 127.f;
  const bool zero = !(top > 0x1p-100f);
  scale = zero ? 0.f : top * (1.f / kTop);
  inv = zero ? 0.f : (1.f / top) * kTop;
}

// Workgroup (x, head) of a sequence: block len / 32 + x of the head if the call
// fills it; x = 0 also writes the rows that stay in the tail, after it has read
// the tail's old rows.  K: 16 elements of one row per thread (rotation pairs in
// one thread).  V: 8 rows x 2 elements per thread, which is 16 consecutive
// bytes of the stored block.  Memory bound on long prompts: a block's codes
// wait for its largest magnitude, so its 32 rows stay in registers and are read
// once (four prompts of 8192 to 16384 tokens, 8 bf16 heads of 128, 344 MB: 79 us, 4.3 TB/s;
// a copy of as many bytes 69).  One token for 16 sequences: 5.6 us, launch and
// the chain lengths -> tail -> maximum -> codes.
template <int D, bool kF32, int kFmt>
__global__ __launch_bounds__(256, kF32 ? 4 : 6) void append_kernel(PagedArgs a) {
  using E = Elem<kF32>;
  constexpr int kLanes = D / 16;                 // K threads per row
  constexpr int kUse = 32 * kLanes;              // threads at work: 256 or 128
  const int tid = threadIdx.x, hk = a.c.n_kv_heads;
  // The heads of one row range run side by side: their rows lie next to each
  // other in a projection, and they share the rotation table's rows.  With
  // eight ranges or more the heads of a range are eight workgroups apart, so on
  // one XCD and its L2.
  const int id = blockIdx.x;
  const int nth = a.append_by8 ? id / (8 * hk) * 8 + id % 8 : id / hk;
  const int h = a.append_by8 ? id % (8 * hk) / 8 : id % hk;
  const int unit = blockIdx.y * hk + h;
  const Span p = append_span(a, unit);
  if (!p.ok) {
    if (nth == 0 && tid == 0) {
      paged_status(a.status, kStatusBadItem);
      if (a.lens_out != a.c.lens) a.lens_out[unit] = a.c.lens[unit];
    }
    return;
  }
  const int end = p.len + p.n;
  const int first = p.len / kBlock, open = end / kBlock;
  const int b = first + nth;
  char* kt = static_cast<char*>(a.c.k_tail) + int64_t(unit) * kBlock * D * E::kBytes;
  char* vt = static_cast<char*>(a.c.v_tail) + int64_t(unit) * kBlock * D * E::kBytes;
  const int krow = tid / kLanes, kj = tid % kLanes;
  const Runs r = runs_of(kj, a.rope.rot_dim);
  const int vg = tid / (D / 2), vd = tid % (D / 2) * 2;
  const bool on = tid < kUse;
  bool bad = false, off_table = false;

  // Where new row i (uniform or per thread) starts.
  auto k_at = [&](int64_t i) {
    return static_cast<const char*>(a.k.p) + ((p.row0 + i) * a.k.row_stride + h * a.k.head_stride) * E::kBytes;
  };
  auto v_at = [&](int64_t i) {
    return static_cast<const char*>(a.v.p) + ((p.row0 + i) * a.v.row_stride + h * a.v.head_stride) * E::kBytes;
  };
  // Rotates and rounds the K elements of new row i.
  auto turn_k = [&](int i, float (&x)[8], float (&y)[8]) {
    if (r.rot)
      rotate_runs<double>(x, y, table_row(a.rope, p.row0 + i, off_table), kj, a.rope.rot_dim, a.rope.style);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = E::round(x[e]);
      y[e] = E::round(y[e]);
    }
  };
  auto clear = [&](float (&x)[8], float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = finite_or_zero(x[e], bad);
      y[e] = finite_or_zero(y[e], bad);
    }
  };

  if (b < open) {   // this call fills block b (uniform over the workgroup)
    const int page = a.c.table[int64_t(unit) * a.c.max_pages + (b >> a.page_shift)];
    const bool page_ok = page >= 0 && page < a.c.n_pages;
    float kx[8] = {}, ky[8] = {}, vx[8] = {}, vy[8] = {};
    if (on) {
      const int new0 = b * kBlock - p.len;      // new row at the block's start (< 0: the tail's rows come first)
      if (new0 >= 0) {
        // Uniform bases, 32-bit offsets.  V's and K's loads are on their way
        // before K waits for its table row.
        const int vstep = int(a.v.row_stride) * E::kBytes;
        const Buf vb(v_at(new0), 0x7FFFFFFF), kb(k_at(new0), 0x7FFFFFFF);
        typename E::Pair w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = E::ld_pair(vb, vg * 8 * vstep + vd * E::kBytes, i * vstep);
        const int koff = krow * (int(a.k.row_stride) * E::kBytes);
        E::unpack8(kb.ld16(koff + r.d0 * E::kBytes), kF32 ? kb.ld16(koff + r.d0 * E::kBytes + 16) : uint4{}, kx);
        E::unpack8(kb.ld16(koff + r.d1 * E::kBytes), kF32 ? kb.ld16(koff + r.d1 * E::kBytes + 16) : uint4{}, ky);
        turn_k(new0 + krow, kx, ky);
#pragma unroll
        for (int i = 0; i < 8; ++i) E::split(w[i], vx[i], vy[i]);
      } else {
        const int t = new0 + krow, tv = new0 + vg * 8;
        if (t < 0) {
          E::load8(kt + (krow * D + r.d0) * E::kBytes, kx);
          E::load8(kt + (krow * D + r.d1) * E::kBytes, ky);
        } else {
          E::load8(k_at(t) + r.d0 * E::kBytes, kx);
          E::load8(k_at(t) + r.d1 * E::kBytes, ky);
          turn_k(t, kx, ky);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (tv + i < 0) {
            vx[i] = E::load1(vt + ((vg * D + vd) * 8 + i) * E::kBytes);
            vy[i] = E::load1(vt + ((vg * D + vd + 1) * 8 + i) * E::kBytes);
          } else {
            E::load2(v_at(tv + i) + vd * E::kBytes, vx[i], vy[i]);
          }
        }
      }
    }
    // Magnitudes are compared as integers, where NaN and infinity come last.
    uint32_t km = top_bits(kx, ky), vm = top_bits(vx, vy);
    if (__builtin_expect(max(km, vm) >= 0x7F800000u, 0)) {
      clear(kx, ky);
      clear(vx, vy);
      km = top_bits(kx, ky);
      vm = top_bits(vx, vy);
    }
    km = wave_top(km);
    vm = wave_top(vm);
    __shared__ uint32_t red[2][4];
    if (tid % 64 == 0) {
      red[0][tid / 64] = km;
      red[1][tid / 64] = vm;
    }
    // The maxima depend on every tail row read above, so past this barrier the
    // tail may be overwritten.
    __syncthreads();
    const float ktop = __builtin_bit_cast(float, max(max(red[0][0], red[0][1]), max(red[0][2], red[0][3])));
    const float vtop = __builtin_bit_cast(float, max(max(red[1][0], red[1][1]), max(red[1][2], red[1][3])));
    float kscale, kinv, vscale, vinv;
    block_scale<kFmt>(ktop, kscale, kinv);
    block_scale<kFmt>(vtop, vscale, vinv);
    if (!page_ok) {
      if (tid == 0) paged_status(a.status, kStatusBadItem);
    } else if (on) {
      const int64_t slot = (int64_t(page) << a.page_shift) + (b & ((1 << a.page_shift) - 1));
      char* kc = static_cast<char*>(a.c.k_codes) + slot * kBlock * D;
      char* vc = static_cast<char*>(a.c.v_codes) + slot * kBlock * D;
      const u32x2_t k0 = codes8<kFmt>(kx, kinv), k1 = codes8<kFmt>(ky, kinv);
      const u32x2_t v0 = codes8<kFmt>(vx, vinv), v1 = codes8<kFmt>(vy, vinv);
      const u32x4_t v = {v0.x, v0.y, v1.x, v1.y};
      const Buf kb(kc, kBlock * D), vb(vc, kBlock * D);
      auto put = [&](auto aux) {
        __builtin_amdgcn_raw_buffer_store_b64(k0, kb.r, krow * D + r.d0, 0, aux.value);
        __builtin_amdgcn_raw_buffer_store_b64(k1, kb.r, krow * D + r.d1, 0, aux.value);
        __builtin_amdgcn_raw_buffer_store_b128(v, vb.r, (vg * D + vd) * 8, 0, aux.value);
      };
      if (a.stream_nt) put(std::integral_constant<int, kNonTemporal>{});
      else put(std::integral_constant<int, 0>{});
      if (tid == 0) {
        a.c.k_scale[slot] = kscale;
        a.c.v_scale[slot] = vscale;
      }
    }
  }
  if (nth == 0) {
    // New rows of the block that stays open.
    if (on) {
      const int t = open * kBlock + krow;
      if (t >= p.len && t < end) {
        float x[8], y[8];
        E::load8(k_at(t - p.len) + r.d0 * E::kBytes, x);
        E::load8(k_at(t - p.len) + r.d1 * E::kBytes, y);
        turn_k(t - p.len, x, y);
        clear(x, y);
        E::store8(kt + (krow * D + r.d0) * E::kBytes, x);
        E::store8(kt + (krow * D + r.d1) * E::kBytes, y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tv = open * kBlock + vg * 8 + i;
        if (tv >= p.len && tv < end) {
          float x, y;
          E::load2(v_at(tv - p.len) + vd * E::kBytes, x, y);
          char* e = vt + ((vg * D + vd) * 8 + i) * E::kBytes;
          E::store1(e, finite_or_zero(x, bad));
          E::store1(e + 8 * E::kBytes, finite_or_zero(y, bad));
        }
      }
    }
    // In place the count may change only when every wavefront has read it.
    __syncthreads();
    if (tid == 0 && !a.bump) a.lens_out[unit] = end;
  }
  if (bad) paged_status(a.status, kStatusNonFinite);
  if (off_table) paged_status(a.status, kStatusBadItem);
}

// ---- gather ----

__device__ inline void decode4(int fmt, uint32_t w, float s, float* x) {
  if (fmt == NX_CACHE_E4M3) {
    const h2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, false);
    const h2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, true);
    x[0] = float(lo.x) * s; x[1] = float(lo.y) * s; x[2] = float(hi.x) * s; x[3] = float(hi.y) * s;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = float(int8_t(w >> (8 * i))) * s;
  }
}

// Workgroup (block, unit): 32 rows, or the tail's.  Reads are 16 bytes a
// thread; K rows are written 16 or 32 bytes a thread, V rows two elements a
// thread (a row's D elements by consecutive threads).  Memory bound, and at the
// rate of a large copy (16 heads of 65536 to 131077 rows, 1.25 GB: 246 us, 5.1 TB/s;
// 8 heads of 6810 rows, 42 MB: 9 us).
template <int D, bool kF32, int kFmt>
__global__ __launch_bounds__(256) void gather_kernel(PagedArgs a) {
  using E = Elem<kF32>;
  constexpr int kLanes = D / 16;
  const int unit = blockIdx.y, tid = threadIdx.x, b = blockIdx.x;
  const int len = a.c.lens[unit];
  if (len < 0 || len > a.max_tokens || int64_t(len) > (int64_t(a.c.max_pages) << a.page_shift) * kBlock) {
    if (b == 0 && tid == 0) paged_status(a.status, kStatusBadItem);
    return;
  }
  if (b * kBlock >= len || tid >= 32 * kLanes) return;
  const int s = unit / a.c.n_kv_heads, h = unit % a.c.n_kv_heads;
  const int64_t at = (s * a.out_seq_stride + h * a.out_head_stride + int64_t(b) * kBlock * D) * E::kBytes;
  char* ok = static_cast<char*>(a.out_k) + at;
  char* ov = static_cast<char*>(a.out_v) + at;
  const int krow = tid / kLanes, kd = tid % kLanes * 16;
  const int vg = tid / (D / 2), vd = tid % (D / 2) * 2;
  if (b == len / kBlock) {
    const int n = len % kBlock;
    const char* kt = static_cast<const char*>(a.c.k_tail) + int64_t(unit) * kBlock * D * E::kBytes;
    const char* vt = static_cast<const char*>(a.c.v_tail) + int64_t(unit) * kBlock * D * E::kBytes;
    if (krow < n) {
      float x[8];
      E::load8(kt + (krow * D + kd) * E::kBytes, x);
      E::store8(ok + (krow * D + kd) * E::kBytes, x);
      E::load8(kt + (krow * D + kd + 8) * E::kBytes, x);
      E::store8(ok + (krow * D + kd + 8) * E::kBytes, x);
    }
    float x[8], y[8];
    E::load8(vt + (vg * D + vd) * 8 * E::kBytes, x);
    E::load8(vt + (vg * D + vd + 1) * 8 * E::kBytes, y);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (vg * 8 + i < n) E::store2(ov + ((vg * 8 + i) * D + vd) * E::kBytes, x[i], y[i]);
    return;
  }
  const int page = a.c.table[int64_t(unit) * a.c.max_pages + (b >> a.page_shift)];
  if (page < 0 || page >= a.c.n_pages) {
    if (tid == 0) paged_status(a.status, kStatusBadItem);
    return;
  }
  const int64_t slot = (int64_t(page) << a.page_shift) + (b & ((1 << a.page_shift) - 1));
  const uint4 kw = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.c.k_codes) +
                                                   slot * kBlock * D + krow * D + kd);
  const uint4 vw = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.c.v_codes) +
                                                   slot * kBlock * D + (vg * D + vd) * 8);
  const float ksc = a.c.k_scale[slot], vsc = a.c.v_scale[slot];
  float x[8], y[8];
  decode4(kFmt, kw.x, ksc, x);
  decode4(kFmt, kw.y, ksc, x + 4);
  decode4(kFmt, kw.z, ksc, y);
  decode4(kFmt, kw.w, ksc, y + 4);
  E::store8(ok + (krow * D + kd) * E::kBytes, x);
  E::store8(ok + (krow * D + kd + 8) * E::kBytes, y);
  decode4(kFmt, vw.x, vsc, x);
  decode4(kFmt, vw.y, vsc, x + 4);
  decode4(kFmt, vw.z, vsc, y);
  decode4(kFmt, vw.w, vsc, y + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) E::store2(ov + ((vg * 8 + i) * D + vd) * E::kBytes, x[i], y[i]);
}

// Calls f.template operator()<D, kF32, kFmt>() for the call's shape.
template <typename F>
void dispatch(const nx_paged& c, F&& f) {
  const bool d128 = c.head_dim == 128, f32 = c.dtype == NX_F32, i8 = c.format == NX_CACHE_I8;
  if (d128) {
    if (f32) i8 ? f.template operator()<128, true, 1>() : f.template operator()<128, true, 0>();
    else i8 ? f.template operator()<128, false, 1>() : f.template operator()<128, false, 0>();
  } else {
    if (f32) i8 ? f.template operator()<64, true, 1>() : f.template operator()<64, true, 0>();
    else i8 ? f.template operator()<64, false, 1>() : f.template operator()<64, false, 0>();
  }
}

struct AppendLaunch {
  const PagedArgs& a;
  dim3 grid;
  hipStream_t s;
  template <int D, bool kF32, int kFmt> void operator()() const {
    hipLaunchKernelGGL((append_kernel<D, kF32, kFmt>), grid, dim3(256), 0, s, a);
  }
};
struct GatherLaunch {
  const PagedArgs& a;
  dim3 grid;
  hipStream_t s;
  template <int D, bool kF32, int kFmt> void operator()() const {
    hipLaunchKernelGGL((gather_kernel<D, kF32, kFmt>), grid, dim3(256), 0, s, a);
  }
};

}  // namespace

hipError_t launch_norm_rope(const NormArgs& a, hipStream_t s) {
  const int64_t heads = int64_t(a.n_rows) * (a.heads[0] + a.heads[1]);
  const int per = 256 / (a.head_dim / 16);
  const dim3 grid(uint32_t((heads + per - 1) / per));
  if (a.head_dim == 128) {
    if (a.dtype == NX_F32) hipLaunchKernelGGL((norm_rope_kernel<128, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((norm_rope_kernel<128, false>), grid, dim3(256), 0, s, a);
  } else {
    if (a.dtype == NX_F32) hipLaunchKernelGGL((norm_rope_kernel<64, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((norm_rope_kernel<64, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_paged_append(const PagedArgs& a, hipStream_t s) {
  const int units = a.c.n_seqs * a.c.n_kv_heads;
  // Blocks that max_new rows can fill from any starting row, at least one workgroup.
  const int64_t fills = a.max_new > 0 ? (a.max_new + kBlock - 1) / kBlock : 1;
  PagedArgs x = a;
  // In place, counts read by several workgroups are advanced by a launch of their own.
  x.bump = a.lens_out == a.c.lens && fills > 1;
  x.append_by8 = fills >= 8;
  const int64_t ranges = x.append_by8 ? (fills + 7) / 8 * 8 : fills;
  dispatch(a.c, AppendLaunch{x, dim3(uint32_t(ranges * a.c.n_kv_heads), a.c.n_seqs), s});
  if (x.bump)
    hipLaunchKernelGGL(bump_kernel, dim3((units + 255) / 256), dim3(256), 0, s, x, units);
  return hipGetLastError();
}

hipError_t launch_paged_gather(const PagedArgs& a, hipStream_t s) {
  const int units = a.c.n_seqs * a.c.n_kv_heads;
  dispatch(a.c, GatherLaunch{a, dim3((a.max_tokens + kBlock - 1) / kBlock, units), s});
  return hipGetLastError();
}

}  // namespace nx
