// The decode step around the attention: norm and rotation of query and key
// heads, appending rows to the paged 8-bit cache, and reading it back.
#include "paged.hpp"

namespace nx {
namespace {

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

// Table row of call row `row`; a position outside the table is reported and reads row 0.
__device__ inline const float* table_row(const nx_rope& r, int64_t row, uint32_t* status) {
  int64_t p = r.positions != nullptr ? int64_t(r.positions[row]) : row;
  if (p < 0 || p >= r.n_pos) {
    paged_status(status, kStatusBadItem);
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
// written once, in 16-byte accesses.
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
  if (r.rot)
    rotate_runs<float>(x, y, table_row(a.rope, row, a.status), j, a.rope.rot_dim, a.rope.style);
  char* dst = static_cast<char*>(out.p) + (row * out.row_stride + h * out.head_stride) * E::kBytes;
  E::store8(dst + r.d0 * E::kBytes, x);
  E::store8(dst + r.d1 * E::kBytes, y);
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

// 4 values -> 4 codes, round to nearest even.  |x| exceeds the largest code by
// fp32 roundings at most, so neither conversion overflows.
template <int kFmt>
__device__ inline uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (kFmt == NX_CACHE_E4M3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
  } else {
    const uint32_t x = uint32_t(int(rintf(a))) & 0xFFu, y = uint32_t(int(rintf(b))) & 0xFFu;
    const uint32_t z = uint32_t(int(rintf(c))) & 0xFFu, t = uint32_t(int(rintf(d)));
    return x | (y << 8) | (z << 16) | (t << 24);
  }
}

// Scale and inverse of a block whose largest magnitude is `top`.
template <int kFmt>
__device__ inline void block_scale(float top, float& scale, float& inv) {
  constexpr float kTop = kFmt == NX_CACHE_E4M3 ? 448.f : 127.f;
  const bool zero = !(top > 0x1p-100f);
  scale = zero ? 0.f : top * (1.f / kTop);
  inv = zero ? 0.f : (1.f / top) * kTop;
}

// Workgroup (x, unit): block len / 32 + x of the (sequence, head) if the call
// fills it; x = 0 also writes the rows that stay in the tail, after it has read
// the tail's old rows.  K: 16 elements of one row per thread (rotation pairs in
// one thread).  V: 8 rows x 2 elements per thread, which is 16 consecutive
// bytes of the stored block.
template <int D, bool kF32, int kFmt>
__global__ __launch_bounds__(256) void append_kernel(PagedArgs a) {
  using E = Elem<kF32>;
  constexpr int kLanes = D / 16;                 // K threads per row
  constexpr int kUse = 32 * kLanes;              // threads at work: 256 or 128
  const int unit = blockIdx.y, tid = threadIdx.x;
  const int h = unit % a.c.n_kv_heads;
  const Span p = append_span(a, unit);
  if (!p.ok) {
    if (blockIdx.x == 0 && tid == 0) {
      paged_status(a.status, kStatusBadItem);
      if (a.lens_out != a.c.lens) a.lens_out[unit] = a.c.lens[unit];
    }
    return;
  }
  const int end = p.len + p.n;
  const int first = p.len / kBlock, open = end / kBlock;
  const int b = first + blockIdx.x;
  const char* ks = static_cast<const char*>(a.k.p) + h * a.k.head_stride * E::kBytes;
  const char* vs = static_cast<const char*>(a.v.p) + h * a.v.head_stride * E::kBytes;
  char* kt = static_cast<char*>(a.c.k_tail) + int64_t(unit) * kBlock * D * E::kBytes;
  char* vt = static_cast<char*>(a.c.v_tail) + int64_t(unit) * kBlock * D * E::kBytes;
  const int krow = tid / kLanes, kj = tid % kLanes;
  const Runs r = runs_of(kj, a.rope.rot_dim);
  const int vg = tid / (D / 2), vd = tid % (D / 2) * 2;
  const bool on = tid < kUse;
  bool bad = false;

  // Rotated and rounded K elements of new row i.
  auto new_k = [&](int i, float (&x)[8], float (&y)[8]) {
    const int64_t row = p.row0 + i;
    const char* src = ks + row * a.k.row_stride * E::kBytes;
    E::load8(src + r.d0 * E::kBytes, x);
    E::load8(src + r.d1 * E::kBytes, y);
    if (r.rot)
      rotate_runs<double>(x, y, table_row(a.rope, row, a.status), kj, a.rope.rot_dim, a.rope.style);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = finite_or_zero(E::round(x[e]), bad);
      y[e] = finite_or_zero(E::round(y[e]), bad);
    }
  };
  auto new_v = [&](int i, float& x, float& y) {
    E::load2(vs + ((p.row0 + i) * a.v.row_stride + vd) * E::kBytes, x, y);
    x = finite_or_zero(x, bad);
    y = finite_or_zero(y, bad);
  };

  if (b < open) {   // this call fills block b (uniform over the workgroup)
    const int page = a.c.table[int64_t(unit) * a.c.max_pages + (b >> a.page_shift)];
    const bool page_ok = page >= 0 && page < a.c.n_pages;
    float kx[8] = {}, ky[8] = {}, vx[16] = {};
    if (on) {
      const int t = b * kBlock + krow;
      if (t < p.len) {
        E::load8(kt + (krow * D + r.d0) * E::kBytes, kx);
        E::load8(kt + (krow * D + r.d1) * E::kBytes, ky);
      } else {
        new_k(t - p.len, kx, ky);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tv = b * kBlock + vg * 8 + i;
        if (tv < p.len) {
          const char* e = vt + ((vg * D + vd) * 8 + i) * E::kBytes;
          if constexpr (kF32) {
            vx[i] = *reinterpret_cast<const float*>(e);
            vx[8 + i] = *reinterpret_cast<const float*>(e + 32);
          } else {
            vx[i] = float(*reinterpret_cast<const __bf16*>(e));
            vx[8 + i] = float(*reinterpret_cast<const __bf16*>(e + 16));
          }
        } else {
          new_v(tv - p.len, vx[i], vx[8 + i]);
        }
      }
    }
    float km = 0.f, vm = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      km = fmaxf(km, fmaxf(fabsf(kx[i]), fabsf(ky[i])));
      vm = fmaxf(vm, fmaxf(fabsf(vx[i]), fabsf(vx[8 + i])));
    }
    km = fmaxf(half_max(km), __shfl_xor(half_max(km), 32, 64));
    vm = fmaxf(half_max(vm), __shfl_xor(half_max(vm), 32, 64));
    __shared__ float red[2][4];
    if (tid % 64 == 0) {
      red[0][tid / 64] = km;
      red[1][tid / 64] = vm;
    }
    // The maxima depend on every tail row read above, so past this barrier the
    // tail may be overwritten.
    __syncthreads();
    km = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    vm = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    float kscale, kinv, vscale, vinv;
    block_scale<kFmt>(km, kscale, kinv);
    block_scale<kFmt>(vm, vscale, vinv);
    if (!page_ok) {
      if (tid == 0) paged_status(a.status, kStatusBadItem);
    } else if (on) {
      const int64_t slot = (int64_t(page) << a.page_shift) + (b & ((1 << a.page_shift) - 1));
      char* kc = static_cast<char*>(a.c.k_codes) + slot * kBlock * D;
      char* vc = static_cast<char*>(a.c.v_codes) + slot * kBlock * D;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        kx[i] *= kinv;
        ky[i] *= kinv;
        vx[i] *= vinv;
        vx[8 + i] *= vinv;
      }
      const uint32_t k0 = codes4<kFmt>(kx[0], kx[1], kx[2], kx[3]);
      const uint32_t k1 = codes4<kFmt>(kx[4], kx[5], kx[6], kx[7]);
      const uint32_t k2 = codes4<kFmt>(ky[0], ky[1], ky[2], ky[3]);
      const uint32_t k3 = codes4<kFmt>(ky[4], ky[5], ky[6], ky[7]);
      *reinterpret_cast<uint2*>(kc + krow * D + r.d0) = make_uint2(k0, k1);
      *reinterpret_cast<uint2*>(kc + krow * D + r.d1) = make_uint2(k2, k3);
      *reinterpret_cast<uint4*>(vc + (vg * D + vd) * 8) =
          make_uint4(codes4<kFmt>(vx[0], vx[1], vx[2], vx[3]), codes4<kFmt>(vx[4], vx[5], vx[6], vx[7]),
                     codes4<kFmt>(vx[8], vx[9], vx[10], vx[11]),
                     codes4<kFmt>(vx[12], vx[13], vx[14], vx[15]));
      if (tid == 0) {
        a.c.k_scale[slot] = kscale;
        a.c.v_scale[slot] = vscale;
      }
    }
  }
  if (blockIdx.x == 0) {
    // New rows of the block that stays open.
    if (on) {
      const int t = open * kBlock + krow;
      if (t >= p.len && t < end) {
        float x[8], y[8];
        new_k(t - p.len, x, y);
        E::store8(kt + (krow * D + r.d0) * E::kBytes, x);
        E::store8(kt + (krow * D + r.d1) * E::kBytes, y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tv = open * kBlock + vg * 8 + i;
        if (tv >= p.len && tv < end) {
          float x, y;
          new_v(tv - p.len, x, y);
          char* e = vt + ((vg * D + vd) * 8 + i) * E::kBytes;
          E::store1(e, x);
          E::store1(e + 8 * E::kBytes, y);
        }
      }
    }
    if (tid == 0 && !a.bump) a.lens_out[unit] = end;
  }
  if (bad) paged_status(a.status, kStatusNonFinite);
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
// thread (a row's D elements by consecutive threads).
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
  const int fills = a.max_new > 0 ? (a.max_new + kBlock - 1) / kBlock : 1;
  PagedArgs x = a;
  // In place, counts read by several workgroups are advanced by a launch of their own.
  x.bump = a.lens_out == a.c.lens && fills > 1;
  dispatch(a.c, AppendLaunch{x, dim3(fills, units), s});
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
