// Internal interface of the decode-step operators (paged 8-bit cache, norm and
// rotation): argument blocks, launchers, and device helpers shared by
// paged.hip and paged_attn.hip.
#pragma once

#include "nx_device.hpp"

namespace nx {

constexpr int kBlock = NX_CACHE_BLOCK;     // rows that share one scale

// Kernel argument block of the nx_paged_* calls, passed by value.
struct PagedArgs {
  nx_paged c;
  nx_rope rope;            // append; rot_dim 0: no rotation
  nx_rows k, v;            // append: new rows
  nx_rows q, out;          // attention
  int32_t n_rows;          // rows of k / v or q / out
  int32_t max_new;         // append: bound on a sequence's rows (uniform count without starts)
  const int32_t* start;    // new_start / q_start
  const int32_t* head_new;
  int32_t* lens_out;       // append: where the new counts go (never null)
  int32_t bump;            // append: 1: a second launch advances lens_out == lens
  int32_t append_by8;      // append: 1: a range's heads are eight workgroups apart
  int32_t page_shift;      // log2(page_blocks)
  int32_t stream_nt;       // 1: the codes are read or written past the caches
  uint32_t* status;
  // attention
  int32_t group, max_q, n_rt, n_wg;   // query-row tiles, workgroups wanted
  int32_t min_share;       // fewest blocks of a full piece
  int32_t whole;           // 1: a workgroup per head, no pieces
  float scale_log2;        // scale * log2(e)
  float* lse;
  int2* pieces;            // [units]: a head's pieces (0: written at once) and its first partial
  float* part_o;           // [2 * n_wg][n_rt][tile rows][D]
  float* part_ml;          // [2 * n_wg][n_rt][tile rows][2]: (base, sum), log2 units
  // gather
  int32_t max_tokens;
  void* out_k;
  void* out_v;
  int64_t out_seq_stride, out_head_stride;
};

struct NormArgs {
  nx_rope rope;
  nx_rows in[2], out[2];   // q, k
  const void* weight[2];
  int32_t heads[2];        // heads of each side (0: side absent)
  int32_t n_rows;
  int32_t head_dim, dtype;
  float eps;
  uint32_t* status;
};

hipError_t launch_paged_append(const PagedArgs& a, hipStream_t s);
hipError_t launch_paged_attn(const PagedArgs& a, hipStream_t s);
hipError_t launch_paged_gather(const PagedArgs& a, hipStream_t s);
hipError_t launch_norm_rope(const NormArgs& a, hipStream_t s);

// Query rows per tile of a call with `rows` = queries * group rows per
// (sequence, KV head).
int paged_tile_rows(int64_t rows);

// ---- device side ----

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Element types of the rows: 8 consecutive elements to and from fp32.
template <bool kF32> struct Elem;
template <> struct Elem<false> {
  static constexpr int kBytes = 2;
  // 8 elements from one 16-byte word (fp32: two).
  static __device__ void unpack8(uint4 w, uint4, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __builtin_bit_cast(float, u[i] << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
    }
  }
  static __device__ void load8(const void* p, float (&x)[8]) {
    unpack8(*static_cast<const uint4*>(p), uint4{}, x);
  }
  static __device__ float round(float x) { return float(__bf16(x)); }
  static __device__ uint32_t pack2(float a, float b) {
    return uint32_t(__builtin_bit_cast(uint16_t, __bf16(a))) |
           (uint32_t(__builtin_bit_cast(uint16_t, __bf16(b))) << 16);
  }
  static __device__ void store8(void* p, const float (&x)[8]) {
    *static_cast<uint4*>(p) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
  using Pair = uint32_t;   // two elements as loaded
  static __device__ Pair ld_pair(const Buf& b, int off, int uniform) {
    return __builtin_amdgcn_raw_buffer_load_b32(b.r, off, uniform, 0);
  }
  static __device__ void split(Pair u, float& a, float& b) {
    a = __builtin_bit_cast(float, u << 16);
    b = __builtin_bit_cast(float, u & 0xFFFF0000u);
  }
  static __device__ void load2(const void* p, float& a, float& b) { split(*static_cast<const Pair*>(p), a, b); }
  static __device__ float load1(const void* p) { return float(*static_cast<const __bf16*>(p)); }
  static __device__ void store2(void* p, float a, float b) {
    *static_cast<uint32_t*>(p) = pack2(a, b);
  }
  static __device__ void store1(void* p, float a) { *static_cast<__bf16*>(p) = __bf16(a); }
};
template <> struct Elem<true> {
  static constexpr int kBytes = 4;
  static __device__ void unpack8(uint4 v, uint4 w, float (&x)[8]) {
    const float4 a = __builtin_bit_cast(float4, v), b = __builtin_bit_cast(float4, w);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ void load8(const void* p, float (&x)[8]) {
    unpack8(static_cast<const uint4*>(p)[0], static_cast<const uint4*>(p)[1], x);
  }
  static __device__ float round(float x) { return x; }
  static __device__ void store8(void* p, const float (&x)[8]) {
    static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
  using Pair = float2;
  static __device__ Pair ld_pair(const Buf& b, int off, int uniform) {
    return __builtin_bit_cast(float2, __builtin_amdgcn_raw_buffer_load_b64(b.r, off, uniform, 0));
  }
  static __device__ void split(Pair u, float& a, float& b) {
    a = u.x;
    b = u.y;
  }
  static __device__ void load2(const void* p, float& a, float& b) { split(*static_cast<const Pair*>(p), a, b); }
  static __device__ float load1(const void* p) { return *static_cast<const float*>(p); }
  static __device__ void store2(void* p, float a, float b) {
    *static_cast<float2*>(p) = make_float2(a, b);
  }
  static __device__ void store1(void* p, float a) { *static_cast<float*>(p) = a; }
};

__device__ inline void paged_status(uint32_t* status, uint32_t bits) { atomicOr(status, bits); }

// Rows [lo, lo + n) of sequence s in the call's row arrays; n = -1: out of range.
__device__ inline int seq_rows(const PagedArgs& a, int s, int most, int64_t* lo) {
  if (a.start == nullptr) {
    *lo = int64_t(s) * most;
    return most;
  }
  const int x = a.start[s], y = a.start[s + 1];
  *lo = x;
  return x < 0 || y < x || y > a.n_rows || y - x > most ? -1 : y - x;
}

}  // namespace nx
