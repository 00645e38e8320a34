// Internals of the dense 8-bit operators: row norm + quantisation, 8-bit products.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

constexpr int kNormMaxWidth = 32768;    // widest row: 1024 threads x 4 chunks of 8
constexpr int kI8MaxWidth = 65536;      // |sum| <= 65536 * 128 * 128 = 2^30: int32 sums are exact
// A launch has fewer than 2^32 threads: rows (a workgroup of up to 1024 each in the norm), columns
// (16 per workgroup of 512) and outputs (at least 8192 per workgroup of 512 where there are many)
constexpr int64_t kMaxRows = int64_t(1) << 21, kMaxOutputs = int64_t(1) << 35;
constexpr int kMaxColumns = 1 << 24;

struct NormQuant {
  int64_t rows;
  int width, act, format;
  const void* x;
  const void* res;     // null: no residual
  const void* gamma;   // null: no norm
  float eps;
  void* x_sum;
  void* out;
  void* scales;
};
int launch_norm_quant(const NormQuant& q, hipStream_t st);

// y = act(x w^T * scales): one weight matrix, or gate and up for the gated product
struct I8Product {
  int64_t T;
  int K, N;
  int out;                 // MOE_F32 | MOE_BF16
  const int8_t* x;         // [T, K]
  const float* sx;         // [T]
  const int8_t* w;         // [N, K]
  const float* sw;         // [N]
  const int8_t* w_up;      // gated product: the up matrix, else null
  const float* s_up;
  const void* res;         // [T, N] out type, or null
  void* y;                 // [T, N] out type
};
int launch_i8_product(const I8Product& p, hipStream_t st);

// The gated product with h as int16 codes and group maxima ([T, N] and [T, ceil(N / 32)]; out is
// ignored), where one of the two widest tiles is chosen; and the int8 codes of such rows.
bool glu_h16_ok(int64_t T, int K, int N);
int launch_glu_h16(const I8Product& p, float* hmax, hipStream_t st);
int launch_h16_codes(const void* h, const float* hmax, int64_t T, int I, int8_t* codes, float* scales,
                     hipStream_t st);

// The dense layer of a few tokens in two launches
struct DenseFew {
  int64_t T;
  int H, I, act;
  const void* x;
  const void* gamma;
  float eps;
  const moe_dense_weights* w;
  float* h;                // [T, I]
  float* hmax;             // dense_few_hmax_bytes()
  void* x_out;
};
bool dense_few_ok(int64_t T, int H, int I);
size_t dense_few_hmax_bytes(int64_t T, int I);
int launch_dense_few(const DenseFew& d, hipStream_t st);

#ifdef __HIPCC__
// 1 / sqrt(mean square + eps) of a row: once per row, so in 64 bits (an error here would shift
// every code of the row).  A row without squares and without eps is left as it is, at zero.
__device__ __forceinline__ float inv_rms(float sum_sq, int width, float eps) {
  const double ms = double(sum_sq) / width + double(eps);
  return ms == 0.0 ? 0.0f : float(1.0 / sqrt(ms));
}
// Maximum that keeps a NaN (one v_maximum3_f32 for two of them): 8-bit codes cannot hold one, so
// a row's or block's scale carries it on to whatever reads the codes.
__device__ __forceinline__ float nmax(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_nmax(float v) {
  v = nmax(v, dppf<0xB1>(v));
  v = nmax(v, dppf<0x4E>(v));
  v = nmax(v, dppf<0x141>(v));
  v = nmax(v, dppf<0x140>(v));
  return nmax(nmax(lanef(v, 0), lanef(v, 16)), nmax(lanef(v, 32), lanef(v, 48)));
}
// Per-row int8: scale = amax / 127.  A row whose amax is so small that the scale would leave
// the normal floats (or is zero) has scale 1 and codes 0, so no division overflows.
__device__ __forceinline__ float i8_scale(float amax) {
  const float s = amax / 127.0f;
  return s < 1.17549435e-38f ? 1.0f : s;
}
// the block-FP8 rule of quant_e4m3_wave with the same guard
__device__ __forceinline__ float e4m3_scale(float amax) {
  const float s = amax / 448.0f;
  return s < 1.17549435e-38f ? 1.0f : s;
}
// v / scale for many values of one scale: the product with the reciprocal and one correction
// step, within an ulp of the quotient, in three operations where the division sequence takes
// about ten.
struct Divider {
  float scale, inv;
  __device__ __forceinline__ explicit Divider(float s) : scale(s), inv(1.0f / s) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * inv;
    return fmaf(fmaf(-q, scale, v), inv, q);
  }
};
// SiLU with the hardware reciprocal (an ulp), for outputs of 16 bits.  The denominator is taken at
// a sixteenth, so that its reciprocal stays a normal float up to where exp(-g) overflows.
__device__ __forceinline__ float silu16(float g) {
  return (g * 0.0625f) * __builtin_amdgcn_rcpf(fmaf(__expf(-g), 0.0625f, 0.0625f));
}
// Eight values -> eight int8 codes, round to nearest even (|v| / scale <= 127 up to the
// division's rounding, which the clamp takes back).
__device__ __forceinline__ uint2 i8x8(const float (&v)[8], const Divider& by) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rintf(by(v[i])), -127.f), 127.f);
    w[i / 4] |= (uint32_t(int(q)) & 0xFFu) << (8 * (i % 4));
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = uint32_t(f32_to_bf16(v[2 * i])) | (uint32_t(f32_to_bf16(v[2 * i + 1])) << 16);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// p = round(a + b); a is replaced by the rounded sum
template <typename TA>
__device__ __forceinline__ void add_store8(TA* p, float (&a)[8], const float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = to_f32<TA>(from_f32<TA>(a[i] + b[i]));
  store8(p, a);
}
#endif

}  // namespace moe
