// Products of 8-bit integer rows and 8-bit integer weights with a scale per token and per
// output channel, alone (k_i8_few<..., false>) or as the gated pair h = silu(g) * u.
//   y[t, n] = sx[t] * sw[n] * sum_k x[t, k] w[n, k]
// The sum is exact in int32 (widths are bounded for that), so its order, and with it how
// the work is split, never changes a result; it becomes fp32 once (exact below 2^24, half
// an fp32 ulp above), is scaled in fp32 and rounded once to the output type.
#include "moe_dense.h"

namespace moe {

// sx * sw * acc in fp32
__device__ __forceinline__ float i8_scaled(int acc, float sx, float sw) { return float(acc) * sx * sw; }

// Four consecutive outputs of one row (n .. n+3; `vec`: rows are 16-byte aligned, N % 8 == 0).
template <typename TO>
__device__ __forceinline__ void store_out4(TO* y, const TO* res, int64_t row_off, int n, int N,
                                           bool vec, float (&v)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (res && n + r < N) v[r] += to_f32<TO>(res[row_off + n + r]);
  if (vec) {
    if (n >= N) return;
    if constexpr (sizeof(TO) == 4) {
      *reinterpret_cast<float4*>(y + row_off + n) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(y + row_off + n) =
          make_uint2(uint32_t(f32_to_bf16(v[0])) | (uint32_t(f32_to_bf16(v[1])) << 16),
                     uint32_t(f32_to_bf16(v[2])) | (uint32_t(f32_to_bf16(v[3])) << 16));
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < N) y[row_off + n + r] = from_f32<TO>(v[r]);
}

// Few rows: bound by the weight stream.  A workgroup of eight waves owns 16 output columns
// (of both matrices when gated) and 16 * TB tokens; the waves split K in units of 128 bytes
// and meet in LDS.  Weights are the MFMA's A operand and tokens its B operand, both loaded
// from global memory straight into the registers the matrix core reads: lane l holds row
// l % 16 and 32 contiguous bytes of a unit at (l / 16) * 32, as two k-slots of a 16x16x64
// step (which k an MFMA slot stands for is free as long as both operands agree), so a row's
// unit is one 128-byte line.  Two units per wave are in flight beside the two in use.
// grid = (ceil(N / 16), ceil(T / (16 TB))), block = 512.
template <typename TO, int TB, bool GLU>
__global__ __launch_bounds__(512) void k_i8_few(const int8_t* __restrict__ x,
                                                const float* __restrict__ sx,
                                                const int8_t* __restrict__ w,
                                                const float* __restrict__ sw,
                                                const int8_t* __restrict__ wu,
                                                const float* __restrict__ su, const TO* res, TO* y,
                                                int64_t T, int K, int N, bool vec) {
  constexpr int NW = 8, NA = GLU ? 2 : 1;
  __shared__ i32x4 part[NW][NA * TB][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int64_t t0 = int64_t(blockIdx.y) * (16 * TB);
  const int64_t nrow = int64_t(min(n0 + r16, N - 1)) * K;   // rows past the end: the last one,
  const int8_t* wp[NA];                                      // computed and not stored
  wp[0] = w + nrow;
  if (GLU) wp[NA - 1] = wu + nrow;
  const int8_t* xp[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) xp[b] = x + min<int64_t>(t0 + 16 * b + r16, T - 1) * K;

  i32x4 acc[NA][TB];
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[a][b] = i32x4{0, 0, 0, 0};

  struct Unit { i32x4 a[NA][2], b[TB][2]; };
  const int nu = (K + 127) >> 7;
  auto load = [&](int u, Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = u * 128 + q * 32 + h * 16;
      const int ko = min(k, K - 16);               // chunks past K: a valid address, x as zeros
#pragma unroll
      for (int a = 0; a < NA; ++a) f.a[a][h] = *reinterpret_cast<const i32x4*>(wp[a] + ko);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        f.b[b][h] = *reinterpret_cast<const i32x4*>(xp[b] + ko);
        if (k >= K) f.b[b][h] = i32x4{0, 0, 0, 0};
      }
    }
  };
  auto mul = [&](const Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[a][h], f.b[b][h], acc[a][b], 0, 0, 0);
  };
  Unit f0, f1;
  int u = wv;
  if (u < nu) load(u, f0);
  for (; u < nu; u += 2 * NW) {
    if (u + NW < nu) load(u + NW, f1);
    mul(f0);
    if (u + 2 * NW < nu) load(u + 2 * NW, f0);
    if (u + NW < nu) mul(f1);
  }

#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int b = 0; b < TB; ++b) part[wv][a * TB + b][lane] = acc[a][b];
  __syncthreads();
  // one thread per four outputs: columns n .. n+3 of token t
  for (int e = threadIdx.x; e < TB * 64; e += 512) {
    const int b = e >> 6, l = e & 63;
    i32x4 s[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      s[a] = part[0][a * TB + b][l];
#pragma unroll
      for (int i = 1; i < NW; ++i) s[a] += part[i][a * TB + b][l];
    }
    const int64_t t = t0 + 16 * b + (l & 15);
    const int n = n0 + 4 * (l >> 4);
    if (t >= T) continue;
    const float st = sx[t];
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nr = min(n + r, N - 1);
      v[r] = i8_scaled(s[0][r], st, sw[nr]);
      if (GLU) v[r] = silu(v[r]) * i8_scaled(s[NA - 1][r], st, su[nr]);
    }
    store_out4<TO>(y, res, t * N, n, N, vec, v);
  }
}

template <typename TO, bool GLU>
static int launch_few(const I8Product& p, bool vec, hipStream_t st) {
  const int tb = p.T <= 16 ? 1 : p.T <= 32 ? 2 : 4;
  const int64_t gy = (p.T + 16 * tb - 1) / (16 * tb);
  auto go = [&](auto kern) {
    // the second grid dimension ends at 65535: longer batches go in slices of rows
    for (int64_t y0 = 0; y0 < gy; y0 += 65535) {
      const int64_t t0 = y0 * 16 * tb, rows = std::min<int64_t>(p.T - t0, int64_t(65535) * 16 * tb);
      hipLaunchKernelGGL(kern, dim3(unsigned((p.N + 15) / 16), unsigned(std::min<int64_t>(gy - y0, 65535))),
                         dim3(512), 0, st, p.x + t0 * p.K, p.sx + t0, p.w, p.sw, p.w_up, p.s_up,
                         p.res ? static_cast<const TO*>(p.res) + t0 * p.N : nullptr,
                         static_cast<TO*>(p.y) + t0 * p.N, rows, p.K, p.N, vec);
    }
  };
  if (tb == 1) go(k_i8_few<TO, 1, GLU>);
  else if (tb == 2) go(k_i8_few<TO, 2, GLU>);
  else go(k_i8_few<TO, 4, GLU>);
  return check_launch();
}

int launch_i8_product(const I8Product& p, hipStream_t st) {
  auto aligned = [](const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15) == 0; };
  const bool vec = p.N % 8 == 0 && aligned(p.y) && (!p.res || aligned(p.res));
  if (p.out == MOE_F32)
    return p.w_up ? launch_few<float, true>(p, vec, st) : launch_few<float, false>(p, vec, st);
  return p.w_up ? launch_few<bf16_t, true>(p, vec, st) : launch_few<bf16_t, false>(p, vec, st);
}

}  // namespace moe
