// Residual add, RMSNorm and 8-bit quantisation of rows in one pass:
//   s = round(x + res);  v = s / sqrt(mean(s^2) + eps) * gamma;  out = rows or codes of v.
// Memory bound: every row is read once into registers, its statistics are reduced there and
// the result is written from the same registers, so the bytes moved are the operator's own.
#include "moe_dense.h"

namespace moe {

// One row is held by WPR waves with NCH chunks of 8 consecutive elements per lane (chunk
// c = j * 64 * WPR + position of the lane in the row's waves), so that
//   * a load is 16 bytes (bf16) or 32 bytes (fp32) per lane, contiguous over the wave;
//   * a 128-column FP8 block is one chunk of a 16-lane DPP row and a 32-column MXFP8 block
//     one chunk of a quad: their maxima need no LDS (H is a multiple of the block, so a
//     block is either all inside the row or all outside).
// WPR is 1 for batches (a wave needs no barrier), 4 or 16 where few rows have to fill the
// chip or the row is too wide for one wave's registers.
// The 8-bit codes are taken from the fp32 v, not from rows rounded to the activation type:
// one rounding instead of two.  The sum s is rounded to the activation type first, since
// that is what the residual stream keeps: the norm of a fused call is the norm of the row
// that the next layer reads back.
// x, res and x_sum may be the same memory (a lane stores only chunks it has loaded itself).
// grid = ceil(T / (4 / WPR)) blocks of 256 threads, or T blocks of 1024 for WPR = 16.
template <typename TA, int FMT, int WPR, int NCH>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 256) void k_norm_quant(NormQuant a) {
  const TA* const x = static_cast<const TA*>(a.x);
  const TA* const res = static_cast<const TA*>(a.res);
  const TA* const gamma = static_cast<const TA*>(a.gamma);
  TA* const x_sum = static_cast<TA*>(a.x_sum);
  void* const out = a.out;
  void* const scales = a.scales;
  const int64_t T = a.rows;
  const int H = a.width;
  constexpr int NW = WPR == 16 ? 16 : 4;         // waves per workgroup
  constexpr int RPB = NW / WPR;                  // rows per workgroup
  __shared__ float part[WPR == 1 ? 1 : 2 * NW];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t t = int64_t(blockIdx.x) * RPB + wv / WPR;
  if (WPR == 1 && t >= T) return;                // (other shapes have a workgroup per row)
  const int pos = (wv % WPR) * 64 + lane;
  const int n8 = H / 8;
  const int64_t base = t * H;

  float v[NCH][8];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = j * 64 * WPR + pos;
    if (c < n8) {
      load8(x + base + c * 8, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    }
  }
  if (res) {
    float r[NCH][8];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = j * 64 * WPR + pos;
      if (c < n8) load8(res + base + c * 8, r[j]);
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = j * 64 * WPR + pos;
      if (c < n8) add_store8(x_sum + base + c * 8, v[j], r[j]);   // v becomes the rounded sum
    }
  }
  if (gamma) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float sj = v[j][0] * v[j][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) sj = fmaf(v[j][i], v[j][i], sj);
      ss += sj;
    }
    ss = wave_sum(ss);
    if (WPR > 1) {
      if (lane == 0) part[wv] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) ss += part[wv / WPR * WPR + i];
    }
    const float rinv = inv_rms(ss, H, a.eps);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = j * 64 * WPR + pos;
      if (c < n8) {
        float g[8];
        load8(gamma + c * 8, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rinv * g[i];
      }
    }
  }

  float row_scale = 1.f;
  if (FMT == MOE_ROWS_I8) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = nmax(m, fabsf(v[j][i]));
    m = wave_nmax(m);
    if (WPR > 1) {
      if (lane == 0) part[NW + wv] = m;
      __syncthreads();
      m = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) m = nmax(m, part[NW + wv / WPR * WPR + i]);
    }
    row_scale = i8_scale(m);
    if (pos == 0) static_cast<float*>(scales)[t] = row_scale;
  }
  const Divider row_by(row_scale);
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = j * 64 * WPR + pos;
    const bool live = c < n8;
    const int64_t off = base + int64_t(c) * 8;
    if (FMT == MOE_ROWS_ACT) {
      if (live) store8(static_cast<TA*>(out) + off, v[j]);
    } else if (FMT == MOE_ROWS_I8) {
      if (live)
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(out) + off) = i8x8(v[j], row_by);
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = nmax(m, fabsf(v[j][i]));
      m = nmax(m, dppf<0xB1>(m));    // quad_perm [1,0,3,2]
      m = nmax(m, dppf<0x4E>(m));    // quad_perm [2,3,0,1]
      uint32_t c0, c1;
      if (FMT == MOE_ROWS_E4M3_B128) {
        m = nmax(m, dppf<0x141>(m));   // row_half_mirror
        m = nmax(m, dppf<0x140>(m));   // row_mirror
        const float s = e4m3_scale(m);
        const Divider by(s);
        c0 = e4m3x4(by(v[j][0]), by(v[j][1]), by(v[j][2]), by(v[j][3]));
        c1 = e4m3x4(by(v[j][4]), by(v[j][5]), by(v[j][6]), by(v[j][7]));
        if (live && (lane & 15) == 0) static_cast<float*>(scales)[t * (H / 128) + c / 16] = s;
      } else {
        const int X = mx_exponent(m);
        const float inv = mx_inv_scale(X);
        c0 = e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv);
        c1 = e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv);
        if (live && (lane & 3) == 0)
          static_cast<uint8_t*>(scales)[t * (H / 32) + c / 4] = m < INFINITY ? uint8_t(X + 127) : 255;
      }
      if (live) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + off) = make_uint2(c0, c1);
    }
  }
}

template <typename TA, int FMT>
static void launch_fmt(const NormQuant& q, hipStream_t st) {
  auto go = [&](auto kern, int wpr) {
    const int rpb = wpr == 1 ? 4 : 1;
    hipLaunchKernelGGL(kern, dim3(unsigned((q.rows + rpb - 1) / rpb)), dim3(wpr == 16 ? 1024 : 256),
                       0, st, q);
  };
  // A wave per row where there are rows enough to fill the chip (8 waves per CU) and its
  // registers hold one row, not two: 8192 x 2048 bf16 to int8 13.3 us against 15.9 with four
  // waves, with the residual 28.0 against 23.1; 1024 x 2048 4.0 against 3.7.
  const bool batch = q.rows >= 2048 && (!q.res || q.width <= 1024);
  const int H = q.width;
  if (H <= 512) return go(k_norm_quant<TA, FMT, 1, 1>, 1);
  if (batch && H <= 1024) return go(k_norm_quant<TA, FMT, 1, 2>, 1);
  if (batch && H <= 2048) return go(k_norm_quant<TA, FMT, 1, 4>, 1);
  if (H <= 2048) return go(k_norm_quant<TA, FMT, 4, 1>, 4);
  if (H <= 8192) return go(k_norm_quant<TA, FMT, 4, 4>, 4);
  go(k_norm_quant<TA, FMT, 16, 4>, 16);
}

template <typename TA>
static void launch_act(const NormQuant& q, hipStream_t st) {
  switch (q.format) {
    case MOE_ROWS_ACT: return launch_fmt<TA, MOE_ROWS_ACT>(q, st);
    case MOE_ROWS_I8: return launch_fmt<TA, MOE_ROWS_I8>(q, st);
    case MOE_ROWS_E4M3_B128: return launch_fmt<TA, MOE_ROWS_E4M3_B128>(q, st);
    default: return launch_fmt<TA, MOE_ROWS_MXFP8>(q, st);
  }
}

int launch_norm_quant(const NormQuant& q, hipStream_t st) {
  if (q.act == MOE_F32)
    launch_act<float>(q, st);
  else
    launch_act<bf16_t>(q, st);
  return check_launch();
}

}  // namespace moe
