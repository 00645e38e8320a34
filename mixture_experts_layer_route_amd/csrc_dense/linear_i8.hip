// Products of 8-bit integer rows and 8-bit integer weights with a scale per token and per
// output channel, alone (k_i8_few<..., false>) or as the gated pair h = silu(g) * u.
//   y[t, n] = sx[t] * sw[n] * sum_k x[t, k] w[n, k]
// The sum is exact in int32 (widths are bounded for that), so its order, and with it how
// the work is split, never changes a result; it becomes fp32 once (exact below 2^24, half
// an fp32 ulp above), is scaled in fp32 and rounded once to the output type.
#include "gemm_common.h"
#include "moe_dense.h"

namespace moe {

// sx * sw * acc in fp32
__device__ __forceinline__ float i8_scaled(int acc, float sx, float sw) { return float(acc) * sx * sw; }

// Four consecutive outputs of one row (n .. n+3; `vec`: rows are 16-byte aligned, N % 8 == 0).
template <typename TO>
__device__ __forceinline__ void store_out4(TO* y, int64_t row_off, int n, int N, bool vec,
                                           float4 v) {
  if (vec) {
    if (n >= N) return;
    if constexpr (sizeof(TO) == 4) {
      *reinterpret_cast<float4*>(y + row_off + n) = v;
    } else {
      *reinterpret_cast<uint2*>(y + row_off + n) =
          make_uint2(uint32_t(f32_to_bf16(v.x)) | (uint32_t(f32_to_bf16(v.y)) << 16),
                     uint32_t(f32_to_bf16(v.z)) | (uint32_t(f32_to_bf16(v.w)) << 16));
    }
    return;
  }
  if (n < N) y[row_off + n] = from_f32<TO>(v.x);
  if (n + 1 < N) y[row_off + n + 1] = from_f32<TO>(v.y);
  if (n + 2 < N) y[row_off + n + 2] = from_f32<TO>(v.z);
  if (n + 3 < N) y[row_off + n + 3] = from_f32<TO>(v.w);
}

// What a kernel of this file reads and writes.  One argument by value: on the host a launch
// costs about 0.1 us per kernel argument (2.9 us for this struct, 3.9 us for twelve arguments),
// which is what the smallest calls are made of.
struct I8Args {
  const int8_t* x;         // [T, K] codes and
  const float* sx;         // [T] scales (unless the kernel makes them itself)
  const int8_t* w;         // [N, K], [N]
  const float* sw;
  const int8_t* wu;        // the up matrix of a gated product
  const float* su;
  const void* res;         // [T, N] or null
  void* y;                 // [T, N]
  int64_t T;
  int K, N;
  int mtiles, ntiles;      // tiled kernel
  int vec;                 // rows of y and res are 16-byte aligned and N % 8 == 0
  // sources of the kernels that make their own codes
  const void* rows;        // kNorm: [T, K] activation rows; kQuant: h, fp32 [T, K]
  const void* gamma;       // kNorm: [K]
  float eps;
  float* hmax;             // [T, groups of columns]: largest |h| of a group, out (kNorm: of 16;
                           // h16_t: of 32) or in (kQuant: of 16)
};

// Output of a gated product that goes on to be quantised: int16 codes with one fp32 maximum per
// row and 32 columns, h = code * max / 32767.  Half the bytes of fp32, and an error of at most
// 0.5 / 32767 of the group's maximum, 0.002 of a step of the int8 codes made from it (h in bf16
// moved 3% of those codes).
struct h16_t { int16_t code; };

// Where a few-row kernel's token codes come from: memory; or made by every workgroup for
// itself in LDS, from activation rows (RMSNorm in front) or from the fp32 h of the gated product.
enum FewSrc { kCodes, kNorm, kQuant };

// LDS row stride of the codes: 16 tokens' equal chunks fall on 16 different bank groups
// (a row is a whole number of 256-byte bank lines for the usual widths).
__host__ __device__ inline int few_stride(int K) { return (K + 255) / 256 * 256 + 16; }

// RMSNorm and int8 codes of up to eight rows in LDS, by the definitions of k_norm_quant: wave wv
// has row wv, four chunks of 8 elements per lane (K <= 2048).  load() only issues loads, so that
// the weights' can follow before the first value is waited for.
template <typename TA>
struct FewNorm {
  static constexpr int NCH = 4;
  Chunk8<TA> x[NCH], g[NCH];
  __device__ __forceinline__ void load(const I8Args& a, int lane, int wv) {
    if (wv >= a.T) return;                   // uniform over the wave
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = j * 64 + lane;
      if (c < a.K / 8) {
        x[j].load(static_cast<const TA*>(a.rows) + int64_t(wv) * a.K + c * 8);
        g[j].load(static_cast<const TA*>(a.gamma) + c * 8);
      }
    }
  }
  __device__ __forceinline__ void store(const I8Args& a, int lane, int wv, int8_t* codes, float* sx) {
    if (wv >= a.T) return;
    float v[NCH][8], ss = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      if (j * 64 + lane < a.K / 8) {
        x[j].get(v[j]);
        float sj = v[j][0] * v[j][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) sj = fmaf(v[j][e], v[j][e], sj);
        ss += sj;
      }
    }
    const float rinv = inv_rms(wave_sum(ss), a.K, a.eps);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
      if (j * 64 + lane < a.K / 8) {
        float gv[8];
        g[j].get(gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[j][e] = v[j][e] * rinv * gv[e];
          m = nmax(m, fabsf(v[j][e]));
        }
      }
    const float scale = i8_scale(wave_nmax(m));
    if (lane == 0) sx[wv] = scale;
    const Divider by(scale);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = j * 64 + lane;
      if (c < a.K / 8) *reinterpret_cast<uint2*>(codes + wv * few_stride(a.K) + c * 8) = i8x8(v[j], by);
    }
  }
};

// int8 codes of up to eight rows of h in LDS: the 8 waves share the rows (all eight on one row,
// four on each of two, two on each of four, one each beyond).  A row's largest value comes from
// its tiles' maxima, so h is read once; a lane's first chunks and maxima are on their way before
// the weights, the rest comes in groups, a round trip each.
struct FewQuant {
  static constexpr int PRE = 4, HM = 6;
  Chunk8<float> h[PRE];
  float hm[HM];
  int wpr, t;
  __device__ __forceinline__ void group(const I8Args& a, int c0) {
#pragma unroll
    for (int j = 0; j < PRE; ++j) {
      const int c = c0 + j * 64 * wpr;
      if (c < a.K / 8) h[j].load(static_cast<const float*>(a.rows) + int64_t(t) * a.K + c * 8);
    }
  }
  __device__ __forceinline__ void load(const I8Args& a, int lane, int wv) {
    wpr = a.T == 1 ? 8 : a.T == 2 ? 4 : a.T <= 4 ? 2 : 1;
    t = wv / wpr;
    if (t >= a.T) return;                    // uniform over the wave
    const int nt = (a.K + 15) / 16;
#pragma unroll
    for (int j = 0; j < HM; ++j) hm[j] = a.hmax[int64_t(t) * nt + min(j * 64 + lane, nt - 1)];
    group(a, (wv % wpr) * 64 + lane);
  }
  __device__ __forceinline__ void store(const I8Args& a, int lane, int wv, int8_t* codes, float* sx) {
    if (t >= a.T) return;
    const int nt = (a.K + 15) / 16;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < HM; ++j) m = nmax(m, hm[j]);
    for (int c = HM * 64 + lane; c < nt; c += 64) m = nmax(m, a.hmax[int64_t(t) * nt + c]);
    const float scale = i8_scale(wave_nmax(m));
    if (lane == 0) sx[t] = scale;            // (the waves of a row write the same value)
    const Divider by(scale);
    int8_t* const row = codes + t * few_stride(a.K);
    const int step = PRE * 64 * wpr;
    for (int c0 = (wv % wpr) * 64 + lane;;) {
#pragma unroll
      for (int j = 0; j < PRE; ++j) {
        const int c = c0 + j * 64 * wpr;
        if (c < a.K / 8) {
          float v[8];
          h[j].get(v);
          *reinterpret_cast<uint2*>(row + c * 8) = i8x8(v, by);
        }
      }
      c0 += step;
      if (c0 - lane >= a.K / 8) break;       // uniform over the wave
      group(a, c0);
    }
  }
};
struct FewNone {
  __device__ __forceinline__ void load(const I8Args&, int, int) {}
  __device__ __forceinline__ void store(const I8Args&, int, int, int8_t*, float*) {}
};

// Few rows: bound by the weight stream.  A workgroup of eight waves owns 16 output columns
// (of both matrices when gated) of every token; the waves split K in units of 128 bytes
// and meet in LDS.  Weights are the MFMA's A operand and tokens its B operand, weights (and
// codes that lie in memory) loaded straight into the registers the matrix core reads: lane l
// holds row l % 16 and 32 contiguous bytes of a unit at (l / 16) * 32, as two k-slots of a
// 16x16x64 step (which k an MFMA slot stands for is free as long as both operands agree), so a
// row's unit is one 128-byte line.  Two units per wave are in flight while codes are made and
// beside the two in use.
// T <= 16 TB (<= 8 unless kCodes); grid = ceil(N / 16), block = 512, dynamic LDS = T *
// few_stride(K) unless kCodes.  At most 128 registers, so that two workgroups share a CU: a grid is
// often a little over one per CU.
template <typename TO, int TB, bool GLU, FewSrc SRC, class Make>
__global__ __launch_bounds__(512, 4) void k_i8_few(I8Args a) {
  constexpr int NW = 8, NA = GLU ? 2 : 1;
  __shared__ i32x4 part[NW][NA * TB][64];
  __shared__ float own_sx[8];
  extern __shared__ __align__(16) int8_t own_codes[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int K = a.K, N = a.N;
  const int T = int(a.T);
  const int64_t nrow = int64_t(min(n0 + r16, N - 1)) * K;   // rows past the end: the last one,
  const int8_t* wp[NA];                                      // computed and not stored
  wp[0] = a.w + nrow;
  if (GLU) wp[NA - 1] = a.wu + nrow;
  const int8_t* xp[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    const int t = min(16 * b + r16, T - 1);
    xp[b] = SRC == kCodes ? a.x + int64_t(t) * K : own_codes + t * few_stride(K);
  }

  i32x4 acc[NA][TB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[i][b] = i32x4{0, 0, 0, 0};

  struct Unit { i32x4 w[NA][2], x[TB][2]; };
  const int nu = (K + 127) >> 7;
  auto load_w = [&](int u, Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ko = min(u * 128 + q * 32 + h * 16, K - 16);   // chunks past K: a valid address
#pragma unroll
      for (int i = 0; i < NA; ++i) f.w[i][h] = *reinterpret_cast<const i32x4*>(wp[i] + ko);
    }
  };
  auto load_x = [&](int u, Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = u * 128 + q * 32 + h * 16;
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        f.x[b][h] = *reinterpret_cast<const i32x4*>(xp[b] + min(k, K - 16));
        if (k >= K) f.x[b][h] = i32x4{0, 0, 0, 0};             // ... that counts as zero
      }
    }
  };
  auto mul = [&](const Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int b = 0; b < TB; ++b)
          acc[i][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[i][h], f.x[b][h], acc[i][b], 0, 0, 0);
  };
  // What the end needs of scales and residual follows the first weights: after the sums it would
  // be one more round trip to cold memory (layer of one token, down product 6.4 against 5.9 us),
  // before the token rows it would delay their codes.  With the norm in front there are no
  // registers for it (9.3 us with, 7.6 without).
  const int ob = min(wv, TB - 1), on = n0 + 4 * q, ot = 16 * ob + r16;
  float es0[4], es1[4] = {0.f, 0.f, 0.f, 0.f}, er[4] = {0.f, 0.f, 0.f, 0.f}, est = 0.f;
  auto load_end = [&] {
    if (wv >= TB) return;
    if (SRC == kCodes) est = a.sx[min(ot, T - 1)];
    const TO* const res = GLU ? nullptr : static_cast<const TO*>(a.res);
    const int64_t rrow = int64_t(min(ot, T - 1)) * N;
    // (four statements: as a loop the arrays went to scratch memory for fp32 outputs)
    auto column = [&](int r, float& s0, float& s1, float& e) {
      const int nr = min(on + r, N - 1);
      s0 = a.sw[nr];
      if (GLU) s1 = a.su[nr];
      if (res) e = to_f32<TO>(res[rrow + nr]);
    };
    column(0, es0[0], es1[0], er[0]);
    column(1, es0[1], es1[1], er[1]);
    column(2, es0[2], es1[2], er[2]);
    column(3, es0[3], es1[3], er[3]);
  };
  Unit f0, f1;
  int u = wv;
  Make make;
  make.load(a, lane, wv);
  if (u < nu) load_w(u, f0);
  if (SRC == kCodes) {
    if (u < nu) load_x(u, f0);
    load_end();
  } else {
    if (u + NW < nu) load_w(u + NW, f1);
    if (SRC != kNorm) load_end();
    make.store(a, lane, wv, own_codes, own_sx);
    __syncthreads();
  }
  for (bool first = true; u < nu; u += 2 * NW, first = false) {
    if (SRC != kCodes) load_x(u, f0);
    if (u + NW < nu) {
      if (SRC == kCodes || !first) load_w(u + NW, f1);
      if (SRC == kCodes) load_x(u + NW, f1);
    }
    mul(f0);
    if (u + 2 * NW < nu) {
      load_w(u + 2 * NW, f0);
      if (SRC == kCodes) load_x(u + 2 * NW, f0);
    }
    if (u + NW < nu) {
      if (SRC != kCodes) load_x(u + NW, f1);
      mul(f1);
    }
  }

#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int b = 0; b < TB; ++b) part[wv][i * TB + b][lane] = acc[i][b];
  __syncthreads();
  // a wave per 16 tokens, a thread per four outputs: columns n .. n + 3 of token t
  if (wv >= TB) return;
  if (SRC == kNorm) load_end();
  const int b = wv, n = on, t = ot;
  i32x4 s[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    s[i] = part[0][i * TB + b][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) s[i] += part[k][i * TB + b][lane];
  }
  const float st = SRC == kCodes ? est : own_sx[min(t, T - 1)];
  float v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] = i8_scaled(s[0][r], st, es0[r]);
    if (GLU) v[r] = silu(v[r]) * i8_scaled(s[NA - 1][r], st, es1[r]);
    if (!GLU) v[r] += er[r];                 // (zeros without a residual)
  }
  if (SRC == kNorm) {
    float m = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) m = nmax(m, fabsf(v[r]));
    m = nmax(m, __shfl_xor(m, 16));
    m = nmax(m, __shfl_xor(m, 32));
    if (q == 0 && t < T) a.hmax[int64_t(t) * gridDim.x + blockIdx.x] = m;
  }
  if (t < T)
    store_out4<TO>(static_cast<TO*>(a.y), int64_t(t) * N, n, N, a.vec,
                   make_float4(v[0], v[1], v[2], v[3]));
}

// 16-byte chunks of the tile's LDS rows are XOR-swizzled so that the 16 consecutive rows one
// ds_read_b128 serves together at one chunk lie in 16 different 16-byte slots of a bank line.
template <int BK> __device__ __forceinline__ int i8_swz(int row) {
  static_assert(BK == 128 || BK == 256, "a row is half a bank line or a whole one");
  return BK == 128 ? (row >> 1) & 7 : row & 15;
}

// Tile of a workgroup: workgroup b runs on XCD b % 8, every XCD takes one contiguous run
// of the tiles in an order that walks GM token tiles per weight tile, so that the tiles in flight
// on an XCD share rows and weights in its L2.
__device__ __forceinline__ bool i8_tile_item(int mtiles, int ntiles, int& mt, int& nt) {
  constexpr int GM = 4;     // (2 and 8 measured alike)
  const int n = mtiles * ntiles, per = (n + 7) >> 3;
  const int j = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
  if (int(blockIdx.x >> 3) >= per || j >= n) return false;
  const int band = j / (GM * ntiles), first = band * GM;
  const int rows = min(GM, mtiles - first), in = j - band * GM * ntiles;
  mt = first + in % rows;
  nt = in / rows;
  return true;
}

// A wave's accumulators -> outputs.  A lane holds four consecutive columns of one token per
// block (for a gated product the gate's and the up's), so the arithmetic is done there; the
// results then pass through a 32-token piece of LDS that only this wave uses, to leave as 16
// bytes per lane, contiguous over the lanes.  ST is the type they are staged in: the output's
// own, or fp32 where a residual is still to be added before the rounding.
// sx, sw: the scales of the wave's tokens and weight rows, in LDS.
template <typename TO, typename ST, bool GLU, class C>
__device__ __forceinline__ void i8_epilogue(unsigned char* stg, const i32x4 (&acc)[C::FN][C::FM],
                                            const I8Args& a, int64_t tw, int nw, int lane,
                                            const float* sx, const float* sw) {
  constexpr bool H16 = std::is_same<TO, h16_t>::value;
  constexpr int FO = GLU ? C::FN / 2 : C::FN, OC = FO * 16;   // output blocks and columns
  constexpr int EPL = sizeof(ST) == 4 && sizeof(TO) == 4 ? 4 : 8;   // elements a lane leaves with
  constexpr int LPR = OC / EPL, RPP = 64 / LPR;               // lanes per row, rows per pass
  constexpr int RS = OC * sizeof(ST) + 16;                    // bytes per staged row
  const int64_t T = a.T;
  const int N = a.N;
  const int l16 = lane & 15, q = lane >> 4;
  float s0[FO][4], s1[FO][4];
#pragma unroll
  for (int f = 0; f < FO; ++f)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s0[f][r] = sw[f * 16 + 4 * q + r];
      s1[f][r] = GLU ? sw[OC + f * 16 + 4 * q + r] : 0.f;
    }
  const int ce = (lane % LPR) * EPL, n = nw + ce;
  // the residual of a piece is loaded a piece ahead (y may be the residual itself, so the
  // compiler could not move a load over the stores before it)
  constexpr int PP = 32 / RPP;                                // passes per piece
  constexpr bool RES = sizeof(ST) == 4 && !GLU;
  uint4 rb[2][RES ? PP : 1];
  auto load_res = [&](int mp, uint4 (&r)[RES ? PP : 1]) {
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      const int64_t t = min<int64_t>(tw + mp * 32 + p * RPP + lane / LPR, T - 1);
      r[p] = *reinterpret_cast<const uint4*>(static_cast<const TO*>(a.res) + t * N + min(n, N - EPL));
    }
  };
  const bool fast_res = RES && a.res && a.vec;
  if constexpr (RES) {
    if (fast_res) load_res(0, rb[0]);
  }
#pragma unroll
  for (int mp = 0; mp < C::FM / 2; ++mp) {
    if constexpr (RES) {
      if (fast_res && mp + 1 < C::FM / 2) load_res(mp + 1, rb[(mp + 1) & 1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int m = 2 * mp + e;
      const float ts = sx[m * 16 + l16];
      float v[FO][4];
#pragma unroll
      for (int f = 0; f < FO; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[f][r] = i8_scaled(acc[f][m][r], ts, s0[f][r]);
          if (GLU) {
            const float u = i8_scaled(acc[FO + f][m][r], ts, s1[f][r]);
            v[f][r] = (sizeof(TO) == 4 ? silu(v[f][r]) : silu16(v[f][r])) * u;
          }
        }
      unsigned char* const row = stg + (16 * e + l16) * RS + 4 * q * sizeof(ST);
      if constexpr (H16) {
        // the wave's 32 columns are one group; four lanes hold a token's part of it
        static_assert(GLU && OC == 32, "groups of 32 columns");
        float mx = 0.f;
#pragma unroll
        for (int f = 0; f < FO; ++f)
          if (nw + f * 16 < N) {                         // (N is a multiple of 16 here)
#pragma unroll
            for (int r = 0; r < 4; ++r) mx = nmax(mx, fabsf(v[f][r]));
          }
        mx = nmax(mx, __shfl_xor(mx, 16));
        mx = nmax(mx, __shfl_xor(mx, 32));
        const int64_t t = tw + m * 16 + l16;
        if (q == 0 && t < T && nw < N) a.hmax[t * ((N + 31) / 32) + nw / 32] = mx;
        const float up = mx >= 1.17549435e-38f ? 32767.0f / mx : 0.0f;
#pragma unroll
        for (int f = 0; f < FO; ++f) {
          uint32_t w[2];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            w[r] = (uint32_t(int(rintf(v[f][2 * r] * up))) & 0xFFFFu) |
                   (uint32_t(int(rintf(v[f][2 * r + 1] * up))) << 16);
          *reinterpret_cast<uint2*>(row + f * 32) = make_uint2(w[0], w[1]);
        }
      } else if constexpr (sizeof(ST) == 4) {
#pragma unroll
        for (int f = 0; f < FO; ++f)
          *reinterpret_cast<float4*>(row + f * 64) = make_float4(v[f][0], v[f][1], v[f][2], v[f][3]);
      } else {
#pragma unroll
        for (int f = 0; f < FO; ++f)
          *reinterpret_cast<uint2*>(row + f * 32) =
              make_uint2(uint32_t(f32_to_bf16(v[f][0])) | (uint32_t(f32_to_bf16(v[f][1])) << 16),
                         uint32_t(f32_to_bf16(v[f][2])) | (uint32_t(f32_to_bf16(v[f][3])) << 16));
      }
    }
#pragma unroll
    for (int p = 0; p < 32 / RPP; ++p) {
      const int row = p * RPP + lane / LPR;
      const int64_t t = tw + mp * 32 + row;
      const unsigned char* const from = stg + row * RS + ce * sizeof(ST);
      if (t >= T || n >= N) continue;
      const int64_t at = t * N + n;
      if constexpr (sizeof(ST) == 2) {
        const uint4 o = *reinterpret_cast<const uint4*>(from);
        if (a.vec) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at) = o;
        } else {
          const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < N) static_cast<uint16_t*>(a.y)[at + i] = uint16_t(w[i / 2] >> (16 * (i % 2)));
        }
      } else {
        const TO* const res = static_cast<const TO*>(a.res);
        TO* const y = static_cast<TO*>(a.y);
        float v[EPL];
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
          const float4 o = *reinterpret_cast<const float4*>(from + 16 * i);
          v[4 * i] = o.x; v[4 * i + 1] = o.y; v[4 * i + 2] = o.z; v[4 * i + 3] = o.w;
        }
        if (a.vec) {
          if constexpr (EPL == 4) {
            if constexpr (RES) {
              if (fast_res) {
                const float4 r = __builtin_bit_cast(float4, rb[mp & 1][p]);
                v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
              }
            }
            *reinterpret_cast<float4*>(y + at) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            Chunk8<TO> c;
            c.v = rb[mp & 1][p];
            float r[8];
            c.get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
            store8(y + at, v);
          }
        } else {
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (n + i < N) y[at + i] = from_f32<TO>(res ? v[i] + to_f32<TO>(res[at + i]) : v[i]);
        }
      }
    }
  }
}

// Geometry of the tiled kernel: BM tokens x BN weight rows per workgroup (gated: BN / 2 columns
// of h, each with its gate and its up row), NWM x NWN wave positions, K slabs of BK bytes in a
// ring of S; at each position KW waves share the slab's K steps (small tiles: more loads in
// flight per tile) and add their sums at the end.
template <int BM_, int BN_, int NWM_, int NWN_, int BK_, int S_, int KW_ = 1>
struct I8Tile {
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, BK = BK_, S = S_, KW = KW_;
  static constexpr int NP = NWM * NWN, NW = NP * KW, TM = BM / NWM, TN = BN / NWN;   // a wave's part
  static constexpr int FM = TM / 16, FN = TN / 16, FH = FM / 2;        // 16x16 blocks of it
  static constexpr int KS = BK / 64 / KW;                              // MFMA steps per slab and wave
  static constexpr int CPR = BK / 16;                                  // 16-byte chunks per row
  // fragments of two whole slabs fit in registers beside the sums: phases are slabs
  static constexpr bool WHOLE = 4 * (FM * FN + 2 * KS * (FM + FN)) <= 144;
  static constexpr int SLAB = (BM + BN) * BK;                          // bytes
  static constexpr int L = SLAB / 1024 / NW;                           // loads per lane and slab
  static constexpr int STG = 32 * (TN * 4 + 16);                       // epilogue bytes per wave
  static constexpr int RED = FM * FN * 1024;                           // a wave's sums
  static constexpr int END = NP * (STG > (KW - 1) * RED ? STG : (KW - 1) * RED);
  static constexpr int RING = S * SLAB > END ? S * SLAB : END;
  static constexpr int LDS = RING + (BM + BN) * 4;                     // + the tile's scales
  static_assert(L * NW * 1024 == SLAB && S >= 2 && FM % 2 == 0 && KS >= 1 && LDS <= 163840,
                "tile geometry");
};

// Address of the scale of row r of a tile's slab (tokens first, then weight rows in slab order).
template <bool GLU, class C>
__device__ __forceinline__ const float* i8_scale_of(const I8Args& a, int r, int64_t t0, int n0) {
  constexpr int OC = GLU ? C::TN / 2 : C::TN;
  if (r < C::BM) return a.sx + min<int64_t>(t0 + r, a.T - 1);
  const int q = r - C::BM, s = q % C::TN;
  const int n = min(GLU ? n0 + q / C::TN * OC + s % OC : n0 + q, a.N - 1);
  return (GLU && s >= OC ? a.su : a.sw) + n;
}

// All but the N newest loads of this wave have landed and its LDS reads are done, then the
// workgroup meets.  The fences keep the compiler from moving LDS accesses across either.
template <int N>
__device__ __forceinline__ void i8_slab_sync() {
  asm volatile("" ::: "memory");
  wait_vm_lgkm0<N>();
  block_sync_nowait();
}

// The tiled product.  Tokens are the MFMA's B operand and weights its A operand, so that a
// lane ends with four consecutive columns of one token; 16x16x64 steps, because at this card's
// power limit they run faster on data than 32x32x32 (register-only loop, all CUs: 4.2e15
// against 3.5e15 op/s; 4.8e15 for both on zeros).
// Both operands move global -> LDS by direct 16-byte loads, a 128-byte line per row and slab
// (with 64-byte slabs the loads alone ran at 28 instead of 40 bytes per clock and CU).  A slab's
// slot is refilled as soon as the last fragments of it are in registers, half a phase before
// the slab's end, which is also where the one barrier per slab is; each phase's fragments are
// read during the phase before.
// 8192 x 4096 x 8192: 221 us, 2.49e15 op/s; 8192 x 8192 x 2048: 109 us, 2.52e15; gated 4096 x
// 2048 x 8192: 129 us, 2.13e15.  A persistent form that loads the next tile's first slabs while the
// results leave was no faster (220 us for the first): on data the card's power bounds the rate.
template <typename TO, bool GLU, class C>
__global__ __launch_bounds__(C::NW * 64) void k_i8_tile(I8Args a) {
  constexpr int OC = GLU ? C::TN / 2 : C::TN;              // output columns per wave
  __shared__ __align__(16) unsigned char lds[C::LDS];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int pos = wv % C::NP, kw = wv / C::NP;
  const int wm = pos / C::NWN, wn = pos % C::NWN;
  const int64_t T = a.T;
  const int K = a.K, N = a.N;

  int mt, nt;
  if (!i8_tile_item(a.mtiles, a.ntiles, mt, nt)) return;
  const int64_t t0 = int64_t(mt) * C::BM;
  const int n0 = nt * (GLU ? C::BN / 2 : C::BN);

  // one load instruction of a wave fills 64 / CPR rows; lane L writes chunk position L % CPR, of
  // rows that are equal modulo the swizzle's period in all of its loads
  constexpr int RPL = 64 / C::CPR;
  static_assert(C::NW * RPL % 16 == 0, "one chunk for all loads of a lane");
  const int kc = ((lane % C::CPR) ^ i8_swz<C::BK>(wv * RPL + lane / C::CPR)) * 16;
  const int8_t* src[C::L];
#pragma unroll
  for (int i = 0; i < C::L; ++i) {
    const int r = (wv + C::NW * i) * RPL + lane / C::CPR;
    if (r < C::BM) {
      src[i] = a.x + min<int64_t>(t0 + r, T - 1) * K;
    } else {
      const int q = r - C::BM;
      if (GLU) {
        const int s = q % C::TN;
        const int n = min(n0 + q / C::TN * OC + s % OC, N - 1);
        src[i] = (s < OC ? a.w : a.wu) + int64_t(n) * K;
      } else {
        src[i] = a.w + int64_t(min(n0 + q, N - 1)) * K;
      }
    }
  }
  // the tile's scales, tokens then weight rows, by loads older than every slab's
  float* const scales = reinterpret_cast<float*>(lds + C::RING);
  static_assert((C::BM + C::BN) % 32 == 0, "whole pieces of scales");
  for (int i = wv; i < (C::BM + C::BN + 63) / 64; i += C::NW) {
    const int r = i * 64 + lane;
    if (r < C::BM + C::BN) dma4(i8_scale_of<GLU, C>(a, r, t0, n0), scales + i * 64);
  }
  const int nk = (K + C::BK - 1) / C::BK;
  auto load = [&](int i, int kt, int slot) {
    dma16(src[i] + min(kt * C::BK + kc, K - 16), lds + slot * C::SLAB + (wv + C::NW * i) * 1024);
  };

  const int l16 = lane & 15, q = lane >> 4;
  int foff[C::KS];                                       // this lane's chunk of each MFMA step
#pragma unroll
  for (int s = 0; s < C::KS; ++s) foff[s] = l16 * C::BK + ((4 * (kw * C::KS + s) + q) ^ i8_swz<C::BK>(l16)) * 16;
  const unsigned char* const xrow = lds + wm * C::TM * C::BK;
  const unsigned char* const wrow = lds + (C::BM + wn * C::TN) * C::BK;
  auto read_frag = [&](const unsigned char* rows, int slot, int s, int i) {
    return *reinterpret_cast<const i32x4*>(rows + slot * C::SLAB + foff[s] + i * 16 * C::BK);
  };
  // chunks past K hold whatever lies at the clamped address: there x counts as zero
  auto past = [&](int kt, int s) { return kt * C::BK + (4 * (kw * C::KS + s) + q) * 16 >= K; };
  for (int k = 0; k < C::S; ++k)
    if (k < nk) {
#pragma unroll
      for (int i = 0; i < C::L; ++i) load(i, k, k);
    }
  i32x4 acc[C::FN][C::FM];
#pragma unroll
  for (int n = 0; n < C::FN; ++n)
#pragma unroll
    for (int m = 0; m < C::FM; ++m) acc[n][m] = i32x4{0, 0, 0, 0};
  if (nk >= C::S) i8_slab_sync<(C::S - 1) * C::L>(); else i8_slab_sync<0>();
  int slot = 0;
  using Buf0 = std::integral_constant<int, 0>;
  using Buf1 = std::integral_constant<int, 1>;
  if constexpr (C::WHOLE) {
    i32x4 fx[2][C::KS][C::FM], fw[2][C::KS][C::FN];
    auto read_slab = [&](int sl, int kt, auto buf) {
      constexpr int B = decltype(buf)::value;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
#pragma unroll
        for (int n = 0; n < C::FN; ++n) fw[B][s][n] = read_frag(wrow, sl, s, n);
#pragma unroll
        for (int m = 0; m < C::FM; ++m) fx[B][s][m] = read_frag(xrow, sl, s, m);
        if (kt == nk - 1 && past(kt, s)) {
#pragma unroll
          for (int m = 0; m < C::FM; ++m) fx[B][s][m] = i32x4{0, 0, 0, 0};
        }
      }
    };
    auto slab = [&](int kt, auto buf, auto other) {
      constexpr int B = decltype(buf)::value;
      const int next = slot + 1 == C::S ? 0 : slot + 1;
      if (kt + 1 < nk) {
        // this slab is in registers everywhere, so its slot is free, and the next one is in LDS
        if (kt + C::S <= nk) i8_slab_sync<(C::S - 2) * C::L>(); else i8_slab_sync<0>();
        if (kt + C::S < nk) {
#pragma unroll
          for (int i = 0; i < C::L; ++i) load(i, kt + C::S, slot);
        }
        read_slab(next, kt + 1, other);
      }
#pragma unroll
      for (int s = 0; s < C::KS; ++s)
#pragma unroll
        for (int m = 0; m < C::FM; ++m)
#pragma unroll
          for (int n = 0; n < C::FN; ++n)
            acc[n][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[B][s][n], fx[B][s][m], acc[n][m], 0, 0, 0);
      slot = next;
    };
    read_slab(0, 0, Buf0());
    int kt = 0;
    for (; kt + 1 < nk; kt += 2) {
      slab(kt, Buf0(), Buf1());
      slab(kt + 1, Buf1(), Buf0());
    }
    if (kt < nk) slab(kt, Buf0(), Buf1());
  } else {
    static_assert(C::KS % 2 == 0, "a slab starts and ends on the same weight buffer");
    i32x4 fx[2][C::FH], fw[2][C::FN];
    auto read_w = [&](int sl, int s, int buf) {
#pragma unroll
      for (int n = 0; n < C::FN; ++n) fw[buf][n] = read_frag(wrow, sl, s, n);
    };
    auto read_x = [&](int sl, int s, int kt, int half) {
#pragma unroll
      for (int m = 0; m < C::FH; ++m) fx[half][m] = read_frag(xrow, sl, s, half * C::FH + m);
      if (kt == nk - 1 && past(kt, s)) {
#pragma unroll
        for (int m = 0; m < C::FH; ++m) fx[half][m] = i32x4{0, 0, 0, 0};
      }
    };
    // half of the wave's tokens; with `lk` >= 0 the loads of slab lk go out between the steps
    auto mul = [&](int half, int buf, int lk) {
      constexpr int N = C::FH * C::FN, EVERY = N / C::L;
      static_assert(EVERY >= 1 && EVERY * C::L == N, "a load every so many steps");
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int m = j / C::FN, n = j % C::FN;
        if (j % EVERY == 0 && lk >= 0) load(j / EVERY, lk, slot);
        acc[n][half * C::FH + m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            fw[buf][n], fx[half][m], acc[n][half * C::FH + m], 0, 0, 0);
      }
    };
    read_w(0, 0, 0);
    read_x(0, 0, 0, 0);
    // Every phase multiplies half of the wave's tokens by one step's weights while the next
    // phase's fragments are read.
    for (int kt = 0; kt < nk; ++kt) {
      const int next = slot + 1 == C::S ? 0 : slot + 1;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        int lk = -1;
        read_x(slot, s, kt, 1);
        mul(0, s & 1, -1);
        if (s + 1 < C::KS) {
          read_w(slot, s + 1, (s + 1) & 1);
          read_x(slot, s + 1, kt, 0);
        } else if (kt + 1 < nk) {
          // every fragment of this slab is in registers: once all waves are here its slot is
          // free, and slab kt + 1 (older than the S - 2 slabs that may still be on their way)
          // can be read
          if (kt + C::S <= nk) i8_slab_sync<(C::S - 2) * C::L>(); else i8_slab_sync<0>();
          if (kt + C::S < nk) lk = kt + C::S;
          read_w(next, 0, 0);
          read_x(next, 0, kt + 1, 0);
        }
        mul(1, s & 1, lk);
      }
      slot = next;
    }
  }
  i8_slab_sync<0>();               // the ring becomes the waves' own staging memory
  if constexpr (C::KW > 1) {
    i32x4* const red = reinterpret_cast<i32x4*>(lds) + lane;
    if (kw > 0) {
#pragma unroll
      for (int n = 0; n < C::FN; ++n)
#pragma unroll
        for (int m = 0; m < C::FM; ++m)
          red[(((kw - 1) * C::NP + pos) * C::FM * C::FN + n * C::FM + m) * 64] = acc[n][m];
    }
    __syncthreads();
    if (kw == 0) {
#pragma unroll
      for (int k = 0; k < C::KW - 1; ++k)
#pragma unroll
        for (int n = 0; n < C::FN; ++n)
#pragma unroll
          for (int m = 0; m < C::FM; ++m)
            acc[n][m] += red[((k * C::NP + pos) * C::FM * C::FN + n * C::FM + m) * 64];
    }
    __syncthreads();
    if (kw > 0) return;
  }
  auto leave = [&](auto staged) {
    i8_epilogue<TO, decltype(staged), GLU, C>(lds + pos * C::STG, acc, a, t0 + wm * C::TM,
                                              n0 + wn * OC, lane, scales + wm * C::TM,
                                              scales + C::BM + wn * C::TN);
  };
  if constexpr (sizeof(TO) == 2 && !GLU) {
    if (a.res) leave(0.f); else leave(TO());
  } else {
    leave(TO());
  }
}

static I8Args i8_args(const I8Product& p) {
  auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  I8Args a{};
  a.x = p.x; a.sx = p.sx; a.w = p.w; a.sw = p.sw; a.wu = p.w_up; a.su = p.s_up;
  a.res = p.res; a.y = p.y; a.T = p.T; a.K = p.K; a.N = p.N;
  a.vec = p.N % 8 == 0 && aligned(p.y) && (!p.res || aligned(p.res));
  return a;
}

template <typename TO, bool GLU, int TB>
static void launch_few(const I8Product& p, hipStream_t st) {
  hipLaunchKernelGGL((k_i8_few<TO, TB, GLU, kCodes, FewNone>), dim3(unsigned((p.N + 15) / 16)),
                     dim3(512), 0, st, i8_args(p));
}

template <typename TO, bool GLU, class C>
static void launch_tile(const I8Product& p, hipStream_t st, float* hmax = nullptr) {
  const int64_t mt = (p.T + C::BM - 1) / C::BM, oc = GLU ? C::BN / 2 : C::BN;
  const int64_t nt = (p.N + oc - 1) / oc;
  I8Args a = i8_args(p);
  a.mtiles = int(mt);
  a.ntiles = int(nt);
  a.hmax = hmax;
  hipLaunchKernelGGL((k_i8_tile<TO, GLU, C>), dim3(xcd_grid(mt * nt)), dim3(C::NW * 64), 0, st, a);
}

// The tiles: one workgroup per CU of 256, 128 and 64 deep (96 to 130 KB of LDS), two or three of
// the others.
using Tile256 = I8Tile<256, 256, 2, 4, 128, 2>;
using Tile128 = I8Tile<128, 128, 4, 2, 128, 3>;
using Tile64Deep = I8Tile<64, 64, 1, 2, 256, 3, 4>;
using Tile64 = I8Tile<64, 64, 2, 2, 128, 3, 2>;
using Tile32 = I8Tile<32, 64, 1, 2, 256, 3, 4>;
using Tile32Narrow = I8Tile<32, 32, 1, 1, 256, 3, 4>;

// Which kernel: the one whose estimated time (us) is least.  For a tile that is
//   (128-wide K slabs) * (tiles on the fullest CU) * (time of a slab) + (start and end) +
//   (the ends of a CU's further tiles, as far as they show),
// and at least the weight stream from memory, fitted to measurements from 1 to 8192
// tokens and widths from 512 to 32768.  Up to 16 tokens (32 without the gate) there is also the
// kernel that streams the weights past every token at once: a time per MB of weights and one per
// token for the codes that each workgroup reads for itself, on at least 256 CUs, the last round
// of workgroups counted half; widths up to 2048 have all their weights on the way from the start.
// Measured on either side of a switch (us; few rows / narrow 32x32 / 32x64): 1 x 2048 x 16384
// 7.5 / 8.0 / 7.9; 4 x 4096 x 16384 14.3 / 12.3 / 12.3; 16 x 2048 x 2048 4.2 / 5.2; 16 x 8192 x
// 8192 16.8 / 12.6 / 13.4; 16 x 1536 x 32768 13.1 / 11.6 / 10.3; 17 x 5120 x 1536 7.1 / 8.4 / 9.0;
// 32 x 5120 x 1536 8.9 / 8.4 / 9.0; 32 x 4096 x 16384 23.5 / 12.7 / 12.8; gated 4 x 1536 x 5120 6.4 /
// 6.2 / 5.9, 16 x 2048 x 1024 4.9 / 5.1 / 5.5.  64 x 5120 x 1536 narrow 8.6, 32x64 9.3, 64x64 14.4;
// 64 x 4096 x 8192 9.8, 8.8, 12.3; 48 x 2048 x 16384 11.1, 9.0, 8.4; 333 x 4112 x 1536 14.1, 14.3,
// 13.2, deep 12.2; 512 x 2048 x 2048 32x64 8.9, 64x64 8.4, deep 8.2, 128x128 13.0; 2048 x 2048 x 2048
// 64x64 18.3, deep 25.5, 128x128 14.1; 8192 x 8192 x 2048 128x128 148, 256x256 109; gated 333 x
// 1536 x 4112 64x64 14.7, 128x128 11.2, 1485 x 288 x 13584 64x64 47.0, 128x128 47.6, 256x256 36.7.
enum I8Kernel { kFew16, kFew32, kTile32Narrow, kTile32, kTile64, kTile64Deep, kTile128, kTile256 };
static I8Kernel pick_kernel(int64_t T, int K, int N, bool glu) {
  const double slabs = double((K + 127) / 128), mats = glu ? 2.0 : 1.0;
  const double mb = mats * K * N * 1e-6;                     // of weights
  auto per_cu = [&](int bm, int bn) {
    const int oc = glu ? bn / 2 : bn;
    return std::ceil(double((T + bm - 1) / bm) * double((N + oc - 1) / oc) / 256.0);
  };
  const double c32 = per_cu(32, 64), c64 = per_cu(64, 64), c128 = per_cu(128, 128);
  double least = std::max(slabs * c32 * (c32 == 1.0 ? 0.16 : 0.19) + 2.85 + 0.5 * (c32 - 1.0), mb * 0.14 + 3.2);
  I8Kernel pick = kTile32;
  auto offer = [&](I8Kernel k, double us) {
    if (us < least) {
      least = us;
      pick = k;
    }
  };
  if (per_cu(32, 32) == 1.0) offer(kTile32Narrow, std::max(slabs * 0.145 + 2.85, mb * 0.144 + 3.2));
  offer(kTile64, std::max(slabs * c64 * 0.26 + 3.3 + 0.3 * (c64 - 1.0), mb * 0.14 + 3.6));
  if (c64 == 1.0) offer(kTile64Deep, std::max(slabs * 0.20 + 3.9, mb * 0.14 + 4.0));
  offer(kTile128, slabs * (c128 == 1.0 ? 0.56 : c128 * 0.65) + 3.7 + 2.0 * (c128 - 1.0));
  offer(kTile256, per_cu(256, 256) * (slabs * 1.6 + 4.0) + 3.0);
  if (T <= 16 || (T <= 32 && !glu)) {
    const double wgs = (N + 15) / 16, rounds = std::ceil(wgs / 256.0) * 256.0;
    const double stream = 16e-6 * mats * K * (wgs <= 256.0 ? 256.0 : (wgs + rounds) / 2);
    const double start = wgs <= 256.0 && K <= 2048 ? 2.0 : 2.6;
    if (T <= 16) offer(kFew16, stream * (0.152 + 0.0034 * T / mats) + start);
    else offer(kFew32, stream * (0.145 + 0.0053 * T) + start);
  }
  return pick;
}
// (a wave of these two tiles has the 32 columns of a group)
bool glu_h16_ok(int64_t T, int K, int N) {
  const I8Kernel k = pick_kernel(T, K, N, true);
  return k == kTile128 || k == kTile256;
}

template <typename TO, bool GLU>
static int launch_product(const I8Product& p, hipStream_t st) {
  switch (pick_kernel(p.T, p.K, p.N, GLU)) {
    case kFew16: launch_few<TO, GLU, 1>(p, st); break;
    case kFew32:
      if constexpr (!GLU) launch_few<TO, GLU, 2>(p, st);
      break;
    case kTile32Narrow: launch_tile<TO, GLU, Tile32Narrow>(p, st); break;
    case kTile32: launch_tile<TO, GLU, Tile32>(p, st); break;
    case kTile64: launch_tile<TO, GLU, Tile64>(p, st); break;
    case kTile64Deep: launch_tile<TO, GLU, Tile64Deep>(p, st); break;
    case kTile128: launch_tile<TO, GLU, Tile128>(p, st); break;
    case kTile256: launch_tile<TO, GLU, Tile256>(p, st); break;
  }
  return check_launch();
}

int launch_glu_h16(const I8Product& p, float* hmax, hipStream_t st) {
  if (pick_kernel(p.T, p.K, p.N, true) == kTile128)
    launch_tile<h16_t, true, Tile128>(p, st, hmax);
  else
    launch_tile<h16_t, true, Tile256>(p, st, hmax);
  return check_launch();
}

// int8 codes and scales of rows of h held as h16_t; a workgroup per row, every value read once
// (the row's maximum comes from its groups').  grid = T, block = 256.
__global__ __launch_bounds__(256) void k_h16_codes(const int16_t* h, const float* hmax, int I,
                                                   int8_t* codes, float* scales) {
  constexpr int PRE = 4;
  __shared__ float part[4];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, n8 = I / 8, ng = (I + 31) / 32;
  const int16_t* const row = h + t * I;
  const float* const gm = hmax + t * ng;
  uint4 c[PRE];
  float m32[PRE];
#pragma unroll
  for (int j = 0; j < PRE; ++j) {
    const int k = min(j * 256 + tid, n8 - 1);
    c[j] = *reinterpret_cast<const uint4*>(row + k * 8);
    m32[j] = gm[k / 4];
  }
  float m = 0.f;
  for (int g = tid; g < ng; g += 256) m = nmax(m, gm[g]);
  m = wave_nmax(m);
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  m = nmax(nmax(part[0], part[1]), nmax(part[2], part[3]));
  const float scale = i8_scale(m);
  if (tid == 0) scales[t] = scale;
  const float step = 1.0f / (32767.0f * scale);     // codes of h16 -> codes, times the group's maximum
  auto put = [&](int k, const uint4& v, float mg) {
    const float f = mg * step;
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = int(in[i / 2] << (i % 2 ? 0 : 16)) >> 16;
      const float q = fminf(fmaxf(rintf(float(x) * f), -127.f), 127.f);
      w[i / 4] |= (uint32_t(int(q)) & 0xFFu) << (8 * (i % 4));
    }
    *reinterpret_cast<uint2*>(codes + t * I + k * 8) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int j = 0; j < PRE; ++j)
    if (j * 256 + tid < n8) put(j * 256 + tid, c[j], m32[j]);
  for (int k = PRE * 256 + tid; k < n8; k += 256)
    put(k, *reinterpret_cast<const uint4*>(row + k * 8), gm[k / 4]);
}

int launch_h16_codes(const void* h, const float* hmax, int64_t T, int I, int8_t* codes, float* scales,
                     hipStream_t st) {
  hipLaunchKernelGGL(k_h16_codes, dim3(unsigned(T)), dim3(256), 0, st, static_cast<const int16_t*>(h),
                     hmax, I, codes, scales);
  return check_launch();
}

int launch_i8_product(const I8Product& p, hipStream_t st) {
  if (p.out == MOE_F32)
    return p.w_up ? launch_product<float, true>(p, st) : launch_product<float, false>(p, st);
  return p.w_up ? launch_product<bf16_t, true>(p, st) : launch_product<bf16_t, false>(p, st);
}

// The dense layer of up to 8 tokens in two launches: norm, codes and gated product; codes of
// h, down product and residual.  Every workgroup makes the codes it needs (a few rows, from L2)
// while its first weights are on their way, as long as a wave has one row to normalise and a lane at
// most eight chunks of h (FewQuant's sharing).  Against the four launches (us, bf16,
// hidden x intermediate): 1536 x 5120 1 token 13.6 / 16.0, 4 tokens 15.1 / 16.9, 5 tokens (10
// chunks) 17.3 / 17.0; 2048 x 4096 8 tokens 15.5 / 16.2; 2048 x 8192 4 tokens 19.0 / 21.0, 5 tokens
// 22.9 / 21.3; 2048 x 16384 4 tokens 37.9 / 33.2; with 4096 x 8192 and two rows' registers per wave 4
// tokens took 33.7 / 30.7.
bool dense_few_ok(int64_t T, int H, int I) {
  const int rows = T == 1 ? 1 : T == 2 ? 2 : T <= 4 ? 4 : 8;
  return T <= 8 && H <= 2048 && rows * I <= 8 * 8 * 64 * 8;
}
size_t dense_few_hmax_bytes(int64_t T, int I) { return size_t(T) * ((I + 15) / 16) * sizeof(float); }

template <typename TA>
static int launch_dense_few_act(const DenseFew& d, hipStream_t st) {
  I8Args up{};
  up.w = d.w->w_gate; up.sw = d.w->s_gate; up.wu = d.w->w_up; up.su = d.w->s_up;
  up.y = d.h; up.T = d.T; up.K = d.H; up.N = d.I; up.vec = d.I % 8 == 0;
  up.rows = d.x; up.gamma = d.gamma; up.eps = d.eps; up.hmax = d.hmax;
  const dim3 gu(unsigned((d.I + 15) / 16)), gd(unsigned((d.H + 15) / 16));
  const size_t lu = size_t(d.T) * few_stride(d.H), ld = size_t(d.T) * few_stride(d.I);
  hipLaunchKernelGGL((k_i8_few<float, 1, true, kNorm, FewNorm<TA>>), gu, dim3(512), lu, st, up);
  MOE_TRY(check_launch());
  I8Args down{};
  down.w = d.w->w_down; down.sw = d.w->s_down; down.res = d.x; down.y = d.x_out;
  down.T = d.T; down.K = d.I; down.N = d.H; down.vec = d.H % 8 == 0;
  down.rows = d.h; down.hmax = d.hmax;
  hipLaunchKernelGGL((k_i8_few<TA, 1, false, kQuant, FewQuant>), gd, dim3(512), ld, st, down);
  return check_launch();
}

int launch_dense_few(const DenseFew& d, hipStream_t st) {
  return d.act == MOE_F32 ? launch_dense_few_act<float>(d, st) : launch_dense_few_act<bf16_t>(d, st);
}

}  // namespace moe
