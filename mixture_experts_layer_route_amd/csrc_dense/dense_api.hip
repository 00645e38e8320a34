// C ABI of the dense 8-bit operators: validation and launch sequences.  As in moe_api.hip
// every call validates its arguments before enqueuing anything, never synchronises, never
// copies to the host and never allocates.
#include "moe_dense.h"

namespace moe {

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
static size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
static int act_bytes(int act) { return act == MOE_F32 ? 4 : 2; }

static int check_norm_quant(const NormQuant& q) {
  if (q.rows < 1 || q.width < 1) return MOE_ERR_ARG;
  if (!q.x || !q.out || (q.res && !q.x_sum)) return MOE_ERR_ARG;
  if (q.format != MOE_ROWS_ACT && !q.scales) return MOE_ERR_ARG;
  if (!(q.eps >= 0.f)) return MOE_ERR_ARG;
  if (!aligned16(q.x) || !aligned16(q.res) || !aligned16(q.gamma) || !aligned16(q.x_sum) ||
      !aligned16(q.out))
    return MOE_ERR_ARG;
  if (q.format != MOE_ROWS_MXFP8 && !aligned4(q.scales)) return MOE_ERR_ARG;
  if (q.act != MOE_F32 && q.act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const int step = q.format == MOE_ROWS_ACT || q.format == MOE_ROWS_I8 ? 8
                   : q.format == MOE_ROWS_E4M3_B128                    ? 128
                   : q.format == MOE_ROWS_MXFP8                        ? 32
                                                                       : 0;
  if (!step || q.width % step || q.width > kNormMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (q.rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

static int check_product(const I8Product& p, bool glu) {
  if (p.T < 1 || p.K < 1 || p.N < 1) return MOE_ERR_ARG;
  if (!p.x || !p.sx || !p.w || !p.sw || !p.y) return MOE_ERR_ARG;
  if (glu && (!p.w_up || !p.s_up)) return MOE_ERR_ARG;
  if (!aligned16(p.x) || !aligned16(p.w) || !aligned16(p.w_up)) return MOE_ERR_ARG;
  if (!aligned4(p.sx) || !aligned4(p.sw) || !aligned4(p.s_up)) return MOE_ERR_ARG;
  if (p.out != MOE_F32 && p.out != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const uintptr_t natural = act_bytes(p.out) - 1;
  if ((reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.res)) & natural)
    return MOE_ERR_ARG;
  if (p.K % 16 || p.K > kI8MaxWidth) return MOE_ERR_UNSUPPORTED;
  if (p.T > kMaxRows || p.N > kMaxColumns || p.T * p.N > kMaxOutputs) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace of the dense layer: codes and scales of the normalised rows and of h, and h.
struct DensePlan {
  int64_t T;
  int H, I, act;
  bool few;                // up to 8 tokens: codes never leave the kernels
  bool h16;                // wide batches: h as int16 codes with group maxima, else fp32
  size_t o_xq, o_sx, o_h, o_hq, o_sh, o_hmax, total;
};

static int make_dense_plan(const moe_dense_config* c, DensePlan* out) {
  if (!c) return MOE_ERR_ARG;
  if (c->num_tokens < 1 || c->hidden < 1 || c->intermediate < 1) return MOE_ERR_ARG;
  if (c->act_dtype != MOE_F32 && c->act_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (c->hidden % 16 || c->intermediate % 16 || c->hidden > kNormMaxWidth ||
      c->intermediate > kNormMaxWidth || c->num_tokens > kMaxRows ||
      c->num_tokens * std::max(c->hidden, c->intermediate) > kMaxOutputs)
    return MOE_ERR_UNSUPPORTED;
  DensePlan q{};
  q.T = c->num_tokens;
  q.H = c->hidden;
  q.I = c->intermediate;
  q.act = c->act_dtype;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align256(o + bytes); return at; };
  q.few = dense_few_ok(q.T, q.H, q.I);
  q.o_xq = take(q.few ? 0 : size_t(q.T) * q.H);
  q.o_sx = take(q.few ? 0 : size_t(q.T) * 4);
  q.h16 = !q.few && glu_h16_ok(q.T, q.H, q.I);
  q.o_h = take(size_t(q.T) * q.I * (q.h16 ? 2 : 4));
  q.o_hq = take(q.few ? 0 : size_t(q.T) * q.I);
  q.o_sh = take(q.few ? 0 : size_t(q.T) * 4);
  q.o_hmax = take(q.few   ? dense_few_hmax_bytes(q.T, q.I)
                  : q.h16 ? size_t(q.T) * ((q.I + 31) / 32) * 4
                          : 0);
  q.total = o;
  *out = q;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_quant_rows(int64_t rows, int32_t width, int32_t act_dtype, int32_t format,
                        const void* x, const void* residual, const void* norm_weight,
                        float norm_eps, void* x_sum, void* out, void* scales, hipStream_t stream) {
  const NormQuant q{rows, width, act_dtype, format, x, residual, norm_weight, norm_eps, x_sum, out, scales};
  MOE_TRY(check_norm_quant(q));
  return launch_norm_quant(q, stream);
}

int moe_linear_i8(int64_t rows, int32_t in_width, int32_t out_width, int32_t out_dtype,
                  const int8_t* x, const float* x_scales, const int8_t* w, const float* w_scales,
                  const void* residual, void* y, hipStream_t stream) {
  const I8Product p{rows, in_width, out_width, out_dtype, x, x_scales, w, w_scales, nullptr, nullptr, residual, y};
  MOE_TRY(check_product(p, false));
  return launch_i8_product(p, stream);
}

int moe_glu_i8(int64_t rows, int32_t in_width, int32_t out_width, int32_t out_dtype,
               const int8_t* x, const float* x_scales, const int8_t* w_gate, const float* s_gate,
               const int8_t* w_up, const float* s_up, void* h, hipStream_t stream) {
  const I8Product p{rows, in_width, out_width, out_dtype, x, x_scales, w_gate, s_gate, w_up, s_up, nullptr, h};
  MOE_TRY(check_product(p, true));
  return launch_i8_product(p, stream);
}

int moe_dense_workspace_size(const moe_dense_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ERR_ARG;
  DensePlan q;
  MOE_TRY(make_dense_plan(cfg, &q));
  *bytes = q.total;
  return MOE_OK;
}

int moe_dense_residual_i8(const moe_dense_config* cfg, const void* x, const void* norm_weight,
                          float norm_eps, const moe_dense_weights* w, void* x_out, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  DensePlan q;
  MOE_TRY(make_dense_plan(cfg, &q));
  if (!x || !norm_weight || !w || !x_out || !ws || !(norm_eps >= 0.f)) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0 || !aligned16(x_out)) return MOE_ERR_ARG;
  if (ws_bytes < q.total) return MOE_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  int8_t* xq = reinterpret_cast<int8_t*>(base + q.o_xq);
  float* sx = reinterpret_cast<float*>(base + q.o_sx);
  void* h = base + q.o_h;
  int8_t* hq = reinterpret_cast<int8_t*>(base + q.o_hq);
  float* sh = reinterpret_cast<float*>(base + q.o_sh);
  const NormQuant nx{q.T, q.H, q.act, MOE_ROWS_I8, x, nullptr, norm_weight, norm_eps, nullptr, xq, sx};
  const I8Product up{q.T, q.H, q.I, MOE_F32, xq, sx, w->w_gate, w->s_gate, w->w_up, w->s_up, nullptr, h};
  const NormQuant nh{q.T, q.I, MOE_F32, MOE_ROWS_I8, h, nullptr, nullptr, 0.f, nullptr, hq, sh};
  const I8Product down{q.T, q.I, q.H, q.act, hq, sh, w->w_down, w->s_down, nullptr, nullptr, x, x_out};
  MOE_TRY(check_norm_quant(nx));
  MOE_TRY(check_product(up, true));
  MOE_TRY(check_norm_quant(nh));
  MOE_TRY(check_product(down, false));
  float* hmax = reinterpret_cast<float*>(base + q.o_hmax);
  if (q.few) {
    const DenseFew d{q.T, q.H, q.I, q.act, x, norm_weight, norm_eps, w, static_cast<float*>(h),
                     hmax, x_out};
    return launch_dense_few(d, stream);
  }
  MOE_TRY(launch_norm_quant(nx, stream));
  if (q.h16) {
    MOE_TRY(launch_glu_h16(up, hmax, stream));
    MOE_TRY(launch_h16_codes(h, hmax, q.T, q.I, hq, sh, stream));
  } else {
    MOE_TRY(launch_i8_product(up, stream));
    MOE_TRY(launch_norm_quant(nh, stream));
  }
  return launch_i8_product(down, stream);
}

}  // extern "C"
