// The C ABI of the decoder block's operators around the mixer (norms, linear, mixture of
// experts): host-side validation, workspace sizing and dispatch.
#include <string.h>

#include "jmix_internal.cuh"

#define JM_API extern "C" __attribute__((visibility("default")))

namespace jmix {
namespace {

constexpr int64_t kMaxNormCols = 16384;

// A named device pointer of a call, the bytes it covers and whether it is required.
struct Arg {
  const char* name;
  const void* p;
  size_t bytes;
  bool required;
};

bool overlap(const Arg& a, const Arg& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

jm_status check_args(const Arg* args, int n) {
  for (int i = 0; i < n; ++i) {
    if (!args[i].p) {
      if (!args[i].required) continue;
      set_error("%s is NULL", args[i].name);
      return JM_ERR_INVALID_ARG;
    }
    if (reinterpret_cast<uintptr_t>(args[i].p) % 16) {
      set_error("%s is not 16-byte aligned", args[i].name);
      return JM_ERR_INVALID_ARG;
    }
  }
  return JM_OK;
}

jm_status refuse_overlap(const Arg& a, const Arg& b) {
  set_error("%s overlaps %s", a.name, b.name);
  return JM_ERR_INVALID_ARG;
}

jm_status check_workspace(const char* who, const void* ws, size_t given, size_t need) {
  if (!ws) {
    set_error("%s: workspace is NULL", who);
    return JM_ERR_WORKSPACE;
  }
  if (reinterpret_cast<uintptr_t>(ws) % 256) {
    set_error("%s: workspace must be 256-byte aligned", who);
    return JM_ERR_WORKSPACE;
  }
  if (given < need) {
    set_error("%s: workspace too small: %zu bytes given, %zu needed", who, given, need);
    return JM_ERR_WORKSPACE;
  }
  return JM_OK;
}

jm_status check_norm_dims(const jm_norm_dims* d) {
  if (!d) {
    set_error("dims is NULL");
    return JM_ERR_INVALID_ARG;
  }
  if (d->io != JM_F32 && d->io != JM_BF16) {
    set_error("io dtype must be JM_F32 or JM_BF16");
    return JM_ERR_INVALID_ARG;
  }
  if (d->kind != JM_NORM_RMS && d->kind != JM_NORM_LAYER) {
    set_error("kind must be JM_NORM_RMS or JM_NORM_LAYER");
    return JM_ERR_INVALID_ARG;
  }
  if (d->reserved != 0) {
    set_error("jm_norm_dims.reserved must be 0");
    return JM_ERR_INVALID_ARG;
  }
  if (d->rows < 0 || d->cols <= 0 || d->x_stride < d->cols) {
    set_error("rows must be >= 0, cols > 0 and x_stride >= cols");
    return JM_ERR_INVALID_ARG;
  }
  if (!(d->eps >= 0.0f) || d->eps > 1e30f) {
    set_error("eps must be finite and >= 0");
    return JM_ERR_INVALID_ARG;
  }
  if (d->cols > kMaxNormCols) {
    set_error("cols > %lld is not built (got %lld)", (long long)kMaxNormCols, (long long)d->cols);
    return JM_ERR_UNSUPPORTED;
  }
  if (d->rows > 0x7fffffffLL || (double)d->rows * (double)d->x_stride > 1.0e15) {
    set_error("problem too large");
    return JM_ERR_INVALID_ARG;
  }
  return JM_OK;
}

size_t esize(jm_dtype io) { return io == JM_BF16 ? 2 : 4; }

size_t strided_bytes(const jm_norm_dims* d) {
  return d->rows ? (size_t)((d->rows - 1) * d->x_stride + d->cols) * esize(d->io) : 0;
}

// The outputs may not overlap an input or one another, except that an output
// named in `same` may be exactly that input's buffer (each value is read before
// the thread that read it writes it).
jm_status check_norm_overlap(const Arg* out, int n_out, const Arg* in, int n_in,
                             const bool* same) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j) {
      const bool ok = same[i * n_in + j] && out[i].p == in[j].p && out[i].bytes == in[j].bytes;
      if (!ok && overlap(out[i], in[j])) return refuse_overlap(out[i], in[j]);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return refuse_overlap(out[i], out[j]);
  }
  return JM_OK;
}

}  // namespace
}  // namespace jmix

using namespace jmix;

JM_API jm_status jm_norm_fwd(const jm_norm_dims* dims, const void* x, const void* residual,
                             const void* weight, const void* bias, void* y, void* sum,
                             float* stats, jm_stream_t stream) {
  jm_status st = check_norm_dims(dims);
  if (st != JM_OK) return st;
  const size_t es = esize(dims->io), act = (size_t)dims->rows * dims->cols * es,
               vec = (size_t)dims->cols * es;
  const bool any = dims->rows > 0;
  if (bias && dims->kind == JM_NORM_RMS) {
    set_error("bias must be NULL for JM_NORM_RMS");
    return JM_ERR_INVALID_ARG;
  }
  if (sum && !residual) {
    set_error("sum must be NULL without a residual (it would be x)");
    return JM_ERR_INVALID_ARG;
  }
  const Arg in[] = {{"x", x, strided_bytes(dims), any},
                    {"residual", residual, act, false},
                    {"weight", weight, vec, true},
                    {"bias", bias, vec, false}};
  const Arg out[] = {{"y", y, act, any},
                     {"sum", sum, act, any && residual},
                     {"stats", stats, (size_t)dims->rows * 8, false}};
  if ((st = check_args(in, 4)) != JM_OK || (st = check_args(out, 3)) != JM_OK) return st;
  const bool packed = dims->x_stride == dims->cols;
  const bool same[] = {packed, true,  false, false,   // y
                       packed, true,  false, false,   // sum
                       false,  false, false, false};  // stats
  if ((st = check_norm_overlap(out, 3, in, 4, same)) != JM_OK) return st;
  Problem p;
  begin_call(p, stream);
  if (!any) return finish_call(p, cudaSuccess);
  NormFwdArgs a{};
  a.rows = dims->rows;
  a.cols = dims->cols;
  a.x_stride = dims->x_stride;
  a.eps = dims->eps;
  a.layer = dims->kind == JM_NORM_LAYER;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.sum = sum;
  a.stats = stats;
  return finish_call(p, run_norm_fwd(a, dims->io, p));
}

JM_API size_t jm_norm_bwd_workspace_size(const jm_norm_dims* dims) {
  if (check_norm_dims(dims) != JM_OK) return 0;
  return norm_bwd_ws_bytes(dims->rows, dims->cols, dims->x_stride, dims->io);
}

JM_API jm_status jm_norm_bwd(const jm_norm_dims* dims, const void* g_y, const void* x,
                             const void* weight, const float* stats, const void* g_sum, void* g_x,
                             void* g_weight, void* g_bias, void* workspace, size_t ws_bytes,
                             jm_stream_t stream) {
  jm_status st = check_norm_dims(dims);
  if (st != JM_OK) return st;
  const size_t es = esize(dims->io), act = (size_t)dims->rows * dims->cols * es,
               vec = (size_t)dims->cols * es;
  const bool any = dims->rows > 0;
  if (g_bias && dims->kind == JM_NORM_RMS) {
    set_error("g_bias must be NULL for JM_NORM_RMS");
    return JM_ERR_INVALID_ARG;
  }
  const size_t need = jm_norm_bwd_workspace_size(dims);
  const Arg in[] = {{"g_y", g_y, act, any},
                    {"x", x, strided_bytes(dims), any},
                    {"weight", weight, vec, true},
                    {"stats", stats, (size_t)dims->rows * 8, any},
                    {"g_sum", g_sum, act, false}};
  const Arg out[] = {{"g_x", g_x, act, any},
                     {"g_weight", g_weight, vec, false},
                     {"g_bias", g_bias, vec, false},
                     {"workspace", workspace, need, false}};
  if ((st = check_args(in, 5)) != JM_OK || (st = check_args(out, 3)) != JM_OK) return st;
  if ((st = check_workspace("jm_norm_bwd", workspace, ws_bytes, need)) != JM_OK) return st;
  const bool same[20] = {true, false, false, false, true};  // g_x: g_y or g_sum
  if ((st = check_norm_overlap(out, 4, in, 5, same)) != JM_OK) return st;
  Problem p;
  begin_call(p, stream);
  NormBwdArgs a{};
  a.rows = dims->rows;
  a.cols = dims->cols;
  a.x_stride = dims->x_stride;
  a.layer = dims->kind == JM_NORM_LAYER;
  a.gy = g_y;
  a.x = x;
  a.weight = weight;
  a.stats = stats;
  a.g_sum = g_sum;
  a.g_x = g_x;
  return finish_call(p, run_norm_bwd(a, g_weight, g_bias, static_cast<char*>(workspace), dims->io,
                                     p));
}

namespace jmix {
namespace {

jm_status check_linear_dims(const jm_linear_dims* d) {
  if (!d) {
    set_error("dims is NULL");
    return JM_ERR_INVALID_ARG;
  }
  if (d->io != JM_F32 && d->io != JM_BF16) {
    set_error("io dtype must be JM_F32 or JM_BF16");
    return JM_ERR_INVALID_ARG;
  }
  if (d->io != JM_BF16) {
    set_error("the linear operators are built for bf16 io only");
    return JM_ERR_UNSUPPORTED;
  }
  if (d->act < JM_ACT_NONE || d->act > JM_ACT_SILU) {
    set_error("act must be one of JM_ACT_*");
    return JM_ERR_INVALID_ARG;
  }
  if (d->rows < 0 || d->in_features <= 0 || d->out_features <= 0) {
    set_error("sizes must be positive (rows >= 0)");
    return JM_ERR_INVALID_ARG;
  }
  if (d->in_features % 8 || d->out_features % 8) {
    set_error("in_features and out_features must be multiples of 8 (got %lld, %lld)",
              (long long)d->in_features, (long long)d->out_features);
    return JM_ERR_INVALID_ARG;
  }
  const int64_t most = 0x7fffff00LL;  // coordinates of the tensor maps are 32-bit
  if (d->rows > most || d->in_features > most || d->out_features > most ||
      (double)d->rows * (double)d->in_features > 1.0e12 ||
      (double)d->rows * (double)d->out_features > 1.0e12 ||
      (double)d->in_features * (double)d->out_features > 1.0e12) {
    set_error("problem too large");
    return JM_ERR_INVALID_ARG;
  }
  return JM_OK;
}

// No output may overlap an input or another output.
jm_status check_disjoint(const Arg* out, int n_out, const Arg* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return refuse_overlap(out[i], in[j]);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return refuse_overlap(out[i], out[j]);
  }
  return JM_OK;
}

}  // namespace
}  // namespace jmix

JM_API size_t jm_linear_fwd_workspace_size(const jm_linear_dims* dims) {
  if (check_linear_dims(dims) != JM_OK) return 0;
  return linear_fwd_ws_bytes(dims->rows, dims->in_features, dims->out_features);
}

JM_API size_t jm_linear_bwd_workspace_size(const jm_linear_dims* dims) {
  if (check_linear_dims(dims) != JM_OK) return 0;
  return linear_bwd_ws_bytes(dims->rows, dims->in_features, dims->out_features, dims->act);
}

JM_API jm_status jm_linear_fwd(const jm_linear_dims* dims, const void* x, const void* w,
                               const void* bias, const void* residual, void* out, void* pre,
                               void* workspace, size_t ws_bytes, jm_stream_t stream) {
  jm_status st = check_linear_dims(dims);
  if (st != JM_OK) return st;
  const size_t M = (size_t)dims->rows, K = (size_t)dims->in_features,
               N = (size_t)dims->out_features;
  const bool any = M > 0;
  const size_t need = jm_linear_fwd_workspace_size(dims);
  // the residual is checked apart: it may be exactly out's buffer, since every value of it is
  // read before out is written there: by the same thread in the few-row kernel and the sum of
  // K splits; in the pairs' kernel box by box, where a residual box and an output box are the
  // same 64 columns x 128 rows of one epilogue group and the load has landed before the store
  // is issued
  const Arg in[] = {{"x", x, M * K * 2, any},
                    {"w", w, N * K * 2, true},
                    {"bias", bias, N * 2, false},
                    {"residual", residual, M * N * 2, false}};
  const Arg outs[] = {{"out", out, M * N * 2, any},
                      {"pre", pre, M * N * 2, false},
                      {"workspace", workspace, need, false}};
  if ((st = check_args(in, 4)) != JM_OK || (st = check_args(outs, 2)) != JM_OK) return st;
  if ((st = check_workspace("jm_linear_fwd", workspace, ws_bytes, need)) != JM_OK) return st;
  if ((st = check_disjoint(outs, 3, in, residual == out ? 3 : 4)) != JM_OK) return st;
  if (residual == out)
    for (int i = 1; i < 3; ++i)
      if (overlap(outs[i], in[3])) return refuse_overlap(outs[i], in[3]);
  Problem p;
  begin_call(p, stream);
  LinearArgs a{};
  a.M = dims->rows;
  a.K = dims->in_features;
  a.N = dims->out_features;
  a.act = dims->act;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.pre = pre;
  a.ws = static_cast<char*>(workspace);
  return finish_call(p, run_linear_fwd(a, p));
}

JM_API jm_status jm_linear_bwd(const jm_linear_dims* dims, const void* g_out, const void* x,
                               const void* w, const void* pre, void* g_x, void* g_w, void* g_bias,
                               void* workspace, size_t ws_bytes, jm_stream_t stream) {
  jm_status st = check_linear_dims(dims);
  if (st != JM_OK) return st;
  const size_t M = (size_t)dims->rows, K = (size_t)dims->in_features,
               N = (size_t)dims->out_features;
  const bool any = M > 0, act = dims->act != JM_ACT_NONE;
  if (pre && !act) {
    set_error("pre must be NULL for JM_ACT_NONE");
    return JM_ERR_INVALID_ARG;
  }
  const size_t need = jm_linear_bwd_workspace_size(dims);
  const Arg in[] = {{"g_out", g_out, M * N * 2, any},
                    {"x", x, M * K * 2, any && g_w},
                    {"w", w, N * K * 2, any && g_x},
                    {"pre", pre, M * N * 2, any && act}};
  const Arg outs[] = {{"g_x", g_x, M * K * 2, false},
                      {"g_w", g_w, N * K * 2, false},
                      {"g_bias", g_bias, N * 2, false},
                      {"workspace", workspace, need, false}};
  if ((st = check_args(in, 4)) != JM_OK || (st = check_args(outs, 3)) != JM_OK) return st;
  if ((st = check_workspace("jm_linear_bwd", workspace, ws_bytes, need)) != JM_OK) return st;
  if ((st = check_disjoint(outs, 4, in, 4)) != JM_OK) return st;
  Problem p;
  begin_call(p, stream);
  LinearArgs a{};
  a.M = dims->rows;
  a.K = dims->in_features;
  a.N = dims->out_features;
  a.act = dims->act;
  a.g_out = g_out;
  a.x = x;
  a.w = w;
  a.pre = const_cast<void*>(pre);
  a.g_x = g_x;
  a.g_w = g_w;
  a.g_bias = g_bias;
  a.ws = static_cast<char*>(workspace);
  return finish_call(p, run_linear_bwd(a, p));
}

namespace jmix {
namespace {

jm_status check_moe_dims(const jm_moe_dims* d, MoeArgs* m) {
  if (!d) {
    set_error("dims is NULL");
    return JM_ERR_INVALID_ARG;
  }
  if (d->io != JM_F32 && d->io != JM_BF16) {
    set_error("io dtype must be JM_F32 or JM_BF16");
    return JM_ERR_INVALID_ARG;
  }
  if (d->io != JM_BF16) {
    set_error("the mixture-of-experts layer is built for bf16 io only");
    return JM_ERR_UNSUPPORTED;
  }
  if (d->router != JM_ROUTE_SOFTMAX_ALL && d->router != JM_ROUTE_SOFTMAX_TOPK) {
    set_error("router must be one of JM_ROUTE_*");
    return JM_ERR_INVALID_ARG;
  }
  if (d->tokens < 0 || d->d_model <= 0 || d->d_ff <= 0 || d->n_experts <= 0 || d->top_k <= 0) {
    set_error("sizes must be positive (tokens >= 0)");
    return JM_ERR_INVALID_ARG;
  }
  if (d->d_model % 8 || d->d_ff % 8) {
    set_error("d_model and d_ff must be multiples of 8 (got %lld, %lld)", (long long)d->d_model,
              (long long)d->d_ff);
    return JM_ERR_INVALID_ARG;
  }
  if (d->top_k > d->n_experts) {
    set_error("top_k %lld is more than n_experts %lld", (long long)d->top_k,
              (long long)d->n_experts);
    return JM_ERR_INVALID_ARG;
  }
  if (d->tokens > 256 || d->n_experts > 256 || d->top_k > 8) {
    set_error("more than 256 tokens, 256 experts or top_k 8 is not built (got %lld, %lld, %lld)",
              (long long)d->tokens, (long long)d->n_experts, (long long)d->top_k);
    return JM_ERR_UNSUPPORTED;
  }
  const int64_t most = 1LL << 24;
  m->T = d->tokens;
  m->D = d->d_model;
  m->F = d->d_ff;
  m->E = d->n_experts;
  m->topk = d->top_k;
  m->topk_softmax = d->router == JM_ROUTE_SOFTMAX_TOPK;
  if (m->D > most || m->F > most || !moe_fits(*m)) {
    set_error("problem too large");
    return JM_ERR_INVALID_ARG;
  }
  return JM_OK;
}

}  // namespace
}  // namespace jmix

JM_API size_t jm_moe_fwd_workspace_size(const jm_moe_dims* dims) {
  MoeArgs m{};
  if (check_moe_dims(dims, &m) != JM_OK) return 0;
  return moe_ws_bytes(m);
}

JM_API jm_status jm_moe_fwd(const jm_moe_dims* dims, const void* x, const void* router_w,
                            const void* w_gate, const void* w_up, const void* w_down,
                            const void* residual, void* out, int32_t* topk_idx, float* topk_w,
                            void* workspace, size_t ws_bytes, jm_stream_t stream) {
  MoeArgs m{};
  jm_status st = check_moe_dims(dims, &m);
  if (st != JM_OK) return st;
  const size_t td = (size_t)m.T * m.D * 2, w = (size_t)m.E * m.F * m.D * 2,
               pairs = (size_t)m.T * m.topk * 4;
  const bool any = m.T > 0;
  const size_t need = moe_ws_bytes(m);
  // the residual last: it may be exactly out's buffer (each value is read by the thread
  // that then writes it)
  const Arg in[] = {{"x", x, td, any},           {"router_w", router_w, (size_t)m.E * m.D * 2, true},
                    {"w_gate", w_gate, w, true}, {"w_up", w_up, w, true},
                    {"w_down", w_down, w, true}, {"residual", residual, td, false}};
  const Arg outs[] = {{"out", out, td, any},
                      {"topk_idx", topk_idx, pairs, false},
                      {"topk_w", topk_w, pairs, false},
                      {"workspace", workspace, need, false}};
  if ((st = check_args(in, 6)) != JM_OK || (st = check_args(outs, 3)) != JM_OK) return st;
  if ((st = check_workspace("jm_moe_fwd", workspace, ws_bytes, need)) != JM_OK) return st;
  if ((st = check_disjoint(outs, 4, in, residual == out ? 5 : 6)) != JM_OK) return st;
  Problem p;
  begin_call(p, stream);
  if (!any) {
    return finish_call(p, cudaMemsetAsync(workspace, 0, sizeof(ErrFlags), p.stream));
  }
  m.x = x;
  m.router_w = router_w;
  m.w_gate = w_gate;
  m.w_up = w_up;
  m.w_down = w_down;
  m.residual = residual;
  m.out = out;
  m.topk_idx = topk_idx;
  m.topk_w = topk_w;
  m.ws = static_cast<char*>(workspace);
  return finish_call(p, run_moe(m, p));
}
