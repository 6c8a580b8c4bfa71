// pkm_block_api.cu -- the extern "C" entry points of the transformer-block operators
// declared in include/pkm.h: argument validation and launches. Each call is an NVTX range
// of its name; the stage trace covers the layer's own passes only.
#include <math.h>

#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "../../include/pkm.h"
#include "pkm_block.h"
#include "pkm_linear.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool is_dtype(int t) { return t == PKM_F32 || t == PKM_BF16; }

template <int N>
bool all_aligned16(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

// An array of a call; empty where it is not given.
struct Array {
  uintptr_t at, end;
  int dtype;
  Array(const void* p, int64_t n, int t)
      : at(reinterpret_cast<uintptr_t>(p)),
        end(at + (p ? static_cast<uintptr_t>(n) * (t == PKM_BF16 ? 2 : 4) : 0)), dtype(t) {}
};
bool apart(const Array& a, const Array& b) {
  return a.at == a.end || b.at == b.end || a.end <= b.at || b.end <= a.at;
}
// Apart, or one and the same array.
bool apart_or_same(const Array& a, const Array& b) {
  return (a.at == b.at && a.end == b.end && a.dtype == b.dtype) || apart(a, b);
}
// `outs` are apart from each other and from `ins`.
bool all_apart(std::initializer_list<Array> outs, std::initializer_list<Array> ins) {
  for (const Array* o = outs.begin(); o != outs.end(); ++o) {
    for (const Array* p = outs.begin(); p != o; ++p)
      if (!apart(*o, *p)) return false;
    for (const Array& i : ins)
      if (!apart(*o, i)) return false;
  }
  return true;
}

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

int finish(cudaError_t e, int launches) {
  if (e != cudaSuccess) return PKM_ERR_CUDA;
  pkm::count_launches(launches);
  return PKM_OK;
}

// rows and d, which every call of the norm reads.
int validate_norm_size(const pkm_norm_shape* s) {
  if (!s || s->rows < 0 || s->d < 1) return PKM_ERR_INVALID_ARG;
  if (s->d > pkm::kNormMaxD || s->rows > 0x7fffffffLL) return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

int validate_norm(const pkm_norm_shape* s, bool has_add) {
  const int rc = validate_norm_size(s);
  if (rc != PKM_OK) return rc;
  if (!is_dtype(s->x_dtype) || !is_dtype(s->y_dtype) || (has_add && !is_dtype(s->add_dtype)))
    return PKM_ERR_INVALID_ARG;
  return PKM_OK;
}

pkm::NormArgs norm_args(const pkm_norm_shape* s) {
  return {s->rows, s->d, s->x_dtype, s->add_dtype, s->y_dtype, s->grad_dtype, s->eps};
}

int validate_linear(const pkm_linear_shape* s) {
  if (!s || s->M < 0 || s->N < 1 || s->K < 1 || !is_dtype(s->dtype) || !is_dtype(s->out_dtype) ||
      s->activation < PKM_ACT_NONE || s->activation > PKM_ACT_SILU)
    return PKM_ERR_INVALID_ARG;
  const int64_t wide = s->N > s->K ? s->N : s->K;
  if (s->M > 0x7fffffffLL - 256 || wide > pkm::kLinearMaxWidth || s->M * wide >= 1LL << 38)
    return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

pkm::LinearArgs linear_args(const pkm_linear_shape* s) {
  return {s->M, s->N, s->K, s->dtype, s->out_dtype, s->activation};
}

Array scratch(const void* workspace, size_t bytes) {
  return {workspace, static_cast<int64_t>(bytes / sizeof(float)), PKM_F32};
}

}  // namespace

extern "C" {

int pkm_layernorm_forward(const pkm_norm_shape* s, const void* x, const void* add,
                          const float* gamma, const float* beta, void* y, void* sum, float* mean,
                          float* rstd, void* stream) {
  const int rc = validate_norm(s, add != nullptr);
  if (rc != PKM_OK) return rc;
  if (!(s->eps >= 0.f) || s->eps > 1e30f) return PKM_ERR_INVALID_ARG;
  if (!gamma || (s->rows > 0 && (!x || !y || (add != nullptr) != (sum != nullptr))))
    return PKM_ERR_INVALID_ARG;
  if (!all_aligned16({x, add, gamma, beta, y, sum, mean, rstd})) return PKM_ERR_UNSUPPORTED;
  if (s->rows == 0) return PKM_OK;
  const int64_t n = s->rows * s->d;
  const Array ax(x, n, s->x_dtype), aa(add, n, s->add_dtype), ay(y, n, s->y_dtype),
      as(sum, n, s->x_dtype), am(mean, s->rows, PKM_F32), ar(rstd, s->rows, PKM_F32),
      ag(gamma, s->d, PKM_F32), ab(beta, s->d, PKM_F32);
  if (!all_apart({ay, as, am, ar}, {ag, ab}) || !all_apart({am, ar}, {ax, aa}) ||
      !apart_or_same(ay, ax) || !apart_or_same(ay, aa) || !apart_or_same(as, ax) ||
      !apart_or_same(as, aa))
    return PKM_ERR_INVALID_ARG;
  const Range range("pkm.layernorm_forward");
  return finish(pkm::launch_layernorm_forward(norm_args(s), x, add, gamma, beta, y, sum, mean,
                                              rstd, static_cast<cudaStream_t>(stream)),
                1);
}

size_t pkm_norm_workspace_size(const pkm_norm_shape* s) {
  if (validate_norm_size(s) != PKM_OK) return 0;
  return static_cast<size_t>(pkm::norm_workspace_blocks(s->rows)) * 2 * s->d * sizeof(float);
}

int pkm_layernorm_backward(const pkm_norm_shape* s, const void* grad_y, const void* x,
                           const float* mean, const float* rstd, const float* gamma,
                           const void* grad_sum, void* grad_x, float* grad_gamma,
                           float* grad_beta, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const int rc = validate_norm(s, grad_sum != nullptr);
  if (rc != PKM_OK) return rc;
  if (!is_dtype(s->grad_dtype)) return PKM_ERR_INVALID_ARG;
  if (!gamma || (s->rows > 0 && (!grad_y || !x || !mean || !rstd || !grad_x)))
    return PKM_ERR_INVALID_ARG;
  if (!all_aligned16({grad_y, x, mean, rstd, gamma, grad_sum, grad_x, grad_gamma, grad_beta}))
    return PKM_ERR_UNSUPPORTED;
  const size_t need = pkm_norm_workspace_size(s);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return PKM_ERR_WORKSPACE;
  const int64_t n = s->rows * s->d;
  const Array ay(grad_y, n, s->y_dtype), ax(x, n, s->x_dtype), am(mean, s->rows, PKM_F32),
      ar(rstd, s->rows, PKM_F32), ag(gamma, s->d, PKM_F32), as(grad_sum, n, s->add_dtype),
      ox(grad_x, n, s->grad_dtype), og(grad_gamma, s->d, PKM_F32), ob(grad_beta, s->d, PKM_F32),
      aw = scratch(workspace, need);
  if (s->rows > 0 &&
      (!all_apart({ox, og, ob, aw}, {am, ar, ag}) || !all_apart({og, ob, aw}, {ay, ax, as}) ||
       !apart_or_same(ox, ay) || !apart_or_same(ox, ax) || !apart_or_same(ox, as)))
    return PKM_ERR_INVALID_ARG;
  const Range range("pkm.layernorm_backward");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->rows == 0) {
    for (float* g : {grad_gamma, grad_beta})
      if (g && cudaMemsetAsync(g, 0, sizeof(float) * s->d, st) != cudaSuccess) return PKM_ERR_CUDA;
    return PKM_OK;
  }
  return finish(pkm::launch_layernorm_backward(norm_args(s), grad_y, x, mean, rstd, gamma,
                                               grad_sum, grad_x, grad_gamma, grad_beta,
                                               static_cast<float*>(workspace), st),
                grad_gamma || grad_beta ? 2 : 1);
}

size_t pkm_linear_workspace_size(const pkm_linear_shape* s, int for_backward) {
  if (validate_linear(s) != PKM_OK) return 0;
  return pkm::linear_workspace_bytes(linear_args(s), for_backward != 0);
}

int pkm_linear_forward(const pkm_linear_shape* s, const void* x, const void* W, const float* bias,
                       const void* residual, void* y, void* pre, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const int rc = validate_linear(s);
  if (rc != PKM_OK) return rc;
  if (!W || (s->M > 0 && (!x || !y))) return PKM_ERR_INVALID_ARG;
  if (!all_aligned16({x, W, bias, residual, y, pre})) return PKM_ERR_UNSUPPORTED;
  const pkm::LinearArgs a = linear_args(s);
  const size_t need = pkm::linear_workspace_bytes(a, false);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return PKM_ERR_WORKSPACE;
  if (s->M == 0) return PKM_OK;
  const Array ax(x, s->M * s->K, s->dtype), aw(W, static_cast<int64_t>(s->N) * s->K, s->dtype),
      ab(bias, s->N, PKM_F32), ar(residual, s->M * s->N, s->out_dtype),
      oy(y, s->M * s->N, s->out_dtype), op(pre, s->M * s->N, s->dtype), ow = scratch(workspace, need);
  if (!all_apart({oy, op, ow}, {ax, aw, ab}) || !all_apart({op, ow}, {ar}) || !apart_or_same(oy, ar))
    return PKM_ERR_INVALID_ARG;
  const Range range("pkm.linear_forward");
  int launches = 0;
  const cudaError_t e = pkm::launch_linear_forward(a, x, W, bias, residual, y, pre, workspace,
                                                   &launches, static_cast<cudaStream_t>(stream));
  return finish(e, launches);
}

int pkm_linear_backward(const pkm_linear_shape* s, const void* x, const void* W,
                        const void* grad_y, const void* pre, void* grad_x, float* grad_W,
                        float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = validate_linear(s);
  if (rc != PKM_OK) return rc;
  const bool act = s->activation != PKM_ACT_NONE;
  if (!W || (s->M > 0 && (!x || !grad_y || (act && !pre)))) return PKM_ERR_INVALID_ARG;
  if (!all_aligned16({x, W, grad_y, pre, grad_x, grad_W, grad_bias})) return PKM_ERR_UNSUPPORTED;
  const pkm::LinearArgs a = linear_args(s);
  const size_t need = pkm::linear_workspace_bytes(a, true);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return PKM_ERR_WORKSPACE;
  // What is read: x for grad_W, W for grad_x.
  const Array ax(grad_W ? x : nullptr, s->M * s->K, s->dtype),
      aw(grad_x ? W : nullptr, static_cast<int64_t>(s->N) * s->K, s->dtype),
      ay(grad_y, s->M * s->N, s->dtype), ap(act ? pre : nullptr, s->M * s->N, s->dtype),
      ox(grad_x, s->M * s->K, s->out_dtype), oW(grad_W, static_cast<int64_t>(s->N) * s->K, PKM_F32),
      ob(grad_bias, s->N, PKM_F32), ow = scratch(workspace, need);
  if (s->M > 0 && !all_apart({ox, oW, ob, ow}, {ax, aw, ay, ap})) return PKM_ERR_INVALID_ARG;
  const Range range("pkm.linear_backward");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->M == 0) {
    if (grad_W && cudaMemsetAsync(grad_W, 0, sizeof(float) * s->N * s->K, st) != cudaSuccess)
      return PKM_ERR_CUDA;
    if (grad_bias && cudaMemsetAsync(grad_bias, 0, sizeof(float) * s->N, st) != cudaSuccess)
      return PKM_ERR_CUDA;
    return PKM_OK;
  }
  int launches = 0;
  const cudaError_t e = pkm::launch_linear_backward(a, x, W, grad_y, pre, grad_x, grad_W,
                                                    grad_bias, workspace, &launches, st);
  return finish(e, launches);
}

int pkm_adamw_step(const pkm_adamw_tensor* tensors, int64_t count, const pkm_adamw_hyper* h,
                   const float* dyn, void* stream) {
  if (!h || count < 0 || (count > 0 && !tensors)) return PKM_ERR_INVALID_ARG;
  // Written so that a NaN fails. eps must stay above 0 in fp32: an element without
  // gradients has m = v = 0, and 0 / (0 + eps) has to be 0.
  const bool rates = h->lr >= 0 && h->lr < 1e30 && h->beta1 >= 0 && h->beta1 < 1 &&
                     h->beta2 >= 0 && h->beta2 < 1 && h->eps >= 1e-30 && h->eps < 1e30 &&
                     fabs(h->grad_scale) < 1e30 && h->step >= 1;
  if (!rates || (h->zero_grad != 0 && h->zero_grad != 1)) return PKM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(dyn) & 3u) return PKM_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    const pkm_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !is_dtype(t.param_dtype) || !is_dtype(t.grad_dtype) ||
        (t.state_bits != 32 && t.state_bits != 8))
      return PKM_ERR_INVALID_ARG;
    if (!(t.weight_decay >= 0.f && t.weight_decay < 1e30f && t.lr_scale >= 0.f &&
          t.lr_scale < 1e30f))
      return PKM_ERR_INVALID_ARG;
    if (t.n >= 1LL << 38) return PKM_ERR_UNSUPPORTED;
    if (t.n == 0) continue;
    const bool eight = t.state_bits == 8;
    if (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale)) ||
        (!eight && (t.m_scale || t.v_scale)) || (t.master && t.param_dtype != PKM_BF16))
      return PKM_ERR_INVALID_ARG;
    if (!all_aligned16({t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale}))
      return PKM_ERR_UNSUPPORTED;
  }
  const Range range("pkm.adamw_step");
  int launches = 0;
  const cudaError_t e =
      pkm::launch_adamw(tensors, count, *h, dyn, &launches, static_cast<cudaStream_t>(stream));
  return finish(e, launches);
}

}  // extern "C"
