// prompt_attn.cu -- causal attention of grouped heads over packed prompts.
#include "attn_plain.cuh"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

struct RowSource {
  const uint16_t *k, *v;
  int64_t k_stride_t, v_stride_t;
  const int32_t* cu_k;
  int Tk, d;
  FM_DEV int begin(int b) const { return cu_k ? offset_at(cu_k, b, Tk) : 0; }
  FM_DEV int keys(int b) const { return max((cu_k ? offset_at(cu_k, b + 1, Tk) : Tk) - begin(b), 0); }
  FM_DEV int64_t past(int b, int n) const { return (int64_t)keys(b) - n; }
  FM_DEV int64_t clamp(int64_t j) const { return j; }
  FM_DEV bool held(int, int64_t) const { return true; }
  FM_DEV float value(int b, int64_t j, int head, int e, bool is_k) const {
    const uint16_t* x = is_k ? k + (begin(b) + j) * k_stride_t : v + (begin(b) + j) * v_stride_t;
    return __uint_as_float((uint32_t)x[head * d + e] << 16);
  }
};

}  // namespace
}  // namespace fm

using namespace fm;

FM_API fm_status fm_prompt_attn(const fm_prompt_attn_args* a) {
  const char* who = "fm_prompt_attn";
  if (!a) return set_error(FM_ERR_INVALID_ARG, "%s: args is NULL", who);
  const char* bad = bad_heads(a->n_h, a->n_k, a->d);
  if (bad) return set_error(FM_ERR_INVALID_ARG, "%s: n_h=%d n_k=%d d=%d (%s)", who, a->n_h, a->n_k, a->d, bad);
  if (a->T < 0 || a->Tk < 0 || a->T >= 1 << 30 || a->Tk >= 1 << 30 || a->B < 0 || a->B > 1 << 24)
    return set_error(FM_ERR_INVALID_ARG, "%s: T=%d Tk=%d B=%d (0 <= T, Tk < 2^30, 0 <= B <= 2^24)", who, a->T, a->Tk, a->B);
  if (a->window < 0) return set_error(FM_ERR_INVALID_ARG, "%s: window=%lld", who, (long long)a->window);
  if (!(a->scale > 0.0f) || isinf(a->scale * 1.4426950408889634f))
    return set_error(FM_ERR_INVALID_ARG, "%s: scale=%g", who, (double)a->scale);
  if (!a->cu_q && (a->B != 1 || a->cu_k))
    return set_error(FM_ERR_INVALID_ARG, "%s: without cu_q there is one sequence (B=%d) and no cu_k", who, a->B);
  if (a->cu_q && !a->cu_k && a->T != a->Tk)
    return set_error(FM_ERR_INVALID_ARG, "%s: without cu_k T=%d must be Tk=%d", who, a->T, a->Tk);
  if (a->T == 0 || a->B == 0) return FM_OK;
  if (bad_rows(a->q, a->q_stride_t, a->n_h, a->d) ||
      (a->Tk > 0 && (bad_rows(a->k, a->k_stride_t, a->n_k, a->d) || bad_rows(a->v, a->v_stride_t, a->n_k, a->d))))
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: q, k, v need 16-byte aligned pointers and token strides that are multiples of 8 and hold the heads",
                     who);
  if (!a->out || !aligned(a->out, 16) || !aligned(a->lse_out, 4) || !aligned(a->cu_q, 4) || !aligned(a->cu_k, 4) ||
      !aligned(a->sink_logit, 4))
    return set_error(FM_ERR_INVALID_ARG, "%s: out is NULL, or a pointer misaligned", who);
  fm_status st = check_device(nullptr);
  if (st != FM_OK) return st;
  RowSource src = {a->k, a->v, a->k_stride_t, a->v_stride_t, a->cu_k ? a->cu_k : a->cu_q, a->Tk, a->d};
  PlainParams p = {a->q, a->q_stride_t, a->cu_q, a->out, a->lse_out, a->sink_logit, a->window, a->scale, a->T, a->n_h, a->n_k, a->d, 1};
  if (a->cu_q) p.B = a->B;
  const cudaError_t e = launch_plain(p, src, reinterpret_cast<cudaStream_t>(a->stream));
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}
