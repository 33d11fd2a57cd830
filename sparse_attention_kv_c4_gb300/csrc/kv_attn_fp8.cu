// kv_attn_fp8.cu -- attention of grouped heads over the paged 8-bit cache.
#include <cuda_fp8.h>

#include "attn_plain.cuh"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

struct CacheSource {
  const uint8_t *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  int64_t P, page_stride, scale_stride;
  const int32_t* table;
  int R, d;
  const int64_t* start;
  unsigned int* status;
  FM_DEV int64_t past(int b, int n) const {  // a position past 2^62 sees nothing, as a negative one
    const int64_t s = start[b];
    return s < 0 || s >= (int64_t(1) << 62) ? -(int64_t)n : s;
  }
  FM_DEV int64_t clamp(int64_t j) const {
    if (j < (int64_t)R * kKvPage) return j;
    atomicOr(status, FM_DEV_PAGE_RANGE);
    return (int64_t)R * kKvPage - 1;
  }
  FM_DEV bool held(int b, int64_t j) const {
    const int page = table[(int64_t)b * R + j / kKvPage];
    if (page >= P) atomicOr(status, FM_DEV_PAGE_RANGE);
    return page >= 0 && page < P;
  }
  FM_DEV float value(int b, int64_t j, int head, int e, bool is_k) const {
    const int64_t page = table[(int64_t)b * R + j / kKvPage];
    const int row = (int)(j % kKvPage);
    const uint8_t c = (is_k ? k_pool : v_pool)[page * page_stride + ((int64_t)head * kKvPage + row) * d + e];
    const float s = (is_k ? k_scale : v_scale)[page * scale_stride + head * kBlocksPerPage + row / kKvBlock];
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3))) * s;
  }
};

}  // namespace
}  // namespace fm

using namespace fm;

FM_API size_t fm_kv_attn_fp8_workspace(int T, int n_h, int n_k, int d) {
  if (T < 0 || bad_heads(n_h, n_k, d)) return 0;
  return 0;
}

FM_API fm_status fm_kv_attn_fp8(const fm_kv_attn_fp8_args* a) {
  const char* who = "fm_kv_attn_fp8";
  if (!a) return set_error(FM_ERR_INVALID_ARG, "%s: args is NULL", who);
  const char* bad = bad_heads(a->n_h, a->n_k, a->d);
  if (bad) return set_error(FM_ERR_INVALID_ARG, "%s: n_h=%d n_k=%d d=%d (%s)", who, a->n_h, a->n_k, a->d, bad);
  if (a->T < 0 || a->T >= 1 << 24) return set_error(FM_ERR_INVALID_ARG, "%s: T=%d (0 <= T < 2^24)", who, a->T);
  bad = bad_cache(a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->P, a->page_stride, a->scale_stride, a->page_table, a->B,
                  a->R, a->n_k, a->d);
  if (bad) return set_error(FM_ERR_INVALID_ARG, "%s: %s", who, bad);
  if (a->window < 0) return set_error(FM_ERR_INVALID_ARG, "%s: window=%lld", who, (long long)a->window);
  if (!(a->scale > 0.0f) || isinf(a->scale * 1.4426950408889634f))
    return set_error(FM_ERR_INVALID_ARG, "%s: scale=%g", who, (double)a->scale);
  if (!a->cu_tokens && a->T != a->B)
    return set_error(FM_ERR_INVALID_ARG, "%s: without cu_tokens T=%d must be B=%d", who, a->T, a->B);
  if (a->T == 0 || a->B == 0) return FM_OK;
  if (bad_rows(a->q, a->q_stride_t, a->n_h, a->d))
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: q needs a 16-byte aligned pointer and a token stride that is a multiple of 8 and holds the heads", who);
  if (!a->out || !aligned(a->out, 16) || !aligned(a->lse_out, 4) || !a->start || !aligned(a->start, 8) ||
      !aligned(a->cu_tokens, 4) || !aligned(a->sink_logit, 4))
    return set_error(FM_ERR_INVALID_ARG, "%s: out or start is NULL, or a pointer misaligned", who);
  const size_t need = fm_kv_attn_fp8_workspace(a->T, a->n_h, a->n_k, a->d);
  if (need > 0 && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < need))
    return set_error(FM_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 256-byte aligned", who, need);
  fm_status st = check_device(nullptr);
  if (st != FM_OK) return st;
  CacheSource src = {a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->P, a->page_stride, a->scale_stride, a->page_table, a->R, a->d, a->start, nullptr};
  if ((st = status_word(&src.status)) != FM_OK) return st;
  PlainParams p = {a->q, a->q_stride_t, a->cu_tokens, a->out, a->lse_out, a->sink_logit, a->window, a->scale, a->T, a->n_h, a->n_k, a->d, a->B};
  const cudaError_t e = launch_plain(p, src, reinterpret_cast<cudaStream_t>(a->stream));
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}
