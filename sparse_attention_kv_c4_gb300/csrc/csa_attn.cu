// csa_attn.cu -- attention of a CSA layer: one softmax per head over the
// selected chunk cells, the first tokens and a sliding window of the sequence's
// tokens ("DeepSeek-V4 CSA + HCA explained", sec. 4), also for a tree of drafted
// tokens.  A cell c (512 elements) is key and value of every head:
//     s_j = scale (q_h . c_j),  out_h = sum_j e^{s_j} c_j / (sum_j e^{s_j} + e^{sink_h})
//
// One CTA per (token, eight heads), one warp per head: the warp walks the
// token's keys with the running maximum and sum of the softmax, each lane
// holding 16 elements of q and of the output in registers.
#include <cuda_bf16.h>

#include "fm_common.cuh"
#include "fm_internal.h"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kWidth = 512;
constexpr int kPage = 64;
constexpr int kMaxCells = 1024;

struct AttnParams {
  const uint16_t* q;
  const uint16_t* kv_pool;
  const int32_t* page_table;
  const int32_t* seq;
  const int64_t* pos;
  const uint16_t* cell_pool;
  const int32_t* cells;
  const float* sink_logit;
  const uint32_t* tree_mask;
  const int64_t* tree_base;
  uint16_t* out;
  float* lse;
  unsigned int* status;
  int64_t kv_page_rows, cell_page_rows;  // rows (of 512 elements) from page to page
  int64_t window;
  int64_t cell_limit;                    // Pc * 64
  int T, n_h, P, B, R, k, n_sink, tree_words;
  float scale;
};

// A token's keys, in order: k listed cells, n_first first tokens, n_win window
// tokens from slot low, then the drafted slots from base.
struct TokenKeys {
  int64_t low, base;
  int b;
  int n_first, n_win, n_tree;
};

FM_DEV TokenKeys token_keys(const AttnParams& p, int64_t t) {
  TokenKeys r = {0, 0, -1, 0, 0, 0};
  const int64_t b = p.seq != nullptr ? p.seq[t] : t;
  const int64_t pos = p.pos[t];
  if (b < 0 || pos < 0) return r;
  if (b >= p.B) {
    atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return r;
  }
  int64_t end = pos + 1;  // cached tokens below end
  if (p.tree_mask != nullptr) {
    r.base = p.tree_base[b];
    if (r.base < 0) return r;
    if (r.base < end) end = r.base;
    r.n_tree = 32 * p.tree_words;
  }
  r.b = (int)b;
  const int64_t held = (int64_t)p.R * kPage;
  if (end > held) {
    end = held;
    atomicOr(p.status, FM_DEV_PAGE_RANGE);
  }
  r.low = p.window > pos ? 0 : pos + 1 - p.window;
  if (r.low > end) r.low = end;
  r.n_first = (int)(p.n_sink < r.low ? p.n_sink : r.low);
  r.n_win = (int)(end - r.low);
  return r;
}

// Pool row of a cached token, or -1.
FM_DEV int token_row(const AttnParams& p, int b, int64_t slot) {
  const int64_t pg = slot / kPage;
  if (pg >= p.R) {
    atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return -1;
  }
  const int page = __ldg(p.page_table + (int64_t)b * p.R + pg);
  if (page >= p.P) {
    atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return -1;
  }
  return page < 0 ? -1 : (int)(page * p.kv_page_rows + slot % kPage);
}

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) csa_attn_kernel(const __grid_constant__ AttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (h >= p.n_h) return;
  const TokenKeys tk = token_keys(p, t);
  float q[16], o[16], m = -INFINITY, l = 0.f;
  const uint16_t* qrow = p.q + (t * p.n_h + h) * kWidth + 16 * lane;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    q[i] = __uint_as_float((uint32_t)qrow[i] << 16);
    o[i] = 0.f;
  }
  const int n = p.k + tk.n_first + tk.n_win + tk.n_tree;
  for (int j = 0; j < n; ++j) {
    const uint16_t* row = nullptr;
    if (j < p.k) {
      const int64_t cell = __ldg(p.cells + t * p.k + j);
      if (cell >= p.cell_limit) atomicOr(p.status, FM_DEV_PAGE_RANGE);
      if (cell >= 0 && cell < p.cell_limit)
        row = p.cell_pool + ((cell / kPage) * p.cell_page_rows + cell % kPage) * kWidth;
    } else {
      const int i = j - p.k;
      int64_t slot = i < tk.n_first ? i : tk.low + (i - tk.n_first);
      bool seen = true;
      if (i >= tk.n_first + tk.n_win) {
        const int d = i - tk.n_first - tk.n_win;
        seen = (__ldg(p.tree_mask + t * p.tree_words + (d >> 5)) >> (d & 31)) & 1u;
        slot = tk.base + d;
      }
      const int r = seen ? token_row(p, tk.b, slot) : -1;
      if (r >= 0) row = p.kv_pool + (int64_t)r * kWidth;
    }
    if (row == nullptr) continue;
    float c[16], s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * lane + 8 * i);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[8 * i + 2 * e] = __uint_as_float(u[e] << 16);
        c[8 * i + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(q[i], c[i], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    const float f = m == mn ? 1.f : expf(m - mn), w = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = o[i] * f + w * c[i];
  }
  float below = l;
  if (p.sink_logit != nullptr && l > 0.f) below += expf(p.sink_logit[h] - m);
  const float inv = l == 0.f ? 0.f : 1.f / below;
  uint16_t* dst = p.out + (t * p.n_h + h) * kWidth + 16 * lane;
#pragma unroll
  for (int i = 0; i < 16; ++i) dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  if (p.lse != nullptr && lane == 0) p.lse[t * p.n_h + h] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t attn_workspace_bytes(int, int) { return 0; }

fm_status launch_attn(const AttnParams& p, int, void*, cudaStream_t stream) {
  csa_attn_kernel<<<dim3((unsigned)p.T, (unsigned)((p.n_h + kWarps - 1) / kWarps)), 32 * kWarps, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "fm_csa_attn: launch: %s", cudaGetErrorString(e));
  return FM_OK;
}

fm_status csa_attn(const char* who, bool tree, const uint16_t* q, int T, int n_h, int d, const uint16_t* kv_pool,
                   int64_t P, int64_t kv_page_stride, const int32_t* page_table, int B, int R, const int32_t* seq,
                   const int64_t* pos, int64_t window, int n_sink, const uint16_t* cell_pool, int64_t Pc,
                   int64_t cell_page_stride, const int32_t* cells, int k, const float* sink_logit, float scale,
                   const uint32_t* tree_mask, int tree_words, const int64_t* tree_base, uint16_t* out, float* lse_out,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (d != kWidth) return set_error(FM_ERR_INVALID_ARG, "%s: d=%d (need 512)", who, d);
  if (T < 0 || n_h < 1 || n_h > 1024 || (int64_t)T * n_h >= (int64_t(1) << 31))
    return set_error(FM_ERR_INVALID_ARG, "%s: bad sizes T=%d n_h=%d (1 <= n_h <= 1024, T * n_h < 2^31)", who, T, n_h);
  if (B < 0 || R < 0 || R > (1 << 24) || window < 0 || n_sink < 0 || k < 0 || k > kMaxCells)
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: bad sizes B=%d R=%d window=%lld n_sink=%d k=%d (R <= 2^24, 0 <= k <= 1024)", who, B, R,
                     (long long)window, n_sink, k);
  if (!(scale > 0.0f) || isinf(scale)) return set_error(FM_ERR_INVALID_ARG, "%s: scale=%g", who, (double)scale);
  if (tree && (tree_words < 1 || tree_words > 32))
    return set_error(FM_ERR_INVALID_ARG, "%s: tree_words=%d (1..32)", who, tree_words);
  // a pool's rows are counted in 31 bits
  auto bad_pool = [](const uint16_t* pool, int64_t pages, int64_t stride) {
    if (pages == 0) return false;
    return pages < 0 || !pool || !aligned(pool, 16) || stride < (int64_t)kPage * kWidth || stride % kWidth != 0 ||
           stride / kWidth >= (int64_t(1) << 31) || pages >= (int64_t(1) << 31) / (stride / kWidth);
  };
  if (bad_pool(kv_pool, P, kv_page_stride) || (k > 0 && bad_pool(cell_pool, Pc, cell_page_stride)))
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: a pool needs a 16-byte aligned pointer, a page stride that is a multiple of 512 and at least "
                     "64 * 512, and fewer than 2^31 rows of 512 elements",
                     who);
  if (T == 0) return FM_OK;
  if (seq == nullptr && T > B)
    return set_error(FM_ERR_INVALID_ARG, "%s: without seq, token t is row t of the page table: T=%d > B=%d", who, T, B);
  if (!q || !pos || !out || (k > 0 && !cells) || (B > 0 && R > 0 && !page_table) || (tree && (!tree_mask || !tree_base)))
    return set_error(FM_ERR_INVALID_ARG, "%s: required pointer is NULL", who);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pos, 8) || (page_table && !aligned(page_table, 4)) ||
      (seq && !aligned(seq, 4)) || (k > 0 && !aligned(cells, 4)) || (sink_logit && !aligned(sink_logit, 4)) ||
      (lse_out && !aligned(lse_out, 4)) || (tree && (!aligned(tree_mask, 4) || !aligned(tree_base, 8))))
    return set_error(FM_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  const size_t need = attn_workspace_bytes(T, n_h);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return set_error(FM_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 256-byte aligned", who, need);
  int sms = 0;
  fm_status st = check_device(&sms);
  if (st != FM_OK) return st;
  AttnParams p = {};
  if ((st = status_word(&p.status)) != FM_OK) return st;
  p.q = q;
  p.kv_pool = kv_pool;
  p.page_table = page_table;
  p.seq = seq;
  p.pos = pos;
  p.cell_pool = cell_pool;
  p.cells = cells;
  p.sink_logit = sink_logit;
  p.tree_mask = tree ? tree_mask : nullptr;
  p.tree_base = tree_base;
  p.out = out;
  p.lse = lse_out;
  p.kv_page_rows = kv_page_stride / kWidth;
  p.cell_page_rows = cell_page_stride / kWidth;
  p.window = window;
  p.cell_limit = k > 0 ? Pc * kPage : 0;
  p.T = T;
  p.n_h = n_h;
  p.P = (int)P;
  p.B = B;
  p.R = R;
  p.k = k;
  p.n_sink = n_sink;
  p.tree_words = tree_words;
  p.scale = scale;
  return launch_attn(p, sms, workspace, stream);
}

}  // namespace
}  // namespace fm

FM_API size_t fm_csa_attn_workspace(int T, int n_h) {
  if (T < 0 || n_h < 1 || n_h > 1024) return 0;
  return fm::attn_workspace_bytes(T, n_h);
}

FM_API fm_status fm_csa_attn(const uint16_t* q, int T, int n_h, int d, const uint16_t* kv_pool, int64_t P,
                             int64_t kv_page_stride, const int32_t* page_table, int B, int R, const int32_t* seq,
                             const int64_t* pos, int64_t window, int n_sink, const uint16_t* cell_pool, int64_t Pc,
                             int64_t cell_page_stride, const int32_t* cells, int k, const float* sink_logit,
                             float scale, uint16_t* out, float* lse_out, void* workspace, size_t workspace_bytes,
                             fm_stream_t stream) {
  return fm::csa_attn("fm_csa_attn", false, q, T, n_h, d, kv_pool, P, kv_page_stride, page_table, B, R, seq, pos, window,
                      n_sink, cell_pool, Pc, cell_page_stride, cells, k, sink_logit, scale, nullptr, 0, nullptr, out,
                      lse_out, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

FM_API fm_status fm_csa_attn_tree(const uint16_t* q, int T, int n_h, int d, const uint16_t* kv_pool, int64_t P,
                                  int64_t kv_page_stride, const int32_t* page_table, int B, int R, const int32_t* seq,
                                  const int64_t* pos, int64_t window, int n_sink, const uint16_t* cell_pool, int64_t Pc,
                                  int64_t cell_page_stride, const int32_t* cells, int k, const float* sink_logit,
                                  float scale, const uint32_t* tree_mask, int tree_words, const int64_t* tree_base,
                                  uint16_t* out, float* lse_out, void* workspace, size_t workspace_bytes,
                                  fm_stream_t stream) {
  return fm::csa_attn("fm_csa_attn_tree", true, q, T, n_h, d, kv_pool, P, kv_page_stride, page_table, B, R, seq, pos,
                      window, n_sink, cell_pool, Pc, cell_page_stride, cells, k, sink_logit, scale, tree_mask, tree_words,
                      tree_base, out, lse_out, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}
