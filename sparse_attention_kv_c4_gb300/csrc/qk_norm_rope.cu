// qk_norm_rope.cu -- RMSNorm of each query and key head and the rotation of its
// last rope_dim entries by the token's position, in one pass; key heads may go
// straight to their cache cells ("DeepSeek-V4 CSA + HCA explained", sec. 2:
// norm and rotary on the chunk cells; "FlashMemory-DeepSeek-V4" README,
// "Hyperparameters": YaRN).
//     y = x / sqrt(mean(x^2) + eps) * g
//     (y[2i], y[2i+1]) -> (y[2i] c - y[2i+1] s, y[2i] s + y[2i+1] c)
// with (c, s) of the angle pos * theta'_i.
//
// Every element is read once and written once, so the kernel is bound by HBM at
// large sizes and by one memory round trip at small ones.  A row (one head of
// one token) is held in registers by a group of lanes, eight elements (16
// bytes) per lane and step: the sum of squares is one shuffle tree, and nothing
// goes through shared memory.  A lane's elements have the same place in every
// row that it handles, so their sines are worked out once per token, a pair to a
// lane, passed by shuffle and kept in registers.
//
// Measured (4096 tokens x 65 heads x 512, 545 MB): 87.5 us, 6.2 TB/s, 92% of the
// measured copy rate.  What it took: the next row's load ahead of the current
// row's sums (107 -> 92 us with the sines below), and few registers -- the gains held
// in registers as well cost an occupancy step and 16 us.
//
// The angle: theta'_i / 2 pi is a 64-bit fixed-point fraction of a turn, so
// pos * fraction modulo 2^64 is the fraction of a turn at pos, exactly reduced
// by the wrap of one integer product (an fp32 angle would lose whole radians at
// positions of 2^20, and FP64 is slow on this chip).
#include <cuda_bf16.h>

#include "fm_common.cuh"
#include "fm_internal.h"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;
constexpr int kPage = 64;

struct NormRopeParams {
  const int64_t* pos;
  const uint16_t* q;
  const uint16_t* q_gain;
  uint16_t* q_out;
  const uint16_t* k;
  const uint16_t* k_gain;
  uint16_t* k_out;
  uint16_t* k_pool;
  const int32_t* k_cell;
  int64_t q_stride_t, k_stride_t, k_page_stride, pool_rows;
  int n_q, n_k, d, rope_start, chunks, rows_per_chunk;
  float inv_d, eps;
  unsigned int* status;
  uint64_t turn[kMaxPairs];  // theta'_i / 2 pi in units of 2^-64 turns
};

FM_DEV float2 unpack2(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
FM_DEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// LPR lanes per row, VPL 16-byte vectors per lane: lane l of a row's group has
// vectors l, l + LPR, ...
template <int LPR, int VPL>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kRowsPerWarp = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPR;
  const int64_t t = blockIdx.x / p.chunks;
  const int chunk = (int)(blockIdx.x % p.chunks);
  const int rows = p.n_q + p.n_k;
  const int row_end = min(rows, (chunk + 1) * p.rows_per_chunk);
  const int nvec = p.d >> 3;
  // programmatic dependent launch: this kernel's launch overlaps the one before
  // it, whose output may be read from here on; the kernel after may get ready
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The warp's first row is on its way before anything else is done.
  const int first = chunk * p.rows_per_chunk + warp * kRowsPerWarp + lane / LPR;
  constexpr int kStep = kWarps * kRowsPerWarp;
  uint4 next[VPL];
  auto fetch = [&](int r) {
    const uint16_t* src = r < p.n_q ? p.q + t * p.q_stride_t + (int64_t)r * p.d
                                    : p.k + t * p.k_stride_t + (int64_t)(r - p.n_q) * p.d;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int v = l + j * LPR;
      next[j] = make_uint4(0, 0, 0, 0);
      if (r < row_end && v < nvec) next[j] = *reinterpret_cast<const uint4*>(src + 8 * v);
    }
  };
  fetch(first);

  // (cos, sin) of the lane's pairs; c = 1, s = 0 before the rotated part.  Lane i
  // works out pairs i, i + 32, ..., and the ones it needs come by shuffle.
  float cs[VPL][4], sn[VPL][4];
#pragma unroll
  for (int j = 0; j < VPL; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[j][i] = 1.f;
      sn[j][i] = 0.f;
    }
  const int pairs = (p.d - p.rope_start) >> 1;
  const uint64_t position = (uint64_t)p.pos[t];
  for (int base = 0; base < pairs; base += 32) {
    float c = 1.f, s = 0.f;
    if (base + lane < pairs) {
      const uint64_t phase = position * p.turn[base + lane];
      // the signed top word counts half turns in units of 2^-31
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * (l + j * LPR) + 2 * i - p.rope_start;  // even
        const int pair = (e >> 1) - base;
        const float cc = __shfl_sync(0xffffffffu, c, pair & 31), ss = __shfl_sync(0xffffffffu, s, pair & 31);
        if (e >= 0 && pair >= 0 && pair < 32) {
          cs[j][i] = cc;
          sn[j][i] = ss;
        }
      }
  }

  for (int r0 = first - lane / LPR; r0 < row_end; r0 += kStep) {
    const int r = r0 + lane / LPR;
    const bool live = r < row_end;
    const bool is_q = r < p.n_q;
    const int head = is_q ? r : r - p.n_q;
    const uint16_t* gain = is_q ? p.q_gain : p.k_gain;
    uint4 x[VPL];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      x[j] = next[j];
      const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(u[i]);
        ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
      }
    }
    fetch(r + kStep);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!live) continue;
    const float inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));

    uint16_t *dst0 = nullptr, *dst1 = nullptr;
    if (is_q) {
      dst0 = p.q_out + (t * p.n_q + head) * p.d;
    } else {
      if (p.k_out != nullptr) dst0 = p.k_out + (t * p.n_k + head) * p.d;
      if (p.k_pool != nullptr) {
        const int64_t cell = p.k_cell[t];
        if (cell >= p.pool_rows) {
          if (l == 0 && head == 0) atomicOr(p.status, FM_DEV_PAGE_RANGE);
        } else if (cell >= 0) {
          dst1 = p.k_pool + (cell / kPage) * p.k_page_stride + ((cell % kPage) * p.n_k + head) * p.d;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int v = l + j * LPR;
      if (v >= nvec) continue;
      uint4 g = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);  // ones
      if (gain != nullptr) g = *reinterpret_cast<const uint4*>(gain + 8 * v);
      const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w}, w[4] = {g.x, g.y, g.z, g.w};
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(u[i]), gg = unpack2(w[i]);
        const float a = f.x * inv * gg.x, b = f.y * inv * gg.y;
        // the unrotated part is written as it is: 0 * inf would make it NaN
        y[i] = 8 * v + 2 * i >= p.rope_start ? pack2(a * cs[j][i] - b * sn[j][i], a * sn[j][i] + b * cs[j][i])
                                             : pack2(a, b);
      }
      const uint4 o = make_uint4(y[0], y[1], y[2], y[3]);
      if (dst0 != nullptr) *reinterpret_cast<uint4*>(dst0 + 8 * v) = o;
      if (dst1 != nullptr) *reinterpret_cast<uint4*>(dst1 + 8 * v) = o;
    }
  }
}

template <int LPR, int VPL>
cudaError_t launch(NormRopeParams& p, int T, int sms, cudaStream_t stream) {
  constexpr int kStep = kWarps * (32 / LPR);  // rows that a block handles at once
  const int rows = p.n_q + p.n_k;
  const int steps = (rows + kStep - 1) / kStep;
  // One block per token where four times the SMs are tokens, else the rows of a
  // token go to several blocks: a 128-thread block at four to an SM took 6.4 us for
  // 76 tokens of 65 x 512, one of 256 threads at eight to an SM 8.3 us (1021 tokens
  // of 40 x 128: 8.5 and 12.4 us).
  int chunks = (int)((4LL * sms + T - 1) / T);
  if (chunks > steps) chunks = steps;
  p.rows_per_chunk = (steps + chunks - 1) / chunks * kStep;
  p.chunks = (rows + p.rows_per_chunk - 1) / p.rows_per_chunk;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)T * p.chunks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<LPR, VPL>, (const NormRopeParams)p);
}

}  // namespace
}  // namespace fm

using namespace fm;

FM_API fm_status fm_qk_norm_rope(const int64_t* pos, int T, int d, int rope_dim, double rope_base, double rope_factor,
                                 double rope_orig_len, double rope_beta_fast, double rope_beta_slow, float eps,
                                 const uint16_t* q, int64_t q_stride_t, int n_q, const uint16_t* q_gain,
                                 uint16_t* q_out, const uint16_t* k, int64_t k_stride_t, int n_k,
                                 const uint16_t* k_gain, uint16_t* k_out, uint16_t* k_pool, int64_t P,
                                 int64_t k_page_stride, const int32_t* k_cell, fm_stream_t stream) {
  const char* who = "fm_qk_norm_rope";
  if (T < 0 || n_q < 0 || n_k < 0 || n_q > 4096 || n_k > 4096 || n_q + n_k > 4096)
    return set_error(FM_ERR_INVALID_ARG, "%s: bad sizes T=%d n_q=%d n_k=%d (n_q + n_k <= 4096)", who, T, n_q, n_k);
  if (d < 8 || d > 1024 || d % 8 != 0 || rope_dim < 0 || rope_dim > d || rope_dim > 2 * kMaxPairs || rope_dim % 2 != 0)
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: d=%d rope_dim=%d (d: a multiple of 8 up to 1024; rope_dim: even, up to min(d, 256))", who, d,
                     rope_dim);
  if (rope_dim > 0 && (!(rope_base > 1.0) || !(rope_factor >= 1.0) || !(rope_orig_len > 0.0) ||
                       !(rope_beta_fast > rope_beta_slow) || isinf(rope_base) || isinf(rope_factor) ||
                       isinf(rope_orig_len) || isinf(rope_beta_fast - rope_beta_slow)))
    return set_error(FM_ERR_INVALID_ARG, "%s: bad rotary parameters", who);
  if (!(eps >= 0.0f)) return set_error(FM_ERR_INVALID_ARG, "%s: eps=%g", who, (double)eps);
  if (T == 0 || n_q + n_k == 0) return FM_OK;
  if (!pos || (n_q > 0 && (!q || !q_out)) || (n_k > 0 && (!k || (!k_out && !k_pool))))
    return set_error(FM_ERR_INVALID_ARG, "%s: required pointer is NULL", who);
  const bool pool = n_k > 0 && k_pool != nullptr;
  if (pool && (!k_cell || P < 0 || P > (int64_t(1) << 25) || k_page_stride < (int64_t)kPage * n_k * d ||
               k_page_stride % 8 != 0))
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: a pool needs k_cell, 0 <= P <= 2^25 and a page stride (%lld) of at least 64 * n_k * d, a "
                     "multiple of 8",
                     who, (long long)k_page_stride);
  if ((n_q > 0 && (q_stride_t < (int64_t)n_q * d || q_stride_t % 8 != 0)) ||
      (n_k > 0 && (k_stride_t < (int64_t)n_k * d || k_stride_t % 8 != 0)))
    return set_error(FM_ERR_INVALID_ARG, "%s: token strides must be multiples of 8 and hold the heads", who);
  if (!aligned(pos, 8) ||
      (n_q > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || (q_gain && !aligned(q_gain, 16)))) ||
      (n_k > 0 && (!aligned(k, 16) || (k_out && !aligned(k_out, 16)) || (k_gain && !aligned(k_gain, 16)))) ||
      (pool && (!aligned(k_pool, 16) || !aligned(k_cell, 4))))
    return set_error(FM_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  int sms = 0;
  fm_status st = check_device(&sms);
  if (st != FM_OK) return st;
  NormRopeParams p = {};
  if ((st = status_word(&p.status)) != FM_OK) return st;
  p.pos = pos;
  p.q = q;
  p.q_gain = q_gain;
  p.q_out = q_out;
  p.k = k;
  p.k_gain = k_gain;
  p.k_out = k_out;
  p.k_pool = pool ? k_pool : nullptr;
  p.k_cell = k_cell;
  p.q_stride_t = q_stride_t;
  p.k_stride_t = k_stride_t;
  p.k_page_stride = k_page_stride;
  p.pool_rows = P * kPage;
  p.n_q = n_q;
  p.n_k = n_k;
  p.d = d;
  p.rope_start = d - rope_dim;
  p.inv_d = 1.0f / (float)d;
  p.eps = eps;
  // the frequencies of this thread's last parameters are kept: 32 powers take 2 us
  struct Table {
    int rope_dim;
    double base, factor, orig_len, beta_fast, beta_slow;
    uint64_t turn[kMaxPairs];
  };
  static thread_local Table kept = {};
  if (rope_dim > 0 && (kept.rope_dim != rope_dim || kept.base != rope_base || kept.factor != rope_factor ||
                       kept.orig_len != rope_orig_len || kept.beta_fast != rope_beta_fast ||
                       kept.beta_slow != rope_beta_slow)) {
    kept.rope_dim = 0;
    for (int i = 0; i < rope_dim / 2; ++i) {
      const double f = yarn_freq(i, rope_dim, rope_base, rope_factor, rope_orig_len, rope_beta_fast, rope_beta_slow);
      kept.turn[i] = (uint64_t)ldexp(f / 6.283185307179586476925286766559, 64);  // f <= 1: at most 2^61.4
    }
    kept.base = rope_base;
    kept.factor = rope_factor;
    kept.orig_len = rope_orig_len;
    kept.beta_fast = rope_beta_fast;
    kept.beta_slow = rope_beta_slow;
    kept.rope_dim = rope_dim;
  }
  for (int i = 0; i < rope_dim / 2; ++i) p.turn[i] = kept.turn[i];
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int nvec = d / 8;
  cudaError_t e;
  if (nvec <= 4)
    e = launch<4, 1>(p, T, sms, s);
  else if (nvec <= 8)
    e = launch<8, 1>(p, T, sms, s);
  else if (nvec <= 16)
    e = launch<16, 1>(p, T, sms, s);
  else if (nvec <= 32)
    e = launch<32, 1>(p, T, sms, s);
  else if (nvec <= 64)
    e = launch<32, 2>(p, T, sms, s);
  else
    e = launch<32, 4>(p, T, sms, s);
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}

FM_API fm_status fm_qk_norm_rope_packed(const fm_qk_norm_rope_args* a) {
  if (!a) return set_error(FM_ERR_INVALID_ARG, "fm_qk_norm_rope_packed: args is NULL");
  return fm_qk_norm_rope(a->pos, a->T, a->d, a->rope_dim, a->rope_base, a->rope_factor, a->rope_orig_len,
                         a->rope_beta_fast, a->rope_beta_slow, a->eps, a->q, a->q_stride_t, a->n_q, a->q_gain, a->q_out,
                         a->k, a->k_stride_t, a->n_k, a->k_gain, a->k_out, a->k_pool, a->P, a->k_page_stride, a->k_cell,
                         a->stream);
}
