// attn_plain.cuh -- causal attention of grouped heads on the CUDA cores: 16 rows
// (token, head of a group) of one sequence and key head to a block, keys in tiles of
// 32 through shared memory, one pass with the running maximum and sum.
#pragma once

#include "grouped.cuh"

namespace fm {

constexpr int kPlainRows = 16, kPlainKeys = 32, kPlainThreads = 256;

struct PlainParams {
  const uint16_t* q;
  int64_t q_stride_t;
  const int32_t* cu_q;
  uint16_t* out;
  float* lse;
  const float* sink;
  int64_t window;
  float scale;
  int T, n_h, n_k, d, B;
};

// Source: past(b, n) the keys before query 0 of sequence b; clamp(j) the last key at or before
// position j that there can be; held(b, j); value(b, j, head, e, is_k).
template <class Source>
__global__ void __launch_bounds__(kPlainThreads) plain_attn_kernel(const PlainParams p, const Source src) {
  __shared__ float qs[kPlainRows][128], ks[kPlainKeys][129], vs[kPlainKeys][128], ps[kPlainRows][kPlainKeys], f[kPlainRows],
      inv[kPlainRows];
  __shared__ int held[kPlainKeys];
  const int G = p.n_h / p.n_k, head = blockIdx.y, tid = threadIdx.x;
  int b = 0, begin = 0, n = p.T;
  if (p.cu_q) {
    b = warp_find(p.B, blockIdx.x, [&](int i) { return (int64_t)offset_at(p.cu_q, i, p.T) * G / kPlainRows + i; });
    begin = offset_at(p.cu_q, b, p.T);
    n = offset_at(p.cu_q, b + 1, p.T) - begin;
  } else if (p.B != 1) {
    b = begin = blockIdx.x / ((G + kPlainRows - 1) / kPlainRows);
    n = 1;
  }
  const int64_t slot0 = p.cu_q ? (int64_t)begin * G / kPlainRows + b : p.B != 1 ? (int64_t)b * ((G + kPlainRows - 1) / kPlainRows) : 0;
  const int64_t row0 = (blockIdx.x - slot0) * kPlainRows;
  if (row0 < 0 || row0 >= (int64_t)n * G) return;
  const int rows = (int)min((int64_t)kPlainRows, (int64_t)n * G - row0);
  const int64_t past = src.past(b, n);
  for (int i = tid; i < kPlainRows * p.d; i += kPlainThreads) {
    const int r = i / p.d, e = i % p.d;
    float x = 0.f;
    if (r < rows)
      x = __uint_as_float((uint32_t)p.q[(begin + (row0 + r) / G) * p.q_stride_t + (head * G + (row0 + r) % G) * p.d + e] << 16);
    qs[r][e] = x;
  }
  int64_t last = past + (row0 + rows - 1) / G, low = past + row0 / G;
  low = low < p.window ? 0 : low - p.window + 1;
  last = src.clamp(last);
  const int r = tid >> 4, c = tid & 15;  // row, and keys c, c + 16; elements c, c + 16, ...
  const int64_t pos = past + (row0 + r) / G;
  float m = -INFINITY, l = 0.f, o[8] = {};
  for (int64_t j0 = low; j0 <= last; j0 += kPlainKeys) {
    __syncthreads();
    if (tid < kPlainKeys) held[tid] = j0 + tid <= last && src.held(b, j0 + tid);
    __syncthreads();
    for (int i = tid; i < kPlainKeys * p.d; i += kPlainThreads) {
      const int k = i / p.d, e = i % p.d;
      ks[k][e] = held[k] ? src.value(b, j0 + k, head, e, true) : 0.f;
      vs[k][e] = held[k] ? src.value(b, j0 + k, head, e, false) : 0.f;
    }
    __syncthreads();
    float s[2], top = m;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = c + 16 * i;
      float x = 0.f;
      for (int e = 0; e < p.d; ++e) x = fmaf(qs[r][e], ks[k][e], x);
      const int64_t j = j0 + k;
      const bool seen = held[k] && j <= pos && pos - j < p.window;
      s[i] = seen ? x * p.scale : -INFINITY;
      top = fmaxf(top, s[i]);
    }
    for (int o2 = 8; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - base);
    m = top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = expf(s[i] - base);
      ps[r][c + 16 * i] = w;
      sum += w;
    }
    for (int o2 = 8; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
    l = l * keep + sum;
    __syncwarp();
    for (int i = 0; i < 8 && c + 16 * i < p.d; ++i) {
      float x = o[i] * keep;
      for (int k = 0; k < kPlainKeys; ++k)
        if (ps[r][k] != 0.f) x = fmaf(ps[r][k], vs[k][c + 16 * i], x);
      o[i] = x;
    }
  }
  if (r >= rows) return;
  const int64_t t = begin + (row0 + r) / G;
  const int h = head * G + (int)((row0 + r) % G);
  float z = l;
  if (p.sink && l != 0.f) z += expf(p.sink[h] - m);
  for (int i = 0; i < 8 && c + 16 * i < p.d; ++i)
    p.out[(t * p.n_h + h) * p.d + c + 16 * i] = (uint16_t)(floats_bf16x2(l != 0.f ? o[i] / z : 0.f, 0.f) & 0xFFFF);
  if (c == 0 && p.lse) p.lse[t * p.n_h + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

template <class Source>
cudaError_t launch_plain(const PlainParams& p, const Source& src, cudaStream_t s) {
  const int G = p.n_h / p.n_k;
  const int64_t per = (G + kPlainRows - 1) / kPlainRows;
  const int64_t x = p.cu_q ? (int64_t)p.T * G / kPlainRows + p.B + 1 : p.B != 1 ? p.B * per : ((int64_t)p.T * G + kPlainRows - 1) / kPlainRows;
  plain_attn_kernel<<<dim3((unsigned)x, p.n_k), kPlainThreads, 0, s>>>(p, src);
  return cudaGetLastError();
}

}  // namespace fm
