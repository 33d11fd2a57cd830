// kv_append.cu -- keys and values of new tokens into the paged 8-bit cache, the
// keys turned by their positions on the way, and the tokens' queries turned alike
// ("FlashMemory-DeepSeek-V4" README, "Hyperparameters": YaRN; "compressed_k
// format": E4M3 with fp32 scales).
//     (x[2i], x[2i+1]) -> (x[2i] c - x[2i+1] s, x[2i] s + x[2i+1] c),  (c, s) of pos * theta'_i
//     code = e4m3(x / scale),  scale = 2^e, one for 16 positions of a page and head
// A scale that is a power of two costs a floating format no precision, makes x / scale
// exact, and lets a block that grows be brought to its new scale by an exact product
// and one rounding.
//
// Every element is read once and written once, so the kernel is bound by HBM at large
// sizes and by the chain of dependent loads (offsets, start, page table) at small ones.
// A warp has a block of 16 positions of one head's keys or values in its registers: a
// lane 16 elements (32 bytes in, 16 out) of up to four positions; the largest
// magnitude is one shuffle tree.  The block's (cos, sin) are worked out once per CTA
// for its eight heads, from a 64-bit fixed-point fraction of a turn (as in
// qk_norm_rope.cu: the wrap of one integer product is the reduction).
// Measured: 4096 tokens x (64 + 2 x 8) heads x 128 39.5 us (4.0 TB/s; 66% of the issue slots, then waits for shared memory: more
// than half of the loads' wavefronts are bank conflicts, of the sines), one token 4.4 us.
// A CTA finds its block by itself: sequence b's blocks begin at slot cu[b] / 16 + 2 b,
// which leaves room for the two blocks that a sequence may touch beyond n / 16.
#include <cuda_fp8.h>

#include "grouped.cuh"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;
constexpr int kQVectors = 8 * kThreads;  // 16-byte vectors of queries to a CTA
constexpr int kQTokens = 16;

struct AppendParams {
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  uint8_t *k_pool, *v_pool;
  float *k_scale, *v_scale;
  const int32_t *page_table, *cu;
  const int64_t* start;
  int64_t k_stride_t, v_stride_t, q_stride_t, P, page_stride, scale_stride;
  int T, n_k, d, n_h, B, R, rope_start;
  int slots, slot_ctas;              // CTAs to a slot
  int q_tokens, q_chunks;            // tokens to a CTA, or CTAs to a token
  uint32_t by_pairs, by_chunks, by_token, by_head;  // ceil(2^32 / divisor): of pairs, of 16-element chunks of a head, of a token's and a head's vectors
  unsigned int* status;
  uint64_t turn[kMaxPairs];          // theta'_i / 2 pi in units of 2^-64 turns
};

struct Shared {
  float2 cs[kQTokens][kMaxPairs];
  uint64_t turn[kMaxPairs];
  int64_t pos[kQTokens];
};

// x / divisor for x < 2^16 and divisors up to 2^14 (0: 1): the product's excess stays below 2^32 / divisor.
FM_DEV int quotient(int x, uint32_t by) { return by == 0 ? x : (int)__umulhi((uint32_t)x, by); }

// (cos, sin) of `rows` tokens at sh.pos (negative: left out), by the whole CTA.
FM_DEV void fill_turns(const AppendParams& p, Shared& sh, int rows) {
  const int pairs = (p.d - p.rope_start) >> 1;
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
    const int r = quotient(i, p.by_pairs), j = i - r * pairs;
    if (sh.pos[r] < 0) continue;
    const uint64_t phase = (uint64_t)sh.pos[r] * sh.turn[j];
    float c, s;
    // the signed top word counts half turns in units of 2^-31
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);
    sh.cs[r][j] = make_float2(c, s);
  }
}

FM_DEV float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// The least power of two >= 2^-100 that brings amax to at most 448 = 1.75 * 2^8.
FM_DEV float need_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);  // biased
  e = max(e, 127 - 100);
  return __uint_as_float((uint32_t)e << 23);
}

// Whether y may lie on the other side of the middle between two E4M3 values if it is off by `off`.
FM_DEV bool near_middle(float y, float off) {
  y = fabsf(y);
  const uint32_t exponent = max(__float_as_uint(y) & 0x7F800000u, 121u << 23);  // the steps below 2^-6 are those of 2^-6
  const float per_step = __uint_as_float(((254u << 23) - exponent) + (3u << 23));  // 2^3 / 2^e
  const float q = y * per_step;
  return fabsf(q - floorf(q) - 0.5f) <= off * per_step;
}
// A pair of bf16 entries turned in 64 bits: cos and sin of the phase in units of 2^-64 turns.
FM_DEV double2 turned(float a, float b, uint64_t phase) {
  double s, c;
  sincospi((double)(int64_t)phase * 1.0842021724855044e-19, &s, &c);
  return make_double2(a * c - b * s, a * s + b * c);
}
__device__ __noinline__ float2 turn_exactly(float a, float b, uint64_t phase, float times) {
  const double2 x = turned(a, b, phase);
  return make_float2((float)(x.x * times), (float)(x.y * times));
}

// Whether fp32's rounding of the turn, under 2^-20 of the largest entry (2^-21 of a pair's two, and neither is more than
// 1.42 times the larger turned one), may have carried a block's largest over a border between two scales.
FM_DEV bool near_border(float amax) {
  const int from = (int)(__float_as_uint(amax) & 0x7FFFFFu) - 0x600000;  // in units of 2^-23 of its power of two
  return from >= -16 && from <= 16;  // 2^-20 of 1.75 are 14.7
}
FM_DEV uint32_t codes4(float a, float b, float c, float d) {
  auto fix = [](float x) { return isinf(x) ? __int_as_float(0x7FC00000) : x; };  // the conversion would make it 448
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(fix(a), fix(b)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(fix(c), fix(d)), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

FM_DEV float2 code2_floats(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// A block of keys whose largest entry is a turned one within fp32's error of a border: whether some entry is over it is found
// with the turns in 64 bits, then all is as in append_block.  By a whole warp, from memory; row 0 would be token `t`.  Some
// block in 10^5 needs it.
__device__ __noinline__ void append_at_border(const AppendParams& p, const Shared& sh, int t, int head, int lo, int hi, uint8_t* cells,
                                              float* scale_at, float amax) {
  const int pairs = p.d / 2, lane = threadIdx.x & 31;
  const uint16_t* x = p.k + (int64_t)t * p.k_stride_t + head * p.d;
  const float border = __uint_as_float((__float_as_uint(amax) & 0x7F800000u) | 0x600000u);
  bool over = false;
#pragma unroll 1
  for (int i = lo * pairs + lane; i < hi * pairs; i += 32) {
    const int row = i / pairs, e = 2 * (i - row * pairs);
    const float2 f = bf16x2_floats(*reinterpret_cast<const uint32_t*>(x + row * p.k_stride_t + e));
    const float a = f.x / border, b = f.y / border;
    double2 y = make_double2(f.x, f.y);
    if (e >= p.rope_start) {
      if (!(a * a + b * b > 0.999f)) continue;  // no turned entry is larger than the pair
      y = turned(f.x, f.y, (uint64_t)sh.pos[row] * sh.turn[(e - p.rope_start) >> 1]);
    }
    over |= (finite_abs((float)y.x) > 0.f && fabs(y.x) > border) || (finite_abs((float)y.y) > 0.f && fabs(y.y) > border);
  }
  const float need = need_scale(__any_sync(0xffffffffu, over) ? __uint_as_float(__float_as_uint(border) + 1) : border);
  const float old = lo > 0 ? *scale_at : 0.f;
  const bool keep = lo > 0 && old >= need;
  const float scale = keep ? old : need, inv = 1.f / scale, shrink = old * inv;
#pragma unroll 1
  for (int i = (keep ? lo : 0) * pairs + lane; i < hi * pairs; i += 32) {
    const int row = i / pairs, e = 2 * (i - row * pairs);
    uint16_t* cell = reinterpret_cast<uint16_t*>(cells + row * p.d + e);
    float2 f;
    if (row < lo) {
      f = code2_floats(*cell);
      f = make_float2(f.x * shrink, f.y * shrink);
    } else {
      const float2 v = bf16x2_floats(*reinterpret_cast<const uint32_t*>(x + row * p.k_stride_t + e));
      f = make_float2(v.x * inv, v.y * inv);
      if (e >= p.rope_start) {
        const float2 c = sh.cs[row][(e - p.rope_start) >> 1];
        f = make_float2((v.x * c.x - v.y * c.y) * inv, (v.x * c.y + v.y * c.x) * inv);
        const float off = (fabsf(f.x) + fabsf(f.y)) * 4.76837158e-7f;
        if (near_middle(f.x, off) || near_middle(f.y, off))
          f = turn_exactly(v.x, v.y, (uint64_t)sh.pos[row] * sh.turn[(e - p.rope_start) >> 1], inv);
      }
    }
    *cell = (uint16_t)codes4(f.x, f.y, 0.f, 0.f);
  }
  __syncwarp();
  if (lane == 0 && !keep) *scale_at = scale;
}

FM_DEV uint4 load16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

FM_DEV void append_block(const AppendParams& p, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = blockIdx.x / p.slot_ctas;
  const int item = (blockIdx.x - slot * p.slot_ctas) * kWarps + warp;  // head * 2 + (keys, values)
  // the slot's sequence, and its tokens
  int b = slot, begin = slot, n = 1;
  if (p.cu) {
    b = warp_find(p.B, slot, [&](int i) { return (int64_t)(offset_at(p.cu, i, p.T) / kKvBlock) + 2 * (int64_t)i; });
    begin = offset_at(p.cu, b, p.T);
    n = offset_at(p.cu, b + 1, p.T) - begin;
  }
  const int j = p.cu ? slot - (begin / kKvBlock + 2 * b) : 0;
  const int64_t start = p.start[b];
  if (n <= 0 || j < 0 || start < 0) return;  // the whole CTA, as below
  if (start >= (int64_t)kMaxTable * kKvPage) {
    if (threadIdx.x == 0) atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return;
  }
  const int64_t first = (start / kKvBlock + j) * kKvBlock;  // position of the block's first cell
  if (first >= start + n) return;
  const int64_t page_at = first / kKvPage;
  int page = -1;
  if (page_at < p.R) {
    page = p.page_table[(int64_t)b * p.R + page_at];
    if (page >= p.P) page = -2;
  } else {
    page = -2;
  }
  if (page < 0) {
    if (page == -2 && threadIdx.x == 0) atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return;
  }
  const int lo = (int)(first < start ? start - first : 0);                       // cells below: earlier tokens
  const int hi = (int)(start + n - first < kKvBlock ? start + n - first : kKvBlock);  // from here on: not this call's
  const int sub = (int)(first % kKvPage) / kKvBlock;

  const bool live = item < 2 * p.n_k;
  const int head = item >> 1;
  const bool is_k = (item & 1) == 0;
  uint8_t* cells = (is_k ? p.k_pool : p.v_pool) + page * p.page_stride +
                   ((int64_t)head * kKvPage + first % kKvPage) * p.d;
  float* scale_at = (is_k ? p.k_scale : p.v_scale) + page * p.scale_stride + head * kBlocksPerPage + sub;
  const uint16_t* src = is_k ? p.k : p.v;
  const int64_t stride = is_k ? p.k_stride_t : p.v_stride_t;
  const int chunks = p.d >> 4;  // of 16 elements
  // lane's chunks lane, lane + 32, ...: 32 bytes of a new token, 16 bytes of codes of an earlier one
  uint4 raw[4][2];
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    row[i] = quotient(c, p.by_chunks);
    const int e = 16 * (c - row[i] * chunks);
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    if (!live || row[i] >= hi) {
      row[i] = -1;
    } else if (row[i] >= lo) {
      const uint16_t* x = src + (int64_t)(begin + (int)(first - start) + row[i]) * stride + head * p.d + e;
      raw[i][0] = load16(x);
      raw[i][1] = load16(x + 8);
    } else {
      raw[i][0] = load16(cells + row[i] * p.d + e);
    }
  }
  const float old = live && lo > 0 ? *scale_at : 0.f;
  if (threadIdx.x < kKvBlock) sh.pos[threadIdx.x] = threadIdx.x >= lo && threadIdx.x < hi ? first + threadIdx.x : -1;
  __syncthreads();
  fill_turns(p, sh, kKvBlock);
  __syncthreads();
  if (!live) return;

  // entries 2 m and 2 m + 1 of the lane's chunk i, turned.  Worked out twice, for the largest and for the codes: 64
  // of them kept would halve the blocks of an SM.
  auto entry = [&](int i, int m) {
    const uint4 u = raw[i][m / 4];
    const uint32_t v = m % 4 == 0 ? u.x : m % 4 == 1 ? u.y : m % 4 == 2 ? u.z : u.w;
    float2 f = bf16x2_floats(v);
    const int e = 16 * (lane + 32 * i - row[i] * chunks) + 2 * m - p.rope_start;  // even
    if (is_k && e >= 0) {
      const float2 t = sh.cs[row[i]][e >> 1];
      f = make_float2(f.x * t.x - f.y * t.y, f.x * t.y + f.y * t.x);
    }
    return f;
  };
  float amax = 0.f, turned_amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row[i] >= lo) {
      float x = 0.f;
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const float2 f = entry(i, m);
        x = fmaxf(x, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
      amax = fmaxf(amax, x);
      if (16 * (lane + 32 * i - row[i] * chunks) + 14 >= p.rope_start) turned_amax = fmaxf(turned_amax, x);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const bool at_border = is_k && __any_sync(0xffffffffu, near_border(turned_amax) && turned_amax > 0.99f * amax);
  if (at_border) {  // nothing of the warp's is used behind the call, which so costs the others no registers
    append_at_border(p, sh, begin + (int)(first - start), head, lo, hi, cells, scale_at, amax);
    return;
  }
  const float need = need_scale(amax);
  const bool keep = lo > 0 && old >= need;  // the block's earlier codes stay as they are
  const float scale = keep ? old : need;
  const float inv = 1.f / scale;
  const float shrink = old * inv;
  // Entries over the scale.  One that the turn's rounding in 32 bits (under 2^-21 of the pair) may have carried over a
  // middle between two codes, some 1 of 10^5, is turned again in 64.
  auto scaled = [&](int i, int m) {
    float2 f = entry(i, m);
    f = make_float2(f.x * inv, f.y * inv);
    const int e = 16 * (lane + 32 * i - row[i] * chunks) + 2 * m - p.rope_start;
    if (is_k && e >= 0) {
      const float off = (fabsf(f.x) + fabsf(f.y)) * 4.76837158e-7f;
      if (near_middle(f.x, off) || near_middle(f.y, off)) {
        const uint4 u = raw[i][m / 4];
        const float2 x = bf16x2_floats(m % 4 == 0 ? u.x : m % 4 == 1 ? u.y : m % 4 == 2 ? u.z : u.w);
        f = turn_exactly(x.x, x.y, (uint64_t)sh.pos[row[i]] * sh.turn[e >> 1], inv);
      }
    }
    return f;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row[i] < 0 || (row[i] < lo && keep)) continue;
    const int e = 16 * (lane + 32 * i - row[i] * chunks);
    uint4 out;
    if (row[i] >= lo) {
      uint32_t w[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 a = scaled(i, 2 * m), c = scaled(i, 2 * m + 1);
        w[m] = codes4(a.x, a.y, c.x, c.y);
      }
      out = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t w[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 a = code2_floats(w[m]), c = code2_floats(w[m] >> 16);
        w[m] = codes4(a.x * shrink, a.y * shrink, c.x * shrink, c.y * shrink);
      }
      out = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(cells + row[i] * p.d + e) = out;
  }
  if (lane == 0 && !keep) *scale_at = scale;
}

FM_DEV void turn_queries(const AppendParams& p, Shared& sh, int block) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = p.q_chunks > 1 ? block / p.q_chunks : block * p.q_tokens;
  const int per = p.n_h * (p.d >> 3);  // vectors of a token
  const int v0 = p.q_chunks > 1 ? (block % p.q_chunks) * kQVectors : 0;
  const int tokens = min(p.q_tokens, p.T - t0);
  const int vectors = min(tokens * per - v0, kQVectors);
  uint4 raw[kQVectors / kThreads];
#pragma unroll
  for (int i = 0; i < kQVectors / kThreads; ++i) {
    const int v = v0 + threadIdx.x + i * kThreads;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (v - v0 < vectors) {
      const int t = quotient(v, p.by_token);
      raw[i] = load16(p.q + (int64_t)(t0 + t) * p.q_stride_t + 8 * (v - t * per));
    }
  }
  for (int i = warp; i < tokens; i += kWarps) {
    int b = t0 + i, begin = b;
    bool in = true;
    if (p.cu) {
      b = warp_find(p.B, t0 + i, [&](int s) { return (int64_t)offset_at(p.cu, s, p.T); });
      begin = offset_at(p.cu, b, p.T);
      in = t0 + i >= begin && t0 + i < offset_at(p.cu, b + 1, p.T);
    }
    const int64_t start = p.start[b];
    if (lane == 0) sh.pos[i] = in && start >= 0 ? start + (t0 + i - begin) : -1;
  }
  __syncthreads();
  fill_turns(p, sh, tokens);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQVectors / kThreads; ++i) {
    const int v = v0 + threadIdx.x + i * kThreads;
    if (v - v0 >= vectors) continue;
    const int t = quotient(v, p.by_token);
    if (sh.pos[t] < 0) continue;
    const int in = v - t * per;  // the vector's place in its token, then in its head
    const int e = 8 * (in - quotient(in, p.by_head) * (p.d >> 3));
    uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (e + 2 * m < p.rope_start) continue;
      const float2 f = bf16x2_floats(u[m]), c = sh.cs[t][(e + 2 * m - p.rope_start) >> 1];
      u[m] = floats_bf16x2(f.x * c.x - f.y * c.y, f.x * c.y + f.y * c.x);
    }
    *reinterpret_cast<uint4*>(p.q_out + (int64_t)t0 * p.n_h * p.d + 8 * (int64_t)v) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ Shared sh;
  if (threadIdx.x < ((p.d - p.rope_start) >> 1)) sh.turn[threadIdx.x] = p.turn[threadIdx.x];
  // programmatic dependent launch: what a kernel before wrote may be read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kv = p.slots * p.slot_ctas;
  if ((int)blockIdx.x < kv)
    append_block(p, sh);
  else
    turn_queries(p, sh, blockIdx.x - kv);
}

}  // namespace
}  // namespace fm

using namespace fm;

FM_API fm_status fm_kv_append_fp8(const fm_kv_append_fp8_args* a) {
  const char* who = "fm_kv_append_fp8";
  if (!a) return set_error(FM_ERR_INVALID_ARG, "%s: args is NULL", who);
  const bool q = a->q != nullptr;
  const char* bad = bad_heads(q ? a->n_h : a->n_k, a->n_k, a->d);
  if (bad) return set_error(FM_ERR_INVALID_ARG, "%s: n_h=%d n_k=%d d=%d (%s)", who, a->n_h, a->n_k, a->d, bad);
  if (a->T < 0 || a->T >= 1 << 24) return set_error(FM_ERR_INVALID_ARG, "%s: T=%d (0 <= T < 2^24)", who, a->T);
  bad = bad_cache(a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->P, a->page_stride, a->scale_stride, a->page_table, a->B,
                  a->R, a->n_k, a->d);
  if (bad) return set_error(FM_ERR_INVALID_ARG, "%s: %s", who, bad);
  if (a->rope_dim < 0 || a->rope_dim > a->d || a->rope_dim % 2 != 0)
    return set_error(FM_ERR_INVALID_ARG, "%s: rope_dim=%d (even, 0..d)", who, a->rope_dim);
  if (a->rope_dim > 0 &&
      (!(a->rope_base > 1.0) || !(a->rope_factor >= 1.0) || !(a->rope_orig_len > 0.0) ||
       !(a->rope_beta_fast > a->rope_beta_slow) || isinf(a->rope_base) || isinf(a->rope_factor) ||
       isinf(a->rope_orig_len) || isinf(a->rope_beta_fast - a->rope_beta_slow)))
    return set_error(FM_ERR_INVALID_ARG, "%s: bad rotary parameters", who);
  if (!a->cu_tokens && a->T != a->B)
    return set_error(FM_ERR_INVALID_ARG, "%s: without cu_tokens T=%d must be B=%d", who, a->T, a->B);
  if (a->T == 0 || a->B == 0) return FM_OK;
  if (bad_rows(a->k, a->k_stride_t, a->n_k, a->d) || bad_rows(a->v, a->v_stride_t, a->n_k, a->d) ||
      (q && (bad_rows(a->q, a->q_stride_t, a->n_h, a->d) || !a->q_out || !aligned(a->q_out, 16))))
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: k, v (and q, q_out) need 16-byte aligned pointers and token strides that are multiples of 8 "
                     "and hold the heads",
                     who);
  if (!a->start || !aligned(a->start, 8) || !aligned(a->cu_tokens, 4))
    return set_error(FM_ERR_INVALID_ARG, "%s: start is NULL, or start or cu_tokens misaligned", who);
  AppendParams p = {};
  p.slot_ctas = (2 * a->n_k + kWarps - 1) / kWarps;
  const int64_t slots = a->cu_tokens ? (int64_t)a->T / kKvBlock + 2 * (int64_t)a->B : a->B;
  const int64_t per = q ? (int64_t)a->n_h * a->d / 8 : 0;
  p.q_chunks = (int)((per + kQVectors - 1) / kQVectors);
  p.q_tokens = q && per <= kQVectors ? (int)(kQVectors / per < kQTokens ? kQVectors / per : kQTokens) : 1;
  const int64_t q_ctas = !q ? 0 : p.q_chunks > 1 ? (int64_t)a->T * p.q_chunks : (a->T + p.q_tokens - 1) / p.q_tokens;
  if (slots * p.slot_ctas + q_ctas >= int64_t(1) << 31)
    return set_error(FM_ERR_INVALID_ARG, "%s: T=%d B=%d are too many for %d heads", who, a->T, a->B, a->n_k);
  fm_status st = check_device(nullptr);
  if (st != FM_OK) return st;
  if ((st = status_word(&p.status)) != FM_OK) return st;
  p.slots = (int)slots;
  p.k = a->k;
  p.v = a->v;
  p.q = a->q;
  p.q_out = a->q_out;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.page_table = a->page_table;
  p.cu = a->cu_tokens;
  p.start = a->start;
  p.k_stride_t = a->k_stride_t;
  p.v_stride_t = a->v_stride_t;
  p.q_stride_t = a->q_stride_t;
  p.P = a->P;
  p.page_stride = a->page_stride;
  p.scale_stride = a->scale_stride;
  p.T = a->T;
  p.n_k = a->n_k;
  p.d = a->d;
  p.n_h = q ? a->n_h : 0;
  p.B = a->B;
  p.R = a->R;
  p.rope_start = a->d - a->rope_dim;
  auto by = [](int divisor) { return divisor <= 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + divisor - 1) / divisor); };
  p.by_pairs = by(a->rope_dim / 2);
  p.by_chunks = by(a->d / 16);
  p.by_token = by((int)per);
  p.by_head = by(a->d / 8);
  rope_turns(a->rope_dim, a->rope_base, a->rope_factor, a->rope_orig_len, a->rope_beta_fast, a->rope_beta_slow, p.turn);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(slots * p.slot_ctas + q_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(a->stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_append_kernel, (const AppendParams)p);
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}
