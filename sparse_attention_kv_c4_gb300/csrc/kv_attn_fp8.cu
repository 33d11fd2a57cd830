// kv_attn_fp8.cu -- attention of grouped heads over the paged 8-bit cache: decode
// steps and a few (drafted) tokens a sequence ("FlashMemory-DeepSeek-V4" README,
// "compressed_k format": E4M3 codes with fp32 scales).
//     s_j = scale (q . k_j),  out = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink}),
// k_j = e4m3(code) * scale of its block of 16 tokens and head, v_j alike.
//
// A cell is read once for each tile of up to 24 (d <= 64: 32) of the rows (token, query head) that share
// its head, 2 d bytes for 4 d flops a row: bound by HBM up to 16 rows, by the warps' own work beyond.
//
// The work is the list of units (sequence, key head, row tile, page of 64 tokens), cut into
// as many equal runs as there are warps, seven to an SM, whatever the sequences' lengths;
// a warp works out its run from the offsets by itself, and a lane of the CTA's eighth warp brings its tiles
// (a page of a head) by TMA (two or three stages each, swizzled):
//   S^T = K Q^T   m16n8k16, 16 keys (one block of scales) x 8 rows, fp16 operands:
//                 E4M3 is exact in fp16, queries are scaled to 2^14 by row
//   softmax       against a running reference that moves only when a score
//                 passes it by 8 (in log2): most tiles need no reduction over lanes
//   O^T += V^T P^T  the weights times the block's scale of V in fp16, kept in its range by
//                 a unit of their own, which follows the tiles' largest weight times scale up and down
// The transposed products take rows in eights, and their operands come from the
// cache's rows as they lie: a lane's 16 bytes of a key are four steps of K16 (the order of
// the contraction is free), ldmatrix transposes V by pairs of bytes.  mma.sync, not tcgen05:
// codes have to pass through registers to become fp16, and a few rows leave either idle.
// An item (sequence, key head, row tile) that spans runs is joined by kv_join_kernel, in a fixed order.
// (With a run to an SM and a join of its warps' results at each item's end, an end cost some 4 us: 30 requests
// of 1K to 32K took 209 us where 30 of 17K took 164.)
// Measured, calls queued on a stream, inputs in rotation: 30 tokens x 64 heads over 1K to 32K cells of 8 x 128
// 173 us (6.0 TB/s; 161 us the first kernel, 96% of the measured copy rate), one token x 32 heads over 1M cells of
// 4 x 128 176 us, 8 x 5 drafted tokens x 40 heads over 8191 cells of 8 x 64 43.5 us, 37 cells 10 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "grouped.cuh"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kWarps = 7;                // with the producer two to a scheduler: 255 registers each
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kScan = 128;               // parts of the sequences whose units are counted
constexpr int kMaxCtas = 160;
constexpr int kMaxRuns = kMaxCtas * kWarps;
constexpr int kRunsPerBlock = 4;        // of the join
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;           // how far a score (in log2) may pass its reference
// Weights times V's scale go to fp16 as 2^(x + g), x the logarithm of such a product relative to the row's reference of
// scores.  A row's g puts a tile's largest at 2^12, so that the heaviest weight is a power of two and loses nothing, and
// moves, up or down, when a tile's largest passes 2^15 (fp16 ends at 65504) or stays below 2^-3: each is then off by 2^-11
// of itself or 2^-22 of its tile's largest (half of fp16's smallest step).  (With a range that only went up, a key e^16
// over the others whose value was zero left them to fp16's subnormals: 12% off.)  O, in fp32, is in units of 2^-g; g goes
// up no further than leaves O below 2^kTop.  All of it is relative to the reference: scores of 10^9 lose
// fp32's digits, but no range.
constexpr float kLead = 12.f, kMost = 15.f, kLeast = -3.f, kTop = 100.f;
constexpr float kUnset = 3e38f;         // g of a row that has not met a key
constexpr float kNoKey = -3.402823466e38f;  // a part's reference where it has none

template <int D>
struct Layout {
  static constexpr int kTile = kKvPage * D;          // bytes of a page and head's keys, and of its values
  static constexpr int kDepth = D == 64 ? 3 : 2;     // tiles of a warp in shared memory
};

struct KvParams {
  const uint16_t* q;
  const float *k_scale, *v_scale, *sink;
  const int32_t *page_table, *cu;
  const int64_t* start;
  uint16_t* out;
  float* lse;
  float* part_o;      // [2 runs][rows][D] unnormalised outputs
  float4* part_ml;    // [2 runs][rows] (reference of scores, g, sum)
  int4* part_item;    // [runs] (sequence, head, row tile, runs that follow) of the item that a run begins and does not end
  int64_t q_stride_t, scale_stride, window;
  int T, n_h, n_k, d, G, P, B, R, runs;
  float scale;
  unsigned int* status;
};

template <int D>
struct Smem {
  static constexpr int kDepth = Layout<D>::kDepth;
  uint8_t kv[kWarps][kDepth][2][Layout<D>::kTile];  // 1024-byte aligned
  float scales[kWarps][kDepth][2][kBlocksPerPage];
  uint64_t full[kWarps][kDepth], empty[kWarps][kDepth];
  int held[kWarps][kDepth];
  int64_t before[kScan + 1];                        // units before each part's sequences
  int abort;
};

// A sequence of the call and the pages that its rows see.
struct Seq {
  int64_t start;
  int begin, n, tiles, low, pages;  // low page, number of pages (at least one unit: a row without keys is written too)
  bool none;                        // no page at all
};

template <int NT>
FM_DEV Seq sequence(const KvParams& p, int b) {
  Seq s;
  s.begin = b;
  s.n = 1;
  if (p.cu) {
    s.begin = offset_at(p.cu, b, p.T);
    s.n = max(offset_at(p.cu, b + 1, p.T) - s.begin, 0);
  }
  s.start = p.start[b];
  s.tiles = (int)(((int64_t)s.n * p.G + 8 * NT - 1) / (8 * NT));
  const int64_t last = s.start + s.n - 1, limit = (int64_t)p.R * kKvPage;
  const int64_t low = s.start < p.window ? 0 : s.start - p.window + 1;
  s.none = s.start < 0 || s.start >= (int64_t(1) << 62) || p.window == 0 || low >= limit || p.R == 0;
  s.low = s.none ? 0 : (int)(low / kKvPage);
  s.pages = s.none ? 1 : (int)((last < limit ? last : limit - 1) / kKvPage) - s.low + 1;
  return s;
}
template <int NT>
FM_DEV int64_t units_of(const KvParams& p, int b) {
  const Seq s = sequence<NT>(p, b);
  return (int64_t)s.tiles * p.n_k * s.pages;
}

// First unit of run r.
FM_DEV int64_t run_begin(int64_t units, int r, int runs) {
  const int64_t each = units / runs, more = units % runs;
  return r * each + min((int64_t)r, more);
}

FM_DEV uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
FM_DEV uint32_t floats_half2(float a, float b) { return half2_bits(__floats2half2_rn(a, b)); }
// Four codes as two pairs of fp16 (exact).
FM_DEV void codes_halves(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
FM_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
FM_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
FM_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
FM_DEV void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FM_DEV uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
FM_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

FM_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Row r of eight in a fragment is key row_key(r) of its eight keys, and a cell's 16-byte
// chunk lies where the TMA's swizzle put it: with this order the eight lanes of a
// 16-byte load, and the eight rows of an ldmatrix, meet eight different chunks.
template <int D>
FM_DEV int row_key(int r) { return D == 128 ? (r >> 1) | ((r & 1) << 2) : r; }
template <int D>
FM_DEV uint32_t chunk_at(int key, int chunk) {
  return key * D + 16 * (D == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3));
}

// ---------------------------------------------------------------------------------------
// consumers

template <int D, int NT>
struct Rows {
  uint32_t q[D / 16][NT][2];    // B fragments: row g of each eight, elements of the lane's chunks
  float f[NT][2];               // columns 2c, 2c + 1: factor from q . code to scores in log2 (times K's scale)
  int pos[NT][2], low[NT][2];   // the last and the first position that they see (last below first: no row)
  float m[NT][2], g[NT][2], l[NT][2];  // reference of scores, unit of the weights, sum
  float o[D / 16][NT][4];       // (d = 16 j + 2 g, column 2c), (.., 2c + 1), (d + 1, 2c), (d + 1, 2c + 1)
  int least, most, low_least, low_most;  // of the tile's first and last row
};

template <int D, int NT>
FM_DEV void load_rows(const KvParams& p, const Seq& s, int head, int tile, Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rows = s.n * p.G, row0 = tile * 8 * NT;
  // positions past the table's reach are alike: 2^30 is one
  auto last_of = [&](int row) { return (int)max(min(s.start + row / p.G, (int64_t)1 << 30), (int64_t)-1); };
  auto low_of = [&](int row) {
    const int64_t pos = s.start + row / p.G;
    return pos < p.window ? 0 : (int)min(pos - p.window + 1, (int64_t)1 << 30);
  };
  const int row1 = min(rows, row0 + 8 * NT) - 1;
  w.least = last_of(row0);
  w.most = last_of(row1);
  w.low_least = low_of(row0);
  w.low_most = low_of(row1);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + 8 * nt + g;
    const bool in = r < rows;
    const int t = in ? r / p.G : 0;
    const uint16_t* src = p.q + (int64_t)(s.begin + t) * p.q_stride_t + (head * p.G + (in ? r - t * p.G : 0)) * p.d;
    uint32_t raw[D / 64][8];
    float top = 0.f;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const int e = 16 * (c + 4 * h);
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (in && e < p.d) {
        a = *reinterpret_cast<const uint4*>(src + e);
        b = *reinterpret_cast<const uint4*>(src + e + 8);
      }
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        raw[h][i] = u[i];
        const float2 x = bf16x2_floats(u[i]);
        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(14 - exponent) brings the row's largest to [2^14, 2^15); the two factors of a scaling by
    // more than 2^127 are applied one after the other
    int e = top > 0.f && top < INFINITY ? (int)(__float_as_uint(top) >> 23) - 127 : 14;
    e = max(e, -110) - 14;
    const float down = __uint_as_float((uint32_t)(127 - (e >> 1)) << 23), down2 = __uint_as_float((uint32_t)(127 - (e - (e >> 1))) << 23);
    const float up = __uint_as_float((uint32_t)(127 + (e >> 1)) << 23), up2 = __uint_as_float((uint32_t)(127 + (e - (e >> 1))) << 23);
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = bf16x2_floats(raw[h][i]);
        w.q[4 * h + (i >> 1)][nt][i & 1] = floats_half2(x.x * down * down2, x.y * down * down2);
      }
    const float factor = p.scale * kLog2e * up * up2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.f[nt][i] = __shfl_sync(0xffffffffu, factor, 4 * (2 * c + i));
      const int row = row0 + 8 * nt + 2 * c + i;
      w.pos[nt][i] = row < rows ? last_of(row) : -1;
      w.low[nt][i] = row < rows ? low_of(row) : 0;
      w.m[nt][i] = 0.f;
      w.g[nt][i] = kUnset;
      w.l[nt][i] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[j][nt][i] = 0.f;
}

// Blocks of 16 keys from block `at` of a page on, `Blocks` of them.  partial: some row does not see some key.
template <int D, int NT, int Blocks>
FM_DEV void key_blocks(uint32_t kv_smem, const float (*scales)[kBlocksPerPage], int at, int page_first, bool partial,
                       Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint32_t k_smem = kv_smem + 16 * at * D, v_smem = k_smem + Layout<D>::kTile;  // 16 rows keep the swizzle's phase
  const int first = page_first + 16 * at;
  float s[Blocks][NT][4];
#pragma unroll
  for (int block = 0; block < Blocks; ++block) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[block][nt][i] = 0.f;
    const int key = 16 * block + row_key<D>(g);
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const uint4 lo = lds16(k_smem + chunk_at<D>(key, c + 4 * h)), hi = lds16(k_smem + chunk_at<D>(key + 8, c + 4 * h));
      const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a0, a1, a2, a3;
        codes_halves(a[i], a0, a2);
        codes_halves(b[i], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(s[block][nt], a0, a1, a2, a3, w.q[4 * h + i][nt][0], w.q[4 * h + i][nt][1]);
      }
    }
  }
  float ks[Blocks], vs[Blocks], log_vs[Blocks];
#pragma unroll
  for (int block = 0; block < Blocks; ++block) {
    ks[block] = scales[0][at + block];
    vs[block] = scales[1][at + block];
    log_vs[block] = fmaxf(__log2f(vs[block]), -200.f);  // a scale of zero has one too
  }
  // scores in log2
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int block = 0; block < Blocks; ++block)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[block][nt][i] *= ks[block] * w.f[nt][i & 1];
  if (partial) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int block = 0; block < Blocks; ++block)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = first + 16 * block + row_key<D>(g) + 8 * (i >> 1);
          if (j > w.pos[nt][i & 1] || j < w.low[nt][i & 1]) s[block][nt][i] = -INFINITY;
        }
  }
  // the largest of the lane's over their references, and of them times V's scale
  bool passes = false, low = false;
  float top[NT][2], topv[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[nt][i] = topv[nt][i] = -INFINITY;
#pragma unroll
      for (int block = 0; block < Blocks; ++block) {
        const float x = fmaxf(s[block][nt][i], s[block][nt][i + 2]) - w.m[nt][i];
        top[nt][i] = fmaxf(top[nt][i], x);
        topv[nt][i] = fmaxf(topv[nt][i], x + log_vs[block]);
      }
      const float x = topv[nt][i] + w.g[nt][i];
      passes |= top[nt][i] > kSlack || x > kMost;
      low |= x < kLeast;
    }
  if (__any_sync(0xffffffffu, passes || low)) {
    if (__any_sync(0xffffffffu, low)) {  // the lane's keys are; the column's?
      uint32_t some = 0, near = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t bit = 1u << (8 * nt + 4 * i);
          some |= topv[nt][i] > -INFINITY ? bit : 0u;
          near |= topv[nt][i] + w.g[nt][i] >= kLeast ? bit : 0u;
        }
      some = __reduce_or_sync(0xffffffffu, some << c);
      near = __reduce_or_sync(0xffffffffu, near << c);
      if ((some & ~near) != 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = topv[nt][i], most = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) most = fmaxf(most, fmaxf(fabsf(w.o[j][nt][i]), fabsf(w.o[j][nt][i + 2])));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            float up = 0.f;
            if (x > -INFINITY && x + w.g[nt][i] < kLeast) up = fminf(kLead - x - w.g[nt][i], fmaxf(kTop - __log2f(most), 0.f));
            w.g[nt][i] += up;
            // 2^up may pass 2^127 where O is small; where O is zero any factor will do
            const float keep = exp2_fast(fminf(0.5f * up, 126.f));
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              w.o[j][nt][i] = w.o[j][nt][i] * keep * keep;
              w.o[j][nt][i + 2] = w.o[j][nt][i + 2] * keep * keep;
            }
          }
      }
    }
    if (__any_sync(0xffffffffu, passes)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = -INFINITY, xv = -INFINITY;
#pragma unroll
          for (int block = 0; block < Blocks; ++block) x = fmaxf(x, fmaxf(s[block][nt][i], s[block][nt][i + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          // the reference of scores: the largest so far; of the row's first keys even if it is below zero
          const bool first_keys = w.g[nt][i] == kUnset && x > -INFINITY;
          const float m = first_keys ? x : fmaxf(w.m[nt][i], x), by = m - w.m[nt][i];
#pragma unroll
          for (int block = 0; block < Blocks; ++block) xv = fmaxf(xv, fmaxf(s[block][nt][i], s[block][nt][i + 2]) - m + log_vs[block]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) xv = fmaxf(xv, __shfl_xor_sync(0xffffffffu, xv, o));
          const float from = first_keys ? INFINITY : w.g[nt][i] + by, to = fminf(from, kLead - xv), keep = exp2_fast(to - from);
          w.l[nt][i] *= first_keys ? 0.f : exp2_fast(-by);
          w.m[nt][i] = m;
          w.g[nt][i] = to;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            w.o[j][nt][i] *= keep;
            w.o[j][nt][i + 2] *= keep;
          }
        }
    }
  }
  // weights, their sums, and the weights times V's scale in fp16 as the second product's operand
  uint32_t pt[Blocks][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float half[2];  // of the way to the weights' unit: the whole may pass 2^127
#pragma unroll
    for (int i = 0; i < 2; ++i) half[i] = exp2_fast(fminf(0.5f * w.g[nt][i], 126.f));
#pragma unroll
    for (int block = 0; block < Blocks; ++block) {
      float x[4], unit[2];
      // Rounded towards zero, so that what passes fp32 ends at its largest number: the weight it then meets is
      // below 2^-112 of the row's largest, or zero, and zero times infinity is no zero.
#pragma unroll
      for (int i = 0; i < 2; ++i) unit[i] = __fmul_rz(__fmul_rz(vs[block], half[i]), half[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = exp2_fast(s[block][nt][i] - w.m[nt][i & 1]);
        w.l[nt][i & 1] += e;
        x[i] = e * unit[i & 1];
      }
      pt[block][nt][0] = transpose8x8(floats_half2(x[0], x[1]));
      pt[block][nt][1] = transpose8x8(floats_half2(x[2], x[3]));
    }
  }
  // O^T += V^T P^T.  Lanes 0-7 address the rows of the matrix (keys 0-7, chunk 2j), 8-15 (8-15, 2j), 16-23 (0-7,
  // 2j + 1), 24-31 (8-15, 2j + 1)
#pragma unroll
  for (int block = 0; block < Blocks; ++block) {
    const int key = 16 * block + 8 * ((lane >> 3) & 1) + row_key<D>(lane & 7);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint32_t r[4];
      ldmatrix4_trans(r, v_smem + chunk_at<D>(key, 2 * j + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a0, a1, a2, a3;
        codes_halves(__byte_perm(r[2 * i], 0, 0x3120), a0, a1);
        codes_halves(__byte_perm(r[2 * i + 1], 0, 0x3120), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(w.o[2 * j + i][nt], a0, a1, a2, a3, pt[block][nt][0], pt[block][nt][1]);
      }
    }
  }
}

// Cells of V that are no keys of any row become zeros: they may hold NaN, and zero times that is NaN.  A NaN
// that some rows see and others do not is made a zero too, and put into the outputs of those that
// see it (E4M3 has no infinities).  The same for the scales of V: a block that is no row's may have any scale, and one that is
// no number stays with the rows that see the block.
template <int D, int NT>
FM_DEV void clean_values(uint8_t* v, float* scales, int first, Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  bool bad = false;
#pragma unroll 1
  for (int i = lane; i < kKvPage * (D / 16); i += 32) {
    const int key = first + i / (D / 16);
    uint4* cell = reinterpret_cast<uint4*>(v + 16 * i);  // some chunk of the key's row: the swizzle stays within it
    if (key > w.most || key < w.low_least) {
      *cell = make_uint4(0, 0, 0, 0);
    } else if (key > w.least || key < w.low_most) {
      const uint4 u = *cell;
      const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) bad |= (((a[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
    }
  }
  __syncwarp();
  if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
    for (int key = 0; key < kKvPage; ++key) {
      const int at = first + key;
      if (at > w.most || at < w.low_least || (at <= w.least && at >= w.low_most)) continue;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint8_t* cell = v + chunk_at<D>(key, j) + 2 * g + k;
          const bool nan = (*cell & 0x7F) == 0x7F;
          __syncwarp();
          if (!nan) continue;
          *cell = 0;  // of the four lanes that read it, all
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (at <= w.pos[nt][i] && at >= w.low[nt][i]) w.o[j][nt][i + 2 * k] = __int_as_float(0x7FC00000);
        }
    }
  }
#pragma unroll 1
  for (int block = 0; block < kBlocksPerPage; ++block) {
    const int at = first + kKvBlock * block, end = at + kKvBlock - 1;
    const bool none = at > w.most || end < w.low_least;
    if (!none && fabsf(scales[block]) < INFINITY) continue;  // the same in all lanes
    __syncwarp();
    scales[block] = 0.f;
    if (none) continue;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (at <= w.pos[nt][i] && end >= w.low[nt][i])
#pragma unroll
          for (int j = 0; j < D / 16; ++j) w.o[j][nt][i] = w.o[j][nt][i + 2] = __int_as_float(0x7FC00000);
  }
  __syncwarp();
}

// A row's factors from its sum of weights times codes, in units of 2^e relative to the reference m, to the output, one after
// the other (the product may leave fp32's range), and its log-sum-exp.
FM_DEV float2 row_factors(const KvParams& p, int h, float m, float e, float l) {
  if (l == 0.f) return make_float2(0.f, 0.f);
  float z = l, down = 0.f;
  if (p.sink) {  // it may be far over the scores, or far below
    const float sink = p.sink[h] * kLog2e - m;
    down = fmaxf(sink, 0.f);
    z = l * exp2_fast(-down) + exp2_fast(sink > 0.f ? 0.f : sink);
  }
  const float half = exp2_fast(0.5f * (e - down));
  return make_float2(half, half / z);
}
FM_DEV float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f; }

// Whether the phase with the given parity is complete, without a wait.
FM_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The producer: lane w brings the tiles of warp w's run, as they become free.
template <int D, int NT>
FM_DEV void bring_tiles(const KvParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, Smem<D>& sh, int64_t units, int runs,
                        int share) {
  using L = Layout<D>;
  constexpr int kDepth = L::kDepth;
  const int warp = threadIdx.x & 31;   // whose tiles the lane brings
  const int run = warp * gridDim.x + blockIdx.x;
  int64_t left = 0, local = 0;
  int b = 0;
  Seq s = {};
  auto enter = [&]() {
    s = sequence<NT>(p, b);
    if (s.tiles > 0 && p.window > 0 && (s.none ? s.start >= 0 : s.start + s.n - 1 >= (int64_t)p.R * kKvPage))
      atomicOr(p.status, FM_DEV_PAGE_RANGE);
  };
  if (warp < kWarps && run < runs) {
    const int64_t u0 = run_begin(units, run, runs);
    left = run_begin(units, run + 1, runs) - u0;
    if (left > 0) {
      int lo = 0;
      for (int hi = kScan; hi - lo > 1;) {
        const int mid = (lo + hi) / 2;
        (sh.before[mid] <= u0 ? lo : hi) = mid;
      }
      b = lo * share;
      local = u0 - sh.before[lo];
      for (int64_t mine; local >= (mine = units_of<NT>(p, b)); ++b) local -= mine;
      enter();
    }
  }
  int item = 0, page = 0, row = 0, entry = -1, stage = 0;
  uint32_t round = 0, issued = 0;
  auto look_up = [&]() { entry = s.none ? -1 : p.page_table[(int64_t)b * p.R + s.low + page]; };
  if (left > 0) {
    item = (int)(local / s.pages);
    page = (int)(local - (int64_t)item * s.pages);
    row = item / s.tiles * kKvPage;
    look_up();
  }
  uint64_t since = 0;
  bool ok = true;
#pragma unroll 1
  for (uint32_t idle = 0; __any_sync(0xffffffffu, left > 0);) {
    const bool ready = left > 0 && (issued < kDepth || mbar_test(&sh.empty[warp][stage], round ^ 1));
    if (ready) {
      int at = entry;
      if (at >= p.P) {
        atomicOr(p.status, FM_DEV_PAGE_RANGE);
        at = -1;
      }
      uint64_t* full = &sh.full[warp][stage];
      sh.held[warp][stage] = at >= 0;
      if (at >= 0) {
        mbar_arrive_expect_tx(full, 2 * L::kTile + 2 * kBlocksPerPage * 4);
        tma_load_3d(sh.kv[warp][stage][0], &k_map, full, 0, row, at);
        tma_load_3d(sh.kv[warp][stage][1], &v_map, full, 0, row, at);
        const int64_t x = at * p.scale_stride + row / kKvBlock;
        bulk_load(sh.scales[warp][stage][0], p.k_scale + x, 16, full);
        bulk_load(sh.scales[warp][stage][1], p.v_scale + x, 16, full);
      } else {
        mbar_arrive(full);
      }
      ++issued;
      stage = stage + 1 == kDepth ? 0 : stage + 1;
      round ^= stage == 0;
      --left;
      if (++page == s.pages) {
        page = 0;
        if (++item == s.tiles * p.n_k && left > 0) {
          item = 0;
          do {
            ++b;
            enter();
          } while (s.tiles == 0);
        }
        row = item / s.tiles * kKvPage;
      }
      if (left > 0) look_up();
    }
    if (__any_sync(0xffffffffu, ready)) {
      idle = 0;
      continue;
    }
    __nanosleep(100);  // looking again at once would take issue slots from the warps that work
    if ((++idle & 63) == 1) {  // a bounded wait, as wait_bar's
      const uint64_t now = globaltimer();
      if (idle == 1) since = now;
      const bool late = now - since > FM_WAIT_LIMIT_NS;
      if (late && *(volatile int*)&sh.abort == 0) atomicOr(p.status, FM_DEV_TIMEOUT);
      if (late) *(volatile int*)&sh.abort = 1;
      if (__any_sync(0xffffffffu, *(volatile int*)&sh.abort != 0)) {
        ok = false;
        break;
      }
    }
  }
  if (ok || warp >= kWarps) return;
  // gave up: the copies in flight land before the CTA's memory is another's
  for (uint32_t i = issued > kDepth ? issued - kDepth : 0; i < issued; ++i)
    mbar_wait_drain(&sh.full[warp][i % kDepth], (i / kDepth) & 1);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_kernel(const __grid_constant__ CUtensorMap k_map,
                                                              const __grid_constant__ CUtensorMap v_map,
                                                              const __grid_constant__ KvParams p) {
  constexpr int kDepth = Layout<D>::kDepth;
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  Smem<D>& sh = *reinterpret_cast<Smem<D>*>(raw_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    tma_prefetch(&k_map);
    tma_prefetch(&v_map);
    sh.abort = 0;
  }
  if (warp < kWarps && lane < kDepth) {
    mbar_init(&sh.full[warp][lane], 1);
    mbar_init(&sh.empty[warp][lane], 1);
  }
  fence_mbar_init();
  // programmatic dependent launch: what a kernel before wrote may be read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // units before each of kScan shares of the sequences
  const int share = (p.B + kScan - 1) / kScan;
  if (warp < kScan / 32) {
    int64_t mine = 0;
    for (int i = 0; i < share && tid * (int64_t)share + i < p.B; ++i) mine += units_of<NT>(p, tid * share + i);
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sh.before[warp] = incl;
    named_bar_sync(1, kScan);
    for (int i = 0; i < warp; ++i) incl += sh.before[i];
    named_bar_sync(1, kScan);
    sh.before[tid + 1] = incl;
    if (tid == 0) sh.before[0] = 0;
  }
  __syncthreads();
  const int64_t units = sh.before[kScan];
  // an item's part costs a run as much as a page: no more runs than make four pages each, if the SMs have one
  const int runs = (int)min((int64_t)p.runs, max(units / 4, (int64_t)gridDim.x));
  if (warp == kWarps) {
    bring_tiles<D, NT>(p, k_map, v_map, sh, units, runs, share);
    return;
  }
  // neighbouring runs go to different SMs
  const int run = warp * gridDim.x + blockIdx.x;
  if (lane == 0) p.part_item[run] = make_int4(-1, 0, 0, 0);
  if (run >= runs) return;
  const int64_t u0 = run_begin(units, run, runs), u1 = run_begin(units, run + 1, runs);
  if (u0 >= u1) return;
  // the sequence that holds the run's first unit
  int lo = 0;
  for (int hi = kScan; hi - lo > 1;) {
    const int mid = (lo + hi) / 2;
    (sh.before[mid] <= u0 ? lo : hi) = mid;
  }
  int b = lo * share;
  int64_t local = u0 - sh.before[lo];
  for (int base = b;; base += 32) {  // 32 of the share's sequences at a time
    const int64_t mine = lane + base < min(p.B, (lo + 1) * share) ? units_of<NT>(p, lane + base) : 0;
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, incl > local);
    if (past) {
      const int at = __ffs(past) - 1;
      b = base + at;
      local -= __shfl_sync(0xffffffffu, incl - mine, at);
      break;
    }
    local -= __shfl_sync(0xffffffffu, incl, 31);
  }

  Seq s = sequence<NT>(p, b);
  int item = (int)(local / s.pages), page0 = (int)(local - (int64_t)item * s.pages);
  Rows<D, NT> w;
  int stage = 0;
  uint32_t turn = 0;
  bool ok = true;
#pragma unroll 1
  for (int64_t u = u0; u < u1 && ok;) {
    if (item == s.tiles * p.n_k) {
      item = 0;
      do s = sequence<NT>(p, ++b);
      while (s.tiles == 0);
    }
    const int head = item / s.tiles, tile = item - head * s.tiles;
    const int64_t from = u;
    const int pages = (int)min((int64_t)(s.pages - page0), u1 - u);  // of this segment
    u += pages;
    load_rows<D, NT>(p, s, head, tile, w);
    const int first0 = (s.low + page0) * kKvPage;
#pragma unroll 1
    for (int i = 0; i < pages; ++i) {
      ok = wait_bar(&sh.full[warp][stage], turn, &sh.abort, p.status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int first = first0 + i * kKvPage;
      if (sh.held[warp][stage] && first <= w.most && first + kKvPage > w.low_least) {
        const bool partial = first + kKvPage - 1 > w.least || first < w.low_most;
        if (partial) clean_values<D, NT>(sh.kv[warp][stage][1], sh.scales[warp][stage][1], first, w);
        // all keys at once where registers allow, else in halves
        constexpr int kBlocks = D * NT < 256 || (D == 128 && NT == 2) ? 4 : 2;
#pragma unroll 1
        for (int block = 0; block < kBlocksPerPage; block += kBlocks)
          key_blocks<D, NT, kBlocks>(smem_u32(sh.kv[warp][stage][0]), sh.scales[warp][stage], block, first, partial, w);
        if (partial) fence_async_smem();  // the next tile comes through the other proxy
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[warp][stage]);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
      turn ^= stage == 0;
    }
    if (!ok) break;
    // the item's rows: out, or to the workspace where other runs have a part
    const bool begins = page0 == 0, ends = page0 + pages == s.pages;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) w.l[nt][i] += __shfl_xor_sync(0xffffffffu, w.l[nt][i], o);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float l = w.l[nt][i];
        const int row = 8 * nt + 2 * c + i, r = tile * 8 * NT + row;
        if (r >= s.n * p.G) continue;
        if (begins && ends) {
          const int t = r / p.G, h = head * p.G + r - t * p.G;
          const int64_t at = (int64_t)(s.begin + t) * p.n_h + h;
          const float2 f = row_factors(p, h, w.m[nt][i], -w.g[nt][i], l);
          uint16_t* out = p.out + at * p.d + 2 * g;
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            if (16 * j < p.d)
              *reinterpret_cast<uint32_t*>(out + 16 * j) =
                  l == 0.f ? 0u : floats_bf16x2(w.o[j][nt][i] * f.x * f.y, w.o[j][nt][i + 2] * f.x * f.y);
          if (g == 0 && p.lse) p.lse[at] = row_lse(w.m[nt][i], l);
        } else {
          const int64_t part = ((int64_t)2 * run + begins) * 8 * NT + row;
          float* out = p.part_o + part * D + 2 * g;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) *reinterpret_cast<float2*>(out + 16 * j) = make_float2(w.o[j][nt][i], w.o[j][nt][i + 2]);
          if (g == 0) p.part_ml[part] = make_float4(l == 0.f ? kNoKey : w.m[nt][i], w.g[nt][i], l, 0.f);
        }
      }
    __syncwarp();
    if (begins && !ends && lane == 0) {
      // the runs that have the rest of the item: up to the one with its last unit
      const int64_t last = from + s.pages - 1, each = units / runs, more = units % runs;
      const int64_t to = last < more * (each + 1) ? last / (each + 1) : more + (last - more * (each + 1)) / each;
      p.part_item[run] = make_int4(b, head, tile, (int)(to - run));
    }
    ++item;
    page0 = 0;
  }
  if (!ok)  // gave up: the copies in flight land before the CTA's memory is another's
    for (int i = 0; i < kDepth; ++i, turn ^= stage == 0) {
      if (lane == 0) mbar_wait_drain(&sh.full[warp][stage], turn);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
}

// Joins the parts of the items that span runs: block (x, row) those that runs 4 x, ... , 4 x + 3 begin.  Eight
// groups of threads take an item's parts in turn, four elements to a thread; their sums are added in order.
template <int D, int NT>
__global__ void __launch_bounds__(2 * D) kv_join_kernel(const __grid_constant__ KvParams p) {
  constexpr int kGroups = 8, kLanes = D / 4;
  __shared__ float4 sums[kGroups][kLanes];
  const int tid = threadIdx.x, lane = tid & 31, row = blockIdx.y, group = tid / kLanes, e = 4 * (tid % kLanes);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int run0 = blockIdx.x * kRunsPerBlock;
  const int follow = lane < kRunsPerBlock && run0 + lane < p.runs && p.part_item[run0 + lane].x >= 0;
  for (uint32_t todo = __ballot_sync(0xffffffffu, follow); todo != 0; todo &= todo - 1) {
    const int run = run0 + __ffs(todo) - 1;
    const int4 item = p.part_item[run];
    auto part = [&](int i) { return ((int64_t)2 * (run + i) + (i == 0)) * 8 * NT + row; };
    // one round of loads: what most items need is under way at once
    float4 mine = make_float4(kNoKey, kUnset, 0.f, 0.f), x_ml = mine, x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane <= item.w) mine = p.part_ml[part(lane)];
    if (group <= item.w) x = *reinterpret_cast<const float4*>(p.part_o + part(group) * D + e), x_ml = p.part_ml[part(group)];
    const int begin = p.cu ? offset_at(p.cu, item.x, p.T) : item.x;
    const int n = p.cu ? offset_at(p.cu, item.x + 1, p.T) - begin : 1;
    const int r = item.z * 8 * NT + row;
    if (r >= n * p.G) continue;  // the whole block
    float m = mine.x;
    for (int i = lane + 32; i <= item.w; i += 32) m = fmaxf(m, p.part_ml[part(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // a part's unit relative to the common reference; the highest becomes the common unit
    auto unit = [&](const float4& s) { return s.x - m - s.y; };
    float l = mine.z * exp2_fast(mine.x - m), high = unit(mine);
    for (int i = lane + 32; i <= item.w; i += 32) {
      const float4 s = p.part_ml[part(i)];
      l += s.z * exp2_fast(s.x - m);
      high = fmaxf(high, unit(s));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    }
    const float f0 = exp2_fast(unit(x_ml) - high);
    x = make_float4(x.x * f0, x.y * f0, x.z * f0, x.w * f0);
#pragma unroll 8
    for (int i = group + kGroups; i <= item.w; i += kGroups) {
      const float f = exp2_fast(unit(p.part_ml[part(i)]) - high);
      const float4 y = *reinterpret_cast<const float4*>(p.part_o + part(i) * D + e);
      x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
    }
    sums[group][e / 4] = x;
    __syncthreads();
    if (group == 0 && e < p.d) {
#pragma unroll
      for (int i = 1; i < kGroups; ++i) {
        const float4 y = sums[i][e / 4];
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
      const int t = r / p.G, h = item.y * p.G + r - t * p.G;
      const int64_t at = (int64_t)(begin + t) * p.n_h + h;
      const float2 f = row_factors(p, h, m, high, l);
      *reinterpret_cast<uint2*>(p.out + at * p.d + e) =
          l == 0.f ? make_uint2(0u, 0u)
                   : make_uint2(floats_bf16x2(x.x * f.x * f.y, x.y * f.x * f.y), floats_bf16x2(x.z * f.x * f.y, x.w * f.x * f.y));
      if (e == 0 && p.lse) p.lse[at] = row_lse(m, l);
    }
    __syncthreads();
  }
}

// Rows in eights to a tile: those that a sequence's tokens have on average, so that its pages are read
// once, or equal parts of them; at most what registers hold.
int row_eights(int64_t rows, int d) {
  const int64_t most = d <= 64 ? 4 : 3, eights = (rows + 7) / 8, tiles = (eights + most - 1) / most;
  const int64_t need = (eights + tiles - 1) / tiles;
  return d <= 64 && need == 3 ? 4 : (int)need;
}

// The most that row_eights gives for up to that many rows.
int most_eights(int64_t rows, int d) {
  const int64_t eights = (rows + 7) / 8;
  return eights >= 3 ? (d <= 64 ? 4 : 3) : eights < 1 ? 1 : (int)eights;
}

size_t workspace_bytes(int eights, int d) {
  return (size_t)kMaxRuns * (sizeof(int4) + 2 * 8 * (size_t)eights * (sizeof(float4) + (d <= 64 ? 64 : 128) * sizeof(float)));
}

template <int D, int NT>
cudaError_t launch(KvParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, int sms, uint8_t* workspace, cudaStream_t stream) {
  p.part_o = reinterpret_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float4*>(workspace + (size_t)kMaxRuns * 2 * 8 * NT * D * sizeof(float));
  p.part_item = reinterpret_cast<int4*>(p.part_ml + (size_t)kMaxRuns * 2 * 8 * NT);
  static_assert(sizeof(Smem<D>) <= 227 * 1024, "shared memory of an SM");
  const int smem = (int)sizeof(Smem<D>);
  static std::atomic<uint64_t> said{0};
  const int64_t most = (int64_t)p.T * p.n_h * (p.R > 0 ? p.R : 1);  // units
  int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  if (most < ctas) ctas = (int)most;
  p.runs = ctas * kWarps;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = launch_with_smem(said, smem, cfg, kv_attn_kernel<D, NT>, k_map, v_map, p);
  if (e != cudaSuccess) return e;
  if (p.R <= 1) return cudaSuccess;  // items of one page are one run's
  cfg.gridDim = dim3((unsigned)((p.runs + kRunsPerBlock - 1) / kRunsPerBlock), 8 * NT);
  cfg.blockDim = dim3(2 * D);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT>, (const KvParams)p);
}

}  // namespace
}  // namespace fm

using namespace fm;

FM_API size_t fm_kv_attn_fp8_workspace(int T, int n_h, int n_k, int d) {
  if (T < 0 || bad_heads(n_h, n_k, d)) return 0;
  return workspace_bytes(most_eights((int64_t)T * (n_h / n_k), d), d);
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
  int sms = 0;
  fm_status st = check_device(&sms);
  if (st != FM_OK) return st;
  KvParams p = {};
  if ((st = status_word(&p.status)) != FM_OK) return st;
  const int D = a->d <= 64 ? 64 : 128;
  CUtensorMap k_map, v_map;
  const uint64_t dims[3] = {(uint64_t)a->d, (uint64_t)a->n_k * kKvPage, a->P > 0 ? (uint64_t)a->P : 1};
  const uint64_t strides[2] = {(uint64_t)a->d, (uint64_t)a->page_stride};
  const uint32_t box[3] = {(uint32_t)D, kKvPage, 1};
  const CUtensorMapSwizzle swizzle = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  // without pages nothing is read: any address will do for the maps
  const void *k_base = a->P > 0 ? (const void*)a->k_pool : a->q, *v_base = a->P > 0 ? (const void*)a->v_pool : a->q;
  if ((st = make_tmap(&k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, k_base, dims, strides, box, swizzle)) != FM_OK) return st;
  if ((st = make_tmap(&v_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, v_base, dims, strides, box, swizzle)) != FM_OK) return st;
  p.q = a->q;
  p.q_stride_t = a->q_stride_t;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.scale_stride = a->scale_stride;
  p.sink = a->sink_logit;
  p.page_table = a->page_table;
  p.cu = a->cu_tokens;
  p.start = a->start;
  p.out = a->out;
  p.lse = a->lse_out;
  p.window = a->window;
  p.T = a->T;
  p.n_h = a->n_h;
  p.n_k = a->n_k;
  p.d = a->d;
  p.G = a->n_h / a->n_k;
  p.P = (int)a->P;
  p.B = a->B;
  p.R = a->R;
  p.scale = a->scale;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(a->stream);
  const int eights = row_eights(((int64_t)a->T + a->B - 1) / a->B * p.G, a->d);
  cudaError_t e;
  if (D == 64)
    e = eights == 1   ? launch<64, 1>(p, k_map, v_map, sms, ws, stream)
        : eights == 2 ? launch<64, 2>(p, k_map, v_map, sms, ws, stream)
                      : launch<64, 4>(p, k_map, v_map, sms, ws, stream);
  else
    e = eights == 1   ? launch<128, 1>(p, k_map, v_map, sms, ws, stream)
        : eights == 2 ? launch<128, 2>(p, k_map, v_map, sms, ws, stream)
                      : launch<128, 3>(p, k_map, v_map, sms, ws, stream);
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}
