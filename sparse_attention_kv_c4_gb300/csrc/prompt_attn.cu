// prompt_attn.cu -- causal attention of grouped heads over packed prompts
// ("FlashMemory-DeepSeek-V4" README, "Two-level recall algorithm": the prompt's dense pass).
//     s_j = scale (q . k_j),  out = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink}),  keys up to the query's own
//
// 4 d flops for each query head and key that it sees: bound by the tensor cores.  A CTA
// has two tiles of 128 rows of one key head against tiles of 128 keys.  A row is a (token, head of
// the group), tokens first: a tile spans 128 / G tokens, so that short prompts fill it, the
// diagonal cuts few of its key tiles, and keys are read once for a group.
//   producer   (warp 8)  finds the items; Q by 3-D TMA boxes [128 / G tokens, G heads, 64 elements]; keys
//              and values in turn into a ring of tiles (SWIZZLE_128B)
//   issuers    (warps 9, 10)  one to a row tile: S = Q K^T (tcgen05 M128 N128 K16), then O += P V with P
//              from TMEM, in two halves; one row tile's products run while the other's softmax
//              does.  At D = 128 P takes the place of S, so the next S of a tile waits for its O
//   softmax    (warps 0-3, 4-7)  one row to a thread: scores from TMEM, a running reference
//              that moves only after a score has passed it by 2^8 (O is scaled in TMEM then), weights in
//              bf16 back to TMEM.  Sums are taken of the weights before they are rounded
//   sweeper    (warp 11)  tiles of keys that some rows do not see: an infinity or NaN among the
//              values would reach those rows as 0 * inf, so it is zeroed in shared memory and added
//              by the epilogue to the rows that do see it
// TMEM: S 2 x 128 columns, O 2 x D, P 2 x 64 (at D = 128 in S's place).
// A block takes over the items of blocks that have not started (cluster launch control).
// What bounds it: at D = 128 a step of both row tiles takes 2940 cycles, 2048 of them products; S starts some 450
// after the O before it has ended (its end has to be known, as P lies in S's place), twice a step.  At D = 64 a
// step takes some 3000, three times what its products or its exponentials need: the softmax warps' chain (scores from
// TMEM, all maxima, then all exponentials, then the stores), one tile after the other.
// Measured, calls queued on a stream, inputs in rotation: 8192 tokens x 32 heads x 128 391 us (1.41 PFLOP/s,
// 75% of a library product's burst rate), 4 x up to 4096 x 32 x 64 in a window of 1021 168 us, 2935 tokens of
// five prompts x 20 x 96 25 us, 37 tokens 8 us.
#include "grouped.cuh"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kRows = 128;       // of a tile
constexpr int kKeys = 128;
constexpr int kThreads = 12 * 32;
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 elements
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLow = -1e30f;   // below every score (past 2^24 a reference's own rounding shows in the weights)
constexpr float kSlack = 8.f;    // how far a score (in log2) may pass its reference for long,
constexpr float kFar = 16.f;     // and at all: weights of up to 2^16 leave values room in fp32
constexpr int kMaxEdge = 16;     // tiles of an item that the mask cuts: at most 2 (256 + 127) / 128 + 2
constexpr uint32_t kBIsMnMajor = 1u << 16;

struct PromptParams {
  const uint16_t* v;
  const int32_t *cu_q, *cu_k;
  const float* sink;
  uint16_t* out;
  float* lse;
  int64_t v_stride_t, window;
  int T, Tk, n_h, n_k, d, G, B, tokens, slots;  // tokens of a row tile
  int more;                                     // there are more blocks than SMs
  float scale;
  unsigned int* status;
};

// Columns of P: its own where TMEM has room, else those of S.
template <int D>
constexpr bool kOwnP = D == 64;
template <int D>
FM_DEV uint32_t p_column(int i) { return kOwnP<D> ? 2 * kKeys + 2 * D + i * (kKeys / 2) : i * kKeys; }

// A row tile: its tokens in the sequence and the key tiles that they see.
struct Tile {
  int t0, tokens;     // first token, number (0: an empty tile)
  int j0, j1;         // key tiles [j0, j1)
  int whole0, whole1; // those of them that every row sees whole
};
struct Item {
  int q0, k0, nk;     // the sequence's first query and key rows, its keys
  int head;
  int shift;          // nk - nq: query i is at position i + shift
  int j0, j1;         // key tiles of both
  int end;            // no item: the block's work is done
  Tile tile[2];
};

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 5 : 8;
  uint8_t q[2][D / 64][kChunkBytes];           // 1024-byte aligned
  uint8_t kv[kStages][D / 64][kChunkBytes];
  uint64_t q_full, q_empty, full[kStages], ready[kStages], empty[kStages];  // ready: full and checked
  uint64_t s_full[2], s_read[2], p_full[2][2], o_done[2], turn[2], drain[2];  // p_full: of the first 64 keys' weights, of the others'
  uint64_t item_full[2], item_empty[2], claimed;
  uint4 claim;                                 // a block of the grid that this one takes over
  Item item[2];
  int bad_tile[2][kMaxEdge];                   // an item's key tiles that held an infinity or NaN
  int bad[2];
  uint32_t tmem;
  int abort;
};

FM_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Descriptor of an MN-major SWIZZLE_128B operand: 64 elements of N to a 128-byte row, one row per K;
// 8-row groups 1024 bytes apart (stride offset), the next 64 elements of N a chunk further (leading offset).
FM_DEV uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kChunkBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
FM_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
FM_DEV float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
FM_DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
FM_DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// One lane of a warp that runs as a whole.
FM_DEV bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 x;\n\telect.sync x|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}
// Takes over a block of this grid that has not started (cluster launch control); the answer arrives at `bar`.
FM_DEV void claim_block(uint4* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
constexpr uint32_t kNoBlock = 0xFFFFFFFFu;
FM_DEV uint32_t claimed_block(const uint4* answer) {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.u32 %0, 0xFFFFFFFF;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return x;
}
FM_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

FM_DEV int last_key(const Item& w, int token) { return token + w.shift; }
FM_DEV int first_key(const PromptParams& p, const Item& w, int token) {
  const int pos = token + w.shift;
  return pos < p.window ? 0 : (int)(pos - p.window + 1);
}
// Whether the mask or the sequence's end cuts key tile j for a row of either tile.
FM_DEV bool cut(const Item& w, int j) {
  auto one = [j](const Tile& t) { return j >= t.j0 && j < t.j1 && (j < t.whole0 || j >= t.whole1); };
  return one(w.tile[0]) || one(w.tile[1]);
}

// The item of a block of the grid; false where the slot is empty.
FM_DEV bool find_item(const PromptParams& p, uint32_t block, Item& w) {
  const int slot = p.slots - 1 - (int)(block / p.n_k);  // later tokens, which see more keys, go first
  w.head = block % p.n_k;
  w.end = 0;
  const int pair = 2 * p.tokens;
  int b = 0, nq = p.T;
  w.q0 = w.k0 = 0;
  w.nk = p.Tk;
  if (p.cu_q) {
    b = warp_find(p.B, slot, [&](int i) { return (int64_t)(offset_at(p.cu_q, i, p.T) / pair) + i; });
    w.q0 = offset_at(p.cu_q, b, p.T);
    nq = offset_at(p.cu_q, b + 1, p.T) - w.q0;
    w.k0 = offset_at(p.cu_k, b, p.Tk);
    w.nk = max(offset_at(p.cu_k, b + 1, p.Tk) - w.k0, 0);
  }
  const int first = (slot - (p.cu_q ? w.q0 / pair + b : 0)) * pair;
  if (first < 0 || first >= nq) return false;
  w.shift = w.nk - nq;
  w.j0 = 1 << 30;
  w.j1 = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Tile& t = w.tile[i];
    t.t0 = first + i * p.tokens;
    t.tokens = max(min(p.tokens, nq - t.t0), 0);
    t.j0 = t.j1 = t.whole0 = t.whole1 = 0;
    if (t.tokens == 0) continue;
    const int last = last_key(w, t.t0 + t.tokens - 1);
    const int low = max(first_key(p, w, max(t.t0, -w.shift)), 0);
    if (last < low) continue;
    t.j0 = low / kKeys;
    t.j1 = last / kKeys + 1;
    t.whole0 = (first_key(p, w, t.t0 + t.tokens - 1) + kKeys - 1) / kKeys;
    t.whole1 = (max(last_key(w, t.t0), -1) + 1) / kKeys;
    w.j0 = min(w.j0, t.j0);
    w.j1 = max(w.j1, t.j1);
  }
  return true;
}

// One item's softmax and output.  `before`: key tiles of this row tile in the items before.
template <int D>
FM_DEV bool softmax_item(const PromptParams& p, Smem<D>& sh, int slot, uint32_t tmem, int which, uint32_t before) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const Item& w = sh.item[slot];
  const Tile tile = w.tile[which];
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  const uint32_t s_at = tmem + lanes + which * kKeys, o_at = tmem + lanes + 2 * kKeys + which * D;
  const uint32_t p_at = tmem + lanes + p_column<D>(which);
  const int r = 32 * quarter + lane;
  const int t = r / p.G;
  const bool live = t < tile.tokens;
  const int token = tile.t0 + t;
  const int last = live ? last_key(w, token) : -1, first = live ? first_key(p, w, token) : 0;
  const float c = p.scale * kLog2e;
  float m = kLow;          // the reference, in log2 units
  float last_most = kLow;  // the last tile's largest
  bool behind = false;     // some row's last tile passed its reference by more than kSlack
  float2 l = make_float2(0.f, 0.f);
  bool ok = true;
  for (int j = tile.j0; j < tile.j1; ++j) {
    const int n = j - tile.j0;
    if (ok) ok = wait_bar(&sh.s_full[which], (before + n) & 1, &sh.abort, p.status);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after();
    uint32_t s[4][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
    tmem_ld_wait();
    if (kOwnP<D>) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_read[which]);
    }
    const int lo = first - j * kKeys, hi = last - j * kKeys;  // the row's keys in the tile: lo .. hi
    if (j < tile.whole0 || j >= tile.whole1) {  // the mask cuts the tile
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int from = lo - 32 * i, to = hi - 32 * i;  // bits from .. to of the word are keys that the row sees
        const uint32_t below = to >= 31 ? 0xFFFFFFFFu : to < 0 ? 0u : (2u << to) - 1u;
        const uint32_t seen = from > 31 ? 0u : from <= 0 ? below : below & (0xFFFFFFFFu << from);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(seen >> e & 1)) s[i][e] = 0xFF800000u;  // -inf
      }
    }
    float top[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top[i] = __uint_as_float(s[i][0]);
#pragma unroll
      for (int e = 1; e + 1 < 32; e += 2) top[i] = max3(top[i], __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
      top[i] = fmaxf(top[i], __uint_as_float(s[i][31]));
    }
    const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c;
    // The reference moves before this tile's weights where they would leave fp32's range, and after
    // them where they are merely large: floating point loses nothing by it, and O is not
    // waited for.  The tile's other rows have no vote: the next sequence's, what lies behind the last, or what shared
    // memory held where the group's tokens do not fill 128 rows.
    const bool must = __any_sync(0xffffffffu, live && most > m + kFar);
    if (must || behind) {
      const float next = must ? fmaxf(m, most) : fmaxf(m, last_most);
      const float keep = exp2_fast(m - next);
      m = next;
      l.x *= keep;
      l.y *= keep;
      if (n > 0) {  // the products so far, in TMEM
        if (!wait_bar(&sh.o_done[which], (before + n - 1) & 1, &sh.abort, p.status)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
          tmem_st32(o_at + 32 * i, o);
        }
      }
    }
    behind = __any_sync(0xffffffffu, live && most > m + kSlack);
    last_most = most;
    const float2 cc = make_float2(c, c), mm = make_float2(-m, -m);
    float2 sums[4] = {l, make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t packed[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint32_t* x = s[2 * half + e / 16];
        const int at = 2 * (e % 16);
        float2 y = fma2(make_float2(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), cc, mm);
        y = make_float2(exp2_fast(y.x), exp2_fast(y.y));
        sums[e % 4] = add2(sums[e % 4], y);
        packed[e] = floats_bf16x2(y.x, y.y);
      }
      if (kOwnP<D> && half == 0 && n > 0) {  // the product that reads the last weights is over
        if (!wait_bar(&sh.o_done[which], (before + n - 1) & 1, &sh.abort, p.status)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      tmem_st32(p_at + 32 * half, packed);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[which][half]);
    }
    l = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
  }
  // epilogue
  const int n = tile.j1 - tile.j0;
  if (n > 0 && ok) {
    if (!wait_bar(&sh.o_done[which], (before + n - 1) & 1, &sh.abort, p.status)) ok = false;
    tc_fence_after();
  }
  if (!__all_sync(0xffffffffu, ok)) return false;
  const float sum = l.x + l.y;
  const int h = w.head * p.G + r - t * p.G;
  float z = sum, half = 1.f;
  if (live && p.sink) {  // it may be far over the scores: the output is then scaled in two steps
    const float sink = p.sink[h] * kLog2e - m, down = fmaxf(sink, 0.f);
    half = exp2_fast(-0.5f * down);
    z = sum * exp2_fast(-down) + exp2_fast(sink > 0.f ? 0.f : sink);
  }
  const bool some = n > 0 && sum != 0.f;  // the row sees a key
  const float inv = some ? half / z : 0.f;
  const int64_t at = (int64_t)(w.q0 + token) * p.n_h + h;
  uint16_t* out = p.out + at * p.d;
#pragma unroll 1
  for (int i = 0; i < D / 32; ++i) {
    uint32_t o[32];
    if (n > 0) {
      tmem_ld32(o_at + 32 * i, o);
      tmem_ld_wait();
    }
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      if (!live || 32 * i + e >= p.d) continue;
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = some ? floats_bf16x2(__uint_as_float(o[e + 2 * k]) * half * inv, __uint_as_float(o[e + 2 * k + 1]) * half * inv) : 0u;
      *reinterpret_cast<uint4*>(out + 32 * i + e) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    __syncwarp();  // the next load from TMEM is the whole warp's
  }
  const int bad = sh.bad[slot];
  if (live && some && bad) {  // infinities and NaN of tiles that the mask cuts, in the keys that the row sees
#pragma unroll 1
    for (int x = 0; x < kMaxEdge; ++x) {
      if (!(bad >> x & 1)) continue;
      const int j = sh.bad_tile[slot][x];
#pragma unroll 1
      for (int key = max(first, j * kKeys); key <= min(last, j * kKeys + kKeys - 1); ++key) {
        const uint16_t* v = p.v + (int64_t)(w.k0 + key) * p.v_stride_t + w.head * p.d;
#pragma unroll 1
        for (int e = 0; e < p.d; ++e) {
          if ((v[e] & 0x7F80u) != 0x7F80u) continue;
          const float sum_e = __uint_as_float((uint32_t)out[e] << 16) + __uint_as_float((uint32_t)v[e] << 16);
          out[e] = (uint16_t)(floats_bf16x2(sum_e, 0.f) & 0xFFFFu);
        }
      }
    }
  }
  if (live && p.lse) p.lse[at] = some ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  return true;
}

// A place in the ring.
template <int Stages>
struct Place {
  int stage = 0;
  uint32_t turn = 0;  // parity of the round
  FM_DEV void next(int by) {
    stage += by;
    if (stage >= Stages) {
      stage -= Stages;
      turn ^= 1;
    }
  }
};

// A value that is the same in all lanes, in a form that the compiler knows to be: an MMA whose operands
// are not takes its issuer several times as long.
FM_DEV uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// One warp issues a row tile's products.  Where a tile's S waits for its O, the two warps take turns, a tile's
// O and next S at a time: left to themselves the tiles fall into step, their products mix and end
// together, and the tensor cores idle through both softmaxes.  (One warp for both tiles: the hundred
// instructions between two products are then nobody else's time, 2 x 800 cycles of a step of 4000.)
template <int D>
FM_DEV void issue_products(const PromptParams& p, Smem<D>& sh, uint32_t I) {
  constexpr int kStages = Smem<D>::kStages;
  constexpr uint32_t s_idesc = idesc_bf16_f32(kRows, kKeys), o_idesc = idesc_bf16_f32(kRows, D) | kBIsMnMajor;
  constexpr uint32_t kTileStep = (D / 64) * (kChunkBytes >> 4);
  const bool one = elect_one();
  const uint32_t tmem = uniform(sh.tmem), s_at = tmem + I * kKeys, o_at = tmem + 2 * kKeys + I * D, p_at = tmem + p_column<D>(I);
  int tiles = 0, first = 0, end = 0, slot = 0;     // of the item; key tiles count from its first
  uint32_t before = 0, turns = 0, q_turn = 0;      // this row tile's key tiles, all, and items with keys, before it
  const uint64_t q_desc = sdesc_sw128(smem_u32(sh.q[I][0])), k_desc = sdesc_sw128(smem_u32(sh.kv[0][0])),
                 v_desc = sdesc_mn_sw128(smem_u32(sh.kv[0][0]));
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_call(bar, parity, &sh.abort, p.status));
  };
  // S of key tile j, whose keys are in stage `at`.  The stage's phase is waited for even where the row tile
  // does not see the keys: a wait tells only the last phase from the one before.
  auto scores = [&](int j, const Place<kStages>& at) {
    if (!wait(&sh.full[at.stage], at.turn)) return false;
    const int done = j - first;
    if (done < 0 || j >= end) {
      if (one) mbar_arrive(&sh.empty[at.stage]);
      return true;
    }
    const uint64_t b = k_desc + at.stage * kTileStep;
    // S is free: its last scores are read, or, where P lies in its place, the product that reads P is over
    if (before + done > 0 && !wait(kOwnP<D> ? &sh.s_read[I] : &sh.o_done[I], (before + done - 1) & 1)) return false;
    tc_fence_after();
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      const uint64_t o = (uint64_t)((x / 4) * (kChunkBytes >> 4) + (x % 4) * 2);
      if (one) umma_bf16_ss(s_at, q_desc + o, b + o, s_idesc, x > 0);
    }
    if (one) {
      umma_commit(&sh.empty[at.stage]);
      umma_commit(&sh.s_full[I]);
    }
    return true;
  };
  // O += P V, half of the keys as soon as their weights are there.
  auto values = [&](int j, const Place<kStages>& at) {
    if (!wait(&sh.full[at.stage], at.turn)) return false;
    const int done = j - first;
    const bool sees = done >= 0 && j < end;
    if (sees && cut(sh.item[slot], sh.item[slot].j0 + j) && !wait(&sh.ready[at.stage], at.turn)) return false;
    if (sees && !wait(&sh.p_full[I][0], (before + done) & 1)) return false;
    if (!kOwnP<D> && !wait(&sh.turn[I], (turns + j) & 1)) return false;
    if (!sees) {
      if (one) mbar_arrive(&sh.empty[at.stage]);
      return true;
    }
    const uint64_t b = v_desc + at.stage * kTileStep;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1 && !wait(&sh.p_full[I][1], (before + done) & 1)) return false;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < kKeys / 32; ++x) {
        const int k = half * (kKeys / 32) + x;
        if (one) umma_bf16_ts(o_at, p_at + 8 * k, b + (uint64_t)(k * (2048 >> 4)), o_idesc, done > 0 || k > 0);
      }
    }
    if (one) {
      umma_commit(&sh.empty[at.stage]);
      umma_commit(&sh.o_done[I]);
    }
    return true;
  };
  Place<kStages> k_at, v_at;  // of the keys after, and of the values of, tile j
  v_at.next(1);
  bool ok = true;
#pragma unroll 1
  for (uint32_t k = 0; ok; ++k) {
    slot = k & 1;
    if (!(ok = wait(&sh.item_full[slot], (k >> 1) & 1)) || sh.item[slot].end) break;
    const Item& w = sh.item[slot];
    tiles = (int)uniform((uint32_t)max(w.j1 - w.j0, 0));
    first = (int)uniform(max(w.tile[I].j0 - w.j0, 0));
    end = (int)uniform(max(w.tile[I].j1 - w.j0, 0));
    if (tiles > 0) ok = wait(&sh.q_full, q_turn++ & 1);
#pragma unroll 1
    for (int j = -1; ok && j < tiles; ++j) {
      const bool more = j + 1 < tiles;
      if (kOwnP<D> && more) ok = scores(j + 1, k_at);
      if (ok && j >= 0) ok = values(j, v_at);
      if (!kOwnP<D> && ok && more) ok = scores(j + 1, k_at);
      if (one && more && j + 2 == tiles) umma_commit(&sh.q_empty);
      if (!kOwnP<D> && one && (I == 0 || more) && j + (int)I >= 0) mbar_arrive(&sh.turn[1 - I]);
      if (more) k_at.next(2);
      if (j >= 0) v_at.next(2);
    }
    if (end > first) before += end - first;
    turns += tiles;
    __syncwarp();
    if (one) mbar_arrive(&sh.item_empty[slot]);
  }
  if (!ok && one) {  // gave up: the products in flight end before TMEM is freed
    umma_commit(&sh.drain[I]);
    mbar_wait_drain(&sh.drain[I], 0);
  }
}

// Zeroes infinities and NaN of the values in a stage; an item's edge number `edge`, key tile j.
template <int D>
FM_DEV void check_values(Smem<D>& sh, int stage, int slot, int edge, int j) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll 1
  for (int x = 0; x < D / 64; ++x) {
    const uint4* cells = reinterpret_cast<const uint4*>(sh.kv[stage][x]);
#pragma unroll 8
    for (int i = lane; i < kChunkBytes / 16; i += 32) {
      const uint4 u = cells[i];
      const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)  // a carry out of an all-ones exponent, of either half
        bad |= (((a[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0;
    }
  }
  if (!__any_sync(0xffffffffu, bad)) return;
#pragma unroll 1
  for (int x = 0; x < D / 64; ++x) {
    uint16_t* cells = reinterpret_cast<uint16_t*>(sh.kv[stage][x]);
#pragma unroll 1
    for (int i = lane; i < kChunkBytes / 2; i += 32)
      if ((cells[i] & 0x7F80u) == 0x7F80u) cells[i] = 0;
  }
  if (lane == 0) {
    sh.bad_tile[slot][edge] = j;
    sh.bad[slot] |= 1 << edge;
  }
  fence_async_smem();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                  const __grid_constant__ CUtensorMap k_map,
                                                                  const __grid_constant__ CUtensorMap v_map,
                                                                  const __grid_constant__ PromptParams p) {
  using S = Smem<D>;
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  S& sh = *reinterpret_cast<S*>(raw_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 2);
    mbar_init(&sh.claimed, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], 11);  // softmax warps, issuers and the sweeper
    }
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.ready[i], 1);
      mbar_init(&sh.empty[i], 3);  // both row tiles and the sweeper
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i][0], 4);
      mbar_init(&sh.p_full[i][1], 4);
      mbar_init(&sh.s_read[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.turn[i], 1);
      mbar_init(&sh.drain[i], 1);
    }
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch(&q_map);
    tma_prefetch(&k_map);
    tma_prefetch(&v_map);
  }
  if (warp == 8) {
    tmem_alloc(&sh.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // programmatic dependent launch: what a kernel before wrote may be read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = sh.tmem;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int which = warp >> 2;
    uint32_t before = 0;
#pragma unroll 1
    for (uint32_t k = 0;; ++k) {
      const int slot = k & 1;
      const bool ok = wait_bar(&sh.item_full[slot], (k >> 1) & 1, &sh.abort, p.status);
      if (!__all_sync(0xffffffffu, ok) || sh.item[slot].end) break;
      if (!softmax_item<D>(p, sh, slot, tmem, which, before)) break;
      before += sh.item[slot].tile[which].j1 - sh.item[slot].tile[which].j0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      // ------------------------------------------------------------ producer
      // It also finds the items: this block's own, then those of blocks that have not started yet, which it
      // takes over one at a time, so that the last item's output runs beside the next one's first products.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_call(bar, parity, &sh.abort, p.status));
      };
      bool ok = true;
      uint32_t block = blockIdx.x, claims = 0, items = 0, q_items = 0;
      int n = 0;  // stages filled
#pragma unroll 1
      for (;; ++claims) {
        Item w;
        if (find_item(p, block, w)) {
          const int slot = items & 1;
          if (items >= 2 && !(ok = wait(&sh.item_empty[slot], ((items >> 1) - 1) & 1))) break;
          if (lane == 0) {
            sh.item[slot] = w;
            sh.bad[slot] = 0;
            mbar_arrive(&sh.item_full[slot]);
          }
          ++items;
          if (w.j1 > w.j0) {
            if (q_items > 0 && !(ok = wait(&sh.q_empty, (q_items - 1) & 1))) break;
            ++q_items;
            if (lane == 0) {
              const int tiles = w.tile[1].tokens > 0 ? 2 : 1;
              mbar_arrive_expect_tx(&sh.q_full, tiles * (D / 64) * p.tokens * p.G * 128);
              for (int i = 0; i < tiles; ++i)
                for (int x = 0; x < D / 64; ++x)
                  tma_load_3d(sh.q[i][x], &q_map, &sh.q_full, 64 * x, w.head * p.G, w.q0 + w.tile[i].t0);
              for (int j = w.j0; ok && j < w.j1; ++j)
                for (int v = 0; v < 2; ++v, ++n) {
                  const int stage = n % S::kStages, turn = n / S::kStages;
                  if (turn > 0 && !(ok = wait_call(&sh.empty[stage], (turn - 1) & 1, &sh.abort, p.status))) break;
                  mbar_arrive_expect_tx(&sh.full[stage], (D / 64) * kChunkBytes);
                  for (int x = 0; x < D / 64; ++x)
                    tma_load_3d(sh.kv[stage][x], v ? &v_map : &k_map, &sh.full[stage], 64 * x, w.head, w.k0 + j * kKeys);
                }
            }
            n = __shfl_sync(0xffffffffu, n, 0);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
          }
        }
        if (!p.more) break;
        // asked for when the item's last copies are under way: asked for before, the first blocks take what
        // is left whether they finish early or not
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.claimed, 16);
          claim_block(&sh.claim, &sh.claimed);
        }
        if (!(ok = wait(&sh.claimed, claims & 1))) break;
        const uint32_t next = claimed_block(&sh.claim);
        fence_async_smem();  // the next claim is written through the other proxy
        if (next == kNoBlock) break;
        block = next;
        __syncwarp();
      }
      const int slot = items & 1;
      if (ok && items >= 2) ok = wait(&sh.item_empty[slot], ((items >> 1) - 1) & 1);
      if (ok && lane == 0) {
        sh.item[slot].end = 1;
        mbar_arrive(&sh.item_full[slot]);
      }
      // the issuers' last arrivals come before the block ends
      for (int i = max(n - S::kStages, 0); ok && i < n; ++i) ok = wait(&sh.empty[i % S::kStages], (i / S::kStages) & 1);
      if (ok && q_items > 0) ok = wait(&sh.q_empty, (q_items - 1) & 1);
      if (!ok && lane == 0) {  // gave up: the copies in flight land before the block's memory is another's
        if (q_items > 0) mbar_wait_drain(&sh.q_full, (q_items - 1) & 1);
        for (int i = max(n - S::kStages, 0); i < n; ++i) mbar_wait_drain(&sh.full[i % S::kStages], (i / S::kStages) & 1);
      }
    } else if (warp == 9 || warp == 10) {
      issue_products<D>(p, sh, uniform(warp - 9));
    } else {
      // ------------------------------------------------------------ sweeper
      // Every stage of the ring passes through its hands, keys too, so that its barriers keep step
      // with the ring's.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_call(bar, parity, &sh.abort, p.status));
      };
      Place<S::kStages> at;
      bool ok = true;
#pragma unroll 1
      for (uint32_t k = 0; ok; ++k) {
        const int slot = k & 1;
        if (!(ok = wait(&sh.item_full[slot], (k >> 1) & 1)) || sh.item[slot].end) break;
        const Item& w = sh.item[slot];
        const int stages = 2 * max(w.j1 - w.j0, 0);
        int edges = 0;
#pragma unroll 1
        for (int n = 0; n < stages; ++n, at.next(1)) {
          if (!(ok = wait(&sh.full[at.stage], at.turn))) break;
          const int j = w.j0 + n / 2;
          if (n % 2 == 1 && cut(w, j)) {
            check_values<D>(sh, at.stage, slot, edges, j);
            ++edges;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.ready[at.stage]);
            mbar_arrive(&sh.empty[at.stage]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const PromptParams& p, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                   cudaStream_t stream) {
  constexpr int smem = (int)sizeof(Smem<D>);
  static_assert(smem <= 227 * 1024, "shared memory of an SM");
  static std::atomic<uint64_t> said{0};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)p.slots * p.n_k));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_with_smem(said, smem, cfg, prompt_attn_kernel<D>, q_map, k_map, v_map, p);
}

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
  PromptParams p = {};
  p.G = a->n_h / a->n_k;
  p.tokens = kRows / p.G;
  const int64_t slots = a->cu_q ? (int64_t)a->T / (2 * p.tokens) + a->B : (a->T + 2 * p.tokens - 1) / (2 * p.tokens);
  if (slots * a->n_k >= int64_t(1) << 31)
    return set_error(FM_ERR_INVALID_ARG, "%s: T=%d B=%d are too many for %d heads", who, a->T, a->B, a->n_h);
  int sms = 0;
  fm_status st = check_device(&sms);
  if (st != FM_OK) return st;
  if ((st = status_word(&p.status)) != FM_OK) return st;
  const int D = a->d <= 64 ? 64 : 128;
  CUtensorMap maps[3];
  for (int i = 0; i < 3; ++i) {
    const bool q = i == 0, none = !q && a->Tk == 0;  // without keys nothing is read: any address will do
    const void* base = q || none ? a->q : i == 1 ? a->k : a->v;
    const int64_t stride = q || none ? a->q_stride_t : i == 1 ? a->k_stride_t : a->v_stride_t;
    const uint64_t dims[3] = {(uint64_t)a->d, (uint64_t)(q || none ? a->n_h : a->n_k), (uint64_t)(q || none ? a->T : a->Tk)};
    const uint64_t strides[2] = {(uint64_t)a->d * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, (uint32_t)(q ? p.G : 1), (uint32_t)(q ? p.tokens : kKeys)};
    if ((st = make_tmap(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) != FM_OK)
      return st;
  }
  p.v = a->v;
  p.v_stride_t = a->v_stride_t;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k ? a->cu_k : a->cu_q;
  p.sink = a->sink_logit;
  p.out = a->out;
  p.lse = a->lse_out;
  p.window = a->window;
  p.T = a->T;
  p.Tk = a->Tk;
  p.n_h = a->n_h;
  p.n_k = a->n_k;
  p.d = a->d;
  p.B = a->B;
  p.slots = (int)slots;
  p.more = slots * a->n_k > sms;
  p.scale = a->scale;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(a->stream);
  const cudaError_t e = D == 64 ? launch<64>(p, maps[0], maps[1], maps[2], stream) : launch<128>(p, maps[0], maps[1], maps[2], stream);
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return FM_OK;
}
