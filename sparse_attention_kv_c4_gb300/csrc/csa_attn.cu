// csa_attn.cu -- attention of a CSA layer: one softmax per head over the
// selected chunk cells, the first tokens and a sliding window of the sequence's
// tokens ("DeepSeek-V4 CSA + HCA explained", sec. 4), also for a tree of drafted
// tokens.  A cell c (512 elements) is key and value of every head:
//     s_j = scale (q_h . c_j),  out_h = sum_j e^{s_j} c_j / (sum_j e^{s_j} + e^{sink_h})
//
// GB300 mapping.  Every token has keys of its own, shared by its heads, so the
// unit of work is one token's block of 64 heads against tiles of 64 keys
// (131 kFLOP per key of 1 KB).  A persistent CTA per SM walks its items (token,
// head block, split of the keys):
//   resolver    (warp 1)  each item's key ranges, and each tile's 64 row addresses
//               and mask (a key that is none is a zero bit).  An item's first tile
//               is its 64 query rows
//   producers   (warps 16-19)  the rows by 16-byte cp.async, 16 rows to a warp,
//               into SWIZZLE_128B chunks [64 rows x 64 elements] (a TMA gather of
//               four rows costs its warp some 90 cycles to issue, 128 of them a
//               tile).  The ring holds three tiles and is freed in quarters; a key
//               that is none is filled with zeros without a read
//   S issuer    (warp 0)  S = Q C^T: tcgen05 M64 N64, 32 steps of K16
//   O issuer    (warp 2)  O^T += C^T P^T: M128 N64, four blocks of 128 elements x
//               four steps of K16.  The cell tile is read twice from shared
//               memory, K-major as keys and MN-major as values, and loaded once
//   softmax     (warps 4-11)  S from TMEM, the running maximum and sum, P in
//               bf16 to shared memory: 16 heads x 32 keys to a warp
//   epilogue    (warps 12-15)  O^T from TMEM, times 1 / (sum + sink), to out; and
//               the next item's queries from the ring to their place
// TMEM: O^T 4 x 64 columns, S 64, three quarters of Q 192.  The output is kept
// transposed (rows = elements) because 64 rows of heads x 512 columns would fill
// TMEM.
// What bounds it: a tile takes some 2200 cycles (2400 where its cells are scattered),
// a third of what its slot of the ring goes through: the copies (128 cp.async of 512
// bytes, 16 cycles of the SM each with four and with eight producer warps alike, and
// not much less without the reads: 2080), S (32 steps of 32 cycles), the softmax
// (some 1500) and O (16 steps of at least 48: it takes 64 KB of cells and 32 KB of
// weights from shared memory at 128 bytes a cycle).  Copies of the kernel with a part
// removed (2 x 61 drafted tokens, 77 us): three quarters of O and half of S gone 72,
// half of the copies gone too 65, all copies gone 55, only the copies gone 81 (S and O
// then interleave more, and each switch between the two costs).  Between items
// another 3900 cycles: the queries hold a third of the ring, and the item's second
// tile waits for the slot of the last item's last one.  What all roles pay for is
// code: a kernel of 107 KB (the waits' loops inlined, 64-bit divisions) took 3 to 9%
// longer than this one of 80.  With all of Q in shared memory the ring held 2.25
// tiles (515 us for the prefill below).
// Measured, calls on the same inputs queued on a stream: 4096 tokens x 64 heads x 644 keys 399 us (866
// TFLOP/s, 44% of the burst peak of a library's product); 2 x 61 drafted tokens over
// a window of 4096 76.5 us (766 TFLOP/s on 122 of the 152 SMs); 3065 tokens x 20
// heads x 186 keys on average 114 us (items of three tiles, and the scores' product
// is padded to 64 heads); 30 tokens x 644 keys 16.1 us; 76 tokens x 128 heads x 644
// keys 21.2 us; 8 tokens x 32832 keys 59.4 us (4.5 TB/s); one token x 37 keys 8.2 us.
//
// Few tokens: the keys of an item are split over several CTAs.  Two, four or eight of
// them are a cluster and join their outputs through distributed shared memory:
// each CTA sends every other one that one's slice of the 512 elements of its output,
// and sums the slices that it gets by the splits' shares of the common softmax, worked
// out beside the sends (30 tokens: 16.3 -> 16.05 us).  Where a split over all SMs
// saves a CTA more than eight tiles (few tokens with long key lists), the splits, two
// or more, write unnormalised fp32 outputs with their maximum and sum to the
// workspace, and csa_merge_kernel joins those.  Both in a fixed order.
// 30 tokens x 644 keys, in cycles from the end of the kernel before: a tile's
// rows known 5400, copied 8800, the split's three tiles done 17100, all of the cluster's
// 19300, outputs sent 24900 (131 KB, 23 bytes a cycle), all arrived 27300, stored 29600.
#include <cuda_bf16.h>

#include <atomic>

#include "fm_common.cuh"
#include "fm_internal.h"

#define FM_API extern "C" __attribute__((visibility("default")))

namespace fm {
namespace {

constexpr int kWidth = 512;
constexpr int kPage = 64;
constexpr int kMaxCells = 1024;
constexpr int kMaxTable = 1 << 19;              // pages of a sequence: its 2^25 tokens take less than a wait's limit
constexpr int kHeadsPerItem = 64;
constexpr int kTileKeys = 64;
constexpr int kChunkBytes = 64 * 128;           // 64 rows x 64 elements
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr int kPairsPerTile = kWidth / 128;     // 4
constexpr int kTileSlots = 3;
constexpr int kPairs = kTileSlots * kPairsPerTile;
constexpr int kQBytes = kPairBytes;             // the first quarter of Q; the rest is in TMEM
constexpr int kPBytes = kHeadsPerItem * kTileKeys * 2;
constexpr int kThreads = 20 * 32;
constexpr int kSoftmaxWarps = 8;
constexpr int kProducerWarps = 4;
constexpr int kKeysPerProducer = kTileKeys / kProducerWarps;
constexpr int kTmemCols = 512;                  // allocations are powers of two
constexpr int kSCol = 256;                      // S behind O^T's 256 columns
constexpr int kQCol = 320;                      // and three quarters of Q, 32 columns to a chunk of 64 elements
constexpr int kInfoSlots = 4;
constexpr int kInfoReaders = 2 + kSoftmaxWarps + 4;           // issuers, softmax and epilogue warps
constexpr int kKvArrivals = 33 * kProducerWarps;              // the producers' copies, and their first lanes
constexpr int kMaxParts = 256;                  // partial results of one call
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxItems = int64_t(1) << 23;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
  const uint16_t* q;
  const uint16_t* kv_pool;
  const uint16_t* cell_pool;
  const int32_t* page_table;
  const int32_t* seq;
  const int64_t* pos;
  const int32_t* cells;
  const float* sink_logit;
  const uint32_t* tree_mask;
  const int64_t* tree_base;
  uint16_t* out;
  float* lse;
  float* part_o;                         // [parts][64][512] unnormalised outputs
  float2* part_ml;                       // [parts][64] (maximum in units of S, sum)
  unsigned int* status;
  int64_t kv_page_rows, cell_page_rows;  // rows (of 512 elements) from page to page
  int64_t window;
  int64_t cell_limit;                    // Pc * 64
  int T, n_h, P, B, R, k, n_sink, tree_words;
  int head_blocks, splits, items;        // items = T * head_blocks * splits
  int cluster;                           // the splits of an item are a cluster
  float scale;
};

// A token's keys, in order: the listed cells, n_first first tokens, n_win window
// tokens from slot low, then n_tree drafted slots from base.
struct TokenKeys {
  int64_t low, base;
  int b;
  int n_first, n_win, n_tree;
};

FM_DEV TokenKeys token_keys(const AttnParams& p, int64_t b, int64_t pos) {
  TokenKeys r = {0, 0, -1, 0, 0, 0};
  if (b < 0 || pos < 0) return r;
  if (b >= p.B) {
    atomicOr(p.status, FM_DEV_PAGE_RANGE);
    return r;
  }
  int64_t last = pos;  // the last cached token that is not after the query
  if (p.tree_mask != nullptr) {
    r.base = p.tree_base[b];
    if (r.base < 0) return r;
    if (r.base <= last) last = r.base - 1;
    if (r.base > int64_t(1) << 62) r.base = int64_t(1) << 62;  // past every table, and sums stay in 64 bits
    r.n_tree = 32 * p.tree_words;
  }
  r.b = (int)b;
  // the window has tokens past the table, or the first tokens reach past it
  const int64_t held = (int64_t)p.R * kPage;
  if (last >= held && (pos - last < p.window || p.n_sink > held)) atomicOr(p.status, FM_DEV_PAGE_RANGE);
  const int64_t end = (last < held ? last : held - 1) + 1;
  r.low = p.window > pos ? 0 : p.window == 0 ? end : pos - p.window + 1;
  if (r.low > end) r.low = end;
  r.n_first = (int)(p.n_sink < r.low ? p.n_sink : r.low);
  r.n_win = (int)(end - r.low);
  return r;
}

// What the roles know of one item.
struct ItemInfo {
  int t, head_block;
  int part;   // index of the partial result, -1 = whole
  int tiles;  // of keys, at least one; the tile of queries before them is not counted
};

// 16 bytes global -> shared, or 16 zero bytes where `bytes` is 0: nothing is read then.
FM_DEV void cp_async16(uint32_t dst, uint64_t src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrive on `bar` when this thread's copies so far have landed.
FM_DEV void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
FM_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
FM_DEV void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 lanes x 32 columns: thread i gets, of columns 8j + 2 (i % 4) + {0, 1}, lane
// i / 4 in r[4j], r[4j + 1] and lane i / 4 + 8 in r[4j + 2], r[4j + 3].
FM_DEV void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Descriptor of an MN-major SWIZZLE_128B operand: 64 elements of M or N to a
// 128-byte row, one row per K; 8-row groups 1024 bytes apart (stride offset),
// the next 64 elements of M or N a chunk further (leading offset).
FM_DEV uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kChunkBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kAIsMnMajor = 1u << 15;

FM_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four 8 x 8 matrices of 16-bit elements to shared memory: x[k] is matrix k, thread
// i holding row i / 4, columns 2 (i % 4) + {0, 1}; thread i's address is that of row
// i % 8 of matrix i / 8.
FM_DEV void store_8x8_x4(uint32_t addr, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x0), "r"(x1),
               "r"(x2), "r"(x3)
               : "memory");
}

// The same, each matrix transposed.
FM_DEV void store_8x8_x4_trans(uint32_t addr, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x0), "r"(x1),
               "r"(x2), "r"(x3)
               : "memory");
}
FM_DEV void store_shared_16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
FM_DEV uint4 load_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

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

// OR of a predicate over the softmax warps' threads (and a barrier for them).
FM_DEV bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(32 * kSoftmaxWarps)
      : "memory");
  return r != 0;
}

FM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

FM_DEV uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

// A warp's wait for a phase, given up after FM_WAIT_LIMIT_NS or when another
// warp has given up.  Lane 0 polls.  A function of its own: some twenty copies
// of this loop would not leave the roles' loops room in the instruction cache.
__device__ __noinline__ bool warp_wait_poll(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t t0 = timer_lo();
#pragma unroll 1
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
      if ((n & 31) != 0) continue;
      const bool late = timer_lo() - t0 > (uint32_t)FM_WAIT_LIMIT_NS;
      if (late && *abort == 0) atomicOr(status, FM_DEV_TIMEOUT);
      if (late) *abort = 1;
      if (*abort != 0) {
        ok = 0;
        break;
      }
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}
__device__ __noinline__ void wait_drain(uint64_t* bar) { mbar_wait_drain(bar, 0); }
FM_DEV bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_poll(bar, parity, abort, status);
}

// The issuers' warps run as a whole and elect the lane that issues, so that the
// operands of an MMA stay uniform values.
FM_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x;\n\t"
      "elect.sync x|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// What the roles share besides the tiles.
struct Shared {
  uint64_t kv_full[kTileSlots], kv_empty[kPairs];
  uint64_t s_full, s_empty, p_full[2], pv_done[2];
  uint64_t q_full, q_empty, o_full, o_empty[kPairsPerTile], stat_full, stat_empty, stage_free[2];
  uint64_t info_full[kInfoSlots], info_empty[kInfoSlots], rows_full[2], rows_empty[2], drain[2];
  uint2 key_mask[8];                     // the resolver is up to four tiles ahead of the softmax
  ItemInfo info[kInfoSlots];
  alignas(16) uint64_t rows[2][kTileKeys];  // addresses: key 16 w + 2 c + x at 16 w + 8 x + c
  float2 stat[kHeadsPerItem];            // maximum in units of S, sum of an item's heads
  alignas(16) float rescale[kHeadsPerItem];
  float top_half[2][kHeadsPerItem];
  uint32_t tmem_slot;
  int abort_flag;
};
constexpr int kSmemBytes = kQBytes + kPairs * kPairBytes + 2 * kPBytes + (int)sizeof(Shared);
static_assert(kSmemBytes <= 232448, "227 KB of shared memory to a CTA");
static_assert(offsetof(Shared, rows) % 16 == 0, "vector accesses");

// The output of an item, 32 heads x 32 elements (of TMEM quadrant `quad`) at a time:
// half block x has heads 32 (x % 2) .. of the 128 elements x / 2.
constexpr int kStageBytes = 32 * 32 * 2;
struct Output {
  const AttnParams& p;
  uint32_t tmem, stage;  // stage: kStageBytes of shared memory of the warp's own
  int t, h0, part;

  // Scaled by the heads' factors (f[2 j + e]: of head 8 j + 2 (lane % 4) + e), to
  // bf16, transposed through `stage`; `loaded` runs once TMEM has been read.
  template <typename Loaded>
  FM_DEV void half_block(int x, int quad, int lane, const float (&f)[8], Loaded loaded) const {
    const int heads = min(kHeadsPerItem, p.n_h - h0);
    // rows of 64 bytes (32 elements of a head), their 16-byte units swizzled: unit u
    // of row h at u ^ (h / 2) % 4
    const uint32_t put = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
    const uint32_t get = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    uint16_t* dst = p.out + ((int64_t)t * p.n_h + h0 + (x & 1) * 32 + lane / 4) * kWidth + (x >> 1) * 128 + quad * 32 +
                    (lane & 3) * 8;
    const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + 32 * x;
    uint32_t a[16], b[16];
    tmem_ld_16x256b_x4(from, a);
    tmem_ld_16x256b_x4(from + (16u << 16), b);
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    loaded();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t e[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        e[r] = pack_bf16(__uint_as_float(a[4 * j + 2 * r]) * f[2 * j], __uint_as_float(a[4 * j + 2 * r + 1]) * f[2 * j + 1]);
        e[2 + r] = pack_bf16(__uint_as_float(b[4 * j + 2 * r]) * f[2 * j], __uint_as_float(b[4 * j + 2 * r + 1]) * f[2 * j + 1]);
      }
      store_8x8_x4_trans(put + 8 * j * 64, e[0], e[1], e[2], e[3]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 v = load_shared_16(get + 8 * j * 64);
      if ((x & 1) * 32 + 8 * j + lane / 4 < heads) *reinterpret_cast<uint4*>(dst + 8 * j * kWidth) = v;
    }
    __syncwarp();
  }

  // As it is, fp32, to the partial results.
  FM_DEV void half_block_partial(int x, int quad, int lane) const {
    const int heads = min(kHeadsPerItem, p.n_h - h0);
    uint32_t o[32];
    tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + 32 * x, o);
    tmem_ld_wait();
    float* dst = p.part_o + ((int64_t)part * kHeadsPerItem + (x & 1) * 32) * kWidth + (x >> 1) * 128 + quad * 32 + lane;
#pragma unroll
    for (int h = 0; h < 32; ++h)
      if ((x & 1) * 32 + h < heads) dst[h * kWidth] = __uint_as_float(o[h]);
  }
};

FM_DEV void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
FM_DEV void grid_dep_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

FM_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
FM_DEV uint32_t in_cta(uint32_t smem_addr, uint32_t rank) {  // the same place in another CTA of the cluster
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  return a;
}

// The end of an item whose splits are a cluster, by all threads of its CTAs.
// CTA r writes elements r * 512 / splits .. of the output; `buf` (the idle ring,
// the same in every CTA) takes the slices of all CTAs: [split][64 heads][512 / splits],
// and `share` (an idle P buffer) the splits' shares [split][64].
FM_DEV void join_cluster(const AttnParams& p, Shared& sh, float* buf, float* share, uint32_t tmem) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)blockIdx.x & (p.splits - 1), th = (int)blockIdx.x >> (__ffs(p.splits) - 1);
  const int t = th / p.head_blocks, h0 = th % p.head_blocks * kHeadsPerItem;
  const int heads = min(kHeadsPerItem, p.n_h - h0);
  const int log_splits = __ffs(p.splits) - 1, slice = kWidth >> log_splits;  // (a power of two)
  const float c = p.scale * kLog2e;
  cluster_sync();  // every CTA is done with its ring, and its maxima and sums are in place
  // 32 heads x 32 elements at a time to the CTA whose slice they are in
#pragma unroll 1
  for (int x = warp >> 2; x < 8; x += kThreads / 128) {
    if ((x & 1) && heads <= 32) continue;
    const int d = (x >> 1) * 128 + (warp & 3) * 32, to = d >> (9 - log_splits);
    uint32_t o[32];
    tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + 32 * x, o);
    tmem_ld_wait();
    const uint32_t dst = in_cta(smem_u32(buf + (rank * kHeadsPerItem + (x & 1) * 32) * slice + (d & (slice - 1)) + lane), to);
#pragma unroll
    for (int h = 0; h < 32; ++h)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst + (uint32_t)(h * slice * 4)), "r"(o[h]) : "memory");
  }
  // each split's share of the common softmax
  if (warp >= 16 && warp < 18) {  // (which have the least to send)
    const int h = threadIdx.x - 16 * 32;
    const uint32_t at = smem_u32(&sh.stat[h]);
    float2 ml[kMaxCluster];
    float top = -INFINITY, total = 0.f;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      ml[s] = make_float2(-INFINITY, 0.f);
      if (s < p.splits)
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml[s].x), "=f"(ml[s].y) : "r"(in_cta(at, s)));
      top = fmaxf(top, ml[s].x);
    }
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s)
      if (ml[s].y != 0.f) total = fmaf(ml[s].y, exp2_fast((ml[s].x - top) * c), total);
    const float sink = p.sink_logit != nullptr && h < heads ? p.sink_logit[h0 + h] * kLog2e : -INFINITY;
    const float norm = 1.f / (total + exp2_fast(fmaf(-c, top, sink)));
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s)
      share[s * kHeadsPerItem + h] = ml[s].y == 0.f ? 0.f : exp2_fast((ml[s].x - top) * c) * norm;
    if (rank == 0 && p.lse != nullptr && h < heads)
      p.lse[(int64_t)t * p.n_h + h0 + h] = total == 0.f ? -INFINITY : fmaf(top, p.scale, logf(total));
  }
  cluster_sync();
#pragma unroll 1
  for (int i = threadIdx.x; i < heads * slice / 4; i += kThreads) {
    const int h = i >> (7 - log_splits), d = (i * 4) & (slice - 1);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int s = 0; s < p.splits; ++s) {
      const float4 v = *reinterpret_cast<const float4*>(buf + (s * kHeadsPerItem + h) * slice + d);
      const float f = share[s * kHeadsPerItem + h];
      sum.x = fmaf(f, v.x, sum.x);
      sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z);
      sum.w = fmaf(f, v.w, sum.w);
    }
    const uint2 v = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
    *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.n_h + h0 + h) * kWidth + rank * slice + d) = v;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    csa_attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + kQBytes;
  uint8_t* p_smem = ring + kPairs * kPairBytes;
  Shared& sh = *reinterpret_cast<Shared*>(p_smem + 2 * kPBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort = &sh.abort_flag;
  unsigned int* status = p.status;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need 1024-byte alignment: never seen otherwise
    if (threadIdx.x == 0) atomicOr(status, FM_DEV_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kTileSlots; ++i) mbar_init(&sh.kv_full[i], kKvArrivals);
    for (int i = 0; i < kPairs; ++i) mbar_init(&sh.kv_empty[i], 1);
    mbar_init(&sh.s_full, 2);
    mbar_init(&sh.s_empty, kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.p_full[i], kSoftmaxWarps);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.stage_free[i], 4);
    }
    mbar_init(&sh.q_full, 4);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.stat_full, 4);
    mbar_init(&sh.stat_empty, 4);
    for (int i = 0; i < kPairsPerTile; ++i) mbar_init(&sh.o_empty[i], 4);
    for (int i = 0; i < kInfoSlots; ++i) {
      mbar_init(&sh.info_full[i], 1);
      mbar_init(&sh.info_empty[i], kInfoReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.rows_full[i], 1);
      mbar_init(&sh.rows_empty[i], kProducerWarps);
    }
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_slot;
  // What is above overlaps the kernel before this one; what it wrote is read from
  // here on (by plain loads: a read-only one is for what no kernel before this one
  // can still be writing).  The kernel after may get ready likewise.
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int n_mine = (p.items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;

  if (warp == 1) {
    // -------------------------------- resolver ------------------------------
    bool ok = true;
    uint32_t g = 0;
    // the addresses and the mask of the next tile: rows lane and lane + 32
    auto publish = [&](const uint64_t (&row)[2], const bool (&seen)[2]) -> bool {
      uint2 mask;
      mask.x = __ballot_sync(0xffffffffu, seen[0]);
      mask.y = __ballot_sync(0xffffffffu, seen[1]);
      if (!warp_wait(&sh.rows_empty[g & 1], ((g >> 1) & 1) ^ 1, abort, status)) return false;
      const int to = (lane >> 4) * 16 + (lane & 1) * 8 + ((lane & 15) >> 1);
      sh.rows[g & 1][to] = row[0];
      sh.rows[g & 1][32 + to] = row[1];
      if (lane == 0) sh.key_mask[g & 7] = mask;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.rows_full[g & 1]);
      ++g;
      return true;
    };
#pragma unroll 1
    for (int i = 0; i < n_mine && ok; ++i) {
      const int slot = i % kInfoSlots;
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int split = item % p.splits, th = item / p.splits;
      const int t = th / p.head_blocks;
      const int64_t b = p.seq != nullptr ? p.seq[t] : t, pos = p.pos[t];
      // the tile of queries
      uint64_t row[2];
      bool seen[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int h = th % p.head_blocks * kHeadsPerItem + 32 * x + lane;
        seen[x] = h < p.n_h;
        row[x] = reinterpret_cast<uint64_t>(p.q + ((int64_t)t * p.n_h + (seen[x] ? h : 0)) * kWidth);
      }
      if (!(ok = publish(row, seen))) break;
      // listed cells up to the last one that is not empty
      int last = -1;
      const int32_t* cells = p.cells + (int64_t)t * p.k;
#pragma unroll 8
      for (int c = lane; c < p.k; c += 32)
        if (cells[c] >= 0) last = c;
      const int n_cells = __reduce_max_sync(0xffffffffu, last) + 1;
      const TokenKeys tk = token_keys(p, b, pos);
      const int end_first = n_cells + tk.n_first, end_win = end_first + tk.n_win, end = end_win + tk.n_tree;
      const uint32_t tiles = (uint32_t)(end + kTileKeys - 1) / kTileKeys;  // < 2^20, and at most 2^8 splits
      int tile = (int)(tiles * (uint32_t)split / (uint32_t)p.splits);
      int tile_end = (int)(tiles * (uint32_t)(split + 1) / (uint32_t)p.splits);
      if (tile == tile_end) {  // a split without keys still runs one tile, of no keys
        tile = (int)tiles;
        tile_end = tile + 1;
      }
      if (!warp_wait(&sh.info_empty[slot], ((i / kInfoSlots) & 1) ^ 1, abort, status)) break;
      if (lane == 0) {
        sh.info[slot] = ItemInfo{t, th % p.head_blocks, p.splits > 1 && !p.cluster ? item : -1, tile_end - tile};
        mbar_arrive(&sh.info_full[slot]);
      }
      const int tile_begin = tile;
      // The keys' indexes are read a tile ahead of their use.  Lane l resolves
      // keys l and l + 32: `raw` is a cell, or a page with `offset` in it, or -1.
      int raw[2], offset[2];
      auto fetch = [&](int at_tile) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int s = at_tile * kTileKeys + 32 * x + lane;
          raw[x] = -1;
          offset[x] = 0;
          if (s < n_cells) {
            raw[x] = cells[s];
          } else if (s < end) {
            int64_t at = s - n_cells;
            bool seen = true;
            if (s >= end_win) {
              const int d = s - end_win;
              seen = (p.tree_mask[(int64_t)t * p.tree_words + (d >> 5)] >> (d & 31)) & 1u;
              at = tk.base + d;
            } else if (s >= end_first) {
              at = tk.low + (s - end_first);
            }
            if (seen && at >= (int64_t)p.R * kPage) {
              atomicOr(status, FM_DEV_PAGE_RANGE);
            } else if (seen) {
              raw[x] = p.page_table[(int64_t)tk.b * p.R + (uint32_t)at / kPage];
              offset[x] = (int)((uint32_t)at % kPage);
            }
          }
        }
      };
      raw[0] = raw[1] = -1;
#pragma unroll 1
      for (--tile; tile < tile_end; ++tile) {  // the first pass only fetches
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool cell = tile * kTileKeys + 32 * x + lane < n_cells;
          seen[x] = raw[x] >= 0 && raw[x] < (cell ? p.cell_limit : p.P);
          if (raw[x] >= 0 && !seen[x]) atomicOr(status, FM_DEV_PAGE_RANGE);
          const int64_t r = cell ? (int64_t)((uint32_t)raw[x] / kPage) * p.cell_page_rows + (uint32_t)raw[x] % kPage
                                 : raw[x] * p.kv_page_rows + offset[x];
          // where nothing is read, an address all the same: a copy's source is on a
          // 16-byte border whatever its size, and q is the one input that is never
          // NULL and on such a border
          row[x] = seen[x] ? reinterpret_cast<uint64_t>((cell ? p.cell_pool : p.kv_pool) + r * kWidth)
                           : reinterpret_cast<uint64_t>(p.q);
        }
        if (tile + 1 < tile_end) fetch(tile + 1);
        if (tile >= tile_begin && !(ok = publish(row, seen))) break;
      }
    }
  } else if (warp >= 16) {
    // ------------------------------- producers ------------------------------
    // Producer w takes the tile's keys 16 w .. 16 w + 15.  Copy c of a pair moves
    // the rows of keys 2 c and 2 c + 1: lane l < 16 the 16-byte unit l of the
    // first, the others those of the second.
    const int me = warp - 16, hi = lane >> 4, unit = lane & 15;
    const uint32_t lane_dst = smem_u32(ring) + me * kKeysPerProducer * 128 + (unit >> 3) * kChunkBytes + hi * 128 +
                              (((unit & 7) ^ hi) << 4);
    uint32_t at_phase = 1, g = 0;
    int tile_slot = 0;
    int i = 0, left = 0;  // the current item, its tiles not yet copied
    uint64_t src[8];
    uint32_t valid = 0;   // bit 2 c: copy c reads
    auto take_rows = [&](uint32_t tile) {
      const ulonglong2* r = reinterpret_cast<const ulonglong2*>(&sh.rows[tile & 1][me * 16 + hi * 8]);
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const ulonglong2 x = r[c / 2];
        src[c] = x.x + unit * 16;
        src[c + 1] = x.y + unit * 16;
      }
      valid = (me & 2 ? sh.key_mask[tile & 7].y : sh.key_mask[tile & 7].x) >> ((me & 1) * 16 + hi);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.rows_empty[tile & 1]);
    };
    bool taken = false;
    // (the loops here stay rolled: unrolled, the roles' code outgrows the instruction cache)
#pragma unroll 1
    while (i < n_mine) {
      if (!taken) {
        if (!warp_wait(&sh.rows_full[g & 1], (g >> 1) & 1, abort, status)) break;
        take_rows(g);
      }
      if (left == 0) {  // the item's tile of queries: its info may come later
        left = -1;
      } else {
        if (left < 0) left = sh.info[i % kInfoSlots].tiles;
        if (--left == 0) ++i;
      }
      taken = false;
      bool ok = true;
      uint64_t from[8];
      uint32_t size[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        from[c] = src[c];
        size[c] = (valid >> (2 * c) & 1u) << 4;
      }
      // (only these four addresses and constant offsets: the issue of the copies is
      // one of the two things that bound a tile)
      const uint32_t slot_dst = lane_dst + tile_slot * (kPairsPerTile * kPairBytes);
      const uint32_t dst[4] = {slot_dst, slot_dst ^ 32, slot_dst ^ 64, slot_dst ^ 96};
      ++g;
#pragma unroll 1
      for (int j = 0; j < kPairsPerTile; ++j) {
        // the next tile's rows, where they are there already, before the last wait
        if (j == kPairsPerTile - 1 && i < n_mine &&
            __all_sync(0xffffffffu, mbar_test(&sh.rows_full[g & 1], (g >> 1) & 1))) {
          take_rows(g);
          taken = true;
        }
        if (!(ok = warp_wait(&sh.kv_empty[tile_slot * kPairsPerTile + j], at_phase, abort, status))) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) cp_async16(dst[c & 3] + c * 256 + j * kPairBytes, from[c] + 256 * j, size[c]);
      }
      if (!ok) break;
      cp_async_arrive(&sh.kv_full[tile_slot]);
      if (lane == 0) mbar_arrive(&sh.kv_full[tile_slot]);  // passes the mask on
      if (++tile_slot == kTileSlots) {
        tile_slot = 0;
        at_phase ^= 1;
      }
    }
    cp_async_wait_all();
  } else if (warp == 0) {
    // ------------------------------- S issuer -------------------------------
    const bool one = elect_one();
    const uint32_t idesc = idesc_bf16_f32(64, kTileKeys);
    const uint64_t q_desc = sdesc_sw128(smem_u32(q_smem));
    const uint64_t k_desc = sdesc_sw128(smem_u32(ring));
    uint32_t g = 0;                // key tiles
    uint32_t at = 0, at_phase = 0; // the current tile's slot in the ring, query tiles among them
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n_mine && ok; ++i) {
      const int slot = i % kInfoSlots;
      if (!warp_wait(&sh.info_full[slot], (i / kInfoSlots) & 1, abort, status)) break;
      const int tiles = sh.info[slot].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
      if (!warp_wait(&sh.q_full, i & 1, abort, status)) break;
      if (one)  // they have left the ring
        for (int j = 0; j < kPairsPerTile; ++j) mbar_arrive(&sh.kv_empty[at * kPairsPerTile + j]);
#pragma unroll 1
      for (int tile = 0; tile < tiles; ++tile, ++g) {
        if (++at == kTileSlots) {
          at = 0;
          at_phase ^= 1;
        }
        // (one wait to a tile: with one to each half or quarter the scores start earlier,
        // but the two issuers' products interleave more: tree of 61 tokens 77 -> 87 us)
        if (!(ok = warp_wait(&sh.kv_full[at], at_phase, abort, status))) break;
        if (!(ok = warp_wait(&sh.s_empty, (g & 1) ^ 1, abort, status))) break;
        fence_proxy_async();  // the copies were written through the generic proxy
        tc_fence_after();
        uint64_t b = k_desc + (uint64_t)(at * (kPairsPerTile * kPairBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t o = (uint64_t)((kk >> 2) * (kChunkBytes >> 4) + (kk & 3) * 2);
          if (one) umma_bf16_ss(tmem + kSCol, q_desc + o, b + o, idesc, kk == 0 ? 0u : 1u);
        }
        uint32_t a = tmem + kQCol;
#pragma unroll 1
        for (int j = 1; j < kPairsPerTile; ++j) {
          b += (uint64_t)(kPairBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kChunkBytes >> 4) + (kk & 3) * 2);
            if (one) umma_bf16_ts(tmem + kSCol, a + 8 * kk, b + o, idesc, 1u);
          }
          a += 64;
        }
        if (one) {
          umma_commit(&sh.s_full);
          mbar_arrive(&sh.s_full);  // passes the mask on
        }
      }
      if (ok && one) umma_commit(&sh.q_empty);
      if (++at == kTileSlots) {  // the next item's queries
        at = 0;
        at_phase ^= 1;
      }
    }
    if (one) umma_commit(&sh.drain[0]);
    if (one) wait_drain(&sh.drain[0]);
  } else if (warp == 2) {
    // ------------------------------- O issuer -------------------------------
    const bool one = elect_one();
    const uint64_t v_desc = sdesc_mn_sw128(smem_u32(ring));
    const uint64_t p_desc = sdesc_sw128(smem_u32(p_smem));
    uint32_t g = 0, at = 0;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n_mine && ok; ++i) {
      const int slot = i % kInfoSlots;
      if (!warp_wait(&sh.info_full[slot], (i / kInfoSlots) & 1, abort, status)) break;
      const int tiles = sh.info[slot].tiles, heads = min(kHeadsPerItem, p.n_h - sh.info[slot].head_block * kHeadsPerItem);
      // N: the heads there are, to a multiple of 16 (a reduction's result is a uniform
      // value, and an MMA whose operands are not costs its issuer twice the time)
      const uint32_t idesc = (idesc_bf16_f32(128, 0) | kAIsMnMajor) | ((uint32_t)__reduce_max_sync(0xffffffffu, (heads + 15) / 16) << 18);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
      at += kPairsPerTile;  // the tile of queries
      if (at == (uint32_t)kPairs) at = 0;
#pragma unroll 1
      for (int tile = 0; tile < tiles && ok; ++tile, ++g) {
        if (!(ok = warp_wait(&sh.p_full[g & 1], (g >> 1) & 1, abort, status))) break;
        tc_fence_after();
        const uint64_t b = p_desc + (uint64_t)((g & 1) * (kPBytes >> 4));
#pragma unroll
        for (int m = 0; m < kPairsPerTile; ++m) {  // a pair of chunks is a block of 128 elements
          if (tile == 0) {  // the block of the last item has been read
            if (!(ok = warp_wait(&sh.o_empty[m], (i & 1) ^ 1, abort, status))) break;
            tc_fence_after();
          }
          const uint64_t a = v_desc + (uint64_t)(at * (kPairBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < kTileKeys / 16; ++kk)
            if (one) umma_bf16_ss(tmem + m * kHeadsPerItem, a + kk * (2048 >> 4), b + kk * 2, idesc, kk == 0 ? (uint32_t)tile : 1u);
          if (one) umma_commit(&sh.kv_empty[at]);
          if (++at == (uint32_t)kPairs) at = 0;
        }
        if (!ok) break;
        if (one) umma_commit(&sh.pv_done[g & 1]);
      }
      if (ok && one) umma_commit(&sh.o_full);
    }
    if (one) umma_commit(&sh.drain[1]);
    if (one) wait_drain(&sh.drain[1]);
  } else if (warp >= 4 && warp < 4 + kSoftmaxWarps) {
    // ------------------------------- softmax --------------------------------
    // Warps quad and quad + 4 hold heads 16 quad .. 16 quad + 15 of the block (S's
    // rows in the first 16 lanes of TMEM quadrant quad), each 32 of the tile's
    // keys; a thread has two heads, r0 and r0 + 8, and eight keys of each.
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r0 = quad * 16 + lane / 4;
    const float c = p.scale * kLog2e;
    // P is K-major in rows (heads) of 128 bytes, SWIZZLE_128B: this lane's row of
    // the eight 8 x 8 matrices that the warp stores
    const uint32_t p_dst = smem_u32(p_smem) + (quad * 16 + (lane & 7)) * 128 + (((4 * half + (lane >> 3)) ^ (lane & 7)) << 4);
    uint32_t g = 0;
    uint32_t staged = 0;  // bit b: P buffer b is lent to an epilogue; bit 2 + b: the phase it ends with
    bool dead = false;
#pragma unroll 1
    for (int i = 0; i < n_mine; ++i) {
      const int slot = i % kInfoSlots;
      bool ok = !dead && warp_wait(&sh.info_full[slot], (i / kInfoSlots) & 1, abort, status);
      if (softmax_any(!ok)) break;
      const int tiles = sh.info[slot].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // m in units of S, l of this thread's keys
      bool left = false;
#pragma unroll 1
      for (int tile = 0; tile < tiles; ++tile, ++g) {
        ok = !dead && warp_wait(&sh.s_full, g & 1, abort, status);
        uint32_t raw[16], w[8];
        float top[2] = {-INFINITY, -INFINITY}, sum[2];
        bool need = false, p_free = false;
        if (ok) {
          tc_fence_after();
          tmem_ld_16x256b_x4(tmem + ((uint32_t)(quad * 32) << 16) + kSCol + 32 * half, raw);
          const uint32_t mask = half ? sh.key_mask[(g + i + 1) & 7].y : sh.key_mask[(g + i + 1) & 7].x;
          p_free = mbar_test(&sh.pv_done[g & 1], ((g >> 1) & 1) ^ 1);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_empty);
          if (mask != 0xffffffffu) {
            const uint32_t seen = mask >> (2 * (lane & 3));
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (((seen >> (8 * j + e)) & 1u) == 0) raw[4 * j + e] = raw[4 * j + 2 + e] = 0xFF800000u;  // -inf
          }
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              top[r] = fmaxf(top[r], fmaxf(__uint_as_float(raw[4 * j + 2 * r]), __uint_as_float(raw[4 * j + 2 * r + 1])));
          // the maximum in use may be passed by up to 2^8 before the sums so far
          // are rescaled: the weights' bf16 and the fp32 sums lose nothing by it
          need = top[0] * c > m[0] * c + 8.f || top[1] * c > m[1] * c + 8.f;
        }
        // Weights under the maximum in use, before it is known whether that
        // holds; where it does not, once more under the new one.
#pragma unroll 1
        for (bool renew = tile == 0, last = false;; renew = true) {
          if (!renew || last) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float mc = m[r] == -INFINITY ? 0.f : m[r] * c;
              sum[r] = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float a = exp2_fast(fmaf(__uint_as_float(raw[4 * j + 2 * r]), c, -mc));
                const float b = exp2_fast(fmaf(__uint_as_float(raw[4 * j + 2 * r + 1]), c, -mc));
                sum[r] += a + b;
                w[4 * r + j] = pack_bf16(a, b);
              }
            }
            if (last || !softmax_any(need || !ok)) break;
          }
          // a new maximum: the heads' tops over both halves of the keys
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            if ((lane & 3) == 0) sh.top_half[half][r0 + 8 * r] = top[r];
          }
          left = softmax_any(!ok);
          if (left) break;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], sh.top_half[half ^ 1][r0 + 8 * r]);
            if (tile == 0) {
              m[r] = top[r];
            } else {
              float f = 1.f;
              if (top[r] * c > m[r] * c + 8.f) {
                f = m[r] == -INFINITY ? 0.f : exp2_fast((m[r] - top[r]) * c);
                m[r] = top[r];
              }
              l[r] *= f;
              if (half == 0 && (lane & 3) == 0) sh.rescale[r0 + 8 * r] = f;
            }
          }
          if (tile > 0) {
            const uint32_t gp = g - 1;
            ok = warp_wait(&sh.pv_done[gp & 1], (gp >> 1) & 1, abort, status);
            left = softmax_any(!ok);
            if (left) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 4 * half; x < 4 * half + 4; ++x) {
              uint32_t o[32];
              const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + 32 * x;
              tmem_ld32(addr, o);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 32; ++h)
                o[h] = __float_as_uint(__uint_as_float(o[h]) * sh.rescale[(x & 1) * 32 + h]);
              tmem_st32(addr, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          last = true;
        }
        if (left) break;
        l[0] += sum[0];
        l[1] += sum[1];
        if (!__all_sync(0xffffffffu, p_free) && !warp_wait(&sh.pv_done[g & 1], ((g >> 1) & 1) ^ 1, abort, status)) {
          dead = true;  // leave together with the others, at the next tile or item
          continue;
        }
        // an epilogue staged its output in this buffer
        if (staged >> (g & 1) & 1u) {
          staged ^= 1u << (g & 1);
          if (!warp_wait(&sh.stage_free[g & 1], staged >> (2 + (g & 1)) & 1u, abort, status)) {
            dead = true;
            continue;
          }
          staged ^= 4u << (g & 1);
        }
        const uint32_t dst = p_dst + (g & 1) * kPBytes;
        store_8x8_x4(dst, w[0], w[1], w[2], w[3]);
        store_8x8_x4(dst + 8 * 128, w[4], w[5], w[6], w[7]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[g & 1]);
      }
      if (left) break;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
      staged |= 1u << ((g - 1) & 1);
      if (!dead && !warp_wait(&sh.stat_empty, (i & 1) ^ 1, abort, status)) dead = true;
      // the upper halves' sums pass to the lower ones
      if (!dead && half == 1 && (lane & 3) == 0) {
        sh.stat[r0].y = l[0];
        sh.stat[r0 + 8].y = l[1];
      }
      if (softmax_any(dead)) break;
      if (half == 0) {
        if ((lane & 3) == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r) sh.stat[r0 + 8 * r] = make_float2(m[r], l[r] + sh.stat[r0 + 8 * r].y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.stat_full);
      }
    }
  } else if (warp >= 12) {  // (warp 3 has no role)
    // ------------------------------- epilogue -------------------------------
    // A warp has 32 elements (TMEM lanes) of every head.  The output is staged,
    // transposed, 32 heads x 32 elements at a time in a quarter of the P buffer
    // that the item's last tile is done with.
    const int quad = warp & 3;
    const float c = p.scale * kLog2e;
    uint32_t g = 0;
    uint32_t at = 0;  // the current item's tile of queries: its number in the ring's stream, modulo 2 * kTileSlots
    // The queries of item i, from the ring to their place: the first two chunks to
    // shared memory as they are, the others to TMEM: heads 16 quad .. 16 quad + 15,
    // head r in lanes r and r + 16 of the quadrant (an M of 64 has its rows in 16
    // lanes of each quadrant), elements 2 x and 2 x + 1 of a chunk in its column x.
    auto queries = [&](int i) -> bool {
      const uint32_t tile = at % kTileSlots;
      // (in this order: the slot's phases before this one, which these warps do not
      // wait for, are over once the last item's scores are)
      if (!warp_wait(&sh.q_empty, (i & 1) ^ 1, abort, status)) return false;
      if (!warp_wait(&sh.kv_full[tile], at / kTileSlots, abort, status)) return false;
      tc_fence_after();
      const uint32_t from = smem_u32(ring) + tile * kPairsPerTile * kPairBytes;
      const uint32_t copy = (quad * 32 + lane) * 16;
#pragma unroll
      for (int x = 0; x < kQBytes / 2048; ++x) store_shared_16(smem_u32(q_smem) + copy + x * 2048, load_shared_16(from + copy + x * 2048));
      const int row = quad * 16 + (lane & 15);
#pragma unroll 1
      for (int c = 2; c < 8; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint4 u = load_shared_16(from + c * kChunkBytes + row * 128 + ((x ^ (row & 7)) << 4));
          v[4 * x] = u.x;
          v[4 * x + 1] = u.y;
          v[4 * x + 2] = u.z;
          v[4 * x + 3] = u.w;
        }
        tmem_st32(tmem + ((uint32_t)(quad * 32) << 16) + kQCol + 32 * (c - 2), v);
      }
      tmem_st_wait();
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      return true;
    };
    bool ok = n_mine == 0 || queries(0);
#pragma unroll 1
    for (int i = 0; i < n_mine && ok; ++i) {
      const int slot = i % kInfoSlots;
      if (!warp_wait(&sh.info_full[slot], (i / kInfoSlots) & 1, abort, status)) break;
      const int t = sh.info[slot].t, h0 = sh.info[slot].head_block * kHeadsPerItem, part = sh.info[slot].part;
      g += (uint32_t)sh.info[slot].tiles;
      at = (at + 1u + (uint32_t)sh.info[slot].tiles) % (2 * kTileSlots);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
      const int heads = min(kHeadsPerItem, p.n_h - h0);
      float sink[2] = {-INFINITY, -INFINITY};  // of heads lane and lane + 32
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (p.sink_logit != nullptr && lane + 32 * r < heads) sink[r] = p.sink_logit[h0 + lane + 32 * r] * kLog2e;
      if (i + 1 < n_mine && !(ok = queries(i + 1))) break;
      if (!warp_wait(&sh.stat_full, i & 1, abort, status)) break;
      if (p.cluster) {  // the whole CTA sees to it, below
        (void)warp_wait(&sh.o_full, i & 1, abort, status);
        break;
      }
      const float2 stat[2] = {sh.stat[lane], sh.stat[lane + 32]};
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.stat_empty);
      float factor[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        factor[r] = stat[r].y == 0.f ? 0.f : 1.f / (stat[r].y + exp2_fast(fmaf(-c, stat[r].x, sink[r])));
        if (quad == 0) {
          if (part >= 0)
            p.part_ml[(int64_t)part * kHeadsPerItem + lane + 32 * r] = stat[r];
          else if (p.lse != nullptr && lane + 32 * r < heads)
            p.lse[(int64_t)t * p.n_h + h0 + lane + 32 * r] = 
                stat[r].y == 0.f ? -INFINITY : fmaf(stat[r].x, p.scale, logf(stat[r].y));
        }
      }
      if (!warp_wait(&sh.o_full, i & 1, abort, status)) break;
      if (i == n_mine - 1) {  // the whole CTA stores the last item, below
        if (quad == 0) {
          sh.rescale[lane] = factor[0];
          sh.rescale[lane + 32] = factor[1];
        }
        break;
      }
      tc_fence_after();
      const Output out = {p, tmem, smem_u32(p_smem) + ((g - 1) & 1) * kPBytes + quad * kStageBytes, t, h0, -1};
#pragma unroll 1
      for (int x = 0; x < 8; ++x) {
        if ((x & 1) && heads <= 32) {
          if (lane == 0) mbar_arrive(&sh.o_empty[x >> 1]);
          continue;
        }
        const float mine = x & 1 ? factor[1] : factor[0];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __shfl_sync(0xffffffffu, mine, 8 * (j >> 1) + 2 * (lane & 3) + (j & 1));
        out.half_block(x, quad, lane, f, [&] {
          if ((x & 1) && lane == 0) mbar_arrive(&sh.o_empty[x >> 1]);
        });
      }
      if (lane == 0) mbar_arrive(&sh.stage_free[(g - 1) & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.cluster) {
    join_cluster(p, sh, reinterpret_cast<float*>(ring), reinterpret_cast<float*>(p_smem), tmem);
  } else if (n_mine > 0 && sh.abort_flag == 0) {
    // the last item, by all warps: a half block of its output at a time each
    const ItemInfo f = sh.info[(n_mine - 1) % kInfoSlots];
    const Output out = {p, tmem, smem_u32(ring) + warp * kStageBytes, f.t, f.head_block * kHeadsPerItem, f.part};
#pragma unroll 1
    for (int x = warp >> 2; x < 8; x += kThreads / 128) {
      if ((x & 1) && p.n_h - out.h0 <= 32) continue;
      float fac[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) fac[j] = sh.rescale[(x & 1) * 32 + 8 * (j >> 1) + 2 * (lane & 3) + (j & 1)];
      if (f.part >= 0)
        out.half_block_partial(x, warp & 3, lane);
      else
        out.half_block(x, warp & 3, lane, fac, [] {});
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits of one (token, head): out = sum_s 2^(m_s - M) O_s / (sum_s
// 2^(m_s - M) l_s + sink).  Four groups of 128 threads (four elements to a thread)
// take every fourth split, eight of them in flight; their sums meet in shared
// memory.  The order of all sums is fixed.
constexpr int kMergeGroups = 4;
constexpr int kMergeThreads = 128 * kMergeGroups;
__global__ void __launch_bounds__(kMergeThreads) csa_merge_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float weight[kMaxParts], warp_top[kMaxParts / 32], warp_sum[kMaxParts / 32];
  __shared__ float4 group_sum[kMergeGroups - 1][128];
  static_assert(kMaxParts <= kMergeThreads, "a split to a thread");
  const int64_t th = blockIdx.x;
  const int h = (int)(th % p.n_h), hl = h % kHeadsPerItem;
  const int64_t t = th / p.n_h;
  const int64_t part0 = (t * p.head_blocks + h / kHeadsPerItem) * p.splits;
  const int tid = threadIdx.x, group = tid / 128, d = 4 * (tid % 128);
  const float c = p.scale * kLog2e;
  grid_dep_wait();  // for the partial results
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid < p.splits) ml = p.part_ml[(part0 + tid) * kHeadsPerItem + hl];
  if (tid < kMaxParts) {
    float top = ml.x;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (tid % 32 == 0) warp_top[tid / 32] = top;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) top = fmaxf(top, warp_top[i]);
  if (tid < kMaxParts) {
    const float w = ml.y == 0.f ? 0.f : exp2_fast((ml.x - top) * c);  // a split without keys holds zeros
    weight[tid] = w;
    float part = w * ml.y;
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (tid % 32 == 0) warp_sum[tid / 32] = part;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) sum += warp_sum[i];
  const float sink = p.sink_logit != nullptr ? p.sink_logit[h] * kLog2e : -INFINITY;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* from = p.part_o + (part0 * kHeadsPerItem + hl) * kWidth + d;
  for (int s0 = group; s0 < p.splits; s0 += 8 * kMergeGroups) {
    float4 o[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int s = s0 + x * kMergeGroups;
      o[x] = s < p.splits ? *reinterpret_cast<const float4*>(from + (int64_t)s * kHeadsPerItem * kWidth)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float w = weight[(s0 + x * kMergeGroups) % kMaxParts];  // (past the last split: of zeros)
      acc.x = fmaf(w, o[x].x, acc.x);
      acc.y = fmaf(w, o[x].y, acc.y);
      acc.z = fmaf(w, o[x].z, acc.z);
      acc.w = fmaf(w, o[x].w, acc.w);
    }
  }
  if (group > 0) group_sum[group - 1][tid % 128] = acc;
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int g = 0; g < kMergeGroups - 1; ++g) {
    const float4 v = group_sum[g][tid];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float f = sum == 0.f ? 0.f : 1.f / (sum + exp2_fast(fmaf(-c, top, sink)));
  const uint2 v = make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
  *reinterpret_cast<uint2*>(p.out + th * kWidth + d) = v;
  if (p.lse != nullptr && tid == 0) p.lse[th] = sum == 0.f ? -INFINITY : fmaf(top, p.scale, logf(sum));
}

int head_blocks_of(int n_h) { return (n_h + kHeadsPerItem - 1) / kHeadsPerItem; }

size_t attn_workspace_bytes(int T, int n_h) {
  const int64_t items = (int64_t)T * head_blocks_of(n_h);
  if (items == 0 || items > kMaxParts / 2) return 0;  // such calls never split
  const int64_t parts = kMaxParts / items * items;
  return (size_t)parts * kHeadsPerItem * (kWidth * sizeof(float) + sizeof(float2));
}

// Clusters of c CTAs of the attention kernel that fit the current device at once.
// (Asked once per device and size: it does not change.)
int max_clusters(int c) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  std::atomic<int>* slot = dev < 64 ? &known[dev][c] : nullptr;
  if (slot != nullptr && slot->load(std::memory_order_relaxed) > 0) return slot->load(std::memory_order_relaxed);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)c, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, csa_attn_kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (slot != nullptr) slot->store(n, std::memory_order_relaxed);
  return n;
}

fm_status launch_attn(AttnParams& p, int sms, void* workspace, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(csa_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return set_error(FM_ERR_CUDA, "fm_csa_attn: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  p.head_blocks = head_blocks_of(p.n_h);
  const int64_t items = (int64_t)p.T * p.head_blocks;
  // tiles that a token can have at most
  const int64_t held = (int64_t)p.R * kPage;
  const int64_t slots = (p.window < held ? p.window : held) + (p.n_sink < held ? p.n_sink : held) + p.k +
                        (p.tree_mask != nullptr ? 32 * p.tree_words : 0);
  const int64_t max_tiles = (slots + kTileKeys - 1) / kTileKeys;
  const int64_t free_sms = items <= kMaxParts / 2 ? (sms < kMaxParts ? sms : kMaxParts) / items : 1;
  int64_t splits = free_sms < max_tiles ? free_sms : max_tiles;
  if (splits < 1) splits = 1;
  p.cluster = 0;
  if (splits > 1) {
    // The largest cluster of which enough fit at once; the split over all SMs
    // through memory where it saves a CTA more than eight tiles: a tile is some
    // 1.1 us, the partial results' way through memory and the second kernel some 8 us.
    int c = kMaxCluster;
    while (c > 1 && (c > splits || max_clusters(c) < items)) c /= 2;
    if ((max_tiles + c - 1) / c <= (max_tiles + splits - 1) / splits + 8) {
      p.cluster = c > 1;
      splits = c;
    }
  }
  p.splits = (int)splits;
  p.items = (int)(items * splits);
  const size_t parts = (size_t)p.items;
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + parts * kHeadsPerItem * sizeof(float2));

  // programmatic dependent launch: a kernel's set-up overlaps the one before it
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(p.cluster || p.items < sms ? p.items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.cluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)p.splits, 1, 1};
    cfg.numAttrs = 2;
  }
  if ((e = cudaLaunchKernelEx(&cfg, csa_attn_kernel, (const AttnParams)p)) != cudaSuccess)
    return set_error(FM_ERR_CUDA, "fm_csa_attn: launch: %s", cudaGetErrorString(e));
  if (p.splits > 1 && !p.cluster) {
    cfg.gridDim = dim3((unsigned)((int64_t)p.T * p.n_h));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, csa_merge_kernel, (const AttnParams)p)) != cudaSuccess)
      return set_error(FM_ERR_CUDA, "fm_csa_attn: merge launch: %s", cudaGetErrorString(e));
  }
  return FM_OK;
}

fm_status csa_attn(const char* who, bool tree, const uint16_t* q, int T, int n_h, int d, const uint16_t* kv_pool,
                   int64_t P, int64_t kv_page_stride, const int32_t* page_table, int B, int R, const int32_t* seq,
                   const int64_t* pos, int64_t window, int n_sink, const uint16_t* cell_pool, int64_t Pc,
                   int64_t cell_page_stride, const int32_t* cells, int k, const float* sink_logit, float scale,
                   const uint32_t* tree_mask, int tree_words, const int64_t* tree_base, uint16_t* out, float* lse_out,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (d != kWidth) return set_error(FM_ERR_INVALID_ARG, "%s: d=%d (need 512)", who, d);
  if (T < 0 || n_h < 1 || n_h > 1024 || (int64_t)T * head_blocks_of(n_h) >= kMaxItems)
    return set_error(FM_ERR_INVALID_ARG, "%s: bad sizes T=%d n_h=%d (1 <= n_h <= 1024, T * ceil(n_h / 64) < 2^23)", who,
                     T, n_h);
  if (B < 0 || R < 0 || R > kMaxTable || window < 0 || n_sink < 0 || k < 0 || k > kMaxCells)
    return set_error(FM_ERR_INVALID_ARG,
                     "%s: bad sizes B=%d R=%d window=%lld n_sink=%d k=%d (R <= 2^19, 0 <= k <= 1024)", who, B, R,
                     (long long)window, n_sink, k);
  if (!(scale > 0.0f) || isinf(scale * kLog2e)) return set_error(FM_ERR_INVALID_ARG, "%s: scale=%g", who, (double)scale);
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
  p.cell_pool = cell_pool;
  p.page_table = page_table;
  p.seq = seq;
  p.pos = pos;
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

FM_API fm_status fm_csa_attn_packed(const fm_csa_attn_args* a) {
  if (!a) return fm::set_error(FM_ERR_INVALID_ARG, "fm_csa_attn_packed: args is NULL");
  const bool tree = a->tree != 0;
  return fm::csa_attn(tree ? "fm_csa_attn_tree" : "fm_csa_attn", tree, a->q, a->T, a->n_h, a->d, a->kv_pool, a->P,
                      a->kv_page_stride, a->page_table, a->B, a->R, a->seq, a->pos, a->window, a->n_sink, a->cell_pool,
                      a->Pc, a->cell_page_stride, a->cells, a->k, a->sink_logit, a->scale, tree ? a->tree_mask : nullptr,
                      tree ? a->tree_words : 0, tree ? a->tree_base : nullptr, a->out, a->lse_out, a->workspace,
                      a->workspace_bytes, reinterpret_cast<cudaStream_t>(a->stream));
}
