// Causal attention of a chunk of new tokens over the KV cache (include/mfa.h:
// mfa_chunk_attn), on the sm_100a tensor cores, for bf16 and FP8 (e4m3) caches:
//     out[t][h] = sum_{j <= p_t} softmax_j(scale q[t][h] . K[j]) V[j],  p_t the token's position.
//
// All 64 heads share K and V, so the rows of q ([token][head], 256 dimensions) of consecutive
// tokens form one tall matrix against the same keys. A tile is 4 tokens = 256 rows, worked on
// by a pair of CTAs on two neighbouring SMs (tcgen05 cta_group::2, M = 256: 128 rows a CTA).
// Per block of 128 keys
//     S[256 x 128] = Q[256 x 256] . K^T          O[256 x 256] += P[256 x 128] . V
// Each CTA loads half of K (64 keys) and half of V (128 of the 256 dimensions); the tensor
// cores of both read both halves, so a pair streams 128 KB (bf16) per block for 256 rows: 32
// bytes per SM and cycle at full tensor rate, half of what one CTA by itself would need from
// L2. A pair keeps up with HBM even when one token a sequence leaves 3/4 of its rows idle
// (a block takes the tensor cores 2048 cycles, and 1/74 of the measured bandwidth ~2800), so
// the same kernel serves decoding and prompts.
//
// Tensor memory (512 columns): O in 256, two S buffers of 128. P overwrites its own S (16-bit:
// the first 64 of the 128 columns) and is read by the product as the tensor-memory operand, so
// it never passes through shared memory. Shared memory: Q 64 KB, and a ring of nine 16 KB
// slots for K and V halves. Warps:
//   warp 0      TMA producer of this CTA's halves (rows of 64 keys a box, 128-byte swizzle)
//   warp 1      in the pair's first CTA: issues the products of both (one elected lane), in
//               the order S(t + 1), O += P(t) V(t), so that S(t + 1) runs during the softmax
//               of t; owns the tensor memory
//   warps 2..9  softmax: two threads per row, 64 of the 128 keys each. Scores stay raw; a
//               row's running maximum is raised only when a block exceeds it by more than 8
//               in log2 (4 for FP8), so O is rarely rescaled; the pair of warps that shares 32
//               rows agrees on that with one barrier a block. Sums in float32, of the
//               unrounded weights.
// FP8 caches: the codes go to the tensor cores as they are (kind::f8f6f4). Q becomes a pair of
// e4m3 matrices, high part and rounded remainder, P an e4m3 and an e5m2 matrix (split_weights),
// both accumulated into the same S or O: twice the products at twice the rate, and half the bytes
// of K and V. Q's scale is a power of two per row. P is 2^8 where the score is the running maximum
// and below 2^12 everywhere. (With 2^8.75 as the limit no weight would need its e5m2 part first, but
// the running maximum would rise more often: 957 us instead of 846 for two prompts of 1500 over
// 4500, where e4m3 pairs up to 2^8 took 808.)
//
// Work split: tiles of all sequences laid end to end, each costing its blocks plus
// kTileCost; pair g takes the g-th of G equal contiguous ranges, so causal chunks, prompts
// and decoding sequences balance to within a block whatever the mix. A range that starts or
// ends inside a tile leaves (m, l, O) partials in one of the pair's two slots, merged in a
// fixed order by chunk_combine_kernel. Where there are fewer tiles than pairs, each tile is
// instead cut evenly among pairs of its own if that is about as short: half as many partials,
// and no pair has two items (32 sequences of 4096 and 4 tokens: 46.2 -> 44.7 us).
//
// Blocks that hold keys some token of the tile does not see are "special": at most the last
// two of a tile. Their scores are masked by selection, so nothing a hidden key holds reaches a
// weight; and as 0 x NaN is NaN, V rows past the tile's last position are zeroed on chip, and
// rows that only its later tokens see are zeroed if they hold an infinity or NaN and then
// added in float32 for the tokens that do see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "chunk.cuh"
#include "sm100.cuh"

namespace mfa {
namespace {

using namespace sm100;

constexpr int kTokens = kChunkRows / kHeads;  // 4 tokens a tile
constexpr int kRows = 128;                    // rows of a CTA (tensor-memory lanes)
constexpr int kCtaTokens = kRows / kHeads;    // 2
constexpr int kBlock = 128;                   // keys of a block
constexpr int kSlotBytes = 16384;
constexpr int kSlots = 9;
constexpr int kBoxBytes = kChunkBoxRows * 128;  // [64 rows x 128 bytes]
constexpr int kQChunkBytes = kRows * 128;       // [128 rows x 128 bytes]
constexpr int kSoftmaxWarps = 8;
constexpr int kHelperWarp = 2 + kSoftmaxWarps;
constexpr int kThreads = 32 * (kHelperWarp + 1);
constexpr int kStageSlots = 4;  // ring slots that a finished tile's 128 x 256 bf16 results take
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemCols = 512;
constexpr int kTileCost = 3;  // a tile's fixed cost, in blocks (Q, first softmax, epilogue)
constexpr int kPartCost = 2;  // what a second part in a pair costs over a tile's start, in blocks
constexpr int kMaxShared = 128;  // (pairs of SMs, at most)
static_assert(2 * kMaxShared >= kMaxAttnGrid, "every pair");
constexpr uint64_t kLandNs = 1000000;  // by when a copy in flight has landed (they take ~1 us)
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kIdescE5m2A = 1u << 7;  // kind::f8f6f4: A's format is e5m2 (0: e4m3)

template <bool kFp8>
struct Cfg {
  static constexpr int kKSlots = kFp8 ? 1 : 2;  // ring slots of a CTA's half of a K block
  static constexpr int kVSlots = kFp8 ? 1 : 2;
  static constexpr float kRescale = kFp8 ? 4.0f : 8.0f;  // log2 units
  static constexpr float kPExp = kFp8 ? 8.0f : 0.0f;     // P = 2^(s - m + kPExp)
  static constexpr uint32_t kIdescS = idesc_f16(256, kBlock, !kFp8, false, false);
  static constexpr uint32_t kIdescPV = idesc_f16(256, kHeadDim, !kFp8, false, true);
};

struct Plan {
  int32_t cost[kMaxBatch + 1];   // exclusive prefix of the sequences' costs
  int32_t start[kMaxBatch + 1];  // q_start
  int32_t len[kMaxBatch];        // seq_lens; -1: refused, its rows get zeros
  const int32_t* pages;          // paged: the page table, `page_stride` entries a sequence
  int32_t page_stride;
  // this pair's share: units [begin, end), the first of them in tile `tile` of sequence b, which
  // begins at unit pos; or (shared, see share_tiles) blocks [begin, end) of that tile alone,
  // one of `parts`
  int32_t begin, end, pos, b, tile, shared, parts;
  int32_t pairs;                 // pairs with a share
  int32_t tile_blk[kMaxShared];  // share_tiles: every tile's blocks
};

struct __align__(1024) Smem {
  uint8_t q[4 * kQChunkBytes];
  uint8_t ring[kSlots * kSlotBytes];
  Plan plan;
  float xch[2][kRows];        // exchange between the two threads of a row: their maxima of a block
  // their sums of an item. (Not in xch: a thread may come here before its partner has read the
  // last block's maximum. Rows of missing tokens have neither, and no barrier: the next write
  // here lies behind a barrier of a row that has, and so behind this item's reads.)
  float sum[2][kRows];
  // FP8: exponent of each row's scale of Q, by the item's parity (warps write the next item's
  // before all have read this one's; the barrier behind those orders the item after it)
  int32_t q_exp[2][kRows];
  uint64_t kv_full[kSlots];   // first CTA: both halves of a slot have landed (and are clean)
  uint64_t kv_empty[kSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2];
  // this CTA: the V half of its i-th special block has landed, by i modulo kSlots. (Not by the
  // slot: only the helper warp waits for these, and it may be several uses of a slot behind
  // the producer or ahead of it. Special block i + kSlots cannot be loaded before block i is
  // used up, and the helper sees every one of them.)
  uint64_t v_full[kSlots];
  uint64_t pv_done[2];        // by the block's parity: a waiter is at most one block behind
  uint64_t o_free;
  uint64_t stage_free;        // the ring slots for a tile's results are free
  uint64_t staged;            // this CTA's results of a tile are in them
  uint64_t mma_done;
  // [item parity][V half]: late rows held out of the product (bad_flag). The item's number tells
  // it from an older one, so nobody has to put it back to zero and wait for those who read it.
  uint32_t bad[2][2];
  uint32_t tmem_base;
  int32_t abort_flag;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory per CTA");

// ---------------------------------------------------------------------------------------
// pair (cluster of two CTAs) primitives
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// True on one lane of the (converged) warp. Unlike a lane test, it tells the compiler that one
// thread runs what depends on it: descriptors then go through uniform registers, and eight
// products are issued in ~100 cycles instead of ~500 (they take the tensor core 512).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}

// shared::cluster address of this CTA's `p` in CTA `rank` of the pair
__device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// Arrive on a barrier of either CTA. The plain form is for what the tensor cores read: tensor
// memory (with tcgen05.fence) and the arriving CTA's own shared memory (with fence.proxy.async).
// The release form also orders what threads of the other CTA read, and waits ~1000 cycles for
// that: for flags only.
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void remote_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void remote_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ void remote_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// TMA loads into this CTA that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                             uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, int x, int y,
                                             int z, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// A box of shared memory to a tensor in global memory.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Wait until all but the last N groups of stores of this thread have read their shared memory.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "n"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
               "n"(kTmemCols)
               : "memory");
}

// Arrive on `bar` of both CTAs when every tcgen05 operation issued so far is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "{\n"
      ".reg .b16 m;\n"
      "mov.b16 m, 3;\n"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], m;\n"
      "}\n" ::"r"(smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptors of the tiles here (128-byte swizzle, 8-row groups 1024 bytes
// apart): the low word, to which a byte offset of x adds x / 16, and the constant high word.
// lbo: the distance of 64-element column groups of an MN-major operand (else ignored).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A . B over the pair; A in shared memory (SS) or tensor memory (TS).
template <bool kFp8>
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t acc) {
  if constexpr (kFp8)
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 a, b;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "mov.b64 a, {%1, %5};\n"
        "mov.b64 b, {%2, %5};\n"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n"
        "}\n" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
  else
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 a, b;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "mov.b64 a, {%1, %5};\n"
        "mov.b64 b, {%2, %5};\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n"
        "}\n" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
}
template <bool kFp8>
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                            uint32_t acc) {
  if constexpr (kFp8)
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 b;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "mov.b64 b, {%2, %5};\n"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [%1], b, %3, p;\n"
        "}\n" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
  else
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 b;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "mov.b64 b, {%2, %5};\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n"
        "}\n" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
}

// ---------------------------------------------------------------------------------------
// the work split
// ---------------------------------------------------------------------------------------

// sum_{i = 1}^{m} ceil((p + 4 i) / 128): with a = p + 127 = 4 c + r, floor((a + 4 i) / 128) =
// floor((c + i) / 32), so it is a difference of G(x) = sum_{j <= x} floor(j / 32).
__device__ __forceinline__ int block_sum(int p, int m) {
  auto G = [](int x) {
    const int q = x >> 5;
    return 16 * q * (q - 1) + q * ((x & 31) + 1);
  };
  const int c = (p + kBlock - 1) >> 2;
  return G(c + m) - G(c);
}

// Cost of the tiles before tile m of a sequence whose chunk starts at position p.
__device__ __forceinline__ int tile_offset(int p, int m) { return m * kTileCost + block_sum(p, m); }

// Cost of n new tokens that end at position len (all their tiles; the last may be short).
__device__ __forceinline__ int seq_cost(int n, int len) {
  const int tiles = (n + kTokens - 1) / kTokens;
  return tile_offset(len - n, tiles - 1) + kTileCost + (len + kBlock - 1) / kBlock;
}
static_assert(kTokens == 4 && kBlock == 128, "block_sum's closed form");

// Of G nearly equal ranges of [0, total) -- the first total mod G one longer -- the one that
// holds unit t. (total is below 2^30: at most 2^20 + 2^10 tiles of at most 513 + kTileCost
// units.)
__device__ __forceinline__ int range_of(int t, int G, int total) {
  const int q = total / G, r = total - q * G, cut = r * (q + 1);
  return t < cut ? t / (q + 1) : r + (t - cut) / q;
}
static_assert((MFA_MAX_ROWS / kTokens + kMaxBatch) * (int64_t)(MFA_MAX_CONTEXT / kBlock + 1 + kTileCost) <
                  (1ll << 30),
              "costs fit 32 bits");

struct Item {
  int b;          // sequence
  int row0;       // first token's row of q
  int ntok;       // tokens of the tile, 1 .. 4
  int p0;         // position of the first
  int blk0, blk1; // blocks of this item
  int nblk;       // blocks of the tile
  int parts;      // items of the tile, where this is the first of several
  __device__ int kend() const { return p0 + ntok; }          // one past the last key seen
  __device__ int special() const { return (p0 + 1) / kBlock; }  // first special block
  __device__ bool whole() const { return blk0 == 0 && blk1 == nblk; }
};

// The last i of [0, n) with pred(i), which holds from 0 up to some i; by a whole warp, which
// looks at 32 places a step.
template <class F>
__device__ __forceinline__ int last_true(int n, F&& pred) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int step = n > 1024 ? 1024 : n > 32 ? 32 : 1;; step /= 32) {
    const int i = lo + lane * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, i < n && pred(i));
    lo += (31 - __clz(yes)) * step;  // (lane 0 says yes)
    if (step == 1) return lo;
  }
}

// A pair's items, in order.
struct Cursor {
  const Plan* P;
  int batch, g, begin, end, pos, b, tile;

  __device__ void init(const Plan& plan, int batch_, int g_) {
    P = &plan;
    batch = batch_;
    g = g_;
    begin = plan.begin;
    end = plan.end;
    pos = plan.pos;
    b = plan.b;
    tile = plan.tile;
  }

  // The tile `tile` of sequence b.
  __device__ void describe(Item& it) const {
    const int n = P->start[b + 1] - P->start[b];
    it.b = b;
    it.ntok = min(kTokens, n - kTokens * tile);
    it.row0 = P->start[b] + kTokens * tile;
    it.p0 = P->len[b] - n + kTokens * tile;
    it.nblk = (it.kend() + kBlock - 1) / kBlock;
    it.parts = 0;
  }

  __device__ bool next(Item& it) {
    if (P->shared) {
      if (begin >= end) return false;
      describe(it);
      it.blk0 = begin;
      it.blk1 = end;
      it.parts = P->parts;
      begin = end;
      return true;
    }
    while (pos < end) {
      describe(it);
      const int first = pos + kTileCost;  // the tile's first block
      it.blk0 = max(0, begin - first);
      it.blk1 = min(it.nblk, end - first);
      if (it.blk0 == 0 && it.blk1 > 0 && it.blk1 < it.nblk)
        it.parts = range_of(first + it.nblk - 1, P->pairs, P->cost[batch]) - g + 1;
      pos = first + it.nblk;
      ++tile;
      if (kTokens * tile >= P->start[b + 1] - P->start[b]) {
        tile = 0;
        do ++b; while (b < batch && P->cost[b + 1] == P->cost[b]);
      }
      if (it.blk1 > it.blk0) return true;
    }
    return false;
  }
};

// Warp 0, when there are no more tiles than pairs: the least M for which cutting every tile into
// ceil(blocks / M) even parts takes no more parts than pairs, and this pair's part. Taken if
// the longest part is about as short as a range of the other kind, whose pairs have two parts
// each. (Each lane has a run of sequences [b0, b1) with `mine` tiles from t0 on, of lo .. hi
// blocks.)
__device__ __forceinline__ bool share_tiles(Plan& P, int tiles, int t0, int mine, int lo, int hi, int b0,
                                            int b1, int batch, int g, int pairs) {
  const int lane = threadIdx.x & 31;
  lo = __reduce_min_sync(0xffffffffu, mine > 0 ? lo : 1 << 30);
  hi = __reduce_max_sync(0xffffffffu, mine > 0 ? hi : 0);
  // a block takes 1.1 us and merging a part 0.1 to 0.5 us, so parts shorter than this do not pay
  // (one token over 60,000 positions: 29.1 us in parts of 10 blocks, 31.4 of 7, 30.6 of 13)
  const int least = max(1, static_cast<int>(sqrtf(0.2f * hi) + 0.5f));
  const int total = P.cost[batch], most = max(least, (total + pairs - 1) / pairs + kPartCost);
  int tile, part, k, blk = hi;
  if (lo == hi) {  // all alike (decoding, or one tile): no search
    const int split = min(pairs / tiles, hi);
    const int M = max(least, (hi + split - 1) / split);
    if (M > most) return false;
    k = (hi + M - 1) / M;
    tile = g / k;
    part = g - tile * k;
  } else {
    constexpr int kPer = kMaxShared / 32;
    for (int b = b0, t = t0; b < b1; ++b) {
      if (P.cost[b + 1] == P.cost[b]) continue;
      const int n = P.start[b + 1] - P.start[b], p = P.len[b] - n;
      for (int i = 0; kTokens * i < n; ++i, ++t)
        P.tile_blk[t] = (p + min(n, kTokens * (i + 1)) + kBlock - 1) / kBlock;
    }
    __syncwarp();
    int c[kPer], ks[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) c[j] = kPer * lane + j < tiles ? P.tile_blk[kPer * lane + j] : 0;
    int M = max(least, (total - tiles * kTileCost + pairs - 1) / pairs), sum = 0;
    for (;; ++M) {
      if (M > most) return false;
      const float r = 1.f / M;
      sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        // ceil(c / M), exact: both are below 1024, so the quotient is 2^-11 from a whole number
        ks[j] = static_cast<int>((c[j] + M - 1 + 0.5f) * r);
        sum += ks[j];
      }
      if (__reduce_add_sync(0xffffffffu, sum) <= pairs) break;
    }
    int first = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, first, o);
      if (lane >= o) first += y;
    }
    first -= sum;
    int found = -1;
    tile = tiles, part = 0, k = 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (g >= first && g < first + ks[j]) {
        found = kPer * lane + j;
        part = g - first;
        k = ks[j];
        blk = c[j];
      }
      first += ks[j];
    }
    const uint32_t who = __ballot_sync(0xffffffffu, found >= 0);
    if (who != 0) {
      const int l = __ffs(who) - 1;
      tile = __shfl_sync(0xffffffffu, found, l);
      part = __shfl_sync(0xffffffffu, part, l);
      k = __shfl_sync(0xffffffffu, k, l);
      blk = __shfl_sync(0xffffffffu, blk, l);
    }
  }
  if (lane == 0) {
    P.shared = 1;
    P.begin = P.end = 0;
    P.b = P.tile = 0;
    P.parts = k;
  }
  __syncwarp();
  if (tile >= t0 && tile < t0 + mine) {  // the lane whose sequences it is in
    int t = tile - t0, b = b0;
    for (;; ++b) {
      const int n = P.cost[b + 1] != P.cost[b] ? (P.start[b + 1] - P.start[b] + kTokens - 1) / kTokens : 0;
      if (t < n) break;
      t -= n;
    }
    P.b = b;
    P.tile = t;
    P.begin = part * blk / k;
    P.end = (part + 1) * blk / k;
  }
  return true;
}

// What is asked of sequence b: its range of rows, its length (-1: refused, its rows get zeros) and
// its cost; the returned bits say why it is refused. A table or ranges of rows that do not hold
// together (kErrLayout) refuse all.
__device__ __forceinline__ uint32_t read_sequence(const ChunkAttnArgs& a, int b, int& s0, int& s1, int& len,
                                                  int& cost) {
  s0 = a.q_start[b], s1 = a.q_start[b + 1], len = a.seq_lens[b];
  const KvSeq& kv = a.kv[b];
  cost = 0;
  if (!has_chunk_maps(kv) || kv.page_size != a.page_size || s0 < 0 || s1 < s0 || s1 > a.n_rows)
    return kErrLayout;
  if (s1 == s0) return 0;
  const uint32_t bits = len > kv.capacity ? kErrCapacity : len < s1 - s0 ? kErrEmpty : 0u;
  if (bits != 0)
    len = -1;
  else
    cost = seq_cost(s1 - s0, len);
  return bits;
}

// Every thread of the CTA: the sequences, from the lengths on the device, and this pair's share.
// Up to 32 sequences are read by the lanes of warp 0, which goes on with them.
__device__ __forceinline__ void build_plan(Smem& S, const ChunkAttnArgs& a, int g, int pairs, bool report) {
  Plan& P = S.plan;
  const bool few = a.batch <= 32;
  uint32_t bits = 0;
  if (threadIdx.x == kThreads - 1) {
    // (rows of one table, a fixed distance apart)
    P.pages = a.kv[0].pages;
    P.page_stride = a.batch > 1 ? static_cast<int>(a.kv[1].pages - a.kv[0].pages) : 0;
  }
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    int s0, s1, len, cost;
    bits |= read_sequence(a, b, s0, s1, len, cost);
    P.start[b] = s0;
    P.len[b] = len;
    P.cost[b] = cost;
    if (b == a.batch - 1) P.start[a.batch] = s1;
  }
  if (report && bits != 0) atomicOr(a.err, bits);
  const bool none = few ? __any_sync(0xffffffffu, (bits & kErrLayout) != 0)
                        : __syncthreads_or(bits & kErrLayout) != 0;
  if (threadIdx.x < 32) {
    // exclusive prefix of the costs, each lane a run of sequences
    const int lane = threadIdx.x, per = (a.batch + 31) / 32;
    const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
    __syncwarp();
    int sum = 0, mine = 0, lo = 1 << 30, hi = 0;
    for (int b = b0; b < b1; ++b) {
      if (none) P.cost[b] = 0, P.len[b] = -2;
      const int c = P.cost[b];
      sum += c;
      if (c != 0) {
        // (blocks of a sequence's first and last tile: the least and the most of its tiles)
        const int n = P.start[b + 1] - P.start[b], len = P.len[b];
        mine += (n + kTokens - 1) / kTokens;
        lo = min(lo, (len - n + min(n, kTokens) + kBlock - 1) / kBlock);
        hi = max(hi, (len + kBlock - 1) / kBlock);
      }
    }
    int incl = sum, tiles = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, tiles, o);
      if (lane >= o) incl += y, tiles += z;
    }
    int run = incl - sum;
    for (int b = b0; b < b1; ++b) {
      const int c = P.cost[b];
      P.cost[b] = run;
      run += c;
    }
    if (lane == 31) P.cost[a.batch] = incl;
    __syncwarp();
    const int total = P.cost[a.batch], all = __shfl_sync(0xffffffffu, tiles, 31);
    const bool shared = all > 0 && all <= min(pairs, kMaxShared) &&
                        share_tiles(P, all, tiles - mine, mine, lo, hi, b0, b1, a.batch, g, pairs);
    if (!shared) {
      // range g of G nearly equal ones of all units, the first total mod G one longer
      const int G = min(pairs, total);
      int begin = 0, end = 0, b = 0, tile = 0, pos = 0;
      if (g < G) {
        const int q = total / G, r = total - q * G;
        begin = g * q + min(g, r);
        end = begin + q + (g < r);
        // the sequence, then the tile, that hold unit `begin`: the last that starts there or before
        b = last_true(a.batch, [&](int i) { return P.cost[i] <= begin; });
        const int n = P.start[b + 1] - P.start[b], p = P.len[b] - n, c = P.cost[b];
        tile = last_true((n + kTokens - 1) / kTokens, [&](int i) { return c + tile_offset(p, i) <= begin; });
        pos = c + tile_offset(p, tile);
      }
      if (lane == 0) {
        P.begin = begin, P.end = end, P.pos = pos;
        P.b = b, P.tile = tile;
        P.pairs = G;
        P.shared = 0;
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ float* slot_m(float* base, int slot) {
  return base + slot * kChunkPartialFloats;
}
__device__ __forceinline__ float* slot_l(float* base, int slot) {
  return base + slot * kChunkPartialFloats + kChunkRows;
}
__device__ __forceinline__ float* slot_acc(float* base, int slot) {
  return base + slot * kChunkPartialFloats + 2 * kChunkRows;
}

// ---------------------------------------------------------------------------------------
// warp 0: TMA producer
// ---------------------------------------------------------------------------------------

// The page ids of a sequence's 64-row groups, 32 ahead in a register of each lane and the
// next 32 on their way, so that no copy waits for the page table.
struct Groups {
  const int32_t* pages;
  int base, last, shift;  // shift: log2(rows of a page) - 6
  int now, ahead;
  __device__ int fetch(int g0, int lane) const {
    const int g = g0 + lane;
    return g <= last ? pages[g >> shift] : 0;
  }
  __device__ void init(const int32_t* pages_, int g0, int last_, int shift_, int lane) {
    pages = pages_;
    last = last_;
    shift = shift_;
    base = g0;
    now = fetch(base, lane);
    ahead = fetch(base + 32, lane);
  }
  __device__ int page(int g, int lane) {
    if (g >= base + 32) {
      base += 32;
      now = ahead;
      ahead = fetch(base + 32, lane);
    }
    return __shfl_sync(0xffffffffu, now, g - base);
  }
};

// bf16: an item's Q, 64 KB a CTA. Tokens that the tile lacks are rows past the end of q, which read
// as zeros. (One lane.)
__device__ __forceinline__ void load_q(Smem& S, const CUtensorMap* q_map, const ChunkAttnArgs& a,
                                       const Item& it, uint32_t rank) {
  const uint32_t bar = map_to(&S.q_full, 0);
  const uint64_t once = policy_evict_first();
  if (rank == 0) mbar_arrive_expect_tx(&S.q_full, 2 * 4 * kQChunkBytes);
#pragma unroll 1
  for (int i = 0; i < 4 * kCtaTokens; ++i) {
    const int k = i / 4, c = i % 4, tok = kCtaTokens * static_cast<int>(rank) + k;
    const int y = (tok < it.ntok ? it.row0 + tok : a.n_rows) * kHeads;
    pair_load_2d(S.q + c * kQChunkBytes + k * kHeads * 128, q_map, 64 * c, y, bar, once);
  }
}

template <bool kFp8, bool kPaged>
__device__ void run_producer(Smem& S, const CUtensorMap* q_map, const ChunkAttnArgs& a, int g,
                             uint32_t rank) {
  using C = Cfg<kFp8>;
  volatile int* abort = &S.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  const uint64_t once = policy_evict_first(), keep = policy_evict_normal();
  const int page_shift = kPaged ? 31 - __clz(a.page_size) : 0;
  uint32_t chunk = 0, specials = 0;
  // what has been issued: uses of slots, special blocks' V, items' Q (the first by the helper)
  uint32_t issued = 0, v_issued = 0;
  int q_issued = 1;
  int item = 0;
  Cursor cur;
  cur.init(S.plan, a.batch, g);
  Item it, nx;
  bool has = cur.next(it);
  const bool any = has;
  if (!kPaged && has && leader) {
    prefetch_tensormap(&chunk_maps(a.kv[it.b])->k);
    prefetch_tensormap(&chunk_maps(a.kv[it.b])->v);
  }
  while (has) {
    const KvChunkMaps* map = chunk_maps(a.kv[kPaged ? 0 : it.b]);  // (paged: one pool)
    if constexpr (!kFp8) {
      if (item > 0) {  // (the first item's Q is loaded by the helper warp meanwhile)
        mbar_wait(&S.q_empty, (item - 1) & 1, abort);
        if (leader && !*abort) {
          load_q(S, q_map, a, it, rank);
          q_issued = item + 1;
        }
      }
    }
    // one tile of the sequence reads its rows once; several find them in L2
    const uint64_t policy =
        S.plan.start[it.b + 1] - S.plan.start[it.b] <= kTokens ? once : keep;
    const int last_group = (it.kend() - 1) / kChunkBoxRows;
    Groups kg, vg;
    if constexpr (kPaged) {
      kg.init(S.plan.pages + static_cast<long long>(it.b) * S.plan.page_stride, 2 * it.blk0,
              last_group, page_shift - 6, lane);
      vg = kg;
    }
    // 64 rows from group gr on, `boxes` boxes of 128 bytes a row from column x on
    auto load = [&](uint8_t* dst, const CUtensorMap* m, Groups& groups, int gr, int x,
                    int boxes, uint32_t bar) {
      int page = 0, y = gr * kChunkBoxRows;
      if constexpr (kPaged) {
        page = groups.page(gr, lane);
        // groups past the last key: rows outside the page, which read as zeros
        y = gr <= last_group ? y & (a.page_size - 1) : a.page_size;
      }
      if (leader && !*abort) {
        for (int i = 0; i < boxes; ++i) {
          const int xx = x + i * (kFp8 ? 128 : 64);
          if constexpr (kPaged)
            pair_load_3d(dst + i * kBoxBytes, m, xx, y, page, bar, policy);
          else
            pair_load_2d(dst + i * kBoxBytes, m, xx, y, bar, policy);
        }
      }
    };
    // The next slot of the ring, free. Each use of a slot is a phase of the pair's barrier, with
    // an arrival for each CTA: its producer's here, or for a special block's V that of its
    // helper, once it has looked the values over.
    auto take = [&](uint32_t& slot) {
      slot = chunk % kSlots;
      const uint32_t use = chunk / kSlots;
      if (use > 0) mbar_wait(&S.kv_empty[slot], (use - 1) & 1, abort);
      ++chunk;
      return map_to(&S.kv_full[slot], 0);
    };
    auto load_k = [&](int blk) {
      // this CTA's 64 keys, all dimensions
      for (int c = 0; c < C::kKSlots; ++c) {
        uint32_t slot;
        const uint32_t bar = take(slot);
        if (leader && !*abort) {
          remote_arrive_expect_tx(bar, kSlotBytes);
          issued = chunk;
        }
        load(S.ring + slot * kSlotBytes, &map->k, kg, 2 * blk + rank, c * 128, 2, bar);
      }
    };
    auto load_v = [&](int blk) {
      // all keys, this CTA's 128 dimensions. Special blocks land on a barrier of this CTA's own,
      // where its helper warp waits for them.
      const bool special = blk >= it.special();
      const int x = 128 * rank;
      uint64_t* own = &S.v_full[specials % kSlots];
      for (int c = 0; c < C::kVSlots; ++c) {
        uint32_t slot;
        uint32_t bar = take(slot);
        if (leader && !*abort) {
          if (!special)
            remote_arrive_expect_tx(bar, kSlotBytes);
          else if (c == 0)
            mbar_arrive_expect_tx(own, C::kVSlots * kSlotBytes);
          if (special) v_issued = specials + 1;
          issued = chunk;
        }
        if (special) bar = smem_u32(own);
        uint8_t* dst = S.ring + slot * kSlotBytes;
        if constexpr (kFp8) {
          load(dst, &map->v, vg, 2 * blk, x, 1, bar);
          load(dst + kBoxBytes, &map->v, vg, 2 * blk + 1, x, 1, bar);
        } else {
          load(dst, &map->v, vg, 2 * blk + c, x, 2, bar);
        }
      }
      specials += special;
    };
    load_k(it.blk0);
    const bool has_nx = cur.next(nx);
    if (has_nx && leader) {
      // the next item's Q (read once from HBM) on its way to L2, and its tensor maps
      for (int tok = kCtaTokens * rank; tok < min(kCtaTokens * static_cast<int>(rank + 1), nx.ntok); ++tok)
        for (int c = 0; c < 4; ++c) tma_prefetch_2d(q_map, 64 * c, (nx.row0 + tok) * kHeads);
      if constexpr (!kPaged) {
        prefetch_tensormap(&chunk_maps(a.kv[nx.b])->k);
        prefetch_tensormap(&chunk_maps(a.kv[nx.b])->v);
      }
    }
    for (int blk = it.blk0; blk < it.blk1; ++blk) {
      if (blk + 1 < it.blk1) load_k(blk + 1);
      load_v(blk);
    }
    if (it.whole()) {
      for (int c = 0; c < kStageSlots; ++c) {
        uint32_t slot;
        const uint32_t bar = take(slot);
        if (leader && !*abort) remote_arrive(bar);
      }
      if (leader && !*abort) mbar_arrive(&S.stage_free);
    }
    it = nx;
    has = has_nx;
    ++item;
  }
  // Before the CTAs may exit, every copy must have landed (after an abort; else all were used):
  // those that the pair's barriers count are waited for in the first CTA, as far as both have
  // issued them. A wait that gives up has been long enough for all of them; the second CTA
  // cannot see those barriers and waits a while.
  if (*abort && leader && any) {
    bool wait = true;
    for (uint32_t c = v_issued > kSlots ? v_issued - kSlots : 0; c < v_issued && wait; ++c)
      wait = mbar_wait_drain(&S.v_full[c % kSlots], (c / kSlots) & 1);
    if (rank == 0) {
      for (uint32_t c = issued > kSlots ? issued - kSlots : 0; c < issued && wait; ++c)
        wait = mbar_wait_drain(&S.kv_full[c % kSlots], (c / kSlots) & 1);
      if (!kFp8 && wait) mbar_wait_drain(&S.q_full, (q_issued - 1) & 1);
    } else {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < kLandNs) {
      }
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------------------
// warp 1 of the first CTA: the products
// ---------------------------------------------------------------------------------------
template <bool kFp8>
__device__ void run_mma(Smem& S, const ChunkAttnArgs& a, int g, uint32_t tmem) {
  using C = Cfg<kFp8>;
  volatile int* abort = &S.abort_flag;
  const bool leader = elect_one();
  uint32_t chunk = 0, gt = 0;
  int item = 0;
  const uint32_t q_lo = desc_lo(smem_u32(S.q), 16), ring = smem_u32(S.ring);

  auto issue_s = [&](uint32_t t) {
    const uint32_t d = tmem + kTmemS + kBlock * (t & 1);
#pragma unroll
    for (int c = 0; c < C::kKSlots; ++c, ++chunk) {
      const uint32_t slot = chunk % kSlots;
      mbar_wait(&S.kv_full[slot], (chunk / kSlots) & 1, abort);
      tc_fence_after();
      if (leader && !*abort) {
        const uint32_t k_lo = desc_lo(ring + slot * kSlotBytes, 16);
        if constexpr (kFp8) {
          // high parts, then low parts of Q, over the same keys
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int part = i >> 3, box = (i >> 2) & 1, kk = i & 3;
            pair_mma_ss<true>(d, q_lo + ((2 * part + box) * kQChunkBytes + 32 * kk) / 16,
                              k_lo + (box * kBoxBytes + 32 * kk) / 16, C::kIdescS, i != 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int box = i >> 2, kk = i & 3;
            pair_mma_ss<false>(d, q_lo + ((2 * c + box) * kQChunkBytes + 32 * kk) / 16,
                               k_lo + (box * kBoxBytes + 32 * kk) / 16, C::kIdescS,
                               (c | i) != 0);
          }
        }
        pair_commit(&S.kv_empty[slot]);
      }
    }
    if (leader && !*abort) pair_commit(&S.s_full[t & 1]);
  };

  auto issue_pv = [&](uint32_t t, bool first) {
    // V first: it has landed long before P, and a wait costs ~150 cycles even so
    uint32_t v_lo[C::kVSlots], slot[C::kVSlots];
#pragma unroll
    for (int c = 0; c < C::kVSlots; ++c, ++chunk) {
      slot[c] = chunk % kSlots;
      mbar_wait(&S.kv_full[slot[c]], (chunk / kSlots) & 1, abort);
      v_lo[c] = desc_lo(ring + slot[c] * kSlotBytes, kBoxBytes);
    }
    if (first && item > 0) mbar_wait(&S.o_free, (item - 1) & 1, abort);
    mbar_wait(&S.p_full[t & 1], (t >> 1) & 1, abort);
    tc_fence_after();
    const uint32_t d = tmem + kTmemO, p = tmem + kTmemS + kBlock * (t & 1);
    if (leader && !*abort) {
#pragma unroll
      for (int c = 0; c < C::kVSlots; ++c) {
        if constexpr (kFp8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int part = i >> 2, kt = i & 3;  // 32 keys each
            pair_mma_ts<true>(d, p + 32 * part + 8 * kt, v_lo[c] + 4096 * kt / 16,
                              part == 0 ? C::kIdescPV : C::kIdescPV | kIdescE5m2A, !(first && i == 0));
          }
        } else {
#pragma unroll
          for (int kt = 0; kt < 4; ++kt)  // 16 keys each
            pair_mma_ts<false>(d, p + 8 * (4 * c + kt), v_lo[c] + 2048 * kt / 16, C::kIdescPV,
                               !(first && c == 0 && kt == 0));
        }
        pair_commit(&S.kv_empty[slot[c]]);
      }
      pair_commit(&S.pv_done[t & 1]);
    }
  };

  Cursor cur;
  cur.init(S.plan, a.batch, g);
  Item it;
  while (cur.next(it)) {
    const int n = it.blk1 - it.blk0;
    mbar_wait(&S.q_full, item & 1, abort);
    tc_fence_after();
    issue_s(gt);
    for (int t = 0; t < n; ++t) {
      if (t + 1 < n) issue_s(gt + t + 1);
      if (t + 1 == n && !kFp8 && leader && !*abort) pair_commit(&S.q_empty);
      if (t + 1 == n && it.whole()) {
        // both producers have counted the uses of the slots behind V that take the results, so
        // that a CTA which is done with them early cannot count its next use into this one
        for (int c = 0; c < kStageSlots; ++c) {
          const uint32_t sc = chunk + C::kVSlots + c;
          mbar_wait(&S.kv_full[sc % kSlots], (sc / kSlots) & 1, abort);
        }
      }
      issue_pv(gt + t, t == 0);
    }
    if (it.whole()) chunk += kStageSlots;
    gt += n;
    ++item;
  }
  // every product must be done before the tensor memory is released
  if (leader) pair_commit(&S.mma_done);
  mbar_wait_drain(&S.mma_done, 0);
}

// ---------------------------------------------------------------------------------------
// warps 2..9: softmax, rescale, epilogue
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of three, NaN if one is: a row with a NaN score has a NaN maximum, and every
// weight of it is NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two floats at a time.
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// f16x2 as e4m3 high and low parts: hi = e4m3(v), lo = e4m3(v - hi) (exact difference)
__device__ __forceinline__ void split_e4m3x2(uint32_t v, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t back, rest;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(v));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(v), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(rest));
  hi = h;
  lo = l;
}
// Weights (f16x2, 0 <= v < 2^12) as sums of an e4m3 and an e5m2 value: from 256 up the value's first
// three bits as e5m2 and the rest (at most 256) as e4m3, below e4m3 and the rest as e5m2. Either
// way the sum is within 2^-8 of the value's power of two, down to 2^-6; below, the rest is at most
// 2^-10 and off by at most 1/8 of itself or 2^-17. (An e4m3 rest has no step below 2^-9, and a row
// of one large weight and thousands of small ones, which an e4m3 pair rounded to nothing, lost all
// of the small ones: 80 % of the result at 65,536 keys, 0.1 % so.)
__device__ __forceinline__ void split_weights(uint32_t v, uint32_t& e4, uint32_t& e5) {
  uint32_t large, rest, back;
  uint16_t a, b;
  asm("set.ge.u32.f16x2 %0, %1, %2;" : "=r"(large) : "r"(v), "r"(0x5C005C00u));
  // (e5m2 is f16's first byte)
  const uint32_t first = (v + 0x00800080u) & 0xFF00FF00u & large;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(v), "r"(first));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(rest));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(v), "r"(back));
  // (what e4m3 left of a large one does not reach its first three bits)
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(rest));
  e4 = a;
  e5 = b;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight consecutive values of a cache row (element offset `at`), as float32.
template <bool kFp8>
__device__ __forceinline__ void load8(const void* base, long long at, float (&f)[8]) {
  if constexpr (kFp8) {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at);
    const uint16_t h[4] = {static_cast<uint16_t>(v.x), static_cast<uint16_t>(v.x >> 16),
                           static_cast<uint16_t>(v.y), static_cast<uint16_t>(v.y >> 16)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(h[i]));
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

// FP8: Q of an item, split into e4m3 high and low parts scaled by 2^-e with the row's largest
// magnitude in [128, 256); e goes to S.q_exp of the item's parity. (bf16 times a power of two is exact in f16 down
// to 2^-24 of 256; smaller elements round there.) Each softmax warp takes 16 of the CTA's rows,
// 16 lanes a row and 16 dimensions a lane, so that its loads cover whole lines (one row a
// thread took 12000 cycles). The Q buffer must be free: every S of the previous item has
// completed.
__device__ __noinline__ void split_q(Smem& S, const ChunkAttnArgs& a, const Item& it, int parity,
                                     int rank, int swarp, int lane) {
  constexpr int kRowsWarp = kRows / kSoftmaxWarps;
  const int part = lane % 16, r0 = swarp * kRowsWarp + lane / 16;
  const long long row0 = (static_cast<long long>(it.row0) + kCtaTokens * rank) * kHeads;
  const int rows = (it.ntok - kCtaTokens * rank) * kHeads;  // (those of missing tokens are zero)
  uint4 v[kRowsWarp / 2][2];
#pragma unroll
  for (int i = 0; i < kRowsWarp / 2; ++i) {
    const int r = r0 + 2 * i;
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (row0 + r) * kHeadDim + 16 * part);
    v[i][0] = r < rows ? src[0] : make_uint4(0, 0, 0, 0);
    v[i][1] = r < rows ? src[1] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kRowsWarp / 2; ++i) {
    const int r = r0 + 2 * i;
    const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w,
                           v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 128 <= mx 2^-e < 256; e >= -100 keeps 2^-e finite; a row of zeros takes 0. (A subnormal mx
    // counts as 2^-127.) A row with an infinity becomes NaN: its scores are infinities or NaN, which
    // e4m3 has no infinity to form, and their softmax is NaN whatever the keys.
    const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
    const int e = mx > 0.f && ex < 255 ? max(ex - 127 - 7, -100) : 0;
    const float sc = ex < 255 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : NAN;
    if (part == 0) S.q_exp[parity][r] = e;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h0, l0, h1, l1;
      split_e4m3x2(pack_f16x2(bf16_lo(w[2 * k]) * sc, bf16_hi(w[2 * k]) * sc), h0, l0);
      split_e4m3x2(pack_f16x2(bf16_lo(w[2 * k + 1]) * sc, bf16_hi(w[2 * k + 1]) * sc), h1, l1);
      hi[k] = h0 | (h1 << 16);
      lo[k] = l0 | (l1 << 16);
    }
    uint8_t* dst = S.q + (part / 8) * kQChunkBytes + r * 128 + (((part % 8) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + 2 * kQChunkBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

__device__ __forceinline__ uint32_t bad_flag(int item, uint32_t rows) {
  return (static_cast<uint32_t>(item + 1) << 3) | rows;
}
static_assert(kTokens - 1 <= 3, "a bit for each late row");

// A special block's V half in this CTA's ring (its first slot's use `chunk`), by one warp: rows
// of keys that no token of the tile sees are zeroed; rows that only its later tokens see (key
// p0 + 1 + i, i < ntok - 1) are zeroed too if they hold an infinity or NaN, and their bits i
// returned.
template <bool kFp8>
__device__ __forceinline__ uint32_t clean_v(Smem& S, const Item& it, int blk, uint32_t chunk,
                                            int lane) {
  constexpr int kBoxes = kFp8 ? 1 : 2;  // boxes of 128 bytes across this CTA's 128 dimensions
  uint8_t* slot0 = S.ring + (chunk % kSlots) * kSlotBytes;
  uint8_t* slot1 = kFp8 ? slot0 + kBoxBytes : S.ring + ((chunk + 1) % kSlots) * kSlotBytes;
  // late rows: lane = 16-byte piece of the row
  uint32_t bad = 0;
  uint4 v[kTokens - 1];
  uint4* at[kTokens - 1];
#pragma unroll
  for (int i = 0; i < kTokens - 1; ++i) {
    const int r = it.p0 + 1 + i - blk * kBlock;
    const bool here = i + 1 < it.ntok && r >= 0 && r < kBlock && lane < 8 * kBoxes;
    at[i] = here ? reinterpret_cast<uint4*>((r < kChunkBoxRows ? slot0 : slot1) + (lane / 8) * kBoxBytes +
                                            (r % kChunkBoxRows) * 128 + (lane % 8) * 16)
                 : nullptr;
    v[i] = here ? *at[i] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kTokens - 1; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    bool odd = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (kFp8)  // a byte of 0x7F or 0xFF
        odd |= (((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
      else
        odd |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
    }
    if (__any_sync(0xffffffffu, odd)) {
      bad |= 1u << i;
      if (at[i] != nullptr) *at[i] = make_uint4(0, 0, 0, 0);
    }
  }
  // the rows from kend on are the rest of each box
  const int from = max(0, it.kend() - blk * kBlock);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int f = max(0, from - h * kChunkBoxRows);
    for (int i = f * 8 + lane; i < kChunkBoxRows * 8; i += 32) {
      uint4* p = reinterpret_cast<uint4*>(h == 0 ? slot0 : slot1) + i;
      p[0] = make_uint4(0, 0, 0, 0);
      if constexpr (kBoxes == 2) p[kBoxBytes / 16] = make_uint4(0, 0, 0, 0);
    }
  }
  return bad;
}

// The weights 2^(s - base) of the held-out keys p0 + 1 + i for this row, 0 where it does not
// see them.
template <bool kFp8>
__device__ __noinline__ void late_weights(const ChunkAttnArgs& a, const Item& it, uint32_t bad,
                                          int tok, int head, float base, float (&w)[3]) {
  const float mul = a.scale * kLog2e * (kFp8 ? a.k_scale : 1.f);
  for (int i = 0; i < 3; ++i) {
    w[i] = 0.f;
    const long long at = kv_row_index(a.kv[it.b], it.p0 + 1 + i);
    if (!((bad >> i) & 1) || tok < i + 1 || tok >= it.ntok || at < 0) continue;
    float s = 0.f;
    for (int d = 0; d < kHeadDim; d += 8) {
      float q[8], k[8];
      load8<false>(a.q, (static_cast<long long>(it.row0 + tok) * kHeads + head) * kHeadDim + d, q);
      load8<kFp8>(a.kv[it.b].k, at * kHeadDim + d, k);
      for (int j = 0; j < 8; ++j) s = fmaf(q[j], k[j], s);
    }
    w[i] = ex2(fmaf(s, mul, -base));
  }
}

// Rows that were held out of the products, added to this thread's half of its row of O in
// tensor memory.
template <bool kFp8>
__device__ __noinline__ void add_late(const ChunkAttnArgs& a, const Item& it, uint32_t bad, int tok,
                                      int head, int half, float base, uint32_t o_addr) {
  float w[3];
  late_weights<kFp8>(a, it, bad, tok, head, base, w);
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t o[16];
    tmem_ld_32x32b_x16(o_addr + 16 * c, o);
    tmem_wait_ld();
    for (int i = 0; i < 3; ++i) {
      if (!((bad >> i) & 1) || tok < i + 1 || tok >= it.ntok) continue;
      const long long at = kv_row_index(a.kv[it.b], it.p0 + 1 + i);
      if (at < 0) continue;
#pragma unroll
      for (int d = 0; d < 16; d += 8) {
        float v[8];
        load8<kFp8>(a.kv[it.b].v, at * kHeadDim + 128 * half + 16 * c + d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          o[d + j] = __float_as_uint(fmaf(w[i], v[j], __uint_as_float(o[d + j])));
      }
    }
    __syncwarp();
    tmem_st_32x32b_x16(o_addr + 16 * c, o);
  }
  tmem_wait_st();
}

template <bool kFp8>
__device__ void run_softmax(Smem& S, const ChunkAttnArgs& a, int g, uint32_t rank,
                            uint32_t tmem) {
  using C = Cfg<kFp8>;
  volatile int* abort = &S.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int swarp = warp - 2, st = threadIdx.x - 64;
  const int quad = warp & 3, half = swarp >> 2;  // lanes of tensor memory; half of the keys
  const int row = quad * 32 + lane;
  const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t bar = 1 + quad;  // named barrier of the two warps that share these rows
  const int tok = kCtaTokens * rank + row / kHeads;  // token of the tile
  const int head = row % kHeads;
  const float mul0 = a.scale * kLog2e * (kFp8 ? a.k_scale : 1.f);
  const float v_mul = kFp8 ? a.v_scale : 1.f;
  const uint32_t p_bar[2] = {map_to(&S.p_full[0], 0), map_to(&S.p_full[1], 0)};
  const uint32_t o_bar = map_to(&S.o_free, 0);
  const uint32_t q_bar = map_to(&S.q_full, 0);
  uint32_t gt = 0, chunk = 0;
  int item = 0, tiles = 0;

  // rows of refused sequences
  for (int b = g; b < a.batch; b += gridDim.x / 2) {
    if (S.plan.len[b] != -1) continue;
    const size_t r0 = static_cast<size_t>(S.plan.start[b]) * (kQWidth / 8);
    const size_t r1 = static_cast<size_t>(S.plan.start[b + 1]) * (kQWidth / 8);
    uint4* out = reinterpret_cast<uint4*>(a.out);
    for (size_t i = r0 + rank * 256 + st; i < r1; i += 512) out[i] = make_uint4(0, 0, 0, 0);
  }
  int2 info = make_int2(0, 0);  // for the combine kernel: rows of the tile and its parts

  Cursor cur;
  cur.init(S.plan, a.batch, g);
  Item it, nx;
  bool has = cur.next(it);
  float mul = mul0;
  // FP8: the next item's Q into the buffer, once every S of this one is done, and its rows'
  // factor of the scores
  auto next_q = [&](const Item& x, int parity) {
    split_q(S, a, x, parity, rank, swarp, lane);
    fence_proxy_async_smem();
    named_bar_sync(7, 32 * kSoftmaxWarps);  // q_exp (and every warp's part is in place)
    if (st == 0) remote_arrive(q_bar);
    // (not 0, by which a hidden key's -infinity would become NaN: scores this small are all alike)
    return fmaxf(mul0 * __uint_as_float(static_cast<uint32_t>(127 + S.q_exp[parity][row]) << 23), FLT_MIN);
  };
  if constexpr (kFp8) {
    if (has) mul = next_q(it, 0);
  }
  while (has) {
    const int n = it.blk1 - it.blk0;
    float next_mul = mul0;
    // keys this row's token sees: positions below lim
    const int lim = it.p0 + min(tok, it.ntok - 1) + 1;
    // (the same for the whole warp)
    const bool real = tok < it.ntok;
    float m = -INFINITY, base = 0.f, l = 0.f;  // m: raw; base = m mul (0 while m is -inf)
    const float thr_step = C::kRescale / mul;
    float thr = -INFINITY;

    for (int t = 0; t < n; ++t) {
      const uint32_t j = (gt + t) & 1;
      const int blk = it.blk0 + t;
      const bool special = blk >= it.special();
      const uint32_t sa = tmem + lane_addr + kTmemS + kBlock * j;
      mbar_wait(&S.s_full[j], ((gt + t) >> 1) & 1, abort);
      tc_fence_after();
      if (!real) {
        // rows of tokens that the tile lacks: weights of zero. (Their Q is zero too: products of
        // zeros cost a fraction of the power, and decoding steps, three of four rows of which
        // are such, ran at 1.6 GHz under the power limit without this.)
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
        tmem_st_32x32b_x32(sa + 32 * half, z);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) remote_arrive(p_bar[j]);
        continue;
      }
      float s[64];
      {
        uint32_t r0[32], r1[32];
        tmem_ld_32x32b_x32(sa + 64 * half, r0);
        tmem_ld_32x32b_x32(sa + 64 * half + 32, r1);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r0[i]), s[32 + i] = __uint_as_float(r1[i]);
      }
      if (special) {
        // of these 64 keys those below lim are seen (the same number in the whole warp); eight
        // at a time, so that only the eight that lim falls into are compared one by one
        const int left = lim - (blk * kBlock + 64 * half);
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          if (left < e + 8) {
#pragma unroll
            for (int i = e; i < e + 8; ++i) s[i] = i < left ? s[i] : -INFINITY;
          }
        }
      }
      float mx = max3(s[0], s[1], s[2]);
      {
        float m1 = max3(s[3], s[4], s[5]);
#pragma unroll
        for (int i = 6; i < 62; i += 4) {
          mx = max3(mx, s[i], s[i + 1]);
          m1 = max3(m1, s[i + 2], s[i + 3]);
        }
        mx = max3(max3(mx, m1, s[62]), s[63], s[63]);
      }
      // (also: both warps have read their scores, which P will overwrite)
      // (a NaN maximum counts as a larger one, once)
      if (named_bar_or(bar, 64, !(mx <= thr) && m == m)) {
        S.xch[half][row] = mx;
        named_bar_sync(bar, 64);
        const float mn = max3(m, mx, S.xch[half ^ 1][row]);
        const float alpha = m == mn ? 1.f : ex2((m - mn) * mul);
        m = mn;
        // an infinite maximum makes the row's weights NaN (inf - inf), as the softmax's are
        base = mn == -INFINITY ? 0.f : mn * mul + (mn - mn);
        thr = mn + thr_step;
        l *= alpha;
        if (t > 0) {
          // O holds PV(t - 1) before it is rescaled
          mbar_wait(&S.pv_done[(gt + t - 1) & 1], ((gt + t - 1) >> 1) & 1, abort);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            const uint32_t oa = tmem + lane_addr + kTmemO + 128 * half + 32 * c;
            tmem_ld_32x32b_x32(oa, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(oa, o);
          }
        }
      }
      // weights 2^(s - base); a hidden key's score is -inf and its weight 0. They are rounded to what
      // the tensor cores read: bf16, off by at most 2^-8 of themselves, up or down (FP8: f16, 2^-11,
      // then split_weights); their sum is of the float32 values. All exponentials go
      // through the special-function unit, which they keep busy for half of a block's products:
      // a quarter of them by polynomial made the softmax shorter and long calls 2 to 4 %
      // slower, since those run at the power limit and the polynomial takes more of it.
      const uint64_t mul2 = pair_f32(mul, mul), off2 = pair_f32(C::kPExp - base, C::kPExp - base);
      uint32_t pw[32];
      uint64_t l2 = pair_f32(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint64_t x = fma2(pair_f32(s[2 * i], s[2 * i + 1]), mul2, off2);
        float p0, p1;
        unpair_f32(x, p0, p1);
        p0 = ex2(p0);
        p1 = ex2(p1);
        l2 = add2(l2, pair_f32(p0, p1));
        pw[i] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
      }
      {
        float l0, l1;
        unpair_f32(l2, l0, l1);
        l += l0 + l1;
      }
      if constexpr (kFp8) {
        uint32_t hl[32];  // 16 words of e4m3 parts, 16 of e5m2 parts
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t a0, b0, a1, b1;
          split_weights(pw[2 * i], a0, b0);
          split_weights(pw[2 * i + 1], a1, b1);
          hl[i] = a0 | (a1 << 16);
          hl[16 + i] = b0 | (b1 << 16);
        }
        uint32_t w0[16], w1[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w0[i] = hl[i], w1[i] = hl[16 + i];
        tmem_st_32x32b_x16(sa + 16 * half, w0);
        tmem_st_32x32b_x16(sa + 32 + 16 * half, w1);
      } else {
        tmem_st_32x32b_x32(sa + 32 * half, pw);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(p_bar[j]);
    }
    gt += n;
    chunk += n * (C::kKSlots + C::kVSlots);

    // ---- epilogue ----
    // what the next item needs goes first, while the last product runs
    if (real) S.sum[half][row] = l;
    const bool has_nx = cur.next(nx);
    if (real) {
      named_bar_sync(bar, 64);
      l += S.sum[half ^ 1][row];
    }
    const bool whole = it.whole();
    if constexpr (kFp8) {
      if (has_nx) next_mul = next_q(nx, (item + 1) & 1);
    }
    if (whole) {
      mbar_wait(&S.stage_free, tiles & 1, abort);
      ++tiles;
    }
    mbar_wait(&S.pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, abort);
    tc_fence_after();
    const bool ok = *abort == 0;
    const uint32_t o_addr = tmem + lane_addr + kTmemO + 128 * half;
    // (volatile: written by the other CTA too; the same in the whole warp, even where that happens
    // meanwhile, after an abort)
    const uint32_t flag = *static_cast<volatile uint32_t*>(&S.bad[item & 1][half]);
    uint32_t bad = bad_flag(item, 0) ^ __shfl_sync(0xffffffffu, flag, 0);
    if (bad >= 8) bad = 0;  // (an older item's)
    if (bad != 0) add_late<kFp8>(a, it, bad, tok, head, half, base - C::kPExp, o_addr);
    const int slot = 2 * g + (it.blk0 == 0 ? 1 : 0);
    if (whole) {
      // rounded into the ring, as boxes of [128 rows x 64 dimensions] with 128-byte swizzle,
      // for the helper warp to store (stores of each lane's own row touch 32 lines each: the
      // epilogue took 12000 cycles that way, 3300 after a transposition by shuffles, 1000 so)
      const float inv = v_mul / l;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[2][32];
        tmem_ld_32x32b_x32(o_addr + 64 * c, r[0]);
        tmem_ld_32x32b_x32(o_addr + 64 * c + 32, r[1]);
        tmem_wait_ld();
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(o_bar);
        }
        uint8_t* dst = S.ring + ((chunk + 2 * half + c) % kSlots) * kSlotBytes + row * 128;
#pragma unroll
        for (int piece = 0; piece < 8; ++piece) {
          const uint32_t* v = r[piece / 4] + 8 * (piece % 4);
          *reinterpret_cast<uint4*>(dst + ((piece ^ (row & 7)) << 4)) = make_uint4(
              pack_bf16x2(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv),
              pack_bf16x2(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv),
              pack_bf16x2(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv),
              pack_bf16x2(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv));
        }
      }
      chunk += kStageSlots;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.staged);
    } else {
      // partials: [4 dimensions][row] so that a store is 512 bytes of consecutive rows
      float* acc = slot_acc(a.partials, slot) + (32 * half * kChunkRows + rank * kRows + row) * 4;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(o_addr + 32 * c, r);
        tmem_wait_ld();
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(o_bar);
        }
        if (ok && real) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(acc + (8 * c + i) * kChunkRows * 4) =
                make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
    }
    if (!whole) {
      if (ok && real && half == 0) {
        // (a part none of whose keys the row sees: m stays -inf, its weight will be 0)
        slot_m(a.partials, slot)[rank * kRows + row] = m == -INFINITY ? -INFINITY : base;
        slot_l(a.partials, slot)[rank * kRows + row] = l;
      }
      if (it.blk0 == 0) info = make_int2(it.row0, it.parts * 8 + it.ntok);
    }
    it = nx;
    has = has_nx;
    mul = next_mul;
    ++item;
  }
  if (rank == 0 && st == 0) a.info[g] = info;
}

// ---------------------------------------------------------------------------------------
// the helper warp: looks special blocks' V over, stores finished tiles
// ---------------------------------------------------------------------------------------
template <bool kFp8>
__device__ void run_helper(Smem& S, const CUtensorMap* q_map, const CUtensorMap* out_map,
                           const ChunkAttnArgs& a, int g, uint32_t rank) {
  using C = Cfg<kFp8>;
  volatile int* abort = &S.abort_flag;
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  uint32_t chunk = 0, specials = 0;
  int item = 0, tiles = 0;
  Cursor cur;
  cur.init(S.plan, a.batch, g);
  Item it;
  while (cur.next(it)) {
    const int n = it.blk1 - it.blk0;
    if (!kFp8 && item == 0 && leader) load_q(S, q_map, a, it, rank);
    uint32_t bad = 0;
    for (int blk = max(it.blk0, it.special()); blk < it.blk1; ++blk) {
      const int t = blk - it.blk0;
      // the use of V's first slot: K of blocks 0 .. t + 1 and V of 0 .. t - 1 come before it
      const uint32_t vc = chunk + C::kKSlots + t * (C::kKSlots + C::kVSlots) +
                          (t + 1 < n ? C::kKSlots : 0);
      mbar_wait(&S.v_full[specials % kSlots], (specials / kSlots) & 1, abort);
      ++specials;
      if (__shfl_sync(0xffffffffu, *abort, 0) != 0) break;
      bad |= clean_v<kFp8>(S, it, blk, vc, lane);
      if (bad != 0 && lane < 2)  // for the epilogues of both CTAs
        remote_store(map_to(&S.bad[item & 1][rank], lane), bad_flag(item, bad));
      fence_proxy_async_smem();
      __syncwarp();
      if (leader) {
#pragma unroll
        for (int c = 0; c < C::kVSlots; ++c) {
          const uint32_t bar = map_to(&S.kv_full[(vc + c) % kSlots], 0);
          if (bad != 0)
            remote_arrive_release(bar);
          else
            remote_arrive(bar);
        }
      }
      __syncwarp();
    }
    chunk += n * (C::kKSlots + C::kVSlots);
    if (it.whole()) {
      mbar_wait(&S.staged, tiles & 1, abort);
      if (leader && !*abort) {
        const int rows = min(kCtaTokens, it.ntok - kCtaTokens * static_cast<int>(rank));
        for (int c = 0; c < kStageSlots; ++c) {
          for (int k = 0; k < rows; ++k)
            tma_store_2d(out_map, 64 * c, (it.row0 + kCtaTokens * rank + k) * kHeads,
                         S.ring + ((chunk + c) % kSlots) * kSlotBytes + k * kHeads * 128);
          tma_store_commit();
        }
        // each slot is free once its store has read it
        tma_store_wait_read<3>();
        mbar_arrive(&S.kv_empty[chunk % kSlots]);
        tma_store_wait_read<2>();
        mbar_arrive(&S.kv_empty[(chunk + 1) % kSlots]);
        tma_store_wait_read<1>();
        mbar_arrive(&S.kv_empty[(chunk + 2) % kSlots]);
        tma_store_wait_read<0>();
        mbar_arrive(&S.kv_empty[(chunk + 3) % kSlots]);
        static_assert(kStageSlots == 4, "the waits above");
      }
      __syncwarp();
      chunk += kStageSlots;
      ++tiles;
    }
    ++item;
  }
  if (leader) tma_store_wait_done();
  __syncwarp();
}

template <bool kFp8, bool kPaged>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap out_map,
                      const __grid_constant__ ChunkAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                     ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cta_rank();
  const int g = blockIdx.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&S.kv_full[i], 2);
      mbar_init(&S.kv_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
    }
    mbar_init(&S.q_full, kFp8 ? 2 : 1);
    mbar_init(&S.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.p_full[i], 2 * kSoftmaxWarps);
    }
    mbar_init(&S.o_free, 2 * kSoftmaxWarps);
    mbar_init(&S.stage_free, 1);
    mbar_init(&S.staged, kSoftmaxWarps);
    mbar_init(&S.mma_done, 1);
    S.bad[0][0] = S.bad[0][1] = S.bad[1][0] = S.bad[1][1] = 0;
    S.abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&out_map);
    if (kPaged) {  // (the table is the host's; no kernel writes it)
      const KvChunkMaps* maps = chunk_maps(a.kv[0]);
      prefetch_tensormap(&maps->k);
      prefetch_tensormap(&maps->v);
    }
  }
  if (warp == 1) pair_tmem_alloc(&S.tmem_base);
  tc_fence_before();
  __syncwarp();
  cluster_arrive();  // this CTA's barriers are set up
  pdl_wait();
  build_plan(S, a, g, static_cast<int>(gridDim.x) / 2, blockIdx.x == 0);
  cluster_wait();  // and the other's
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp == 0) {
    run_producer<kFp8, kPaged>(S, &q_map, a, g, rank);
  } else if (warp == 1) {
    if (rank == 0) run_mma<kFp8>(S, a, g, tmem);
  } else if (warp == kHelperWarp) {
    run_helper<kFp8>(S, &q_map, &out_map, a, g, rank);
  } else {
    run_softmax<kFp8>(S, a, g, rank, tmem);
  }

  tc_fence_before();
  __syncthreads();
  // (not earlier: see the merge)
  pdl_launch_dependents();
  if (threadIdx.x == 0 && S.abort_flag) atomicOr(a.err, kErrTimeout);
  // the last commit of the products reaches both CTAs: neither may be gone by then
  if (warp == 1 && rank != 0) mbar_wait_drain(&S.mma_done, 0);
  __syncwarp();
  cluster_arrive();
  cluster_wait();  // the other CTA's products and arrivals are done with this one's memory
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    pair_tmem_dealloc(tmem);
  }
}

// ---------------------------------------------------------------------------------------
// merge of the tiles that several pairs share, in a fixed order. A block takes 32 rows (half a
// token) of one tile: lane = row, four warps of kDims dimensions each. Bound by the latency of its
// loads and by how evenly its blocks lie: their launch is triggered at the end of a pair's work, so
// that they do not gather on the SMs that have none (12 sequences of one token over 4000 positions:
// 24.4 us when triggered at the start, 20.7 so).
// ---------------------------------------------------------------------------------------
constexpr int kCombineRows = 32, kCombineWarps = 4;
static_assert(kHeads == 2 * kCombineRows, "a token is two blocks of rows");
// By a whole warp: the `token`-th token of all split tiles, as its tile's info, the pair in which
// that begins, and the token of the tile; zeros if there are fewer. (Each lane looks at kPer pairs
// in a row.)
__device__ __forceinline__ int4 find_token(const ChunkAttnArgs& a, int token) {
  constexpr int kPer = kMaxShared / 32;
  const int lane = threadIdx.x & 31;
  int2 info[kPer];
  int mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int g = kPer * lane + j;
    info[j] = g < a.pairs ? __ldcg(&a.info[g]) : make_int2(0, 0);
    mine += info[j].y & 7;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  int4 r = make_int4(0, 0, 0, 0);
  int left = token - (upto - mine);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int n = info[j].y & 7;
    if (left >= 0 && left < n) r = make_int4(info[j].x, info[j].y, kPer * lane + j, left);
    left -= n;
  }
  const uint32_t who = __ballot_sync(0xffffffffu, r.y != 0);
  const int from = who != 0 ? __ffs(who) - 1 : 0;
  r.x = __shfl_sync(0xffffffffu, r.x, from);
  r.y = __shfl_sync(0xffffffffu, r.y, from);
  r.z = __shfl_sync(0xffffffffu, r.z, from);
  r.w = __shfl_sync(0xffffffffu, r.w, from);
  return r;
}

// Up to this many tiles, which may have a dozen parts and more each, 8 dimensions a thread and 16
// parts' loads at a time; above it 16 dimensions and four parts. Measured, the first and the second:
// one token over 60,000 positions 29.1 and 42.6 us, 12 over 30,000 29.3 and 36.3; 12 sequences of
// one token over 200 11.9 and 11.3, 64 over 1500 28.0 and 26.8.
constexpr int kFewTiles = 6;
// Up to this many tokens, blocks for the tokens that there are, which look for their tile; above it
// blocks for every pair and row, most of which end at once. The first and the second: 24 tokens over
// 3000 positions 18.0 and 24.2 us, 64 sequences of one over 200 14.3 and 15.4; 25 of 4 over 500 17.8
// and 16.5, 100 tokens over 900 19.0 and 18.1 (and a prompt of 1111 tokens 63 and 56: every block
// reads the pairs' few lines).
constexpr int kFewTokens = 64;

template <int kDims, int kAtOnce, bool kSearch>
__global__ void __launch_bounds__(32 * kCombineWarps) chunk_combine_kernel(ChunkAttnArgs a) {
  constexpr int kBlockDims = kDims * kCombineWarps;
  __shared__ __align__(16) uint4 tile[kCombineRows][kBlockDims / 8 + 1];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int dim0 = blockIdx.y * kBlockDims;
  // the tile, the pair g in which it begins, and its row
  int2 info;
  int g, row0;
  if constexpr (kSearch) {
    // Block x takes half x % 2 of the (x / 2)-th token of all split tiles.
    __shared__ int4 found;
    if (warp == 0) found = find_token(a, blockIdx.x / 2);
    __syncthreads();
    info = make_int2(found.x, found.y);
    g = found.z;
    row0 = found.w * kHeads + (blockIdx.x & 1) * kCombineRows;
    if (info.y == 0) return;
  } else {
    g = blockIdx.x;
    info = __ldcg(&a.info[g]);
    row0 = blockIdx.z * kCombineRows;
    if (row0 >= (info.y & 7) * kHeads) return;
  }
  const int parts = info.y >> 3, row = row0 + lane;
  // part i of the tile lies in the first slot of pair g + i, part 0 in g's second
  auto slot = [&](int i) { return i == 0 ? 2 * g + 1 : 2 * (g + i); };
  // two, then kAtOnce parts' loads at a time, none of which waits for a maximum: the sums so far are
  // scaled down when it rises
  float M = -INFINITY, L = 0.f, o[kDims] = {};
  auto merge = [&](int i0, auto ahead) {
    constexpr int kAhead = decltype(ahead)::value;
    float m[kAhead], l[kAhead];
    float4 x[kAhead][kDims / 4];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool there = i0 + j < parts;
      const int sl = slot(i0 + j);
      const float* acc = slot_acc(a.partials, sl) + ((dim0 + kDims * warp) * kChunkRows + row * 4);
      m[j] = there ? __ldcg(slot_m(a.partials, sl) + row) : -INFINITY;
      l[j] = there ? __ldcg(slot_l(a.partials, sl) + row) : 0.f;
#pragma unroll
      for (int k = 0; k < kDims / 4; ++k)
        x[j][k] = there ? __ldcg(reinterpret_cast<const float4*>(acc + k * kChunkRows * 4))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mn = M;
#pragma unroll
    for (int j = 0; j < kAhead; j += 2) mn = max3(mn, m[j], m[j + 1]);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float down = ex2(M - base);  // (0 at first)
    M = mn;
    L *= down;
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] *= down;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float w = ex2(m[j] - base);
      L = fmaf(w, l[j], L);
#pragma unroll
      for (int k = 0; k < kDims / 4; ++k) {
        o[4 * k] = fmaf(w, x[j][k].x, o[4 * k]);
        o[4 * k + 1] = fmaf(w, x[j][k].y, o[4 * k + 1]);
        o[4 * k + 2] = fmaf(w, x[j][k].z, o[4 * k + 2]);
        o[4 * k + 3] = fmaf(w, x[j][k].w, o[4 * k + 3]);
      }
    }
  };
  merge(0, std::integral_constant<int, 2>());
  int i = 2;
  constexpr int kRest = kAtOnce > 8 ? kAtOnce / 2 : 0;  // (what the last, smaller step takes)
#pragma unroll 1
  for (; i + kRest < parts; i += kAtOnce) merge(i, std::integral_constant<int, kAtOnce>());
  if constexpr (kRest > 0)
    if (i < parts) merge(i, std::integral_constant<int, kRest>());
  const float inv = (a.kv_dtype == MFA_KV_FP8_E4M3 ? a.v_scale : 1.f) / L;
#pragma unroll
  for (int k = 0; k < kDims / 8; ++k)
    tile[lane][kDims / 8 * warp + k] = make_uint4(
        pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
        pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
        pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
        pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
  __syncthreads();
  // whole sectors of the rows
  for (int p = threadIdx.x; p < kCombineRows * (kBlockDims / 8); p += 32 * kCombineWarps) {
    const int r = p / (kBlockDims / 8), piece = p % (kBlockDims / 8);
    *reinterpret_cast<uint4*>(a.out + (static_cast<size_t>(info.x) * kHeads + row0 + r) * kHeadDim + dim0 +
                              8 * piece) = tile[r][piece];
  }
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, ChunkAttnArgs);
constexpr int kSmemBytes = sizeof(Smem) + 1024;

// The kernel of a call's cache type and layout, its shared-memory limit raised; null on error.
Kernel kernel_of(const ChunkAttnArgs& a) {
  const Kernel all[4] = {chunk_attn_kernel<false, false>, chunk_attn_kernel<false, true>,
                         chunk_attn_kernel<true, false>, chunk_attn_kernel<true, true>};
  static std::atomic<uint64_t> smem_set[4];
  const int i = 2 * (a.kv_dtype == MFA_KV_FP8_E4M3) + (a.page_size != 0);
  if (!set_smem_limit_once(reinterpret_cast<const void*>(all[i]), kSmemBytes, &smem_set[i]))
    return nullptr;
  return all[i];
}

}  // namespace

int chunk_attn_pairs(const ChunkAttnArgs& a) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::atomic<int> cached[64];
  const bool known = dev >= 0 && dev < 64;
  if (known && cached[dev].load() > 0) return cached[dev].load();
  const Kernel kernel = kernel_of(a);
  if (kernel == nullptr) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kMaxAttnGrid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  int n = 0;
  // (every instantiation fills an SM alike: one CTA of kSmemBytes)
  if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kernel), &cfg) != cudaSuccess)
    return 0;
  if (known) cached[dev].store(n);
  return n;
}

cudaError_t launch_chunk_attn(const CUtensorMap& q_map, const CUtensorMap& out_map,
                              const ChunkAttnArgs& a, cudaStream_t s) {
  const Kernel kernel = kernel_of(a);
  if (kernel == nullptr) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_pdl(kernel, dim3(2 * a.pairs), dim3(kThreads), kSmemBytes, s, q_map, out_map, a);
  if (e != cudaSuccess) return e;
  const dim3 block(32 * kCombineWarps);
  const auto dims = [](int n) { return kHeadDim / (n * kCombineWarps); };
  if (a.n_rows > kFewTokens)
    return launch_pdl(chunk_combine_kernel<16, 4, false>, dim3(a.pairs, dims(16), kChunkRows / kCombineRows),
                      block, 0, s, a);
  // (at most)
  const int tiles = a.n_rows < a.batch ? a.n_rows : (a.n_rows + (kTokens - 1) * a.batch) / kTokens;
  if (tiles <= kFewTiles)
    return launch_pdl(chunk_combine_kernel<8, 16, true>, dim3(2 * a.n_rows, dims(8)), block, 0, s, a);
  return launch_pdl(chunk_combine_kernel<16, 4, true>, dim3(2 * a.n_rows, dims(16)), block, 0, s, a);
}

}  // namespace mfa
