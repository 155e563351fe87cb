// Attention of the newest tokens of each sequence over the paged latent cache (dsa_latent_attn),
// on the 5th-generation tensor cores.
//
//   l_j = scale q.row_j (576 dims),  O = sum_j softmax(l)_j row_j[0:512]
//
// All heads of a token (and, over every cached key, all new tokens of a sequence) share the
// cached rows, so the (token, head) pairs are the 128 lanes of a tile and the keys its columns:
//
//   S_c = Q [128 x 576] . K_c^T       O += P_c [128 x 48] . K_c[:, 0:512]
//
// One row of fp32 O is all 512 columns of an SM's TMEM, with no room for S. A cluster of two
// CTAs therefore shares a tile by dims: CTA r holds latent dims [256 r, 256 r + 256) and
// positional dims [32 r, 32 r + 32) of Q and of every key, so that each key byte is loaded into
// one of the two, S is a partial sum in each, and O's columns are split. The partial sums (fp32)
// cross over through distributed shared memory once per chunk; both CTAs then add the same two
// numbers and work out the same P. (Computing S whole in both would load every key twice and cost
// 832 products a key and lane instead of 544.)
//
// Work is split over the cache's length: the chunks of 48 keys of all tiles, one tile after the
// other, are cut into one even range per cluster, whatever the lengths. A tile whose chunks lie in
// one range is written out there; the others leave (O, m, l) in the workspace and
// latent_join_kernel adds them up. Lengths are read on the device only.
//
// Warp-specialised CTA, 512 threads (four warps a scheduler, 128 registers a thread):
//   warps 0-7   softmax / output, one (token, head) row per thread: warps 0-3 the even chunks,
//               warps 4-7 the odd ones. A chunk's way through a softmax warp is a chain of
//               latencies (S out of TMEM, the peer's half of it, the exponentials), about three
//               times what its products take, so two of them run side by side. They share the
//               running maximum, which passes from chunk to chunk in order; each keeps the sum
//               of its own chunks.
//   warps 8, 9  single-thread UMMA issuers, one for S and one for P V: the waits and commits of
//               a single one took as long as the products (18 of them for S, and one with few
//               columns takes 45 cycles whatever they are). Warp 8 owns TMEM.
//   warps 10-15 gather, eight keys of each chunk per warp: the slots of four chunks are looked up
//               at once, one key per lane, a batch ahead for the page and two for the list entry;
//               then 16-byte cp.async into 128B-swizzled tiles. e4m3 rows go through a raw ring
//               two chunks ahead and are widened to bf16, exactly, since their scales are powers
//               of two.
// Shared prefixes (dsa_latent_attn_shared): the rows of a group of sequences are tiled together over its
// prefix, whatever sequences they are of, in front of the sequences' own tiles in the same even ranges.
// Every tile leaves its (O, m, l) in the workspace, and shared_join_kernel adds those of a row up: 64
// sequences, 16 heads, a prefix of 32768 bf16 rows: 114 us, and 11 more for own rows of up to 1024 (one
// sequence with as many rows over the prefix 109). As 64 sequences by themselves, the prefix's pages in front
// of each one's own, they take 538 us; with 32 / 64 / 128 heads 209 / 378 / 716 against 539 / 561 / 707: what
// the tiling saves are the empty rows of a tile, and with 128 rows a sequence there are none.
// P goes to the tensor cores through shared memory, so that a chunk's S columns are free again
// once they have been read. TMEM: [Q: 144][S: 2 x 48][pad 16][O: 256] = 512 columns.
//
// Measured (device time): four sequences of 131072 e4m3 rows, 128 heads: 221 us, 660 TFLOP/s,
// 1.56 TB/s; 32 sequences of 256 to 8192 bf16 rows: 69 us. A chunk takes about 1900 cycles in
// steady state (bf16; 2600 with e4m3) of which the products are 1190: with bf16 the hand-offs
// between the warps pace it, with e4m3 a gather warp's way through a chunk (copies 600, widening
// 650, lookups 250, the fence and the waits), all of it in reach of the same shared memory.

#include <mutex>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "latent_row.cuh"

namespace dsa {
namespace {

constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kNK = 48;                  // keys per chunk
constexpr int kHalf = kDc / 2;           // latent dims (and O columns) per CTA
constexpr int kHalfR = kDr / 2;          // positional dims per CTA
constexpr int kSteps = (kHalf + kHalfR) / 16;   // MMA k-steps of S
constexpr int kAtoms = 5;                // 64-dim atoms per key; the last one half filled
constexpr uint32_t kAtom = kNK * 128;
constexpr uint32_t kStage = kAtoms * kAtom;
constexpr uint32_t kExch = 128 * kNK * 4;   // one buffer of the peer's partial S
constexpr uint32_t kPTile = 128 * 32;       // P of 16 keys: one k-step of P V
constexpr uint32_t kPBuf = kNK / 16 * kPTile;
constexpr int kIssueWarp = 8, kIssuePvWarp = 9;
constexpr int kGatherWarp0 = 10, kGatherWarps = 6;
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr int kKeysPerWarp = kNK / kGatherWarps;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);
constexpr uint32_t kColQ = 0, kColS = 144, kColO = 256;
constexpr int kMinChunks = 3;            // chunks that a cluster takes at least: 1000 keys of
                                         // four sequences 16.3 us, with two 18.4, four 18.6
constexpr int kTileCost = 5;             // chunks that a change of tiles is worth: 128 ragged
                                         // sequences up to 2000 keys 86 us, 154 with none
constexpr int kMaxClusters = 80;         // clusters that the workspace has room for
constexpr float kRescaleLog2 = 8.f;      // refresh the running max when it grows by > 2^8
constexpr int kErrIdx = DSA_STAGE_LATENT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_LATENT | DSA_DEVERR_BAD_PAGE;
constexpr int kErrTime = DSA_STAGE_LATENT | DSA_DEVERR_TIMEOUT;
static_assert(kKeysPerWarp == 8, "the keys of a gather warp are one byte of the chunk's mask");
constexpr int kMaxGroups = kLatentGroups;   // groups of sequences that share a prefix
constexpr int kAllSee = -0x7fffffff - 1;   // Header::lim0 of a prefix's tile: every row sees every key

// e4m3: 48 keys x 16 pieces of 16 codes and 48 x 4 of positional dims, four and one per gather
// thread, and two scales per key, in a ring of raw chunks
constexpr int kCodeReps = kNK * (kHalf / 16) / kGatherThreads;
constexpr uint32_t kRawRope = kCodeReps * kGatherThreads * 16;
constexpr uint32_t kRawScale = kRawRope + kGatherThreads * 16;
constexpr uint32_t kRaw = kRawScale + kNK * 8;
constexpr int kAhead = 2;
static_assert(kNK * (kHalfR / 8) == kGatherThreads, "one piece of positional dims per thread");

template <bool FP8>
struct Layout {
  static constexpr int kStages = FP8 ? 4 : 5;
  static constexpr uint32_t kExchOff = kStages * kStage;   // the peer's S of an even / odd chunk
  static constexpr uint32_t kPOff = kExchOff + 2 * kExch;  // P of an even / odd chunk
  static constexpr uint32_t kRawOff = kPOff + 2 * kPBuf;
  static constexpr uint32_t kTailOff = kRawOff + (FP8 ? kAhead * kRaw : 0);
};
constexpr int kMaxStages = 5;
constexpr size_t kSmemMost = 232448;   // of a block

struct Header {
  int item;    // tile
  int cf;      // 16 * (chunk of the tile) + 1: its first chunk here, 2: its last one here, 4: the
               // whole tile is here, 8: the next chunk is its last one here
  int lim0;    // keys that the tile's first row sees (every cached key); unused with lists
  uint32_t valid[2];   // the chunk's 48 keys: a byte from each gather warp
};

struct Tail {
  Header hdr[kMaxStages];
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  // by parity of the chunk; x_full / x_free (the peer's partial S is there / was read by the
  // peer) and turn (the chunk has settled the running maximum) also by softmax warp
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t x_full[2][4], x_free[2][4], turn[2][4];
  uint64_t q_full, o_free, drain[2];
  float mref[128];            // running maximum of each row (raw logits)
  float lsum[2][2][128];      // [parity][every second chunk of it]: the sum of its chunks so far
  uint32_t tmem_base;
  int abort_flag;
  long long sums[kThreads / 32];
  // this cluster's range: its first tile, that tile's first chunk here, the chunks of all tiles in
  // front of the range and of its end, and a range's weight
  int item0, c0;
  long long first, end;
  int each;
  // shared prefixes: first sequence of each group and the end of the last, first tile of each group's
  // rows and their number, keys of its prefix
  int gstart[kMaxGroups + 1], gtile[kMaxGroups + 1], gkeys[kMaxGroups];
};

static_assert(Layout<false>::kTailOff + sizeof(Tail) <= kSmemMost &&
                  Layout<true>::kTailOff + sizeof(Tail) <= kSmemMost &&
                  Layout<true>::kTailOff % 8 == 0,
              "shared memory of a block");

struct Params {
  LatentArgs a;
  int tiles;        // tiles per sequence (lists: one per token, B * Sq in all)
  int items;
  int list_chunks;  // chunks of a list (lists only)
  int clusters;
  int act_warps;    // softmax warps with rows
  int prow;         // rows of a workspace part (32 * act_warps)
  int page_shift;   // log2 of the page size, -1 where it is no power of two
  float scale_log2;
  float4* part;     // [2 * clusters][128 groups of 4 dims][prow]
  float2* ml;       // [2 * clusters][prow]: running max (of the logits before scale) and sum
  int2* joins;      // [clusters]: the tile that begins in a cluster's range and goes on behind it
                    // (-1: none), and the last cluster that works on it
  // Shared prefixes: the tiles of the groups' rows over their prefixes come first, then those of the
  // sequences over their own keys. Each leaves parts, tile i's of cluster c at i + c (which goes up
  // along the work, so that no two have the same); part, ml: [most tiles + clusters].
  int most_items;   // tiles that there can be
  int2* spans;      // [most tiles]: the first and the last cluster of each
  int* groups;      // the tables of Tail, for the join: gstart, gtile
};

// ------------------------------------------------------------------ the split

__device__ __forceinline__ int seq_len(const LatentArgs& a, int b, bool report) {
  const int cap = a.max_pages * a.page_size;
  const int len = __ldg(a.lens + b);
  if (report && (len < 0 || len > cap)) report_error(a.err, kErrPage);
  return max(0, min(len, cap));
}

// rows of tile mt of a sequence: [128 mt, 128 mt + rows)
__device__ __forceinline__ int tile_rows(const Params& p, int mt) {
  return min(128, p.a.Sq * p.a.H - mt * 128);
}

// the group whose tiles `item` is one of (item < gtile[G])
__device__ __forceinline__ int group_of(const Params& p, const Tail* tail, int item) {
  int g = 0;
  for (int n = p.a.G; n > 1;) {   // the last one that begins at or in front of it
    const int half = n >> 1;
    if (tail->gtile[g + half] <= item) g += half;
    n -= half;
  }
  return g;
}

// first row of tile `item` in Q, O and lse, and the rows it has
template <bool SHARED>
__device__ __forceinline__ long long rows_of(const Params& p, const Tail* tail, int item, int& rows) {
  if (SHARED) {
    const int prefix_tiles = tail->gtile[p.a.G];
    if (item < prefix_tiles) {
      const int g = group_of(p, tail, item), row = (item - tail->gtile[g]) * 128;
      const int per = p.a.Sq * p.a.H;
      rows = min(128, (tail->gstart[g + 1] - tail->gstart[g]) * per - row);
      return static_cast<long long>(tail->gstart[g]) * per + row;
    }
    item -= prefix_tiles;
  } else if (p.a.idx) {
    rows = p.a.H;
    return static_cast<long long>(item) * p.a.H;
  }
  const int b = item / p.tiles, mt = item - b * p.tiles;
  rows = tile_rows(p, mt);
  return static_cast<long long>(b) * p.a.Sq * p.a.H + mt * 128;
}

// keys that the last row of a tile sees
__device__ __forceinline__ int tile_keys(const Params& p, int len, int mt) {
  const int i1 = (mt * 128 + tile_rows(p, mt) - 1) / p.a.H;
  return max(0, len - p.a.Sq + i1 + 1);
}

// a tile without a key has one (empty) chunk, which writes its rows
// (keys + kNK - 1 may be past 32 bits)
__device__ __forceinline__ int chunks_of(int keys) { return keys > 0 ? (keys - 1) / kNK + 1 : 1; }

template <bool SHARED>
__device__ __forceinline__ int item_chunks(const Params& p, const Tail* tail, int item) {
  if (SHARED) {
    if (item < tail->gtile[p.a.G]) return chunks_of(tail->gkeys[group_of(p, tail, item)]);
    item -= tail->gtile[p.a.G];
  } else if (p.a.idx) {
    return p.list_chunks;
  }
  const int b = item / p.tiles;
  return chunks_of(tile_keys(p, seq_len(p.a, b, false), item - b * p.tiles));
}

// What a cluster takes of the chunks of all tiles, into the tail: [c0, ...) of tile item0, n chunks
// in all. Every thread of the block calls it, before a barrier.
//
// The chunks are cut by weight: going on to another tile costs about as much as kTileCost chunks
// (its Q, an empty pipeline, an output), so a tile weighs that much in front of its chunks. Cluster
// c has the chunks at weights [each c, each (c + 1)). Short ranges count no such cost: they would be
// cut into setups alone. With shared prefixes they do: there are as many short tiles as sequences, which
// would else fall to a few clusters one after the other. (3 / 5 / 8 / 12 chunks: 32 sequences behind 8192
// keys with 128 heads 141 / 129 / 132 / 136 us, 96 behind 3000 with 32 heads 62 / 64 / 69 / 77.)
template <bool SHARED>
__device__ __forceinline__ void my_chunks(const Params& p, int cluster, Tail* tail) {
  const int items = SHARED ? tail->gtile[p.a.G] + p.items : p.items;
  long long total, before = 0, s = 0;   // chunks: of all tiles, in front of this thread's, of its own
  int i0 = 0, i1 = 0;                   // this thread's tiles
  if (!SHARED && p.a.idx) {
    total = static_cast<long long>(p.items) * p.list_chunks;
  } else {
    const int q = (items + kThreads - 1) / kThreads;
    i0 = min(items, static_cast<int>(threadIdx.x) * q);
    i1 = min(items, i0 + q);
    for (int i = i0; i < i1; ++i) s += item_chunks<SHARED>(p, tail, i);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) tail->sums[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += tail->sums[w];
      total += tail->sums[w];
    }
    before += incl - s;
  }
  const int cost = SHARED || (total + p.clusters - 1) / p.clusters >= 4 * kTileCost ? kTileCost : 0;
  const long long weight = total + static_cast<long long>(cost) * items;
  const long long each =
      max((weight + p.clusters - 1) / p.clusters, static_cast<long long>(kMinChunks));
  const long long w0 = each * cluster, w1 = min(w0 + each, weight);
  if (threadIdx.x == 0) tail->each = static_cast<int>(each);
  if (w0 >= weight) return;   // first and end stay 0
  if (w1 == weight && threadIdx.x == 0) tail->end = total;
  if (!SHARED && p.a.idx) {
    if (threadIdx.x != 0) return;
    const int per = cost + p.list_chunks;
    // chunks in front of weight w
    auto chunk_at = [&](long long w, int& item, int& c) {
      item = static_cast<int>(w / per);
      c = max(0, static_cast<int>(w - static_cast<long long>(item) * per) - cost);
      return static_cast<long long>(item) * p.list_chunks + c;
    };
    int item, c;
    if (w1 < weight) tail->end = chunk_at(w1, item, c);
    tail->first = chunk_at(w0, tail->item0, tail->c0);
    return;
  }
  long long at = before + static_cast<long long>(cost) * i0;   // weight in front of tile i
  for (int i = i0; i < i1; ++i) {
    const int m = i1 - i0 == 1 ? static_cast<int>(s) : item_chunks<SHARED>(p, tail, i);
    const long long end = at + cost + m;
    if (w0 >= at && w0 < end) {
      const int c = max(0, static_cast<int>(w0 - at) - cost);
      tail->item0 = i;
      tail->c0 = c;
      tail->first = before + c;
    }
    if (w1 >= at && w1 < end) tail->end = before + max(0, static_cast<int>(w1 - at) - cost);
    at = end;
    before += m;
  }
}

// The groups of sequences that share a prefix, into the tail: starts that go down or out of [0, B] are
// taken as the nearest that do not, a group without rows or keys has no tiles. Every thread of the
// block calls it.
__device__ __forceinline__ void my_groups(const Params& p, bool report, Tail* tail) {
  const int t = threadIdx.x, G = p.a.G;
  if (t <= G) tail->gstart[t] = __ldg(p.a.starts + t);
  if (t < G) {
    const int cap = p.a.max_prefix * p.a.page_size, keys = __ldg(p.a.prefix_lens + t);
    if (report && (keys < 0 || keys > cap)) report_error(p.a.err, kErrPage);
    tail->gkeys[t] = max(0, min(keys, cap));
  }
  __syncthreads();
  if (t == 0) {
    int at = 0, tiles = 0;
    bool bad = false;
    for (int g = 0; g <= G; ++g) {
      const int want = tail->gstart[g], got = max(at, min(want, p.a.B));
      bad = bad || want != got;
      if (g > 0) {
        if (tail->gkeys[g - 1] > 0) tiles += ((got - at) * p.a.Sq * p.a.H + 127) / 128;
      }
      tail->gstart[g] = at = got;
      tail->gtile[g] = tiles;
    }
    if (report && bad) report_error(p.a.err, kErrIdx);
  }
  __syncthreads();
}

// ------------------------------------------------------------------ small helpers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// 16 bytes into the peer's shared memory, counted on the peer's barrier
__device__ __forceinline__ void st_peer(uint32_t dst, uint32_t bar, uint32_t a, uint32_t b,
                                        uint32_t c, uint32_t d) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::
          "r"(dst),
      "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d)
      : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Tells the peer that what it sent has been read, by every lane of the warp; `used` is worked out from
// all that the lane has read. Relaxed: a release at cluster scope waits for what the warp itself
// has on its way to the peer, and at every place for it, in this warp or in an issuer's, it took 3 to
// 10% (four sequences of 131072 e4m3 rows 223 to 241 us instead of 220, and 222 this way; 32 ragged
// bf16 ones 75 to 78 instead of 72). The order comes from a chain of dependencies: the arrival hangs on a vote over
// values worked out from the reads, the peer's next stores hang on the arrival, and no value comes
// out of thin air, so no read can return what those stores write. (Reads and stores are of the same
// size and place.) kNoMaximum is a NaN that no addition or maximum gives: the vote always passes.
constexpr uint32_t kNoMaximum = 0x7fa5a5a5u;
__device__ __forceinline__ void arrive_peer(uint32_t bar, float used, int lane) {
  if (__any_sync(0xffffffffu, __float_as_uint(used) != kNoMaximum) && lane == 0)
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

// mbar_wait for what the peer CTA sends
__device__ __forceinline__ bool wait_peer(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* err) {
  const uint32_t a = smem_u32(bar);
  if (try_wait_cluster(a, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait_cluster(a, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      report_error(err, kErrTime);
      return false;
    }
  }
}

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations per instruction, and a maximum of three.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}

// widen4 gives the bytes as (0, 2) and (1, 3): of every four latent dims the middle two are swapped in
// the tile, in Q's columns (load_q) and in O's, and O is written the right way round. (With the dims in
// order: selected e4m3 keys 138.6 us, long 240; 133 and 225 this way, the rest by the loads and stores
// around it.)

// two bf16 with infinities and NaNs replaced by zero
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// Keys [from, to) of a chunk: infinities and NaNs of their latent dims replaced by zero (four atoms of
// 64 dims, a row of 128 bytes of each per key), by thread t of n.
__device__ __forceinline__ void drop_non_finite(uint8_t* stage, int from, int to, int t, int n) {
#pragma unroll 1
  for (int i = from * 32 + t; i < to * 32; i += n) {
    uint4* at = reinterpret_cast<uint4*>(stage + ((i >> 3) & 3) * kAtom + (i >> 5) * 128) + (i & 7);
    const uint4 w = *at;
    const uint4 f = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
    if (f.x != w.x || f.y != w.y || f.z != w.z || f.w != w.w) *at = f;
  }
}

// log sum exp of a row with largest logit m (before scale) and sum l; a row without a key has l = 0
__device__ __forceinline__ float lse_of(const Params& p, float m, float l) {
  return l == 0.f ? -INFINITY : m * p.a.scale + log2f(l) * 0.69314718055994530942f;
}

// ------------------------------------------------------------------ the kernel

// where a gather warp stands in its cluster's chunks
struct Cursor {
  int item, c, nch, len, keys, b, lim0;
};

template <bool SHARED>
__device__ __forceinline__ void enter_item(const Params& p, const Tail* tail, int item, Cursor& k) {
  k.item = item;
  if (SHARED) {
    const int prefix_tiles = tail->gtile[p.a.G];
    if (item < prefix_tiles) {
      const int g = group_of(p, tail, item);
      k.b = ~g;
      k.keys = k.len = tail->gkeys[g];
      k.nch = chunks_of(k.keys);
      k.lim0 = kAllSee;
      return;
    }
    item -= prefix_tiles;
  }
  k.b = item / (p.a.idx ? p.a.Sq : p.tiles);
  const int at = item - k.b * (p.a.idx ? p.a.Sq : p.tiles);   // the token, or the tile
  k.len = seq_len(p.a, k.b, true);
  if (p.a.idx) {
    k.keys = max(0, k.len - p.a.Sq + at + 1);
    k.nch = p.list_chunks;
    k.lim0 = 0;
  } else {
    k.keys = tile_keys(p, k.len, at);
    k.nch = chunks_of(k.keys);
    k.lim0 = k.len - p.a.Sq + 1 + (at * 128) / p.a.H;
  }
}

template <bool FP8, bool SHARED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const Params p) {
  using L = Layout<FP8>;
  constexpr int kStages = L::kStages;
  constexpr uint32_t kExchOff = L::kExchOff, kPOff = L::kPOff;
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail* tail = reinterpret_cast<Tail*>(smem + L::kTailOff);
  volatile int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;
  int* err = p.a.err;
  // the same in both CTAs of a cluster (one layout), so both leave
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) report_error(err, DSA_STAGE_LATENT | DSA_DEVERR_MISALIGNED);
    return;
  }

  if (threadIdx.x == 0) {
    const int act_threads = 32 * p.act_warps;   // softmax threads of a chunk
    for (int i = 0; i < kStages; ++i) {
      // every gather thread when its part has landed, and one per gather warp for the header
      mbar_init(&tail->kv_full[i], kGatherThreads + kGatherWarps);
      mbar_init(&tail->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->s_full[i], 1);
      mbar_init(&tail->s_free[i], act_threads);
      mbar_init(&tail->p_full[i], act_threads);
      mbar_init(&tail->pv_done[i], 1);
      for (int w = 0; w < 4; ++w) {
        mbar_init(&tail->x_full[i][w], 1);
        mbar_init(&tail->x_free[i][w], 1);
        mbar_init(&tail->turn[i][w], 1);
      }
    }
    mbar_init(&tail->q_full, act_threads);
    mbar_init(&tail->o_free, act_threads);
    mbar_init(&tail->drain[0], 1);
    mbar_init(&tail->drain[1], 1);
    tail->abort_flag = 0;
    tail->first = tail->end = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&tail->tmem_base, 512);
    tmem_relinquish();
  }
  // thread 0 has made this CTA's barriers; the peer's are ready once cluster_wait returns
  cluster_arrive();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (SHARED) {
    my_groups(p, blockIdx.x == 0, tail);
    if (blockIdx.x == 0 && threadIdx.x <= p.a.G) {
      p.groups[threadIdx.x] = tail->gstart[threadIdx.x];
      p.groups[kMaxGroups + 1 + threadIdx.x] = tail->gtile[threadIdx.x];
    }
  }
  my_chunks<SHARED>(p, cluster, tail);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  const int n = static_cast<int>(tail->end - tail->first), item0 = tail->item0, c0 = tail->c0;

  if (n == 0) {
    // nothing here (both CTAs agree)
    if (!SHARED && threadIdx.x == 0 && rank == 0) p.joins[cluster] = make_int2(-1, 0);
    cluster_wait();
  } else if (warp >= kGatherWarp0) {
    // ================================================================ gather
    const int gw = warp - kGatherWarp0;
    const int mykey = gw * kKeysPerWarp + (lane & 7);
    const long long row_bytes = FP8 ? kDc + 16 + 2 * kDr : 2 * kD;
    Cursor k;
    enter_item<SHARED>(p, tail, item0, k);
    k.c = c0;
    const bool scribe = gw == 0 && lane == 0 && rank == 0;
    if (SHARED && scribe && c0 == 0) p.spans[item0].x = cluster;
    int made = 0;   // chunks handed out
    // Three steps for the keys of four chunks, lane 8 i + j the warp's key j of the i-th of them:
    // the chunk and its list entry, the page of its position, its slot.
    struct Entry {
      int raw, len, keys, b, item, cf, lim0;
    };
    struct Paged {
      int page, off, item, cf, lim0;   // off: row of the page, -1 without a key
    };
    struct Slot {
      int slot, item, cf, lim0;
    };
    // the next tile's Q, to be read by the softmax warps some chunks later, on its way to L2
    auto prefetch_q = [&](int item) {
      int rows;
      const long long r0 = rows_of<SHARED>(p, tail, item, rows);
      for (int i = gw * 32 + lane; i < rows * 5; i += kGatherThreads) {
        const int row = i / 5, piece = i - row * 5;
        const uint16_t* at = p.a.Q + (r0 + row) * kD +
                             (piece < 4 ? rank * kHalf + piece * 64 : kDc + rank * kHalfR);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
      }
    };
    auto look = [&]() {
      Entry e = {-1, 0, 0, 0, 0, 0, 0};
      // chunk k.c + i of the tile, the (made + i)-th of the range
      auto take = [&](int i) {
        const int c = k.c + i, m = made + i;
        const int to_go = min(n - 1 - m, k.nch - 1 - c);   // chunks of the tile behind it
        e.cf = 16 * c + (m == 0 || c == 0 ? 1 : 0) + (to_go == 0 ? 2 : 0) + (to_go == 1 ? 8 : 0);
        // the whole tile is in this range: its first chunk was here, and its last one is
        if (c <= m && k.nch - c <= n - m) e.cf += 4;
        e.len = k.len;
        e.keys = k.keys;
        e.b = k.b;
        e.item = k.item;
        e.lim0 = k.lim0;
        const uint32_t j = static_cast<uint32_t>(c) * kNK + mykey;   // past 2^31 in a last chunk
        e.raw = j < static_cast<uint32_t>(!SHARED && p.a.idx ? p.a.k : k.keys) ? static_cast<int>(j) : -1;
      };
      if (made + 4 < n && k.c + 4 < k.nch) {
        take(lane >> 3);
        made += 4;
        k.c += 4;
      } else {
#pragma unroll 1
        for (int i = 0; i < 4 && made < n; ++i) {
          if ((lane >> 3) == i) take(0);
          if (++made == n) {
            // a tile that begins here and goes on in later clusters
            const int left = k.nch - 1 - k.c;
            if (SHARED && scribe && left == 0) p.spans[k.item].y = cluster;
            if (!SHARED && scribe)
              p.joins[cluster] =
                  left > 0 && k.c < n
                      ? make_int2(k.item, cluster + (left + tail->each - 1) / tail->each)
                      : make_int2(-1, 0);
          } else if (++k.c == k.nch) {
            if (SHARED && scribe) {
              p.spans[k.item].y = cluster;
              p.spans[k.item + 1].x = cluster;
            }
            enter_item<SHARED>(p, tail, k.item + 1, k);
            k.c = 0;
            prefetch_q(k.item);
          }
        }
      }
      if (!SHARED && p.a.idx && e.raw >= 0)
        e.raw = __ldg(p.a.idx + static_cast<long long>(e.item) * p.a.k + e.raw);
      return e;
    };
    auto page_of = [&](const Entry& e) {
      Paged q = {-1, -1, e.item, e.cf, e.lim0};
      if (e.raw < -1 || e.raw >= e.len) {
        if (e.raw != -1) report_error(err, kErrIdx);
      } else if (e.raw >= 0 && e.raw < e.keys) {
        const int pg = p.page_shift >= 0 ? e.raw >> p.page_shift : e.raw / p.a.page_size;
        q.off = e.raw - pg * p.a.page_size;
        q.page = __ldg((SHARED && e.b < 0
                            ? p.a.prefix_table + static_cast<long long>(~e.b) * p.a.max_prefix
                            : p.a.page_table + static_cast<long long>(e.b) * p.a.max_pages) + pg);
      }
      return q;
    };
    auto slot_of = [&](const Paged& q) {
      Slot r = {-1, q.item, q.cf, q.lim0};
      if (q.off >= 0) {
        if (q.page < 0 || q.page >= p.a.num_pages)
          report_error(err, kErrPage);
        else
          r.slot = q.page * p.a.page_size + q.off;
      }
      return r;
    };
    Entry e0 = {-1, 0, 0, 0, 0, 0, 0};
    Paged q0 = {-1, -1, 0, 0, 0};
    Slot now = {-1, 0, 0, 0};
    int steps = 3;   // to the first batch's slots
    auto next_batch = [&]() {
#pragma unroll 1
      for (; steps > 0; --steps) {
        now = slot_of(q0);
        q0 = page_of(e0);
        e0 = look();
      }
      steps = 1;
    };
    const uint32_t base = smem_u32(smem);

    if (!FP8) {
      for (int g = 0; g < n; ++g) {
        const int b8 = (g & 3) * 8;   // the lanes with this chunk's keys
        if (b8 == 0) next_batch();
        const int st = g % kStages;
        const uint32_t par = ((g / kStages) & 1) ^ 1u;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&tail->kv_empty[st], par, abort_flag, err, kErrTime)))
          break;
        const uint32_t bal = __ballot_sync(0xffffffffu, now.slot >= 0);
        if (lane == b8) {
          Header& h = tail->hdr[st];
          reinterpret_cast<uint8_t*>(h.valid)[gw] = static_cast<uint8_t>(bal >> b8);
          if (gw == 0) {
            h.item = now.item;
            h.cf = now.cf;
            h.lim0 = now.lim0;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->kv_full[st]);   // the header
        const uint32_t stage = base + st * kStage;
#pragma unroll
        for (int i = 0; i < kKeysPerWarp; ++i) {
          const int s = __shfl_sync(0xffffffffu, now.slot, b8 + i);
          const int key = gw * kKeysPerWarp + i;
          const uint8_t* src = p.a.cache + (s >= 0 ? s : 0) * row_bytes + rank * (2 * kHalf);
          cp_async_16(stage + (lane >> 3) * kAtom + key * 128 + (((lane & 7) ^ (key & 7)) << 4),
                      src + lane * 16, s >= 0 ? 16u : 0u);
        }
        {
          const int i = lane >> 2, pc = lane & 3;   // four pieces of positional dims per key
          const int s = __shfl_sync(0xffffffffu, now.slot, b8 + i);
          const int key = gw * kKeysPerWarp + i;
          const uint8_t* src =
              p.a.cache + (s >= 0 ? s : 0) * row_bytes + 2 * kDc + rank * (2 * kHalfR);
          cp_async_16(stage + 4 * kAtom + key * 128 + ((pc ^ (key & 7)) << 4), src + pc * 16,
                      s >= 0 ? 16u : 0u);
        }
        // arrives, by the copy hardware, once this thread's copies have landed
        cp_async_mbar_arrive(&tail->kv_full[st]);
      }
      cp_async_wait<0>();
    } else {
      // Raw ring: a thread copies in the codes and positional dims that it converts itself; the
      // scales are the warp's.
      uint8_t* const raw = smem + L::kRawOff;
      const int gt = gw * 32 + lane;
      // A thread's codes: piece pc of the warp's keys odd, 2 + odd, ... Eight lanes have the four
      // pieces of an atom of an even and an odd key, which the tile's swizzle puts in eight
      // different bank groups.
      const int odd = (lane >> 2) & 1, pc = (lane >> 3) * 4 + (lane & 3);
      struct Ahead {
        uint32_t valid;
        int item, cf, lim0;
      };
      auto fetch = [&](Ahead& r, int g) {
        const int b8 = (g & 3) * 8;   // the lanes with this chunk's keys
        if (b8 == 0) next_batch();
        if (gw == 0) {
          r.item = __shfl_sync(0xffffffffu, now.item, b8);
          r.cf = __shfl_sync(0xffffffffu, now.cf, b8);
          r.lim0 = __shfl_sync(0xffffffffu, now.lim0, b8);
        }
        r.valid = (__ballot_sync(0xffffffffu, now.slot >= 0) >> b8) & 0xffu;
        const uint32_t rs = smem_u32(raw) + (g % kAhead) * kRaw;
#pragma unroll
        for (int j = 0; j < kCodeReps; ++j) {
          const int s = __shfl_sync(0xffffffffu, now.slot, b8 + 2 * j + odd);
          cp_async_16(rs + (j * kGatherThreads + gt) * 16,
                      p.a.cache + (s >= 0 ? s : 0) * row_bytes + rank * kHalf + pc * 16,
                      s >= 0 ? 16u : 0u);
        }
        {
          const int s = __shfl_sync(0xffffffffu, now.slot, b8 + (lane >> 2));
          cp_async_16(rs + kRawRope + gt * 16,
                      p.a.cache + (s >= 0 ? s : 0) * row_bytes + kDc + 16 + rank * (2 * kHalfR) +
                          (lane & 3) * 16,
                      s >= 0 ? 16u : 0u);
        }
        {
          // scale lane & 1 of key (lane >> 1) & 7, so that the four of a thread are 16 bytes
          const int s = __shfl_sync(0xffffffffu, now.slot, b8 + ((lane >> 1) & 7));
          if (lane < 16)
            cp_async_4(rs + kRawScale + gw * 64 + ((lane & 3) * 4 + (lane >> 2)) * 4,
                       p.a.cache + (s >= 0 ? s : 0) * row_bytes + kDc + rank * 8 + (lane & 1) * 4,
                       s >= 0 ? 4u : 0u);
        }
        cp_async_commit();
      };
      static_assert(kAhead == 2, "two chunks on their way");
      Ahead a0 = {0, 0, 0, 0}, a1 = a0;
      for (int f = 0; f < n + kAhead; ++f) {
        const int g = f - kAhead;
        const Ahead r = a0;
        uint4 code[kCodeReps], rope, scales;
        if (g >= 0) {
          cp_async_wait<kAhead - 1>();
          __syncwarp();
          const uint8_t* rs = raw + (g % kAhead) * kRaw;
#pragma unroll
          for (int j = 0; j < kCodeReps; ++j)
            code[j] = *reinterpret_cast<const uint4*>(rs + (j * kGatherThreads + gt) * 16);
          scales = *reinterpret_cast<const uint4*>(rs + kRawScale + gw * 64 +
                                                   (odd * 2 + (lane >> 4)) * 16);
          rope = *reinterpret_cast<const uint4*>(rs + kRawRope + gt * 16);
          __syncwarp();
        }
        a0 = a1;
        fetch(a1, f);   // no keys behind the end
        if (g >= 0) {
          const int st = g % kStages;
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->kv_empty[st], ((g / kStages) & 1) ^ 1u,
                                                 abort_flag, err, kErrTime)))
            break;
          if (lane == 0) {
            Header& h = tail->hdr[st];
            reinterpret_cast<uint8_t*>(h.valid)[gw] = static_cast<uint8_t>(r.valid);
            if (gw == 0) {
              h.item = r.item;
              h.cf = r.cf;
              h.lim0 = r.lim0;
            }
            mbar_arrive(&tail->kv_full[st]);
          }
          uint8_t* stage = smem + st * kStage;
          // the scales' upper halves: 2^k as bf16. (A key that is not there has codes and scale
          // bits of zero.)
          const uint32_t e[kCodeReps] = {scales.x >> 16, scales.y >> 16, scales.z >> 16,
                                         scales.w >> 16};
          // keys 2 j + odd of the warp's eight: rows of 128 bytes, their pieces swizzled by 2 j
          uint8_t* const at = stage + (lane >> 3) * kAtom + (gw * kKeysPerWarp + odd) * 128;
          const int put = ((lane & 3) * 2 ^ odd) << 4;
          bool wide = false;
#pragma unroll
          for (int j = 0; j < kCodeReps; ++j) {
            // 2^(120 + k) twice, or 2^127 and the rest below
            const uint32_t up = widen_factor(e[j]);
            wide = wide || e[j] > kScaleMost;
            uint4 w0, w1;
            widen4(code[j].x, up, w0.x, w0.y);
            widen4(code[j].y, up, w0.z, w0.w);
            widen4(code[j].z, up, w1.x, w1.y);
            widen4(code[j].w, up, w1.z, w1.w);
            *reinterpret_cast<uint4*>(at + j * 256 + (put ^ (j * 32))) = w0;
            *reinterpret_cast<uint4*>(at + j * 256 + (put ^ (j * 32) ^ 16)) = w1;
            // Two keys' pieces at a time: the compiler else mixes all four and runs out of
            // registers (16 ragged sequences up to 32768, 64 heads: 104 us, not 98).
            if (j == 1) asm volatile("" ::: "memory");
          }
          if (wide) {   // a scale of more than 2^7, or of NaN
#pragma unroll 1
            for (int i = 0; i < 2 * kCodeReps; ++i) {
              const int j = i >> 1;
              const uint32_t ej = (j & 2 ? (j & 1 ? scales.w : scales.z)
                                         : (j & 1 ? scales.y : scales.x)) >> 16;
              if (ej <= kScaleMost) continue;
              const uint32_t more = widen_rest(ej);
              uint4* const piece = reinterpret_cast<uint4*>(at + j * 256 + (put ^ (i * 16)));
              uint4 w = *piece;
              w.x = mul_bf16x2(w.x, more);
              w.y = mul_bf16x2(w.y, more);
              w.z = mul_bf16x2(w.z, more);
              w.w = mul_bf16x2(w.w, more);
              *piece = w;
            }
          }
          {
            const int key = gw * kKeysPerWarp + (lane >> 2), pc = lane & 3;
            *reinterpret_cast<uint4*>(stage + 4 * kAtom + key * 128 + ((pc ^ (key & 7)) << 4)) =
                rope;
          }
          fence_proxy_async_smem();
          mbar_arrive(&tail->kv_full[st]);
        }
      }
      cp_async_wait<0>();
    }
    cluster_wait();
  } else if (warp == kIssueWarp || warp == kIssuePvWarp) {
    // ================================================================ UMMA issuers
    if (lane == 0) {
      const uint32_t base = smem_u32(smem);
      if (warp == kIssueWarp) {
        constexpr uint32_t idesc = umma_idesc_bf16_mn(128, kNK, false);
        uint32_t q_par = 0;
        for (int g = 0; g < n; ++g) {
          const int st = g % kStages, sb = g & 1;
          if (!mbar_wait(&tail->kv_full[st], (g / kStages) & 1, abort_flag, err, kErrTime)) break;
          if (tail->hdr[st].cf & 1) {
            if (!mbar_wait(&tail->q_full, q_par, abort_flag, err, kErrTime)) break;
            q_par ^= 1u;
          }
          if (!mbar_wait(&tail->s_free[sb], ((g >> 1) & 1) ^ 1u, abort_flag, err, kErrTime)) break;
          if (!FP8) fence_proxy_async_smem();   // cp.async wrote the rows by the generic proxy
          tc_fence_after();
          const uint64_t k0 = umma_sdesc(base + st * kStage, 1024, kLayoutSw128);
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk)
            umma_bf16_ts(tmem + kColS + sb * kNK, tmem + kColQ + kk * 8,
                         umma_desc_adv(k0, (kk >> 2) * kAtom + (kk & 3) * 32), idesc,
                         kk > 0 ? 1u : 0u);
          umma_commit(&tail->s_full[sb]);
        }
      } else {
        constexpr uint32_t idesc = umma_idesc_bf16_mn(128, kHalf, true);
        uint32_t o_par = 1;
        for (int g = 0; g < n; ++g) {
          const int st = g % kStages, sb = g & 1;
          if (!mbar_wait(&tail->kv_full[st], (g / kStages) & 1, abort_flag, err, kErrTime)) break;
          const bool first = (tail->hdr[st].cf & 1) != 0;
          if (!FP8) fence_proxy_async_smem();
          if (first) {   // the previous tile's O has been read out
            if (!mbar_wait(&tail->o_free, o_par, abort_flag, err, kErrTime)) break;
            o_par ^= 1u;
          }
          if (!mbar_wait(&tail->p_full[sb], (g >> 1) & 1, abort_flag, err, kErrTime)) break;
          tc_fence_after();
          const uint64_t p0 = umma_sdesc(base + kPOff + sb * kPBuf, 256, kLayoutSw32);
          const uint64_t v0 = umma_sdesc_lbo(base + st * kStage, kAtom, 1024, kLayoutSw128);
#pragma unroll
          for (int ks = 0; ks < kNK / 16; ++ks)
            umma_bf16(tmem + kColO, umma_desc_adv(p0, ks * kPTile), umma_desc_adv(v0, ks * 2048),
                      idesc, (first && ks == 0) ? 0u : 1u);
          umma_commit(&tail->kv_empty[st]);
          umma_commit(&tail->pv_done[sb]);
        }
      }
      uint64_t* drain = &tail->drain[warp == kIssueWarp ? 0 : 1];
      umma_commit(drain);
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(drain), 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          report_error(err, kErrTime);
          break;
        }
      }
    }
    cluster_wait();
  } else if ((warp & 3) < p.act_warps) {
    // ================================================================ softmax / output
    // (a warp whose 32 rows no tile has takes no part: its lanes of S and O hold anything)
    const int wg = warp >> 2, quarter = warp & 3;   // chunks wg, wg + 2, ...; TMEM lanes
    const int hrow = threadIdx.x & 127;             // TMEM lane = row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = p.scale_log2;
    const int H = p.a.H;
    const uint32_t peer = rank ^ 1u;
    // this CTA's dims of the row of Q, packed bf16 pairs, into the thread's TMEM lane
    auto load_q = [&](int item) {
      int rows;
      const long long r0 = rows_of<SHARED>(p, tail, item, rows);
      const bool in = hrow < rows;
      const uint4* src = reinterpret_cast<const uint4*>(p.a.Q + (in ? r0 + hrow : 0) * kD);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      // 96 dims at a time, so that enough loads are on their way: a row is a line of its own to
      // every lane
#pragma unroll
      for (int t = 0; t < kSteps / 6; ++t) {
        uint4 x[12];
#pragma unroll
        for (int q = 0; q < 12; ++q) {
          const int i = 12 * t + q;   // of this CTA's 16-byte pieces of the row
          const int at = i < kHalf / 8 ? rank * (kHalf / 8) + i
                                       : kDc / 8 + rank * (kHalfR / 8) + i - kHalf / 8;
          x[q] = in ? __ldg(src + at) : zero;
        }
#pragma unroll
        for (int a = 0; a < 3; ++a) {
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v = x[4 * a + q];
            if (FP8 && 12 * t + 4 * a + q < kHalf / 8)   // the middle two of four dims swapped
              v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                             __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
            w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
          }
          tmem_st_x16(tmem + lane_off + kColQ + (3 * t + a) * 16, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&tail->q_full);
    };

    if (wg == 0) load_q(item0);
    cluster_wait();   // the peer is ready to receive
    const uint32_t sbase = tmem + lane_off + kColS + wg * kNK;
    const uint32_t xb = smem_u32(smem + kExchOff + wg * kExch) + hrow * 16;
    const uint32_t x_dst = peer_addr(xb, peer);
    const uint32_t x_bar = peer_addr(smem_u32(&tail->x_full[wg][quarter]), peer);
    const uint32_t x_ack = peer_addr(smem_u32(&tail->x_free[wg][quarter]), peer);
    constexpr int c1 = FP8 ? 2 : 1, c2nd = 3 - c1;   // O's columns of the middle two of four dims
    const float4* xr = reinterpret_cast<const float4*>(smem + kExchOff + wg * kExch) + hrow;
    // P: this row's 32 bytes of each k-step's tile, 32B-swizzled
    uint8_t* prow_s = smem + kPOff + wg * kPBuf + hrow * 32;
    const int psw = ((hrow >> 2) & 1) << 4;

    float m = -INFINITY, l = 0.f;   // the running max last seen (raw logits), own chunks' sum
    int rows = 0, lim = 0, cur = -1;
    long long r0 = 0;
    for (int g = wg; g < n; g += 2) {
      const int st = g % kStages;
      const uint32_t par = (g >> 1) & 1;
      if (lane == 0) mbar_arrive_expect_tx(&tail->x_full[wg][quarter], 32 * kNK * 4);
      // what does not wait for S first: the header (the gather warps' writes), and the peer has read
      // what was sent two chunks ago
      bool ok = mbar_wait(&tail->kv_full[st], (g / kStages) & 1, abort_flag, err, kErrTime);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Header& h = tail->hdr[st];
      const int item = h.item, flags = h.cf & 15, c = h.cf >> 4;
      unsigned long long vm =
          h.valid[0] | static_cast<unsigned long long>(h.valid[1] & 0xffffu) << 32;
      if (item != cur) {
        cur = item;
        m = -INFINITY;
        l = 0.f;
        r0 = rows_of<SHARED>(p, tail, item, rows);
        // keys that this row sees: the tile's first token sees lim0, each later one one more
        if (SHARED || !p.a.idx) lim = h.lim0 + (static_cast<int>(r0 % H) + hrow) / H;
      }
      if (SHARED ? h.lim0 != kAllSee : !p.a.idx) {
        const int left = lim - c * kNK;   // keys of the chunk that the row sees
        if (left < kNK) vm = left <= 0 ? 0ull : vm & ((1ull << left) - 1);
      }
      ok = wait_peer(&tail->x_free[wg][quarter], par ^ 1u, abort_flag, err);
      ok = ok && mbar_wait(&tail->s_full[wg], par, abort_flag, err, kErrTime);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float2 s[kNK / 2];
      uint32_t lo[32], hi[16];
      tmem_ld_x32(sbase, lo);
      tmem_ld_16(sbase + 32, hi);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&tail->s_free[wg]);
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        st_peer(x_dst + j * 512, x_bar, lo[j], lo[j + 1], lo[j + 2], lo[j + 3]);
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        st_peer(x_dst + (32 + j) * 512, x_bar, hi[j], hi[j + 1], hi[j + 2], hi[j + 3]);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        s[j] = make_float2(__uint_as_float(lo[2 * j]), __uint_as_float(lo[2 * j + 1]));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s[16 + j] = make_float2(__uint_as_float(hi[2 * j]), __uint_as_float(hi[2 * j + 1]));
      // while the peer's half is on its way: the chunk before has settled the running maximum, and
      // the P buffer's previous chunk has gone through the tensor cores
      ok = g == 0 || mbar_wait(&tail->turn[wg ^ 1][quarter], ((g - 1) >> 1) & 1, abort_flag, err,
                               kErrTime);
      if (g >= 2) ok = ok && mbar_wait(&tail->pv_done[wg], par ^ 1u, abort_flag, err, kErrTime);
      ok = ok && wait_peer(&tail->x_full[wg][quarter], par, abort_flag, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float mr = (flags & 1) ? -INFINITY : tail->mref[hrow];
#pragma unroll
      for (int j = 0; j < kNK / 4; ++j) {
        const float4 x = xr[j * 128];
        s[2 * j] = add2(s[2 * j], make_float2(x.x, x.y));
        s[2 * j + 1] = add2(s[2 * j + 1], make_float2(x.z, x.w));
      }
      if (vm != (1ull << kNK) - 1) {
#pragma unroll
        for (int j = 0; j < kNK / 2; ++j) {
          s[j].x = ((vm >> (2 * j)) & 1u) ? s[j].x : -INFINITY;
          s[j].y = ((vm >> (2 * j + 1)) & 1u) ? s[j].y : -INFINITY;
        }
      }
      float m4[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) m4[j] = fmaxf(s[j].x, s[j].y);
#pragma unroll
      for (int j = 4; j < kNK / 2; ++j) m4[j & 3] = max3(m4[j & 3], s[j].x, s[j].y);
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      arrive_peer(x_ack, mx, lane);

      // in the order of the chunks: the running maximum
      float mn = mx;
      if (!(flags & 1)) {
        mn = mr;
        if (__any_sync(0xffffffffu,
                       mx > mr && (mr == -INFINITY || (mx - mr) * c2 > kRescaleLog2))) {
          // refresh the warp's running maxima: rescale O (once every earlier P V is done)
          const int pg = g - 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->pv_done[pg & 1], (pg >> 1) & 1,
                                                 abort_flag, err, kErrTime)))
            break;
          tc_fence_after();
          mn = fmaxf(mr, mx);
          const float f = mr == -INFINITY ? 0.f : exp2f((mr - mn) * c2);
#pragma unroll 1
          for (int d0 = 0; d0 < kHalf; d0 += 16) {
            uint32_t ov[16];
            tmem_ld_16(tmem + lane_off + kColO + d0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * f);
            tmem_st_x16(tmem + lane_off + kColO + d0, ov);
          }
          tmem_st_wait();
        }
      }
      tail->mref[hrow] = mn;
      float other = 0.f;
      if ((flags & 3) == 2) {
        // the tile ends here: the other warps' sum, from their chunk before this one (scaled by
        // the maximum of then, mr). It is awaited before the turn passes on, since their next
        // chunk takes the barrier further.
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->p_full[wg ^ 1], ((g - 1) >> 1) & 1,
                                               abort_flag, err, kErrTime)))
          break;
        other = tail->lsum[wg ^ 1][((g - 1) >> 1) & 1][hrow];
        if (mr != -INFINITY) other *= exp2f((mr - mn) * c2);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->turn[wg][quarter]);
      if (m != mn) {
        l *= m == -INFINITY ? 0.f : exp2f((m - mn) * c2);
        m = mn;
      }
      // P = exp2((S - m) c2) over the valid keys (exp2(-inf) = 0 elsewhere). The difference comes
      // first: S c2 and m c2 by themselves may be past fp32, and far from zero their own roundings
      // would move P. For its product with the rows, which are bf16, P is rounded to bf16 too: half a
      // step of 2^-8 at most, of either sign from key to key. Its sum l, and so lse, takes it unrounded.
      const float base = m == -INFINITY ? 0.f : m;
      const float2 cc = make_float2(c2, c2), bb = make_float2(-base, -base);
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int t = 0; t < kNK / 16; ++t) {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2 e = mul2(add2(s[t * 8 + j], bb), cc);
          e.x = ex2f(e.x);
          e.y = ex2f(e.y);
          ls[j & 1] = add2(ls[j & 1], e);
          pk[j] = pack_bf16(e.x, e.y);
        }
        uint8_t* dst = prow_s + t * kPTile;
        *reinterpret_cast<uint4*>(dst + psw) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(dst + (psw ^ 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
      l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      tail->lsum[wg][par][hrow] = l;
      l += other;
      if (p.a.Sq > 1 && (SHARED ? h.lim0 != kAllSee : !p.a.idx) && h.lim0 - c * kNK < kNK) {
        // Keys that the tile's later tokens see and its earlier ones do not: an infinity or a NaN in
        // one would go through the earlier ones' weight of zero. S has been worked out, and a token
        // that sees the key has it in its logit; in V it is dropped. (Here, where few registers are
        // in use: in front of the loads of S it took four long e4m3 sequences from 218 to 237 us,
        // here to 220; bf16 is level.)
        const int from = h.lim0 - c * kNK;
        drop_non_finite(smem + st * kStage, max(0, from),
                        min(kNK, from + (static_cast<int>(r0 % H) + rows - 1) / H), hrow,
                        32 * p.act_warps);
      }
      fence_proxy_async_smem();
      mbar_arrive(&tail->p_full[wg]);
      // The next tile's Q replaces this one's once the last S of this one is done. The warps of
      // the chunk before the last load it, since those of the last have the output to write.
      if ((flags & 8) && g + 2 < n) {
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->s_full[wg ^ 1], ((g + 1) >> 1) & 1, abort_flag,
                                               err, kErrTime)))
          break;
        tc_fence_after();
        load_q(item + 1);
      }
      if (!(flags & 2)) continue;

      if ((flags & 1) && g + 1 < n) load_q(item + 1);   // the tile's only chunk here
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&tail->pv_done[wg], par, abort_flag, err, kErrTime)))
        break;
      tc_fence_after();
      const long long row = r0 + hrow;
      if (!SHARED && (flags & 4)) {
        const float inv = l == 0.f ? 0.f : 1.f / l;   // NaN stays NaN
        uint4* out = reinterpret_cast<uint4*>(p.a.O + row * kDc + rank * kHalf);
#pragma unroll 1
        for (int d0 = 0; d0 < kHalf; d0 += 32) {
          uint32_t ov[32];
          tmem_ld_x32(tmem + lane_off + kColO + d0, ov);
          tmem_ld_wait();
          if (hrow < rows) {
#pragma unroll
            for (int d = 0; d < 32; d += 8) {
              uint4 w;
              w.x = pack_bf16(__uint_as_float(ov[d]) * inv, __uint_as_float(ov[d + c1]) * inv);
              w.y = pack_bf16(__uint_as_float(ov[d + c2nd]) * inv, __uint_as_float(ov[d + 3]) * inv);
              w.z = pack_bf16(__uint_as_float(ov[d + 4]) * inv, __uint_as_float(ov[d + 4 + c1]) * inv);
              w.w = pack_bf16(__uint_as_float(ov[d + 4 + c2nd]) * inv,
                              __uint_as_float(ov[d + 7]) * inv);
              out[(d0 + d) / 8] = w;
            }
          }
        }
        if (rank == 0 && hrow < rows)
          p.a.lse[row] = lse_of(p, m, l);
      } else {
        // part 0 of this cluster: a tile begun before its range; part 1: one that goes on behind
        const int part = SHARED ? item + cluster : 2 * cluster + (item == item0 && c0 > 0 ? 0 : 1);
        float4* out = p.part + static_cast<long long>(part) * (kDc / 4) * p.prow +
                      static_cast<long long>(rank * (kHalf / 4)) * p.prow + hrow;
        // (a warp's rows go out together, and of a tile of few rows the first warps alone)
#pragma unroll 1
        for (int d0 = SHARED && quarter * 32 >= rows ? kHalf : 0; d0 < kHalf; d0 += 32) {
          uint32_t ov[32];
          tmem_ld_x32(tmem + lane_off + kColO + d0, ov);
          tmem_ld_wait();
#pragma unroll
          for (int d = 0; d < 32; d += 4)
            out[static_cast<long long>((d0 + d) / 4) * p.prow] =
                make_float4(__uint_as_float(ov[d]), __uint_as_float(ov[d + c1]),
                            __uint_as_float(ov[d + c2nd]), __uint_as_float(ov[d + 3]));
        }
        if (rank == 0)
          p.ml[static_cast<long long>(part) * p.prow + hrow] = make_float2(m, l);
      }
      tc_fence_before();
      mbar_arrive(&tail->o_free);
    }
    if (*abort_flag) {
      // what this thread has sent to the peer lands before the cluster ends
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000ull) {
      }
    }
  } else {
    cluster_wait();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
  cluster_arrive();
  cluster_wait();   // no CTA leaves while its peer may still write to it
}

// Joins the parts of a tile that several clusters worked on: block (c, y, z) the tile that begins
// in cluster c's range and goes on behind it, rows [32 y, 32 y + 32), one per lane. With few parts
// a tile each warp takes 16 of the block's 128 dims. With many (SHARE: a single long sequence has
// one per cluster) a block has 16 dims and its warps share the parts, since one after the other
// their latencies took longer than the attention itself: 32768 keys 39 us instead of 66. The
// other way round 75 tiles of two parts take 30 us longer shared.
constexpr int kJoinWarps = 8, kJoinD4 = 4;   // warps of a block, groups of four dims of a warp
template <bool SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps) latent_join_kernel(const Params p) {
  __shared__ float2 ml[kMaxClusters][32];
  __shared__ float4 acc[SHARE ? kJoinWarps : 1][kJoinD4][33];
  __shared__ float sum[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 tile = __ldcg(p.joins + blockIdx.x);
  const int first = blockIdx.x, parts = tile.y - first + 1;
  // nothing to join, or not written: a cluster whose waits ran out (recorded) leaves what was there
  if (tile.x < 0 || tile.x >= p.items || tile.y <= first || tile.y >= p.clusters) return;
  int rows;
  long long r0 = rows_of<false>(p, nullptr, tile.x, rows);
  rows -= blockIdx.y * 32;   // left from this block's first on
  r0 += blockIdx.y * 32;
  if (rows <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * 32 + lane;
  // part 1 of the first cluster, part 0 of the others
  auto part_of = [&](int i) { return static_cast<long long>(2 * (first + i) + (i == 0)); };
  for (int i = warp; i < parts; i += kJoinWarps)
    ml[i][lane] = __ldcg(p.ml + part_of(i) * p.prow + row);
  __syncthreads();
  float top = -INFINITY, l = 0.f;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, ml[i][lane].x);
  // a part without a key has m = -inf, l = 0 and O = 0; one with a NaN keeps it in l
  auto weight = [&](float2 q) {
    return q.x == -INFINITY ? (q.y == 0.f ? 0.f : 1.f) : exp2f((q.x - top) * p.scale_log2);
  };
  const int d4 = SHARE ? blockIdx.z * kJoinD4 : (blockIdx.z * kJoinWarps + warp) * kJoinD4;
  float4 o[kJoinD4];
#pragma unroll
  for (int d = 0; d < kJoinD4; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = SHARE ? warp : 0; i < parts; i += SHARE ? kJoinWarps : 1) {
    const float4* src = p.part + (part_of(i) * (kDc / 4) + d4) * p.prow + row;
    float4 x[kJoinD4];
#pragma unroll
    for (int d = 0; d < kJoinD4; ++d) x[d] = __ldcg(src + d * p.prow);
    const float w = weight(ml[i][lane]);
#pragma unroll
    for (int d = 0; d < kJoinD4; ++d) {
      o[d].x += w * x[d].x;
      o[d].y += w * x[d].y;
      o[d].z += w * x[d].z;
      o[d].w += w * x[d].w;
    }
  }
  if (!SHARE || warp == 0)
    for (int i = 0; i < parts; ++i) l += weight(ml[i][lane]) * ml[i][lane].y;
  if (blockIdx.z == 0 && warp == 0 && lane < rows)
    p.a.lse[r0 + lane] = lse_of(p, top, l);
  auto pack4 = [](float4 v, float inv) {
    return make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  };
  if (!SHARE) {
    if (lane >= rows) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint4* out = reinterpret_cast<uint4*>(p.a.O + (r0 + lane) * kDc + d4 * 4);
#pragma unroll
    for (int d = 0; d < kJoinD4; d += 2) {
      const uint2 a = pack4(o[d], inv), b = pack4(o[d + 1], inv);
      out[d / 2] = make_uint4(a.x, a.y, b.x, b.y);
    }
    return;
  }
  if (warp == 0) sum[lane] = l;
#pragma unroll
  for (int d = 0; d < kJoinD4; ++d) acc[SHARE ? warp : 0][d][lane] = o[d];
  __syncthreads();
  // four threads per row, four dims each
  const int out_row = threadIdx.x / kJoinD4, d = threadIdx.x % kJoinD4;
  if (out_row >= min(rows, 32)) return;
  float4 v = acc[0][d][out_row];
#pragma unroll
  for (int w = 1; w < (SHARE ? kJoinWarps : 1); ++w) {
    const float4 x = acc[w][d][out_row];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  *reinterpret_cast<uint2*>(p.a.O + (r0 + out_row) * kDc + (d4 + d) * 4) =
      pack4(v, sum[out_row] == 0.f ? 0.f : 1.f / sum[out_row]);
}

// The join of shared prefixes: block (x, y, z) rows [32 y, 32 y + 32) of a sequence's own tile x, one
// per lane. A row's parts are those of its own tile and those of the tile of its group's rows that it
// is in; the warps share the dims or the parts, as above.
template <bool SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps) shared_join_kernel(const Params p) {
  __shared__ __align__(16) uint8_t buffer[2 * kMaxClusters * 32 * sizeof(float2)];
  float2(*ml)[32] = reinterpret_cast<float2(*)[32]>(buffer);
  // the warps' sums, in the same place later
  float4(*acc)[kJoinD4][33] = reinterpret_cast<float4(*)[kJoinD4][33]>(buffer);
  static_assert(sizeof(float4[kJoinWarps][kJoinD4][33]) <= sizeof(buffer), "they fit");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.a.G;
  const int b = blockIdx.x / p.tiles, mt = blockIdx.x - b * p.tiles;
  const int at = blockIdx.y * 32 + lane;   // row of the tile
  if (static_cast<int>(blockIdx.y) * 32 >= tile_rows(p, mt)) return;
  const bool in = at < tile_rows(p, mt);
  const int per = p.a.Sq * p.a.H, row = mt * 128 + at;
  // a token that has no place in its sequence (padding) has no key
  const bool there = in && seq_len(p.a, b, false) - p.a.Sq + row / p.a.H >= 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* gstart = p.groups;
  const int* gtile = p.groups + kMaxGroups + 1;
  int g = 0;   // groups that end at or in front of b: the starts go up
#pragma unroll
  for (int i = 0; i < kMaxGroups; i += 32)
    g += __popc(__ballot_sync(0xffffffffu, i + lane < G && b >= __ldcg(gstart + i + lane + 1)));
  const int prefix_tiles = __ldcg(gtile + G);
  // parts first[k] + i, i < n[k], at row where[k] of each: k = 0 the prefix's, k = 1 the own keys'
  int first[2] = {0, 0}, n[2] = {0, 0}, where[2] = {0, at};
  auto find = [&](int k, int item) {
    if (item < 0 || item >= p.most_items) return;
    const int2 s = __ldcg(p.spans + item);
    // not written: a cluster whose waits ran out (recorded)
    if (s.x < 0 || s.y < s.x || s.y >= p.clusters) return;
    first[k] = item + s.x;
    n[k] = s.y - s.x + 1;
  };
  if (there) {
    find(1, prefix_tiles + blockIdx.x);
    if (g < G && b >= __ldcg(gstart + g) && __ldcg(gtile + g + 1) > __ldcg(gtile + g)) {
      const int off = (b - __ldcg(gstart + g)) * per + row;
      where[0] = off & 127;
      find(0, __ldcg(gtile + g) + (off >> 7));
    }
  }
  const int parts = n[0] + n[1];
  const int most = __reduce_max_sync(0xffffffffu, parts);
  auto part_of = [&](int i) {
    return static_cast<long long>(i < n[0] ? first[0] + i : first[1] + i - n[0]);
  };
  for (int i = warp; i < most; i += kJoinWarps)
    if (i < parts) ml[i][lane] = __ldcg(p.ml + part_of(i) * p.prow + where[i >= n[0]]);
  __syncthreads();
  float top = -INFINITY, l = 0.f;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, ml[i][lane].x);
  // a part without a key has m = -inf, l = 0 and O = 0; one with a NaN keeps it in l
  auto weight = [&](float2 q) {
    return q.x == -INFINITY ? (q.y == 0.f ? 0.f : 1.f) : exp2f((q.x - top) * p.scale_log2);
  };
  const int d4 = SHARE ? blockIdx.z * kJoinD4 : (blockIdx.z * kJoinWarps + warp) * kJoinD4;
  float4 o[kJoinD4];
#pragma unroll
  for (int d = 0; d < kJoinD4; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = SHARE ? warp : 0; i < parts; i += SHARE ? kJoinWarps : 1) {
    const float4* src = p.part + (part_of(i) * (kDc / 4) + d4) * p.prow + where[i >= n[0]];
    float4 x[kJoinD4];
#pragma unroll
    for (int d = 0; d < kJoinD4; ++d) x[d] = __ldcg(src + d * p.prow);
    const float w = weight(ml[i][lane]);
#pragma unroll
    for (int d = 0; d < kJoinD4; ++d) {
      o[d].x += w * x[d].x;
      o[d].y += w * x[d].y;
      o[d].z += w * x[d].z;
      o[d].w += w * x[d].w;
    }
  }
  for (int i = 0; i < parts; ++i) l += weight(ml[i][lane]) * ml[i][lane].y;
  const long long out_row = static_cast<long long>(b) * per + row;
  if (blockIdx.z == 0 && warp == 0 && in) p.a.lse[out_row] = lse_of(p, top, l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  auto pack4 = [](float4 v, float inv) {
    return make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  };
  if (!SHARE) {
    if (!in) return;
    uint4* out = reinterpret_cast<uint4*>(p.a.O + out_row * kDc + d4 * 4);
#pragma unroll
    for (int d = 0; d < kJoinD4; d += 2) {
      const uint2 a = pack4(o[d], inv), b = pack4(o[d + 1], inv);
      out[d / 2] = make_uint4(a.x, a.y, b.x, b.y);
    }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int d = 0; d < kJoinD4; ++d) acc[warp][d][lane] = o[d];
  __syncthreads();
  if (warp >= kJoinD4 || !in) return;   // warp d: four dims of the lane's row
  float4 v = acc[0][warp][lane];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 x = acc[w][warp][lane];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  *reinterpret_cast<uint2*>(p.a.O + out_row * kDc + (d4 + warp) * 4) = pack4(v, inv);
}

int part_rows(int Sq, int H, int k) {
  const long long rows = k > 0 ? H : static_cast<long long>(Sq) * H;
  return static_cast<int>(rows < 128 ? (rows + 31) / 32 * 32 : 128);
}

// Clusters of the kernel that fit on the current device at once; the first call on a device also
// raises the kernel's shared-memory limit there.
template <bool FP8, bool SHARED>
int resident_clusters(size_t smem) {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices] = {};
  static std::mutex lock;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> guard(lock);
  if (known[dev] == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (cudaFuncSetAttribute(latent_attn_kernel<FP8, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return 0;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, latent_attn_kernel<FP8, SHARED>, &cfg) != cudaSuccess || c < 1)
      return 0;
    known[dev] = c < kMaxClusters ? c : kMaxClusters;
  }
  return known[dev];
}

template <bool FP8>
int launch(Params p, cudaStream_t stream) {
  constexpr bool SHARED = false;
  const size_t smem = Layout<FP8>::kTailOff + sizeof(Tail);
  p.clusters = resident_clusters<FP8, SHARED>(smem);
  if (p.clusters < 1) return DSA_ERR_CUDA;
  // no more clusters than the longest possible sequences have work for
  const long long cap = static_cast<long long>(p.a.max_pages) * p.a.page_size;
  const long long most = p.a.idx ? p.list_chunks : (cap + kNK - 1) / kNK;
  const long long wanted = (p.items * most + kMinChunks - 1) / kMinChunks;
  if (wanted < p.clusters) p.clusters = static_cast<int>(wanted);
  p.ml = reinterpret_cast<float2*>(p.part + 2ll * p.clusters * (kDc / 4) * p.prow);
  p.joins = reinterpret_cast<int2*>(p.ml + 2ll * p.clusters * p.prow);
  latent_attn_kernel<FP8, SHARED><<<2 * p.clusters, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (p.clusters == 1) return DSA_OK;   // nothing is split
  // its blocks may be set up while the last clusters finish; they wait for the parts
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // shared while the tiles' blocks (32 for 32 rows) all fit on the SMs at once, six on each: eight
  // sequences of 500 keys and 128 heads take 25 us unshared, 31 shared
  const bool share = static_cast<long long>(p.items) * p.prow <= 152 * 6;
  cfg.gridDim = dim3(p.clusters - 1, p.prow / 32, kDc / (4 * kJoinD4) / (share ? 1 : kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, share ? latent_join_kernel<true> : latent_join_kernel<false>,
                            p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

// tiles of the groups' rows that there can be: each group's rows are rounded up
long long most_prefix_tiles(int B, int Sq, int H, int G) {
  return static_cast<long long>(B) * Sq * H / 128 + (G < B ? G : B);
}

template <bool FP8>
int launch_shared(Params p, cudaStream_t stream) {
  const size_t smem = Layout<FP8>::kTailOff + sizeof(Tail);
  p.clusters = resident_clusters<FP8, true>(smem);
  if (p.clusters < 1) return DSA_ERR_CUDA;
  // no more clusters than the longest possible sequences and prefixes have work for
  const long long own = (static_cast<long long>(p.a.max_pages) * p.a.page_size + kNK - 1) / kNK;
  const long long pre = (static_cast<long long>(p.a.max_prefix) * p.a.page_size + kNK - 1) / kNK;
  const long long wanted =
      (p.items * own + (p.most_items - p.items) * pre + kMinChunks - 1) / kMinChunks;
  if (wanted < p.clusters) p.clusters = static_cast<int>(wanted);
  const long long parts = static_cast<long long>(p.most_items) + kMaxClusters;
  p.ml = reinterpret_cast<float2*>(p.part + parts * (kDc / 4) * p.prow);
  p.spans = reinterpret_cast<int2*>(p.ml + parts * p.prow);
  p.groups = reinterpret_cast<int*>(p.spans + p.most_items);
  latent_attn_kernel<FP8, true><<<2 * p.clusters, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  // its blocks may be set up while the last clusters finish; they wait for the parts
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int rows = part_rows(p.a.Sq, p.a.H, 0);   // of the largest own tile
  const bool share = static_cast<long long>(p.items) * rows <= 152 * 6;
  cfg.gridDim = dim3(p.items, rows / 32, kDc / (4 * kJoinD4) / (share ? 1 : kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, share ? shared_join_kernel<true> : shared_join_kernel<false>,
                            p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace

size_t latent_attn_workspace(int B, int Sq, int H, int k) {
  (void)B;
  const size_t rows = static_cast<size_t>(part_rows(Sq, H, k));
  return 2ull * kMaxClusters * rows * (kDc * sizeof(float) + sizeof(float2)) +
         kMaxClusters * sizeof(int2);
}

int launch_latent_attn(const LatentArgs& a, int fmt, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.tiles = static_cast<int>((static_cast<long long>(a.Sq) * a.H + 127) / 128);
  const long long items = a.idx ? static_cast<long long>(a.B) * a.Sq
                                : static_cast<long long>(a.B) * p.tiles;
  p.items = static_cast<int>(items);   // at most B * Sq * H < 2^31
  p.list_chunks = a.idx ? (a.k - 1) / kNK + 1 : 0;
  p.prow = part_rows(a.Sq, a.H, a.k);
  p.act_warps = p.prow / 32;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.part = static_cast<float4*>(a.ws);
  return fmt == DSA_CACHE_E4M3 ? launch<true>(p, stream) : launch<false>(p, stream);
}

size_t latent_attn_shared_workspace(int B, int Sq, int H, int G) {
  const long long rows = static_cast<long long>(B) * Sq * H;
  const long long tiles = (static_cast<long long>(Sq) * H + 127) / 128;
  const size_t items = static_cast<size_t>(most_prefix_tiles(B, Sq, H, G) + B * tiles);
  const size_t prow = rows < 128 ? (rows + 31) / 32 * 32 : 128;
  return (items + kMaxClusters) * prow * (kDc * sizeof(float) + sizeof(float2)) +
         items * sizeof(int2) + 2 * (kMaxGroups + 1) * sizeof(int);
}

int launch_latent_attn_shared(const LatentArgs& a, int fmt, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.tiles = static_cast<int>((static_cast<long long>(a.Sq) * a.H + 127) / 128);
  const long long items = static_cast<long long>(a.B) * p.tiles;
  const long long most = items + most_prefix_tiles(a.B, a.Sq, a.H, a.G);
  p.items = static_cast<int>(items);   // at most B * Sq * H
  p.most_items = static_cast<int>(most);
  const long long rows = static_cast<long long>(a.B) * a.Sq * a.H;
  p.prow = rows < 128 ? static_cast<int>((rows + 31) / 32 * 32) : 128;
  p.act_warps = p.prow / 32;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.part = static_cast<float4*>(a.ws);
  return fmt == DSA_CACHE_E4M3 ? launch_shared<true>(p, stream) : launch_shared<false>(p, stream);
}

}  // namespace dsa
