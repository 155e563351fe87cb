// The attention weight that each cached position receives from the newest tokens (dsa_cache_mass), on
// the 5th-generation tensor cores.
//
//   mass[j] = decay prev[j] + sum over tokens i and heads h that see j of exp(scale q_ih . row_j - lse_ih)
//
// with lse from the attention itself, so that one more product of queries and rows is all it takes. The
// keys are the lanes of a tile and the (token, head) pairs its columns, so that a key's sum over
// tokens and heads stays within one thread:
//
//   S [256 keys x 128 pairs] = K [256 x 576] . Q^T,   sum_c exp(scale S_c - lse_c)
//
// A tile is the pair instruction's (cta_group::2): each CTA of a cluster of two has 128 of the keys and
// half of the pairs' rows in its shared memory, so that a query's row is fetched once for 256 keys and
// takes half the room. Both operands go through shared memory in atoms of 64 dims. Up to 128 pairs a
// sequence (a token with a list always is): Q stays, the rows stream through a ring, and memory is the
// bound. More pairs: a tile's rows stay and the pairs stream past them, 128 at a time; the tensor cores
// are the bound. The work, tiles or (tile, 128 pairs), is cut into one even range per cluster whatever
// the lengths. A tile whose pairs lie in several ranges leaves a part in each, which
// join_kernel adds up in order. Lengths are read on the device only.
//
// The tensor cores cut off, not round, what an addition moves behind the last bit, always towards zero.
// Over all 576 dims that would move a weight by 1.5e-6 of itself; so the first five atoms and the
// last four have an accumulator each (7e-7), added up in the epilogue.
//
// Warp-specialised CTA, 896 threads:
//   warps 0-7    epilogue, one key per thread: warps 0-3 the first 64 pairs, 4-7 the others
//   warp 8       in the first CTA the single-thread UMMA issuer; owns TMEM: two buffers of two
//                accumulators of 128 columns
//   warp 9       Q by TMA
//   warp 10      the pairs' lse and limits, a unit ahead
//   warps 12-27  rows, a quarter of a key's atom per thread: cp.async, bf16 into the operand's place, e4m3
//                into a ring of raw atoms, then widened to bf16, exactly

// Measured (device time): 32 sequences of 256 to 8192 rows, 128 heads: bf16 33 us (4.9 TB/s; 6.3 in
// steady state, the rest is the start of a launch and the last round of tiles), e4m3 33 us (2.9 TB/s); 32
// tokens over 2 x 16384 rows, bf16 131 us (1180 TFLOP/s), e4m3 135. What bounds it: bf16 memory; e4m3 no unit
// but the chain between them: of about 8300 cycles a tile the products take 2304, the rows' way from memory
// about 3900, what goes through shared memory (raw codes in and out, bf16 in, the products' reads) about 4000
// at 128 bytes a cycle, and the issuer waits 1800 to 2600 for rows, whose ring of two groups ties the gather
// to the products (without the copies, the widening, the fence or most of the epilogue the batch takes
// 31.0, 31.7, 32.7 or 31.6 us); many pairs the products, 36 of 256 x 128 x 16 at 64 cycles of about 4300 a
// unit, beside which one thread waits and commits and which take the 128 bytes a cycle of shared memory too,
// and the epilogue, whose steps of eight columns each wait for TMEM (with an eighth of them 118 us).

#include <mutex>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "latent_row.cuh"
#include "tensor_map.h"

namespace dsa {
namespace {

constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kKeys = 128, kTile = 2 * kKeys;   // keys of a CTA and of a tile
constexpr int kPairs = 128;              // pairs at a time
constexpr int kAtoms = kD / 64;
constexpr int kGroup = 3, kGroups = kAtoms / kGroup;   // atoms that are handed over together
constexpr int kFirstAtoms = 5;           // atoms of the first accumulator
constexpr uint32_t kKeyAtom = kKeys * 128, kQueryAtom = kPairs / 2 * 128;
constexpr uint32_t kRawAtom = kKeys * 64;   // of codes; one of positional dims is two
constexpr int kRawSteps = 10;            // raw atoms of a tile: eight of codes, two of positional dims
constexpr int kEpilogueWarps = 8;
constexpr int kIssueWarp = 8, kQueryWarp = 9, kStageWarp = 10, kGatherWarp0 = 12, kGatherWarps = 16;
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);
constexpr int kMaxClusters = 128;
constexpr int kErrIdx = DSA_STAGE_EVICT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_EVICT | DSA_DEVERR_BAD_PAGE;
constexpr int kErrTime = DSA_STAGE_EVICT | DSA_DEVERR_TIMEOUT;
static_assert(kGatherThreads == 4 * kKeys, "a quarter of a key's atom per thread");

// 224 KB in 28 pieces of 8 KB: groups of atoms of rows, groups of atoms of Q, raw atoms
template <bool FP8, bool MULTI>
struct Layout {
  static constexpr int kKeySlots = MULTI || !FP8 ? kGroups : 2;
  static constexpr int kQuerySlots = MULTI && FP8 ? 2 : kGroups;
  static constexpr int kRawSlots = FP8 ? (MULTI ? 4 : 7) : 0;
  static constexpr uint32_t kQueryOff = kKeySlots * kGroup * kKeyAtom;
  static constexpr uint32_t kRawOff = kQueryOff + kQuerySlots * kGroup * kQueryAtom;
  static constexpr uint32_t kTailOff = kRawOff + kRawSlots * kRawAtom;
};

// Columns of the product for so many pairs: half of them are rows in each CTA. A multiple of 32, which the
// pair instruction takes at 256 rows without doubt: whether steps of 16 are among its shapes there, the
// descriptions that are known disagree. (The columns behind the last pair cost nothing that shows: 32
// sequences of up to 8192 e4m3 rows with 16 / 48 / 80 / 112 heads 32.1 / 31.6 / 32.4 / 33.5 us, with steps
// of 16 32.5 / 31.5 / 32.4 / 33.6.)
constexpr int pair_columns(int pairs) { return pairs < kPairs ? (pairs + 31) / 32 * 32 : kPairs; }
constexpr bool shapes_are_sound() {
  for (int pairs = 1; pairs <= 2 * kPairs; ++pairs) {
    const int n = pair_columns(pairs);
    if (n % 32 != 0 || n < 32 || n > kPairs || (pairs <= kPairs && n < pairs)) return false;
  }
  return true;
}
static_assert(shapes_are_sound(), "columns of the pair instruction");

struct Tail {
  float nlse[2][kPairs];     // -lse of the pairs
  int lim[2][kPairs];        // positions below it are seen by the pair; a pair that adds nothing: none
  int group_lim[2][4];       // the least of 32 pairs
  uint32_t valid[3][kGatherWarps];   // the tile's keys that are there: four bits a key
  float other[kKeys];        // the sums of the second 64 pairs
  uint64_t k_full[kGroups], k_empty[kGroups], q_full[kGroups], q_empty[kGroups];
  uint64_t d_full[2], d_empty[2], valid_full[3], staged_full[2], staged_empty[2], other_full, other_empty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  // this cluster's range: its first item and the first unit of it here, and how many units
  int item0;
  long long first, count;
};
static_assert(Layout<true, true>::kTailOff + sizeof(Tail) <= 232448 &&
                  Layout<true, false>::kTailOff + sizeof(Tail) <= 232448 &&
                  Layout<false, true>::kTailOff + sizeof(Tail) <= 232448,
              "shared memory of a block");

struct Params {
  MassArgs a;
  int items;        // sequences, or tokens with a list each
  int nts;          // columns of 128 pairs
  int box;          // columns at a time (pair_columns), half of them in each CTA
  int page_shift;   // log2 of the page size, -1 where it is no power of two
  float* w;         // lists: the weight of each entry [B, Sq, k]
  float* part;      // [2 * clusters][256]
  int4* joins;      // [clusters]: (sequence, tile, last cluster that has a part of it) or (-1, ...)
};

__device__ __forceinline__ int seq_len(const MassArgs& a, int b, bool report) {
  const int cap = a.max_pages * a.page_size;
  const int len = __ldg(a.lens + b);
  if (report && (len < 0 || len > cap || len > a.n)) report_error(a.err, kErrPage);
  return max(0, min(len, cap));
}

__device__ __forceinline__ int item_tiles(const Params& p, int item) {
  const int keys = p.a.idx ? p.a.k : min(p.a.n, seq_len(p.a, item, false));
  return keys > 0 ? (keys - 1) / kTile + 1 : 0;
}

// this cluster's range of units, into the tail; every thread of the block calls it, before a barrier
template <bool MULTI>
__device__ __forceinline__ void my_units(const Params& p, Tail* tail) {
  const long long per_tile = MULTI ? p.nts : 1;
  long long* sums = reinterpret_cast<long long*>(tail->nlse);   // not in use yet
  long long total, before = 0, s = 0;
  int i0 = 0, i1 = 0;   // this thread's items
  if (p.a.idx) {
    total = static_cast<long long>(p.items) * item_tiles(p, 0);
  } else {
    const int q = (p.items + kThreads - 1) / kThreads;
    i0 = min(p.items, static_cast<int>(threadIdx.x) * q);
    i1 = min(p.items, i0 + q);
    for (int i = i0; i < i1; ++i) s += item_tiles(p, i) * per_tile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    before += incl - s;
  }
  const int clusters = gridDim.x >> 1, cluster = blockIdx.x >> 1;
  const long long each = (total + clusters - 1) / clusters;
  const long long u0 = min(total, each * cluster), u1 = min(total, u0 + each);
  if (u0 == u1) return;   // count stays 0
  if (p.a.idx) {
    if (threadIdx.x != 0) return;
    const int tiles = item_tiles(p, 0);
    tail->item0 = static_cast<int>(u0 / tiles);
    tail->first = u0 - static_cast<long long>(tail->item0) * tiles;
    tail->count = u1 - u0;
    return;
  }
  for (int i = i0; i < i1; ++i) {
    const long long m = item_tiles(p, i) * per_tile;
    if (u0 >= before && u0 < before + m) {
      tail->item0 = i;
      tail->first = u0 - before;
      tail->count = u1 - u0;
    }
    before += m;
  }
}

// where a warp stands in its cluster's range
template <bool MULTI>
struct Cursor {
  int item, tile, nt, tiles;
  __device__ __forceinline__ Cursor(const Params& p, const Tail* t) {
    item = t->item0;
    tiles = item_tiles(p, item);
    tile = static_cast<int>(MULTI ? t->first / p.nts : t->first);
    nt = MULTI ? static_cast<int>(t->first - static_cast<long long>(tile) * p.nts) : 0;
  }
  __device__ __forceinline__ void next_tile(const Params& p) {
    nt = 0;
    if (++tile < tiles) return;
    tile = 0;
    do {
      ++item;
      tiles = item < p.items ? item_tiles(p, item) : 1;
    } while (tiles == 0);
  }
  __device__ __forceinline__ void next(const Params& p) {
    if (!MULTI || ++nt == p.nts) next_tile(p);
  }
};

// ------------------------------------------------------------------ small helpers

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return r;
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the address of a barrier of the first CTA, from either
__device__ __forceinline__ uint32_t first_cta(const uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
// Arrives at a barrier of the first CTA, without a scope of its own: a release at cluster scope waits
// for all that the warp has on its way, copies too, and took 88 us instead of 44 (32 ragged e4m3
// sequences). What has to be in order here is in the writer's own SM, where the tensor cores read it:
// its shared memory, which fence.proxy.async has made theirs in front of this, or TMEM, read in front of
// tcgen05.wait::ld. Nothing that another thread reads by plain loads hangs on these barriers.
__device__ __forceinline__ void arrive_first_cta(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// tma_load_2d that counts on a barrier of the first CTA, from either
__device__ __forceinline__ void tma2_load_2d(void* dst, const void* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// The pair instruction: A is 128 rows of each CTA, B half of the columns of each, at the same places.
__device__ __forceinline__ void umma2_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on `bar` of both CTAs when every earlier tcgen05.mma of this thread has completed.
__device__ __forceinline__ void umma2_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// Waits for the last commit. It was issued behind all others, so that by then none of them has an arrival at
// this CTA's barriers left to make: no CTA may leave its shared memory in front of that. (Not mbar_wait: that
// gives up as soon as the block does.)
__device__ __forceinline__ void drain_wait(uint64_t* bar, int* err) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(smem_u32(bar), 0)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      report_error(err, kErrTime);
      break;
    }
  }
}

// the slot counter of a ring, and the parity to wait for
template <int N>
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      round ^= 1u;
    }
  }
};

// ------------------------------------------------------------------ the kernel

template <bool FP8, bool MULTI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mass_kernel(const Params p, const __grid_constant__ CUtensorMap qmap) {
  using L = Layout<FP8, MULTI>;
  constexpr int kKeySlots = L::kKeySlots, kQuerySlots = L::kQuerySlots;
  constexpr int kNone = -0x7fffffff - 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const qsmem = smem + L::kQueryOff;
  Tail* tail = reinterpret_cast<Tail*>(smem + L::kTailOff);
  volatile int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;
  const MassArgs& a = p.a;
  int* err = a.err;
  // the same in both CTAs of a cluster (one layout), so both leave
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) report_error(err, DSA_STAGE_EVICT | DSA_DEVERR_MISALIGNED);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&tail->k_full[i], 2 * kGatherWarps);   // of the first CTA: both CTAs' rows
      mbar_init(&tail->k_empty[i], 1);
      mbar_init(&tail->q_full[i], 1);                  // of the first CTA: both CTAs' halves
      mbar_init(&tail->q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->d_full[i], 1);
      mbar_init(&tail->d_empty[i], 2 * kEpilogueWarps);   // of the first CTA: both CTAs' epilogue warps
      mbar_init(&tail->staged_full[i], 1);
      mbar_init(&tail->staged_empty[i], kEpilogueWarps);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&tail->valid_full[i], kGatherWarps);
    mbar_init(&tail->other_full, 4);
    mbar_init(&tail->other_empty, 4);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    tail->count = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tail->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  my_units<MULTI>(p, tail);
  tc_fence_before();
  cluster_sync();   // and both CTAs' barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  const long long n = tail->count;   // the same in both CTAs

  const int pairs = a.idx ? a.H : a.Sq * a.H;   // of an item
  if (warp < kEpilogueWarps) {
    // ================================================================ epilogue
    if (!a.idx) {
      // zeros behind the sequences' ends, shared out among the CTAs
      for (int b = warp; b < a.B; b += kEpilogueWarps) {
        const int len = seq_len(a, b, blockIdx.x == 0 && lane == 0), end = min(len, a.n);
        const long long room = a.n - end;
        const int z0 = end + static_cast<int>(room * blockIdx.x / gridDim.x);
        const int z1 = end + static_cast<int>(room * (blockIdx.x + 1) / gridDim.x);
        for (int j = z0 + lane; j < z1; j += 32) a.mass[static_cast<long long>(b) * a.n + j] = 0.f;
      }
    }
    const int me = threadIdx.x & 127;    // TMEM lane
    const int half = warp >> 2;          // pairs 64 half, ...
    const int key = rank * kKeys + me;   // of the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 scale2 = make_float2(a.scale, a.scale);
    const float2 log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
    const uint32_t d_empty0 = first_cta(&tail->d_empty[0]);
    if (n > 0) {
      Cursor<MULTI> c(p, tail);
      int cur_item = -1, len = 0;
      float sum = 0.f;
      bool whole = false;        // the tile's first pairs were here
      Ring<3> vr;                // tiles whose flags have been taken
      Ring<2> sr;                // sets of lse and limits
      uint32_t done = 0;         // tiles that are done
      bool there = false;
#pragma unroll 1
      for (long long u = 0; u < n; ++u) {
        const int buf = static_cast<int>(u) & 1;
        const uint32_t par = static_cast<uint32_t>(u >> 1) & 1u;
        if (c.item != cur_item) {
          cur_item = c.item;
          len = seq_len(a, a.idx ? c.item / a.Sq : c.item, false);
        }
        bool ok = true;
        if (u == 0 || c.nt == 0) {
          sum = 0.f;
          whole = c.nt == 0;
          ok = mbar_wait(&tail->valid_full[vr.slot], vr.round, abort_flag, err, kErrTime);
        }
        // the earlier weight, on its way while the tile is
        float before = 0.f;
        if (half == 0 && a.prev && !a.idx && (!MULTI || c.nt == p.nts - 1) && c.tile * kTile + key < min(len, a.n))
          before = a.prev[static_cast<long long>(c.item) * a.n + c.tile * kTile + key];
        ok = ok && mbar_wait(&tail->staged_full[sr.slot], sr.round, abort_flag, err, kErrTime);
        ok = ok && mbar_wait(&tail->d_full[buf], par, abort_flag, err, kErrTime);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (u == 0 || c.nt == 0) {
          there = (tail->valid[vr.slot][me >> 3] >> (4 * (me & 7)) & 1u) != 0;
          vr.next();
        }
        const int j0 = c.tile * kTile;   // (below 2^31: n and k are)
        // lists: a key that its token does not see is not there
        const int last = a.idx ? kNone : min(j0 + (kTile - 1), len - 1) + 1;
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const uint32_t d = tmem + lane_off + buf * 2 * kPairs;
        // eight pairs at a time, the next ones on their way (sixteen would not fit the registers)
        const int c1 = min(64 * half + 64, pairs - c.nt * kPairs);
        uint32_t s0[8], s1[8];
        tmem_ld_8(d + half * 64, s0);
        tmem_ld_8(d + kPairs + half * 64, s1);
#pragma unroll 1
        for (int c0 = 64 * half; c0 < c1; c0 += 8) {
          tmem_ld_wait();
          float2 s[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            s[q] = add2(make_float2(__uint_as_float(s0[2 * q]), __uint_as_float(s0[2 * q + 1])),
                        make_float2(__uint_as_float(s1[2 * q]), __uint_as_float(s1[2 * q + 1])));
          const int next = (c0 + 8) & (kPairs - 1);   // (behind the last one: read, not used)
          tmem_ld_8(d + next, s0);
          tmem_ld_8(d + kPairs + next, s1);
          const float4* nl = reinterpret_cast<const float4*>(&tail->nlse[sr.slot][c0]);
          const int least = tail->group_lim[sr.slot][c0 >> 5];
          if (least != kNone && least >= last) {
            // every pair of the group sees every key of the tile
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 v = nl[q];
              // the difference first, in one rounding: far from zero those of the products with
              // log2(e) would move the weight
              float2 x = fma2(s[2 * q], scale2, make_float2(v.x, v.y));
              float2 y = fma2(s[2 * q + 1], scale2, make_float2(v.z, v.w));
              x = mul2(x, log2e);
              y = mul2(y, log2e);
              acc[0] = add2(acc[0], make_float2(ex2f(x.x), ex2f(x.y)));
              acc[1] = add2(acc[1], make_float2(ex2f(y.x), ex2f(y.y)));
            }
          } else {
            const int* lims = &tail->lim[sr.slot][c0];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float v = tail->nlse[sr.slot][c0 + q];
              const float x = ex2f(fmaf(q & 1 ? s[q / 2].y : s[q / 2].x, a.scale, v) * log2e.x);
              const bool sees = lims[q] != kNone && (a.idx || j0 + key < lims[q]);
              (q & 1 ? acc[0].y : acc[0].x) += sees ? x : 0.f;
            }
          }
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        const bool end = !MULTI || c.nt == p.nts - 1 || u == n - 1;   // of the tile, here
        if (lane == 0) {
          arrive_first_cta(d_empty0 + buf * 8);
          if (MULTI || u == n - 1 || c.tile == c.tiles - 1) mbar_arrive(&tail->staged_empty[sr.slot]);
        }
        if (MULTI || u == n - 1 || c.tile == c.tiles - 1) sr.next();
        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        if (end) {
          // the second half's sums go to the first half's threads
          if (half == 1) {
            ok = mbar_wait(&tail->other_empty, (done & 1u) ^ 1u, abort_flag, err, kErrTime);
            if (!__all_sync(0xffffffffu, ok)) break;
            tail->other[me] = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->other_full);
          } else {
            ok = mbar_wait(&tail->other_full, done & 1u, abort_flag, err, kErrTime);
            if (!__all_sync(0xffffffffu, ok)) break;
            sum = there ? sum + tail->other[me] : 0.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->other_empty);
            if (a.idx) {
              if (j0 + key < a.k) p.w[static_cast<long long>(c.item) * a.k + j0 + key] = sum;
            } else if (whole && (!MULTI || c.nt == p.nts - 1)) {
              if (j0 + key < min(len, a.n)) {
                const long long at = static_cast<long long>(c.item) * a.n + j0 + key;
                a.mass[at] = fmaf(a.decay, before, sum);
              }
            } else {
              // part 0: a tile begun in front of the range; part 1: one that goes on behind it
              p.part[(2ll * cluster + (whole ? 1 : 0)) * kTile + key] = sum;
            }
          }
          ++done;
        }
        if (MULTI && u == n - 1 && half == 0 && key == 0) {
          const int left = p.nts - 1 - c.nt;
          const int each = static_cast<int>(min(n, 0x40000000ll));   // this range is not the last one
          p.joins[cluster] = whole && left > 0 ? make_int4(c.item, c.tile, cluster + (left + each - 1) / each, 0)
                                               : make_int4(-1, 0, 0, 0);
        }
        c.next(p);
      }
    } else if (MULTI && half == 0 && key == 0) {
      p.joins[cluster] = make_int4(-1, 0, 0, 0);
    }
  } else if (warp == kStageWarp) {
    // ================================================================ the pairs' lse and limits
    if (n > 0) {
      Cursor<MULTI> c(p, tail);
      Ring<2> sr;
      int cur_item = -1, len = 0;
#pragma unroll 1
      for (long long u = 0; u < n; ++u) {
        if (MULTI || c.item != cur_item) {
          if (c.item != cur_item) {
            cur_item = c.item;
            len = seq_len(a, a.idx ? c.item / a.Sq : c.item, false);
          }
          float lse[kPairs / 32];
#pragma unroll
          for (int i = 0; i < kPairs / 32; ++i) {
            const int pr = c.nt * kPairs + i * 32 + lane;
            lse[i] = pr < pairs ? __ldg(a.lse + static_cast<long long>(c.item) * pairs + pr) : -INFINITY;
          }
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->staged_empty[sr.slot], sr.round ^ 1u, abort_flag,
                                                 err, kErrTime)))
            break;
#pragma unroll
          for (int i = 0; i < kPairs / 32; ++i) {
            const int pr = c.nt * kPairs + i * 32 + lane;
            // a pair without a key, and one that is not there, adds nothing
            const int lim = lse[i] == -INFINITY ? kNone
                                                : len - a.Sq + (a.idx ? c.item % a.Sq : pr / a.H) + 1;
            tail->nlse[sr.slot][i * 32 + lane] = -lse[i];
            tail->lim[sr.slot][i * 32 + lane] = lim;
            const int least = __reduce_min_sync(0xffffffffu, lim);
            if (lane == 0) tail->group_lim[sr.slot][i] = least;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->staged_full[sr.slot]);
          sr.next();
        }
        c.next(p);
      }
    }
  } else if (warp == kIssueWarp) {
    // ================================================================ UMMA issuer
    if (lane == 0 && n > 0 && rank == 0) {
      const uint32_t idesc = umma_idesc_bf16(kTile, p.box);
      const uint64_t k0 = umma_sdesc(smem_u32(smem), 1024, kLayoutSw128);
      const uint64_t q0 = umma_sdesc(smem_u32(qsmem), 1024, kLayoutSw128);
      Cursor<MULTI> c(p, tail);
      Ring<kKeySlots> kr;
      Ring<kQuerySlots> qr;
      bool ok = true;
#pragma unroll 1
      for (long long u = 0; ok && u < n; ++u) {
        const int buf = static_cast<int>(u) & 1;
        // the operand that stays is new here, or is used for the last time
        const bool first = u == 0 || (MULTI ? c.nt == 0 : c.tile == 0);
        const bool last = u == n - 1 || (MULTI ? c.nt == p.nts - 1 : c.tile == c.tiles - 1);
        ok = mbar_wait(&tail->d_empty[buf], (static_cast<uint32_t>(u >> 1) & 1u) ^ 1u, abort_flag, err,
                       kErrTime);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          if (ok && (!MULTI || first))
            ok = mbar_wait(&tail->k_full[kr.slot], kr.round, abort_flag, err, kErrTime);
          if (ok && (MULTI || first))
            ok = mbar_wait(&tail->q_full[qr.slot], qr.round, abort_flag, err, kErrTime);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = umma_desc_adv(k0, kr.slot * (kGroup * kKeyAtom));
          const uint64_t qd = umma_desc_adv(q0, qr.slot * (kGroup * kQueryAtom));
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int d = g * kGroup + i;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma2_bf16(tmem + (2 * buf + (d >= kFirstAtoms ? 1 : 0)) * kPairs,
                         umma_desc_adv(kd, i * kKeyAtom + kk * 32),
                         umma_desc_adv(qd, i * kQueryAtom + kk * 32), idesc,
                         (d == 0 || d == kFirstAtoms) && kk == 0 ? 0u : 1u);
          }
          if (!MULTI || last) umma2_commit(&tail->k_empty[kr.slot]);
          if (MULTI || last) umma2_commit(&tail->q_empty[qr.slot]);
          kr.next();
          qr.next();
        }
        // what stays is read again: its phase is over only with the last use
        if (!last) {
          if (MULTI)
            kr.round ^= 1u;
          else
            qr.round ^= 1u;
        }
        if (ok) umma2_commit(&tail->d_full[buf]);
        c.next(p);
      }
      umma2_commit(&tail->drain);
      drain_wait(&tail->drain, err);
    }
  } else if (warp == kQueryWarp) {
    // ================================================================ Q
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&qmap);
      const uint32_t full0 = first_cta(&tail->q_full[0]);
      Cursor<MULTI> c(p, tail);
      Ring<kQuerySlots> qr;
      bool ok = true;
#pragma unroll 1
      for (long long u = 0; ok && u < n; ++u) {
        if (MULTI || u == 0 || c.tile == 0) {
          const int row = c.item * pairs + c.nt * kPairs + rank * (p.box / 2);
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) {
            ok = mbar_wait(&tail->q_empty[qr.slot], qr.round ^ 1u, abort_flag, err, kErrTime);
            if (!ok) break;
            // (the second CTA's half may come in front of this: its bytes are only taken off)
            if (rank == 0) mbar_arrive_expect_tx(&tail->q_full[qr.slot], kGroup * p.box * 128);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
              tma2_load_2d(qsmem + (qr.slot * kGroup + i) * kQueryAtom, &qmap, full0 + qr.slot * 8,
                           (g * kGroup + i) * 64, row);
            qr.next();
          }
        }
        c.next(p);
      }
      // The commits arrive in both CTAs, and the second one waits for them too: from its last query on, or, where
      // a query may stay for a whole range, from its last row on, so that the wait is of a few units. (In the
      // epilogue, behind the last products, it took 2% of the time of many pairs.)
      if (MULTI && rank == 1) drain_wait(&tail->drain, err);
      if (*abort_flag) {
        // what is on its way lands before the block ends: some time for it, since the barrier's phase
        // may hang on the other CTA
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp >= kGatherWarp0 && n > 0) {
    // ================================================================ rows
    const int t = threadIdx.x - 32 * kGatherWarp0, key = t >> 2, sub = t & 3;
    const long long row_bytes = FP8 ? kDc + 16 + 2 * kDr : 2 * kD;
    // the tiles of the range: from the cursor's on, until its units are used up
    Cursor<MULTI> ahead(p, tail);
    long long left = n + (MULTI ? ahead.nt : 0);   // units from the tile's first on
    auto more = [&]() { return left > 0; };
    auto advance = [&]() {
      left -= MULTI ? p.nts : 1;
      if (left > 0) ahead.next_tile(p);
    };
    // Three steps for the thread's key of a tile: its position (or list entry), its page, its row.
    struct Found {
      int raw, len, limit, b;
    };
    auto look = [&]() {
      Found f = {-1, 0, 0, 0};
      if (!more()) return f;
      f.b = a.idx ? ahead.item / a.Sq : ahead.item;
      f.len = seq_len(a, f.b, false);
      f.limit = a.idx ? f.len - a.Sq + ahead.item % a.Sq + 1 : min(f.len, a.n);
      const uint32_t j = static_cast<uint32_t>(ahead.tile) * kTile + rank * kKeys + key;
      if (a.idx)   // (k may be within a tile of 2^31)
        f.raw = j < static_cast<uint32_t>(a.k)
                    ? __ldg(a.idx + static_cast<long long>(ahead.item) * a.k + j)
                    : -1;
      else
        f.raw = static_cast<int>(j);   // n is at most 2^30
      return f;
    };
    struct Paged {
      int page, off;
    };
    auto page_of = [&](const Found& f) {
      Paged q = {-1, -1};
      if (a.idx && (f.raw < -1 || f.raw >= f.len)) {
        if (f.raw != -1) report_error(err, kErrIdx);
      } else if (f.raw >= 0 && f.raw < f.limit) {
        const int pg = p.page_shift >= 0 ? f.raw >> p.page_shift : f.raw / a.page_size;
        q.off = f.raw - pg * a.page_size;
        q.page = __ldg(a.page_table + static_cast<long long>(f.b) * a.max_pages + pg);
      }
      return q;
    };
    auto row_of = [&](const Paged& q) -> const uint8_t* {
      if (q.off < 0) return nullptr;
      if (q.page < 0 || q.page >= a.num_pages) {
        report_error(err, kErrPage);
        return nullptr;
      }
      return a.cache + (static_cast<long long>(q.page) * a.page_size + q.off) * row_bytes;
    };
    Ring<kKeySlots> kr;
    const uint32_t base = smem_u32(smem);
    auto wait_empty = [&]() {
      return __all_sync(0xffffffffu, mbar_wait(&tail->k_empty[kr.slot], kr.round ^ 1u, abort_flag, err,
                                               kErrTime)) != 0;
    };
    auto tell_valid = [&](int tiles, bool there) {
      const uint32_t bits = __ballot_sync(0xffffffffu, there);
      if (lane == 0) {
        tail->valid[tiles % 3][warp - kGatherWarp0] = bits;
        mbar_arrive(&tail->valid_full[tiles % 3]);
      }
    };
    // A warp's part of an atom is written: one arrival for it. (One per thread, 512 an atom, is level:
    // what took the time were the loads.)
    const uint32_t full0 = first_cta(&tail->k_full[0]);
    auto tell_full = [&](int slot) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_first_cta(full0 + slot * 8);
    };
    const uint32_t at = key * 128;
    if constexpr (!FP8) {
      // copies of a group behind the newest are on their way
      Ring<kKeySlots> landed;
      bool flying = false;
      const uint8_t* row = row_of(page_of(look()));
      bool ok = true;
#pragma unroll 1
      for (int tiles = 0; ok && more(); ++tiles) {
        advance();
        const Found f = look();   // of the next tile
        Paged q = {-1, -1};
        const uint8_t* src = (row ? row : a.cache) + sub * 16;
        const uint32_t bytes = row ? 16u : 0u;
        const uint32_t lo = at + ((sub ^ (key & 7)) << 4), hi = at + (((sub + 4) ^ (key & 7)) << 4);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          ok = ok && wait_empty();
          if (!ok) break;
          if (g == 0) tell_valid(tiles, row != nullptr);
          const uint32_t dst = base + kr.slot * (kGroup * kKeyAtom);
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            cp_async_16(dst + i * kKeyAtom + lo, src + (g * kGroup + i) * 128, bytes);
            cp_async_16(dst + i * kKeyAtom + hi, src + (g * kGroup + i) * 128 + 64, bytes);
          }
          cp_async_commit();
          kr.next();
          if (flying) {
            cp_async_wait<1>();
            tell_full(landed.slot);
            landed.next();
          }
          flying = true;
          if (g == 0) q = page_of(f);
        }
        row = row_of(q);
        // the last ones; a tile that stays is waited for as a whole before its slots come free again
        if (ok && (MULTI || !more())) {
          cp_async_wait<0>();
          tell_full(landed.slot);
          landed.next();
          flying = false;
        }
      }
      cp_async_wait<0>();
    } else {
      // Raw ring: a thread copies in what it widens itself, step by step: eight pieces of 16 codes, two of
      // positional dims, kAhead steps ahead. The scales come by way of a register, a tile ahead.
      constexpr int kAhead = L::kRawSlots;
      static_assert(kAhead < kRawSteps && kAhead >= 4, "one tile's steps, and a group's");
      const uint32_t raw0 = base + L::kRawOff + t * 16;
      struct Source {
        const uint8_t* at;
        uint32_t bytes;
      };
      auto source = [&](const uint8_t* row) {
        return Source{(row ? row : a.cache) + sub * 16, row ? 16u : 0u};
      };
      auto fetch = [&](const Source& from, int step, uint32_t dst) {
        cp_async_16(dst, from.at + (step < 8 ? step * 64 : kDc + 16 + (step - 8) * 64), from.bytes);
        cp_async_commit();
      };
      auto scales_of = [&](const Source& from) {
        return from.bytes ? __ldg(reinterpret_cast<const uint4*>(from.at - sub * 16 + kDc))
                          : make_uint4(0, 0, 0, 0);
      };
      Source row = source(row_of(page_of(look())));   // of the tile that is widened
      long long togo = left;                          // units of it and of those behind it
      uint4 scale = scales_of(row);
      advance();
      Source next = source(row_of(page_of(look())));
      if (more()) advance();
      Found f = look();                               // the tile two ahead
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(row, i, raw0 + i * kRawAtom);
      uint32_t raw = raw0;
      bool ok = true;
#pragma unroll 1
      for (int tiles = 0; ok && togo > 0; ++tiles, togo -= MULTI ? p.nts : 1) {
        const uint4 next_scale = scales_of(next);
        Paged q = {-1, -1};
        // step i: its piece out of the ring, and the piece kAhead steps on into the same place
        auto step = [&](int i) {
          uint4 x;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(raw)
                       : "memory");
          fetch(i + kAhead < kRawSteps ? row : next, (i + kAhead) % kRawSteps, raw);
          raw = raw == raw0 + (kAhead - 1) * kRawAtom ? raw0 : raw + kRawAtom;
          return x;
        };
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          uint4 x[kGroup + 1];
          cp_async_wait<kAhead - (kGroup + 1)>();   // (one more than the first groups need)
#pragma unroll
          for (int i = 0; i < kGroup + (g == 2 ? 1 : 0); ++i) x[i] = step(g * kGroup + i);
          ok = ok && wait_empty();
          if (!ok) break;
          if (g == 0) tell_valid(tiles, row.bytes != 0);
          uint8_t* dst = smem + kr.slot * (kGroup * kKeyAtom) + at;
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int d = g * kGroup + i;
            if (d == 8) {
              *reinterpret_cast<uint4*>(dst + i * kKeyAtom + ((sub ^ (key & 7)) << 4)) = x[i];
              *reinterpret_cast<uint4*>(dst + i * kKeyAtom + (((sub + 4) ^ (key & 7)) << 4)) = x[i + 1];
              continue;
            }
            const uint32_t e = (d < 2 ? scale.x : d < 4 ? scale.y : d < 6 ? scale.z : scale.w) >> 16;
            const uint32_t up = widen_factor(e);
            uint4 w0, w1;
            widen4_in_order(x[i].x, up, w0.x, w0.y);
            widen4_in_order(x[i].y, up, w0.z, w0.w);
            widen4_in_order(x[i].z, up, w1.x, w1.y);
            widen4_in_order(x[i].w, up, w1.z, w1.w);
            if (e > kScaleMost) {   // a scale of more than 2^7, or of NaN
              const uint32_t rest = widen_rest(e);
              w0 = make_uint4(mul_bf16x2(w0.x, rest), mul_bf16x2(w0.y, rest), mul_bf16x2(w0.z, rest),
                              mul_bf16x2(w0.w, rest));
              w1 = make_uint4(mul_bf16x2(w1.x, rest), mul_bf16x2(w1.y, rest), mul_bf16x2(w1.z, rest),
                              mul_bf16x2(w1.w, rest));
            }
            *reinterpret_cast<uint4*>(dst + i * kKeyAtom + (((2 * sub) ^ (key & 7)) << 4)) = w0;
            *reinterpret_cast<uint4*>(dst + i * kKeyAtom + (((2 * sub + 1) ^ (key & 7)) << 4)) = w1;
          }
          tell_full(kr.slot);
          kr.next();
          if (g == 1) q = page_of(f);
        }
        if (!ok) break;
        row = next;
        scale = next_scale;
        next = source(row_of(q));
        if (more()) advance();
        f = look();
      }
      cp_async_wait<0>();
    }
    if (!MULTI && rank == 1 && t == 0) drain_wait(&tail->drain, err);
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();   // no CTA leaves while the other may still write to it
  tc_fence_after();
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A tile that begins in cluster c's range and goes on behind it: its parts, one after the other.
__global__ void __launch_bounds__(kTile) join_kernel(const Params p, int clusters) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MassArgs& a = p.a;
  const int4 t = __ldcg(p.joins + blockIdx.x);
  // nothing to join, or not written: a cluster whose waits ran out (recorded) leaves what was there
  if (t.x < 0 || t.x >= a.B || t.y < 0 || t.z <= static_cast<int>(blockIdx.x) || t.z >= clusters) return;
  const int len = min(seq_len(a, t.x, false), a.n);
  if (t.y >= (len + kTile - 1) / kTile) return;
  const int j = t.y * kTile + threadIdx.x;
  if (j >= len) return;
  float sum = __ldcg(p.part + (2ll * blockIdx.x + 1) * kTile + threadIdx.x);
  for (int c = blockIdx.x + 1; c <= t.z; ++c) sum += __ldcg(p.part + 2ll * c * kTile + threadIdx.x);
  const long long at = static_cast<long long>(t.x) * a.n + j;
  a.mass[at] = a.prev ? fmaf(a.decay, a.prev[at], sum) : sum;
}

// Lists: a block has kSlice positions of sequence b in shared memory, adds the lists' weights to
// them token by token (a list's entries are distinct, so the order is fixed) and writes them out.
constexpr int kSlice = 8192, kAddThreads = 512;
__global__ void __launch_bounds__(kAddThreads) add_lists_kernel(const Params p) {
  __shared__ float m[kSlice];
  const MassArgs& a = p.a;
  const int slices = (a.n + kSlice - 1) / kSlice, b = blockIdx.x / slices;
  const int lo = (blockIdx.x - b * slices) * kSlice, size = min(kSlice, a.n - lo);
  const int len = seq_len(a, b, lo == 0 && threadIdx.x == 0);
  const long long at = static_cast<long long>(b) * a.n + lo;
#pragma unroll 4
  for (int j = threadIdx.x; j < size; j += kAddThreads)
    m[j] = a.prev && lo + j < len ? a.decay * a.prev[at + j] : 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // for the weights, nothing else
  __syncthreads();
  for (int i = 0; i < a.Sq; ++i) {
    const long long list = (static_cast<long long>(b) * a.Sq + i) * a.k;
    const int limit = len - a.Sq + i + 1;
    constexpr int kAtOnce = 4;
    for (long long s0 = threadIdx.x; s0 < a.k; s0 += kAtOnce * kAddThreads) {
      int j[kAtOnce];
      float w[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const long long s = s0 + q * kAddThreads;
        j[q] = s < a.k ? __ldg(a.idx + list + s) : -1;
        w[q] = s < a.k ? __ldcg(p.w + list + s) : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (j[q] >= lo && j[q] - lo < size && j[q] < limit) atomicAdd(m + (j[q] - lo), w[q]);
    }
    __syncthreads();
  }
  for (int j = threadIdx.x; j < size; j += kAddThreads) a.mass[at + j] = m[j];
}

// Q [rows, 576] bf16 in boxes of 64 dims x box rows, 128B-swizzled
bool query_map(CUtensorMap* map, const void* Q, long long rows, int box) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  cuuint32_t boxes[2] = {64, static_cast<cuuint32_t>(box)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(Q), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of the kernel that fit on the current device at once; the first call on a device also
// raises the kernel's shared-memory limit there.
template <bool FP8, bool MULTI>
int resident_clusters(size_t smem) {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices] = {};
  static std::mutex lock;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> guard(lock);
  if (known[dev] == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (cudaFuncSetAttribute(mass_kernel<FP8, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    if (cudaOccupancyMaxActiveClusters(&c, mass_kernel<FP8, MULTI>, &cfg) != cudaSuccess || c < 1) return 0;
    known[dev] = c < kMaxClusters ? c : kMaxClusters;
  }
  return known[dev];
}

template <bool FP8, bool MULTI>
int launch(Params p, cudaStream_t stream) {
  const MassArgs& a = p.a;
  const int pairs = a.idx ? a.H : a.Sq * a.H;
  p.items = a.idx ? a.B * a.Sq : a.B;
  p.nts = (pairs - 1) / kPairs + 1;
  p.box = pair_columns(pairs);
  CUtensorMap map;
  if (!query_map(&map, a.Q, static_cast<long long>(a.B) * a.Sq * a.H, p.box / 2)) return DSA_ERR_CUDA;
  const size_t smem = Layout<FP8, MULTI>::kTailOff + sizeof(Tail);
  int clusters = resident_clusters<FP8, MULTI>(smem);
  if (clusters < 1) return DSA_ERR_CUDA;
  // no more clusters than the longest possible sequences have work for
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  const long long keys = a.idx ? a.k : cap < a.n ? cap : a.n;
  const long long most = p.items * ((keys + kTile - 1) / kTile) * (MULTI ? p.nts : 1);
  if (most < clusters) clusters = static_cast<int>(most);
  if (MULTI) {
    p.part = static_cast<float*>(a.ws);
    p.joins = reinterpret_cast<int4*>(p.part + 2 * kMaxClusters * kTile);
  }
  p.w = static_cast<float*>(a.ws);
  mass_kernel<FP8, MULTI><<<2 * clusters, kThreads, smem, stream>>>(p, map);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (!a.idx && (!MULTI || clusters == 1)) return DSA_OK;   // nothing is split
  // the second kernel's blocks may be set up while the last clusters finish; they wait for the weights, or
  // the parts
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (a.idx) {
    const long long blocks = static_cast<long long>(a.B) * ((a.n + kSlice - 1) / kSlice);
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kAddThreads);
    return cudaLaunchKernelEx(&cfg, add_lists_kernel, p) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  }
  cfg.gridDim = dim3(clusters - 1);
  cfg.blockDim = dim3(kTile);
  return cudaLaunchKernelEx(&cfg, join_kernel, p, clusters) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

size_t cache_mass_workspace(int B, int Sq, int H, int k) {
  if (k > 0) return static_cast<size_t>(B) * Sq * k * sizeof(float);
  if (static_cast<long long>(Sq) * H <= kPairs) return 0;
  return 2 * kMaxClusters * kTile * sizeof(float) + kMaxClusters * sizeof(int4);
}

int launch_cache_mass(const MassArgs& a, int fmt, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  const bool multi = !a.idx && static_cast<long long>(a.Sq) * a.H > kPairs;
  if (fmt == DSA_CACHE_E4M3)
    return multi ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return multi ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace dsa
