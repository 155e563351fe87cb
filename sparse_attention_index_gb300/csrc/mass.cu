// The attention weight that each cached position receives from the newest tokens (dsa_cache_mass), on
// the 5th-generation tensor cores.
//
//   mass[j] = decay prev[j] + sum over tokens i and heads h that see j of exp(scale q_ih . row_j - lse_ih)
//
// with lse from the attention itself, so that one more product of queries and rows is all it takes. The
// keys are the 128 lanes of a tile and the (token, head) pairs its columns, so that a key's sum over
// tokens and heads stays within one thread:
//
//   S [128 keys x 128 pairs] = K [128 x 576] . Q^T,   sum_c exp(scale S_c - lse_c)
//
// Both operands go through shared memory in atoms of 64 dims (16 KB). Up to 128 pairs a sequence (a
// token with a list always is): Q stays, the rows stream through a ring of five atoms, and memory is
// the bound. More pairs: a tile's rows stay and the pairs stream past them, 128 at a time; the tensor
// cores are the bound. The work, tiles or (tile, 128 pairs), is cut into one even range per CTA whatever
// the lengths. A tile whose pairs lie in several ranges leaves a part in each, which
// join_kernel adds up in order. Lengths are read on the device only.
//
// Warp-specialised CTA, 704 threads:
//   warps 0-3   epilogue, one key per thread
//   warp 4      single-thread UMMA issuer; owns TMEM: two buffers of 128 columns
//   warp 5      Q by TMA
//   warps 6-21  rows, a quarter of a key's atom per thread: bf16 by cp.async, e4m3 by way of
//               registers (a tile ahead), widened to bf16, exactly

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "latent_row.cuh"

namespace dsa {
namespace {

constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kTile = 128;               // keys of a tile, and pairs at a time
constexpr int kAtoms = kD / 64;
constexpr uint32_t kAtom = kTile * 128;
constexpr int kRing = 5;                 // atoms of the operand that streams; the other has all nine
constexpr int kSlots = kRing + kAtoms;
constexpr int kIssueWarp = 4, kQueryWarp = 5, kGatherWarp0 = 6, kGatherWarps = 16;
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);
constexpr int kMaxCtas = 256;
constexpr int kErrIdx = DSA_STAGE_EVICT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_EVICT | DSA_DEVERR_BAD_PAGE;
constexpr int kErrTime = DSA_STAGE_EVICT | DSA_DEVERR_TIMEOUT;
static_assert(kGatherThreads == 4 * kTile, "a quarter of a key's atom per thread");

struct Tail {
  float nlse[2][kTile];      // -lse of the pairs
  int lim[2][kTile];         // positions below it are seen by the pair; a pair that adds nothing: none
  int group_lim[2][4];       // the least of 32 pairs
  uint32_t valid[4][kGatherWarps];   // the tile's keys that are there: four bits a key
  uint64_t k_full[kAtoms], k_empty[kAtoms], q_full[kAtoms], q_empty[kAtoms];   // of ring or residents
  uint64_t d_full[2], d_empty[2], valid_full[4], staged, drain;
  uint32_t tmem_base;
  int abort_flag;
  long long sums[kThreads / 32];
  // this CTA's range: its first item and the first unit of it here, and how many units
  int item0;
  long long first, count;
};
constexpr size_t kSmem = kSlots * kAtom + sizeof(Tail);
static_assert(kSmem <= 232448, "shared memory of a block");

struct Params {
  MassArgs a;
  int items;        // sequences, or tokens with a list each
  int nts;          // columns of 128 pairs
  int box;          // pairs loaded at a time (a multiple of 16)
  int page_shift;   // log2 of the page size, -1 where it is no power of two
  float* w;         // lists: the weight of each entry [B, Sq, k]
  float* part;      // [2 * ctas][128]
  int4* joins;      // [ctas]: (sequence, tile, last CTA that has a part of it) or (-1, ...)
};

__device__ __forceinline__ int seq_len(const MassArgs& a, int b, bool report) {
  const int cap = a.max_pages * a.page_size;
  const int len = __ldg(a.lens + b);
  if (report && (len < 0 || len > cap || len > a.n)) report_error(a.err, kErrPage);
  return max(0, min(len, cap));
}

__device__ __forceinline__ int item_tiles(const Params& p, int item) {
  const int keys = p.a.idx ? p.a.k : min(p.a.n, seq_len(p.a, item, false));
  return (keys + kTile - 1) / kTile;   // (n and k are at most 2^30)
}

// this CTA's range of units, into the tail; every thread of the block calls it, before a barrier
template <bool MULTI>
__device__ __forceinline__ void my_units(const Params& p, Tail* tail) {
  const long long per_tile = MULTI ? p.nts : 1;
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
    if (lane == 31) tail->sums[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += tail->sums[w];
      total += tail->sums[w];
    }
    before += incl - s;
  }
  const long long each = (total + gridDim.x - 1) / gridDim.x;
  const long long u0 = min(total, each * blockIdx.x), u1 = min(total, u0 + each);
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

// where a warp stands in its CTA's range
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
__global__ void __launch_bounds__(kThreads, 1)
    mass_kernel(const Params p, const __grid_constant__ CUtensorMap qmap) {
  constexpr int kKeySlots = MULTI ? kAtoms : kRing, kQuerySlots = MULTI ? kRing : kAtoms;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const qsmem = smem + kKeySlots * kAtom;
  Tail* tail = reinterpret_cast<Tail*>(smem + kSlots * kAtom);
  volatile int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MassArgs& a = p.a;
  int* err = a.err;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) report_error(err, DSA_STAGE_EVICT | DSA_DEVERR_MISALIGNED);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kAtoms; ++i) {
      mbar_init(&tail->k_full[i], kGatherThreads);
      mbar_init(&tail->k_empty[i], 1);
      mbar_init(&tail->q_full[i], 1);
      mbar_init(&tail->q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->d_full[i], 1);
      mbar_init(&tail->d_empty[i], kTile);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&tail->valid_full[i], kGatherWarps);
    mbar_init(&tail->staged, kTile);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    tail->count = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&tail->tmem_base, 256);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  my_units<MULTI>(p, tail);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  const long long n = tail->count;

  if (warp < 4) {
    // ================================================================ epilogue
    if (!a.idx) {
      // zeros behind the sequences' ends, shared out among the CTAs
      for (int b = warp; b < a.B; b += 4) {
        const int len = seq_len(a, b, blockIdx.x == 0 && lane == 0), end = min(len, a.n);
        const long long room = a.n - end;
        const int z0 = end + static_cast<int>(room * blockIdx.x / gridDim.x);
        const int z1 = end + static_cast<int>(room * (blockIdx.x + 1) / gridDim.x);
        for (int j = z0 + lane; j < z1; j += 32) a.mass[static_cast<long long>(b) * a.n + j] = 0.f;
      }
    }
    const int key = threadIdx.x;   // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const int pairs = a.idx ? a.H : a.Sq * a.H;   // of an item
    const float2 scale2 = make_float2(a.scale, a.scale);
    const float2 log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
    if (n > 0) {
      Cursor<MULTI> c(p, tail);
      int cur_item = -1, len = 0;
      float sum = 0.f;
      bool whole = false;        // the tile's first pairs were here
      int tiles_done = 0;        // tiles whose flags have been taken
      int stages = 0;            // times that pairs' lse and limits have been written
      bool there = false;
#pragma unroll 1
      for (long long u = 0; u < n; ++u) {
        const int buf = static_cast<int>(u) & 1;
        const uint32_t par = static_cast<uint32_t>(u >> 1) & 1u;
        const bool fresh_item = c.item != cur_item;
        if (fresh_item) {
          cur_item = c.item;
          len = seq_len(a, a.idx ? c.item / a.Sq : c.item, false);
        }
        // The pairs' lse and limits: with several columns per tile they change with each unit. (The
        // buffer was last read two stages ago, before every thread's arrival at the last one.)
        if (MULTI || fresh_item) {
          const int w = stages & 1;
          const int pr = c.nt * kTile + key;
          float v = 0.f;
          int lim = -0x7fffffff - 1;
          if (pr < pairs) {
            const long long row = static_cast<long long>(c.item) * pairs + pr;
            const float lse = __ldg(a.lse + row);
            const int token = a.idx ? c.item % a.Sq : pr / a.H;
            v = -lse;
            if (lse != -INFINITY) lim = len - a.Sq + token + 1;
          }
          tail->nlse[w][key] = v;
          tail->lim[w][key] = lim;
          lim = __reduce_min_sync(0xffffffffu, lim);
          if (lane == 0) tail->group_lim[w][warp] = lim;
          __syncwarp();
          mbar_arrive(&tail->staged);
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->staged, w, abort_flag, err, kErrTime))) break;
          ++stages;
        }
        const int sb = (stages & 1) ^ 1;
        if (u == 0 || c.nt == 0) {
          sum = 0.f;
          whole = c.nt == 0;
          const int vb = tiles_done & 3;
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->valid_full[vb], (tiles_done >> 2) & 1,
                                                 abort_flag, err, kErrTime)))
            break;
          there = (tail->valid[vb][key >> 3] >> (4 * (key & 7)) & 1u) != 0;
          ++tiles_done;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->d_full[buf], par, abort_flag, err, kErrTime)))
          break;
        tc_fence_after();
        const int j0 = c.tile * kTile;
        // lists: a key that its token does not see is not there
        const int last = a.idx ? -0x7fffffff - 1 : min(j0 + kTile, len);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float some = 0.f;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          if (c.nt * kTile + g * 32 >= pairs) break;
          uint32_t s[32];
          tmem_ld_x32(tmem + lane_off + buf * kTile + g * 32, s);
          tmem_ld_wait();
          const float4* nl = reinterpret_cast<const float4*>(&tail->nlse[sb][g * 32]);
          const int least = tail->group_lim[sb][g];
          if (least != -0x7fffffff - 1 && least >= last) {
            // every pair of the group sees every key of the tile
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 v = nl[q];
              // the difference first, in one rounding: far from zero those of the products with
              // log2(e) would move the weight
              float2 x = fma2(make_float2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])),
                              scale2, make_float2(v.x, v.y));
              float2 y = fma2(make_float2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])),
                              scale2, make_float2(v.z, v.w));
              x = mul2(x, log2e);
              y = mul2(y, log2e);
              acc[0] = add2(acc[0], make_float2(ex2f(x.x), ex2f(x.y)));
              acc[1] = add2(acc[1], make_float2(ex2f(y.x), ex2f(y.y)));
            }
          } else {
            const int j = a.idx ? -0x7fffffff - 1 : j0 + key;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const int lim = tail->lim[sb][g * 32 + q];
              const float x = fmaf(__uint_as_float(s[q]), a.scale, tail->nlse[sb][g * 32 + q]);
              // (with lists j is below every limit but that of a pair that adds nothing)
              if (lim != -0x7fffffff - 1 && j < lim) some += ex2f(x * log2e.x);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&tail->d_empty[buf]);
        sum += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) + some;
        if (!MULTI || c.nt == p.nts - 1 || u == n - 1) {
          if (!there) sum = 0.f;
          if (a.idx) {
            if (j0 + key < a.k) p.w[static_cast<long long>(c.item) * a.k + j0 + key] = sum;
          } else if (whole && (!MULTI || c.nt == p.nts - 1)) {
            if (j0 + key < min(len, a.n)) {
              const long long at = static_cast<long long>(c.item) * a.n + j0 + key;
              a.mass[at] = a.prev ? fmaf(a.decay, a.prev[at], sum) : sum;
            }
          } else {
            // part 0: a tile begun in front of the range; part 1: one that goes on behind it
            p.part[(2ll * blockIdx.x + (whole ? 1 : 0)) * kTile + key] = sum;
          }
        }
        if (MULTI && u == n - 1 && key == 0) {
          const int left = p.nts - 1 - c.nt;
          const int each = static_cast<int>(min(n, 0x40000000ll));   // this range is not the last one
          p.joins[blockIdx.x] = whole && left > 0
                                    ? make_int4(c.item, c.tile, blockIdx.x + (left + each - 1) / each, 0)
                                    : make_int4(-1, 0, 0, 0);
        }
        c.next(p);
      }
    } else if (MULTI && key == 0) {
      p.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
  } else if (warp == kIssueWarp) {
    // ================================================================ UMMA issuer
    if (lane == 0 && n > 0) {
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
#pragma unroll 1
        for (int d = 0; ok && d < kAtoms; ++d) {
          if (!MULTI || first)
            ok = mbar_wait(&tail->k_full[kr.slot], kr.round, abort_flag, err, kErrTime);
          if (ok && (MULTI || first))
            ok = mbar_wait(&tail->q_full[qr.slot], qr.round, abort_flag, err, kErrTime);
          if (!ok) break;
          fence_proxy_async_smem();   // the rows were written by the generic proxy
          tc_fence_after();
          const uint64_t kd = umma_desc_adv(k0, kr.slot * kAtom), qd = umma_desc_adv(q0, qr.slot * kAtom);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + buf * kTile, umma_desc_adv(kd, kk * 32), umma_desc_adv(qd, kk * 32), idesc,
                      d > 0 || kk > 0 ? 1u : 0u);
          if (!MULTI || last) umma_commit(&tail->k_empty[kr.slot]);
          if (MULTI || last) umma_commit(&tail->q_empty[qr.slot]);
          kr.next();
          qr.next();
          // what stays is read again: its phase is over only with the last use
          if (MULTI && !last && kr.slot == 0) kr.round ^= 1u;
          if (!MULTI && !last && qr.slot == 0) qr.round ^= 1u;
        }
        if (ok) umma_commit(&tail->d_full[buf]);
        c.next(p);
      }
      umma_commit(&tail->drain);
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&tail->drain), 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          report_error(err, kErrTime);
          break;
        }
      }
    }
  } else if (warp == kQueryWarp) {
    // ================================================================ Q
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&qmap);
      const int pairs = a.idx ? a.H : a.Sq * a.H;
      Cursor<MULTI> c(p, tail);
      Ring<kQuerySlots> qr;
      bool ok = true;
      long long loads = 0;
#pragma unroll 1
      for (long long u = 0; ok && u < n; ++u) {
        if (MULTI || u == 0 || c.tile == 0) {
          const int row = c.item * pairs + c.nt * kTile;
#pragma unroll 1
          for (int d = 0; d < kAtoms; ++d) {
            ok = mbar_wait(&tail->q_empty[qr.slot], qr.round ^ 1u, abort_flag, err, kErrTime);
            if (!ok) break;
            mbar_arrive_expect_tx(&tail->q_full[qr.slot], p.box * 128);
            tma_load_2d(qsmem + qr.slot * kAtom, &qmap, &tail->q_full[qr.slot], d * 64, row);
            qr.next();
            ++loads;
          }
        }
        c.next(p);
      }
      if (*abort_flag) {
        // what is on its way lands before the block ends: the last load of each slot
        const unsigned long long t0 = globaltimer_ns();
        for (int i = 0; i < kQuerySlots && i < loads; ++i) {
          const uint32_t round = i < qr.slot ? qr.round : qr.round ^ 1u;
          while (!mbar_try_wait(smem_u32(&tail->q_full[i]), round) &&
                 globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (n > 0) {
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
      f.raw = ahead.tile * kTile + key;
      if (a.idx)
        f.raw = f.raw < a.k ? __ldg(a.idx + static_cast<long long>(ahead.item) * a.k + f.raw) : -1;
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
        tail->valid[tiles & 3][warp - kGatherWarp0] = bits;
        mbar_arrive(&tail->valid_full[tiles & 3]);
      }
    };
    const uint32_t at = key * 128;
    if (!FP8) {
      const uint8_t* row = row_of(page_of(look()));
      bool ok = true;
#pragma unroll 1
      for (int tiles = 0; ok && more(); ++tiles) {
        advance();
        const Found f = look();   // of the next tile
        Paged q = {-1, -1};
        const uint8_t* src = row ? row : a.cache;
        const uint32_t bytes = row ? 16u : 0u;
#pragma unroll 1
        for (int d = 0; d < kAtoms; ++d) {
          ok = wait_empty();
          if (!ok) break;
          if (d == 0) tell_valid(tiles, row != nullptr);
          const uint32_t dst = base + kr.slot * kAtom + at;
          cp_async_16(dst + ((sub ^ (key & 7)) << 4), src + d * 128 + sub * 16, bytes);
          cp_async_16(dst + (((sub + 4) ^ (key & 7)) << 4), src + d * 128 + 64 + sub * 16, bytes);
          cp_async_mbar_arrive(&tail->k_full[kr.slot]);
          kr.next();
          if (d == 3) q = page_of(f);
        }
        row = row_of(q);
      }
      cp_async_wait<0>();
    } else {
      // A tile's codes, scales and positional dims are loaded into registers a tile ahead.
      uint4 code[8], rope[2], scale, next_scale;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      auto load_code = [&](const uint8_t* row, int d) {
        code[d] = row ? __ldg(reinterpret_cast<const uint4*>(row + d * 64 + sub * 16)) : zero;
      };
      auto load_rope = [&](const uint8_t* row) {
        rope[0] = row ? __ldg(reinterpret_cast<const uint4*>(row + kDc + 16 + sub * 16)) : zero;
        rope[1] = row ? __ldg(reinterpret_cast<const uint4*>(row + kDc + 16 + 64 + sub * 16)) : zero;
      };
      auto load_scale = [&](const uint8_t* row) {
        next_scale = row ? __ldg(reinterpret_cast<const uint4*>(row + kDc)) : zero;
      };
      const uint8_t* row = row_of(page_of(look()));   // of the tile in registers
      load_scale(row);
#pragma unroll
      for (int d = 0; d < 8; ++d) load_code(row, d);
      load_rope(row);
      bool there = row != nullptr;
      advance();
      row = row_of(page_of(look()));                  // of the one to be loaded
      long long togo = n + (MULTI ? Cursor<MULTI>(p, tail).nt : 0);   // units of the tiles left
      bool ok = true;
#pragma unroll 1
      for (int tiles = 0; ok && togo > 0; ++tiles, togo -= MULTI ? p.nts : 1) {
        if (more()) advance();
        const Found f = look();   // two tiles ahead
        Paged q = {-1, -1};
        scale = next_scale;
        load_scale(row);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          ok = wait_empty();
          if (!ok) break;
          if (d == 0) tell_valid(tiles, there);
          uint8_t* dst = smem + kr.slot * kAtom + at;
          const uint32_t e = (d < 2 ? scale.x : d < 4 ? scale.y : d < 6 ? scale.z : scale.w) >> 16;
          const uint32_t up = widen_factor(e);
          const uint4 x = code[d];
          load_code(row, d);
          uint4 w0, w1;
          // (bytes 0 2 1 3, so that they come out in order)
          widen4(__byte_perm(x.x, 0, 0x3120), up, w0.x, w0.y);
          widen4(__byte_perm(x.y, 0, 0x3120), up, w0.z, w0.w);
          widen4(__byte_perm(x.z, 0, 0x3120), up, w1.x, w1.y);
          widen4(__byte_perm(x.w, 0, 0x3120), up, w1.z, w1.w);
          if (e > kScaleMost) {   // a scale of more than 2^7, or of NaN
            const uint32_t rest = widen_rest(e);
            w0 = make_uint4(mul_bf16x2(w0.x, rest), mul_bf16x2(w0.y, rest), mul_bf16x2(w0.z, rest),
                            mul_bf16x2(w0.w, rest));
            w1 = make_uint4(mul_bf16x2(w1.x, rest), mul_bf16x2(w1.y, rest), mul_bf16x2(w1.z, rest),
                            mul_bf16x2(w1.w, rest));
          }
          *reinterpret_cast<uint4*>(dst + (((2 * sub) ^ (key & 7)) << 4)) = w0;
          *reinterpret_cast<uint4*>(dst + (((2 * sub + 1) ^ (key & 7)) << 4)) = w1;
          fence_proxy_async_smem();
          mbar_arrive(&tail->k_full[kr.slot]);
          kr.next();
          if (d == 3) q = page_of(f);
        }
        if (!ok) break;
        ok = wait_empty();
        if (!ok) break;
        uint8_t* dst = smem + kr.slot * kAtom + at;
        *reinterpret_cast<uint4*>(dst + ((sub ^ (key & 7)) << 4)) = rope[0];
        *reinterpret_cast<uint4*>(dst + (((sub + 4) ^ (key & 7)) << 4)) = rope[1];
        load_rope(row);
        fence_proxy_async_smem();
        mbar_arrive(&tail->k_full[kr.slot]);
        kr.next();
        there = row != nullptr;
        row = row_of(q);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 256);
}

// A tile that begins in CTA c's range and goes on behind it: its parts, one after the other.
__global__ void __launch_bounds__(kTile) join_kernel(const Params p, int ctas) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MassArgs& a = p.a;
  const int4 t = __ldcg(p.joins + blockIdx.x);
  // nothing to join, or not written: a CTA whose waits ran out (recorded) leaves what was there
  if (t.x < 0 || t.x >= a.B || t.y < 0 || t.z <= static_cast<int>(blockIdx.x) || t.z >= ctas) return;
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
  for (int j = threadIdx.x; j < size; j += kAddThreads)
    m[j] = a.prev && lo + j < len ? a.decay * a.prev[at + j] : 0.f;
  __syncthreads();
  for (int i = 0; i < a.Sq; ++i) {
    const long long list = (static_cast<long long>(b) * a.Sq + i) * a.k;
    const int limit = len - a.Sq + i + 1;
    for (int s = threadIdx.x; s < a.k; s += kAddThreads) {
      const int j = __ldg(a.idx + list + s);
      if (j >= lo && j - lo < size && j < limit) atomicAdd(m + (j - lo), __ldcg(p.w + list + s));
    }
    __syncthreads();
  }
  for (int j = threadIdx.x; j < size; j += kAddThreads) a.mass[at + j] = m[j];
}

typedef CUresult (*EncodeTiledFnMass)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                      const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                      const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                      CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Q [rows, 576] bf16 in boxes of 64 dims x box rows, 128B-swizzled
bool query_map(CUtensorMap* map, const void* Q, long long rows, int box) {
  static EncodeTiledFnMass fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<EncodeTiledFnMass>(ptr);
  }
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  cuuint32_t boxes[2] = {64, static_cast<cuuint32_t>(box)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(Q), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, bool MULTI>
int launch(Params p, cudaStream_t stream) {
  const MassArgs& a = p.a;
  const int pairs = a.idx ? a.H : a.Sq * a.H;
  p.items = a.idx ? a.B * a.Sq : a.B;
  p.nts = (pairs + kTile - 1) / kTile;
  p.box = pairs < kTile ? (pairs + 15) / 16 * 16 : kTile;
  CUtensorMap map;
  if (!query_map(&map, a.Q, static_cast<long long>(a.B) * a.Sq * a.H, p.box)) return DSA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (cudaFuncSetAttribute(mass_kernel<FP8, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmem)) != cudaSuccess)
    return DSA_ERR_CUDA;
  // no more CTAs than the longest possible sequences have work for
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  const long long keys = a.idx ? a.k : cap < a.n ? cap : a.n;
  const long long most = p.items * ((keys + kTile - 1) / kTile) * (MULTI ? p.nts : 1);
  int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  if (most < ctas) ctas = static_cast<int>(most);
  if (MULTI) {
    p.part = static_cast<float*>(a.ws);
    p.joins = reinterpret_cast<int4*>(p.part + 2 * kMaxCtas * kTile);
  }
  p.w = static_cast<float*>(a.ws);
  mass_kernel<FP8, MULTI><<<ctas, kThreads, kSmem, stream>>>(p, map);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (a.idx) {
    const long long blocks = static_cast<long long>(a.B) * ((a.n + kSlice - 1) / kSlice);
    add_lists_kernel<<<static_cast<unsigned>(blocks), kAddThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  }
  if (!MULTI || ctas == 1) return DSA_OK;   // nothing is split
  // its blocks may be set up while the last CTAs finish; they wait for the parts
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas - 1);
  cfg.blockDim = dim3(kTile);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, p, ctas) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

size_t cache_mass_workspace(int B, int Sq, int H, int k) {
  if (k > 0) return static_cast<size_t>(B) * Sq * k * sizeof(float);
  if (static_cast<long long>(Sq) * H <= kTile) return 0;
  return 2 * kMaxCtas * kTile * sizeof(float) + kMaxCtas * sizeof(int4);
}

int launch_cache_mass(const MassArgs& a, int fmt, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  const bool multi = !a.idx && static_cast<long long>(a.Sq) * a.H > kTile;
  if (fmt == DSA_CACHE_E4M3)
    return multi ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return multi ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace dsa
