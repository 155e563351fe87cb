// Eviction from the paged latent cache by accumulated attention weight: choosing the positions that
// stay (dsa_cache_keep) and moving their rows (dsa_cache_compact). The weights themselves come from
// mass.cu.
//
// Choosing. A cluster of CTAs has a sequence, each CTA an even slice of the positions that go by
// their weight. The weights are mapped to integers that order like them and the budget's last one is
// found digit by digit (11, 11 and 10 bits): a histogram per CTA in shared memory, added up over the
// cluster through distributed shared memory. Ties at that value go to the lower positions: one pass
// over the slice counts, an exclusive sum over warps and CTAs places, one more writes. The weights are
// read from memory once and kept in shared memory as far as it holds them.
// Bound: latency. 64 sequences of up to 8192 weights (1 MB) take 9 us, 2 of 131072 20 us: the passes over
// the slice and the barriers between them.
//
// Moving. Rows are copied 16 bytes a thread; memory is the bound (64 x 2048 e4m3 rows 33 us, 4.7 TB/s read
// and written, 2 x 16384 bf16 rows 16.6 us, 4.6 TB/s, of which the first lookups take about 4; copies of
// whole rows by the bulk engine are level on the former, 31 us, and slower on the latter, 20). To other
// pages, all rows at once. In place (62 and 43 us: a chain of loads and a barrier per chunk of rows), row
// keep[j] goes to position j <= keep[j] and ascending lists never overwrite a row that is still to be read,
// as long as rows go in order: so a CTA takes a column slice of all rows of a sequence and walks down, the
// slices being independent of one another. Weights in place walk the same way, one CTA a sequence in front
// of the rows (66 and 59 us with them).

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kErrIdx = DSA_STAGE_EVICT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_EVICT | DSA_DEVERR_BAD_PAGE;

// ------------------------------------------------------------------ choosing

constexpr int kBins = 2048;
constexpr int kMostHeld = 49152;   // weights that a CTA keeps in shared memory (192 KB)

struct KeepParams {
  const float* mass;
  const int32_t* lens;
  int32_t *keep, *count;
  int n, budget, sink, recent;
  int held;   // weights per CTA that shared memory has room for
  int* err;
};

struct __align__(16) KeepTail {
  int hist[3][kBins];      // one per digit
  int above[32], equal[32];   // of each warp's part
  int2 total;              // of the CTA
  int sums[32];
  int shares[8];           // weights in each CTA's share of the bins
  int4 found;              // the digit, what is left to take of its bin, whether that is all of it
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Shared memory of another CTA. (No memory clobber: the loads of one histogram from all CTAs are on their
// way together; what they read is settled at the barrier in front of them, which no load passes.)
__device__ __forceinline__ uint32_t of_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int4 ld_cluster4(uint32_t a) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t a, int4 v) {
  asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ int2 ld_cluster2(uint32_t a) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// An integer that orders like the weight: -0 like +0, a NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int C, int kKeepThreads>   // CTAs of a cluster, threads of a CTA
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ KeepTail s;
  constexpr int kKeepWarps = kKeepThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C == 1 ? 0 : cluster_rank(), b = blockIdx.x / C;
  int len = __ldg(p.lens + b);
  if (len < 0 || len > p.n) {
    if (tid == 0) report_error(p.err, kErrPage);
    len = max(0, min(len, p.n));
  }
  int32_t* keep = p.keep + static_cast<long long>(b) * p.budget;
  const float* mass = p.mass + static_cast<long long>(b) * p.n;
  if (rank == 0 && tid == 0) p.count[b] = min(len, p.budget);
  if (len <= p.budget) {   // everything stays (the whole cluster leaves)
    for (int j = rank * kKeepThreads + tid; j < p.budget; j += C * kKeepThreads)
      keep[j] = j < len ? j : -1;
    return;
  }
  const int m = p.budget - p.sink - p.recent;   // to be chosen by weight
  for (int j = rank * kKeepThreads + tid; j < p.sink + p.recent; j += C * kKeepThreads) {
    if (j < p.sink)
      keep[j] = j;
    else
      keep[m + j] = len - (p.sink + p.recent) + j;
  }
  if (m == 0) return;

  // this CTA's slice of the positions between the first and the newest ones, m < all
  const int all = len - p.sink - p.recent;
  const int per = ((all + C - 1) / C + 31) / 32 * 32;
  const int at0 = min(all, rank * per), mine = min(all, at0 + per) - at0;
  mass += p.sink + at0;
  const bool held = per <= p.held;
  // the first weights, on their way while the histograms are cleared
  constexpr int kFirst = 8;
  float first[kFirst];
#pragma unroll
  for (int j = 0; j < kFirst; ++j)
    first[j] = tid + j * kKeepThreads < mine ? __ldg(mass + tid + j * kKeepThreads) : 0.f;
#pragma unroll
  for (int i = tid; i < 3 * kBins / 4; i += kKeepThreads)
    reinterpret_cast<int4*>(&s.hist[0][0])[i] = make_int4(0, 0, 0, 0);
  __syncthreads();
  auto take = [&](int i, float x) {
    const uint32_t k = order_key(x);
    if (held) keys[i] = k;
    atomicAdd(&s.hist[0][k >> 21], 1);
  };
#pragma unroll
  for (int j = 0; j < kFirst; ++j)
    if (tid + j * kKeepThreads < mine) take(tid + j * kKeepThreads, first[j]);
#pragma unroll 8
  for (int i = tid + kFirst * kKeepThreads; i < mine; i += kKeepThreads) take(i, __ldg(mass + i));
  // four weights from i on (a multiple of four; those behind the last one are 0)
  auto keys_at = [&](int i, uint32_t (&k)[4]) {
    if (held && i + 3 < mine) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      k[0] = v.x;
      k[1] = v.y;
      k[2] = v.z;
      k[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        k[j] = i + j < mine ? (held ? keys[i + j] : order_key(__ldg(mass + i + j))) : 0u;
    }
  };

  // the m-th heaviest: its digits, and how many of the equal ones are taken
  uint32_t found = 0;
  int left = m;
  bool exact = false;   // every weight with the digits found so far is taken
  int shift = 21;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    if (C == 1)
      __syncthreads();
    else
      cluster_sync();
    // Each CTA adds up a share of the bins over the cluster, the first one the topmost, four bins a
    // thread; then all know each share's weights, and the one that the border is in finds it.
    // (Every CTA of eight reading all bins of all took 8000 cycles a digit; with two, that is what they do:
    // 2500 cycles instead of 4200.)
    constexpr bool kShared = C > 2;
    const int bins = d == 2 ? 1024 : 2048, share = kShared ? bins / C : bins;
    const int low4 = bins - (kShared ? rank * share : 0) - 4 - 4 * tid;
    int c[4] = {0, 0, 0, 0};
    if (tid < share / 4) {
      int4 v[C];
#pragma unroll
      for (int r = 0; r < C; ++r)
        v[r] = C == 1 ? *reinterpret_cast<const int4*>(&s.hist[d][low4]) : ld_cluster4(of_cta(&s.hist[d][low4], r));
#pragma unroll
      for (int r = 0; r < C; ++r) {
        c[0] += v[r].w;
        c[1] += v[r].z;
        c[2] += v[r].y;
        c[3] += v[r].x;
      }
    }
    const int own = (c[0] + c[1]) + (c[2] + c[3]);
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? s.sums[lane] : 0) + incl - own;
    if (kShared) {
      if (warp == 0) {
        const int total = __reduce_add_sync(0xffffffffu, lane < kKeepWarps ? s.sums[lane] : 0);
        if (lane < C) st_cluster(of_cta(&s.shares[rank], lane), total);
      }
      cluster_sync();
      before += __reduce_add_sync(0xffffffffu, lane < rank ? s.shares[lane & 7] : 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < left && before + c[j] >= left) {
        const int4 f = make_int4(low4 + 3 - j, left - before, before + c[j] == left, 0);
        if (!kShared)
          s.found = f;
        else
          for (int r = 0; r < C; ++r) st_cluster4(of_cta(&s.found, r), f);
      }
      before += c[j];
    }
    if (kShared)
      cluster_sync();
    else
      __syncthreads();
    found = (found << (d == 2 ? 10 : 11)) | static_cast<uint32_t>(s.found.x);
    left = s.found.y;
    exact = s.found.z != 0;
    if (d == 2 || exact) break;
    const int next = d == 0 ? 10 : 0;   // the next digit's lowest bit
    for (int i = tid * 4; i < (mine + 127) / 128 * 128; i += 4 * kKeepThreads) {
      uint32_t k[4];
      keys_at(i, k);   // (a key of 0 is no weight's)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = k[j] != 0 && k[j] >> shift == found;
        const uint32_t lanes = __ballot_sync(0xffffffffu, in);
        if (lanes == 0) continue;
        const uint32_t bin = (k[j] >> next) & (d == 0 ? 2047u : 1023u);
        // equal weights fall into one bin: the lanes with the same one count together
        const uint32_t first_bin = __shfl_sync(0xffffffffu, bin, __ffs(lanes) - 1);
        const uint32_t same = __ballot_sync(0xffffffffu, in && bin == first_bin);
        if (lane == __ffs(lanes) - 1) atomicAdd(&s.hist[d + 1][bin], __popc(same));
        if (in && bin != first_bin) atomicAdd(&s.hist[d + 1][bin], 1);
      }
    }
    shift = next;
  }
  const uint32_t low = found << shift;   // exact: the lightest that stays, or what is below it

  // counts of each warp's part, then what is in front of it
  const int part = ((per + 127) / 128 + kKeepWarps - 1) / kKeepWarps * 128;
  const int w0 = min(mine, warp * part), w1 = min(mine, w0 + part);
  auto above = [&](uint32_t k) { return k != 0 && (exact ? k >= low : k > low); };
  auto equal = [&](uint32_t k) { return !exact && k == low && k != 0; };
  int na = 0, ne = 0;
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    uint32_t k[4];
    keys_at(i, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      na += above(k[j]);
      ne += equal(k[j]);
    }
  }
  na = __reduce_add_sync(0xffffffffu, na);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    s.above[warp] = na;
    s.equal[warp] = ne;
  }
  __syncthreads();
  if (warp == 0) {
    const int a = __reduce_add_sync(0xffffffffu, lane < kKeepWarps ? s.above[lane] : 0);
    const int e = __reduce_add_sync(0xffffffffu, lane < kKeepWarps ? s.equal[lane] : 0);
    if (lane == 0) s.total = make_int2(a, e);
  }
  if (C == 1)
    __syncthreads();
  else
    cluster_sync();
  int fa = lane < warp ? s.above[lane] : 0, fe = lane < warp ? s.equal[lane] : 0;
  if (C > 1 && lane < rank) {
    const int2 t = ld_cluster2(of_cta(&s.total, lane));
    fa += t.x;
    fe += t.y;
  }
  fa = __reduce_add_sync(0xffffffffu, fa);
  fe = __reduce_add_sync(0xffffffffu, fe);
  for (int i0 = w0; i0 < w1; i0 += 128) {
    uint32_t k[4];
    keys_at(i0 + 4 * lane, k);
    // four weights a lane: how many of either kind are in front of the lane's, in the two halves of a word
    int mine4 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine4 += above(k[j]) + (equal(k[j]) << 16);
    int incl = mine4;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int a = fa + ((incl - mine4) & 0xffff), e = fe + ((incl - mine4) >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool is_above = above(k[j]), is_equal = equal(k[j]);
      if (is_above || (is_equal && e < left)) keep[p.sink + a + min(e, left)] = p.sink + at0 + i0 + 4 * lane + j;
      a += is_above;
      e += is_equal;
    }
    const int all4 = __shfl_sync(0xffffffffu, incl, 31);
    fa += all4 & 0xffff;
    fe += all4 >> 16;
  }
  if (C > 1) cluster_sync();   // no CTA leaves while another may still read its counts
}

// ------------------------------------------------------------------ moving

constexpr int kMoveThreads = 256, kMoveRows = 8;   // rows of a warp
// 16-byte pieces per lane at a time: three rounds are the 576 of eight bf16 rows. 64 x 2048 e4m3 and 2 x
// 16384 bf16 rows: 8 rows and 6 pieces 32.8 and 16.1 us, 16 and 6 31.5 and 18.4, 16 and 8 39.0 and 23.8,
// 8 and 11 41.3 and 24.9.
constexpr int kMoveDepth = 6;
constexpr int kWalkThreads = 512;
constexpr int kWalkDepth = 4;   // 16-byte pieces per thread and chunk

struct MoveParams {
  uint8_t* cache;
  const int32_t *page_table, *lens, *keep, *new_table;
  const float* mass;           // moved with the rows, or nullptr
  float *new_mass, *tail;      // tail: new_mass where its rows' ends are to be cleared
  long long num_pages, rows;   // rows: B * budget
  int page_size, max_pages, new_max_pages, budget, upr;   // upr: 16-byte units per row
  int page_shift;              // log2 of the page size, -1 where it is no power of two
  int n, new_n;                // columns of mass and new_mass
  int B, unit_slice;
  int* err;
};

__device__ __forceinline__ int seq_len(const MoveParams& p, int b) {
  const int cap = p.max_pages * p.page_size;
  const int len = __ldg(p.lens + b);
  if (len < 0 || len > cap) report_error(p.err, kErrPage);
  return max(0, min(len, cap));
}

// the page that position j is in, of its sequence's
__device__ __forceinline__ int page_of(const MoveParams& p, int j) {
  return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
}

// the slot of position j, -1 where its page is not one of the cache
__device__ __forceinline__ long long slot_of(const MoveParams& p, const int32_t* table, int j) {
  const int pg = page_of(p, j);
  const int page = __ldg(table + pg);
  if (page < 0 || page >= p.num_pages) {
    report_error(p.err, kErrPage);
    return -1;
  }
  return static_cast<long long>(page) * p.page_size + (j - pg * p.page_size);
}

// a list entry, -1 where it names no row
__device__ __forceinline__ int entry(const MoveParams& p, long long row, int len) {
  const int e = __ldg(p.keep + row);
  if (e < -1 || e >= len) {
    report_error(p.err, kErrIdx);
    return -1;
  }
  return e;
}

// zeros behind the budget in every row of new_mass, shared out among the blocks
__device__ __forceinline__ void clear_tails(const MoveParams& p, long long block, long long blocks) {
  if (p.tail == nullptr || p.new_n <= p.budget) return;
  const int tail = p.new_n - p.budget;
  const long long count = static_cast<long long>(p.B) * tail, each = (count + blocks - 1) / blocks;
  const long long end = min(count, (block + 1) * each);
  for (long long i = block * each + threadIdx.x; i < end; i += blockDim.x) {
    const long long b = i / tail;
    p.tail[b * p.new_n + p.budget + (i - b * tail)] = 0.f;
  }
}

// To other pages: a warp takes kMoveRows rows. A lane each looks them up (list entry, pages, slots: three
// waits for memory), then the warp copies their 16-byte pieces one after the other, whatever rows they
// are of, kMoveDepth a lane at a time. (A block per 32 rows with the slots in shared memory: 34.2 us for
// 64 x 2048 e4m3 rows.)
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  const int lane = threadIdx.x & 31;
  const long long warp = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const long long row = warp * kMoveRows + lane;
  int src = -1, dst = -1;   // slots (below 2^31)
  if (lane < kMoveRows && row < p.rows) {
    const int b = static_cast<int>(row / p.budget), j = static_cast<int>(row - static_cast<long long>(b) * p.budget);
    const int e = entry(p, row, seq_len(p, b));
    float w = 0.f;
    if (e >= 0) {
      src = static_cast<int>(slot_of(p, p.page_table + static_cast<long long>(b) * p.max_pages, e));
      dst = static_cast<int>(slot_of(p, p.new_table + static_cast<long long>(b) * p.new_max_pages, j));
      if (src < 0) dst = -1;
      if (dst < 0) src = -1;
      if (p.mass) {
        if (e < p.n)
          w = __ldg(p.mass + static_cast<long long>(b) * p.n + e);
        else
          report_error(p.err, kErrIdx);   // a row without a weight
      }
    }
    if (p.mass) p.new_mass[static_cast<long long>(b) * p.new_n + j] = w;
  }
  const uint4* in = reinterpret_cast<const uint4*>(p.cache);
  uint4* out = reinterpret_cast<uint4*>(p.cache);
  const uint32_t upr = p.upr, units = kMoveRows * upr;
  // u / upr as (u magic) >> 20: magic is at most one above 2^20 / upr, so the quotient is right as long as
  // u upr < 2^20
  constexpr uint32_t kMostPieces = 2 * (kCacheMostDc + kCacheMostDr) / 16;   // of the widest row, in bf16
  static_assert(kMoveRows * kMostPieces * kMostPieces <= 1u << 20, "the division of a warp's pieces");
  const uint32_t magic = (1u << 20) / upr + 1;
#pragma unroll 1
  for (uint32_t u0 = lane; u0 < units + lane; u0 += 32 * kMoveDepth) {   // the same for every lane
    uint4 v[kMoveDepth];
#pragma unroll
    for (int k = 0; k < kMoveDepth; ++k) {
      const uint32_t u = u0 + 32 * k, r = (u * magic) >> 20, c = u - r * upr;
      const int s = __shfl_sync(0xffffffffu, src, r);   // (past the last row: a lane without one)
      if (u < units && s >= 0) v[k] = __ldcs(in + static_cast<long long>(s) * upr + c);
    }
#pragma unroll
    for (int k = 0; k < kMoveDepth; ++k) {
      const uint32_t u = u0 + 32 * k, r = (u * magic) >> 20, c = u - r * upr;
      const int d = __shfl_sync(0xffffffffu, dst, r);
      if (u < units && d >= 0) out[static_cast<long long>(d) * upr + c] = v[k];
    }
  }
  clear_tails(p, blockIdx.x, gridDim.x);
}

// In place: block (slice, b) walks down the rows of sequence b, chunk after chunk of kWalkDepth rows a
// thread (of `per` threads). List entries are read three chunks ahead, pages two, pieces one.
template <int T>
__global__ void __launch_bounds__(T) walk_kernel(const MoveParams p) {
  const int b = blockIdx.y, per = p.unit_slice;
  const int u = blockIdx.x * per + threadIdx.x % per;
  const int step = T / per, chunk = step * kWalkDepth, j0 = threadIdx.x / per;
  const int len = seq_len(p, b);
  const int32_t* table = p.page_table + static_cast<long long>(b) * p.max_pages;
  const int32_t* list = p.keep + static_cast<long long>(b) * p.budget;
  uint4* data = reinterpret_cast<uint4*>(p.cache);
  const int end = u < p.upr ? min(p.budget, len) : 0;   // row j comes from a position j or later
  // the rows that move: their entries (-1: none), pages, then pieces and where they go (a slot, or -1)
  int e[kWalkDepth], from[kWalkDepth], to[kWalkDepth], at[kWalkDepth], dst[2][kWalkDepth];
  uint4 v[2][kWalkDepth];
  auto entries = [&](int c) {
#pragma unroll
    for (int k = 0; k < kWalkDepth; ++k) {
      const int j = c * chunk + k * step + j0;
      e[k] = j < end ? __ldg(list + j) : -1;
    }
  };
  auto pages = [&](int c) {
#pragma unroll
    for (int k = 0; k < kWalkDepth; ++k) {
      const int j = c * chunk + k * step + j0;
      at[k] = -1;
      if (e[k] == -1 || e[k] == j) continue;
      if (e[k] < j || e[k] >= len) {   // outside the sequence, or not an ascending list
        report_error(p.err, kErrIdx);
        continue;
      }
      at[k] = e[k];
      from[k] = __ldg(table + page_of(p, e[k]));
      to[k] = __ldg(table + page_of(p, j));
    }
  };
  auto pieces = [&](int c, uint4 (&x)[kWalkDepth], int (&d)[kWalkDepth]) {
#pragma unroll
    for (int k = 0; k < kWalkDepth; ++k) {
      const int j = c * chunk + k * step + j0;
      d[k] = -1;
      if (at[k] < 0) continue;
      if (from[k] < 0 || from[k] >= p.num_pages || to[k] < 0 || to[k] >= p.num_pages) {
        report_error(p.err, kErrPage);
        continue;
      }
      // (a slot is below 2^31; a page's first one and the position together may be past it)
      const int src = from[k] * p.page_size + (at[k] - page_of(p, at[k]) * p.page_size);
      d[k] = to[k] * p.page_size + (j - page_of(p, j) * p.page_size);
      x[k] = data[static_cast<long long>(src) * p.upr + u];
    }
  };
  auto store = [&](const uint4 (&x)[kWalkDepth], const int (&d)[kWalkDepth]) {
#pragma unroll
    for (int k = 0; k < kWalkDepth; ++k)
      if (d[k] >= 0) data[static_cast<long long>(d[k]) * p.upr + u] = x[k];
  };
  // What chunk c + 1 reads lies behind all that chunks up to c write, so its loads go first; what
  // chunk c reads may be what it writes itself, so a barrier parts the two.
  const int chunks = (min(p.budget, len) + chunk - 1) / chunk;   // the same for every thread
  if (blockIdx.x == 0)   // behind the sequence's end there are no rows to name
    for (int j = len + threadIdx.x; j < p.budget; j += T)
      if (__ldg(list + j) != -1) report_error(p.err, kErrIdx);
  entries(0);
  pages(0);
  entries(1);
  pieces(0, v[0], dst[0]);
  pages(1);
  entries(2);
#pragma unroll 1
  for (int c = 0; c < chunks; c += 2) {
    __syncthreads();
    pieces(c + 1, v[1], dst[1]);
    pages(c + 2);
    entries(c + 3);
    store(v[0], dst[0]);
    __syncthreads();
    pieces(c + 2, v[0], dst[0]);
    pages(c + 3);
    entries(c + 4);
    store(v[1], dst[1]);
  }
  clear_tails(p, static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x,
              static_cast<long long>(gridDim.x) * gridDim.y);
}

// The weights of sequence b, walked down the same way (new_mass may be mass). The kernel that moves the
// rows comes after it and clears what is behind them.
__global__ void __launch_bounds__(kWalkThreads) walk_mass_kernel(const MoveParams p) {
  const int b = blockIdx.x;
  const int len = seq_len(p, b);
  const float* mass = p.mass + static_cast<long long>(b) * p.n;
  float* out = p.new_mass + static_cast<long long>(b) * p.new_n;
  constexpr int kDepth = 8, kChunk = kWalkThreads * kDepth;
  for (int j0 = 0; j0 < p.budget; j0 += kChunk) {
    float x[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      const int j = j0 + k * kWalkThreads + threadIdx.x;
      x[k] = 0.f;
      if (j < p.budget) {
        const int e = entry(p, static_cast<long long>(b) * p.budget + j, len);
        if (e >= j && e < p.n)
          x[k] = mass[e];
        else if (e >= 0)   // overwritten by now, or a row without a weight
          report_error(p.err, kErrIdx);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      const int j = j0 + k * kWalkThreads + threadIdx.x;
      if (j < p.budget) out[j] = x[k];
    }
  }
}

}  // namespace

namespace {

template <int C, int kKeepThreads>
int launch_keep(const KeepParams& p, int B, cudaStream_t stream) {
  if (static_cast<long long>(B) * C > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(keep_kernel<C, kKeepThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMostHeld * 4) != cudaSuccess)
    return DSA_ERR_CUDA;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * C);
  cfg.blockDim = dim3(kKeepThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.held) * 4;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, keep_kernel<C, kKeepThreads>, p) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

int launch_cache_keep(const float* mass, int n, const int32_t* lens, int B, int budget, int sink,
                      int recent, int32_t* keep, int32_t* count, cudaStream_t stream) {
  KeepParams p = {mass, lens, keep, count, n, budget, sink, recent, 0, device_error_word()};
  // More CTAs a cluster share out the passes over the weights and pay for it at the barriers, and dearly as
  // soon as not all of them are resident at once. With 1 / 2 / 4 / 8 CTAs, us from a graph: 2 x 131072
  // weights 126 / 101 / 27.5 / 19.5 (up to 49152 a CTA stay in shared memory), 16 x 32768 23 / 18.6 / 13.7 /
  // 19.0, 64 x 8192 10.9 / 9.5 / 18.7 / 42, 128 x 4096 7.1 / 9.8 / 32 / 74. Between these sizes the rule may
  // take half of what would be quickest: 4 x 65536 four (19.2; eight 14.3), 32 x 16384 two (13.1; four 11.5).
  int C = 1;
  while (C < 8 && n / C > 4096 * C && 2ll * C * B <= 304) C *= 2;
  const int per = ((n + C - 1) / C + 31) / 32 * 32;
  p.held = per <= kMostHeld ? per : 0;
  switch (C) {
    case 8: return launch_keep<8, 1024>(p, B, stream);
    case 4: return launch_keep<4, 1024>(p, B, stream);
    case 2: return launch_keep<2, 512>(p, B, stream);
    // (many long sequences: one CTA each)
    default: return per > 8192 ? launch_keep<1, 1024>(p, B, stream) : launch_keep<1, 512>(p, B, stream);
  }
}

int launch_cache_compact(const CompactArgs& a, cudaStream_t stream) {
  MoveParams p = {};
  p.cache = a.cache;
  p.page_table = a.page_table;
  p.lens = a.lens;
  p.keep = a.keep;
  p.new_table = a.new_table;
  p.num_pages = a.num_pages;
  p.rows = static_cast<long long>(a.B) * a.budget;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.new_max_pages = a.new_max_pages;
  p.budget = a.budget;
  p.upr = a.row_bytes / 16;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.n = a.n;
  p.new_n = a.new_n;
  p.B = a.B;
  p.err = device_error_word();
  p.tail = a.mass ? a.new_mass : nullptr;
  const long long per = kMoveThreads / 32 * kMoveRows, blocks = (p.rows + per - 1) / per;
  if (a.new_table && blocks > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;   // before anything is launched
  const bool walk_mass = a.mass && (!a.new_table || a.new_mass == a.mass);
  if (walk_mass) {
    MoveParams w = p;
    w.mass = a.mass;
    w.new_mass = a.new_mass;
    walk_mass_kernel<<<a.B, kWalkThreads, 0, stream>>>(w);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  } else {
    p.mass = a.mass;
    p.new_mass = a.new_mass;
  }
  if (a.new_table) {
    move_kernel<<<static_cast<unsigned>(blocks), kMoveThreads, 0, stream>>>(p);
  } else {
    p.unit_slice = 8;
    while (p.unit_slice > 2 && static_cast<long long>(a.B) * (p.upr / p.unit_slice) < 304)
      p.unit_slice /= 2;
    const dim3 grid((p.upr + p.unit_slice - 1) / p.unit_slice, a.B);
    // few blocks: as many threads as a block can have
    if (static_cast<long long>(grid.x) * a.B <= 152)
      walk_kernel<1024><<<grid, 1024, 0, stream>>>(p);
    else
      walk_kernel<256><<<grid, 256, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
