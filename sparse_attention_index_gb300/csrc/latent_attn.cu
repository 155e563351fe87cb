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
// Warp-specialised CTA, 416 threads:
//   warps 0-3   softmax / output: one (token, head) row per thread
//   warp  4     TMEM owner and single-thread UMMA issuer
//   warps 5-12  gather, six keys of each chunk per warp: page lookup two chunks ahead, then
//               16-byte cp.async into 128B-swizzled tiles. An e4m3 row goes through a raw ring
//               (each thread copies in what it will convert itself, so no barrier is needed)
//               and is widened to bf16, exactly, since its scales are powers of two.
// TMEM: [Q: 144][S/P: 2 x 48][pad 16][O: 256] = 512 columns.

#include <mutex>

#include "dsa_common.cuh"
#include "dsa_internal.h"

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
constexpr int kGatherWarp0 = 5, kGatherWarps = 8;
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr int kKeysPerWarp = kNK / kGatherWarps;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);
constexpr uint32_t kColQ = 0, kColS = 144, kColO = 256;
constexpr int kMinChunks = 4;            // chunks that a cluster takes at least
constexpr int kMaxClusters = 80;         // clusters that the workspace has room for
constexpr float kRescaleLog2 = 8.f;      // refresh the running max when it grows by > 2^8
constexpr int kErrIdx = DSA_STAGE_LATENT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_LATENT | DSA_DEVERR_BAD_PAGE;
constexpr int kErrTime = DSA_STAGE_LATENT | DSA_DEVERR_TIMEOUT;
static_assert(kKeysPerWarp * kGatherWarps == kNK, "six keys per gather warp");

// e4m3: 48 keys x 16 pieces of 16 codes, three per gather thread, each with its scale, and
// 48 x 4 pieces of positional dims
constexpr int kCodeReps = kNK * (kHalf / 16) / kGatherThreads;
constexpr uint32_t kRawScale = kCodeReps * kGatherThreads * 16;
constexpr uint32_t kRawRope = kRawScale + kCodeReps * kGatherThreads * 4;
constexpr uint32_t kRaw = kRawRope + kNK * (kHalfR / 8) * 16;
constexpr int kRawStages = 4;

template <bool FP8>
struct Layout {
  static constexpr int kStages = FP8 ? 3 : 5;
  static constexpr uint32_t kExchOff = kStages * kStage;
  static constexpr uint32_t kRawOff = kExchOff + 2 * kExch;
  static constexpr uint32_t kTailOff = kRawOff + (FP8 ? kRawStages * kRaw : 0);
};

struct Header {
  int item;    // tile
  int c;       // chunk of the tile
  int lim0;    // keys that the tile's first row sees (every cached key); unused with lists
  int flags;   // 1: first chunk of the tile here, 2: last one here, 4: the whole tile is here
  uint8_t valid[kGatherWarps];   // six keys each
};

struct Tail {
  Header hdr[5];
  uint64_t kv_full[5], kv_empty[5];
  uint64_t s_full[2], s_empty[2], p_full[2], x_full[2];
  uint64_t q_full, o_free, drain;
  uint32_t tmem_base;
  int abort_flag;
  long long sums[kThreads / 32];
  // this cluster's range: its first tile, that tile's first chunk here, chunks in all
  int item0, c0, n;
};

struct Params {
  LatentArgs a;
  int tiles;        // tiles per sequence (lists: one per token, B * Sq in all)
  int items;
  int list_chunks;  // chunks of a list (lists only)
  int clusters;
  int act_warps;    // softmax warps with rows
  int prow;         // rows of a workspace part (32 * act_warps)
  float scale_log2;
  float4* part;     // [2 * clusters][128 groups of 4 dims][prow]
  float2* ml;       // [2 * clusters][prow]: running max (scaled, log2) and sum
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

// keys that the last row of a tile sees
__device__ __forceinline__ int tile_keys(const Params& p, int len, int mt) {
  const int i1 = (mt * 128 + tile_rows(p, mt) - 1) / p.a.H;
  return max(0, len - p.a.Sq + i1 + 1);
}

// a tile without a key has one (empty) chunk, which writes its rows
__device__ __forceinline__ int chunks_of(int keys) { return keys > 0 ? (keys + kNK - 1) / kNK : 1; }

__device__ __forceinline__ int item_chunks(const Params& p, int item) {
  if (p.a.idx) return p.list_chunks;
  const int b = item / p.tiles;
  return chunks_of(tile_keys(p, seq_len(p.a, b, false), item - b * p.tiles));
}

struct Place {
  int item;
  long long start;   // first chunk of the tile among all chunks
};

// Chunks of all tiles; with at >= 0, also the tile that chunk `at` lies in. Every thread of the
// block calls it.
__device__ __forceinline__ long long total_chunks(const Params& p, long long* sums) {
  if (p.a.idx) return static_cast<long long>(p.items) * p.list_chunks;
  const int q = (p.items + blockDim.x - 1) / blockDim.x;
  const int i0 = min(p.items, static_cast<int>(threadIdx.x) * q), i1 = min(p.items, i0 + q);
  long long s = 0;
  for (int i = i0; i < i1; ++i) s += item_chunks(p, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += sums[w];
  return s;
}

// the tile that chunk `at` lies in, in the one thread that finds it (true there)
__device__ __forceinline__ bool find_item(const Params& p, long long at, const long long* sums,
                                          Place& out) {
  if (p.a.idx) {
    out.item = static_cast<int>(at / p.list_chunks);
    out.start = static_cast<long long>(out.item) * p.list_chunks;
    return threadIdx.x == 0;
  }
  const int q = (p.items + blockDim.x - 1) / blockDim.x;
  const int i0 = min(p.items, static_cast<int>(threadIdx.x) * q), i1 = min(p.items, i0 + q);
  const int lane = threadIdx.x & 31;
  long long s = 0;
  for (int i = i0; i < i1; ++i) s += item_chunks(p, i);
  long long incl = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  long long before = incl - s;
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) before += sums[w];
  if (at < before || at >= before + s) return false;
  for (int i = i0; i < i1; ++i) {
    const int n = item_chunks(p, i);
    if (at < before + n) {
      out.item = i;
      out.start = before;
      return true;
    }
    before += n;
  }
  return false;
}

__device__ __forceinline__ long long chunks_each(const Params& p, long long total) {
  return max((total + p.clusters - 1) / p.clusters, static_cast<long long>(kMinChunks));
}

// ------------------------------------------------------------------ small helpers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
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

// mbar_wait for data that the peer CTA sends
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

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four e4m3 bytes to bf16. The 7 magnitude bits, moved to the top of the bf16 mantissa and the
// bottom of its exponent, are the value times 2^-120 (biases 127 and 7; the subnormals of one are
// subnormals of the other), so one exact multiply by 2^(120 + k) widens and scales. `up` holds
// that power twice, `more` what it lacks above 2^127 (1 but for k > 7).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t up, uint32_t more, uint32_t& lo,
                                       uint32_t& hi) {
  const uint32_t t0 = __byte_perm(w, 0, 0x1404), t1 = __byte_perm(w, 0, 0x3424);
  lo = mul_bf16x2((t0 & 0x80008000u) | ((t0 >> 4) & 0x07f007f0u), up);
  hi = mul_bf16x2((t1 & 0x80008000u) | ((t1 >> 4) & 0x07f007f0u), up);
  if (more != 0x3f803f80u) {
    lo = mul_bf16x2(lo, more);
    hi = mul_bf16x2(hi, more);
  }
}

// ------------------------------------------------------------------ the kernel

// where a gather warp stands in its cluster's chunks
struct Cursor {
  int item, c, nch, len, keys, b, mt;
};

__device__ __forceinline__ void enter_item(const Params& p, int item, Cursor& k) {
  k.item = item;
  if (p.a.idx) {
    k.b = item / p.a.Sq;
    k.mt = item - k.b * p.a.Sq;   // the token
    k.len = seq_len(p.a, k.b, true);
    k.keys = max(0, k.len - p.a.Sq + k.mt + 1);
    k.nch = p.list_chunks;
  } else {
    k.b = item / p.tiles;
    k.mt = item - k.b * p.tiles;
    k.len = seq_len(p.a, k.b, true);
    k.keys = tile_keys(p, k.len, k.mt);
    k.nch = chunks_of(k.keys);
  }
}

template <bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const Params p) {
  using L = Layout<FP8>;
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
    for (int i = 0; i < L::kStages; ++i) {
      // every gather thread when its part has landed, and one per gather warp for the header
      mbar_init(&tail->kv_full[i], kGatherThreads + kGatherWarps);
      mbar_init(&tail->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->s_full[i], 1);
      mbar_init(&tail->s_empty[i], 1);
      mbar_init(&tail->p_full[i], 128);
      mbar_init(&tail->x_full[i], 1);
    }
    mbar_init(&tail->q_full, 128);
    mbar_init(&tail->o_free, 128);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    tail->n = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(&tail->tmem_base, 512);
    tmem_relinquish();
  }
  {
    // this cluster's range of chunks
    const long long total = total_chunks(p, tail->sums);
    const long long each = chunks_each(p, total);
    const long long g0 = each * cluster;
    if (g0 < total) {
      Place at;
      if (find_item(p, g0, tail->sums, at)) {
        tail->item0 = at.item;
        tail->c0 = static_cast<int>(g0 - at.start);
        tail->n = static_cast<int>(min(each, total - g0));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();   // the peer's barriers are ready
  const uint32_t tmem = tail->tmem_base;
  const int n = tail->n, item0 = tail->item0, c0 = tail->c0;

  if (n == 0) {
    // nothing here (both CTAs agree)
  } else if (warp >= kGatherWarp0) {
    // ================================================================ gather
    const int gw = warp - kGatherWarp0, gt = threadIdx.x - 32 * kGatherWarp0;
    const int mykey = gw * kKeysPerWarp + lane;   // lanes 0-5: the chunk's key of this lane
    const bool holder = lane < kKeysPerWarp;
    const long long row_bytes = FP8 ? kDc + 16 + 2 * kDr : 2 * kD;
    Cursor k;
    enter_item(p, item0, k);
    k.c = c0;
    int made = 0;   // chunks handed out by next()
    // the lane's position in the next chunk (-1: no key), with the chunk's header
    struct Ahead {
      int pos, b, item, c, lim0, flags;
    };
    auto next = [&]() {
      Ahead h;
      h.pos = -1;
      h.b = k.b;
      h.item = k.item;
      h.c = k.c;
      h.flags = 0;
      h.lim0 = 0;
      if (made >= n) return h;
      const bool first = made == 0 || k.c == 0;
      const bool last = made == n - 1 || k.c == k.nch - 1;
      h.flags = (first ? 1 : 0) | (last ? 2 : 0);
      // the whole tile is in this range: its first chunk was here, and its last one is
      if (k.c <= made && k.nch - k.c <= n - made) h.flags |= 4;
      h.lim0 = k.len - p.a.Sq + 1 + (p.a.idx ? 0 : (k.mt * 128) / p.a.H);
      if (holder) {
        const int j = k.c * kNK + mykey;
        if (p.a.idx) {
          if (j < p.a.k) {
            const int s = __ldg(p.a.idx + static_cast<long long>(k.item) * p.a.k + j);
            if (s < -1 || s >= k.len)
              report_error(err, kErrIdx);
            else if (s < k.keys)
              h.pos = s;
          }
        } else if (j < k.keys) {
          h.pos = j;
        }
      }
      ++made;
      if (made < n && ++k.c == k.nch) {
        enter_item(p, k.item + 1, k);
        k.c = 0;
      }
      return h;
    };
    // the page of a position, then its slot
    auto page_of = [&](const Ahead& h) {
      return h.pos >= 0 ? __ldg(p.a.page_table + static_cast<long long>(h.b) * p.a.max_pages +
                                h.pos / p.a.page_size)
                        : -1;
    };
    auto slot_of = [&](const Ahead& h, int page) {
      if (h.pos < 0) return -1;
      if (page < 0 || page >= p.a.num_pages) {
        report_error(err, kErrPage);
        return -1;
      }
      return page * p.a.page_size + h.pos % p.a.page_size;
    };
    const uint32_t base = smem_u32(smem);
    Ahead h0 = next();
    int page0 = page_of(h0);
    Ahead h1 = next();
    int slot = slot_of(h0, page0);

    if (!FP8) {
      for (int g = 0; g < n; ++g) {
        const int page1 = page_of(h1);
        const Ahead h2 = next();
        const int st = g % L::kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->kv_empty[st], ((g / L::kStages) & 1) ^ 1u,
                                               abort_flag, err, kErrTime)))
          break;
        const uint32_t bal = __ballot_sync(0xffffffffu, holder && slot >= 0);
        if (lane == 0) {
          Header& h = tail->hdr[st];
          h.valid[gw] = static_cast<uint8_t>(bal);
          if (gw == 0) {
            h.item = h0.item;
            h.c = h0.c;
            h.lim0 = h0.lim0;
            h.flags = h0.flags;
          }
          mbar_arrive(&tail->kv_full[st]);
        }
        const uint32_t stage = base + st * kStage;
#pragma unroll
        for (int i = 0; i < kKeysPerWarp; ++i) {
          const int s = __shfl_sync(0xffffffffu, slot, i);
          const int key = gw * kKeysPerWarp + i;
          const uint8_t* src = p.a.cache + (s >= 0 ? s : 0) * row_bytes + rank * (2 * kHalf);
          cp_async_16(stage + (lane >> 3) * kAtom + key * 128 + (((lane & 7) ^ (key & 7)) << 4),
                      src + lane * 16, s >= 0 ? 16u : 0u);
        }
        {
          const int i = lane >> 2, pc = lane & 3;   // four pieces of positional dims per key
          const int s = __shfl_sync(0xffffffffu, slot, i < kKeysPerWarp ? i : 0);
          const int key = gw * kKeysPerWarp + i;
          const uint8_t* src =
              p.a.cache + (s >= 0 ? s : 0) * row_bytes + 2 * kDc + rank * (2 * kHalfR);
          if (i < kKeysPerWarp)
            cp_async_16(stage + 4 * kAtom + key * 128 + ((pc ^ (key & 7)) << 4), src + pc * 16,
                        s >= 0 ? 16u : 0u);
        }
        cp_async_mbar_arrive(&tail->kv_full[st]);
        slot = slot_of(h1, page1);
        h0 = h1;
        h1 = h2;
      }
      cp_async_wait<0>();
    } else {
      // raw ring: chunk g's codes, scales and positional dims in slots of this thread's own
      const uint32_t raw = base + L::kRawOff;
      auto fetch = [&](int g, int sl) {
        const uint32_t rs = raw + (g % kRawStages) * kRaw;
#pragma unroll
        for (int j = 0; j < kCodeReps; ++j) {
          const int i = 2 * j + (lane >> 4), pc = lane & 15;   // two keys per instruction
          const int s = __shfl_sync(0xffffffffu, sl, i);
          const uint8_t* src = p.a.cache + (s >= 0 ? s : 0) * row_bytes;
          const uint32_t at = static_cast<uint32_t>(j) * kGatherThreads + gt;
          cp_async_16(rs + at * 16, src + rank * kHalf + pc * 16, s >= 0 ? 16u : 0u);
          cp_async_4(rs + kRawScale + at * 4, src + kDc + (rank * 2 + (pc >> 3)) * 4);
        }
        const int i = lane >> 2, pc = lane & 3;
        const int s = __shfl_sync(0xffffffffu, sl, i < kKeysPerWarp ? i : 0);
        const uint8_t* src =
            p.a.cache + (s >= 0 ? s : 0) * row_bytes + kDc + 16 + rank * (2 * kHalfR) + pc * 16;
        if (i < kKeysPerWarp)
          cp_async_16(rs + kRawRope + (gw * kKeysPerWarp * 4 + lane) * 16, src, s >= 0 ? 16u : 0u);
        cp_async_commit();
      };
      // chunks fetched ahead: their headers and key masks wait in registers
      Ahead hq[kRawStages - 1];
      uint32_t vq[kRawStages - 1];
#pragma unroll
      for (int d = 0; d < kRawStages - 1; ++d) {
        hq[d] = h0;
        vq[d] = __ballot_sync(0xffffffffu, holder && slot >= 0);
        if (d < n)
          fetch(d, slot);
        else
          cp_async_commit();
        const int page1 = page_of(h1);
        const Ahead h2 = next();
        slot = slot_of(h1, page1);
        h0 = h1;
        h1 = h2;
      }
      for (int g = 0; g < n; ++g) {
        const int page1 = page_of(h1);
        const Ahead h2 = next();
        const uint32_t bal = __ballot_sync(0xffffffffu, holder && slot >= 0);
        if (g + kRawStages - 1 < n)
          fetch(g + kRawStages - 1, slot);
        else
          cp_async_commit();
        const int st = g % L::kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->kv_empty[st], ((g / L::kStages) & 1) ^ 1u,
                                               abort_flag, err, kErrTime)))
          break;
        if (lane == 0) {
          Header& h = tail->hdr[st];
          h.valid[gw] = static_cast<uint8_t>(vq[0]);
          if (gw == 0) {
            h.item = hq[0].item;
            h.c = hq[0].c;
            h.lim0 = hq[0].lim0;
            h.flags = hq[0].flags;
          }
          mbar_arrive(&tail->kv_full[st]);
        }
        cp_async_wait<kRawStages - 1>();
        const uint8_t* rs = smem + L::kRawOff + (g % kRawStages) * kRaw;
        uint8_t* stage = smem + st * kStage;
#pragma unroll
        for (int j = 0; j < kCodeReps; ++j) {
          const int i = 2 * j + (lane >> 4), pc = lane & 15, key = gw * kKeysPerWarp + i;
          const int at = j * kGatherThreads + gt;
          const uint4 q = *reinterpret_cast<const uint4*>(rs + at * 16);
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(rs + kRawScale + at * 4);
          uint4 w[2];
          if ((vq[0] >> i) & 1u) {
            // 2^k as bf16 bits; 2^(120 + k), or 2^127 and the rest of it
            const uint32_t e = sc >> 16;
            uint32_t up = e + (120u << 7), more = 0x3f80u;
            if (e > (134u << 7)) {   // k > 7, or NaN
              up = e > 0x7f80u ? e : 254u << 7;
              more = e > 0x7f80u ? e : e - (7u << 7);
            }
            up |= up << 16;
            more |= more << 16;
            widen4(q.x, up, more, w[0].x, w[0].y);
            widen4(q.y, up, more, w[0].z, w[0].w);
            widen4(q.z, up, more, w[1].x, w[1].y);
            widen4(q.w, up, more, w[1].z, w[1].w);
          } else {
            w[0] = w[1] = make_uint4(0, 0, 0, 0);
          }
          // the two 16-byte halves, in the other order in every second atom: eight lanes then
          // store to eight different bank groups
          uint8_t* row = stage + (pc >> 2) * kAtom + key * 128;
          const int sw = (pc >> 2) & 1, c = (pc & 3) * 2;
          *reinterpret_cast<uint4*>(row + (((c + sw) ^ (key & 7)) << 4)) = sw ? w[1] : w[0];
          *reinterpret_cast<uint4*>(row + (((c + 1 - sw) ^ (key & 7)) << 4)) = sw ? w[0] : w[1];
        }
        if (lane < 4 * kKeysPerWarp) {
          const int key = gw * kKeysPerWarp + (lane >> 2), pc = lane & 3;
          *reinterpret_cast<uint4*>(stage + 4 * kAtom + key * 128 + ((pc ^ (key & 7)) << 4)) =
              *reinterpret_cast<const uint4*>(rs + kRawRope + (gw * kKeysPerWarp * 4 + lane) * 16);
        }
        fence_proxy_async_smem();
        mbar_arrive(&tail->kv_full[st]);
        slot = slot_of(h1, page1);
#pragma unroll
        for (int d = 0; d + 1 < kRawStages - 1; ++d) {
          hq[d] = hq[d + 1];
          vq[d] = vq[d + 1];
        }
        hq[kRawStages - 2] = h0;
        vq[kRawStages - 2] = bal;
        h0 = h1;
        h1 = h2;
      }
      cp_async_wait<0>();
    }
  } else if (warp == 4) {
    // ================================================================ UMMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16_mn(128, kNK, false);
      constexpr uint32_t idesc_pv = umma_idesc_bf16_mn(128, kHalf, true);
      const uint32_t base = smem_u32(smem);
      uint32_t q_par = 0, of_par = 1;
      int pend_flags = 0;
      // PV of chunk g (its P is awaited here)
      auto pv = [&](int g, int flags) {
        const int sb = g & 1, st = g % L::kStages;
        if (!mbar_wait(&tail->p_full[sb], (g >> 1) & 1, abort_flag, err, kErrTime)) return false;
        if (flags & 1) {   // the previous tile's O has been read out
          if (!mbar_wait(&tail->o_free, of_par, abort_flag, err, kErrTime)) return false;
          of_par ^= 1u;
        }
        tc_fence_after();
        const uint64_t v0 = umma_sdesc_lbo(base + st * kStage, kAtom, 1024, kLayoutSw128);
#pragma unroll
        for (int ks = 0; ks < kNK / 16; ++ks)
          umma_bf16_ts(tmem + kColO, tmem + kColS + sb * kNK + ks * 8, umma_desc_adv(v0, ks * 2048),
                       idesc_pv, ((flags & 1) && ks == 0) ? 0u : 1u);
        umma_commit(&tail->kv_empty[st]);
        umma_commit(&tail->s_empty[sb]);
        return true;
      };
      for (int g = 0; g < n; ++g) {
        const int st = g % L::kStages, sb = g & 1;
        if (!mbar_wait(&tail->kv_full[st], (g / L::kStages) & 1, abort_flag, err, kErrTime)) break;
        const int flags = tail->hdr[st].flags;
        if (flags & 1) {
          if (!mbar_wait(&tail->q_full, q_par, abort_flag, err, kErrTime)) break;
          q_par ^= 1u;
        }
        if (!mbar_wait(&tail->s_empty[sb], ((g >> 1) & 1) ^ 1u, abort_flag, err, kErrTime)) break;
        // cp.async wrote the rows through the generic proxy
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t k0 = umma_sdesc(base + st * kStage, 1024, kLayoutSw128);
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          umma_bf16_ts(tmem + kColS + sb * kNK, tmem + kColQ + kk * 8,
                       umma_desc_adv(k0, (kk >> 2) * kAtom + (kk & 3) * 32), idesc_s,
                       kk > 0 ? 1u : 0u);
        umma_commit(&tail->s_full[sb]);
        if (g > 0 && !(pend_flags & 2) && !pv(g - 1, pend_flags)) break;
        // a tile's last chunk: its PV right away, so that O is complete before the next tile
        if ((flags & 2) && !pv(g, flags)) break;
        pend_flags = flags;
      }
      umma_commit(&tail->drain);
      const uint32_t a = smem_u32(&tail->drain);
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(a, 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          report_error(err, kErrTime);
          break;
        }
      }
    }
  } else {
    // ================================================================ softmax / output
    const int hrow = threadIdx.x;   // TMEM lane = row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const bool act = warp < p.act_warps;
    const float c2 = p.scale_log2;
    const int H = p.a.H;
    const uint32_t peer = rank ^ 1u;
    const uint32_t x_bytes = p.act_warps * 32 * kNK * 4;
    // the tile's first row of Q / O / lse, and the rows it has
    auto rows_at = [&](int item, int& rows) {
      if (p.a.idx) {
        rows = H;
        return static_cast<long long>(item) * H;
      }
      const int b = item / p.tiles, mt = item - b * p.tiles;
      rows = tile_rows(p, mt);
      return static_cast<long long>(b) * p.a.Sq * H + mt * 128;
    };
    // this CTA's dims of the row of Q, packed bf16 pairs, into the thread's TMEM lane
    auto load_q = [&](int item) {
      if (act) {
        int rows;
        const long long r0 = rows_at(item, rows);
        const bool in = hrow < rows;
        const uint4* src = reinterpret_cast<const uint4*>(p.a.Q + (in ? r0 + hrow : 0) * kD);
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int a = 0; a < kSteps / 2; ++a) {   // 32 dims: 16 columns
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = a < kHalf / 32 ? rank * (kHalf / 8) + a * 4 + q
                                          : kDc / 8 + rank * (kHalfR / 8) + q;
            const uint4 x = in ? __ldg(src + at) : zero;
            w[4 * q] = x.x; w[4 * q + 1] = x.y; w[4 * q + 2] = x.z; w[4 * q + 3] = x.w;
          }
          tmem_st_x16(tmem + lane_off + kColQ + a * 16, w);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(&tail->q_full);
    };

    load_q(item0);
    float m = -INFINITY, l = 0.f;   // running max (raw logits) and sum
    int rows = 0, lim = 0;
    long long r0 = 0;
    for (int g = 0; g < n; ++g) {
      const int sb = g & 1, st = g % L::kStages;
      const uint32_t par = (g >> 1) & 1;
      if (threadIdx.x == 0) mbar_arrive_expect_tx(&tail->x_full[sb], x_bytes);
      bool ok = mbar_wait(&tail->s_full[sb], par, abort_flag, err, kErrTime);
      // acquires the gather warps' header writes
      ok = ok && mbar_wait(&tail->kv_full[st], (g / L::kStages) & 1, abort_flag, err, kErrTime);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const Header& h = tail->hdr[st];
      const int item = h.item, flags = h.flags, c = h.c;
      unsigned long long vm = 0;
#pragma unroll
      for (int w = 0; w < kGatherWarps; ++w)
        vm |= static_cast<unsigned long long>(h.valid[w]) << (w * kKeysPerWarp);
      if (flags & 1) {
        m = -INFINITY;
        l = 0.f;
        r0 = rows_at(item, rows);
        // keys that this row sees: the tile's first token sees lim0, each later one one more
        if (!p.a.idx) lim = h.lim0 + (static_cast<int>(r0 % H) + hrow) / H;
      }
      if (!p.a.idx) {
        const int left = lim - c * kNK;   // keys of the chunk that the row sees
        if (left < kNK) vm = left <= 0 ? 0ull : vm & ((1ull << left) - 1);
      }
      if (act) {
        const uint32_t sbase = tmem + lane_off + kColS + sb * kNK;
        float s[kNK];
        {
          uint32_t lo[32], hi[16];
          tmem_ld_x32(sbase, lo);
          tmem_ld_16(sbase + 32, hi);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(lo[j]);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[32 + j] = __uint_as_float(hi[j]);
        }
        // partial sums to the peer, and the peer's
        {
          const uint32_t xb = smem_u32(smem + L::kExchOff + sb * kExch) + hrow * 16;
          const uint32_t dst = peer_addr(xb, peer);
          const uint32_t bar = peer_addr(smem_u32(&tail->x_full[sb]), peer);
#pragma unroll
          for (int j = 0; j < kNK / 4; ++j)
            st_peer(dst + j * 2048, bar, __float_as_uint(s[4 * j]), __float_as_uint(s[4 * j + 1]),
                    __float_as_uint(s[4 * j + 2]), __float_as_uint(s[4 * j + 3]));
        }
        if (!__all_sync(0xffffffffu, wait_peer(&tail->x_full[sb], par, abort_flag, err))) break;
        const float4* xr =
            reinterpret_cast<const float4*>(smem + L::kExchOff + sb * kExch) + hrow;
        float mx = -INFINITY;
        const bool all = vm == (1ull << kNK) - 1;
#pragma unroll
        for (int j = 0; j < kNK / 4; ++j) {
          const float4 x = xr[j * 128];
          s[4 * j] += x.x;
          s[4 * j + 1] += x.y;
          s[4 * j + 2] += x.z;
          s[4 * j + 3] += x.w;
        }
        if (all) {
#pragma unroll
          for (int j = 0; j < kNK; ++j) mx = fmaxf(mx, s[j]);
        } else {
#pragma unroll
          for (int j = 0; j < kNK; ++j)
            if ((vm >> j) & 1u) mx = fmaxf(mx, s[j]);
        }
        if (flags & 1) {
          m = mx;
        } else if (__any_sync(0xffffffffu,
                              mx > m && (m == -INFINITY || (mx - m) * c2 > kRescaleLog2))) {
          // refresh the warp's running maxima: rescale O (every earlier PV is done) and l
          const int pg = g - 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&tail->s_empty[pg & 1], (pg >> 1) & 1, abort_flag,
                                                 err, kErrTime)))
            break;
          tc_fence_after();
          const float mnew = fmaxf(m, mx);
          const float f = m == -INFINITY ? 0.f : exp2f((m - mnew) * c2);
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
          l *= f;
          m = mnew;
        }
        // P = exp2(S*c2 - m*c2) over the valid keys, bf16 pairs in the S buffer's first columns
        const float base = m == -INFINITY ? 0.f : m * c2;
        float ls = 0.f;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t pk[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const int jj = part * 16 + j;
            float e0 = ex2f(fmaf(s[jj], c2, -base));
            float e1 = ex2f(fmaf(s[jj + 1], c2, -base));
            if (!all) {
              e0 = ((vm >> jj) & 1u) ? e0 : 0.f;
              e1 = ((vm >> (jj + 1)) & 1u) ? e1 : 0.f;
            }
            ls += e0 + e1;
            pk[j >> 1] = pack_bf16(e0, e1);
          }
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                  sbase + part * 8),
              "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]),
              "r"(pk[7])
              : "memory");
        }
        tmem_st_wait();
        l += ls;
      }
      tc_fence_before();
      mbar_arrive(&tail->p_full[sb]);
      if (!(flags & 2)) continue;

      // the tile's last chunk here: every S of it is done, the next tile's Q may replace its own
      if (g + 1 < n) load_q(item + 1);
      if (act) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&tail->s_empty[sb], par, abort_flag, err, kErrTime)))
          break;
        tc_fence_after();
        const long long row = r0 + hrow;
        if (flags & 4) {
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
                w.x = pack_bf16(__uint_as_float(ov[d]) * inv, __uint_as_float(ov[d + 1]) * inv);
                w.y = pack_bf16(__uint_as_float(ov[d + 2]) * inv, __uint_as_float(ov[d + 3]) * inv);
                w.z = pack_bf16(__uint_as_float(ov[d + 4]) * inv, __uint_as_float(ov[d + 5]) * inv);
                w.w = pack_bf16(__uint_as_float(ov[d + 6]) * inv, __uint_as_float(ov[d + 7]) * inv);
                out[(d0 + d) / 8] = w;
              }
            }
          }
          if (rank == 0 && hrow < rows)
            p.a.lse[row] = l == 0.f ? -INFINITY : (m * c2 + log2f(l)) * 0.69314718055994530942f;
        } else {
          // part 0 of this cluster: a tile begun before its range; part 1: one that goes on behind
          const int part = 2 * cluster + (item == item0 && c0 > 0 ? 0 : 1);
          float4* out = p.part + static_cast<long long>(part) * (kDc / 4) * p.prow +
                        static_cast<long long>(rank * (kHalf / 4)) * p.prow + hrow;
#pragma unroll 1
          for (int d0 = 0; d0 < kHalf; d0 += 32) {
            uint32_t ov[32];
            tmem_ld_x32(tmem + lane_off + kColO + d0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int d = 0; d < 32; d += 4)
              out[static_cast<long long>((d0 + d) / 4) * p.prow] =
                  make_float4(__uint_as_float(ov[d]), __uint_as_float(ov[d + 1]),
                              __uint_as_float(ov[d + 2]), __uint_as_float(ov[d + 3]));
          }
          if (rank == 0)
            p.ml[static_cast<long long>(part) * p.prow + hrow] =
                make_float2(m == -INFINITY ? -INFINITY : m * c2, l);
        }
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
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, 512);
  cluster_sync_all();   // no CTA leaves while its peer may still write to it
}

// Joins the parts of a tile that several clusters worked on: block (c, y) the tile that begins in
// cluster c's range and goes on behind it, dims [32 y, 32 y + 32). One row per thread.
__global__ void __launch_bounds__(128) latent_join_kernel(const Params p) {
  __shared__ long long sums[4];
  __shared__ int item_s;
  __shared__ long long start_s, end_s;
  const int cluster = blockIdx.x;
  const long long total = total_chunks(p, sums);
  const long long each = chunks_each(p, total);
  const long long g0 = each * cluster, g1 = g0 + each;
  if (g1 >= total) return;
  Place at;
  if (find_item(p, g1 - 1, sums, at)) {
    item_s = at.item;
    start_s = at.start;
    end_s = at.start + item_chunks(p, at.item);
  }
  __syncthreads();
  if (start_s < g0 || end_s <= g1) return;
  const int last = static_cast<int>((end_s - 1) / each);
  int rows = p.a.H;
  long long r0 = static_cast<long long>(item_s) * p.a.H;
  if (!p.a.idx) {
    const int b = item_s / p.tiles, mt = item_s - b * p.tiles;
    rows = tile_rows(p, mt);
    r0 = static_cast<long long>(b) * p.a.Sq * p.a.H + mt * 128;
  }
  const int row = threadIdx.x;
  if (row >= rows) return;
  // part 1 of the first cluster, part 0 of the others
  float top = -INFINITY;
  for (int c = cluster; c <= last; ++c)
    top = fmaxf(top, p.ml[static_cast<long long>(2 * c + (c == cluster)) * p.prow + row].x);
  float l = 0.f;
  float4 o[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = cluster; c <= last; ++c) {
    const long long part = 2 * c + (c == cluster);
    const float2 ml = p.ml[part * p.prow + row];
    // a part without a key has m = -inf and l = 0 (and O = 0); one with a NaN keeps it in l
    const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
    if (w == 0.f) continue;
    l += w * ml.y;
    const float4* src = p.part + part * (kDc / 4) * p.prow + blockIdx.y * 8 * p.prow + row;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const float4 x = src[d * p.prow];
      o[d].x += w * x.x;
      o[d].y += w * x.y;
      o[d].z += w * x.z;
      o[d].w += w * x.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* out = reinterpret_cast<uint4*>(p.a.O + (r0 + row) * kDc + blockIdx.y * 32);
#pragma unroll
  for (int d = 0; d < 4; ++d)
    out[d] = make_uint4(pack_bf16(o[2 * d].x * inv, o[2 * d].y * inv),
                        pack_bf16(o[2 * d].z * inv, o[2 * d].w * inv),
                        pack_bf16(o[2 * d + 1].x * inv, o[2 * d + 1].y * inv),
                        pack_bf16(o[2 * d + 1].z * inv, o[2 * d + 1].w * inv));
  if (blockIdx.y == 0)
    p.a.lse[r0 + row] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
}

int part_rows(int Sq, int H, int k) {
  const long long rows = k > 0 ? H : static_cast<long long>(Sq) * H;
  return static_cast<int>(rows < 128 ? (rows + 31) / 32 * 32 : 128);
}

// clusters of the kernel that fit on the current device at once
template <bool FP8>
int resident_clusters(size_t smem) {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices] = {};
  static std::mutex lock;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> guard(lock);
  if (known[dev] == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
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
    if (cudaOccupancyMaxActiveClusters(&c, latent_attn_kernel<FP8>, &cfg) != cudaSuccess || c < 1)
      return 0;
    known[dev] = c < kMaxClusters ? c : kMaxClusters;
  }
  return known[dev];
}

template <bool FP8>
int launch(Params p, cudaStream_t stream) {
  const size_t smem = Layout<FP8>::kTailOff + sizeof(Tail);
  if (cudaFuncSetAttribute(latent_attn_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return DSA_ERR_CUDA;
  p.clusters = resident_clusters<FP8>(smem);
  if (p.clusters < 1) return DSA_ERR_CUDA;
  // no more clusters than the longest possible sequences have work for
  const long long cap = static_cast<long long>(p.a.max_pages) * p.a.page_size;
  const long long most = p.a.idx ? p.list_chunks : (cap + kNK - 1) / kNK;
  const long long wanted = (p.items * most + kMinChunks - 1) / kMinChunks;
  if (wanted < p.clusters) p.clusters = static_cast<int>(wanted);
  p.ml = reinterpret_cast<float2*>(p.part + 2ll * p.clusters * (kDc / 4) * p.prow);
  latent_attn_kernel<FP8><<<2 * p.clusters, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (p.clusters == 1) return DSA_OK;   // nothing is split
  latent_join_kernel<<<dim3(p.clusters, kDc / 32), 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

size_t latent_attn_workspace(int B, int Sq, int H, int k) {
  (void)B;
  const size_t rows = static_cast<size_t>(part_rows(Sq, H, k));
  return 2ull * kMaxClusters * rows * (kDc * sizeof(float) + sizeof(float2));
}

int launch_latent_attn(const LatentArgs& a, int fmt, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.tiles = static_cast<int>((static_cast<long long>(a.Sq) * a.H + 127) / 128);
  const long long items = a.idx ? static_cast<long long>(a.B) * a.Sq
                                : static_cast<long long>(a.B) * p.tiles;
  p.items = static_cast<int>(items);   // at most B * Sq * H < 2^31
  p.list_chunks = a.idx ? (a.k + kNK - 1) / kNK : 0;
  p.prow = part_rows(a.Sq, a.H, a.k);
  p.act_warps = p.prow / 32;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part = static_cast<float4*>(a.ws);
  return fmt == DSA_CACHE_E4M3 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace dsa
