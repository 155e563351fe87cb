// The paged latent cache: writing rows (quantising them on the way) and reading them back.
//
// A row's work is cut into units of 128 dims, eight lanes with 16 dims each: the Dc / 128
// quantised groups, then the positional dims (the last unit may be partly idle). A group's
// largest magnitude is an integer maximum of the bf16 magnitudes' bits (which order like the
// values, with infinities and NaNs on top) over the lane and three shuffles; the power-of-two
// scale comes from its exponent field, so that no division or logarithm rounds.
//
// Bound: memory. Each input byte is read once and each output byte written once, 32 bytes of
// bf16 and 16 of e4m3 per lane; bf16 rows are copied 16 bytes a thread. 131072 rows of 576 dims
// at slots in no order, calls replayed from a graph: read back in 39.6 us from e4m3 (6.0 TB/s) and
// 43.1 us from bf16 (7.0), written in 44.9 us (5.3) and 46.9 us (6.4); through the Python binding 2 to
// 3 us more. What holds the e4m3 rows back is not known: they are 656 bytes, so that neighbours
// share a 32-byte sector, but that is one sector in twenty.

#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kErrSlot = DSA_STAGE_CACHE | DSA_DEVERR_BAD_INDEX;

struct CacheParams {
  uint8_t* cache;
  uint16_t* kv;   // written by the read kernels, read by the write kernels
  const int32_t* slots;
  long long num_slots;
  long long units;   // rows * units per row
  int upr;           // units (e4m3) or 16-byte vectors (bf16) per row
  int Dc, Dr, row_bytes;
  int* err;
};

// the slot of a row, -1 where there is none
__device__ __forceinline__ long long slot_of(const CacheParams& p, long long row) {
  const int s = __ldg(p.slots + row);
  if (s >= p.num_slots || s < -1) {
    report_error(p.err, kErrSlot);
    return -1;
  }
  return s;
}

// Row and unit in it of unit `local` of this block's `per`, without dividing 64-bit numbers.
__device__ __forceinline__ long long row_of(const CacheParams& p, uint32_t per, uint32_t local,
                                            int& u) {
  const uint32_t upr = p.upr, q = blockIdx.x / upr, r = blockIdx.x - q * upr;
  const uint32_t v = r * per + local;   // units behind the first of row q * per
  const uint32_t d = v / upr;
  u = static_cast<int>(v - d * upr);
  return static_cast<long long>(q) * per + d;
}

// K vectors per thread, a block apart, loaded before any is stored
template <int K>
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const CacheParams p, int to_cache) {
  const long long i0 = static_cast<long long>(blockIdx.x) * (kThreads * K) + threadIdx.x;
  uint4 v[K];
  uint4* dst[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    dst[k] = nullptr;
    if (i0 + k * kThreads >= p.units) continue;
    int c;
    const long long row = row_of(p, kThreads * K, k * kThreads + threadIdx.x, c);
    const long long slot = slot_of(p, row);
    uint4* kv = reinterpret_cast<uint4*>(p.kv) + i0 + k * kThreads;
    uint4* at = reinterpret_cast<uint4*>(p.cache) + slot * p.upr + c;
    v[k] = make_uint4(0, 0, 0, 0);
    if (slot >= 0) v[k] = __ldg(to_cache ? kv : at);
    if (slot >= 0 || !to_cache) dst[k] = to_cache ? at : kv;
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (dst[k] != nullptr) *dst[k] = v[k];
}

// k of the scale 2^k: the smallest with amax <= 448 * 2^k, at least -120; 0 for amax = 0.
// `bits` is amax in bf16, finite: 1.f * 2^(e - 127), and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  if (bits == 0) return 0;
  const int k = static_cast<int>(bits >> 7) - 135 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return max(k, -120);
}

__device__ __forceinline__ uint32_t quant4(uint32_t lo, uint32_t hi, float inv) {
  const float2 a = make_float2(__uint_as_float(lo << 16) * inv,
                               __uint_as_float(lo & 0xffff0000u) * inv);
  const float2 b = make_float2(__uint_as_float(hi << 16) * inv,
                               __uint_as_float(hi & 0xffff0000u) * inv);
  const uint32_t x = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
  const uint32_t y = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
  return x | (y << 16);
}

// K units per eight lanes, a block apart, loaded before any is stored
template <int K>
__global__ void __launch_bounds__(kThreads) write_e4m3_kernel(const CacheParams p) {
  constexpr int kPer = kThreads / 8;
  const long long i0 = static_cast<long long>(blockIdx.x) * (kPer * K) + (threadIdx.x >> 3);
  const int sub = threadIdx.x & 7;
  const int G = p.Dc >> 7;
  long long slot[K];
  int u[K];
  uint4 v[K][2];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long row = row_of(p, kPer * K, k * kPer + (threadIdx.x >> 3), u[k]);
    slot[k] = i0 + k * kPer < p.units ? slot_of(p, row) : -1;
    const int d = u[k] * 128 + sub * 16;   // first dim of this lane
    const int left = p.Dc + p.Dr - d;      // dims left in the row: 8 in a half-filled last lane
    v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
    if (slot[k] >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(p.kv + row * (p.Dc + p.Dr) + d);
      if (left > 0) v[k][0] = __ldg(src);
      if (left > 8) v[k][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    // every lane takes part in the shuffles; the eight lanes of a unit agree on everything else
    const uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                           v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
    uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (slot[k] < 0) continue;
    uint8_t* out = p.cache + slot[k] * p.row_bytes;
    const int d = u[k] * 128 + sub * 16, left = p.Dc + p.Dr - d;
    if (u[k] < G) {
      float scale = __int_as_float(0x7fc00000), inv = scale;   // an infinity or a NaN: NaN
      if (top < 0x7f80u) {
        const int e = scale_exponent(top);
        scale = __int_as_float((127 + e) << 23);
        inv = __int_as_float((127 - e) << 23);
      }
      uint4 q;
      q.x = quant4(w[0], w[1], inv);
      q.y = quant4(w[2], w[3], inv);
      q.z = quant4(w[4], w[5], inv);
      q.w = quant4(w[6], w[7], inv);
      *reinterpret_cast<uint4*>(out + d) = q;
      float* sc = reinterpret_cast<float*>(out + p.Dc);
      if (sub == 0) sc[u[k]] = scale;
      // the scales' padding
      if (u[k] == G - 1 && sub > 0 && sub < 4 && u[k] + sub < (G + 3) / 4 * 4)
        sc[u[k] + sub] = 0.f;
    } else {
      uint4* dst = reinterpret_cast<uint4*>(out + p.row_bytes - 2 * p.Dr + 2 * (d - p.Dc));
      if (left > 0) dst[0] = v[k][0];
      if (left > 8) dst[1] = v[k][1];
    }
  }
}

__device__ __forceinline__ uint32_t dequant2(uint32_t two, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two),
                                                   __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x * scale, f.y * scale);
}

template <int K>
__global__ void __launch_bounds__(kThreads) read_e4m3_kernel(const CacheParams p) {
  constexpr int kPer = kThreads / 8;
  const long long i0 = static_cast<long long>(blockIdx.x) * (kPer * K) + (threadIdx.x >> 3);
  const int sub = threadIdx.x & 7;
  uint4 v[K][2];   // the codes in the first, or the positional dims as they are
  float scale[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
    scale[k] = 1.f;
    if (i0 + k * kPer >= p.units) continue;
    int u;
    const long long row = row_of(p, kPer * K, k * kPer + (threadIdx.x >> 3), u);
    const long long slot = slot_of(p, row);
    if (slot < 0) continue;
    const int d = u * 128 + sub * 16, left = p.Dc + p.Dr - d;
    const uint8_t* in = p.cache + slot * p.row_bytes;
    if (d < p.Dc) {
      v[k][0] = __ldg(reinterpret_cast<const uint4*>(in + d));
      scale[k] = __ldg(reinterpret_cast<const float*>(in + p.Dc) + u);
    } else {
      const uint4* src =
          reinterpret_cast<const uint4*>(in + p.row_bytes - 2 * p.Dr + 2 * (d - p.Dc));
      if (left > 0) v[k][0] = __ldg(src);
      if (left > 8) v[k][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (i0 + k * kPer >= p.units) continue;
    int u;
    const long long row = row_of(p, kPer * K, k * kPer + (threadIdx.x >> 3), u);
    const int d = u * 128 + sub * 16, left = p.Dc + p.Dr - d;
    if (d < p.Dc) {
      const uint4 q = v[k][0];
      const float sc = scale[k];
      v[k][0] = make_uint4(dequant2(q.x & 0xffffu, sc), dequant2(q.x >> 16, sc),
                           dequant2(q.y & 0xffffu, sc), dequant2(q.y >> 16, sc));
      v[k][1] = make_uint4(dequant2(q.z & 0xffffu, sc), dequant2(q.z >> 16, sc),
                           dequant2(q.w & 0xffffu, sc), dequant2(q.w >> 16, sc));
    }
    uint4* dst = reinterpret_cast<uint4*>(p.kv + row * (p.Dc + p.Dr) + d);
    if (left > 0) dst[0] = v[k][0];
    if (left > 8) dst[1] = v[k][1];
  }
}

template <int K>
int launch(const CacheParams& p, int fmt, bool write, cudaStream_t stream) {
  const int per = K * (fmt == DSA_CACHE_BF16 ? kThreads : kThreads / 8);
  const long long blocks = (p.units + per - 1) / per;
  if (blocks > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (fmt == DSA_CACHE_BF16)
    copy_rows_kernel<K><<<grid, kThreads, 0, stream>>>(p, write);
  else if (write)
    write_e4m3_kernel<K><<<grid, kThreads, 0, stream>>>(p);
  else
    read_e4m3_kernel<K><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int run(CacheParams p, int rows, int fmt, bool write, cudaStream_t stream) {
  p.row_bytes = static_cast<int>(cache_row_bytes(fmt, p.Dc, p.Dr));
  p.err = device_error_word();
  p.upr = fmt == DSA_CACHE_BF16 ? p.row_bytes / 16 : p.Dc / 128 + (p.Dr + 127) / 128;
  p.units = static_cast<long long>(rows) * p.upr;
  // Several units per thread once one each would fill the SMs' eight resident blocks that often:
  // 131072 rows of 576 dims, 1 / 2 / 4 per thread, calls through the binding: e4m3 read back 46.4 /
  // 41.9 / 46.3 us, written 47.7 / 47.7 / 60.0; bf16 read 62.1 / 50.0 / 45.6, written 63.9 / 53.9 /
  // 49.6. At 16384 rows
  // they are level, below that one is the quickest.
  const long long wave = 152ll * 8 * (kThreads / (fmt == DSA_CACHE_BF16 ? 1 : 8));
  if (fmt == DSA_CACHE_BF16)
    return p.units >= 4 * wave ? launch<4>(p, fmt, write, stream) : launch<1>(p, fmt, write, stream);
  return p.units >= 2 * wave ? launch<2>(p, fmt, write, stream) : launch<1>(p, fmt, write, stream);
}

}  // namespace

size_t cache_row_bytes(int fmt, int Dc, int Dr) {
  if (Dc < 128 || Dc > 1024 || Dc % 128 != 0 || Dr < 0 || Dr > 256 || Dr % 8 != 0) return 0;
  if (fmt == DSA_CACHE_BF16) return 2 * static_cast<size_t>(Dc + Dr);
  if (fmt != DSA_CACHE_E4M3) return 0;
  return static_cast<size_t>(Dc) + (Dc / 128 * 4 + 15) / 16 * 16 + 2 * static_cast<size_t>(Dr);
}

int launch_cache_write(const void* kv, const int32_t* slots, int T, int Dc, int Dr, int fmt,
                       void* cache, int64_t num_slots, cudaStream_t stream) {
  CacheParams p = {};
  p.cache = static_cast<uint8_t*>(cache);
  p.kv = const_cast<uint16_t*>(static_cast<const uint16_t*>(kv));
  p.slots = slots;
  p.num_slots = num_slots;
  p.Dc = Dc;
  p.Dr = Dr;
  return run(p, T, fmt, true, stream);
}

int launch_cache_read(const void* cache, int64_t num_slots, int fmt, const int32_t* slots, int N,
                      int Dc, int Dr, void* kv, cudaStream_t stream) {
  CacheParams p = {};
  p.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
  p.kv = static_cast<uint16_t*>(kv);
  p.slots = slots;
  p.num_slots = num_slots;
  p.Dc = Dc;
  p.Dr = Dr;
  return run(p, N, fmt, false, stream);
}

}  // namespace dsa
