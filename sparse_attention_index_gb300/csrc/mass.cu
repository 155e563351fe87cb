// The attention weight that each cached position receives from the newest tokens (dsa_cache_mass):
//
//   mass[j] = decay prev[j] + sum over tokens i and heads h that see j of exp(scale q_ih . row_j - lse_ih)
//
// with lse from the attention itself, so that one more product of queries and rows is all it takes. A
// key's sum stays with one thread block, in a fixed order: the same bits every time.

#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kThreads = 256, kKeys = 4;   // keys per warp
constexpr int kErrIdx = DSA_STAGE_EVICT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_EVICT | DSA_DEVERR_BAD_PAGE;

struct Params {
  MassArgs a;
  float* w;   // lists: the weight of each entry [B, Sq, k]
};

__device__ __forceinline__ int seq_len(const MassArgs& a, int b, bool report) {
  const int cap = a.max_pages * a.page_size;
  const int len = __ldg(a.lens + b);
  if (report && (len < 0 || len > cap || len > a.n)) report_error(a.err, kErrPage);
  return max(0, min(len, cap));
}

template <bool FP8>
__device__ __forceinline__ float value(const uint8_t* row, int d) {
  if (!FP8 || d >= kDc) {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(row + (FP8 ? kDc + 16 - 2 * kDc : 0));
    return bf16_bits_to_float(__ldg(v + d));
  }
  const __half_raw h = __nv_cvt_fp8_to_halfraw(__ldg(row + d), __NV_E4M3);
  return __half2float(__half(h)) * __ldg(reinterpret_cast<const float*>(row + kDc) + (d >> 7));
}

// Warp w of block (x, b): keys 4 (8 x + w) ... of sequence b, or, with lists, entries of token b's list.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) mass_kernel(const Params p) {
  const MassArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kKeys;
  const int b = a.idx ? blockIdx.y / a.Sq : blockIdx.y, i0 = a.idx ? blockIdx.y - b * a.Sq : 0;
  const int len = seq_len(a, b, j0 == 0 && lane == 0);
  const int count = a.idx ? a.k : a.n;
  if (j0 >= count) return;
  const long long row_bytes = FP8 ? kDc + 16 + 2 * kDr : 2 * kD;
  float key[kKeys][kD / 32], sum[kKeys];
  int pos[kKeys];
#pragma unroll
  for (int t = 0; t < kKeys; ++t) {
    sum[t] = 0.f;
    int j = j0 + t < count ? j0 + t : -1;
    if (a.idx && j >= 0) {
      j = __ldg(a.idx + static_cast<long long>(blockIdx.y) * a.k + j);
      if (j < -1 || j >= len) {
        if (lane == 0) report_error(a.err, kErrIdx);
        j = -1;
      }
    }
    if (j >= len) j = -1;
    long long slot = -1;
    if (j >= 0) {
      const int pg = j / a.page_size;
      const int page = __ldg(a.page_table + static_cast<long long>(b) * a.max_pages + pg);
      if (page >= 0 && page < a.num_pages)
        slot = static_cast<long long>(page) * a.page_size + (j - pg * a.page_size);
      else if (lane == 0)
        report_error(a.err, kErrPage);
    }
    pos[t] = slot >= 0 ? j : 0x7fffffff;
#pragma unroll
    for (int d = 0; d < kD / 32; ++d)
      key[t][d] = slot >= 0 ? value<FP8>(a.cache + slot * row_bytes, d * 32 + lane) : 0.f;
  }
  for (int i = i0; i < (a.idx ? i0 + 1 : a.Sq); ++i) {
    const int limit = len - a.Sq + i + 1;
    for (int h = 0; h < a.H; ++h) {
      const long long row = (static_cast<long long>(b) * a.Sq + i) * a.H + h;
      const float lse = __ldg(a.lse + row);
      float s[kKeys] = {};
#pragma unroll
      for (int d = 0; d < kD / 32; ++d) {
        const float q = bf16_bits_to_float(__ldg(a.Q + row * kD + d * 32 + lane));
#pragma unroll
        for (int t = 0; t < kKeys; ++t) s[t] = fmaf(q, key[t][d], s[t]);
      }
#pragma unroll
      for (int t = 0; t < kKeys; ++t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[t] += __shfl_xor_sync(0xffffffffu, s[t], o);
        if (pos[t] < limit && lse != -INFINITY) sum[t] += expf(fmaf(s[t], a.scale, -lse));
      }
    }
  }
  if (lane != 0) return;
  for (int t = 0; t < kKeys && j0 + t < count; ++t) {
    if (a.idx) {
      p.w[static_cast<long long>(blockIdx.y) * a.k + j0 + t] = sum[t];
    } else {
      const long long at = static_cast<long long>(b) * a.n + j0 + t;
      float m = sum[t];
      if (a.prev && j0 + t < len) m += a.decay * a.prev[at];
      a.mass[at] = m;
    }
  }
}

// Lists: block (x, b) has kSlice positions of sequence b in shared memory, adds the lists' weights to
// them token by token (a list's entries are distinct, so the order is fixed) and writes them out.
constexpr int kSlice = 8192, kAddThreads = 512;
__global__ void __launch_bounds__(kAddThreads) add_lists_kernel(const Params p) {
  __shared__ float m[kSlice];
  const MassArgs& a = p.a;
  const int b = blockIdx.y, lo = blockIdx.x * kSlice, size = min(kSlice, a.n - lo);
  const int len = seq_len(a, b, false);
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

template <bool FP8>
int launch(const Params& p, cudaStream_t stream) {
  const MassArgs& a = p.a;
  const int count = a.idx ? a.k : a.n;
  const dim3 grid((count + kKeys * kThreads / 32 - 1) / (kKeys * kThreads / 32), a.idx ? a.B * a.Sq : a.B);
  mass_kernel<FP8><<<grid, kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (a.idx) {
    add_lists_kernel<<<dim3((a.n + kSlice - 1) / kSlice, a.B), kAddThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace

size_t cache_mass_workspace(int B, int Sq, int k) {
  return static_cast<size_t>(B) * Sq * k * sizeof(float);
}

int launch_cache_mass(const MassArgs& a, int fmt, cudaStream_t stream) {
  Params p = {a, static_cast<float*>(a.ws)};
  return fmt == DSA_CACHE_E4M3 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace dsa
