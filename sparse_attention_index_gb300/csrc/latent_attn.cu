// Attention of the newest tokens of each sequence over the paged latent cache (dsa_latent_attn).
//
// One warp per (sequence, token, head): the 576 dims of a row over its lanes, an online softmax
// over the row's keys.

#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kErrIdx = DSA_STAGE_LATENT | DSA_DEVERR_BAD_INDEX;
constexpr int kErrPage = DSA_STAGE_LATENT | DSA_DEVERR_BAD_PAGE;

__device__ __forceinline__ float e4m3(uint8_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <bool FP8>
__global__ void __launch_bounds__(256) latent_simple_kernel(const LatentArgs p) {
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(p.B) * p.Sq * p.H) return;
  const long long tok = w / p.H;
  const int b = static_cast<int>(tok / p.Sq), i = static_cast<int>(tok % p.Sq);
  const int cap = p.max_pages * p.page_size;
  int len = p.lens[b];
  if (len < 0 || len > cap) report_error(p.err, kErrPage);
  len = max(0, min(len, cap));
  const int limit = len - p.Sq + i + 1;
  float q[18], o[16];
  for (int c = 0; c < 18; ++c) q[c] = bf16_bits_to_float(p.Q[w * kD + c * 32 + lane]);
  for (int c = 0; c < 16; ++c) o[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int n = p.idx ? p.k : limit;
  for (int j = 0; j < n; ++j) {
    int pos = j;
    if (p.idx) {
      pos = p.idx[tok * p.k + j];
      if (pos < -1 || pos >= len) {
        report_error(p.err, kErrIdx);
        continue;
      }
      if (pos < 0 || pos >= limit) continue;
    }
    const int page = p.page_table[static_cast<long long>(b) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      report_error(p.err, kErrPage);
      continue;
    }
    const long long slot = static_cast<long long>(page) * p.page_size + pos % p.page_size;
    float kv[18];
    if (FP8) {
      const uint8_t* row = p.cache + slot * (kDc + 16 + 2 * kDr);
      for (int c = 0; c < 16; ++c)
        kv[c] = e4m3(row[c * 32 + lane]) * reinterpret_cast<const float*>(row + kDc)[c >> 2];
      for (int c = 0; c < 2; ++c)
        kv[16 + c] = bf16_bits_to_float(
            reinterpret_cast<const uint16_t*>(row + kDc + 16)[c * 32 + lane]);
    } else {
      const uint16_t* row = reinterpret_cast<const uint16_t*>(p.cache) + slot * kD;
      for (int c = 0; c < 18; ++c) kv[c] = bf16_bits_to_float(row[c * 32 + lane]);
    }
    float s = 0.f;
    for (int c = 0; c < 18; ++c) s = fmaf(q[c], kv[c], s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn), e = __expf(s - mn);
    for (int c = 0; c < 16; ++c) o[c] = o[c] * f + e * kv[c];
    l = l * f + e;
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;   // NaN stays NaN
  for (int c = 0; c < 16; ++c)
    p.O[w * kDc + c * 32 + lane] = static_cast<uint16_t>(pack_bf16(o[c] * inv, 0.f));
  if (lane == 0) p.lse[w] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t latent_attn_workspace(int B, int Sq, int H, int k) {
  (void)B; (void)Sq; (void)H; (void)k;
  return 0;
}

int launch_latent_attn(const LatentArgs& a, int fmt, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.B) * a.Sq * a.H;
  const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
  if (fmt == DSA_CACHE_E4M3)
    latent_simple_kernel<true><<<grid, 256, 0, stream>>>(a);
  else
    latent_simple_kernel<false><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
