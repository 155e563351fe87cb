// Rotary positions on part of each head (dsa_rope): (x_a, x_b) turned by pos * inv_freq.
//
// Angle. One turn is 2^64: F = inv_freq / (2 pi) turns per position as a 64-bit fraction, and
// pos * F mod 2^64 is the turned fraction, with the whole turns dropped by the wrap. The
// product is exact, so a far position loses nothing but F's own rounding (2^-53 of F, in
// fp64 once per block and frequency): 2^-25 turns at the farthest position, 2^-36 at 2^20.
// (An fp32 product pos * inv_freq is off by 2^-24 of the angle: 0.008 rad at 131072. In fp64
// per angle it would cost as much as the memory traffic when there is one head to share it.)
// The top 32 bits of the fraction, as a float in [-1/2, 1/2), go to sincospif.
//
// Bound: one read and one write of x. A thread moves 16-byte vectors and loads all of its
// own before the block works out its angles; each (token, frequency) angle is computed once
// per block and shared by the heads through shared memory. In the half layout a vector's
// partner is rot/2 dims away. Where the rotated part is a power of two of vectors, aligned in the
// head, the partner is in the same warp and comes by shuffle; otherwise the thread with the vector
// of the first half loads and turns both and the other does nothing (all that is read of a
// rotated part is read before it is written either way, so rotating in place is safe).
//
// Measured, calls replayed from a graph (through the Python binding 2 us more): 128 heads of 192 dims,
// 64 of them turned, 16384 tokens, bf16: 235 us, 6.9 TB/s (two or eight vectors per thread: 260 and 257
// us). 4097 tokens of 64 fp32 heads of 128 dims, 64 turned in halves: 43 us, 6.3 TB/s. 16384 tokens of 32
// bf16 heads, all 128 dims in halves: 72 us, 3.7 TB/s, held back by the angles' reads from shared
// memory (eight of 8 bytes for each vector). Reading two angles at once gives 2% in the interleaved layout and costs
// 5% in halves (16384 tokens of 32 bf16 heads, all 128 dims: 77.2 us instead of 73.5).

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr long long kL2Bytes = 129ll << 20;

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack<float>(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack<uint16_t>(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

struct RopeParams {
  const uint4* x;
  uint4* y;
  const int32_t* pos;
  const float* inv_freq;
  long long total;   // vectors
  int vpt;           // vectors per token (H * D / E)
  int vpd;           // vectors per head
  int off, rot;      // in elements
  float mscale;
  int inverse;
};

template <bool STREAM>
__device__ __forceinline__ void store(uint4* to, const uint4& a) {
  if (STREAM)
    __stcs(to, a);
  else
    *to = a;
}

// how the vectors of the rotated part are turned
enum Layout { kInterleaved, kHalfShuffle, kHalfPairs };

// V vectors per thread, strided by the block. STREAM: x and y are more than L2 holds and are marked
// to leave it first.
template <typename T, int LAYOUT, int V, bool STREAM>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int nf = p.rot >> 1;
  unsigned long long* F = reinterpret_cast<unsigned long long*>(smem_raw);
  float2* cs = reinterpret_cast<float2*>(smem_raw + nf * sizeof(unsigned long long));
  const int tid = threadIdx.x;
  const bool inplace = p.x == p.y;
  const long long v0 = static_cast<long long>(blockIdx.x) * (kThreads * V);
  const long long v1 = min(v0 + kThreads * V, p.total);
  const long long t0 = v0 / p.vpt;
  const int ntok = static_cast<int>((v1 - 1) / p.vpt - t0) + 1;
  const int first = static_cast<int>(v0 - t0 * p.vpt);   // of the block, within token t0

  // what this thread's vectors are: copied, turned, or (pairs) the second, which the thread of
  // the first turns
  uint4 a[V], b[V];
  int tok[V], fi[V];   // fi: -2 none, -1 copied, else the vector's first frequency
  bool second[V];      // of the second half (shuffled)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const long long v = v0 + tid + i * kThreads;
    fi[i] = -2;
    tok[i] = 0;
    second[i] = false;
    a[i] = make_uint4(0, 0, 0, 0);
    if (v < v1) {
      const int in = first + tid + i * kThreads;
      tok[i] = in / p.vpt;
      const int d = ((in - tok[i] * p.vpt) % p.vpd) * E - p.off;
      if (d < 0 || d >= p.rot)
        fi[i] = inplace ? -2 : -1;
      else if (LAYOUT == kInterleaved)
        fi[i] = d >> 1;
      else if (d < nf)
        fi[i] = d;
      else if (LAYOUT == kHalfShuffle) {
        fi[i] = d - nf;
        second[i] = true;
      }
      if (fi[i] != -2) a[i] = STREAM ? __ldcs(p.x + v) : p.x[v];
      if (LAYOUT == kHalfPairs && fi[i] >= 0) b[i] = p.x[v + nf / E];
    }
  }

  for (int f = tid; f < nf; f += kThreads) {
    double turns = static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577;
    turns -= floor(turns);
    F[f] = static_cast<unsigned long long>(turns * 18446744073709551616.0);
  }
  __syncthreads();
  for (int i = tid; i < ntok * nf; i += kThreads) {
    const int t = i / nf;
    const long long at = p.pos[t0 + t];
    const unsigned long long u = static_cast<unsigned long long>(at) * F[i - t * nf];
    const float half_turns = static_cast<float>(static_cast<int>(u >> 32)) * 4.6566128730773926e-10f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[i] = make_float2(c * p.mscale, (p.inverse ? -s : s) * p.mscale);
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < V; ++i) {
    const long long v = v0 + tid + i * kThreads;
    if (LAYOUT == kHalfShuffle) {
      const int o = nf / E;
      b[i] = make_uint4(
          __shfl_xor_sync(0xffffffffu, a[i].x, o), __shfl_xor_sync(0xffffffffu, a[i].y, o),
          __shfl_xor_sync(0xffffffffu, a[i].z, o), __shfl_xor_sync(0xffffffffu, a[i].w, o));
    }
    if (fi[i] >= 0) {
      const float2* w = cs + tok[i] * nf + fi[i];
      float fa[E], fb[E];
      unpack<T>(a[i], fa);
      if (LAYOUT == kHalfShuffle) {
        unpack<T>(b[i], fb);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float2 r = w[e];
          fa[e] = second[i] ? fb[e] * r.y + fa[e] * r.x : fa[e] * r.x - fb[e] * r.y;
        }
      } else if (LAYOUT == kHalfPairs) {
        unpack<T>(b[i], fb);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float2 r = w[e];
          const float x = fa[e], y = fb[e];
          fa[e] = x * r.x - y * r.y;
          fb[e] = x * r.y + y * r.x;
        }
        store<STREAM>(p.y + v + nf / E, pack(fb));
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {   // two angles at a time
          const float4 r = *reinterpret_cast<const float4*>(w + (e >> 1));
          const float x0 = fa[e], y0 = fa[e + 1], x1 = fa[e + 2], y1 = fa[e + 3];
          fa[e] = x0 * r.x - y0 * r.y;
          fa[e + 1] = x0 * r.y + y0 * r.x;
          fa[e + 2] = x1 * r.z - y1 * r.w;
          fa[e + 3] = x1 * r.w + y1 * r.z;
        }
      }
      store<STREAM>(p.y + v, pack(fa));
    } else if (fi[i] == -1) {
      store<STREAM>(p.y + v, a[i]);
    }
  }
}

template <typename T, int LAYOUT, int V, bool STREAM>
int launch(const RopeParams& p, cudaStream_t stream) {
  const int nf = p.rot / 2;
  // tokens that a block's vectors touch
  const long long ntok = (kThreads * V + p.vpt - 2) / p.vpt + 1;
  const size_t smem = nf * sizeof(unsigned long long) + ntok * nf * sizeof(float2);
  // at most 1024 * 8 / D vectors' tokens of D / 2 angles and two partial ones: below 48 KB
  const long long blocks = (p.total + kThreads * V - 1) / (kThreads * V);
  if (blocks > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
  rope_kernel<T, LAYOUT, V, STREAM><<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <typename T, int LAYOUT>
int launch_v(const RopeParams& p, cudaStream_t stream) {
  // few vectors: one per thread, so that they spread over the SMs
  if (p.total <= 152 * 4 * kThreads) return launch<T, LAYOUT, 1, false>(p, stream);
  // streamed: 243.3 us down to 238.3 for 16384 tokens of 128 heads, 44.9 to 43.0 for 4097 tokens of
  // 64 fp32 heads in halves, but 48.6 up to 49.6 for those in pairs
  if (LAYOUT != kHalfPairs && p.total * 32 > kL2Bytes)
    return launch<T, LAYOUT, 4, LAYOUT != kHalfPairs>(p, stream);
  return launch<T, LAYOUT, 4, false>(p, stream);
}

}  // namespace

int launch_rope(const void* x, void* y, int is_f32, const int32_t* pos, const float* inv_freq,
                int T, int H, int D, int off, int rot, int half, float mscale, int inverse,
                cudaStream_t stream) {
  const int E = is_f32 ? 4 : 8;
  if (static_cast<long long>(H) * (D / E) > 0x3fffffffLL) return DSA_ERR_UNSUPPORTED;
  RopeParams p;
  p.x = static_cast<const uint4*>(x);
  p.y = static_cast<uint4*>(y);
  p.pos = pos;
  p.inv_freq = inv_freq;
  p.vpd = D / E;
  p.vpt = H * p.vpd;
  p.total = static_cast<long long>(T) * p.vpt;
  p.off = off;
  p.rot = rot;
  p.mscale = mscale;
  p.inverse = inverse;
  if (!half)
    return is_f32 ? launch_v<float, kInterleaved>(p, stream)
                  : launch_v<uint16_t, kInterleaved>(p, stream);
  // by shuffle: 16384 tokens as above 290 us instead of 311; 4097 tokens of 64 fp32 heads of 128
  // dims 47.6 us instead of 50.3
  const int n = rot / E;   // vectors of the rotated part
  if (n <= 32 && (n & (n - 1)) == 0 && (off / E) % n == 0 && p.vpd % n == 0)
    return is_f32 ? launch_v<float, kHalfShuffle>(p, stream)
                  : launch_v<uint16_t, kHalfShuffle>(p, stream);
  return is_f32 ? launch_v<float, kHalfPairs>(p, stream)
                : launch_v<uint16_t, kHalfPairs>(p, stream);
}

}  // namespace dsa
