// pkv_rope.cu -- the pass between the QKV projection and attention: norms of
// query and key heads, rotation by position, and the KV-cache write, in one launch.
//
// Mathematics.  For a head's row x of D elements, in fp32: y = x w / sqrt(mean(x^2) +
// eps) where there is a weight w, else y = x; then, for the first R elements, the pairs
// (y_i, y_{i + R/2}), or (y_2i, y_{2i+1}), are turned by the angle whose cosine and
// sine are cos_sin[position][i] and [R/2 + i]; one rounding at the end (e4m3: of
// y / scale).  V rows are copied, or quantised as pkv_write_fp8 does.
//
// Layout.  A row is 4 to 32 lanes of one 16-byte load each (a "group": D = 128 bf16:
// 16 lanes), the sum of squares is a shuffle reduction over them, a partner element
// is R/2 elements on: in the lane R/(2 elements per lane) further where that divides,
// else through shared memory.  A group takes the rows r, r + groups, ... of one token,
// kRows loads in flight, and keeps the token's cosines and sines in registers for all of
// them; tokens with few heads share a CTA.
#include <cuda_fp8.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRows = 4;   // rows of a group in flight

// VEC elements of type T in one 16-byte register quartet <-> fp32.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)), __NV_SATFINITE,
        __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)),
        __NV_SATFINITE, __NV_E4M3);
    w[i] = (lo & 0xFFFFu) | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Where the partner of an element is: the other half of a pair in the same lane, in the
// lane kShift further, or anywhere (through shared memory).
enum Pairing { kInLane, kShuffle, kShared };

template <typename T, int D, Pairing PAIR, bool FP8>
__global__ void __launch_bounds__(kRopeThreads) pkv_rope_kernel(const RopeArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N, LANES = D / N, GROUPS = kRopeThreads / LANES;
  static_assert(!FP8 || N == 8, "e4m3 codes of bf16 rows");
  __shared__ float stage[PAIR == kShared ? kRopeThreads * N : 1];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int per_token = a.groups_per_token;          // a power of two
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (GROUPS / per_token) + group / per_token;
  const bool live = t < a.num_tokens;
  const int first = group % per_token;
  const int rows = a.num_q_heads + (a.v != nullptr ? 2 : 1) * a.num_kv_heads;
  const int e0 = lane * N;                           // this lane's first element of a row

  auto source = [&](int r) -> const T* {
    const T* p;
    if (r < a.num_q_heads) p = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
    else if ((r -= a.num_q_heads) < a.num_kv_heads)
      p = static_cast<const T*>(a.k) + t * a.k_stride + r * D;
    else p = static_cast<const T*>(a.v) + t * a.v_stride + (r - a.num_kv_heads) * D;
    return p + e0;
  };

  int64_t slot = -1, pos = 0;
  if (live) {
    pos = __ldg(a.positions + t);
    if (a.slot_mapping != nullptr) slot = __ldg(a.slot_mapping + t);
  }
  // a token to skip: padding, or one that the table or the cache does not have
  bool skip = !live || (a.slot_mapping != nullptr && slot < 0);
  if (!skip) {
    const int32_t bad = (pos < 0 || pos >= a.max_position ? PKV_ERR_POSITION : 0) |
                        (a.slot_mapping != nullptr && slot >= a.num_slots ? PKV_ERR_SLOT : 0);
    if (bad != 0) {
      if (first == 0 && lane == 0) raise_error(a.err, bad);
      skip = true;
    }
  }
  const int half = a.rot_dim / 2;
  // cosine and sine of each of this lane's elements, the sine negative for the first of a pair
  float c[N], s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i;
    c[i] = 1.f;
    s[i] = 0.f;
    if (!skip && e < a.rot_dim) {
      const int p = PAIR == kInLane ? e >> 1 : (e < half ? e : e - half);
      const bool is_first = PAIR == kInLane ? (e & 1) == 0 : e < half;
      const float* row = a.cos_sin + pos * a.rot_dim;
      c[i] = __ldg(row + p);
      const float sine = __ldg(row + half + p);
      s[i] = is_first ? -sine : sine;
    }
  }

  // (the same steps for every group: the shuffles take whole warps)
  for (int b = 0; b < rows; b += kRows * per_token) {
    const int r0 = b + first;
    uint4 in[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * per_token;
      in[u] = !skip && r < rows ? *reinterpret_cast<const uint4*>(source(r)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * per_token;
      float x[N];
      V::unpack(in[u], x);
      const bool is_q = r < a.num_q_heads;
      const bool is_v = r >= a.num_q_heads + a.num_kv_heads;
      const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
      // (every lane of the warp takes part in the shuffles)
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (w != nullptr && !is_v) {
          const float inv = rsqrtf(sum * (1.f / D) + a.eps);
          float f[N];
          V::unpack(*reinterpret_cast<const uint4*>(w + e0), f);
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] = x[i] * inv * f[i];
        }
      }
      float y[N];   // the other element of each pair
      if constexpr (PAIR == kInLane) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = x[i ^ 1];
      } else if constexpr (PAIR == kShuffle) {
        const int shift = half / N, at = threadIdx.x & 31;
        const int from = at - lane + (lane < shift ? lane + shift : (lane < 2 * shift ? lane - shift : lane));
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
      } else {
        float* row = stage + threadIdx.x / LANES * D;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) row[e0 + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int e = e0 + i;
          y[i] = e < a.rot_dim ? row[e < half ? e + half : e - half] : 0.f;
        }
      }
      if (skip || r >= rows) continue;
      if (!is_v) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (e0 + i < a.rot_dim) x[i] = fmaf(x[i], c[i], y[i] * s[i]);
      }
      const int h = is_q ? r : (is_v ? r - a.num_kv_heads : r) - a.num_q_heads;
      if (is_q) {
        T* out = static_cast<T*>(a.q_out) + t * a.q_out_stride + h * D + e0;
        *reinterpret_cast<uint4*>(out) = V::pack(x);
      } else if (a.slot_mapping == nullptr) {
        T* out = static_cast<T*>(a.k_out) + t * a.k_out_stride + h * D + e0;
        *reinterpret_cast<uint4*>(out) = V::pack(x);
      } else {
        const int64_t at = (slot * a.num_kv_heads + h) * D + e0;
        if constexpr (FP8) {
          uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
          *reinterpret_cast<uint2*>(cache + at) =
              to_e4m3(x, __ldg((is_v ? a.v_scale : a.k_scale) + h));
        } else {
          T* cache = static_cast<T*>(is_v ? a.v_cache : a.k_cache);
          *reinterpret_cast<uint4*>(cache + at) = V::pack(x);
        }
      }
    }
  }
}

template <typename T, int D, bool FP8>
cudaError_t launch_t(RopeArgs a, cudaStream_t stream) {
  constexpr int N = Vec<T>::N, GROUPS = kRopeThreads / (D / N);
  const int rows = a.num_q_heads + (a.v != nullptr ? 2 : 1) * a.num_kv_heads;
  a.groups_per_token = 1;
  while (a.groups_per_token < GROUPS && a.groups_per_token * kRows < rows) a.groups_per_token *= 2;
  const int tokens = GROUPS / a.groups_per_token;
  const unsigned grid = static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens);
  if (a.interleaved || a.rot_dim == 0)
    pkv_rope_kernel<T, D, kInLane, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  else if (a.rot_dim % (2 * N) == 0)
    pkv_rope_kernel<T, D, kShuffle, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  else
    pkv_rope_kernel<T, D, kShared, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int head_size, bool f32, bool fp8, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (f32) return head_size == 128 ? launch_t<float, 128, false>(a, stream)
                                   : launch_t<float, 64, false>(a, stream);
  if (fp8) return head_size == 128 ? launch_t<__nv_bfloat16, 128, true>(a, stream)
                                   : launch_t<__nv_bfloat16, 64, true>(a, stream);
  return head_size == 128 ? launch_t<__nv_bfloat16, 128, false>(a, stream)
                          : launch_t<__nv_bfloat16, 64, false>(a, stream);
}

}  // namespace pkv
