// pkv_rope.cu -- the pass between the QKV projection and attention: norms of
// query and key heads, rotation by position, and the KV-cache write, in one launch.
//
// Mathematics.  For a head's row x of D elements, in fp32: y = x w / sqrt(mean(x^2) +
// eps) where there is a weight w, else y = x; then, for the first R elements, the pairs
// (y_i, y_{i + R/2}), or (y_2i, y_{2i+1}), are turned by the angle whose cosine and
// sine are cos_sin[position][i] and [R/2 + i]; one rounding at the end (e4m3: of
// y / scale).  V rows are copied, or quantised as pkv_write_fp8 does.
//
// Layout.  A row is D / 8 lanes (bf16; fp32: D / 4) with two 8-byte chunks each (a "group"):
// a chunk and the one with its pairs' other halves, so that a rotation needs no other
// lane; the sum of squares is a shuffle reduction.  (Rotations whose half does not
// fill chunks take their pairs through shared memory.)  A thread has the same kRows rows
// of every token that its CTA walks, so that what depends on the row alone (kind, pointers)
// is found once: the kernel is bound by its instructions (0.7 issued a cycle) before it is
// by memory.  The next token's rows, position and slot are on their way while a token is
// computed.  16384 tokens of 32 q / 8 kv heads of 128, bf16, normalised: 81 us, 5.1 TB/s, 0.75
// of the copy rate (rows found anew for every token: 123 us; partners exchanged by
// shuffles of 16-byte loads: 123 to 145; 256 threads and 3 rows each: 86; 8 CTAs an SM: 89); 1024 tokens of 32 /
// 32 heads without norms 8.2 us; 1 token 2.7; 8192 tokens in fp32 79 us, 0.76 of the copy rate; 16384 tokens
// into an e4m3 cache 105 us, 3.6 TB/s, 0.53 of it (59 % of the issue slots; K and V are
// divided and converted element by element).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kCtasPerSm = 6;
constexpr int kRows = 2;   // of a thread

// Elements of type T in an 8-byte chunk <-> fp32.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint2& u, float* x) {
    x[0] = bf16_lo(u.x);
    x[1] = bf16_hi(u.x);
    x[2] = bf16_lo(u.y);
    x[3] = bf16_hi(u.y);
  }
  static __device__ __forceinline__ uint2 pack(const float* x) {
    return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
};
template <>
struct Chunk<float> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void unpack(const uint2& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
  }
  static __device__ __forceinline__ uint2 pack(const float* x) {
    return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
  }
};

__device__ __forceinline__ uint32_t to_e4m3(const float* x, float scale) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | (hi << 16);
}

// How the pairs of a rotation lie: two neighbours; half a rotation apart, in whole chunks;
// half a rotation apart, anyhow.
enum Pairing { kNeighbours, kChunks, kAnyhow };

template <typename T, int D, Pairing PAIR, bool FP8>
__global__ void __launch_bounds__(kRopeThreads, kCtasPerSm) pkv_rope_kernel(const RopeArgs a) {
  using C = Chunk<T>;
  constexpr int N = C::N, LANES = D / (2 * N), GROUPS = kRopeThreads / LANES;
  constexpr int kIn = sizeof(T), kOut = FP8 ? 1 : sizeof(T);   // bytes of an element, of a cached one
  static_assert(!FP8 || N == 4, "e4m3 codes of bf16 rows");
  __shared__ float stage[PAIR == kAnyhow ? GROUPS * D : 1];
  __shared__ alignas(16) float weights[2][D];        // of q, of k
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int per_token = a.groups_per_token;          // a power of two
  const int tokens = GROUPS / per_token;             // of a CTA at a time
  const int hq = a.num_q_heads, hk = hq + a.num_kv_heads;   // rows: q below hq, k below hk, v
  const int rows = hk + (a.v != nullptr ? a.num_kv_heads : 0);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * tokens;
  const int half = a.rot_dim / 2;
  // this lane's elements: ea .. ea + N - 1 and eb .. eb + N - 1
  int ea = 2 * N * lane, eb = ea + N;
  if (PAIR == kChunks && lane < half / N) {
    ea = N * lane;
    eb = ea + half;
  }
  const bool turn = PAIR == kNeighbours ? ea < a.rot_dim : lane < half / N;
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
    const T* w = static_cast<const T*>(i < D ? a.q_weight : a.k_weight);
    weights[i / D][i % D] = w != nullptr ? static_cast<float>(w[i % D]) : 1.f;
  }
  __syncthreads();

  // This thread's rows: where they come from (and the way to the next token's), where
  // they go (q, and k without a cache: a token on by out_step; else from the token's slot on).
  enum Kind { kNone, kQ, kK, kV };
  int64_t t = static_cast<int64_t>(blockIdx.x) * tokens + group / per_token;
  int kind[kRows], head[kRows];
  const char* src[kRows];
  char* dst[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    int r = (blockIdx.y * kRows + u) * per_token + group % per_token;
    kind[u] = r < hq ? kQ : (r < hk ? kK : (r < rows ? kV : kNone));
    r -= kind[u] == kQ ? 0 : (kind[u] == kK ? hq : hk);
    head[u] = r;
    src[u] = static_cast<const char*>(kind[u] == kQ ? a.q : (kind[u] == kK ? a.k : a.v)) +
             (t * (kind[u] == kQ ? a.q_stride : (kind[u] == kK ? a.k_stride : a.v_stride)) +
              static_cast<int64_t>(r) * D + ea) * kIn;
    if (kind[u] == kQ)
      dst[u] = static_cast<char*>(a.q_out) + (t * a.q_out_stride + static_cast<int64_t>(r) * D + ea) * kIn;
    else if (a.slot_mapping == nullptr)
      dst[u] = static_cast<char*>(a.k_out) + (t * a.k_out_stride + static_cast<int64_t>(r) * D + ea) * kIn;
    else
      dst[u] = static_cast<char*>(kind[u] == kK ? a.k_cache : a.v_cache) +
               (static_cast<int64_t>(r) * D + ea) * kOut;
  }
  const int64_t q_step = stride * a.q_stride * kIn, k_step = stride * a.k_stride * kIn,
                v_step = stride * a.v_stride * kIn, qo_step = stride * a.q_out_stride * kIn,
                ko_step = stride * a.k_out_stride * kIn;
  const int64_t slot_bytes = static_cast<int64_t>(a.num_kv_heads) * D * kOut;

  uint2 in[kRows][2];
  auto load = [&](bool live, uint2 (&to)[kRows][2]) {
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (live && kind[u] != kNone) {
        to[u][0] = *reinterpret_cast<const uint2*>(src[u]);
        to[u][1] = *reinterpret_cast<const uint2*>(src[u] + (eb - ea) * kIn);
      }
  };
  int64_t next_pos = 0, next_slot = -1;
  auto look = [&](int64_t at) {
    if (at < a.num_tokens) {
      next_pos = __ldg(a.positions + at);
      if (a.slot_mapping != nullptr) next_slot = __ldg(a.slot_mapping + at);
    }
  };
  look(t);
  load(t < a.num_tokens, in);

  // (the same steps for every group: the shuffles take whole warps)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * tokens; base < a.num_tokens; base += stride) {
    const int64_t pos = next_pos, slot = next_slot;
    // a token to skip: padding, or one that the table or the cache does not have
    bool skip = t >= a.num_tokens || (a.slot_mapping != nullptr && slot < 0);
    if (!skip) {
      const int32_t bad = (pos < 0 || pos >= a.max_position ? PKV_ERR_POSITION : 0) |
                          (a.slot_mapping != nullptr && slot >= a.num_slots ? PKV_ERR_SLOT : 0);
      if (bad != 0) {
        if (blockIdx.y == 0 && group % per_token == 0 && lane == 0) raise_error(a.err, bad);
        skip = true;
      }
    }
    // cosines and sines of this lane's N pairs (of its 2 N elements, where they lie anyhow)
    constexpr int M = PAIR == kAnyhow ? 2 * N : N;
    float c[M], s[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (!skip) {
      const float* row = a.cos_sin + pos * a.rot_dim;
      if constexpr (PAIR == kAnyhow) {
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const int e = ea + i, p = e < half ? e : e - half;   // (eb = ea + N)
          if (e < a.rot_dim) {
            c[i] = __ldg(row + p);
            const float sine = __ldg(row + half + p);
            s[i] = e < half ? -sine : sine;
          }
        }
      } else if (turn) {
        const int p = PAIR == kNeighbours ? ea / 2 : ea;
        if (half % N == 0) {   // (rows and halves begin on a vector)
          using F = std::conditional_t<N == 4, float4, float2>;
          *reinterpret_cast<F*>(c) = __ldg(reinterpret_cast<const F*>(row + p));
          *reinterpret_cast<F*>(s) = __ldg(reinterpret_cast<const F*>(row + half + p));
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (p + i < half) {
              c[i] = __ldg(row + p + i);
              s[i] = __ldg(row + half + p + i);
            }
        }
      }
    }
    t += stride;
    look(t);
    uint2 ahead[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      src[u] += kind[u] == kQ ? q_step : (kind[u] == kK ? k_step : v_step);
    load(t < a.num_tokens, ahead);
    const int64_t slot_at = slot * slot_bytes;

#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float x[2 * N];
      C::unpack(in[u][0], x);
      C::unpack(in[u][1], x + N);
      const bool is_q = kind[u] == kQ, is_v = kind[u] == kV;
      // (every lane of the warp takes part in the shuffles)
      if (norm_q || norm_k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (!is_v && (is_q ? norm_q : norm_k)) {
          const float inv = rsqrtf(fmaf(sum, 1.f / D, a.eps));
          const float* w = weights[is_q ? 0 : 1];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x[i] *= inv * w[ea + i];
            x[N + i] *= inv * w[eb + i];
          }
        }
      }
      if constexpr (PAIR == kNeighbours) {
        if (!is_v) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (ea + 2 * i < a.rot_dim) {
              const float y = x[2 * i], z = x[2 * i + 1];
              x[2 * i] = fmaf(y, c[i], -z * s[i]);
              x[2 * i + 1] = fmaf(z, c[i], y * s[i]);
            }
        }
      } else if constexpr (PAIR == kChunks) {
        if (turn && !is_v) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float y = x[i], z = x[N + i];
            x[i] = fmaf(y, c[i], -z * s[i]);
            x[N + i] = fmaf(z, c[i], y * s[i]);
          }
        }
      } else {
        float* row = stage + group * D;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) row[ea + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
          const int e = ea + i;
          if (e < a.rot_dim && !is_v) x[i] = fmaf(x[i], c[i], row[e < half ? e + half : e - half] * s[i]);
        }
      }
      if (!skip && kind[u] != kNone) {
        if (is_q || a.slot_mapping == nullptr) {
          *reinterpret_cast<uint2*>(dst[u]) = C::pack(x);
          *reinterpret_cast<uint2*>(dst[u] + (eb - ea) * kIn) = C::pack(x + N);
        } else if constexpr (FP8) {
          const float scale = __ldg((is_v ? a.v_scale : a.k_scale) + head[u]);
          *reinterpret_cast<uint32_t*>(dst[u] + slot_at) = to_e4m3(x, scale);
          *reinterpret_cast<uint32_t*>(dst[u] + slot_at + (eb - ea)) = to_e4m3(x + N, scale);
        } else {
          *reinterpret_cast<uint2*>(dst[u] + slot_at) = is_v ? in[u][0] : C::pack(x);
          *reinterpret_cast<uint2*>(dst[u] + slot_at + (eb - ea) * kIn) = is_v ? in[u][1] : C::pack(x + N);
        }
      }
      if (is_q) dst[u] += qo_step;
      else if (a.slot_mapping == nullptr) dst[u] += ko_step;
      in[u][0] = ahead[u][0];
      in[u][1] = ahead[u][1];
    }
  }
}

template <typename T, int D, bool FP8>
cudaError_t launch_t(RopeArgs a, int num_sms, cudaStream_t stream) {
  constexpr int N = Chunk<T>::N, GROUPS = kRopeThreads / (D / (2 * N));
  const int rows = a.num_q_heads + (a.v != nullptr ? 2 : 1) * a.num_kv_heads;
  a.groups_per_token = 1;
  while (a.groups_per_token < GROUPS && a.groups_per_token * kRows < rows) a.groups_per_token *= 2;
  const int tokens = GROUPS / a.groups_per_token, step = a.groups_per_token * kRows;
  const int parts = (rows + step - 1) / step;   // CTAs that share a token's rows
  const dim3 grid(std::min((a.num_tokens - 1) / tokens + 1, std::max(num_sms * kCtasPerSm / parts, 1)), parts);
  if (a.interleaved || a.rot_dim == 0)
    pkv_rope_kernel<T, D, kNeighbours, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  else if (a.rot_dim % (2 * N) == 0)
    pkv_rope_kernel<T, D, kChunks, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  else
    pkv_rope_kernel<T, D, kAnyhow, FP8><<<grid, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int head_size, bool f32, bool fp8, int num_sms,
                        cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (f32) return head_size == 128 ? launch_t<float, 128, false>(a, num_sms, stream)
                                   : launch_t<float, 64, false>(a, num_sms, stream);
  if (fp8) return head_size == 128 ? launch_t<__nv_bfloat16, 128, true>(a, num_sms, stream)
                                   : launch_t<__nv_bfloat16, 64, true>(a, num_sms, stream);
  return head_size == 128 ? launch_t<__nv_bfloat16, 128, false>(a, num_sms, stream)
                          : launch_t<__nv_bfloat16, 64, false>(a, num_sms, stream);
}

}  // namespace pkv
