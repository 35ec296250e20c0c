// Device helpers for matrices that stay in the caller's layout: eight consecutive elements of a
// stored row as fp32, whatever the storage type, and the power-of-two factors of the fp16 iterates.
#pragma once

#include "muon_device.cuh"

namespace muon {

__device__ __forceinline__ void widen8(const uint4& q, int type, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = type == kViewBF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]))
                                       : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float load_one(const void* base, int type, long long at) {
  if (type == kViewF32) return static_cast<const float*>(base)[at];
  if (type == kViewBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  return __half2float(static_cast<const __half*>(base)[at]);
}
__device__ __forceinline__ void store_one(void* base, int type, long long at, float x) {
  if (type == kViewF32)
    static_cast<float*>(base)[at] = x;
  else if (type == kViewBF16)
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(base)[at] = __float2half_rn(x);
}

// Elements at .. at + 7 of a stored row; the first `have` exist, the others come back as 0.
// The row starts 16-byte aligned and `at` is a multiple of 8 elements into it.
__device__ __forceinline__ void load_eight(const void* base, int type, long long at, int have, float (&v)[8]) {
  if (have >= 8) {
    if (type == kViewF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at), type, v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < have ? load_one(base, type, at + i) : 0.0f;
}

__device__ __forceinline__ void store_eight(void* base, int type, long long at, int have, const float (&v)[8]) {
  if (have >= 8) {
    if (type == kViewF32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (type == kViewBF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < have) store_one(base, type, at + i, v[i]);
}

// Sums of squares of values of any size.  The squares of fp32 values outside 2^-63 .. 2^64 are not fp32 values: a thread
// whose sum is outside 2^-100 .. 2^100 takes its values, by eights, times a power of two into sums of their own.
// (Far smaller ones beside values of the usual size would not show; a matrix of nothing else has a norm all the same.
// A test for every eight values took 24 x 1536 x 6144 of momentum, bound by its instructions, from 430 to 444 us.)
constexpr float kSquaresLow = 0x1p-100f, kSquaresHigh = 0x1p100f;
template <typename T>
__device__ __forceinline__ bool usual_sum(T sum) { return sum >= kSquaresLow && sum <= kSquaresHigh; }
__device__ __forceinline__ float squares8(const float (&v)[8]) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
  return sum;
}
struct Squares {
  float usual, large = 0.0f, small = 0.0f;
  // `sum`: the squares8 of all of the thread's eights together, which each(add) hands to add one by one where it is not usual.
  // `any`: whether there are any (a thread beyond the matrix has none to look for).
  template <typename Each>
  __device__ __forceinline__ Squares(float sum, bool any, Each each) : usual(sum) {
    if (usual_sum(sum) || !any) return;
    usual = 0.0f;
    each([&](const float (&v)[8]) {
      const float part = squares8(v);
      if (usual_sum(part)) {
        usual += part;
        return;
      }
      const bool down = !(part < 1.0f);  // (NaN too)
      const float f = down ? 0x1p-80f : 0x1p100f;
      float far = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) far = fmaf(v[i] * f, v[i] * f, far);
      if (down) large += far;
      else small += far;
    });
  }
};

// The sum over a CTA of THREADS threads, in thread 0; `red` holds a value for each of its warps.
template <int THREADS, typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // `red` may be in use
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T t = 0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += red[i];
  }
  return t;
}
// The same of squares, a CTA's first use of `red`: with one barrier where all are of the usual size.
template <int THREADS>
__device__ __forceinline__ double block_sum(const Squares& q, double* red) {
  float* red32 = reinterpret_cast<float*>(red);
  float v = q.usual;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red32[threadIdx.x >> 5] = v;
  const bool far = __syncthreads_or(q.large != 0.0f || q.small != 0.0f);
  float usual = 0.0f;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) usual += red32[i];
  }
  double t = usual;
  if (far)
    t += static_cast<double>(block_sum<THREADS>(q.large, red32)) * 0x1p160 +
         static_cast<double>(block_sum<THREADS>(q.small, red32)) * 0x1p-200;
  return t;
}
// Thread 0 leaves `sum` at `part`; true in the CTA that is the last of `parts` to do so, which may then read them all.
__device__ __forceinline__ bool last_to_leave(double* part, double sum, unsigned int* arrivals, int parts, bool* last) {
  if (threadIdx.x == 0) {
    *part = sum;
    __threadfence();
    *last = atomicAdd(arrivals, 1u) == static_cast<unsigned>(parts) - 1u;
  }
  __syncthreads();
  if (!*last) return false;
  __threadfence();
  return true;
}
// This thread's share of the sum of the parts, in a fixed order.
template <int THREADS>
__device__ __forceinline__ double sum_parts(const double* part, int parts) {
  double t = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) t += __ldcg(part + i);
  return t;
}

// The norm of a matrix whose squares add up to `sum` (infinite where fp32 has no such value), and the factor that makes
// x into the stored 2^12 x / (norm + eps).  The denominator counts as 2^-100 at least, so that its reciprocal is
// finite; a sum that is not finite, of a matrix that is not, gives NaN.
__device__ __forceinline__ float norm_of(double sum) {
  return usual_sum(sum) ? sqrtf(static_cast<float>(sum)) : static_cast<float>(sqrt(sum));
}
__device__ __forceinline__ float normaliser(double sum, float eps) {
  if (usual_sum(sum)) return kHalfX / (sqrtf(static_cast<float>(sum)) + eps);
  if (!isfinite(sum)) return __uint_as_float(0x7FC00000u);
  return static_cast<float>(kHalfX / fmax(sqrt(sum) + eps, 0x1p-100));
}

}  // namespace muon
