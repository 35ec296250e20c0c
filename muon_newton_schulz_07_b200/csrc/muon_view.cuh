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
// `vec`: the row starts 16-byte aligned and `at` is a multiple of 8 elements into it.
__device__ __forceinline__ void load_eight(const void* base, int type, long long at, int have, bool vec,
                                           float (&v)[8]) {
  if (vec && have >= 8) {
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

__device__ __forceinline__ void store_eight(void* base, int type, long long at, int have, bool vec,
                                            const float (&v)[8]) {
  if (vec && have >= 8) {
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

// The sum over a CTA of THREADS threads, in thread 0; `red` holds a value for each of its warps.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // `red` may be in use
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += red[i];
  }
  return t;
}
// Thread 0 leaves `sum` at `part`; true in the CTA that is the last of `parts` to do so, which may then read them all.
__device__ __forceinline__ bool last_to_leave(float* part, float sum, unsigned int* arrivals, int parts, bool* last) {
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
__device__ __forceinline__ float sum_parts(const float* part, int parts) {
  float t = 0.0f;
  for (int i = threadIdx.x; i < parts; i += THREADS) t += __ldcg(part + i);
  return t;
}

// The factor that makes x into the stored 2^12 x / (norm + eps).  The denominator counts as 2^-100 at
// least, so that its reciprocal is finite; a NaN stays one.
__device__ __forceinline__ float normaliser(float norm, float eps) {
  const float den = norm + eps;
  return kHalfX / (den < 0x1p-100f ? 0x1p-100f : den);
}

}  // namespace muon
