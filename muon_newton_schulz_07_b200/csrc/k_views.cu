// The ends of the fp16 Newton-Schulz iteration (MUON_MODE_HALF) for matrices that stay where and
// how the caller holds them: slices of fused weights, stacks, transposed storage, bf16, fp16 or fp32.
//
//   view_sumsq_kernel   ||x||_F from partial sums of squares, one per 64 x 128 tile
//   view_orient_kernel  X0 = 2^12 x / (||x||_F + eps), oriented to min x max, zero-padded, fp16
//   view_write_kernel   dst = decay dst + coef X_k, oriented back
//
// The norm must be known before the first rounding to fp16: gradients reach far below fp16's
// range, normalised matrices do not.  So the source is read twice; the second read finds it in L2
// when the set fits (126 MB).  The last CTA of a matrix to leave its partial sum adds them all, in a
// fixed order.  That costs each CTA a fence and an atomic, but no launch: one that only added them took 3 us more of
// small calls (7 of 331 x 1003: 162 us for 158) and 18 less of the largest.  Added by every CTA of the second pass,
// they were work that grows with the square of the matrix's tiles (4 GB from L2 for 16384 x 16384).  All three are bound by
// memory traffic: 2 x 2 + 2 bytes an element in, 2 + 2 out for bf16.  Measured with 113 M bf16 values (12 of
// 1536 x 6144): norms 58 us (3.9 TB/s), X0 71 us (6.4 TB/s).
#include "muon_view.cuh"

namespace muon {
namespace {

constexpr int TR = kEwTileR, TC = kEwTileC;  // 64 x 128 of the oriented matrix
constexpr int THREADS = kEwThreads;
static_assert(TR * TC == THREADS * 32, "four groups of eight elements a thread");

struct Where {
  int seg, e;        // view and matrix of it
  int tile;          // within the matrix
  int r0, c0;        // first row and column of the oriented matrix
};
__device__ __forceinline__ Where find(const ViewParams& p) {
  const int cta = static_cast<int>(blockIdx.x);
  int lo = 0, hi = p.nseg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seg[mid].tile_begin <= cta) lo = mid; else hi = mid - 1;
  }
  const ViewSeg& s = p.seg[lo];
  Where w;
  w.seg = lo;
  const int at = cta - s.tile_begin;
  w.e = at / s.tiles;
  w.tile = at - w.e * s.tiles;
  w.r0 = w.tile / s.tiles_c * TR;
  w.c0 = w.tile % s.tiles_c * TC;
  return w;
}

// The 32 stored elements a thread handles.  Where every stored row is 16-byte aligned, four groups of
// eight: rows of the tile when the storage runs along X's rows, of the transposed tile otherwise.
__device__ __forceinline__ void place(bool tr, int q, int& row, int& col) {
  const int c = threadIdx.x + q * THREADS;
  row = tr ? c >> 3 : c >> 4;          // stored row within the tile
  col = (tr ? c & 7 : c & 15) * 8;     // first stored element
}
// Otherwise single elements, a warp's 32 lanes side by side in a stored row.
__device__ __forceinline__ void place_one(bool tr, int i, int& row, int& col) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  row = warp + 8 * (tr ? i >> 1 : i >> 2);
  col = lane + 32 * (tr ? i & 1 : i & 3);
}

// A tile of the source (DST: of the destination, before it is updated) as a thread's 32 values:
// groups of eight where `grouped`, single elements otherwise.  The loads of a thread are all
// issued before any value is used.
template <bool DST>
__device__ __forceinline__ bool load_tile(const ViewSeg& s, const Where& w, float (&v)[4][8]) {
  const bool tr = (DST ? s.dst_tr : s.src_tr) != 0;
  const int type = DST ? s.dst_type : s.src_type;
  const void* base = DST ? s.dst : s.src;
  const long long ld = DST ? s.dst_ld : s.src_ld, bs = DST ? s.dst_bs : s.src_bs;
  const bool vec = (DST ? s.dst_vec : s.src_vec) != 0;
  const int rows = tr ? s.n : s.m, cols = tr ? s.m : s.n;  // as stored
  const int r0 = tr ? w.c0 : w.r0, c0 = tr ? w.r0 : w.c0;
  if (vec && r0 + (tr ? TC : TR) <= rows && c0 + (tr ? TR : TC) <= cols) {  // whole and aligned
    const long long at = w.e * bs + r0 * ld + c0;
    if (type != kViewF32) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int r, c;
        place(tr, i, r, c);
        q[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at + r * ld + c));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) widen8(q[i], type, v[i]);
    } else {
      float4 q[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int r, c;
        place(tr, i, r, c);
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + r * ld + c);
        q[2 * i] = __ldg(p);
        q[2 * i + 1] = __ldg(p + 1);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float* to = &v[i >> 1][(i & 1) * 4];
        to[0] = q[i].x; to[1] = q[i].y; to[2] = q[i].z; to[3] = q[i].w;
      }
    }
    return true;
  }
  if (vec) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int r, c;
      place(tr, q, r, c);
      const int have = r0 + r < rows ? cols - (c0 + c) : 0;
      load_eight(base, type, w.e * bs + (r0 + r) * ld + c0 + c, have, v[q]);
    }
    return true;
  }
  const long long at = w.e * bs + r0 * ld + c0;
  auto each = [&](auto load) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      int r, c;
      place_one(tr, i, r, c);
      v[i >> 3][i & 7] = r0 + r < rows && c0 + c < cols ? load(at + r * ld + c) : 0.0f;
    }
  };
  if (type == kViewF32)
    each([&](long long i) { return __ldg(static_cast<const float*>(base) + i); });
  else if (type == kViewBF16)
    each([&](long long i) { return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]); });
  else
    each([&](long long i) { return __half2float(static_cast<const __half*>(base)[i]); });
  return false;
}

__global__ void __launch_bounds__(THREADS, 6) view_sumsq_kernel(const __grid_constant__ ViewParams p) {
  __shared__ double red[THREADS / 32];
  __shared__ bool last;
  const Where w = find(p);
  const ViewSeg& s = p.seg[w.seg];
  float v[4][8];
  load_tile<false>(s, w, v);
  float sum32 = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) sum32 += squares8(v[q]);
  const Squares squares(sum32, true, [&](auto add) {
#pragma unroll
    for (int q = 0; q < 4; ++q) add(v[q]);
  });
  const double ss = block_sum<THREADS>(squares, red);
  double* part = p.partials + s.part_begin + w.e * s.parts;
  if (!last_to_leave(part + w.tile, ss, p.arrivals + s.caller_idx + w.e, s.parts, &last)) return;
  const double sum = block_sum<THREADS>(sum_parts<THREADS>(part, s.parts), red);
  if (threadIdx.x == 0) {
    p.norms[s.caller_idx + w.e] = norm_of(sum);
    p.factors[s.caller_idx + w.e] = normaliser(sum, p.eps);
  }
}

__global__ void __launch_bounds__(THREADS, 4) view_orient_kernel(const __grid_constant__ ViewParams p) {
  __shared__ __half stage[TR][TC + 2];
  const Where w = find(p);
  const ViewSeg& s = p.seg[w.seg];
  float v[4][8];
  const bool grouped = load_tile<false>(s, w, v);
  const float mul = p.normalised ? 1.0f : p.factors[s.caller_idx + w.e];
  __half* x = static_cast<__half*>(s.x) + static_cast<size_t>(w.e) * s.mp * s.np;
  const bool tr = s.src_tr != 0;
  const bool staged = tr || !grouped;
  if (staged) {
    if (grouped) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int r, c;
        place(true, q, r, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) stage[c + i][r] = __float2half_rn(v[q][i] * mul);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        int r, c;
        place_one(tr, i, r, c);
        stage[tr ? c : r][tr ? r : c] = __float2half_rn(v[i >> 3][i & 7] * mul);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(false, q, r, c);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 t;
      if (staged)
        t = *reinterpret_cast<const __half2*>(&stage[r][c + 2 * i]);
      else
        t = __floats2half2_rn(v[q][2 * i] * mul, v[q][2 * i + 1] * mul);
      h[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(x + static_cast<size_t>(w.r0 + r) * s.np + w.c0 + c) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

__global__ void __launch_bounds__(THREADS, 3) view_write_kernel(const __grid_constant__ ViewParams p) {
  __shared__ float stage[TR][TC + 1];
  const Where w = find(p);
  const ViewSeg& s = p.seg[w.seg];
  const bool tr = s.dst_tr != 0, grouped = s.dst_vec != 0;
  const bool staged = tr || !grouped;
  const __half* x = static_cast<const __half*>(s.x) + static_cast<size_t>(w.e) * s.mp * s.np;
  float d[4][8];
  if (p.decay != 0.0f) load_tile<true>(s, w, d);
  float o[4][8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(false, q, r, c);
    widen8(*reinterpret_cast<const uint4*>(x + static_cast<size_t>(w.r0 + r) * s.np + w.c0 + c), kViewF16, o[q]);
    if (staged) {
#pragma unroll
      for (int i = 0; i < 8; ++i) stage[r][c + i] = o[q][i];
    }
  }
  if (staged) __syncthreads();
  const int rows = tr ? s.n : s.m, cols = tr ? s.m : s.n;  // as stored
  const int r0 = tr ? w.c0 : w.r0, c0 = tr ? w.r0 : w.c0;
  const long long at = w.e * s.dst_bs + r0 * s.dst_ld + c0;
  if (!grouped) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      int r, c;
      place_one(tr, i, r, c);
      const float y = s.coef * stage[tr ? c : r][tr ? r : c];
      o[i >> 3][i & 7] = p.decay != 0.0f ? fmaf(p.decay, d[i >> 3][i & 7], y) : y;
    }
    auto each = [&](auto store) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        int r, c;
        place_one(tr, i, r, c);
        if (r0 + r < rows && c0 + c < cols) store(at + r * s.dst_ld + c, o[i >> 3][i & 7]);
      }
    };
    if (s.dst_type == kViewF32)
      each([&](long long i, float y) { static_cast<float*>(s.dst)[i] = y; });
    else if (s.dst_type == kViewBF16)
      each([&](long long i, float y) { static_cast<__nv_bfloat16*>(s.dst)[i] = __float2bfloat16_rn(y); });
    else
      each([&](long long i, float y) { static_cast<__half*>(s.dst)[i] = __float2half_rn(y); });
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(tr, q, r, c);
    const int have = r0 + r < rows ? cols - (c0 + c) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = s.coef * (tr ? stage[c + i][r] : o[q][i]);
      o[q][i] = p.decay != 0.0f ? fmaf(p.decay, d[q][i], y) : y;
    }
    store_eight(s.dst, s.dst_type, at + r * s.dst_ld + c, have, o[q]);
  }
}

}  // namespace

cudaError_t launch_view_sumsq(const ViewParams& p, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  view_sumsq_kernel<<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_view_orient(const ViewParams& p, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  view_orient_kernel<<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_view_write(const ViewParams& p, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  view_write_kernel<<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace muon
