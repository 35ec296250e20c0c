// The ends of the fp16 Newton-Schulz iteration (MUON_MODE_HALF) for matrices that stay where and
// how the caller holds them: slices of fused weights, stacks, transposed storage, bf16, fp16 or fp32.
//
//   view_sumsq_kernel   partial sums of squares, fp32, one per 64 x 128 tile
//   view_orient_kernel  X0 = 2^12 x / (||x||_F + eps), oriented to min x max, zero-padded, fp16
//   view_write_kernel   dst = decay dst + coef X_k, oriented back
//
// The norm must be known before the first rounding to fp16: gradients reach far below fp16's
// range, normalised matrices do not.  So the source is read twice; the second read finds it in L2
// when the set fits (126 MB).  Every CTA of the second pass adds its matrix's partial sums itself,
// in a fixed order, which saves the launch that would do only that.  All three are bound by
// memory traffic: 2 x 2 + 2 bytes an element in, 2 + 2 out for bf16.
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

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += red[i];
  return t;
}

// The four groups of eight stored elements a thread handles: rows of the tile when the storage
// runs along X's rows, rows of the transposed tile otherwise.
__device__ __forceinline__ void place(bool tr, int q, int& row, int& col) {
  const int c = threadIdx.x + q * THREADS;
  row = tr ? c >> 3 : c >> 4;          // stored row within the tile
  col = (tr ? c & 7 : c & 15) * 8;     // first stored element
}

__device__ __forceinline__ void load_tile(const ViewSeg& s, const Where& w, float (&v)[4][8]) {
  const bool tr = s.src_tr != 0;
  const int rows = tr ? s.n : s.m, cols = tr ? s.m : s.n;  // as stored
  const int r0 = tr ? w.c0 : w.r0, c0 = tr ? w.r0 : w.c0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(tr, q, r, c);
    const int have = r0 + r < rows ? cols - (c0 + c) : 0;
    load_eight(s.src, s.src_type, w.e * s.src_bs + (r0 + r) * s.src_ld + c0 + c, have, s.src_vec != 0, v[q]);
  }
}

__global__ void __launch_bounds__(THREADS, 4) view_sumsq_kernel(const __grid_constant__ ViewParams p) {
  const Where w = find(p);
  const ViewSeg& s = p.seg[w.seg];
  float v[4][8];
  load_tile(s, w, v);
  float ss = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[q][i], v[q][i], ss);
  ss = block_sum(ss);
  if (threadIdx.x == 0) p.partials[s.part_begin + w.e * s.parts + w.tile] = ss;
}

__global__ void __launch_bounds__(THREADS, 4) view_orient_kernel(const __grid_constant__ ViewParams p) {
  __shared__ __half stage[TR][TC + 2];
  const Where w = find(p);
  const ViewSeg& s = p.seg[w.seg];
  float v[4][8];
  load_tile(s, w, v);
  const float* part = p.partials + s.part_begin + w.e * s.parts;
  float ss = 0.0f;
  for (int i = threadIdx.x; i < s.parts; i += THREADS) ss += part[i];
  const float norm = sqrtf(block_sum(ss));
  if (w.tile == 0 && threadIdx.x == 0) p.norms[s.caller_idx + w.e] = norm;
  const float mul = normaliser(norm, p.eps);
  __half* x = static_cast<__half*>(s.x) + static_cast<size_t>(w.e) * s.mp * s.np;
  if (s.src_tr) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int r, c;
      place(true, q, r, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) stage[c + i][r] = __float2half_rn(v[q][i] * mul);
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
      if (s.src_tr)
        t = __halves2half2(stage[r][c + 2 * i], stage[r][c + 2 * i + 1]);
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
  const bool tr = s.dst_tr != 0;
  const __half* x = static_cast<const __half*>(s.x) + static_cast<size_t>(w.e) * s.mp * s.np;
  float o[4][8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(false, q, r, c);
    widen8(*reinterpret_cast<const uint4*>(x + static_cast<size_t>(w.r0 + r) * s.np + w.c0 + c), kViewF16, o[q]);
    if (tr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) stage[r][c + i] = o[q][i];
    }
  }
  const int rows = tr ? s.n : s.m, cols = tr ? s.m : s.n;  // as stored
  const int r0 = tr ? w.c0 : w.r0, c0 = tr ? w.r0 : w.c0;
  if (tr) __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int r, c;
    place(tr, q, r, c);
    const int have = r0 + r < rows ? cols - (c0 + c) : 0;
    const long long at = w.e * s.dst_bs + (r0 + r) * s.dst_ld + c0 + c;
    if (tr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[q][i] = stage[c + i][r];
    }
    float d[8];
    if (p.decay != 0.0f) {
      load_eight(s.dst, s.dst_type, at, have, s.dst_vec != 0, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = fmaf(p.decay, d[i], s.coef * o[q][i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = s.coef * o[q][i];
    }
    store_eight(s.dst, s.dst_type, at, have, s.dst_vec != 0, d);
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
