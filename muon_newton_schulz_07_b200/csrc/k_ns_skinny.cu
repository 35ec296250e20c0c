// Newton-Schulz for matrices of few rows (attention heads, low-rank factors): every iteration on chip.
//
//   X0 = X / (||X||_F + eps);   k times: A = X X^T, B' = a I + b A + c A A, X <- B' X
//
// for min(rows, cols) = m <= 128 and n = max(rows, cols) up to 8 x 512, in fp16 operands
// (MUON_MODE_HALF).  The general path pads m to 256, which costs a 64-row head 4 (update) to 16
// (Gram) times its work, and takes 3 k launches that each read X or A from L2.  Here a cluster of
// C CTAs owns a tile of 128 rows x n: CTA c keeps columns [c w, c w + w) of X in shared memory
// for the whole iteration, and the matrix is read from and written to global memory in the
// caller's own layout, once each (the norm's pass reads it too; the second read is an L2 hit).
//
// Several small matrices share a tile: a matrix takes h rows, h the power of two >= m, and 128 / h
// of them make the tile's X a stack whose A is masked to its h x h diagonal blocks.  B' is then
// block diagonal and B' X the stack of the updates, so a tile costs the tensor cores the same
// however many matrices it holds.  A matrix that is not finite would reach its neighbours through 0 x NaN,
// so its rows are taken out of the tile (and its output is NaN) as soon as its norm or a diagonal
// entry of its A says so.
//
// Shared memory: X as w / 64 chunks of 128 rows x 64 columns (16 KB, 128-byte swizzle).  One layout
// serves both products: read along k = n it is the K-major operand of the Gram product, read along
// k = m the MN-major second operand of the update.  Then A, replaced by B' (32 KB, K-major), and
// for C > 1 the CTA's fp32 share of A (64 KB): CTA c adds rows 128 c / C .. of all shares in a
// fixed order and stores them, rounded once, into every CTA's A through distributed shared memory.
// TMEM (512 columns): A | A A in columns 0..255, and the update in 256-column blocks that alternate
// between 256..511 and 0..255 (A and A A have been read by then), in place: the update of
// a column block reads no other column.
//
// All waits are bounded; a CTA whose wait runs out records the timeout, stops its work, and still
// takes every barrier of the schedule.
#include <algorithm>
#include <atomic>

#include "muon_view.cuh"

namespace muon {
namespace {

constexpr int THREADS = 256;                 // 8 warps, two per TMEM lane quadrant
constexpr uint32_t CHUNK = 16384;            // 128 rows x 64 columns of fp16
constexpr uint32_t ABUF_BYTES = 2 * CHUNK;
constexpr uint32_t PART_BYTES = 128 * 128 * 4;
constexpr uint32_t MISC_BYTES = 512;
constexpr size_t SMEM_LIMIT = 232448;
constexpr size_t SMEM_ONE = 120 * 1024;      // at least this much, so that an SM holds one CTA

__host__ __device__ constexpr size_t smem_bytes(int width, int cluster) {
  const size_t need = 1024 + static_cast<size_t>(width / 64) * CHUNK + ABUF_BYTES + (cluster > 1 ? PART_BYTES : 0) + MISC_BYTES;
  // More than half of an SM: every CTA takes all of TMEM, so two clusters that shared two SMs could
  // each hold what the other waits for.
  return need > SMEM_ONE ? need : SMEM_ONE;
}
static_assert(smem_bytes(kSkinnyColsOne, 1) <= SMEM_LIMIT, "one CTA");
static_assert(smem_bytes(kSkinnyColsPart, 2) <= SMEM_LIMIT, "a CTA of a cluster");

__device__ __forceinline__ uint4 pack8h(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16-byte group u (8 columns) of row r in a 128-row chunk.
__device__ __forceinline__ uint32_t group_at(int r, int u) {
  return static_cast<uint32_t>(u >> 3) * CHUNK + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(THREADS, 1) ns_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nch = p.width / 64;
  const int C = p.cluster;
  uint8_t* xbuf = smem;
  uint8_t* abuf = smem + nch * CHUNK;
  float* share = reinterpret_cast<float*>(abuf + ABUF_BYTES);  // C > 1 only
  uint8_t* misc = abuf + ABUF_BYTES + (C > 1 ? PART_BYTES : 0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  const uint32_t mma_bar = smem_u32(bars), upd_bar = smem_u32(bars + 1);  // upd_bar: two
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3);
  volatile uint8_t* poison = misc + 64;  // per matrix of the tile
  const uint32_t xaddr = smem_u32(xbuf), aaddr = smem_u32(abuf);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / C;
  const int lh = __ffs(p.slot_rows) - 1;         // log2 of the rows of a matrix in the tile
  const int used = p.slots << lh;                // rows of the tile in use
  const int col0 = rank * p.width;               // this CTA's first column
  const int first_mat = tile * p.slots;
  const uint64_t tmo = p.timeout_ns;
  auto sync_all = [&]() {                        // every thread of the tile
    tc_fence_before();
    if (C > 1) cluster_arrive_wait();
    else __syncthreads();
    tc_fence_after();
  };
  // The view of a row of the tile; returns its matrix within the view, or -1 (no such row).
  auto view_of = [&](int r, int& seg) -> int {
    const int mat = first_mat + (r >> lh);
    if (r >= used || mat >= p.total || (r & (p.slot_rows - 1)) >= p.m) return -1;
    int s = 0;
    while (s + 1 < p.nseg && p.seg[s + 1].mat_begin <= mat) ++s;
    seg = s;
    return mat - p.seg[s].mat_begin;
  };

  if (tid == 0) {
    mbar_init(mma_bar, 1);
    mbar_init(upd_bar, 1);
    mbar_init(upd_bar + 8, 1);
    fence_barrier_init();
  }
  if (tid < 128) poison[tid] = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- norms
  float* rowpart = reinterpret_cast<float*>(abuf);   // [2][128], then totals and factors; A is not there yet
  float* rowtot = rowpart + 256;
  float* rowall = rowtot + 128;
  float2* factor = reinterpret_cast<float2*>(rowall + 128);
  const int groups = p.width / 8;
  int seg0 = 0;
  const bool tr = view_of(0, seg0) >= 0 && p.seg[seg0].src_tr != 0;  // decides the order of the reads only
  auto read_group = [&](int r, int u, float (&v)[8]) {
    int seg;
    const int e = view_of(r, seg);
    const int i = r & (p.slot_rows - 1), j = col0 + u * 8;
    if (e < 0 || j >= p.n) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = 0.0f;
      return;
    }
    const ViewSeg& s = p.seg[seg];
    if (!s.src_tr) {
      load_eight(s.src, s.src_type, e * s.src_bs + i * s.src_ld + j, p.n - j, s.src_vec != 0, v);
    } else {
      const long long at = e * s.src_bs + i;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = j + q < p.n ? load_one(s.src, s.src_type, at + (j + q) * s.src_ld) : 0.0f;
    }
  };
  if (!tr) {
    for (int r = warp; r < 128; r += THREADS / 32) {
      float ss = 0.0f;
      for (int u = lane; u < groups; u += 32) {
        float v[8];
        read_group(r, u, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(v[q], v[q], ss);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (lane == 0) rowtot[r] = ss;
    }
  } else {
    const int r = (warp & 3) * 32 + lane;
    float ss = 0.0f;
    for (int u = warp >> 2; u < groups; u += 2) {
      float v[8];
      read_group(r, u, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(v[q], v[q], ss);
    }
    rowpart[(warp >> 2) * 128 + r] = ss;
    __syncthreads();
    if (tid < 128) rowtot[tid] = rowpart[tid] + rowpart[128 + tid];
  }
  sync_all();  // (also: barriers initialised, TMEM allocated)
  const uint32_t tmem = *tmem_slot;
  if (tid < 128) {
    float t = 0.0f;
    for (int c = 0; c < C; ++c)
      t += C > 1 ? ld_cluster_f32(map_to_rank(smem_u32(rowtot + tid), c)) : rowtot[tid];
    rowall[tid] = t;
  }
  __syncthreads();
  if (tid < p.slots) {
    float t = 0.0f;
    for (int i = 0; i < p.m; ++i) t += rowall[(tid << lh) + i];
    const float norm = sqrtf(t);
    int seg;
    const int e = view_of(tid << lh, seg);
    if (e >= 0 && rank == 0) p.norms[p.seg[seg].caller_idx + e] = norm;
    const Normaliser nz = normaliser(norm, p.eps);
    const bool fine = isfinite(norm);
    if (!fine) poison[tid] = 1;
    factor[tid] = make_float2(nz.pre, fine ? nz.mul : 0.0f);
  }
  __syncthreads();

  // ---------------------------------------------------------------- X0 into shared memory
  for (int idx = tid; idx < 128 * groups; idx += THREADS) {
    const int r = tr ? idx & 127 : idx / groups;
    const int u = tr ? idx >> 7 : idx - r * groups;
    float v[8];
    read_group(r, u, v);
    const int slot = min(r >> lh, p.slots - 1);
    const float2 f = factor[slot];
    const bool out = poison[slot] != 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = out ? 0.0f : v[q] * f.x * f.y;
    *reinterpret_cast<uint4*>(xbuf + group_at(r, u)) = pack8h(v);
  }
  sync_all();  // the factors have been read, here and (the row totals) by the whole cluster
  for (uint32_t i = tid * 16; i < ABUF_BYTES; i += THREADS * 16)
    *reinterpret_cast<uint4*>(abuf + i) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  sync_all();

  const int quad = warp & 3, half = warp >> 2;
  const int r = quad * 32 + lane;                       // this thread's row of the tile
  const bool active = quad * 32 < used;                 // rows that hold a matrix (warp-uniform)
  const int slot = r >> lh;
  const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const int nblk = (p.width + 255) / 256;
  bool ok = true;
  uint32_t mma_par = 0, upd_par0 = 0, upd_par1 = 0;
  auto wait_on = [&](uint32_t bar, uint32_t& par) {
    if (ok) ok = mbar_wait_bounded(bar, par, tmo, nullptr, p.status);
    par ^= 1u;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  };
  // keep columns c .. c + 31 of this row that belong to its own matrix
  auto masked = [&](int c, float (&v)[32]) {
    if (lh < 7) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = ((c + i) >> lh) == slot ? v[i] : 0.0f;
    }
  };
  auto put_a = [&](int c, const float (&v)[32]) {  // columns c .. of this row of A / B'
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(abuf + group_at(r, (c >> 3) + q)) = pack8h(v + 8 * q);
  };
  auto issue_update = [&](int b) {  // one thread: block b of the update
    const int n = min(256, p.width - b * 256);
    const uint32_t idesc = idesc_f16_f32(true, 128, n, 0, 1);
    const uint32_t d = tmem + ((b & 1) ? 0 : 256);
    tc_fence_after();
#pragma unroll 1
    for (int kb = 0; kb < 2; ++kb) {
      const uint64_t ad = smem_desc_sw128(aaddr + kb * CHUNK, 16, 1024);
      const uint64_t bd = smem_desc_sw128(xaddr + b * 4 * CHUNK + kb * 8192, CHUNK, 1024);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        tc_mma_bf16(d, ad + ((32u * j) >> 4), bd + ((2048u * j) >> 4), idesc, (kb | j) != 0 ? 1u : 0u);
    }
    tc_commit(upd_bar + 8 * (b & 1));
  };

  constexpr float kGram = kHalfA / (kHalfX * kHalfX);
  const uint32_t idesc_sym = idesc_f16_f32(true, 128, 128, 0, 0);
#pragma unroll 1
  for (int it = 0; it < p.k; ++it) {
    // -------------------------------------------------------------- A = X X^T
    if (tid == 0 && ok) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        const uint64_t d = smem_desc_sw128(xaddr + c * CHUNK, 16, 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc_mma_bf16(tmem, d + ((32u * j) >> 4), d + ((32u * j) >> 4), idesc_sym, (c | j) != 0 ? 1u : 0u);
      }
      tc_commit(mma_bar);
    }
    wait_on(mma_bar, mma_par);
    if (ok && (active || C > 1)) {
#pragma unroll 1
      for (int c = half * 64; c < half * 64 + 64; c += 32) {
        float v[32];
        tmem_ld_32cols(t_row + c, v);
        if (C == 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= kGram;
          masked(c, v);
          put_a(c, v);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(share + r * 128 + (((c >> 2) + q) ^ (r & 7)) * 4) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
    }
    if (C > 1) {
      sync_all();
      // rows 128 rank / C .. of A: the shares of every CTA, in order, then one rounding
      const int rows = 128 / C;
      for (int idx = tid; idx < rows * 16; idx += THREADS) {
        const int rr = rank * rows + (idx >> 4), u = idx & 15;
        float s[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = 0.0f;
        for (int c = 0; c < C; ++c) {
#pragma unroll
          for (int hq = 0; hq < 2; ++hq) {
            const uint32_t at = smem_u32(share + rr * 128 + ((u * 2 + hq) ^ (rr & 7)) * 4);
            const float4 t = ld_cluster_v4(map_to_rank(at, c));
            s[4 * hq] += t.x; s[4 * hq + 1] += t.y; s[4 * hq + 2] += t.z; s[4 * hq + 3] += t.w;
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = ((u * 8 + q) >> lh) == (rr >> lh) ? s[q] * kGram : 0.0f;
        const uint4 h = pack8h(s);
        for (int c = 0; c < C; ++c) st_cluster_v4(map_to_rank(aaddr + group_at(rr, u), c), h);
      }
      fence_async_all();
      sync_all();
    } else {
      fence_async_smem();
      sync_all();
    }
    // -------------------------------------------------------------- B' = a I + b A + c A A
    if (tid == 0 && ok) {
      tc_fence_after();
#pragma unroll 1
      for (int kb = 0; kb < 2; ++kb) {
        const uint64_t d = smem_desc_sw128(aaddr + kb * CHUNK, 16, 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc_mma_bf16(tmem + 128, d + ((32u * j) >> 4), d + ((32u * j) >> 4), idesc_sym, (kb | j) != 0 ? 1u : 0u);
      }
      tc_commit(mma_bar);
    }
    if (tid < 128) {  // a row of X that left fp16's range shows on the diagonal of A
      const __half d = *reinterpret_cast<const __half*>(abuf + group_at(tid, tid >> 3) + (tid & 7) * 2);
      if (__hisinf(d) || __hisnan(d)) poison[tid >> lh] = 1;
    }
    wait_on(mma_bar, mma_par);
    __syncthreads();
    if (ok && active) {
      const bool out = poison[slot] != 0;
      const float ca = p.coef[it][0] * kHalfB, cb = p.coef[it][1] * (kHalfB / kHalfA),
                  cc = p.coef[it][2] * (kHalfB / (kHalfA * kHalfA));
#pragma unroll 1
      for (int c = half * 64; c < half * 64 + 64; c += 32) {
        float v[32];
        tmem_ld_32cols(t_row + 128 + c, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a8[8];
          widen8(*reinterpret_cast<const uint4*>(abuf + group_at(r, (c >> 3) + q)), kViewF16, a8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float diag = c + q * 8 + i == r ? ca : 0.0f;
            v[8 * q + i] = fmaf(cc, v[8 * q + i], fmaf(cb, a8[i], diag));
          }
        }
        masked(c, v);
        if (out) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
        put_a(c, v);
      }
      if (out) {  // nothing of this matrix may meet the others' rows
        for (int u = half; u < groups; u += 2)
          *reinterpret_cast<uint4*>(xbuf + group_at(r, u)) = make_uint4(0, 0, 0, 0);
      }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    // -------------------------------------------------------------- X <- B' X
    if (tid == 0 && ok) {
      issue_update(0);
      if (nblk > 1) issue_update(1);
    }
#pragma unroll 1
    for (int b = 0; b < nblk; ++b) {
      if (b & 1) wait_on(upd_bar + 8, upd_par1);
      else wait_on(upd_bar, upd_par0);
      const int chunks = min(256, p.width - b * 256) / 32;
      const uint32_t d = t_row + ((b & 1) ? 0 : 256);
      if (ok && active) {
#pragma unroll 1
        for (int ch = half; ch < chunks; ch += 2) {
          float v[32];
          tmem_ld_32cols(d + ch * 32, v);
          const int jl = b * 256 + ch * 32;  // first column, within this CTA's
          if (it + 1 < p.k) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kHalfB;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(xbuf + group_at(r, (jl >> 3) + q)) = pack8h(v + 8 * q);
          } else {
            int seg;
            const int e = view_of(r, seg);
            const int j = col0 + jl;
            if (e >= 0 && j < p.n) {
              const ViewSeg& s = p.seg[seg];
              const int i0 = r & (p.slot_rows - 1);
              const float coef = poison[slot] != 0 ? __uint_as_float(0x7FC00000u) : s.coef * (1.0f / kHalfB);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = coef * v[8 * q + i];
                const int jq = j + 8 * q;
                if (!s.dst_tr) {
                  const long long at = e * s.dst_bs + i0 * s.dst_ld + jq;
                  if (p.decay != 0.0f) {
                    float w[8];
                    load_eight(s.dst, s.dst_type, at, p.n - jq, s.dst_vec != 0, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = fmaf(p.decay, w[i], o[i]);
                  }
                  store_eight(s.dst, s.dst_type, at, p.n - jq, s.dst_vec != 0, o);
                } else {
                  const long long at = e * s.dst_bs + i0;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    if (jq + i < p.n) {
                      const long long to = at + (jq + i) * s.dst_ld;
                      const float w = p.decay != 0.0f ? load_one(s.dst, s.dst_type, to) : 0.0f;
                      store_one(s.dst, s.dst_type, to, p.decay != 0.0f ? fmaf(p.decay, w, o[i]) : o[i]);
                    }
                  }
                }
              }
            }
          }
        }
      }
      if (b + 2 < nblk) {  // the block's TMEM columns have been read: the next but one may take them
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && ok) issue_update(b + 2);
      }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
  }

  if (p.k == 0) {  // no iteration: O = X0
    for (int idx = tid; idx < 128 * groups; idx += THREADS) {
      const int row = tr ? idx & 127 : idx / groups;
      const int u = tr ? idx >> 7 : idx - row * groups;
      int seg;
      const int e = view_of(row, seg);
      const int j = col0 + u * 8;
      if (e < 0 || j >= p.n) continue;
      const ViewSeg& s = p.seg[seg];
      float v[8];
      widen8(*reinterpret_cast<const uint4*>(xbuf + group_at(row, u)), kViewF16, v);
      const float coef = poison[row >> lh] != 0 ? __uint_as_float(0x7FC00000u) : s.coef;
      const int i0 = row & (p.slot_rows - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (j + i >= p.n) break;
        const long long to = e * s.dst_bs + (s.dst_tr ? i0 + (j + i) * s.dst_ld : i0 * s.dst_ld + j + i);
        const float w = p.decay != 0.0f ? load_one(s.dst, s.dst_type, to) : 0.0f;
        store_one(s.dst, s.dst_type, to, p.decay != 0.0f ? fmaf(p.decay, w, coef * v[i]) : coef * v[i]);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  sync_all();  // no CTA leaves while its shared memory may be read
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_ns_skinny(const SkinnyParams& p, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  // The shared-memory limit is a property of the function on each device: set it once per device.
  static std::atomic<unsigned long long> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((attr_set.load() & bit) == 0) {
    e = cudaFuncSetAttribute(ns_skinny_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SMEM_LIMIT));
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(bit);
  }
  const int tiles = (p.total + p.slots - 1) / p.slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * p.cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes(p.width, p.cluster);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ns_skinny_kernel, p);
}

}  // namespace muon
