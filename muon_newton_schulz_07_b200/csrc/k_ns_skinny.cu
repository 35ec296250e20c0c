// Newton-Schulz for matrices of few rows (attention heads, low-rank factors): every iteration on chip.
//
//   X0 = X / (||X||_F + eps);   k times: A = X X^T, B' = a I + b A + c A A, X <- B' X
//
// for min(rows, cols) = m <= 128 and n = max(rows, cols) up to 8 x 512, in fp16 operands
// (MUON_MODE_HALF).  The general path pads m to 256, which costs a 64-row head 4 (update) to 16
// (Gram) times its work, and takes 3 k launches that each read X or A from L2.  Here a cluster of
// C CTAs owns a tile of 128 rows x n: CTA c keeps columns [c w, c w + w) of X in shared memory
// for the whole iteration, and the matrix is read from and written to global memory in the
// caller's own layout, once each (fp32 sources twice: the second read is an L2 hit).
//
// Several small matrices share a tile: a matrix takes h rows, h the power of two >= m (8 at least), and
// up to 128 / h of them make the tile's X a stack whose A is masked to its h x h diagonal blocks.
// B' is then block diagonal and B' X the stack of the updates.  A matrix that is not finite would reach
// its neighbours through 0 x NaN, so its rows are taken out of the tile (and its output is NaN) as
// soon as its norm or a diagonal entry of its A says so.
//
// Shared memory: X as w / 64 chunks of 128 rows x 64 columns (16 KB, 128-byte swizzle).  One layout
// serves both products: read along k = n it is the K-major operand of the Gram product, read along
// k = m the MN-major second operand of the update.  Then A, replaced by B' (32 KB, K-major).  The
// fp32 shares of A that the CTAs of a cluster hold are added in a fixed order through
// distributed shared memory: for C = 2 each CTA receives the other's share of its 64 rows in the
// place of A (which nothing reads then), for C > 2 in 64 KB of its own.
// TMEM (512 columns): A | A A | two 128-column buffers of the update.
//
// Warp 8 issues the MMAs, warps 0..7 do the rest.  The update runs in blocks of 128 columns, in
// place (a block reads no other block's columns): while the warps turn block b into the new X, the tensor
// core computes block b + 1, and block b enters the next iteration's Gram product as soon as it
// is stored.  So an iteration costs its MMAs (2 x 128 x 128 x w) plus the A -> B' chain.
//
// Rounding: X, A and B' are fp16 (2^-11), products and sums fp32.  B' is dominated by its
// diagonal, where one rounding shifts a whole row of the update the same way; that remainder is kept in fp32 and
// added in the update's epilogue, which costs a read of the old X and an FMA a value and takes a
// third off the error of the result (64 x 768, five quintic iterations: 1.9e-3 -> 1.2e-3).
//
// All waits are bounded; a CTA whose wait runs out records the timeout, stops its work, and still
// takes every barrier of the schedule.
#include <algorithm>
#include <atomic>

#include "muon_view.cuh"

namespace muon {
namespace {

constexpr int EPI_WARPS = 8;                 // two per TMEM lane quadrant
constexpr int EPI = 32 * EPI_WARPS;
constexpr int THREADS = EPI + 32;            // and the MMA issuer
constexpr uint32_t CHUNK = 16384;            // 128 rows x 64 columns of fp16
constexpr uint32_t ABUF_BYTES = 2 * CHUNK;
constexpr uint32_t PART_BYTES = 128 * 128 * 4;
constexpr uint32_t MISC_BYTES = 1024;
constexpr size_t SMEM_LIMIT = 232448;
constexpr size_t SMEM_ONE = 120 * 1024;      // at least this much, so that an SM holds one CTA
constexpr uint32_t T_A = 0, T_AA = 128, T_UPD = 256;  // TMEM columns

__host__ __device__ constexpr size_t smem_bytes(int width, int cluster) {
  const size_t need = 1024 + static_cast<size_t>(width / 64) * CHUNK + ABUF_BYTES +
                      (cluster > 2 ? PART_BYTES : 0) + MISC_BYTES;
  // More than half of an SM: every CTA takes all of TMEM, so two clusters that shared two SMs could
  // each hold what the other waits for.
  return need > SMEM_ONE ? need : SMEM_ONE;
}
static_assert(smem_bytes(kSkinnyColsOne, 2) <= SMEM_LIMIT, "one CTA, or two");
static_assert(smem_bytes(kSkinnyColsPart, 4) <= SMEM_LIMIT, "a CTA of a larger cluster");

__device__ __forceinline__ uint32_t pack2h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8h(const float* v) {
  return make_uint4(pack2h(v[0], v[1]), pack2h(v[2], v[3]), pack2h(v[4], v[5]), pack2h(v[6], v[7]));
}
// 16-byte group u (8 columns) of row r in a 128-row operand.
__device__ __forceinline__ uint32_t group_at(int r, int u) {
  return static_cast<uint32_t>(u >> 3) * CHUNK + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}
// Place of a 16-byte group (4 columns) of fp32 row r in a 128-column share of A.
__device__ __forceinline__ uint32_t share_at(int r, int q) { return (r * 32 + (q ^ (r & 7))) * 16; }

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
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(EPI) : "memory"); }

// 8 x 8 transposition of 16-bit values: q[k] holds eight values of row k, then of column k.
__device__ __forceinline__ void transpose8(uint4 (&q)[8]) {
  uint32_t in[8][4], out[8][4];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    in[k][0] = q[k].x; in[k][1] = q[k].y; in[k][2] = q[k].z; in[k][3] = q[k].w;
  }
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      out[2 * w][h] = __byte_perm(in[2 * h][w], in[2 * h + 1][w], 0x5410);
      out[2 * w + 1][h] = __byte_perm(in[2 * h][w], in[2 * h + 1][w], 0x7632);
    }
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
}

__global__ void __launch_bounds__(THREADS, 1) ns_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nch = p.width / 64;
  const int C = p.cluster;
  uint8_t* xbuf = smem;
  uint8_t* abuf = smem + nch * CHUNK;
  uint8_t* share = abuf + ABUF_BYTES;  // C > 2 only
  uint8_t* misc = share + (C > 2 ? PART_BYTES : 0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t a_full = bar0, a_ready = bar0 + 8, aa_full = bar0 + 16, b_ready = bar0 + 24, upd_full = bar0 + 32,
                 upd_done = bar0 + 48;  // upd_full, upd_done: two each, for even and odd blocks
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 64);
  volatile uint8_t* poison = misc + 128;                               // per matrix of the tile
  volatile float* remainder = reinterpret_cast<float*>(misc + 256);    // of each row's diagonal entry of B'
  const uint32_t xaddr = smem_u32(xbuf), aaddr = smem_u32(abuf), saddr = smem_u32(share);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / C;
  const int lh = __ffs(p.slot_rows) - 1;         // log2 of the rows of a matrix in the tile
  const int used = p.slots << lh;                // rows of the tile in use
  const int used16 = (used + 15) & ~15;
  const int col0 = rank * p.width;               // this CTA's first column
  const int first_mat = tile * p.slots;
  const int nblk = (p.width + 127) / 128;
  const uint64_t tmo = p.timeout_ns;
  auto sync_all = [&]() {                        // every thread of the tile
    tc_fence_before();
    if (C > 1) cluster_arrive_wait();
    else __syncthreads();
    tc_fence_after();
  };
  bool ok = true;
  auto wait_on = [&](uint32_t bar, uint32_t par) {
    if (ok) ok = mbar_wait_bounded(bar, par, tmo, nullptr, p.status);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  };

  if (tid == 0) {
    mbar_init(a_full, 1);
    mbar_init(a_ready, EPI_WARPS);
    mbar_init(aa_full, 1);
    mbar_init(b_ready, EPI_WARPS);
    mbar_init(upd_full, 1);
    mbar_init(upd_full + 8, 1);
    mbar_init(upd_done, EPI_WARPS);
    mbar_init(upd_done + 8, EPI_WARPS);
    fence_barrier_init();
  }
  if (tid < 128) {
    poison[tid] = 0;
    remainder[tid] = 0.0f;
  }
  if (warp == EPI_WARPS) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- X0 into shared memory
  // In blocks of 8 rows x 8 columns, eight 16-byte loads of 16-bit sources each: rows of the
  // storage are rows of the block or, for transposed storage, its columns.  Eight lanes take
  // neighbouring columns and a thread always the same rows, so of one matrix.  16-bit values wait
  // for their norm in shared memory as they came; fp32 ones are read again.
  const int groups = p.width / 8;                // a multiple of 8
  const int ig = (tid >> 3) & 15;                // rows 8 ig .. 8 ig + 7
  const int i0 = (ig * 8) & (p.slot_rows - 1);   // the first of them, within the matrix
  const int slot_l = (ig * 8) >> lh;
  int seg = 0, e = -1;                           // view of those rows, and matrix within it (-1: none)
  if (ig * 8 < used && first_mat + slot_l < p.total && i0 < p.m) {
    while (seg + 1 < p.nseg && p.seg[seg + 1].mat_begin <= first_mat + slot_l) ++seg;
    e = first_mat + slot_l - p.seg[seg].mat_begin;
  }
  const ViewSeg& sg = p.seg[seg];
  const int u0 = ((tid >> 7) << 3) + (tid & 7);  // first group of this thread, then every 16th
  const bool wide_src = sg.src_type == kViewF32;
  float* part = reinterpret_cast<float*>(abuf);  // [2][16] sums of squares; A is not there yet
  float* total = part + 32;                      // [16]
  float2* factor = reinterpret_cast<float2*>(total + 16);  // [16] by slot
  // the storage rows of block (ig, u): address of the first, distance, how many, values in each
  struct Block { long long at; long long ld; int rows, have; };
  auto block_of = [&](int u, bool tr, long long ld, long long bs) {
    const int j = col0 + u * 8;
    Block b;
    b.ld = ld;
    b.at = e * bs + (tr ? j * ld + i0 : i0 * ld + j);
    b.rows = tr ? p.n - j : p.m - i0;
    b.have = tr ? p.m - i0 : p.n - j;
    if (e < 0 || b.have <= 0) b.rows = 0;
    return b;
  };
  auto load_f32 = [&](const Block& b, float (&v)[8][8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      load_eight(sg.src, kViewF32, b.at + k * b.ld, k < b.rows ? b.have : 0, sg.src_vec != 0, v[k]);
  };
  if (warp < EPI_WARPS) {
    float ss = 0.0f;
#pragma unroll 1
    for (int u = u0; u < groups; u += 16) {
      const Block b = block_of(u, sg.src_tr != 0, sg.src_ld, sg.src_bs);
      if (wide_src) {
        float v[8][8];
        load_f32(b, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[k][i], v[k][i], ss);
      } else {
        uint4 q[8];
        const uint16_t* src = static_cast<const uint16_t*>(sg.src) + b.at;
        if (sg.src_vec && b.rows >= 8 && b.have >= 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = __ldg(reinterpret_cast<const uint4*>(src + k * b.ld));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = k < b.rows && 2 * i < b.have ? src[k * b.ld + 2 * i] : 0;
              const uint32_t hi = k < b.rows && 2 * i + 1 < b.have ? src[k * b.ld + 2 * i + 1] : 0;
              w[i] = lo | hi << 16;
            }
            q[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float v[8];
          widen8(q[k], sg.src_type, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        }
        if (sg.src_tr) transpose8(q);
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = q[k];
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 7) == 0) part[(tid >> 7) * 16 + ig] = ss;
  }
  sync_all();  // (also: barriers initialised, TMEM allocated)
  const uint32_t tmem = *tmem_slot;
  if (tid < 16) {
    float t = 0.0f;
    for (int c = 0; c < C; ++c)
      for (int h = 0; h < 2; ++h)
        t += C > 1 ? ld_cluster_f32(map_to_rank(smem_u32(part + h * 16 + tid), c)) : part[h * 16 + tid];
    total[tid] = t;
  }
  __syncthreads();
  if (tid < 128 && (tid & (p.slot_rows - 1)) == 0 && tid < used) {  // one thread a matrix
    const int slot = tid >> lh;
    float t = 0.0f;
    for (int i = 0; i * 8 < p.slot_rows; ++i) t += total[(tid >> 3) + i];
    const float norm = sqrtf(t);
    const Normaliser nz = normaliser(norm, p.eps);
    const bool fine = isfinite(norm);
    if (!fine) poison[slot] = 1;
    factor[slot] = make_float2(nz.pre, fine ? nz.mul : 0.0f);
    if (first_mat + slot < p.total && rank == 0) {
      int s = 0;
      while (s + 1 < p.nseg && p.seg[s + 1].mat_begin <= first_mat + slot) ++s;
      p.norms[p.seg[s].caller_idx + first_mat + slot - p.seg[s].mat_begin] = norm;
    }
  }
  __syncthreads();
  if (warp < EPI_WARPS) {
    const bool out = slot_l >= p.slots || poison[slot_l] != 0;
    const float2 f = out ? make_float2(0.0f, 0.0f) : factor[slot_l];
#pragma unroll 1
    for (int u = u0; u < groups; u += 16) {
      uint4 q[8];
      if (wide_src) {
        float v[8][8];
        load_f32(block_of(u, sg.src_tr != 0, sg.src_ld, sg.src_bs), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[k][i] = out ? 0.0f : v[k][i] * f.x * f.y;
          q[k] = pack8h(v[k]);
        }
        if (sg.src_tr) transpose8(q);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float v[8];
          widen8(*reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u)), sg.src_type, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = out ? 0.0f : v[i] * f.x * f.y;
          q[k] = pack8h(v);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = q[k];
    }
  }
  sync_all();  // the sums and factors have been read, here and by the whole cluster
  for (uint32_t i = tid * 16; i < ABUF_BYTES; i += THREADS * 16)
    *reinterpret_cast<uint4*>(abuf + i) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  sync_all();

  if (warp == EPI_WARPS) {
    // -------------------------------------------------------------- MMA issuer
    const uint32_t idesc_sym = idesc_f16_f32(true, 128, used16, 0, 0);
    const int ksteps = used16 / 16;
    auto gram_block = [&](int b) {
      for (int c = 2 * b; c < min(nch, 2 * b + 2); ++c) {
        const uint64_t d = smem_desc_sw128(xaddr + c * CHUNK, 16, 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc_mma_bf16(tmem + T_A, d + ((32u * j) >> 4), d + ((32u * j) >> 4), idesc_sym, (c | j) != 0 ? 1u : 0u);
      }
    };
    auto update_block = [&](int b) {
      const uint32_t idesc = idesc_f16_f32(true, 128, min(128, p.width - b * 128), 0, 1);
      const uint32_t d = tmem + T_UPD + (b & 1) * 128;
      for (int j = 0; j < ksteps; ++j) {
        const uint64_t ad = smem_desc_sw128(aaddr + (j >> 2) * CHUNK + (j & 3) * 32, 16, 1024);
        const uint64_t bd = smem_desc_sw128(xaddr + b * 2 * CHUNK + j * 2048, CHUNK, 1024);
        tc_mma_bf16(d, ad, bd, idesc, j != 0 ? 1u : 0u);
      }
      tc_commit(upd_full + 8 * (b & 1));
    };
    uint32_t done[2] = {0, 0};  // phases of upd_done
    if (lane == 0 && p.k > 0) {
      for (int b = 0; b < nblk; ++b) gram_block(b);
      tc_commit(a_full);
    }
#pragma unroll 1
    for (int it = 0; it < p.k; ++it) {
      __syncwarp();
      if (C > 1) {
        for (int i = 0; i < (C == 2 ? 4 : 2); ++i) cluster_arrive_wait();
      }
      wait_on(a_ready, it & 1);
      if (lane == 0 && ok) {
        for (int j = 0; j < ksteps; ++j) {
          const uint64_t d = smem_desc_sw128(aaddr + (j >> 2) * CHUNK + (j & 3) * 32, 16, 1024);
          tc_mma_bf16(tmem + T_AA, d, d, idesc_sym, j != 0 ? 1u : 0u);
        }
        tc_commit(aa_full);
      }
      __syncwarp();
      wait_on(b_ready, it & 1);
      if (lane == 0 && ok) {
        update_block(0);
        if (nblk > 1) update_block(1);
      }
      __syncwarp();
      for (int b = 0; b < nblk; ++b) {
        // block b is the new X and its TMEM columns are free.  (A barrier each for even and odd
        // blocks: the warps may finish block b + 1 before this wait, but not b + 2.)
        wait_on(upd_done + 8 * (b & 1), done[b & 1] & 1);
        ++done[b & 1];
        if (lane == 0 && ok) {
          if (b + 2 < nblk) update_block(b + 2);
          if (it + 1 < p.k) {
            gram_block(b);
            if (b + 1 == nblk) tc_commit(a_full);
          }
        }
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------- the other warps
    const int quad = warp & 3, half = warp >> 2;
    const int r = quad * 32 + lane;                       // this thread's row of the tile
    const bool active = quad * 32 < used;                 // rows that hold a matrix (warp-uniform)
    const int slot = r < used ? r >> lh : -1;             // -1: no matrix, the row stays 0
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int ca0 = half * 64;                            // this thread's columns of A
    uint32_t uses[2] = {0, 0};                            // phases of upd_full
    constexpr float kGram = kHalfA / (kHalfX * kHalfX);
    // columns ca0 + c .. + 31 of this row's A: scaled, outside the row's own matrix 0, as fp16
    auto pack_a = [&](int c, float (&v)[32], uint4 (&q)[4]) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = ((ca0 + c + i) >> lh) == slot ? v[i] * kGram : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = pack8h(v + 8 * i);
    };
#pragma unroll 1
    for (int it = 0; it < p.k; ++it) {
      // ------------------------------------------------------------ A
      wait_on(a_full, it & 1);
      if (C == 1) {
        if (ok && active) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float v[32];
            uint4 q[4];
            tmem_ld_32cols(t_row + T_A + ca0 + c, v);
            pack_a(c, v, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(abuf + group_at(r, ((ca0 + c) >> 3) + i)) = q[i];
          }
        }
        fence_async_smem();
      } else if (C == 2) {
        // rank 0 adds up rows 0..63, rank 1 rows 64..127
        const bool mine = (quad >> 1) == rank;
        const uint32_t peer = static_cast<uint32_t>(rank ^ 1);
        uint4 q[8];
        tc_fence_before();
        cluster_arrive_wait();  // neither tensor core reads A any more
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32];
          if (!mine && ok) {
            tmem_ld_32cols(t_row + T_A + ca0 + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_cluster_v4(map_to_rank(aaddr + share_at(r & 63, ((ca0 + c) >> 2) + i), peer),
                            make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                       __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
          }
        }
        tc_fence_before();
        cluster_arrive_wait();  // the shares have arrived
        tc_fence_after();
        if (mine && ok) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float v[32];
            uint4 h[4];
            tmem_ld_32cols(t_row + T_A + ca0 + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 t = *reinterpret_cast<const float4*>(abuf + share_at(r & 63, ((ca0 + c) >> 2) + i));
              v[4 * i] += t.x; v[4 * i + 1] += t.y; v[4 * i + 2] += t.z; v[4 * i + 3] += t.w;
            }
            pack_a(c, v, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) q[(c >> 3) + i] = h[i];
          }
        }
        cluster_arrive_wait();  // and been read
        if (mine && ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = group_at(r, (ca0 >> 3) + i);
            *reinterpret_cast<uint4*>(abuf + at) = q[i];
            st_cluster_v4(map_to_rank(aaddr + at, peer), q[i]);
          }
        }
        fence_async_all();
        tc_fence_before();
        cluster_arrive_wait();
      } else {
        if (ok) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float v[32];
            tmem_ld_32cols(t_row + T_A + ca0 + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(share + share_at(r, ((ca0 + c) >> 2) + i)) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        tc_fence_before();
        cluster_arrive_wait();
        // rows 128 rank / C .. of A: the shares of every CTA, in order, then one rounding
        const int rows = 128 / C;
        for (int idx = tid; idx < rows * 16; idx += EPI) {
          const int rr = rank * rows + (idx >> 4), u = idx & 15;
          float s[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = 0.0f;
          for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 t = ld_cluster_v4(map_to_rank(saddr + share_at(rr, u * 2 + h), c));
              s[4 * h] += t.x; s[4 * h + 1] += t.y; s[4 * h + 2] += t.z; s[4 * h + 3] += t.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = ((u * 8 + i) >> lh) == (rr >> lh) ? s[i] * kGram : 0.0f;
          const uint4 h = pack8h(s);
          for (int c = 0; c < C; ++c) st_cluster_v4(map_to_rank(aaddr + group_at(rr, u), c), h);
        }
        fence_async_all();
        tc_fence_before();
        cluster_arrive_wait();
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_ready);
      epi_sync();
      if (tid < 128) {  // a row of X that left fp16's range shows on the diagonal of A
        const __half d = *reinterpret_cast<const __half*>(abuf + group_at(tid, tid >> 3) + (tid & 7) * 2);
        if (tid < used && (__hisinf(d) || __hisnan(d))) poison[tid >> lh] = 1;
      }
      // ------------------------------------------------------------ B' = a I + b A + c A A
      wait_on(aa_full, it & 1);
      epi_sync();
      if (ok && active) {
        const bool out = slot < 0 || poison[slot] != 0;
        const float ca = p.coef[it][0], cb = p.coef[it][1] * (1.0f / kHalfA),
                    cc = p.coef[it][2] * (1.0f / (kHalfA * kHalfA));
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32];
          tmem_ld_32cols(t_row + T_AA + ca0 + c, v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint8_t* at = abuf + group_at(r, ((ca0 + c) >> 3) + q);
            float a8[8];
            widen8(*reinterpret_cast<const uint4*>(at), kViewF16, a8);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int col = ca0 + c + q * 8 + i;
              const float diag = col == r ? ca : 0.0f;
              float x = fmaf(cc, v[8 * q + i], fmaf(cb, a8[i], diag));
              x = (col >> lh) == slot && !out ? x : 0.0f;
              v[8 * q + i] = x;
              if (col == r) remainder[r] = x - __half2float(__float2half_rn(x));
            }
            *reinterpret_cast<uint4*>(at) = pack8h(v + 8 * q);
          }
        }
        if (out && slot >= 0) {  // nothing of this matrix may meet the others' rows
          for (int u = half; u < groups; u += 2)
            *reinterpret_cast<uint4*>(xbuf + group_at(r, u)) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_ready);
      epi_sync();  // the remainders
      const float rest = active ? remainder[r] : 0.0f;
      // ------------------------------------------------------------ X <- B' X
#pragma unroll 1
      for (int b = 0; b < nblk; ++b) {
        wait_on(upd_full + 8 * (b & 1), uses[b & 1] & 1);
        ++uses[b & 1];
        const int chunks = min(128, p.width - b * 128) / 32;
        if (ok && active) {
#pragma unroll 1
          for (int ch = half; ch < chunks; ch += 2) {
            float v[32];
            tmem_ld_32cols(t_row + T_UPD + (b & 1) * 128 + ch * 32, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint8_t* at = xbuf + group_at(r, b * 16 + ch * 4 + q);
              float x[8];
              widen8(*reinterpret_cast<const uint4*>(at), kViewF16, x);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[8 * q + i] = fmaf(rest, x[i], v[8 * q + i]);
              *reinterpret_cast<uint4*>(at) = pack8h(v + 8 * q);
            }
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(upd_done + 8 * (b & 1));
      }
    }
    epi_sync();  // X_k is complete

    // -------------------------------------------------------------- X_k to its view
    if (e >= 0) {
      const bool nan = poison[slot_l] != 0;
      const float coef = nan ? __uint_as_float(0x7FC00000u) : sg.coef;
#pragma unroll 1
      for (int u = u0; u < groups; u += 16) {
        const Block b = block_of(u, sg.dst_tr != 0, sg.dst_ld, sg.dst_bs);
        uint4 q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = *reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u));
        if (sg.dst_tr) transpose8(q);
        if (p.decay != 0.0f) {
          float w[8][8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            load_eight(sg.dst, sg.dst_type, b.at + k * b.ld, k < b.rows ? b.have : 0, sg.dst_vec != 0, w[k]);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v[8];
            widen8(q[k], kViewF16, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(p.decay, w[k][i], coef * v[i]);
            store_eight(sg.dst, sg.dst_type, b.at + k * b.ld, k < b.rows ? b.have : 0, sg.dst_vec != 0, v);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v[8];
            widen8(q[k], kViewF16, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= coef;
            store_eight(sg.dst, sg.dst_type, b.at + k * b.ld, k < b.rows ? b.have : 0, sg.dst_vec != 0, v);
          }
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  sync_all();  // no CTA leaves while its shared memory may be read
  if (warp == EPI_WARPS) {
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
