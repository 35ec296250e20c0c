// Newton-Schulz for matrices of few rows (attention heads, low-rank factors): every iteration on chip.
//
//   X0 = X / (||X||_F + eps);   k times: A = X X^T, B' = a I + b A + c A A, X <- B' X
//
// for min(rows, cols) = m <= 128 and n = max(rows, cols) up to 8 x 512 (of at most 64 rows, cut into column ranges, up to
// that for each: 16 x 4096 for 8 rows), in fp16 operands (MUON_MODE_HALF).  The general path pads m to 256, which costs a 64-row head 4 (update) to 16
// (Gram) times its work, and takes 3 k launches that each read X or A from L2.  Here a cluster of
// C CTAs owns a tile of 128 rows x n: CTA c keeps columns [c w, c w + w) of X in shared memory
// for the whole iteration, and the matrix is read from and written to global memory in the
// caller's own layout, once each (fp32 sources twice: the second read is an L2 hit).
//
// A matrix of h rows, h the power of two >= m (8 at least), fills the 128 rows as F column ranges below
// each other (a 64 x 768 matrix is 128 x 384): the Gram product's h x h diagonal blocks then add up to its A,
// and the update multiplies each range by the same B', a block diagonal of F copies.  And several
// matrices share a tile in the same way, each with diagonal blocks of its own.  A matrix that is not finite would reach
// its neighbours through 0 x NaN, so its rows are taken out of the tile (and its output is NaN) as
// soon as its norm or a diagonal entry of its A says so.
//
// Shared memory: X as w / 64 chunks of 128 rows x 64 columns (16 KB, 128-byte swizzle).  One layout
// serves both products: read along k = n it is the K-major operand of the Gram product, read along
// k = m the MN-major second operand of the update.  Then A (32 KB, K-major).  The fp32 shares of A
// that the CTAs of a cluster hold are added by rows: each CTA sends the owner of a row its share
// (st.async, counted by a barrier of the owner), the owner adds the shares in a fixed order, rounds
// once, and copies its rows of A to the others.  The shares arrive in 64 KB of their own or, for
// C = 2, in the place of A, which nothing reads then: that leaves room for 768 columns a CTA.
// TMEM (512 columns): A | two 128-column buffers of the update, the odd one also A A | B'.  B' and the
// freshly updated blocks of X are first operands from TMEM: with both operands in shared memory, a
// 128 x 128 MMA reads its full 128 bytes a cycle and leaves none to the epilogue.
//
// Warp 16 issues the MMAs, warps 0..15 do the rest.  The update runs in blocks of 128 columns, in
// place (a block reads no other block's columns): while the warps turn block b into the new X, the tensor
// core computes block b + 1, and block b enters the next iteration's Gram product as soon as it
// is stored.  So an iteration costs its MMAs (2 x 128 x 128 x w) plus the A -> B' chain.
//
// Rounding: X, A and B' are fp16 (2^-11), products and sums fp32.  B' is dominated by its
// diagonal, where one rounding scales a whole row of the update; the update's epilogue multiplies
// the row by the exact diagonal entry over the rounded one, which takes a third off the error
// of the result (64 x 768, five quintic iterations: 1.9e-3 -> 1.2e-3).
//
// Measured, five iterations: 12 of 64 x 768 44 us, 288 of 1536 x 128 (clusters of two) 322 us.  An iteration of 128 x 768
// a CTA takes 13 k cycles, 7 k of them the six blocks (their MMAs at the rate of the tensor core), 5 k the chain from A to the first
// block, 1 k the last block's Gram product; a cluster of two adds 6 k for the exchange of A.  Loading, converting
// and storing a tile is 30 to 45 k once, which one CTA an SM has nothing to hide behind.
//
// All waits are bounded; a CTA whose wait runs out records the timeout, stops its work, and still
// takes every barrier of the schedule.
#include <algorithm>
#include <atomic>

#include "muon_view.cuh"

namespace muon {
namespace {

constexpr int EPI_WARPS = 16;                // four per TMEM lane quadrant
constexpr int EPI = 32 * EPI_WARPS;
constexpr int THREADS = EPI + 32;            // and the MMA issuer
constexpr uint32_t CHUNK = 16384;            // 128 rows x 64 columns of fp16
constexpr uint32_t ABUF_BYTES = 2 * CHUNK;
constexpr uint32_t PART_BYTES = 128 * 128 * 4;
constexpr uint32_t MISC_BYTES = 1024;
constexpr size_t SMEM_LIMIT = 232448;
constexpr size_t SMEM_ONE = 120 * 1024;      // at least this much, so that an SM holds one CTA
constexpr uint32_t T_A = 0, T_UPD = 128, T_AA = 256, T_B = 384;  // TMEM columns (A A: the odd update buffer)

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


// 16 bytes into another CTA's shared memory, counted by a barrier of that CTA.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, float a, float b, float c, float d) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}
// A piece of this CTA's shared memory into another CTA's, counted by a barrier of that CTA.
__device__ __forceinline__ void copy_to_cta(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}
// 16 bytes from global to shared memory without passing through registers.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
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

template <int TYPE>
__device__ __forceinline__ void add_squares(const uint4& q, float2& ss) {
  float v[8];
  widen8(q, TYPE, v);
#pragma unroll
  for (int i = 0; i < 8; i += 2) ss = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(v[i], v[i + 1]), ss);
}

// Eight 16-bit values times f, from one 16-bit type to another.
template <int FROM, int TO>
__device__ __forceinline__ uint4 rescale8(const uint4& q, float f) {
  float v[8];
  widen8(q, FROM, v);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(f, f));
    if (TO == kViewBF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[i] = pack2h(x.x, x.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight neighbouring values of the result (decay 0: without reading what was there).  Not inlined: it is
// called from unrolled code that runs once.
__device__ __noinline__ void write_eight(void* dst, int type, long long at, uint4 q, float coef, float decay) {
  float v[8];
  widen8(q, kViewF16, v);
  if (decay != 0.0f) {
    float w[8];
    load_eight(dst, type, at, 8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(decay, w[i], coef * v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= coef;
  }
  store_eight(dst, type, at, 8, v);
}

// The squares of up to eight neighbouring values whatever their size.
__device__ __noinline__ double far_squares(const void* src, int type, long long at, int have) {
  double sum = 0.0;
#pragma unroll 1
  for (int c = 0; c < min(have, 8); ++c) {
    const double v = load_one(src, type, at + c);
    sum = fma(v, v, sum);
  }
  return sum;
}

// CLUSTER: 1, 2, or 4 for any larger cluster.  FOLDED: matrices are cut into column ranges (their sums in code
// that every tile carried took 288 of 1536 x 128 from 320 to 328 us).
template <int CLUSTER, bool FOLDED>
__global__ void __launch_bounds__(THREADS, 1) ns_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nch = p.width / 64;
  const int C = CLUSTER <= 2 ? CLUSTER : p.cluster;
  uint8_t* xbuf = smem;
  uint8_t* abuf = smem + nch * CHUNK;
  uint8_t* share = abuf + ABUF_BYTES;  // C > 2 only
  uint8_t* misc = share + (C > 2 ? PART_BYTES : 0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t a_full = bar0, a_ready = bar0 + 8, aa_full = bar0 + 16, b_ready = bar0 + 24, upd_full = bar0 + 32,
                 upd_done = bar0 + 48,  // upd_full, upd_done: two each, for even and odd blocks
      share_full = bar0 + 64, rows_full = bar0 + 72, peer_free = bar0 + 80, peer_read = bar0 + 88, peer_got = bar0 + 96;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 112);
  volatile uint8_t* poison = misc + 128;                               // per matrix of the tile
  volatile float* row_factor = reinterpret_cast<float*>(misc + 256);   // of each row of the update
  const uint32_t xaddr = smem_u32(xbuf), aaddr = smem_u32(abuf), saddr = smem_u32(share);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / C;
  const int lh = __ffs(p.slot_rows) - 1;         // log2 of the rows of a matrix in the tile
  const int folds = FOLDED ? p.folds : 1;        // column ranges a matrix is cut into
  const int lf = __ffs(folds) - 1;
  const int ls = lh + lf;                        // log2 of the tile's rows that hold a matrix
  const int used = p.slots << ls;                // rows of the tile in use
  const int used16 = (used + 15) & ~15;
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
    mbar_init(upd_done, EPI_WARPS / 2);
    mbar_init(upd_done + 8, EPI_WARPS / 2);
    mbar_init(share_full, 1);
    mbar_init(rows_full, 1);
    mbar_init(peer_free, 1);
    mbar_init(peer_read, 1);
    mbar_init(peer_got, C > 1 ? C - 1 : 1);
    fence_barrier_init();
  }
  if (tid < 128) {
    poison[tid] = 0;
    row_factor[tid] = 1.0f;
  }
  if (warp == EPI_WARPS) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- X0 into shared memory
  // In blocks of 8 rows x 8 columns, eight 16-byte copies of 16-bit sources each: rows of the
  // storage are rows of the block or, for transposed storage, its columns.  Eight lanes take
  // neighbouring columns and a thread always the same rows, so of one matrix.  A block's copies go,
  // all of a thread's blocks at once (cp.async), to the eight places its rows will have; there the values
  // wait for their norm, and are transposed on their way through the conversion.  fp32 sources
  // are read twice instead.
  const int groups = p.width / 8;                // a multiple of 8
  const int ig = (tid >> 3) & 15;                // rows 8 ig .. 8 ig + 7
  const int i0 = (ig * 8) & (p.slot_rows - 1);   // the first of them, within the matrix
  const int slot_l = (ig * 8) >> ls;             // the matrix of the tile
  const int col0 = ((((ig * 8) >> lh) & (folds - 1)) * C + rank) * p.width;  // first column of those rows
  int seg = 0, e = -1;                           // view of those rows, and matrix within it (-1: none)
  if (ig * 8 < used && first_mat + slot_l < p.total && i0 < p.m) {
    while (seg + 1 < p.nseg && p.seg[seg + 1].mat_begin <= first_mat + slot_l) ++seg;
    e = first_mat + slot_l - p.seg[seg].mat_begin;
  }
  const ViewSeg& sg = p.seg[seg];
  const int u0 = ((tid >> 7) << 3) + (tid & 7);  // first group of this thread, then every 32nd
  const bool wide_src = sg.src_type == kViewF32;
  double* part = reinterpret_cast<double*>(abuf);          // [4][16] sums of squares; A is not there yet
  double* total = part + 64;                               // [16]
  float* factor = reinterpret_cast<float*>(total + 16);    // [16] by matrix of the tile
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
  // Blocks that reach over the matrix's edge or whose rows are not aligned go value by value, in
  // loops: this code runs once per tile, and what it costs is fetching its instructions.
  auto whole = [&](const Block& b, bool vec) { return vec && b.rows >= 8 && b.have >= 8; };
  const bool src_tr = sg.src_tr != 0, src_vec = sg.src_vec != 0;
  if (warp < EPI_WARPS) {
    float ss = 0.0f;
    float2 ss2 = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int u = u0; u < groups; u += EPI / 16) {
      const Block b = block_of(u, src_tr, sg.src_ld, sg.src_bs);
      if (wide_src) {
        if (whole(b, src_vec)) {
          const float* src = static_cast<const float*>(sg.src) + b.at;
          float4 q[8];
#pragma unroll 1
          for (int h = 0; h < 8; h += 4) {
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k] = __ldg(reinterpret_cast<const float4*>(src + (k >> 1) * b.ld + (k & 1) * 4));
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(q[k].x, q[k].x, fmaf(q[k].y, q[k].y, fmaf(q[k].z, q[k].z, fmaf(q[k].w, q[k].w, ss))));
            src += 4 * b.ld;
          }
        } else {
#pragma unroll 2
          for (int k = 0; k < min(b.rows, 8); ++k) {
            float v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = c < b.have ? static_cast<const float*>(sg.src)[b.at + k * b.ld + c] : 0.0f;
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = fmaf(v[c], v[c], ss);
          }
        }
      } else if (whole(b, src_vec)) {
        const uint16_t* src = static_cast<const uint16_t*>(sg.src) + b.at;
        if (!src_tr) {
#pragma unroll
          for (int k = 0; k < 8; ++k) copy_async16(xaddr + group_at(ig * 8 + k, u), src + k * b.ld);
        } else {  // 64 bytes of a row by a warp, the next by its neighbour: through L1
          uint4 q[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = __ldg(reinterpret_cast<const uint4*>(src + k * b.ld));
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = q[k];
        }
      } else {
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = k < b.rows && c < b.have ? static_cast<const uint16_t*>(sg.src)[b.at + k * b.ld + c] : 0u;
          *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) =
              make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
      }
    }
    if (!wide_src) {
      copy_async_wait();  // a thread reads only what it copied itself
#pragma unroll 1
      for (int u = u0; u < groups; u += EPI / 16) {
        if (sg.src_type == kViewBF16) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            add_squares<kViewBF16>(*reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u)), ss2);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            add_squares<kViewF16>(*reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u)), ss2);
        }
      }
    }
    ss += ss2.x + ss2.y;
    double sum = ss;
    if (e >= 0 && !usual_sum(sum)) {  // squares that fp32 has no values for (see Squares): once more, in fp64
      sum = 0.0;
#pragma unroll 1
      for (int u = u0; u < groups; u += EPI / 16) {
        const Block b = block_of(u, src_tr, sg.src_ld, sg.src_bs);
#pragma unroll 1
        for (int k = 0; k < min(b.rows, 8); ++k)
          sum += wide_src ? far_squares(sg.src, kViewF32, b.at + k * b.ld, b.have)
                          : far_squares(xbuf + group_at(ig * 8 + k, u), sg.src_type, 0, b.have);
      }
    }
    if (__any_sync(0xffffffffu, sum != ss)) {
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    } else {
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sum = ss;
    }
    if ((tid & 7) == 0) part[(tid >> 7) * 16 + ig] = sum;
  }
  sync_all();  // (also: barriers initialised, TMEM allocated)
  const uint32_t tmem = *tmem_slot;
  if (tid < 16) {
    double t = 0.0;
    for (int c = 0; c < C; ++c)
      for (int h = 0; h < EPI / 128; ++h)
        t += C > 1 ? ld_cluster_f64(map_to_rank(smem_u32(part + h * 16 + tid), c)) : part[h * 16 + tid];
    total[tid] = t;
  }
  __syncthreads();
  if (tid < 128 && (tid & ((1 << ls) - 1)) == 0 && tid < used) {  // one thread a matrix
    const int slot = tid >> ls;
    double t = 0.0;
    for (int i = 0; i < (1 << ls) / 8; ++i) t += total[(tid >> 3) + i];
    if (!isfinite(t)) poison[slot] = 1;
    factor[slot] = p.normalised ? 1.0f : normaliser(t, p.eps);
    if (first_mat + slot < p.total && rank == 0 && !p.normalised) {
      int s = 0;
      while (s + 1 < p.nseg && p.seg[s + 1].mat_begin <= first_mat + slot) ++s;
      p.norms[p.seg[s].caller_idx + first_mat + slot - p.seg[s].mat_begin] = norm_of(t);
    }
  }
  __syncthreads();
  if (warp < EPI_WARPS) {
    const bool out = slot_l >= p.slots || poison[slot_l] != 0;
    const float f = out ? 0.0f : factor[slot_l];
#pragma unroll 1
    for (int u = u0; u < groups; u += EPI / 16) {
      const Block b = block_of(u, src_tr, sg.src_ld, sg.src_bs);
      if (out || b.rows <= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = make_uint4(0, 0, 0, 0);
      } else if (wide_src) {
        const bool full = whole(b, src_vec);
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {  // (fp32: the second read, an L2 hit)
          float v[8];
          if (full) {
            load_eight(sg.src, kViewF32, b.at + k * b.ld, 8, v);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = k < b.rows && i < b.have ? static_cast<const float*>(sg.src)[b.at + k * b.ld + i] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= f;
          if (!src_tr) {
            *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = pack8h(v);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<__half*>(xbuf + group_at(ig * 8 + i, u) + k * 2) = __float2half_rn(v[i]);
          }
        }
      } else {
        uint4 q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = *reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u));
        if (sg.src_type == kViewBF16) {
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = rescale8<kViewBF16, kViewF16>(q[k], f);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = rescale8<kViewF16, kViewF16>(q[k], f);
        }
        if (src_tr) transpose8(q);
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(xbuf + group_at(ig * 8 + k, u)) = q[k];
      }
    }
  }
  fence_async_smem();
  sync_all();  // (and the sums and factors have been read, here and by the whole cluster)

  if (warp == EPI_WARPS) {
    // -------------------------------------------------------------- MMA issuer
    {
      const uint32_t lead = elect_one();
      const uint32_t idesc_sym = idesc_f16_f32(true, 128, used16, 0, 0);
      const uint32_t idesc_128 = idesc_f16_f32(true, 128, 128, 0, 1), idesc_64 = idesc_f16_f32(true, 128, 64, 0, 1);
      const uint64_t x_rows = smem_desc_sw128(xaddr, 16, 1024);     // X, K-major: 16 columns are 32 bytes
      const uint64_t x_cols = smem_desc_sw128(xaddr, CHUNK, 1024);  // X, MN-major: 16 rows are 2 KB
      const uint64_t a_rows = smem_desc_sw128(aaddr, 16, 1024);
      constexpr uint64_t BLOCK = 2 * CHUNK >> 4;                    // 128 columns, in descriptor units
      // MMAs go out four at a time (64 columns, or 64 rows of X), each descriptor the first one's plus a
      // constant: what is computed between two MMAs adds to their time.  Rows beyond the tile's
      // matrices are zero in X and B', so rounding their number up to 64 changes nothing.
      // Block b's share of A: the first time from shared memory on both sides, later with the first
      // operand where the update's epilogue left it in TMEM, 16 columns of X in 8 of 32 bits.
      auto gram_first = [&](int b) {
#pragma unroll 1
        for (int c = 2 * b; c < min(nch, 2 * b + 2); ++c) {
          const uint64_t d = x_rows + (CHUNK >> 4) * static_cast<uint64_t>(c);
#pragma unroll
          for (int j = 0; j < 4; ++j) tc_mma_lead(lead, tmem + T_A, d + 2 * j, d + 2 * j, idesc_sym, (c | j) != 0 ? 1u : 0u);
        }
      };
      auto gram_next = [&](int b) {
#pragma unroll 1
        for (int c = 2 * b; c < min(nch, 2 * b + 2); ++c) {
          const uint64_t d = x_rows + (CHUNK >> 4) * static_cast<uint64_t>(c);
          const uint32_t t = tmem + T_UPD + (c & 3) * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_tmem_a_lead(lead, tmem + T_A, t + (j >> 1) * 32 + (j & 1) * 8, d + 2 * j, idesc_sym, (c | j) != 0 ? 1u : 0u);
        }
      };
      auto update_block = [&](int b) {
        const uint64_t d = x_cols + BLOCK * b;
        const uint32_t t = tmem + T_UPD + (b & 1) * 128, idesc = 2 * b + 1 < nch ? idesc_128 : idesc_64;
#pragma unroll 1
        for (int g = 0; g < used; g += 64) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_tmem_a_lead(lead, t, tmem + T_B + g / 2 + j * 8, d + 8 * g + j * 128, idesc, (g | j) != 0 ? 1u : 0u);
        }
        tc_commit_lead(lead, upd_full + 8 * (b & 1));
      };
      uint32_t done = 0;  // parities of upd_done, a bit each
      if (p.k > 0) {
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) gram_first(b);
        tc_commit_lead(lead, a_full);
      }
#pragma unroll 1
      for (int it = 0; it < p.k; ++it) {
        wait_on(a_ready, it & 1);
        if (ok) {
#pragma unroll 1
          for (int g = 0; g < used; g += 64) {
            const uint64_t d = a_rows + (CHUNK >> 4) * static_cast<uint64_t>(g >> 6);
#pragma unroll
            for (int j = 0; j < 4; ++j) tc_mma_lead(lead, tmem + T_AA, d + 2 * j, d + 2 * j, idesc_sym, (g | j) != 0 ? 1u : 0u);
          }
          tc_commit_lead(lead, aa_full);
        }
        wait_on(b_ready, it & 1);
        if (ok) {
          update_block(0);
          if (nblk > 1) update_block(1);
        }
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          // block b is the new X.  (A barrier each for even and odd blocks: the warps may finish
          // block b + 1 before this wait, but not b + 2.)
          wait_on(upd_done + 8 * (b & 1), (done >> (b & 1)) & 1);
          done ^= 1u << (b & 1);
          if (ok && it + 1 < p.k) {
            gram_next(b);  // before the update that takes the same TMEM columns
            if (b + 1 == nblk) tc_commit_lead(lead, a_full);
          }
          if (ok && b + 2 < nblk) update_block(b + 2);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- the other warps
    const int quad = warp & 3, part4 = warp >> 2;
    const int r = quad * 32 + lane;                       // this thread's row of the tile
    const int ca0 = part4 * 32;                           // its columns of A, and of a block of the update
    const bool active = quad * 32 < used;                 // rows that hold a matrix (warp-uniform)
    const int slot = r < used ? r >> ls : -1;             // its matrix (-1: none, the row stays 0)
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t uses = 0;                                    // parity of upd_full
    uint32_t own = 0;                                     // columns ca0 + i of the row's own block, a bit each
    for (int i = 0; i < 32; ++i) own |= static_cast<uint32_t>(((ca0 + i) >> lh) == (r < used ? r >> lh : -1)) << i;
    constexpr float kGram = kHalfA / (kHalfX * kHalfX);
    // keep the row's own block; of 32 rows and more, rows are all in or all out
    auto masked = [&](float (&v)[32]) {
      if (own == 0xffffffffu) return;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = (own >> i) & 1u ? v[i] : 0.0f;
    };
    const int rows_c = 128 / C;                           // rows of A that each CTA of the cluster adds up
    const int owner = r / rows_c, in_slice = r & (rows_c - 1);
    // the place of 16 bytes of a share of A in its owner's memory: neighbouring rows side by side
    const uint32_t share_base = C == 2 ? aaddr : saddr;
    const int helper = C == 2 ? 2 * (1 - rank) : 0;       // a warp that sends the signals: for C = 2 one without rows to add
    auto share_at = [&](int from, int q) {
      return static_cast<uint32_t>((C == 2 ? 0 : from * rows_c * 32) + q * rows_c + in_slice) * 16;
    };
#pragma unroll 1
    for (int it = 0; it < p.k; ++it) {
      const uint32_t par = it & 1;
      // ------------------------------------------------------------ A
      wait_on(a_full, par);
      uint4 h[4];
      {
        float v[32];
        if (ok && (active || C > 1)) tmem_ld_32cols(t_row + T_A + ca0, v);
        if (FOLDED) {
          // The matrix's A is the sum of its column ranges' blocks: through the place of A, fp32, each row
          // its h columns in groups of four.  Of h >= 32 a warp's 32 columns are all its rows' own or none.
          const int lq = lh - 2, q0 = (ca0 & (p.slot_rows - 1)) >> 2, swz = r & min(7, (1 << lq) - 1);
          const uint32_t mine = aaddr + (r << lq) * 16;                      // this row
          const uint32_t first = aaddr + ((((r >> ls) << ls) + (r & (p.slot_rows - 1))) << lq) * 16;  // in the first block
          const uint32_t step = (p.slot_rows << lq) * 16;                    // to the next block
          const bool all = own == 0xffffffffu;
          if (ok && own != 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (all || ((own >> (4 * i)) & 1u))
                st_shared_v4(mine + ((lh >= 5 ? q0 + i : i & ((1 << lq) - 1)) ^ swz) * 16, v[4 * i], v[4 * i + 1], v[4 * i + 2],
                             v[4 * i + 3]);
            }
          }
          epi_sync();
          if (ok && own != 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 1
            for (int f = 0; f < folds; ++f) {
              const uint32_t from = first + f * step;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (all || ((own >> (4 * i)) & 1u)) {
                  const float4 t = ld_shared_v4(from + ((lh >= 5 ? q0 + i : i & ((1 << lq) - 1)) ^ swz) * 16);
                  v[4 * i] += t.x; v[4 * i + 1] += t.y; v[4 * i + 2] += t.z; v[4 * i + 3] += t.w;
                }
              }
            }
          }
          epi_sync();
          if (C == 2 && tid == 0 && ok) mbar_arrive_remote(map_to_rank(peer_free, rank ^ 1));  // the place is free
        }
        if (C > 1) {
          // Each CTA sends every owner its share of the owner's rows; the owner adds its own and the
          // others' in a fixed order, rounds once, and copies its rows of A to the others.
          if (tid == 0 && ok) {
            mbar_arrive_expect_tx(share_full, (C - 1) * rows_c * 512);
            mbar_arrive_expect_tx(rows_full, (C - 1) * rows_c * 256);
          }
          __syncwarp();
          if (C == 2 && FOLDED) wait_on(peer_free, par);
          else if (C == 2 && it > 0) wait_on(peer_free, par ^ 1);
          if (ok && owner != rank) {
            const uint32_t bar = map_to_rank(share_full, owner);
            const uint32_t to = map_to_rank(share_base + share_at(rank, ca0 >> 2), owner);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_async_v4(to + i * rows_c * 16, bar, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
          __syncwarp();
          wait_on(share_full, par);
          if (ok && owner == rank) {
            for (int c = 0; c < C; ++c) {
              if (c == rank) continue;
              const uint8_t* sh = (C == 2 ? abuf : share) + share_at(c, ca0 >> 2);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 t = *reinterpret_cast<const float4*>(sh + i * rows_c * 16);
                v[4 * i] += t.x; v[4 * i + 1] += t.y; v[4 * i + 2] += t.z; v[4 * i + 3] += t.w;
              }
            }
          }
          if (C == 2) {
            epi_sync();  // the share has been read: its place takes A
            if (warp == helper && lane == 0 && ok) mbar_arrive_remote(map_to_rank(peer_read, rank ^ 1));
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= kGram;
        masked(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = pack8h(v + 8 * i);
      }
      if (ok && (C == 1 ? active : owner == rank)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(abuf + group_at(r, (ca0 >> 3) + i)) = h[i];
      }
      fence_async_smem();
      if (C > 1) {
        epi_sync();
        if (warp == helper) {
          if (C == 2) wait_on(peer_read, par);
          if (lane < C && lane != rank && ok) {
            for (int c = 0; c < 2; ++c) {
              const uint32_t at = aaddr + c * CHUNK + rank * rows_c * 128;
              copy_to_cta(map_to_rank(at, lane), at, rows_c * 128, map_to_rank(rows_full, lane));
            }
          }
          __syncwarp();
        }
        wait_on(rows_full, par);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_ready);
      if (C > 1 && tid < C && tid != rank && ok) mbar_arrive_remote(map_to_rank(peer_got, tid));
      if (C > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const uint4*>(abuf + group_at(r, (ca0 >> 3) + i));
      }
      if (part4 == quad && slot >= 0) {  // a row of X that left fp16's range shows on the diagonal of A
        const unsigned short d =
            *reinterpret_cast<const unsigned short*>(abuf + group_at(r, r >> 3) + (r & 7) * 2);
        if ((d & 0x7C00) == 0x7C00) poison[slot] = 1;
      }
      // ------------------------------------------------------------ B' = a I + b A + c A A
      const float ca = p.coef[it][0], cb = p.coef[it][1] * (1.0f / kHalfA),
                  cc = p.coef[it][2] * (1.0f / (kHalfA * kHalfA));
      wait_on(aa_full, par);
      if (C > 1) wait_on(peer_got, par);  // the rows of A that this CTA copied have been read
      epi_sync();
      if (C == 2 && !FOLDED && tid == 0 && ok)
        mbar_arrive_remote(map_to_rank(peer_free, rank ^ 1));  // A has been read
      if (ok && active) {
        const bool out = slot >= 0 && poison[slot] != 0;
        float v[32];
        tmem_ld_32cols(t_row + T_AA + ca0, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a8[8];
          widen8(h[q], kViewF16, a8);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 x = __ffma2_rn(make_float2(cc, cc), make_float2(v[8 * q + i], v[8 * q + i + 1]),
                                        __fmul2_rn(make_float2(cb, cb), make_float2(a8[i], a8[i + 1])));
            v[8 * q + i] = x.x;
            v[8 * q + i + 1] = x.y;
          }
        }
        masked(v);
        if (part4 == quad) {  // the diagonal: entry `lane` of this thread
          float d = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (i == lane) {
              v[i] += ca;
              d = v[i];
            }
          }
          const float rounded = __half2float(__float2half_rn(d));
          row_factor[r] = fabsf(rounded) > 0x1p-10f ? __fdividef(d, rounded) : 1.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = pack8h(v + 8 * q);
        if (out) {  // nothing of this matrix may meet the others' rows
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = make_uint4(0, 0, 0, 0);
          for (int u = part4; u < groups; u += 4)
            *reinterpret_cast<uint4*>(xbuf + group_at(r, u)) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
        }
        tmem_st_16cols(t_row + T_B + part4 * 16, h);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_ready);
      epi_sync();  // the row factors
      const float g = active ? row_factor[r] : 1.0f;
      // ------------------------------------------------------------ X <- B' X
      // Warps 0..7 take the even blocks, 8..15 the odd ones, 64 columns a warp: a block's chain of
      // TMEM read, conversion, stores and fence is latency, which two blocks at a time hide.
      const int grp = warp >> 3;
#pragma unroll 1
      for (int b = grp; b < nblk; b += 2) {
        wait_on(upd_full + 8 * grp, uses);
        uses ^= 1u;
        if (ok && active) {
#pragma unroll 1
          for (int c = (part4 & 1) * 64; c < min((part4 & 1) * 64 + 64, p.width - b * 128); c += 32) {
            const uint32_t t = t_row + T_UPD + grp * 128 + c;
            float v[32];
            tmem_ld_32cols(t, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const float2 x = __fmul2_rn(make_float2(v[8 * q + i], v[8 * q + i + 1]), make_float2(g, g));
                v[8 * q + i] = x.x;
                v[8 * q + i + 1] = x.y;
              }
              h[q] = pack8h(v + 8 * q);
            }
            if (it + 1 < p.k) tmem_st_16cols(t, h);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(xbuf + group_at(r, b * 16 + (c >> 3) + q)) = h[q];
          }
          fence_async_smem();
          if (it + 1 < p.k) tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(upd_done + 8 * grp);
      }
    }
    epi_sync();  // X_k is complete

    // -------------------------------------------------------------- X_k to its view
    if (e >= 0) {
      const float coef = poison[slot_l] != 0 ? __uint_as_float(0x7FC00000u) : sg.coef;
      const bool dst_tr = sg.dst_tr != 0;
#pragma unroll 1
      for (int u = u0; u < groups; u += EPI / 16) {
        const Block b = block_of(u, dst_tr, sg.dst_ld, sg.dst_bs);
        if (whole(b, sg.dst_vec != 0)) {
          uint4 q[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = *reinterpret_cast<const uint4*>(xbuf + group_at(ig * 8 + k, u));
          if (dst_tr) transpose8(q);
          if (p.decay == 0.0f && sg.dst_type == kViewBF16) {
            uint16_t* dst = static_cast<uint16_t*>(sg.dst) + b.at;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(dst + k * b.ld) = rescale8<kViewF16, kViewBF16>(q[k], coef);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) write_eight(sg.dst, sg.dst_type, b.at + k * b.ld, q[k], coef, p.decay);
        } else {
#pragma unroll 1
          for (int k = 0; k < min(b.rows, 8); ++k) {
            float w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
              w[c] = p.decay != 0.0f && c < b.have ? load_one(sg.dst, sg.dst_type, b.at + k * b.ld + c) : 0.0f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int row = ig * 8 + (dst_tr ? c : k), col = dst_tr ? k : c;
              const float x = coef * __half2float(*reinterpret_cast<const __half*>(xbuf + group_at(row, u) + col * 2));
              if (c < b.have)
                store_one(sg.dst, sg.dst_type, b.at + k * b.ld + c, p.decay != 0.0f ? fmaf(p.decay, w[c], x) : x);
            }
          }
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  if (!ok && C > 1) {  // after a wait that ran out, let what is on its way between the CTAs arrive
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
  __syncwarp();
  sync_all();  // no CTA leaves while its shared memory may be read
  if (warp == EPI_WARPS) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

namespace {
template <int CLUSTER, bool FOLDED>
cudaError_t launch(const SkinnyParams& p, cudaStream_t s) {
  // The shared-memory limit is a property of the function on each device: set it once per device.
  static std::atomic<unsigned long long> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((attr_set.load() & bit) == 0) {
    e = cudaFuncSetAttribute(ns_skinny_kernel<CLUSTER, FOLDED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  return cudaLaunchKernelEx(&cfg, ns_skinny_kernel<CLUSTER, FOLDED>, p);
}
}  // namespace

cudaError_t launch_ns_skinny(const SkinnyParams& p, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  if (p.cluster == 1) return p.folds > 1 ? launch<1, true>(p, s) : launch<1, false>(p, s);
  if (p.cluster == 2) return p.folds > 1 ? launch<2, true>(p, s) : launch<2, false>(p, s);
  return p.folds > 1 ? launch<4, true>(p, s) : launch<4, false>(p, s);
}

}  // namespace muon
