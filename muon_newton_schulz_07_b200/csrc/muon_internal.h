// Internal launch interfaces between the C ABI (muon_api.cu) and the kernels.
// Nothing here is exported from libmuon.so.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

namespace muon {

// Device status codes (written to the workspace status word; match muon_status_t).
constexpr unsigned int kDevTimeout = 5;
constexpr unsigned int kDevFault = 6;

// Every workspace buffer is padded to multiples of this many rows/columns.
constexpr int kPad = 256;

// ------------------------------------------------------------------ elementwise
// Elementwise kernels work on X-coordinate tiles of 64 x 128 (X is the oriented
// matrix, min(rows,cols) x max(rows,cols), padded to multiples of kPad).
constexpr int kEwTileR = 64;
constexpr int kEwTileC = 128;
constexpr int kEwThreads = 256;
constexpr int kEwMinCtasPerSm = 4;  // resident momentum/norm CTAs per SM the register budget allows (bf16 sources)
constexpr int kEwMatsPerLaunch = 192;

enum Dtype : int { kBF16 = 0, kF32 = 1 };

struct EwMat {
  const void* src;   // G (step) or X (orthogonalize), rows x cols, caller's layout
  void* mom;         // M, updated in place; nullptr: no momentum (U = src)
  void* x;           // workspace X buffer of this matrix, mp x np, row stride np
  int rows, cols;    // caller's shape
  int mp, np;        // padded oriented shape
  int trans;         // rows > cols: X = U^T
  int tile_begin;    // first tile of this matrix in the launch's tile list
  int tiles_c;       // X tiles along np
  int ntiles;        // X tiles of the padded matrix (mp/64 * np/128)
  int scal_idx;      // slot of this matrix in the scalar / counter tables
  int caller_idx;    // position in the caller's matrix list
  int part_begin;    // first CTA of this matrix in the launch (= tile_begin: one CTA per tile)
  int nparts;        // CTAs of this matrix, each with one partial-sum slot per warp (= ntiles)
};

// The momentum/norm launch: one CTA per tile, matrix j's CTAs part_begin .. part_begin + nparts - 1.
struct EwParams {
  EwMat mat[kEwMatsPerLaunch];
  int nmat;
  int total_tiles;
  int grid;                // CTAs of the launch: the sum of the matrices' nparts
  float beta;
  float eps;
  int nesterov;
  int vec_ok;              // every row of every matrix starts 16-byte aligned
  float* partials;         // per (CTA, warp) sums of squares
  float* scal;             // per matrix: {||U||_F, 1/(||U||_F + eps)}
  float* norms;            // ||U||_F per matrix, caller order
  unsigned int* status;    // device status word (a bounded wait that ran out)
};

struct WrMat {
  void* w;           // W (updated in place) or O (written)
  const void* x;     // final X of this matrix, mp x np, row stride np
  int rows, cols, mp, np, trans;
  int tile_begin;    // first CTA of this matrix
  int tiles_c;       // tiles along the real n
  int scal_idx;
  float shape_scale; // sqrt(max(1, rows/cols))
};

struct WrParams {
  WrMat mat[kEwMatsPerLaunch];
  int nmat;
  int total_ctas;
  float lr, wd;
  int store_only;   // 1: O = X (orthogonalize); 0: W = (1 - lr*wd) W - lr*s*X
  int use_alpha;    // 1: X still unnormalised (k = 0), multiply by 1/(||U||+eps)
  int vec_ok;
  const float* scal;
};

cudaError_t launch_momentum_norm(const EwParams& p, Dtype io, Dtype xt, cudaStream_t s);
cudaError_t launch_param_write(const WrParams& p, Dtype io, Dtype xt, cudaStream_t s);

// ------------------------------------------------------------------ tcgen05 GEMMs
constexpr int kTcBM = 128;
constexpr int kTcBN = 256;
constexpr int kTcBK = 64;
constexpr int kTcMaxGroups = 6;
constexpr int kTcEpiWarps = 8;     // two per TMEM lane quadrant, each on half of the tile's columns
constexpr int kTcThreads = 64 + 32 * kTcEpiWarps;  // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue

enum TcKind : int { kGram = 0, kPoly = 1, kUpdate = 2 };

struct alignas(64) TcGroup {
  CUtensorMap tm_a;     // operand A source, row view: box 64 (k) x 128 (rows) x 1, 128B swizzle
  CUtensorMap tm_at;    // the same buffer, chunked view for MN-major reads: box 64 x 64 (k) x 2 chunks x 1
  CUtensorMap tm_b;     // operand B source, row view
  CUtensorMap tm_bt;    // operand B source, chunked view
  CUtensorMap tm_out;   // output, store view: box 32 x 32 x 1, 64B swizzle
  CUtensorMap tm_aux;   // Poly's epilogue input A, store view (box 32 x 32, 64B swizzle), loaded by TMA
  void* out;            // [cnt][rows][ld] bf16
  int cnt, mp, np;
  int tiles_per_mat;
  int tile_begin;
  int kblocks;
  int scal_base;
  int tdim;             // Gram/Poly: mp/256 (triangle side); Update: np/256
  int out_ld;
  int m_real;           // real (unpadded) rows: Poly adds its diagonal term only there
  int n_real;           // real (unpadded) columns of X
  int pad_;
};

// Largest number of matrices whose parameter write can be fused into the last
// Update launch (their pointers travel in the kernel parameters).
constexpr int kTcMaxFused = 1024;
// Words of NsParams::round for the launches of one call: one, or one per stage of up to 64 iterations.
constexpr int kNsRounds = 2 * 3 * 64;

struct TcParams {
  TcGroup g[kTcMaxGroups];
  int ngroups;
  int total_tiles;
  int kind;
  int wide;              // Update with 256 x 512 pair tiles (every group's np a multiple of 512)
  int half;              // operands are fp16 (MUON_MODE_HALF), not bf16
  int use_scal;          // first iteration: fold the normalisation in
  float c_acc, c_aux;    // out = s * (c_acc * acc + c_aux * aux) (+ c_diag on the real diagonal)
  float c_diag;
  const float* scal;
  unsigned int* status;
  unsigned long long timeout_ns;
  // Fused parameter write (last Update only).  Instead of storing X_k, the epilogue
  // writes W = w_decay * W + wcoef[slot] * X_k into the caller's bf16 matrix of each
  // slot (the scalar-table index), transposed back when wtrans[slot] is set.  With
  // w_decay == 0 it stores wcoef * X_k without reading W (the orthogonaliser output).
  int fuse_write;
  float w_decay;
  void* wptr[kTcMaxFused];
  float wcoef[kTcMaxFused];
  int wld[kTcMaxFused];  // elements between rows of the matrix as it is stored
  unsigned char wtrans[kTcMaxFused];
};

size_t tc_smem_bytes();
cudaError_t launch_tc_gemm(const TcParams& p, int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ every iteration in one launch
// One persistent launch runs all k x {Gram, Poly, Update} stages of every matrix of up to
// kTcMaxGroups shape groups.  Tiles are listed stage after stage (iteration-major, then
// Gram / Poly / Update, then group, matrix and tile) and dealt round-robin to the CTA pairs that run;
// before loading a tile, a pair waits (bounded) until the stage the tile reads is complete for
// its matrix: every epilogue warp that finishes a tile adds 1 to a per (stage, matrix)
// completion counter in the workspace.
struct alignas(64) NsGroup {
  CUtensorMap x_row[2], x_chk[2], x_st[2];  // X0 / X1: row, chunked and store views
  CUtensorMap a_row, a_chk, a_st;           // A
  CUtensorMap b_row, b_chk, b_st;           // B'
  int cnt, mp, np;
  int m_real, n_real;
  int scal_base;        // first slot of the group in the scalar / counter tables
  int tdim;             // mp / 256
  int pad_[7];
};

struct NsParams {
  NsGroup g[kTcMaxGroups];
  int ngroups;
  int k;                 // iterations, >= 1
  int nslots;            // matrices of the launch (the counter table's row length)
  int tiles_iter;        // tiles of an iteration other than the last
  int total_tiles;
  int t_begin, t_end;    // the tiles this launch runs: [0, total_tiles), or one stage of them
  int upd_tw[2];         // Update tile width (128, 256 or 512) of [other, last] iterations
  int sym_tw;            // Gram and Poly tile width (128 or 256)
  int fuse_write;        // the last Update writes the parameters (see TcParams)
  // first tile of (stage, group) within an iteration, [other, last][stage][group];
  // [..][stage][ngroups] is the end of the stage
  int begin[2][3][kTcMaxGroups + 1];
  int half;              // operands are fp16 (MUON_MODE_HALF), not bf16; X0 is normalised
  float gram;            // A = gram * (the Gram product)
  float coef[64][3];     // B' = coef[0] I + coef[1] A + coef[2] A A, by iteration
  const float* scal;
  unsigned int* status;
  unsigned int* deps;    // [3 k][nslots] completion counters, zero before the launch
  unsigned int* round;   // two words: pairs that have come, and how many the tiles are dealt to; zero before the launch
  unsigned long long timeout_ns;
  float w_decay;
  void* wptr[kTcMaxFused];
  float wcoef[kTcMaxFused];
  int wld[kTcMaxFused];
  unsigned char wtrans[kTcMaxFused];
};

// Tiles per matrix of a symmetric stage (Gram, Poly) over the T x T blocks of the upper triangle: one
// per block of 256 x 256, or two of 256 x 128.
__host__ __device__ inline int sym_tiles(int T, int tw) { return T * (T + 1) / 2 * (256 / tw); }

size_t fused_smem_bytes();
cudaError_t launch_ns_fused(const NsParams& p, int num_sms, cudaStream_t s);
// Host-side consistency check of a single-launch tile list (number of problems found).
long long check_fused_tiles(const NsParams& p);
// Host-side consistency check of one momentum/norm launch's tables (number of problems found).
long long check_front_tables(const EwParams& p);

// ------------------------------------------------------------------ small matrices, all iterations in one kernel
// Every matrix of the set fits one 256 x 256 tile (max(rows, cols) <= 256; the workspace
// pads it to 256 x 256).  One CTA pair runs all k Newton-Schulz iterations of a matrix.
constexpr int kSmallTile = 256;

struct alignas(64) SmGroup {
  CUtensorMap tm_row;   // X0, row view (box 64 x 128 x 1): this CTA's 128 rows, one 64-wide k chunk
  CUtensorMap tm_col;   // X0, chunked view (box 64 x 64 x 2 x 1): 64 rows of this CTA's 128 columns
  void* out;            // [cnt][256][256] bf16: X_k
  int mat_begin;        // first matrix of the group in the launch's numbering
  int cnt;
  int scal_base;
  int m_real;           // real rows of the Gram matrix (the polynomial's a I stops there)
};

struct SmallParams {
  SmGroup g[kTcMaxGroups];
  int ngroups;
  int total;            // matrices in the launch
  int k;                // Newton-Schulz iterations, >= 1
  int half;             // operands are fp16 (MUON_MODE_HALF), not bf16; X0 is normalised
  float gram;           // A = gram * (the Gram product)
  float coef[64][3];    // B' = coef[0] I + coef[1] A + coef[2] A A, by iteration
  const float* scal;    // per matrix {||U||, 1/(||U||+eps)}
  unsigned int* status;
  unsigned long long timeout_ns;
};

size_t small_smem_bytes();
cudaError_t launch_ns_small(const SmallParams& p, int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ fp16 operands (MUON_MODE_HALF)
// The iteration's operands are stored in fp16 (11 significant bits, three more than bf16) times
// powers of two, folded into the epilogues' coefficients, that keep what matters in fp16's normal
// range: after Frobenius normalisation a typical entry of X is 1/sqrt(mn) and of A 1/(m sqrt(n)),
// down to 2^-20, while no entry of X or A exceeds the largest singular value (squared).  Singular
// values up to 4 fit.
constexpr float kHalfX = 4096.0f;  // stored X  = 2^12 X
constexpr float kHalfA = 4096.0f;  // stored A  = 2^12 A
constexpr float kHalfB = 1.0f;     // B' as it is: its diagonal is of the order of a

// Storage types of a view (MUON_BF16, MUON_FP32, MUON_FP16).
enum ViewType : int { kViewBF16 = 0, kViewF32 = 1, kViewF16 = 2 };

// `count` equal matrices of a call: how their elements are stored on the source and destination
// side, and their place in the launch's and the handle's tables.  A side is stored as rows of
// contiguous elements, `ld` apart; `tr` says that those rows are the columns of the oriented X
// (min x max), so that the tile is transposed on its way.  Matrix e starts at e * bs.
struct ViewSeg {
  const void* src;
  void* dst;
  long long src_ld, src_bs, dst_ld, dst_bs;
  int src_type, dst_type;
  int src_tr, dst_tr;
  int src_vec, dst_vec;  // every stored row starts 16-byte aligned
  void* x;               // workspace X of the first matrix, [count][mp][np] fp16
  int m, n, mp, np;
  int count;
  int mat_begin;         // first matrix of the launch's numbering
  int tile_begin;        // first tile (CTA) of the launch
  int tiles_c, tiles;    // tiles along a row of X, tiles of one matrix
  int part_begin;        // first partial sum; `parts` for each matrix
  int parts;
  int caller_idx;        // first matrix's place in the handle's list
  float coef;            // the write: dst = decay * dst + coef * X (X as stored, 2^12 X)
};

constexpr int kViewSegs = 96;
struct ViewParams {
  ViewSeg seg[kViewSegs];
  int nseg;
  int total;             // CTAs
  int normalised;        // the source is 2^12 X already: no norm is taken
  float eps;
  float decay;           // 0: dst is not read
  double* partials;
  float* norms;          // each matrix's last CTA of the sums puts its norm there ...
  float* factors;        // ... and here what its elements are multiplied by
  unsigned int* arrivals;  // CTAs of each matrix that have left their part, zero before the call's first launch
};

// The norms of the sources, from one partial sum of squares per CTA (a 64 x 128 tile).
cudaError_t launch_view_sumsq(const ViewParams& p, cudaStream_t s);
// X0 = 2^12 src / (||src|| + eps), oriented and zero-padded.
cudaError_t launch_view_orient(const ViewParams& p, cudaStream_t s);
// dst = decay * dst + coef * X.
cudaError_t launch_view_write(const ViewParams& p, cudaStream_t s);

// Matrices of few rows: every iteration on chip, one cluster per 128-row tile (k_ns_skinny.cu).
constexpr int kSkinnyRows = 128;       // most rows (of the oriented matrix)
constexpr int kSkinnyColsOne = 768;    // most columns of one CTA, or of each of two
constexpr int kSkinnyColsPart = 512;   // most columns of each CTA of a larger cluster
constexpr int kSkinnyCluster = 8;      // most CTAs of a cluster
inline int skinny_block(int m) {       // rows of a block
  int h = 8;
  while (h < m) h *= 2;
  return h;
}
// Whether matrices of m rows and n columns (m <= n) fit.
inline bool skinny_fits(long long m, long long n) {
  return m <= kSkinnyRows && n <= static_cast<long long>(kSkinnyRows / skinny_block(static_cast<int>(m))) * kSkinnyCluster * kSkinnyColsPart;
}
constexpr int kSkinnySegs = 64;
constexpr int kMaxSteps = 64;

struct SkinnyParams {
  ViewSeg seg[kSkinnySegs];  // mat_begin numbers the launch's matrices; the workspace is not used
  int nseg;
  int total;                 // matrices
  int m, n;
  int slot_rows;             // rows of a block of the tile: a power of two >= m, 8 at least
  int folds;                 // blocks below each other that hold a matrix, each a range of its columns
  int slots;                 // matrices in a tile; slots * folds * slot_rows <= 128
  int cluster;               // CTAs of a tile
  int width;                 // columns of a block that each CTA holds, a multiple of 64
  int normalised;            // the source is 2^12 X already: no norm is taken
  int k;
  float coef[kMaxSteps][3];  // (a, b, c) of each iteration
  float eps;
  float decay;
  float* norms;
  unsigned int* status;
  unsigned long long timeout_ns;
};
cudaError_t launch_ns_skinny(const SkinnyParams& p, cudaStream_t s);

// ------------------------------------------------------------------ 8-bit state
constexpr int kStateBlock = 128;   // columns that share a scale
constexpr int kStateUnits = 64;    // (row, block) units of one CTA
enum StateFormat : int { kStateInt8 = 0, kStateE4M3 = 1, kStateDense = 2 };

struct StateSeg {
  const void* in;        // quantise: X; momentum: G
  void* out;             // dequantise: X; momentum: U
  void* codes;           // int8 / e4m3 codes, or the dense momentum
  float* scales;
  long long in_ld, in_bs, out_ld, out_bs;
  int in_type, out_type;
  int vec;               // every row of every side is a multiple of 4 long and aligned to 4 values
  int linear;            // and whole blocks, the matrices and their rows back to back on every side
  int rows, cols, blocks;
  int count;
  int mat_begin;         // first matrix's number in the call (the random bits' key)
  int unit_ctas;         // CTAs of one matrix
  int cta_begin;
  int caller_idx;        // momentum: first matrix's place in the handle's list
};
// Parameters are copied at each launch: 128 segments cost the host 1.1 us more than 32, which bounds a call on
// one small matrix (2.2 us); beyond 32 states another launch is 2.2 us of many.
constexpr int kStateSegs = 32;
struct StateParams {
  StateSeg seg[kStateSegs];
  int nseg;
  int total;             // CTAs
  int linear;            // every segment is: whole blocks, every side contiguous and aligned
  int stochastic;
  unsigned int seed;
  float beta;
  int nesterov;
  double* partials;      // momentum: one sum of squares per CTA
  float eps;             // momentum
  float* norms;          // momentum: each matrix's last CTA puts its norm there ...
  float* factors;        // ... and here what kPassStep multiplies u by
  unsigned int* arrivals;  // CTAs of each matrix that have left their part, zero before the call's first launch
};
cudaError_t launch_state_quantize(const StateParams& p, StateFormat f, cudaStream_t s);
cudaError_t launch_state_dequantize(const StateParams& p, StateFormat f, cudaStream_t s);
// What a momentum launch does: write u (in the type of G) and m1, with the norms; the norms alone,
// leaving everything as it was; or, knowing the norms, write 2^12 u / (norm + eps) in fp16 and m1.  A step
// runs the second and the third: u is then rounded once, after it has been normalised, where a pass that
// wrote it first would have to keep it in 32 bits.
enum StatePass : int { kPassMomentum = 0, kPassNorm = 1, kPassStep = 2 };
// G and a dense momentum have one type, bf16 or fp32.
cudaError_t launch_state_momentum(const StateParams& p, StateFormat f, StatePass pass, cudaStream_t s);

// ------------------------------------------------------------------ fp32 reference GEMMs
struct SgParams {
  const float* a; const float* b; float* c; const float* aux;
  int M, N, K;
  int lda, ldb, ldc;
  long long sa, sb, sc;   // batch strides (elements)
  int cnt;
  int b_trans;            // 1: second operand is b^T (b row-major N x K)
  float c_acc, c_aux;
  const float* scal; int scal_base; int scal_mode;  // 0: none, 1: alpha^2, 2: alpha
  float c_diag; int diag_n;  // add c_diag to C[i][i] for i < diag_n
};
cudaError_t launch_sgemm(const SgParams& p, cudaStream_t s);

// ------------------------------------------------------------------ self-test
cudaError_t launch_timeout_selftest(unsigned int* status, unsigned long long timeout_ns, cudaStream_t s);

}  // namespace muon
