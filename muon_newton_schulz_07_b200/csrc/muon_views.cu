// C ABI of libmuon.so, second part (declared in include/muon.h): the orthogonaliser on views, the
// 8-bit state, and the steps of MUON_MODE_HALF handles.  All arithmetic runs in the kernels; this file
// only checks, plans and enqueues.
//
// A HALF call enqueues, on the caller's stream and without any host sync:
//   state_momentum_kernel   (steps only, twice) the norms; then m1 written back and the normalised u as
//                           X0 itself, or in the caller's layout where it has to be transposed or padded
//   view_sumsq_kernel       (orthogonaliser only) the norms
//   view_orient_kernel      X0, oriented and padded, fp16
//   k x { Gram, Poly, Update }   tcgen05 kernels, the last Update writes the result when it can
//   view_write_kernel       otherwise
//   ns_skinny_kernel        instead of the last four, for shape groups of at most 128 rows
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>
#include <vector>

#include "muon_ctx.h"

using namespace muon;

namespace {

// One side of a view: rows of `len` contiguous elements, `ld` apart; by_cols: those are the
// matrix's columns.
struct Side {
  char* data;
  int type;
  long long ld, bs;
  bool by_cols;
  bool vec;   // every stored row starts 16-byte aligned
};

struct Item {   // equal matrices of the call, consecutive in the handle's list
  int first, count;
  Side src, dst;
  int part_begin, parts;  // of the first matrix; partial sums of each matrix
  bool is_x0;             // the source is X0 already
};

size_t type_bytes(int type) { return type == kViewF32 ? 4 : 2; }

bool count_ok(int64_t v) { return v >= 1 && v <= MUON_MAX_MATRICES; }

muon_status_t make_side(const muon_view_t& v, int64_t rows, int64_t cols, bool output, Side* s) {
  if (v.data == nullptr || !count_ok(v.count)) return MUON_ERR_INVALID_ARG;
  if (v.dtype != MUON_BF16 && v.dtype != MUON_FP32 && v.dtype != MUON_FP16) return MUON_ERR_INVALID_ARG;
  if (v.batch_stride < 0 || v.row_stride < 0 || v.col_stride < 0) return MUON_ERR_INVALID_ARG;
  s->data = static_cast<char*>(v.data);
  s->type = static_cast<int>(v.dtype);
  int64_t len, nrow;
  if (cols == 1 && (v.row_stride == 1 || rows == 1)) {
    s->by_cols = true;
    s->ld = rows;  // one stored row
  } else if (v.col_stride == 1 || cols == 1) {
    s->by_cols = false;
    s->ld = rows == 1 ? cols : v.row_stride;
  } else if (v.row_stride == 1 || rows == 1) {
    s->by_cols = true;
    s->ld = v.col_stride;
  } else {
    return MUON_ERR_UNSUPPORTED;
  }
  len = s->by_cols ? rows : cols;
  nrow = s->by_cols ? cols : rows;
  s->bs = v.count == 1 ? 0 : v.batch_stride;
  const size_t es = type_bytes(s->type);
  if ((reinterpret_cast<uintptr_t>(v.data) % es) != 0) return MUON_ERR_INVALID_ARG;
  if (output) {
    // distinct elements at distinct addresses: matrix after matrix, or row after row of all matrices
    const bool inner = nrow == 1 || s->ld >= len;
    const bool outer = v.count == 1 || s->bs >= (nrow - 1) * s->ld + len;
    const bool inner2 = v.count == 1 || s->bs >= len;
    const bool outer2 = nrow == 1 || s->ld >= (v.count - 1) * s->bs + len;
    if (!(inner && outer) && !(inner2 && outer2)) return MUON_ERR_INVALID_ARG;
  }
  s->vec = (reinterpret_cast<uintptr_t>(v.data) & 15u) == 0 && (nrow == 1 || s->ld * es % 16 == 0) &&
           (v.count == 1 || s->bs * es % 16 == 0);
  return MUON_OK;
}

muon_view_t contiguous(const void* data, const muon_shape_t& sh, muon_dtype_t dtype) {
  return muon_view_t{const_cast<void*>(data), 1, sh.rows * sh.cols, sh.cols, 1, dtype};
}

// The handle's matrices covered by n views' counts: the first matrix of each, which must add up and
// be of one shape each.
muon_status_t cover(const muon_ctx* h, const muon_view_t* v, int n, std::vector<int>* first) {
  int at = 0;
  first->clear();
  for (int j = 0; j < n; ++j) {
    if (!count_ok(v[j].count) || at + v[j].count > h->n) return MUON_ERR_INVALID_ARG;
    for (int e = 1; e < v[j].count; ++e)
      if (h->shapes[at + e].rows != h->shapes[at].rows || h->shapes[at + e].cols != h->shapes[at].cols)
        return MUON_ERR_INVALID_ARG;
    first->push_back(at);
    at += static_cast<int>(v[j].count);
  }
  return at == h->n ? MUON_OK : MUON_ERR_INVALID_ARG;
}

// Outputs at one address, or at another matrix's input, would race: the same tensor twice in a list,
// or a list given back in another order.  (Views that overlap in part are the caller's to avoid.)
bool distinct(std::vector<const void*>& at) {
  std::sort(at.begin(), at.end());
  return std::adjacent_find(at.begin(), at.end()) == at.end();
}
bool apart(const std::vector<const void*>& in, const std::vector<const void*>& out) {
  if (out.size() == 1) return true;
  std::vector<std::pair<const void*, size_t>> sorted;
  for (size_t j = 0; j < out.size(); ++j) sorted.emplace_back(out[j], j);
  std::sort(sorted.begin(), sorted.end());
  for (size_t j = 1; j < sorted.size(); ++j)
    if (sorted[j].first == sorted[j - 1].first) return false;
  for (size_t j = 0; j < in.size(); ++j) {
    const auto it = std::lower_bound(sorted.begin(), sorted.end(), std::make_pair(in[j], size_t{0}));
    if (it != sorted.end() && it->first == in[j] && it->second != j) return false;
  }
  return true;
}
bool states_distinct(const muon_state_t* S, int n) {
  if (n == 1) return true;
  std::vector<const void*> at;
  for (int j = 0; j < n; ++j) {
    at.push_back(S[j].codes);
    at.push_back(S[j].scales);
  }
  return distinct(at);
}

// (a, b, c) of iteration t.
const float* coef_of(const muon_ctx* h, const muon_hparams_t* hp, int t, float (&own)[3]) {
  if (!h->coef.empty()) return &h->coef[3 * static_cast<size_t>(t)];
  own[0] = hp->a;
  own[1] = hp->b;
  own[2] = hp->c;
  return own;
}
bool steps_ok(const muon_ctx* h, const muon_hparams_t* hp) {
  return h->coef.empty() || static_cast<size_t>(hp->ns_steps) * 3 <= h->coef.size();
}

// The factors of A and B' in a kernel that runs every iteration.
template <typename Params>
void fill_iterations(const muon_ctx* h, const muon_hparams_t* hp, Params* p) {
  p->gram = kHalfA / (kHalfX * kHalfX);
  for (int t = 0; t < hp->ns_steps; ++t) {
    float own[3];
    const float* abc = coef_of(h, hp, t, own);
    p->coef[t][0] = abc[0];
    p->coef[t][1] = abc[1] * (1.0f / kHalfA);
    p->coef[t][2] = abc[2] * (1.0f / (kHalfA * kHalfA));
  }
}

const GroupPlan& group_of(const muon_ctx* h, int mat) { return h->plan.groups[h->plan.mat_group[mat]]; }
bool tall(const muon_ctx* h, int mat) { return h->shapes[mat].rows > h->shapes[mat].cols; }

bool small_tiles(const muon_ctx* h, int k);

// A view segment without its place in a launch.  `store`: the result is O itself, else the step
// of the parameters.
void fill_seg(const muon_ctx* h, const Item& it, bool store, float lr, ViewSeg* s) {
  std::memset(s, 0, sizeof(*s));
  const GroupPlan& gp = group_of(h, it.first);
  const bool t = tall(h, it.first);
  s->src = it.src.data;
  s->src_ld = it.src.ld;
  s->src_bs = it.src.bs;
  s->src_type = it.src.type;
  s->src_tr = t != it.src.by_cols;
  s->src_vec = it.src.vec;
  s->dst = it.dst.data;
  s->dst_ld = it.dst.ld;
  s->dst_bs = it.dst.bs;
  s->dst_type = it.dst.type;
  s->dst_tr = t != it.dst.by_cols;
  s->dst_vec = it.dst.vec;
  s->m = gp.m;
  s->n = gp.n;
  s->mp = gp.mp;
  s->np = gp.np;
  s->count = it.count;
  s->caller_idx = it.first;
  s->part_begin = it.part_begin;
  s->parts = it.parts;
  const float r = static_cast<float>(h->shapes[it.first].rows), c = static_cast<float>(h->shapes[it.first].cols);
  s->coef = (store ? 1.0f : -lr * std::sqrt(std::max(1.0f, r / c))) / kHalfX;
}

enum ViewPass { kSumsq, kOrient, kWrite };

// One pass over the views of the groups that go through the workspace, as few launches as fit.
cudaError_t view_pass(muon_ctx* h, const std::vector<Item>& items, ViewPass pass, const muon_hparams_t* hp, bool store,
                      bool normalised, int fin, cudaStream_t st) {
  ViewParams& p = h->vw;
  size_t i = 0;
  while (i < items.size()) {
    p.nseg = 0;
    p.total = 0;
    p.normalised = normalised ? 1 : 0;
    p.eps = hp->eps;
    p.decay = store ? 0.0f : 1.0f - hp->lr * hp->weight_decay;
    p.partials = reinterpret_cast<double*>(h->d_partials);
    p.norms = h->d_norms;
    p.factors = h->d_scal;
    p.arrivals = reinterpret_cast<unsigned int*>(h->ws + h->plan.off_arrivals);
    for (; i < items.size() && p.nseg < kViewSegs; ++i) {
      const Item& it = items[i];
      const GroupPlan& gp = group_of(h, it.first);
      if (gp.skinny || (pass == kOrient && it.is_x0)) continue;
      const int rows = pass == kOrient ? gp.mp : gp.m, cols = pass == kOrient ? gp.np : gp.n;
      const int tiles_c = (cols + kEwTileC - 1) / kEwTileC;
      const long long tiles = static_cast<long long>((rows + kEwTileR - 1) / kEwTileR) * tiles_c;
      if (p.total + tiles * it.count > 0x7fffffffll) {
        if (p.nseg == 0) return cudaErrorInvalidConfiguration;
        break;
      }
      ViewSeg& s = p.seg[p.nseg++];
      fill_seg(h, it, store, hp->lr, &s);
      s.x = h->ws + gp.off_x[pass == kWrite ? fin : 0] +
            static_cast<size_t>(h->plan.mat_slot[it.first]) * gp.mp * gp.np * 2;
      s.tile_begin = p.total;
      s.tiles_c = tiles_c;
      s.tiles = static_cast<int>(tiles);
      p.total += static_cast<int>(tiles * it.count);
    }
    if (p.nseg == 0) break;
    const cudaError_t e = pass == kSumsq ? launch_view_sumsq(p, st)
                          : pass == kOrient ? launch_view_orient(p, st)
                                            : launch_view_write(p, st);
    if (e != cudaSuccess) return e;
    trace(h, pass == kWrite ? MUON_KERNEL_WRITE : MUON_KERNEL_MOMENTUM_NORM, st);
  }
  return cudaSuccess;
}

// The last Update can write the result itself when every destination of the workspace groups is
// bf16 with aligned rows and every real dimension is a multiple of 32.
bool result_fusable(const muon_ctx* h, const std::vector<Item>& items, int k) {
  if (k < 1 || h->n > kTcMaxFused || small_tiles(h, k)) return false;
  for (const Item& it : items) {
    const GroupPlan& gp = group_of(h, it.first);
    if (gp.skinny) continue;
    if (it.dst.type != kViewBF16 || !it.dst.vec || gp.m % 32 != 0 || gp.n % 32 != 0 || it.dst.ld > 0x7fffffffll)
      return false;
  }
  return true;
}

std::vector<const GroupPlan*> tiled_groups(const muon_ctx* h) {
  std::vector<const GroupPlan*> v;
  for (const GroupPlan& gp : h->plan.groups)
    if (!gp.skinny) v.push_back(&gp);
  return v;
}

// Whether every group that goes through the workspace is one 256 x 256 tile a matrix, which the
// small-matrix kernel iterates on chip.
bool small_tiles(const muon_ctx* h, int k) {
  const std::vector<const GroupPlan*> groups = tiled_groups(h);
  if (k < 1 || groups.empty() || groups.size() > static_cast<size_t>(kTcMaxGroups)) return false;
  for (const GroupPlan* gp : groups)
    if (gp->mp != kSmallTile || gp->np != kSmallTile) return false;
  return true;
}

cudaError_t enqueue_small(muon_ctx* h, const muon_hparams_t* hp, cudaStream_t st) {
  NvtxRange range("muon: Newton-Schulz, all iterations (small matrices)");
  SmallParams& sp = h->sm;
  std::memset(&sp, 0, sizeof(sp));
  small_groups(h, tiled_groups(h), hp->ns_steps & 1, &sp);
  sp.k = hp->ns_steps;
  sp.half = 1;
  fill_iterations(h, hp, &sp);
  sp.scal = h->d_scal;
  sp.status = h->d_status;
  sp.timeout_ns = kTimeoutNs;
  const cudaError_t e = launch_ns_small(sp, h->num_sms, st);
  if (e == cudaSuccess) trace(h, MUON_KERNEL_NS_SMALL, st);
  return e;
}

// 256 x 256 tiles of an Update over every group, and the CTA pairs that share them.
long long update_tiles(const std::vector<const GroupPlan*>& groups) {
  long long tiles = 0;
  for (const GroupPlan* gp : groups) tiles += static_cast<long long>(gp->cnt) * (gp->mp / 256) * (gp->np / 256);
  return tiles;
}

// Whether the k iterations of the groups that go through the workspace run as one launch.  AUTO
// does so up to eight Update tiles a pair: there the launch boundaries (a ramp, a tail and a gap each)
// cost more than the single launch's waits on completion counters.  Measured, five iterations,
// one launch against one per stage, the orthogonaliser on bf16 by itself: 4 x 768 x 768 (half a tile a pair) 158 and 218 us,
// 16 x 1024 x 1024 (3.5) 381 and 497, 48 x 768 x 768 (5.8) 540 and 653, 16 x 1536 x 1536 (7.8) 1231 and 1326.  Beyond,
// where the power cap sets the pace, it depends on the set and on what else the call does: 40 x 1024 x 1024 (8.6) 1069
// and 1192, 24 x 1536 x 1536 (12) 1903 and 1895, 12 x 1536 x 6144 (23) 2820 and 2928; steps on an 8-bit state, 24 x 1536 x 1536
// 1998 and 1956, 12 x 1536 x 6144 3194 and 3092.
bool single_launch(const muon_ctx* h, int k) {
  if (k < 1 || !half_fused_possible(h)) return false;
  if (h->schedule != MUON_SCHEDULE_AUTO) return h->schedule != MUON_SCHEDULE_STAGED;
  return update_tiles(tiled_groups(h)) <= 8ll * (h->num_sms / 2);
}

// 256 x 512 Update tiles only when there are more 256-wide ones than CTA pairs: below that a wide
// tile leaves pairs idle and takes twice as long.
bool wide_pays(const muon_ctx* h, const std::vector<const GroupPlan*>& groups) {
  return update_tiles(groups) > h->num_sms / 2;
}

// Where the last Update writes matrix e of an item: destination, factor and layout by slot.
template <typename Params>
void fill_results(const muon_ctx* h, const std::vector<Item>& items, const muon_hparams_t* hp, bool store, Params* p) {
  p->fuse_write = 1;
  p->w_decay = store ? 0.0f : 1.0f - hp->lr * hp->weight_decay;
  for (const Item& it : items) {
    if (group_of(h, it.first).skinny) continue;
    ViewSeg s;
    fill_seg(h, it, store, hp->lr, &s);
    for (int e = 0; e < it.count; ++e) {
      const int slot = h->plan.scal_idx[it.first + e];
      p->wptr[slot] = it.dst.data + static_cast<size_t>(e) * it.dst.bs * 2;
      p->wcoef[slot] = s.coef;
      p->wld[slot] = static_cast<int>(it.dst.ld);
      p->wtrans[slot] = static_cast<unsigned char>(s.dst_tr);
    }
  }
}

// All iterations in one launch (or, for measurements, its tiles with a launch per stage).
cudaError_t enqueue_single(muon_ctx* h, const std::vector<Item>& items, const muon_hparams_t* hp, bool store, bool fuse,
                           cudaStream_t st) {
  NvtxRange range("muon: Newton-Schulz, every iteration in one launch");
  const std::vector<const GroupPlan*> groups = tiled_groups(h);
  const int k = hp->ns_steps;
  cudaError_t e;
  NsParams& q = h->ns;
  fused_tables(groups, h->n, k, fuse, wide_pays(h, groups), h->num_sms / 2, &q);
  fused_maps(groups, &q);
  q.half = 1;
  fill_iterations(h, hp, &q);
  q.scal = h->d_scal;
  q.status = h->d_status;
  q.deps = reinterpret_cast<unsigned int*>(h->ws + h->plan.off_deps);  // zero, as the rounds: clear_counters
  unsigned int* rounds = reinterpret_cast<unsigned int*>(h->ws + h->plan.off_rounds);
  q.round = rounds;
  q.timeout_ns = kTimeoutNs;
  if (fuse) fill_results(h, items, hp, store, &q);
  if (h->schedule != MUON_SCHEDULE_SPLIT) {
    q.t_begin = 0;
    q.t_end = q.total_tiles;
    e = launch_ns_fused(q, h->num_sms, st);
    if (e == cudaSuccess) trace(h, MUON_KERNEL_NS_FUSED, st);
    return e;
  }
  for (int s = 0; s < 3 * k; ++s) {
    const int it = s / 3, kind = s % 3, L = it == k - 1 ? 1 : 0;
    q.t_begin = it * q.tiles_iter + q.begin[L][kind][0];
    q.t_end = it * q.tiles_iter + q.begin[L][kind][q.ngroups];
    q.round = rounds + 2 * s;
    e = launch_ns_fused(q, h->num_sms, st);
    if (e != cudaSuccess) return e;
    trace(h, MUON_KERNEL_GRAM + kind, st);
  }
  return cudaSuccess;
}

cudaError_t enqueue_tiles(muon_ctx* h, const std::vector<Item>& items, const muon_hparams_t* hp, bool store,
                          bool fuse, cudaStream_t st) {
  const std::vector<const GroupPlan*> groups = tiled_groups(h);
  if (groups.empty()) return cudaSuccess;
  if (small_tiles(h, hp->ns_steps)) return enqueue_small(h, hp, st);
  if (single_launch(h, hp->ns_steps)) return enqueue_single(h, items, hp, store, fuse, st);
  const int k = hp->ns_steps;
  for (int t = 0; t < k; ++t) {
    float own[3];
    const float* abc = coef_of(h, hp, t, own);
    for (int kind = kGram; kind <= kUpdate; ++kind) {
      NvtxRange range(kind == kGram ? "muon: Gram" : kind == kPoly ? "muon: polynomial" : "muon: update");
      for (size_t g0 = 0; g0 < groups.size(); g0 += kTcMaxGroups) {
        TcParams& prm = h->tc;
        std::memset(&prm, 0, sizeof(prm));
        const int ng = static_cast<int>(std::min<size_t>(kTcMaxGroups, groups.size() - g0));
        prm.ngroups = ng;
        prm.kind = kind;
        prm.half = 1;
        prm.scal = h->d_scal;
        prm.status = h->d_status;
        prm.timeout_ns = kTimeoutNs;
        const bool last = kind == kUpdate && t + 1 == k && fuse;
        // 256 x 512 Update tiles where there are enough of them (wide_pays) and, as on the bf16 path, every
        // padded width allows them and, where the launch writes the result, the k loops are long (mean m >= 2048)
        bool wide = kind == kUpdate && wide_pays(h, groups);
        double wsum = 0.0, wm = 0.0;
        for (int gi = 0; gi < ng; ++gi) {
          const GroupPlan& gp = *groups[g0 + gi];
          wide = wide && gp.np % 512 == 0;
          const double f = static_cast<double>(gp.cnt) * gp.mp * gp.mp * gp.np;
          wsum += f;
          wm += f * gp.mp;
        }
        if (last) wide = wide && wm >= 2048.0 * wsum;
        prm.wide = wide ? 1 : 0;
        if (kind == kGram) prm.c_acc = kHalfA / (kHalfX * kHalfX);
        if (kind == kPoly) {
          prm.c_acc = abc[2] * (kHalfB / (kHalfA * kHalfA));
          prm.c_aux = abc[1] * (kHalfB / kHalfA);
          prm.c_diag = abc[0] * kHalfB;
        }
        if (kind == kUpdate) prm.c_acc = 1.0f / kHalfB;
        if (last) fill_results(h, items, hp, store, &prm);
        int tiles = 0;
        for (int gi = 0; gi < ng; ++gi) {
          TcGroup& G = prm.g[gi];
          G.tile_begin = tiles;
          stage_group(h, *groups[g0 + gi], kind, t & 1, (t + 1) & 1, wide ? 512 : 256, &G);
          tiles += G.tiles_per_mat * G.cnt;
        }
        prm.total_tiles = tiles;
        const cudaError_t e = launch_tc_gemm(prm, h->num_sms, st);
        if (e != cudaSuccess) return e;
        trace(h, MUON_KERNEL_GRAM + kind, st);
      }
    }
  }
  return cudaSuccess;
}

// How `cnt` m x n matrices are laid over tiles and clusters: how many share a tile, into how many column
// ranges of at least 64 each is cut, and the fewest CTAs that hold them, by what the waves of tiles would take.
// Measured, an iteration of a tile takes about 7 k cycles for the A -> B' chain, 6 k more to add up
// the A of a cluster, 2.7 k more to add up column ranges, and 1.6 k for each 128 columns (1.15 k in the
// update, the rest its share of loading and storing the tile): 12 of 64 x 768 take 43 us in two ranges and
// 51 in one, 9 of 25 x 626 51 us in four and 83 in one.
void skinny_layout(const GroupPlan& gp, int cnt, int num_sms, SkinnyParams* p) {
  p->m = gp.m;
  p->n = gp.n;
  p->slot_rows = skinny_block(gp.m);
  const int most = kSkinnyRows / p->slot_rows;
  double best = -1.0;
  for (int slots = 1; slots <= most; slots *= 2) {
    for (int folds = 1; folds <= most / slots && (folds == 1 || (gp.n + folds - 1) / folds >= 64); folds *= 2) {
      int cluster = 1;
      while (cluster <= kSkinnyCluster &&
             gp.n > static_cast<long long>(folds) * cluster * (cluster <= 2 ? kSkinnyColsOne : kSkinnyColsPart))
        cluster *= 2;
      if (cluster > kSkinnyCluster) continue;
      const int width = ((gp.n + folds * cluster - 1) / (folds * cluster) + 63) / 64 * 64;
      const long long ctas = (static_cast<long long>(cnt) + slots - 1) / slots * cluster;
      const double waves = static_cast<double>((ctas + num_sms - 1) / num_sms);
      const double cost =
          waves * (7.0 + (cluster > 1 ? 6.0 : 0.0) + (folds > 1 ? 2.7 : 0.0) + 1.6 * ((width + 127) / 128));
      if (best < 0.0 || cost < best) {
        best = cost;
        p->slots = slots;
        p->folds = folds;
        p->cluster = cluster;
        p->width = width;
      }
    }
  }
}

cudaError_t enqueue_skinny(muon_ctx* h, const std::vector<Item>& items, const muon_hparams_t* hp, bool store,
                           bool normalised, cudaStream_t st) {
  for (size_t g = 0; g < h->plan.groups.size(); ++g) {
    const GroupPlan& gp = h->plan.groups[g];
    if (!gp.skinny) continue;
    SkinnyParams& p = h->sk;
    size_t i = 0;
    while (i < items.size()) {
      p.nseg = 0;
      p.total = 0;
      for (; i < items.size() && p.nseg < kSkinnySegs; ++i) {
        if (h->plan.mat_group[items[i].first] != static_cast<int>(g)) continue;
        ViewSeg& s = p.seg[p.nseg++];
        fill_seg(h, items[i], store, hp->lr, &s);
        s.mat_begin = p.total;
        p.total += items[i].count;
      }
      if (p.nseg == 0) break;
      skinny_layout(gp, p.total, h->num_sms, &p);
      p.normalised = normalised ? 1 : 0;
      p.k = hp->ns_steps;
      for (int t = 0; t < p.k; ++t) {
        float own[3];
        const float* abc = coef_of(h, hp, t, own);
        std::copy(abc, abc + 3, p.coef[t]);
      }
      p.eps = hp->eps;
      p.decay = store ? 0.0f : 1.0f - hp->lr * hp->weight_decay;
      p.norms = h->d_norms;
      p.status = h->d_status;
      p.timeout_ns = kTimeoutNs;
      const cudaError_t e = launch_ns_skinny(p, st);
      if (e != cudaSuccess) return e;
      trace(h, MUON_KERNEL_NS_SMALL, st);
    }
  }
  return cudaSuccess;
}

// Whether the workspace groups' iterations count completed tiles (enqueue_single), and of how many iterations.
int counted_iterations(const muon_ctx* h, int k) {
  return !tiled_groups(h).empty() && !small_tiles(h, k) && single_launch(h, k) ? k : 0;
}

// From sources in the caller's layout to the results.  `normalised`: the sources are 2^12 X already.
cudaError_t half_run(muon_ctx* h, std::vector<Item>& items, const muon_hparams_t* hp, bool store, bool normalised,
                     cudaStream_t st) {
  const int k = hp->ns_steps;
  cudaError_t e = cudaSuccess;
  if (!normalised) {
    if (!tiled_groups(h).empty()) e = clear_counters(h, counted_iterations(h, k), st);
    // view_sumsq_kernel's partial sums, one a tile
    int at = 0;
    for (Item& it : items) {
      const GroupPlan& gp = group_of(h, it.first);
      it.parts = ((gp.m + kEwTileR - 1) / kEwTileR) * ((gp.n + kEwTileC - 1) / kEwTileC);
      it.part_begin = at;
      at += it.parts * it.count;
    }
    if (e == cudaSuccess) e = view_pass(h, items, kSumsq, hp, store, normalised, 0, st);
  }
  if (e == cudaSuccess) e = view_pass(h, items, kOrient, hp, store, normalised, 0, st);
  const bool fuse = result_fusable(h, items, k);
  if (e == cudaSuccess) e = enqueue_tiles(h, items, hp, store, fuse, st);
  if (e == cudaSuccess && !fuse) e = view_pass(h, items, kWrite, hp, store, normalised, k & 1, st);
  if (e == cudaSuccess) e = enqueue_skinny(h, items, hp, store, normalised, st);
  return e;
}

// ---------------------------------------------------------------- state

StateFormat format_of(muon_state_format_t f) { return f == MUON_STATE_INT8 ? kStateInt8 : kStateE4M3; }
bool format_ok(muon_state_format_t f) { return f == MUON_STATE_INT8 || f == MUON_STATE_E4M3; }

muon_status_t check_state(const muon_state_t& s) {
  if (s.codes == nullptr || s.scales == nullptr || s.count < 1 || s.rows < 1 || s.cols < 1)
    return MUON_ERR_INVALID_ARG;
  if (s.count > 0x7fffffffll || s.rows > 0x7fffffffll || s.cols > 0x7fffffffll) return MUON_ERR_UNSUPPORTED;
  const int64_t blocks = (s.cols + kStateBlock - 1) / kStateBlock;
  if (s.rows * blocks >= 0x7fffffffll) return MUON_ERR_UNSUPPORTED;
  const int64_t ctas = (s.rows * blocks + kStateUnits - 1) / kStateUnits;
  if (ctas > 0x7fffffffll / s.count) return MUON_ERR_UNSUPPORTED;
  return (reinterpret_cast<uintptr_t>(s.scales) & 3u) == 0 ? MUON_OK : MUON_ERR_INVALID_ARG;
}

// The value side of a state: rows of contiguous elements.
struct Rows {
  char* data;
  int type;
  long long ld, bs;
  bool vec, linear;
};
muon_status_t make_rows(const muon_view_t& v, const muon_state_t& s, bool output, Rows* r) {
  if (v.data == nullptr || v.count != s.count) return MUON_ERR_INVALID_ARG;
  if (v.dtype != MUON_BF16 && v.dtype != MUON_FP32 && v.dtype != MUON_FP16) return MUON_ERR_INVALID_ARG;
  if (v.batch_stride < 0 || v.row_stride < 0 || v.col_stride < 0) return MUON_ERR_INVALID_ARG;
  if (v.col_stride != 1 && s.cols > 1) return MUON_ERR_UNSUPPORTED;
  const size_t es = type_bytes(static_cast<int>(v.dtype));
  if ((reinterpret_cast<uintptr_t>(v.data) % es) != 0) return MUON_ERR_INVALID_ARG;
  r->data = static_cast<char*>(v.data);
  r->type = static_cast<int>(v.dtype);
  r->ld = s.rows == 1 ? s.cols : v.row_stride;
  r->bs = s.count == 1 ? 0 : v.batch_stride;
  if (output) {
    const bool a = (s.rows == 1 || r->ld >= s.cols) && (s.count == 1 || r->bs >= (s.rows - 1) * r->ld + s.cols);
    const bool b = (s.count == 1 || r->bs >= s.cols) && (s.rows == 1 || r->ld >= (s.count - 1) * r->bs + s.cols);
    if (!a && !b) return MUON_ERR_INVALID_ARG;
  }
  r->vec = reinterpret_cast<uintptr_t>(v.data) % (4 * es) == 0 && s.cols % 4 == 0 &&
           (s.rows == 1 || r->ld % 4 == 0) && (s.count == 1 || r->bs % 4 == 0);
  // back to back (a stack's stride may still differ: matrices are found by it)
  r->linear = (reinterpret_cast<uintptr_t>(v.data) & 15u) == 0 && s.cols % kStateBlock == 0 &&
              (s.rows == 1 || r->ld == s.cols) && (s.count == 1 || r->bs * es % 16 == 0);
  return MUON_OK;
}

void fill_state(const muon_state_t& s, const Rows* in, const Rows* out, int mat, StateSeg* g) {
  std::memset(g, 0, sizeof(*g));
  g->codes = s.codes;
  g->scales = s.scales;
  g->rows = static_cast<int>(s.rows);
  g->cols = static_cast<int>(s.cols);
  g->blocks = static_cast<int>((s.cols + kStateBlock - 1) / kStateBlock);
  g->count = static_cast<int>(s.count);
  g->mat_begin = mat;
  g->unit_ctas = static_cast<int>((s.rows * g->blocks + kStateUnits - 1) / kStateUnits);
  bool vec = (reinterpret_cast<uintptr_t>(s.codes) & 3u) == 0;
  bool linear = (reinterpret_cast<uintptr_t>(s.codes) & 7u) == 0 && s.cols % kStateBlock == 0;
  if (in != nullptr) {
    g->in = in->data;
    g->in_ld = in->ld;
    g->in_bs = in->bs;
    g->in_type = in->type;
    vec = vec && in->vec;
    linear = linear && in->linear;
  }
  if (out != nullptr) {
    g->out = out->data;
    g->out_ld = out->ld;
    g->out_bs = out->bs;
    g->out_type = out->type;
    vec = vec && out->vec;
    linear = linear && out->linear;
  }
  g->vec = vec ? 1 : 0;
  g->linear = linear ? 1 : 0;
}

// Quantise (X read) or dequantise (X written).
muon_status_t convert(const muon_view_t* X, const muon_state_t* S, int n, muon_state_format_t format,
                      const uint32_t* seed, bool write_state, cudaStream_t st) {
  if (n < 0 || !format_ok(format)) return MUON_ERR_INVALID_ARG;
  if (n == 0) return MUON_OK;
  if (X == nullptr || S == nullptr) return MUON_ERR_INVALID_ARG;
  long long mats = 0;
  for (int j = 0; j < n; ++j) {
    muon_status_t r = check_state(S[j]);
    if (r != MUON_OK) return r;
    Rows rows;
    r = make_rows(X[j], S[j], !write_state, &rows);
    if (r != MUON_OK) return r;
    if (X[j].dtype != X[0].dtype) return MUON_ERR_INVALID_ARG;
    mats += S[j].count;
    if (mats > 0x7fffffffll) return MUON_ERR_UNSUPPORTED;
  }
  if (write_state) {
    if (!states_distinct(S, n)) return MUON_ERR_INVALID_ARG;
  } else if (n > 1) {
    std::vector<const void*> at;
    for (int j = 0; j < n; ++j) at.push_back(X[j].data);
    if (!distinct(at)) return MUON_ERR_INVALID_ARG;
  }
  static thread_local StateParams p;  // 4 KB that need no clearing
  int j = 0, mat = 0;
  while (j < n) {
    p.nseg = 0;
    p.total = 0;
    p.linear = 1;
    p.stochastic = seed != nullptr;
    p.seed = seed != nullptr ? *seed : 0u;
    for (; j < n && p.nseg < kStateSegs; ++j) {
      StateSeg g;
      Rows rows;
      make_rows(X[j], S[j], !write_state, &rows);
      fill_state(S[j], write_state ? &rows : nullptr, write_state ? nullptr : &rows, mat, &g);
      const long long ctas = static_cast<long long>(g.unit_ctas) * g.count;
      if (p.total + ctas > 0x7fffffffll) break;  // (one state fits: check_state)
      g.cta_begin = p.total;
      p.linear &= g.linear;
      p.seg[p.nseg++] = g;
      p.total += static_cast<int>(ctas);
      mat += g.count;
    }
    const StateFormat f = format_of(format);
    const cudaError_t e = write_state ? launch_state_quantize(p, f, st) : launch_state_dequantize(p, f, st);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

// A momentum's sources and results: G, the state (or, as its codes, the dense momentum), and U.
struct MomentumIn {
  muon_state_t state;
  Rows g, u;
  int first;
};
// One pass over every matrix of the call.
cudaError_t momentum_pass(muon_ctx* h, const std::vector<MomentumIn>& in, StateFormat f, StatePass pass,
                          const muon_hparams_t* hp, const uint32_t* seed, cudaStream_t st) {
  NvtxRange range(pass == kPassNorm ? "muon: norm" : "muon: momentum");
  StateParams& p = h->st;
  size_t j = 0;
  int part = 0;
  while (j < in.size()) {
    p.nseg = 0;
    p.total = 0;
    p.linear = 1;
    p.stochastic = seed != nullptr;
    p.seed = seed != nullptr ? *seed : 0u;
    p.beta = hp->beta;
    p.nesterov = hp->nesterov ? 1 : 0;
    p.eps = hp->eps;
    p.partials = reinterpret_cast<double*>(h->d_partials) + part;
    p.norms = h->d_norms;
    p.factors = h->d_scal;
    p.arrivals = reinterpret_cast<unsigned int*>(h->ws + h->plan.off_arrivals);
    for (; j < in.size() && p.nseg < kStateSegs; ++j) {
      StateSeg g;
      fill_state(in[j].state, &in[j].g, pass == kPassNorm ? nullptr : &in[j].u, in[j].first, &g);
      if (f == kStateDense && (reinterpret_cast<uintptr_t>(g.codes) & 15u) != 0) g.vec = g.linear = 0;
      p.linear &= g.linear;
      g.caller_idx = in[j].first;
      g.cta_begin = p.total;
      p.seg[p.nseg++] = g;
      p.total += g.unit_ctas * g.count;  // (bounded by the workspace's partial sums)
    }
    part += p.total;
    const cudaError_t e = launch_state_momentum(p, f, pass, st);
    if (e != cudaSuccess) return e;
    trace(h, MUON_KERNEL_MOMENTUM_NORM, st);
  }
  return cudaSuccess;
}

// Where a step's normalised direction goes: X0 itself where the caller's layout is X0's, else a place in
// the workspace that the orientation or the on-chip kernel reads.
void stage(muon_ctx* h, int mat, int count, Item* item, Rows* rows) {
  const GroupPlan& gp = group_of(h, mat);
  const muon_shape_t& sh = h->shapes[mat];
  item->is_x0 = !gp.skinny && !tall(h, mat) && gp.mp == gp.m && gp.np == gp.n;
  const size_t at = item->is_x0 ? gp.off_x[0] + static_cast<size_t>(h->plan.mat_slot[mat]) * gp.mp * gp.np * 2
                                : h->plan.off_u[mat];
  muon_view_t v = contiguous(h->ws + at, sh, MUON_FP16);
  v.count = count;
  if (count > 1 && !item->is_x0) v.batch_stride = static_cast<int64_t>((h->plan.off_u[mat + 1] - h->plan.off_u[mat]) / 2);
  make_side(v, sh.rows, sh.cols, false, &item->src);
  const muon_state_t s{nullptr, nullptr, count, sh.rows, sh.cols};
  make_rows(v, s, false, rows);
}

cudaError_t run_step(muon_ctx* h, std::vector<Item>& items, const std::vector<MomentumIn>& in, StateFormat f,
                     const muon_hparams_t* hp, const uint32_t* seed, cudaStream_t st) {
  cudaError_t e = clear_counters(h, counted_iterations(h, hp->ns_steps), st);
  if (e == cudaSuccess) e = momentum_pass(h, in, f, kPassNorm, hp, nullptr, st);
  if (e == cudaSuccess) e = momentum_pass(h, in, f, kPassStep, hp, seed, st);
  if (e == cudaSuccess) e = half_run(h, items, hp, false, true, st);
  return e;
}

}  // namespace

muon_status_t muon::half_orthogonalize(muon_ctx* h, const void* const* X, void* const* O, const muon_hparams_t* hp,
                                       cudaStream_t stream) {
  return no_throw([&]() -> muon_status_t {
    std::vector<muon_view_t> x, o;
    for (int i = 0; i < h->n; ++i) {
      x.push_back(contiguous(X[i], h->shapes[i], h->dtype));
      o.push_back(contiguous(O[i], h->shapes[i], h->dtype));
    }
    return muon_orthogonalize_views(h, x.data(), o.data(), h->n, hp, stream);
  });
}

muon_status_t muon::half_step(muon_ctx* h, void* const* W, const void* const* G, void* const* M,
                              const muon_hparams_t* hp, cudaStream_t stream) {
  return no_throw([&]() -> muon_status_t {
    if (!steps_ok(h, hp)) return MUON_ERR_INVALID_ARG;
    std::vector<const void*> outs(W, W + h->n);
    outs.insert(outs.end(), M, M + h->n);
    if (!distinct(outs)) return MUON_ERR_INVALID_ARG;
    std::vector<Item> items(h->n);
    std::vector<MomentumIn> in(h->n);
    for (int i = 0; i < h->n; ++i) {
      const muon_shape_t& sh = h->shapes[i];
      const muon_view_t w = contiguous(W[i], sh, h->dtype), g = contiguous(G[i], sh, h->dtype);
      const size_t es = h->dtype == MUON_BF16 ? 2 : 4;
      if ((reinterpret_cast<uintptr_t>(M[i]) % es) != 0) return MUON_ERR_INVALID_ARG;
      items[i].first = in[i].first = i;
      items[i].count = 1;
      in[i].state = muon_state_t{M[i], nullptr, 1, sh.rows, sh.cols};
      muon_status_t r = make_side(w, sh.rows, sh.cols, true, &items[i].dst);
      if (r == MUON_OK) r = make_rows(g, in[i].state, false, &in[i].g);
      if (r != MUON_OK) return r;
      stage(h, i, 1, &items[i], &in[i].u);
    }
    DeviceGuard guard(h->device);
    NvtxRange range("muon_step");
    trace(h, -1, stream);
    const cudaError_t e = run_step(h, items, in, kStateDense, hp, nullptr, stream);
    trace_call_end(h);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  });
}

bool muon::half_fused_possible(const muon_ctx* h) {
  const size_t n = tiled_groups(h).size();
  return n >= 1 && n <= static_cast<size_t>(kTcMaxGroups);
}

int muon::half_launches(const muon_ctx* h, int k) {
  // a muon_step: every matrix is a view of its own
  int tiled = 0, ngroups = 0, skinny = 0;
  for (const GroupPlan& gp : h->plan.groups) {
    if (gp.skinny) {
      skinny += (gp.cnt + kSkinnySegs - 1) / kSkinnySegs;
    } else {
      tiled += gp.cnt;
      ++ngroups;
    }
  }
  const int views = (tiled + kViewSegs - 1) / kViewSegs;
  int turned = 0;  // matrices whose direction is transposed or padded on its way to X0
  for (int i = 0; i < h->n; ++i) {
    const GroupPlan& gp = group_of(h, i);
    turned += !gp.skinny && (tall(h, i) || gp.mp != gp.m || gp.np != gp.n);
  }
  bool fused = k >= 1 && h->dtype == MUON_BF16 && h->n <= kTcMaxFused && !small_tiles(h, k);
  for (const GroupPlan& gp : h->plan.groups)
    if (!gp.skinny && (gp.m % 32 != 0 || gp.n % 32 != 0)) fused = false;
  const int stages = ngroups == 0            ? 0
                     : small_tiles(h, k)     ? 1
                     : single_launch(h, k)   ? (h->schedule == MUON_SCHEDULE_SPLIT ? 3 * k : 1)
                                             : 3 * k * ((ngroups + kTcMaxGroups - 1) / kTcMaxGroups);
  return 2 * ((h->n + kStateSegs - 1) / kStateSegs) + (turned + kViewSegs - 1) / kViewSegs + stages +
         (fused ? 0 : views) + skinny;
}

extern "C" {

muon_status_t muon_set_coefficients(muon_handle_t h, const float* abc, int steps) {
  if (h == nullptr || steps < 0 || steps > kMaxSteps || (steps > 0 && abc == nullptr)) return MUON_ERR_INVALID_ARG;
  if (h->mode != MUON_MODE_HALF) return MUON_ERR_UNSUPPORTED;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(abc[i])) return MUON_ERR_INVALID_ARG;
  return no_throw([&]() -> muon_status_t {
    h->coef.assign(abc, abc + 3 * steps);
    return MUON_OK;
  });
}

muon_status_t muon_orthogonalize_views(muon_handle_t h, const muon_view_t* X, const muon_view_t* O, int n,
                                       const muon_hparams_t* hp, cudaStream_t stream) {
  if (h == nullptr || X == nullptr || O == nullptr || n < 1 || !hp_ok(hp, false)) return MUON_ERR_INVALID_ARG;
  if (h->mode != MUON_MODE_HALF) return MUON_ERR_UNSUPPORTED;
  if (!steps_ok(h, hp)) return MUON_ERR_INVALID_ARG;
  return no_throw([&]() -> muon_status_t {
    std::vector<int> first;
    muon_status_t r = cover(h, X, n, &first);
    if (r != MUON_OK) return r;
    std::vector<Item> items(n);
    std::vector<const void*> ins, outs;
    for (int j = 0; j < n; ++j) {
      if (O[j].count != X[j].count) return MUON_ERR_INVALID_ARG;
      const muon_shape_t& sh = h->shapes[first[j]];
      items[j].first = first[j];
      items[j].count = static_cast<int>(X[j].count);
      r = make_side(X[j], sh.rows, sh.cols, false, &items[j].src);
      if (r == MUON_OK) r = make_side(O[j], sh.rows, sh.cols, true, &items[j].dst);
      if (r != MUON_OK) return r;
      const Side &a = items[j].src, &b = items[j].dst;  // in place: an element is written where it was read
      if (a.data == b.data && (a.type != b.type || a.by_cols != b.by_cols || a.ld != b.ld || a.bs != b.bs))
        return MUON_ERR_INVALID_ARG;
      ins.push_back(X[j].data);
      outs.push_back(O[j].data);
    }
    if (!apart(ins, outs)) return MUON_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    NvtxRange range("muon_orthogonalize_views");
    muon_hparams_t q = *hp;
    q.lr = 0.0f;
    q.weight_decay = 0.0f;
    trace(h, -1, stream);
    const cudaError_t e = half_run(h, items, &q, true, false, stream);
    trace_call_end(h);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  });
}

muon_status_t muon_state_quantize(const muon_view_t* X, const muon_state_t* S, int n, muon_state_format_t format,
                                  const uint32_t* seed, cudaStream_t stream) {
  return no_throw([&] { return convert(X, S, n, format, seed, true, stream); });
}

muon_status_t muon_state_dequantize(const muon_state_t* S, const muon_view_t* X, int n, muon_state_format_t format,
                                    cudaStream_t stream) {
  return no_throw([&] { return convert(X, S, n, format, nullptr, false, stream); });
}

muon_status_t muon_momentum_state(muon_handle_t h, const muon_view_t* G, const muon_state_t* S, const muon_view_t* U,
                                  int n, muon_state_format_t format, const muon_hparams_t* hp, const uint32_t* seed,
                                  cudaStream_t stream) {
  if (h == nullptr || G == nullptr || S == nullptr || U == nullptr || n < 1 || !format_ok(format) || hp == nullptr ||
      !std::isfinite(hp->beta) || hp->beta < 0.0f || hp->beta > 1.0f)
    return MUON_ERR_INVALID_ARG;
  return no_throw([&]() -> muon_status_t {
    std::vector<int> first;
    muon_status_t r = cover(h, G, n, &first);
    if (r != MUON_OK) return r;
    std::vector<MomentumIn> in(n);
    std::vector<const void*> ins, outs;
    for (int j = 0; j < n; ++j) {
      const muon_shape_t& sh = h->shapes[first[j]];
      if (S[j].rows != sh.rows || S[j].cols != sh.cols || G[j].dtype != h->dtype || U[j].dtype != h->dtype)
        return MUON_ERR_INVALID_ARG;
      r = check_state(S[j]);
      if (r == MUON_OK) r = make_rows(G[j], S[j], false, &in[j].g);
      if (r == MUON_OK) r = make_rows(U[j], S[j], true, &in[j].u);
      if (r != MUON_OK) return r;
      if (U[j].data == G[j].data && (in[j].u.ld != in[j].g.ld || in[j].u.bs != in[j].g.bs)) return MUON_ERR_INVALID_ARG;
      ins.push_back(G[j].data);
      outs.push_back(U[j].data);
      in[j].state = S[j];
      in[j].first = first[j];
    }
    if (!apart(ins, outs) || !states_distinct(S, n)) return MUON_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    trace(h, -1, stream);
    cudaError_t e = clear_counters(h, 0, stream);
    if (e == cudaSuccess) e = momentum_pass(h, in, format_of(format), kPassMomentum, hp, seed, stream);
    trace_call_end(h);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  });
}

muon_status_t muon_step_state(muon_handle_t h, const muon_view_t* W, const muon_view_t* G, const muon_state_t* S,
                              int n, muon_state_format_t format, const muon_hparams_t* hp, const uint32_t* seed,
                              cudaStream_t stream) {
  if (h == nullptr || W == nullptr || G == nullptr || S == nullptr || n < 1 || !format_ok(format) ||
      !hp_ok(hp, true))
    return MUON_ERR_INVALID_ARG;
  if (h->mode != MUON_MODE_HALF) return MUON_ERR_UNSUPPORTED;
  if (!steps_ok(h, hp)) return MUON_ERR_INVALID_ARG;
  return no_throw([&]() -> muon_status_t {
    std::vector<int> first;
    muon_status_t r = cover(h, W, n, &first);
    if (r != MUON_OK) return r;
    std::vector<Item> items(n);
    std::vector<MomentumIn> in(n);
    for (int j = 0; j < n; ++j) {
      const muon_shape_t& sh = h->shapes[first[j]];
      if (S[j].rows != sh.rows || S[j].cols != sh.cols || S[j].count != W[j].count || G[j].dtype != h->dtype ||
          W[j].dtype != h->dtype)
        return MUON_ERR_INVALID_ARG;
      items[j].first = in[j].first = first[j];
      items[j].count = static_cast<int>(W[j].count);
      r = check_state(S[j]);
      if (r == MUON_OK) r = make_rows(G[j], S[j], false, &in[j].g);
      if (r == MUON_OK) r = make_side(W[j], sh.rows, sh.cols, true, &items[j].dst);
      if (r != MUON_OK) return r;
      in[j].state = S[j];
      stage(h, first[j], items[j].count, &items[j], &in[j].u);
    }
    std::vector<const void*> outs;
    for (int j = 0; j < n; ++j) outs.push_back(W[j].data);
    if (!distinct(outs) || !states_distinct(S, n)) return MUON_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    NvtxRange range("muon_step_state");
    trace(h, -1, stream);
    const cudaError_t e = run_step(h, items, in, format_of(format), hp, seed, stream);
    trace_call_end(h);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  });
}

}  // extern "C"
