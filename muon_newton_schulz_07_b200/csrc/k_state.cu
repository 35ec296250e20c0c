// 8-bit optimizer state: quantised as it is written, read back, and updated in place by the
// momentum of the next step.
//
// A state holds one code a value and one fp32 scale for every 128 columns of a row (the last block
// of a row may be shorter).  With t the largest magnitude of the block and T the largest code (127
// for int8, 448 for e4m3):
//   write   y = x * (T / t);  int8: code = rint(y), e4m3: code = y rounded to e4m3;  scale = t / T
//   read    x = code * scale
// A block whose t is below 2^-100 is written as zeros with scale 0; a block holding an infinity
// or a NaN gets the scale NaN, so that what is read back shows it.  Rounding is to nearest even, or
// stochastic: with u in [0, 1) from 16 random bits, floor(y + u) in units of the code's spacing (for
// e4m3 on the magnitude), whose expectation is y up to 2^-17 of the spacing.  An average with a decay of a few percent a
// step needs that: a change below half a code is otherwise lost every time.
//   momentum  m1 = beta m + (1 - beta) g;  u = (1 - beta) g + beta m1, or m1;  m1 written back
// Every operation is rounded by itself (no contraction), so that the codes are the same function
// of the inputs wherever the formula is evaluated in fp32.
//
// All three are bound by memory traffic (bf16: 3.03 bytes a value to write, 3.03 to read back, 6.06
// for the momentum).  A unit is one block of one row, 16 lanes of 8 values; consecutive units are
// consecutive in memory, so a CTA of 64 units streams up to 8192 contiguous values whatever the
// row length, and a thread has the loads of all four of its units in flight before it computes.
// Rows that are not a multiple of 8 long (or not aligned) interleave the 16 lanes instead, one
// value each, which keeps the accesses of a half-warp contiguous.
#include <cuda_fp8.h>

#include "muon_view.cuh"

namespace muon {
namespace {

constexpr int THREADS = 256;
constexpr int LANES = 16;                       // lanes of a unit
constexpr int PASSES = kStateUnits * LANES / THREADS;
static_assert(PASSES == 4 && kStateBlock == LANES * 8, "a CTA takes its units in four passes");

// ---------------------------------------------------------------- random bits

// Two xor-shift and multiply rounds (odd factors: the leading bits of the square roots of 2 and 3).
__host__ __device__ __forceinline__ uint32_t mixed(uint32_t h) {
  h ^= h >> 16;
  h *= 0x6A09E667u;
  h ^= h >> 15;
  h *= 0xBB67AE85u;
  h ^= h >> 16;
  return h;
}
__device__ __forceinline__ uint32_t matrix_key(uint32_t seed, uint32_t matrix) { return mixed(mixed(seed) ^ matrix); }
// The 32 bits that places 2 pair and 2 pair + 1 of a matrix share, the lower half first.
__device__ __forceinline__ uint32_t pair_bits(uint32_t key, unsigned long long pair) {
  return mixed(static_cast<uint32_t>(pair) + key + static_cast<uint32_t>(pair >> 32) * 0x9E3779B1u);
}

// ---------------------------------------------------------------- codes

// Four int8 codes in a word, widened: the byte, offset by 128, becomes the low mantissa bits of 2^23.
__device__ __forceinline__ void widen_int8(uint32_t w, float* v) {
  const uint32_t b = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + i)) - 8388736.0f;  // 2^23 + 128
}
__device__ __forceinline__ void widen_e4m3(uint32_t w, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <int F>
struct Range;
template <>
struct Range<kStateInt8> {
  static constexpr float top = 127.0f;
};
template <>
struct Range<kStateE4M3> {
  static constexpr float top = 448.0f;
};

// Four values, scaled to the codes' range, as a word of codes; r: two words of 16 random bits each.
// The kernels that round stochastically are bound by the integer and logic pipe, whose rate is half
// of the FMA pipe's (and conversions and floor() run at a quarter): so the random bits become a float by one
// byte permutation and an addition, and rounding down is an addition that rounds down.
template <int F, bool STOCHASTIC>
__device__ __forceinline__ uint32_t encode4(const float* y, const uint32_t (&r)[2]) {
  uint32_t b[4];
  float g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 2^23 + the 16 bits, as the bits of a float
    const float bits = STOCHASTIC ? __uint_as_float(__byte_perm(r[i >> 1], 0x4B000000u, (i & 1) ? 0x7632 : 0x7610)) : 0.0f;
    const float u = STOCHASTIC ? __fsub_rn(bits, 8388608.0f) : 0.0f;  // 2^16 u
    if (F == kStateInt8) {
      if (STOCHASTIC)
        b[i] = __float_as_uint(__fadd_rd(fminf(fmaxf(__fmaf_rn(u, 0x1p-16f, y[i]), -127.0f), 127.0f), 12582912.0f));
      else
        b[i] = __float_as_uint(__fadd_rn(y[i], 12582912.0f));  // 1.5 * 2^23: negative values too
    } else if (STOCHASTIC) {
      // The spacing at |y| is an eighth of its binade, and of 2^-6 below that.  |y| + u spacing is exact
      // (or passes into the next binade, whose first code it then is), and adding 2^23 spacings,
      // rounded down, and taking them off again leaves whole spacings.
      const uint32_t bits_y = __float_as_uint(y[i]);
      const float binade = __uint_as_float(max(bits_y & 0x7F800000u, 0x3C800000u));
      const float z = __fmaf_rn(u, binade * 0x1p-19f, fabsf(y[i]));
      const float v = __fsub_rn(__fadd_rd(z, binade * 0x1p20f), binade * 0x1p20f);
      g[i] = __uint_as_float(__float_as_uint(v) | (bits_y & 0x80000000u));
    } else {
      g[i] = y[i];
    }
  }
  if (F == kStateE4M3) {  // exact for values on the grid; 448 is the largest
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(g[0], g[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(g[2], g[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// max(a, |b|), NaN above all.
__device__ __forceinline__ float max_size(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// Factor and scale of a block from its largest magnitude (as bits: NaN above infinity above all).
template <int F>
__device__ __forceinline__ void unit_scale(uint32_t top_bits, float& mul, float& scale) {
  const float t = __uint_as_float(top_bits);
  mul = 0.0f;
  scale = 0.0f;
  if (top_bits >= 0x7F800000u) {
    scale = __uint_as_float(0x7FC00000u);
  } else if (t >= 0x1p-100f) {
    mul = __fdiv_rn(Range<F>::top, t);
    scale = __fdiv_rn(t, Range<F>::top);
  }
}

// ---------------------------------------------------------------- units

struct Unit {
  int row, col;        // the unit's row, its first column
  int have;            // values of the unit (0: beyond the matrix)
};
struct Cta {
  int seg, e;
  uint32_t first;      // first unit of this CTA in its matrix
};
__device__ __forceinline__ Cta find(const StateParams& p) {
  const int cta = static_cast<int>(blockIdx.x);
  int lo = 0, hi = p.nseg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seg[mid].cta_begin <= cta) lo = mid; else hi = mid - 1;
  }
  const StateSeg& s = p.seg[lo];
  const int at = cta - s.cta_begin;
  Cta c;
  c.seg = lo;
  c.e = at / s.unit_ctas;
  c.first = static_cast<uint32_t>(at - c.e * s.unit_ctas) * kStateUnits;
  return c;
}
constexpr int UNITS = THREADS / LANES;  // of a pass
// The units of this thread's 16 lanes, one a pass: one division, then steps of UNITS.
__device__ __forceinline__ void units_of(const StateSeg& s, const Cta& c, Unit (&u)[PASSES]) {
  const uint32_t at = c.first + threadIdx.x / LANES;  // below 2^31 + 64
  uint32_t row = at / static_cast<uint32_t>(s.blocks), block = at - row * s.blocks;
  const uint32_t rows = UNITS / static_cast<uint32_t>(s.blocks), blocks = UNITS - rows * s.blocks;
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    u[q].row = static_cast<int>(row);
    u[q].col = static_cast<int>(block) * kStateBlock;
    u[q].have = row < static_cast<uint32_t>(s.rows) ? min(kStateBlock, s.cols - u[q].col) : 0;
    row += rows;
    block += blocks;
    if (block >= static_cast<uint32_t>(s.blocks)) {
      block -= s.blocks;
      ++row;
    }
  }
}
__device__ __forceinline__ int unit_lane() { return threadIdx.x % LANES; }
// Of a unit's first value in the codes of the stack, and of its scale.
__device__ __forceinline__ long long code_at(const StateSeg& s, const Cta& c, const Unit& u) {
  return (static_cast<long long>(c.e) * s.rows + u.row) * s.cols + u.col;
}
__device__ __forceinline__ long long scale_at(const StateSeg& s, const Cta& c, const Unit& u) {
  return (static_cast<long long>(c.e) * s.rows + u.row) * s.blocks + u.col / kStateBlock;
}
// Value i of a lane sits at this place of the unit: eight neighbours, or interleaved lanes.
__device__ __forceinline__ int place(bool vec, int lane, int i) { return vec ? lane * 8 + i : lane + LANES * i; }

// Eight values of a stored row as they come from memory (widened only when they are used, so that
// the loads of several units can be in flight).
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(int i, const float* p) { v[i] = __ldcs(p); }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
};
template <typename T>
struct Eight16 {
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  }
  __device__ __forceinline__ void set(int i, const T* p) {
    const uint32_t b = __ldcs(reinterpret_cast<const unsigned short*>(p));
    w[i >> 1] = (i & 1) ? (w[i >> 1] | b << 16) : b;
  }
};
template <>
struct Eight<__nv_bfloat16> : Eight16<__nv_bfloat16> {
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    widen8(make_uint4(w[0], w[1], w[2], w[3]), kViewBF16, x);
  }
};
template <>
struct Eight<__half> : Eight16<__half> {
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    widen8(make_uint4(w[0], w[1], w[2], w[3]), kViewF16, x);
  }
};
template <typename T>
struct TypeOf;
template <>
struct TypeOf<float> { static constexpr int id = kViewF32; };
template <>
struct TypeOf<__nv_bfloat16> { static constexpr int id = kViewBF16; };
template <>
struct TypeOf<__half> { static constexpr int id = kViewF16; };

// Store a lane's eight values.
template <typename T>
__device__ __forceinline__ void store_unit(T* base, bool vec, const Unit& u, const float (&x)[8]) {
  const int lane = unit_lane();
  if (vec) {
    if (lane * 8 < u.have) store_eight(base, TypeOf<T>::id, lane * 8, 8, true, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = place(false, lane, i);
      if (at < u.have) store_one(base, TypeOf<T>::id, at, x[i]);
    }
  }
}

// Write the four units of these 16 lanes.  The largest magnitudes of all four go through one
// exchange: each step halves the units a lane still holds, so that quarter q of the lanes ends with
// unit q's, divides once, and hands factor and scale back.
template <int F, bool STOCHASTIC>
__device__ __forceinline__ void write_units(const StateSeg& s, const Cta& c, bool vec, const Unit (&u)[PASSES],
                                            uint32_t key, float (&x)[PASSES][8]) {
  const int lane = unit_lane();
  uint32_t top[PASSES];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    float m = fabsf(x[q][0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_size(m, x[q][i]);
    top[q] = __float_as_uint(m) & 0x7FFFFFFFu;
  }
  const bool hi8 = lane & 8, hi4 = lane & 4;
  uint32_t a = hi8 ? top[2] : top[0], b = hi8 ? top[3] : top[1];
  a = max(a, __shfl_xor_sync(0xffffffffu, hi8 ? top[0] : top[2], 8));
  b = max(b, __shfl_xor_sync(0xffffffffu, hi8 ? top[1] : top[3], 8));
  uint32_t t = max(hi4 ? b : a, __shfl_xor_sync(0xffffffffu, hi4 ? a : b, 4));
  t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
  t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
  float my_mul, my_scale;
  unit_scale<F>(t, my_mul, my_scale);
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    const float mul = __shfl_sync(0xffffffffu, my_mul, q * 4, LANES);
    const bool fine = __shfl_sync(0xffffffffu, t, q * 4, LANES) < 0x7F800000u;
    if (lane == q * 4 && u[q].have > 0) s.scales[scale_at(s, c, u[q])] = my_scale;
    uint8_t* codes = static_cast<uint8_t*>(s.codes) + code_at(s, c, u[q]);
    const unsigned long long at = static_cast<unsigned long long>(u[q].row) * s.cols + u[q].col;  // in the matrix
#pragma unroll
    for (int i = 0; i < 8; ++i) x[q][i] = __fmul_rn(x[q][i], mul);
    if (!fine) {  // rare: not finite
#pragma unroll
      for (int i = 0; i < 8; ++i) x[q][i] = 0.0f;
    }
    uint32_t r[4] = {0, 0, 0, 0};
    if (STOCHASTIC) {
      if (vec) {  // eight neighbours from an even place: four pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = pair_bits(key, (at + lane * 8) / 2 + i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned long long here = at + place(false, lane, i);
          const uint32_t h = pair_bits(key, here >> 1) >> (16 * (here & 1)) & 0xFFFFu;
          r[i >> 1] |= h << (16 * (i & 1));
        }
      }
    }
    const uint32_t r0[2] = {r[0], r[1]}, r1[2] = {r[2], r[3]};
    const uint32_t lo = encode4<F, STOCHASTIC>(x[q], r0), hi = encode4<F, STOCHASTIC>(x[q] + 4, r1);
    if (vec) {
      if (lane * 8 < u[q].have) __stcs(reinterpret_cast<uint2*>(codes + lane * 8), make_uint2(lo, hi));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int to = place(false, lane, i);
        if (to < u[q].have) codes[to] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
}

// The codes of a lane's eight values, as loaded.
struct Codes {
  uint32_t w[2];
  float scale;
};
__device__ __forceinline__ void load_codes(const StateSeg& s, const Cta& cta, bool vec, const Unit& u, Codes& c) {
  const int lane = unit_lane();
  const uint8_t* p = static_cast<const uint8_t*>(s.codes) + code_at(s, cta, u);
  c.w[0] = c.w[1] = 0;
  c.scale = u.have > 0 ? s.scales[scale_at(s, cta, u)] : 0.0f;
  if (vec) {
    if (lane * 8 < u.have) {
      const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p + lane * 8));
      c.w[0] = q.x;
      c.w[1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = place(false, lane, i);
      if (at < u.have) c.w[i >> 2] |= static_cast<uint32_t>(p[at]) << (8 * (i & 3));
    }
  }
}
template <int F>
__device__ __forceinline__ void read_codes(const Codes& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (F == kStateInt8) widen_int8(c.w[i], x + 4 * i);
    else widen_e4m3(c.w[i], x + 4 * i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], c.scale);
}

template <typename T>
__device__ __forceinline__ void load_values(const T* base, bool vec, const Unit& u, Eight<T>& x) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(x) / 4); ++i) reinterpret_cast<uint32_t*>(&x)[i] = 0;
  const int lane = unit_lane();
  if (vec) {
    if (lane * 8 < u.have) x.load(base + lane * 8);  // rows are multiples of 8: all or nothing
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = place(false, lane, i);
      if (at < u.have) x.set(i, base + at);
    }
  }
}

template <typename T>
__device__ __forceinline__ const T* in_row(const StateSeg& s, const Cta& c, const Unit& u) {
  return static_cast<const T*>(s.in) + c.e * s.in_bs + u.row * s.in_ld + u.col;
}
template <typename T>
__device__ __forceinline__ T* out_row(const StateSeg& s, const Cta& c, const Unit& u) {
  return static_cast<T*>(s.out) + c.e * s.out_bs + u.row * s.out_ld + u.col;
}

template <typename T, int F, bool STOCHASTIC>
__global__ void __launch_bounds__(THREADS) state_quantize_kernel(const __grid_constant__ StateParams p) {
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  const uint32_t key = STOCHASTIC ? matrix_key(p.seed, static_cast<uint32_t>(s.mat_begin + c.e)) : 0u;
  Unit u[PASSES];
  units_of(s, c, u);
  Eight<T> raw[PASSES];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) load_values<T>(in_row<T>(s, c, u[q]), vec, u[q], raw[q]);
  float x[PASSES][8];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) raw[q].widen(x[q]);
  write_units<F, STOCHASTIC>(s, c, vec, u, key, x);
}

template <typename T, int F>
__global__ void __launch_bounds__(THREADS) state_dequantize_kernel(const __grid_constant__ StateParams p) {
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  Unit u[PASSES];
  units_of(s, c, u);
  Codes raw[PASSES];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) load_codes(s, c, vec, u[q], raw[q]);
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    float x[8];
    read_codes<F>(raw[q], x);
    store_unit<T>(out_row<T>(s, c, u[q]), vec, u[q], x);
  }
}

// Momentum and Nesterov blend of one CTA's units; F = kStateDense keeps m in T.
template <typename T, int F, bool STOCHASTIC>
__global__ void __launch_bounds__(THREADS) state_momentum_kernel(const __grid_constant__ StateParams p) {
  __shared__ float red[THREADS / 32];
  constexpr bool DENSE = F == kStateDense;
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  const uint32_t key = STOCHASTIC ? matrix_key(p.seed, static_cast<uint32_t>(s.mat_begin + c.e)) : 0u;
  const float beta = p.beta, rest = __fsub_rn(1.0f, p.beta);
  Unit u[PASSES];
  units_of(s, c, u);
  Eight<T> raw[PASSES];
  Codes codes[DENSE ? 1 : PASSES];
  Eight<T> dense[DENSE ? PASSES : 1];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    load_values<T>(in_row<T>(s, c, u[q]), vec, u[q], raw[q]);
    if (DENSE)
      load_values<T>(static_cast<const T*>(s.codes) + code_at(s, c, u[q]), vec, u[q], dense[DENSE ? q : 0]);
    else
      load_codes(s, c, vec, u[q], codes[DENSE ? 0 : q]);
  }
  float ss = 0.0f;
  float m[PASSES][8];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    float g[8];
    raw[q].widen(g);
    if (DENSE)
      dense[DENSE ? q : 0].widen(m[q]);
    else
      read_codes<DENSE ? kStateInt8 : F>(codes[DENSE ? 0 : q], m[q]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = __fmul_rn(g[i], rest);
      m[q][i] = __fadd_rn(__fmul_rn(m[q][i], beta), g[i]);
      g[i] = p.nesterov ? __fadd_rn(g[i], __fmul_rn(m[q][i], beta)) : m[q][i];
      ss = fmaf(g[i], g[i], ss);
    }
    store_unit<T>(out_row<T>(s, c, u[q]), vec, u[q], g);
    if (DENSE) store_unit<T>(static_cast<T*>(s.codes) + code_at(s, c, u[q]), vec, u[q], m[q]);
  }
  if (!DENSE) write_units<DENSE ? kStateInt8 : F, STOCHASTIC>(s, c, vec, u, key, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += red[i];
    p.partials[blockIdx.x] = t;
  }
}

// The norms of one momentum launch: CTA j adds matrix j's partial sums in a fixed order.
__global__ void __launch_bounds__(THREADS) state_norm_kernel(const __grid_constant__ StateParams p) {
  __shared__ float red[THREADS / 32];
  int at = static_cast<int>(blockIdx.x), seg = 0;
  while (at >= p.seg[seg].count) at -= p.seg[seg++].count;
  const StateSeg& s = p.seg[seg];
  const float* part = p.partials + s.cta_begin + at * s.unit_ctas;
  float t = 0.0f;
  for (int i = threadIdx.x; i < s.unit_ctas; i += THREADS) t += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    float n = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) n += red[i];
    p.norms[s.caller_idx + at] = sqrtf(n);
  }
}

template <typename T, int F>
cudaError_t quantize(const StateParams& p, cudaStream_t s) {
  if (p.stochastic)
    state_quantize_kernel<T, F, true><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  else
    state_quantize_kernel<T, F, false><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t quantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  return f == kStateInt8 ? quantize<T, kStateInt8>(p, s) : quantize<T, kStateE4M3>(p, s);
}
template <typename T>
cudaError_t dequantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  if (f == kStateInt8)
    state_dequantize_kernel<T, kStateInt8><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  else
    state_dequantize_kernel<T, kStateE4M3><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int F>
cudaError_t momentum(const StateParams& p, cudaStream_t s) {
  if (F != kStateDense && p.stochastic)
    state_momentum_kernel<T, F, true><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  else
    state_momentum_kernel<T, F, false><<<static_cast<unsigned>(p.total), THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t momentum(const StateParams& p, StateFormat f, cudaStream_t s) {
  if (f == kStateInt8) return momentum<T, kStateInt8>(p, s);
  if (f == kStateE4M3) return momentum<T, kStateE4M3>(p, s);
  return momentum<T, kStateDense>(p, s);
}

}  // namespace

cudaError_t launch_state_quantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  const int t = p.seg[0].in_type;
  if (t == kViewF32) return quantize<float>(p, f, s);
  if (t == kViewBF16) return quantize<__nv_bfloat16>(p, f, s);
  return quantize<__half>(p, f, s);
}

cudaError_t launch_state_dequantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  const int t = p.seg[0].out_type;
  if (t == kViewF32) return dequantize<float>(p, f, s);
  if (t == kViewBF16) return dequantize<__nv_bfloat16>(p, f, s);
  return dequantize<__half>(p, f, s);
}

cudaError_t launch_state_momentum(const StateParams& p, StateFormat f, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  cudaError_t e = p.seg[0].in_type == kViewF32 ? momentum<float>(p, f, s) : momentum<__nv_bfloat16>(p, f, s);
  if (e != cudaSuccess || p.norms == nullptr) return e;
  int mats = 0;
  for (int i = 0; i < p.nseg; ++i) mats += p.seg[i].count;
  state_norm_kernel<<<mats, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace muon
