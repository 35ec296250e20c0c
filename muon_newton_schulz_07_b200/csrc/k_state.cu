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
// for the momentum) or, with stochastic rounding, by the integer and logic pipe.  Measured with 226 M bf16
// values: read back 101 us (6.8 TB/s, the rate of a copy), written as e4m3 with stochastic rounding 193 us,
// momentum on int8 with it 312 us (4.4 TB/s); to nearest, 57 M values as int8 38 us (4.5 TB/s).  A unit is one block of one row, 16 lanes of 8 values; consecutive units are
// consecutive in memory, so a CTA of 64 units streams up to 8192 contiguous values whatever the
// row length, and a thread has the loads of all four of its units in flight before it computes.
// Three or four CTAs an SM (the launch bounds): the loads of one hide behind the arithmetic of the others (30 of
// 1001 x 1001 bf16, value by value: momentum on int8 113 us unbounded, 89 with three).  Momentum on fp32 rows of whole
// blocks is not held to a number (one CTA fewer fits; 24 of 1536 x 1536 as int8, to nearest, 116 us a call with the norms).
// Rows that are not whole blocks back to back interleave the 16 lanes instead, four values each where
// rows are multiples of 4 and aligned so, else one, which keeps the accesses of a half-warp contiguous.
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
// Places 2 pair and 2 pair + 1 of a matrix share the 32 bits mixed(pair_counter(key, pair)), the lower half first.  (Of
// a matrix of more than 2^33 values, those 2^33 apart have the same bits.)
__device__ __forceinline__ uint32_t pair_counter(uint32_t key, unsigned long long pair) {
  return static_cast<uint32_t>(pair) + key;
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
    // the 16 bits below the leading one of 2^7 (int8) or 2^-16 (e4m3): taking that off leaves u, or 2^-23 u
    constexpr uint32_t one = F == kStateInt8 ? 0x43000000u : 0x37800000u;
    const uint32_t bits = STOCHASTIC ? __byte_perm(r[i >> 1], one, (i & 1) ? 0x7632 : 0x7610) : one;
    const float u = STOCHASTIC ? __fsub_rn(__uint_as_float(bits), __uint_as_float(one)) : 0.0f;
    if (F == kStateInt8) {
      if (STOCHASTIC)
        b[i] = __float_as_uint(__fadd_rd(fminf(fmaxf(__fadd_rn(y[i], u), -127.0f), 127.0f), 12582912.0f));
      else
        b[i] = __float_as_uint(__fadd_rn(y[i], 12582912.0f));  // 1.5 * 2^23: negative values too
    } else if (STOCHASTIC) {
      // The spacing at |y| is an eighth of its binade, and of 2^-6 below that.  |y| + u spacing is exact
      // (or passes into the next binade, whose first code it then is), and adding 2^23 spacings,
      // rounded down, and taking them off again leaves whole spacings.
      const uint32_t bits_y = __float_as_uint(y[i]);
      const float whole = __uint_as_float(max(bits_y & 0x7F800000u, 0x3C800000u)) * 0x1p20f;  // 2^23 spacings
      const float z = __fmaf_rn(u, whole, fabsf(y[i]));
      const float v = __fsub_rn(__fadd_rd(z, whole), whole);
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
__device__ __forceinline__ int unit_lane() { return threadIdx.x % LANES; }
constexpr uint32_t UNITS = THREADS / LANES;  // of a pass

// Where the units of this thread's 16 lanes are, one a pass.  LINEAR: rows are whole blocks and every
// side is contiguous, so unit i of a matrix is its values 128 i .. everywhere, and a pass is a constant further
// on: one address a side, computed once (computed for each pass they were a sixth of the instructions,
// which bound the kernels that round stochastically).  Otherwise the row and column of a unit: one division, then
// steps.
template <bool LINEAR>
struct Sites {
  uint32_t unit0, total;                        // LINEAR
  long long code0, scale0;                      // LINEAR, of pass 0
  int row[LINEAR ? 1 : PASSES], col[LINEAR ? 1 : PASSES], vals[LINEAR ? 1 : PASSES];
  const StateSeg& s;
  const Cta& c;
  __device__ __forceinline__ Sites(const StateSeg& seg, const Cta& cta) : s(seg), c(cta) {
    unit0 = cta.first + threadIdx.x / LANES;  // below 2^31 + 64
    if (LINEAR) {
      total = static_cast<uint32_t>(s.rows) * s.blocks;
      scale0 = static_cast<long long>(c.e) * total + unit0;
      code0 = scale0 * kStateBlock;  // (rows are whole blocks)
      return;
    }
    uint32_t r = unit0 / static_cast<uint32_t>(s.blocks), block = unit0 - r * s.blocks;
    const uint32_t rows = UNITS / static_cast<uint32_t>(s.blocks), blocks = UNITS - rows * s.blocks;
#pragma unroll
    for (int q = 0; q < (LINEAR ? 0 : PASSES); ++q) {
      row[LINEAR ? 0 : q] = static_cast<int>(r);
      col[LINEAR ? 0 : q] = static_cast<int>(block) * kStateBlock;
      vals[LINEAR ? 0 : q] = r < static_cast<uint32_t>(s.rows) ? min(kStateBlock, s.cols - static_cast<int>(block) * kStateBlock) : 0;
      r += rows;
      block += blocks;
      if (block >= static_cast<uint32_t>(s.blocks)) {
        block -= s.blocks;
        ++r;
      }
    }
  }
  static constexpr int kPass = UNITS * kStateBlock;  // LINEAR: values from one pass to the next
  // values of the unit that exist (0: beyond the matrix)
  __device__ __forceinline__ int have(int q) const {
    return LINEAR ? (unit0 + q * UNITS < total ? kStateBlock : 0) : vals[LINEAR ? 0 : q];
  }
  // of the unit's first value: within the matrix, in the codes of the stack, and its scale
  __device__ __forceinline__ unsigned long long place_of(int q) const {
    return LINEAR ? static_cast<unsigned long long>(unit0) * kStateBlock + q * kPass
                  : static_cast<unsigned long long>(row[LINEAR ? 0 : q]) * s.cols + col[LINEAR ? 0 : q];
  }
  __device__ __forceinline__ long long code_at(int q) const {
    return LINEAR ? code0 + q * kPass : static_cast<long long>(c.e) * s.rows * s.cols + place_of(q);
  }
  __device__ __forceinline__ long long scale_at(int q) const {
    return LINEAR ? scale0 + q * static_cast<int>(UNITS)
                  : static_cast<long long>(c.e) * s.rows * s.blocks +
                        (static_cast<long long>(row[LINEAR ? 0 : q]) * s.blocks + col[LINEAR ? 0 : q] / kStateBlock);
  }
  __device__ __forceinline__ long long value_at(int q, long long ld, long long bs) const {
    return LINEAR ? c.e * bs + static_cast<long long>(unit0) * kStateBlock + q * kPass
                  : c.e * bs + row[LINEAR ? 0 : q] * ld + col[LINEAR ? 0 : q];
  }
  template <typename T>
  __device__ __forceinline__ const T* in(int q) const {
    return static_cast<const T*>(s.in) + value_at(q, s.in_ld, s.in_bs);
  }
  template <typename T>
  __device__ __forceinline__ T* out(int q) const {
    return static_cast<T*>(s.out) + value_at(q, s.out_ld, s.out_bs);
  }
};
// Value i of a lane sits at this place of the unit: eight neighbours (LINEAR), two runs of four (vec), or
// single values.
__device__ __forceinline__ int run(int lane, int h) { return (lane + LANES * h) * 4; }
__device__ __forceinline__ int single(int lane, int i) { return lane + LANES * i; }

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
  __device__ __forceinline__ void load4(int h, const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
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
  __device__ __forceinline__ void load4(int h, const T* p) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p));
    w[2 * h] = q.x; w[2 * h + 1] = q.y;
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

template <bool LINEAR, typename T>
__device__ __forceinline__ void load_values(const T* base, bool vec, int have, Eight<T>& x) {
  const int lane = unit_lane();
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(x) / 4); ++i) reinterpret_cast<uint32_t*>(&x)[i] = 0;
  if (LINEAR) {
    if (have > 0) x.load(base + lane * 8);
    return;
  }
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (run(lane, h) < have) x.load4(h, base + run(lane, h));  // rows are multiples of 4: all or nothing
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = single(lane, i);
      if (at < have) x.set(i, base + at);
    }
  }
}

template <bool LINEAR, typename T>
__device__ __forceinline__ void store_values(T* base, bool vec, int have, const float (&x)[8]) {
  const int lane = unit_lane();
  if (LINEAR) {
    if (lane * 8 < have) store_eight(base, TypeOf<T>::id, lane * 8, 8, x);
  } else if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* v = x + 4 * h;
      if (run(lane, h) >= have) continue;
      if (TypeOf<T>::id == kViewF32) {
        *reinterpret_cast<float4*>(base + run(lane, h)) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        alignas(8) T q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) store_one(q, TypeOf<T>::id, i, v[i]);
        *reinterpret_cast<uint2*>(base + run(lane, h)) = *reinterpret_cast<const uint2*>(q);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = single(lane, i);
      if (at < have) store_one(base, TypeOf<T>::id, at, x[i]);
    }
  }
}

// Write the four units of these 16 lanes.  The largest magnitudes of all four go through one
// exchange: each step halves the units a lane still holds, so that quarter q of the lanes ends with
// unit q's, divides once, and hands factor and scale back.
template <int F, bool STOCHASTIC, bool LINEAR>
__device__ __forceinline__ void write_units(const Sites<LINEAR>& at, bool vec, uint32_t key, float (&x)[PASSES][8]) {
  const StateSeg& s = at.s;
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
    const int have = at.have(q);
    if (lane == q * 4 && have > 0) s.scales[at.scale_at(q)] = my_scale;
    uint8_t* codes = static_cast<uint8_t*>(s.codes) + at.code_at(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[q][i] = __fmul_rn(x[q][i], mul);
    if (!fine) {  // rare: not finite
#pragma unroll
      for (int i = 0; i < 8; ++i) x[q][i] = 0.0f;
    }
    uint32_t r[4] = {0, 0, 0, 0};
    if (STOCHASTIC) {
      const unsigned long long first = at.place_of(q);
      if (LINEAR) {  // eight neighbours from an even place: four pairs
        const uint32_t counter = pair_counter(key, (at.place_of(0) + lane * 8) / 2) + q * (Sites<LINEAR>::kPass / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = mixed(counter + i);
      } else if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t counter = pair_counter(key, (first + run(lane, h)) / 2);  // (even)
          r[2 * h] = mixed(counter);
          r[2 * h + 1] = mixed(counter + 1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned long long here = first + single(lane, i);
          const uint32_t h = mixed(pair_counter(key, here >> 1)) >> (16 * (here & 1)) & 0xFFFFu;
          r[i >> 1] |= h << (16 * (i & 1));
        }
      }
    }
    const uint32_t r0[2] = {r[0], r[1]}, r1[2] = {r[2], r[3]};
    const uint32_t lo = encode4<F, STOCHASTIC>(x[q], r0), hi = encode4<F, STOCHASTIC>(x[q] + 4, r1);
    if (LINEAR) {
      if (lane * 8 < have) __stcs(reinterpret_cast<uint2*>(codes + lane * 8), make_uint2(lo, hi));
    } else if (vec) {
      if (run(lane, 0) < have) __stcs(reinterpret_cast<uint32_t*>(codes + run(lane, 0)), lo);
      if (run(lane, 1) < have) __stcs(reinterpret_cast<uint32_t*>(codes + run(lane, 1)), hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int to = single(lane, i);
        if (to < have) codes[to] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
}

// The codes of a lane's eight values, as loaded.
struct Codes {
  uint32_t w[2];
  float scale;
};
template <bool LINEAR>
__device__ __forceinline__ void load_codes(const Sites<LINEAR>& at, int q, bool vec, Codes& c) {
  const int lane = unit_lane(), have = at.have(q);
  const uint8_t* p = static_cast<const uint8_t*>(at.s.codes) + at.code_at(q);
  c.w[0] = c.w[1] = 0;
  c.scale = have > 0 ? at.s.scales[at.scale_at(q)] : 0.0f;
  if (LINEAR) {
    if (have > 0) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p + lane * 8));
      c.w[0] = v.x;
      c.w[1] = v.y;
    }
  } else if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (run(lane, h) < have) c.w[h] = __ldcs(reinterpret_cast<const uint32_t*>(p + run(lane, h)));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int to = single(lane, i);
      if (to < have) c.w[i >> 2] |= static_cast<uint32_t>(p[to]) << (8 * (i & 3));
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

template <typename T, int F, bool STOCHASTIC, bool LINEAR>
__global__ void __launch_bounds__(THREADS, 4) state_quantize_kernel(const __grid_constant__ StateParams p) {
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  const uint32_t key = STOCHASTIC ? matrix_key(p.seed, static_cast<uint32_t>(s.mat_begin + c.e)) : 0u;
  const Sites<LINEAR> at(s, c);
  Eight<T> raw[PASSES];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) load_values<LINEAR, T>(at.template in<T>(q), vec, at.have(q), raw[q]);
  float x[PASSES][8];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) raw[q].widen(x[q]);
  write_units<F, STOCHASTIC, LINEAR>(at, vec, key, x);
}

template <typename T, int F, bool LINEAR>
__global__ void __launch_bounds__(THREADS, 4) state_dequantize_kernel(const __grid_constant__ StateParams p) {
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  const Sites<LINEAR> at(s, c);
  Codes raw[PASSES];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) load_codes<LINEAR>(at, q, vec, raw[q]);
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    float x[8];
    read_codes<F>(raw[q], x);
    store_values<LINEAR, T>(at.template out<T>(q), vec, at.have(q), x);
  }
}

// Momentum and Nesterov blend of one CTA's units; F = kStateDense keeps m in T.  PASS says what a
// launch does with u and m1 (see StatePass).
template <typename T, int F, bool STOCHASTIC, bool LINEAR, int PASS>
__global__ void __launch_bounds__(THREADS, !LINEAR || sizeof(T) == 2 ? 3 : 1)
    state_momentum_kernel(const __grid_constant__ StateParams p) {
  constexpr bool DENSE = F == kStateDense;
  __shared__ double red[THREADS / 32];
  __shared__ bool last;
  const Cta c = find(p);
  const StateSeg& s = p.seg[c.seg];
  const bool vec = s.vec != 0;
  const uint32_t key = STOCHASTIC ? matrix_key(p.seed, static_cast<uint32_t>(s.mat_begin + c.e)) : 0u;
  const float mul = PASS == kPassStep ? p.factors[s.caller_idx + c.e] : 1.0f;
  const float beta = p.beta, rest = __fsub_rn(1.0f, p.beta);
  const Sites<LINEAR> at(s, c);
  Eight<T> raw[PASSES];
  Codes codes[DENSE ? 1 : PASSES];
  Eight<T> dense[DENSE ? PASSES : 1];
  auto load = [&](int q, Eight<T>& g, Codes& m8, Eight<T>& m) {
    load_values<LINEAR, T>(at.template in<T>(q), vec, at.have(q), g);
    if (DENSE)
      load_values<LINEAR, T>(static_cast<const T*>(s.codes) + at.code_at(q), vec, at.have(q), m);
    else
      load_codes<LINEAR>(at, q, vec, m8);
  };
  // m1 and u of eight values
  auto moments = [&](const Eight<T>& g8, const Codes& m8, const Eight<T>& m, float (&m1)[8], float (&u)[8]) {
    g8.widen(u);
    if (DENSE)
      m.widen(m1);
    else
      read_codes<DENSE ? kStateInt8 : F>(m8, m1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = __fmul_rn(u[i], rest);
      m1[i] = __fadd_rn(__fmul_rn(m1[i], beta), u[i]);
      if (p.nesterov)
        u[i] = __fadd_rn(u[i], __fmul_rn(m1[i], beta));
      else
        u[i] = m1[i];
    }
  };
#pragma unroll
  for (int q = 0; q < PASSES; ++q) load(q, raw[q], codes[DENSE ? 0 : q], dense[DENSE ? q : 0]);
  float sum = 0.0f;
  float m[PASSES][8];
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    float u[8];
    moments(raw[q], codes[DENSE ? 0 : q], dense[DENSE ? q : 0], m[q], u);
    if (PASS != kPassStep) sum += at.have(q) > 0 ? squares8(u) : 0.0f;
    if (PASS == kPassStep) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] *= mul;
      store_values<LINEAR, __half>(at.template out<__half>(q), vec, at.have(q), u);
    }
    if (PASS == kPassMomentum) store_values<LINEAR, T>(at.template out<T>(q), vec, at.have(q), u);
    if (DENSE && PASS != kPassNorm) store_values<LINEAR, T>(static_cast<T*>(s.codes) + at.code_at(q), vec, at.have(q), m[q]);
  }
  if (!DENSE && PASS != kPassNorm) write_units<DENSE ? kStateInt8 : F, STOCHASTIC, LINEAR>(at, vec, key, m);
  if (PASS == kPassStep) return;
  // The values of an unusual sum come from memory again: u as this thread stored it (held until now, in registers or in
  // shared memory, u costs every call 2 to 10 %), or what it is made of where nothing has been written.
  const Squares squares(sum, at.have(0) > 0, [&](auto add) {
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      Eight<T> g8, m8;
      Codes c8;
      float m1[8], u[8];
      if (PASS == kPassMomentum) {
        load_values<LINEAR, T>(at.template out<T>(q), vec, at.have(q), g8);
        g8.widen(u);
      } else {
        load(q, g8, c8, m8);
        moments(g8, c8, m8, m1, u);
      }
      add(u);  // (values beyond the matrix: zeros)
    }
  });
  const double ss = block_sum<THREADS>(squares, red);
  if (!last_to_leave(p.partials + blockIdx.x, ss, p.arrivals + s.caller_idx + c.e, s.unit_ctas, &last)) return;
  const double* part = p.partials + s.cta_begin + c.e * s.unit_ctas;
  const double total = block_sum<THREADS>(sum_parts<THREADS>(part, s.unit_ctas), red);
  if (threadIdx.x == 0) {
    p.norms[s.caller_idx + c.e] = norm_of(total);
    p.factors[s.caller_idx + c.e] = normaliser(total, p.eps);
  }
}

template <typename T, int F, bool LINEAR>
cudaError_t quantize(const StateParams& p, cudaStream_t s) {
  if (p.stochastic)
    state_quantize_kernel<T, F, true, LINEAR><<<p.total, THREADS, 0, s>>>(p);
  else
    state_quantize_kernel<T, F, false, LINEAR><<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int F>
cudaError_t quantize(const StateParams& p, cudaStream_t s) {
  return p.linear ? quantize<T, F, true>(p, s) : quantize<T, F, false>(p, s);
}
template <typename T>
cudaError_t quantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  return f == kStateInt8 ? quantize<T, kStateInt8>(p, s) : quantize<T, kStateE4M3>(p, s);
}
template <typename T, int F>
cudaError_t dequantize(const StateParams& p, cudaStream_t s) {
  if (p.linear)
    state_dequantize_kernel<T, F, true><<<p.total, THREADS, 0, s>>>(p);
  else
    state_dequantize_kernel<T, F, false><<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t dequantize(const StateParams& p, StateFormat f, cudaStream_t s) {
  return f == kStateInt8 ? dequantize<T, kStateInt8>(p, s) : dequantize<T, kStateE4M3>(p, s);
}
template <typename T, int F, bool LINEAR>
cudaError_t momentum(const StateParams& p, StatePass pass, cudaStream_t s) {
  constexpr bool CODES = F != kStateDense;  // (a dense momentum has steps only)
  if (pass == kPassNorm)
    state_momentum_kernel<T, F, false, LINEAR, kPassNorm><<<p.total, THREADS, 0, s>>>(p);
  else if (pass == kPassStep && !(CODES && p.stochastic))
    state_momentum_kernel<T, F, false, LINEAR, kPassStep><<<p.total, THREADS, 0, s>>>(p);
  else if constexpr (!CODES)
    return cudaErrorInvalidValue;
  else if (pass == kPassStep)
    state_momentum_kernel<T, F, true, LINEAR, kPassStep><<<p.total, THREADS, 0, s>>>(p);
  else if (p.stochastic)
    state_momentum_kernel<T, F, true, LINEAR, kPassMomentum><<<p.total, THREADS, 0, s>>>(p);
  else
    state_momentum_kernel<T, F, false, LINEAR, kPassMomentum><<<p.total, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int F>
cudaError_t momentum(const StateParams& p, StatePass pass, cudaStream_t s) {
  return p.linear ? momentum<T, F, true>(p, pass, s) : momentum<T, F, false>(p, pass, s);
}
template <typename T>
cudaError_t momentum(const StateParams& p, StateFormat f, StatePass pass, cudaStream_t s) {
  if (f == kStateInt8) return momentum<T, kStateInt8>(p, pass, s);
  if (f == kStateE4M3) return momentum<T, kStateE4M3>(p, pass, s);
  return momentum<T, kStateDense>(p, pass, s);
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

cudaError_t launch_state_momentum(const StateParams& p, StateFormat f, StatePass pass, cudaStream_t s) {
  if (p.total <= 0) return cudaSuccess;
  return p.seg[0].in_type == kViewF32 ? momentum<float>(p, f, pass, s) : momentum<__nv_bfloat16>(p, f, pass, s);
}

}  // namespace muon
