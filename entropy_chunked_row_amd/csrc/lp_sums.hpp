// Softmax sums of a row without the entropy's term, and the order of logits:
// shared by the kernels that choose from a row and that distil from one.
#pragma once

#include "lp_device.hpp"

namespace lp {

// RowStat without `a`: m the largest value (-inf: none yet), s the sum of 2^t
// over exponents t relative to m c, near and far as there; values whose m c leaves
// fp32 are far ones too.
struct SumStat {
  float m, s;
};

struct LaneSum : SumStat {
  float nmc = 0.f;  // -RN(m c); 0 while m is -inf
};

__device__ __forceinline__ LaneSum sum_none() { return LaneSum{{neg_inf(), 0.f}}; }

// s 2^d, d <= 0.  A sum relative to a value that a kernel took early may be as large as
// kMostSum, so that something is left of it where 2^d alone is below fp32: two halves.
__device__ __forceinline__ float sum_scaled(float s, float d) {
  const float r = fast_exp2(0.5f * d);
  return s * r * r;
}

// The largest sum of a workgroup or wave relative to such a value that is kept: 2^27 of
// them still add up.
constexpr float kMostSum = 1.2676506e30f;  // 2^100

// Folds N values whose largest is vm into the state.  -inf weighs 0; a NaN stays
// a NaN in s.
template <int N, int CH>
__device__ __forceinline__ void sum_push(LaneSum& st, const float* x, float vm, float c) {
  if (vm > st.m) {
    st.s = sum_scaled(st.s, stat_shift(st.m, vm, c));
    st.m = vm;
    st.nmc = -(vm * c);
  }
  auto fold = [&](auto exponent) {
#pragma unroll
    for (int g = 0; g < N; g += CH) {
      float ps = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) ps += fast_exp2(exponent(x[g + k]));
      st.s += ps;
    }
  };
  if (is_near(st.nmc))
    fold([&](float v) { return fmaf(v, c, st.nmc); });
  else
    fold([&](float v) { return (v - st.m) * c; });
}

__device__ __forceinline__ void sum_push1(LaneSum& st, float x, float c) { sum_push<1, 1>(st, &x, x, c); }

// The whole of N states of N neighbouring lanes, in each of them.
template <int N>
__device__ __forceinline__ SumStat sum_merge(SumStat st, float c) {
  const float m = lanes_reduce<N>(st.m, [](float x, float y) { return fmaxf(x, y); });
  return SumStat{m, lanes_reduce<N>(sum_scaled(st.s, stat_shift(st.m, m, c)), [](float x, float y) { return x + y; })};
}

__device__ __forceinline__ SumStat sum_add(SumStat x, SumStat y, float c) {
  const float m = fmaxf(x.m, y.m);
  return SumStat{m, sum_scaled(x.s, stat_shift(x.m, m, c)) + sum_scaled(y.s, stat_shift(y.m, m, c))};
}

// The workgroup's whole state, in every thread; sm holds NT / 64 states.  Ends
// with no barrier: sm may be written again only after one.
template <int NT>
__device__ __forceinline__ SumStat sum_block(SumStat st, float c, SumStat* sm) {
  constexpr int W = NT / 64;
  st = sum_merge<64>(st, c);
  if (W == 1) return st;
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = st;
  __syncthreads();
  return sum_merge<W>(sm[threadIdx.x & (W - 1)], c);
}

// log-sum-exp of z / tau less m / tau, natural, in fp64 (scores of different rows are
// compared and differences of nearly equal ones formed: fp32 would leave a few 2^-24 of
// their magnitude).  m c carries the rounding of c and of the product; both are
// taken out again, so that only the exponents' own roundings remain.  Whatever is taken
// from a log-sum or added to one is taken relative to m first: in rows of finite masks (m of
// 1e38) fp64 holds nothing of the logs beside m itself.
__device__ __forceinline__ double sum_log(SumStat st, float c) {
  if (st.s == 0.f) return -__builtin_inf();
  const float mc = st.m * c;
  const double l2s = log2(static_cast<double>(st.s));
  const double off = is_near(mc) ? static_cast<double>(st.m) * c - static_cast<double>(mc) : 0.0;
  return (l2s - off) * 0.69314718055994530942;
}

// (x - m) / tau
__device__ __forceinline__ double below(float x, float m, double inv_tau) {
  return (static_cast<double>(x) - static_cast<double>(m)) * inv_tau;
}

// The log-sum-exp itself, and a part's less the whole row's, from states and their sum_log.
__device__ __forceinline__ double sum_lse(SumStat st, double log_sum, double inv_tau) {
  return st.s == 0.f ? -__builtin_inf() : static_cast<double>(st.m) * inv_tau + log_sum;
}
__device__ __forceinline__ double sum_gap(SumStat part, double part_log, SumStat whole, double whole_log, double inv_tau) {
  return part.s == 0.f ? -__builtin_inf() : below(part.m, whole.m, inv_tau) + (part_log - whole_log);
}

// Whole numbers in the order of the values (-0 = 0); NaN of either sign lies outside the infinities.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

// Which piece of work a workgroup takes: a workgroup runs on XCD blockIdx.x % 8,
// and rows that a mask leaves out often come in a period of 8 (rows 0 .. 3 of every 16:
// half the XCDs would have twice the work of the others, 335 us for 290 on 8192 x
// 151936).  So each eight neighbours go round by another offset.
__device__ __forceinline__ unsigned spread_block() {
  const unsigned b = blockIdx.x;
  return (b | 7u) < gridDim.x ? (b & ~7u) | ((b + (b >> 3) + (b >> 6)) & 7u) : b;
}

// A row's vector v of n columns: whole, or what is left at the end with -inf
// behind it.  Rows may start at any element.
template <class Tr>
__device__ __forceinline__ u32x4 row_vector(const char* xp, int v, int n) {
  constexpr int P = Tr::kPerVec;
  if ((v + 1) * P <= n) return load_vec(xp + static_cast<size_t>(v) * 16);
  float x[P];
#pragma unroll
  for (int k = 0; k < P; ++k) x[k] = v * P + k < n ? Tr::load1(xp, v * P + k) : neg_inf();
  return Tr::pack(x);
}

template <class Tr>
__device__ __forceinline__ u32x4 no_vector() {
  const uint32_t w = Tr::kBytes == 2 ? Tr::neg_inf_bits() * 0x10001u : Tr::neg_inf_bits();
  return u32x4{w, w, w, w};
}

__device__ __forceinline__ float largest3(float a, float b, float c) {
#if defined(__HIP_DEVICE_COMPILE__)
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
#else
  return fmaxf(fmaxf(a, b), c);
#endif
}

// NaN are passed over.  Three at a time by hand: the compiler first brings each
// value of a pair to canonical form, which widened logits already have.
template <int N>
__device__ __forceinline__ float largest_of(const float* x) {
  float m = x[0];
  int k = 1;
#pragma unroll
  for (; k + 2 <= N; k += 2) m = largest3(m, x[k], x[k + 1]);
  if (k < N) m = fmaxf(m, x[k]);
  return m;
}

}  // namespace lp
