// Device-side building blocks shared by the row-reduction kernels and the
// fused LM-head epilogues.
//
// Row state.  For one row (or any subset of its vocabulary) the kernels keep
//   mc = RN(max_z * c)            reference exponent, log2 units
//   s  = sum_j 2^{t_j}            t_j = RN(z_j * c - mc)
//   a  = sum_j 2^{t_j} * t_j
// with c = log2(e) / tau (tau = 1 when the temperature does not apply).  Then
//   log-sum-exp of z / tau = ln2 * (mc + log2 s)
//   log p(y)               = ln2 * (t_y - log2 s)
//   entropy                = ln2 * (log2 s - a / s)
// Two states over disjoint parts of a row merge exactly (up to rounding) by
// moving both to the larger reference exponent.  Every sum is fp32; the
// model-precision values are only ever widened, never accumulated in place.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace lp {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kLog2e = 1.44269504088896340736f;
// Reference exponent of a state that has seen nothing.  Finite on purpose: a
// -inf element then gives t = -inf (probability 0) instead of NaN.
constexpr float kNegBig = -3.402823466e38f;

struct Stat {
  float mc, s, a;
};

__device__ __forceinline__ Stat stat_empty() { return Stat{kNegBig, 0.f, 0.f}; }

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Merge two partial states of the same row.  A side that has seen nothing
// (s == 0) adds nothing; a NaN side makes the whole NaN.
__device__ __forceinline__ Stat stat_merge(Stat x, Stat y) {
  const float mc = fmaxf(x.mc, y.mc);
  float s = 0.f, a = 0.f;
  if (x.s != 0.f) {
    const float d = x.mc - mc;
    const float r = fast_exp2(d);
    s += x.s * r;
    a += (x.a + x.s * d) * r;
  }
  if (y.s != 0.f) {
    const float d = y.mc - mc;
    const float r = fast_exp2(d);
    s += y.s * r;
    a += (y.a + y.s * d) * r;
  }
  return Stat{mc, s, a};
}

// Move a state to a new, larger reference exponent nmc.
__device__ __forceinline__ void stat_rebase(Stat& st, float nmc) {
  if (st.s != 0.f) {
    const float d = st.mc - nmc;
    const float r = fast_exp2(d);
    st.a = (st.a + st.s * d) * r;
    st.s *= r;
  }
  st.mc = nmc;
}

// Fold N widened values into the state: one max test, then CH-long partial
// sums (short chains keep fp32 rounding low).  GUARD clamps t in `a`, so that a
// -inf value contributes 0 * finite instead of 0 * -inf (a NaN stays in s).
template <bool GUARD, int N, int CH>
__device__ __forceinline__ void stat_push(Stat& st, const float* x, float c) {
  float vm = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) vm = fmaxf(vm, x[k]);
  const float vmc = vm * c;
  if (vmc > st.mc) stat_rebase(st, vmc);
  const float nmc = -st.mc;
#pragma unroll
  for (int g = 0; g < N; g += CH) {
    float ps = 0.f, pa = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const float t = fmaf(x[g + k], c, nmc);
      const float e = fast_exp2(t);
      ps += e;
      pa = fmaf(e, GUARD ? fmaxf(t, kNegBig) : t, pa);
    }
    st.s += ps;
    st.a += pa;
  }
}

// Butterfly over a wave64: every lane ends with the merge of all 64 lanes.
__device__ __forceinline__ Stat stat_wave_allreduce(Stat st) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    Stat o;
    o.mc = __shfl_xor(st.mc, off, 64);
    o.s = __shfl_xor(st.s, off, 64);
    o.a = __shfl_xor(st.a, off, 64);
    st = stat_merge(st, o);
  }
  return st;
}

// Block-wide merge; every thread returns the same state (fixed order, so the
// result is bitwise reproducible).  `sm` holds NT/64 states.
template <int NT>
__device__ __forceinline__ Stat stat_block_allreduce(Stat st, Stat* sm) {
  constexpr int NW = NT / 64;
  st = stat_wave_allreduce(st);
  if (NW == 1) return st;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) sm[w] = st;
  __syncthreads();
  Stat r = sm[0];
#pragma unroll
  for (int k = 1; k < NW; ++k) r = stat_merge(r, sm[k]);
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------------------
// states of rows that may hold finite values of any size
// ---------------------------------------------------------------------------

constexpr float kNoWeight = -1024.f;  // exponents below weigh exactly 0 in fp32

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Softmax state of some of a row's columns under an exponent scale c: m their
// largest value that has weight (-inf: none yet), s = sum 2^t and a = sum 2^t t
// over exponents t relative to m c.  Where |m c| is below kFar ("near") they
// are t = fma(x, c, -RN(m c)), which rounds once.  The rounding of m c itself,
// which then stands in every t alike, is an exponent of its own: 1/2 at 2^24, 512
// at 1e10, 1e22 at 1e30.  Past kFar, where finite masks lie, t = (x - m) c
// instead, two operations but 0 at m whatever its size (in every column they
// would cost one instruction more of 13).
struct RowStat {
  float m, s, a;
};

constexpr float kFar = 16777216.f;
constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ bool is_near(float mc) { return fabsf(mc) < kFar; }

// What exponents relative to m0 gain when they are taken relative to m1.  The
// products are rounded here as they are in the exponents: no contraction.
__device__ __forceinline__ float reference_gap(float m0, float m1, float c) {
#pragma clang fp contract(off)
  const float r0 = m0 * c, r1 = m1 * c;
  float d = r0 - r1;
  if (!is_near(r0) || !is_near(r1)) {
    d = (m0 - m1) * c;
    // of near ones the rounding of their product is part
    if (is_near(r0)) d -= fmaf(m0, c, -r0);
    if (is_near(r1)) d += fmaf(m1, c, -r1);
  }
  return d;
}

// The same for m1 >= m0.  Below kNoWeight nothing is left of a weight; the
// bound keeps s times the shift finite, and takes an empty side (m0 = -inf) to
// nothing whatever m1.
__device__ __forceinline__ float stat_shift(float m0, float m1, float c) {
  return fmaxf(reference_gap(m0, m1, c), kNoWeight);
}

// A lane's state while it takes columns: with its reference exponent, which
// moves only when a larger value comes.
struct LaneStat : RowStat {
  float nmc = 0.f;  // -RN(m c); 0 while m is -inf, whose exponents are then -inf or NaN
};

__device__ __forceinline__ LaneStat stat_none() { return LaneStat{{neg_inf(), 0.f, 0.f}}; }

// Folds N values into the state.  They may be -inf, or so low that their
// product with c leaves fp32: those weigh 0 and add nothing to `a`.  A NaN
// stays a NaN in s and a.
template <int N, int CH>
__device__ __forceinline__ void stat_push_masked(LaneStat& st, const float* x, float c) {
  float vm = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) vm = fmaxf(vm, x[k]);
  if (vm > st.m && vm * c >= -kLargest) {
    const float d = stat_shift(st.m, vm, c), r = fast_exp2(d);
    st.a = (st.a + st.s * d) * r;
    st.s *= r;
    st.m = vm;
    st.nmc = -(vm * c);
  }
  auto fold = [&](auto exponent) {
#pragma unroll
    for (int g = 0; g < N; g += CH) {
      float ps = 0.f, pa = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float t = exponent(x[g + k]);
        const float e = fast_exp2(t);
        ps += e;
        pa = fmaf(e, fmaxf(t, kNoWeight), pa);
      }
      st.s += ps;
      st.a += pa;
    }
  };
  if (is_near(st.nmc))
    fold([&](float v) { return fmaf(v, c, st.nmc); });
  else
    fold([&](float v) { return (v - st.m) * c; });
}

// op over N neighbouring lanes (a power of two), in each of them: moves inside
// the registers (through LDS the twelve steps of a merge cost rows of 2344 to
// 16609 columns 3 % of their time).  Halves of 8 and 16 lanes may be mirrored,
// their lanes hold one value by then.
template <int N, class Op>
__device__ __forceinline__ float lanes_reduce(float x, Op op) {
  auto moved = [](float v, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  if constexpr (N >= 2) x = op(x, moved(x, std::integral_constant<int, 0xb1>{}));    // quad: 1 0 3 2
  if constexpr (N >= 4) x = op(x, moved(x, std::integral_constant<int, 0x4e>{}));    // quad: 2 3 0 1
  if constexpr (N >= 8) x = op(x, moved(x, std::integral_constant<int, 0x141>{}));   // mirrored in 8
  if constexpr (N >= 16) x = op(x, moved(x, std::integral_constant<int, 0x140>{}));  // mirrored in 16
  if constexpr (N >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if constexpr (N >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return x;
}

// The whole of N states of N neighbouring lanes, in each: all move to the
// largest value first, then sums and nothing else.  An empty state adds nothing
// and a NaN one wins.
template <int N>
__device__ __forceinline__ RowStat stat_merge(RowStat st, float c) {
  const float m = lanes_reduce<N>(st.m, [](float x, float y) { return fmaxf(x, y); });
  const float d = stat_shift(st.m, m, c), r = fast_exp2(d);
  auto sum = [](float x, float y) { return x + y; };
  return RowStat{m, lanes_reduce<N>(st.s * r, sum), lanes_reduce<N>((st.a + st.s * d) * r, sum)};
}

// As stat_merge, of two states in one lane.
__device__ __forceinline__ RowStat stat_add(RowStat x, RowStat y, float c) {
  const float m = fmaxf(x.m, y.m);
  const float dx = stat_shift(x.m, m, c), rx = fast_exp2(dx), dy = stat_shift(y.m, m, c), ry = fast_exp2(dy);
  return RowStat{m, x.s * rx + y.s * ry, (x.a + x.s * dx) * rx + (y.a + y.s * dy) * ry};
}

// ---------------------------------------------------------------------------
// element types: 16-byte vectors and exact widening to fp32
// ---------------------------------------------------------------------------

// Two fp32 values rounded to nearest even and packed (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, (f16x2_t{static_cast<_Float16>(lo), static_cast<_Float16>(hi)}));
}

struct Bf16 {
  static constexpr int kBytes = 2;
  static constexpr int kPerVec = 8;
  __device__ static __forceinline__ constexpr uint32_t neg_inf_bits() { return 0xff80u; }
  __device__ static __forceinline__ void unpack(u32x4 w, float* x) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
    x[4] = __uint_as_float(w.z << 16);
    x[5] = __uint_as_float(w.z & 0xffff0000u);
    x[6] = __uint_as_float(w.w << 16);
    x[7] = __uint_as_float(w.w & 0xffff0000u);
  }
  __device__ static __forceinline__ float load1(const char* p, int64_t i) {
    const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
  __device__ static __forceinline__ u32x4 pack(const float* x) {
    return u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  }
  __device__ static __forceinline__ void store1(char* p, int64_t i, float x) {
    reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
  }
};

__device__ __forceinline__ float half_bits_to_float(uint32_t b) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
}

struct Fp16 {
  static constexpr int kBytes = 2;
  static constexpr int kPerVec = 8;
  __device__ static __forceinline__ constexpr uint32_t neg_inf_bits() { return 0xfc00u; }
  __device__ static __forceinline__ void unpack(u32x4 w, float* x) {
    x[0] = half_bits_to_float(w.x & 0xffffu);
    x[1] = half_bits_to_float(w.x >> 16);
    x[2] = half_bits_to_float(w.y & 0xffffu);
    x[3] = half_bits_to_float(w.y >> 16);
    x[4] = half_bits_to_float(w.z & 0xffffu);
    x[5] = half_bits_to_float(w.z >> 16);
    x[6] = half_bits_to_float(w.w & 0xffffu);
    x[7] = half_bits_to_float(w.w >> 16);
  }
  __device__ static __forceinline__ float load1(const char* p, int64_t i) {
    return half_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]);
  }
  __device__ static __forceinline__ u32x4 pack(const float* x) {
    return u32x4{pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]), pack_f16x2(x[6], x[7])};
  }
  __device__ static __forceinline__ void store1(char* p, int64_t i, float x) {
    reinterpret_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
  }
};

struct Fp32 {
  static constexpr int kBytes = 4;
  static constexpr int kPerVec = 4;
  __device__ static __forceinline__ constexpr uint32_t neg_inf_bits() { return 0xff800000u; }
  __device__ static __forceinline__ void unpack(u32x4 w, float* x) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  __device__ static __forceinline__ float load1(const char* p, int64_t i) {
    return reinterpret_cast<const float*>(p)[i];
  }
  __device__ static __forceinline__ u32x4 pack(const float* x) {
    return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
  __device__ static __forceinline__ void store1(char* p, int64_t i, float x) { reinterpret_cast<float*>(p)[i] = x; }
};

// Dual (student u, teacher v) state for KL(teacher || student).
// Student u: (mcu, su).  Teacher v: (mcv, sv) and C = sum_j 2^{tv_j} (v_j - u_j)
// on the teacher's reference.  Then, with natural-log normalisers
// lse = ln2 (mc + log2 s):  KL = C / sv - (lse_v - lse_u).

struct KLState {
  float mcu, su, mcv, sv, C;
};

template <bool GUARD, int N, int CH>
__device__ __forceinline__ void kl_push(KLState& st, const float* xu, const float* xv, float c) {
  float mu = xu[0], mv = xv[0];
#pragma unroll
  for (int k = 1; k < N; ++k) {
    mu = fmaxf(mu, xu[k]);
    mv = fmaxf(mv, xv[k]);
  }
  const float muc = mu * c, mvc = mv * c;
  if (muc > st.mcu) {
    if (st.su != 0.f) st.su *= fast_exp2(st.mcu - muc);
    st.mcu = muc;
  }
  if (mvc > st.mcv) {
    if (st.sv != 0.f) {
      const float r = fast_exp2(st.mcv - mvc);
      st.sv *= r;
      st.C *= r;
    }
    st.mcv = mvc;
  }
  const float nu = -st.mcu, nv = -st.mcv;
#pragma unroll
  for (int g = 0; g < N; g += CH) {
    float pu = 0.f, pv = 0.f, pc = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const float eu = fast_exp2(fmaf(xu[g + k], c, nu));
      const float ev = fast_exp2(fmaf(xv[g + k], c, nv));
      pu += eu;
      pv += ev;
      const float d = xv[g + k] - xu[g + k];
      if (GUARD)
        pc += (ev > 0.f) ? ev * d : 0.f;
      else
        pc = fmaf(ev, d, pc);
    }
    st.su += pu;
    st.sv += pv;
    st.C += pc;
  }
}

__device__ __forceinline__ KLState kl_merge(KLState x, KLState y) {
  KLState r;
  r.mcu = fmaxf(x.mcu, y.mcu);
  r.su = 0.f;
  if (x.su != 0.f) r.su += x.su * fast_exp2(x.mcu - r.mcu);
  if (y.su != 0.f) r.su += y.su * fast_exp2(y.mcu - r.mcu);
  r.mcv = fmaxf(x.mcv, y.mcv);
  r.sv = 0.f;
  r.C = 0.f;
  if (x.sv != 0.f) {
    const float f = fast_exp2(x.mcv - r.mcv);
    r.sv += x.sv * f;
    r.C += x.C * f;
  }
  if (y.sv != 0.f) {
    const float f = fast_exp2(y.mcv - r.mcv);
    r.sv += y.sv * f;
    r.C += y.C * f;
  }
  return r;
}

// The dual state for rows that may hold finite values of any size: the largest
// values instead of their exponents (RowStat).
struct KLFar {
  float mu, su, mv, sv, C;
};

__device__ __forceinline__ float far_exponent(float x, float m, float c) {
  const float mc = m * c;
  if (mc < -kLargest) return x * c;  // none yet: -inf or NaN
  return is_near(mc) ? fmaf(x, c, -mc) : (x - m) * c;
}

// To the references of mu and mv, which are no smaller.  C may be infinite
// (the student gives no weight to what the teacher does); with no weight left
// of it, it is 0.
__device__ __forceinline__ void kl_far_move(KLFar& st, float mu, float mv, float c) {
  st.su *= fast_exp2(stat_shift(st.mu, mu, c));
  const float r = fast_exp2(stat_shift(st.mv, mv, c));
  st.sv *= r;
  st.C = r == 0.f ? 0.f : st.C * r;
  st.mu = mu;
  st.mv = mv;
}

__device__ __forceinline__ void kl_far_push(KLFar& st, float xu, float xv, float c) {
  const float mu = xu > st.mu && xu * c >= -kLargest ? xu : st.mu, mv = xv > st.mv && xv * c >= -kLargest ? xv : st.mv;
  if (mu != st.mu || mv != st.mv) kl_far_move(st, mu, mv, c);
  st.su += fast_exp2(far_exponent(xu, st.mu, c));
  const float ev = fast_exp2(far_exponent(xv, st.mv, c));
  st.sv += ev;
  if (ev > 0.f) st.C += ev * (xv - xu);
}

// The whole of N states of N neighbouring lanes, in each.
template <int N>
__device__ __forceinline__ KLFar kl_far_merge(KLFar st, float c) {
  auto most = [](float x, float y) { return fmaxf(x, y); };
  auto sum = [](float x, float y) { return x + y; };
  kl_far_move(st, lanes_reduce<N>(st.mu, most), lanes_reduce<N>(st.mv, most), c);
  return KLFar{st.mu, lanes_reduce<N>(st.su, sum), st.mv, lanes_reduce<N>(st.sv, sum), lanes_reduce<N>(st.C, sum)};
}

// 16 bytes of a row from any element on: one load, also off the 16-byte grid.
typedef unsigned int u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4 load_vec(const char* p) { return *reinterpret_cast<const u32x4_a2*>(p); }

// Split of a row of `n` elements at `p` into a scalar head (up to the first
// 16-byte boundary), whole 16-byte vectors, and a scalar tail.
template <class Tr>
struct RowSplit {
  int head;
  int nvec;
  int tail;
  __device__ __forceinline__ RowSplit(const char* p, int n) {
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
    int hd = mis ? (16 - mis) / Tr::kBytes : 0;
    head = hd < n ? hd : n;
    nvec = (n - head) / Tr::kPerVec;
    tail = n - head - nvec * Tr::kPerVec;
  }
};

}  // namespace lp
