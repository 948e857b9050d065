// Logits of few rows through an output head held in 4 bits with group scales:
//   out[t][v] = sum over groups g of s[v][g] * sum over k in g of x[t][k] (q[v][k] - 8)
// with q in 0..15, two to a byte (even column in the low half), s bf16, x
// bf16 or fp16 and every sum in fp32.
//
// The head's bytes are the floor: h / 2 + 2 h / group bytes a vocabulary row,
// read once for up to 64 rows of x.  Matrix cores do the products also for a
// single row of x, because the vector unit is what the unpacking needs:
//  * A nibble n becomes the 16-bit float 16 + n by one shift and one
//    and-or on two nibbles at a time (its bits go into the top of the mantissa of
//    16.0), exact in bf16 and fp16.
//  * sum x (q - 8) = sum x (16 + q) - 24 sum x.  The second sum does not depend on
//    v: one MFMA with a constant operand gives it to every row tile as
//    the start value of its accumulator.
//  * Nibbles s and s + 4 of a 32-bit word share a register, so x's columns take
//    the order 0 4 1 5 2 6 3 7 within each 8 (a permutation of the sum).
// A lane loads 16 bytes, 32 columns of a row; the 4 x 4 words of a row's four
// lanes are transposed in registers (v_permlane32_swap, v_permlane16_swap), so that one
// MFMA takes 32 neighbouring columns and stays inside one group, whose sum is
// then scaled in fp32.
#include <type_traits>

#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct XBf16 {
  static constexpr uint32_t kBase = 0x41804180u, kMask = 0x00780078u, kNeg24 = 0xc1c0c1c0u;
  static constexpr int kBit = 3;  // mantissa position of a nibble's bit 0
  __device__ static __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  }
};

struct XFp16 {
  static constexpr uint32_t kBase = 0x4c004c00u, kMask = 0x03c003c0u, kNeg24 = 0xce00ce00u;
  static constexpr int kBit = 6;
  __device__ static __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// Eight nibbles as 16 + n, in the order 0 4 1 5 2 6 3 7.
template <class X>
__device__ __forceinline__ u32x4 widen_nibbles(uint32_t w) {
  u32x4 r;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int sh = X::kBit - 4 * s;
    const uint32_t v = sh >= 0 ? w << (sh >= 0 ? sh : 0) : w >> (sh < 0 ? -sh : 0);
    r[s] = (v & X::kMask) | X::kBase;
  }
  return r;
}

// Eight 16-bit values in the same order.
__device__ __forceinline__ u32x4 order_x(u32x4 d) {
  return u32x4{__builtin_amdgcn_perm(d.z, d.x, 0x05040100u), __builtin_amdgcn_perm(d.z, d.x, 0x07060302u),
               __builtin_amdgcn_perm(d.w, d.y, 0x05040100u), __builtin_amdgcn_perm(d.w, d.y, 0x07060302u)};
}

__device__ __forceinline__ void store_logit(void* out, int dtype, int64_t i, float x) {
  switch (dtype) {
    case 0: Bf16::store1(static_cast<char*>(out), i, x); break;
    case 1: Fp16::store1(static_cast<char*>(out), i, x); break;
    default: Fp32::store1(static_cast<char*>(out), i, x); break;
  }
}

// w[a] of lane row q becomes w[q] of lane row a (lane rows: 16 lanes each).
__device__ __forceinline__ u32x4 transpose_rows(u32x4 w) {
  auto p = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
  auto r = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
  auto lo = __builtin_amdgcn_permlane16_swap(p[0], r[0], false, false);
  auto hi = __builtin_amdgcn_permlane16_swap(p[1], r[1], false, false);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

template <int N>
struct ScaleVec;  // N bf16 values at any 2-byte boundary
template <>
struct ScaleVec<2> {
  typedef uint32_t type __attribute__((ext_vector_type(1), aligned(2)));
};
template <>
struct ScaleVec<4> {
  typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct ScaleVec<8> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};

constexpr int kSpan = 256;  // columns a wave takes at a time: a row's 128-byte line

// One workgroup: 16 RT vocabulary rows x 16 NT rows of x.  Its four waves take
// every fourth span of columns and add their sums through LDS at the end.
template <class X, int G, int NT, int RT>
__global__ void __launch_bounds__(256) k_w4_logits(W4Args a) {
  constexpr int kGroups = kSpan / G, kSteps = G / 32;  // per span, per group
  __shared__ float sm[4][RT * 4][64];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int h = a.h, spans = h / kSpan;  // whole ones; a last, short one follows

  // rows past the end repeat the last one: their results are not stored
  const char* wrow[RT];
  const uint16_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t v = v0 + r * 16 + r16;
    v = v < a.V ? v : a.V - 1;
    wrow[r] = static_cast<const char*>(a.packed) + v * a.ld_p;
    srow[r] = a.scales + v * a.ld_s;
  }
  const uint16_t* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int64_t row = t0 + t * 16 + r16;
    row = row < a.T ? row : a.T - 1;
    xrow[t] = a.hidden + row * a.ld_h;
  }

  f32x4 tot[NT][RT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) tot[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};

  const u32x4 neg24{X::kNeg24, X::kNeg24, X::kNeg24, X::kNeg24};

  struct Span {
    u32x4 w[RT][2];
    uint32_t s[RT][kGroups / 2];
  };
  auto load = [&](int c, Span& d, auto whole) {
    constexpr bool full = decltype(whole)::value;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        // a lane's 32 columns lie inside the head or past its end as a whole
        int k = c * kSpan + f * 128 + q * 32;
        k = full || k < h ? k : 0;
        d.w[r][f] = *reinterpret_cast<const u32x4*>(wrow[r] + k / 2);
      }
      if (full) {
        const auto v = *reinterpret_cast<const typename ScaleVec<kGroups>::type*>(srow[r] + c * kGroups);
#pragma unroll
        for (int i = 0; i < kGroups / 2; ++i) d.s[r][i] = v[i];
      } else {
        const int last = (h - 1) / G;
#pragma unroll
        for (int i = 0; i < kGroups / 2; ++i) {
          const int g0 = c * kGroups + 2 * i, g1 = g0 + 1;
          d.s[r][i] = srow[r][g0 < last ? g0 : last] | static_cast<uint32_t>(srow[r][g1 < last ? g1 : last]) << 16;
        }
      }
    }
  };

  auto add = [&](int c, const Span& cur, auto whole) {
    constexpr bool full = decltype(whole)::value;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      u32x4 x[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = c * kSpan + f * 128 + i * 32 + q * 8;
          u32x4 d = *reinterpret_cast<const u32x4*>(xrow[t] + (full || k < h ? k : 0));
          if (!full && k >= h) d = u32x4{0, 0, 0, 0};
          x[t][i] = order_x(d);
        }
      u32x4 words[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) words[r] = transpose_rows(cur.w[r][f]);
#pragma unroll
      for (int g = 0; g < 128 / G; ++g) {
        f32x4 shift[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          shift[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kSteps; ++i) shift[t] = X::mfma(x[t][g * kSteps + i], neg24, shift[t]);
        }
        const int gs = f * (128 / G) + g;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const uint32_t pair = cur.s[r][gs / 2];
          const float sc = __uint_as_float(gs & 1 ? pair & 0xffff0000u : pair << 16);
          u32x4 b[kSteps];
#pragma unroll
          for (int i = 0; i < kSteps; ++i) b[i] = widen_nibbles<X>(words[r][g * kSteps + i]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x4 acc = shift[t];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) acc = X::mfma(x[t][g * kSteps + i], b[i], acc);
#pragma unroll
            for (int j = 0; j < 4; ++j) tot[t][r][j] = fmaf(sc, acc[j], tot[t][r][j]);
          }
        }
      }
    }
  };

  Span cur;
  if (w < spans) load(w, cur, std::true_type());
  for (int c = w; c < spans; c += 4) {
    Span nxt;
    if (c + 4 < spans) load(c + 4, nxt, std::true_type());
    add(c, cur, std::true_type());
    cur = nxt;
  }
  if (spans * kSpan < h && (spans & 3) == w) {
    load(spans, cur, std::false_type());
    add(spans, cur, std::false_type());
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm[w][r * 4 + j][lane] = tot[t][r][j];
    __syncthreads();
    for (int e = w; e < RT * 4; e += 4) {
      const float sum = (sm[0][e][lane] + sm[1][e][lane]) + (sm[2][e][lane] + sm[3][e][lane]);
      const int64_t row = t0 + t * 16 + q * 4 + (e & 3);
      const int64_t v = v0 + (e >> 2) * 16 + r16;
      if (row < a.T && v < a.V) store_logit(a.out, a.out_dtype, row * a.ld_out + v, sum);
    }
  }
}

template <class X, int G>
hipError_t launch_logits(const W4Args& a, hipStream_t s) {
  // grid.y is at most 65535 blocks of 64 rows
  constexpr int64_t kRows = int64_t(65535) * 64;
  for (int64_t r0 = 0; r0 < a.T; r0 += kRows) {
    W4Args b = a;
    b.T = a.T - r0 < kRows ? a.T - r0 : kRows;
    b.hidden = a.hidden + r0 * a.ld_h;
    b.out = static_cast<char*>(a.out) + r0 * a.ld_out * (a.out_dtype == 2 ? 4 : 2);
    const int nt = b.T >= 64 ? 4 : static_cast<int>((b.T + 15) / 16);
    const unsigned gy = static_cast<unsigned>((b.T + 63) / 64);
    TimedLaunch tl("k_w4_logits", s);
    auto grid = [&](int rt) { return dim3(static_cast<unsigned>((int64_t(a.V) + 16 * rt - 1) / (16 * rt)), gy); };
    switch (nt) {
      case 1: hipLaunchKernelGGL((k_w4_logits<X, G, 1, 2>), grid(2), dim3(256), 0, s, b); break;
      case 2: hipLaunchKernelGGL((k_w4_logits<X, G, 2, 2>), grid(2), dim3(256), 0, s, b); break;
      case 3: hipLaunchKernelGGL((k_w4_logits<X, G, 3, 4>), grid(4), dim3(256), 0, s, b); break;
      default: hipLaunchKernelGGL((k_w4_logits<X, G, 4, 4>), grid(4), dim3(256), 0, s, b); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class X>
hipError_t launch_logits_g(const W4Args& a, hipStream_t s) {
  switch (a.group) {
    case 32: return launch_logits<X, 32>(a, s);
    case 64: return launch_logits<X, 64>(a, s);
    default: return launch_logits<X, 128>(a, s);
  }
}

// Eight columns a lane; the group / 8 lanes of a group agree on its scale.
template <class Tr>
__global__ void __launch_bounds__(256) k_w4_quantize(W4QuantArgs a) {
  const int group = a.group, words = a.groups * (group / 8);  // per row, whole groups
  const int64_t n = static_cast<int64_t>(a.V) * words;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  // n and stride are multiples of a group's lanes, which so stay together
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += stride) {
    const int64_t v = i / words;
    const int wd = static_cast<int>(i - v * words);
    const bool in = wd * 8 < a.h;
    const char* row = static_cast<const char*>(a.weight) + v * a.ld_w * Tr::kBytes;
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = 0.f;
    if (in) {
      const char* p = row + static_cast<int64_t>(wd) * 8 * Tr::kBytes;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
        for (int k = 0; k < 8; k += Tr::kPerVec) Tr::unpack(*reinterpret_cast<const u32x4*>(p + k * Tr::kBytes), x + k);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = Tr::load1(p, k);
      }
    }
    // largest magnitude as bits: a NaN is larger than anything and stays
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __float_as_uint(x[k]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    for (int off = 1; off < group / 8; off <<= 1) {
      const uint32_t o = __shfl_xor(m, off, 64);
      m = o > m ? o : m;
    }
    // a group with an infinity gets a NaN for its scale too
    const uint32_t sb = m >= 0x7f800000u ? 0x7fc0u : pack_bf16x2(__fdiv_rn(__uint_as_float(m), 7.f), 0.f) & 0xffffu;
    const float s = __uint_as_float(sb << 16);
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y = s == 0.f ? 0.f : rintf(__fdiv_rn(x[k], s));
      y = fminf(fmaxf(y, -8.f), 7.f);
      word |= static_cast<uint32_t>(static_cast<int>(y) + 8) << (4 * k);
    }
    if (in) {
      reinterpret_cast<uint32_t*>(static_cast<char*>(a.packed) + v * a.ld_p)[wd] = word;
      if (wd % (group / 8) == 0) a.scales[v * a.ld_s + wd / (group / 8)] = static_cast<uint16_t>(sb);
    }
  }
}

}  // namespace

hipError_t launch_w4_logits(int dtype, const W4Args& a, hipStream_t s) {
  return dtype == 0 ? launch_logits_g<XBf16>(a, s) : launch_logits_g<XFp16>(a, s);
}

hipError_t launch_w4_quantize(int dtype, const W4QuantArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.V) * a.groups * (a.group / 8);
  int64_t blocks = (n + 255) / 256;
  if (blocks > 16384) blocks = 16384;
  const dim3 g(static_cast<unsigned>(blocks)), b(256);
  TimedLaunch tl("k_w4_quantize", s);
  switch (dtype) {
    case 0: hipLaunchKernelGGL(k_w4_quantize<Bf16>, g, b, 0, s, a); break;
    case 1: hipLaunchKernelGGL(k_w4_quantize<Fp16>, g, b, 0, s, a); break;
    default: hipLaunchKernelGGL(k_w4_quantize<Fp32>, g, b, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace lp
