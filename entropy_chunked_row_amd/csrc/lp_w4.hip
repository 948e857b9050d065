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
// A lane loads 16 bytes, 32 columns of a row, and lanes exchange words in
// registers until each MFMA stays inside one group, whose sum is then scaled
// in fp32.
#include "lp_device.hpp"
#include "lp_internal.hpp"

// Measured: one row of 5120 x 151936, groups of 128: 73 us (5.5 TB/s); 8 rows,
// groups of 64: 89 us; 40 rows of 7168 x 129280, groups of 32: 195 us.  Few rows
// are bound by HBM (and short of it by the waves' meeting once per 32 rows),
// many by no unit alone: unpacking and scaling take half of the vector unit's time
// and the products 0.3 of the matrix unit's, 145 us together without the
// loads, with one workgroup a CU to hide what is left.

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

// The two constants of the unpacking, in registers: as literals they would
// make the and-or two instructions.  The instruction itself is left to the
// compiler, which knows how many cycles lie between it and a matrix
// instruction that reads its result.
template <class X>
struct Nibbles {
  uint32_t mask, base;

  __device__ __forceinline__ Nibbles() : mask(X::kMask), base(X::kBase) {
    asm volatile("" : "+s"(mask));
    asm volatile("" : "+v"(base));
  }

  // Eight nibbles as 16 + n, in the order 0 4 1 5 2 6 3 7.
  __device__ __forceinline__ u32x4 widen(uint32_t w) const {
    u32x4 r;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int sh = X::kBit - 4 * s;
      const uint32_t v = sh >= 0 ? w << (sh >= 0 ? sh : 0) : w >> (sh < 0 ? -sh : 0);
      r[s] = (v & mask) | base;
    }
    return r;
  }
};

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

// A lane row is 16 lanes; lane row q loads columns 32 q .. 32 q + 31 of a
// chunk of 128 as four words.  words_of exchanges words between lane rows until each
// word index i holds columns of one group only (none for groups of 128, one
// exchange for 64, a full 4 x 4 transpose for 32); column_of is the first of
// the eight columns that lane row q then holds in word i.
template <int G>
__device__ __forceinline__ u32x4 words_of(u32x4 w) {
  if constexpr (G == 128) return w;
  const auto p = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
  const auto r = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
  if constexpr (G == 64) return u32x4{p[0], r[0], p[1], r[1]};
  const auto lo = __builtin_amdgcn_permlane16_swap(p[0], r[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(p[1], r[1], false, false);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

template <int G>
__device__ __forceinline__ int column_of(int i, int q) {
  if (G == 128) return 32 * q + 8 * i;
  if (G == 64) return 64 * (i >> 1) + 32 * (q & 1) + 16 * (q >> 1) + 8 * (i & 1);
  return 32 * i + 8 * q;
}

// Columns are taken in chunks of 128, and the chunks of a row fall into
// kRanges ranges of equal length.  Every kernel adds a range's groups in order
// and then the ranges in order, so a row's logits have the same bits
// whichever kernel computes them.
constexpr int kChunk = 128;
constexpr int kRanges = 8;

// Words and scales of a 16-row tile for KC neighbouring chunks, as loaded:
// scales are unpacked where they are used, for any work on a loaded value
// next to its load would wait for the load.  TAIL: columns may end inside the
// chunks (otherwise loads need no branch, which would part them from the
// products they run ahead of).  EXIST: all KC chunks exist, so that with TAIL
// only the last one's columns may end, and its scales are loaded one by one.
template <int G, int KC, bool TAIL, bool EXIST = false>
struct Tile {
  static constexpr int kGroups = kChunk / G, kScales = KC * kGroups;
  static constexpr bool kSingly = TAIL && EXIST;
  u32x4 w[KC];
  uint32_t s[(kScales + 1) / 2];
  uint32_t last_s[kSingly ? kGroups : 1];

  // `Loaded` of the scales from p on
  template <int Loaded>
  __device__ __forceinline__ void load_scales(const uint16_t* p) {
    typedef u32x4 x4 __attribute__((aligned(2)));
    typedef uint32_t x2 __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t x1 __attribute__((aligned(2)));
#pragma unroll
    for (int i = 0; i + 8 <= Loaded; i += 8) {
      const u32x4 v = *reinterpret_cast<const x4*>(p + i);
      s[i / 2] = v.x, s[i / 2 + 1] = v.y, s[i / 2 + 2] = v.z, s[i / 2 + 3] = v.w;
    }
    constexpr int r4 = Loaded / 8 * 8, r2 = Loaded / 4 * 4, r1 = Loaded / 2 * 2;
    if constexpr (r2 > r4) {
      const auto v = *reinterpret_cast<const x2*>(p + r4);
      s[r4 / 2] = v.x, s[r4 / 2 + 1] = v.y;
    }
    if constexpr (r1 > r2) s[r2 / 2] = *reinterpret_cast<const x1*>(p + r2);
    if constexpr (Loaded > r1) s[r1 / 2] = p[r1];
  }

  // wrow: the lane's row from its own 16 bytes of chunk 0 on; srow: the row's
  // scales.  Chunks c .. c + KC - 1; what lies past column h is read from
  // elsewhere in the row (x is 0 there).
  __device__ __forceinline__ void load(const char* wrow, const uint16_t* srow, int c, int q, int h) {
    if constexpr (kSingly) {
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const bool in = k + 1 < KC || (c + k) * kChunk + q * 32 < h;
        w[k] = *reinterpret_cast<const u32x4*>(wrow + (in ? (c + k) * (kChunk / 2) : -q * 16));
      }
      load_scales<kScales - kGroups>(srow + c * kGroups);
      const int last = (h - 1) / G;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int at = (c + KC - 1) * kGroups + g;
        last_s[g] = srow[at < last ? at : last];
      }
    } else if (!TAIL || (c + KC) * kChunk <= h) {
#pragma unroll
      for (int k = 0; k < KC; ++k) w[k] = *reinterpret_cast<const u32x4*>(wrow + (c + k) * (kChunk / 2));
      load_scales<kScales>(srow + c * kGroups);
    } else {
      const int last = (h - 1) / G;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        // a lane's 32 columns lie inside the head or past its end as a whole
        const int at = (c + k) * kChunk + q * 32 < h ? (c + k) * (kChunk / 2) : -q * 16;
        w[k] = *reinterpret_cast<const u32x4*>(wrow + at);
      }
#pragma unroll
      for (int i = 0; i < (kScales + 1) / 2; ++i) {
        const int a = c * kGroups + 2 * i, b = a + 1;
        s[i] = srow[a < last ? a : last] | static_cast<uint32_t>(srow[b < last ? b : last]) << 16;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // issued here, not where registers would be saved
  }

  __device__ __forceinline__ float scale(int k, int g) const {
    if (kSingly && k == KC - 1) return __uint_as_float(last_s[g] << 16);
    const int i = k * kGroups + g;
    return __uint_as_float(i & 1 ? s[i / 2] & 0xffff0000u : s[i / 2] << 16);
  }
};

// Columns k .. k + 7 of a row of x; zero past the end.
template <bool TAIL>
__device__ __forceinline__ u32x4 load_x(const uint16_t* xrow, int k, int h) {
  u32x4 d = *reinterpret_cast<const u32x4*>(xrow + (!TAIL || k < h ? k : 0));
  if (TAIL && k >= h) d = u32x4{0, 0, 0, 0};
  return d;
}

// Start value of a group's sums: -24 sum x.
template <class X, int S>
__device__ __forceinline__ f32x4 shift_of(const u32x4* x, uint32_t n = X::kNeg24) {
  const u32x4 neg24{n, n, n, n};
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < S; ++i) acc = X::mfma(x[i], neg24, acc);
  return acc;
}

// Up to 16 rows of x and 8 KC chunks: x stays in registers.  A workgroup is
// resident and walks over pairs of 16-row tiles of the head; its wave w holds x's
// chunks of range w and reads that part of every tile, one tile ahead.  Per
// word of the head that leaves the unpacking, the products and a share of a
// multiply-add per group: no traffic for x, which at 16 rows would be four
// times that of the head.  The waves' sums meet in LDS once per pair.
template <class X, int G, int KC, bool TAIL>
__global__ void __launch_bounds__(512) k_w4_few(W4Args a) {
  constexpr int kGroups = kChunk / G, S = G / 32;
  // the groups' start values, kept where they take no more registers than this
  constexpr bool kKeepShift = KC * kGroups * 4 <= 40;
  __shared__ f32x4 red[2][2][kRanges][64];  // [turn][tile of the pair][wave][lane]
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, q = lane >> 4;
  const int h = a.h, chunks = (h + kChunk - 1) / kChunk;
  // the window of KC chunks read, all of which exist: it ends with the row
  // where the wave's own range does, and x is 0 in chunks before the range
  const int own = w * KC, c0 = own < chunks - KC ? own : chunks - KC;
  const int64_t tiles = (static_cast<int64_t>(a.V) + 15) / 16;
  const Nibbles<X> nibbles;

  u32x4 x[KC][4];
  f32x4 shift[KC][kGroups];
  {
    const uint16_t* xrow = a.hidden + (r16 < a.T ? r16 : a.T - 1) * a.ld_h;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[c][i] = order_x(load_x<true>(xrow, c0 + c >= own ? (c0 + c) * kChunk + column_of<G>(i, q) : h, h));
      if (kKeepShift) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) shift[c][g] = shift_of<X, S>(x[c] + g * S);
      }
    }
  }

  // Two buffers in turn, so that a load's registers are next touched when its
  // tile's turn comes (moving them would wait for the load).  A third buffer
  // measured no faster.
  Tile<G, KC, TAIL, true> buf[2];
  auto load = [&](int64_t tile, Tile<G, KC, TAIL, true>& d) {
    int64_t v = tile * 16 + r16;
    v = v < a.V ? v : a.V - 1;  // rows past the end repeat the last one
    d.load(static_cast<const char*>(a.packed) + v * a.ld_p + q * 16, a.scales + v * a.ld_s, c0, q, h);
  };
  auto add = [&](const Tile<G, KC, TAIL, true>& d) {
    f32x4 tot{0.f, 0.f, 0.f, 0.f};
    uint32_t neg24 = X::kNeg24;
    if (!kKeepShift) asm volatile("" : "+v"(neg24));  // or the compiler would keep the start values all the same
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const u32x4 words = words_of<G>(d.w[c]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 acc = kKeepShift ? shift[c][g] : shift_of<X, S>(x[c] + g * S, neg24);
#pragma unroll
        for (int i = 0; i < S; ++i) acc = X::mfma(x[c][g * S + i], nibbles.widen(words[g * S + i]), acc);
        const float sc = d.scale(c, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[j] = fmaf(sc, acc[j], tot[j]);
      }
      // x and the buffers fill the registers: no chunk may run ahead
      if (!kKeepShift) __builtin_amdgcn_sched_barrier(0);
    }
    return tot;
  };

  const int64_t step = 2 * static_cast<int64_t>(gridDim.x);
  int64_t tile = 2 * static_cast<int64_t>(blockIdx.x);
  load(tile, buf[0]);
  for (int b = 0; tile < tiles; tile += step, b ^= 1) {
    load(tile + 1, buf[1]);
    red[b][0][w][lane] = add(buf[0]);
    load(tile + step, buf[0]);
    red[b][1][w][lane] = add(buf[1]);  // of a tile past the end: not stored
    __syncthreads();
    // 512 sums; the buffer is written again two turns on, behind the next barrier
    const int l = (threadIdx.x & 255) >> 2, j = threadIdx.x & 3, second = threadIdx.x >> 8;
    const int64_t row = (l >> 4) * 4 + j, v = (tile + second) * 16 + (l & 15);
    if (row < a.T && v < a.V) {
      float sum = red[b][second][0][l][j];
#pragma unroll
      for (int k = 1; k < kRanges; ++k) sum += red[b][second][k][l][j];
      store_logit(a.out, a.out_dtype, row * a.ld_out + v, sum);
    }
  }
}

// Any number of rows of x and columns.  A workgroup takes 16 RT rows of the head
// per wave and 16 NT rows of x, which its waves share: x's chunk pairs pass
// through LDS, two buffers in turn, already in the products' order.
template <class X, int G, int NT, int RT, int NW, bool TAIL>
__global__ void __launch_bounds__(64 * NW, 2) k_w4_wide(W4Args a) {
  constexpr int kGroups = kChunk / G, S = G / 32;
  __shared__ u32x4 xs[2][2 * 4 * NT][64];  // [buffer][chunk, step, x tile][lane]
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t v0 = (static_cast<int64_t>(blockIdx.x) * NW + w) * (16 * RT);
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int h = a.h, chunks = (h + kChunk - 1) / kChunk;
  const int per = (chunks + kRanges - 1) / kRanges;

  const char* wrow[RT];
  const uint16_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t v = v0 + r * 16 + r16;
    v = v < a.V ? v : a.V - 1;  // rows past the end repeat the last one: not stored
    wrow[r] = static_cast<const char*>(a.packed) + v * a.ld_p + q * 16;
    srow[r] = a.scales + v * a.ld_s;
  }
  const Nibbles<X> nibbles;
  // each wave brings an equal share of the eight steps of a chunk pair
  const uint16_t* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int64_t row = t0 + t * 16 + r16;
    row = row < a.T ? row : a.T - 1;
    xrow[t] = a.hidden + row * a.ld_h;
  }

  // A lane's sums: of the range in hand in registers, of the ranges before it in
  // LDS where the registers would not hold two tiles of the head beside four
  // of x (64 rows of 5120 x 129280, groups of 128: 205 us with one tile, 160
  // so; with three tiles of x both fit, and LDS is 2 % slower).
  constexpr bool kTotInLds = NT == 4;
  __shared__ f32x4 lds_tot[kTotInLds ? NW : 1][kTotInLds ? NT : 1][RT][64];
  f32x4 reg_tot[NT][RT], part[NT][RT];
  auto tot = [&](int t, int r) -> f32x4& { return kTotInLds ? lds_tot[w][t][r][lane] : reg_tot[t][r]; };
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) tot(t, r) = part[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int XS = 8 / NW;
  u32x4 xn[XS][NT];
  auto fetch_x = [&](int c) {
#pragma unroll
    for (int i = 0; i < XS; ++i) {
      const int step = w * XS + i;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xn[i][t] = load_x<TAIL>(xrow[t], (c + (step >> 2)) * kChunk + column_of<G>(step & 3, q), h);
    }
  };
  auto put_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < XS; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) xs[buf][(w * XS + i) * NT + t][lane] = order_x(xn[i][t]);
  };

  // two buffers in turn: moving a load's registers would wait for it
  Tile<G, 2, TAIL> buf[2][RT];
  auto load = [&](int c, Tile<G, 2, TAIL>(&d)[RT]) {
#pragma unroll
    for (int r = 0; r < RT; ++r) d[r].load(wrow[r], srow[r], c, q, h);
  };
  int left = per;  // chunks to the end of the range
  auto add = [&](int c, const Tile<G, 2, TAIL>(&d)[RT], int b) {
    constexpr int kAll = 2 * kGroups;
    u32x4 x[NT][S];  // of a group; the next one's replaces it step by step
    f32x4 acc[2][NT][RT];
    // The products of a group run while the sums of the one before it are
    // scaled, which would otherwise wait for the last product.
    auto scale_in = [&](int group) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float sc = d[r].scale(group / kGroups, group % kGroups);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[t][r][j] = fmaf(sc, acc[group & 1][t][r][j], part[t][r][j]);
      }
      if (group % kGroups == kGroups - 1 && (--left == 0 || c + group / kGroups + 1 >= chunks)) {  // end of a range
        left = per;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            tot(t, r) += part[t][r];
            part[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
      }
    };
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t][i] = xs[b][i * NT + t][lane];
    u32x4 words[RT];
#pragma unroll
    for (int group = 0; group < kAll; ++group) {
      const int f = group / kGroups, g = group % kGroups;
      if (g == 0) {
#pragma unroll
        for (int r = 0; r < RT; ++r) words[r] = words_of<G>(d[r].w[f]);
      }
      f32x4 start[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) start[t] = shift_of<X, S>(x[t]);
#pragma unroll
      for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const u32x4 bw = nibbles.widen(words[r][g * S + i]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const f32x4 from = i == 0 ? start[t] : acc[group & 1][t][r];
            acc[group & 1][t][r] = X::mfma(x[t][i], bw, from);
          }
        }
        if (group + 1 < kAll) {
#pragma unroll
          for (int t = 0; t < NT; ++t) x[t][i] = xs[b][((group + 1) * S + i) * NT + t][lane];
        }
      }
      if (group > 0) scale_in(group - 1);
    }
    scale_in(kAll - 1);
  };

  fetch_x(0);
  load(0, buf[0]);
  put_x(0);
  __syncthreads();
  // The loads ahead carry no condition (past the end they repeat the last
  // pair): behind a branch the wait for the older loads would wait for them too.
  const int last = (chunks - 1) / 2 * 2;
  int c = 0;
  while (true) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int next = c < last ? c + 2 : last;
      fetch_x(next);
      load(next, buf[k ^ 1]);
      add(c, buf[k], k);
      if (c == last) goto done;
      // this buffer of x was last read before the barrier that ended the
      // previous turn
      put_x(k ^ 1);
      __syncthreads();
      c += 2;
    }
  }
done:
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const f32x4 sum = tot(t, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t row = t0 + t * 16 + q * 4 + j, v = v0 + r * 16 + r16;
        if (row < a.T && v < a.V) store_logit(a.out, a.out_dtype, row * a.ld_out + v, sum[j]);
      }
    }
}

// Chunks per range up to which x's registers leave room for two buffers; with
// groups of 32 the buffers' scales take more (one row of 7168 x 129280: 328 us
// spilling, 126 us through k_w4_wide; with groups of 128 83 us here, 99 there).
constexpr int most_chunks(int group) { return group == 32 ? 5 : 7; }

template <class X, int G, bool TAIL>
hipError_t launch_few(const W4Args& a, int per, hipStream_t s) {
  // one resident workgroup a CU, two where the registers of x leave room
  const int64_t pairs = (int64_t(a.V) + 31) / 32, most = per <= 3 ? 512 : 256;
  const dim3 g(static_cast<unsigned>(pairs < most ? pairs : most)), b(512);
  TimedLaunch tl("k_w4_logits", s);
  switch (per) {
    case 1: hipLaunchKernelGGL((k_w4_few<X, G, 1, TAIL>), g, b, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_w4_few<X, G, 2, TAIL>), g, b, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_w4_few<X, G, 3, TAIL>), g, b, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_w4_few<X, G, 4, TAIL>), g, b, 0, s, a); break;
    case 5: hipLaunchKernelGGL((k_w4_few<X, G, 5, TAIL>), g, b, 0, s, a); break;
    default:
      if constexpr (most_chunks(G) == 7) {
        if (per == 6)
          hipLaunchKernelGGL((k_w4_few<X, G, 6, TAIL>), g, b, 0, s, a);
        else
          hipLaunchKernelGGL((k_w4_few<X, G, 7, TAIL>), g, b, 0, s, a);
      }
  }
  return hipGetLastError();
}

template <class X, int G, bool TAIL>
hipError_t launch_wide(const W4Args& a, hipStream_t s) {
  // grid.y is at most 65535 blocks of 64 rows
  constexpr int64_t kRows = int64_t(65535) * 64;
  constexpr int NW = 8;  // four waves measured the same
  for (int64_t r0 = 0; r0 < a.T; r0 += kRows) {
    W4Args b = a;
    b.T = a.T - r0 < kRows ? a.T - r0 : kRows;
    b.hidden = a.hidden + r0 * a.ld_h;
    b.out = static_cast<char*>(a.out) + r0 * a.ld_out * (a.out_dtype == 2 ? 4 : 2);
    const int nt = b.T >= 64 ? 4 : static_cast<int>((b.T + 15) / 16);
    constexpr int RT = 2;  // two tiles of the head a wave share its x operands
    const dim3 g(static_cast<unsigned>((int64_t(a.V) + 16 * NW * RT - 1) / (16 * NW * RT)),
                 static_cast<unsigned>((b.T + 63) / 64));
    TimedLaunch tl("k_w4_logits", s);
    switch (nt) {
      case 1: hipLaunchKernelGGL((k_w4_wide<X, G, 1, RT, NW, TAIL>), g, dim3(64 * NW), 0, s, b); break;
      case 2: hipLaunchKernelGGL((k_w4_wide<X, G, 2, RT, NW, TAIL>), g, dim3(64 * NW), 0, s, b); break;
      case 3: hipLaunchKernelGGL((k_w4_wide<X, G, 3, RT, NW, TAIL>), g, dim3(64 * NW), 0, s, b); break;
      default: hipLaunchKernelGGL((k_w4_wide<X, G, 4, RT, NW, TAIL>), g, dim3(64 * NW), 0, s, b); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class X, int G>
hipError_t launch_logits(const W4Args& a, hipStream_t s) {
  const int per = ((a.h + kChunk - 1) / kChunk + kRanges - 1) / kRanges;
  if (a.T <= 16 && per <= most_chunks(G))
    return a.h % kChunk ? launch_few<X, G, true>(a, per, s) : launch_few<X, G, false>(a, per, s);
  return a.h % (2 * kChunk) ? launch_wide<X, G, true>(a, s) : launch_wide<X, G, false>(a, s);
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
