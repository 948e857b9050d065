// An output head in 8-bit floats (e4m3) with a scale for each block of 128 x 128:
//   out[t][v] = sum over blocks b of 128 columns
//               sx[t][b] sw[v / 128][b] sum_{k in b} qx[t][k] qw[v][k]
// The hidden rows are brought to 8 bits first, with a scale for each 128 columns
// of a row (k_fp8_rows), into the workspace.  Products run on the matrix cores at
// the rate of 8-bit operands, one block of K at a time from zero; the block's
// partial sums times the two scales are added to fp32 accumulators.
#include "lp_gemm.hpp"
#include "lp_internal.hpp"
#include "lp_sums.hpp"

namespace lp {

namespace {

constexpr int kBlock = 128;
constexpr float kLargestE4m3 = 448.f, kPerLargest = 1.f / kLargestE4m3;
constexpr float kLeastScale = 1.1754943508e-38f;  // 2^-126: a quotient by it is no larger than the value's own scale allows

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Two e4m3 bytes, rounded to nearest even (NaN stays NaN).
template <bool HIGH>
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi, uint32_t old) {
#if defined(__HIP_DEVICE_COMPILE__)
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, static_cast<int>(old), HIGH));
#else
  (void)lo, (void)hi;
  return old;
#endif
}

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x2_t quantize8(const float* x, float scale) {
  uint32_t w0 = 0, w1 = 0;
  w0 = to_e4m3x2<false>(x[0] / scale, x[1] / scale, w0);
  w0 = to_e4m3x2<true>(x[2] / scale, x[3] / scale, w0);
  w1 = to_e4m3x2<false>(x[4] / scale, x[5] / scale, w1);
  w1 = to_e4m3x2<true>(x[6] / scale, x[7] / scale, w1);
  return u32x2_t{w0, w1};
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax * kPerLargest, kLeastScale); }

// Eight columns from j on of a row of n, zeros behind its end.
template <class Tr>
__device__ __forceinline__ void load8(const char* row, int64_t j, int64_t n, float* x) {
  if (j + 8 <= n) {
#pragma unroll
    for (int i = 0; i < 8 / Tr::kPerVec; ++i)
      Tr::unpack(load_vec(row + (j + i * Tr::kPerVec) * Tr::kBytes), x + i * Tr::kPerVec);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = j + k < n ? Tr::load1(row, j + k) : 0.f;
  }
}

// 16 lanes a block of a row, 16 blocks a workgroup.  xq [T x hp], zeros behind
// column h; sx [blocks x pitch].
template <class Tr>
__global__ void __launch_bounds__(256) k_fp8_rows(Fp8Args a, uint8_t* xq, float* sx, int64_t pitch, int blocks, int64_t first) {
  const int64_t i = first + static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (i >= a.T * blocks) return;
  const int64_t t = i / blocks;
  const int b = static_cast<int>(i - t * blocks), lane = threadIdx.x & 15;
  float x[8];
  load8<Tr>(reinterpret_cast<const char*>(a.hidden) + t * a.ld_h * Tr::kBytes, b * kBlock + lane * 8, a.h, x);
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
  m = lanes_reduce<16>(m, [](float p, float q) { return fmaxf(p, q); });
  const float scale = scale_of(m);
  *reinterpret_cast<u32x2_t*>(xq + (t * blocks + b) * kBlock + lane * 8) = quantize8(x, scale);
  if (lane == 0) sx[b * pitch + t] = scale;
}

// A workgroup a block of 128 x 128, which stays in registers between the search for its
// largest magnitude and the rounding.  Bound by HBM: 5120 x 151936 bf16 445 us, 5.2 TB/s read
// and written (6.1 is an elementwise kernel's), fp32 713 us, 5.5.
template <class Tr>
__global__ void __launch_bounds__(256) k_fp8_quantize(Fp8QuantArgs a, int blocks, int64_t first) {
  __shared__ float sm[4];
  const int64_t block = first + blockIdx.x;
  const int vb = static_cast<int>(block / blocks), kb = static_cast<int>(block % blocks);
  const int lane = threadIdx.x & 15, r0 = threadIdx.x >> 4, j = kb * kBlock + lane * 8;
  float x[8][8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t v = static_cast<int64_t>(vb) * kBlock + r0 + i * 16;
    if (v < a.V) {
      load8<Tr>(static_cast<const char*>(a.weight) + v * a.ld_w * Tr::kBytes, j, a.h, x[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[i][k]));
    }
  }
  m = lanes_reduce<64>(m, [](float p, float q) { return fmaxf(p, q); });
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  const float scale = scale_of(fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])));
  if (threadIdx.x == 0) a.scales[vb * a.ld_s + kb] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t v = static_cast<int64_t>(vb) * kBlock + r0 + i * 16;
    if (v < a.V && j < a.h) *reinterpret_cast<u32x2_t*>(a.q + v * a.ld_q + j) = quantize8(x[i], scale);
  }
}

// ---------------------------------------------------------------------------
// many rows: tiles of 256 (vocabulary) x BN (rows)
// ---------------------------------------------------------------------------

struct TileArgs {
  const uint8_t* weight;
  int64_t ld_w;
  const float* sw;
  int64_t ld_s;
  const uint8_t* xq;  // [T x hp]
  const float* sx;    // [blocks x pitch_sx], 256 more behind them
  int64_t T;
  int64_t pitch_sx;  // T up to a multiple of 4
  int h, V, blocks;
  int n_vb, n_nb;
  int64_t t0;  // first row of the launch
  void* out;
  int out_dtype;
  int64_t ld_out;
};

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
               static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}

__device__ __forceinline__ f32x4_t mfma_16(i32x8 a, i32x8 b, f32x4_t c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
#else
  (void)a, (void)b;
  return c;
#endif
}

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// Eight e4m3 values as fp16, exactly.
__device__ __forceinline__ f16x8_t widen8(uint32_t lo, uint32_t hi) {
#if defined(__HIP_DEVICE_COMPILE__)
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(static_cast<int>(lo), 1.f, false);
  const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(static_cast<int>(lo), 1.f, true);
  const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(static_cast<int>(hi), 1.f, false);
  const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(static_cast<int>(hi), 1.f, true);
  return f16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#else
  (void)lo, (void)hi;
  return f16x8_t{};
#endif
}

// 32 bytes of K a lane, as fp16: four operands of 16x16x32 products.
struct Wide {
  f16x8_t k[4];
};

__device__ __forceinline__ Wide widen(i32x8 a) {
  return Wide{{widen8(a[0], a[1]), widen8(a[2], a[3]), widen8(a[4], a[5]), widen8(a[6], a[7])}};
}

__device__ __forceinline__ f32x4_t mfma_16(const Wide& a, const Wide& b, f32x4_t c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.k[i], b.k[i], c, 0, 0, 0);
  return c;
}

// Neighbouring results of one row to out, rounded once.
template <int N>
__device__ __forceinline__ void store_results(void* out, int dtype, int64_t at, const float* x, int valid) {
  char* p = static_cast<char*>(out);
  if (N % 4 == 0 && valid >= N) {
    if (dtype == 2) {
#pragma unroll
      for (int k = 0; k < N; k += 4) *reinterpret_cast<u32x4_a2*>(p + (at + k) * 4) = Fp32::pack(x + k);
      return;
    }
    if (N == 8) {
      *reinterpret_cast<u32x4_a2*>(p + at * 2) = dtype == 0 ? Bf16::pack(x) : Fp16::pack(x);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k >= valid) continue;
    if (dtype == 0)
      Bf16::store1(p, at + k, x[k]);
    else if (dtype == 1)
      Fp16::store1(p, at + k, x[k]);
    else
      Fp32::store1(p, at + k, x[k]);
  }
}

// To LDS, with no registers between: 16 bytes a lane (read once, so not kept in
// the caches), and one float that all lanes take.
__device__ __forceinline__ void load16_once(const dtl_rsrc_t& rsrc, unsigned char* to, uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)(to), 16, at, 0, 0, 2);
#else
  (void)rsrc, (void)to, (void)at;
#endif
}
__device__ __forceinline__ void load4_same(const dtl_rsrc_t& rsrc, unsigned char* to) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)(to), 4, 0, 0, 0, 0);
#else
  (void)rsrc, (void)to;
#endif
}

// The 16-byte chunk c of row r of 128 bytes lies at place c ^ chunk_swz(r): reads
// of 16 bytes take 16 lanes at a time, here the same 8 places of two chunks, which
// then differ in a bit (0.9 M cycles of conflicts a CU in 4096 rows without).
__device__ __forceinline__ int chunk_swz(int r) { return r & 7; }

template <int BM_, int BN, int WGM, int WGN, int STAGES_>
struct Fp8Tile {
  static constexpr int BM = BM_, STAGES = STAGES_, NW = WGM * WGN;
  static constexpr int MI = BM / WGM / 16, NI = BN / WGN / 16;     // 16 x 16 products of a wave
  static constexpr int A_INST = BM / 8 / NW, B_INST = BN / 8 / NW;  // 1 KB loads a wave and stage
  static constexpr int ROWS = (BM + BN) * kBlock;                   // bytes of both operands' rows
  static constexpr int STAGE = ROWS + 1024 + NW * 256;              // and the scales of up to 256 rows of x and of each wave's rows of the head
  static constexpr int OUT_PITCH = MI * 16 + 4;                     // floats of a row staged for output
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BN <= 256, "whole loads a wave");
  static_assert(BM / WGM <= kBlock, "a wave's rows of the head lie in one block of scales");
  static_assert(NW * 32 * OUT_PITCH * 4 <= STAGES * STAGE, "output staging fits the stages");
};

// One block of BM x BN: K in steps of 128 (one scale block) through LDS stages,
// filled direct to LDS with the step's scales.  A step's products are 16x16x128, a
// whole scale block each, so a partial sum takes four registers and is scaled while
// the next products run.  The step's last column of products is held back: behind it
// the next stage has arrived and this one is free (one barrier a step), and the first
// operands of the next step are read while it runs.
// 4096 x 7168 x 129280 to bf16: 3.5 ms, 2160 TFLOP/s, the matrix cores busy in 51% of
// the cycles and the clock near 2.05 GHz; a step of 256 x 256 is 2048 cycles of
// products, some 1300 of scaling on the same SIMDs and 1500 of LDS, which two waves a
// SIMD overlap in part.
template <int BM, int BN, int WGM, int WGN, int STAGES, bool WIDE>
__global__ void __launch_bounds__(64 * WGM * WGN, 2) k_fp8_tile(TileArgs a) {
  using C = Fp8Tile<BM, BN, WGM, WGN, STAGES>;
  constexpr int MI = C::MI, NI = C::NI, NW = C::NW;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[STAGES * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  int vb, nb;
  {
    // each XCD (workgroup b runs on XCD b % 8) walks one contiguous range of the
    // order: groups of 4 vocabulary blocks, in them the row blocks
    const int all = a.n_vb * a.n_nb, b = blockIdx.x, x = b & 7;
    const int L = (all >> 3) * x + min(x, all & 7) + (b >> 3);
    constexpr int G = 4;
    const int g = L / (G * a.n_nb), size = min(G, a.n_vb - g * G), in = L - g * G * a.n_nb;
    nb = in / size;
    vb = g * G + in % size;
  }
  const int v0 = vb * C::BM;
  const int64_t t0 = a.t0 + static_cast<int64_t>(nb) * BN;
  const int M = a.V - v0, N = static_cast<int>(a.T - t0 < BN ? a.T - t0 : BN);
  const int hp = a.blocks * kBlock;

  // Loads: slot (j NW + wave) 64 + lane of a stage's 16-byte chunks; its row r and
  // chunk kc ^ swizzle(r), the same kc for every j.  Rows past the operand are its
  // last one again; behind the last column the chunk in front of the row's last
  // block stands in, against zeros of x.
  const int r = wave * 8 + (lane >> 3), kc = (lane & 7) ^ chunk_swz(r);
  const dtl_rsrc_t wrsrc = dtl_rsrc(a.weight + static_cast<int64_t>(v0) * a.ld_w), xrsrc = dtl_rsrc(a.xq + t0 * hp);
  const uint32_t tail = static_cast<uint32_t>(kc * 16) >= static_cast<uint32_t>(a.h - (a.blocks - 1) * kBlock) ? kc * 16u : 0u;
  // row r of every 8 NW of an operand, no further than its last
  auto offset = [&](int j, uint32_t last, uint32_t ld) {
    return min(static_cast<uint32_t>(r) * ld + static_cast<uint32_t>(j * NW * 8) * ld, last) + kc * 16u;
  };
  const uint32_t ld_w = static_cast<uint32_t>(a.ld_w), ld_x = static_cast<uint32_t>(hp);
  const uint32_t last_w = static_cast<uint32_t>(min(M, C::BM) - 1) * ld_w, last_x = static_cast<uint32_t>(N - 1) * ld_x;
  // this wave's rows of the head lie in one block of scales
  const float* sw = a.sw + static_cast<int64_t>(min(v0 + wm * C::MI * 16, a.V - 1) / kBlock) * a.ld_s;
  auto issue = [&](int kt, unsigned char* stage) {
    const uint32_t back = kt == a.blocks - 1 ? tail : 0u;
#pragma unroll
    for (int j = 0; j < C::A_INST; ++j)
      dtl_load16(wrsrc, reinterpret_cast<uint16_t*>(stage + (j * NW + wave) * 1024), offset(j, last_w, ld_w) - back,
                 static_cast<uint32_t>(kt) * kBlock);
#pragma unroll
    for (int j = 0; j < C::B_INST; ++j)
      dtl_load16(xrsrc, reinterpret_cast<uint16_t*>(stage + C::BM * kBlock + (j * NW + wave) * 1024),
                 offset(j, last_x, ld_x), static_cast<uint32_t>(kt) * kBlock);
    if (wave == 0)
      dtl_load16(dtl_rsrc(a.sx + static_cast<int64_t>(kt) * a.pitch_sx + t0), reinterpret_cast<uint16_t*>(stage + C::ROWS), lane * 16u,
                 0);
    load4_same(dtl_rsrc(sw + kt), stage + C::ROWS + 1024 + wave * 256);
  };
  // 32 bytes of K of one operand row: chunks g and 4 + g, for both operands alike
  // (the order within K is free).
  const int r16 = lane & 15, g = lane >> 4, z16 = chunk_swz(r16);
  auto fragment = [&](const unsigned char* rows, int row) {
    const unsigned char* p = rows + (row + r16) * kBlock;
    return join(*reinterpret_cast<const u32x4*>(p + ((g ^ z16) << 4)), *reinterpret_cast<const u32x4*>(p + (((4 + g) ^ z16) << 4)));
  };
  auto frag_a = [&](const unsigned char* stage, int mi) { return fragment(stage, (wm * MI + mi) * 16); };
  auto frag_b = [&](const unsigned char* stage, int ni) { return fragment(stage + C::BM * kBlock, (wn * NI + ni) * 16); };
  auto scale_b = [&](const unsigned char* stage, int ni) {
    return reinterpret_cast<const float*>(stage + C::ROWS)[(wn * NI + ni) * 16 + r16];
  };

  auto scale_a = [&](const unsigned char* stage) { return *reinterpret_cast<const float*>(stage + C::ROWS + 1024 + wave * 256); };

  f32x4_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  using Frag = std::conditional_t<WIDE, Wide, i32x8>;
  auto as_operand = [](i32x8 x) {
    if constexpr (WIDE)
      return widen(x);
    else
      return x;
  };
  Frag fa[MI];
  i32x8 fb[2];
  float fx[2];
  // the oldest of the stages under way has arrived when only the others' loads are not back
  constexpr int LOADS = C::A_INST + C::B_INST + 1;
#define LP_FP8_ARRIVED(others)                                                                \
  if (wave == 0)                                                                              \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((others) * (LOADS + 1)) : "memory"); \
  else                                                                                        \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((others) * LOADS) : "memory")
#pragma unroll
  for (int i = 0; i < STAGES; ++i)
    if (i < a.blocks) issue(i, lds + i * C::STAGE);
  if (a.blocks >= STAGES) {
    LP_FP8_ARRIVED(STAGES - 1);
  } else {
    LP_FP8_ARRIVED(0);
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) fa[mi] = as_operand(frag_a(lds, mi));
  fb[0] = frag_b(lds, 0);
  fx[0] = scale_b(lds, 0);
  float w = scale_a(lds), w_next = 0.f;

  // Products of a column and, between them, the scaling of those of the column
  // before (of the last step's last column at first).
  const f32x4_t zero{0.f, 0.f, 0.f, 0.f};
  f32x4_t part[2][MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) part[1][mi] = zero;
  float f_before = 0.f;
  auto add = [&](f32x4_t& to, f32x4_t p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = fmaf(p[i], f_before, to[i]);
    asm volatile("" : "+v"(to));  // here, or the compiler keeps a whole step's parts for the end
  };
  int stage = 0;
  for (int kt = 0; kt < a.blocks; ++kt) {
    unsigned char* X = lds + stage * C::STAGE;
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    unsigned char* Y = lds + stage * C::STAGE;
    const bool next = kt + 1 < a.blocks;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const int cur = ni & 1;
      if (ni + 1 < NI) {
        fb[cur ^ 1] = frag_b(X, ni + 1);
        fx[cur ^ 1] = scale_b(X, ni + 1);
      } else {
        // every operand of this step is in registers
        if (STAGES > 2 && kt + STAGES <= a.blocks) {
          LP_FP8_ARRIVED(STAGES - 2);
        } else {
          LP_FP8_ARRIVED(0);
        }
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (next) {
          if (kt + STAGES < a.blocks) issue(kt + STAGES, X);
          fb[cur ^ 1] = frag_b(Y, 0);
          fx[cur ^ 1] = scale_b(Y, 0);
          w_next = scale_a(Y);
        }
      }
      const float f = w * fx[cur];
      const Frag b = as_operand(fb[cur]);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        part[cur][mi] = mfma_16(fa[mi], b, zero);
        if (ni + 1 == NI && next) fa[mi] = as_operand(frag_a(Y, mi));
        add(acc[mi][(ni + NI - 1) % NI], part[cur ^ 1][mi]);
      }
      f_before = f;
      __builtin_amdgcn_sched_barrier(0);  // no column's operands ahead of their turn
    }
    static_assert(NI % 2 == 0, "the next step's first column goes to buffer 0");
    w = w_next;
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) add(acc[mi][NI - 1], part[1][mi]);
#undef LP_FP8_ARRIVED
  __syncthreads();

  // Out: 32 rows at a time through LDS of the wave's own, so that a row's
  // neighbouring results are stored together.
  float* own = reinterpret_cast<float*>(lds) + wave * 32 * C::OUT_PITCH;
  const int vw = v0 + wm * MI * 16;
  const int per = a.out_dtype == 2 ? 4 : 8, lanes = MI * 16 / per, rows = 64 / lanes;
  const int col = lane % lanes * per, row0 = lane / lanes;
#pragma unroll
  for (int ni = 0; ni < NI; ni += 2) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<f32x4_t*>(own + (q * 16 + r16) * C::OUT_PITCH + mi * 16 + g * 4) = acc[mi][ni + q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = row0; q < 32; q += rows) {
      const int t = (wn * NI + ni) * 16 + q, v = vw + col;
      const float* p = own + q * C::OUT_PITCH + col;
      float x[8];
      *reinterpret_cast<f32x4_t*>(x) = *reinterpret_cast<const f32x4_t*>(p);
      if (t >= N || v >= a.V) continue;
      const int64_t at = (t0 + t) * a.ld_out + v;
      if (per == 8) {
        *reinterpret_cast<f32x4_t*>(x + 4) = *reinterpret_cast<const f32x4_t*>(p + 4);
        store_results<8>(a.out, a.out_dtype, at, x, a.V - v);
      } else {
        store_results<4>(a.out, a.out_dtype, at, x, a.V - v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// few rows: the head passes by once
// ---------------------------------------------------------------------------

// Up to 16 XT rows of x.  K is split over the 8 waves of a workgroup, whose blocks
// of x stay in registers; the workgroups walk over the head 16 rows at a time.  A
// wave's pieces of 16 rows x 128 columns, with the piece's scale, come through a
// ring of its own in LDS, whose other slots are on their way: whole lines of 128
// bytes a row, and no registers held by what is in flight (8 rows of 5120 x 151936
// 125 us, 6.3 TB/s, bound by reading the head; with pieces of 16 bytes a row through
// registers 184, with loads that stay in the caches 148).
constexpr int few_slots(int XT) { return XT == 1 ? 8 : XT == 2 ? 7 : 5; }

template <int NB, int XT, bool WIDE>
__global__ void __launch_bounds__(512, 2) k_fp8_few(TileArgs a) {
  constexpr int R = few_slots(XT), SLOT = 16 * kBlock + 256;
  __shared__ __attribute__((aligned(256))) unsigned char ring[8 * R * SLOT];
  __shared__ float sums[2][XT][8][256];
  static_assert(sizeof(ring) + sizeof(sums) <= 160 * 1024, "LDS of a CU");
  using Operand = std::conditional_t<WIDE, Wide, i32x8>;
  auto as_operand = [](i32x8 x) {
    if constexpr (WIDE)
      return widen(x);
    else
      return x;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int T = static_cast<int>(a.T), hp = a.blocks * kBlock, tiles = (a.V + 15) / 16;
  // wave's blocks: wave, wave + 8, ...; of them only the last may not be there
  const bool all = wave + (NB - 1) * 8 < a.blocks;
  const int mine = all ? NB : NB - 1;
  i32x8 x[XT][NB];
  float sx[XT][NB];
#pragma unroll
  for (int n = 0; n < XT; ++n)
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int kb = i < mine ? wave + i * 8 : 0, t = min(n * 16 + r, T - 1);
      const u32x4* p = reinterpret_cast<const u32x4*>(a.xq + static_cast<int64_t>(t) * hp + kb * kBlock);
      x[n][i] = join(p[g], p[4 + g]);
      sx[n][i] = a.sx[static_cast<int64_t>(kb) * a.pitch_sx + t];
    }

  // A piece: two loads of 8 rows (lane: row lane / 8, chunk kc) and one of the
  // scale (every lane the same).  Rows behind the head are its last one again;
  // behind the last column the row's first chunk of that block stands in, against zeros of x.
  unsigned char* const own = ring + wave * (R * SLOT);
  const int row = lane >> 3, kc0 = (lane & 7) ^ chunk_swz(row), kc1 = (lane & 7) ^ chunk_swz(row + 8);
  const int last_bytes = a.h - (a.blocks - 1) * kBlock;
  const uint32_t ld = static_cast<uint32_t>(a.ld_w);
  int put_tile = blockIdx.x, put_i = 0, put_slot = 0;
  auto put = [&]() {
    const int v = put_tile * 16, kb = wave + put_i * 8, last = min(15, a.V - 1 - v);
    const int end = kb == a.blocks - 1 ? last_bytes : kBlock;
    const dtl_rsrc_t w = dtl_rsrc(a.weight + static_cast<int64_t>(v) * a.ld_w + kb * kBlock);
    unsigned char* to = own + put_slot * SLOT;
    load16_once(w, to, static_cast<uint32_t>(min(row, last)) * ld + (kc0 * 16 < end ? kc0 * 16 : 0));
    load16_once(w, to + 1024, static_cast<uint32_t>(min(row + 8, last)) * ld + (kc1 * 16 < end ? kc1 * 16 : 0));
    load4_same(dtl_rsrc(a.sw + static_cast<int64_t>(put_tile / 8) * a.ld_s + kb), to + 2048);
    if (++put_i == mine) put_i = 0, put_tile += gridDim.x;
    put_slot = put_slot + 1 == R ? 0 : put_slot + 1;
  };
  if (mine > 0)
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (put_tile < tiles) put();

  const int z = chunk_swz(r);
  int slot = 0, buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    f32x4_t acc[XT];
#pragma unroll
    for (int n = 0; n < XT; ++n) acc[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (i + 1 == NB && !all) continue;
      // the oldest piece has arrived when only the others' loads are under way
      if (put_tile < tiles)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * (R - 1)) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const unsigned char* p = own + slot * SLOT;
      const i32x8 wq = join(*reinterpret_cast<const u32x4*>(p + r * kBlock + ((g ^ z) << 4)),
                            *reinterpret_cast<const u32x4*>(p + r * kBlock + (((4 + g) ^ z) << 4)));
      const float sw = *reinterpret_cast<const float*>(p + 2048);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (put_tile < tiles) put();  // into the slot just read
      slot = slot + 1 == R ? 0 : slot + 1;
      const Operand w = as_operand(wq);
#pragma unroll
      for (int n = 0; n < XT; ++n) {
        if (WIDE && NB * XT > 8) asm volatile("" : "+v"(x[n][i]));  // widened anew: the registers hold no more
        const f32x4_t q = mfma_16(w, as_operand(x[n][i]), f32x4_t{0.f, 0.f, 0.f, 0.f});
        const float f = sw * sx[n][i];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[n][k] = fmaf(q[k], f, acc[n][k]);
      }
    }
    // lane: rows 4 g .. + 3 of the head, row r of x
#pragma unroll
    for (int n = 0; n < XT; ++n) *reinterpret_cast<f32x4_t*>(&sums[buf][n][wave][r * 16 + g * 4]) = acc[n];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // not for the loads under way
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int e = threadIdx.x; e < XT * 256; e += 512) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += sums[buf][e >> 8][k][e & 255];
      const int t = e >> 4, v = tile * 16 + (e & 15);
      if (t < T && v < a.V) store_results<1>(a.out, a.out_dtype, (a.t0 + t) * a.ld_out + v, &s, 1);
    }
  }
}

template <int BM, int BN, int WGM, int WGN, int STAGES, bool WIDE>
hipError_t launch_tile(TileArgs a, hipStream_t s) {
  a.n_vb = (a.V + BM - 1) / BM;
  // blocks of a launch: below 2^32 work-items whatever T
  const int64_t most = (int64_t(1) << 22) / a.n_vb > 0 ? (int64_t(1) << 22) / a.n_vb : 1;
  const int64_t T = a.T;
  for (int64_t t0 = 0; t0 < T; t0 += most * BN) {
    const int64_t rows = T - t0 < most * BN ? T - t0 : most * BN;
    a.t0 = t0;
    a.n_nb = static_cast<int>((rows + BN - 1) / BN);
    TimedLaunch tl("k_fp8_tile", s);
    hipLaunchKernelGGL((k_fp8_tile<BM, BN, WGM, WGN, STAGES, WIDE>), dim3(static_cast<unsigned>(a.n_vb * a.n_nb)), dim3(64 * WGM * WGN), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int XT, bool WIDE, int NB = 8>
hipError_t launch_few(const TileArgs& a, hipStream_t s) {
  if constexpr (NB > 1)
    if ((a.blocks + 7) / 8 < NB) return launch_few<XT, WIDE, NB - 1>(a, s);
  const int tiles = (a.V + 15) / 16;
  TimedLaunch tl("k_fp8_few", s);
  hipLaunchKernelGGL((k_fp8_few<NB, XT, WIDE>), dim3(tiles < 256 ? tiles : 256), dim3(512), 0, s, a);
  return hipGetLastError();
}

constexpr int64_t kMostGroups = int64_t(1) << 23;  // of 256 threads in a launch: below 2^32 work-items

int64_t sx_pitch(int64_t T) { return (T + 3) / 4 * 4; }

size_t rows_bytes(int64_t T, int64_t h) { return (size_t(T) * ((h + kBlock - 1) / kBlock) * kBlock + 255) / 256 * 256; }

}  // namespace

size_t fp8_workspace_bytes(int64_t T, int64_t h, int64_t V) {
  (void)V;
  return rows_bytes(T, h) + ((size_t(sx_pitch(T)) * ((h + kBlock - 1) / kBlock) + 256) * 4 + 255) / 256 * 256;
}

hipError_t launch_fp8_logits(int dtype, const Fp8Args& f, char* ws, hipStream_t s) {
  TileArgs a{};
  a.weight = f.weight;
  a.ld_w = f.ld_w;
  a.sw = f.scales;
  a.ld_s = f.ld_s;
  a.T = f.T;
  a.h = f.h;
  a.V = f.V;
  a.blocks = (f.h + kBlock - 1) / kBlock;
  a.out = f.out;
  a.out_dtype = f.out_dtype;
  a.ld_out = f.ld_out;
  uint8_t* xq = reinterpret_cast<uint8_t*>(ws);
  float* sx = reinterpret_cast<float*>(ws + rows_bytes(f.T, f.h));
  a.xq = xq;
  a.sx = sx;
  a.pitch_sx = sx_pitch(f.T);
  const int64_t parts = (f.T * a.blocks + 15) / 16;
  for (int64_t p = 0; p < parts; p += kMostGroups) {
    const dim3 grid(static_cast<unsigned>(parts - p < kMostGroups ? parts - p : kMostGroups));
    TimedLaunch tl("k_fp8_rows", s);
    if (dtype == 0)
      hipLaunchKernelGGL(k_fp8_rows<Bf16>, grid, dim3(256), 0, s, f, xq, sx, sx_pitch(f.T), a.blocks, p * 16);
    else
      hipLaunchKernelGGL(k_fp8_rows<Fp16>, grid, dim3(256), 0, s, f, xq, sx, sx_pitch(f.T), a.blocks, p * 16);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // The ring reads each line of the head once, the tiles read x again for each block of
  // it; rows beyond 32 find no registers (17 rows of 5120 x 129280 127 us against 141
  // in tiles, 32 rows of 8192 x 129280 190 against 210).
  if (a.T <= 16 && a.blocks <= 64) return launch_few<1, true>(a, s);
  if (a.T <= 32 && a.blocks <= 64) return a.out_dtype == 2 ? launch_few<2, true>(a, s) : launch_few<2, false>(a, s);
  // fp32 results: widened operands, whose products keep every bit.  Before a rounding to 16
  // bits (2e-4 or 2e-3 of a value) the 8-bit products' own error, 1e-5 to 5e-5 of the logits'
  // rms, is small, and widening would take twice the time (512 rows 773 us against 430).
  // Tiles no wider than the rows need, and two workgroups a CU where they fit: 64 rows
  // of 5120 x 151936 182 us against 219 in tiles of 256 x 64, 128 rows 209 against 234
  // in 256 x 128, 512 rows to fp32 807 against 875.
  if (a.out_dtype == 2) {
    if (a.T <= 64) return launch_tile<128, 64, 2, 2, 3, true>(a, s);
    return launch_tile<128, 128, 2, 2, 2, true>(a, s);
  }
  if (a.T <= 64) return launch_tile<128, 64, 2, 2, 3, false>(a, s);
  if (a.T <= 128) return launch_tile<128, 128, 2, 2, 2, false>(a, s);
  return launch_tile<256, 256, 4, 2, 2, false>(a, s);
}

hipError_t launch_fp8_quantize(int dtype, const Fp8QuantArgs& a, hipStream_t s) {
  const int blocks = (a.h + kBlock - 1) / kBlock;
  const int64_t all = (int64_t(a.V) + kBlock - 1) / kBlock * blocks;
  for (int64_t p = 0; p < all; p += kMostGroups) {
    const dim3 grid(static_cast<unsigned>(all - p < kMostGroups ? all - p : kMostGroups));
    TimedLaunch tl("k_fp8_quantize", s);
    if (dtype == 0)
      hipLaunchKernelGGL(k_fp8_quantize<Bf16>, grid, dim3(256), 0, s, a, blocks, p);
    else if (dtype == 1)
      hipLaunchKernelGGL(k_fp8_quantize<Fp16>, grid, dim3(256), 0, s, a, blocks, p);
    else
      hipLaunchKernelGGL(k_fp8_quantize<Fp32>, grid, dim3(256), 0, s, a, blocks, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lp
