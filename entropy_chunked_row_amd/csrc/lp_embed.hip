// Embedding lookup with a scale, and its weight gradient by sorted tokens.
//
// Lookup: out[i] = RN(scale * W[token[i]]), one fp32 product per element.
//
// Gradient: dW[v] (+)= scale * sum over i with token[i] = v of g[i].  The
// positions are sorted by token (a stable radix sort: equal tokens keep their
// order), so that each row of dW has one owner that adds its gradients in a
// fixed order: no float atomics, the same bits on every call.  Only the token
// ids are sorted; the gradients are read where they lie, once.
//
// Frequent tokens: blocks of kChunk sorted positions that hold a single token
// are summed first, by a workgroup each, into partial rows; the owner then
// adds the partial rows of its run's whole blocks and, one by one, the
// positions before and after them.  The same launch writes the zeros of the
// rows that no token names, which are most of dW's bytes.
//
// Bound: HBM.  Measured: lookup of 32768 x 5120 bf16 101 us a call among others, 85 us
// repeated on the same tokens (a third of the rows, repeated tokens, comes out of
// the caches), gradient of 32768 x 5120 bf16 over a
// vocabulary of 151936 0.69 ms, of which 0.46 ms is the least that 3.1 GB of
// dW can take at the rate of a fill: sort 27 us, partial rows 30 us, runs and
// zeros 0.63 ms.
//
// Up to kTinyN positions nothing is sorted: every owner finds its positions
// among all of them with ballots, in one launch.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kChunk = 64;      // sorted positions per partial row
constexpr int kSortNT = 256;    // threads of a sorting workgroup
constexpr int kMaxTiles = 128;  // sorting workgroups
constexpr int kMaxDigit = 10;   // bits per pass
constexpr int kSmallN = 4096;   // sorted by one workgroup in LDS up to here
constexpr int kSmallNT = 1024;
constexpr int kTinyN = 256;     // not sorted up to here
constexpr int kSumNT = 128;     // threads of a summing workgroup
constexpr int kRunSpan = 16;    // sorted positions whose run starts a workgroup owns
constexpr uint32_t kAbsent = 0xffffffffu;

typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------

template <class Tr>
__global__ void __launch_bounds__(256) k_embedding(EmbedArgs a) {
  constexpr int P = Tr::kPerVec;
  const int lane = threadIdx.x & 63;
  const int64_t waves = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); i < a.N; i += waves) {
    const int64_t v = a.tokens[i];
    const bool known = v >= 0 && v < a.V;
    const char* src = static_cast<const char*>(a.weight) + (known ? v : 0) * a.ld_w * Tr::kBytes;
    char* dst = static_cast<char*>(a.out) + i * a.ld_out * Tr::kBytes;
    const RowSplit<Tr> sp(dst, a.h);  // stores on the 16-byte grid, loads where they fall
    if (lane < sp.head) Tr::store1(dst, lane, known ? Tr::load1(src, lane) * a.scale : 0.f);
    const char* vp = src + sp.head * Tr::kBytes;
    u32x4* wp = reinterpret_cast<u32x4*>(dst + sp.head * Tr::kBytes);
    for (int j = lane; j < sp.nvec; j += 64) {
      float x[P];
      Tr::unpack(load_vec(vp + static_cast<int64_t>(j) * 16), x);
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = known ? x[k] * a.scale : 0.f;
      __builtin_nontemporal_store(Tr::pack(x), wp + j);
    }
    for (int j = a.h - sp.tail + lane; j < a.h; j += 64)
      Tr::store1(dst, j, known ? Tr::load1(src, j) * a.scale : 0.f);
  }
}

// ---------------------------------------------------------------------------
// stable sort of (token, position)
// ---------------------------------------------------------------------------

// Token of position i as a sort key; ids outside [0, V) become V and sort last.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t i) {
  const int64_t v = a.tokens[i];
  return v >= 0 && v < a.V ? static_cast<uint32_t>(v) : static_cast<uint32_t>(a.V);
}

// Lanes of the wave with the same digit of `bits` bits (among live lanes).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool live, int bits) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const uint64_t s = __ballot((d >> b) & 1u);
    m &= ((d >> b) & 1u) ? s : ~s;
  }
  return m;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
}

// Orders the wave's LDS accesses before and after it (they run in order; the
// compiler must keep them so).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Whole sort of N <= kSmallN positions in one workgroup.  Wave w ranks a
// contiguous share of the positions in order, so equal digits keep theirs.
__global__ void __launch_bounds__(kSmallNT) k_embed_sort_small(EmbedGradArgs a) {
  constexpr int W = kSmallNT / 64;
  __shared__ uint32_t key[2][kSmallN];
  __shared__ uint32_t pos[2][kSmallN];
  __shared__ uint32_t cnt[W][256];
  __shared__ uint32_t base[256];
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int n = static_cast<int>(a.N);
  for (int i = tid; i < n; i += kSmallNT) {
    key[0][i] = key_of(a, i);
    pos[0][i] = i;
  }
  if (a.first) {
    for (int v = tid; v < a.V; v += kSmallNT) a.first[v] = kAbsent;
  }
  const int share = ((n + W - 1) / W + 63) / 64 * 64;
  const int i0 = w * share, i1 = i0 + share < n ? i0 + share : n;
  int cur = 0;
  for (int shift = 0; shift < a.key_bits; shift += 8, cur ^= 1) {
    for (int i = tid; i < W * 256; i += kSmallNT) (&cnt[0][0])[i] = 0;
    __syncthreads();
    for (int i = i0; i < i1; i += 64) {
      const bool live = i + lane < i1;
      const uint32_t d = live ? (key[cur][i + lane] >> shift) & 255u : 0;
      const uint64_t m = same_digit(d, live, 8);
      if (live && lanes_below(m) == 0) cnt[w][d] += __popcll(m);
      wave_sync();
    }
    __syncthreads();
    if (tid < 256) {  // digit totals, and each wave's start within its digit
      uint32_t s = 0;
      for (int k = 0; k < W; ++k) {
        const uint32_t c = cnt[k][tid];
        cnt[k][tid] = s;
        s += c;
      }
      base[tid] = s;
    }
    __syncthreads();
    if (w == 0) {  // exclusive scan of 256 totals, four a lane
      uint32_t v[4], s = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = s;
        s += base[lane * 4 + k];
      }
      uint32_t x = s;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const uint32_t y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) base[lane * 4 + k] = v[k] + x - s;
    }
    __syncthreads();
    for (int i = i0; i < i1; i += 64) {
      const bool live = i + lane < i1;
      const uint32_t kx = live ? key[cur][i + lane] : 0;
      const uint32_t px = live ? pos[cur][i + lane] : 0;
      const uint32_t d = (kx >> shift) & 255u;
      const uint64_t m = same_digit(d, live, 8);
      const int below = lanes_below(m);
      uint32_t at = 0;
      if (live) at = base[d] + cnt[w][d] + below;
      // every lane has read the counter before its leader moves it on
      wave_sync();
      if (live && below == 0) cnt[w][d] += __popcll(m);
      wave_sync();
      if (live) {
        key[cur ^ 1][at] = kx;
        pos[cur ^ 1][at] = px;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < n; i += kSmallNT) {
    const uint32_t k = key[cur][i];
    a.keys[0][i] = k;
    a.pos[0][i] = pos[cur][i];
  }
}

// One pass over `bits` bits of the keys, two kernels: digit counts per tile,
// and the stable scatter, whose workgroups each add up the counts before them
// (there are at most kMaxTiles tiles, so this costs less than a scan's launch).
__device__ __forceinline__ uint32_t load_key(const EmbedGradArgs& a, int src, int64_t i) {
  return src < 0 ? key_of(a, i) : a.keys[src][i];
}

__global__ void __launch_bounds__(kSortNT) k_embed_count(EmbedGradArgs a, int shift, int bits, int src) {
  __shared__ uint32_t cnt[1 << kMaxDigit];
  const int bins = 1 << bits;
  for (int d = threadIdx.x; d < bins; d += kSortNT) cnt[d] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile, t1 = t0 + a.tile < a.N ? t0 + a.tile : a.N;
  for (int64_t i = t0 + threadIdx.x; i < t1; i += kSortNT)
    atomicAdd(&cnt[(load_key(a, src, i) >> shift) & (bins - 1)], 1u);
  if (src < 0 && a.first) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kSortNT;
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kSortNT + threadIdx.x; v < a.V; v += stride) a.first[v] = kAbsent;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortNT) a.counts[static_cast<int64_t>(blockIdx.x) * bins + d] = cnt[d];
}

__global__ void __launch_bounds__(kSortNT) k_embed_scatter(EmbedGradArgs a, int shift, int bits, int src, int dst) {
  constexpr int W = kSortNT / 64, kPer = (1 << kMaxDigit) / kSortNT;
  __shared__ uint32_t cnt[W][1 << kMaxDigit];
  __shared__ uint32_t wsum[W];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int bins = 1 << bits;
  for (int d = threadIdx.x; d < bins; d += kSortNT)
#pragma unroll
    for (int k = 0; k < W; ++k) cnt[k][d] = 0;
  __syncthreads();
  const int share = a.tile / W;  // a multiple of 64
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * a.tile + static_cast<int64_t>(w) * share;
  const int64_t s1 = s0 + share < a.N ? s0 + share : a.N;
  for (int64_t i = s0 + lane; i < s1; i += 64) atomicAdd(&cnt[w][(load_key(a, src, i) >> shift) & (bins - 1)], 1u);
  // digits of this thread: kPer neighbours, so that the scan over digits is
  // one over threads
  uint32_t before[kPer], total[kPer], mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) before[k] = total[k] = 0;
  static_assert(kPer == 4, "a thread's digits are one 16-byte load");
  if (static_cast<int>(threadIdx.x) * kPer < bins) {  // bins is a multiple of 4
    const uint32_t* p = a.counts + threadIdx.x * kPer;
#pragma unroll 16
    for (int t = 0; t < a.tiles; ++t) {
      const u32x4 c = *reinterpret_cast<const u32x4*>(p + static_cast<int64_t>(t) * bins);
      const uint32_t on = t < static_cast<int>(blockIdx.x) ? ~0u : 0u;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        total[k] += c[k];
        before[k] += c[k] & on;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) mine += total[k];
  uint32_t x = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  uint32_t base = x - mine;
#pragma unroll
  for (int k = 0; k < W; ++k)
    if (k < w) base += wsum[k];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = threadIdx.x * kPer + k;
    if (d < bins) {
      uint32_t s = base + before[k];
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const uint32_t c = cnt[u][d];
        cnt[u][d] = s;
        s += c;
      }
    }
    base += total[k];
  }
  __syncthreads();
  for (int64_t i0 = s0; i0 < s1; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool live = i < s1;
    const uint32_t kx = live ? load_key(a, src, i) : 0;
    const uint32_t d = (kx >> shift) & (bins - 1);
    const uint64_t m = same_digit(d, live, bits);
    const int below = lanes_below(m);
    const uint32_t at = cnt[w][d] + below;
    wave_sync();
    if (live && below == 0) cnt[w][d] += __popcll(m);
    wave_sync();
    if (live) {
      a.keys[dst][at] = kx;
      a.pos[dst][at] = src < 0 ? static_cast<uint32_t>(i) : a.pos[src][i];
    }
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------

// x[0..P) = the P columns from `col` of the gradient at position i.
template <class Tr, bool VEC>
__device__ __forceinline__ void load_cols(const EmbedGradArgs& a, uint32_t i, int64_t col, float* x) {
  const char* p = static_cast<const char*>(a.grad) + static_cast<int64_t>(i) * a.ld_g * Tr::kBytes;
  if constexpr (VEC)
    Tr::unpack(load_vec(p + col * Tr::kBytes), x);
  else
    x[0] = Tr::load1(p, col);
}

// acc[0..P) += the gradients at sorted positions [i0, i1), in that order, kAhead
// rows in flight.
template <class Tr, bool VEC, int kAhead>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, float* acc, int64_t i0, int64_t i1, int64_t col) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  int64_t i = i0;
  for (; i + kAhead <= i1; i += kAhead) {
    float x[kAhead][P];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load_cols<Tr, VEC>(a, a.sorted_pos[i + u], col, x[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int k = 0; k < P; ++k) acc[k] += x[u][k];
  }
  for (; i < i1; ++i) {
    float x[P];
    load_cols<Tr, VEC>(a, a.sorted_pos[i], col, x);
#pragma unroll
    for (int k = 0; k < P; ++k) acc[k] += x[k];
  }
}

// A lane's P columns end with the row: the last lane's begin before `col`, and
// it stores those from the skip(col)-th on, the ones before are its neighbour's.
template <int P>
__device__ __forceinline__ int skip(const EmbedGradArgs& a, int64_t col) {
  return P > 1 && col + P > a.h ? static_cast<int>(col + P - a.h) : 0;
}

// Stores the P columns of a finished row of dW, but the first `from`.
template <int P, bool ACC>
__device__ __forceinline__ void store_row(const EmbedGradArgs& a, uint32_t v, int64_t col, int from, const float* acc) {
  float* out = a.grad_weight + static_cast<int64_t>(v) * a.h + col;
  if (from > 0) {
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (j >= from) out[j] = ACC ? out[j] + acc[j] * a.scale : acc[j] * a.scale;
  } else if constexpr (P % 4 == 0) {
#pragma unroll
    for (int j = 0; j < P; j += 4) {
      f32x4_a4 x{acc[j] * a.scale, acc[j + 1] * a.scale, acc[j + 2] * a.scale, acc[j + 3] * a.scale};
      f32x4_a4* q = reinterpret_cast<f32x4_a4*>(out + j);
      *q = ACC ? *q + x : x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < P; ++j) out[j] = ACC ? out[j] + acc[j] * a.scale : acc[j] * a.scale;
  }
}

// Workgroups below `parts`: partial rows of the whole blocks that hold one
// token.  The others note where each token's run begins.
template <class Tr, bool VEC>
__global__ void __launch_bounds__(kSumNT) k_embed_partial(EmbedGradArgs a) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  if (blockIdx.x >= a.parts) {
    const int64_t i = static_cast<int64_t>(blockIdx.x - a.parts) * kSumNT + threadIdx.x;
    if (i < a.N) {
      const uint32_t k = a.sorted_keys[i];
      if (k != static_cast<uint32_t>(a.V) && (i == 0 || a.sorted_keys[i - 1] != k)) a.first[k] = static_cast<uint32_t>(i);
    }
    return;
  }
  const int64_t c = blockIdx.x / a.col_blocks + a.row0;
  int64_t col = (static_cast<int64_t>(blockIdx.x % a.col_blocks) * kSumNT + threadIdx.x) * P;
  const uint32_t k = a.sorted_keys[c * kChunk];
  if (k == static_cast<uint32_t>(a.V) || a.sorted_keys[c * kChunk + kChunk - 1] != k || col >= a.h) return;
  col -= skip<P>(a, col);  // what two lanes then store is the same
  float acc[P];
#pragma unroll
  for (int j = 0; j < P; ++j) acc[j] = 0.f;
  add_rows<Tr, VEC, 16>(a, acc, c * kChunk, (c + 1) * kChunk, col);
  float* out = a.partial + c * a.h + col;
#pragma unroll
  for (int j = 0; j < P; ++j) out[j] = acc[j];
}

// Zeros in the rows v0 + k of dW, k the set bits: neighbours among them are one
// stretch of memory, whose stores start on the 128-byte grid.
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, int64_t v0, uint64_t todo) {
  while (todo) {
    const int at = __builtin_ctzll(todo);
    const uint64_t rest = ~(todo >> at);
    const int rows = rest ? __builtin_ctzll(rest) : 64;
    todo = at + rows < 64 ? todo >> (at + rows) << (at + rows) : 0;
    float* out = a.grad_weight + (v0 + at) * a.h;
    const int64_t n = static_cast<int64_t>(rows) * a.h;
    const int64_t lead = (32 - (reinterpret_cast<uintptr_t>(out) >> 2 & 31u)) & 31u, head = lead < n ? lead : n;
    if (static_cast<int64_t>(threadIdx.x) < head) out[threadIdx.x] = 0.f;
    const int64_t vecs = (n - head) / 4;
    u32x4* grid = reinterpret_cast<u32x4*>(out + head);
    for (int64_t j = threadIdx.x; j < vecs; j += kSumNT) grid[j] = u32x4{0, 0, 0, 0};
    const int64_t left = head + vecs * 4 + threadIdx.x;
    if (left < n) out[left] = 0.f;
  }
}

// Zeros in the rows of dW that no token names.
__device__ __forceinline__ void fill_rows(const EmbedGradArgs& a, int64_t block) {
  const int64_t v0 = block * a.fill_rows;
  const int lane = threadIdx.x & 63;
  for (int r0 = 0; r0 < a.fill_rows; r0 += 64) {
    const int64_t v = v0 + r0 + lane;
    zero_rows(a, v0 + r0, __ballot(r0 + lane < a.fill_rows && v < a.V && a.first[v] == kAbsent));
  }
}

// Rows of dW that some token names: a workgroup owns the runs that start in
// its kRunSpan sorted positions, for one block of columns.  Workgroups from
// `parts` on write zeros instead: their stores keep the memory busy while the
// others wait for theirs.
template <class Tr, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumNT) k_embed_runs(EmbedGradArgs a) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  if (!ACC && blockIdx.x >= a.parts) return fill_rows(a, blockIdx.x - a.parts);
  const int64_t p0 = (blockIdx.x / a.col_blocks + a.row0) * kRunSpan;
  const int64_t first_col = (static_cast<int64_t>(blockIdx.x % a.col_blocks) * kSumNT + threadIdx.x) * P;
  const int from = skip<P>(a, first_col);
  const int64_t col = first_col - from;
  const int lane = threadIdx.x & 63;
  const int64_t p = p0 + lane;
  const bool there = lane < kRunSpan && p < a.N;
  const uint32_t key = there ? a.sorted_keys[p] : 0;
  const bool start = there && key != static_cast<uint32_t>(a.V) && (p == 0 || a.sorted_keys[p - 1] != key);
  const uint64_t ends = __ballot(there && (p == 0 || a.sorted_keys[p - 1] != key));  // also the unknown ids' start
  for (uint64_t todo = __ballot(start); todo; todo &= todo - 1) {
    const int at = __builtin_ctzll(todo);
    const uint32_t v = __shfl(key, at, 64);
    const int64_t i = p0 + at;
    const uint64_t later = at < 63 ? ends >> (at + 1) : 0;
    int64_t e;
    if (later) {
      e = i + 1 + __builtin_ctzll(later);
    } else {
      // end of the run: the next 64 positions, then ever finer 64ths of the
      // rest (keys are sorted, so the run's positions come first in a sample)
      e = i;
      int64_t rest = a.N - i, step = 1;
      while (rest > 0) {
        const bool in = (lane + 1) * step <= rest && a.sorted_keys[e + (lane + 1) * step - 1] == v;
        const uint64_t m = __ballot(in);
        const int full = ~m ? __builtin_ctzll(~m) : 64;
        e += full * step;
        rest -= full * step;
        if (step > 1) {
          rest = rest < step - 1 ? rest : step - 1;  // the end lies within the next step
        } else if (full < 64) {
          break;
        }
        step = (rest + 63) / 64;
      }
    }
    if (first_col >= a.h) continue;
    float acc[P];
#pragma unroll
    for (int j = 0; j < P; ++j) acc[j] = 0.f;
    const int64_t c0 = (i + kChunk - 1) / kChunk, c1 = e / kChunk;
    if (c0 < c1) {
      add_rows<Tr, VEC, 8>(a, acc, i, c0 * kChunk, col);
      for (int64_t c = c0; c < c1; ++c) {
        const float* q = a.partial + c * a.h + col;
#pragma unroll
        for (int j = 0; j < P; ++j) acc[j] += q[j];
      }
      add_rows<Tr, VEC, 8>(a, acc, c1 * kChunk, e, col);
    } else {
      add_rows<Tr, VEC, 8>(a, acc, i, e, col);
    }
    store_row<P, ACC>(a, v, col, from, acc);
  }
}

// Up to kTinyN positions, unsorted.  ACC: a workgroup per position, which
// owns the row of its token if no earlier position has it.  Otherwise a
// workgroup per `rows` rows of dW.  A wave holds all tokens in its lanes.
template <class Tr, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumNT) k_embed_tiny(EmbedGradArgs a, int rows) {
  constexpr int P = VEC ? Tr::kPerVec : 1, K = kTinyN / 64;
  const int lane = threadIdx.x & 63;
  uint32_t key[K];
#pragma unroll
  for (int k = 0; k < K; ++k) key[k] = k * 64 + lane < a.N ? key_of(a, k * 64 + lane) : static_cast<uint32_t>(a.V);
  uint64_t absent = 0;  // of the workgroup's rows, at most 64
  for (int r = 0; r < rows; ++r) {
    int64_t v = static_cast<int64_t>(blockIdx.x) * rows + r;
    if (ACC) {
      const int i = static_cast<int>(blockIdx.x);
      v = key_of(a, i);
      if (v == a.V) return;
      bool earlier = false;
#pragma unroll
      for (int k = 0; k < K; ++k) earlier |= k * 64 + lane < i && key[k] == static_cast<uint32_t>(v);
      if (__any(earlier)) return;
    } else if (v >= a.V) {
      break;
    }
    uint64_t hit[K], any = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) any |= hit[k] = __ballot(key[k] == static_cast<uint32_t>(v));
    if (!ACC && !any) {
      absent |= uint64_t(1) << r;
      continue;
    }
    for (int64_t own = static_cast<int64_t>(threadIdx.x) * P; own < a.h; own += kSumNT * P) {
      const int from = skip<P>(a, own);
      const int64_t col = own - from;
      float acc[P];
#pragma unroll
      for (int j = 0; j < P; ++j) acc[j] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        for (uint64_t m = hit[k]; m; m &= m - 1) {
          float x[P];
          load_cols<Tr, VEC>(a, k * 64 + __builtin_ctzll(m), col, x);
#pragma unroll
          for (int j = 0; j < P; ++j) acc[j] += x[j];
        }
      }
      store_row<P, ACC>(a, static_cast<uint32_t>(v), col, from, acc);
    }
  }
  if (!ACC) zero_rows(a, static_cast<int64_t>(blockIdx.x) * rows, absent);
}

template <class Tr, bool VEC>
hipError_t launch_tiny(const EmbedGradArgs& a, hipStream_t s) {
  TimedLaunch tl("k_embedding_grad", s);
  if (a.accumulate) {
    hipLaunchKernelGGL((k_embed_tiny<Tr, VEC, true>), dim3(static_cast<unsigned>(a.N)), dim3(kSumNT), 0, s, a, 1);
  } else {
    // several rows a workgroup once there are workgroups enough to fill the chip
    int rows = a.V / 4096;
    rows = rows < 1 ? 1 : rows > 64 ? 64 : rows;
    hipLaunchKernelGGL((k_embed_tiny<Tr, VEC, false>), dim3((a.V + rows - 1) / rows), dim3(kSumNT), 0, s, a, rows);
  }
  return hipGetLastError();
}

template <class Tr, bool VEC>
hipError_t launch_sums(EmbedGradArgs a, hipStream_t s) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  a.col_blocks = static_cast<int>((a.h + int64_t(kSumNT) * P - 1) / (int64_t(kSumNT) * P));
  TimedLaunch tl("k_embedding_grad", s);
  // workgroups per launch: far below 2^32 work-items
  const int64_t per = (int64_t(1) << 23) / a.col_blocks;
  a.fill_rows = 16 > a.V >> 22 ? 16 : a.V >> 22;
  const int64_t chunks = a.N / kChunk, fills = a.accumulate ? 0 : (int64_t(a.V) + a.fill_rows - 1) / a.fill_rows;
  for (int64_t r0 = 0; r0 < chunks; r0 += per) {
    a.row0 = r0;
    const int64_t n = chunks - r0 < per ? chunks - r0 : per;
    a.parts = static_cast<unsigned>(n * a.col_blocks);
    const int64_t more = a.first && r0 + n == chunks ? (a.N + kSumNT - 1) / kSumNT : 0;
    hipLaunchKernelGGL((k_embed_partial<Tr, VEC>), dim3(static_cast<unsigned>(a.parts + more)), dim3(kSumNT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t spans = (a.N + kRunSpan - 1) / kRunSpan;
  for (int64_t r0 = 0; r0 < spans; r0 += per) {
    a.row0 = r0;
    const int64_t n = spans - r0 < per ? spans - r0 : per;
    a.parts = static_cast<unsigned>(n * a.col_blocks);
    const dim3 g(static_cast<unsigned>(a.parts + (r0 + n == spans ? fills : 0)));
    if (a.accumulate)
      hipLaunchKernelGGL((k_embed_runs<Tr, VEC, true>), g, dim3(kSumNT), 0, s, a);
    else
      hipLaunchKernelGGL((k_embed_runs<Tr, VEC, false>), g, dim3(kSumNT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class Tr>
hipError_t launch_sums_t(const EmbedGradArgs& a, hipStream_t s) {
  // 16 bytes a lane where rows are whole vectors on the 16-byte grid, and for
  // long rows on any boundary; short ones leave too few lanes at work (30000
  // positions, V = 30000 and 1000: h = 257 64 and 50 us by vectors, 61 and 47
  // singly; h = 801 73 and 55, 78 and 51; 32768 x 5119, V = 40000: 299, 492).
  const bool whole = reinterpret_cast<uintptr_t>(a.grad) % 16 == 0 && (a.ld_g * Tr::kBytes) % 16 == 0 &&
                     a.h % Tr::kPerVec == 0;
  const bool vec = whole || a.h >= 768;
  if (a.N <= kTinyN) return vec ? launch_tiny<Tr, true>(a, s) : launch_tiny<Tr, false>(a, s);
  return vec ? launch_sums<Tr, true>(a, s) : launch_sums<Tr, false>(a, s);
}

// Sorting tiles: 512 positions at least, kMaxTiles tiles at most.
void set_tiles(EmbedGradArgs& a) {
  int64_t n = (a.N + 511) / 512;
  n = n < 1 ? 1 : n < kMaxTiles ? n : kMaxTiles;
  a.tile = ((a.N + n - 1) / n + 255) / 256 * 256;
  a.tiles = static_cast<int>((a.N + a.tile - 1) / a.tile);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

bool embedding_workspace_layout(int64_t N, int64_t h, int64_t V, EmbedWorkspace* w) {
  // positions are 32-bit; 2^31 keeps tile and block counts far below 2^32
  if (N < 0 || N > 0x7fffffff || h <= 0 || h > (int64_t(1) << 30) || V <= 0 || V > (int64_t(1) << 30)) return false;
  const size_t n = static_cast<size_t>(N);
  size_t off = 0;
  for (int k = 0; k < 2; ++k) {
    w->keys_off[k] = off;
    off += round256(n * 4);
    w->pos_off[k] = off;
    off += round256(n * 4);
  }
  w->counts_off = off;
  off += round256(size_t(kMaxTiles) * (1 << kMaxDigit) * 4);
  w->first_off = off;
  off += round256(static_cast<size_t>(V) * 4);
  w->partial_off = off;
  off += round256(n / kChunk * static_cast<size_t>(h) * 4);
  w->total = off > 256 ? off : 256;
  return true;
}

hipError_t launch_embedding(int dtype, const EmbedArgs& a, hipStream_t s) {
  int64_t blocks = (a.N + 3) / 4;
  if (blocks > 16384) blocks = 16384;
  TimedLaunch tl("k_embedding", s);
  const dim3 g(static_cast<unsigned>(blocks)), b(256);
  switch (dtype) {
    case 0: hipLaunchKernelGGL(k_embedding<Bf16>, g, b, 0, s, a); break;
    case 1: hipLaunchKernelGGL(k_embedding<Fp16>, g, b, 0, s, a); break;
    default: hipLaunchKernelGGL(k_embedding<Fp32>, g, b, 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_embedding_backward(int dtype, const EmbedGradArgs& args, char* ws, const EmbedWorkspace& w,
                                     hipStream_t s) {
  EmbedGradArgs a = args;
  for (int k = 0; k < 2; ++k) {
    a.keys[k] = reinterpret_cast<uint32_t*>(ws + w.keys_off[k]);
    a.pos[k] = reinterpret_cast<uint32_t*>(ws + w.pos_off[k]);
  }
  a.counts = reinterpret_cast<uint32_t*>(ws + w.counts_off);
  a.first = a.accumulate ? nullptr : reinterpret_cast<uint32_t*>(ws + w.first_off);
  a.partial = reinterpret_cast<float*>(ws + w.partial_off);
  set_tiles(a);
  a.key_bits = 0;
  while ((static_cast<int64_t>(a.V) >> a.key_bits) != 0) ++a.key_bits;  // V itself is the key of unknown ids
  hipError_t e;
  int last = 0;
  if (a.N > kSmallN) {
    TimedLaunch tl("k_embedding_sort", s);
    const int passes = (a.key_bits + kMaxDigit - 1) / kMaxDigit, least = (a.key_bits + passes - 1) / passes;
    const int bits = least < 2 ? 2 : least;
    for (int k = 0, src = -1; k < passes; ++k, src = last) {
      last = src == 0 ? 1 : 0;
      hipLaunchKernelGGL(k_embed_count, dim3(a.tiles), dim3(kSortNT), 0, s, a, k * bits, bits, src);
      hipLaunchKernelGGL(k_embed_scatter, dim3(a.tiles), dim3(kSortNT), 0, s, a, k * bits, bits, src, last);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  } else if (a.N > kTinyN) {
    TimedLaunch tl("k_embedding_sort", s);
    hipLaunchKernelGGL(k_embed_sort_small, dim3(1), dim3(kSmallNT), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  a.sorted_keys = a.keys[last];
  a.sorted_pos = a.pos[last];
  switch (dtype) {
    case 0: return launch_sums_t<Bf16>(a, s);
    case 1: return launch_sums_t<Fp16>(a, s);
    default: return launch_sums_t<Fp32>(a, s);
  }
}

}  // namespace lp
