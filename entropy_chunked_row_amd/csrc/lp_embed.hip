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
// positions before and after them.  A run's length so costs its owner
// length / kChunk + 2 kChunk additions.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kChunk = 64;       // sorted positions per partial row
constexpr int kSortNT = 256;     // threads of a sorting workgroup
constexpr int kSortTile = 2048;  // positions per sorting workgroup
constexpr int kSmallN = 4096;    // sorted by one workgroup in LDS up to here
constexpr int kSmallNT = 1024;

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
    RowSplit<Tr> sp(src, a.h);
    if ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) {
      sp.head = 0;
      sp.nvec = 0;
      sp.tail = a.h;
    }
    if (lane < sp.head) Tr::store1(dst, lane, known ? Tr::load1(src, lane) * a.scale : 0.f);
    const u32x4* vp = reinterpret_cast<const u32x4*>(src + sp.head * Tr::kBytes);
    u32x4* wp = reinterpret_cast<u32x4*>(dst + sp.head * Tr::kBytes);
    for (int j = lane; j < sp.nvec; j += 64) {
      float x[P];
      Tr::unpack(vp[j], x);
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

// Lanes of the wave with the same 8-bit digit (among live lanes).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool live) {
  uint64_t m = __ballot(live);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
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
  const int share = ((n + W - 1) / W + 63) / 64 * 64;
  const int i0 = w * share, i1 = i0 + share < n ? i0 + share : n;
  int cur = 0;
  for (int shift = 0; shift < a.key_bits; shift += 8, cur ^= 1) {
    for (int i = tid; i < W * 256; i += kSmallNT) (&cnt[0][0])[i] = 0;
    __syncthreads();
    for (int i = i0; i < i1; i += 64) {
      const bool live = i + lane < i1;
      const uint32_t d = live ? (key[cur][i + lane] >> shift) & 255u : 0;
      const uint64_t m = same_digit(d, live);
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
      const uint64_t m = same_digit(d, live);
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
    a.keys[0][i] = key[cur][i];
    a.pos[0][i] = pos[cur][i];
  }
}

// One pass over 8 bits of the keys, three kernels: digit counts per tile,
// their scan in (digit, tile) order, and the stable scatter.
__device__ __forceinline__ uint32_t load_key(const EmbedGradArgs& a, int src, int64_t i) {
  return src < 0 ? key_of(a, i) : a.keys[src][i];
}

__global__ void __launch_bounds__(kSortNT) k_embed_count(EmbedGradArgs a, int shift, int src) {
  __shared__ uint32_t cnt[256];
  cnt[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kSortTile;
#pragma unroll
  for (int k = 0; k < kSortTile / kSortNT; ++k) {
    const int64_t i = t0 + k * kSortNT + threadIdx.x;
    if (i < a.N) atomicAdd(&cnt[(load_key(a, src, i) >> shift) & 255u], 1u);
  }
  __syncthreads();
  a.counts[static_cast<int64_t>(threadIdx.x) * a.tiles + blockIdx.x] = cnt[threadIdx.x];
}

// Exclusive scan of 256 x tiles counts by one workgroup.
__global__ void __launch_bounds__(1024) k_embed_scan(EmbedGradArgs a) {
  __shared__ uint32_t wsum[16];
  const int64_t n = static_cast<int64_t>(a.tiles) * 256;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 4096) {
    const int64_t i = i0 + threadIdx.x * 4;  // n is a multiple of 256
    u32x4 v{0, 0, 0, 0};
    if (i < n) v = *reinterpret_cast<const u32x4*>(a.counts + i);
    const uint32_t s = v.x + v.y + v.z + v.w;
    uint32_t x = s;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) wsum[w] = x;
    __syncthreads();
    uint32_t before = carry, total = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < w) before += wsum[k];
      total += wsum[k];
    }
    carry += total;
    uint32_t e = before + x - s;
    if (i < n) *reinterpret_cast<u32x4*>(a.counts + i) = u32x4{e, e + v.x, e + v.x + v.y, e + v.x + v.y + v.z};
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortNT) k_embed_scatter(EmbedGradArgs a, int shift, int src, int dst) {
  constexpr int W = kSortNT / 64, kShare = kSortTile / W;
  __shared__ uint32_t cnt[W][256];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < W; ++k) cnt[k][threadIdx.x] = 0;
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kSortTile + w * kShare;
  uint32_t kx[kShare / 64];
#pragma unroll
  for (int k = 0; k < kShare / 64; ++k) {
    const int64_t i = s0 + k * 64 + lane;
    kx[k] = i < a.N ? load_key(a, src, i) : 0;
  }
#pragma unroll
  for (int k = 0; k < kShare / 64; ++k) {
    const bool live = s0 + k * 64 + lane < a.N;
    const uint32_t d = (kx[k] >> shift) & 255u;
    const uint64_t m = same_digit(d, live);
    if (live && lanes_below(m) == 0) cnt[w][d] += __popcll(m);
    wave_sync();
  }
  __syncthreads();
  uint32_t s = a.counts[static_cast<int64_t>(threadIdx.x) * a.tiles + blockIdx.x];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const uint32_t c = cnt[k][threadIdx.x];
    cnt[k][threadIdx.x] = s;
    s += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kShare / 64; ++k) {
    const int64_t i = s0 + k * 64 + lane;
    const bool live = i < a.N;
    const uint32_t d = (kx[k] >> shift) & 255u;
    const uint64_t m = same_digit(d, live);
    const int below = lanes_below(m);
    const uint32_t at = cnt[w][d] + below;
    wave_sync();
    if (live && below == 0) cnt[w][d] += __popcll(m);
    wave_sync();
    if (live) {
      a.keys[dst][at] = kx[k];
      a.pos[dst][at] = src < 0 ? static_cast<uint32_t>(i) : a.pos[src][i];
    }
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------

// First sorted position of each token (0xffffffff: not there), for the form
// that writes every row of dW.
__global__ void __launch_bounds__(256) k_embed_clear(uint32_t* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0xffffffffu;
}

__global__ void __launch_bounds__(256) k_embed_first(EmbedGradArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.N) return;
  const uint32_t k = a.sorted_keys[i];
  if (k < static_cast<uint32_t>(a.V) && (i == 0 || a.sorted_keys[i - 1] != k)) a.first[k] = static_cast<uint32_t>(i);
}

// acc[0..P) += the P columns from `col` of the gradients at sorted positions
// [i0, i1), in that order.
template <class Tr, bool VEC>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, float* acc, int64_t i0, int64_t i1, int64_t col) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  int64_t i = i0;
  for (; i + 4 <= i1; i += 4) {
    float x[4][P];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const char* p = static_cast<const char*>(a.grad) + static_cast<int64_t>(a.sorted_pos[i + u]) * a.ld_g * Tr::kBytes;
      if constexpr (VEC)
        Tr::unpack(*reinterpret_cast<const u32x4*>(p + col * Tr::kBytes), x[u]);
      else
        x[u][0] = Tr::load1(p, col);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < P; ++k) acc[k] += x[u][k];
  }
  for (; i < i1; ++i) {
    float x[P];
    const char* p = static_cast<const char*>(a.grad) + static_cast<int64_t>(a.sorted_pos[i]) * a.ld_g * Tr::kBytes;
    if constexpr (VEC)
      Tr::unpack(*reinterpret_cast<const u32x4*>(p + col * Tr::kBytes), x);
    else
      x[0] = Tr::load1(p, col);
#pragma unroll
    for (int k = 0; k < P; ++k) acc[k] += x[k];
  }
}

// Partial rows of the whole blocks that hold one token.
template <class Tr, bool VEC, int NT>
__global__ void __launch_bounds__(NT) k_embed_partial(EmbedGradArgs a) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  const int64_t c = blockIdx.x / a.col_blocks + a.row0;
  const int64_t col = (static_cast<int64_t>(blockIdx.x % a.col_blocks) * NT + threadIdx.x) * P;
  const uint32_t k = a.sorted_keys[c * kChunk];
  if (k == static_cast<uint32_t>(a.V) || a.sorted_keys[c * kChunk + kChunk - 1] != k || col >= a.h) return;
  float acc[P];
#pragma unroll
  for (int j = 0; j < P; ++j) acc[j] = 0.f;
  add_rows<Tr, VEC>(a, acc, c * kChunk, (c + 1) * kChunk, col);
  float* out = a.partial + c * a.h + col;
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (col + j < a.h) out[j] = acc[j];
}

// One workgroup per row of dW and column block.  ACC: the rows that some
// position names, found as run starts; otherwise every row.
template <class Tr, bool VEC, bool ACC, int NT>
__global__ void __launch_bounds__(NT) k_embed_rows(EmbedGradArgs a) {
  constexpr int P = VEC ? Tr::kPerVec : 1;
  const int64_t b = blockIdx.x / a.col_blocks + a.row0;
  const int64_t col = (static_cast<int64_t>(blockIdx.x % a.col_blocks) * NT + threadIdx.x) * P;
  int64_t i = b;
  uint32_t v;
  if (ACC) {
    v = a.sorted_keys[i];
    if (v == static_cast<uint32_t>(a.V) || (i > 0 && a.sorted_keys[i - 1] == v)) return;
  } else {
    v = static_cast<uint32_t>(b);
    const uint32_t f = a.first[b];
    i = f == 0xffffffffu ? a.N : f;
  }
  // end of the run: the next 64 positions, then ever finer 64ths of the rest
  // (keys are sorted, so the run's positions come first in every sample)
  int64_t e = i, rest = a.N - i, step = 1;
  const int lane = threadIdx.x & 63;
  while (rest > 0) {
    const bool in = (lane + 1) * step <= rest && a.sorted_keys[e + (lane + 1) * step - 1] == v;
    const uint64_t m = __ballot(in);
    const int full = ~m ? __builtin_ctzll(~m) : 64;
    e += full * step;
    rest -= full * step;
    if (step > 1) {
      // the end lies within the next step
      rest = rest < step - 1 ? rest : step - 1;
      step = (rest + 63) / 64;
    } else {
      if (full < 64) break;
      step = (rest + 63) / 64;
    }
  }
  if (col >= a.h) return;
  float acc[P];
#pragma unroll
  for (int j = 0; j < P; ++j) acc[j] = 0.f;
  const int64_t c0 = (i + kChunk - 1) / kChunk, c1 = e / kChunk;
  if (c0 < c1) {
    add_rows<Tr, VEC>(a, acc, i, c0 * kChunk, col);
    for (int64_t c = c0; c < c1; ++c) {
      const float* p = a.partial + c * a.h + col;
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (col + j < a.h) acc[j] += p[j];
    }
    add_rows<Tr, VEC>(a, acc, c1 * kChunk, e, col);
  } else {
    add_rows<Tr, VEC>(a, acc, i, e, col);
  }
  float* out = a.grad_weight + static_cast<int64_t>(v) * a.h + col;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (col + j < a.h) {
      const float x = acc[j] * a.scale;
      out[j] = ACC ? out[j] + x : x;
    }
  }
}

template <class Tr, bool VEC>
hipError_t launch_sums(EmbedGradArgs a, hipStream_t s) {
  constexpr int NT = 128;
  constexpr int P = VEC ? Tr::kPerVec : 1;
  a.col_blocks = static_cast<int>((a.h + int64_t(NT) * P - 1) / (int64_t(NT) * P));
  TimedLaunch tl("k_embedding_grad", s);
  // workgroups per launch: far below 2^32 work-items
  const int64_t per = (int64_t(1) << 23) / a.col_blocks;
  const int64_t chunks = a.N / kChunk;
  for (int64_t r0 = 0; r0 < chunks; r0 += per) {
    a.row0 = r0;
    const int64_t n = chunks - r0 < per ? chunks - r0 : per;
    hipLaunchKernelGGL((k_embed_partial<Tr, VEC, NT>), dim3(static_cast<unsigned>(n * a.col_blocks)), dim3(NT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t rows = a.accumulate ? a.N : a.V;
  for (int64_t r0 = 0; r0 < rows; r0 += per) {
    a.row0 = r0;
    const int64_t n = rows - r0 < per ? rows - r0 : per;
    const dim3 g(static_cast<unsigned>(n * a.col_blocks));
    if (a.accumulate)
      hipLaunchKernelGGL((k_embed_rows<Tr, VEC, true, NT>), g, dim3(NT), 0, s, a);
    else
      hipLaunchKernelGGL((k_embed_rows<Tr, VEC, false, NT>), g, dim3(NT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

template <class Tr>
hipError_t launch_sums_t(const EmbedGradArgs& a, hipStream_t s) {
  // 16-byte loads need every gradient row on the 16-byte grid and whole vectors
  const bool vec = reinterpret_cast<uintptr_t>(a.grad) % 16 == 0 && (a.ld_g * Tr::kBytes) % 16 == 0 &&
                   a.h % Tr::kPerVec == 0;
  return vec ? launch_sums<Tr, true>(a, s) : launch_sums<Tr, false>(a, s);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

bool embedding_workspace_layout(int64_t N, int64_t h, int64_t V, EmbedWorkspace* w) {
  // positions are 32-bit; 2^31 keeps tile and block counts far below 2^32
  if (N < 0 || N > 0x7fffffff || h <= 0 || h > (int64_t(1) << 30) || V <= 0 || V > (int64_t(1) << 30)) return false;
  const size_t n = static_cast<size_t>(N), tiles = (n + kSortTile - 1) / kSortTile;
  size_t off = 0;
  for (int k = 0; k < 2; ++k) {
    w->keys_off[k] = off;
    off += round256(n * 4);
    w->pos_off[k] = off;
    off += round256(n * 4);
  }
  w->counts_off = off;
  off += round256(tiles * 256 * 4);
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
  a.first = reinterpret_cast<uint32_t*>(ws + w.first_off);
  a.partial = reinterpret_cast<float*>(ws + w.partial_off);
  a.tiles = static_cast<int>((a.N + kSortTile - 1) / kSortTile);
  a.key_bits = 0;
  while ((static_cast<int64_t>(a.V) >> a.key_bits) != 0) ++a.key_bits;  // V itself is the key of unknown ids
  hipError_t e;
  int last = 0;
  if (a.N <= kSmallN) {
    TimedLaunch tl("k_embedding_sort", s);
    hipLaunchKernelGGL(k_embed_sort_small, dim3(1), dim3(kSmallNT), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    TimedLaunch tl("k_embedding_sort", s);
    int src = -1;
    for (int shift = 0; shift < a.key_bits; shift += 8) {
      last = src == 0 ? 1 : 0;
      hipLaunchKernelGGL(k_embed_count, dim3(a.tiles), dim3(kSortNT), 0, s, a, shift, src);
      hipLaunchKernelGGL(k_embed_scan, dim3(1), dim3(1024), 0, s, a);
      hipLaunchKernelGGL(k_embed_scatter, dim3(a.tiles), dim3(kSortNT), 0, s, a, shift, src, last);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      src = last;
    }
  }
  a.sorted_keys = a.keys[last];
  a.sorted_pos = a.pos[last];
  if (!a.accumulate) {
    hipLaunchKernelGGL(k_embed_clear, dim3(static_cast<unsigned>((a.V + 255) / 256)), dim3(256), 0, s, a.first,
                       static_cast<int64_t>(a.V));
    if (a.N > 0)
      hipLaunchKernelGGL(k_embed_first, dim3(static_cast<unsigned>((a.N + 255) / 256)), dim3(256), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  switch (dtype) {
    case 0: return launch_sums_t<Bf16>(a, s);
    case 1: return launch_sums_t<Fp16>(a, s);
    default: return launch_sums_t<Fp32>(a, s);
  }
}

}  // namespace lp
