// Logit rules (penalties for repeated tokens, sparse biases, a grammar mask)
// and what is computed under them: the processed logits, the log-prob and
// entropy of the distribution they leave, and the gradient with respect to
// the raw logits.
//
// Row t, column j, with n = times j stands in the row's output and
// seen = j stands in its prompt or output:
//   z1 = seen ? (z > 0 ? z / rho : z * rho) : z
//   z2 = z1 - f * n          z3 = z2 - p * (n > 0)
//   z4 = z3 + b_j            z5 = allowed_j ? z4 : -inf
// each step one fp32 operation, rounded on its own (no contraction).
//
// The row is cut into slices of columns, one workgroup each.  A workgroup
// counts the history tokens that fall into its slice in an LDS word per
// column (bit 31: stands in the prompt; below: times in the output), then
// streams the slice.  Counts are integers, so the order of the LDS atomics
// does not change any result.  Nothing of size V is kept between calls and no
// dense count matrix passes through memory: a dense one would cost 4 bytes a
// column where the logits themselves cost 2.  Every slice rereads the row's
// history (4 bytes a token, from L2).
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr uint32_t kPromptBit = 0x80000000u;
constexpr int kLdsPad = 16;

enum RulesOp { kProcess = 0, kScore = 1, kGrad = 2 };

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Like stat_push with guards for -inf (weight 0, adds nothing to `a`); a NaN
// stays a NaN in s and a.
template <int N>
__device__ __forceinline__ void stat_push_masked(Stat& st, const float* x, float c) {
  float vm = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) vm = fmaxf(vm, x[k]);
  const float vmc = vm * c;
  if (vmc > st.mc) stat_rebase(st, vmc);
  const float nmc = -st.mc;
  float ps = 0.f, pa = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float t = fmaf(x[k], c, nmc);
    const float e = fast_exp2(t);
    ps += e;
    pa = fmaf(e, t == neg_inf() ? 0.f : t, pa);
  }
  st.s += ps;
  st.a += pa;
}

// Merge in which an empty side (s == 0) adds nothing and a NaN side wins.
__device__ __forceinline__ Stat stat_merge_nan(Stat x, Stat y) {
  const float mc = fmaxf(x.mc, y.mc);
  float s = 0.f, a = 0.f;
  if (x.s != 0.f) {
    const float d = x.mc - mc, r = fast_exp2(d);
    s += x.s * r;
    a += (x.a + x.s * d) * r;
  }
  if (y.s != 0.f) {
    const float d = y.mc - mc, r = fast_exp2(d);
    s += y.s * r;
    a += (y.a + y.s * d) * r;
  }
  return Stat{mc, s, a};
}

__device__ __forceinline__ Stat stat_wave_merge_nan(Stat st) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    Stat o;
    o.mc = __shfl_xor(st.mc, off, 64);
    o.s = __shfl_xor(st.s, off, 64);
    o.a = __shfl_xor(st.a, off, 64);
    st = stat_merge_nan(st, o);
  }
  return st;
}

// One row's scalars.
struct RowRules {
  float rho, f, p;
  const uint32_t* words;  // LDS words of the slice, or null: no history
  const uint32_t* bias;   // LDS: 1 + list position of the column's bias, 0 = none; or null
  const float* values;    // the row's bias values
  const uint32_t* allowed;
  // gradient
  float g, gh, nlse2, H, c, inv_tau;
  int64_t y;
};

// Rules on N columns from `col`, whose LDS words start at `at`.  slope: d
// processed / d raw (kGrad only).  Returns a bit per column: 1 = not allowed.
template <int N, bool SLOPE>
__device__ __forceinline__ uint32_t apply_rules(const RowRules& r, float* z, float* slope, int at, int col) {
  if (SLOPE) {
#pragma unroll
    for (int k = 0; k < N; ++k) slope[k] = 1.f;
  }
  if (r.words) {
    uint32_t w[N];
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(r.words + at + k);
        w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) w[k] = r.words[at + k];
    }
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) any |= w[k];
    if (any) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (w[k]) {
          const bool up = z[k] > 0.f;
          if (SLOPE) slope[k] = up ? __frcp_rn(r.rho) : r.rho;
          z[k] = up ? __fdiv_rn(z[k], r.rho) : __fmul_rn(z[k], r.rho);
          const uint32_t n = w[k] & ~kPromptBit;
          if (n) z[k] = __fsub_rn(__fsub_rn(z[k], __fmul_rn(r.f, static_cast<float>(n))), r.p);
        }
      }
    }
  }
  if (r.bias) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t w = r.bias[at + k];
      if (w) z[k] = __fadd_rn(z[k], r.values[w - 1]);
    }
  }
  uint32_t shut = 0;
  if (r.allowed) {
    const int wi = col >> 5, sh = col & 31;
    uint32_t bits = r.allowed[wi] >> sh;
    if (N > 1 && sh > 32 - N) bits |= r.allowed[wi + 1] << (32 - sh);
    shut = ~bits;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if ((shut >> k) & 1u) z[k] = neg_inf();
  }
  return shut;
}

// dL/draw of N columns from `col`; z holds the processed logits on entry.  A
// column that is not allowed gets 0 whatever its value and the row's.
template <int N>
__device__ __forceinline__ void grad_cols(const RowRules& r, float* z, const float* slope, uint32_t shut, int col) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float t = fmaf(z[k], r.c, r.nlse2);
    const float p = fast_exp2(t);
    const float lt = t == neg_inf() ? 0.f : t * kLn2;
    float d = -p * fmaf(r.gh, lt + r.H, r.g);
    if (col + k == r.y) d += r.g;
    d = d * r.inv_tau * slope[k];
    z[k] = (shut >> k) & 1u ? 0.f : d;
  }
}

template <class Tr, int OP, int N>
__device__ __forceinline__ void finish_cols(const RowRules& r, float* z, Stat& st, int at, int col) {
  float slope[N];
  const uint32_t shut = apply_rules<N, OP == kGrad>(r, z, slope, at, col);
  if (OP == kScore) stat_push_masked<N>(st, z, r.c);
  if (OP == kGrad) grad_cols<N>(r, z, slope, shut, col);
}

template <class Tr, int OP, int NT, int U>
__global__ void __launch_bounds__(NT) k_rules(RulesArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int P = Tr::kPerVec;
  const int tid = threadIdx.x;
  const unsigned rel = blockIdx.x / static_cast<unsigned>(a.nslices);
  const int slice = static_cast<int>(blockIdx.x - rel * static_cast<unsigned>(a.nslices));
  const int64_t row = a.row0 + rel;
  const int c0 = slice * a.slice;
  const int n = a.V - c0 < a.slice ? a.V - c0 : a.slice;
  const char* xp = static_cast<const char*>(a.x) + (row * a.ld + c0) * Tr::kBytes;
  char* op = OP == kScore ? nullptr : static_cast<char*>(a.out) + (row * a.ld_out + c0) * Tr::kBytes;
  if (a.mask && a.mask[row] == 0) {
    if (OP == kGrad) {
      const RowSplit<Tr> sp(op, n);
      if (tid < sp.head) Tr::store1(op, tid, 0.f);
      u32x4* vp = reinterpret_cast<u32x4*>(op + sp.head * Tr::kBytes);
      for (int i = tid; i < sp.nvec; i += NT) vp[i] = u32x4{0, 0, 0, 0};
      if (tid < sp.tail) Tr::store1(op, sp.head + sp.nvec * P + tid, 0.f);
    }
    return;
  }
  // Columns [0, head) and the tail go one by one, the rest as 16-byte vectors;
  // where input and output rows differ in their 16-byte phase, all go singly.
  RowSplit<Tr> sp(xp, n);
  if (OP != kScore && ((reinterpret_cast<uintptr_t>(xp) ^ reinterpret_cast<uintptr_t>(op)) & 15u)) {
    sp.head = 0;
    sp.nvec = 0;
    sp.tail = n;
  }
  const int base = 8 - sp.head;  // LDS position of column c0: vectors start at a multiple of 8

  RowRules r;
  r.rho = a.repetition ? a.repetition[row] : 1.f;
  r.f = a.frequency ? a.frequency[row] : 0.f;
  r.p = a.presence ? a.presence[row] : 0.f;
  r.words = nullptr;
  r.bias = nullptr;
  r.values = nullptr;
  r.allowed = a.allowed ? a.allowed + row * a.ld_allowed : nullptr;
  r.c = a.c;
  if (OP == kGrad) {
    r.g = a.grad_logprob[row];
    r.gh = a.grad_entropy ? a.grad_entropy[row] : 0.f;
    r.nlse2 = -a.lse[row] * kLog2e;
    r.H = a.grad_entropy ? a.entropy[row] : 0.f;
    r.inv_tau = a.inv_tau;
    r.y = a.targets[row];
  }

  int64_t len = 0, buf = row, b0 = 0, nb = 0;
  if (a.tokens) {
    if (a.row_buffer) buf = a.row_buffer[row];
    len = a.hist_len[row];
    len = len < a.max_len ? len : a.max_len;
    if (buf < 0 || buf >= a.buffers) len = 0;
  }
  if (a.bias_offsets) {
    b0 = a.bias_offsets[row];
    int64_t b1 = a.bias_offsets[row + 1];
    b0 = b0 > 0 ? b0 : 0;
    b1 = b1 < a.bias_count ? b1 : a.bias_count;
    nb = b1 > b0 ? b1 - b0 : 0;
  }
  const int span = n + kLdsPad;
  uint32_t* words = lds;
  uint32_t* bias = lds + (a.tokens ? a.slice + kLdsPad : 0);
  if (len > 0) {
    r.words = words;
    for (int i = tid; i < span; i += NT) words[i] = 0;
  }
  if (nb > 0) {
    r.bias = bias;
    r.values = a.bias_values + b0;
    for (int i = tid; i < span; i += NT) bias[i] = 0;
  }
  if (len > 0 || nb > 0) {  // the same for the whole workgroup
    __syncthreads();
    if (len > 0) {
      const int32_t* tok = a.tokens + buf * a.ld_tokens;
      const int64_t prompt = a.prompt_len ? a.prompt_len[row] : 0;
#pragma unroll 4
      for (int64_t i = tid; i < len; i += NT) {
        // a token outside the vocabulary is negative or past every slice
        const int64_t j = static_cast<int64_t>(tok[i]) - c0;
        if (j >= 0 && j < n) {
          if (i < prompt)
            atomicOr(words + base + j, kPromptBit);
          else
            atomicAdd(words + base + j, 1u);
        }
      }
    }
    // the last entry listed for a column counts
    for (int64_t i = tid; i < nb; i += NT) {
      const int64_t j = static_cast<int64_t>(a.bias_tokens[b0 + i]) - c0;
      if (j >= 0 && j < n) atomicMax(bias + base + j, static_cast<uint32_t>(i) + 1u);
    }
    __syncthreads();
  }

  Stat st = stat_empty();
  if (tid < sp.head) {
    float z = Tr::load1(xp, tid);
    finish_cols<Tr, OP, 1>(r, &z, st, base + tid, c0 + tid);
    if (OP != kScore) Tr::store1(op, tid, z);
  }
  const u32x4* vp = reinterpret_cast<const u32x4*>(xp + sp.head * Tr::kBytes);
  u32x4* wp = reinterpret_cast<u32x4*>(op + sp.head * Tr::kBytes);
  int i = tid;
  for (; i + (U - 1) * NT < sp.nvec; i += U * NT) {
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = __builtin_nontemporal_load(vp + i + u * NT);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[P];
      Tr::unpack(w[u], z);
      const int at = (i + u * NT) * P;
      finish_cols<Tr, OP, P>(r, z, st, 8 + at, c0 + sp.head + at);
      if (OP != kScore) __builtin_nontemporal_store(Tr::pack(z), wp + i + u * NT);
    }
  }
  for (; i < sp.nvec; i += NT) {
    float z[P];
    Tr::unpack(__builtin_nontemporal_load(vp + i), z);
    finish_cols<Tr, OP, P>(r, z, st, 8 + i * P, c0 + sp.head + i * P);
    if (OP != kScore) __builtin_nontemporal_store(Tr::pack(z), wp + i);
  }
  for (int j = n - sp.tail + tid; j < n; j += NT) {
    float z = Tr::load1(xp, j);
    finish_cols<Tr, OP, 1>(r, &z, st, base + j, c0 + j);
    if (OP != kScore) Tr::store1(op, j, z);
  }

  if (OP == kScore) {
    __shared__ Stat sm[NT / 64];
    st = stat_wave_merge_nan(st);
    if ((tid & 63) == 0) sm[tid >> 6] = st;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int k = 1; k < NT / 64; ++k) st = stat_merge_nan(st, sm[k]);
      float* pt = a.part + (row * a.nslices + slice) * 3;
      pt[0] = st.mc;
      pt[1] = st.s;
      pt[2] = st.a;
      const int64_t y = a.targets[row];
      if (y >= c0 && y < c0 + n) {
        const int j = static_cast<int>(y) - c0;
        float z = Tr::load1(xp, j);
        float unused;
        apply_rules<1, false>(r, &z, &unused, base + j, static_cast<int>(y));
        a.zy[row] = z;
      }
    }
  }
}

// One wave per row: the slices' states in a fixed order, then the outputs.
__global__ void __launch_bounds__(256) k_rules_join(RulesArgs a) {
  const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.T) return;
  if (a.mask && a.mask[row] == 0) {
    if (lane == 0) {
      a.logprob[row] = 0.f;
      if (a.entropy_out) a.entropy_out[row] = 0.f;
      if (a.lse_out) a.lse_out[row] = 0.f;
    }
    return;
  }
  Stat st = stat_empty();
  for (int i = lane; i < a.nslices; i += 64) {
    const float* pt = a.part + (row * a.nslices + i) * 3;
    st = stat_merge_nan(st, Stat{pt[0], pt[1], pt[2]});
  }
  st = stat_wave_merge_nan(st);
  if (lane == 0) {
    const float l2s = log2f(st.s);
    const int64_t y = a.targets[row];
    float lp = __builtin_nanf("");
    if (y >= 0 && y < a.V) lp = (fmaf(a.zy[row], a.c, -st.mc) - l2s) * kLn2;
    a.logprob[row] = lp;
    if (a.entropy_out) a.entropy_out[row] = (l2s - st.a / st.s) * kLn2;
    if (a.lse_out) a.lse_out[row] = (st.mc + l2s) * kLn2;
  }
}

// Columns per workgroup: the widest slice that still gives every CU four
// workgroups, so that long calls reread the history few times and a single
// decode row still spreads over the chip.
int slice_of(int64_t T, int64_t V) {
  for (int s : {4096, 2048})
    if (T * ((V + s - 1) / s) >= 1024) return s;
  return 1024;
}

template <class Tr, int OP>
hipError_t launch_rules_t(const RulesArgs& args, const char* name, hipStream_t s) {
  constexpr int NT = 256;
  RulesArgs a = args;
  a.slice = slice_of(a.T, a.V);
  a.nslices = static_cast<int>((int64_t(a.V) + a.slice - 1) / a.slice);
  const size_t lds = size_t(a.slice + kLdsPad) * 4 * ((a.tokens ? 1 : 0) + (a.bias_offsets ? 1 : 0));
  // workgroups of a launch: far below 2^32 work-items whatever T
  const int64_t rows_per = (int64_t(1) << 22) / a.nslices > 0 ? (int64_t(1) << 22) / a.nslices : 1;
  for (int64_t r0 = 0; r0 < a.T; r0 += rows_per) {
    const int64_t rows = a.T - r0 < rows_per ? a.T - r0 : rows_per;
    a.row0 = r0;
    TimedLaunch tl(name, s);
    hipLaunchKernelGGL((k_rules<Tr, OP, NT, 2>), dim3(static_cast<unsigned>(rows * a.nslices)), dim3(NT), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int OP>
hipError_t launch_rules(int dtype, const RulesArgs& a, const char* name, hipStream_t s) {
  switch (dtype) {
    case 0: return launch_rules_t<Bf16, OP>(a, name, s);
    case 1: return launch_rules_t<Fp16, OP>(a, name, s);
    default: return launch_rules_t<Fp32, OP>(a, name, s);
  }
}

}  // namespace

size_t processed_workspace_bytes(int64_t T, int64_t V) {
  const int64_t slice = slice_of(T, V);
  const int64_t ns = (V + slice - 1) / slice;
  const size_t per_row = size_t(ns) * 12 + 4;
  if (size_t(T) > (size_t(1) << 60) / per_row) return 0;
  return (size_t(T) * per_row + 255) / 256 * 256;
}

hipError_t launch_process_logits(int dtype, const RulesArgs& a, hipStream_t s) {
  return launch_rules<kProcess>(dtype, a, "k_process_logits", s);
}

hipError_t launch_processed_score(int dtype, const RulesArgs& args, char* ws, hipStream_t s) {
  RulesArgs a = args;
  a.slice = slice_of(a.T, a.V);
  a.nslices = static_cast<int>((int64_t(a.V) + a.slice - 1) / a.slice);
  a.part = reinterpret_cast<float*>(ws);
  a.zy = a.part + a.T * a.nslices * 3;
  hipError_t e = launch_rules<kScore>(dtype, a, "k_processed_score", s);
  if (e != hipSuccess) return e;
  constexpr int64_t kRows = int64_t(1) << 22;
  for (int64_t r0 = 0; r0 < a.T; r0 += kRows) {
    RulesArgs b = a;
    b.row0 = r0;
    const int64_t rows = a.T - r0 < kRows ? a.T - r0 : kRows;
    TimedLaunch tl("k_processed_join", s);
    hipLaunchKernelGGL(k_rules_join, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s, b);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_processed_grad(int dtype, const RulesArgs& a, hipStream_t s) {
  return launch_rules<kGrad>(dtype, a, "k_processed_grad", s);
}

}  // namespace lp
