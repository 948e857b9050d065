// Distillation from a teacher's top logits: KL from a list of K entries a row,
// and on request the mass outside it, to the student's whole row, and the
// gradient with respect to the student's raw logits.
//
//   p_k = exp(t_k), P = sum p_k over entries inside the vocabulary, r = exp(t_rest)
//   loss = sum_k p_k (t_k - log q_{id_k}) + r (t_rest - (lse_rest - lse))
// with q = softmax(z / tau) and lse_rest the log-sum-exp over the columns that no
// entry names.  With m = P + r, r_q = exp(lse_rest - lse) and g = grad / tau,
//   d loss / d z_j = g (q_j m - sum of p_k over entries that name j)   listed
//                  = g w_j (m r_q - r),  w_j = exp(z_j / tau - lse_rest)  others
// (q_j m - r w_j, of which neither part can overflow this way).
//
// A row is read once.  The listed columns lie in at most K of its 16-byte
// vectors.  A lane streams vectors tid, tid + NT, ... of its slice, at most 64
// of them, so which of its own are listed fits one 64-bit word, set in LDS
// before the stream: a vector costs one bit test.  Listed vectors are left out
// of the stream; each is taken by the first entry that lies in it, which looks
// through the list for the others: so an id listed twice counts once in the
// sums and with both its masses in the gradient, in a fixed order, and the sum over
// unlisted columns is a sum of its own.
#include "lp_internal.hpp"
#include "lp_sums.hpp"

namespace lp {

namespace {

constexpr int kMinDistillSlice = 2048;

// Where a slice's vectors lie: vector v holds columns v P - pad .. + P, those
// outside [0, n) missing at either end.  The gradient takes pad from its output,
// so that whole vectors are stored on the 16-byte grid.
template <class Tr>
struct Vectors {
  static constexpr int P = Tr::kPerVec;
  int n, pad;
  __device__ __forceinline__ int first() const { return pad ? 1 : 0; }
  __device__ __forceinline__ int whole_end() const { return (n + pad) / P; }
  __device__ __forceinline__ int end() const { return (n + pad + P - 1) / P; }
  __device__ __forceinline__ bool whole(int v) const { return v >= first() && v < whole_end(); }
  __device__ __forceinline__ u32x4 load(const char* xp, int v) const {
    if (whole(v)) return load_vec(xp + (static_cast<int64_t>(v) * P - pad) * Tr::kBytes);
    float x[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = v * P - pad + k;
      x[k] = j >= 0 && j < n ? Tr::load1(xp, j) : neg_inf();
    }
    return Tr::pack(x);
  }
  __device__ __forceinline__ void store(char* op, int v, const float* x) const {
    if (whole(v)) {
      __builtin_nontemporal_store(Tr::pack(x), reinterpret_cast<u32x4*>(op + (static_cast<int64_t>(v) * P - pad) * Tr::kBytes));
      return;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = v * P - pad + k;
      if (j >= 0 && j < n) Tr::store1(op, j, x[k]);
    }
  }
};

__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// By one wave: the outputs of a row from the states of its unlisted and its
// listed columns.  The loss is a difference of nearly equal numbers: fp64.
template <class Tr>
__device__ void store_loss(const DistillArgs& a, int64_t row, SumStat rest, SumStat listed) {
  const int lane = threadIdx.x & 63;
  const char* xp = static_cast<const char*>(a.x) + row * a.ld * Tr::kBytes;
  const double lse = sum_lse(sum_add(rest, listed, a.c), a.c, a.inv_tau);
  const double lse_rest = sum_lse(rest, a.c, a.inv_tau);
  double sum = 0.0;
  for (int k = lane; k < a.K; k += 64) {
    const int64_t id = a.ids[row * a.K + k];
    if (id < 0 || id >= a.V) continue;
    const float t = a.logprob[row * a.K + k];
    if (t == neg_inf()) continue;  // no mass
    const double logq = static_cast<double>(Tr::load1(xp, id)) * a.inv_tau - lse;
    sum += exp(static_cast<double>(t)) * (static_cast<double>(t) - logq);
  }
  sum = lanes_sum(sum);
  if (lane != 0) return;
  if (a.rest && a.rest[row] != neg_inf()) {
    const double t = a.rest[row];
    sum += exp(t) * (t - (lse_rest - lse));
  }
  a.loss[row] = static_cast<float>(sum);
  if (a.lse_out) a.lse_out[row] = static_cast<float>(lse);
  if (a.lse_rest_out) a.lse_rest_out[row] = static_cast<float>(lse_rest);
}

__device__ __forceinline__ void store_no_loss(const DistillArgs& a, int64_t row) {
  a.loss[row] = 0.f;
  if (a.lse_out) a.lse_out[row] = 0.f;
  if (a.lse_rest_out) a.lse_rest_out[row] = 0.f;
}

// The gradient's scalars of a row: listed columns get exp2(z c + nl) all - mass gt,
// others exp2(z c + nr) others.
struct GradRow {
  float nl, all, gt, nr, others;
  int zero;  // nothing is left of the probabilities: the row's gradient is 0
};

// |lse| up to which fp32 says anything of exp(z - lse)
constexpr float kFarLse = kFar * kLn2;

template <class Tr, int NT, int U, bool GRAD>
__global__ void __launch_bounds__(NT) k_distill(DistillArgs a) {
  constexpr int P = Tr::kPerVec, W = NT / 64;
  __shared__ int cols[kMaxTop];  // column of the slice that an entry names, or -1
  __shared__ float mass[GRAD ? kMaxTop : 1];
  __shared__ unsigned long long held[NT];
  __shared__ SumStat sm[2][W];
  __shared__ GradRow shared_row;
  const int tid = threadIdx.x;
  const unsigned rel_row = blockIdx.x / static_cast<unsigned>(a.nslices);
  const int slice = static_cast<int>(blockIdx.x - rel_row * static_cast<unsigned>(a.nslices));
  const int64_t row = a.row0 + rel_row;
  const int c0 = slice * a.slice;
  const char* xp = static_cast<const char*>(a.x) + (row * a.ld + c0) * Tr::kBytes;
  char* op = GRAD ? static_cast<char*>(a.out) + (row * a.ld_out + c0) * Tr::kBytes : nullptr;
  Vectors<Tr> vs;
  vs.n = a.V - c0 < a.slice ? a.V - c0 : a.slice;
  vs.pad = GRAD ? static_cast<int>((reinterpret_cast<uintptr_t>(op) & 15u) / Tr::kBytes) : 0;
  const float c = a.c;
  auto clear = [&] {
    float x[P];
#pragma unroll
    for (int k = 0; k < P; ++k) x[k] = 0.f;
    for (int v = tid; v < vs.end(); v += NT) vs.store(op, v, x);
  };
  if (a.mask && a.mask[row] == 0) {
    if (GRAD)
      clear();
    else if (a.nslices == 1 && tid == 0)
      store_no_loss(a, row);
    return;
  }

  held[tid] = 0;
  __syncthreads();
  if (tid < 64) {
    double all = 0.0;
    for (int k = tid; k < a.K; k += 64) {
      const int64_t id = a.ids[row * a.K + k], rel = id - c0;
      const bool inside = id >= 0 && id < a.V, here = rel >= 0 && rel < vs.n;
      cols[k] = here ? static_cast<int>(rel) : -1;
      if (GRAD) {
        const double p = inside ? exp(static_cast<double>(a.logprob[row * a.K + k])) : 0.0;
        all += p;
        mass[k] = static_cast<float>(p);
      }
      if (here) {
        const int v = (static_cast<int>(rel) + vs.pad) / P;
        atomicOr(held + v % NT, 1ull << (v / NT));
      }
    }
    if (GRAD) {
      all = lanes_sum(all);
      const double r = a.rest ? exp(static_cast<double>(a.rest[row])) : 0.0;
      const double g = static_cast<double>(a.grad_loss[row]) * a.inv_tau;
      const float lse = a.lse[row], lse_rest = a.lse_rest[row];
      all += r;
      GradRow q;
      q.zero = fabsf(lse) > kFarLse;
      q.nl = -lse * kLog2e;
      q.all = static_cast<float>(all * g);
      q.gt = static_cast<float>(g);
      // with no weight outside the list, or none that fp32 tells apart, those columns get 0
      const bool none = fabsf(lse_rest) > kFarLse;
      q.nr = none ? neg_inf() : -lse_rest * kLog2e;
      q.others = none ? 0.f : static_cast<float>((all * exp(static_cast<double>(lse_rest) - static_cast<double>(lse)) - r) * g);
      if (tid == 0) shared_row = q;
    }
  }
  __syncthreads();
  GradRow gr{};
  if (GRAD) {
    gr = shared_row;
    if (gr.zero) {
      clear();
      return;
    }
  }
  const unsigned long long own = held[tid];

  LaneSum st = sum_none(), listed = sum_none();
  auto load = [&](int v) {
    return static_cast<u32x4>(__builtin_nontemporal_load(
        reinterpret_cast<const u32x4_a2*>(xp + (static_cast<int64_t>(v) * P - vs.pad) * Tr::kBytes)));
  };
  auto other = [&](float z) { return fast_exp2(fmaf(z, c, gr.nr)) * gr.others; };
  const int whole_end = vs.whole_end(), first = vs.first();
  const int steps = (vs.end() + NT - 1) / NT;
  // U vectors at a time; a bit of `skip` leaves one out
  auto skips = [&](int q) {
    uint32_t s = static_cast<uint32_t>(own >> q);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = tid + (q + u) * NT;
      if (v < first || v >= whole_end) s |= 1u << u;
    }
    return s;
  };
  u32x4 w[U];
  uint32_t skip = skips(0);
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = skip >> u & 1 ? no_vector<Tr>() : load(tid + u * NT);
  for (int q = 0; q < steps; q += U) {
    float x[U * P];
#pragma unroll
    for (int u = 0; u < U; ++u) Tr::unpack(w[u], x + u * P);
    const uint32_t now = skip;
    if (q + U < steps) {
      skip = skips(q + U);
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = skip >> u & 1 ? no_vector<Tr>() : load(tid + (q + U + u) * NT);
    }
    if (GRAD) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (now >> u & 1) continue;
#pragma unroll
        for (int k = 0; k < P; ++k) x[u * P + k] = other(x[u * P + k]);
        __builtin_nontemporal_store(Tr::pack(x + u * P),
                                    reinterpret_cast<u32x4*>(op + (static_cast<int64_t>(tid + (q + u) * NT) * P - vs.pad) * Tr::kBytes));
      }
    } else {
      sum_push<U * P, P>(st, x, largest_of<U * P>(x), c);
    }
  }
  // what is not whole, unless an entry lies in it
  auto partial = [&](int v) {
    if (v % NT != tid || (own >> (v / NT) & 1)) return;
    float x[P];
    Tr::unpack(vs.load(xp, v), x);
    if (GRAD) {
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = other(x[k]);
      vs.store(op, v, x);
    } else {
      sum_push<P, P>(st, x, largest_of<P>(x), c);
    }
  };
  if (first) partial(0);
  if (whole_end < vs.end() && (whole_end > 0 || !first)) partial(whole_end);

  for (int k = tid; k < a.K; k += NT) {
    if (cols[k] < 0) continue;
    const int v = (cols[k] + vs.pad) / P;
    bool mine = true;
    uint32_t bits = 0;
    double ps[P];  // many entries may name one column
#pragma unroll
    for (int e = 0; e < P; ++e) ps[e] = 0.0;
    for (int j = 0; j < a.K; ++j) {
      if (cols[j] < 0) continue;
      const int at = cols[j] + vs.pad;
      if (at / P != v) continue;
      mine = mine && j >= k;
      bits |= 1u << (at % P);
      if (GRAD) {
#pragma unroll
        for (int e = 0; e < P; ++e)
          if (at % P == e) ps[e] += mass[j];
      }
    }
    if (!mine) continue;
    float x[P];
    Tr::unpack(vs.load(xp, v), x);
    if (GRAD) {
#pragma unroll
      for (int e = 0; e < P; ++e)
        x[e] = bits >> e & 1 ? fmaf(fast_exp2(fmaf(x[e], c, gr.nl)), gr.all, -static_cast<float>(ps[e]) * gr.gt) : other(x[e]);
      vs.store(op, v, x);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (bits >> e & 1)
          sum_push1(listed, x[e], c);
        else
          sum_push1(st, x[e], c);
      }
    }
  }
  if (GRAD) return;
  const SumStat rest = sum_block<NT>(st, c, sm[0]), top = sum_block<NT>(listed, c, sm[1]);
  if (a.nslices == 1) {
    if (tid < 64) store_loss<Tr>(a, row, rest, top);
  } else if (tid == 0) {
    float* p = a.part + (row * a.nslices + slice) * 4;
    p[0] = rest.m;
    p[1] = rest.s;
    p[2] = top.m;
    p[3] = top.s;
  }
}

// One wave per row: the slices' states in a fixed order, then the outputs.
template <class Tr>
__global__ void __launch_bounds__(256) k_distill_join(DistillArgs a) {
  const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.T) return;
  if (a.mask && a.mask[row] == 0) {
    if (lane == 0) store_no_loss(a, row);
    return;
  }
  SumStat rest{neg_inf(), 0.f}, listed{neg_inf(), 0.f};
  for (int i = lane; i < a.nslices; i += 64) {
    const float* p = a.part + (row * a.nslices + i) * 4;
    rest = sum_add(rest, SumStat{p[0], p[1]}, a.c);
    listed = sum_add(listed, SumStat{p[2], p[3]}, a.c);
  }
  store_loss<Tr>(a, row, sum_merge<64>(rest, a.c), sum_merge<64>(listed, a.c));
}

// Slices per row: one where there are rows for three workgroups a CU, else as
// many as that takes; a lane's word takes 64 vectors of a slice.
void set_slices(DistillArgs& a, int dtype) {
  const int64_t longest = int64_t(64) * 512 * (dtype == 2 ? 4 : 8) - 128;
  const int64_t most = (int64_t(a.V) + kMinDistillSlice - 1) / kMinDistillSlice, least = (int64_t(a.V) + longest - 1) / longest;
  int64_t n = (768 + a.T - 1) / (a.T > 0 ? a.T : 1);
  n = n < most ? n : most;
  n = n > least ? n : least;
  a.slice = static_cast<int>(((int64_t(a.V) + n - 1) / n + 127) / 128 * 128);
  a.nslices = static_cast<int>((int64_t(a.V) + a.slice - 1) / a.slice);
}

template <class Tr, int NT, bool GRAD>
hipError_t launch_distill_nt(DistillArgs a, hipStream_t s) {
  constexpr int U = GRAD ? 2 : 4;
  const int64_t rows_per = (int64_t(1) << 22) / a.nslices > 0 ? (int64_t(1) << 22) / a.nslices : 1;
  for (int64_t r0 = 0; r0 < a.T; r0 += rows_per) {
    const int64_t rows = a.T - r0 < rows_per ? a.T - r0 : rows_per;
    a.row0 = r0;
    TimedLaunch tl(GRAD ? "k_distill_grad" : "k_distill", s);
    hipLaunchKernelGGL((k_distill<Tr, NT, U, GRAD>), dim3(static_cast<unsigned>(rows * a.nslices)), dim3(NT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class Tr, bool GRAD>
hipError_t launch_distill_t(const DistillArgs& a, hipStream_t s) {
  if (a.slice >= 16384) return launch_distill_nt<Tr, 512, GRAD>(a, s);
  if (a.slice >= 4096) return launch_distill_nt<Tr, 256, GRAD>(a, s);
  return launch_distill_nt<Tr, 128, GRAD>(a, s);
}

template <bool GRAD>
hipError_t launch_distill_any(int dtype, const DistillArgs& a, hipStream_t s) {
  switch (dtype) {
    case 0: return launch_distill_t<Bf16, GRAD>(a, s);
    case 1: return launch_distill_t<Fp16, GRAD>(a, s);
    default: return launch_distill_t<Fp32, GRAD>(a, s);
  }
}

}  // namespace

size_t distill_workspace_bytes(int dtype, int64_t T, int64_t V) {
  DistillArgs a{};
  a.T = T;
  a.V = static_cast<int>(V);
  set_slices(a, dtype);
  if (a.nslices == 1) return 256;
  const size_t per_row = size_t(a.nslices) * 16;
  if (size_t(T) > (size_t(1) << 60) / per_row) return 0;
  return (size_t(T) * per_row + 255) / 256 * 256;
}

hipError_t launch_distill(int dtype, const DistillArgs& args, char* ws, hipStream_t s) {
  DistillArgs a = args;
  set_slices(a, dtype);
  a.part = reinterpret_cast<float*>(ws);
  hipError_t e = launch_distill_any<false>(dtype, a, s);
  if (e != hipSuccess || a.nslices == 1) return e;
  constexpr int64_t kRows = int64_t(1) << 22;
  for (int64_t r0 = 0; r0 < a.T; r0 += kRows) {
    a.row0 = r0;
    const int64_t rows = a.T - r0 < kRows ? a.T - r0 : kRows;
    const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
    TimedLaunch tl("k_distill_join", s);
    if (dtype == 0)
      hipLaunchKernelGGL(k_distill_join<Bf16>, grid, dim3(256), 0, s, a);
    else if (dtype == 1)
      hipLaunchKernelGGL(k_distill_join<Fp16>, grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL(k_distill_join<Fp32>, grid, dim3(256), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_distill_grad(int dtype, const DistillArgs& args, hipStream_t s) {
  DistillArgs a = args;
  set_slices(a, dtype);
  return launch_distill_any<true>(dtype, a, s);
}

}  // namespace lp
