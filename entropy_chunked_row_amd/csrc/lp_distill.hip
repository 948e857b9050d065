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
// vectors.  A lane streams vectors tid, tid + NT, ... of its slice; which of its own are
// listed is a bit each in LDS, 32 to a word, so a vector costs one bit test.
// Listed vectors are left out of the stream; each is taken by the first entry that lies
// in it, which looks through the list for the others: so an id listed twice counts
// once in the sums and with both its masses in the gradient, in a fixed order, and
// the sum over unlisted columns is a sum of its own.
// Bound by HBM: lists of 64 on 6144 scored rows of 151936 bf16 289 us, 6.5 TB/s of
// reading (6.8 is what reading alone reaches); the gradient of 4096 such rows 412 us,
// 6.0 TB/s read and written (6.1 is an elementwise kernel's).
#include "lp_internal.hpp"
#include "lp_sums.hpp"

namespace lp {

namespace {

constexpr int kMinDistillSlice = 2048;
constexpr int kNoCol = 0x7fffffff;
constexpr int kMaskWords = 8;  // of 32 of a lane's vectors each: the longest slice

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

// exp(t) to within 2^-23 of it: a teacher's log-probs are no better known, and the
// fp64 function alone takes longer than all else in a short row.  The same in every
// place, so that a row's masses agree with their sum.  0 from about -104 down: an entry
// without mass adds nothing to the loss, also where the student's log is -inf and the
// term would be 0 times infinity (finite masks in the teacher's logits, -inf in the student's).
__device__ __forceinline__ double mass_of(float t) { return static_cast<double>(expf(t)); }

// What listed entries add to a row's loss before its log-sum-exps are known: with m the
// largest value of the row's state and l = lse - m / tau,
//   loss = sum over waves (terms + mass ((m - ref) / tau + l)) + r (t_rest - (lse_rest - lse)).
// The loss is a difference of nearly equal numbers: fp64; and relative to the largest
// value that a wave's entries name, since beside values of finite masks fp64 holds nothing else.
struct Entries {
  double terms, mass;  // sums of p_k (t_k - (z_k - ref) / tau) and of p_k
  float ref;           // the largest finite z_k of an entry with mass, 0 if there is none
};

// z, or nothing where an entry has no mass
__device__ __forceinline__ float candidate_ref(float z, double p) { return p != 0.0 ? z : neg_inf(); }
__device__ __forceinline__ float reduce_ref(float z) {
  const float m = lanes_reduce<64>(z, [](float x, float y) { return fmaxf(x, y); });
  return m > neg_inf() ? m : 0.f;
}

// By one wave, in every lane of it.
template <class Tr>
__device__ __forceinline__ Entries sum_entries(const DistillArgs& a, int64_t row) {
  const char* xp = static_cast<const char*>(a.x) + row * a.ld * Tr::kBytes;
  Entries e{0.0, 0.0, neg_inf()};
  constexpr int E = kMaxTop / 64;
  float t[E], z[E];
  double p[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int k = static_cast<int>(threadIdx.x & 63) + i * 64;
    p[i] = 0.0;
    if (i * 64 >= a.K) continue;  // for the whole wave
    const int64_t id = k < a.K ? a.ids[row * a.K + k] : -1;
    t[i] = k < a.K ? a.logprob[row * a.K + k] : neg_inf();
    const bool inside = id >= 0 && id < a.V;  // else padding
    z[i] = inside ? Tr::load1(xp, id) : 0.f;
    p[i] = inside ? mass_of(t[i]) : 0.0;
    e.mass += p[i];
    e.ref = fmaxf(e.ref, candidate_ref(z[i], p[i]));
  }
  e.ref = reduce_ref(e.ref);
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i * 64 < a.K && p[i] != 0.0) e.terms += p[i] * (static_cast<double>(t[i]) - below(z[i], e.ref, a.inv_tau));
  e.terms = lanes_sum(e.terms);
  e.mass = lanes_sum(e.mass);
  return e;
}

// By one thread: the outputs of a row from the entries of N waves and the states of
// its unlisted and its listed columns.
template <int N>
__device__ __forceinline__ void store_loss(const DistillArgs& a, int64_t row, const Entries* e, float t_rest, SumStat rest,
                                           SumStat listed) {
  const SumStat whole = sum_add(rest, listed, a.c);
  const double log_sum = sum_log(whole, a.c), log_rest = sum_log(rest, a.c);
  double loss = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) loss += e[i].terms + e[i].mass * (below(whole.m, e[i].ref, a.inv_tau) + log_sum);
  const double r = mass_of(t_rest);
  if (r != 0.0) loss += r * (static_cast<double>(t_rest) - sum_gap(rest, log_rest, whole, log_sum, a.inv_tau));
  a.loss[row] = static_cast<float>(loss);
  if (a.lse_out) a.lse_out[row] = static_cast<float>(sum_lse(whole, log_sum, a.inv_tau));
  if (a.lse_rest_out) a.lse_rest_out[row] = static_cast<float>(sum_lse(rest, log_rest, a.inv_tau));
}

__device__ __forceinline__ void store_no_loss(const DistillArgs& a, int64_t row) {
  a.loss[row] = 0.f;
  if (a.lse_out) a.lse_out[row] = 0.f;
  if (a.lse_rest_out) a.lse_rest_out[row] = 0.f;
}

// The gradient's scalars of a row: listed columns get exp2(z cl + nl) all - mass gt
// (two nearly equal parts where the student is near its teacher: their exponent is
// taken in fp64), others exp2(z c + nr) others.
struct GradRow {
  double cl, nl;
  float all, gt, nr, others;
};

constexpr double kLog2e64 = 1.4426950408889634;

// |lse| up to which fp32 says anything of exp(z - lse)
constexpr float kFarLse = kFar * kLn2;

template <class Tr, int NT, int U, bool GRAD>
__global__ void __launch_bounds__(NT) k_distill(DistillArgs a) {
  constexpr int P = Tr::kPerVec, W = NT / 64;
  static_assert(32 % U == 0, "a group's bits lie in one word");
  __shared__ __attribute__((aligned(16))) int cols[kMaxTop];  // of every entry
  __shared__ float mass[GRAD ? kMaxTop : 1];
  __shared__ uint32_t held[kMaskWords][NT];
  __shared__ SumStat sm[2][W];
  __shared__ Entries parts[W];  // of the entries of each wave's threads
  const int tid = threadIdx.x;
  const unsigned block = spread_block(), rel_row = block / static_cast<unsigned>(a.nslices);
  const int slice = static_cast<int>(block - rel_row * static_cast<unsigned>(a.nslices));
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

  const int whole_end = vs.whole_end(), first = vs.first();
  const int steps = (vs.end() + NT - 1) / NT;
  const char* base = xp - vs.pad * Tr::kBytes;  // 32-bit offsets: a slice is far shorter
  // U vectors at a time, unconditionally: those outside read one inside
  auto load = [&](int v) {
    const int at = min(max(v, first), whole_end - 1);
    return static_cast<u32x4>(__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(base + static_cast<uint32_t>(at) * 16u)));
  };
  // Thread k has entry k (and k + NT).  What follows from its id is under way
  // before anything waits: the vector it lies in, its logit, the first vectors of
  // the stream, the row's scalars.
  constexpr int E = (kMaxTop + NT - 1) / NT;
  int64_t id[E];
  float t[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int k = tid + i * NT;
    id[i] = k < a.K ? a.ids[row * a.K + k] : -1;
    t[i] = k < a.K ? a.logprob[row * a.K + k] : neg_inf();
  }
  const float t_rest = a.rest ? a.rest[row] : neg_inf();
  const float lse = GRAD ? a.lse[row] : 0.f, lse_rest = GRAD ? a.lse_rest[row] : 0.f, g_loss = GRAD ? a.grad_loss[row] : 0.f;
  u32x4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = whole_end > first ? load(tid + u * NT) : no_vector<Tr>();
  for (int i = 0; i * 32 < steps; ++i) held[i][tid] = 0;
  __syncthreads();
  u32x4 in[E];  // the vector that the entry lies in
  float z[E];
  int col[E];  // on the grid of vectors, or outside
  Entries e{0.0, 0.0, neg_inf()};
  double p[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int k = tid + i * NT;
    const int64_t rel = id[i] - c0;
    const bool inside = id[i] >= 0 && id[i] < a.V, here = rel >= 0 && rel < vs.n;
    col[i] = here ? static_cast<int>(rel) + vs.pad : kNoCol;
    if (here) {
      const int v = col[i] / P;
      in[i] = vs.load(xp, v);
      atomicOr(&held[v / (32 * NT)][v % NT], 1u << (v / NT % 32));
    }
    z[i] = !GRAD && inside && a.nslices == 1 ? Tr::load1(xp, id[i]) : 0.f;
    if (k < kMaxTop) cols[k] = col[i];
    if (GRAD || a.nslices == 1) {
      p[i] = inside ? mass_of(t[i]) : 0.0;
      e.mass += p[i];
      if (GRAD && k < kMaxTop) mass[k] = static_cast<float>(p[i]);
      if (!GRAD) e.ref = fmaxf(e.ref, candidate_ref(z[i], p[i]));
    }
  }
  if ((tid & ~63) < a.K && (GRAD || a.nslices == 1)) {  // waves with entries
    if (!GRAD) {
      e.ref = reduce_ref(e.ref);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (p[i] != 0.0) e.terms += p[i] * (static_cast<double>(t[i]) - below(z[i], e.ref, a.inv_tau));
      e.terms = lanes_sum(e.terms);
    }
    e.mass = lanes_sum(e.mass);
  } else {
    e.ref = 0.f;
  }
  if ((tid & 63) == 0) parts[tid >> 6] = e;
  __syncthreads();
  GradRow gr{};
  if (GRAD) {
    double all = a.rest ? mass_of(t_rest) : 0.0;
    const double r = all, g = static_cast<double>(g_loss) * a.inv_tau;
#pragma unroll
    for (int i = 0; i < W; ++i) all += parts[i].mass;
    if (fabsf(lse) > kFarLse) {  // nothing is left of the probabilities
      clear();
      return;
    }
    gr.cl = a.inv_tau * kLog2e64;
    gr.nl = -lse * kLog2e64;
    gr.all = static_cast<float>(all * g);
    gr.gt = static_cast<float>(g);
    // with no weight outside the list, or none that fp32 tells apart, those columns get 0
    const bool none = fabsf(lse_rest) > kFarLse;
    // What rounding lse_rest log2(e) to fp32 takes off every exponent of the row (1e-6
    // of the weights at 20) goes into the row's factor; the product is taken with the
    // log2(e) / tau that c holds, so that both of an exponent's terms are off alike.
    const double er = -lse_rest * (static_cast<double>(c) / a.inv_tau);
    gr.nr = none ? neg_inf() : static_cast<float>(er);
    const double down = static_cast<double>(lse_rest) - static_cast<double>(lse);
    const float near = static_cast<float>(down);
    const double rq = static_cast<double>(expf(near)) * (1.0 + (down - near));
    gr.others = none ? 0.f : static_cast<float>((all * rq - r) * g) * fast_exp2(static_cast<float>(er - gr.nr));
  }

  LaneSum st = sum_none(), listed = sum_none();
  auto other = [&](float z) { return fast_exp2(fmaf(z, c, gr.nr)) * gr.others; };
  auto listed_at = [&](float z) {
    const double e = fma(static_cast<double>(z), gr.cl, gr.nl);
    const float near = static_cast<float>(e);  // -inf: its rest is a NaN
    const float p = fast_exp2(near);
    return p == 0.f ? p : p * fast_exp2(static_cast<float>(e - near));
  };
  auto own = [&](int q) { return held[q >> 5][tid] >> (q & 31) & 1u; };

  // Listed vectors, each by its first entry.
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (col[i] == kNoCol) continue;
    const int k = tid + i * NT, v = col[i] / P;
    bool mine = true;
    uint32_t bits = 0;
    double ps[P];  // many entries may name one column
#pragma unroll
    for (int j = 0; j < P; ++j) ps[j] = 0.0;
    for (int j0 = 0; j0 < a.K; j0 += 32) {  // behind entry K lie none
      typedef int i32x4 __attribute__((ext_vector_type(4)));
      uint32_t match = 0;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const i32x4 quad = *reinterpret_cast<const i32x4*>(cols + j0 + j);
#pragma unroll
        for (int n = 0; n < 4; ++n) match |= static_cast<uint32_t>(quad[n]) / P == static_cast<uint32_t>(v) ? 1u << (j + n) : 0u;
      }
      for (; match; match &= match - 1) {
        const int at = j0 + __ffs(static_cast<int>(match)) - 1, in_vec = cols[at] % P;
        mine = mine && at >= k;
        bits |= 1u << in_vec;
        if (GRAD) {
          const double p = mass[at];
#pragma unroll
          for (int m = 0; m < P; ++m) ps[m] += in_vec == m ? p : 0.0;
        }
      }
    }
    if (!mine) continue;
    float x[P];
    Tr::unpack(in[i], x);
    if (GRAD) {
#pragma unroll
      for (int m = 0; m < P; ++m)
        x[m] = bits >> m & 1 ? fmaf(listed_at(x[m]), gr.all, -static_cast<float>(ps[m]) * gr.gt) : other(x[m]);
      vs.store(op, v, x);
    } else {
      float y[P];
#pragma unroll
      for (int m = 0; m < P; ++m) {
        y[m] = bits >> m & 1 ? x[m] : neg_inf();
        x[m] = bits >> m & 1 ? neg_inf() : x[m];
      }
      sum_push<P, P>(listed, y, largest_of<P>(y), c);
      sum_push<P, P>(st, x, largest_of<P>(x), c);
    }
  }
  // what is not whole, unless an entry lies in it
  auto partial = [&](int v) {
    if (v % NT != tid || own(v / NT)) return;
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

  // The stream.  Sums are relative to the largest of the wave's first vectors,
  // without a running maximum.  Where a wave's sum passes 2^100 that way, or is so
  // small that what was added as 0 (126 octaves below the reference) may count, or
  // where that reference is far from 0, the slice is summed again with one.
  SumStat low{neg_inf(), 0.f};
  if (whole_end > first) {
    float nmc = 0.f;
    if (!GRAD) {
      float m = neg_inf();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[P];
        Tr::unpack(w[u], x);
        m = fmaxf(m, largest_of<P>(x));
      }
      low.m = lanes_reduce<64>(m, [](float p, float q) { return fmaxf(p, q); });
      nmc = is_near(low.m * c) ? -(low.m * c) : -__builtin_inff();  // far: no sum
    }
    uint32_t word = 0;
    for (int q = 0; q < steps; q += U) {
      if ((q & 31) == 0) word = held[q >> 5][tid];
      float x[U * P];
#pragma unroll
      for (int u = 0; u < U; ++u) Tr::unpack(w[u], x + u * P);
      if (q + U < steps) {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load(tid + (q + U + u) * NT);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = tid + (q + u) * NT;
        const bool on = !(word >> u & 1) && v >= first && v < whole_end;
        if (GRAD) {
          if (!on) continue;
#pragma unroll
          for (int k = 0; k < P; ++k) x[u * P + k] = other(x[u * P + k]);
          __builtin_nontemporal_store(Tr::pack(x + u * P),
                                      reinterpret_cast<u32x4*>(op + (static_cast<int64_t>(v) * P - vs.pad) * Tr::kBytes));
        } else {
          float ps = fast_exp2(fmaf(x[u * P], c, nmc));
#pragma unroll
          for (int k = 1; k < P; ++k) ps += fast_exp2(fmaf(x[u * P + k], c, nmc));
          low.s += on ? ps : 0.f;
        }
      }
      word >>= U;
    }
    if (!GRAD) {
      const float whole = lanes_reduce<64>(low.s, [](float p, float q) { return p + q; });
      if (__syncthreads_or(!(whole >= 8.5e-22f && whole <= kMostSum))) {
        LaneSum over = sum_none();
        for (int q = 0; q < steps; ++q) {
          const int v = tid + q * NT;
          if (v < first || v >= whole_end || own(q)) continue;
          float x[P];
          Tr::unpack(load(v), x);
          sum_push<P, P>(over, x, largest_of<P>(x), c);
        }
        low = over;
      }
    }
  }
  if (GRAD) return;
  // both states of the workgroup, in every lane of its first wave
  const SumStat mine[2] = {sum_merge<64>(sum_add(st, low, c), c), sum_merge<64>(listed, c)};
  if ((tid & 63) == 0) {
    sm[0][tid >> 6] = mine[0];
    sm[1][tid >> 6] = mine[1];
  }
  __syncthreads();
  if (tid >= 64) return;
  const SumStat rest = sum_merge<W>(sm[0][tid & (W - 1)], c), top = sum_merge<W>(sm[1][tid & (W - 1)], c);
  if (tid != 0) return;
  if (a.nslices == 1) {
    store_loss<W>(a, row, parts, t_rest, rest, top);
  } else {
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
  const Entries e = sum_entries<Tr>(a, row);
  rest = sum_merge<64>(rest, a.c);
  listed = sum_merge<64>(listed, a.c);
  if (lane == 0) store_loss<1>(a, row, &e, a.rest ? a.rest[row] : neg_inf(), rest, listed);
}

// Slices per row: as many as make three workgroups a CU where rows are few; the
// bits hold kMaskWords x 32 of a lane's vectors.  For the gradient slices of about
// kGradSlice columns, whatever the rows: what is read and what is written then lie
// close together (4096 x 151936 bf16 422 us back to back, 446 with 16384 columns, 472 with 32768).
// Short rows are not cut for the loss: a join would cost more than it saves (1 to 256
// rows of 32000 15 us, 18 with slices).
constexpr int64_t kRowGroups = 768, kGradSlice = 8192, kWholeRow = 32768;

void set_slices(DistillArgs& a, int dtype, bool grad) {
  const int64_t longest = int64_t(32) * kMaskWords * 256 * (dtype == 2 ? 4 : 8) - 128;
  const int64_t most = (int64_t(a.V) + kMinDistillSlice - 1) / kMinDistillSlice, least = (int64_t(a.V) + longest - 1) / longest;
  int64_t n = (kRowGroups + a.T - 1) / (a.T > 0 ? a.T : 1);
  if (grad && n < a.V / kGradSlice) n = a.V / kGradSlice;
  n = n < most ? n : most;
  if (!grad && a.V <= kWholeRow) n = 1;
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
  // 128 threads where that leaves a few vectors each (2000 rows of 4099: 19 us, 23 with
  // 256; of 7300 columns the same), 256 for long slices (8192 x 151936 292 us, 305 with
  // 128; gradient 435 and 451; all of these before listed vectors took less)
  if (a.slice >= 6144) return launch_distill_nt<Tr, 256, GRAD>(a, s);
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
  set_slices(a, dtype, false);
  if (a.nslices == 1) return 256;
  const size_t per_row = size_t(a.nslices) * 16;
  if (size_t(T) > (size_t(1) << 60) / per_row) return 0;
  return (size_t(T) * per_row + 255) / 256 * 256;
}

hipError_t launch_distill(int dtype, const DistillArgs& args, char* ws, hipStream_t s) {
  DistillArgs a = args;
  set_slices(a, dtype, false);
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
  set_slices(a, dtype, true);
  return launch_distill_any<true>(dtype, a, s);
}

}  // namespace lp
