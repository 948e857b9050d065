// The largest logits of rows, and what is chosen from them: the top K of a row
// with their log-probs and the mass of all others (lp_top_logits), and the best
// N continuations over the beams of a request (lp_beam_select).
//
// A row is read once.  A workgroup owns a row, or a slice of one where rows are
// few, and
//   1. reads a first piece of it, spread over its whole length, and takes each
//      lane's largest value: the K-th largest of these, the floor, is no larger
//      than the K-th largest of the row, so nothing below it can be chosen;
//   2. streams the row.  Vectors of 16 bytes that hold a value at or above the
//      floor are kept in LDS, all others are added to a sum of exponentials
//      relative to the floor, which needs no running maximum.  The floor is taken
//      anew after 1, 2, 4, 8 ... steps: of 152000 columns about 5 K vectors are kept;
//   3. repeats step 1 on the kept vectors, ranks what reaches the new floor by
//      counting, and sums what was not chosen.
// Short slices are kept whole.  The mass outside the list is a sum of its own,
// never a difference of two nearly equal ones.  Every result is the same bits on
// every call: only the order of the keys that are ranked depends on LDS atomics.
// Order is (value descending, column ascending), as one 64-bit key.  More kept
// vectors than LDS holds (rows that rise steadily, or have most values equal) are
// counted by digits of the keys instead: right for any row, several more reads of it.
// Bound by reading: 6144 scored rows of 151936 bf16, 64 of each, 322 us, 5.8 TB/s
// (6.8 is what reading alone reaches); what is missing are the waits of a row's end,
// which the other workgroups of a CU cover in part.  One row of 151936 is 16 us a
// call, two launches; 512 of 129280 fp16, 16 of each, 38 us, 9 of them the join.
#include "lp_internal.hpp"
#include "lp_sums.hpp"

namespace lp {

namespace {

constexpr int kMaxBuffered = 4096;  // keys of a row's or a request's slices that a join takes

// Significant leading bits of order_of for values of a type.
template <class Tr>
constexpr int kOrderBits = 32;
template <>
constexpr int kOrderBits<Bf16> = 16;
template <>
constexpr int kOrderBits<Fp16> = 19;

// By one wave: a t with at most BITS leading bits such that at least `want` of N
// words are >= t, and either exactly as many are or t is the largest such; 0 if even
// that many are not there (empty places hold 0).
template <int N, int BITS>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t* words, int want) {
  uint32_t w[N / 64];
#pragma unroll
  for (int i = 0; i < N / 64; ++i) w[i] = words[(threadIdx.x & 63) + 64 * i];
  uint32_t t = 0;
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t cand = t | 1u << b;
    int count = 0;
#pragma unroll
    for (int i = 0; i < N / 64; ++i) count += __popcll(__ballot(w[i] >= cand));
    if (count >= want) t = cand;
    if (count == want) break;
  }
  return t;
}

__device__ __forceinline__ uint64_t key_of(float x, int col) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ float key_value(uint64_t key) { return value_of(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int key_col(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }

// As a threshold: values at or above it.  Never -inf, which is not chosen.
__device__ __forceinline__ float threshold_of(uint32_t t) {
  const float x = value_of(t);
  return x >= -kLargest ? x : -kLargest;  // NaN (t = 0) too
}

// Keys greater than `key` among n (a 0 behind them where n is odd).
__device__ __forceinline__ int rank_among(const uint64_t* keys, int n, uint64_t key) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  int r = 0;
  for (int i = 0; i < n; i += 2) {
    const u64x2 q = *reinterpret_cast<const u64x2*>(keys + i);
    r += (q.x > key) + (q.y > key);
  }
  return r;
}

// Adds 1 to a bin; lanes that share the first lane's bin do so as one (rows of
// equal values would queue up at one address).
__device__ __forceinline__ void count_bin(uint32_t* hist, bool on, uint32_t bin) {
  const uint64_t live = __ballot(on);
  if (!live) return;
  const int first = __ffsll(static_cast<unsigned long long>(live)) - 1;
  const uint32_t lead = __shfl(bin, first, 64);
  const uint64_t same = __ballot(on && bin == lead);
  if (on && bin != lead) atomicAdd(hist + bin, 1u);
  if ((threadIdx.x & 63) == first) atomicAdd(hist + lead, static_cast<uint32_t>(__popcll(same)));
}

// The top `want` finite values of n columns by digits of their keys, whatever
// the row.  Their keys to `chosen` (unordered), their number returned; all else
// folded into st.  hist: 256 words and two more of LDS.
template <class Tr, int NT>
__device__ int choose_by_digits(const char* xp, int n, int c0, int want, float c, LaneSum& st, uint64_t* chosen,
                                uint32_t* hist) {
  constexpr int P = Tr::kPerVec;
  const int tid = threadIdx.x, vectors = (n + P - 1) / P, rounds = (vectors + NT - 1) / NT;
  uint32_t* found = hist + 256;  // digit, keys above it
  uint64_t prefix = 0;
  int need = want, shift = 64;
  while (shift > 0) {
    shift -= 8;
    __syncthreads();
    for (int i = tid; i < 256; i += NT) hist[i] = 0;
    __syncthreads();
    for (int q = 0; q < rounds; ++q) {
      const int v = tid + q * NT;
      float x[P];
      Tr::unpack(v < vectors ? row_vector<Tr>(xp, v, n) : no_vector<Tr>(), x);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const uint64_t key = key_of(x[k], c0 + v * P + k);
        const bool on = x[k] >= -kLargest && (shift == 56 || (key >> (shift + 8)) == prefix);
        count_bin(hist, on, static_cast<uint32_t>(key >> shift) & 255u);
      }
    }
    __syncthreads();
    if (tid < 64) {
      // lane l: digits 4 (63 - l) .. + 3, so that lower lanes hold larger ones
      const int d0 = 4 * (63 - tid);
      uint32_t h[4], mine = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine += h[k] = hist[d0 + k];
      uint32_t upto = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const uint32_t y = __shfl_up(upto, off, 64);
        if (tid >= off) upto += y;
      }
      uint32_t above = upto - mine;
      if (tid == 63 && upto < static_cast<uint32_t>(need)) found[0] = 0xffffffffu;  // not that many
      if (above < static_cast<uint32_t>(need) && upto >= static_cast<uint32_t>(need)) {
        int k = 3;
        while (above + h[k] < static_cast<uint32_t>(need)) above += h[k--];
        found[0] = d0 + k;
        found[1] = above;
      }
    }
    __syncthreads();
    const uint32_t digit = found[0];
    if (digit == 0xffffffffu) {  // only in the first round: every finite value is chosen
      shift = 64;
      break;
    }
    need -= static_cast<int>(found[1]);
    prefix = prefix << 8 | digit;
    if (hist[digit] == static_cast<uint32_t>(need)) break;  // the whole bin
  }
  const uint64_t least = shift >= 64 ? 0 : prefix << shift;
  __syncthreads();
  if (tid == 0) hist[0] = 0;
  __syncthreads();
  for (int q = 0; q < rounds; ++q) {
    const int v = tid + q * NT;
    float x[P];
    Tr::unpack(v < vectors ? row_vector<Tr>(xp, v, n) : no_vector<Tr>(), x);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const uint64_t key = key_of(x[k], c0 + v * P + k);
      if (x[k] >= -kLargest && key >= least) {
        const uint32_t at = atomicAdd(hist, 1u);
        if (at < static_cast<uint32_t>(want)) chosen[at] = key;  // never more; a bound all the same
        x[k] = neg_inf();
      }
    }
    sum_push<P, P>(st, x, largest_of<P>(x), c);
  }
  __syncthreads();
  const int got = static_cast<int>(hist[0]);
  return got < want ? got : want;
}

// The outputs of a row from its list in order (LDS) and the states of the list
// and of all else.
template <int NT>
__device__ __forceinline__ void store_top(const TopArgs& a, int64_t row, const uint64_t* top, int got, SumStat rest,
                                          SumStat listed) {
  const SumStat whole = sum_add(rest, listed, a.c);
  const bool bad = !(whole.s > 0.f && whole.s <= kLargest);  // a NaN or +inf in the row, or only -inf
  const float nan = __builtin_nanf("");
  if (static_cast<int>(threadIdx.x) >= a.K) return;
  const double log_sum = sum_log(whole, a.c);
  for (int k = threadIdx.x; k < a.K; k += NT) {
    float lp = bad ? nan : neg_inf();
    int64_t id = -1;
    if (k < got && !bad) {
      lp = static_cast<float>(below(key_value(top[k]), whole.m, a.inv_tau) - log_sum);
      id = key_col(top[k]);
    }
    a.ids[row * a.K + k] = id;
    a.logprob[row * a.K + k] = lp;
  }
  if (threadIdx.x == 0) {
    if (a.rest) a.rest[row] = bad ? nan : static_cast<float>(sum_gap(rest, sum_log(rest, a.c), whole, log_sum, a.inv_tau));
    if (a.lse) a.lse[row] = static_cast<float>(sum_lse(whole, log_sum, a.inv_tau));
  }
}

template <int NT>
__device__ __forceinline__ void store_no_top(const TopArgs& a, int64_t row) {
  for (int k = threadIdx.x; k < a.K; k += NT) {
    a.ids[row * a.K + k] = -1;
    a.logprob[row * a.K + k] = 0.f;
  }
  if (threadIdx.x == 0) {
    if (a.rest) a.rest[row] = 0.f;
    if (a.lse) a.lse[row] = 0.f;
  }
}

// Whether row `row` takes part: scored, or of a beam that goes on.
__device__ __forceinline__ bool row_live(const TopArgs& a, int64_t row) {
  if (a.beam_scores) return a.beam_scores[row] >= -kLargest && a.beam_scores[row] <= kLargest && !(a.finished && a.finished[row]);
  return !(a.mask && a.mask[row] == 0);
}

// Kept vectors a lane: of a slice kept whole (SHORT) 4, in registers.  Of a stream with 256
// threads (K up to 64) 192 a wave, twice what is expected, so that seven
// workgroups fit a CU; with 512 (K up to 256) 256, of which 170 are expected.
template <int NT, bool SHORT>
constexpr int kHeld = SHORT || NT > 256 ? 4 : 3;
constexpr int kFewTop = 64;  // most K of the first of these

// SHORT: the slice is at most kHeld vectors a lane, all of which are kept.
template <class Tr, int NT, bool SHORT>
__global__ void __launch_bounds__(NT) k_top(TopArgs a) {
  constexpr int P = Tr::kPerVec, U = 4, W = NT / 64, kLane = kHeld<NT, SHORT>, kKept = kLane * NT, kWave = kKept / W, kKeys = 2 * NT, kWords = 2 * NT;
  __shared__ u32x4 kept[SHORT ? 1 : kKept];
  __shared__ uint32_t kept_at[SHORT ? 1 : kKept];
  __shared__ __attribute__((aligned(16))) uint64_t keys[kKeys];
  __shared__ uint32_t best[kWords];  // later the digits' counts
  __shared__ uint64_t top[SHORT || NT > 256 ? kMaxTop : kFewTop];
  __shared__ SumStat sm[2][W];
  __shared__ uint32_t count, bar;
  __shared__ int held_by[W];
  static_assert(kWords >= 258, "digits' counts");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned block = spread_block(), rel_row = block / static_cast<unsigned>(a.nslices);
  const int slice = static_cast<int>(block - rel_row * static_cast<unsigned>(a.nslices));
  const int64_t row = a.row0 + rel_row;
  if (!row_live(a, row)) {
    if (!a.part_keys) store_no_top<NT>(a, row);
    return;
  }
  const int c0 = slice * a.slice;
  const int n = a.V - c0 < a.slice ? a.V - c0 : a.slice;
  const char* xp = static_cast<const char*>(a.x) + (row * a.ld + c0) * Tr::kBytes;
  const float c = a.c;
  if (tid == 0) count = 0;  // read behind the barriers of take_floor
  auto word = [](float x) { return x > neg_inf() ? order_of(x) : 0u; };
  // the floor that `best` gives, in every lane
  auto take_floor = [&](auto words) {
    __syncthreads();
    if (wave == 0) {
      const uint32_t t = kth_largest<decltype(words)::value, kOrderBits<Tr>>(best, a.K);
      if (lane == 0) bar = t;
    }
    __syncthreads();
    return threshold_of(bar);
  };

  SumStat low{neg_inf(), 0.f};  // of what was streamed and not kept: this lane's
  bool digits = false;
  u32x4 short_kept[SHORT ? kLane : 1];
  if (SHORT) {
    const int vectors = (n + P - 1) / P;
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const int v = tid + i * NT;
      short_kept[i] = v < vectors ? row_vector<Tr>(xp, v, n) : no_vector<Tr>();
    }
  } else {
    // U W pieces of `steps` times 64 vectors, so that one step of the workgroup is a
    // sample of the whole; a wave goes from piece to piece, so that each has its
    // share of a piece that holds more of what is kept.  What is left over behind
    // the pieces comes last.  There is at least one step: n >= 4 NT P (set_slices; the
    // loop below ends all the same without one).
    const int vectors = n / P, steps = vectors / (64 * U * W);
    const char* base = xp;  // 32-bit offsets: a slice has at most 2^32 bytes
    auto load = [&](uint32_t v) {
      return static_cast<u32x4>(__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(base + v * 16u)));
    };
    auto number = [&](int u, int q) { return static_cast<uint32_t>(((u * W + ((wave + q) & (W - 1))) * steps + q) * 64) + lane; };
    int held = 0;  // vectors that this wave has kept
    auto keep = [&](bool on, u32x4 vec, uint32_t v) {
      const uint64_t mask = __ballot(on);
      if (mask) {
        const int k = held + static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                                                      __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0)));
        if (on && k < kWave) {
          kept[wave * kWave + k] = vec;
          kept_at[wave * kWave + k] = v;
        }
        held += __popcll(mask);
      }
    };
    u32x4 w[U];
    float most = neg_inf();  // the lane's largest value so far
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load(number(u, 0));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[P];
      Tr::unpack(w[u], x);
      most = fmaxf(most, largest_of<P>(x));
    }
    best[tid] = word(most);
    float floor = take_floor(std::integral_constant<int, NT>{});
    // Exponents are relative to the floor.  With the lowest floor every finite value
    // is kept and the others' exponents only have to be -inf or NaN.  Floors far
    // from 0 otherwise (finite masks in all but a few columns) are left to the digits.
    float fc = floor > -kLargest ? floor * c : 0.f;
    digits = !is_near(fc);
    auto sum = [&](const float* x, bool on) {
      float ps = fast_exp2(fmaf(x[0], c, -fc));
#pragma unroll
      for (int k = 1; k < P; ++k) ps += fast_exp2(fmaf(x[k], c, -fc));
      low.s += on ? ps : 0.f;
    };
    for (int q = 0; !digits;) {
      float x[U * P];
      bool hit[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Tr::unpack(w[u], x + u * P);
        const float m = largest_of<P>(x + u * P);
        hit[u] = m >= floor;
        most = fmaxf(most, m);
        keep(hit[u], w[u], number(u, q));
      }
      const bool last = ++q >= steps;
      if (!last) {  // in flight while the exponentials are taken
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load(number(u, q));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) sum(x + u * P, !hit[u]);
      if (last) break;
      if ((q & (q - 1)) == 0) {
        best[tid] = word(most);
        const float was = floor;
        floor = take_floor(std::integral_constant<int, NT>{});
        fc = floor > -kLargest ? floor * c : 0.f;
        digits = !is_near(fc);
        low.s *= fast_exp2(stat_shift(was, floor, c));
      }
    }
    for (int v0 = steps * 64 * U * W; v0 * P < n; v0 += NT) {
      const int v = v0 + tid;
      const u32x4 vec = v * P < n ? row_vector<Tr>(xp, v, n) : no_vector<Tr>();
      float x[P];
      Tr::unpack(vec, x);
      const bool on = largest_of<P>(x) >= floor;
      keep(on, vec, v);
      sum(x, !on);
    }
    low.m = floor;
    if (lane == 0) held_by[wave] = held;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) digits |= held_by[i] > kWave;
  }

  // The kept vectors of this lane, f(values, number of the vector, whether it is
  // an odd one of the lane's).
  auto each_kept = [&](auto f) {
    if constexpr (SHORT) {
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        float x[P];
        Tr::unpack(short_kept[i], x);
        f(x, tid + i * NT, (i & 1) != 0);
      }
    } else {
      const int m = held_by[wave];
      for (int k = lane; k < m; k += 64) {
        float x[P];
        Tr::unpack(kept[wave * kWave + k], x);
        f(x, static_cast<int>(kept_at[wave * kWave + k]), (k / 64 & 1) != 0);
      }
    }
  };
  int got = 0;
  // the columns of vector v that are in the list weigh nothing in the rest
  auto leave_out = [&](float* x, int v) {
    const uint64_t least = got > 0 ? top[got - 1] : ~0ull;
    const float value = got > 0 ? key_value(least) : __builtin_inff();
    const int col = (got > 0 ? key_col(least) : -1) - c0 - v * P;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (x[i] > value || (x[i] == value && i <= col)) x[i] = neg_inf();
  };
  LaneSum st = sum_none();
  bool relative = false;
  if (!digits) {
    // Two words a lane, of every other vector; of the halves of its vector where
    // no lane has two: with fewer words than K nothing could be left out.
    const bool halves = SHORT ? n <= NT * P : held_by[wave] <= 64;
    float even = neg_inf(), odd = neg_inf();
    each_kept([&](const float* x, int, bool second) {
      const float lo = largest_of<P / 2>(x), hi = largest_of<P / 2>(x + P / 2);
      even = fmaxf(even, halves ? lo : second ? neg_inf() : fmaxf(lo, hi));
      odd = fmaxf(odd, halves ? hi : second ? fmaxf(lo, hi) : neg_inf());
    });
    best[tid] = word(even);
    best[NT + tid] = word(odd);
    const float floor = take_floor(std::integral_constant<int, kWords>{});
    each_kept([&](const float* x, int v, bool) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (x[i] >= floor) {
          const uint32_t k = atomicAdd(&count, 1u);
          if (k < static_cast<uint32_t>(kKeys)) keys[k] = key_of(x[i], c0 + v * P + i);
        }
      }
    });
    __syncthreads();
    const int m = static_cast<int>(count);
    digits = m > kKeys;
    if (!digits) {
      if (tid == 0 && (m & 1)) keys[m] = 0;
      __syncthreads();
      for (int i = tid; i < m; i += NT) {
        const uint64_t key = keys[i];
        const int r = rank_among(keys, m, key);
        if (r < a.K) top[r] = key;
      }
      got = m < a.K ? m : a.K;
      __syncthreads();
      // what is left of the kept vectors, relative to the floor as well where it is
      // near 0 (a streamed slice's is, or the lowest: others went to the digits); elsewhere
      // the state stays empty, since one of no weight at the floor would hide lower ones
      if (SHORT && is_near(floor * c)) low.m = floor;
      relative = low.m > -kLargest && is_near(low.m * c);
      const float mc = low.m * c;
      each_kept([&](float* x, int v, bool) {
        leave_out(x, v);
        if (relative) {
          float ps = fast_exp2(fmaf(x[0], c, -mc));
#pragma unroll
          for (int i = 1; i < P; ++i) ps += fast_exp2(fmaf(x[i], c, -mc));
          low.s += ps;
        } else {
          sum_push<P, P>(st, x, largest_of<P>(x), c);
        }
      });
    }
  }
  if (digits) {  // the same for the whole workgroup
    __syncthreads();
    st = sum_none();
    got = choose_by_digits<Tr, NT>(xp, n, c0, a.K, c, st, keys, best);
    if (tid == 0 && (got & 1)) keys[got] = 0;
    __syncthreads();
    for (int i = tid; i < got; i += NT) top[rank_among(keys, got, keys[i])] = keys[i];
  }
  SumStat rest = sum_block<NT>(digits ? st : sum_add(low, st, c), c, sm[0]);
  // What lies more than 126 octaves below the floor was added as 0, and what lies 128
  // above it as infinity.  Where the first is not small beside what is left, or that is
  // too large to be added up with others, the rest is summed once more.  (Below the
  // lowest floor lies nothing.)
  if (relative && !(rest.s >= 8.5e-22f && rest.s <= kMostSum)) {
    st = sum_none();
    for (int v = tid; v * P < n; v += NT) {
      float x[P];
      Tr::unpack(row_vector<Tr>(xp, v, n), x);
      leave_out(x, v);
      sum_push<P, P>(st, x, largest_of<P>(x), c);
    }
    __syncthreads();
    rest = sum_block<NT>(st, c, sm[0]);
  }
  __syncthreads();
  if (a.part_keys) {
    const int64_t part = row * a.nslices + slice;
    for (int k = tid; k < a.K; k += NT) a.part_keys[part * a.K + k] = k < got ? top[k] : 0;
    if (tid == 0) {
      a.part_sums[part * 2] = rest.m;
      a.part_sums[part * 2 + 1] = rest.s;
    }
    return;
  }
  LaneSum of_list = sum_none();
  for (int k = tid; k < got; k += NT) sum_push1(of_list, key_value(top[k]), c);
  store_top<NT>(a, row, top, got, rest, sum_block<NT>(of_list, c, sm[1]));
}

// A row's slices: their keys are ranked like a slice's own.
template <int NT>
__global__ void __launch_bounds__(NT) k_top_join(TopArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t keys[];  // nslices * K and one more
  __shared__ uint32_t best[NT];
  __shared__ uint64_t top[kMaxTop];
  __shared__ SumStat sm[2][NT / 64];
  __shared__ uint32_t count, bar;
  const int tid = threadIdx.x;
  const int64_t row = a.row0 + blockIdx.x;
  if (!row_live(a, row)) {
    store_no_top<NT>(a, row);
    return;
  }
  const float c = a.c;
  const int n = a.nslices * a.K;
  const uint64_t* all = a.part_keys + row * n;
  if (tid == 0) count = 0;
  // the first keys stay in registers
  constexpr int R = 4;
  uint64_t first[R];
#pragma unroll
  for (int i = 0; i < R; ++i) first[i] = tid + i * NT < n ? all[tid + i * NT] : 0;
  auto each_key = [&](auto f) {
#pragma unroll
    for (int i = 0; i < R; ++i) f(first[i]);
    for (int i = tid + R * NT; i < n; i += NT) f(all[i]);
  };
  uint32_t most = 0;
  each_key([&](uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    most = o > most ? o : most;
  });
  best[tid] = most;
  __syncthreads();
  if (tid < 64) {
    const uint32_t t = kth_largest<NT, 32>(best, a.K);
    if (tid == 0) bar = t;
  }
  __syncthreads();
  LaneSum st = sum_none();
  each_key([&](uint64_t key) {
    if (key != 0 && static_cast<uint32_t>(key >> 32) >= bar) keys[atomicAdd(&count, 1u)] = key;
  });
  for (int i = tid; i < a.nslices; i += NT) {
    const float* p = a.part_sums + (row * a.nslices + i) * 2;
    const SumStat both = sum_add(st, SumStat{p[0], p[1]}, c);
    st.m = both.m;
    st.s = both.s;
    st.nmc = both.m > neg_inf() ? -(both.m * c) : 0.f;
  }
  __syncthreads();
  const int m = static_cast<int>(count);
  if (tid == 0 && (m & 1)) keys[m] = 0;
  __syncthreads();
  for (int i = tid; i < m; i += NT) {
    const uint64_t key = keys[i];
    const int r = rank_among(keys, m, key);
    if (r < a.K) top[r] = key;
  }
  __syncthreads();
  const int got = m < a.K ? m : a.K;
  const uint64_t least = got > 0 ? top[got - 1] : 0;
  each_key([&](uint64_t key) {
    if (key != 0 && key < least) sum_push1(st, key_value(key), c);
  });
  LaneSum of_list = sum_none();
  for (int k = tid; k < got; k += NT) sum_push1(of_list, key_value(top[k]), c);
  const SumStat rest = sum_block<NT>(st, c, sm[0]);
  store_top<NT>(a, row, top, got, rest, sum_block<NT>(of_list, c, sm[1]));
}

// ---------------------------------------------------------------------------
// beams
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t order_of64(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of64(uint64_t order) {
  return __longlong_as_double(static_cast<long long>(order & 0x8000000000000000ull ? order ^ 0x8000000000000000ull : ~order));
}

// place orders candidates of equal scores: the lowest beam, its largest logit, the
// lowest column (a beam's lists are in the order of its columns' slices).
struct Candidate {
  uint64_t order;  // of its score
  uint64_t place;  // beam << 48 | ~order of its logit << 16 | number of its key among the request's
};
static_assert(kMaxBuffered <= 1 << 16 && kMaxBeamLists <= kMaxBuffered, "a key's number in 16 bits");

// One request: the lists of its beams' slices, scored and ranked.  Scores are fp64
// (sum_log).  Where the sum so far takes up the differences of a beam's logits (1e20, or
// the largest finite number, for beams that are not there; temperatures as large), place
// keeps their order.
template <int NT>
__global__ void __launch_bounds__(NT) k_beam_join(TopArgs a) {
  extern __shared__ __attribute__((aligned(16))) Candidate cand[];  // W * nslices * K of them
  __shared__ uint32_t best[NT];
  __shared__ double gain[kMaxBeams];  // what a beam adds to (z - m) / tau; NaN: no continuation
  __shared__ float most[kMaxBeams];   // m
  __shared__ uint32_t count, bar;
  const int tid = threadIdx.x;
  const int64_t b = a.row0 + blockIdx.x;
  const int W = a.W, N = a.K, per = a.nslices * N, n = W * per;
  const float c = a.c;
  if (tid == 0) count = 0;
  // a wave a beam
  for (int w = tid >> 6; w < W; w += NT / 64) {
    const int64_t row = b * W + w;
    double g = __builtin_nan("");
    if (row_live(a, row)) {
      LaneSum st = sum_none();
      for (int i = tid & 63; i < a.nslices; i += 64) {
        const float* p = a.part_sums + (row * a.nslices + i) * 2;
        const SumStat both = sum_add(st, SumStat{p[0], p[1]}, c);
        st.m = both.m;
        st.s = both.s;
      }
      st.nmc = st.m > neg_inf() ? -(st.m * c) : 0.f;
      for (int i = tid & 63; i < per; i += 64) {
        const uint64_t key = a.part_keys[row * per + i];
        if (key) sum_push1(st, key_value(key), c);
      }
      const SumStat whole = sum_merge<64>(st, c);
      if (whole.s > 0.f && whole.s <= kLargest) g = static_cast<double>(a.beam_scores[row]) - sum_log(whole, c);
      if ((tid & 63) == 0) most[w] = whole.m;
    }
    if ((tid & 63) == 0) gain[w] = g;
  }
  __syncthreads();
  // candidate i of beam i / per; 0: none
  auto order_at = [&](int i, uint64_t& place) -> uint64_t {
    const int w = i / per;
    const int64_t row = b * W + w;
    place = static_cast<uint64_t>(w) << 48 | static_cast<uint64_t>(i);
    if (a.finished && a.finished[row]) {
      const float s = a.beam_scores[row];
      return i == w * per && s >= -kLargest && s <= kLargest ? order_of64(s) : 0;
    }
    if (__builtin_isnan(gain[w])) return 0;
    const uint64_t key = a.part_keys[b * n + i];
    if (!key) return 0;
    place |= static_cast<uint64_t>(~static_cast<uint32_t>(key >> 32)) << 16;
    return order_of64(gain[w] + below(key_value(key), most[w], a.inv_tau));
  };
  // the first candidates stay in registers
  constexpr int R = 2;
  Candidate first[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    first[i].order = 0;
    if (tid + i * NT < n) first[i].order = order_at(tid + i * NT, first[i].place);
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < R; ++i) f(first[i]);
    for (int i = tid + R * NT; i < n; i += NT) {
      Candidate q;
      q.order = order_at(i, q.place);
      f(q);
    }
  };
  uint32_t first_word = 0;
  each([&](const Candidate& q) {
    const uint32_t o = static_cast<uint32_t>(q.order >> 32);
    first_word = o > first_word ? o : first_word;
  });
  best[tid] = first_word;
  __syncthreads();
  if (tid < 64) {
    const uint32_t t = kth_largest<NT, 32>(best, N);
    if (tid == 0) bar = t;
  }
  __syncthreads();
  each([&](const Candidate& q) {
    if (q.order && static_cast<uint32_t>(q.order >> 32) >= bar) cand[atomicAdd(&count, 1u)] = q;
  });
  __syncthreads();
  const int m = static_cast<int>(count);
  for (int i = tid; i < m; i += NT) {
    const Candidate q = cand[i];
    int r = 0;
    for (int j = 0; j < m; ++j) {
      const Candidate p = cand[j];
      r += p.order > q.order || (p.order == q.order && p.place < q.place);
    }
    if (r < N) {
      const int w = static_cast<int>(q.place >> 48);
      const bool ended = a.finished && a.finished[b * W + w];
      a.scores[b * N + r] = static_cast<float>(value_of64(q.order));
      a.parents[b * N + r] = w;
      a.ids[b * N + r] = ended ? a.end_token : key_col(a.part_keys[b * n + static_cast<int>(q.place & 0xffffu)]);
    }
  }
  for (int r = m + tid; r < N; r += NT) {
    a.scores[b * N + r] = neg_inf();
    a.parents[b * N + r] = -1;
    a.ids[b * N + r] = -1;
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Threads of k_top: the K-th largest of the lanes' values cuts the better the more
// lanes there are, which K = 200 needs; with K = 20 fewer threads wait less for each
// other (256 rows of 151936: 30 us with 256, 45 with 512).
int threads_of(int K) { return K > kFewTop ? 512 : 256; }

// Columns of a slice that k_top keeps whole.
int short_slice(int dtype, int threads) { return 4 * threads * (dtype == 2 ? 4 : 8); }

// Slices per row: one where there are rows for four workgroups a CU and more, else as
// many as that takes (256 rows of 151936, K = 20: 30 us, 33 with half as many).  With K
// past 64 joins take longer: one workgroup a CU, and 1024 keys a join (K = 200, 256 rows
// 40 us, 49 with twice as many; 37 rows 29 us, 38 with 4096 keys).  None is
// shorter than what a workgroup keeps whole.  Slices are either short ones that are
// kept whole or each of them, a row's last one too, has the columns of a step of
// the stream, which has no end without one.  Short rows are not cut, but for beams,
// which are joined anyway: up to 128 KB a row a join costs about what it saves.  us a call,
// whole and in slices, K = 20, 1 / 64 / 256 rows: 20000 bf16 13 / 13 / 14 and 17 / 18 / 19, 65000 bf16
// 18 / 20 / 21 and 17 / 18 / 24, 32000 fp32 18 / 19 / 21 and 16 / 17 / 21 (500 rows 23 and 26), 65000
// fp32 25 / 25 / 29 and 16 / 18 / 27; K = 200: 65000 bf16 25 / 26 / 27 either way, 65000 fp32
// 32 / 32 / 36 and 25 / 28 / 35.
constexpr int64_t kWholeRow = 131072;  // bytes

void set_slices(TopArgs& a, int dtype) {
  const int64_t lists = (a.W > 0 ? a.W : 1) * static_cast<int64_t>(a.K);
  const bool many = a.K > kFewTop;
  const int64_t keys = many ? 1024 : kMaxBuffered, most_keys = keys / lists > 1 ? keys / lists : 1;
  const int64_t least = short_slice(dtype, 256);
  const int64_t groups = many ? 256 : 1024;
  int64_t n = (groups + a.T - 1) / (a.T > 0 ? a.T : 1);
  const int64_t most = (int64_t(a.V) + least - 1) / least;
  n = n < most ? n : most;
  n = n < most_keys ? n : most_keys;
  if (a.W == 0 && int64_t(a.V) * (dtype == 2 ? 4 : 2) <= kWholeRow) n = 1;
  const int64_t kept = short_slice(dtype, threads_of(a.K));
  int64_t last;
  do {
    a.slice = static_cast<int>(((int64_t(a.V) + n - 1) / n + 63) / 64 * 64);
    a.nslices = static_cast<int>((int64_t(a.V) + a.slice - 1) / a.slice);
    last = a.V - int64_t(a.nslices - 1) * a.slice;
    n = a.nslices - 1;  // fewer, longer ones; one alone is longer than `kept` if it is not short
  } while (a.slice > kept && last < kept);
}

template <class Tr, int NT, bool SHORT>
hipError_t launch_top_nt(TopArgs a, hipStream_t s) {
  // workgroups of a launch: far below 2^32 work-items whatever T
  const int64_t rows_per = (int64_t(1) << 21) / a.nslices > 0 ? (int64_t(1) << 21) / a.nslices : 1;
  for (int64_t r0 = 0; r0 < a.T; r0 += rows_per) {
    const int64_t rows = a.T - r0 < rows_per ? a.T - r0 : rows_per;
    a.row0 = r0;
    TimedLaunch tl("k_top", s);
    hipLaunchKernelGGL((k_top<Tr, NT, SHORT>), dim3(static_cast<unsigned>(rows * a.nslices)), dim3(NT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class Tr, int NT>
hipError_t launch_top_t(const TopArgs& a, int dtype, hipStream_t s) {
  if (a.slice <= short_slice(dtype, NT)) return launch_top_nt<Tr, NT, true>(a, s);
  return launch_top_nt<Tr, NT, false>(a, s);
}

template <class Tr>
hipError_t launch_top_t(const TopArgs& a, int dtype, hipStream_t s) {
  return threads_of(a.K) == 512 ? launch_top_t<Tr, 512>(a, dtype, s) : launch_top_t<Tr, 256>(a, dtype, s);
}

hipError_t launch_top_slices(int dtype, const TopArgs& a, hipStream_t s) {
  switch (dtype) {
    case 0: return launch_top_t<Bf16>(a, dtype, s);
    case 1: return launch_top_t<Fp16>(a, dtype, s);
    default: return launch_top_t<Fp32>(a, dtype, s);
  }
}

}  // namespace

// Keys of every slice, then their sums.
static size_t part_bytes(const TopArgs& a, size_t* sums_off) {
  const size_t per_row = size_t(a.nslices) * (size_t(a.K) * 8 + 8);
  if (size_t(a.T) > (size_t(1) << 60) / per_row) return 0;
  *sums_off = size_t(a.T) * a.nslices * a.K * 8;
  return (size_t(a.T) * per_row + 255) / 256 * 256;
}

size_t top_workspace_bytes(int dtype, int64_t T, int64_t V, int64_t K) {
  TopArgs a{};
  a.T = T;
  a.V = static_cast<int>(V);
  a.K = static_cast<int>(K);
  set_slices(a, dtype);
  size_t off;
  return a.nslices == 1 ? 256 : part_bytes(a, &off);
}

size_t beam_workspace_bytes(int dtype, int64_t B, int64_t W, int64_t V, int64_t N) {
  TopArgs a{};
  a.T = B * W;
  a.V = static_cast<int>(V);
  a.K = static_cast<int>(N);
  a.W = static_cast<int>(W);
  set_slices(a, dtype);
  size_t off;
  return part_bytes(a, &off);
}

hipError_t launch_top_logits(int dtype, const TopArgs& args, char* ws, hipStream_t s) {
  TopArgs a = args;
  set_slices(a, dtype);
  if (a.nslices == 1) return launch_top_slices(dtype, a, s);
  size_t off = 0;
  part_bytes(a, &off);
  a.part_keys = reinterpret_cast<uint64_t*>(ws);
  a.part_sums = reinterpret_cast<float*>(ws + off);
  hipError_t e = launch_top_slices(dtype, a, s);
  if (e != hipSuccess) return e;
  const size_t lds = (size_t(a.nslices) * a.K + 1 + 1) / 2 * 2 * 8;
  constexpr int64_t kRows = int64_t(1) << 21;
  for (int64_t r0 = 0; r0 < a.T; r0 += kRows) {
    const int64_t rows = a.T - r0 < kRows ? a.T - r0 : kRows;
    a.row0 = r0;
    TimedLaunch tl("k_top_join", s);
    hipLaunchKernelGGL(k_top_join<256>, dim3(static_cast<unsigned>(rows)), dim3(256), lds, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_beam_select(int dtype, const TopArgs& args, int64_t B, char* ws, hipStream_t s) {
  TopArgs a = args;
  set_slices(a, dtype);
  size_t off = 0;
  part_bytes(a, &off);
  a.part_keys = reinterpret_cast<uint64_t*>(ws);
  a.part_sums = reinterpret_cast<float*>(ws + off);
  hipError_t e = launch_top_slices(dtype, a, s);
  if (e != hipSuccess) return e;
  const size_t lds = size_t(a.W) * a.nslices * a.K * sizeof(Candidate);
  constexpr int64_t kRows = int64_t(1) << 21;
  for (int64_t r0 = 0; r0 < B; r0 += kRows) {
    const int64_t rows = B - r0 < kRows ? B - r0 : kRows;
    a.row0 = r0;
    TimedLaunch tl("k_beam_join", s);
    hipLaunchKernelGGL(k_beam_join<256>, dim3(static_cast<unsigned>(rows)), dim3(256), lds, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// states that follow their beams
// ---------------------------------------------------------------------------

// A workgroup takes a piece of one beam's row, reads it once and writes it to
// every slot that goes on from that beam; beam W stands for slots whose parent
// is none, which get zeros.  Vec: the widest type that every address and the
// width are multiples of.  Bound by the copy: 48 x 256 rows of 256 KB, 5.1 GB, in
// 930 us, 5.5 TB/s (stores that stay in the caches 963; 2 vectors a lane 1004, 8 989).
template <class Vec, int U>
__global__ void __launch_bounds__(256) k_beam_reorder(ReorderArgs a) {
  constexpr int kPiece = 256 * U;
  unsigned i = blockIdx.x;
  const unsigned piece = i % a.pieces;
  i /= a.pieces;
  const int w = static_cast<int>(i % static_cast<unsigned>(a.W + 1));
  i /= static_cast<unsigned>(a.W + 1);
  i += a.seg0;  // request, then mid, then outer
  const unsigned nb = static_cast<unsigned>(a.B), nm = static_cast<unsigned>(a.mid);
  const int64_t b = i % nb, mid = i / nb % nm, outer = i / nb / nm;
  const int32_t* parents = a.parents + b * a.N;
  auto takes = [&](int p) { return w == a.W ? p < 0 || p >= a.W : p == w; };
  bool any = false;
  for (int k = threadIdx.x & 63; k < a.N; k += 64) any |= takes(parents[k]);
  if (!__any(any)) return;
  const int64_t width = a.width / static_cast<int64_t>(sizeof(Vec)), at = static_cast<int64_t>(piece) * kPiece + threadIdx.x;
  const Vec* src = reinterpret_cast<const Vec*>(static_cast<const char*>(a.src) + outer * a.src_outer + mid * a.src_mid +
                                                (b * a.W + (w < a.W ? w : 0)) * a.src_row);
  Vec v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = w < a.W && at + u * 256 < width ? src[at + u * 256] : Vec{};
  for (int k = 0; k < a.N; ++k) {
    if (!takes(parents[k])) continue;
    Vec* dst = reinterpret_cast<Vec*>(static_cast<char*>(a.dst) + outer * a.dst_outer + mid * a.dst_mid +
                                      (b * a.N + k) * a.dst_row);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at + u * 256 < width) __builtin_nontemporal_store(v[u], dst + at + u * 256);
  }
}

namespace {

constexpr int kReorderU = 4;  // vectors a lane
constexpr int64_t kReorderGroups = int64_t(1) << 23;  // workgroups of a launch: 2^31 work-items

// Bytes of the widest type that every address, stride and the width allow.
int64_t reorder_bytes(const ReorderArgs& a) {
  const uint64_t all = reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) |
                       static_cast<uint64_t>(a.width | a.src_outer | a.src_mid | a.src_row | a.dst_outer | a.dst_mid | a.dst_row);
  const int64_t low = static_cast<int64_t>(all & (~all + 1));
  return low < 16 ? low : 16;
}

int64_t reorder_pieces(const ReorderArgs& a) {
  const int64_t piece = reorder_bytes(a) * 256 * kReorderU;
  return (a.width + piece - 1) / piece;
}

template <class Vec>
hipError_t launch_reorder_t(ReorderArgs a, hipStream_t s) {
  a.pieces = static_cast<unsigned>(reorder_pieces(a));
  const int64_t per_seg = static_cast<int64_t>(a.pieces) * (a.W + 1), segs = a.B * a.mid * a.outer;
  const int64_t most = kReorderGroups / per_seg;
  for (int64_t s0 = 0; s0 < segs; s0 += most) {
    const int64_t n = segs - s0 < most ? segs - s0 : most;
    a.seg0 = static_cast<unsigned>(s0);
    TimedLaunch tl("k_beam_reorder", s);
    hipLaunchKernelGGL((k_beam_reorder<Vec, kReorderU>), dim3(static_cast<unsigned>(n * per_seg)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool beam_reorder_fits(const ReorderArgs& a) { return reorder_pieces(a) <= kReorderGroups / (a.W + 1); }

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
  switch (reorder_bytes(a)) {
    case 16: return launch_reorder_t<u32x4>(a, s);
    case 8: return launch_reorder_t<uint64_t>(a, s);
    case 4: return launch_reorder_t<uint32_t>(a, s);
    case 2: return launch_reorder_t<uint16_t>(a, s);
    default: return launch_reorder_t<uint8_t>(a, s);
  }
}

}  // namespace lp
