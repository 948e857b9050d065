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
// each step one fp32 operation, rounded on its own (touched_col).
//
// Few columns of a row are touched by a history or a bias, and all others
// pass unchanged, so the two are kept apart.  A workgroup owns a slice of a
// row's columns (the whole row where there are rows enough) and
//   1. sets a bit per touched column in an LDS bitmap, and counts the bits
//      before each group of 128 columns: a touched column's rank in the slice
//      is that count plus a popcount;
//   2. counts by rank: a word per touched column (bit 31: stands in the prompt; below: times in
//      the output), its column, and the last bias entry that names it;
//   3. computes what touched columns give: a thread each, from a gathered
//      logit, the first kRanks of them before the stream, into LDS;
//   4. streams the slice, 16 bytes a lane; the grammar's bits decide what an
//      untouched column gives, and touched ones are filled in from step 3.
//      Scoring only leaves them out of the stream and adds them by themselves;
//      the others store whole vectors this way (storing touched columns singly
//      behind the stream cost 100 of 600 us at 4096 x 151936: each is a
//      partial write of memory that the stream's store has left the cache for).
// Bound: HBM and, when scoring, the vector unit.  Measured: scoring 8192 x 151936
// bf16 0.51 ms (5.2 TB/s of what it must read, 6.6 TB/s with the lines fetched again
// for touched columns; vector unit 85 % busy; without any rule 0.38 ms), gradient
// of 4096 x 151936 bf16 0.52 ms (5.0 TB/s), processing 256 x 129280 fp16 with
// histories of up to 4096 tokens 32 us (of which 9 us are the histories' latency:
// every workgroup of so short a call starts with its history), one row of
// 151936 7 us.  An LDS word per column in place of bitmap and ranks took 2.5 ms
// on the first (slices of 4096 columns, each with its own history pass).
// Counts are integers and the bias entry is a maximum, so the order of the
// LDS atomics does not change any result.  Nothing of size V is kept between
// calls and no dense count matrix passes through memory (it would cost 4 bytes
// a column where the logits cost 2); a history is read twice per slice.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr uint32_t kPromptBit = 0x80000000u;
constexpr int kRanks = 2048;     // touched columns dealt with at a time
constexpr int kMinSlice = 1024;
constexpr int kMaxSlice = 163840;  // columns: 20 KB of bits and 5 KB of counts before them

enum RulesOp { kProcess = 0, kScore = 1, kGrad = 2 };

// One row's scalars.
struct RowRules {
  float rho, f, p;
  const float* values;      // the row's bias values
  const uint32_t* allowed;  // the row's grammar, or null
  const uint32_t* bits;     // LDS: touched columns of the slice, or null
  const uint32_t* pre;      // LDS: bits before each 128 columns
  const uint32_t* given;    // LDS: what the touched columns of ranks < ranks give (fp32 bits)
  int ranks;
  float c;
  // gradient: d = [j = y] gy - p_j (ga + gb t_j), t_j the log2 of p_j
  float nlse2, ga, gb, gy;
  int64_t y;
};

// N bits from position `pos` of a bit array (bit k of the result = pos + k).
// The word behind is read only if they reach it.
template <int N>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int pos) {
  const int w = pos >> 5, sh = pos & 31;
  if (N == 1) return words[w] >> sh;
  const int more = sh > 32 - N ? 1 : 0;
  return __builtin_amdgcn_alignbit(words[w + more], words[w], sh);
}

// x where the bit is set, -inf elsewhere, without a compare.
__device__ __forceinline__ float keep_if(uint32_t bits, int k, float x) {
  const uint32_t m = static_cast<uint32_t>(static_cast<int32_t>(bits << (31 - k)) >> 31);
  return __uint_as_float((m & __float_as_uint(x)) | (~m & 0xff800000u));
}

// The target's own term, gy, is added by its caller.
__device__ __forceinline__ float grad_of(const RowRules& r, float z) {
  const float t = fmaf(z, r.c, r.nlse2);
  const float p = fast_exp2(t);
  return -p * fmaf(r.gb, fmaxf(t, kNoWeight), r.ga);
}

// Touched columns before slice column j.
__device__ __forceinline__ uint32_t rank_of(const uint32_t* bits, const uint32_t* pre, int j) {
  const u32x4 q = *reinterpret_cast<const u32x4*>(bits + (j >> 7) * 4);
  const int k = (j >> 5) & 3;
  const uint32_t word = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
  uint32_t rk = pre[j >> 7] + __popc(word & ((1u << (j & 31)) - 1u));
  if (k > 0) rk += __popc(q.x);
  if (k > 1) rk += __popc(q.y);
  if (k > 2) rk += __popc(q.z);
  return rk;
}

// A bit per column that takes part in the stream.
template <int OP>
__device__ __forceinline__ uint32_t live_bits(const RowRules& r, uint32_t allowed, uint32_t touched) {
  uint32_t live = ~0u;
  if (r.allowed) live = allowed;
  if (OP == kScore && r.bits) live &= ~touched;
  return live;
}

// -inf over the columns of a vector of 16-bit logits whose bit is not set, two
// at a time before they are widened: three instructions a pair, where
// keep_if would take four.
__device__ __forceinline__ u32x4 mask_vector(u32x4 w, uint32_t live, uint32_t neg_inf_pair) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  live &= 0xffu;
  const s16x2 both = __builtin_bit_cast(s16x2, live | live << 16);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const s16x2 up = both << s16x2{static_cast<short>(15 - 2 * k), static_cast<short>(14 - 2 * k)};
    uint32_t m = __builtin_bit_cast(uint32_t, up >> s16x2{15, 15});
    asm("" : "+v"(m));  // stays a mask: as compares and selects it would be six instructions
    w[k] = (m & w[k]) | (~m & neg_inf_pair);
  }
  return w;
}

// What N streamed columns give, from slice column `rel` on; `allowed` and
// `touched` hold a bit per column, bit 0 first (only looked at where the row
// has such bits):
//   kProcess  -inf where not allowed, else the raw value
//   kScore    touched columns and those not allowed become -inf (weigh nothing)
//   kGrad     their gradient without the target's own term, 0 where not allowed
// and for kProcess and kGrad touched columns what step 3 gave them.  Those of
// later ranks are written over later; in place they may only be the raw value
// or, where not allowed, the final -inf.
// MASKED: the -inf are in place already (mask_vector).
template <int OP, int N, bool MASKED = false>
__device__ __forceinline__ void stream_cols(const RowRules& r, float* z, uint32_t allowed, uint32_t touched, int rel) {
  const uint32_t live = live_bits<OP>(r, allowed, touched);
  if (OP == kGrad) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float d = grad_of(r, z[k]);
      // bits, not a product: a NaN beside the grammar gives 0 too
      const uint32_t m = static_cast<uint32_t>(static_cast<int32_t>(live << (31 - k)) >> 31);
      z[k] = r.allowed ? __uint_as_float(__float_as_uint(d) & m) : d;
    }
  } else if (!MASKED && (r.allowed || (OP == kScore && r.bits))) {
#pragma unroll
    for (int k = 0; k < N; ++k) z[k] = keep_if(live, k, z[k]);
  }
  if (OP != kScore && (touched & ((1u << N) - 1u))) {
    const int first = static_cast<int>(rank_of(r.bits, r.pre, rel));
    float got[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int at = first + __popc(touched & ((1u << k) - 1u));
      got[k] = __uint_as_float(r.given[at < r.ranks ? at : 0]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (((touched >> k) & 1u) && first + __popc(touched & ((1u << k) - 1u)) < r.ranks) z[k] = got[k];
  }
}

// The rules on one touched column: w its count word, b its bias entry + 1.
// False if the grammar does not allow it.  The pragma keeps every product and
// sum an operation of its own: it has to cover the operators themselves, the
// rounding functions of the HIP headers (__fmul_rn and the like) are plain
// operators there, and the product f n went unrounded into a multiply-add.
__device__ __forceinline__ bool touched_col(const RowRules& r, uint32_t w, uint32_t b, int col, float& z,
                                            float& slope) {
#pragma clang fp contract(off)
  slope = 1.f;
  if (w) {
    const bool up = z > 0.f;
    slope = up ? 1.f / r.rho : r.rho;
    z = up ? z / r.rho : z * r.rho;
    const uint32_t n = w & ~kPromptBit;
    if (n) {
      z = z - r.f * static_cast<float>(n);
      z = z - r.p;
    }
  }
  if (b) z = z + r.values[b - 1];
  if (r.allowed && !(bits_at<1>(r.allowed, col) & 1u)) {
    z = neg_inf();
    return false;
  }
  return true;
}

// Exclusive sum over the workgroup; *total = the whole.
template <int NT>
__device__ __forceinline__ uint32_t block_exclusive_sum(uint32_t v, uint32_t* sm, uint32_t* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) sm[w] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < NT / 64; ++k) {
    if (k < w) before += sm[k];
    all += sm[k];
  }
  *total = all;
  return before + x - v;
}

// The outputs of a row from its whole state and its target's processed logit.
// s == 0: nothing has weight (shut out, -inf, or so low that z c leaves fp32).
__device__ __forceinline__ void store_score(const RulesArgs& a, int64_t row, RowStat st, float zy) {
#pragma clang fp contract(off)  // s is relative to the rounded product
  const float mc = st.m * a.c, l2s = log2f(st.s);
  const bool near = is_near(mc);
  const int64_t y = a.targets[row];
  float lp = __builtin_nanf("");
  if (y >= 0 && y < a.V && st.s != 0.f) lp = ((near ? fmaf(zy, a.c, -mc) : (zy - st.m) * a.c) - l2s) * kLn2;
  a.logprob[row] = lp;
  if (a.entropy_out) a.entropy_out[row] = (l2s - st.a / st.s) * kLn2;
  // m / tau may be a number where m c is none
  if (a.lse_out) a.lse_out[row] = near ? (mc + l2s) * kLn2 : fmaf(st.m, a.c * kLn2, l2s * kLn2);
}

__device__ __forceinline__ void store_unscored(const RulesArgs& a, int64_t row) {
  a.logprob[row] = 0.f;
  if (a.entropy_out) a.entropy_out[row] = 0.f;
  if (a.lse_out) a.lse_out[row] = 0.f;
}

// The slice's 16-byte vectors, U of them in flight a lane.  The bits are
// loaded ahead of the vectors, so that the first vector's work waits for
// nothing issued behind it.  ALIGNED: head == 0, and a vector's bits are one
// byte (half of one with fp32).  Addresses are a base that the workgroup shares plus a
// 32-bit offset: one instruction a load.  ahead: the lane's first U vectors,
// loaded by the caller where the slice has that many for every lane (kProcess).
template <class Tr, int OP, int NT, int U, bool ALIGNED>
__device__ __forceinline__ void stream_vectors(const RowRules& r, LaneStat& st, const char* xp, char* op, int nvec, int head,
                                               int c0, const u32x4* ahead) {
  constexpr int P = Tr::kPerVec;
  constexpr bool kPairs = Tr::kBytes == 2 && OP != kGrad;
  const uint32_t neg_inf_pair = Tr::neg_inf_bits() * 0x10001u;
  const char* xv = xp + head * Tr::kBytes;
  char* ov = op + head * Tr::kBytes;
  const uint8_t* allowed_bytes = reinterpret_cast<const uint8_t*>(r.allowed) + (c0 >> 3);
  const uint8_t* touched_bytes = reinterpret_cast<const uint8_t*>(r.bits);
  auto byte_bits = [&](const uint8_t* p, uint32_t i) {
    return P == 8 ? static_cast<uint32_t>(p[i]) : static_cast<uint32_t>(p[i >> 1]) >> ((i & 1) * 4);
  };
  auto allowed_of = [&](uint32_t i) {
    return ALIGNED ? byte_bits(allowed_bytes, i) : bits_at<P>(r.allowed, c0 + head + static_cast<int>(i) * P);
  };
  auto touched_of = [&](uint32_t i) {
    return ALIGNED ? byte_bits(touched_bytes, i) : bits_at<P>(r.bits, head + static_cast<int>(i) * P);
  };
  const bool masked = r.allowed || (OP == kScore && r.bits);
  auto finish = [&](u32x4 w, float* z, uint32_t ok, uint32_t hit, uint32_t i) {
    if (kPairs && masked) w = mask_vector(w, live_bits<OP>(r, ok, hit), neg_inf_pair);
    Tr::unpack(w, z);
    stream_cols<OP, P, kPairs>(r, z, ok, hit, head + static_cast<int>(i) * P);
    if (OP != kScore) __builtin_nontemporal_store(Tr::pack(z), reinterpret_cast<u32x4*>(ov + i * 16u));
  };
  // Scored rows pass by once: non-temporal loads (8192 x 151936 without rules
  // 0.42 -> 0.38 ms, gradient of 4096 rows 0.52 -> 0.50-0.515).  The logits of a
  // decode step were written just before, and what is left of them in the
  // caches counts (256 x 129280: non-temporal loads take 1.1 times as long).
  auto load = [&](uint32_t i) {
    if (OP == kProcess) return load_vec(xv + i * 16u);
    return static_cast<u32x4>(__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(xv + i * 16u)));
  };
  uint32_t i = threadIdx.x;
  const uint32_t n = nvec;
  auto several = [&](uint32_t i, const u32x4* have) {
    uint32_t ok[U], hit[U];
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ok[u] = hit[u] = 0;
    if (r.allowed) {
#pragma unroll
      for (int u = 0; u < U; ++u) ok[u] = allowed_of(i + u * NT);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = have ? have[u] : load(i + u * NT);
    if (r.bits) {
#pragma unroll
      for (int u = 0; u < U; ++u) hit[u] = touched_of(i + u * NT);
    }
    float z[U * P];
#pragma unroll
    for (int u = 0; u < U; ++u) finish(w[u], z + u * P, ok[u], hit[u], i + u * NT);
    if (OP == kScore) stat_push_masked<U * P, P>(st, z, r.c);
  };
  if (OP == kProcess && n >= U * NT) {
    several(i, ahead);
    i += U * NT;
  }
  for (; i + (U - 1) * NT < n; i += U * NT) several(i, nullptr);
  for (; i < n; i += NT) {
    const uint32_t ok = r.allowed ? allowed_of(i) : 0u, hit = r.bits ? touched_of(i) : 0u;
    float z[P];
    finish(load(i), z, ok, hit, i);
    if (OP == kScore) stat_push_masked<P, P>(st, z, r.c);
  }
}

template <class Tr, int OP, int NT, int U>
__global__ void __launch_bounds__(NT) k_rules(RulesArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  __shared__ uint32_t sums[NT / 64];
  __shared__ RowStat sm[NT / 64];
  __shared__ float zy;  // processed logit of the target, if it is a touched column
  constexpr int P = Tr::kPerVec;
  const int tid = threadIdx.x;
  const unsigned rel_row = blockIdx.x / static_cast<unsigned>(a.nslices);
  const int slice = static_cast<int>(blockIdx.x - rel_row * static_cast<unsigned>(a.nslices));
  const int64_t row = a.row0 + rel_row;
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
    if (OP == kScore && a.nslices == 1 && tid == 0) store_unscored(a, row);
    return;
  }

  RowRules r;
  r.rho = a.repetition ? a.repetition[row] : 1.f;
  r.f = a.frequency ? a.frequency[row] : 0.f;
  r.p = a.presence ? a.presence[row] : 0.f;
  r.values = nullptr;
  r.allowed = a.allowed ? a.allowed + row * a.ld_allowed : nullptr;
  r.bits = nullptr;
  r.pre = r.given = nullptr;
  r.c = a.c;
  if (OP == kGrad) {
    const float g = a.grad_logprob[row] * a.inv_tau;
    const float gh = a.grad_entropy ? a.grad_entropy[row] * a.inv_tau : 0.f;
    r.nlse2 = -a.lse[row] * kLog2e;
    r.ga = a.grad_entropy ? fmaf(gh, a.entropy[row], g) : g;
    r.gb = gh * kLn2;
    r.gy = g;
    // Nothing has weight, or an lse so far out that its rounding to fp32 is a
    // factor of e and more of every probability: no gradient.
    if (fabsf(r.nlse2) >= kFar) {
      r.nlse2 = neg_inf();
      r.ga = r.gb = r.gy = 0.f;
    }
  }
  if (OP != kProcess) r.y = a.targets[row];

  int64_t len = 0, buf = row, b0 = 0, nb = 0, prompt = 0;
  if (a.tokens) {
    if (a.row_buffer) buf = a.row_buffer[row];
    if (a.prompt_len) prompt = a.prompt_len[row];
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
  const int32_t* tok = a.tokens + buf * a.ld_tokens;
  const int32_t* btok = a.bias_tokens + b0;

  // Columns [0, head) and the tail go one by one, the rest as 16-byte vectors
  // on the grid of what is stored; loads go off it where the input's rows do.
  const RowSplit<Tr> sp(OP == kScore ? xp : op, n);
  // All workgroups of a decode step read their histories at once: the first
  // logits come in meanwhile (4 % of 256 x 129280 fp16; four vectors a lane
  // instead of two take registers that cost a workgroup a CU, and 12 %).
  u32x4 ahead[U];
  if (OP == kProcess && sp.nvec >= U * NT) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      ahead[u] = load_vec(xp + sp.head * Tr::kBytes + (tid + u * NT) * 16u);
  }

  const int ranks = a.slice < kRanks ? a.slice : kRanks;
  uint32_t* bits = lds;                   // [slice / 32]
  uint32_t* pre = bits + a.slice / 32;    // [slice / 128]
  uint32_t* list = pre + a.slice / 128;   // [ranks]
  uint32_t* cnt = list + ranks;           // [ranks]
  uint32_t* bidx = cnt + ranks;           // [ranks], only with biases
  uint32_t touched = 0;                   // columns of the slice

  // Column of a token within the slice; one outside the vocabulary is
  // negative or past every slice.
  auto in_slice = [&](int32_t t, int& j) {
    const int64_t d = static_cast<int64_t>(t) - c0;
    j = static_cast<int>(d);
    return d >= 0 && d < n;
  };
  // The first kHeld x NT tokens stay in registers between the two steps.
  constexpr int kHeld = 8;
  int held[kHeld];  // column within the slice, -1: none
  auto note = [&](int j, int64_t i, uint32_t r0) {
    const uint32_t k = rank_of(bits, pre, j) - r0;
    if (k < static_cast<uint32_t>(ranks)) {
      list[k] = j;
      if (i < prompt)
        atomicOr(cnt + k, kPromptBit);
      else
        atomicAdd(cnt + k, 1u);
    }
  };
  // Step 2 for ranks [r0, r0 + ranks).
  auto count = [&](uint32_t r0) {
    for (int i = tid; i < ranks; i += NT) {
      cnt[i] = 0;
      if (nb > 0) bidx[i] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (held[k] >= 0) note(held[k], tid + k * NT, r0);
    for (int64_t i = tid + kHeld * NT; i < len; i += NT) {
      int j;
      if (in_slice(tok[i], j)) note(j, i, r0);
    }
    for (int64_t i = tid; i < nb; i += NT) {
      int j;
      if (in_slice(btok[i], j)) {
        const uint32_t k = rank_of(bits, pre, j) - r0;
        if (k < static_cast<uint32_t>(ranks)) {
          list[k] = j;
          atomicMax(bidx + k, static_cast<uint32_t>(i) + 1u);  // the last entry listed counts
        }
      }
    }
    __syncthreads();
  };

  if (len > 0 || nb > 0) {  // the same for the whole workgroup
    // loaded while the bits are cleared; a position past the end reads the
    // first token and drops it
    int32_t t[kHeld];
    if (len > 0) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) t[k] = tok[tid + k * NT < len ? tid + k * NT : 0];
    }
    for (int i = tid; i < a.slice / 128; i += NT) reinterpret_cast<u32x4*>(bits)[i] = u32x4{0, 0, 0, 0};
    __syncthreads();
    int j;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      held[k] = tid + k * NT < len && in_slice(t[k], j) ? j : -1;
      if (held[k] >= 0) atomicOr(bits + (held[k] >> 5), 1u << (held[k] & 31));
    }
    for (int64_t i = tid + kHeld * NT; i < len; i += NT)
      if (in_slice(tok[i], j)) atomicOr(bits + (j >> 5), 1u << (j & 31));
    for (int64_t i = tid; i < nb; i += NT)
      if (in_slice(btok[i], j)) atomicOr(bits + (j >> 5), 1u << (j & 31));
    __syncthreads();
    const int per = (a.slice / 128 + NT - 1) / NT;
    uint32_t mine = 0;
    for (int k = 0; k < per; ++k) {
      const int g = tid * per + k;
      if (g < a.slice / 128) {
        const u32x4 q = reinterpret_cast<const u32x4*>(bits)[g];
        mine += __popc(q.x) + __popc(q.y) + __popc(q.z) + __popc(q.w);
      }
    }
    uint32_t at = block_exclusive_sum<NT>(mine, sums, &touched);
    for (int k = 0; k < per; ++k) {
      const int g = tid * per + k;
      if (g < a.slice / 128) {
        const u32x4 q = reinterpret_cast<const u32x4*>(bits)[g];
        pre[g] = at;
        at += __popc(q.x) + __popc(q.y) + __popc(q.z) + __popc(q.w);
      }
    }
    __syncthreads();
    if (touched) {
      r.bits = bits;
      r.values = a.bias_values + b0;
      count(0);
    }
  }

  // What the touched column of rank r0 + k gives.
  auto touched_gives = [&](int k) {
    const int j = static_cast<int>(list[k]);
    float z = Tr::load1(xp, j), slope;
    const bool ok = touched_col(r, cnt[k], nb > 0 ? bidx[k] : 0u, c0 + j, z, slope);
    if (OP == kGrad) z = ok ? (grad_of(r, z) + (c0 + j == r.y ? r.gy : 0.f)) * slope : 0.f;
    return z;
  };
  if (OP != kScore && touched) {
    const int m = touched < static_cast<uint32_t>(ranks) ? static_cast<int>(touched) : ranks;
    for (int k = tid; k < m; k += NT) {
      const float z = touched_gives(k);
      cnt[k] = __float_as_uint(z);
    }
    r.pre = pre;
    r.given = cnt;
    r.ranks = ranks;
    __syncthreads();
  }

  LaneStat st = stat_none();
  auto single = [&](int j) {
    float z = Tr::load1(xp, j);
    stream_cols<OP, 1>(r, &z, r.allowed ? bits_at<1>(r.allowed, c0 + j) : 0u, r.bits ? bits_at<1>(r.bits, j) : 0u, j);
    if (OP == kScore)
      stat_push_masked<1, 1>(st, &z, r.c);
    else
      Tr::store1(op, j, z);
  };
  if (tid < sp.head) single(tid);
  if (sp.head == 0)
    stream_vectors<Tr, OP, NT, U, true>(r, st, xp, op, sp.nvec, 0, c0, ahead);
  else
    stream_vectors<Tr, OP, NT, U, false>(r, st, xp, op, sp.nvec, sp.head, c0, ahead);
  for (int j = n - sp.tail + tid; j < n; j += NT) single(j);

  const bool mine = OP != kProcess && r.y >= c0 && r.y < c0 + n;  // the target is in this slice
  // What is stored singly from here on lies between the stream's stores.
  if (OP != kScore && (mine || touched > static_cast<uint32_t>(ranks))) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // those are done
    __syncthreads();
  }
  if (OP == kGrad && mine && tid == 0) {
    const int j = static_cast<int>(r.y) - c0;
    if (!(r.bits && (bits_at<1>(bits, j) & 1u)) && !(r.allowed && !(bits_at<1>(r.allowed, c0 + j) & 1u)))
      Tr::store1(op, j, grad_of(r, Tr::load1(xp, j)) + r.gy);
  }
  for (uint32_t r0 = OP == kScore ? 0 : ranks; r0 < touched; r0 += ranks) {
    if (r0 > 0) {
      __syncthreads();
      count(r0);
    }
    const int m = touched - r0 < static_cast<uint32_t>(ranks) ? static_cast<int>(touched - r0) : ranks;
    for (int k = tid; k < m; k += NT) {
      const float z = touched_gives(k);
      const int j = static_cast<int>(list[k]);
      if (OP == kScore) {
        stat_push_masked<1, 1>(st, &z, r.c);
        if (c0 + j == r.y) zy = z;
      } else {
        Tr::store1(op, j, z);
      }
    }
  }

  if (OP == kScore) {
    constexpr int W = NT / 64;
    RowStat whole = stat_merge<64>(st, a.c);
    if ((tid & 63) == 0) sm[tid >> 6] = whole;
    __syncthreads();
    if (tid < 64) whole = stat_merge<W>(sm[tid & (W - 1)], a.c);
    if (tid == 0) {
      float z = 0.f;
      if (mine) {
        const int j = static_cast<int>(r.y) - c0;
        if (r.bits && (bits_at<1>(bits, j) & 1u)) {
          z = zy;
        } else {
          z = Tr::load1(xp, j);
          if (r.allowed && !(bits_at<1>(r.allowed, c0 + j) & 1u)) z = neg_inf();
        }
      }
      if (a.nslices == 1) {
        store_score(a, row, whole, z);
      } else {
        float* pt = a.part + (row * a.nslices + slice) * 3;
        pt[0] = whole.m;
        pt[1] = whole.s;
        pt[2] = whole.a;
        if (mine) a.zy[row] = z;
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
    if (lane == 0) store_unscored(a, row);
    return;
  }
  RowStat st{neg_inf(), 0.f, 0.f};
  for (int i = lane; i < a.nslices; i += 64) {
    const float* pt = a.part + (row * a.nslices + i) * 3;
    st = stat_add(st, RowStat{pt[0], pt[1], pt[2]}, a.c);
  }
  st = stat_merge<64>(st, a.c);
  // a target outside the vocabulary has no processed logit: not read
  const int64_t y = a.targets[row];
  if (lane == 0) store_score(a, row, st, y >= 0 && y < a.V ? a.zy[row] : 0.f);
}

// Slices per row: one where there are rows enough for three workgroups a CU,
// which is what their registers let be resident, else as many as that takes, of
// at least kMinSlice columns.  (256 x 129280 fp16: 1024 workgroups take 1.1
// times as long as 768, 2048 1.3, 8192 2 times; 4096 rows of 151936: one slice 0.61 ms, two 0.59, but scoring
// 0.52 ms with one, 0.525 with two.)
void set_slices(RulesArgs& a) {
  const int64_t most = (int64_t(a.V) + kMinSlice - 1) / kMinSlice, least = (int64_t(a.V) + kMaxSlice - 1) / kMaxSlice;
  int64_t n = (768 + a.T - 1) / (a.T > 0 ? a.T : 1);
  n = n < most ? n : most;
  n = n > least ? n : least;
  a.slice = static_cast<int>(((a.V + n - 1) / n + 127) / 128 * 128);
  a.nslices = static_cast<int>((int64_t(a.V) + a.slice - 1) / a.slice);
}

template <class Tr, int OP, int NT>
hipError_t launch_rules_nt(RulesArgs a, const char* name, hipStream_t s) {
  size_t lds = 0;
  if (a.tokens || a.bias_offsets) {
    const int ranks = a.slice < kRanks ? a.slice : kRanks;
    lds = size_t(a.slice) / 8 + a.slice / 32 + size_t(ranks) * 4 * (a.bias_offsets ? 3 : 2);
  }
  // workgroups of a launch: far below 2^32 work-items whatever T
  const int64_t rows_per = (int64_t(1) << 22) / a.nslices > 0 ? (int64_t(1) << 22) / a.nslices : 1;
  for (int64_t r0 = 0; r0 < a.T; r0 += rows_per) {
    const int64_t rows = a.T - r0 < rows_per ? a.T - r0 : rows_per;
    a.row0 = r0;
    TimedLaunch tl(name, s);
    hipLaunchKernelGGL((k_rules<Tr, OP, NT, OP == kScore ? 4 : 2>), dim3(static_cast<unsigned>(rows * a.nslices)), dim3(NT), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class Tr, int OP>
hipError_t launch_rules_t(const RulesArgs& a, const char* name, hipStream_t s) {
  // A few vectors a lane at least, so that short slices do not idle waves.
  // Long ones: 256 threads score 8192 x 151936 in 0.59 ms, 512 in 0.54, 1024 in 0.69.
  if (a.slice >= 16384) return launch_rules_nt<Tr, OP, 512>(a, name, s);
  if (a.slice >= 4096) return launch_rules_nt<Tr, OP, 256>(a, name, s);
  return launch_rules_nt<Tr, OP, 128>(a, name, s);
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
  RulesArgs a;
  a.T = T;
  a.V = static_cast<int>(V);
  set_slices(a);
  const size_t per_row = size_t(a.nslices) * 12 + 4;
  if (size_t(T) > (size_t(1) << 60) / per_row) return 0;
  return (size_t(T) * per_row + 255) / 256 * 256;
}

hipError_t launch_process_logits(int dtype, const RulesArgs& args, hipStream_t s) {
  RulesArgs a = args;
  set_slices(a);
  return launch_rules<kProcess>(dtype, a, "k_process_logits", s);
}

hipError_t launch_processed_score(int dtype, const RulesArgs& args, char* ws, hipStream_t s) {
  RulesArgs a = args;
  set_slices(a);
  a.part = reinterpret_cast<float*>(ws);
  a.zy = a.part + a.T * a.nslices * 3;
  hipError_t e = launch_rules<kScore>(dtype, a, "k_processed_score", s);
  if (e != hipSuccess || a.nslices == 1) return e;
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

hipError_t launch_processed_grad(int dtype, const RulesArgs& args, hipStream_t s) {
  RulesArgs a = args;
  set_slices(a);
  return launch_rules<kGrad>(dtype, a, "k_processed_grad", s);
}

}  // namespace lp
