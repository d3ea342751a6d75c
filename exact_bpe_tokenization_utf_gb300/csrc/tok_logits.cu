// The rules on the scores of the next token (tok_logits_process), their
// gradient (tok_logits_backward) and the bit sets of prompts (tok_seen_bits).
//
// For row b and token v, with c = occurrences of v among the generated ids:
//   z = logit;  c > 0 or seen: z = z > 0 ? z / r : z * r;  z -= f c;  c > 0: z -= p
//   z += bias(v);  masked: z = -inf;  y = z / T
//   top = argmax z (lowest index of equals),  lse = log sum exp y
// and backwards, with p(v) = exp(y(v) - lse),
//   dy(v) = grad_out(v) + (grad_lse - grad_logprob) p(v) + [v == pick] grad_logprob
//   grad_logit(v) = allowed(v) dy(v) / T * (1, 1 / r or r),  grad_bias(i) = dy(id(i)) / T
// Scores, maxima and sums are in 32 bits; a score is rounded to the logits'
// type once, when it is written.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "tok_handle.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr int LG_THREADS = 256;
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr int VEC = 8;            // scores per thread and step
constexpr int EDGE = 16;          // places before a slice's first vector, for the scores that come before it (fewer)
constexpr int SLOTS = 4096;       // of the table of tokens with entries
constexpr int MOST_TOKENS = 3072; // tokens that it takes
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float REF_MAX = 1e37f;  // references of a sum of exponentials stay within this

template <class T> struct Num;
template <> struct Num<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  // scores 2 i and 2 i + 1 of a vector's words
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  static __device__ __forceinline__ void put_pair(uint32_t* w, int i, float a, float b) {
    w[2 * i] = __float_as_uint(a);
    w[2 * i + 1] = __float_as_uint(b);
  }
};
template <> struct Num<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) {
    return __half22float2(*reinterpret_cast<const __half2*>(w + i));
  }
  static __device__ __forceinline__ void put_pair(uint32_t* w, int i, float a, float b) {
    *reinterpret_cast<__half2*>(w + i) = __floats2half2_rn(a, b);
  }
};
template <> struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void put_pair(uint32_t* w, int i, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(w + i) = __floats2bfloat162_rn(a, b);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// with results below 2^-126 kept: a gradient scales them up again
__device__ __forceinline__ float ex2_small(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Grad {
  const void* out;
  long long out_stride;
  const float* lse;
  const float* logprob;
  void* logits;
  long long logits_stride;
  float* bias;
};

// a row's rules
struct Row {
  const uint32_t* mask;  // nullptr: everything is allowed
  bool none;             // nothing is
  const uint32_t* seen;
  const int32_t* gen;
  int gen_len;
  const int32_t* bias_id;
  const float* bias;
  int bias_n;
  float rep, inv_rep, freq, pres, inv_t;
};

__device__ __forceinline__ Row load_row(const tok_logits_args& a, uint32_t b) {
  Row r;
  long long m = b;
  if (a.d_mask && a.d_mask_row) m = a.d_mask_row[b];
  r.none = a.d_mask && m == -1;
  r.mask = a.d_mask && m >= 0 ? a.d_mask + m * a.mask_stride : nullptr;
  r.seen = a.d_seen ? a.d_seen + (long long)b * a.seen_stride : nullptr;
  r.gen_len = a.d_gen ? max(a.d_gen_len[b], 0) : 0;
  r.gen = a.d_gen ? a.d_gen + a.d_gen_start[b] : nullptr;
  r.bias_n = 0;
  if (a.d_bias_off) {
    const long long o = a.d_bias_off[b], n = a.d_bias_off[b + 1] - o;
    r.bias_n = n > 0 ? (int)min(n, (long long)0x7fffffff) : 0;
    r.bias_id = a.d_bias_id + o;
    r.bias = a.d_bias + o;
  }
  r.rep = a.d_repetition ? a.d_repetition[b] : 1.f;
  r.inv_rep = __fdiv_rn(1.f, r.rep);
  r.freq = a.d_frequency ? a.d_frequency[b] : 0.f;
  r.pres = a.d_presence ? a.d_presence[b] : 0.f;
  r.inv_t = a.d_temperature ? __fdiv_rn(1.f, a.d_temperature[b]) : 1.f;
  return r;
}

// How a row's scores fall into vectors of 8: vector i holds v0 + 8 i ..
// v0 + 8 i + 7, at a 16-byte boundary of the array that is written (of the
// logits where none is).  The scores before and after are taken one by one,
// and where another array's rows lie differently so are the first and the
// last vector: reading them takes whole 16-byte pieces around them.
struct Grid {
  uint32_t v0, n_vec;
};

template <class T, bool SHIFTED>
__device__ __forceinline__ Grid vectors(const void* row, uint32_t n_logits) {
  Grid g;
  g.v0 = (uint32_t)((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (uint32_t)sizeof(T);
  g.n_vec = n_logits > g.v0 ? (n_logits - g.v0) / VEC : 0;
  if (SHIFTED) {
    if (g.n_vec <= 2) {
      g.v0 = 0;
      g.n_vec = 0;
    } else {
      g.v0 += VEC;
      g.n_vec -= 2;
    }
  }
  return g;
}

// The words of one vector as they come from memory: whole 16-byte pieces, one
// more where the row is shifted against the vectors.
template <class T, bool SHIFTED> struct Raw {
  static constexpr int WORDS = VEC * (int)sizeof(T) / 4;
  static constexpr int PIECES = WORDS / 4 + (SHIFTED ? 1 : 0);
  uint4 p[PIECES];

  __device__ __forceinline__ void load(const T* row, uint32_t v) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + v) & ~uintptr_t(SHIFTED ? 15 : 0));
#pragma unroll
    for (int i = 0; i < PIECES; ++i) p[i] = __ldcs(q + i);
  }
  // the vector's own words; shift: the row's bytes past a 16-byte boundary at each vector
  __device__ __forceinline__ void words(uint32_t* w, uint32_t shift) const {
    uint32_t a[PIECES * 4];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      a[4 * i] = p[i].x;
      a[4 * i + 1] = p[i].y;
      a[4 * i + 2] = p[i].z;
      a[4 * i + 3] = p[i].w;
    }
    if constexpr (!SHIFTED) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = a[i];
    } else {
      const bool two = shift & 8u, one = shift & 4u;
#pragma unroll
      for (int i = 0; i < WORDS + 2; ++i) a[i] = two ? a[i + 2] : a[i];
#pragma unroll
      for (int i = 0; i < WORDS + 1; ++i) a[i] = one ? a[i + 1] : a[i];
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = sizeof(T) == 4 ? a[i] : __funnelshift_r(a[i], a[i + 1], (shift & 2u) * 8u);
    }
  }
};

// the 8 bits from v on
__device__ __forceinline__ uint32_t bits8(const uint32_t* words, uint32_t v) {
  if ((v & 7u) == 0) return __ldg(reinterpret_cast<const uint8_t*>(words) + (v >> 3));
  return __funnelshift_r(__ldg(words + (v >> 5)), __ldg(words + ((v + 7u) >> 5)), v & 31u) & 255u;
}

__device__ __forceinline__ bool bit_of(const uint32_t* words, uint32_t v) { return (__ldg(words + (v >> 5)) >> (v & 31)) & 1u; }

// What the lists (generated ids, biases) say about the tokens of a slice, in
// shared memory: a bit for each token with entries, and a table of these
// tokens (linear probing from a multiplicative hash) with the number of
// occurrences and the smallest index of the bias entries (its top bit: there
// are more), or NO_BIAS.  Once all entries are in, the scores of the table's
// tokens are computed, all loads in flight at once, and replace the counts;
// whoever meets a token's bit looks its score up.  A table that would hold
// more than MOST_TOKENS tokens is made for half of the range, and so on down
// to a single step's 2,048 tokens, which always fit.
constexpr uint32_t NO_BIAS = 0x7fffffffu;
constexpr uint32_t NO_TOKEN = 0xffffffffu;
constexpr uint32_t GENERATED = 0x80000000u;  // with a key: the token is among the generated ids
static_assert(LG_THREADS * VEC <= MOST_TOKENS && MOST_TOKENS < SLOTS, "a step's tokens fit the table");

struct Lists {
  uint32_t* bits;
  uint32_t* key;
  uint32_t* val;    // occurrences, then the score
  uint32_t* first;  // nullptr: no biases
  uint16_t* used;   // the slots in use
  uint32_t* n_used;
  uint32_t lo;      // token of bit 0 (modulo 2^32)
  uint32_t mask;    // slots - 1
};

__host__ __device__ constexpr uint32_t bit_words(uint32_t per) { return (per * VEC + 48 + 31) / 32; }
size_t lists_bytes(uint32_t per, bool bias) {
  return (SLOTS * (bias ? 3 : 2) + 4 + bit_words(per)) * sizeof(uint32_t) + MOST_TOKENS * sizeof(uint16_t);
}

__device__ __forceinline__ Lists place_lists(uint32_t* mem, bool bias, uint32_t n_entries) {
  Lists l;
  l.key = mem;
  l.val = mem + SLOTS;
  l.first = bias ? mem + 2 * SLOTS : nullptr;
  uint32_t* at = mem + SLOTS * (bias ? 3 : 2);
  l.used = reinterpret_cast<uint16_t*>(at);
  l.n_used = at + MOST_TOKENS / 2;
  l.bits = l.n_used + 4;
  l.lo = 0;
  uint32_t slots = 256;
  while (slots < SLOTS && slots / 2 < n_entries) slots *= 2;
  l.mask = slots - 1;
  return l;
}

__device__ __forceinline__ uint32_t first_slot(const Lists& l, uint32_t v) { return (v * 0x9E3779B1u >> 16) & l.mask; }

__device__ __forceinline__ uint32_t slot_of(const Lists& l, uint32_t v) {
  uint32_t s = first_slot(l, v);
  while ((l.key[s] & ~GENERATED) != v) s = (s + 1) & l.mask;
  return s;
}

// a token's slot, taken if it has none; NO_TOKEN: the table is full
__device__ __forceinline__ uint32_t take_slot(const Lists& l, uint32_t v) {
  uint32_t s = first_slot(l, v);
  for (;;) {
    uint32_t k = *static_cast<volatile uint32_t*>(l.key + s);
    if (k == NO_TOKEN) {
      k = atomicCAS(&l.key[s], NO_TOKEN, v);
      if (k == NO_TOKEN) {
        const uint32_t n = atomicAdd(l.n_used, 1u);
        if (n >= MOST_TOKENS) return NO_TOKEN;  // (at most one per thread beyond: the table keeps free slots)
        l.used[n] = (uint16_t)s;
        const uint32_t at = v - l.lo;
        atomicOr(&l.bits[at >> 5], 1u << (at & 31));
        return s;
      }
    }
    if (k == v) return s;
    s = (s + 1) & l.mask;
  }
}

// The score of a token with c occurrences and bias entries from fb on, from
// its logit; with the divisions and the order of the definition, so that equal
// scores are equal.
__device__ __forceinline__ float score(const Row& r, uint32_t v, uint32_t c, uint32_t fb, bool seen, float x) {
  if (c || seen) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (c) {
    x = __fsub_rn(x, __fmul_rn(r.freq, (float)c));
    x = __fsub_rn(x, r.pres);
  }
  if ((fb & NO_BIAS) != NO_BIAS) {
    float s = r.bias[fb & NO_BIAS];
    if (fb >> 31)  // more than one entry: their sum in the list's order
      for (int i = (int)(fb & NO_BIAS) + 1; i < r.bias_n; ++i)
        if ((uint32_t)r.bias_id[i] == v) s = __fadd_rn(s, r.bias[i]);
    x = __fadd_rn(x, s);
  }
  return x;
}

// The table of the tokens from .. from + n - 1, with their scores.  False (in
// every thread): it is too small for them.
template <class T>
__device__ __forceinline__ bool take_lists(const Row& r, const Lists& l, uint32_t from, uint32_t n, const T* x) {
  for (uint32_t i = threadIdx.x; i <= l.mask; i += LG_THREADS) {
    l.key[i] = NO_TOKEN;
    l.val[i] = 0;
    if (l.first) l.first[i] = NO_BIAS;
  }
  if (threadIdx.x == 0) *l.n_used = 0;
  __syncthreads();
  bool full = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < r.gen_len; i += LG_THREADS) {
    const uint32_t v = (uint32_t)r.gen[i];
    if (v - from < n && !full) {
      const uint32_t s = take_slot(l, v);
      if (s == NO_TOKEN) full = true;
      else atomicAdd(&l.val[s], 1u);
    }
  }
  if (l.first)
    for (int i = threadIdx.x; i < r.bias_n; i += LG_THREADS) {
      const uint32_t v = (uint32_t)r.bias_id[i];
      if (v - from < n && !full) {
        const uint32_t s = take_slot(l, v);
        if (s == NO_TOKEN) full = true;
        else atomicMin(&l.first[s], (uint32_t)i);
      }
    }
  if (__syncthreads_or(full)) return false;
  if (l.first && r.bias_n > 1) {
    for (int i = threadIdx.x; i < r.bias_n; i += LG_THREADS) {
      const uint32_t v = (uint32_t)r.bias_id[i];
      if (v - from < n) {
        const uint32_t s = slot_of(l, v);
        if ((l.first[s] & NO_BIAS) != (uint32_t)i) atomicOr(&l.first[s], 0x80000000u);
      }
    }
    __syncthreads();
  }
  const uint32_t used = *l.n_used;
  for (uint32_t j = threadIdx.x; j < used; j += LG_THREADS) {
    const uint32_t s = l.used[j], v = l.key[s], c = l.val[s];
    const float z = score(r, v, c, l.first ? l.first[s] : NO_BIAS, r.seen && bit_of(r.seen, v), Num<T>::get(x[v]));
    l.val[s] = __float_as_uint(z);
    if (c) l.key[s] = v | GENERATED;
  }
  __syncthreads();
  return true;
}

// The scores of a vector; special: its tokens with entries, generated (where
// asked for): those among the generated ids.  The repetition penalty of the
// others is a product with its reciprocal, within 2^-22 of the quotient:
// where that can decide which score is the largest, they are taken again with
// score().
__device__ __forceinline__ void scores(const Row& r, const Lists& l, uint32_t v, uint32_t seen, uint32_t special,
                                       float* z, uint32_t* generated) {
  if (seen) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float f = z[e] > 0.f ? r.inv_rep : r.rep;
      if ((seen >> e) & 1u) z[e] *= f;
    }
  }
  for (uint32_t m = special; m; m &= m - 1) {
    const int at = __ffs((int)m) - 1;
    const uint32_t s = slot_of(l, v + at);
    const float zs = __uint_as_float(l.val[s]);
    if (generated) *generated |= (l.key[s] >> 31) << at;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e == at) z[e] = zs;
  }
}

// the largest score and its token (the lowest of equals) as one word; 0: none above -inf
__device__ __forceinline__ unsigned long long top_key(float z, uint32_t v) {
  const uint32_t b = __float_as_uint(z + 0.f);  // (-0 counts as 0)
  if (!(z > -INFINITY)) return 0;
  return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - v);
}
__device__ __forceinline__ float key_score(unsigned long long k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return k ? __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b) : -INFINITY;
}

// What is known of a part of a row: its largest score, and the sum of
// exp2(k z - ref) for k = log2(e) / T.  ref follows the scores loosely: the sum
// is in range while ref is within 2^6 or so of the largest k z.
struct Part {
  unsigned long long key;
  float ref, sum, z_pick;
};

// sums in one fixed order: the result does not depend on which CTA or warp comes first
__device__ __forceinline__ void join_sum(float& ref, float& sum, float ref2, float sum2) {
  const float m = fmaxf(ref, ref2);
  sum = sum * ex2(ref - m) + sum2 * ex2(ref2 - m);
  ref = m;
}

struct LogitsCall {
  tok_logits_args a;
  uint32_t per;   // vectors per CTA
  int lists;      // there are generated ids or biases
};

// Forward.  A row is cut into the slices of a cluster's CTAs (one CTA: the
// whole row); each thread takes vectors of 8 scores, up to three of them in
// flight, with the mask's, the seen tokens' and the lists' bits of a vector as
// a byte each.  Scores that the mask hides are not read.
template <class T, bool SHIFTED>
__global__ void __launch_bounds__(LG_THREADS, 3) k_logits(LogitsCall call) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t s_lists[];
  __shared__ Part s_part[16];
  __shared__ float s_ref[LG_WARPS], s_sum[LG_WARPS], s_z_pick;
  __shared__ unsigned long long s_key;
  __shared__ float s_best;  // a score that some token of this CTA has: what is below it is not the top
  const tok_logits_args& a = call.a;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  const uint32_t b = blockIdx.x / n_ranks, tid = threadIdx.x, lane = tid & 31u;
  const Row r = load_row(a, b);
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  T* out = a.d_out ? static_cast<T*>(a.d_out) + (long long)b * a.out_stride : nullptr;
  const uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  const float k = r.inv_t * LOG2E;
  const Grid g = vectors<T, SHIFTED>(out ? static_cast<const void*>(out) : x, a.n_logits);
  const uint32_t shift = (uint32_t)(reinterpret_cast<uintptr_t>(x + g.v0) & 15u);
  const uint32_t i_begin = min(rank * call.per, g.n_vec), i_end = min(i_begin + call.per, g.n_vec);
  Lists l{};
  const bool lists = call.lists && (r.gen_len || r.bias_n);
  if (lists) {
    l = place_lists(s_lists, a.d_bias_off != nullptr, (uint32_t)r.gen_len + (uint32_t)r.bias_n);
    for (uint32_t i = tid; i < bit_words(call.per); i += LG_THREADS) l.bits[i] = 0;
  }
  l.lo = g.v0 + i_begin * VEC - EDGE;
  if (tid == 0) {
    s_key = 0;
    s_best = -INFINITY;
    s_z_pick = -INFINITY;
  }
  cluster.sync();  // (every CTA of the cluster runs before its shared memory is written)

  float ref = -REF_MAX, sum = 0.f;
  auto allowed8 = [&](uint32_t i) -> uint32_t {
    if (i >= i_end || r.none) return 0u;
    return r.mask ? bits8(r.mask, g.v0 + i * VEC) : 255u;
  };
  auto seen8 = [&](uint32_t i) -> uint32_t { return r.seen && i < i_end ? bits8(r.seen, g.v0 + i * VEC) : 0u; };
  // the next three vectors of this thread and their bits
  constexpr int DEPTH = 3;
  Raw<T, SHIFTED> raw[DEPTH];
  uint32_t ok[DEPTH], sn[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    ok[d] = allowed8(i_begin + tid + d * LG_THREADS);
    sn[d] = seen8(i_begin + tid + d * LG_THREADS);
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (ok[d]) raw[d].load(x, g.v0 + (i_begin + tid + d * LG_THREADS) * VEC);

  const uint32_t steps = max(1u, (i_end - i_begin + LG_THREADS - 1) / LG_THREADS);
  uint32_t range = steps, next = 0;  // steps that the table is made for, and the step of the next table
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step) {
    const uint32_t i = i_begin + step * LG_THREADS + tid, v = g.v0 + i * VEC;
    if (step == next) {
      // the scores of this range: its vectors, the first with those before all vectors, the last with those after
      const uint32_t i0 = i_begin + step * LG_THREADS;
      const uint32_t from = rank == 0 && step == 0 ? 0u : g.v0 + i0 * VEC;
      uint32_t i1, to;
      for (;;) {
        i1 = min(i0 + range * LG_THREADS, i_end);
        to = rank == n_ranks - 1 && i1 == i_end ? a.n_logits : g.v0 + i1 * VEC;
        if (!lists) break;
        __syncthreads();
        if (take_lists(r, l, from, to - from, x)) break;
        range = (range + 1) / 2;
      }
      next = step + range;
      if (tid < 32) {  // the scores outside the vectors
        const uint32_t head = g.v0 + i0 * VEC - from, n = head + (to - (g.v0 + i1 * VEC));
        if (tid < n) {
          const uint32_t u = tid < head ? from + tid : g.v0 + i1 * VEC + (tid - head);
          float z = -INFINITY;
          if (!r.none && (!r.mask || bit_of(r.mask, u))) {
            const uint32_t at = u - l.lo;
            if (lists && (l.bits[at >> 5] >> (at & 31) & 1u)) z = __uint_as_float(l.val[slot_of(l, u)]);
            else z = score(r, u, 0, NO_BIAS, r.seen && bit_of(r.seen, u), Num<T>::get(x[u]));
            const float t = z * k;
            if (t > ref + 24.f) {
              const float m = fminf(t, REF_MAX);
              sum *= ex2(ref - m);
              ref = m;
            }
            sum += ex2(fmaf(z, k, -ref));
            atomicMax(&s_key, top_key(z, u));
          }
          if (out) out[u] = Num<T>::put(z * r.inv_t);
          if (u == pick) s_z_pick = z;
        }
      }
    }
    const uint32_t allowed = ok[0], seen = sn[0];
    float z[VEC];
    {
      uint32_t w[Raw<T, SHIFTED>::WORDS];
      raw[0].words(w, shift);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 p = Num<T>::pair(w, e);
        z[2 * e] = p.x;
        z[2 * e + 1] = p.y;
      }
    }
#pragma unroll
    for (int d = 0; d + 1 < DEPTH; ++d) {
      ok[d] = ok[d + 1];
      sn[d] = sn[d + 1];
      raw[d] = raw[d + 1];
    }
    ok[DEPTH - 1] = allowed8(i + DEPTH * LG_THREADS);
    sn[DEPTH - 1] = seen8(i + DEPTH * LG_THREADS);
    if (ok[DEPTH - 1]) raw[DEPTH - 1].load(x, v + DEPTH * LG_THREADS * VEC);

    const bool mine = i < i_end;
    uint32_t special = 0;
    if (lists && mine) special = reinterpret_cast<const uint8_t*>(l.bits)[(v - l.lo) >> 3];
    float vmax = -INFINITY;
    if (allowed) {
      scores(r, l, v, seen, special, z, nullptr);
      if (allowed != 255u) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (!((allowed >> e) & 1u)) z[e] = -INFINITY;
      }
      vmax = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
      const float t = vmax * k;
      if (t > ref + 24.f) {
        const float m = fminf(t, REF_MAX);
        sum *= ex2(ref - m);
        ref = m;
      }
      float q[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) q[e] = ex2(fmaf(z[e], k, -ref));
      sum += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) z[e] = -INFINITY;
    }
    // scores that may be the largest, once more and exactly
    const float best = *static_cast<volatile float*>(&s_best);
    const float near = best < INFINITY ? best - fabsf(best) * 0x1p-20f : best;
    if (__any_sync(0xffffffffu, vmax > -INFINITY && vmax >= near)) {
      float wmax = vmax;
#pragma unroll
      for (int o = 16; o; o >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
      const float at_least = fmaxf(near, wmax - fabsf(wmax) * 0x1p-20f);
      if (vmax >= at_least) {
        unsigned long long key = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (z[e] >= at_least) {
            float zx = z[e];
            if (((seen & ~special) >> e) & 1u) zx = score(r, v + e, 0, NO_BIAS, true, Num<T>::get(x[v + e]));
            key = max(key, top_key(zx, v + e));
          }
        atomicMax(&s_key, key);
        const float zx = key_score(key);
        if (zx > best) s_best = zx;
      }
    }
    if (mine && pick - v < (uint32_t)VEC) {
      float zp = -INFINITY;
      if ((allowed >> (pick - v)) & 1u) {
        if ((special >> (pick - v)) & 1u) zp = __uint_as_float(l.val[slot_of(l, pick)]);
        else zp = score(r, pick, 0, NO_BIAS, (seen >> (pick - v)) & 1u, Num<T>::get(x[pick]));
      }
      s_z_pick = zp;
    }
    // (last: out may be the logits, which the lines above read again)
    if (out && mine) {
      uint32_t w[Raw<T, false>::WORDS];
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) Num<T>::put_pair(w, e, z[2 * e] * r.inv_t, z[2 * e + 1] * r.inv_t);
      uint4* q = reinterpret_cast<uint4*>(out + v);
#pragma unroll
      for (int j = 0; j < Raw<T, false>::PIECES; ++j) __stcs(q + j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
    }
  }

  // the CTA's sum, then the cluster's, and the row's results
#pragma unroll
  for (int o = 16; o; o >>= 1)
    join_sum(ref, sum, __shfl_xor_sync(0xffffffffu, ref, o), __shfl_xor_sync(0xffffffffu, sum, o));
  if (lane == 0) {
    s_ref[tid >> 5] = ref;
    s_sum[tid >> 5] = sum;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < LG_WARPS; ++w) join_sum(ref, sum, s_ref[w], s_sum[w]);
    Part* to = n_ranks == 1 ? s_part : cluster.map_shared_rank(s_part, 0);
    to[rank] = Part{s_key, ref, sum, s_z_pick};
  }
  if (n_ranks > 1) cluster.sync();
  if (rank == 0 && tid == 0) {
    unsigned long long key = s_part[0].key;
    ref = s_part[0].ref;
    sum = s_part[0].sum;
    float z_pick = s_part[0].z_pick;
    for (uint32_t q = 1; q < n_ranks; ++q) {
      key = max(key, s_part[q].key);
      join_sum(ref, sum, s_part[q].ref, s_part[q].sum);
      z_pick = fmaxf(z_pick, s_part[q].z_pick);
    }
    const bool nan = sum != sum;
    const float z_top = key_score(key), y_top = z_top * r.inv_t;
    // beyond the references' range all of the sum is its largest term
    float lse = nan ? sum : fabsf(y_top) < 1e36f ? LN2 * (ref + log2f(sum)) : y_top;
    if (a.d_top) a.d_top[b] = nan || !key ? -1 : (int32_t)(0xffffffffu - (uint32_t)key);
    if (a.d_lse) a.d_lse[b] = lse;
    if (a.d_logprob) {
      const float y = (int32_t)pick >= 0 ? z_pick * r.inv_t : y_top;
      a.d_logprob[b] = nan ? lse : y == -INFINITY ? -INFINITY : y - lse;
    }
  }
}

struct GradCall {
  tok_logits_args a;
  Grad g;
  uint32_t per, ranks;
  int lists;
};

// Gradient: slices as in k_logits, but independent CTAs.  exp(y - lse) is
// 2^-24 exp2(z k - lse log2(e) + 24): what is scaled by the gradient and the
// temperature is not lost below 2^-126.  For 32-bit gradients k and lse
// log2(e) are sums of two numbers each (their rounding would weigh |y| times
// on the result) and nothing is added to the exponent.
template <class T, bool SHIFTED>
__global__ void __launch_bounds__(LG_THREADS, 3) k_logits_grad(GradCall call) {
  extern __shared__ __align__(16) uint32_t s_lists[];
  const tok_logits_args& a = call.a;
  const Grad& gr = call.g;
  const uint32_t rank = blockIdx.x % call.ranks, b = blockIdx.x / call.ranks, tid = threadIdx.x;
  const Row r = load_row(a, b);
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  const T* go = gr.out ? static_cast<const T*>(gr.out) + (long long)b * gr.out_stride : nullptr;
  T* gx = static_cast<T*>(gr.logits) + (long long)b * gr.logits_stride;
  const float glp = gr.logprob ? gr.logprob[b] : 0.f;
  float cp = (gr.lse ? gr.lse[b] : 0.f) - glp, lse = 0.f;
  if (gr.lse || gr.logprob) lse = a.d_lse[b];
  if (fabsf(lse) >= 1e36f) cp = lse = 0.f;  // (nothing but -inf or a type's lowest value)
  uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  if ((int32_t)pick < 0 && gr.logprob) pick = (uint32_t)a.d_top[b];
  const double kd = 1.4426950408889634 / (a.d_temperature ? (double)a.d_temperature[b] : 1.0);
  const float up = sizeof(T) == 4 ? 0.f : 24.f;
  const double ld = (double)lse * 1.4426950408889634 - (double)up;
  const float k = (float)kd, k_lo = (float)(kd - (double)k), lh = (float)ld, l_lo = (float)(ld - (double)lh);
  const float cpt = cp * r.inv_t * (sizeof(T) == 4 ? 1.f : 0x1p-24f);
  const Grid g = vectors<T, SHIFTED>(gx, a.n_logits);
  const uint32_t shift = (uint32_t)(reinterpret_cast<uintptr_t>(x + g.v0) & 15u);
  const uint32_t go_shift = (uint32_t)(reinterpret_cast<uintptr_t>(go + g.v0) & 15u);
  const uint32_t i_begin = min(rank * call.per, g.n_vec), i_end = min(i_begin + call.per, g.n_vec);
  Lists l{};
  const bool lists = call.lists && (r.gen_len || r.bias_n);
  if (lists) {
    l = place_lists(s_lists, a.d_bias_off != nullptr, (uint32_t)r.gen_len + (uint32_t)r.bias_n);
    for (uint32_t i = tid; i < bit_words(call.per); i += LG_THREADS) l.bits[i] = 0;
  }
  l.lo = g.v0 + i_begin * VEC - EDGE;
  if (rank == 0 && gr.bias)
    for (int i = tid; i < r.bias_n; i += LG_THREADS)
      if ((uint32_t)r.bias_id[i] >= a.n_logits) gr.bias[(r.bias - a.d_bias) + i] = 0.f;

  // the gradient of a score before the temperature, from the score and grad_out
  auto d_score = [&](float z, float d) -> float {
    d *= r.inv_t;
    if (cpt != 0.f) {
      if (sizeof(T) == 4) {
        z = fmaxf(z, -FLT_MAX);  // (-inf times k_lo is no number)
        d = fmaf(cpt, ex2_small(fmaf(z, k, -lh) + fmaf(z, k_lo, -l_lo)), d);
      } else {
        d = fmaf(cpt, ex2(fmaf(z, k, -lh)), d);
      }
    }
    return d;
  };
  // the gradients of a token's bias entries
  auto bias_grad = [&](uint32_t v, uint32_t s, float dz) {
    const uint32_t fb = l.first ? l.first[s] : NO_BIAS;
    if (!gr.bias || (fb & NO_BIAS) == NO_BIAS) return;
    float* to = gr.bias + (r.bias - a.d_bias);
    to[fb & NO_BIAS] = dz;
    if (fb >> 31)
      for (int i = (int)(fb & NO_BIAS) + 1; i < r.bias_n; ++i)
        if ((uint32_t)r.bias_id[i] == v) to[i] = dz;
  };
  auto allowed8 = [&](uint32_t i) -> uint32_t {
    if (i >= i_end || r.none) return 0u;
    return r.mask ? bits8(r.mask, g.v0 + i * VEC) : 255u;
  };
  auto seen8 = [&](uint32_t i) -> uint32_t { return r.seen && i < i_end ? bits8(r.seen, g.v0 + i * VEC) : 0u; };
  constexpr int DEPTH = 2;
  Raw<T, SHIFTED> raw[DEPTH], graw[DEPTH];
  uint32_t ok[DEPTH], sn[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    ok[d] = allowed8(i_begin + tid + d * LG_THREADS);
    sn[d] = seen8(i_begin + tid + d * LG_THREADS);
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (ok[d]) {
      const uint32_t v = g.v0 + (i_begin + tid + d * LG_THREADS) * VEC;
      raw[d].load(x, v);
      if (go) graw[d].load(go, v);
    }

  const uint32_t steps = max(1u, (i_end - i_begin + LG_THREADS - 1) / LG_THREADS);
  uint32_t range = steps, next = 0;
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step) {
    const uint32_t i = i_begin + step * LG_THREADS + tid, v = g.v0 + i * VEC;
    if (step == next) {
      const uint32_t i0 = i_begin + step * LG_THREADS;
      const uint32_t from = rank == 0 && step == 0 ? 0u : g.v0 + i0 * VEC;
      uint32_t i1, to;
      for (;;) {
        i1 = min(i0 + range * LG_THREADS, i_end);
        to = rank == call.ranks - 1 && i1 == i_end ? a.n_logits : g.v0 + i1 * VEC;
        if (!lists) break;
        __syncthreads();
        if (take_lists(r, l, from, to - from, x)) break;
        range = (range + 1) / 2;
      }
      next = step + range;
      if (tid < 32) {
        const uint32_t head = g.v0 + i0 * VEC - from, n = head + (to - (g.v0 + i1 * VEC));
        if (tid < n) {
          const uint32_t u = tid < head ? from + tid : g.v0 + i1 * VEC + (tid - head), at = u - l.lo;
          const bool special = lists && (l.bits[at >> 5] >> (at & 31) & 1u);
          const uint32_t s = special ? slot_of(l, u) : 0;
          float dz = 0.f, f = 1.f;
          if (!r.none && (!r.mask || bit_of(r.mask, u))) {
            const bool seen = r.seen && bit_of(r.seen, u);
            const float xu = Num<T>::get(x[u]);
            if (seen || (special && l.key[s] >> 31)) f = xu > 0.f ? r.inv_rep : r.rep;
            dz = d_score(special ? __uint_as_float(l.val[s]) : score(r, u, 0, NO_BIAS, seen, xu), go ? Num<T>::get(go[u]) : 0.f);
            if (u == pick) dz += glp * r.inv_t;
          }
          gx[u] = Num<T>::put(dz * f);
          if (special) bias_grad(u, s, dz);
        }
      }
    }
    const uint32_t allowed = ok[0], seen = sn[0];
    float z[VEC], d[VEC];
    {
      uint32_t w[Raw<T, SHIFTED>::WORDS];
      raw[0].words(w, shift);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 p = Num<T>::pair(w, e);
        z[2 * e] = p.x;
        z[2 * e + 1] = p.y;
      }
      if (go) {
        graw[0].words(w, go_shift);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 p = Num<T>::pair(w, e);
          d[2 * e] = p.x;
          d[2 * e + 1] = p.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q + 1 < DEPTH; ++q) {
      ok[q] = ok[q + 1];
      sn[q] = sn[q + 1];
      raw[q] = raw[q + 1];
      if (go) graw[q] = graw[q + 1];
    }
    ok[DEPTH - 1] = allowed8(i + DEPTH * LG_THREADS);
    sn[DEPTH - 1] = seen8(i + DEPTH * LG_THREADS);
    if (ok[DEPTH - 1]) {
      raw[DEPTH - 1].load(x, v + DEPTH * LG_THREADS * VEC);
      if (go) graw[DEPTH - 1].load(go, v + DEPTH * LG_THREADS * VEC);
    }
    if (i >= i_end) continue;
    uint32_t special = 0;
    if (lists) special = reinterpret_cast<const uint8_t*>(l.bits)[(v - l.lo) >> 3];
    if (allowed) {
      uint32_t positive = 0, hit = seen;
      if (seen | special) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) positive |= (z[e] > 0.f ? 1u : 0u) << e;
      }
      scores(r, l, v, seen, special, z, &hit);
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[e] = d_score(z[e], d[e]);
      if (pick - v < (uint32_t)VEC) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (v + e == pick) d[e] = fmaf(glp, r.inv_t, d[e]);
      }
      if (allowed != 255u) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (!((allowed >> e) & 1u)) d[e] = 0.f;
      }
      if (special && gr.bias) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if ((special >> e) & 1u) bias_grad(v + e, slot_of(l, v + e), d[e]);
      }
      if (hit) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float f = (positive >> e) & 1u ? r.inv_rep : r.rep;
          if ((hit >> e) & 1u) d[e] *= f;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        d[e] = 0.f;
        if (gr.bias && ((special >> e) & 1u)) bias_grad(v + e, slot_of(l, v + e), 0.f);
      }
    }
    uint32_t w[Raw<T, false>::WORDS];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) Num<T>::put_pair(w, e, d[2 * e], d[2 * e + 1]);
    uint4* q = reinterpret_cast<uint4*>(gx + v);
#pragma unroll
    for (int j = 0; j < Raw<T, false>::PIECES; ++j) __stcs(q + j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
  }
}

// One CTA per row: the bits in shared memory, then the row.
__global__ void __launch_bounds__(LG_THREADS) k_seen_bits(const int32_t* ids, const long long* off, uint32_t n_logits,
                                                          uint32_t* seen, long long stride, int keep) {
  extern __shared__ uint32_t s_bits[];
  const uint32_t words = (n_logits + 31) / 32;
  uint32_t* row = seen + (long long)blockIdx.x * stride;
  for (uint32_t w = threadIdx.x; w < words; w += LG_THREADS) s_bits[w] = keep ? row[w] : 0u;
  __syncthreads();
  const long long end = off[blockIdx.x + 1];
  for (long long i = off[blockIdx.x] + threadIdx.x; i < end; i += LG_THREADS) {
    const uint32_t v = (uint32_t)ids[i];
    if (v < n_logits) atomicOr(&s_bits[v >> 5], 1u << (v & 31));
  }
  __syncthreads();
  for (uint32_t w = threadIdx.x; w < words; w += LG_THREADS) row[w] = s_bits[w];
}

// Slices of a row: enough CTAs to fill the GPU a few times over while a slice
// keeps some thousand scores, at most the 16 CTAs of a cluster.
uint32_t slices(const tok_handle* h, const tok_logits_args& a) {
  uint32_t s = 1;
  while (s < 16 && (unsigned long long)a.rows * s < 4ull * (unsigned)h->n_sms && a.n_logits / (2 * s) >= 2048) s *= 2;
  return s;
}

// whether rows of an array lie like those of another towards 16-byte boundaries
bool alike(const void* p, int64_t stride, const void* q, int64_t q_stride, uint32_t rows, size_t size) {
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) != 0) return false;
  return rows == 1 || ((uint64_t)(stride - q_stride) * size & 15u) == 0;
}

size_t size_of(int dtype) { return dtype == TOK_F32 ? 4 : 2; }

template <class K, class C>
cudaError_t launch(K kernel, const C& call, unsigned ctas, unsigned cluster, size_t smem, cudaStream_t s) {
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(LG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (cluster > 1) {
    if (cluster > 8) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, call);
}

template <class T>
cudaError_t launch_forward(const LogitsCall& c, bool shifted, unsigned ctas, unsigned cluster, size_t smem, cudaStream_t s) {
  return shifted ? launch(k_logits<T, true>, c, ctas, cluster, smem, s) : launch(k_logits<T, false>, c, ctas, cluster, smem, s);
}
template <class T>
cudaError_t launch_grad(const GradCall& c, bool shifted, unsigned ctas, size_t smem, cudaStream_t s) {
  return shifted ? launch(k_logits_grad<T, true>, c, ctas, 1, smem, s) : launch(k_logits_grad<T, false>, c, ctas, 1, smem, s);
}

int launched(tok_handle* h, cudaError_t e) {
  h->launches += 1;
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
}

// nullptr, or what is wrong with the arguments
const char* check_logits(const tok_logits_args* a) {
  if (!a || !a->d_logits) return "logits: the arguments or the logits are NULL";
  if (a->dtype != TOK_F32 && a->dtype != TOK_F16 && a->dtype != TOK_BF16) return "logits: unknown type";
  if (a->n_logits == 0 || a->n_logits > MAX_LOGITS) return "logits: n_logits is out of range";
  if (a->rows > 0x7ffffffu) return "logits: too many rows";
  const int64_t n = a->n_logits, words = (n + 31) / 32;
  if (a->logits_stride < n || (a->d_out && a->out_stride < n)) return "logits: a row stride is below n_logits";
  if ((a->d_seen && a->seen_stride < words) || (a->d_mask && a->mask_stride < words))
    return "logits: a stride of bits is below a row's words";
  if ((a->d_gen && (!a->d_gen_start || !a->d_gen_len)) || (a->d_bias_off && (!a->d_bias_id || !a->d_bias)))
    return "logits: generated ids need their starts and lengths, bias offsets their ids and values";
  if (a->d_mask_row && !a->d_mask) return "logits: mask rows without masks";
  return nullptr;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_logits_process(tok_handle* h, const tok_logits_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (const char* w = check_logits(a)) return fail(h, TOK_EINVAL, w);
  if (a->rows == 0) return TOK_OK;
  DeviceGuard g(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LogitsCall c{};
  c.a = *a;
  c.lists = a->d_gen || a->d_bias_off;
  const uint32_t n = slices(h, *a);
  c.per = (a->n_logits / VEC + n - 1) / n;
  const size_t smem = c.lists ? lists_bytes(c.per, a->d_bias_off != nullptr) : 0;
  const bool shifted = a->d_out && !alike(a->d_logits, a->logits_stride, a->d_out, a->out_stride, a->rows, size_of(a->dtype));
  const unsigned ctas = a->rows * n;
  const cudaError_t e = a->dtype == TOK_F32   ? launch_forward<float>(c, shifted, ctas, n, smem, s)
                        : a->dtype == TOK_F16 ? launch_forward<__half>(c, shifted, ctas, n, smem, s)
                                              : launch_forward<__nv_bfloat16>(c, shifted, ctas, n, smem, s);
  return launched(h, e);
} catch (...) {
  return TOK_ENOMEM;
}

int tok_logits_backward(tok_handle* h, const tok_logits_args* a, const tok_logits_grad_args* ga, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (const char* w = check_logits(a)) return fail(h, TOK_EINVAL, w);
  if (!ga || !ga->d_grad_logits) return fail(h, TOK_EINVAL, "logits: the gradient's arguments or buffer are NULL");
  if (ga->grad_logits_stride < (int64_t)a->n_logits || (ga->d_grad_out && ga->grad_out_stride < (int64_t)a->n_logits))
    return fail(h, TOK_EINVAL, "logits: a row stride is below n_logits");
  if ((ga->d_grad_lse || ga->d_grad_logprob) && !a->d_lse)
    return fail(h, TOK_EINVAL, "logits: the gradient of lse or logprob needs the forward pass's lse");
  if (ga->d_grad_logprob && !a->d_top && !a->d_pick)
    return fail(h, TOK_EINVAL, "logits: the gradient of logprob needs the picks or the forward pass's top");
  if (a->rows == 0) return TOK_OK;
  DeviceGuard gd(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GradCall c{};
  c.a = *a;
  c.g = Grad{ga->d_grad_out, ga->grad_out_stride, ga->d_grad_lse,  ga->d_grad_logprob,
               ga->d_grad_logits, ga->grad_logits_stride, a->d_bias_off ? ga->d_grad_bias : nullptr};
  c.lists = a->d_gen || a->d_bias_off;
  c.ranks = slices(h, *a);
  c.per = (a->n_logits / VEC + c.ranks - 1) / c.ranks;
  const size_t smem = c.lists ? lists_bytes(c.per, a->d_bias_off != nullptr) : 0, size = size_of(a->dtype);
  const bool shifted = !alike(a->d_logits, a->logits_stride, ga->d_grad_logits, ga->grad_logits_stride, a->rows, size) ||
                       (ga->d_grad_out && !alike(ga->d_grad_out, ga->grad_out_stride, ga->d_grad_logits,
                                                 ga->grad_logits_stride, a->rows, size));
  const unsigned ctas = a->rows * c.ranks;
  const cudaError_t e = a->dtype == TOK_F32   ? launch_grad<float>(c, shifted, ctas, smem, s)
                        : a->dtype == TOK_F16 ? launch_grad<__half>(c, shifted, ctas, smem, s)
                                              : launch_grad<__nv_bfloat16>(c, shifted, ctas, smem, s);
  return launched(h, e);
} catch (...) {
  return TOK_ENOMEM;
}

int tok_seen_bits(tok_handle* h, const int32_t* d_ids, const int64_t* d_item_off, uint32_t n, uint32_t n_logits,
                  uint32_t* d_seen, int64_t seen_stride, int keep, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (!d_ids || !d_item_off || !d_seen || n == 0) return fail(h, TOK_EINVAL, "seen bits: a buffer is NULL, or n is 0");
  const uint32_t words = (n_logits + 31) / 32;
  if (n > 0x7fffffffu || n_logits == 0 || n_logits > MAX_LOGITS || seen_stride < (int64_t)words)
    return fail(h, TOK_EINVAL, "seen bits: n, n_logits or seen_stride is out of range");
  DeviceGuard g(h->dev);
  const size_t bytes = words * sizeof(uint32_t);
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_seen_bits, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return cuda_fail(h, e, "seen bits");
  }
  k_seen_bits<<<n, LG_THREADS, bytes, static_cast<cudaStream_t>(stream)>>>(
      d_ids, reinterpret_cast<const long long*>(d_item_off), n_logits, d_seen, seen_stride, keep);
  return launched(h, cudaGetLastError());
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
