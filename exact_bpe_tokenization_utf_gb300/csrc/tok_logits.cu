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
#include "tok_scan.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr int LG_THREADS = 256;
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr int PER = 16;           // scores per thread and step
constexpr int STEP = LG_THREADS * PER;
constexpr int EDGE = 16;          // places before a slice's first vector, for the scores that come before it (fewer)
constexpr int TABLE = STEP + 64;  // listed tokens of a table: at least as many as a step has scores
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float REF_MAX = 1e37f;  // references of a sum of exponentials stay within this

template <class T> struct Num;
template <> struct Num<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  static constexpr int VEC = 4;  // scores of a vector: 16 bytes
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
  static constexpr int VEC = 8;
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
  static constexpr int VEC = 8;
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// two 32-bit operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c;"
      " mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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

// How a row's scores fall into vectors of 16 bytes: vector i holds the VEC
// scores from v0 + VEC i on, at a 16-byte boundary of the array that is
// written (of the logits where none is).  The scores before and after are
// taken one by one, and where another array's rows lie differently (SHIFTED)
// so are the first and the last vector: reading them takes whole 16-byte
// pieces around them.
struct Grid {
  uint32_t v0, n_vec;
};

template <class T, bool SHIFTED>
__device__ __forceinline__ Grid vectors(const void* row, uint32_t n_logits) {
  constexpr uint32_t VEC = Num<T>::VEC;
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

// A row's vectors on their way from memory: each thread keeps its vectors of
// the next steps in flight (cp.async into slots of its own warp), so that
// about 24 KB per CTA are under way whatever the warps are doing.  Vector i of
// a shifted row lies in the pieces i and i + 1.
template <class T, bool SHIFTED> struct Stream {
  static constexpr int VEC = Num<T>::VEC;
  static constexpr int U = PER / VEC;                       // vectors per thread and step
  static constexpr int DEPTH = sizeof(T) == 4 ? 3 : 4;      // steps in flight
  static constexpr int SLOT = (SHIFTED ? 33 : 32) * 16;     // bytes of a warp's 32 vectors
  static constexpr int STAGE = LG_WARPS * U * SLOT;         // bytes of a step
  static constexpr size_t BYTES = (size_t)DEPTH * STAGE;

  const uint8_t* base;  // the piece of vector 0
  uint32_t shift;       // bytes of the vectors past a 16-byte boundary
  uint8_t* mine;        // this lane's slot of stage 0
  uint32_t i_end;

  __device__ __forceinline__ void open(const T* row, uint32_t v0, uint32_t end, uint8_t* mem) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + v0);
    shift = (uint32_t)(at & 15u);
    base = reinterpret_cast<const uint8_t*>(at - (SHIFTED ? shift : 0u));
    mine = mem + (threadIdx.x >> 5) * U * SLOT + (threadIdx.x & 31u) * 16;
    i_end = end;
  }
  static __device__ __forceinline__ void copy(uint8_t* to, const uint8_t* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
  }
  // the thread's u-th vector, i; want: whether its scores matter (for a shifted row: any of the warp's)
  __device__ __forceinline__ void issue(uint32_t stage, int u, uint32_t i, bool want) const {
    uint8_t* to = mine + stage * STAGE + u * SLOT;
    if (!SHIFTED) {
      if (want && i < i_end) copy(to, base + (size_t)i * 16);
    } else if (want) {
      if (i <= i_end && i_end) copy(to, base + (size_t)i * 16);
      if ((threadIdx.x & 31u) == 0 && i + 32 <= i_end) copy(to + 512, base + (size_t)(i + 32) * 16);
    }
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    if (SHIFTED) __syncwarp();
  }
  // score e of the u-th vector
  __device__ __forceinline__ float score(uint32_t stage, uint32_t u, uint32_t e) const {
    return Num<T>::get(*reinterpret_cast<const T*>(mine + stage * STAGE + u * SLOT + (SHIFTED ? shift : 0u) + e * sizeof(T)));
  }
  __device__ __forceinline__ void scores(uint32_t stage, int u, float* z) const {
    const uint4* q = reinterpret_cast<const uint4*>(mine + stage * STAGE + u * SLOT);
    uint32_t w[5];
    const uint4 a = q[0];
    if constexpr (!SHIFTED) {
      w[0] = a.x;
      w[1] = a.y;
      w[2] = a.z;
      w[3] = a.w;
    } else {
      const uint4 b = q[1];
      const bool two = shift & 8u, one = shift & 4u;
      const uint32_t c0 = two ? a.z : a.x, c1 = two ? a.w : a.y, c2 = two ? b.x : a.z, c3 = two ? b.y : a.w,
                     c4 = two ? b.z : b.x, c5 = two ? b.w : b.y;
      w[0] = one ? c1 : c0;
      w[1] = one ? c2 : c1;
      w[2] = one ? c3 : c2;
      w[3] = one ? c4 : c3;
      w[4] = one ? c5 : c4;
      if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2u) * 8u);
      }
    }
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 f = Num<T>::pair(w, e);
      z[2 * e] = f.x;
      z[2 * e + 1] = f.y;
    }
  }
};

template <class T>
__device__ __forceinline__ void store_scores(T* to, const float* z, float factor) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < Num<T>::VEC / 2; ++e) {
    const float2 y = mul2(make_float2(z[2 * e], z[2 * e + 1]), make_float2(factor, factor));
    Num<T>::put_pair(w, e, y.x, y.y);
  }
  __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
}

// A slice's bits in shared memory, moved so that the bits of a vector lie in
// one byte: bit p is that of token lo + p (lo modulo 2^32: it may be negative).
__host__ __device__ constexpr uint32_t bit_words(uint32_t tokens) { return (tokens + 48 + 31) / 32; }

__device__ __forceinline__ void move_bits(uint32_t* to, const uint32_t* from, uint32_t n_logits, uint32_t lo, uint32_t n) {
  const int n_words = (int)((n_logits + 31) / 32);
  for (uint32_t j = threadIdx.x; j < n; j += LG_THREADS) {
    const int first = (int)(lo + 32 * j) >> 5;
    const uint32_t a = first >= 0 && first < n_words ? __ldg(from + first) : 0u;
    const uint32_t b = first + 1 >= 0 && first + 1 < n_words ? __ldg(from + first + 1) : 0u;
    to[j] = __funnelshift_r(a, b, lo & 31u);
  }
}

// the bits of the slice's vector ii
template <class T>
__device__ __forceinline__ uint32_t vector_bits(const uint32_t* bits, uint32_t ii) {
  const uint8_t* b = reinterpret_cast<const uint8_t*>(bits) + EDGE / 8;
  if (Num<T>::VEC == 8) return b[ii];
  return (uint32_t)b[ii >> 1] >> (4 * (ii & 1u)) & 15u;
}

// The tokens of the lists (generated ids, biases) have a bit each in a slice;
// the number of bits before a token's is its place in a table with the number
// of its occurrences and the smallest index of its bias entries (its top bit:
// there are more), or NO_BIAS.  The table holds TABLE tokens: where a slice
// lists more, it is made for as many steps as it has room for, at least one.
// The main pass leaves listed tokens out; each warp collects those that it
// meets and scores 32 of them at a time.
constexpr uint32_t NO_BIAS = 0x7fffffffu;
constexpr int QUEUE = 64;  // collected tokens of a warp

struct Table {
  uint32_t* count;
  uint32_t* first;   // nullptr: no biases
  uint32_t* bits;    // of the slice
  uint32_t* before;  // bits before each word of them
  uint32_t lo;       // token of bit 0 (modulo 2^32)
  uint32_t base;     // place of the first token of the table
};

constexpr uint32_t table_bytes(bool bias) { return TABLE * (bias ? 8u : 4u); }

// f(i, ids[i]) for this thread's entries of a list, four loads at a time
template <class F>
__device__ __forceinline__ void each_id(const int32_t* ids, int n, F f) {
  for (int i0 = (int)threadIdx.x; i0 < n; i0 += 4 * LG_THREADS) {
    int32_t id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = i0 + j * LG_THREADS < n ? __ldg(ids + i0 + j * LG_THREADS) : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * LG_THREADS < n) f(i0 + j * LG_THREADS, (uint32_t)id[j]);
  }
}

// the bits of the slice's listed tokens, from .. from + n - 1, and their sums
__device__ __forceinline__ void list_bits(const Row& r, const Table& t, uint32_t words, uint32_t from, uint32_t n,
                                          uint32_t* sh) {
  auto one = [&](int, uint32_t v) {
    const uint32_t bit = v - t.lo;
    if (v - from < n) atomicOr(&t.bits[bit >> 5], 1u << (bit & 31));
  };
  each_id(r.gen, r.gen_len, one);
  each_id(r.bias_id, r.bias_n, one);
  __syncthreads();
  const uint32_t each = (words + LG_THREADS - 1) / LG_THREADS, w0 = min(threadIdx.x * each, words), w1 = min(w0 + each, words);
  uint32_t sum = 0, total;
  for (uint32_t w = w0; w < w1; ++w) sum += (uint32_t)__popc(t.bits[w]);
  sum = block_excl_sum(sum, &total, sh);
  for (uint32_t w = w0; w < w1; ++w) {
    t.before[w] = sum;
    sum += (uint32_t)__popc(t.bits[w]);
  }
  if (threadIdx.x == 0) t.before[words] = total;
  __syncthreads();
}

// listed tokens before v
__device__ __forceinline__ uint32_t place_of(const Table& t, uint32_t v) {
  const uint32_t bit = v - t.lo;
  return t.before[bit >> 5] + (uint32_t)__popc(t.bits[bit >> 5] & ((1u << (bit & 31)) - 1u));
}

// The table of the listed tokens from place t.base on, n of them.
__device__ __forceinline__ void fill_table(const Row& r, const Table& t, uint32_t from, uint32_t n_tokens, uint32_t n) {
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += LG_THREADS) {
    t.count[i] = 0;
    if (t.first) t.first[i] = NO_BIAS;
  }
  __syncthreads();
  each_id(r.gen, r.gen_len, [&](int, uint32_t v) {
    if (v - from < n_tokens) atomicAdd(&t.count[place_of(t, v) - t.base], 1u);
  });
  if (t.first && r.bias_n) {
    each_id(r.bias_id, r.bias_n, [&](int i, uint32_t v) {
      if (v - from < n_tokens) atomicMin(&t.first[place_of(t, v) - t.base], (uint32_t)i);
    });
    if (r.bias_n > 1) {
      __syncthreads();
      each_id(r.bias_id, r.bias_n, [&](int i, uint32_t v) {
        if (v - from >= n_tokens) return;
        uint32_t* f = &t.first[place_of(t, v) - t.base];
        if ((*f & NO_BIAS) != (uint32_t)i) atomicOr(f, 0x80000000u);
      });
    }
  }
  __syncthreads();
}

// the number of occurrences of a listed token, and its first bias entry
__device__ __forceinline__ void entries_of(const Table& t, uint32_t v, uint32_t* c, uint32_t* fb) {
  const uint32_t i = place_of(t, v) - t.base;
  *c = t.count[i];
  *fb = t.first ? t.first[i] : NO_BIAS;
}

// The range of steps from `step` on that a table has room for: its end, and the table.
template <int VEC, int U>
__device__ __forceinline__ uint32_t next_table(const Row& r, Table& t, uint32_t step, uint32_t steps, uint32_t v_begin,
                                               uint32_t from, uint32_t to) {
  // listed tokens before the vectors of a step (the first and the last step: before all, and all)
  auto until = [&](uint32_t s) { return place_of(t, s == 0 ? from : s < steps ? v_begin + s * STEP : to); };
  const uint32_t base = until(step);
  uint32_t end = steps;
  while (end > step + 1 && until(end) - base > TABLE) end = step + (end - step + 1) / 2;
  t.base = base;
  const uint32_t t0 = step == 0 ? from : v_begin + step * STEP, t1 = end < steps ? v_begin + end * STEP : to;
  fill_table(r, t, t0, t1 - t0, until(end) - base);
  return end;
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

// The repetition penalty of a thread's seen scores, as a product with its
// reciprocal, within 2^-22 of the quotient: where that can decide which score
// is the largest, they are taken again with score().
__device__ __forceinline__ void penalise(const Row& r, uint32_t seen, float* z) {
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const float f = z[q] > 0.f ? r.inv_rep : r.rep;
    if ((seen >> q) & 1u) z[q] *= f;
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

// the two halves of a cluster's barrier
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct LogitsCall {
  tok_logits_args a;
  uint32_t per;    // vectors per CTA
  uint32_t words;  // of a slice's bits
  uint32_t bits_at; // where they are in shared memory
  int lists;       // there are generated ids or biases
};

// Forward.  A row is cut into the slices of a cluster's CTAs (one CTA: the
// whole row); a step gives each thread 16 scores.  Scores that the mask hides
// are not read.
template <class T, bool SHIFTED>
__global__ void __launch_bounds__(LG_THREADS, 2) k_logits(LogitsCall call) {
  namespace cg = cooperative_groups;
  using S = Stream<T, SHIFTED>;
  constexpr int VEC = S::VEC, U = S::U, DEPTH = S::DEPTH;
  constexpr uint32_t FULL = (1u << PER) - 1u;
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ Part s_part[16];
  __shared__ float s_ref[LG_WARPS], s_sum[LG_WARPS], s_z_pick;
  __shared__ unsigned long long s_key;
  __shared__ uint32_t s_scan[LG_WARPS];
  __shared__ uint2 s_queue[LG_WARPS][QUEUE];
  __shared__ float s_best;  // a score that some token of this CTA has: what is below it is not the top
  const tok_logits_args& a = call.a;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  if (n_ranks > 1) cluster_arrive();  // (waited for before another CTA's shared memory is written)
  const uint32_t b = blockIdx.x / n_ranks, tid = threadIdx.x, lane = tid & 31u;
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  T* out = a.d_out ? static_cast<T*>(a.d_out) + (long long)b * a.out_stride : nullptr;
  const Grid g = vectors<T, SHIFTED>(out ? static_cast<const void*>(out) : x, a.n_logits);
  const uint32_t i_begin = min(rank * call.per, g.n_vec), i_end = min(i_begin + call.per, g.n_vec);
  S in;
  in.open(x, g.v0, i_end, s_mem);
  const Row r = load_row(a, b);
  // the first steps' scores, before it is known which of them are hidden
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
    for (int u = 0; u < U; ++u) in.issue(d, u, i_begin + (d * U + u) * LG_THREADS + tid, !r.none);
    S::commit();
  }
  const bool lists = call.lists && (r.gen_len || r.bias_n);
  const uint32_t lo = g.v0 + i_begin * VEC - EDGE;
  uint32_t* words = reinterpret_cast<uint32_t*>(s_mem + call.bits_at);
  uint32_t *m_bits = nullptr, *s_bits = nullptr, *l_bits = nullptr;
  if (a.d_mask) m_bits = words, words += call.words;
  if (a.d_seen) s_bits = words, words += call.words;
  if (call.lists) l_bits = words, words += call.words;
  if (r.mask) move_bits(m_bits, r.mask, a.n_logits, lo, call.words);
  if (r.seen) move_bits(s_bits, r.seen, a.n_logits, lo, call.words);
  // the slice's tokens: those of its vectors, the first slice's from the row's start, the last one's to its end
  const uint32_t from = rank == 0 ? 0u : g.v0 + i_begin * VEC;
  const uint32_t to = rank == n_ranks - 1 ? a.n_logits : g.v0 + i_end * VEC;
  Table table{};
  table.lo = lo;
  if (lists) {
    table.bits = l_bits;
    table.before = words;
    table.count = reinterpret_cast<uint32_t*>(s_mem + S::BYTES);
    table.first = a.d_bias_off ? table.count + TABLE : nullptr;
    for (uint32_t i = tid; i < call.words; i += LG_THREADS) l_bits[i] = 0;
    __syncthreads();
    list_bits(r, table, call.words, from, to - from, s_scan);
  }
  const uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  const float k = r.inv_t * LOG2E;
  if (tid == 0) {
    s_key = 0;
    s_best = -INFINITY;
    s_z_pick = -INFINITY;
  }
  __syncthreads();

  // the bits of a thread's vectors from i on
  auto bits_at = [&](const uint32_t* bits, uint32_t i) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * LG_THREADS < i_end) m |= vector_bits<T>(bits, i - i_begin + u * LG_THREADS) << (u * VEC);
    return m;
  };
  auto inside = [&](uint32_t i) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * LG_THREADS < i_end) m |= ((1u << VEC) - 1u) << (u * VEC);
    return m;
  };
  auto allowed_at = [&](uint32_t i) { return r.none ? 0u : r.mask ? bits_at(m_bits, i) : inside(i); };

  float ref = -REF_MAX, sum = 0.f;
  const uint32_t steps = max(1u, (i_end - i_begin + U * LG_THREADS - 1) / (U * LG_THREADS));
  uint32_t stage = 0, next = 0, queued = 0;
  // one score outside the vectors or of a listed token, into the sum; the top is left to the caller
  auto one = [&](float z) {
    const float y = z * k;
    if (y > ref + 24.f) {
      const float m = fminf(y, REF_MAX);
      sum *= ex2(ref - m);
      ref = m;
    }
    sum += ex2(fmaf(z, k, -ref));
  };
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step) {
    const uint32_t i = i_begin + step * (U * LG_THREADS) + tid;
    if (lists && step == next) next = next_table<VEC, U>(r, table, step, steps, g.v0 + i_begin * VEC, from, to);
    // the scores outside the vectors: before the first step's, after the last one's
    if ((step == 0 || step + 1 == steps) && tid < 32) {
      const uint32_t head = step == 0 ? g.v0 + i_begin * VEC - from : 0u;
      const uint32_t n = head + (step + 1 == steps ? to - (g.v0 + i_end * VEC) : 0u);
      if (tid < n) {
        const uint32_t t = tid < head ? from + tid : g.v0 + i_end * VEC + (tid - head), at = t - lo;
        float z = -INFINITY;
        if (!r.none && (!r.mask || (m_bits[at >> 5] >> (at & 31) & 1u))) {
          uint32_t c = 0, fb = NO_BIAS;
          if (lists && (l_bits[at >> 5] >> (at & 31) & 1u)) entries_of(table, t, &c, &fb);
          z = score(r, t, c, fb, r.seen && (s_bits[at >> 5] >> (at & 31) & 1u), Num<T>::get(x[t]));
          one(z);
          atomicMax(&s_key, top_key(z, t));
        }
        if (out) out[t] = Num<T>::put(z * r.inv_t);
        if (t == pick) s_z_pick = z;
      }
    }
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = g.v0 + (i + u * LG_THREADS) * VEC;
    const uint32_t special = lists ? bits_at(l_bits, i) : 0u;
    const uint32_t loaded = allowed_at(i), allowed = loaded & ~special, seen = r.seen ? bits_at(s_bits, i) : 0u;
    S::wait();
    float z[PER], vmax = -INFINITY;
    if (allowed) {
#pragma unroll
      for (int u = 0; u < U; ++u) in.scores(stage, u, z + u * VEC);
      if (seen) penalise(r, seen, z);
      if (allowed != FULL) {
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (!((allowed >> q) & 1u)) z[q] = -INFINITY;
      }
#pragma unroll
      for (int q = 0; q < PER; q += 2) vmax = max3(z[q], z[q + 1], vmax);
      const float y = vmax * k;
      if (y > ref + 24.f) {
        const float m = fminf(y, REF_MAX);
        sum *= ex2(ref - m);
        ref = m;
      }
      float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int q = 0; q < PER; q += 2) {
        const float2 w = fma2(make_float2(z[q], z[q + 1]), make_float2(k, k), make_float2(-ref, -ref));
        part[q / 2 & 1] = add2(part[q / 2 & 1], make_float2(ex2(w.x), ex2(w.y)));
      }
      part[0] = add2(part[0], part[1]);
      sum += part[0].x + part[0].y;
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q) z[q] = -INFINITY;
    }
    if (out) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * LG_THREADS < i_end) store_scores(out + v[u], z + u * VEC, r.inv_t);
    }
    // scores that may be the largest, once more and exactly
    const float best = *static_cast<volatile float*>(&s_best);
    const float near = best < INFINITY ? best - fabsf(best) * 0x1p-20f : best;
    unsigned long long key = 0;
    if (__any_sync(0xffffffffu, vmax > -INFINITY && vmax >= near)) {
      float wmax = vmax;
#pragma unroll
      for (int o = 16; o; o >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
      const float at_least = fmaxf(near, wmax - fabsf(wmax) * 0x1p-20f);
      if (vmax >= at_least) {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) m |= (z[q] >= at_least && z[q] > -INFINITY ? 1u : 0u) << q;
        for (; m; m &= m - 1) {
          const uint32_t q = (uint32_t)__ffs((int)m) - 1u, t = v[0] + q / VEC * (LG_THREADS * VEC) + q % VEC;
          key = max(key, top_key(score(r, t, 0, NO_BIAS, (seen >> q) & 1u, in.score(stage, q / VEC, q % VEC)), t));
        }
      }
    }
    // the listed tokens: collected, and scored as soon as there are 32 of them or the table changes
    if (lists) {
      const bool flush = step + 1 == next;
      for (uint32_t m = special & loaded;;) {
        const uint32_t with = __ballot_sync(0xffffffffu, m != 0);
        if (with) {
          if (m) {
            const uint32_t q = (uint32_t)__ffs((int)m) - 1u, t = v[0] + q / VEC * (LG_THREADS * VEC) + q % VEC;
            s_queue[tid >> 5][queued + __popc(with & ((1u << lane) - 1u))] =
                make_uint2(t | ((seen >> q) & 1u) << 31, __float_as_uint(in.score(stage, q / VEC, q % VEC)));
            m &= m - 1;
          }
          queued += __popc(with);
        }
        if (queued >= 32 || (!with && flush && queued)) {
          __syncwarp();
          const uint32_t n = min(queued, 32u);
          if (lane < n) {
            const uint2 e = s_queue[tid >> 5][queued - n + lane];
            const uint32_t t = e.x & 0x7fffffffu;
            uint32_t c, fb;
            entries_of(table, t, &c, &fb);
            const float zs = score(r, t, c, fb, e.x >> 31, __uint_as_float(e.y));
            one(zs);
            if (zs >= best) key = max(key, top_key(zs, t));
            if (out) out[t] = Num<T>::put(zs * r.inv_t);
            if (t == pick) s_z_pick = zs;
          }
          queued -= n;
          __syncwarp();
        }
        if (!with) break;
      }
    }
    if (key) {
      atomicMax(&s_key, key);
      const float zx = key_score(key);
      if (zx > best) s_best = zx;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (pick - v[u] < (uint32_t)VEC && i + u * LG_THREADS < i_end) {
        const uint32_t e = pick - v[u], q = u * VEC + e;
        if ((allowed >> q) & 1u) s_z_pick = score(r, pick, 0, NO_BIAS, (seen >> q) & 1u, in.score(stage, u, e));
      }
    // this stage's slots are free: the step DEPTH later
    __syncwarp();
    {
      const uint32_t later = i + DEPTH * U * LG_THREADS;
      uint32_t want = step + DEPTH < steps ? allowed_at(later) : 0u;
      if (SHIFTED) want = __any_sync(0xffffffffu, want != 0) ? FULL : 0u;
#pragma unroll
      for (int u = 0; u < U; ++u)
        in.issue(stage, u, later + u * LG_THREADS, (want >> (u * VEC)) & ((1u << VEC) - 1u));
      S::commit();
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
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
  if (n_ranks > 1) cluster_wait();
  if (tid == 0) {
    for (int w = 1; w < LG_WARPS; ++w) join_sum(ref, sum, s_ref[w], s_sum[w]);
    Part* parts = n_ranks == 1 ? s_part : cluster.map_shared_rank(s_part, 0);
    parts[rank] = Part{s_key, ref, sum, s_z_pick};
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
    const float lse = nan ? sum : fabsf(y_top) < 1e36f ? LN2 * (ref + log2f(sum)) : y_top;
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
  uint32_t per, words, table_at, bits_at, ranks;
  int lists;
};

// Gradient: slices as in k_logits, but independent CTAs.  exp(y - lse) is
// 2^-24 exp2(z k - lse log2(e) + 24): what is scaled by the gradient and the
// temperature is not lost below 2^-126.  For 32-bit gradients k and lse
// log2(e) are sums of two numbers each (their rounding would weigh |y| times
// on the result) and nothing is added to the exponent.
template <class T, bool SHIFTED>
__global__ void __launch_bounds__(LG_THREADS, 2) k_logits_grad(GradCall call) {
  using S = Stream<T, SHIFTED>;
  constexpr int VEC = S::VEC, U = S::U, DEPTH = S::DEPTH;
  constexpr uint32_t FULL = (1u << PER) - 1u;
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ uint32_t s_scan[LG_WARPS];
  __shared__ uint2 s_queue[LG_WARPS][QUEUE];
  __shared__ float s_queue_grad[LG_WARPS][QUEUE];
  const tok_logits_args& a = call.a;
  const Grad& gr = call.g;
  const uint32_t rank = blockIdx.x % call.ranks, b = blockIdx.x / call.ranks, tid = threadIdx.x, lane = tid & 31u;
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  const T* go = gr.out ? static_cast<const T*>(gr.out) + (long long)b * gr.out_stride : nullptr;
  T* gx = static_cast<T*>(gr.logits) + (long long)b * gr.logits_stride;
  const Grid g = vectors<T, SHIFTED>(gx, a.n_logits);
  const uint32_t i_begin = min(rank * call.per, g.n_vec), i_end = min(i_begin + call.per, g.n_vec);
  S in, gin;
  in.open(x, g.v0, i_end, s_mem);
  if (go) gin.open(go, g.v0, i_end, s_mem + S::BYTES);
  const Row r = load_row(a, b);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i_begin + (d * U + u) * LG_THREADS + tid;
      in.issue(d, u, i, !r.none);
      if (go) gin.issue(d, u, i, !r.none);
    }
    S::commit();
  }
  const bool lists = call.lists && (r.gen_len || r.bias_n);
  const uint32_t lo = g.v0 + i_begin * VEC - EDGE;
  uint32_t* words = reinterpret_cast<uint32_t*>(s_mem + call.bits_at);
  uint32_t *m_bits = nullptr, *s_bits = nullptr, *l_bits = nullptr;
  if (a.d_mask) m_bits = words, words += call.words;
  if (a.d_seen) s_bits = words, words += call.words;
  if (call.lists) l_bits = words, words += call.words;
  if (r.mask) move_bits(m_bits, r.mask, a.n_logits, lo, call.words);
  if (r.seen) move_bits(s_bits, r.seen, a.n_logits, lo, call.words);
  const uint32_t from = rank == 0 ? 0u : g.v0 + i_begin * VEC;
  const uint32_t to = rank == call.ranks - 1 ? a.n_logits : g.v0 + i_end * VEC;
  Table table{};
  table.lo = lo;
  if (lists) {
    table.bits = l_bits;
    table.before = words;
    table.count = reinterpret_cast<uint32_t*>(s_mem + call.table_at);
    table.first = a.d_bias_off ? table.count + TABLE : nullptr;
    for (uint32_t i = tid; i < call.words; i += LG_THREADS) l_bits[i] = 0;
    __syncthreads();
    list_bits(r, table, call.words, from, to - from, s_scan);
  }
  const float glp = gr.logprob ? gr.logprob[b] : 0.f;
  float cp = (gr.lse ? gr.lse[b] : 0.f) - glp, lse = 0.f;
  if (gr.lse || gr.logprob) lse = a.d_lse[b];
  if (fabsf(lse) >= 1e36f) cp = lse = 0.f;  // (nothing but -inf or a type's lowest value)
  uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  if ((int32_t)pick < 0 && gr.logprob) pick = (uint32_t)a.d_top[b];
  const float up = sizeof(T) == 4 ? 0.f : 24.f;
  const double kd = 1.4426950408889634 / (a.d_temperature ? (double)a.d_temperature[b] : 1.0);
  const double ld = (double)lse * 1.4426950408889634 - (double)up;
  const float k = (float)kd, k_lo = (float)(kd - (double)k), lh = (float)ld, l_lo = (float)(ld - (double)lh);
  const float cpt = cp * r.inv_t * (sizeof(T) == 4 ? 1.f : 0x1p-24f);
  if (rank == 0 && gr.bias)
    for (int i = tid; i < r.bias_n; i += LG_THREADS)
      if ((uint32_t)r.bias_id[i] >= a.n_logits) gr.bias[(r.bias - a.d_bias) + i] = 0.f;
  __syncthreads();

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
  auto bits_at = [&](const uint32_t* bits, uint32_t i) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * LG_THREADS < i_end) m |= vector_bits<T>(bits, i - i_begin + u * LG_THREADS) << (u * VEC);
    return m;
  };
  auto inside = [&](uint32_t i) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * LG_THREADS < i_end) m |= ((1u << VEC) - 1u) << (u * VEC);
    return m;
  };
  auto allowed_at = [&](uint32_t i) { return r.none ? 0u : r.mask ? bits_at(m_bits, i) : inside(i); };

  const uint32_t steps = max(1u, (i_end - i_begin + U * LG_THREADS - 1) / (U * LG_THREADS));
  uint32_t stage = 0, next = 0, queued = 0;
  // the gradient of one score; special: with its entries in the lists, whose biases' gradients are written too
  auto one = [&](uint32_t t, bool allowed, bool seen, bool special, float xt, float gt) {
    uint32_t c = 0, fb = NO_BIAS;
    if (special) entries_of(table, t, &c, &fb);
    float dz = 0.f, f = 1.f;
    if (allowed) {
      if (seen || c) f = xt > 0.f ? r.inv_rep : r.rep;
      dz = d_score(score(r, t, c, fb, seen, xt), gt);
      if (t == pick) dz = fmaf(glp, r.inv_t, dz);
    }
    gx[t] = Num<T>::put(dz * f);
    if (gr.bias && (fb & NO_BIAS) != NO_BIAS) {
      float* gb = gr.bias + (r.bias - a.d_bias);
      gb[fb & NO_BIAS] = dz;
      if (fb >> 31)
        for (int e = (int)(fb & NO_BIAS) + 1; e < r.bias_n; ++e)
          if ((uint32_t)r.bias_id[e] == t) gb[e] = dz;
    }
  };
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step) {
    const uint32_t i = i_begin + step * (U * LG_THREADS) + tid;
    if (lists && step == next) next = next_table<VEC, U>(r, table, step, steps, g.v0 + i_begin * VEC, from, to);
    if ((step == 0 || step + 1 == steps) && tid < 32) {  // the scores outside the vectors
      const uint32_t head = step == 0 ? g.v0 + i_begin * VEC - from : 0u;
      const uint32_t n = head + (step + 1 == steps ? to - (g.v0 + i_end * VEC) : 0u);
      if (tid < n) {
        const uint32_t t = tid < head ? from + tid : g.v0 + i_end * VEC + (tid - head), at = t - lo;
        one(t, !r.none && (!r.mask || (m_bits[at >> 5] >> (at & 31) & 1u)), r.seen && (s_bits[at >> 5] >> (at & 31) & 1u),
            lists && (l_bits[at >> 5] >> (at & 31) & 1u), Num<T>::get(x[t]), go ? Num<T>::get(go[t]) : 0.f);
      }
    }
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = g.v0 + (i + u * LG_THREADS) * VEC;
    const uint32_t special = lists ? bits_at(l_bits, i) : 0u, loaded = allowed_at(i), allowed = loaded & ~special;
    const uint32_t seen = r.seen ? bits_at(s_bits, i) : 0u;
    S::wait();
    float z[PER], d[PER];
    if (allowed) {
#pragma unroll
      for (int u = 0; u < U; ++u) in.scores(stage, u, z + u * VEC);
      if (go) {
#pragma unroll
        for (int u = 0; u < U; ++u) gin.scores(stage, u, d + u * VEC);
      } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) d[q] = 0.f;
      }
      uint32_t positive = 0;
      if (seen) {
#pragma unroll
        for (int q = 0; q < PER; ++q) positive |= (z[q] > 0.f ? 1u : 0u) << q;
        penalise(r, seen, z);
      }
#pragma unroll
      for (int q = 0; q < PER; ++q) d[q] = d_score(z[q], d[q]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (pick - v[u] < (uint32_t)VEC) {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (v[u] + e == pick) d[u * VEC + e] = fmaf(glp, r.inv_t, d[u * VEC + e]);
        }
      if (allowed != FULL) {
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (!((allowed >> q) & 1u)) d[q] = 0.f;
      }
      if (seen) {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const float f = (positive >> q) & 1u ? r.inv_rep : r.rep;
          if ((seen >> q) & 1u) d[q] *= f;
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q) d[q] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * LG_THREADS < i_end) store_scores(gx + v[u], d + u * VEC, 1.f);
    // the listed tokens: collected, and taken as soon as there are 32 of them or the table changes
    if (lists) {
      const bool flush = step + 1 == next;
      for (uint32_t m = special;;) {
        const uint32_t with = __ballot_sync(0xffffffffu, m != 0);
        if (with) {
          if (m) {
            const uint32_t q = (uint32_t)__ffs((int)m) - 1u, u = q / VEC, e = q % VEC;
            const uint32_t at = queued + __popc(with & ((1u << lane) - 1u)), ok = (loaded >> q) & 1u;
            s_queue[tid >> 5][at] = make_uint2(v[0] + u * (LG_THREADS * VEC) + e | ((seen >> q) & 1u) << 31 | ok << 30,
                                               ok ? __float_as_uint(in.score(stage, u, e)) : 0u);
            if (go) s_queue_grad[tid >> 5][at] = ok ? gin.score(stage, u, e) : 0.f;
            m &= m - 1;
          }
          queued += __popc(with);
        }
        if (queued >= 32 || (!with && flush && queued)) {
          __syncwarp();
          const uint32_t n = min(queued, 32u);
          if (lane < n) {
            const uint2 e = s_queue[tid >> 5][queued - n + lane];
            one(e.x & 0x3fffffffu, e.x >> 30 & 1u, e.x >> 31, true, __uint_as_float(e.y),
                go ? s_queue_grad[tid >> 5][queued - n + lane] : 0.f);
          }
          queued -= n;
          __syncwarp();
        }
        if (!with) break;
      }
    }
    __syncwarp();
    {
      const uint32_t later = i + DEPTH * U * LG_THREADS;
      uint32_t want = step + DEPTH < steps ? allowed_at(later) : 0u;
      if (SHIFTED) want = __any_sync(0xffffffffu, want != 0) ? FULL : 0u;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool w = (want >> (u * VEC)) & ((1u << VEC) - 1u);
        in.issue(stage, u, later + u * LG_THREADS, w);
        if (go) gin.issue(stage, u, later + u * LG_THREADS, w);
      }
      S::commit();
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    }
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
// keeps some thousand scores, at most the 16 CTAs of a cluster; a slice's
// bits stay within 16 KB each.
uint32_t slices(const tok_handle* h, const tok_logits_args& a) {
  uint32_t s = 1;
  while (s < 16 && ((unsigned long long)a.rows * s < 4ull * (unsigned)h->n_sms || a.n_logits / s > (1u << 17)) &&
         a.n_logits / (2 * s) >= 2048)
    s *= 2;
  return s;
}

size_t stage_bytes(int dtype, bool shifted) {
  if (dtype == TOK_F32) return shifted ? Stream<float, true>::BYTES : Stream<float, false>::BYTES;
  return shifted ? Stream<__half, true>::BYTES : Stream<__half, false>::BYTES;
}

size_t bits_bytes(const tok_logits_args& a, uint32_t words, bool lists) {
  return (size_t)((a.d_mask ? words : 0) + (a.d_seen ? words : 0) + (lists ? 2 * words + 1 : 0)) * sizeof(uint32_t);
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
  const uint32_t vec = 16 / (uint32_t)size_of(a->dtype);
  c.per = (a->n_logits / vec + n - 1) / n;
  c.words = bit_words(c.per * vec);
  const bool shifted = a->d_out && !alike(a->d_logits, a->logits_stride, a->d_out, a->out_stride, a->rows, size_of(a->dtype));
  c.bits_at = (uint32_t)stage_bytes(a->dtype, shifted) + (c.lists ? table_bytes(a->d_bias_off != nullptr) : 0);
  const size_t smem = c.bits_at + bits_bytes(*a, c.words, c.lists);
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
  const size_t size = size_of(a->dtype);
  const uint32_t vec = 16 / (uint32_t)size;
  c.per = (a->n_logits / vec + c.ranks - 1) / c.ranks;
  c.words = bit_words(c.per * vec);
  const bool shifted = !alike(a->d_logits, a->logits_stride, ga->d_grad_logits, ga->grad_logits_stride, a->rows, size) ||
                       (ga->d_grad_out && !alike(ga->d_grad_out, ga->grad_out_stride, ga->d_grad_logits,
                                                 ga->grad_logits_stride, a->rows, size));
  c.table_at = (uint32_t)stage_bytes(a->dtype, shifted) * (ga->d_grad_out ? 2 : 1);
  c.bits_at = c.table_at + (c.lists ? table_bytes(a->d_bias_off != nullptr) : 0);
  const size_t smem = c.bits_at + bits_bytes(*a, c.words, c.lists);
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
