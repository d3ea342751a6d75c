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
//
// Both directions are one pass over the scores, which reads and writes each
// once.  What bounds it is neither the bytes nor the issue of instructions alone:
// for 512 rows of 100,257 bf16 scores with seen sets and lists of 2,000 ids on a
// GB300, 32 us of bytes, 48.7M warp instructions (39 us if one were issued in
// every cycle) and 74 us measured, with instructions issued in 54% of all cycles
// and DRAM at 29%.  The row's scalars, bits and listed tokens take a CTA 8 to 15
// us before its first step and after its last, which do not overlap its own
// scores, and the SM's other CTAs' only in part.  Of those 30 instructions of a
// thread for each score the main pass has 22 or fewer: 13 without rules, 6 for a
// seen set, up to 3 where the input's rows and the output's lie differently
// towards 16 bytes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "tok_handle.cuh"
#include "tok_scan.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
// 256 threads, 3 CTAs per SM (80 registers).  Six CTAs of 128 threads: one row
// 12.0 us against 10.3, 64 rows 21.3 against 18.4, 512 rows 75.2 against 73.6.
constexpr int LG_THREADS = 256;
constexpr int LG_CTAS = 3;        // per SM, where shared memory has room for them
constexpr int SB_THREADS = 512;   // of k_seen_bits
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr int PER = 16;           // scores per thread and step
constexpr int EDGE = 16;          // places before a slice's first vector, for the scores that come before it (fewer)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// References of a sum of exponentials stay within this: up to there z k lies no
// more than half a spacing (32) above a reference that was rounded from it, and
// no sum overflows below the largest reference.  Y_MAX: from here on (in natural
// units, well within REF_MAX) scores are 32 apart or more, and so is what 32 bits
// tell apart of their log-sum-exp: the largest score is all of it.
constexpr float REF_MAX = 0x1p30f;
constexpr float Y_MAX = 0x1p29f;
// From here on the rounding of an lse is 2^-4 or more, and exp(y - lse) only makes
// sense with the y that lse was formed from, rounded alike.
constexpr float Y_FAR = 0x1p20f;

template <class T> struct Num;
template <> struct Num<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  static constexpr int VEC = 4;  // scores of a vector: 16 bytes
  static constexpr uint32_t MINUS_INF = 0xff800000u;  // in all of a word's scores
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
  static constexpr uint32_t MINUS_INF = 0xfc00fc00u;
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
  static constexpr uint32_t MINUS_INF = 0xff80ff80u;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void put_pair(uint32_t* w, int i, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(w + i) = __floats2bfloat162_rn(a, b);
  }
};

// Of the words of a thread's u-th vector (scores u VEC on), the scores whose
// bit of m is clear become those of fill.  For 16-bit scores the bits of two
// neighbours are moved to the tops of bytes and prmt spreads them: six
// instructions for four scores, where a test and a choice each take eight.
template <class T>
__device__ __forceinline__ void hide(uint32_t* w, uint32_t m, int u, uint32_t fill) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (sizeof(T) == 4) {
      if (!((m >> (u * 4 + e)) & 1u)) w[e] = fill;
    } else {
      uint32_t keep;
      asm("prmt.b32 %0, %1, %2, %3;" : "=r"(keep) : "r"(m << (7 - 2 * e)), "r"(m << (6 - 2 * e)), "r"(u == 0 ? 0xcc88 : 0xdd99));
      w[e] = (w[e] & keep) | (fill & ~keep);
    }
  }
}

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

// two 32-bit numbers, and operations on both in one instruction
struct Two {
  float2 v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float x, float y) : v(make_float2(x, y)) {}
  __device__ __forceinline__ explicit Two(float2 x) : v(x) {}
  __device__ __forceinline__ void get(float& x, float& y) const {
    x = v.x;
    y = v.y;
  }
};
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { return Two(__ffma2_rn(a.v, b.v, c.v)); }
__device__ __forceinline__ Two add2(Two a, Two b) { return Two(__fadd2_rn(a.v, b.v)); }
__device__ __forceinline__ Two mul2(Two a, Two b) { return Two(__fmul2_rn(a.v, b.v)); }

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
  r.bias_id = nullptr;
  r.bias = nullptr;
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

  const uint8_t* from;  // this lane's piece of the next step to be issued
  uint32_t shift;       // bytes of the vectors past a 16-byte boundary
  uint8_t* mine;        // this lane's slot of stage 0
  uint32_t slot;        // the same as a shared address

  __device__ __forceinline__ void open(const T* row, uint32_t v0, uint32_t i_begin, uint8_t* mem) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + v0);
    shift = (uint32_t)(at & 15u);
    from = reinterpret_cast<const uint8_t*>(at - (SHIFTED ? shift : 0u)) + ((size_t)i_begin + threadIdx.x) * 16;
    mine = mem + (threadIdx.x >> 5) * U * SLOT + (threadIdx.x & 31u) * 16;
    slot = (uint32_t)__cvta_generic_to_shared(mine);
  }
  static __device__ __forceinline__ void copy(uint32_t to, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
  }
  // The next step into a stage, all of whose vectors exist; bit u of want:
  // whether scores of the u-th vector matter (for a shifted row: any).
  __device__ __forceinline__ void issue(uint32_t stage, uint32_t want) {
    const uint32_t to = slot + stage * STAGE;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (want >> u & 1u) copy(to + u * SLOT, from + u * (LG_THREADS * 16));
      if (SHIFTED && (want & 1u) && (threadIdx.x & 31u) == 0) copy(to + u * SLOT + 512, from + u * (LG_THREADS * 16) + 512);
    }
    from += U * LG_THREADS * 16;
  }
  // The same of a slice's last steps: only what lies within its n vectors, the
  // thread's first one being ii.  (A shifted row's last piece belongs to the
  // last vector, which another lane may hold.)
  __device__ __forceinline__ void issue_end(uint32_t stage, uint32_t want, uint32_t ii, uint32_t n) {
    const uint32_t to = slot + stage * STAGE, end = n ? n + (SHIFTED ? 1u : 0u) : 0u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = ii + u * LG_THREADS;
      if ((want >> u & 1u) && i < end) copy(to + u * SLOT, from + u * (LG_THREADS * 16));
      if (SHIFTED && (want & 1u) && (threadIdx.x & 31u) == 0 && i + 32 < end) copy(to + u * SLOT + 512, from + u * (LG_THREADS * 16) + 512);
    }
    from += U * LG_THREADS * 16;
  }
  // the copies issued since the last call are a step
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    if (SHIFTED) __syncwarp();
  }
  // before the slots serve as other memory
  static __device__ __forceinline__ void close() { asm volatile("cp.async.wait_all;" ::: "memory"); }
  // score e of the u-th vector
  __device__ __forceinline__ float score(uint32_t stage, uint32_t u, uint32_t e) const {
    return Num<T>::get(*reinterpret_cast<const T*>(mine + stage * STAGE + u * SLOT + (SHIFTED ? shift : 0u) + e * sizeof(T)));
  }
  // the four words of the u-th vector
  __device__ __forceinline__ void words(uint32_t stage, int u, uint32_t* to) const {
    const uint8_t* q = mine + stage * STAGE + u * SLOT;
    if constexpr (!SHIFTED) {
      const uint4 a = *reinterpret_cast<const uint4*>(q);
      to[0] = a.x;
      to[1] = a.y;
      to[2] = a.z;
      to[3] = a.w;
    } else {
      uint32_t w[5];
      // (8 bytes at a time, so that the place of the first takes care of half of the shift)
      const uint2* p = reinterpret_cast<const uint2*>(q + (shift & 8u));
      const uint2 a = p[0], b = p[1], c = p[2];
      const bool one = shift & 4u;
      w[0] = one ? a.y : a.x;
      w[1] = one ? b.x : a.y;
      w[2] = one ? b.y : b.x;
      w[3] = one ? c.x : b.y;
      w[4] = one ? c.y : c.x;
      if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2u) * 8u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = w[i];
    }
  }
  // the thread's scores, those without a bit in m as -inf (HIDE)
  template <bool HIDE>
  __device__ __forceinline__ void scores(uint32_t stage, float* z, uint32_t m) const {
    uint32_t w[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) words(stage, u, w[u]);
    if (HIDE && m != (1u << PER) - 1u) {
#pragma unroll
      for (int u = 0; u < U; ++u) hide<T>(w[u], m, u, Num<T>::MINUS_INF);
    }
#pragma unroll
    for (int q = 0; q < PER; q += 2) {
      const float2 f = Num<T>::pair(w[q / VEC], q % VEC / 2);
      z[q] = f.x;
      z[q + 1] = f.y;
    }
  }
};

template <class T>
__device__ __forceinline__ void store_scores(T* to, const float* z, float factor) {
  const Two f(factor, factor);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < Num<T>::VEC / 2; ++e) {
    float a, b;
    mul2(Two(z[2 * e], z[2 * e + 1]), f).get(a, b);
    Num<T>::put_pair(w, e, a, b);
  }
  __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
}

// the vector of a masked place
template <class T>
__device__ __forceinline__ void store_all(T* to, float x) {
  uint32_t w[1 + sizeof(T) / 4];
  Num<T>::put_pair(w, 0, x, x);
  __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[0], w[0], w[0]));
}

// the sums of a slice's words, four words each, in whole 16 bytes
__host__ __device__ constexpr uint32_t fours_of(uint32_t words) { return (words / 4 + 3) / 4 * 4; }

// A slice's bits in shared memory, moved so that the bits of a vector lie in
// one byte: bit p is that of token lo + p (lo modulo 2^32: it may be negative).
__host__ __device__ constexpr uint32_t bit_words(uint32_t tokens) { return ((tokens + 48 + 31) / 32 + 3) / 4 * 4; }

__device__ __forceinline__ void move_bits(uint32_t* to, const uint32_t* from, uint32_t n_logits, uint32_t lo, uint32_t n) {
  const int n_words = (int)((n_logits + 31) / 32);
#pragma unroll 4
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

// The tokens of the lists (generated ids, biases) have a bit each in a slice,
// and the main pass leaves them out.  The number of bits before a token's is
// its place among them; after the main pass a table in shared memory takes,
// by place, the token, the number of its occurrences and the smallest index of
// its bias entries (its top bit: there are more), or NO_BIAS, and each thread
// scores every LG_THREADS-th of them.  Where a slice lists more tokens than the
// table holds, it is filled several times.
constexpr uint32_t NO_BIAS = 0x7fffffffu;

struct Table {
  uint32_t* token;
  uint32_t* count;
  uint32_t* first;   // where there are biases
  uint32_t* bits;    // of the slice
  uint32_t* before;  // bits before every fourth word of them
  uint32_t lo;       // token of bit 0 (modulo 2^32)
  uint32_t total;    // listed tokens
  uint32_t room;     // of the table
};

__device__ __forceinline__ bool listed(const Table& t, uint32_t v) {
  return (t.bits[(v - t.lo) >> 5] >> ((v - t.lo) & 31)) & 1u;
}

// f(i, ids[i]) for this thread's entries of a list, four loads at a time
template <class F>
__device__ __forceinline__ void each_id(const int32_t* ids, int n, F f) {
  const uint32_t end = (uint32_t)n;  // (the last i0 may pass 2^31)
  for (uint32_t i0 = threadIdx.x; i0 < end; i0 += 4 * LG_THREADS) {
    int32_t id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = i0 + j * LG_THREADS < end ? __ldg(ids + i0 + j * LG_THREADS) : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * LG_THREADS < end) f((int)(i0 + j * LG_THREADS), (uint32_t)id[j]);
  }
}

// the bits of the slice's listed tokens, from .. from + n - 1, and their sums
__device__ __forceinline__ void list_bits(const Row& r, Table& t, uint32_t words, uint32_t from, uint32_t n, uint32_t* sh) {
  auto one = [&](int, uint32_t v) {
    const uint32_t bit = v - t.lo;
    if (v - from < n) atomicOr(&t.bits[bit >> 5], 1u << (bit & 31));
  };
  each_id(r.gen, r.gen_len, one);
  each_id(r.bias_id, r.bias_n, one);
  __syncthreads();
  // sums of four words each (16 bytes a thread, side by side), then their scan, four sums a thread
  const uint32_t fours = (words + 3) / 4;
  for (uint32_t f = threadIdx.x; f < fours; f += LG_THREADS) {
    const uint4 b = reinterpret_cast<const uint4*>(t.bits)[f];
    t.before[f] = (uint32_t)(__popc(b.x) + __popc(b.y) + __popc(b.z) + __popc(b.w));
  }
  __syncthreads();
  uint32_t carry = 0;
  for (uint32_t f0 = 0; f0 < fours; f0 += 4 * LG_THREADS) {
    const uint32_t f = f0 + 4 * threadIdx.x;
    uint4 n = make_uint4(0, 0, 0, 0);
    if (f < fours) n = reinterpret_cast<const uint4*>(t.before)[f / 4];
    if (f + 1 >= fours) n.y = 0;
    if (f + 2 >= fours) n.z = 0;
    if (f + 3 >= fours) n.w = 0;
    uint32_t all;
    const uint32_t at = carry + block_excl_sum(n.x + n.y + n.z + n.w, &all, sh);
    if (f < fours) reinterpret_cast<uint4*>(t.before)[f / 4] = make_uint4(at, at + n.x, at + n.x + n.y, at + n.x + n.y + n.z);
    carry += all;
  }
  t.total = carry;
}

// the place of a listed token
__device__ __forceinline__ uint32_t place_of(const Table& t, uint32_t v) {
  const uint32_t bit = v - t.lo, word = bit >> 5;
  uint32_t n = t.before[bit >> 7] + (uint32_t)__popc(t.bits[word] & ((1u << (bit & 31)) - 1u));
#pragma unroll
  for (uint32_t back = 1; back < 4; ++back)
    if ((word & 3u) >= back) n += (uint32_t)__popc(t.bits[word - back]);
  return n;
}

// one(token, occurrences, first bias entry, load(token)) for this thread's
// listed tokens, in the order of the tokens, four loads at a time
template <class L, class F>
__device__ __forceinline__ void each_listed(const Row& r, Table& t, void* mem, uint32_t bytes, bool bias, uint32_t from,
                                            uint32_t n_tokens, L load, F one) {
  t.room = bytes / (bias ? 12u : 8u);
  t.token = static_cast<uint32_t*>(mem);
  t.count = t.token + t.room;
  t.first = bias ? t.count + t.room : t.count;  // (read with biases only)
  for (uint32_t base = 0; base < t.total; base += t.room) {
    const uint32_t n = min(t.room, t.total - base);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n; i += LG_THREADS) {
      t.count[i] = 0;
      if (bias) t.first[i] = NO_BIAS;
    }
    __syncthreads();
    each_id(r.gen, r.gen_len, [&](int, uint32_t v) {
      if (v - from >= n_tokens) return;
      const uint32_t i = place_of(t, v) - base;
      if (i >= n) return;
      t.token[i] = v;  // (the same from every occurrence)
      atomicAdd(&t.count[i], 1u);
    });
    if (bias && r.bias_n) {
      each_id(r.bias_id, r.bias_n, [&](int e, uint32_t v) {
        if (v - from >= n_tokens) return;
        const uint32_t i = place_of(t, v) - base;
        if (i >= n) return;
        t.token[i] = v;
        atomicMin(&t.first[i], (uint32_t)e);
      });
      if (r.bias_n > 1) {
        __syncthreads();
        each_id(r.bias_id, r.bias_n, [&](int e, uint32_t v) {
          if (v - from >= n_tokens) return;
          const uint32_t i = place_of(t, v) - base;
          if (i < n && (t.first[i] & NO_BIAS) != (uint32_t)e) atomicOr(&t.first[i], 0x80000000u);
        });
      }
    }
    __syncthreads();
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 4 * LG_THREADS) {
      uint32_t v[4];
      float2 x[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        v[j] = i0 + j * LG_THREADS < n ? t.token[i0 + j * LG_THREADS] : 0xffffffffu;
        x[j] = make_float2(0.f, 0.f);
        if (v[j] != 0xffffffffu) x[j] = load(v[j]);
      }
#pragma unroll 1
      for (uint32_t i = i0; i < n && i < i0 + 4 * LG_THREADS; i += LG_THREADS) {
        one(v[0], t.count[i], bias ? t.first[i] : NO_BIAS, x[0]);
        // (moved up, so that the body stands here once)
        v[0] = v[1];
        v[1] = v[2];
        v[2] = v[3];
        x[0] = x[1];
        x[1] = x[2];
        x[2] = x[3];
      }
    }
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
    x = __fadd_rn(x, r.bias[fb & NO_BIAS]);
    if (fb >> 31)  // more than one entry: one after another, in the list's order
      for (int i = (int)(fb & NO_BIAS) + 1; i < r.bias_n; ++i)
        if ((uint32_t)r.bias_id[i] == v) x = __fadd_rn(x, r.bias[i]);
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

__device__ __forceinline__ float max16(const float* z) {
  const float a = max3(z[0], z[1], z[2]), b = max3(z[3], z[4], z[5]), c = max3(z[6], z[7], z[8]),
              d = max3(z[9], z[10], z[11]), e = max3(z[12], z[13], z[14]);
  return max3(max3(a, b, c), max3(d, e, z[15]), z[15]);
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
// exp2(k z - ref) for k = log2(e) / T.  ref follows the scores loosely: a warp
// raises it when a score passes it by 24, so that a sum stays below 2^24 times
// its number of terms.
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

// A row's slice as a CTA takes it, for both kernels: its vectors, its bits in
// shared memory and its listed tokens.
constexpr size_t BITS_ROOM = 16 * LG_THREADS / 8 + 64;  // read, not used, behind a slice's last bits: a step's
struct Shape {
  uint32_t per;      // vectors per CTA
  uint32_t words;    // of a slice's bits
  uint32_t front;    // bytes of shared memory for the scores in flight, later the table of listed tokens
  int lists;         // there are generated ids or biases
};

template <class T> struct Slice {
  static constexpr int VEC = Num<T>::VEC, U = PER / VEC;
  static constexpr uint32_t FULL = (1u << PER) - 1u;
  uint32_t v0, i_begin, i_end;  // the first vector's first token; the vectors
  uint32_t from, to;            // the tokens
  uint32_t *mask, *seen;        // bits, where there are any (pointers into the slice's memory in any case)
  bool none, masked, marked, lists;
  Table table;

  __device__ __forceinline__ void open(const tok_logits_args& a, const Shape& sh, const Grid& g, uint32_t rank, uint32_t n_ranks) {
    v0 = g.v0;
    i_begin = min(rank * sh.per, g.n_vec);
    i_end = min(i_begin + sh.per, g.n_vec);
    // the first slice's tokens from the row's start, the last one's to its end
    from = rank == 0 ? 0u : v0 + i_begin * VEC;
    to = rank == n_ranks - 1 ? a.n_logits : v0 + i_end * VEC;
    table.lo = v0 + i_begin * VEC - EDGE;
  }
  // (ends with a barrier)
  __device__ __forceinline__ void fill(const tok_logits_args& a, const Shape& sh, const Row& r, uint8_t* mem, uint32_t* scan) {
    uint32_t* w = reinterpret_cast<uint32_t*>(mem + sh.front);
    none = r.none;
    masked = r.mask != nullptr;
    marked = r.seen != nullptr;
    lists = sh.lists && (r.gen_len || r.bias_n);
    table.token = table.count = table.first = reinterpret_cast<uint32_t*>(mem);
    table.bits = table.before = mask = seen = w;
    table.total = table.room = 0;
    if (lists) {
      table.before = w + sh.words;
      w += sh.words + fours_of(sh.words);
      for (uint32_t i = threadIdx.x; i < sh.words; i += LG_THREADS) table.bits[i] = 0;
    }
    if (masked) {
      mask = w;
      w += sh.words;
      move_bits(mask, r.mask, a.n_logits, table.lo, sh.words);
    }
    if (marked) {
      seen = w;
      move_bits(seen, r.seen, a.n_logits, table.lo, sh.words);
    }
    __syncthreads();
    if (lists) list_bits(r, table, sh.words, from, to - from, scan);
    __syncthreads();
  }
  __device__ __forceinline__ uint32_t n_vec() const { return i_end - i_begin; }
  // the bits of a thread's vectors, the first one ii after the slice's first
  // (beyond the slice: of what follows in memory)
  __device__ __forceinline__ uint32_t bits_at(const uint32_t* bits, uint32_t ii) const {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) m |= vector_bits<T>(bits, ii + u * LG_THREADS) << (u * VEC);
    return m;
  }
  // the scores of a thread's vectors that are the slice's
  __device__ __forceinline__ uint32_t inside(uint32_t ii) const {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ii + u * LG_THREADS < n_vec()) m |= ((1u << VEC) - 1u) << (u * VEC);
    return m;
  }
  // those that the mask allows; whole: the slice has all of the step's vectors
  __device__ __forceinline__ uint32_t allowed_at(uint32_t ii, bool whole) const {
    uint32_t m = masked ? bits_at(mask, ii) : none ? 0u : FULL;
    if (!whole) m &= inside(ii);
    return m;
  }
  // which of a thread's vectors have allowed scores; for a shifted row: whether any of the warp's has
  template <bool SHIFTED>
  __device__ __forceinline__ uint32_t wanted(uint32_t ii, bool whole) const {
    if (!masked) return none ? 0u : 0xffu;
    const uint32_t m = allowed_at(ii, whole);
    if (SHIFTED) return __any_sync(0xffffffffu, m != 0) ? 0xffu : 0u;
    uint32_t w = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) w |= (m >> (u * VEC) & ((1u << VEC) - 1u) ? 1u : 0u) << u;
    return w;
  }
  __device__ __forceinline__ bool allows(uint32_t t) const {
    const uint32_t at = t - table.lo;
    return !none && (!masked || (mask[at >> 5] >> (at & 31) & 1u));
  }
  __device__ __forceinline__ bool saw(uint32_t t) const {
    const uint32_t at = t - table.lo;
    return marked && (seen[at >> 5] >> (at & 31) & 1u);
  }
  // the tid-th score outside the vectors (fewer than 32), or NO_TOKEN
  __device__ __forceinline__ uint32_t outside(uint32_t tid) const {
    const uint32_t head = v0 + i_begin * VEC - from, n = head + (to - (v0 + i_end * VEC));
    return tid < n ? (tid < head ? from + tid : v0 + i_end * VEC + (tid - head)) : 0xffffffffu;
  }
};

struct LogitsCall {
  tok_logits_args a;
  Shape shape;
};

// Forward.  A row is cut into the slices of a cluster's CTAs (one CTA: the
// whole row); a step gives each thread 16 scores.  Scores that the mask hides
// are not read.  The largest score is found among products with reciprocals
// (within 2^-22); only those that come near it are taken once more with the
// definition's divisions, so that the choice is exact.  IN_PLACE: out is logits.
//
// Measured, with all rules on unless stated: one row of 100,257 bf16 scores
// 10.3 us (the launch is 7); 64 rows of 50,257 f16 scores 18.4 us; 200 rows of
// 100,257 f32 scores, half of them masked and nothing written, 28.1 us (2.9 TB/s of
// logits); 512 rows of 100,257 bf16 scores, no mask, 74 us (2.9 TB/s read and
// written).
template <class T, bool SHIFTED, bool IN_PLACE>
__global__ void __launch_bounds__(LG_THREADS, LG_CTAS) k_logits(LogitsCall call) {
  namespace cg = cooperative_groups;
  using S = Stream<T, SHIFTED>;
  constexpr int VEC = S::VEC, U = S::U, DEPTH = S::DEPTH;
  constexpr uint32_t ALL = 0xffffffffu;
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ Part s_part[16];
  __shared__ float s_ref[LG_WARPS], s_sum[LG_WARPS], s_z_pick;
  __shared__ uint32_t s_scan[LG_WARPS];
  __shared__ unsigned long long s_key;
  __shared__ float s_best;  // a score that some token of this CTA has: what is below it is not the top
  const tok_logits_args& a = call.a;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  if (n_ranks > 1) cluster_arrive_only();  // (waited for before another CTA's shared memory is written)
  const uint32_t b = blockIdx.x / n_ranks, tid = threadIdx.x, lane = tid & 31u;
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  T* out = a.d_out ? static_cast<T*>(a.d_out) + (long long)b * a.out_stride : nullptr;
  Slice<T> c;
  c.open(a, call.shape, vectors<T, SHIFTED>(out ? static_cast<const void*>(out) : x, a.n_logits), rank, n_ranks);
  S in;
  in.open(x, c.v0, c.i_begin, s_mem);
  // the first steps' scores, before it is known which of them are hidden
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    in.issue_end(d, 0xffu, tid + d * U * LG_THREADS, c.n_vec());
    S::commit();
  }
  const Row r = load_row(a, b);
  const uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  const float x_pick = pick - c.from < c.to - c.from ? Num<T>::get(x[pick]) : 0.f;
  if (tid == 0) {
    s_key = 0;
    s_best = -INFINITY;
    s_z_pick = -INFINITY;
  }
  c.fill(a, call.shape, r, s_mem, s_scan);

  // ref is the same in all threads of a warp
  const float k = r.inv_t * LOG2E;
  const Two k2(k, k);
  float ref = -REF_MAX, sum = 0.f;
  unsigned long long key = 0;
  auto raise = [&](float y) {  // ref to y or higher
    const float m = fmaxf(ref, fminf(y, REF_MAX));
    sum *= ex2(ref - m);
    ref = m;
  };
  if (tid == 0 && pick - c.from < c.to - c.from && c.allows(pick) && !(c.lists && listed(c.table, pick)))
    s_z_pick = score(r, pick, 0, NO_BIAS, c.saw(pick), x_pick);
  if (tid < 32) {  // the scores outside the vectors
    const uint32_t t = c.outside(tid);
    float z = -INFINITY;
    if (t != 0xffffffffu && !(c.lists && listed(c.table, t))) {
      if (c.allows(t)) z = score(r, t, 0, NO_BIAS, c.saw(t), Num<T>::get(x[t]));
      if (out) out[t] = Num<T>::put(z * r.inv_t);
      key = top_key(z, t);
    }
    float y = z * k;
#pragma unroll
    for (int o = 16; o; o >>= 1) y = fmaxf(y, __shfl_xor_sync(ALL, y, o));
    raise(y);
    sum = ex2(fmaf(z, k, -ref));
  }
  const uint32_t n = c.n_vec(), steps = (n + U * LG_THREADS - 1) / (U * LG_THREADS), whole = n / (U * LG_THREADS);
  T* to = out + c.v0 + (c.i_begin + tid) * VEC;
  uint32_t stage = 0, ii = tid;
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step, ii += U * LG_THREADS) {
    const uint32_t special = c.lists ? c.bits_at(c.table.bits, ii) : 0u;
    const uint32_t loaded = c.allowed_at(ii, step < whole), allowed = loaded & ~special;
    S::wait();
    // (in two versions: rows without seen tokens do not pay for the penalty)
    auto take = [&](auto marked) {
      uint32_t seen = 0;
      if constexpr (marked) seen = c.bits_at(c.seen, ii);
      float z[PER];
      in.template scores<true>(stage, z, allowed);
      if constexpr (marked) penalise(r, seen, z);  // (-inf stays)
      const float vmax = max16(z);
      // scores that may be the largest, once more and exactly (which those are
      // depends on the order of the warps, the largest does not); and ref where
      // the warp's own scores leave its range: the sum has the same bits each time
      const float best = *static_cast<volatile float*>(&s_best);
      const float near = best < INFINITY ? best - fabsf(best) * 0x1p-20f : best;
      if (__any_sync(ALL, (vmax >= near && vmax > -INFINITY) || vmax * k > ref + 24.f)) {
        float wmax = vmax;
#pragma unroll
        for (int o = 16; o; o >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(ALL, wmax, o));
        if (wmax * k > ref + 24.f) raise(wmax * k);
        const float at_least = fmaxf(near, wmax - fabsf(wmax) * 0x1p-20f);
        if (vmax >= at_least) {
          uint32_t m = 0;
#pragma unroll
          for (int q = 0; q < PER; ++q) m |= (z[q] >= at_least && z[q] > -INFINITY ? 1u : 0u) << q;
          unsigned long long top = 0;
          for (; m; m &= m - 1) {
            const uint32_t q = (uint32_t)__ffs((int)m) - 1u;
            const uint32_t t = c.v0 + (c.i_begin + ii + q / VEC * LG_THREADS) * VEC + q % VEC;
            top = max(top, top_key(score(r, t, 0, NO_BIAS, (seen >> q) & 1u, in.score(stage, q / VEC, q % VEC)), t));
          }
          key = max(key, top);
          const float zx = key_score(top);
          if (zx > best) s_best = zx;
        }
      }
      const Two ref2(-ref, -ref);
      Two part[2] = {Two(0.f, 0.f), Two(0.f, 0.f)};
#pragma unroll
      for (int q = 0; q < PER; q += 2) {
        float p0, p1;
        fma2(Two(z[q], z[q + 1]), k2, ref2).get(p0, p1);
        part[q / 2 & 1] = add2(part[q / 2 & 1], Two(ex2(p0), ex2(p1)));
      }
      float p0, p1;
      add2(part[0], part[1]).get(p0, p1);
      sum += p0 + p1;
      if (out) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (step < whole || ii + u * LG_THREADS < n) store_scores(to + u * (LG_THREADS * VEC), z + u * VEC, r.inv_t);
      }
    };
    if (__any_sync(ALL, allowed != 0)) {
      if (c.marked) take(std::true_type());
      else take(std::false_type());
    } else if (out) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (step < whole || ii + u * LG_THREADS < n) store_all(to + u * (LG_THREADS * VEC), -INFINITY);
    }
    if (out) {
      if constexpr (IN_PLACE)  // the logits of listed tokens are still needed
        for (uint32_t m = special & loaded; m; m &= m - 1) {
          const uint32_t q = (uint32_t)__ffs((int)m) - 1u;
          to[q / VEC * (LG_THREADS * VEC) + q % VEC] = Num<T>::put(in.score(stage, q / VEC, q % VEC));
        }
      to += U * LG_THREADS * VEC;
    }
    // this stage's slots are free: the step DEPTH later
    __syncwarp();
    {
      const uint32_t later = step + DEPTH, i_later = ii + DEPTH * U * LG_THREADS;
      if (later < whole) in.issue(stage, c.template wanted<SHIFTED>(i_later, true));
      else if (later < steps) in.issue_end(stage, c.template wanted<SHIFTED>(i_later, false), i_later, n);
      S::commit();
    }
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
  }
  S::close();

  // the listed tokens
  if (c.lists)
    each_listed(r, c.table, s_mem, call.shape.front, a.d_bias_off != nullptr, c.from, c.to - c.from,
                [&](uint32_t t) { return make_float2(Num<T>::get(x[t]), 0.f); },
                [&](uint32_t t, uint32_t times, uint32_t fb, float2 xt) {
                  float z = -INFINITY;
                  if (c.allows(t)) z = score(r, t, times, fb, c.saw(t), xt.x);
                  if (z * k > ref + 24.f) raise(z * k);
                  sum += ex2(fmaf(z, k, -ref));
                  key = max(key, top_key(z, t));
                  if (t == pick) s_z_pick = z;
                  if (out) out[t] = Num<T>::put(z * r.inv_t);
                });

  // the CTA's sum, then the cluster's, and the row's results
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    join_sum(ref, sum, __shfl_xor_sync(ALL, ref, o), __shfl_xor_sync(ALL, sum, o));
    key = max(key, __shfl_xor_sync(ALL, key, o));
  }
  if (lane == 0) {
    s_ref[tid >> 5] = ref;
    s_sum[tid >> 5] = sum;
    atomicMax(&s_key, key);
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
    key = s_part[0].key;
    ref = s_part[0].ref;
    sum = s_part[0].sum;
    float z_pick = s_part[0].z_pick;
    for (uint32_t q = 1; q < n_ranks; ++q) {
      key = max(key, s_part[q].key);
      join_sum(ref, sum, s_part[q].ref, s_part[q].sum);
      z_pick = fmaxf(z_pick, s_part[q].z_pick);
    }
    const bool nan = sum != sum;
    const float z_top = key_score(key), y_top = __fmul_rn(z_top, r.inv_t);
    const float lse = nan ? sum : fabsf(y_top) < Y_MAX ? __fadd_rn(y_top, LN2 * (log2f(sum) - fmaf(z_top, k, -ref))) : y_top;
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
  Shape shape;
  uint32_t ranks;
};

// Gradient: slices as in k_logits, but independent CTAs.  Measured: 2,048 rows of
// 50,257 bf16 scores with masks, seen sets and lists of 2,047 ids in 130 us (3.4
// TB/s read and written), issuing in 53% of all cycles, DRAM at 37%.  exp(y - lse) is
// 2^-24 exp2(z k - lse log2(e) + 24): what is scaled by the gradient and the
// temperature is not lost below 2^-126.  For 32-bit gradients k and lse
// log2(e) are sums of two numbers each (their rounding would weigh |y| times
// on the result) and nothing is added to the exponent.
// DENSE: out has a gradient.
template <class T, bool SHIFTED, bool DENSE>
__global__ void __launch_bounds__(LG_THREADS, LG_CTAS) k_logits_grad(GradCall call) {
  using S = Stream<T, SHIFTED>;
  constexpr int VEC = S::VEC, U = S::U, DEPTH = S::DEPTH;
  constexpr uint32_t FULL = Slice<T>::FULL, ALL = 0xffffffffu;
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ uint32_t s_scan[LG_WARPS];
  const tok_logits_args& a = call.a;
  const Grad& gr = call.g;
  const uint32_t rank = blockIdx.x % call.ranks, b = blockIdx.x / call.ranks, tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  const T* go = DENSE ? static_cast<const T*>(gr.out) + (long long)b * gr.out_stride : x;
  T* gx = static_cast<T*>(gr.logits) + (long long)b * gr.logits_stride;
  Slice<T> c;
  c.open(a, call.shape, vectors<T, SHIFTED>(gx, a.n_logits), rank, call.ranks);
  S in, gin;
  in.open(x, c.v0, c.i_begin, s_mem);
  gin.open(go, c.v0, c.i_begin, s_mem + (DENSE ? S::BYTES : 0));
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    in.issue_end(d, 0xffu, tid + d * U * LG_THREADS, c.n_vec());
    if (DENSE) gin.issue_end(d, 0xffu, tid + d * U * LG_THREADS, c.n_vec());
    S::commit();
  }
  const Row r = load_row(a, b);
  const float glp = gr.logprob ? gr.logprob[b] : 0.f;
  float cp = (gr.lse ? gr.lse[b] : 0.f) - glp, lse = 0.f;
  if (gr.lse || gr.logprob) lse = a.d_lse[b];
  if (fabsf(lse) >= 1e36f) cp = lse = 0.f;  // (nothing but -inf or a type's lowest value)
  // a masked row, or next to no temperature: every score is taken one by one
  const bool far = fabsf(lse) >= Y_FAR && cp != 0.f;
  uint32_t pick = a.d_pick ? (uint32_t)a.d_pick[b] : 0xffffffffu;
  if ((int32_t)pick < 0 && gr.logprob) pick = a.d_top ? (uint32_t)a.d_top[b] : 0xffffffffu;
  const double kd = 1.4426950408889634 / (a.d_temperature ? (double)a.d_temperature[b] : 1.0);
  const double ld = (double)lse * 1.4426950408889634 - (sizeof(T) == 4 ? 0.0 : 24.0);
  const float k = (float)kd, k_lo = (float)(kd - (double)k), lh = (float)ld, l_lo = (float)(ld - (double)lh);
  const float cpt = cp * r.inv_t * (sizeof(T) == 4 ? 1.f : 0x1p-24f);
  // the second part of a 32-bit exponent; where z is -inf or z k overflows, the first part is -inf and this one
  // may be +inf or no number: it is kept finite
  auto second = [](float x) { return fminf(x, FLT_MAX); };
  if (rank == 0 && gr.bias)
    for (int i = tid; i < r.bias_n; i += LG_THREADS)
      if ((uint32_t)r.bias_id[i] >= a.n_logits) gr.bias[(r.bias - a.d_bias) + i] = 0.f;
  c.fill(a, call.shape, r, s_mem, s_scan);

  // the gradient of one score and, returned, the one before the repetition penalty
  auto load = [&](uint32_t t) { return make_float2(Num<T>::get(x[t]), DENSE ? Num<T>::get(go[t]) : 0.f); };
  auto one = [&](uint32_t t, uint32_t times, uint32_t fb, float2 in) {
    float dz = 0.f, f = 1.f;
    if (c.allows(t)) {
      const bool seen = c.saw(t);
      const float xt = in.x;
      if (seen || times) f = xt > 0.f ? r.inv_rep : r.rep;
      dz = in.y * r.inv_t;
      if (cpt != 0.f) {
        const float z = score(r, t, times, fb, seen, xt);
        float e;
        if (far) e = fmaf(fminf(__fsub_rn(__fmul_rn(z, r.inv_t), lse), 0.f), LOG2E, sizeof(T) == 4 ? 0.f : 24.f);
        else e = sizeof(T) == 4 ? fmaf(z, k, -lh) + second(fmaf(z, k_lo, -l_lo)) : fmaf(z, k, -lh);
        dz = fmaf(cpt, sizeof(T) == 4 ? ex2_small(e) : ex2(e), dz);
      }
      if (t == pick) dz = fmaf(glp, r.inv_t, dz);
    }
    gx[t] = Num<T>::put(dz * f);
    return dz;
  };
  // the scores outside the vectors (fewer than 32), or all of them
  for (uint32_t i = tid, some = far ? c.to - c.from : 32u; i < some; i += LG_THREADS) {
    const uint32_t t = far ? c.from + i : c.outside(i);
    if (t != 0xffffffffu && !(c.lists && listed(c.table, t))) one(t, 0, NO_BIAS, load(t));
  }
  const Two k2(k, k), lh2(-lh, -lh), klo2(k_lo, k_lo), llo2(-l_lo, -l_lo), cpt2(cpt, cpt);
  const uint32_t n = far ? 0u : c.n_vec(), steps = (n + U * LG_THREADS - 1) / (U * LG_THREADS), whole = n / (U * LG_THREADS);
  T* to = gx + c.v0 + (c.i_begin + tid) * VEC;
  uint32_t stage = 0, ii = tid;
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step, ii += U * LG_THREADS, to += U * LG_THREADS * VEC) {
    const uint32_t allowed = c.allowed_at(ii, step < whole) & ~(c.lists ? c.bits_at(c.table.bits, ii) : 0u);
    S::wait();
    if (__any_sync(ALL, allowed != 0)) {
      float z[PER], d[PER];
      in.template scores<false>(stage, z, 0);
      if constexpr (DENSE) {
        gin.template scores<false>(stage, d, 0);
#pragma unroll
        for (int q = 0; q < PER; ++q) d[q] *= r.inv_t;
      } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) d[q] = 0.f;
      }
      // (in two versions: rows without seen tokens carry no factors)
      auto slope = [&](auto factors) {
        float f[PER];
        if constexpr (factors) {
          const uint32_t seen = c.bits_at(c.seen, ii);
#pragma unroll
          for (int q = 0; q < PER; ++q) {
            f[q] = (seen >> q) & 1u ? (z[q] > 0.f ? r.inv_rep : r.rep) : 1.f;
          }
#pragma unroll
          for (int q = 0; q < PER; q += 2) mul2(Two(z[q], z[q + 1]), Two(f[q], f[q + 1])).get(z[q], z[q + 1]);
        }
        if (cpt != 0.f) {
#pragma unroll
          for (int q = 0; q < PER; q += 2) {
            const Two z2(z[q], z[q + 1]);
            Two e2 = fma2(z2, k2, lh2);
            float p0, p1;
            if (sizeof(T) == 4) {
              fma2(z2, klo2, llo2).get(p0, p1);
              e2 = add2(e2, Two(second(p0), second(p1)));
            }
            e2.get(p0, p1);
            const Two p2 = sizeof(T) == 4 ? Two(ex2_small(p0), ex2_small(p1)) : Two(ex2(p0), ex2(p1));
            (DENSE ? fma2(cpt2, p2, Two(d[q], d[q + 1])) : mul2(cpt2, p2)).get(d[q], d[q + 1]);
          }
        }
        if constexpr (factors) {
#pragma unroll
          for (int q = 0; q < PER; q += 2) mul2(Two(d[q], d[q + 1]), Two(f[q], f[q + 1])).get(d[q], d[q + 1]);
        }
      };
      if (c.marked) slope(std::true_type());
      else slope(std::false_type());
      uint32_t w[U][4];
#pragma unroll
      for (int q = 0; q < PER; q += 2) Num<T>::put_pair(w[q / VEC], q % VEC / 2, d[q], d[q + 1]);
      if (allowed != FULL) {
#pragma unroll
        for (int u = 0; u < U; ++u) hide<T>(w[u], allowed, u, 0u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (step < whole || ii + u * LG_THREADS < n)
          __stcs(reinterpret_cast<uint4*>(to + u * (LG_THREADS * VEC)), make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]));
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (step < whole || ii + u * LG_THREADS < n) store_all(to + u * (LG_THREADS * VEC), 0.f);
    }
    __syncwarp();
    const uint32_t later = step + DEPTH, i_later = ii + DEPTH * U * LG_THREADS;
    if (later < whole) {
      const uint32_t want = c.template wanted<SHIFTED>(i_later, true);
      in.issue(stage, want);
      if (DENSE) gin.issue(stage, want);
    } else if (later < steps) {
      const uint32_t want = c.template wanted<SHIFTED>(i_later, false);
      in.issue_end(stage, want, i_later, n);
      if (DENSE) gin.issue_end(stage, want, i_later, n);
    }
    S::commit();
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
  }
  S::close();
  __syncthreads();
  if (tid == 0 && pick - c.from < c.to - c.from && !(c.lists && listed(c.table, pick))) one(pick, 0, NO_BIAS, load(pick));

  // the listed tokens, with their biases' gradients
  if (c.lists)
    each_listed(r, c.table, s_mem, call.shape.front, a.d_bias_off != nullptr, c.from, c.to - c.from,
                load, [&](uint32_t t, uint32_t times, uint32_t fb, float2 in) {
                  const float dz = one(t, times, fb, in);
                  if (!gr.bias || (fb & NO_BIAS) == NO_BIAS) return;
                  float* gb = gr.bias + (r.bias - a.d_bias);
                  gb[fb & NO_BIAS] = dz;
                  if (fb >> 31)
                    for (int e = (int)(fb & NO_BIAS) + 1; e < r.bias_n; ++e)
                      if ((uint32_t)r.bias_id[e] == t) gb[e] = dz;
                });
}

// One cluster per row: each CTA sets the bits of its share of the ids in its
// own shared memory; then each joins all CTAs' bits for its share of the row.
// Setting bits that are set already is left out, so that shared memory sees
// mostly reads.  Measured: 64 prompts of up to 180,001 ids 10.3 us (0.45 TB/s:
// a call's latencies, the launch of 7 us among them).
__global__ void __launch_bounds__(SB_THREADS) k_seen_bits(const int32_t* ids, const long long* off, uint32_t n_logits,
                                                          uint32_t* seen, long long stride, int keep) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t s_bits[];
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks(), b = blockIdx.x / n_ranks;
  const uint32_t words = (n_logits + 31) / 32;
  const long long begin = off[b], n = off[b + 1] - begin, each = n > 0 ? (n + n_ranks - 1) / n_ranks : 0;
  const long long i0 = min(each * rank, max(n, 0ll)), i1 = min(i0 + each, max(n, 0ll));
  for (uint32_t w = threadIdx.x; w < words; w += SB_THREADS) s_bits[w] = 0;
  __syncthreads();
  constexpr int AHEAD = 8;  // loads of a thread in flight
  for (long long i = i0 + threadIdx.x; i < i1; i += AHEAD * SB_THREADS) {
    uint32_t v[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      v[j] = i + j * SB_THREADS < i1 ? (uint32_t)__ldcs(ids + begin + i + j * SB_THREADS) : 0xffffffffu;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      // (text repeats its words: most bits are set already, and reading one is cheaper than setting it again)
      const uint32_t bit = 1u << (v[j] & 31);
      if (v[j] < n_logits && !(*static_cast<volatile uint32_t*>(s_bits + (v[j] >> 5)) & bit)) atomicOr(&s_bits[v[j] >> 5], bit);
    }
  }
  __syncthreads();
  if (n_ranks > 1) {
    cluster_arrive();
    cluster_wait();
  }
  uint32_t* row = seen + (long long)b * stride;
  const uint32_t share = (words + n_ranks - 1) / n_ranks, w1 = min((rank + 1) * share, words);
  for (uint32_t w = rank * share + threadIdx.x; w < w1; w += SB_THREADS) {
    uint32_t m = keep ? row[w] : 0u;
    if (n_ranks == 1) m |= s_bits[w];
    else
      for (uint32_t q = 0; q < n_ranks; ++q) m |= cluster.map_shared_rank(s_bits, q)[w];
    row[w] = m;
  }
  if (n_ranks > 1) {  // until the others have read this CTA's bits
    cluster_arrive_only();
    cluster_wait();
  }
}

size_t stage_bytes(int dtype, bool shifted) {
  if (dtype == TOK_F32) return shifted ? Stream<float, true>::BYTES : Stream<float, false>::BYTES;
  return shifted ? Stream<__half, true>::BYTES : Stream<__half, false>::BYTES;
}

size_t size_of(int dtype) { return dtype == TOK_F32 ? 4 : 2; }

// A row in n slices; arrays: of scores that are read.
Shape shape(const tok_logits_args& a, bool shifted, int arrays, uint32_t n, size_t* smem) {
  const uint32_t vec = 16 / (uint32_t)size_of(a.dtype);
  Shape s{};
  s.lists = a.d_gen || a.d_bias_off;
  s.per = (a.n_logits / vec + n - 1) / n;
  s.words = bit_words(s.per * vec);
  s.front = (uint32_t)stage_bytes(a.dtype, shifted) * arrays;
  *smem = s.front + BITS_ROOM + sizeof(uint32_t) * ((size_t)s.words * ((a.d_mask ? 1 : 0) + (a.d_seen ? 1 : 0) + (s.lists ? 1 : 0)) +
                                        (s.lists ? fours_of(s.words) : 0));
  return s;
}

// The slices of a row, at most the 16 CTAs of a cluster: as few rounds of CTAs
// as possible, weighing a CTA's start and end (about 8 us) like 64 KB of its
// scores.  A slice keeps 2,048 scores or more.  Rows of 100,257 bf16 scores, us
// with 1, 2, 4, 8 and 16 slices, the rule's choice in brackets:
//   1 row     25.0  18.8  15.2  12.6 [10.8]    152 rows  31.3 [29.2] 39.7  48.4  81.7
//   16 rows   28.5  20.8  16.7  14.6 [14.8]    304 rows [45.4] 53.9  64.9  89.4 155.7
//   64 rows   29.1  21.0 [20.9] 26.0  37.1     512 rows  73.5 [74.4] 98.1 141.9 253.2
uint32_t slices(const tok_handle* h, const tok_logits_args& a, bool shifted, int arrays) {
  uint32_t best = 0;
  double least = 0;
  for (uint32_t n = 1; n <= 16; n *= 2) {  // (clusters of other sizes leave slots of an SM group empty)
    if (best && a.n_logits / n < 2048) break;
    size_t smem;
    shape(a, shifted, arrays, n, &smem);
    if (smem > MOST_SHARED) continue;
    const unsigned fit = (unsigned)std::min<size_t>(LG_CTAS, (228 * 1024) / (smem + 2048));
    const unsigned long long room = (unsigned long long)fit * (unsigned)h->n_sms;
    const unsigned long long rounds = ((unsigned long long)a.rows * n + room - 1) / room;
    const double cost = (double)rounds * (fit * (double)a.n_logits * (double)size_of(a.dtype) / n + LG_CTAS * 65536.0);
    if (!best || cost < least) {
      best = n;
      least = cost;
    }
  }
  return best ? best : 16;
}

// whether rows of an array lie like those of another towards 16-byte boundaries
bool alike(const void* p, int64_t stride, const void* q, int64_t q_stride, uint32_t rows, size_t size) {
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) != 0) return false;
  return rows == 1 || ((uint64_t)(stride - q_stride) * size & 15u) == 0;
}

template <class T>
cudaError_t launch_forward(int dev, const LogitsCall& c, bool shifted, bool in_place, unsigned ctas, unsigned cluster, size_t smem,
                           cudaStream_t s) {
  if (in_place) return launch_clusters<k_logits<T, false, true>>(dev, ctas, LG_THREADS, cluster, smem, s, c);
  return shifted ? launch_clusters<k_logits<T, true, false>>(dev, ctas, LG_THREADS, cluster, smem, s, c)
                 : launch_clusters<k_logits<T, false, false>>(dev, ctas, LG_THREADS, cluster, smem, s, c);
}
template <class T>
cudaError_t launch_grad(int dev, const GradCall& c, bool shifted, unsigned ctas, size_t smem, cudaStream_t s) {
  if (c.g.out)
    return shifted ? launch_clusters<k_logits_grad<T, true, true>>(dev, ctas, LG_THREADS, 1, smem, s, c)
                   : launch_clusters<k_logits_grad<T, false, true>>(dev, ctas, LG_THREADS, 1, smem, s, c);
  return shifted ? launch_clusters<k_logits_grad<T, true, false>>(dev, ctas, LG_THREADS, 1, smem, s, c)
                 : launch_clusters<k_logits_grad<T, false, false>>(dev, ctas, LG_THREADS, 1, smem, s, c);
}

int launched(tok_handle* h, cudaError_t e) {
  h->launches += 1;
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
}

// (addresses come without a type: one that no score can have would fault on the device)
bool lies_at_scores(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % size_of(dtype) == 0; }

// nullptr, or what is wrong with the arguments
const char* check_logits(const tok_logits_args* a) {
  if (!a || !a->d_logits) return "logits: the arguments or the logits are NULL";
  if (a->dtype != TOK_F32 && a->dtype != TOK_F16 && a->dtype != TOK_BF16) return "logits: unknown type";
  if (a->n_logits == 0 || a->n_logits > MAX_LOGITS) return "logits: n_logits is out of range";
  if (a->rows > 0x7ffffffu) return "logits: too many rows";
  if (!lies_at_scores(a->d_logits, a->dtype) || !lies_at_scores(a->d_out, a->dtype))
    return "logits: an array does not lie at a multiple of its type's size";
  const int64_t n = a->n_logits, words = (n + 31) / 32;
  if (a->logits_stride < n || (a->d_out && a->out_stride < n)) return "logits: a row stride is below n_logits";
  if ((a->d_seen && a->seen_stride < words) || (a->d_mask && a->mask_stride < words))
    return "logits: a stride of bits is below a row's words";
  if ((a->d_gen && (!a->d_gen_start || !a->d_gen_len)) || (a->d_bias_off && (!a->d_bias_id || !a->d_bias)))
    return "logits: generated ids need their starts and lengths, bias offsets their ids and values";
  if (a->d_mask_row && !a->d_mask) return "logits: mask rows without masks";
  if (a->d_out == a->d_logits && a->out_stride != a->logits_stride && a->rows > 1)
    return "logits: out is the logits with another stride";
  return nullptr;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_logits_process(tok_handle* h, const tok_logits_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->rows == 0) return TOK_OK;  // (an empty batch's buffers are often NULL)
  if (const char* w = check_logits(a)) return fail(h, TOK_EINVAL, w);
  DeviceGuard g(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LogitsCall c{};
  c.a = *a;
  const size_t size = size_of(a->dtype);
  const bool shifted = a->d_out && !alike(a->d_logits, a->logits_stride, a->d_out, a->out_stride, a->rows, size);
  const uint32_t n = slices(h, *a, shifted, 1);
  size_t smem;
  c.shape = shape(*a, shifted, 1, n, &smem);
  const bool in_place = a->d_out == a->d_logits;
  const unsigned ctas = a->rows * n;
  const cudaError_t e = a->dtype == TOK_F32   ? launch_forward<float>(h->dev, c, shifted, in_place, ctas, n, smem, s)
                        : a->dtype == TOK_F16 ? launch_forward<__half>(h->dev, c, shifted, in_place, ctas, n, smem, s)
                                              : launch_forward<__nv_bfloat16>(h->dev, c, shifted, in_place, ctas, n, smem, s);
  return launched(h, e);
} catch (...) {
  return TOK_ENOMEM;
}

int tok_logits_backward(tok_handle* h, const tok_logits_args* a, const tok_logits_grad_args* ga, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->rows == 0) return TOK_OK;
  if (const char* w = check_logits(a)) return fail(h, TOK_EINVAL, w);
  if (!ga || !ga->d_grad_logits) return fail(h, TOK_EINVAL, "logits: the gradient's arguments or buffer are NULL");
  if (!lies_at_scores(ga->d_grad_logits, a->dtype) || !lies_at_scores(ga->d_grad_out, a->dtype))
    return fail(h, TOK_EINVAL, "logits: an array does not lie at a multiple of its type's size");
  if (ga->grad_logits_stride < (int64_t)a->n_logits || (ga->d_grad_out && ga->grad_out_stride < (int64_t)a->n_logits))
    return fail(h, TOK_EINVAL, "logits: a row stride is below n_logits");
  if ((ga->d_grad_lse || ga->d_grad_logprob) && !a->d_lse)
    return fail(h, TOK_EINVAL, "logits: the gradient of lse or logprob needs the forward pass's lse");
  if (ga->d_grad_logprob && !a->d_top && !a->d_pick)
    return fail(h, TOK_EINVAL, "logits: the gradient of logprob needs the picks or the forward pass's top");
  DeviceGuard gd(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GradCall c{};
  c.a = *a;
  c.g = Grad{ga->d_grad_out, ga->grad_out_stride, ga->d_grad_lse,  ga->d_grad_logprob,
               ga->d_grad_logits, ga->grad_logits_stride, a->d_bias_off ? ga->d_grad_bias : nullptr};
  const size_t size = size_of(a->dtype);
  const bool shifted = !alike(a->d_logits, a->logits_stride, ga->d_grad_logits, ga->grad_logits_stride, a->rows, size) ||
                       (ga->d_grad_out && !alike(ga->d_grad_out, ga->grad_out_stride, ga->d_grad_logits,
                                                 ga->grad_logits_stride, a->rows, size));
  const int arrays = ga->d_grad_out ? 2 : 1;
  c.ranks = slices(h, *a, shifted, arrays);
  size_t smem;
  c.shape = shape(*a, shifted, arrays, c.ranks, &smem);
  const unsigned ctas = a->rows * c.ranks;
  const cudaError_t e = a->dtype == TOK_F32   ? launch_grad<float>(h->dev, c, shifted, ctas, smem, s)
                        : a->dtype == TOK_F16 ? launch_grad<__half>(h->dev, c, shifted, ctas, smem, s)
                                              : launch_grad<__nv_bfloat16>(h->dev, c, shifted, ctas, smem, s);
  return launched(h, e);
} catch (...) {
  return TOK_ENOMEM;
}

int tok_seen_bits(tok_handle* h, const int32_t* d_ids, const int64_t* d_item_off, uint32_t n, uint32_t n_logits,
                  uint32_t* d_seen, int64_t seen_stride, int keep, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (!d_ids || !d_item_off || !d_seen || n == 0) return fail(h, TOK_EINVAL, "seen bits: a buffer is NULL, or n is 0");
  const uint32_t words = (n_logits + 31) / 32;
  if (n > 0x7ffffffu || n_logits == 0 || n_logits > MAX_LOGITS || seen_stride < (int64_t)words)
    return fail(h, TOK_EINVAL, "seen bits: n, n_logits or seen_stride is out of range");
  DeviceGuard g(h->dev);
  // few rows: more CTAs for each, up to a cluster of 16 (prompts of up to 180,001
  // ids, us with 1, 4 and 16: 8 rows 21, 10, 8; 64 rows 35, 15, 11; 600 rows alike)
  uint32_t ranks = 16;
  while (ranks > 1 && (unsigned long long)n * ranks > 4ull * (unsigned)h->n_sms) ranks /= 2;
  return launched(h, launch_clusters<k_seen_bits>(h->dev, n * ranks, SB_THREADS, ranks, words * sizeof(uint32_t),
                                                  static_cast<cudaStream_t>(stream), d_ids,
                                                  reinterpret_cast<const long long*>(d_item_off), n_logits, d_seen,
                                                  (long long)seen_stride, keep));
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
