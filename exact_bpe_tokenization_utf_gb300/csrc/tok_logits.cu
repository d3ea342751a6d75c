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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "tok_handle.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr int LG_THREADS = 256;
constexpr int LG_TILE = 4096;  // tokens whose counts are in shared memory at a time
constexpr float LOG2E = 1.4426950408889634f;

template <class T> struct Num;
template <> struct Num<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Num<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <> struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
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
  float rep, freq, pres, inv_t;
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
  r.freq = a.d_frequency ? a.d_frequency[b] : 0.f;
  r.pres = a.d_presence ? a.d_presence[b] : 0.f;
  r.inv_t = a.d_temperature ? __fdiv_rn(1.f, a.d_temperature[b]) : 1.f;
  return r;
}

// Counts of the generated ids and places of the bias entries, for the tokens
// of one tile: first[v] holds the smallest index of v's bias entries (its top
// bit: more than one), or NO_BIAS.
constexpr uint32_t NO_BIAS = 0x7fffffffu;
struct Tile {
  uint32_t* count;
  uint32_t* first;
  uint32_t lo, n;
};

__device__ __forceinline__ void fill_tile(const Row& r, const Tile& t) {
  for (uint32_t i = threadIdx.x; i < t.n; i += blockDim.x) {
    t.count[i] = 0;
    t.first[i] = NO_BIAS;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < r.gen_len; i += blockDim.x) {
    const uint32_t v = (uint32_t)r.gen[i] - t.lo;
    if (v < t.n) atomicAdd(&t.count[v], 1u);
  }
  for (int i = threadIdx.x; i < r.bias_n; i += blockDim.x) {
    const uint32_t v = (uint32_t)r.bias_id[i] - t.lo;
    if (v < t.n) atomicMin(&t.first[v], (uint32_t)i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < r.bias_n; i += blockDim.x) {
    const uint32_t v = (uint32_t)r.bias_id[i] - t.lo;
    if (v < t.n && (t.first[v] & NO_BIAS) != (uint32_t)i) atomicOr(&t.first[v], 0x80000000u);
  }
  __syncthreads();
}

__device__ __forceinline__ bool bit_of(const uint32_t* words, uint32_t v) { return (words[v >> 5] >> (v & 31)) & 1u; }

__device__ __forceinline__ bool allowed(const Row& r, uint32_t v) { return !r.none && (!r.mask || bit_of(r.mask, v)); }

// the score of token v before the temperature, from its logit; *factor: of the repetition penalty
__device__ __forceinline__ float score(const Row& r, const Tile& t, uint32_t v, float x, float* factor) {
  const uint32_t c = t.count[v - t.lo], fb = t.first[v - t.lo];
  *factor = 1.f;
  if (c || (r.seen && bit_of(r.seen, v))) {
    *factor = x > 0.f ? __fdiv_rn(1.f, r.rep) : r.rep;
    x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  }
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

// What is known of a part of a row: its largest score before the temperature
// and that score's token (the lowest of equals), the maximum m of y, kept
// within the finite numbers, and the sum of exp(y - m).
struct Stats {
  float best;
  int top;
  float m, s;
};

__device__ __forceinline__ Stats no_stats() { return Stats{-INFINITY, -1, -FLT_MAX, 0.f}; }

__device__ __forceinline__ void add(Stats& s, float z, float y, int v) {
  if (z > s.best) {
    s.best = z;
    s.top = v;
    const float m = fmaxf(s.m, fminf(y, FLT_MAX));
    s.s *= ex2((s.m - m) * LOG2E);
    s.m = m;
  }
  s.s += ex2((y - s.m) * LOG2E);
}

__device__ __forceinline__ Stats join(const Stats& a, const Stats& b) {
  Stats r;
  const bool left = a.best > b.best || (a.best == b.best && (uint32_t)a.top < (uint32_t)b.top);
  r.best = left ? a.best : b.best;
  r.top = left ? a.top : b.top;
  r.m = fmaxf(a.m, b.m);
  r.s = a.s * ex2((a.m - r.m) * LOG2E) + b.s * ex2((b.m - r.m) * LOG2E);
  return r;
}

__device__ __forceinline__ Stats join_block(Stats s, Stats* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Stats x{__shfl_xor_sync(0xffffffffu, s.best, o), __shfl_xor_sync(0xffffffffu, s.top, o),
                  __shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.s, o)};
    s = join(s, x);
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  s = sh[0];
  for (uint32_t k = 1; k < blockDim.x / 32; ++k) s = join(s, sh[k]);
  return s;
}

__device__ __forceinline__ void write_stats(const tok_logits_args& a, const Row& r, uint32_t b, const Stats& s,
                                            float z_pick, int pick) {
  const float lse = s.m + logf(s.s);
  const bool nan = s.s != s.s;
  if (a.d_top) a.d_top[b] = nan ? -1 : s.top;
  if (a.d_lse) a.d_lse[b] = lse;
  if (a.d_logprob) {
    const float y = (pick >= 0 ? z_pick : s.best) * r.inv_t;
    a.d_logprob[b] = nan ? lse : y == -INFINITY ? -INFINITY : y - lse;
  }
}

template <class T>
__global__ void __launch_bounds__(LG_THREADS) k_logits(tok_logits_args a) {
  __shared__ uint32_t s_count[LG_TILE], s_first[LG_TILE];
  __shared__ Stats s_st[LG_THREADS / 32];
  __shared__ float s_pick;
  const uint32_t b = blockIdx.x;
  const Row r = load_row(a, b);
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  T* out = a.d_out ? static_cast<T*>(a.d_out) + (long long)b * a.out_stride : nullptr;
  const int pick = a.d_pick ? a.d_pick[b] : -1;
  Stats st = no_stats();
  if (threadIdx.x == 0) s_pick = -INFINITY;
  Tile t{s_count, s_first, 0, 0};
  for (t.lo = 0; t.lo < a.n_logits; t.lo += LG_TILE) {
    t.n = min((uint32_t)LG_TILE, a.n_logits - t.lo);
    __syncthreads();
    fill_tile(r, t);
    for (uint32_t v = t.lo + threadIdx.x; v < t.lo + t.n; v += LG_THREADS) {
      float z = -INFINITY, f;
      if (allowed(r, v)) z = score(r, t, v, Num<T>::get(x[v]), &f);
      const float y = z * r.inv_t;
      add(st, z, y, (int)v);
      if (out) out[v] = Num<T>::put(y);
      if ((int)v == pick) s_pick = z;
    }
  }
  __syncthreads();
  st = join_block(st, s_st);
  if (threadIdx.x == 0) write_stats(a, r, b, st, s_pick, pick);
}

template <class T>
__global__ void __launch_bounds__(LG_THREADS) k_logits_grad(tok_logits_args a, Grad g) {
  __shared__ uint32_t s_count[LG_TILE], s_first[LG_TILE];
  const uint32_t b = blockIdx.x;
  const Row r = load_row(a, b);
  const T* x = static_cast<const T*>(a.d_logits) + (long long)b * a.logits_stride;
  const T* go = g.out ? static_cast<const T*>(g.out) + (long long)b * g.out_stride : nullptr;
  T* gx = static_cast<T*>(g.logits) + (long long)b * g.logits_stride;
  const float glp = g.logprob ? g.logprob[b] : 0.f;
  float cp = (g.lse ? g.lse[b] : 0.f) - glp, lse = 0.f;
  if (g.lse || g.logprob) lse = a.d_lse[b];
  if (lse == -INFINITY) cp = 0.f;
  int pick = a.d_pick ? a.d_pick[b] : -1;
  if (pick < 0 && g.logprob) pick = a.d_top[b];
  Tile t{s_count, s_first, 0, 0};
  for (t.lo = 0; t.lo < a.n_logits; t.lo += LG_TILE) {
    t.n = min((uint32_t)LG_TILE, a.n_logits - t.lo);
    __syncthreads();
    fill_tile(r, t);
    auto dz = [&](uint32_t v, float* f) {
      if (!allowed(r, v)) return *f = 0.f;
      const float y = score(r, t, v, Num<T>::get(x[v]), f) * r.inv_t;
      float d = go ? Num<T>::get(go[v]) : 0.f;
      if (cp != 0.f) d += cp * ex2_small((y - lse) * LOG2E);
      if ((int)v == pick) d += glp;
      return d * r.inv_t;
    };
    if (g.bias)
      for (int i = threadIdx.x; i < r.bias_n; i += LG_THREADS) {
        const uint32_t v = (uint32_t)r.bias_id[i];
        float f;
        if (v - t.lo < t.n) g.bias[(r.bias - a.d_bias) + i] = dz(v, &f);
        else if (v >= a.n_logits && t.lo == 0) g.bias[(r.bias - a.d_bias) + i] = 0.f;
      }
    for (uint32_t v = t.lo + threadIdx.x; v < t.lo + t.n; v += LG_THREADS) {
      float f;
      const float d = dz(v, &f);
      gx[v] = Num<T>::put(d * f);
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

int launched(tok_handle* h) {
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
}

// nullptr, or what is wrong with the arguments
const char* check_logits(const tok_logits_args* a) {
  if (!a || !a->d_logits) return "logits: the arguments or the logits are NULL";
  if (a->dtype != TOK_F32 && a->dtype != TOK_F16 && a->dtype != TOK_BF16) return "logits: unknown type";
  if (a->n_logits == 0 || a->n_logits > MAX_LOGITS) return "logits: n_logits is out of range";
  if (a->rows > 0x7fffffffu) return "logits: too many rows";
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
  if (a->dtype == TOK_F32) k_logits<float><<<a->rows, LG_THREADS, 0, s>>>(*a);
  else if (a->dtype == TOK_F16) k_logits<__half><<<a->rows, LG_THREADS, 0, s>>>(*a);
  else k_logits<__nv_bfloat16><<<a->rows, LG_THREADS, 0, s>>>(*a);
  return launched(h);
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
  const Grad g{ga->d_grad_out, ga->grad_out_stride, ga->d_grad_lse,  ga->d_grad_logprob,
               ga->d_grad_logits, ga->grad_logits_stride, a->d_bias_off ? ga->d_grad_bias : nullptr};
  if (a->dtype == TOK_F32) k_logits_grad<float><<<a->rows, LG_THREADS, 0, s>>>(*a, g);
  else if (a->dtype == TOK_F16) k_logits_grad<__half><<<a->rows, LG_THREADS, 0, s>>>(*a, g);
  else k_logits_grad<__nv_bfloat16><<<a->rows, LG_THREADS, 0, s>>>(*a, g);
  return launched(h);
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
  return launched(h);
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
