// Token masks of a byte automaton (tok_grammar_load, tok_grammar_mask).
//
// A token may follow in state s iff the automaton, read byte by byte from s,
// never meets a byte that is not allowed: walk(s, bytes) = next(... next(next(s,
// b0), b1) ...) stays defined.  mask[k][t] = walk(state_k, bytes of t) is
// defined; the end token's bit is whether state_k accepts.
#include <new>

#include "tok_handle.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr uint32_t DEAD = 0xffffu;
constexpr int GR_THREADS = 256;

struct DevGrammar {
  const uint16_t* next;   // n_states rows of 256
  const uint8_t* accept;
  uint32_t n_states;
};

struct MaskCall {
  const int32_t* state;
  const int32_t* ids;
  const long long* item_off;
  uint32_t n;
  int32_t eos;
  int32_t* state_out;
  uint32_t n_logits;
  uint32_t* mask;
  long long mask_stride;
};

__device__ __forceinline__ uint32_t walk(const DevGrammar& g, const DevTokens& v, uint32_t s, uint32_t t) {
  const uint32_t end = v.off[t + 1];
  for (uint32_t i = v.off[t]; i < end && s != DEAD; ++i) s = __ldg(g.next + s * 256u + __ldg(v.bytes + i));
  return s;
}

// the state of row k after its tokens
__device__ __forceinline__ uint32_t row_state(const DevGrammar& g, const DevTokens& v, const MaskCall& c, uint32_t k) {
  const int32_t s0 = c.state[k];
  uint32_t s = s0 >= 0 && (uint32_t)s0 < g.n_states ? (uint32_t)s0 : DEAD;
  if (!c.ids) return s;
  long long i = c.item_off ? c.item_off[k] : k;
  const long long end = c.item_off ? c.item_off[k + 1] : i + 1;
  for (; i < end && s != DEAD; ++i) {
    const int32_t t = c.ids[i];
    if (t < 0) continue;
    if ((uint32_t)t >= v.n || t == c.eos) s = DEAD;
    else s = walk(g, v, s, (uint32_t)t);
  }
  return s;
}

// One CTA per row, a thread per token.
__global__ void __launch_bounds__(GR_THREADS) k_grammar_mask(DevGrammar g, DevTokens v, MaskCall c) {
  __shared__ uint32_t s_state;
  const uint32_t k = blockIdx.x;
  if (threadIdx.x == 0) {
    const uint32_t s = row_state(g, v, c, k);
    s_state = s;
    if (c.state_out) c.state_out[k] = s == DEAD ? -1 : (int32_t)s;
  }
  __syncthreads();
  if (!c.mask) return;
  const uint32_t s = s_state;
  const uint32_t words = (c.n_logits + 31) / 32;
  uint32_t* row = c.mask + (long long)k * c.mask_stride;
  for (uint32_t w = threadIdx.x / 32; w < words; w += GR_THREADS / 32) {
    const uint32_t t = w * 32 + (threadIdx.x & 31);
    bool ok = false;
    if (s != DEAD && t < c.n_logits) {
      if ((int32_t)t == c.eos) ok = g.accept[s] != 0;
      else if (t < v.n) ok = walk(g, v, s, t) != DEAD;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, ok);
    if ((threadIdx.x & 31) == 0) row[w] = bits;
  }
}

// the vocabulary's bytes on the device, once per handle
int ensure_tokens(tok_handle* h) {
  if (h->d_tokens) return TOK_OK;
  const size_t n = h->vocab_off.size() - 1, nb = h->vocab_bytes.size();
  if (nb > 0xffffffffull) return fail(h, TOK_EINVAL, "grammar: a vocabulary of 4 GiB or more");
  std::vector<uint32_t> off(n + 1);
  for (size_t t = 0; t <= n; ++t) off[t] = (uint32_t)h->vocab_off[t];
  uint8_t* p = nullptr;
  const size_t ob = off.size() * sizeof(uint32_t);
  cudaError_t e = halloc(h, &p, ob + nb);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(h, TOK_ENOMEM, "grammar: allocation failed");
  }
  e = cudaMemcpy(p, off.data(), ob, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(p + ob, h->vocab_bytes.data(), nb, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaFree(p);
    return cuda_fail(h, e, "grammar: vocabulary copy");
  }
  h->d_tokens = p;
  h->tokens = DevTokens{p + ob, reinterpret_cast<const uint32_t*>(p), (uint32_t)n};
  return TOK_OK;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

struct tok_grammar {
  tok_handle* h = nullptr;
  DevGrammar g{};
  uint8_t* d_mem = nullptr;
};

extern "C" {

int tok_grammar_load(tok_handle* h, const int32_t* next, const uint8_t* accept, uint32_t n_states,
                     tok_grammar** out) try {
  if (!h) return TOK_EINVAL;
  if (!out) return fail(h, TOK_EINVAL, "grammar: out is NULL");
  *out = nullptr;
  if (!next || !accept) return fail(h, TOK_EINVAL, "grammar: next or accept is NULL");
  if (n_states == 0 || n_states > DEAD) return fail(h, TOK_EINVAL, "grammar: n_states is out of range");
  std::vector<uint16_t> t((size_t)n_states * 256);
  for (size_t i = 0; i < t.size(); ++i) {
    if (next[i] < -1 || next[i] >= (int32_t)n_states) return fail(h, TOK_EINVAL, "grammar: a next state is out of range");
    t[i] = next[i] < 0 ? (uint16_t)DEAD : (uint16_t)next[i];
  }
  DeviceGuard dg(h->dev);
  int rc = ensure_tokens(h);
  if (rc) return rc;
  tok_grammar* g = new tok_grammar();
  const size_t tb = t.size() * sizeof(uint16_t);
  cudaError_t e = halloc(h, &g->d_mem, tb + n_states);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete g;
    return fail(h, TOK_ENOMEM, "grammar: allocation failed");
  }
  e = cudaMemcpy(g->d_mem, t.data(), tb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(g->d_mem + tb, accept, n_states, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaFree(g->d_mem);
    delete g;
    return cuda_fail(h, e, "grammar: copy");
  }
  g->h = h;
  g->g = DevGrammar{reinterpret_cast<const uint16_t*>(g->d_mem), g->d_mem + tb, n_states};
  *out = g;
  return TOK_OK;
} catch (...) {
  return fail(h, TOK_ENOMEM, "grammar: out of host memory");
}

void tok_grammar_free(tok_grammar* g) {
  if (!g) return;
  DeviceGuard dg(g->h->dev);
  cudaFree(g->d_mem);
  delete g;
}

int tok_grammar_mask(tok_handle* h, const tok_grammar* g, const int32_t* d_state, const int32_t* d_ids,
                     const int64_t* d_item_off, uint32_t n, int32_t eos, int32_t* d_state_out, uint32_t n_logits,
                     uint32_t* d_mask, int64_t mask_stride, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (!g || g->h != h) return fail(h, TOK_EINVAL, "grammar mask: the grammar is NULL or belongs to another handle");
  if (n == 0) return TOK_OK;
  if (!d_state || (!d_mask && !d_state_out)) return fail(h, TOK_EINVAL, "grammar mask: a buffer is NULL");
  if (d_state_out == d_state) return fail(h, TOK_EINVAL, "grammar mask: state_out is state");
  if (n > 0x7fffffffu || (d_item_off && !d_ids) ||
      (d_mask && (n_logits == 0 || n_logits > MAX_LOGITS || mask_stride < (int64_t)((n_logits + 31) / 32))))
    return fail(h, TOK_EINVAL, "grammar mask: n, n_logits or mask_stride is out of range, or offsets without ids");
  DeviceGuard dg(h->dev);
  const MaskCall c{d_state, d_ids, reinterpret_cast<const long long*>(d_item_off), n, eos, d_state_out, n_logits,
                   d_mask, mask_stride};
  k_grammar_mask<<<n, GR_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(g->g, h->tokens, c);
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
