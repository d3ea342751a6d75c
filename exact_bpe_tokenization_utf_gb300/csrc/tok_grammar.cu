// Token masks of a byte automaton (tok_grammar_load, tok_grammar_mask).
//
// A token may follow in state s iff the automaton, read byte by byte from s,
// never meets a byte that is not allowed: walk(s, bytes) = next(... next(next(s,
// b0), b1) ...) stays defined.  mask[k][t] = walk(state_k, bytes of t) is
// defined; the end token's bit is whether state_k accepts.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "tok_handle.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr uint32_t DEAD = 0xffffu;
constexpr uint32_t NO_TOKEN = 0xffffffffu;
constexpr int GR_THREADS = 512;

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

// The rows' states alone.
__global__ void __launch_bounds__(128) k_grammar_states(DevGrammar g, DevTokens v, MaskCall c) {
  const uint32_t k = blockIdx.x * 128 + threadIdx.x;
  if (k >= c.n) return;
  const uint32_t s = row_state(g, v, c, k);
  c.state_out[k] = s == DEAD ? -1 : (int32_t)s;
}

// One cluster per row.  A thread walks a group's common first bytes, so that
// one step decides over up to 32 tokens; where the state survives, a warp walks
// the group's tokens, one per lane (sorted tokens read neighbouring bytes from
// equal states).  Allowed tokens set their bits in the CTA's shared memory;
// the cluster's CTAs then join their bits, a share of the row each, and write it.
// Rows (of GR_THREADS at a time) in equal states are walked once, by the
// first one's cluster, which writes all of them.
__global__ void __launch_bounds__(GR_THREADS) k_grammar_mask(DevGrammar g, DevTokens v, MaskCall c) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t s_mem[];
  __shared__ uint32_t s_live, s_row[GR_THREADS / 32], s_state;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks(), k = blockIdx.x / n_ranks;
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t n_words = (c.n_logits + 31) / 32;
  uint32_t* bits = s_mem;                               // a row's
  uint32_t* live = s_mem + ((n_words + 3) / 4) * 4;     // group | state << 16
  const uint32_t per = (v.n_groups + n_ranks - 1) / n_ranks;
  // this thread's group, on its way while the states are walked
  const uint32_t g0 = min(rank * per, v.n_groups), g1 = min(g0 + per, v.n_groups);

  // the states of this row's window, and the rows among them that equal it
  const uint32_t w0 = k / GR_THREADS * GR_THREADS, j = w0 + tid;
  uint32_t sj = DEAD;
  if (j < c.n) sj = row_state(g, v, c, j);
  if (j == k) {
    s_state = sj;
    s_live = 0;
    if (rank == 0 && c.state_out) c.state_out[k] = sj == DEAD ? -1 : (int32_t)sj;
  }
  for (uint32_t w = tid; w < n_words; w += GR_THREADS) bits[w] = 0;
  __syncthreads();
  const uint32_t s0 = s_state;
  const bool same = j < c.n && sj == s0;
  const uint32_t mine = __ballot_sync(0xffffffffu, same);
  if (lane == 0) s_row[warp] = mine;
  if (__syncthreads_or(same && j < k)) return;  // (in every CTA of the cluster alike)

  if (s0 != DEAD) {
    for (uint32_t q = g0 + tid; q < g1; q += GR_THREADS) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(v.group + q));
      unsigned long long head = (unsigned long long)r.y << 32 | r.x;
      uint32_t s = s0;
      for (uint32_t i = r.z & 15u; i && s != DEAD; --i) {
        s = __ldg(g.next + s * 256u + (uint32_t)(head & 255u));
        head >>= 8;
      }
      if (s != DEAD) live[atomicAdd(&s_live, 1u)] = q | s << 16;
    }
    __syncthreads();
    const uint32_t n_live = s_live;
    // two groups at a time: their walks do not depend on one another
    for (uint32_t e = warp; e < n_live; e += 2 * (GR_THREADS / 32)) {
      uint32_t s[2], id[2], rest[2], at[2], words = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t f = e + h * (GR_THREADS / 32);
        const bool any = f < n_live;
        const uint32_t x = live[any ? f : e], q = x & 0xffffu;
        const TokenGroup* r = v.group + q;
        s[h] = x >> 16;
        id[h] = any ? __ldg(v.id + q * 32 + lane) : NO_TOKEN;
        rest[h] = id[h] == NO_TOKEN ? 0u : __ldg(v.rest + q * 32 + lane);
        at[h] = __ldg(&r->at) + lane;
        words = max(words, any ? __ldg(&r->shape) >> 4 : 0u);
      }
      for (uint32_t w = 0; w < words; ++w) {
        uint32_t b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) b[h] = rest[h] > 4 * w && s[h] != DEAD ? __ldg(v.words + at[h] + 32 * w) : 0u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (4 * w + i < rest[h] && s[h] != DEAD) s[h] = __ldg(g.next + s[h] * 256u + (b[h] >> (8 * i) & 255u));
        }
        if (!__any_sync(0xffffffffu, (rest[0] > 4 * w + 4 && s[0] != DEAD) || (rest[1] > 4 * w + 4 && s[1] != DEAD))) break;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (s[h] != DEAD && id[h] < c.n_logits) atomicOr(&bits[id[h] >> 5], 1u << (id[h] & 31));
    }
  }
  if (n_ranks > 1) cluster.sync();
  else __syncthreads();
  const uint32_t share = (n_words + n_ranks - 1) / n_ranks, b0 = min(rank * share, n_words), b1 = min(b0 + share, n_words);
  for (uint32_t w = b0 + tid; w < b1; w += GR_THREADS) {
    uint32_t m = 0;
    if (n_ranks == 1) m = bits[w];
    else
      for (uint32_t q = 0; q < n_ranks; ++q) m |= cluster.map_shared_rank(bits, q)[w];
    if (c.eos >= 0 && (uint32_t)c.eos < c.n_logits && (uint32_t)c.eos / 32 == w) {
      m &= ~(1u << (c.eos & 31));
      if (s0 != DEAD && g.accept[s0]) m |= 1u << (c.eos & 31);
    }
    for (uint32_t i = 0; i < GR_THREADS / 32; ++i)
      for (uint32_t x = s_row[i]; x; x &= x - 1)
        c.mask[(long long)(w0 + i * 32 + (uint32_t)__ffs((int)x) - 1u) * c.mask_stride + w] = m;
  }
  if (n_ranks > 1) cluster.sync();  // (until the others have read this CTA's bits)
}

// CTAs of a row's cluster: 16 while few rows leave SMs without work, 4 where
// there are enough of them (their groups then keep a CTA's warps busy).
uint32_t mask_ranks(const tok_handle* h, uint32_t n) {
  uint32_t s = 16;
  while (s > 4 && (unsigned long long)n * s > 4ull * (unsigned)h->n_sms) s /= 2;
  return s;
}

// the vocabulary's bytes on the device, once per handle
int ensure_tokens(tok_handle* h) {
  if (h->d_tokens) return TOK_OK;
  const uint32_t n = (uint32_t)h->vocab_off.size() - 1;
  const size_t nb = h->vocab_bytes.size();
  if (nb > 0x7fffffffull) return fail(h, TOK_EINVAL, "grammar: a vocabulary of 2 GiB or more");
  const uint8_t* bytes = h->vocab_bytes.data();
  auto len = [&](uint32_t t) { return (uint32_t)(h->vocab_off[t + 1] - h->vocab_off[t]); };
  auto at = [&](uint32_t t) { return bytes + h->vocab_off[t]; };
  std::vector<uint32_t> order(n);
  for (uint32_t t = 0; t < n; ++t) order[t] = t;
  std::sort(order.begin(), order.end(), [&](uint32_t a, uint32_t b) {
    const uint32_t la = len(a), lb = len(b);
    const int d = std::memcmp(at(a), at(b), std::min(la, lb));
    return d ? d < 0 : la < lb;
  });
  std::vector<TokenGroup> group;
  std::vector<uint32_t> words, id;
  std::vector<uint16_t> rest;
  for (uint32_t i = 0; i < n;) {
    uint32_t m = 1;
    while (m < 32 && i + m < n && *at(order[i + m]) == *at(order[i])) ++m;
    const uint32_t a = order[i], b = order[i + m - 1];
    uint32_t p = 0;
    while (p < 8 && p < len(a) && p < len(b) && at(a)[p] == at(b)[p]) ++p;  // (sorted: common to all between)
    TokenGroup r{0, 0, (uint32_t)words.size()};
    uint32_t most = 0;
    for (uint32_t j = 0; j < p; ++j) r.head |= (unsigned long long)at(a)[j] << (8 * j);
    for (uint32_t q = 0; q < m; ++q) most = std::max(most, len(order[i + q]) - p);
    const uint32_t nw = (most + 3) / 4;
    r.shape = p | nw << 4;
    words.resize(words.size() + (size_t)nw * 32, 0u);
    for (uint32_t q = 0; q < 32; ++q) {
      id.push_back(q < m ? order[i + q] : NO_TOKEN);
      const uint32_t l = q < m ? len(order[i + q]) - p : 0u;
      rest.push_back((uint16_t)l);
      for (uint32_t j = 0; j < l; ++j) words[r.at + (size_t)(j / 4) * 32 + q] |= (uint32_t)at(order[i + q])[p + j] << (8 * (j & 3));
    }
    group.push_back(r);
    i += m;
  }
  if (words.size() > 0x7fffffffull || group.size() > 0xffffull)
    return fail(h, TOK_EINVAL, "grammar: too large a vocabulary");
  std::vector<uint32_t> off(n + 1);
  for (uint32_t t = 0; t <= n; ++t) off[t] = (uint32_t)h->vocab_off[t];
  // one allocation; the parts by falling alignment
  const void* part[6] = {group.data(), words.data(), id.data(), off.data(), rest.data(), bytes};
  const size_t size[6] = {group.size() * sizeof(TokenGroup), words.size() * 4, id.size() * 4, off.size() * 4, rest.size() * 2, nb};
  size_t place[7] = {0};
  for (int i = 0; i < 6; ++i) place[i + 1] = place[i] + (size[i] + 15) / 16 * 16;
  uint8_t* p = nullptr;
  cudaError_t e = halloc(h, &p, place[6]);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(h, TOK_ENOMEM, "grammar: allocation failed");
  }
  for (int i = 0; i < 6 && e == cudaSuccess; ++i)
    if (size[i]) e = cudaMemcpy(p + place[i], part[i], size[i], cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaFree(p);
    return cuda_fail(h, e, "grammar: vocabulary copy");
  }
  h->d_tokens = p;
  h->tokens.group = reinterpret_cast<const TokenGroup*>(p + place[0]);
  h->tokens.words = reinterpret_cast<const uint32_t*>(p + place[1]);
  h->tokens.id = reinterpret_cast<const uint32_t*>(p + place[2]);
  h->tokens.off = reinterpret_cast<const uint32_t*>(p + place[3]);
  h->tokens.rest = reinterpret_cast<const uint16_t*>(p + place[4]);
  h->tokens.bytes = p + place[5];
  h->tokens.n = n;
  h->tokens.n_groups = (uint32_t)group.size();
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
  if (n > 0x7ffffffu || (d_item_off && !d_ids) ||
      (d_mask && (n_logits == 0 || n_logits > MAX_LOGITS || mask_stride < (int64_t)((n_logits + 31) / 32))))
    return fail(h, TOK_EINVAL, "grammar mask: n, n_logits or mask_stride is out of range, or offsets without ids");
  DeviceGuard dg(h->dev);
  MaskCall c{d_state, d_ids, reinterpret_cast<const long long*>(d_item_off), n, eos, d_state_out, n_logits, d_mask, mask_stride};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // many rows with tokens: their states first, once (each row's cluster looks at those of GR_THREADS rows)
  if (!d_mask || (d_ids && d_state_out && n > 64)) {
    k_grammar_states<<<(n + 127) / 128, 128, 0, st>>>(g->g, h->tokens, c);
    h->launches += 1;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(h, e, "kernel launch");
    if (!d_mask) return TOK_OK;
    c.state = d_state_out;
    c.ids = nullptr;
    c.item_off = nullptr;
    c.state_out = nullptr;
  }
  const uint32_t ranks = mask_ranks(h, n), groups = (h->tokens.n_groups + ranks - 1) / ranks;
  const size_t smem = (((size_t)(n_logits + 31) / 32 + 3) / 4 * 4 + groups) * sizeof(uint32_t);
  const cudaError_t e = launch_clusters<k_grammar_mask>(h->dev, n * ranks, GR_THREADS, ranks, smem, st, g->g, h->tokens, c);
  h->launches += 1;
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_fail(h, e, "kernel launch");
  }
  return TOK_OK;
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
