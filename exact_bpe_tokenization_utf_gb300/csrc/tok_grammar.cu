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
#include "tok_scan.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MAX_LOGITS = 1u << 20;
constexpr uint32_t DEAD = 0xffffu;
constexpr uint32_t NO_TOKEN = 0xffffffffu;
constexpr int GR_THREADS = 512;

struct DevGrammar {
  const uint16_t* next;   // n_states rows of 256
  const uint32_t* leaves; // per state: the kinds of bytes of which some change the state
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

// (eight bytes at a time, whose loads need not wait for the states)
__device__ __forceinline__ uint32_t walk(const DevGrammar& g, const DevTokens& v, uint32_t s, uint32_t t) {
  const uint32_t begin = v.off[t], end = v.off[t + 1];
  for (uint32_t i = begin; i < end && s != DEAD; i += 8) {
    uint32_t b[8];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) b[j] = i + j < end ? __ldg(v.bytes + i + j) : 0u;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (i + j < end && s != DEAD) s = __ldg(g.next + s * 256u + b[j]);
  }
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

// The rows' states alone: a thread walks a row, one load after another.
__global__ void __launch_bounds__(128) k_grammar_states(DevGrammar g, DevTokens v, MaskCall c) {
  const uint32_t k = blockIdx.x * 128 + threadIdx.x;
  if (k >= c.n) return;
  const uint32_t s = row_state(g, v, c, k);
  c.state_out[k] = s == DEAD ? -1 : (int32_t)s;
}

// read once: kept out of L1, where the automaton's rows are
__device__ __forceinline__ uint32_t load_once(const uint32_t* p) {
  uint32_t x;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// a lane's token of a group whose common bytes lead to state s
struct Item {
  uint32_t s, place, rest, at, word, kinds;
};

// A row's window of GR_THREADS rows: its state, and the rows in equal states.
// Each thread looks at one row.  sh holds GR_THREADS / 32 + 1 words.
struct Window {
  uint32_t state;
  bool first;            // no earlier row of the window is in this state
  const uint32_t* same;  // bits of the rows that are
  uint32_t begin;
};

__device__ __forceinline__ Window look_around(const DevGrammar& g, const DevTokens& v, const MaskCall& c, uint32_t k, uint32_t* sh) {
  Window w;
  w.begin = k / GR_THREADS * GR_THREADS;
  const uint32_t j = w.begin + threadIdx.x;
  uint32_t sj = DEAD;
  if (j < c.n) sj = row_state(g, v, c, j);
  if (j == k) sh[GR_THREADS / 32] = sj;
  __syncthreads();
  w.state = sh[GR_THREADS / 32];
  const bool same = j < c.n && sj == w.state;
  const uint32_t b = __ballot_sync(0xffffffffu, same);
  if ((threadIdx.x & 31u) == 0) sh[threadIdx.x >> 5] = b;
  w.first = !__syncthreads_or(same && j < k);
  w.same = sh;
  return w;
}

// f(row's mask) for each row of a window that is in its state
template <class F>
__device__ __forceinline__ void each_same(const Window& win, const MaskCall& c, F f) {
  for (uint32_t i = 0; i < GR_THREADS / 32; ++i)
    for (uint32_t x = win.same[i]; x; x &= x - 1)
      f(c.mask + (long long)(win.begin + i * 32 + (uint32_t)__ffs((int)x) - 1u) * c.mask_stride);
}

// A CTA's groups: 32 in turn with the others of its row (long tokens lie together).
struct Share {
  uint32_t rank, n_ranks;
  __device__ __forceinline__ uint32_t group(uint32_t i) const { return (i / 32 * n_ranks + rank) * 32 + i % 32; }
  __device__ __forceinline__ uint32_t count(const DevTokens& v) const { return ((v.n_groups + 31) / 32 + n_ranks - 1) / n_ranks * 32; }
};

// a thread's first group, on its way while the states are looked at
struct First {
  uint4 r;
  uint32_t kinds;
};
__device__ __forceinline__ First first_group(const DevTokens& v, const Share& sh) {
  First f{make_uint4(0, 0, 0, 0), 0};
  if (threadIdx.x < sh.count(v) && sh.group(threadIdx.x) < v.n_groups) {
    f.r = __ldg(reinterpret_cast<const uint4*>(v.group + sh.group(threadIdx.x)));
    f.kinds = __ldg(v.group_kinds + sh.group(threadIdx.x));
  }
  return f;
}

// A thread walks a group's common first bytes, so that one step decides over up
// to 32 tokens.  The groups that survive are listed: from the front those whose
// tokens have to be walked (group | state << 16, place of their words), from
// the back those whose other bytes are all of kinds that do not change the
// state.  n_live[0] and n_live[1] (0 before, behind a barrier) receive their
// numbers.  Ends with a barrier.
__device__ __forceinline__ void find_live(const DevGrammar& g, const DevTokens& v, const Share& sh, First f, uint32_t s0, uint2* live,
                                          uint32_t room, uint32_t* n_live) {
  const uint32_t tid = threadIdx.x, lane = tid & 31u, n = sh.count(v);
  for (uint32_t base = 0; base < n; base += GR_THREADS) {
    const uint32_t q = base + tid < n ? sh.group(base + tid) : v.n_groups;
    unsigned long long head = (unsigned long long)f.r.y << 32 | f.r.x;
    uint32_t s = q < v.n_groups ? s0 : DEAD;
    const uint32_t kinds = f.kinds, words = f.r.w;
    uint32_t i = f.r.z;
    if (base + GR_THREADS + tid < n) {  // the next one
      const uint32_t next = sh.group(base + GR_THREADS + tid);
      if (next < v.n_groups) {
        f.r = __ldg(reinterpret_cast<const uint4*>(v.group + next));
        f.kinds = __ldg(v.group_kinds + next);
      }
    }
    if (i == 0 && s != DEAD && __ldg(g.next + s * 256u + (uint32_t)(head & 255u)) == DEAD) s = DEAD;
    for (; i && s != DEAD; --i) {
      s = __ldg(g.next + s * 256u + (uint32_t)(head & 255u));
      head >>= 8;
    }
    const bool whole = s != DEAD && (kinds & __ldg(g.leaves + s)) == 0;
#pragma unroll
    for (uint32_t l = 0; l < 2; ++l) {
      const uint32_t in = __ballot_sync(0xffffffffu, s != DEAD && whole == (l == 1));
      uint32_t at = 0;
      if (lane == 0 && in) at = atomicAdd(n_live + l, (uint32_t)__popc(in));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(in & ((1u << lane) - 1u));
      if (in >> lane & 1u) live[l ? room - 1 - at : at] = make_uint2(q | s << 16, words);
    }
  }
  __syncthreads();
}

// A warp takes a listed group's tokens, one per lane, and sets the allowed ones'
// bits: at once where no byte changes the state (inside a string that is most
// groups), the others by a walk, two groups at a time with the next two on
// their way.  Four bytes are looked up at once, as if the state stayed; where it
// changes, the lookups after that are done again.  A token's leading bytes of one
// kind are passed over where that kind does not change the state: the longest
// tokens are runs, and a warp that walked them kept its CTA waiting.
__device__ __forceinline__ void walk_live(const DevGrammar& g, const DevTokens& v, const uint2* live, uint32_t room,
                                          const uint32_t* n_live, uint32_t n_logits, uint32_t* bits) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  constexpr uint32_t W = GR_THREADS / 32;
  auto allow = [&](uint32_t id) {
    if (id < n_logits) atomicOr(&bits[id >> 5], 1u << (id & 31));
  };
  const uint32_t n_whole = n_live[1], n_walk = n_live[0];
  for (uint32_t e = warp; e < n_whole; e += 4 * W) {
    uint32_t id[4];
#pragma unroll
    for (uint32_t h = 0; h < 4; ++h)
      id[h] = e + h * W < n_whole ? load_once(v.id + (live[room - 1 - (e + h * W)].x & 0xffffu) * 32 + lane) : NO_TOKEN;
#pragma unroll
    for (uint32_t h = 0; h < 4; ++h) allow(id[h]);
  }
  auto load = [&](uint32_t f) {
    Item t{DEAD, 0, 0, 0, 0, 0};
    if (f < n_walk) {  // (every group has a first word, so that these loads need not wait for one another)
      const uint2 e = live[f];
      t.s = e.x >> 16;
      t.place = (e.x & 0xffffu) * 32 + lane;
      t.at = e.y + lane;
      t.word = load_once(v.words + t.at);
      t.rest = load_once(v.rest + t.place);
      t.kinds = load_once(v.kinds + t.place);
    }
    return t;
  };
  Item now[2] = {load(warp), load(warp + W)};
  for (uint32_t e = warp; e < n_walk; e += 2 * W) {
    const Item next[2] = {load(e + 2 * W), load(e + 3 * W)};  // (used in the next turn: nothing waits for it here)
    uint32_t id[2], from[2];  // the bytes of a word to be read: from here
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      id[h] = now[h].s != DEAD ? load_once(v.id + now[h].place) : NO_TOKEN;
      const uint32_t leaves = now[h].s != DEAD ? __ldg(g.leaves + now[h].s) : 0u;
      const uint32_t r = now[h].rest, skip = leaves >> (r >> 16 & 31u) & 1u ? 0u : r >> 21;
      from[h] = skip & 3u;
      now[h].rest = now[h].kinds & leaves ? (r & 0xffffu) - (skip & ~3u) : 0u;
      now[h].at += 8 * (skip & ~3u);
      if (skip > 3 && now[h].rest) now[h].word = load_once(v.words + now[h].at);
    }
    while (__any_sync(0xffffffffu, now[0].rest | now[1].rest)) {
      uint32_t ahead[2], to[2];  // the tokens' next words; to here
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        now[h].at += 32;
        ahead[h] = now[h].rest > 4 ? load_once(v.words + now[h].at) : 0u;
        to[h] = min(now[h].rest, 4u);
      }
      while (__any_sync(0xffffffffu, from[0] < to[0] || from[1] < to[1])) {
        uint32_t t[2][4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            t[h][i] = i >= from[h] && i < to[h] ? (uint32_t)__ldg(g.next + now[h].s * 256u + (now[h].word >> (8 * i) & 255u)) : now[h].s;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s = now[h].s;
          // the first byte that changes the state is the last one that counts
          const uint32_t stop = t[h][0] != s ? 0 : t[h][1] != s ? 1 : t[h][2] != s ? 2 : 3;
          now[h].s = stop == 0 ? t[h][0] : stop == 1 ? t[h][1] : stop == 2 ? t[h][2] : t[h][3];
          from[h] = now[h].s == DEAD ? to[h] : stop + 1;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        now[h].word = ahead[h];
        now[h].rest = now[h].s == DEAD ? 0u : now[h].rest - to[h];
        from[h] = 0;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (now[h].s != DEAD) allow(id[h]);
      now[h] = next[h];
    }
  }
}

// word w of a mask with the end token's bit as the state has it (the token's own bytes do not count)
__device__ __forceinline__ uint32_t with_eos(const DevGrammar& g, const MaskCall& c, uint32_t s, uint32_t w, uint32_t m) {
  if (c.eos >= 0 && (uint32_t)c.eos < c.n_logits && (uint32_t)c.eos / 32 == w) {
    m &= ~(1u << (c.eos & 31));
    if (s != DEAD && g.accept[s]) m |= 1u << (c.eos & 31);
  }
  return m;
}

__device__ __forceinline__ uint2* list_behind(uint32_t* bits, uint32_t n_words) {
  return reinterpret_cast<uint2*>(bits + (n_words + 3) / 4 * 4);
}

// A cluster for each row.  The CTAs share the groups; then each sends its
// words that are not empty to the CTAs that write them, a share of the row
// each.  Rows in equal states are walked once, by the first one's cluster,
// which writes all of them.
//
// Bound by barriers and by the chains of lookups (every row's cluster looks at
// all groups, whatever its state allows): 473 states of a grammar over 100,257
// tokens (47M decisions) in 49 us, issuing in 43% of all cycles, of which the
// masks' 6 MB are 1 us; one row in 8 to 12 us, the launch 7 of them.  A
// CTA per row, with rows that have many live groups finished in 16 parts by a
// second kernel, took 49 us for those 473 states (clusters then 62) but 122
// instead of 42 for 400 rows that share states.
__global__ void __launch_bounds__(GR_THREADS, 3) k_grammar_mask(DevGrammar g, DevTokens v, MaskCall c) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t s_mem[];
  __shared__ uint32_t s_live[2], s_row[GR_THREADS / 32 + 1];
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), n_ranks = cluster.num_blocks(), k = blockIdx.x / n_ranks, tid = threadIdx.x;
  const uint32_t n_words = (c.n_logits + 31) / 32;
  uint32_t* bits = s_mem;
  uint2* live = list_behind(bits, n_words);
  const Share share{rank, n_ranks};
  const First f = first_group(v, share);
  for (uint32_t i = tid; i < (n_words + 3) / 4; i += GR_THREADS) reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 2) s_live[tid] = 0;
  const Window win = look_around(g, v, c, k, s_row);
  if (tid == 0 && rank == 0 && c.state_out) c.state_out[k] = win.state == DEAD ? -1 : (int32_t)win.state;
  if (!win.first) return;  // (in every CTA of the cluster alike)
  cluster_arrive();        // (waited for before another CTA's bits are set; they are 0 since the window's barriers)
  if (win.state != DEAD) {
    find_live(g, v, share, f, win.state, live, share.count(v), s_live);
    walk_live(g, v, live, share.count(v), s_live, c.n_logits, bits);
  }
  const uint32_t each = (n_words + n_ranks - 1) / n_ranks;
  __syncthreads();
  cluster_wait();
  if (s_live[0] | s_live[1])
    for (uint32_t w = tid; w < n_words; w += GR_THREADS)
      if (bits[w] && w / each != rank) atomicOr(cluster.map_shared_rank(bits, w / each) + w, bits[w]);
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  const uint32_t w1 = min((rank + 1) * each, n_words);
  for (uint32_t w = rank * each + tid; w < w1; w += GR_THREADS) {
    const uint32_t m = with_eos(g, c, win.state, w, bits[w]);
    each_same(win, c, [&](uint32_t* row) { row[w] = m; });
  }
}

// bytes of shared memory of a CTA: a row's bits, and a list of groups
size_t mask_bytes(uint32_t n_logits, uint32_t groups) {
  return ((size_t)(n_logits + 31) / 32 + 3) / 4 * 16 + groups * sizeof(uint2);
}
uint32_t share_of(const tok_handle* h, uint32_t ranks) { return ((h->tokens.n_groups + 31) / 32 + ranks - 1) / ranks * 32; }

// CTAs of a row's cluster, for the times of a vocabulary of 100,257 tokens with
// 16, 8 and 4: 16 while that makes no more than four for each SM (a row 10.3, 10.4
// and 10.4 us; 32 rows of one grammar 15.6, 16.5 and 16.5 or, of another, 22.7,
// 18.5 and 22.7; 76 rows 32.2, 21.6 and 26.7), 8 while those are no more than
// eight (120 rows 40.3, 23.6 and 22.7), else 4 (400 rows 101, 50 and 33, with two
// 41; 473 rows in as many states 138, 69 and 50.6, with two 50.2).  And 64 groups
// for each CTA (1,257 tokens: 60 rows 20.6, 12.3 and 10.3; 120 rows 32.1, 16.8 and
// 11.6).
uint32_t mask_ranks(const tok_handle* h, uint32_t n, uint32_t n_logits) {
  const unsigned long long sms = (unsigned)h->n_sms;
  uint32_t s = 16;
  while (s > 4 && ((unsigned long long)n * s > (s == 16 ? 4 : 8) * sms || h->tokens.n_groups < 64 * s) &&
         mask_bytes(n_logits, share_of(h, s / 2)) <= MOST_SHARED)
    s /= 2;
  return s;
}

// length of the well-formed UTF-8 sequence of two bytes or more (RFC 3629) at s[0..n), or 0
uint32_t sequence(const uint8_t* s, uint32_t n) {
  const uint8_t b = s[0];
  const uint32_t len = b >= 0xc2 && b <= 0xdf ? 2 : b >= 0xe0 && b <= 0xef ? 3 : b >= 0xf0 && b <= 0xf4 ? 4 : 0;
  if (len == 0 || len > n) return 0;
  const uint8_t lo = b == 0xe0 ? 0xa0 : b == 0xf0 ? 0x90 : 0x80, hi = b == 0xed ? 0x9f : b == 0xf4 ? 0x8f : 0xbf;
  if (s[1] < lo || s[1] > hi) return 0;
  for (uint32_t i = 2; i < len; ++i)
    if ((s[i] & 0xc0) != 0x80) return 0;
  return len;
}

// the kinds of a token's bytes; well-formed sequences are a kind of their own
uint32_t kinds_of(const uint8_t* s, uint32_t n) {
  uint32_t k = 0;
  for (uint32_t i = 0; i < n;) {
    const uint32_t len = sequence(s + i, n - i);
    k |= 1u << (len ? KIND_SEQUENCE : byte_kind(s[i]));
    i += len ? len : 1;
  }
  return k;
}

// the bytes of one kind that a text begins with, sequences whole
struct Run {
  uint32_t kind, bytes;
};
Run first_run(const uint8_t* s, uint32_t n) {
  Run r{0, 0};
  while (r.bytes < n) {
    const uint32_t seq = sequence(s + r.bytes, n - r.bytes), len = seq ? seq : 1, k = seq ? KIND_SEQUENCE : byte_kind(s[r.bytes]);
    if ((r.bytes && k != r.kind) || r.bytes + len > MOST_RUN) break;
    r.kind = k;
    r.bytes += len;
  }
  return r;
}

// Whether every well-formed sequence of two bytes or more leads from state s
// back to s.  (Answers no where more than a few states are on the way.)
bool sequences_return(const int32_t* next, uint32_t s) {
  for (uint32_t b = 0xc2; b <= 0xf4; ++b) {
    std::vector<int32_t> at{next[(size_t)s * 256 + b]}, to;
    const uint32_t len = b <= 0xdf ? 2 : b <= 0xef ? 3 : 4;
    for (uint32_t i = 1; i < len; ++i) {
      const uint32_t lo = i > 1 ? 0x80 : b == 0xe0 ? 0xa0 : b == 0xf0 ? 0x90 : 0x80;
      const uint32_t hi = i > 1 ? 0xbf : b == 0xed ? 0x9f : b == 0xf4 ? 0x8f : 0xbf;
      to.clear();
      for (int32_t a : at) {
        if (a < 0) return false;
        for (uint32_t x = lo; x <= hi; ++x) {
          const int32_t y = next[(size_t)a * 256 + x];
          if (std::find(to.begin(), to.end(), y) == to.end()) to.push_back(y);
        }
        if (to.size() > 8) return false;
      }
      at.swap(to);
    }
    if (at.size() != 1 || at[0] != (int32_t)s) return false;
  }
  return true;
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
  std::vector<uint32_t> words, id, kinds, group_kinds, rest;
  for (uint32_t i = 0; i < n;) {
    uint32_t m = 1;
    while (m < 32 && i + m < n && *at(order[i + m]) == *at(order[i])) ++m;
    const uint32_t a = order[i], b = order[i + m - 1];
    uint32_t p = 0;
    while (p < 8 && p < len(a) && p < len(b) && at(a)[p] == at(b)[p]) ++p;  // (sorted: common to all between)
    // not inside a code point, whose rest would have to be walked
    auto splits = [&] {
      for (uint32_t q = 0; q < m; ++q)
        if (len(order[i + q]) > p && (at(order[i + q])[p] & 0xc0) == 0x80) return true;
      return false;
    };
    while (p > 0 && splits()) --p;
    TokenGroup r{0, 0, (uint32_t)words.size()};
    uint32_t most = 0;
    for (uint32_t j = 0; j < std::max(p, 1u); ++j) r.head |= (unsigned long long)at(a)[j] << (8 * j);
    for (uint32_t q = 0; q < m; ++q) most = std::max(most, len(order[i + q]) - p);
    const uint32_t nw = std::max(1u, (most + 3) / 4);
    uint32_t all = 0;
    r.prefix = p;
    words.resize(words.size() + (size_t)nw * 32, 0u);
    for (uint32_t q = 0; q < 32; ++q) {
      id.push_back(q < m ? order[i + q] : NO_TOKEN);
      const uint32_t l = q < m ? len(order[i + q]) - p : 0u;
      const Run run = q < m ? first_run(at(order[i + q]) + p, l) : Run{0, 0};
      rest.push_back(l | run.kind << 16 | run.bytes << 21);
      for (uint32_t j = 0; j < l; ++j)
        words[r.at + (size_t)(j / 4) * 32 + q] |= (uint32_t)at(order[i + q])[p + j] << (8 * (j & 3));
      const uint32_t some = q < m ? kinds_of(at(order[i + q]) + p, l) : 0u;
      kinds.push_back(some);
      all |= some;
    }
    group_kinds.push_back(all);
    group.push_back(r);
    i += m;
  }
  if (words.size() > 0x7fffffffull || group.size() > 0xffffull)
    return fail(h, TOK_EINVAL, "grammar: too large a vocabulary");
  std::vector<uint32_t> off(n + 1);
  for (uint32_t t = 0; t <= n; ++t) off[t] = (uint32_t)h->vocab_off[t];
  // one allocation; the parts by falling alignment
  constexpr int N_PARTS = 8;
  const void* part[N_PARTS] = {group.data(), words.data(), id.data(), kinds.data(), group_kinds.data(), off.data(), rest.data(), bytes};
  const size_t size[N_PARTS] = {group.size() * sizeof(TokenGroup), words.size() * 4, id.size() * 4, kinds.size() * 4,
                              group_kinds.size() * 4, off.size() * 4, rest.size() * 4, nb};
  size_t place[N_PARTS + 1] = {0};
  for (int i = 0; i < N_PARTS; ++i) place[i + 1] = place[i] + (size[i] + 15) / 16 * 16;
  uint8_t* p = nullptr;
  cudaError_t e = halloc(h, &p, place[N_PARTS]);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(h, TOK_ENOMEM, "grammar: allocation failed");
  }
  for (int i = 0; i < N_PARTS && e == cudaSuccess; ++i)
    if (size[i]) e = cudaMemcpy(p + place[i], part[i], size[i], cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaFree(p);
    return cuda_fail(h, e, "grammar: vocabulary copy");
  }
  h->d_tokens = p;
  h->tokens.group = reinterpret_cast<const TokenGroup*>(p + place[0]);
  h->tokens.words = reinterpret_cast<const uint32_t*>(p + place[1]);
  h->tokens.id = reinterpret_cast<const uint32_t*>(p + place[2]);
  h->tokens.kinds = reinterpret_cast<const uint32_t*>(p + place[3]);
  h->tokens.group_kinds = reinterpret_cast<const uint32_t*>(p + place[4]);
  h->tokens.off = reinterpret_cast<const uint32_t*>(p + place[5]);
  h->tokens.rest = reinterpret_cast<const uint32_t*>(p + place[6]);
  h->tokens.bytes = p + place[7];
  h->tokens.n = n;
  h->tokens.n_groups = (uint32_t)group.size();
  return TOK_OK;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

struct tok_grammar {
  const tok_handle* h = nullptr;  // compared, not read: the grammar may outlive it
  int dev = 0;
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
  std::vector<uint32_t> leaves(n_states, 0u);
  for (size_t i = 0; i < t.size(); ++i) {
    if (next[i] < -1 || next[i] >= (int32_t)n_states) return fail(h, TOK_EINVAL, "grammar: a next state is out of range");
    t[i] = next[i] < 0 ? (uint16_t)DEAD : (uint16_t)next[i];
    if (next[i] != (int32_t)(i / 256)) leaves[i / 256] |= 1u << byte_kind((uint8_t)(i & 255));
  }
  for (uint32_t s = 0; s < n_states; ++s)
    if (!sequences_return(next, s)) leaves[s] |= 1u << KIND_SEQUENCE;
  DeviceGuard dg(h->dev);
  int rc = ensure_tokens(h);
  if (rc) return rc;
  tok_grammar* g = new tok_grammar();
  const size_t tb = t.size() * sizeof(uint16_t), lb = n_states * sizeof(uint32_t);
  cudaError_t e = halloc(h, &g->d_mem, tb + lb + n_states);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete g;
    return fail(h, TOK_ENOMEM, "grammar: allocation failed");
  }
  e = cudaMemcpy(g->d_mem, t.data(), tb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(g->d_mem + tb, leaves.data(), lb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(g->d_mem + tb + lb, accept, n_states, cudaMemcpyHostToDevice);
  // (a copy from pageable memory may return with its last part still on its way, the vocabulary's copies above
  // too, and a caller's stream need not wait for the default one)
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  if (e != cudaSuccess) {
    cudaFree(g->d_mem);
    delete g;
    return cuda_fail(h, e, "grammar: copy");
  }
  g->h = h;
  g->dev = h->dev;
  g->g = DevGrammar{reinterpret_cast<const uint16_t*>(g->d_mem), reinterpret_cast<const uint32_t*>(g->d_mem + tb),
                    g->d_mem + tb + lb, n_states};
  *out = g;
  return TOK_OK;
} catch (...) {
  return fail(h, TOK_ENOMEM, "grammar: out of host memory");
}

void tok_grammar_free(tok_grammar* g) {
  if (!g) return;
  DeviceGuard dg(g->dev);
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
  // Each row's cluster finds the states of its window of GR_THREADS rows, unless
  // they are found first, once, by a kernel of their own: for rows of one token
  // each beyond a window (1,000 rows: 50 us with that kernel, 66 without; 4,000:
  // 158 and 245; 400 rows, which are one window, 43 and 41 in one grammar, 29 and
  // 33 in another), for rows of any number of tokens early (64 rows of 8 tokens:
  // 35 and 34; of 100 tokens: 176 and 341).
  if (!d_mask || (d_ids && d_state_out && n > (d_item_off ? 16u : (uint32_t)GR_THREADS))) {
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
  const uint32_t ranks = mask_ranks(h, n, n_logits);
  const cudaError_t e = launch_clusters<k_grammar_mask>(h->dev, n * ranks, GR_THREADS, ranks, mask_bytes(n_logits, share_of(h, ranks)), st,
                                                        g->g, h->tokens, c);
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
