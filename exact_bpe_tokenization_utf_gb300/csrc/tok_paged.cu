// Paged cache: the blocks and slots of a batch's tokens (tok_paged_assign) and
// the blocks of finished requests (tok_paged_release).
//
// With new_k = off[k+1] - off[k], have_k = ceil(ctx_k / bs) and need_k =
// ceil((ctx_k + new_k) / bs), request k takes the need_k - have_k blocks that
// follow the ones taken by the requests before it: base_k = sum of (need - have)
// over the requests before k, and its j-th new block is
// free[n_free - 1 - (base_k + j)].  A token's block is a new one or an old
// entry of its row of the table, by its position alone, so tokens are
// independent once base is known.  A new block's first position always
// belongs to a new token, which writes the block into the table.
#include "tok_handle.cuh"
#include "tok_scan.cuh"

namespace tokgb {
namespace {

constexpr int PG_THREADS = 1024;                   // most threads of a CTA
constexpr int PG_THREADS_4 = 256;                  // of one that takes four tokens a thread,
constexpr int PG_CTAS_4 = 4;                       // and how many of those an SM runs at once (56 registers)
constexpr int PG_MAX_LEN = 0x7fffffff;             // tokens of a request

struct PagedCall {
  tok_paged_args a;
  long long span;      // tokens per CTA, a multiple of its tile
  int wide;            // slot, pos and req lie at 16-byte boundaries
  uint32_t* done;      // the handle's counter of finished CTAs (0 between calls), or nullptr: CTA 0 completes the call
};

struct Req {
  long long off, end, ctx;
  bool bad;       // its own numbers make no sense
  bool wide;      // its row of the table is too narrow
  int have, extra;
};

__device__ __forceinline__ Req load_req(const tok_paged_args& a, uint32_t k) {
  Req r;
  r.off = a.d_item_off[k];
  r.end = a.d_item_off[k + 1];
  r.ctx = a.d_ctx_len ? a.d_ctx_len[k] : 0;
  const long long len = r.end - r.off;
  r.bad = len < 0 || r.ctx < 0 || len > PG_MAX_LEN || r.ctx > PG_MAX_LEN - len || (k == 0 && r.off != 0);
  r.wide = false;
  r.have = r.extra = 0;
  if (!r.bad) {
    const uint32_t bs = a.block_size;
    const uint32_t have = ((uint32_t)r.ctx + bs - 1u) / bs, need = ((uint32_t)(r.ctx + len) + bs - 1u) / bs;
    r.have = (int)have;
    r.extra = (int)(need - have);
    r.wide = need > a.max_blocks && len > 0;
  }
  return r;
}

// sums of two numbers over the block, in every thread; sh: 2 * 32 words
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  if (lane == 0) {
    sh[warp] = a;
    sh[32 + warp] = b;
  }
  __syncthreads();
  a = lane < n ? sh[lane] : 0;
  b = lane < n ? sh[32 + lane] : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
}

// true in one CTA of the grid: the one that gets here last (done is 0 again
// then), or without a counter the first one.  Either way all of its threads are
// here: in place, what is written next is what the others of them read.
__device__ __forceinline__ bool completes(uint32_t* done, unsigned* sh) {
  __syncthreads();
  if (!done) return blockIdx.x == 0;
  if (threadIdx.x == 0) {
    __threadfence();
    const bool last = atomicAdd(done, 1u) == gridDim.x - 1;
    if (last) *done = 0;
    *sh = last;
  }
  __syncthreads();
  return *sh != 0;
}

// One CTA takes a span of tokens, PER a thread at a time.  It reads every
// request once: the blocks of those that end before its span are its base,
// the sum over all of them and their checks decide (alike in every CTA)
// whether the call goes through.  This redundant pass over 20 bytes a request
// costs less than a second launch, or a CTA's wait for another's sums.
//
// Bound by the chain offsets - sums - table or stack entry - store, and in a
// small call by the launch (7 us with its host side).  Measured: a decode step of
// 64 requests 6.5 us, of 4,096 requests 10.2 us (in place, with the counter of
// finished CTAs, 12.4); a prefill of 64 requests with 0.9M tokens 10.3 to 11.2 us
// (15 MB, 1.4 TB/s).
template <int PER>
__global__ void __launch_bounds__(PER == 1 ? PG_THREADS : PG_THREADS_4, PER == 1 ? 1 : PG_CTAS_4) k_paged_assign(PagedCall c) {
  const tok_paged_args& a = c.a;
  constexpr int MOST = (PER == 1 ? PG_THREADS : PG_THREADS_4) * PER;
  __shared__ long long sh[64];
  __shared__ unsigned s_bad, s_wide, s_kf, s_last;
  __shared__ int s_req[MOST], s_add[MOST + 1];
  __shared__ int s_w[32], s_m[32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int tile = nt * PER;
  const long long n_free = *a.d_n_free, n_tok = a.d_item_off[a.n];
  const long long t_begin = (long long)blockIdx.x * c.span;
  if (tid == 0) s_bad = s_wide = s_kf = 0xffffffffu;
  __syncthreads();
  long long total = 0, carry = 0;
#pragma unroll 4
  for (uint32_t k = tid; k < a.n; k += nt) {
    const Req r = load_req(a, k);
    total += r.extra;
    if (r.bad) atomicMin(&s_bad, k);
    else if (r.wide) atomicMin(&s_wide, k);
    else if (r.end <= t_begin) carry += r.extra;
    else if (r.off < r.end) atomicMin(&s_kf, k);
  }
  block_sums(total, carry, sh);  // (its barrier also completes the words above)
  int code = ST_OK;
  if (s_bad != 0xffffffffu || n_free < 0) code = TOK_EINVAL;
  else if (s_wide != 0xffffffffu || (unsigned long long)n_tok > a.cap || total > n_free) code = TOK_EBUF;
  const uint32_t bs = a.block_size;
  uint32_t kf = s_kf;
  const long long t_end = min(t_begin + c.span, (long long)a.cap);
  for (long long t0 = t_begin; t0 < t_end; t0 += tile) {
    const long long mine = t0 + (long long)tid * PER;
    long long slot[PER];
    int pos[PER], req[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      slot[j] = -1;
      pos[j] = req[j] = -1;
    }
    // a request that covers the whole tile, as in a prefill: nothing to find
    bool alone = false;
    Req r{};
    int of = -1;  // r is this request's
    if (code == ST_OK && t0 < n_tok) {
      r = load_req(a, kf);
      of = (int)kf;
      alone = r.off <= t0 && r.end >= t0 + tile;
    }
    int m[PER], w[PER], em = -1, ew = 0;
    long long next_carry = carry;
    if (alone) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        m[j] = of;
        w[j] = 0;
      }
    } else if (code == ST_OK && t0 < n_tok) {
      // the requests with tokens in the tile mark their first one there, and
      // add their blocks at the first token after them
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        s_req[j * nt + tid] = -1;
        s_add[j * nt + tid] = 0;
      }
      if (tid == 0) s_add[tile] = 0;
      __syncthreads();
      const long long t1 = t0 + tile;
      for (uint32_t k0 = kf; k0 < a.n && a.d_item_off[k0] < t1; k0 += nt) {
        const uint32_t k = k0 + tid;
        if (k < a.n) {
          const Req x = load_req(a, k);
          if (x.off < x.end && x.off < t1 && x.end > t0) {
            s_req[x.off > t0 ? (int)(x.off - t0) : 0] = (int)k;
            if (x.end <= t1) s_add[(int)(x.end - t0)] = x.extra;
            if (x.end >= t1) s_last = k;  // (one request covers the tile's last token)
          }
        }
      }
      __syncthreads();
      // each token's request (a running maximum) and base (a running sum)
      int mm = -1, ww = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        mm = max(mm, s_req[tid * PER + j]);
        ww += s_add[tid * PER + j];
        m[j] = mm;
        w[j] = ww;
      }
      int im = mm, iw = ww;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, im, o), y = __shfl_up_sync(0xffffffffu, iw, o);
        if (lane >= o) {
          im = max(im, x);
          iw += y;
        }
      }
      if (lane == 31) {
        s_m[warp] = im;
        s_w[warp] = iw;
      }
      em = __shfl_up_sync(0xffffffffu, im, 1);
      ew = iw - ww;
      if (lane == 0) em = -1;
      __syncthreads();
      // the warps before this one, and all
      const bool in = lane < nt / 32, before = lane < warp;
      int am = before ? s_m[lane] : -1, aw = before ? s_w[lane] : 0, tot = in ? s_w[lane] : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
        aw += __shfl_xor_sync(0xffffffffu, aw, o);
        tot += __shfl_xor_sync(0xffffffffu, tot, o);
      }
      em = max(em, am);
      ew += aw;
      next_carry = carry + tot + s_add[tile];
      if (t1 < n_tok) kf = s_last;
    }
    if (code == ST_OK && t0 < n_tok) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const long long t = mine + j;
        if (t < n_tok) {
          req[j] = max(em, m[j]);
          if (req[j] != of) r = load_req(a, (uint32_t)(of = req[j]));
          pos[j] = (int)(r.ctx + (t - r.off));
          const uint32_t col = (uint32_t)pos[j] / bs, in = (uint32_t)pos[j] - col * bs;
          int32_t* entry = a.d_table + (long long)req[j] * a.table_stride + col;
          int blk;
          if ((int)col >= r.have) {
            blk = a.d_free[n_free - 1 - (carry + ew + w[j] + ((int)col - r.have))];
            if (in == 0) *entry = blk;
          } else {
            blk = *entry;
          }
          slot[j] = (long long)blk * bs + in;
        }
      }
      if (alone && r.end == t0 + tile) next_carry += r.extra;
      carry = next_carry;
      if (!alone) __syncthreads();
    }
    if (PER == 4 && c.wide && mine + PER <= t_end) {
      longlong2* q = reinterpret_cast<longlong2*>(a.d_slot + mine);
      q[0] = make_longlong2(slot[0], slot[1 % PER]);
      q[1] = make_longlong2(slot[2 % PER], slot[3 % PER]);
      if (a.d_pos) *reinterpret_cast<int4*>(a.d_pos + mine) = make_int4(pos[0], pos[1 % PER], pos[2 % PER], pos[3 % PER]);
      if (a.d_req) *reinterpret_cast<int4*>(a.d_req + mine) = make_int4(req[0], req[1 % PER], req[2 % PER], req[3 % PER]);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (mine + j < t_end) {
          a.d_slot[mine + j] = slot[j];
          if (a.d_pos) a.d_pos[mine + j] = pos[j];
          if (a.d_req) a.d_req[mine + j] = req[j];
        }
    }
  }
  // seq_len, n_free_out and the status: by the CTA that finishes last where
  // they may replace what the others still read, else by the first
  if (!completes(c.done, &s_last)) return;
  if (a.d_seq_len)
    for (uint32_t k = tid; k < a.n; k += nt) {
      const long long ctx = a.d_ctx_len ? a.d_ctx_len[k] : 0;
      a.d_seq_len[k] = code == ST_OK ? ctx + (a.d_item_off[k + 1] - a.d_item_off[k]) : ctx;
    }
  if (tid == 0) {
    const unsigned first = min(s_bad, s_wide);
    *a.d_n_free_out = code == ST_OK ? n_free - total : n_free;
    a.d_status[0] = code;
    a.d_status[1] = code == TOK_EINVAL ? 0 : total;
    a.d_status[2] = n_tok;
    a.d_status[3] = first == 0xffffffffu ? -1 : (long long)first;
  }
}

struct ReleaseCall {
  const long long* len;
  const uint8_t* fin;
  uint32_t n, block_size, per;  // per: requests per CTA
  const int32_t* table;
  long long stride;
  uint32_t max_blocks;
  int32_t* free_stack;
  unsigned long long free_cap;
  const long long* n_free;
  long long* n_free_out;
  long long* status;
  uint32_t* done;
};

__device__ __forceinline__ long long release_count(const ReleaseCall& c, uint32_t k, bool* bad) {
  if (!c.fin[k]) return 0;
  const long long len = c.len[k];
  if (len < 0 || len > (long long)c.max_blocks * c.block_size) {
    *bad = true;
    return 0;
  }
  if (len < 0x7fffffffll - c.block_size) return ((uint32_t)len + c.block_size - 1u) / c.block_size;
  return (len + c.block_size - 1) / c.block_size;
}

// One CTA takes a range of requests; as in k_paged_assign each CTA reads all
// of them once for its base and for the checks.  Bound like it, and by a CTA's
// requests being copied one after another; a quarter of 1,000 requests of up to
// 20,011 tokens in blocks of 16 in 8.7 to 12.6 us, in place the same.
__global__ void __launch_bounds__(PG_THREADS, 1) k_paged_release(ReleaseCall c) {
  __shared__ long long sh[64], s_cnt[PG_THREADS];
  __shared__ unsigned s_bad, s_last;
  const int tid = threadIdx.x, nt = blockDim.x;
  const long long n_free = *c.n_free;
  const uint32_t k_begin = min(blockIdx.x * c.per, c.n), k_end = min(k_begin + c.per, c.n);
  if (tid == 0) s_bad = 0xffffffffu;
  __syncthreads();
  long long total = 0, carry = 0;
#pragma unroll 4
  for (uint32_t k = tid; k < c.n; k += nt) {
    bool bad = false;
    const long long m = release_count(c, k, &bad);
    if (bad) atomicMin(&s_bad, k);
    total += m;
    if (k < k_begin) carry += m;
  }
  block_sums(total, carry, sh);
  int code = ST_OK;
  if (s_bad != 0xffffffffu || n_free < 0) code = TOK_EINVAL;
  else if ((unsigned long long)(n_free + total) > c.free_cap) code = TOK_EBUF;
  if (code == ST_OK) {
    long long base = n_free + carry;
    for (uint32_t k0 = k_begin; k0 < k_end; k0 += nt) {
      bool bad = false;
      __syncthreads();
      s_cnt[tid] = k0 + tid < k_end ? release_count(c, k0 + tid, &bad) : 0;
      __syncthreads();
      for (uint32_t i = 0; i < (uint32_t)nt && k0 + i < k_end; ++i) {
        const long long cnt = s_cnt[i];
        const int32_t* row = c.table + (long long)(k0 + i) * c.stride;
#pragma unroll 4
        for (long long j = tid; j < cnt; j += nt) c.free_stack[base + j] = row[j];
        base += cnt;
      }
    }
  }
  if (!completes(c.done, &s_last)) return;
  if (tid == 0) {
    *c.n_free_out = code == ST_OK ? n_free + total : n_free;
    c.status[0] = code;
    c.status[1] = code == TOK_EINVAL ? 0 : total;
    c.status[2] = 0;
    c.status[3] = s_bad == 0xffffffffu ? -1 : (long long)s_bad;
  }
}

// threads of a CTA for n things at a time: 128 to most
unsigned threads_for(unsigned long long n, int most) {
  unsigned t = 128;
  while (t < (unsigned)most && t < n) t *= 2;
  return t;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_paged_assign(tok_handle* h, const tok_paged_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (!a || !a->d_item_off || !a->d_table || !a->d_free || !a->d_n_free || !a->d_n_free_out || !a->d_status ||
      (a->cap && !a->d_slot) || a->n == 0)
    return fail(h, TOK_EINVAL, "paged assign: a buffer is NULL, or n is 0");
  if (a->n > 0x7fffffffu || a->block_size == 0 || a->block_size > (1u << 20) || a->max_blocks > 0x7fffffffu ||
      a->table_stride < (int64_t)a->max_blocks || a->cap > (1ull << 40))
    return fail(h, TOK_EINVAL, "paged assign: n, block_size, max_blocks, table_stride or cap is out of range");
  DeviceGuard g(h->dev);
  PagedCall c{};
  c.a = *a;
  // one token a thread while all of them fit two CTAs per SM (a decode step's
  // tokens are of as many requests: one's loads would wait for another's), else
  // four.  4,096 requests of a token 10.3 us with one, 16.5 with four; prefills of
  // 64 requests of up to 20,001 tokens 6.2 and 6.7, of up to 180,001 16.4 and 10.3.
  // Threads of a CTA: many CTAs hide one another's latencies, but each reads every
  // request.  One token a thread, 512 and 1,024 threads: 1,000 requests 7.2 and
  // 8.3 us, 4,096 10.3 both, 15,000 24.7 and 18.5.  Four, 128 and 256: 64 long
  // requests 10.3 and 12.5, 4,096 requests with 3.1M tokens 38.8 and 34.9.
  unsigned threads = threads_for(std::max<unsigned long long>(a->n, a->cap), a->n > 4096 ? PG_THREADS : 512);
  const bool one = a->cap <= 2ull * (unsigned)h->n_sms * threads;
  if (!one) threads = a->n > 512 ? PG_THREADS_4 : 128;
  const long long tile = (long long)threads * (one ? 1 : 4);
  const long long tiles = std::max<long long>(1, ((long long)a->cap + tile - 1) / tile);
  const long long ctas = std::min<long long>(tiles, (one ? 2u : PG_CTAS_4 * PG_THREADS_4 / threads) * (long long)h->n_sms);
  c.span = (tiles + ctas - 1) / ctas * tile;
  c.wide = ((reinterpret_cast<uintptr_t>(a->d_slot) | reinterpret_cast<uintptr_t>(a->d_pos) |
             reinterpret_cast<uintptr_t>(a->d_req)) & 15u) == 0;
  const bool in_place = a->d_n_free_out == a->d_n_free || (a->d_seq_len && a->d_seq_len == a->d_ctx_len);
  c.done = in_place && ctas > 1 ? h->d_done : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (one) k_paged_assign<1><<<(unsigned)ctas, threads, 0, s>>>(c);
  else k_paged_assign<4><<<(unsigned)ctas, threads, 0, s>>>(c);
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

int tok_paged_release(tok_handle* h, const int64_t* d_seq_len, const uint8_t* d_done, uint32_t n, uint32_t block_size,
                      const int32_t* d_table, int64_t table_stride, uint32_t max_blocks, int32_t* d_free,
                      uint64_t free_cap, const int64_t* d_n_free, int64_t* d_n_free_out, int64_t* d_status,
                      void* stream) try {
  if (!h) return TOK_EINVAL;
  if (!d_seq_len || !d_done || !d_table || !d_free || !d_n_free || !d_n_free_out || !d_status || n == 0)
    return fail(h, TOK_EINVAL, "paged release: a buffer is NULL, or n is 0");
  if (n > 0x7fffffffu || block_size == 0 || block_size > (1u << 20) || max_blocks > 0x7fffffffu ||
      table_stride < (int64_t)max_blocks)
    return fail(h, TOK_EINVAL, "paged release: n, block_size, max_blocks or table_stride is out of range");
  DeviceGuard g(h->dev);
  ReleaseCall c{};
  c.len = reinterpret_cast<const long long*>(d_seq_len);
  c.fin = d_done;
  c.n = n;
  c.block_size = block_size;
  c.table = d_table;
  c.stride = table_stride;
  c.max_blocks = max_blocks;
  c.free_stack = d_free;
  c.free_cap = free_cap;
  c.n_free = reinterpret_cast<const long long*>(d_n_free);
  c.n_free_out = reinterpret_cast<long long*>(d_n_free_out);
  c.status = reinterpret_cast<long long*>(d_status);
  const uint32_t ctas = std::min<uint32_t>((n + 3) / 4, 2u * (uint32_t)h->n_sms);
  c.per = (n + ctas - 1) / ctas;
  c.done = d_n_free_out == d_n_free && ctas > 1 ? h->d_done : nullptr;
  k_paged_release<<<ctas, threads_for(n, 512), 0, static_cast<cudaStream_t>(stream)>>>(c);
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
