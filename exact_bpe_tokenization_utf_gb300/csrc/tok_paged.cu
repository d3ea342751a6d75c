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

constexpr int PG_THREADS = 256;
constexpr int PG_PER = 4;                          // tokens per thread and tile
constexpr int PG_TILE = PG_THREADS * PG_PER;       // tokens per tile
constexpr int PG_MAX_LEN = 0x7fffffff;             // tokens of a request

struct PagedCall {
  tok_paged_args a;
  long long span;      // tokens per CTA, a multiple of PG_TILE
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

// One CTA takes a span of tokens.  It reads every request once: the blocks of
// those that end before its span are its base, the sum over all of them and
// their checks decide (alike in every CTA) whether the call goes through.
__global__ void __launch_bounds__(PG_THREADS) k_paged_assign(PagedCall c) {
  const tok_paged_args& a = c.a;
  __shared__ long long sh[PG_THREADS / 32], sh_first;
  __shared__ unsigned s_bad, s_kf, s_last;
  __shared__ int s_req[PG_TILE], s_add[PG_TILE + 1];
  __shared__ int s_w[PG_THREADS / 32], s_m[PG_THREADS / 32];
  const int tid = threadIdx.x;
  const long long n_free = *a.d_n_free;
  const long long t_begin = (long long)blockIdx.x * c.span;
  if (tid == 0) {
    s_bad = s_kf = 0xffffffffu;
    s_last = 0;
    sh_first = 0;
  }
  __syncthreads();
  long long sum = 0, before = 0;
  bool bad = false;
  for (uint32_t k = tid; k < a.n; k += PG_THREADS) {
    const Req r = load_req(a, k);
    if (r.bad || r.wide) {
      atomicMin(&s_bad, k);
      bad |= r.bad;
      sum += r.extra;
      continue;
    }
    sum += r.extra;
    if (r.end <= t_begin) before += r.extra;
    else if (r.off < r.end) atomicMin(&s_kf, k);
  }
  const int any_bad = __syncthreads_or(bad);
  long long total, carry;
  block_excl_sum(sum, &total, sh);
  block_excl_sum(before, &carry, sh);
  const long long n_tok = a.d_item_off[a.n];
  int code = ST_OK;
  if (any_bad || n_free < 0) code = TOK_EINVAL;
  else if (s_bad != 0xffffffffu || (unsigned long long)n_tok > a.cap || total > n_free) code = TOK_EBUF;
  const uint32_t bs = a.block_size;
  uint32_t kf = s_kf;
  long long t_end = t_begin + c.span;
  if (t_end > (long long)a.cap) t_end = (long long)a.cap;
  for (long long t0 = t_begin; t0 < t_end; t0 += PG_TILE) {
    if (code != ST_OK || t0 >= n_tok) {  // padding
      for (int i = tid; i < PG_TILE && t0 + i < t_end; i += PG_THREADS) {
        a.d_slot[t0 + i] = -1;
        if (a.d_pos) a.d_pos[t0 + i] = -1;
        if (a.d_req) a.d_req[t0 + i] = -1;
      }
      continue;
    }
    // the requests with tokens in the tile mark their first one there, and
    // add their blocks at the first token after them
    for (int i = tid; i <= PG_TILE; i += PG_THREADS) {
      if (i < PG_TILE) s_req[i] = -1;
      s_add[i] = 0;
    }
    __syncthreads();
    const long long t1 = t0 + PG_TILE;
    uint32_t k0 = kf;
    for (; k0 < a.n && a.d_item_off[k0] < t1; k0 += PG_THREADS) {
      const uint32_t k = k0 + tid;
      if (k < a.n) {
        const Req r = load_req(a, k);
        if (r.off < r.end && r.off < t1 && r.end > t0) {
          s_req[r.off > t0 ? (int)(r.off - t0) : 0] = (int)k;
          if (r.end <= t1) s_add[(int)(r.end - t0)] = r.extra;
          if (r.end >= t1) s_last = k;  // (one request covers the tile's last token)
        }
      }
    }
    __syncthreads();
    // each token's request (a running maximum) and base (a running sum)
    int m[PG_PER], w[PG_PER];
    int mm = -1, ww = 0;
#pragma unroll
    for (int j = 0; j < PG_PER; ++j) {
      mm = max(mm, s_req[tid * PG_PER + j]);
      ww += s_add[tid * PG_PER + j];
      m[j] = mm;
      w[j] = ww;
    }
    const int lane = tid & 31, warp = tid >> 5;
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
    int em = __shfl_up_sync(0xffffffffu, im, 1), ew = iw - ww;
    if (lane == 0) em = -1;
    __syncthreads();
    int tot = 0;
#pragma unroll
    for (int q = 0; q < PG_THREADS / 32; ++q) {
      if (q < warp) {
        em = max(em, s_m[q]);
        ew += s_w[q];
      }
      tot += s_w[q];
    }
#pragma unroll
    for (int j = 0; j < PG_PER; ++j) {
      const long long t = t0 + tid * PG_PER + j;
      if (t >= t_end) break;
      long long slot = -1;
      int pos = -1, req = -1;
      if (t < n_tok) {
        req = max(em, m[j]);
        const Req r = load_req(a, (uint32_t)req);
        pos = (int)(r.ctx + (t - r.off));
        const uint32_t col = (uint32_t)pos / bs, in = (uint32_t)pos - col * bs;
        int32_t* entry = a.d_table + (long long)req * a.table_stride + col;
        int blk;
        if ((int)col >= r.have) {
          blk = a.d_free[n_free - 1 - (carry + ew + w[j] + ((int)col - r.have))];
          if (in == 0) *entry = blk;
        } else {
          blk = *entry;
        }
        slot = (long long)blk * bs + in;
      }
      a.d_slot[t] = slot;
      if (a.d_pos) a.d_pos[t] = pos;
      if (a.d_req) a.d_req[t] = req;
    }
    carry += tot + s_add[PG_TILE];
    if (t1 < n_tok) kf = s_last;
    __syncthreads();
  }
  // seq_len, n_free_out and the status: by the CTA that finishes last where
  // they may replace what the others still read, else by the first
  if (c.done) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const uint32_t d = atomicAdd(c.done, 1u);
      s_last = d == gridDim.x - 1;
      if (s_last) *c.done = 0;
    }
    __syncthreads();
    if (!s_last) return;
  } else if (blockIdx.x != 0) {
    return;
  }
  if (a.d_seq_len)
    for (uint32_t k = tid; k < a.n; k += PG_THREADS) {
      const long long ctx = a.d_ctx_len ? a.d_ctx_len[k] : 0;
      a.d_seq_len[k] = code == ST_OK ? ctx + (a.d_item_off[k + 1] - a.d_item_off[k]) : ctx;
    }
  if (tid == 0) {
    *a.d_n_free_out = code == ST_OK ? n_free - total : n_free;
    a.d_status[0] = code;
    a.d_status[1] = total;
    a.d_status[2] = n_tok;
    a.d_status[3] = s_bad == 0xffffffffu ? -1 : (long long)s_bad;
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
  return (len + c.block_size - 1) / c.block_size;
}

// One CTA takes a range of requests; as in k_paged_assign each CTA reads all
// of them once for its base and for the checks.
__global__ void __launch_bounds__(PG_THREADS) k_paged_release(ReleaseCall c) {
  __shared__ long long sh[PG_THREADS / 32], s_cnt[PG_THREADS];
  __shared__ unsigned s_bad, s_last;
  const int tid = threadIdx.x;
  const long long n_free = *c.n_free;
  const uint32_t k_begin = min(blockIdx.x * c.per, c.n), k_end = min(k_begin + c.per, c.n);
  if (tid == 0) s_bad = 0xffffffffu;
  __syncthreads();
  long long sum = 0, before = 0;
  for (uint32_t k = tid; k < c.n; k += PG_THREADS) {
    bool bad = false;
    const long long m = release_count(c, k, &bad);
    if (bad) atomicMin(&s_bad, k);
    sum += m;
    if (k < k_begin) before += m;
  }
  long long total, carry;
  block_excl_sum(sum, &total, sh);
  block_excl_sum(before, &carry, sh);
  int code = ST_OK;
  if (s_bad != 0xffffffffu || n_free < 0) code = TOK_EINVAL;
  else if ((unsigned long long)(n_free + total) > c.free_cap) code = TOK_EBUF;
  if (code == ST_OK) {
    for (uint32_t k0 = k_begin; k0 < k_end; k0 += PG_THREADS) {
      const uint32_t k = k0 + tid;
      bool bad = false;
      const long long m = k < k_end ? release_count(c, k, &bad) : 0;
      long long tile;
      block_excl_sum(m, &tile, sh);
      s_cnt[tid] = m;
      __syncthreads();
      long long base = n_free + carry;
      for (uint32_t i = 0; i < PG_THREADS && k0 + i < k_end; ++i) {
        const long long cnt = s_cnt[i];
        const int32_t* row = c.table + (long long)(k0 + i) * c.stride;
        for (long long j = tid; j < cnt; j += PG_THREADS) c.free_stack[base + j] = row[j];
        base += cnt;
      }
      carry += tile;
      __syncthreads();
    }
  }
  if (c.done) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const uint32_t d = atomicAdd(c.done, 1u);
      s_last = d == gridDim.x - 1;
      if (s_last) *c.done = 0;
    }
    __syncthreads();
    if (!s_last) return;
  } else if (blockIdx.x != 0) {
    return;
  }
  if (tid == 0) {
    *c.n_free_out = code == ST_OK ? n_free + total : n_free;
    c.status[0] = code;
    c.status[1] = total;
    c.status[2] = 0;
    c.status[3] = s_bad == 0xffffffffu ? -1 : (long long)s_bad;
  }
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
  const long long tiles = std::max<long long>(1, ((long long)a->cap + PG_TILE - 1) / PG_TILE);
  const long long ctas = std::min<long long>(tiles, 2ll * h->n_sms);
  c.span = (tiles + ctas - 1) / ctas * PG_TILE;
  const bool in_place = a->d_n_free_out == a->d_n_free || (a->d_seq_len && a->d_seq_len == a->d_ctx_len);
  c.done = in_place && ctas > 1 ? h->d_done : nullptr;
  k_paged_assign<<<(unsigned)ctas, PG_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(c);
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
  const uint32_t ctas = std::min<uint32_t>(n, 2u * (uint32_t)h->n_sms);
  c.per = (n + ctas - 1) / ctas;
  c.done = d_n_free_out == d_n_free && ctas > 1 ? h->d_done : nullptr;
  k_paged_release<<<ctas, PG_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(c);
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
