// The rows of a batch's ids (tok_embed) and the gradient of the weights
// (tok_embed_backward).
//
//   out[t] = scale * W[ids[t]],   dW[v] = scale * sum of dout[t] over ids[t] == v
//
// Both are bound by the bytes: the rows that ids name and what is written; the
// gradients that come in and the rows of dW.
//
// The gradient sorts the tokens by their ids (a stable radix sort in two passes
// of up to 11 bits, one where the ids have no more), so that a row's tokens lie
// side by side and are added in their order: sums in 32 bits, the same bits each
// time, without atomics on them.  The sorted tokens are cut into chunks of equal
// length; a warp adds a chunk's rows over 256 columns.  A run of equal ids inside
// a chunk is a finished row of dW; what a chunk's first and last run share with
// the neighbours goes to d_work, and a second kernel adds those parts in order.
//
// The rows that no token names are written as zeros by CTAs of their own, as bulk
// copies out of shared memory (131,057 tokens by 2,048 columns 185 us, with stores 201);
// which rows these are the first kernel of the sort says, with a bit for each.  A part
// of them beside the sort's kernels: 4,096 tokens 52 us instead of 56, but 1,000,000
// tokens 330 instead of 311.
#include "types.cuh"

namespace tokgb {
namespace {

constexpr uint32_t MOST_ROWS = 1u << 20, MOST_DIM = 1u << 20;
constexpr int EM_THREADS = 256;
constexpr int COLS = 256;            // columns of a warp's step: eight a lane
constexpr uint32_t ALL = 0xffffffffu;

// --- the rows ------------------------------------------------------------------

struct EmbedCall {
  const int32_t* ids;
  const long long* n_dev;
  uint32_t n, n_rows, dim, segs;  // segs: warps of a row
  const void* weight;
  long long weight_stride;
  void* out;
  long long out_stride;
  float scale;
};

constexpr int EM_COLS = 1024;        // columns of a warp, all of whose loads are under way at once

// N elements side by side: 8 or 16 bytes
template <class T, int N> struct Pack {
  uint32_t w[N * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N * sizeof(T) == 16) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x; w[1] = q.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (N * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return to_f32(reinterpret_cast<const T*>(w)[i]);
  }
  __device__ __forceinline__ void put(int i, float x) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x);
    else reinterpret_cast<T*>(w)[i] = from_f32<T>(x);
  }
};

// A lane takes N columns at a time, so that no access is of more than 16 bytes and a
// warp's lie side by side.  Bound by the bytes: 60,000 rows of 1,024 bf16 columns in 31
// us (5.5 TB/s), to 32 bits in 50 (5.9 TB/s; with eight columns a lane, in two accesses
// with gaps between the lanes, 66); 60,001 of 2,048 32-bit columns to bf16 in 82 (5.3).
template <class TI, class TO>
__global__ void __launch_bounds__(EM_THREADS) k_embed(EmbedCall c) {
  constexpr int N = sizeof(TI) == 4 || sizeof(TO) == 4 ? 4 : 8, U = EM_COLS / (32 * N);
  const uint32_t n = count_of(c.n_dev, c.n);
  const uint64_t unit = (uint64_t)blockIdx.x * (EM_THREADS / 32) + (threadIdx.x >> 5);
  const uint32_t t = (uint32_t)(unit / c.segs), seg = (uint32_t)(unit % c.segs), lane = threadIdx.x & 31u;
  if (t >= n) return;
  const int32_t id = c.ids[t];
  const bool there = (uint32_t)id < c.n_rows;
  const TI* row = static_cast<const TI*>(c.weight) + (there ? (long long)id * c.weight_stride : 0);
  TO* to = static_cast<TO*>(c.out) + (long long)t * c.out_stride;
  const uint32_t col = seg * EM_COLS + lane * N;
  Pack<TI, N> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (there && col + u * 32 * N < c.dim) x[u].load(row + col + u * 32 * N);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (col + u * 32 * N >= c.dim) break;
    Pack<TO, N> y;
#pragma unroll
    for (int i = 0; i < N; ++i) y.put(i, there ? x[u].get(i) * c.scale : 0.f);
    y.store(to + col + u * 32 * N);
  }
}

// rows that do not lie at 16-byte boundaries, or of a width that is no multiple of eight,
// an element at a time (60,000 rows of 1,031 bf16 columns in 58 us)
template <class TI, class TO>
__global__ void __launch_bounds__(EM_THREADS) k_embed_any(EmbedCall c) {
  const uint32_t n = count_of(c.n_dev, c.n);
  const uint64_t unit = (uint64_t)blockIdx.x * (EM_THREADS / 32) + (threadIdx.x >> 5);
  const uint32_t t = (uint32_t)(unit / c.segs), seg = (uint32_t)(unit % c.segs), lane = threadIdx.x & 31u;
  if (t >= n) return;
  const int32_t id = c.ids[t];
  const bool there = (uint32_t)id < c.n_rows;
  const TI* row = static_cast<const TI*>(c.weight) + (there ? (long long)id * c.weight_stride : 0);
  TO* to = static_cast<TO*>(c.out) + (long long)t * c.out_stride;
  const uint32_t col = seg * EM_COLS + lane;
#pragma unroll
  for (int u = 0; u < EM_COLS / COLS; ++u) {
    TI x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (there && col + u * COLS + i * 32 < c.dim) x[i] = row[col + u * COLS + i * 32];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + u * COLS + i * 32 < c.dim) to[col + u * COLS + i * 32] = from_f32<TO>(there ? to_f32(x[i]) * c.scale : 0.f);
  }
}

// --- the tokens sorted by their ids ----------------------------------------------

// Bound by latencies: 131,057 tokens over 100,257 rows in 6 us of counting and 13 and 12
// us of placing (64 CTAs; tiles of 4,096 tokens, 32 CTAs: 2 us more for both, of 1,024
// tokens: the gradient 242 us instead of 222), 4,096 tokens in 4, 9 and 8 (all of it by one
// CTA in its shared memory: the gradient 54 us instead of 55).
// A pass of the sort: every CTA takes a span of the tokens, in tiles.  A tile's
// warps take 256 tokens each, 32 at a time, so that a token's place among those
// of its digit is their order; counts of the digits by CTA (the table `counts`,
// a row of n_digits for each CTA) give the places of the spans.
constexpr int ST_THREADS = 512, ST_WARPS = ST_THREADS / 32, ST_PER = 4;
constexpr int ST_TILE = ST_THREADS * ST_PER;
constexpr int MOST_BITS = 11, MOST_DIGITS = 1 << MOST_BITS;
constexpr uint32_t MOST_SPANS = 152;

struct SortCall {
  const int32_t* ids;
  const long long* n_dev;
  uint32_t n, n_rows;
  uint32_t span;       // tokens of a CTA, a multiple of a tile
  uint32_t spans;      // CTAs
  uint32_t bits0, bits1;
  uint32_t* counts0;   // spans rows of 2^bits0
  uint32_t* counts1;   // spans rows of 2^bits1
  uint32_t* named;     // spans rows of a bit for each row of the weights: whether the span's ids name it; or nullptr
  uint2* half;         // (key, token) after the first pass of two
  uint2* sorted;       // and at the end
  uint32_t* n_runs;    // set to 0 for the sums
};

// an id's key: ids without a row come last
__device__ __forceinline__ uint32_t key_of(int32_t id, uint32_t n_rows) { return min((uint32_t)id, n_rows); }

// lanes with the same digit
template <int BITS_MOST>
__device__ __forceinline__ uint32_t alike(uint32_t d, bool in, uint32_t bits) {
  uint32_t m = __ballot_sync(ALL, in);
#pragma unroll
  for (int b = 0; b < BITS_MOST; ++b) {
    if (b >= (int)bits) break;
    const uint32_t one = __ballot_sync(ALL, d >> b & 1u);
    m &= d >> b & 1u ? one : ~one;
  }
  return in ? m : 0u;
}

// rows of the weights that get zeros, in blocks of 32
struct Empty {
  const uint32_t* named;
  uint32_t spans, n_rows, words;
  uint8_t* rows;
  long long stride;       // bytes
  unsigned long long row; // bytes
  int eights;             // rows are multiples of 16 bytes and lie at such
  uint32_t element;       // bytes
};

// block b's rows by all threads of the CTA.  Rows of whole 16-byte pieces are bulk
// copies of zeros in shared memory: a lane issues a row's, no thread waits for a store.
constexpr uint32_t ZEROS = 8192;
__device__ __forceinline__ void write_empty(const Empty& e, uint32_t b) {
  __shared__ uint32_t s_named;
  __shared__ __align__(128) uint4 s_zero[ZEROS / 16];
  if (threadIdx.x < 32) {
    uint32_t m = 0;
    for (uint32_t s = threadIdx.x; s < e.spans; s += 32) m |= e.named[(size_t)s * e.words + b];
    m = __reduce_or_sync(ALL, m);
    if (threadIdx.x == 0) s_named = m;
  }
  if (e.eights) {
    for (uint32_t i = threadIdx.x; i < ZEROS / 16; i += blockDim.x) s_zero[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  uint32_t left = ~s_named;
  const uint32_t rows = min(32u, e.n_rows - b * 32);
  if (rows < 32) left &= (1u << rows) - 1u;
  if (e.eights) {
    if (threadIdx.x < 32) {
      if (left >> threadIdx.x & 1u) {
        uint8_t* to = e.rows + (long long)(b * 32 + threadIdx.x) * e.stride;
        const uint32_t from = (uint32_t)__cvta_generic_to_shared(s_zero);
        for (uint32_t i = 0; i < (uint32_t)e.row; i += ZEROS)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + i), "r"(from),
                       "r"(min(ZEROS, (uint32_t)e.row - i)) : "memory");
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    return;
  }
  // each warp takes rows in turn
  for (uint32_t k = 0; left; left &= left - 1, ++k) {
    if (k % (blockDim.x >> 5) != threadIdx.x >> 5) continue;
    uint8_t* to = e.rows + (long long)(b * 32 + __ffs(left) - 1) * e.stride;
    const uint32_t lane = threadIdx.x & 31u;
    if (e.element == 4) {
      for (uint32_t i = lane; i < (uint32_t)(e.row / 4); i += 32) reinterpret_cast<uint32_t*>(to)[i] = 0;
    } else {
      for (uint32_t i = lane; i < (uint32_t)(e.row / 2); i += 32) reinterpret_cast<uint16_t*>(to)[i] = 0;
    }
  }
}

// counts of the first digit in each span, and the rows that it names; the second
// digit's counts are set to 0
__global__ void __launch_bounds__(ST_THREADS) k_sort_count(SortCall c) {
  extern __shared__ __align__(16) uint8_t mem[];
  uint32_t* s_count = reinterpret_cast<uint32_t*>(mem);
  uint32_t* s_named = s_count + (1u << c.bits0);
  let_next_start();
  if (blockIdx.x == 0 && threadIdx.x < 2) c.n_runs[threadIdx.x] = 0;
  const uint32_t n = count_of(c.n_dev, c.n), digits = 1u << c.bits0, words = (c.n_rows + 31) / 32, tid = threadIdx.x;
  for (uint32_t d = tid; d < digits + (c.named ? words : 0u); d += ST_THREADS) s_count[d] = 0;
  __syncthreads();
  const uint32_t begin = min(blockIdx.x * c.span, n), end = min(begin + c.span, n);
#pragma unroll 4
  for (uint32_t t = begin + tid; t < end; t += ST_THREADS) {
    const uint32_t k = key_of(c.ids[t], c.n_rows);
    atomicAdd(&s_count[k & (digits - 1)], 1u);
    if (c.named && k < c.n_rows) atomicOr(&s_named[k >> 5], 1u << (k & 31u));
  }
  __syncthreads();
  for (uint32_t d = tid; d < digits; d += ST_THREADS) c.counts0[(size_t)blockIdx.x * digits + d] = s_count[d];
  if (c.named)
    for (uint32_t w = tid; w < words; w += ST_THREADS) c.named[(size_t)blockIdx.x * words + w] = s_named[w];
  if (c.bits1)
    for (uint32_t d = tid; d < (1u << c.bits1); d += ST_THREADS) c.counts1[((size_t)blockIdx.x << c.bits1) + d] = 0;
}

template <int PASS>
__global__ void __launch_bounds__(ST_THREADS) k_sort_place(SortCall c) {
  extern __shared__ __align__(16) uint8_t mem[];
  wait_for_previous();
  let_next_start();
  const uint32_t bits = PASS == 0 ? c.bits0 : c.bits1, digits = 1u << bits, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  uint32_t* base = reinterpret_cast<uint32_t*>(mem);                    // [digits] where a digit's next token goes
  uint16_t* count = reinterpret_cast<uint16_t*>(base + digits);         // [ST_WARPS][digits]
  __shared__ uint32_t s_sum[ST_WARPS];
  const uint32_t n = count_of(c.n_dev, c.n);
  const uint32_t* counts = PASS == 0 ? c.counts0 : c.counts1;
  const uint32_t begin = min(blockIdx.x * c.span, n), end = min(begin + c.span, n);
  // places: all tokens of lower digits, then those of the digit in earlier spans
  uint32_t* total = reinterpret_cast<uint32_t*>(count);                 // [digits][2], before the counts of tiles
  for (uint32_t d = tid; d < digits; d += ST_THREADS) {
    uint32_t mine = 0, before = 0;
#pragma unroll 16
    for (uint32_t s = 0; s < c.spans; ++s) {
      const uint32_t m = counts[(size_t)s * digits + d];
      mine += m;
      before += s < blockIdx.x ? m : 0u;
    }
    total[2 * d] = mine;
    total[2 * d + 1] = before;
  }
  __syncthreads();
  // (up to four digits of a thread side by side)
  constexpr int PER = MOST_DIGITS / ST_THREADS;
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (tid * PER + i < digits) all += total[2 * (tid * PER + i)];
  uint32_t inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(ALL, inc, o);
    if (lane >= (uint32_t)o) inc += v;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  uint32_t lower = inc - all;
  for (uint32_t w = 0; w < warp; ++w) lower += s_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t d = tid * PER + i;
    if (d < digits) {
      base[d] = lower + total[2 * d + 1];
      lower += total[2 * d];
    }
  }
  for (uint32_t t0 = begin; t0 < end; t0 += ST_TILE) {
    __syncthreads();
    for (uint32_t i = tid; i < ST_WARPS * digits / 2; i += ST_THREADS) reinterpret_cast<uint32_t*>(count)[i] = 0;
    __syncthreads();
    uint32_t key[ST_PER], tok[ST_PER], rank[ST_PER];
    uint16_t* my = count + warp * digits;
#pragma unroll
    for (int j = 0; j < ST_PER; ++j) {
      const uint32_t t = t0 + warp * (ST_PER * 32) + j * 32 + lane;
      key[j] = tok[j] = 0;
      if (t < end) {
        if (PASS == 0) {
          key[j] = key_of(c.ids[t], c.n_rows);
          tok[j] = t;
        } else {
          const uint2 kt = c.half[t];
          key[j] = kt.x;
          tok[j] = kt.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < ST_PER; ++j) {
      const bool in = t0 + warp * (ST_PER * 32) + j * 32 + lane < end;
      const uint32_t d = PASS == 0 ? key[j] & (digits - 1) : key[j] >> c.bits0;
      const uint32_t same = alike<MOST_BITS>(d, in, bits), below = __popc(same & ((1u << lane) - 1u));
      uint32_t at = in ? my[d] : 0;
      __syncwarp();
      if (in && below == 0) my[d] = (uint16_t)(at + __popc(same));
      __syncwarp();
      rank[j] = at + below;
    }
    __syncthreads();
    // a digit's counts by warp become places, its base moves on
    for (uint32_t d = tid; d < digits; d += ST_THREADS) {
      uint32_t run = 0;
#pragma unroll
      for (int w = 0; w < ST_WARPS; ++w) {
        const uint32_t m = count[w * digits + d];
        count[w * digits + d] = (uint16_t)run;
        run += m;
      }
      // (kept in the place of a 17th warp's: the base without this tile's)
      base[d] += run;
      count[ST_WARPS * digits + d] = (uint16_t)run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ST_PER; ++j) {
      const bool in = t0 + warp * (ST_PER * 32) + j * 32 + lane < end;
      const uint32_t d = PASS == 0 ? key[j] & (digits - 1) : key[j] >> c.bits0;
      uint32_t to = 0;
      if (in) {
        to = base[d] - count[ST_WARPS * digits + d] + count[warp * digits + d] + rank[j];
        const uint2 kt = make_uint2(key[j], tok[j]);
        if (PASS == 0 && c.bits1) c.half[to] = kt;
        else c.sorted[to] = kt;
      }
      if (PASS == 0 && c.bits1) {
        // the next pass's counts; equal keys of a warp lie side by side (but where a
        // span ends between them)
        const uint32_t slot = in ? ((to / c.span) << c.bits1) + (key[j] >> c.bits0) : ALL;
        const uint32_t same = __match_any_sync(ALL, slot);
        if (in && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&c.counts1[slot], (uint32_t)__popc(same));
      }
    }
  }
}

// --- the rows' sums ----------------------------------------------------------------

struct SumCall {
  const uint2* sorted;
  const long long* n_dev;
  uint32_t n, n_rows, dim, segs;  // segs: warps of a row
  uint32_t chunk;                 // sorted tokens of a warp, a multiple of 32
  uint32_t chunks;
  float scale;
  const void* grad_out;
  long long grad_out_stride;
  void* grad_weight;
  long long grad_weight_stride;
  float* parts;                   // [chunks][2][dim rounded up to COLS]: first and last run of a chunk
  uint32_t* runs;                 // [chunks]: chunks in which a run begins that others end; from the end, long ones
  uint32_t* n_runs;               // how many of both
  uint32_t sum_ctas;              // CTAs that add; the others write rows without tokens
};

// a lane's eight columns: side by side (VEC), or 32 apart
template <bool VEC> __device__ __forceinline__ uint32_t column(uint32_t seg, uint32_t lane, int i) {
  return seg * COLS + (VEC ? lane * 8 + i : lane + i * 32);
}

template <class TG, class TW, bool VEC>
__device__ __forceinline__ void write_row(const SumCall& c, uint32_t v, uint32_t seg, uint32_t lane, const float* s, bool add) {
  TW* to = static_cast<TW*>(c.grad_weight) + (long long)v * c.grad_weight_stride;
  if (VEC) {
    const uint32_t col = column<true>(seg, lane, 0);
    if (col >= c.dim) return;
    Eight<TW> y;
    if (add) {
      Eight<TW> old;
      old.load(to + col);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y.put_pair(i, fmaf(s[2 * i], c.scale, old.get(2 * i)), fmaf(s[2 * i + 1], c.scale, old.get(2 * i + 1)));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y.put_pair(i, s[2 * i] * c.scale, s[2 * i + 1] * c.scale);
    }
    y.store(to + col);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t col = column<false>(seg, lane, i);
      if (col < c.dim) to[col] = from_f32<TW>(add ? fmaf(s[i], c.scale, to_f32(to[col])) : s[i] * c.scale);
    }
  }
}

__device__ __forceinline__ float* part_of(const SumCall& c, uint32_t chunk, int last, uint32_t seg, uint32_t lane) {
  return c.parts + (((size_t)chunk * 2 + last) * c.segs + seg) * COLS + lane * 8;
}
__device__ __forceinline__ void put_part(float* p, const float* s) {
  reinterpret_cast<float4*>(p)[0] = make_float4(s[0], s[1], s[2], s[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// Bound by the bytes: 131,057 rows of 2,048 bf16 columns in, 100,257 rows out, in 145 us
// (6.5 TB/s); chunks of 32 tokens while a warp's columns and chunks are 8,192 or fewer,
// then longer ones, up to 128: parts that go to d_work are two rows of 32 bits a chunk.
constexpr int AHEAD = 8;  // rows whose loads are under way
constexpr uint32_t LONG_RUN = 8;  // chunks of a run that a whole CTA adds

template <class TG, class TW, bool VEC, bool ADD>
__global__ void __launch_bounds__(EM_THREADS) k_embed_sum(SumCall c, Empty empty) {
  wait_for_previous();
  let_next_start();
  if (blockIdx.x >= c.sum_ctas) {
    write_empty(empty, blockIdx.x - c.sum_ctas);
    return;
  }
  const uint32_t n = count_of(c.n_dev, c.n), lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint64_t unit = (uint64_t)blockIdx.x * (EM_THREADS / 32) + warp;
  const uint32_t chunk = (uint32_t)(unit / c.segs), seg = (uint32_t)(unit % c.segs);
  const uint32_t begin = chunk * c.chunk, end = min(begin + c.chunk, n);
  if (chunk >= c.chunks || begin >= n) return;
  uint32_t run_key = begin ? c.sorted[begin - 1].x : ALL;  // the key of the tokens before
  bool first = true;                                       // the run began before the chunk
  const uint32_t next_key = end < n ? c.sorted[end].x : ALL;
  float s[8] = {};
  for (uint32_t b = begin; b < end; b += 32) {
    const uint2 kt = b + lane < end ? c.sorted[b + lane] : make_uint2(ALL, 0);
    const uint32_t m = min(32u, end - b);
    for (uint32_t j0 = 0; j0 < m; j0 += AHEAD) {
      Eight<TG> x[AHEAD];
      float xs[VEC ? 1 : AHEAD][8];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const uint32_t t = __shfl_sync(ALL, kt.y, (j0 + j) & 31u), k = __shfl_sync(ALL, kt.x, (j0 + j) & 31u);
        const bool in = j0 + j < m && k < c.n_rows;
        const TG* row = static_cast<const TG*>(c.grad_out) + (long long)t * c.grad_out_stride;
        if (VEC) {
          const uint32_t col = column<true>(seg, lane, 0);
          if (in && col < c.dim) x[j].load_once(row + col);
          else x[j].zero();
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t col = column<false>(seg, lane, i);
            xs[VEC ? 0 : j][i] = in && col < c.dim ? to_f32(row[col]) : 0.f;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= m) break;
        const uint32_t k = __shfl_sync(ALL, kt.x, (j0 + j) & 31u);
        if (k != run_key) {  // (the same in all lanes)
          if (run_key != ALL && run_key < c.n_rows) {
            if (!first) write_row<TG, TW, VEC>(c, run_key, seg, lane, s, ADD);
            else if (b + j0 + j > begin) put_part(part_of(c, chunk, 0, seg, lane), s);
          }
          first = false;
          run_key = k;
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += VEC ? x[j].get(i) : xs[VEC ? 0 : j][i];
      }
    }
  }
  if (run_key >= c.n_rows) return;
  if (first) {
    put_part(part_of(c, chunk, 0, seg, lane), s);
  } else if (next_key == run_key) {
    put_part(part_of(c, chunk, 1, seg, lane), s);
    if (seg == 0 && lane == 0) {
      const uint64_t far = (uint64_t)begin + (uint64_t)c.chunk * LONG_RUN;
      if (far < n && c.sorted[far].x == run_key) c.runs[c.chunks - 1 - atomicAdd(c.n_runs + 1, 1u)] = chunk;
      else c.runs[atomicAdd(c.n_runs, 1u)] = chunk;
    }
  } else {
    write_row<TG, TW, VEC>(c, run_key, seg, lane, s, ADD);
  }
}

// Runs that reach over chunks, as the chunks in which they begin (in any order: each
// is a row of its own).  A warp adds a run's parts over 256 columns in order; of a
// long run each warp of a CTA takes a share, and the shares are added in order.
template <class TG, class TW, bool VEC, bool ADD>
__global__ void __launch_bounds__(EM_THREADS) k_embed_join(SumCall c) {
  __shared__ __align__(16) float s_part[EM_THREADS / 32][COLS];
  wait_for_previous();
  constexpr uint32_t WARPS = EM_THREADS / 32;
  const uint32_t n = count_of(c.n_dev, c.n), lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  // parts of the run that begins in a chunk: its own, and those of the chunks after it that begin with the key
  auto parts_of = [&](uint32_t chunk, uint32_t key) {
    uint32_t m = 1;
    for (uint64_t k0 = chunk + 1;; k0 += 32) {
      const uint64_t at = (k0 + lane) * c.chunk;
      const uint32_t same = __ballot_sync(ALL, at < n && c.sorted[at].x == key);
      m += same == ALL ? 32 : __ffs(~same) - 1;
      if (same != ALL) return m;
    }
  };
  auto sum = [&](uint32_t chunk, uint32_t seg, uint32_t from, uint32_t to, float* s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll 4
    for (uint32_t i = from; i < to; ++i) {
      const float4* p = reinterpret_cast<const float4*>(part_of(c, chunk + i, i == 0, seg, lane));
      const float4 a = p[0], b = p[1];
      s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
      s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
    }
  };
  float s[8];
  const uint64_t short_items = (uint64_t)c.n_runs[0] * c.segs, long_items = (uint64_t)c.n_runs[1] * c.segs;
  for (uint64_t item = (uint64_t)blockIdx.x * WARPS + warp; item < short_items; item += (uint64_t)gridDim.x * WARPS) {
    const uint32_t chunk = c.runs[item / c.segs], seg = (uint32_t)(item % c.segs);
    const uint32_t key = c.sorted[(uint64_t)(chunk + 1) * c.chunk].x;
    sum(chunk, seg, 0, parts_of(chunk, key), s);
    write_row<TG, TW, VEC>(c, key, seg, lane, s, ADD);
  }
  for (uint64_t item = blockIdx.x; item < long_items; item += gridDim.x) {
    const uint32_t chunk = c.runs[c.chunks - 1 - item / c.segs], seg = (uint32_t)(item % c.segs);
    const uint32_t key = c.sorted[(uint64_t)(chunk + 1) * c.chunk].x;
    const uint32_t m = parts_of(chunk, key), per = (m + WARPS - 1) / WARPS;
    sum(chunk, seg, min(warp * per, m), min((warp + 1) * per, m), s);
    put_part(&s_part[warp][lane * 8], s);
    __syncthreads();
    if (warp == 0) {
      for (uint32_t w = 1; w < WARPS; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += s_part[w][lane * 8 + i];
      write_row<TG, TW, VEC>(c, key, seg, lane, s, ADD);
    }
    __syncthreads();
  }
}

// --- the host's side -----------------------------------------------------------------

constexpr uint64_t MOST_SHORT = 8192;   // chunks times warps of a row, with chunks below 128 tokens

uint64_t up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

struct Plan {
  uint32_t bits0, bits1, span, spans, chunk, chunks, segs;
  uint64_t counts0, counts1, named, half, sorted, parts, runs, bytes;  // places in d_work
};

Plan plan_of(uint64_t n, uint32_t n_rows, uint32_t dim) {
  Plan p{};
  uint32_t bits = 1;
  while (bits < 21 && (n_rows >> bits)) ++bits;  // keys are 0 .. n_rows
  p.bits0 = bits <= (uint32_t)MOST_BITS ? bits : (bits + 1) / 2;
  p.bits1 = bits - p.bits0;
  const uint64_t tiles = std::max<uint64_t>(1, (n + ST_TILE - 1) / ST_TILE);
  const uint64_t per = (tiles + MOST_SPANS - 1) / MOST_SPANS;
  p.span = (uint32_t)(per * ST_TILE);
  p.spans = (uint32_t)((tiles + per - 1) / per);
  p.segs = (dim + COLS - 1) / COLS;
  p.chunk = 32;
  while (p.chunk < 128 && n / p.chunk * p.segs > MOST_SHORT) p.chunk *= 2;
  p.chunks = (uint32_t)((n + p.chunk - 1) / p.chunk);
  // room for fewer ids, too, of which there may be more spans or chunks
  const uint64_t spans = std::min<uint64_t>(tiles, MOST_SPANS);
  const uint64_t chunks = std::min<uint64_t>((n + 31) / 32, std::max<uint64_t>(MOST_SHORT / p.segs + 1, (n + 127) / 128));
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) { const uint64_t here = at; at = up(at + bytes, 256); return here; };
  p.counts0 = take(spans * 4 << p.bits0);
  p.counts1 = take(p.bits1 ? spans * 4 << p.bits1 : 0);
  p.named = take(spans * ((n_rows + 31) / 32) * 4);
  p.half = take(p.bits1 ? n * 8 : 0);
  p.sorted = take(n * 8);
  p.parts = take(chunks * 2 * p.segs * COLS * 4);
  p.runs = take(chunks * 4 + 8);
  p.bytes = at;
  return p;
}

bool sizes_ok(uint64_t n, uint32_t n_rows, uint32_t dim) {
  return n < (1ull << 31) && n_rows && n_rows <= MOST_ROWS && dim && dim <= MOST_DIM;
}

int finish(tok_handle* h, unsigned launches) {
  h->launches += launches;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
}

// f(T{}) for an element type
template <class F> void with_type(int dtype, F f) {
  if (dtype == TOK_F32) f(float{});
  else if (dtype == TOK_F16) f(__half{});
  else f(__nv_bfloat16{});
}

// whether rows can be taken eight elements at a time
bool in_eights(const void* p, int64_t stride, int dtype, uint32_t dim) {
  return lies_at(p, 16) && (uint64_t)stride * element_size(dtype) % 16 == 0 && dim % 8 == 0;
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_embed(tok_handle* h, const tok_embed_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->n == 0) return TOK_OK;
  if (!a || !a->d_ids || !a->d_weight || !a->d_out) return fail(h, TOK_EINVAL, "embed: a buffer is NULL");
  if (!element_size(a->weight_dtype) || !element_size(a->out_dtype)) return fail(h, TOK_EINVAL, "embed: unknown type");
  if (!sizes_ok(a->n, a->n_rows, a->dim) || a->weight_stride < (int64_t)a->dim || a->out_stride < (int64_t)a->dim)
    return fail(h, TOK_EINVAL, "embed: n, n_rows, dim or a stride is out of range");
  if (!lies_at(a->d_ids, 4) || !lies_at(a->d_n, 8) || !lies_at(a->d_weight, element_size(a->weight_dtype)) ||
      !lies_at(a->d_out, element_size(a->out_dtype)))
    return fail(h, TOK_EINVAL, "embed: an array does not lie at a multiple of its type's size");
  DeviceGuard g(h->dev);
  EmbedCall c{a->d_ids, reinterpret_cast<const long long*>(a->d_n), (uint32_t)a->n, a->n_rows, a->dim,
              (a->dim + EM_COLS - 1) / EM_COLS, a->d_weight, a->weight_stride, a->d_out, a->out_stride, a->scale};
  const uint64_t ctas = (a->n * c.segs + EM_THREADS / 32 - 1) / (EM_THREADS / 32);
  if (ctas > 0x7fffffffull) return fail(h, TOK_EINVAL, "embed: n times dim is out of range");
  const bool eights = in_eights(a->d_weight, a->weight_stride, a->weight_dtype, a->dim) &&
                      in_eights(a->d_out, a->out_stride, a->out_dtype, a->dim);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  with_type(a->weight_dtype, [&](auto ti) {
    with_type(a->out_dtype, [&](auto to) {
      if (eights) k_embed<decltype(ti), decltype(to)><<<(unsigned)ctas, EM_THREADS, 0, s>>>(c);
      else k_embed_any<decltype(ti), decltype(to)><<<(unsigned)ctas, EM_THREADS, 0, s>>>(c);
    });
  });
  return finish(h, 1);
} catch (...) {
  return TOK_ENOMEM;
}

uint64_t tok_embed_work_bytes(uint64_t n, uint32_t n_rows, uint32_t dim) {
  return sizes_ok(n, n_rows, dim) ? plan_of(n, n_rows, dim).bytes : 0;
}

int tok_embed_backward(tok_handle* h, const tok_embed_grad_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->n == 0 && a->accumulate) return TOK_OK;
  if (!a || !a->d_grad_weight || (a->n && (!a->d_ids || !a->d_grad_out)))
    return fail(h, TOK_EINVAL, "embed gradient: a buffer is NULL");
  if (!element_size(a->grad_weight_dtype) || !element_size(a->grad_out_dtype))
    return fail(h, TOK_EINVAL, "embed gradient: unknown type");
  if (!sizes_ok(a->n, a->n_rows, a->dim) || a->grad_weight_stride < (int64_t)a->dim ||
      (a->n && a->grad_out_stride < (int64_t)a->dim))
    return fail(h, TOK_EINVAL, "embed gradient: n, n_rows, dim or a stride is out of range");
  if (!lies_at(a->d_ids, 4) || !lies_at(a->d_n, 8) || !lies_at(a->d_grad_weight, element_size(a->grad_weight_dtype)) ||
      !lies_at(a->d_grad_out, element_size(a->grad_out_dtype)))
    return fail(h, TOK_EINVAL, "embed gradient: an array does not lie at a multiple of its type's size");
  const Plan p = plan_of(a->n, a->n_rows, a->dim);
  if (!a->d_work || !lies_at(a->d_work, 256) || a->work_bytes < p.bytes)
    return fail(h, TOK_EINVAL, "embed gradient: d_work is NULL, not at a multiple of 256 bytes or too small");
  DeviceGuard g(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* work = static_cast<uint8_t*>(a->d_work);
  const long long* n_dev = reinterpret_cast<const long long*>(a->d_n);
  SortCall sc{a->d_ids, n_dev, (uint32_t)a->n, a->n_rows, p.span, p.spans, p.bits0, p.bits1,
              reinterpret_cast<uint32_t*>(work + p.counts0), reinterpret_cast<uint32_t*>(work + p.counts1),
              a->accumulate ? nullptr : reinterpret_cast<uint32_t*>(work + p.named),
              reinterpret_cast<uint2*>(work + p.half), reinterpret_cast<uint2*>(work + p.sorted),
              reinterpret_cast<uint32_t*>(work + p.runs)};
  SumCall c{sc.sorted, n_dev, (uint32_t)a->n, a->n_rows, a->dim, p.segs, p.chunk, p.chunks, a->scale, a->d_grad_out,
            a->grad_out_stride, a->d_grad_weight, a->grad_weight_stride, reinterpret_cast<float*>(work + p.parts), sc.n_runs + 2, sc.n_runs, 0};
  constexpr uint64_t WARPS = EM_THREADS / 32;
  if ((uint64_t)p.chunks * p.segs > 0x7fffffffull / 2) return fail(h, TOK_EINVAL, "embed gradient: n times dim is out of range");
  c.sum_ctas = (uint32_t)(((uint64_t)p.chunks * p.segs + WARPS - 1) / WARPS);
  const uint64_t join_ctas = p.chunks > 1 ? std::min<uint64_t>((uint64_t)(p.chunks - 1) * p.segs, 6ull * (uint32_t)h->n_sms) : 0;
  const size_t size = element_size(a->grad_weight_dtype);
  const bool eights = in_eights(a->d_grad_out, a->grad_out_stride, a->grad_out_dtype, a->dim) &&
                      in_eights(a->d_grad_weight, a->grad_weight_stride, a->grad_weight_dtype, a->dim);
  const Empty em{sc.named, p.spans, a->n_rows, (a->n_rows + 31) / 32, static_cast<uint8_t*>(a->d_grad_weight),
                 (long long)(a->grad_weight_stride * (int64_t)size), (unsigned long long)a->dim * size,
                 in_eights(a->d_grad_weight, a->grad_weight_stride, a->grad_weight_dtype, a->dim), (uint32_t)size};
  const uint32_t m = a->accumulate ? 0 : em.words;   // blocks of 32 rows
  cudaError_t e = allow_all<k_sort_count>(h->dev);
  if (e == cudaSuccess) e = allow_all<k_sort_place<0>>(h->dev);
  if (e == cudaSuccess) e = allow_all<k_sort_place<1>>(h->dev);
  if (e != cudaSuccess) return cuda_fail(h, e, "shared memory of a kernel");
  unsigned launches = 1;
  const size_t bitmap = sc.named ? (size_t)em.words * 4 : 0;
  auto room = [](uint32_t bits) { return ((size_t)4 << bits) + ((size_t)2 * (ST_WARPS + 1) << bits); };
  k_sort_count<<<p.spans, ST_THREADS, ((size_t)4 << p.bits0) + bitmap, s>>>(sc);
  launch_behind(k_sort_place<0>, p.spans, ST_THREADS, room(p.bits0), s, sc);
  ++launches;
  if (p.bits1) {
    launch_behind(k_sort_place<1>, p.spans, ST_THREADS, room(p.bits1), s, sc);
    ++launches;
  }
  with_type(a->grad_out_dtype, [&](auto tg) {
    with_type(a->grad_weight_dtype, [&](auto tw) {
      using TG = decltype(tg);
      using TW = decltype(tw);
      auto both = [&](auto vec, auto add) {
        if (c.sum_ctas + m) {
          launch_behind(k_embed_sum<TG, TW, vec.value, add.value>, c.sum_ctas + m, EM_THREADS, 0, s, c, em);
          ++launches;
        }
        if (join_ctas) {
          launch_behind(k_embed_join<TG, TW, vec.value, add.value>, (unsigned)join_ctas, EM_THREADS, 0, s, c);
          ++launches;
        }
      };
      if (eights && a->accumulate) both(std::true_type{}, std::true_type{});
      else if (eights) both(std::true_type{}, std::false_type{});
      else if (a->accumulate) both(std::false_type{}, std::true_type{});
      else both(std::false_type{}, std::false_type{});
    });
  });
  return finish(h, launches);
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
