// New tokens' keys and values into the paged cache (tok_paged_store) and the
// attention of one new token of each request over it (tok_paged_attend).
//
// For query head j of request k, over the tokens p that it may read,
//   s(p) = scale * (q . key(p)),  out = sum exp(s(p)) value(p) / sum exp(s(p)),  lse = log sum exp(s(p))
// Bound by the keys' and values' bytes: 2 * 2 * head_dim bytes for each token and
// key head, 4 * head_dim * group operations on them (group: query heads of a key head).
//
// Tokens are taken in tiles of 64 of one request and key head.  All tiles of all
// requests form one row; each CTA (as many as the SMs hold at once) takes an equal
// piece of it, so that long and short requests share the GPU evenly.  A warp takes
// 16 tokens at a time, which it copies into shared memory of its own (cp.async, two
// steps ahead, five for widths of 64), so that warps never wait for one another; it keeps
// the maximum, the sum and the output of its tokens, and the CTA joins its warps'
// when the piece of a request and head ends.  What a CTA has only a part of goes to
// d_work and a second kernel joins the parts, in order: the same bits each time.
// A piece's start costs about as much as two of its tiles (its first tokens' places
// and copies, the queries, the join of the warps): pieces are cut by that measure.
//
// The products are on mma.sync (m16n8k16): 16 tokens by 8 query heads, so that
// groups of eight fill it; S^T = K Q^T and O^T = V^T P^T both read the cache's rows
// as they lie (ldmatrix, transposed for the values), and P^T comes from S^T by
// movmatrix.  The matrix work is a small part of the time that the bytes take: at
// group 8 and width 128, 32 instructions (bf16; f16: 24, and 32 sums) of 2,048
// multiply-adds for 8 KB.
//
// Measured on a GB300 (6.7 TB/s of plain copying): 256 requests of up to 4,801 tokens, 8
// key heads of 128, group 8, in 397 us (6.4 TB/s); 64 requests of 0 to 16,381 tokens in 82
// us (5.4); one of 32,749 in 35 us (3.8): of these 2 are the way to the first copies, 24
// the bytes, 4 the warps' and CTAs' joins, the rest the second kernel, which the first lets
// start early.  Without the starts' share in the pieces the 64 requests took 133 us.
#include "types.cuh"

#include <cfloat>

namespace tokgb {
namespace {

constexpr uint32_t ALL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int STEP = 16;                // tokens of a warp's step
constexpr int TILE = STEP * WARPS;      // tokens of a CTA's step, the unit that pieces are cut at
constexpr uint32_t START = 2;           // what the start of a request and head counts, in tiles
constexpr uint32_t MOST_REQUESTS = 1u << 20, MOST_GROUP = 64;
// A weight's exponent is relative to a reference that is replaced once a score lies
// more than this above it (in powers of 2): weights stay below 2^8.
constexpr float SLACK = 8.f;

// Kernels are made for widths of 64, 128 and 256; others take the next one's, with zeros
// in shared memory (256 requests of up to 4,000 tokens, 8 key heads of 80: 317 us, and 331
// with kernels for 96 and 192, too: what bounds it is that 160 bytes of a token lie in
// three or four of the 64-byte pieces that DRAM is read in).
template <int D> struct Shape {
  static constexpr int ROW = D * 2;                    // bytes of a token in shared memory
  static constexpr int STAGE = 2 * STEP * ROW;         // keys and values of a step
  static constexpr int DEPTH = D == 64 ? 6 : 3;        // steps in shared memory
  static constexpr int WARP_BYTES = DEPTH * STAGE;     // 24 KB for widths of 64 and 128, 48 KB for 256
  static constexpr size_t BYTES = (size_t)WARPS * WARP_BYTES;
  static constexpr int CTAS = D == 256 ? 1 : 2;        // per SM
};

struct AttendCall {
  const void* k;
  const void* v;
  long long block_stride, token_stride, head_stride;
  uint32_t n_blocks, block_size, kv_heads, head_dim;
  const void* q;
  long long q_stride, q_head_stride;
  void* out;
  long long out_stride, out_head_stride;
  float* lse;
  uint32_t n, heads, group, parts;  // parts: CTAs' shares of a group (gt query heads each)
  uint32_t gt;
  float scale_log2;
  uint32_t window;
  const int32_t* table;
  long long table_stride;
  long long most_len;               // tokens that a row of the table has room for
  const long long* seq_len;
  uint4* splits;                    // [ctas]: what a CTA began and others end: request, key head and share, last CTA, 1
  float* sums;                      // [ctas][2][16][2]: reference and sum of a part
  float* outs;                      // [ctas][2][16][D]
  uint32_t ctas;
};

struct Span { long long begin, end; };  // tokens that a request's query reads
__device__ __forceinline__ Span span_of(const AttendCall& c, uint32_t r) {
  long long m = c.seq_len[r];
  m = m < 0 ? 0 : m > c.most_len ? c.most_len : m;
  return Span{c.window && m > (long long)c.window ? m - (long long)c.window : 0, m};
}
__device__ __forceinline__ uint32_t tiles_of(const Span& s) { return (uint32_t)((s.end - s.begin + TILE - 1) / TILE); }
// of all its key heads and shares
__device__ __forceinline__ unsigned long long cost_of(const AttendCall& c, const Span& s) {
  return s.end > s.begin ? (unsigned long long)(tiles_of(s) + START) * (c.kv_heads * c.parts) : 0ull;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The products of a type, and a weight as PARTS numbers of the type: three of bf16 add up
// to its 24 bits.  Weights are taken UNIT times.  bf16 holds values near the 32-bit numbers'
// end: with weights of 2^-32 at most, sums over 2^31 tokens stay finite.  f16 holds no
// number below 2^-24: there the largest weight lies near the type's upper end, and what
// rounding to f16 left is taken 2^11 times, in sums of its own.  Together they are off by at
// most 2^-23 of the weight or 2^-43 of the largest one.  (As two f16 numbers in one sum,
// without either, weights were off by 2^-25 of the largest one: a token that took nearly the
// whole weight hid all others.)
template <class T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
  static constexpr int PARTS = 3;
  static constexpr float UNIT = 0x1p-40f;   // (SLACK: 2^-32 at most)
  static __device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // two weights' parts, x's in the lower halves; each is the rest's upper half
  static __device__ __forceinline__ void split(float x, float y, uint32_t* part) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      part[p] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
      x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    }
  }
  // c += a times the weights whose parts are w[.][0] and w[.][1]
  static __device__ __forceinline__ void add(float* c, const uint32_t* a, const uint32_t (*w)[2]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) mma(c, a, w[p][0], w[p][1]);
  }
};
template <> struct Mma<__half> {
  static constexpr int PARTS = 2;
  static constexpr float UNIT = 0x1p7f;     // (2^15 at most)
  static __device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void split(float x, float y, uint32_t* part) {
    part[0] = pack(x, y);
    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&part[0]));
    part[1] = pack((x - back.x) * 2048.f, (y - back.y) * 2048.f);
  }
  static __device__ __forceinline__ void add(float* c, const uint32_t* a, const uint32_t (*w)[2]) {
    float rest[4] = {0.f, 0.f, 0.f, 0.f};
    mma(c, a, w[0][0], w[0][1]);
    mma(rest, a, w[1][0], w[1][1]);
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(rest[e], 1.f / 2048.f, c[e]);
  }
};

__device__ __forceinline__ void ldmatrix(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16 bytes, or zeros where there is nothing to read
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// The steps of one warp over the tokens begin .. end of a request and key head:
// where the tokens' rows are, and their copies into the warp's shared memory.
template <class T, int D> struct Loader {
  static constexpr int CPR = D / 8;            // copies of a row
  static constexpr int RPI = 32 / CPR;         // rows that the warp's lanes copy at once
  const AttendCall& c;
  const int32_t* row;                          // of the table
  long long end;
  long long head_off;
  uint32_t slot;                               // the warp's shared memory

  // the place of token p, in elements; -1: nothing to read
  __device__ __forceinline__ long long place(long long p) const {
    if (p >= end) return -1;
    const uint32_t b = (uint32_t)p / c.block_size, in = (uint32_t)p - b * c.block_size;  // (rows hold fewer than 2^31 tokens)
    const int32_t id = row[b];
    if ((uint32_t)id >= c.n_blocks) return -1;
    return (long long)id * c.block_stride + (long long)in * c.token_stride + head_off;
  }
  // copies of the 16 tokens whose places are at (lane i: token i) into a stage
  __device__ __forceinline__ void issue(uint32_t stage, long long at) const {
    const uint32_t lane = threadIdx.x & 31u, chunk = lane % CPR;
    const uint32_t to = slot + stage * Shape<D>::STAGE;
#pragma unroll
    for (int i = 0; i < STEP / RPI; ++i) {
      const uint32_t r = i * RPI + lane / CPR;
      const long long from = __shfl_sync(ALL, at, r);
      const bool there = from >= 0 && chunk * 8 < c.head_dim;
      const long long off = there ? from + chunk * 8 : 0;
      const uint32_t dst = to + r * Shape<D>::ROW + (chunk ^ (r & 7u)) * 16;
      copy16(dst, static_cast<const T*>(c.k) + off, there);
      copy16(dst + STEP * Shape<D>::ROW, static_cast<const T*>(c.v) + off, there);
    }
  }
};

// a + v f for a part v of an output, however small f is: an infinity or a NaN stays what it is
__device__ __forceinline__ float plus(float a, float v, float f) { return fabsf(v) < INFINITY ? fmaf(v, f, a) : a + v; }

// Where the values hold an infinity, the products of matrices give a NaN: weights and their
// rests may be 0, or of both signs.  Every weight is above 0, so what such a column's
// output is follows from the values alone: the warp passes over those of its tokens (at p,
// a step's 16 by the lanes) once more and sets that column for all of its query heads.
template <class T, int D>
__device__ __forceinline__ void set_infinities(const Loader<T, D>& in, long long p, uint32_t steps, float* out, uint32_t pitch,
                                               const float* tot, uint32_t heads) {
  constexpr uint32_t INF = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
  const uint32_t lane = threadIdx.x & 31u;
  uint32_t seen = 0;   // of each of the lane's columns, two side by side in every 64: 1 for inf, 2 for -inf, both for a NaN
  for (uint32_t step = 0; step < steps; ++step, p += TILE) {
    const long long at = in.place(p);
    for (int r = 0; r < STEP; ++r) {
      const long long from = __shfl_sync(ALL, at, r);
      if (from < 0) continue;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const uint32_t d = k * 64 + lane * 2;
        if (d >= in.c.head_dim) continue;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const T*>(in.c.v) + from + d);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u = e ? w >> 16 : w & 0xffffu;
          if ((u & INF) == INF) seen |= ((u & 0x7fffu) != INF ? 3u : u >> 15 ? 2u : 1u) << (4 * k + 2 * e);
        }
      }
    }
  }
  for (int c = 0; c < D / 32; ++c) {
    const uint32_t what = seen >> (2 * c) & 3u;
    if (!what) continue;
    for (uint32_t j = 0; j < heads; ++j)
      if (tot[j] == tot[j])   // (a NaN among the scores is a NaN everywhere)
        out[j * pitch + c / 2 * 64 + lane * 2 + (c & 1)] = what == 3 ? NAN : what == 2 ? -INFINITY : INFINITY;
  }
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(THREADS, Shape<D>::CTAS) k_attend(AttendCall c) {
  extern __shared__ __align__(128) uint8_t mem[];
  __shared__ unsigned long long s_sum[WARPS], s_base;
  __shared__ uint32_t s_req;
  __shared__ float s_ref[WARPS][16], s_tot[WARPS][16];
  using S = Shape<D>;
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g = lane >> 2, t = lane & 3u;

  let_next_start();
  // the cost of all requests, and the request in which this CTA's piece begins
  const uint32_t per = (c.n + THREADS - 1) / THREADS, r0 = min(tid * per, c.n), r1 = min(r0 + per, c.n);
  unsigned long long mine = 0;
  for (uint32_t r = r0; r < r1; ++r) mine += cost_of(c, span_of(c, r));
  unsigned long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(ALL, inc, o);
    if (lane >= (uint32_t)o) inc += x;
  }
  if (lane == 31) s_sum[warp] = inc;
  if (tid == 0) s_req = c.n;
  __syncthreads();
  unsigned long long total = 0, at = inc - mine;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < (int)warp) at += s_sum[w];
    total += s_sum[w];
  }
  const unsigned long long share = (total + c.ctas - 1) / c.ctas;
  const unsigned long long begin = min(share * blockIdx.x, total), stop = min(begin + share, total);
  for (uint32_t r = r0; r < r1; ++r) {
    const unsigned long long m = cost_of(c, span_of(c, r));
    if (begin >= at && begin < at + m) {
      s_req = r;
      s_base = at;
    }
    at += m;
    if (m == 0 && r % c.ctas == blockIdx.x) {
      // a request without tokens
      for (uint32_t j = 0; j < c.heads; ++j) {
        T* to = static_cast<T*>(c.out) + (long long)r * c.out_stride + (long long)j * c.out_head_stride;
        for (uint32_t d = 0; d < c.head_dim; d += 8) *reinterpret_cast<uint4*>(to + d) = make_uint4(0, 0, 0, 0);
        if (c.lse) c.lse[(size_t)r * c.heads + j] = -INFINITY;
      }
    }
  }
  if (tid == 0) c.splits[blockIdx.x] = make_uint4(0, 0, 0, 0);
  if (begin >= stop) return;  // (all threads: nothing in this piece)
  __syncthreads();
  uint32_t r = s_req;
  unsigned long long r_base = s_base, u = begin;

  Loader<T, D> in{c, nullptr, 0, 0, (uint32_t)__cvta_generic_to_shared(mem + warp * S::WARP_BYTES)};
  while (u < stop) {
    // the piece's part of one request, key head and share of the group
    Span sp = span_of(c, r);
    while (sp.end == sp.begin) sp = span_of(c, ++r);   // (u < total: a request with tokens follows)
    const uint32_t tiles = tiles_of(sp), cost = tiles + START;
    const uint32_t which = (uint32_t)((u - r_base) / cost), off = (uint32_t)((u - r_base) % cost);
    const uint32_t until = (uint32_t)min((unsigned long long)cost, off + (stop - u));
    const uint32_t tile0 = off > START ? off - START : 0u, tile1 = until > START ? until - START : 0u;
    u += until - off;
    const unsigned long long next_base = r_base + (unsigned long long)cost * (c.kv_heads * c.parts);
    const uint32_t r_now = r;
    if (u == next_base) {
      r_base = next_base;
      ++r;
    }
    if (tile0 == tile1) continue;   // (only the start's share)
    const uint32_t part = which % c.parts, head = which / c.parts;
    const uint32_t j0 = head * c.group + part * c.gt, heads = min(c.gt, c.group - part * c.gt);  // query heads
    const long long p0 = sp.begin + (long long)tile0 * TILE, p1 = min(sp.end, sp.begin + (long long)tile1 * TILE);
    in.row = c.table + (long long)r_now * c.table_stride;
    in.end = p1;
    in.head_off = (long long)head * c.head_stride;
    const uint32_t tiles_here = tile1 - tile0;

    // the first steps' copies, their places looked up together; then the place of each
    // step's tokens is looked up a step early
    long long p = p0 + warp * STEP + (lane & 15u), next[S::DEPTH];
    uint32_t ring[S::DEPTH - 1];   // which tokens of the steps under way are there
#pragma unroll
    for (int i = 0; i < S::DEPTH; ++i) next[i] = in.place(p + i * TILE);
#pragma unroll
    for (int i = 0; i < S::DEPTH - 1; ++i) {
      ring[i] = __ballot_sync(ALL, next[i] >= 0) & 0xffffu;
      if ((uint32_t)i < tiles_here) in.issue(i, next[i]);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    long long ahead_at = next[S::DEPTH - 1];
    p += (S::DEPTH - 1) * TILE;
    // the queries, as the matrices' second operand
    uint32_t q[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t j = nt * 8 + g;
      const T* from = static_cast<const T*>(c.q) + (long long)r_now * c.q_stride + (long long)(j0 + (j < heads ? j : 0)) * c.q_head_stride;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t d = i * 16 + b * 8 + t * 2;
          q[nt][i][b] = j < heads && d < c.head_dim ? *reinterpret_cast<const uint32_t*>(from + d) : 0u;
        }
    }
    float o[NT][D / 16][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      ref[nt][0] = ref[nt][1] = -FLT_MAX;
      sum[nt][0] = sum[nt][1] = 0.f;
    }

    uint32_t stage = 0;
#pragma unroll 1
    for (uint32_t step = 0; step < tiles_here; ++step) {
      // the copies DEPTH - 1 steps ahead, into the stage that was read last
      const uint32_t ahead = stage == 0 ? S::DEPTH - 1 : stage - 1;
      __syncwarp();
      const uint32_t seen = __ballot_sync(ALL, ahead_at >= 0) & 0xffffu;
      if (step + S::DEPTH - 1 < tiles_here) {
        in.issue(ahead, ahead_at);
        p += TILE;
        ahead_at = in.place(p);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      uint32_t live = ring[0];
#pragma unroll
      for (int i = 0; i < S::DEPTH - 2; ++i) ring[i] = ring[i + 1];
      ring[S::DEPTH - 2] = seen;
      asm volatile("cp.async.wait_group %0;" ::"n"(S::DEPTH - 1) : "memory");
      __syncwarp();
      const uint32_t ks = in.slot + stage * S::STAGE, vs = ks + STEP * S::ROW;
      stage = stage + 1 == S::DEPTH ? 0 : stage + 1;

      // scores: tokens g and g + 8 of query heads 2 t and 2 t + 1
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        const uint32_t row = lane & 15u, chunk = 2 * i + (lane >> 4);
        ldmatrix(a, ks + row * S::ROW + (chunk ^ (row & 7u)) * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Mma<T>::mma(s[nt], a, q[nt][i][0], q[nt][i][1]);
      }
      const bool has0 = live >> g & 1u, has8 = live >> (g + 8) & 1u;
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = (e < 2 ? has0 : has8) ? s[nt][e] * c.scale_log2 : -INFINITY;
          above |= s[nt][e] - ref[nt][e & 1] > SLACK;
        }
      if (__any_sync(ALL, above)) {
        // a new reference: the largest score so far of each query head (its 8 lanes agree)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[nt][e], s[nt][e + 2]);
            m = fmaxf(m, __shfl_xor_sync(ALL, m, 4));
            m = fmaxf(m, __shfl_xor_sync(ALL, m, 8));
            m = fmaxf(m, __shfl_xor_sync(ALL, m, 16));
            m = fmaxf(m, ref[nt][e]);
            const float f = ex2(ref[nt][e] - m);
            ref[nt][e] = m;
            sum[nt][e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][e] *= f;
              o[nt][i][e + 2] *= f;
            }
          }
      }
      // weights, in parts: with one alone they would be off by half a step of the type, as
      // much as the rounding of out
      constexpr int PARTS = Mma<T>::PARTS;
      uint32_t w[NT][PARTS][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = ex2(s[nt][2 * e] - ref[nt][0]) * Mma<T>::UNIT, y = ex2(s[nt][2 * e + 1] - ref[nt][1]) * Mma<T>::UNIT;
          sum[nt][0] += x;
          sum[nt][1] += y;
          uint32_t part[PARTS];
          Mma<T>::split(x, y, part);
#pragma unroll
          for (int p = 0; p < PARTS; ++p) w[nt][p][e] = transposed(part[p]);
        }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        const uint32_t row = (lane & 7u) + (lane >> 4) * 8, chunk = 2 * i + (lane >> 3 & 1u);
        ldmatrix_trans(a, vs + row * S::ROW + (chunk ^ (row & 7u)) * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Mma<T>::add(o[nt][i], a, w[nt]);
      }
    }

    // the warps' parts into shared memory (each into its own), then joined
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    constexpr int PITCH = D + 4;
    float* my = reinterpret_cast<float*>(mem + warp * S::WARP_BYTES);
    float finite = 0.f;   // a NaN once a number is not
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = sum[nt][e];
        x += __shfl_xor_sync(ALL, x, 4);
        x += __shfl_xor_sync(ALL, x, 8);
        x += __shfl_xor_sync(ALL, x, 16);
        const uint32_t j = nt * 8 + t * 2 + e;
        if (g == 0) {
          s_ref[warp][j] = ref[nt][e];
          s_tot[warp][j] = x;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          my[j * PITCH + i * 16 + g] = o[nt][i][e];
          my[j * PITCH + i * 16 + g + 8] = o[nt][i][e + 2];
          finite = fmaf(o[nt][i][e], 0.f, finite);
          finite = fmaf(o[nt][i][e + 2], 0.f, finite);
        }
      }
    if (__any_sync(ALL, finite != 0.f)) {
      __syncwarp();
      set_infinities(in, p0 + warp * STEP + (lane & 15u), tiles_here, my, PITCH, s_tot[warp], heads);
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == tiles;
    // a part that the CTA before began is its first; one that the next CTA ends its second
    const size_t part_at = (size_t)blockIdx.x * 2 + (tile0 == 0 ? 1 : 0);
    for (uint32_t i = tid; i < heads * (D / 2); i += THREADS) {
      const uint32_t j = i / (D / 2), d = i % (D / 2) * 2;
      float m = s_ref[0][j];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) m = fmaxf(m, s_ref[w][j]);
      float x = 0.f, y = 0.f, tot = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ex2(s_ref[w][j] - m);
        const float2 v = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(mem + w * S::WARP_BYTES) + j * PITCH + d);
        x = plus(x, v.x, f);
        y = plus(y, v.y, f);
        tot = fmaf(s_tot[w][j], f, tot);
      }
      if (whole) {
        if (d < c.head_dim) {
          const float inv = tot == 0.f ? 0.f : 1.f / tot;
          T* to = static_cast<T*>(c.out) + (long long)r_now * c.out_stride + (long long)(j0 + j) * c.out_head_stride + d;
          *reinterpret_cast<uint32_t*>(to) = Mma<T>::pack(x * inv, y * inv);
        }
        if (d == 0 && c.lse) c.lse[(size_t)r_now * c.heads + j0 + j] = tot == 0.f ? -INFINITY : (m + log2f(tot * (1.f / Mma<T>::UNIT))) * LN2;
      } else {
        *reinterpret_cast<float2*>(c.outs + (part_at * 16 + j) * D + d) = make_float2(x, y);
        if (d == 0) *reinterpret_cast<float2*>(c.sums + (part_at * 16 + j) * 2) = make_float2(m, tot);
      }
    }
    if (tid == 0 && tile0 == 0 && !whole) {
      // who ends it: the CTA that has its last tile
      const unsigned long long end = (u - until) + cost;
      c.splits[blockIdx.x] = make_uint4(r_now, which, (uint32_t)((end - 1) / share), 1);
    }
    __syncthreads();
  }
}

// A CTA for each query head of what a CTA above began and others end: their parts
// joined in order (every GROUPS-th one by the same threads, then these).
template <class T, int D>
__global__ void __launch_bounds__(THREADS) k_attend_join(AttendCall c) {
  constexpr int LANES = D / 2, GROUPS = THREADS / LANES, MOST = 1024;
  __shared__ float s_f[MOST], s_x[GROUPS][D], s_m[THREADS / 32], s_t[GROUPS];
  const uint32_t first = blockIdx.x / c.gt, j = blockIdx.x % c.gt, tid = threadIdx.x, group = tid / LANES, d = tid % LANES * 2;
  wait_for_previous();
  const uint4 split = c.splits[first];
  if (!split.w) return;
  const uint32_t r = split.x, part = split.y % c.parts, head = split.y / c.parts, n = split.z - first + 1;
  const uint32_t j0 = head * c.group + part * c.gt, heads = min(c.gt, c.group - part * c.gt);
  if (j >= heads) return;
  // part k is the second of CTA `first`, or the first of a CTA after it
  auto place = [&](uint32_t k) { return ((size_t)(first + k) * 2 + (k == 0 ? 1 : 0)) * 16 + j; };
  float m = -FLT_MAX;
  for (uint32_t k = tid; k < n; k += THREADS) m = fmaxf(m, c.sums[place(k) * 2]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(ALL, m, o));
  if ((tid & 31u) == 0) s_m[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = fmaxf(m, s_m[w]);
  float x = 0.f, y = 0.f, tot = 0.f;
  for (uint32_t k0 = 0; k0 < n; k0 += MOST) {   // (as many CTAs as the GPU holds at once: a few hundred)
    const uint32_t some = min(n - k0, (uint32_t)MOST);
    __syncthreads();
    for (uint32_t k = tid; k < some; k += THREADS) s_f[k] = ex2(c.sums[place(k0 + k) * 2] - m);
    __syncthreads();
#pragma unroll 8
    for (uint32_t k = group; k < some; k += GROUPS) {
      const size_t at = place(k0 + k);
      const float2 v = *reinterpret_cast<const float2*>(c.outs + at * D + d);
      const float f = s_f[k];
      x = plus(x, v.x, f);
      y = plus(y, v.y, f);
      tot = fmaf(c.sums[at * 2 + 1], f, tot);
    }
  }
  s_x[group][d] = x;
  s_x[group][d + 1] = y;
  if (d == 0) s_t[group] = tot;
  __syncthreads();
  if (group) return;
  for (int g = 1; g < GROUPS; ++g) {
    x += s_x[g][d];
    y += s_x[g][d + 1];
    tot += s_t[g];
  }
  if (d < c.head_dim) {
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    T* to = static_cast<T*>(c.out) + (long long)r * c.out_stride + (long long)(j0 + j) * c.out_head_stride + d;
    *reinterpret_cast<uint32_t*>(to) = Mma<T>::pack(x * inv, y * inv);
  }
  if (d == 0 && c.lse) c.lse[(size_t)r * c.heads + j0 + j] = tot == 0.f ? -INFINITY : (m + log2f(tot * (1.f / Mma<T>::UNIT))) * LN2;
}

struct StoreCall {
  uint4* k;  // (in units of 16 bytes, as all strides here)
  uint4* v;
  long long block_stride, token_stride, head_stride;
  uint32_t block_size, kv_heads, row;  // row: of a head
  unsigned long long slots;
  const uint4* new_k;
  const uint4* new_v;
  long long new_token_stride, new_head_stride;
  const long long* slot;
  uint32_t n;
};

// A copy of 2 * row units a head and token; a thread takes one of the keys and one of
// the values.  Bound by the bytes: 16,381 tokens of 8 heads of 128 in 24.6 us (5.5 TB/s; 18.5
// where one call is repeated, whose bytes stay in L2 in part).  64 tokens: a launch, 1.7 us
// in a graph, 6.3 a call through the binding.
__global__ void __launch_bounds__(256) k_store(StoreCall c) {
  const uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const uint32_t per = c.kv_heads * c.row;
  const uint32_t t = (uint32_t)(i / per), e = (uint32_t)(i % per);
  if (t >= c.n) return;
  const long long slot = c.slot[t];
  if ((unsigned long long)slot >= c.slots) return;
  const uint32_t h = e / c.row, x = e % c.row;
  const long long from = (long long)t * c.new_token_stride + (long long)h * c.new_head_stride + x;
  const long long to = slot / c.block_size * c.block_stride + slot % c.block_size * c.token_stride + (long long)h * c.head_stride + x;
  const uint4 a = __ldcs(c.new_k + from), b = __ldcs(c.new_v + from);
  c.k[to] = a;
  c.v[to] = b;
}

// nullptr, or what is wrong with a cache
const char* check_cache(const tok_kv_cache* c) {
  if (!c || !c->d_k || !c->d_v) return "paged cache: the keys or the values are NULL";
  if (c->dtype != TOK_F16 && c->dtype != TOK_BF16) return "paged cache: unknown type";
  if (c->n_blocks == 0 || c->n_blocks > 0x7fffffffu || c->block_size == 0 || c->block_size > (1u << 20) || c->kv_heads == 0 ||
      c->kv_heads > 1024 || c->head_dim == 0 || c->head_dim > 256 || c->head_dim % 8)
    return "paged cache: n_blocks, block_size, kv_heads or head_dim is out of range";
  if (!lies_at(c->d_k, 16) || !lies_at(c->d_v, 16) || c->block_stride % 8 || c->token_stride % 8 || c->head_stride % 8 ||
      c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return "paged cache: the arrays lie at multiples of 16 bytes, their strides are multiples of 8";
  return nullptr;
}

struct Sizes {
  int d;              // width that kernels are made for
  uint32_t gt, parts, ctas;
  uint64_t splits, sums, outs, bytes;
};

bool sizes_of(const tok_handle* h, uint32_t n, uint32_t heads, uint32_t kv_heads, uint32_t head_dim, Sizes* s) {
  if (n > MOST_REQUESTS || kv_heads == 0 || kv_heads > 1024 || heads == 0 || heads % kv_heads || heads / kv_heads > MOST_GROUP ||
      head_dim == 0 || head_dim > 256 || head_dim % 8)
    return false;
  const uint32_t group = heads / kv_heads;
  s->d = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  // (a share of eight query heads or, where the registers have room, sixteen)
  s->gt = group <= 8 || s->d == 256 ? 8 : 16;
  s->parts = (group + s->gt - 1) / s->gt;
  s->ctas = (uint32_t)h->n_sms * (s->d == 256 ? 1 : 2);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) { const uint64_t here = at; at = (at + bytes + 255) / 256 * 256; return here; };
  s->splits = take((uint64_t)s->ctas * 16);
  s->sums = take((uint64_t)s->ctas * 2 * 16 * 2 * 4);
  s->outs = take((uint64_t)s->ctas * 2 * 16 * (uint64_t)s->d * 4);
  s->bytes = at;
  return true;
}

template <class T, int D, int NT>
cudaError_t launch_attend(int dev, const AttendCall& c, cudaStream_t s) {
  cudaError_t e = launch_clusters<k_attend<T, D, NT>>(dev, c.ctas, THREADS, 1, Shape<D>::BYTES, s, c);
  if (e != cudaSuccess) return e;
  return launch_behind(k_attend_join<T, D>, c.ctas * c.gt, THREADS, 0, s, c);
}

template <class T>
cudaError_t launch_type(int dev, int d, const AttendCall& c, cudaStream_t s) {
  if (d == 64) return c.gt == 8 ? launch_attend<T, 64, 1>(dev, c, s) : launch_attend<T, 64, 2>(dev, c, s);
  if (d == 128) return c.gt == 8 ? launch_attend<T, 128, 1>(dev, c, s) : launch_attend<T, 128, 2>(dev, c, s);
  return launch_attend<T, 256, 1>(dev, c, s);
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_paged_store(tok_handle* h, const tok_kv_cache* c, const tok_store_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->n == 0) return TOK_OK;
  if (const char* w = check_cache(c)) return fail(h, TOK_EINVAL, w);
  if (!a || !a->d_k || !a->d_v || !a->d_slot) return fail(h, TOK_EINVAL, "paged store: a buffer is NULL");
  if (a->n >= (1ull << 31)) return fail(h, TOK_EINVAL, "paged store: n is out of range");
  if (!lies_at(a->d_k, 16) || !lies_at(a->d_v, 16) || !lies_at(a->d_slot, 8) || a->token_stride % 8 || a->head_stride % 8)
    return fail(h, TOK_EINVAL, "paged store: the arrays lie at multiples of 16 bytes, their strides are multiples of 8");
  DeviceGuard g(h->dev);
  StoreCall s{static_cast<uint4*>(c->d_k), static_cast<uint4*>(c->d_v), c->block_stride / 8, c->token_stride / 8, c->head_stride / 8,
              c->block_size, c->kv_heads, c->head_dim / 8, (unsigned long long)c->n_blocks * c->block_size,
              static_cast<const uint4*>(a->d_k), static_cast<const uint4*>(a->d_v), a->token_stride / 8, a->head_stride / 8,
              reinterpret_cast<const long long*>(a->d_slot), (uint32_t)a->n};
  const uint64_t ctas = (a->n * s.kv_heads * s.row + 255) / 256;
  if (ctas > 0x7fffffffull) return fail(h, TOK_EINVAL, "paged store: n times a token's size is out of range");
  k_store<<<(unsigned)ctas, 256, 0, static_cast<cudaStream_t>(stream)>>>(s);
  h->launches += 1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

uint64_t tok_paged_attend_work_bytes(tok_handle* h, uint32_t n, uint32_t heads, uint32_t kv_heads, uint32_t head_dim) {
  Sizes s;
  return h && sizes_of(h, n, heads, kv_heads, head_dim, &s) ? s.bytes : 0;
}

int tok_paged_attend(tok_handle* h, const tok_kv_cache* c, const tok_attend_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->n == 0) return TOK_OK;
  if (const char* w = check_cache(c)) return fail(h, TOK_EINVAL, w);
  if (!a || !a->d_q || !a->d_out || !a->d_table || !a->d_seq_len) return fail(h, TOK_EINVAL, "paged attend: a buffer is NULL");
  Sizes z;
  if (!sizes_of(h, a->n, a->heads, c->kv_heads, c->head_dim, &z) || a->max_blocks > 0x7fffffffu ||
      a->table_stride < (int64_t)a->max_blocks)
    return fail(h, TOK_EINVAL, "paged attend: n, heads, max_blocks or table_stride is out of range");
  if (!lies_at(a->d_q, 16) || !lies_at(a->d_out, 16) || a->q_stride % 8 || a->q_head_stride % 8 || a->out_stride % 8 ||
      a->out_head_stride % 8 || !lies_at(a->d_lse, 4) || !lies_at(a->d_table, 4) || !lies_at(a->d_seq_len, 8))
    return fail(h, TOK_EINVAL, "paged attend: queries and out lie at multiples of 16 bytes, their strides are multiples of 8");
  if (!a->d_work || !lies_at(a->d_work, 256) || a->work_bytes < z.bytes)
    return fail(h, TOK_EINVAL, "paged attend: d_work is NULL, not at a multiple of 256 bytes or too small");
  DeviceGuard g(h->dev);
  uint8_t* work = static_cast<uint8_t*>(a->d_work);
  AttendCall k{};
  k.k = c->d_k;
  k.v = c->d_v;
  k.block_stride = c->block_stride;
  k.token_stride = c->token_stride;
  k.head_stride = c->head_stride;
  k.n_blocks = c->n_blocks;
  k.block_size = c->block_size;
  k.kv_heads = c->kv_heads;
  k.head_dim = c->head_dim;
  k.q = a->d_q;
  k.q_stride = a->q_stride;
  k.q_head_stride = a->q_head_stride;
  k.out = a->d_out;
  k.out_stride = a->out_stride;
  k.out_head_stride = a->out_head_stride;
  k.lse = a->d_lse;
  k.n = a->n;
  k.heads = a->heads;
  k.group = a->heads / c->kv_heads;
  k.gt = z.gt;
  k.parts = z.parts;
  k.scale_log2 = a->scale * LOG2E;
  k.window = a->window;
  k.table = a->d_table;
  k.table_stride = a->table_stride;
  // (a token's place in its row is a 32-bit number)
  k.most_len = std::min<long long>((long long)a->max_blocks * c->block_size, 0x7fffffffll);
  k.seq_len = reinterpret_cast<const long long*>(a->d_seq_len);
  k.splits = reinterpret_cast<uint4*>(work + z.splits);
  k.sums = reinterpret_cast<float*>(work + z.sums);
  k.outs = reinterpret_cast<float*>(work + z.outs);
  k.ctas = z.ctas;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->dtype == TOK_F16 ? launch_type<__half>(h->dev, z.d, k, s) : launch_type<__nv_bfloat16>(h->dev, z.d, k, s);
  h->launches += 2;
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
