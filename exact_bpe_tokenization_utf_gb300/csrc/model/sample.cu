// The choice of a token for each row of scores (tok_sample).
//
// With M = the largest score and T = the temperature, w(v) = exp((x(v) - M) / T).  The
// tokens in the order of falling scores, equal ones by their ids, form a list from
// which min-p keeps those with w >= m, top-k the first k of these, top-p the shortest
// beginning whose sum reaches p times the whole; the choice is the first at which
// the running sum exceeds u times the sum of what is left.
//
// Every border lies where a running sum reaches a number, so that two sums formed
// differently could disagree about it.  Weights are therefore 43-bit fixed-point
// numbers, formed with 38 bits or more, and sums are whole numbers: they do not depend
// on the order in which threads add.
//
// Rows of 32-bit scores: a cluster of CTAs holds the row in shared memory, so that it
// is read once.  After the maximum, each token is counted in one of 2,048 bins of equal
// width of log w, with its weight.  The bins' sums say in which bin a border lies; the
// tokens of that bin (a few hundred, as a rule) go to the cluster's first CTA, which
// sorts them.  Where there are more, bins of keys (scores as whole numbers of the same
// order) come in between, until a bin holds few tokens or a single score.  Where top-k or
// min-p leave few tokens, their number is found without weights and they go there at once.
// Bound by instructions: a weight takes about 45.
//
// Rows of 16-bit scores have few different scores.  They are counted score by score, with
// an atomic on shared memory for each token and two tokens in each operation before it; a
// weight is formed once for a score, and a border is met by counts alone.  The choice's
// id is then searched in the row, which is read again from L2.  512 rows of 100,257 bf16
// scores 70 us on a GB300 (the bytes: 15 us): 25 to 50 of counting (bound by the atomics,
// 3 cycles for a warp's 32), 8 of weights, 3 of borders, 6 to 14 of the search.
#include "types.cuh"

#include <cooperative_groups.h>

namespace tokgb {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t ALL = 0xffffffffu;
constexpr uint32_t MOST_LOGITS = 1u << 20;
constexpr int MOST_WARPS = 32;                // of a CTA
constexpr uint32_t LIST = 1024;               // most tokens that are sorted
constexpr double ONE = 8796093022208.0;       // the largest weight, 2^43; 2^20 of them fit 64 bits
constexpr int MOST_COMMANDS = 64;             // three goals of at most 8 each; a limit, so that the kernel ends
constexpr float LOWEST = -62.f;               // log2 of weights that count (below 2^-43 they are 0 anyway)
constexpr int LOWEST_K = -(1 << 22);          // of log2 w in units of 2^-16

// --- weights ---------------------------------------------------------------------

// 2^(i / 256) and 2^(i / 65536) - 1 by their series, evaluated by the compiler
struct Pow { unsigned long long whole; uint32_t top; float near; };   // 2^39, 2^31 times, and as it is
struct Fine { uint32_t less; float near; };                          // 2^40 times, and as it is
struct Powers { Pow a[256]; Fine b[256]; };
constexpr double exp_less_1(double x) {   // |x| < 0.7
  double term = x, sum = 0;
  for (int i = 2; i < 30; ++i) {
    sum += term;
    term = term * x / i;
  }
  return sum;
}
constexpr Powers make_powers() {
  Powers p{};
  constexpr double ln2 = 0.693147180559945309417;
  for (int i = 0; i < 256; ++i) {
    const double x = 1.0 + exp_less_1(i * ln2 / 256), y = exp_less_1(i * ln2 / 65536);
    p.a[i] = Pow{(unsigned long long)(x * 549755813888.0 + 0.5), (uint32_t)(x * 2147483648.0 + 0.5), (float)x};
    p.b[i] = Fine{(uint32_t)(y * 1099511627776.0 + 0.5), (float)y};
  }
  return p;
}
__device__ const Powers g_powers = make_powers();

// a row's temperature and maximum, for weights
struct Rule {
  float shrink;         // scores are taken times it, so that differences are finite and c is not too small:
                        // 1/2, or 2^-64 for temperatures from 2^64 on
  float c_hi, c_lo;     // log2(e) / T, for those
  float top;            // the largest score, so taken
  float x_max;          // and as it is
  bool only_max;        // no other weight is above 0
};

// all but top and x_max
__device__ __forceinline__ void set_temperature(Rule& r, float temp) {
  r.shrink = temp >= 0x1p64f ? 0x1p-64f : 0.5f;
  r.only_max = temp < 0x1p-100f;
  const double k = 1.4426950408889634074 / (r.only_max ? 1.0 : (double)temp * r.shrink);   // (0 for an infinite one: all weights are 1)
  r.c_hi = (float)k;
  r.c_lo = (float)(k - (double)(float)k);
}
__device__ __forceinline__ void set_largest(Rule& r, float x) {
  r.x_max = x;
  r.top = x * r.shrink;
}

// log2 w in two parts: hi rounded to 32 bits, and the rest.  The difference to the largest
// score comes first, exactly in two parts: the product is off by 2^-46 of log2 w, however
// far from 0 the scores lie.  hi never rises where x falls (but by its last place, where
// two scores differ by less than 2^-46 of their difference to the largest).
__device__ __forceinline__ void log2_weight(const Rule& r, float x, float& hi, float& lo) {
  const float y = __fmul_rn(x, r.shrink), d = y - r.top, back = d - y;
  const float err = (y - (d - back)) + (-r.top - back);
  const float p = __fmul_rn(d, r.c_hi);   // (not to be joined with the sums after it)
  float e = fmaf(d, r.c_hi, -p);
  e = fmaf(d, r.c_lo, fmaf(err, r.c_hi, e));
  hi = p + e;
  lo = e - (hi - p);
  if (r.only_max || !(p > -1e4f)) {
    hi = x == r.x_max ? 0.f : -1e4f;
    lo = 0.f;
  }
}

// log2 w in units of 2^-16 (at most 0), and what is left of it
__device__ __forceinline__ int fixed_log2(float hi, float lo, float& rest) {
  if (hi < LOWEST) return LOWEST_K;
  constexpr float MAGIC = 192.f;                     // 1.5 * 2^7: its last place is 2^-16
  const float m = hi + MAGIC;
  rest = (hi - (m - MAGIC)) + lo;
  return min(__float_as_int(m) - __float_as_int(MAGIC), 0);
}

// 2^43 times w: 2^(k / 65536 + rest) is a whole power of 2, two factors from the
// tables and 1 + q for the rest (below 2^-17), so that 32-bit arithmetic on q is enough.
__device__ __forceinline__ unsigned long long weight(const Pow* a, const Fine* b, int k, float rest) {
  if (k == LOWEST_K) return 0;
  const Pow x = a[(k >> 8) & 255];
  const Fine y = b[k & 255];
  constexpr float L1 = 0.693147180559945f, L2 = 0.240226506959101f;   // ln 2, (ln 2)^2 / 2
  const float q = rest * fmaf(rest, L2, L1);
  const int v = __float2int_rn(fmaf(x.near, y.near, x.near) * 549755813888.f * q);
  const unsigned long long s = x.whole + __umulhi(x.top, y.less) + (long long)v;   // 2^39 times
  return (((s << 5) >> -(k >> 16)) + 1) >> 1;
}

__device__ __forceinline__ uint32_t key_of(float x) {   // whole numbers of the same order
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);   // (-0 is 0)
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

__device__ __forceinline__ double t_ln(float temp, float min_p) {
  return !(min_p > 0.f) ? 0.0 : temp < INFINITY ? (double)temp * log((double)min_p) : -INFINITY;
}
// scores below this are not kept: M + T ln(min_p) (T = 0: M)
__device__ __forceinline__ float least_of(const Rule& r, float temp, float min_p, double t_ln_m) {
  if (!(min_p > 0.f)) return -INFINITY;
  if (min_p > 1.f) return INFINITY;
  return __double2float_ru(temp >= 0x1p-100f ? (double)r.x_max + t_ln_m : (double)r.x_max);
}

// The sums that top-p's list and the choice have to reach, with all bits of p (below
// 1) and u: the least whole number from p times the mass on, and above u times it.
__device__ __forceinline__ unsigned long long enough(float p, unsigned long long mass) {
  const unsigned long long f = __double2ull_rd((double)fmaxf(p, 0.f) * 18446744073709551616.0);
  const unsigned long long m = __umul64hi(f, mass) + (f * mass != 0 ? 1 : 0);
  return m ? m : 1;
}
__device__ __forceinline__ unsigned long long chosen_at(float u, unsigned long long mass) {
  const float v = u >= 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f;
  return __umul64hi(__double2ull_rd((double)v * 18446744073709551616.0), mass) + 1;
}

// --- the kernel --------------------------------------------------------------------

enum Op { OP_DONE, OP_BINS, OP_GATHER, OP_NTH };

struct Command {
  int op;
  uint32_t lo, hi;      // keys: the tokens that it is about
  uint32_t shift;       // OP_BINS: bin = (hi - key) >> shift
  uint32_t nth;         // OP_NTH: which of the tokens of key lo, in the order of ids
  int by_bin;           // the tokens of a bin of log w instead, or -1
  int through;          // OP_GATHER: of all bins up to it
};

// Bins are of 2^BIN_SHIFT units of log2 w, to 2^-64; the last one is for all below, too.
template <int BIN_SHIFT> struct Shared {
  static constexpr int BINS = 1 << (22 - BIN_SHIFT);
  Pow pow[256];
  Fine fine[256];
  uint32_t cnt[BINS], low[BINS], high[BINS];         // this CTA's bins
  // the first CTA's: sums over all bins up to each
  unsigned long long mass[BINS];
  uint32_t upto[BINS];
  union {
    struct { unsigned long long mass[BINS]; uint32_t upto[BINS]; } sub;   // of bins of keys
    unsigned long long list[LIST];                                        // (~key, id)
  };
  unsigned long long scan_m[MOST_WARPS];
  uint32_t scan_c[MOST_WARPS];
  float part_max[16];
  uint32_t part_cnt[16], part_lo[16], part_hi[16];
  Rule rule;
  double t_ln_m;                                     // T ln(min_p), for the threshold
  uint32_t listed;
  Command cmd;
  int brief;                                         // apart from cmd, which the first CTA may set again before all have read it
  uint32_t found;
  unsigned long long answer_mass;
  uint32_t answer_cnt, answer_key;
};

struct Slice {
  const void* at;        // element `from` (in shared memory, or the row's)
  uint32_t from, to;
};

// By all threads: one(place, element) for the elements before and after the 16-byte
// pieces that the slice has, piece(place, its elements) for these.
template <class T, int N, int UNROLL, class F, class G>
__device__ __forceinline__ void for_vectors(const Slice& s, F one, G piece) {
  const T* x = static_cast<const T*>(s.at);
  const uint32_t n = s.to - s.from;
  constexpr uint32_t VEC = 16 / sizeof(T);
  const uint32_t head = min(n, (uint32_t)((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / (uint32_t)sizeof(T));
  const uint32_t vecs = (n - head) / VEC, tail = head + vecs * VEC;
  for (uint32_t i = threadIdx.x; i < head + (n - tail); i += N) {
    const uint32_t e = i < head ? i : tail + (i - head);
    one(e, x[e]);
  }
#pragma unroll UNROLL
  for (uint32_t i = threadIdx.x; i < vecs; i += N) piece(head + i * VEC, reinterpret_cast<const uint4*>(x + head)[i]);
}
// f(score, id) for every element
template <class T, int N, class F>
__device__ __forceinline__ void for_each(const Slice& s, F f) {
  for_vectors<T, N, sizeof(T) == 4 ? 2 : 1>(s, [&](uint32_t e, T x) { f(to_f32(x), s.from + e); }, [&](uint32_t e, uint4 q) {
    const T* y = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (uint32_t i = 0; i < 16 / sizeof(T); ++i) f(to_f32(y[i]), s.from + e + i);
  });
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

struct SampleCall {
  tok_sample_args a;
  uint32_t ranks;     // CTAs of a row
  uint32_t per;       // elements of a CTA
  int resident;       // its elements are kept in shared memory
};

// sums over the threads before, and of all (in every thread)
template <int WARPS, class S>
__device__ __forceinline__ void block_scan(S& sh, uint32_t& c, unsigned long long& m, uint32_t& all_c, unsigned long long& all_m) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  uint32_t ic = c;
  unsigned long long im = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t pc = __shfl_up_sync(ALL, ic, o);
    const unsigned long long pm = __shfl_up_sync(ALL, im, o);
    if (lane >= (uint32_t)o) {
      ic += pc;
      im += pm;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sh.scan_c[warp] = ic;
    sh.scan_m[warp] = im;
  }
  __syncthreads();
  uint32_t bc = 0;
  unsigned long long bm = 0;
  all_c = 0;
  all_m = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < (int)warp) {
      bc += sh.scan_c[w];
      bm += sh.scan_m[w];
    }
    all_c += sh.scan_c[w];
    all_m += sh.scan_m[w];
  }
  c = bc + ic - c;
  m = bm + im - m;
}

template <class T, int THREADS, int BIN_SHIFT>
__device__ __forceinline__ void choose(const SampleCall& c, uint8_t* mem) {
  using Shared = tokgb::Shared<BIN_SHIFT>;
  constexpr int BINS = Shared::BINS, WARPS = THREADS / 32, PER_BIN = BINS / THREADS, PER_LIST = LIST / THREADS;
  Shared& sh = *reinterpret_cast<Shared*>(mem);
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), row = blockIdx.x / c.ranks, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t V = c.a.n_logits;
  Slice s;
  s.from = min(rank * c.per, V);
  s.to = min(s.from + c.per, V);
  const T* src = static_cast<const T*>(c.a.d_scores) + (long long)row * c.a.scores_stride + s.from;
  const float temp = c.a.d_temperature ? c.a.d_temperature[row] : 1.f;
  const float min_p = c.a.d_min_p ? c.a.d_min_p[row] : 0.f;

  // the largest score; the slice into shared memory, lying towards 16 bytes as it does in the row
  float most = -INFINITY;
  s.at = src;
  if (c.resident) {
    T* keep = reinterpret_cast<T*>(mem + ((sizeof(Shared) + 15) & ~size_t(15)) + (reinterpret_cast<uintptr_t>(src) & 15u));
    for_vectors<T, THREADS, 4>(s, [&](uint32_t e, T x) {
      most = max_nan(most, to_f32(x));
      keep[e] = x;
    }, [&](uint32_t e, uint4 q) {
      *reinterpret_cast<uint4*>(keep + e) = q;
      const T* y = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (uint32_t i = 0; i < 16 / sizeof(T); ++i) most = max_nan(most, to_f32(y[i]));
    });
    s.at = keep;
  } else {
    for_each<T, THREADS>(s, [&](float x, uint32_t) { most = max_nan(most, x); });
  }
  for (uint32_t i = tid; i < 256; i += THREADS) {
    sh.pow[i] = g_powers.a[i];
    sh.fine[i] = g_powers.b[i];
  }
  for (uint32_t i = tid; i < BINS; i += THREADS) sh.cnt[i] = sh.low[i] = sh.high[i] = 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(ALL, most, o));
  if (lane == 0) sh.scan_c[warp] = __float_as_uint(most);
  if (tid == 32) {
    set_temperature(sh.rule, temp);
    sh.t_ln_m = t_ln(temp, min_p);
  }
  __syncthreads();
  most = __uint_as_float(sh.scan_c[lane % WARPS]);
#pragma unroll
  for (int o = WARPS / 2; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(ALL, most, o));
  if (tid < c.ranks) cluster.map_shared_rank(&sh, tid)->part_max[rank] = most;
  cluster.sync();
  most = -INFINITY;
  for (uint32_t i = 0; i < c.ranks; ++i) most = max_nan(most, sh.part_max[i]);
  if (!(temp >= 0.f) || !(most > -INFINITY && most < INFINITY)) {   // (all CTAs of the row)
    if (rank == 0 && tid == 0) {
      c.a.d_pick[row] = -1;
      if (c.a.d_kept) c.a.d_kept[row] = 0;
      if (c.a.d_logprob) c.a.d_logprob[row] = -INFINITY;
    }
    return;
  }
  Rule r = sh.rule;
  set_largest(r, most);
  const float least = least_of(r, temp, min_p, sh.t_ln_m);
  auto bin_of = [](int k) { return min((uint32_t)-k >> BIN_SHIFT, (uint32_t)BINS - 1u); };
  // what a token of the row is counted as; false: it is not kept
  auto look = [&](float x, int& k, float& rest) {
    if (!(x >= least) || x == -INFINITY) return false;
    float hi, lo;
    log2_weight(r, x, hi, lo);
    k = fixed_log2(hi, lo, rest);
    return true;
  };
  auto count_in = [&](uint32_t bin, unsigned long long w) {
    atomicAdd(&sh.cnt[bin], 1u);
    const uint32_t w_lo = (uint32_t)w, old = atomicAdd(&sh.low[bin], w_lo);
    const uint32_t carry = (uint32_t)(w >> 32) + (old + w_lo < old ? 1u : 0u);
    if (carry) atomicAdd(&sh.high[bin], carry);
  };
  // a bin of the same width without the care that weights take: off by one at most (but
  // for the last ones), and it never falls where x falls either
  const float bin_scale = (float)(65536 >> BIN_SHIFT) * r.c_hi;
  auto rough_bin = [&](float x) {
    if (r.only_max) return x == r.x_max ? 0u : (uint32_t)BINS - 1u;
    return (uint32_t)min((int)(fmaf(x, -r.shrink, r.top) * bin_scale), BINS - 1);
  };
  // the row's bins: each CTA adds a share of them, for the first one
  auto add_up = [&](bool sub, bool weights) {
    Shared* first = cluster.map_shared_rank(&sh, 0);
    // (ranks lanes side by side read a bin of a CTA each)
    const uint32_t i = tid & (c.ranks - 1), b0 = rank * (BINS / c.ranks) + tid / c.ranks;
    const Shared* o = cluster.map_shared_rank(&sh, i);
    uint32_t n[PER_BIN];
    unsigned long long m[PER_BIN];
#pragma unroll
    for (int k = 0; k < PER_BIN; ++k) {
      const uint32_t b = b0 + k * (THREADS / c.ranks);
      n[k] = o->cnt[b];
      m[k] = weights ? o->low[b] + ((unsigned long long)o->high[b] << 32) : 0ull;
    }
#pragma unroll
    for (int k = 0; k < PER_BIN; ++k) {
      for (uint32_t d = 1; d < c.ranks; d *= 2) {
        n[k] += __shfl_xor_sync(ALL, n[k], d);
        if (weights) m[k] += __shfl_xor_sync(ALL, m[k], d);
      }
      const uint32_t b = b0 + k * (THREADS / c.ranks);
      if (i == 0) {
        (sub ? first->sub.upto : first->upto)[b] = n[k];
        (sub ? first->sub.mass : first->mass)[b] = m[k];
      }
    }
  };

  // sums of the bins up to each (in the first CTA)
  uint32_t all_c = 0;
  unsigned long long all_m = 0;
  auto run_up = [&](uint32_t* upto, unsigned long long* mass) {
    uint32_t n[PER_BIN], bc = 0;
    unsigned long long m[PER_BIN], bm = 0;
#pragma unroll
    for (int i = 0; i < PER_BIN; ++i) {
      n[i] = upto[tid * PER_BIN + i];
      m[i] = mass[tid * PER_BIN + i];
      bc += n[i];
      bm += m[i];
    }
    block_scan<WARPS>(sh, bc, bm, all_c, all_m);
#pragma unroll
    for (int i = 0; i < PER_BIN; ++i) {
      bc += n[i];
      bm += m[i];
      upto[tid * PER_BIN + i] = bc;
      mass[tid * PER_BIN + i] = bm;
    }
    __syncthreads();
  };
  // the first bin at which a sum reaches a number
  auto bin_at = [&](const uint32_t* upto, const unsigned long long* mass, bool by_count, unsigned long long target) {
    uint32_t lo = 0, hi = BINS - 1;
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if ((by_count ? (unsigned long long)upto[mid] : mass[mid]) >= target) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };

  // The goals in turn: the last token of top-k (by count), of top-p (by mass), the
  // choice (by mass).  The first CTA decides, all CTAs carry out.
  enum { GOAL_K, GOAL_P, GOAL_U, GOAL_END };
  int goal = GOAL_K;
  bool started = false;                    // a goal's bin is being looked into
  bool listed = false;                     // all goals' tokens have been listed
  uint32_t kept = 0;                       // tokens kept so far
  unsigned long long kept_m = 0;           // and their mass
  unsigned long long target = 0;           // of the goal
  uint32_t before_c = 0;                   // tokens before the range that is looked into
  unsigned long long before_m = 0;
  uint32_t pick_key = 0;
  float top_p = 1.f, u = 0.f;
  int top_k = 0;
  if (rank == 0) {
    top_k = c.a.d_top_k ? c.a.d_top_k[row] : 0;
    top_p = c.a.d_top_p ? c.a.d_top_p[row] : 1.f;
    u = c.a.d_random[row];
  }
  // Where top-k or min-p leave few tokens, their number is enough to list them; no
  // other token's weight is formed.
  bool brief = false;
  if (min_p > 0.f || (c.a.d_top_k && c.a.d_top_k[row] > 0)) {
    for_each<T, THREADS>(s, [&](float x, uint32_t) {
      if (x >= least && x > -INFINITY) atomicAdd(&sh.cnt[rough_bin(x)], 1u);
    });
    cluster.sync();
    add_up(false, false);
    cluster.sync();
    if (rank == 0) {
      run_up(sh.upto, sh.mass);
      kept = all_c;
      const uint32_t b = bin_at(sh.upto, sh.mass, true, top_k > 0 ? min((uint32_t)top_k, kept) : kept);
      Command next{};
      next.by_bin = (int)b;
      next.op = sh.upto[b] <= LIST ? OP_GATHER : OP_BINS;
      if (tid < c.ranks) cluster.map_shared_rank(&sh, tid)->brief = next.op == OP_GATHER;
      if (tid == 0) sh.cmd = next;
    }
    cluster.sync();
    brief = sh.brief;
    if (!brief)
      for (uint32_t i = tid; i < BINS; i += THREADS) sh.cnt[i] = 0;
    __syncthreads();
  }
  if (!brief) {
    for_each<T, THREADS>(s, [&](float x, uint32_t) {
      int k;
      float rest = 0.f;
      if (look(x, k, rest)) count_in(bin_of(k), weight(sh.pow, sh.fine, k, rest));
    });
    cluster.sync();
    add_up(false, true);
    cluster.sync();
    if (rank == 0) {
      run_up(sh.upto, sh.mass);
      kept = all_c;
      kept_m = all_m;
    }
  }
  // The number that the goal's sum has to reach; false: there is no such rule.
  auto aim = [&]() {
    if (goal == GOAL_K) {
      target = (unsigned long long)max(top_k, 0);
      return target != 0 && target < kept;
    }
    if (goal == GOAL_P) {
      target = enough(top_p, kept_m);
      return top_p < 1.f;
    }
    target = chosen_at(u, kept_m);
    return true;
  };
  // The state after an answer: the first at which the goal's sum is reached is the
  // cnt-th token, the sum up to it mass.
  auto answered = [&](uint32_t cnt, unsigned long long mass) {
    if (goal != GOAL_U) {
      kept = cnt;
      kept_m = mass;
    }
    ++goal;
    started = false;
  };
  for (int commands = 0;; ++commands) {
    if (rank == 0) {
      Command cmd{};
      cmd.by_bin = -1;
      // (all threads of the first CTA come to the same decision)
      while (goal != GOAL_END && kept && !started) {
        if (brief) {   // (the list's command is set; its goals are aimed at when its weights are known)
          listed = started = true;
          break;
        }
        if (!aim()) {
          ++goal;
          continue;
        }
        const uint32_t b = bin_at(sh.upto, sh.mass, goal == GOAL_K, target);
        // where everything up to the first goal's bin fits the list, the goals after it
        // lie there too: one list for all
        if (!listed && sh.upto[b] <= LIST) {
          listed = started = true;
          before_c = 0;
          before_m = 0;
          cmd.by_bin = (int)b;
          cmd.through = 1;
          cmd.op = OP_GATHER;
          continue;
        }
        before_c = b ? sh.upto[b - 1] : 0;
        before_m = b ? sh.mass[b - 1] : 0;
        const uint32_t n = sh.upto[b] - before_c;
        if (goal != GOAL_U && (goal == GOAL_K ? target == sh.upto[b] : n == 1)) {
          answered(sh.upto[b], sh.mass[b]);
          continue;
        }
        started = true;
        cmd.by_bin = (int)b;
        cmd.op = n <= LIST ? OP_GATHER : OP_BINS;   // (OP_BINS with by_bin: only the range of its keys)
      }
      if (goal != GOAL_END && kept && cmd.by_bin < 0 && started) cmd = sh.cmd;   // set by the last answer
      if (commands >= MOST_COMMANDS) cmd.op = OP_DONE;
      if (tid < c.ranks) cluster.map_shared_rank(&sh, tid)->cmd = cmd;
      if (tid == 0) {
        sh.listed = 0;
        sh.found = ALL;
      }
    }
    cluster.sync();
    const Command cmd = sh.cmd;
    if (cmd.op == OP_DONE) break;
    auto wanted = [&](float x, int& k, float& rest) {
      if (cmd.by_bin >= 0) {
        const int rough = (int)rough_bin(x);
        if (brief) return rough <= cmd.by_bin && look(x, k, rest);
        if (cmd.by_bin < BINS - 64 && (rough > cmd.by_bin + 1 || (!cmd.through && rough < cmd.by_bin - 1))) return false;
        if (!look(x, k, rest)) return false;
        const uint32_t b = bin_of(k);
        return b == (uint32_t)cmd.by_bin || (cmd.through && b < (uint32_t)cmd.by_bin);
      }
      const uint32_t key = key_of(x);
      if (key < cmd.lo || key > cmd.hi) return false;
      return look(x, k, rest);
    };
    if (cmd.op == OP_GATHER) {
      Shared* first = cluster.map_shared_rank(&sh, 0);
      for_each<T, THREADS>(s, [&](float x, uint32_t id) {
        int k;
        float rest;
        if (wanted(x, k, rest)) {
          const uint32_t at = atomicAdd(&first->listed, 1u);
          if (at < LIST) first->list[at] = (unsigned long long)(~key_of(x)) << 32 | id;
        }
      });
      cluster.sync();
      if (rank == 0) {
        const uint32_t n = min(sh.listed, LIST);
        uint32_t size = 32;
        while (size < n) size *= 2;
        for (uint32_t i = n + tid; i < size; i += THREADS) sh.list[i] = ~0ull;
        __syncthreads();
        for (uint32_t k = 2; k <= size; k *= 2)
          for (uint32_t j = k / 2; j; j /= 2) {
            for (uint32_t i = tid; i < size / 2; i += THREADS) {
              const uint32_t a = 2 * i - (i & (j - 1)), b = a + j;
              const unsigned long long x = sh.list[a], y = sh.list[b];
              if ((x > y) == ((a & k) == 0)) {
                sh.list[a] = y;
                sh.list[b] = x;
              }
            }
            __syncthreads();
          }
        // sums up to each token, and the first that reaches the target
        unsigned long long w[PER_LIST], sum = 0;
        uint32_t cnt = 0;
#pragma unroll
        for (int i = 0; i < PER_LIST; ++i) {
          w[i] = 0;
          if (tid * PER_LIST + i < n) {
            int k;
            float rest = 0.f;
            look(of_key(~(uint32_t)(sh.list[tid * PER_LIST + i] >> 32)), k, rest);
            w[i] = weight(sh.pow, sh.fine, k, rest);
            ++cnt;
          }
          sum += w[i];
        }
        uint32_t ac;
        unsigned long long am;
        block_scan<WARPS>(sh, cnt, sum, ac, am);
        if (listed) {
          if (brief && !(goal == GOAL_K && aim())) kept_m = am;   // (the list is all that is kept)
          while (goal < GOAL_U && !aim()) ++goal;
          aim();
        }
        do {
          unsigned long long m = before_m + sum;
#pragma unroll
          for (int i = 0; i < PER_LIST; ++i)
            if (tid * PER_LIST + i < n) {
              const unsigned long long next = m + w[i];
              const uint32_t at = before_c + tid * PER_LIST + i + 1;
              if (goal == GOAL_K ? at == target : m < target && next >= target) {
                sh.answer_cnt = at;
                sh.answer_mass = next;
                sh.found = (uint32_t)sh.list[tid * PER_LIST + i];
                sh.answer_key = ~(uint32_t)(sh.list[tid * PER_LIST + i] >> 32);
              }
              m = next;
            }
          __syncthreads();
          pick_key = sh.answer_key;
          answered(sh.answer_cnt, sh.answer_mass);
          __syncthreads();
          // (a list of all tokens that matter serves the next goals)
          if (listed)
            while (goal < GOAL_U && !aim()) ++goal;
        } while (listed && goal != GOAL_END && aim());
      }
    } else if (cmd.op == OP_BINS && cmd.by_bin >= 0) {
      // the range of the bin's keys
      uint32_t lo = ALL, hi = 0;
      for_each<T, THREADS>(s, [&](float x, uint32_t) {
        int k;
        float rest;
        if (wanted(x, k, rest)) {
          lo = min(lo, key_of(x));
          hi = max(hi, key_of(x));
        }
      });
      lo = __reduce_min_sync(ALL, lo);
      hi = __reduce_max_sync(ALL, hi);
      if (tid == 0) {
        sh.scan_c[0] = ALL;
        sh.scan_c[1] = 0;
      }
      __syncthreads();
      if (lane == 0) {
        atomicMin(&sh.scan_c[0], lo);
        atomicMax(&sh.scan_c[1], hi);
      }
      __syncthreads();
      if (tid == 0) {
        cluster.map_shared_rank(&sh, 0)->part_lo[rank] = sh.scan_c[0];
        cluster.map_shared_rank(&sh, 0)->part_hi[rank] = sh.scan_c[1];
      }
      cluster.sync();
      if (rank == 0) {
        Command next{};
        next.by_bin = -1;
        next.op = OP_BINS;
        next.lo = ALL;
        for (uint32_t i = 0; i < c.ranks; ++i) {
          next.lo = min(next.lo, sh.part_lo[i]);
          next.hi = max(next.hi, sh.part_hi[i]);
        }
        while ((next.hi - next.lo) >> next.shift >= BINS) ++next.shift;
        __syncthreads();
        if (tid == 0) sh.cmd = next;
        __syncthreads();
      }
    } else if (cmd.op == OP_BINS) {
      for (uint32_t i = tid; i < BINS; i += THREADS) sh.cnt[i] = sh.low[i] = sh.high[i] = 0;
      __syncthreads();
      for_each<T, THREADS>(s, [&](float x, uint32_t) {
        int k;
        float rest = 0.f;
        if (wanted(x, k, rest)) count_in((cmd.hi - key_of(x)) >> cmd.shift, weight(sh.pow, sh.fine, k, rest));
      });
      cluster.sync();
      add_up(true, true);
      cluster.sync();
      if (rank == 0) {
        uint32_t keep_c = all_c;
        const unsigned long long keep_m = all_m;
        run_up(sh.sub.upto, sh.sub.mass);
        all_c = keep_c;
        all_m = keep_m;
        const unsigned long long rest = target - (goal == GOAL_K ? (unsigned long long)before_c : before_m);
        const uint32_t b = bin_at(sh.sub.upto, sh.sub.mass, goal == GOAL_K, rest);
        const uint32_t bc = b ? sh.sub.upto[b - 1] : 0, n = sh.sub.upto[b] - bc;
        const unsigned long long bm = b ? sh.sub.mass[b - 1] : 0, m = sh.sub.mass[b] - bm;
        Command next{};
        next.by_bin = -1;
        next.hi = cmd.hi - (b << cmd.shift);
        const uint32_t down = (1u << cmd.shift) - 1u;
        next.lo = next.hi - cmd.lo > down ? next.hi - down : cmd.lo;
        before_c += bc;
        before_m += bm;
        __syncthreads();
        if (n <= LIST) {
          next.op = OP_GATHER;
        } else if (cmd.shift) {
          next.op = OP_BINS;
          while ((next.hi - next.lo) >> next.shift >= BINS) ++next.shift;
        } else {
          // tokens of one score, all of the same weight: by their number
          const unsigned long long one = m / n, left = target - (goal == GOAL_K ? (unsigned long long)before_c : before_m);
          const uint32_t nth = goal == GOAL_K ? (uint32_t)left : one ? (uint32_t)((left + one - 1) / one) : 1u;
          pick_key = next.lo;
          if (goal == GOAL_U) {
            next.op = OP_NTH;
            next.nth = nth;
          } else {
            answered(before_c + nth, before_m + nth * one);
          }
        }
        if (tid == 0) sh.cmd = next;
        __syncthreads();
      }
    } else {
      // the nth token of one score, in the order of ids: each thread counts its run of elements
      const T* x = static_cast<const T*>(s.at);
      const uint32_t n = s.to - s.from, per = (n + THREADS - 1) / THREADS, e0 = min(tid * per, n), e1 = min(e0 + per, n);
      uint32_t mine = 0;
      for (uint32_t e = e0; e < e1; ++e) mine += key_of(to_f32(x[e])) == cmd.lo;
      uint32_t at = mine, all;
      unsigned long long zero = 0, zeros;
      block_scan<WARPS>(sh, at, zero, all, zeros);
      if (tid < c.ranks) cluster.map_shared_rank(&sh, tid)->part_cnt[rank] = all;
      cluster.sync();
      for (uint32_t i = 0; i < rank; ++i) at += sh.part_cnt[i];
      if (at < cmd.nth && cmd.nth <= at + mine) {
        for (uint32_t e = e0; e < e1; ++e)
          if (key_of(to_f32(x[e])) == cmd.lo && ++at == cmd.nth) cluster.map_shared_rank(&sh, 0)->found = s.from + e;
      }
      cluster.sync();
      if (rank == 0) answered(0, 0);
    }
    if (rank == 0 && goal == GOAL_END) {
      __syncthreads();
      if (tid == 0) {
        c.a.d_pick[row] = (int32_t)sh.found;
        if (c.a.d_kept) c.a.d_kept[row] = (int32_t)kept;
        if (c.a.d_logprob) {
          float hi, lo;
          log2_weight(r, of_key(pick_key), hi, lo);
          c.a.d_logprob[row] = (float)(((double)hi + lo) * 0.693147180559945309417 - log((double)kept_m / ONE));
        }
      }
      __syncthreads();
    }
  }
  // (min-p above 1 keeps nothing; commands do not run out)
  if (rank == 0 && tid == 0 && (kept == 0 || goal != GOAL_END)) {
    c.a.d_pick[row] = -1;
    if (c.a.d_kept) c.a.d_kept[row] = 0;
    if (c.a.d_logprob) c.a.d_logprob[row] = -INFINITY;
  }
}

constexpr int SAMPLE_THREADS = 512, SAMPLE_BINS = 11, FEW_BINS = 12;   // (BIN_SHIFT; fewer where counts share the memory)
template <class T>
__global__ void __launch_bounds__(SAMPLE_THREADS, 2) k_sample(const __grid_constant__ SampleCall c) {
  extern __shared__ __align__(16) uint8_t mem[];
  choose<T, SAMPLE_THREADS, SAMPLE_BINS>(c, mem);
}

// --- 16-bit scores -------------------------------------------------------------------

// A row of 16-bit scores has few different ones: they are counted, score by score, and
// a weight is formed once for each.  What lies below -2^11 is only counted, and must have
// no weight; a row with other scores (2^11 or more, below 2^-27 in bf16, NaN) takes the
// way above.
template <class T> struct Places;
template <> struct Places<__nv_bfloat16> {
  static constexpr uint32_t LOW = 100u << 7, HIGH = 138u << 7, INF = 0x7f80;   // the bits of 2^-27, 2^11
  static constexpr int THREADS = 256, ROUNDS = 8;                              // four CTAs per SM
  using Count = uint32_t;
};
template <> struct Places<__half> {
  static constexpr uint32_t LOW = 0, HIGH = 26u << 10, INF = 0x7c00;           // all but 0, 2^11
  static constexpr int THREADS = 1024, ROUNDS = 2;                             // one
  using Count = uint16_t;                                                      // (as words they would not fit)
};
constexpr float FAR = -2048.f;
constexpr int GROUP = 256;                 // places of a warp's step

// Counts lie by size, positive scores first, then negative ones, then 0.  In the order
// of falling scores (places): the positive ones backwards, a group with 0, the others.
template <class T> struct Counts {
  static constexpr uint32_t RANGE = Places<T>::HIGH - Places<T>::LOW, N = 2 * RANGE + GROUP, GROUPS = N / GROUP;
  static_assert(RANGE % GROUP == 0);
  using Count = typename Places<T>::Count;
  static constexpr bool WORDS = sizeof(Count) == 4;
  Pow pow[256];
  Fine fine[256];
  __align__(16) Count at[N];
  // the first CTA's: of eight places each (up to them in the group), and of each group, then up to each
  unsigned long long lane_mass[GROUPS * 32], mass[GROUPS];
  uint32_t upto[GROUPS];
  uint32_t part_best[16], part_far[16], part_odd[16], part_cnt[16];
  uint32_t part_some[16][(GROUPS + 31) / 32];   // which groups have tokens in each CTA
  uint32_t best, far, odd, some[(GROUPS + 31) / 32];
  uint32_t cell[64];                       // of the search
  Rule rule;
  double t_ln_m;
  uint32_t pick_bits, nth;                 // the choice is the nth of this score (nth 0: there is none)

  // a place's score, and where its count lies
  static __device__ __forceinline__ uint32_t bits(uint32_t place) {
    return place < RANGE ? Places<T>::HIGH - 1 - place : place < RANGE + GROUP ? 0u : 0x8000u | (place - RANGE - GROUP + Places<T>::LOW);
  }
  static __device__ __forceinline__ float score(uint32_t place) {
    if (WORDS) return __uint_as_float(bits(place) << 16);
    return __half2float(__ushort_as_half((unsigned short)bits(place)));
  }
  static __device__ __forceinline__ uint32_t lies(uint32_t place) {
    return place < RANGE ? RANGE - 1 - place : place < RANGE + GROUP ? place + RANGE : place - GROUP;
  }
  __device__ __forceinline__ void add(uint32_t lies, uint32_t n) {
    if (WORDS) atomicAdd(reinterpret_cast<uint32_t*>(at) + lies, n);
    else atomicAdd(reinterpret_cast<uint32_t*>(at) + (lies >> 1), n << (lies & 1u) * 16);
  }
  // one more, without a branch (from: the shared address of at)
  static __device__ __forceinline__ void add_if(uint32_t from, uint32_t lies, bool really) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p red.shared.add.u32 [%0], %1; }" ::
                 "r"(WORDS ? from + lies * 4 : from + (lies >> 1) * 4), "r"(WORDS ? 1u : 1u << (lies & 1u) * 16), "r"((uint32_t)really) : "memory");
  }
  // the counts of eight places side by side are added to n (place: a multiple of 8)
  __device__ __forceinline__ void eight(uint32_t place, uint32_t* n) const {
    const uint4* p = reinterpret_cast<const uint4*>(at + (place < RANGE ? RANGE - 8 - place : lies(place)));
    const uint4 a = p[0], b = WORDS ? p[1] : a;
    uint32_t v[8];
    if (WORDS) {
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = a.x & 0xffffu; v[1] = a.x >> 16; v[2] = a.y & 0xffffu; v[3] = a.y >> 16;
      v[4] = a.z & 0xffffu; v[5] = a.z >> 16; v[6] = a.w & 0xffffu; v[7] = a.w >> 16;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] += place < RANGE ? v[7 - i] : v[i];
  }
};

// sums over the lanes before, and up to this one
__device__ __forceinline__ void warp_scan(uint32_t& c, unsigned long long& m) {
  const uint32_t lane = threadIdx.x & 31u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t pc = __shfl_up_sync(ALL, c, o);
    const unsigned long long pm = __shfl_up_sync(ALL, m, o);
    if (lane >= (uint32_t)o) {
      c += pc;
      m += pm;
    }
  }
}

// true: the row is done; false: it has scores that this way does not take (in all CTAs alike)
template <class T>
__device__ __forceinline__ bool choose_counted(const SampleCall& c, uint8_t* mem) {
  using C = Counts<T>;
  constexpr int COUNT_THREADS = Places<T>::THREADS, COUNT_WARPS = COUNT_THREADS / 32;
  constexpr uint32_t ROUNDS = Places<T>::ROUNDS;   // of the search for the choice, of 256 pieces a warp, at most
  constexpr uint32_t RANGE = C::RANGE, LOW = Places<T>::LOW;
  C& sh = *reinterpret_cast<C*>(mem);
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), row = blockIdx.x / c.ranks, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t V = c.a.n_logits;
  Slice s;
  s.from = min(rank * c.per, V);
  s.to = min(s.from + c.per, V);
  const uint16_t* src = static_cast<const uint16_t*>(c.a.d_scores) + (long long)row * c.a.scores_stride + s.from;
  s.at = src;
  const float temp = c.a.d_temperature ? c.a.d_temperature[row] : 1.f;
  const float min_p = c.a.d_min_p ? c.a.d_min_p[row] : 0.f;
  for (uint32_t i = tid; i < sizeof(sh.at) / 16; i += COUNT_THREADS) reinterpret_cast<uint4*>(sh.at)[i] = make_uint4(0, 0, 0, 0);
  for (uint32_t i = tid; i < 256; i += COUNT_THREADS) {
    sh.pow[i] = g_powers.a[i];
    sh.fine[i] = g_powers.b[i];
  }
  if (tid == 32) {
    set_temperature(sh.rule, temp);
    sh.t_ln_m = t_ln(temp, min_p);
  }
  if (tid == 0) {
    sh.best = ALL;
    sh.far = sh.odd = 0;
    for (uint32_t& x : sh.some) x = 0;
  }
  if (tid < 64) sh.cell[tid] = 0;
  __syncthreads();

  // the scores are counted
  uint32_t best = ALL, far = 0, odd = 0, zero = 0;
  auto count = [&](uint32_t u) {
    const uint32_t m = u & 0x7fffu, q = m - LOW, neg = u >> 15;
    if (m == 0) {
      ++zero;
    } else if (q < RANGE) {
      sh.add(q + neg * RANGE, 1);
    } else if (neg && m > LOW && m <= Places<T>::INF) {
      far += m < Places<T>::INF;   // (-inf is no token)
    } else {
      odd = 1;
    }
  };
  const uint32_t n_mine = s.to - s.from;
  const uint32_t head = min(n_mine, (uint32_t)((16u - (reinterpret_cast<uintptr_t>(src) & 15u)) & 15u) / 2u);
  const uint32_t vecs = (n_mine - head) / 8, tail = head + vecs * 8;
  const uint4* pieces = reinterpret_cast<const uint4*>(src + head);
  if (tid < head + (n_mine - tail)) count(src[tid < head ? tid : tail + (tid - head)]);   // (14 at most)
  const uint32_t counts = (uint32_t)__cvta_generic_to_shared(sh.at);
  auto count_piece = [&](const uint4& q) {
    // two scores in each operation: their sizes' range, their places, an atomic for each
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = w[i] & 0x7fff7fffu;
    const uint32_t hi = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
    const uint32_t lo = __vminu2(__vminu2(m[0], m[1]), __vminu2(m[2], m[3]));
    if (max(hi & 0xffffu, hi >> 16) < Places<T>::HIGH && min(lo & 0xffffu, lo >> 16) >= max(LOW, 1u)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at2 = m[i] + (w[i] >> 15 & 0x00010001u) * RANGE;
        sh.add((at2 & 0xffffu) - LOW, 1);
        sh.add((at2 >> 16) - LOW, 1);
      }
    } else {
      // (masked rows: what is -inf is passed over, what else has no place comes after)
      uint32_t left = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu, x = u & 0x7fffu;
        const bool in = x - LOW < RANGE && x;
        C::add_if(counts, x - LOW + (u >> 15) * RANGE, in);
        left |= (in || u == (0x8000u | Places<T>::INF) ? 0u : 1u) << i;
      }
      for (; left; left &= left - 1) {
        const uint32_t i = __ffs(left) - 1;
        const uint32_t x = i & 4u ? (i & 2u ? w[3] : w[2]) : (i & 2u ? w[1] : w[0]);
        count(i & 1u ? x >> 16 : x & 0xffffu);
      }
    }
  };
  constexpr int AHEAD = 3;   // pieces under way while as many are counted
  uint4 q[AHEAD];
  auto fetch = [&](uint32_t i) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (i + u * COUNT_THREADS < vecs) q[u] = __ldg(pieces + i + u * COUNT_THREADS);
  };
  fetch(tid);
  for (uint32_t i = tid; i < vecs; i += AHEAD * COUNT_THREADS) {
    uint4 now[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) now[u] = q[u];
    fetch(i + AHEAD * COUNT_THREADS);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (i + u * COUNT_THREADS < vecs) count_piece(now[u]);
  }
  zero = __reduce_add_sync(ALL, zero);
  if (lane == 0 && zero) sh.add(2 * RANGE, zero);
  __syncthreads();
  // the groups that have tokens, and the largest score: the first place that has one
  for (uint32_t g = warp; g < C::GROUPS; g += COUNT_WARPS) {
    uint32_t n[8] = {};
    sh.eight(g * GROUP + lane * 8, n);
    uint32_t mine = ALL;
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (n[i]) mine = g * GROUP + lane * 8 + i;
    const bool any = __any_sync(ALL, mine != ALL);
    if (any && lane == 0) atomicOr(&sh.some[g >> 5], 1u << (g & 31u));
    best = min(best, mine);
  }
  best = __reduce_min_sync(ALL, best);
  far = __reduce_add_sync(ALL, far);
  odd = __any_sync(ALL, odd);
  if (lane == 0) {
    atomicMin(&sh.best, best);
    if (far) atomicAdd(&sh.far, far);
    if (odd) sh.odd = 1;
  }
  __syncthreads();
  if (tid < c.ranks) {
    C* o = cluster.map_shared_rank(&sh, tid);
    o->part_best[rank] = sh.best;
    o->part_far[rank] = sh.far;
    o->part_odd[rank] = sh.odd;
    for (uint32_t i = 0; i < (C::GROUPS + 31) / 32; ++i) o->part_some[rank][i] = sh.some[i];
  }
  cluster.sync();
  best = ALL;
  far = odd = 0;
  for (uint32_t i = 0; i < c.ranks; ++i) {
    best = min(best, sh.part_best[i]);
    far += sh.part_far[i];
    odd |= sh.part_odd[i];
  }
  if (odd || (best == ALL && far) || !(temp >= 0.f)) {
    cluster.sync();
    return false;
  }
  if (best == ALL) {
    if (rank == 0 && tid == 0) {
      c.a.d_pick[row] = -1;
      if (c.a.d_kept) c.a.d_kept[row] = 0;
      if (c.a.d_logprob) c.a.d_logprob[row] = -INFINITY;
    }
    return true;
  }
  Rule r = sh.rule;
  set_largest(r, C::score(best));
  const float least = least_of(r, temp, min_p, sh.t_ln_m);
  const int top_k = c.a.d_top_k ? c.a.d_top_k[row] : 0;
  if (far) {
    // the scores far down have no weight, and no rule reaches in among them
    float hi, lo;
    log2_weight(r, FAR, hi, lo);
    if (hi >= LOWEST || (min_p > 0.f && least <= FAR)) {
      cluster.sync();
      return false;
    }
    if (min_p > 0.f) far = 0;
  }
  auto weight_of = [&](uint32_t place, uint32_t& n) {   // (n 0: below min-p's scores)
    const float x = C::score(place);
    if (!(x >= least)) n = 0;
    float hi, lo, rest = 0.f;
    log2_weight(r, x, hi, lo);
    const int k = fixed_log2(hi, lo, rest);
    return weight(sh.pow, sh.fine, k, rest);
  };
  C* first = cluster.map_shared_rank(&sh, 0);
  C* second = cluster.map_shared_rank(&sh, c.ranks > 1 ? 1 : 0);
  for (uint32_t g = warp * c.ranks + rank; g < C::GROUPS; g += COUNT_WARPS * c.ranks) {
    const uint32_t place = g * GROUP + lane * 8;
    uint32_t n[8] = {}, all = 0;
    unsigned long long m = 0;
#pragma unroll 4
    for (uint32_t k = 0; k < c.ranks; ++k)   // (reading another CTA's memory is slow: only where it has tokens)
      if (sh.part_some[k][g >> 5] >> (g & 31u) & 1u) cluster.map_shared_rank(&sh, k)->eight(place, n);
    if (__any_sync(ALL, n[0] | n[1] | n[2] | n[3] | n[4] | n[5] | n[6] | n[7])) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!__any_sync(ALL, n[i])) continue;
        const unsigned long long w = weight_of(place + i, n[i]);
        all += n[i];
        m += n[i] * w;
      }
      // the row's counts stay with the first CTA (or 16 bits of them, the others with the second)
      if (c.ranks > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          first->at[C::lies(place + i)] = (typename C::Count)n[i];
          if (!C::WORDS) second->at[C::lies(place + i)] = (typename C::Count)(n[i] >> 16);
        }
      }
    }
    warp_scan(all, m);
    first->lane_mass[g * 32 + lane] = m;
    if (lane == 31) {
      first->upto[g] = all;
      first->mass[g] = m;
    }
  }
  cluster.sync();

  // the first CTA's first warp finds the borders
  uint32_t kept = 0, pick_place = 0;
  unsigned long long kept_m = 0;
  if (rank == 0 && warp == 0) {
    for (uint32_t g0 = 0; g0 < C::GROUPS; g0 += 32) {
      uint32_t n = g0 + lane < C::GROUPS ? sh.upto[g0 + lane] : 0;
      unsigned long long m = g0 + lane < C::GROUPS ? sh.mass[g0 + lane] : 0;
      warp_scan(n, m);
      n += kept;
      m += kept_m;
      if (g0 + lane < C::GROUPS) {
        sh.upto[g0 + lane] = n;
        sh.mass[g0 + lane] = m;
      }
      kept = __shfl_sync(ALL, n, 31);
      kept_m = __shfl_sync(ALL, m, 31);
    }
    __syncwarp();
    const uint32_t near = kept;
    uint32_t place = 0, nth = 0;
    // the token at which a sum reaches the target: its place, its number among that
    // score's, how many tokens and what mass there are up to it
    auto reach = [&](bool by_count, unsigned long long target, uint32_t& cnt, unsigned long long& mass) {
      uint32_t g = 0;
      for (uint32_t g0 = 0; g0 < C::GROUPS; g0 += 32) {
        const bool below = g0 + lane < C::GROUPS && (by_count ? (unsigned long long)sh.upto[g0 + lane] : sh.mass[g0 + lane]) < target;
        g += __popc(__ballot_sync(ALL, below));
      }
      g = min(g, C::GROUPS - 1);
      uint32_t at_n = g ? sh.upto[g - 1] : 0;
      unsigned long long at_m = g ? sh.mass[g - 1] : 0;
      // the eight places, then the place, by a lane for each
      uint32_t n8[8] = {}, lane_n = 0;
      sh.eight(g * GROUP + lane * 8, n8);
      if (!C::WORDS && c.ranks > 1) {
        uint32_t top[8] = {};
        second->eight(g * GROUP + lane * 8, top);
#pragma unroll
        for (int i = 0; i < 8; ++i) n8[i] |= top[i] << 16;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (C::score(g * GROUP + lane * 8 + i) >= least) lane_n += n8[i];
      unsigned long long no_mass = 0;
      warp_scan(lane_n, no_mass);
      lane_n += at_n;
      const unsigned long long lane_m = at_m + sh.lane_mass[g * 32 + lane];
      const uint32_t e = min((uint32_t)__popc(__ballot_sync(ALL, (by_count ? (unsigned long long)lane_n : lane_m) < target)), 31u);
      if (e) {
        at_n = __shfl_sync(ALL, lane_n, e - 1);
        at_m = __shfl_sync(ALL, lane_m, e - 1);
      }
      const uint32_t p = g * GROUP + e * 8 + (lane & 7u);
      uint32_t n = sh.at[C::lies(p)];
      if (!C::WORDS && c.ranks > 1) n |= (uint32_t)second->at[C::lies(p)] << 16;
      if (lane >= 8) n = 0;
      const unsigned long long w = weight_of(p, n);
      uint32_t upto_n = n;
      unsigned long long upto_m = n * w;
      warp_scan(upto_n, upto_m);
      upto_n += at_n - n;
      upto_m += at_m - n * w;
      // (the place's first token's sums are above upto, without it)
      const bool in = n && (by_count ? upto_n < target && upto_n + n >= target : upto_m < target && upto_m + n * w >= target);
      uint32_t nth_here = 0;
      if (in) nth_here = by_count ? (uint32_t)(target - upto_n) : (uint32_t)((target - upto_m + w - 1) / w);
      const uint32_t who = __ffs(__ballot_sync(ALL, in)) - 1;
      place = __shfl_sync(ALL, p, who);
      nth = __shfl_sync(ALL, nth_here, who);
      cnt = __shfl_sync(ALL, upto_n + nth_here, who);
      mass = __shfl_sync(ALL, upto_m + nth_here * w, who);
    };
    kept += far;
    if (top_k > 0 && (uint32_t)top_k < kept) {
      if ((uint32_t)top_k > near) kept = (uint32_t)top_k;   // (among those without weight)
      else reach(true, (uint32_t)top_k, kept, kept_m);
    }
    const float top_p = c.a.d_top_p ? c.a.d_top_p[row] : 1.f;
    if (kept && top_p < 1.f) {
      reach(false, enough(top_p, kept_m), kept, kept_m);
    }
    uint32_t bits = 0;
    if (kept) {
      uint32_t n;
      unsigned long long m;
      reach(false, chosen_at(c.a.d_random[row], kept_m), n, m);
      bits = C::bits(place);
    }
    if (lane < c.ranks) {
      C* o = cluster.map_shared_rank(&sh, lane);
      o->pick_bits = bits;
      o->nth = kept ? nth : 0;
    }
    pick_place = place;
  }
  cluster.sync();
  const uint32_t nth = sh.nth;
  auto finish = [&] {   // (by the first warp, which has no part in the search below)
    if (rank || tid) return;
    if (c.a.d_kept) c.a.d_kept[row] = (int32_t)kept;
    if (c.a.d_logprob) {
      float hi, lo;
      log2_weight(r, C::score(pick_place), hi, lo);
      c.a.d_logprob[row] = kept ? (float)(((double)hi + lo) * 0.693147180559945309417 - log((double)kept_m / ONE)) : -INFINITY;
    }
    if (!kept) c.a.d_pick[row] = -1;
  };
  if (nth == 0) {
    finish();
    return true;
  }
  // The nth token of that score in the order of ids.  The slice is searched in rounds,
  // in each of which a warp has a run of 256 pieces; a row that one CTA has is searched
  // no further than needed.  Cells, in order: the scores before the first piece, each
  // round's warps, the scores after the last piece.
  const uint32_t want = sh.pick_bits, mask = want ? 0xffffu : 0x7fffu, want2 = want | want << 16, mask2 = mask | mask << 16;
  auto same = [&](uint32_t u) { return (u & mask) == want; };
  auto match = [&](const uint4& q) {   // of the eight scores of a piece, as bits
    const uint32_t x[4] = {(q.x & mask2) ^ want2, (q.y & mask2) ^ want2, (q.z & mask2) ^ want2, (q.w & mask2) ^ want2};
    const uint32_t least = __vminu2(__vminu2(x[0], x[1]), __vminu2(x[2], x[3]));
    uint32_t m = 0;
    if (!(least & 0xffffu) || !(least >> 16)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) m |= (x[i] & 0xffffu ? 0u : 1u) << (2 * i) | (x[i] >> 16 ? 0u : 2u) << (2 * i);
    }
    return m;
  };
  constexpr uint32_t SEARCH = COUNT_WARPS - 1, LAST = 1 + ROUNDS * SEARCH;
  const bool has_head = warp == 1 && lane < head && same(src[lane]);
  const bool has_tail = warp == 1 && lane < n_mine - tail && same(src[tail + lane]);
  if (warp == 1) {
    const uint32_t h = __popc(__ballot_sync(ALL, has_head)), t = __popc(__ballot_sync(ALL, has_tail));
    if (lane == 0) {
      sh.cell[0] = h;
      sh.cell[LAST] = t;
    }
  }
  unsigned long long steps = 0;   // in which the lane found some
  uint4 p[8];                     // the pieces of the next round
  auto get = [&](uint32_t k) {
    const uint32_t v0 = (k * SEARCH + warp - 1) * 256 + lane;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (warp && v0 + i * 32 < vecs) p[i] = __ldg(pieces + v0 + i * 32);
  };
  get(0);
  for (uint32_t k = 0; k * SEARCH * 256 < vecs; ++k) {
    uint32_t mine = 0;
    if (warp) {
      const uint32_t v0 = (k * SEARCH + warp - 1) * 256 + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = v0 + i * 32 < vecs ? match(p[i]) : 0u;
        mine += __popc(m);
        if (m) steps |= 1ull << (k * 8 + i);
      }
      get(k + 1);
      mine = __reduce_add_sync(ALL, mine);
      if (lane == 0) sh.cell[1 + k * SEARCH + warp - 1] = mine;
    }
    if (c.ranks == 1) {
      __syncthreads();
      uint32_t found = lane <= (k + 1) * SEARCH ? sh.cell[lane] : 0;
      if (lane + 32 <= (k + 1) * SEARCH) found += sh.cell[lane + 32];
      if (__reduce_add_sync(ALL, found) >= nth) break;   // (all warps alike)
    }
  }
  __syncthreads();
  const uint32_t c0 = sh.cell[lane], c1 = sh.cell[lane + 32];
  uint32_t before = 0;
  if (c.ranks > 1) {
    const uint32_t all = __reduce_add_sync(ALL, c0 + c1);
    if (tid < c.ranks) cluster.map_shared_rank(&sh, tid)->part_cnt[rank] = all;
    cluster.sync();
    for (uint32_t i = 0; i < rank; ++i) before += sh.part_cnt[i];
  }
  // sums up to each cell: in which one it is, and as which of its tokens
  uint32_t s0 = c0, s1 = c1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t p0 = __shfl_up_sync(ALL, s0, o), p1 = __shfl_up_sync(ALL, s1, o);
    if (lane >= (uint32_t)o) {
      s0 += p0;
      s1 += p1;
    }
  }
  s0 += before;
  s1 += __shfl_sync(ALL, s0, 31);
  const uint32_t in0 = __ballot_sync(ALL, s0 - c0 < nth && nth <= s0), in1 = __ballot_sync(ALL, s1 - c1 < nth && nth <= s1);
  finish();
  if (!(in0 | in1)) return true;   // (another CTA's)
  const uint32_t cell = in0 ? __ffs(in0) - 1 : 31 + __ffs(in1);
  uint32_t left = nth - (in0 ? __shfl_sync(ALL, s0 - c0, cell) : __shfl_sync(ALL, s1 - c1, cell - 32));
  if (cell == 0 || cell == LAST) {
    if (warp == 1) {
      const uint32_t m = __ballot_sync(ALL, cell ? has_tail : has_head);
      if (lane == 0) c.a.d_pick[row] = (int32_t)(s.from + (cell ? tail : 0u) + __fns(m, 0, (int)left));
    }
    return true;
  }
  const uint32_t k = (cell - 1) / SEARCH;
  if (warp != 1 + (cell - 1) % SEARCH) return true;
  for (uint32_t i = 0; i < 8; ++i) {
    const bool some = steps >> (k * 8 + i) & 1;
    if (!__any_sync(ALL, some)) continue;
    const uint32_t v = (cell - 1) * 256 + i * 32 + lane, m = some ? match(__ldg(pieces + v)) : 0u, mine = __popc(m);
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t p = __shfl_up_sync(ALL, upto, o);
      if (lane >= (uint32_t)o) upto += p;
    }
    if (upto - mine < left && left <= upto)
      c.a.d_pick[row] = (int32_t)(s.from + head + v * 8 + __fns(m, 0, (int)(left - (upto - mine))));
    const uint32_t total = __shfl_sync(ALL, upto, 31);
    if (total >= left) break;
    left -= total;
  }
  return true;
}

template <class T>
__device__ __noinline__ void choose_any(const SampleCall& c, uint8_t* mem) { choose<T, Places<T>::THREADS, FEW_BINS>(c, mem); }

template <class T>
__global__ void __launch_bounds__(Places<T>::THREADS, 1024 / Places<T>::THREADS) k_sample_counted(const __grid_constant__ SampleCall c) {
  extern __shared__ __align__(16) uint8_t mem[];
  if (!choose_counted<T>(c, mem)) choose_any<T>(c, mem);
}

// More CTAs for a row while all of them run at once (fit: on an SM) and each keeps `few`
// scores: adding up bins over a cluster costs more than it gains from there.  us with 1,
// 2, 4 and 8 CTAs for a row of bf16 (16,384 scores): 64 rows of 50,257 27, 23, 25, 32; 512
// of 100,257 70, 78, 119, 192; one of 100,257 27, 25, 23, 21; 150 39, 33, 47, 70.  Of f16 (16,384): one
// row of 50,257 33, 35, 36, 35; 64 33, 37, 74, 155; 150 35, 72, 157, 317; of 100,257 from 2 on
// (counts of 16 bits take 63,000 scores) one 37, 38, 36; 512 253, 510, 1,091.  Of f32 (4,096), with
// 16 CTAs last: one row of 100,257 with top-p 108, 65, 43, 33, 31; 16 147, 93, 62, 48, 70; 64 166, 103,
// 78, 95, 190; 150 163, 125, 144, 197; 512 388, 358, 416, 615 (`most` is 65,536: at least 2 there,
// where 300 rows take 227, 233); of 50,257 300 124, 146, 179; of 8,192 one 23, 21, 19, 21; 64 39, 36, 37,
// 60; 300 47, 61, 99.
void split(const tok_handle* h, uint32_t fit, uint32_t most, uint32_t few, SampleCall& c) {
  const uint32_t V = c.a.n_logits;
  uint32_t n = 1;
  while (n < 16 && (V / n > most || (V / n > few && (uint64_t)c.a.rows * n * 2 <= (uint64_t)fit * (uint32_t)h->n_sms))) n *= 2;
  c.ranks = n;
  c.per = ((V + n - 1) / n + 7) / 8 * 8;
}

template <class T>
cudaError_t launch(tok_handle* h, const tok_sample_args* a, cudaStream_t s) {
  SampleCall c{};
  c.a = *a;
  if constexpr (sizeof(T) == 2) {
    // a CTA's counts have to fit their type, and its slice the search for the choice
    constexpr bool WORDS = Counts<T>::WORDS;
    constexpr uint32_t most = std::min<uint32_t>(WORDS ? MOST_LOGITS : 63000u, (Places<T>::THREADS / 32 - 1) * Places<T>::ROUNDS * 2048 - 8);
    const size_t room = std::max(sizeof(Shared<FEW_BINS>), sizeof(Counts<T>));
    split(h, (uint32_t)std::min<size_t>(1024 / Places<T>::THREADS, 228 * 1024 / (room + 1024)), most, 16384, c);
    // (2^20 f16 scores are too many for 16 CTAs)
    if (WORDS || c.per <= most + 8)
      return launch_clusters<k_sample_counted<T>>(h->dev, a->rows * c.ranks, Places<T>::THREADS, c.ranks, room, s, c);
  }
  if constexpr (!std::is_same_v<T, __nv_bfloat16>) {
    split(h, 2, 65536, 4096, c);
    const size_t base = (sizeof(Shared<SAMPLE_BINS>) + 15) & ~size_t(15), slice = (size_t)c.per * sizeof(T) + 16;
    c.resident = base + slice <= 112 * 1024;   // (two CTAs per SM: 256 rows of 100,257 scores 226 us, with one that keeps them 330)
    return launch_clusters<k_sample<T>>(h->dev, a->rows * c.ranks, SAMPLE_THREADS, c.ranks, base + (c.resident ? slice : 0), s, c);
  }
  return cudaErrorInvalidValue;   // (not reached)
}

}  // namespace
}  // namespace tokgb

using namespace tokgb;

extern "C" {

int tok_sample(tok_handle* h, const tok_sample_args* a, void* stream) try {
  if (!h) return TOK_EINVAL;
  if (a && a->rows == 0) return TOK_OK;
  if (!a || !a->d_scores || !a->d_random || !a->d_pick) return fail(h, TOK_EINVAL, "sample: a buffer is NULL");
  if (!element_size(a->dtype)) return fail(h, TOK_EINVAL, "sample: unknown type");
  if (a->n_logits == 0 || a->n_logits > MOST_LOGITS || a->rows > 0x7ffffffu || a->scores_stride < (int64_t)a->n_logits)
    return fail(h, TOK_EINVAL, "sample: rows, n_logits or scores_stride is out of range");
  if (!lies_at(a->d_scores, element_size(a->dtype)) || !lies_at(a->d_temperature, 4) || !lies_at(a->d_min_p, 4) ||
      !lies_at(a->d_top_k, 4) || !lies_at(a->d_top_p, 4) || !lies_at(a->d_random, 4) || !lies_at(a->d_pick, 4) ||
      !lies_at(a->d_kept, 4) || !lies_at(a->d_logprob, 4))
    return fail(h, TOK_EINVAL, "sample: an array does not lie at a multiple of its type's size");
  DeviceGuard g(h->dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == TOK_F32 ? launch<float>(h, a, s) : a->dtype == TOK_F16 ? launch<__half>(h, a, s)
                                                                                             : launch<__nv_bfloat16>(h, a, s);
  h->launches += 1;
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TOK_OK : cuda_fail(h, e, "kernel launch");
} catch (...) {
  return TOK_ENOMEM;
}

}  // extern "C"
