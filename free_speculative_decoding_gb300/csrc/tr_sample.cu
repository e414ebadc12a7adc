// Sampling: one token of each row of logits, with temperature, top-k, top-p and min-p,
// from given uniforms.
//
// Weights w = 2^((x - m) log2(e) / T), m the row's maximum, are held as integers in units of
// 2^-S, so their sums are exact and do not depend on the order: top-p's edge is found
// from sums over any grouping, and equal calls give equal bits.  A token is left when its key
// (the order of its logit) is above the row's edge, or at it with an ID up to the edge's.
//
// A row is worked on by a cluster of one to eight CTAs.  Few rows lie in its shared memory, copied once; many
// are read from global memory in every pass (the first from DRAM, the others mostly from L2).
// The first pass finds the largest logit, and of each warp a logit that a known number of tokens reach.  top-k's
// candidates are the tokens that reach enough of these, some k to 3 k of them; top-p's are found
// from a histogram of the weights' first 16 bits over a linear scale of the logits, whose error is
// bounded, as the tokens of the bins that the edge must lie in, a few hundred at most.  The candidates go to a
// list, which is merged over the cluster and sorted, and the edge is read off exact sums.  Where they
// are more than the list holds (long runs of equal logits) the key is narrowed down by eight
// bits a pass instead.  The draw then goes from the warps' sums to one warp's range, an eighth of it, a batch and a
// token.  With a temperature alone, in rows that are read from global memory, the weights are summed in the first pass
// already, relative to the warp's largest logit so far.  These sums are cut whenever that rises, so they are not the exact
// ones: by two units for each lane and one for the warp, within the stated bound, but a row that lies in shared
// memory in a call of fewer rows can differ in a last bit, or in its token next to a border.
//
// What bounds it: single rows a chain of latencies (some fifteen passes and barriers, those of a cluster about 1 us each,
// instructions fetched for the first time); many rows the latencies of their passes (1280 rows of mixed rules: issue slots
// 36% busy, warps wait for L2, at barriers and for instructions).  Measured in a graph,
// 1280 x 32000 fp32 (the bytes alone take 24 us): greedy 44 us, temperature 86, min_p 90, top-k 50 97, top-p 0.9 185 to
// 200, top-k 900 248, rows of mixed rules 178.  One row of 32000: 4.0, 7.8, 8.4, 12, 18 and 32 us.  64 x 128256 bf16:
// 8.5, 24, 25, 20, 43 to 58 and 67 us.
#include <cfloat>
#include <cmath>
#include <cstddef>
#include <cstring>

#include <atomic>

#include <cooperative_groups.h>

#include "tr_internal.cuh"

namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

struct SampleArgs {
  const void *x;
  long long ld, rows;
  int V, S;  // weights are in units of 2^-S
  const float *temperature, *top_p, *min_p, *U;
  const int32_t *top_k;
  int32_t *token;
  float *logprob;
  int granules;  // of a CTA's slice, its threads or a multiple
  int full;      // warps of a row's cluster whose ranges hold nothing but tokens, at least
  int drop;      // bits that top-p's histogram gives up
};

// The order of a logit; NaN and -inf (never drawn) are 0x007FFFFF, below every other.
constexpr uint32_t kNever = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float x) { return x == x ? tr_ord(x) : kNever; }

// Two fp32 values in one register pair, and one instruction.
struct F2 {
  u64 v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {  // a b + c
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c.v) : "l"(a.v), "l"(b.v));
  return c;
}

// Weights of a row: 2^S 2^(x c - K), c = log2(e) / T and K a whole number above m c by 1.02 at most, rounded
// down.  x c is split into a multiple of 1 / 64 (adding and taking away 1.5 2^17 rounds to it) and a
// rest whose error is below 2^-31; the multiple's power of two comes from a table, the rest's from a
// polynomial.  Where |m c| passes 2^15, x is taken relative to m first: what has weight then
// lies so near to m that the difference is exact.  A weight below 2^-S is 0.
constexpr float kL1 = 6.931471805599453e-1f, kL2 = 2.402265069591007e-1f, kL3 = 5.550410866482158e-2f;  // ln2^i / i!
struct Weight {
  float m, base, c_hi, c_lo;
  float floor;          // logits up to this one have no weight
  int shift, S;         // shift: (K - (bits of 0 + 1.5 2^17) / 64) + 63 - S, see whole()
  bool infinite;        // the largest logit is +inf
  bool far;
  const float2 *table;  // 2^(j / 64): 2^31 times it as a float, and as an integer (in its bits)
  __device__ __forceinline__ void set(float m_, float2 c, int S_, const float2 *t) {
    m = m_;
    S = S_;
    table = t;
    c_hi = c.x;
    c_lo = c.y;
    infinite = m == INFINITY;
    const float mc = m * c_hi;
    far = !(fabsf(mc) < 32700.f);  // infinite too
    base = far ? m : 0.f;
    const int K = far ? 1 : (int)ceilf(mc + 0.01f);  // m c is off by 2^-9 at most
    shift = K + (0x48400000 >> 6) + 63 - S;
    floor = infinite ? FLT_MAX : m - (float)(S - 2) / c_hi;  // an infinite temperature: -inf
    if (floor == m) floor = tr_unord(tr_ord(m) - 1);         // the next number already is too far below
  }
  // From p = q + 1.5 2^17, whose bits are 64 q more than those of 1.5 2^17, and e = 2^r - 1: the
  // mantissa, times 2^32 and shifted right by less than 64 (for what lies above `floor`).
  __device__ __forceinline__ u64 whole(float p, float e, bool there = true) const {
    const int n = __float_as_int(p);
    const float2 f = table[n & 63];
    const unsigned mant = __float_as_uint(f.y) + (unsigned)__float2int_rn(e * f.x);
    return ((u64)(there ? mant : 0) << 32) >> (shift - (n >> 6));
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    if (infinite) return x == m ? 1ull << S : 0;
    if (!(x > floor)) return 0;
    const float y = x - base, p = fmaf(y, c_hi, 0x1.8p17f), q = p - 0x1.8p17f;
    const float r = fmaf(y, c_lo, fmaf(y, c_hi, -q));  // |r| <= 1 / 128 and a little
    float e = fmaf(r, kL3, kL2);                       // 2^r - 1
    e = fmaf(r, e, kL1);
    return whole(p, e * r);
  }
  // ln(weight of x / all).  The whole number of a small weight has lost too much: its power of two itself then.
  __device__ __forceinline__ double log_share(float x, u64 all) const {
    const u64 n = (*this)(x);
    const bool small = n < 1u << 30 && !infinite;
    double r = log((double)(small ? 1 : n) / (double)all);
    if (small)  // seldom, and a single row waits 0.2 us for it
      r += 0.6931471805599453 * (((double)x - (double)base) * ((double)c_hi + (double)c_lo) + ((0x48400000 >> 6) + 63 - shift));
    return r;
  }
  // The weights of N logits, the same arithmetic, two to an instruction; 0 for those whose bit of `there` is not set: of
  // all that lie up to `floor` or are NaN.
  template <int N>
  __device__ __forceinline__ void of(const float (&x)[N], const bool (&there)[N], u64 (&w)[N]) const {
    if (infinite) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = there[i] && x[i] == m ? 1ull << S : 0;
      return;
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const F2 c = f2(c_hi, c_hi), magic = f2(0x1.8p17f, 0x1.8p17f);
      const F2 y = f2(x[i] - base, x[i + 1] - base);
      const F2 p = fma(y, c, magic), q = fma(p, f2(-1.f, -1.f), magic);
      const F2 r = fma(y, f2(c_lo, c_lo), fma(y, c, q));
      F2 e = fma(r, f2(kL3, kL3), f2(kL2, kL2));
      e = fma(r, e, f2(kL1, kL1)) * r;
      const float2 p1 = split(p), e1 = split(e);
      w[i] = whole(p1.x, e1.x, there[i]);
      w[i + 1] = whole(p1.y, e1.y, there[i + 1]);
    }
  }
};
// c of a temperature, in two numbers (2^-47 of it).
__device__ __forceinline__ float2 log2e_over(float temp) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;  // log2(e)
  const float hi = kHi / temp;
  return make_float2(hi, hi > 0.f ? (fmaf(-hi, temp, kHi) + kLo) / temp : 0.f);
}

// 2^(j / 64) 2^31, j = 0 .. 63, as a number and as an integer: worked out once on the host.
struct Table {
  float2 of[64];
};
__device__ __forceinline__ void fill_table(float2 *table, const Table &t) {
  if (threadIdx.x < 64) table[threadIdx.x] = t.of[threadIdx.x];
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// floor(f * n) and whether it is exact, for a float f in [0, 1) and n < 2^63.
__device__ __forceinline__ u64 part_of(float f, u64 n, bool *exact) {
  *exact = true;
  if (!(f > 0.f)) return 0;
  int e = ilogbf(f);                                  // f = man * 2^(e - 23)
  const u64 man = (u64)scalbnf(f, 23 - e);            // 24 bits
  const int shift = 23 - e;                           // at least 24
  const u64 lo = man * n, hi = __umul64hi(man, n);    // up to 87 bits
  if (shift >= 128) {
    *exact = false;
    return 0;
  }
  if (shift >= 64) {
    *exact = lo == 0 && (shift == 64 || (hi << (128 - shift)) == 0);
    return shift == 64 ? hi : hi >> (shift - 64);
  }
  *exact = (lo << (64 - shift)) == 0;
  return (lo >> shift) | (hi << (64 - shift));
}
// The sum that top-p asks for: the least whole number that is at least p times `all`, at least 1.
__device__ __forceinline__ u64 share_of(float p, u64 all) {
  bool exact;
  u64 n = part_of(p, all, &exact);
  n += !exact;
  return n > 0 ? n : 1;
}

template <typename T>
__device__ __forceinline__ float get(const T *x, int v) {
  return (float)x[v];
}
template <>
__device__ __forceinline__ float get(const __nv_bfloat16 *x, int v) {
  return __bfloat162float(x[v]);
}

// Of the tokens with the edge's key those with an ID up to the edge's are left, and all above.
struct Edge {
  uint32_t key;
  int id;
};
// The same on logits: NaN and -inf are never left.
struct Left {
  float at;
  int id;
  __device__ __forceinline__ Left(Edge e)
      : at(e.key <= kNever ? -INFINITY : tr_unord(e.key)), id(e.key <= kNever ? -1 : e.id) {}
  __device__ __forceinline__ bool operator()(float x, int v) const { return x > at || (x == at && v <= id); }
  // Of these, the ones above `floor`.
  __device__ __forceinline__ Left above(float floor) const {
    Left l = *this;
    if (floor >= at) {
      l.at = floor;
      l.id = -1;
    }
    return l;
  }
};

// min_p's edge: the key of the least logit whose weight is at least min_p of the largest one's (0: off).
// below: T ln(min(min_p, 1)), how far that is below the largest logit; NaN: off.
__device__ __forceinline__ double min_p_below(float mp, float temp) {
  // with an infinite temperature all weights are 1
  return mp > 0.f && temp < INFINITY ? (double)temp * log(fmin((double)mp, 1.0)) : __longlong_as_double(~0ll);
}
__device__ __forceinline__ uint32_t min_p_key(double below, float m) {
  return below == below ? key_of(__double2float_ru((double)m + below)) : 0;
}
__device__ __forceinline__ Edge with_min_p(Edge e, uint32_t key) { return key > e.key ? Edge{key, INT_MAX} : e; }

__device__ __forceinline__ float uniform_of(float u) { return fminf(fmaxf(u, 0.f), 1.f - 0x1p-24f); }  // NaN: 0

// ---------------------------------------------------------------------------
// rows that a cluster's shared memory holds
// ---------------------------------------------------------------------------

// Threads of a CTA: where it has an SM to itself (long slices in shared memory), and where it shares one.  64 x 128256 in
// two CTAs of 512 to an SM took 56 us instead of 54.
constexpr int kAlone = 512, kShared = 256;
constexpr int kMaxWarps = kAlone / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;       // 64 to a power of two, where they are weighted
constexpr int kList = 1024;

struct alignas(128) Smem {  // the slice lies behind it
  float2 table[64];
  u64 box[2][kMaxCluster][2 + kMaxWarps / 2];  // what the cluster's CTAs have told this one, in this exchange and the last
  u64 wsum[kMaxWarps];
  u64 kept[kMaxWarps];            // the weights that are left in the warps' ranges, where they are known
  unsigned listed;                // tokens that were to go to this CTA's list
  uint32_t listed_low;            // the key that at least k tokens lie at or above
  float u;
  double below;
  unsigned found[3];
  int id;
  u64 cum;
  union {
    alignas(16) unsigned hist[kBins];
    u64 wide[256];
    u64 list[kList];              // key << 32 | ~ID of the candidates, all of the cluster's CTAs
  };
  u64 own[kList];                 // the ones in this CTA's slice
  u64 groups[kMaxCluster][64];    // sums of the histograms' groups
};

static_assert(sizeof(Smem) % 16 == 0 && offsetof(Smem, hist) % 16 == 0);

// HELD: the CTA's slice is in shared memory; else it is read from global memory (L2) in every pass.
template <typename T, bool HELD, int NT>
struct Row {
  static constexpr int VEC = 16 / sizeof(T);
  static constexpr int NW = NT / 32;
  const SampleArgs &a;
  Smem &s;
  const uint4 *data;   // held: the slice's 16-byte granules; what is no token is -inf
  const T *x;          // the row
  int whole0, whole1;  // granules of the slice whose elements are all tokens
  int CS, rank, parity = 0;
  int warp, lane;
  int id0;             // ID of the slice's first element (below 0: no token)
  int g0, g1;          // the warp's granules
  Weight w;

  __device__ __forceinline__ Row(const SampleArgs &a_, Smem &s_) : a(a_), s(s_) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
  }

  __device__ __forceinline__ void sync() {
    if (CS == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;" ::: "memory");
  }

  // Granule g of the slice, some of whose elements may be no tokens.
  __device__ __forceinline__ uint4 edge(int g) const {
    union {
      uint4 v;
      T e[VEC];
    } u;
    const int id = id0 + g * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) u.e[e] = id + e >= 0 && id + e < a.V ? x[id + e] : (T)-INFINITY;
    return u.v;
  }
  __device__ __forceinline__ const uint4 *granules() const {
    return HELD ? data : reinterpret_cast<const uint4 *>(x + id0);
  }
  __device__ __forceinline__ uint4 fetch(int g) const {
    return HELD || (g >= whole0 && g < whole1) ? granules()[g] : edge(g);
  }
  // f(granule, first ID) for the warp's granules, a batch of 32 at a time, N batches under way; all lanes call f
  // alike.
  template <int N, typename F>
  __device__ __forceinline__ void scan(F f) const {
    if constexpr (HELD) {
#pragma unroll 1
      for (int g = g0 + lane; g < g1; g += 32) f(data[g], id0 + g * VEC);
      return;
    }
    const int n = (g1 - g0) / 32;  // batches; those from i0 to i1 hold nothing but tokens
    const int i0 = g0 >= whole0 ? 0 : 1, i1 = min(n, (whole1 - g0) >> 5);
    const uint4 *p = granules() + g0 + lane;
    int id = id0 + (g0 + lane) * VEC;
    for (int i = 0; i < n;) {
      if (i >= i0 && i + N <= i1) {
        uint4 v[N];
#pragma unroll
        for (int b = 0; b < N; ++b) v[b] = p[b * 32];
#pragma unroll
        for (int b = 0; b < N; ++b) f(v[b], id + b * (32 * VEC));
        i += N;
        p += N * 32;
        id += N * 32 * VEC;
      } else {
        f(i >= i0 && i < i1 ? *p : fetch(g0 + i * 32 + lane), id);
        ++i;
        p += 32;
        id += 32 * VEC;
      }
    }
  }
  // f(x[4], first ID), where any of the warp's elements is at or above `floor`.
  template <int N, typename F>
  __device__ __forceinline__ void each(float floor, F f) const {
    scan<N>([&](const uint4 &v, int id) {
      if (__any_sync(~0u, most(v) >= floor)) by_four(v, id, f);
    });
  }
  template <typename F>
  static __device__ __forceinline__ void by_four(const uint4 &v, int id, F f) {
    if constexpr (VEC == 4) {
      const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
      f(x, id);
    } else {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x[4] = {__uint_as_float(u[2 * h] << 16), __uint_as_float(u[2 * h] & 0xFFFF0000u),
                            __uint_as_float(u[2 * h + 1] << 16), __uint_as_float(u[2 * h + 1] & 0xFFFF0000u)};
        f(x, id + 4 * h);
      }
    }
  }
  // Batches under way, of passes that do little or much (1280 x 32000 fp32: with four and 16 instead of eight in light
  // passes greedy takes 46 and 58 us instead of 44; with four instead of two in heavy ones min_p 86 instead of 90, but
  // rows of mixed rules 203 instead of 178, whose code the SM's CTAs fetch by turns).  From shared memory one: more
  // copies of a pass's code, each of which a short row runs through once, cost more in fetching instructions (gathering
  // from 4096 logits a CTA took 9 us with four).
  static constexpr int kLight = HELD ? 1 : 32 / VEC, kHeavy = HELD ? 1 : 8 / VEC;
  // A granule's largest element.
  static __device__ __forceinline__ float most(const uint4 &v) {
    if constexpr (VEC == 4) {
      float m;
      asm("max.f32 %0, %1, %2, %3;"
          : "=f"(m)
          : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)), "f"(__uint_as_float(v.z)));
      return fmaxf(m, __uint_as_float(v.w));
    } else {
      auto b = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
      const __nv_bfloat162 m = __hmax2(__hmax2(b(v.x), b(v.y)), __hmax2(b(v.z), b(v.w)));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }

  // Sum of v over the CTA, in every thread (two barriers).
  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = warp_sum(v);
    if (lane == 0) s.wsum[warp] = v;
    __syncthreads();
    u64 r = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) r += s.wsum[i];
    __syncthreads();
    return r;
  }

  // Tells every CTA of the cluster up to three numbers of this one (the same in all threads) and waits for
  // theirs: heard(r, i).
  __device__ __forceinline__ void tell(u64 x, u64 y = 0, u64 z = 0) {
    if ((int)threadIdx.x < CS) {
      u64 *to = &s.box[parity][rank][0];
      if (CS > 1) to = cg::this_cluster().map_shared_rank(to, threadIdx.x);
      to[0] = x;
      to[1] = y;
      to[2] = z;
    }
    sync();
    parity ^= 1;
  }
  // The same with 32 bits of every warp, which its lane 0 has in s.wsum.
  __device__ __forceinline__ void tell_warps(u64 x) {
    for (int i = threadIdx.x; i < CS * (1 + NW / 2); i += NT) {
      const int r = i / (1 + NW / 2), w = i - r * (1 + NW / 2);
      u64 *to = &s.box[parity][rank][w];
      if (CS > 1) to = cg::this_cluster().map_shared_rank(to, r);
      *to = w == 0 ? x : (s.wsum[2 * w - 2] & 0xFFFFFFFFu) | s.wsum[2 * w - 1] << 32;
    }
    sync();
    parity ^= 1;
  }
  __device__ __forceinline__ uint32_t heard_warp(int i) const {  // i: of the cluster's
    const int r = i / NW, w = i - r * NW;
    return (uint32_t)(s.box[parity ^ 1][r][1 + w / 2] >> (w & 1) * 32);
  }
  __device__ __forceinline__ u64 heard(int r, int i) const { return s.box[parity ^ 1][r][i]; }

  // Inclusive sum over the CTA's threads (two barriers).
  __device__ __forceinline__ u64 block_scan(u64 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) s.wsum[warp] = v;
    __syncthreads();
    u64 before = 0;
    for (int i = 0; i < warp; ++i) before += s.wsum[i];
    __syncthreads();
    return before + v;
  }

  // The lowest ID at which the running sum over ascending IDs passes target_of(whole sum), in the one CTA that
  // holds it; -1 in the others.  amounts(x[4], first ID) is the sum of four tokens, none of which lies below `floor`,
  // amount(x, ID) one's.  known: the sums of the warps' ranges are in s.kept, and those that are not 0 hold a token whose
  // amount is not.
  template <typename F, typename A, typename G>
  __device__ __forceinline__ int first_past(float floor, F amounts, A amount, G target_of, u64 *all, bool known = false) {
    const int keep0 = g0, keep1 = g1, seg = a.granules / NW;
    u64 before = 0, target = 0, mine;
    bool here = true;
    // the sums of the warps' ranges; then, in the CTA that holds the place, of an eighth of the range that does
#pragma unroll 1
    for (int round = 0;; ++round) {
      mine = 0;
      if (round || !known) each<kHeavy>(floor, [&](const float (&x)[4], int v) { mine += amounts(x, v); });
      mine = warp_sum(mine);
      if (round == 0 && known) mine = s.kept[warp];
      __syncthreads();
      if (lane == 0) s.wsum[warp] = mine;
      if (threadIdx.x == 0) s.id = -1;
      __syncthreads();
      if (round) break;
      u64 cta = 0, sum = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) cta += s.wsum[i];
      tell(cta);
      for (int r = 0; r < CS; ++r) {
        if (r < rank) before += heard(r, 0);
        sum += heard(r, 0);
      }
      *all = sum;
      target = target_of(sum);
      here = before <= target && before + cta > target;
      if (!here) break;
      int q = 0;
      while (q < NW - 1 && before + s.wsum[q] <= target) before += s.wsum[q++];
      const int part = ((seg + NW - 1) / NW + 31) & ~31, hi = (q + 1) * seg;
      g0 = min(hi, q * seg + warp * part);
      g1 = min(hi, g0 + part);
    }
    if (here) {
      if (known) {  // sums that were made otherwise may differ in their last places (but 0 they are together)
        u64 all_parts = 0;
        for (int i = 0; i < NW; ++i) all_parts += s.wsum[i];
        target = min(target, before + all_parts - 1);
      }
      for (int i = 0; i < warp; ++i) before += s.wsum[i];
      if (before <= target && before + mine > target) {  // one warp: batch by batch, then a granule
        bool done = false;
        scan<1>([&](const uint4 &v, int id) {
          if (done) return;
          u64 own = 0;
          by_four(v, id, [&](const float (&x)[4], int i) { own += amounts(x, i); });
          u64 c = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(~0u, c, o);
            if (lane >= o) c += y;
          }
          const unsigned past = __ballot_sync(~0u, before + c > target);
          if (past) {
            if (lane == __ffs(past) - 1) {
              u64 run = before + c - own;
              int at = id;
              for (; at < id + VEC - 1; ++at) {
                run += at >= 0 && at < a.V ? amount(get(x, at), at) : 0;
                if (run > target) break;
              }
              s.id = at;
            }
            done = true;
          }
          before += __shfl_sync(~0u, c, 31);
        });
      }
    }
    g0 = keep0;
    g1 = keep1;
    __syncthreads();
    return here ? s.id : -1;
  }

  // A token's place on the histogram's scale: falling logits, rising bins.
  static __device__ __forceinline__ int bin_of(float m, float x, float scale) {
    return (int)fminf((m - x) * scale, (float)(kBins - 1));
  }

  // The sum of the cluster's histograms, found in two steps: each CTA tells the others the sums of its kGroups groups of
  // bins; of the groups that matter the bins are read from all CTAs.  Found are the first bins at which the running sum
  // reaches lo_of(all) and hi_of(all) (kBins where it does not), the sum before the first of them, and its own entry in
  // 32 bits.
  static constexpr int kGroups = 64, kGroup = kBins / kGroups;
  template <typename F, typename G, typename H>
  __device__ __forceinline__ void crossing(F value, G lo_of, H hi_of, int *b0, int *b1, u64 *base, unsigned *own) {
    if (threadIdx.x < 3) s.found[threadIdx.x] = kBins;
    __syncthreads();  // the histogram is whole
    static_assert(kGroup == 32);
#pragma unroll 1
    for (int g = warp; g < kGroups; g += NW) {
      const u64 v = warp_sum(value(g * 32 + lane, s.hist[g * 32 + lane]));
      if (lane < CS) {
        u64 *to = &s.groups[rank][g];
        if (CS > 1) to = cg::this_cluster().map_shared_rank(to, lane);
        *to = v;
      }
    }
    sync();
    // every warp: a lane has groups 2 lane and 2 lane + 1
    u64 v0 = 0, v1 = 0;
    for (int r = 0; r < CS; ++r) {
      v0 += s.groups[r][2 * lane];
      v1 += s.groups[r][2 * lane + 1];
    }
    u64 incl = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    const u64 all = __shfl_sync(~0u, incl, 31), lo = lo_of(all), hi = hi_of(all);
    if (warp < 2) {  // one for lo, one for hi
      const u64 mark = warp ? hi : lo;
      const unsigned past = __ballot_sync(~0u, incl >= mark);
      if (past && mark > 0) {
        const int l = __ffs(past) - 1;
        const u64 e = __shfl_sync(~0u, incl, l), w0 = __shfl_sync(~0u, v0, l), w1 = __shfl_sync(~0u, v1, l);
        u64 before = e - w0 - w1;
        const int g = 2 * l + (before + w0 < mark);
        if (before + w0 < mark) before += w0;
        u64 n = 0;
        for (int r = 0; r < CS; ++r) {
          const unsigned *h = &s.hist[g * 32 + lane];
          n += value(g * 32 + lane, CS > 1 ? *cg::this_cluster().map_shared_rank(h, r) : *h);
        }
        u64 c = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(~0u, c, o);
          if (lane >= o) c += y;
        }
        const unsigned in = __ballot_sync(~0u, before + c >= mark);
        if (in && lane == __ffs(in) - 1) {
          s.found[warp] = g * 32 + lane;
          if (warp == 0) {
            s.found[2] = (unsigned)n;
            s.cum = before + c - n;
          }
        }
      }
    }
    __syncthreads();
    *b0 = s.found[0];
    *b1 = s.found[1];
    *own = s.found[2];
    *base = s.cum;
  }

  // Clears the histogram and the list before anybody adds to them.
  __device__ __forceinline__ void clear() {
    __syncthreads();  // the last list has been read
    for (int i = threadIdx.x; i < kBins; i += NT) s.hist[i] = 0;
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
  }

  // Puts those of the tokens v .. v + 3 whose bits are set on the CTA's list.
  __device__ __forceinline__ void gather(unsigned bits, const float (&x)[4], int v) {
    if (bits == 0) return;
    unsigned at = atomicAdd(&s.listed, __popc(bits));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((bits >> e & 1) && at < kList) s.own[at++] = (u64)key_of(x[e]) << 32 | (0xFFFFFFFFu - (unsigned)(v + e));
  }

  // The cluster's lists, the largest entry first: every CTA makes its own copy.  The CTAs have told each other
  // how long theirs are: heard(r, 0).  Their number, more than kList where they do not fit.
  __device__ __forceinline__ int merge_lists() {
    u64 n = 0, before = 0;
    for (int r = 0; r < CS; ++r) {
      if (r < warp) before += heard(r, 0);
      n += heard(r, 0);
    }
    if (n > kList) return kList + 1;
    if (warp < CS) {  // warp r takes CTA r's
      const int mine = (int)heard(warp, 0);
      const u64 *from = CS > 1 ? cg::this_cluster().map_shared_rank(s.own, warp) : s.own;
      for (int i = lane; i < mine; i += 32) s.list[before + i] = from[i];
    }
    __syncthreads();
    sort_list((int)n);
    return (int)n;
  }

  // Sorts the list's n <= kList entries (none is 0), the largest first: 32 of them by each warp in registers, then every
  // entry's place is its place among these plus the numbers of larger ones in the other groups, found by bisection,
  // four groups at a time.
  __device__ __forceinline__ void sort_list(int n) {
    constexpr int kMine = kList / NT;  // entries of a thread
    for (int i = n + threadIdx.x; i < ((n + 127) & ~127); i += NT) s.list[i] = 0;
    __syncthreads();
    u64 e[kMine];
    int at[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int i = threadIdx.x + j * NT;
      if (i - lane >= n) break;
      u64 v = s.list[i];
#pragma unroll 1
      for (int k = 2; k <= 32; k *= 2)
#pragma unroll 1
        for (int d = k / 2; d; d /= 2) {
          const u64 o = __shfl_xor_sync(~0u, v, d);
          v = (((lane & k) == 0 || k == 32) == ((lane & d) == 0)) == (v > o) ? v : o;
        }
      s.list[i] = e[j] = v;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int i = threadIdx.x + j * NT;
      if (i - lane >= n) break;
      at[j] = 0;  // its own group among them: the entries before it there
#pragma unroll 1
      for (int g = 0; g < n; g += 128) {
        int c[4] = {};
#pragma unroll
        for (int d = 16; d; d /= 2)
#pragma unroll
          for (int q = 0; q < 4; ++q) c[q] += s.list[g + q * 32 + c[q] + d - 1] > e[j] ? d : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) at[j] += c[q] + (s.list[g + q * 32 + c[q]] > e[j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      if ((int)threadIdx.x + j * NT - lane >= n) break;
      if (e[j]) s.list[at[j]] = e[j];
    }
    __syncthreads();
  }

  static constexpr int kPer = kList / NT;
  // The place in the sorted list of n entries at which the running sum of the weights,
  // from `base` on, reaches target_of(base + their sum); n where it does not.
  template <typename G>
  __device__ __forceinline__ int place(int n, u64 base, G target_of) {
    u64 v[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x * (kPer) + j;
      v[j] = i < n ? w(tr_unord((uint32_t)(s.list[i] >> 32))) : 0;
      sum += v[j];
    }
    const u64 incl = block_scan(sum);
    if (threadIdx.x == NT - 1) s.cum = incl;
    if (threadIdx.x == 0) s.id = n;
    __syncthreads();
    const u64 target = target_of(base + s.cum);
    u64 run = base + incl - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (run < target && run + v[j] >= target) s.id = threadIdx.x * (kPer) + j;
      run += v[j];
    }
    __syncthreads();
    const int at = s.id;
    __syncthreads();
    return at;
  }

  __device__ __forceinline__ Edge edge_at(int i) const {
    const u64 e = s.list[min(max(i, 0), kList - 1)];
    return {(uint32_t)(e >> 32), (int)(0xFFFFFFFFu - (uint32_t)e)};
  }

  // The edge that leaves, of the tokens that `old` leaves, the first ones in falling order whose
  // amounts sum to at least `target`: the key is narrowed down by eight bits a pass, then the
  // lowest IDs among equal keys.
  template <typename F>
  __device__ __forceinline__ Edge narrow_down(u64 target, Left old, F amount) {
    uint32_t prefix = 0;
    u64 base = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      sync();  // the first CTA has read the last pass's sums
      for (int i = threadIdx.x; i < 256; i += NT) s.wide[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      each<kHeavy>(-FLT_MAX, [&](const float (&x)[4], int v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t k = key_of(x[e]);
          const u64 n = (k & mask) == prefix && old(x[e], v + e) ? amount(x[e]) : 0;
          const unsigned m = __ballot_sync(~0u, n != 0), b = (k >> shift) & 255;
          if (m == 0) continue;
          int same;  // a warp whose tokens all share a bin adds once
          __match_all_sync(~0u, b, &same);
          if (same) {
            const u64 t = warp_sum(n);
            if (lane == 0) atomicAdd(&s.wide[b], t);
          } else if (n) {
            atomicAdd(&s.wide[b], n);
          }
        }
      });
      sync();
      if (rank == 0) {
        // thread t has the bin that is t-th from above
        const int b = 255 - (int)threadIdx.x;
        u64 n = 0;
        for (int r = 0; b >= 0 && r < CS; ++r) n += CS > 1 ? *cg::this_cluster().map_shared_rank(&s.wide[b], r) : s.wide[b];
        const u64 incl = base + block_scan(n);
        if (incl >= target && incl - n < target) {
          s.found[0] = b;
          s.cum = incl - n;
        }
        __syncthreads();
      }
      tell(s.found[0], s.cum);
      prefix |= (uint32_t)(heard(0, 0) & 255) << shift;
      base = heard(0, 1);
    }
    const u64 each_ = amount(tr_unord(prefix));
    const u64 take = each_ ? (target - base + each_ - 1) / each_ : 0;
    u64 n;
    const float at = tr_unord(prefix);
    auto one = [&](float x, int v) -> u64 { return x == at && old(x, v); };
    const int id = first_past(at,
                              [&](const float (&x)[4], int v) {
                                u64 t = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) t += one(x[e], v + e);
                                return t;
                              },
                              one, [&](u64) -> u64 { return take - 1; }, &n);
    tell(id >= 0, (u64)(unsigned)id);
    Edge e = {prefix, INT_MAX};
    for (int r = 0; r < CS; ++r)
      if (heard(r, 0)) e.id = (int)(unsigned)heard(r, 1);
    return e;
  }

  // Adds the weights of the sorted list's first n entries to s.kept of the warps in whose ranges they lie.
  __device__ __forceinline__ void add_listed(int n) {
    const int seg = a.granules / NW * VEC;  // a warp's range
    for (int i = threadIdx.x; i < n; i += NT) {
      const u64 e = s.list[i];
      const unsigned at = (0xFFFFFFFFu - (uint32_t)e) - (unsigned)id0;
      if (at < (unsigned)(NW * seg)) atomicAdd(&s.kept[at / seg], w(tr_unord((uint32_t)(e >> 32))));
    }
    __syncthreads();
  }

  // top-k, and the other rules with it where the list takes all tokens at or above the edge: then *left is the number of
  // its entries that are left (else -1).
  // low: at least k tokens lie at or above it where it is `sure`, else fewer, a known part of k; or -inf.
  __device__ __forceinline__ Edge top_k(int k, float p, uint32_t min_p_key, float low, bool sure, int *left) {
    const Edge none = {kNever, -1};
    *left = -1;
    bool whole = sure;
    int need = k;
    Edge edge = none;
    auto found = [&] {  // from the gathered tokens
      __syncthreads();
      tell(s.listed);
      const int n = merge_lists();
      if (n > kList) return false;
      if (whole) {
        int keep = min(k, n);
        if (p < 1.f) keep = min(keep, place(keep, 0, [&](u64 all) { return share_of(p, all); }) + 1);
        *left = keep = at_least(keep, min_p_key);
        edge = edge_at(keep - 1);
      } else {
        edge = edge_at(need - 1);
      }
      return true;
    };
    bool ok = false;
    if (whole) {
      // often the list takes all tokens from `low` on
      each<kLight>(low, [&](const float (&x)[4], int v) {
        unsigned bits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) bits |= x[e] >= low ? 1u << e : 0;
        gather(bits, x, v);
      });
      ok = found();
    }
    if (!ok) {
      // bins from `low` on; where it is not sure twice as far down, and over all logits if these are too few
      const float m = w.m;
      float least = sure ? low : low - (m - low), scale;
      int b0, b1;
      u64 above;
      unsigned at_edge;
#pragma unroll 1
      for (bool last = sure;;) {
        if (!sure && !(least > -INFINITY && least < m)) {
          last = true;
          least = INFINITY;
          each<kHeavy>(-FLT_MAX, [&](const float (&x)[4], int) {
#pragma unroll
            for (int e = 0; e < 4; ++e) least = x[e] > -INFINITY ? fminf(least, x[e]) : least;
          });
#pragma unroll
          for (int o = 16; o; o >>= 1) least = fminf(least, __shfl_xor_sync(~0u, least, o));
          if (lane == 0) s.wsum[warp] = __float_as_uint(least);
          __syncthreads();
          for (int i = 0; i < NW; ++i) least = fminf(least, __uint_as_float((unsigned)s.wsum[i]));
          tell(__float_as_uint(least));
          for (int r = 0; r < CS; ++r) least = fminf(least, __uint_as_float((unsigned)heard(r, 0)));
        }
        const float span = m - least;
        if (!(span > 0.f && span < INFINITY)) return narrow_down_k(k);
        scale = fminf((float)(kBins - 1) / span, FLT_MAX);
        clear();
        each<kHeavy>(least, [&](const float (&x)[4], int) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[e] >= least) atomicAdd(&s.hist[bin_of(m, x[e], scale)], 1u);
        });
        crossing([](int, u64 n) { return n; }, [&](u64) -> u64 { return (u64)k; }, [&](u64) -> u64 { return (u64)k; }, &b0,
                 &b1, &above, &at_edge);
        if (b0 < kBins) break;
        if (last) return none;  // fewer than k tokens: all are left
        least = -INFINITY;
      }
      whole = above + at_edge <= kList;  // the list takes them all, else those of the edge's bin
      if (!whole) need = k - (int)above;
      // (a logit of bin b lies at or above m - (b + 1) / scale, but for the roundings: half a bin covers them)
      each<kLight>(fmaxf(least, m - (b0 + 1.5f) / scale), [&](const float (&x)[4], int v) {
        unsigned bits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = x[e] >= least ? bin_of(m, x[e], scale) : kBins;
          bits |= (whole ? b <= b0 : b == b0) ? 1u << e : 0;
        }
        gather(bits, x, v);
      });
      ok = found();
    }
    if (!ok) return narrow_down_k(k);
    if (whole) {
      if (threadIdx.x < NW) s.kept[threadIdx.x] = 0;
      __syncthreads();
      add_listed(*left);
    }
    return edge;
  }
  // How many of the sorted list's first n entries have at least this key (the first one has).
  __device__ __forceinline__ int at_least(int n, uint32_t key) {
    int c = 0;
    for (int i = threadIdx.x; i < n; i += NT) c += (uint32_t)(s.list[i] >> 32) >= key;
    return (int)block_sum(c);
  }
  __device__ __noinline__ Edge narrow_down_k(int k) {
    u64 n = 0;
    each<kHeavy>(-FLT_MAX, [&](const float (&x)[4], int) {
#pragma unroll
      for (int e = 0; e < 4; ++e) n += x[e] > -INFINITY;
    });
    n = block_sum(n);
    tell(n);
    n = 0;
    for (int r = 0; r < CS; ++r) n += heard(r, 0);
    const Edge none = {kNever, -1};
    return n <= (u64)k ? none : narrow_down((u64)k, Left(none), [](float) -> u64 { return 1; });
  }

  // top-p among the tokens that `old` leaves; *known: the weights that are left, by warps, are in s.kept (unless min_p
  // takes more).
  template <bool PLAIN>
  __device__ __forceinline__ Edge top_p(float p, Left old, uint32_t min_p_key, bool *known) {
    // 64 bins to a power of two; a token adds its weight's first 16 bits, in units of its bin's power of two
    // (2^16 of them: the sum of a slice of 65000 tokens stays below 2^32; of longer ones some bits are dropped).  A
    // token beyond the last bin but one has a weight below 2^-31.9 and is left out; a bin's sum is below the true
    // one by less than 2^-15 of it (and fp32's errors).  PLAIN: `old` leaves all (1280 x 32000, p = 0.9: its
    // comparisons cost 12 of 209 us when the histogram was slower).
    const float m = w.m, scale = fminf(w.c_hi * 64.f, FLT_MAX);
    const Left weighted = old.above(w.floor);
    const uint32_t hist = (uint32_t)__cvta_generic_to_shared(s.hist) - 4 * 0x4B400000u;
    clear();
    each<kHeavy>(fmaxf(old.at, m - 32.f / w.c_hi), [&](const float (&x)[4], int v) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const F2 y = fma(f2(x[i], x[i + 1]), f2(-1.f, -1.f), f2(m, m));
        const F2 t2 = fma(y, f2(scale, scale), f2(-0.5f, -0.5f));
        const float2 t = split(t2), b = split(fma(t2, f2(1.f, 1.f), f2(0x1.8p23f, 0x1.8p23f)));
        const float2 at = split(fma(t2, f2(-1.f / 64, -1.f / 64), f2(-0.5f / 64, -0.5f / 64)));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned bin = __float_as_uint(e ? b.y : b.x);  // + 0x4B400000: the whole number nearest to t, below t + 0.5
          float f;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(e ? at.y : at.x));
          // in [2^-(o + 1), 2^-o], o = bin / 64: 16 bits of it, from 2^15 on, out of the float's own
          const unsigned n = (__float_as_uint(f) + ((bin & ~63u) << 17) + ((1u << 23) - (126u << 23))) >> (8 + a.drop);
          if ((e ? t.y : t.x) < (float)(kBins - 1) && (PLAIN || old(x[i + e], v + i + e)))
            asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(hist + bin * 4), "r"(n) : "memory");
        }
      }
    });
    int b0, b1;
    u64 base;
    unsigned own;
    // in units of 2^-S
    const int off = 14 - a.drop;  // sums are off by less than 2^-off
    crossing([&](int b, u64 n) { return (n << (a.S - 16 + a.drop)) >> (b >> 6); },
             [&](u64 all) -> u64 { return share_of(p, all - (all >> off)); },
             [&](u64 all) -> u64 { return share_of(p, all + (all >> off) + ((u64)a.V << max(a.S - 31, 0))); }, &b0, &b1,
             &base, &own);
    // the exact sums, of all and of what lies above the bins that hold the edge (they end at logits `hi` and `lo`, with 2^-7
    // of a bin for the roundings)
    u64 rest = 0, above = 0;
    const float hi = __fsub_ru(m, ((float)b0 - 0x1p-7f) / scale);
    const float lo = b1 < kBins ? __fsub_rd(m, ((float)b1 + (1.f + 0x1p-7f)) / scale) : -INFINITY;
    each<kHeavy>(weighted.at, [&](const float (&x)[4], int v) {
      u64 q[4];
      bool there[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) there[e] = PLAIN ? x[e] > weighted.at : weighted(x[e], v + e);
      w.of(x, there, q);
      bool some = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (x[e] > hi) above += q[e];
        else rest += q[e];
        some |= x[e] <= hi && x[e] >= lo;
      }
      if (some) {
        unsigned in = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) in |= x[e] <= hi && x[e] >= lo && q[e] ? 1u << e : 0;
        gather(in, x, v);
      }
    });
    above = warp_sum(above);
    if (lane == 0) s.kept[warp] = above;
    u64 all = block_sum(rest);  // (its barrier makes s.kept known)
    above = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) above += s.kept[i];
    all += above;
    tell(s.listed, all, above);
    all = above = 0;
    for (int r = 0; r < CS; ++r) {
      all += heard(r, 1);
      above += heard(r, 2);
    }
    const u64 target = share_of(p, all);
    *known = false;
    const int n = above < target ? merge_lists() : kList + 1;
    if (n > kList) return narrow_down_p(target, old);
    const int at = place(n, above, [&](u64) { return target; });
    if (at >= n) return narrow_down_p(target, old);
    const Edge edge = edge_at(at);
    *known = edge.key >= min_p_key;
    if (*known) add_listed(at + 1);
    return edge;
  }
  __device__ __noinline__ Edge narrow_down_p(u64 target, Left old) { return narrow_down(target, old, w); }
};

template <typename T, bool HELD, int NT>
__global__ void __launch_bounds__(NT, NT == kAlone ? 1 : HELD ? 2 : 3) sample_kernel(const SampleArgs a, int CS,
                                                             const __grid_constant__ Table table) {
  extern __shared__ __align__(128) unsigned char smem[];
  Smem &s = *reinterpret_cast<Smem *>(smem);
  using R = Row<T, HELD, NT>;
  R r(a, s);
  constexpr int VEC = R::VEC, NW = R::NW;
  const long long row = blockIdx.x / CS;
  r.CS = CS;
  r.rank = blockIdx.x - (int)row * CS;
  uint4 *const data = reinterpret_cast<uint4 *>(smem + sizeof(Smem));
  r.data = data;
  r.g0 = r.warp * (a.granules / NW);
  r.g1 = r.g0 + a.granules / NW;
  fill_table(s.table, table);
  if (threadIdx.x == 0) s.listed = 0;
  // a CTA's shared memory may be written from others only once it has started: waited for before the first number is told
  if (CS > 1) asm volatile("barrier.cluster.arrive;" ::: "memory");
  tr_let_next_start();
  tr_wait_for_previous();
  // the slice, in granules that start on 16-byte boundaries; each lane copies what it reads
  const T *const x = reinterpret_cast<const T *>(a.x) + row * a.ld;
  const int off = (int)(((uintptr_t)x & 15) / sizeof(T));
  r.id0 = (int)((long long)r.rank * a.granules * VEC) - off;
  r.x = x;
  r.whole0 = r.id0 < 0 ? 1 : 0;
  r.whole1 = r.id0 >= a.V ? 0 : (int)min((long long)a.granules, ((long long)a.V - r.id0) / VEC);
  if (HELD) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(data);
    const T *from = x + r.id0;
#pragma unroll 4
    for (int g = r.g0 + r.lane; g < r.g1; g += 32) {
      if (g >= r.whole0 && g < r.whole1) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + g * 16), "l"(from + g * VEC) : "memory");
      } else {
        T *edge = reinterpret_cast<T *>(data + g);
        const int id = r.id0 + g * VEC;
        for (int e = 0; e < VEC; ++e) edge[e] = id + e >= 0 && id + e < a.V ? x[id + e] : (T)-INFINITY;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const float temp = a.temperature ? a.temperature[row] : 1.f, p = a.top_p ? a.top_p[row] : 1.f,
              min_p = a.min_p ? a.min_p[row] : 0.f;
  int k = a.top_k ? a.top_k[row] : 0;
  if (k >= a.V) k = 0;
  const float2 c = log2e_over(temp);
  if (threadIdx.x == NT - 1) {  // the rules, while the slice is under way; 64-bit arithmetic once
    s.u = uniform_of(a.U[row]);
    s.below = min_p_below(min_p, temp);
  }
  if (HELD) asm volatile("cp.async.wait_group 0;" ::: "memory");

  // The largest logit; and, for top-k, one that at least k lie at or above: of each of the a.full warps whose ranges are
  // full of tokens the j-th of the lanes' largest, of these the ceil(k / j)-th.
  float most = -INFINITY;
  int where = 0;  // the first ID of the granule that has the lane's largest
  // Temperature alone, from global memory: the weights are summed in the same pass, relative to the largest logit that
  // the warp has seen yet.
  const bool once = !HELD && k == 0 && !(p < 1.f) && !(min_p > 0.f) && temp >= FLT_MIN;
  bool known = false;  // the weights that are left, by warps
  u64 sum = 0;
  if (once) {
    __syncthreads();  // the table
    r.w.set(-INFINITY, c, a.S, s.table);
    r.w.floor = FLT_MAX;
    known = true;
    r.template scan<16 / VEC>([&](const uint4 &v, int id) {
      const float top = R::most(v);
      if (__any_sync(~0u, top > most)) {
        most = fmaxf(most, top);
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        const int shift = r.w.shift;
        const bool first = r.w.m == -INFINITY;
        r.w.set(most, c, a.S, s.table);
        if (r.w.far) known = false;  // not a shift: the sums are found in a pass of their own
        if (!first) sum >>= min(r.w.shift - shift, 63);
      }
      R::by_four(v, id, [&](const float (&x)[4], int) {
        u64 q[4];
        const float f = r.w.floor;
        r.w.of(x, {x[0] > f, x[1] > f, x[2] > f, x[3] > f}, q);
        sum += (q[0] + q[1]) + (q[2] + q[3]);
      });
    });
    sum = warp_sum(sum);
  } else {
    r.template scan<R::kLight>([&](const uint4 &v, int id) {
      const float top = R::most(v);
      where = top > most ? id : where;
      most = fmaxf(most, top);
    });
  }
  const float lane_most = most;
  const int own_shift = r.w.shift;
  const int full_j = k > 0 && a.full > 0 ? (int)(((long long)k + a.full - 1) / a.full) : INT_MAX;
  const bool sure = full_j <= 32;  // beyond, up to an eighth of k are known to lie at or above the least of the 32nd
  const int j = sure ? full_j : full_j <= 8 * 32 ? 32 : 33;
  float bound = -INFINITY;
  if (j <= 32) {
    float v = most;  // the lanes' in falling order
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
      for (int d = n / 2; d; d /= 2) {
        const float o = __shfl_xor_sync(~0u, v, d);
        v = ((r.lane & n) == 0 || n == 32) == ((r.lane & d) == 0) ? fmaxf(v, o) : fminf(v, o);
      }
    bound = __shfl_sync(~0u, v, j - 1);
    most = __shfl_sync(~0u, v, 0);
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
  }
  if (r.lane == 0) s.wsum[r.warp] = (u64)key_of(most) << 32 | key_of(bound);
  __syncthreads();
  uint32_t top = 0, low = 0;
  for (int i = 0; i < NW; ++i) top = max(top, (uint32_t)(s.wsum[i] >> 32));
  const uint32_t own_top = top;
  if (CS > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
  r.tell_warps(top);
  int owner = 0;  // the first CTA that has the largest
  for (int i = CS - 1; i >= 0; --i) {
    const uint32_t t = (uint32_t)r.heard(i, 0);
    if (t >= top) {
      top = t;
      owner = i;
    }
  }
  if (j <= 32) {
    const int n = a.full, rank = sure ? (k + j - 1) / j : n;
    if ((int)threadIdx.x < n) {
      const uint32_t mine = r.heard_warp(threadIdx.x);
      int above = 0;
      for (int i = 0; i < n; ++i) {
        const uint32_t o = r.heard_warp(i);
        above += o > mine || (o == mine && i < (int)threadIdx.x);
      }
      if (above == rank - 1) s.listed_low = mine;
    }
    __syncthreads();
    low = s.listed_low;
  }
  if (top <= kNever || !(temp >= FLT_MIN) || k == 1) {
    if (top <= kNever) {
      if (r.rank == 0 && threadIdx.x == 0) {
        a.token[row] = -1;
        if (a.logprob) a.logprob[row] = -INFINITY;
      }
    } else if (r.rank == owner && own_top == top) {
      if (threadIdx.x == 0) s.id = INT_MAX;
      __syncthreads();
      int first = INT_MAX;
      if (key_of(lane_most) == top) {
        for (int e = VEC - 1; e >= 0; --e) {
          const int v = where + e;
          if (v >= 0 && v < a.V && key_of(get(x, v)) == top) first = v;
        }
      }
      atomicMin(&s.id, first);
      __syncthreads();
      if (threadIdx.x == 0) {
        a.token[row] = s.id;
        if (a.logprob) a.logprob[row] = 0.f;
      }
    }
    return;
  }
  r.w.set(tr_unord(top), c, a.S, s.table);

  Edge edge = {kNever, -1};
  const uint32_t mp = min_p_key(s.below, r.w.m);
  if (once) {
    known = !__syncthreads_or(!known || r.w.far);
    // tokens that count beside the warp's largest may all lie too low beside the row's: then the range has none to draw
    if (known && r.lane == 0) s.kept[r.warp] = most > r.w.floor ? sum >> min(r.w.shift - own_shift, 63) : 0;
    __syncwarp();
  }
  int listed = -1;
  if (k > 0) {
    edge = r.top_k(k, p, mp, low > kNever ? tr_unord(low) : -INFINITY, sure && low > kNever, &listed);
    known = listed >= 0;
  }
  if (p < 1.f && listed < 0) {
    if (edge.key <= kNever) edge = r.template top_p<true>(p, Left(edge), mp, &known);
    else edge = r.template top_p<false>(p, Left(edge), mp, &known);
  }
  const Left left = Left(with_min_p(edge, mp)).above(r.w.floor);
  const float u = s.u;
  u64 all;
  const int id = r.first_past(left.at,
                              [&](const float (&y)[4], int v) {
                                u64 q[4];
                                r.w.of(y, {left(y[0], v), left(y[1], v + 1), left(y[2], v + 2), left(y[3], v + 3)}, q);
                                return (q[0] + q[1]) + (q[2] + q[3]);
                              },
                              [&](float y, int v) -> u64 { return left(y, v) ? r.w(y) : 0; },
                              [&](u64 sum) {
                                bool exact;
                                return part_of(u, sum, &exact);
                              },
                              &all, known);
  if (id >= 0 && threadIdx.x == 0) {
    a.token[row] = id;
    const float y = get(x, id);
    if (a.logprob) a.logprob[row] = (float)r.w.log_share(y, all);
  }
}

const Table &table() {
  static const Table t = [] {
    Table x;
    for (int j = 0; j < 64; ++j) {
      const double p = std::exp2(j / 64.0) * 0x1p31;
      const uint32_t bits = (uint32_t)std::llround(p);
      x.of[j].x = (float)p;
      memcpy(&x.of[j].y, &bits, 4);
    }
    return x;
  }();
  return t;
}

// Slices that a CTA can hold in shared memory, alone on an SM and as one of two; tokens of any slice, see top_p.
constexpr long long kAloneSlice = 192 * 1024, kSharedSlice = 88 * 1024;
static_assert(sizeof(Smem) + kAloneSlice <= 227 * 1024 && 2 * (sizeof(Smem) + kSharedSlice + 1024) <= 228 * 1024);
constexpr int kMostTokens = 65000;

template <typename T, bool HELD, int NT>
constexpr size_t most_shared() {
  return sizeof(Smem) + (HELD ? NT == kAlone ? kAloneSlice : kSharedSlice : 0);
}

// Clusters of 2^n CTAs that the device runs at once (those of eight do not fill its groups of SMs: 38 rows in clusters of
// eight are 304 CTAs, two to an SM, and take two waves, 16 us instead of 10 for 33 rows).  Asked once for a device.
template <typename T, bool HELD, int NT>
int clusters_at_once(int n, long long *count) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];  // and one more
  int dev = 0;
  TR_TRY_CUDA(cudaGetDevice(&dev));
  int c = dev < kDevices ? known[dev][n].load(std::memory_order_relaxed) : 0;
  if (c == 0) {
    TR_TRY_CUDA(cudaFuncSetAttribute(sample_kernel<T, HELD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)most_shared<T, HELD, NT>()));
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1 << n;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1 << n);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = most_shared<T, HELD, NT>();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    TR_TRY_CUDA(cudaOccupancyMaxActiveClusters(&c, sample_kernel<T, HELD, NT>, &cfg));
    ++c;
    if (dev < kDevices) known[dev][n].store(c, std::memory_order_relaxed);
  }
  *count = c - 1;
  return TR_OK;
}

// A row's share of the chip: 2^n CTAs, as many as leave all rows' a place at once and each CTA 4 KB.
struct Shape {
  int n, granules;
  bool fits;  // all rows are under way at once
};
template <typename T, bool HELD, int NT>
int shape_of(const SampleArgs &a, Shape *out) {
  constexpr int VEC = 16 / sizeof(T), kMostN = 3;
  static_assert(1 << kMostN == kMaxCluster);
  const long long all = ((long long)a.V + 2 * VEC - 2) / VEC;  // granules, wherever the row starts in the first
  int n = 0;
  long long count = 0;
  while (n < kMostN && (all >> n) * 16 > 4096) {
    const int rc = clusters_at_once<T, HELD, NT>(n + 1, &count);
    if (rc != TR_OK) return rc;
    if (a.rows > count) break;
    ++n;
  }
  while (n < kMostN && (all >> n) * VEC > kMostTokens - 2 * kAlone * VEC) ++n;
  const int rc = clusters_at_once<T, HELD, NT>(n, &count);
  if (rc != TR_OK) return rc;
  const long long one = (all + (1 << n) - 1) >> n;
  *out = {n, (int)((one + NT - 1) / NT * NT), a.rows <= count};
  return TR_OK;
}

template <typename T, bool HELD, int NT>
int launch(SampleArgs a, const Shape &shape, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const int cs = 1 << shape.n;
  a.granules = shape.granules;
  a.full = (int)(((long long)a.V - (VEC - 1)) / ((long long)a.granules / (NT / 32) * VEC));
  a.drop = 0;
  while (((long long)a.granules * VEC >> a.drop) > kMostTokens) ++a.drop;
  return tr_launch_next(sample_kernel<T, HELD, NT>,
                        {dim3((unsigned)(a.rows * cs)), NT, sizeof(Smem) + (HELD ? (size_t)a.granules * 16 : 0), cs}, s, a,
                        cs, table());
}

// Rows are held in shared memory where all of them are at once: 64 x 128256 bf16 in four slices each take 43 to 57 us so
// (top-p) and 54 to 74 read from L2, 67 and 82 (top-k 900), 8.6 and 7.7 (greedy).  Many rows held by clusters, wave
// after wave, lose by it (1280 x 32000, when it was tried: temperature 156 instead of 108 us, top-k 50 185 instead
// of 99): fewer CTAs fit on an SM, and the barriers are clusters' instead of CTAs'.  CTAs of 512 threads with an SM to
// themselves pay from 8192 tokens a CTA on: 1 x 128256 bf16 22.0 instead of 23.8 us (top-p), 10.9 / 12.2 (temperature),
// but 1 x 32000 18.7 / 17.9 and 8.6 / 7.9, 2 x 8000 17.9 / 15.9 and 8.3 / 6.7.
template <typename T>
int launch(const SampleArgs &a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  Shape alone, shared;
  int rc = shape_of<T, true, kAlone>(a, &alone);
  if (rc != TR_OK) return rc;
  if (alone.fits && alone.granules * VEC > 8192 && alone.n == 3 && alone.granules * 16LL <= kAloneSlice)
    return launch<T, true, kAlone>(a, alone, s);
  rc = shape_of<T, true, kShared>(a, &shared);
  if (rc != TR_OK) return rc;
  if (shared.fits && shared.granules * 16LL <= kSharedSlice) return launch<T, true, kShared>(a, shared, s);
  rc = shape_of<T, false, kShared>(a, &shared);
  if (rc != TR_OK) return rc;
  return launch<T, false, kShared>(a, shared, s);
}

}  // namespace

extern "C" int tr_sample(const void *logits, tr_ftype ftype, int64_t rows, int64_t V, int64_t ld,
                         const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                         const float *U, int32_t *token, float *logprob, tr_stream_t stream) {
  if (ftype != TR_F32 && ftype != TR_BF16) return TR_E_INVAL;
  if (rows < 0 || V < 1 || ld < V) return TR_E_INVAL;
  if (rows == 0) return TR_OK;
  if (!logits || !U || !token) return TR_E_INVAL;
  if (((uintptr_t)logits & (ftype == TR_F32 ? 3 : 1)) ||
      (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)U |
        (uintptr_t)token | (uintptr_t)logprob) & 3))
    return TR_E_INVAL;
  if (V > (1LL << 30) || rows > (1LL << 24) || ld > (1LL << 60) / rows) return TR_E_UNSUPPORTED;
  const int rc = tr_check_device();
  if (rc != TR_OK) return rc;
  SampleArgs a = {logits, ld, rows, (int)V, 62, temperature, top_p, min_p, U, top_k, token, logprob};
  while (a.S > 30 && (V >> (62 - a.S)) > 1) --a.S;  // V weights of 2^S and less stay below 2^63
  cudaStream_t s = (cudaStream_t)stream;
  return ftype == TR_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}
