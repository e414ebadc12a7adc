// Sampling: one token of each row of logits, with temperature, top-k, top-p and min-p,
// from given uniforms.
//
// Weights w = 2^((x - m) log2(e) / T), m the row's maximum, are held as integers in units of
// 2^-S, so their sums are exact and do not depend on the order: top-p's edge is found
// from sums over any grouping, and equal calls give equal bits.  A token is left when its key
// (the order of its logit) is above the row's edge, or at it with an ID up to the edge's.
#include <cfloat>
#include <cmath>

#include "tr_internal.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
typedef unsigned long long u64;

struct SampleArgs {
  const void *x;
  long long ld;
  int V, S;  // weights are in units of 2^-S
  const float *temperature, *top_p, *min_p, *U;
  const int32_t *top_k;
  int32_t *token;
  float *logprob;
};

// The order of a logit; NaN and -inf (never drawn) are 0x007FFFFF, below every other.
constexpr uint32_t kNever = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float x) { return x == x ? tr_ord(x) : kNever; }

// Weights of a row.  The exponent (m - x) log2(e) / T is carried in two fp32 numbers, its
// fraction's power of two comes from a table of 2^(-j / 64) and a polynomial in the rest.
struct Weight {
  float m, c_hi, c_lo;
  int S;
  const float2 *table;  // 2^(-j / 64): as a float, and (as bits) 2^31 times it
  // 2^S w, rounded down
  __device__ __forceinline__ u64 operator()(float x) const {
    if (x == m) return 1ull << S;
    // d = m - x exactly, as d + e
    const float d = m - x, z = d - m, e = (m - (d - z)) - (x + z);
    const float t = d * c_hi;
    if (!(t < 63.f)) return 0;  // below every S, or not a number: x is -inf
    const float lo = fmaf(d, c_hi, -t) + fmaf(d, c_lo, e * c_hi);
    const float n = rintf(t * 64.f);
    const float r = fmaf(n, -1.f / 64.f, t) + lo;  // |r| <= 1 / 128 and a little
    // 2^-r - 1
    float y = fmaf(r, 9.618129107628477e-3f, -5.550410866482158e-2f);  // ln2^4 / 24, -ln2^3 / 6
    y = fmaf(r, y, 2.402265069591007e-1f);
    y = fmaf(r, y, -6.931471805599453e-1f);
    y *= r;
    const int j = (int)n;
    const float2 p = table[j & 63];
    const unsigned mant = __float_as_uint(p.y) + (unsigned)__float2int_rn(y * p.x * 0x1p31f);
    const int shift = (j >> 6) + 31 - S;  // the weight is mant 2^-31 2^-(j >> 6)
    return shift >= 0 ? (u64)mant >> min(shift, 63) : (u64)mant << -shift;
  }
};

struct Smem {
  float2 table[64];
  u64 hist[256];
  u64 wsum[kWarps];
  u64 best;
  u64 base;      // of the keys above
  uint32_t prefix;
  int id;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// Sum over the block, in every thread (two barriers).
__device__ __forceinline__ u64 block_sum(u64 v, u64 *wsum) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) wsum[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
  for (int i = 0; i < kWarps; ++i) s += wsum[i];
  __syncthreads();
  return s;
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

// The range of IDs of a warp: consecutive ones.
struct Range {
  int lo, hi;
};

template <typename T>
__device__ __forceinline__ float get(const T *x, int v) {
  return (float)x[v];
}
template <>
__device__ __forceinline__ float get(const __nv_bfloat16 *x, int v) {
  return __bfloat162float(x[v]);
}

// The lowest ID at which the running sum of weight_of(id) over ascending IDs passes
// `target` (V if it never does).  Every thread gets it.
template <typename F>
__device__ __forceinline__ int first_past(u64 target, Range r, Smem &s, F weight_of) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 sum = 0;
  for (int v = r.lo + lane; v < r.hi; v += 32) sum += weight_of(v);
  sum = warp_sum(sum);
  if (threadIdx.x == 0) s.id = INT_MAX;
  if (lane == 0) s.wsum[warp] = sum;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += s.wsum[i];
  if (before <= target && before + sum > target) {  // one warp at most
    for (int v0 = r.lo; v0 < r.hi; v0 += 32) {
      u64 c = v0 + lane < r.hi ? weight_of(v0 + lane) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(~0u, c, o);
        if (lane >= o) c += y;
      }
      const unsigned past = __ballot_sync(~0u, before + c > target);
      if (past) {
        if (lane == 0) s.id = v0 + __ffs(past) - 1;
        break;
      }
      before += __shfl_sync(~0u, c, 31);
    }
  }
  __syncthreads();
  const int id = s.id;
  __syncthreads();
  return id;
}

// The edge that leaves, of the tokens whose key is above `never`, the first ones in
// falling order whose amounts sum to at least `target` (>= 1): the key is narrowed down by
// eight bits a pass.  amount(x) of equal keys is equal.
struct Edge {
  uint32_t key;
  int id;  // of the tokens with that key the ones up to this ID are left
};
template <typename T, typename F>
__device__ __forceinline__ Edge select(const T *x, int V, Range r, u64 target, Edge old, Smem &s, F amount) {
  uint32_t prefix = 0;
  u64 base = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) s.hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int v = threadIdx.x; v < V; v += kThreads) {
      const float y = get(x, v);
      const uint32_t k = key_of(y);
      if ((k & mask) != prefix || !(k > old.key || (k == old.key && v <= old.id))) continue;
      const u64 a = amount(y);
      if (a) atomicAdd(&s.hist[(k >> shift) & 255], a);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 sum = base;
      int b = 255;
      for (; b > 0; --b) {
        if (sum + s.hist[b] >= target) break;
        sum += s.hist[b];
      }
      s.base = sum;
      s.prefix = prefix | (uint32_t)b << shift;
    }
    __syncthreads();
    base = s.base;
    prefix = s.prefix;
    __syncthreads();
  }
  // of the tokens at the edge the lowest IDs, as many as are needed
  const u64 each = amount(tr_unord(prefix));
  const u64 take = each ? (target - base + each - 1) / each : 0;
  Edge e = {prefix, INT_MAX};
  if (take)
    e.id = first_past(take - 1, r, s, [&](int v) -> u64 {
      return key_of(get(x, v)) == prefix && !(prefix == old.key && v > old.id);
    });
  return e;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  __shared__ Smem s;
  tr_let_next_start();
  tr_wait_for_previous();
  const long long row = blockIdx.x;
  const T *x = reinterpret_cast<const T *>(a.x) + row * a.ld;
  const int V = a.V, warp = threadIdx.x >> 5;
  const int seg = (int)(((long long)V + kWarps - 1) / kWarps);
  const Range r = {(int)min((long long)V, (long long)warp * seg), (int)min((long long)V, (long long)(warp + 1) * seg)};
  if (threadIdx.x < 64) {
    const double p = exp2(-(double)threadIdx.x / 64.0);
    s.table[threadIdx.x] = make_float2((float)p, __uint_as_float((unsigned)__double2ll_rn(p * 0x1p31)));
  }
  if (threadIdx.x == 0) s.best = 0;
  __syncthreads();

  // the largest logit and its lowest ID
  u64 best = 0;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    const u64 k = (u64)key_of(get(x, v)) << 32 | (0xFFFFFFFFu - (uint32_t)v);
    best = k > best ? k : best;
  }
  atomicMax(&s.best, best);
  __syncthreads();
  best = s.best;
  const uint32_t top = (uint32_t)(best >> 32);
  const float temp = a.temperature ? a.temperature[row] : 1.f;
  if (top <= kNever || !(temp >= FLT_MIN)) {
    if (threadIdx.x == 0) {
      a.token[row] = top <= kNever ? -1 : (int)(0xFFFFFFFFu - (uint32_t)best);
      if (a.logprob) a.logprob[row] = top <= kNever ? -INFINITY : 0.f;
    }
    return;
  }
  Weight w;
  w.m = tr_unord(top);
  w.S = a.S;
  w.table = s.table;
  const double c = 1.4426950408889634 / (double)temp;
  w.c_hi = (float)c;
  w.c_lo = (float)(c - (double)w.c_hi);

  Edge edge = {kNever, -1};
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < V) {
    // fewer than k tokens in all: the edge stays below them
    u64 n = 0;
    for (int v = threadIdx.x; v < V; v += kThreads) n += key_of(get(x, v)) > kNever;
    n = block_sum(n, s.wsum);
    if (n > (u64)k) edge = select(x, V, r, (u64)k, edge, s, [](float) -> u64 { return 1; });
  }
  auto left = [&](uint32_t key, int v) { return key > edge.key || (key == edge.key && v <= edge.id); };
  const float p = a.top_p ? a.top_p[row] : 1.f;
  if (p < 1.f) {
    u64 all = 0;
    for (int v = threadIdx.x; v < V; v += kThreads) {
      const float y = get(x, v);
      if (left(key_of(y), v)) all += w(y);
    }
    all = block_sum(all, s.wsum);
    bool exact;
    u64 need = part_of(p, all, &exact);
    need += !exact;
    edge = select(x, V, r, need > 0 ? need : 1, edge, s, w);
  }
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  if (mp > 0.f && temp < INFINITY) {  // with an infinite temperature all weights are 1
    const float f = __double2float_ru((double)w.m + (double)temp * log(fmin((double)mp, 1.0)));
    const uint32_t lk = key_of(f);
    if (lk > edge.key) edge = {lk, INT_MAX};
  }
  auto weight_of = [&](int v) -> u64 {
    const float y = get(x, v);
    return left(key_of(y), v) ? w(y) : 0;
  };
  u64 all = 0;
  for (int v = threadIdx.x; v < V; v += kThreads) all += weight_of(v);
  all = block_sum(all, s.wsum);
  const float u = fminf(fmaxf(a.U[row], 0.f), 1.f - 0x1p-24f);  // NaN: 0
  bool exact;
  const int id = first_past(part_of(u, all, &exact), r, s, weight_of);
  if (threadIdx.x == 0) {
    a.token[row] = id;
    if (a.logprob) a.logprob[row] = (float)log((double)w(get(x, id)) / (double)all);
  }
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
  SampleArgs a = {logits, ld, (int)V, 62, temperature, top_p, min_p, U, top_k, token, logprob};
  while (a.S > 30 && (V >> (62 - a.S)) > 1) --a.S;  // V weights of 2^S and less stay below 2^63
  auto go = [&](auto kernel) {
    return tr_launch_next(kernel, {dim3((unsigned)rows), kThreads}, (cudaStream_t)stream, a);
  };
  return ftype == TR_F32 ? go(sample_kernel<float>) : go(sample_kernel<__nv_bfloat16>);
}
