// Norms of queries and keys per head with the position rotation in the same pass,
// into dense rows (tr_qkv_rope) or, for keys and values, into a KV cache
// (tr_kv_append_rope).
//
// A row x of d elements: y = x w / sqrt(mean x^2 + eps), then pairs of elements turned
// by the angle p f_i.  Every element is read once and written once and takes a few
// flops: bytes bound the large calls, a chain of latencies the small ones.
//
// A head's row is held by d / 16 lanes of a warp, 16 elements each in two 16-byte
// pieces that make whole pairs: pieces c and c + rot / 16 where halves are paired, else 2 c
// and 2 c + 1.  A lane then turns its own pairs, and one set of eight cosines and sines
// serves it for all heads of the token.  A task is a token's next U groups of heads (32 / (d / 16)
// heads a group) of one kind (queries, keys or values), whose loads are all requested before
// the first is used; a warp takes consecutive tasks, so that a token's angles and a
// kind's weights are worked out once.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "tr_append.cuh"

namespace {

constexpr int kMaxWarps = 16;

struct RopeArgs {
  const char *x[3];               // queries, keys, values
  long long stride[3][3];         // bytes between sequences, rows, heads
  char *out[3];                   // dense; keys and values only without a cache
  int heads[3];                   // 0: not there
  int B, T, rot;
  const float *inv_freq, *norm[2];
  float eps;
  const int32_t *pos, *count;
  const int2 *todo;               // cache: (old length, rows) of each sequence, or NULL: found here
  unsigned *status;
  int batches[3], all_batches;    // tasks of a token, of each kind
  int per;                        // tasks of a warp
};

// Depths of a tree's nodes; without nodes the positions follow the rows.
struct Depths {
  int nodes;
  uint8_t of[TR_MAX_NODES];
};

__device__ __forceinline__ float2 widen(uint32_t w, bool bf) {
  if (bf) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t narrow(float lo, float hi, bool bf) {
  if (bf) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
  }
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&r);
}

// Turns a position as a fraction of 2^64: a multiplication by the position wraps around
// with the whole turns, so far positions lose nothing.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  const double t = (double)f * 0.15915494309189535;  // 1 / (2 pi)
  return __double2ull_rz((t - floor(t)) * 0x1p64);
}
// cos and sin at position p: the nearest 2^-32 of a turn, as half turns in fp32.
__device__ __forceinline__ float2 turn(long long p, unsigned long long f) {
  const int phase = (int)(((unsigned long long)p * f) >> 32);
  float2 r;
  sincospif((float)phase * 0x1p-31f, &r.y, &r.x);
  return r;
}

// What a warp keeps of a token and a kind.
struct Held {
  float2 cs[8];       // cosines and sines of the lane's pairs
  float w[16];        // norm weights of the lane's elements
};

enum { kDense, kCache, kCache8 };  // where keys and values go

template <bool BF, int D, bool PAIRS, int DST, int U>
struct Rows {
  static constexpr int LPH = D / 16, HPG = 32 / LPH;  // lanes of a head, heads of a group
  const RopeArgs &a;
  const KvDev &c;
  float2 *table;      // the warp's, D / 2
  int lane, sub, head, pa, pb;  // lane of its head, head of the group, the lane's pieces
  bool turned;
  unsigned long long f[D / 64];

  __device__ __forceinline__ Rows(const RopeArgs &a_, const KvDev &c_, float2 *t) : a(a_), c(c_), table(t) {
    lane = threadIdx.x & 31;
    sub = lane % LPH;
    head = lane / LPH;
    turned = sub < a.rot / 16;
    const bool apart = turned && !PAIRS;
    pa = apart ? sub : 2 * sub;
    pb = apart ? sub + a.rot / 16 : 2 * sub + 1;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) f[e] = lane + 32 * e < a.rot / 2 ? turns_of(a.inv_freq[lane + 32 * e]) : 0;
  }

  __device__ __forceinline__ void angles(long long p, Held &k) {
    if (a.rot == 0) return;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      if (lane + 32 * e < a.rot / 2) table[lane + 32 * e] = turn(p, f[e]);
    __syncwarp();
    if (!turned) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 x = reinterpret_cast<const float4 *>(table + sub * 8)[e];
      k.cs[2 * e] = make_float2(x.x, x.y);
      k.cs[2 * e + 1] = make_float2(x.z, x.w);
    }
  }

  __device__ __forceinline__ void weights(int kind, Held &k) {
    const float *w = kind < 2 ? a.norm[kind] : nullptr;
    if (!w) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      k.w[e] = w[pa * 8 + e];
      k.w[8 + e] = w[pb * 8 + e];
    }
  }

  __device__ __forceinline__ void load(int kind, int b, int i, int h0, uint4 (&x)[U][2]) {
    const char *src = a.x[kind] + b * a.stride[kind][0] + i * a.stride[kind][1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPG + head;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (h < a.heads[kind]) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src + h * a.stride[kind][2]);
        x[u][0] = p[pa];
        x[u][1] = p[pb];
      }
    }
  }

  // The task's rows of token i of sequence b, whose place in the cache is p.
  __device__ __forceinline__ void finish(int kind, int b, int i, int p, int h0, const uint4 (&x)[U][2], const Held &k) {
    const bool dense = DST == kDense || kind == 0;
    const long long block = dense ? 0 : kv_block(c, b, p) + kv_row(c, p);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPG + head;
      if (h0 + u * HPG >= a.heads[kind]) break;
      float y[16];
      uint4 out[2] = {x[u][0], x[u][1]};
      if (kind < 2 || DST == kCache8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w[4] = {x[u][q].x, x[u][q].y, x[u][q].z, x[u][q].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = widen(w[e], BF);
            y[8 * q + 2 * e] = v.x;
            y[8 * q + 2 * e + 1] = v.y;
          }
        }
      }
      if (kind < 2) {
        if (a.norm[kind]) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s0 = fmaf(y[e], y[e], s0);
            s1 = fmaf(y[8 + e], y[8 + e], s1);
          }
          float s = s0 + s1;
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
          const float r = rsqrtf(fmaf(s, 1.f / D, a.eps));
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] *= r * k.w[e];
        }
        if (turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float &p0 = y[PAIRS ? 2 * e : e], &p1 = y[PAIRS ? 2 * e + 1 : 8 + e];
            const float z0 = fmaf(p0, k.cs[e].x, -(p1 * k.cs[e].y)), z1 = fmaf(p1, k.cs[e].x, p0 * k.cs[e].y);
            p0 = z0;
            p1 = z1;
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          out[q] = make_uint4(narrow(y[8 * q], y[8 * q + 1], BF), narrow(y[8 * q + 2], y[8 * q + 3], BF),
                              narrow(y[8 * q + 4], y[8 * q + 5], BF), narrow(y[8 * q + 6], y[8 * q + 7], BF));
      }
      if (h >= a.heads[kind]) continue;
      if (dense) {
        uint4 *dst = reinterpret_cast<uint4 *>(a.out[kind] + (((long long)b * a.T + i) * a.heads[kind] + h) * (D * 2));
        dst[pa] = out[0];
        dst[pb] = out[1];
      } else {
        char *dst = (kind == 1 ? c.K : c.V) + block + (long long)h * c.head_stride;
        if constexpr (DST == kCache8) {
          const Scale s = make_scale((kind == 1 ? c.k_scale : c.v_scale)[h]);
          float lo[8], hi[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            lo[e] = y[e];
            hi[e] = y[8 + e];
          }
          reinterpret_cast<uint2 *>(dst)[pa] = e4m3_of(lo, s);
          reinterpret_cast<uint2 *>(dst)[pb] = e4m3_of(hi, s);
        } else {
          reinterpret_cast<uint4 *>(dst)[pa] = out[0];
          reinterpret_cast<uint4 *>(dst)[pb] = out[1];
        }
        if (kind == 1 && c.scores && sub == 0) c.scores[((long long)b * c.Hkv + h) * c.scores_ld + p] = 0.f;
      }
    }
  }

  // Kind and first head of a token's task.
  __device__ __forceinline__ int place(int t, int &h0) const {
    int kind = 0;
    while (t >= a.batches[kind]) t -= a.batches[kind++];
    h0 = t * U * HPG;
    return kind;
  }
};

// Tasks of all tokens in order, a.per consecutive ones to a warp.  CACHE: with the lengths
// that the plan kernel has left in todo.
template <bool BF, int D, bool PAIRS, int DST, int U>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a, const KvDev c, const __grid_constant__ Depths tree) {
  __shared__ __align__(16) float2 tables[8][D / 2];
  tr_let_next_start();
  tr_wait_for_previous();
  const int warp = threadIdx.x >> 5;
  const long long tasks = (long long)a.B * a.T * a.all_batches;
  long long t = ((long long)blockIdx.x * 8 + warp) * a.per;
  const long long t1 = min(tasks, t + a.per);
  if (t >= t1) return;
  Rows<BF, D, PAIRS, DST, U> r(a, c, tables[warp]);
  long long row = t / a.all_batches;
  int at = (int)(t - row * a.all_batches), b = (int)(row / a.T), i = (int)(row - (long long)b * a.T);
  int angle_of = -1, weights_of = -1, p = 0;
  bool there = true;
  Held k;
  for (; t < t1; ++t) {
    int h0;
    const int kind = r.place(at, h0);
    if (angle_of != i) {
      if (DST != kDense) {
        const int2 todo = a.todo[b];
        there = i < todo.y;
        p = todo.x + i;
      }
    }
    if (there) {
      uint4 x[U][2];
      r.load(kind, b, i, h0, x);
      if (angle_of != i && kind < 2) {
        r.angles(a.pos ? (long long)a.pos[b] + (tree.nodes ? tree.of[i] : i) : p, k);
        angle_of = i;
      }
      if (weights_of != kind) r.weights(weights_of = kind, k);
      r.finish(kind, b, i, p, h0, x, k);
    }
    if (++at == a.all_batches) {
      at = 0;
      angle_of = -1;
      if (++i == a.T) {
        i = 0;
        ++b;
      }
    }
  }
}

// Few rows: a cluster takes a sequence, checks it, copies its rows and advances its length,
// so that no kernel is needed before this one.
template <bool BF, int D, bool PAIRS, int DST, int U>
__global__ void __launch_bounds__(kMaxWarps * 32) append_rope_kernel(const RopeArgs a, const KvDev c) {
  __shared__ __align__(16) float2 tables[kMaxWarps][D / 2];
  tr_let_next_start();
  tr_wait_for_previous();
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int b = blockIdx.y, Lb = c.L[b], n0 = a.count ? a.count[b] : a.T;
  const int step = gridDim.x * warps;
  Rows<BF, D, PAIRS, DST, U> r(a, c, tables[warp]);
  int t = blockIdx.x * warps + warp, i = t / a.all_batches, at = t - i * a.all_batches, h0;
  int kind = r.place(at, h0);
  // the first task's rows are requested before the checks (they are read even if these fail)
  uint4 x[U][2];
  if (i < a.T) r.load(kind, b, i, h0, x);
  const long long base = a.pos ? (long long)a.pos[b] : Lb;
  const int n = append_rows(c, b, Lb, n0, a.T, a.status);
  int angle_of = -1, weights_of = -1;
  Held k;
  while (i < n) {
    if (angle_of != i && kind < 2) r.angles(base + (angle_of = i), k);
    if (weights_of != kind) r.weights(weights_of = kind, k);
    r.finish(kind, b, i, Lb + i, h0, x, k);
    t += step;
    i = t / a.all_batches;
    at = t - i * a.all_batches;
    kind = r.place(at, h0);
    if (i < n) r.load(kind, b, i, h0, x);
  }
  if (gridDim.x > 1) {  // the sequence's other CTAs have read the old length
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && n > 0) c.L[b] = Lb + n;
}

// Checks the rows and the rotation on the host and fills what the kernel needs of them.
int fill(const tr_qkv *x, const tr_rope *r, const int32_t *pos, RopeArgs *out) {
  if (!x || !r || x->B < 1 || x->T < 1) return TR_E_INVAL;
  if (x->type != TR_KV_BF16 && x->type != TR_KV_F16) return TR_E_INVAL;
  if (!x->Q && !x->K && !x->V) return TR_E_INVAL;
  if ((x->Q && x->Hq < 1) || ((x->K || x->V) && x->Hkv < 1)) return TR_E_INVAL;
  if (r->d < 1 || r->rot < 0 || r->rot > r->d || (r->rot && !r->inv_freq)) return TR_E_INVAL;
  if (((uintptr_t)r->inv_freq | (uintptr_t)r->q_norm | (uintptr_t)r->k_norm | (uintptr_t)pos) & 3) return TR_E_INVAL;
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return TR_E_INVAL;
  RopeArgs a = {};
  const void *p[3] = {x->Q, x->K, x->V};
  const int64_t *st[3] = {x->q_stride, x->k_stride, x->v_stride};
  const int heads[3] = {x->Hq, x->Hkv, x->Hkv};
  long long all = 0;
  for (int i = 0; i < 3; ++i) {
    if (!p[i]) continue;
    if ((uintptr_t)p[i] & 15) return TR_E_INVAL;
    a.x[i] = (const char *)p[i];
    a.heads[i] = heads[i];
    all += heads[i];
    const int n[3] = {x->B, x->T, heads[i]};
    for (int j = 0; j < 3; ++j) {
      const int64_t s = n[j] == 1 ? 0 : st[i][j];
      if (s < 0 || s > (1LL << 58) / n[j] || (s & 7)) return TR_E_INVAL;
      a.stride[i][j] = s * 2;
    }
  }
  if ((r->d != 64 && r->d != 128) || r->rot % 16) return TR_E_UNSUPPORTED;
  if ((long long)x->B * x->T >= (1LL << 31) || all > (1 << 20)) return TR_E_UNSUPPORTED;
  a.B = x->B;
  a.T = x->T;
  a.rot = r->rot;
  a.inv_freq = r->inv_freq;
  a.norm[0] = r->q_norm;
  a.norm[1] = r->k_norm;
  a.eps = r->eps;
  a.pos = pos;
  *out = a;
  return TR_OK;
}

// Groups of a task in a large call, and in a small one.
constexpr int kWide = 4, kShort = 2;

// Tasks of a token; returns their number.
int plan(RopeArgs *a, int d, int U) {
  const int heads = 32 / (d / 16) * U;
  a->all_batches = 0;
  for (int i = 0; i < 3; ++i) a->all_batches += a->batches[i] = (a->heads[i] + heads - 1) / heads;
  return a->all_batches;
}

template <bool BF, int D, bool PAIRS, int DST>
int launch(RopeArgs a, const KvDev &c, const Depths &tree, cudaStream_t s) {
  auto go = [&](auto kernel, int U) {
    const long long tasks = (long long)a.B * a.T * plan(&a, D, U);
    a.per = tasks >= 64LL * tr_sm_count() ? a.all_batches : 1;
    const long long ctas = (tasks + 8LL * a.per - 1) / (8LL * a.per);
    if (ctas >= (1LL << 31)) return (int)TR_E_UNSUPPORTED;
    return tr_launch_next(kernel, {dim3((unsigned)ctas), 256}, s, a, c, tree);
  };
  const long long wide = (long long)a.B * a.T * plan(&a, D, kWide);
  if (wide >= 16LL * tr_sm_count()) return go(rope_kernel<BF, D, PAIRS, DST, kWide>, kWide);
  return go(rope_kernel<BF, D, PAIRS, DST, kShort>, kShort);
}

// One kernel for a sequence's rows up to this many tasks of a warp.
constexpr int kRounds = 4, kMostCluster = 8;

template <bool BF, int D, bool PAIRS, int DST>
int launch_append(RopeArgs a, const KvDev &c, const int32_t *count, void *ws, cudaStream_t s) {
  const long long tasks = (long long)a.T * plan(&a, D, kShort);
  if (tasks <= (long long)kMostCluster * kMaxWarps * kRounds) {
    int cs = 1;
    while (cs < kMostCluster && tasks > (long long)cs * kMaxWarps) cs *= 2;
    const int warps = (int)std::min<long long>(kMaxWarps, (tasks + cs - 1) / cs);
    a.count = count;
    a.status = tr_status_dev();
    return tr_launch_next(append_rope_kernel<BF, D, PAIRS, DST, kShort>, {dim3(cs, a.B), warps * 32, 0, cs}, s, a, c);
  }
  a.todo = (const int2 *)ws;
  const int rc = kv_append_plan(c, a.T, count, (int2 *)ws, s);
  return rc != TR_OK ? rc : launch<BF, D, PAIRS, DST>(a, c, Depths{}, s);
}

// f(BF, D, PAIRS) as compile-time constants.
template <typename F>
int with(bool bf, int d, bool pairs, F f) {
  using T = std::true_type;
  using N = std::false_type;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  auto second = [&](auto t) {
    return d == 64 ? (pairs ? f(t, D64{}, T{}) : f(t, D64{}, N{})) : (pairs ? f(t, D128{}, T{}) : f(t, D128{}, N{}));
  };
  return bf ? second(T{}) : second(N{});
}

}  // namespace

extern "C" int tr_qkv_rope(const tr_qkv *rows, const tr_rope *rope, const int32_t *pos, const struct tr_tree *tree,
                           void *Qo, void *Ko, void *Vo, tr_stream_t stream) {
  RopeArgs a;
  int rc = fill(rows, rope, pos, &a);
  if (rc != TR_OK) return rc;
  if (!rows->Q != !Qo || !rows->K != !Ko || !rows->V != !Vo) return TR_E_INVAL;
  if (((uintptr_t)Qo | (uintptr_t)Ko | (uintptr_t)Vo) & 15) return TR_E_INVAL;
  if (rope->rot && !pos) return TR_E_INVAL;
  if (tree && tree->dev.N != rows->T) return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  a.out[0] = (char *)Qo;
  a.out[1] = (char *)Ko;
  a.out[2] = (char *)Vo;
  Depths depths = {};
  if (tree) {
    depths.nodes = tree->dev.N;
    memcpy(depths.of, tree->dev.depth, sizeof(depths.of));
  }
  return with(rows->type == TR_KV_BF16, rope->d, rope->pairs != 0, [&](auto bf, auto d, auto pairs) {
    return launch<bf.value, d.value, pairs.value, kDense>(a, KvDev{}, depths, (cudaStream_t)stream);
  });
}

extern "C" int tr_kv_append_rope(const tr_qkv *rows, const tr_rope *rope, const int32_t *pos, const int32_t *count,
                                 const tr_kv_cache *cache, void *Qo, void *ws, size_t ws_bytes, tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  RopeArgs a;
  rc = fill(rows, rope, pos, &a);
  if (rc != TR_OK) return rc;
  if (!rows->K || !rows->V || !rows->Q != !Qo || ((uintptr_t)Qo & 15)) return TR_E_INVAL;
  if ((uintptr_t)count & 3) return TR_E_INVAL;
  if (rows->B != cache->B || rows->Hkv != cache->Hkv || rope->d != cache->d) return TR_E_INVAL;
  if (rows->type != (cache->type == TR_KV_F16 ? TR_KV_F16 : TR_KV_BF16)) return TR_E_INVAL;
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < tr_kv_append_workspace_bytes(cache)) return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  a.out[0] = (char *)Qo;
  cudaStream_t s = (cudaStream_t)stream;
  return with(rows->type == TR_KV_BF16, rope->d, rope->pairs != 0, [&](auto bf, auto d, auto pairs) {
    if constexpr (bf.value)
      if (cache->type == TR_KV_E4M3) return launch_append<true, d.value, pairs.value, kCache8>(a, c, count, ws, s);
    return launch_append<bf.value, d.value, pairs.value, kCache>(a, c, count, ws, s);
  });
}
