// Norms of queries and keys per head with the position rotation in the same pass,
// into dense rows (tr_qkv_rope) or, for keys and values, into a KV cache
// (tr_kv_append_rope).
//
// A row x of d elements: y = x w / sqrt(mean x^2 + eps), then pairs of elements turned
// by the angle p f_i.  Every element is read once and written once; a few flops each.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "tr_kv.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct RopeArgs {
  const char *x[3];               // queries, keys, values
  long long stride[3][3];         // bytes between sequences, rows, heads
  char *out[3];                   // dense; keys and values only without a cache
  int heads[3];                   // 0: not there
  int T, rot, pairs;
  const float *inv_freq, *norm[2];
  float eps;
  const int32_t *pos;
  const int2 *todo;               // cache: (old length, rows) of each sequence
};

template <bool BF>
__device__ __forceinline__ float load16(const char *p, int i) {
  if (BF) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(reinterpret_cast<const __half *>(p)[i]);
}
template <bool BF>
__device__ __forceinline__ void store16(char *p, int i, float x) {
  if (BF) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half *>(p)[i] = __float2half_rn(x);
}

// cos and sin of position p times the frequency f: the angle in turns in 64 bits, its
// whole turns dropped, so that far positions lose nothing.
__device__ __forceinline__ float2 turn(long long p, float f) {
  const double t = (double)p * ((double)f * 0.15915494309189535);  // 1 / (2 pi)
  const float half_turns = (float)(2.0 * (t - rint(t)));
  float2 r;
  sincospif(half_turns, &r.y, &r.x);
  return r;
}

// One warp per (row, head).  CACHE: keys and values go to the cache.
template <bool BF, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, const KvDev c, int d, int B,
                                                        const __grid_constant__ TreeDev tree, bool has_tree) {
  tr_let_next_start();
  tr_wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int all = a.heads[0] + a.heads[1] + a.heads[2];
  const long long items = (long long)B * a.T * all;
  for (long long it = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items;
       it += (long long)gridDim.x * kWarps) {
    const long long row = it / all;
    int h = (int)(it - row * all);
    const int b = (int)(row / a.T), i = (int)(row - (long long)b * a.T);
    int kind = 0;
    while (h >= a.heads[kind]) h -= a.heads[kind++];
    int2 todo = make_int2(0, 0);
    if (CACHE) {
      todo = a.todo[b];
      if (i >= todo.y) continue;
    }
    const char *src = a.x[kind] + b * a.stride[kind][0] + i * a.stride[kind][1] + h * a.stride[kind][2];
    float x[4];
    const int n = d / 32;
    for (int e = 0; e < n; ++e) x[e] = load16<BF>(src, lane + 32 * e);
    if (kind < 2) {
      if (a.norm[kind]) {
        float sum = 0.f;
        for (int e = 0; e < n; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float r = rsqrtf(sum / d + a.eps);
        for (int e = 0; e < n; ++e) x[e] = x[e] * r * a.norm[kind][lane + 32 * e];
      }
      if (a.rot) {
        const long long p = (a.pos ? a.pos[b] : todo.x) + (long long)(has_tree ? tree.depth[i] : i);
        // a pair's elements lie in different lanes: through shared memory, a row for each warp
        __shared__ float rows[kWarps][128];
        float *y = rows[threadIdx.x >> 5];
        __syncwarp();
        for (int e = 0; e < n; ++e) y[lane + 32 * e] = x[e];
        __syncwarp();
        for (int e = 0; e < n; ++e) {
          const int at = lane + 32 * e;
          if (at >= a.rot) continue;
          const int half = a.rot / 2;
          const int pair = a.pairs ? at / 2 : at % half;
          const bool second = a.pairs ? at & 1 : at >= half;
          const float mate = y[a.pairs ? at ^ 1 : second ? at - half : at + half];
          const float2 cs = turn(p, a.inv_freq[pair]);
          x[e] = second ? fmaf(x[e], cs.x, mate * cs.y) : fmaf(x[e], cs.x, -(mate * cs.y));
        }
      }
    }
    if (!CACHE || kind == 0) {
      char *dst = a.out[kind] + (row * a.heads[kind] + h) * d * 2;
      for (int e = 0; e < n; ++e) store16<BF>(dst, lane + 32 * e, x[e]);
      continue;
    }
    const int p = todo.x + i;
    char *dst = (kind == 1 ? c.K : c.V) + kv_block(c, b, p) + (long long)h * c.head_stride + kv_row(c, p);
    if (c.k_scale) {
      const float s = (kind == 1 ? c.k_scale : c.v_scale)[h];
      for (int e = 0; e < n; ++e)
        dst[lane + 32 * e] = (char)__nv_cvt_float_to_fp8(__fdiv_rn(x[e], s), __NV_SATFINITE, __NV_E4M3);
    } else {
      for (int e = 0; e < n; ++e) store16<BF>(dst, lane + 32 * e, x[e]);
    }
    if (kind == 1 && c.scores && lane == 0) c.scores[((long long)b * c.Hkv + h) * c.scores_ld + p] = 0.f;
  }
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
  a.T = x->T;
  a.rot = r->rot;
  a.pairs = r->pairs;
  a.inv_freq = r->inv_freq;
  a.norm[0] = r->q_norm;
  a.norm[1] = r->k_norm;
  a.eps = r->eps;
  a.pos = pos;
  *out = a;
  return TR_OK;
}

unsigned grid_of(const RopeArgs &a, int B) {
  const long long items = (long long)B * a.T * (a.heads[0] + a.heads[1] + a.heads[2]);
  const long long ctas = (items + kWarps - 1) / kWarps, most = 64LL * tr_sm_count();
  return (unsigned)(ctas < most ? ctas : most);
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
  const TreeDev none = {};
  auto go = [&](auto kernel) {
    return tr_launch_next(kernel, {dim3(grid_of(a, rows->B)), kThreads}, (cudaStream_t)stream, a, KvDev{}, rope->d,
                          rows->B, tree ? tree->dev : none, tree != nullptr);
  };
  return rows->type == TR_KV_BF16 ? go(rope_kernel<true, false>) : go(rope_kernel<false, false>);
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
  a.todo = (const int2 *)ws;
  cudaStream_t s = (cudaStream_t)stream;
  rc = kv_append_plan(c, rows->T, count, (int2 *)ws, s);
  if (rc != TR_OK) return rc;
  auto go = [&](auto kernel) {
    return tr_launch_next(kernel, {dim3(grid_of(a, rows->B)), kThreads}, s, a, c, rope->d, rows->B, TreeDev{}, false);
  };
  return rows->type == TR_KV_BF16 ? go(rope_kernel<true, true>) : go(rope_kernel<false, true>);
}
