// Attention of one new token per sequence over a KV cache.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "tr_kv.cuh"
#include "tr_sm100.cuh"

namespace {

constexpr int kWarps = 8;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeArgs {
  const void *Q;
  float *O, *lse;
  float *s;  // workspace: logits (log2 units) [B, Hq, ld]
  long long s_ld;
  int Hq, G, accumulate;
  float scale_log2;
  unsigned *status;
};

template <int TYPE, int N>
__device__ __forceinline__ void load_row(const char *p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (TYPE == TR_KV_BF16) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p + 2 * i));
      x[i] = f.x;
      x[i + 1] = f.y;
    } else if constexpr (TYPE == TR_KV_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(p + 2 * i));
      x[i] = f.x;
      x[i + 1] = f.y;
    } else {
      const __half2 v = __half2(__nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const unsigned short *>(p + i), __NV_E4M3));
      const float2 f = __half22float2(v);
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}

// One CTA per (KV head, sequence), one query head after the other: each warp
// takes every eighth key with a running maximum and sum, the warps' parts are
// joined in shared memory.
template <int TYPE, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const KvDev c, const DecodeArgs a) {
  constexpr int N = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int L = c.L[b];
  if (L < 0 || L > c.cap) {
    if (h == 0 && threadIdx.x == 0) tr_flag(a.status, TR_DEV_BAD_LENGTH);
    L = 0;
  }
  const float ks = TYPE == TR_KV_E4M3 ? __ldg(c.k_scale + h) : 1.f, vs = TYPE == TR_KV_E4M3 ? __ldg(c.v_scale + h) : 1.f;
  constexpr int ESZ = TYPE == TR_KV_E4M3 ? 1 : 2;
  constexpr int QT = TYPE == TR_KV_F16 ? TR_KV_F16 : TR_KV_BF16;
  for (int g = 0; g < a.G; ++g) {
    const long long row = (long long)b * a.Hq + h * a.G + g;
    float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
    load_row<QT, N>((const char *)a.Q + (row * D + lane * N) * 2, q);
    for (int p = warp; p < L; p += kWarps) {
      const long long blk = kv_block(c, b, p);
      if (blk < 0) {
        if (lane == 0) tr_flag(a.status, TR_DEV_BAD_PAGE);
        continue;
      }
      const long long at = blk + (long long)h * c.head_stride + kv_row(c, p) + lane * N * ESZ;
      float k[N], v[N], s = 0.f;
      load_row<TYPE, N>(c.K + at, k);
      load_row<TYPE, N>(c.V + at, v);
#pragma unroll
      for (int i = 0; i < N; ++i) s += q[i] * k[i];
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
      s *= a.scale_log2 * ks;
      if (a.accumulate && lane == 0) a.s[row * a.s_ld + p] = s;
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
      l = l * f + w;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = o[i] * f + w * v[i];
      m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < N; ++i) so[warp][lane * N + i] = o[i];
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) sum += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
      float x = 0.f;
      for (int w = 0; w < kWarps; ++w) x += sm[w] == -INFINITY ? 0.f : so[w][d] * exp2f(sm[w] - M);
      a.O[row * D + d] = sum > 0.f ? x / sum * vs : 0.f;
    }
    const float lse2 = sum > 0.f ? M + log2f(sum) : -INFINITY;
    if (a.lse && threadIdx.x == 0) a.lse[row] = lse2 * kLn2;
    if (a.accumulate)
      for (int p = threadIdx.x; p < L; p += kWarps * 32)
        if (kv_block(c, b, p) >= 0)
          c.scores[((long long)b * c.Hkv + h) * c.scores_ld + p] += exp2f(a.s[row * a.s_ld + p] - lse2);
    __syncthreads();
  }
}

template <int TYPE>
void launch(int d, dim3 grid, cudaStream_t s, const KvDev &c, const DecodeArgs &a) {
  if (d == 64)
    decode_kernel<TYPE, 64><<<grid, kWarps * 32, 0, s>>>(c, a);
  else
    decode_kernel<TYPE, 128><<<grid, kWarps * 32, 0, s>>>(c, a);
}

}  // namespace

extern "C" size_t tr_decode_attn_workspace_bytes(const tr_kv_cache *cache, int Hq, int accumulate) {
  KvDev c;
  if (kv_check(cache, &c) != TR_OK || Hq < 1 || Hq % c.Hkv) return 0;
  return accumulate ? (size_t)c.B * Hq * tr_align_up(c.cap, 16) * 4 : 256;
}

extern "C" int tr_decode_attn(const void *Q, const tr_kv_cache *cache, int Hq, float scale, float *O, float *lse,
                              int accumulate, void *ws, size_t ws_bytes, tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  if (!Q || !O || Hq < 1 || Hq % c.Hkv || !(scale > 0.f) || !(scale < INFINITY)) return TR_E_INVAL;
  if ((((uintptr_t)Q | (uintptr_t)O) & 15) || ((uintptr_t)lse & 3)) return TR_E_INVAL;
  if (accumulate && !c.scores) return TR_E_INVAL;
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < tr_decode_attn_workspace_bytes(cache, Hq, accumulate))
    return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  DecodeArgs a;
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.s = (float *)ws;
  a.s_ld = (long long)tr_align_up(c.cap, 16);
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.accumulate = accumulate;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = tr_status_dev();
  const dim3 grid(c.Hkv, c.B);
  cudaStream_t s = (cudaStream_t)stream;
  if (cache->type == TR_KV_BF16)
    launch<TR_KV_BF16>(cache->d, grid, s, c, a);
  else if (cache->type == TR_KV_F16)
    launch<TR_KV_F16>(cache->d, grid, s, c, a);
  else
    launch<TR_KV_E4M3>(cache->d, grid, s, c, a);
  TR_LAUNCH_CHECK();
  return TR_OK;
}
