// Appending rows to a KV cache and evicting rows from it by accumulated
// attention weight.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "tr_kv.cuh"

namespace {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;  // 16-byte pieces of K and of V per thread

// Eight bf16 values divided by the head's scale and rounded to e4m3: IEEE
// division and one rounding to nearest even (the conversion clamps to +-448).
__device__ __forceinline__ uint2 e4m3_of(const uint4 &x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
    r[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// One thread per 16-byte piece of a new row (8 elements), K and V together.
// Every CTA of a sequence decides alike whether the sequence can take its
// rows; the last one to finish advances L[b], so that none reads a changed
// length.
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const KvDev c, const uint4 *Kn, const uint4 *Vn, int T,
                                                                const int32_t *count, unsigned *counters,
                                                                unsigned *status) {
  const int b = blockIdx.y;
  const int Lb = c.L[b], n = count ? count[b] : T;
  const bool bad_len = Lb < 0 || Lb > c.cap || n < 0 || n > T;
  const bool full = !bad_len && n > c.cap - Lb;
  bool bad_page = false;
  if (!bad_len && !full) bad_page = kv_bad_pages(c, b, Lb, Lb + n);
  if (!bad_len && !full && !bad_page) {
    const int pieces = c.row_bytes / (E4M3 ? 8 : 16);  // of a row
    const long long total = (long long)n * c.Hkv * pieces;
    const long long base = (long long)b * T * c.Hkv * pieces;
    const long long i0 = (long long)blockIdx.x * (kAppendThreads * kAppendUnroll) + threadIdx.x;
    uint4 kx[kAppendUnroll], vx[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const long long i = i0 + u * kAppendThreads;
      if (i < total) {
        kx[u] = __ldcs(Kn + base + i);
        vx[u] = __ldcs(Vn + base + i);
      }
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const long long i = i0 + u * kAppendThreads;
      if (i >= total) continue;
      const int piece = (int)(i % pieces);
      const long long th = i / pieces;
      const int h = (int)(th % c.Hkv), p = Lb + (int)(th / c.Hkv);
      const long long at = kv_block(c, b, p) + (long long)h * c.head_stride + kv_row(c, p) + piece * (E4M3 ? 8 : 16);
      if constexpr (E4M3) {
        *reinterpret_cast<uint2 *>(c.K + at) = e4m3_of(kx[u], __ldg(c.k_scale + h));
        *reinterpret_cast<uint2 *>(c.V + at) = e4m3_of(vx[u], __ldg(c.v_scale + h));
      } else {
        *reinterpret_cast<uint4 *>(c.K + at) = kx[u];
        *reinterpret_cast<uint4 *>(c.V + at) = vx[u];
      }
      if (c.scores && piece == 0) c.scores[((long long)b * c.Hkv + h) * c.scores_ld + p] = 0.f;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned G = gridDim.x;
    bool last = true;
    if (G > 1) {
      __threadfence();
      last = atomicAdd(&counters[b], 1u) == G - 1;
    }
    if (last) {
      if (bad_len) tr_flag(status, TR_DEV_BAD_LENGTH);
      else if (full) tr_flag(status, TR_DEV_CACHE_FULL);
      else if (bad_page) tr_flag(status, TR_DEV_BAD_PAGE);
      else c.L[b] = Lb + n;
      if (G > 1) counters[b] = 0u;
    }
  }
}

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;
constexpr int kPartBytes = 64;  // columns of a row that one CTA moves

// Order of the scores: larger first, -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t score_key(float s) { return s != s ? 0u : tr_ord(s); }

struct SelSmem {
  unsigned hist[256];
  unsigned warp_sel[kSelThreads / 32], warp_eq[kSelThreads / 32];
  unsigned prefix, need;
};

// One CTA per (KV head, sequence).  Finds the key of the k-th largest score
// among the rows before the protected ones (radix select, eight bits a pass),
// then walks all rows in order, writes the positions that stay to keep and
// moves their scores up.  A score only moves down in position and every chunk
// is read before it is written, so the walk can work in place.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const KvDev c, int budget, int recent, int32_t *keep,
                                                                   int32_t *old_len, unsigned *status) {
  __shared__ SelSmem s;
  const int h = blockIdx.x, b = blockIdx.y;
  const int Lb = c.L[b];
  const bool bad_len = Lb < 0 || Lb > c.cap;
  const bool active = !bad_len && Lb > budget;
  const bool bad_page = active && kv_bad_pages(c, b, 0, Lb);
  if (h == 0 && threadIdx.x == 0) {
    old_len[b] = active && !bad_page ? Lb : -1;
    if (bad_len) tr_flag(status, TR_DEV_BAD_LENGTH);
    if (bad_page) tr_flag(status, TR_DEV_BAD_PAGE);
  }
  if (!active || bad_page) return;
  float *sc = c.scores + ((long long)b * c.Hkv + h) * c.scores_ld;
  keep += ((long long)b * c.Hkv + h) * budget;
  const int n = Lb - recent, k = budget - recent;  // k < n
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // key of the k-th largest: `prefix` holds its leading bits, `need` how many
  // of the rows that share them are still to be taken
  unsigned prefix = 0, need = k;
  if (k > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) s.hist[i] = 0;
      __syncthreads();
      const unsigned mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int i = threadIdx.x; i < n; i += kSelThreads) {
        const unsigned key = score_key(sc[i]);
        if ((key & mask) == prefix) atomicAdd(&s.hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l owns bins 255-8l .. 248-8l: running count from the largest key down
        unsigned sum = 0;
        for (int j = 0; j < 8; ++j) sum += s.hist[255 - 8 * lane - j];
        unsigned incl = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_up_sync(~0u, incl, o);
          if (lane >= o) incl += v;
        }
        unsigned before = incl - sum;
        if (before < need && need <= incl) {
          int bin = 255 - 8 * lane;
          while (before + s.hist[bin] < need) before += s.hist[bin--];
          s.prefix = prefix | ((unsigned)bin << shift);
          s.need = need - before;
        }
      }
      __syncthreads();
      prefix = s.prefix;
      need = s.need;
    }
  }
  // rows in order: all above the k-th key, the first `need` of those equal to it, all protected ones
  unsigned taken = 0, equal = 0;
  for (int i0 = 0; i0 < Lb; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    const float v = i < Lb ? sc[i] : 0.f;
    const unsigned key = score_key(v);
    const bool eq = k > 0 && i < n && key == prefix;
    const unsigned eqs = __ballot_sync(~0u, eq), below = (1u << lane) - 1;
    if (lane == 0) s.warp_eq[warp] = __popc(eqs);
    __syncthreads();
    unsigned eq_before = equal, eq_all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) eq_before += s.warp_eq[w];
      eq_all += s.warp_eq[w];
    }
    eq_before += __popc(eqs & below);
    const bool sel = i < Lb && (i >= n || (k > 0 && (key > prefix || (eq && eq_before < need))));
    const unsigned sels = __ballot_sync(~0u, sel);
    if (lane == 0) s.warp_sel[warp] = __popc(sels);
    __syncthreads();
    unsigned at = taken, all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) at += s.warp_sel[w];
      all += s.warp_sel[w];
    }
    at += __popc(sels & below);
    if (sel) {
      keep[at] = i;
      sc[at] = v;
    }
    taken += all;
    equal += eq_all;
    __syncthreads();
  }
}

// Moves the kept rows of K and V up, in place.  A CTA owns 64 bytes of every
// row of one (sequence, KV head), of K or of V, so no two CTAs touch the same
// bytes, and walks the kept rows in order.  Row r comes from keep[r] >= r:
// writing rows [r0, r0 + n) can only hit sources of rows < r0 + n, so it is
// enough that a batch is read before it is written, which a barrier ensures.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const KvDev c, int budget, const int32_t *keep,
                                                                  const int32_t *old_len) {
  constexpr int kLanes = kPartBytes / 16, kRows = kMoveThreads / kLanes;
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  if (old_len[b] < 0) return;
  const int per = c.row_bytes / kPartBytes;
  char *base = (part < per ? c.K : c.V) + (long long)h * c.head_stride + (part % per) * kPartBytes +
               (threadIdx.x % kLanes) * 16;
  keep += ((long long)b * c.Hkv + h) * budget;
  const int row = threadIdx.x / kLanes;
  for (int r0 = 0; r0 < budget; r0 += kRows * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    bool moves[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int r = r0 + u * kRows + row;
      const int src = r < budget ? __ldg(keep + r) : r;
      moves[u] = src != r;
      if (moves[u]) x[u] = *reinterpret_cast<const uint4 *>(base + kv_block(c, b, src) + kv_row(c, src));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int r = r0 + u * kRows + row;
      if (moves[u]) *reinterpret_cast<uint4 *>(base + kv_block(c, b, r) + kv_row(c, r)) = x[u];
    }
  }
  if (part == 0 && h == 0 && threadIdx.x == 0) c.L[b] = budget;
}

// Workspace: the kept positions of every (sequence, KV head), then the old
// lengths.  A budget that no sequence can exceed keeps no positions.
size_t keep_bytes(const KvDev &c, int budget) {
  return budget < c.cap ? tr_align_up((size_t)c.B * c.Hkv * (size_t)budget * 4, 256) : 0;
}

size_t evict_bytes(const KvDev &c, int budget) { return keep_bytes(c, budget) + tr_align_up((size_t)c.B * 4, 256); }

}  // namespace

// ---------------------------------------------------------------------------
// ABI
// ---------------------------------------------------------------------------

extern "C" size_t tr_kv_append_workspace_bytes(const tr_kv_cache *cache) {
  return cache && cache->B > 0 ? tr_align_up((size_t)cache->B * 4, 256) : 0;
}

extern "C" int tr_kv_append(const void *Kn, const void *Vn, int T, const int32_t *count, const tr_kv_cache *cache,
                            void *ws, size_t ws_bytes, tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  if (!Kn || !Vn || T < 1 || (((uintptr_t)Kn | (uintptr_t)Vn) & 15)) return TR_E_INVAL;
  const bool e4m3 = cache->type == TR_KV_E4M3;
  const long long pieces = (long long)T * c.Hkv * (cache->d / 8);
  const long long per = kAppendThreads * kAppendUnroll;
  const long long grid = (pieces + per - 1) / per;
  if (grid >= (1LL << 31)) return TR_E_UNSUPPORTED;
  if (grid > 1 && (!ws || ((uintptr_t)ws & 15) || ws_bytes < tr_kv_append_workspace_bytes(cache))) return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  const dim3 g((unsigned)grid, (unsigned)c.B);
  cudaStream_t s = (cudaStream_t)stream;
  if (e4m3)
    append_kernel<true><<<g, kAppendThreads, 0, s>>>(c, (const uint4 *)Kn, (const uint4 *)Vn, T, count, (unsigned *)ws,
                                                     tr_status_dev());
  else
    append_kernel<false><<<g, kAppendThreads, 0, s>>>(c, (const uint4 *)Kn, (const uint4 *)Vn, T, count,
                                                      (unsigned *)ws, tr_status_dev());
  TR_LAUNCH_CHECK();
  return TR_OK;
}

extern "C" size_t tr_kv_evict_workspace_bytes(const tr_kv_cache *cache, int budget) {
  KvDev c;
  return budget >= 1 && kv_check(cache, &c) == TR_OK ? evict_bytes(c, budget) : 0;
}

extern "C" int tr_kv_evict(const tr_kv_cache *cache, int budget, int recent, void *ws, size_t ws_bytes,
                           tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  if (!c.scores || budget < 1 || recent < 0 || recent > budget) return TR_E_INVAL;
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < evict_bytes(c, budget)) return TR_E_INVAL;
  if (c.Hkv > 65535) return TR_E_UNSUPPORTED;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  int32_t *old_len = (int32_t *)((char *)ws + keep_bytes(c, budget));
  cudaStream_t s = (cudaStream_t)stream;
  // with a budget that the cache cannot exceed this still reports bad lengths
  evict_select_kernel<<<dim3(c.Hkv, c.B), kSelThreads, 0, s>>>(c, budget, recent, (int32_t *)ws, old_len,
                                                               tr_status_dev());
  TR_LAUNCH_CHECK();
  if (budget < c.cap) {
    evict_move_kernel<<<dim3(2 * c.row_bytes / kPartBytes, c.Hkv, c.B), kMoveThreads, 0, s>>>(
        c, budget, (const int32_t *)ws, old_len);
    TR_LAUNCH_CHECK();
  }
  return TR_OK;
}
