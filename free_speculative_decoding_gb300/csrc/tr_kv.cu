// Appending rows to a KV cache and evicting rows from it by accumulated
// attention weight.
//
// Both move bytes and are bound by HBM where there are enough of them.  Measured
// (one GB300, in a graph, fractions of the 6675 GB/s of a copy over the bytes
// that the call cannot do without): 8 prompts of up to 4096 rows into an 8-bit
// cache 28 us = 66% (its floor 18.6 us; the kernel is bound by the instructions of the
// division: 22.6 M of them with one IEEE division per value took 49 us), into a 16-bit
// one 29 us = 86%; one new row for each of 16 sequences 2.2 us behind another kernel, a
// launch (8-bit 2.7); 16 x 32 heads of 4096 rows cut to 1024, 100 us = 82% (choosing
// 16 us, moving 81 us = 98%; of 128-byte rows 68 us = 62%, of 64-byte ones 50 us =
// 43%); one sequence of 131072 rows x 8 heads cut to 32768, 76 us = 54% (choosing
// 20 us; moving 11 + 13 + 33 us; of 128-byte rows 57 us = 37%, of 64-byte ones 50 us = 22%).
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "tr_kv.cuh"

namespace {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;  // 16-byte pieces of K and of V per thread

// x / s rounded to the nearest fp32, as far as its rounding to e4m3 can tell, from
// r = RN(1 / s): q0 = x r, q = q0 + r (x - q0 s) (Markstein 1990: with fused
// multiply-adds the last step rounds correctly).  For s in [2^-60, 2^60]: x is
// first held to +-most, a bf16 number between 1024 s and 1033 s (the quotient is
// past 448 either way, and nothing overflows; NaN stays), and where the remainder
// underflows the quotient is below 2^-40, which rounds to 0 either way.  The remainder
// is exact and a zero one is made -0, which takes no sign from q0: -0 / s stays -0.
// Other scales (r = 0) take the division itself, which costs two to three times as much.
struct Scale {
  float s, r;
  uint32_t most;  // twice
};
__device__ __forceinline__ Scale make_scale(float s) {
  const uint32_t m = (__float_as_uint(1024.f * s) + 0xFFFFu) >> 16;
  return {s, s >= 0x1p-60f && s <= 0x1p60f ? __frcp_rn(s) : 0.f, m | (m << 16)};
}

// Two fp32 values in one instruction: a * b, and a * b + c.
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b, float m) {
  asm("{ .reg .b64 p, q; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mul.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m));
}
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float m, float c, float d) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mov.b64 r, {%5, %6};"
      " fma.rn.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m), "f"(c), "f"(d));
}
// The same rounded down: where the sum is exact only the sign of a zero differs, which is -0
// unless both terms are +0.
__device__ __forceinline__ void fma2_down(float &x, float &y, float a, float b, float m, float c, float d) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mov.b64 r, {%5, %6};"
      " fma.rm.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m), "f"(c), "f"(d));
}
// bf16 pairs held to +-most; NaN stays.
__device__ __forceinline__ uint32_t hold2(uint32_t x, uint32_t most) {
  uint32_t r;
  asm("{ .reg .b32 p; min.NaN.bf16x2 p, %1, %2; max.NaN.bf16x2 %0, p, %3; }"
      : "=r"(r)
      : "r"(x), "r"(most), "r"(most | 0x80008000u));
  return r;
}

// Eight bf16 values divided by the head's scale and rounded to e4m3 (one
// rounding of the fp32 quotient to nearest even, clamped to +-448).
__device__ __forceinline__ uint2 e4m3_of(const uint4 &x, const Scale &sc) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
  if (sc.r != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = hold2(w[i], sc.most);
      const float lo = __uint_as_float(h << 16), hi = __uint_as_float(h & 0xFFFF0000u);
      float p, q, u, v;
      mul2(p, q, lo, hi, sc.r);
      fma2_down(u, v, p, q, -sc.s, lo, hi);
      fma2(p, q, u, v, sc.r, p, q);
      r[i] = __nv_cvt_float2_to_fp8x2(make_float2(p, q), __NV_SATFINITE, __NV_E4M3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
      r[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(lo, sc.s), __fdiv_rn(hi, sc.s)), __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Whether a sequence can take its rows (the same answer in every thread of the
// block; contains a barrier): the rows to copy, or -1 with the status bit set.
__device__ __forceinline__ int append_rows(const KvDev &c, int b, int Lb, int n, int T, unsigned *status) {
  const bool bad_len = Lb < 0 || Lb > c.cap || n < 0 || n > T;
  const bool full = !bad_len && n > c.cap - Lb;
  const bool bad_page = kv_bad_pages(c, b, Lb, bad_len || full ? Lb : Lb + n);
  if (!bad_len && !full && !bad_page) return n;
  if (threadIdx.x == 0) tr_flag(status, bad_len ? TR_DEV_BAD_LENGTH : full ? TR_DEV_CACHE_FULL : TR_DEV_BAD_PAGE);
  return -1;
}

// The checks of all sequences and their new lengths; what append_kernel has to
// copy goes to todo[b] = (old length, rows).
__global__ void __launch_bounds__(kAppendThreads) append_plan_kernel(const KvDev c, int T, const int32_t *count,
                                                                     int2 *todo, unsigned *status) {
  tr_let_next_start();
  tr_wait_for_previous();
  const int b = blockIdx.x, Lb = c.L[b];
  const int n = append_rows(c, b, Lb, count ? count[b] : T, T, status);
  if (threadIdx.x == 0) {
    todo[b] = make_int2(Lb, max(n, 0));
    if (n > 0) c.L[b] = Lb + n;
  }
}

// One thread per 16-byte piece of a new row (8 elements), K and V together.
// todo: the plan kernel's; NULL when a sequence's rows are one CTA's work (a
// decoding step), which then checks and advances the length itself.
template <bool E4M3, int D>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const KvDev c, const uint4 *Kn, const uint4 *Vn, int T,
                                                                const int32_t *count, const int2 *todo,
                                                                unsigned *status) {
  constexpr int kPieces = D / 8, kOut = E4M3 ? 8 : 16;  // of a row; bytes of a piece in the cache
  const int b = blockIdx.y;
  tr_let_next_start();
  tr_wait_for_previous();
  int Lb, n;
  if (todo) {
    const int2 x = todo[b];
    Lb = x.x;
    n = x.y;
  } else {
    Lb = c.L[b];
    n = append_rows(c, b, Lb, count ? count[b] : T, T, status);  // its barrier lies between reads and write of L
    if (threadIdx.x == 0 && n > 0) c.L[b] = Lb + n;
  }
  if (n <= 0 || blockIdx.x * (kAppendThreads * kAppendUnroll) >= (unsigned)n * c.Hkv * kPieces) return;
  // the heads' scales and their reciprocals, once per CTA where they fit
  constexpr int kHeads = E4M3 ? 256 : 1;
  __shared__ Scale scales[2][kHeads];
  const bool shared_scales = c.Hkv <= kHeads;
  const unsigned total = (unsigned)n * c.Hkv * kPieces;
  const long long base = (long long)b * T * c.Hkv * kPieces;
  const unsigned i0 = blockIdx.x * (kAppendThreads * kAppendUnroll) + threadIdx.x;
  uint4 kx[kAppendUnroll], vx[kAppendUnroll];
  long long at[kAppendUnroll];
  int head[kAppendUnroll];
  // row th = token * Hkv + head; the next piece of this thread is kAppendThreads / kPieces rows on
  constexpr unsigned kNext = kAppendThreads / kPieces;
  const unsigned piece = threadIdx.x % kPieces, tok_next = kNext / (unsigned)c.Hkv, h_next = kNext % (unsigned)c.Hkv;
  unsigned th = i0 / kPieces, tok = th / (unsigned)c.Hkv, h = th - tok * c.Hkv;
#pragma unroll
  for (int u = 0; u < kAppendUnroll; ++u) {
    head[u] = h;
    if (i0 + u * kAppendThreads < total) {
      const unsigned i = i0 + u * kAppendThreads;
      kx[u] = __ldcs(Kn + base + i);
      vx[u] = __ldcs(Vn + base + i);
      const int p = Lb + (int)tok;
      at[u] = kv_block(c, b, p) + (long long)h * c.head_stride + kv_row(c, p) + piece * kOut;
      if (c.scores && piece == 0) c.scores[((long long)b * c.Hkv + h) * c.scores_ld + p] = 0.f;
    }
    tok += tok_next;
    h += h_next;
    if (h >= (unsigned)c.Hkv) {
      h -= c.Hkv;
      ++tok;
    }
  }
  if constexpr (E4M3) {
    if (shared_scales) {
      if ((int)threadIdx.x < c.Hkv) {
        scales[0][threadIdx.x] = make_scale(c.k_scale[threadIdx.x]);
        scales[1][threadIdx.x] = make_scale(c.v_scale[threadIdx.x]);
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int u = 0; u < kAppendUnroll; ++u) {
    if (i0 + u * kAppendThreads >= total) continue;
    if constexpr (E4M3) {
      const Scale ks = shared_scales ? scales[0][head[u]] : make_scale(c.k_scale[head[u]]);
      const Scale vs = shared_scales ? scales[1][head[u]] : make_scale(c.v_scale[head[u]]);
      *reinterpret_cast<uint2 *>(c.K + at[u]) = e4m3_of(kx[u], ks);
      *reinterpret_cast<uint2 *>(c.V + at[u]) = e4m3_of(vx[u], vs);
    } else {
      *reinterpret_cast<uint4 *>(c.K + at[u]) = kx[u];
      *reinterpret_cast<uint4 *>(c.V + at[u]) = vx[u];
    }
  }
}

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMost = 32;  // keys of a thread in registers, at most
constexpr int kMoveThreads = 512;

// Order of the scores: larger first, -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t score_key(float s) { return s != s ? 0u : tr_ord(s); }

template <int BITS>
struct SelSmem {
  __align__(16) unsigned hist[(32 + BITS - 1) / BITS][1 << BITS];
  unsigned wsum[kSelWarps];
  unsigned cnt[kSelMost * kSelWarps];  // (rows above the edge << 16) + rows at it, of 32 rows
  unsigned wgt[kSelWarps], weq[kSelWarps];
  unsigned bin, need;
  unsigned gt, eq;  // of the CTA
};

// Inclusive sum over the block's threads (two barriers).
__device__ __forceinline__ unsigned block_sum(unsigned v, unsigned *wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) wsum[warp] = v;
  __syncthreads();
  unsigned w = lane < kSelWarps ? wsum[lane] : 0u;
#pragma unroll
  for (int o = 1; o < kSelWarps; o <<= 1) {
    const unsigned x = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += x;
  }
  w = __shfl_sync(~0u, w, max(warp - 1, 0));
  __syncthreads();
  return v + (warp ? w : 0u);
}

// One cluster per (KV head, sequence): finds the key of the k-th largest score
// among the rows before the protected ones and writes the k positions that stay,
// ascending, to keep.  Each CTA holds one slice of the keys, KPT to a thread in
// registers (a slice that is longer is read again in every pass).  The key is
// found by a radix select, BITS a pass: the CTAs' histograms are added through
// distributed shared memory and every CTA walks the sum alike.  11 bits (three
// passes) suit one CTA, 8 bits (four) a cluster, whose exchange is an eighth
// (131072 rows, clusters of 8: 38 us with 11 bits, 20 us with 8).  A row's place
// in keep is the number of rows above the edge before it plus the number of edge
// rows taken before it.  split[pair], where asked for, gets the number of kept rows
// at positions below the budget.
// Four CTAs of the short form share an SM, for which it spills 36 to 44 bytes.
template <int KPT, int BITS>
__global__ void __launch_bounds__(kSelThreads, KPT <= 8 ? 4 : 2)
    evict_select_kernel(const KvDev c, int budget, int recent, int32_t *keep, int32_t *old_len, int32_t *split,
                        unsigned *status) {
  constexpr int kSelBins = 1 << BITS, kPasses = (32 + BITS - 1) / BITS;
  __shared__ SelSmem<BITS> s;
  tr_let_next_start();
  tr_wait_for_previous();
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int h = blockIdx.x / CS, b = blockIdx.y;
  const int Lb = c.L[b];
  const bool bad_len = Lb < 0 || Lb > c.cap;
  const bool active = !bad_len && Lb > budget;
  const int n = Lb - recent, k = budget - recent;  // k < n where active
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = active ? ((n + CS - 1) / CS + 31) & ~31 : 0;
  const int lo = active ? min(n, rank * slice) : 0, len = active ? min(n - lo, slice) : 0;
  const float *sc = c.scores + ((long long)b * c.Hkv + h) * c.scores_ld + lo;
  const bool held = slice <= KPT * kSelThreads;
  unsigned keys[KPT];  // rows threadIdx.x + j * kSelThreads, read while the pages are looked over
  if (held) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int i = threadIdx.x + j * kSelThreads;
      keys[j] = i < len ? __float_as_uint(sc[i]) : 0u;
    }
  }
  for (int i = threadIdx.x; i < kPasses * kSelBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
  const bool bad_page = active && kv_bad_pages(c, b, 0, Lb);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    old_len[b] = active && !bad_page ? Lb : -1;
    if (bad_len) tr_flag(status, TR_DEV_BAD_LENGTH);
    if (bad_page) tr_flag(status, TR_DEV_BAD_PAGE);
  }
  if (!active || bad_page || k == 0) return;  // the same for the whole cluster
  keep += ((long long)b * c.Hkv + h) * budget;
  if (held) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) keys[j] = score_key(__uint_as_float(keys[j]));
  }
  // `prefix` holds the leading bits of the key of the k-th largest, `need` how
  // many of the rows that share them are still to be taken
  unsigned prefix = 0, need = k;
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = max(32 - BITS * (pass + 1), 0), width = min(BITS, 32 - BITS * pass);
    const unsigned mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + width), low = (1u << width) - 1u;
    unsigned *hist = s.hist[pass];
    auto count = [&](unsigned key) {
      if ((key & mask) == prefix) atomicAdd(&hist[kSelBins - 1 - ((key >> shift) & low)], 1u);
    };
    if (held) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (threadIdx.x + j * kSelThreads < len) count(keys[j]);
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < len; i += kSelThreads) count(score_key(sc[i]));
    }
    // bins lie from the largest key down; a thread owns four of them
    constexpr int kOwners = kSelBins / 4;
    unsigned cnt[4] = {}, sum = 0;
    uint4 *own_bins = reinterpret_cast<uint4 *>(hist) + threadIdx.x;
    auto add = [&](const uint4 &x) {
      cnt[0] += x.x;
      cnt[1] += x.y;
      cnt[2] += x.z;
      cnt[3] += x.w;
    };
    if (CS == 1) __syncthreads();
    else cluster.sync();
    if (threadIdx.x < kOwners) {
      if (CS == 1) {
        add(*own_bins);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < CS) add(*cluster.map_shared_rank(own_bins, r));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += cnt[j];
    const unsigned incl = block_sum(sum, s.wsum);
    unsigned before = incl - sum;
    if (before < need && need <= incl) {
      int bin = kSelBins - 1 - 4 * threadIdx.x;
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (before + cnt[j] < need) {
          before += cnt[j];
          --bin;
        } else {
          break;
        }
      s.bin = bin;
      s.need = need - before;
    }
    __syncthreads();
    prefix |= s.bin << shift;
    need = s.need;
  }
  // rows above the edge and at it before each 32 rows of the slice
  unsigned gt = 0, eq = 0;  // of the CTA, then before its slice
  const unsigned below = (1u << lane) - 1;
  const int stretch = ((slice + kSelWarps - 1) / kSelWarps + 31) & ~31;  // of a warp, where the slice is not held
  const int w0 = min(len, warp * stretch), w1 = min(len, w0 + stretch);
  if (held) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const bool in = threadIdx.x + j * kSelThreads < len;
      const unsigned x = __popc(__ballot_sync(~0u, in && keys[j] > prefix)),
                     y = __popc(__ballot_sync(~0u, in && keys[j] == prefix));
      if (lane == 0) s.cnt[j * kSelWarps + warp] = (x << 16) + y;
    }
    __syncthreads();
    const unsigned v = threadIdx.x < KPT * kSelWarps ? s.cnt[threadIdx.x] : 0u;
    const unsigned incl = block_sum(v, s.wsum);
    if (threadIdx.x < KPT * kSelWarps) s.cnt[threadIdx.x] = incl - v;
    if (threadIdx.x == kSelThreads - 1) {
      s.gt = incl >> 16;
      s.eq = incl & 0xFFFFu;
    }
  } else {
#pragma unroll 2
    for (int i = w0; i < w1; i += 32) {
      const bool in = i + lane < w1;
      const unsigned key = in ? score_key(sc[i + lane]) : 0u;
      gt += __popc(__ballot_sync(~0u, in && key > prefix));
      eq += __popc(__ballot_sync(~0u, in && key == prefix));
    }
    if (lane == 0) {
      s.wgt[warp] = gt;
      s.weq[warp] = eq;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned x = 0, y = 0;
      for (int w = 0; w < kSelWarps; ++w) {
        x += s.wgt[w];
        y += s.weq[w];
      }
      s.gt = x;
      s.eq = y;
    }
  }
  gt = eq = 0;
  if (CS == 1) {
    __syncthreads();
  } else {
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      gt += *cluster.map_shared_rank(&s.gt, r);
      eq += *cluster.map_shared_rank(&s.eq, r);
    }
    cluster.sync();  // no CTA of the cluster is read from here on
  }
  auto place = [&](int i, bool in, unsigned key) {
    const bool above = in && key > prefix, edge = in && key == prefix;
    const unsigned gts = __ballot_sync(~0u, above), eqs = __ballot_sync(~0u, edge);
    const unsigned eq_before = eq + __popc(eqs & below);
    const unsigned at = gt + __popc(gts & below) + min(eq_before, need);
    if (above || (edge && eq_before < need)) keep[at] = lo + i;
    if (split && in && lo + i == budget) split[(long long)b * c.Hkv + h] = at;
    gt += __popc(gts);
    eq += __popc(eqs);
  };
  if (held) {
    const unsigned gt0 = gt, eq0 = eq;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const unsigned x = s.cnt[j * kSelWarps + warp];
      gt = gt0 + (x >> 16);
      eq = eq0 + (x & 0xFFFFu);
      const int i = threadIdx.x + j * kSelThreads;
      place(i, i < len, keys[j]);
    }
  } else {
    for (int w = 0; w < warp; ++w) {
      gt += s.wgt[w];
      eq += s.weq[w];
    }
    for (int i = w0; i < w1; i += 32) {
      const bool in = i + lane < w1;
      place(i + lane, in, in ? score_key(sc[i + lane]) : 0u);
    }
  }
}

// Where there are few pairs, the kept rows of one are cut at two places: rows
// [one, budget) come from positions at or behind the budget, rows [two, one) from
// positions at or behind one, so that within either stretch nothing is read
// where something is written, and each can be moved in any order once the
// stretches before it have been read.  two is the first eighth of one that will do.
struct Cuts {
  int two, one;
};
__device__ __forceinline__ Cuts cuts_of(int budget, int k, int Lb, const int32_t *keep, const int32_t *split) {
  Cuts u;
  u.one = k > 0 && budget < Lb - (budget - k) ? *split : max(0, 2 * budget - Lb);
  u.two = u.one;
  int at[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (int)((long long)u.one * i / 8);
    at[i] = r < k ? __ldcg(keep + r) : r + Lb - budget;
  }
#pragma unroll
  for (int i = 7; i >= 0; --i)
    if (at[i] >= u.one) u.two = (int)((long long)u.one * i / 8);
  return u;
}

// Moves one of the two stretches, scores included: 16 bytes of K and of V per
// thread and turn.
constexpr int kApartUnroll = 4;
template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) evict_apart_kernel(const KvDev c, int budget, int recent, bool second,
                                                                   const int32_t *keep, const int32_t *old_len,
                                                                   const int32_t *split) {
  constexpr int kLanes = ROW / 16, kRows = kMoveThreads / kLanes;
  const int h = blockIdx.y, b = blockIdx.z;
  tr_let_next_start();
  tr_wait_for_previous();
  const int Lb = old_len[b];
  if (Lb < 0) return;
  const int k = budget - recent, shift = Lb - budget;
  const long long pair = (long long)b * c.Hkv + h;
  keep += pair * budget;
  const Cuts cuts = cuts_of(budget, k, Lb, keep, split + pair);
  const int first = second ? cuts.two : cuts.one, last = second ? cuts.one : budget;
  const long long head = (long long)h * c.head_stride + (threadIdx.x % kLanes) * 16;
  float *sc = c.scores + pair * c.scores_ld;
  const bool scorer = threadIdx.x % kLanes == 0;
  for (int r0 = first + blockIdx.x * kRows * kApartUnroll; r0 < last; r0 += gridDim.x * kRows * kApartUnroll) {
    long long from[kApartUnroll];
    uint4 x[kApartUnroll], y[kApartUnroll];
    float z[kApartUnroll];
#pragma unroll
    for (int u = 0; u < kApartUnroll; ++u) {  // a row behind the last one is read twice, and not written
      const int r = min(r0 + u * kRows + (int)threadIdx.x / kLanes, last - 1);
      const int src = r < k ? __ldcg(keep + r) : r + shift;
      from[u] = head + kv_block(c, b, src) + kv_row(c, src);
      if (scorer) z[u] = sc[src];
    }
#pragma unroll
    for (int u = 0; u < kApartUnroll; ++u) {
      x[u] = __ldcs(reinterpret_cast<const uint4 *>(c.K + from[u]));
      y[u] = __ldcs(reinterpret_cast<const uint4 *>(c.V + from[u]));
    }
#pragma unroll
    for (int u = 0; u < kApartUnroll; ++u) {
      const int r = r0 + u * kRows + threadIdx.x / kLanes;
      if (r >= last) continue;
      const long long to = head + kv_block(c, b, r) + kv_row(c, r);
      *reinterpret_cast<uint4 *>(c.K + to) = x[u];
      *reinterpret_cast<uint4 *>(c.V + to) = y[u];
      if (scorer) sc[r] = z[u];
    }
  }
}

// Moves the kept rows of K and V up, in place, and their scores.  A CTA owns
// PART bytes of every row of one (sequence, KV head), of K or of V (or the
// scores), so no two CTAs touch the same bytes, and walks the kept rows in
// order.  Row r comes from keep[r] >= r.  Writing a batch of rows [r0, r1) can
// only hit sources of rows < r1: their reads lie before the barrier that the write
// waits for.  The next batch's sources lie at or behind r1, so it is read before the
// barrier too, which keeps loads in flight while the batch is written; its
// addresses come from keep and the page table, read one and two batches before that.
// With few pairs (split given) it ends where evict_apart_kernel takes over.  The
// first CTA of a sequence sets its new length.
template <int PART, int kMoveUnroll>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const KvDev c, int budget, int recent,
                                                                  const int32_t *keep, const int32_t *old_len,
                                                                  const int32_t *split) {
  constexpr int kLanes = PART / 16, kRows = kMoveThreads / kLanes, kBatch = kRows * kMoveUnroll;
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  tr_let_next_start();
  tr_wait_for_previous();
  const int Lb = old_len[b];
  if (Lb < 0) return;
  const int k = budget - recent, shift = Lb - budget;  // a protected row moves by `shift`
  keep += ((long long)b * c.Hkv + h) * budget;
  const int rows = split ? cuts_of(budget, k, Lb, keep, split + (long long)b * c.Hkv + h).two : budget;
  auto source = [&](int r) { return r >= budget ? r : r < k ? __ldcg(keep + r) : r + shift; };
  const int per = c.row_bytes / PART;
  if (part == 2 * per) {
    float *sc = c.scores + ((long long)b * c.Hkv + h) * c.scores_ld;
    constexpr int kPer = 8;
    for (int r0 = 0; r0 < rows; r0 += kMoveThreads * kPer) {
      float x[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = r0 + u * kMoveThreads + threadIdx.x;
        if (r < rows) x[u] = sc[source(r)];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = r0 + u * kMoveThreads + threadIdx.x;
        if (r < rows) sc[r] = x[u];
      }
    }
    if (h == 0 && threadIdx.x == 0) c.L[b] = budget;
    return;
  }
  char *base = (part < per ? c.K : c.V) + (long long)h * c.head_stride + (part % per) * PART +
               (threadIdx.x % kLanes) * 16;
  const int row = threadIdx.x / kLanes;
  uint4 x[2][kMoveUnroll];
  long long from[2][kMoveUnroll];  // byte offset of the source, -1: the row stays
  int src[kMoveUnroll];
  auto sources = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int r = r0 + u * kRows + row;
      src[u] = r < rows ? source(r) : r;
    }
  };
  auto offsets = [&](int r0, long long(&f)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      f[u] = src[u] == r0 + u * kRows + row ? -1 : kv_block(c, b, src[u]) + kv_row(c, src[u]);
  };
  auto load = [&](const long long(&f)[kMoveUnroll], uint4(&y)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (f[u] >= 0) y[u] = *reinterpret_cast<const uint4 *>(base + f[u]);
  };
  auto store = [&](int r0, const long long(&f)[kMoveUnroll], const uint4(&y)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int r = r0 + u * kRows + row;
      if (f[u] >= 0) *reinterpret_cast<uint4 *>(base + kv_block(c, b, r) + kv_row(c, r)) = y[u];
    }
  };
  // on entry of a turn: batch r0 loaded, offsets of r0 + kBatch and sources of r0 + 2 kBatch at hand
  sources(0);
  offsets(0, from[0]);
  load(from[0], x[0]);
  sources(kBatch);
  offsets(kBatch, from[1]);
  sources(2 * kBatch);
  auto turn = [&](int r0, long long(&f)[kMoveUnroll], uint4(&y)[kMoveUnroll], long long(&nf)[kMoveUnroll],
                  uint4(&ny)[kMoveUnroll]) {
    load(nf, ny);
    __syncthreads();
    store(r0, f, y);
    offsets(r0 + 2 * kBatch, f);
    sources(r0 + 3 * kBatch);
  };
  for (int r0 = 0; r0 < rows; r0 += 2 * kBatch) {
    turn(r0, from[0], x[0], from[1], x[1]);
    turn(r0 + kBatch, from[1], x[1], from[0], x[0]);
  }
}

// Workspace: the kept positions of every (sequence, KV head), then the old
// lengths, then each pair's first row to come from behind the budget.  A budget that no sequence can exceed keeps no positions.
size_t keep_bytes(const KvDev &c, int budget) {
  return budget < c.cap ? tr_align_up((size_t)c.B * c.Hkv * (size_t)budget * 4, 256) : 0;
}

size_t evict_bytes(const KvDev &c, int budget) {
  return keep_bytes(c, budget) + tr_align_up((size_t)c.B * 4, 256) + tr_align_up((size_t)c.B * c.Hkv * 4, 256);
}

}  // namespace

// ---------------------------------------------------------------------------
// ABI
// ---------------------------------------------------------------------------

extern "C" size_t tr_kv_append_workspace_bytes(const tr_kv_cache *cache) {
  return cache && cache->B > 0 ? tr_align_up((size_t)cache->B * sizeof(int2), 256) : 0;
}

extern "C" int tr_kv_append(const void *Kn, const void *Vn, int T, const int32_t *count, const tr_kv_cache *cache,
                            void *ws, size_t ws_bytes, tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  if (!Kn || !Vn || T < 1 || (((uintptr_t)Kn | (uintptr_t)Vn) & 15) || ((uintptr_t)count & 3)) return TR_E_INVAL;
  const bool e4m3 = cache->type == TR_KV_E4M3;
  const long long pieces = (long long)T * c.Hkv * (cache->d / 8);
  const long long per = kAppendThreads * kAppendUnroll;
  const long long grid = (pieces + per - 1) / per;
  if (pieces >= (1LL << 31)) return TR_E_UNSUPPORTED;
  if (grid > 1 && (!ws || ((uintptr_t)ws & 15) || ws_bytes < tr_kv_append_workspace_bytes(cache))) return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  const dim3 g((unsigned)grid, (unsigned)c.B);
  cudaStream_t s = (cudaStream_t)stream;
  int2 *todo = grid > 1 ? (int2 *)ws : nullptr;
  if (todo) {
    rc = tr_launch_next(append_plan_kernel, {dim3(c.B), kAppendThreads}, s, c, T, count, todo, tr_status_dev());
    if (rc != TR_OK) return rc;
  }
  auto run = [&](auto kernel) {
    return tr_launch_next(kernel, {g, kAppendThreads}, s, c, (const uint4 *)Kn, (const uint4 *)Vn, T, count,
                          (const int2 *)todo, tr_status_dev());
  };
  if (cache->d == 64) return e4m3 ? run(append_kernel<true, 64>) : run(append_kernel<false, 64>);
  return e4m3 ? run(append_kernel<true, 128>) : run(append_kernel<false, 128>);
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
  int32_t *keep = (int32_t *)ws, *old_len = (int32_t *)((char *)ws + keep_bytes(c, budget));
  cudaStream_t s = (cudaStream_t)stream;
  // CTAs per (sequence, KV head): more where there are few of these and their rows are many
  const long long pairs = (long long)c.B * c.Hkv;
  int cs = 1;
  while (cs < 8 && c.cap / (2 * cs) >= 4096 && pairs * 2 * cs <= 4 * tr_sm_count()) cs *= 2;
  // Whole rows, one CTA for K and one for V of each pair, or, with few pairs of
  // many rows, narrow columns for the rows that move within the budget and the others
  // apart.  Whole rows take 9 ns a row of 256 bytes and CTA until HBM is full, the
  // other way 1.3 of HBM's time and 15 us.  Measured (bf16, d = 128; whole / apart):
  // 8 pairs, 2048 rows kept 27 / 25 us, 16384 155 / 46 us, 32768 300 / 85 us;
  // 32 pairs, 2048 rows 32 / 43 us; 128 pairs, 2048 rows 59 / 70 us; 1 pair, 1024
  // rows 15 / 18 us.  The host knows no lengths: pairs within the budget count too, so
  // one sequence of 131072 rows among eight short ones goes as whole rows (8 heads cut
  // to 32768: 430 us, alone 76).  Shorter rows follow by their bytes; that rule was
  // measured with rows of 256 bytes only.
  const int row = c.row_bytes;
  const bool few = pairs < 45 && (double)budget * row * (45 - pairs) > 19e6;
  int32_t *split = few ? (int32_t *)((char *)old_len + tr_align_up((size_t)c.B * 4, 256)) : nullptr;
  // with a budget that the cache cannot exceed this still reports bad lengths
  const dim3 select(c.Hkv * cs, c.B);
  auto pick = [&](auto kernel) {
    return tr_launch_next(kernel, {select, kSelThreads, 0, cs}, s, c, budget, recent, keep, old_len, split,
                          tr_status_dev());
  };
  const bool small = c.cap <= (long long)cs * 8 * kSelThreads;
  rc = cs == 1 ? (small ? pick(evict_select_kernel<8, 11>) : pick(evict_select_kernel<kSelMost, 11>))
               : (small ? pick(evict_select_kernel<8, 8>) : pick(evict_select_kernel<kSelMost, 8>));
  if (rc != TR_OK || budget >= c.cap) return rc;
  int part = row;
  while (few && part > 32 && pairs * 2 * (row / part) < 2LL * tr_sm_count()) part /= 2;
  const dim3 move(2 * (row / part) + 1, c.Hkv, c.B);
  auto go = [&](auto kernel) {
    return tr_launch_next(kernel, {move, kMoveThreads}, s, c, budget, recent, keep, old_len, split);
  };
  rc = part == 256   ? go(evict_move_kernel<256, 4>)
       : part == 128 ? go(evict_move_kernel<128, 4>)
       : part == 64  ? go(evict_move_kernel<64, 4>)
                     : go(evict_move_kernel<32, 8>);  // few CTAs: more in flight for each
  if (!few) return rc;
  const long long rows = kMoveThreads / (row / 16) * kApartUnroll;  // of one turn of a CTA
  const long long turns = (budget + rows - 1) / rows, fill = (4LL * tr_sm_count() + pairs - 1) / pairs;
  const dim3 apart((unsigned)(turns < fill ? turns : fill), c.Hkv, c.B);
  for (int level = 2; level >= 1 && rc == TR_OK; --level) {
    auto rest = [&](auto kernel) {
      return tr_launch_next(kernel, {apart, kMoveThreads}, s, c, budget, recent, level == 2, keep, old_len, split);
    };
    rc = row == 256   ? rest(evict_apart_kernel<256>)
         : row == 128 ? rest(evict_apart_kernel<128>)
                      : rest(evict_apart_kernel<64>);
  }
  return rc;
}
