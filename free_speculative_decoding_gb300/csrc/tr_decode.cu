// Attention of one new token per sequence over a KV cache.
//
// For query head hq with KV head g, O = sum_p w_p V[g, p] with w the softmax of
// scale * Q[hq] . K[g, p] over the cached rows p < L[b].  Every cached row is
// needed once and used for the few query heads of its group, so the cache's
// bytes bound the work: 4 G d flops for 4 d bytes of a 16-bit row, G flops a byte.
// The 5th-generation tensor cores' 128-row tile would be empty but for G rows, so
// the products run on the warp-level matrix instructions, which keep up with
// HBM here (tensor pipe 28% active while DRAM delivers 6.5 TB/s).
//
// Split.  A pair is (sequence, KV head) with ceil(L / kTile) tiles.  All pairs'
// tiles are laid end to end and cut into equal ranges, one per WARP of a
// one-CTA-per-SM grid.  A warp streams its own tiles through its own ring in
// shared memory (cp.async) and meets no barrier on the way, whatever the mix of
// lengths.  With little work only as many warps of each CTA take part as leave
// each about kMinRows rows, so that it spreads over every SM.  A pair that lies
// inside one range is finished by its warp.  When a CTA's whole range lies in
// one pair its warps' sums are joined in shared memory first.  What remains are
// (m, l, O) partials, which join_kernel joins in a fixed order.  Where all pairs
// of a small cache fit on the SMs at once each is the work of a cluster of one
// to eight CTAs that join their parts through distributed shared memory, and
// nothing is left for a second kernel.
//
// Tile.  S = Q K^T with m16n8k16 instructions: the group's query heads are the 16
// rows (8 of them empty when the group has at most 8 heads), cached rows are
// the columns.  The contraction runs over d in an order of its own: a lane's
// 16-byte piece of a row of K is used as the B fragments of two (8-bit: four)
// instructions, and Q is loaded in the same order, so that K needs no
// transposing load.  The accumulators of S are laid out as the A fragments of
// P V.  V's B fragments pair two rows: transposing loads bring 16-bit ones; of
// 8-bit rows a lane reads the same 16-byte piece of four rows, interleaves them
// with byte permutes and widens the pairs.
//
// Precision.  The output is fp32, so P must not be rounded to the cache's type:
// p is split exactly into three bf16 parts (8 + 8 + 8 bits), or into two fp16 parts
// (22 bits; p is scaled up to between 2^7 and 2^15 at the largest, so that what
// fp16 cannot hold is below 2^-32 of the weights' sum), and each part is
// multiplied with V.  With at most 8 heads the empty half of the
// instruction's rows carries the second part at no extra cost.  The matrix
// unit's own adds cut off what does not fit, always towards zero, so its sums
// last 16 rows only and are added to O with rounded adds (kept in the unit over a
// whole range, the loss grew with the range: 7e-6 of the result's norm at 3400
// rows a warp against 1e-6 for fp32 products and sums; now 5e-7).
// An 8-bit row is widened to fp16 (exact); Q is scaled by a power of two per
// head so that narrowing bf16 to fp16 is exact for all elements down to 2^-31 of
// the head's largest.
//
// Measured (one GB300, whole calls in a graph, fractions of the 6675 GB/s of a
// copy): 4 x 32768 rows of 32 heads, bf16, 308 us = 105%; 16 x 1k-4k rows of 32
// heads in pages of 64, 112 us = 96%; 64 sequences of 1-8191 rows, 8 heads of
// groups of 4, 8-bit, weights gathered, 116 us = 74% (98 us without weights;
// bound by instructions: each 8-bit pair is widened); 8 x 4096 rows of 8 heads,
// weights gathered, 33 us = 61%, 24 x 17-2011 rows, d = 64, 13 us = 36%, and one
// sequence of 512 rows of 32 heads, 5.4 us (6.5 where L2 does not hold its rows), are
// bound by latency: 2 us of launch,
// 1 to 2 us until the first rows are there, then 0.7 us for a tile of a warp by itself
// and about 1 us beside the SM's others (350 to 400 instructions in chains), 2 to 3 us
// for each kernel behind this one.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include <cooperative_groups.h>

#include "tr_kv.cuh"
#include "tr_sm100.cuh"

namespace {

namespace cg = cooperative_groups;
using sm100::ex2;
using sm100::smem_u32;

constexpr int kMaxB = 1024;
constexpr int kMaxOwn = 8;               // CTAs of a cluster that share a pair
constexpr int kRings = 192 * 1024;       // bytes of a CTA's rings
constexpr int kMinRows = 32;            // cached rows of a warp's range, about, at least
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;            // the running maximum follows once it is 2^8 behind

struct DecodeArgs {
  const void *Q;
  float *O, *lse;
  float *part_o;     // [row tiles][warps][2][MT][d]
  float2 *part_ml;   // [row tiles][warps][2][MT] (reference maximum, sum), log2 units
  float *lse2;       // [B, Hq] log2 of the softmax denominators
  float *s;          // [B, Hq, s_ld] logits, log2 units (accumulate)
  int *plan;         // tiles per warp, warps per CTA, then for each sequence the tiles of one head before it
  long long s_ld;
  int Hq, G, accumulate;
  int own;           // CTAs (a cluster) that share one pair and row tile; 0: ranges over all pairs
  float scale_log2;
  float scale_man;   // scale_log2 = scale_man * 2^scale_exp, scale_man in [1, 2)
  int scale_exp;
  unsigned *status;
};

template <int TYPE, int D, int NW>
struct Shape {
  static constexpr bool F8 = TYPE == TR_KV_E4M3;
  static constexpr bool BF = TYPE == TR_KV_BF16;
  static constexpr int ROW = D * (F8 ? 1 : 2);          // bytes
  static constexpr int CPR = ROW / 16;                  // 16-byte pieces of a row
  // cached rows per tile: 16 (one contraction step of P V), or 32 of the shorter rows, so
  // that a tile's chain of dependent steps is paid once per 4 KB or more
  static constexpr int KB = ROW == 256 ? 1 : 2;
  static constexpr int kTile = 16 * KB;
  static constexpr int STAGE = 2 * kTile * ROW;         // K tile, V tile
  static constexpr int WARPS = NW;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int RING = kRings / WARPS;           // bytes of a warp's ring
  static constexpr int STAGES = RING / STAGE;
  static constexpr int NT = D / 8;                      // column blocks of O
  static constexpr int QR = D / 8;                      // registers of one query row's fragments
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, bool bf) {
  if (bf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// a + b, two fp32 values in one instruction.
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
  asm("{ .reg .b64 p, q; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %3}; add.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// 16 bytes from global to shared memory; of the second form 16 zero bytes where not valid.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 bytes from global memory where valid, else zero; not moved behind the copies that follow.
__device__ __forceinline__ uint4 ldg16(const uint4 *p, bool valid) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (valid)
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// Four 8 x 8 blocks of 16-bit values, transposed; lane l gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void ldsm_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Two e4m3 values widened to fp16 (exact): those in the low, or high, half of w.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A place in the global order of tiles: tile kt of (b, h), whose nt tiles hold L rows.
struct Cursor {
  int b, h, kt, nt, L;
};

template <typename Prefix>
__device__ __forceinline__ void seek(Cursor &u, const Prefix &tp, const int *Ls, int B, int Hkv, int t) {
  // the last sequence whose first tile is at or before t (skips empty ones)
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)tp[mid] * Hkv <= t) lo = mid;
    else hi = mid - 1;
  }
  u.b = lo;
  u.nt = tp[lo + 1] - tp[lo];
  const int r = t - tp[lo] * Hkv;
  u.h = r / u.nt;
  u.kt = r - u.h * u.nt;
  u.L = Ls[lo];
}

template <int kTile>
__device__ __forceinline__ void step(Cursor &u, const int *Ls, int B, int Hkv) {
  if (++u.kt < u.nt) return;
  u.kt = 0;
  if (++u.h < Hkv) return;
  u.h = 0;
  while (++u.b < B && Ls[u.b] == 0) {
  }
  if (u.b < B) {
    u.L = Ls[u.b];
    u.nt = (u.L + kTile - 1) / kTile;
  }
}

// Swizzles of the 16-byte pieces of row r, so that the fragment reads below
// meet no bank conflict (8-bit rows of 64 bytes: two-way ones on V).
template <int CPR>
__device__ __forceinline__ int swz_k(int r, int ch) {
  return CPR >= 8 ? ch ^ ((r & 1) << 2) : ch;
}
template <int CPR, bool F8>
__device__ __forceinline__ int swz_v(int r, int ch) {
  return !F8 ? ch ^ (r & 7) : CPR >= 8 ? ch ^ (((r >> 1) & 3) << 1) : ch ^ ((r >> 1) & 3);
}

// What a product of the scaled query (2^up) and an 8-bit row is multiplied with:
// scale * ks * 2^-up in log2 units.  The softmax below takes the largest product
// for the largest logit and masks rows with a product of -inf, so the factor must
// be a positive number.  2^-126 stands for everything below it, a scale of 0
// included: products are below 2^31, so all such weights are equal as they should be.
// Mantissas and exponents apart: no intermediate leaves the range that the factor is in.
__device__ __forceinline__ float logit_factor(const DecodeArgs &a, float ks, int up) {
  if (!(ks < INFINITY)) return ks * 0.f;  // NaN: so is every logit
  const int e = ks > 0.f ? ilogbf(ks) : 0;
  const float f = scalbnf(a.scale_man * scalbnf(ks, -e), a.scale_exp + e - up);
  return fminf(fmaxf(f, 0x1p-126f), FLT_MAX);
}

// 8-bit V: columns of a lane's piece of a row, and its pieces per row.
__host__ __device__ constexpr int piece_cols(int D) { return D == 128 ? 16 : 8; }
__host__ __device__ constexpr int pieces(int D) { return D / (8 * piece_cols(D)); }

// The warps that a range of pairs is cut for, from the tiles' number alone.
struct Cut {
  int warps, per;  // per CTA, tiles per warp
};
__device__ __forceinline__ Cut cut_of(int T, int ctas, int kTile, int most) {
  const int min_tiles = max(kMinRows / kTile, 1);
  Cut c;
  c.warps = min(max((T + ctas * min_tiles - 1) / (ctas * min_tiles), 1), most);
  c.per = max((T + ctas * c.warps - 1) / (ctas * c.warps), 1);
  return c;
}

// Registers of a thread: 168 with 12 warps, up to 246 with 8; with 16 query rows 255,
// and at d = 128 12 (bf16) or 20 (8-bit) bytes spilled.
template <int TYPE, int D, int MT, int NW>
__global__ void __launch_bounds__(NW * 32, 1) split_kernel(const KvDev c, const DecodeArgs a) {
  using S = Shape<TYPE, D, NW>;
  constexpr int kTile = S::kTile, KB = S::KB, kWarps = S::WARPS, kThreads = S::THREADS;
  constexpr int kOwn = (kMaxB + kThreads - 1) / kThreads;  // sequences of a thread, in the prefix sum
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int Ls[kMaxB], tp[kMaxB + 1], wsum[kWarps];
  __shared__ float2 jml[kWarps][MT], cml[MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  tr_let_next_start();
  tr_wait_for_previous();

  // the CTA's range of tiles, [c0, c1) in the order of all pairs' tiles, and its first pair
  long long c0;
  int c1;
  Cursor cur, ld;
  Cut cut;
  if (a.own) {
    // of one pair alone: counted from the pair's first tile
    const int pair_id = blockIdx.x / a.own, part = blockIdx.x % a.own;
    cur.b = pair_id / c.Hkv;
    cur.h = pair_id - cur.b * c.Hkv;
    cur.L = c.L[cur.b];
    const bool bad = cur.L < 0 || cur.L > c.cap;
    if (bad && part == 0 && cur.h == 0 && blockIdx.y == 0 && threadIdx.x == 0) tr_flag(a.status, TR_DEV_BAD_LENGTH);
    if (bad || cur.L == 0) {  // the whole cluster
      const int m0 = blockIdx.y * MT;
      const long long hq = (long long)cur.b * a.Hq + (long long)cur.h * a.G + m0;
      if (part == 0)
        for (int i = threadIdx.x; i < min(MT, a.G - m0) * D; i += kThreads) {
          a.O[hq * D + i] = 0.f;
          if (a.lse && i < min(MT, a.G - m0)) a.lse[hq + i] = -INFINITY;
        }
      return;
    }
    cur.nt = (cur.L + kTile - 1) / kTile;
    cut.warps = kWarps;
    cut.per = (cur.nt + a.own * kWarps - 1) / (a.own * kWarps);
    cur.kt = min(cur.nt, part * kWarps * cut.per);
    c0 = cur.kt;
    c1 = cur.kt + min(cur.nt - cur.kt, kWarps * cut.per);
  } else {
    // lengths and, for one head, the tiles before each sequence
    int mine[kOwn], sum = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int b = threadIdx.x * kOwn + i;
      int L = b < c.B ? c.L[b] : 0;
      if (L < 0 || L > c.cap) {
        if (blockIdx.x == 0 && blockIdx.y == 0) tr_flag(a.status, TR_DEV_BAD_LENGTH);
        L = 0;
      }
      if (b < kMaxB) Ls[b] = L;
      mine[i] = sum;
      sum += (L + kTile - 1) / kTile;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += wsum[w];
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (threadIdx.x * kOwn + i <= kMaxB) tp[threadIdx.x * kOwn + i] = before + mine[i];
    if (threadIdx.x == kThreads - 1 && kThreads * kOwn == kMaxB) tp[kMaxB] = before + sum;
    __syncthreads();
    const int T = tp[c.B] * c.Hkv;
    cut = cut_of(T, gridDim.x, kTile, kWarps);
    if (blockIdx.x == 0 && blockIdx.y == 0)
      for (int i = threadIdx.x; i <= c.B + 2; i += kThreads)
        a.plan[i] = i == 0 ? cut.per : i == 1 ? cut.warps : tp[i - 2];
    // sequences without rows belong to no warp's range
    if (blockIdx.y == 0)
      for (int b = blockIdx.x; b < c.B; b += gridDim.x)
        if (Ls[b] == 0)
          for (unsigned i = threadIdx.x; i < (unsigned)a.Hq * D; i += kThreads) {  // up to 2^31 - 128
            a.O[(long long)b * a.Hq * D + i] = 0.f;
            if (a.lse && i < (unsigned)a.Hq) a.lse[(long long)b * a.Hq + i] = -INFINITY;
          }
    c0 = (long long)blockIdx.x * cut.warps * cut.per;
    if (c0 >= T) return;
    c1 = (int)min((long long)T, c0 + (long long)cut.warps * cut.per);
    seek(cur, tp, Ls, c.B, c.Hkv, (int)c0);
  }
  const int w = blockIdx.x * cut.warps + warp;
  const int t0 = warp < cut.warps ? (int)min((long long)c1, c0 + (long long)warp * cut.per) : c1;
  const int t1 = warp < cut.warps ? min(c1, t0 + cut.per) : c1;
  const uint32_t ring = smem_u32(smem) + warp * S::RING;
  const int row0 = blockIdx.y * MT;  // first query head of this row tile inside its group

  // joined: the CTA's whole range lies in its first pair
  const bool joined = a.own || (cut.warps > 1 && c1 - (int)c0 <= cur.nt - cur.kt);
  const Cursor pair = cur;
  if (t0 >= t1 && !joined) return;
  if (t0 < t1) {
    if (joined) cur.kt += t0 - (int)c0;
    else seek(cur, tp, Ls, c.B, c.Hkv, t0);
  }
  ld = cur;
  int t_ld = t0;

  // Queries of a pair, raw: requested before the rows, which would keep them waiting.
  constexpr int R = MT / 8;                           // query rows of a lane: g, g + 8
  uint32_t q[R][S::QR];
  auto fetch_q = [&](const Cursor &u) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int m_row = row0 + g + r * 8;
      const uint4 *src = reinterpret_cast<const uint4 *>(a.Q) +
                         ((long long)u.b * a.Hq + (long long)u.h * a.G + m_row) * (D / 8);
#pragma unroll
      for (int s = 0; s < S::QR / 4; ++s) {
        // 16-bit rows: a lane's pieces are 8 elements apart by four; 8-bit ones: 16
        const uint4 x = ldg16(src + (S::F8 ? (4 * (s / 2) + t) * 2 + s % 2 : 4 * s + t), m_row < a.G);
        q[r][s * 4] = x.x;
        q[r][s * 4 + 1] = x.y;
        q[r][s * 4 + 2] = x.z;
        q[r][s * 4 + 3] = x.w;
      }
    }
  };
  if (t0 < t1) fetch_q(cur);

  // The loader.  `run` whole tiles lie right behind the last one in the same page (or
  // dense sequence): they take two pointer steps each.  Any other tile is looked up
  // by its rows' pages; lane l holds that of row l, read ahead of its use.
  const int blocks = c.page_table ? c.num_pages : c.B;
  const bool whole_tile = !c.page_table || (1 << c.page_log2) >= kTile;  // a tile lies in one page
  constexpr int kCopies = KB * S::CPR / 2, kStep = 32 / S::CPR;  // per lane and tensor; rows apart
  const int ch = lane % S::CPR, r0 = lane / S::CPR;
  const char *kp = nullptr, *vp = nullptr;
  int run = 0, page = 0;
  auto page_of = [&](Cursor u, int ahead) {
    u.kt += ahead;
    if (u.kt >= u.nt) {  // behind the pair's last tile: the next one's first
      u.kt = u.nt - 1;
      step<kTile>(u, Ls, c.B, c.Hkv);
    }
    const int p = u.kt * kTile + lane;
    page = !c.page_table ? u.b
           : lane < kTile && p < u.L ? c.page_table[(long long)u.b * c.max_pages + (p >> c.page_log2)]
                                     : 0;
  };
  if (t0 < t1) page_of(ld, 0);
  auto issue = [&](int stage) {
    if (t_ld < t1) {
      const uint32_t dk = ring + stage * S::STAGE, dv = dk + kTile * S::ROW;
      bool whole = run > 0;
      if (!whole) {
        const int p0 = ld.kt * kTile, left = ld.L - p0;
        const long long head = (long long)ld.h * c.head_stride + ch * 16;
        const bool bad = lane < min(kTile, left) && (unsigned)page >= (unsigned)blocks;
        if (whole_tile && left >= kTile && !__any_sync(~0u, bad)) {
          const long long at = (long long)__shfl_sync(~0u, page, 0) * c.block_stride + head + kv_row(c, p0 + r0);
          kp = c.K + at;
          vp = c.V + at;
          whole = true;
          // whole tiles of the pair and tiles of the page behind this one
          run = left / kTile - 1;
          if (c.page_table) {
            const int per_page = (1 << c.page_log2) / kTile;
            run = min(run, per_page - 1 - (ld.kt & (per_page - 1)));
          }
          run = min(run, t1 - 1 - t_ld) + 1;
        } else {  // small pages, a pair's last tile, or a page that is not there: row by row
          if (bad) tr_flag(a.status, TR_DEV_BAD_PAGE);
          if (left >= kTile && !__any_sync(~0u, bad)) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
              const int r = r0 + i * kStep;
              const long long at = (long long)__shfl_sync(~0u, page, r) * c.block_stride + head + kv_row(c, p0 + r);
              copy16(dk + r * S::ROW + swz_k<S::CPR>(r, ch) * 16, c.K + at);
              copy16(dv + r * S::ROW + swz_v<S::CPR, S::F8>(r, ch) * 16, c.V + at);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
              const int r = r0 + i * kStep, pg = __shfl_sync(~0u, page, r);
              const bool valid = r < left && (unsigned)pg < (unsigned)blocks;
              const long long at = valid ? (long long)pg * c.block_stride + head + kv_row(c, p0 + r) : 0;
              copy16(dk + r * S::ROW + swz_k<S::CPR>(r, ch) * 16, c.K + at, valid);
              copy16(dv + r * S::ROW + swz_v<S::CPR, S::F8>(r, ch) * 16, c.V + at, valid);
            }
          }
          run = 1;
        }
        if (t_ld + run < t1) page_of(ld, run);
      }
      if (whole) {
        auto copy = [&](long long next) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int r = r0 + i * kStep;
            copy16(dk + r * S::ROW + swz_k<S::CPR>(r, ch) * 16, kp + i * next);
            copy16(dv + r * S::ROW + swz_v<S::CPR, S::F8>(r, ch) * 16, vp + i * next);
          }
        };
        if (c.row_stride == S::ROW) copy(kStep * S::ROW);  // the offsets are part of the instructions
        else copy(kStep * c.row_stride);
        kp += kTile * c.row_stride;
        vp += kTile * c.row_stride;
      }
      --run;
      ++t_ld;
      if (t_ld < t1) step<kTile>(ld, Ls, c.B, c.Hkv);
    }
    copy_commit();
  };
  for (int i = 0; i < S::STAGES - 1; ++i) issue(i);

  constexpr float kOff = S::BF ? 0.f : 7.f;           // fp16 weights run up to 2^15
  float mul[R], m[R], l[R], o[S::NT][2 * R];
  float *logits[R];  // where a lane's logits of the next tile go
  int kt0 = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    logits[r] = nullptr;
  }

  // a lane's columns of query row g + 8 r, times f
  auto store_row = [&](float *dst, int r, float f) {
    if constexpr (!S::F8) {
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
        *reinterpret_cast<float2 *>(dst + n * 8 + 2 * t) = make_float2(o[n][2 * r] * f, o[n][2 * r + 1] * f);
    } else {
#pragma unroll
      for (int v = 0; v < pieces(D); ++v)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < piece_cols(D); e += 4) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = o[v * piece_cols(D) + e + k][2 * r + n] * f;
            *reinterpret_cast<float4 *>(dst + (2 * t + n + 8 * v) * piece_cols(D) + e) = make_float4(y[0], y[1], y[2], y[3]);
          }
    }
  };

  for (int i = t0; i < t1; ++i) {
    const int stage = (i - t0) % S::STAGES;
    if (i == t0 || cur.kt == 0) {
      // a new pair: its queries, empty sums
      kt0 = cur.kt;
      if (i > t0) fetch_q(cur);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mul[r] = a.scale_log2;
        logits[r] = a.s + ((long long)cur.b * a.Hq + (long long)cur.h * a.G + row0 + g + r * 8) * a.s_ld +
                    cur.kt * kTile + 2 * t;
        if constexpr (S::F8) {
          // narrowed to fp16 after scaling the head's largest to 2^14
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < S::QR; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(q[r][e] << 16)), fabsf(__uint_as_float(q[r][e] & 0xFFFF0000u))));
          amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
          const int up = amax > 0.f ? max(14 - ilogbf(amax), -114) : 0;  // -114: infinite
          const float ks = c.k_scale[cur.h];
          const uint32_t flip = ks < 0.f ? 0x80008000u : 0u;  // the scale's sign goes to the query
          // 2^up, up to 2^147, in two factors; neither product rounds what fp16 can hold
          const float f0 = __int_as_float((127 + (up >> 1)) << 23), f1 = __int_as_float((127 + up - (up >> 1)) << 23);
#pragma unroll
          for (int e = 0; e < S::QR; ++e)
            q[r][e] = pack_half2(__uint_as_float(q[r][e] << 16) * f0 * f1,
                                 __uint_as_float(q[r][e] & 0xFFFF0000u) * f0 * f1) ^ flip;
          mul[r] = logit_factor(a, fabsf(ks), up);
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
#pragma unroll
        for (int e = 0; e < 2 * R; ++e) o[n][e] = 0.f;
    }

    copy_wait<S::STAGES - 2>();
    __syncwarp();
    const uint32_t sk = ring + stage * S::STAGE, sv = sk + kTile * S::ROW;

    // S = Q K^T: column n of block j is row j * 8 + n of the tile.  With two blocks only the
    // contraction runs in two halves, so that four chains of instructions are under way
    constexpr int kHalves = KB == 1 ? 2 : 1, kPieces = S::CPR / 4;
    float s2[kHalves][2 * KB][4] = {};
#pragma unroll
    for (int e = 0; e < kPieces / kHalves; ++e)
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j) {
          const int r = j * 8 + g, pc = hf * (kPieces / kHalves) + e;
          const uint4 x = lds16(sk + r * S::ROW + swz_k<S::CPR>(r, pc * 4 + t) * 16);
          auto &acc = s2[hf][j];
          if constexpr (S::F8) {
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int at = pc * 8 + f * 2;
              mma(acc, q[0][at], R > 1 ? q[R - 1][at] : 0u, q[0][at + 1], R > 1 ? q[R - 1][at + 1] : 0u,
                  widen_lo(y[f]), widen_hi(y[f]), false);
            }
          } else {
            const int at = pc * 4;
            mma(acc, q[0][at], R > 1 ? q[R - 1][at] : 0u, q[0][at + 1], R > 1 ? q[R - 1][at + 1] : 0u, x.x, x.y, S::BF);
            mma(acc, q[0][at + 2], R > 1 ? q[R - 1][at + 2] : 0u, q[0][at + 3], R > 1 ? q[R - 1][at + 3] : 0u, x.z, x.w,
                S::BF);
          }
        }
    // the stage read in the previous turn; its addresses are worked out while the products are under way
    issue((i - t0 + S::STAGES - 1) % S::STAGES);
    float s[2 * KB][4];
#pragma unroll
    for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = kHalves == 2 ? s2[0][j][e] + s2[kHalves - 1][j][e] : s2[0][j][e];

    // softmax weights, relative to a maximum that follows lazily; rows behind the last get none
    const int rows = cur.L - cur.kt * kTile;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (rows < kTile) {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (j * 8 + 2 * t + e >= rows) s[j][2 * r + e] = -INFINITY;
      }
      float mx = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
      for (int j = 1; j < 2 * KB; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
      if (a.accumulate) {
        if (row0 + g + r * 8 < a.G)
#pragma unroll
          for (int j = 0; j < 2 * KB; ++j)
            *reinterpret_cast<float2 *>(logits[r] + j * 8) = make_float2(s[j][2 * r] * mul[r], s[j][2 * r + 1] * mul[r]);
        logits[r] += kTile;
      }
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2)) * mul[r];
      const bool grow = mx > m[r] + (kOff + kLazy);
      if (__any_sync(~0u, grow)) {
        const float mn = grow ? mx - kOff : m[r];
        const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int n = 0; n < S::NT; ++n) {
          o[n][2 * r] *= f;
          o[n][2 * r + 1] *= f;
        }
      }
      const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[j][2 * r + e] = ex2(fmaf(s[j][2 * r + e], mul[r], -base));
          l[r] += s[j][2 * r + e];
        }
    }

    // P in parts: pt[kb][part][r][j] holds rows 2t, 2t + 1 of half j of 16 rows for query row g + 8 r
    constexpr int kParts = S::BF ? 3 : 2;
    uint32_t pt[KB][kParts][R][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = s[2 * kb + j][2 * r], y = s[2 * kb + j][2 * r + 1];
          if constexpr (S::BF) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              pt[kb][k][r][j] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
              if (k < 2) {
                x -= __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
                y -= __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
              }
            }
          } else {
            pt[kb][0][r][j] = pack_half2(x, y);
            const __half2 h = *reinterpret_cast<const __half2 *>(&pt[kb][0][r][j]);
            pt[kb][1][r][j] = pack_half2(x - __low2float(h), y - __high2float(h));
          }
        }
    // O += P V of 16 rows and one column block
    auto pv = [&](float(&to)[2 * R], int kb, uint32_t b0, uint32_t b1) {
      const uint32_t(&p)[kParts][R][2] = pt[kb];
      float acc[4] = {};
      if constexpr (R == 1) {
        mma(acc, p[0][0][0], p[1][0][0], p[0][0][1], p[1][0][1], b0, b1, S::BF);
        if constexpr (S::BF) mma(acc, p[kParts - 1][0][0], 0u, p[kParts - 1][0][1], 0u, b0, b1, true);
        add2(acc[0], acc[1], acc[2], acc[3]);
        add2(to[0], to[1], acc[0], acc[1]);
      } else {
#pragma unroll
        for (int k = 0; k < kParts; ++k) mma(acc, p[k][0][0], p[k][R - 1][0], p[k][0][1], p[k][R - 1][1], b0, b1, S::BF);
        add2(to[0], to[1], acc[0], acc[1]);
        add2(to[2 * R - 2], to[2 * R - 1], acc[2], acc[3]);
      }
    };
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if constexpr (!S::F8) {
        // column block n holds columns 8 n ..: transposing loads bring two blocks' fragments
        const int r = kb * 16 + (lane & 15);
#pragma unroll
        for (int n = 0; n < S::NT; n += 2) {
          uint32_t x[4];
          ldsm_trans(x, sv + r * S::ROW + swz_v<S::CPR, false>(r, n + (lane >> 4)) * 16);
          pv(o[n], kb, x[0], x[1]);
          pv(o[n + 1], kb, x[2], x[3]);
        }
      } else {
        // a lane reads the same piece of four rows and interleaves them: block n = VW * v + e
        // holds columns (lane / 4 + 8 v) * VW + e
#pragma unroll
        for (int v = 0; v < pieces(D); ++v) {
          constexpr int kWords = piece_cols(D) / 4;  // of a piece
          uint32_t x[4][kWords];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = kb * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
            if constexpr (kWords == 4) {
              const uint4 y = lds16(sv + r * S::ROW + swz_v<S::CPR, true>(r, g + 8 * v) * 16);
              x[k][0] = y.x;
              x[k][1] = y.y;
              x[k][2] = y.z;
              x[k][3] = y.w;
            } else {
              const uint2 y = lds8(sv + r * S::ROW + swz_v<S::CPR, true>(r, g >> 1) * 16 + (g & 1) * 8);
              x[k][0] = y.x;
              x[k][1] = y.y;
            }
          }
#pragma unroll
          for (int e = 0; e < kWords; ++e)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint32_t sel = f ? 0x7362 : 0x5140;
              const uint32_t lo = __byte_perm(x[0][e], x[1][e], sel), hi = __byte_perm(x[2][e], x[3][e], sel);
              pv(o[v * piece_cols(D) + e * 4 + f * 2], kb, widen_lo(lo), widen_lo(hi));
              pv(o[v * piece_cols(D) + e * 4 + f * 2 + 1], kb, widen_hi(lo), widen_hi(hi));
            }
        }
      }
    }

    if (!joined && (cur.kt == cur.nt - 1 || i == t1 - 1)) {
      // the range leaves this pair: the result, or a partial
      const bool whole = kt0 == 0 && cur.kt == cur.nt - 1;
      const long long slot = ((long long)blockIdx.y * gridDim.x * kWarps + w) * 2 + (kt0 > 0 ? 0 : 1);
      const float vs = S::F8 ? c.v_scale[cur.h] : 1.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        l[r] += __shfl_xor_sync(~0u, l[r], 1);
        l[r] += __shfl_xor_sync(~0u, l[r], 2);
        const int row = g + r * 8;
        if (row0 + row >= a.G) continue;
        const long long hq = (long long)cur.b * a.Hq + (long long)cur.h * a.G + row0 + row;
        const float f = whole ? vs / l[r] : 1.f;
        float *dst = whole ? a.O + hq * D : a.part_o + (slot * MT + row) * D;
        if (t == 0) {
          if (whole) {
            const float x = m[r] + log2f(l[r]);
            if (a.lse) a.lse[hq] = x * kLn2;
            a.lse2[hq] = x;
          } else {
            a.part_ml[slot * MT + row] = make_float2(m[r], l[r]);
          }
        }
        store_row(dst, r, f);
      }
    }
    if (i + 1 < t1) step<kTile>(cur, Ls, c.B, c.Hkv);
  }
  if (!joined) return;

  // the CTA's warps hold parts of one pair: join them through their rings
  float *const rings = reinterpret_cast<float *>(smem);
  copy_wait<0>();
  __syncwarp();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    l[r] += __shfl_xor_sync(~0u, l[r], 1);
    l[r] += __shfl_xor_sync(~0u, l[r], 2);
    if (t == 0) jml[warp][g + r * 8] = make_float2(m[r], l[r]);
    if (t0 >= t1 || row0 + g + r * 8 >= a.G) continue;
    float *dst = rings + warp * (S::RING / 4) + (g + r * 8) * D;
    store_row(dst, r, 1.f);
  }
  __syncthreads();
  // one CTA has the whole pair, or its part goes to the cluster (through the first ring,
  // behind its warp's sums), or to the workspace
  const bool whole = pair.kt == 0 && c1 - (int)c0 == pair.nt;
  const bool shared = a.own > 1;
  float *const part = rings + MT * D;
  const long long slot = ((long long)blockIdx.y * gridDim.x * kWarps + blockIdx.x * cut.warps) * 2;
  const float vs = S::F8 ? c.v_scale[pair.h] : 1.f;
  const int used = (c1 - (int)c0 + cut.per - 1) / cut.per;  // warps with tiles
  const int rows_here = min(MT, a.G - row0);
  const long long hq0 = (long long)pair.b * a.Hq + (long long)pair.h * a.G + row0;
  for (int i = threadIdx.x; i < rows_here * (D / 4); i += kThreads) {
    const int row = i / (D / 4), col = i % (D / 4) * 4;
    float M = -INFINITY, sum = 0.f;
    for (int k = 0; k < used; ++k) M = fmaxf(M, jml[k][row].x);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < used; ++k) {
      const float f = jml[k][row].x == -INFINITY ? 0.f : ex2(jml[k][row].x - M);
      const float4 x = *reinterpret_cast<const float4 *>(rings + k * (S::RING / 4) + row * D + col);
      sum += jml[k][row].y * f;
      y.x += x.x * f;
      y.y += x.y * f;
      y.z += x.z * f;
      y.w += x.w * f;
    }
    const float f = whole && !shared ? vs / sum : 1.f;
    float *dst = shared ? part + row * D : whole ? a.O + (hq0 + row) * D : a.part_o + (slot * MT + row) * D;
    *reinterpret_cast<float4 *>(dst + col) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
    if (col == 0) {
      if (shared) {
        cml[row] = make_float2(M, sum);
      } else if (whole) {
        const float x = M + log2f(sum);
        if (a.lse) a.lse[hq0 + row] = x * kLn2;
        a.lse2[hq0 + row] = x;
      } else {
        a.part_ml[slot * MT + row] = make_float2(M, sum);
      }
    }
  }
  if (!shared) return;
  // the cluster's CTAs join the parts, each some of the columns
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int i = cluster.block_rank() * kThreads + threadIdx.x; i < rows_here * (D / 4); i += a.own * kThreads) {
    const int row = i / (D / 4), col = i % (D / 4) * 4;
    float2 ml[kMaxOwn];
    float4 x[kMaxOwn];
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxOwn; ++k) {
      if (k >= a.own) break;
      ml[k] = *cluster.map_shared_rank(&cml[row], k);
      x[k] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(part + row * D + col, k));
      M = fmaxf(M, ml[k].x);
    }
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMaxOwn; ++k) {
      if (k >= a.own) break;
      const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
      sum += ml[k].y * f;
      y.x += x[k].x * f;
      y.y += x[k].y * f;
      y.z += x[k].z * f;
      y.w += x[k].w * f;
    }
    const float f = vs / sum;
    *reinterpret_cast<float4 *>(a.O + (hq0 + row) * D + col) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
    if (col == 0) {
      const float z = M + log2f(sum);
      if (a.lse) a.lse[hq0 + row] = z * kLn2;
      a.lse2[hq0 + row] = z;
    }
  }
  cluster.sync();  // no CTA leaves while its part may still be read
}

// The parts of pair (b, h), in order.  A CTA whose range lies in the pair
// has left one (slot 0 of its first warp); the CTAs at the pair's two ends, where
// other pairs take part of the range, one per warp: in slot 1 where the pair starts
// inside the warp's range, else in slot 0.
struct Parts {
  int per, warps;
  int w0, w1;            // first and last warp
  int head, mid, tail;   // parts of the first CTA, of whole CTAs, of the last one
};
__device__ __forceinline__ int parts_of(const KvDev &c, const DecodeArgs &a, int b, int h, Parts &u) {
  u.per = a.plan[0];
  u.warps = a.plan[1];
  const int p0 = a.plan[2 + b], nt = a.plan[3 + b] - p0;
  const int T = a.plan[2 + c.B] * c.Hkv;  // tiles are at most 2^27
  const int first = p0 * c.Hkv + h * nt, last = first + nt - 1;
  if (nt == 0) return 0;
  u.w0 = first / u.per;
  u.w1 = last / u.per;
  const int cr = u.per * u.warps;  // tiles of a CTA
  const int k0 = first / cr, k1 = last / cr;
  // whole CTAs: all tiles of the CTA's range in the pair
  const bool whole0 = u.warps > 1 && first == k0 * cr && last >= min(T, (k0 + 1) * cr) - 1;
  const bool whole1 = u.warps > 1 && k1 > k0 && last == min(T, (k1 + 1) * cr) - 1;
  if (u.warps == 1) {
    u.head = u.w1 - u.w0 + 1;
    u.mid = u.tail = 0;
  } else if (k0 == k1) {
    u.head = whole0 ? 0 : u.w1 - u.w0 + 1;
    u.mid = whole0 ? 1 : 0;
    u.tail = 0;
  } else {
    u.head = whole0 ? 0 : (k0 + 1) * u.warps - u.w0;
    u.tail = whole1 ? 0 : u.w1 - k1 * u.warps + 1;
    u.mid = k1 - k0 - 1 + (whole0 ? 1 : 0) + (whole1 ? 1 : 0);
  }
  return u.head + u.mid + u.tail;
}
// Warp slot (warp * 2 + slot) of part i.
__device__ __forceinline__ long long part_slot(const Parts &u, int i) {
  if (i < u.head) return (long long)(u.w0 + i) * 2 + (i == 0);
  const int k0 = (u.w0 + u.head + u.warps - 1) / u.warps;  // first whole CTA
  if (i < u.head + u.mid) return (long long)(k0 + i - u.head) * u.warps * 2;
  return ((long long)(k0 + u.mid) * u.warps + (i - u.head - u.mid)) * 2;
}

constexpr int kFinThreads = 128;
constexpr int kFinWarps = kFinThreads / 32;

// Joins the partials of one query head (a row of O), in the order of the parts.
template <int D>
__device__ __forceinline__ void join(const KvDev &c, const DecodeArgs &a, int W, int MT, int id) {
  __shared__ float sm[kFinWarps], sl[kFinWarps];
  __shared__ float4 acc[kFinWarps][D / 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = id % a.Hq, b = id / a.Hq, h = hq / a.G, m = hq % a.G;
  Parts u;
  const int parts = parts_of(c, a, b, h, u);
  if (parts <= 1) return;  // empty, or finished by one warp or CTA
  const long long base = (long long)(m / MT) * W * 2;
  const int row = m % MT;
  auto slot = [&](int i) { return (base + part_slot(u, i)) * MT + row; };
  // each lane holds four columns; with d = 64 a warp takes two partials at a time.  Parts
  // are read once: a warp's sums follow its own maximum, the four are levelled at the end
  constexpr int kPer = 128 / D;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f, M = -INFINITY;
#pragma unroll 4
  for (int i = warp * kPer + lane / (D / 4); i < parts; i += kFinWarps * kPer) {
    const long long s = slot(i);
    const float2 ml = __ldcg(a.part_ml + s);
    const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.part_o + s * D + (lane % (D / 4)) * 4));
    const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
    const float e = ex2(M - base), f = ex2(ml.x - base);
    M = mn;
    l = l * e + ml.y * f;
    x.x = x.x * e + y.x * f;
    x.y = x.y * e + y.y * f;
    x.z = x.z * e + y.z * f;
    x.w = x.w * e + y.w * f;
  }
  if constexpr (kPer == 2) {
    const float mn = fmaxf(M, __shfl_xor_sync(~0u, M, 16));
    const float e = ex2(M - (mn == -INFINITY ? 0.f : mn));
    M = mn;
    l *= e;
    l += __shfl_xor_sync(~0u, l, 16);
    x = make_float4(x.x * e, x.y * e, x.z * e, x.w * e);
    x.x += __shfl_xor_sync(~0u, x.x, 16);
    x.y += __shfl_xor_sync(~0u, x.y, 16);
    x.z += __shfl_xor_sync(~0u, x.z, 16);
    x.w += __shfl_xor_sync(~0u, x.w, 16);
  }
  if (lane == 0) sm[warp] = M;
  if (lane < D / 4) acc[warp][lane] = x;
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  float f4[kFinWarps];
  M = sm[0];
  for (int i = 1; i < kFinWarps; ++i) M = fmaxf(M, sm[i]);
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kFinWarps; ++i) {
    f4[i] = ex2(sm[i] - (M == -INFINITY ? 0.f : M));
    l += sl[i] * f4[i];
  }
  if (threadIdx.x < D / 4) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kFinWarps; ++i) {
      y.x += acc[i][threadIdx.x].x * f4[i];
      y.y += acc[i][threadIdx.x].y * f4[i];
      y.z += acc[i][threadIdx.x].z * f4[i];
      y.w += acc[i][threadIdx.x].w * f4[i];
    }
    const float f = (c.v_scale ? c.v_scale[h] : 1.f) / l;
    *reinterpret_cast<float4 *>(a.O + (long long)id * D + threadIdx.x * 4) =
        make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
  }
  if (threadIdx.x == 0) {
    const float lse2 = M + log2f(l);
    a.lse2[id] = lse2;
    if (a.lse) a.lse[id] = lse2 * kLn2;
  }
}

template <int D>
__global__ void __launch_bounds__(kFinThreads) join_kernel(const KvDev c, const DecodeArgs a, int W, int MT) {
  tr_let_next_start();
  tr_wait_for_previous();
  join<D>(c, a, W, MT, blockIdx.x);
}

// Adds the weights of a pair's rows, summed over its query heads, to the
// rows' scores; bound by the logits' bytes.  SPLIT (more than 8 heads): a CTA
// takes 128 rows, each warp every fourth head; else 512 rows and every thread all
// heads of four rows.  With 4 heads and 262 k rows the split form took 20 us
// and the other 12 us; with 40 heads and 50 k rows 8 us and 19 us.
// lse2_of(m): the log2 of query head m's softmax denominator.
template <bool SPLIT, typename Lse2>
__device__ __forceinline__ void add_scores(const KvDev &c, const DecodeArgs &a, int b, int h, int L, int p0,
                                           Lse2 lse2_of) {
  __shared__ float4 sums[SPLIT ? kFinWarps : 1][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p = p0 + (SPLIT ? lane : threadIdx.x) * 4;
  const float *src = a.s + ((long long)b * a.Hq + (long long)h * a.G) * a.s_ld + p;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p < L) {
#pragma unroll 4
    for (int m = SPLIT ? warp : 0; m < a.G; m += SPLIT ? kFinWarps : 1) {
      const float lse2 = lse2_of(m);
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + m * a.s_ld));  // behind the last row: not used
      w.x += ex2(x.x - lse2);
      w.y += ex2(x.y - lse2);
      w.z += ex2(x.z - lse2);
      w.w += ex2(x.w - lse2);
    }
  }
  float *dst = c.scores + ((long long)b * c.Hkv + h) * c.scores_ld;
  if constexpr (SPLIT) {
    sums[warp][lane] = w;
    __syncthreads();
    const int r = p0 + threadIdx.x;
    if (r >= L) return;
    const float *all = reinterpret_cast<const float *>(sums);
    float x = all[threadIdx.x];
#pragma unroll
    for (int i = 1; i < kFinWarps; ++i) x += all[i * 128 + threadIdx.x];
    dst[r] += x;
  } else {
    const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i < L) dst[p + i] += x[i];
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kFinThreads) score_kernel(const KvDev c, const DecodeArgs a) {
  const int h = blockIdx.y, b = blockIdx.z, p0 = blockIdx.x * (SPLIT ? 128 : 512);
  tr_wait_for_previous();
  const int L = c.L[b];
  if (L < 0 || L > c.cap || p0 >= L) return;
  const float *lse2 = a.lse2 + (long long)b * a.Hq + (long long)h * a.G;
  add_scores<SPLIT>(c, a, b, h, L, p0, [&](int m) { return __ldcg(lse2 + m); });
}

// Joins and scores in one kernel: the first B * Hq CTAs join a query head each,
// those behind them (`chunks` for each pair, at most 8 heads a group) take their
// denominators from the parts' (m, l) themselves, a warp for each head.  It saves
// waiting for the joins and costs every one of these CTAs the denominators:
// 8 sequences of 4096 rows of 8 heads (512 of them) 35.5 us with two kernels, 33.1
// with one; 64 of up to 8191 (8192 of them) 113.6 and 117.1 us.
constexpr long long kOneFinish = 1024;
template <int D>
__global__ void __launch_bounds__(kFinThreads) finish_kernel(const KvDev c, const DecodeArgs a, int W, int MT,
                                                             unsigned joins, unsigned chunks) {
  __shared__ float lse2[8];
  tr_wait_for_previous();
  if (blockIdx.x < joins) {
    join<D>(c, a, W, MT, blockIdx.x);
    return;
  }
  const unsigned k = blockIdx.x - joins, pair = k / chunks;
  const int b = pair / c.Hkv, h = pair % c.Hkv, p0 = (k % chunks) * 512, L = c.L[b];
  if (L < 0 || L > c.cap || p0 >= L) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Parts u;
  const int parts = parts_of(c, a, b, h, u);
  const long long hq = (long long)b * a.Hq + (long long)h * a.G;
  for (int m = warp; m < a.G; m += kFinWarps) {
    float x;
    if (parts <= 1) {
      x = __ldcg(a.lse2 + hq + m);
    } else {
      float M = -INFINITY, l = 0.f;
      for (int i = lane; i < parts; i += 32) {
        const float2 y = __ldcg(a.part_ml + part_slot(u, i) * MT + m);
        const float mn = fmaxf(M, y.x), base = mn == -INFINITY ? 0.f : mn;
        l = l * ex2(M - base) + y.y * ex2(y.x - base);
        M = mn;
      }
      const float own = M;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
      l *= ex2(own - (M == -INFINITY ? 0.f : M));
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      x = M + log2f(l);
    }
    if (lane == 0) lse2[m] = x;
  }
  __syncthreads();
  add_scores<false>(c, a, b, h, L, p0, [&](int m) { return lse2[m]; });
}

// bf16 products can pass fp32's range where the scaled logits do not.  Below a scale
// of 2^-64 half of its exponent is multiplied into a copy of the queries first, so
// logits below 2^64 are right with any scale.  What that rounds is queries below 2^-51,
// by 2^-134 at most, which moves a logit by less than 2^-30 whatever the rows hold.  A
// kernel of its own: the multiplication inside split_kernel took every call of one
// sequence of 512 rows from 5.37 to 5.47 us.
constexpr int kPlainScale = -64;
constexpr int kScaleThreads = 256;
__global__ void __launch_bounds__(kScaleThreads) scale_queries_kernel(const uint4 *Q, uint4 *to, long long pieces,
                                                                      uint32_t factor) {
  tr_let_next_start();
  tr_wait_for_previous();
  for (long long i = (long long)blockIdx.x * kScaleThreads + threadIdx.x; i < pieces;
       i += (long long)gridDim.x * kScaleThreads) {
    const uint4 x = Q[i];
    to[i] = make_uint4(mul_bf16x2(x.x, factor), mul_bf16x2(x.y, factor), mul_bf16x2(x.z, factor),
                       mul_bf16x2(x.w, factor));
  }
}

// A CTA's share of a pair's bytes up to which clusters own pairs.  Measured (bf16,
// d = 128, calls in a graph; clusters against ranges over all pairs): 32 pairs,
// 512 rows 5.7 / 7.6 us, 2048 rows 9.2 / 9.9 us; 8 pairs of 4 heads, 4096 rows
// 9.5 / 9.9 us; one pair of 32 heads, 2048 rows 9.4 / 11.9 us, 4096 rows
// 12.1 / 20.5 us.  With larger shares the SMs that no cluster uses are missed.
// The host knows no lengths, so this and the rule below go by the positions that a
// sequence can hold; the figures are of caches that are full.  With room the same
// rows take the way of longer ones (rows not in L2): 32 pairs of 512 rows 6.6 us in a
// full cache, 8.9 with 8192 positions, 11.0 with 32768; 128 pairs of 4 heads 9.9 us,
// 17.3 with 8192.
constexpr long long kOwnBytes = 256 * 1024;
// Cache bytes from which 12 warps of two stages each are launched instead of 8
// of three.  Large reads gain from more warps (16 x 4k rows of 32 heads: 112
// against 116 us; 8-bit, 64 sequences: 115 against 121 us), short ranges from more
// tiles in flight at their start (24 sequences of up to 2k rows, d = 64: 14.2
// against 12.8 us; 8 x 4k rows of 8 heads, 134 MB: 36.9 against 35.5 us).  With room
// for 32768 rows the latter take 31.8 us without weights, 29.1 in a full cache.
constexpr long long kManyBytes = 512ll << 20;

// Launch shape and workspace: [partial O | partial (m, l) | lse2 | plan | scaled queries (bf16) | logits]
struct Plan {
  int MT, warps, row_tiles, grid;  // grid: CTAs per row tile
  int own;
  size_t ml_off, lse_off, plan_off, q_off, s_off, total;
};

Plan make_plan(const KvDev &c, tr_kvtype type, int Hq, int d, int accumulate) {
  Plan p;
  const int G = Hq / c.Hkv;
  const long long pairs = (long long)c.B * c.Hkv, bytes = (long long)c.cap * c.row_bytes * 2;  // of a pair
  p.MT = G <= 8 ? 8 : 16;
  p.row_tiles = (G + p.MT - 1) / p.MT;
  p.warps = p.MT == 8 && pairs * bytes >= kManyBytes ? 12 : 8;
  const long long most = pairs * ((c.cap + kMinRows - 1) / kMinRows);  // ranges worth a warp
  p.grid = (int)std::max<long long>(1, std::min<long long>(tr_sm_count() / p.row_tiles, most));
  // clusters as large as fit on the SMs and leave each warp a tile
  p.own = 0;
  if (pairs * p.row_tiles <= tr_sm_count()) {
    int cs = 1;
    while (cs < kMaxOwn && pairs * p.row_tiles * cs * 2 <= tr_sm_count() && c.cap > cs * 128) cs *= 2;
    if (bytes <= kOwnBytes * cs) p.own = cs;
  }
  if (p.own) {
    p.warps = 8;
    p.grid = (int)pairs * p.own;
  }
  const size_t rows = p.own ? 0 : (size_t)p.row_tiles * p.grid * p.warps * 2 * p.MT;  // clusters leave no partials
  p.ml_off = tr_align_up(rows * d * 4, 256);
  p.lse_off = p.ml_off + tr_align_up(rows * 8, 256);
  p.plan_off = p.lse_off + tr_align_up((size_t)c.B * Hq * 4, 256);
  p.q_off = p.plan_off + tr_align_up((size_t)(c.B + 3) * 4, 256);
  p.s_off = p.q_off + (type == TR_KV_BF16 ? tr_align_up((size_t)c.B * Hq * d * 2, 256) : 0);
  p.total = p.s_off + (accumulate ? (size_t)c.B * Hq * tr_align_up(c.cap, 32) * 4 : 0);
  return p;
}

template <int TYPE, int D, int MT, int NW>
int launch_split(const Plan &p, cudaStream_t s, const KvDev &c, const DecodeArgs &a) {
  static std::atomic<bool> set[64];  // per device
  int dev = 0;
  TR_TRY_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    TR_TRY_CUDA(cudaFuncSetAttribute(split_kernel<TYPE, D, MT, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRings));
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  return tr_launch_next(split_kernel<TYPE, D, MT, NW>, {dim3(p.grid, p.row_tiles), NW * 32, kRings, p.own > 1 ? p.own : 1},
                        s, c, a);
}

template <int TYPE, int D>
int launch(const Plan &p, cudaStream_t s, const KvDev &c, const DecodeArgs &a) {
  int rc = p.MT == 16     ? launch_split<TYPE, D, 16, 8>(p, s, c, a)
           : p.warps == 8 ? launch_split<TYPE, D, 8, 8>(p, s, c, a)
                          : launch_split<TYPE, D, 8, 12>(p, s, c, a);
  if (rc != TR_OK) return rc;
  const long long chunks = (c.cap + 511) / 512, pairs = (long long)c.B * c.Hkv;
  if (!p.own && a.accumulate && a.G <= 8 && pairs * chunks <= kOneFinish) {
    const unsigned joins = c.B * a.Hq;
    return tr_launch_next(finish_kernel<D>, {dim3(joins + (unsigned)(pairs * chunks)), kFinThreads}, s, c, a,
                          p.grid * p.warps, p.MT, joins, (unsigned)chunks);
  }
  if (!p.own) rc = tr_launch_next(join_kernel<D>, {dim3(c.B * a.Hq), kFinThreads}, s, c, a, p.grid * p.warps, p.MT);
  if (rc != TR_OK || !a.accumulate) return rc;
  return a.G > 8 ? tr_launch_next(score_kernel<true>, {dim3((c.cap + 127) / 128, c.Hkv, c.B), kFinThreads}, s, c, a)
                 : tr_launch_next(score_kernel<false>, {dim3((unsigned)chunks, c.Hkv, c.B), kFinThreads}, s, c, a);
}

template <int TYPE>
int launch(int d, const Plan &p, cudaStream_t s, const KvDev &c, const DecodeArgs &a) {
  return d == 64 ? launch<TYPE, 64>(p, s, c, a) : launch<TYPE, 128>(p, s, c, a);
}

// Launch grids hold B * Hq in 31 bits, the KV heads and the row tiles in 16.
bool fits(const KvDev &c, int Hq) {
  return (long long)c.B * Hq < (1LL << 31) && Hq < (1 << 24) && c.Hkv <= 65535 && Hq / c.Hkv <= 65535 * 8;
}

}  // namespace

extern "C" size_t tr_decode_attn_workspace_bytes(const tr_kv_cache *cache, int Hq, int accumulate) {
  KvDev c;
  if (kv_check(cache, &c) != TR_OK || Hq < 1 || Hq % c.Hkv || !fits(c, Hq)) return 0;
  return make_plan(c, cache->type, Hq, cache->d, accumulate).total;
}

extern "C" int tr_decode_attn(const void *Q, const tr_kv_cache *cache, int Hq, float scale, float *O, float *lse,
                              int accumulate, void *ws, size_t ws_bytes, tr_stream_t stream) {
  KvDev c;
  int rc = kv_check(cache, &c);
  if (rc != TR_OK) return rc;
  if (!Q || !O || Hq < 1 || Hq % c.Hkv || !(scale > 0.f) || !(scale < 0x1p127f)) return TR_E_INVAL;
  if ((((uintptr_t)Q | (uintptr_t)O) & 15) || ((uintptr_t)lse & 3)) return TR_E_INVAL;
  if (accumulate && !c.scores) return TR_E_INVAL;
  if (!fits(c, Hq)) return TR_E_UNSUPPORTED;
  const Plan p = make_plan(c, cache->type, Hq, cache->d, accumulate);
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < p.total) return TR_E_INVAL;
  rc = tr_check_device();
  if (rc != TR_OK) return rc;
  DecodeArgs a;
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.part_o = (float *)ws;
  a.part_ml = (float2 *)((char *)ws + p.ml_off);
  a.lse2 = (float *)((char *)ws + p.lse_off);
  a.plan = (int *)((char *)ws + p.plan_off);
  a.s = (float *)((char *)ws + p.s_off);
  a.s_ld = (long long)tr_align_up(c.cap, 32);
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.accumulate = accumulate != 0;
  a.own = p.own;
  const double scale_log2 = (double)scale * 1.4426950408889634f;  // exact: the smallest scales keep their bits
  a.scale_log2 = (float)scale_log2;
  a.scale_man = 2.f * (float)std::frexp(scale_log2, &a.scale_exp);
  --a.scale_exp;
  a.status = tr_status_dev();
  cudaStream_t s = (cudaStream_t)stream;
  if (cache->type == TR_KV_BF16 && a.scale_exp < kPlainScale) {
    const int half = a.scale_exp / 2;
    const uint32_t f = (uint32_t)(127 + half) << 7;
    const long long pieces = (long long)cache->B * Hq * cache->d / 8;
    const long long ctas = std::min<long long>((pieces + kScaleThreads - 1) / kScaleThreads, 8LL * tr_sm_count());
    uint4 *const to = (uint4 *)((char *)ws + p.q_off);
    rc = tr_launch_next(scale_queries_kernel, {dim3((unsigned)ctas), kScaleThreads}, s, (const uint4 *)Q, to, pieces,
                        f | f << 16);
    if (rc != TR_OK) return rc;
    a.Q = to;
    a.scale_log2 = (float)std::ldexp(scale_log2, -half);
  }
  if (cache->type == TR_KV_BF16) return launch<TR_KV_BF16>(cache->d, p, s, c, a);
  if (cache->type == TR_KV_F16) return launch<TR_KV_F16>(cache->d, p, s, c, a);
  return launch<TR_KV_E4M3>(cache->d, p, s, c, a);
}
