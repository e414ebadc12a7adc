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
// serves it for all heads of the token.  The weights of the norm are multiplied into these, the norm's factor comes
// last: 16 elements take some 60 packed instructions.  A warp's step is a group of 32 / (d / 16) heads of one kind
// (queries, keys or values), 1 KB.
//
// Measured in a graph (rows not in L2; of a copy's rate): 4 x 8192 tokens of 32/8 heads of 128, bf16, norms 135 us (88%),
// fp16 137, 16 x 8192 519 (91%), without norms 140 (85%), pairs of neighbours 132 (90%), 32/32 heads 274 (87%), heads of 64
// 71 (84%), 64/8 heads 122 of 2 x 8192 (81%), 8/2 heads 35 of 4 x 4096 (43%: keys and values are half a group each, and a
// token's angles and factors serve four groups; 1377 instructions a token, issue slots 58% busy); 8 x 700 28 (71%); a tree
// of 80 nodes 3.7, 8 trees of 128 with 32/8 heads 8.5; into pages, 8 prompts up to 4096 long 84 (86%), e4m3 99 (68%: a
// division by the scale, found anew for every group); one token for each of 64 sequences 3.8 to 4.1, e4m3, 4.4 to 4.8.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "tr_append.cuh"

namespace {

constexpr int kMaxWarps = 8;
constexpr int kCtas = 2;    // of rope_kernel on an SM
constexpr int kStages = 6;  // groups in a warp's ring
constexpr int kShort = 2;   // groups of a task in append_rope_kernel, at most

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
  int groups[3], all_groups;      // of heads: of a kind, of a token
  int parts, per;                 // shares of a token, groups of a share (append_rope_kernel: of a task)
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

__device__ __forceinline__ void copy16(uint32_t dst, const char *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// Turns a position as a fraction of 2^64: a multiplication by the position wraps around
// with the whole turns, so far positions lose nothing.  Of f = man 2^e, man of 24 bits, in whole numbers:
// off by 1 + f units at most, from 2^24 on (whose next number is more than a turn away) by two: there
// 1 / (2 pi) is taken from its e-th bit on, what is above being whole turns (Payne and Hanek 1983).
__device__ __forceinline__ unsigned long long turns_of(float f) {
  typedef unsigned long long u64;
  constexpr u64 kInv = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi), rounded down, and its next 128 bits
  constexpr u64 kInv1 = 0x7F09D5F47D4D3770ull, kInv2 = 0x36D8A5664F10E410ull;
  const unsigned bits = __float_as_uint(f), power = bits >> 23 & 255;
  const int right = 150 - (int)power;                         // -e
  const u64 man = power ? (bits & 0x7FFFFFu) | 0x800000u : 0;  // below 2^-126: no turn
  u64 t;
  if (right < 0) {
    const int e = -right, by = e & 63;  // e is 104 at most
    const u64 a = e < 64 ? kInv : kInv1, b = e < 64 ? kInv1 : kInv2, c = e < 64 ? kInv2 : 0;
    const u64 hi = by ? a << by | b >> (64 - by) : a, lo = by ? b << by | c >> (64 - by) : b;
    t = man * hi + __umul64hi(man, lo);
  } else {
    const u64 lo = man * kInv, hi = __umul64hi(man, kInv);
    t = right == 0 ? lo : right < 64 ? hi << (64 - right) | lo >> right : right < 128 ? hi >> (right - 64) : 0;
  }
  return bits >> 31 ? 0 - t : t;
}
// cos and sin at position p: its phase rounded down to 2^-32 of a turn, as half turns in fp32.
__device__ __forceinline__ float2 turn(long long p, unsigned long long f) {
  const int phase = (int)(((unsigned long long)p * f) >> 32);
  float2 r;
  sincospif((float)phase * 0x1p-31f, &r.y, &r.x);
  return r;
}

// Two fp32 values in one register pair, and one instruction.
struct F2 {
  unsigned long long v;
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
__device__ __forceinline__ F2 operator-(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }

// What a warp keeps of a token and a kind: z0 = x0 a0 - x1 b0, z1 = x1 a1 + x0 b1 with the
// angles' cosines in a and sines in b, each times the weight of its element of x; two
// pairs of elements to a register pair.
struct Held {
  F2 a0[4], b0[4], a1[4], b1[4];  // b0 negated
};

enum { kDense, kCache, kCache8 };  // where keys and values go

template <bool BF, int D, bool PAIRS, int DST>
struct Rows {
  static constexpr int LPH = D / 16, HPG = 32 / LPH;  // lanes of a head, heads of a group
  const RopeArgs &a;
  const KvDev &c;
  float2 *table;      // the warp's, D / 2; behind it the frequencies' turns, of each lane its own
  int lane, sub, head, pa, pb;  // lane of its head, head of the group, the lane's pieces
  bool turned;
  Held k;
  int held;           // the kind that k is of

  __device__ __forceinline__ Rows(const RopeArgs &a_, const KvDev &c_, float2 *t) : a(a_), c(c_), table(t) {
    lane = threadIdx.x & 31;
    sub = lane % LPH;
    head = lane / LPH;
    turned = sub < a.rot / 16;
    const bool apart = turned && !PAIRS;
    pa = apart ? sub : 2 * sub;
    pb = apart ? sub + a.rot / 16 : 2 * sub + 1;
    held = -1;
  }

  __device__ __forceinline__ unsigned long long *turns() { return reinterpret_cast<unsigned long long *>(table + D / 2); }
  __device__ __forceinline__ void frequencies() {
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      if (lane + 32 * e < a.rot / 2) turns()[lane + 32 * e] = turns_of(a.inv_freq[lane + 32 * e]);
  }

  // Cosines and sines of the token at position p into the table.
  __device__ __forceinline__ void angles(long long p) {
    held = -1;
    if (a.rot == 0) return;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      if (lane + 32 * e < a.rot / 2) table[lane + 32 * e] = turn(p, turns()[lane + 32 * e]);
    __syncwarp();
  }

  // The lane's factors for a kind: eight pairs of elements, (x0, x1) = elements e of
  // its two pieces, or neighbours.
  __device__ __forceinline__ void factors(int kind) {
    if (held == kind) return;
    held = kind;
    const float *w = a.norm[kind];
    float wa[8], wb[8];
    if (w) {
      // one 16-byte load for four where the array's address allows it
      if (((uintptr_t)w & 15) == 0) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 x = reinterpret_cast<const float4 *>(w + pa * 8)[q], y = reinterpret_cast<const float4 *>(w + pb * 8)[q];
          wa[4 * q] = x.x, wa[4 * q + 1] = x.y, wa[4 * q + 2] = x.z, wa[4 * q + 3] = x.w;
          wb[4 * q] = y.x, wb[4 * q + 1] = y.y, wb[4 * q + 2] = y.z, wb[4 * q + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wa[e] = w[pa * 8 + e];
          wb[e] = w[pb * 8 + e];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float4 cs = make_float4(1.f, 0.f, 1.f, 0.f);
      if (turned) cs = reinterpret_cast<const float4 *>(table + sub * 8)[q];
      F2 c2 = f2(cs.x, cs.z), s2 = f2(cs.y, cs.w);
      if (w) {
        // PAIRS: pairs 2q, 2q + 1 are elements 4q .. 4q + 3 of the 16
        const F2 w0 = PAIRS ? (q < 2 ? f2(wa[(4 * q) & 7], wa[(4 * q + 2) & 7]) : f2(wb[(4 * q) & 7], wb[(4 * q + 2) & 7]))
                            : f2(wa[2 * q], wa[2 * q + 1]);
        const F2 w1 = PAIRS ? (q < 2 ? f2(wa[(4 * q + 1) & 7], wa[(4 * q + 3) & 7]) : f2(wb[(4 * q + 1) & 7], wb[(4 * q + 3) & 7]))
                            : f2(wb[2 * q], wb[2 * q + 1]);
        k.a0[q] = c2 * w0;
        k.b0[q] = -(s2 * w1);
        k.a1[q] = c2 * w1;
        k.b1[q] = s2 * w0;
      } else {
        k.a0[q] = k.a1[q] = c2;
        k.b0[q] = -s2;
        k.b1[q] = s2;
      }
    }
  }

  // Whether a kind's rows go to dense rows, and whether they are narrowed to 8 bits.
  static constexpr bool to_rows(int kind) { return DST == kDense || kind == 0; }
  static constexpr bool to_8(int kind) { return !to_rows(kind) && DST == kCache8; }

  // Where head h of token i of sequence b goes, p being its place in the cache, and bytes between heads there.
  template <int KIND>
  __device__ __forceinline__ char *target(int b, int i, int p, int h) const {
    if (to_rows(KIND)) return a.out[KIND] + (((long long)b * a.T + i) * a.heads[KIND] + h) * (D * 2);
    return (KIND == 1 ? c.K : c.V) + kv_block(c, b, p) + kv_row(c, p) + h * c.head_stride;
  }
  template <int KIND>
  __device__ __forceinline__ long long pitch() const {
    return to_rows(KIND) ? D * 2 : c.head_stride;
  }

  // Norms and turns the lane's pieces x of head h and stores them, where the head is there
  // (else they may be anything).
  template <int KIND>
  __device__ __forceinline__ void store(char *dst, int h, bool there, const uint4 (&x)[2]) {
    constexpr bool kNarrow = to_8(KIND);
    uint4 out[2] = {x[0], x[1]};
    F2 x0[4], x1[4];  // the two elements of pairs 2q and 2q + 1
    if (KIND < 2 || kNarrow) {
      const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 m = widen(PAIRS ? w[2 * q] : w[q], BF), n = widen(PAIRS ? w[2 * q + 1] : w[4 + q], BF);
        x0[q] = PAIRS ? f2(m.x, n.x) : f2(m.x, m.y);
        x1[q] = PAIRS ? f2(m.y, n.y) : f2(n.x, n.y);
      }
    }
    if (KIND < 2) {
      const bool norm = a.norm[KIND < 2 ? KIND : 0] != nullptr;
      F2 r2;
      if (norm) {
        F2 s0 = x0[0] * x0[0], s1 = x1[0] * x1[0];
#pragma unroll
        for (int q = 1; q < 4; ++q) {
          s0 = fma(x0[q], x0[q], s0);
          s1 = fma(x1[q], x1[q], s1);
        }
        const float2 y0 = split(s0), y1 = split(s1);
        float s = (y0.x + y0.y) + (y1.x + y1.y);
#pragma unroll
        for (int o = LPH / 2; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        const float r = rsqrtf(fmaf(s, 1.f / D, a.eps));
        r2 = f2(r, r);
      }
      if (turned) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const F2 z0 = fma(x1[q], k.b0[q], x0[q] * k.a0[q]), z1 = fma(x0[q], k.b1[q], x1[q] * k.a1[q]);
          x0[q] = z0;
          x1[q] = z1;
        }
      } else if (norm) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x0[q] = x0[q] * k.a0[q];
          x1[q] = x1[q] * k.a1[q];
        }
      }
      if (norm) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x0[q] = x0[q] * r2;
          x1[q] = x1[q] * r2;
        }
      }
    }
    float y[16];  // in the order of the pieces
    if (KIND < 2 || kNarrow) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 z0 = split(x0[q]), z1 = split(x1[q]);
        y[PAIRS ? 4 * q : 2 * q] = z0.x;
        y[PAIRS ? 4 * q + 2 : 2 * q + 1] = z0.y;
        y[PAIRS ? 4 * q + 1 : 8 + 2 * q] = z1.x;
        y[PAIRS ? 4 * q + 3 : 8 + 2 * q + 1] = z1.y;
      }
    }
    if (!there) return;
    if constexpr (kNarrow) {
      const Scale s = make_scale((KIND == 1 ? c.k_scale : c.v_scale)[h]);
      float lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = y[e];
        hi[e] = y[8 + e];
      }
      reinterpret_cast<uint2 *>(dst)[pa] = e4m3_of(lo, s);
      reinterpret_cast<uint2 *>(dst)[pb] = e4m3_of(hi, s);
    } else {
      if (KIND < 2) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          out[q] = make_uint4(narrow(y[8 * q], y[8 * q + 1], BF), narrow(y[8 * q + 2], y[8 * q + 3], BF),
                              narrow(y[8 * q + 4], y[8 * q + 5], BF), narrow(y[8 * q + 6], y[8 * q + 7], BF));
      }
      reinterpret_cast<uint4 *>(dst)[pa] = out[0];
      reinterpret_cast<uint4 *>(dst)[pb] = out[1];
    }
  }

  // Kind and first head of a token's group; the address of its rows.
  __device__ __forceinline__ int place(int g, int &h0) const {
    int kind = 0;
    if (g >= a.groups[0]) g -= a.groups[0], kind = 1;
    if (kind == 1 && g >= a.groups[1]) g -= a.groups[1], kind = 2;
    h0 = g * HPG;
    return kind;
  }
  __device__ __forceinline__ const uint4 *source(int kind, int b, int i, int h) const {
    return reinterpret_cast<const uint4 *>(a.x[kind] + b * a.stride[kind][0] + i * a.stride[kind][1] +
                                           h * a.stride[kind][2]);
  }
};

// All tokens: an item is a token, or one of a.parts shares of its groups, and a warp takes every
// gridDim * 8-th item.  Groups come through the warp's ring in shared memory (cp.async), kStages - 1
// ahead of the one in work and across items, so that the bytes under way need no registers: loads into registers took
// 4 x 8192 tokens 146 to 150 us when they were tried, 16 stages 160 (the L1 that they take is the stores'), three CTAs on an
// SM with 80 registers 303 (they spill; with two on an SM only the variants that write e4m3 do, 8 to 16 bytes).
// With a cache the lengths are what the plan kernel has left in todo.
template <bool BF, int D, bool PAIRS, int DST>
__global__ void __launch_bounds__(256, kCtas) rope_kernel(const RopeArgs a, const KvDev c,
                                                          const __grid_constant__ Depths tree) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5;
  using R = Rows<BF, D, PAIRS, DST>;
  R r(a, c, reinterpret_cast<float2 *>(smem) + warp * D);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + 8 * D * 8 + warp * (kStages * 1024);
  // a group's heads lie one behind the other in a stage: copied in order, read by pieces
  const uint32_t copy_at = ring + r.head * (D * 2) + r.sub * 16;
  const uint32_t read_a = ring + r.head * (D * 2) + r.pa * 16, read_b = ring + r.head * (D * 2) + r.pb * 16;
  tr_let_next_start();
  tr_wait_for_previous();
  const unsigned items = (unsigned)a.B * a.T * a.parts, stride = gridDim.x * 8;
  struct Cursor {
    unsigned it;
    int g, b, i, len;  // g: first group
  };
  auto enter = [&](Cursor &u) {  // item u.it, or the next one that there is
    for (; u.it < items; u.it += stride) {
      const unsigned row = a.parts == 1 ? u.it : u.it / a.parts;
      u.b = row / a.T;
      u.i = row - u.b * a.T;
      u.g = (u.it - row * a.parts) * a.per;
      if (DST == kDense) return;
      const int2 todo = a.todo[u.b];
      u.len = todo.x;
      if (u.i < todo.y) return;
    }
  };
  Cursor u, ld;
  u.it = blockIdx.x * 8 + warp;
  enter(u);
  ld = u;
  // the loader's place: `run` groups of one kind from src on, the lane's head among the kind's `left` ones
  const char *src = nullptr;
  long long src_step = 0;
  int run = 0, left = 0;
  auto find = [&] {
    int h0;
    const int kind = r.place(ld.g, h0);
    src_step = a.stride[kind][2] * R::HPG;
    src = reinterpret_cast<const char *>(r.source(kind, ld.b, ld.i, h0 + r.head)) + r.sub * 16;
    left = a.heads[kind] - h0 - r.head;
    const int end = min(a.all_groups, (ld.g / a.per + 1) * a.per);
    run = min((a.heads[kind] - h0 + R::HPG - 1) / R::HPG, end - ld.g);
    ld.g += run;
    if (ld.g == end) {
      ld.it += stride;
      enter(ld);
    }
  };
  auto issue = [&](uint32_t stage) {
    if (run == 0 && ld.it < items) find();
    if (run > 0) {
      if (left > 0) {
        copy16(copy_at + stage, src);
        copy16(copy_at + stage + R::LPH * 16, src + R::LPH * 16);
      }
      src += src_step;
      left -= R::HPG;
      --run;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k * 1024);
  r.frequencies();
  uint32_t stage = 0;
  // groups [g0, g1) of a kind, counted from its first
  auto groups = [&](auto K, int g0, int g1, int p) {
    constexpr int KIND = decltype(K)::value;
    if (g0 >= g1) return;
    if (KIND < 2) r.factors(KIND);
    int h = g0 * R::HPG + r.head;
    char *dst = r.template target<KIND>(u.b, u.i, p, h);
    const long long step = r.template pitch<KIND>() * R::HPG;
    if (!R::to_rows(KIND) && KIND == 1 && c.scores)  // of all the groups' heads
      for (int k = g0 * R::HPG + r.lane; k < min(a.heads[1], g1 * R::HPG); k += 32)
        c.scores[((long long)u.b * c.Hkv + k) * c.scores_ld + p] = 0.f;
    for (int g = g0; g < g1; ++g) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // every lane's copies are there, and the stage before this one is free
      const uint4 x[2] = {lds16(read_a + stage), lds16(read_b + stage)};
      issue((stage + (kStages - 1) * 1024) % (kStages * 1024));
      r.template store<KIND>(dst, h, h < a.heads[KIND], x);
      dst += step;
      h += R::HPG;
      stage = (stage + 1024) % (kStages * 1024);
    }
  };
  for (; u.it < items; u.it += stride, enter(u)) {
    const int g0 = u.g, g1 = min(a.all_groups, g0 + a.per), p = u.len + u.i;
    const int k1 = a.groups[0], k2 = k1 + a.groups[1];
    if (g0 < k2) r.angles(a.pos ? (long long)a.pos[u.b] + (tree.nodes ? tree.of[u.i] : u.i) : p);
    groups(std::integral_constant<int, 0>{}, g0, min(g1, k1), p);
    groups(std::integral_constant<int, 1>{}, max(g0, k1) - k1, min(g1, k2) - k1, p);
    groups(std::integral_constant<int, 2>{}, max(g0, k2) - k2, g1 - k2, p);
  }
}

// Few rows: a cluster takes a sequence, checks it, copies its rows and advances its length,
// so that no kernel is needed before this one.  A task is the next U groups of a token, whose loads are requested
// before the sequence is checked; a warp takes every (gridDim * warps)-th.  Latency bounds it: one token 3.4 to 3.6 us, of
// which the launch is most.
template <bool BF, int D, bool PAIRS, int DST>
__global__ void __launch_bounds__(kMaxWarps * 32, 2) append_rope_kernel(const RopeArgs a, const KvDev c) {
  constexpr int U = kShort;
  __shared__ __align__(16) float2 tables[kMaxWarps][D];
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Rows<BF, D, PAIRS, DST> r(a, c, tables[warp]);
  tr_let_next_start();
  tr_wait_for_previous();
  const int b = blockIdx.y, Lb = c.L[b], n0 = a.count ? a.count[b] : a.T;
  const int step = gridDim.x * warps, tasks = (a.all_groups + a.per - 1) / a.per;
  uint4 x[U][2];
  int i, g;
  auto load = [&](int t) {
    i = t / tasks;
    g = (t - i * tasks) * a.per;
    if (i >= a.T) return;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      int h0;
      const int kind = r.place(g + k, h0);
      x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
      if (k >= a.per || g + k >= a.all_groups || h0 + r.head >= a.heads[kind]) continue;
      const uint4 *src = r.source(kind, b, i, h0 + r.head);
      x[k][0] = src[r.pa];
      x[k][1] = src[r.pb];
    }
  };
  int t = blockIdx.x * warps + warp;
  load(t);  // before the checks (the rows are read even if these fail)
  r.frequencies();
  const long long base = a.pos ? (long long)a.pos[b] : Lb;
  const int n = append_rows(c, b, Lb, n0, a.T, a.status);
  int angle_of = -1;
  while (i < n) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      int h0;
      const int kind = r.place(g + k, h0);
      if (k >= a.per || g + k >= a.all_groups) break;
      if (kind < 2) {
        if (angle_of != i) r.angles(base + (angle_of = i));
        r.factors(kind);
      }
      const int h = h0 + r.head;
      const bool there = h < a.heads[kind];
      if (kind == 0) {
        r.template store<0>(r.template target<0>(b, i, Lb + i, h), h, there, x[k]);
      } else if (kind == 1) {
        r.template store<1>(r.template target<1>(b, i, Lb + i, h), h, there, x[k]);
        if (c.scores && r.sub == 0 && there) c.scores[((long long)b * c.Hkv + h) * c.scores_ld + Lb + i] = 0.f;
      } else {
        r.template store<2>(r.template target<2>(b, i, Lb + i, h), h, there, x[k]);
      }
    }
    load(t += step);
  }
  if (gridDim.x > 1) {  // the sequence's other CTAs have read the old length
    asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;" ::: "memory");
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && n > 0) c.L[b] = Lb + n;
}

void count_groups(RopeArgs *a, int d) {
  const int heads = 32 / (d / 16);
  a->all_groups = 0;
  for (int i = 0; i < 3; ++i) a->all_groups += a->groups[i] = (a->heads[i] + heads - 1) / heads;
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
  // (two shares a token, and the warps' steps behind the last one, are counted in 32 bits)
  if ((long long)x->B * x->T >= (1LL << 30) || all > (1 << 20)) return TR_E_UNSUPPORTED;
  a.B = x->B;
  a.T = x->T;
  a.rot = r->rot;
  a.inv_freq = r->inv_freq;
  a.norm[0] = r->q_norm;
  a.norm[1] = r->k_norm;
  a.eps = r->eps;
  count_groups(&a, r->d);
  a.pos = pos;
  *out = a;
  return TR_OK;
}

template <bool BF, int D, bool PAIRS, int DST>
int launch(RopeArgs a, const KvDev &c, const Depths &tree, cudaStream_t s) {
  constexpr int kSmem = 8 * (kStages * 1024 + D * 8);
  static std::atomic<bool> set[64];  // per device
  int dev = 0;
  TR_TRY_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    TR_TRY_CUDA(cudaFuncSetAttribute(rope_kernel<BF, D, PAIRS, DST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  const long long rows = (long long)a.B * a.T, most = (long long)kCtas * tr_sm_count();
  // Shares of a token: as many as give every warp one, where tokens are few.  Where they are many, one, but two of tokens
  // with 12 groups and more whose halves are paired behind a norm (its work is more than the angles that both halves
  // then need), unless there are 16 groups and as many of them are keys' and values' as queries' (the cut then falls into
  // the keys).  One against two, 32 queries' and 8 keys' heads of 128, dense: 4 x 8192 tokens 145 / 135 us, 3 x 8192
  // 107 / 103, 4 x 5000 87 / 85; without norms 141 / 147 us, pairs of neighbours 137 / 143 us, 8 x 700 tokens 27.9 / 28.6
  // us; into a cache, ragged, 88 / 99 us.  Other heads, 4 x 8192: of 128, 32/4 (10 groups) 107 / 127, 16/16 (12) 145 / 137,
  // 24/12 (12) 146 / 132, 40/8 (14) 170 / 149, 48/8 (16) 194 / 172, 32/16 (16) 191 / 195, 24/24 (18) 211 / 224, 64/8 (20)
  // 240 / 236, 48/16 (20) 238 / 237, 64/16 (24) 283 / 284, 32/32 (24) 274 / 295, 64/32 (32) 364 / 377; of 64, 32/8 (6)
  // 71 / 90, 64/8 (10) 119 / 118, 64/16 (12) 146 / 128, 32/32 (12) 144 / 147, 128/8 (18) 217 / 215.
  const bool two = DST == kDense && !PAIRS && a.norm[0] && a.norm[1] && a.all_groups >= 12 &&
                   (a.all_groups < 16 || 2 * a.groups[0] > a.all_groups) && rows >= 8 * most * 8;
  a.parts = (int)std::max<long long>(two ? 2 : 1, std::min<long long>(a.all_groups, most * 8 / rows));
  a.per = (a.all_groups + a.parts - 1) / a.parts;
  a.parts = (a.all_groups + a.per - 1) / a.per;
  const long long ctas = (rows * a.parts + 7) / 8;
  return tr_launch_next(rope_kernel<BF, D, PAIRS, DST>, {dim3((unsigned)std::min(ctas, most)), 256, kSmem}, s, a, c, tree);
}

// One kernel for a sequence's rows up to this many tasks of a warp, else a plan and rope_kernel.  In a graph, one against
// two, 32/8 heads of 128: 64 x 1 tokens 3.8 / 5.0 us, 1 x 10 4.6 / 5.1, 24 x 16 7.5 / 6.4, 24 x 33 13.5 / 9.5, 8 x 85
// 19.1 / 8.1; the second launch takes the host 2.4 us.
constexpr int kRounds = 2, kMostCluster = 8;

template <bool BF, int D, bool PAIRS, int DST>
int launch_append(RopeArgs a, const KvDev &c, const int32_t *count, void *ws, cudaStream_t s) {
  // A task is a group where every warp of a cluster gets one at most and the clusters fill the SMs once, else two.  One
  // against two, in us: one token of 32/32 heads 3.5 / 4.1 (e4m3 4.1 / 5.0), 1 x 4 of 32/8 3.5 / 4.1, 16 x 1 3.6 / 3.8,
  // 32 x 1 3.8 / 3.8, 64 x 1 4.05 / 3.9 (e4m3 4.4 / 5.5), 72 x 1 3.9 / 4.0, 24 x 4 4.1 / 4.4, 64 x 1 of 8/2 3.3 / 3.6;
  // with one always 64 x 4 9.0 / 5.8, 24 x 21 10.1 / 8.4.
  const long long alone = (long long)a.T * a.all_groups;
  a.per = alone <= kMostCluster * kMaxWarps && a.B * ((alone + kMaxWarps - 1) / kMaxWarps) <= tr_sm_count() ? 1 : kShort;
  const long long tasks = (long long)a.T * ((a.all_groups + a.per - 1) / a.per);
  if (tasks <= (long long)kMostCluster * kMaxWarps * kRounds) {
    int cs = 1;
    while (cs < kMostCluster && tasks > (long long)cs * kMaxWarps) cs *= 2;
    const int warps = (int)std::min<long long>(kMaxWarps, (tasks + cs - 1) / cs);
    a.count = count;
    a.status = tr_status_dev();
    return tr_launch_next(append_rope_kernel<BF, D, PAIRS, DST>, {dim3(cs, a.B), warps * 32, 0, cs}, s, a, c);
  }
  a.todo = (const int2 *)ws;
  const int rc = kv_append_plan(c, a.T, count, (int2 *)ws, s);
  return rc != TR_OK ? rc : launch<BF, D, PAIRS, DST>(a, c, Depths{}, s);
}

// Whether numbers of the sequences overlap the cache's lengths without being these: a sequence's could then be read
// after another one's length was advanced.
bool part_of_lengths(const int32_t *x, const tr_kv_cache &c) {
  const uintptr_t a = (uintptr_t)x, l = (uintptr_t)c.L, bytes = (uintptr_t)c.B * sizeof(int32_t);
  return x && a != l && (a < l ? l - a : a - l) < bytes;
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
  if (part_of_lengths(pos, *cache) || part_of_lengths(count, *cache)) return TR_E_INVAL;
  // the lengths before the call, which the plan kernel has advanced before rope_kernel would read them
  if (pos == cache->L) a.pos = nullptr;
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
