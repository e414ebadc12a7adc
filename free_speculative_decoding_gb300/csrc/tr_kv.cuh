// Addressing and host checks of a tr_kv_cache, shared by the single-token
// attention, the append and the eviction.
#pragma once

#include "tr_internal.cuh"

// A cache as the kernels see it: strides in bytes, the page size as a shift.
// The kernels may be set up before the one before them ends (tr_launch_next), so
// nothing that it can have written is read through the non-coherent path (__ldg).
struct KvDev {
  char *K, *V;
  int B, Hkv;
  int row_bytes;  // d * element size
  int32_t *L;
  const int32_t *page_table;  // NULL: dense
  int max_pages, num_pages, page_log2;
  int cap;  // positions a sequence can hold
  long long block_stride, head_stride, row_stride;
  const float *k_scale, *v_scale;
  float *scores;
  long long scores_ld;
};

// Byte offset of the page (or dense sequence) that holds position p of
// sequence b, -1 for a page table entry that points nowhere.
__device__ __forceinline__ long long kv_block(const KvDev &c, int b, int p) {
  if (!c.page_table) return (long long)b * c.block_stride;
  const int page = c.page_table[(long long)b * c.max_pages + (p >> c.page_log2)];
  return (unsigned)page < (unsigned)c.num_pages ? (long long)page * c.block_stride : -1;
}

// Byte offset of position p inside its block.
__device__ __forceinline__ long long kv_row(const KvDev &c, int p) {
  return (long long)(c.page_table ? p & ((1 << c.page_log2) - 1) : p) * c.row_stride;
}

// Whether the whole block finds a bad page among those of positions [p0, p1)
// of sequence b (the same answer in every thread; contains a barrier).
__device__ __forceinline__ bool kv_bad_pages(const KvDev &c, int b, int p0, int p1) {
  int bad = 0;
  if (c.page_table && p1 > p0)
    for (int i = (p0 >> c.page_log2) + threadIdx.x; i <= (p1 - 1) >> c.page_log2; i += blockDim.x)
      bad |= (unsigned)c.page_table[(long long)b * c.max_pages + i] >= (unsigned)c.num_pages;
  return __syncthreads_or(bad);
}

// Checks a cache on the host and fills its device view.
static inline int kv_check(const tr_kv_cache *c, KvDev *out) {
  if (!c || !c->K || !c->V || !c->L || c->B < 1 || c->Hkv < 1) return TR_E_INVAL;
  if (c->type != TR_KV_BF16 && c->type != TR_KV_F16 && c->type != TR_KV_E4M3) return TR_E_INVAL;
  const bool e4m3 = c->type == TR_KV_E4M3;
  if (e4m3 != (c->k_scale != nullptr) || e4m3 != (c->v_scale != nullptr)) return TR_E_INVAL;
  if (c->d < 1) return TR_E_INVAL;
  if (c->d != 64 && c->d != 128) return TR_E_UNSUPPORTED;
  long long cap, blocks;
  KvDev v;
  v.page_log2 = 0;
  if (c->page_table) {
    if (c->max_pages < 1 || c->num_pages < 1 || c->page_size < 1) return TR_E_INVAL;
    if (c->page_size & (c->page_size - 1)) return TR_E_UNSUPPORTED;
    while ((1 << v.page_log2) < c->page_size) ++v.page_log2;
    cap = (long long)c->max_pages * c->page_size;
    blocks = c->num_pages;
  } else {
    if (c->cap < 1) return TR_E_INVAL;
    cap = c->cap;
    blocks = c->B;
  }
  const long long esz = e4m3 ? 1 : 2;
  if (((uintptr_t)c->K | (uintptr_t)c->V) & 15) return TR_E_INVAL;
  if (((uintptr_t)c->L | (uintptr_t)c->page_table | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale | (uintptr_t)c->scores) & 3)
    return TR_E_INVAL;
  const long long rows = c->page_table ? c->page_size : cap;
  // strides: 16-byte aligned wherever they are used, and no two rows overlap
  // (sorted by stride, each dimension steps over what the smaller ones span)
  long long n[3] = {blocks, c->Hkv, rows}, st[3] = {c->block_stride, c->head_stride, c->row_stride};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) st[i] = 0;
    if (st[i] < 0 || st[i] >= (1LL << 58) || (st[i] * esz) & 15) return TR_E_INVAL;
  }
  long long span = c->d;
  bool used[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (at < 0 || st[i] < st[at])) at = i;
    if (at < 0) break;
    used[at] = true;
    if (st[at] < span) return TR_E_INVAL;
    if (st[at] > (1LL << 60) / n[at]) return TR_E_INVAL;
    span += st[at] * (n[at] - 1);
  }
  const long long pairs = (long long)c->B * c->Hkv;
  if (c->scores && (c->scores_ld < cap || c->scores_ld > (1LL << 60) / pairs)) return TR_E_INVAL;
  if (c->B > 1024 || cap > (1LL << 30) || pairs > ((1LL << 31) - 1) / cap) return TR_E_UNSUPPORTED;
  v.K = (char *)c->K;
  v.V = (char *)c->V;
  v.B = c->B;
  v.Hkv = c->Hkv;
  v.row_bytes = (int)(c->d * esz);
  v.L = c->L;
  v.page_table = c->page_table;
  v.max_pages = c->page_table ? c->max_pages : 0;
  v.num_pages = c->page_table ? c->num_pages : 0;
  v.cap = (int)cap;
  v.block_stride = st[0] * esz;
  v.head_stride = st[1] * esz;
  v.row_stride = st[2] * esz;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.scores = c->scores;
  v.scores_ld = c->scores ? c->scores_ld : 0;
  *out = v;
  return TR_OK;
}

// The first kernel of an append (tr_kv.cu): the checks of all sequences and their new
// lengths; the rows that each takes go to todo[b] = (old length, rows).
int kv_append_plan(const KvDev &c, int T, const int32_t *count, int2 *todo, cudaStream_t s);
