// Upkeep of the paged K/V cache: writing the keys and values of new tokens, and cutting a
// cache to a budget of keys by accumulated attention weight.  Bound by HBM (and by launch
// latency for small calls): every row moves once, 16 bytes a lane.  Append of 4 x 2048 tokens
// x 4 kv-heads, d = 128 9 us (3 TB/s), of 32 tokens 4.4 us; 16 caches of 16384 to 32768 keys x 4
// kv-heads cut to 4096 keys 78 us (31 us of them the selection, one CTA a (cache, kv-head),
// bound by the counting passes over shared memory; 3.5 TB/s in all).
#include <algorithm>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

// ---------------------------------------------------------------------------- append
// New token i of a sequence with L cached tokens (Lq of them new) goes to position
// L - Lq + i.  One thread a 16-byte piece of K or V.
__global__ void __launch_bounds__(256) append_kernel(Seqs s, Keys c, const uint4* __restrict__ k_new,
                                                     const uint4* __restrict__ v_new, __nv_bfloat16* k_pages,
                                                     __nv_bfloat16* v_pages, float* weights, int hkv, int d) {
  const int per = hkv * d / 8;  // pieces of a token's K
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tok = e / (2 * per);
  if (tok >= s.tokens) return;
  const int which = (int)(e / per & 1), ch = (int)(e % per);
  const int seq = seq_of_token(s, tok);
  const int64_t i = tok - seq_start(s, seq);
  const int Lq = seq_len(s, seq);
  if (i < 0 || i >= Lq) return;  // a row of no sequence
  const int64_t cap = (int64_t)c.max_pages << c.page_log2, pos = (int64_t)c.lens[seq] - Lq + i;
  if (pos < 0 || pos >= cap) return;
  const int pid = page_of(c, seq, (int)pos);
  if (pid < 0) return;
  const int slot = (int)pos & ((1 << c.page_log2) - 1);
  __nv_bfloat16* dst = (which ? v_pages : k_pages) + pid * c.page_stride + (int64_t)slot * hkv * d;
  reinterpret_cast<uint4*>(dst)[ch] = (which ? v_new : k_new)[tok * per + ch];
  if (weights && !which && ch < hkv) weights[(((int64_t)pid * hkv + ch) << c.page_log2) + slot] = 0.f;
}

// ---------------------------------------------------------------------------- evict
constexpr int kSelThreads = 1024;
constexpr int kSelCached = 49152;  // keys whose ranks shared memory holds (192 KB)
// Copies of the histogram: a warp's lanes count into the copy of their lane % 4, since many
// keys share a digit (weights within a few octaves, or zeros) and counts of one address are
// taken one after another.
constexpr int kCopies = 4, kHistBytes = 2048 * kCopies * 4;

// Order of a weight as an unsigned key: larger weights have larger keys, -0 equals +0, NaN
// (and a key in a missing page) is the lowest.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The `budget` keys of one (sequence, kv-head) that stay, ascending: the first n_sink, the
// last n_recent, and the best of the others by weight (equal weights: the lower index).
// A radix selection on 11, 11 and 10 bits (three counting passes, the first while the
// weights are read; 43 us for 64 caches of 16384 to 32768 keys with four passes of 8 bits)
// finds the rank of the last key that stays and how many keys of exactly that rank do; then
// every warp takes a contiguous run of keys, counts what it keeps, and after one scan over
// the warps writes its run in order.  Counting in shared-memory integers, so the result is
// the same on every run.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(Keys c, const float* __restrict__ weights, int hkv,
                                                                   int budget, int n_sink, int n_recent, int room,
                                                                   int32_t* __restrict__ keep) {
  extern __shared__ int s_hist[];  // [2048][kCopies], then the ranks
  launch_dependents();
  __shared__ int s_gt[32], s_eq[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int seq = blockIdx.x, g = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* s_rank = reinterpret_cast<uint32_t*>(s_hist + 2048 * kCopies);
  const int L = cached_len(c, seq);
  int32_t* out = keep + ((int64_t)seq * hkv + g) * budget;
  if (L <= budget) {  // everything stays
    for (int i = tid; i < budget; i += kSelThreads) out[i] = i < L ? i : -1;
    return;
  }
  const int page = 1 << c.page_log2;
  const bool cached = L <= room;  // the ranks fit the launch's shared memory
  // (no branches: the loads of several keys have to be in flight together)
  auto place = [&](int i) -> int64_t {  // of key i's weight (-1: in no page)
    const int pid = page_of(c, seq, i);
    return pid < 0 ? -1 : (((int64_t)pid * hkv + g) << c.page_log2) + (i & (page - 1));
  };
  auto order = [&](int i, int64_t at, float w) -> uint32_t {
    const uint32_t r = at < 0 ? 0u : rank_of(w);
    return i < n_sink || i >= L - n_recent ? 0xffffffffu : r;  // above +inf
  };
  auto rank = [&](int i) -> uint32_t {
    const int64_t at = place(i);
    return order(i, at, __ldg(weights + (at < 0 ? 0 : at)));
  };
  auto get = [&](int i) { return cached ? s_rank[i] : rank(i); };
  uint32_t prefix = 0;
  int left = budget;  // keys still to take among those that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass < 2 ? 2048 : 1024;
#pragma unroll
    for (int i = 0; i < 2048 * kCopies / kSelThreads; ++i) s_hist[tid + i * kSelThreads] = 0;
    __syncthreads();
    if (pass == 0) {
      constexpr int U = 8;  // weights in flight a thread
      for (int b = 0; b < L; b += U * kSelThreads) {
        int64_t at[U];
        uint32_t r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) at[u] = place(min(b + u * kSelThreads + tid, L - 1));
#pragma unroll
        for (int u = 0; u < U; ++u)
          r[u] = order(b + u * kSelThreads + tid, at[u], __ldg(weights + (at[u] < 0 ? 0 : at[u])));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = b + u * kSelThreads + tid;
          if (i < L) {
            if (cached) s_rank[i] = r[u];
            atomicAdd(&s_hist[(r[u] >> 21) * kCopies + lane % kCopies], 1);
          }
        }
      }
    } else {
      const uint32_t mask = pass == 1 ? 0xffe00000u : 0xfffffc00u;
#pragma unroll 8
      for (int i = tid; i < L; i += kSelThreads) {
        const uint32_t r = get(i);
        if ((r & mask) == prefix) atomicAdd(&s_hist[((r >> shift) & (digits - 1)) * kCopies + lane % kCopies], 1);
      }
    }
    __syncthreads();
    // the digit of the last key that stays, from the top: thread tid has digits 2047 - 2 tid
    // and 2046 - 2 tid
    const int d0 = 2047 - 2 * tid;
    const int4 c0 = reinterpret_cast<const int4*>(s_hist)[d0], c1 = reinterpret_cast<const int4*>(s_hist)[d0 - 1];
    const int h0 = c0.x + c0.y + c0.z + c0.w, sum = h0 + c1.x + c1.y + c1.z + c1.w;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_gt[warp] = incl;
    __syncthreads();
    const int others = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
    const int before = others + incl - sum;
    if (before < left && before + sum >= left) {
      const bool second = before + h0 < left;
      s_prefix = prefix | ((uint32_t)(d0 - second) << shift);
      s_left = left - before - (second ? h0 : 0);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // keys of rank > prefix stay, and the first `left` of rank == prefix
  const int run = (L + 31) / 32, i0 = min(L, warp * run), i1 = min(L, i0 + run);
  int gt = 0, eq = 0;
#pragma unroll 8
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t r = get(i);
    gt += r > prefix;
    eq += r == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int at = 0, ties = 0;
  for (int w = 0; w < warp; ++w) {
    at += s_gt[w] + min(s_eq[w], max(0, left - ties));
    ties += s_eq[w];
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    const uint32_t r = i < i1 ? get(i) : 0u;
    uint32_t stay = __ballot_sync(0xffffffffu, i < i1 && r > prefix);
    const uint32_t tie = __ballot_sync(0xffffffffu, i < i1 && r == prefix);
    if (tie && ties < left) {  // the first left - ties of them
      const int room_left = left - ties;
      const bool in = ((tie >> lane) & 1u) && __popc(tie & below) < room_left;
      stay |= __ballot_sync(0xffffffffu, in);
    }
    if ((stay >> lane) & 1u) out[at + __popc(stay & below)] = i;
    at += __popc(stay);
    ties += __popc(tie);
  }
}

// Row keep[i] of a (sequence, kv-head) to position i of the new table's pages: K, V and
// weight.  A half-warp (d = 128) or quarter-warp (d = 64) moves a row of K and of V.
template <int D>
__global__ void __launch_bounds__(256) evict_copy_kernel(Keys c, Keys to, __nv_bfloat16* k_pages,
                                                         __nv_bfloat16* v_pages, float* weights, int hkv, int budget,
                                                         const int32_t* __restrict__ keep, int32_t* new_lens) {
  constexpr int CH = D / 8, PER = 256 / CH;  // lanes a row, rows a block
  const int seq = blockIdx.z, g = blockIdx.y;
  const int32_t* list = keep + ((int64_t)seq * hkv + g) * budget;
  const int i = blockIdx.x * PER + threadIdx.x / CH, ch = threadIdx.x % CH;
  const int64_t cap = (int64_t)to.max_pages << to.page_log2;
  wait_primary();
  if (i >= budget) return;
  const int src = list[i];
  // the kept count of head 0 (the same for every head): the list is filled from the front
  if (g == 0 && ch == 0 && new_lens) {
    if (src >= 0 && (i + 1 == budget || list[i + 1] < 0)) new_lens[seq] = i + 1;
    if (i == 0 && src < 0) new_lens[seq] = 0;
  }
  if (src < 0 || i >= cap) return;
  const int pd = page_of(to, seq, i);
  if (pd < 0) return;
  const int page = 1 << c.page_log2, ss = src & (page - 1), ds = i & (page - 1);
  const int ps = page_of(c, seq, src);
  uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
  float w = 0.f;
  if (ps >= 0) {  // (a row of a missing page is copied as zeros)
    const int64_t from = ps * c.page_stride + ((int64_t)ss * hkv + g) * D + ch * 8;
    kx = *reinterpret_cast<const uint4*>(k_pages + from);
    vx = *reinterpret_cast<const uint4*>(v_pages + from);
    if (ch == 0) w = weights[(((int64_t)ps * hkv + g) << c.page_log2) + ss];
  }
  const int64_t dst = pd * c.page_stride + ((int64_t)ds * hkv + g) * D + ch * 8;
  *reinterpret_cast<uint4*>(k_pages + dst) = kx;
  *reinterpret_cast<uint4*>(v_pages + dst) = vx;
  if (ch == 0) weights[(((int64_t)pd * hkv + g) << c.page_log2) + ds] = w;
}

}  // namespace span

cudaError_t launch_paged_append(const Seqs& s, const void* k_new, const void* v_new, const PagedView& cache,
                                void* k_pages, void* v_pages, float* weights, int hkv, int d, cudaStream_t st) {
  const int64_t n = s.tokens * 2 * (hkv * d / 8);
  if (n == 0 || s.n_seqs == 0) return cudaSuccess;
  span::append_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(
      s, span::keys_of(&cache, nullptr, nullptr), (const uint4*)k_new, (const uint4*)v_new, (__nv_bfloat16*)k_pages,
      (__nv_bfloat16*)v_pages, weights, hkv, d);
  return cudaGetLastError();
}

cudaError_t launch_paged_evict(int n_seqs, const PagedView& cache, const PagedView& to, void* k_pages,
                               void* v_pages, float* weights, int hkv, int d, int budget, int n_sink, int n_recent,
                               int32_t* keep, int32_t* new_lens, cudaStream_t st) {
  if (n_seqs == 0) return cudaSuccess;
  const span::Keys c = span::keys_of(&cache, k_pages, v_pages), t = span::keys_of(&to, k_pages, v_pages);
  const int room = (int)std::min<int64_t>(span::kSelCached, (int64_t)cache.max_pages << cache.page_log2);
  cudaError_t e = cudaFuncSetAttribute(span::evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       span::kSelCached * 4 + span::kHistBytes);
  if (e != cudaSuccess) return e;
  span::evict_select_kernel<<<dim3(n_seqs, hkv), span::kSelThreads, span::kHistBytes + room * 4, st>>>(c, weights, hkv, budget, n_sink,
                                                                                   n_recent, room, keep);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int per = 256 / (d / 8);
  const dim3 grid((budget + per - 1) / per, hkv, n_seqs);
  return span::launch_second(d == 64 ? span::evict_copy_kernel<64> : span::evict_copy_kernel<128>, grid, 256, 0, st, c, t,
                             (__nv_bfloat16*)k_pages, (__nv_bfloat16*)v_pages, weights, hkv, budget, keep, new_lens);
}

}  // namespace nsa
