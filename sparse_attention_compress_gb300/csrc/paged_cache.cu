// Upkeep of the paged K/V cache: writing the keys and values of new tokens, and cutting a
// cache to a budget of keys by accumulated attention weight.  Bound by HBM (and by launch
// latency for small calls): every row moves once, 16 bytes a lane.  Times on the device (a call from
// Python takes 12 us and more on the host): append of 4 x 2048 tokens
// x 4 kv-heads, d = 128 9 us (3 TB/s), of 32 tokens 4.4 us; 16 caches of 16384 to 32768 keys x 4
// kv-heads cut to 4096 keys 70 us (25 us of them the selection, one CTA a (cache, kv-head),
// bound by its instructions on 64 of 152 SMs; the copy runs at 6 TB/s).
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
// weights are read; 43 us for 64 caches of 16384 to 32768 keys with four passes of 8 bits, 33
// a key at a time, 25 with four consecutive keys a lane)
// finds the rank of the last key that stays and how many keys of exactly that rank do; then
// every warp takes a contiguous run of keys, counts what it keeps, and after one scan over
// the warps writes its run in order.  Counting in shared-memory integers, so the result is
// the same on every run.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(Keys c, const float* __restrict__ weights, int hkv,
                                                                   int budget, int n_sink, int n_recent, int room,
                                                                   bool vec, int32_t* __restrict__ keep) {
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
  // weights of keys i .. i + 3 (i a multiple of 4: a page holds all four, be they keys or not)
  auto load4 = [&](int64_t at) -> float4 {
    const float* src = weights + (at < 0 ? 0 : at);
    return vec ? __ldg(reinterpret_cast<const float4*>(src))
               : make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
  };
  auto order4 = [&](int i, int64_t at, float4 w) {
    return make_uint4(order(i, at, w.x), order(i + 1, at, w.y), order(i + 2, at, w.z), order(i + 3, at, w.w));
  };
  auto get4 = [&](int i) -> uint4 {
    if (cached) return *reinterpret_cast<const uint4*>(s_rank + i);
    const int64_t at = place(i);
    return order4(i, at, load4(at));
  };
  uint32_t prefix = 0;
  int left = budget;  // keys still to take among those that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass < 2 ? 2048 : 1024;
#pragma unroll
    for (int i = 0; i < 2048 * kCopies / kSelThreads; ++i) s_hist[tid + i * kSelThreads] = 0;
    __syncthreads();
    if (pass == 0) {
      constexpr int U = 4;  // loads in flight a thread
      for (int b = 0; b < L; b += U * 4 * kSelThreads) {
        int64_t at[U];
        float4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) at[u] = place(min(b + (u * kSelThreads + tid) * 4, (L - 1) & ~3));
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load4(at[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = b + (u * kSelThreads + tid) * 4;
          if (i < L) {
            const uint4 r = order4(i, at[u], w[u]);
            if (cached) *reinterpret_cast<uint4*>(s_rank + i) = r;
            const uint32_t re[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (i + e < L) atomicAdd(&s_hist[(re[e] >> 21) * kCopies + lane % kCopies], 1);
          }
        }
      }
    } else {
      const uint32_t mask = pass == 1 ? 0xffe00000u : 0xfffffc00u;
#pragma unroll 4
      for (int i = tid * 4; i < L; i += 4 * kSelThreads) {
        const uint4 r = get4(i);
        const uint32_t re[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((re[e] & mask) == prefix && i + e < L)
            atomicAdd(&s_hist[((re[e] >> shift) & (digits - 1)) * kCopies + lane % kCopies], 1);
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
  const int run = ((L + 31) / 32 + 3) & ~3, i0 = min(L, warp * run), i1 = min(L, i0 + run);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = i0 + lane * 4; i < i1; i += 128) {
    const uint4 r = get4(i);
    const uint32_t re[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += i + e < i1 && re[e] > prefix;
      eq += i + e < i1 && re[e] == prefix;
    }
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
#pragma unroll 2
  for (int b = i0; b < i1; b += 128) {
    const int i = b + lane * 4;
    const uint4 r = i < i1 ? get4(i) : make_uint4(0, 0, 0, 0);
    const uint32_t re[4] = {r.x, r.y, r.z, r.w};
    uint32_t stay[4], tie[4];  // by key of a lane: a bit a lane
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      stay[e] = __ballot_sync(0xffffffffu, i + e < i1 && re[e] > prefix);
      tie[e] = __ballot_sync(0xffffffffu, i + e < i1 && re[e] == prefix);
    }
    const int n_ties = __popc(tie[0]) + __popc(tie[1]) + __popc(tie[2]) + __popc(tie[3]);
    if (n_ties && ties < left) {  // the first left - ties of them
      int before = ties + __popc(tie[0] & below) + __popc(tie[1] & below) + __popc(tie[2] & below) + __popc(tie[3] & below);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is = (tie[e] >> lane) & 1u;
        stay[e] |= __ballot_sync(0xffffffffu, is && before < left);
        before += is;
      }
    }
    int to = at + __popc(stay[0] & below) + __popc(stay[1] & below) + __popc(stay[2] & below) + __popc(stay[3] & below);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((stay[e] >> lane) & 1u) out[to++] = i + e;
    at += __popc(stay[0]) + __popc(stay[1]) + __popc(stay[2]) + __popc(stay[3]);
    ties += n_ties;
  }
}

// Row keep[i] of a (sequence, kv-head) to position i of the new table's pages: K, V and
// weight.  A half-warp (d = 128) or quarter-warp (d = 64) moves a row of K and of V.  (keep is
// written while this kernel starts: no read-only loads of it.)
template <int D>
__global__ void __launch_bounds__(256) evict_copy_kernel(Keys c, Keys to, __nv_bfloat16* k_pages,
                                                         __nv_bfloat16* v_pages, float* weights, int hkv, int budget,
                                                         const int32_t* keep, int32_t* new_lens) {
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
  const bool vec = (reinterpret_cast<uintptr_t>(weights) & 15u) == 0;
  cudaError_t e = cudaFuncSetAttribute(span::evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       span::kSelCached * 4 + span::kHistBytes);
  if (e != cudaSuccess) return e;
  span::evict_select_kernel<<<dim3(n_seqs, hkv), span::kSelThreads, span::kHistBytes + room * 4, st>>>(
      c, weights, hkv, budget, n_sink, n_recent, room, vec, keep);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int per = 256 / (d / 8);
  const dim3 grid((budget + per - 1) / per, hkv, n_seqs);
  return span::launch_second(d == 64 ? span::evict_copy_kernel<64> : span::evict_copy_kernel<128>, grid, 256, 0, st, c, t,
                             (__nv_bfloat16*)k_pages, (__nv_bfloat16*)v_pages, weights, hkv, budget, keep, new_lens);
}

}  // namespace nsa
