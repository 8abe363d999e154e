// Accumulated attention weights of cached keys, the input of eviction by weight: for key j
// of kv-head g, sum over the chunk's queries i that see j and the group's heads of
// exp(scale q_i.k_j - lse_i), with the lse of the attention call on the same inputs, added
// to decay times the weight so far.
//
// Every key's sum stays in one thread's fp32 registers: no atomics, the same result on every
// run, K read once (FEW reads all cached keys, seen or not: under a window that is many times what
// its queries see).  The product is taken transposed, S^T = K Q^T (M = 128 keys, N = the
// tile's rows), so that a TMEM lane is a key and the sum over queries needs no exchange
// between threads.  One operand of a CTA stays and the other streams through a ring:
//   many rows   128 keys stay, the query tiles that see them stream.  Four groups of summing
//               warps take the tiles in turn, each with an S buffer of its own, and add their
//               sums at the end (one group and two CTAs an SM took 1.2 times as long).  An
//               exponential per product of 128 terms: the exponential unit and the tensor
//               cores, both at 40%, and the issue of the sums at 35% bound it together:
//               2 x 1000 queries x 16 heads over caches of 14746 to 16384 keys 140 us
//               (840 TFLOP/s).
//   FEW         (a sequence's rows fit one tile of 48) the queries stay and a run of key
//               tiles streams: bound by HBM; one group, two CTAs an SM.  32 tokens over
//               caches of 16384 to 32768 keys x 2 kv-heads 74 us (5.6 TB/s, 83% of a copy).
// Roles: groups of four warps sum (one key a thread), then a warp that loads and one that
// issues the products.
#include <algorithm>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

struct WeightParams {
  Seqs seqs;
  Keys keys;
  const float* lse;
  const float* w_in;  // optional
  float* w_out;
  int h, hkv, R, tpc, cols, window, n_sink;  // cols: columns of a full query tile, up to a multiple of 16
  int q_group, n_splits;                     // bytes between Q's 64-column groups; FEW: CTAs of a (sequence, kv-head)
  uint32_t tmem_cols, buf_cols;
  float scale_log2, decay;
};

template <int D, bool FEW>
struct WCfg {
  static constexpr int K_BYTES = KT * D * 2;
  static constexpr int NS = FEW ? (D == 64 ? 6 : 3) : 4;  // slots of the streamed operand
  static constexpr int NG = FEW ? 1 : 4;                  // groups of summing warps
  static constexpr int NB = FEW ? 2 : 4;                  // S buffers: item i in i % NB, summed by group i % NG
  static constexpr int THREADS = (4 * NG + 2) * 32;
  // TMEM columns of an S buffer for query tiles of `cols` columns, of all of them (powers of two)
  static constexpr int buf_cols(int cols) { return cols <= 32 ? 32 : cols <= 64 ? 64 : 128; }
  // Shared memory of a launch, so much that no more CTAs come onto an SM than its 512 TMEM columns
  // serve (228 KB, 1 KB of it per CTA reserved); and of the largest.
  static constexpr int smem(int cols) {
    const int q = (D / 64) * cols * 128, own = (FEW ? q + NS * K_BYTES : K_BYTES + NS * q) + 1024;
    const int least = 228 * 1024 / (512 / (NB * buf_cols(cols)) + 1) - 1024 + 16;
    return own > least ? own : least;
  }
  static constexpr int max_smem() {
    int most = 0;
    for (int c = GRAN; c <= ROWS; c += GRAN) most = smem(c) > most ? smem(c) : most;
    return most;
  }
};

template <int D, bool FEW>
__global__ void __launch_bounds__(WCfg<D, FEW>::THREADS, FEW ? 2 : 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_k16, const WeightParams p) {
  using C = WCfg<D, FEW>;
  constexpr int NS = C::NS, NG = C::NG, NB = C::NB, kLoad = 4 * NG, kIssue = kLoad + 1;
  enum : int { FIXED = 0, FULL = 1, EMPTY = FULL + NS, SFULL = EMPTY + NS, SFREE = SFULL + NB, DRAIN = SFREE + NB, COUNT };
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[COUNT];
  __shared__ __align__(16) float s_lse[4 * NG][ROWS];  // by summing warp: minus the base-2 lse of its tile's rows
  __shared__ float s_sum[NG][ROWS];                    // the groups' sums (many rows)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t q_bytes = (D / 64) * p.q_group, slot_bytes = FEW ? C::K_BYTES : q_bytes;
  const uint32_t fixed_s = base, ring_s = fixed_s + (FEW ? q_bytes : C::K_BYTES);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  if (stopped()) return;
  const Waits wait(abort);
  const int seq = blockIdx.y, g = blockIdx.z;
  const int kv_len = cached_len(p.keys, seq);
  const int64_t start = seq_start(p.seqs, seq);
  const int Lq = seq_len(p.seqs, seq);
  const int off = kv_len - Lq;
  // this CTA's key tiles, and (many rows) the queries [t_lo, t_hi) that see some key of its one
  const int n_kt = (kv_len + KT - 1) / KT;
  const int kt0 = FEW ? (int)((int64_t)n_kt * blockIdx.x / p.n_splits) : (int)blockIdx.x;
  const int kt1 = FEW ? (int)((int64_t)n_kt * (blockIdx.x + 1) / p.n_splits) : kt0 + 1;
  if (kt0 >= min(kt1, n_kt)) return;
  const int fkey0 = kt0 * KT;
  const int t_lo = FEW ? 0 : max(0, fkey0 - off);
  const int t_hi = !FEW && p.window > 0 && fkey0 >= p.n_sink ? min(Lq, fkey0 + KT - 1 + p.window - off) : Lq;  // (sums below 2^31: every size is at most 2^28)
  const int n_q = t_hi > t_lo ? (t_hi - t_lo + p.tpc - 1) / p.tpc : 0;
  const int n = FEW ? kt1 - kt0 : n_q;  // streamed items
  const bool any = n_q > 0;             // without queries nothing is loaded

  if (tid == 0) {
    tc::mbar_init(bar(FIXED), 1);
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(bar(FULL + i), 1);
      tc::mbar_init(bar(EMPTY + i), 1);
    }
    for (int i = 0; i < NB; ++i) {
      tc::mbar_init(bar(SFULL + i), 1);
      tc::mbar_init(bar(SFREE + i), 4);  // one arrival a summing warp
    }
    tc::mbar_init(bar(DRAIN), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  auto place = [&](int key) -> int64_t {  // of the key's weight, or -1 (no key, or in no page)
    if (key >= kv_len) return -1;
    const int pid = page_of(p.keys, seq, key);
    return pid < 0 ? -1 : (((int64_t)pid * p.hkv + g) << p.keys.page_log2) + (key & ((1 << p.keys.page_log2) - 1));
  };
  auto finish = [&](float sum, float before, int64_t at) {
    if (at >= 0) p.w_out[at] = p.w_in ? fmaf(p.decay, before, sum) : sum;
  };
  if (warp == kIssue) {
    tmem_alloc(smem_u32(&s_tmem), p.tmem_cols);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_item = -1;
  if (warp == kLoad) {
    // ------------------------------------------------------------------ loads
    auto load_q = [&](uint32_t to, int t, uint32_t full) {
      if (lane == 0) {
        tc::mbar_expect_tx(full, (uint32_t)(p.tpc * p.R * D * 2));
        for (int c = 0; c < D / 64; ++c)
          tc::tma3d(to + c * p.q_group, &tm_q, c * 64, g * p.R, (int)(start + t), full);
      }
      __syncwarp();
    };
    auto load_k = [&](uint32_t to, int key0, uint32_t full) {
      load_tile<D, true>(to, &tm_k, &tm_k16, p.keys.k, p.keys, p.hkv, g, seq, start, key0, 0, 0,
                         min(KT, up16(kv_len - key0)), kv_len, full, lane);
    };
    if (any && FEW) load_q(fixed_s, 0, bar(FIXED));
    if (any && !FEW) load_k(fixed_s, fkey0, bar(FIXED));
    int slot = 0;
    uint32_t phase = 1;
    for (int i = 0; any && i < n; ++i) {
      if (i >= NS && !wait(bar(EMPTY + slot), phase)) break;
      if (FEW) {
        load_k(ring_s + slot * slot_bytes, (kt0 + i) * KT, bar(FULL + slot));
      } else {
        load_q(ring_s + slot * slot_bytes, t_lo + i * p.tpc, bar(FULL + slot));
      }
      last_item = i;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------------------ products
    bool ok = !any || wait(bar(FIXED), 0);
    const uint32_t lead = elect(), id = tc::idesc(KT, p.cols), fixed_d = desc_k(fixed_s), ring_d = desc_k(ring_s);
    int slot = 0;
    uint32_t phase = 0;
    for (int i = 0; ok && any && i < n; ++i) {
      const int b = i % NB;
      if (i >= NB && !(ok = wait(bar(SFREE + b), (i / NB - 1) & 1))) break;
      if (!(ok = wait(bar(FULL + slot), phase))) break;
      tc::fence_after();
      const uint32_t at = ring_d + slot * (slot_bytes >> 4);
      const uint32_t kd = FEW ? at : fixed_d, qd = FEW ? fixed_d : at, qg = p.q_group >> 4;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        mma_ss(tmem + b * p.buf_cols, kd + (s >> 2) * (KT * 128 >> 4) + (s & 3) * 2, qd + (s >> 2) * qg + (s & 3) * 2,
               id, s > 0, lead);
      commit(bar(SFULL + b), lead);
      commit(bar(EMPTY + slot), lead);
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------------ sums, one key a thread
    const int row = tid & 127;  // the thread's key of a tile
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
    float acc = 0.f;
    bool ok = true;
    // minus the base-2 lse of a query tile's rows (-inf for a row of no query or without keys,
    // so that it adds 0), four a lane, fetched a turn of the group ahead
    float nl[ROWS / 32];
    int tok[ROWS / 32], ofs[ROWS / 32];
#pragma unroll
    for (int e = 0; e < ROWS / 32; ++e) {
      const int r = lane + e * 32;
      tok[e] = r < p.tpc * p.R ? r / p.R : 1 << 30;
      ofs[e] = r / p.R * p.h + r % p.R;
    }
    auto fetch = [&](int i) {
      const int t = FEW ? 0 : t_lo + i * p.tpc;
      const float* src = p.lse + (start + t) * p.h + g * p.R;
#pragma unroll
      for (int e = 0; e < ROWS / 32; ++e) nl[e] = any && i < n && tok[e] < Lq - t ? __ldg(src + ofs[e]) : kNegInf;
    };
    fetch(warp >> 2);
    for (int i = warp >> 2; i < n; i += NG) {
      const int b = i % NB, key = FEW ? (kt0 + i) * KT + row : fkey0 + row, t = FEW ? 0 : t_lo + i * p.tpc;
      int64_t at = -1;
      float before = 0.f;
      if (FEW) {  // (read ahead of the product)
        at = place(key);
        if (at >= 0 && p.w_in) before = p.w_in[at];
        acc = 0.f;
      }
      if (any) {
        // columns [c_lo, c_hi) are rows whose query sees this key
        const int64_t first = (int64_t)(key - off - t) * p.R;
        int64_t end = (int64_t)min(p.tpc, Lq - t) * p.R;
        if (p.window > 0 && key >= p.n_sink) end = min(end, ((int64_t)key + p.window - off - t) * p.R);
        const int c_lo = (int)max((int64_t)0, min(first, (int64_t)ROWS));
        const int c_hi = key < kv_len ? (int)max((int64_t)0, end) : 0;
        float* lse = s_lse[warp];
        if (!FEW || i == 0) {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < ROWS / 32; ++e) lse[lane + e * 32] = nl[e] > kNegInf ? -nl[e] * kLog2e : kNegInf;
          __syncwarp();
          if (!FEW) fetch(i + NG);
        }
        if (!(ok = wait(bar(SFULL + b), (i / NB) & 1))) break;
        tc::fence_after();
        uint64_t a2[4] = {0, 0, 0, 0};
        const uint32_t s_t = t_lane + b * p.buf_cols;
        // (a tile whose every column is seen goes without masks, in code of its own: joined, the
        // two ways would meet in copies of the scores)
        auto sum = [&](auto full, float (&sv)[32], int c) {
          const float4* l4 = reinterpret_cast<const float4*>(lse + c);
          if constexpr (!decltype(full)::value) {
            const uint32_t see = bits(c_lo - c, c_hi - c);
            // (a column of no query holds whatever lies past the tile's rows)
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[e] = (see >> e) & 1u ? sv[e] : kNegInf;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l = l4[e / 4];
            const float2 y = unpair(fma2(pair(sv[e], sv[e + 1]), scale2, pair(l.x, l.y)));
            const float2 z = unpair(fma2(pair(sv[e + 2], sv[e + 3]), scale2, pair(l.z, l.w)));
            a2[(e >> 1) & 3] = add2(a2[(e >> 1) & 3], pair(ex2(y.x), ex2(y.y)));
            a2[((e >> 1) + 1) & 3] = add2(a2[((e >> 1) + 1) & 3], pair(ex2(z.x), ex2(z.y)));
          }
        };
        auto release = [&]() {  // the buffer's scores are in registers
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(SFREE + b));
        };
        // 32 columns at a time, the next ones on their way while these are summed
        float sa[32], sb[32];
        tc::tmem_ld32_nowait(s_t, sa);
        tmem_wait_ld(sa);
        if (!FEW && __all_sync(0xffffffffu, c_lo == 0 && c_hi >= ROWS)) {
          constexpr std::true_type full{};
          tc::tmem_ld32_nowait(s_t + 32, sb);
          sum(full, sa, 0);
          tmem_wait_ld(sb);
          tc::tmem_ld32_nowait(s_t + 64, sa);
          sum(full, sb, 32);
          tmem_wait_ld(sa);
          tc::tmem_ld32_nowait(s_t + 96, sb);
          sum(full, sa, 64);
          tmem_wait_ld(sb);
          release();
          sum(full, sb, 96);
        } else {
          constexpr std::false_type full{};
          sum(full, sa, 0);
#pragma unroll 1
          for (int c = 32; c < p.cols; c += 32) {
            tc::tmem_ld32_nowait(s_t + c, sa);
            tmem_wait_ld(sa);
            sum(full, sa, c);
          }
          release();
        }
        const float2 s2 = unpair(add2(add2(a2[0], a2[1]), add2(a2[2], a2[3])));
        acc += s2.x + s2.y;
      }
      if (FEW) finish(acc, before, at);
    }
    s_sum[warp >> 2][row] = acc;
  }

  __syncthreads();
  if (!FEW && tid < ROWS && !*abort) {
    const int64_t at = place(fkey0 + tid);
    float sum = s_sum[0][tid];
#pragma unroll
    for (int i = 1; i < NG; ++i) sum += s_sum[i][tid];
    finish(sum, at >= 0 && p.w_in ? p.w_in[at] : 0.f, at);
  }
  if (*abort) {
    // copies and products still in flight land before the CTA leaves
    if (warp == kLoad) {
      if (any) tc::warp_drain(bar(FIXED), 0);
      for (int st = 0; st < NS; ++st)
        if (last_item >= st) tc::warp_drain(bar(FULL + st), ((last_item - st) / NS) & 1);
    } else if (warp == kIssue) {
      commit(bar(DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(DRAIN), 0);
    }
  } else if (warp == kLoad) {
    for (int st = 0; st < NS; ++st)
      if (last_item >= st) tc::warp_drain(bar(EMPTY + st), ((last_item - st) / NS) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_free(tmem, p.tmem_cols);
}

template <int D, bool FEW>
cudaError_t launch_weights_d(WeightParams& p, const void* q, cudaStream_t st) {
  using C = WCfg<D, FEW>;
  p.cols = up16(p.tpc * p.R);
  p.q_group = p.cols * 128;
  p.buf_cols = C::buf_cols(p.cols);
  p.tmem_cols = C::NB * p.buf_cols;
  CUtensorMap mq, mk, mk16;
  // (a map needs rows; without queries none is ever loaded)
  const bool any = p.seqs.tokens > 0;
  if (!query_map(&mq, any ? q : p.keys.k, any ? p.seqs.tokens : 1, p.h, D, p.R, p.tpc) ||
      !key_maps(&mk, &mk16, p.keys.k, p.keys, p.hkv, D, 0))
    return cudaErrorInvalidValue;
  auto kern = weights_kernel<D, FEW>;
  // (the limit belongs to the kernel, and other threads launch it too: the same for every call)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::max_smem());
  if (e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)p.keys.max_pages << p.keys.page_log2) + KT - 1) / KT;
  const int64_t units = (int64_t)p.seqs.n_seqs * p.hkv;
  // FEW: at most three rounds of two CTAs an SM, so that ragged caches even out
  p.n_splits = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, 3 * 2 * 152 / units));
  const dim3 grid((unsigned)(FEW ? p.n_splits : tiles), p.seqs.n_seqs, p.hkv);
  kern<<<grid, C::THREADS, C::smem(p.cols), st>>>(mq, mk, mk16, p);
  return cudaGetLastError();
}

}  // namespace span

cudaError_t launch_span_weights(const Seqs& s, const void* q, const PagedView& cache, const void* k, int h, int hkv,
                                int d, int window, int n_sink, float scale, float decay,
                                const float* lse, const float* w_in, float* w_out, cudaStream_t st) {
  if (s.n_seqs == 0) return cudaSuccess;
  span::WeightParams p{};
  p.seqs = s;
  p.keys = span::keys_of(&cache, k, nullptr);
  p.lse = lse;
  p.w_in = w_in;
  p.w_out = w_out;
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.tpc = std::max(1, std::min(span::ROWS / p.R, s.max_len));
  p.window = window;
  p.n_sink = n_sink;
  p.scale_log2 = scale * kLog2e;
  p.decay = decay;
  // a sequence's queries fit one tile of at most 48 rows (what leaves room for two CTAs an SM)
  if ((int64_t)s.max_len * p.R <= 48)
    return d == 64 ? span::launch_weights_d<64, true>(p, q, st) : span::launch_weights_d<128, true>(p, q, st);
  return d == 64 ? span::launch_weights_d<64, false>(p, q, st) : span::launch_weights_d<128, false>(p, q, st);
}

NSA_STATUS_ACCESSOR(span_weights)

}  // namespace nsa
