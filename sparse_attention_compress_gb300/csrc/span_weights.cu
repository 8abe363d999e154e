// Accumulated attention weights of cached keys, the input of eviction by weight: for key j
// of kv-head g, sum over the chunk's queries i that see j and the group's heads of
// exp(scale q_i.k_j - lse_i), with the lse of the attention call on the same inputs, added
// to decay times the weight so far.
//
// One CTA owns 128 keys and walks the query tiles that see them, so every key's sum stays
// in one thread's fp32 registers: no atomics, the same result on every run, K read once.
// The product is taken transposed, S^T = K Q^T (M = 128 keys, N = the tile's rows), so that
// a TMEM lane is a key and the sum over queries needs no exchange between threads.  Roles:
// warps 0-3 sum (one key a thread), warp 4 loads, warp 5 issues.  A decode step has few
// columns: its Q stages and TMEM buffers are sized to them, so that up to five CTAs share
// an SM and their loads overlap.
#include <algorithm>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

constexpr int kWThreads = 192;
constexpr int kWStages = 2;

struct WeightParams {
  Seqs seqs;
  Keys keys;
  const float* lse;
  const float* w_in;  // optional
  float* w_out;
  int h, hkv, R, tpc, cols, q_bytes, window, n_sink;  // cols: columns of a full query tile, up to a multiple of 16
  uint32_t tmem_cols, buf_cols;
  float scale_log2, decay;
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 3)
    weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_k16, const WeightParams p) {
  enum : int { K = 0, QFULL = 1, QEMPTY = 3, SFULL = 5, SFREE = 7, DRAIN = 9, COUNT = 10 };
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[COUNT];
  __shared__ __align__(16) float s_lse[4][ROWS];  // by summing warp: the tile's base-2 lse
  __shared__ uint32_t s_tmem, s_bad;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t k_s = base, q_s = base + KT * D * 2;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  if (tc::device_status_set()) return;
  const int seq = blockIdx.y, g = blockIdx.z, key0 = (int)blockIdx.x * KT;
  const int kv_len = cached_len(p.keys, seq);
  if (key0 >= kv_len) return;
  const int64_t start = seq_start(p.seqs, seq);
  const int Lq = seq_len(p.seqs, seq);
  const int off = kv_len - Lq;
  const int w = min(KT, up16(kv_len - key0));
  // queries [t_lo, t_hi) see some key of the tile
  const int t_lo = max(0, key0 - off);
  const int t_hi = p.window > 0 && key0 >= p.n_sink ? min(Lq, key0 + KT - 1 + p.window - off) : Lq;
  const int n = t_hi > t_lo ? (t_hi - t_lo + p.tpc - 1) / p.tpc : 0;

  if (tid == 0) {
    tc::mbar_init(bar(K), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(QFULL + i), 1);
      tc::mbar_init(bar(QEMPTY + i), 1);
      tc::mbar_init(bar(SFULL + i), 1);
      tc::mbar_init(bar(SFREE + i), 128);
    }
    tc::mbar_init(bar(DRAIN), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&s_tmem), p.tmem_cols);
    tc::fence_before();
  }
  if (warp == 4) {
    const uint32_t bad = missing_groups(p.keys, seq, key0, w, kv_len, lane);
    if (lane == 0) s_bad = bad;
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_q = -1;
  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    if (n > 0)
      load_tile<D, true>(k_s, &tm_k, &tm_k16, p.keys.k, p.keys, p.hkv, g, seq, start, key0, w, kv_len, bar(K), lane);
    for (int j = 0; j < n; ++j) {
      const int st = j & 1;
      if (j >= 2 && !tc::warp_wait(bar(QEMPTY + st), ((j >> 1) - 1) & 1, abort)) break;
      if (lane == 0) {
        tc::mbar_expect_tx(bar(QFULL + st), (uint32_t)(p.tpc * p.R * D * 2));
        for (int c = 0; c < D / 64; ++c)
          tc::tma3d(q_s + st * p.q_bytes + c * (p.q_bytes / (D / 64)), &tm_q, c * 64, g * p.R,
                    (int)(start + t_lo + j * p.tpc), bar(QFULL + st));
      }
      __syncwarp();
      last_q = j;
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------------ products
    bool ok = n == 0 || tc::warp_wait(bar(K), 0, abort);
    for (int j = 0; ok && j < n; ++j) {
      const int st = j & 1;
      if (j >= 2 && !(ok = tc::warp_wait(bar(SFREE + st), ((j >> 1) - 1) & 1, abort))) break;
      if (!(ok = tc::warp_wait(bar(QFULL + st), (j >> 1) & 1, abort))) break;
      if (lane == 0) {
        tc::fence_after();
        const uint32_t id = tc::idesc(KT, p.cols), qh = p.q_bytes / (D / 64);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc::mma_ss(tmem + st * p.buf_cols, tc::sdesc(k_s + (s >> 2) * (KT * 128) + (s & 3) * 32),
                     tc::sdesc(q_s + st * p.q_bytes + (s >> 2) * qh + (s & 3) * 32), id, s > 0);
        tc::commit(bar(SFULL + st));
        tc::commit(bar(QEMPTY + st));
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ sums, one key a thread
    const int key = key0 + tid;
    const bool have = key < kv_len && !((s_bad >> (tid / GRAN)) & 1u);
    const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
    float acc = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int st = j & 1, t = t_lo + j * p.tpc;
      // this tile's lse, a copy for each warp (rows of no query: +inf, so that they add 0)
      __syncwarp();
#pragma unroll
      for (int e = lane; e < ROWS; e += 32) {
        float le = __builtin_inff();
        if (e < p.tpc * p.R && t + e / p.R < Lq) {
          le = p.lse[(start + t + e / p.R) * p.h + g * p.R + e % p.R];
          le = le == kNegInf ? __builtin_inff() : le * kLog2e;
        }
        s_lse[warp][e] = le;
      }
      __syncwarp();
      // columns [c_lo, c_hi) are rows whose query sees this key
      int c_lo = 0, c_hi = 0;
      if (have) {
        const int64_t first = (int64_t)(key - off - t) * p.R;
        int64_t end = (int64_t)min(p.tpc, Lq - t) * p.R;
        if (p.window > 0 && key >= p.n_sink) end = min(end, (int64_t)(key + (int64_t)p.window - off - t) * p.R);
        c_lo = first > 0 ? (int)min(first, (int64_t)ROWS) : 0;
        c_hi = end > 0 ? (int)end : 0;
      }
      if (!(ok = tc::warp_wait(bar(SFULL + st), (j >> 1) & 1, abort))) break;
      tc::fence_after();
      float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = 0; c < p.cols; c += 32) {
        float sv[32];
        tc::tmem_ld32(t_lane + st * p.buf_cols + c, sv);
        const float4* l4 = reinterpret_cast<const float4*>(&s_lse[warp][c]);
        if (__all_sync(0xffffffffu, c_lo <= c && c_hi >= c + 32)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 l = l4[e];
            a4[0] += ex2(fmaf(sv[4 * e], p.scale_log2, -l.x));
            a4[1] += ex2(fmaf(sv[4 * e + 1], p.scale_log2, -l.y));
            a4[2] += ex2(fmaf(sv[4 * e + 2], p.scale_log2, -l.z));
            a4[3] += ex2(fmaf(sv[4 * e + 3], p.scale_log2, -l.w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 l = l4[e];
            const int cc = c + 4 * e;
            a4[0] += cc >= c_lo && cc < c_hi ? ex2(fmaf(sv[4 * e], p.scale_log2, -l.x)) : 0.f;
            a4[1] += cc + 1 >= c_lo && cc + 1 < c_hi ? ex2(fmaf(sv[4 * e + 1], p.scale_log2, -l.y)) : 0.f;
            a4[2] += cc + 2 >= c_lo && cc + 2 < c_hi ? ex2(fmaf(sv[4 * e + 2], p.scale_log2, -l.z)) : 0.f;
            a4[3] += cc + 3 >= c_lo && cc + 3 < c_hi ? ex2(fmaf(sv[4 * e + 3], p.scale_log2, -l.w)) : 0.f;
          }
        }
      }
      acc += (a4[0] + a4[1]) + (a4[2] + a4[3]);
      tc::fence_before();
      tc::mbar_arrive(bar(SFREE + st));
    }
    if (ok && have) {
      const int64_t at = ((int64_t)page_of(p.keys, seq, key) * p.hkv + g << p.keys.page_log2) +
                         (key & ((1 << p.keys.page_log2) - 1));
      p.w_out[at] = p.w_in ? fmaf(p.decay, p.w_in[at], acc) : acc;
    }
  }

  __syncthreads();
  if (*abort) {
    if (warp == 4) {
      if (n > 0) tc::warp_drain(bar(K), 0);
      for (int st = 0; st < 2; ++st)
        if (last_q >= st) tc::warp_drain(bar(QFULL + st), ((last_q - ((last_q ^ st) & 1)) >> 1) & 1);
    } else if (warp == 5) {
      if (lane == 0) tc::commit(bar(DRAIN));
      __syncwarp();
      tc::warp_drain(bar(DRAIN), 0);
    }
  } else if (warp == 4) {
    for (int st = 0; st < 2; ++st)
      if (last_q >= st) tc::warp_drain(bar(QEMPTY + st), ((last_q - ((last_q ^ st) & 1)) >> 1) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 5) tmem_free(tmem, p.tmem_cols);
}

template <int D>
cudaError_t launch_weights_d(WeightParams& p, const void* q, cudaStream_t st) {
  p.R = p.h / p.hkv;
  p.tpc = std::max(1, std::min(ROWS / p.R, p.seqs.max_len));
  p.cols = up16(p.tpc * p.R);
  p.q_bytes = p.cols * D * 2;
  // 128-byte-swizzled tiles start on 1024 bytes: 16 rows of 128 bytes are 2048
  p.buf_cols = 32;
  while ((int)p.buf_cols < p.cols) p.buf_cols *= 2;
  p.tmem_cols = 2 * p.buf_cols;
  CUtensorMap mq, mk, mk16;
  // (a map needs rows; without queries none is ever loaded)
  const bool any = p.seqs.tokens > 0;
  if (!query_map(&mq, any ? q : p.keys.k, any ? p.seqs.tokens : 1, p.h, D, p.R, p.tpc) ||
      !key_maps(&mk, &mk16, p.keys.k, p.keys, p.hkv, D, 0))
    return cudaErrorInvalidValue;
  int smem = KT * D * 2 + kWStages * p.q_bytes + 1024;
  // no more CTAs on an SM than its 512 TMEM columns serve (228 KB, 1 KB of it per CTA reserved)
  smem = std::max(smem, 228 * 1024 / (512 / (int)p.tmem_cols + 1) - 1024 + 16);
  auto kern = weights_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t cap = (int64_t)p.keys.max_pages << p.keys.page_log2;
  const dim3 grid((unsigned)((cap + KT - 1) / KT), p.seqs.n_seqs, p.hkv);
  kern<<<grid, kWThreads, smem, st>>>(mq, mk, mk16, p);
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
  p.window = window;
  p.n_sink = n_sink;
  p.scale_log2 = scale * kLog2e;
  p.decay = decay;
  return d == 64 ? span::launch_weights_d<64>(p, q, st) : span::launch_weights_d<128>(p, q, st);
}

NSA_STATUS_ACCESSOR(span_weights)

}  // namespace nsa
