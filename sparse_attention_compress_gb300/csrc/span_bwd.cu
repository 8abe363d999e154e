// Backward of the sliding window with sinks (span_attn.cu on packed sequences).  Per row
// with seen keys j:  p_j = exp(scale q.k_j - lse),  dp_j = dO.v_j,  D = sum_j p_j dp_j,
//   ds_j = p_j (dp_j - D),  dq = scale sum_j ds_j k_j,
//   dk_j = scale sum_rows ds_j q,  dv_j = sum_rows p_j dO.
// S, dP and all accumulators are fp32 (TMEM); P and dS enter the last products as bf16: one
// rounding of at most 2^-8 relative per weight, of either sign over a sum's terms, which adds to a
// gradient's error about what its own rounding to bf16 does.  In tiles with a row of at most
// kFewKeys keys, where one term is much of a sum, the remainders x - bf16(x) pass through a second
// product, so that P and dS count to about 16 bits there.  D equals dO.o;
// where a row's ds_j are formed before all its dp_j are known it is taken so, from the bf16
// o, and the difference (the sum of the ds_j, which is 0 for the true D) is added for the
// gradients of k.  Rows of at most kFewKeys keys, in whose ds_j the rounding of o would show (it
// adds to dq's error the share 1 / sqrt(keys) of a bf16 rounding), have them in one tile, and
// their D is the sum itself.
//
// Two kernels, each a chain of M = 128 products over 128-wide tiles with eight softmax
// warps (two threads a TMEM lane, 64 columns each):
//   dq_kernel   a CTA owns 128 rows and walks the key tiles they see (S, dP, dQ).  It also
//               stores each row's base-2 lse and D (negated) for the second kernel.
//   dkv_kernel  a CTA owns 128 keys and walks the query tiles that see them, transposed
//               (S^T = K Q^T, dP^T = V dO^T), so that P^T and dS^T are, in place in TMEM,
//               the A operands of dV += P^T dO and dK += dS^T Q, and nothing passes through
//               shared memory but the tiles.
// Sinks are seen by every later query, so the queries past a sink tile's window are cut
// into chunks with a CTA each, and where there are fewer key tiles than SMs their own queries
// are divided too; the fp32 partials are summed in order by key_sum_kernel.
// No atomics: results are the same on every run.
//
// 65536 tokens x 64 heads (4 kv-heads, d = 128), window 512: dq 2.28 ms, dkv 1.98 ms, together
// 650 TFLOP/s.  dkv keeps the tensor cores busy 70% of its time.  dq is bound by its CTAs' starts
// and ends (five key tiles each, and 227 KB leave room for one on an SM) and by the chain S - P - dS
// of a tile: tensor cores 31%.  Small calls are bound by the four kernels' own lengths: 3 sequences
// of at most 1001 tokens x 16 heads, window 256, forward and backward 78 us on the device.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

constexpr uint32_t kBwdTmem = 512;
// A row at token t has min(t + 1, window + n_sink) keys.  Those of rows with at most this many lie
// in one key tile: bwd_layout sees to it.  (A test of P's values instead, for any row with a p of
// 1/4 or more, took 7% of the whole backward at window 512 and 11% at 1024: the softmax warps, which
// everything else waits for, would do it in every tile.  The remainders' code, a copy of its own
// that a tile chooses, takes 1% of it at 65536 tokens and window 512, 3 - 5% of small calls, and 17%
// under a window of 24 and 4 sinks, where every tile has few keys.)
constexpr int kFewKeys = 32;
// Remainders of a half's 64 values lie this many TMEM columns behind the values.
constexpr uint32_t kRest = 32;

struct BwdParams {
  Seqs seqs;
  Keys keys;  // packed
  const __nv_bfloat16 *q, *o, *dout;
  const float* lse;
  float* nlse2;  // [tokens, h] workspace: minus the base-2 lse (-inf for rows without keys)
  float* ndsum;  // [tokens, h] workspace: minus D
  __nv_bfloat16 *dq, *dk, *dv;
  float* part;  // [n_seqs][hkv][sink tiles][1 + n_far][2][sink_rows][D] fp32 (0: the near queries, undivided)
  float* near;  // [n_seqs][hkv][key tiles][n_near][2][KT][D] fp32, where n_near > 1
  int h, hkv, R, tpc, cols, window, n_sink;
  int n_far, far_tokens, sink_tiles, sink_rows, n_near;
  float scale, scale_log2;
};

__device__ __forceinline__ int last_in(int last, int st, int ns) { return last < st ? -1 : last - (last - st) % ns; }

// (+)= A[128 x w] (bf16 in TMEM: columns 0..31 hold the first 64, 64..95 the others)
// B[w x D], a tile of w rows read MN-major.
// b: desc_mn of the tile.
template <int D>
__device__ __forceinline__ void mma_split_a(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, int w, bool first,
                                            uint32_t lead) {
  constexpr uint32_t id = tc::idesc(ROWS, D) | kBMn;
  auto step = [&](int s) {
    mma_ts(d_tmem, a_tmem + (s < 4 ? s * 8 : 64 + (s - 4) * 8), b + s * (2048 >> 4), id, s == 0 ? !first : 1u, lead);
  };
  if (w == KT) {
#pragma unroll
    for (int s = 0; s < KT / 16; ++s) step(s);
  } else {
#pragma unroll
    for (int s = 0; s < KT / 16; ++s)
      if (s * 16 < w) step(s);
  }
}

// Two values as bf16.
__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
  const float2 d = unpair(x);
  return pack_bf16(d.x, d.y);
}
// What that leaves of them, as bf16.
__device__ __forceinline__ uint32_t rest_pair(uint64_t x) {
  const float2 v = unpair(x);
  const uint32_t hi = pack_bf16(v.x, v.y);
  const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
  return pack_bf16(v.x - h.x, v.y - h.y);
}

// ---------------------------------------------------------------------------- dQ
// Warps 0-7 softmax, 8 loads, 9 issues S, 10 dP, 11 dQ.  TMEM: S / dS of tile j at
// 128 (j & 1), dP at 256, dQ at 384: S of the next tile is computed while this one's dS is
// formed, dP once this tile's dP has been read.
constexpr int kDqThreads = 384, kNK = 3, kNV = 2;

template <int D>
constexpr int dq_smem() {
  return (2 + kNK + kNV) * KT * D * 2 + 1024;
}

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k16,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v16,
              const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_dq,
              const BwdParams p) {
  enum : int {
    Q = 0,
    KFULL = 1,
    KEMPTY = KFULL + kNK,
    VFULL = KEMPTY + kNK,
    VEMPTY = VFULL + kNV,
    SFULL = VEMPTY + kNV,  // [2] by S buffer
    PFULL = SFULL + 2,     // dP computed
    PFREE = PFULL + 1,     // dP read
    DSFULL = PFREE + 1,    // [2] dS written
    DQDONE = DSFULL + 2,   // [2] dQ product of that buffer done
    DRAIN = DQDONE + 2,
    COUNT
  };
  constexpr int TB = KT * D * 2;  // bytes of a tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[COUNT];
  __shared__ float s_dsum[ROWS], s_half[2][ROWS];  // dO.o of the rows; the halves' parts of a row sum
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t q_s = base, do_s = q_s + TB, k_s = do_s + TB, v_s = k_s + kNK * TB;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  launch_dependents();
  if (stopped()) return;
  const Waits wait(abort);
  const int seq = blockIdx.y, g = blockIdx.z;
  const int64_t start = seq_start(p.seqs, seq);
  const int L = seq_len(p.seqs, seq);
  const int t0 = ((L + p.tpc - 1) / p.tpc - 1 - (int)blockIdx.x) * p.tpc;
  if (t0 < 0) return;
  const Tiles tiles(t0, min(t0 + p.tpc, L) - 1, p.window, p.n_sink);
  const int n = tiles.n;
  const bool few = min(t0 + 1, p.window + p.n_sink) <= kFewKeys;  // some row has few keys

  if (tid == 0) {
    tc::mbar_init(bar(Q), 1);
    for (int i = 0; i < kNK; ++i) {
      tc::mbar_init(bar(KFULL + i), 1);
      tc::mbar_init(bar(KEMPTY + i), 1);
    }
    for (int i = 0; i < kNV; ++i) {
      tc::mbar_init(bar(VFULL + i), 1);
      tc::mbar_init(bar(VEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(SFULL + i), 1);
      tc::mbar_init(bar(DSFULL + i), 8);  // one arrival a softmax warp
      tc::mbar_init(bar(DQDONE + i), 1);
    }
    tc::mbar_init(bar(PFULL), 1);
    tc::mbar_init(bar(PFREE), 8);
    tc::mbar_init(bar(DRAIN), 3);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), kBwdTmem);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_k = -1, last_v = -1;
  if (warp == 8) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      tc::mbar_expect_tx(bar(Q), (uint32_t)(2 * p.tpc * p.R * D * 2));
      for (int c = 0; c < D / 64; ++c) {
        tc::tma3d(q_s + c * (ROWS * 128), &tm_q, c * 64, g * p.R, (int)(start + t0), bar(Q));
        tc::tma3d(do_s + c * (ROWS * 128), &tm_do, c * 64, g * p.R, (int)(start + t0), bar(Q));
      }
    }
    __syncwarp();
    // o passes through the V ring's first slot (its rows' D is formed there): by plain loads it
    // took three times as long to arrive as Q and dO do
    if (lane == 0) {
      tc::mbar_expect_tx(bar(VFULL), (uint32_t)(p.tpc * p.R * D * 2));
      for (int c = 0; c < D / 64; ++c)
        tc::tma3d(v_s + c * (ROWS * 128), &tm_o, c * 64, g * p.R, (int)(start + t0), bar(VFULL));
    }
    __syncwarp();
    last_v = 0;
    for (int j = 0; j < n; ++j) {
      const int w = tiles.width(j), sk = j % kNK, sv = (j + 1) % kNV;
      if (j >= kNK && !wait(bar(KEMPTY + sk), ((j / kNK) - 1) & 1)) break;
      load_tile<D, false>(k_s + sk * TB, &tm_k, &tm_k16, p.keys.k, p.keys, p.hkv, g, seq, start, j * KT, tiles.sink_end,
                          tiles.shift, w, L, bar(KFULL + sk), lane);
      last_k = j;
      if (j + 1 >= kNV && !wait(bar(VEMPTY + sv), (((j + 1) / kNV) - 1) & 1)) break;
      load_tile<D, false>(v_s + sv * TB, &tm_v, &tm_v16, p.keys.v, p.keys, p.hkv, g, seq, start, j * KT, tiles.sink_end,
                          tiles.shift, w, L, bar(VFULL + sv), lane);
      last_v = j + 1;
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ S
    const uint32_t lead = elect();
    bool ok = wait(bar(Q), 0);
    for (int j = 0; ok && j < n; ++j) {
      const int b = j & 1, sk = j % kNK;
      if (j >= 2 && !(ok = wait(bar(DQDONE + b), ((j >> 1) - 1) & 1))) break;
      if (!(ok = wait(bar(KFULL + sk), (j / kNK) & 1))) break;
      tc::fence_after();
      mma_abt<D>(tmem + b * 128, desc_k(q_s), desc_k(k_s) + sk * (TB >> 4), tiles.width(j), lead);
      commit(bar(SFULL + b), lead);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------------ dP
    const uint32_t lead = elect();
    bool ok = wait(bar(Q), 0);
    for (int j = 0; ok && j < n; ++j) {
      const int sv = (j + 1) % kNV;
      if (j >= 1 && !(ok = wait(bar(PFREE), (j - 1) & 1))) break;
      if (!(ok = wait(bar(VFULL + sv), ((j + 1) / kNV) & 1))) break;
      tc::fence_after();
      mma_abt<D>(tmem + 256, desc_k(do_s), desc_k(v_s) + sv * (TB >> 4), tiles.width(j), lead);
      commit(bar(PFULL), lead);
      commit(bar(VEMPTY + sv), lead);
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------------ dQ += dS K
    const uint32_t lead = elect();
    bool ok = true;
    for (int j = 0; ok && j < n; ++j) {
      const int b = j & 1, sk = j % kNK;
      // (dS of this tile was formed from S, so its K tile is in place)
      if (!(ok = wait(bar(DSFULL + b), (j >> 1) & 1))) break;
      tc::fence_after();
      mma_split_a<D>(tmem + 384, tmem + b * 128, desc_mn(k_s) + sk * (TB >> 4), tiles.width(j), j == 0, lead);
      if (few)
        mma_split_a<D>(tmem + 384, tmem + b * 128 + kRest, desc_mn(k_s) + sk * (TB >> 4), tiles.width(j), false, lead);
      commit(bar(DQDONE + b), lead);
      commit(bar(KEMPTY + sk), lead);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;  // columns 64 x .. 64 x + 63 of every tile
    const int tl = row / p.R, hd = row % p.R, t = t0 + tl;
    const bool valid = tl < p.tpc && t < L;
    const int pos = valid ? t : -1;
    const int64_t rr = (start + t) * p.h + g * p.R + hd;
    bool ok = true;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // D of the CTA's rows, sixteen lanes (d = 128) a row
    constexpr int CH = D / 8, RPW = 32 / CH, NIT = ROWS / (8 * RPW);  // chunks a row, rows a warp at a time
    const float lse = valid ? p.lse[rr] : kNegInf;
    ok = wait(bar(Q), 0) && wait(bar(VFULL), 0);
    {
      float sum[NIT];
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        const int r = (i * 8 + warp) * RPW + lane / CH;
        const uint4 ov = ld_shared(stage_at(v_s, ROWS * 128, r, lane % CH));
        const uint4 dv = ld_shared(stage_at(do_s, ROWS * 128, r, lane % CH));
        const uint32_t av[4] = {ov.x, ov.y, ov.z, ov.w}, bv[4] = {dv.x, dv.y, dv.z, dv.w};
        sum[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&av[e]));
          const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv[e]));
          sum[i] = fmaf(u.x, v.x, fmaf(u.y, v.y, sum[i]));
        }
      }
#pragma unroll
      for (int o = CH / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < NIT; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
      for (int i = 0; i < NIT; ++i)
        if (lane % CH == 0) s_dsum[(i * 8 + warp) * RPW + lane / CH] = sum[i];
    }
    named_barrier(1, 256);  // (after a timeout too: every softmax warp comes here)
    // (a thread that gave up on o does not hand its slot on: the copy may still be in flight)
    if (tid == 0 && ok) tc::mbar_arrive(bar(VEMPTY));
    float l2 = __builtin_inff(), dsum = 0.f;
    if (valid) {
      l2 = lse == kNegInf ? __builtin_inff() : lse * kLog2e;
      dsum = s_dsum[row];
    }
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), nl2 = pair(-l2, -l2);
    uint64_t nd2 = pair(-dsum, -dsum), e2 = 0;  // e2: this half's sum of ds
    // the sum of both halves' parts of a row (every softmax warp comes here)
    auto row_sum = [&](float part) {
      s_half[x][row] = part;
      named_barrier(2, 256);
      return s_half[0][row] + s_half[1][row];
    };
    // (with one tile a warp that gave up, here or before, still comes to the barrier of row_sum:
    // the others may not have)
    // (remainders or none in code of their own: what the one keeps alive would cost the other)
    auto walk = [&](auto with_rest) {
      for (int j = 0; (ok || n == 1) && j < n; ++j) {
        const int b = j & 1, key0 = tiles.key0(j), w = tiles.width(j);
        ok = wait(bar(SFULL + b), (j >> 1) & 1) && ok;
        if (!ok && n > 1) break;
        tc::fence_after();
        const uint32_t s_t = tmem + b * 128 + x * 64 + lane_base, p_t = tmem + 256 + x * 64 + lane_base;
        const int c0 = x * 64, nc = min(64, w - c0);  // columns of this half (nc <= 0: none)
        float sv[64];
#pragma unroll
        for (int c = 0; c < 64; c += 32)
          tc::tmem_ld32_nowait(s_t + c, sv + c);
        const int j_hi = min(pos + 1 - key0, w), j_lo = pos - p.window + 1 - key0, j_sink = tiles.sinks(j, p.n_sink);
        const bool all = __all_sync(0xffffffffu, j_hi >= c0 + 64 && (j_lo <= c0 || j_sink >= c0 + 64));
        tmem_wait_ld(sv);
        tmem_wait_ld(sv + 32);
        if (!all) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            const uint32_t see = bits(j_lo - c0 - c, j_hi - c0 - c) | bits(0, min(j_sink, j_hi) - c0 - c);
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[c + e] = (see >> e) & 1u ? sv[c + e] : kNegInf;
          }
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 y = unpair(fma2(pair(sv[c], sv[c + 1]), scale2, nl2));
          sv[c] = ex2(y.x);
          sv[c + 1] = ex2(y.y);
        }
        ok = wait(bar(PFULL), j & 1) && ok;
        if (!ok && n > 1) break;
        tc::fence_after();
        float dp[64];
#pragma unroll
        for (int c = 0; c < 64; c += 32)
          tc::tmem_ld32_nowait(p_t + c, dp + c);
        tmem_wait_ld(dp);
        tmem_wait_ld(dp + 32);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(PFREE));
        // (an unseen key's p is 0 and its dp finite; columns past the tile's hold anything)
#pragma unroll
        for (int c = 0; c < 64; c += GRAN)
          if (c >= nc) {
#pragma unroll
            for (int e = 0; e < GRAN; ++e) dp[c + e] = 0.f;
          }
        if (n == 1) {
          uint64_t d2 = 0;
#pragma unroll
          for (int c = 0; c < 64; c += 2) d2 = fma2(pair(sv[c], sv[c + 1]), pair(dp[c], dp[c + 1]), d2);
          const float2 d = unpair(d2);
          dsum = row_sum(d.x + d.y);
          nd2 = pair(-dsum, -dsum);
          if (!ok) break;
        }
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          if (c >= nc) break;
          uint32_t pk[16];
          auto ds = [&](int e) {  // (an unseen key has p = 0)
            return mul2(pair(sv[c + e], sv[c + e + 1]), add2(pair(dp[c + e], dp[c + e + 1]), nd2));
          };
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t d = ds(e);
            e2 = add2(e2, d);
            pk[e / 2] = pack_pair(d);
          }
          tmem_st16_nowait(s_t + c / 2, pk);
          if constexpr (decltype(with_rest)::value) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) pk[e / 2] = rest_pair(ds(e));
            tmem_st16_nowait(s_t + kRest + c / 2, pk);
          }
        }
        tmem_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(DSFULL + b));
      }
    };
    if (few)
      walk(std::true_type{});
    else
      walk(std::false_type{});
    if (ok) {
      ok = wait(bar(DQDONE + ((n - 1) & 1)), ((n - 1) >> 1) & 1);
      tc::fence_after();
    }
    if (n > 1) {
      const float2 e = unpair(e2);
      dsum += row_sum(e.x + e.y);  // (the sum of p is 1)
    }
    if (ok && valid && x == 0) {
      p.nlse2[rr] = -l2;
      p.ndsum[rr] = -dsum;
    }
    if (ok) {
      // staged over Q, which every S has read
#pragma unroll 1
      for (int c = x * (D / 2); c < (x + 1) * (D / 2); c += 32) {
        float v[32];
        tc::tmem_ld32(tmem + 384 + lane_base + c, v);
        stage_cols(q_s, ROWS * 128, row, c, v, p.scale);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    named_barrier(1, 256);
    if (ok && t0 + p.tpc <= L) {
      if (tid == 0) store_tile<D>(&tm_dq, q_s, ROWS * 128, g * p.R, (int)(start + t0));
    } else if (ok) {  // the box would reach into the next sequence
      unstage_rows<D>(q_s, ROWS * 128, p.tpc * p.R, p.R, p.h, L - t0, p.dq + ((start + t0) * p.h + g * p.R) * D, tid,
                      256);
    }
  }

  __syncthreads();
  if (*abort) {
    if (warp == 8) {
      tc::warp_drain(bar(Q), 0);
      for (int st = 0; st < kNK; ++st)
        if (const int i = last_in(last_k, st, kNK); i >= 0) tc::warp_drain(bar(KFULL + st), (i / kNK) & 1);
      for (int st = 0; st < kNV; ++st)
        if (const int i = last_in(last_v, st, kNV); i >= 0) tc::warp_drain(bar(VFULL + st), (i / kNV) & 1);
    } else if (warp > 8) {
      commit(bar(DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(DRAIN), 0);
    }
  } else if (warp == 8) {
    for (int st = 0; st < kNK; ++st)
      if (const int i = last_in(last_k, st, kNK); i >= 0) tc::warp_drain(bar(KEMPTY + st), (i / kNK) & 1);
    for (int st = 0; st < kNV; ++st)
      if (const int i = last_in(last_v, st, kNV); i >= 0) tc::warp_drain(bar(VEMPTY + st), (i / kNV) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 9) tmem_free(tmem, kBwdTmem);
}

// ---------------------------------------------------------------------------- dK, dV
// Warps 0-7 softmax, 8 loads, 9 issues S^T and dV, 10 dP^T and dK.  TMEM: S^T (then P^T) at
// 0, dP^T (then dS^T) at 128, dV at 256, dK at 384.  The two issuers' chains interleave on
// the tensor pipe: while P^T is formed dK of the tile before and dP^T run, while dS^T is
// formed dV and the next S^T do.  (S^T of a tile overwrites P^T of the one before, and dP^T
// its dS^T: the same lane issued the products that read them, and products execute in
// issue order.)
// A tile's Q is read from its S^T to its dK, its dO from dP^T to dV, hence three slots and
// two: all that 227 KB hold at d = 128, to within the alignment of the first.
constexpr int kDkvThreads = 352, kNQ = 3, kND = 2, kSmemMax = 227 * 1024;

template <int D>
constexpr int dkv_tiles() {
  return (2 + kNQ + kND) * KT * D * 2;
}

template <int D>
__global__ void __launch_bounds__(kDkvThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k16,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v16,
               const BwdParams p) {
  enum : int {
    KV = 0,      // [2] K, V
    QFULL = 2,             // by slot: Q rows
    QEMPTY = QFULL + kNQ,
    DFULL = QEMPTY + kNQ,  // by slot: dO rows, lse, D
    DEMPTY = DFULL + kND,
    SFULL = DEMPTY + kND,
    PFULL,   // P^T written
    DVDONE,  // every dV product is done
    DPFULL,
    DSFULL,  // dS^T written
    DKDONE,  // every dK product is done
    DRAIN,
    COUNT
  };
  constexpr int TB = KT * D * 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[COUNT];
  // minus the rows' base-2 lse (of tile j at j % 2: a tile's dV is done, and its lse read, before
  // the next but one is loaded) and D (at j % 3: read after that, but before the next tile's P^T)
  __shared__ __align__(16) float s_l2[2][ROWS], s_d[3][ROWS];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t k_s = base, v_s = k_s + TB, q_s = v_s + TB, do_s = q_s + kNQ * TB;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  {  // (the tiles fit what the launch gave, wherever the static shared memory ends)
    uint32_t given;
    asm("mov.u32 %0, %%dynamic_smem_size;\n" : "=r"(given));
    if (base + dkv_tiles<D>() > smem_u32(smem_raw) + given) {
      if (threadIdx.x == 0) atomicExch(&g_device_status, (int)NSA_ERR_CUDA);
      return;
    }
  }
  launch_dependents();
  if (stopped()) {
    wait_primary();
    return;
  }
  const Waits wait(abort);
  // items of a (sequence, kv-head): the chunks of far queries of the sink tiles, then every
  // key tile with the queries within its window
  const int n_far_items = p.sink_tiles * p.n_far;
  const int seq = blockIdx.y, g = blockIdx.z;
  const int64_t start = seq_start(p.seqs, seq);
  const int L = seq_len(p.seqs, seq);
  const bool far = (int)blockIdx.x < n_far_items;
  const int kt = far ? (int)blockIdx.x / p.n_far : ((int)blockIdx.x - n_far_items) / p.n_near;
  const int chunk = far ? (int)blockIdx.x % p.n_far : -1;
  const int share = far ? 0 : ((int)blockIdx.x - n_far_items) % p.n_near;
  const int key0 = kt * KT;
  if (key0 >= L) return;  // (some block of the call has keys, and waits)
  const int near_end = min(L, key0 + KT - 1 + p.window);
  const int near_tiles = (near_end - key0 + p.tpc - 1) / p.tpc;
  const int t_lo = far ? near_end + chunk * p.far_tokens : key0 + near_tiles * share / p.n_near * p.tpc;
  const int t_hi = far ? min(L, t_lo + p.far_tokens) : min(near_end, key0 + near_tiles * (share + 1) / p.n_near * p.tpc);
  if (t_lo >= t_hi) return;  // (an empty chunk or share: key_sum_kernel does not read it)
  const int n = (t_hi - t_lo + p.tpc - 1) / p.tpc;
  const int used = p.tpc * p.R;  // rows of a tile
  // Tiles that have a row with few keys come first: all, or those of a sequence's first tokens (where
  // the round begins with the first tile).
  const int n_few = p.window + p.n_sink <= kFewKeys ? n : min(n, (max(0, kFewKeys - t_lo) + p.tpc - 1) / p.tpc);
  // A query tile is seen by the key tiles of its whole window, CTAs that run side by side.
  // Each begins its round of query tiles where the others do (at the tile whose index is a
  // multiple of a full round's length), so that they ask for the same tile at about the same
  // time and all but one find it in L2: begun at the first tile instead, 8192 tokens x 64
  // heads read 1.30 GB from HBM for 0.27 GB of q and dO.
  const int round = (KT - 1 + p.window + p.tpc - 1) / p.tpc;
  const int first = far || p.n_near > 1 ? 0 : (round - t_lo / p.tpc % round) % round;
  auto token_of = [&](int j) {  // first token of the round's tile j
    const int i = j + (first < n ? first : 0);
    return t_lo + (i < n ? i : i - n) * p.tpc;
  };

  if (tid == 0) {
    tc::mbar_init(bar(KV), 1);
    tc::mbar_init(bar(KV + 1), 1);
    for (int i = 0; i < kNQ; ++i) {
      tc::mbar_init(bar(QFULL + i), 1);
      tc::mbar_init(bar(QEMPTY + i), 1);
    }
    for (int i = 0; i < kND; ++i) {
      tc::mbar_init(bar(DFULL + i), 1);
      tc::mbar_init(bar(DEMPTY + i), 2);  // dP^T and dV have read dO
    }
    tc::mbar_init(bar(SFULL), 1);
    tc::mbar_init(bar(PFULL), 8);  // one arrival a softmax warp
    tc::mbar_init(bar(DVDONE), 1);
    tc::mbar_init(bar(DPFULL), 1);
    tc::mbar_init(bar(DSFULL), 8);
    tc::mbar_init(bar(DKDONE), 1);
    tc::mbar_init(bar(DRAIN), 2);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  // rows between the tile's own and the next multiple of 16 (group sizes that do not divide
  // 128) enter the products as zeros; no copy ever writes them
  for (int e = tid; e < (p.cols - used) * (kNQ + kND) * (D / 8); e += kDkvThreads) {
    const int ch = e % (D / 8), which = e / (D / 8) % (kNQ + kND), r = used + e / ((kNQ + kND) * (D / 8));
    const uint32_t to = q_s + which * TB + (ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(to), "r"(0u) : "memory");
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), kBwdTmem);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_q = -1, last_d = -1;
  if (warp == 8) {
    // ------------------------------------------------------------------ loads
    const int w = min(KT, up16(L - key0));
    load_tile<D, false>(k_s, &tm_k, &tm_k16, p.keys.k, p.keys, p.hkv, g, seq, start, key0, 0, 0, w, L, bar(KV),
                        lane);
    load_tile<D, false>(v_s, &tm_v, &tm_v16, p.keys.v, p.keys, p.hkv, g, seq, start, key0, 0, 0, w, L,
                        bar(KV + 1), lane);
    // Rows of tokens t .. t + tpc - 1 (those past the sequence as zeros: they are another
    // sequence's, or lie past the tensors); returns the bytes to come.
    auto load_rows = [&](uint32_t to, const CUtensorMap* map, const __nv_bfloat16* src, int t, uint32_t full) {
      if (t + p.tpc <= L) {
        if (lane < D / 64) tc::tma3d(to + lane * (ROWS * 128), map, lane * 64, g * p.R, (int)(start + t), full);
        return (uint32_t)(used * D * 2);
      }
      for (int e = lane; e < used * (D / 8); e += 32) {
        const int r = e / (D / 8), ch = e % (D / 8), tt = t + r / p.R;
        const bool in = tt < L;
        cp_async16(to + (ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                   in ? (const void*)(src + ((start + tt) * p.h + g * p.R + r % p.R) * D + ch * 8) : (const void*)src,
                   in ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      return 0u;
    };
    // minus the base-2 lse and D of a tile's rows, four a lane, fetched a tile ahead
    float nl[ROWS / 32], nd[ROWS / 32];
    int tok[ROWS / 32], at[ROWS / 32];  // a row's token (past every sequence: no row) and place in the tile
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i) {
      const int e = lane + i * 32;
      tok[i] = e < used ? e / p.R : 1 << 30;
      at[i] = e / p.R * p.h + e % p.R;
    }
    auto fetch = [&](int t) {
      const int64_t r0 = (start + t) * p.h + g * p.R;
#pragma unroll
      for (int i = 0; i < ROWS / 32; ++i) {
        const bool in = tok[i] < L - t;
        nl[i] = in ? __ldcg(p.nlse2 + r0 + at[i]) : kNegInf;  // (written while this kernel starts)
        nd[i] = in ? __ldcg(p.ndsum + r0 + at[i]) : 0.f;
      }
    };
    wait_primary();  // (K and V are on their way)
    fetch(token_of(0));
    Ring<kNQ> rq;
    Ring<kND> rd;
    for (int j = 0; j < n; ++j) {
      const int t = token_of(j);
      if (j >= kNQ && !wait(bar(QEMPTY + rq.slot), rq.phase ^ 1u)) break;
      uint32_t bytes = load_rows(q_s + rq.slot * TB, &tm_q, p.q, t, bar(QFULL + rq.slot));
      __syncwarp();
      if (lane == 0) tc::mbar_expect_tx(bar(QFULL + rq.slot), bytes);
      last_q = j;
      if (j >= kND && !wait(bar(DEMPTY + rd.slot), rd.phase ^ 1u)) break;
      bytes = load_rows(do_s + rd.slot * TB, &tm_do, p.dout, t, bar(DFULL + rd.slot));
#pragma unroll
      for (int i = 0; i < ROWS / 32; ++i) {
        s_l2[j & 1][lane + i * 32] = nl[i];
        s_d[rq.slot][lane + i * 32] = nd[i];
      }
      __syncwarp();
      if (lane == 0) tc::mbar_expect_tx(bar(DFULL + rd.slot), bytes);
      if (j + 1 < n) fetch(token_of(j + 1));
      last_d = j;
      rq.next();
      rd.next();
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ S^T, dV += P^T dO
    const uint32_t lead = elect(), kd = desc_k(k_s), qd = desc_k(q_s), dd = desc_mn(do_s);
    Ring<kNQ> rq;
    Ring<kND> rd;
    // (what a product needs beside P^T is waited for before it, so that dV and the next S^T go
    // out together)
    auto issue_s = [&]() {
      mma_abt<D>(tmem, kd, qd + rq.slot * (TB >> 4), p.cols, lead);
      commit(bar(SFULL), lead);
      rq.next();
    };
    bool ok = wait(bar(KV), 0) && wait(bar(QFULL), 0);
    if (ok) {
      tc::fence_after();
      issue_s();
    }
    auto walk = [&](auto with_rest, int j0, int j1) {
      for (int j = j0; ok && j < j1; ++j) {
        if (!(ok = wait(bar(DFULL + rd.slot), rd.phase))) break;
        if (j + 1 < n && !(ok = wait(bar(QFULL + rq.slot), rq.phase))) break;
        if (!(ok = wait(bar(PFULL), j & 1))) break;
        tc::fence_after();
        mma_split_a<D>(tmem + 256, tmem, dd + rd.slot * (TB >> 4), p.cols, j == 0, lead);
        if constexpr (decltype(with_rest)::value)
          mma_split_a<D>(tmem + 256, tmem + kRest, dd + rd.slot * (TB >> 4), p.cols, false, lead);
        commit(bar(DEMPTY + rd.slot), lead);
        if (j + 1 < n)
          issue_s();
        else
          commit(bar(DVDONE), lead);
        rd.next();
      }
    };
    walk(std::true_type{}, 0, n_few);
    walk(std::false_type{}, n_few, n);
  } else if (warp == 10) {
    // ------------------------------------------------------------------ dP^T, dK += dS^T Q
    const uint32_t lead = elect(), vd = desc_k(v_s), dd = desc_k(do_s), qd = desc_mn(q_s);
    Ring<kNQ> rq;
    Ring<kND> rd;
    auto issue_dp = [&]() {
      mma_abt<D>(tmem + 128, vd, dd + rd.slot * (TB >> 4), p.cols, lead);
      commit(bar(DPFULL), lead);
      commit(bar(DEMPTY + rd.slot), lead);
      rd.next();
    };
    bool ok = wait(bar(KV + 1), 0) && wait(bar(DFULL), 0);
    if (ok) {
      tc::fence_after();
      issue_dp();
    }
    auto walk = [&](auto with_rest, int j0, int j1) {
      for (int j = j0; ok && j < j1; ++j) {
        if (j + 1 < n && !(ok = wait(bar(DFULL + rd.slot), rd.phase))) break;
        if (!(ok = wait(bar(DSFULL), j & 1))) break;
        tc::fence_after();
        mma_split_a<D>(tmem + 384, tmem + 128, qd + rq.slot * (TB >> 4), p.cols, j == 0, lead);
        if constexpr (decltype(with_rest)::value)
          mma_split_a<D>(tmem + 384, tmem + 128 + kRest, qd + rq.slot * (TB >> 4), p.cols, false, lead);
        commit(bar(QEMPTY + rq.slot), lead);  // (S^T of the tile was done before its dS^T)
        if (j + 1 < n)
          issue_dp();
        else
          commit(bar(DKDONE), lead);
        rq.next();
      }
    };
    walk(std::true_type{}, 0, n_few);
    walk(std::false_type{}, n_few, n);
  } else {
    // ------------------------------------------------------------------ softmax
    const int x = warp >> 2, row = (warp & 3) * 32 + lane, key = key0 + row, c0 = x * 64;
    const bool have = key < L;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + c0 + lane_base, p_t = tmem + 128 + c0 + lane_base;
    const int nc = min(64, p.cols - c0);
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
    Ring<kNQ> rq;  // (D's buffers go with Q's slots: three of each)
    Ring<kND> rd;
    bool ok = true;
    // (remainders or none in code of their own, as above)
    auto tile = [&](auto with_rest, int j) -> bool {
      const int t = token_of(j);
      // columns [c_lo, c_hi) of this half are rows whose query sees this key
      int c_lo = 0, c_hi = 0;
      if (have) {
        int64_t end = (int64_t)min(p.tpc, t_hi - t) * p.R;
        if (key >= p.n_sink) end = min(end, ((int64_t)key + p.window - t) * p.R);
        c_lo = (int)max((int64_t)0, min((int64_t)(key - t) * p.R, (int64_t)ROWS)) - c0;
        c_hi = (int)max((int64_t)0, end) - c0;
      }
      if (!wait(bar(DFULL + rd.slot), rd.phase)) return false;  // lse and D
      if (!wait(bar(SFULL), j & 1)) return false;
      tc::fence_after();
      float sv[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32)
        tc::tmem_ld32_nowait(s_t + c, sv + c);
      const bool all = c_lo <= 0 && c_hi >= 64;
      const float4* l4 = reinterpret_cast<const float4*>(&s_l2[j & 1][c0]);
      tmem_wait_ld(sv);
      tmem_wait_ld(sv + 32);
      if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          const uint32_t see = bits(c_lo - c, c_hi - c);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[c + e] = (see >> e) & 1u ? sv[c + e] : kNegInf;
        }
      }
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = l4[(c + e) / 4];
          const float2 y = unpair(fma2(pair(sv[c + e], sv[c + e + 1]), scale2, pair(l.x, l.y)));
          const float2 z = unpair(fma2(pair(sv[c + e + 2], sv[c + e + 3]), scale2, pair(l.z, l.w)));
          sv[c + e] = ex2(y.x);
          sv[c + e + 1] = ex2(y.y);
          sv[c + e + 2] = ex2(z.x);
          sv[c + e + 3] = ex2(z.y);
          pk[e / 2] = pack_bf16(sv[c + e], sv[c + e + 1]);
          pk[e / 2 + 1] = pack_bf16(sv[c + e + 2], sv[c + e + 3]);
        }
        if (c < nc) tmem_st16_nowait(s_t + c / 2, pk);
        if constexpr (decltype(with_rest)::value) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) pk[e / 2] = rest_pair(pair(sv[c + e], sv[c + e + 1]));
          if (c < nc) tmem_st16_nowait(s_t + kRest + c / 2, pk);
        }
      }
      tmem_wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(PFULL));
      if (!wait(bar(DPFULL), j & 1)) return false;
      tc::fence_after();
      const float4* d4 = reinterpret_cast<const float4*>(&s_d[rq.slot][c0]);
      float dp[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32)
        tc::tmem_ld32_nowait(p_t + c, dp + c);
      tmem_wait_ld(dp);
      tmem_wait_ld(dp + 32);
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        if (c >= nc) break;
        uint32_t pk[16];
        // (zero rows past the sequence have dp = 0, so p = 0 gives ds = 0)
        auto ds = [&](int e, float x, float y) {
          return mul2(pair(sv[c + e], sv[c + e + 1]), add2(pair(dp[c + e], dp[c + e + 1]), pair(x, y)));
        };
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = d4[(c + e) / 4];
          pk[e / 2] = pack_pair(ds(e, d.x, d.y));
          pk[e / 2 + 1] = pack_pair(ds(e + 2, d.z, d.w));
        }
        tmem_st16_nowait(p_t + c / 2, pk);
        if constexpr (decltype(with_rest)::value) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 d = d4[(c + e) / 4];
            pk[e / 2] = rest_pair(ds(e, d.x, d.y));
            pk[e / 2 + 1] = rest_pair(ds(e + 2, d.z, d.w));
          }
          tmem_st16_nowait(p_t + kRest + c / 2, pk);
        }
      }
      tmem_wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(DSFULL));
      return true;
    };
    for (int j = 0; j < n; ++j, rq.next(), rd.next())
      if (!(ok = j < n_few ? tile(std::true_type{}, j) : tile(std::false_type{}, j))) break;
    if (ok) {
      ok = wait(bar(DVDONE), 0) && wait(bar(DKDONE), 0);
      tc::fence_after();
    }
    if (ok) {
      // half 0 writes dK, half 1 dV
      const float f = x ? 1.f : p.scale;
      const bool divided = !far && p.n_near > 1;
      const bool to_part = divided || (kt < p.sink_tiles && p.n_far > 0 && key < p.n_sink);
      float* part;
      if (divided) {
        const int n_kt = ((int)gridDim.x - n_far_items) / p.n_near;
        part = p.near + (((((int64_t)seq * p.hkv + g) * n_kt + kt) * p.n_near + share) * 2 + x) * KT * D + row * D;
      } else {
        part = p.part + (((((int64_t)seq * p.hkv + g) * p.sink_tiles + kt) * (1 + p.n_far) + (chunk + 1)) * 2 + x) *
                            p.sink_rows * D + (int64_t)row * D;
      }
      __nv_bfloat16* dst = (x ? p.dv : p.dk) + ((start + key) * p.hkv + g) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        tc::tmem_ld32(tmem + (x ? 256 : 384) + lane_base + c, v);
        if (have && to_part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else if (have && !far) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 u;
            u.x = pack_bf16(v[e] * f, v[e + 1] * f);
            u.y = pack_bf16(v[e + 2] * f, v[e + 3] * f);
            u.z = pack_bf16(v[e + 4] * f, v[e + 5] * f);
            u.w = pack_bf16(v[e + 6] * f, v[e + 7] * f);
            *reinterpret_cast<uint4*>(dst + c + e) = u;
          }
        }
      }
    }
  }

  __syncthreads();
  if (*abort) {
    if (warp == 8) {
      tc::warp_drain(bar(KV), 0);
      tc::warp_drain(bar(KV + 1), 0);
      for (int st = 0; st < kNQ; ++st)
        if (const int i = last_in(last_q, st, kNQ); i >= 0) tc::warp_drain(bar(QFULL + st), (i / kNQ) & 1);
      for (int st = 0; st < kND; ++st)
        if (const int i = last_in(last_d, st, kND); i >= 0) tc::warp_drain(bar(DFULL + st), (i / kND) & 1);
    } else if (warp > 8) {
      commit(bar(DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(DRAIN), 0);
    }
  } else if (warp == 8) {
    for (int st = 0; st < kNQ; ++st)
      if (const int i = last_in(last_q, st, kNQ); i >= 0) tc::warp_drain(bar(QEMPTY + st), (i / kNQ) & 1);
    for (int st = 0; st < kND; ++st)
      if (const int i = last_in(last_d, st, kND); i >= 0) tc::warp_drain(bar(DEMPTY + st), (i / kND) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 9) tmem_free(tmem, kBwdTmem);
}

// dK and dV of the keys that several CTAs hold parts of: the near parts and, for sinks, the
// far chunks, in order.  One block a (key, kv-head, sequence); thread: column of dK (first D
// threads) or dV.
template <int D>
__global__ void __launch_bounds__(2 * D) key_sum_kernel(const BwdParams p, int n_kt) {
  wait_primary();
  const int key = blockIdx.x, g = blockIdx.y, seq = blockIdx.z;
  const int L = seq_len(p.seqs, seq);
  if (key >= L) return;
  const int x = threadIdx.x / D, c = threadIdx.x % D, kt = key / KT;
  const int near_end = min(L, kt * KT + KT - 1 + p.window);
  float acc = 0.f;
  if (p.n_near > 1) {
    const int tiles = (near_end - kt * KT + p.tpc - 1) / p.tpc;
    const float* src = p.near + ((((int64_t)seq * p.hkv + g) * n_kt + kt) * p.n_near * 2 + x) * KT * D +
                       (int64_t)(key % KT) * D + c;
    for (int i = 0; i < p.n_near; ++i)
      if (tiles * (i + 1) / p.n_near > tiles * i / p.n_near) acc += src[(int64_t)i * 2 * KT * D];
  }
  if (p.n_far > 0 && key < p.n_sink) {
    const int64_t step = (int64_t)2 * p.sink_rows * D;
    const float* src = p.part + (((int64_t)seq * p.hkv + g) * p.sink_tiles + kt) * (1 + p.n_far) * step +
                       ((int64_t)x * p.sink_rows + key % KT) * D + c;
    // (no more than there are, should a sequence be longer than the call's longest length)
    const int parts = 1 + min(p.n_far, (L - near_end + p.far_tokens - 1) / p.far_tokens);
#pragma unroll 4
    for (int i = p.n_near > 1; i < parts; ++i) acc += src[i * step];
  }
  __nv_bfloat16* dst = (x ? p.dv : p.dk) + ((seq_start(p.seqs, seq) + key) * (int64_t)p.hkv + g) * D + c;
  *dst = __float2bfloat16_rn(x ? acc : acc * p.scale);
}

struct BwdLayout {
  int tpc, n_far, far_tokens, sink_tiles, sink_rows, n_near;
  size_t dsum, part, near, bytes;
};
BwdLayout bwd_layout(const Seqs& s, int h, int hkv, int D, int window, int n_sink) {
  BwdLayout l{};
  const int R = h / hkv;
  l.tpc = std::max(1, std::min(ROWS / R, s.max_len));
  // The sinks and windows of a tile's rows in one key tile (its first token is a multiple of 16 where
  // this bites: group 1 alone, 80 to 112 rows a tile instead of 128).
  if ((int64_t)window + n_sink <= kFewKeys) l.tpc = std::min(l.tpc, KT - up16(window - 1) - up16(n_sink));
  const int sinks = std::min(n_sink, s.max_len);
  const int64_t far = sinks > 0 ? (int64_t)s.max_len - (KT - 1) - window : 0;  // queries past the first tile's window
  const int64_t own = (int64_t)window + KT - 1;                                // queries of a key tile
  const int64_t n_kt = ((int64_t)s.max_len + KT - 1) / KT, units = (int64_t)s.n_seqs * hkv;
  l.sink_tiles = far > 0 ? (sinks + KT - 1) / KT : 0;
  // Fewer key tiles (and chunks of a tile's length) than SMs: their queries are divided as far
  // as one round of the SMs holds the shares, none below eight query tiles.  3 sequences of at
  // most 1001 tokens x 16 heads, window 256 (60 CTAs that walk 48 query tiles each): 65 us whole,
  // 39 us and 10 us to sum in 2 shares.
  const int64_t far_chunks = far > 0 ? std::min<int64_t>(64, (far + own - 1) / own) : 0;
  const int64_t walk = (std::min<int64_t>(s.max_len, own) + l.tpc - 1) / l.tpc;
  const int64_t ctas = std::max<int64_t>(1, (n_kt + l.sink_tiles * far_chunks) * units);
  l.n_near = (int)std::max<int64_t>(1, std::min<int64_t>(152 / ctas, walk / 8));
  if (far > 0) {
    // a chunk is about as long as a share of a key tile's own queries, at most 64 chunks
    const int64_t len = std::max<int64_t>((own + l.n_near - 1) / l.n_near, (far + 63) / 64);
    l.far_tokens = (int)((len + l.tpc - 1) / l.tpc * l.tpc);
    l.n_far = (int)((far + l.far_tokens - 1) / l.far_tokens);
    l.sink_rows = std::min(sinks, KT);
  }
  auto a256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  l.dsum = a256((size_t)s.tokens * h * 4);
  l.part = 2 * l.dsum;
  l.near = a256(l.part + (size_t)s.n_seqs * hkv * l.sink_tiles * (1 + l.n_far) * 2 * l.sink_rows * D * 4);
  l.bytes = l.near + (l.n_near > 1 ? (size_t)(n_kt * units) * l.n_near * 2 * KT * D * 4 : 0);
  return l;
}

template <int D>
cudaError_t launch_bwd_d(BwdParams& p, const BwdLayout& l, cudaStream_t st) {
  const Seqs& s = p.seqs;
  CUtensorMap mq, md, mo, mdq, mk, mk16, mv, mv16;
  if (!query_map(&mo, p.o, s.tokens, p.h, D, p.R, p.tpc) || !query_map(&mdq, p.dq, s.tokens, p.h, D, p.R, p.tpc) ||
      !query_map(&mq, p.q, s.tokens, p.h, D, p.R, p.tpc) || !query_map(&md, p.dout, s.tokens, p.h, D, p.R, p.tpc) ||
      !key_maps(&mk, &mk16, p.keys.k, p.keys, p.hkv, D, s.tokens) ||
      !key_maps(&mv, &mv16, p.keys.v, p.keys, p.hkv, D, s.tokens))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq_smem<D>());
  if (e != cudaSuccess) return e;
  // the tiles start on the first multiple of 1024 after the static shared memory
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, dkv_kernel<D>)) != cudaSuccess) return e;
  const int fixed = (int)at.sharedSizeBytes, dkv_smem = (fixed + 1023) / 1024 * 1024 + dkv_tiles<D>() - fixed;
  if (fixed + dkv_smem > kSmemMax) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, dkv_smem);
  if (e != cudaSuccess) return e;
  dq_kernel<D><<<dim3((s.max_len + p.tpc - 1) / p.tpc, s.n_seqs, p.hkv), kDqThreads, dq_smem<D>(), st>>>(
      mq, md, mk, mk16, mv, mv16, mo, mdq, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int n_kt = (s.max_len + KT - 1) / KT, items = l.sink_tiles * l.n_far + n_kt * l.n_near;
  e = launch_second(dkv_kernel<D>, dim3(items, s.n_seqs, p.hkv), kDkvThreads, dkv_smem, st, mq, md, mk, mk16, mv, mv16, p);
  if (e != cudaSuccess || (l.n_far == 0 && l.n_near == 1)) return e;
  const int keys = l.n_near > 1 ? s.max_len : std::min(p.n_sink, s.max_len);
  return launch_second(key_sum_kernel<D>, dim3(keys, p.hkv, s.n_seqs), 2 * D, 0, st, p, n_kt);
}

}  // namespace span

size_t span_bwd_workspace_bytes(const Seqs& s, int h, int hkv, int d, int window, int n_sink) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return 0;
  return span::bwd_layout(s, h, hkv, d, window, n_sink).bytes;
}

cudaError_t launch_span_bwd(const Seqs& s, const void* q, const void* k, const void* v, int h, int hkv, int d,
                            int window, int n_sink, float scale, const void* o, const float* lse, const void* dout,
                            void* dq, void* dk, void* dv, void* workspace, cudaStream_t st) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return cudaSuccess;
  const span::BwdLayout l = span::bwd_layout(s, h, hkv, d, window, n_sink);
  span::BwdParams p{};
  p.seqs = s;
  p.keys = span::keys_of(nullptr, k, v);
  p.q = (const __nv_bfloat16*)q;
  p.o = (const __nv_bfloat16*)o;
  p.dout = (const __nv_bfloat16*)dout;
  p.lse = lse;
  p.nlse2 = (float*)workspace;
  p.ndsum = (float*)((uint8_t*)workspace + l.dsum);
  p.part = (float*)((uint8_t*)workspace + l.part);
  p.near = (float*)((uint8_t*)workspace + l.near);
  p.n_near = l.n_near;
  p.dq = (__nv_bfloat16*)dq;
  p.dk = (__nv_bfloat16*)dk;
  p.dv = (__nv_bfloat16*)dv;
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.tpc = l.tpc;
  p.cols = span::up16(l.tpc * p.R);
  p.window = window;
  p.n_sink = n_sink;
  p.n_far = l.n_far;
  p.far_tokens = l.far_tokens;
  p.sink_tiles = l.sink_tiles;
  p.sink_rows = l.sink_rows;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  return d == 64 ? span::launch_bwd_d<64>(p, l, st) : span::launch_bwd_d<128>(p, l, st);
}

NSA_STATUS_ACCESSOR(span_bwd)

}  // namespace nsa
