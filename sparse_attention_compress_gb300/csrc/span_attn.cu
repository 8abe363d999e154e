// Attention of a chunk of new tokens over a paged cache, and of packed sequences under a
// sliding window with sinks: per (token, head) row at position p,
//   s_j = scale q.k_j over the keys p sees (span.cuh),  lse = log sum_j exp s_j,
//   o = sum_j exp(s_j - lse) v_j;   a row that sees no key gets o = 0, lse = -inf.
// One pass over the keys with a running maximum and sum, base-2 exponentials, all
// statistics and accumulators in fp32; P enters the second product as bf16 (half a step,
// 2^-8 relative on each weight, which averages out over a row's keys and stays below the
// rounding of the bf16 output itself).
//
// A tile is 128 rows = 128 / group tokens x the heads of a kv-group, so each K / V tile is
// read once for the whole group.  A CTA holds two such row tiles ("halves", four softmax
// warps each, one row a thread) over one K / V ring: while one half's softmax runs, the
// tensor cores work for the other.  With few rows (a decode step, or chunks whose rows fit
// one tile: SPLIT) both halves take the same rows and alternate key tiles instead, and the
// keys are also divided over CTAs; every part leaves (max, sum, unnormalised o) in the
// workspace and combine_kernel joins them in a fixed order.  Roles: warps 0-7 softmax,
// warps 8 and 11 load (TMA, span.cuh), warp 9 (SPLIT: and 10) issues the products.
// TMEM (512 columns): S of half x at 128 x with P over its first columns, O at 256 + 128 x.
// V is used as it lies (MN-major B operand), so nothing is transposed.
#include <algorithm>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

constexpr int kThreads = 384;
// Registers a thread: the softmax warps keep a row of 128 scores, the others next to nothing.
constexpr int kSoftRegs = 208, kOtherRegs = 56, kMinRegs = 160;  // 256 * 208 + 128 * 56 <= 384 * 160
constexpr uint32_t kTmemCols = 512;
// P may exceed 1 by 2^kLazy before the running maximum moves: the floating-point formats of
// P, of the sums and of O hold it with the same relative precision.
constexpr float kLazy = 16.f;

template <int D, bool SPLIT>
struct Cfg {
  static constexpr int NQ = SPLIT ? 1 : 2;  // row tiles in shared memory
  static constexpr int Q_BYTES = ROWS * D * 2;
  static constexpr int KV_BYTES = KT * D * 2;
  // Two rings of tiles.  Otherwise K tiles go through ring 0 and V tiles through ring 1, read
  // by both halves; SPLIT: ring x is half x's own and holds its K and V tiles in turn, so
  // that every wait sees every phase of its slot (halves that took alternate items of one
  // ring would skip phases, and mistake the one before for the one they wait for).
  static constexpr int N0 = D == 64 ? (SPLIT ? 6 : 5) : 3, N1 = D == 64 ? (SPLIT ? 6 : 5) : (SPLIT ? 3 : 2);
  static constexpr int SMEM = NQ * Q_BYTES + (N0 + N1) * KV_BYTES + 1024;
};

// Position in a ring of n slots: the slot and the parity of its phase.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

struct AttnParams {
  Seqs seqs;
  Keys keys;
  __nv_bfloat16* o;
  float* lse;     // optional
  float* part_o;  // [parts][tokens * h][D] fp32, or null: one part, written to o
  float2* part_ml;  // [parts][tokens * h] (running max in base-2 units, sum)
  int h, hkv, R, tpc, window, n_sink, n_splits;
  float scale_log2;
};

template <int NS>
struct Bars {
  enum : int {
    Q = 0,
    FULL = 1,             // [NS] ring 0's slots, then ring 1's
    EMPTY = FULL + NS,
    SFULL = EMPTY + NS,   // [2] by half
    PFULL = SFULL + 2,    // [2][2] by half and 64-key part
    ODONE = PFULL + 4,    // [2] the half's last product is done
    DRAIN = ODONE + 2,
    COUNT = DRAIN + 1
  };
};

// Index of the last of tiles 0..last that went to ring stage st (-1 if none).
__device__ __forceinline__ int last_in_stage(int last, int st, int ns) {
  return last < st ? -1 : last - (last - st) % ns;
}

template <int D, bool PAGED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_v16, const AttnParams p) {
  using C = Cfg<D, SPLIT>;
  constexpr int N0 = C::N0, N1 = C::N1, NS = N0 + N1;
  using B = Bars<NS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B::COUNT];
  __shared__ uint32_t s_tmem, s_bad[2][8];  // s_bad: missing 16-row groups of a half's (else any) tile i, at i % 8
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t q_s = base, slots = q_s + C::NQ * C::Q_BYTES;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  if (tc::device_status_set()) return;
  const Waits wait(abort);
  const int seq = blockIdx.y, g = blockIdx.z / p.n_splits, split = blockIdx.z % p.n_splits;
  const int64_t start = seq_start(p.seqs, seq);
  const int Lq = seq_len(p.seqs, seq);
  const int rows_tok = C::NQ * p.tpc;  // tokens of this CTA
  const int t0 = ((Lq + rows_tok - 1) / rows_tok - 1 - (int)blockIdx.x) * rows_tok;  // longest spans first
  if (t0 < 0) return;
  const int kv_len = PAGED ? cached_len(p.keys, seq) : Lq;
  const int off = kv_len - Lq;  // position of the sequence's first query
  const Tiles tiles(off + t0, off + min(t0 + rows_tok, Lq) - 1, p.window, p.n_sink);
  const int a = (int)((int64_t)tiles.n * split / p.n_splits);
  const int n = (int)((int64_t)tiles.n * (split + 1) / p.n_splits) - a;  // this CTA's tiles: a .. a + n - 1
  const bool two = SPLIT || t0 + p.tpc < Lq;  // the second half has rows
  // tiles of half x: every one, or (SPLIT) every second one
  auto count_of = [&](int x) { return SPLIT ? (n + 1 - x) >> 1 : (x == 0 || two ? n : 0); };
  auto tile_of = [&](int x, int it) { return SPLIT ? 2 * it + x : it; };

  if (tid == 0) {
    const int users = !SPLIT && two ? 2 : 1;
    tc::mbar_init(bar(B::Q), 1);
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(bar(B::FULL + i), 1);
      tc::mbar_init(bar(B::EMPTY + i), users);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(B::SFULL + i), 1);
      tc::mbar_init(bar(B::PFULL + 2 * i), 128);
      tc::mbar_init(bar(B::PFULL + 2 * i + 1), 128);
      tc::mbar_init(bar(B::ODONE + i), 1);
    }
    tc::mbar_init(bar(B::DRAIN), 2);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_item = -1;  // loading warps: the last item handed to their ring
  // (each warpgroup states its register share in its own branch: the compiler allots by branch)
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
  if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------------ loads of ring y
    const int y = warp == 8 ? 0 : 1;
    if (y == 0 && lane == 0 && n > 0) {
      const int nq = two && !SPLIT ? 2 : 1;
      tc::mbar_expect_tx(bar(B::Q), (uint32_t)(nq * p.tpc * p.R * D * 2));
      for (int x = 0; x < nq; ++x)
        for (int c = 0; c < D / 64; ++c)
          tc::tma3d(q_s + x * C::Q_BYTES + c * (ROWS * 128), &tm_q, c * 64, g * p.R, (int)(start + t0 + x * p.tpc),
                    bar(B::Q));
    }
    __syncwarp();
    const int cnt = SPLIT ? 2 * count_of(y) : n, ns = y ? N1 : N0, first = y ? N0 : 0;
    int slot = 0;
    uint32_t phase = 1;
    for (int i = 0; i < cnt; ++i) {
      const int it = SPLIT ? i >> 1 : i, j = SPLIT ? 2 * it + y : i;
      const bool is_v = SPLIT ? (i & 1) : y == 1;
      const int key0 = tiles.key0(a + j), w = tiles.width(a + j);
      if (i >= ns && !wait(bar(B::EMPTY + first + slot), phase)) break;
      // the flags of a tile are read by its softmax after S, so they are in place before the
      // K tile's arrival; the missing pages of K and V are the same
      if (PAGED && !is_v) {
        const uint32_t bad = missing_groups(p.keys, seq, key0, w, kv_len, lane);
        if (lane == 0) s_bad[SPLIT ? y : 0][it & 7] = bad;
        __syncwarp();
      }
      load_tile<D, PAGED>(slots + (first + slot) * C::KV_BYTES, is_v ? &tm_v : &tm_k, is_v ? &tm_v16 : &tm_k16,
                          is_v ? p.keys.v : p.keys.k, p.keys, p.hkv, g, seq, start, key0, w, kv_len,
                          bar(B::FULL + first + slot), lane);
      last_item = i;
      if (++slot == ns) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 9 || (SPLIT && warp == 10)) {
    // ------------------------------------------------------------------ products
    // SPLIT: each warp issues for its own half, as its softmax proceeds.  Otherwise one warp
    // issues for both in turn: PV and the next S of a half go out together, so the halves run
    // half a tile apart.  (Two issuers' products interleave on the pipe and end together;
    // the halves then form their P at the same time and the tensor cores wait for both.)
    const int x0 = SPLIT ? warp - 9 : 0, nx = SPLIT ? 1 : (two ? 2 : 1), cnt = count_of(x0);
    bool ok = cnt == 0 || wait(bar(B::Q), 0);
    // K and V items: one ring of the half's own (SPLIT), or the two common rings
    Ring<N0> rk;
    Ring<N1> rv;
    const int first_k = SPLIT ? x0 * N0 : 0, first_v = SPLIT ? x0 * N0 : N0;
    if (SPLIT) rv.next();
    auto next = [&](auto& r) {
      r.next();
      if (SPLIT) r.next();
    };
    const uint32_t lead = elect(), q_d = desc_k(q_s), slots_k = desc_k(slots), slots_v = desc_mn(slots);
    constexpr uint32_t kSlot = C::KV_BYTES >> 4;  // in descriptor units
    auto issue_s = [&](int x, int w) {
      mma_abt<D>(tmem + x * 128, q_d + (SPLIT ? 0 : x * (C::Q_BYTES >> 4)), slots_k + (first_k + rk.slot) * kSlot, w,
                 lead);
      commit(bar(B::SFULL + x), lead);
      commit(bar(B::EMPTY + first_k + rk.slot), lead);
    };
    int w = tiles.width(a + tile_of(x0, 0));
    if (ok && cnt > 0) {
      ok = wait(bar(B::FULL + first_k + rk.slot), rk.phase);
      if (ok) {
        tc::fence_after();
        for (int q = 0; q < nx; ++q) issue_s(x0 + q, w);
      }
      next(rk);
    }
    for (int it = 0; ok && it < cnt; ++it) {
      const bool more = it + 1 < cnt;
      const int w_next = more ? tiles.width(a + tile_of(x0, it + 1)) : 0;
      const uint32_t vs = slots_v + (first_v + rv.slot) * kSlot;
      if (!(ok = wait(bar(B::FULL + first_v + rv.slot), rv.phase))) break;
      for (int x = x0; ok && x < x0 + nx; ++x) {
        const uint32_t s_t = tmem + x * 128, o_t = tmem + 256 + x * 128;
        // the first 64 keys' product runs while the softmax forms the others
        if (!(ok = wait(bar(B::PFULL + 2 * x), it & 1))) break;
        tc::fence_after();
        mma_pv<D, 0, 4>(o_t, s_t, vs, w, it == 0, lead);
        if (more && !(ok = wait(bar(B::FULL + first_k + rk.slot), rk.phase))) break;
        if (!(ok = wait(bar(B::PFULL + 2 * x + 1), it & 1))) break;
        tc::fence_after();
        mma_pv<D, 4, 8>(o_t, s_t, vs, w, false, lead);
        commit(bar(B::EMPTY + first_v + rv.slot), lead);
        if (more)  // over P(it): this lane issued its product, and products execute in issue order
          issue_s(x, w_next);
        else
          commit(bar(B::ODONE + x), lead);
      }
      next(rk);
      next(rv);
      w = w_next;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax of half x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    const int x = warp >> 2, row = tid & 127, cnt = count_of(x);
    const int tl = row / p.R, hd = row % p.R, t = t0 + (SPLIT ? 0 : x * p.tpc) + tl;
    const bool valid = tl < p.tpc && t < Lq;
    const int pos = valid ? off + t : -1;
    const bool work = __any_sync(0xffffffffu, pos >= 0);  // warps without rows only keep the barriers moving
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + x * 128 + lane_base, o_t = tmem + 256 + x * 128 + lane_base;
    float m = kNegInf, l = 0.f;
    bool ok = true;
    for (int it = 0; it < cnt; ++it) {
      const int j = tile_of(x, it), key0 = tiles.key0(a + j), w = tiles.width(a + j);
      if (!(ok = wait(bar(B::SFULL + x), it & 1))) break;
      tc::fence_after();
      if (work) {
        float sv[KT];
        tc::tmem_ld32_nowait(s_t, sv);
        if (w > 32) tc::tmem_ld32_nowait(s_t + 32, sv + 32);
        // seen columns: [j_lo, j_hi) and, of those before j_lo, the sinks [0, j_sink)
        const int j_hi = min(pos + 1 - key0, w);
        const int j_lo = p.window > 0 ? pos - p.window + 1 - key0 : 0, j_sink = p.n_sink - key0;
        const uint32_t bad = PAGED ? s_bad[SPLIT ? x : 0][it & 7] : 0u;
        const bool all =
            __all_sync(0xffffffffu, j_hi == KT && (j_lo <= 0 || j_sink >= KT) && bad == 0);
        // columns c .. c + 31 that are not seen get -inf
        auto mask = [&](int c) {
          uint32_t see = bits(j_lo - c, j_hi - c) | bits(0, min(j_sink, j_hi) - c);
          if (PAGED) {
            const uint32_t b2 = (bad >> (c / GRAN)) & 3u;
            see &= ~((b2 & 1u ? 0xffffu : 0u) | (b2 & 2u ? 0xffff0000u : 0u));
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[c + e] = (see >> e) & 1u ? sv[c + e] : kNegInf;
        };
        float mx4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
        auto max_of = [&](int c) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            mx4[0] = max3(mx4[0], sv[c + e], sv[c + e + 1]);
            mx4[1] = max3(mx4[1], sv[c + e + 2], sv[c + e + 3]);
            mx4[2] = max3(mx4[2], sv[c + e + 4], sv[c + e + 5]);
            mx4[3] = max3(mx4[3], sv[c + e + 6], sv[c + e + 7]);
          }
        };
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
        uint64_t mu2, l2[4];  // minus the maximum, twice; four chains of two row sums
        uint32_t pk[32];
        // P of columns c .. c + 31 to pk[at ..]
        auto exps = [&](int c, int at) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = unpair(fma2(pair(sv[c + e], sv[c + e + 1]), scale2, mu2));
            const float e0 = ex2(y.x), e1 = ex2(y.y);
            l2[(e >> 1) & 3] = add2(l2[(e >> 1) & 3], pair(e0, e1));
            pk[at + e / 2] = pack_bf16(e0, e1);
          }
        };
        auto first_half = [&]() {
          const float mu = m == kNegInf ? 0.f : -m;
          mu2 = pair(mu, mu);
#pragma unroll
          for (int e = 0; e < 4; ++e) l2[e] = 0;
          exps(0, 0);
          exps(32, 16);
        };
        tmem_wait_ld(sv);
        tmem_wait_ld(sv + 32);
        if (w > 64) tc::tmem_ld32_nowait(s_t + 64, sv + 64);
        if (w > 96) tc::tmem_ld32_nowait(s_t + 96, sv + 96);
        if (!all) {
          mask(0);
          mask(32);
        }
        // the first 64 exponentials are taken with the maximum so far, while the other scores
        // arrive and the tile's own maximum is found; the running maximum moves (and they are
        // taken again) only when a score exceeds it by 2^kLazy
        if (it > 0) first_half();
        max_of(0);
        max_of(32);
        tmem_wait_ld(sv + 64);
        tmem_wait_ld(sv + 96);
        if (!all) {
          mask(64);
          mask(96);
        }
        max_of(64);
        max_of(96);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
        const bool need = mx > m + kLazy;
        if (__any_sync(0xffffffffu, need) || it == 0) {
          const float alpha = need ? ex2(m - mx) : 1.f;
          if (it > 0) {
            // S(it) followed PV(it - 1) on the tensor pipe, so O is complete here
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float ov[32];
              tc::tmem_ld32(o_t + c, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] *= alpha;
              tc::tmem_st32(o_t + c, reinterpret_cast<const uint32_t*>(ov));
            }
          }
          if (need) {
            l *= alpha;
            m = mx;
          }
          first_half();
        }
        tmem_st16_nowait(s_t, pk);
        if (w > 32) tmem_st16_nowait(s_t + 16, pk + 16);
        if (w > 64) exps(64, 0);
        tmem_wait_st();
        tc::fence_before();
        tc::mbar_arrive(bar(B::PFULL + 2 * x));  // P of the first 64 keys
        if (w > 64) {
          tmem_st16_nowait(s_t + 32, pk);
          if (w > 96) {
            exps(96, 16);
            tmem_st16_nowait(s_t + 48, pk + 16);
          }
          tmem_wait_st();
        }
        const float2 la = unpair(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
        l += la.x + la.y;
      } else {
        tc::fence_before();
        tc::mbar_arrive(bar(B::PFULL + 2 * x));
      }
      tc::fence_before();
      tc::mbar_arrive(bar(B::PFULL + 2 * x + 1));
    }
    if (ok && cnt > 0) {
      ok = wait(bar(B::ODONE + x), 0);
      tc::fence_after();
    }
    if (ok && (SPLIT || x == 0 || two)) {
      const int64_t rr = (start + t) * p.h + g * p.R + hd;
      if (SPLIT || p.part_o) {
        const int64_t at = (int64_t)(SPLIT ? split * 2 + x : split) * p.seqs.tokens * p.h + rr;
        if (valid) p.part_ml[at] = make_float2(m, l);
        if (__any_sync(0xffffffffu, l > 0.f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tc::tmem_ld32(o_t + c, ov);
            if (l > 0.f) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(p.part_o + at * D + c + e) =
                    make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            }
          }
        }
      } else {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          if (cnt > 0) tc::tmem_ld32(o_t + c, ov);
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (l > 0.f) {  // (a row without keys holds no product)
                v.x = pack_bf16(ov[e] * inv, ov[e + 1] * inv);
                v.y = pack_bf16(ov[e + 2] * inv, ov[e + 3] * inv);
                v.z = pack_bf16(ov[e + 4] * inv, ov[e + 5] * inv);
                v.w = pack_bf16(ov[e + 6] * inv, ov[e + 7] * inv);
              }
              *reinterpret_cast<uint4*>(p.o + rr * D + c + e) = v;
            }
          }
        }
        if (p.lse && valid) p.lse[rr] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
      }
    }
  }

  __syncthreads();
  if (*abort) {
    // copies and products still in flight land before the CTA leaves
    if (warp == 8 || warp == 11) {
      if (warp == 8 && n > 0) tc::warp_drain(bar(B::Q), 0);
      const int ns = warp == 8 ? N0 : N1, first = warp == 8 ? 0 : N0;
      for (int st = 0; st < ns; ++st)
        if (const int i = last_in_stage(last_item, st, ns); i >= 0)
          tc::warp_drain(bar(B::FULL + first + st), (i / ns) & 1);
    } else if (warp == 9 || warp == 10) {
      if (lane == 0) tc::commit(bar(B::DRAIN));
      __syncwarp();
      tc::warp_drain(bar(B::DRAIN), 0);
    }
  } else if (warp == 8 || warp == 11) {
    // the last release of every slot lands before the CTA leaves
    const int ns = warp == 8 ? N0 : N1, first = warp == 8 ? 0 : N0;
    for (int st = 0; st < ns; ++st)
      if (const int i = last_in_stage(last_item, st, ns); i >= 0)
        tc::warp_drain(bar(B::EMPTY + first + st), (i / ns) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 9) tmem_free(tmem, kTmemCols);
}

// Joins the parts of a row in order: PW warps a (token, head) row, each every PW-th part
// (eight warps where there are many parts, whose loads would otherwise wait for one
// another), then a sum over the warps.  Reads every part once (a part without keys is
// skipped), writes bf16 o and the lse.
template <int D, int PW>
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p, int parts) {
  constexpr int E = D / 32;
  __shared__ float s_acc[8][D + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pw = warp % PW;
  const int64_t rows = p.seqs.tokens * p.h;
  const int64_t rr = (int64_t)blockIdx.x * (8 / PW) + warp / PW;
  bool mine = rr < rows;
  if (mine) {
    const int64_t tok = rr / p.h;
    const int seq = seq_of_token(p.seqs, tok);
    const int64_t i = tok - seq_start(p.seqs, seq);
    mine = i >= 0 && i < seq_len(p.seqs, seq);  // (a row of no sequence is left alone)
  }
  float m = kNegInf, acc[E] = {}, l = 0.f;
  if (mine) {
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[i * rows + rr].x);
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    if (m > kNegInf) {
      for (int i0 = pw; i0 < parts; i0 += 32 * PW) {
        float wl = 0.f, w = 0.f;
        if (i0 + lane * PW < parts) {
          const float2 ml = p.part_ml[(int64_t)(i0 + lane * PW) * rows + rr];
          if (ml.y > 0.f) {
            w = ex2(ml.x - m);
            wl = w * ml.y;
          }
        }
        const int e1 = min(32, (parts - i0 + PW - 1) / PW);
#pragma unroll 4
        for (int i = 0; i < e1; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, wl, i);
          l += li;
          if (li > 0.f) {  // (an underflowed weight would only add zeros)
            const float* src = p.part_o + ((int64_t)(i0 + i * PW) * rows + rr) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float2 v = *reinterpret_cast<const float2*>(src + e);
              acc[e] += wi * v.x;
              acc[e + 1] += wi * v.y;
            }
          }
        }
      }
    }
  }
  if (PW > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
    if (lane == 0) s_acc[warp][D] = l;
    __syncthreads();
    if (pw != 0) return;
#pragma unroll
    for (int w = 1; w < PW; ++w) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += s_acc[warp + w][lane * E + e];
      l += s_acc[warp + w][D];
    }
  }
  if (!mine) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.o + rr * D + lane * E + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse && lane == 0) p.lse[rr] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
}

// How a call is cut.  Key tiles are bounded by the longest cache and the window.
struct Plan {
  bool split;    // one row tile a CTA, halves alternate key tiles
  int tpc, row_ctas, n_splits, parts;
  size_t ml, bytes;  // workspace: part_o at 0, part_ml at `ml`
};
Plan make_plan(const Seqs& s, int h, int hkv, int D, int max_keys, int window, int n_sink) {
  Plan pl{};
  const int R = h / hkv;
  pl.tpc = std::max(1, std::min(ROWS / R, s.max_len));
  // Few rows: every sequence's queries fit one row tile, so a second row tile would idle.
  pl.split = s.max_len <= pl.tpc;
  const int rows_tok = pl.split ? pl.tpc : 2 * pl.tpc;
  pl.row_ctas = (s.max_len + rows_tok - 1) / rows_tok;
  int64_t keys = max_keys;
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + rows_tok + up16(n_sink) + 2 * GRAN);
  const int64_t tiles = std::max<int64_t>(1, (keys + KT - 1) / KT);
  const int64_t ctas = std::max<int64_t>(1, (int64_t)pl.row_ctas * s.n_seqs * hkv);
  // Enough CTAs for about four rounds of the 152 SMs (ragged caches then even out), but no
  // part below two key tiles (a tile for each half).
  int64_t want = pl.split ? (4 * 152 + ctas - 1) / ctas : (152 + ctas - 1) / ctas;
  want = std::max<int64_t>(1, std::min<int64_t>(want, (tiles + 1) / 2));
  pl.n_splits = (int)std::min<int64_t>(want, std::min(256, 65535 / hkv));
  pl.parts = pl.split ? 2 * pl.n_splits : pl.n_splits;
  if (pl.parts > 1) {
    const size_t rows = (size_t)s.tokens * h;
    pl.ml = (pl.parts * rows * D * 4 + 255) & ~size_t(255);
    pl.bytes = pl.ml + pl.parts * rows * 8;
  }
  return pl;
}

template <int D, bool PAGED, bool SPLIT>
cudaError_t run_attn(const CUtensorMap* m, const AttnParams& p, dim3 grid, cudaStream_t st) {
  auto kern = attn_kernel<D, PAGED, SPLIT>;
  constexpr int smem = Cfg<D, SPLIT>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // the softmax warps' share must come out of what the block is launched with
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
  if (at.numRegs < kMinRegs) return cudaErrorInvalidConfiguration;
  kern<<<grid, kThreads, smem, st>>>(m[0], m[1], m[2], m[3], m[4], p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Seqs& s, const void* q, const Keys& keys, int h, int hkv, int max_keys, int window,
                     int n_sink, float scale, void* o, float* lse, void* workspace, cudaStream_t st) {
  const Plan pl = make_plan(s, h, hkv, D, max_keys, window, n_sink);
  AttnParams p{};
  p.seqs = s;
  p.keys = keys;
  p.o = (__nv_bfloat16*)o;
  p.lse = lse;
  if (pl.parts > 1) {
    p.part_o = (float*)workspace;
    p.part_ml = (float2*)((uint8_t*)workspace + pl.ml);
  }
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.tpc = pl.tpc;
  p.window = window;
  p.n_sink = n_sink;
  p.n_splits = pl.n_splits;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap m[5];
  if (!query_map(&m[0], q, s.tokens, h, D, p.R, p.tpc) || !key_maps(&m[1], &m[2], keys.k, keys, hkv, D, s.tokens) ||
      !key_maps(&m[3], &m[4], keys.v, keys, hkv, D, s.tokens))
    return cudaErrorInvalidValue;
  const dim3 grid(pl.row_ctas, s.n_seqs, hkv * pl.n_splits);
  cudaError_t e = keys.table ? (pl.split ? run_attn<D, true, true>(m, p, grid, st) : run_attn<D, true, false>(m, p, grid, st))
                             : (pl.split ? run_attn<D, false, true>(m, p, grid, st) : run_attn<D, false, false>(m, p, grid, st));
  if (e != cudaSuccess || pl.parts == 1) return e;
  const int64_t rows = s.tokens * h;
  if (pl.parts >= 8)
    combine_kernel<D, 8><<<(unsigned)rows, 256, 0, st>>>(p, pl.parts);
  else
    combine_kernel<D, 1><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p, pl.parts);
  return cudaGetLastError();
}

}  // namespace span

size_t span_attn_workspace_bytes(const Seqs& s, int h, int hkv, int d, int max_keys, int window, int n_sink) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return 0;
  return span::make_plan(s, h, hkv, d, max_keys, window, n_sink).bytes;
}

cudaError_t launch_span_attn(const Seqs& s, const void* q, const PagedView* cache, const void* k, const void* v, int h,
                             int hkv, int d, int max_keys, int window, int n_sink, float scale, void* o, float* lse,
                             void* workspace, cudaStream_t st) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return cudaSuccess;
  const span::Keys keys = span::keys_of(cache, k, v);
  return d == 64 ? span::launch_d<64>(s, q, keys, h, hkv, max_keys, window, n_sink, scale, o, lse, workspace, st)
                 : span::launch_d<128>(s, q, keys, h, hkv, max_keys, window, n_sink, scale, o, lse, workspace, st);
}

NSA_STATUS_ACCESSOR(span_attn)

}  // namespace nsa
