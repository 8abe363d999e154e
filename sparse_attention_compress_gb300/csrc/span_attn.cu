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
// read once for the whole group.  Three forms of one kernel:
//   long        a CTA (one an SM) holds two row tiles ("halves", four softmax warps each, one
//               row a thread) over common K and V rings; while one half's softmax runs the
//               tensor cores work for the other.  Bound by the tensor cores and, beside them,
//               by the instructions that turn S into P: 2048 tokens x 64 heads at 32768 keys,
//               d = 128, 1.46 ms (1460 TFLOP/s, 77% of a large library product).
//   short       (spans of at most 16 key tiles) a CTA holds one row tile over one ring, so
//               that two CTAs share an SM and a start or an end, which the few tiles do not
//               hide, runs beside the other's products: 65536 tokens x 64 heads, window 512,
//               1.54 ms (1.65 in the long form).
//   few         (a decode step, a few speculative tokens: at most 48 rows a sequence and
//               kv-head) as short, Q taking only the rows it has and the ring the rest, for
//               HBM: 32 tokens over caches of 16384 to 32768 keys x 2 kv-heads 146 us
//               (5.5 TB/s, 81% of a copy); one token over 4096 keys 15 us on the device (25 us
//               a call from Python), the length of its two launches and of one CTA's start
//               and end.  The rows past Q's are whatever lies there and stay in their own lanes.
// Work units (row tile, sequence, kv-head) that would not fill the SMs evenly have their keys
// divided over several CTAs: each leaves (max, sum, unnormalised o) in the workspace and
// combine_kernel joins them in a fixed order.  Roles: softmax warps (one row a thread),
// loading warps (TMA, span.cuh), one warp that issues the products.
// TMEM: S of half x at 128 x with P over its first columns, then O of the halves.
// V is used as it lies (MN-major B operand), so nothing is transposed.
#include <algorithm>
#include <atomic>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

// Registers a thread: the softmax warps keep a row of 128 scores, the others next to nothing.
constexpr int kSoftRegs = 208;
// P may exceed 1 by 2^kLazy before the running maximum moves: the floating-point formats of
// P, of the sums and of O hold it with the same relative precision.
constexpr float kLazy = 16.f;
// But a key that outweighs half of all before it moves the maximum at once: its P is then 1, which bf16
// holds, where otherwise the rounding of the one P that makes up the row would show.  (Window 512
// 1.520 -> 1.535 ms at 65536 tokens x 64 heads, window 64 19.7 -> 20.5 us at 8192 x 8, longer ones unchanged.)
constexpr float kOutweighs = -1.f;  // log2
constexpr int kFewRows = 48;  // what leaves room for two such CTAs on an SM beside three tiles each
constexpr int kSms = 152;
// Key tiles of a row tile up to which its CTA shares an SM.  32768 tokens x 64 heads (4 kv-heads,
// d = 128) short and long: window 64 392 and 461 us, 512 774 and 835, 1024 1127 and 1176, 2048
// 1838 and 1848, 4096 3202 and 3128; 1024 tokens x 16 heads, window 512, 14.8 and 16.9.
constexpr int kShortTiles = 16;

enum Form { kLong, kShort, kFew };

template <int D, int FORM>
struct Cfg {
  static constexpr bool ONE = FORM != kLong;
  static constexpr int NH = ONE ? 1 : 2;  // row tiles (halves)
  static constexpr int THREADS = ONE ? 256 : 384;
  static constexpr int KV_BYTES = KT * D * 2;
  // Two rings of tiles, for K and for V.  ONE: one ring holds K and V tiles in turn.
  static constexpr int N0 = D == 64 ? (FORM == kFew ? 6 : 5) : (FORM == kShort ? 2 : 3), N1 = ONE ? 0 : (D == 64 ? 5 : 2);
  static constexpr uint32_t TMEM = ONE ? 256 : 512;
  static constexpr int OTHER_REGS = ONE ? 40 : 56;
  // what the launch must give a thread for the shares to add up
  static constexpr int MIN_REGS = (NH * 128 * kSoftRegs + 128 * OTHER_REGS + THREADS - 1) / THREADS;
  // Shared memory of a launch whose Q has `rows` rows a half (few rows: as many as the call's,
  // to 16), and of the largest.
  static constexpr int smem(int rows) { return NH * (D / 64) * rows * 128 + (N0 + N1) * KV_BYTES + 1024; }
  static constexpr int MAX_SMEM = smem(FORM == kFew ? (kFewRows + GRAN - 1) / GRAN * GRAN : ROWS);
};

struct AttnParams {
  Seqs seqs;
  Keys keys;
  __nv_bfloat16* o;
  float* lse;     // optional
  float* part_o;    // [divided units][n_splits][cta_rows][D] fp32: unnormalised o
  float2* part_ml;  // [divided units][n_splits][cta_rows]: (running max in base-2 units, sum)
  int h, hkv, R, tpc, window, n_sink;
  int n_whole, n_splits, cta_rows, q_group;  // units 0 .. n_whole - 1 are not divided; q_group: bytes
                                             // between Q's 64-column groups
  float scale_log2;
};

// Unit u: row tile `rev` from a sequence's last (the longest spans first), sequence, kv-head.
struct Unit {
  int seq, g, t0, Lq;  // t0 < 0: no such rows
  int64_t start;
  __device__ __forceinline__ Unit(const AttnParams& p, int64_t u, int rows_tok) {
    g = (int)(u % p.hkv);
    seq = (int)(u / p.hkv % p.seqs.n_seqs);
    const int rev = (int)(u / p.hkv / p.seqs.n_seqs);
    start = seq_start(p.seqs, seq);
    Lq = seq_len(p.seqs, seq);
    t0 = ((Lq + rows_tok - 1) / rows_tok - 1 - rev) * rows_tok;
  }
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

template <int D, bool PAGED, int FORM>
__global__ void __launch_bounds__(Cfg<D, FORM>::THREADS, FORM == kLong ? 1 : 2)
    attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ CUtensorMap tm_o,
                const AttnParams p) {
  using C = Cfg<D, FORM>;
  constexpr bool ONE = C::ONE;  // one row tile, one ring of K and V in turn
  constexpr int NH = C::NH, N0 = C::N0, N1 = C::N1, NS = N0 + N1;
  using B = Bars<NS>;
  constexpr int kLoad0 = 4 * NH, kIssue = 4 * NH + 1, kLoad1 = ONE ? -1 : 4 * NH + 2;  // warps; 0 .. 4 NH - 1: softmax
  constexpr uint32_t kO = NH * 128;  // TMEM column of O
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B::COUNT];
  __shared__ uint32_t s_tmem, s_bad[8];  // s_bad: missing 16-row groups of tile i, at i % 8
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t q_bytes = (D / 64) * p.q_group;  // of a half
  const uint32_t q_s = base, slots = q_s + NH * q_bytes;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  if (stopped()) return;
  const Waits wait(abort);
  const int rows_tok = NH * p.tpc;  // tokens of this CTA
  const bool whole = (int64_t)blockIdx.x < p.n_whole;
  const int64_t part_unit = whole ? 0 : ((int64_t)blockIdx.x - p.n_whole) / p.n_splits;
  const int split = whole ? 0 : (int)(((int64_t)blockIdx.x - p.n_whole) % p.n_splits), n_splits = whole ? 1 : p.n_splits;
  const Unit un(p, whole ? (int64_t)blockIdx.x : p.n_whole + part_unit, rows_tok);
  if (un.t0 < 0) return;
  const int seq = un.seq, g = un.g, t0 = un.t0, Lq = un.Lq;
  const int64_t start = un.start;
  const int kv_len = PAGED ? cached_len(p.keys, seq) : Lq;
  const int off = kv_len - Lq;  // position of the sequence's first query
  const Tiles tiles(off + t0, off + min(t0 + rows_tok, Lq) - 1, p.window, p.n_sink);
  const int a = (int)((int64_t)tiles.n * split / n_splits);
  const int n = (int)((int64_t)tiles.n * (split + 1) / n_splits) - a;  // this CTA's tiles: a .. a + n - 1
  const int nh = !ONE && t0 + p.tpc < Lq ? 2 : 1;  // halves that have rows

  if (tid == 0) {
    tc::mbar_init(bar(B::Q), 1);
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(bar(B::FULL + i), 1);
      tc::mbar_init(bar(B::EMPTY + i), nh);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(B::SFULL + i), 1);
      tc::mbar_init(bar(B::PFULL + 2 * i), 4);  // one arrival a softmax warp
      tc::mbar_init(bar(B::PFULL + 2 * i + 1), 4);
      tc::mbar_init(bar(B::ODONE + i), 1);
    }
    tc::mbar_init(bar(B::DRAIN), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kIssue) {
    tmem_alloc(smem_u32(&s_tmem), C::TMEM);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_item = -1;  // loading warps: the last item handed to their ring
  // (each warpgroup states its register share in its own branch: the compiler allots by branch)
  if (warp >= 4 * NH) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::OTHER_REGS));
  if (warp == kLoad0 || warp == kLoad1) {
    // ------------------------------------------------------------------ loads of ring y
    const int y = warp == kLoad0 ? 0 : 1;
    if (y == 0 && lane == 0 && n > 0) {
      tc::mbar_expect_tx(bar(B::Q), (uint32_t)(nh * p.tpc * p.R * D * 2));
      for (int x = 0; x < nh; ++x)
        for (int c = 0; c < D / 64; ++c)
          tc::tma3d(q_s + x * q_bytes + c * p.q_group, &tm_q, c * 64, g * p.R, (int)(start + t0 + x * p.tpc), bar(B::Q));
    }
    __syncwarp();
    const int cnt = ONE ? 2 * n : n, ns = y ? N1 : N0, first = y ? N0 : 0;
    int slot = 0;
    uint32_t phase = 1;
    for (int i = 0; i < cnt; ++i) {
      const int j = ONE ? i >> 1 : i;
      const bool is_v = ONE ? (i & 1) : y == 1;
      if (i >= ns && !wait(bar(B::EMPTY + first + slot), phase)) break;
      // the flags of a tile are read by its softmax after S, so they are in place before the
      // K tile's arrival; the missing pages of K and V are the same
      if (PAGED && !is_v) {
        const uint32_t bad = missing_groups(p.keys, seq, tiles, a + j, kv_len, lane);
        if (lane == 0) s_bad[j & 7] = bad;
        __syncwarp();
      }
      load_tile<D, PAGED>(slots + (first + slot) * C::KV_BYTES, is_v ? &tm_v : &tm_k, is_v ? &tm_v16 : &tm_k16,
                          is_v ? p.keys.v : p.keys.k, p.keys, p.hkv, g, seq, start, (a + j) * KT,
                          tiles.sink_end, tiles.shift, tiles.width(a + j), kv_len, bar(B::FULL + first + slot), lane);
      last_item = i;
      if (++slot == ns) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------------------ products
    // One warp issues for both halves in turn: PV and the next S of a half go out together,
    // so the halves run half a tile apart.  (Two issuers' products interleave on the pipe and
    // end together; the halves then form their P at the same time and the tensor cores wait
    // for both.)
    bool ok = n == 0 || wait(bar(B::Q), 0);
    Ring<N0> rk;
    Ring<ONE ? N0 : N1> rv;  // ONE: the same ring, one item on
    constexpr int first_v = ONE ? 0 : N0;
    if (ONE) rv.next();
    auto next = [&](auto& r) {
      r.next();
      if (ONE) r.next();
    };
    const uint32_t lead = elect(), q_d = desc_k(q_s), slots_k = desc_k(slots), slots_v = desc_mn(slots);
    constexpr uint32_t kSlot = C::KV_BYTES >> 4;  // in descriptor units
    auto issue_s = [&](int x, int w) {
      mma_abt<D>(tmem + x * 128, q_d + x * (q_bytes >> 4), slots_k + rk.slot * kSlot, w, lead, p.q_group >> 4);
      commit(bar(B::SFULL + x), lead);
      commit(bar(B::EMPTY + rk.slot), lead);
    };
    int w = tiles.width(a);
    if (ok && n > 0) {
      ok = wait(bar(B::FULL + rk.slot), rk.phase);
      if (ok) {
        tc::fence_after();
        for (int x = 0; x < nh; ++x) issue_s(x, w);
      }
      next(rk);
    }
    for (int it = 0; ok && it < n; ++it) {
      const bool more = it + 1 < n;
      const int w_next = more ? tiles.width(a + it + 1) : 0;
      const uint32_t vs = slots_v + (first_v + rv.slot) * kSlot;
      if (!(ok = wait(bar(B::FULL + first_v + rv.slot), rv.phase))) break;
      for (int x = 0; ok && x < nh; ++x) {
        const uint32_t s_t = tmem + x * 128, o_t = tmem + kO + x * 128;
        // the first 64 keys' product runs while the softmax forms the others
        if (!(ok = wait(bar(B::PFULL + 2 * x), it & 1))) break;
        tc::fence_after();
        mma_pv<D, 0, 4>(o_t, s_t, vs, w, it == 0, lead);
        if (more && !(ok = wait(bar(B::FULL + rk.slot), rk.phase))) break;
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
  } else if (warp < 4 * NH) {
    // ------------------------------------------------------------------ softmax of half x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    const int x = warp >> 2, row = tid & 127, cnt = x < nh ? n : 0;
    const int tl = row / p.R, hd = row % p.R, t = t0 + x * p.tpc + tl;
    const bool valid = tl < p.tpc && t < Lq;
    const int pos = valid ? off + t : -1;
    const bool work = __any_sync(0xffffffffu, pos >= 0);  // warps without rows only keep the barriers moving
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + x * 128 + lane_base, o_t = tmem + kO + x * 128 + lane_base;
    float m = kNegInf, l = 0.f, lim = kNegInf;  // lim: what a score must exceed for the maximum to move
    bool ok = true;
    for (int it = 0; it < cnt; ++it) {
      const int key0 = tiles.key0(a + it), w = tiles.width(a + it);
      if (!(ok = wait(bar(B::SFULL + x), it & 1))) break;
      tc::fence_after();
      if (work) {
        float sv[KT];
        tc::tmem_ld32_nowait(s_t, sv);
        tmem_ld32_if(w > 32, s_t + 32, sv + 32);
        // seen columns: [j_lo, j_hi) and the sinks [0, j_sink) before j_hi
        const int j_hi = min(pos + 1 - key0, w);
        const int j_lo = p.window > 0 ? pos - p.window + 1 - key0 : 0, j_sink = tiles.sinks(a + it, p.n_sink);
        const uint32_t bad = PAGED ? s_bad[it & 7] : 0u;
        const bool all =
            __all_sync(0xffffffffu, j_hi == KT && (j_lo <= 0 || j_sink >= KT) && bad == 0);
        // columns c .. c + 31 that are not seen get -inf
        auto mask = [&](int c) {
          uint32_t see = bits(j_lo - c, j_hi - c) | bits(0, min(j_sink, j_hi) - c);
          if (PAGED) {
            const uint32_t b2 = (bad >> (c / GRAN)) & 3u;
            see &= ~((b2 & 1u ? 0xffffu : 0u) | (b2 & 2u ? 0xffff0000u : 0u));
          }
          if (__all_sync(0xffffffffu, see == ~0u)) return;  // (a boundary crosses one or two of the four)
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
        tmem_ld32_if(w > 64, s_t + 64, sv + 64);
        tmem_ld32_if(w > 96, s_t + 96, sv + 96);
        if (!all) {
          mask(0);
          mask(32);
        }
        // the first 64 exponentials are taken with the maximum so far, while the other scores
        // arrive and the tile's own maximum is found; the running maximum moves (and they are
        // taken again) only when a score exceeds it by 2^kLazy or outweighs the row so far
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
        const bool need = mx > lim;
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
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::PFULL + 2 * x));  // P of the first 64 keys
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
        lim = m + fminf(kLazy, __log2f(l) + kOutweighs);
      } else if (lane == 0) {
        tc::mbar_arrive(bar(B::PFULL + 2 * x));
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B::PFULL + 2 * x + 1));
    }
    if (ok && cnt > 0) {
      ok = wait(bar(B::ODONE + x), 0);
      tc::fence_after();
    }
    if (ok && x < nh) {
      const int64_t rr = (start + t) * p.h + g * p.R + hd;
      if (!whole) {
        const int64_t at = (part_unit * p.n_splits + split) * p.cta_rows + x * p.tpc * p.R + row;
        if (valid) p.part_ml[at] = make_float2(m, l);
        if (__any_sync(0xffffffffu, l > 0.f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tc::tmem_ld32(o_t + c, ov);
            if (valid && l > 0.f) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(p.part_o + at * D + c + e) =
                    make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            }
          }
        }
      } else {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const uint32_t stage = q_s + x * q_bytes;  // the half's Q, which its last S has read
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          tmem_ld32_if(n > 0, o_t + c, ov);  // (the whole warp's load)
          tmem_wait_ld(ov);
          if (!(l > 0.f)) {  // a row without keys holds no product
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = 0.f;
          }
          if (row < p.tpc * p.R) stage_cols(stage, p.q_group, row, c, ov, inv);
        }
        if (p.lse && valid) p.lse[rr] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
      }
    }
    if (whole && x < nh) {
      const int tx = t0 + x * p.tpc;
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      named_barrier(1 + x, 128);  // (also after a timeout: every warp of the half comes here)
      if (ok && tx + p.tpc <= Lq) {
        if (row == 0) store_tile<D>(&tm_o, q_s + x * q_bytes, p.q_group, g * p.R, (int)(start + tx));
      } else if (ok) {  // the box would reach into the next sequence
        unstage_rows<D>(q_s + x * q_bytes, p.q_group, p.tpc * p.R, p.R, p.h, Lq - tx,
                        p.o + ((start + tx) * p.h + g * p.R) * D, row, 128);
      }
    }
  }

  __syncthreads();
  if (*abort) {
    // copies and products still in flight land before the CTA leaves
    if (warp == kLoad0 || warp == kLoad1) {
      if (warp == kLoad0 && n > 0) tc::warp_drain(bar(B::Q), 0);
      const int ns = warp == kLoad0 ? N0 : N1, first = warp == kLoad0 ? 0 : N0;
      for (int st = 0; st < ns; ++st)
        if (const int i = last_in_stage(last_item, st, ns); i >= 0)
          tc::warp_drain(bar(B::FULL + first + st), (i / ns) & 1);
    } else if (warp == kIssue) {
      commit(bar(B::DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(B::DRAIN), 0);
    }
  } else if (warp == kLoad0 || warp == kLoad1) {
    // the last release of every slot lands before the CTA leaves
    const int ns = warp == kLoad0 ? N0 : N1, first = warp == kLoad0 ? 0 : N0;
    for (int st = 0; st < ns; ++st)
      if (const int i = last_in_stage(last_item, st, ns); i >= 0)
        tc::warp_drain(bar(B::EMPTY + first + st), (i / ns) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_free(tmem, C::TMEM);
}

// Joins the parts of a row in order: PW warps a (token, head) row, each every PW-th part
// (eight warps where there are many parts, whose loads would otherwise wait for one
// another), then a sum over the warps.  Reads every part once (a part without keys is
// skipped), writes bf16 o and the lse.
template <int D, int PW>
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p, int64_t rows) {
  constexpr int E = D / 32;
  __shared__ float s_acc[8][D + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pw = warp % PW;
  const int64_t row = (int64_t)blockIdx.x * (8 / PW) + warp / PW;  // of the divided units
  const int parts = p.n_splits, R = p.R;
  const Unit un(p, p.n_whole + row / p.cta_rows, p.cta_rows / R);
  const int t = un.t0 + (int)(row % p.cta_rows) / R;
  const bool mine = row < rows && un.t0 >= 0 && t < un.Lq;
  const int64_t rr = (un.start + t) * p.h + un.g * R + (int)(row % p.cta_rows) % R;
  const int64_t at = row / p.cta_rows * parts * p.cta_rows + row % p.cta_rows;  // of part 0
  float m = kNegInf, acc[E] = {}, l = 0.f;
  if (mine) {
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[at + (int64_t)i * p.cta_rows].x);
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    if (m > kNegInf) {
      for (int i0 = pw; i0 < parts; i0 += 32 * PW) {
        float wl = 0.f, w = 0.f;
        if (i0 + lane * PW < parts) {
          const float2 ml = p.part_ml[at + (int64_t)(i0 + lane * PW) * p.cta_rows];
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
            const float* src = p.part_o + (at + (int64_t)(i0 + i * PW) * p.cta_rows) * D + lane * E;
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

// How a call is cut.  The number of key tiles follows from the longest cache and the window.
struct Plan {
  int form;
  int tpc, cta_rows, n_splits;
  int64_t units, whole;  // units 0 .. whole - 1 take one CTA, the others n_splits
  size_t ml, bytes;      // workspace: part_o at 0, part_ml at `ml`
};
Plan make_plan(const Seqs& s, int h, int hkv, int D, int max_keys, int window, int n_sink) {
  Plan pl{};
  const int R = h / hkv;
  pl.tpc = std::max(1, std::min(ROWS / R, s.max_len));
  int64_t span = max_keys;  // keys of a row tile
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + pl.tpc + up16(n_sink) + 2 * GRAN);
  pl.form = (int64_t)s.max_len * R <= kFewRows ? kFew : span <= kShortTiles * KT ? kShort : kLong;
  const int rows_tok = pl.form != kLong ? pl.tpc : 2 * pl.tpc;
  pl.cta_rows = rows_tok * R;
  pl.units = ((int64_t)s.max_len + rows_tok - 1) / rows_tok * s.n_seqs * hkv;
  int64_t keys = max_keys;
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + rows_tok + up16(n_sink) + 2 * GRAN);
  const int64_t tiles = std::max<int64_t>(1, (keys + KT - 1) / KT);
  if (pl.form == kShort) {
    pl.n_splits = 1;
    pl.whole = pl.units;
  } else if (pl.form == kFew) {
    // At most four rounds of CTAs (two an SM): ragged caches then even out, and a round is not
    // begun for a few.  32 caches of 16384 to 32768 keys: 146 us with 19 parts (four rounds),
    // 154 with 10 (2.1 rounds), 152 with 15 (3.2), 157 with 29 (6.1).
    const int64_t want = 4 * 2 * kSms / pl.units;
    pl.n_splits = (int)std::max<int64_t>(1, std::min<int64_t>({want, tiles, 256}));
    pl.whole = pl.n_splits == 1 ? pl.units : 0;
  } else {
    // Whole rounds of the SMs as they are; the units of the last, partial round are divided
    // where that shortens it.  In the time of a key tile (1.6 us at d = 128): a CTA takes its
    // tiles and about 5 more to start and end, each part about 3 to pass through memory.  The
    // chunk of 2048 tokens x 64 heads at 32768 keys (512 units, 56 of them in the last round)
    // takes 1463 us with those in 5 parts, 1507 in 8 and 1684 undivided; 224 units of 10
    // tiles 30 us undivided and 43 us with the last 72 halved.
    const int64_t rest = pl.units % kSms;
    double best = 1e30;
    pl.n_splits = 1;
    for (int sp = 1; rest > 0 && sp <= 16 && (sp == 1 || 2 * sp <= tiles); ++sp) {
      const double cost = (double)((rest * sp + kSms - 1) / kSms) * ((double)tiles / sp + 5.0) + (sp > 1 ? 3.0 * sp : 0.0);
      if (cost < best) {
        best = cost;
        pl.n_splits = sp;
      }
    }
    pl.whole = pl.n_splits == 1 ? pl.units : pl.units - rest;
  }
  const size_t rows = (size_t)(pl.units - pl.whole) * pl.n_splits * pl.cta_rows;
  pl.ml = (rows * D * 4 + 255) & ~size_t(255);
  pl.bytes = rows ? pl.ml + rows * 8 : 0;
  return pl;
}

template <int D, bool PAGED, int FORM>
cudaError_t run_attn(const CUtensorMap* m, const AttnParams& p, int64_t ctas, cudaStream_t st) {
  using C = Cfg<D, FORM>;
  auto kern = attn_kernel<D, PAGED, FORM>;
  // (the limit belongs to the kernel, and other threads launch it too: the same for every call)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::MAX_SMEM);
  if (e != cudaSuccess) return e;
  // the softmax warps' share must come out of what the block is launched with
  static std::atomic<int> kernel_regs{0};
  int regs = kernel_regs.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    kernel_regs.store(regs = at.numRegs, std::memory_order_relaxed);
  }
  if (regs < C::MIN_REGS) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)ctas, C::THREADS, C::smem(p.q_group / 128), st>>>(m[0], m[1], m[2], m[3], m[4], m[5], p);
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
  p.part_o = (float*)workspace;
  p.part_ml = (float2*)((uint8_t*)workspace + pl.ml);
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.tpc = pl.tpc;
  p.window = window;
  p.n_sink = n_sink;
  p.n_whole = (int)pl.whole;
  p.n_splits = pl.n_splits;
  p.cta_rows = pl.cta_rows;
  p.q_group = pl.form == kFew ? up16(pl.cta_rows) * 128 : ROWS * 128;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap m[6];
  if (!query_map(&m[5], o, s.tokens, h, D, p.R, p.tpc) ||
      !query_map(&m[0], q, s.tokens, h, D, p.R, p.tpc) || !key_maps(&m[1], &m[2], keys.k, keys, hkv, D, s.tokens) ||
      !key_maps(&m[3], &m[4], keys.v, keys, hkv, D, s.tokens))
    return cudaErrorInvalidValue;
  const int64_t ctas = pl.whole + (pl.units - pl.whole) * pl.n_splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto run = [&](auto form) {
    constexpr int F = decltype(form)::value;
    return keys.table ? run_attn<D, true, F>(m, p, ctas, st) : run_attn<D, false, F>(m, p, ctas, st);
  };
  cudaError_t e = pl.form == kFew     ? run(std::integral_constant<int, kFew>{})
                  : pl.form == kShort ? run(std::integral_constant<int, kShort>{})
                                      : run(std::integral_constant<int, kLong>{});
  if (e != cudaSuccess || pl.bytes == 0) return e;
  const int64_t rows = (pl.units - pl.whole) * pl.cta_rows;
  if (pl.n_splits >= 8)
    combine_kernel<D, 8><<<(unsigned)rows, 256, 0, st>>>(p, rows);
  else
    combine_kernel<D, 1><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p, rows);
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
