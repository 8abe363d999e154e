// Attention over a paged cache held in 8 bits: keys and values are e4m3 codes times a scale for each
// block of tokens and kv-head (paged_rope.cu), and the codes go to the tensor cores as they
// are.  Per (token, head) row at position p, over the keys that p sees (span.cuh),
//   t_j = scale sk_j q.k_j,   lse = log sum_j exp t_j,   o = sum_j exp(t_j - lse) sv_j v_j.
//
// The cache is the wide operand of both products, so that a few rows (a decode step) fill the
// tensor cores' M with keys and not with rows that do not exist:
//   S^T [128 keys x rows]  = K tile [128 keys x d] Q^T
//   O^T [d x rows]        += V tile^T [d x 128 keys] P^T
// (kind::f8f6f4; V is read MN-major, so nothing is transposed or converted).  Both partners
// have to be e4m3 as well, whose 4 significant bits would be too few, so they are sums of
// e4m3 terms that lie side by side in N, each with an accumulator column of its own:
//   Q  = 2^-a (q1 + q2 / 32)            a per row, so that max |Q 2^a| is in [128, 256)
//   P' = p1 + p2 / 32 + p3 / 1024       of P' = exp(t - m) sv 2^6 rounded to f16
// q1 + q2 / 32 holds a bf16 exactly down to 2^-14 of its row's largest, and to 2^-22 of that below.
// p1 + p2 / 32 + p3 / 1024 is within 2^-12 of P' (and P' within 2^-11 of its value, half a step
// of f16; a bf16 P has 2^-8), down to 2^-26 of the row's largest weight.
// A key's value scale sv is part of its weight, and the running maximum is that of t + log2 sv:
// what is held in few bits is what the sum is made of.  The row sum takes exp(t - m) alone.
//
// A thread of the softmax has one key and HR rows, so a mask is a bit mask over rows, scales are
// scalars of the thread, and only the running maximum has to be agreed on: it moves when some
// key exceeds it by 2^2 (P' has that room), which a vote finds out for each tile.
//
// Work units (row tile, sequence, kv-head) that would not fill the SMs have their keys divided
// over several CTAs, which leave (max, sum, unnormalised o); q8_combine_kernel joins them in order.
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

constexpr int kSms8 = 152;
constexpr float kRoom = 6.f, kMoves = 8.f;  // log2 of P' at the running maximum, and at which it moves
constexpr float kNone = -3e38f;             // running maximum of a row that has seen no key

struct Keys8 {
  const uint8_t *k, *v;
  const float *ks, *vs;  // [n_pages, hkv, page / block]
  Keys c;                // table, lens, sizes (page_stride in bytes; k, v unused)
  int block_log2;
};

template <int D, int NR>
struct Cfg8 {
  static constexpr int HR = NR / 2;  // rows a thread
  static constexpr int PER_SM = NR == 64 ? 1 : 2;
  static constexpr int THREADS = 352;  // 8 softmax warps, loads, products, scales
  static constexpr int TILE = KT * D;
  static constexpr int QN = 2 * NR, PN = 3 * NR;             // columns of S^T and O^T
  static constexpr int PG = (PN + 127) / 128;                // 128-column groups of P
  static constexpr int Q_BYTES = QN * D, P_BYTES = PG * KT * 128;  // of one P buffer
  static constexpr int NS = ((PER_SM == 2 ? 108 : 220) * 1024 - 2 * P_BYTES - Q_BYTES) / TILE > 16
                                ? 16
                                : ((PER_SM == 2 ? 108 : 220) * 1024 - 2 * P_BYTES - Q_BYTES) / TILE;
  static constexpr int SMEM = 2 * P_BYTES + NS * TILE + Q_BYTES + 1024;
  static constexpr uint32_t TMEM = NR == 64 ? 512 : NR == 32 ? 256 : 128;
  static constexpr uint32_t O_COL = 2 * QN;
  static_assert(O_COL + PN <= TMEM, "");
  static_assert(NS >= 4, "");
};

struct Q8Params {
  Seqs seqs;
  Keys8 keys;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;       // optional
  float* part_o;    // [units][n_splits][NR][D]
  float2* part_ml;  // [units][n_splits][NR]: (running maximum, sum)
  int h, hkv, R, window, n_sink, row_tiles, n_splits;
  float scale_log2;
};

// Unit u: row tile (rows are (token, head of the group), heads fastest), kv-head, sequence.
struct Unit8 {
  int seq, g, Lq, row0;
  int64_t start;
  __device__ __forceinline__ Unit8(const Q8Params& p, int64_t u, int nr) {
    const int rt = (int)(u % p.row_tiles);
    u /= p.row_tiles;
    g = (int)(u % p.hkv);
    seq = (int)(u / p.hkv);
    start = seq_start(p.seqs, seq);
    Lq = seq_len(p.seqs, seq);
    row0 = rt * nr;
  }
};

template <int NS>
struct Bars8 {
  enum : int {
    FULL = 0,
    EMPTY = NS,
    SFULL = 2 * NS,       // [2] S^T of a tile
    PFULL = SFULL + 2,    // [2] P of a tile
    PVDONE = PFULL + 2,   // [2] its product
    SCFULL = PVDONE + 2,  // [4] scales of four tiles
    SCEMPTY = SCFULL + 4,
    DRAIN = SCEMPTY + 4,
    COUNT
  };
};

// ------------------------------------------------------------------ byte tiles
// Row r of a tile of D-byte rows, 16-byte chunk ch, in the swizzle of D bytes (as TMA writes it).
template <int D>
__device__ __forceinline__ uint32_t at8(uint32_t base, int r, int ch) {
  return base + r * D + ((ch ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}
template <int D>
__device__ __forceinline__ void load_tile8(uint32_t dst, const CUtensorMap* big, const CUtensorMap* small,
                                           const uint8_t* src, const Keys& c, int hkv, int g, int seq, int place0,
                                           int sink_end, int shift, int w, int kv_len, uint32_t bar, int lane) {
  const int page = 1 << c.page_log2;
  const int box = page < KT ? page : KT;
  const int first = place0 + shift;
  const bool whole = w == KT && place0 >= sink_end && first + KT <= kv_len && (first & (box - 1)) == 0;
  const int br = whole ? box : GRAN;
  const int n = w / br;
  const bool mine = lane < n;
  const int place = place0 + lane * br, key = place < sink_end ? place : place + shift;
  const int pid = mine && key < kv_len ? page_of(c, seq, key) : 0;
  const bool ok = pid >= 0;
  const bool plain = mine && (!ok || key + br > kv_len);
  if (mine && !plain) tc::tma3d(dst + lane * br * D, whole ? big : small, g * D, key & (page - 1), pid, bar);
  const uint32_t bad = __ballot_sync(0xffffffffu, mine && !ok);
  uint32_t todo = __ballot_sync(0xffffffffu, plain);
  const int bytes = (n - __popc(todo)) * br * D;
  if (todo) {
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const bool okc = !((bad >> l) & 1u);
      const int64_t pidc = __shfl_sync(0xffffffffu, pid, l);
      const int keyc = __shfl_sync(0xffffffffu, key, l);
      for (int e = lane; e < br * (D / 16); e += 32) {
        const int r = l * br + e / (D / 16), ch = e % (D / 16), kk = keyc + e / (D / 16);
        const bool in = okc && kk < kv_len;
        const int64_t row = pidc * c.page_stride + (int64_t)(kk & (page - 1)) * hkv * D;
        cp_async16(at8<D>(dst, r, ch), in ? src + row + g * D + ch * 16 : src, in ? 16 : 0);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncwarp();
  if (lane == 0) tc::mbar_expect_tx(bar, (uint32_t)bytes);
}

// ------------------------------------------------------------------ products
// High word of a descriptor of tiles of B-byte rows in the B-byte swizzle: 8 rows to an atom.
template <int B>
constexpr uint32_t kDescHi8 = (uint32_t)(8 * B >> 4) | (1u << 14) | ((B == 128 ? 2u : 4u) << 29);
// e4m3 x e4m3 -> fp32, M x N; A and B MN-major where said.
constexpr uint32_t idesc8(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
template <uint32_t AHI, uint32_t BHI>
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum, uint32_t lead) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "mov.b64 x, {%1, %6};\nmov.b64 y, {%2, %7};\n"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accum), "r"(lead), "n"(AHI), "n"(BHI)
      : "memory");
}
// S^T[128 x QN] = K[128 x D] Q[QN x D]^T, both K-major.
template <int D, int QN>
__device__ __forceinline__ void mma_s8(uint32_t d_tmem, uint32_t k, uint32_t q, uint32_t lead) {
#pragma unroll
  for (int s = 0; s < D / 32; ++s)
    mma8<kDescHi8<D>, kDescHi8<D>>(d_tmem, k + s * 2, q + s * 2, idesc8(128, QN, false, false), s > 0, lead);
}
// O^T[128 x PN] (+)= V[w x D]^T P[w x PN], both MN-major (D = 64: the lanes from 64 on repeat the
// first ones, V's second column group lying 0 bytes behind the first).
template <int D, int PN>
__device__ __forceinline__ void mma_o8(uint32_t d_tmem, uint32_t v, uint32_t p, int w, bool first, uint32_t lead) {
#pragma unroll
  for (int s = 0; s < KT / 32; ++s)
    if (s * 32 < w)
      mma8<kDescHi8<D>, kDescHi8<128>>(d_tmem, v + s * (32 * D >> 4), p + s * (32 * 128 >> 4),
                                       idesc8(128, PN, true, true), s > 0 || !first, lead);
}

// N TMEM columns of a lane (8, 16 or 32), without the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_nowait(uint32_t a, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
  } else {
    static_assert(N == 32, "");
    tc::tmem_ld32_nowait(a, v);
  }
}
// Waits for every load of the thread and makes v's registers depend on it.
template <int N>
__device__ __forceinline__ void tmem_landed(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+f"(v[e]));
}
template <int N>
__device__ __forceinline__ void tmem_st_nowait(uint32_t a, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
  for (int e = 0; e < N; e += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a + e), "r"(r[e]),
                 "r"(r[e + 1]), "r"(r[e + 2]), "r"(r[e + 3]), "r"(r[e + 4]), "r"(r[e + 5]), "r"(r[e + 6]), "r"(r[e + 7])
                 : "memory");
}

// Barrier of a group's 128 threads that also joins a condition.
__device__ __forceinline__ bool bar_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, %2, 128, p;\nselp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint16_t e4m3x2_of(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(c));
  return r;
}
// 32 (h - c) for pairs of f16: exact, since c is h rounded to fewer bits.
__device__ __forceinline__ uint32_t rest32(uint32_t h, uint32_t c) {
  uint32_t r;
  asm("{\n.reg .b32 d;\nsub.rn.f16x2 d, %1, %2;\nmul.rn.f16x2 %0, d, %3;\n}\n" : "=r"(r) : "r"(h), "r"(c), "r"(0x50005000u));
  return r;
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg8<D, NR>::THREADS, Cfg8<D, NR>::PER_SM)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k16,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v16,
                   const Q8Params p) {
  using C = Cfg8<D, NR>;
  constexpr int HR = C::HR, NS = C::NS, QN = C::QN, PN = C::PN;
  using B = Bars8<NS>;
  constexpr int kLoad = 8, kIssue = 9, kScale = 10;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B::COUNT];
  __shared__ __align__(16) float4 s_sc[16 * 8];  // of tile i % 16, 16-key group: (sk, log2 sv, 1 / sv, whether there is a page)
  __shared__ __align__(16) float s_rs[NR];       // scale log2(e) 2^-a of a row
  __shared__ float s_max[2][4][HR], s_sum[2][4][HR];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t p_s = base, slots = p_s + 2 * C::P_BYTES, q_s = slots + NS * C::TILE;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  if (stopped()) return;
  const Waits wait(abort);
  const int64_t unit = (int64_t)blockIdx.x / p.n_splits;
  const int split = (int)((int64_t)blockIdx.x % p.n_splits);
  const Unit8 un(p, unit, NR);
  const int seq = un.seq, g = un.g, R = p.R;
  const int64_t rows_all = (int64_t)un.Lq * R;
  if (un.row0 >= rows_all) return;
  const int rows = (int)min((int64_t)NR, rows_all - un.row0);
  const int kv_len = cached_len(p.keys.c, seq);
  const int off = kv_len - un.Lq;  // position of the sequence's first query
  const Tiles tiles(off + un.row0 / R, off + (un.row0 + rows - 1) / R, p.window, p.n_sink);
  const int a = (int)((int64_t)tiles.n * split / p.n_splits);
  const int n = (int)((int64_t)tiles.n * (split + 1) / p.n_splits) - a;  // this CTA's tiles: a .. a + n - 1
  const int groups = rows > HR ? 2 : 1;                                  // softmax groups that have rows
  // whole steps of 32 keys (the product's K): what lies past the keys is zeros
  auto width = [&](int i) { return min(KT, (tiles.width(i) + 31) & ~31); };

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(bar(B::FULL + i), 1);
      tc::mbar_init(bar(B::EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(B::SFULL + i), 1);
      tc::mbar_init(bar(B::PFULL + i), 4 * groups);
      tc::mbar_init(bar(B::PVDONE + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(bar(B::SCFULL + i), 1);
      tc::mbar_init(bar(B::SCEMPTY + i), 4 * groups);
    }
    tc::mbar_init(bar(B::DRAIN), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kIssue) {
    tmem_alloc(smem_u32(&s_tmem), C::TMEM);
    tc::fence_before();
  }
  if (warp < 8) {
    // Q's rows as two e4m3 terms: row r and row NR + r of the operand
    constexpr int E = D / 32;  // values a lane
    for (int r = warp; r < NR; r += 8) {
      float x[E];
      if (r < rows) {
        const int64_t rho = un.row0 + r;
        const __nv_bfloat16* src = p.q + ((un.start + rho / R) * p.h + g * R + rho % R) * D + lane * E;
        if constexpr (E == 4) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
          x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
        } else {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(src);
          x[0] = __uint_as_float(u << 16), x[1] = __uint_as_float(u & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
      }
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      const int ex = min(120, max(-120, 7 + 127 - (int)(top >> 23)));  // max |x| 2^ex in [128, 256)
      const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
      uint32_t c1 = 0, c2 = 0;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float y0 = x[e] * up, y1 = x[e + 1] * up;
        uint16_t h1, h2;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(h1) : "f"(y1), "f"(y0));
        const uint32_t b = f16x2_of(h1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(h2) : "f"((y1 - f.y) * 32.f), "f"((y0 - f.x) * 32.f));
        c1 |= (uint32_t)h1 << (8 * e);
        c2 |= (uint32_t)h2 << (8 * e);
      }
      const int ch = lane * E / 16, in = lane * E % 16;
      if constexpr (E == 4) {
        asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(at8<D>(q_s, r, ch) + in), "r"(c1) : "memory");
        asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(at8<D>(q_s, NR + r, ch) + in), "r"(c2) : "memory");
      } else {
        asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(at8<D>(q_s, r, ch) + in), "h"((uint16_t)c1) : "memory");
        asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(at8<D>(q_s, NR + r, ch) + in), "h"((uint16_t)c2) : "memory");
      }
      if (lane == 0) s_rs[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  int last_item = -1;  // loading warp: the last item handed to the ring
  if (warp == kLoad) {
    // ------------------------------------------------------------------ K and V tiles in turn
    int slot = 0;
    uint32_t phase = 1;
    for (int i = 0; i < 2 * n; ++i) {
      const int j = a + (i >> 1);
      const bool is_v = i & 1;
      if (i >= NS && !wait(bar(B::EMPTY + slot), phase)) break;
      load_tile8<D>(slots + slot * C::TILE, is_v ? &tm_v : &tm_k, is_v ? &tm_v16 : &tm_k16,
                    is_v ? p.keys.v : p.keys.k, p.keys.c, p.hkv, g, seq, j * KT, tiles.sink_end, tiles.shift, width(j),
                    kv_len, bar(B::FULL + slot), lane);
      last_item = i;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == kScale) {
    // ------------------------------------------------------------------ scales of four tiles
    const int batches = (n + 3) / 4;
    for (int i = 0; i < batches; ++i) {
      if (i >= 4 && !wait(bar(B::SCEMPTY + (i & 3)), ((i >> 2) - 1) & 1)) break;
      const int tile = a + i * 4 + (lane >> 3), place = tile * KT + (lane & 7) * GRAN;
      const int key = place < tiles.sink_end ? place : place + tiles.shift;
      float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tile < a + n && place < tiles.total && key < kv_len) {
        const int pid = page_of(p.keys.c, seq, key);
        if (pid >= 0) {
          const int pl = p.keys.c.page_log2, bl = p.keys.block_log2;
          const int64_t at = (((int64_t)pid * p.hkv + g) << (pl - bl)) + ((key & ((1 << pl) - 1)) >> bl);
          const float sv = __ldg(p.keys.vs + at);
          sc = make_float4(__ldg(p.keys.ks + at), log2f(sv), 1.f / sv, 1.f);
        }
      }
      s_sc[(i & 3) * 32 + lane] = sc;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B::SCFULL + (i & 3)));
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------------------ products
    const uint32_t lead = elect();
    const uint32_t q_d = desc_k(q_s), k_d = desc_k(slots);
    // V: the second group of 64 columns (D = 64) is the first again; P: groups P_BYTES / PG apart
    const uint32_t v_d = (slots & 0x3FFFF) >> 4, p_d = ((p_s & 0x3FFFF) >> 4) | ((uint32_t)(KT * 128 >> 4) << 16);
    Ring<NS> rk, rv;
    rv.next();
    bool ok = true;
    auto issue_s = [&](int b) {
      ok = wait(bar(B::FULL + rk.slot), rk.phase);
      if (!ok) return;
      tc::fence_after();
      mma_s8<D, QN>(tmem + b * QN, k_d + rk.slot * (C::TILE >> 4), q_d, lead);
      commit(bar(B::SFULL + b), lead);
      commit(bar(B::EMPTY + rk.slot), lead);
      rk.next();
      rk.next();
    };
    if (n > 0) issue_s(0);
    if (ok && n > 1) issue_s(1);
    for (int it = 0; ok && it < n; ++it) {
      const int b = it & 1;
      if (!(ok = wait(bar(B::FULL + rv.slot), rv.phase))) break;
      if (!(ok = wait(bar(B::PFULL + b), (it >> 1) & 1))) break;
      tc::fence_after();
      mma_o8<D, PN>(tmem + C::O_COL, v_d + rv.slot * (C::TILE >> 4), p_d + b * (C::P_BYTES >> 4), width(a + it), it == 0,
                    lead);
      commit(bar(B::EMPTY + rv.slot), lead);
      commit(bar(B::PVDONE + b), lead);
      rv.next();
      rv.next();
      if (it + 2 < n) issue_s(b);  // (its scores were read before P was written)
    }
  } else if (warp < 4 * groups) {
    // ------------------------------------------------------------------ softmax: one key, HR rows
    const int x = warp >> 2, krow = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_t = tmem + C::O_COL + x * HR + lane_base;
    float m[HR], l[HR];  // m: the running maximum less kRoom, so that P' = exp2(t - m)
#pragma unroll
    for (int e = 0; e < HR; ++e) {
      m[e] = kNone;
      l[e] = 0.f;
    }
    bool ok = true;
    int it = 0;
    for (; it < n; ++it) {
      const int b = it & 1;
      const uint32_t s_t = tmem + b * QN + x * HR + lane_base;
      float t[HR];
      float inv_sv = 0.f;
      uint32_t see = 0;
      bool move = false;
      ok = ok && wait(bar(B::SCFULL + ((it >> 2) & 3)), (it >> 4) & 1) && wait(bar(B::SFULL + b), (it >> 1) & 1);
      if (ok) {
        tc::fence_after();
        float lo[HR];
        tmem_ld_nowait<HR>(s_t, t);
        tmem_ld_nowait<HR>(s_t + NR, lo);
        const float4 sc = s_sc[(it & 15) * 8 + (krow >> 4)];
        inv_sv = sc.z;
        // rows that see the key: from the first at its position on, to the last whose window reaches it
        const int place = (a + it) * KT + krow, key = place < tiles.sink_end ? place : place + tiles.shift;
        const int64_t r0 = un.row0 + x * HR;
        if (sc.w != 0.f && place < tiles.total && key < kv_len && !(place < tiles.sink_end && key >= p.n_sink)) {
          const int64_t from = (int64_t)(key - off) * R - r0;
          const int64_t to = p.window > 0 && key >= p.n_sink ? ((int64_t)key + p.window - off) * R - r0 : HR;
          see = bits((int)min((int64_t)32, max((int64_t)0, from)), (int)min((int64_t)32, max((int64_t)0, to)));
        }
        tmem_landed<HR>(t);
#pragma unroll
        for (int e = 0; e < HR; ++e) asm volatile("" : "+f"(lo[e]));
        float most = kNegInf;
#pragma unroll
        for (int e = 0; e < HR; ++e) {
          const float s = fmaf(lo[e], 0.03125f, t[e]);
          t[e] = (see >> e) & 1u ? fmaf(s, s_rs[x * HR + e] * sc.x, sc.y) : kNegInf;
          most = fmaxf(most, t[e] - m[e]);
        }
        move = most > kMoves;
      }
      if (bar_or(1 + x, move || !ok)) {
        // the tile's maxima; a row that one of them exceeds moves
#pragma unroll
        for (int e = 0; e < HR; ++e) {
          float v = ok ? t[e] : kNegInf;
#pragma unroll
          for (int s = 16; s; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
          if (lane == 0) s_max[x][warp & 3][e] = v;
        }
        if (it > 0) ok = ok && wait(bar(B::PVDONE + (b ^ 1)), ((it - 1) >> 1) & 1);  // O is complete
        if (bar_or(1 + x, !ok || *abort)) {  // (every warp of the group leaves here, or none)
          ok = false;
          break;
        }
        tc::fence_after();
#pragma unroll
        for (int e0 = 0; e0 < HR; e0 += 8) {
          float al[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            const float v = fmaxf(fmaxf(s_max[x][0][e], s_max[x][1][e]), fmaxf(s_max[x][2][e], s_max[x][3][e]));
            const float now = v - m[e] > kMoves ? v - kRoom : m[e];
            al[i] = ex2(m[e] - now);
            l[e] *= al[i];
            m[e] = now;
          }
          if (it > 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              float ov[8];
              tmem_ld_nowait<8>(o_t + k * NR + e0, ov);
              tmem_landed<8>(ov);
#pragma unroll
              for (int i = 0; i < 8; ++i) ov[i] *= al[i];
              tmem_st_nowait<8>(o_t + k * NR + e0, ov);
            }
          }
        }
        tmem_wait_st();
      }
      if (it >= 2 && ok) ok = wait(bar(B::PVDONE + b), ((it - 2) >> 1) & 1);  // P's buffer is free
      if (!ok) continue;  // (to the next vote)
      const uint32_t p_b = p_s + b * C::P_BYTES;
      // eight rows at a time: three terms of P' each, to bytes (term NR + row) of the key's line
#pragma unroll
      for (int e0 = 0; e0 < HR; e0 += 8) {
        uint32_t c1[2], c2[2], c3[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint16_t d1[2], d2[2], d3[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int e = e0 + q * 4 + y * 2;
            const float w0 = ex2(t[e] - m[e]), w1 = ex2(t[e + 1] - m[e + 1]);
            l[e] = fmaf(w0, inv_sv, l[e]);
            l[e + 1] = fmaf(w1, inv_sv, l[e + 1]);
            const __half2 hh = __floats2half2_rn(w0, w1);
            const uint32_t h = *reinterpret_cast<const uint32_t*>(&hh);
            d1[y] = e4m3x2_of(h);
            const uint32_t h2 = rest32(h, f16x2_of(d1[y]));
            d2[y] = e4m3x2_of(h2);
            d3[y] = e4m3x2_of(rest32(h2, f16x2_of(d2[y])));
          }
          c1[q] = d1[0] | (uint32_t)d1[1] << 16;
          c2[q] = d2[0] | (uint32_t)d2[1] << 16;
          c3[q] = d3[0] | (uint32_t)d3[1] << 16;
        }
        auto put = [&](int term, const uint32_t* c) {
          const int col = term * NR + x * HR + e0;
          const uint32_t at = at8<128>(p_b + (col >> 7) * (KT * 128), krow, (col & 127) >> 4) + (col & 15);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at), "r"(c[0]), "r"(c[1]) : "memory");
        };
        put(0, c1);
        put(1, c2);
        put(2, c3);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(bar(B::PFULL + b));
        if ((it & 3) == 3) tc::mbar_arrive(bar(B::SCEMPTY + ((it >> 2) & 3)));
      }
    }
    if (n > 1) ok = ok && wait(bar(B::PVDONE + (n & 1)), ((n - 2) >> 1) & 1);
    if (n > 0) ok = ok && wait(bar(B::PVDONE + ((n - 1) & 1)), ((n - 1) >> 1) & 1);
    tc::fence_after();
#pragma unroll
    for (int e = 0; e < HR; ++e) {
#pragma unroll
      for (int s = 16; s; s >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], s);
      if (lane == 0) s_sum[x][warp & 3][e] = l[e];
    }
    named_barrier(1 + x, 128);  // (also after a timeout: every warp of the group comes here)
    if (ok) {
#pragma unroll
      for (int e = 0; e < HR; ++e)
        l[e] = (s_sum[x][0][e] + s_sum[x][1][e]) + (s_sum[x][2][e] + s_sum[x][3][e]);
      int64_t tok = un.row0 + x * HR;  // token and head of the row
      int head = (int)(tok % R);
      tok = un.start + tok / R;
#pragma unroll
      for (int e0 = 0; e0 < HR; e0 += 8) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.f;
        if (n > 0) {
          float u[24];
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_ld_nowait<8>(o_t + k * NR + e0, u + 8 * k);
          tmem_landed<24>(u);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fmaf(fmaf(u[16 + i], 0.03125f, u[8 + i]), 0.03125f, u[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i, r = x * HR + e;
          if (r < rows) {
            if (p.n_splits == 1) {
              const int64_t rr = tok * p.h + g * R + head;
              if (krow < D) p.o[rr * D + krow] = __float2bfloat16(l[e] > 0.f ? o[i] / l[e] : 0.f);
              if (p.lse && krow == 0) p.lse[rr] = l[e] > 0.f ? (m[e] + log2f(l[e])) * kLn2 : kNegInf;
            } else {
              const int64_t at = (unit * p.n_splits + split) * NR + r;
              if (krow < D && l[e] > 0.f) p.part_o[at * D + krow] = o[i];
              if (krow == 0) p.part_ml[at] = make_float2(m[e], l[e]);
            }
          }
          if (++head == R) {
            head = 0;
            ++tok;
          }
        }
      }
    }
  }

  __syncthreads();
  if (*abort) {
    // copies and products still in flight land before the CTA leaves
    if (warp == kLoad) {
      for (int st = 0; st < NS; ++st)
        if (last_item >= st) {
          const int i = last_item - (last_item - st) % NS;
          tc::warp_drain(bar(B::FULL + st), (i / NS) & 1);
        }
    } else if (warp == kIssue) {
      commit(bar(B::DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(B::DRAIN), 0);
    }
  } else if (warp == kLoad) {
    // the last release of every slot lands before the CTA leaves
    for (int st = 0; st < NS; ++st)
      if (last_item >= st) {
        const int i = last_item - (last_item - st) % NS;
        tc::warp_drain(bar(B::EMPTY + st), (i / NS) & 1);
      }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_free(tmem, C::TMEM);
}

// Joins the parts of a row in order, a warp a row.
template <int D, int NR>
__global__ void __launch_bounds__(256) q8_combine_kernel(const Q8Params p, int64_t rows) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int64_t unit = row / NR;
  const Unit8 un(p, unit, NR);
  const int r = (int)(row % NR);
  const int64_t rho = un.row0 + r;
  if (rho >= (int64_t)un.Lq * p.R) return;
  const int64_t rr = (un.start + rho / p.R) * p.h + un.g * p.R + rho % p.R;
  const int parts = p.n_splits;
  const int64_t at = unit * parts * NR + r;  // of part 0
  float m = kNone, acc[E] = {}, l = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float2 ml = p.part_ml[at + (int64_t)i * NR];
    if (ml.y > 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f, wl = 0.f;
    if (i0 + lane < parts) {
      const float2 ml = p.part_ml[at + (int64_t)(i0 + lane) * NR];
      if (ml.y > 0.f) {
        w = ex2(ml.x - m);
        wl = w * ml.y;
      }
    }
    const int e1 = min(32, parts - i0);
#pragma unroll 4
    for (int i = 0; i < e1; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, wl, i);
      l += li;
      if (wi > 0.f) {
        const float* src = p.part_o + (at + (int64_t)(i0 + i) * NR) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, src[e], acc[e]);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.o + rr * D + lane * E + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse && lane == 0) p.lse[rr] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
}

// How a call is cut.
struct Plan8 {
  int nr, row_tiles, n_splits;
  int64_t units;
  size_t ml, bytes;  // workspace: part_o at 0, part_ml at `ml`
};
static Plan8 make_plan8(const Seqs& s, int h, int hkv, int D, int max_keys, int window, int n_sink) {
  Plan8 pl{};
  const int R = h / hkv;
  const int64_t rows = (int64_t)s.max_len * R;
  pl.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  pl.row_tiles = (int)((rows + pl.nr - 1) / pl.nr);
  pl.units = (int64_t)pl.row_tiles * s.n_seqs * hkv;
  int64_t keys = max_keys;
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + pl.nr / R + 1 + up16(n_sink) + 2 * GRAN);
  const int64_t tiles = std::max<int64_t>(1, (keys + KT - 1) / KT);
  const int64_t want = 4 * (pl.nr == 64 ? 1 : 2) * kSms8 / pl.units;
  pl.n_splits = (int)std::max<int64_t>(1, std::min<int64_t>({want, tiles, 256}));
  const size_t part = pl.n_splits == 1 ? 0 : (size_t)pl.units * pl.n_splits * pl.nr;
  pl.ml = (part * D * 4 + 255) & ~size_t(255);
  pl.bytes = part ? pl.ml + part * 8 : 0;
  return pl;
}

// Maps of the codes of K (or V): the tile box and the 16-row box.
static bool byte_maps(CUtensorMap* big, CUtensorMap* small, const void* ptr, const Keys& c, int hkv, int D) {
  const uint32_t page = 1u << c.page_log2;
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[3] = {(uint64_t)hkv * D, page, (uint64_t)c.n_pages};
    const uint64_t strides[2] = {(uint64_t)hkv * D, (uint64_t)c.page_stride};
    const uint32_t box[3] = {(uint32_t)D, i ? (uint32_t)GRAN : (page < KT ? page : (uint32_t)KT), 1};
    if (!tc::make_map(i ? small : big, ptr, 3, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return false;
  }
  return true;
}

template <int D, int NR>
static cudaError_t run_q8(const CUtensorMap* m, const Q8Params& p, const Plan8& pl, cudaStream_t st) {
  using C = Cfg8<D, NR>;
  auto kern = attn_q8_kernel<D, NR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t ctas = pl.units * pl.n_splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)ctas, C::THREADS, C::SMEM, st>>>(m[0], m[1], m[2], m[3], p);
  if ((e = cudaGetLastError()) != cudaSuccess || pl.n_splits == 1) return e;
  const int64_t rows = pl.units * NR;
  q8_combine_kernel<D, NR><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p, rows);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_q8_d(const Seqs& s, const void* q, const Keys8& keys, int h, int hkv, int max_keys,
                               int window, int n_sink, float scale, void* o, float* lse, void* workspace,
                               cudaStream_t st) {
  const Plan8 pl = make_plan8(s, h, hkv, D, max_keys, window, n_sink);
  Q8Params p{};
  p.seqs = s;
  p.keys = keys;
  p.q = (const __nv_bfloat16*)q;
  p.o = (__nv_bfloat16*)o;
  p.lse = lse;
  p.part_o = (float*)workspace;
  p.part_ml = (float2*)((uint8_t*)workspace + pl.ml);
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.window = window;
  p.n_sink = n_sink;
  p.row_tiles = pl.row_tiles;
  p.n_splits = pl.n_splits;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap m[4];
  if (!byte_maps(&m[0], &m[1], keys.k, keys.c, hkv, D) || !byte_maps(&m[2], &m[3], keys.v, keys.c, hkv, D))
    return cudaErrorInvalidValue;
  return pl.nr == 16   ? run_q8<D, 16>(m, p, pl, st)
         : pl.nr == 32 ? run_q8<D, 32>(m, p, pl, st)
                       : run_q8<D, 64>(m, p, pl, st);
}

}  // namespace span

size_t span_q8_workspace_bytes(const Seqs& s, int h, int hkv, int d, int max_keys, int window, int n_sink) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return 0;
  return span::make_plan8(s, h, hkv, d, max_keys, window, n_sink).bytes;
}

cudaError_t launch_span_q8(const Seqs& s, const void* q, const PagedView& cache, const void* k, const void* v,
                           const float* k_scales, const float* v_scales, int block_log2, int h, int hkv, int d,
                           int max_keys, int window, int n_sink, float scale, void* o, float* lse, void* workspace,
                           cudaStream_t st) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return cudaSuccess;
  span::Keys8 keys{};
  keys.k = (const uint8_t*)k;
  keys.v = (const uint8_t*)v;
  keys.ks = k_scales;
  keys.vs = v_scales;
  keys.c = span::keys_of(&cache, nullptr, nullptr);
  keys.block_log2 = block_log2;
  return d == 64 ? span::launch_q8_d<64>(s, q, keys, h, hkv, max_keys, window, n_sink, scale, o, lse, workspace, st)
                 : span::launch_q8_d<128>(s, q, keys, h, hkv, max_keys, window, n_sink, scale, o, lse, workspace, st);
}

NSA_STATUS_ACCESSOR(span_q8)

}  // namespace nsa
