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
// have to be 8-bit floats as well, whose few significant bits would be too few, so they are sums of terms:
//   Q  = 2^-a (q1 + q2 + q3)  a per row, so that max |Q 2^a| is in [128, 256); q1 in e4m3, the rest in e5m2
//   P' = p1 + p2 + p3       of P' = exp(t - m) sv 2^9 rounded to f16; all in e5m2
// q1 leaves at most 8 units of bf16's last place, which the 3 significant bits of e5m2 hold, where it is
// normal: from 2^-6 on.  Below, it leaves up to 2^-10, of which q2 leaves up to 2^-14 (without q3, 2^-21 of
// the row's largest element would go), and q3 half a step of e5m2's subnormals, 2^-17: so Q is
// exact down to 2^-16 of its row's largest element, and to 2^-24 of that below.  p1 + p2 + p3 is within
// 2^-9 of P' (and P' within 2^-11 of its value, half a step of f16; a bf16 P has 2^-8), down
// to 2^-26 of the row's largest weight.  q1, q2 and q3 share an accumulator (K is read three times); p1, p2 and p3
// lie side by side in N with accumulator columns of their own, so that V is read once.
// A key's value scale sv is part of its weight, and the running maximum is that of t + log2 sv:
// what is held in few bits is what the sum is made of.  The row sum takes exp(t - m) alone.
//
// A thread of the softmax has one key and HR rows, so a mask is a bit mask over rows, scales are
// scalars of the thread, and only the running maximum has to be agreed on: it moves when some
// key exceeds it by 2^6 (P' has that room), which a vote finds out for each tile.
//
// The key tiles of all units (row tile, sequence, kv-head) are cut into equal runs, one for each CTA
// that fits the GPU: a run may start and end inside a unit, whose parts (max, sum, unnormalised
// o) q8_combine_kernel joins in order.  So ragged caches even out, and a CTA sets itself
// up once.  The barriers of a turn cost more than its arithmetic, so a turn takes two key tiles.
//
// Decode, 32 caches of 16384 .. 32768 keys, 16 heads over 2 kv-heads of 128 (403 MB of codes): 81 us, 5.0 TB/s
// of a copy's 6.7 (80 with Q in two terms); the same values in a bf16 cache take 143.  Of the rest, 8 us go before
// the first scores (launch, set-up, first copies) and 5 into the join; in between HBM runs at 6.0 TB/s.  The tensor cores are far from
// their limit (one row of 8 in use of N = 16 costs as much as 16), but not from sight: a product with M = 128
// takes 40 cycles or more however small its N.  From 33 rows on the other form is faster (attn_q8_rows_kernel).
#include <algorithm>

#include <cuda_fp16.h>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

constexpr int kSms8 = 152;
constexpr float kRoom = 9.f, kMoves = 15.f;  // log2 of P' at the running maximum, and at which it moves
constexpr float kNone = -3e38f;             // running maximum of a row that has seen no key

struct Keys8 {
  const uint8_t *k, *v;
  const float *ks, *vs;  // [n_pages, hkv, page / block]
  Keys c;                // table, lens, sizes (page_stride in bytes; k, v unused)
  int block_log2;
};

template <int D, int NR>
struct Cfg8 {
  static constexpr int HR = 8, SUB = 2;   // rows (as many as tmem_ld8_nowait's columns) and keys of a thread: a turn takes SUB key tiles
  static constexpr int GROUPS = NR / HR;  // softmax groups of four warps
  static constexpr int PER_SM = NR <= 16 ? 2 : 1;
  // softmax warps; then loads of K, loads of V, products, queries and scales
  static constexpr int SOFT = 4 * GROUPS, THREADS = (SOFT + 4) * 32;
  static constexpr int TILE = KT * D;
  // Columns of S^T, columns of O^T: three terms of P; the products want multiples of 16.  Q's terms lie NR rows apart: with
  // 8 rows a product reads the next term's, too, into columns that no one reads
  static constexpr int SN = NR < 16 ? 16 : NR, PN = (3 * NR + 15) / 16 * 16;
  static constexpr int PW = NR == 8 ? 32 : NR == 16 ? 64 : 128;  // bytes of a key's line of P (PN, and room for the swizzle)
  static constexpr int Q_BYTES = (2 * NR + SN) * D, P_TILE = KT * PW;  // of one of two Q buffers, of a key tile's P
  // Slots of a turn's K tiles and of its V tiles
  static constexpr int TURN = SUB * TILE, ROOM = ((PER_SM == 2 ? 108 : 219) * 1024 - SUB * P_TILE - 2 * Q_BYTES) / TURN;
  static constexpr int NS = ROOM > 8 ? 8 : ROOM, NK = NS / 2, NV = NS - NK;
  static constexpr int SMEM = SUB * P_TILE + NS * TURN + 2 * Q_BYTES + 1024;
  static constexpr uint32_t O_COL = 2 * SUB * SN;  // behind two turns' S^T
  static constexpr uint32_t TMEM = NR == 32 ? 256 : 128;
  static_assert(O_COL + PN <= TMEM, "");
  static_assert(NK >= 1 && NV >= 1, "");
};

struct Q8Params {
  Seqs seqs;
  Keys8 keys;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;       // optional
  float* part_o;    // [CTAs][2][NR][D]: unnormalised o of a CTA's last unit (1) and of its first (0)
  float2* part_ml;  // [CTAs][2][NR]: (running maximum, sum)
  int2* info;       // [units]: (first CTA, CTAs) that a unit's tiles went to
  int h, hkv, R, window, n_sink, row_tiles;
  int ctas;         // of a streamed call
  int streamed;     // the tiles of all units in equal runs; else a CTA a unit
  int min_places;   // of a run
  float scale_log2;
};

// Rows of a unit and the key tiles that they see.  Unit ((seq * hkv) + g) * row_tiles + rt: rows rt * NR ..
// of (token, head of the group), heads fastest.
template <int NR>
struct Seq8 {
  int64_t start;
  int Lq, kv_len;
  __device__ __forceinline__ void load(const Q8Params& p, int seq) {
    start = seq_start(p.seqs, seq);
    Lq = seq_len(p.seqs, seq);
    kv_len = cached_len(p.keys.c, seq);
  }
  __device__ __forceinline__ int rows(const Q8Params& p, int rt) const {
    return (int)max((int64_t)0, min((int64_t)NR, (int64_t)Lq * p.R - (int64_t)rt * NR));
  }
  __device__ __forceinline__ Tiles tiles(const Q8Params& p, int rt) const {
    const int64_t row0 = (int64_t)rt * NR;
    const int off = kv_len - Lq;  // position of the sequence's first query
    return Tiles(off + (int)(row0 / p.R), off + (int)((row0 + rows(p, rt) - 1) / p.R), p.window, p.n_sink);
  }
  // Tiles that a unit counts for: a unit whose rows see nothing has an empty one, which writes them.
  __device__ __forceinline__ int count(const Q8Params& p, int rt) const {
    return rt >= p.row_tiles || rows(p, rt) == 0 ? 0 : max(1, tiles(p, rt).n);
  }
};

// The units of a CTA's run of tiles, one after another.  Every role walks the run for itself.
// A run is cut in places: a unit has kSwitch places that stand for the time that it takes to begin one (the
// joining of the row sums, O's way out, the first maxima), then one for each tile.
// 32 x 16384 .. 32768 keys, 8 rows: 0 places 85 us, 4 80.4, 8 79.5, 12 79.6, 24 80.6; 8 x 8192 keys x 8 kv-heads 46.2,
// 40.4, 37.1, 37.4, 38.9; 32 rows over 16 x 16384 keys x 4 kv-heads 88, 86, 84, 82, 76 (24 is the most that was tried);
// 128 rows over 16 x up to 8192 keys x 4 kv-heads with 6 places 72.2, 8 72.5, 12 74.2, 24 81.6.  16 rows take the 8-row
// form's number.
template <int NR>
struct Walk {
  static constexpr int kSwitch = NR == 128 ? 8 : NR == 32 ? 24 : 12;
  Seq8<NR> s;
  int seq, g, rt;
  int a, n, all;  // tiles a .. a + n - 1 of the unit's `all`; n = 0: the run has no tile (left)
  int left;       // places of the run from the unit's first on
  int at, took;   // where in the unit's places it starts, and how many of them it takes
  Walk() = default;
  __device__ __forceinline__ void enter(const Q8Params& p, int place) {
    at = place;
    all = s.count(p, rt);
    took = min(all + kSwitch - at, left);
    a = max(0, at - kSwitch);
    n = max(0, at + took - kSwitch) - a;
  }
  __device__ __forceinline__ Walk(const Q8Params& p, int seq0, int64_t place, int run) : seq(seq0), g(0), rt(0), left(run) {
    s.load(p, seq);
    int64_t per = 0;
    for (int i = 0; i < p.row_tiles; ++i)
      if (const int c = s.count(p, i)) per += c + kSwitch;
    g = (int)(place / per);
    place -= g * per;
    for (int c; place >= (c = s.count(p, rt) + kSwitch); ++rt) place -= c;
    enter(p, (int)place);
    if (n == 0) next(p);
  }
  // one whole unit
  __device__ __forceinline__ Walk(const Q8Params& p, int64_t unit) {
    rt = (int)(unit % p.row_tiles);
    unit /= p.row_tiles;
    g = (int)(unit % p.hkv);
    seq = (int)(unit / p.hkv);
    s.load(p, seq);
    a = 0;
    n = all = s.count(p, rt);
    left = at = took = 0;
  }
  __device__ __forceinline__ bool next(const Q8Params& p) {
    n = 0;
    left -= took;
    if (left <= kSwitch) return false;  // (no tile of the next unit)
    if (s.count(p, ++rt) == 0) {
      rt = 0;
      if (++g == p.hkv) {
        g = 0;
        do {
          if (++seq >= p.seqs.n_seqs) return false;
          s.load(p, seq);
        } while (s.count(p, 0) == 0);
      }
    }
    enter(p, 0);
    return true;
  }
};

// The turns of a run (SUB tiles of a unit each).
template <int NR, int SUB>
struct Turns {
  Walk<NR> u;
  Tiles tl;
  int j = 0;
  bool more = true;
  __device__ __forceinline__ Turns(const Q8Params& p, const Walk<NR>& w) : u(w), tl(w.s.tiles(p, w.rt)) {}
  __device__ __forceinline__ void next(const Q8Params& p) {
    if ((j += SUB) < u.n) return;
    j = 0;
    if ((more = u.next(p))) tl = u.s.tiles(p, u.rt);
  }
};

// A CTA's run: places first .. first + places - 1 of `total`, which `ctas` CTAs share.
struct Run8 {
  int places = 0, ctas = 0;
  int64_t first = 0, total = 0;
};
// False: there is nothing for this CTA.  A streamed call's run begins in sequence *s_seq, *s_at places on (known
// after the block's next synchronisation).
template <int NR, int WARPS>
__device__ __forceinline__ bool find_run(const Q8Params& p, Run8& r, int64_t* s_scan, int* s_seq, int64_t* s_at) {
  if (!p.streamed) return Walk<NR>(p, (int64_t)blockIdx.x).n != 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.seqs.n_seqs + WARPS * 32 - 1) / (WARPS * 32), i0 = min(p.seqs.n_seqs, tid * per),
            i1 = min(p.seqs.n_seqs, i0 + per);
  auto places_of = [&](int i) {
    Seq8<NR> s;
    s.load(p, i);
    int64_t c = 0;
    for (int rt = 0; rt < p.row_tiles; ++rt)
      if (const int n = s.count(p, rt)) c += n + Walk<NR>::kSwitch;
    return c * p.hkv;
  };
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += places_of(i);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  r.total = total;
  r.ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, total / p.min_places));
  if (total == 0 || blockIdx.x >= r.ctas) return false;
  r.first = total * blockIdx.x / r.ctas;
  r.places = (int)(total * (blockIdx.x + 1) / r.ctas - r.first);
  before += incl - mine;
  if (before <= r.first && r.first < before + mine) {
    int i = i0;
    for (int64_t c; before + (c = places_of(i)) <= r.first; ++i) before += c;
    *s_seq = i;
    *s_at = r.first - before;
  }
  return true;
}

// What the softmax has to know of a unit, in shared memory (its registers hold rows).
struct Part8 {
  int64_t start;
  int seq, g, rt, a, n, all, rows, off, kv_len, ctas;  // ctas: how many the unit's tiles go to
  int more;  // whether the run goes on
  int sink_end, shift, total, full_lo, full_hi;  // tiles full_lo .. full_hi - 1: every row sees every key that has a page
};
template <int NR>
__device__ __forceinline__ void describe(const Q8Params& p, const Walk<NR>& u, const Run8& r, Part8* s) {
  const Tiles tl = u.s.tiles(p, u.rt);
  const int off = u.s.kv_len - u.s.Lq, rows = u.s.rows(p, u.rt);
  const int64_t row0 = (int64_t)u.rt * NR;
  const int p0 = off + (int)(row0 / p.R), p1 = off + (int)((row0 + rows - 1) / p.R);
  s->start = u.s.start;
  s->seq = u.seq, s->g = u.g, s->rt = u.rt;
  s->a = u.a, s->n = u.n, s->all = u.all;
  s->rows = rows, s->off = off, s->kv_len = u.s.kv_len;
  s->sink_end = tl.sink_end, s->shift = tl.shift, s->total = tl.total;
  s->full_hi = max(0, p0 + 1 - tl.shift) / KT - u.a;  // the last key is at most the first position
  s->full_lo = p.window > 0 ? max(0, (max(tl.sink_end, p1 - p.window + 1 - tl.shift) + KT - 1) / KT) - u.a : 0;
  // (of a unit that begins here, at place t) the CTA that has place e - 1 of all: floor((e ctas - 1) / total)
  const int64_t t = r.first + r.places - u.left - u.at;
  s->ctas = p.streamed ? (int)(((t + u.kSwitch + u.all) * r.ctas - 1) / r.total) - (int)blockIdx.x + 1 : 1;
  s->more = u.left - u.took > u.kSwitch;
}

// Index of the last of items 0 .. last that went to slot st of ns (-1 if none).
__device__ __forceinline__ int last_in_stage(int last, int st, int ns) {
  return last < st ? -1 : last - (last - st) % ns;
}

template <int NS>
struct Bars8 {
  enum : int {
    FULL = 0,             // [NS] K's slots, then V's
    EMPTY = NS,
    SFULL = 2 * NS,       // [2] S^T of a turn
    PFULL = SFULL + 2,    // P of a turn
    PVDONE = PFULL + 1,   // its product
    SCFULL = PVDONE + 1,  // [4] scales of up to four tiles
    SCEMPTY = SCFULL + 4,
    QFULL = SCEMPTY + 4,  // [2] queries of a unit
    QEMPTY = QFULL + 2,
    DRAIN = QEMPTY + 2,
    COUNT
  };
};

// ------------------------------------------------------------------ byte tiles
// Row r of a tile of D-byte rows (32, 64 or 128), 16-byte chunk ch, in the swizzle of D bytes (as TMA writes it).
template <int D>
__device__ __forceinline__ uint32_t at8(uint32_t base, int r, int ch) {
  return base + r * D + ((ch ^ (D == 128 ? r & 7 : D == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4);
}
// Page of the 16 keys at place `place` (a lane's) of a unit: -1 where the table names none, 0 where there are no keys.
__device__ __forceinline__ int page_at(const Keys& c, int seq, int place, int sink_end, int shift, int kv_len) {
  const int key = place < sink_end ? place : place + shift;
  return key < kv_len ? page_of(c, seq, key) : 0;
}
// One warp fills a tile of w (a multiple of 32) rows as load_tile (span.cuh) does; pid16: page_at of a lane's 16 rows
// (lanes 0 .. 7).
template <int D>
__device__ __forceinline__ void load_tile8(uint32_t dst, const CUtensorMap* big, const CUtensorMap* small,
                                           const uint8_t* src, const Keys& c, int hkv, int g, int pid16, int place0,
                                           int sink_end, int shift, int w, int kv_len, uint32_t bar, int lane) {
  const int page = 1 << c.page_log2;
  const int box = page < KT ? page : KT;
  const int first = place0 + shift;
  const uint32_t bad = __ballot_sync(0xffffffffu, lane < w / GRAN && pid16 < 0);
  if (w == KT && place0 >= sink_end && first + KT <= kv_len && (first & (box - 1)) == 0 && bad == 0) {
    // whole pages (or parts of one)
    if (lane == 0) tc::mbar_expect_tx(bar, KT * D);
    const int pid = __shfl_sync(0xffffffffu, pid16, (lane * box / GRAN) & 7);
    if (lane * box < KT) tc::tma3d(dst + lane * box * D, big, g * D, (first + lane * box) & (page - 1), pid, bar);
    __syncwarp();
    return;
  }
  const int place = place0 + lane * GRAN, key = place < sink_end ? place : place + shift;
  const bool mine = lane < w / GRAN, plain = mine && (pid16 < 0 || key + GRAN > kv_len);
  if (mine && !plain) tc::tma3d(dst + lane * GRAN * D, small, g * D, key & (page - 1), pid16, bar);
  uint32_t todo = __ballot_sync(0xffffffffu, plain);
  const int bytes = (w / GRAN - __popc(todo)) * GRAN * D;
  if (todo) {
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const bool okc = !((bad >> l) & 1u);
      const int64_t pidc = __shfl_sync(0xffffffffu, pid16, l);
      const int keyc = __shfl_sync(0xffffffffu, key, l);
      for (int e = lane; e < GRAN * (D / 16); e += 32) {
        const int r = l * GRAN + e / (D / 16), ch = e % (D / 16), kk = keyc + e / (D / 16);
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
constexpr uint32_t kDescHi8 = (uint32_t)(8 * B >> 4) | (1u << 14) | ((B == 128 ? 2u : B == 64 ? 4u : 6u) << 29);
// e4m3 x (e4m3 or e5m2) -> fp32, M x N; A and B MN-major where said.
constexpr uint32_t idesc8(int M, int N, bool b_e5m2, bool mn) {
  return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)mn << 15) | ((uint32_t)mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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
// S^T[128 x SN] = K[128 x D] (Q1 + Q2 + Q3)[SN x D]^T, all K-major, Q's terms NR rows apart.
template <int D, int NR, int SN>
__device__ __forceinline__ void mma_s8(uint32_t d_tmem, uint32_t k, uint32_t q, uint32_t lead) {
#pragma unroll
  for (int z = 0; z < 3; ++z)
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      mma8<kDescHi8<D>, kDescHi8<D>>(d_tmem, k + s * 2, q + z * (NR * D >> 4) + s * 2, idesc8(128, SN, z > 0, false),
                                     z > 0 || s > 0, lead);
}
// O^T[128 x PN] (+)= V[128 x D]^T P[128 x PN], both MN-major (D = 64: the lanes from 64 on repeat the
// first ones, V's second column group lying 0 bytes behind the first).
template <int D, int PN, int PW>
__device__ __forceinline__ void mma_o8(uint32_t d_tmem, uint32_t v, uint32_t p, bool first, uint32_t lead) {
#pragma unroll
  for (int s = 0; s < KT / 32; ++s)
    mma8<kDescHi8<D>, kDescHi8<PW>>(d_tmem, v + s * (32 * D >> 4), p + s * (32 * PW >> 4), idesc8(128, PN, true, true),
                                    s > 0 || !first, lead);
}
// The same for a tile of w keys.
template <int D, int PN, int PW>
__device__ __forceinline__ void mma_o8_cut(uint32_t d_tmem, uint32_t v, uint32_t p, int w, bool first, uint32_t lead) {
#pragma unroll
  for (int s = 0; s < KT / 32; ++s)
    if (s * 32 < w)
      mma8<kDescHi8<D>, kDescHi8<PW>>(d_tmem, v + s * (32 * D >> 4), p + s * (32 * PW >> 4), idesc8(128, PN, true, true),
                                      s > 0 || !first, lead);
}

// Eight TMEM columns of a lane, without the wait.
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t a, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
// Waits for every load of the thread and makes v's registers depend on it.
template <int N>
__device__ __forceinline__ void tmem_landed(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+f"(v[e]));
}
__device__ __forceinline__ void tmem_st8_nowait(uint32_t a, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ bool device_stopped() { return tc::device_status_set(); }

// Barrier of `threads` threads that also joins a condition.
__device__ __forceinline__ bool bar_or(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, %2, %3, p;\nselp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint16_t e5m2x2_of(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(h2));
  return r;
}
// Two e5m2 are the high bytes of two f16.
__device__ __forceinline__ uint32_t f16x2_of_e5m2(uint16_t c) { return __byte_perm(c, 0, 0x1404); }
// h less its two e5m2: exact, since they are h rounded to fewer bits.
__device__ __forceinline__ uint32_t rest_of(uint32_t h, uint16_t c) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(h), "r"(f16x2_of_e5m2(c)));
  return r;
}

// Query rows r0, r0 + step, ... of a unit as three terms: rows r, NR + r and 2 NR + r of the operand; what
// turns their scores into exponents of 2; and the running maximum of no keys.  A warp's call.
template <int D, int NR>
__device__ __forceinline__ void load_q8(const Q8Params& p, const Walk<NR>& u, uint32_t q_s, float* s_rs, float* s_nm,
                                        int r0, int step, int lane) {
  constexpr int E = D / 32;  // values a lane
  const int rows = u.s.rows(p, u.rt);
#pragma unroll 4
  for (int r = r0; r < NR; r += step) {
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (r < rows) {
      const uint32_t rho = (uint32_t)u.rt * NR + r, R = p.R;  // (a call of many rows does not come here)
      const __nv_bfloat16* src = p.q + ((u.s.start + rho / R) * p.h + u.g * p.R + rho % R) * D + lane * E;
      if constexpr (E == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src);
        x[0] = __uint_as_float(w << 16), x[1] = __uint_as_float(w & 0xffff0000u);
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const int ex = min(120, max(-120, 7 + 127 - (int)(top >> 23)));  // max |x| 2^ex in [128, 256)
    const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
    uint32_t c[3] = {};
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float y0 = x[e] * up, y1 = x[e + 1] * up;
      uint16_t h[3];
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(h[0]) : "f"(y1), "f"(y0));
      const uint32_t b = f16x2_of_e4m3(h[0]);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
      const float d0 = y0 - f.x, d1 = y1 - f.y;  // (what is left is exact)
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(h[1]) : "f"(d1), "f"(d0));
      const uint32_t b2 = f16x2_of_e5m2(h[1]);
      const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&b2));
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(h[2]) : "f"(d1 - f2.y), "f"(d0 - f2.x));
#pragma unroll
      for (int z = 0; z < 3; ++z) c[z] |= (uint32_t)h[z] << (8 * e);
    }
    const int ch = lane * E / 16, in = lane * E % 16;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
      const uint32_t to = at8<D>(q_s, z * NR + r, ch) + in;
      if constexpr (E == 4)
        asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(to), "r"(c[z]) : "memory");
      else
        asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(to), "h"((uint16_t)c[z]) : "memory");
    }
    if (lane == 0) {
      // (a row with an infinity or NaN: an infinity's terms are finite, so its scores are made NaN here)
      s_rs[r] = p.scale_log2 * __uint_as_float(top < 0x7f800000u ? (uint32_t)(127 - ex) << 23 : 0x7fc00000u);
      s_nm[r] = -kNone;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg8<D, NR>::THREADS, Cfg8<D, NR>::PER_SM)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k16,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v16,
                   const Q8Params p) {
  using C = Cfg8<D, NR>;
  constexpr int HR = C::HR, NS = C::NS, PN = C::PN, SUB = C::SUB, SOFT = C::SOFT, WARPS = C::THREADS / 32;
  using B = Bars8<NS>;
  constexpr int kLoadK = SOFT, kLoadV = SOFT + 1, kIssue = SOFT + 2, kAux = SOFT + 3, NK = C::NK, NV = C::NV;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B::COUNT];
  __shared__ __align__(16) float4 s_sc[4][4][8];  // batch, tile, 16 keys: (sk, log2 sv, 1 / sv, whether there is a page)
  __shared__ __align__(16) float s_rs[2][NR];    // scale log2(e) 2^-a of a row
  __shared__ __align__(16) float s_nm[4][2][NR];  // of unit k at k % 4: minus the running maximum less kRoom (twice: see the moves)
  __shared__ float s_max[C::GROUPS][4][HR], s_sum[C::GROUPS][4][HR];
  __shared__ int64_t s_scan[WARPS], s_at;
  __shared__ uint32_t s_tmem;
  __shared__ Part8 s_part[4];  // of unit k of the run, at k % 4
  __shared__ int s_abort, s_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t p_s = base, slots = p_s + C::SUB * C::P_TILE, q_s = slots + NS * C::TURN;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  launch_dependents();
  if (stopped()) return;
  const Waits wait(abort);
  // ------------------------------------------------------------------ this CTA's run of tiles
  Run8 r;
  if (!find_run<NR, WARPS>(p, r, s_scan, &s_seq, &s_at)) return;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(bar(B::FULL + i), SUB);
      tc::mbar_init(bar(B::EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(B::SFULL + i), 1);
      tc::mbar_init(bar(B::QFULL + i), 1);
      tc::mbar_init(bar(B::QEMPTY + i), SOFT);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(bar(B::SCFULL + i), 1);
      tc::mbar_init(bar(B::SCEMPTY + i), SOFT);
    }
    tc::mbar_init(bar(B::PFULL), SOFT);
    tc::mbar_init(bar(B::PVDONE), 1);
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
  Walk<NR> u = p.streamed ? Walk<NR>(p, s_seq, s_at, r.places) : Walk<NR>(p, (int64_t)blockIdx.x);
  // whole steps of 32 keys (the product's K): what lies past the keys is zeros
  auto width = [&](const Tiles& tl, int i) { return max(0, min(KT, (tl.width(i) + 31) & ~31)); };

  int last_item = -1;  // loading warps: the last turn handed to their ring
  if (u.n == 0) {
    // (a run that lies between two units)
  } else if (warp == kLoadK || warp == kLoadV) {
    // ------------------------------------------------------------------ K tiles, or V tiles
    // (one code for both: instructions of warps that run rarely come from far)
    const bool is_v = warp == kLoadV;
    const int first = is_v ? NK : 0, ns = is_v ? NV : NK;
    const CUtensorMap *big = is_v ? &tm_v : &tm_k, *small = is_v ? &tm_v16 : &tm_k16;
    const uint8_t* src = is_v ? p.keys.v : p.keys.k;
    Turns<NR, SUB> t(p, u);
    int slot = 0;
    uint32_t phase = 1;
    auto pages = [&](int i) {
      return page_at(p.keys.c, t.u.seq, (t.u.a + i) * KT + (lane & 7) * GRAN, t.tl.sink_end, t.tl.shift, t.u.s.kv_len);
    };
    for (; t.more; t.next(p)) {
      int pid = pages(t.j);
      if (last_item + 1 >= ns && !wait(bar(B::EMPTY + first + slot), phase)) break;
#pragma unroll 1
      for (int y = 0; y < SUB; ++y) {
        const int j = t.j + y;
        if (j < t.u.n)
          load_tile8<D>(slots + (first + slot) * C::TURN + y * C::TILE, big, small, src, p.keys.c, p.hkv, t.u.g, pid,
                        (t.u.a + j) * KT, t.tl.sink_end, t.tl.shift, width(t.tl, t.u.a + j), t.u.s.kv_len,
                        bar(B::FULL + first + slot), lane);
        else if (lane == 0)
          tc::mbar_arrive(bar(B::FULL + first + slot));
        pid = pages(j + 1);
      }
      ++last_item;
      if (++slot == ns) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == kAux) {
    // ------------------------------------------------------------------ per unit: description, queries, scales
    // The first unit's queries are the softmax warps' own; a later one's are loaded once the scales of the
    // unit before are on their way.
    Ring<2> rq;
    Ring<4> rs;
    bool ok = true, again = false;
    for (int k = 0; ok; ++k) {
      if (k > 1 && !(ok = wait(bar(B::QEMPTY + rq.slot), rq.phase ^ 1u))) break;
      if (lane == 0) describe<NR>(p, u, r, &s_part[k & 3]);
      if (k > 0)
        load_q8<D, NR>(p, u, q_s + rq.slot * C::Q_BYTES, s_rs[rq.slot], s_nm[k & 3][0], 0, 1, lane);
      else
        named_barrier(1, (SOFT + 1) * 32);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B::QFULL + rq.slot));
      rq.next();
      const Tiles tl = u.s.tiles(p, u.rt);
      for (int i = 0; i < u.n; i += 4) {
        if (again && !(ok = wait(bar(B::SCEMPTY + rs.slot), rs.phase ^ 1u))) break;
        const int tile = u.a + i + (lane >> 3), place = tile * KT + (lane & 7) * GRAN;
        const int key = place < tl.sink_end ? place : place + tl.shift;
        float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tile < u.a + u.n && place < tl.total && key < u.s.kv_len) {
          const int pid = page_of(p.keys.c, u.seq, key);
          if (pid >= 0) {
            const int pl = p.keys.c.page_log2, bl = p.keys.block_log2;
            const int64_t at = (((int64_t)pid * p.hkv + u.g) << (pl - bl)) + ((key & ((1 << pl) - 1)) >> bl);
            const float sv = __ldg(p.keys.vs + at);
            sc = make_float4(__ldg(p.keys.ks + at), log2f(sv), 1.f / sv, 1.f);
          }
        }
        s_sc[rs.slot][lane >> 3][lane & 7] = sc;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::SCFULL + rs.slot));
        rs.next();
        again |= rs.slot == 0;
      }
      if (!u.next(p)) break;
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------------------ products
    // S^T runs up to two turns ahead of O^T, across the units of the run.
    const uint32_t lead = elect(), q_d = desc_k(q_s), k_d = desc_k(slots);
    // V: the second group of 64 columns (D = 64) is the first again
    const uint32_t v_d = ((slots + NK * C::TURN) & 0x3FFFF) >> 4, p_d = (p_s & 0x3FFFF) >> 4;
    Turns<NR, SUB> ts(p, u), to = ts;
    Ring<NK> rk;
    Ring<NV> rv;
    Ring<2> rq;
    bool ok = true;
    for (uint32_t it = 0; ok && to.more; ++it) {
      // turn it's scores, and from the third turn on the product of turn it - 2 before them
      if (it >= 2) {
        const int left = to.u.n - to.j;  // of the unit
        if (!(ok = wait(bar(B::FULL + NK + rv.slot), rv.phase) && wait(bar(B::PFULL), it & 1))) break;
        tc::fence_after();
        const uint32_t vv = v_d + rv.slot * (C::TURN >> 4);
        if (left > SUB) {  // (no branch between the products)
#pragma unroll
          for (int y = 0; y < SUB; ++y)
            mma_o8<D, PN, C::PW>(tmem + C::O_COL, vv + y * (C::TILE >> 4), p_d + y * (C::P_TILE >> 4), to.j + y == 0, lead);
        } else {
#pragma unroll 1
          for (int y = 0; y < left; ++y)
            mma_o8_cut<D, PN, C::PW>(tmem + C::O_COL, vv + y * (C::TILE >> 4), p_d + y * (C::P_TILE >> 4),
                                     width(to.tl, to.u.a + to.j + y), to.j + y == 0, lead);
        }
        commit(bar(B::PVDONE), lead);
        commit(bar(B::EMPTY + NK + rv.slot), lead);
        rv.next();
        to.next(p);
      }
      if (ts.more) {
        const int b = it & 1;
        // (S^T of turn it - 2 was read before its P was written)
        if (!(ok = (ts.j != 0 || wait(bar(B::QFULL + rq.slot), rq.phase)) && wait(bar(B::FULL + rk.slot), rk.phase))) break;
        tc::fence_after();
        const uint32_t q = q_d + rq.slot * (C::Q_BYTES >> 4), kk = k_d + rk.slot * (C::TURN >> 4);
        const uint32_t s_t = tmem + b * SUB * C::SN;
        // (without a second tile, at the end of a unit, old keys give scores that no one reads)
#pragma unroll
        for (int y = 0; y < SUB; ++y) mma_s8<D, NR, C::SN>(s_t + y * C::SN, kk + y * (C::TILE >> 4), q, lead);
        commit(bar(B::SFULL + b), lead);
        commit(bar(B::EMPTY + rk.slot), lead);
        rk.next();
        ts.next(p);
        if (ts.j == 0) rq.next();
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax: one key, HR rows
    const int x = warp >> 2, krow = (warp & 3) * 32 + lane, x0 = x * HR, vote = 2 + x;  // (vote: the group's barrier)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_t = tmem + C::O_COL + x0 + lane_base;
    load_q8<D, NR>(p, u, q_s, s_rs[0], s_nm[0][0], warp, SOFT, lane);
    named_barrier(1, (SOFT + 1) * 32);
    Ring<4> rsc;
    Ring<2> rq;
    bool ok = true;
    uint32_t it = 0;  // turns of the run
    for (int k = 0;; ++k) {
      ok = ok && wait(bar(B::QFULL + rq.slot), rq.phase);
      // (one answer for all that meet at the unit's end: they go through the same turns)
      if (bar_or(vote, 128, !ok)) break;
      const volatile Part8& u = s_part[k & 3];
      const int n = u.n, full_lo = u.full_lo, full_hi = u.full_hi;
      const int rows = u.rows - x0;  // of the group; without any it only keeps the barriers moving
      const float* nm = s_nm[k & 3][0] + x0;
      float l[HR];
#pragma unroll
      for (int e = 0; e < HR; ++e) l[e] = 0.f;
#pragma unroll 1
      for (int i = 0; i < n; i += SUB, ++it) {
        const int b = it & 1;
        const uint32_t s_t = tmem + b * SUB * C::SN + x0 + lane_base;
        if ((i & 3) == 0) ok = ok && wait(bar(B::SCFULL + rsc.slot), rsc.phase);
        ok = ok && wait(bar(B::SFULL + b), (it >> 1) & 1);
        tc::fence_after();
        float4 sc[SUB];
        // rows that see the thread's keys: from the first at its position on, to the last whose window reaches it
        uint32_t see[SUB];
        bool all = true;
#pragma unroll
        for (int y = 0; y < SUB; ++y) {
          sc[y] = s_sc[rsc.slot][(i & 3) + y][krow >> 4];
          see[y] = sc[y].w != 0.f ? (1u << HR) - 1u : 0u;  // (0 past the unit's tiles too)
          if (i + y < full_lo || i + y >= full_hi) {
            const int place = (u.a + i + y) * KT + krow, sink_end = u.sink_end;
            const int key = place < sink_end ? place : place + u.shift, off = u.off;
            const int64_t r0 = (int64_t)u.rt * NR + x0;
            const bool in = place < u.total && key < u.kv_len && !(place < sink_end && key >= p.n_sink);
            const int64_t from = (int64_t)(key - off) * p.R - r0;
            const int64_t to = p.window > 0 && key >= p.n_sink ? ((int64_t)key + p.window - off) * p.R - r0 : HR;
            if (in)
              see[y] &= bits((int)min((int64_t)HR, max((int64_t)0, from)), (int)min((int64_t)HR, max((int64_t)0, to)));
            else
              see[y] = 0;
          }
          all = all && see[y] == (1u << HR) - 1u;
        }
        all = __all_sync(0xffffffffu, all);
        // exponents t of the scores (raw), or t + nm: P' = exp2(t + nm)
        float v[SUB][HR];
        auto scores = [&](bool raw) {
#pragma unroll
          for (int y = 0; y < SUB; ++y) tmem_ld8_nowait(s_t + y * C::SN, v[y]);
          tmem_landed<SUB * HR>(&v[0][0]);
          const float* rs = s_rs[rq.slot] + x0;
#pragma unroll
          for (int e = 0; e < HR; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(rs + e);
            float2 m = make_float2(0.f, 0.f);
            if (!raw) m = *reinterpret_cast<const float2*>(nm + e);
#pragma unroll
            for (int y = 0; y < SUB; ++y) {
              const float2 t = unpair(fma2(pair(v[y][e], v[y][e + 1]), mul2(pair(f.x, f.y), pair(sc[y].x, sc[y].x)),
                                           add2(pair(sc[y].y, sc[y].y), pair(m.x, m.y))));
              v[y][e] = t.x;
              v[y][e + 1] = t.y;
            }
          }
          if (!all) {
#pragma unroll
            for (int y = 0; y < SUB; ++y)
#pragma unroll
              for (int e = 0; e < HR; ++e) v[y][e] = (see[y] >> e) & 1u ? v[y][e] : kNegInf;
          }
        };
        bool move = i == 0;  // (a unit's first turn has its maxima found in any case)
        if (!move) {
          if (ok && rows > 0) {
            scores(false);
            float most = kNegInf;
#pragma unroll
            for (int y = 0; y < SUB; ++y)
#pragma unroll
              for (int e = 0; e < HR; e += 2) most = max3(most, v[y][e], v[y][e + 1]);
            move = most > kMoves;
          }
          move = bar_or(vote, 128, move || !ok);
        }
        if (move) {
          // the turn's maxima; a row that one of them exceeds moves
          if (ok && rows > 0) {
            scores(true);
#pragma unroll
            for (int e = 0; e < HR; ++e) {
              float top = v[0][e];
#pragma unroll
              for (int y = 1; y < SUB; ++y) top = fmaxf(top, v[y][e]);
              top = warp_max(top);
              if (lane == 0) s_max[x][warp & 3][e] = top;
            }
          }
          if (it > 0) ok = ok && wait(bar(B::PVDONE), (it - 1) & 1);  // O is complete
          if (bar_or(vote, 128, !ok || *abort)) {  // (every warp of the group leaves here, or none)
            ok = false;
            break;
          }
          tc::fence_after();
          // Every warp writes the new maxima (the same) where the next turn finds them; the old ones stay
          // for the warps that are still here, and their place is taken at the next move, after its vote.
          float* to = s_nm[k & 3][nm == s_nm[k & 3][0] + x0] + x0;
          float al[HR];
#pragma unroll
          for (int e = 0; e < HR; ++e) {
            const float was = nm[e];
            const float top = fmaxf(fmaxf(s_max[x][0][e], s_max[x][1][e]), fmaxf(s_max[x][2][e], s_max[x][3][e]));
            const float now = rows > 0 && top + was > kMoves ? kRoom - top : was;
            al[e] = ex2(now - was);
            l[e] *= al[e];
#pragma unroll
            for (int y = 0; y < SUB; ++y) v[y][e] += now;
            if (lane == e) to[e] = now;
          }
          if (i > 0) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              float ov[HR];
              tmem_ld8_nowait(o_t + z * NR, ov);
              tmem_landed<HR>(ov);
#pragma unroll
              for (int e = 0; e < HR; ++e) ov[e] *= al[e];
              tmem_st8_nowait(o_t + z * NR, ov);
            }
            tmem_wait_st();
          }
          nm = to;
          __syncwarp();
        } else if (it > 0) {
          ok = ok && wait(bar(B::PVDONE), (it - 1) & 1);  // P's room is free
        }
        if (!ok) continue;  // (to the next vote)
        if (rows > 0) {
          // three terms of P', to bytes (term NR + row) of the key's line
#pragma unroll
          for (int y = 0; y < SUB; ++y) {
            uint32_t c[3][2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint16_t d[3][2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int e = q * 4 + z * 2;
                const float w0 = ex2(v[y][e]), w1 = ex2(v[y][e + 1]);
                const float2 ll = unpair(fma2(pair(w0, w1), pair(sc[y].z, sc[y].z), pair(l[e], l[e + 1])));
                l[e] = ll.x;
                l[e + 1] = ll.y;
                const __half2 hh = __floats2half2_rn(w0, w1);
                uint32_t h = *reinterpret_cast<const uint32_t*>(&hh);
                d[0][z] = e5m2x2_of(h);
                h = rest_of(h, d[0][z]);
                d[1][z] = e5m2x2_of(h);
                d[2][z] = e5m2x2_of(rest_of(h, d[1][z]));
              }
#pragma unroll
              for (int z = 0; z < 3; ++z) c[z][q] = d[z][0] | (uint32_t)d[z][1] << 16;
            }
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              const int col = z * NR + x0;
              const uint32_t to = at8<C::PW>(p_s + y * C::P_TILE, krow, col >> 4) + (col & 15);
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(to), "r"(c[z][0]), "r"(c[z][1]) : "memory");
            }
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        }
        tc::fence_before();
        __syncwarp();
        const bool last = i + SUB >= n, release = last || (i & 3) + SUB == 4;
        if (lane == 0) {
          tc::mbar_arrive(bar(B::PFULL));
          if (release) tc::mbar_arrive(bar(B::SCEMPTY + rsc.slot));
          if (last) tc::mbar_arrive(bar(B::QEMPTY + rq.slot));
        }
        if (release) rsc.next();
      }
      // ---------------------------------------------------------------- the unit's rows, or its part of them
      ok = ok && wait(bar(B::PVDONE), (it - 1) & 1);
      tc::fence_after();
      if (rows > 0) {
#pragma unroll
        for (int e = 0; e < HR; ++e) {
#pragma unroll
          for (int s = 16; s; s >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], s);
          if (lane == 0) s_sum[x][warp & 3][e] = l[e];
        }
      }
      if (bar_or(vote, 128, !ok)) break;  // (also after a timeout: every warp of the group comes here)
      if (rows > 0) {
        const bool whole = n == u.all;
        const int g = u.g;
        const int64_t slot = (int64_t)blockIdx.x * 2 + (u.a == 0);
        if (p.streamed && u.a == 0 && tid == 0)
          p.info[((int64_t)u.seq * p.hkv + g) * p.row_tiles + u.rt] = make_int2(blockIdx.x, u.ctas);
        int64_t tok = (int64_t)u.rt * NR + x0;  // token and head of the row
        int head = (int)(tok % p.R);
        tok = u.start + tok / p.R;
        float w[24];
#pragma unroll
        for (int y = 0; y < 3; ++y) tmem_ld8_nowait(o_t + y * NR, w + 8 * y);
        tmem_landed<24>(w);
#pragma unroll
        for (int e = 0; e < HR; ++e) {
          const float o = w[e] + (w[8 + e] + w[16 + e]);
          const float sum = (s_sum[x][0][e] + s_sum[x][1][e]) + (s_sum[x][2][e] + s_sum[x][3][e]), neg = nm[e];
          if (e < rows) {
            if (whole) {
              const int64_t rr = tok * p.h + g * p.R + head;
              if (krow < D) p.o[rr * D + krow] = __float2bfloat16(sum != 0.f ? o / sum : 0.f);
              if (p.lse && krow == 0) p.lse[rr] = sum != 0.f ? (log2f(sum) - neg) * kLn2 : kNegInf;
            } else {
              if (krow < D && sum != 0.f) p.part_o[(slot * NR + x0 + e) * D + krow] = o;
              if (krow == 0) p.part_ml[slot * NR + x0 + e] = make_float2(-neg, sum);
            }
          }
          if (++head == p.R) {
            head = 0;
            ++tok;
          }
        }
      }
      if (!u.more) break;
      rq.next();
    }
  }

  __syncthreads();
  if (warp == kLoadK || warp == kLoadV) {
    // After a timeout the copies still in flight land before the CTA leaves, else the last release of every slot.
    const int which = *abort ? B::FULL : B::EMPTY, first = warp == kLoadV ? NK : 0, ns = warp == kLoadV ? NV : NK;
    for (int st = 0; st < ns; ++st)
      if (const int i = last_in_stage(last_item, st, ns); i >= 0) tc::warp_drain(bar(which + first + st), (i / ns) & 1);
  } else if (warp == kIssue && *abort) {
    // products still in flight, too
    commit(bar(B::DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
    __syncwarp();
    tc::warp_drain(bar(B::DRAIN), 0);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_free(tmem, C::TMEM);
}

// ---------------------------------------------------------------------------- many rows over long caches
// More rows than the form above is made for: the rows are the products' M, as in span_attn.cu, and four warps
// turn the codes into f16 tiles (exact) beside the products,
//   S [128 rows x 128 keys] = Q K^T,   O [128 rows x d] += P V,
// with Q 2^a in f16 (exact down to 2^-32 of the row's largest element), P' = exp(t - m) sv 2^9 in f16, in TMEM
// over the scores it came from.  Scales stay with the scores and the weights, as above.  Four
// threads share a row, 32 keys each, and agree on its running maximum by a vote of their warps.  S of the next
// tile is issued before this one's P is waited for.
// 16 caches of up to 8192 keys, 8 tokens, 64 heads over 4 kv-heads of 128: 72.5 us, of which HBM 17 (136 in tiles of
// 32 rows by the form above, whose three terms of P cost too many conversions; 122 with those terms and the rows as M).
// A key tile takes about 3000 cycles: the conversion of its K and V 1600 and the softmax of its rows 2100, beside
// each other; shared memory moves 220 KB for it, 1750 cycles.  A CTA's 22 tiles are so 33 of the 72.5 us; the join takes 10,
// and the rest goes into starts and changes of unit, at which Q's one buffer and the converting warps' load of
// it let everything behind them run empty.
template <int D>
struct CfgR {
  static constexpr int NR = 128, SOFT = 16, CONV = 4, WARPS = SOFT + CONV + 3, THREADS = WARPS * 32;
  static constexpr int CODES = KT * D, TILE = KT * D * 2;  // bytes of a tile of codes, of a tile (or of Q) in f16
  static constexpr int NC = D == 64 ? 6 : 3, NF = D == 64 ? 6 : 4;  // slots of codes and of tiles, K and V in turn
  static constexpr int SMEM = TILE + NF * TILE + NC * CODES + 1024;
  static constexpr uint32_t TMEM = 512, O_COL = 256;
};
template <int NC, int NF>
struct BarsR {
  enum : int {
    CFULL = 0,           // [NC] codes
    CEMPTY = NC,
    FFULL = 2 * NC,      // [NF] tiles
    FEMPTY = FFULL + NF,
    SFULL = FEMPTY + NF,  // [2] S of a tile
    PFULL = SFULL + 2,   // [2] its P
    PVDONE = PFULL + 2,  // [2] its product
    SCFULL = PVDONE + 2,  // [4] scales of up to four tiles
    SCEMPTY = SCFULL + 4,
    QFULL = SCEMPTY + 4,
    QEMPTY = QFULL + 1,  // the unit's last S, and every softmax warp has begun the unit
    DRAIN = QEMPTY + 1,
    COUNT
  };
};

constexpr uint32_t idesc_f16(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

// 16 codes to 16 f16.
__device__ __forceinline__ void f16_of_codes(uint4 c, uint4* lo, uint4* hi) {
  lo->x = f16x2_of_e4m3((uint16_t)c.x), lo->y = f16x2_of_e4m3((uint16_t)(c.x >> 16));
  lo->z = f16x2_of_e4m3((uint16_t)c.y), lo->w = f16x2_of_e4m3((uint16_t)(c.y >> 16));
  hi->x = f16x2_of_e4m3((uint16_t)c.z), hi->y = f16x2_of_e4m3((uint16_t)(c.z >> 16));
  hi->z = f16x2_of_e4m3((uint16_t)c.w), hi->w = f16x2_of_e4m3((uint16_t)(c.w >> 16));
}

// Query rows 32 cw .. 32 cw + 31 of a unit as f16, max |q 2^a| in [2^14, 2^15), and what turns their scores into
// exponents of 2.  A warp's call; 16 bytes a lane, eight loads under way at a time.
template <int D>
__device__ __forceinline__ void load_q_f16(const Q8Params& p, const Walk<128>& u, uint32_t q_s, float* s_rs, int cw,
                                           int lane) {
  constexpr int LANES = D / 8, STEP = 32 / LANES;  // lanes of a row, rows of a load
  const int rows = u.s.rows(p, u.rt), col = lane % LANES * 8;
  const uint32_t group = (LANES == 16 ? 0xffffu : 0xffu) << (lane / LANES * LANES);
#pragma unroll 1
  for (int r0 = cw * 32 + lane / LANES; r0 < cw * 32 + 32; r0 += 8 * STEP) {
    uint4 w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = r0 + e * STEP;
      w[e] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const uint32_t rho = (uint32_t)u.rt * 128 + r, R = p.R;  // (a call of many rows does not come here)
        w[e] = *reinterpret_cast<const uint4*>(p.q + ((u.s.start + rho / R) * p.h + u.g * p.R + rho % R) * D + col);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = r0 + e * STEP;
      const uint32_t b[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
      uint32_t top = 0, h[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) top = max(top, max(b[z] << 16 & 0x7fffffffu, b[z] & 0x7fff0000u));
      top = __reduce_max_sync(group, top);
      const int ex = min(120, max(-120, 14 + 127 - (int)(top >> 23)));
      const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const __half2 y = __floats2half2_rn(__uint_as_float(b[z] << 16) * up, __uint_as_float(b[z] & 0xffff0000u) * up);
        h[z] = *reinterpret_cast<const uint32_t*>(&y);
      }
      st_shared(stage_at(q_s, KT * 128, r, col / 8), make_uint4(h[0], h[1], h[2], h[3]));
      // (a row with an infinity or NaN: its scores are NaN)
      if (col == 0)
        s_rs[r] = p.scale_log2 * __uint_as_float(top < 0x7f800000u ? (uint32_t)(127 - ex) << 23 : 0x7fc00000u);
      __syncwarp();
    }
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(CfgR<D>::THREADS, 1)
    attn_q8_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k16,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v16,
                        const Q8Params p) {
  using C = CfgR<D>;
  constexpr int NR = C::NR, NC = C::NC, NF = C::NF, SOFT = C::SOFT, CONV = C::CONV;
  using B = BarsR<NC, NF>;
  constexpr int kConv = SOFT, kLoad = SOFT + CONV, kIssue = kLoad + 1, kAux = kLoad + 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B::COUNT];
  __shared__ __align__(16) float4 s_sc[4][4][8];  // batch, tile, 16 keys: (sk, log2 sv, 1 / sv, whether there is a page)
  __shared__ float s_rs[2][NR];                   // scale log2(e) 2^-a of a row of unit k at k % 2
  __shared__ float s_max[4][NR], s_sum[4][NR];
  __shared__ int64_t s_scan[C::WARPS], s_at;
  __shared__ uint32_t s_tmem;
  __shared__ Part8 s_part[8];  // of unit k of the run, at k % 8
  __shared__ int s_abort, s_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = (smem_u32(smem_raw) + 1023) & ~1023u, tiles_s = q_s + C::TILE, codes_s = tiles_s + NF * C::TILE;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  volatile int* abort = &s_abort;

  launch_dependents();
  if (stopped()) return;
  const Waits wait(abort);
  Run8 r;
  if (!find_run<NR, C::WARPS>(p, r, s_scan, &s_seq, &s_at)) return;

  if (tid == 0) {
    for (int i = 0; i < NC; ++i) {
      tc::mbar_init(bar(B::CFULL + i), 1);
      tc::mbar_init(bar(B::CEMPTY + i), CONV);
    }
    for (int i = 0; i < NF; ++i) {
      tc::mbar_init(bar(B::FFULL + i), CONV);
      tc::mbar_init(bar(B::FEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(B::SFULL + i), 1);
      tc::mbar_init(bar(B::PFULL + i), SOFT);
      tc::mbar_init(bar(B::PVDONE + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(bar(B::SCFULL + i), 1);
      tc::mbar_init(bar(B::SCEMPTY + i), SOFT);
    }
    tc::mbar_init(bar(B::QFULL), CONV);
    tc::mbar_init(bar(B::QEMPTY), SOFT + 1);
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
  Walk<NR> u = p.streamed ? Walk<NR>(p, s_seq, s_at, r.places) : Walk<NR>(p, (int64_t)blockIdx.x);
  // whole steps of 32 keys: what lies past the keys is zeros
  auto width = [&](const Tiles& tl, int i) { return max(0, min(KT, (tl.width(i) + 31) & ~31)); };

  int last_item = -1;  // loading warp: the last tile handed to the ring of codes; issuing warp: the last one used
  if (u.n == 0) {
    // (a run that lies between two units)
  } else if (warp == kLoad) {
    // ------------------------------------------------------------------ codes of K and V tiles, in turn
    Turns<NR, 1> t(p, u);
    Ring<NC> rc;
    bool ok = true;
    for (; ok && t.more; t.next(p)) {
      const int i = t.u.a + t.j;
      const int pid = page_at(p.keys.c, t.u.seq, i * KT + (lane & 7) * GRAN, t.tl.sink_end, t.tl.shift, t.u.s.kv_len);
#pragma unroll 1
      for (int y = 0; y < 2; ++y) {
        if (last_item + 1 >= NC && !(ok = wait(bar(B::CEMPTY + rc.slot), rc.phase ^ 1u))) break;
        load_tile8<D>(codes_s + rc.slot * C::CODES, y ? &tm_v : &tm_k, y ? &tm_v16 : &tm_k16, y ? p.keys.v : p.keys.k,
                      p.keys.c, p.hkv, t.u.g, pid, i * KT, t.tl.sink_end, t.tl.shift, width(t.tl, i), t.u.s.kv_len,
                      bar(B::CFULL + rc.slot), lane);
        ++last_item;
        rc.next();
      }
    }
  } else if (warp >= kConv && warp < kConv + CONV) {
    // ------------------------------------------------------------------ codes to f16; queries
    const int cw = warp - kConv, ct = tid - kConv * 32;
    Turns<NR, 1> t(p, u);
    Ring<NC> rc;
    Ring<NF> rf;
    bool ok = true;
    int item = 0;
    for (int k = 0; ok && t.more;) {
      if (t.j == 0) {
        if (k > 0 && !(ok = wait(bar(B::QEMPTY), (k - 1) & 1))) break;
        load_q_f16<D>(p, t.u, q_s, s_rs[k & 1], cw, lane);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::QFULL));
        ++k;
      }
#pragma unroll 1
      for (int y = 0; y < 2; ++y, ++item) {
        if (!(ok = wait(bar(B::CFULL + rc.slot), rc.phase) &&
                   (item < NF || wait(bar(B::FEMPTY + rf.slot), rf.phase ^ 1u))))
          break;
        const uint32_t from = codes_s + rc.slot * C::CODES, to = tiles_s + rf.slot * C::TILE;
        // Eight lanes take four 16-byte chunks of two rows whose numbers differ in bits 0 and 2 (d = 128; of two rows
        // that follow one another for d = 64): other banks for each, of the codes and of the f16.
        constexpr int N = KT * (D / 16) / (CONV * 32);  // chunks of a thread
        const int j = ct >> 3, sub = ct >> 2 & 1;
#pragma unroll 1
        for (int e0 = 0; e0 < N; e0 += 4) {
          uint4 c[4];
          auto row_of = [&](int e) {
            return D == 128 ? (ct >> 5) * 8 + (e >> 1) * 32 + ((j & 3) * 2 ^ (sub ? 5 : 0)) : e * 32 + j * 2 + sub;
          };
          auto chunk_of = [&](int e) { return (ct & 3) + (D == 128 ? (e & 1) * 4 : 0); };
#pragma unroll
          for (int e = 0; e < 4; ++e) c[e] = ld_shared(at8<D>(from, row_of(e0 + e), chunk_of(e)));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 lo, hi;
            f16_of_codes(c[e], &lo, &hi);
            const int row = row_of(e0 + e), ch = 2 * chunk_of(e);
            st_shared(stage_at(to, KT * 128, row, ch), lo);
            st_shared(stage_at(to, KT * 128, row, ch + 1), hi);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar(B::FFULL + rf.slot));
          tc::mbar_arrive(bar(B::CEMPTY + rc.slot));
        }
        rc.next();
        rf.next();
      }
      if (ok) t.next(p);
    }
  } else if (warp == kAux) {
    // ------------------------------------------------------------------ per unit: description, scales
    Ring<4> rs;
    bool ok = true, again = false;
    for (int k = 0; ok; ++k) {
      const Tiles tl = u.s.tiles(p, u.rt);
      for (int i = 0; i < u.n; i += 4) {
        if (again && !(ok = wait(bar(B::SCEMPTY + rs.slot), rs.phase ^ 1u))) break;
        // (four batches are under way at most, so unit k - 8's description is no longer in use)
        if (i == 0 && lane == 0) describe<NR>(p, u, r, &s_part[k & 7]);
        const int tile = u.a + i + (lane >> 3), place = tile * KT + (lane & 7) * GRAN;
        const int key = place < tl.sink_end ? place : place + tl.shift;
        float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tile < u.a + u.n && place < tl.total && key < u.s.kv_len) {
          const int pid = page_of(p.keys.c, u.seq, key);
          if (pid >= 0) {
            const int pl = p.keys.c.page_log2, bl = p.keys.block_log2;
            const int64_t at = (((int64_t)pid * p.hkv + u.g) << (pl - bl)) + ((key & ((1 << pl) - 1)) >> bl);
            const float sv = __ldg(p.keys.vs + at);
            sc = make_float4(__ldg(p.keys.ks + at), log2f(sv), 1.f / sv, 1.f);
          }
        }
        s_sc[rs.slot][lane >> 3][lane & 7] = sc;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::SCFULL + rs.slot));
        rs.next();
        again |= rs.slot == 0;
      }
      if (!u.next(p)) break;
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------------------ products: S of tile it, then O of tile it - 1
    const uint32_t lead = elect(), q_d = desc_k(q_s), k_d = desc_k(tiles_s), v_d = desc_mn(tiles_s);
    constexpr uint32_t kSlot = C::TILE >> 4, kGroup = KT * 128 >> 4;
    Turns<NR, 1> ts(p, u), to = ts;
    Ring<NF> rk, rv;
    rv.next();
    bool ok = true;
    int k = 0;
    for (uint32_t it = 0; ok && to.more; ++it) {
      if (ts.more) {
        const int w = width(ts.tl, ts.u.a + ts.j);
        if (ts.j == 0 && !(ok = wait(bar(B::QFULL), k++ & 1))) break;
        if (!(ok = wait(bar(B::FFULL + rk.slot), rk.phase))) break;
        tc::fence_after();
        // (over the P of two tiles ago, whose product was issued before: products execute in issue order)
        const uint32_t s_t = tmem + (it & 1) * 128, kk = k_d + rk.slot * kSlot;
        const uint32_t id_s = idesc_f16(0) | (uint32_t)(w >> 3) << 17;
        if (w > 0) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_ss(s_t, q_d + (s >> 2) * kGroup + (s & 3) * 2, kk + (s >> 2) * kGroup + (s & 3) * 2, id_s, s > 0, lead);
        }
        commit(bar(B::SFULL + (it & 1)), lead);
        commit(bar(B::FEMPTY + rk.slot), lead);
        rk.next();
        rk.next();
        ts.next(p);
        if (ts.more && ts.j == 0) commit(bar(B::QEMPTY), lead);
      }
      if (it > 0) {
        const uint32_t b = (it - 1) & 1;
        if (!(ok = wait(bar(B::FFULL + rv.slot), rv.phase) && wait(bar(B::PFULL + b), ((it - 1) >> 1) & 1))) break;
        tc::fence_after();
        const int w = width(to.tl, to.u.a + to.j);
        const uint32_t vv = v_d + rv.slot * kSlot, p_t = tmem + b * 128;
        constexpr uint32_t id = idesc_f16(D) | kBMn;
        if (w == KT) {
#pragma unroll
          for (int s = 0; s < KT / 16; ++s)
            mma_ts(tmem + C::O_COL, p_t + s * 8, vv + s * (2048 >> 4), id, s > 0 || to.j > 0, lead);
        } else {
#pragma unroll
          for (int s = 0; s < KT / 16; ++s)
            if (s * 16 < w) mma_ts(tmem + C::O_COL, p_t + s * 8, vv + s * (2048 >> 4), id, s > 0 || to.j > 0, lead);
        }
        commit(bar(B::PVDONE + b), lead);
        commit(bar(B::FEMPTY + rv.slot), lead);
        last_item += 2;
        rv.next();
        rv.next();
        to.next(p);
      }
    }
  } else if (warp < SOFT) {
    // ------------------------------------------------------------------ softmax: quarter x of a row's keys
    constexpr int OC = D / 4;  // columns of O that a thread rescales and writes
    const int x = warp >> 2, row = tid & 127, vote = 1 + (warp & 3);  // (vote: the barrier of a row's warps)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16, o_t = tmem + C::O_COL + x * OC + lane_base;
    Ring<4> rsc;
    bool ok = true;
    uint32_t it = 0;  // tiles of the run
    for (int k = 0;; ++k) {
      ok = ok && wait(bar(B::SCFULL + rsc.slot), rsc.phase) && wait(bar(B::QFULL), k & 1);
      if (bar_or(vote, 128, !ok)) break;
      __syncwarp();
      const float rs = s_rs[k & 1][row];
      const volatile Part8& u = s_part[k & 7];
      const int n = u.n, rows = u.rows;
      const bool valid = row < rows, work = (warp & 3) * 32 < rows;
      const int pos = valid ? u.off + (int)(((uint32_t)u.rt * NR + row) / (uint32_t)p.R) : -1;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B::QEMPTY));
      // nm: minus the running maximum less kRoom; lim: what moves it (at first, any key)
      float nm = 0.f, l = 0.f, lim = kNegInf;
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++it) {
        const uint32_t b = it & 1, s_t = tmem + b * 128 + lane_base;
        if (i > 0 && (i & 3) == 0) ok = ok && wait(bar(B::SCFULL + rsc.slot), rsc.phase);
        ok = ok && wait(bar(B::SFULL + b), (it >> 1) & 1);
        tc::fence_after();
        const float4* sc = &s_sc[rsc.slot][i & 3][x * 2];
        float v[32];
        bool need = false;
        float top = kNegInf;
        if (ok && work) {
          tc::tmem_ld32_nowait(s_t + x * 32, v);
          tmem_wait_ld(v);
          uint32_t pages = 0;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 c = sc[g];
            pages |= (uint32_t)(c.w != 0.f) << g;
            const uint64_t f = pair(rs * c.x, rs * c.x), a = pair(c.y + nm, c.y + nm);
#pragma unroll
            for (int e = 16 * g; e < 16 * g + 16; e += 2) {
              const float2 y = unpair(fma2(pair(v[e], v[e + 1]), f, a));
              v[e] = y.x;
              v[e + 1] = y.y;
            }
          }
          if (i < u.full_lo || i >= u.full_hi || pages != 3u) {
            // seen columns: [j_lo, j_hi) and the sinks [0, j_sink) before j_hi
            const int at = u.a + i, key0 = at * KT + u.shift, w = min(KT, up16(u.total - at * KT));
            const int j_hi = min(pos + 1 - key0, w), j_lo = p.window > 0 ? pos - p.window + 1 - key0 : 0;
            const int j_sink = p.n_sink - at * KT - (u.sink_end > 0 ? 0 : u.shift);
            uint32_t see = bits(j_lo - x * 32, j_hi - x * 32) | bits(0, min(j_sink, j_hi) - x * 32);
            see &= (pages & 1u ? 0xffffu : 0u) | (pages & 2u ? 0xffff0000u : 0u);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (see >> e) & 1u ? v[e] : kNegInf;
          }
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], v[e], v[e + 1]);
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          need = valid && top > lim;
        }
        tc::fence_before();
        // (also: all four warps have read S, over which P goes)
        const bool move = bar_or(vote, 128, need || !ok);
        tc::fence_after();
        if (move) {
          if (ok) s_max[x][row] = top;
          if (it > 0) ok = ok && wait(bar(B::PVDONE + ((it - 1) & 1)), ((it - 1) >> 1) & 1);  // O is complete
          if (bar_or(vote, 128, !ok || *abort)) {
            ok = false;
            break;
          }
          tc::fence_after();
          if (work) {
            const float joint = fmaxf(fmaxf(s_max[0][row], s_max[1][row]), fmaxf(s_max[2][row], s_max[3][row]));
            const bool mine = valid && joint > lim;
            const float up = mine ? kRoom - joint : 0.f, al = lim == kNegInf ? 1.f : ex2(up);
            nm += up;
            l *= al;
            if (mine) lim = kMoves;
            const uint64_t up2 = pair(up, up);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = unpair(add2(pair(v[e], v[e + 1]), up2));
              v[e] = y.x;
              v[e + 1] = y.y;
            }
            if (i > 0) {
              __syncwarp();
#pragma unroll 1
              for (int c = 0; c < OC; c += 8) {
                float ov[8];
                tmem_ld8_nowait(o_t + c, ov);
                tmem_landed<8>(ov);
#pragma unroll
                for (int e = 0; e < 8; ++e) ov[e] *= al;
                tmem_st8_nowait(o_t + c, ov);
              }
              tmem_wait_st();
            }
          }
        }
        if (!ok) continue;  // (to the next vote)
        if (work) {
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint64_t sum = 0;
#pragma unroll
            for (int e = 16 * g; e < 16 * g + 16; e += 2) {
              const float e0 = ex2(v[e]), e1 = ex2(v[e + 1]);
              sum = add2(sum, pair(e0, e1));
              const __half2 h = __floats2half2_rn(e0, e1);
              pk[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const float2 y = unpair(sum);
            l = fmaf(y.x + y.y, sc[g].z, l);
          }
          tmem_st16_nowait(s_t + x * 16, pk);
          tmem_wait_st();
        }
        tc::fence_before();
        __syncwarp();
        const bool release = i + 1 == n || (i & 3) == 3;
        if (lane == 0) {
          tc::mbar_arrive(bar(B::PFULL + b));
          if (release) tc::mbar_arrive(bar(B::SCEMPTY + rsc.slot));
        }
        if (release) rsc.next();
      }
      // ---------------------------------------------------------------- the unit's rows, or its part of them
      ok = ok && wait(bar(B::PVDONE + ((it - 1) & 1)), ((it - 1) >> 1) & 1);
      tc::fence_after();
      s_sum[x][row] = l;
      if (bar_or(vote, 128, !ok)) break;  // (also after a timeout: all four warps come here)
      if (work) {
        const float sum = (s_sum[0][row] + s_sum[1][row]) + (s_sum[2][row] + s_sum[3][row]);
        const bool whole = n == u.all;
        const int g = u.g;
        const int64_t slot = (int64_t)blockIdx.x * 2 + (u.a == 0);
        const uint32_t rho = (uint32_t)u.rt * NR + row, R = p.R;
        const int64_t rr = (u.start + rho / R) * p.h + g * p.R + rho % R;
        if (p.streamed && u.a == 0 && tid == 0)
          p.info[((int64_t)u.seq * p.hkv + g) * p.row_tiles + u.rt] = make_int2(blockIdx.x, u.ctas);
        if (x == 0 && valid) {
          if (whole && p.lse) p.lse[rr] = sum != 0.f ? (log2f(sum) - nm) * kLn2 : kNegInf;
          if (!whole) p.part_ml[slot * NR + row] = make_float2(sum != 0.f ? -nm : kNone, sum);
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < OC; c += 8) {
          float ov[8];
          tmem_ld8_nowait(o_t + c, ov);
          tmem_landed<8>(ov);
          if (valid && whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ov[e] = sum != 0.f ? ov[e] * inv : 0.f;  // (a row without keys may hold no product)
            *reinterpret_cast<uint4*>(p.o + rr * D + x * OC + c) =
                make_uint4(pack_bf16(ov[0], ov[1]), pack_bf16(ov[2], ov[3]), pack_bf16(ov[4], ov[5]), pack_bf16(ov[6], ov[7]));
          } else if (valid && sum != 0.f) {
            float* to = p.part_o + (slot * NR + row) * D + x * OC + c;
            *reinterpret_cast<float4*>(to) = make_float4(ov[0], ov[1], ov[2], ov[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(ov[4], ov[5], ov[6], ov[7]);
          }
          __syncwarp();
        }
        tc::fence_before();  // (the next unit's first product writes O after these loads)
      }
      if (!u.more) break;
    }
  }

  __syncthreads();
  if (warp == kLoad && *abort) {
    // after a timeout the copies still in flight land before the CTA leaves
    for (int st = 0; st < NC; ++st)
      if (const int i = last_in_stage(last_item, st, NC); i >= 0) tc::warp_drain(bar(B::CFULL + st), (i / NC) & 1);
  } else if (warp == kIssue) {
    // and the products, and the last release of every slot
    if (u.n > 0) {
      commit(bar(B::DRAIN), elect());  // (the lane that issued: a commit covers its own products alone)
      __syncwarp();
      tc::warp_drain(bar(B::DRAIN), 0);
    }
    if (!*abort)
      for (int st = 0; st < NF; ++st)
        if (const int i = last_in_stage(last_item, st, NF); i >= 0) tc::warp_drain(bar(B::FEMPTY + st), (i / NF) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_free(tmem, C::TMEM);
}

// Joins the parts of a row in order: PW warps a row, each every PW-th part, then a sum over the warps.
// (The parts are written while this kernel starts: no read-only loads of them.)
template <int D, int NR, int PW>
__global__ void __launch_bounds__(256) q8_combine_kernel(const Q8Params p) {
  constexpr int E = D / 32, PER = 8 / PW;  // rows a block
  __shared__ float s_acc[8][D + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pw = warp % PW;
  const int64_t unit = blockIdx.x / (NR / PER);
  const int r = (int)(blockIdx.x % (NR / PER)) * PER + warp / PW;
  const int rt = (int)(unit % p.row_tiles), g = (int)(unit / p.row_tiles % p.hkv), seq = (int)(unit / p.row_tiles / p.hkv);
  Seq8<NR> s;
  s.load(p, seq);
  const bool mine = r < s.rows(p, rt);
  const int64_t rho = (int64_t)rt * NR + r, rr = (s.start + rho / p.R) * p.h + g * p.R + rho % p.R;
  wait_primary();
  if (device_stopped()) return;
  int2 who = make_int2(0, 0);
  if (mine) who = p.info[unit];
  who.x = max(0, min(who.x, p.ctas - 1));  // (whatever changed cu_seqlens meanwhile: within the workspace)
  const int parts = min(who.y, p.ctas - who.x);
  if (PW == 8 ? parts < 2 : __syncthreads_and(parts < 2)) return;  // (one part wrote the row itself)
  // part i: the first CTA's last unit, the others' first
  auto slot = [&](int i) { return ((int64_t)(who.x + i) * 2 + (i == 0)) * NR + r; };
  float m = kNone, acc[E] = {}, l = 0.f;
  if (parts > 1) {
    for (int i = lane; i < parts; i += 32) {
      const float2 ml = p.part_ml[slot(i)];
      if (ml.y != 0.f) m = fmaxf(m, ml.x);  // (NaN counts: it has to reach the row)
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int i0 = pw; i0 < parts; i0 += 32 * PW) {
      float w = 0.f, wl = 0.f;
      if (i0 + lane * PW < parts) {
        const float2 ml = p.part_ml[slot(i0 + lane * PW)];
        if (ml.y != 0.f) {
          w = ex2(ml.x - m);
          wl = w * ml.y;
        }
      }
      const int e1 = min(32, (parts - i0 + PW - 1) / PW);
#pragma unroll 4
      for (int i = 0; i < e1; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        l += __shfl_sync(0xffffffffu, wl, i);
        if (wi > 0.f) {
          const float* src = p.part_o + slot(i0 + i * PW) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 y = *reinterpret_cast<const float2*>(src + e);
            acc[e] = fmaf(wi, y.x, acc[e]);
            acc[e + 1] = fmaf(wi, y.y, acc[e + 1]);
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
  if (parts < 2) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.o + rr * D + lane * E + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse && lane == 0) p.lse[rr] = l != 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
}

// How a call is cut.
// Rows of a (sequence, kv-head) up to which the cache is the products' M.  16 caches of 6550 keys x 4 kv-heads,
// d = 128, us, as M and as N: 32 rows 46 and 61, 48 67 and 60, 64 66 and 61, 128 122 and 63.
constexpr int kFewRows8 = 32;
struct Plan8 {
  int nr, row_tiles, ctas;
  bool streamed;
  int64_t units;
  size_t ml, info, bytes;  // workspace: part_o at 0, part_ml at `ml`, info at `info`
};
static Plan8 make_plan8(const Seqs& s, int h, int hkv, int D) {
  Plan8 pl{};
  const int64_t rows = (int64_t)s.max_len * (h / hkv);
  pl.nr = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kFewRows8 ? 32 : 128;
  pl.row_tiles = (int)((rows + pl.nr - 1) / pl.nr);
  pl.units = (int64_t)pl.row_tiles * s.n_seqs * hkv;
  pl.ctas = (pl.nr <= 16 ? 2 : 1) * kSms8;
  pl.streamed = pl.units <= 4 * pl.ctas;
  if (!pl.streamed) return pl;
  const size_t part = (size_t)pl.ctas * 2 * pl.nr;
  pl.ml = part * D * 4;
  pl.info = pl.ml + part * 8;
  pl.bytes = pl.info + (size_t)pl.units * 8;
  return pl;
}

// ---------------------------------------------------------------------------- many rows
// With many rows a sequence the products bound the call, and each key is met by many row tiles: the seen
// part of the caches is expanded to bf16 pages of the workspace once (value = code * scale: exact
// for scales that are powers of two, else rounded once), and span_attn.cu's kernels read those.
struct Expand8 {
  Keys8 keys;
  Seqs seqs;
  int hkv, window, seq0;          // sequences seq0 .. of the call
  int bound;                      // table entries that lengths within the caller's bound reach
  int pages;                      // workspace pages of a sequence: those of the sinks, then those of the window
  int sink_pages;
  __nv_bfloat16 *k, *v;           // [sequences][pages][page][hkv][D]
  int32_t* table;                 // [sequences][bound]
  int32_t* lens;                  // [sequences]
};
// A block takes a page of a sequence (blockIdx.x: entry of the table) for all kv-heads.
template <int D>
__global__ void __launch_bounds__(256) expand_q8_kernel(const Expand8 x) {
  const int seq = x.seq0 + blockIdx.y, pl = x.keys.c.page_log2, page = 1 << pl, e = blockIdx.x;
  const int len = cached_len(x.keys.c, seq), Lq = seq_len(x.seqs, seq);
  const int kv_len = len > (int64_t)x.bound << pl ? 0 : len;  // (longer than the caller said: no keys, to be seen by that)
  // pages that some query sees: those of the sinks and from the first query's window on
  const int first = x.window > 0 ? max(0, kv_len - Lq - x.window + 1) >> pl : 0;
  const bool sink = e < x.sink_pages && e < first, seen = Lq > 0 && (e << pl) < kv_len && (sink || e >= first);
  const int at = sink || first <= x.sink_pages ? e : e - first + x.sink_pages;  // its place in the workspace
  const int pid = seen && at < x.pages ? page_of(x.keys.c, seq, e << pl) : -1;
  if (threadIdx.x == 0) {
    x.table[(int64_t)blockIdx.y * x.bound + e] = pid < 0 ? -1 : (int)blockIdx.y * x.pages + at;
    if (e == 0) x.lens[blockIdx.y] = kv_len;
  }
  if (pid < 0) return;
  constexpr int CH = D / 16;  // 16-byte chunks of a row
  const int bl = x.keys.block_log2, rows = min(page, kv_len - (e << pl)) * x.hkv;
  const int64_t to = ((int64_t)blockIdx.y * x.pages + at) * page * x.hkv * D, from = pid * x.keys.c.page_stride;
#pragma unroll 2
  for (int i = threadIdx.x; i < 2 * rows * CH; i += 256) {
    const bool is_v = i >= rows * CH;
    const int j = is_v ? i - rows * CH : i, r = j / CH / x.hkv, g = j / CH % x.hkv;
    const int64_t row = (int64_t)(j / CH) * D + j % CH * 16;
    const uint4 c = *reinterpret_cast<const uint4*>((is_v ? x.keys.v : x.keys.k) + from + row);
    const float s = __ldg((is_v ? x.keys.vs : x.keys.ks) + (((int64_t)pid * x.hkv + g) << (pl - bl)) + (r >> bl));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = f16x2_of_e4m3((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      o[k] = pack_bf16(f.x * s, f.y * s);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? x.v : x.k) + to + row);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// How a call of many rows is cut: sequences by groups whose pages fit the room, one after another.
// Rows a (sequence, kv-head) from which the caches are expanded: more than two row tiles.  Codes and expanded, us, d =
// 128: 8 caches of 16384 keys, 160 rows 47 and 67, 256 48 and 71, 512 67 and 73; 16 of 2048
// keys, 256 rows 34 and 43, 512 both 43; d = 64, 8 of 16384, 256 rows 42 and 52, 512 60 and 53.
constexpr int kManyRows = 257;
constexpr size_t kExpandRoom = (size_t)512 << 20;  // bytes of a group's pages, where more than a sequence's
struct Groups8 {
  int seqs, bound, pages, sink_pages;  // sequences of a group; table entries and workspace pages of each
  size_t v, table, lens, attn, bytes;  // workspace: K's pages at 0, the others there
};
static Groups8 make_groups8(const Seqs& s, int h, int hkv, int D, int max_keys, int page, int max_pages, int window,
                            int n_sink) {
  Groups8 gr{};
  int64_t pages = std::min<int64_t>(max_pages, ((int64_t)max_keys + page - 1) / page);
  gr.bound = (int)pages;
  if (window > 0) {
    gr.sink_pages = (int)std::min<int64_t>(pages, ((int64_t)n_sink + page - 1) / page);
    pages = std::min<int64_t>(pages, gr.sink_pages + ((int64_t)window + s.max_len + page - 1) / page + 1);
  }
  gr.pages = (int)pages;
  const size_t one = (size_t)pages * page * hkv * D * 2;
  gr.seqs = (int)std::max<int64_t>(1, std::min<int64_t>(s.n_seqs, (int64_t)(kExpandRoom / (2 * one))));
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  gr.v = up(one * gr.seqs);
  gr.table = 2 * gr.v;
  gr.lens = gr.table + up((size_t)gr.seqs * gr.bound * 4);
  gr.attn = gr.lens + up((size_t)gr.seqs * 4);
  Seqs part = s;
  part.n_seqs = gr.seqs;
  size_t need = span_attn_workspace_bytes(part, h, hkv, D, max_keys, window, n_sink);
  part.n_seqs = s.n_seqs % gr.seqs;  // the last group
  if (part.n_seqs) need = std::max(need, span_attn_workspace_bytes(part, h, hkv, D, max_keys, window, n_sink));
  gr.bytes = gr.attn + need;
  return gr;
}
static bool many_rows(const Seqs& s, int h, int hkv) { return (int64_t)s.max_len * (h / hkv) >= kManyRows; }

static cudaError_t launch_expanded(const Seqs& s, const void* q, const Keys8& keys, int h, int hkv, int D, int max_keys,
                                   int window, int n_sink, float scale, void* o, float* lse, void* workspace,
                                   cudaStream_t st) {
  const int page = 1 << keys.c.page_log2;
  const Groups8 gr = make_groups8(s, h, hkv, D, max_keys, page, keys.c.max_pages, window, n_sink);
  uint8_t* w = (uint8_t*)workspace;
  Expand8 x{};
  x.keys = keys;
  x.seqs = s;
  x.hkv = hkv;
  x.window = window;
  x.bound = gr.bound;
  x.pages = gr.pages;
  x.sink_pages = gr.sink_pages;
  x.k = (__nv_bfloat16*)w;
  x.v = (__nv_bfloat16*)(w + gr.v);
  x.table = (int32_t*)(w + gr.table);
  x.lens = (int32_t*)(w + gr.lens);
  for (int s0 = 0; s0 < s.n_seqs; s0 += gr.seqs) {
    Seqs part = s;
    part.n_seqs = std::min(gr.seqs, s.n_seqs - s0);
    x.seq0 = s0;
    const dim3 grid(gr.bound, part.n_seqs);
    if (D == 64)
      expand_q8_kernel<64><<<grid, 256, 0, st>>>(x);
    else
      expand_q8_kernel<128><<<grid, 256, 0, st>>>(x);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    PagedView c{};
    c.table = x.table;
    c.lens = x.lens;
    c.n_pages = part.n_seqs * gr.pages;
    c.page_log2 = keys.c.page_log2;
    c.max_pages = gr.bound;
    c.page_stride = (int64_t)page * hkv * D;
    const char* qs = (const char*)q;
    char* os = (char*)o;
    float* ls = lse;
    if (s.cu) {
      part.cu = s.cu + s0;  // (rows are counted from the packed start)
    } else {
      const int64_t row = (int64_t)s0 * s.T * h;
      qs += row * D * 2;
      os += row * D * 2;
      if (ls) ls += row;
      part.tokens = (int64_t)part.n_seqs * s.T;
    }
    e = launch_span_attn(part, qs, &c, x.k, x.v, h, hkv, D, max_keys, window, n_sink, scale, os, ls, w + gr.attn, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Maps of the codes of K (or V): the tile box and the 16-row box.
static bool byte_maps(CUtensorMap* big, CUtensorMap* small, const void* ptr, const Keys& c, int hkv, int D) {
  const uint32_t page = 1u << c.page_log2;
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[3] = {(uint64_t)hkv * D, page, (uint64_t)c.n_pages};
    const uint64_t strides[2] = {(uint64_t)hkv * D, (uint64_t)c.page_stride};
    const uint32_t box[3] = {(uint32_t)D, i ? (uint32_t)GRAN : (page < KT ? page : (uint32_t)KT), 1};
    if (!tc::make_map(i ? small : big, ptr, 3, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
      return false;
  }
  return true;
}

template <int D, int NR, typename C, typename Kern>
static cudaError_t run_q8(Kern kern, const CUtensorMap* m, const Q8Params& p, const Plan8& pl, cudaStream_t st) {
  // (the limit belongs to the kernel, and other threads launch it too: the same for every call)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t ctas = pl.streamed ? pl.ctas : pl.units;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)ctas, C::THREADS, C::SMEM, st>>>(m[0], m[1], m[2], m[3], p);
  if ((e = cudaGetLastError()) != cudaSuccess || !pl.streamed) return e;
  if (pl.units * 8 <= pl.ctas)
    return launch_second(q8_combine_kernel<D, NR, 8>, dim3((unsigned)(pl.units * NR)), 256, 0, st, p);
  return launch_second(q8_combine_kernel<D, NR, 1>, dim3((unsigned)(pl.units * NR / 8)), 256, 0, st, p);
}

template <int D>
static cudaError_t launch_q8_d(const Seqs& s, const void* q, const Keys8& keys, int h, int hkv, int window, int n_sink,
                               float scale, void* o, float* lse, void* workspace, cudaStream_t st) {
  const Plan8 pl = make_plan8(s, h, hkv, D);
  Q8Params p{};
  p.seqs = s;
  p.keys = keys;
  p.q = (const __nv_bfloat16*)q;
  p.o = (__nv_bfloat16*)o;
  p.lse = lse;
  p.part_o = (float*)workspace;
  p.part_ml = (float2*)((uint8_t*)workspace + pl.ml);
  p.info = (int2*)((uint8_t*)workspace + pl.info);
  p.h = h;
  p.hkv = hkv;
  p.R = h / hkv;
  p.window = window;
  p.n_sink = n_sink;
  p.row_tiles = pl.row_tiles;
  p.streamed = pl.streamed;
  p.ctas = pl.ctas;
  p.min_places = 2;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap m[4];
  if (!byte_maps(&m[0], &m[1], keys.k, keys.c, hkv, D) || !byte_maps(&m[2], &m[3], keys.v, keys.c, hkv, D))
    return cudaErrorInvalidValue;
  return pl.nr == 8    ? run_q8<D, 8, Cfg8<D, 8>>(attn_q8_kernel<D, 8>, m, p, pl, st)
         : pl.nr == 16 ? run_q8<D, 16, Cfg8<D, 16>>(attn_q8_kernel<D, 16>, m, p, pl, st)
         : pl.nr == 32 ? run_q8<D, 32, Cfg8<D, 32>>(attn_q8_kernel<D, 32>, m, p, pl, st)
                       : run_q8<D, 128, CfgR<D>>(attn_q8_rows_kernel<D>, m, p, pl, st);
}

}  // namespace span

size_t span_q8_workspace_bytes(const Seqs& s, int h, int hkv, int d, int max_keys, int page, int max_pages, int window,
                               int n_sink) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return 0;
  if (span::many_rows(s, h, hkv))
    return span::make_groups8(s, h, hkv, d, max_keys, page, max_pages, window, n_sink).bytes;
  return span::make_plan8(s, h, hkv, d).bytes;
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
  if (span::many_rows(s, h, hkv))
    return span::launch_expanded(s, q, keys, h, hkv, d, max_keys, window, n_sink, scale, o, lse, workspace, st);
  return d == 64 ? span::launch_q8_d<64>(s, q, keys, h, hkv, window, n_sink, scale, o, lse, workspace, st)
                 : span::launch_q8_d<128>(s, q, keys, h, hkv, window, n_sink, scale, o, lse, workspace, st);
}

NSA_STATUS_ACCESSOR(span_q8)

}  // namespace nsa
