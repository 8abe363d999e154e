// Pieces shared by the kernels whose queries see a span of a sequence's keys: attention
// over a paged cache (span_attn.cu), the accumulated attention weights (span_weights.cu)
// and the sliding window with sinks and its backward (span_attn.cu, span_bwd.cu).
//
// A query at position p sees key j when j <= p and (window == 0, or j > p - window, or
// j < n_sink).  The rows of one CTA are consecutive positions p_first .. p_last, so the
// keys any of them sees are at most two spans: the sinks [0, n_sink) and
// [p_first - window + 1, p_last].  The spans, one after the other (each starting on a
// multiple of 16 keys), are walked in 128-key tiles whose last one is cut to a multiple of
// 16 (the granularity of the tensor-core N and K extents), so a few sinks cost 16 columns of
// a tile and not a tile.
#pragma once

#include "launch.h"
#include "sm100.cuh"

namespace nsa {
namespace span {

constexpr int KT = 128;     // keys per tile
constexpr int ROWS = 128;   // (token, head) rows per tile
constexpr int GRAN = 16;    // key granularity of a tile's width

// Keys and values.  table == nullptr: packed rows [tokens, hkv, D] of the query sequences
// themselves.  Otherwise pages [n_pages][page_stride elements] of 2^page_log2 rows
// [hkv, D]; row `seq` of the table lists a sequence's pages.
struct Keys {
  const __nv_bfloat16 *k, *v;
  const int32_t* table;
  const int32_t* lens;  // cached tokens of each sequence, its new tokens included
  int n_pages, page_log2, max_pages;
  int64_t page_stride;
};

// Cached tokens of a sequence, within what its table row can hold.
__device__ __forceinline__ int cached_len(const Keys& c, int seq) {
  const int64_t cap = (int64_t)c.max_pages << c.page_log2;
  const int n = c.lens[seq];
  return n < 0 ? 0 : (n > cap ? (int)cap : n);
}

// Page of key `key` of a sequence, or -1 when the table holds no valid page for it.
__device__ __forceinline__ int page_of(const Keys& c, int seq, int key) {
  const int pid = __ldg(c.table + (int64_t)seq * c.max_pages + (key >> c.page_log2));
  return (unsigned)pid < (unsigned)c.n_pages ? pid : -1;
}

inline Keys keys_of(const PagedView* c, const void* k, const void* v) {
  Keys r{};
  r.k = (const __nv_bfloat16*)k;
  r.v = (const __nv_bfloat16*)v;
  if (c) {
    r.table = c->table;
    r.lens = c->lens;
    r.n_pages = c->n_pages;
    r.page_log2 = c->page_log2;
    r.max_pages = c->max_pages;
    r.page_stride = c->page_stride;
  }
  return r;
}

__host__ __device__ __forceinline__ int up16(int x) { return (x + GRAN - 1) & ~(GRAN - 1); }

// The key tiles that rows at positions p_first .. p_last see (at least in part).  Column c of
// tile i is place 128 i + c of the two spans: key `place` below sink_end, place + shift from
// there on.
struct Tiles {
  int sink_end, shift, total, n;
  __device__ __forceinline__ Tiles(int p_first, int p_last, int window, int n_sink) {
    const int hi = p_last + 1;
    int lo = window > 0 ? max(0, p_first - window + 1) & ~(GRAN - 1) : 0;
    sink_end = up16(n_sink);
    if (window == 0 || n_sink == 0) sink_end = 0;
    if (lo <= sink_end && sink_end > 0) lo = sink_end = 0;  // the spans meet: one span
    shift = lo - sink_end;
    total = hi > lo ? sink_end + hi - lo : 0;
    n = (total + KT - 1) / KT;
  }
  __device__ __forceinline__ int width(int i) const { return min(KT, up16(total - i * KT)); }
  // key of column 0 of tile i, counted in the last span
  __device__ __forceinline__ int key0(int i) const { return i * KT + shift; }
  // columns of tile i before this one are sinks
  __device__ __forceinline__ int sinks(int i, int n_sink) const {
    return n_sink - i * KT - (sink_end > 0 ? 0 : shift);
  }
};

// One warp fills a tile of `w` (a multiple of 16) rows x D of kv-head g, the keys at places
// place0 .. place0 + w - 1 (Tiles: key `place` below sink_end, place + shift from there on),
// in the 128-byte-swizzled layout (64-column groups KT * 128 bytes apart), and lane 0 arrives
// on `bar` with the bytes still to come.  The rows travel as TMA boxes, issued by as many
// lanes as there are boxes: whole pages (at most 128 rows) when the tile is whole and starts
// on a page, else 16 rows.  What holds no key (rows at or past kv_len, rows of a page the
// table does not name) is written as zeros by plain bounds-checked copies, so whatever lies
// there (NaN included) never meets a product.
template <int D, bool PAGED>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* big, const CUtensorMap* small,
                                          const __nv_bfloat16* src, const Keys& c, int hkv, int g, int seq,
                                          int64_t start, int place0, int sink_end, int shift, int w, int kv_len,
                                          uint32_t bar, int lane) {
  constexpr int H = D / 64;
  const int page = PAGED ? 1 << c.page_log2 : KT;
  const int box = page < KT ? page : KT;
  const int first = place0 + shift;
  const bool whole =
      w == KT && place0 >= sink_end && first + KT <= kv_len && (!PAGED || (first & (box - 1)) == 0);
  const int br = whole ? box : GRAN;
  const int n = w / br;
  const int ci = lane / H, hf = lane % H;
  const bool mine = ci < n;
  const int place = place0 + ci * br, key = place < sink_end ? place : place + shift;
  int pid = 0;
  if (PAGED) pid = mine && key < kv_len ? page_of(c, seq, key) : 0;
  const bool ok = pid >= 0;
  const bool plain = mine && (!ok || key + br > kv_len);
  if (mine && !plain) {
    const uint32_t to = dst + hf * (KT * 128) + ci * br * 128;
    if (PAGED)
      tc::tma3d(to, whole ? big : small, g * D + hf * 64, key & (page - 1), pid, bar);
    else
      tc::tma2d(to, whole ? big : small, g * D + hf * 64, (int)(start + key), bar);
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, mine && !ok && hf == 0);
  uint32_t todo = __ballot_sync(0xffffffffu, plain && hf == 0);
  const int bytes = (n - __popc(todo)) * br * D * 2;
  if (todo) {
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int cc = l / H;
      const bool okc = !((bad >> l) & 1u);
      const int64_t pidc = __shfl_sync(0xffffffffu, pid, l);
      const int keyc = __shfl_sync(0xffffffffu, key, l);
      for (int e = lane; e < br * (D / 8); e += 32) {
        const int r = cc * br + e / (D / 8), ch = e % (D / 8);
        const int kk = keyc + e / (D / 8);
        const bool in = okc && kk < kv_len;
        const int64_t row = PAGED ? pidc * c.page_stride + (int64_t)(kk & (page - 1)) * hkv * D
                                  : (start + kk) * hkv * D;
        cp_async16(dst + (ch >> 3) * (KT * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                   in ? (const void*)(src + row + g * D + ch * 8) : (const void*)src, in ? 16 : 0);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncwarp();
  if (lane == 0) tc::mbar_expect_tx(bar, (uint32_t)bytes);
}

// A bit for every 16-row group of a tile that the table names no page for (a warp's call).
__device__ __forceinline__ uint32_t missing_groups(const Keys& c, int seq, const Tiles& t, int i, int kv_len, int lane) {
  const int place = i * KT + lane * GRAN, key = place < t.sink_end ? place : place + t.shift;
  return __ballot_sync(0xffffffffu, lane * GRAN < t.width(i) && key < kv_len && page_of(c, seq, key) < 0);
}

// ------------------------------------------------------------------ products
// The issuing warp shares its scheduler with softmax warps, so every instruction it needs
// per product shows up as tensor-core time.  All its lanes run the same code (operands then
// stay in uniform registers) and one elected lane's products and commits take effect;
// descriptors differ from a per-tile base by constants.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n.reg .pred q;\n.reg .b32 l;\nelect.sync l|q, 0xffffffff;\nselp.b32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Low words of the shared-memory descriptors (address and leading offset); the high word is
// the same for both: 8 rows of 128 bytes to an atom, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major tile (tc::sdesc), and MN-major tile with 64-element groups KT * 128 bytes apart.
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFF) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) {
  return ((saddr & 0x3FFFF) >> 4) | ((uint32_t)(KT * 128 >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum, uint32_t lead) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "mov.b64 x, {%1, %6};\nmov.b64 y, {%2, %6};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accum), "r"(lead), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum, uint32_t lead) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 y;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "mov.b64 y, {%2, %6};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accum), "r"(lead), "n"(kDescHi)
      : "memory");
}
constexpr uint32_t kBMn = 1u << 16;  // instruction descriptor: B is MN-major

// S[128 x w] = A[128 x D] B[w x D]^T, both K-major tiles (64-column groups 16 KB apart, A's
// a_group descriptor units); a and b: desc_k of their bases.
template <int D>
__device__ __forceinline__ void mma_abt(uint32_t d_tmem, uint32_t a, uint32_t b, int w, uint32_t lead,
                                        uint32_t a_group = KT * 128 >> 4) {
  const uint32_t id = tc::idesc(ROWS, w);
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    mma_ss(d_tmem, a + (s >> 2) * a_group + (s & 3) * 2, b + (s >> 2) * (KT * 128 >> 4) + (s & 3) * 2, id, s > 0,
           lead);
}
// O[128 x D] (+)= P[128 x w] (bf16 in TMEM) V[w x D], V a tile of w rows read MN-major (v:
// desc_mn of its base): the steps S0 .. S1 - 1 of 16 keys.
template <int D, int S0, int S1>
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v, int w, bool first, uint32_t lead) {
  constexpr uint32_t id = tc::idesc(ROWS, D) | kBMn;
  if (w >= S1 * 16) {
#pragma unroll
    for (int s = S0; s < S1; ++s)
      mma_ts(d_tmem, p_tmem + s * 8, v + s * (2048 >> 4), id, s == 0 ? !first : 1u, lead);
  } else {
#pragma unroll
    for (int s = S0; s < S1; ++s)
      if (s * 16 < w) mma_ts(d_tmem, p_tmem + s * 8, v + s * (2048 >> 4), id, s == 0 ? !first : 1u, lead);
  }
}

// A wait ran out in an earlier kernel or CTA: the block leaves.  One answer for all its threads
// (the word may change between their reads, and some would go on without the others' set-up).
__device__ __forceinline__ bool stopped() { return __syncthreads_or(tc::device_status_set()); }

// Bounded wait of a warp for phase `parity` (tc::warp_wait's rules: abort flag, time limit,
// status word), inline: a call would keep the caller's registers in local memory across it,
// and with nearly all of L1 given to shared memory that is a trip to L2 or DRAM per wait.
// `quick`: the limit is below tc::kQuickNs (one unsuccessful probe gives up).
struct Waits {
  volatile int* abort;
  bool quick;
  __device__ __forceinline__ explicit Waits(volatile int* a) : abort(a), quick(tc::wait_limit() < tc::kQuickNs) {}
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    bool ok = quick ? tc::mbar_test(bar, parity) : tc::mbar_try(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
      const unsigned long long t0 = tc::globaltimer(), lim = tc::wait_limit();
      const uint32_t hint = lim < 10000000ull ? (uint32_t)lim : 10000000u;
      while (!quick && !ok && !(ok = tc::mbar_try_for(bar, parity, hint)) && !*abort && tc::globaltimer() - t0 < lim) {
      }
      if (!ok && !*abort) {
        *abort = 1;
        atomicExch(&g_device_status, (int)NSA_ERR_TIMEOUT);
      }
      return __all_sync(0xffffffffu, ok);
    }
    return true;
  }
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

// 32 TMEM columns whose load was issued with tc::tmem_ld32_nowait: waits for every load of
// the thread so far and makes v's registers depend on the wait.
__device__ __forceinline__ void tmem_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])::"memory");
}

// Starts the load of 32 columns if `on`; else the registers get a value all the same (what a
// skipped load would leave in them is their last one, which would keep them occupied from
// tile to tile).
__device__ __forceinline__ void tmem_ld32_if(bool on, uint32_t taddr, float* v) {
  if (on) {
    tc::tmem_ld32_nowait(taddr, v);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = 0.f;
  }
}

// Two fp32 operations in one instruction (a pair in a 64-bit register).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Bits lo .. hi - 1 of a word, clamped to 0 .. 32.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : (hi <= 0 ? 0u : (1u << hi) - 1u);
  const uint32_t below_lo = lo >= 32 ? ~0u : (lo <= 0 ? 0u : (1u << lo) - 1u);
  return below_hi & ~below_lo;
}

// TMEM stores of 16 words without the wait (the caller issues tmem_wait_st).
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t holder, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(holder), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols) : "memory");
}

// A call's kernels follow one another without the gap of a launch: the second one's blocks start
// as the first one's last blocks leave room, set themselves up, and wait for the first to be
// complete before they read what it wrote.  (Every block of a first kernel says so at its start;
// every block of a second one waits, so that whoever waits for the second waits for both.)
// On the device, 3 x 1001 tokens forward and backward 80 -> 76 us (77 now), a cache of 4096 keys cut to
// 1024 13.6 -> 12.8 (12.3 now);
// the attention's parts, whose waiting blocks would take room from the last round of others, gain
// nothing (decode 146 -> 148) and are joined by an ordinary launch.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_primary() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Output rows staged in shared memory (the layout of the tiles: 64-column groups `group`
// bytes apart, 16-byte chunk ch of row r at chunk ch ^ (r & 7)), so that they leave by TMA
// or in whole lines: a warp whose threads wrote a row each would touch 32 lines per store.
__device__ __forceinline__ uint32_t stage_at(uint32_t base, uint32_t group, int r, int ch) {
  return base + (ch >> 3) * group + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 32 columns c .. c + 31 of a row, times f, as bf16 to the stage.
__device__ __forceinline__ void stage_cols(uint32_t base, uint32_t group, int r, int c, const float* v, float f) {
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    uint4 u;
    u.x = pack_bf16(v[e] * f, v[e + 1] * f);
    u.y = pack_bf16(v[e + 2] * f, v[e + 3] * f);
    u.z = pack_bf16(v[e + 4] * f, v[e + 5] * f);
    u.w = pack_bf16(v[e + 6] * f, v[e + 7] * f);
    st_shared(stage_at(base, group, r, (c + e) / 8), u);
  }
}
// A staged tile of D / 64 column groups to the rows of a query map (one thread, after every
// writer's fence and a barrier); returns once shared memory has been read.
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t base, uint32_t group, int head, int tok) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c * 64), "r"(head), "r"(tok), "r"(base + c * group)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
// The staged rows 0 .. rows - 1 (token r / R, head r % R; those of the first t_left tokens)
// to dst, the first row's place; `threads` threads, this one `i`.
template <int D>
__device__ __forceinline__ void unstage_rows(uint32_t base, uint32_t group, int rows, int R, int h, int t_left,
                                             __nv_bfloat16* dst, int i, int threads) {
  constexpr int CH = D / 8;
#pragma unroll 4
  for (int e = i; e < rows * CH; e += threads) {
    const int r = e / CH, ch = e % CH, tl = r / R;
    if (tl < t_left)
      *reinterpret_cast<uint4*>(dst + ((int64_t)tl * h + r % R) * D + ch * 8) = ld_shared(stage_at(base, group, r, ch));
  }
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------------- host side
template <typename... P, typename... A>
cudaError_t launch_second(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, static_cast<P>(args)...);
}
// Maps of K (or V): the tile box and the 16-row box.
inline bool key_maps(CUtensorMap* big, CUtensorMap* small, const void* ptr, const Keys& c, int hkv, int D,
                     int64_t packed_rows) {
  for (int i = 0; i < 2; ++i) {
    if (c.table) {
      const uint32_t page = 1u << c.page_log2;
      const uint64_t dims[3] = {(uint64_t)hkv * D, page, (uint64_t)c.n_pages};
      const uint64_t strides[2] = {(uint64_t)hkv * D * 2, (uint64_t)c.page_stride * 2};
      const uint32_t box[3] = {64, i ? (uint32_t)GRAN : (page < KT ? page : (uint32_t)KT), 1};
      if (!tc::make_map(i ? small : big, ptr, 3, dims, strides, box)) return false;
    } else {
      const uint64_t dims[2] = {(uint64_t)hkv * D, (uint64_t)packed_rows};
      const uint64_t strides[1] = {(uint64_t)hkv * D * 2};
      const uint32_t box[2] = {64, i ? (uint32_t)GRAN : (uint32_t)KT};
      if (!tc::make_map(i ? small : big, ptr, 2, dims, strides, box)) return false;
    }
  }
  return true;
}
// Map of query rows [tokens, h, D]: a box is 64 columns of R heads of tpc tokens.
inline bool query_map(CUtensorMap* m, const void* ptr, int64_t tokens, int h, int D, int R, int tpc) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)h, (uint64_t)tokens};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)h * D * 2};
  const uint32_t box[3] = {64, (uint32_t)R, (uint32_t)tpc};
  return tc::make_map(m, ptr, 3, dims, strides, box);
}

}  // namespace span
}  // namespace nsa
