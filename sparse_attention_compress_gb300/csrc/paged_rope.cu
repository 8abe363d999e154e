// Appending new tokens to a paged cache with the rotary rotation applied on the way: into the
// bf16 cache (append_rope_kernel) and into the cache held in 8 bits (append_q8_kernel).
//
// Rotation of a token at position p, pair i of n = rot / 2 (dimensions (i, i + n), or (2i, 2i + 1)):
//   a = p f_i;   (x, y) -> (x cos a - y sin a, x sin a + y cos a)
// in fp32, the angle reduced to a fraction of a turn without rounding that grows with p: f_i / 2pi
// is held as a 64-bit fixed-point fraction (turn_step), its product with the integer p wraps
// by itself, and the top 32 bits (2^-32 turns) go to sincospi.  fp64 would take 5 operations
// an angle at 2 a clock and SM.
//
// 8-bit blocks: value = code * s, code e4m3, s a power of two for each (page, kv-head, block of
// B tokens), the least with max |x| <= 448 s.  e4m3 has an exponent of its own, so a power of two
// costs no precision but at the ends of its range, and a scale that grows moves the earlier codes
// by whole binades: they are rounded again only where they reach e4m3's subnormals.
//
// Single tokens cost one launch (3.1 us for 32 tokens into the bf16 cache, 4.1 into 8 bits).  Four sequences
// of up to 2048 new tokens (16 query heads, 4 kv-heads of 128) take 18.3 us into the bf16 cache (81 MB read and
// written: 4.4 TB/s; its 1639 blocks are one and a half rounds, and two synchronisations come before a block's first
// load of values) and 24.2 us into 8 bits (74 MB; loads, angles, conversions and a block-wide maximum behind one
// another, three and a half rounds).
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "span.cuh"

namespace nsa {
namespace span {

// frac(f / 2pi) in units of 2^-64 turns: the 24-bit mantissa times 2^128 / 2pi, shifted.  (What
// is cut off is below 2^-63 turns per position for |f| <= 2pi.)
__device__ __forceinline__ uint64_t turn_step(float f) {
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // 2^128 / 2pi
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23 & 255u);
  const uint64_t m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int sh = (ex ? ex : 1) - 150;  // f = m 2^sh
  const uint64_t p0 = m * kLo, p1 = m * kHi + __umul64hi(m, kLo);
  const uint64_t p2 = __umul64hi(m, kHi) + (p1 < m * kHi ? 1u : 0u);
  uint64_t u;
  if (sh <= -128)
    u = 0;
  else if (sh <= -64)
    u = p2 >> (-sh - 64);
  else if (sh < 0)
    u = p1 >> -sh | p2 << (64 + sh);
  else if (sh == 0)
    u = p1;
  else
    u = sh < 64 ? p1 << sh | p0 >> (64 - sh) : 0;
  return b >> 31 ? 0 - u : u;
}
// (cos, sin) of position `pos`.
__device__ __forceinline__ float2 turn(uint64_t step, int pos) {
  const int t = (int)((step * (uint64_t)(int64_t)pos + 0x80000000ull) >> 32);  // 2^-32 turns
  float2 r;
  sincospif((float)t * 0x1p-31f, &r.y, &r.x);
  return r;
}

struct Rope {
  const float* inv_freq;   // [rot / 2]
  const int32_t* positions;  // [tokens], or NULL: the position in the cache
  int rot;                 // multiple of 16, at most d; 0: nothing is rotated
  int interleaved;
  const uint4* q;          // [tokens, h, d], or NULL
  uint4* q_out;
};

// A thread's item is two 16-byte chunks of a head, those of 8 pairs where the head is rotated:
// item j's pairs are 8j .. 8j + 7.
__device__ __forceinline__ int2 item_chunks(const Rope& rp, int j) {
  return j < rp.rot / 16 && !rp.interleaved ? make_int2(j, j + rp.rot / 16) : make_int2(2 * j, 2 * j + 1);
}
__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// x[0..7] and x[8..15]: the two chunks; cs(e): (cos, sin) of pair 8j + e.
template <typename CS>
__device__ __forceinline__ void rotate_item(float* x, bool interleaved, CS cs) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 c = cs(e);
    if (interleaved) {
      const float u = x[2 * e], v = x[2 * e + 1];
      x[2 * e] = fmaf(u, c.x, -v * c.y);
      x[2 * e + 1] = fmaf(u, c.y, v * c.x);
    } else {
      const float u = x[e], v = x[8 + e];
      x[e] = fmaf(u, c.x, -v * c.y);
      x[8 + e] = fmaf(u, c.y, v * c.x);
    }
  }
}

// Where a token goes (a warp's call): the sequence by a search of 32 probes a step.
struct Place {
  int seq;        // -1: a row of no sequence
  int64_t pos;    // position in the cache
};
__device__ __forceinline__ Place place_of(const Seqs& s, const int32_t* lens, int64_t tok, int lane) {
  Place r{-1, 0};
  if (tok >= s.tokens) return r;
  int lo = 0, n = s.n_seqs;  // the sequence is one of lo .. lo + n - 1
  if (!s.cu) {
    lo = (int)(tok / s.T);
  } else {
    while (n > 1) {
      const int step = (n + 31) / 32, i = lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, i < n && __ldg(s.cu + lo + i) <= tok);
      const int at = max(0, 31 - __clz(below)) * step;
      lo += at;
      n = min(step, n - at);
    }
  }
  const int64_t i = tok - seq_start(s, lo);
  const int Lq = seq_len(s, lo);
  if (i < 0 || i >= Lq) return r;
  r.seq = lo;
  r.pos = (int64_t)lens[lo] - Lq + i;
  return r;
}

// ---------------------------------------------------------------------------- bf16 cache
constexpr int kTok = 4;  // tokens a block of 256 threads: 64 angles each

// The heads of kTok tokens: h query heads, then K and V heads (q_only: the query heads alone).
// Angles once a token, in shared memory, for all its heads.
__device__ __forceinline__ void rope_tokens(const Seqs& s, const Keys& c, const Rope& rp, int64_t tok0, int n_tok,
                                            const uint4* k_new, const uint4* v_new, __nv_bfloat16* k_pages,
                                            __nv_bfloat16* v_pages, float* weights, int h, int hkv, int d, bool q_only) {
  __shared__ __align__(16) float2 s_cs[kTok * 64];
  __shared__ int64_t s_row[kTok], s_cell[kTok];  // element of the pool and cell of the weights (-1: no place)
  __shared__ int s_pos[kTok], s_ok[kTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp < n_tok) {
    const int64_t tok = tok0 + warp;
    const Place p = place_of(s, c.lens, tok, lane);
    int64_t row = -1, cell = 0;
    const int64_t cap = (int64_t)c.max_pages << c.page_log2;
    if (p.seq >= 0 && p.pos >= 0 && p.pos < cap) {
      const int pid = page_of(c, p.seq, (int)p.pos);
      const int slot = (int)p.pos & ((1 << c.page_log2) - 1);
      if (pid >= 0) {
        row = pid * c.page_stride + (int64_t)slot * hkv * d;
        cell = ((int64_t)pid * hkv << c.page_log2) + slot;
      }
    }
    if (lane == 0) {
      s_row[warp] = row;
      s_cell[warp] = cell;
      s_ok[warp] = p.seq >= 0;
      s_pos[warp] = p.seq < 0 ? 0 : rp.positions ? rp.positions[tok] : (int)p.pos;
    }
  }
  __syncthreads();
  const int pairs = rp.rot / 2;
  for (int i = tid; i < n_tok * pairs; i += blockDim.x) {
    const int t = i / pairs, e = i % pairs;
    s_cs[t * 64 + e] = turn(turn_step(__ldg(rp.inv_freq + e)), s_pos[t]);
  }
  __syncthreads();
  // A thread keeps its item j of a head and goes through the heads of the tokens, one after another: no divisions.
  const int per_log2 = d == 128 ? 3 : 2, j = tid & ((1 << per_log2) - 1), step = blockDim.x >> per_log2;
  const int nq = rp.q ? h : 0, heads = q_only ? nq : nq + 2 * hkv, cd = d / 8;
  const bool turned = j < rp.rot / 16;
  const int2 ch_k = item_chunks(rp, j), ch_v = make_int2(2 * j, 2 * j + 1);
  for (int t = 0, head = tid >> per_log2;; head += step) {
    while (head >= heads) {
      head -= heads;
      ++t;
    }
    if (t >= n_tok) break;
    if (!s_ok[t]) continue;
    const int64_t tok = tok0 + t;
    const uint4* src;
    uint4* dst;
    bool is_v = false;
    if (head < nq) {
      const int64_t row = (tok * h + head) * cd;
      src = rp.q + row;
      dst = rp.q_out + row;
    } else {
      if (s_row[t] < 0) continue;
      int g = head - nq;
      is_v = g >= hkv;
      if (is_v) g -= hkv;
      src = (is_v ? v_new : k_new) + (tok * hkv + g) * cd;
      dst = reinterpret_cast<uint4*>((is_v ? v_pages : k_pages) + s_row[t]) + g * cd;
      if (weights && !is_v && j == 0) weights[s_cell[t] + ((int64_t)g << c.page_log2)] = 0.f;
    }
    const int2 ch = is_v ? ch_v : ch_k;
    uint4 a = src[ch.x], b = src[ch.y];
    if (turned && !is_v) {
      float x[16];
      float4 cs[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = *reinterpret_cast<const float4*>(s_cs + t * 64 + j * 8 + 2 * e);
      unpack8(a, x);
      unpack8(b, x + 8);
      rotate_item(x, rp.interleaved != 0,
                  [&](int e) { return e & 1 ? make_float2(cs[e >> 1].z, cs[e >> 1].w) : make_float2(cs[e >> 1].x, cs[e >> 1].y); });
      a = pack8(x);
      b = pack8(x + 8);
    }
    dst[ch.x] = a;
    dst[ch.y] = b;
  }
}

__global__ void __launch_bounds__(256) append_rope_kernel(Seqs s, Keys c, Rope rp, int n_tok,
                                                          const uint4* __restrict__ k_new,
                                                          const uint4* __restrict__ v_new, __nv_bfloat16* k_pages,
                                                          __nv_bfloat16* v_pages, float* weights, int h, int hkv, int d) {
  rope_tokens(s, c, rp, (int64_t)blockIdx.x * n_tok, n_tok, k_new, v_new, k_pages, v_pages, weights, h, hkv, d, false);
}

// ---------------------------------------------------------------------------- 8-bit cache
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}
// Least power of two s in [2^-60, 2^60] with top <= 448 s.
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);  // 448 = 1.75 * 2^8
  return __uint_as_float((uint32_t)(min(60, max(-60, e)) + 127) << 23);
}

// Block b < kv_blocks takes one block of B cache positions of a (sequence, kv-head), of K or of V: its new
// values to registers (K rotated), their largest to the scale, the earlier codes rounded again where it
// grew, the new ones written.  The others, which take less time, rotate queries, kTok tokens each.
// kItems: items a thread holds in registers.  Blocks wait for memory, one load after another, so that the
// blocks an SM holds are what counts: 4 x 2048 tokens (h 16, h_kv 4, d 128) 42 us with
// 4 items and two blocks an SM, 29 with 2 and four, 26.5 with these blocks ahead of the queries, 25.2 with
// the values requested before the page is known, 24.2 with five (a few spilled registers; six: 25.2).
template <int kItems>
__global__ void __launch_bounds__(256, kItems == 4 ? 2 : 5)
    append_q8_kernel(Seqs s, Keys c, Rope rp, int kv_blocks, int n_tok, int block_log2, int blocks,
                     const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, uint8_t* k_pages,
                     uint8_t* v_pages, float* k_scales, float* v_scales, int h, int hkv, int d) {
  if ((int)blockIdx.x >= kv_blocks) {
    rope_tokens(s, c, rp, (int64_t)((int)blockIdx.x - kv_blocks) * n_tok, n_tok, nullptr, nullptr, nullptr, nullptr,
                nullptr, h, hkv, d, true);
    return;
  }
  __shared__ uint32_t s_top[8];
  const int tid = threadIdx.x, threads = blockDim.x;
  int u = (int)blockIdx.x;
  const bool is_v = u & 1;
  u >>= 1;
  const int g = u % hkv;
  u /= hkv;
  const int bi = u % blocks, seq = u / blocks;
  const int B = 1 << block_log2, Lq = seq_len(s, seq);
  const int64_t cap = (int64_t)c.max_pages << c.page_log2, end = min((int64_t)c.lens[seq], cap);
  const int64_t first = (int64_t)c.lens[seq] - Lq;  // the first new position
  const int64_t start = ((max(first, (int64_t)0) >> block_log2) + bi) << block_log2;
  if (start >= end) return;
  const int r0 = (int)(max(first, start) - start), r1 = (int)(min(start + B, end) - start);  // new rows of the block
  const int64_t tok0 = seq_start(s, seq) + start - first;  // row of the block's position 0
  const uint4* src = is_v ? v_new : k_new;
  const int per_log2 = d == 128 ? 3 : 2, j = tid & ((1 << per_log2) - 1);
  const int2 ch = is_v ? make_int2(2 * j, 2 * j + 1) : item_chunks(rp, j);
  const bool rotated = !is_v && j < rp.rot / 16;
  // (the values are requested before the page is looked up, and the angles' steps found while they arrive)
  uint4 in[kItems][2];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int r = r0 + ((tid + k * threads) >> per_log2);
    in[k][0] = in[k][1] = make_uint4(0, 0, 0, 0);
    if (r < r1) {
      const uint4* row = src + ((tok0 + r) * hkv + g) * (d / 8);
      in[k][0] = row[ch.x];
      in[k][1] = row[ch.y];
    }
  }
  const int pid = page_of(c, seq, (int)start);
  if (pid < 0) return;
  const int slot = (int)start & ((1 << c.page_log2) - 1);
  uint8_t* pages = (is_v ? v_pages : k_pages) + pid * c.page_stride + ((int64_t)slot * hkv + g) * d;
  float* scale = (is_v ? v_scales : k_scales) + (((int64_t)pid * hkv + g) << (c.page_log2 - block_log2)) +
                 (slot >> block_log2);
  const bool fresh = r0 == 0;
  const float was = fresh ? 0.f : *scale;

  float x[kItems][16];
  if (rotated) {
    uint64_t step[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) step[e] = turn_step(__ldg(rp.inv_freq + j * 8 + e));
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = r0 + ((tid + k * threads) >> per_log2);
      const int pos = r < r1 ? (rp.positions ? __ldg(rp.positions + tok0 + r) : (int)start + r) : 0;
      unpack8(in[k][0], x[k]);
      unpack8(in[k][1], x[k] + 8);
      rotate_item(x[k], rp.interleaved != 0, [&](int e) { return turn(step[e], pos); });
    }
  } else {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      unpack8(in[k][0], x[k]);
      unpack8(in[k][1], x[k] + 8);
    }
  }
  // the largest finite value (bits of non-negative floats are in their order)
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kItems; ++k)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t b = __float_as_uint(x[k][e]) & 0x7fffffffu;
      top = max(top, b < 0x7f800000u ? b : 0u);
    }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
  for (int w = 0; w < threads / 32; ++w) top = max(top, s_top[w]);
  const float need = scale_for(__uint_as_float(top));
  const float sc = was > need ? was : need;
  if (!fresh && need > was) {
    const float ratio = was / need;
    for (int i = tid; i < r0 << per_log2; i += threads) {
      uint4* at = reinterpret_cast<uint4*>(pages + (int64_t)(i >> per_log2) * hkv * d) + j;
      const uint4 old = *at;
      const uint32_t w[4] = {old.x, old.y, old.z, old.w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = from_e4m3x2((uint16_t)w[e]), b = from_e4m3x2((uint16_t)(w[e] >> 16));
        o[e] = to_e4m3x2(a.x * ratio, a.y * ratio) | (uint32_t)to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
      }
      *at = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (tid == 0) *scale = sc;
  const float inv = 1.f / sc;
  const bool whole = (__float_as_uint(sc) & 0x7fffffu) == 0;  // a power of two: x inv is x / sc
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int r = r0 + ((tid + k * threads) >> per_log2);
    if (r >= r1) break;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[k][e] = whole ? x[k][e] * inv : __fdiv_rn(x[k][e], sc);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = to_e4m3x2(x[k][4 * e], x[k][4 * e + 1]) | (uint32_t)to_e4m3x2(x[k][4 * e + 2], x[k][4 * e + 3]) << 16;
    uint2* at = reinterpret_cast<uint2*>(pages + (int64_t)r * hkv * d);
    at[ch.x] = make_uint2(o[0], o[1]);
    at[ch.y] = make_uint2(o[2], o[3]);
  }
}

static Rope rope_of(const RopeArgs* a) {
  Rope r{};
  if (!a) return r;
  r.inv_freq = a->inv_freq;
  r.positions = a->positions;
  r.rot = a->rot;
  r.interleaved = a->interleaved;
  r.q = (const uint4*)a->q;
  r.q_out = (uint4*)a->q_out;
  return r;
}
// Tokens a block: single tokens spread over the SMs, chunks share the angles' set-up.
static int tokens_a_block(int64_t tokens) { return tokens >= 1024 ? kTok : 1; }

}  // namespace span

cudaError_t launch_paged_append_rope(const Seqs& s, const void* k_new, const void* v_new, const RopeArgs& rope,
                                     const PagedView& cache, void* k_pages, void* v_pages, float* weights, int h,
                                     int hkv, int d, cudaStream_t st) {
  if (s.tokens == 0 || s.n_seqs == 0) return cudaSuccess;
  const int n = span::tokens_a_block(s.tokens);
  span::append_rope_kernel<<<(unsigned)((s.tokens + n - 1) / n), 256, 0, st>>>(
      s, span::keys_of(&cache, nullptr, nullptr), span::rope_of(&rope), n, (const uint4*)k_new, (const uint4*)v_new,
      (__nv_bfloat16*)k_pages, (__nv_bfloat16*)v_pages, weights, h, hkv, d);
  return cudaGetLastError();
}

cudaError_t launch_paged_q8_append(const Seqs& s, const void* k_new, const void* v_new, const RopeArgs* rope,
                                   const PagedView& cache, void* k_pages, void* v_pages, float* k_scales,
                                   float* v_scales, int block_log2, int h, int hkv, int d, cudaStream_t st) {
  if (s.tokens == 0 || s.n_seqs == 0 || s.max_len == 0) return cudaSuccess;
  const int n = span::tokens_a_block(s.tokens), B = 1 << block_log2;
  const int64_t q_blocks = rope && rope->q ? (s.tokens + n - 1) / n : 0;
  // a run of max_len positions touches at most this many blocks
  const int blocks = (s.max_len - 1 + B - 1) / B + 1;
  const int64_t kv_blocks = (int64_t)blocks * s.n_seqs * hkv * 2, all = q_blocks + kv_blocks;
  if (all > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int items = std::min(B, s.max_len) * (d / 16), threads = items <= 128 ? 128 : 256;
  auto go = [&](auto kern) {
    kern<<<(unsigned)all, threads, 0, st>>>(s, span::keys_of(&cache, nullptr, nullptr), span::rope_of(rope),
                                            (int)kv_blocks, n, block_log2, blocks, (const uint4*)k_new, (const uint4*)v_new,
                                            (uint8_t*)k_pages, (uint8_t*)v_pages, k_scales, v_scales, h, hkv, d);
  };
  if (items <= threads)
    go(span::append_q8_kernel<1>);
  else if (items <= 2 * threads)
    go(span::append_q8_kernel<2>);
  else
    go(span::append_q8_kernel<4>);
  return cudaGetLastError();
}

}  // namespace nsa
