// paged_cache.cuh -- the paged key-value cache's writers for sm_100a: a step's
// keys and values appended to the pages a block table names (rotated, bf16 or
// fp8), and the mean key of every completed block.
//
// Both move each byte once and compute next to nothing, so memory bounds the
// long bf16 calls and the launch the short ones; the fp8 format (a maximum, a
// scale and a conversion per feature) makes the long fp8 calls bound by
// instructions. A head row (128 features) lies across 8 or 16 neighbouring
// lanes: the rotation's partner features sit in the same lane (interleaved
// pairs) or a fixed number of lanes away (halves), and so do the 32 features of
// an e8m0 scale.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace dsa {

constexpr int kRowD = 128;               // features of a head row

struct PagedGeom {
  int num_seqs, H_kv;
  int page_shift;                        // log2(page_size)
  int pages_per_seq, num_pages;
  int64_t page_stride, slot_stride, head_stride;   // elements
  const int *table;

  __host__ __device__ int64_t capacity() const {
    return static_cast<int64_t>(pages_per_seq) << page_shift;
  }
};

// Element offset of slot `slot` of sequence `seq` for head 0, or -1 where the
// table has no page of the pool for it. 0 <= seq < num_seqs, 0 <= slot <
// capacity.
__device__ __forceinline__ int64_t paged_slot(const PagedGeom &g, int seq, int slot) {
  const int page = __ldg(g.table + static_cast<int64_t>(seq) * g.pages_per_seq +
                         (slot >> g.page_shift));
  if (page < 0 || page >= g.num_pages) return -1;
  return page * g.page_stride + (slot & ((1 << g.page_shift) - 1)) * g.slot_stride;
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t *>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Two fp32 values as e4m3 (nearest, ties to even; |x| <= 448 here).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// Two e4m3 bytes (low 16 bits of v) as fp32, exactly.
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

// The e8m0 byte of 32 features whose largest magnitude has the bits `top`, or
// 255 where one is a NaN or an infinity (their bits compare above every
// number's). 448 = 1.75 * 2^8, so the least e with amax <= 448 * 2^e is
// amax's exponent less 8, plus one where its fraction is above .75: one integer
// addition to amax's bits carries exactly then.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t top) {
  return top < 0x7f800000u ? max(0, static_cast<int>((top + 0x1fffffu) >> 23) - 8) : 255;
}

// The largest magnitude's bits, a NaN's where there is one: one instruction a
// feature (its result's sign, the product of the signs, is dropped).
template <int kN>
__device__ __forceinline__ uint32_t largest_bits(const float (&x)[kN]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kN; ++i)
    asm("max.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(top) : "f"(x[i]));
  return __float_as_uint(top) & 0x7fffffffu;
}

// Two products, each rounded to fp32; where they are summands, the compiler makes
// an fma of product and sum all the same (rounded_products keeps them apart).
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%4, %5};\n\t"
      "mul.rn.f32x2 pd, pa, pb;\n\t"
      "mov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Two products, each rounded to fp32 whatever is done with them: minus_zero is
// -0, which adds nothing to any product, but known at run time alone.
__device__ __forceinline__ float2 rounded_products(float2 a, float2 b, float minus_zero) {
  return ffma2(a, b, make_float2(minus_zero, minus_zero));
}

// Two sums, each rounded to fp32.
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%4, %5};\n\t"
      "add.rn.f32x2 pd, pa, pb;\n\t"
      "mov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// kN features (a multiple of 4) over 2^(e - 127) as e4m3 bytes; zeros for 255.
template <int kN>
__device__ __forceinline__ void quantize(const float (&x)[kN], uint32_t e, uint32_t (&out)[kN / 4]) {
  // 2^(127 - e) by its exponent bits: e <= 247, so 254 - e >= 7
  const float inv = __uint_as_float(e == 255 ? 0u : (254 - e) << 23);
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    const float2 a = fmul2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(inv, inv));
    const float2 b = fmul2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(inv, inv));
    out[i] = e == 255 ? 0u : __byte_perm(e4m3x2(a.x, a.y), e4m3x2(b.x, b.y), 0x5410);
  }
}

// ---- append --------------------------------------------------------------------

struct AppendParams {
  PagedGeom g;
  int T, H, rows;            // tokens, query heads, head rows a token (q, k, v)
  int units;                 // kAppendRows-row groups a token
  int half;                  // rope_dim / 2
  bool vec;                  // cos and sin rows can be read 16 bytes at a time
  float minus_zero;          // -0 (rounded_products)
  int64_t q_stride, k_stride, v_stride;
  const uint16_t *q, *k, *v;
  const float *cos, *sin;
  const int *positions, *seq_ids;
  void *q_out, *k_cache, *v_cache;
  uint8_t *q_scale, *k_scale, *v_scale;
};

constexpr int kAppendRows = 4;           // head rows a group of lanes holds at once
constexpr int kAppendThreads = 128;

// Lanes of a head row: 16 of 8 features (a row's lines are read and written by
// consecutive lanes) where rows stay bf16; eight of 16 where some become
// fp8, whose per-row work (the scale, the address) then costs half.
template <bool kFp8>
constexpr int kAppendLanes = kFp8 ? 8 : 16;

// A group of lanes takes kAppendRows head rows of one token, whose cosines and
// sines it reads once; four rows' loads are in flight a lane. Products and sums
// of the rotation are rounded one by one (no fma), so that the result is the
// formula's in fp32. Measured on a B200: 16 tokens (64 query heads, 8 key heads)
// 2.5 us in a graph, a launch; 8,192 tokens bf16 65 us, 5.2 TB/s (copying reaches
// 6.6); 12,345 tokens' 64 query heads and one key head to fp8 74 us, 4.2 TB/s, bound
// by instructions (with an fma for a product and the sum 72 us, bf16 64).
template <bool kQFp8, bool kKvFp8, bool kHalves>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
  constexpr int kLanes = kAppendLanes<kQFp8 || kKvFp8>;
  constexpr int kF = kRowD / kLanes, kP = kF / 8;    // a lane's features, its 8-feature pieces
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int l = threadIdx.x & (kLanes - 1);
  const uint32_t unit = (blockIdx.x * kAppendThreads + threadIdx.x) / kLanes;
  int t = static_cast<int>(unit / static_cast<uint32_t>(p.units));
  const int r0 = static_cast<int>(unit - static_cast<uint32_t>(t) * p.units) * kAppendRows;
  const bool in = t < p.T;
  if (!in) t = 0;
  const int pos = __ldg(p.positions + t);
  const bool live = in && pos >= 0;
  const int kv0 = p.H, v0 = p.H + p.g.H_kv;          // first key row, first value row

  uint4 raw[kAppendRows][kP];
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int r = r0 + i;
#pragma unroll
    for (int u = 0; u < kP; ++u) raw[i][u] = make_uint4(0u, 0u, 0u, 0u);
    if (in && r < p.rows) {                          // (a padded token's too: no wait for its position)
      const uint16_t *src = r < kv0  ? p.q + t * p.q_stride + r * kRowD
                            : r < v0 ? p.k + t * p.k_stride + (r - kv0) * kRowD
                                     : p.v + t * p.v_stride + (r - v0) * kRowD;
#pragma unroll
      for (int u = 0; u < kP; ++u) raw[i][u] = reinterpret_cast<const uint4 *>(src)[kP * l + u];
    }
  }
  // the token's slot
  int64_t slot = -1;
  if (live && r0 + kAppendRows > kv0) {
    const int seq = p.seq_ids ? __ldg(p.seq_ids + t) : t;
    if (seq >= 0 && seq < p.g.num_seqs && pos < p.g.capacity()) slot = paged_slot(p.g, seq, pos);
  }
  // cosines and sines of this lane's pieces: eight (halves) or four (pairs) each
  constexpr int kC = kHalves ? 8 : 4;
  float c[kP][kC], s[kP][kC];
#pragma unroll
  for (int u = 0; u < kP; ++u) {
    const int f = 8 * (kP * l + u);                   // the piece's first feature
    const int c0 = kHalves ? (f < p.half ? f : f - p.half) : f / 2;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      c[u][i] = 1.f;
      s[u][i] = 0.f;
    }
    if (f < 2 * p.half && in && r0 < v0) {
      const float *cr = p.cos + static_cast<int64_t>(t) * p.half + c0;
      const float *sr = p.sin + static_cast<int64_t>(t) * p.half + c0;
      if (p.vec) {
#pragma unroll
        for (int i = 0; i < kC; i += 4) {
          *reinterpret_cast<float4 *>(&c[u][i]) = *reinterpret_cast<const float4 *>(cr + i);
          *reinterpret_cast<float4 *>(&s[u][i]) = *reinterpret_cast<const float4 *>(sr + i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kC; ++i)
          if (c0 + i < p.half) {
            c[u][i] = cr[i];
            s[u][i] = sr[i];
          }
      }
      if (kHalves && f < p.half) {
#pragma unroll
        for (int i = 0; i < kC; ++i) s[u][i] = -s[u][i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int r = r0 + i;
    float x[kF];
#pragma unroll
    for (int u = 0; u < kP; ++u) unpack8(raw[i][u], *reinterpret_cast<float (*)[8]>(&x[8 * u]));
    if constexpr (kHalves) {
      // features j and j + half sit half / 8 pieces apart: in the lane that
      // holds that piece, as its same or (two pieces a lane, half / 8 odd) its
      // other one
      const int apart = p.half / 8;
#pragma unroll
      for (int u = 0; u < kP; ++u) {
        const int piece = kP * l + u;
        const bool low = piece < apart, turn = piece < 2 * apart;
        const int from = (turn ? (low ? piece + apart : piece - apart) : piece) / kP;
        const uint4 give = kP == 2 && (apart & 1) ? raw[i][kP - 1 - u] : raw[i][u];
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, give.x, from, kLanes);
        o.y = __shfl_sync(0xffffffffu, give.y, from, kLanes);
        o.z = __shfl_sync(0xffffffffu, give.z, from, kLanes);
        o.w = __shfl_sync(0xffffffffu, give.w, from, kLanes);
        if (turn && r < v0) {
          // (the low half's sines were negated: a cos + b (-sin) rounds as a cos - b sin)
          float y[8];
          unpack8(o, y);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float &a = x[8 * u + j], &b = x[8 * u + j + 1];
            const float2 z = fadd2(
                rounded_products(make_float2(a, b), make_float2(c[u][j], c[u][j + 1]), p.minus_zero),
                rounded_products(make_float2(y[j], y[j + 1]), make_float2(s[u][j], s[u][j + 1]), p.minus_zero));
            a = z.x;
            b = z.y;
          }
        }
      }
    } else if (kF * l < 2 * p.half && r < v0) {
#pragma unroll
      for (int j = 0; j < kF / 2; ++j)
        if (kF / 2 * l + j < p.half) {
          // (a cos, a sin) + (-b sin, b cos)
          const float a = x[2 * j], b = x[2 * j + 1], cj = c[j >> 2][j & 3], sj = s[j >> 2][j & 3];
          const float2 y = fadd2(rounded_products(make_float2(a, a), make_float2(cj, sj), p.minus_zero),
                                 rounded_products(make_float2(b, b), make_float2(-sj, cj), p.minus_zero));
          x[2 * j] = y.x;
          x[2 * j + 1] = y.y;
        }
    }
    // where the row goes (the fp8 rows' shuffles below are the whole warp's)
    const bool is_q = r < kv0, is_k = !is_q && r < v0;
    const bool write = live && r < p.rows && (is_q || slot >= 0);
    const int64_t at = is_q ? (static_cast<int64_t>(t) * p.H + r) * kRowD
                            : slot + (is_k ? r - kv0 : r - v0) * p.g.head_stride;
    void *const data = is_q ? p.q_out : is_k ? p.k_cache : p.v_cache;
    if constexpr (kQFp8 || kKvFp8) {
      uint32_t top = largest_bits(x);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const uint32_t e = e8m0_of(top);
      uint32_t word = e << (8 * (l >> 1));           // the row's four scales
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      if (write && (is_q ? kQFp8 : kKvFp8)) {
        uint32_t d[4];
        quantize(x, e, d);
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(data) + at + 16 * l) =
            make_uint4(d[0], d[1], d[2], d[3]);
        uint8_t *const scale = is_q ? p.q_scale : is_k ? p.k_scale : p.v_scale;
        if (l == 0) *reinterpret_cast<uint32_t *>(scale + at / 32) = word;
      }
    }
    if (!(kQFp8 && kKvFp8) && write && !(is_q ? kQFp8 : kKvFp8)) {
      uint4 *const dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(data) + at) + kP * l;
#pragma unroll
      for (int u = 0; u < kP; ++u) dst[u] = pack8(*reinterpret_cast<const float (*)[8]>(&x[8 * u]));
    }
  }
}

// ---- block pooling -----------------------------------------------------------------

struct PoolParams {
  PagedGeom g;
  int block_size;
  int block_shift;           // log2 of it, where it is a power of two
  int share;                 // half warps that sum one pooled row (1 .. kPoolGroups, a power of two)
  int64_t S_pool, seq_stride, head_stride;
  const void *k;
  const uint8_t *k_scale;
  const int *start, *positions;
  void *pooled;
  uint8_t *pooled_scale;
  int *last_block;
};

constexpr int kPoolThreads = 256;
constexpr int kPoolLanes = 16;           // lanes a key row, 8 features each
constexpr int kPoolGroups = kPoolThreads / kPoolLanes;
constexpr int kPoolRun = 16;             // key rows a half warp has in flight
constexpr int kPoolSeqs = 1024;          // sequences the CTAs share out at once
template <bool kFp8>
constexpr int kPoolCtasPerSm = kFp8 ? 3 : 2;   // a run is 64 or 32 registers

// One pooled row, 8 features a lane; called by whole warps.
template <bool kFp8>
__device__ __forceinline__ void pool_store(const float (&x)[8], const PoolParams &p, int seq, int h,
                                           int b, int l, bool write) {
  const int64_t at = seq * p.seq_stride + h * p.head_stride + static_cast<int64_t>(b) * kRowD;
  if constexpr (kFp8) {
    uint32_t top = largest_bits(x);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t e = e8m0_of(top);
    uint32_t word = e << (8 * (l >> 2));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (write) {
      uint32_t d[2];
      quantize(x, e, d);
      reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.pooled) + at)[l] = make_uint2(d[0], d[1]);
      if (l == 0) *reinterpret_cast<uint32_t *>(p.pooled_scale + at / 32) = word;
    }
  } else {
    if (write) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.pooled) + at)[l] = pack8(x);
  }
}

// First fresh block of a sequence, and one past the last to write.
template <bool kPow2>
__device__ __forceinline__ int2 pool_range(const PoolParams &p, int seq, int &done) {
  const int cap = static_cast<int>(p.g.capacity());
  const int pos = __ldg(p.positions + seq);
  const int n = max(0, pos < cap ? pos + 1 : cap);          // slots held
  done = kPow2 ? n >> p.block_shift : n / p.block_size;
  const int start = p.start ? max(0, __ldg(p.start + seq)) : 0;
  const int first = kPow2 ? start >> p.block_shift : start / p.block_size;
  return make_int2(first, static_cast<int>(min(static_cast<int64_t>(done), p.S_pool)));
}

// A lane's 8 features of a key row, as loaded.
template <bool kFp8>
struct PoolRaw {
  uint4 w;
};
template <>
struct PoolRaw<true> {
  uint2 w;
};

template <bool kFp8>
__device__ __forceinline__ PoolRaw<kFp8> pool_load(const PoolParams &p, int64_t at, int l) {
  PoolRaw<kFp8> r;
  if constexpr (kFp8)
    r.w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.k) + at) + l);
  else
    r.w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) + at) + l);
  return r;
}

// acc += the row's features times `part`, a power of two that is at most the
// share of a row in its block, so that a sum passes fp32's range only where the mean
// does (fp8: under the scale byte number blk of e, as an fp32 exponent: 0 makes 0,
// and 255 an infinity, which makes NaN of the zeros beside it)
template <bool kFp8>
__device__ __forceinline__ void pool_add(float2 (&acc)[4], const PoolRaw<kFp8> &r, uint32_t e, int blk,
                                         float part) {
  if constexpr (kFp8) {
    const float f = __uint_as_float(__byte_perm(e, 0, blk << 12 | 0x444) >> 1) * part;
    const uint32_t q[4] = {r.w.x & 0xffffu, r.w.x >> 16, r.w.y & 0xffffu, r.w.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = ffma2(e4m3x2_f32(q[i]), make_float2(f, f), acc[i]);
  } else {
    float v[8];
    unpack8(r.w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = ffma2(make_float2(v[2 * i], v[2 * i + 1]), make_float2(part, part), acc[i]);
  }
}

// All sequences' fresh blocks (`together` blocks of a head: an item) are
// counted by every CTA, which then takes an equal share of them, so that
// sequences of any lengths fill the GPU evenly. kR > 0: block sizes that are
// powers of two, kR = min(block_size, 16). A half warp reads the 16 rows of a
// run (one page's, 16 slots from a multiple of 16 on) at once, looking the next
// item's run up meanwhile: 16 / kR blocks, or 1/16 of a larger block's rows and
// on, which `share` half warps sum and the first of them joins (in order, so
// that the result does not depend on timing). kR = 0: any block size, each row
// looked up by itself, four in flight. Measured on a B200: a step of 64 sequences
// 5.8 us (the chain start, positions, table, row), 3.9 in a graph; 240,000 bf16 keys
// by fours 12.2 us on resident rows and 17 on rows not in L2, 4.7 TB/s; 1.1 million
// fp8 rows by 64s 38 us, 3.8 TB/s, bound by instructions (four conversions to f16x2,
// eight to fp32, four packed fmas and a scale's product a lane and row).
template <bool kFp8, int kR>
__global__ void __launch_bounds__(kPoolThreads, kPoolCtasPerSm<kFp8>)
    block_pool_kernel(const PoolParams p) {
  constexpr int kTogether = kR > 0 ? kPoolRun / (kR > 0 ? kR : 1) : 1;   // blocks of an item
  __shared__ float4 part[2][kPoolGroups][2][kPoolLanes];    // (turns take one after the other)
  __shared__ uint32_t ends[kPoolSeqs];                      // items up to and with a sequence's
  __shared__ uint32_t warp_sum[kPoolThreads / 32];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int l = threadIdx.x & (kPoolLanes - 1), grp = threadIdx.x / kPoolLanes;
  const int per_cta = kPoolGroups / p.share;
  const int mine = grp / p.share, part_of = grp - mine * p.share;
  const bool warp_joins = (grp & ~1 & (p.share - 1)) == 0;  // a first half warp is in this warp
  // a power of two's reciprocal is the mean's whole factor; else the power of two
  // below it, and the sum over the rest of the size (above 1/2) is the same quotient
  const float size = static_cast<float>(p.block_size);
  const float part_of_sum = kR > 0 && kR < kPoolRun ? 1.f / (kR > 0 ? kR : 1)
                            : kR > 0                ? 1.f / size
                                                    : 1.f / static_cast<float>(2 << (31 - __clz(p.block_size)));
  const float rest = size * part_of_sum;
  int turn = 0;
  for (int seq0 = 0; seq0 < p.g.num_seqs; seq0 += kPoolSeqs) {
    const int seqs = min(kPoolSeqs, p.g.num_seqs - seq0);
    // ---- items of each sequence, summed up: four sequences a thread ----
    constexpr int kEach = kPoolSeqs / kPoolThreads;
    uint32_t count[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int s = threadIdx.x * kEach + i;
      int done = 0;
      count[i] = 0;
      if (s < seqs) {
        const int2 r = pool_range<(kR > 0)>(p, seq0 + s, done);
        // items lie at multiples of kTogether blocks
        if (r.y > r.x)
          count[i] = static_cast<uint32_t>((r.y + kTogether - 1) / kTogether - r.x / kTogether) * p.g.H_kv;
        if (p.last_block && blockIdx.x == 0)
          for (int h = 0; h < p.g.H_kv; ++h)
            p.last_block[static_cast<int64_t>(seq0 + s) * p.g.H_kv + h] = done - 1;
      }
      sum += count[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if ((threadIdx.x & 31) >= off) incl += o;
    }
    __syncthreads();                                        // the last turn's readers are done
    if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = incl;
    __syncthreads();
    uint32_t items = 0, at0 = incl - sum;
#pragma unroll
    for (int w = 0; w < kPoolThreads / 32; ++w) {
      if (w < threadIdx.x >> 5) at0 += warp_sum[w];
      items += warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) ends[threadIdx.x * kEach + i] = at0 += count[i];
    __syncthreads();
    // ---- this CTA's share, in turns of per_cta items ----
    const uint64_t turns_all = (items + per_cta - 1) / per_cta;
    const uint32_t begin = static_cast<uint32_t>(turns_all * blockIdx.x / gridDim.x) * per_cta;
    const uint32_t end =
        min(items, static_cast<uint32_t>(turns_all * (blockIdx.x + 1) / gridDim.x) * per_cta);
    int s = 0;                                              // the sequence of this half warp's item
    for (int hi = seqs - 1; s < hi;) {
      const int mid = (s + hi) / 2;
      if (begin + mine < ends[mid]) hi = mid;
      else s = mid + 1;
    }
    // Where an item is: its sequence and head, its first block and those to
    // write ([lo, hi)), and element offset and page of this half warp's first run.
    struct Item {
      int seq, h, b0, lo, hi;
      int64_t at;
    };
    int known = -1;                                         // the sequence of `range`
    int2 range = make_int2(0, 0);
    uint32_t first = 0;                                     // its first item
    auto locate = [&](uint32_t it) -> Item {
      Item x{0, 0, 0, 0, 0, -1};
      if (it >= end) return x;
      while (it >= ends[s]) ++s;
      if (s != known) {
        int done;
        range = pool_range<(kR > 0)>(p, seq0 + s, done);
        first = s > 0 ? ends[s - 1] : 0;
        known = s;
      }
      x.seq = seq0 + s;
      const uint32_t set = (it - first) / static_cast<uint32_t>(p.g.H_kv);
      x.h = static_cast<int>(it - first - set * p.g.H_kv);
      x.b0 = (range.x / kTogether + static_cast<int>(set)) * kTogether;
      x.lo = max(x.b0, range.x);
      x.hi = min(x.b0 + kTogether, range.y);
      if constexpr (kR > 0) x.at = paged_slot(p.g, x.seq, x.b0 * p.block_size + part_of * kPoolRun);
      return x;
    };
    Item next = locate(begin + mine);
    for (uint32_t it0 = begin; it0 < end; it0 += per_cta) {
      const Item cur = next;
      float2 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
      if constexpr (kR > 0) {
        const bool in = cur.hi > cur.lo;
        for (int j0 = part_of * kPoolRun;;) {
          const int64_t at = j0 == part_of * kPoolRun
                                 ? cur.at
                                 : paged_slot(p.g, cur.seq, cur.b0 * p.block_size + j0);
          const int64_t base = at + cur.h * p.g.head_stride;
          PoolRaw<kFp8> w[kPoolRun];
          uint32_t sc = 0x7f7f7f7fu;                        // scales of the run's row l
#pragma unroll
          for (int u = 0; u < kPoolRun; ++u) {
            w[u].w = {};
            if (at >= 0) w[u] = pool_load<kFp8>(p, base + u * p.g.slot_stride, l);
          }
          if (kFp8 && at >= 0)
            sc = __ldg(reinterpret_cast<const uint32_t *>(p.k_scale + (base + l * p.g.slot_stride) / 32));
          if (j0 == part_of * kPoolRun) next = locate(it0 + per_cta + mine);
          j0 += kPoolRun * p.share;
          const bool on = kR == 16 && j0 < p.block_size;    // the same for all lanes
#pragma unroll
          for (int u = 0; u < kPoolRun; ++u) {
            uint32_t e = 0;
            if constexpr (kFp8) e = __shfl_sync(0xffffffffu, sc, u, kPoolLanes);
            pool_add<kFp8>(acc, w[u], e, l >> 2, part_of_sum);
            if (kR < 16 && u % (kR > 0 ? kR : 1) == kR - 1) {
              // a block ends
              const int b = cur.b0 + u / (kR > 0 ? kR : 1);
              float x[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[2 * i] = acc[i].x;
                x[2 * i + 1] = acc[i].y;
                acc[i] = make_float2(0.f, 0.f);
              }
              pool_store<kFp8>(x, p, cur.seq, cur.h, b, l, in && b >= cur.lo && b < cur.hi);
            }
          }
          if (!on) break;
        }
      } else {
        // rows part_of, part_of + share, ..: four in flight
        const bool in = cur.hi > cur.lo;
        for (int j0 = part_of; j0 < p.block_size; j0 += 4 * p.share) {
          PoolRaw<kFp8> w[4];
          uint32_t e[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * p.share;
            int64_t at = -1;
            if (in && j < p.block_size) at = paged_slot(p.g, cur.seq, cur.b0 * p.block_size + j);
            w[u].w = {};
            e[u] = 127;
            if (at >= 0) {
              at += cur.h * p.g.head_stride;
              w[u] = pool_load<kFp8>(p, at, l);
              if (kFp8) e[u] = __ldg(p.k_scale + at / 32 + (l >> 2));
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) pool_add<kFp8>(acc, w[u], e[u], 0, part_of_sum);
        }
        next = locate(it0 + per_cta + mine);
      }
      if (kR == 16 || kR == 0) {
        if (p.share > 1) {
          float4 (&at)[kPoolGroups][2][kPoolLanes] = part[turn & 1];
          ++turn;
          at[grp][0][l] = make_float4(acc[0].x, acc[0].y, acc[1].x, acc[1].y);
          at[grp][1][l] = make_float4(acc[2].x, acc[2].y, acc[3].x, acc[3].y);
          __syncthreads();
          if (!warp_joins) continue;
          if (part_of == 0)
            for (int u = 1; u < p.share; ++u) {
              const float4 a = at[grp + u][0][l], b = at[grp + u][1][l];
              acc[0] = fadd2(acc[0], make_float2(a.x, a.y));
              acc[1] = fadd2(acc[1], make_float2(a.z, a.w));
              acc[2] = fadd2(acc[2], make_float2(b.x, b.y));
              acc[3] = fadd2(acc[3], make_float2(b.z, b.w));
            }
        }
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = kR > 0 ? acc[i].x : __fdiv_rn(acc[i].x, rest);
          x[2 * i + 1] = kR > 0 ? acc[i].y : __fdiv_rn(acc[i].y, rest);
        }
        pool_store<kFp8>(x, p, cur.seq, cur.h, cur.b0, l, cur.hi > cur.lo && part_of == 0);
      }
    }
  }
}

}  // namespace dsa
