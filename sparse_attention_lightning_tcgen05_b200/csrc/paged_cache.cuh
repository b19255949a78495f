// paged_cache.cuh -- the paged key-value cache's writers for sm_100a: a step's
// keys and values appended to the pages a block table names (rotated, bf16 or
// fp8), and the mean key of every completed block.
//
// Both move each byte once and compute next to nothing, so memory bounds the
// long calls and the launch the short ones. A head row (128 features) is one
// half warp's work: a lane holds 8 features, one 16-byte load, so that a
// row is whole 128-byte lines; the rotation's partner features sit in the
// same lane (interleaved pairs) or a fixed number of lanes away (halves), and
// the 32 features of an e8m0 scale in four neighbouring lanes.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace dsa {

constexpr int kRowD = 128;               // features of a head row
constexpr int kRowLanes = 16;            // lanes a row

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

// The value 2^(b - 127) of an e8m0 byte (255: NaN; 0: 2^-127, a denormal).
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fffffffu : b << 23);
}

// A half warp's row in the block-32 fp8 format: 8 e4m3 bytes a lane and, in
// every lane, the row's four scale bytes as one word. Called by whole warps.
// 448 = 1.75 * 2^8, so the least e with amax <= 448 * 2^e is amax's exponent
// less 8, plus one where its fraction is above .75: one integer addition to
// amax's bits carries exactly then.
__device__ __forceinline__ uint2 quantize_row(const float (&x)[8], uint32_t &scales) {
  uint32_t top = 0;                       // magnitudes as integers: NaN > inf > numbers
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool finite = top < 0x7f800000u;
  const int e = max(0, static_cast<int>((top + 0x1fffffu) >> 23) - 8);   // e + 127
  uint2 data = make_uint2(0u, 0u);
  if (finite) {
    // 2^-e by its exponent bits: e + 127 <= 247, so 254 - (e + 127) >= 7
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
    data.x = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
    data.y = e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16;
  }
  uint32_t word = static_cast<uint32_t>(finite ? e : 255) << (8 * ((threadIdx.x >> 2) & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
  scales = word;
  return data;
}

// ---- append --------------------------------------------------------------------

struct AppendParams {
  PagedGeom g;
  int T, H, rows;            // tokens, query heads, head rows a token (q, k, v)
  int units;                 // kAppendRows-row groups a token
  int half;                  // rope_dim / 2
  bool vec;                  // cos and sin rows can be read 16 bytes at a time
  int64_t q_stride, k_stride, v_stride;
  const uint16_t *q, *k, *v;
  const float *cos, *sin;
  const int *positions, *seq_ids;
  void *q_out, *k_cache, *v_cache;
  uint8_t *q_scale, *k_scale, *v_scale;
};

constexpr int kAppendRows = 4;           // head rows a half warp holds at once
constexpr int kAppendThreads = 256;

// Writes one row (8 features a lane) at element offset `at` of a buffer.
template <bool kFp8>
__device__ __forceinline__ void store_row(const float (&x)[8], void *data, uint8_t *scale,
                                          int64_t at, int l, bool write) {
  if constexpr (kFp8) {
    uint32_t scales;
    const uint2 d = quantize_row(x, scales);
    if (write) {
      *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(data) + at + 8 * l) = d;
      if (l == 0) *reinterpret_cast<uint32_t *>(scale + at / 32) = scales;
    }
  } else {
    if (write)
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(data) + at + 8 * l) = pack8(x);
  }
}

// A half warp takes kAppendRows head rows of one token, whose cosines and
// sines it reads once. Products and sums of the rotation are rounded one by
// one (no fma), so that the result is the formula's in fp32.
template <bool kQFp8, bool kKvFp8, bool kHalves>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int l = threadIdx.x & (kRowLanes - 1);
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) / kRowLanes;
  int t = static_cast<int>(unit / p.units);
  const int r0 = static_cast<int>(unit - static_cast<int64_t>(t) * p.units) * kAppendRows;
  const bool in = t < p.T;
  if (!in) t = 0;
  const int pos = __ldg(p.positions + t);
  const bool live = in && pos >= 0;

  uint4 raw[kAppendRows];
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int r = r0 + i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live && r < p.rows) {
      const uint16_t *src;
      if (r < p.H) src = p.q + t * p.q_stride + static_cast<int64_t>(r) * kRowD;
      else if (r < p.H + p.g.H_kv) src = p.k + t * p.k_stride + static_cast<int64_t>(r - p.H) * kRowD;
      else src = p.v + t * p.v_stride + static_cast<int64_t>(r - p.H - p.g.H_kv) * kRowD;
      raw[i] = *reinterpret_cast<const uint4 *>(src + 8 * l);
    }
  }
  // the token's slot
  int64_t slot = -1;
  if (live && r0 + kAppendRows > p.H) {
    const int seq = p.seq_ids ? __ldg(p.seq_ids + t) : t;
    if (seq >= 0 && seq < p.g.num_seqs && pos < p.g.capacity()) slot = paged_slot(p.g, seq, pos);
  }
  // this lane's cosines and sines
  constexpr int kC = kHalves ? 8 : 4;
  const int c0 = kHalves ? (8 * l < p.half ? 8 * l : 8 * l - p.half) : 4 * l;
  const bool turn = 8 * l < 2 * p.half;
  float c[kC], s[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (turn && live && r0 < p.H + p.g.H_kv) {
    const float *cr = p.cos + static_cast<int64_t>(t) * p.half + c0;
    const float *sr = p.sin + static_cast<int64_t>(t) * p.half + c0;
    if (p.vec) {
#pragma unroll
      for (int i = 0; i < kC; i += 4) {
        *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(cr + i);
        *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(sr + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (c0 + i < p.half) {
          c[i] = cr[i];
          s[i] = sr[i];
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int r = r0 + i;
    float x[8];
    unpack8(raw[i], x);
    if constexpr (kHalves) {
      // features j and j + half sit half / 8 lanes apart
      const int apart = p.half / 8;
      const bool low = 8 * l < p.half;
      const int from = turn ? (low ? l + apart : l - apart) : l;
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw[i].x, from, kRowLanes);
      o.y = __shfl_sync(0xffffffffu, raw[i].y, from, kRowLanes);
      o.z = __shfl_sync(0xffffffffu, raw[i].z, from, kRowLanes);
      o.w = __shfl_sync(0xffffffffu, raw[i].w, from, kRowLanes);
      if (turn && r < p.H + p.g.H_kv) {
        float y[8];
        unpack8(o, y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = low ? __fsub_rn(__fmul_rn(x[j], c[j]), __fmul_rn(y[j], s[j]))
                     : __fadd_rn(__fmul_rn(y[j], s[j]), __fmul_rn(x[j], c[j]));
      }
    } else if (turn && r < p.H + p.g.H_kv) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * l + j < p.half) {
          const float a = x[2 * j], b = x[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(a, s[j]), __fmul_rn(b, c[j]));
        }
    }
    // r is the same in both half warps only by chance: the branch below does
    // not hold the warp-wide shuffles of the fp8 rows
    const bool is_q = r < p.H, is_k = !is_q && r < p.H + p.g.H_kv;
    const int64_t q_at = (static_cast<int64_t>(t) * p.H + r) * kRowD;
    if constexpr (kQFp8 == kKvFp8) {
      const int64_t at = is_q ? q_at : slot + (is_k ? r - p.H : r - p.H - p.g.H_kv) * p.g.head_stride;
      store_row<kQFp8>(x, is_q ? p.q_out : is_k ? p.k_cache : p.v_cache,
                       is_q ? p.q_scale : is_k ? p.k_scale : p.v_scale, at, l,
                       live && r < p.rows && (is_q || slot >= 0));
    } else {
      store_row<kQFp8>(x, p.q_out, p.q_scale, q_at, l, live && is_q);
      store_row<kKvFp8>(x, is_k ? p.k_cache : p.v_cache, is_k ? p.k_scale : p.v_scale,
                        slot + (is_k ? r - p.H : r - p.H - p.g.H_kv) * p.g.head_stride, l,
                        live && !is_q && r < p.rows && slot >= 0);
    }
  }
}

// ---- block pooling -----------------------------------------------------------------

struct PoolParams {
  PagedGeom g;
  int block_size;
  int share;                 // half warps a pooled row (1 .. kPoolRows, a power of two)
  int ctas_per_seq;
  int64_t S_pool, seq_stride, head_stride;
  const void *k;
  const uint8_t *k_scale;
  const int *start, *positions;
  void *pooled;
  uint8_t *pooled_scale;
  int *last_block;
};

constexpr int kPoolThreads = 256;
constexpr int kPoolRows = kPoolThreads / kRowLanes;
constexpr int kPoolBatch = 4;            // key rows a half warp has in flight

// ctas_per_seq CTAs walk a sequence's fresh (block, head) rows; `share` half
// warps sum a row's slots and the first of them joins their sums (in order,
// so that the result does not depend on timing) and writes it.
template <bool kFp8>
__global__ void __launch_bounds__(kPoolThreads) block_pool_kernel(const PoolParams p) {
  __shared__ float part[kPoolRows][kRowD];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seq = blockIdx.x / p.ctas_per_seq;
  const int cta = blockIdx.x - seq * p.ctas_per_seq;
  const int l = threadIdx.x & (kRowLanes - 1), grp = threadIdx.x / kRowLanes;
  const int64_t cap = p.g.capacity();
  const int64_t n = min(static_cast<int64_t>(__ldg(p.positions + seq)) + 1, cap);   // slots held
  const int64_t done = n > 0 ? n / p.block_size : 0;
  if (p.last_block && cta == 0)
    for (int h = threadIdx.x; h < p.g.H_kv; h += kPoolThreads)
      p.last_block[static_cast<int64_t>(seq) * p.g.H_kv + h] = static_cast<int>(done) - 1;
  const int64_t first = p.start ? max(0, __ldg(p.start + seq)) / p.block_size : 0;
  const int64_t items = (min(done, p.S_pool) - first) * p.g.H_kv;
  const int per_cta = kPoolRows / p.share;
  const int row = grp / p.share, part_of = grp - row * p.share;
  for (int64_t it0 = static_cast<int64_t>(cta) * per_cta; it0 < items;
       it0 += static_cast<int64_t>(p.ctas_per_seq) * per_cta) {
    const int64_t it = it0 + row;
    const bool in = it < items;
    const int64_t b = first + (in ? it / p.g.H_kv : 0);
    const int h = in ? static_cast<int>(it % p.g.H_kv) : 0;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      const int s0 = static_cast<int>(b * p.block_size);
      for (int j0 = part_of; j0 < p.block_size; j0 += p.share * kPoolBatch) {
        int64_t at[kPoolBatch];
#pragma unroll
        for (int u = 0; u < kPoolBatch; ++u) {
          const int j = j0 + u * p.share;
          at[u] = j < p.block_size ? paged_slot(p.g, seq, s0 + j) : -1;
        }
        if constexpr (kFp8) {
          uint2 w[kPoolBatch];
          uint32_t sc[kPoolBatch];
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u) {
            w[u] = make_uint2(0u, 0u);
            sc[u] = 127;
            if (at[u] >= 0) {
              const int64_t o = at[u] + h * p.g.head_stride;
              w[u] = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.k) + o + 8 * l);
              sc[u] = p.k_scale[o / 32 + l / 4];
            }
          }
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u) {
            const float f = e8m0_f32(sc[u]);
            const uint32_t q[4] = {w[u].x & 0xffffu, w[u].x >> 16, w[u].y & 0xffffu, w[u].y >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = e4m3x2_f32(q[i]);
              acc[2 * i] += v.x * f;
              acc[2 * i + 1] += v.y * f;
            }
          }
        } else {
          uint4 w[kPoolBatch];
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u) {
            w[u] = make_uint4(0u, 0u, 0u, 0u);
            if (at[u] >= 0)
              w[u] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) + at[u] +
                                                      h * p.g.head_stride + 8 * l);
          }
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u) {
            float v[8];
            unpack8(w[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
          }
        }
      }
    }
    if (p.share > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) part[grp][8 * l + i] = acc[i];
      __syncthreads();
      if (part_of == 0)
        for (int u = 1; u < p.share; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += part[grp + u][8 * l + i];
      __syncthreads();
    }
    const float size = static_cast<float>(p.block_size);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __fdiv_rn(acc[i], size);
    store_row<kFp8>(acc, p.pooled, p.pooled_scale,
                    seq * p.seq_stride + h * p.head_stride + b * kRowD, l, in && part_of == 0);
  }
}

}  // namespace dsa
