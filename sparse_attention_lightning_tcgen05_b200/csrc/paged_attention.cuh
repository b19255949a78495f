// paged_attention.cuh -- attention of query tokens over a paged key-value
// cache (all slots of a sequence, or listed blocks of them) for sm_100a.
//
// For query token t, head h (key-value head g = h / G) and its kept slots s:
//   l_s = sm_scale * q[t,h,:] . k[s,g,:]
//   out = sum_s e^{l_s} v[s,g,:] / (sum_s e^{l_s} + e^{sink_h}),
//   lse = ln sum_s e^{l_s}.
// One pass over the slots with a running maximum m and sum, in log2 units:
// p_s = 2^(x_s - m), x = l * log2(e); the accumulated O and the sum are
// rescaled only when the maximum grows by more than 2^8 (p stays <= 256 and
// the final division removes the common factor, so the result is the same).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "paged_cache.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = kPaWarps * 32;
constexpr int kPaChunk = 16;                       // slots of a warp's step
constexpr int kPaTile = kPaWarps * kPaChunk;       // slots the CTA's warps take at once
constexpr int kPaRows = 16;                        // query heads of a work item
constexpr float kPaLazy = 8.f;                     // log2 units
constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PagedAttnParams {
  PagedGeom g;
  int T, H, G, head_tiles;     // head_tiles = ceil(G / kPaRows)
  int window;
  int block_shift, num_blocks, block_heads;
  int gran_shift;              // log2 of the slots one lookup covers (<= 4)
  int list_chunks;             // ceil(num_blocks * block_size / kPaChunk)
  float scale_log2;
  const uint16_t *q;
  const uint8_t *k, *v;        // pools, by byte
  const uint8_t *k_scale, *v_scale;
  const float *sinks;
  const int *positions, *seq_ids, *blocks;
  uint16_t *out;
  float *lse;
  float *part_o;               // [grid, 2, kPaRows, D] unnormalised
  float2 *part_ml;             // [grid, 2, kPaRows] (max in log2 units, sum)
  int4 *chain;                 // [grid] what the combine kernel reads
};

// What a query token attends to: its sequence, last slot and recent slots.
struct PaRow {
  int seq, last;               // last = -1: nothing
  int lo;                      // first recent slot kept (dense: first slot kept)
  int wbase;                   // lo rounded down to a chunk
  int chunks;                  // 16-slot steps in all
};

template <bool kList>
__device__ __forceinline__ PaRow pa_row(const PagedAttnParams &p, int t) {
  PaRow r;
  r.seq = p.seq_ids ? __ldg(p.seq_ids + t) : t;
  const int64_t cap = p.g.capacity();
  int64_t pos = __ldg(p.positions + t);
  if (r.seq < 0 || r.seq >= p.g.num_seqs || pos < 0) {
    r.seq = 0;
    r.last = -1;
    r.lo = r.wbase = r.chunks = 0;
    return r;
  }
  // window counts back from the token, which may stand past the table
  const int64_t lo = (kList || p.window > 0) ? max(int64_t{0}, pos + 1 - p.window) : 0;
  r.last = static_cast<int>(min(pos, cap - 1));
  r.lo = static_cast<int>(min(lo, static_cast<int64_t>(r.last) + 1));
  r.wbase = r.lo & ~(kPaChunk - 1);
  r.chunks = (r.last + 1 - r.wbase + kPaChunk - 1) / kPaChunk;
  if (r.lo > r.last) r.chunks = 0;
  if (kList) r.chunks += p.list_chunks;
  return r;
}

__device__ __forceinline__ int pa_tiles(int chunks) {
  return max(1, (chunks + kPaWarps - 1) / kPaWarps);
}

__device__ __forceinline__ void cp_async4_zfill(void *smem_dst, const void *gmem_src,
                                                uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem_dst)),
               "l"(gmem_src), "r"(src_bytes)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) * b (16 x 8): bf16 or f16 operands.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The e4m3 bytes 0 and 2 (even) or 1 and 3 (odd) of w as two bf16 values. The
// byte's exponent and fraction moved to the top of bf16's fields read as the
// value times 2^-120 (exponent biases 7 and 127; an e4m3 subnormal becomes a
// bf16 subnormal), which one exact multiplication undoes.
__device__ __forceinline__ uint32_t bf16_of_even(uint32_t w) {
  return mul_bf16x2((w << 8 & 0x80008000u) | (w << 4 & 0x07f007f0u), 0x7b807b80u);
}
__device__ __forceinline__ uint32_t bf16_of_odd(uint32_t w) {
  return mul_bf16x2((w & 0x80008000u) | (w >> 4 & 0x07f007f0u), 0x7b807b80u);
}

// Shared memory of a warp: kStages steps of 16 key rows, 16 value rows and
// (fp8) their scale words, each row's 16-byte pieces permuted by its number's
// low three bits so that eight rows' pieces lie in different banks.
template <bool kFp8>
struct PaSmem {
  static constexpr int kStages = kFp8 ? 6 : 3;
  static constexpr int kRowBytes = kFp8 ? 128 : 256;
  static constexpr int kTileBytes = kPaChunk * kRowBytes;
  static constexpr int off_v = kTileBytes;
  static constexpr int off_scale = 2 * kTileBytes;                  // 16 words k, 16 words v
  static constexpr int kStageBytes = 2 * kTileBytes + (kFp8 ? 128 : 0);
  static constexpr int off_mask = kStages * kStageBytes;            // a word a stage
  static constexpr int kWarpBytes = off_mask + 32;
  static constexpr int kTotal = kPaWarps * kWarpBytes;
  // the warp's O [16, 128] and (m, l) [16] replace the stages at an item's end
  static_assert(kStages * kStageBytes >= kPaRows * kRowD * 4 + kPaRows * 8, "merge area");
};

// A CTA walks a contiguous range of 64-slot tiles, an equal share of all
// items' tiles (an item: a token, a key-value head and up to 16 of its query
// heads), so that rows of any lengths fill the GPU evenly. In a tile warp w
// takes slots 16w .. 16w + 15 with its own ring of copies (cp.async), running
// maximum, sum and O (16 heads x 128 in registers), and no barrier with the
// other warps until the item ends. Items that lie in one CTA are finished
// here; the others leave partial results for the combine kernel.
template <bool kFp8, bool kList>
__global__ void __launch_bounds__(kPaThreads) paged_attention_kernel(const PagedAttnParams p) {
  using Smem = PaSmem<kFp8>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ int64_t scan[kPaWarps];
  __shared__ int start_row;
  __shared__ int64_t start_tile;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *const ring = smem_raw + warp * Smem::kWarpBytes;
  uint32_t *const masks = reinterpret_cast<uint32_t *>(ring + Smem::off_mask);
  grid_dep_wait();
  grid_dep_launch_dependents();

  // ---- this CTA's range of tiles, and the row it starts in ----
  const int items_per_row = p.g.H_kv * p.head_tiles;
  const int per = (p.T + kPaThreads - 1) / kPaThreads;
  const int ra = min(p.T, tid * per), rb = min(p.T, ra + per);
  int64_t mine = 0;
  for (int t = ra; t < rb; ++t) mine += pa_tiles(pa_row<kList>(p, t).chunks);
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPaWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  total *= items_per_row;
  // no more CTAs than tiles, so that the working ones are the first ones and
  // an item's CTAs follow one another
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  const int64_t begin = blockIdx.x < ctas ? total * blockIdx.x / ctas : total;
  const int64_t end = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : total;
  const int64_t excl = (before + incl - mine) * items_per_row;
  if (begin < end && begin >= excl && begin < (before + incl) * items_per_row) {
    int64_t at = excl;
    for (int t = ra; t < rb; ++t) {
      const int64_t n = static_cast<int64_t>(pa_tiles(pa_row<kList>(p, t).chunks)) * items_per_row;
      if (begin < at + n) {
        start_row = t;
        start_tile = begin - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  if (begin >= end) {
    if (tid == 0) p.chain[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }

  int t = start_row;
  int64_t left = end - begin;
  PaRow row = pa_row<kList>(p, t);
  int tiles = pa_tiles(row.chunks);
  int item = static_cast<int>(start_tile / tiles);          // of the row
  int tile = static_cast<int>(start_tile % tiles);
  int4 chain = make_int4(-1, 0, 0, 0);                      // head: row, item; inside
  const int gran = 1 << p.gran_shift;
  const int per_chunk = kPaChunk >> p.gran_shift;           // lookups a step
  const int quad = lane & 3, r0 = lane >> 2;

  while (left > 0) {
    const int kvh = item / p.head_tiles, ht = item - kvh * p.head_tiles;
    const int heads = min(kPaRows, p.G - ht * kPaRows);
    const int h0 = kvh * p.G + ht * kPaRows;
    const int tile_end = static_cast<int>(min(static_cast<int64_t>(tiles), tile + left));
    const int64_t head_off = kvh * p.g.head_stride;
    const int64_t list_row =
        kList ? (static_cast<int64_t>(t) * p.block_heads + (p.block_heads > 1 ? kvh : 0)) * p.num_blocks
              : 0;

    // ---- the query heads as matrix fragments ----
    uint32_t qf[8][4];
    float xs[2] = {p.scale_log2, p.scale_log2};               // logit scale of rows r0, r0 + 8
    {
      const uint16_t *qr[2];
      bool ok[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ok[i] = r0 + 8 * i < heads;
        qr[i] = p.q + (static_cast<int64_t>(t) * p.H + h0 + (ok[i] ? r0 + 8 * i : 0)) * kRowD;
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (kFp8) {
            // features 16kk + 4 quad .. + 3: the order the fp8 keys' bytes come in
            const uint2 w = ok[i] ? __ldg(reinterpret_cast<const uint2 *>(qr[i] + 16 * kk + 4 * quad))
                                  : make_uint2(0u, 0u);
            qf[kk][i] = w.x;
            qf[kk][2 + i] = w.y;
          } else {
            qf[kk][i] = ok[i] ? __ldg(reinterpret_cast<const uint32_t *>(qr[i] + 16 * kk + 2 * quad)) : 0u;
            qf[kk][2 + i] = ok[i] ? __ldg(reinterpret_cast<const uint32_t *>(qr[i] + 16 * kk + 8 + 2 * quad)) : 0u;
          }
        }
      if constexpr (kFp8) {
        // e4m3 keys are exact in f16, and so are the query's bf16 values once
        // its largest is brought to 2^13 .. 2^14: f16's 11 bits cover bf16's 8
        // down to 2^-27 of the row's largest, and below that the rounding is
        // 2^-38 of it, far under fp32's own
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t top = 0;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = qf[kk][2 * j + i] & 0x7fff7fffu;
              top = max(top, max(w & 0xffffu, w >> 16));
            }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = static_cast<int>(top >> 7) - 127;      // its exponent
          // inf and NaN stay as they are; 2^shift must be a normal number
          const int shift = top >= 0x7f80u || top == 0 ? 0 : max(-126, min(126, 13 - e));
          const float up = __int_as_float((shift + 127) << 23);
          xs[i] = p.scale_log2 * __int_as_float((127 - shift) << 23);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = qf[kk][2 * j + i];
              qf[kk][2 * j + i] = pack_f16x2(__uint_as_float(w << 16) * up,
                                             __uint_as_float(w & 0xffff0000u) * up);
            }
        }
      }
    }

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    const float neg_inf = __int_as_float(0xff800000);
    float m[2] = {neg_inf, neg_inf}, sum[2] = {0.f, 0.f};

    // this warp's steps: chunks (tile + i) * 4 + warp
    const int first = tile * kPaWarps + warp;
    const int steps = max(0, (min(tile_end * kPaWarps, row.chunks) - first + kPaWarps - 1) / kPaWarps);

    // Lookups of 32 granules at a time: lane l holds granule l's pool row
    // (page << page_shift | slot) and the range of its slots that are kept.
    int look_row = 0, look_lo = 0, look_hi = 0;
    const int steps_per_look = 32 / per_chunk;
    auto look = [&](int step) {
      const int st = step + lane / per_chunk;
      const int ch = first + st * kPaWarps;
      const int within = (lane & (per_chunk - 1)) << p.gran_shift;
      int64_t slot = -1;
      look_lo = 0;
      look_hi = 0;
      if (st < steps) {
        if (kList && ch < p.list_chunks) {
          const int at = ch * kPaChunk + within;
          const int e = at >> p.block_shift;
          if (e < p.num_blocks) {
            const int b = __ldg(p.blocks + list_row + e);
            if (b >= 0) {
              slot = (static_cast<int64_t>(b) << p.block_shift) + (at & ((1 << p.block_shift) - 1));
              // slots before the recent ones, of the table
              look_hi = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.lo - slot)));
            }
          }
        } else {
          slot = row.wbase + (kList ? ch - p.list_chunks : ch) * kPaChunk + within;
          look_lo = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.lo - slot)));
          look_hi = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.last + 1 - slot)));
        }
      }
      look_row = 0;
      if (look_hi > look_lo) {
        const int s = static_cast<int>(slot);
        const int page = __ldg(p.g.table + static_cast<int64_t>(row.seq) * p.g.pages_per_seq +
                               (s >> p.g.page_shift));
        if (page < 0 || page >= p.g.num_pages) look_hi = look_lo;
        else look_row = page << p.g.page_shift | (s & ((1 << p.g.page_shift) - 1));
      }
    };
    auto issue = [&](int step) {
      if (step < steps) {
        if (step % steps_per_look == 0) look(step);
        const int g0 = (step % steps_per_look) * per_chunk;
        uint8_t *const stage = ring + (step % Smem::kStages) * Smem::kStageBytes;
        {
          // slot lane % 16 is kept?
          const int src = g0 + ((lane & 15) >> p.gran_shift), rr = lane & (gran - 1);
          const int lo = __shfl_sync(0xffffffffu, look_lo, src);
          const int hi = __shfl_sync(0xffffffffu, look_hi, src);
          const uint32_t mask = __ballot_sync(0xffffffffu, rr >= lo && rr < hi) & 0xffffu;
          if (lane == 0) masks[step % Smem::kStages] = mask;
          if constexpr (kFp8) {
            const int rb2 = __shfl_sync(0xffffffffu, look_row, src);
            const int64_t at = (rb2 >> p.g.page_shift) * p.g.page_stride +
                               ((rb2 & ((1 << p.g.page_shift) - 1)) + rr) * p.g.slot_stride + head_off;
            const bool keep = rr >= lo && rr < hi;
            cp_async4_zfill(stage + Smem::off_scale + 4 * lane,
                            (lane < 16 ? p.k_scale : p.v_scale) + (keep ? at / 32 : 0), keep ? 4u : 0u);
          }
        }
        constexpr int kPieces = Smem::kRowBytes / 16;           // lanes a row
        constexpr int kRowsAtOnce = 32 / kPieces;
        const int c = lane & (kPieces - 1);
#pragma unroll
        for (int i = 0; i < kPaChunk / kRowsAtOnce; ++i) {
          const int r = i * kRowsAtOnce + lane / kPieces;
          const int src = g0 + (r >> p.gran_shift), rr = r & (gran - 1);
          const int base = __shfl_sync(0xffffffffu, look_row, src);
          const int lo = __shfl_sync(0xffffffffu, look_lo, src);
          const int hi = __shfl_sync(0xffffffffu, look_hi, src);
          const bool keep = rr >= lo && rr < hi;
          int64_t at = (base >> p.g.page_shift) * p.g.page_stride +
                       ((base & ((1 << p.g.page_shift) - 1)) + rr) * p.g.slot_stride + head_off;
          if (!kFp8) at *= 2;
          at = keep ? at + 16 * c : 0;
          uint8_t *const dst = stage + r * Smem::kRowBytes + ((c ^ (r & 7)) << 4);
          cp_async16_zfill(dst, p.k + at, keep ? 16u : 0u);
          cp_async16_zfill(dst + Smem::off_v, p.v + at, keep ? 16u : 0u);
        }
      }
      cp_async_commit();
    };

#pragma unroll
    for (int i = 0; i < Smem::kStages - 1; ++i) issue(i);
    for (int step = 0; step < steps; ++step) {
      issue(step + Smem::kStages - 1);
      cp_async_wait<Smem::kStages - 1>();
      __syncwarp();
      const uint8_t *const stage = ring + (step % Smem::kStages) * Smem::kStageBytes;
      const uint32_t mask = masks[step % Smem::kStages];
      const uint32_t ks = smem_u32(stage), vs = ks + Smem::off_v;
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t b[4];
          const int r = (lane & 7) + 8 * (lane >> 4), c = 2 * kk + ((lane >> 3) & 1);
          ldsm4(b, ks + r * 256 + ((c ^ (r & 7)) << 4));
          mma_bf16(s[0], qf[kk], b[0], b[1]);
          mma_bf16(s[1], qf[kk], b[2], b[3]);
        }
      } else {
        const uint32_t *const sc = reinterpret_cast<const uint32_t *>(stage + Smem::off_scale);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 w = *reinterpret_cast<const uint2 *>(sc + 8 * j + 2 * quad);   // two slots' scales
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t b[4];
            const int r = (lane & 7) + 8 * j, c = 4 * half + (lane >> 3);
            ldsm4(b, ks + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
              float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t v = b[2 * blk + i];
                mma_f16(x, qf[4 * half + 2 * blk + i], f16x2_of_e4m3x2(v & 0xffffu), f16x2_of_e4m3x2(v >> 16));
              }
              const int sh = 8 * (2 * half + blk);
              const float f0 = __uint_as_float((w.x >> sh & 0xffu) << 23);
              const float f1 = __uint_as_float((w.y >> sh & 0xffu) << 23);
              s[j][0] = fmaf(x[0], f0, s[j][0]);
              s[j][1] = fmaf(x[1], f1, s[j][1]);
              s[j][2] = fmaf(x[2], f0, s[j][2]);
              s[j][3] = fmaf(x[3], f1, s[j][3]);
            }
          }
        }
      }
      // ---- softmax: rows r0 and r0 + 8, slots 8j + 2 quad + {0, 1} ----
      float mx[2] = {neg_inf, neg_inf};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[j][i] * xs[i >> 1];
          if (!((mask >> (8 * j + 2 * quad + (i & 1))) & 1u)) x = neg_inf;
          s[j][i] = x;
          mx[i >> 1] = fmaxf(mx[i >> 1], x);
        }
      bool grow = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        grow = grow || mx[i] > m[i] + kPaLazy;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], mx[i]);
          const float a = m[i] == neg_inf ? 0.f : ex2_approx(m[i] - mn);
          m[i] = mn;
          sum[i] *= a;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[n][2 * i] *= a;
            o[n][2 * i + 1] *= a;
          }
        }
      }
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) base[i] = m[i] == neg_inf ? 0.f : m[i];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[j][i] = ex2_approx(s[j][i] - base[i >> 1]);
          sum[i >> 1] += s[j][i];
        }
      // ---- O += P V ----
      if constexpr (!kFp8) {
        const uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
        for (int dd = 0; dd < 8; ++dd) {
          uint32_t b[4];
          const int r = (lane & 7) + 8 * ((lane >> 3) & 1), c = 2 * dd + (lane >> 4);
          ldsm4_t(b, vs + r * 256 + ((c ^ (r & 7)) << 4));
          mma_bf16(o[2 * dd], pf, b[0], b[1]);
          mma_bf16(o[2 * dd + 1], pf, b[2], b[3]);
        }
      } else {
        // the slots' scales go into P: one set of fragments per 32 features
        const uint32_t *const sc = reinterpret_cast<const uint32_t *>(stage + Smem::off_scale) + 16;
        const uint2 w0 = *reinterpret_cast<const uint2 *>(sc + 2 * quad);
        const uint2 w1 = *reinterpret_cast<const uint2 *>(sc + 8 + 2 * quad);
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          const float f0 = __uint_as_float((w0.x >> (8 * blk) & 0xffu) << 23);
          const float f1 = __uint_as_float((w0.y >> (8 * blk) & 0xffu) << 23);
          const float f2 = __uint_as_float((w1.x >> (8 * blk) & 0xffu) << 23);
          const float f3 = __uint_as_float((w1.y >> (8 * blk) & 0xffu) << 23);
          const uint32_t pf[4] = {pack_bf16x2(s[0][0] * f0, s[0][1] * f1),
                                  pack_bf16x2(s[0][2] * f0, s[0][3] * f1),
                                  pack_bf16x2(s[1][0] * f2, s[1][1] * f3),
                                  pack_bf16x2(s[1][2] * f2, s[1][3] * f3)};
          uint32_t b[4];                       // 16 features x slots 0-7, 8-15; the next 16
          const int r = (lane & 7) + 8 * ((lane >> 3) & 1), c = 2 * blk + (lane >> 4);
          ldsm4_t(b, vs + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // a transposed 16-bit unit is two features of a slot: even and
            // odd features make a tile each
            mma_bf16(o[4 * blk + 2 * i], pf, bf16_of_even(b[2 * i]), bf16_of_even(b[2 * i + 1]));
            mma_bf16(o[4 * blk + 2 * i + 1], pf, bf16_of_odd(b[2 * i]), bf16_of_odd(b[2 * i + 1]));
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the four warps' results ----
    float *const so = reinterpret_cast<float *>(ring);
    float2 *const sml = reinterpret_cast<float2 *>(ring + kPaRows * kRowD * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
      if (quad == 0) sml[r0 + 8 * i] = make_float2(m[i], sum[i]);
#pragma unroll
      for (int n = 0; n < 16; n += 2) {
        float *const dst = so + (r0 + 8 * i) * kRowD;
        if constexpr (!kFp8) {
          *reinterpret_cast<float2 *>(dst + 8 * n + 2 * quad) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
          *reinterpret_cast<float2 *>(dst + 8 * n + 8 + 2 * quad) =
              make_float2(o[n + 1][2 * i], o[n + 1][2 * i + 1]);
        } else {
          // tiles n, n + 1: the even and odd features of a 16-feature piece
          *reinterpret_cast<float4 *>(dst + 8 * n + 4 * quad) =
              make_float4(o[n][2 * i], o[n + 1][2 * i], o[n][2 * i + 1], o[n + 1][2 * i + 1]);
        }
      }
    }
    __syncthreads();
    const bool whole = tile == 0 && tile_end == tiles;
    {
      const int r = tid >> 3, c0 = tid & 7;                   // row, 4-feature pieces c0 + 8i
      if (r < heads) {
        float M = neg_inf, L = 0.f, a[kPaWarps];
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) {
          const float2 ml = *reinterpret_cast<const float2 *>(
              smem_raw + w * Smem::kWarpBytes + kPaRows * kRowD * 4 + 8 * r);
          a[w] = ml.x;
          M = fmaxf(M, ml.x);
        }
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) {
          const float2 ml = *reinterpret_cast<const float2 *>(
              smem_raw + w * Smem::kWarpBytes + kPaRows * kRowD * 4 + 8 * r);
          a[w] = a[w] == neg_inf ? 0.f : ex2_approx(a[w] - M);
          L += a[w] * ml.y;
        }
        const int64_t orow = static_cast<int64_t>(t) * p.H + h0 + r;
        float inv = 1.f;
        if (whole) {
          float den = L;
          if (p.sinks && M != neg_inf) den += ex2_approx(__ldg(p.sinks + h0 + r) * kPaLog2e - M);
          inv = M == neg_inf ? 0.f : 1.f / den;
          if (c0 == 0 && p.lse) p.lse[orow] = M == neg_inf ? neg_inf : (M + log2f(L)) * kPaLn2;
        }
        const int64_t prow = (static_cast<int64_t>(blockIdx.x) * 2 + (tile == 0 ? 1 : 0)) * kPaRows + r;
        if (!whole && c0 == 0) p.part_ml[prow] = make_float2(M, L);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 4 * (c0 + 8 * i);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kPaWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(smem_raw + w * Smem::kWarpBytes +
                                                               (r * kRowD + d) * 4);
            acc.x += a[w] * x.x;
            acc.y += a[w] * x.y;
            acc.z += a[w] * x.z;
            acc.w += a[w] * x.w;
          }
          if (whole) {
            *reinterpret_cast<uint2 *>(p.out + orow * kRowD + d) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          } else {
            *reinterpret_cast<float4 *>(p.part_o + prow * kRowD + d) = acc;
          }
        }
      }
    }
    __syncthreads();

    // ---- the next item ----
    left -= tile_end - tile;
    if (tile_end < tiles) {                                   // the range ends inside the item
      if (tile == 0) chain.x = t, chain.y = item;
      else chain.z = 1;
      break;
    }
    tile = 0;
    if (++item == items_per_row && left > 0) {
      item = 0;
      ++t;
      row = pa_row<kList>(p, t);
      tiles = pa_tiles(row.chunks);
    }
  }
  if (tid == 0) p.chain[blockIdx.x] = chain;
}

// Joins the items that several CTAs share: an item begins in CTA a (chain.x,
// chain.y: its row and item) and goes on through CTAs a + 1, .. up to the
// first that does not lie inside it (chain.z). Two heads a block; a thread
// joins one 4-feature piece per head over the partials in CTA order.
constexpr int kPaJoinThreads = 64;
__global__ void __launch_bounds__(kPaJoinThreads) paged_attention_join_kernel(const PagedAttnParams p,
                                                                             int grid) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int a = blockIdx.x / (kPaRows / 2);
  const int r = (blockIdx.x % (kPaRows / 2)) * 2 + (threadIdx.x >> 5);
  const int4 c = p.chain[a];
  if (c.x < 0) return;
  const int kvh = c.y / p.head_tiles, ht = c.y - kvh * p.head_tiles;
  if (r >= min(kPaRows, p.G - ht * kPaRows)) return;
  const int lane = threadIdx.x & 31;
  const float neg_inf = __int_as_float(0xff800000);
  int b = a + 1;                                              // the last CTA of the chain
  while (b < grid - 1 && p.chain[b].z) ++b;
  float M = neg_inf;
  for (int i = a + lane; i <= b; i += 32)
    M = fmaxf(M, p.part_ml[(static_cast<int64_t>(i) * 2 + (i == a)) * kPaRows + r].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
  for (int i0 = a; i0 <= b; i0 += 32) {
    float w = 0.f, l = 0.f;
    if (i0 + lane <= b) {
      const int i = i0 + lane;
      const float2 ml = p.part_ml[(static_cast<int64_t>(i) * 2 + (i == a)) * kPaRows + r];
      w = ml.x == neg_inf ? 0.f : ex2_approx(ml.x - M);
      l = ml.y;
    }
    L += w * l;
    const int n = min(32, b - i0 + 1);
    for (int j = 0; j < n; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int i = i0 + j;
      const float4 x = *reinterpret_cast<const float4 *>(
          p.part_o + ((static_cast<int64_t>(i) * 2 + (i == a)) * kPaRows + r) * kRowD + 4 * lane);
      acc.x += wj * x.x;
      acc.y += wj * x.y;
      acc.z += wj * x.z;
      acc.w += wj * x.w;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  const int h = kvh * p.G + ht * kPaRows + r;
  const int64_t orow = static_cast<int64_t>(c.x) * p.H + h;
  float den = L;
  if (p.sinks && M != neg_inf) den += ex2_approx(__ldg(p.sinks + h) * kPaLog2e - M);
  const float inv = M == neg_inf ? 0.f : 1.f / den;
  if (lane == 0 && p.lse) p.lse[orow] = M == neg_inf ? neg_inf : (M + log2f(L)) * kPaLn2;
  reinterpret_cast<uint2 *>(p.out + orow * kRowD)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace dsa
