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

constexpr int kPaWarps = 4;                        // consumer warps
constexpr int kPaThreads = (kPaWarps + 1) * 32;    // and the producer
constexpr int kPaStep = 32;                        // slots of a pipeline stage
constexpr int kPaRows = 16;                        // query heads of a work item
constexpr float kPaLazy = 8.f;                     // log2 units
constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PagedAttnParams {
  PagedGeom g;
  int T, H, G, head_tiles;     // head_tiles = ceil(G / kPaRows)
  int window;
  int block_shift, num_blocks, block_heads;
  int gran_shift;              // log2 of the slots one lookup and one box cover (<= 5)
  int list_steps;              // ceil(num_blocks * block_size / kPaStep)
  float scale_log2;
  const uint8_t *k_scale, *v_scale;
  const float *sinks;
  const int *positions, *seq_ids, *blocks;
  uint16_t *out;
  float *lse;
  float *part_o;               // [grid, 2, kPaRows, D] unnormalised
  float2 *part_ml;             // [grid, 2, kPaRows] (max in log2 units, sum)
  int4 *chain;                 // [grid] items that several CTAs share
  unsigned int *err, *err_info;
  uint64_t wait_limit_ns, drain_limit_ns;
};

// What a query token attends to: its sequence, last slot and recent slots.
struct PaRow {
  int seq, last;               // last = -1: nothing
  int lo;                      // first recent slot kept (dense: first slot kept)
  int wbase;                   // lo rounded down to a step
  int steps;                   // 32-slot steps, at least one
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
    r.lo = r.wbase = 0;
    r.steps = 1;
    return r;
  }
  // window counts back from the token, which may stand past the table
  const int64_t lo = (kList || p.window > 0) ? max(int64_t{0}, pos + 1 - p.window) : 0;
  r.last = static_cast<int>(min(pos, cap - 1));
  r.lo = static_cast<int>(min(lo, static_cast<int64_t>(r.last) + 1));
  r.wbase = r.lo & ~(kPaStep - 1);
  r.steps = r.lo <= r.last ? (r.last + kPaStep - r.wbase) / kPaStep : 0;
  if (kList) r.steps += p.list_steps;
  r.steps = max(1, r.steps);
  return r;
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

// A bounded wait whose fast path is one instruction (see mbar_wait).
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, const WaitCtl &ctl,
                                        uint32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, ctl, site);
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

// What the producer tells the consumers of an item.
struct PaItem {
  int row, item;               // token (-1: no more items), its (kv head, head tile)
  int steps;                   // of this CTA
  int slot;                    // -1: the whole item; else where the partial result goes (0, 1)
};

// Shared memory. A stage holds 32 slots: bf16 rows as two 128-byte halves
// ([32 x 64] each), fp8 rows whole, keys then values, in TMA's 128-byte swizzle
// (16-byte piece c of row r at c ^ (r & 7): the eight rows of a matrix
// fragment lie in different banks).
template <bool kFp8>
struct PaSmem {
  // a multiple of the consumer warps: a stage is always the same warp's, so
  // that no warp waits for a phase before the last one of its barrier is over
  static constexpr int kStages = kFp8 ? 8 : 4;
  static constexpr int kHalf = kPaStep * 128;                       // one [32 x 128 B] box
  static constexpr int kBoxes = kFp8 ? 1 : 2;                       // of a row
  static constexpr int off_v = kBoxes * kHalf;
  static constexpr int kStageBytes = 2 * kBoxes * kHalf;
  static constexpr int kQBytes = kPaRows * kRowD * 2;               // [2][16 x 64] bf16
  static constexpr int off_q = kStages * kStageBytes;               // two of them
  static constexpr int off_merge = off_q + 2 * kQBytes;
  static constexpr int kMergeBytes = 68 * 32 * 4;                   // O, m and sum of a warp
  static constexpr int off_scale = off_merge + (kPaWarps - 1) * kMergeBytes;
  static constexpr int off_mask = off_scale + (kFp8 ? kStages * 2 * kPaStep * 4 : 0);
  static constexpr int off_bar = off_mask + 16 * 4;
  static constexpr int off_misc = off_bar + 32 * 8;
  static constexpr int kTotal = off_misc + 128 + 1024;              // + alignment slack
  static_assert(2 * (kTotal + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(kStages % kPaWarps == 0, "a stage's warp");
};

// A CTA walks a contiguous range of 32-slot steps, an equal share of all
// items' steps (an item: a token, a key-value head and up to 16 of its query
// heads), so that rows of any lengths fill the GPU evenly. Warp 4 produces:
// it looks the steps' pages up, 32 of them at a time, and keeps a ring of
// stages full with TMA loads, running ahead over the items' ends. Consumer
// warp w takes every fourth step with a running maximum, sum and O
// (16 heads x 128 in registers) of its own; at the item's end three warps hand
// theirs to the fourth (a different one each time), which joins and writes.
// Items that lie in one CTA are finished here; of the others each CTA leaves a
// partial result for the join kernel.
template <bool kFp8, bool kList>
__global__ void __launch_bounds__(kPaThreads, 2)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                           const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const PagedAttnParams p) {
  using Smem = PaSmem<kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint32_t *const masks = reinterpret_cast<uint32_t *>(smem + Smem::off_mask);
  uint64_t *const full = reinterpret_cast<uint64_t *>(smem + Smem::off_bar);
  uint64_t *const empty = full + Smem::kStages;
  uint64_t *const q_full = empty + Smem::kStages;
  uint64_t *const q_empty = q_full + 2;
  uint64_t *const merge_full = q_empty + 2;
  uint64_t *const merge_empty = merge_full + 1;
  PaItem *const info = reinterpret_cast<PaItem *>(smem + Smem::off_misc);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(info + 2);
  int *const start_row = reinterpret_cast<int *>(info + 2) + 1;
  int64_t *const start_step = reinterpret_cast<int64_t *>(smem + Smem::off_misc + 48);
  int64_t *const scan = start_step + 1;                             // [kPaWarps + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Smem::kStages; ++i) {
      mbar_init(full + i, kFp8 ? 33 : 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, kPaWarps);
    }
    mbar_init(merge_full, kPaWarps - 1);
    mbar_init(merge_empty, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  grid_dep_wait();
  grid_dep_launch_dependents();

  // ---- this CTA's range of steps, and the row it starts in ----
  const int items_per_row = p.g.H_kv * p.head_tiles;
  const int per = (p.T + kPaThreads - 1) / kPaThreads;
  const int ra = min(p.T, tid * per), rb = min(p.T, ra + per);
  int64_t mine = 0;
  for (int t = ra; t < rb; ++t) mine += pa_row<kList>(p, t).steps;
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
  for (int w = 0; w <= kPaWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  total *= items_per_row;
  // no more CTAs than give each warp a step, and the working ones are the
  // first ones, so that an item's CTAs follow one another
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + kPaWarps - 1) / kPaWarps);
  const int64_t begin = blockIdx.x < ctas ? total * blockIdx.x / ctas : total;
  const int64_t end = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : total;
  const int64_t excl = (before + incl - mine) * items_per_row;
  if (begin < end && begin >= excl && begin < (before + incl) * items_per_row) {
    int64_t at = excl;
    for (int t = ra; t < rb; ++t) {
      const int64_t n = static_cast<int64_t>(pa_row<kList>(p, t).steps) * items_per_row;
      if (begin < at + n) {
        *start_row = t;
        *start_step = begin - at;
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
  const WaitCtl ctl{abort_flag, p.err, p.err_info, p.wait_limit_ns};

  if (warp == kPaWarps) {
    // ---------------- producer ----------------
    int t = *start_row;
    PaRow row = pa_row<kList>(p, t);
    int item = static_cast<int>(*start_step / row.steps);     // of the row
    int first = static_cast<int>(*start_step % row.steps);
    int64_t at = begin;
    int4 chain = make_int4(-1, 0, 0, 0);
    const int gran = 1 << p.gran_shift;
    const int per_step = kPaStep >> p.gran_shift;             // lookups and boxes a step
    const int steps_per_look = 32 / per_step;
    uint32_t g = 0, st = 0, ph = 0, n_items = 0;
    bool ok = true, published = false;
    while (ok) {
      const bool more = at < end;
      const int steps = more ? static_cast<int>(min(static_cast<int64_t>(row.steps - first), end - at)) : 0;
      const bool whole = more && first == 0 && steps == row.steps;
      const int kvh = item / p.head_tiles, ht = item - kvh * p.head_tiles;
      const uint32_t qb = n_items & 1u;
      if (!pa_wait(q_empty + qb, ((n_items >> 1) & 1u) ^ 1u, ctl, 60)) break;
      if (lane == 0) {
        info[qb] = PaItem{more ? t : -1, item, steps, whole ? -1 : first == 0 ? 1 : 0};
        if (more) {
          uint8_t *const dst = smem + Smem::off_q + qb * Smem::kQBytes;
          const int q_row = t * p.H + kvh * p.G + ht * kPaRows;
          mbar_arrive_expect_tx(q_full + qb, Smem::kQBytes);
          tma_load_2d(dst, &tmap_q, q_full + qb, 0, q_row);
          tma_load_2d(dst + Smem::kQBytes / 2, &tmap_q, q_full + qb, 64, q_row);
        } else {
          mbar_arrive(q_full + qb);
        }
      }
      __syncwarp();
      if (!more) {
        published = true;
        break;
      }
      ++n_items;
      if (!whole && first == 0) {
        // the CTA that holds the item's last step
        const int64_t last = at + row.steps - 1;
        chain = make_int4(t, item, static_cast<int>(((last + 1) * ctas - 1) / total), 0);
      }
      const int64_t list_row =
          kList ? (static_cast<int64_t>(t) * p.block_heads + (p.block_heads > 1 ? kvh : 0)) * p.num_blocks
                : 0;
      // Lane l's lookup: a granule's page and slot there, and which of its
      // slots are kept.
      int look_page = 0, look_slot = 0;
      uint32_t look_lo = 0, look_hi = 0;
      for (int step = 0; step < steps; ++step) {
        const int in_look = step & (steps_per_look - 1);
        if (in_look == 0) {
          const int s = step + lane / per_step;
          const int ch = first + s;
          const int within = (lane & (per_step - 1)) << p.gran_shift;
          int64_t slot = -1;
          int lo = 0, hi = 0;
          if (s < steps) {
            if (kList && ch < p.list_steps) {
              const int a = ch * kPaStep + within;
              const int e = a >> p.block_shift;
              if (e < p.num_blocks) {
                const int b = __ldg(p.blocks + list_row + e);
                if (b >= 0) {
                  // slots before the recent ones; row.lo lies in the table
                  slot = (static_cast<int64_t>(b) << p.block_shift) + (a & ((1 << p.block_shift) - 1));
                  hi = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.lo - slot)));
                }
              }
            } else {
              slot = row.wbase + static_cast<int64_t>(kList ? ch - p.list_steps : ch) * kPaStep + within;
              lo = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.lo - slot)));
              hi = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(gran), row.last + 1 - slot)));
            }
          }
          if (hi > lo) {
            const int sl = static_cast<int>(slot);
            look_page = __ldg(p.g.table + static_cast<int64_t>(row.seq) * p.g.pages_per_seq +
                              (sl >> p.g.page_shift));
            look_slot = sl & ((1 << p.g.page_shift) - 1);
            if (look_page < 0 || look_page >= p.g.num_pages) hi = lo;
          }
          look_lo = lo;
          look_hi = hi;
        }
        if (!pa_wait(empty + st, ph ^ 1u, ctl, 61)) {
          ok = false;
          break;
        }
        uint8_t *const stage = smem + st * Smem::kStageBytes;
        // slot `lane` of the step is kept?
        const int src = in_look * per_step + (lane >> p.gran_shift);
        const uint32_t rr = lane & (gran - 1);
        const uint32_t lo = __shfl_sync(0xffffffffu, look_lo, src);
        const uint32_t hi = __shfl_sync(0xffffffffu, look_hi, src);
        const bool keep = rr >= lo && rr < hi;
        const uint32_t mask = __ballot_sync(0xffffffffu, keep);
        const uint32_t live = __popc(__ballot_sync(0xffffffffu, hi > lo && rr == 0));
        if constexpr (kFp8) {
          const int pg = __shfl_sync(0xffffffffu, look_page, src);
          const int sl = __shfl_sync(0xffffffffu, look_slot, src);
          const int64_t o = keep ? (pg * p.g.page_stride + static_cast<int64_t>(sl + rr) * p.g.slot_stride +
                                    kvh * p.g.head_stride) / 32
                                 : 0;
          uint8_t *const sc = smem + Smem::off_scale + st * (2 * kPaStep * 4) + 4 * lane;
          cp_async4_zfill(sc, p.k_scale + o, keep ? 4u : 0u);
          cp_async4_zfill(sc + kPaStep * 4, p.v_scale + o, keep ? 4u : 0u);
          cp_async_mbar_arrive_noinc(full + st);
        }
        if (lane == 0) {
          masks[st] = mask;
          mbar_arrive_expect_tx(full + st, live * (gran * 128 * 2 * Smem::kBoxes));
        }
        __syncwarp();
        // boxes: granule, keys or values, half of the row
        const int boxes = per_step * 2 * Smem::kBoxes;
        for (int b0 = 0; b0 < boxes; b0 += 32) {
          const int b = b0 + lane;
          const int gr = b / (2 * Smem::kBoxes), part = b & (2 * Smem::kBoxes - 1);
          const int from = (in_look * per_step + gr) & 31;
          const int pg = __shfl_sync(0xffffffffu, look_page, from);
          const int sl = __shfl_sync(0xffffffffu, look_slot, from);
          const uint32_t l2 = __shfl_sync(0xffffffffu, look_lo, from);
          const uint32_t h2 = __shfl_sync(0xffffffffu, look_hi, from);
          if (b < boxes && h2 > l2)
            tma_load_4d(stage + part * Smem::kHalf + gr * gran * 128,
                        part >= Smem::kBoxes ? &tmap_v : &tmap_k, full + st,
                        (part & (Smem::kBoxes - 1)) * 64, sl, kvh, pg);
        }
        ++g;
        if (++st == Smem::kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      at += steps;
      first = 0;
      if (++item == items_per_row && at < end) {
        item = 0;
        ++t;
        row = pa_row<kList>(p, t);
      }
    }
    if (lane == 0) p.chain[blockIdx.x] = chain;
    // every copy started here lands before the CTA can exit, whatever the
    // consumers' waits come to
    if constexpr (kFp8) cp_async_wait<0>();
    for (uint32_t i = 0; i < min(g, static_cast<uint32_t>(Smem::kStages)); ++i) {
      if (st == 0) {
        st = Smem::kStages;
        ph ^= 1u;
      }
      --st;
      mbar_drain(full + st, ph, p.drain_limit_ns);
    }
    // (before the end is published the consumers have had all queries but the
    // last two items')
    for (uint32_t i = 1; i <= 2; ++i)
      if (n_items >= i) {
        const uint32_t n = n_items - i;
        if (!(published && i == 2)) mbar_drain(q_full + (n & 1u), (n >> 1) & 1u, p.drain_limit_ns);
      }
    return;
  }

  // ---------------- consumers ----------------
  const int quad = lane & 3, r0 = lane >> 2;
  const float neg_inf = __int_as_float(0xff800000);
  uint32_t base_g = 0;                                        // stages before this item
  for (uint32_t n = 0;; ++n) {
    const uint32_t qb = n & 1u;
    if (!pa_wait(q_full + qb, (n >> 1) & 1u, ctl, 62)) return;
    const PaItem it = info[qb];
    if (it.row < 0) return;
    const int kvh = it.item / p.head_tiles, ht = it.item - kvh * p.head_tiles;
    const int heads = min(kPaRows, p.G - ht * kPaRows);
    const int h0 = kvh * p.G + ht * kPaRows;

    // ---- the query heads as matrix fragments ----
    uint32_t qf[8][4];
    float xs[2] = {p.scale_log2, p.scale_log2};               // logit scale of rows r0, r0 + 8
    {
      const uint8_t *const sq = smem + Smem::off_q + qb * Smem::kQBytes;
      const uint32_t qs = smem_u32(sq);
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // matrices: rows 0-7, 8-15 of features 16kk .. + 7, then of + 8 .. + 15
          const int r = lane & 15, c = (2 * kk + (lane >> 4)) & 7;
          ldsm4(qf[kk], qs + (kk >> 2) * (kPaRows * 128) + r * 128 + ((c ^ (r & 7)) << 4));
        }
      } else {
        // features 16kk + 4 quad .. + 3: the order the fp8 keys' bytes come in
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = r0 + 8 * i, c = (2 * kk + (quad >> 1)) & 7;
            const uint2 w = *reinterpret_cast<const uint2 *>(
                sq + (kk >> 2) * (kPaRows * 128) + r * 128 + ((c ^ (r & 7)) << 4) +
                8 * (quad & 1));
            qf[kk][i] = w.x;
            qf[kk][2 + i] = w.y;
          }
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
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty + qb);

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {neg_inf, neg_inf}, sum[2] = {0.f, 0.f};

    for (int step = (warp - base_g) & (kPaWarps - 1); step < it.steps; step += kPaWarps) {
      const uint32_t gs = base_g + step;
      const uint32_t st = gs % Smem::kStages;
      if (!pa_wait(full + st, (gs / Smem::kStages) & 1u, ctl, 63)) return;
      uint8_t *const stage = smem + st * Smem::kStageBytes;
      const uint32_t mask = masks[st];
      const uint32_t ks = smem_u32(stage), vs = ks + Smem::off_v;
      if (mask != 0xffffffffu) {
        // value rows of slots that are not kept: their weight is 0, and 0
        // times whatever is there has to be 0
        if (!(mask >> lane & 1u)) {
#pragma unroll
          for (int i = 0; i < Smem::kBoxes * 8; ++i)
            *reinterpret_cast<uint4 *>(stage + Smem::off_v + (i >> 3) * Smem::kHalf + lane * 128 +
                                       ((i & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();             // the stage's next load comes from TMA
        __syncwarp();
      }
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            uint32_t b[4];
            const int r = (lane & 7) + 8 * (lane >> 4) + 16 * jj, c = (2 * kk + ((lane >> 3) & 1)) & 7;
            ldsm4(b, ks + (kk >> 2) * Smem::kHalf + r * 128 + ((c ^ (r & 7)) << 4));
            mma_bf16(s[2 * jj], qf[kk], b[0], b[1]);
            mma_bf16(s[2 * jj + 1], qf[kk], b[2], b[3]);
          }
      } else {
        const uint32_t *const sc =
            reinterpret_cast<const uint32_t *>(smem + Smem::off_scale + st * (2 * kPaStep * 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
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
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] *= xs[i >> 1];
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(mask >> (8 * j + 2 * quad + (i & 1)) & 1u)) s[j][i] = neg_inf;
      }
      float mx[2] = {neg_inf, neg_inf};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], s[j][i]);
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
          for (int k = 0; k < 16; ++k) {
            o[k][2 * i] *= a;
            o[k][2 * i + 1] *= a;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float base = m[i] == neg_inf ? 0.f : m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j][2 * i] = ex2_approx(s[j][2 * i] - base);
          s[j][2 * i + 1] = ex2_approx(s[j][2 * i + 1] - base);
          sum[i] += s[j][2 * i] + s[j][2 * i + 1];
        }
      }
      // ---- O += P V ----
      if constexpr (!kFp8) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const uint32_t pf[4] = {
              pack_bf16x2(s[2 * jj][0], s[2 * jj][1]), pack_bf16x2(s[2 * jj][2], s[2 * jj][3]),
              pack_bf16x2(s[2 * jj + 1][0], s[2 * jj + 1][1]),
              pack_bf16x2(s[2 * jj + 1][2], s[2 * jj + 1][3])};
#pragma unroll
          for (int dd = 0; dd < 8; ++dd) {
            uint32_t b[4];
            const int r = (lane & 15) + 16 * jj, c = (2 * dd + (lane >> 4)) & 7;
            ldsm4_t(b, vs + (dd >> 2) * Smem::kHalf + r * 128 + ((c ^ (r & 7)) << 4));
            mma_bf16(o[2 * dd], pf, b[0], b[1]);
            mma_bf16(o[2 * dd + 1], pf, b[2], b[3]);
          }
        }
      } else {
        // the slots' scales go into P: one set of fragments per 32 features
        const uint32_t *const sc = reinterpret_cast<const uint32_t *>(
            smem + Smem::off_scale + st * (2 * kPaStep * 4) + kPaStep * 4);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const uint2 w0 = *reinterpret_cast<const uint2 *>(sc + 16 * jj + 2 * quad);
          const uint2 w1 = *reinterpret_cast<const uint2 *>(sc + 16 * jj + 8 + 2 * quad);
#pragma unroll
          for (int blk = 0; blk < 4; ++blk) {
            const float f0 = __uint_as_float((w0.x >> (8 * blk) & 0xffu) << 23);
            const float f1 = __uint_as_float((w0.y >> (8 * blk) & 0xffu) << 23);
            const float f2 = __uint_as_float((w1.x >> (8 * blk) & 0xffu) << 23);
            const float f3 = __uint_as_float((w1.y >> (8 * blk) & 0xffu) << 23);
            const float(&sa)[4] = s[2 * jj], (&sb)[4] = s[2 * jj + 1];
            const uint32_t pf[4] = {pack_bf16x2(sa[0] * f0, sa[1] * f1), pack_bf16x2(sa[2] * f0, sa[3] * f1),
                                    pack_bf16x2(sb[0] * f2, sb[1] * f3), pack_bf16x2(sb[2] * f2, sb[3] * f3)};
            uint32_t b[4];                     // 16 features x slots 0-7, 8-15; the next 16
            const int r = (lane & 15) + 16 * jj, c = 2 * blk + (lane >> 4);
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
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
    }
    base_g += it.steps;

    // ---- join the four warps' results ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    const int joiner = n & (kPaWarps - 1);
    // the last item's join is over (the joiner waits too: its own wait below
    // must not meet the phase before)
    if (!pa_wait(merge_empty, (n & 1u) ^ 1u, ctl, 64)) return;
    if (warp != joiner) {
      float *const to = reinterpret_cast<float *>(
          smem + Smem::off_merge + ((warp - joiner - 1) & (kPaWarps - 1)) * Smem::kMergeBytes) + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        to[32 * i] = m[i];
        to[32 * (2 + i)] = sum[i];
      }
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[32 * (4 + 4 * k + j)] = o[k][j];
      __syncwarp();
      if (lane == 0) mbar_arrive(merge_full);
      continue;
    }
    if (!pa_wait(merge_full, n & 1u, ctl, 65)) return;
    {
      const float *const from = reinterpret_cast<const float *>(smem + Smem::off_merge) + lane;
      constexpr int kNext = Smem::kMergeBytes / 4;
      float a[kPaWarps][2], M[2], L[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        M[i] = m[i];
#pragma unroll
        for (int w = 0; w < kPaWarps - 1; ++w) M[i] = fmaxf(M[i], from[w * kNext + 32 * i]);
        a[kPaWarps - 1][i] = m[i] == neg_inf ? 0.f : ex2_approx(m[i] - M[i]);
        L[i] = a[kPaWarps - 1][i] * sum[i];
#pragma unroll
        for (int w = 0; w < kPaWarps - 1; ++w) {
          const float mw = from[w * kNext + 32 * i];
          a[w][i] = mw == neg_inf ? 0.f : ex2_approx(mw - M[i]);
          L[i] += a[w][i] * from[w * kNext + 32 * (2 + i)];
        }
      }
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = o[k][j] * a[kPaWarps - 1][j >> 1];
#pragma unroll
          for (int w = 0; w < kPaWarps - 1; ++w) x += a[w][j >> 1] * from[w * kNext + 32 * (4 + 4 * k + j)];
          o[k][j] = x;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(merge_empty);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        if (r >= heads) continue;
        if (it.slot < 0) {
          const int64_t row = static_cast<int64_t>(it.row) * p.H + h0 + r;
          float den = L[i];
          if (p.sinks && M[i] != neg_inf) den += ex2_approx(__ldg(p.sinks + h0 + r) * kPaLog2e - M[i]);
          const float inv = M[i] == neg_inf ? 0.f : 1.f / den;
          if (quad == 0 && p.lse) p.lse[row] = M[i] == neg_inf ? neg_inf : (M[i] + log2f(L[i])) * kPaLn2;
          uint16_t *const dst = p.out + row * kRowD;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            if constexpr (!kFp8) {
              *reinterpret_cast<uint32_t *>(dst + 8 * k + 2 * quad) =
                  pack_bf16x2(o[k][2 * i] * inv, o[k][2 * i + 1] * inv);
              *reinterpret_cast<uint32_t *>(dst + 8 * k + 8 + 2 * quad) =
                  pack_bf16x2(o[k + 1][2 * i] * inv, o[k + 1][2 * i + 1] * inv);
            } else {
              // tiles k, k + 1: the even and odd features of a 16-feature piece
              *reinterpret_cast<uint2 *>(dst + 8 * k + 4 * quad) =
                  make_uint2(pack_bf16x2(o[k][2 * i] * inv, o[k + 1][2 * i] * inv),
                             pack_bf16x2(o[k][2 * i + 1] * inv, o[k + 1][2 * i + 1] * inv));
            }
          }
        } else {
          const int64_t row = (static_cast<int64_t>(blockIdx.x) * 2 + it.slot) * kPaRows + r;
          if (quad == 0) p.part_ml[row] = make_float2(M[i], L[i]);
          float *const dst = p.part_o + row * kRowD;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            if constexpr (!kFp8) {
              *reinterpret_cast<float2 *>(dst + 8 * k + 2 * quad) = make_float2(o[k][2 * i], o[k][2 * i + 1]);
              *reinterpret_cast<float2 *>(dst + 8 * k + 8 + 2 * quad) =
                  make_float2(o[k + 1][2 * i], o[k + 1][2 * i + 1]);
            } else {
              *reinterpret_cast<float4 *>(dst + 8 * k + 4 * quad) =
                  make_float4(o[k][2 * i], o[k + 1][2 * i], o[k][2 * i + 1], o[k + 1][2 * i + 1]);
            }
          }
        }
      }
    }
  }
}

// Joins the items that several CTAs share: an item that begins in CTA a
// (chain.x, chain.y: its row and item) goes on through CTAs a + 1 .. chain.z.
// Two heads a block; a lane joins one 4-feature piece of a head over the
// partials in CTA order.
constexpr int kPaJoinThreads = 64;
__global__ void __launch_bounds__(kPaJoinThreads) paged_attention_join_kernel(
    const PagedAttnParams p) {
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
  const int b = c.z;                                          // the last CTA of the item
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
