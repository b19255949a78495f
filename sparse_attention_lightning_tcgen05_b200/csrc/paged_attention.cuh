// paged_attention.cuh -- attention of query tokens over a paged key-value
// cache (all slots of a sequence, or listed blocks of them) for sm_100a.
//
// For query token t, head h (key-value head g = h / G) and its kept slots s:
//   l_s = sm_scale * q[t,h,:] . k[s,g,:]
//   out = sum_s e^{l_s} v[s,g,:] / (sum_s e^{l_s} + e^{sink_h}),
//   lse = ln sum_s e^{l_s}.
// One pass over the slots with a running maximum m and sum, in log2 units:
// p_s = 2^(x_s - m), x = l * log2(e); the accumulated O and the sum are
// rescaled only when the maximum grows by more than 8 (p stays <= 2^8 and the
// final division removes the common factor, so the result is the same).
// P is rounded to bf16 for its product with V, as V is: an error of half a
// step (2^-9 on average) of each weight, which averages out over the slots.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "paged_cache.cuh"
#include "paged_schedule.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

constexpr int kPaRows = 16;                        // query heads of a work item

__device__ __forceinline__ void cp_async4_zfill(void *smem_dst, const void *gmem_src,
                                                uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem_dst)),
               "l"(gmem_src), "r"(src_bytes)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// c (16 x 8, fp32) += a (16 x 16) * b (16 x 8): bf16 or f16 operands.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
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

// What the producer tells the consumers of an item.
struct PaItem {
  int row, item;               // token (-1: no more items), its (kv head, head tile)
  int steps;                   // of this CTA
  int slot;                    // -1: the whole item; else where the partial result goes (0, 1)
};

// Shared memory. A stage holds kStep slots: bf16 rows as two 128-byte halves
// ([kStep x 64] each), fp8 rows whole, keys then values, in TMA's 128-byte
// swizzle (16-byte piece c of row r at c ^ (r & 7): the eight rows of a matrix
// fragment lie in different banks).
template <bool kFp8>
struct PaSmem {
  static constexpr int kStep = kFp8 ? 32 : 16;
  // Consumer warps: 12 warps an SM have the same 168 registers as 10. The fp8
  // batch below: five with two stages each 241 us, four with three 250; bf16: 189
  // and 175, where the fewer stages cost more than the fifth warp brings.
  static constexpr int kWarps = kFp8 ? 5 : 4;
  static constexpr int kThreads = (kWarps + 1) * 32;                // and the producer
  // Steps worth a CTA: one a consumer warp. One, two and three of them, us: one
  // context of 4,000 slots, 8 key heads, bf16 10.9, 11.4, 13.6, fp8 11.7, 14.5, 15.0;
  // 16 of 200 to 1,000 slots 15.0, 15.0, 15.0 and 17.3, 19.7, 22.2.
  static constexpr int kLeast = kWarps;
  // three (bf16) or two a consumer warp; a stage is always the same warp's, so that no warp
  // waits for a phase before the last one of its barrier is over
  static constexpr int kStages = (kFp8 ? 2 : 3) * kWarps;
  static constexpr int kBox = kStep * 128;                          // one [kStep x 128 B] box
  static constexpr int kBoxes = kFp8 ? 1 : 2;                       // of a row
  static constexpr int off_v = kBoxes * kBox;
  static constexpr int kStageBytes = 2 * kBoxes * kBox;
  static constexpr int off_q = kStages * kStageBytes;               // [2][16 x 64] bf16
  static constexpr int kQBytes = kPaRows * kRowD * 2;
  static constexpr int off_hand = off_q + kQBytes;                  // O, m and sum of a warp
  static constexpr int off_scale = off_hand + 68 * 32 * 4;          // a stage: k words, v words
  static constexpr int kScaleBytes = kFp8 ? 2 * kStep * 4 : 0;
  static constexpr int off_mask = off_scale + kStages * kScaleBytes;
  static constexpr int off_bar = off_mask + 64;
  static constexpr int off_misc = off_bar + 32 * 8;
  static constexpr int kTotal = off_misc + 128;
  static_assert(2 * (kTotal + 1024) <= 228 * 1024, "two CTAs an SM");
};

// A CTA walks a contiguous range of the items' steps. The last warp produces:
// it keeps a ring of stages full with TMA loads, running ahead over the items'
// ends. A consumer warp takes every kWarps-th step with a running maximum, sum
// and O (16 heads x 128 in registers) of its own, and (bf16) has the next step's
// logits multiplied while it works on the present one's softmax. At an item's
// end the warps add up from the first to the next, and the last one writes: always
// in this order, so that from the second item on a warp ends when its turn comes (a
// different first one each time, with a fence at every hand-over: 243 us where this
// takes 234, below). Items that lie in one CTA are finished here; of the others each
// CTA leaves a partial result for the join kernel.
//
// With up to 16 heads on a key-value head the products cost 8 flops a byte of
// the cache at most, which mma.sync sustains beside HBM's rate; its fragments
// also leave each warp its softmax in registers, where tcgen05 would spend its
// 128 rows on 16 heads and take a trip through TMEM a tile. Two CTAs an SM with
// 192 KB (bf16) of stages between them cover HBM's latency. Measured on a B200:
// (calls one by one; graph replays in brackets) 16 contexts of 2,048 to 32,768
// slots, 8 key heads, bf16: 176 us (173), 6.6 TB/s, HBM; 64 contexts of 1,024 to
// 32,768, 4 key heads, fp8: 249 us (216), 4.6 TB/s, bound by the chain from a stage's
// bytes to fragments (about 700 instructions a step of 32 slots; the loads alone take
// 181 us). One context of 1,000 slots: 12.2 us (11.6), a chain of launches, prologue,
// loads, hand-over and join. 1,024 tokens that each list 16 blocks of 64 and the last
// 64 slots: 233 us (208), of them 9.1 a block (2 GB through the L2 in all, 13.9 TB/s),
// 15 fixed and 25 for the items' ends.
template <bool kFp8, bool kList>
__global__ void __launch_bounds__(PaSmem<kFp8>::kThreads, 2)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                           const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const PagedAttnParams p) {
  using Smem = PaSmem<kFp8>;
  constexpr int kStep = Smem::kStep, kWarps = Smem::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t *const masks = reinterpret_cast<uint32_t *>(smem + Smem::off_mask);
  uint64_t *const full = reinterpret_cast<uint64_t *>(smem + Smem::off_bar);
  uint64_t *const empty = full + Smem::kStages;
  uint64_t *const q_full = empty + Smem::kStages;
  uint64_t *const q_empty = q_full + 1;
  uint64_t *const hand_full = q_empty + 1;                          // [kWarps - 1]
  uint64_t *const hand_empty = hand_full + kWarps - 1;
  PaItem *const info = reinterpret_cast<PaItem *>(smem + Smem::off_misc);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(info + 1);
  int *const start_row = reinterpret_cast<int *>(info + 1) + 1;
  int64_t *const start_step = reinterpret_cast<int64_t *>(smem + Smem::off_misc + 32);
  int64_t *const scan = start_step + 1;                             // [kWarps + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Smem::kStages; ++i) {
      mbar_init(full + i, kFp8 ? 33 : 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, kWarps);
    for (int i = 0; i < kWarps - 1; ++i) mbar_init(hand_full + i, 1);
    mbar_init(hand_empty, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  const PaRange range =
      pa_range<kList, kStep, Smem::kThreads>(p, Smem::kLeast, tid, scan, start_row, start_step);
  if (range.begin >= range.end) {
    PaChain{}.finish(p, tid);
    return;
  }
  const WaitCtl ctl{abort_flag, p.err, p.err_info, p.wait_limit_ns};

  if (warp == kWarps) {
    // ---------------- producer ----------------
    PaCursor<kList, kStep> cur;
    cur.start(p, range.kvh, *start_row, *start_step, range.end - range.begin);
    PaLookup<kList, kStep, kStep> look;
    look.start(p, lane, cur);
    PaChain chain;
    const int gran = 1 << p.gran_shift;
    const int per_step = look.per_unit(p);                    // lookups and boxes a step
    uint32_t g = 0, st = 0, ph = 0, n_items = 0;
    uint32_t my_st = 0, my_ph = 0, round = 0;                 // the round's stage of this lane; heads that went
    bool ok = true, published = false;
    while (ok) {
      const bool more = cur.steps > 0;
      const bool whole = cur.steps == cur.row.steps;
      const int id = cur.id(p);
      const int kvh = id / p.head_tiles, ht = id - kvh * p.head_tiles;
      if (!pa_wait(q_empty, (n_items & 1u) ^ 1u, ctl, 60)) break;
      if (lane == 0) {
        *info = PaItem{more ? cur.t : -1, id, cur.steps, whole ? -1 : cur.first == 0 ? 1 : 0};
        if (more) {
          const int q_row = cur.t * p.H + kvh * p.G + ht * kPaRows;
          mbar_arrive_expect_tx(q_full, Smem::kQBytes);
          tma_load_2d(smem + Smem::off_q, &tmap_q, q_full, 0, q_row);
          tma_load_2d(smem + Smem::off_q + Smem::kQBytes / 2, &tmap_q, q_full, 64, q_row);
        } else {
          mbar_arrive(q_full);
        }
      }
      __syncwarp();
      if (!more) {
        published = true;
        break;
      }
      ++n_items;
      chain.add(p, range, lane, cur.t, id, range.end - cur.left, cur.first, cur.steps, cur.row.steps);
      // Rounds of up to four steps, a lane a granule: the first lane of a step
      // watches its stage, and as soon as that is free the step's lanes issue
      // their boxes. (A step at a time, with its lookup broadcast to the warp,
      // took 425 cycles before any load was issued, and bounded the kernel.)
      uint32_t mask = 0, live = 0;                            // of this lane's step
      for (int step = 0; step < cur.steps;) {
        const int in_look = step & (look.batch(p) - 1);
        if (in_look == 0) {
          look.next(p, lane);
          live = look.hi > look.lo;
          mask = live ? ((2u << (look.hi - 1)) - (1u << look.lo)) << look.within(p, lane) : 0u;
          for (int off = 1; off < per_step; off <<= 1) {
            mask |= __shfl_xor_sync(0xffffffffu, mask, off);
            live += __shfl_xor_sync(0xffffffffu, live, off);
          }
        }
        const int count = min(min(4, look.batch(p) - in_look), cur.steps - step);
        const int mine = (lane / per_step) - in_look;         // this lane's step of the round
        bool todo = mine >= 0 && mine < count;
        my_st = st + (todo ? mine : 0);
        my_ph = ph;
        if (my_st >= Smem::kStages) {
          my_st -= Smem::kStages;
          my_ph ^= 1u;
        }
        const int head = lane & ~(per_step - 1);
        PaPatience patience;
        while (ok) {
          const uint32_t free_heads =
              __ballot_sync(0xffffffffu, todo && lane == head && mbar_test_wait(empty + my_st, my_ph ^ 1u));
          const bool go = todo && (free_heads >> head & 1u);
          if (go && lane == head) {
            masks[my_st] = mask;
            mbar_arrive_expect_tx(full + my_st, live * (gran * 128 * 2 * Smem::kBoxes));
          }
          __syncwarp();
          if (go && look.hi > look.lo) {
            uint8_t *const dst = smem + my_st * Smem::kStageBytes + look.within(p, lane) * 128;
            if (per_step == 1) {
              tma_load_5d(dst, &tmap_k, full + my_st, 0, look.slot, 0, kvh, look.page);
              tma_load_5d(dst + Smem::off_v, &tmap_v, full + my_st, 0, look.slot, 0, kvh, look.page);
            } else {
              // a box smaller than the stage's halves is loaded half by half
#pragma unroll
              for (int b = 0; b < Smem::kBoxes; ++b) {
                tma_load_5d(dst + b * Smem::kBox, &tmap_k, full + my_st, 0, look.slot, b, kvh, look.page);
                tma_load_5d(dst + Smem::off_v + b * Smem::kBox, &tmap_v, full + my_st, 0, look.slot, b, kvh,
                            look.page);
              }
            }
          }
          if constexpr (kFp8) {
            // the scales of the steps that just went, a lane a slot
            for (uint32_t left = free_heads; left != 0; left &= left - 1) {
              const int h = __ffs(left) - 1;
              const uint32_t stage = __shfl_sync(0xffffffffu, my_st, h);
              const bool keep = __shfl_sync(0xffffffffu, mask, h) >> lane & 1u;
              const int pg = __shfl_sync(0xffffffffu, look.page, h + (lane >> p.gran_shift));
              const int sl = __shfl_sync(0xffffffffu, look.slot, h + (lane >> p.gran_shift));
              const int64_t o = keep ? (pg * p.g.page_stride +
                                        static_cast<int64_t>(sl + (lane & (gran - 1))) * p.g.slot_stride +
                                        kvh * p.g.head_stride) / 32
                                     : 0;
              uint8_t *const sc = smem + Smem::off_scale + stage * Smem::kScaleBytes + 4 * lane;
              cp_async4_zfill(sc, p.k_scale + o, keep ? 4u : 0u);
              cp_async4_zfill(sc + kStep * 4, p.v_scale + o, keep ? 4u : 0u);
              cp_async_mbar_arrive_noinc(full + stage);
            }
          }
          round |= free_heads;
          todo = todo && !go;
          if (!__any_sync(0xffffffffu, todo)) break;
          ok = patience.more(ctl, 61);
        }
        if (!ok) break;
        round = 0;
        g += count;
        step += count;
        st += count;
        if (st >= Smem::kStages) {
          st -= Smem::kStages;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      cur.advance(p);
    }
    chain.finish(p, lane);
    // every copy started here lands before the CTA can exit, whatever the
    // consumers' waits come to: the last round's (where it was given up), and
    // the last one of each stage before it
    if constexpr (kFp8) cp_async_wait<0>();
    uint32_t again = 0;                                       // stages that last round filled
    for (uint32_t left = round; left != 0; left &= left - 1) {
      const int h = __ffs(left) - 1;
      const uint32_t i = __shfl_sync(0xffffffffu, my_st, h);
      mbar_drain(full + i, __shfl_sync(0xffffffffu, my_ph, h), p.drain_limit_ns);
      again |= 1u << i;
    }
    for (uint32_t i = 0; i < min(g, static_cast<uint32_t>(Smem::kStages)); ++i) {
      if (st == 0) {
        st = Smem::kStages;
        ph ^= 1u;
      }
      --st;
      if (!(again >> st & 1u)) mbar_drain(full + st, ph, p.drain_limit_ns);
    }
    // (before their end is published the consumers have had all queries)
    if (!published && n_items > 0) mbar_drain(q_full, (n_items - 1) & 1u, p.drain_limit_ns);
    return;
  }

  // ---------------- consumers ----------------
  constexpr int kJ = kStep / 8;                               // 8-slot tiles of a step
  constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : (1u << (kStep & 31)) - 1u;
  const int quad = lane & 3, r0 = lane >> 2;
  const float neg_inf = __int_as_float(0xff800000);
  uint32_t base_g = 0;                                        // stages before this item
  for (uint32_t n = 0;; ++n) {
    if (!pa_wait(q_full, n & 1u, ctl, 62)) return;
    const PaItem it = *info;
    if (it.row < 0) return;
    const int kvh = it.item / p.head_tiles, ht = it.item - kvh * p.head_tiles;
    const int heads = min(kPaRows, p.G - ht * kPaRows);
    const int h0 = kvh * p.G + ht * kPaRows;

    // ---- the query heads as matrix fragments ----
    uint32_t qf[8][4];
    // logit scale of rows r0, r0 + 8: a negative one's sign goes to the query, so
    // that the largest product is the largest logit; 0 counts as the least number
    // above it, so that a masked logit stays -infinity
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const float scale = fabsf(p.scale_log2), least = __int_as_float(1);
    float xs[2] = {fmaxf(scale, least), fmaxf(scale, least)};
    {
      const uint8_t *const sq = smem + Smem::off_q;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // matrices: rows 0-7, 8-15 of features 16kk .. + 7, then of + 8 .. + 15
          const int r = lane & 15, c = (2 * kk + (lane >> 4)) & 7;
          ldsm4(qf[kk], smem_u32(sq) + (kk >> 2) * (kPaRows * 128) + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[kk][i] ^= flip;
        }
      } else {
        // features 16kk + 4 quad .. + 3: the order the fp8 keys' bytes come in
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = r0 + 8 * i, c = (2 * kk + (quad >> 1)) & 7;
            const uint2 w = *reinterpret_cast<const uint2 *>(
                sq + (kk >> 2) * (kPaRows * 128) + r * 128 + ((c ^ (r & 7)) << 4) + 8 * (quad & 1));
            qf[kk][i] = w.x ^ flip;
            qf[kk][2 + i] = w.y ^ flip;
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
          xs[i] = fmaxf(scale * __int_as_float((127 - shift) << 23), least);
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
    pa_release(q_empty, lane);

    // S = Q K^T of the step in stage gs (unscaled), once its copies are there
    auto logits = [&](uint32_t gs, float (&s)[kJ][4], uint32_t &mask) -> bool {
      const uint32_t st = gs % Smem::kStages;
      if (!pa_wait(full + st, (gs / Smem::kStages) & 1u, ctl, 63)) return false;
      const uint32_t ks = smem_u32(smem + st * Smem::kStageBytes);
      mask = masks[st];
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int jj = 0; jj < kJ / 2; ++jj) {
            uint32_t b[4];
            const int r = (lane & 7) + 8 * (lane >> 4) + 16 * jj, c = (2 * kk + ((lane >> 3) & 1)) & 7;
            ldsm4(b, ks + (kk >> 2) * Smem::kBox + r * 128 + ((c ^ (r & 7)) << 4));
            mma_bf16(s[2 * jj], qf[kk], b[0], b[1]);
            mma_bf16(s[2 * jj + 1], qf[kk], b[2], b[3]);
          }
      } else {
        const uint32_t *const sc =
            reinterpret_cast<const uint32_t *>(smem + Smem::off_scale + st * Smem::kScaleBytes);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
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
      return true;
    };

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    // The running maximum (of unscaled logits until the item's end), 0 instead of
    // it while there is none, and the logit past which O is rescaled (four lanes
    // share a row's). The maximum is taken off before the scaling: the largest
    // weight is then exactly 1 however large the logits are, where an fma of scaled
    // ones leaves what the maximum's own rounding dropped, hundreds at 2^33.
    float m[2] = {neg_inf, neg_inf}, mb[2] = {0.f, 0.f}, limit[2] = {neg_inf, neg_inf};
    float sum[2] = {0.f, 0.f};
    // The next step's logits ahead: not for fp8 (no registers), and not for listed
    // blocks, which L2 feeds: holding two stages at once then costs more loads in
    // flight than it hides (1,024 tokens, 16 blocks of 64 each: 243 us with, 210
    // without; a batch over all its slots, which HBM feeds: 173 and 181).
    constexpr bool kAhead = !kFp8 && !kList;
    float s[kJ][4], s_next[kAhead ? kJ : 1][4];
    uint32_t mask = 0, mask_next = 0;
    const int step0 = static_cast<int>((warp + kWarps - base_g % kWarps) % kWarps);
    if (kAhead && step0 < it.steps && !logits(base_g + step0, s, mask)) return;
    for (int step = step0; step < it.steps; step += kWarps) {
      if constexpr (kAhead) {
        if (step + kWarps < it.steps && !logits(base_g + step + kWarps, s_next, mask_next)) return;
      } else {
        if (!logits(base_g + step, s, mask)) return;
      }
      const uint32_t st = (base_g + step) % Smem::kStages;
      uint8_t *const stage = smem + st * Smem::kStageBytes;
      const uint32_t vs = smem_u32(stage) + Smem::off_v;
      // ---- softmax: rows r0 and r0 + 8, slots 8j + 2 quad + {0, 1} ----
      if (mask != kAll) {
        // value rows of slots that are not kept: their weight is 0, and 0
        // times whatever is there has to be 0
        if (lane < kStep && !(mask >> lane & 1u)) {
#pragma unroll
          for (int i = 0; i < Smem::kBoxes * 8; ++i)
            *reinterpret_cast<uint4 *>(stage + Smem::off_v + (i >> 3) * Smem::kBox + lane * 128 +
                                       ((i & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(mask >> (8 * j + 2 * quad + (i & 1)) & 1u)) s[j][i] = neg_inf;
      }
      float mx[2] = {neg_inf, neg_inf};
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], s[j][i]);
      if (__any_sync(0xffffffffu, mx[0] > limit[0] || mx[1] > limit[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          const float mn = fmaxf(m[i], mx[i]);
          if (mn == neg_inf) continue;
          const float a = m[i] == neg_inf ? 0.f : ex2_approx((m[i] - mn) * xs[i]);
          m[i] = mb[i] = mn;
          limit[i] = __fadd_rd(mn, __fdividef(kPaLazy, xs[i]));
          sum[i] *= a;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            o[k][2 * i] *= a;
            o[k][2 * i + 1] *= a;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = fmul2(fadd2(make_float2(s[j][2 * i], s[j][2 * i + 1]), make_float2(-mb[i], -mb[i])),
                                 make_float2(xs[i], xs[i]));
          s[j][2 * i] = ex2_approx(x.x);
          s[j][2 * i + 1] = ex2_approx(x.y);
          sum[i] += s[j][2 * i];
          sum[i] += s[j][2 * i + 1];
        }
      // ---- O += P V ----
      if constexpr (!kFp8) {
#pragma unroll
        for (int jj = 0; jj < kJ / 2; ++jj) {
          const uint32_t pf[4] = {
              pack_bf16x2(s[2 * jj][0], s[2 * jj][1]), pack_bf16x2(s[2 * jj][2], s[2 * jj][3]),
              pack_bf16x2(s[2 * jj + 1][0], s[2 * jj + 1][1]),
              pack_bf16x2(s[2 * jj + 1][2], s[2 * jj + 1][3])};
#pragma unroll
          for (int dd = 0; dd < 8; ++dd) {
            uint32_t b[4];
            const int r = (lane & 15) + 16 * jj, c = (2 * dd + (lane >> 4)) & 7;
            ldsm4_t(b, vs + (dd >> 2) * Smem::kBox + r * 128 + ((c ^ (r & 7)) << 4));
            mma_bf16(o[2 * dd], pf, b[0], b[1]);
            mma_bf16(o[2 * dd + 1], pf, b[2], b[3]);
          }
        }
      } else {
        // the slots' scales go into P: one set of fragments per 32 features (exact
        // where the product is 2^-126 or more: bf16 keeps its bits from there on)
        const uint32_t *const sc =
            reinterpret_cast<const uint32_t *>(smem + Smem::off_scale + st * Smem::kScaleBytes) + kStep;
#pragma unroll
        for (int jj = 0; jj < kJ / 2; ++jj) {
          const uint2 w0 = *reinterpret_cast<const uint2 *>(sc + 16 * jj + 2 * quad);
          const uint2 w1 = *reinterpret_cast<const uint2 *>(sc + 16 * jj + 8 + 2 * quad);
          const float(&sa)[4] = s[2 * jj], (&sb)[4] = s[2 * jj + 1];
          const uint32_t pr[4] = {pack_bf16x2(sa[0], sa[1]), pack_bf16x2(sa[2], sa[3]),
                                  pack_bf16x2(sb[0], sb[1]), pack_bf16x2(sb[2], sb[3])};
#pragma unroll
          for (int blk = 0; blk < 4; ++blk) {
            // two slots' scale bytes as two bf16 powers of two (255: infinity,
            // which makes a NaN of the zero data beside it)
            const uint32_t f0 = __byte_perm(w0.x, w0.y, 0x4400 + 0x1111 * blk) << 7 & 0x7f807f80u;
            const uint32_t f1 = __byte_perm(w1.x, w1.y, 0x4400 + 0x1111 * blk) << 7 & 0x7f807f80u;
            const uint32_t pf[4] = {mul_bf16x2(pr[0], f0), mul_bf16x2(pr[1], f0), mul_bf16x2(pr[2], f1),
                                    mul_bf16x2(pr[3], f1)};
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
      pa_release(empty + st, lane);
      if constexpr (kAhead) {
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][i] = s_next[j][i];
        mask = mask_next;
      }
    }
    base_g += it.steps;

    // ---- add the warps' results up, from warp 0 to the last ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
      // in log2 units from here on; no maximum although slots were kept, their
      // logits being NaN: any number, so that the sum is not taken for an empty one
      if (m[i] != neg_inf) m[i] *= xs[i];
      else if (sum[i] != 0.f) m[i] = 0.f;
    }
    // the last item's sum is taken over (every warp waits: a wait below must
    // not meet the phase before)
    if (!pa_wait(hand_empty, (n & 1u) ^ 1u, ctl, 64)) return;
    float4 *const hand = reinterpret_cast<float4 *>(smem + Smem::off_hand) + lane;
    if (warp > 0) {
      if (!pa_wait(hand_full + warp - 1, n & 1u, ctl, 65)) return;
      const float4 got = hand[0];
      float a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mo = i ? got.y : got.x, M = fmaxf(m[i], mo);
        a[i] = m[i] == neg_inf ? 0.f : ex2_approx(m[i] - M);
        b[i] = mo == neg_inf ? 0.f : ex2_approx(mo - M);
        sum[i] = a[i] * sum[i] + b[i] * (i ? got.w : got.z);
        m[i] = M;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float4 x = hand[32 * (1 + k)];
        o[k][0] = fmaf(b[0], x.x, a[0] * o[k][0]);
        o[k][1] = fmaf(b[0], x.y, a[0] * o[k][1]);
        o[k][2] = fmaf(b[1], x.z, a[1] * o[k][2]);
        o[k][3] = fmaf(b[1], x.w, a[1] * o[k][3]);
      }
    }
    if (warp < kWarps - 1) {
      hand[0] = make_float4(m[0], m[1], sum[0], sum[1]);
#pragma unroll
      for (int k = 0; k < 16; ++k) hand[32 * (1 + k)] = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
      __syncwarp();                                           // (read by a warp, not by TMA: no fence)
      if (lane == 0 && !(p.selftest_stall && warp == 0)) mbar_arrive(hand_full + warp);
      continue;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(hand_empty);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      if (r >= heads) continue;
      if (m[i] == neg_inf) {
        // nothing kept but logits of -infinity, whose weights of 0 make NaN of an
        // infinite value
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k][2 * i] = o[k][2 * i + 1] = 0.f;
      }
      if (it.slot < 0) {
        const int64_t row = static_cast<int64_t>(it.row) * p.H + h0 + r;
        float den = sum[i];
        if (p.sinks && m[i] != neg_inf) den += ex2_approx(__ldg(p.sinks + h0 + r) * kPaLog2e - m[i]);
        const float inv = m[i] == neg_inf ? 0.f : 1.f / den;
        if (quad == 0 && p.lse) p.lse[row] = m[i] == neg_inf ? neg_inf : (m[i] + log2f(sum[i])) * kPaLn2;
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
        if (quad == 0) p.part_ml[row] = make_float2(m[i], sum[i]);
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

// Joins the items that several CTAs share: an item that begins in CTA a
// (chain: a row, its item there, a and the last CTA) left a partial result in
// a's second place and in the first place of a + 1 .. last. kWays warps a head,
// a 4-feature piece a lane, each over every kWays-th partial with kBatch of
// them in flight, added up through shared memory in warp order. Eight ways
// where items are few and their partials many (4 contexts of 65,000 to 131,072
// slots under 128 heads, 37 partials an item: the whole call 66 us by one warp a
// head, 61 so); one way, and fewer blocks, where most items lie in one or two
// CTAs (16 contexts of 2,048 to 32,768 slots, 8 key heads: 183 us by eight ways,
// 176 by one; 64 contexts, fp8: 260 and 249).
constexpr int kPaJoinThreads = 512;
template <int kWays>
constexpr int kPaJoinHeads = kPaJoinThreads / 32 / kWays;     // of a block
template <int kWays>
__global__ void __launch_bounds__(kPaJoinThreads) paged_attention_join_kernel(
    const PagedAttnParams p) {
  constexpr int kBatch = kWays > 1 ? 8 : 4;
  __shared__ float4 acc_of[kPaJoinHeads<kWays>][kWays][32];
  __shared__ float2 ml_of[kPaJoinHeads<kWays>][kWays];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int blocks = p.rows / kPaJoinHeads<kWays>;
  const int entry = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = warp / kWays, way = warp - head * kWays;
  const int r = (blockIdx.x - entry * blocks) * kPaJoinHeads<kWays> + head;
  const int4 c = p.chain[entry];
  // -1: nothing to join; out of range: left by another call where a wait that
  // ran out kept this one's entry from being written
  if (c.x < 0 || c.x >= p.T || c.y < 0 || c.y >= p.g.H_kv * p.head_tiles || c.z < 0 || c.w >= p.ctas) return;
  const int kvh = c.y / p.head_tiles, ht = c.y - kvh * p.head_tiles;
  const bool in = r < min(p.rows, p.G - ht * p.rows);
  const float neg_inf = __int_as_float(0xff800000);
  const int a = c.z, b = c.w;
  // this warp's partials
  float M = neg_inf, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = a + way; in && i0 <= b; i0 += kBatch * kWays) {
    float2 ml[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kWays;
      const int64_t row = (static_cast<int64_t>(i) * 2 + (i == a)) * p.rows + r;
      ml[j] = make_float2(neg_inf, 0.f);
      x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i <= b) {
        ml[j] = __ldcg(p.part_ml + row);
        x[j] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + row * kRowD) + lane);
      }
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
    if (top == neg_inf) continue;
    const float old = M == neg_inf ? 0.f : ex2_approx(M - top);
    M = top;
    L *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float w = ml[j].x == neg_inf ? 0.f : ex2_approx(ml[j].x - M);
      L = fmaf(w, ml[j].y, L);
      acc.x = fmaf(w, x[j].x, acc.x);
      acc.y = fmaf(w, x[j].y, acc.y);
      acc.z = fmaf(w, x[j].z, acc.z);
      acc.w = fmaf(w, x[j].w, acc.w);
    }
  }
  acc_of[head][way][lane] = acc;
  if (lane == 0) ml_of[head][way] = make_float2(M, L);
  __syncthreads();
  if (way != 0 || !in) return;
  for (int w = 0; w < kWays; ++w) M = fmaxf(M, ml_of[head][w].x);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kWays; ++w) {
    const float2 ml = ml_of[head][w];
    const float4 x = acc_of[head][w][lane];
    const float f = ml.x == neg_inf ? 0.f : ex2_approx(ml.x - M);
    L = fmaf(f, ml.y, L);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  const int h = kvh * p.G + ht * p.rows + r;
  const int64_t orow = static_cast<int64_t>(c.x) * p.H + h;
  float den = L;
  if (p.sinks && M != neg_inf) den += ex2_approx(__ldg(p.sinks + h) * kPaLog2e - M);
  const float inv = M == neg_inf ? 0.f : 1.f / den;
  if (lane == 0 && p.lse) p.lse[orow] = M == neg_inf ? neg_inf : (M + log2f(L)) * kPaLn2;
  reinterpret_cast<uint2 *>(p.out + orow * kRowD)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace dsa
