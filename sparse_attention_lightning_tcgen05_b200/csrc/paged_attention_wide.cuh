// paged_attention_wide.cuh -- attention over a paged cache on tcgen05, for
// sm_100a: more than 16 (fp8: 48) query heads on a key-value head.
//
// The same sums as paged_attention.cuh, all of a key-value head's query heads
// (up to 128) being the M = 128 rows of both products, so that a slot is loaded
// once for all of them:
//   S = Q K^T  (128 rows x 128 slots, K = D) from shared memory into TMEM,
//   O += P V   (128 rows x D, K = 128 slots) with P read from TMEM, where the
//              softmax wrote it over S, and V MN-major from its tile.
// Tiles of 128 slots alternate between two streams, each with its own S (128
// TMEM columns), O (128 columns), running maxima and sums, and softmax warps,
// so that one stream's products run under the other's softmax; the streams
// are added up at the item's end. Warps 0-3 and 4-7: the streams' softmax, a
// thread a row; warp 8 issues the products; warp 9 loads. With G heads on a
// key the products cost 4 G D flops for the 4 D bytes of a bf16 key and value,
// past what mma.sync sustains at HBM speed from about 32 heads on.
//
// An fp8 cache is loaded as it is and turned into bf16 tiles by warps 10 to 15
// (e4m3 times a power of two is exact in bf16); the rest is as for bf16.
//
// Measured on a B200 with 128 heads: 4 contexts of 65,000 to 131,072 slots, bf16:
// 61 us, in graph replays 57, of them 18 fixed (launches, prologue, hand-over, join)
// and the rest HBM's rate; 4 x 65,536 slots in graph replays: bf16 39 us, fp8 55 (63
// with two converting warps; 40 without the conversion, 40 without the softmax, 34
// without both: they share the issue slots, and a staged tile waits for both).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "paged_attention.cuh"
#include "paged_schedule.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

constexpr int kPwTile = 128;                       // slots a tile
constexpr int kPwUnit = 32;                        // slots a lookup round's unit
constexpr int kPwRows = 128;                       // query heads of a work item, at most
constexpr int kPwLeast = 2;                        // tiles worth a CTA
constexpr int kPwMmaWarp = 8;
constexpr int kPwConvertWarp = 10;                 // fp8: and the next five, to the block's 16
constexpr int kPwConvertWarps = 6;

// Shared memory: bf16 tiles as two halves of their rows ([128 x 128 bytes]
// each, 128-byte swizzle), loaded directly or (fp8) converted from slots of a
// staging ring, in which a tile's keys and values take a slot each.
template <bool kFp8>
struct PwSmem {
  static constexpr int kThreads = (kPwConvertWarp + (kFp8 ? kPwConvertWarps : 0)) * 32;
  // fp8: K's tile is free again while V's is being converted
  static constexpr int kKStages = kFp8 ? 1 : 3, kVStages = kFp8 ? 2 : 3;
  static constexpr int kSlots = kFp8 ? 5 : 0;
  static constexpr int kHalf = kPwTile * 128;                       // [128 x 128 B]
  static constexpr int kTileBytes = 2 * kHalf;
  static constexpr int off_q = 0;
  static constexpr int off_k = kTileBytes;
  static constexpr int off_v = off_k + kKStages * kTileBytes;
  static constexpr int off_slot = off_v + kVStages * kTileBytes;
  static constexpr int kSlotBytes = kHalf;                          // [128 x 128 B] e4m3
  static constexpr int off_scale = off_slot + kSlots * kSlotBytes;  // [slots][128] words
  static constexpr int off_ml = off_scale + kSlots * kPwTile * 4;   // [2 streams][128 rows] (max, sum)
  // kept slots of a tile, in a ring that outlasts every stage between the
  // producer and the softmax
  static constexpr int kMasks = 8;
  static constexpr int off_mask = off_ml + 2 * kPwRows * 8;         // [kMasks][4]
  static constexpr int off_bar = off_mask + kMasks * 16;
  static constexpr int off_misc = off_bar + 40 * 8;
  static constexpr int kTotal = off_misc + 192;
  static_assert(kTotal <= 227 * 1024, "one CTA an SM");
};

// D[tmem] (+)= A[tmem] * B[smem desc]: bf16, A's row i in lane i, two
// consecutive K elements a 32-bit column.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Eight floats, a whole 32-byte sector, in one store (dst 32-byte aligned).
__device__ __forceinline__ void st_global_v8(float *dst, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// This thread's lane of 16 TMEM columns from taddr on.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

// 16 e4m3 features of a row as 16 bf16 values times a power of two: f1 is
// 2^(s - 127 + 120) (bf16_of_even: a byte's bits read as bf16 are its value
// times 2^-120), or 2^120 with f2 the scale where that is past bf16's exponents.
__device__ __forceinline__ void bf16_of_e4m3x16(uint4 w, uint32_t f1, uint32_t f2, bool two,
                                                uint4 (&out)[2]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __byte_perm(in[i >> 1], 0, i & 1 ? 0x3424 : 0x1404);   // byte, 0, next, 0
    r[i] = mul_bf16x2((u & 0x80008000u) | (u >> 4 & 0x07f007f0u), f1);
    if (two) r[i] = mul_bf16x2(r[i], f2);
  }
  out[0] = make_uint4(r[0], r[1], r[2], r[3]);
  out[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// A slot's staged row (with its scale word) as a row of a bf16 tile.
__device__ __forceinline__ void convert_row(const uint8_t *slot, uint32_t scales, uint8_t *tile, int r) {
  // two multiplications where a scale is 2^8 or more (or NaN): rare
  const bool two = ((scales & 0x7f7f7f7fu) + 0x79797979u & scales & 0x80808080u) != 0;
  uint4 in[8];                                                // (read before any store)
#pragma unroll
  for (int c = 0; c < 8; ++c)
    in[c] = *reinterpret_cast<const uint4 *>(slot + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 w = in[c];
    const uint32_t s = scales >> (8 * (c >> 1)) & 0xffu;
    uint32_t f1 = (s + 120u) << 7, f2 = 0;
    if (two) {
      f1 = 0x7b80u;                                          // 2^120
      f2 = s == 255u ? 0x7fc0u : s == 0u ? 0x0040u : s << 7;
      f2 |= f2 << 16;
    }
    uint4 out[2];
    bf16_of_e4m3x16(w, f1 | f1 << 16, f2, two, out);
    uint8_t *const row = tile + (c >> 2) * (kPwTile * 128) + r * 128;
    *reinterpret_cast<uint4 *>(row + ((((2 * c) & 7) ^ (r & 7)) << 4)) = out[0];
    *reinterpret_cast<uint4 *>(row + ((((2 * c + 1) & 7) ^ (r & 7)) << 4)) = out[1];
  }
}

template <bool kFp8, bool kList>
__global__ void __launch_bounds__(PwSmem<kFp8>::kThreads, 1)
    paged_attention_wide_kernel(const __grid_constant__ CUtensorMap tmap_q,
                                const __grid_constant__ CUtensorMap tmap_k,
                                const __grid_constant__ CUtensorMap tmap_v, const PagedAttnParams p) {
  using Smem = PwSmem<kFp8>;
  constexpr int kKStages = Smem::kKStages, kVStages = Smem::kVStages;
  constexpr int kSub = kPwTile / kPwUnit;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t *const masks = reinterpret_cast<uint32_t *>(smem + Smem::off_mask);
  uint64_t *const k_full = reinterpret_cast<uint64_t *>(smem + Smem::off_bar);
  uint64_t *const v_full = k_full + kKStages;
  uint64_t *const k_empty = v_full + kVStages;
  uint64_t *const v_empty = k_empty + kKStages;
  uint64_t *const slot_full = v_empty + kVStages;
  uint64_t *const slot_empty = slot_full + Smem::kSlots;
  uint64_t *const q_full = slot_empty + Smem::kSlots;
  uint64_t *const q_empty = q_full + 1;
  uint64_t *const s_full = q_empty + 1;                             // [2]
  uint64_t *const p_full = s_full + 2;                              // [2]
  uint64_t *const pv_done = p_full + 2;                             // [2]
  uint64_t *const item_done = pv_done + 2;
  uint64_t *const ml_full = item_done + 1;
  uint64_t *const o_free = ml_full + 1;
  PaItem *const info = reinterpret_cast<PaItem *>(smem + Smem::off_misc);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(info + 1);
  int *const start_row = reinterpret_cast<int *>(info + 1) + 1;
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(info + 1) + 2;
  int64_t *const start_step = reinterpret_cast<int64_t *>(smem + Smem::off_misc + 32);
  int64_t *const scan = start_step + 1;                             // [kThreads / 32]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kPwMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    // tiles are filled by four units' loads, or by the converting warps
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(k_full + i, kFp8 ? kPwConvertWarps : kSub);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(v_full + i, kFp8 ? kPwConvertWarps : kSub);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < Smem::kSlots; ++i) {
      mbar_init(slot_full + i, kSub * 33);        // a unit's loads and its 32 scale words
      mbar_init(slot_empty + i, kPwConvertWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 9);                         // the softmax warps and the last Q K^T
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(item_done, 1);
    mbar_init(ml_full, 8);
    mbar_init(o_free, 8);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  tc_fence_before_sync();
  const PaRange range =
      pa_range<kList, kPwTile, Smem::kThreads>(p, kPwLeast, tid, scan, start_row, start_step);
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.err, p.err_info, p.wait_limit_ns};

  if (range.begin >= range.end) {
    PaChain{}.finish(p, tid);
  } else if (kFp8 && warp >= kPwConvertWarp) {
    // ---------------- conversion: a unit a warp, a slot's row a thread ----------------
    // units in turn, so that six warps share the four of a load evenly; every
    // warp waits and arrives for every load, so that none is a phase apart
    int sub = warp - kPwConvertWarp;                          // this warp's unit, from the load's first
    const uint32_t tiles = static_cast<uint32_t>(range.end - range.begin);
    for (uint32_t c = 0; c < 2 * tiles; ++c) {
      const uint32_t t = c >> 1, is_v = c & 1u;
      const uint32_t slot = c % (Smem::kSlots + !kFp8), lap = c / (Smem::kSlots + !kFp8);
      const uint32_t st = is_v ? t % kVStages : t % kKStages, use = is_v ? t / kVStages : t / kKStages;
      if (!pa_wait(slot_full + slot, lap & 1u, ctl, 84) ||
          !pa_wait((is_v ? v_empty : k_empty) + st, (use & 1u) ^ 1u, ctl, 85))
        break;
      const uint8_t *const from = smem + Smem::off_slot + slot * Smem::kSlotBytes;
      uint8_t *const to = smem + (is_v ? Smem::off_v : Smem::off_k) + st * Smem::kTileBytes;
      const uint32_t *const scales = reinterpret_cast<const uint32_t *>(smem + Smem::off_scale) + slot * kPwTile;
      if (sub < kSub) {
        const int r = sub * kPwUnit + lane;
        if (masks[t % Smem::kMasks * kSub + sub] >> lane & 1u) {
          convert_row(from, scales[r], to, r);
        } else {
          // a slot that is not kept: whatever was staged, its row is zero
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint4 *>(to + (i >> 3) * Smem::kHalf + r * 128 + ((i & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        sub += kPwConvertWarps;
      }
      sub -= kSub;
      pa_release((is_v ? v_full : k_full) + st, lane);        // read by the products (async proxy)
      if (lane == 0) mbar_arrive(slot_empty + slot);
    }
  } else if (warp > kPwMmaWarp) {
    // ---------------- producer ----------------
    PaCursor<kList, kPwTile> cur;
    cur.start(p, range.kvh, *start_row, *start_step, range.end - range.begin);
    PaLookup<kList, kPwTile, kPwUnit> look;
    look.start(p, lane, cur);
    PaChain chain;
    const int gran = 1 << p.gran_shift;
    const int per_unit = look.per_unit(p);
    const int q_rows = min(kPwRows, p.G);
    uint32_t g = 0, n_items = 0;                              // units before this round, items
    uint32_t round = 0;                                       // heads of the round that went
    bool ok = true, published = false;
    while (ok) {
      const bool more = cur.steps > 0;
      const bool whole = cur.steps == cur.row.steps;
      const int kvh = cur.id(p);                              // one item a head
      if (!pa_wait(q_empty, (n_items & 1u) ^ 1u, ctl, 70)) break;
      if (lane == 0) {
        *info = PaItem{more ? cur.t : -1, kvh, cur.steps, whole ? -1 : cur.first == 0 ? 1 : 0};
        if (more) {
          const int q_row = cur.t * p.H + kvh * p.G;
          mbar_arrive_expect_tx(q_full, 2 * q_rows * 128);
          tma_load_2d(smem + Smem::off_q, &tmap_q, q_full, 0, q_row);
          tma_load_2d(smem + Smem::off_q + Smem::kHalf, &tmap_q, q_full, 64, q_row);
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
      chain.add(p, range, lane, cur.t, kvh, range.end - cur.left, cur.first, cur.steps, cur.row.steps);
      uint32_t mask = 0, live = 0;                            // of this lane's unit
      const int units = cur.steps * kSub;
      for (int unit = 0; unit < units;) {
        const int in_look = unit & (look.batch(p) - 1);
        if (in_look == 0) {
          look.next(p, lane);
          live = look.hi > look.lo;
          mask = live ? ((2u << (look.hi - 1)) - (1u << look.lo)) << look.within(p, lane) : 0u;
          for (int off = 1; off < per_unit; off <<= 1) {
            mask |= __shfl_xor_sync(0xffffffffu, mask, off);
            live += __shfl_xor_sync(0xffffffffu, live, off);
          }
        }
        const int count = min(min(4, look.batch(p) - in_look), units - unit);
        const int mine = (lane / per_unit) - in_look;         // this lane's unit of the round
        bool todo = mine >= 0 && mine < count;
        const uint32_t my_unit = g + (todo ? mine : 0);
        const uint32_t tile = my_unit / kSub, sub = my_unit % kSub;
        // where the unit's keys and values go: tiles, or two staging slots
        uint64_t *kf, *vf, *ke, *ve;
        uint8_t *kd, *vd;
        uint32_t kp, vp;
        if constexpr (kFp8) {
          const uint32_t c = 2 * tile, ks = c % Smem::kSlots, vs = (c + 1) % Smem::kSlots;
          kf = slot_full + ks;
          vf = slot_full + vs;
          ke = slot_empty + ks;
          ve = slot_empty + vs;
          kp = (c / Smem::kSlots) & 1u;
          vp = ((c + 1) / Smem::kSlots) & 1u;
          kd = smem + Smem::off_slot + ks * Smem::kSlotBytes;
          vd = smem + Smem::off_slot + vs * Smem::kSlotBytes;
        } else {
          const uint32_t st = tile % kKStages;
          kf = k_full + st;
          vf = v_full + st;
          ke = k_empty + st;
          ve = v_empty + st;
          kp = vp = (tile / kKStages) & 1u;
          kd = smem + Smem::off_k + st * Smem::kTileBytes;
          vd = smem + Smem::off_v + st * Smem::kTileBytes;
        }
        const int head = lane & ~(per_unit - 1);
        PaPatience patience;
        while (ok) {
          const uint32_t free_heads =
              __ballot_sync(0xffffffffu, todo && lane == head && mbar_test_wait(ke, kp ^ 1u) &&
                                             mbar_test_wait(ve, vp ^ 1u));
          const bool go = todo && (free_heads >> head & 1u);
          if (go && lane == head) {
            masks[tile % Smem::kMasks * kSub + sub] = mask;
            const uint32_t bytes = live * (gran * (kFp8 ? 128 : 256));
            mbar_arrive_expect_tx(kf, bytes);
            mbar_arrive_expect_tx(vf, bytes);
          }
          __syncwarp();
          if (go && look.hi > look.lo) {
            const int at = (sub * kPwUnit + look.within(p, lane)) * 128;
#pragma unroll
            for (int b = 0; b < (kFp8 ? 1 : 2); ++b) {
              tma_load_5d(kd + b * Smem::kHalf + at, &tmap_k, kf, 0, look.slot, b, kvh, look.page);
              tma_load_5d(vd + b * Smem::kHalf + at, &tmap_v, vf, 0, look.slot, b, kvh, look.page);
            }
          }
          if constexpr (kFp8) {
            // the scales of the units that just went, a lane a slot
            for (uint32_t left = free_heads; left != 0; left &= left - 1) {
              const int h = __ffs(left) - 1;
              const uint32_t unit_no = __shfl_sync(0xffffffffu, my_unit, h);
              const bool keep = __shfl_sync(0xffffffffu, mask, h) >> lane & 1u;
              const int pg = __shfl_sync(0xffffffffu, look.page, h + (lane >> p.gran_shift));
              const int sl = __shfl_sync(0xffffffffu, look.slot, h + (lane >> p.gran_shift));
              const int64_t o = keep ? (pg * p.g.page_stride +
                                        static_cast<int64_t>(sl + (lane & (gran - 1))) * p.g.slot_stride +
                                        kvh * p.g.head_stride) / 32
                                     : 0;
              const uint32_t c = 2 * (unit_no / kSub), row = unit_no % kSub * kPwUnit + lane;
              uint32_t *const sc = reinterpret_cast<uint32_t *>(smem + Smem::off_scale);
              const uint32_t ks = c % Smem::kSlots, vs = (c + 1) % Smem::kSlots;
              cp_async4_zfill(sc + ks * kPwTile + row, p.k_scale + o, keep ? 4u : 0u);
              cp_async_mbar_arrive_noinc(slot_full + ks);
              cp_async4_zfill(sc + vs * kPwTile + row, p.v_scale + o, keep ? 4u : 0u);
              cp_async_mbar_arrive_noinc(slot_full + vs);
            }
          }
          round |= free_heads;
          todo = todo && !go;
          if (!__any_sync(0xffffffffu, todo)) break;
          ok = patience.more(ctl, 71);
        }
        if (!ok) break;
        round = 0;
        g += count;
        unit += count;
      }
      if (!ok) break;
      cur.advance(p);
    }
    chain.finish(p, lane);
    // every copy started here lands before the CTA can exit: the last tiles'
    // barriers. (Where a wait was given up inside a tile its barriers lack the
    // arrivals of the units that never started; they are made here.)
    if constexpr (kFp8) cp_async_wait<0>();
    __syncwarp();
    const uint32_t started = g + __popc(round);
    if (lane == 0) {
      auto barrier = [&](uint32_t c, uint32_t &phase) -> uint64_t * {
        if constexpr (kFp8) {
          phase = (c / Smem::kSlots) & 1u;
          return slot_full + c % Smem::kSlots;
        } else {
          phase = (c / 2 / kKStages) & 1u;
          return (c & 1u ? v_full : k_full) + c / 2 % kKStages;
        }
      };
      const uint32_t loads = 2 * ((started + kSub - 1) / kSub);          // keys and values of a tile
      uint32_t phase;
      for (uint32_t u = started; u % kSub != 0; ++u)
        for (uint32_t c = loads - 2; c < loads; ++c)
          for (int i = 0; i < (kFp8 ? 33 : 1); ++i) mbar_arrive(barrier(c, phase));
      constexpr uint32_t kLast = kFp8 ? Smem::kSlots : 2 * kKStages;
      for (uint32_t c = loads > kLast ? loads - kLast : 0; c < loads; ++c) {
        uint64_t *const bar = barrier(c, phase);
        mbar_drain(bar, phase, p.drain_limit_ns);
      }
      if (!published && n_items > 0) mbar_drain(q_full, (n_items - 1) & 1u, p.drain_limit_ns);
    }
    __syncwarp();
  } else if (warp == kPwMmaWarp) {
    // ---------------- products ----------------
    const uint32_t idesc_s = idesc_bf16_f32(128, kPwTile);
    const uint32_t idesc_o = idesc_bf16_f32_bmn(128, kRowD);
    const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(smem + Smem::off_q));
    uint64_t *last_commit = nullptr;
    uint32_t last_phase = 0;
    uint32_t g = 0;                                           // tiles before this item
    bool ok = true;
    // O += P V of tile `t` (global number); fresh: its stream's first of the item
    auto pv = [&](uint32_t t, bool fresh, uint32_t n) -> bool {
      const uint32_t sb = t & 1u, st = t % kVStages;
      if (!pa_wait(p_full + sb, (t >> 1) & 1u, ctl, 72) ||
          !pa_wait(v_full + st, (t / kVStages) & 1u, ctl, 73) ||
          (fresh && n > 0 && !pa_wait(o_free, (n - 1) & 1u, ctl, 74)))
        return false;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t v_base = smem_u32(smem + Smem::off_v + st * Smem::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < kPwTile / 16; ++kk)
          // V: 16 slots = two 8-row atoms further along K; the halves of D apart
          mma_f16_ts(tmem + 256 + sb * 128, tmem + sb * 128 + kk * 8,
                     sdesc_mnmajor_sw128(v_base + kk * 2048, Smem::kHalf, 1024), idesc_o,
                     fresh && kk == 0 ? 0u : 1u);
        mma_commit(pv_done + sb);
        mma_commit(v_empty + st);
        last_commit = pv_done + sb;
        last_phase = (t >> 1) & 1u;
      }
      __syncwarp();
      return true;
    };
    for (uint32_t n = 0; ok; ++n) {
      if (!pa_wait(q_full, n & 1u, ctl, 75)) break;
      const PaItem it = *info;
      if (it.row < 0) break;
      tc_fence_after_sync();
      for (int i = 0; i < it.steps; ++i) {
        const uint32_t t = g + i, sb = t & 1u, st = t % kKStages;
        // S's buffer is free: P V of tile t - 2, which reads P there, was
        // issued before and products run in order
        if (!pa_wait(k_full + st, (t / kKStages) & 1u, ctl, 76)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (lane == 0) {
          const uint64_t k_desc = sdesc_kmajor_sw128(smem_u32(smem + Smem::off_k + st * Smem::kTileBytes));
#pragma unroll
          for (int kk = 0; kk < kRowD / 16; ++kk) {
            const uint32_t off = (kk / 4) * (Smem::kHalf >> 4) + (kk % 4) * 2;
            mma_f16_ss(tmem + sb * 128, q_desc + off, k_desc + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(s_full + sb);
          mma_commit(k_empty + st);
          if (i == it.steps - 1) mma_commit(q_empty);
          last_commit = s_full + sb;
          last_phase = (t >> 1) & 1u;
        }
        __syncwarp();
        if (i >= 1 && !pv(t - 1, i <= 2, n)) {
          ok = false;
          break;
        }
      }
      if (!ok || !pv(g + it.steps - 1, it.steps <= 2, n)) break;
      if (lane == 0) mma_commit(item_done);
      __syncwarp();
      g += it.steps;
    }
    if (lane == 0 && last_commit) mbar_drain(last_commit, last_phase, p.drain_limit_ns);
    __syncwarp();
  } else {
    // ---------------- softmax and epilogue: a thread a row ----------------
    const int stream = warp >> 2, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + stream * 128, t_o = tmem + lane_base + 256 + stream * 128;
    float2 *const ml = reinterpret_cast<float2 *>(smem + Smem::off_ml);
    const float neg_inf = __int_as_float(0xff800000);
    const bool mine = r < p.G;                                // rows past G hold no head
    const bool warp_rows = (warp & 3) * 32 < p.G;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!pa_wait(q_full, n & 1u, ctl, 77)) break;
      const PaItem it = *info;
      if (it.row < 0) break;
      pa_release(q_empty, lane);
      // (the maximum unscaled until the item's end, as in the other kernel)
      float m = neg_inf, mb = 0.f, lazy = neg_inf, sum = 0.f;
      bool first = true;
      for (int i = (stream ^ g) & 1; i < it.steps; i += 2) {
        const uint32_t t = g + i, st = t % kVStages, mt = t % Smem::kMasks * kSub;
        // (bf16: V's tile too, for the rows zeroed below)
        if (!pa_wait(s_full + stream, (t >> 1) & 1u, ctl, 78) ||
            (!kFp8 && !pa_wait(v_full + st, (t / kVStages) & 1u, ctl, 79))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t mw[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) mw[w] = masks[mt + w];
        const bool every = (mw[0] & mw[1] & mw[2] & mw[3]) == 0xffffffffu;
        if (!kFp8 && !every && !(masks[mt + (r >> 5)] >> (r & 31) & 1u)) {
          // a value row that is not kept: its weight is 0, and 0 times
          // whatever is there has to be 0
          uint8_t *const row = smem + Smem::off_v + st * Smem::kTileBytes + r * 128;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4 *>(row + (c >> 3) * Smem::kHalf + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (warp_rows) {
          // S is read twice, 32 logits at a time: for the maximum, and once O is
          // on the right reference for P, which takes S's place as packed
          // pairs (columns already read)
          // (the next 32 on their way meanwhile)
          float v[2][32];
          auto ahead = [&](int q4) { tmem_ld32_async(t_s + 32 * q4, v[q4 & 1]); };
          const bool down_scale = p.scale_log2 < 0.f;
          float m4[4] = {neg_inf, neg_inf, neg_inf, neg_inf};
          ahead(0);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            float (&x)[32] = v[q4 & 1];
            tmem_wait_ld32(x);
            if (q4 < 3) ahead(q4 + 1);
            if (!every || down_scale) {
              // masked logits out; a negative scale turns the order around
#pragma unroll
              for (int c = 0; c < 32; ++c)
                x[c] = mw[q4] >> c & 1u ? (down_scale ? -x[c] : x[c]) : neg_inf;
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) m4[c & 3] = fmaxf(m4[c & 3], x[c]);
          }
          ahead(0);                                           // for the second reading
          const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // the row's largest logit before its scaling (-inf: nothing is kept)
          const float mx = down_scale ? -top : top;
          const bool grow = mine && top != neg_inf && (mx - mb) * p.scale_log2 > lazy;
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mx : mb;                  // the row's new reference
            const float a = !grow ? 1.f : m == neg_inf ? 0.f : ex2_approx((m - mn) * p.scale_log2);
            if (!first) {
              // O holds the stream's earlier tiles: their P V ended before this
              // tile's S, which products issued in order
              tmem_wait_ld32(v[0]);
              float (&o)[32] = v[1];
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                tmem_ld32_wait(t_o + 32 * q4, o);
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] *= a;
                tmem_st32(t_o + 32 * q4, o);
              }
              tmem_wait_st();
            }
            sum *= a;
            if (grow) {
              m = mb = mn;
              lazy = kPaLazy;
            }
          }
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            float pk[16];
            float (&x)[32] = v[q4 & 1];
            tmem_wait_ld32(x);
            if (q4 < 3) ahead(q4 + 1);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 y = fmul2(fadd2(make_float2(x[c], x[c + 1]), make_float2(-mb, -mb)),
                                     make_float2(p.scale_log2, p.scale_log2));
              x[c] = y.x;
              x[c + 1] = y.y;
            }
            if (!every) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(mw[q4] >> c & 1u)) x[c] = neg_inf;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float e0 = ex2_approx(x[2 * c]), e1 = ex2_approx(x[2 * c + 1]);
              s4[c & 3] += e0 + e1;
              pk[c] = __uint_as_float(pack_bf16x2(e0, e1));
            }
            // columns 16 q4 .. + 15: their logits have been read twice
            tmem_st16(t_s + 16 * q4, pk);
          }
          sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          tmem_wait_st();
        }
        first = false;
        fence_proxy_async_smem();                             // zeroed value rows
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + stream);
      }
      if (!ok) break;
      // in log2 units from here on; all kept logits NaN: not an empty row
      if (m != neg_inf) m *= p.scale_log2;
      else if (sum != 0.f) m = 0.f;
      // ---- add the two streams up: this one writes half of the features ----
      // (once everyone has read the last item's maxima and sums)
      if (n > 0 && !pa_wait(o_free, (n - 1) & 1u, ctl, 83)) break;
      ml[stream * kPwRows + r] = make_float2(m, sum);
      if (!(p.selftest_stall && warp == 0)) pa_release(ml_full, lane);
      if (!pa_wait(ml_full, n & 1u, ctl, 81) || !pa_wait(item_done, n & 1u, ctl, 82)) break;
      tc_fence_after_sync();
      if (warp_rows) {
        const float2 x0 = ml[r], x1 = ml[kPwRows + r];
        const float M = fmaxf(x0.x, x1.x);
        const bool any0 = x0.x != neg_inf, any1 = x1.x != neg_inf;
        const float a0 = any0 ? ex2_approx(x0.x - M) : 0.f, a1 = any1 ? ex2_approx(x1.x - M) : 0.f;
        const float L = a0 * x0.y + a1 * x1.y;
        const int64_t row = it.slot < 0 ? static_cast<int64_t>(it.row) * p.H + it.item * p.G + r
                                        : (static_cast<int64_t>(blockIdx.x) * 2 + it.slot) * kPwRows + r;
        float inv = 1.f;
        if (it.slot < 0) {
          float den = L;
          if (mine && p.sinks && M != neg_inf)
            den += ex2_approx(__ldg(p.sinks + it.item * p.G + r) * kPaLog2e - M);
          inv = M == neg_inf ? 0.f : 1.f / den;
          if (mine && stream == 0 && p.lse) p.lse[row] = M == neg_inf ? neg_inf : (M + log2f(L)) * kPaLn2;
        } else if (mine && stream == 0) {
          p.part_ml[row] = make_float2(M, L);
        }
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          const int c0 = 64 * stream + 32 * q2;
          float o0[32], o1[32];
          __syncwarp();
          tmem_ld32_wait(tmem + lane_base + 256 + c0, o0);
          tmem_ld32_wait(tmem + lane_base + 384 + c0, o1);
          // a stream without a tile (or a kept slot) left no O of this item
#pragma unroll
          for (int c = 0; c < 32; ++c)
            o0[c] = ((any0 ? a0 * o0[c] : 0.f) + (any1 ? a1 * o1[c] : 0.f)) * inv;
          if (!mine) {
          } else if (it.slot < 0) {
            uint4 *const dst = reinterpret_cast<uint4 *>(p.out + row * kRowD + c0);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              dst[c] = make_uint4(pack_bf16x2(o0[8 * c], o0[8 * c + 1]), pack_bf16x2(o0[8 * c + 2], o0[8 * c + 3]),
                                  pack_bf16x2(o0[8 * c + 4], o0[8 * c + 5]),
                                  pack_bf16x2(o0[8 * c + 6], o0[8 * c + 7]));
          } else {
            float *const dst = p.part_o + row * kRowD + c0;
#pragma unroll
            for (int c = 0; c < 4; ++c) st_global_v8(dst + 8 * c, &o0[8 * c]);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      g += it.steps;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kPwMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace dsa
