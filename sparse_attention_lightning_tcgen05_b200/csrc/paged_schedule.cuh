// paged_schedule.cuh -- what the kernels that attend over a paged cache share:
// the slots a query token keeps, the order of the work items and a CTA's even
// share of them, the page lookups ahead of the loads, and the pipeline's
// waits.
//
// A work item is a token, a key-value head and a tile of its query heads; it
// takes the token's kept slots in steps of kStep. All items' steps in a row are
// cut into equal ranges, one a CTA, so that rows of any lengths fill the GPU;
// an item cut by a border leaves partial results that a second kernel joins.
#pragma once

#include <cstdint>

#include "paged_cache.cuh"
#include "paged_rows.h"
#include "sm100_ptx.cuh"

namespace dsa {

constexpr float kPaLazy = 8.f;                     // log2 units: rescale when a logit passes the maximum by more
constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PagedAttnParams {
  PagedGeom g;
  int T, H, G;
  int head_tiles;              // work items a key-value head, of `rows` query heads each
  int rows;
  int window;
  int block_shift, num_blocks, block_heads;
  int gran_shift;              // log2 of the slots one lookup and one box cover
  int list_steps;              // steps that the listed blocks take
  float scale_log2;
  const uint8_t *k_scale, *v_scale;
  const float *sinks;
  const int *positions, *seq_ids, *blocks;
  uint16_t *out;
  float *lse;
  float *part_o;               // [grid, 2, rows, D] unnormalised
  float2 *part_ml;             // [grid, 2, rows] (max in log2 units, sum)
  int4 *chain;                 // items that several CTAs share (PaChain)
  bool chain_by_item;          // an entry an item, else one a CTA
  int ctas;                    // of the attention kernel
  bool selftest_stall;         // warp 0's results never reach the others
  unsigned int *err, *err_info;
  uint64_t wait_limit_ns, drain_limit_ns;
};

// The items' order is (key-value head, token, tile of query heads): neighbouring
// CTAs are at tokens of one sequence and one head, which read the same slots. All
// heads pass at the same time, each in its share of the CTAs, so that L2 holds what
// their tokens read of all of them.

// A CTA's range of all items' steps, [begin, end) of `total`, one of `ctas` that
// have any; and the key-value head it starts in.
struct PaRange {
  int64_t begin, end, total, ctas;
  int kvh;
};

// The entries that tell the join kernel which items several CTAs share, written
// by the CTA in which an item begins: (row, item of the row, first and last
// CTA), row -1 for an item that lies in one CTA. By item where there are no
// more of them than CTAs, else by CTA: one, since only its last item can go on.
struct PaChain {
  int4 mine = {-1, 0, 0, 0};

  // an item of which this CTA has `steps` of `of` steps from `first` on, the
  // first of them number `at` of all
  __device__ __forceinline__ void add(const PagedAttnParams &p, const PaRange &range, int lane, int row,
                                      int id, int64_t at, int first, int steps, int of) {
    if (first != 0) return;
    int4 e = {-1, 0, 0, 0};
    if (steps < of)
      e = make_int4(row, id, static_cast<int>(blockIdx.x),
                    static_cast<int>(((at + of) * range.ctas - 1) / range.total));
    if (p.chain_by_item) {
      if (lane == 0) p.chain[static_cast<int64_t>(row) * p.g.H_kv * p.head_tiles + id] = e;
    } else {
      mine = e;
    }
  }
  __device__ __forceinline__ void finish(const PagedAttnParams &p, int lane) const {
    if (!p.chain_by_item && lane == 0) p.chain[blockIdx.x] = mine;
  }
};

template <bool kList, int kStep>
__device__ __forceinline__ PaRow pa_row_of(const PagedAttnParams &p, int seq, int at) {
  return pa_row_at(p.g.capacity(), p.g.num_seqs, p.window, kList, p.list_steps, kStep, seq, at);
}

template <bool kList, int kStep>
__device__ __forceinline__ PaRow pa_row(const PagedAttnParams &p, int t) {
  return pa_row_of<kList, kStep>(p, p.seq_ids ? __ldg(p.seq_ids + t) : t, __ldg(p.positions + t));
}

// A place in a CTA's range of steps: an item and this CTA's steps of it. The
// next row's position is loaded one row ahead.
template <bool kList, int kStep>
struct PaCursor {
  int kvh, t, item;            // key-value head, token, tile
  int first, steps;            // 0 steps: the range is over
  int64_t left;                // steps to the range's end, this item's among them
  PaRow row;
  int next_seq, next_pos;

  __device__ __forceinline__ void fetch(const PagedAttnParams &p) {
    const int n = t + 1 < p.T ? t + 1 : 0;
    next_seq = p.seq_ids ? __ldg(p.seq_ids + n) : n;
    next_pos = __ldg(p.positions + n);
  }
  // `offset` steps into row t of head `kvh`, for `count` steps
  __device__ __forceinline__ void start(const PagedAttnParams &p, int kvh_, int t_, int64_t offset,
                                        int64_t count) {
    kvh = kvh_;
    t = t_;
    row = pa_row<kList, kStep>(p, t);
    fetch(p);
    item = static_cast<int>(offset / row.steps);
    first = static_cast<int>(offset % row.steps);
    left = count;
    steps = static_cast<int>(min(static_cast<int64_t>(row.steps - first), left));
  }
  __device__ __forceinline__ void advance(const PagedAttnParams &p) {
    left -= steps;
    first = 0;
    if (left > 0 && ++item == p.head_tiles) {
      item = 0;
      if (++t == p.T) {
        t = 0;
        ++kvh;
      }
      row = pa_row_of<kList, kStep>(p, next_seq, next_pos);
      fetch(p);
    }
    steps = static_cast<int>(min(static_cast<int64_t>(row.steps), left));
  }
  // of the row's H_kv * head_tiles items
  __device__ __forceinline__ int id(const PagedAttnParams &p) const {
    return kvh * p.head_tiles + item;
  }
};

// Looks up the granules (2^gran_shift slots of one page) of a CTA's steps, 32
// at a time, a lane each, in the order the producer loads them: a step is
// kStep / kUnit units of kUnit slots, a unit kUnit >> gran_shift granules. The
// entries of a block list are read two batches ahead and the pages one, so
// that no lookup waits for memory.
template <bool kList, int kStep, int kUnit>
struct PaLookup {
  static constexpr int kSub = kStep / kUnit;
  static constexpr int kUnitShift = kUnit == 16 ? 4 : 5;
  static_assert(kUnit == 1 << kUnitShift, "a unit is 16 or 32 slots");
  PaCursor<kList, kStep> cur;
  int sub;                     // the batch's first unit of the item
  // first level: this lane's list entry and what it belongs to
  PaRow e_row;
  int e_unit, e_block;         // unit in the item's row (-1: none)
  // second level: the page as the table has it
  int t_page, t_slot, t_lo, t_hi;
  // looked up: page, slot in the page, and which of the granule's slots are
  // kept (none: lo >= hi)
  int page, slot;
  uint32_t lo, hi;

  // granules a unit, and units a batch
  static __device__ __forceinline__ int per_unit(const PagedAttnParams &p) {
    return kUnit >> p.gran_shift;
  }
  static __device__ __forceinline__ int batch(const PagedAttnParams &p) {
    return 32 >> (kUnitShift - p.gran_shift);
  }
  static __device__ __forceinline__ int within(const PagedAttnParams &p, int lane) {
    return (lane & (per_unit(p) - 1)) << p.gran_shift;
  }
  __device__ __forceinline__ void load_list(const PagedAttnParams &p, int lane) {
    const int u = sub + (lane >> (kUnitShift - p.gran_shift));
    e_row = cur.row;
    e_unit = u < cur.steps * kSub ? cur.first * kSub + u : -1;
    e_block = -1;
    if (kList && e_unit >= 0 && e_unit < p.list_steps * kSub) {
      const int e = (e_unit * kUnit + within(p, lane)) >> p.block_shift;
      const int list = cur.t * p.block_heads + (p.block_heads > 1 ? cur.kvh : 0);
      if (e < p.num_blocks) e_block = __ldg(p.blocks + static_cast<int64_t>(list) * p.num_blocks + e);
    }
    sub += batch(p);
    if (sub >= cur.steps * kSub && cur.steps > 0) {
      cur.advance(p);
      sub = 0;
    }
  }
  __device__ __forceinline__ void load_page(const PagedAttnParams &p, int lane) {
    const int64_t gran = 1 << p.gran_shift;
    int64_t s = 0, l = 0, h = 0;
    if (kList && e_unit < p.list_steps * kSub) {
      if (e_block >= 0) {
        // slots before the recent ones; e_row.lo lies in the table
        s = (static_cast<int64_t>(e_block) << p.block_shift) +
            ((e_unit * kUnit + within(p, lane)) & ((1 << p.block_shift) - 1));
        h = max(int64_t{0}, min(gran, e_row.lo - s));
      }
    } else if (e_unit >= 0) {
      s = e_row.wbase + static_cast<int64_t>(kList ? e_unit - p.list_steps * kSub : e_unit) * kUnit +
          within(p, lane);
      l = max(int64_t{0}, min(gran, e_row.lo - s));
      h = max(int64_t{0}, min(gran, e_row.last + 1 - s));
    }
    t_lo = static_cast<int>(l);
    t_hi = static_cast<int>(max(l, h));
    t_page = -1;
    t_slot = static_cast<int>(s & ((int64_t{1} << p.g.page_shift) - 1));
    if (h > l)
      t_page = __ldg(p.g.table + static_cast<int64_t>(e_row.seq) * p.g.pages_per_seq +
                     (s >> p.g.page_shift));
  }
  __device__ __forceinline__ void start(const PagedAttnParams &p, int lane,
                                        const PaCursor<kList, kStep> &from) {
    cur = from;
    sub = 0;
    load_list(p, lane);
    load_page(p, lane);
    load_list(p, lane);
  }
  __device__ __forceinline__ void next(const PagedAttnParams &p, int lane) {
    page = t_page;
    slot = t_slot;
    lo = t_lo;
    hi = page < 0 || page >= p.g.num_pages ? t_lo : t_hi;
    load_page(p, lane);
    load_list(p, lane);
  }
};

// Called by all kThreads threads. `least`: steps below which a CTA is not worth
// its part of the join.
template <bool kList, int kStep, int kThreads>
__device__ __forceinline__ PaRange pa_range(const PagedAttnParams &p, int least, int tid, int64_t *scan,
                                            int *start_row, int64_t *start_step) {
  constexpr int kWarps = kThreads / 32;
  const int lane = tid & 31, warp = tid >> 5;
  const int inner = p.head_tiles;
  const int per = (p.T + kThreads - 1) / kThreads;
  const int ra = min(p.T, tid * per), rb = min(p.T, ra + per);
  int64_t mine = 0;
  for (int t = ra; t < rb; ++t) mine += pa_row<kList, kStep>(p, t).steps;
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, group = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    group += scan[w];
  }
  group *= inner;
  PaRange r;
  r.total = group * p.g.H_kv;
  // no more CTAs than get `least` steps, and the working ones are the first
  // ones, so that an item's CTAs follow one another
  r.ctas = min(static_cast<int64_t>(gridDim.x), (r.total + least - 1) / least);
  const bool in = blockIdx.x < r.ctas;
  r.begin = in ? r.total * blockIdx.x / r.ctas : r.total;
  r.end = in ? r.total * (blockIdx.x + 1) / r.ctas : r.total;
  r.kvh = in ? static_cast<int>(r.begin / group) : 0;
  const int64_t at = r.begin - r.kvh * group;
  const int64_t excl = (before + incl - mine) * inner;
  if (r.begin < r.end && at >= excl && at < (before + incl) * inner) {
    int64_t x = excl;
    for (int t = ra; t < rb; ++t) {
      const int64_t n = static_cast<int64_t>(pa_row<kList, kStep>(p, t).steps) * inner;
      if (at < x + n) {
        *start_row = t;
        *start_step = at - x;
        break;
      }
      x += n;
    }
  }
  __syncthreads();
  return r;
}

// A whole warp's bounded wait, whose fast path is one instruction (see
// mbar_wait). The vote brings the lanes together again, as the warp-wide
// instructions that follow need, and gives all of them one answer.
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, const WaitCtl &ctl,
                                        uint32_t site) {
  const bool ok = mbar_try_wait(bar, parity) || mbar_wait(bar, parity, ctl, site);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The bound of a warp's polling loop: false (after recording the timeout and
// raising the CTA's abort flag) once it outlives ctl.limit_ns or another role
// has aborted. The time is looked at every 64 polls.
struct PaPatience {
  uint64_t t0 = 0;
  uint32_t polls = 0;
  __device__ __forceinline__ bool more(const WaitCtl &ctl, uint32_t site) {
    if ((++polls & 63u) != 0) return true;
    bool on = !*ctl.abort;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (on && (now - t0 > ctl.limit_ns || polls >= 1u << 30)) {
      *ctl.abort = 1;
      if (atomicCAS(ctl.err, 0u, kStatusTimeout) == 0u) atomicExch(ctl.err_info, site);
      on = false;
    }
    return __all_sync(0xffffffffu, on);
  }
};

// A warp gives shared memory that it has read back to TMA: its reads (generic
// proxy) come before the loads (async proxy) that the arrival lets start.
// Without the fence, reads issued last were seen to return the next load's
// data.
__device__ __forceinline__ void pa_release(uint64_t *bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3,
                                            int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3), "r"(c4)
      : "memory");
}

}  // namespace dsa
