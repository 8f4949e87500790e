// Shared-prefix decode (pad_decode_shared): partial softmax over the units of
// the work line (pad_shared.h), then one merge of each query row's partials.
//
// Per unit and row, over the unit's tokens:  m = max s, l = sum 2^(s - m),
//   o = sum 2^(s - m) v / l,  lse2 = m + log2 l   (s = scale * log2(e) * q.k)
// and per row over its units:  out = sum 2^(lse2_u - lse2) o_u.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pad_device.cuh"
#include "pad_shared.h"
#include "pad_shared_walk.cuh"
#include "pad_tc.cuh"

namespace pad {
namespace {

// One warp per query row, one token at a time: the definition, as a kernel.
template <int D, bool F8>
__global__ void __launch_bounds__(256) shared_kernel(const __grid_constant__ SharedParams p) {
  constexpr int VEC = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  shared_walk<D>(p, blockIdx.x, blockIdx.x == 0 && warp == 0 ? p.cum : nullptr, [&](const SharedUnit &u) {
    for (int r = warp; r < u.rows; r += 8) {
      const int b = u.b0 + r / p.gt, j = r % p.gt;
      if (j >= u.heads) continue;
      const int h = u.kvh * p.g + u.ht * p.gt + j;
      float qv[VEC], acc[VEC], m = -INFINITY, l = 0.f;
      for (int i = 0; i < VEC; ++i) {
        qv[i] = __uint_as_float((uint32_t)p.q[b * p.q_sb + (int64_t)h * p.q_sh + lane * VEC + i] << 16) * p.scale_log2;
        acc[i] = 0.f;
      }
      for (int t = u.tok0; t < u.tok1; ++t) {
        const int pg = t >> p.bs_log2, slot = t & ((1 << p.bs_log2) - 1);
        const int id = pg < p.n_shared ? p.shared_table[pg] : p.tables[b * p.table_stride + pg];
        const bool ok = (unsigned)id < (unsigned)p.num_blocks;
        if (!ok && lane == 0) atomicOr(p.err, kErrBlockId);
        const int64_t ko = id * p.k_sblk + u.kvh * p.k_sh + slot * p.k_ss + lane * VEC;
        const int64_t vo = id * p.v_sblk + u.kvh * p.v_sh + slot * p.v_ss + lane * VEC;
        auto at = [&](const void *c, int64_t o) -> float {
          if (!ok) return 0.f;
          if constexpr (F8) {
            const uint32_t h2 = e4m3x2_to_f16x2(static_cast<const uint8_t *>(c)[o]);
            return __half2float(__ushort_as_half((unsigned short)h2));
          } else {
            return __uint_as_float((uint32_t)static_cast<const uint16_t *>(c)[o] << 16);
          }
        };
        float s = 0.f;
        for (int i = 0; i < VEC; ++i) s += qv[i] * at(p.k, ko + i);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - ref), w = exp2f(s - ref);
        m = mn;
        l = l * a + w;
        for (int i = 0; i < VEC; ++i) acc[i] = acc[i] * a + w * at(p.v, vo + i);
      }
      const int64_t row = u.part + r;
      for (int i = 0; i < VEC; ++i) p.o_part[row * D + lane * VEC + i] = acc[i] / l;
      if (lane == 0) {
        p.lse_part[row] = m + log2f(l);
        if (shared_part_rows(u.rows, D) != u.rows) p.lse_part[row + u.rows] = -INFINITY;
      }
    }
  });
}

// ---- the partial kernel -------------------------------------------------------
//
// One persistent CTA per SM, warp-specialised; every role goes through the CTA's
// units in order, each as far ahead as its buffers let it:
//
//   schedule warp   walks the work line and puts units into a queue of kQueue
//   copy warps      TMA of the unit's q rows and K chunks into one ring, and of its V
//                   chunks into another, boxes of one 128-byte column block x one page
//                   (or a chunk's worth of a larger page)
//   MMA warp        S = Q . K^T  (128 rows x chunk) into one of two S buffers, then
//                   O += P . V  with P read from tensor memory
//   softmax warps   two threads per row, half a chunk's columns each: scores out of
//                   tensor memory, running maximum and sum, P back over the scores
//
// A step is (query tile, chunk): S buffer of a step = its parity, so one step's
// softmax runs under the other's products.  A two-tile unit takes both tiles
// through each chunk; a one-tile unit alternates its even and odd chunks between
// the two accumulators, which leave two partials per row.  At D = 256 there is one
// accumulator (256 of the 512 columns), one softmax group, and still two S buffers.
//
// The P of a step overlays its S: PV(j) is issued before QK(j + 2), and the tensor
// core runs one thread's products in order, so a QK never overwrites a P that is
// still to be read.
template <int D>
struct SharedCfg {
  static constexpr int CT = shared_chunk(D), NACC = shared_accs(D), CB = D / 64;
  static constexpr int QR = shared_rows(D);
  static constexpr uint32_t kSlot = CT * D * 2;         // bytes of a K or V chunk
  static constexpr uint32_t kBlock = CT * 128;          // one column block of it
  static constexpr uint32_t kQBlock = QR * 128;         // one column block of q
  static constexpr uint32_t kQ = CB * kQBlock;
  // Ring slots: what is left beside q.  V's slots are held longer, from the copy
  // to the value product two steps behind the score product.
  static constexpr int NK = D == 64 ? 4 : 2, NV = D == 64 ? 4 : 3, NS = NK + NV;
  static constexpr int kQueue = 4;
  static constexpr int kGroupWarps = 8;                 // a softmax group: 4 x 32 rows, two halves of the columns
  static constexpr int kSoftmaxWarps = kGroupWarps * NACC;
  static constexpr int kCopyKWarp = kSoftmaxWarps, kCopyVWarp = kSoftmaxWarps + 1, kMmaWarp = kSoftmaxWarps + 2,
                       kScheduleWarp = kSoftmaxWarps + 3;
  static constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
  static constexpr uint32_t ring = kQ, queue = ring + NS * kSlot, bars = queue + kQueue * 64;
  static constexpr uint32_t total = bars + 512 + 1024 /* alignment slack */;
  static constexpr uint32_t kSCol = 128, kOCol = 256;   // S buffers at 0 and 128, O behind them
};
static_assert(sizeof(SharedUnit) <= 64, "queue entry");

template <int D>
__global__ void __launch_bounds__(SharedCfg<D>::kThreads, 1) shared_tc_kernel(const __grid_constant__ SharedParams p) {
  using C = SharedCfg<D>;
  constexpr int CT = C::CT, NACC = C::NACC, NS = C::NS, CB = C::CB;
  static_assert(C::total <= (uint32_t)kSmemBudget, "shared-memory plan over budget");
  static_assert(C::kOCol + NACC * D <= 512, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sq = smem_addr(smem), sring = sq + C::ring;
  SharedUnit *queue = reinterpret_cast<SharedUnit *>(smem + C::queue);  // entries 64 bytes apart
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::bars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t full = bar0, empty = full + 8 * NS, q_full = empty + 8 * NS, q_empty = q_full + 16,
                 s_full = q_empty + 16, p_full = s_full + 16, pv_done = p_full + 16, o_free = pv_done + 16,
                 u_full = o_free + 16, u_empty = u_full + 8 * C::kQueue, idle = u_empty + 8 * C::kQueue;
  constexpr int kBars = 2 * NS + 12 + 2 * C::kQueue + 1;
  static_assert(kBars * 8 + 8 <= 512, "barrier area");
  uint32_t *words = reinterpret_cast<uint32_t *>(bars + kBars);  // [0] tmem, [1] abort
  volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, C::kGroupWarps);
      mbar_init(pv_done + 8 * i, 1);
      mbar_init(o_free + 8 * i, C::kGroupWarps);
    }
    for (int i = 0; i < C::kQueue; ++i) {
      mbar_init(u_full + 8 * i, 1);
      mbar_init(u_empty + 8 * i, C::kSoftmaxWarps + 3);  // every role's warps
    }
    mbar_init(idle, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::alloc(smem_addr(words), 512);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[0], 0);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the merge may come up as CTAs end

  auto wait = [&](uint32_t bar, uint32_t parity, bool drain = false) {
    return tc::wait(bar, parity, p.err, abort_flag, drain);
  };
  // Unit k of the queue, by a whole warp; false: give up.  chunks == 0 ends.
  auto next_unit = [&](int k, SharedUnit &u) -> bool {
    const int e = k % C::kQueue;
    if (!__all_sync(0xffffffffu, wait(u_full + 8 * e, (k / C::kQueue) & 1))) return false;
    u = *reinterpret_cast<const SharedUnit *>(reinterpret_cast<const uint8_t *>(queue) + 64 * e);
    __syncwarp();
    if (lane == 0) tc::arrive(u_empty + 8 * e);
    return true;
  };
  // Half of the q buffer a unit's rows take: both when its box has more than 128
  // rows, else each half in turn (one at D = 256).
  auto q_box_rows = [&](const SharedUnit &u) { return p.gt * (u.rest ? 1 : p.nseq); };

  if (warp == C::kScheduleWarp) {
    int k = 0;
    bool ok = true;
    auto put = [&](const SharedUnit &u) {
      const int e = k % C::kQueue;
      ok = ok && (k < C::kQueue || __all_sync(0xffffffffu, wait(u_empty + 8 * e, (k / C::kQueue - 1) & 1)));
      if (ok && lane == 0) {
        *reinterpret_cast<SharedUnit *>(reinterpret_cast<uint8_t *>(queue) + 64 * e) = u;
        tc::arrive(u_full + 8 * e);
      }
      ++k;
    };
    shared_walk<D>(p, blockIdx.x, blockIdx.x == 0 ? p.cum : nullptr, put);
    SharedUnit end{};
    put(end);
  } else if (warp == C::kCopyKWarp || warp == C::kCopyVWarp) {
    const bool is_k = warp == C::kCopyKWarp;
    const CUtensorMap *map = is_k ? &p.tmk : &p.tmv;
    const int box_log2 = min(p.bs_log2, CT == 128 ? 7 : 6), box = 1 << box_log2, nbox = CT >> box_log2;
    const int slot_mask = (1 << p.bs_log2) - 1;
    const int first_slot = is_k ? 0 : C::NK, slots = is_k ? C::NK : C::NV;
    uint32_t item = 0;               // chunks copied
    uint32_t qn[2] = {0, 0};         // uses of each half of q
    int half = 0;
    bool ok = true;
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      const int32_t *table = u.rest ? p.tables + u.b0 * p.table_stride : p.shared_table;
      // Block of each box of a chunk, box j's in lane j % 32: num_blocks (reads as
      // zeros) behind the unit's tokens and for an id that is not one.  Fetched a
      // chunk ahead, so that the table's latency is not in the copies' way.
      int ids[CT / 32];
      auto fetch = [&](int c) {
#pragma unroll
        for (int w = 0; w < CT / 32; ++w) {
          const int t = u.tok0 + c * CT + ((32 * w + lane) << box_log2);
          ids[w] = p.num_blocks;
          if (32 * w < nbox && 32 * w + lane < nbox && t < u.tok1) {
            const int id = __ldg(table + (t >> p.bs_log2));
            if ((unsigned)id < (unsigned)p.num_blocks) ids[w] = id;
            else atomicOr(p.err, kErrBlockId);
          }
        }
      };
      fetch(0);
      if (is_k) {  // ---- q
        const int box_rows = q_box_rows(u);
        const bool both = NACC == 2 && box_rows > kTileRows;
        const int h = both || NACC == 1 ? 0 : half;
        if (!both && NACC == 2) half ^= 1;
        ok = qn[h] == 0 || __all_sync(0xffffffffu, wait(q_empty + 8 * h, (qn[h] - 1) & 1));
        if (both) ok = ok && (qn[1] == 0 || __all_sync(0xffffffffu, wait(q_empty + 8, (qn[1] - 1) & 1)));
        if (!ok) break;
        if (tc::elect()) {
          mbar_arrive_expect_tx(q_full + 8 * h, (uint32_t)box_rows * 128 * CB);
          if (both) tc::arrive(q_full + 8);
          for (int cb = 0; cb < CB; ++cb)
            tma_load_4d(sq + cb * C::kQBlock + h * (kTileRows * 128), u.rest ? &p.tmqr : &p.tmqp, 0,
                        u.kvh * p.g + u.ht * p.gt, cb, u.b0, q_full + 8 * h);
        }
        __syncwarp();
        ++qn[h];
        if (both) ++qn[1];
      }
      // ---- this warp's chunks
      for (int c = 0; ok && c < u.chunks; ++c) {
        const int slot = first_slot + item % slots;
        if (item >= slots && !__all_sync(0xffffffffu, wait(empty + 8 * slot, (item / slots - 1) & 1))) {
          ok = false;
          break;
        }
        const uint32_t bar = full + 8 * slot, dst = sring + slot * C::kSlot;
        const int tb = u.tok0 + c * CT;
        // V's box that a sequence ends in: row by row, so that the slots behind the
        // sequence are zeros, whatever they hold (a weight of 0 times NaN is NaN)
        const int part = !is_k && u.tok1 < tb + CT && (u.tok1 & (box - 1)) != 0 ? (u.tok1 - tb) >> box_log2 : -1;
        const bool one = tc::elect();
        if (one) mbar_arrive_expect_tx(bar, C::kSlot);
#pragma unroll
        for (int w = 0; w < CT / 32; ++w) {
#pragma unroll 1
          for (int jj = 0; jj < 32 && 32 * w + jj < nbox; ++jj) {
            const int j = 32 * w + jj, id = __shfl_sync(0xffffffffu, ids[w], jj);
            const uint32_t to = dst + ((uint32_t)j << (box_log2 + 7));
            if (j == part) {
              for (int i = 0; i < box; ++i)
                if (one)
#pragma unroll
                  for (int cb = 0; cb < CB; ++cb)
                    tma_load_5d(to + cb * C::kBlock + i * 128, &p.tmv1, 0, (tb + (j << box_log2) + i) & slot_mask, cb,
                                u.kvh, tb + (j << box_log2) + i < u.tok1 ? id : p.num_blocks, bar);
            } else if (one) {
#pragma unroll
              for (int cb = 0; cb < CB; ++cb)
                tma_load_5d(to + cb * C::kBlock, map, 0, (tb + (j << box_log2)) & slot_mask, cb, u.kvh, id, bar);
            }
          }
        }
        __syncwarp();
        ++item;
        if (c + 1 < u.chunks) fetch(c + 1);
      }
    }
    // Leave no copy in flight, whoever gives up: a chunk is copied once its slot's
    // earlier one has been read, so only the last `slots` can be open.
    if (lane == 0) {
      for (uint32_t i = item > (uint32_t)slots ? item - slots : 0; i < item; ++i)
        wait(full + 8 * (first_slot + i % slots), (i / slots) & 1, true);
      for (int h = 0; h < 2; ++h)
        if (qn[h] > 0) wait(q_full + 8 * h, (qn[h] - 1) & 1, true);
    }
  } else if (warp == C::kMmaWarp) {
    constexpr uint32_t IQK = tc::idesc(CT, false, false), IPV = tc::idesc(D, true, false);
    // Two cursors over the CTA's steps, the score product's up to two steps ahead
    // of the value product's (there are two S buffers), across units.
    struct Cursor {
      int k, j, steps, chunks, h;   // next unit of the queue; step of the unit; its q half
      uint32_t item, step;          // chunks and steps of the units before it
      bool two, both;
    };
    Cursor cq{-1, 0, 0, 0, 0, 0, 0, false, false}, cp = cq;
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0}, on[2] = {0, 0};
    int half = 0;
    bool ok = true, more = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    SharedUnit u;
    int queued_steps[2], queued_chunks[2];  // the units between the cursors: at most two, by parity
    bool queued_two[2];
    // The score product's cursor on its next step; false: no unit left (or gave up).
    auto next_qk = [&]() -> bool {
      if (cq.j < cq.steps) return true;
      if (!more) return false;
      cq.item += cq.chunks;
      cq.step += cq.steps;
      ++cq.k;
      ok = next_unit(cq.k, u);
      if (!ok || u.chunks == 0) {
        more = false;
        cq.steps = cq.chunks = cq.j = 0;
        return false;
      }
      cq.two = NACC == 2 && u.rows > kTileRows;
      cq.both = NACC == 2 && q_box_rows(u) > kTileRows;
      cq.h = cq.both || NACC == 1 ? 0 : half;
      if (!cq.both && NACC == 2) half ^= 1;
      cq.chunks = u.chunks;
      cq.steps = cq.two ? 2 * u.chunks : u.chunks;
      cq.j = 0;
      queued_steps[cq.k & 1] = cq.steps;
      queued_chunks[cq.k & 1] = cq.chunks;
      queued_two[cq.k & 1] = cq.two;
      ok = all(wait(q_full + 8 * cq.h, qn[cq.h] & 1)) && (!cq.both || all(wait(q_full + 8, qn[1] & 1)));
      ++qn[cq.h];
      if (cq.both) ++qn[1];
      return ok;
    };
    auto qk = [&]() -> bool {
      const int c = cq.two ? cq.j >> 1 : cq.j, tile = cq.two ? cq.j & 1 : 0, buf = (cq.step + cq.j) & 1;
      const uint32_t it = cq.item + c, slot = it % C::NK;
      if (!all(wait(full + 8 * slot, (it / C::NK) & 1))) return false;
      tc::fence_after();
      const uint64_t qd = tc::smem_desc(sq + (cq.h + tile) * (kTileRows * 128), 16, 1024);
      const uint64_t kd = tc::smem_desc(sring + slot * C::kSlot, 16, 1024);
      if (tc::elect()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(tmem + buf * C::kSCol, qd + (((kk >> 2) * C::kQBlock + (kk & 3) * 32) >> 4),
                     kd + (((kk >> 2) * C::kBlock + (kk & 3) * 32) >> 4), IQK, kk > 0);
        tc::commit(s_full + 8 * buf);
        if (!cq.two || tile == 1) tc::commit(empty + 8 * slot);
        if (cq.j == cq.steps - 1) {
          tc::commit(q_empty + 8 * cq.h);
          if (cq.both) tc::commit(q_empty + 8);
        }
      }
      __syncwarp();
      ++cq.j;
      return true;
    };
    auto pv = [&]() -> bool {
      if (cp.j == cp.steps) {  // on to the next unit, which the other cursor has been given
        cp.item += cp.chunks;
        cp.step += cp.steps;
        ++cp.k;
        cp.steps = queued_steps[cp.k & 1];
        cp.chunks = queued_chunks[cp.k & 1];
        cp.two = queued_two[cp.k & 1];
        cp.j = 0;
      }
      const int c = cp.two ? cp.j >> 1 : cp.j, buf = (cp.step + cp.j) & 1, acc = NACC == 2 ? buf : 0;
      const bool first = cp.j < NACC;
      const uint32_t it = cp.item + c, slot = C::NK + it % C::NV;
      if (first) {  // the last unit's sums have been read
        if (on[acc] > 0 && !all(wait(o_free + 8 * acc, (on[acc] - 1) & 1))) return false;
        ++on[acc];
      }
      if (!all(wait(full + 8 * slot, (it / C::NV) & 1))) return false;
      if (!all(wait(p_full + 8 * buf, pn[buf] & 1))) return false;
      ++pn[buf];
      tc::fence_after();
      const uint64_t vd = tc::smem_desc(sring + slot * C::kSlot, C::kBlock, 1024);
      if (tc::elect()) {
#pragma unroll
        for (int kk = 0; kk < CT / 16; ++kk)
          tc::mma_ts(tmem + C::kOCol + acc * D, tmem + buf * C::kSCol + kk * 8, vd + (kk * 2048 >> 4), IPV,
                     !first || kk > 0);
        tc::commit(pv_done + 8 * acc);
        if (!cp.two || (cp.j & 1)) tc::commit(empty + 8 * slot);
      }
      __syncwarp();
      ++cp.j;
      return true;
    };
    int ahead = 0;
    while (ok) {
      while (ok && ahead < 2 && next_qk()) {
        ok = qk();
        ++ahead;
      }
      if (!ok || ahead == 0) break;
      ok = pv();
      --ahead;
    }
    if (tc::elect()) tc::commit(idle);  // every product issued above has completed when this arrives
  } else {
    // ---- softmax: a row's columns in two halves, one thread each
    constexpr int HC = CT / 2;
    const int w = warp / C::kGroupWarps, half = warp >> 2 & 1, wq = warp & 3, row_in_tile = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t ocol = lanes + C::kOCol + w * D + half * (D / 2);
    // The two warps of the same rows exchange a value per row through a column of
    // tensor memory each (shared memory is full): own, then a barrier, then other.
    auto exchange = [&](uint32_t own, uint32_t other, float v) -> float {
      tc::st1(own, v);
      tc::wait_st();
      tc::fence_before();
      asm volatile("bar.sync %0, 64;\n" ::"r"(1 + w * 4 + wq) : "memory");
      tc::fence_after();
      return tc::ld1(other);
    };
    const float sl2 = p.scale_log2;
    const float none = sl2 >= 0.f ? -INFINITY : INFINITY;  // below every score
    uint32_t step = 0;               // steps of all units so far
    uint32_t sn[2] = {0, 0};         // S buffer uses
    uint32_t vn = 0;                 // products into this group's accumulator
    bool ok = true;
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      const bool two = NACC == 2 && u.rows > kTileRows;
      const int steps = two ? 2 * u.chunks : u.chunks;
      const int j0 = NACC == 2 ? (w ^ (int)step) & 1 : 0;  // the unit's first step of this group
      const int tile = two ? j0 : 0;
      const int r = tile * kTileRows + row_in_tile;
      const bool live = tile * kTileRows + wq * 32 < u.rows;  // the warp has a row
      float m = -INFINITY, l = 0.f;
      for (int j = j0; ok && j < steps; j += NACC) {
        const int buf = (int)(step + j) & 1;
        ok = __all_sync(0xffffffffu, wait(s_full + 8 * buf, sn[buf] & 1));
        ++sn[buf];
        if (!ok) break;
        if (live) {
          tc::fence_after();
          const uint32_t scol = lanes + buf * C::kSCol;
          float s[HC];
#pragma unroll
          for (int i = 0; i < HC; i += 32) tc::ld32(scol + half * HC + i, s + i);
          tc::wait_ld();
          const int nv = u.tok1 - (u.tok0 + (two ? j >> 1 : j) * CT) - half * HC;  // columns in range
          if (nv < HC) {
#pragma unroll
            for (int i = 0; i < HC; ++i)
              if (i >= nv) s[i] = none;
          }
          float mx[4] = {none, none, none, none};
          if (sl2 >= 0.f) {
#pragma unroll
            for (int i = 0; i < HC; i += 2) mx[i >> 1 & 3] = fmaxf(mx[i >> 1 & 3], fmaxf(s[i], s[i + 1]));
            mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          } else {
#pragma unroll
            for (int i = 0; i < HC; i += 2) mx[i >> 1 & 3] = fminf(mx[i >> 1 & 3], fminf(s[i], s[i + 1]));
            mx[0] = fminf(fminf(mx[0], mx[1]), fminf(mx[2], mx[3]));
          }
          // Each half's maximum travels in its last column of S, which it has read.
          // Behind the exchange all of S has been read: P, in its first half, may
          // overwrite it.
          float top = mx[0] * sl2;
          top = fmaxf(top, exchange(scol + half * HC + HC - 1, scol + (half ^ 1) * HC + HC - 1, top));
          // The reference moves only when a score passes it by 2^8: any
          // reference gives the same result as long as l and O share it, and the
          // rescale of O is skipped on almost every chunk.
          if (__any_sync(0xffffffffu, top > m + 8.f)) {
            const float mn = fmaxf(m, top);
            const float a = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= a;
            if (j != j0) {  // O holds the earlier chunks once their product is done
              ok = __all_sync(0xffffffffu, wait(pv_done + 8 * w, (vn - 1) & 1));
              if (!ok) break;
              tc::fence_after();
#pragma unroll 1
              for (int i = 0; i < D / 2; i += 16) {
                float o[16];
                tc::ld16(ocol + i, o);
                tc::wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] *= a;
                tc::st16(ocol + i, reinterpret_cast<const uint32_t *>(o));
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < HC; i += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float e0 = fast_exp2(s[i + x] * sl2 - ref), e1 = fast_exp2(s[i + x + 1] * sl2 - ref);
              ls[x & 2] += e0;
              ls[(x & 2) + 1] += e1;
              pk[x / 2] = pack_bf16x2(e0, e1);
            }
            tc::st16(scol + (half * HC + i) / 2, pk);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);  // fp32 weights: rounded ones would move lse by up to 2^-9
          if (j + NACC >= steps) l += exchange(scol + HC + half, scol + HC + (half ^ 1), l);  // the unit's sum
          tc::wait_st();
          tc::fence_before();
        }
        ++vn;
        __syncwarp();
        if (lane == 0) tc::arrive(p_full + 8 * buf);
      }
      if (ok && steps > j0) {
        // (a parity tells only neighbouring phases apart: with one accumulator the
        // last two products may both be open)
        if (NACC == 1 && steps > 1) ok = __all_sync(0xffffffffu, wait(pv_done + 8 * w, (vn - 2) & 1));
        ok = ok && __all_sync(0xffffffffu, wait(pv_done + 8 * w, (vn - 1) & 1));
        if (ok && live) {
          tc::fence_after();
          const float inv = 1.f / l;
          const int64_t row = u.part + (two || NACC == 1 ? 0 : (int64_t)j0 * u.rows) + r;
          float4 *dst = reinterpret_cast<float4 *>(p.o_part + row * D + half * (D / 2));
#pragma unroll
          for (int i = 0; i < D / 2; i += 32) {
            float o[32];
            tc::ld32(ocol + i, o);
            tc::wait_ld();
            if (r < u.rows) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[i / 4 + x] = make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
            }
          }
          if (half == 0 && r < u.rows) p.lse_part[row] = m + log2f(l);
          tc::fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::arrive(o_free + 8 * w);
      }
      step += steps;
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    wait(idle, 0, true);  // no product may write tensor memory that is given back
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// One warp per query row: the row's prefix units and rest units, found again
// from the cumulative costs, weighted by their log-sum-exp.
template <int D>
__global__ void __launch_bounds__(128) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int VEC = D / 32;
  constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)p.B * p.Hq) return;
  const int b = (int)(row / p.Hq), h = (int)(row % p.Hq);
  const int kvh = h / p.g, ht = h % p.g / p.gt, j = h % p.g % p.gt;
  const SharedPrefix pre = shared_prefix<D>(p);
  bool bad;
  const int L = shared_len(p, b, &bad), Lp = p.n_shared << p.bs_log2;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the partials and the cumulative costs are written
  const int64_t q = p.cum[p.B];

  // An item's candidate parts: (CTA, accumulator) pairs over the CTAs that its
  // cost range touches; one that took no chunk is none.
  struct Item {
    int64_t start, cta0, part;  // cost, first CTA, part row of CTA 0 and row
    int w, chunks, accs, stride, rows, n;
  };
  auto make = [&](int64_t start, int64_t cost, int w, int chunks, int64_t part0, int stride, int rows, int r) {
    Item it;
    it.start = start;
    it.cta0 = shared_div(start, q);
    it.part = part0 + r;
    it.w = w;
    it.chunks = chunks;
    it.accs = shared_part_rows(rows, D) / rows;
    it.stride = stride;
    it.rows = rows;
    it.n = (int)(shared_div(start + cost - 1, q) - it.cta0 + 1) * it.accs;
    return it;
  };
  Item pi{}, ri{};
  if (L > 0 && pre.chunks > 0) {
    const int grp = kvh * p.HT + ht, rb = b / p.nseq;
    const bool lastrb = rb == p.nrb - 1;
    const int rows = (lastrb ? pre.last_nb : p.nseq) * p.gt;
    pi = make(grp * pre.group + rb * pre.full, lastrb ? pre.last : pre.full, rows > kTileRows ? p.w_pre2 : p.w_pre1,
              pre.chunks, ((int64_t)grp * p.nrb + rb) * p.pre_rows, p.pre_rows, rows, (b - rb * p.nseq) * p.gt + j);
  }
  if (L > Lp) {
    const int64_t cost = shared_rest_cost<D>(p, L);
    const int k = kvh * p.HT + ht;
    ri = make(p.cum[b] + k * cost, cost, p.w_rest, (L - Lp + shared_chunk(D) - 1) / shared_chunk(D),
              p.rest_row0 + ((int64_t)b * p.Hkv * p.HT + k) * p.rest_rows, p.rest_rows, p.gt, j);
  }
  float m = -INFINITY, l = 0.f, acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  for (int i0 = 0; i0 < pi.n + ri.n; i0 += 32) {  // lane: one candidate
    const int i = i0 + lane;
    float s = -INFINITY;
    int64_t r = 0;
    if (i < pi.n + ri.n) {
      const Item &it = i < pi.n ? pi : ri;
      const int x = i < pi.n ? i : i - pi.n;
      const int64_t c = it.cta0 + x / it.accs;
      const int a = x % it.accs;
      const int n = shared_cut(p, (c + 1) * q - it.start, it.w, it.chunks) - shared_cut(p, c * q - it.start, it.w, it.chunks);
      if (a < n) {
        r = it.part + c * it.stride + a * it.rows;
        s = p.lse_part[r];
      }
    }
    float top = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - ref), w = exp2f(s - ref);
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * a + sum;
    m = mn;
#pragma unroll
    for (int x = 0; x < VEC; ++x) acc[x] *= a;
    uint32_t todo = __ballot_sync(0xffffffffu, s != -INFINITY);
    while (todo != 0) {  // four partials in flight
      float o[4][VEC], wj[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int jl = todo != 0 ? __ffs(todo) - 1 : 0;
        const int64_t rj = __shfl_sync(0xffffffffu, r, jl);
        wj[y] = todo != 0 ? __shfl_sync(0xffffffffu, w, jl) : 0.f;
        if (todo != 0) {
          const float *src = p.o_part + rj * D + lane * VEC;
#pragma unroll
          for (int x = 0; x < VEC; x += 2) {
            const float2 f = *reinterpret_cast<const float2 *>(src + x);
            o[y][x] = f.x;
            o[y][x + 1] = f.y;
          }
        } else {
#pragma unroll
          for (int x = 0; x < VEC; ++x) o[y][x] = 0.f;
        }
        todo &= todo - 1;
      }
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < VEC; ++x) acc[x] += wj[y] * o[y][x];
    }
  }
  float lse2 = m + log2f(l);  // no token: m = -inf
  if (p.sinks != nullptr) {
    const float sg = p.sinks[h] * kLog2e;
    const float top = fmaxf(m, sg);
    const float z = (m == -INFINITY ? 0.f : l * exp2f(m - top)) + (sg == -INFINITY ? 0.f : exp2f(sg - top));
    lse2 = top + log2f(z);
  }
  if (m == -INFINITY && p.sinks == nullptr) lse2 = -INFINITY;
  const float w = m == -INFINITY ? 0.f : exp2f(m - lse2) * p.v_scale;
  uint16_t *o = p.out + b * p.o_sb + (int64_t)h * p.o_sh + lane * VEC;
#pragma unroll
  for (int i = 0; i < VEC; i += 2)
    *reinterpret_cast<uint32_t *>(o + i) = pack_bf16x2(acc[i] * w, acc[i + 1] * w);
  if (lane == 0 && p.lse != nullptr) p.lse[b * p.lse_sb + (int64_t)h * p.lse_sh] = lse2 * kLn2;
}

template <int D, bool F8>
cudaError_t launch_t(const SharedParams &p, cudaStream_t s) {
  cudaError_t e;
  if constexpr (F8) {
    shared_kernel<D, F8><<<p.ctas, 256, 0, s>>>(p);
  } else {
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(shared_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)SharedCfg<D>::total);
      if (e != cudaSuccess) return e;
      attr_done.fetch_or(bit, std::memory_order_acq_rel);
    }
    shared_tc_kernel<D><<<p.ctas, SharedCfg<D>::kThreads, SharedCfg<D>::total, s>>>(p);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.B * p.Hq;
  // comes up while the partial kernel's last CTAs run; waits for them before its first read
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, p);
}

}  // namespace

cudaError_t launch_shared(const SharedParams &p, int D, bool kv_fp8, cudaStream_t s) {
  switch (D) {
    case 64: return kv_fp8 ? launch_t<64, true>(p, s) : launch_t<64, false>(p, s);
    case 128: return kv_fp8 ? launch_t<128, true>(p, s) : launch_t<128, false>(p, s);
    case 256: return kv_fp8 ? launch_t<256, true>(p, s) : launch_t<256, false>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pad
