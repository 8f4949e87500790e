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
#include <type_traits>

#include "pad_device.cuh"
#include "pad_f32x2.cuh"
#include "pad_shared.h"
#include "pad_shared_walk.cuh"
#include "pad_tc.cuh"

namespace pad {
namespace {

// ---- the partial kernel -------------------------------------------------------
//
// One persistent CTA per SM, warp-specialised; every role goes through the CTA's
// units in order, each as far ahead as its buffers let it:
//
//   unit warp       walks the work line, puts units into a queue of kQueue, copies
//                   (TMA) their q rows
//   K and V warps   a unit's chunks, each into a ring of its own
//   QK warp         S = Q . K^T  (128 rows x chunk) into one of the S buffers
//   PV warp         O += P . V, P read from tensor memory
//   softmax warps   thread = row: scores out of tensor memory, running maximum and
//                   sum, P back over the scores
//   widening warps  (E4M3 cache) the copies' codes, from a small ring of their own, to
//                   f16 operands: four warps for K, four for V, q's rows by all
//
// Every E4M3 code is an f16 value, and q is scaled per row by a power of two that
// puts its largest element into [2^14, 2^15), where its bf16 values are f16 values
// too (down to 2^-28 of that element); the row's score scale takes the inverse.  P is
// f16 then, three bits finer than bf16 down to 2^-14, and a fixed point of 2^-24 below.  So
// weights stand 2^7 higher than their exponents say (they reach 2^8 over the row's
// reference, f16 2^15): a weight of 2^-21 of the largest has its full bits, and one is lost
// from 2^-32 on, with 2^20 of those 2^-12 of the output; 2^-25, without, would be 3 %.
//
// A step is (query tile, chunk); step n of the CTA uses S buffer n % NBUF and is the
// buffer's use n / NBUF, which gives every barrier's phase.  A two-tile unit takes both
// tiles through each chunk, a tile per accumulator; a one-tile unit alternates its
// even and odd chunks between the accumulators, which leave two partials per row.
// At D = 256 there is one accumulator (256 of the 512 columns) and one softmax group.
//
// The P of a step overlays its S, so QK(n + NBUF) waits for PV(n).  Four buffers of 64
// tokens keep the next scores ready when a group has written P.  The products are
// issued by two warps because between two of them a warp spends about as long on its
// waits and counters as the tensor core on a product: from one warp the products' issue
// was half of its time.
//
// Rounding: P to 16 bits (bf16; f16 with an E4M3 cache), the operand's type; l sums the
// weights before that, in fp32, as O and the partials are.
//
// Measured on B200 (bf16 unless said; merge included):
//   256 sequences of 32 / 8 heads of 128 behind 32768 tokens: 145 us, 945 TFLOP/s, 57 %
//     of the measured matrix peak; 64 of 40 / 8, 8192 tokens of their own each: 344 us,
//     6.2 TB/s, 95 % of the measured copy rate.  The first is bound by the chain scores ->
//     exponentials -> product of two tiles taking turns, the second by HBM.  With up to 400
//     tokens behind the first's prefix (198 us) the tensor pipe is busy 40 %, the
//     exponentials' 35 %, issue slots 32 %, DRAM 45 %: 745 MB are read where 346 would do, as
//     row blocks cut at different chunks read a page at different times.
//   Two buffers of 128 tokens with two threads per row 161 us where this kernel, then,
//     took 153; a quarter of the exponentials on the FMA pipe instead of ex2 154, half
//     163; a pair of issuing warps per accumulator the same within 1 %.
//   Rest items (a few rows, a few chunks) are bound by latency and by instruction
//     fetches: a unit change runs every role's code, and warps then wait for instructions
//     longer than for anything but data (64 sequences with up to 700 tokens behind 8192:
//     tensor pipe 23 %, exponentials' 14 %, DRAM 33 %).  Scores read from tensor memory twice, a half at
//     a time in loops that are not unrolled, instead of once into 64 registers: 256
//     sequences with up to 400 tokens behind those 32768 206 -> 195 us.
//   E4M3, 48 sequences of 32 / 8 heads behind 6000 tokens: 44 us (tensor pipe 14 %, DRAM
//     11 %), of which q's conversion
//     with a thread per row took 10 and two widening warps per ring instead of four 2.
template <int D, bool F8>
struct SharedCfg {
  static constexpr int CT = kSharedChunk, NBUF = 4, NACC = shared_accs(D), CB = D / 64;
  static constexpr int QR = shared_rows(D);
  static constexpr uint32_t kSlot = CT * D * 2;         // bytes of a K or V chunk
  // A chunk's rows lie in groups of 8, a group's 128-byte column blocks one after
  // another: a page arrives with one copy, and the groups keep one stride.
  static constexpr uint32_t kGroup = CB * 1024;
  static constexpr uint32_t kQBlock = QR * 128;         // one column block of q
  static constexpr uint32_t kQ = CB * kQBlock;
  // Ring slots: what is left beside q.  V's slots are held longer, from the copy
  // to the value product two steps behind the score product.
  static constexpr int NK = 512 / D, NV = D == 64 ? 8 : F8 ? NK : D == 128 ? 6 : 3, NS = NK + NV;
  // E4M3: slots of codes, per ring; rows of boxes of at least 128 bytes
  static constexpr int NR = F8 ? (D == 256 ? 1 : 2) : 0;
  static constexpr uint32_t kRaw = CT * (D < 128 ? 128 : D);
  static constexpr int kQueue = 4;
  static constexpr int kGroupWarps = 4;                 // a softmax group: a tile's rows
  static constexpr int kSoftmaxWarps = kGroupWarps * NACC;
  static constexpr int kKWarp = kSoftmaxWarps, kVWarp = kSoftmaxWarps + 1, kQkWarp = kSoftmaxWarps + 2,
                       kPvWarp = kSoftmaxWarps + 3, kWidenWarp = kSoftmaxWarps + 4,
                       kUnitWarp = kSoftmaxWarps + (F8 ? 12 : 4);
  static constexpr int kWarps = kUnitWarp + 1, kThreads = kWarps * 32;
  static constexpr uint32_t ring = kQ, raw = ring + NS * kSlot, unscale = raw + 2 * NR * kRaw,
                            queue = unscale + (F8 ? QR * 4 : 0),
                            bars = queue + kQueue * 64;
  static constexpr uint32_t kBarBytes = 640, total = bars + kBarBytes + 1024 /* alignment slack */;
  static constexpr float kRaise = F8 ? 7.f : 0.f;       // weights are 2^(s - m + kRaise)
  static constexpr uint32_t kSCol = CT, kOCol = NBUF * CT;  // tensor memory: S buffers, then O
};
static_assert(sizeof(SharedUnit) <= 64, "queue entry");

// Power of two that scales a row of bf16 q whose largest magnitude is that of either half
// into f16's range, as an exponent; 0 for a row of zeros or one that is not finite.  From
// -113 for bf16's largest to 126, above which its inverse is no normal fp32: rows that
// would take more (below 2^-112) get to 2^0 at least, where f16 holds them to 2^-25 of
// their largest element.
__device__ __forceinline__ int q_exponent(uint32_t halves) {
  const uint32_t abs_bits = max(halves & 0xffffu, halves >> 16);
  return abs_bits == 0 || abs_bits >= 0x7f80u ? 0 : min(126, 141 - (int)(abs_bits >> 7));
}
// Largest magnitudes of the even and of the odd values so far, a half each.
__device__ __forceinline__ uint32_t max_abs(uint32_t m, const uint4 &c) {
  const uint32_t k = 0x7fff7fffu;
  return __vmaxu2(m, __vmaxu2(__vmaxu2(c.x & k, c.y & k), __vmaxu2(c.z & k, c.w & k)));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

// A piece's sums (a lane's row of tensor memory, 1 / l, lse) joined with what the row's
// earlier pieces left in its part row, by a whole warp.  Pieces without a weight, lse =
// -inf, add nothing.  A function of its own: units of one piece do not fetch it.
template <int D>
__device__ __noinline__ void fold_sums(uint32_t ocol, float4 *dst, float *lse_at, bool some, float lse, float inv) {
  const float had = some ? *lse_at : -INFINITY;
  const float top = fmaxf(had, lse), ref = top == -INFINITY ? 0.f : top;
  const float a = exp2f(had - ref), b = exp2f(lse - ref);  // (NaN stays NaN)
  const float keep = had == -INFINITY ? 0.f : a / (a + b);
  inv = lse == -INFINITY ? 0.f : inv * b / (a + b);
#pragma unroll 1
  for (int i = 0; i < D; i += 16) {
    float o[16];
    tc::ld16(ocol + i, o);
    tc::wait_ld16(o);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (!some) break;
      float4 v = make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
      if (keep != 0.f) {
        const float4 w = dst[i / 4 + x];
        v = make_float4(v.x + keep * w.x, v.y + keep * w.y, v.z + keep * w.z, v.w + keep * w.w);
      }
      dst[i / 4 + x] = v;
    }
  }
  if (some) *lse_at = top + log2f(a + b);
}

template <int D, bool F8>
__global__ void __launch_bounds__(SharedCfg<D, F8>::kThreads, 1)
    shared_kernel(const __grid_constant__ SharedParams p) {
  using C = SharedCfg<D, F8>;
  constexpr int CT = C::CT, NACC = C::NACC, NBUF = C::NBUF, NS = C::NS, CB = C::CB;
  static_assert(C::total <= (uint32_t)kSmemBudget, "shared-memory plan over budget");
  static_assert(C::kOCol + NACC * D <= 512, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sq = smem_addr(smem), sring = sq + C::ring;
  SharedUnit *queue = reinterpret_cast<SharedUnit *>(smem + C::queue);  // entries 64 bytes apart
  float *unscale = reinterpret_cast<float *>(smem + C::unscale);  // E4M3: 1 / the power of two of each q row
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::bars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t full = bar0, empty = full + 8 * NS, q_full = empty + 8 * NS, q_empty = q_full + 16,
                 s_full = q_empty + 16, p_full = s_full + 8 * NBUF, pv_done = p_full + 8 * NBUF,
                 o_free = pv_done + 8 * NBUF,
                 u_full = o_free + 16, u_empty = u_full + 8 * C::kQueue, idle = u_empty + 8 * C::kQueue,
                 q_tx = F8 ? idle + 8 : q_full, raw_full = q_tx + 16, raw_empty = raw_full + 16 * C::NR;
  constexpr int kBars = 2 * NS + 3 * NBUF + 6 + 2 * C::kQueue + 1 + (F8 ? 2 + 4 * C::NR : 0);
  static_assert(kBars * 8 + 8 <= C::kBarBytes, "barrier area");
  uint32_t *words = reinterpret_cast<uint32_t *>(bars + kBars);  // [0] tmem, [1] abort
  volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, F8 ? 4 : 1);  // a ring's widening warps, or the copy
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, F8 ? 8 : 1);  // the widening warps, or the copy
      if (F8) mbar_init(q_tx + 8 * i, 1);
      mbar_init(q_empty + 8 * i, F8 ? 1 + C::kSoftmaxWarps : 1);  // its products; E4M3: and its rows' powers read
      mbar_init(o_free + 8 * i, C::kGroupWarps);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, C::kGroupWarps);
      mbar_init(pv_done + 8 * i, 1);
    }
    for (int i = 0; i < C::kQueue; ++i) {
      mbar_init(u_full + 8 * i, 1);
      mbar_init(u_empty + 8 * i, C::kWarps - 1);  // every warp but the one that fills it
    }
    for (int i = 0; i < 2 * C::NR; ++i) {
      mbar_init(raw_full + 8 * i, 1);
      mbar_init(raw_empty + 8 * i, 4);
    }
    mbar_init(idle, 2);
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
  // What is above may run beside the kernel before this one; nothing below does.  The
  // merge may come up from here on: it reads the lengths, which that kernel may write.
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;\n" ::: "memory");

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

  // One ring's chunks of a unit, by a whole warp: K's or V's.  (E4M3: its codes' ring.)
  const uint32_t copied = F8 ? raw_full : full, freed = F8 ? raw_empty : empty;
  uint32_t slot = 0, phase = 1, used = 0;  // a first filling's wait passes at once
  auto copy_chunks = [&](const SharedUnit &u, auto which) -> bool {
    constexpr bool kIsK = decltype(which)::value;
    const CUtensorMap *map = kIsK ? &p.tmk : &p.tmv;
    constexpr uint32_t first_slot = kIsK ? 0 : F8 ? C::NR : C::NK, slots = F8 ? C::NR : kIsK ? C::NK : C::NV;
    const int32_t *table = u.rest ? p.tables + u.b0 * p.table_stride : p.shared_table;
    const int box_log2 = p.box_log2, nbox = CT >> box_log2;
    // Block of box 32 w + lane of a chunk: num_blocks (reads as zeros) behind the
    // unit's tokens and for an id that is not one.
    auto fetch = [&](int c, int w) -> int {
      const int t = u.tok0 + c * CT + ((32 * w + lane) << box_log2);
      if (c >= u.chunks || t >= u.tok1) return p.num_blocks;
      const int id = __ldg(table + (t >> p.bs_log2));
      if ((unsigned)id < (unsigned)p.num_blocks) return id;
      atomicOr(p.err, kErrBlockId);
      return p.num_blocks;
    };
    int id_next = fetch(0, 0);
    for (int c = 0; c < u.chunks; ++c) {
      int id = id_next;
      id_next = fetch(c + 1, 0);  // a chunk ahead: the table's latency is not in the copies' way
      const uint32_t bar = copied + 8 * (first_slot + slot);
      const uint32_t dst = F8 ? sq + C::raw + (first_slot + slot) * C::kRaw : sring + (first_slot + slot) * C::kSlot;
      if (!__all_sync(0xffffffffu, wait(freed + 8 * (first_slot + slot), phase))) return false;
      if (lane == 0) mbar_arrive_expect_tx(bar, F8 ? CT * D : C::kSlot);
      __syncwarp();
      // A lane per box: measured 118 cycles a copy, against 280 for a loop of one
      // elected lane, which sets up the copy's uniform operands each time.
      // (a box's first row inside its page: only pages larger than a box have several)
      const int in_page = u.tok0 + c * CT, mask = (1 << p.bs_log2) - 1;
      for (int j = lane; j < nbox; j += 32) {
        if (j >= 32) id = fetch(c, j >> 5);  // (pages of 1 token)
        const int row = j << box_log2, at = (in_page + row) & mask;
        if constexpr (F8) {
          tma_load_4d(dst + j * p.box_pitch, map, 0, at, u.kvh, id, bar);
        } else {
          const uint32_t to = dst + (row >> 3) * C::kGroup + (row & 7) * 128;
          if (p.box_kind == kBoxPage) {  // a page, or a chunk's worth of a larger one
            tma_load_5d(to, map, 0, 0, 0, at >> 3, id * p.blk_heads + u.kvh, bar);
          } else if (p.box_kind == kBoxGroup) {  // 8 rows
            tma_load_5d(to, map, 0, at, 0, u.kvh, id, bar);
          } else {  // pages below 8 tokens: a column block of a page
            for (int cb = 0; cb < CB; ++cb) tma_load_5d(to + cb * 1024, map, 0, 0, cb, u.kvh, id, bar);
          }
        }
      }
      __syncwarp();
      ++used;
      if (++slot == slots) {
        slot = 0;
        phase ^= 1;
      }
    }
    return true;
  };
  // Leaves no copy in flight, whoever gives up: a chunk is copied once its slot's
  // earlier one has been read, so only a ring's last round can be open.
  auto drain = [&](uint32_t first_slot, uint32_t slots) {
    if (lane == 0)
      for (uint32_t i = used > slots ? used - slots : 0; i < used; ++i)
        wait(copied + 8 * (first_slot + i % slots), (i / slots) & 1, true);
  };

  if (warp == C::kUnitWarp) {
    uint32_t qphase = 3;  // a bit per half of q
    int k = 0, half = 0;
    bool ok = true, q_used[2] = {false, false};
    auto put = [&](const SharedUnit &u) {
      const int e = k % C::kQueue;
      ok = ok && (k < C::kQueue || __all_sync(0xffffffffu, wait(u_empty + 8 * e, (k / C::kQueue - 1) & 1)));
      if (ok && lane == 0) {
        *reinterpret_cast<SharedUnit *>(reinterpret_cast<uint8_t *>(queue) + 64 * e) = u;
        tc::arrive(u_full + 8 * e);
      }
      ++k;
    };
    shared_walk<D>(p, blockIdx.x, [&](const SharedUnit &u) {
      put(u);
      const int box_rows = q_box_rows(u);
      const bool both = NACC == 2 && box_rows > kTileRows;
      const int h = both || NACC == 1 ? 0 : half;
      if (!both && NACC == 2) half ^= 1;
      ok = ok && __all_sync(0xffffffffu, wait(q_empty + 8 * h, qphase >> h & 1));
      if (both) ok = ok && __all_sync(0xffffffffu, wait(q_empty + 8, qphase >> 1));
      if (!ok) return;
      if (tc::elect()) {
        mbar_arrive_expect_tx(q_tx + 8 * h, (uint32_t)box_rows * 128 * CB);
        if (both) tc::arrive(q_tx + 8);
        for (int cb = 0; cb < CB; ++cb)
          tma_load_4d(sq + cb * C::kQBlock + h * (kTileRows * 128), u.rest ? &p.tmqr : &p.tmqp, 0,
                      u.kvh * p.g + u.ht * p.gt, cb, u.b0, q_tx + 8 * h);
      }
      __syncwarp();
      qphase ^= both ? 3 : 1 << h;
      q_used[h] = true;
    });
    put(SharedUnit{});  // chunks == 0: the end
    if (lane == 0)
      for (int h = 0; h < 2; ++h)
        if (q_used[h]) wait(q_tx + 8 * h, qphase >> h & 1, true);
  } else if (warp == C::kKWarp) {
    bool ok = true;
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) ok = copy_chunks(u, std::true_type{});
    drain(0, F8 ? C::NR : C::NK);
  } else if (warp == C::kVWarp) {
    bool ok = true;
    SharedUnit u;
    constexpr uint32_t first = F8 ? C::NR : C::NK, slots = F8 ? C::NR : C::NV;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) ok = copy_chunks(u, std::false_type{});
    drain(first, slots);
  } else if (warp == C::kQkWarp) {
    const uint32_t idesc = tc::idesc(CT, false, F8) | (p.scale_log2 < 0.f ? tc::kNegateA : 0u);
    const uint64_t qd0 = tc::smem_desc(sq, 16, 1024), kd0 = tc::smem_desc(sring, 16, C::kGroup);
    uint32_t kslot = 0, kphase = 0, n = 0;  // ring slot and its phase, steps so far
    uint32_t qphase = 0;                    // a bit per half of q
    int half = 0;
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      const bool two = NACC == 2 && u.rows > kTileRows, both = NACC == 2 && q_box_rows(u) > kTileRows;
      const int h = both || NACC == 1 ? 0 : half;
      if (!both && NACC == 2) half ^= 1;
      ok = all(wait(q_full + 8 * h, qphase >> h & 1)) && (!both || all(wait(q_full + 8, qphase >> 1)));
      qphase ^= both ? 3 : 1 << h;
      const uint64_t qd = qd0 + (uint32_t)h * (kTileRows * 128 >> 4);
      auto step = [&](int tile, bool last_tile, bool last) -> bool {
        const uint32_t buf = n % NBUF;
        if (n >= NBUF && !all(wait(pv_done + 8 * buf, (n / NBUF - 1) & 1))) return false;
        tc::fence_after();
        const uint64_t a = qd + (uint32_t)tile * (kTileRows * 128 >> 4), b = kd0 + kslot * (C::kSlot >> 4);
        const uint32_t d = tmem + buf * C::kSCol;
        if (tc::elect()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ss(d, a + (((kk >> 2) * C::kQBlock + (kk & 3) * 32) >> 4),
                       b + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc, kk > 0);
          tc::commit(s_full + 8 * buf);
          if (last_tile) tc::commit(empty + 8 * kslot);
          if (last) {
            tc::commit(q_empty + 8 * h);
            if (both) tc::commit(q_empty + 8);
          }
        }
        __syncwarp();
        ++n;
        return true;
      };
      for (int c = 0; ok && c < u.chunks; ++c) {
        ok = all(wait(full + 8 * kslot, kphase)) && step(0, !two, !two && c + 1 == u.chunks) &&
             (!two || step(1, true, c + 1 == u.chunks));
        if (++kslot == C::NK) {
          kslot = 0;
          kphase ^= 1;
        }
      }
    }
    if (tc::elect()) tc::commit(idle);  // every product issued above has completed when this arrives
  } else if (warp == C::kPvWarp) {
    constexpr uint32_t idesc = tc::idesc(D, true, F8);
    const uint64_t vd0 = tc::smem_desc(sring + C::NK * C::kSlot, 1024, C::kGroup);
    uint32_t vslot = 0, vphase = 0, n = 0;
    uint32_t ophase = 3;  // a bit per accumulator; the first wait on each passes at once
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      const bool two = NACC == 2 && u.rows > kTileRows;
      auto step = [&](bool first, bool last_tile) -> bool {
        const uint32_t buf = n % NBUF, acc = NACC == 2 ? n & 1 : 0;
        if (first) {  // the last unit's sums have been read
          if (!all(wait(o_free + 8 * acc, ophase >> acc & 1))) return false;
          ophase ^= 1 << acc;
        }
        if (!all(wait(p_full + 8 * buf, n / NBUF & 1))) return false;
        tc::fence_after();
        const uint64_t b = vd0 + vslot * (C::kSlot >> 4);
        const uint32_t d = tmem + C::kOCol + acc * D, a = tmem + buf * C::kSCol;
        if (tc::elect()) {
#pragma unroll
          for (int kk = 0; kk < CT / 16; ++kk) tc::mma_ts(d, a + kk * 8, b + (kk * 2 * C::kGroup >> 4), idesc, !first || kk > 0);
          tc::commit(pv_done + 8 * buf);
          if (last_tile) tc::commit(empty + 8 * (C::NK + vslot));
        }
        __syncwarp();
        ++n;
        return true;
      };
      for (int c = 0; ok && c < u.chunks; ++c) {
        ok = all(wait(full + 8 * (C::NK + vslot), vphase));
        const int nv = u.tok1 - (u.tok0 + c * CT), bs = 1 << p.bs_log2;
        if (!F8 && ok && nv < CT && (u.tok1 & (bs - 1)) != 0) {
          // The page the sequence ends in arrived whole: zeros over the slots behind
          // the sequence, whatever they hold (a weight of 0 times NaN is NaN).
          const int end = min(CT, nv + bs - (u.tok1 & (bs - 1)));
          uint8_t *v = smem + C::ring + (C::NK + vslot) * C::kSlot;
          for (int x = lane; x < (end - nv) * (D / 8); x += 32) {
            const int row = nv + x / (D / 8), at = x % (D / 8) * 16;  // (the swizzle stays inside the 128 bytes)
            *reinterpret_cast<uint4 *>(v + (row >> 3) * C::kGroup + (at >> 7) * 1024 + (row & 7) * 128 + (at & 127)) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ok = ok && step(two ? c == 0 : c < NACC, !two) && (!two || step(c == 0, true));
        if (++vslot == C::NV) {
          vslot = 0;
          vphase ^= 1;
        }
      }
    }
    if (tc::elect()) tc::commit(idle);
  } else if (F8 && warp >= C::kWidenWarp) {
    const bool is_k = warp < C::kWidenWarp + 4;
    const int t = (warp & 3) * 32 + lane;  // (kWidenWarp is a multiple of 4) of the ring's 128 threads
    constexpr int LR = D / 16;             // threads of a row: 16 codes each
    const uint32_t first = is_k ? 0 : C::NK, slots = is_k ? C::NK : C::NV, raw0 = is_k ? 0 : C::NR;
    uint32_t slot = 0, phase = 1, rslot = 0, rphase = 0, qphase = 0;
    int half = 0;
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      {  // ---- q: bf16 to f16 in place, by both rings' warps
        const bool both = NACC == 2 && q_box_rows(u) > kTileRows;
        const int h = both || NACC == 1 ? 0 : half;
        if (!both && NACC == 2) half ^= 1;
        ok = all(wait(q_tx + 8 * h, qphase >> h & 1)) && (!both || all(wait(q_tx + 8, qphase >> 1)));
        if (!ok) break;
        qphase ^= both ? 3 : 1 << h;
        // 16 bytes of a row per lane: a thread per row would take a rest unit, with its
        // few rows, as long as a full tile.
        constexpr int QL = D / 8, RI = 32 / QL, kRows = 2;  // lanes of a row; rows of a warp at a time, times kRows in flight
        const int c = lane % QL;
        for (int r0 = (warp - C::kWidenWarp) * RI + lane / QL; r0 - lane / QL < u.rows; r0 += 8 * RI * kRows) {
          uint4 v[kRows];
          auto at = [&](int i) {
            const int r = r0 + i * 8 * RI;
            return reinterpret_cast<uint4 *>(smem + (h * kTileRows + r) * 128 + (c >> 3) * C::kQBlock + ((c ^ r) & 7) * 16);
          };
#pragma unroll
          for (int i = 0; i < kRows; ++i) v[i] = r0 + i * 8 * RI < u.rows ? *at(i) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            if (r0 - lane / QL + i * 8 * RI >= u.rows) break;
            uint32_t m = max_abs(0, v[i]);
#pragma unroll
            for (int off = QL / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float f = pow2(q_exponent(m));
            auto scaled = [&](uint32_t x) { return pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
            if (c == 0 && r0 + i * 8 * RI < u.rows) unscale[h * kTileRows + r0 + i * 8 * RI] = pow2(-q_exponent(m));
            if (r0 + i * 8 * RI < u.rows) *at(i) = make_uint4(scaled(v[i].x), scaled(v[i].y), scaled(v[i].z), scaled(v[i].w));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::arrive(q_full + 8 * h);
          if (both) tc::arrive(q_full + 8);
        }
      }
      for (int c = 0; c < u.chunks; ++c) {
        const uint32_t r = raw0 + rslot, s = first + slot;
        ok = all(wait(raw_full + 8 * r, rphase)) && all(wait(empty + 8 * s, phase));
        if (!ok) break;
        const uint8_t *raw = smem + C::raw + r * C::kRaw;
        uint8_t *to = smem + C::ring + s * C::kSlot;
        const int nv = is_k ? CT : u.tok1 - (u.tok0 + c * CT);  // V: zeros behind the unit's tokens
        const int in_box = (1 << p.box_log2) - 1;
        constexpr int kFlight = LR < 8 ? 2 : 4;  // loads in flight, all before the first store
#pragma unroll 1
        for (int i0 = 0; i0 < LR / 2; i0 += kFlight) {
          uint4 code[kFlight];
#pragma unroll
          for (int i = 0; i < kFlight; ++i) {
            const int row = (i0 + i) * (128 / LR) + t / LR, x = t % LR;
            code[i] = row < nv ? *reinterpret_cast<const uint4 *>(raw + (row >> p.box_log2) * p.box_pitch +
                                                                  (row & in_box) * D + x * 16)
                               : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < kFlight; ++i) {
            const int row = (i0 + i) * (128 / LR) + t / LR, x = t % LR;
            uint4 a, b;  // codes 0-7 and 8-15
            e4m3x4_to_f16x2x2(code[i].x, a.x, a.y);
            e4m3x4_to_f16x2x2(code[i].y, a.z, a.w);
            e4m3x4_to_f16x2x2(code[i].z, b.x, b.y);
            e4m3x4_to_f16x2x2(code[i].w, b.z, b.w);
            uint8_t *d = to + (row >> 3) * C::kGroup + (x >> 2) * 1024 + (row & 7) * 128;
            const int c0 = (2 * (x & 3)) ^ (row & 7), odd = x >> 2 & 1;  // odd blocks store their second chunk first:
            *reinterpret_cast<uint4 *>(d + (c0 ^ odd) * 16) = odd ? b : a;  // eight threads, eight 16-byte banks
            *reinterpret_cast<uint4 *>(d + (c0 ^ odd ^ 1) * 16) = odd ? a : b;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::arrive(full + 8 * s);
          tc::arrive(raw_empty + 8 * r);
        }
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
        if (++rslot == (uint32_t)C::NR) {
          rslot = 0;
          rphase ^= 1;
        }
      }
    }
  } else {
    // ---- softmax: thread = row of the group's tile
    const int w = warp / C::kGroupWarps, wq = warp & 3, row_in_tile = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t ocol = lanes + C::kOCol + w * D;
    float sl2 = fabsf(p.scale_log2);  // a negative scale's sign is in the score product
    uint32_t step = 0;               // steps of all units so far
    uint32_t qphase = 0;             // E4M3: a bit per half of q
    int half = 0;
    bool ok = true;
    SharedUnit u;
    for (int k = 0; ok && (ok = next_unit(k, u)) && u.chunks > 0; ++k) {
      const bool two = NACC == 2 && u.rows > kTileRows;
      const int steps = two ? 2 * u.chunks : u.chunks;
      const int j0 = NACC == 2 ? (w ^ (int)step) & 1 : 0;  // the unit's first step of this group
      const int tile = two ? j0 : 0;
      const int r = tile * kTileRows + row_in_tile;
      const bool live = tile * kTileRows + wq * 32 < u.rows;  // the warp has a row
      int nv = u.tok1 - u.tok0 - (two ? 0 : j0) * CT;         // tokens of the step's chunk and behind it
      float m = -INFINITY, l = 0.f;
      if constexpr (F8) {  // the power of two that the row's q was scaled by
        const bool both = NACC == 2 && q_box_rows(u) > kTileRows;
        const int h = both || NACC == 1 ? 0 : half;
        if (!both && NACC == 2) half ^= 1;
        ok = __all_sync(0xffffffffu, wait(q_full + 8 * h, qphase >> h & 1) && (!both || wait(q_full + 8, qphase >> 1)));
        if (!ok) break;
        qphase ^= both ? 3 : 1 << h;
        // not 0, however small: a masked score, -inf, has to stay -inf
        sl2 = fmaxf(fabsf(p.scale_log2) * (r < u.rows ? unscale[h * kTileRows + r] : 1.f), kTinyScale);
        __syncwarp();
        if (lane == 0) {
          tc::arrive(q_empty + 8 * h);
          if (both) tc::arrive(q_empty + 8);
        }
      }
      const uint64_t scale = duo(sl2, sl2);
      for (int j = j0; ok && j < steps; j += NACC, nv -= (two ? 1 : NACC) * CT) {
        const uint32_t n = step + j, buf = n % NBUF;
        ok = __all_sync(0xffffffffu, wait(s_full + 8 * buf, n / NBUF & 1));
        if (!ok) break;
        if (live) {
          tc::fence_after();
          const uint32_t scol = lanes + buf * C::kSCol;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
// Not unrolled, and the scores read twice: with a tile's 64 scores held, the roles of a
// unit change did not fit the instruction cache beside one another.
#pragma unroll 1
          for (int i0 = 0; i0 < CT; i0 += 32) {
            float s[32];
            tc::ld32(scol + i0, s);
            tc::wait_ld32(s);
            if (nv < i0 + 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i0 + i >= nv) s[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx[i >> 1 & 3] = fmaxf(fmaxf(mx[i >> 1 & 3], s[i]), s[i + 1]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
          // The reference moves only when a score passes it by 2^8: any
          // reference gives the same result as long as l and O share it, and the
          // rescale of O is skipped on almost every chunk.
          if (__any_sync(0xffffffffu, r < u.rows && top > m + 8.f)) {
            const float mn = fmaxf(m, top);
            const float a = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= a;
            if (j != j0) {  // O holds the earlier chunks once their product is done
              const uint32_t before = n - NACC;
              ok = __all_sync(0xffffffffu, wait(pv_done + 8 * (before % NBUF), before / NBUF & 1));
              if (!ok) break;
              tc::fence_after();
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                float o[16];
                tc::ld16(ocol + i, o);
                tc::wait_ld16(o);
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] *= a;
                tc::st16(ocol + i, reinterpret_cast<const uint32_t *>(o));
              }
            }
          }
          const float ref = (m == -INFINITY ? 0.f : m) - C::kRaise;
          const uint64_t shift = duo(-ref, -ref);
          uint64_t ls[2] = {0, 0};
#pragma unroll 1
          for (int i = 0; i < CT; i += 32) {
            float s[32];
            tc::ld32(scol + i, s);
            tc::wait_ld32(s);
            if (nv < i + 32) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (i + x >= nv) s[x] = -INFINITY;
            }
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float2 e = parts(fma2(duo(s[x], s[x + 1]), scale, shift));
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              ls[x >> 1 & 1] = add2(ls[x >> 1 & 1], duo(e.x, e.y));
              pk[x / 2] = F8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
            }
            tc::st16(scol + i / 2, pk);
          }
          const float2 sum = parts(add2(ls[0], ls[1]));
          l += sum.x + sum.y;  // fp32 weights: rounded ones would move lse by up to 2^-9
          tc::wait_st();
          tc::fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::arrive(p_full + 8 * buf);
      }
      if (ok && steps > j0) {
        const uint32_t n = step + j0 + (steps - 1 - j0) / NACC * NACC;  // the group's last step
        ok = __all_sync(0xffffffffu, wait(pv_done + 8 * (n % NBUF), n / NBUF & 1));
        if (ok && live) {
          tc::fence_after();
          const float inv = 1.f / l, lse = m - C::kRaise + log2f(l);
          const int64_t row = u.part + (two || NACC == 1 ? 0 : (int64_t)j0 * u.rows) + r;
          float4 *dst = reinterpret_cast<float4 *>(p.o_part + row * D);
          if (__builtin_expect(u.fold, 0)) {
            fold_sums<D>(ocol, dst, p.lse_part + row, r < u.rows, lse, inv);
          } else {
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              float o[32];
              tc::ld32(ocol + i, o);
              tc::wait_ld32(o);
              if (r < u.rows) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  dst[i / 4 + x] = make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
              }
            }
            if (r < u.rows) p.lse_part[row] = lse;
          }
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

// One to four warps per query row: the row's prefix units and rest units, found again
// from the lengths, weighted by their log-sum-exp.  What needs only the lengths is
// done before the partial kernel has ended.
constexpr int kMergeWarps = 8;
__host__ __device__ __forceinline__ int merge_ctas(int Hq, int wpr) { return (Hq * wpr + kMergeWarps - 1) / kMergeWarps; }
// Sum over a warp of values in [0, 2^58): two halves' worth of bits at a time, which
// one instruction adds up without a carry out of 32.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
  int64_t sum = (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)v & 0x3ffffffu) +
                ((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 26) & 0x3ffffffu) << 26);
  if (__any_sync(0xffffffffu, v >> 52 != 0)) sum += (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 52)) << 52;
  return sum;
}
template <int D, int VEC>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int WPR = D / (32 * VEC);  // warps of a row
  constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;
  __shared__ int64_t sums[2][kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = merge_ctas(p.Hq, WPR);
  const int b = (int)(blockIdx.x / per_seq), wh = (int)(blockIdx.x % per_seq) * kMergeWarps + warp;
  const int h = wh / WPR, col = (wh % WPR * 32 + lane) * VEC;
  // costs of all rest items, and of those of the sequences before b
  int64_t all = 0, before = 0;
  bool bad;
  for (int x = threadIdx.x; x < p.B; x += kMergeWarps * 32) {
    const int64_t c = shared_rest_cost(p, shared_len(p, x, &bad));
    all += c;
    if (x < b) before += c;
  }
  all = warp_sum(all);
  before = warp_sum(before);
  if (lane == 0) {
    sums[0][warp] = all;
    sums[1][warp] = before;
  }
  __syncthreads();
  if (h >= p.Hq) return;  // (counts as having let the next kernel start)
  all = before = 0;
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) {
    all += sums[0][i];
    before += sums[1][i];
  }
  const int kvh = h / p.g, ht = h % p.g / p.gt, j = h % p.g % p.gt;
  const SharedPrefix pre = shared_prefix(p);
  const int L = shared_len(p, b, &bad), Lp = p.n_shared << p.bs_log2;
  const int64_t hh = (int64_t)p.Hkv * p.HT;
  const int64_t q = shared_div(pre.total + all * hh + p.ctas - 1, p.ctas);

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
    const int64_t cost = shared_rest_cost(p, L);
    const int k = kvh * p.HT + ht;
    ri = make(pre.total + before * hh + k * cost, cost, p.w_rest, (L - Lp + kSharedChunk - 1) / kSharedChunk,
              p.rest_row0 + ((int64_t)b * p.Hkv * p.HT + k) * p.rest_rows, p.rest_rows, p.gt, j);
  }
  float m = -INFINITY, l = 0.f, acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the partials are written
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the next kernel's start may be beside what is left
  for (int i0 = 0; i0 < pi.n + ri.n; i0 += 32) {  // lane: one candidate
    const int i = i0 + lane;
    float s = -INFINITY;
    uint32_t r = 0;  // (2^32 part rows would be a workspace of a terabyte)
    if (i < pi.n + ri.n) {
      const Item &it = i < pi.n ? pi : ri;
      const int x = i < pi.n ? i : i - pi.n;
      const int64_t c = it.cta0 + x / it.accs;
      const int a = x % it.accs;
      const int n = shared_cut(p, (c + 1) * q - it.start, it.w, it.chunks) -
                    shared_cut(p, c * q - it.start, it.w, it.chunks);
      if (a < n) {
        r = (uint32_t)(it.part + c * it.stride + a * it.rows);
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
    constexpr int kFlight = 32 / VEC;
    while (todo != 0) {  // several partials in flight
      float o[kFlight][VEC], wj[kFlight];
#pragma unroll
      for (int y = 0; y < kFlight; ++y) {
        const int jl = todo != 0 ? __ffs(todo) - 1 : 0;
        const uint32_t rj = __shfl_sync(0xffffffffu, r, jl);
        wj[y] = todo != 0 ? __shfl_sync(0xffffffffu, w, jl) : 0.f;
        if (todo != 0) {
          const float *src = p.o_part + (int64_t)rj * D + col;
          if constexpr (VEC == 2) {
            const float2 f = *reinterpret_cast<const float2 *>(src);
            o[y][0] = f.x, o[y][1] = f.y;
          } else {
#pragma unroll
            for (int x = 0; x < VEC; x += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(src + x);
              o[y][x] = f.x, o[y][x + 1] = f.y, o[y][x + 2] = f.z, o[y][x + 3] = f.w;
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < VEC; ++x) o[y][x] = 0.f;
        }
        todo &= todo - 1;
      }
#pragma unroll
      for (int y = 0; y < kFlight; ++y)
#pragma unroll
        for (int x = 0; x < VEC; ++x) acc[x] += wj[y] * o[y][x];
    }
  }
  // No weight at all: no token, or scores of -inf alone.  (A row whose scores are NaN has
  // m = -inf too, as a maximum passes them over, but l is NaN then, and so is its lse.)
  const bool none = m == -INFINITY && l == 0.f;
  float lse2 = none ? -INFINITY : m + log2f(l);
  if (p.sinks != nullptr) {
    const float sg = p.sinks[h] * kLog2e;
    const float top = fmaxf(m, sg);
    const float z = (none ? 0.f : l * exp2f(m - top)) + (sg == -INFINITY ? 0.f : exp2f(sg - top));
    lse2 = top + log2f(z);
  }
  const float w = none ? 0.f : exp2f(m - lse2) * p.v_scale;
  uint16_t *o = p.out + b * p.o_sb + (int64_t)h * p.o_sh + col;
#pragma unroll
  for (int i = 0; i < VEC; i += 2)
    *reinterpret_cast<uint32_t *>(o + i) = pack_bf16x2(acc[i] * w, acc[i + 1] * w);
  if (col == 0 && p.lse != nullptr) p.lse[b * p.lse_sb + (int64_t)h * p.lse_sh] = lse2 * kLn2;
}

template <int D, bool F8>
cudaError_t launch_t(const SharedParams &p, cudaStream_t s) {
  using C = SharedCfg<D, F8>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(shared_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  // Both come up beside the kernel before them, and wait for it before their first use
  // of memory that it may write (6 sequences behind 1040 tokens 13.4 -> 12.5 us, 131 of 32
  // heads behind 4096 37.6 -> 36.3).
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::total;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, shared_kernel<D, F8>, p)) != cudaSuccess) return e;
  // Two elements a lane, so more warps for a row, each with more of its partials in
  // flight, while all the warps fit the SMs at once (24 each: three CTAs of 80 registers a
  // thread at head_dim 64 and 128, and at 256, where 94 allow two, the sizes below gain
  // with the same bound); four beyond.  Two against four: 24
  // sequences of 16 heads of 256 31.7 / 32.5 us in all, 48 of 32 of 128 43.1 / 44.2;
  // 64 of 40 of 128 52.6 / 49.7, 131 of 32 40.5 / 37.8.
  constexpr int kWide = D == 64 ? 2 : 4, kFine = 2;
  const int64_t fine_warps = (int64_t)p.B * p.Hq * (D / (32 * kFine));
  const bool fine = fine_warps <= (int64_t)p.ctas * 24;
  cfg.gridDim = dim3((unsigned)p.B * (unsigned)merge_ctas(p.Hq, D / (32 * (fine ? kFine : kWide))));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return fine ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, kFine>, p)
              : cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, kWide>, p);
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
