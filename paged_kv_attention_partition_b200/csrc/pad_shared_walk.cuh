// Device side of the work line of pad_shared.h: the units of a CTA, and what the
// merge needs to find a row's units again (both from the lengths alone).
#pragma once

#include "pad_shared.h"

namespace pad {

struct SharedUnit {
  int32_t rest;         // 0: prefix, 1: rest
  int32_t kvh, ht;
  int32_t b0, nb;       // sequences b0 .. b0 + nb - 1
  int32_t rows;         // nb * gt
  int32_t fold;         // 1: a later piece of a long unit, added to what the part rows hold
  int32_t tok0, tok1;   // tokens, tok0 a chunk's start
  int32_t chunks;
  int64_t part;         // first part row
};

// Costs fit 32 bits but for the very largest problems, and a 64-bit division is
// tens of instructions.
__device__ __forceinline__ int64_t shared_div(int64_t a, int64_t b) {
  return ((uint64_t)a | (uint64_t)b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A sequence's length as the kernels use it: outside [0, capacity], or shorter
// than the prefix it claims, is an error; it counts as the nearest valid one (0
// for a sequence shorter than the prefix).
__device__ __forceinline__ int shared_len(const SharedParams &p, int b, bool *bad) {
  const int cap = p.max_blocks << p.bs_log2, Lp = p.n_shared << p.bs_log2;
  const int L = __ldg(p.seq_lens + b);
  *bad = L < 0 || L > cap || (L > 0 && L < Lp);
  return L > cap ? cap : L < Lp ? 0 : L;
}

// Cost of a rest item of a sequence of this length.
__device__ __forceinline__ int64_t shared_rest_cost(const SharedParams &p, int L) {
  const int n = L - (p.n_shared << p.bs_log2);
  return n <= 0 ? 0 : p.w_item + (int64_t)((n + kSharedChunk - 1) / kSharedChunk) * p.w_rest;
}

// The prefix part of the line: items (kvh, ht, rb), rb innermost; every row block
// is full but the last.
struct SharedPrefix {
  int chunks, last_nb;
  int64_t full, last, group, total;  // costs: a full block's item, the last one's, a (kvh, ht)'s, all
};
__device__ __forceinline__ SharedPrefix shared_prefix(const SharedParams &p) {
  SharedPrefix s;
  s.chunks = ((p.n_shared << p.bs_log2) + kSharedChunk - 1) / kSharedChunk;
  s.last_nb = p.B - (p.nrb - 1) * p.nseq;
  auto cost = [&](int nb) -> int64_t {
    return s.chunks == 0 ? 0 : p.w_item + (int64_t)s.chunks * (nb * p.gt > kTileRows ? p.w_pre2 : p.w_pre1);
  };
  s.full = cost(p.nseq);
  s.last = cost(s.last_nb);
  s.group = (p.nrb - 1) * s.full + s.last;
  s.total = s.group * p.Hkv * p.HT;
  return s;
}

// First chunk of an item at or behind `at` (a cost counted from the item's start).
__device__ __forceinline__ int shared_cut(const SharedParams &p, int64_t at, int w, int chunks) {
  if (at <= p.w_item) return 0;
  const int64_t c = shared_div(at - p.w_item + w - 1, w);
  return c > chunks ? chunks : (int)c;
}

// Calls emit(unit) for each unit of CTA `cta`, in order, a long one in pieces of
// kSharedPiece chunks; all lanes of a warp call it together, and emit is called by all of
// them with the same unit.
template <int D, class Emit>
__device__ __forceinline__ void shared_walk(const SharedParams &p, int cta, Emit &&emit) {
  constexpr int CT = kSharedChunk;
  const int lane = threadIdx.x & 31;
  auto pieces = [&](SharedUnit &u) {
    const int chunks = u.chunks, tok0 = u.tok0, tok1 = u.tok1;
    for (int c = 0; c < chunks; c += kSharedPiece) {
      u.fold = c > 0;
      u.chunks = min(kSharedPiece, chunks - c);
      u.tok0 = tok0 + c * CT;
      u.tok1 = min(tok1, u.tok0 + u.chunks * CT);
      emit(u);
    }
  };
  const SharedPrefix pre = shared_prefix(p);
  const int Lp = p.n_shared << p.bs_log2;
  const int hh = p.Hkv * p.HT;
  auto length = [&](int b, bool *bad) -> int {
    *bad = false;
    return b < p.B ? shared_len(p, b, bad) : 0;
  };
  int64_t sum = 0;
  bool any_bad = false;
  for (int b = lane; b < p.B; b += 8 * 32) {  // eight loads in flight
    int L[8];
    bool bad[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) L[i] = length(b + 32 * i, &bad[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += shared_rest_cost(p, L[i]);
      any_bad |= bad[i];
    }
  }
  if (any_bad && cta == 0) atomicOr(p.err, kErrSeqLen);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const int64_t total = pre.total + sum * hh;
  const int64_t q = shared_div(total + p.ctas - 1, p.ctas);
  int64_t pos = cta * q;
  const int64_t end = pos + q < total ? pos + q : total;

  while (pos < end && pos < pre.total) {
    const int grp = (int)shared_div(pos, pre.group);
    const int64_t in = pos - grp * pre.group;
    int rb = (int)shared_div(in, pre.full);
    if (rb > p.nrb - 1) rb = p.nrb - 1;
    const int64_t start = grp * pre.group + rb * pre.full;
    SharedUnit u;
    u.rest = 0;
    u.kvh = grp / p.HT;
    u.ht = grp % p.HT;
    u.b0 = rb * p.nseq;
    u.nb = rb == p.nrb - 1 ? pre.last_nb : p.nseq;
    u.rows = u.nb * p.gt;
    const int w = u.rows > kTileRows ? p.w_pre2 : p.w_pre1;
    const int c0 = shared_cut(p, pos - start, w, pre.chunks), c1 = shared_cut(p, end - start, w, pre.chunks);
    u.tok0 = c0 * CT;
    u.tok1 = min(c1 * CT, Lp);
    u.chunks = c1 - c0;
    u.part = ((int64_t)grp * p.nrb + rb + cta) * p.pre_rows;
    if (c1 > c0) pieces(u);
    pos = start + (rb == p.nrb - 1 ? pre.last : pre.full);
  }

  int64_t base = pre.total;  // cost before these 32 sequences
  bool bad;
  int next = length(lane, &bad);
  for (int b0 = 0; b0 < p.B && pos < end; b0 += 32) {
    const int L = next;
    next = length(b0 + 32 + lane, &bad);  // in flight meanwhile
    const int64_t item = shared_rest_cost(p, L);
    int64_t incl = item * hh;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const int64_t first = base + incl - item * hh;
    uint32_t todo = __ballot_sync(0xffffffffu, item > 0 && first < end && first + item * hh > pos);
    while (todo != 0) {
      const int j = __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t f = __shfl_sync(0xffffffffu, first, j), it = __shfl_sync(0xffffffffu, item, j);
      const int Lj = __shfl_sync(0xffffffffu, L, j);
      const int chunks = (Lj - Lp + CT - 1) / CT;
      while (pos < end && pos < f + it * hh) {
        const int k = (int)shared_div(pos - f, it);
        const int64_t start = f + k * it;
        SharedUnit u;
        u.rest = 1;
        u.kvh = k / p.HT;
        u.ht = k % p.HT;
        u.b0 = b0 + j;
        u.nb = 1;
        u.rows = p.gt;
        const int c0 = shared_cut(p, pos - start, p.w_rest, chunks), c1 = shared_cut(p, end - start, p.w_rest, chunks);
        u.tok0 = Lp + c0 * CT;
        u.tok1 = min(Lp + c1 * CT, Lj);
        u.chunks = c1 - c0;
        u.part = p.rest_row0 + (((int64_t)u.b0 * hh + k) + cta) * p.rest_rows;
        if (c1 > c0) pieces(u);
        pos = start + it;
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

}  // namespace pad
