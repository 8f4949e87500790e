// Shared-prefix decode (pad_decode_shared): partial softmax over the units of
// the work line (pad_shared.h), then one merge of each query row's partials.
//
// Per unit and row, over the unit's tokens:  m = max s, l = sum 2^(s - m),
//   o = sum 2^(s - m) v / l,  lse2 = m + log2 l   (s = scale * log2(e) * q.k)
// and per row over its units:  out = sum 2^(lse2_u - lse2) o_u.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pad_device.cuh"
#include "pad_shared.h"
#include "pad_shared_walk.cuh"

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
  const int64_t q = p.cum[p.B];

  float m = -INFINITY, l = 0.f, acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  auto add = [&](int64_t r) {
    const float s = p.lse_part[r];
    if (s == -INFINITY) return;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = acc[i] * a + w * p.o_part[r * D + lane * VEC + i];
  };
  auto item = [&](int64_t start, int64_t cost, int w, int chunks, int64_t part0, int stride, int rows, int r) {
    const int accs = shared_part_rows(rows, D) / rows;
    for (int64_t c = start / q; c <= (start + cost - 1) / q; ++c) {
      const int n = shared_cut(p, (c + 1) * q - start, w, chunks) - shared_cut(p, c * q - start, w, chunks);
      for (int a = 0; a < accs && a < n; ++a) add(part0 + c * stride + a * rows + r);
    }
  };
  if (L > 0 && pre.chunks > 0) {
    const int grp = kvh * p.HT + ht, rb = b / p.nseq;
    const bool lastrb = rb == p.nrb - 1;
    const int rows = (lastrb ? pre.last_nb : p.nseq) * p.gt;
    item(grp * pre.group + rb * pre.full, lastrb ? pre.last : pre.full, rows > kTileRows ? p.w_pre2 : p.w_pre1,
         pre.chunks, ((int64_t)grp * p.nrb + rb) * p.pre_rows, p.pre_rows, rows, (b - rb * p.nseq) * p.gt + j);
  }
  if (L > Lp) {
    const int64_t cost = shared_rest_cost<D>(p, L);
    const int k = kvh * p.HT + ht;
    item(p.cum[b] + k * cost, cost, p.w_rest, (L - Lp + shared_chunk(D) - 1) / shared_chunk(D),
         p.rest_row0 + ((int64_t)b * p.Hkv * p.HT + k) * p.rest_rows, p.rest_rows, p.gt, j);
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
  shared_kernel<D, F8><<<p.ctas, 256, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.B * p.Hq;
  shared_merge_kernel<D><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(p);
  return cudaGetLastError();
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
