// Per-head rows: RMS norm, position rotation, and the append into the paged
// cache, in one pass over the rows (pad_qk_norm_rope, pad_append_kv).
//
//   n = x * rsqrt(mean(x^2) + eps) * w
//   (y1, y2) = (n1 cos a - n2 sin a, n2 cos a + n1 sin a),   a = position * inv_freq[i]
// in fp32, rounded once to the output's type.
//
// D / 16 lanes share a row: lane c holds two 16-byte chunks whose elements
// rotate with one another (half style: chunk c of the first half and chunk c of
// the second; neighbours: any), so the rotation needs no exchange between lanes
// and the norm one reduction over D / 16 lanes.  A warp keeps one token, so its
// angles are computed once for all the heads it handles.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pad_device.cuh"
#include "pad_internal.h"
#include "pad_rows.h"

namespace pad {
namespace {

constexpr int kRowsWarps = 4;

__device__ __forceinline__ void unpack8(const uint4 &c, float (&x)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// Two E4M3 codes, round to nearest even, beyond +-448 to +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  return make_uint2(e4m3x2(x[0] / scale, x[1] / scale) | e4m3x2(x[2] / scale, x[3] / scale) << 16,
                    e4m3x2(x[4] / scale, x[5] / scale) | e4m3x2(x[6] / scale, x[7] / scale) << 16);
}
__device__ __forceinline__ float weight_at(const void *w, int f32, int i) {
  return f32 ? __ldg(static_cast<const float *>(w) + i)
             : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(w) + i) << 16);
}
// cos and sin of position * freq.  The product and its reduction to half turns
// are in 64 bits: in 32 a position of 10^5 alone would lose the angle's last two
// decimal digits.
__device__ __forceinline__ void angle(int pos, float freq, float &c, float &s) {
  double half_turns = (double)pos * (double)freq * 0.31830988618379067154;  // / pi
  half_turns -= 2.0 * rint(half_turns * 0.5);
  sincospif((float)half_turns, &s, &c);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kRowsWarps * 32) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes per row, rows per warp step
  constexpr bool kCache = MODE != kRowsOut;
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int rows = p.Hq + p.Hkv * (kCache ? 2 : 1);
  const int steps = (rows + RPW - 1) / RPW;
  const int parts = (steps + p.steps_per_warp - 1) / p.steps_per_warp;
  const int64_t w = (int64_t)blockIdx.x * kRowsWarps + (threadIdx.x >> 5);
  const int64_t t = w / parts;
  if (t >= p.T) return;
  const int s0 = (int)(w % parts) * p.steps_per_warp, s1 = min(s0 + p.steps_per_warp, steps);

  // this lane's chunks: a rotating pair (half style), or two neighbours
  const int hc = p.inv_freq != nullptr ? p.rot / 16 : 0;  // rotating chunk pairs
  const bool turn = c < hc;
  int c0 = 2 * c, c1 = 2 * c + 1;
  if (turn && !p.interleaved) {
    c0 = c;
    c1 = c + hc;
  }
  float cs[8], sn[8];
  if (turn) {
    const int pos = __ldg(p.positions + t);
#pragma unroll
    for (int i = 0; i < 8; ++i) angle(pos, __ldg(p.inv_freq + 8 * c + i), cs[i], sn[i]);
  }
  // where the token goes; block < 0: nowhere
  int block = -1, slot = 0;
  if (kCache) {
    const int seq = p.seq_ids != nullptr ? __ldg(p.seq_ids + t) : (int)t;
    if (seq >= 0) {
      const int pos = __ldg(p.positions + t);
      const bool seq_ok = seq < p.B, pos_ok = pos >= 0 && (pos >> p.bs_log2) < p.max_blocks;
      if (seq_ok && pos_ok) {
        block = __ldg(p.tables + seq * p.table_stride + (pos >> p.bs_log2));
        slot = pos & ((1 << p.bs_log2) - 1);
      }
      if (block < 0 || block >= p.num_blocks) {
        if (lane == 0) atomicOr(p.err, seq_ok && !pos_ok ? kErrSeqLen : kErrBlockId);
        block = -1;
      }
    }
  }

  for (int st = s0; st < s1; ++st) {
    const int r = st * RPW + sub;
    const bool live = r < rows;
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
    const int h = is_q ? r : is_v ? r - p.Hq - p.Hkv : r - p.Hq;
    const uint16_t *src = is_q ? p.q + t * p.q_st + h * p.q_sh
                               : is_v ? p.v + t * p.v_st + h * p.v_sh : p.k + t * p.k_st + h * p.k_sh;
    float x[8], y[8];
    float ss = 0.f;
    if (live) {
      unpack8(*reinterpret_cast<const uint4 *>(src + c0 * 8), x);
      unpack8(*reinterpret_cast<const uint4 *>(src + c1 * 8), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (!live) continue;
    const void *wt = is_q ? p.qw : is_v ? nullptr : p.kw;
    if (wt != nullptr) {
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const int f32 = is_q ? p.qw_f32 : p.kw_f32;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= inv * weight_at(wt, f32, c0 * 8 + i);
        y[i] *= inv * weight_at(wt, f32, c1 * 8 + i);
      }
    }
    if (turn && !is_v) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x1 = x[2 * i], x2 = x[2 * i + 1], y1 = y[2 * i], y2 = y[2 * i + 1];
          x[2 * i] = x1 * cs[i] - x2 * sn[i];
          x[2 * i + 1] = x2 * cs[i] + x1 * sn[i];
          y[2 * i] = y1 * cs[4 + i] - y2 * sn[4 + i];
          y[2 * i + 1] = y2 * cs[4 + i] + y1 * sn[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x1 = x[i], x2 = y[i];
          x[i] = x1 * cs[i] - x2 * sn[i];
          y[i] = x2 * cs[i] + x1 * sn[i];
        }
      }
    }
    if (is_q || !kCache) {
      uint16_t *o = is_q ? p.q_out + t * p.qo_st + h * p.qo_sh : p.k_out + t * p.ko_st + h * p.ko_sh;
      *reinterpret_cast<uint4 *>(o + c0 * 8) = pack8(x);
      *reinterpret_cast<uint4 *>(o + c1 * 8) = pack8(y);
    } else if (block >= 0) {
      const int64_t at = is_v ? block * p.vc_sb + h * p.vc_sh + slot * p.vc_ss
                              : block * p.kc_sb + h * p.kc_sh + slot * p.kc_ss;
      if constexpr (MODE == kRowsCacheE4m3) {
        uint8_t *o = static_cast<uint8_t *>(is_v ? p.vc : p.kc) + at;
        const float sc = is_v ? p.v_scale : p.k_scale;
        *reinterpret_cast<uint2 *>(o + c0 * 8) = pack8_e4m3(x, sc);
        *reinterpret_cast<uint2 *>(o + c1 * 8) = pack8_e4m3(y, sc);
      } else {
        uint16_t *o = static_cast<uint16_t *>(is_v ? p.vc : p.kc) + at;
        *reinterpret_cast<uint4 *>(o + c0 * 8) = pack8(x);
        *reinterpret_cast<uint4 *>(o + c1 * 8) = pack8(y);
      }
    }
  }
}

template <int D, int MODE>
cudaError_t launch_t(RowsParams p, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (D / 16);
  const int rows = p.Hq + p.Hkv * (MODE != kRowsOut ? 2 : 1), steps = (rows + RPW - 1) / RPW;
  // One step per warp while the launch has room for it (latency), then as many
  // of a token's heads per warp as keep every SM at 16 warps: each further step
  // reuses the warp's angles.
  int64_t spw = p.T * steps / ((int64_t)sms * 16);
  p.steps_per_warp = (int)(spw < 1 ? 1 : spw > steps ? steps : spw);
  const int64_t warps = p.T * ((steps + p.steps_per_warp - 1) / p.steps_per_warp);
  const int64_t grid = (warps + kRowsWarps - 1) / kRowsWarps;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  rows_kernel<D, MODE><<<(unsigned)grid, kRowsWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RowsParams &p, int mode, int sms, cudaStream_t s) {
  return mode == kRowsOut ? launch_t<D, kRowsOut>(p, sms, s)
         : mode == kRowsCacheBf16 ? launch_t<D, kRowsCacheBf16>(p, sms, s) : launch_t<D, kRowsCacheE4m3>(p, sms, s);
}

}  // namespace

cudaError_t launch_rows(const RowsParams &p, int D, int mode, int sms, cudaStream_t s) {
  switch (D) {
    case 64: return launch_d<64>(p, mode, sms, s);
    case 128: return launch_d<128>(p, mode, sms, s);
    case 256: return launch_d<256>(p, mode, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pad
