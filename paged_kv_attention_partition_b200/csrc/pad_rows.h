// Launch parameters of the per-head row kernel: norm, rotation and the append.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pad {

struct RowsParams {
  int64_t T;
  int32_t Hq, Hkv;  // rows of q (0: none) and of k (and v) per token
  const uint16_t *q, *k, *v;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // element strides over (token, head)
  const void *qw, *kw;                          // norm weights (null: no norm)
  int32_t qw_f32, kw_f32;                       // 1: fp32 weights, 0: bf16
  float eps;
  const int32_t *positions;
  const float *inv_freq;  // null: no rotation
  int32_t rot;            // rotary dims, a multiple of 16
  int32_t interleaved;
  uint16_t *q_out, *k_out;
  int64_t qo_st, qo_sh, ko_st, ko_sh;
  // the append's caches (element strides over block, head, slot)
  void *kc, *vc;
  int64_t kc_sb, kc_sh, kc_ss, vc_sb, vc_sh, vc_ss;
  const int32_t *tables;
  int64_t table_stride;
  const int32_t *seq_ids;  // null: token t is sequence t's
  int32_t B, max_blocks, num_blocks, bs_log2;
  float k_scale, v_scale;
  int32_t steps_per_warp;
  uint32_t *err;
};

enum RowsMode { kRowsOut = 0, kRowsCacheBf16 = 1, kRowsCacheE4m3 = 2 };

cudaError_t launch_rows(const RowsParams &p, int D, int mode, int sms, cudaStream_t s);

}  // namespace pad
