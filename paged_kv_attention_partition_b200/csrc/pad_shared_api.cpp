// Host side of pad_decode_shared: argument validation, the workspace, the
// launch.  Declared in include/pad.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pad.h"
#include "pad_host.h"
#include "pad_internal.h"
#include "pad_shared.h"

namespace {

using pad::host_fail;

struct Shape {
  int64_t B, Hq, Hkv, D, bs, W, n;
  bool fp8;
};

pad_status check_shape(const Shape &s) {
  if (s.n < 0 || s.n > s.W)
    return host_fail(PAD_ERR_INVALID_ARG, "shared_table has %lld pages, a table row holds %lld", (long long)s.n,
                     (long long)s.W);
  return pad::host_check_shape(s.B, s.Hq, s.Hkv, s.D, s.bs, s.W);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t o_part, lse_part, total;
};

// Geometry and scratch of one shape: how rows are grouped into units, and room
// for every (item, CTA) number's part rows.
Layout layout(const Shape &s, int ctas, pad::SharedParams *p) {
  const int64_t g = s.Hq / s.Hkv, R = pad::shared_rows((int)s.D);
  const int64_t gt = g < R ? g : R;
  p->B = (int32_t)s.B;
  p->Hq = (int32_t)s.Hq;
  p->Hkv = (int32_t)s.Hkv;
  p->g = (int32_t)g;
  p->gt = (int32_t)gt;
  p->HT = (int32_t)((g + gt - 1) / gt);
  int64_t nseq = p->HT > 1 ? 1 : R / gt;
  if (nseq > s.B) nseq = s.B > 0 ? s.B : 1;
  p->nseq = (int32_t)nseq;
  p->nrb = (int32_t)((s.B + nseq - 1) / nseq);
  p->ctas = ctas;
  p->n_shared = (int32_t)s.n;
  p->max_blocks = (int32_t)s.W;
  p->bs_log2 = 0;
  while ((1ll << p->bs_log2) < s.bs) ++p->bs_log2;
  // In hundreds of cycles: begun with the kernel's own clocks on B200, then swept on
  // seven bf16 and six E4M3 shapes (head_dim 64 to 256, 6 to 256 sequences).  bf16, 64
  // sequences of 40 / 8 heads behind 8192 tokens and 256 of 32 / 8 behind 32768:
  // 30 / 11 / 20 / 11 51.9 and 196 us, 40 / 11 / 20 / 9 49.8 and 196, 20 / 11 / 20 / 9
  // 47.8 and 225: the shapes pull apart (equal cuts keep row blocks of a long prefix in
  // step, cheap items spread short rests), and these are between.  E4M3, 48 sequences of
  // 32 / 8 heads behind 6000 tokens: 80 / 14 / 26 / 18 46.7 us, 60 / 14 / 26 / 14 43.3.
  p->w_item = s.fp8 ? 60 : 40;
  p->w_pre1 = s.fp8 ? 14 : 11;
  p->w_pre2 = s.fp8 ? 26 : 20;
  p->w_rest = s.fp8 ? 14 : 9;
  const int full = pad::shared_part_rows((int)(nseq * gt), (int)s.D);
  const int last = pad::shared_part_rows((int)((s.B - (p->nrb - 1) * nseq) * gt), (int)s.D);
  p->pre_rows = full > last ? full : last;
  p->rest_rows = pad::shared_part_rows((int)gt, (int)s.D);
  const int64_t groups = s.Hkv * p->HT;
  const int64_t pre_units = s.n > 0 ? groups * p->nrb + ctas : 0;
  p->rest_row0 = pre_units * p->pre_rows;
  const int64_t rows = p->rest_row0 + (s.B * groups + ctas) * p->rest_rows;
  Layout l;
  l.o_part = 0;
  l.lse_part = align256((size_t)(rows * s.D * 4));
  l.total = l.lse_part + align256((size_t)(rows * 4));
  return l;
}

// How a cache's pages are copied (SharedBox), K and V alike.
void choose_box(const pad_tensor *k, const pad_tensor *v, int chunk, pad::SharedParams *p) {
  const int64_t NB = k->shape[0], H = k->shape[1], bs = k->shape[2];
  p->blk_heads = 1;
  if (k->dtype == PAD_FP8_E4M3) {
    p->box_log2 = 0;
    while ((1 << p->box_log2) < chunk && (1 << p->box_log2) < bs) ++p->box_log2;
    p->box_pitch = (int32_t)(k->shape[3] << p->box_log2);
    if (p->box_pitch < 128) p->box_pitch = 128;
    return;
  }
  if (bs < 8) {
    p->box_kind = pad::kBoxRows;
    p->box_log2 = p->bs_log2;
    return;
  }
  p->box_kind = pad::kBoxGroup;
  p->box_log2 = 3;
  // block and head as one coordinate, block * (block stride / head stride) + head
  auto ratio = [&](const pad_tensor *t) -> int64_t {
    if (NB == 1) return H;
    if (H == 1) return 1;
    return t->stride[1] > 0 && t->stride[0] % t->stride[1] == 0 ? t->stride[0] / t->stride[1] : 0;
  };
  const int64_t r = ratio(k);
  if (r < H || r != ratio(v) || NB * r + H > 0x7fffffffll) return;  // (r >= H: block num_blocks is out of range)
  p->box_kind = pad::kBoxPage;
  p->blk_heads = (int32_t)r;
  while ((1 << p->box_log2) < chunk && (1 << p->box_log2) < bs) ++p->box_log2;
}

// A cache's tensor map for the boxes of `p`: bf16 with the 128-byte swizzle, E4M3
// codes as they are (they are widened on the way to the operand).
pad_status cache_map(CUtensorMap *map, const pad_tensor *t, const pad::SharedParams &p, const char *name) {
  pad::TensorMapEncodeFn enc = pad::host_tensor_map_encoder();
  if (enc == nullptr) return host_fail(PAD_ERR_CUDA, "the CUDA driver does not provide cuTensorMapEncodeTiled");
  const cuuint64_t NB = t->shape[0], H = t->shape[1], bs = t->shape[2], CB = t->shape[3] / 64;
  const bool fp8 = t->dtype == PAD_FP8_E4M3;
  const int64_t eb = fp8 ? 1 : 2;
  auto bytes = [&](int i, int64_t natural) { return (cuuint64_t)(t->shape[i] > 1 ? t->stride[i] * eb : natural); };
  const cuuint64_t row = bytes(2, t->shape[3] * eb), head = bytes(1, bs * row), block = bytes(0, H * head);
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  CUresult r;
  if (fp8) {
    const cuuint64_t dims[4] = {(cuuint64_t)t->shape[3], bs, H, NB};
    const cuuint64_t strides[3] = {row, head, block};
    const cuuint32_t box[4] = {(cuuint32_t)t->shape[3], (cuuint32_t)(1 << p.box_log2), 1, 1};
    r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, t->data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else if (p.box_kind == pad::kBoxPage) {
    const cuuint64_t dims[5] = {64, 8, CB, bs / 8, (NB - 1) * p.blk_heads + H};
    const cuuint64_t strides[4] = {row, 128, 8 * row, H > 1 ? head : block};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)CB, (cuuint32_t)(1 << p.box_log2) / 8, 1};
    r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, t->data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[5] = {64, bs, CB, H, NB};
    const cuuint64_t strides[4] = {row, 128, head, block};
    const cuuint32_t box[5] = {64, (cuuint32_t)(1 << p.box_log2), p.box_kind == pad::kBoxGroup ? (cuuint32_t)CB : 1, 1,
                               1};
    r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, t->data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS)
    return host_fail(PAD_ERR_INVALID_ARG, "%s: strides/shape not expressible as a TMA tensor (cuTensorMapEncodeTiled %d)",
                     name, (int)r);
  return PAD_OK;
}

// q as (64 head_dim elements, head, the rest of head_dim, sequence), boxes of 64
// x `heads` x 1 x `seqs`.
pad_status query_map(CUtensorMap *map, const pad_tensor *q, int heads, int seqs) {
  pad::TensorMapEncodeFn enc = pad::host_tensor_map_encoder();
  if (enc == nullptr) return host_fail(PAD_ERR_CUDA, "the CUDA driver does not provide cuTensorMapEncodeTiled");
  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const cuuint64_t dims[4] = {64, (cuuint64_t)Hq, (cuuint64_t)(D / 64), (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)(Hq > 1 ? q->stride[1] * 2 : D * 2), 128,
                                 (cuuint64_t)(B > 1 ? q->stride[0] * 2 : Hq * D * 2)};
  const cuuint32_t box[4] = {64, (cuuint32_t)heads, 1, (cuuint32_t)seqs}, one[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q->data, dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return host_fail(PAD_ERR_INVALID_ARG, "q: strides/shape not expressible as a TMA tensor (%d)", (int)r);
  return PAD_OK;
}

// The current device, its context made current too: in a thread that has made no
// CUDA call of its own yet the tensor-map encoder, a driver call, would find none.
pad_status current_device(int *device) {
  cudaError_t e = cudaGetDevice(device);
  if (e == cudaSuccess) e = cudaSetDevice(*device);
  return e == cudaSuccess ? PAD_OK : pad::host_cuda_fail(e, "cudaGetDevice");
}

}  // namespace

extern "C" pad_status pad_decode_shared_plan(int64_t batch, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                                             int64_t block_size, int64_t max_blocks_per_seq, int64_t shared_blocks,
                                             int32_t kv_dtype, int32_t device, pad_shared_plan *plan) {
  if (plan == nullptr) return host_fail(PAD_ERR_INVALID_ARG, "plan is NULL");
  if (kv_dtype != PAD_BF16 && kv_dtype != PAD_FP8_E4M3)
    return host_fail(PAD_ERR_INVALID_ARG, "kv_dtype must be PAD_BF16 or PAD_FP8_E4M3 (got %d)", kv_dtype);
  const Shape s{batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, shared_blocks,
                kv_dtype == PAD_FP8_E4M3};
  pad_status st = check_shape(s);
  if (st != PAD_OK) return st;
  if (device < 0) {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) {
      cudaGetLastError();
      d = -1;
    }
    device = d;
  }
  pad::SharedParams p{};
  const Layout l = layout(s, pad::host_sm_count(device < 0 ? 0 : device), &p);
  plan->ctas = p.ctas;
  plan->chunk_tokens = pad::kSharedChunk;
  plan->prefix_rows = p.nseq * p.gt;
  plan->prefix_blocks = p.nrb * p.HT;
  plan->workspace_bytes = batch == 0 ? 0 : (int64_t)l.total;
  return PAD_OK;
}

extern "C" pad_status pad_decode_shared(const pad_tensor *q, const pad_tensor *k_cache, const pad_tensor *v_cache,
                                        const pad_tensor *shared_table, const pad_tensor *block_tables,
                                        const pad_tensor *seq_lens, float scale, const pad_decode_options *options,
                                        pad_tensor *out, pad_tensor *lse, void *workspace, size_t workspace_bytes,
                                        void *stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  pad_status st;
  if ((st = pad::host_check_tensor(q, "q", PAD_BF16, 3)) != PAD_OK) return st;
  const bool fp8 = k_cache != nullptr && k_cache->dtype == PAD_FP8_E4M3;
  const pad_dtype kv = fp8 ? PAD_FP8_E4M3 : PAD_BF16;
  if ((st = pad::host_check_tensor(k_cache, "k_cache", kv, 4)) != PAD_OK) return st;
  if ((st = pad::host_check_tensor(v_cache, "v_cache", kv, 4)) != PAD_OK) return st;
  if (shared_table == nullptr) return host_fail(PAD_ERR_INVALID_ARG, "shared_table is NULL");
  const bool some = shared_table->ndim != 1 || shared_table->shape[0] != 0;  // an empty one may have no data
  if (some && (st = pad::host_check_tensor(shared_table, "shared_table", PAD_I32, 1)) != PAD_OK) return st;
  if ((st = pad::host_check_tensor(block_tables, "block_tables", PAD_I32, 2)) != PAD_OK) return st;
  if ((st = pad::host_check_tensor(seq_lens, "seq_lens", PAD_I32, 1)) != PAD_OK) return st;
  if ((st = pad::host_check_tensor(out, "out", PAD_BF16, 3)) != PAD_OK) return st;
  if (lse != nullptr && (st = pad::host_check_tensor(lse, "lse", PAD_F32, 2)) != PAD_OK) return st;

  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t NB = k_cache->shape[0], Hkv = k_cache->shape[1], bs = k_cache->shape[2];
  for (int i = 0; i < 4; ++i)
    if (v_cache->shape[i] != k_cache->shape[i])
      return host_fail(PAD_ERR_INVALID_ARG, "v_cache.shape[%d]=%lld differs from k_cache", i,
                       (long long)v_cache->shape[i]);
  if (k_cache->shape[3] != D)
    return host_fail(PAD_ERR_INVALID_ARG, "k_cache head_dim %lld != q head_dim %lld", (long long)k_cache->shape[3],
                     (long long)D);
  if (shared_table->shape[0] > 1 && shared_table->stride[0] != 1)
    return host_fail(PAD_ERR_INVALID_ARG, "shared_table must be contiguous");
  if (block_tables->shape[0] != B || (block_tables->stride[1] != 1 && block_tables->shape[1] > 1))
    return host_fail(PAD_ERR_INVALID_ARG, "block_tables must be [%lld, blocks] with contiguous rows", (long long)B);
  if (seq_lens->shape[0] != B || (seq_lens->stride[0] != 1 && B > 1))
    return host_fail(PAD_ERR_INVALID_ARG, "seq_lens must be contiguous [%lld]", (long long)B);
  if (out->shape[0] != B || out->shape[1] != Hq || out->shape[2] != D)
    return host_fail(PAD_ERR_INVALID_ARG, "out shape must equal q shape [%lld, %lld, %lld]", (long long)B,
                     (long long)Hq, (long long)D);
  if (lse != nullptr && (lse->shape[0] != B || lse->shape[1] != Hq))
    return host_fail(PAD_ERR_INVALID_ARG, "lse shape must be [B, Hq] = [%lld, %lld]", (long long)B, (long long)Hq);
  if (!isfinite(scale)) return host_fail(PAD_ERR_INVALID_ARG, "scale must be finite");
  if (NB <= 0 || NB > 0x7fffffffll) return host_fail(PAD_ERR_INVALID_ARG, "num_blocks %lld out of range", (long long)NB);
  if ((st = pad::host_check_rows16(q, "q", 2)) != PAD_OK) return st;
  if ((st = pad::host_check_rows16(k_cache, "k_cache", fp8 ? 1 : 2)) != PAD_OK) return st;
  if ((st = pad::host_check_rows16(v_cache, "v_cache", fp8 ? 1 : 2)) != PAD_OK) return st;
  if ((st = pad::host_check_rows16(out, "out", 2)) != PAD_OK) return st;
  if (reinterpret_cast<uintptr_t>(shared_table->data) % 4 || reinterpret_cast<uintptr_t>(block_tables->data) % 4 ||
      reinterpret_cast<uintptr_t>(seq_lens->data) % 4 || (lse != nullptr && reinterpret_cast<uintptr_t>(lse->data) % 4))
    return host_fail(PAD_ERR_INVALID_ARG, "int32/fp32 tensors must be 4-byte aligned");
  const Shape s{B, Hq, Hkv, D, bs, block_tables->shape[1], shared_table->shape[0], fp8};
  if ((st = check_shape(s)) != PAD_OK) return st;

  float k_scale = 1.f, v_scale = 1.f;
  const pad_tensor *sinks = nullptr;
  if (options != nullptr) {
    if (options->window_left != 0)
      return host_fail(options->window_left < 0 ? PAD_ERR_INVALID_ARG : PAD_ERR_UNSUPPORTED,
                       "window_left must be 0: a window moves with each sequence's length, so it shares no prefix");
    k_scale = options->k_scale == 0.f ? 1.f : options->k_scale;
    v_scale = options->v_scale == 0.f ? 1.f : options->v_scale;
    if (!(isfinite(k_scale) && k_scale > 0.f) || !(isfinite(v_scale) && v_scale > 0.f))
      return host_fail(PAD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive (or 0 for 1)");
    if (!fp8 && (k_scale != 1.f || v_scale != 1.f))
      return host_fail(PAD_ERR_INVALID_ARG, "k_scale / v_scale apply to an E4M3 cache only (bf16 cache: 0 or 1)");
    sinks = options->sinks;
    if (sinks != nullptr) {
      if ((st = pad::host_check_tensor(sinks, "sinks", PAD_F32, 1)) != PAD_OK) return st;
      if (sinks->shape[0] != Hq || (sinks->stride[0] != 1 && Hq > 1) ||
          reinterpret_cast<uintptr_t>(sinks->data) % 4)
        return host_fail(PAD_ERR_INVALID_ARG, "sinks must be contiguous fp32 [Hq] = [%lld]", (long long)Hq);
    }
  }
  if (B == 0) return PAD_OK;

  int device = 0;
  if ((st = current_device(&device)) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(q->data, device, "q")) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(k_cache->data, device, "k_cache")) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(v_cache->data, device, "v_cache")) != PAD_OK) return st;
  if (some && (st = pad::host_check_device_ptr(shared_table->data, device, "shared_table")) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(block_tables->data, device, "block_tables")) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(seq_lens->data, device, "seq_lens")) != PAD_OK) return st;
  if ((st = pad::host_check_device_ptr(out->data, device, "out")) != PAD_OK) return st;
  if (lse != nullptr && (st = pad::host_check_device_ptr(lse->data, device, "lse")) != PAD_OK) return st;
  if (sinks != nullptr && (st = pad::host_check_device_ptr(sinks->data, device, "sinks")) != PAD_OK) return st;

  pad::SharedParams p{};
  const Layout l = layout(s, pad::host_sm_count(device), &p);
  if (workspace != nullptr) {
    if (workspace_bytes < l.total)
      return host_fail(PAD_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes, l.total);
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
      return host_fail(PAD_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if ((st = pad::host_check_device_ptr(workspace, device, "workspace")) != PAD_OK) return st;
  }
  choose_box(k_cache, v_cache, pad::kSharedChunk, &p);
  if ((st = cache_map(&p.tmk, k_cache, p, "k_cache")) != PAD_OK) return st;
  if ((st = cache_map(&p.tmv, v_cache, p, "v_cache")) != PAD_OK) return st;
  if ((st = query_map(&p.tmqp, q, p.gt, p.nseq)) != PAD_OK) return st;
  if ((st = query_map(&p.tmqr, q, p.gt, 1)) != PAD_OK) return st;
  p.shared_table = static_cast<const int32_t *>(shared_table->data);
  p.tables = static_cast<const int32_t *>(block_tables->data);
  p.table_stride = block_tables->stride[0];
  p.seq_lens = static_cast<const int32_t *>(seq_lens->data);
  p.num_blocks = (int32_t)NB;
  p.scale_log2 = (float)((double)scale * (double)k_scale * 1.4426950408889634);
  // a scale of 0 weighs every token alike; the smallest positive one does too, and
  // keeps a masked score, -inf, at -inf
  if (p.scale_log2 == 0.f) p.scale_log2 = pad::kTinyScale;
  p.v_scale = v_scale;
  p.sinks = sinks != nullptr ? static_cast<const float *>(sinks->data) : nullptr;
  p.out = static_cast<uint16_t *>(out->data);
  p.o_sb = out->stride[0];
  p.o_sh = out->stride[1];
  p.lse = lse != nullptr ? static_cast<float *>(lse->data) : nullptr;
  p.lse_sb = lse != nullptr ? lse->stride[0] : 0;
  p.lse_sh = lse != nullptr ? lse->stride[1] : 0;
  cudaError_t e = pad::device_error_word(device, &p.err);
  if (e != cudaSuccess) return pad::host_cuda_fail(e, "error word");
  // Two threads on one stream share its scratch, held over the launches: neither's kernels
  // between the other's two, nor a larger buffer between the other's look and its launches.
  // (A workspace of the caller's needs no lock: another call's kernel between the two only
  // adds to what the merge waits for.)
  pad::ScratchHold scratch;
  if (workspace == nullptr) {
    if ((st = pad::host_scratch(device, stream, l.total, &scratch)) != PAD_OK) return st;
    workspace = scratch.ptr;
  }
  char *base = static_cast<char *>(workspace);
  p.o_part = reinterpret_cast<float *>(base + l.o_part);
  p.lse_part = reinterpret_cast<float *>(base + l.lse_part);
  e = pad::launch_shared(p, (int)D, fp8, stream);
  return e == cudaSuccess ? PAD_OK : pad::host_cuda_fail(e, "shared-prefix decode launch");
}
