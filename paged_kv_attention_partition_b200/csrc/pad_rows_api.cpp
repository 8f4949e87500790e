// Host side of pad_qk_norm_rope and pad_append_kv: argument validation and the
// launch.  Declared in include/pad.h.
#include <cuda_runtime.h>
#include <math.h>

#include "pad.h"
#include "pad_host.h"
#include "pad_internal.h"
#include "pad_rows.h"

namespace {

using pad::host_fail;

// Whether rows of D elements at these (size, stride) dims are apart: taken by
// ascending stride, each dim steps over everything below it.  (Rows that
// overlap would be written by two lanes at once.)
bool rows_apart(const pad_tensor *t) {
  int64_t span = t->shape[t->ndim - 1];
  bool used[3] = {};
  for (int round = 0; round < t->ndim - 1; ++round) {
    int best = -1;
    for (int i = 0; i < t->ndim - 1; ++i)
      if (!used[i] && (best < 0 || t->stride[i] < t->stride[best])) best = i;
    used[best] = true;
    if (t->shape[best] <= 1) continue;
    if (t->stride[best] < span) return false;
    span += t->stride[best] * (t->shape[best] - 1);
  }
  return true;
}

// rows [T, H, D] of one token range; *D is taken from the first one seen
pad_status check_rows(const pad_tensor *t, const char *name, int64_t *T, int64_t *D) {
  pad_status st;
  if ((st = pad::host_check_tensor(t, name, PAD_BF16, 3)) != PAD_OK) return st;
  if ((st = pad::host_check_rows16(t, name, 2)) != PAD_OK) return st;
  if (*T < 0) *T = t->shape[0];
  if (*D < 0) *D = t->shape[2];
  if (t->shape[0] != *T || t->shape[2] != *D)
    return host_fail(PAD_ERR_INVALID_ARG, "%s is [%lld, %lld, %lld], expected [%lld, heads, %lld]", name,
                     (long long)t->shape[0], (long long)t->shape[1], (long long)t->shape[2], (long long)*T, (long long)*D);
  if (t->shape[1] <= 0 || t->shape[1] > 65536)
    return host_fail(PAD_ERR_UNSUPPORTED, "%s has %lld heads (1 to 65536)", name, (long long)t->shape[1]);
  return PAD_OK;
}

pad_status check_like(const pad_tensor *t, const pad_tensor *like, const char *name) {
  int64_t T = like->shape[0], D = like->shape[2];
  pad_status st = check_rows(t, name, &T, &D);
  if (st != PAD_OK) return st;
  if (t->shape[1] != like->shape[1])
    return host_fail(PAD_ERR_INVALID_ARG, "%s has %lld heads, expected %lld", name, (long long)t->shape[1],
                     (long long)like->shape[1]);
  if (!rows_apart(t)) return host_fail(PAD_ERR_INVALID_ARG, "%s: its rows overlap", name);
  return PAD_OK;
}

pad_status check_vector(const pad_tensor *t, const char *name, pad_dtype dt, int64_t n) {
  pad_status st = pad::host_check_tensor(t, name, dt, 1);
  if (st != PAD_OK) return st;
  if (t->shape[0] != n || (t->stride[0] != 1 && n > 1))
    return host_fail(PAD_ERR_INVALID_ARG, "%s must be contiguous [%lld]", name, (long long)n);
  if (reinterpret_cast<uintptr_t>(t->data) % (dt == PAD_BF16 ? 2 : 4))
    return host_fail(PAD_ERR_INVALID_ARG, "%s is misaligned", name);
  return PAD_OK;
}

pad_status check_weight(const pad_tensor *t, const char *name, int64_t D) {
  if (t == nullptr) return PAD_OK;
  pad_status st = check_vector(t, name, t->dtype == PAD_F32 ? PAD_F32 : PAD_BF16, D);
  if (st != PAD_OK) return st;
  if (reinterpret_cast<uintptr_t>(t->data) % 16)
    return host_fail(PAD_ERR_INVALID_ARG, "%s: data must be 16-byte aligned", name);
  return PAD_OK;
}

pad_status check_rotation(const pad_tensor *inv_freq, int64_t D) {
  if (inv_freq == nullptr) return PAD_OK;
  const int64_t half = inv_freq->ndim == 1 ? inv_freq->shape[0] : -1;
  pad_status st = check_vector(inv_freq, "inv_freq", PAD_F32, half);
  if (st != PAD_OK) return st;
  if (half <= 0 || 2 * half > D)
    return host_fail(PAD_ERR_INVALID_ARG, "inv_freq has %lld entries: 1 to head_dim / 2 = %lld", (long long)half,
                     (long long)(D / 2));
  if (half % 8 != 0)
    return host_fail(PAD_ERR_UNSUPPORTED, "inv_freq has %lld entries: a multiple of 8 is supported", (long long)half);
  return PAD_OK;
}

pad_status check_dim(int64_t D) {
  return D == 64 || D == 128 || D == 256
             ? PAD_OK
             : host_fail(PAD_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)D);
}

pad_status check_eps(float eps) {
  return isfinite(eps) && eps >= 0.f ? PAD_OK : host_fail(PAD_ERR_INVALID_ARG, "eps must be finite and >= 0");
}

pad_status on_device(const pad_tensor *t, int device, const char *name) {
  return t == nullptr ? PAD_OK : pad::host_check_device_ptr(t->data, device, name);
}

void set_weights(pad::RowsParams *p, const pad_tensor *qw, const pad_tensor *kw, float eps) {
  p->qw = qw != nullptr ? qw->data : nullptr;
  p->qw_f32 = qw != nullptr && qw->dtype == PAD_F32;
  p->kw = kw != nullptr ? kw->data : nullptr;
  p->kw_f32 = kw != nullptr && kw->dtype == PAD_F32;
  p->eps = eps;
}

void set_rotation(pad::RowsParams *p, const pad_tensor *positions, const pad_tensor *inv_freq, int32_t interleaved) {
  p->positions = static_cast<const int32_t *>(positions->data);
  p->inv_freq = inv_freq != nullptr ? static_cast<const float *>(inv_freq->data) : nullptr;
  p->rot = inv_freq != nullptr ? (int32_t)(2 * inv_freq->shape[0]) : 0;
  p->interleaved = interleaved != 0;
}

void set_query(pad::RowsParams *p, const pad_tensor *q, const pad_tensor *q_out) {
  p->Hq = (int32_t)q->shape[1];
  p->q = static_cast<const uint16_t *>(q->data);
  p->q_st = q->stride[0];
  p->q_sh = q->stride[1];
  p->q_out = static_cast<uint16_t *>(q_out->data);
  p->qo_st = q_out->stride[0];
  p->qo_sh = q_out->stride[1];
}

pad_status launch(const pad::RowsParams &p, int64_t D, int mode, int device, void *stream) {
  const cudaError_t e =
      pad::launch_rows(p, (int)D, mode, pad::host_sm_count(device), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAD_OK : pad::host_cuda_fail(e, "row kernel launch");
}

}  // namespace

extern "C" pad_status pad_qk_norm_rope(const pad_tensor *q, const pad_tensor *k, const pad_tensor *q_weight,
                                       const pad_tensor *k_weight, float eps, const pad_tensor *positions,
                                       const pad_tensor *inv_freq, int32_t interleaved, pad_tensor *q_out,
                                       pad_tensor *k_out, void *stream) {
  pad_status st;
  int64_t T = -1, D = -1;
  if ((st = check_rows(q, "q", &T, &D)) != PAD_OK) return st;
  if ((st = check_like(q_out, q, "q_out")) != PAD_OK) return st;
  if ((k == nullptr) != (k_out == nullptr))
    return host_fail(PAD_ERR_INVALID_ARG, "k and k_out go together: both or neither");
  if (k != nullptr && (st = check_rows(k, "k", &T, &D)) != PAD_OK) return st;
  if (k != nullptr && (st = check_like(k_out, k, "k_out")) != PAD_OK) return st;
  if ((st = check_dim(D)) != PAD_OK) return st;
  if ((st = check_weight(q_weight, "q_weight", D)) != PAD_OK) return st;
  if ((st = check_weight(k_weight, "k_weight", D)) != PAD_OK) return st;
  if (k == nullptr && k_weight != nullptr) return host_fail(PAD_ERR_INVALID_ARG, "k_weight without k");
  if ((st = check_eps(eps)) != PAD_OK) return st;
  if ((st = check_rotation(inv_freq, D)) != PAD_OK) return st;
  if ((positions == nullptr) != (inv_freq == nullptr))
    return host_fail(PAD_ERR_INVALID_ARG, "positions and inv_freq go together: both or neither");
  if (positions != nullptr && (st = check_vector(positions, "positions", PAD_I32, T)) != PAD_OK) return st;
  if (T == 0) return PAD_OK;

  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return pad::host_cuda_fail(e, "cudaGetDevice");
  const struct { const pad_tensor *t; const char *name; } all[] = {
      {q, "q"}, {k, "k"}, {q_weight, "q_weight"}, {k_weight, "k_weight"}, {positions, "positions"},
      {inv_freq, "inv_freq"}, {q_out, "q_out"}, {k_out, "k_out"}};
  for (const auto &x : all)
    if ((st = on_device(x.t, device, x.name)) != PAD_OK) return st;

  pad::RowsParams p{};
  p.T = T;
  set_query(&p, q, q_out);
  if (k != nullptr) {
    p.Hkv = (int32_t)k->shape[1];
    p.k = static_cast<const uint16_t *>(k->data);
    p.k_st = k->stride[0];
    p.k_sh = k->stride[1];
    p.k_out = static_cast<uint16_t *>(k_out->data);
    p.ko_st = k_out->stride[0];
    p.ko_sh = k_out->stride[1];
  }
  set_weights(&p, q_weight, k_weight, eps);
  if (positions != nullptr) set_rotation(&p, positions, inv_freq, interleaved);
  return launch(p, D, pad::kRowsOut, device, stream);
}

extern "C" pad_status pad_append_kv(const pad_tensor *k, const pad_tensor *v, const pad_tensor *positions,
                                    const pad_tensor *seq_ids, const pad_tensor *block_tables,
                                    const pad_append_options *options, pad_tensor *k_cache, pad_tensor *v_cache,
                                    void *stream) {
  static const pad_append_options none{};
  const pad_append_options &o = options != nullptr ? *options : none;
  pad_status st;
  int64_t T = -1, D = -1;
  if ((st = check_rows(k, "k", &T, &D)) != PAD_OK) return st;
  if ((st = check_rows(v, "v", &T, &D)) != PAD_OK) return st;
  const int64_t Hkv = k->shape[1];
  if (v->shape[1] != Hkv)
    return host_fail(PAD_ERR_INVALID_ARG, "v has %lld heads, k %lld", (long long)v->shape[1], (long long)Hkv);
  if ((st = check_vector(positions, "positions", PAD_I32, T)) != PAD_OK) return st;
  if ((st = pad::host_check_tensor(block_tables, "block_tables", PAD_I32, 2)) != PAD_OK) return st;
  const int64_t B = block_tables->shape[0], W = block_tables->shape[1];
  if (block_tables->stride[1] != 1 && W > 1)
    return host_fail(PAD_ERR_INVALID_ARG, "block_tables rows must be contiguous");
  if (reinterpret_cast<uintptr_t>(block_tables->data) % 4)
    return host_fail(PAD_ERR_INVALID_ARG, "int32 tensors must be 4-byte aligned");
  if (seq_ids != nullptr && (st = check_vector(seq_ids, "seq_ids", PAD_I32, T)) != PAD_OK) return st;
  if (seq_ids == nullptr && T != B)
    return host_fail(PAD_ERR_INVALID_ARG, "without seq_ids token t is sequence t's: %lld tokens, %lld table rows",
                     (long long)T, (long long)B);
  const bool fp8 = k_cache != nullptr && k_cache->dtype == PAD_FP8_E4M3;
  const pad_dtype kv = fp8 ? PAD_FP8_E4M3 : PAD_BF16;
  const struct { const pad_tensor *t; const char *name; } caches[] = {{k_cache, "k_cache"}, {v_cache, "v_cache"}};
  for (const auto &x : caches) {
    if ((st = pad::host_check_tensor(x.t, x.name, kv, 4)) != PAD_OK) return st;
    if ((st = pad::host_check_rows16(x.t, x.name, fp8 ? 1 : 2)) != PAD_OK) return st;
    if (x.t->shape[1] != Hkv || x.t->shape[3] != D)
      return host_fail(PAD_ERR_INVALID_ARG, "%s is [blocks, %lld, block_size, %lld], k has %lld heads of %lld", x.name,
                       (long long)x.t->shape[1], (long long)x.t->shape[3], (long long)Hkv, (long long)D);
    if (!rows_apart(x.t)) return host_fail(PAD_ERR_INVALID_ARG, "%s: its slots overlap", x.name);
  }
  for (int i = 0; i < 4; ++i)
    if (v_cache->shape[i] != k_cache->shape[i])
      return host_fail(PAD_ERR_INVALID_ARG, "v_cache.shape[%d]=%lld differs from k_cache", i,
                       (long long)v_cache->shape[i]);
  const int64_t NB = k_cache->shape[0], bs = k_cache->shape[2];
  if (NB <= 0 || NB > 0x7fffffffll) return host_fail(PAD_ERR_INVALID_ARG, "num_blocks %lld out of range", (long long)NB);
  if ((st = check_dim(D)) != PAD_OK) return st;
  if (W <= 0 || bs <= 0) return host_fail(PAD_ERR_INVALID_ARG, "sizes must be positive: bs=%lld W=%lld", (long long)bs, (long long)W);
  if ((bs & (bs - 1)) != 0 || bs > 256)
    return host_fail(PAD_ERR_UNSUPPORTED, "block_size %lld must be a power of two in [1, 256]", (long long)bs);
  if (W > ((int64_t)1 << 30) || W * bs > ((int64_t)1 << 30) || B > 0x7fffffffll)
    return host_fail(PAD_ERR_UNSUPPORTED, "table of %lld rows x %lld blocks x %lld tokens too large", (long long)B,
                     (long long)W, (long long)bs);
  if ((o.q == nullptr) != (o.q_out == nullptr))
    return host_fail(PAD_ERR_INVALID_ARG, "q and q_out go together: both or neither");
  if (o.q != nullptr && (st = check_rows(o.q, "q", &T, &D)) != PAD_OK) return st;
  if (o.q != nullptr && (st = check_like(o.q_out, o.q, "q_out")) != PAD_OK) return st;
  if (o.q == nullptr && o.q_weight != nullptr) return host_fail(PAD_ERR_INVALID_ARG, "q_weight without q");
  if ((st = check_weight(o.q_weight, "q_weight", D)) != PAD_OK) return st;
  if ((st = check_weight(o.k_weight, "k_weight", D)) != PAD_OK) return st;
  if ((st = check_eps(o.eps)) != PAD_OK) return st;
  if ((st = check_rotation(o.inv_freq, D)) != PAD_OK) return st;
  const float k_scale = o.k_scale == 0.f ? 1.f : o.k_scale, v_scale = o.v_scale == 0.f ? 1.f : o.v_scale;
  if (!(isfinite(k_scale) && k_scale > 0.f) || !(isfinite(v_scale) && v_scale > 0.f))
    return host_fail(PAD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive (or 0 for 1)");
  if (!fp8 && (k_scale != 1.f || v_scale != 1.f))
    return host_fail(PAD_ERR_INVALID_ARG, "k_scale / v_scale apply to an E4M3 cache only (bf16 cache: 0 or 1)");
  for (float s : {k_scale, v_scale})
    if (s < 0x1p-100f || s > 0x1p100f)
      return host_fail(PAD_ERR_UNSUPPORTED, "scale %g outside [2^-100, 2^100]", (double)s);
  if (T == 0) return PAD_OK;

  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return pad::host_cuda_fail(e, "cudaGetDevice");
  const struct { const pad_tensor *t; const char *name; } all[] = {
      {k, "k"}, {v, "v"}, {positions, "positions"}, {seq_ids, "seq_ids"}, {block_tables, "block_tables"},
      {k_cache, "k_cache"}, {v_cache, "v_cache"}, {o.q, "q"}, {o.q_out, "q_out"}, {o.q_weight, "q_weight"},
      {o.k_weight, "k_weight"}, {o.inv_freq, "inv_freq"}};
  for (const auto &x : all)
    if ((st = on_device(x.t, device, x.name)) != PAD_OK) return st;

  pad::RowsParams p{};
  p.T = T;
  p.Hkv = (int32_t)Hkv;
  p.k = static_cast<const uint16_t *>(k->data);
  p.k_st = k->stride[0];
  p.k_sh = k->stride[1];
  p.v = static_cast<const uint16_t *>(v->data);
  p.v_st = v->stride[0];
  p.v_sh = v->stride[1];
  if (o.q != nullptr) set_query(&p, o.q, o.q_out);
  set_weights(&p, o.q_weight, o.k_weight, o.eps);
  set_rotation(&p, positions, o.inv_freq, o.interleaved);
  p.kc = k_cache->data;
  p.vc = v_cache->data;
  p.kc_sb = k_cache->stride[0];
  p.kc_sh = k_cache->stride[1];
  p.kc_ss = k_cache->stride[2];
  p.vc_sb = v_cache->stride[0];
  p.vc_sh = v_cache->stride[1];
  p.vc_ss = v_cache->stride[2];
  p.tables = static_cast<const int32_t *>(block_tables->data);
  p.table_stride = block_tables->stride[0];
  p.seq_ids = seq_ids != nullptr ? static_cast<const int32_t *>(seq_ids->data) : nullptr;
  p.B = (int32_t)B;
  p.max_blocks = (int32_t)W;
  p.num_blocks = (int32_t)NB;
  while ((1ll << p.bs_log2) < bs) ++p.bs_log2;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const cudaError_t ee = pad::device_error_word(device, &p.err);
  if (ee != cudaSuccess) return pad::host_cuda_fail(ee, "error word");
  return launch(p, D, fp8 ? pad::kRowsCacheE4m3 : pad::kRowsCacheBf16, device, stream);
}
