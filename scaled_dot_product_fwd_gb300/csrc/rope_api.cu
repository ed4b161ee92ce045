// rope_api.cu — the C entry points of the rotary operators (include/sdpa.h):
// argument checks.
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "rotate.cuh"
#include "sdpa.h"

namespace gb300 {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

sdpa_status_t check_strides(const int64_t* s, int es) {
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || s[i] > (int64_t(1) << 40)) return SDPA_ERR_INVALID_ARGUMENT;
    if ((s[i] * es) % 16 != 0) return SDPA_ERR_MISALIGNED;
  }
  return SDPA_OK;
}

// A tensor and its rotated form: strides, alignment, an output with a place for
// every row, and the input's layout where it is the input itself.
sdpa_status_t check_pair(const sdpa_rope_params_t& p, int heads, const void* x, const void* out,
                         const int64_t* xs, const int64_t* os) {
  if (heads == 0) return SDPA_OK;
  const int es = p.dtype == SDPA_F32 ? 4 : 2;
  sdpa_status_t st = check_strides(xs, es);
  if (st == SDPA_OK) st = check_strides(os, es);
  if (st != SDPA_OK) return st;
  if (!x || !out) return SDPA_ERR_INVALID_ARGUMENT;
  const int64_t n[3] = {p.batch, heads, p.seq_len};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (os[i] == 0 || (x == out && xs[i] != os[i]))) return SDPA_ERR_INVALID_ARGUMENT;
  return aligned(x, 16) && aligned(out, 16) ? SDPA_OK : SDPA_ERR_MISALIGNED;
}

}  // namespace

sdpa_status_t check_rotation(const sdpa_rotation_t& r, int head_dim) {
  if (r.rotary_dim < 1 || r.rotary_dim > head_dim || r.table_len < 0 ||
      (r.table_len > 0 && !r.table))
    return SDPA_ERR_INVALID_ARGUMENT;
  if (r.rotary_dim % 16 != 0 || r.table_len > (int64_t(1) << 40)) return SDPA_ERR_UNSUPPORTED;
  if (!aligned(r.table, 16) || !aligned(r.positions, 4)) return SDPA_ERR_MISALIGNED;
  return SDPA_OK;
}

}  // namespace gb300

using namespace gb300;

extern "C" {

sdpa_status_t sdpa_rope_table(float* table, int64_t length, int32_t rotary_dim,
                              const double* inv_freq, double gain, void* stream) {
  set_last_launches(0);
  if (length < 0 || rotary_dim < 1 || !inv_freq || !isfinite(gain))
    return SDPA_ERR_INVALID_ARGUMENT;
  if (rotary_dim % 16 != 0 || rotary_dim > 512 || length > (int64_t(1) << 31))
    return SDPA_ERR_UNSUPPORTED;
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!isfinite(inv_freq[i])) return SDPA_ERR_INVALID_ARGUMENT;
  if (length == 0) return SDPA_OK;
  if (!table) return SDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(table, 16)) return SDPA_ERR_MISALIGNED;
  const sdpa_status_t st = launch_rope_table(table, length, rotary_dim, inv_freq, gain,
                                             static_cast<cudaStream_t>(stream));
  if (st == SDPA_OK) set_last_launches(1);
  return st;
}

sdpa_status_t sdpa_rope(const sdpa_rope_params_t* p, const void* q, const void* k, void* q_out,
                        void* k_out, void* stream) {
  set_last_launches(0);
  if (!p || p->batch < 0 || p->num_q_heads < 0 || p->num_kv_heads < 0 || p->seq_len < 0 ||
      p->flags != 0 || p->position_stride < 0)
    return SDPA_ERR_INVALID_ARGUMENT;
  if (p->dtype != SDPA_F32 && p->dtype != SDPA_F16 && p->dtype != SDPA_BF16)
    return SDPA_ERR_INVALID_ARGUMENT;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 512)
    return p->head_dim < 1 ? SDPA_ERR_INVALID_ARGUMENT : SDPA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->batch) * p->seq_len > (1 << 30) ||
      static_cast<int64_t>(p->num_q_heads) + p->num_kv_heads > (1 << 24))
    return SDPA_ERR_UNSUPPORTED;
  sdpa_status_t st = check_rotation(p->rotation, p->head_dim);
  if (st != SDPA_OK) return st;
  if (p->batch == 0 || p->seq_len == 0 || p->num_q_heads + p->num_kv_heads == 0) return SDPA_OK;
  st = check_pair(*p, p->num_q_heads, q, q_out, p->q_stride, p->q_out_stride);
  if (st == SDPA_OK)
    st = check_pair(*p, p->num_kv_heads, k, k_out, p->k_stride, p->k_out_stride);
  if (st != SDPA_OK) return st;
  if (p->num_q_heads > 0 && p->num_kv_heads > 0 && q_out == k_out)
    return SDPA_ERR_INVALID_ARGUMENT;
  LaunchEnv env;
  env.wait_limit_ns = current_wait_limit_ns();
  env.stream = static_cast<cudaStream_t>(stream);
  if (!current_device(&env.status, &env.num_sms)) return SDPA_ERR_CUDA;
  st = launch_rope(*p, q, k, q_out, k_out, env);
  if (st == SDPA_OK) set_last_launches(1);
  return st;
}

}  // extern "C"
