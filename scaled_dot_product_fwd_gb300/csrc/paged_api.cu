// paged_api.cu — the C entry points over the paged KV cache (include/sdpa.h):
// argument checks, workspace size, kernel choice by type and page size.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "sdpa.h"

namespace gb300 {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
int elem_size(const sdpa_paged_params_t& p) { return p.dtype == SDPA_F32 ? 4 : 2; }

sdpa_status_t check_strides(const int64_t* s, int n, int es) {
  for (int i = 0; i < n; ++i) {
    if (s[i] < 0 || s[i] > (int64_t(1) << 40)) return SDPA_ERR_INVALID_ARGUMENT;
    if ((s[i] * es) % 16 != 0) return SDPA_ERR_MISALIGNED;
  }
  return SDPA_OK;
}

// An output whose rows lie on one another would be written by several CTAs.
bool overlaps(int64_t stride, int64_t count) { return stride == 0 && count > 1; }

enum : unsigned { kUsesQ = 1, kUsesO = 2, kUsesV = 4 };

// Host-only checks of the problem description (no CUDA call).
sdpa_status_t validate(const sdpa_paged_params_t* p, unsigned uses) {
  if (!p) return SDPA_ERR_INVALID_ARGUMENT;
  if (p->num_seqs < 0 || p->num_tokens < 0 || p->num_kv_heads < 1 || p->num_pages < 0 ||
      p->page_size < 1 || p->max_pages < 0 || p->page_table_stride < 0 || p->flags != 0)
    return SDPA_ERR_INVALID_ARGUMENT;
  if (p->dtype != SDPA_F32 && p->dtype != SDPA_F16 && p->dtype != SDPA_BF16)
    return SDPA_ERR_INVALID_ARGUMENT;
  if (uses & kUsesQ) {
    if (p->num_q_heads < 0 || p->num_q_heads % p->num_kv_heads != 0)
      return SDPA_ERR_INVALID_ARGUMENT;
    if (!isfinite(p->scale)) return SDPA_ERR_INVALID_ARGUMENT;
  }
  const int es = elem_size(*p);
  sdpa_status_t st = check_strides(p->k_stride, 3, es);
  if (st == SDPA_OK && (uses & kUsesV)) st = check_strides(p->v_stride, 3, es);
  if (st == SDPA_OK && (uses & kUsesQ)) st = check_strides(p->q_stride, 2, es);
  if (st == SDPA_OK && (uses & kUsesO)) st = check_strides(p->o_stride, 2, es);
  if (st != SDPA_OK) return st;
  if (p->head_dim != 64 && p->head_dim != 128)
    return p->head_dim < 1 ? SDPA_ERR_INVALID_ARGUMENT : SDPA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->max_pages) * p->page_size > (1 << 30) ||
      p->num_tokens > (1 << 30))
    return SDPA_ERR_UNSUPPORTED;
  // (sequence, kv head, slice) counts of the one-dimensional grids
  if (static_cast<int64_t>(p->num_seqs) * p->num_kv_heads > (1 << 24))
    return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

// The device arrays of the description.
sdpa_status_t check_arrays(const sdpa_paged_params_t& p) {
  if (!p.seq_lens_kv || (p.max_pages > 0 && !p.page_table)) return SDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(p.seq_lens_kv, 4) || !aligned(p.page_table, 4) || !aligned(p.cu_seqlens_q, 4) ||
      !aligned(p.sinks, 4))
    return SDPA_ERR_MISALIGNED;
  return SDPA_OK;
}

// A cache that is written to has a place of its own for every row.
bool cache_overlaps(const sdpa_paged_params_t& p) {
  const int64_t n[3] = {p.num_pages, p.num_kv_heads, p.page_size};
  for (int i = 0; i < 3; ++i)
    if (overlaps(p.k_stride[i], n[i]) || overlaps(p.v_stride[i], n[i])) return true;
  return false;
}

// Whether two tensors of one base address are the same one: strides of
// dimensions of one element do not count.
template <int N>
bool same_layout(const int64_t* x, const int64_t* y, const int64_t (&n)[N]) {
  for (int i = 0; i < N; ++i)
    if (n[i] > 1 && x[i] != y[i]) return false;
  return true;
}

int device_sms() {
  int* status = nullptr;
  int sms = 0;
  if (!current_device(&status, &sms)) {
    cudaGetLastError();  // no device: plan for a full GB300
    return 152;
  }
  return sms;
}

paged::Args make_args(const sdpa_paged_params_t& p) {
  using paged::fast_div;
  paged::Args a = {};
  a.B = p.num_seqs;
  a.T = p.num_tokens;
  a.Hq = p.num_q_heads;
  a.Hkv = p.num_kv_heads;
  a.G = p.num_q_heads / p.num_kv_heads;
  a.causal = p.causal ? 1 : 0;
  a.num_pages = p.num_pages;
  a.page_size = p.page_size;
  a.max_pages = p.max_pages;
  a.cap = p.max_pages * p.page_size;
  a.table = p.page_table;
  a.table_stride = p.page_table_stride;
  a.cu = p.cu_seqlens_q;
  a.lens = p.seq_lens_kv;
  a.sinks = p.sinks;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = p.q_stride[i];
    a.os[i] = p.o_stride[i];
  }
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = p.k_stride[i];
    a.vs[i] = p.v_stride[i];
  }
  a.sl2 = p.scale * 1.4426950408889634f;
  a.gu = a.w = a.nsub = 1;
  a.by_page = fast_div(p.page_size);
  a.by_gu = a.by_nsub = a.by_w = fast_div(1);
  return a;
}

// The workspace: descriptors of the CTAs that share a call's work (at most
// kMaxCtas an SM), then two slots of partial results each: one CTA an SM with
// slots of kMaxRows rows, or several with as many rows together.
size_t desc_bytes(int sms) {
  return align256(static_cast<size_t>(paged::kMaxCtas * sms) * paged::kDesc * sizeof(int));
}
size_t workspace(const sdpa_paged_params_t& p, int sms) {
  const size_t slot = static_cast<size_t>(paged::kMaxRows) * (p.head_dim + 2) * sizeof(float);
  return desc_bytes(sms) + 2 * static_cast<size_t>(sms) * slot;
}

bool make_env(LaunchEnv* env, void* stream) {
  env->wait_limit_ns = current_wait_limit_ns();
  env->stream = static_cast<cudaStream_t>(stream);
  return current_device(&env->status, &env->num_sms);
}

// What sdpa_paged_forward and sdpa_paged_scores share before their launch.
sdpa_status_t enter(const sdpa_paged_params_t& p, void* ws, size_t ws_bytes, void* stream,
                    paged::Args* a, LaunchEnv* env) {
  const int sms = device_sms();
  if (!ws || ws_bytes < workspace(p, sms)) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return SDPA_ERR_MISALIGNED;
  if (!make_env(env, stream)) return SDPA_ERR_CUDA;
  *a = make_args(p);
  a->desc = static_cast<int*>(ws);
  a->ws = reinterpret_cast<float*>(static_cast<char*>(ws) + desc_bytes(sms));
  const int forced = debug_option(SDPA_DEBUG_PAGED_CTAS);  // test hook
  a->max_ctas = forced > 0 ? forced : paged::kMaxCtas * sms;
  a->nctas = std::min(a->max_ctas, sms);
  a->status = env->status;
  a->wait_ns = env->wait_limit_ns;
  return SDPA_OK;
}

// Whether a problem runs on the tensor cores: a 16-bit type, pages of whole
// groups of 8 rows (the 128-byte-swizzled tiles' unit), strides that a tensor
// map takes, and a positive scale (the softmax takes its maximum over the raw
// scores).
bool tc_fits(const sdpa_paged_params_t& p, bool values) {
  if (p.dtype == SDPA_F32 || p.page_size % 8 != 0 || p.num_pages < 1 || !(p.scale > 0.f))
    return false;
  if (debug_option(SDPA_DEBUG_PAGED_SIMT) == 1) return false;  // test hook
  const int64_t kv[3] = {p.num_pages, p.num_kv_heads, p.page_size};
  const int64_t qn[2] = {p.num_tokens, p.num_q_heads};
  for (int i = 0; i < 3; ++i)
    for (const int64_t* s : {p.k_stride, p.v_stride})
      if ((s == p.k_stride || values) && kv[i] > 1 && (s[i] <= 0 || s[i] >= (int64_t(1) << 35)))
        return false;
  // the (page, head) blocks are numbered in 31 bits
  paged::CacheBlocks c;
  long long unit;
  const long long ks[3] = {p.k_stride[0], p.k_stride[1], p.k_stride[2]};
  const long long vs[3] = {p.v_stride[0], p.v_stride[1], p.v_stride[2]};
  if (!paged::cache_blocks(ks, p.num_pages, p.num_kv_heads, &c, &unit) ||
      (values && !paged::cache_blocks(vs, p.num_pages, p.num_kv_heads, &c, &unit)))
    return false;
  for (int i = 0; i < 2; ++i)
    if (qn[i] > 1 && (p.q_stride[i] <= 0 || p.q_stride[i] >= (int64_t(1) << 35))) return false;
  return true;
}

bool no_rows(const sdpa_paged_params_t& p) {
  return p.num_seqs == 0 || p.num_tokens == 0 || p.num_q_heads == 0;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

size_t sdpa_paged_workspace_size(const sdpa_paged_params_t* p) {
  if (validate(p, kUsesQ) != SDPA_OK || no_rows(*p)) return 0;
  return workspace(*p, device_sms());
}

sdpa_status_t sdpa_paged_write(const sdpa_paged_params_t* p, const void* k, const void* v,
                               const int64_t* k_new_stride, const int64_t* v_new_stride,
                               void* k_pages, void* v_pages, void* stream) {
  set_last_launches(0);
  sdpa_status_t st = validate(p, kUsesV);
  if (st != SDPA_OK) return st;
  if (p->num_seqs == 0 || p->num_tokens == 0) return SDPA_OK;
  if (!k || !v || !k_new_stride || !v_new_stride || (p->num_pages > 0 && (!k_pages || !v_pages)) ||
      cache_overlaps(*p))
    return SDPA_ERR_INVALID_ARGUMENT;
  const int es = elem_size(*p);
  if ((st = check_strides(k_new_stride, 2, es)) != SDPA_OK) return st;
  if ((st = check_strides(v_new_stride, 2, es)) != SDPA_OK) return st;
  if ((st = check_arrays(*p)) != SDPA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return SDPA_ERR_MISALIGNED;
  // One cache for both: every row is written twice, with the same values only
  // where both come from the same place and go to the same one.
  const int64_t rows[2] = {p->num_tokens, p->num_kv_heads};
  const int64_t places[3] = {p->num_pages, p->num_kv_heads, p->page_size};
  if (p->num_pages > 0 && k_pages == v_pages &&
      (k != v || !same_layout(k_new_stride, v_new_stride, rows) ||
       !same_layout(p->k_stride, p->v_stride, places)))
    return SDPA_ERR_INVALID_ARGUMENT;
  LaunchEnv env;
  if (!make_env(&env, stream)) return SDPA_ERR_CUDA;
  paged::Args a = make_args(*p);
  a.status = env.status;
  st = launch_paged_write(a, p->head_dim * es, k, v, k_new_stride, v_new_stride, k_pages,
                          v_pages, es, env.stream);
  if (st == SDPA_OK) set_last_launches(1);
  return st;
}

sdpa_status_t sdpa_paged_forward(const sdpa_paged_params_t* p, const void* q,
                                 const void* k_pages, const void* v_pages, void* o, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  set_last_launches(0);
  sdpa_status_t st = validate(p, kUsesQ | kUsesO | kUsesV);
  if (st != SDPA_OK) return st;
  if (no_rows(*p)) return SDPA_OK;
  if (overlaps(p->o_stride[0], p->num_tokens) || overlaps(p->o_stride[1], p->num_q_heads))
    return SDPA_ERR_INVALID_ARGUMENT;
  if (!q || !o || (p->num_pages > 0 && (!k_pages || !v_pages)))
    return SDPA_ERR_INVALID_ARGUMENT;
  if ((st = check_arrays(*p)) != SDPA_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(lse, 4))
    return SDPA_ERR_MISALIGNED;
  paged::Args a;
  LaunchEnv env;
  if ((st = enter(*p, ws, ws_bytes, stream, &a, &env)) != SDPA_OK) return st;
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.o = o;
  a.lse = lse;
  if (!tc_fits(*p, true)) {
    const int rows = p->dtype == SDPA_F32 ? paged_vector_rows(a) : 0;
    st = rows ? launch_paged_vector_f32(a, p->head_dim, rows, env)
              : launch_paged_simt(a, p->head_dim, p->dtype, env);
  }
  else if (const int rows = paged_decode_rows(a))
    st = launch_paged_decode_tc(a, p->head_dim, p->dtype, rows, env);
  else
    st = p->head_dim == 64 ? launch_paged_tc_d64(a, p->dtype, env)
                           : launch_paged_tc_d128(a, p->dtype, env);
  if (st == SDPA_OK) set_last_launches(2);
  return st;
}

sdpa_status_t sdpa_paged_scores(const sdpa_paged_params_t* p, const void* q,
                                const void* k_pages, const float* lse, float* scores,
                                const int64_t* score_stride, int32_t score_len, void* ws,
                                size_t ws_bytes, void* stream) {
  set_last_launches(0);
  sdpa_status_t st = validate(p, kUsesQ);
  if (st != SDPA_OK) return st;
  if (score_len < 0) return SDPA_ERR_INVALID_ARGUMENT;
  if (no_rows(*p) || score_len == 0) return SDPA_OK;
  if (!q || !lse || !scores || !score_stride || score_stride[0] < 0 || score_stride[1] < 0 ||
      (p->num_pages > 0 && !k_pages) || overlaps(score_stride[0], p->num_seqs) ||
      overlaps(score_stride[1], p->num_kv_heads))
    return SDPA_ERR_INVALID_ARGUMENT;
  if ((st = check_arrays(*p)) != SDPA_OK) return st;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(lse, 4) || !aligned(scores, 4))
    return SDPA_ERR_MISALIGNED;
  paged::Args a;
  LaunchEnv env;
  if ((st = enter(*p, ws, ws_bytes, stream, &a, &env)) != SDPA_OK) return st;
  a.q = q;
  a.k = k_pages;
  a.lse = const_cast<float*>(lse);
  a.scores = scores;
  a.ss[0] = score_stride[0];
  a.ss[1] = score_stride[1];
  a.score_len = score_len;
  int launches = 2;
  // (the few-row kernel counts a sequence's steps, key tiles times blocks of
  // rows, in 32 bits)
  const int rows = p->dtype == SDPA_F32 && (a.cap / 64 + 1LL) * a.T <= INT32_MAX
                       ? paged_vector_rows(a) : 0;
  if (tc_fits(*p, false)) {
    st = launch_paged_scores_tc(a, p->head_dim, p->dtype, env);
  } else if (rows) {
    launches = 1;
    st = launch_paged_scores_vector_f32(a, p->head_dim, rows, env);
  } else {
    st = launch_paged_scores_simt(a, p->head_dim, p->dtype, env);
  }
  if (st == SDPA_OK) set_last_launches(launches);
  return st;
}

sdpa_status_t sdpa_paged_evict(const sdpa_paged_params_t* p, int32_t keep, int32_t recent,
                               void* k_pages, void* v_pages, const float* scores,
                               float* scores_out, const int64_t* score_stride,
                               int32_t score_len, int32_t* kept, int32_t* seq_lens_out,
                               void* stream) {
  set_last_launches(0);
  sdpa_status_t st = validate(p, kUsesV);
  if (st != SDPA_OK) return st;
  if (keep < 1 || recent < 0 || score_len < 0) return SDPA_ERR_INVALID_ARGUMENT;
  // (as for the positions: loops over either step past them in 32 bits)
  if (keep > (1 << 30) || score_len > (1 << 30)) return SDPA_ERR_UNSUPPORTED;
  if (p->num_seqs == 0) return SDPA_OK;
  if (!scores || !score_stride || score_stride[0] < 0 || score_stride[1] < 0 || !kept ||
      (p->num_pages > 0 && (!k_pages || !v_pages)) || cache_overlaps(*p) ||
      (scores_out && (overlaps(score_stride[0], p->num_seqs) ||
                      overlaps(score_stride[1], p->num_kv_heads))))
    return SDPA_ERR_INVALID_ARGUMENT;
  if ((st = check_arrays(*p)) != SDPA_OK) return st;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(scores, 4) ||
      !aligned(scores_out, 4) || !aligned(kept, 4) || !aligned(seq_lens_out, 4))
    return SDPA_ERR_MISALIGNED;
  // (K and V move side by side: rows of one cache would move twice)
  if (p->num_pages > 0 && k_pages == v_pages) return SDPA_ERR_INVALID_ARGUMENT;
  LaunchEnv env;
  if (!make_env(&env, stream)) return SDPA_ERR_CUDA;
  paged::Args a = make_args(*p);
  a.status = env.status;
  const int es = elem_size(*p);
  int launches = 0;
  st = launch_paged_evict(a, p->head_dim * es, es, keep, recent, k_pages, v_pages, scores,
                          scores_out, score_stride, score_len, kept, seq_lens_out, env.stream,
                          &launches);
  if (st == SDPA_OK) set_last_launches(launches);
  return st;
}

}  // extern "C"
