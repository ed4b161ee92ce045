// paged_append.cuh — host interface of paged_append.cu.
#pragma once

#include "internal.h"
#include "paged.cuh"
#include "sdpa.h"

namespace gb300 {
namespace paged {
// What sdpa_paged_append and sdpa_paged_append_fp4 were given besides the
// problem (fp4 null: a cache of the tensors' type).
struct AppendIo {
  const sdpa_rotation_t* rotation;
  const sdpa_fp4_cache_t* fp4;
  const void* k;
  const void* v;
  void* q_out;
  const int64_t* k_new_stride;
  const int64_t* v_new_stride;
  void* k_pages;
  void* v_pages;
  void* k_out;
  void* v_out;
  const int64_t* out_stride;
};
}  // namespace paged

sdpa_status_t launch_paged_append(const paged::Args& a, int head_dim, int dtype,
                                  const paged::AppendIo& io, const LaunchEnv& env);

}  // namespace gb300
