// paged_tc_d128.cu — the head_dim-128 instantiation of paged_tc.cuh (a
// translation unit of its own, so that the head sizes compile in parallel).
#include "paged_tc.cuh"

namespace gb300 {

sdpa_status_t launch_paged_tc_d128(paged::Args a, int dtype, const LaunchEnv& env) {
  return paged::launch_tc<128>(a, dtype, env);
}

}  // namespace gb300
