// paged_fp4_tc_d64.cu — the head_dim-64 instantiation of paged_fp4_tc.cuh (a
// translation unit of its own, so that the head sizes compile in parallel).
#include "paged_fp4_tc.cuh"

namespace gb300 {

sdpa_status_t launch_paged_fp4_tc_d64(paged::Args a, int dtype, const LaunchEnv& env) {
  return paged::launch_fp4_tc<64>(a, dtype, env);
}

}  // namespace gb300
