#include "adapter_project.cuh"

namespace moe {
namespace adapter {

moe_status project_pair(const ProjectArgs& a, const Operands& o, bool kmaj, cudaStream_t s) {
  moe_status st = MOE_ERR_CUDA;
  if (kmaj) launch_project_as<256, 1, 2, true>(a, o, s, st);
  else launch_project_as<256, 1, 2, false>(a, o, s, st);
  return st;
}

}  // namespace adapter
}  // namespace moe
