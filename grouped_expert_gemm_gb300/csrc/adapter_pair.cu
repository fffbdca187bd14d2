#include "adapter_project.cuh"

namespace moe {
namespace adapter {

moe_status project_pair(const ProjectArgs& a, const Operands& o, bool kmaj, cudaStream_t s) {
  return kmaj ? launch_project_as<256, 1, 2, true>(a, o, s) : launch_project_as<256, 1, 2, false>(a, o, s);
}

}  // namespace adapter
}  // namespace moe
