#include "adapter_project.cuh"

namespace moe {
namespace adapter {

moe_status project_flat64(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s) {
  return launch_flat<64, false>(a, o, split, s);
}

}  // namespace adapter
}  // namespace moe
