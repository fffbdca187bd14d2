#include "adapter_project.cuh"

namespace moe {
namespace adapter {

moe_status project_flat128_kmaj(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s) {
  return launch_flat<128, true>(a, o, split, s);
}

}  // namespace adapter
}  // namespace moe
