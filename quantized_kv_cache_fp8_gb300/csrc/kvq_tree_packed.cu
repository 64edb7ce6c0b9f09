#include "kvq_internal.cuh"
namespace kvq {
bool tree_packed_reads(const kvq_mla_tree_problem&) { return false; }
size_t tree_packed_workspace(const kvq_mla_tree_problem&) { return 0; }
cudaError_t launch_tree_packed(const kvq_mla_tree_problem&, void*, float*, void*, uint32_t*, cudaStream_t) { return cudaErrorNotSupported; }
}
