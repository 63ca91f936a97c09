// fm_seqs_tree_tc.cu -- the tensor-core attention kernels of fm_seqs_tc.cuh for trees of drafted tokens.
#include "fm_seqs_tc.cuh"

namespace fm {

cudaError_t seqs_tree_tc_prepare() { return prepare_tc<true>(); }
cudaError_t launch_seqs_tree_tc(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  return launch_tc<true>(a, g, s, st);
}

}  // namespace fm
