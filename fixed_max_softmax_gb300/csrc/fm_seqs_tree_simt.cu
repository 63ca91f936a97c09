// fm_seqs_tree_simt.cu -- the CUDA-core attention kernels of fm_seqs_simt.cuh for trees of drafted tokens.
#include "fm_seqs_simt.cuh"

namespace fm {

cudaError_t seqs_tree_simt_prepare() { return prepare_simt<true>(); }
cudaError_t launch_seqs_tree_simt(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  return launch_simt<true>(a, g, s, st);
}

}  // namespace fm
