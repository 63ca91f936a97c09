// fm_seqs_simt.cu -- the CUDA-core attention kernels of fm_seqs_simt.cuh for causal, windowed and full
// masks, and how their work is cut (trees of drafted tokens: fm_seqs_tree_simt.cu).
#include "fm_seqs_simt.cuh"

namespace fm {

SeqsGeom seqs_geom_simt(int64_t T, int group, int rows) {
  SeqsGeom g;
  g.group = group;
  g.tq = rows / group;
  g.bk = kK;
  g.slot_rows = (int)(g.tq < T ? g.tq : T) * group;
  g.ctas = 2 * current_device_sm_count();
  g.n_slots = 4 * g.ctas;
  g.min_tiles = rows < kR ? 4 : 1;  // of few rows: a step of every warp
  g.stream = 0;
  return g;
}

cudaError_t seqs_simt_prepare() { return prepare_simt<false>(); }
cudaError_t launch_seqs_simt(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  return launch_simt<false>(a, g, s, st);
}

}  // namespace fm
