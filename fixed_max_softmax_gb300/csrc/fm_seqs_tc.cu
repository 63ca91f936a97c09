// fm_seqs_tc.cu -- the tensor-core attention kernels of fm_seqs_tc.cuh for causal, windowed and full
// masks, and how their work is cut (trees of drafted tokens: fm_seqs_tree_tc.cu).
#include "fm_seqs_tc.cuh"

namespace fm {

// The tensor-core kernel takes 16-bit types whose rows a tensor map describes, and pages that
// divide its key tiles or are made of them.
bool seqs_tc_supported(const SeqsArgs &a) {
  if (a.q.dtype == FM_F32) return false;
  if (a.k.S < 1 || a.k.B < 1) return false;
  const int64_t ps = a.k.S;
  if (a.paged && !(ps == 8 || ps == 16 || ps == 32 || ps == 64 || ps % 128 == 0)) return false;
  return rows_aligned(a.q, 2, 16) && rows_aligned(a.k, 2, 16) && rows_aligned(a.v, 2, 16) &&
         rows_aligned(a.o, a.o.dtype == FM_F32 ? 4 : 2, 16);
}

SeqsGeom seqs_geom_tc(int64_t T, int64_t n, int group, bool tree) {
  SeqsGeom g;
  g.group = group;
  g.tq = 2 * (128 / group);
  g.bk = 128;
  g.slot_rows = (int)(g.tq < T ? g.tq : T) * group;
  g.ctas = current_device_sm_count();
  g.n_slots = 8 * g.ctas;
  g.min_tiles = 4;
  // few queries a request: a tile of rows holds all of most requests' queries of a key head.  Even runs
  // against the list: decode batch of 64 149 and 158 us, 4 requests of 131k 149 and 171, a step of 120
  // decoding requests and 3 chunks 203 and 208; 24 packed prompts of up to 4,096 751 and 674.
  // The rule knows the arrays, not the lengths in them, which are on the device: the decode batch in
  // buffers of 2,048 rows takes the list (146 -> 155 us), a prompt of 6,000 among 255 idle rows even runs
  // (325 -> 351).
  // Trees have tens of tokens over long contexts, where the list's three launches and uneven pieces cost more:
  // one tree of 64 over 8k 35 and 39, 4 of 64 over 65k (8 heads to one) 177 and 219, one of 1,024 over 30k 372 and
  // 444, 3 chunks of 500 beside a tree 85 and 90 (3,100 rows a request); chunks of 2,000 beside a tree 103 and 94
  // (7,600), of 4,000 112 and 106 (8,000).
  g.stream = T * group <= (tree ? 4096 : 128) * n ? 1 : 0;
  return g;
}

cudaError_t seqs_tc_prepare() { return prepare_tc<false>(); }
cudaError_t launch_seqs_tc(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  return launch_tc<false>(a, g, s, st);
}

}  // namespace fm
