// fm_tree.cu -- trees of drafted tokens: what each node sees.
//
// fm_tree_mask: of a request whose new tokens are the nodes of a tree (parent[t] < t, -1: a root),
//   bit j of row t  <=>  j = t, or j is an ancestor of t;   positions[t] = base + (number of ancestors)
// A CTA a request stages the parents in shared memory; a thread walks up from its node.  Ancestors come
// in descending order, so a row's words are finished one after another from its last: a node of depth d
// in a mask of W words takes d + W steps, and nothing waits for another node.  Bound by latency: the
// parents' load, then the walk.
#include "fm_tree.cuh"

namespace fm {
namespace {

constexpr int kMaskThreads = 128;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const TreeMaskArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int par[FM_MAX_NODES];
  const int b = blockIdx.x, words = (int)a.words;
  const Rows r = rows_of(a.cu_q, b, a.T, threadIdx.x == 0 ? a.err : nullptr);
  const int base = a.kv_len[b] - r.count;
  if (r.count > 32 * words) {  // causal: more tokens than a row has bits
    for (int64_t i = threadIdx.x; i < (int64_t)r.count * words; i += kMaskThreads)
      a.mask[(r.first + i / words) * a.stride + i % words] = 0u;
    if (a.positions)
      for (int t = threadIdx.x; t < r.count; t += kMaskThreads) a.positions[r.first + t] = base + t;
    return;
  }
  for (int t = threadIdx.x; t < r.count; t += kMaskThreads) {
    int p = a.parent[r.first + t];
    if (p >= t || p < -1) {  // no tree: the node is taken for a root
      report(a.err, kDevErrParent, (unsigned)b, (unsigned)t, (unsigned)p, 0u);
      p = -1;
    }
    par[t] = p;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < r.count; t += kMaskThreads) {
    uint32_t *row = a.mask + (int64_t)(r.first + t) * a.stride;
    int at = t, depth = -1;
    for (int w = words - 1; w >= 0; --w) {
      uint32_t bits = 0u;
      for (; at >= 32 * w; at = par[at]) {  // (at = -1 ends it: above the root)
        bits |= 1u << (at & 31);
        ++depth;
      }
      row[w] = bits;
    }
    if (a.positions) a.positions[r.first + t] = base + depth;
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs &a, cudaStream_t st) {
  return launch_pdl(tree_mask_kernel, dim3((unsigned)a.n), dim3(kMaskThreads), 0, st, a);
}

}  // namespace fm
