// attend_tree.cu -- attention of a tree of drafted tokens over the cache.
#include "attend_set.cuh"

namespace up {

size_t attend_tree_workspace(int64_t T, int num_seqs, int Hq, int Hk, int d) {
    return layout_of(T, num_seqs, Hq, Hk, d).total + (size_t)T * kTreeWords * sizeof(uint32_t);
}

cudaError_t launch_attend_tree(const AttendArgs &a, int num_sms, cudaStream_t st) {
    return launch_set<kTree>(a, num_sms, st);
}

}  // namespace up
