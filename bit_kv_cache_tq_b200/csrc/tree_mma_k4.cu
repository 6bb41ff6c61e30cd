// Tree attention on the tensor cores: keys of 4 bits (8: int8).

#include "tree_mma_impl.cuh"

namespace tq {
namespace tree {

cudaError_t launch_mma_k4(int vb, const Args& a, int blocks, cudaStream_t s) {
    switch (vb) {
        case 2: return mma::launch_typed<4, 2>(a, blocks, s);
        case 3: return mma::launch_typed<4, 3>(a, blocks, s);
        case 4: return mma::launch_typed<4, 4>(a, blocks, s);
        default: return mma::launch_typed<4, 8>(a, blocks, s);
    }
}

}  // namespace tree
}  // namespace tq
