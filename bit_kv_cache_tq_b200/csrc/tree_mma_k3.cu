// Tree attention on the tensor cores: keys of 3 bits (8: int8).

#include "tree_mma_impl.cuh"

namespace tq {
namespace tree {

cudaError_t launch_mma_k3(int vb, const Args& a, int blocks, cudaStream_t s) {
    switch (vb) {
        case 2: return mma::launch_typed<3, 2>(a, blocks, s);
        case 3: return mma::launch_typed<3, 3>(a, blocks, s);
        case 4: return mma::launch_typed<3, 4>(a, blocks, s);
        default: return mma::launch_typed<3, 8>(a, blocks, s);
    }
}

}  // namespace tree
}  // namespace tq
