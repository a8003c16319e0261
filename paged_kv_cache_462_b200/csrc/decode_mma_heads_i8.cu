// Instantiations of the warp-MMA decode kernels for KvI8 caches whose producer resolves every KV
// head of a unit for itself (selected blocks, block scales).
#include "decode_mma_dispatch.cuh"

namespace pkv {

int decode_mma_heads_dispatch_i8(int D, int BS, int G, int HG, const MmaOp& op)
{
    return mma_by_d<KvI8, false, true>(D, BS, G, HG, op);
}

}  // namespace pkv
