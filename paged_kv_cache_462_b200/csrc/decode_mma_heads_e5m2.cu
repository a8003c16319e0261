// Instantiations of the warp-MMA decode kernels for KvE5M2 caches whose producer resolves every KV
// head of a unit for itself (selected blocks, block scales).
#include "decode_mma_dispatch.cuh"

namespace pkv {

int decode_mma_heads_dispatch_e5m2(int D, int BS, int G, int HG, const MmaOp& op)
{
    return mma_by_d<KvE5M2, false, true>(D, BS, G, HG, op);
}

}  // namespace pkv
