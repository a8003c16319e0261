// Shape dispatch of the warp-MMA decode kernels: run-time (head_dim, block size, group, head
// group) -> template instantiation, for one cache type per translation unit (decode_mma_*.cu).
#pragma once

#include "decode_mma.cuh"

namespace pkv {

// PH: the kernels that resolve every KV head for itself, in translation units of their own
// (decode_mma_heads_*.cu)
template <class KV, int D, int BS, int G, int HG, bool PH>
int mma_run(const MmaOp& op)
{
    if constexpr (PH) {
        using L = MmaLauncher<KV, __nv_bfloat16, D, BS, G, HG, false, true>;
        if (op.kind == MmaOp::kLaunchPerHead)
            return L::launch(*op.p, op.nruns, op.stream);
        if (op.kind == MmaOp::kPerHeadOccupancy) {
            *op.occ = L::occupancy(op.p->num_seqs);
            return PKV_OK;
        }
        return PKV_ERR_SHAPE;
    } else {
        using L = MmaLauncher<KV, __nv_bfloat16, D, BS, G, HG>;
        switch (op.kind) {
        case MmaOp::kLaunch:
            return L::launch(*op.p, op.nruns, op.stream);
        case MmaOp::kOccupancy:
            *op.occ = L::occupancy(op.p->num_seqs);
            return PKV_OK;
        case MmaOp::kLaunchSharedPrefix:
            return L::launch_shared_prefix(*op.p, *op.pp, op.nruns, op.runs_p, op.stream);
        case MmaOp::kPrefixOccupancy:
            *op.occ = MmaLauncher<KV, __nv_bfloat16, D, BS, 8, 1, true>::occupancy(op.p->num_seqs);
            return PKV_OK;
        default:
            return PKV_ERR_SHAPE;
        }
    }
}

template <class KV, int D, int BS, int G, bool PH>
int mma_by_hg(int HG, const MmaOp& op)
{
    switch (HG) {
    case 1: return mma_run<KV, D, BS, G, 1, PH>(op);
    case 2: return mma_run<KV, D, BS, G, 2, PH>(op);
    case 4: return mma_run<KV, D, BS, G, 4, PH>(op);
    default: return PKV_ERR_SHAPE;
    }
}

template <class KV, int D, int BS, bool PH>
int mma_by_g(int G, int HG, const MmaOp& op)
{
    switch (G) {
    case 1: return mma_by_hg<KV, D, BS, 1, PH>(HG, op);
    case 2: return mma_by_hg<KV, D, BS, 2, PH>(HG, op);
    case 4: return mma_by_hg<KV, D, BS, 4, PH>(HG, op);
    case 5: return mma_by_hg<KV, D, BS, 5, PH>(HG, op);
    case 8: return mma_by_hg<KV, D, BS, 8, PH>(HG, op);
    default: return PKV_ERR_SHAPE;
    }
}

template <class KV, int D, bool PH>
int mma_by_bs(int BS, int G, int HG, const MmaOp& op)
{
    switch (BS) {
    case 16: return mma_by_g<KV, D, 16, PH>(G, HG, op);
    case 32: return mma_by_g<KV, D, 32, PH>(G, HG, op);
    default: return PKV_ERR_SHAPE;
    }
}

// head_dim 128 for every cache type; 64 as well for bf16 caches (WITH_D64)
template <class KV, bool WITH_D64, bool PH = false>
int mma_by_d(int D, int BS, int G, int HG, const MmaOp& op)
{
    if (D == 128)
        return mma_by_bs<KV, 128, PH>(BS, G, HG, op);
    if constexpr (WITH_D64) {
        if (D == 64)
            return mma_by_bs<KV, 64, PH>(BS, G, HG, op);
    }
    return PKV_ERR_SHAPE;
}

}  // namespace pkv
