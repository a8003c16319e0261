// The smallest and largest value of each key dimension over a block of tokens, for every KV head
// (update_key_bounds): what select_blocks scores a block by without reading its keys.
//
//   key_bounds[b][h][0][d] = max over the block's tokens of K[b][h][token][d]
//   key_bounds[b][h][1][d] = min of the same
//
// in bf16: exact for bf16 keys, the nearest bf16 of code * scale for 8-bit ones (rounding keeps
// the order, so the extremes are found among the codes and scaled once). Only a sequence's own
// tokens count: what lies behind its last one in a block is not read. A block is taken from the
// cache as a whole each time, so a call can be repeated and its result depends on no earlier one.
//
// One warp per (touched block, KV head), 16-byte loads, all of a block's rows in flight; the rows
// of a pass meet in a butterfly at the end. Bound: HBM for prompts (the keys once; the bounds are
// an eighth of them): 16 x 8192 tokens of 8 heads, bf16 (302 MB) 49.3 us, 6.1 TB/s, 94 % of the copy
// rate. Launch and dependent loads for a decode step: 64 tokens 3.1 us.
#include <cstdint>
#include <type_traits>

#include "touched.cuh"

namespace pkv {

namespace {

constexpr int kBoundsThreads = 128;

struct BoundsArgs {
    __nv_bfloat16* bounds;      // [num_blocks][num_kv_heads][2][head_dim]
    const uint8_t* k_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* row_offsets;
    const float* k_block_scales;   // [num_blocks][num_kv_heads] or null
    int32_t* err;
    float k_scale;
    long long work;             // items * num_kv_heads
    int num_tokens, num_seqs, num_kv_heads, max_blocks, num_blocks;
};

// Pairs of elements, compared with NaN winning (as a score built from it would be NaN).
__device__ __forceinline__ __nv_bfloat162 top(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 low(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __half2 top(__half2 a, __half2 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __half2 low(__half2 a, __half2 b) { return __hmin2_nan(a, b); }

template <class P>
__device__ __forceinline__ P shfl_pair(P x, int o)
{
    const uint32_t u = __shfl_xor_sync(kFullMask, *reinterpret_cast<const uint32_t*>(&x), o);
    return *reinterpret_cast<const P*>(&u);
}

__device__ __forceinline__ float2 pair_to_float2(__nv_bfloat162 x) { return __bfloat1622float2(x); }
__device__ __forceinline__ float2 pair_to_float2(__half2 x) { return __half22float2(x); }

// Code pair i (of two in a 32-bit word) as an exact f16 pair.
template <int KVDT>
__device__ __forceinline__ __half2 code_pair(uint32_t w, int i)
{
    if constexpr (KVDT == PKV_INT8)
        return __halves2half2(__int2half_rn((int)(int8_t)(w >> (16 * i))), __int2half_rn((int)(int8_t)(w >> (16 * i + 8))));
    else
        return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)),
                                                   KVDT == PKV_FP8_E4M3 ? __NV_E4M3 : __NV_E5M2));
}

template <int KVDT, int D, int BS>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(const BoundsArgs p)
{
    constexpr int EB = KVDT == PKV_BF16 ? 2 : 1;
    constexpr int LPR = D * EB / 16;     // lanes per row, 16 bytes each
    constexpr int RPP = 32 / LPR;        // rows a warp reads at a time
    constexpr int NP = BS >= RPP ? BS / RPP : 1;
    constexpr int E = 16 / EB;           // elements a lane holds of a row
    using P = typename std::conditional<KVDT == PKV_BF16, __nv_bfloat162, __half2>::type;
    const int lane = threadIdx.x & 31;
    const long long thread = (long long)blockIdx.x * kBoundsThreads + threadIdx.x;
    touched_flag(p.row_offsets, p.seq_lens, p.num_seqs, p.num_tokens, p.max_blocks * BS, thread, p.err);
    const long long w = thread >> 5;
    if (w >= p.work)
        return;
    const int h = (int)(w % p.num_kv_heads);
    const Touched t = touched_find(p.row_offsets, p.seq_lens, p.block_tables, p.num_seqs, p.num_tokens, BS,
                                   p.max_blocks, p.num_blocks, w / p.num_kv_heads, lane, h == 0 ? p.err : nullptr);
    if (t.phys < 0)
        return;
    const int held = min(BS, t.len - t.block * BS);   // >= 1
    const long long tile_id = (long long)t.phys * p.num_kv_heads + h;
    const uint8_t* tile = p.k_cache + tile_id * (BS * D * EB) + (lane % LPR) * 16;
    uint4 raw[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        // past the last token its row is read again: the extremes stay the same
        const int o = min(i * RPP + lane / LPR, held - 1);
        raw[i] = *reinterpret_cast<const uint4*>(tile + o * (D * EB));
    }
    P hi[E / 2], lo[E / 2];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t word[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            P x;
            if constexpr (KVDT == PKV_BF16)
                x = *reinterpret_cast<const P*>(&word[e]);
            else
                x = code_pair<KVDT>(word[e / 2], e & 1);
            hi[e] = i == 0 ? x : top(hi[e], x);
            lo[e] = i == 0 ? x : low(lo[e], x);
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            hi[e] = top(hi[e], shfl_pair(hi[e], o));
            lo[e] = low(lo[e], shfl_pair(lo[e], o));
        }
    if (lane < 2 * LPR) {   // the first row's lanes store the maxima, the second's the minima
        const bool is_min = lane >= LPR;
        float ks = 1.0f;
        if constexpr (KVDT != PKV_BF16)
            ks = p.k_block_scales ? __ldg(p.k_block_scales + tile_id) : p.k_scale;
        uint32_t out[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const P x = is_min ? lo[e] : hi[e];
            if constexpr (KVDT == PKV_BF16) {
                out[e] = *reinterpret_cast<const uint32_t*>(&x);
            } else {
                const float2 f = pair_to_float2(x);
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * ks, f.y * ks);
                out[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        __nv_bfloat16* dst = p.bounds + (tile_id * 2 + is_min) * D + (lane % LPR) * E;
#pragma unroll
        for (int e = 0; e < E / 2; e += 4)
            *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(out[e], out[e + 1], out[e + 2], out[e + 3]);
    }
}

template <int KVDT, int D, int BS>
int launch_bounds(const BoundsArgs& p, cudaStream_t stream)
{
    const long long grid = (p.work * 32 + kBoundsThreads - 1) / kBoundsThreads;
    key_bounds_kernel<KVDT, D, BS><<<(unsigned)grid, kBoundsThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <int KVDT, int D>
int bounds_by_bs(int BS, const BoundsArgs& p, cudaStream_t stream)
{
    switch (BS) {
    case 8: return launch_bounds<KVDT, D, 8>(p, stream);
    case 16: return launch_bounds<KVDT, D, 16>(p, stream);
    default: return launch_bounds<KVDT, D, 32>(p, stream);
    }
}

template <int KVDT>
int bounds_by_d(int D, int BS, const BoundsArgs& p, cudaStream_t stream)
{
    return D == 128 ? bounds_by_bs<KVDT, 128>(BS, p, stream) : bounds_by_bs<KVDT, 64>(BS, p, stream);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int update_key_bounds(void* key_bounds, const void* k_cache, const int32_t* block_tables,
                                         const int32_t* seq_lens, const int32_t* row_offsets, int num_tokens,
                                         int num_seqs, int num_kv_heads, int head_dim, int block_size,
                                         int max_blocks_per_seq, int num_blocks, int kv_dtype, float k_scale,
                                         const float* k_block_scales, int32_t* device_error, void* stream)
{
    const int st = touched_host_check(num_tokens, num_seqs, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                      num_blocks);
    if (st != PKV_OK)
        return st;
    const bool coded = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_FP8_E5M2 || kv_dtype == PKV_INT8;
    if ((kv_dtype != PKV_BF16 && !coded) || (k_block_scales && !coded))
        return PKV_ERR_DTYPE;
    if (coded && !k_block_scales && !(k_scale > 0.0f))
        return PKV_ERR_SHAPE;
    if (num_seqs == 0 || num_tokens == 0)
        return PKV_OK;
    if (!key_bounds || !k_cache || !block_tables || !seq_lens || !row_offsets)
        return PKV_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(key_bounds) & 15u) != 0 || (reinterpret_cast<uintptr_t>(k_cache) & 15u) != 0)
        return PKV_ERR_SHAPE;
    BoundsArgs p{};
    p.bounds = static_cast<__nv_bfloat16*>(key_bounds);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.row_offsets = row_offsets;
    p.k_block_scales = k_block_scales;
    p.err = device_error;
    p.k_scale = k_scale;
    p.work = touched_items(num_tokens, num_seqs, block_size) * num_kv_heads;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (kv_dtype) {
    case PKV_BF16: return bounds_by_d<PKV_BF16>(head_dim, block_size, p, s);
    case PKV_FP8_E4M3: return bounds_by_d<PKV_FP8_E4M3>(head_dim, block_size, p, s);
    case PKV_FP8_E5M2: return bounds_by_d<PKV_FP8_E5M2>(head_dim, block_size, p, s);
    default: return bounds_by_d<PKV_INT8>(head_dim, block_size, p, s);
    }
}
