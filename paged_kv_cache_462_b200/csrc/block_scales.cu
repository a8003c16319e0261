// Append into an 8-bit cache with one scale for each block of tokens and KV head
// (reshape_and_cache_block_scales).
//
// A block's scale is a power of two: the smallest 2^e, e in [-50, 50], with absmax <= qmax * 2^e
// (qmax 448, 57344 or 127) over what the block holds, so that x / scale and code * scale are exact
// in fp32 and every code is the one nearest rounding of its value. Rows that join a block with
// older tokens can only raise its scale; the older codes are then re-encoded from their values
// (exact for FP8 codes that stay normal, rounded once more for INT8 and subnormal ones).
//
// One warp per (touched block, KV head, K or V): it reads the block's new rows once, keeps them in
// registers through the maximum and encodes them, so nothing is read twice and no two warps meet
// in a block. Bound: HBM for prompts (rows in, codes out): 16 ragged chunks of 801 to 2047 rows, INT8,
// 8 heads of 128 (142 MB) 28.1 us, 5.1 TB/s, 77 % of the copy rate, of which the arithmetic of rounding
// hides all but a quarter (68 us with a compare and a conversion per element instead of the packed
// maximum and the one-FMA rounding). The launch and four dependent loads (offsets, lengths, table,
// rows) for a decode step: 128 tokens 4.3 us.
#include <cstdint>

#include "touched.cuh"

namespace pkv {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;
// CTAs up to which a block's tiles are shared between several: 128 single tokens (1056 CTAs) 4.3 us
// against 5.3 us with a CTA per block, 256 tokens (2112) 6.7 against 5.7 us, 16 chunks of 256 (1152)
// 6.7 against 7.1 us
constexpr long long kAppendSplit = 148 * 12;
constexpr int kScaleLo = -50, kScaleHi = 50;

template <int KVDT>
struct Code;
template <>
struct Code<PKV_FP8_E4M3> {
    static constexpr __nv_fp8_interpretation_t kFmt = __NV_E4M3;
    static constexpr int kTop = 8;                 // qmax = 1.75 * 2^8
    static constexpr uint32_t kTopMantissa = 0x600000u;
};
template <>
struct Code<PKV_FP8_E5M2> {
    static constexpr __nv_fp8_interpretation_t kFmt = __NV_E5M2;
    static constexpr int kTop = 15;                // qmax = 1.75 * 2^15
    static constexpr uint32_t kTopMantissa = 0x600000u;
};
template <>
struct Code<PKV_INT8> {
    static constexpr __nv_fp8_interpretation_t kFmt = __NV_E4M3;   // unused
    static constexpr int kTop = 6;                 // qmax = 127/64 * 2^6
    static constexpr uint32_t kTopMantissa = 0x7e0000u;
};

// The smallest power of two 2^e with `absmax` (finite, >= 0) <= qmax * 2^e, e clamped.
template <int KVDT>
__device__ __forceinline__ float scale_for(float absmax)
{
    const uint32_t u = __float_as_uint(absmax);
    int e = (int)(u >> 23) - 127 - Code<KVDT>::kTop + ((u & 0x7fffffu) > Code<KVDT>::kTopMantissa ? 1 : 0);
    e = e < kScaleLo ? kScaleLo : (e > kScaleHi ? kScaleHi : e);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// x / scale; exact by the reciprocal when the scale is a power of two (inv != 0)
__device__ __forceinline__ float over(float x, float scale, float inv) { return inv != 0.f ? x * inv : __fdiv_rn(x, scale); }

// Eight values -> eight codes of x / scale, nearest even, saturated (NaN: a NaN code, INT8 0).
template <int KVDT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float scale, float inv)
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t packed = 0;
        if constexpr (KVDT == PKV_INT8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = over(f[4 * h + i], scale, inv);
                const int c = (y != y) ? 0 : __float2int_rn(fminf(fmaxf(y, -127.0f), 127.0f));
                packed |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 y = make_float2(over(f[4 * h + 2 * i], scale, inv), over(f[4 * h + 2 * i + 1], scale, inv));
                packed |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, Code<KVDT>::kFmt))
                          << (16 * i);
            }
        }
        w[h] = packed;
    }
    return make_uint2(w[0], w[1]);
}

// The same for values that no code saturates for (finite ones, |x| <= qmax * scale, a power of two).
// INT8: x * inv + 1.5 * 2^23 rounds to an integer in the low bits, nearest even, two's complement.
template <int KVDT>
__device__ __forceinline__ uint2 encode8_inside(const float (&f)[8], float inv)
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (KVDT == PKV_INT8) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = __float_as_uint(fmaf(f[4 * h + i], inv, 12582912.0f));
            w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        } else {
            uint32_t packed = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                packed |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                              make_float2(f[4 * h + 2 * i] * inv, f[4 * h + 2 * i + 1] * inv), __NV_SATFINITE,
                              Code<KVDT>::kFmt))
                          << (16 * i);
            w[h] = packed;
        }
    }
    return make_uint2(w[0], w[1]);
}

// Eight codes -> their values in units of the scale, exactly.
template <int KVDT>
__device__ __forceinline__ void decode8(uint2 c, float (&f)[8])
{
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (KVDT == PKV_INT8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[4 * h + i] = (float)(int8_t)(w[h] >> (8 * i));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[h] >> (16 * i)), Code<KVDT>::kFmt);
                const float2 y = __half22float2(__half2(r));
                f[4 * h + 2 * i] = y.x;
                f[4 * h + 2 * i + 1] = y.y;
            }
        }
    }
}

struct AppendBlockArgs {
    const void* k;
    const void* v;
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scales;    // [num_blocks][num_kv_heads]
    float* v_scales;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* row_offsets;
    int32_t* err;
    long long k_stride, v_stride;
    int num_tokens, num_seqs, num_kv_heads, max_blocks, num_blocks;
};

// Eight consecutive elements as they lie.
template <class TIN>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    // the largest magnitude's bits, NaN above infinity above the rest
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
        float f[8];
        get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ uint32_t top() const
    {
        constexpr uint32_t M = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        widen_word(KvBF16{}, a.x, f + 0);
        widen_word(KvBF16{}, a.y, f + 2);
        widen_word(KvBF16{}, a.z, f + 4);
        widen_word(KvBF16{}, a.w, f + 6);
    }
};

template <class TIN, int KVDT, int D, int BS>
__global__ void __launch_bounds__(kAppendThreads, BS / (32 / (D / 8)) * sizeof(TIN) <= 16 ? 5 : 3) append_block_scales_kernel(const AppendBlockArgs p)
{
    constexpr int LPR = D / 8;           // lanes per row, 8 elements each
    constexpr int RPP = 32 / LPR;        // rows a warp reads at a time
    constexpr int NP = BS / RPP;         // passes over a whole block
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    if (blockIdx.y == 0)
        touched_flag(p.row_offsets, p.seq_lens, p.num_seqs, p.num_tokens, p.max_blocks * BS,
                     (long long)blockIdx.x * kAppendThreads + threadIdx.x, p.err);
    // (only an item's first warp reports its block id)
    const Touched t = touched_find(p.row_offsets, p.seq_lens, p.block_tables, p.num_seqs, p.num_tokens, BS,
                                   p.max_blocks, p.num_blocks, blockIdx.x, lane,
                                   blockIdx.y == 0 && warp == 0 ? p.err : nullptr);
    if (t.phys < 0)
        return;
    const int begin = max(0, t.first - t.block * BS);        // this block's new offsets: [begin, end)
    const int end = min(BS, t.len - t.block * BS);
    const long long row0 = (long long)t.row + t.block * BS - t.first;   // row of offset 0 (may be before the call's)
    // the block's tiles: KV head job / 2, K or V
    for (int job = blockIdx.y * kAppendWarps + warp; job < 2 * p.num_kv_heads; job += gridDim.y * kAppendWarps) {
        const bool is_v = job & 1;
        const int h = job >> 1;
        const long long stride = is_v ? p.v_stride : p.k_stride;
        const TIN* src = static_cast<const TIN*>(is_v ? p.v : p.k) + (long long)h * D + (lane % LPR) * 8;
        uint8_t* tile = (is_v ? p.v_cache : p.k_cache) + ((long long)t.phys * p.num_kv_heads + h) * (BS * D) + (lane % LPR) * 8;
        float* scale_at = (is_v ? p.v_scales : p.k_scales) + (long long)t.phys * p.num_kv_heads + h;
        const float before = begin > 0 ? *scale_at : 0.f;

        Raw8<TIN> raw[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int o = i * RPP + lane / LPR;
            if (o >= begin && o < end)
                raw[i].load(src + (row0 + o) * stride);
            else
                raw[i].clear();
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            top = max(top, raw[i].top());
        top = __reduce_max_sync(kFullMask, top);
        const bool all_finite = top < 0x7f800000u;
        float mx = __uint_as_float(top);
        if (!all_finite) {                   // infinities and NaN set no scale
            mx = 0.f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float f[8];
                raw[i].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = fabsf(f[e]);
                    mx = a <= 3.402823466e38f ? fmaxf(mx, a) : mx;
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, o));
        }
        const float need = scale_for<KVDT>(mx);
        const float after = fmaxf(before, need);
        const bool power = (__float_as_uint(after) & 0x7fffffu) == 0u;
        const float inv = power ? __uint_as_float((254u << 23) - __float_as_uint(after)) : 0.f;
        // below the largest scale no finite value lies beyond the codes
        const bool inside = all_finite && power && after < __uint_as_float((uint32_t)(kScaleHi + 127) << 23);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int o = i * RPP + lane / LPR;
            if (o >= begin && o < end) {
                float f[8];
                raw[i].get(f);
                *reinterpret_cast<uint2*>(tile + o * D) =
                    inside ? encode8_inside<KVDT>(f, inv) : encode8<KVDT>(f, after, inv);
            }
        }
        if (begin > 0 && after > before) {   // the scale grew: the older codes in its units
            for (int o = lane / LPR; o < begin; o += RPP) {
                float f[8];
                decode8<KVDT>(*reinterpret_cast<const uint2*>(tile + o * D), f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] *= before;
                *reinterpret_cast<uint2*>(tile + o * D) = encode8<KVDT>(f, after, inv);
            }
        }
        if (lane == 0 && !(before == after))
            *scale_at = after;
    }
}

template <class TIN, int KVDT, int D, int BS>
int launch_append(const AppendBlockArgs& p, cudaStream_t stream)
{
    const long long items = touched_items(p.num_tokens, p.num_seqs, BS);
    // a CTA per block; where there are few, several, so that no warp has two tiles
    const int jobs = (2 * p.num_kv_heads + kAppendWarps - 1) / kAppendWarps;
    const int split = items * jobs <= kAppendSplit ? jobs : 1;
    append_block_scales_kernel<TIN, KVDT, D, BS><<<dim3((unsigned)items, split), kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <class TIN, int KVDT, int D>
int append_by_bs(int BS, const AppendBlockArgs& p, cudaStream_t stream)
{
    switch (BS) {
    case 8: return launch_append<TIN, KVDT, D, 8>(p, stream);
    case 16: return launch_append<TIN, KVDT, D, 16>(p, stream);
    default: return launch_append<TIN, KVDT, D, 32>(p, stream);
    }
}

template <class TIN, int KVDT>
int append_by_d(int D, int BS, const AppendBlockArgs& p, cudaStream_t stream)
{
    return D == 128 ? append_by_bs<TIN, KVDT, 128>(BS, p, stream) : append_by_bs<TIN, KVDT, 64>(BS, p, stream);
}

template <class TIN>
int append_by_code(int kv_dtype, int D, int BS, const AppendBlockArgs& p, cudaStream_t stream)
{
    switch (kv_dtype) {
    case PKV_FP8_E4M3: return append_by_d<TIN, PKV_FP8_E4M3>(D, BS, p, stream);
    case PKV_FP8_E5M2: return append_by_d<TIN, PKV_FP8_E5M2>(D, BS, p, stream);
    default: return append_by_d<TIN, PKV_INT8>(D, BS, p, stream);
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int reshape_and_cache_block_scales(const void* k, const void* v, void* k_cache, void* v_cache,
                                                      float* k_block_scales, float* v_block_scales,
                                                      const int32_t* block_tables, const int32_t* seq_lens,
                                                      const int32_t* row_offsets, int num_tokens, int num_seqs,
                                                      int num_kv_heads, int head_dim, int block_size,
                                                      int max_blocks_per_seq, int num_blocks, int64_t k_stride,
                                                      int64_t v_stride, int in_dtype, int kv_dtype,
                                                      int32_t* device_error, void* stream)
{
    const int st = touched_host_check(num_tokens, num_seqs, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                      num_blocks);
    if (st != PKV_OK)
        return st;
    if ((in_dtype != PKV_F32 && in_dtype != PKV_BF16) ||
        (kv_dtype != PKV_FP8_E4M3 && kv_dtype != PKV_FP8_E5M2 && kv_dtype != PKV_INT8))
        return PKV_ERR_DTYPE;
    if (num_seqs == 0 || num_tokens == 0)
        return PKV_OK;
    if (!k || !v || !k_cache || !v_cache || !k_block_scales || !v_block_scales || !block_tables || !seq_lens ||
        !row_offsets)
        return PKV_ERR_NULL;
    const int elt = in_dtype == PKV_F32 ? 4 : 2;
    auto off16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    if (off16(k) || off16(v) || off16(k_cache) || off16(v_cache))
        return PKV_ERR_SHAPE;
    if (num_tokens > 1 && (k_stride < (int64_t)num_kv_heads * head_dim || v_stride < (int64_t)num_kv_heads * head_dim ||
                           k_stride * elt % 16 != 0 || v_stride * elt % 16 != 0))
        return PKV_ERR_SHAPE;
    AppendBlockArgs p{};
    p.k = k;
    p.v = v;
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scales = k_block_scales;
    p.v_scales = v_block_scales;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.row_offsets = row_offsets;
    p.err = device_error;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return in_dtype == PKV_F32 ? append_by_code<float>(kv_dtype, head_dim, block_size, p, s)
                               : append_by_code<__nv_bfloat16>(kv_dtype, head_dim, block_size, p, s);
}
