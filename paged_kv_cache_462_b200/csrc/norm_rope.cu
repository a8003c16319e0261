// Per-head RMS norm of queries and keys, position rotation and the append of K and V to the
// paged cache, in one pass over the rows (qk_norm_rope, qk_norm_rope_and_cache).
//
//   y = x / sqrt(mean(x^2) + eps) * w           over the head_dim elements of one head's row
//   (a, b) -> (a c - b s, b c + a s)            for the rotary_dim / 2 pairs of the row, c and s
//                                               the token's row of the cos / sin table
//
// Everything is fp32 from the load to the one rounding of each stored element; the sum of
// squares is fp32 too. Bound: HBM (each row is read once and written once, about 8 operations an
// element).
//
// Layout: a row is held by head_dim / 8 lanes (16 or 8), 8 elements each, as two chunks of four
// chosen so that both elements of a rotation pair lie in one lane: chunks (4c, rotary/2 + 4c) for
// half-split pairs, (8c, 8c + 4) for interleaved ones and for the part that is not rotated. The
// only exchange is the butterfly sum of squares. A CTA takes one token (several when a token has
// few rows), so that a lane reads its cos and sin once for all its rows.
#include <cstdint>
#include <type_traits>

#include "device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormUnroll = 4;   // rows a lane group has in flight

struct NormRopeArgs {
    void* q_out;          // [T][Hq][D]
    void* k_out;          // [T][Hkv][D] (no cache) or null
    const void* q;        // rows of head_dim elements, heads contiguous, tokens *_stride apart
    const void* k;
    const void* v;        // null without a cache
    const void* q_weight;
    const void* k_weight;
    const float* cos_sin; // [num_positions][rotary]: cosines, then sines
    const int64_t* positions;
    const int64_t* slots;
    void* k_cache;
    void* v_cache;
    int32_t* err;
    long long q_stride, k_stride, v_stride;
    long long capacity;
    int num_tokens, num_heads, num_kv_heads, rotary, num_positions, block_size;
    int interleaved;
    int groups_per_token;   // lane groups that share a token's rows (a power of two)
    float eps, k_scale, v_scale;
};

// Four consecutive elements as they lie, widened when they are used.
template <class TIN>
struct Raw4;
template <>
struct Raw4<float> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void clear() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float4 get() const { return u; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void clear() { u = make_uint2(0u, 0u); }
    __device__ __forceinline__ float4 get() const
    {
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
};

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Four elements into the cache: as they are, or as codes of x / scale (IEEE division, nearest
// even, saturated; the conversions reshape_and_cache uses).
template <class TC, __nv_fp8_interpretation_t FMT>
__device__ __forceinline__ void cache4(TC* p, float4 x, float scale)
{
    if constexpr (sizeof(TC) > 1) {
        store4(p, x);
    } else if constexpr (std::is_same<TC, int8_t>::value) {
        const float v[4] = {x.x, x.y, x.z, x.w};
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float y = __fdiv_rn(v[i], scale);
            const int c = (y != y) ? 0 : __float2int_rn(fminf(fmaxf(y, -127.0f), 127.0f));
            w |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * i);
        }
        *reinterpret_cast<uint32_t*>(p) = w;
    } else {
        const float2 a = make_float2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale));
        const float2 b = make_float2(__fdiv_rn(x.z, scale), __fdiv_rn(x.w, scale));
        *reinterpret_cast<uint32_t*>(p) =
            static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, FMT)) |
            (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, FMT)) << 16);
    }
}

__device__ __forceinline__ float4 times(float4 a, float4 b)
{
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

template <class TIN, class TC, int D, __nv_fp8_interpretation_t FMT = __NV_E4M3>
__global__ void __launch_bounds__(kNormThreads, sizeof(TIN) == 2 ? 4 : 3) norm_rope_kernel(const NormRopeArgs p)
{
    constexpr int LPR = D / 8;                    // lanes per row
    constexpr int kGroups = kNormThreads / LPR;   // rows a CTA has at a time
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int per_token = p.groups_per_token, first = group % per_token;
    const long long t = (long long)blockIdx.x * (kGroups / per_token) + group / per_token;
    // (shuffles below: whole warps stay together, a group without a token works on nothing)
    const bool real = t < p.num_tokens;
    const int Hq = p.num_heads, Hkv = p.num_kv_heads;
    const int rows = Hq + Hkv + (p.v ? Hkv : 0);

    // this lane's two chunks of a row
    const int half = p.rotary / 2;
    const bool rotated = 8 * lane < p.rotary;
    const bool split = rotated && !p.interleaved;
    const int d0 = split ? 4 * lane : 8 * lane;
    const int d1 = split ? half + 4 * lane : 8 * lane + 4;

    const TIN* qrow = static_cast<const TIN*>(p.q) + t * p.q_stride;
    const TIN* krow = static_cast<const TIN*>(p.k) + t * p.k_stride;
    const TIN* vrow = static_cast<const TIN*>(p.v) + t * p.v_stride;
    Raw4<TIN> a[kNormUnroll], b[kNormUnroll];
    auto load_rows = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const int r = r0 + u * per_token;
            if (real && r < rows) {
                const TIN* x = r < Hq ? qrow + r * D : r < Hq + Hkv ? krow + (r - Hq) * D : vrow + (r - Hq - Hkv) * D;
                a[u].load(x + d0);
                b[u].load(x + d1);
            } else {
                a[u].clear();
                b[u].clear();
            }
        }
    };
    load_rows(first);    // before anything that waits for a load: the rows are what takes time

    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    bool live = real;
    long long slot = -1;
    if (real) {
        const long long pos = __ldg(p.positions + t);
        if (p.slots)
            slot = __ldg(p.slots + t);
        if (pos < 0 || pos >= p.num_positions) {
            if (lane == 0 && first == 0 && p.err)
                atomicOr(p.err, PKV_DEVERR_POSITION);
            live = false;
        } else {
            if (rotated) {
                const float* cs = p.cos_sin + pos * p.rotary;
                c = __ldg(reinterpret_cast<const float4*>(cs + 4 * lane));
                s = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * lane));
            }
            if (slot >= p.capacity) {
                if (lane == 0 && first == 0 && p.err)
                    atomicOr(p.err, PKV_DEVERR_SLOT);
                slot = -1;
            }
        }
    }
    Raw4<TIN> qw0, qw1, kw0, kw1;
    qw0.load(static_cast<const TIN*>(p.q_weight) + d0);
    qw1.load(static_cast<const TIN*>(p.q_weight) + d1);
    kw0.load(static_cast<const TIN*>(p.k_weight) + d0);
    kw1.load(static_cast<const TIN*>(p.k_weight) + d1);
    // offset of this token's row of KV head 0 in the caches; heads lie block_size rows apart
    const long long head_rows = (long long)p.block_size * D;
    const long long blk = slot >= 0 ? slot / p.block_size : 0;
    const long long at = blk * Hkv * head_rows + (slot >= 0 ? slot - blk * p.block_size : 0) * D;

    for (int r0 = first;;) {
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const int r = r0 + u * per_token;
            const float4 xa = a[u].get(), xb = b[u].get();
            float ss = xa.x * xa.x + xa.y * xa.y + xa.z * xa.z + xa.w * xa.w + xb.x * xb.x + xb.y * xb.y +
                       xb.z * xb.z + xb.w * xb.w;
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1)
                ss += __shfl_xor_sync(kFullMask, ss, o);
            if (!live || r >= rows)
                continue;
            if (r >= Hq + Hkv) {   // a V row: only appended
                if (slot >= 0) {
                    TC* dst = static_cast<TC*>(p.v_cache) + at + (r - Hq - Hkv) * head_rows;
                    cache4<TC, FMT>(dst + d0, xa, p.v_scale);
                    cache4<TC, FMT>(dst + d1, xb, p.v_scale);
                }
                continue;
            }
            const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
            const bool is_q = r < Hq;
            const float4 i4 = make_float4(inv, inv, inv, inv);
            const float4 x = times(times(xa, i4), is_q ? qw0.get() : kw0.get());
            const float4 y = times(times(xb, i4), is_q ? qw1.get() : kw1.get());
            float4 u0 = x, u1 = y;
            if (split) {
                u0 = make_float4(x.x * c.x - y.x * s.x, x.y * c.y - y.y * s.y, x.z * c.z - y.z * s.z,
                                 x.w * c.w - y.w * s.w);
                u1 = make_float4(y.x * c.x + x.x * s.x, y.y * c.y + x.y * s.y, y.z * c.z + x.z * s.z,
                                 y.w * c.w + x.w * s.w);
            } else if (rotated) {
                u0 = make_float4(x.x * c.x - x.y * s.x, x.y * c.x + x.x * s.x, x.z * c.y - x.w * s.y,
                                 x.w * c.y + x.z * s.y);
                u1 = make_float4(y.x * c.z - y.y * s.z, y.y * c.z + y.x * s.z, y.z * c.w - y.w * s.w,
                                 y.w * c.w + y.z * s.w);
            }
            if (is_q || !p.slots) {
                TIN* dst = is_q ? static_cast<TIN*>(p.q_out) + (t * Hq + r) * D
                                : static_cast<TIN*>(p.k_out) + (t * Hkv + (r - Hq)) * D;
                store4(dst + d0, u0);
                store4(dst + d1, u1);
            } else if (slot >= 0) {
                TC* dst = static_cast<TC*>(p.k_cache) + at + (r - Hq) * head_rows;
                cache4<TC, FMT>(dst + d0, u0, p.k_scale);
                cache4<TC, FMT>(dst + d1, u1, p.k_scale);
            }
        }
        r0 += kNormUnroll * per_token;
        if (r0 - first >= rows)
            break;
        load_rows(r0);
    }
}

template <class TIN, class TC, int D, __nv_fp8_interpretation_t FMT = __NV_E4M3>
int launch_norm_rope(NormRopeArgs p, cudaStream_t stream)
{
    constexpr int kGroups = kNormThreads / (D / 8);
    const int rows = p.num_heads + p.num_kv_heads + (p.v ? p.num_kv_heads : 0);
    int per = 1;
    while (per < kGroups && per < rows)
        per *= 2;
    p.groups_per_token = per;
    const int tokens_per_cta = kGroups / per;
    const int grid = (p.num_tokens + tokens_per_cta - 1) / tokens_per_cta;
    norm_rope_kernel<TIN, TC, D, FMT><<<grid, kNormThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <class TIN, int D>
int norm_rope_by_cache(const NormRopeArgs& p, int kv_dtype, cudaStream_t stream)
{
    switch (kv_dtype) {
    case PKV_FP8_E4M3: return launch_norm_rope<TIN, uint8_t, D, __NV_E4M3>(p, stream);
    case PKV_FP8_E5M2: return launch_norm_rope<TIN, uint8_t, D, __NV_E5M2>(p, stream);
    case PKV_INT8: return launch_norm_rope<TIN, int8_t, D>(p, stream);
    default: return launch_norm_rope<TIN, TIN, D>(p, stream);
    }
}

// Bytes [a, a + na) and [b, b + nb) have one in common.
bool overlap(const void* a, long long na, const void* b, long long nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Output rows (contiguous) against the input rows they must not reach: allowed are no byte in
// common, or the very rows they are made from, in the same order.
bool rows_clash(const void* out, long long out_row, const void* in, long long in_row, long long in_stride, long long T,
                int elt, bool same)
{
    if (same && out == in && (T == 1 || in_stride == in_row))
        return false;
    return overlap(out, T * out_row * elt, in, ((T - 1) * in_stride + in_row) * elt);
}

int norm_rope_impl(NormRopeArgs p, int head_dim, int num_blocks, int in_dtype, int kv_dtype, bool cached,
                   cudaStream_t stream)
{
    if (p.num_tokens < 0 || p.num_heads <= 0 || p.num_kv_heads <= 0 || (head_dim != 64 && head_dim != 128) ||
        p.rotary < 0 || p.rotary > head_dim || p.rotary % 8 != 0 || p.num_positions < 0 || !(p.eps >= 0.0f))
        return PKV_ERR_SHAPE;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16)
        return PKV_ERR_DTYPE;
    const bool coded = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_FP8_E5M2 || kv_dtype == PKV_INT8;
    if (cached && kv_dtype != in_dtype && !coded)
        return PKV_ERR_DTYPE;
    if (cached && (num_blocks <= 0 || (p.block_size != 8 && p.block_size != 16 && p.block_size != 32)))
        return PKV_ERR_SHAPE;
    if (cached && coded && !(p.k_scale > 0.0f && p.v_scale > 0.0f))
        return PKV_ERR_SHAPE;
    if (p.num_tokens == 0)
        return PKV_OK;
    if (!p.q_out || !p.q || !p.k || !p.q_weight || !p.k_weight || (p.rotary > 0 && !p.cos_sin) || !p.positions)
        return PKV_ERR_NULL;
    if (cached ? (!p.v || !p.k_cache || !p.v_cache || !p.slots) : !p.k_out)
        return PKV_ERR_NULL;
    const int elt = in_dtype == PKV_F32 ? 4 : 2;
    const long long q_row = (long long)p.num_heads * head_dim, k_row = (long long)p.num_kv_heads * head_dim;
    if (p.num_tokens > 1 && (p.q_stride < q_row || p.k_stride < k_row || (cached && p.v_stride < k_row)))
        return PKV_ERR_SHAPE;
    auto off16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    auto bad_stride = [&](long long s) { return p.num_tokens > 1 && s * elt % 16 != 0; };
    if (off16(p.q) || off16(p.k) || off16(p.q_out) || off16(p.q_weight) || off16(p.k_weight) || off16(p.cos_sin) ||
        bad_stride(p.q_stride) || bad_stride(p.k_stride) || (cached && (off16(p.v) || bad_stride(p.v_stride))) ||
        (cached ? off16(p.k_cache) || off16(p.v_cache) : off16(p.k_out)))
        return PKV_ERR_SHAPE;
    // every CTA reads and writes its own tokens' rows at its own time
    const long long T = p.num_tokens;
    if (rows_clash(p.q_out, q_row, p.q, q_row, p.q_stride, T, elt, true) ||
        rows_clash(p.q_out, q_row, p.k, k_row, p.k_stride, T, elt, false) ||
        (cached && rows_clash(p.q_out, q_row, p.v, k_row, p.v_stride, T, elt, false)))
        return PKV_ERR_SHAPE;
    if (!cached && (rows_clash(p.k_out, k_row, p.k, k_row, p.k_stride, T, elt, true) ||
                    rows_clash(p.k_out, k_row, p.q, q_row, p.q_stride, T, elt, false) ||
                    overlap(p.k_out, T * k_row * elt, p.q_out, T * q_row * elt)))
        return PKV_ERR_SHAPE;
    p.capacity = (long long)num_blocks * p.block_size;
    const int kv = cached ? kv_dtype : in_dtype;
    if (in_dtype == PKV_F32)
        return head_dim == 128 ? norm_rope_by_cache<float, 128>(p, kv, stream)
                               : norm_rope_by_cache<float, 64>(p, kv, stream);
    return head_dim == 128 ? norm_rope_by_cache<__nv_bfloat16, 128>(p, kv, stream)
                           : norm_rope_by_cache<__nv_bfloat16, 64>(p, kv, stream);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API int qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, const void* q_weight,
                         const void* k_weight, float eps, const float* cos_sin, const int64_t* positions,
                         int num_tokens, int num_heads, int num_kv_heads, int head_dim, int rotary_dim,
                         int num_positions, int interleaved, int64_t q_stride, int64_t k_stride, int dtype,
                         int32_t* device_error, void* stream)
{
    NormRopeArgs p{};
    p.q_out = q_out;
    p.k_out = k_out;
    p.q = q;
    p.k = k;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.err = device_error;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary = rotary_dim;
    p.num_positions = num_positions;
    p.block_size = 16;
    p.interleaved = interleaved;
    p.eps = eps;
    return norm_rope_impl(p, head_dim, 1, dtype, dtype, false, static_cast<cudaStream_t>(stream));
}

PKV_API int qk_norm_rope_and_cache(void* q_out, const void* q, const void* k, const void* v, const void* q_weight,
                                   const void* k_weight, float eps, const float* cos_sin, const int64_t* positions,
                                   void* k_cache, void* v_cache, const int64_t* slot_mapping, int num_tokens,
                                   int num_heads, int num_kv_heads, int head_dim, int rotary_dim, int num_positions,
                                   int block_size, int num_blocks, int interleaved, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, int in_dtype, int kv_dtype, float k_scale,
                                   float v_scale, int32_t* device_error, void* stream)
{
    NormRopeArgs p{};
    p.q_out = q_out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.err = device_error;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary = rotary_dim;
    p.num_positions = num_positions;
    p.block_size = block_size;
    p.interleaved = interleaved;
    p.eps = eps;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return norm_rope_impl(p, head_dim, num_blocks, in_dtype, kv_dtype, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
