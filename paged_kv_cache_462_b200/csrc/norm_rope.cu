// Per-head RMS norm of queries and keys, position rotation and the append of K and V to the
// paged cache, in one pass over the rows (qk_norm_rope, qk_norm_rope_and_cache).
//
//   y = x / sqrt(mean(x^2) + eps) * w           over the head_dim elements of one head's row
//   (a, b) -> (a c - b s, b c + a s)            for the rotary_dim / 2 pairs of the row, c and s
//                                               the token's row of the cos / sin table
//
// Everything is fp32 from the load to the one rounding of each stored element; the sum of
// squares is fp32 too. Bound: HBM (each row is read once and written once), with the issue slots not
// far behind. Measured (40 query and 8 KV heads of 128, bf16, 8192 tokens, 239 MB): 44.8 us, 5.3 TB/s,
// 82 % of the copy rate, where a call finds what the one before left in L2, 49.1 us, 75 %, with other
// inputs each time; with a CTA per token and a load per row 63 us, 70 % of the issue slots busy.
// Four tokens: 3.5 us, launch and latency.
//
// Layout: a row is held by head_dim / 8 lanes (16 or 8), 8 elements each, as two chunks of four
// chosen so that both elements of a rotation pair lie in one lane: chunks (4c, rotary/2 + 4c) for
// half-split pairs, (8c, 8c + 4) for interleaved ones and for the part that is not rotated. The
// only exchange is the butterfly sum of squares. A thread has up to four rows of a token and the
// same rows of every token it takes (two or three CTAs an SM, tokens dealt out in turn), so where they
// go is worked out once and a token's cos and sin serve all of them. A warp of its own brings the
// rows into a ring of stages by bulk copies, tokens ahead of the arithmetic: a token's rows of q, of
// k and of v are each one run of memory.
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
    int block_shift;        // log2 of block_size
    int stages, stage_bytes;
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
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = u; }
    __device__ __forceinline__ float4 get() const { return u; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void clear() { u = make_uint2(0u, 0u); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = u; }
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

// Four fp32 numbers as two pairs for the packed fp32 instructions (two products or fused
// multiply-adds each, rounded as the single ones are).
struct Pairs {
    unsigned long long lo, hi;
};
__device__ __forceinline__ Pairs pairs(float4 x)
{
    Pairs p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.lo) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.hi) : "f"(x.z), "f"(x.w));
    return p;
}
__device__ __forceinline__ float4 singles(Pairs p)
{
    float4 x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(p.lo));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.z), "=f"(x.w) : "l"(p.hi));
    return x;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pairs times(Pairs a, Pairs b) { return Pairs{mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Pairs plus_times(Pairs a, Pairs b, Pairs c)   // a b + c
{
    return Pairs{fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)};
}

// Shared memory of a CTA: a ring of stages, each the rows of the tokens a CTA works on at a time, as
// they lie in memory; the weights in fp32; the ring's barriers.
template <class TIN, int D>
struct NormSmem {
    static constexpr int kBudget = sizeof(TIN) == 2 ? 64 * 1024 : 96 * 1024;   // three or two CTAs an SM
    static constexpr int kMaxStages = 8;
    static constexpr int kWeights = 2 * D * 4;
    static constexpr int kBarriers = 2 * kMaxStages * 8 + 16;
    static int stages(int stage_bytes)
    {
        const int n = kBudget / stage_bytes;
        return n > kMaxStages ? kMaxStages : n;
    }
    static size_t bytes(int stages, int stage_bytes) { return (size_t)stages * stage_bytes + kWeights + kBarriers; }
};

// WHOLE: half-split pairs over the whole head (rotary == D), what most models use: the chunks' places
// are known when this is compiled (8192 tokens as above: 44.8 us, the general form 58.7 us; four
// tokens 3.5 and 4.0 us). CACHED: K and V go to the caches.
template <class TIN, class TC, int D, __nv_fp8_interpretation_t FMT, bool WHOLE, bool CACHED>
__global__ void __launch_bounds__(kNormThreads + 32, sizeof(TIN) == 2 ? 3 : 2) norm_rope_kernel(const NormRopeArgs p)
{
    constexpr int LPR = D / 8;                    // lanes per row
    constexpr int kGroups = kNormThreads / LPR;   // rows a CTA has at a time
    constexpr int kWarps = kNormThreads / 32;
    constexpr int kRowBytes = D * sizeof(TIN);
    extern __shared__ __align__(128) uint8_t smem[];
    const int S = p.stages;
    float* weights = reinterpret_cast<float*>(smem + S * p.stage_bytes);          // [2][D]
    uint64_t* full = reinterpret_cast<uint64_t*>(weights + 2 * D);
    uint64_t* empty = full + S;
    volatile int* abort_flag = reinterpret_cast<int*>(empty + S);

    const int per_token = p.groups_per_token, tokens = kGroups / per_token;   // tokens at a time
    const int stride = gridDim.x * tokens;                                     // from one set to the next
    const int Hq = p.num_heads, Hkv = p.num_kv_heads;
    const int rows = Hq + Hkv + (CACHED ? Hkv : 0);
    const int row_lo = blockIdx.y * (kNormUnroll * per_token);                 // this CTA's rows of each token
    const int row_n = min(rows - row_lo, kNormUnroll * per_token);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 2 * D; i += kNormThreads + 32)
        weights[i] = to_float(static_cast<const TIN*>(i < D ? p.q_weight : p.k_weight)[i % D]);
    __syncthreads();

    // =========================== producer warp: lane i brings token i of a set
    if (threadIdx.x >= kNormThreads) {
        const int lane = threadIdx.x & 31;
        // this CTA's rows are up to three runs of memory: of q, of k and of v
        const int nq = max(0, min(Hq, row_lo + row_n) - row_lo);
        const int k_lo = max(0, row_lo - Hq), nk = max(0, min(Hkv, row_lo + row_n - Hq) - k_lo);
        const int v_lo = max(0, row_lo - Hq - Hkv), nv = row_n - nq - nk;
        bool aborted = false;
        int k = 0;
        for (int base = blockIdx.x * tokens; base < p.num_tokens && !aborted; base += stride, ++k) {
            const int st = k % S;
            const int n = min(tokens, p.num_tokens - base);
            if (lane == 0) {
                if (*abort_flag || (k >= S && !mbar_wait_bounded(&empty[st], ((k / S) - 1) & 1)))
                    aborted = true;
                else
                    mbar_arrive_expect_tx(&full[st], n * row_n * kRowBytes);
            }
            aborted = __shfl_sync(kFullMask, aborted ? 1 : 0, 0) != 0;
            __syncwarp();
            if (!aborted && lane < n) {
                const long long t = base + lane;
                uint8_t* dst = smem + st * p.stage_bytes + lane * (row_n * kRowBytes);
                if (nq)
                    bulk_copy_g2s(dst, static_cast<const TIN*>(p.q) + t * p.q_stride + (long long)row_lo * D,
                                  nq * kRowBytes, &full[st]);
                if (nk)
                    bulk_copy_g2s(dst + nq * kRowBytes, static_cast<const TIN*>(p.k) + t * p.k_stride + (long long)k_lo * D,
                                  nk * kRowBytes, &full[st]);
                if (nv)
                    bulk_copy_g2s(dst + (nq + nk) * kRowBytes,
                                  static_cast<const TIN*>(p.v) + t * p.v_stride + (long long)v_lo * D, nv * kRowBytes,
                                  &full[st]);
            }
        }
        if (aborted && lane == 0) {      // a wait gave up: the copies under way end before the CTA does
            *abort_flag = 1;
            if (p.err)
                atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            for (int i = max(0, k - 1 - S); i < k - 1; ++i)
                (void)mbar_wait_bounded(&full[i % S], (i / S) & 1);
        }
        return;
    }

    // =========================== the other warps
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int first = group % per_token, set_token = group / per_token;
    const bool report = lane == 0 && first == 0 && blockIdx.y == 0 && p.err != nullptr;

    // this lane's two chunks of a row
    const int half = WHOLE ? D / 2 : p.rotary / 2;
    const bool rotated = WHOLE || 8 * lane < p.rotary;
    const bool split = WHOLE || (rotated && !p.interleaved);
    const int d0 = split ? 4 * lane : 8 * lane;
    const int d1 = WHOLE ? d0 + D / 2 : split ? half + 4 * lane : 8 * lane + 4;
    const int apart = WHOLE ? D / 2 : d1 - d0;

    // this thread's rows, the same ones of every token it takes, and where they go but for the token
    enum Kind { kQ, kK, kV, kNone };
    int kind[kNormUnroll];
    void* dst[kNormUnroll];
    const long long head_rows = (long long)p.block_size * D;   // elements between a block's KV heads
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        const int r = row_lo + first + u * per_token;
        if (r < Hq) {
            kind[u] = kQ;
            dst[u] = static_cast<TIN*>(p.q_out) + (long long)r * D + d0;
        } else if (r < Hq + Hkv) {
            kind[u] = kK;
            dst[u] = CACHED ? static_cast<void*>(static_cast<TC*>(p.k_cache) + (r - Hq) * head_rows + d0)
                            : static_cast<void*>(static_cast<TIN*>(p.k_out) + (long long)(r - Hq) * D + d0);
        } else if (r < rows) {
            kind[u] = kV;
            dst[u] = static_cast<TC*>(p.v_cache) + (r - Hq - Hkv) * head_rows + d0;
        } else {
            kind[u] = kNone;
            dst[u] = nullptr;
        }
    }
    const TIN* staged = reinterpret_cast<const TIN*>(smem) + (set_token * row_n + first) * D + d0;

    auto load_index = [&](int tok, long long& pos, long long& slot) {
        pos = -1;
        slot = -1;
        if (tok < p.num_tokens) {
            pos = __ldg(p.positions + tok);
            if (CACHED)
                slot = __ldg(p.slots + tok);
        }
    };
    auto load_angles = [&](long long pos, float4& c, float4& s) {
        c = make_float4(1.f, 1.f, 1.f, 1.f);
        s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rotated && pos >= 0 && pos < p.num_positions) {
            const float* cs = p.cos_sin + pos * p.rotary;
            c = __ldg(reinterpret_cast<const float4*>(cs + 4 * lane));
            s = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * lane));
        }
    };
    // the next token's cosines and sines and the position of the one after it are on their way while
    // one is worked on (num_tokens and two strides fit 32 bits: the launcher bounds both)
    int t = blockIdx.x * tokens + set_token;
    float4 c, s, nc, ns;
    long long pos, slot, npos, nslot, npos2, nslot2;
    load_index(t, pos, slot);
    load_index(t + stride, npos, nslot);
    load_angles(pos, c, s);

    int k = 0;
    for (int base = blockIdx.x * tokens; base < p.num_tokens; base += stride, t += stride, ++k) {
        const bool real = t < p.num_tokens;
        load_index(t + 2 * stride, npos2, nslot2);
        load_angles(npos, nc, ns);

        const bool live = real && pos >= 0 && pos < p.num_positions;
        if (real && !live && report)
            atomicOr(p.err, PKV_DEVERR_POSITION);
        if (CACHED && live && slot >= p.capacity) {
            if (report)
                atomicOr(p.err, PKV_DEVERR_SLOT);
            slot = -1;
        }
        // element offsets of this token's outputs and of its row in a block's KV head 0
        const long long q_at = (long long)t * Hq * D, k_at = (long long)t * Hkv * D;
        long long cache_at = 0;
        if (CACHED && slot >= 0) {       // (block sizes are powers of two)
            const long long blk = slot >> p.block_shift;
            cache_at = blk * Hkv * head_rows + (slot & (p.block_size - 1)) * D;
        }
        const Pairs cp = pairs(c), sp = pairs(s), np = pairs(make_float4(-s.x, -s.y, -s.z, -s.w));

        const int st = k % S;
        const bool ok = !*abort_flag && mbar_wait_bounded(&full[st], (k / S) & 1);
        if (!__all_sync(kFullMask, ok)) {
            if ((threadIdx.x & 31) == 0) {
                *abort_flag = 1;
                if (p.err)
                    atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            }
            break;
        }
        const TIN* x0 = staged + st * (p.stage_bytes / (int)sizeof(TIN));
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            Raw4<TIN> a, b;
            a.clear();
            b.clear();
            if (real && kind[u] != kNone) {
                a.load(x0 + u * per_token * D);
                b.load(x0 + u * per_token * D + apart);
            }
            const float4 fa = a.get(), fb = b.get();
            const Pairs xa = pairs(fa), xb = pairs(fb);
            const Pairs sq = plus_times(xa, xa, times(xb, xb));
            const float4 sum4 = singles(sq);
            float ss = (sum4.x + sum4.y) + (sum4.z + sum4.w);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1)
                ss += __shfl_xor_sync(kFullMask, ss, o);
            if (!live || kind[u] == kNone)
                continue;
            if (CACHED && kind[u] == kV) {   // only appended
                if (slot >= 0) {
                    TC* at = static_cast<TC*>(dst[u]) + cache_at;
                    if constexpr (std::is_same<TIN, TC>::value) {   // the bits as they are
                        a.store(at);
                        b.store(at + apart);
                    } else {
                        cache4<TC, FMT>(at, fa, p.v_scale);
                        cache4<TC, FMT>(at + apart, fb, p.v_scale);
                    }
                }
                continue;
            }
            const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
            const float* w = weights + kind[u] * D + d0;
            const Pairs i4 = pairs(make_float4(inv, inv, inv, inv));
            const Pairs x = times(xa, times(i4, pairs(*reinterpret_cast<const float4*>(w))));
            const Pairs y = times(xb, times(i4, pairs(*reinterpret_cast<const float4*>(w + apart))));
            float4 u0, u1;
            if (!rotated) {
                u0 = singles(x);
                u1 = singles(y);
            } else if (split) {
                u0 = singles(plus_times(x, cp, times(y, np)));
                u1 = singles(plus_times(y, cp, times(x, sp)));
            } else {
                const float4 e = singles(x), f = singles(y);
                u0 = make_float4(e.x * c.x - e.y * s.x, e.y * c.x + e.x * s.x, e.z * c.y - e.w * s.y,
                                 e.w * c.y + e.z * s.y);
                u1 = make_float4(f.x * c.z - f.y * s.z, f.y * c.z + f.x * s.z, f.z * c.w - f.w * s.w,
                                 f.w * c.w + f.z * s.w);
            }
            if (!CACHED || kind[u] == kQ) {
                TIN* at = static_cast<TIN*>(dst[u]) + (kind[u] == kQ ? q_at : k_at);
                store4(at, u0);
                store4(at + apart, u1);
            } else if (slot >= 0) {
                TC* at = static_cast<TC*>(dst[u]) + cache_at;
                cache4<TC, FMT>(at, u0, p.k_scale);
                cache4<TC, FMT>(at + apart, u1, p.k_scale);
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(&empty[st]);
        c = nc;
        s = ns;
        pos = npos;
        slot = nslot;
        npos = npos2;
        nslot = nslot2;
    }
}

template <class TIN, class TC, int D, __nv_fp8_interpretation_t FMT, bool WHOLE, bool CACHED>
int launch_norm_rope_kernel(const NormRopeArgs& p, dim3 grid, cudaStream_t stream)
{
    auto kern = norm_rope_kernel<TIN, TC, D, FMT, WHOLE, CACHED>;
    const size_t smem = NormSmem<TIN, D>::bytes(p.stages, p.stage_bytes);
    if (!ensure_smem_attribute((const void*)kern, NormSmem<TIN, D>::bytes(1, NormSmem<TIN, D>::kBudget)))
        return PKV_ERR_LAUNCH;
    kern<<<grid, kNormThreads + 32, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <class TIN, class TC, int D, __nv_fp8_interpretation_t FMT = __NV_E4M3>
int launch_norm_rope(NormRopeArgs p, cudaStream_t stream)
{
    constexpr int kGroups = kNormThreads / (D / 8);
    const bool cached = p.slots != nullptr;
    const int rows = p.num_heads + p.num_kv_heads + (cached ? p.num_kv_heads : 0);
    // three CTAs an SM (fp32 rows: two), each taking every so many tokens
    constexpr int kResident = (sizeof(TIN) == 2 ? 3 : 2) * 148;
    // lane groups to a token: one a row while every CTA has one set of tokens, else as few as hold its
    // rows, so that a thread has up to four and a set more tokens (8192 tokens of 8 + 2 + 2 heads of 64:
    // 8.5 us against 16.4 us with a group a row; 600 of 16 + 8 + 8: 4.2 against 5.1 us)
    int per = 1;
    while (per < kGroups && per < rows)
        per *= 2;
    if ((long long)p.num_tokens * per > (long long)kResident * kGroups)
        for (per = 1; per < kGroups && kNormUnroll * per < rows;)
            per *= 2;
    p.groups_per_token = per;
    const int tokens_per_cta = kGroups / per;
    const int passes = (rows + kNormUnroll * per - 1) / (kNormUnroll * per);
    const int rows_per_pass = rows < kNormUnroll * per ? rows : kNormUnroll * per;
    p.stage_bytes = tokens_per_cta * rows_per_pass * D * (int)sizeof(TIN);   // at most 16 KB (fp32: 32 KB)
    p.stages = NormSmem<TIN, D>::stages(p.stage_bytes);
    int grid = (p.num_tokens + tokens_per_cta - 1) / tokens_per_cta;
    const int most = (kResident + passes - 1) / passes;
    if (grid > most)
        grid = most;
    const bool whole = p.rotary == D && !p.interleaved;
    const dim3 g(grid, passes);
    if (cached)
        return whole ? launch_norm_rope_kernel<TIN, TC, D, FMT, true, true>(p, g, stream)
                     : launch_norm_rope_kernel<TIN, TC, D, FMT, false, true>(p, g, stream);
    if constexpr (std::is_same<TIN, TC>::value)
        return whole ? launch_norm_rope_kernel<TIN, TC, D, FMT, true, false>(p, g, stream)
                     : launch_norm_rope_kernel<TIN, TC, D, FMT, false, false>(p, g, stream);
    return PKV_ERR_DTYPE;
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
    if (p.num_tokens < 0 || p.num_tokens > (1 << 30) || p.num_heads <= 0 || p.num_kv_heads <= 0 ||
        (long long)p.num_heads + 2ll * p.num_kv_heads > 65536 || (head_dim != 64 && head_dim != 128) ||
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
    p.block_shift = p.block_size == 8 ? 3 : p.block_size == 16 ? 4 : 5;
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
