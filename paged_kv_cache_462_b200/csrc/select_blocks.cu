// The blocks a decode step's queries may need most, for every sequence and KV head
// (select_blocks).
//
//   score(j) = max over the group's query heads of sum_d max(q_d kmax_d, q_d kmin_d)
//
// with kmax, kmin the block's key bounds: no key of block j has a larger product with the query (but for
// the rounding of an 8-bit cache's bounds to bf16, up to 2^-8 of sum_d |q_d k_d|).
// Kept are the first num_sink and the last num_recent blocks and the highest scores of the rest,
// ties to the lowest index, in ascending order.
//
// As q_d kmax_d wins where q_d > 0 and q_d kmin_d where q_d < 0, the sum is q+ . kmax + q- . kmin
// with q+ = max(q, 0), q- = min(q, 0): two dot products, for eight query columns at once on the
// warp's tensor cores (m16n8k16: 16 blocks x 8 columns). A lane takes the bounds in 16-byte pieces
// straight into A fragments: the order of d within a product is free, and q is loaded in the same
// one. Bound: HBM, 4 * head_dim bytes per block and KV head.
//
// fp32 sums cannot tell apart scores that lie closer than their rounding, and a wrong choice is a
// wrong block. So the MMAs sum 32 terms at a time, those sums are added in fp32, and with
// A = sum |q_d k_d| every score is within 2^-17 A of the exact one (the truncations of two chained
// MMAs stay under 35 * 2^-23 of their own |terms|, 2 head_dim / 32 <= 8 additions under 2^-24 A each).
// Blocks further than that from the border are decided by the fp32 score; those within it are
// scored again in fp64, where products of bf16 numbers and their sums are exact but for terms
// 2^-30 apart. Products and sums below fp32's normal range lose more than that: 3 head_dim of them by
// 2^-126 at most each, which every border allows for (2^-115 for two scores). A block with a bound that
// is not finite, or a score beyond fp32, ranks first.
//
// Two launches. The first streams the bounds: a block's bounds of neighbouring KV heads are one run of
// memory, so a producer warp brings 16 blocks (or a few times 16) of up to four heads at a time into
// a ring of shared-memory stages by bulk copies, and a warp per head and 16 blocks turns them into
// scores. Two CTAs an SM share all stages of the batch evenly, each a range of them. The second,
// queued behind it as a dependent launch, selects, a CTA per stream: up to 2048 blocks (or 16384, with
// four times the threads) are kept in registers, with as few exchanges as the steps allow: latency is
// all it costs.
//
// Measured (32 query and 8 KV heads of 128, blocks of 16): 64 sequences of 20001 to 32768 tokens, 128 of
// up to 2048 blocks (434 MB) 84.6 us, of which the scores take 74 (5.9 TB/s, 89 % of the copy rate) and
// the selection 11; 16 x 8192 tokens (34 MB) 14.5 us, 8 of them the latency of the two launches' chains
// of loads. One launch, its last CTA of a stream selecting, took 100 us: a CTA that selects streams
// nothing. A warp per stream selected 2048 blocks in 53 us, a CTA in shared memory in 20, in registers
// in 11; one sequence of 131072 tokens (8192 blocks) 50 us in shared memory, 21 us with 1024 threads.
#include <cstdint>

#include "device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kScoreWarps = 4;                // consumer warps, each a KV head's 16 blocks of a stage
constexpr int kScoreThreads = (kScoreWarps + 1) * 32;
constexpr int kScoreStages = 3;
constexpr int kRowPad = 64;                   // bytes behind a block's run: neighbouring rows meet other banks
// selection: threads of a CTA and keys a thread holds, for tables of up to 2048 blocks and for wider ones
constexpr int kSelThreads = 256, kSelPerThread = 8;
constexpr int kSelWideThreads = 1024, kSelWidePerThread = 16;
constexpr int kSelNear = 256;                 // blocks near the border that are ranked in shared memory
constexpr int kSelSmemKeys = 4096;            // what registers cannot settle is selected in shared memory up to this many
constexpr float kSelError = 7.62939453125e-06f;   // 2^-17
constexpr float kSelTiny = 2.407412430484045e-35f; // 2^-115
constexpr uint32_t kChosen = 0xffffffffu;

struct SelectArgs {
    int32_t* selected;            // [num_seqs][num_kv_heads][keep]
    const __nv_bfloat16* q;       // [num_seqs][num_heads][D]
    const __nv_bfloat16* bounds;  // [num_blocks][num_kv_heads][2][D]
    const int32_t* block_tables;
    const int32_t* seq_lens;
    int32_t* err;
    float* magnitude;             // [streams][runs]: the largest A of a run of 16 blocks
    float* scores;                // [streams][max_blocks]
    int32_t* near_list;           // [streams][max_blocks]: blocks near the border
    double* near_score;           // [streams][max_blocks]
    int num_seqs, num_heads, num_kv_heads, max_blocks, num_blocks, block_size;
    int keep, sink, recent;
    int heads, head_groups;       // KV heads a stage holds (the last group may have fewer)
    int tiles;                    // runs of 16 blocks in a stage
    int runs;                     // runs of 16 blocks of the widest sequence
};

// Tokens of sequence s as the table can hold them.
__device__ __forceinline__ int held_tokens(const SelectArgs& p, int s)
{
    const int L = __ldg(p.seq_lens + s), capacity = p.max_blocks * p.block_size;
    return L < 0 ? 0 : min(L, capacity);
}

__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// fp32 order as unsigned order, below kChosen for every finite number.
__device__ __forceinline__ uint32_t sort_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long sort_key(double f)
{
    const unsigned long long u = (unsigned long long)__double_as_longlong(f);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

template <int NW>
__device__ __forceinline__ int block_sum(int v, int* scratch)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(kFullMask, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i)
        s += scratch[i];
    return s;
}

// Both sums in one exchange.
template <int NW>
__device__ __forceinline__ void block_sum2(int& a, int& b, int2* scratch)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(kFullMask, a, o);
        b += __shfl_xor_sync(kFullMask, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = make_int2(a, b);
    __syncthreads();
    a = b = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        a += scratch[i].x;
        b += scratch[i].y;
    }
}

// Exclusive sum over the CTA's threads in order; `total` the sum of all.
template <int NW>
__device__ __forceinline__ int block_scan(int v, int* scratch, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = x;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < warp)
            base += scratch[i];
        total += scratch[i];
    }
    return base + x - v;
}

// Stages of one head group of sequence s: none where everything is kept.
__device__ __forceinline__ int stages_of(const SelectArgs& p, int s)
{
    const int nb = (held_tokens(p, s) + p.block_size - 1) / p.block_size;
    return nb <= p.keep ? 0 : (nb + 16 * p.tiles - 1) / (16 * p.tiles);
}

// A CTA's place in the batch's stages, in (sequence, head group, stage) order.
struct Walk {
    int s, hg, r, n;     // stage r of n of head group hg of sequence s
    __device__ __forceinline__ void next(const SelectArgs& p)
    {
        if (++r < n)
            return;
        r = 0;
        if (++hg < p.head_groups)
            return;
        hg = 0;
        for (n = 0; n == 0 && ++s < p.num_seqs;)
            n = stages_of(p, s);
    }
};

// Stages of the whole batch; `at` = where stage number `share` of `shares` equal parts begins, and
// `count` how many it has. A whole warp; sequences are summed in 32 runs, then within the run.
__device__ __forceinline__ void find_share(const SelectArgs& p, int share, int shares, int lane, Walk& at, int& count)
{
    int lo = 0, n = p.num_seqs;
    long long before = 0, target = -1;
    count = 0;
    while (n > 0) {
        const int per = (n + 31) / 32;
        int mine = 0;
        for (int i = lane * per; i < min(n, (lane + 1) * per); ++i)
            mine += stages_of(p, lo + i) * p.head_groups;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o)
                upto += y;
        }
        if (target < 0) {                // the first time: the whole batch
            const long long total = __shfl_sync(kFullMask, upto, 31);
            target = total * share / shares;
            count = (int)(total * (share + 1) / shares - target);
            if (count == 0)
                return;
        }
        const unsigned past = __ballot_sync(kFullMask, before + upto > target);   // some lane: target < total
        const int l = __ffs(past) - 1;
        before += __shfl_sync(kFullMask, upto - mine, l);
        lo += l * per;
        n = min(per, n - l * per);
        if (n == 1 && per == 1)
            break;
    }
    at.s = lo;
    at.n = stages_of(p, lo);
    const int in = (int)(target - before);
    at.hg = in / at.n;
    at.r = in - at.hg * at.n;
}

template <int D, int G>
__global__ void __launch_bounds__(kScoreThreads, 2) score_blocks_kernel(const SelectArgs p)
{
    constexpr int NC = D / 32;           // 16-byte pieces of one bound a lane takes
    constexpr int kTileBytes = 4 * D;    // one (block, KV head): maxima and minima
    extern __shared__ __align__(128) uint8_t smem[];
    const int row_bytes = p.heads * kTileBytes + kRowPad;      // a block's run in a stage
    const int stage_blocks = 16 * p.tiles;
    const int stage_bytes = stage_blocks * row_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kScoreStages * stage_bytes);
    uint64_t* empty = full + kScoreStages;
    int* held = reinterpret_cast<int*>(empty + kScoreStages);  // [stages][stage_blocks]: a good block id
    volatile int* abort_flag = held + kScoreStages * 16 * kScoreWarps;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * kScoreThreads + tid; i < p.num_seqs; i += gridDim.x * kScoreThreads) {
        const int L = __ldg(p.seq_lens + i);
        if (L < 0 || L > p.max_blocks * p.block_size)
            atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
    }
    if (tid == 0) {
        for (int i = 0; i < kScoreStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kScoreWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    Walk at{};
    int count;
    find_share(p, blockIdx.x, gridDim.x, lane, at, count);
    __syncthreads();

    if (warp == kScoreWarps) {           // the producer: lanes share a stage's blocks
        // (a stage has at most 64 blocks)
        auto entry = [&](const Walk& w, int i) -> int {
            const int j = w.r * stage_blocks + lane + 32 * i;
            const int nb = (held_tokens(p, w.s) + p.block_size - 1) / p.block_size;
            if (lane + 32 * i >= stage_blocks || j >= nb)
                return -2;               // no block
            return __ldg(p.block_tables + (long long)w.s * p.max_blocks + j);
        };
        int next[2] = {-2, -2};
        if (count > 0) {
            next[0] = entry(at, 0);
            next[1] = entry(at, 1);
        }
        bool aborted = false;
        int k = 0;
        for (; k < count; ++k) {
            const int st = k % kScoreStages;
            const int h0 = at.hg * p.heads, heads = min(p.heads, p.num_kv_heads - h0);
            const bool first_group = at.hg == 0;
            const int phys[2] = {next[0], next[1]};
            if (k + 1 < count) {         // the next stage's entries come while this one's copies are issued
                at.next(p);
                next[0] = entry(at, 0);
                next[1] = entry(at, 1);
            }
            bool ok[2];
            int copies = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ok[i] = phys[i] >= 0 && phys[i] < p.num_blocks;
                if (phys[i] != -2 && !ok[i] && first_group)
                    atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                copies += __popc(__ballot_sync(kFullMask, ok[i]));
            }
            if (lane == 0 && (*abort_flag || (k >= kScoreStages &&
                                              !mbar_wait_bounded(&empty[st], ((k / kScoreStages) - 1) & 1))))
                aborted = true;
            aborted = __shfl_sync(kFullMask, aborted ? 1 : 0, 0) != 0;
            if (aborted)
                break;
            __syncwarp();                // lane 0's wait, before other lanes write what consumers have read
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < stage_blocks)
                    held[st * stage_blocks + lane + 32 * i] = ok[i];
            __syncwarp();                // the entries, before the arrival that publishes them
            if (lane == 0) {
                if (copies)
                    mbar_arrive_expect_tx(&full[st], copies * heads * kTileBytes);
                else
                    mbar_arrive(&full[st]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ok[i])
                    bulk_copy_g2s(smem + st * stage_bytes + (lane + 32 * i) * row_bytes,
                                  p.bounds + ((long long)phys[i] * p.num_kv_heads + h0) * (2 * D),
                                  heads * kTileBytes, &full[st]);
        }
        if (aborted && lane == 0) {      // a wait gave up: the copies under way end before the CTA does
            *abort_flag = 1;
            atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            for (int i = max(0, k - kScoreStages); i < k; ++i)
                (void)mbar_wait_bounded(&full[i % kScoreStages], (i / kScoreStages) & 1);
        }
        return;
    }
    // ---- a consumer: of each stage KV head warp % heads, run warp / heads
    const int g = lane >> 2, t = lane & 3;
    uint32_t qp[NC][4], qn[NC][4];       // q+ and q- of column g in the order of the bounds' pieces
    long long stream = -1;               // the one qp and qn are of
    for (int k = 0; k < count; ++k, at.next(p)) {
        const int st = k % kScoreStages;
        const int h0 = at.hg * p.heads, heads = min(p.heads, p.num_kv_heads - h0);
        const int tile = warp / heads, hw = warp - tile * heads, h = h0 + hw;
        const int nb = (held_tokens(p, at.s) + p.block_size - 1) / p.block_size;
        const int first = at.r * stage_blocks + tile * 16;
        const bool active = tile < p.tiles && first < nb;
        if (active && stream != (long long)at.s * p.num_kv_heads + h) {
            stream = (long long)at.s * p.num_kv_heads + h;
            const __nv_bfloat16* q = p.q + ((long long)at.s * p.num_heads + (long long)h * G) * D;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (g < G)
                    u = __ldg(reinterpret_cast<const uint4*>(q + (long long)g * D) + 4 * c + t);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
                    const __nv_bfloat162 a = __hmax2_nan(x, zero), b = __hmin2_nan(x, zero);
                    qp[c][i] = *reinterpret_cast<const uint32_t*>(&a);
                    qn[c][i] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
        }
        const bool arrived = !*abort_flag && mbar_wait_bounded(&full[st], (k / kScoreStages) & 1);
        if (!__all_sync(kFullMask, arrived)) {
            if (lane == 0) {
                *abort_flag = 1;
                atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            }
            break;
        }
        if (!active) {
            if (lane == 0)
                mbar_arrive(&empty[st]);
            continue;
        }
        const int slot = st * stage_blocks + tile * 16 + g;
        const bool ok[2] = {held[slot] != 0, held[slot + 8] != 0};   // rows g and g + 8
        // sc: the scores; ab and an: the sums of |q+ kmax| and of -|q- kmin|. Rows without a block hold
        // what was there before: nothing of theirs is used.
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, ab[4] = {0.f, 0.f, 0.f, 0.f}, an[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* at = smem + st * stage_bytes + (tile * 16 + g) * row_bytes + hw * kTileBytes + t * 16;
        auto product = [&](const uint8_t* from, const uint32_t (&b)[4], float (&size)[4]) {
            constexpr uint32_t M = 0x7fff7fffu;
            const uint4 x = *reinterpret_cast<const uint4*>(from);
            const uint4 y = *reinterpret_cast<const uint4*>(from + 8 * row_bytes);
            float c[4];
            mma_bf16_zero(c, x.x, y.x, x.y, y.y, b[0], b[1]);
            mma_bf16(c, x.z, y.z, x.w, y.w, b[2], b[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sc[i] += c[i];
            mma_bf16(size, x.x & M, y.x & M, x.y & M, y.y & M, b[0], b[1]);
            mma_bf16(size, x.z & M, y.z & M, x.w & M, y.w & M, b[2], b[3]);
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            product(at + 64 * c, qp[c], ab);
            product(at + 64 * c + 2 * D, qn[c], an);
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[st]);
        // rows first + g (sc 0, 1) and first + g + 8 (sc 2, 3), columns 2t and 2t + 1
        float mag = 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float best = -INFINITY, a = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (2 * t + i < G) {
                    const float x = sc[2 * r + i];
                    best = fmaxf(best, finite(x) ? x : INFINITY);
                    a = fmaxf(a, ab[2 * r + i] - an[2 * r + i]);
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                best = fmaxf(best, __shfl_xor_sync(kFullMask, best, o));
                a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
            }
            if (!ok[r])
                best = -INFINITY;        // a bad block id: chosen last
            else if (finite(best))
                mag = fmaxf(mag, a);
            const int j = first + g + 8 * r;
            if (t == 0 && j < nb)
                p.scores[stream * p.max_blocks + j] = best;
        }
        mag = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(mag)));   // (not negative)
        if (lane == 0)
            p.magnitude[stream * p.runs + first / 16] = mag;
    }
}

// The exact score of a block: fp64 sums, the largest over the group's query heads (a whole warp).
template <int D, int G>
__device__ __forceinline__ double exact_score(const __nv_bfloat16* q, const __nv_bfloat16* bounds, int lane)
{
    constexpr int E = D / 32;            // 4 or 2 elements of a row
    __nv_bfloat16 hi[E], lo[E], x[G][E];
    auto load = [&](__nv_bfloat16(&to)[E], const __nv_bfloat16* from) {
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(to) = __ldg(reinterpret_cast<const uint2*>(from) + lane);
        else
            *reinterpret_cast<uint32_t*>(to) = __ldg(reinterpret_cast<const uint32_t*>(from) + lane);
    };
    load(hi, bounds);
    load(lo, bounds + D);
#pragma unroll
    for (int g = 0; g < G; ++g)
        load(x[g], q + g * D);
    double best = 0.0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        double s = 0.0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float f = __bfloat162float(x[g][e]);
            s = fma((double)f, (double)__bfloat162float(f > 0.f ? hi[e] : lo[e]), s);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            s += __shfl_xor_sync(kFullMask, s, o);
        best = g == 0 ? s : fmax(best, s);
    }
    return best;
}

// The keys from `up` on are certainly above a border `key`, those below `down` certainly not: two
// errors (the border's own and the block's), the rounding of this very sum and what is lost below fp32's
// normal range.
__device__ __forceinline__ void border_zone(uint32_t key, float mag, uint32_t& down, uint32_t& up)
{
    const float f = __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
    up = down = key;
    if (finite(f)) {
        const float d = 2.f * kSelError * mag + fabsf(f) * 2.4e-7f + kSelTiny;
        up = max(key, sort_key(f + d));
        down = min(key, sort_key(f - d));
    }
}

// A near block's score in 64 bits (a whole warp); one that is not finite in fp32 keeps its place above
// or below all.
template <int D, int G>
__device__ __forceinline__ double near_score_of(const SelectArgs& p, const __nv_bfloat16* q, const int32_t* table, int h,
                                                int j, uint32_t key, int lane)
{
    if (key >= sort_key(INFINITY))
        return INFINITY;
    if (key <= sort_key(-INFINITY))
        return -INFINITY;
    const long long tile = (long long)__ldg(table + j) * p.num_kv_heads + h;
    return exact_score<D, G>(q, p.bounds + tile * (2 * D), lane);
}

template <int NT, int K>
struct FastShared {
    int hist[4][256];
    int taken[4];                        // keys gathered after each pass; [3]: near blocks
    uint32_t list[32];
    uint32_t reduce[3][NT / 32];
    int above[NT / 32];
    int near_block[kSelNear];
    uint32_t near_key[kSelNear];
    unsigned long long near_val[kSelNear];
    uint32_t chosen[NT * K / 32];
    int counts[NT / 32 * K];
};

// Selection among up to NT * K blocks by the CTA; thread t holds the keys of blocks t, t + NT, ...
// Returns false, having written nothing, if more than kSelNear blocks are too close to the border.
template <int D, int G, int NT, int K>
__device__ __forceinline__ bool select_in_registers(const SelectArgs& p, const __nv_bfloat16* q, const int32_t* table,
                                                    const float* scores, const float* magnitude, int nb, int h,
                                                    int32_t* out, FastShared<NT, K>& sh)
{
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int need = p.keep - p.sink - p.recent;
    uint32_t keys[K];
    float score[K];
    float mag = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int j = i * NT + tid;
        score[i] = j < nb ? __ldcg(scores + j) : 0.f;
    }
    for (int i = tid; i < (nb + 15) / 16; i += NT)
        mag = fmaxf(mag, __ldcg(magnitude + i));
    for (int i = tid; i < 4 * 256; i += NT)
        sh.hist[i / 256][i % 256] = 0;
    if (tid < 4)
        sh.taken[tid] = 0;
    for (int i = tid; i < NT * K / 32; i += NT)
        sh.chosen[i] = 0u;
    uint32_t kmin = 0xffffffffu, kmax = 0u;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int j = i * NT + tid;
        keys[i] = j < nb ? sort_key(score[i]) : 0u;      // behind the last block: below every key
        if (j < p.sink || (j < nb && j >= nb - p.recent)) {
            keys[i] = kChosen;
        } else if (j < nb) {
            kmin = min(kmin, keys[i]);
            kmax = max(kmax, keys[i]);
        }
    }
    kmin = __reduce_min_sync(kFullMask, kmin);
    kmax = __reduce_max_sync(kFullMask, kmax);
    const uint32_t m0 = __reduce_max_sync(kFullMask, __float_as_uint(mag));   // (not negative)
    if (lane == 0) {
        sh.reduce[0][warp] = kmin;
        sh.reduce[1][warp] = kmax;
        sh.reduce[2][warp] = m0;
    }
    __syncthreads();
    uint32_t mbits = 0u;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        kmin = min(kmin, sh.reduce[0][i]);
        kmax = max(kmax, sh.reduce[1][i]);
        mbits = max(mbits, sh.reduce[2][i]);
    }
    mag = __uint_as_float(mbits);

    uint32_t take = kChosen;             // keys from here on are chosen
    if (need > 0) {
        // The border, the need-th largest key: 256 equal bins over the range left, then over the bin
        // it lies in, until that holds few. Every warp reads the counts for itself.
        uint32_t lo = kmin, hi = kmax;
        int rank = need;                 // the rank-th largest of the keys in [lo, hi]
        int left = nb;
#pragma unroll 1
        for (int pass = 0; pass < 4 && lo < hi && left > 32; ++pass) {
            const uint32_t span = hi - lo;
            const int shift = span < 256u ? 0 : 24 - __clz(span);
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (keys[i] >= lo && keys[i] <= hi)
                    atomicAdd(&sh.hist[pass][(keys[i] - lo) >> shift], 1);
            __syncthreads();
            // lane l adds up bins 255 - 8 l .. 248 - 8 l, the largest keys first
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = sh.hist[pass][255 - 8 * lane - i];
                sum += c[i];
            }
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFullMask, upto, o);
                if (lane >= o)
                    upto += y;
            }
            const int l = __ffs(__ballot_sync(kFullMask, upto >= rank)) - 1;
            int before = upto - sum, bin = 0, in = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (in == 0 && before + c[i] >= rank) {
                    bin = 255 - 8 * lane - i;
                    in = c[i];
                } else if (in == 0) {
                    before += c[i];
                }
            }
            bin = __shfl_sync(kFullMask, bin, l);
            left = __shfl_sync(kFullMask, in, l);
            rank -= __shfl_sync(kFullMask, before, l);
            const uint32_t base = lo + ((uint32_t)bin << shift);
            const uint32_t last = base + ((1u << shift) - 1u);
            hi = last < base || last > hi ? hi : last;
            lo = base;
        }
        if (lo < hi) {                   // at most 32 keys are left: ranked against one another
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (keys[i] >= lo && keys[i] <= hi) {
                    const int at = atomicAdd(&sh.taken[0], 1);
                    if (at < 32)
                        sh.list[at] = keys[i];
                }
            __syncthreads();
            const int n = min(sh.taken[0], 32);
            const uint32_t mine = lane < n ? sh.list[lane] : 0u;
            int greater = 0, equal = 0;
            for (int i = 0; i < n; ++i) {
                const uint32_t k = __shfl_sync(kFullMask, mine, i);
                greater += k > mine;
                equal += k == mine;
            }
            const unsigned hit = __ballot_sync(kFullMask, lane < n && greater < rank && rank <= greater + equal);
            lo = __shfl_sync(kFullMask, mine, __ffs(hit) - 1);
        }
        uint32_t down, up;
        border_zone(lo, mag, down, up);
        int above = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            above += keys[i] > up && keys[i] != kChosen;
            if (keys[i] >= down && keys[i] <= up) {
                const int at = atomicAdd(&sh.taken[3], 1);
                if (at < kSelNear) {
                    sh.near_block[at] = i * NT + tid;
                    sh.near_key[at] = keys[i];
                }
            }
        }
        above = __reduce_add_sync(kFullMask, above);
        if (lane == 0)
            sh.above[warp] = above;
        __syncthreads();
        const int near = sh.taken[3];
        int want = need;                 // of the near ones; 1 <= want <= near
#pragma unroll
        for (int i = 0; i < NW; ++i)
            want -= sh.above[i];
        take = down;
        if (want < near) {
            if (near > kSelNear)
                return false;
            take = up + 1u;
            for (int i = warp; i < near; i += NW) {
                const double v = near_score_of<D, G>(p, q, table, h, sh.near_block[i], sh.near_key[i], lane);
                if (lane == 0)
                    sh.near_val[i] = sort_key(v);
            }
            __syncthreads();
            if (tid < near) {            // each is ranked against the others, ties by index
                const unsigned long long mine = sh.near_val[tid];
                const int block = sh.near_block[tid];
                int better = 0;
                for (int i = 0; i < near; ++i) {
                    const unsigned long long k = sh.near_val[i];
                    better += k > mine || (k == mine && sh.near_block[i] < block);
                }
                if (better < want)
                    atomicOr(&sh.chosen[block / 32], 1u << (block % 32));
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (sh.chosen[i * NW + warp] >> lane & 1u)
                    keys[i] = kChosen;
        }
    }
    // ascending order: by i, then by thread
    unsigned m[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        m[i] = __ballot_sync(kFullMask, keys[i] >= take);
        if (lane == 0)
            sh.counts[i * NW + warp] = __popc(m[i]);
    }
    __syncthreads();
    if (warp == 0) {                     // what comes before each of them, K * NW / 32 a lane
        constexpr int E = K * NW / 32;
        int c[E], sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            c[e] = sh.counts[lane * E + e];
            sum += c[e];
        }
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullMask, before, o);
            if (lane >= o)
                before += y;
        }
        before -= sum;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sh.counts[lane * E + e] = before;
            before += c[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int at = sh.counts[i * NW + warp] + __popc(m[i] & ((1u << lane) - 1u));
        if ((m[i] >> lane & 1u) && at < p.keep)
            out[at] = i * NT + tid;
    }
    return true;
}

template <int D, int G, int NT, int K>
__global__ void __launch_bounds__(NT) select_blocks_kernel(const SelectArgs p)
{
    constexpr int NW = NT / 32;
    extern __shared__ uint32_t smem_keys[];
    __shared__ int scratch[NW];
    __shared__ int2 scratch2[NW];
    __shared__ double near_vals[kSelNear];
    __shared__ float fscratch[NW];
    __shared__ int hist[256];
    __shared__ int bcast[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int stream = blockIdx.x, s = stream / p.num_kv_heads, h = stream - s * p.num_kv_heads;
    int32_t* out = p.selected + (long long)stream * p.keep;
    const int nb = (held_tokens(p, s) + p.block_size - 1) / p.block_size;
    // (the scoring grid may still run; the next call's waits for this one's end)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nb <= p.keep) {                  // everything is kept
        for (int i = tid; i < p.keep; i += NT)
            out[i] = i < nb ? i : -1;
        return;
    }
    const __nv_bfloat16* q = p.q + ((long long)s * p.num_heads + (long long)h * G) * D;
    const int32_t* table = p.block_tables + (long long)s * p.max_blocks;
    float* scores = p.scores + (long long)stream * p.max_blocks;
    const float* magnitude = p.magnitude + (long long)stream * p.runs;
    __shared__ FastShared<NT, K> fast;
    if (nb <= NT * K && select_in_registers<D, G, NT, K>(p, q, table, scores, magnitude, nb, h, out, fast))
        return;
    const bool in_smem = nb <= kSelSmemKeys;
    uint32_t* keys = in_smem ? smem_keys : reinterpret_cast<uint32_t*>(scores);
    const int need = p.keep - p.sink - p.recent;   // among blocks [sink, nb - recent), more than `need` of them
    float mag = 0.f;
    for (int i = tid; i < (nb + 15) / 16; i += NT)
        mag = fmaxf(mag, __ldcg(magnitude + i));
    uint32_t kmin = 0xffffffffu, kmax = 0u;
    for (int j = tid; j < nb; j += NT) {
        uint32_t k = sort_key(__ldcg(scores + j));
        if (j < p.sink || j >= nb - p.recent) {
            k = kChosen;
        } else {
            kmin = min(kmin, k);
            kmax = max(kmax, k);
        }
        keys[j] = k;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        mag = fmaxf(mag, __shfl_xor_sync(kFullMask, mag, o));
        kmin = min(kmin, __shfl_xor_sync(kFullMask, kmin, o));
        kmax = max(kmax, __shfl_xor_sync(kFullMask, kmax, o));
    }
    __shared__ uint32_t range[2][NW];
    if (lane == 0) {
        range[0][warp] = kmin;
        range[1][warp] = kmax;
        fscratch[warp] = mag;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        kmin = min(kmin, range[0][i]);
        kmax = max(kmax, range[1][i]);
        mag = fmaxf(mag, fscratch[i]);
    }

    if (need > 0) {
        // the key of the need-th largest: 256 equal bins between the smallest and the largest key
        // left, then the same within the bin it lies in, until that holds at most 256
        uint32_t lo = kmin, hi = kmax;
        int rank = need;                 // the rank-th largest of the keys in [lo, hi]
        int in_bin = nb;
        for (int pass = 0; pass < 5 && lo < hi && in_bin > 256; ++pass) {
            const uint32_t span = hi - lo;
            const int shift = span < 256u ? 0 : 24 - __clz(span);
            if (tid < 256)
                hist[tid] = 0;
            __syncthreads();
            for (int j = tid; j < nb; j += NT) {
                const uint32_t k = keys[j];
                if (k >= lo && k <= hi)
                    atomicAdd(&hist[(k - lo) >> shift], 1);
            }
            __syncthreads();
            int total;
            // thread i holds bin 255 - i: how many keys lie in higher bins
            const int mine = tid < 256 ? hist[255 - tid] : 0;
            const int above = block_scan<NW>(mine, scratch, total);
            if (mine > 0 && above < rank && rank <= above + mine) {
                bcast[0] = 255 - tid;
                bcast[1] = rank - above;
                bcast[2] = mine;
            }
            __syncthreads();
            const uint32_t bin = (uint32_t)bcast[0];
            rank = bcast[1];
            in_bin = bcast[2];
            const uint32_t base = lo + (bin << shift);
            const uint32_t last = base + ((1u << shift) - 1u);
            hi = last < base || last > hi ? hi : last;
            lo = base;
            __syncthreads();
        }
        if (lo < hi) {                   // rank the keys that are left against one another
            if (tid == 0)
                bcast[0] = 0;
            __syncthreads();
            for (int j = tid; j < nb; j += NT) {
                const uint32_t k = keys[j];
                if (k >= lo && k <= hi) {
                    const int at = atomicAdd(&bcast[0], 1);
                    if (at < 256)
                        hist[at] = (int)k;
                }
            }
            __syncthreads();
            const int n = min(bcast[0], 256);
            if (tid < n) {
                const uint32_t k = (uint32_t)hist[tid];
                int greater = 0, equal = 0;
                for (int i = 0; i < n; ++i) {
                    greater += (uint32_t)hist[i] > k;
                    equal += (uint32_t)hist[i] == k;
                }
                if (greater < rank && rank <= greater + equal)
                    bcast[1] = (int)k;   // the same key from every thread that holds it
            }
            __syncthreads();
            lo = (uint32_t)bcast[1];
        }
        // blocks whose order against that one the fp32 scores do not settle
        uint32_t down, up;
        border_zone(lo, mag, down, up);
        int above = 0, near = 0;
        for (int j = tid; j < nb; j += NT) {
            const uint32_t k = keys[j];
            above += k > up && k != kChosen;
            near += k >= down && k <= up;
        }
        block_sum2<NW>(above, near, scratch2);
        int want = need - above;         // of the `near` ones; 1 <= want <= near
        const bool all = want == near;
        uint32_t take = all ? down : up + 1u;        // keys from here on are chosen
        if (!all) {
            int32_t* list = p.near_list + (long long)stream * p.max_blocks;
            double* val = p.near_score + (long long)stream * p.max_blocks;
            // the near blocks in ascending order
            const int seg = (nb + NT - 1) / NT;
            const int b = min(nb, tid * seg), e = min(nb, b + seg);
            int cnt = 0, total;
            for (int j = b; j < e; ++j)
                cnt += keys[j] >= down && keys[j] <= up;
            int at = block_scan<NW>(cnt, scratch, total);
            for (int j = b; j < e; ++j)
                if (keys[j] >= down && keys[j] <= up)
                    list[at++] = j;
            __syncthreads();
            for (int i = warp; i < near; i += NW) {
                const double v = near_score_of<D, G>(p, q, table, h, list[i], keys[list[i]], lane);
                if (lane == 0)
                    (near <= kSelNear ? near_vals : val)[i] = v;
            }
            __syncthreads();
            if (near <= kSelNear) {   // a few: each is ranked against the others, ties by index
                if (tid < near) {
                    const unsigned long long mine = sort_key(near_vals[tid]);
                    int better = 0;
                    for (int i = 0; i < near; ++i) {
                        const unsigned long long k = sort_key(near_vals[i]);
                        better += k > mine || (k == mine && i < tid);
                    }
                    keys[list[tid]] = better < want ? kChosen : 0u;
                }
                __syncthreads();
            } else {
                // the want-th largest exact score, bit by bit
                unsigned long long bound = 0ull;
                for (int bit = 63; bit >= 0; --bit) {
                    const unsigned long long trial = bound | (1ull << bit);
                    int c = 0;
                    for (int i = tid; i < near; i += NT)
                        c += sort_key(val[i]) >= trial;
                    if (block_sum<NW>(c, scratch) >= want)
                        bound = trial;
                }
                int more = 0;
                for (int i = tid; i < near; i += NT)
                    more += sort_key(val[i]) > bound;
                more = block_sum<NW>(more, scratch);
                want -= more;                // of the ties, in order
                const int seg2 = (near + NT - 1) / NT;
                const int b2 = min(near, tid * seg2), e2 = min(near, b2 + seg2);
                int ties = 0;
                for (int i = b2; i < e2; ++i)
                    ties += sort_key(val[i]) == bound;
                int rank2 = block_scan<NW>(ties, scratch, total);
                for (int i = b2; i < e2; ++i) {
                    const unsigned long long k = sort_key(val[i]);
                    const bool chosen = k > bound || (k == bound && rank2 < want);
                    rank2 += k == bound;
                    keys[list[i]] = chosen ? kChosen : 0u;
                }
                __syncthreads();
            }
        }
        // emit in ascending order: chosen keys and those from `take` on
        const int seg = (nb + NT - 1) / NT;
        const int b = min(nb, tid * seg), e = min(nb, b + seg);
        int cnt = 0, total;
        for (int j = b; j < e; ++j)
            cnt += keys[j] >= take;
        int at = block_scan<NW>(cnt, scratch, total);
        for (int j = b; j < e; ++j)
            if (keys[j] >= take && at < p.keep)
                out[at++] = j;
    } else {
        for (int i = tid; i < p.keep; i += NT)
            out[i] = i < p.sink ? i : nb - p.keep + i;
    }
}

struct SelectLayout {
    size_t magnitude, scores, near_list, near_score, bytes;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

SelectLayout select_layout(long long streams, long long max_blocks)
{
    SelectLayout l;
    const size_t parts = (size_t)((max_blocks + 15) / 16);   // runs of 16 blocks
    l.magnitude = kWorkspaceHeader;
    l.scores = l.magnitude + up256((size_t)streams * parts * 4);
    l.near_list = l.scores + up256((size_t)streams * max_blocks * 4);
    l.near_score = l.near_list + up256((size_t)streams * max_blocks * 4);
    l.bytes = l.near_score + up256((size_t)streams * max_blocks * 8);
    return l;
}

bool select_sizes_ok(int num_seqs, int num_kv_heads, int max_blocks)
{
    return num_seqs >= 0 && num_seqs <= kMaxSeqs && num_kv_heads > 0 && max_blocks > 0 &&
           (long long)num_seqs * num_kv_heads * max_blocks < (1ll << 31);
}

template <int D, int G>
int launch_select(SelectArgs p, int num_seqs, cudaStream_t stream)
{
    auto score = score_blocks_kernel<D, G>;
    p.heads = p.num_kv_heads < kScoreWarps ? p.num_kv_heads : kScoreWarps;
    p.head_groups = (p.num_kv_heads + p.heads - 1) / p.heads;
    p.tiles = kScoreWarps / p.heads;
    const int stage_blocks = 16 * p.tiles;
    const int stages = (p.max_blocks + stage_blocks - 1) / stage_blocks;
    p.runs = (p.max_blocks + 15) / 16;
    const long long all = (long long)num_seqs * p.head_groups * stages;
    const unsigned grid = (unsigned)(all < 2 * 148 ? all : 2 * 148);
    const size_t smem = (size_t)kScoreStages * stage_blocks * (p.heads * 4 * D + kRowPad) + kScoreStages * 16 +
                        kScoreStages * 16 * kScoreWarps * 4 + 16;
    if (!ensure_smem_attribute((const void*)score, smem))
        return PKV_ERR_LAUNCH;
    score<<<grid, kScoreThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return PKV_ERR_LAUNCH;
    const bool wide = p.max_blocks > kSelThreads * kSelPerThread;
    auto select = wide ? select_blocks_kernel<D, G, kSelWideThreads, kSelWidePerThread>
                       : select_blocks_kernel<D, G, kSelThreads, kSelPerThread>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_seqs * p.num_kv_heads));
    cfg.blockDim = dim3(wide ? kSelWideThreads : kSelThreads);
    cfg.dynamicSmemBytes = (size_t)(p.max_blocks < kSelSmemKeys ? p.max_blocks : kSelSmemKeys) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select, p) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <int D>
int select_by_group(int group, const SelectArgs& p, int num_seqs, cudaStream_t stream)
{
    switch (group) {
    case 1: return launch_select<D, 1>(p, num_seqs, stream);
    case 2: return launch_select<D, 2>(p, num_seqs, stream);
    case 4: return launch_select<D, 4>(p, num_seqs, stream);
    case 5: return launch_select<D, 5>(p, num_seqs, stream);
    case 8: return launch_select<D, 8>(p, num_seqs, stream);
    default: return PKV_ERR_SHAPE;
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API size_t pkv_select_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq)
{
    if (!select_sizes_ok(num_seqs, num_kv_heads, max_blocks_per_seq))
        return 0;
    return select_layout((long long)num_seqs * num_kv_heads, max_blocks_per_seq).bytes;
}

PKV_API int select_blocks(int32_t* selected, const void* q, const void* key_bounds, const int32_t* block_tables,
                          const int32_t* seq_lens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                          int block_size, int max_blocks_per_seq, int num_blocks, int num_selected,
                          int num_sink_blocks, int num_recent_blocks, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    if (!select_sizes_ok(num_seqs, num_kv_heads, max_blocks_per_seq) || num_heads <= 0 ||
        num_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128) ||
        (block_size != 8 && block_size != 16 && block_size != 32) || num_blocks <= 0 ||
        (long long)num_blocks * num_kv_heads >= (1ll << 31) || (long long)max_blocks_per_seq * block_size >= (1ll << 31) || num_selected < 1 || num_sink_blocks < 0 ||
        num_recent_blocks < 0 || (long long)num_sink_blocks + num_recent_blocks > num_selected ||
        (long long)num_seqs * num_kv_heads * num_selected >= (1ll << 31))
        return PKV_ERR_SHAPE;
    const int group = num_heads / num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 5 && group != 8)
        return PKV_ERR_SHAPE;
    if (num_seqs == 0)
        return PKV_OK;
    if (!selected || !q || !key_bounds || !block_tables || !seq_lens)
        return PKV_ERR_NULL;
    const long long streams = (long long)num_seqs * num_kv_heads;
    const SelectLayout l = select_layout(streams, max_blocks_per_seq);
    if (!workspace || workspace_bytes < l.bytes)
        return PKV_ERR_WORKSPACE;
    auto off16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    if (off16(q) || off16(key_bounds) || off16(workspace))
        return PKV_ERR_SHAPE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    SelectArgs p{};
    p.selected = selected;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.bounds = static_cast<const __nv_bfloat16*>(key_bounds);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.err = reinterpret_cast<int32_t*>(ws);
    p.magnitude = reinterpret_cast<float*>(ws + l.magnitude);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.near_list = reinterpret_cast<int32_t*>(ws + l.near_list);
    p.near_score = reinterpret_cast<double*>(ws + l.near_score);
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.keep = num_selected;
    p.sink = num_sink_blocks;
    p.recent = num_recent_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? select_by_group<128>(group, p, num_seqs, st) : select_by_group<64>(group, p, num_seqs, st);
}

}  // extern "C"
