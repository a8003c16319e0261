// The blocks a call appends to, by sequence: sequence s has the rows row_offsets[s] ..
// row_offsets[s + 1] - 1 of a call, its newest tokens, at positions seq_lens[s] - n ..
// seq_lens[s] - 1 (n of them). A work item is one (sequence, logical block) that holds one of them
// at least.
//
// Items are numbered without a scan: sequence s owns the numbers from row_offsets[s] / block_size +
// 2 s up to the next sequence's, which are at least n / block_size + 2, and n consecutive positions
// lie in at most (n - 2) / block_size + 2 blocks. So the host launches num_tokens / block_size +
// 2 num_seqs items, knowing no length, and the numbers without a block do nothing. (Offsets out of order
// can hide other sequences' numbers from the search below: their blocks are left out, and the
// call has flagged the offsets.)
#pragma once

#include "device.cuh"
#include "pkv_internal.h"

namespace pkv {

struct Touched {
    int seq, block;     // logical block
    int len;            // tokens of the sequence
    int first;          // position of its first new token
    int row;            // the row of that token
    int phys;           // -1: nothing to do
};

__host__ __device__ __forceinline__ long long touched_items(int num_tokens, int num_seqs, int block_size)
{
    return num_tokens / block_size + 2ll * num_seqs;
}

// The PKV_DEVERR_* bits of sequence s's entries: 0 when they can be used.
__device__ __forceinline__ int touched_check(const int32_t* row_offsets, const int32_t* seq_lens, int s,
                                             int num_tokens, int capacity)
{
    const int a = __ldg(row_offsets + s), b = __ldg(row_offsets + s + 1), L = __ldg(seq_lens + s);
    if (a < 0 || b < a || b > num_tokens)
        return PKV_DEVERR_ROWS;
    return L < 0 || L > capacity || b - a > L ? PKV_DEVERR_SEQ_LEN : 0;
}

// Work item `item` (the same for all lanes of the warp). Sequences with bad entries have no items.
__device__ __forceinline__ Touched touched_find(const int32_t* row_offsets, const int32_t* seq_lens,
                                                const int32_t* block_tables, int num_seqs, int num_tokens,
                                                int block_size, int max_blocks, int num_blocks, long long item,
                                                int lane, int32_t* err)
{
    auto start = [&](int s) -> long long { return max(0, __ldg(row_offsets + s)) / block_size + 2ll * s; };
    // the last sequence whose first number is at most `item`, 32 probes at a time
    int lo = 0, n = num_seqs;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int probe = lo + lane * step;
        const bool le = lane * step < n && start(probe) <= item;
        const int at = __popc(__ballot_sync(kFullMask, le));   // in order: a prefix of the probes
        const int skip = at > 0 ? (at - 1) * step : 0;
        lo += skip;
        n = min(step, n - skip);
    }
    Touched t;
    t.seq = lo;
    t.phys = -1;
    t.block = t.len = t.first = t.row = 0;
    if (touched_check(row_offsets, seq_lens, lo, num_tokens, max_blocks * block_size) != 0)
        return t;
    t.row = __ldg(row_offsets + lo);
    const int fresh = __ldg(row_offsets + lo + 1) - t.row;
    t.len = __ldg(seq_lens + lo);
    t.first = t.len - fresh;
    const long long local = item - start(lo);
    const long long block = t.first / block_size + local;
    if (fresh == 0 || local < 0 || block > (t.len - 1) / block_size)
        return t;
    t.block = (int)block;
    const int phys = __ldg(block_tables + (long long)lo * max_blocks + block);
    if (phys < 0 || phys >= num_blocks) {
        if (lane == 0 && err)
            atomicOr(err, PKV_DEVERR_BLOCK_ID);
        return t;
    }
    t.phys = phys;
    return t;
}

// Flags every sequence's bad entries once: thread `i` of the launch looks at sequence i.
__device__ __forceinline__ void touched_flag(const int32_t* row_offsets, const int32_t* seq_lens, int num_seqs,
                                             int num_tokens, int capacity, long long i, int32_t* err)
{
    if (err && i < num_seqs) {
        const int bad = touched_check(row_offsets, seq_lens, (int)i, num_tokens, capacity);
        if (bad)
            atomicOr(err, bad);
    }
}

// Host checks shared by the calls that take row_offsets.
inline int touched_host_check(int num_tokens, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int num_blocks)
{
    if (num_tokens < 0 || num_seqs < 0 || num_seqs > kMaxSeqs || num_kv_heads <= 0 ||
        (head_dim != 64 && head_dim != 128) || (block_size != 8 && block_size != 16 && block_size != 32))
        return PKV_ERR_SHAPE;
    if (num_seqs == 0 || num_tokens == 0)
        return PKV_OK;
    if (max_blocks_per_seq <= 0 || num_blocks <= 0 || (long long)max_blocks_per_seq * block_size >= (1ll << 31) ||
        2 * touched_items(num_tokens, num_seqs, block_size) * num_kv_heads >= (1ll << 31))
        return PKV_ERR_SHAPE;
    return PKV_OK;
}

}  // namespace pkv
