// Sequences of a ragged batch: their rows (both ss_prefill kernels), and the
// order in which the chunked form runs them.
#pragma once
#include "ss_common.cuh"
#include "ss_many.h"

namespace ss {

// The row range of sequence b; false (with REPORT and the status bit) if it is not a range of the call's rows.
template <bool REPORT>
__device__ __forceinline__ bool seq_rows(const PrefillParams& p, int b, int& first, int& count) {
    const int s = p.seq_start[b], e = p.seq_start[b + 1];
    if (s < 0 || e < s || e > p.rows) {
        if (REPORT && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, SS_DEVICE_BAD_ROWS);
        return false;
    }
    first = s;
    count = e - s;
    return true;
}

// The place-th sequence to run, longest first, or -1 where no more have tokens
// (every thread of the block calls it; scratch: PREFILL_ORDER_MAX + 1 ints).  Blocks
// start in order, so the long sequences do not begin last, the blocks that have
// work are dealt out over the SMs, and those that have none end at once: one
// prompt of 512 tokens in a batch of 256 x 32 heads takes 70 us, not 225 (alone
// 53).  The token form does without: its blocks end at once by themselves, and
// the registers that this costs it made every call about a tenth slower.
template <int THREADS>
__device__ __forceinline__ int sequence_at(const PrefillParams& p, int place, int* scratch) {
    const int t = threadIdx.x;
    int with = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + t;
        const int n = b < p.B ? p.seq_start[b + 1] - p.seq_start[b] : 0;
        if (b < p.B) scratch[b] = n;
        with += __syncthreads_count(n > 0);
    }
    if (place >= with) return -1;
    for (int b = t; b < p.B; b += THREADS) {
        const int n = scratch[b];
        if (n <= 0) continue;
        int rank = 0;
        for (int j = 0; j < p.B; ++j) rank += scratch[j] > n || (scratch[j] == n && j < b);
        if (rank == place) scratch[PREFILL_ORDER_MAX] = b;
    }
    __syncthreads();
    const int b = scratch[PREFILL_ORDER_MAX];
    __syncthreads();                       // the scratch is free again
    return b;
}

}  // namespace ss
