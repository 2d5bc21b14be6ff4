// paged.cuh -- what the kernels of the paged key/value cache share.
#pragma once

#include "common.cuh"

namespace pivot {

// A cache as the kernels see it (pivot_cache_t, checked).
struct CacheView {
    uint8_t *k, *v;
    float *ks, *vs;            // NULL for bf16
    int32_t *table, *len, *refs;
    int B, Hkv, D;
    int page_log2, num_pages, max_pages;
    int rowb;                  // bytes of one token's row of K: Hkv * D * value size

    __host__ __device__ __forceinline__ int page_size() const { return 1 << page_log2; }
    // Token row of position t of sequence b, or -1 (a page id out of range).
    __device__ __forceinline__ int row_of(int page, int t) const {
        if ((unsigned)page >= (unsigned)num_pages) return -1;
        return (page << page_log2) + (t & ((1 << page_log2) - 1));
    }
};

// Rows [first, first + n) of the packed new tokens belong to sequence b;
// false (and the error word) if its offsets or length are out of range.
__device__ __forceinline__ bool new_rows(const CacheView& c, const int32_t* cu, int b, int total,
                                         int max_new, int& first, int& n, int& len) {
    first = cu[b];
    const int end = cu[b + 1];
    len = c.len[b];
    n = end - first;
    const bool ok = first >= 0 && end >= first && end <= total && n <= max_new && len >= 0 &&
                    (long long)len <= ((long long)c.max_pages << c.page_log2);
    if (!ok) raise_error(ERRBIT_DATA);
    return ok;
}

// Sequence whose packed rows hold row r, by bisection over cu [B + 1]: the
// last b with cu[b] <= r (0 if there is none).
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int B, int r) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Exclusive prefix sum of one value per thread over a block of up to 1024
// threads; `tot` receives the sum.  tmp: 33 ints of shared memory.
__device__ __forceinline__ int block_exclusive(int v, int* tmp, int& tot) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) tmp[w] = x;
    __syncthreads();
    if (w == 0) {
        const int s = lane < nw ? tmp[lane] : 0;
        int t = s;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += y;
        }
        tmp[lane] = t - s;
        if (lane == 31) tmp[32] = t;
    }
    __syncthreads();
    const int r = tmp[w] + x - v;
    tot = tmp[32];
    __syncthreads();
    return r;
}

}  // namespace pivot
