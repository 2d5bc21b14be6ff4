// attend.h -- attention over the paged cache: parameters and launchers.
#pragma once

#include <utility>

#include "paged.cuh"

namespace pivot {

// Work is counted in units of one key tile for one block of query rows and
// one key/value head.  The units of a call are numbered sequence by
// sequence, head by head, row block by row block, and CTA c of n takes the
// contiguous run [c U / n, (c + 1) U / n): every CTA gets the same work
// whatever the lengths.  A row block ("item") that more than one CTA worked
// on leaves partial sums in the workspace, which a second kernel joins.
//
// The query rows of a sequence for one key/value head are its new tokens'
// heads of that group, token by token: row r is token r / G, head r % G.
struct AttendParams {
    CacheView c;
    const uint16_t* q;          // bf16 [total, Hq, D]
    const int32_t* cu;          // [B + 1]
    const int32_t* idx;         // [total, topk] or NULL
    uint16_t* o;
    float* lse;
    int Hq, G, total, max_new, window, topk;
    float scale_log2;           // scale * log2(e)
    int R, TK;                  // rows of a block, keys of a tile
    // plan of a paged call (the selected call's is arithmetic)
    long long* seq_units;       // [B + 1] units before sequence b
    int32_t* blk_off;           // [B + 1] row blocks before sequence b
    long long* blk_units;       // per row block: tiles of its sequence's blocks up to it
    // partial sums: slots 2c (a CTA's item that began before its run) and
    // 2c + 1 (one that it began): R rows of D sums, then R maxima, R sums
    float* part;
    // per CTA: what to join where its run begins inside an item
    struct JoinRecord* join;
    int ncta;
};

// Partial sums of one item: CTAs c0 .. c1 worked on it (c0 began it); rows = 0
// where there is nothing to join.
struct JoinRecord {
    long long units;
    int c0, c1, ncta;
    int first, h, row0, rows;
    int pad[3];
};
static_assert(sizeof(JoinRecord) == 48, "three 16-byte reads");

// One item and where it lies among the units.
struct Item {
    int b, h;                   // sequence, key/value head
    int row0, rows;             // its query rows (of the sequence's n G)
    int first;                  // packed row of the sequence's first new token
    int pos0;                   // position of that token
    int tile0, tiles;           // key tiles
    long long unit0;            // first unit
    bool ok;
};

// Total units of the call.
__device__ __forceinline__ int blocks_per_token(const AttendParams& p) { return (p.G + p.R - 1) / p.R; }
__device__ __forceinline__ int selected_tiles(const AttendParams& p) { return (p.topk + p.TK - 1) / p.TK; }

template <bool SELECTED>
__device__ __forceinline__ long long total_units(const AttendParams& p) {
    if constexpr (SELECTED) {
        int rows = p.cu[p.c.B];
        if (rows < 0 || rows > p.total) {
            raise_error(ERRBIT_DATA);
            rows = 0;
        }
        return (long long)rows * p.c.Hkv * blocks_per_token(p) * selected_tiles(p);
    } else {
        return p.seq_units[p.c.B];
    }
}

// CTAs that share the units.  On the rows kernel, whose units are small, a call
// of few units keeps to few CTAs, three units each, so that an item leaves few
// partial sums to join.  One new token over 700 (32 heads on 8), with one, three
// and eight units a CTA: 17.4, 19.5 and 23.6 us for one sequence, 27.6, 25.6 and
// 27.6 for eight; from 3000 tokens on the same.
__device__ __forceinline__ int run_count(const AttendParams& p, long long units) {
    const int ncta = p.ncta;
    const long long n = p.R > 32 ? units : units / 3;
    return n < 1 ? 1 : n < ncta ? (int)n : ncta;
}
// First unit of CTA c's run.
__device__ __forceinline__ long long run_begin(long long units, int c, int ncta) {
    return units * c / ncta;
}
// The CTA whose run holds unit u.
__device__ __forceinline__ int run_of(long long units, long long u, int ncta) {
    return (int)(((u + 1) * ncta - 1) / units);
}

// Row blocks and tiles of a paged call's sequence.
__device__ __forceinline__ void block_tiles(const AttendParams& p, int pos0, int row0, int rows,
                                            int& tile0, int& tiles) {
    const int hi = pos0 + (row0 + rows - 1) / p.G;               // the last token's position
    const int lo = p.window ? max(0, pos0 + row0 / p.G - p.window + 1) : 0;
    tile0 = lo / p.TK;
    tiles = hi / p.TK + 1 - tile0;
}

template <bool SELECTED>
__device__ __forceinline__ Item find_item(const AttendParams& p, long long u) {
    Item it;
    it.ok = true;
    if constexpr (SELECTED) {
        const int nt = selected_tiles(p), nb = blocks_per_token(p);
        long long i = u / nt;
        it.unit0 = i * nt;
        const int blk = (int)(i % nb);
        i /= nb;
        it.h = (int)(i % p.c.Hkv);
        const int r = (int)(i / p.c.Hkv);
        it.b = seq_of_row(p.cu, p.c.B, r);
        int first = 0, n = 0, len = 0;
        it.ok = new_rows(p.c, p.cu, it.b, p.total, p.max_new, first, n, len);
        if (it.ok && len < n) {
            raise_error(ERRBIT_DATA);
            it.ok = false;
        }
        if (it.ok && (r < first || r >= first + n)) it.ok = false;   // before the first offset
        it.first = r;
        it.pos0 = len - n + r - first;
        it.row0 = blk * p.R;
        it.rows = min(p.R, p.G - it.row0);
        it.tile0 = 0;
        it.tiles = nt;
    } else {
        int lo = 0, hi = p.c.B - 1;
        while (lo < hi) {                        // last b with seq_units[b] <= u
            const int mid = (lo + hi + 1) >> 1;
            if (p.seq_units[mid] <= u) lo = mid; else hi = mid - 1;
        }
        it.b = lo;
        const int blk0 = p.blk_off[lo], nblk = p.blk_off[lo + 1] - blk0;
        const long long* cum = p.blk_units + blk0;
        const long long per_head = cum[nblk - 1];
        const long long in_seq = u - p.seq_units[lo];
        it.h = (int)(in_seq / per_head);
        const long long in_head = in_seq % per_head;
        int a = 0, z = nblk - 1;
        while (a < z) {                          // first block whose units end after in_head
            const int mid = (a + z) >> 1;
            if (cum[mid] > in_head) z = mid; else a = mid + 1;
        }
        it.unit0 = p.seq_units[lo] + it.h * per_head + (a ? cum[a - 1] : 0);
        it.first = p.cu[lo];
        const int n = p.cu[lo + 1] - it.first;
        it.pos0 = p.c.len[lo] - n;
        it.row0 = a * p.R;
        it.rows = min(p.R, n * p.G - it.row0);
        block_tiles(p, it.pos0, it.row0, it.rows, it.tile0, it.tiles);
    }
    return it;
}

// The reference point m of an e4m3 softmax stands over weight times value
// scale, so that their product fits f16 whatever the scales.  m moves when one
// could pass 2^E4M3_LAG (f16 ends below 2^16); a move puts the largest at about
// 2^E4M3_HEAD (the rows kernel; the tensor-memory kernel, where a move costs
// more, at 2).  11 bits are kept down to 2^-14 and an absolute 2^-25 below:
// down to 2^-24 (2^-15) of the largest, and 2^-35 (2^-26) of it.  l and o are
// in the same units.  The scale of a key without values does not raise m, and
// on the tensor-memory kernel neither does its score: it adds to l only, and m
// follows it at a distance of 2^EMPTY_BELOW, where l still fits fp32 (2^26
// such keys); so it follows keys of scales below 2^-EMPTY_BELOW.
constexpr float E4M3_HEAD = 10.0f, E4M3_LAG = 15.0f, EMPTY_BELOW = 70.0f;
// Beside a larger m fp32 holds no such distances: the largest is then put at 1.
constexpr float HUGE_POINT = 1048576.0f;

// Where m goes for a largest of `top` (it moves if top - m > E4M3_LAG).
__device__ __forceinline__ float point_at(float m, float top, float head) {
    return fmaxf(m, fabsf(top) > HUGE_POINT ? top : top - head);
}

// For scales of a warp's 32 keys: the log2 of the power of two at or above
// their largest size, within [LO, 100] (LO if all are 0).
template <int LO>
__device__ __forceinline__ float log2_above(float scale) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(scale)));
    const int e = (int)((top + 0x007FFFFFu) >> 23) - 127;
    return (float)(e < LO ? LO : e > 100 ? 100 : e);
}
// The lowest, for scales of K; for those of V as far as m follows keys.
constexpr int LOG2_LOW = -100, LOG2_LOW_V = -70;

// One thread of each CTA: the record of the item that holds the first unit of
// its run, if an earlier CTA began it and no other CTA's run begins between.
__device__ __forceinline__ void put_join(const AttendParams& p, const Item& it, long long units, long long u_begin,
                                         int c, int ncta) {
    JoinRecord r{};
    if (it.ok && it.unit0 < u_begin) {
        r.c0 = run_of(units, it.unit0, ncta);
        if (run_begin(units, r.c0 + 1, ncta) == u_begin) {
            r.units = units;
            r.c1 = run_of(units, it.unit0 + it.tiles - 1, ncta);
            r.ncta = ncta;
            r.first = it.first;
            r.h = it.h;
            r.row0 = it.row0;
            r.rows = it.rows;
        }
    }
    p.join[c] = r;
}

// ------------------------------------------------------------- conversions
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes as two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// 2^e of a whole number within [-126, 127].
__device__ __forceinline__ float exp2_whole(float e) { return __uint_as_float((uint32_t)(127 + (int)e) << 23); }

// Programmatic dependent launch: a kernel lets the next one of its call be
// set up beside it, and waits for the one before to be complete.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Dynamic shared memory of kernel `fn` on the current device, set once.
template <class F>
inline cudaError_t allow_smem(F* fn, int smem, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

// after: the kernel waits for the one before itself (wait_for_previous).
template <class... Formal, class... Actual>
inline cudaError_t launch(bool after, void (*fn)(Formal...), dim3 grid, dim3 block, int smem, cudaStream_t st,
                          Actual&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, std::forward<Actual>(args)...);
}

__device__ __forceinline__ size_t slot_words(int R, int D) { return (size_t)R * (D + 2); }

// Bytes of the plan and of the partial sums.
size_t attend_plan_bytes(int B, int total, int G, int R);
size_t attend_part_bytes(int ncta, int R, int D);

cudaError_t launch_attend_plan(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_rows(const AttendParams& p, cudaStream_t st);
// tk, tv: the planes as token rows x Hkv D values, boxes of a page (at
// most 128 tokens) and one head's codes or 64 bf16 values, 128-byte swizzle
// for 128-byte rows
cudaError_t launch_attend_umma(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p,
                               cudaStream_t st);
cudaError_t launch_attend_join(const AttendParams& p, cudaStream_t st);

// CTAs and tile of the rows kernel.
constexpr int ROWS_CTAS_PER_SM = 2;
inline int rows_tile(int dtype) { return dtype == PIVOT_E4M3 ? 128 : 64; }

}  // namespace pivot
