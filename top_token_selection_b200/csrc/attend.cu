// attend.cu -- attention over a paged key/value cache: the plan, the kernel
// for few query rows a key (single tokens, prediction steps, selected
// positions), and the join of partial sums.
//
// One pass over the keys with the running maximum m and sum l of a softmax:
//     m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),
//     o' = o e^(m - m') + e^(s - m') v,
// in base 2 (scores carry log2 e); o / l at the end.  Partial results over
// disjoint key sets join by the same rule.
#include "attend.h"

namespace pivot {

namespace {

// --------------------------------------------------------------- the plan
constexpr int PLAN_THREADS = 1024;

// One block.  Per sequence the row blocks, per row block the key tiles;
// running sums of both.  Offsets that never descend give the sequences rows
// of their own, total at most, and blk_units has room for their blocks;
// sequences between offsets that descend somewhere could claim the same rows
// again and again, so such a call has no units at all.
__global__ void __launch_bounds__(PLAN_THREADS) attend_plan_kernel(const AttendParams p) {
    __shared__ int tmp[33];
    const int B = p.c.B;
    let_next_start();
    // row blocks before each sequence
    int carry = 0;
    bool descends = false;
    for (int b0 = 0; b0 < B; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        int nb = 0;
        if (b < B) {
            int first, n, len;
            bool ok = new_rows(p.c, p.cu, b, p.total, p.max_new, first, n, len);
            descends = descends || p.cu[b + 1] < p.cu[b];
            if (ok && len < n) {
                raise_error(ERRBIT_DATA);
                ok = false;
            }
            if (ok) nb = (int)(((long long)n * p.G + p.R - 1) / p.R);
        }
        int tot;
        const int x = block_exclusive(nb, tmp, tot);
        if (b < B) p.blk_off[b] = carry + x;
        carry += tot;
    }
    if (threadIdx.x == 0) p.blk_off[B] = carry;
    if (__syncthreads_or(descends)) {          // new_rows has set the error word
        if (threadIdx.x == 0) p.seq_units[B] = 0;
        return;
    }
    // tiles of every row block: running sums over the call's blocks first
    const int nblk = carry;
    long long run = 0;
    for (int j0 = 0; j0 < nblk; j0 += PLAN_THREADS) {
        const int j = j0 + threadIdx.x;
        int tiles = 0;
        if (j < nblk) {
            const int b = seq_of_row(p.blk_off, B, j);
            const int first = p.cu[b], n = p.cu[b + 1] - first;
            const int row0 = (j - p.blk_off[b]) * p.R;
            int tile0;
            block_tiles(p, p.c.len[b] - n, row0, min(p.R, n * p.G - row0), tile0, tiles);
        }
        int tot;
        const int x = block_exclusive(tiles, tmp, tot);
        if (j < nblk && PIVOT_CHECK(j < (long long)p.total * p.G / p.R + B)) p.blk_units[j] = run + x + tiles;
        run += tot;
    }
    __syncthreads();
    // units before each sequence, and each block's sum made its sequence's own
    for (int b = threadIdx.x; b <= B; b += PLAN_THREADS) {
        const int j = p.blk_off[b];
        p.seq_units[b] = (j ? p.blk_units[j - 1] : 0) * p.c.Hkv;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < nblk; j += PLAN_THREADS) {
        const int b = seq_of_row(p.blk_off, B, j);
        p.blk_units[j] -= p.seq_units[b] / p.c.Hkv;
    }
}

// ------------------------------------------------------- warp-level pieces
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared, or 16 zero bytes (nothing read).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4_or_zero(uint32_t dst, const void* src, bool live) {
    const int n = live ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// -------------------------------------------------------- the rows kernel
// A CTA of four warps takes a run of units; in each tile a warp owns KW keys
// and all R = 16 MT query rows, with softmax statistics and sums of its own
// and its own ring of STAGES cp.async stages: no barrier inside an item.
// The warps join through shared memory at the item's end.
//
// mma.sync, not tcgen05: the loads should bound up to 32 rows a key, and
// register fragments let each warp run alone on keys gathered from anywhere.
// They do for bf16: a two-token step over 32 caches of 32K to 128K tokens
// takes 765 us for 5.0 GB, 6.5 TB/s, as a plain copy reaches.  e4m3 codes
// become halves first, two a conversion, and the instructions set the pace:
// 519 us for 2.5 GB in turn with other work, 4.8 TB/s (486 in a short run).
// Three CTAs an SM at 168 registers and two stages instead of two at 255 and
// three moved the e4m3 step by 1% and the same step of one key/value head by
// 2% the other way.
template <int D, bool FP8, int MT>
struct RowsShape {
    static constexpr int WARPS = 4;
    static constexpr int R = 16 * MT;
    static constexpr int KW = FP8 ? 32 : 16;             // keys of a warp in a tile
    static constexpr int TK = WARPS * KW;
    static constexpr int ROWB = D * (FP8 ? 1 : 2);       // bytes of a key of one head
    static constexpr int CH = ROWB / 16;
    static constexpr int HALF = KW * ROWB;               // K (or V) of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = STAGE >= 8192 ? 3 : 5;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int SCALES = FP8 ? WARPS * STAGES * 2 * KW * 4 : 0;
    static constexpr int QROW = D * 2 + 16;              // padded: rows fall on different banks
    static constexpr int QBYTES = R * QROW;
    static constexpr int JOIN = WARPS * R * (D + 2) * 4; // the warps' sums, in the drained ring
    static constexpr int RING_ALL = RING > JOIN ? RING : JOIN;
    static constexpr int SMEM = RING_ALL + SCALES + QBYTES + R * 4 + 128;
};

// Byte of 16-byte chunk `c` of key `k` in a warp's K or V stage: chunks are
// permuted so that eight keys' same chunk (ldmatrix) and two keys' four
// chunks (16-byte reads of codes) fall on different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t key_chunk(int k, int c) {
    if constexpr (ROWB >= 128) {
        const int f = ((k & 1) << 2) | ((k >> 1) & 3);
        return (uint32_t)(k * ROWB + ((c ^ f) << 4));
    } else {
        return (uint32_t)(k * ROWB + ((c ^ ((k >> 1) & 3)) << 4));
    }
}

template <int D, bool FP8, int MT, bool SELECTED>
__global__ void __launch_bounds__(128, ROWS_CTAS_PER_SM) attend_rows_kernel(const AttendParams p) {
    using S = RowsShape<D, FP8, MT>;
    constexpr int KW = S::KW, R = S::R, NT = KW / 8, KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* scales = reinterpret_cast<float*>(smem + S::RING_ALL);
    uint8_t* qs = smem + S::RING_ALL + S::SCALES;
    float* qmul = reinterpret_cast<float*>(qs + S::QBYTES);    // [R] factor of a row's scores

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c4 = lane & 3;
    let_next_start();
    if constexpr (!SELECTED) wait_for_previous();
    const long long units = total_units<SELECTED>(p);
    const int ncta = run_count(p, units);
    const bool used = (int)blockIdx.x < ncta;
    const long long u_end = used ? run_begin(units, blockIdx.x + 1, ncta) : 0;
    long long u = used ? run_begin(units, blockIdx.x, ncta) : 0;
    const long long u_begin = u;
    if (u == u_end && threadIdx.x == 0) p.join[blockIdx.x].rows = 0;
    const uint32_t my_ring = smem_u32(ring) + warp * (S::STAGES * S::STAGE);
    float* my_scales = scales + warp * (S::STAGES * 2 * KW);

    // e4m3: where some row's |m| passes HUGE_POINT, fp32 does not hold lv in it,
    // and scales met f16 as they are.  The CTA then goes over the item again,
    // each warp with its scales in units of 2^unit, the largest: its weights
    // are larger by that, and m smaller.
    bool again = false;
    float unit = 0.0f;
    while (u < u_end) {
        const long long u0 = u;
        const Item it = find_item<SELECTED>(p, u);
        const int ta = it.tile0 + (int)(u - it.unit0);
        const int tz = it.tile0 + (int)min((long long)it.tiles, u_end - it.unit0);
        const bool whole = it.unit0 >= u_begin && it.unit0 + it.tiles <= u_end;
        const int slot = 2 * blockIdx.x + (it.unit0 < u_begin ? 0 : 1);
        if (u == u_begin && threadIdx.x == 0) put_join(p, it, units, u_begin, blockIdx.x, ncta);
        u = it.unit0 + (tz - it.tile0);
        if (!it.ok) continue;

        // ---- query rows into shared memory.  For e4m3 keys they become
        // halves: a row is divided by the power of two under its largest
        // value, which keeps 11 bits of values down to 2^-14 of it and an
        // absolute 2^-25 of it below, and its scores are multiplied back.
        for (int r = warp; r < R; r += 4) {
            const bool live = r < it.rows;
            const int rr = it.row0 + r;
            const uint16_t* src =
                p.q + ((size_t)(it.first + rr / p.G) * p.Hq + it.h * p.G + rr % p.G) * D;
            constexpr int PER = D / 64;                 // pairs a lane
            uint32_t x[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                x[i] = live ? reinterpret_cast<const uint32_t*>(src)[lane + 32 * i] : 0u;
            float mul = p.scale_log2;
            if constexpr (FP8) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i] << 16)),
                                             fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
#pragma unroll
                for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                // within [2^-125, 2^124]: 2^e and 2^-e are normal
                const uint32_t e =
                    min(max(__float_as_uint(amax) & 0x7F800000u, 0x01000000u), 0x7D800000u);
                const float down = __uint_as_float(0x7F000000u - e);
                mul = fminf(mul * __uint_as_float(e), 0x1p127f);   // a score of 0 stays 0
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    x[i] = f16x2(__uint_as_float(x[i] << 16) * down,
                                 __uint_as_float(x[i] & 0xFFFF0000u) * down);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                reinterpret_cast<uint32_t*>(qs + r * S::QROW)[lane + 32 * i] = x[i];
            if (lane == 0) qmul[r] = mul;
        }
        __syncthreads();

        // fragments of Q: kept for 16 rows, read again each tile for 32
        uint32_t qf[MT == 1 ? KS : 1][4];
        auto load_q = [&](int mt, int ks, uint32_t (&a)[4]) {
            if constexpr (FP8) {
                // the order of the contraction is free: thread c4 takes the 16
                // values of chunk c4 (then c4 + 4) of its key, four a step
                const int d = (ks >> 2) * 64 + c4 * 16 + (ks & 3) * 4;
                const uint2 lo = *reinterpret_cast<const uint2*>(qs + (mt * 16 + g) * S::QROW + d * 2);
                const uint2 hi =
                    *reinterpret_cast<const uint2*>(qs + (mt * 16 + g + 8) * S::QROW + d * 2);
                a[0] = lo.x; a[1] = hi.x; a[2] = lo.y; a[3] = hi.y;
            } else {
                ldsm4(a, smem_u32(qs) + (mt * 16 + (lane & 15)) * S::QROW + ks * 32 + (lane >> 4) * 16);
            }
        };
        if constexpr (MT == 1) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) load_q(0, ks, qf[ks]);
        }
        float mul[MT][2];
        int lim[MT][2];          // paged: the row's position (rows past the block see nothing)
        int lim_lo = 0x7fffffff, lim_hi = -1;    // of the live rows
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + g + 8 * e;
                mul[mt][e] = qmul[r];
                lim[mt][e] = r < it.rows ? it.pos0 + (it.row0 + r) / p.G : -1;
            }
        lim_lo = it.pos0 + it.row0 / p.G;
        lim_hi = it.pos0 + (it.row0 + it.rows - 1) / p.G;
        const int key_lo = p.window ? max(0, lim_lo - p.window + 1) : 0;   // first position any row reads

        float m[MT][2], l[MT][2], acc[MT][D / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) { m[mt][e] = -INFINITY; l[mt][e] = 0.0f; }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][n][e] = 0.0f;
        }

        // ---- the ring.  Lane kk owns key kk of the warp's step; a step's
        // positions, then its token rows, are read one step ahead of its copy.
        const int kk = lane & (KW - 1);
        const int32_t* sel = SELECTED ? p.idx + (size_t)it.first * p.topk : nullptr;
        const int32_t* pages = p.c.table + (size_t)it.b * p.c.max_pages;
        auto position = [&](int t) -> int {
            const int s = t * S::TK + warp * KW + kk;
            if (t >= tz) return -1;
            if constexpr (SELECTED) {
                const int pos = s < p.topk ? ld_nc_early(sel + s) : -1;
                return pos;
            } else {
                return s >= key_lo && s <= lim_hi ? s : -1;
            }
        };
        auto page_of = [&](int pos) -> int {
            if (SELECTED && pos > it.pos0) return -2;
            return pos >= 0 ? ld_nc_early(pages + (pos >> p.c.page_log2)) : -2;
        };
        if (FP8 && again) {
            float most = 0.0f;
#pragma unroll 1
            for (int t = ta; t < tz; ++t) {
                const int pos = position(t), page = page_of(pos);
                const int row = page == -2 ? -1 : p.c.row_of(page, pos);
                if (row >= 0) most = fmaxf(most, fabsf(p.c.vs[row]));
            }
            unit = __any_sync(0xffffffffu, most > 0.0f) ? log2_above<LOG2_LOW_V>(most) : 0.0f;
        }
        int pos_a = position(ta), page_a = page_of(pos_a);      // step to copy next
        int pos_b = position(ta + 1);                           // and the one after
        uint32_t ring_ok[S::STAGES];                            // keys that count, by stage
#pragma unroll
        for (int i = 0; i < S::STAGES; ++i) ring_ok[i] = 0;
        const size_t head_off = (size_t)it.h * S::ROWB;
        uint32_t put_ok = 0;
        auto copy = [&](int t, int stage) {
            int row = -1;
            if (page_a != -2) {
                row = p.c.row_of(page_a, pos_a);
                if (row < 0) raise_error(ERRBIT_DATA);
                if (!PIVOT_CHECK(row < (long long)p.c.num_pages << p.c.page_log2)) row = -1;
            }
            put_ok = __ballot_sync(0xffffffffu, row >= 0);
            // the next step's page, the one after its positions
            pos_a = pos_b;
            page_a = page_of(pos_a);
            pos_b = position(t + 2);
            const uint32_t dst = my_ring + stage * S::STAGE;
            constexpr int KPI = 32 / S::CH;                    // keys an instruction
            const int ch = lane % S::CH;
#pragma unroll
            for (int i = 0; i < KW / KPI; ++i) {
                const int k = i * KPI + lane / S::CH;
                const int kr = __shfl_sync(0xffffffffu, row, k);
                const size_t off = (size_t)(kr < 0 ? 0 : kr) * p.c.rowb + head_off + ch * 16;
                cp16_or_zero(dst + key_chunk<S::ROWB>(k, ch), p.c.k + off, kr >= 0);
                cp16_or_zero(dst + S::HALF + key_chunk<S::ROWB>(k, ch), p.c.v + off, kr >= 0);
            }
            if constexpr (FP8) {
                const uint32_t sd = smem_u32(my_scales + stage * 2 * KW) + kk * 4;
                const int sr = row < 0 ? 0 : row;
                cp4_or_zero(sd, p.c.ks + sr, row >= 0);
                if (unit == 0.0f) cp4_or_zero(sd + KW * 4, p.c.vs + sr, row >= 0);
                else my_scales[stage * 2 * KW + KW + kk] = row >= 0 ? p.c.vs[sr] * exp2_whole(-unit) : 0.0f;
            }
        };
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) {
            if (ta + i < tz) {
                copy(ta + i, i);
                ring_ok[i] = put_ok;
            }
            cp_async_commit();
        }
        int stage = 0;
        for (int t = ta; t < tz; ++t) {
            cp_async_wait<S::STAGES - 2>();
            __syncwarp();
            const uint32_t ok = ring_ok[0];
            // the stage read in the last step is free: fill it
            {
                int fill = stage + S::STAGES - 1;
                if (fill >= S::STAGES) fill -= S::STAGES;
                put_ok = 0;
                if (t + S::STAGES - 1 < tz) copy(t + S::STAGES - 1, fill);
                cp_async_commit();
#pragma unroll
                for (int i = 0; i < S::STAGES - 2; ++i) ring_ok[i] = ring_ok[i + 1];
                ring_ok[S::STAGES - 2] = put_ok;
            }
            const uint32_t kbase = my_ring + stage * S::STAGE, vbase = kbase + S::HALF;
            float* sc = my_scales + stage * 2 * KW;
            if (++stage == S::STAGES) stage = 0;
            const uint32_t every = KW == 32 ? 0xffffffffu : 0xffffu;
            if ((ok & every) == 0) continue;                   // nothing in this step counts

            // ---- scores
            float s[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.0f;
            if constexpr (FP8) {
#pragma unroll
                for (int half = 0; half < KS / 4; ++half) {
                    uint4 kc[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t a = kbase + key_chunk<S::ROWB>(n * 8 + g, half * 4 + c4);
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(kc[n].x), "=r"(kc[n].y), "=r"(kc[n].z), "=r"(kc[n].w)
                                     : "r"(a));
                    }
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t af[MT][4];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            if constexpr (MT == 1) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) af[0][e] = qf[half * 4 + q4][e];
                            } else {
                                load_q(mt, half * 4 + q4, af[mt]);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t w = q4 == 0 ? kc[n].x : q4 == 1 ? kc[n].y : q4 == 2 ? kc[n].z : kc[n].w;
                            const uint32_t b0 = e4m3x2_f16x2((uint16_t)(w & 0xFFFFu));
                            const uint32_t b1 = e4m3x2_f16x2((uint16_t)(w >> 16));
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) mma_f16(s[mt][n], af[mt], b0, b1);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kb[4];
                    const int k = (lane & 7) + ((lane >> 4) << 3), ch = ks * 2 + ((lane >> 3) & 1);
                    ldsm4(kb, kbase + key_chunk<S::ROWB>(k, ch));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t af[4];
                        if constexpr (MT == 1) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) af[e] = qf[ks][e];
                        } else {
                            load_q(mt, ks, af);
                        }
                        mma_bf16(s[mt][0], af, kb[0], kb[1]);
                        mma_bf16(s[mt][1], af, kb[2], kb[3]);
                    }
                }
            }

            // ---- factors and masks
            const int key0 = t * S::TK + warp * KW;
            float kmul[NT][2];
            if constexpr (FP8) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 x = *reinterpret_cast<const float2*>(sc + n * 8 + c4 * 2);
                    kmul[n][0] = x.x;
                    kmul[n][1] = x.y;
                }
            }
            const bool plain = (ok & every) == every &&
                               (SELECTED || (key0 + KW - 1 <= lim_lo &&
                                             (!p.window || key0 > lim_hi - p.window)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[mt][n][e] * mul[mt][e >> 1];
                        if constexpr (FP8) x *= kmul[n][e & 1];
                        if (!plain) {
                            const int k = n * 8 + c4 * 2 + (e & 1);
                            bool see = (ok >> k) & 1;
                            if constexpr (!SELECTED) {
                                const int d = lim[mt][e >> 1] - (key0 + k);
                                see = see && d >= 0 && (!p.window || d < p.window);
                            }
                            if (!see) x = -INFINITY;
                        }
                        s[mt][n][e] = x;
                    }

            // ---- reference point: the running maximum (e4m3: see E4M3_HEAD, lv
            // is log2 of the step's largest value scale); the sums move only
            // when it does
            float lv = 0.0f;
            if constexpr (FP8) lv = log2_above<LOG2_LOW_V>(sc[KW + lane]);
            uint32_t pf[MT][NT / 2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mx[0] = fmaxf(mx[0], fmaxf(s[mt][n][0], s[mt][n][1]));
                    mx[1] = fmaxf(mx[1], fmaxf(s[mt][n][2], s[mt][n][3]));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                }
                bool move = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (FP8)
                        move = move || (mx[e] + lv) - m[mt][e] > E4M3_LAG;
                    else
                        move = move || mx[e] > m[mt][e];
                }
                if (__any_sync(0xffffffffu, move)) {
                    if constexpr (FP8) {
                        // keys without values, whose scale does not count: a
                        // lane looks at one, as far as it has to
                        uint32_t some = 0;
#pragma unroll 1
                        for (int ch = 0; ch < S::CH && !__all_sync(0xffffffffu, some & 0x7F7F7F7Fu); ++ch) {
                            uint32_t x, y, z, w;
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                                         : "r"(vbase + key_chunk<S::ROWB>(lane, ch)));
                            some |= x | y | z | w;
                        }
                        if (!__all_sync(0xffffffffu, some & 0x7F7F7F7Fu)) {
                            if (!(some & 0x7F7F7F7Fu)) sc[KW + lane] = 0.0f;
                            __syncwarp();
                            lv = log2_above<LOG2_LOW_V>(sc[KW + lane]);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) mx[e] += lv;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (FP8 && !(mx[e] - m[mt][e] > E4M3_LAG)) continue;
                        const float to = FP8 ? point_at(m[mt][e], mx[e], E4M3_HEAD) : fmaxf(mx[e], m[mt][e]);
                        const float f = m[mt][e] == -INFINITY ? 0.0f : ex2(m[mt][e] - to);
                        m[mt][e] = to;
                        l[mt][e] *= f;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            acc[mt][n][2 * e] *= f;
                            acc[mt][n][2 * e + 1] *= f;
                        }
                    }
                }
                const float z0 = m[mt][0] == -INFINITY ? 0.0f : m[mt][0];
                const float z1 = m[mt][1] == -INFINITY ? 0.0f : m[mt][1];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float e0 = ex2(s[mt][n][0] - z0), e1 = ex2(s[mt][n][1] - z0);
                    float e2 = ex2(s[mt][n][2] - z1), e3 = ex2(s[mt][n][3] - z1);
                    // the sum takes the weights as they are (the log-sum-exp
                    // is wanted in fp32); for the product they keep the 8 bits
                    // of the bf16 values they meet (an error of at most 2^-8
                    // of each weight, independent from key to key), or the 11
                    // of f16 beside e4m3 values, which f16 holds exactly
                    l[mt][0] += e0 + e1;
                    l[mt][1] += e2 + e3;
                    if constexpr (FP8) {
                        // the value's scale goes with the weight
                        const float2 v = *reinterpret_cast<const float2*>(sc + KW + n * 8 + c4 * 2);
                        e0 *= v.x; e1 *= v.y; e2 *= v.x; e3 *= v.y;
                    }
                    const uint32_t lo = FP8 ? f16x2(e0, e1) : bf16x2(e0, e1);
                    const uint32_t hi = FP8 ? f16x2(e2, e3) : bf16x2(e2, e3);
                    pf[mt][n >> 1][(n & 1) * 2] = lo;
                    pf[mt][n >> 1][(n & 1) * 2 + 1] = hi;
                }
            }

            // ---- weights times values
            if constexpr (FP8) {
#pragma unroll
                for (int ch = 0; ch < S::CH; ++ch) {
                    // 32 keys x 16 values as byte pairs: thread (g, c4) gets
                    // values 2g, 2g + 1 of keys 2c4, 2c4 + 1 of each eight
                    uint32_t r[4];
                    ldsm4t(r, vbase + key_chunk<S::ROWB>(lane, ch));
                    uint32_t even[4], odd[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = __byte_perm(r[i], 0, 0x3120);
                        even[i] = e4m3x2_f16x2((uint16_t)(w & 0xFFFFu));
                        odd[i] = e4m3x2_f16x2((uint16_t)(w >> 16));
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_f16(acc[mt][2 * ch], pf[mt][0], even[0], even[1]);
                        mma_f16(acc[mt][2 * ch], pf[mt][1], even[2], even[3]);
                        mma_f16(acc[mt][2 * ch + 1], pf[mt][0], odd[0], odd[1]);
                        mma_f16(acc[mt][2 * ch + 1], pf[mt][1], odd[2], odd[3]);
                    }
                }
            } else {
#pragma unroll
                for (int d16 = 0; d16 < D / 16; ++d16) {
                    uint32_t vb[4];
                    ldsm4t(vb, vbase + key_chunk<S::ROWB>(lane & 15, d16 * 2 + (lane >> 4)));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_bf16(acc[mt][2 * d16], pf[mt][0], vb[0], vb[1]);
                        mma_bf16(acc[mt][2 * d16 + 1], pf[mt][0], vb[2], vb[3]);
                    }
                }
            }
        }

        // ---- the four warps' sums, through the drained ring
        cp_async_wait<0>();
        if constexpr (FP8) {
            bool huge = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) huge = huge || (fabsf(m[mt][e]) > HUGE_POINT && m[mt][e] > -INFINITY);
            again = __syncthreads_or(huge) && !again;
            if (again) {
                u = u0;
                continue;
            }
        } else {
            __syncthreads();
        }
        float* join = reinterpret_cast<float*>(ring);
        float* jm = join + S::WARPS * R * D;                   // [WARPS][R] maxima, then sums
        float* jl = jm + S::WARPS * R;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + g + 8 * e;
                float x = l[mt][e], f = 1.0f;
                if constexpr (FP8) {
                    if (unit != 0.0f) {  // back to units of 1; where m cannot take it, the sums
                        const bool sums = fabsf(m[mt][e]) > HUGE_POINT && m[mt][e] > -INFINITY;
                        f = sums ? exp2_whole(unit) : 1.0f;
                        x *= sums ? 1.0f : exp2_whole(-unit);
                        m[mt][e] += sums ? 0.0f : unit;
                    }
                }
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (c4 == 0) {
                    jm[warp * R + r] = m[mt][e];
                    jl[warp * R + r] = x;
                }
                float* to = join + (size_t)(warp * R + r) * D;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    if constexpr (FP8) {
                        // tiles 2i and 2i + 1 hold the even and odd values of 16
                        const int d = (n >> 1) * 16 + c4 * 4 + (n & 1);
                        to[d] = acc[mt][n][2 * e] * f;
                        to[d + 2] = acc[mt][n][2 * e + 1] * f;
                    } else {
                        *reinterpret_cast<float2*>(to + n * 8 + c4 * 2) =
                            make_float2(acc[mt][n][2 * e], acc[mt][n][2 * e + 1]);
                    }
                }
            }
        __syncthreads();
        constexpr int LPR = D / 4;                             // threads a row, four values each
        for (int i = threadIdx.x; i < it.rows * LPR; i += 128) {
            const int r = i / LPR, d = (i % LPR) * 4;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) mx = fmaxf(mx, jm[w * R + r]);
            const float z = mx == -INFINITY ? 0.0f : mx;
            float sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) {
                const float f = ex2(jm[w * R + r] - z);
                sum += jl[w * R + r] * f;
                const float4 x = *reinterpret_cast<const float4*>(join + (size_t)(w * R + r) * D + d);
                o[0] += x.x * f; o[1] += x.y * f; o[2] += x.z * f; o[3] += x.w * f;
            }
            const int rr = it.row0 + r;
            if (whole) {
                const size_t head = (size_t)(it.first + rr / p.G) * p.Hq + it.h * p.G + rr % p.G;
                const bool none = mx == -INFINITY && sum == 0.0f;
                const float inv = none ? 0.0f : 1.0f / sum;
                uint2 y;
                y.x = bf16x2(o[0] * inv, o[1] * inv);
                y.y = bf16x2(o[2] * inv, o[3] * inv);
                *reinterpret_cast<uint2*>(p.o + head * D + d) = y;
                if (p.lse && d == 0)
                    p.lse[head] = none ? -INFINITY : (z + __log2f(sum)) * 0.6931471805599453f;
            } else if (PIVOT_CHECK(slot < 2 * p.ncta)) {
                float* to = p.part + (size_t)slot * slot_words(R, D);
                *reinterpret_cast<float4*>(to + (size_t)r * D + d) = make_float4(o[0], o[1], o[2], o[3]);
                if (d == 0) {
                    to[(size_t)R * D + r] = mx;
                    to[(size_t)R * D + R + r] = sum;
                }
            }
        }
        unit = 0.0f;
        __syncthreads();   // the ring and the query rows are free again
    }
}

// ---------------------------------------------------------------- the join
// A warp a row of the item whose record CTA blockIdx.x + 1 of the call left.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendParams p) {
    wait_for_previous();
    const JoinRecord j = p.join[blockIdx.x + 1];
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (r >= j.rows) return;
    constexpr int PER = D / 32;
    const size_t words = slot_words(p.R, D);
    auto sums = [&](int i) { return p.part + (size_t)(2 * i + (i == j.c0)) * words; };
    // a lane a partial: its maximum and sum
    float m = -INFINITY, l = 0.0f;
    for (int i = j.c0 + lane; i <= j.c1; i += 32) {
        const float* s = sums(i) + (size_t)p.R * D;
        const float mi = s[r], li = s[p.R + r];
        const float top = fmaxf(m, mi);
        const float z = top == -INFINITY ? 0.0f : top;
        l = l * ex2(m - z) + li * ex2(mi - z);
        m = top;
    }
    float mx = m;
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float z = mx == -INFINITY ? 0.0f : mx;
    float sum = l * ex2(m - z), o[PER];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
    for (int k = 0; k < PER; ++k) o[k] = 0.0f;
    // four partials at a time: their loads do not wait for one another
    for (int i0 = j.c0; i0 <= j.c1; i0 += 4) {
        float x[4][PER], f[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const bool ok = i0 + y <= j.c1;
            const float* s = sums(ok ? i0 + y : j.c0);
            f[y] = ok ? ex2(s[(size_t)p.R * D + r] - z) : 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) x[y][k] = s[(size_t)r * D + lane * PER + k];
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int k = 0; k < PER; ++k) o[k] = f[y] == 0.0f ? o[k] : fmaf(x[y][k], f[y], o[k]);
    }
    const int rr = j.row0 + r;
    const size_t head = (size_t)(j.first + rr / p.G) * p.Hq + j.h * p.G + rr % p.G;
    const bool none = mx == -INFINITY && sum == 0.0f;
    const float inv = none ? 0.0f : 1.0f / sum;
    uint32_t* to = reinterpret_cast<uint32_t*>(p.o + head * D + lane * PER);
#pragma unroll
    for (int k = 0; k < PER; k += 2) to[k / 2] = bf16x2(o[k] * inv, o[k + 1] * inv);
    if (p.lse && lane == 0) p.lse[head] = none ? -INFINITY : (z + __log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool FP8, int MT, bool SELECTED>
cudaError_t launch_rows_one(const AttendParams& p, cudaStream_t st) {
    auto fn = attend_rows_kernel<D, FP8, MT, SELECTED>;
    constexpr int smem = RowsShape<D, FP8, MT>::SMEM;
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs an SM");
    static bool done[64] = {false};
    const cudaError_t e = allow_smem(fn, smem, done);
    if (e != cudaSuccess) return e;
    return launch(!SELECTED, fn, p.ncta, 128, smem, st, p);
}

template <int D, bool FP8, bool SELECTED>
cudaError_t launch_rows_mt(const AttendParams& p, cudaStream_t st) {
    return p.R == 16 ? launch_rows_one<D, FP8, 1, SELECTED>(p, st)
                     : launch_rows_one<D, FP8, 2, SELECTED>(p, st);
}

template <int D, bool SELECTED>
cudaError_t launch_rows_type(const AttendParams& p, cudaStream_t st) {
    return p.c.ks ? launch_rows_mt<D, true, SELECTED>(p, st) : launch_rows_mt<D, false, SELECTED>(p, st);
}

}  // namespace

size_t attend_plan_bytes(int B, int total, int G, int R) {
    const size_t blocks = (size_t)((long long)total * G / R) + B;
    return (size_t)(B + 1) * 8 + blocks * 8 + (size_t)(B + 1) * 4;
}
size_t attend_part_bytes(int ncta, int R, int D) {
    return (size_t)ncta * (sizeof(JoinRecord) + (size_t)2 * R * (D + 2) * 4);
}

cudaError_t launch_attend_plan(const AttendParams& p, cudaStream_t st) {
    attend_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attend_rows(const AttendParams& p, cudaStream_t st) {
    if (p.idx) return p.c.D == 128 ? launch_rows_type<128, true>(p, st) : launch_rows_type<64, true>(p, st);
    return p.c.D == 128 ? launch_rows_type<128, false>(p, st) : launch_rows_type<64, false>(p, st);
}

cudaError_t launch_attend_join(const AttendParams& p, cudaStream_t st) {
    if (p.ncta < 2) return cudaSuccess;
    const dim3 grid(p.ncta - 1, p.R / 4);
    return p.c.D == 128 ? launch(true, attend_join_kernel<128>, grid, 128, 0, st, p)
                        : launch(true, attend_join_kernel<64>, grid, 128, 0, st, p);
}

}  // namespace pivot
