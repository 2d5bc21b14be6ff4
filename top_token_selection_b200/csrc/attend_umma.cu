// attend_umma.cu -- attention over a paged key/value cache on the
// 5th-generation tensor cores, for blocks of many query rows a key: chunks
// of new tokens, and selected positions with many query heads a key head.
//
// S = Q K^T and O += P V by tcgen05.mma with the accumulators in TMEM:
// 128 query rows on the M axis (the 128 TMEM lanes), so one thread owns one
// row's softmax and no shuffle is needed; 128 keys a tile.  P goes back to
// TMEM in 16 bits, over the S it came from, and is the A operand of the second
// product (bf16 beside bf16 values; e4m3 codes are converted to f16, which
// holds them exactly, and P is f16 then).  Two such tiles are in flight and take turns: while one's softmax
// runs, the tensor cores work on the other.  They are
//  * the two halves of a block of 256 rows, which share every key tile; or
//  * (SPLIT) the even and odd key tiles of one block of up to 128 rows, each
//    with sums of its own that are joined at the end.
//
// TMEM (512 columns): S/P of tile 0, S/P of tile 1, O of tile 0, O of tile 1.
//
// Warps 0-3 and 4-7: softmax of tiles 0 and 1.  Warps 8-10: loads, every
// third K or V tile each.  Warp 11: MMA issue.  Three warps on each of the
// SM's four register files leave 168 registers a thread: the softmax holds
// its row's 128 scores.
#include "attend.h"

namespace pivot {

namespace {

constexpr int TKEYS = 128;
constexpr int THREADS = 384;
constexpr int LOAD_WARP = 8, MMA_WARP = 11;

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
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 16 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Descriptor of V as the B operand with N (values of a key) contiguous: the
// tile is 8-key x 64-value atoms of 1024 bytes with the 128-byte swizzle;
// leading offset 16 KB to the next 64 values, stride 1 KB to the next 8 keys.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(TKEYS * 128 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

template <int D, bool FP8>
struct UmmaShape {
    static constexpr int TILE = TKEYS * D * 2;               // K or V tile, and 128 rows of Q
    static constexpr int STAGES = FP8 ? 3 : (D == 128 ? 5 : 8);
    // e4m3 codes wait in a staging tile of each load warp and are converted
    // from there; bf16 goes into the tile directly
    static constexpr int STAGING = FP8 ? 3 * TKEYS * D : 0;
    // per tile what the softmax needs besides S: which keys count, and for
    // e4m3 their scales.  A slot is written again once the K tile MS later
    // has a ring slot, which is after its readers are done: 2 MS > STAGES.
    static constexpr int MS = 8;
    static_assert(2 * MS > STAGES, "meta slots outlive the ring");
    static constexpr int META = MS * (16 + (FP8 ? 16 + TKEYS * 8 : 0));
    static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + STAGING + META + 512;
};

template <int D, bool FP8, bool SELECTED, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) attend_umma_kernel(const AttendParams p) {
    using S = UmmaShape<D, FP8>;
    constexpr int STAGES = S::STAGES, MS = S::MS;
    constexpr int R = SPLIT ? 128 : 256;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sQ = smem;                                   // two tiles of 128 rows
    uint8_t* sT = sQ + 2 * S::TILE;                       // K and V tiles in turn
    uint8_t* sC = sT + STAGES * S::TILE;                  // e4m3 codes on their way
    uint8_t* sM = sC + S::STAGING;
    uint32_t* m_ok = reinterpret_cast<uint32_t*>(sM);     // [MS][4]
    float* m_lv = reinterpret_cast<float*>(sM + MS * 16); // [MS][4] see log2_above
    float* m_ks = m_lv + MS * 4;                          // [MS][128]
    float* m_vs = m_ks + MS * TKEYS;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sM + S::META);
    uint64_t* full = bars;                                // [STAGES] tile there
    uint64_t* empty = full + STAGES;                      // [STAGES] tile read
    uint64_t* mfull = empty + STAGES;                     // [MS] meta there
    uint64_t* sfull = mfull + MS;                         // [2] S there
    uint64_t* pfull = sfull + 2;                          // [2] P there
    uint64_t* ofull = pfull + 2;                          // [2] O complete
    uint64_t* qfull = ofull + 2;                          // Q there
    uint64_t* drain = qfull + 1;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drain + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < MS; ++i) mbar_init(&mfull[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&ofull[i], 1);
        }
        mbar_init(qfull, SPLIT ? 4 : 8);
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(tmem_at, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    const long long units = total_units<SELECTED>(p);
    const long long u_begin = run_begin(units, blockIdx.x, p.ncta);
    const long long u_end = run_begin(units, blockIdx.x + 1, p.ncta);

    if (warp >= LOAD_WARP && warp < MMA_WARP) {
        // ------------------------------------------------------------- loads
        // The K and V tiles are numbered in the order of the ring; warp w
        // takes every third.  A lane looks after keys lane, lane + 32, ... of
        // its tile: their positions are read two own tiles ahead, their page
        // ids one.
        const int lw = warp - LOAD_WARP;
        long long entry0 = 0;            // tiles of the items before
        int tile_no = 0;                 // key tiles of the items before
        bool aborted = false;
        constexpr int CH = D * (FP8 ? 1 : 2) / 16;         // 16-byte chunks of a stored row
        constexpr int KPI = 32 / CH;                       // keys an instruction
        const int ch = lane % CH, sub = lane / CH;
        for (long long u = u_begin; u < u_end && !aborted;) {
            const Item it = find_item<SELECTED>(p, u);
            const int ta = it.tile0 + (int)(u - it.unit0);
            const int tz = it.tile0 + (int)min((long long)it.tiles, u_end - it.unit0);
            u = it.unit0 + (tz - it.tile0);
            if (!it.ok) continue;
            const int lim_lo = it.pos0 + it.row0 / p.G;
            const int lim_hi = it.pos0 + (it.row0 + it.rows - 1) / p.G;
            const int key_lo = p.window ? max(0, lim_lo - p.window + 1) : 0;
            const int32_t* sel = SELECTED ? p.idx + (size_t)it.first * p.topk : nullptr;
            const int32_t* pages = p.c.table + (size_t)it.b * p.c.max_pages;
            const size_t head_off = (size_t)it.h * D * (FP8 ? 1 : 2) + ch * 16;
            const int total = 2 * (tz - ta);               // tiles of this item
            int x = (int)((lw + 3 - entry0 % 3) % 3);      // the next one of this warp
            auto position = [&](int x, int g) -> int {
                const int t = ta + (x >> 1), s = t * TKEYS + g * 32 + lane;
                if (x >= total) return -1;
                if constexpr (SELECTED) return s < p.topk ? ld_nc_early(sel + s) : -1;
                else return s >= key_lo && s <= lim_hi ? s : -1;
            };
            auto page_of = [&](int pos) -> int {
                if (SELECTED && pos > it.pos0) return -2;
                return pos >= 0 ? ld_nc_early(pages + (pos >> p.c.page_log2)) : -2;
            };
            int pos_a[4], page_a[4], pos_b[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) pos_a[g] = position(x, g);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                page_a[g] = page_of(pos_a[g]);
                pos_b[g] = position(x + 3, g);
            }
            // Token rows of this lane's keys of tile x; the next own tile's
            // pages and the positions after it are then under way.  All waits
            // come before all loads: a load waited for beside younger ones
            // costs their latency too.
            auto resolve = [&](int x, int (&row)[4]) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    row[g] = -1;
                    if (page_a[g] != -2) {
                        row[g] = p.c.row_of(page_a[g], pos_a[g]);
                        if (row[g] < 0) raise_error(ERRBIT_DATA);
                    }
                    pos_a[g] = pos_b[g];
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) page_a[g] = page_of(pos_a[g]);
#pragma unroll
                for (int g = 0; g < 4; ++g) pos_b[g] = position(x + 6, g);
            };
            auto wait_slot = [&](long long e) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(&empty[e % STAGES], (uint32_t)((e / STAGES) & 1) ^ 1));
            };
            auto publish = [&](long long e) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[e % STAGES]);
            };
            if constexpr (!FP8) {
                for (; x < total; x += 3) {
                    const long long e = entry0 + x;
                    int row[4];
                    uint32_t ok[4];
                    resolve(x, row);
#pragma unroll
                    for (int g = 0; g < 4; ++g) ok[g] = __ballot_sync(0xffffffffu, row[g] >= 0);
                    if (!wait_slot(e)) { aborted = true; break; }
                    if ((x & 1) == 0 && lane < 4)
                        m_ok[((tile_no + (x >> 1)) % MS) * 4 + lane] =
                            lane == 0 ? ok[0] : lane == 1 ? ok[1] : lane == 2 ? ok[2] : ok[3];
                    const uint8_t* plane = ((x & 1) ? p.c.v : p.c.k) + head_off;
                    const uint32_t dst = smem_u32(sT + (e % STAGES) * S::TILE) + (ch >> 3) * (TKEYS * 128);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int i = 0; i < 32 / KPI; ++i) {
                            const int kr = i * KPI + sub;
                            const int r = __shfl_sync(0xffffffffu, row[g], kr);
                            cp16_or_zero(dst + sw128_offset(g * 32 + kr, ch & 7),
                                         plane + (size_t)(r < 0 ? 0 : r) * p.c.rowb, r >= 0);
                        }
                    cp_async_commit();
                    cp_async_wait<0>();
                    publish(e);
                }
            } else {
                // Codes are copied to a staging tile of the warp, 32 keys at a
                // time, and converted from there; the space of 32 converted
                // keys takes the same keys of the warp's next tile at once.  A
                // lane converts the chunks that it copied itself.
                const uint32_t mine = smem_u32(sC) + lw * (TKEYS * D) + lane * 16;
                int row[4];                                // of the tile being copied
                float ks[4], vs[4], ks_n[4], vs_n[4];      // of the tile in staging, and of the next
                uint32_t ok[4], ok_n[4];
                auto look_up = [&](int x) {
                    if (x >= total) return;
                    resolve(x, row);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        ok_n[g] = __ballot_sync(0xffffffffu, row[g] >= 0);
                        ks_n[g] = vs_n[g] = 0.0f;
                        if ((x & 1) == 0 && row[g] >= 0) {
                            ks_n[g] = ld_nc_early(p.c.ks + row[g]);
                            vs_n[g] = ld_nc_early(p.c.vs + row[g]);
                        }
                    }
                };
                auto load = [&](int x, int g) {
                    if (x < total) {
                        const uint8_t* plane = ((x & 1) ? p.c.v : p.c.k) + head_off;
#pragma unroll
                        for (int i = 0; i < 32 / KPI; ++i) {
                            const int r = __shfl_sync(0xffffffffu, row[g], i * KPI + sub);
                            cp16_or_zero(mine + g * (32 * D) + i * 512,
                                         plane + (size_t)(r < 0 ? 0 : r) * p.c.rowb, r >= 0);
                        }
                    }
                    cp_async_commit();
                };
                look_up(x);
#pragma unroll
                for (int g = 0; g < 4; ++g) load(x, g);
                for (; x < total; x += 3) {
                    const long long e = entry0 + x;
                    if (!wait_slot(e)) { aborted = true; break; }
                    const int ms = (tile_no + (x >> 1)) % MS;
                    const uint32_t dst = smem_u32(sT + (e % STAGES) * S::TILE) + (ch >> 2) * (TKEYS * 128);
#pragma unroll
                    for (int g = 0; g < 4; ++g) { ks[g] = ks_n[g]; vs[g] = vs_n[g]; ok[g] = ok_n[g]; }
                    look_up(x + 3);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        cp_async_wait<3>();
                        if ((x & 1) == 0) {
                            const float lv = log2_above(vs[g]);
                            if (lane == 0) {
                                m_ok[ms * 4 + g] = ok[g];
                                m_lv[ms * 4 + g] = lv;
                            }
                            m_ks[ms * TKEYS + g * 32 + lane] = ks[g];
                            m_vs[ms * TKEYS + g * 32 + lane] = vs[g];
                        }
                        // all of the group's reads come first: stores between
                        // them would hold each up behind the last one's chain
                        uint4 w[32 / KPI];
#pragma unroll
                        for (int i = 0; i < 32 / KPI; ++i)
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                                         : "r"(mine + g * (32 * D) + i * 512)
                                         : "memory");
#pragma unroll
                        for (int i = 0; i < 32 / KPI; ++i) {
                            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                y[2 * k] = e4m3x2_f16x2((uint16_t)(v[k] & 0xFFFFu));
                                y[2 * k + 1] = e4m3x2_f16x2((uint16_t)(v[k] >> 16));
                            }
                            const int r = g * 32 + i * KPI + sub, c0 = 2 * (ch & 3);
                            // the upper 64 values' lanes write their second half
                            // first: the eight lanes of a row cover all banks
                            const int s = ch >> 2;
                            const uint32_t d0 = dst + sw128_offset(r, c0 + s);
                            const uint32_t d1 = dst + sw128_offset(r, c0 + 1 - s);
                            sts16(d0, s ? y[4] : y[0], s ? y[5] : y[1], s ? y[6] : y[2], s ? y[7] : y[3]);
                            sts16(d1, s ? y[0] : y[4], s ? y[1] : y[5], s ? y[2] : y[6], s ? y[3] : y[7]);
                        }
                        load(x + 3, g);
                    }
                    publish(e);
                }
                cp_async_wait<0>();
            }
            entry0 += total;
            tile_no += tz - ta;
        }
        cp_async_wait<0>();
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------- MMA
        // The whole warp walks the steps and one lane issues: descriptors
        // then stay in uniform registers.  (Issued from inside a one-lane
        // branch an MMA took about 140 cycles to issue, twice its own time.)
        const bool leader = elect_one();
        const uint32_t id_s = make_idesc(FP8 ? 0u : 1u, 128, TKEYS);            // Q K^T
        const uint32_t id_o = make_idesc(FP8 ? 0u : 1u, 128, D) | (1u << 16);   // P V: V's N contiguous
        const uint64_t dq = smem_desc_k_sw128(smem_u32(sQ));
        const uint64_t dk = smem_desc_k_sw128(smem_u32(sT)), dv = smem_desc_mn_sw128(smem_u32(sT));
        constexpr uint32_t TILE16 = S::TILE >> 4;      // descriptor addresses count 16 bytes
        // ring positions of the next K and V tiles, and their phases
        uint32_t ks = 0, kph = 0, vs = 1, vph = 0, ms = 0;
        auto next = [](uint32_t& slot, uint32_t& ph) {
            slot += 2;
            if (slot >= STAGES) {
                slot -= STAGES;
                ph ^= 1;
            }
        };
        uint32_t pph[2] = {0, 0};        // phase of the next P, per tile
        uint32_t qph = 0;
        bool aborted = false;
        // S of tile t from the K tile at hand; `last`: no other product needs it
        auto do_s = [&](int t) -> bool {
            if (SPLIT || t == 0) {
                if (!mbar_wait(&full[ks], kph)) return false;
                tc_fence_after();
                if (leader) mbar_arrive(&mfull[ms]);
                ms = (ms + 1) % MS;
            }
            if (leader) {
                const uint64_t a = dq + (SPLIT ? 0 : t * TILE16), b = dk + ks * TILE16;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t off = ((i >> 2) * (TKEYS * 128) + (i & 3) * 32) >> 4;
                    umma_ss<KIND_F16>(tmem + t * 128, a + off, b + off, id_s, i > 0);
                }
                umma_commit(&sfull[t]);
                if (SPLIT || t == 1) umma_commit(&empty[ks]);
            }
            __syncwarp();
            if (SPLIT || t == 1) next(ks, kph);
            return true;
        };
        for (long long u = u_begin; u < u_end && !aborted;) {
            const Item it = find_item<SELECTED>(p, u);
            const int ta = it.tile0 + (int)(u - it.unit0);
            const int tz = it.tile0 + (int)min((long long)it.tiles, u_end - it.unit0);
            u = it.unit0 + (tz - it.tile0);
            if (!it.ok) continue;
            const int n = __shfl_sync(0xffffffffu, tz - ta, 0), H = SPLIT ? n : 2 * n;
            if (!mbar_wait(qfull, qph)) break;
            qph ^= 1;
            tc_fence_after();
            aborted = !do_s(0) || (H > 1 && !do_s(1));
            auto step = [&](int h, int t) -> bool {
                if (!mbar_wait(&pfull[t], pph[t])) return false;
                pph[t] ^= 1;
                if ((SPLIT || t == 0) && !mbar_wait(&full[vs], vph)) return false;
                tc_fence_after();
                if (leader) {
                    const uint64_t b = dv + vs * TILE16;
#pragma unroll
                    for (int i = 0; i < TKEYS / 16; ++i)
                        umma_ts(tmem + 256 + t * 128, tmem + t * 128 + i * 8, b + i * (2048 >> 4), id_o,
                                i > 0 ? 1u : (uint32_t)(h > 1));
                    if (SPLIT || t == 1) umma_commit(&empty[vs]);
                    if (h + 2 >= H) umma_commit(&ofull[t]);
                }
                __syncwarp();
                if (SPLIT || t == 1) next(vs, vph);
                return h + 2 >= H || do_s(t);
            };
            for (int h = 0; h < H && !aborted; h += 2)
                aborted = !step(h, 0) || (h + 1 < H && !step(h + 1, 1));
        }
        if (leader) {
            umma_commit(drain);
            mbar_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------- softmax
        const int t = warp >> 2;
        const int r = (threadIdx.x & 127);                 // row of the tile, TMEM lane
        const int rb = SPLIT ? r : t * 128 + r;            // row of the block
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + 256 + t * 128;
        uint32_t steps = 0, ends = 0;
        int tile_no = 0;
        bool aborted = false;
        for (long long u = u_begin; u < u_end;) {
            const Item it = find_item<SELECTED>(p, u);
            const int ta = it.tile0 + (int)(u - it.unit0);
            const int tz = it.tile0 + (int)min((long long)it.tiles, u_end - it.unit0);
            const bool whole = it.unit0 >= u_begin && it.unit0 + it.tiles <= u_end;
            const int slot = 2 * blockIdx.x + (it.unit0 < u_begin ? 0 : 1);
            u = it.unit0 + (tz - it.tile0);
            if (!it.ok) continue;
            const int n = tz - ta;
            const bool live = rb < it.rows;
            const int rr = it.row0 + rb;
            const size_t head = live ? (size_t)(it.first + rr / p.G) * p.Hq + it.h * p.G + rr % p.G : 0;
            const int lim = live ? it.pos0 + rr / p.G : -1;
            const int lim_lo = it.pos0 + it.row0 / p.G;
            const int lim_hi = it.pos0 + (it.row0 + it.rows - 1) / p.G;

            // ---- this thread's query row into the swizzled tile (for e4m3
            // as halves, divided by the power of two under its largest value)
            float c = p.scale_log2;
            if (!SPLIT || t == 0) {
                const uint4* src = reinterpret_cast<const uint4*>(p.q + head * D);
                const uint32_t dst = smem_u32(sQ) + t * S::TILE;
                float down = 1.0f;
                if constexpr (FP8) {
                    float amax = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 x = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                                     fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
                    }
                    const uint32_t e = __float_as_uint(amax) & 0x7F800000u;
                    if (e > 0x01000000u && e < 0x7E000000u) {
                        c *= __uint_as_float(e);
                        down = __uint_as_float(0x7F000000u - e);
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint4 x = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                    if constexpr (FP8) {
                        uint32_t* w[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *w[k] = f16x2(__uint_as_float(*w[k] << 16) * down,
                                          __uint_as_float(*w[k] & 0xFFFF0000u) * down);
                    }
                    sts16(dst + (i >> 3) * (TKEYS * 128) + sw128_offset(r, i & 7), x.x, x.y, x.z, x.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
            } else if constexpr (FP8) {
                // the odd tiles' threads need the row's factor only
                float amax = 0.0f;
                const uint4* src = reinterpret_cast<const uint4*>(p.q + head * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 x = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                                 fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
                }
                const uint32_t e = __float_as_uint(amax) & 0x7F800000u;
                if (e > 0x01000000u && e < 0x7E000000u) c *= __uint_as_float(e);
            }

            float m = -INFINITY, l = 0.0f;
            bool begun = false;                            // O holds sums
            for (int j = SPLIT ? t : 0; j < n; j += SPLIT ? 2 : 1) {
                const int ms = (tile_no + j) % MS;
                const uint32_t mph = (uint32_t)(((tile_no + j) / MS) & 1);
                if (!aborted) {
                    const bool got = mbar_wait(&sfull[t], steps & 1) && mbar_wait(&mfull[ms], mph);
                    if (!__all_sync(0xffffffffu, got)) aborted = true;
                }
                ++steps;
                if (aborted) continue;
                tc_fence_after();
                float s[TKEYS];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(tS + i * 32, s + i * 32);
                const uint4 okv = *reinterpret_cast<const uint4*>(m_ok + ms * 4);
                tmem_ld_wait();
                if constexpr (FP8) {
                    const float4* ks = reinterpret_cast<const float4*>(m_ks + ms * TKEYS);
#pragma unroll
                    for (int i = 0; i < TKEYS / 4; ++i) {
                        const float4 x = ks[i];
                        s[4 * i] *= x.x; s[4 * i + 1] *= x.y; s[4 * i + 2] *= x.z; s[4 * i + 3] *= x.w;
                    }
                }
                const int key0 = (ta + j) * TKEYS;
                const bool plain = (okv.x & okv.y & okv.z & okv.w) == 0xffffffffu &&
                                   (SELECTED || (key0 + TKEYS - 1 <= lim_lo &&
                                                 (!p.window || key0 > lim_hi - p.window)));
                if (!plain) {
                    const uint32_t ok[4] = {okv.x, okv.y, okv.z, okv.w};
                    // keys from..to of the tile are this row's
                    const int to = SELECTED ? TKEYS - 1 : lim - key0;
                    const int from = !SELECTED && p.window ? lim - p.window + 1 - key0 : 0;
#pragma unroll
                    for (int k = 0; k < TKEYS; ++k) {
                        const bool see = ((ok[k >> 5] >> (k & 31)) & 1) && k <= to && k >= from;
                        s[k] = see ? s[k] : -INFINITY;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k < TKEYS; k += 4) {
                    mx[0] = fmaxf(mx[0], s[k]);
                    mx[1] = fmaxf(mx[1], s[k + 1]);
                    mx[2] = fmaxf(mx[2], s[k + 2]);
                    mx[3] = fmaxf(mx[3], s[k + 3]);
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                if constexpr (FP8) {
                    const float4 lv = *reinterpret_cast<const float4*>(m_lv + ms * 4);
                    top += fmaxf(fmaxf(lv.x, lv.y), fmaxf(lv.z, lv.w));
                }
                // The reference point m may lag behind the maximum by up to
                // 8: weights then reach 2^8, which costs no precision, and
                // the sums in TMEM seldom have to be multiplied.  For e4m3
                // it stands over the weights times the values' scales, so
                // that their product fits f16 whatever the scales; the sums
                // of both are in its units, which cancel in o.
                float f = 1.0f;
                if (top > m + 8.0f) {
                    f = m == -INFINITY ? 0.0f : ex2(m - top);
                    m = top;
                }
                l *= f;
                if (__any_sync(0xffffffffu, f != 1.0f) && begun) {
                    // the product that wrote O was complete before this S was
#pragma unroll 1
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t o[16];
                        asm volatile(
                            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                            : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]),
                              "=r"(o[6]), "=r"(o[7]), "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]),
                              "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                            : "r"(tO + i * 16));
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st16(tO + i * 16, o);
                    }
                }
                begun = true;
                const float z = m == -INFINITY ? 0.0f : -m;
                const uint64_t c2 = pack2(c, c), z2 = pack2(z, z);
                const float4* vs = reinterpret_cast<const float4*>(m_vs + ms * TKEYS);
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float* x = s + i * 32 + k;
                        float e[4];
                        unpack2(ffma2(pack2(x[0], x[1]), c2, z2), e[0], e[1]);
                        unpack2(ffma2(pack2(x[2], x[3]), c2, z2), e[2], e[3]);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            e[y] = ex2(e[y]);
                            sum[y] += e[y];
                        }
                        if constexpr (FP8) {
                            const float4 v = vs[(i * 32 + k) / 4];
                            e[0] *= v.x; e[1] *= v.y; e[2] *= v.z; e[3] *= v.w;
                        }
                        pk[k / 2] = FP8 ? f16x2(e[0], e[1]) : bf16x2(e[0], e[1]);
                        pk[k / 2 + 1] = FP8 ? f16x2(e[2], e[3]) : bf16x2(e[2], e[3]);
                    }
                    tmem_st16(tS + i * 16, pk);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[t]);
            }
            tile_no += n;

            // ---- the item's end: O is complete
            if (n > (SPLIT ? t : 0)) {
                if (!aborted) {
                    const bool got = mbar_wait(&ofull[t], ends & 1);
                    if (!__all_sync(0xffffffffu, got)) aborted = true;
                }
                ++ends;
            }
            tc_fence_after();
            float f0 = 1.0f, f1 = 0.0f;
            float* other = reinterpret_cast<float*>(sQ);       // SPLIT: tile 1's sums, [128][D]
            if constexpr (SPLIT) {
                // the odd tiles' sums go through the query rows' memory, which
                // the last product has left: both halves wait for each other
                __shared__ float ml[2][128];
                named_bar_sync(1, 256);
                if (t == 1) {
                    ml[0][r] = m;
                    ml[1][r] = l;
                    if (begun && !aborted) {
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            float o[32];
                            tmem_ld32(tO + i * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                *reinterpret_cast<float4*>(other + r * D + (((i * 8 + k) ^ (r & 7)) * 4)) =
                                    make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        }
                    }
                }
                named_bar_sync(1, 256);
                if (t == 0) {
                    const float m1 = ml[0][r], l1 = ml[1][r];
                    const float mm = fmaxf(m, m1);
                    const float zz = mm == -INFINITY ? 0.0f : mm;
                    f0 = ex2(m - zz);
                    f1 = n > 1 ? ex2(m1 - zz) : 0.0f;
                    l = l * f0 + (n > 1 ? l1 * f1 : 0.0f);
                    m = mm;
                }
            }
            if ((!SPLIT || t == 0) && !aborted) {
                const bool none = m == -INFINITY && l == 0.0f;
                const float inv = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
                float* part = p.part + (size_t)slot * slot_words(R, D);
#pragma unroll 1
                for (int i = 0; i < D / 32; ++i) {
                    float o[32];
                    tmem_ld32(tO + i * 32, o);
                    tmem_ld_wait();
                    if constexpr (SPLIT) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f0;
                        if (n > 1) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float4 x = *reinterpret_cast<const float4*>(
                                    other + r * D + (((i * 8 + k) ^ (r & 7)) * 4));
                                o[4 * k] += x.x * f1; o[4 * k + 1] += x.y * f1;
                                o[4 * k + 2] += x.z * f1; o[4 * k + 3] += x.w * f1;
                            }
                        }
                    }
                    if (live && whole) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 y;
                            y.x = bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv);
                            y.y = bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv);
                            y.z = bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv);
                            y.w = bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv);
                            *reinterpret_cast<uint4*>(p.o + head * D + i * 32 + k * 8) = y;
                        }
                    } else if (live) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4*>(part + (size_t)rb * D + i * 32 + k * 4) =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                    __syncwarp();
                }
                if (live) {
                    if (!whole) {
                        part[(size_t)R * D + rb] = m;
                        part[(size_t)R * D + R + rb] = l;
                    } else if (p.lse) {
                        p.lse[head] = none ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
                    }
                }
            }
            tc_fence_before();
            if constexpr (SPLIT) named_bar_sync(1, 256);       // the query rows' memory is free again
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool FP8, bool SELECTED, bool SPLIT>
cudaError_t launch_one(const AttendParams& p, cudaStream_t st) {
    auto fn = attend_umma_kernel<D, FP8, SELECTED, SPLIT>;
    constexpr int smem = UmmaShape<D, FP8>::SMEM;
    static_assert(smem <= 227 * 1024 - 1024, "shared memory of a CTA (1 KB of it static)");
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    fn<<<p.ncta, THREADS, smem, st>>>(p);
    return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t launch_type(const AttendParams& p, cudaStream_t st) {
    if (p.idx) return launch_one<D, FP8, true, true>(p, st);
    return p.R == 128 ? launch_one<D, FP8, false, true>(p, st) : launch_one<D, FP8, false, false>(p, st);
}

}  // namespace

cudaError_t launch_attend_umma(const AttendParams& p, cudaStream_t st) {
    if (p.c.D == 128) return p.c.ks ? launch_type<128, true>(p, st) : launch_type<128, false>(p, st);
    return p.c.ks ? launch_type<64, true>(p, st) : launch_type<64, false>(p, st);
}

}  // namespace pivot
