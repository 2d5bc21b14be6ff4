// attend_umma.cu -- attention over a paged key/value cache on the
// 5th-generation tensor cores, for blocks of many query rows a key: chunks
// of new tokens, and selected positions with many query heads a key head.
//
// S = Q K^T and O += P V by tcgen05.mma with the accumulators in TMEM:
// 128 query rows on the M axis (the 128 TMEM lanes), so one thread owns one
// row's softmax and no shuffle is needed; 128 keys a tile.  P goes back to
// TMEM in 16 bits, over the S it came from, and is the A operand of the second
// product: bf16 beside bf16 values, f16 beside e4m3 ones, which are converted
// to f16 with their scales.  Two such tiles are in flight and take turns:
// while one's softmax runs, the tensor cores work on the other.  They are
//  * the two halves of a block of 256 rows, which share every key tile; or
//  * (SPLIT) the even and odd key tiles of one block of up to 128 rows, each
//    with sums of its own that are joined at the end.
//
// TMEM (512 columns): S/P of tile 0, S/P of tile 1, O of tile 0, O of tile 1.
//
// Paged keys come by TMA, a page a box.  Selected keys are copied row by row
// with cp.async (tile::gather4 was measured: about 75 cycles for four 128-byte
// rows, a quarter of what the products take).
//
// Warps 0-15: softmax, four warps a tile and half of its keys.  Warp 16: rows
// and TMA loads.  Warp 17: MMA issue.  Warps 18-21 (selected keys, e4m3
// codes): copies, and codes to halves.
//
// What bounds it: the products.  On one SM a 128 x 128 x 16 product takes 96
// cycles with both operands in shared memory and 75 with P in TMEM (64 would
// be the nominal rate; measured back to back), 103 when the two alternate:
// about 3300 cycles for 256 rows x 128 keys at D = 128.  2048 new tokens over
// 32K (bf16, 32 heads on 8) take 1256 us in turn with other work, 900 TFLOP/s
// at the clock that the power limit leaves (1070 us, 1060 TFLOP/s, in a short
// run; e4m3: 1610): a tile's softmax waits for its S, which waits for its last
// product with V, and only two tiles fit into TMEM to fill the gap.  Selected keys, 64 rows of the 128: 1.7 us a tile in
// bf16 and 2.2 in e4m3, the two streams' round trips, not a unit (without the
// copies 1.75, without the conversions 2.1; warps whose lanes hold no row
// leaving the softmax out gained nothing), and 7 to 11 us an item to fill the
// pipeline.
#include "attend.h"

namespace pivot {

namespace {

constexpr int TKEYS = 128;
constexpr int SOFT_WARPS = 16, LOAD_WARP = 16, MMA_WARP = 17;
constexpr int COPY_WARP = 18, COPY_WARPS = 4;      // e4m3 or selected only

// An mbarrier's count; a write to memory also for the compiler, which may move
// it past the block's first barrier otherwise.
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// f16x2 of weights that may pass the type's range: those of keys without
// values, which meet zeros.
__device__ __forceinline__ uint32_t f16x2_sat(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Whether `v` holds for any of the N threads that meet at named barrier `id`.
template <int N>
__device__ __forceinline__ bool group_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "n"(N)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// A number rounded to 7 significant bits.
__device__ __forceinline__ float seven_bits(float a) {
    const uint32_t u = __float_as_uint(a);
    return __uint_as_float((u + 0xFFFFu + ((u >> 17) & 1u)) & 0xFFFE0000u);
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
__device__ __forceinline__ void tmem_st2(uint32_t taddr, uint32_t a, uint32_t b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t& a, uint32_t& b) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Weights 2^(c s + z) of 32 keys of a row (e4m3: 2^(c s rest + z)): to TMEM in
// 16 bits, and added to the sums.
template <bool FP8>
__device__ __forceinline__ void weights(const float* s, float c, float z, const float* rest, uint32_t to,
                                        uint64_t (&sum)[2]) {
    const uint64_t c2 = pack2(c, c), z2 = pack2(z, z);
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        float e[4];
        uint64_t cr[2] = {c2, c2};
        if constexpr (FP8) {
            const float4 r = *reinterpret_cast<const float4*>(rest + k);
            cr[0] = mul2(c2, pack2(r.x, r.y));
            cr[1] = mul2(c2, pack2(r.z, r.w));
        }
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
            unpack2(ffma2(pack2(s[k + y], s[k + y + 1]), cr[y / 2], z2), e[y], e[y + 1]);
            e[y] = ex2(e[y]);
            e[y + 1] = ex2(e[y + 1]);
            sum[y / 2] = add2(sum[y / 2], pack2(e[y], e[y + 1]));
        }
        pk[k / 2] = FP8 ? f16x2_sat(e[0], e[1]) : bf16x2(e[0], e[1]);
        pk[k / 2 + 1] = FP8 ? f16x2_sat(e[2], e[3]) : bf16x2(e[2], e[3]);
    }
    tmem_st16(to, pk);
}

// Which of a lane's four token rows (those in `ask`) hold no code but 0 in the
// D bytes of one head; each is read as far as it has to be.  Called seldom: out
// of line, for the registers.
template <int D>
__device__ __noinline__ uint32_t keys_without_values(const uint8_t* plane, int rowb, int4 row, uint32_t ask) {
    const int r[4] = {row.x, row.y, row.z, row.w};
    uint32_t c[4], none = 0;
    auto word = [&](int i, int d) {
        return __ldg(reinterpret_cast<const uint32_t*>(plane + (size_t)r[i] * rowb) + d) & 0x7F7F7F7Fu;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = (ask >> i) & 1 ? word(i, 0) : 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll 1
        for (int d = 1; d < D / 4 && c[i] == 0; ++d) c[i] = word(i, d);
        if (c[i] == 0) none |= 1u << i;
    }
    __syncwarp();
    return none;
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

template <int D, bool FP8, bool SELECTED, bool SPLIT>
struct UmmaShape {
    static constexpr int TILE = TKEYS * D * 2;               // K or V tile, and 128 rows of Q
    static constexpr int QTILES = SPLIT ? 1 : 2;
    // ring slots: as many as fit beside Q (and the staging tiles)
    static constexpr int STAGES = D == 64 ? 8 : (FP8 ? 3 : 5) + (SPLIT && (FP8 || !SELECTED) ? 1 : 0);
    static constexpr int WARPS = FP8 || SELECTED ? COPY_WARP + COPY_WARPS : COPY_WARP;
    static constexpr int THREADS = WARPS * 32;
    // registers are per SM sub-partition (16K each; warp w runs on w % 4)
    static constexpr int REGS = WARPS > 20 ? 80 : 96;
    static_assert((WARPS + 3) / 4 * 32 * REGS <= 16384, "register file of a sub-partition");
    // bf16 is loaded into the ring; e4m3 codes into staging tiles, from which
    // they are converted into the ring
    static constexpr int CSTAGES = 3;
    static constexpr int STAGING = FP8 ? CSTAGES * TKEYS * D : 0;
    // per tile: which keys count, and for e4m3 their scales; selected: rows.
    // (A load of m_empty, or of the scales, where m moves instead of at the
    // tile's beginning: mixed chunks 218 -> 228 us.)
    static constexpr int MS = 8;
    static constexpr int META = MS * (16 + (FP8 ? 16 + TKEYS * 12 : 0) + (SELECTED ? TKEYS * 4 : 0));
    static constexpr int SMEM = 1024 + QTILES * TILE + STAGES * TILE + STAGING + META + 1024 + 512 + 2 * 48 + TKEYS;
};

// An item as the rows warp passes it on to the others (48 bytes); n = 0: the end.
struct Work {
    int n, ta, b, h;            // key tiles of this CTA, the first, sequence, key/value head
    int first, pos0, row0, rows;
    int slot, whole, pad[2];    // partial sums' slot; all of the item's tiles are this CTA's
};

template <int D, bool FP8, bool SELECTED, bool SPLIT>
__global__ void __maxnreg__((UmmaShape<D, FP8, SELECTED, SPLIT>::REGS))
    attend_umma_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const AttendParams p) {
    using S = UmmaShape<D, FP8, SELECTED, SPLIT>;
    constexpr int STAGES = S::STAGES, MS = S::MS;
    constexpr int R = SPLIT ? 128 : 256;
    constexpr float LAG = FP8 ? E4M3_LAG : 0.0f, HEAD = FP8 ? 1.0f : -24.0f;
    constexpr float FAR = FP8 ? 512.0f : HUGE_POINT;
    constexpr float UP = 7.0f;                            // e4m3: see the tiles' scales
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sQ = smem;                                   // tiles of 128 rows
    uint8_t* sT = sQ + S::QTILES * S::TILE;               // K and V tiles in turn
    uint8_t* sC = sT + STAGES * S::TILE;                  // e4m3 codes on their way
    uint8_t* sM = sC + S::STAGING;
    uint32_t* m_ok = reinterpret_cast<uint32_t*>(sM);     // [MS][4]
    float* m_lv = reinterpret_cast<float*>(sM + MS * 16); // [MS] log2_above of the scales of V
    float* m_lk = m_lv + MS;                              // [MS] and of K
    float* m_empty = m_lk + MS;                           // [MS] not 0: some key has no scale of V
    float* m_ks = m_lv + MS * 4;                          // [MS][128] scales over those
    float* m_rest = m_ks + MS * TKEYS;                    // [MS][128] what m_ks leaves of a key's scale
    float* m_vs = m_rest + MS * TKEYS;
    int* m_row = reinterpret_cast<int*>(FP8 ? m_vs + MS * TKEYS : m_lv);   // [MS][128] token rows
    uint32_t* m_top = reinterpret_cast<uint32_t*>(sM + S::META);   // [2][128] rows' maxima, as ordered_key
    uint64_t* bars = reinterpret_cast<uint64_t*>(sM + S::META + 1024);
    uint64_t* full = bars;                                // [STAGES] tile there
    uint64_t* empty = full + STAGES;                      // [STAGES] tile read
    uint64_t* mfull = empty + STAGES;                     // [MS] meta there
    uint64_t* mempty = mfull + MS;                        // [MS] meta read
    uint64_t* sfull = mempty + MS;                        // [2] S there
    uint64_t* pfull = sfull + 2;                          // [2][2] half of P there
    uint64_t* ofull = pfull + 4;                          // [2] O complete
    uint64_t* qfull = ofull + 2;                          // Q there
    uint64_t* drain = qfull + 1;
    uint64_t* cfull = drain + 1;                          // [CSTAGES] codes there
    uint64_t* cempty = cfull + S::CSTAGES;                // [CSTAGES] codes converted
    uint64_t* raw = cempty + S::CSTAGES;                  // V tile to be mended there
    uint64_t* ifull = raw + 1;                            // [2] item there
    uint64_t* iempty = ifull + 2;                         // [2] item read
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(iempty + 2);
    Work* m_item = reinterpret_cast<Work*>(sM + S::META + 1024 + 512);     // [2]
    float* m_one = reinterpret_cast<float*>(m_item + 2);  // [32] of 1

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&full[i], FP8 || SELECTED ? COPY_WARPS : 1);
            bar_init(&empty[i], 1);
        }
        for (int i = 0; i < S::CSTAGES; ++i) {
            bar_init(&cfull[i], 1);
            bar_init(&cempty[i], COPY_WARPS);
        }
        for (int i = 0; i < MS; ++i) {
            bar_init(&mfull[i], 1);
            bar_init(&mempty[i], (SPLIT ? 8 : 16) + (FP8 ? COPY_WARPS : 0));
        }
        bar_init(raw, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&ifull[i], 1);
            bar_init(&iempty[i], S::WARPS - 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sfull[i], 1);
            bar_init(&pfull[2 * i], 4);
            bar_init(&pfull[2 * i + 1], 4);
            bar_init(&ofull[i], 1);
        }
        bar_init(qfull, SPLIT ? 8 : 16);
        bar_init(drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == 1) m_one[lane] = 1.0f;
    __syncwarp();
    if (warp == MMA_WARP) {
        tmem_alloc(tmem_at, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    let_next_start();
    if constexpr (!SELECTED) wait_for_previous();
    const long long units = total_units<SELECTED>(p);
    const int ncta = run_count(p, units);
    const bool used = (int)blockIdx.x < ncta;
    const long long u_begin = used ? run_begin(units, blockIdx.x, ncta) : 0;
    const long long u_end = used ? run_begin(units, blockIdx.x + 1, ncta) : 0;

    // The next item, from the rows warp (one descriptor read of dependent loads
    // costs some 5000 cycles); false if it never came.
    uint32_t i_at = 0, i_ph = 0;
    auto next_item = [&](Work& w) -> bool {
        const bool got = __all_sync(0xffffffffu, mbar_wait(&ifull[i_at], i_ph));
        if (!got) return false;
        const int4* from = reinterpret_cast<const int4*>(&m_item[i_at]);
        const int4 a = from[0], b = from[1], c = from[2];
        w.n = a.x; w.ta = a.y; w.b = a.z; w.h = a.w;
        w.first = b.x; w.pos0 = b.y; w.row0 = b.z; w.rows = b.w;
        w.slot = c.x; w.whole = c.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[i_at]);
        if (++i_at == 2) {
            i_at = 0;
            i_ph ^= 1;
        }
        return true;
    };

    if (warp == LOAD_WARP) {
        // ------------------------------------------------------- rows, loads
        // A lane looks after keys 4 lane .. 4 lane + 3 of a tile: their
        // positions are read two tiles ahead, their pages one.  The tile's
        // token rows, scales and which keys count go to shared memory.  Paged:
        // this warp then loads the tile, a page (or 128 keys of it) a TMA box.
        bool aborted = false;
        uint32_t ms = 0, mph = 1;        // next meta slot, and the phase of its release
        uint32_t slot = 0, ph = 1;       // the same of the ring (e4m3: of the staging tiles)
        uint32_t loaded = 0, raws = 0;   // tiles issued so far; loads mended before use
        uint64_t* there = FP8 ? cfull : full;
        uint64_t* read = FP8 ? cempty : empty;
        constexpr uint32_t RING = FP8 ? S::CSTAGES : STAGES;
        const int box = min(TKEYS, p.c.page_size());           // keys of a TMA box
        const int boxes = TKEYS / box;
        if (u_begin == u_end && lane == 0) p.join[blockIdx.x].rows = 0;
        auto pass_on = [&](const Work& w) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&iempty[i_at], i_ph ^ 1))) return false;
            if (lane == 0) {
                int4* to = reinterpret_cast<int4*>(&m_item[i_at]);
                to[0] = make_int4(w.n, w.ta, w.b, w.h);
                to[1] = make_int4(w.first, w.pos0, w.row0, w.rows);
                to[2] = make_int4(w.slot, w.whole, 0, 0);
                mbar_arrive(&ifull[i_at]);
            }
            __syncwarp();
            if (++i_at == 2) {
                i_at = 0;
                i_ph ^= 1;
            }
            return true;
        };
        for (long long u = u_begin; u < u_end && !aborted;) {
            Item it = find_item<SELECTED>(p, u);
            // selected: a key that does not count is replaced by the token's
            // own, so that V holds nothing but finite numbers (copies that may
            // be of no bytes instead cost 5% of chunks over 2048 selected
            // e4m3 keys)
            int spare = 0;
            if (SELECTED && it.ok) {
                const int own = it.pos0 + (it.row0 + it.rows - 1) / p.G;
                spare = p.c.row_of(p.c.table[(size_t)it.b * p.c.max_pages + (own >> p.c.page_log2)], own);
                if (spare < 0) {
                    raise_error(ERRBIT_DATA);
                    it.ok = false;
                }
            }
            const int ta = it.tile0 + (int)(u - it.unit0);
            const int tz = it.tile0 + (int)min((long long)it.tiles, u_end - it.unit0);
            if (u == u_begin && lane == 0) put_join(p, it, units, u_begin, blockIdx.x, ncta);
            u = it.unit0 + (tz - it.tile0);
            if (!it.ok) continue;
            if (!pass_on(Work{tz - ta, ta, it.b, it.h, it.first, it.pos0, it.row0, it.rows,
                              2 * (int)blockIdx.x + (it.unit0 < u_begin ? 0 : 1),
                              it.unit0 >= u_begin && it.unit0 + it.tiles <= u_end, {0, 0}})) {
                aborted = true;
                break;
            }
            const int lim_lo = it.pos0 + it.row0 / p.G;
            const int lim_hi = it.pos0 + (it.row0 + it.rows - 1) / p.G;
            const int key_lo = p.window ? max(0, lim_lo - p.window + 1) : 0;
            const int32_t* sel = SELECTED ? p.idx + (size_t)it.first * p.topk : nullptr;
            const int32_t* pages = p.c.table + (size_t)it.b * p.c.max_pages;
            auto position = [&](int t, int i) -> int {
                const int s = t * TKEYS + 4 * lane + i;
                if (t >= tz) return -1;
                if constexpr (SELECTED) return s < p.topk ? ld_nc_early(sel + s) : -1;
                else return s;
            };
            auto counts = [&](int pos) { return pos >= key_lo && pos <= lim_hi; };
            int pos_a[4], page_a[4], pos_b[4];
            bool ones = false;         // e4m3: some token with values has scale 1
            auto pages_of = [&]() {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    page_a[i] = counts(pos_a[i]) ? ld_nc_early(pages + (pos_a[i] >> p.c.page_log2)) : -1;
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pos_a[i] = position(ta, i);
                pos_b[i] = position(ta + 1, i);
            }
            pages_of();
            for (int t = ta; t < tz && !aborted; ++t) {
                // all waits for loads come before the next loads: one waited
                // for beside younger ones costs their latency too
                int row[4];
                // keys of a lane lie on one page; -1 where one does not count
                const int my_page = max(max(page_a[0], page_a[1]), max(page_a[2], page_a[3]));
                uint32_t ok = 0;
                float ks[4], vs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    row[i] = -1;
                    if (counts(pos_a[i])) {
                        row[i] = p.c.row_of(page_a[i], pos_a[i]);
                        if (row[i] < 0) raise_error(ERRBIT_DATA);
                        if (!PIVOT_CHECK(row[i] < (long long)p.c.num_pages << p.c.page_log2)) row[i] = -1;
                    }
                    ok |= (row[i] >= 0 ? 1u : 0u) << i;
                    pos_a[i] = pos_b[i];
                }
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ks[i] = row[i] >= 0 ? ld_nc_early(p.c.ks + row[i]) : 0.0f;
                        vs[i] = row[i] >= 0 ? ld_nc_early(p.c.vs + row[i]) : 0.0f;
                    }
                }
                pages_of();
#pragma unroll
                for (int i = 0; i < 4; ++i) pos_b[i] = position(t + 2, i);
                const uint32_t mine = ok;
                ok <<= 4 * (lane & 7);                         // eight lanes make a word
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) ok |= __shfl_xor_sync(0xffffffffu, ok, d);
                if (!__all_sync(0xffffffffu, mbar_wait(&mempty[ms], mph))) {
                    aborted = true;
                    break;
                }
                if ((lane & 7) == 0) m_ok[ms * 4 + (lane >> 3)] = ok;
                if constexpr (SELECTED)
                    *reinterpret_cast<int4*>(m_row + ms * TKEYS + 4 * lane) =
                        make_int4(row[0] >= 0 ? row[0] : spare, row[1] >= 0 ? row[1] : spare,
                                  row[2] >= 0 ? row[2] : spare, row[3] >= 0 ? row[3] : spare);
                if constexpr (FP8) {
                    // scales relative to the power of two at or above the
                    // tile's largest, times 2^UP: codes of up to 448 then
                    // use f16 from its top
                    const float lk = log2_above<LOG2_LOW>(fmaxf(fmaxf(fabsf(ks[0]), fabsf(ks[1])),
                                                                fmaxf(fabsf(ks[2]), fabsf(ks[3]))));
                    auto top_v = [&]() {
                        return log2_above<LOG2_LOW_V>(fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])),
                                                        fmaxf(fabsf(vs[2]), fabsf(vs[3]))));
                    };
                    float lv = top_v(), empty = 0.0f;
                    // a token without values (its scale is 1, as an append
                    // stores it): no scale, so that it takes no bits from the
                    // tile's values and the softmax knows it.  Not asked for
                    // where tokens with values have that scale too.
                    if (lv >= 0.0f && !ones) {
                        const uint32_t ask =
                            (vs[0] == 1.0f) | (vs[1] == 1.0f) << 1 | (vs[2] == 1.0f) << 2 | (vs[3] == 1.0f) << 3;
                        if (__any_sync(0xffffffffu, ask)) {
                            const uint32_t none = keys_without_values<D>(
                                p.c.v + it.h * D, p.c.rowb, make_int4(row[0], row[1], row[2], row[3]), ask);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if ((none >> i) & 1) vs[i] = 0.0f;
                            empty = __any_sync(0xffffffffu, none) ? 1.0f : 0.0f;
                            ones = __any_sync(0xffffffffu, ask & ~none);
                            lv = top_v();
                        }
                    }
                    const float dk = exp2_whole(UP - lk), dv = exp2_whole(UP - lv);
                    if (lane == 0) {
                        m_lk[ms] = lk - UP;
                        m_lv[ms] = lv;
                        m_empty[ms] = empty;
                    }
                    // a key's scale in two factors: 7 bits that go into its
                    // halves, exactly (a code has 4), and the rest, within
                    // 2^-7 of 1, for the fp32 scores
                    float h[4], rest[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = ks[i] * dk;
                        h[i] = seven_bits(a);
                        rest[i] = h[i] == 0.0f ? 1.0f : __fdividef(a, h[i]);
                    }
                    *reinterpret_cast<float4*>(m_ks + ms * TKEYS + 4 * lane) = make_float4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<float4*>(m_rest + ms * TKEYS + 4 * lane) =
                        make_float4(rest[0], rest[1], rest[2], rest[3]);
                    *reinterpret_cast<float4*>(m_vs + ms * TKEYS + 4 * lane) =
                        make_float4(vs[0] * dv, vs[1] * dv, vs[2] * dv, vs[3] * dv);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&mfull[ms]);
                if (++ms == MS) {
                    ms = 0;
                    mph ^= 1;
                }
                if constexpr (!SELECTED) {
                    // lane i loads box i (of 64-value half i / boxes); a box
                    // with no key that counts is left out
                    const int part = lane % boxes, half = lane / boxes;
                    constexpr int HALVES = FP8 ? 1 : D / 64;
                    const int from = part * box / 4;           // the lane of the box's first keys
                    const uint32_t any = __ballot_sync(0xffffffffu, mine != 0);
                    const uint32_t its = box == TKEYS ? any : (any >> from) & ((1u << (box / 4)) - 1);
                    const int page = __shfl_sync(0xffffffffu, my_page, its ? from + __ffs(its) - 1 : 0);
                    const int at = (page << p.c.page_log2) + ((t * TKEYS + part * box) & (p.c.page_size() - 1));
                    const bool go = half < HALVES && its != 0;
                    const uint32_t bytes =
                        __popc(__ballot_sync(0xffffffffu, go)) * box * (FP8 ? D : 128);
                    const bool every = __all_sync(0xffffffffu, mine == 15u);
#pragma unroll
                    for (int kv = 0; kv < 2 && !aborted; ++kv) {
                        if (!__all_sync(0xffffffffu, mbar_wait(&read[slot], ph))) {
                            aborted = true;
                            break;
                        }
                        // bf16 values of keys that do not count are zeroed
                        // before use (e4m3: by the converting warps)
                        const bool mend = !FP8 && kv && !every;
                        uint64_t* bar = mend ? raw : &there[slot];
                        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                        __syncwarp();
                        if (go) {
                            if constexpr (FP8)
                                tma_load_2d(sC + slot * (TKEYS * D) + part * box * D, kv ? &tmap_v : &tmap_k, bar,
                                            it.h * D, at);
                            else
                                tma_load_2d(sT + slot * S::TILE + half * (TKEYS * 128) + part * box * 128,
                                            kv ? &tmap_v : &tmap_k, bar, it.h * D + half * 64, at);
                        }
                        if (mend) {
                            if (!__all_sync(0xffffffffu, mbar_wait(raw, raws & 1))) aborted = true;
                            ++raws;
                            const uint32_t base = smem_u32(sT + slot * S::TILE);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((mine >> i) & 1) continue;
                                const int k = 4 * lane + i;
                                for (int c = 0; c < D / 8; ++c)
                                    sts16(base + (c >> 3) * (TKEYS * 128) + k * 128 + (c & 7) * 16, 0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&full[slot]);
                        }
                        ++loaded;
                        if (++slot == RING) {
                            slot = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
        }
        if (!aborted) pass_on(Work{});
        // every load has landed before the CTA may end
        for (uint32_t i = 0; i < RING && i < loaded; ++i) {
            const uint32_t e = loaded - 1 - i;
            mbar_wait(&there[e % RING], (e / RING) & 1);
        }
    } else if (warp >= COPY_WARP) {
        // ------------------- selected keys; e4m3 codes to halves (exact)
        // Four warps, 32 keys of each tile each.  Selected keys are copied
        // row by row: bf16 into the ring, codes into the staging tiles.
        if constexpr (FP8 || SELECTED) {
            constexpr int KEYS = TKEYS / COPY_WARPS;           // of a warp
            const int key_w = (warp - COPY_WARP) * KEYS;
            bool aborted = false;
            uint32_t ms = 0, mph = 0;              // meta of the next tile to copy (or convert)
            uint32_t cs = 0, cph = 0, cms = 0;     // staging tile to convert, and its meta
            uint32_t slot = 0, ph = 1;             // ring slot to fill
            uint32_t out = 0;                      // and to publish
            const int es = FP8 ? 1 : 2;
            // e4m3: eight neighbouring lanes take four chunks of two keys
            // whose numbers differ in bits 0 and 2 (D = 64: in bit 0): their
            // reads of codes and writes of halves fall on different banks
            constexpr int CH = D * (FP8 ? 1 : 2) / 16;         // 16-byte chunks of a stored row
            constexpr int KPI = 32 / CH;                       // keys an instruction
            const int ch = !FP8 ? lane % CH : (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0);
            auto key_of = [&](int j) -> int {                  // of instruction j
                if constexpr (FP8 && D == 128) {
                    const int q = (lane >> 2) & 3;
                    return key_w + (j >> 1) * 8 + (((j & 1) * 2 + (q >> 1)) ^ ((q & 1) * 5));
                } else if constexpr (FP8) {
                    return key_w + j * 8 + (lane >> 2);
                } else {
                    return key_w + j * KPI + lane / CH;
                }
            };
            auto code_at = [&](uint32_t stage, int k) -> uint32_t {
                return smem_u32(sC) + stage * (TKEYS * D) +
                       (D == 128 ? k * 128 + ((ch ^ (k & 7)) << 4) : k * 64 + ch * 16);
            };
            auto advance = [](uint32_t& at, uint32_t& phase, uint32_t n) {
                if (++at == n) {
                    at = 0;
                    phase ^= 1;
                }
            };
            Work it;
            while (!aborted && next_item(it) && it.n > 0) {
                const int total = 2 * it.n;                    // K and V tiles of the item
                const size_t head_off = (size_t)it.h * D * es + ch * 16;
                // copies of tile x (K if even) towards shared memory at dst(k)
                auto copy = [&](int x, auto dst) -> bool {
                    if ((x & 1) == 0 && !__all_sync(0xffffffffu, mbar_wait(&mfull[ms], mph))) return false;
                    const uint8_t* plane = ((x & 1) ? p.c.v : p.c.k) + head_off;
#pragma unroll
                    for (int j = 0; j < KEYS / KPI; ++j) {
                        const int k = key_of(j);
                        cp_async16(dst(k), plane + (size_t)m_row[ms * TKEYS + k] * p.c.rowb);
                    }
                    if (x & 1) advance(ms, mph, MS);
                    return true;
                };
                auto publish = [&](uint32_t at) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[at]);
                };
                if constexpr (!FP8) {
                    // Tiles in flight.  The slot of a tile is released once
                    // the tile after it is published at the latest, so the
                    // slot waited for needs all but the STAGES - 2 tiles
                    // before it published.
                    constexpr int PENDING = STAGES - 3 < 3 ? STAGES - 3 : 3;
                    auto publish_next = [&]() {
                        publish(out);
                        if (++out == STAGES) out = 0;
                    };
                    int x = 0;
                    for (; x < total && !aborted; ++x) {
                        if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ph))) aborted = true;
                        const uint32_t base = smem_u32(sT) + slot * S::TILE + (ch >> 3) * (TKEYS * 128);
                        if (!aborted && !copy(x, [&](int k) { return base + sw128_offset(k, ch & 7); }))
                            aborted = true;
                        cp_async_commit();
                        advance(slot, ph, STAGES);
                        if (x >= PENDING) {
                            cp_async_wait<PENDING>();
                            publish_next();
                        }
                    }
                    cp_async_wait<0>();
                    for (int y = min(x, PENDING); y > 0; --y) publish_next();
                } else {
                    // staging tiles are filled two ahead (selected: by these
                    // warps themselves, each its own keys)
                    uint32_t fs = cs;                          // staging tile to fill
                    auto fill = [&](int x) {
                        if (SELECTED && x < total && !aborted) {
                            if (!copy(x, [&](int k) { return code_at(fs, k); })) aborted = true;
                            if (++fs == S::CSTAGES) fs = 0;
                        }
                        if (SELECTED) cp_async_commit();
                    };
                    fill(0);
                    fill(1);
                    for (int x = 0; x < total; ++x) {
                        if constexpr (SELECTED) {
                            cp_async_wait<1>();
                            __syncwarp();
                        }
                        const bool got = (SELECTED || mbar_wait(&cfull[cs], cph)) && mbar_wait(&empty[slot], ph);
                        if (!__all_sync(0xffffffffu, got && !aborted)) {
                            aborted = true;
                            break;
                        }
                        uint32_t ok = 0xffffffffu;
                        if constexpr (!SELECTED) {             // values that do not count: 0
                            if (x & 1) ok = m_ok[cms * 4 + (key_w >> 5)];
                        }
                        const bool every = ok == 0xffffffffu;
                        const uint32_t dst = smem_u32(sT) + slot * S::TILE + (ch >> 2) * (TKEYS * 128);
                        constexpr int BATCH = KEYS / KPI;      // reads before the writes
#pragma unroll
                        for (int j0 = 0; j0 < KEYS / KPI; j0 += BATCH) {
                            uint4 c[BATCH];
#pragma unroll
                            for (int j = 0; j < BATCH; ++j)
                                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(c[j].x), "=r"(c[j].y), "=r"(c[j].z), "=r"(c[j].w)
                                             : "r"(code_at(cs, key_of(j0 + j)))
                                             : "memory");
                            if (!every) {
#pragma unroll
                                for (int j = 0; j < BATCH; ++j) {
                                    if (!((ok >> (key_of(j0 + j) - key_w)) & 1)) c[j] = make_uint4(0, 0, 0, 0);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < BATCH; ++j) {
                                const uint32_t v[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
                                const int k = key_of(j0 + j), c0 = 2 * (ch & 3);
                                uint32_t y[8];
                                // times the key's 7 bits: exact; times the
                                // value's 11: two errors of up to 2^-12
                                const float m = ((x & 1) ? m_vs : m_ks)[cms * TKEYS + k];
                                const uint32_t m2 = f16x2(m, m);
#pragma unroll
                                for (int n = 0; n < 4; ++n) {
                                    y[2 * n] = mul_f16x2(e4m3x2_f16x2((uint16_t)(v[n] & 0xFFFFu)), m2);
                                    y[2 * n + 1] = mul_f16x2(e4m3x2_f16x2((uint16_t)(v[n] >> 16)), m2);
                                }
                                sts16(dst + sw128_offset(k, c0), y[0], y[1], y[2], y[3]);
                                sts16(dst + sw128_offset(k, c0 + 1), y[4], y[5], y[6], y[7]);
                            }
                        }
                        if (x & 1) {                           // the tile's scales are read
                            if (lane == 0) mbar_arrive(&mempty[cms]);
                            if (++cms == MS) cms = 0;
                        }
                        publish(slot);
                        if (!SELECTED && lane == 0) mbar_arrive(&cempty[cs]);
                        advance(cs, cph, S::CSTAGES);
                        advance(slot, ph, STAGES);
                        fill(x + 2);
                    }
                }
            }
            cp_async_wait<0>();
        }
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
        uint32_t ks = 0, kph = 0, vs = 1, vph = 0;
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
        Work it;
        while (!aborted && next_item(it) && it.n > 0) {
            const int n = __shfl_sync(0xffffffffu, it.n, 0), H = SPLIT ? n : 2 * n;
            if (!mbar_wait(qfull, qph)) break;
            qph ^= 1;
            tc_fence_after();
            aborted = !do_s(0) || (H > 1 && !do_s(1));
            auto step = [&](int h, int t) -> bool {
                if ((SPLIT || t == 0) && !mbar_wait(&full[vs], vph)) return false;
                const uint64_t b = dv + vs * TILE16;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!mbar_wait(&pfull[2 * t + half], pph[t])) return false;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int i = 4 * half; i < 4 * half + 4; ++i)
                            umma_ts(tmem + 256 + t * 128, tmem + t * 128 + half * 64 + (i & 3) * 8, b + i * (2048 >> 4),
                                    id_o, i > 0 ? 1u : (uint32_t)(h > 1));
                    }
                    __syncwarp();
                }
                pph[t] ^= 1;
                if (leader) {
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
        // Stream t = tile of rows (or parity of the key tiles); two warps a
        // TMEM lane quarter, x = 0, 1: keys 64 x .. of every tile, of the
        // same rows.  Both weigh from one reference point m.
        const int t = (warp >> 2) & 1, x = warp >> 3;
        const int r = (warp & 3) * 32 + lane;              // row of the tile, TMEM lane
        const int rb = SPLIT ? r : t * 128 + r;            // row of the block
        const int pair = 1 + t * 4 + (warp & 3);           // named barrier of the two warps
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + 256;
        uint32_t sph = 0, oph[2] = {0, 0};
        int tile_no = 0;
        bool aborted = false;
        // All warps of a stream (split: of both) go on or stop together, since
        // they meet at named barriers.
        Work it;
        auto fetch = [&]() -> bool {
            const bool lost = !next_item(it);
            if (SPLIT ? group_any<SOFT_WARPS * 32>(9, lost) : group_any<64>(pair, lost)) return false;
            return it.n > 0;
        };
        // this thread's half of its query row (e4m3: and the row's largest
        // value) is read while the item before ends
        uint4 qh[D / 16];
        float amax = 0.0f;
        auto read_q = [&]() {
            const int rr = it.row0 + rb;
            const bool live = rb < it.rows;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + (live ? (size_t)(it.first + rr / p.G) * p.Hq + it.h * p.G + rr % p.G : 0) * D);
            amax = 0.0f;
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 q = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                                 fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
                }
            }
            if (!SPLIT || t == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    qh[k] = live ? __ldg(src + x * (D / 16) + k) : make_uint4(0, 0, 0, 0);
            }
        };
        bool more = fetch();
        if (more) read_q();
        while (more) {
            const int n = it.n, ta = it.ta, slot = it.slot;
            const bool whole = it.whole != 0, live = rb < it.rows;
            const int rr = it.row0 + rb;
            const size_t head = live ? (size_t)(it.first + rr / p.G) * p.Hq + it.h * p.G + rr % p.G : 0;
            const int lim = live ? it.pos0 + rr / p.G : -1;
            const int lim_lo = it.pos0 + it.row0 / p.G;
            const int lim_hi = it.pos0 + (it.row0 + it.rows - 1) / p.G;

            // ---- this thread's half of its query row into the swizzled tile
            // (for e4m3 as halves, divided by the power of two under the
            // row's largest value)
            float c = p.scale_log2;
            {
                float down = 1.0f;
                if constexpr (FP8) {
                    const uint32_t e =
                        min(max(__float_as_uint(amax) & 0x7F800000u, 0x01000000u), 0x7D800000u);
                    c *= __uint_as_float(e);
                    down = __uint_as_float(0x7F000000u - e);
                }
                if (!SPLIT || t == 0) {
                    const uint32_t dst = smem_u32(sQ) + (SPLIT ? 0 : t * S::TILE);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int i = x * (D / 16) + k;
                        uint32_t w[4] = {qh[k].x, qh[k].y, qh[k].z, qh[k].w};
                        if constexpr (FP8) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = f16x2(__uint_as_float(w[y] << 16) * down,
                                             __uint_as_float(w[y] & 0xFFFF0000u) * down);
                        }
                        sts16(dst + (i >> 3) * (TKEYS * 128) + sw128_offset(r, i & 7), w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qfull);
                }
            }

            float m = -INFINITY, l = 0.0f;                 // l: of this thread's keys
            if (x == 0) m_top[t * 128 + r] = 0;            // below every number; read after a barrier
            bool begun = false;                            // O holds sums
            bool far = false;                              // |m| > FAR in some row of the warp
            for (int j = SPLIT ? t : 0; j < n; j += SPLIT ? 2 : 1) {
                const int ms = (tile_no + j) % MS;
                if (!aborted) {
                    const uint32_t mph = (uint32_t)(((tile_no + j) / MS) & 1);
                    const bool got = mbar_wait(&sfull[t], sph) && mbar_wait(&mfull[ms], mph);
                    if (!__all_sync(0xffffffffu, got)) aborted = true;
                }
                sph ^= 1;
                // e4m3: factor of the tile's scores, and log2 of its values'.
                // Scores are below 2^32 here: a smaller factor is as good as
                // 2^-120, and 0 would make NaN of the masked ones' -inf.
                const float ct = FP8 ? fminf(fmaxf(c * exp2_whole(m_lk[ms]), 0x1p-120f), 0x1p120f) : c,
                            lv = FP8 ? m_lv[ms] : 0.0f;
                const bool empty = FP8 && m_empty[ms] != 0.0f;
                const uint2 ok = *reinterpret_cast<const uint2*>(m_ok + ms * 4 + 2 * x);
                const int key0 = (ta + j) * TKEYS + 64 * x;
                const bool plain = (ok.x & ok.y) == 0xffffffffu &&
                                   (SELECTED || (key0 + 63 <= lim_lo && (!p.window || key0 > lim_hi - p.window)));
                // which of 32 keys count for this row
                auto seen = [&](int i) -> uint32_t {
                    if (plain) return 0xffffffffu;
                    // keys from..to of these 64 are this row's
                    const int to = SELECTED ? 63 : lim - key0;
                    const int from = !SELECTED && p.window ? lim - p.window + 1 - key0 : 0;
                    const int a = min(max(from - 32 * i, 0), 32), z = min(max(to - 32 * i + 1, 0), 32);
                    const uint32_t below = z == 32 ? 0xffffffffu : (1u << z) - 1;
                    const uint32_t above = a == 32 ? 0u : 0xffffffffu << a;
                    return (i ? ok.y : ok.x) & below & above;
                };
                // the scores of keys that do not count
                auto finish = [&](float* s, int i) {
                    if (!plain) {
                        const uint32_t see = seen(i);
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1 ? s[k] : -INFINITY;
                    }
                };
                auto largest = [](const float* s, float (&mx)[4]) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[k + y], s[k + 4 + y]);
                };
                // The maximum may grow under the reference point m, so that m
                // and the sums in TMEM seldom have to move (2048 new tokens
                // over 32K, bf16: 1147 us with room for 2^8, 1088 for 2^24 or
                // 2^64).  bf16 weights have the exponents of fp32: a move puts
                // the largest at 2^-24 and none passes 1, so sums of weight
                // times value stay as small as the values.  For f16 weights
                // see E4M3_LAG: m stands over weight times the tile's lv, and
                // a move puts the largest at 2, not higher (2^10: 295 -> 375
                // us for chunks over 2048 selected keys, for m moves more).
                float top = -INFINITY;
                if (!aborted) {
                    float a[32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        tmem_ld32(tS + 64 * x + 32 * i, a);
                        tmem_ld_wait();
                        finish(a, i);
                        largest(a, mx);
                    }
                    top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * ct + lv;
                    // e4m3: without the rest of the scales, up to 2^-7 off
                    if (FP8 && top > -INFINITY) top += fabsf(top - lv) * 0.0078125f;
                }
                const float* rest = m_rest + ms * TKEYS + 64 * x;
                if (group_any<64>(pair, top - m > LAG)) {
                    if constexpr (FP8) {
                        const float* vs = m_vs + ms * TKEYS + 64 * x;
                        if (__any_sync(0xffffffffu, empty || (fabsf(top) > FAR && top > -INFINITY)) && !aborted) {
                            // with the rest of the scales; keys without values
                            // (scale 0) EMPTY_BELOW below what l or, lv > 0,
                            // their weight here takes
                            const float below = EMPTY_BELOW + fminf(lv, 0.0f);
                            top = -INFINITY;
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) {
                                uint32_t b[8];
                                tmem_ld8(tS + 64 * x + 8 * i, b);
                                tmem_ld_wait();
                                const uint32_t see = seen(i >> 2) >> (8 * (i & 3));
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if ((see >> k) & 1) {
                                        const float a = __fadd_rn(
                                            __fmul_rn(__uint_as_float(b[k]), __fmul_rn(ct, rest[8 * i + k])), lv);
                                        top = fmaxf(top, vs[8 * i + k] != 0.0f ? a : a - below);
                                    }
                            }
                        }
                    }
                    atomicMax(&m_top[t * 128 + r], ordered_key(top));
                    named_bar_sync(pair, 64);
                    top = key_to_float(m_top[t * 128 + r]);
                    float f = 1.0f;
                    if (top - m > LAG) {
                        const float to = point_at(m, top, HEAD);
                        f = m == -INFINITY ? 0.0f : ex2(m - to);
                        m = to;
                    }
                    l *= f;
                    far = __any_sync(0xffffffffu, fabsf(m) > FAR && m > -INFINITY);
                    // the product that wrote O was complete before this S was;
                    // each warp takes half of the values
                    if (begun && !aborted) {
#pragma unroll 1
                        for (int i = x * (D / 32); i < (x + 1) * (D / 32); ++i) {
                            uint32_t o[16];
                            tmem_ld16(tO + t * 128 + i * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(tO + t * 128 + i * 16, o);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    named_bar_sync(pair, 64);      // all of the row's sums have moved
                }
                if (aborted) continue;
                // Beside a reference point that fp32 holds no longer to a small
                // part of 1 (e4m3: where 2^-7 of it, for the rest of the
                // scales, is not small) the scores are rounded as its were
                // before it is subtracted: the largest weight is about 1
                // however large they are.
                if (far) {
                    const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b[16];
                        tmem_ld16(tS + 64 * x + 16 * i, b);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float f = FP8 ? __fmul_rn(ct, rest[16 * i + k]) : ct;
                            b[k] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(b[k]), f), lv) - m0);
                        }
                        tmem_st16(tS + 64 * x + 16 * i, b);
                    }
                    tmem_st_wait();
                }
                const float z = far || m == -INFINITY ? 0.0f : lv - m, cw = far ? 1.0f : ct;
                begun = true;
                // P takes the place of these 64 keys' S, half of it at a time:
                // the scores are read again, for all 64 would not fit in the
                // registers beside the rest
                {
                    uint64_t sum[2] = {0ull, 0ull};
                    float a[32];
                    tmem_ld32(tS + 64 * x, a);
                    tmem_ld_wait();
                    finish(a, 0);
                    weights<FP8>(a, cw, z, far ? m_one : rest, tS + 64 * x, sum);
                    tmem_ld32(tS + 64 * x + 32, a);
                    tmem_ld_wait();
                    finish(a, 1);
                    weights<FP8>(a, cw, z, far ? m_one : rest + 32, tS + 64 * x + 16, sum);
                    float s0, s1, s2, s3;
                    unpack2(sum[0], s0, s1);
                    unpack2(sum[1], s2, s3);
                    l += ((s0 + s1) + (s2 + s3)) * (FP8 ? exp2_whole(-lv) : 1.0f);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&pfull[2 * t + x]);
                    mbar_arrive(&mempty[ms]);
                }
            }
            tile_no += n;

            // ---- the item's end
            more = fetch();
            if (more) read_q();
            if (!aborted) {
                bool got = true;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if ((SPLIT || y == t) && n > (SPLIT ? y : 0)) {
                        got = got && mbar_wait(&ofull[y], oph[y]);
                        oph[y] ^= 1;
                    }
                }
                if (!__all_sync(0xffffffffu, got)) aborted = true;
            }
            // Columns of S that P leaves free carry the statistics from warp
            // to warp (TMEM lanes belong to warps by their number modulo 4).
            // Split key tiles: four warps a row join the two streams' sums, a
            // quarter of the values each.
            if (!aborted) {
                tc_fence_after();
                tmem_st2(tS + 32 + 2 * x, __float_as_uint(m), __float_as_uint(l));
                tmem_st_wait();
            }
            tc_fence_before();
            if constexpr (SPLIT) named_bar_sync(9, SOFT_WARPS * 32);
            else named_bar_sync(pair, 64);
            tc_fence_after();
            if (!aborted) {
                float f0 = 1.0f, f1 = 0.0f;                // of the streams' sums
                if constexpr (SPLIT) {
                    uint32_t sm[2], sl[2], y;
                    float ls[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tmem_ld2(tmem + lane_off + k * 128 + 32, sm[k], sl[0]);
                        tmem_ld2(tmem + lane_off + k * 128 + 34, y, sl[1]);
                        tmem_ld_wait();
                        ls[k] = __uint_as_float(sl[0]) + __uint_as_float(sl[1]);
                    }
                    const float m0 = __uint_as_float(sm[0]), m1 = __uint_as_float(sm[1]);
                    m = fmaxf(m0, m1);                     // a stream without keys: -inf, 0
                    const float zz = m == -INFINITY ? 0.0f : m;
                    f0 = ex2(m0 - zz);
                    f1 = ex2(m1 - zz);
                    l = ls[0] * f0 + ls[1] * f1;
                } else {
                    uint32_t om, ol;
                    tmem_ld2(tS + 32 + 2 * (x ^ 1), om, ol);
                    tmem_ld_wait();
                    l += __uint_as_float(ol);
                }
                const bool none = m == -INFINITY && l == 0.0f;
                const float inv = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
                constexpr int PARTS = SPLIT ? D / 64 : D / 32;     // 16 values each
                const int first = (SPLIT ? 2 * t + x : x) * PARTS;
                float* part = p.part + (size_t)slot * slot_words(R, D);
                f0 *= FP8 ? inv * exp2_whole(-UP) : inv;
                f1 *= FP8 ? inv * exp2_whole(-UP) : inv;
#pragma unroll
                for (int i = first; i < first + PARTS; ++i) {
                    float o[16];
                    tmem_ld16(tO + (SPLIT ? 0 : t * 128) + i * 16, reinterpret_cast<uint32_t*>(o));
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= f0;
                    if constexpr (SPLIT) {
                        if (n > 1) {
                            float o1[16];
                            tmem_ld16(tO + 128 + i * 16, reinterpret_cast<uint32_t*>(o1));
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = fmaf(o1[k], f1, o[k]);
                        }
                    }
                    if (live && whole) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint4 y;
                            y.x = bf16x2(o[8 * k], o[8 * k + 1]);
                            y.y = bf16x2(o[8 * k + 2], o[8 * k + 3]);
                            y.z = bf16x2(o[8 * k + 4], o[8 * k + 5]);
                            y.w = bf16x2(o[8 * k + 6], o[8 * k + 7]);
                            *reinterpret_cast<uint4*>(p.o + head * D + i * 16 + k * 8) = y;
                        }
                    } else if (live && PIVOT_CHECK(slot < 2 * p.ncta)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<float4*>(part + (size_t)rb * D + i * 16 + k * 4) =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                    __syncwarp();
                }
                if (live && x == 0 && (!SPLIT || t == 0)) {
                    if (!whole && PIVOT_CHECK(slot < 2 * p.ncta)) {
                        part[(size_t)R * D + rb] = m;
                        part[(size_t)R * D + R + rb] = l;
                    } else if (whole && p.lse) {
                        p.lse[head] = none ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
                    }
                }
            }
            tc_fence_before();
            // all statistics are read (and, split, all sums and Q)
            if constexpr (SPLIT) named_bar_sync(9, SOFT_WARPS * 32);
            else named_bar_sync(pair, 64);
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
cudaError_t launch_one(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t st) {
    auto fn = attend_umma_kernel<D, FP8, SELECTED, SPLIT>;
    constexpr int smem = UmmaShape<D, FP8, SELECTED, SPLIT>::SMEM;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static bool done[64] = {false};
    const cudaError_t e = allow_smem(fn, smem, done);
    if (e != cudaSuccess) return e;
    return launch(!SELECTED, fn, p.ncta, UmmaShape<D, FP8, SELECTED, SPLIT>::THREADS, smem, st, tk, tv, p);
}

template <int D, bool FP8>
cudaError_t launch_type(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t st) {
    if (p.idx) return launch_one<D, FP8, true, true>(tk, tv, p, st);
    return p.R == 128 ? launch_one<D, FP8, false, true>(tk, tv, p, st)
                      : launch_one<D, FP8, false, false>(tk, tv, p, st);
}

}  // namespace

cudaError_t launch_attend_umma(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p,
                               cudaStream_t st) {
    if (p.c.D == 128)
        return p.c.ks ? launch_type<128, true>(tk, tv, p, st) : launch_type<128, false>(tk, tv, p, st);
    return p.c.ks ? launch_type<64, true>(tk, tv, p, st) : launch_type<64, false>(tk, tv, p, st);
}

}  // namespace pivot
