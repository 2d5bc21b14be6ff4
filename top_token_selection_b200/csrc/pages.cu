// pages.cu -- the pages of a paged key/value cache: appending new tokens,
// forking, cutting, copying and compacting.
//
// The state (table, lengths, reference counts) is kept on the device by
// integer operations whose result does not depend on their order, so equal
// calls leave equal states.  All of it is bound by memory: the bookkeeping
// by latency (a few kilobytes, so as few launches and passes as possible: one
// block plans, a second kernel moves), the copies by bandwidth.  Measured, at
// 6.54 TB/s for a plain copy: an append of 17K bf16 tokens with shared pages
// 41 us (155 MB, 24 us at that rate), a compaction that moves half of a large
// pool 232 us (1.25 GB, 192 us).
#include "pages.h"

namespace pivot {

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PIECE = 16384;          // bytes one block copies at a time: 256 threads x 4 x 16

// Workspace of an append: the verdict, then per sequence its length before
// the call, the shared page it copies (-1: none) and its first index into
// the list of pages taken, then that list.
struct AppendWs {
    int32_t *head, *len0, *cow, *off, *list;
    __host__ __device__ AppendWs(int32_t* ws, int B)
        : head(ws), len0(ws + 4), cow(len0 + B), off(cow + B), list(off + B) {}
};

// Ids of the lowest `want` free pages (refs 0), ascending, to list; returns
// how many there are, up to want.  Whole block; each round reads 16 counts a
// thread.  room: entries of list.
__device__ int lowest_free(const int32_t* refs, int num_pages, int want, int32_t* list, int room, int* tmp) {
    constexpr int PER = 16;
    int found = 0;
    for (int base = 0; base < num_pages && found < want; base += PLAN_THREADS * PER) {
        const int at = base + threadIdx.x * PER;
        unsigned free_bits = 0;
        if (at + PER <= num_pages && ((reinterpret_cast<uintptr_t>(refs) & 15) == 0)) {
            const int4* r4 = reinterpret_cast<const int4*>(refs + at);
            int4 v[PER / 4];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) v[i] = r4[i];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
                free_bits |= (unsigned)(v[i].x == 0) << (4 * i);
                free_bits |= (unsigned)(v[i].y == 0) << (4 * i + 1);
                free_bits |= (unsigned)(v[i].z == 0) << (4 * i + 2);
                free_bits |= (unsigned)(v[i].w == 0) << (4 * i + 3);
            }
        } else {
            for (int i = 0; i < PER; ++i)
                if (at + i < num_pages && refs[at + i] == 0) free_bits |= 1u << i;
        }
        int tot;
        int rank = found + block_exclusive(__popc(free_bits), tmp, tot);
        while (free_bits && rank < want) {
            const int i = __ffs(free_bits) - 1;
            free_bits &= free_bits - 1;
            if (PIVOT_CHECK(rank < room)) list[rank] = at + i;
            ++rank;
        }
        found += tot;
    }
    return found < want ? found : want;
}

// One block: checks the batch, counts the pages each sequence needs, takes
// the lowest free ones and enters them.  Nothing is changed before all of it
// is known to fit.
__global__ void __launch_bounds__(PLAN_THREADS)
    append_plan_kernel(const CacheView c, const int32_t* cu, int total, int max_new, int32_t* lack,
                       int32_t* ws) {
    __shared__ int tmp[33];
    const AppendWs w(ws, c.B);
    const int P = c.page_size();
    int carry = 0;
    bool bad = false;
    for (int b0 = 0; b0 < c.B; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        int need = 0;
        if (b < c.B) {
            int first, n, len;
            bool ok = new_rows(c, cu, b, total, max_new, first, n, len);
            if (ok && (long long)len + n > ((long long)c.max_pages << c.page_log2)) {
                raise_error(ERRBIT_DATA);
                ok = false;
            }
            int cow = -1;
            if (ok && n > 0) {
                const int have = (len + P - 1) >> c.page_log2;
                need = ((len + n + P - 1) >> c.page_log2) - have;
                if (len & (P - 1)) {
                    const int last = c.table[(size_t)b * c.max_pages + have - 1];
                    if ((unsigned)last >= (unsigned)c.num_pages) {
                        raise_error(ERRBIT_DATA);
                        ok = false;
                    } else if (c.refs[last] > 1) {
                        cow = last;
                        ++need;
                    }
                }
            }
            if (!ok) bad = true;
            w.len0[b] = len;
            w.cow[b] = cow;
        }
        int tot;
        const int x = block_exclusive(need, tmp, tot);
        if (b < c.B) w.off[b] = carry + x;
        carry += tot;
    }
    bad = __syncthreads_or(bad);
    int found = 0;
    if (!bad) found = lowest_free(c.refs, c.num_pages, carry, w.list, total / P + 2 * c.B + 1, tmp);
    const bool fits = !bad && found == carry;
    if (threadIdx.x == 0) {
        w.head[0] = fits ? 1 : 0;
        *lack = bad ? -1 : carry - found;
    }
    if (!fits) return;
    __syncthreads();   // the list and the offsets are written
    for (int i = threadIdx.x; i < carry; i += PLAN_THREADS) {
        const int b = seq_of_row(w.off, c.B, i);
        const int have = (w.len0[b] + P - 1) >> c.page_log2;
        const int col = have - (w.cow[b] >= 0 ? 1 : 0) + i - w.off[b];
        const int id = w.list[i];
        c.table[(size_t)b * c.max_pages + col] = id;
        c.refs[id] = 1;
    }
    for (int b = threadIdx.x; b < c.B; b += PLAN_THREADS) {
        if (w.cow[b] >= 0) atomicSub(&c.refs[w.cow[b]], 1);
        c.len[b] = w.len0[b] + cu[b + 1] - cu[b];
    }
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t u, float scale) {
    const uint32_t lo = f32_to_e4m3_satfinite(__fdiv_rn(bf16_lo(u), scale));
    const uint32_t hi = f32_to_e4m3_satfinite(__fdiv_rn(bf16_hi(u), scale));
    return lo | (hi << 8);
}

// A warp a token and plane writes its row of Hkv * D values; the blocks after
// those copy, one sequence each, the tokens of a shared last page into the
// page its sequence got for them.
__global__ void __launch_bounds__(256)
    append_write_kernel(const CacheView c, const uint8_t* k_new, const uint8_t* v_new,
                        const int32_t* cu, int total, int token_blocks, const int32_t* ws) {
    const AppendWs w(const_cast<int32_t*>(ws), c.B);
    if (w.head[0] == 0) return;
    const int P = c.page_size();
    if ((int)blockIdx.x >= token_blocks) {
        const int b = blockIdx.x - token_blocks;
        const int src = w.cow[b];
        if (src < 0) return;
        const int len = w.len0[b], rem = len & (P - 1);
        const int dst = c.table[(size_t)b * c.max_pages + (len >> c.page_log2)];
        const size_t n16 = (size_t)rem * c.rowb / 16, page16 = (size_t)P * c.rowb / 16;
        const uint4 *ks = reinterpret_cast<const uint4*>(c.k) + src * page16,
                    *vs = reinterpret_cast<const uint4*>(c.v) + src * page16;
        uint4 *kd = reinterpret_cast<uint4*>(c.k) + dst * page16,
              *vd = reinterpret_cast<uint4*>(c.v) + dst * page16;
        for (size_t i0 = threadIdx.x; i0 < n16; i0 += 4 * 256) {
            uint4 x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 256 * j < n16) {
                    x[j] = ks[i0 + 256 * j];
                    y[j] = vs[i0 + 256 * j];
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 256 * j < n16) {
                    kd[i0 + 256 * j] = x[j];
                    vd[i0 + 256 * j] = y[j];
                }
        }
        if (c.ks)
            for (int i = threadIdx.x; i < rem; i += blockDim.x) {
                c.ks[(size_t)dst * P + i] = c.ks[(size_t)src * P + i];
                c.vs[(size_t)dst * P + i] = c.vs[(size_t)src * P + i];
            }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int job = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = job >> 1;
    if (r >= total) return;
    const int b = seq_of_row(cu, c.B, r);
    const int first = cu[b];
    if (r < first || r >= cu[b + 1]) return;      // behind the last sequence
    const int pos = w.len0[b] + r - first;
    const int row = c.row_of(c.table[(size_t)b * c.max_pages + (pos >> c.page_log2)], pos);
    if (row < 0) return;
    const bool value = job & 1;
    const int n8 = c.Hkv * c.D / 8;               // groups of eight values
    const uint4* src = reinterpret_cast<const uint4*>(value ? v_new : k_new) + (size_t)r * n8;
    uint8_t* plane = (value ? c.v : c.k) + (size_t)row * c.rowb;
    if (!c.ks) {
        for (int i0 = lane; i0 < n8; i0 += 128) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 32 * j < n8) x[j] = __ldcs(src + i0 + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 32 * j < n8) reinterpret_cast<uint4*>(plane)[i0 + 32 * j] = x[j];
        }
        return;
    }
    float amax = 0.0f;
    for (int i = lane; i < n8; i += 32) {
        const uint4 u = src[i];
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const float scale = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (lane == 0) (value ? c.vs : c.ks)[row] = scale;
    for (int i = lane; i < n8; i += 32) {
        const uint4 u = src[i];
        uint2 y;
        y.x = e4m3_pair(u.x, scale) | (e4m3_pair(u.y, scale) << 16);
        y.y = e4m3_pair(u.z, scale) | (e4m3_pair(u.w, scale) << 16);
        reinterpret_cast<uint2*>(plane)[i] = y;
    }
}

// Whether the n sequence ids and (lengths) those sequences' lengths are in
// range, and (distinct) each is named once; all threads of the block get the
// verdict, the same in every block: a length that another block has changed
// was in range and still is.  seen: B bits of shared memory.
__device__ bool ids_ok(const CacheView& c, const int32_t* ids, int n, bool distinct, bool lengths, uint32_t* seen) {
    const int B = c.B, most = c.max_pages << c.page_log2;
    for (int i = threadIdx.x; i < (B + 31) / 32; i += blockDim.x) seen[i] = 0;
    __syncthreads();
    bool ok = true;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int b = ids[i];
        if ((unsigned)b >= (unsigned)B) ok = false;
        else if (lengths && (unsigned)c.len[b] > (unsigned)most) ok = false;
        else if (distinct && (atomicOr(&seen[b >> 5], 1u << (b & 31)) >> (b & 31)) & 1u) ok = false;
    }
    return __syncthreads_and(ok);
}

// Pair by pair: the source's row is noted and its pages gain a reference...
__global__ void __launch_bounds__(1024)
    fork_take_kernel(const CacheView c, const int32_t* src, const int32_t* dst, int n, int32_t* ws) {
    extern __shared__ uint32_t seen[];
    if (!ids_ok(c, dst, n, true, false, seen) || !ids_ok(c, src, n, false, true, seen)) {
        if (threadIdx.x == 0) raise_error(ERRBIT_DATA);
        return;
    }
    const int i = blockIdx.x, s = src[i];
    int32_t* row = ws + n + (size_t)i * c.max_pages;
    const int32_t* from = c.table + (size_t)s * c.max_pages;
    for (int p = threadIdx.x; p < c.max_pages; p += blockDim.x) {
        int id = from[p];
        if (id >= c.num_pages) {
            raise_error(ERRBIT_DATA);
            id = -1;
        }
        if (id >= 0) atomicAdd(&c.refs[id], 1);
        row[p] = id;
    }
    if (threadIdx.x == 0) ws[i] = c.len[s];
}

// ...then every destination gives up its own pages and gets the noted row.
__global__ void __launch_bounds__(1024)
    fork_give_kernel(const CacheView c, const int32_t* src, const int32_t* dst, int n,
                     const int32_t* ws) {
    extern __shared__ uint32_t seen[];
    if (!ids_ok(c, dst, n, true, false, seen) || !ids_ok(c, src, n, false, true, seen)) return;
    const int i = blockIdx.x, d = dst[i];
    const int32_t* row = ws + n + (size_t)i * c.max_pages;
    int32_t* to = c.table + (size_t)d * c.max_pages;
    for (int p = threadIdx.x; p < c.max_pages; p += blockDim.x) {
        const int id = to[p];
        if ((unsigned)id < (unsigned)c.num_pages) atomicSub(&c.refs[id], 1);
        to[p] = row[p];
    }
    if (threadIdx.x == 0) c.len[d] = ws[i];
}

__global__ void __launch_bounds__(1024)
    free_kernel(const CacheView c, const int32_t* seqs, const int32_t* keep, int n) {
    extern __shared__ uint32_t seen[];
    bool ok = ids_ok(c, seqs, n, true, true, seen);
    bool neg = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) neg |= keep[i] < 0;
    ok = !__syncthreads_or(neg) && ok;
    if (!ok) {
        if (threadIdx.x == 0) raise_error(ERRBIT_DATA);
        return;
    }
    const int b = seqs[blockIdx.x];
    const int len = c.len[b];
    const int left = min(len, keep[blockIdx.x]);
    __syncthreads();   // every thread has the old length
    if (threadIdx.x == 0) c.len[b] = left;
    int32_t* row = c.table + (size_t)b * c.max_pages;
    const int P = c.page_size();
    for (int p = ((left + P - 1) >> c.page_log2) + threadIdx.x; p < c.max_pages; p += blockDim.x) {
        const int id = row[p];
        if (id < 0) continue;
        if (id < c.num_pages) atomicSub(&c.refs[id], 1);
        else raise_error(ERRBIT_DATA);
        row[p] = -1;
    }
}

// One PIECE of a page; bytes is a multiple of 16.  All 256 threads.
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, size_t bytes, size_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(src + at);
    uint4* d = reinterpret_cast<uint4*>(dst + at);
    const int n = (int)((bytes - at < (size_t)PIECE ? bytes - at : (size_t)PIECE) / 16);
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (threadIdx.x + j * 256 < n) v[j] = __ldcs(s + threadIdx.x + j * 256);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (threadIdx.x + j * 256 < n) __stcs(d + threadIdx.x + j * 256, v[j]);
}

__global__ void __launch_bounds__(256)
    copy_kernel(const uint8_t* src, int src_pages, uint8_t* dst, int dst_pages, size_t bytes,
                const int32_t* src_ids, const int32_t* dst_ids, int n) {
    const int pieces = (int)((bytes + PIECE - 1) / PIECE);
    const long long jobs = (long long)n * pieces;
    // the same piece of every page, then the next: copies of one source read
    // it from L2 together (48 branches of 16 caches with 4 MB of indexer keys
    // each, fork and copy: 137 -> 101 us, 64 bytes a thread in flight
    // included; the floor is 74)
    for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int i = (int)(j % n);
        const int a = src_ids[i], b = dst_ids[i];
        if ((unsigned)a >= (unsigned)src_pages || (unsigned)b >= (unsigned)dst_pages) {
            if (threadIdx.x == 0) raise_error(ERRBIT_DATA);
            continue;
        }
        copy_piece(src + (size_t)a * bytes, dst + (size_t)b * bytes, bytes,
                   (size_t)(j / n) * PIECE);
    }
}

// Workspace of a compaction: U and the number of moves, the moves' sources
// and destinations, and every page's new id.
struct CompactWs {
    int32_t *head, *of, *to, *remap;
    __host__ __device__ CompactWs(int32_t* ws, int num_pages)
        : head(ws), of(ws + 4), to(of + num_pages / 2 + 1), remap(to + num_pages / 2 + 1) {}
};

// One block: U, then the i-th used id >= U beside the i-th free id < U (as
// many of one as of the other), and the new ids.
__global__ void __launch_bounds__(PLAN_THREADS)
    compact_plan_kernel(const CacheView c, int32_t* used_out, int32_t* ws) {
    __shared__ int tmp[33];
    const CompactWs w(ws, c.num_pages);
    constexpr int PER = 8;                // pages a thread takes at a time
    int mine = 0;
    for (int p = threadIdx.x; p < c.num_pages; p += PLAN_THREADS) mine += c.refs[p] > 0;
    int used;
    block_exclusive(mine, tmp, used);
    int moves = 0, holes = 0;
    for (int base = 0; base < c.num_pages; base += PLAN_THREADS * PER) {
        const int p0 = base + threadIdx.x * PER;
        uint32_t live = 0, in = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (p0 + i < c.num_pages) {
                in |= 1u << i;
                live |= (uint32_t)(c.refs[p0 + i] > 0) << i;
            }
        uint32_t low = 0;                 // ids below U
#pragma unroll
        for (int i = 0; i < PER; ++i) low |= (uint32_t)(p0 + i < used) << i;
        const uint32_t of = live & ~low, to = in & ~live & low;
        int tot;
        // both ranks in one scan: at most 8192 of each
        const int x = block_exclusive(__popc(of) | (__popc(to) << 16), tmp, tot);
        int a = moves + (x & 0xFFFF), b = holes + (x >> 16);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (((of >> i) & 1) && PIVOT_CHECK(a <= c.num_pages / 2)) w.of[a++] = p0 + i;
            if (((to >> i) & 1) && PIVOT_CHECK(b <= c.num_pages / 2)) w.to[b++] = p0 + i;
            if ((in >> i) & 1) w.remap[p0 + i] = (live >> i) & 1 ? p0 + i : -1;
        }
        moves += tot & 0xFFFF;
        holes += tot >> 16;
    }
    if (threadIdx.x == 0) {
        w.head[0] = used;
        w.head[1] = moves;
        if (used_out) *used_out = used;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += PLAN_THREADS) w.remap[w.of[i]] = w.to[i];
}

__global__ void __launch_bounds__(256)
    compact_move_kernel(const CacheView c, int32_t* remap_out, const int32_t* ws) {
    const CompactWs w(const_cast<int32_t*>(ws), c.num_pages);
    const int moves = w.head[1];
    const size_t bytes = (size_t)c.page_size() * c.rowb;
    const int pieces = (int)((bytes + PIECE - 1) / PIECE);
    const long long jobs = (long long)moves * 2 * pieces;
    for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int piece = (int)(j % pieces);
        const int i = (int)(j / pieces) >> 1;
        const bool value = (j / pieces) & 1;
        const int a = w.of[i], b = w.to[i];
        uint8_t* plane = value ? c.v : c.k;
        copy_piece(plane + (size_t)a * bytes, plane + (size_t)b * bytes, bytes, (size_t)piece * PIECE);
        if (piece == 0) {
            float* scale = value ? c.vs : c.ks;
            const int P = c.page_size();
            if (scale)
                for (int t = threadIdx.x; t < P; t += blockDim.x)
                    scale[(size_t)b * P + t] = scale[(size_t)a * P + t];
            if (!value && threadIdx.x == 0) {
                c.refs[b] = c.refs[a];
                c.refs[a] = 0;
            }
        }
    }
    const long long tid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long nth = (long long)gridDim.x * blockDim.x;
    const long long cells = (long long)c.B * c.max_pages;
    for (long long e = tid; e < cells; e += nth) {
        const int id = c.table[e];
        if (id < 0) continue;
        const int now = id < c.num_pages ? w.remap[id] : -1;
        if (now < 0) raise_error(ERRBIT_DATA);
        if (now != id) c.table[e] = now;
    }
    if (remap_out)
        for (long long p = tid; p < c.num_pages; p += nth) remap_out[p] = w.remap[p];
}

size_t seen_bytes(int B) { return (size_t)((B + 31) / 32) * 4; }
// Threads of a block that walks one table row.
int row_threads(int max_pages) { return max_pages > 512 ? 1024 : 256; }

}  // namespace

size_t append_ws_words(int B, int total, int page) {
    return 4 + 3 * (size_t)B + (size_t)total / page + 2 * (size_t)B + 1;
}
size_t fork_ws_words(int n, int max_pages) { return (size_t)n * (1 + (size_t)max_pages); }
size_t compact_ws_words(int num_pages) { return 4 + 2 * ((size_t)num_pages / 2 + 1) + num_pages; }

cudaError_t launch_append(const CacheView& c, const void* k_new, const void* v_new,
                          const int32_t* cu, int total, int max_new, int32_t* lack, int32_t* ws,
                          cudaStream_t st) {
    append_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(c, cu, total, max_new, lack, ws);
    const int token_blocks = (int)(((long long)total * 2 + 7) / 8);
    append_write_kernel<<<token_blocks + c.B, 256, 0, st>>>(
        c, static_cast<const uint8_t*>(k_new), static_cast<const uint8_t*>(v_new), cu, total,
        token_blocks, ws);
    return cudaGetLastError();
}

cudaError_t launch_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int n,
                        int32_t* ws, cudaStream_t st) {
    fork_take_kernel<<<n, row_threads(c.max_pages), seen_bytes(c.B), st>>>(c, src, dst, n, ws);
    fork_give_kernel<<<n, row_threads(c.max_pages), seen_bytes(c.B), st>>>(c, src, dst, n, ws);
    return cudaGetLastError();
}

cudaError_t launch_free(const CacheView& c, const int32_t* seqs, const int32_t* keep, int n,
                        cudaStream_t st) {
    free_kernel<<<n, row_threads(c.max_pages), seen_bytes(c.B), st>>>(c, seqs, keep, n);
    return cudaGetLastError();
}

cudaError_t launch_copy(const void* src, int src_pages, void* dst, int dst_pages, size_t page_bytes,
                        const int32_t* src_ids, const int32_t* dst_ids, int n, int sms,
                        cudaStream_t st) {
    const long long jobs = (long long)n * (long long)((page_bytes + PIECE - 1) / PIECE);
    const int grid = (int)(jobs < (long long)sms * 8 ? jobs : (long long)sms * 8);
    copy_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(src), src_pages,
                                      static_cast<uint8_t*>(dst), dst_pages, page_bytes, src_ids,
                                      dst_ids, n);
    return cudaGetLastError();
}

cudaError_t launch_compact(const CacheView& c, int32_t* remap, int32_t* used, int32_t* ws, int sms,
                           cudaStream_t st) {
    compact_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(c, used, ws);
    compact_move_kernel<<<sms * 8, 256, 0, st>>>(c, remap, ws);
    return cudaGetLastError();
}

}  // namespace pivot
