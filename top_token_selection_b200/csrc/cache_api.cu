// cache_api.cu -- C entry points of the paged cache: argument checks,
// workspace layout and launches.  See include/pivot.h for the contract.
#include <climits>

#include "attend.h"
#include "host.h"
#include "pages.h"
#include "profile.h"

#include <nvtx3/nvToolsExt.h>

namespace pivot {

namespace {

constexpr size_t WS_ALIGN = 256;
constexpr int MAX_SEQS = 65536;      // sequence ids are marked in one bit each of shared memory
constexpr int MAX_SELECTED = 65536;
constexpr int MAX_TOKENS = 1 << 26;  // the plan counts 1024 row blocks' tiles of 64 tokens in 32 bits

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

size_t up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool ws_ok(const void* ws) { return ws && aligned(ws, WS_ALIGN); }

pivot_status_t check_cache(const pivot_cache_t* c, CacheView* v) {
    if (!c || (c->dtype != PIVOT_F32 && c->dtype != PIVOT_BF16 && c->dtype != PIVOT_E4M3))
        return PIVOT_ERR_INVALID_ARG;
    if (c->B < 1 || c->Hkv < 1 || c->D < 1 || c->page_size < 1 || c->num_pages < 1 || c->max_pages < 1)
        return PIVOT_ERR_INVALID_ARG;
    if (!c->k || !c->v || !c->table || !c->len || !c->refs) return PIVOT_ERR_INVALID_ARG;
    const bool fp8 = c->dtype == PIVOT_E4M3;
    if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr)) return PIVOT_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return PIVOT_ERR_INVALID_ARG;
    if (c->dtype == PIVOT_F32) return PIVOT_ERR_UNSUPPORTED;
    int l2 = 4;
    while (l2 <= 8 && (1 << l2) != c->page_size) ++l2;
    if (l2 > 8 || c->B > MAX_SEQS) return PIVOT_ERR_UNSUPPORTED;
    const int es = fp8 ? 1 : 2;
    if ((c->D * (long long)es) % 16) return PIVOT_ERR_UNSUPPORTED;
    if ((long long)c->num_pages * c->page_size > INT_MAX ||
        (long long)c->max_pages * c->page_size > INT_MAX ||
        (long long)c->Hkv * c->D * es > INT_MAX / 256)
        return PIVOT_ERR_UNSUPPORTED;
    v->k = static_cast<uint8_t*>(c->k);
    v->v = static_cast<uint8_t*>(c->v);
    v->ks = c->k_scale;
    v->vs = c->v_scale;
    v->table = c->table;
    v->len = c->len;
    v->refs = c->refs;
    v->B = c->B;
    v->Hkv = c->Hkv;
    v->D = c->D;
    v->page_log2 = l2;
    v->num_pages = c->num_pages;
    v->max_pages = c->max_pages;
    v->rowb = c->Hkv * c->D * es;
    return PIVOT_OK;
}

pivot_status_t check_attend(const pivot_cache_t* cache, const pivot_attend_t* a, bool selected,
                            AttendParams* p) {
    const pivot_status_t st = check_cache(cache, &p->c);
    if (st != PIVOT_OK) return st;
    if (!a || a->Hq < 1 || a->total < 0 || a->max_new < 0 || a->window < 0) return PIVOT_ERR_INVALID_ARG;
    if (a->Hq % cache->Hkv) return PIVOT_ERR_INVALID_ARG;
    if (!(a->scale > 0.0f) || !(a->scale <= 1e30f)) return PIVOT_ERR_INVALID_ARG;
    if (selected ? (a->topk < 1 || a->window != 0) : (a->topk != 0 || a->idx)) return PIVOT_ERR_INVALID_ARG;
    if (a->total > 0 && (!a->q || !a->cu_new || !a->o || a->max_new < 1 || (selected && !a->idx)))
        return PIVOT_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->o, 16)) return PIVOT_ERR_INVALID_ARG;
    if (cache->D != 64 && cache->D != 128) return PIVOT_ERR_UNSUPPORTED;
    if (a->topk > MAX_SELECTED || (long long)a->total * a->Hq > INT_MAX ||
        (long long)cache->max_pages * cache->page_size > MAX_TOKENS)
        return PIVOT_ERR_UNSUPPORTED;
    p->q = static_cast<const uint16_t*>(a->q);
    p->cu = a->cu_new;
    p->idx = selected ? a->idx : nullptr;
    p->o = static_cast<uint16_t*>(a->o);
    p->lse = a->lse;
    p->Hq = a->Hq;
    p->G = a->Hq / cache->Hkv;
    p->total = a->total;
    p->max_new = a->max_new < a->total ? a->max_new : a->total;
    p->window = a->window;
    p->topk = a->topk;
    p->scale_log2 = a->scale * 1.4426950408889634f;
    // Rows a sequence has for one key/value head: up to 32 on the warp-level
    // kernel (16 or 32 of them share each key read), more on the tensor-memory
    // kernel in blocks of 128 or 256.  Both kernels at 32 rows, us (rows,
    // tensor memory): two tokens over 32 caches of 32K to 128K tokens, e4m3 787
    // and 1095, bf16 867 and 822; over 2048 selected positions of each, e4m3
    // 144 and 202, bf16 134 and 153.  At 16 rows over the caches: 492 and 1088,
    // 773 and 816.
    const long long rows = selected ? p->G : (long long)p->max_new * p->G;
    if (rows > 32) {
        p->R = selected || rows <= 128 ? 128 : 256;
        p->TK = 128;
        p->ncta = sm_count();
    } else {
        p->R = rows <= 16 ? 16 : 32;
        p->TK = rows_tile(cache->dtype);
        p->ncta = sm_count() * ROWS_CTAS_PER_SM;
    }
    return PIVOT_OK;
}

// The plane as rows of tokens: a box is a page (at most 128 tokens) high, and
// 64 bf16 values or one head's e4m3 codes wide.
bool plane_map(CUtensorMap* map, const CacheView& c, void* plane) {
    const TensorMapEncodeFn fn = tensor_map_encode();
    if (!fn) return false;
    const bool fp8 = c.ks != nullptr;
    const cuuint64_t dims[2] = {(cuuint64_t)c.Hkv * c.D, (cuuint64_t)c.num_pages * c.page_size()};
    const cuuint64_t strides[1] = {(cuuint64_t)c.rowb};
    const cuuint32_t rows = c.page_size() < 128 ? c.page_size() : 128;
    const cuuint32_t box[2] = {(cuuint32_t)(fp8 ? c.D : 64), rows}, steps[2] = {1, 1};
    return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, plane, dims,
              strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp8 && c.D == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t attend_layout(AttendParams* p, bool selected, void* ws) {
    size_t at = 0;
    uint8_t* base = static_cast<uint8_t*>(ws);
    if (!selected) {
        const size_t blocks = (size_t)((long long)p->total * p->G / p->R) + p->c.B;
        p->seq_units = reinterpret_cast<long long*>(base);
        p->blk_units = p->seq_units + p->c.B + 1;
        p->blk_off = reinterpret_cast<int32_t*>(p->blk_units + blocks);
        at = up(attend_plan_bytes(p->c.B, p->total, p->G, p->R));
    }
    p->join = reinterpret_cast<JoinRecord*>(base + at);
    p->part = reinterpret_cast<float*>(p->join + p->ncta);
    return at + up(attend_part_bytes(p->ncta, p->R, p->c.D));
}

size_t attend_size(const pivot_cache_t* cache, const pivot_attend_t* a, bool selected) {
    AttendParams p{};
    if (check_attend(cache, a, selected, &p) != PIVOT_OK) return 0;
    return attend_layout(&p, selected, nullptr);
}

pivot_status_t attend(const pivot_cache_t* cache, const pivot_attend_t* a, bool selected, void* ws,
                      size_t ws_bytes, cudaStream_t st) {
    AttendParams p{};
    const pivot_status_t s = check_attend(cache, a, selected, &p);
    if (s != PIVOT_OK) return s;
    if (!ws_ok(ws)) return PIVOT_ERR_INVALID_ARG;
    if (attend_layout(&p, selected, ws) > ws_bytes) return PIVOT_ERR_WORKSPACE;
    if (p.total == 0) return PIVOT_OK;
    cudaError_t e = cudaSuccess;
    CUtensorMap tk, tv;
    if (p.R > 32 && (!plane_map(&tk, p.c, p.c.k) || !plane_map(&tv, p.c, p.c.v))) return PIVOT_ERR_CUDA;
    if (!selected) {
        count_launch();
        e = launch_attend_plan(p, st);
        if (e != cudaSuccess) return status_of(e);
    }
    count_launch();
    e = p.R > 32 ? launch_attend_umma(tk, tv, p, st) : launch_attend_rows(p, st);
    if (e != cudaSuccess) return status_of(e);
    count_launch();
    return status_of(launch_attend_join(p, st));
}

}  // namespace

}  // namespace pivot

using namespace pivot;

extern "C" {

size_t pivot_cache_append_workspace_size(const pivot_cache_t* cache, int32_t total) {
    CacheView c;
    if (check_cache(cache, &c) != PIVOT_OK || total < 0) return 0;
    return up(append_ws_words(c.B, total, c.page_size()) * 4);
}

pivot_status_t pivot_cache_append(const pivot_cache_t* cache, const void* k_new, const void* v_new,
                                  const int32_t* cu_new, int32_t total, int32_t max_new,
                                  int32_t* lack, void* ws, size_t ws_bytes, void* stream) {
    Range range("pivot_cache_append");
    CacheView c;
    const pivot_status_t st = check_cache(cache, &c);
    if (st != PIVOT_OK) return st;
    if (total < 0 || max_new < 0 || !cu_new || !lack) return PIVOT_ERR_INVALID_ARG;
    if (total > 0 && (!k_new || !v_new || max_new < 1)) return PIVOT_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !ws_ok(ws)) return PIVOT_ERR_INVALID_ARG;
    if ((long long)total * 2 > INT_MAX) return PIVOT_ERR_UNSUPPORTED;
    if (ws_bytes < pivot_cache_append_workspace_size(cache, total)) return PIVOT_ERR_WORKSPACE;
    count_launch();
    count_launch();
    return status_of(launch_append(c, k_new, v_new, cu_new, total, max_new, lack,
                                   static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

size_t pivot_pages_fork_workspace_size(const pivot_cache_t* cache, int32_t n) {
    CacheView c;
    if (check_cache(cache, &c) != PIVOT_OK || n < 0 || n > c.B) return 0;
    return up(fork_ws_words(n > 0 ? n : 1, c.max_pages) * 4);
}

pivot_status_t pivot_pages_fork(const pivot_cache_t* cache, const int32_t* src, const int32_t* dst,
                                int32_t n, void* ws, size_t ws_bytes, void* stream) {
    Range range("pivot_pages_fork");
    CacheView c;
    const pivot_status_t st = check_cache(cache, &c);
    if (st != PIVOT_OK) return st;
    // more pairs than sequences would name a destination twice
    if (n < 0 || n > c.B || (n > 0 && (!src || !dst)) || !ws_ok(ws)) return PIVOT_ERR_INVALID_ARG;
    if (ws_bytes < pivot_pages_fork_workspace_size(cache, n)) return PIVOT_ERR_WORKSPACE;
    if (n == 0) return PIVOT_OK;
    count_launch();
    count_launch();
    return status_of(launch_fork(c, src, dst, n, static_cast<int32_t*>(ws),
                                 static_cast<cudaStream_t>(stream)));
}

pivot_status_t pivot_pages_free(const pivot_cache_t* cache, const int32_t* seqs, const int32_t* keep,
                                int32_t n, void* stream) {
    Range range("pivot_pages_free");
    CacheView c;
    const pivot_status_t st = check_cache(cache, &c);
    if (st != PIVOT_OK) return st;
    if (n < 0 || n > c.B || (n > 0 && (!seqs || !keep))) return PIVOT_ERR_INVALID_ARG;
    if (n == 0) return PIVOT_OK;
    count_launch();
    return status_of(launch_free(c, seqs, keep, n, static_cast<cudaStream_t>(stream)));
}

pivot_status_t pivot_pages_copy(const void* src, int32_t src_pages, void* dst, int32_t dst_pages,
                                size_t page_bytes, const int32_t* src_ids, const int32_t* dst_ids,
                                int32_t n, void* stream) {
    Range range("pivot_pages_copy");
    if (!src || !dst || src_pages < 1 || dst_pages < 1 || n < 0) return PIVOT_ERR_INVALID_ARG;
    if (n > 0 && (!src_ids || !dst_ids)) return PIVOT_ERR_INVALID_ARG;
    if (page_bytes < 16 || page_bytes % 16 || !aligned(src, 16) || !aligned(dst, 16))
        return PIVOT_ERR_INVALID_ARG;
    if (page_bytes > (size_t(1) << 40)) return PIVOT_ERR_UNSUPPORTED;
    if (n == 0) return PIVOT_OK;
    count_launch();
    return status_of(launch_copy(src, src_pages, dst, dst_pages, page_bytes, src_ids, dst_ids, n,
                                 sm_count(), static_cast<cudaStream_t>(stream)));
}

size_t pivot_pages_compact_workspace_size(const pivot_cache_t* cache) {
    CacheView c;
    if (check_cache(cache, &c) != PIVOT_OK) return 0;
    return up(compact_ws_words(c.num_pages) * 4);
}

pivot_status_t pivot_pages_compact(const pivot_cache_t* cache, int32_t* remap, int32_t* used, void* ws,
                                   size_t ws_bytes, void* stream) {
    Range range("pivot_pages_compact");
    CacheView c;
    const pivot_status_t st = check_cache(cache, &c);
    if (st != PIVOT_OK) return st;
    if (!ws_ok(ws)) return PIVOT_ERR_INVALID_ARG;
    if (ws_bytes < pivot_pages_compact_workspace_size(cache)) return PIVOT_ERR_WORKSPACE;
    count_launch();
    count_launch();
    return status_of(launch_compact(c, remap, used, static_cast<int32_t*>(ws), sm_count(),
                                    static_cast<cudaStream_t>(stream)));
}

size_t pivot_paged_attention_workspace_size(const pivot_cache_t* cache, const pivot_attend_t* call) {
    return attend_size(cache, call, false);
}

pivot_status_t pivot_paged_attention(const pivot_cache_t* cache, const pivot_attend_t* call, void* ws,
                                     size_t ws_bytes, void* stream) {
    Range range("pivot_paged_attention");
    return attend(cache, call, false, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

size_t pivot_selected_attention_workspace_size(const pivot_cache_t* cache, const pivot_attend_t* call) {
    return attend_size(cache, call, true);
}

pivot_status_t pivot_selected_attention(const pivot_cache_t* cache, const pivot_attend_t* call, void* ws,
                                        size_t ws_bytes, void* stream) {
    Range range("pivot_selected_attention");
    return attend(cache, call, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
