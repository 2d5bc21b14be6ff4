// pages.h -- launchers of the page operations (pages.cu).
#pragma once

#include "paged.cuh"

namespace pivot {

// Workspaces, in 4-byte words.
size_t append_ws_words(int B, int total, int page);
size_t fork_ws_words(int n, int max_pages);
size_t compact_ws_words(int num_pages);

cudaError_t launch_append(const CacheView& c, const void* k_new, const void* v_new,
                          const int32_t* cu, int total, int max_new, int32_t* lack, int32_t* ws,
                          cudaStream_t st);
cudaError_t launch_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int n,
                        int32_t* ws, cudaStream_t st);
cudaError_t launch_free(const CacheView& c, const int32_t* seqs, const int32_t* keep, int n,
                        cudaStream_t st);
cudaError_t launch_copy(const void* src, int src_pages, void* dst, int dst_pages,
                        size_t page_bytes, const int32_t* src_ids, const int32_t* dst_ids, int n,
                        int sms, cudaStream_t st);
cudaError_t launch_compact(const CacheView& c, int32_t* remap, int32_t* used, int32_t* ws, int sms,
                           cudaStream_t st);

}  // namespace pivot
