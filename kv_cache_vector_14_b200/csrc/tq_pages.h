// Internal declarations of the page operators (tq_pages.cu).
#pragma once

#include "tq_internal.h"

namespace tqi {

constexpr int kMaxPageBuffers = TQ_MAX_PAGE_BUFFERS;

struct PageBuffers {
    uint8_t* src[kMaxPageBuffers];
    uint8_t* dst[kMaxPageBuffers];
    uint32_t units[kMaxPageBuffers];     // 16-byte units of a page
    int n;
};
struct PagesArgs {
    int32_t* table;           // [B*Hkv][NB] pages, -1: none
    int32_t* refs;            // [pool] table entries that name each page
    int64_t B, Hkv, NB, pool;
    int* err;
    // workspace
    int32_t* counts;          // [4]: moves, live pages
    int32_t* from;            // [pool] moves: source page (alloc: -1 where nothing is copied)
    int32_t* to;              // [pool] destination page
    int32_t* rank;            // [pool] compact: move that takes a page away
    int32_t* list;            // [pool] alloc: free pages, lowest first; compact: live pages per segment
};
struct PagesWs {
    size_t off_from, off_to, off_rank, off_list, bytes;
};
inline PagesWs pages_ws(int64_t pool) {
    PagesWs w{};
    const size_t each = ((size_t)pool * 4 + 255) / 256 * 256;
    w.off_from = 256;
    w.off_to = w.off_from + each;
    w.off_rank = w.off_to + each;
    w.off_list = w.off_rank + each;
    w.bytes = w.off_list + each;
    return w;
}

constexpr int64_t kMaxForkSequences = 7168;   // a fork stages 8 table columns of all sequences in shared memory

cudaError_t launch_pages_free(const PagesArgs& a, const int32_t* keep, cudaStream_t s);
cudaError_t launch_pages_fork(const PagesArgs& a, const int32_t* parent, cudaStream_t s);
cudaError_t launch_pages_alloc(const PagesArgs& a, const PageBuffers& b, const int32_t* lo, const int32_t* hi, int32_t* info,
                               int num_sms, cudaStream_t s);
cudaError_t launch_pages_compact(const PagesArgs& a, const PageBuffers& b, int32_t* info, int num_sms, cudaStream_t s);
// n >= 0 moves from src[i] to dst[i]; pages outside [0, pool_src) / [0, pool_dst) are skipped (check word), -1 silently
cudaError_t launch_pages_copy(const PageBuffers& b, const int32_t* src, const int32_t* dst, int64_t n, int64_t pool_src,
                              int64_t pool_dst, int* err, int num_sms, cudaStream_t s);

}  // namespace tqi
