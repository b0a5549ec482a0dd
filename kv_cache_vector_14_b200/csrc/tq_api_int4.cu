// C entry points of the 4-bit caches and of the page operators (include/tq.h):
// argument checks and launches.
#include <cmath>

#include "tq_int4.h"
#include "tq_pages.h"

using namespace tqi;

namespace {

tq_status device_ok(const tq_handle* h) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
    return dev == h->device ? TQ_OK : TQ_ERR_INVALID_ARG;
}

// Checks of an encode or expand of one cache; *empty: nothing to do.
tq_status prepare_copy(const tq_handle* h, int group, const void* x, tq_dtype dt, int64_t B, int64_t Hkv, int64_t T,
                       int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos, int64_t t0,
                       Int4CopyArgs* a, int side, bool* empty) {
    *empty = false;
    if (!h || !dtype_ok(dt) || !cache_ok(h, c) || !int4_group_ok(h->d, group)) return TQ_ERR_INVALID_ARG;
    if (B != c->B || Hkv != c->Hkv || T < 0 || (pos && !aligned(pos, 4))) return TQ_ERR_INVALID_ARG;
    if (!pos && (t0 < 0 || t0 > c->Tcap || T > c->Tcap - t0)) return TQ_ERR_INVALID_ARG;
    if (B == 0 || T == 0) {
        *empty = true;
        return TQ_OK;
    }
    if (!x || !aligned(x, dtype_size(dt)) || sb < 0 || sh < 0 || st < 0) return TQ_ERR_INVALID_ARG;
    if (T > c->Tcap) return TQ_ERR_INVALID_ARG;
    // word indices are 32-bit; (B Hkv, T, words) multiplied stepwise, so that no product overflows
    const int64_t most = (int64_t)1 << 31;
    if (B >= most || Hkv >= most || B * Hkv >= most || T >= most || B * Hkv * T >= most || B * Hkv * T * (h->d / 8) >= most)
        return TQ_ERR_UNSUPPORTED;
    a->side[side] = Int4Side{const_cast<void*>(x), static_cast<uint8_t*>(c->base), c->block_table, c->pool_blocks};
    a->nsides = side + 1;
    a->sb = sb; a->sh = sh; a->st = st;
    a->B = B; a->Hkv = Hkv; a->T = T;
    a->pos = pos;
    a->t0 = t0;
    a->Tcap = c->Tcap;
    a->NB = c->Tcap / kBlockT;
    const int64_t es = (int64_t)dtype_size(dt);
    const bool v16 = aligned(x, 16) && (sb * es) % 16 == 0 && (sh * es) % 16 == 0 && (st * es) % 16 == 0;
    a->vec16 = (side == 0 || a->vec16) && v16;
    a->err = h->derr;
    a->fdT = make_fastdiv((uint32_t)T);
    a->fdH = make_fastdiv((uint32_t)Hkv);
    return device_ok(h);
}

tq_status copy_common(bool encode, const tq_handle* h, int group, const void* x, tq_dtype dt, int64_t B, int64_t Hkv,
                      int64_t T, int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos, int64_t t0,
                      void* stream) {
    Int4CopyArgs a{};
    bool empty;
    const tq_status r = prepare_copy(h, group, x, dt, B, Hkv, T, sb, sh, st, c, pos, t0, &a, 0, &empty);
    if (r != TQ_OK || empty) return r;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(encode ? launch_int4_encode(h->d, group, dt, a, h->num_sms, s)
                              : launch_int4_expand(h->d, group, dt, a, h->num_sms, s));
}

struct AttendWs {
    size_t off_ml, off_acc, off_split, bytes;
};
AttendWs attend_ws(int d, int num_sms, int slot_rows) {
    const size_t ctas = num_sms < kInt4MaxCtas ? num_sms : kInt4MaxCtas;
    const size_t slots = ctas * 2 * slot_rows;
    AttendWs w;
    w.off_ml = 0;
    w.off_acc = (slots * 2 * 4 + 255) / 256 * 256;
    w.off_split = w.off_acc + slots * d * 4;
    w.bytes = w.off_split + ctas * sizeof(int4);
    return w;
}

bool attend_sizes_ok(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv) {
    const int64_t most = (int64_t)1 << 31;
    if (B >= most || Lq >= most || Hq >= most) return false;
    const int64_t G = Hq / Hkv;
    if (Lq * G >= most) return false;
    return Hkv * ((Lq * G + 3) / 4) < most;
}

cudaError_t launch_any(const tq_handle* h, int group, tq_dtype dt, const Int4AttendArgs& a, cudaStream_t s) {
    return int4_slot_rows(h->d, dt, a.rows) > 8 ? launch_int4_chunk(h->d, group, dt, a, h->num_sms, s)
                                                : launch_int4_attend(h->d, group, dt, a, h->num_sms, s);
}

// Whether tokens of the two caches may share blocks: contiguous ones whose bytes meet, or one pool
// under one table (two tables over one pool are taken to name different blocks).
bool caches_meet(const tq_handle* h, int group, const tq_cache* x, const tq_cache* y) {
    if (x->block_table || y->block_table) return x->base == y->base && x->block_table == y->block_table;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x->base), b = reinterpret_cast<uintptr_t>(y->base);
    const uintptr_t n = (uintptr_t)(x->B * x->Hkv * (x->Tcap / kBlockT) * int4_block_bytes(h->d, group));
    return a < b + n && b < a + n;                     // (of one size: prepare_attend)
}

// Checks of an attention call and its kernel arguments; *empty: nothing to do.
tq_status prepare_attend(const tq_handle* h, int group, const void* q, tq_dtype qdt, int64_t B, int64_t Lq, int64_t Hq,
                         const tq_cache* kc, const tq_cache* vc, const int32_t* lens, int64_t T, int64_t add, float scale,
                         void* out, void* ws, size_t ws_bytes, Int4AttendArgs* a, bool* empty) {
    *empty = false;
    if (!h || !dtype_ok(qdt) || !cache_ok(h, kc) || !cache_ok(h, vc) || !int4_group_ok(h->d, group))
        return TQ_ERR_INVALID_ARG;
    if (B < 0 || Lq < 0 || Hq <= 0 || kc->B != B || vc->B != B || kc->Hkv != vc->Hkv || kc->Tcap != vc->Tcap ||
        Hq % kc->Hkv || !std::isfinite(scale * kLog2e) || (lens && !aligned(lens, 4)))
        return TQ_ERR_INVALID_ARG;
    if (!lens && (T < 0 || T > kc->Tcap - add)) return TQ_ERR_INVALID_ARG;
    if (!attend_sizes_ok(B, Lq, Hq, kc->Hkv) || kc->Tcap >= ((int64_t)1 << 31)) return TQ_ERR_UNSUPPORTED;
    if (B == 0 || Lq == 0) {
        *empty = true;
        return TQ_OK;
    }
    if (!q || !out || !ws || !aligned(q, dtype_size(qdt)) || !aligned(out, dtype_size(qdt)) || !aligned(ws, 256))
        return TQ_ERR_INVALID_ARG;
    const AttendWs w = attend_ws(h->d, h->num_sms, int4_slot_rows(h->d, qdt, (int)(Lq * (Hq / kc->Hkv))));
    if (ws_bytes < w.bytes) return TQ_ERR_WORKSPACE;
    uint8_t* p = static_cast<uint8_t*>(ws);
    a->q = q;
    a->out = out;
    a->kc = static_cast<const uint8_t*>(kc->base);
    a->vc = static_cast<const uint8_t*>(vc->base);
    a->ktable = kc->block_table;
    a->vtable = vc->block_table;
    a->kpool = kc->pool_blocks;
    a->vpool = vc->pool_blocks;
    a->lens = lens;
    a->T = T;
    a->add = add;
    a->Tcap = kc->Tcap;
    a->NB = kc->Tcap / kBlockT;
    a->B = B; a->Hq = Hq; a->Hkv = kc->Hkv; a->Lq = Lq;
    a->G = (int)(Hq / kc->Hkv);
    a->rows = (int)(Lq * a->G);
    a->scale_log2 = scale * kLog2e;
    a->part_ml = reinterpret_cast<float*>(p + w.off_ml);
    a->part_acc = reinterpret_cast<float*>(p + w.off_acc);
    a->split = reinterpret_cast<int4*>(p + w.off_split);
    a->err = h->derr;
    a->first_wait = h->first_wait >= 0 ? h->first_wait : kDefaultWaitLimit;
    a->vec16 = aligned(q, 16) && aligned(out, 16);
    return device_ok(h);
}

// State (table, refs) of a page call.
tq_status prepare_pages(const tq_handle* h, const tq_pages* p, PagesArgs* a, bool* empty) {
    *empty = false;
    if (!h || !p || !p->block_table || !p->refs || !aligned(p->block_table, 4) || !aligned(p->refs, 4) || p->B < 0 ||
        p->Hkv <= 0 || p->NB <= 0 || p->pool_blocks <= 0)
        return TQ_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 31;
    if (p->pool_blocks >= most || p->B >= most || p->Hkv >= most || p->NB >= most / kBlockT || p->B * p->Hkv >= most ||
        p->B * p->Hkv * p->NB >= most)
        return TQ_ERR_UNSUPPORTED;
    *empty = p->B == 0;
    *a = PagesArgs{};
    a->table = p->block_table;
    a->refs = p->refs;
    a->B = p->B; a->Hkv = p->Hkv; a->NB = p->NB;
    a->pool = p->pool_blocks;
    a->err = h->derr;
    return device_ok(h);
}

bool buffers_ok(const tq_pages* p) {
    if (p->n_buffers < 0 || p->n_buffers > kMaxPageBuffers || (p->n_buffers > 0 && (!p->buffers || !p->block_bytes)))
        return false;
    for (int i = 0; i < p->n_buffers; ++i)
        if (!p->buffers[i] || !aligned(p->buffers[i], 16) || p->block_bytes[i] <= 0 || p->block_bytes[i] % 16 ||
            p->block_bytes[i] >= ((int64_t)1 << 32))
            return false;
    return true;
}
void set_buffers(PageBuffers* b, const tq_pages* from, const tq_pages* to) {
    *b = PageBuffers{};
    b->n = from->n_buffers;
    for (int i = 0; i < b->n; ++i) {
        b->src[i] = static_cast<uint8_t*>(from->buffers[i]);
        b->dst[i] = static_cast<uint8_t*>(to->buffers[i]);
        b->units[i] = (uint32_t)(from->block_bytes[i] / 16);
    }
}
tq_status prepare_pages_ws(const tq_handle* h, const tq_pages* p, void* ws, size_t ws_bytes, PagesArgs* a, PageBuffers* b,
                           bool* empty) {
    const tq_status r = prepare_pages(h, p, a, empty);
    if (r != TQ_OK) return r;
    if (!buffers_ok(p) || !ws || !aligned(ws, 256)) return TQ_ERR_INVALID_ARG;
    const PagesWs w = pages_ws(p->pool_blocks);
    if (ws_bytes < w.bytes) return TQ_ERR_WORKSPACE;
    uint8_t* base = static_cast<uint8_t*>(ws);
    a->counts = reinterpret_cast<int32_t*>(base);
    a->from = reinterpret_cast<int32_t*>(base + w.off_from);
    a->to = reinterpret_cast<int32_t*>(base + w.off_to);
    a->rank = reinterpret_cast<int32_t*>(base + w.off_rank);
    a->list = reinterpret_cast<int32_t*>(base + w.off_list);
    set_buffers(b, p, p);
    return TQ_OK;
}

}  // namespace

extern "C" {

size_t tq_int4_block_bytes(int head_dim, int group) {
    if (!head_dim_ok(head_dim) || !int4_group_ok(head_dim, group)) return 0;
    return (size_t)int4_block_bytes(head_dim, group);
}

size_t tq_int4_cache_bytes(int head_dim, int group, int64_t B, int64_t Hkv, int64_t Tcap) {
    if (B < 0 || Hkv < 0 || Tcap <= 0 || Tcap % kBlockT) return 0;
    return (size_t)(B * Hkv * (Tcap / kBlockT)) * tq_int4_block_bytes(head_dim, group);
}

tq_status tq_encode_int4(const tq_handle* h, int group, const void* x, tq_dtype dt, int64_t B, int64_t Hkv, int64_t T,
                         int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos, int64_t t0,
                         void* stream) {
    return copy_common(true, h, group, x, dt, B, Hkv, T, sb, sh, st, c, pos, t0, stream);
}

tq_status tq_expand_int4(const tq_handle* h, int group, void* x, tq_dtype dt, int64_t B, int64_t Hkv, int64_t T,
                         int64_t sb, int64_t sh, int64_t st, const tq_cache* c, const int32_t* pos, int64_t t0,
                         void* stream) {
    return copy_common(false, h, group, x, dt, B, Hkv, T, sb, sh, st, c, pos, t0, stream);
}

size_t tq_attend_int4_workspace_bytes(const tq_handle* h, int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv) {
    if (!h || B < 0 || Lq < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || !attend_sizes_ok(B, Lq, Hq, Hkv)) return 0;
    // (the largest over the query types)
    return attend_ws(h->d, h->num_sms, int4_slot_rows(h->d, TQ_BF16, (int)(Lq * (Hq / Hkv)))).bytes;
}

tq_status tq_attend_int4(const tq_handle* h, int group, const void* q, tq_dtype qdt, int64_t B, int64_t Lq, int64_t Hq,
                         const tq_cache* kc, const tq_cache* vc, const int32_t* seq_lens, int64_t T, float scale, void* out,
                         void* ws, size_t ws_bytes, void* stream) {
    Int4AttendArgs a{};
    bool empty;
    const tq_status r = prepare_attend(h, group, q, qdt, B, Lq, Hq, kc, vc, seq_lens, T, 0, scale, out, ws, ws_bytes, &a,
                                       &empty);
    if (r != TQ_OK || empty) return r;
    return cuda_status(launch_any(h, group, qdt, a, static_cast<cudaStream_t>(stream)));
}

tq_status tq_append_attend_int4(const tq_handle* h, int group, const void* k_new, const void* v_new, tq_dtype kv_dtype,
                                int64_t Lq, int64_t sb, int64_t sh, int64_t st, const tq_cache* kc, const tq_cache* vc,
                                const int32_t* pos, int64_t t0, const void* q, tq_dtype q_dtype, int64_t Hq, float scale,
                                void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!kc || !vc) return TQ_ERR_INVALID_ARG;
    Int4CopyArgs e{};
    Int4AttendArgs a{};
    bool empty;
    tq_status r = prepare_copy(h, group, k_new, kv_dtype, kc->B, kc->Hkv, Lq, sb, sh, st, kc, pos, t0, &e, 0, &empty);
    if (r == TQ_OK)
        r = prepare_copy(h, group, v_new, kv_dtype, kc->B, kc->Hkv, Lq, sb, sh, st, vc, pos, t0, &e, 1, &empty);
    if (r == TQ_OK)
        r = prepare_attend(h, group, q, q_dtype, kc->B, Lq, Hq, kc, vc, pos, t0, Lq, scale, out, ws, ws_bytes, &a, &empty);
    if (r != TQ_OK || empty) return r;
    if (caches_meet(h, group, kc, vc)) return TQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = launch_int4_encode(h->d, group, kv_dtype, e, h->num_sms, s);
    if (err == cudaSuccess) err = launch_any(h, group, q_dtype, a, s);
    return cuda_status(err);
}

size_t tq_pages_workspace_bytes(const tq_pages* p) {
    if (!p || p->pool_blocks <= 0 || p->pool_blocks >= ((int64_t)1 << 31)) return 0;
    return pages_ws(p->pool_blocks).bytes;
}

tq_status tq_pages_alloc(const tq_handle* h, const tq_pages* p, const int32_t* lo, const int32_t* hi, int32_t* info,
                         void* ws, size_t ws_bytes, void* stream) {
    PagesArgs a;
    PageBuffers b;
    bool empty;
    const tq_status r = prepare_pages_ws(h, p, ws, ws_bytes, &a, &b, &empty);
    if (r != TQ_OK) return r;
    if (!empty && (!lo || !hi || !aligned(lo, 4) || !aligned(hi, 4))) return TQ_ERR_INVALID_ARG;
    if (info && !aligned(info, 4)) return TQ_ERR_INVALID_ARG;
    return cuda_status(launch_pages_alloc(a, b, lo, hi, info, h->num_sms, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_fork(const tq_handle* h, const tq_pages* p, const int32_t* parent, void* stream) {
    PagesArgs a;
    bool empty;
    const tq_status r = prepare_pages(h, p, &a, &empty);
    if (r != TQ_OK || empty) return r;
    if (!parent || !aligned(parent, 4)) return TQ_ERR_INVALID_ARG;
    if (p->B > kMaxForkSequences || p->Hkv > 65535) return TQ_ERR_UNSUPPORTED;
    return cuda_status(launch_pages_fork(a, parent, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_free(const tq_handle* h, const tq_pages* p, const int32_t* keep, void* stream) {
    PagesArgs a;
    bool empty;
    const tq_status r = prepare_pages(h, p, &a, &empty);
    if (r != TQ_OK || empty) return r;
    if (!keep || !aligned(keep, 4)) return TQ_ERR_INVALID_ARG;
    return cuda_status(launch_pages_free(a, keep, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_compact(const tq_handle* h, const tq_pages* p, int32_t* info, void* ws, size_t ws_bytes, void* stream) {
    PagesArgs a;
    PageBuffers b;
    bool empty;
    const tq_status r = prepare_pages_ws(h, p, ws, ws_bytes, &a, &b, &empty);
    if (r != TQ_OK) return r;
    if (info && !aligned(info, 4)) return TQ_ERR_INVALID_ARG;
    return cuda_status(launch_pages_compact(a, b, info, h->num_sms, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_copy(const tq_handle* h, const tq_pages* from, const tq_pages* to, const int32_t* src,
                        const int32_t* dst, int64_t n, void* stream) {
    if (!h || !from || !to || n < 0 || from->pool_blocks <= 0 || to->pool_blocks <= 0 || !buffers_ok(from) ||
        !buffers_ok(to) || from->n_buffers != to->n_buffers)
        return TQ_ERR_INVALID_ARG;
    for (int i = 0; i < from->n_buffers; ++i)
        if (from->block_bytes[i] != to->block_bytes[i]) return TQ_ERR_INVALID_ARG;
    const tq_status r = device_ok(h);
    if (r != TQ_OK) return r;
    if (n == 0 || from->n_buffers == 0) return TQ_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || n >= ((int64_t)1 << 31)) return TQ_ERR_INVALID_ARG;
    PageBuffers b;
    set_buffers(&b, from, to);
    return cuda_status(launch_pages_copy(b, src, dst, n, from->pool_blocks, to->pool_blocks, h->derr, h->num_sms,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
