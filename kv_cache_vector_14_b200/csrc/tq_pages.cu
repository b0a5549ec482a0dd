// Page operators of paged caches, for sm_100a: releasing, forking, supplying
// (with copy on write), compacting and copying pages, on the device, so that a
// captured serving step needs no host bookkeeping.  The state is the block
// table [B*Hkv][NB] (-1: no page) and a reference count per page (the number of
// table entries that name it; 0: free).  There is no free list to keep in step:
// free pages are found by counting over refs, lowest first, so the outcome does
// not depend on the order in which threads run.
//
// What bounds them: the bookkeeping reads the table rows concerned and refs
// (4 bytes a page) and is latency; the moved pages are read and written once.
#include "tq_pages.h"

namespace tqi {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ---------------------------------------------------------------- free
// Entries at logical blocks >= ceil(keep / 64) are released.
__global__ void __launch_bounds__(256) tq_pages_free_kernel(const PagesArgs a, const int32_t* keep) {
    const int64_t n = a.B * a.Hkv * a.NB;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int64_t row = i / a.NB, lb = i - row * a.NB;
        const int64_t k = __ldg(keep + row / a.Hkv);
        if (lb * kBlockT < k) continue;
        const int32_t e = a.table[i];
        if (e < 0) continue;
        if (e >= a.pool) {
            atomicExch(a.err, 1);
            continue;
        }
        a.table[i] = -1;
        atomicSub(a.refs + e, 1);
    }
}

// ---------------------------------------------------------------- fork
// Block (8 columns, kv head): the columns of all sequences are staged, then every
// sequence takes its parent's entries.  An entry that stays the same touches nothing.
constexpr int kForkCols = 8;
__global__ void __launch_bounds__(256) tq_pages_fork_kernel(const PagesArgs a, const int32_t* parent) {
    extern __shared__ int32_t tile[];                  // [B][kForkCols]
    const int x = threadIdx.x % kForkCols, y = threadIdx.x / kForkCols;
    const int64_t lb = (int64_t)blockIdx.x * kForkCols + x;
    for (int64_t b = y; b < a.B; b += 256 / kForkCols)
        tile[b * kForkCols + x] = lb < a.NB ? a.table[(b * a.Hkv + blockIdx.y) * a.NB + lb] : -1;
    __syncthreads();
    if (lb >= a.NB) return;
    for (int64_t b = y; b < a.B; b += 256 / kForkCols) {
        const int64_t p = __ldg(parent + b);
        if (p == b) continue;
        if (p < -1 || p >= a.B) {
            atomicExch(a.err, 1);
            continue;
        }
        const int32_t old = tile[b * kForkCols + x], now = p < 0 ? -1 : tile[p * kForkCols + x];
        if (old == now) continue;
        if (old >= a.pool || now >= a.pool) {
            atomicExch(a.err, 1);
            continue;
        }
        a.table[(b * a.Hkv + blockIdx.y) * a.NB + lb] = now < 0 ? -1 : now;
        if (old >= 0) atomicSub(a.refs + old, 1);
        if (now >= 0) atomicAdd(a.refs + now, 1);
    }
}

// ---------------------------------------------------------------- plans (one CTA)
constexpr int kPlan = 1024;
// exclusive scan of v over the CTA; *total: the sum
__device__ __forceinline__ int scan_cta(int v, int* total) {
    __shared__ int part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();                                   // part may still be read from an earlier scan
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int p = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, p, o);
        if (lane >= o) p += x;
    }
    *total = __shfl_sync(kFull, p, 31);
    const int before = warp ? __shfl_sync(kFull, p, warp - 1) : 0;
    return before + incl - v;
}
// Pages p of the warp's run of the pool, in order: f(p, refs, pages before p in the run that `pick` holds for)
template <typename Pick, typename F>
__device__ __forceinline__ int warp_run(const PagesArgs& a, Pick pick, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t per = ((a.pool + 31) / 32 + 31) / 32 * 32;
    const int64_t p0 = warp * per, p1 = p0 + per < a.pool ? p0 + per : a.pool;
    int n = 0;
    for (int64_t p = p0; p < p1; p += 32) {
        const bool in = p + lane < p1;
        const int r = in ? a.refs[p + lane] : 1;
        const bool yes = in && pick(r);
        const unsigned m = __ballot_sync(kFull, yes);
        if (in) f(p + lane, r, yes, n + __popc(m & ((1u << lane) - 1u)));
        n += __popc(m);
    }
    return n;
}

// Tokens [lo, hi) of every sequence become writable: each of their blocks that has no page,
// or one that other entries name too, gets a fresh page.
__global__ void __launch_bounds__(kPlan) tq_pages_alloc_kernel(const PagesArgs a, const int32_t* lo, const int32_t* hi,
                                                               int32_t* info) {
    const int64_t rows = a.B * a.Hkv, per = (rows + kPlan - 1) / kPlan;
    const int64_t r0 = threadIdx.x * per < rows ? threadIdx.x * per : rows, r1 = r0 + per < rows ? r0 + per : rows;
    // the requests of this thread's rows, in (row, block) order: f(table index, entry)
    auto requests = [&](auto f) {
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t b = row / a.Hkv;
            int64_t l = __ldg(lo + b), h = __ldg(hi + b);
            if (l < 0 || h > a.NB * kBlockT) {
                atomicExch(a.err, 1);
                l = l < 0 ? 0 : l;
                h = h > a.NB * kBlockT ? a.NB * kBlockT : h;
            }
            if (h <= l) continue;
            for (int64_t lb = l >> 6; lb <= (h - 1) >> 6; ++lb) {
                const int32_t e = a.table[row * a.NB + lb];
                if (e >= a.pool) {
                    atomicExch(a.err, 1);
                    continue;
                }
                if (e < 0 || a.refs[e] > 1) f(row * a.NB + lb, e);
            }
        }
    };
    int mine = 0, R, F;
    requests([&](int64_t, int32_t) { ++mine; });
    int rank = scan_cta(mine, &R);
    const int nf = warp_run(a, [](int r) { return r == 0; }, [](int64_t, int, bool, int) {});
    const int f0 = __shfl_sync(kFull, scan_cta((threadIdx.x & 31) == 0 ? nf : 0, &F), 0);
    warp_run(a, [](int r) { return r == 0; },
             [&](int64_t p, int, bool yes, int k) { if (yes && f0 + k < R) a.list[f0 + k] = (int32_t)p; });
    __syncthreads();
    const int got = R < F ? R : F;
    // (refs stay as they were until every request has been looked at again)
    requests([&](int64_t at, int32_t e) {
        if (rank < got) {
            const int32_t p = a.list[rank];
            a.from[rank] = e < 0 ? -1 : e;
            a.to[rank] = p;
            a.table[at] = p;
        }
        ++rank;
    });
    __syncthreads();
    int zeroed = 0;
    for (int k = threadIdx.x; k < got; k += kPlan) {
        a.refs[a.to[k]] = 1;
        if (a.from[k] >= 0 && atomicSub(a.refs + a.from[k], 1) == 1) ++zeroed;
    }
    int z;
    scan_cta(zeroed, &z);
    if (threadIdx.x == 0) {
        a.counts[0] = got;
        if (info) {
            info[0] = F - got + z;
            info[1] = R - got;
        }
    }
}

// The k-th lowest hole below the number of live pages takes the k-th highest live page.
__global__ void __launch_bounds__(kPlan) tq_pages_compact_kernel(const PagesArgs a, int32_t* info) {
    int L, n;
    auto live = [](int r) { return r > 0; };
    const int nl = warp_run(a, live, [](int64_t, int, bool, int) {});
    const int l0 = __shfl_sync(kFull, scan_cta((threadIdx.x & 31) == 0 ? nl : 0, &L), 0);
    int moves = 0;
    warp_run(a, live, [&](int64_t p, int, bool yes, int k) {
        const int before = l0 + k;                     // live pages below p
        if (!yes && p < L) a.to[p - before] = (int32_t)p;
        if (yes && p >= L) {
            const int m = L - 1 - before;
            a.from[m] = (int32_t)p;
            a.rank[p] = m;
            ++moves;
        }
    });
    scan_cta(moves, &n);                               // (its barriers order the lists as well)
    for (int k = threadIdx.x; k < n; k += kPlan) {
        a.refs[a.to[k]] = a.refs[a.from[k]];
        a.refs[a.from[k]] = 0;
    }
    if (threadIdx.x == 0) {
        a.counts[0] = n;
        a.counts[1] = L;
        if (info) {
            info[0] = (int32_t)(a.pool - L);
            info[1] = n;
        }
    }
}

// ---------------------------------------------------------------- moving pages
// One warp copies one page of one buffer at a time, 16 bytes a lane, kDeep of them in flight.
constexpr int kDeep = 8;
__device__ __forceinline__ void copy_page(const uint8_t* src, uint8_t* dst, uint32_t units) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    for (uint32_t i0 = threadIdx.x & 31; i0 < units; i0 += 32 * kDeep) {
        uint4 v[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (i0 + 32 * k < units) v[k] = s[i0 + 32 * k];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (i0 + 32 * k < units) d[i0 + 32 * k] = v[k];
    }
}

// moves from[k] -> to[k], k < *count (or n where count is null); table: entries of moved pages follow (compact)
__global__ void __launch_bounds__(256) tq_pages_move_kernel(const PageBuffers b, const int32_t* from, const int32_t* to,
                                                            const int32_t* count, int64_t n, int64_t pool_src,
                                                            int64_t pool_dst, const PagesArgs a, int remap) {
    pdl_wait();
    const int64_t warps = gridDim.x * 8ll, w = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int64_t moves = count ? (int64_t)count[0] : n;
    for (int64_t it = w; it < moves * b.n; it += warps) {
        const int64_t k = it / b.n;
        const int q = (int)(it - k * b.n);
        const int32_t s = from[k], d = to[k];
        if (s < 0 || d < 0) {
            if ((s < -1 || d < -1) && (threadIdx.x & 31) == 0) atomicExch(a.err, 1);
            continue;
        }
        if (s >= pool_src || d >= pool_dst) {
            if ((threadIdx.x & 31) == 0) atomicExch(a.err, 1);
            continue;
        }
        copy_page(b.src[q] + (int64_t)s * b.units[q] * 16, b.dst[q] + (int64_t)d * b.units[q] * 16, b.units[q]);
    }
    if (remap) {
        const int32_t L = a.counts[1];
        const int64_t entries = a.B * a.Hkv * a.NB;
        for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < entries; i += gridDim.x * 256ll) {
            const int32_t e = a.table[i];
            if (e < L) continue;
            // (a page that no count names cannot be followed)
            if (e >= a.pool || a.rank[e] < 0 || a.rank[e] >= moves || a.from[a.rank[e]] != e) {
                atomicExch(a.err, 1);
                continue;
            }
            a.table[i] = a.to[a.rank[e]];
        }
    }
}

}  // namespace

cudaError_t launch_pages_free(const PagesArgs& a, const int32_t* keep, cudaStream_t s) {
    const int64_t n = (a.B * a.Hkv * a.NB + 255) / 256;
    tq_pages_free_kernel<<<(unsigned)(n < 65536 ? n : 65536), 256, 0, s>>>(a, keep);
    return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesArgs& a, const int32_t* parent, cudaStream_t s) {
    const size_t smem = (size_t)a.B * kForkCols * 4;
    const cudaError_t e = set_smem_once<tq_pages_fork_kernel>((int)(kMaxForkSequences * kForkCols * 4));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.NB + kForkCols - 1) / kForkCols), (unsigned)a.Hkv);
    tq_pages_fork_kernel<<<grid, 256, smem, s>>>(a, parent);
    return cudaGetLastError();
}

cudaError_t launch_pages_alloc(const PagesArgs& a, const PageBuffers& b, const int32_t* lo, const int32_t* hi, int32_t* info,
                               int num_sms, cudaStream_t s) {
    tq_pages_alloc_kernel<<<1, kPlan, 0, s>>>(a, lo, hi, info);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_pages_move_kernel, dim3((unsigned)num_sms * 4), dim3(256), 0, s, b, (const int32_t*)a.from,
                      (const int32_t*)a.to, (const int32_t*)a.counts, (int64_t)0, a.pool, a.pool, a, 0);
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PageBuffers& b, int32_t* info, int num_sms, cudaStream_t s) {
    tq_pages_compact_kernel<<<1, kPlan, 0, s>>>(a, info);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_pages_move_kernel, dim3((unsigned)num_sms * 4), dim3(256), 0, s, b, (const int32_t*)a.from,
                      (const int32_t*)a.to, (const int32_t*)a.counts, (int64_t)0, a.pool, a.pool, a, 1);
}

cudaError_t launch_pages_copy(const PageBuffers& b, const int32_t* src, const int32_t* dst, int64_t n, int64_t pool_src,
                              int64_t pool_dst, int* err, int num_sms, cudaStream_t s) {
    PagesArgs a{};
    a.err = err;
    const int64_t need = (n * b.n + 7) / 8, most = (int64_t)num_sms * 8;
    tq_pages_move_kernel<<<(unsigned)(need < most ? need : most), 256, 0, s>>>(b, src, dst, nullptr, n, pool_src, pool_dst, a,
                                                                             0);
    return cudaGetLastError();
}

}  // namespace tqi
