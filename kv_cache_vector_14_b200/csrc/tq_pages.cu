// Page operators of paged caches, for sm_100a: releasing, forking, supplying
// (with copy on write), compacting and copying pages, on the device, so that a
// captured serving step needs no host bookkeeping.  The state is the block
// table [B*Hkv][NB] (-1: no page) and a reference count per page (the number of
// table entries that name it; 0: free).  There is no free list to keep in step:
// free pages are found by counting over refs, lowest first, so the outcome does
// not depend on the order in which threads run.
//
// Every kernel is launched as a programmatic dependent of the one before it on the stream, lets
// the next one start and then waits for its predecessor to be complete: the launches' set-up
// overlaps (a fork with its supply for 64 sequences 16.4 -> 13.6 us).
//
// What bounds them: the bookkeeping reads the table rows concerned and refs
// (4 bytes a page) and is latency; the moved pages are read and written once.
// Measured: fork and supply for 64 sequences of 8198 tokens, 8 kv heads: 13.6 us in three
// launches; compaction of 49152 pages, a third live: 49 us with the two copies
// that put table and counts back, the moves 30 (the copy rate).  Supplying a whole prompt is
// far from that, a thread walks all blocks of its row: 32768 tokens of one sequence (8 rows,
// 4096 pages) with their release 174 us, of 16 sequences 423 us; a release alone 4.5 us.
#include "tq_pages.h"

namespace tqi {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ---------------------------------------------------------------- free
// Entries at logical blocks >= ceil(keep / 64) are released.
__global__ void __launch_bounds__(256) tq_pages_free_kernel(const PagesArgs a, const int32_t* keep) {
    pdl_trigger();
    pdl_wait();
    const int64_t n = a.B * a.Hkv * a.NB;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int64_t row = i / a.NB, lb = i - row * a.NB;
        const int64_t k = keep[row / a.Hkv];
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
    pdl_trigger();
    pdl_wait();
    const int x = threadIdx.x % kForkCols, y = threadIdx.x / kForkCols;
    const int64_t lb = (int64_t)blockIdx.x * kForkCols + x;
    for (int64_t b = y; b < a.B; b += 256 / kForkCols)
        tile[b * kForkCols + x] = lb < a.NB ? a.table[(b * a.Hkv + blockIdx.y) * a.NB + lb] : -1;
    __syncthreads();
    if (lb >= a.NB) return;
    for (int64_t b = y; b < a.B; b += 256 / kForkCols) {
        const int64_t p = parent[b];
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

// ---------------------------------------------------------------- plans
constexpr int kPlan = 1024;
// exclusive scan of v over the CTA of T threads; *total: the sum
template <int T = kPlan>
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
    int p = lane < T / 32 ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, p, o);
        if (lane >= o) p += x;
    }
    *total = __shfl_sync(kFull, p, 31);
    const int before = warp ? __shfl_sync(kFull, p, warp - 1) : 0;
    return before + incl - v;
}
// The pool in rounds of up to 64 pages per thread (65536 pages per round; thread t holds a run of
// `per` pages, ascending in t): bit i of the mask says whether pick(refs) holds for page p0 + i.
// One round's masks stay in registers, so a pool of that size is read once.
struct Runs {
    int64_t pool;
    int per;          // pages per thread and round, a multiple of 4
    int rounds;
    bool vec;         // refs on a 16-byte boundary
    __device__ explicit Runs(const PagesArgs& a) {
        pool = a.pool;
        const int64_t each = (pool + kPlan - 1) / kPlan;
        per = each < 64 ? (int)((each + 3) / 4 * 4) : 64;
        rounds = (int)((pool + (int64_t)per * kPlan - 1) / ((int64_t)per * kPlan));
        vec = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
    }
    __device__ int64_t first(int round) const { return ((int64_t)round * kPlan + threadIdx.x) * per; }
    template <typename Pick>
    __device__ uint64_t mask(const PagesArgs& a, int round, Pick pick) const {
        const int64_t p0 = first(round);
        uint64_t m = 0;
        if (vec && p0 + per <= pool) {
#pragma unroll 4
            for (int i = 0; i < per; i += 4) {
                const int4 r = *reinterpret_cast<const int4*>(a.refs + p0 + i);
                const uint32_t four = (uint32_t)pick(r.x) | (uint32_t)pick(r.y) << 1 | (uint32_t)pick(r.z) << 2 |
                                      (uint32_t)pick(r.w) << 3;
                m |= (uint64_t)four << i;
            }
        } else {
            for (int i = 0; i < per; ++i)
                if (p0 + i < pool && pick(a.refs[p0 + i])) m |= 1ull << i;
        }
        return m;
    }
};

// Tokens [lo, hi) of every sequence become writable: each of their blocks that has no page,
// or one that other entries name too, gets a fresh page.
__global__ void __launch_bounds__(kPlan) tq_pages_alloc_kernel(const PagesArgs a, const int32_t* lo, const int32_t* hi,
                                                               int32_t* info) {
    pdl_trigger();
    pdl_wait();
    const Runs runs(a);
    auto is_free = [](int r) { return r == 0; };
    const uint64_t free0 = runs.mask(a, 0, is_free);
    const int64_t rows = a.B * a.Hkv, per = (rows + kPlan - 1) / kPlan;
    const int64_t r0 = threadIdx.x * per < rows ? threadIdx.x * per : rows, r1 = r0 + per < rows ? r0 + per : rows;
    // the requests of this thread's rows, in (row, block) order: f(table index, entry)
    auto requests = [&](auto f) {
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t b = row / a.Hkv;
            int64_t l = lo[b], h = hi[b];
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
    // (up to two requests are kept: a decode step asks for one block per row)
    int mine = 0, R;
    int64_t at0 = 0, at1 = 0;
    int32_t e0 = 0, e1 = 0;
    requests([&](int64_t at, int32_t e) {
        if (mine == 0) { at0 = at; e0 = e; }
        if (mine == 1) { at1 = at; e1 = e; }
        ++mine;
    });
    int rank = scan_cta(mine, &R);
    // free pages, lowest first, as far as they are asked for
    int F = 0;
    for (int k = 0; k < runs.rounds; ++k) {
        uint64_t m = k == 0 ? free0 : runs.mask(a, k, is_free);
        int n;
        int at = F + scan_cta(__popcll(m), &n);
        for (; m && at < R; m &= m - 1, ++at) a.list[at] = (int32_t)(runs.first(k) + __ffsll((long long)m) - 1);
        F += n;
    }
    __syncthreads();
    const int got = R < F ? R : F;
    // (refs stay as they were until every request has been looked at again)
    auto give = [&](int64_t at, int32_t e) {
        if (rank < got) {
            const int32_t p = a.list[rank];
            a.from[rank] = e < 0 ? -1 : e;
            a.to[rank] = p;
            a.table[at] = p;
        }
        ++rank;
    };
    if (mine > 2) {
        requests(give);
    } else {
        if (mine > 0) give(at0, e0);
        if (mine > 1) give(at1, e1);
    }
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

// Compaction: the k-th lowest hole below the number of live pages takes the k-th highest live page.
// One CTA per segment of 2048 pages, 8 per thread: a first launch counts the live pages of every
// segment, a second adds up the counts before its segment and lists holes and far pages (one CTA
// alone took 24 to 36 us for 49152 pages; a single segment needs no first launch).  References and
// table follow in the move kernel.
constexpr int kSeg = 2048, kSegThreads = 256;
// live bits of this thread's 8 pages from p0 on
__device__ __forceinline__ uint32_t live8(const PagesArgs& a, int64_t p0) {
    uint32_t m = 0;
    if ((reinterpret_cast<uintptr_t>(a.refs) & 15) == 0 && p0 + 8 <= a.pool) {
        const int4 x = *reinterpret_cast<const int4*>(a.refs + p0), y = *reinterpret_cast<const int4*>(a.refs + p0 + 4);
        m = (uint32_t)(x.x > 0) | (uint32_t)(x.y > 0) << 1 | (uint32_t)(x.z > 0) << 2 | (uint32_t)(x.w > 0) << 3 |
            (uint32_t)(y.x > 0) << 4 | (uint32_t)(y.y > 0) << 5 | (uint32_t)(y.z > 0) << 6 | (uint32_t)(y.w > 0) << 7;
    } else {
        for (int i = 0; i < 8; ++i)
            if (p0 + i < a.pool && a.refs[p0 + i] > 0) m |= 1u << i;
    }
    return m;
}
__global__ void __launch_bounds__(kSegThreads) tq_pages_count_kernel(const PagesArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t p0 = (int64_t)blockIdx.x * kSeg + threadIdx.x * 8;
    int n;
    scan_cta<kSegThreads>(__popc(live8(a, p0)), &n);
    if (threadIdx.x == 0) a.list[blockIdx.x] = n;
}
__global__ void __launch_bounds__(kSegThreads) tq_pages_compact_kernel(const PagesArgs a, int32_t* info) {
    const int64_t s0 = (int64_t)blockIdx.x * kSeg, p0 = s0 + threadIdx.x * 8;
    pdl_trigger();
    pdl_wait();
    const uint32_t m = live8(a, p0);
    int n;
    const int mine = scan_cta<kSegThreads>(__popc(m), &n);
    int64_t L = n, first = 0;                          // live pages in all, and before this segment
    if (gridDim.x > 1) {
        int all = 0, low = 0;
        for (unsigned k = threadIdx.x; k < gridDim.x; k += kSegThreads) {
            const int c = a.list[k];
            all += c;
            low += k < blockIdx.x ? c : 0;
        }
        int t;
        scan_cta<kSegThreads>(all, &t);
        L = t;
        scan_cta<kSegThreads>(low, &t);
        first = t;
    }
    int64_t before = first + mine;                     // live pages below p
    int low = 0;                                       // live pages of this thread below L
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t p = p0 + i;
        if ((m >> i) & 1u) {
            if (p >= L) {
                const int64_t to = L - 1 - before;
                a.from[to] = (int32_t)p;
                a.rank[p] = (int32_t)to;
            } else {
                ++low;
            }
            ++before;
        } else if (p < L && p < a.pool) {
            a.to[p - before] = (int32_t)p;
        }
    }
    // the segment that holds page L (the last one where every page is live) knows the moves
    int under;
    scan_cta<kSegThreads>(low, &under);
    if (threadIdx.x == 0 && ((s0 <= L && L < s0 + kSeg) || (L == a.pool && blockIdx.x == gridDim.x - 1 && L == s0 + kSeg))) {
        const int32_t moves = (int32_t)(L - first - under);
        a.counts[0] = moves;
        a.counts[1] = (int32_t)L;
        if (info) {
            info[0] = (int32_t)(a.pool - L);
            info[1] = moves;
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

// moves from[k] -> to[k], k < *count (or n where count is null); remap: references and table
// entries of moved pages follow (compact)
__global__ void __launch_bounds__(256) tq_pages_move_kernel(const PageBuffers b, const int32_t* from, const int32_t* to,
                                                            const int32_t* count, int64_t n, int64_t pool_src,
                                                            int64_t pool_dst, const PagesArgs a, int remap) {
    pdl_trigger();
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
        for (int64_t k = blockIdx.x * 256ll + threadIdx.x; k < moves; k += gridDim.x * 256ll) {
            a.refs[to[k]] = a.refs[from[k]];           // (a page moves once: sources and destinations are distinct)
            a.refs[from[k]] = 0;
        }
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
    return launch_pdl(tq_pages_free_kernel, dim3((unsigned)(n < 65536 ? n : 65536)), dim3(256), 0, s, a, keep);
}

cudaError_t launch_pages_fork(const PagesArgs& a, const int32_t* parent, cudaStream_t s) {
    const size_t smem = (size_t)a.B * kForkCols * 4;
    const cudaError_t e = set_smem_once<tq_pages_fork_kernel>((int)(kMaxForkSequences * kForkCols * 4));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.NB + kForkCols - 1) / kForkCols), (unsigned)a.Hkv);
    return launch_pdl(tq_pages_fork_kernel, grid, dim3(256), smem, s, a, parent);
}

// blocks of a move kernel whose number of moves only the device knows: enough for a warp per page
// and buffer where there are few, four per SM at most
static unsigned move_grid(const PagesArgs& a, const PageBuffers& b, int num_sms) {
    const int64_t entries = a.B * a.Hkv * a.NB;
    const int64_t pages = entries < a.pool ? entries : a.pool;
    const int64_t need = (pages * (b.n > 0 ? b.n : 1) + 7) / 8, most = (int64_t)num_sms * 4;
    return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}

cudaError_t launch_pages_alloc(const PagesArgs& a, const PageBuffers& b, const int32_t* lo, const int32_t* hi, int32_t* info,
                               int num_sms, cudaStream_t s) {
    const cudaError_t e = launch_pdl(tq_pages_alloc_kernel, dim3(1), dim3(kPlan), 0, s, a, lo, hi, info);
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_pages_move_kernel, dim3(move_grid(a, b, num_sms)), dim3(256), 0, s, b, (const int32_t*)a.from,
                      (const int32_t*)a.to, (const int32_t*)a.counts, (int64_t)0, a.pool, a.pool, a, 0);
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PageBuffers& b, int32_t* info, int num_sms, cudaStream_t s) {
    const unsigned segments = (unsigned)((a.pool + kSeg - 1) / kSeg);
    cudaError_t e = cudaSuccess;
    if (segments > 1) {
        e = launch_pdl(tq_pages_count_kernel, dim3(segments), dim3(kSegThreads), 0, s, a);
        if (e == cudaSuccess) e = launch_pdl(tq_pages_compact_kernel, dim3(segments), dim3(kSegThreads), 0, s, a, info);
    } else {
        e = launch_pdl(tq_pages_compact_kernel, dim3(1), dim3(kSegThreads), 0, s, a, info);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_pages_move_kernel, dim3(move_grid(a, b, num_sms)), dim3(256), 0, s, b, (const int32_t*)a.from,
                      (const int32_t*)a.to, (const int32_t*)a.counts, (int64_t)0, a.pool, a.pool, a, 1);
}

cudaError_t launch_pages_copy(const PageBuffers& b, const int32_t* src, const int32_t* dst, int64_t n, int64_t pool_src,
                              int64_t pool_dst, int* err, int num_sms, cudaStream_t s) {
    PagesArgs a{};
    a.err = err;
    const int64_t need = (n * b.n + 7) / 8, most = (int64_t)num_sms * 8;
    return launch_pdl(tq_pages_move_kernel, dim3((unsigned)(need < most ? need : most)), dim3(256), 0, s, b, src, dst,
                      (const int32_t*)nullptr, n, pool_src, pool_dst, a, 0);
}

}  // namespace tqi
