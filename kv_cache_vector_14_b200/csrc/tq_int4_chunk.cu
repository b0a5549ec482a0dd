// Attention of many query rows over the 4-bit cache (prefill chunks, speculative
// tokens) on the 5th-generation tensor cores (tcgen05, accumulators, query
// operand and softmax weights in tensor memory), head_dim 64 and 128, for sm_100a.
//
// Mathematics as in tq_int4_attend.cu.  A unit is 128 MT query rows (query i,
// head g: row i G + g) of one kv head; its tokens come in tiles of 64, one cache
// block.  A tile is expanded once into shared memory and serves all rows:
//   S[128 rows][64] = Q K^T     (A: Q in shared memory, B: K, both K-major)
//   O[128 rows][D] += P V       (A: P in tensor memory over S, B: V, MN-major)
// The expanded values zero + scale c are rounded to fp16 (65504 at most), bf16 and fp16 queries enter
// exactly (scaled by a power of two per row), P is fp16.  For bf16 that is one product
// each (NL = 1): those roundings are 2^-11 relative and the output's own is 2^-8.  For
// fp16 and fp32 they would show, so K, V and P (and fp32 Q) are kept as fp16 hi + lo
// (NL = 2, 22 bits) and three products are summed, hi hi + lo hi + hi lo, in the same
// fp32 accumulator.
//
// Warp roles: warps 0-3 and 4-7 are two softmax streams, each with its own O
// accumulator and two score buffers; a thread owns a row.  With MT = 2 the streams
// are the two row tiles of the unit, and an expanded tile serves 256 rows; with MT = 1
// (few rows, or fp32 at head_dim 128, whose query limbs leave no shared memory) they
// take the even and the odd tiles and are merged at the unit's end.  Warps 8-11
// expand the blocks, warp 13 fills their ring (bulk copies), warp 12 issues the mma (its
// elected lane), the scores of the next tiles before the values of this one, so that softmax
// and tensor core overlap.  The mma of one
// thread run in issue order, so a score buffer is not overwritten before the product
// with the weights in it has run.  The reference exponent moves only when it is
// exceeded by 2^8 (two limbs: 2^2); then O is rescaled, once the stream's last product is done.
//
// Work: the units' tiles (each unit only as far as its last row sees) laid end
// to end, shared out evenly over one CTA per SM on the device, cut units merged
// by the combine kernel, as in tq_int4_attend.cu.
//
// Measured: 512 queries after 40448 tokens, 32/8 heads, d 128, bf16: 342 to 388 us with encode and
// read-back (0.88 to 1.0 PFLOP/s, 54 to 61 % of cuBLAS); a 256 x 64 tile takes about 2000 clocks, of
// which the tensor pipe and the exponentials fill half each.  What holds it are the softmax warps:
// their chain of waits, loads and stores, at 128 registers a thread (14 warps of equal share) of which
// this kernel spills 356 bytes; how much the spills take of it has not been separated.  The same
// 512 queries: d 128 fp16 1280, fp32 2520 us (three products of limbs); d 64 bf16 285, fp16 797, fp32
// 1093.  5 queries of 16 sequences at 4000 tokens, bf16: 50 us (20 of 128 rows used; a tile's softmax
// again).
//
// NaN: a value group with a non-finite pair is expanded as zeros, and the first
// such token of the segment is kept per group; rows that see it get NaN in that
// group at the end (a row sees a prefix of the tokens, so the first one decides).
// So a NaN does not reach the rows for which it is masked, as a product 0 NaN would.
#include <climits>
#include <type_traits>

#include "tq_frag.cuh"
#include "tq_int4.h"
#include "tq_int4_combine.cuh"
#include "tq_tc.cuh"

namespace tqi {
namespace {

constexpr int kSoft = 256;                // softmax threads: two streams x 128 rows
constexpr int kProd = 128;                // producer threads
constexpr int kThreads = kSoft + kProd + 64;
constexpr float kHuge = 3.40282347e38f;   // the largest finite fp32
constexpr int kSlots = 3;                 // ring of raw tiles (a K and a V block)
template <int D, int GRP, int NL, int QL, int MT>
struct Ch {
    static constexpr int kNG = D / GRP;
    static constexpr int TT = 64;                             // tokens per tile: one cache block
    static constexpr int kBufs = NL == 2 ? 2 : MT == 2 ? 3 : 5;   // operand buffers: what shared memory holds
    static constexpr int kBlockB = 64 * (D / 2 + 4 * kNG);
    static constexpr int kTile = TT * D * 2;                  // one fp16 operand of a tile
    static constexpr int kQ = 128 * D * 2;                    // one limb of a row tile's queries
    static constexpr int kBuf = 2 * NL * kTile;               // K limbs, V limbs
    static constexpr int kOffQ = kBufs * kBuf;                    // [MT][QL]
    static constexpr int kOffRing = kOffQ + MT * QL * kQ;
    static constexpr int kOffBar = kOffRing + kSlots * 2 * kBlockB;
    static constexpr int kOffXch = kOffBar + 38 * 8;          // [2][2][128]: reference, sum
    static constexpr int kOffBad = kOffXch + 4 * 128 * 4;     // [8 segments][4 groups]: first non-finite token
    static constexpr int kOffScan = kOffBad + 32 * 4;         // [kThreads / 32 + 3] int64
    static constexpr int kOffMisc = kOffScan + (kThreads / 32 + 3) * 8;
    static constexpr int kSmem = kOffMisc + 16 + 1024;        // + slack to align the base
    static_assert(kOffRing % 16 == 0 && kOffBar % 8 == 0 && kOffScan % 8 == 0, "alignment");
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    // tensor memory columns
    // Tiles of a segment.  The tensor core truncates its sums: an O of values with a mean loses up to
    // 5e-7 of itself per tile (3.5e-4 in 1100).  So O is taken out after 16 (fp32: 8e-6 of the result)
    // or 256 (fp16: 1.3e-4, a quarter of the half step) of a stream's tiles and added up in the workspace,
    // correctly rounded; a take-out costs 20 to 40 us (loads, stores and a drained pipeline).  bf16 calls go without: their half step is reached in some 10000 tiles of one
    // CTA (include/tq.h says so), and the code alone costs the 512-token step 3 %.
    static constexpr bool kTakeOut = NL == 2;
    static constexpr int kSegStream = !kTakeOut ? INT_MAX / 4 : QL == 2 ? 16 : 256;
    static constexpr int kSegTiles = MT == 2 ? kSegStream : 2 * kSegStream;
    static constexpr int kX = 0;                              // S / P of stream x, buffer b at TT (2 x + b)
    static constexpr int kO = 4 * TT;                         // O of stream x at kO + D x
    static_assert(kO + 2 * D <= 512, "tensor memory");
};

// mbarriers.  A barrier is never two phases ahead of a thread that waits on it: whatever a
// stream's two score buffers allow to run ahead has a barrier per buffer.
enum : int {
    kBarRing = 0,      // [3] a tile's raw K and V blocks in their slot (copy bytes)
    kBarSlot = 3,      // [3] a slot read (kProd arrivals)
    kBarReady = 6,     // [5] operands of a buffer built (kProd arrivals)
    kBarFree = 11,     // [5] operands of a buffer read (commit)
    kBarS = 16,        // [2][2] S of stream x, score buffer b computed (commit)
    kBarP = 20,        // [2][2] P of stream x in score buffer b written (128 arrivals)
    kBarO = 24,        // [2] O of stream x updated (commit)
    kBarSeg = 26,      // O of a segment complete (commit), and the mma warp's own arrival
    kBarQ = 27,        // query operand written (256 arrivals)
    kBarDrain = 28,    // every mma done (commit, at exit)
};

// tokens that the last row of row tile rt sees, and the tiles they take (at least one)
__device__ __forceinline__ int64_t chunk_len(const Int4AttendArgs& a, int64_t b) {
    const int64_t n = (a.lens ? (int64_t)a.lens[b] : a.T) + a.add;
    return n < 0 ? 0 : (n > a.Tcap ? a.Tcap : n);
}
template <int ROWS, int TT>
__device__ __forceinline__ int unit_tiles(const Int4AttendArgs& a, int64_t n, int rt) {
    const int64_t last = (int64_t)rt * ROWS + ROWS - 1 < a.rows ? (int64_t)rt * ROWS + ROWS - 1 : a.rows - 1;
    const int64_t sees = n - a.Lq + 1 + last / a.G;
    const int64_t t = (sees + TT - 1) / TT;
    return t > 1 ? (int)t : 1;
}

// Walks the flattened tiles: (sequence, row tile) pair, kv head, tile.
template <int ROWS, int TT>
struct Walk {
    int64_t n;         // tokens of the sequence
    int b, rt, kv, k, nt, R;
    __device__ void load(const Int4AttendArgs& a) {
        n = chunk_len(a, b);
        nt = unit_tiles<ROWS, TT>(a, n, rt);
    }
    __device__ void next(const Int4AttendArgs& a) {
        if (++k < nt) return;
        k = 0;
        if (++kv < (int)a.Hkv) return;
        kv = 0;
        if (++rt == R) {
            rt = 0;
            if (++b == (int)a.B) { b = 0; return; }           // behind the last tile: not used
        }
        load(a);
    }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(kFull, mbar_wait_bounded(bar, parity));
}
// mma and commit by the warp's elected lane, called by the whole warp: the operands are then
// warp-uniform to the compiler and stay in uniform registers (one diverged thread issued an
// mma every 80 to 100 clocks, more than it takes to run)
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// barrier over the softmax threads that ORs v
__device__ __forceinline__ bool soft_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(kSoft)
        : "memory");
    return r != 0;
}
template <int DT>
__device__ __forceinline__ void put_elem(void* p, int64_t i, float x) {
    if constexpr (DT == TQ_F32) static_cast<float*>(p)[i] = x;
    else if constexpr (DT == TQ_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half*>(p)[i] = __float2half_rn(x);
}
// Operand position p (0 .. 7) of a word's eight values holds value word_value(p): the
// order in which masks pick nibbles r and r + 4
__host__ __device__ constexpr int word_value(int p) { return (p >> 1) + 4 * (p & 1); }

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// The eight values of word w, zero + scale c, as four fp16 pairs: hi, and with NL = 2 lo, what the
// value lies above it.  The scale is a rounded number, so the top of a group may lie above 65504, by
// 15 scale 2^-11 <= 64, where the mma needs a finite hi.  NL = 1: TOP keeps it at 65504.  NL = 2: s2
// is one unit lower then, and lo, from the exact pair, carries the difference (at most 120).
template <int NL, bool TOP>
__device__ __forceinline__ void expand_word(uint32_t w, __half2 s2, __half2 z2, __half2 pair, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const uint32_t w8 = w >> 8;
    const __half2 m1024 = as_h2(0xe400e400u), sixteenth = as_h2(0x2c002c00u), m64 = as_h2(0xd400d400u);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t v = r < 2 ? w : w8;
        // 1024 + c (or 1024 + 16 c) as fp16, then c exactly, then one rounding of zero + scale c
        const __half2 c = (r & 1) ? __hfma2(as_h2((v & 0x00f000f0u) | 0x64006400u), sixteenth, m64)
                                  : __hadd2(as_h2((v & 0x000f000fu) | 0x64006400u), m1024);
        __half2 h = __hfma2(c, s2, z2);
        if constexpr (TOP) h = __hmin2_nan(h, as_h2(0x7bff7bffu));
        hi[r] = h2_bits(h);
        if constexpr (NL == 2) {
            const float2 cf = __half22float2(c), hf = __half22float2(h);
            const float s = __low2float(pair), z = __high2float(pair);
            lo[r] = h2_bits(__floats2half2_rn(fmaf(cf.x, s, z) - hf.x, fmaf(cf.y, s, z) - hf.y));
        }
    }
}

// packed fp32 pairs
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// N consecutive elements of a row as stored (zeros where there is no row); vec: the row is 16-byte aligned
template <int DT, int N>
__device__ __forceinline__ void load_raw(const void* p, int64_t at, bool vec, bool there, uint32_t (&w)[N * (DT == TQ_F32 ? 4 : 2) / 4]) {
    constexpr int kE = DT == TQ_F32 ? 4 : 2, kN = N * kE / 4;
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = 0u;
    if (!there) return;
    const char* s = static_cast<const char*>(p) + at * kE;
    if (vec) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(s)[i];
            w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
        }
    } else if constexpr (DT == TQ_F32) {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = reinterpret_cast<const uint32_t*>(s)[i];
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(s);
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
    }
}
template <int DT, int N>
__device__ __forceinline__ float raw_elem(const uint32_t (&w)[N], int e) {
    if constexpr (DT == TQ_F32) return __uint_as_float(w[e]);
    else if constexpr (DT == TQ_BF16) return __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    else return (e & 1) ? __high2float(as_h2(w[e >> 1])) : __low2float(as_h2(w[e >> 1]));
}
// eight consecutive outputs
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, bool vec, const float (&v)[8]) {
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) put_elem<DT>(p, at + i, v[i]);
    } else if constexpr (DT == TQ_F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == TQ_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                w[k] = h2_bits(__floats2half2_rn(v[2 * k], v[2 * k + 1]));
            }
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(p) + at * 2) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int D, int GRP, int DT, int MT>
__global__ void __launch_bounds__(kThreads, 1) tq_int4_chunk_kernel(const __grid_constant__ Int4AttendArgs a) {
    constexpr int NL = DT == TQ_BF16 ? 1 : 2;                 // limbs of K, V and P
    constexpr int QL = DT == TQ_F32 ? 2 : 1;                  // limbs of Q
    constexpr int ROWS = 128 * MT;
    // P is kept below 2^15 (fp16 holds 65504); two limbs need the room (see tq_int4_attend.cu)
    constexpr float kRoom = NL == 1 ? 7.f : 13.f, kLazy = 15.f - kRoom;
    using C = Ch<D, GRP, NL, QL, MT>;
    constexpr int NG = C::kNG, TT = C::TT;
    using W = Walk<ROWS, TT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    int64_t* sScan = reinterpret_cast<int64_t*>(sm + C::kOffScan);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = kThreads / 32;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bar(kBarRing + i), 1);
            mbar_init(bar(kBarSlot + i), kProd);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(bar(kBarReady + i), kProd);
            mbar_init(bar(kBarFree + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarO + i), 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(bar(kBarS + 2 * i + b), 1);
                mbar_init(bar(kBarP + 2 * i + b), 128);
            }
        }
        mbar_init(bar(kBarSeg), 2);
        mbar_init(bar(kBarQ), kSoft);
        mbar_init(bar(kBarDrain), 1);
        fence_mbar_init();
    }
    int* sBad = reinterpret_cast<int*>(sm + C::kOffBad);
    if (tid < 32) sBad[tid] = INT_MAX;
    if (warp == 0) {
        tc_alloc(smem_u32(tmem_slot), 512);
        tc_relinquish();
    }
    pdl_wait();

    // ---------------- this CTA's share of the tiles: pairs (sequence, row tile) in order, each
    // Hkv units of unit_tiles tiles; a scan over runs of pairs finds the place
    const int R = (a.rows + ROWS - 1) / ROWS;
    const int64_t pairs = a.B * R, per = (pairs + kThreads - 1) / kThreads;
    const int64_t p0 = tid * per < pairs ? tid * per : pairs, p1 = p0 + per < pairs ? p0 + per : pairs;
    auto span_of = [&](int64_t p) -> int64_t {
        const int64_t b = p / R;
        return (int64_t)unit_tiles<ROWS, TT>(a, chunk_len(a, b), (int)(p - b * R)) * a.Hkv;
    };
    int64_t mine = 0;
    for (int64_t p = p0; p < p1; ++p) mine += span_of(p);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sScan[warp] = incl;
    tc_fence_before();
    __syncthreads();                       // (also: mbarriers and tensor memory are set up)
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int64_t before = 0, N = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sScan[w];
        N += sScan[w];
    }
    const int64_t c = blockIdx.x, nC = N < gridDim.x ? N : gridDim.x;
    const int64_t lo = c < nC ? c * N / nC : 0;
    {
        int64_t base = before + incl - mine;
        if (base <= lo && lo < base + mine)
            for (int64_t p = p0; p < p1; ++p) {
                const int64_t span = span_of(p);
                if (lo < base + span) {
                    sScan[kWarps] = p;
                    sScan[kWarps + 1] = lo - base;
                    break;
                }
                base += span;
            }
    }
    __syncthreads();
    if (tid == 0) a.split[c] = make_int4(0, 0, 0, 0);
    const int J = c < nC ? (int)((c + 1) * N / nC - lo) : 0;  // tiles of this CTA
    W w0;
    w0.R = R;
    w0.b = (int)(sScan[kWarps] / R);
    w0.rt = (int)(sScan[kWarps] - (int64_t)w0.b * R);
    w0.load(a);
    w0.kv = (int)(sScan[kWarps + 1] / w0.nt);
    w0.k = (int)(sScan[kWarps + 1] - (int64_t)w0.kv * w0.nt);

    bool failed = false;
    if (warp < 8) {
        // ======================================== softmax: stream x, thread = row r of its row tile
        const int x = warp >> 2, r = tid & 127;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float* xch = reinterpret_cast<float*>(sm + C::kOffXch);
        // values of a row that this thread loads and stores
        constexpr int kCols = MT == 2 ? D : D / 2;
        const int col0 = MT == 2 ? 0 : x * kCols;
        W w = w0;
        int seg = 0, nS = 0;                                  // segments, S of this stream so far
        bool cont = false, ubegins = false;                   // the unit has a part in the workspace; it begins in this CTA
        float fr = 0.f, mrun = -INFINITY, lrun = 0.f;         // its score factor, and that part's reference and sum
        for (int j = 0; j < J; ++seg) {
            // ---- a segment: tiles j .. j1 - 1 of one unit
            const int k0 = w.k, left = w.nt - w.k;
            const int most = left < C::kSegTiles ? left : C::kSegTiles;
            const int j1 = j + most < J ? j + most : J;
            if (!C::kTakeOut || !cont) ubegins = k0 == 0;
            const int ur = MT == 2 ? 128 * x + r : r;         // row of the unit
            const int64_t grow = (int64_t)w.rt * ROWS + ur;
            const bool rvalid = grow < a.rows;
            const int64_t qi = rvalid ? grow / a.G : 0, qg = rvalid ? grow - qi * a.G : 0;
            const int64_t qrow = ((int64_t)w.b * a.Lq + qi) * a.Hq + (int64_t)w.kv * a.G + qg;
            // tokens that the row sees, clamped to 32 bits (a row that is not there sees everything: no
            // masking for it, and nothing of it is stored)
            const int64_t lim64 = rvalid ? w.n - a.Lq + 1 + qi : INT_MAX;
            const int lim = lim64 < 0 ? 0 : (int)lim64;
            // query operand: the row scaled by a power of two (largest element in [2^14, 2^15));
            // position p of a word's eight holds value word_value(p), as in the expanded operands
            if (!C::kTakeOut || !cont) {
                // (all loads at once; 64 registers with MT = 2)
                constexpr int kRegs = kCols * (DT == TQ_F32 ? 4 : 2) / 4;
                uint32_t raw_q[kRegs];
                load_raw<DT, kCols>(a.q, qrow * D + col0, a.vec16, rvalid, raw_q);
                float mx = 0.f;
#pragma unroll
                for (int e = 0; e < kCols; ++e) {
                    const float v = fabsf(raw_elem<DT>(raw_q, e));
                    mx = fmaxf(mx, v <= kHuge ? v : INFINITY); // (a NaN counts as infinite)
                }
                if constexpr (MT == 1) {
                    xch[x * 128 + r] = mx;
                    soft_or(false);
                    mx = fmaxf(mx, xch[(x ^ 1) * 128 + r]);
                }
                int ex = mx > 0.f && mx <= kHuge ? ilogbf(mx) : 0;
                ex = ex < -100 ? -100 : ex;
                const float f = mx <= kHuge ? exp2f((float)(14 - ex)) : 1.f;
                const float fs = a.scale_log2 < 0.f ? -f : f;
                // (above zero: a masked -inf stays one; a query with an infinity or a NaN makes its row NaN)
                fr = mx <= kHuge ? fmaxf(fabsf(a.scale_log2) / f, 1e-37f) : __int_as_float(0x7fc00000);
                uint8_t* sq = sm + C::kOffQ + (MT == 2 ? x * QL * C::kQ : 0);
#pragma unroll
                for (int i = 0; i < kCols; i += 8) {           // eight positions, 16 bytes
                    uint32_t qh[4], qlo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        split_hilo(raw_elem<DT>(raw_q, i + word_value(2 * k)) * fs, raw_elem<DT>(raw_q, i + word_value(2 * k + 1)) * fs,
                                   qh[k], qlo[k]);
                    const uint32_t at = sw128_byte(r, 2 * (col0 + i), 128);
                    *reinterpret_cast<uint4*>(sq + at) = make_uint4(qh[0], qh[1], qh[2], qh[3]);
                    if constexpr (QL == 2) *reinterpret_cast<uint4*>(sq + C::kQ + at) = make_uint4(qlo[0], qlo[1], qlo[2], qlo[3]);
                }
                fence_proxy_async();
            }
            mbar_arrive(bar(kBarQ));
            float mref = -INFINITY, lsum = 0.f;
            bool any = false;                                  // this stream has an O
            const bool idle = !__any_sync(kFull, rvalid);      // none of the warp's rows is there
            const uint64_t fr2 = pack2(fr, fr);
            for (int jj = MT == 2 ? j : j + ((j & 1) ^ x); jj < j1 && !failed; jj += 3 - MT) {
                const int b = 2 * x + (nS & 1);                // score buffer
                const uint32_t tx = tl + C::kX + TT * b;
                const int64_t rest = (int64_t)lim - (int64_t)(k0 + (jj - j)) * TT;
                const int vis = rest >= TT ? TT : (int)(rest > 0 ? rest : 0);
                if (!warp_wait(bar(kBarS + b), (uint32_t)((nS >> 1) & 1))) { failed = true; break; }
                ++nS;
                tc_fence_after();
                if (idle) {                                    // P of these rows may be anything: O's other rows do not see it
                    tc_fence_before();
                    mbar_arrive(bar(kBarP + b));
                    continue;
                }
                uint32_t sv[TT];
                tc_ld64(tx, sv);
                if (vis < TT) {
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        if (t >= vis) sv[t] = 0xff800000u;
                }
                // P = 2^(S fr - mref) over S (tokens 2 i, 2 i + 1 in column i; NL = 2: low limbs in
                // column 32 + i), and its sum; 16 tokens at a time (fewer registers)
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto weights = [&](float m) -> float {
                    const uint64_t m2 = pack2(-m, -m);
                    uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                    for (int qt = 0; qt < 4; ++qt) {
                        uint32_t ph[8], pl[8];
#pragma unroll
                        for (int t = 0; t < 16; t += 2) {
                            const float a0 = __uint_as_float(sv[16 * qt + t]), a1 = __uint_as_float(sv[16 * qt + t + 1]);
                            mx4[(t >> 1) & 3] = fmaxf(mx4[(t >> 1) & 3], fmaxf(a0, a1));
                            float e0, e1;
                            unpack2(fma2(pack2(a0, a1), fr2, m2), e0, e1);
                            e0 = fast_exp2(e0);
                            e1 = fast_exp2(e1);
                            sum2[(t >> 1) & 1] = add2(sum2[(t >> 1) & 1], pack2(e0, e1));
                            if constexpr (NL == 2) split_hilo(e0, e1, ph[t >> 1], pl[t >> 1]);
                            else ph[t >> 1] = h2_bits(__floats2half2_rn(e0, e1));
                        }
                        tc_st8(tx + 8 * qt, ph);
                        if constexpr (NL == 2) tc_st8(tx + 32 + 8 * qt, pl);
                    }
                    float s0, s1;
                    unpack2(add2(sum2[0], sum2[1]), s0, s1);
                    return s0 + s1;
                };
                // The weights are taken with the reference as it is, the maximum beside them (off the
                // critical path); where the reference turns out exceeded by 2^kLazy (always in a unit's
                // first tile) it moves, O is rescaled by whole warps and the weights are taken again.
                float sum = weights(mref == -INFINITY ? 0.f : mref);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fr;
                const bool move = mx - kRoom - kLazy > mref;
                if (__any_sync(kFull, move)) {
                    float f = 1.f;
                    if (move) {
                        f = mref == -INFINITY ? 0.f : fast_exp2(mref - (mx - kRoom));
                        mref = mx - kRoom;
                        lsum *= f;
                    }
                    if (any) {
                        // the product with the stream's tile before (its product nS - 2) is done
                        if (!warp_wait(bar(kBarO + x), (uint32_t)(nS & 1))) { failed = true; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            uint32_t ov[16];
                            tc_ld16(tl + C::kO + D * x + c0, ov);
#pragma unroll
                            for (int cc = 0; cc < 16; ++cc) ov[cc] = __float_as_uint(__uint_as_float(ov[cc]) * f);
                            tc_st16(tl + C::kO + D * x + c0, ov);
                        }
                    }
                    sum = weights(mref == -INFINITY ? 0.f : mref);
                }
                any = true;
                lsum += sum;
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(bar(kBarP + b));
            }
            // ---- the segment's end
            if (!failed && !warp_wait(bar(kBarSeg), (uint32_t)(seg & 1))) failed = true;
            tc_fence_after();
            if (!any) mref = -INFINITY;
            if (lim == 0) {                                    // sees nothing: zeros, whatever its query
                mref = -INFINITY;
                lsum = 0.f;
            }
            // groups with a non-finite pair on a token that this row sees
            uint32_t bad = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) bad |= (uint32_t)(sBad[4 * (seg & 7) + g] < lim) << g;
            if (lsum != lsum && mref == -INFINITY) mref = 0.f;   // nothing but NaN scores
            if constexpr (MT == 1) {
                xch[x * 128 + r] = mref;
                xch[(2 + x) * 128 + r] = lsum;
            }
            if (soft_or(failed)) failed = true;
            const bool ends = j1 - j == left, whole = ubegins && ends;
            const int64_t slot = (2 * c + (ubegins ? 1 : 0)) * ROWS + ur;
            // MT = 1: both streams' results, each stream half of the coordinates
            float m0 = mref, m1 = -INFINITY, l0 = lsum, l1 = 0.f;
            if constexpr (MT == 1) {
                m0 = xch[r];
                m1 = xch[128 + r];
                l0 = xch[2 * 128 + r];
                l1 = xch[3 * 128 + r];
            }
            if (!cont) { mrun = -INFINITY; lrun = 0.f; }
            const float mm = failed ? -INFINITY : fmaxf(fmaxf(m0, m1), mrun);
            const float f0 = m0 == -INFINITY || failed ? 0.f : fast_exp2(m0 - mm);
            const float f1 = m1 == -INFINITY || failed ? 0.f : fast_exp2(m1 - mm);
            const float f2 = mrun == -INFINITY || failed ? 0.f : fast_exp2(mrun - mm);
            // (a sum that is NaN stays in L though its factor is 0; one without a token is 0)
            const float L = mm == -INFINITY ? 0.f : fmaf(f1, l1, fmaf(f0, l0, f2 * lrun));
            const float inv = whole && mm != -INFINITY ? 1.f / L : 1.f;
            float* part = a.part_acc + (slot - ur) * D + ur;   // [D][ROWS]: the lanes of a store are neighbours
            // eight columns of this segment, in value order
            auto take = [&](int col, float (&v)[8]) {
                uint32_t o0[8], o1[8];
                tc_ld8(tl + C::kO + (MT == 2 ? D * x : 0) + col, o0);
                if constexpr (MT == 1) tc_ld8(tl + C::kO + D + col, o1);
                const bool poison = (bad >> (col / GRP)) & 1u; // (a run of 8 lies in one group)
#pragma unroll
                for (int cc = 0; cc < 8; ++cc) {
                    float y = f0 != 0.f ? __uint_as_float(o0[cc]) * f0 : 0.f;
                    if constexpr (MT == 1) y = f1 != 0.f ? fmaf(__uint_as_float(o1[cc]), f1, y) : y;
                    v[word_value(cc)] = poison && mm != -INFINITY ? __uint_as_float(0x7fc00000u) : y;
                }
            };
            auto put = [&](int col, const float (&v)[8]) {
                if (!rvalid) return;
                if (whole) {
                    store8<DT>(a.out, qrow * D + col, a.vec16, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) part[(int64_t)(col + e) * ROWS] = v[e];
                }
            };
            if (C::kTakeOut && cont) {
                // beside what this thread stored there (0 NaN stays NaN), in a loop of its own: one loop for
                // both cost 8 % of a call that takes nothing out.  32 columns in flight, 8 where more
                // registers cost the tiles' loop (512-token step, fp32, head_dim 128: 2640 -> 2525 us)
                constexpr int kStep = D == 128 ? 32 : 8;
#pragma unroll 1
                for (int c0 = 0; c0 < kCols; c0 += kStep) {
                    float pv[kStep];
#pragma unroll
                    for (int e = 0; e < kStep; ++e) pv[e] = rvalid ? part[(int64_t)(col0 + c0 + e) * ROWS] : 0.f;
#pragma unroll
                    for (int q = 0; q < kStep / 8; ++q) {
                        float v[8];
                        take(col0 + c0 + 8 * q, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = fmaf(pv[8 * q + e], f2, v[e]) * inv;
                        put(col0 + c0 + 8 * q, v);
                    }
                }
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < kCols; c0 += 8) {
                    float v[8];
                    take(col0 + c0, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= inv;
                    put(col0 + c0, v);
                }
            }
            if (rvalid && !whole && (MT == 2 || x == 0)) {
                a.part_ml[2 * slot] = mm;
                a.part_ml[2 * slot + 1] = L;
            }
            // a unit that begins here and goes on behind this CTA: up to the CTA of its last tile
            if (tid == 0 && ubegins && !ends && j1 == J) {
                const int64_t end = lo + j + left;             // (flattened index behind its last tile)
                a.split[c] = make_int4(w.b, w.rt * (int)a.Hkv + w.kv, (int)((end * nC - 1) / N), 1);
            }
            // the next segment's queries and exchange overwrite what was read here (the marks of
            // this segment's slot are next used eight segments on; producers are at most kBufs ahead)
            if (tid < 4) sBad[4 * (seg & 7) + tid] = INT_MAX;
            tc_fence_before();
            soft_or(false);
            tc_fence_after();
            if constexpr (C::kTakeOut) {
                cont = !ends;
                mrun = mm;
                lrun = L;
            }
            w.k += j1 - j - 1;                                 // on to the next segment
            w.next(a);
            j = j1;
        }
        if (failed) atomicExch(a.err, 1);
    } else if (warp < 12) {
        // ======================================== producers: K, then V block of a tile; thread =
        // token `tau0` (D = 128: and tau0 + 32) of piece cp (32 values)
        const int pw = warp - 8;
        W w = w0;
        constexpr int kPieces = D / 32, kItems = 64 * kPieces / kProd;   // items per block and thread
        const int cp = pw % kPieces, tau0 = lane + 32 * (pw / kPieces);
        const int src = tau0 * (D / 2) + ((cp * 16) ^ int4_swizzle(D, tau0));
        const int gam = cp * 32 / GRP;
        const int prs = 64 * (D / 2) + (tau0 * NG + gam) * 4;
        uint32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = sw128_byte(tau0, 2 * (32 * cp + 8 * i), TT);
        // (no warp-collective instruction here: a thread whose wait runs out leaves, the others follow)
        int slot = 0, sp = 0, bf = 0, bfp = 0;                 // ring slot and buffer, with their phases
        int seg = 0, inseg = 0;                                // segment, tiles of it
        for (int j = 0; j < J; ++j) {
            if (!mbar_wait_bounded(bar(kBarRing + slot), (uint32_t)sp)) { failed = true; break; }
            const uint8_t* raw_blk = sm + C::kOffRing + slot * 2 * C::kBlockB;
            const int64_t tok0 = (int64_t)w.k * TT, inside = w.n - tok0;
            const int valid = inside < TT ? (int)(inside > 0 ? inside : 0) : TT;           // tokens inside the sequence
            // items: K, then V
            uint4 v[2 * kItems];
            uint32_t bits[2 * kItems], high[2 * kItems];       // pairs; and those of hi (see expand_word)
            bool rare = false;
#pragma unroll
            for (int it = 0; it < 2 * kItems; ++it) {
                const uint8_t* blk = raw_blk + (it / kItems) * C::kBlockB;
                const int dt = 32 * (it % kItems);
                v[it] = *reinterpret_cast<const uint4*>(blk + src + dt * (D / 2));
                bits[it] = *reinterpret_cast<const uint32_t*>(blk + prs + dt * NG * 4);
                if (tau0 + dt >= valid) bits[it] = 0u;         // behind the sequence anything may stand
                // a scale of 2^11 or more, a zero of 2^15 or more, infinity or NaN
                rare |= (bits[it] & 0x7fffu) >= 0x6800u || (bits[it] & 0x7fff0000u) >= 0x78000000u;
                high[it] = bits[it];
            }
            if (j >= C::kBufs && !mbar_wait_bounded(bar(kBarFree + bf), (uint32_t)(bfp ^ 1))) { failed = true; break; }
            if (rare) {                                        // (after the wait: it bounds how far ahead marks are made)
#pragma unroll
                for (int it = 0; it < 2 * kItems; ++it) {
                    if ((bits[it] & 0x7c00u) == 0x7c00u || (bits[it] & 0x7c000000u) == 0x7c000000u) {
                        bits[it] = it < kItems ? 0x7e007e00u : 0u;     // a key: NaN, whatever its codes
                        if (it >= kItems) atomicMin(&sBad[4 * (seg & 7) + gam], (int)tok0 + tau0 + 32 * (it % kItems));
                    }
                    high[it] = bits[it];
                    if (NL == 2 && fmaf(15.f, __low2float(as_h2(bits[it])), __high2float(as_h2(bits[it]))) > 65504.f) high[it] -= 1u;
                }
            }
            uint8_t* buf = sm + bf * C::kBuf;
            auto build = [&](auto top) {
#pragma unroll
                for (int it = 0; it < 2 * kItems; ++it) {
                    const __half2 s2 = __low2half2(as_h2(high[it])), z2 = __high2half2(as_h2(high[it]));
                    const uint32_t wd[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
                    uint8_t* op = buf + (it / kItems) * NL * C::kTile + 32 * (it % kItems) * 128;    // (32 rows: 4 atoms of 1024 bytes)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4], l[4];
                        expand_word<NL, decltype(top)::value>(wd[i], s2, z2, as_h2(bits[it]), h, l);
                        *reinterpret_cast<uint4*>(op + at[i]) = make_uint4(h[0], h[1], h[2], h[3]);
                        if constexpr (NL == 2) *reinterpret_cast<uint4*>(op + C::kTile + at[i]) = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                }
            };
            build(std::false_type{});
            if (NL == 1 && rare) build(std::true_type{});      // again over it (512-token step 345 us; as an else branch 349)
            fence_proxy_async();           // operands for the tensor core; the slot's reads before its next copies
            mbar_arrive(bar(kBarReady + bf));
            mbar_arrive(bar(kBarSlot + slot));
            if (++slot == kSlots) { slot = 0; sp ^= 1; }
            if (++bf == C::kBufs) { bf = 0; bfp ^= 1; }
            if (++inseg == C::kSegTiles || w.k == w.nt - 1) { ++seg; inseg = 0; }
            w.next(a);
        }
        if (failed) atomicExch(a.err, 1);
    } else if (warp == 13) {
        // ======================================== loader: one thread fills the ring, K and V block
        // of each tile
        if (lane == 0) {
            W w = w0;
            int i = 0, slot = 0, sp = 0;                       // tiles loaded
            asm volatile("fence.proxy.async;" ::: "memory");
            for (int j = 0; j < J && !failed; ++j) {
                const int64_t bh = (int64_t)w.b * a.Hkv + w.kv;
                int64_t blk[2] = {0, 0};                       // (an empty sequence reads block 0, all masked)
                if (w.n > 0) {
                    blk[0] = cache_block(a.ktable, a.kpool, a.NB, bh, w.k, a.err);
                    blk[1] = cache_block(a.vtable, a.vpool, a.NB, bh, w.k, a.err);
                }
                if (i >= kSlots && !mbar_wait_bounded(bar(kBarSlot + slot), (uint32_t)(sp ^ 1))) { failed = true; break; }
                const uint32_t br = bar(kBarRing + slot);
                mbar_expect_tx(br, (uint32_t)(2 * C::kBlockB));
#pragma unroll
                for (int k = 0; k < 2; ++k)                    // a bad table entry reads block 0
                    bulk_g2s(smem_u32(sm + C::kOffRing + (2 * slot + k) * C::kBlockB),
                             (k ? a.vc : a.kc) + (blk[k] >= 0 ? blk[k] : 0) * C::kBlockB, C::kBlockB, br);
                ++i;
                if (++slot == kSlots) { slot = 0; sp ^= 1; }
                w.next(a);
            }
            // copies that may still be in flight (the last one into each slot)
            for (int k = i > kSlots ? i - kSlots : 0; k < i; ++k)
                mbar_wait_bounded(bar(kBarRing + k % kSlots), (uint32_t)((k / kSlots) & 1));
            if (failed) atomicExch(a.err, 1);
        }
    } else {
        // ======================================== the mma warp (uniform; its elected lane issues)
        constexpr uint32_t kIdS = idesc_f16(128, TT), kIdO = idesc_f16_bmn(128, D);
        W w = w0;
        bool ok = true;
        // operand descriptors of buffer 0; an offset goes into their address field (16-byte units;
        // shared-memory addresses are below 2^18, so it does not carry)
        const uint64_t qdesc = sw128_desc(sbase + C::kOffQ), kdesc = sw128_desc(sbase);
        const uint64_t vdesc = sw128_desc_mn(sbase + NL * C::kTile, (uint32_t)(TT * 128), 1024u);
        int nS[2] = {0, 0}, nP[2] = {0, 0};    // S issued and P taken of each stream so far
        // S of stream x from buffer bf
        auto mma_s = [&](int x, int bf) {
            const uint64_t kd = kdesc + (uint64_t)(bf * (C::kBuf >> 4));
            const uint64_t qd = qdesc + (uint64_t)(MT == 2 ? x * ((QL * C::kQ) >> 4) : 0);
            const int b = 2 * x + (nS[x]++ & 1);                // score buffer
            const uint32_t xd = tmem + C::kX + TT * b;
            uint32_t acc = 0u;
#pragma unroll
            for (int q = 1; q <= 3; ++q) {                     // lo hi, hi lo, hi hi: the small ones first (truncated sums)
                const int pr = q % 3;
                if ((pr == 1 && QL == 1) || (pr == 2 && NL == 1)) continue;
                const uint32_t ql = pr == 1 ? (uint32_t)C::kQ : 0u, kl = pr == 2 ? (uint32_t)C::kTile : 0u;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    mma_ss(xd, qd + ((ql + (uint32_t)((s >> 2) * (128 * 128) + (s & 3) * 32)) >> 4),
                                  kd + ((kl + (uint32_t)((s >> 2) * (TT * 128) + (s & 3) * 32)) >> 4), kIdS, acc);
                    acc = 1u;
                }
            }
            commit(bar(kBarS + b));
        };
        // O of stream x (+)= P V from buffer bf, once P is there
        auto mma_o = [&](int x, int bf, bool first, bool last) -> bool {
            const int b = 2 * x + (nP[x] & 1);                  // score buffer
            if (!warp_wait(bar(kBarP + b), (uint32_t)((nP[x] >> 1) & 1))) return false;
            ++nP[x];
            const uint32_t od = tmem + C::kO + D * x, pa = tmem + C::kX + TT * b;
            tc_fence_after();
            const uint64_t vd = vdesc + (uint64_t)(bf * (C::kBuf >> 4));
            uint32_t acc = first ? 0u : 1u;
#pragma unroll
            for (int pr = 0; pr < (NL == 2 ? 3 : 1); ++pr) {   // hi hi, lo hi, hi lo
                const uint32_t pl = pr == 1 ? 32u : 0u, vl = pr == 2 ? (uint32_t)C::kTile : 0u;
#pragma unroll
                for (int s = 0; s < TT / 16; ++s) {
                    mma_ts(od, pa + pl + 8 * s, vd + ((vl + 2048 * s) >> 4), kIdO, acc);
                    acc = 1u;
                }
            }
            commit(bar(kBarO + x));
            if (last) commit(bar(kBarFree + bf));           // the tile's last product
            return true;
        };
        // S of tile j (both row tiles, or the tile's stream), once its operands are there
        // tiles whose scores go out before this one's values (fewer than there are buffers)
        constexpr int kAhead = MT == 2 || C::kBufs == 2 ? 1 : 2;
        int sb = 0, sbp = 0;               // buffer of the next scores, and its phase
        auto scores = [&](int j) -> bool {
            if (!warp_wait(bar(kBarReady + sb), (uint32_t)sbp)) return false;
            tc_fence_after();
            if constexpr (MT == 2) {
                mma_s(0, sb);
                mma_s(1, sb);
            } else {
                mma_s(j & 1, sb);
            }
            if (++sb == C::kBufs) { sb = 0; sbp ^= 1; }
            return true;
        };
        int vb = 0;                        // buffer of the next values (its scores have waited for it)
        for (int j = 0, seg = 0; j < J && ok; ++seg) {
            const int left = w.nt - w.k, most = left < C::kSegTiles ? left : C::kSegTiles;
            const int j1 = j + most < J ? j + most : J;        // the segment's tiles
            if (!(ok = warp_wait(bar(kBarQ), (uint32_t)(seg & 1)))) break;
            for (int i = 0; i < kAhead && j + i < j1 && ok; ++i) ok = scores(j + i);
            for (int i = j; i < j1 && ok; ++i) {
                if (i + kAhead < j1 && !(ok = scores(i + kAhead))) break;
                if constexpr (MT == 2) {
                    if (!(ok = mma_o(0, vb, i == j, false))) break;
                    if (!(ok = mma_o(1, vb, i == j, true))) break;
                } else {
                    if (!(ok = mma_o(i & 1, vb, i - j < 2, true))) break;
                }
                if (++vb == C::kBufs) vb = 0;
            }
            if (ok) {
                commit(bar(kBarSeg));
                if (lane == 0) mbar_arrive(bar(kBarSeg));      // (orders what the producers noted, seen through their arrivals)
            }
            w.k += j1 - j - 1;
            w.next(a);
            j = j1;
        }
        // every mma is done before tensor memory is released
        commit(bar(kBarDrain));
        warp_wait(bar(kBarDrain), 0u);
        if (!ok && lane == 0) atomicExch(a.err, 1);
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

template <int D, int GRP, int DT, int MT>
cudaError_t launch_t(const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    using C = Ch<D, GRP, DT == TQ_BF16 ? 1 : 2, DT == TQ_F32 ? 2 : 1, MT>;
    cudaError_t e = set_smem_once<tq_int4_chunk_kernel<D, GRP, DT, MT>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms < kInt4MaxCtas ? num_sms : kInt4MaxCtas;
    e = launch_pdl(tq_int4_chunk_kernel<D, GRP, DT, MT>, dim3(ctas), dim3(kThreads), C::kSmem, s, a);
    if (e != cudaSuccess) return e;
    return launch_int4_combine_tiles<D, DT, MT>(a, ctas, s);
}
template <int D, int GRP>
cudaError_t launch_g(tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    const bool two = int4_slot_rows(D, dt, a.rows) == 256;
    if (dt == TQ_F32) {
        if constexpr (D == 64)
            if (two) return launch_t<D, GRP, TQ_F32, 2>(a, num_sms, s);
        return launch_t<D, GRP, TQ_F32, 1>(a, num_sms, s);
    }
    if (dt == TQ_BF16)
        return two ? launch_t<D, GRP, TQ_BF16, 2>(a, num_sms, s) : launch_t<D, GRP, TQ_BF16, 1>(a, num_sms, s);
    return two ? launch_t<D, GRP, TQ_F16, 2>(a, num_sms, s) : launch_t<D, GRP, TQ_F16, 1>(a, num_sms, s);
}

}  // namespace

// Split kernel (units of 8 rows, each reading its cache) or chunk kernel (128 rows at a time, used or
// not), and one or two row tiles a unit.  Attention, us, 16 sequences of 4000 tokens / one of 40960, 8 kv
// heads:
//   rows            12        16        24        32        64
//   d 128 bf16 split  62 / 43   63 / 43   89 / 57  115 / 70  214 / 123
//              chunk  67 / 62   68 / 61   68 / 62   67 / 62   67 / 63
//         fp16 split  69 / 47   70 / 48  100 / 64  129 / 78  242 / 139
//              chunk 211 / 148 215 / 147 219 / 151 223 / 154 237 / 163
//         fp32 split  74 / 50   75 / 51  107 / 68  138 / 85  262 / 152
//              chunk 244 / 163 252 / 164 258 / 166 261 / 169 271 / 175
//   d 64  bf16 split  46 / 32   47 / 33   65 / 43   83 / 52  154 / 90
//              chunk  53 / 54   53 / 53   53 / 54   54 / 54   55 / 54
//         fp16 split  49 / 34   50 / 35   69 / 45   88 / 55  164 / 96
//              chunk 106 / 84  107 / 84  111 / 86  116 / 88  129 / 98
// so the chunk kernel takes over above 16 rows of bf16 and above 32 of the others.  256-row units above
// 128 rows, against 128-row ones: d 128 bf16 132 rows 96 / 89 (119 / 84), 512 rows 174 / 122 (219 / 138),
// 2048 rows 584 / 340 (769 / 482); fp16 132 rows 322 / 202 (449 / 289); d 64 bf16 132 rows 75 / 70 (92 / 70);
// where two row tiles' query limbs fit into shared memory (fp32 at head_dim 128: 128 KB of them beside
// 128 KB of operands do not).
int int4_slot_rows(int d, tq_dtype dt, int rows) {
    if (d > 128 || rows <= (dt == TQ_BF16 ? 16 : 32)) return 8;
    return rows > 128 && !(d == 128 && dt == TQ_F32) ? 256 : 128;
}

cudaError_t launch_int4_chunk(int d, int group, tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    if (d == 64) return group == 32 ? launch_g<64, 32>(dt, a, num_sms, s) : launch_g<64, 64>(dt, a, num_sms, s);
    return group == 32   ? launch_g<128, 32>(dt, a, num_sms, s)
           : group == 64 ? launch_g<128, 64>(dt, a, num_sms, s)
                         : launch_g<128, 128>(dt, a, num_sms, s);
}

}  // namespace tqi
