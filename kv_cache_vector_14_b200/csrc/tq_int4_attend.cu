// Attention over the 4-bit cache on tensor-core fragments (mma.sync, fp16
// operands, fp32 accumulation), for sm_100a: Lq queries a sequence, causal at
// the end (Lq = 1 is the decode step), any number of query heads per kv head.
//
// Per query row r (query i, head g) and token t, with the codes c of a group G of values:
//   s_t = scale sum_G (ks_{t,G} sum_{j in G} q_j c_{t,j} + kz_{t,G} sum_{j in G} q_j)
//   out = sum_t p_t (vz_{t,G} + vs_{t,G} cv_{t,j}) / sum_t p_t,   p_t = 2^(s_t log2 e - m)
//
// Operands.  What bounds the kernel is the integer pipe that takes codes apart, so
// the operands are chosen for few instructions per code:
//   * Keys enter as int8 operands without being unpacked.  A byte is c0 + 16 c1, so
//     q0 c0 + q1 c1 = (q1 / 16) byte + (q0 - q1 / 16) (byte & 15): the stored words
//     and the words with the high nibbles masked off are the two halves of a k = 32
//     step, one AND per eight codes.  The queries are 32-bit fixed point relative to
//     the row's largest element, in four signed byte limbs; a lane's columns are the
//     limbs of its own head.
//   * A value nibble c in the low mantissa bits of an fp16 is the subnormal number
//     c 2^-24 (16 c 2^-24 one nibble higher), which the tensor core multiplies
//     exactly: one AND per pair and one shift per four pairs, no conversion (fp32
//     calls spend two more, see pick).  A
//     transposing shared-memory load brings the nibbles of two tokens into one
//     register.  The softmax weights times the value scales, p vs, are the other
//     operand: fp16 hi and lo limbs in two columns (22 bits), for bf16 outputs hi
//     alone (2^-11 relative, against 2^-8 of the output's rounding).
// The products with the zeros are rank-one: fp32 sums outside the tensor core.
// To keep p vs inside fp16 whatever the values' magnitude, the reference
// exponent m follows the maximum of s_t + log2 max_G |vs_{t,G}| rather than of s_t.
//   scores  S[16 tok][8] += C[16 tok][32] Q[32][8]                   (int8, group/32 steps per group)
//   values  O^T[16 values][8] += Cv^T[16 values][16 tok] P[16 tok][8], one P per group
// Lane (g, t) = (lane / 4, lane % 4) owns tokens g and g + 8 of a 16-token tile
// and head t (and 4 + t with two n-tiles).
//
// Work.  A unit is (sequence, kv head, up to 8 query rows).  The units' chunks
// of tokens laid end to end are shared out evenly over one CTA per SM, whatever
// the sequences' lengths (each CTA finds its place with a scan of the lengths);
// a CTA deals the chunks of a unit to its warps in turn.  A unit inside one CTA
// is finished there; of a unit cut by CTA borders every CTA writes a partial,
// and the combine kernel merges them.  At most the first and the last unit of a
// CTA are cut, so there are two partial slots per CTA and the workspace does
// not grow with the batch or the context.
//
// Data movement: each warp owns a ring of chunks (codes and pairs of K and V,
// four bulk copies with an mbarrier); waits are bounded as in the other kernels.
//
// Measured: 4 sequences of 102400 tokens, 16/8 heads, d 128, bf16 (floor 72 us): 107 to 112 us,
// 64 to 67 % of the copy rate; the copies alone take 82 and the arithmetic alone 85 us.  fp16 110,
// fp32 128 us; half as many tokens at d 256: bf16 126, fp32 139.  64 ragged sequences up to 8198
// tokens, 32/8 heads, fp16 (floor 55): 118 to 123 us.
#include <type_traits>

#include "tq_frag.cuh"
#include "tq_int4.h"
#include "tq_int4_combine.cuh"

namespace tqi {
namespace {

template <int D, int GRP, int NT>
struct Shape {
    static constexpr int kNG = D / GRP;                       // groups
    static constexpr int kCodeB = D / 2, kPairB = 4 * kNG;    // bytes per token
    static constexpr int kChunk = D <= 128 ? 32 : 16;         // tokens per ring stage
    static constexpr int kTiles = kChunk / 16;
    static constexpr int kNW = (NT == 1 && D <= 128) ? 12 : 8;
    static constexpr int kRing = (NT == 1 || D == 256) ? 3 : 4;
    static constexpr int kOffKc = 0;
    static constexpr int kOffKp = kChunk * kCodeB;
    static constexpr int kOffVc = kOffKp + kChunk * kPairB;
    static constexpr int kOffVp = kOffVc + kChunk * kCodeB;
    static constexpr int kStageB = kOffVp + kChunk * kPairB;
    static constexpr int kBlockB = kBlockT * (kCodeB + kPairB);
    static constexpr int kRows = 4 * NT;                      // query rows of a unit
    static constexpr int kTogether = kTiles;                  // tiles worked on at once
    // shared memory
    static constexpr int kOffAcc = kNW * kRing * kStageB;                 // [NW][kRows][D] merge buffers
    static constexpr int kOffQ = kOffAcc + kNW * kRows * D * 4;           // [kRows][D] scaled queries
    static constexpr int kOffFrag = kOffQ + kRows * D * 4;                // D = 256: query fragments [2 NT][D / 32][32]
    static constexpr int kOffQs = kOffFrag + (D == 256 ? 2 * NT * (D / 32) * 32 * 8 : 0);   // [kRows][kNG]
    static constexpr int kOffF = kOffQs + kRows * kNG * 4;                // [kRows]
    static constexpr int kOffMl = kOffF + kRows * 4;                      // [NW][kRows][2]
    static constexpr int kOffDesc = kOffMl + kNW * kRows * 8;             // [NW][kRing] int
    static constexpr int kOffBar = (kOffDesc + kNW * kRing * 4 + 7) / 8 * 8;
    static constexpr int kOffScan = kOffBar + kNW * kRing * 8;            // [NW + 3] int64
    static constexpr int kSmem = kOffScan + (kNW + 3) * 8;
    static_assert(kOffKp % 16 == 0 && kOffVc % 16 == 0 && kOffVp % 16 == 0 && kStageB % 16 == 0, "bulk copies");
    static_assert(kOffAcc % 16 == 0 && kOffQ % 16 == 0 && kOffBar % 8 == 0 && kOffScan % 8 == 0, "alignment");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

constexpr float kHuge = 3.4e38f;
// p vs is kept below 2^(room + lazy) = 2^15 (fp16 holds 65504), and the reference exponent moves only
// when 2^room is exceeded by 2^lazy.  Two limbs want the room: the low limb of a weight below 2^-3 is
// subnormal.
__host__ __device__ constexpr float room(bool one_limb) { return one_limb ? 7.f : 13.f; }
__host__ __device__ constexpr float lazy(bool one_limb) { return 15.f - room(one_limb); }

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
    if constexpr (DT == TQ_F32) return static_cast<const float*>(p)[i];
    else if constexpr (DT == TQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else return __half2float(static_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float x) {
    if constexpr (DT == TQ_F32) static_cast<float*>(p)[i] = x;
    else if constexpr (DT == TQ_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half*>(p)[i] = __float2half_rn(x);
}
__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tokens of sequence b, and its chunks (at least one, so that an empty sequence's rows are written)
__device__ __forceinline__ int64_t seq_len(const Int4AttendArgs& a, int64_t b) {
    const int64_t n = (a.lens ? (int64_t)a.lens[b] : a.T) + a.add;
    return n < 0 ? 0 : (n > a.Tcap ? a.Tcap : n);
}
template <int CH>
__device__ __forceinline__ int64_t seq_chunks(const Int4AttendArgs& a, int64_t b) {
    const int64_t n = (seq_len(a, b) + CH - 1) / CH;
    return n > 0 ? n : 1;
}

// Place in the units' chunks laid end to end: chunk x is chunk `chunk` of unit `unit` of sequence b.
struct Cursor {
    int64_t base;      // first chunk of sequence b
    int b, nck;
    int64_t span;      // chunks of sequence b over its units
};
template <int CH>
__device__ __forceinline__ void cursor_to(const Int4AttendArgs& a, int64_t units, int64_t x, Cursor& c) {
    while (x >= c.base + c.span) {
        c.base += c.span;
        ++c.b;
        c.nck = (int)seq_chunks<CH>(a, c.b);
        c.span = c.nck * units;
    }
}

// Lane (g, t)'s code words of a 16-token tile, as the stored layout has them.
template <int D, int GRP>
struct Words {
    static constexpr int kK = GRP / 32;                       // words per token and group, K side
    // K: words of group gam of token tok for lane quarter t, from byte key_at of the token codes
    static __device__ __forceinline__ int key_at(int tok, int gam, int t) {
        return tok * (D / 2) + ((gam * (GRP / 2) + t * (GRP / 8)) ^ int4_swizzle(D, tok));
    }
    static __device__ __forceinline__ void key(const uint8_t* p, uint32_t (&w)[kK]) {
        if constexpr (kK == 1) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (kK == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
    }
};
// four 8 x 8 matrices of 16-bit elements, transposed: element rows 2t, 2t + 1 of column g each
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// D += A B, A unsigned and B signed 8-bit, exact 32-bit accumulation
__device__ __forceinline__ void imma_u8s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// nibble R of both halves of x as fp16, the high half's as 15 - c; x8 = x >> 8.  EXACT = false: the
// subnormals c 2^-24 (16 c 2^-24 for odd R), (x & mask) ^ flip in one instruction.  The tensor core
// multiplies them exactly, but aligns its sums by the exponent field, which for a subnormal stands 7
// to 10 bits above the value, so those bits are lost from the sum: 5e-6 of the result.  EXACT = true
// (fp32 calls): c (16 c) as a normal number, two instructions more.
template <int R, bool EXACT>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t x8) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;"
        : "=r"(r)
        : "r"(R < 2 ? x : x8), "r"((R & 1) ? 0x00f000f0u : 0x000f000fu), "r"((R & 1) ? 0x00f00000u : 0x000f0000u));
    if constexpr (EXACT) {
        r |= 0x64006400u;                                     // 1024 + c
        const uint32_t m1024 = 0xe400e400u;
        r = h2_bits(__hadd2(*reinterpret_cast<const __half2*>(&r), *reinterpret_cast<const __half2*>(&m1024)));
    }
    return r;
}
// v as four signed byte digits, v = l0 + 256 l1 + 65536 l2 + 2^24 l3 (adding 128 to each of the
// lower bytes carries, the exclusive or takes it off again), and byte l of four words as one
__device__ __forceinline__ uint32_t digits(int v) { return ((uint32_t)v + 0x00808080u) ^ 0x00808080u; }
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int l) {
    const uint32_t sel = (uint32_t)(l | ((4 + l) << 4));
    return __byte_perm(__byte_perm(a, b, sel), __byte_perm(c, d, sel), 0x5410);
}

// pool block of a block-table entry (contiguous cache: the row itself); bad: -1 and the check word
__device__ __forceinline__ int64_t table_entry(const int32_t* table, int64_t pool, int64_t row, int* err) {
    if (!table) return row;
    const int32_t p = table[row];
    if (p < 0 || (int64_t)p >= pool) {
        atomicExch(err, 1);
        return -1;
    }
    return p;
}

template <int D, int GRP, int NT, int DT>
__global__ void __launch_bounds__(Shape<D, GRP, NT>::kNW * 32, 1) tq_int4_attend_kernel(const Int4AttendArgs a) {
    using S = Shape<D, GRP, NT>;
    using W = Words<D, GRP>;
    constexpr int NG = S::kNG, NW = S::kNW, CH = S::kChunk, ROWS = S::kRows, RING = S::kRing;
    constexpr int kWords = D / 32;                            // key words per lane and token: k-steps of a score
    constexpr int kMT = D / 16;                               // 16-value tiles of the output
    // bf16 outputs: weights as one fp16 limb, columns (head t, head 4 + t); else (hi, lo) of head t per n-tile
    constexpr bool kOneLimb = DT == TQ_BF16;
    constexpr int VT = kOneLimb ? 1 : NT;                     // value n-tiles
    constexpr float kRoom = room(kOneLimb), kLazy = lazy(kOneLimb);
    constexpr float kUnit = DT == TQ_F32 ? 1.f : 16777216.f;  // what one of a value operand's code stands for (see pick)
    constexpr bool kFragSmem = D == 256;
    extern __shared__ __align__(128) uint8_t smem[];
    float* sAcc = reinterpret_cast<float*>(smem + S::kOffAcc);
    uint32_t* sQ = reinterpret_cast<uint32_t*>(smem + S::kOffQ);
    [[maybe_unused]] uint2* sFrag = reinterpret_cast<uint2*>(smem + S::kOffFrag);
    float* sQs = reinterpret_cast<float*>(smem + S::kOffQs);
    float* sF = reinterpret_cast<float*>(smem + S::kOffF);
    float* sMl = reinterpret_cast<float*>(smem + S::kOffMl);
    int* sDesc = reinterpret_cast<int*>(smem + S::kOffDesc);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    int64_t* sScan = reinterpret_cast<int64_t*>(smem + S::kOffScan);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, tq4 = lane & 3;
    uint8_t* ring = smem + (size_t)warp * RING * S::kStageB;
    int* desc = sDesc + warp * RING;                          // first token of each stage's chunk
    uint64_t* bar = bars + warp * RING;

    if (lane == 0)
        for (int s = 0; s < RING; ++s) mbar_init(smem_u32(&bar[s]), 1);
    fence_mbar_init();
    pdl_wait();                                               // (the newest tokens come from the encode before this)

    // ---------------- this CTA's share [lo, hi) of the chunks
    const int rgroups = (a.rows + ROWS - 1) / ROWS;
    const int64_t units = a.Hkv * rgroups;                    // per sequence
    int64_t N;
    Cursor cur;
    // CTAs with work: with fewer chunks than CTAs one chunk each, so that none between the
    // first and the last CTA of a unit is left out
    const int64_t c = blockIdx.x;
    int64_t nC;
    if (!a.lens) {
        const int nck = (int)seq_chunks<CH>(a, 0);
        const int64_t span = nck * units;
        N = a.B * span;
        nC = N < gridDim.x ? N : gridDim.x;
        const int64_t b = (c * N / nC) / span;
        cur = Cursor{b * span, (int)b, nck, span};
        __syncthreads();
    } else {
        // every thread sums the chunks of a run of sequences; a scan over the threads; the
        // thread whose run holds `lo` walks it to the sequence
        const int64_t per = (a.B + NW * 32 - 1) / (NW * 32);
        const int64_t b0 = tid * per < a.B ? tid * per : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
        int64_t mine = 0;
        for (int64_t b = b0; b < b1; ++b) mine += seq_chunks<CH>(a, b) * units;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sScan[warp] = incl;
        __syncthreads();
        int64_t before = 0;
        N = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += sScan[w];
            N += sScan[w];
        }
        nC = N < gridDim.x ? N : gridDim.x;
        const int64_t lo = c < nC ? c * N / nC : 0;
        int64_t base = before + incl - mine;
        if (base <= lo && lo < base + mine) {
            for (int64_t b = b0; b < b1; ++b) {
                const int64_t span = seq_chunks<CH>(a, b) * units;
                if (lo < base + span) {
                    sScan[NW] = base;
                    sScan[NW + 1] = b;
                    break;
                }
                base += span;
            }
        }
        __syncthreads();
        cur.base = sScan[NW];
        cur.b = (int)sScan[NW + 1];
        cur.nck = (int)seq_chunks<CH>(a, cur.b);
        cur.span = cur.nck * units;
    }
    if (tid == 0) a.split[c] = make_int4(0, 0, 0, 0);
    if (c >= nC) return;
    const int64_t lo = c * N / nC, hi = (c + 1) * N / nC;

    // ---------------- the ring: this warp's chunks are lo + warp, lo + warp + NW, ...
    const int nmine = hi - lo > warp ? (int)((hi - lo - warp + NW - 1) / NW) : 0;
    // Where the ring is filled: chunk ck of unit u of sequence b, advanced by NW chunks at a time
    // (no divisions in the loop); the chunk's cache blocks, looked up one chunk ahead of the copy
    int ib, iu, ick, inck, ilen;
    int64_t irow;                                             // block-table row of the unit's first block
    {
        Cursor ci = cur;
        if (nmine > 0) cursor_to<CH>(a, units, lo + warp, ci);
        const int64_t rel = lo + warp - ci.base;
        ib = ci.b;
        inck = ci.nck;
        iu = (int)(rel / inck);
        ick = (int)(rel - (int64_t)iu * inck);
        ilen = (int)seq_len(a, ib);
        irow = ((int64_t)ib * a.Hkv + iu / rgroups) * a.NB;
    }
    int64_t kblk = 0, vblk = 0;
    auto locate = [&]() {
        const int lb = (int)(((int64_t)ick * CH) >> 6);
        kblk = vblk = 0;                                      // (an empty sequence reads block 0, all masked)
        if (ilen > 0) {
            kblk = table_entry(a.ktable, a.kpool, irow + lb, a.err);
            vblk = table_entry(a.vtable, a.vpool, irow + lb, a.err);
        }
    };
    auto advance = [&]() {
        ick += NW;
        if (ick >= inck) {
            do {
                ick -= inck;
                if (++iu == (int)units) {
                    iu = 0;
                    if (++ib == (int)a.B) { ib = 0; inck = NW; ick = 0; break; }        // behind the last chunk
                    ilen = (int)seq_len(a, ib);
                    inck = (int)seq_chunks<CH>(a, ib);
                }
            } while (ick >= inck);
            irow = ((int64_t)ib * a.Hkv + iu / rgroups) * a.NB;
        }
    };
    // lane k issues copy k of a stage: K codes, K pairs, V codes, V pairs
    int cp_off, cp_step, cp_dst, cp_size;
    {
        const bool pairs = lane & 1;
        cp_off = pairs ? kBlockT * S::kCodeB : 0;
        cp_size = cp_step = CH * (pairs ? S::kPairB : S::kCodeB);
        cp_dst = lane == 0 ? S::kOffKc : lane == 1 ? S::kOffKp : lane == 2 ? S::kOffVc : S::kOffVp;
    }
    auto issue = [&](int st) {                                // the chunk that locate() found, into stage st
        const uint32_t br = smem_u32(&bar[st]);
        if (lane == 0) {
            desc[st] = ick * CH;
            mbar_expect_tx(br, S::kStageB);
        }
        __syncwarp();
        if (lane < 4) {
            const int64_t blk = lane < 2 ? kblk : vblk;       // a bad table entry reads block 0
            const uint8_t* src = (lane < 2 ? a.kc : a.vc) + (blk >= 0 ? blk : 0) * S::kBlockB;
            const int sub = ((ick * CH) & 63) / CH;
            bulk_g2s(smem_u32(ring + st * S::kStageB + cp_dst), src + cp_off + sub * cp_step, (uint32_t)cp_size, br);
        }
    };
    // bytes that a kernel before this wrote (the encode) are read by bulk copies
    asm volatile("fence.proxy.async;" ::: "memory");
    for (int i = 0; i < RING && i < nmine; ++i) {
        locate();
        issue(i);
        advance();
    }
    if (RING < nmine) locate();

    // Lane constants: where this lane's key words and value rows sit in a tile (the swizzle repeats
    // every 8 tokens), kept in registers for up to two groups (two 64-value pieces)
    constexpr int kTileB = 16 * (D / 2);
    constexpr int kKeepK = NG <= 2 ? NG : 1, kKeepV = D <= 128 ? D / 64 : 1;
    // value loads: lane l gives row l % 8 of matrix l / 8: tokens 0-7 and 8-15 of one 16-byte piece, then of the next
    const int vtok = 8 * ((lane >> 3) & 1) + (lane & 7), vbase = vtok * (D / 2) + 16 * (lane >> 4);
    int kat[kKeepK], vat[kKeepV];
#pragma unroll
    for (int G_ = 0; G_ < kKeepK; ++G_) kat[G_] = W::key_at(gr, G_, tq4);
#pragma unroll
    for (int c2 = 0; c2 < kKeepV; ++c2) vat[c2] = vbase + ((32 * c2) ^ int4_swizzle(D, vtok));
    auto at_k = [&](int gam) { return NG <= 2 ? kat[gam < kKeepK ? gam : 0] : W::key_at(gr, gam, tq4); };
    auto at_v = [&](int c2) { return D <= 128 ? vat[c2 < kKeepV ? c2 : 0] : vbase + ((32 * c2) ^ int4_swizzle(D, vtok)); };
    const float c15 = (gr & 1) ? 15.f : 0.f, odd = (gr & 1) ? -1.f : 1.f;     // this lane's tokens are odd ones

    // ---------------- units of this CTA, one after the other
    uint32_t bq[kFragSmem ? 1 : 2 * NT][kFragSmem ? 1 : kWords][2];
    float o[VT][kMT][4], oz[NT][NG], mref[NT], mexp[NT], lsum[NT], fq[NT], qs[NT][NG];
    int lim[NT];                                              // tokens visible to this lane's rows
    bool failed = false;
    int i = 0;                                                // this warp's next chunk
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t x0 = lo; x0 < hi;) {
        cursor_to<CH>(a, units, x0, cur);
        const int64_t rel = x0 - cur.base;
        const int u = (int)(rel / cur.nck);
        const int64_t us = cur.base + (int64_t)u * cur.nck, ue = us + cur.nck;
        const int64_t x1 = ue < hi ? ue : hi;
        const int kv = u / rgroups, rg = u - kv * rgroups;
        const int r0 = rg * ROWS;                             // first query row
        const int nrow = a.rows - r0 < ROWS ? a.rows - r0 : ROWS;
        const int64_t len = seq_len(a, cur.b);
        auto out_row = [&](int r) -> int64_t {                // row r of the unit in q and out
            const int64_t qi = (r0 + r) / a.G, g = (r0 + r) - qi * a.G;
            return ((int64_t)cur.b * a.Lq + qi) * a.Hq + (int64_t)kv * a.G + g;
        };
        // queries: row r in fixed point, scaled by a power of two so that its largest element is in
        // [2^28, 2^29); an even value's entry is q0 - q1 / 16, an odd one's q1 / 16
        for (int r = warp; r < ROWS; r += NW) {
            float v[D / 32], mx = 0.f;
            bool bad = false;
            const int64_t at = (r < nrow ? out_row(r) : 0) * D;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                v[e] = r < nrow ? load_elem<DT>(a.q, at + 32 * e + lane) : 0.f;
                mx = fmaxf(mx, fabsf(v[e]));
                bad |= !(fabsf(v[e]) <= kHuge);
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, s));
            bad = __any_sync(kFull, bad);                     // an infinity or a NaN makes the row NaN
            int ex = mx > 0.f && !bad ? ilogbf(mx) : 0;
            ex = ex < -90 ? -90 : ex;
            const float f = exp2f((float)(28 - ex));
            float gs[NG];
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) gs[G_] = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const int fix = __float2int_rn(v[e] * f * ((lane & 1) ? 0.0625f : 1.f));
                const int high = __shfl_xor_sync(kFull, fix, 1);
                sQ[r * D + 32 * e + lane] = digits((lane & 1) ? fix : fix - high);
                gs[e / (GRP / 32)] += v[e];
            }
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) gs[G_] += __shfl_xor_sync(kFull, gs[G_], s);
                if (lane == 0) sQs[r * NG + G_] = a.scale_log2 * gs[G_];
            }
            if (lane == 0) sF[r] = bad ? __int_as_float(0x7fc00000) : a.scale_log2 / f;
        }
        __syncthreads();
        // B operand of k-step (group, word j), n-tile (nt, p): column n is head 4 nt + n / 2, limb
        // 2 p + n % 2, so that this lane's own columns are limbs 2 p, 2 p + 1 of head 4 nt + t.  Rows
        // 4 t + e belong to byte e of lane quarter t's word, rows 16 + 4 t + e to its low nibbles.
        auto frag = [&](int nt, int kw, uint2 (&b)[2]) {      // both n-tiles p of heads 4 nt ..
            const int gam = kw / (GRP / 32), j = kw % (GRP / 32);
            const int w = gam * (GRP / 8) + tq4 * (GRP / 32) + j;
            const uint4* p = reinterpret_cast<const uint4*>(sQ + (4 * nt + (gr >> 1)) * D + 8 * w);
            const uint4 x = p[0], y = p[1];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int l = 2 * q + (gr & 1);
                b[q] = make_uint2(bytes4(x.y, x.w, y.y, y.w, l), bytes4(x.x, x.z, y.x, y.z, l));
            }
        };
        if constexpr (kFragSmem) {
            for (int idx = warp; idx < NT * kWords; idx += NW) {
                uint2 b[2];
                frag(idx / kWords, idx % kWords, b);
#pragma unroll
                for (int q = 0; q < 2; ++q) sFrag[((2 * (idx / kWords) + q) * kWords + idx % kWords) * 32 + lane] = b[q];
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kw = 0; kw < kWords; ++kw) {
                    uint2 b[2];
                    frag(nt, kw, b);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        bq[2 * nt + q][kw][0] = b[q].x;
                        bq[2 * nt + q][kw][1] = b[q].y;
                    }
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = 4 * nt + tq4;
            fq[nt] = sF[h];
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) {
                qs[nt][G_] = sQs[h * NG + G_];
                oz[nt][G_] = 0.f;
            }
            const int64_t l_ = len - a.Lq + 1 + (r0 + h) / a.G;
            lim[nt] = h < nrow && l_ > 0 ? (int)l_ : 0;
            mref[nt] = -INFINITY;
            mexp[nt] = 0.f;                                   // the reference used in exponents (0 before any token)
            lsum[nt] = 0.f;
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) o[vt][mt][0] = o[vt][mt][1] = o[vt][mt][2] = o[vt][mt][3] = 0.f;
        const int64_t minlim = len - a.Lq + 1 + r0 / a.G;     // the unit's first row sees the fewest tokens

        // ---------------- this warp's chunks of the unit
        for (; i < nmine && lo + warp + (int64_t)i * NW < x1 && !failed; ++i) {
            const uint32_t br = smem_u32(&bar[stage]);
            const bool ok = mbar_wait_bounded(br, phase, i == 0 ? a.first_wait : kWaitLimit);
            if (__any_sync(kFull, !ok)) {                     // give up: no more chunks, once the copies in flight are in
                failed = true;
                if (lane == 0) atomicExch(a.err, 1);
                for (int j = i; j < nmine && j < i + RING; ++j)
                    mbar_wait_bounded(smem_u32(&bar[j % RING]), (uint32_t)((j / RING) & 1));
                break;
            }
            const uint8_t* st = ring + stage * S::kStageB;
            const int tok0 = desc[stage];
            // NTILE 16-token tiles from tile k0 on, together: more independent work per warp, and one
            // maximum exchange for all of them
            auto tiles = [&](auto ntile_tag, const int k0, auto partial_tag) {
                constexpr bool PARTIAL = decltype(partial_tag)::value;
                constexpr int NTILE = decltype(ntile_tag)::value;
                constexpr int NP = 2 * NTILE;                 // this lane's tokens: g and g + 8 of every tile
                // ---- scores
                float sc[NT][NP], zc[NT][NP];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < NP; ++k) sc[nt][k] = zc[nt][k] = 0.f;
#pragma unroll
                for (int kt = 0; kt < NTILE; ++kt) {
                    const uint8_t* kc = st + (k0 + kt) * kTileB + S::kOffKc;
                    const uint8_t* kp = st + S::kOffKp + ((k0 + kt) * 16 + gr) * S::kPairB;
#pragma unroll
                    for (int gam = 0; gam < NG; ++gam) {
                        uint32_t wA[W::kK], wB[W::kK];
                        W::key(kc + at_k(gam), wA);
                        W::key(kc + at_k(gam) + 8 * (D / 2), wB);
                        int acc[2 * NT][4];
#pragma unroll
                        for (int np = 0; np < 2 * NT; ++np) acc[np][0] = acc[np][1] = acc[np][2] = acc[np][3] = 0;
#pragma unroll
                        for (int j = 0; j < W::kK; ++j) {
                            const uint32_t ka[4] = {wA[j], wB[j], wA[j] & 0x0f0f0f0fu, wB[j] & 0x0f0f0f0fu};
                            const int kw = gam * (GRP / 32) + j;
#pragma unroll
                            for (int np = 0; np < 2 * NT; ++np) {
                                if constexpr (kFragSmem) {
                                    const uint2 b = sFrag[(np * kWords + kw) * 32 + lane];
                                    imma_u8s8(acc[np], ka, b.x, b.y);
                                } else {
                                    imma_u8s8(acc[np], ka, bq[np][kw][0], bq[np][kw][1]);
                                }
                            }
                        }
                        const float2 pA = __half22float2(*reinterpret_cast<const __half2*>(kp + 4 * gam));
                        const float2 pB = __half22float2(*reinterpret_cast<const __half2*>(kp + 8 * S::kPairB + 4 * gam));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // the four limbs of this lane's head (each sum below 2^22, so a pair fits 32 bits)
                            const int(&lo_)[4] = acc[2 * nt];
                            const int(&hi_)[4] = acc[2 * nt + 1];
                            const float xA = fmaf((float)(hi_[0] + 256 * hi_[1]), 65536.f, (float)(lo_[0] + 256 * lo_[1]));
                            const float xB = fmaf((float)(hi_[2] + 256 * hi_[3]), 65536.f, (float)(lo_[2] + 256 * lo_[3]));
                            sc[nt][2 * kt] = fmaf(pA.x, xA, sc[nt][2 * kt]);
                            sc[nt][2 * kt + 1] = fmaf(pB.x, xB, sc[nt][2 * kt + 1]);
                            zc[nt][2 * kt] = fmaf(pA.y, qs[nt][gam], zc[nt][2 * kt]);
                            zc[nt][2 * kt + 1] = fmaf(pB.y, qs[nt][gam], zc[nt][2 * kt + 1]);
                        }
                    }
                }
                // ---- the values' scales and zeros, and a bound of log2 of the scales' magnitudes (where a
                // group's zero rounds above its maximum the scale is below zero)
                const uint8_t* vp = st + S::kOffVp + (k0 * 16 + gr) * S::kPairB;
                uint32_t vpair[NP][NG];
                float lg[NP];
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    float big = 5.9604645e-8f;                // 2^-24, the least scale above zero
#pragma unroll
                    for (int gam = 0; gam < NG; ++gam) {
                        vpair[k][gam] = *reinterpret_cast<const uint32_t*>(vp + 8 * k * S::kPairB + 4 * gam);
                        big = fmaxf(big, fabsf(__low2float(*reinterpret_cast<const __half2*>(&vpair[k][gam]))));
                    }
                    lg[k] = fast_log2(big);
                }
                // ---- online softmax
                float p[NT][NP];
                [[maybe_unused]] bool ok[NT][NP];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float e = -INFINITY;
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        sc[nt][k] = fmaf(sc[nt][k], fq[nt], zc[nt][k]);
                        if constexpr (PARTIAL) {
                            ok[nt][k] = tok0 + (k0 * 16 + 8 * k + gr) < lim[nt];
                            if (!ok[nt][k]) sc[nt][k] = -INFINITY;
                            e = ok[nt][k] ? fmaxf(e, sc[nt][k] + lg[k]) : e;
                        } else {
                            e = fmaxf(e, sc[nt][k] + lg[k]);
                        }
                    }
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 4));
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 8));
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 16));
                    if (__any_sync(kFull, e - kRoom - kLazy > mref[nt])) {
                        const float mn = e - kRoom > mref[nt] ? e - kRoom : mref[nt];
                        const float f = mref[nt] == -INFINITY ? 0.f : fast_exp2(mref[nt] - mn);   // nothing summed so far
                        mref[nt] = mn;
                        mexp[nt] = mn == -INFINITY ? 0.f : mn;
                        lsum[nt] *= f;
#pragma unroll
                        for (int G_ = 0; G_ < NG; ++G_) oz[nt][G_] *= f;
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) {
                            if constexpr (kOneLimb) {
                                o[0][mt][nt] *= f; o[0][mt][2 + nt] *= f;
                            } else {
                                o[nt][mt][0] *= f; o[nt][mt][1] *= f; o[nt][mt][2] *= f; o[nt][mt][3] *= f;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        p[nt][k] = fast_exp2(sc[nt][k] - mexp[nt]);
                        lsum[nt] += p[nt][k];
                    }
                }
                // ---- values: O^T += Cv^T (p vs).  An odd token enters as p (vz + 15 vs) - p vs (15 - c):
                // codes are all positive and a long flat softmax would sum them to many times the
                // result, with the tensor core's truncated additions (relative error against 64 bits
                // at 4133 tokens 7e-5; this way, and with exact picks for fp32 calls, 5e-7)
#pragma unroll
                for (int kt = 0; kt < NTILE; ++kt) {
                    uint32_t pb[VT][2];
#pragma unroll
                    for (int c2 = 0; c2 < D / 64; ++c2) {      // 64 values: two 16-byte pieces of 16 tokens
                        uint32_t v4[4];
                        ldsm_x4_t(smem_u32(st + (k0 + kt) * kTileB + S::kOffVc + at_v(c2)), v4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = 2 * c2 + h, gam = 32 * c / GRP;
                            if (32 * c % GRP == 0) {           // a new group: its weights
                                float w2[NT][2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&vpair[2 * kt + k][gam]));
                                    const float vs = v.x * odd;
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        float w_ = p[nt][2 * kt + k] * vs, y_ = fmaf(v.x, c15, v.y);
                                        if constexpr (PARTIAL)     // p = 0 there, but the pair may be anything
                                            if (!ok[nt][2 * kt + k]) w_ = y_ = 0.f;
                                        w2[nt][k] = w_;
                                        oz[nt][gam] = fmaf(p[nt][2 * kt + k], y_, oz[nt][gam]);
                                    }
                                }
                                // columns of token A and of token B: (head t, head 4 + t), or (hi, lo) of head t
                                if constexpr (kOneLimb) {
#pragma unroll
                                    for (int k = 0; k < 2; ++k)
                                        pb[0][k] = movmatrix_t(h2_bits(__floats2half2_rn(w2[0][k], NT == 2 ? w2[NT - 1][k] : 0.f)));
                                } else {
#pragma unroll
                                    for (int nt = 0; nt < VT; ++nt) {
                                        uint32_t hi, lo;
                                        split_hilo(w2[nt][0], w2[nt][1], hi, lo);
                                        pb[nt][0] = movmatrix_t(__byte_perm(hi, lo, 0x5410));
                                        pb[nt][1] = movmatrix_t(__byte_perm(hi, lo, 0x7632));
                                    }
                                }
                            }
                            // registers: tokens 2t, 2t + 1 (low, high half) and 8 further on, values 32 c + 4 g ..
                            const uint32_t x = v4[2 * h], y = v4[2 * h + 1], x8 = x >> 8, y8 = y >> 8;
                            const uint32_t va[4] = {pick<0, DT == TQ_F32>(x, x8), pick<1, DT == TQ_F32>(x, x8), pick<0, DT == TQ_F32>(y, y8), pick<1, DT == TQ_F32>(y, y8)};
                            const uint32_t vb[4] = {pick<2, DT == TQ_F32>(x, x8), pick<3, DT == TQ_F32>(x, x8), pick<2, DT == TQ_F32>(y, y8), pick<3, DT == TQ_F32>(y, y8)};
#pragma unroll
                            for (int vt = 0; vt < VT; ++vt) {
                                mma16816(o[vt][2 * c], va, pb[vt][0], pb[vt][1]);
                                mma16816(o[vt][2 * c + 1], vb, pb[vt][0], pb[vt][1]);
                            }
                        }
                    }
                }
            };
            if (tok0 + CH <= minlim) {
                constexpr int kTogether = S::kTogether;
#pragma unroll
                for (int k0 = 0; k0 < S::kTiles; k0 += kTogether)
                    tiles(std::integral_constant<int, kTogether>{}, k0, std::false_type{});
            } else {
#pragma unroll 1
                for (int k0 = 0; k0 < S::kTiles; ++k0)
                    if (tok0 + 16 * k0 < len) tiles(std::integral_constant<int, 1>{}, k0, std::true_type{});
            }
            __syncwarp();
            if (i + RING < nmine) {
                fence_proxy_async();
                issue(stage);
                advance();
                if (i + RING + 1 < nmine) locate();
            }
            if (++stage == RING) { stage = 0; phase ^= 1; }
        }
        // ---------------- merge the warps: accumulators [kRows][D], (reference, sum) [kRows][2]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (failed) { mref[nt] = -INFINITY; lsum[nt] = 0.f; }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                lsum[nt] += __shfl_xor_sync(kFull, lsum[nt], s);
#pragma unroll
                for (int G_ = 0; G_ < NG; ++G_) oz[nt][G_] += __shfl_xor_sync(kFull, oz[nt][G_], s);
            }
            // nothing but NaN scores moves no maximum, and still is no empty row
            if (lsum[nt] != lsum[nt] && mref[nt] == -INFINITY) mref[nt] = 0.f;
            const int h = 4 * nt + tq4;
            if (gr == 0) {
                sMl[(warp * ROWS + h) * 2] = mref[nt];
                sMl[(warp * ROWS + h) * 2 + 1] = lsum[nt];
            }
            if (mref[nt] != -INFINITY) {
                float* dst = sAcc + (warp * ROWS + h) * D;
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                    // tile mt: values 2 (mt % 2) and one more of lane row g's four in the 32 of piece mt / 2
                    const int gam = 16 * mt / GRP, val = 32 * (mt >> 1) + 4 * gr + 2 * (mt & 1);
                    const float x = kOneLimb ? o[0][mt][nt] : o[kOneLimb ? 0 : nt][mt][0] + o[kOneLimb ? 0 : nt][mt][1];
                    const float y = kOneLimb ? o[0][mt][2 + nt] : o[kOneLimb ? 0 : nt][mt][2] + o[kOneLimb ? 0 : nt][mt][3];
                    dst[val] = fmaf(x, kUnit, oz[nt][gam]);
                    dst[val + 1] = fmaf(y, kUnit / 16.f, oz[nt][gam]);
                }
            }
        }
        __syncthreads();
        const bool whole = us >= lo && ue <= hi;
        // a cut unit's partial: slot 1 where it begins in this CTA, else slot 0
        const int64_t slot = (2 * c + (us >= lo ? 1 : 0)) * ROWS;
        for (int idx = tid; idx < nrow * D; idx += NW * 32) {
            const int r = idx / D, j = idx % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, sMl[(w * ROWS + r) * 2]);
            float L = 0.f, A = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float mw = sMl[(w * ROWS + r) * 2];
                    if (mw == -INFINITY) continue;
                    const float f = fast_exp2(mw - M);
                    L = fmaf(f, sMl[(w * ROWS + r) * 2 + 1], L);
                    A = fmaf(f, sAcc[(w * ROWS + r) * D + j], A);
                }
            }
            if (whole) {
                store_elem<DT>(a.out, out_row(r) * D + j, M == -INFINITY ? 0.f : A / L);
            } else {
                a.part_acc[(slot + r) * D + j] = A;
                if (j == 0) {
                    a.part_ml[(slot + r) * 2] = M;
                    a.part_ml[(slot + r) * 2 + 1] = L;
                }
            }
        }
        if (tid == 0 && us >= lo && ue > hi)                  // the combine merges it: up to the CTA of its last chunk
            a.split[c] = make_int4(cur.b, u, (int)((ue * nC - 1) / N), 1);
        x0 = x1;
        if (x0 < hi) __syncthreads();                         // the merge buffers and queries are reused
    }
    pdl_trigger();
}

template <int D, int GRP, int NT, int DT>
cudaError_t launch_t(const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    using S = Shape<D, GRP, NT>;
    cudaError_t e = set_smem_once<tq_int4_attend_kernel<D, GRP, NT, DT>>(S::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms < kInt4MaxCtas ? num_sms : kInt4MaxCtas;
    e = launch_pdl(tq_int4_attend_kernel<D, GRP, NT, DT>, dim3(ctas), dim3(S::kNW * 32), S::kSmem, s, a);
    if (e != cudaSuccess) return e;
    return launch_int4_combine<D, DT>(a, S::kRows, ctas, s);
}
template <int D, int GRP>
cudaError_t launch_g(tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    if (a.rows <= 4)
        return dt == TQ_F32    ? launch_t<D, GRP, 1, TQ_F32>(a, num_sms, s)
               : dt == TQ_BF16 ? launch_t<D, GRP, 1, TQ_BF16>(a, num_sms, s)
                               : launch_t<D, GRP, 1, TQ_F16>(a, num_sms, s);
    return dt == TQ_F32    ? launch_t<D, GRP, 2, TQ_F32>(a, num_sms, s)
           : dt == TQ_BF16 ? launch_t<D, GRP, 2, TQ_BF16>(a, num_sms, s)
                           : launch_t<D, GRP, 2, TQ_F16>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_int4_attend(int d, int group, tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s) {
    if (d == 64) return group == 32 ? launch_g<64, 32>(dt, a, num_sms, s) : launch_g<64, 64>(dt, a, num_sms, s);
    if (d == 128)
        return group == 32   ? launch_g<128, 32>(dt, a, num_sms, s)
               : group == 64 ? launch_g<128, 64>(dt, a, num_sms, s)
                             : launch_g<128, 128>(dt, a, num_sms, s);
    return group == 32   ? launch_g<256, 32>(dt, a, num_sms, s)
           : group == 64 ? launch_g<256, 64>(dt, a, num_sms, s)
                         : launch_g<256, 128>(dt, a, num_sms, s);
}

}  // namespace tqi
