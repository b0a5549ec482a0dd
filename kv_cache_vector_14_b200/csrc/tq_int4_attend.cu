// Attention over the 4-bit cache on tensor-core fragments (mma.sync, fp16
// operands, fp32 accumulation), for sm_100a: Lq queries a sequence, causal at
// the end (Lq = 1 is the decode step), any number of query heads per kv head.
//
// Per query row r (query i, head g) and token t, with the codes c of a group G of values:
//   s_t = scale sum_G (ks_{t,G} sum_{j in G} q_j c_{t,j} + kz_{t,G} sum_{j in G} q_j)
//   out = sum_t p_t (vz_{t,G} + vs_{t,G} cv_{t,j}) / sum_t p_t,   p_t = 2^(s_t log2 e - m)
//
// Operands.  A nibble c placed in the low mantissa bits of an fp16 is the
// subnormal number c 2^-24 (16 c 2^-24 one nibble higher), which the tensor
// core multiplies exactly, so a code costs one AND per pair and one shift per
// four pairs, no conversion.  The factors 2^24 and 16 go into the query
// (power-of-two scaled per row), and into the result.  q enters as fp16 hi and
// lo limbs (22 bits; 16-bit queries need only hi), the softmax weights times
// the value scales, p vs, as hi and lo limbs in the columns of one operand.
// The products with the zeros are rank-one: fp32 sums outside the tensor core.
// To keep p vs inside fp16 whatever the values' magnitude, the reference
// exponent m follows the maximum of s_t + log2 max_G vs_{t,G} rather than of s_t.
//   scores  S[16 tok][8] += C[16 tok][16 values] Q[16 values][8]     (group/16 steps per group)
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
    static constexpr int kNW = (NT == 1 && D <= 128) ? 16 : 8;
    static constexpr int kRing = (NT == 1 && D <= 128) ? 2 : (D <= 128 ? 4 : 3);
    static constexpr int kOffKc = 0;
    static constexpr int kOffKp = kChunk * kCodeB;
    static constexpr int kOffVc = kOffKp + kChunk * kPairB;
    static constexpr int kOffVp = kOffVc + kChunk * kCodeB;
    static constexpr int kStageB = kOffVp + kChunk * kPairB;
    static constexpr int kBlockB = kBlockT * (kCodeB + kPairB);
    static constexpr int kRows = 4 * NT;                      // query rows of a unit
    // shared memory
    static constexpr int kOffAcc = kNW * kRing * kStageB;                 // [NW][kRows][D] merge buffers
    static constexpr int kOffQ = kOffAcc + kNW * kRows * D * 4;           // [kRows][D] scaled queries
    static constexpr int kOffFrag = kOffQ + kRows * D * 4;                // D = 256: query fragments [NT][16][32]
    static constexpr int kOffQs = kOffFrag + (D == 256 ? NT * (D / 16) * 32 * 8 : 0);   // [kRows][kNG]
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

constexpr float kTwo24 = 16777216.f;
constexpr float kRoom = 7.f;      // p vs is kept below 2^(kRoom + kLazy) = 2^15 (fp16 holds 65504) ...
constexpr float kLazy = 8.f;      // ... and the reference exponent moves only when it is exceeded by this much

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
    if constexpr (DT == TQ_F32) return __ldg(static_cast<const float*>(p) + i);
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
    const int64_t n = (a.lens ? (int64_t)__ldg(a.lens + b) : a.T) + a.add;
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
    // V: the GRP / 8 values of group gam that lane row g holds of token tok: 1 or 2 words, or a halfword
    static constexpr int kV = GRP == 128 ? 2 : 1;
    static __device__ __forceinline__ int value_at(int tok, int gam, int g) {
        return tok * (D / 2) + ((gam * (GRP / 2) + g * (GRP / 16)) ^ int4_swizzle(D, tok));
    }
    static __device__ __forceinline__ void value(const uint8_t* p, uint32_t (&w)[kV]) {
        if constexpr (GRP == 32) w[0] = *reinterpret_cast<const uint16_t*>(p);
        else if constexpr (GRP == 64) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        }
    }
};
// nibbles r (and r + 4) of a word as two fp16 subnormals: c 2^-24 for even r, 16 c 2^-24 for odd
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t w8, int r) {
    return (r < 2 ? w : w8) & ((r & 1) ? 0x00f000f0u : 0x000f000fu);
}
// pool block of a block-table entry (contiguous cache: the row itself); bad: -1 and the check word
__device__ __forceinline__ int64_t table_entry(const int32_t* table, int64_t pool, int64_t row, int* err) {
    if (!table) return row;
    const int32_t p = __ldg(table + row);
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
    constexpr int kKC = D / 16;                               // k-steps of a score
    // K n-tiles: with one (NT = 1, or 16-bit queries) the columns are (head, limb) or (head t, head 4 + t)
    constexpr int KNT = (NT == 2 && DT == TQ_F32) ? 2 : 1;
    constexpr bool kTwoHeads = NT == 2 && KNT == 1;
    constexpr bool kFragSmem = D == 256;
    extern __shared__ __align__(128) uint8_t smem[];
    float* sAcc = reinterpret_cast<float*>(smem + S::kOffAcc);
    float* sQ = reinterpret_cast<float*>(smem + S::kOffQ);
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
    if (a.chained) pdl_wait();                                // the newest tokens come from the encode before this

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

    // Lane constants: where this lane's codes sit in a tile (the swizzle repeats every 8 tokens),
    // kept in registers for up to two groups; the order of its value tokens (2t, 2t + 1, the odd
    // one first where t >= 2)
    constexpr int kTileB = 16 * (D / 2);
    constexpr int kKeep = NG <= 2 ? NG : 1;
    const int par = tq4 >> 1, tv0 = 2 * tq4 + par, tv1 = 2 * tq4 + 1 - par;
    const uint32_t sel_lo = par ? 0x1054u : 0x5410u, sel_hi = par ? 0x3276u : 0x7632u;
    int kat[kKeep], vat0[kKeep], vat1[kKeep];
#pragma unroll
    for (int G_ = 0; G_ < kKeep; ++G_) {
        kat[G_] = W::key_at(gr, G_, tq4);
        vat0[G_] = W::value_at(tv0, G_, gr);
        vat1[G_] = W::value_at(tv1, G_, gr);
    }
    auto at_k = [&](int gam) { return NG <= 2 ? kat[gam < kKeep ? gam : 0] : W::key_at(gr, gam, tq4); };
    auto at_v0 = [&](int gam) { return NG <= 2 ? vat0[gam < kKeep ? gam : 0] : W::value_at(tv0, gam, gr); };
    auto at_v1 = [&](int gam) { return NG <= 2 ? vat1[gam < kKeep ? gam : 0] : W::value_at(tv1, gam, gr); };

    // ---------------- units of this CTA, one after the other
    uint32_t bq[kFragSmem ? 1 : KNT][kFragSmem ? 1 : kKC][2];
    float o[NT][kKC][4], oz[NT][NG], mref[NT], lsum[NT], fq[NT], qs[NT][NG];
    bool live[NT];
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
        // queries: row r scaled by a power of two so that its largest element is in [2^14, 2^15)
        for (int r = warp; r < ROWS; r += NW) {
            float v[D / 32], mx = 0.f;
            const int64_t at = (r < nrow ? out_row(r) : 0) * D;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                v[e] = r < nrow ? load_elem<DT>(a.q, at + 32 * e + lane) : 0.f;
                mx = fmaxf(mx, fabsf(v[e]));
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, s));
            int ex = mx > 0.f ? ilogbf(mx) : 0;
            ex = ex < -100 ? -100 : ex;
            const float f = mx <= 3.4e38f ? exp2f((float)(14 - ex)) : 1.f;
            float gs[NG];
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) gs[G_] = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                sQ[r * D + 32 * e + lane] = v[e] * f;
                gs[e / (GRP / 32)] += v[e];
            }
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) gs[G_] += __shfl_xor_sync(kFull, gs[G_], s);
                if (lane == 0) sQs[r * NG + G_] = a.scale_log2 * gs[G_];
            }
            if (lane == 0) sF[r] = a.scale_log2 * (kTwo24 / f);
        }
        __syncthreads();
        // B operand of k-step kc: step (group, word j, half hf) covers, for lane quarter t, values
        // 8 w + r and 8 w + r + 4, r = 2 hf (rows 2t, 2t + 1) and 2 hf + 1 (rows 2t + 8, + 9, scaled by 1/16)
        auto frag = [&](int nt, int kc, uint32_t& b0, uint32_t& b1) {
            const int gam = kc / (GRP / 16), in = kc % (GRP / 16), j = in >> 1, hf = in & 1;
            const int w = gam * (GRP / 8) + tq4 * (GRP / 32) + j;
            const int head = kTwoHeads ? (gr >> 1) + 4 * (gr & 1) : 4 * nt + (gr >> 1);
            const float* p = sQ + head * D + 8 * w + 2 * hf;
            uint32_t h0, l0, h1, l1;
            split_hilo(p[0], p[4], h0, l0);
            split_hilo(p[1] * 0.0625f, p[5] * 0.0625f, h1, l1);
            const bool lolimb = !kTwoHeads && (gr & 1);
            b0 = lolimb ? l0 : h0;
            b1 = lolimb ? l1 : h1;
        };
        if constexpr (kFragSmem) {
            for (int idx = warp; idx < KNT * kKC; idx += NW) {
                uint32_t b0, b1;
                frag(idx / kKC, idx % kKC, b0, b1);
                sFrag[idx * 32 + lane] = make_uint2(b0, b1);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int nt = 0; nt < KNT; ++nt)
#pragma unroll
                for (int kc = 0; kc < kKC; ++kc) frag(nt, kc, bq[nt][kc][0], bq[nt][kc][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = 4 * nt + tq4;
            live[nt] = h < nrow;
            fq[nt] = sF[h];
#pragma unroll
            for (int G_ = 0; G_ < NG; ++G_) {
                qs[nt][G_] = sQs[h * NG + G_];
                oz[nt][G_] = 0.f;
            }
            const int64_t l_ = len - a.Lq + 1 + (r0 + h) / a.G;
            lim[nt] = live[nt] && l_ > 0 ? (int)l_ : 0;
            mref[nt] = -INFINITY;
            lsum[nt] = 0.f;
#pragma unroll
            for (int mt = 0; mt < kKC; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        }
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
            auto tile = [&](const int kt, auto partial_tag) {
                constexpr bool PARTIAL = decltype(partial_tag)::value;
                const int tA = kt * 16 + gr, tB = tA + 8;     // this lane's two tokens
                // ---- scores
                float s0[NT], s1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s0[nt] = s1[nt] = 0.f;
                float z0[NT], z1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) z0[nt] = z1[nt] = 0.f;
#pragma unroll
                for (int gam = 0; gam < NG; ++gam) {
                    uint32_t wA[W::kK], wB[W::kK];
                    W::key(st + kt * kTileB + S::kOffKc + at_k(gam), wA);
                    W::key(st + kt * kTileB + S::kOffKc + at_k(gam) + 8 * (D / 2), wB);
                    float acc[KNT][4];
#pragma unroll
                    for (int nt = 0; nt < KNT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
                    for (int j = 0; j < W::kK; ++j) {
                        const uint32_t wA8 = wA[j] >> 8, wB8 = wB[j] >> 8;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t ka[4] = {pick(wA[j], wA8, 2 * hf), pick(wB[j], wB8, 2 * hf),
                                                    pick(wA[j], wA8, 2 * hf + 1), pick(wB[j], wB8, 2 * hf + 1)};
                            const int kc = gam * (GRP / 16) + 2 * j + hf;
#pragma unroll
                            for (int nt = 0; nt < KNT; ++nt) {
                                if constexpr (kFragSmem) {
                                    const uint2 b = sFrag[(nt * kKC + kc) * 32 + lane];
                                    mma16816(acc[nt], ka, b.x, b.y);
                                } else {
                                    mma16816(acc[nt], ka, bq[nt][kc][0], bq[nt][kc][1]);
                                }
                            }
                        }
                    }
                    const float2 pA = __half22float2(*reinterpret_cast<const __half2*>(st + S::kOffKp + tA * S::kPairB + 4 * gam));
                    const float2 pB = __half22float2(*reinterpret_cast<const __half2*>(st + S::kOffKp + tB * S::kPairB + 4 * gam));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float xA = kTwoHeads ? acc[0][nt] : acc[kTwoHeads ? 0 : nt][0] + acc[kTwoHeads ? 0 : nt][1];
                        const float xB = kTwoHeads ? acc[0][2 + nt] : acc[kTwoHeads ? 0 : nt][2] + acc[kTwoHeads ? 0 : nt][3];
                        s0[nt] = fmaf(pA.x, xA, s0[nt]);
                        s1[nt] = fmaf(pB.x, xB, s1[nt]);
                        z0[nt] = fmaf(pA.y, qs[nt][gam], z0[nt]);
                        z1[nt] = fmaf(pB.y, qs[nt][gam], z1[nt]);
                    }
                }
                // ---- the values' scales and zeros, and a bound of log2 of the scales
                float2 vA[NG], vB[NG];
                float bigA = 5.9604645e-8f, bigB = 5.9604645e-8f;              // 2^-24, the least scale above zero
#pragma unroll
                for (int gam = 0; gam < NG; ++gam) {
                    vA[gam] = __half22float2(*reinterpret_cast<const __half2*>(st + S::kOffVp + tA * S::kPairB + 4 * gam));
                    vB[gam] = __half22float2(*reinterpret_cast<const __half2*>(st + S::kOffVp + tB * S::kPairB + 4 * gam));
                    bigA = fmaxf(bigA, vA[gam].x);
                    bigB = fmaxf(bigB, vB[gam].x);
                }
                const float lgA = fast_log2(bigA), lgB = fast_log2(bigB);
                // ---- online softmax
                float pA[NT], pB[NT];
                [[maybe_unused]] bool okA[NT], okB[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float sA = fmaf(s0[nt], fq[nt], z0[nt]), sB = fmaf(s1[nt], fq[nt], z1[nt]);
                    float eA = sA + lgA, eB = sB + lgB;
                    if constexpr (PARTIAL) {
                        okA[nt] = tok0 + tA < lim[nt];
                        okB[nt] = tok0 + tB < lim[nt];
                        if (!okA[nt]) { sA = -INFINITY; eA = -INFINITY; }
                        if (!okB[nt]) { sB = -INFINITY; eB = -INFINITY; }
                    }
                    float e = fmaxf(eA, eB);
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 4));
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 8));
                    e = fmaxf(e, __shfl_xor_sync(kFull, e, 16));
                    if (__any_sync(kFull, e - kRoom - kLazy > mref[nt])) {
                        const float mn = e - kRoom > mref[nt] ? e - kRoom : mref[nt];
                        const float f = mref[nt] == -INFINITY ? 0.f : fast_exp2(mref[nt] - mn);   // nothing summed so far
                        mref[nt] = mn;
                        lsum[nt] *= f;
#pragma unroll
                        for (int G_ = 0; G_ < NG; ++G_) oz[nt][G_] *= f;
#pragma unroll
                        for (int mt = 0; mt < kKC; ++mt) {
                            o[nt][mt][0] *= f; o[nt][mt][1] *= f; o[nt][mt][2] *= f; o[nt][mt][3] *= f;
                        }
                    }
                    const float m = mref[nt] == -INFINITY ? 0.f : mref[nt];      // no visible token yet: s is -inf
                    pA[nt] = fast_exp2(sA - m);
                    pB[nt] = fast_exp2(sB - m);
                    lsum[nt] += pA[nt] + pB[nt];
                }
                // ---- values: O^T += Cv^T (p vs); lane quarter t takes tokens 2t, 2t + 1 (+ 8), the
                // odd one first where t >= 2 (bank conflicts).  An odd token enters as
                // p (vz + 15 vs) - p vs (15 - c): codes are all positive and a long flat softmax
                // would sum them to many times the result, with the tensor core's truncated
                // additions (relative error against 64 bits at 4133 tokens 7e-5; this way 7e-7)
                const float c15 = (gr & 1) ? 15.f : 0.f;      // this lane's tokens are odd
                float qA[NT], qB[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    qA[nt] = (gr & 1) ? -pA[nt] : pA[nt];
                    qB[nt] = (gr & 1) ? -pB[nt] : pB[nt];
                }
#pragma unroll
                for (int gam = 0; gam < NG; ++gam) {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float wA = qA[nt] * vA[gam].x, wB = qB[nt] * vB[gam].x;
                        float yA = fmaf(vA[gam].x, c15, vA[gam].y), yB = fmaf(vB[gam].x, c15, vB[gam].y);
                        if constexpr (PARTIAL) {              // p = 0 there, but the pair may be anything
                            if (!okA[nt]) wA = yA = 0.f;
                            if (!okB[nt]) wB = yB = 0.f;
                        }
                        oz[nt][gam] = fmaf(pA[nt], yA, fmaf(pB[nt], yB, oz[nt][gam]));
                        uint32_t h, l;
                        split_hilo(wA, wB, h, l);
                        // (hi, lo) of token A and of token B: the two columns of head t
                        pb[nt][0] = movmatrix_t(__byte_perm(h, l, 0x5410));
                        pb[nt][1] = movmatrix_t(__byte_perm(h, l, 0x7632));
                    }
                    uint32_t w0[W::kV], w1[W::kV], w2[W::kV], w3[W::kV];
                    const uint8_t* vp = st + kt * kTileB + S::kOffVc;
                    W::value(vp + at_v0(gam), w0);
                    W::value(vp + at_v1(gam), w1);
                    W::value(vp + at_v0(gam) + 8 * (D / 2), w2);
                    W::value(vp + at_v1(gam) + 8 * (D / 2), w3);
#pragma unroll
                    for (int k = 0; k < W::kV; ++k) {
#pragma unroll
                        for (int half = 0; half < (GRP == 32 ? 1 : 2); ++half) {
                            // four values: the low halfword is token 2t's, the high one token 2t + 1's
                            const uint32_t sel = half ? sel_hi : sel_lo;
                            // (its 15 - c)
                            const uint32_t x = __byte_perm(w0[k], w1[k], sel) ^ 0xffff0000u;
                            const uint32_t y = __byte_perm(w2[k], w3[k], sel) ^ 0xffff0000u;
                            const uint32_t x8 = x >> 8, y8 = y >> 8;
#pragma unroll
                            for (int r = 0; r < 4; r += 2) {
                                const uint32_t va[4] = {pick(x, x8, r), pick(x, x8, r + 1), pick(y, y8, r), pick(y, y8, r + 1)};
                                const int mt = gam * (GRP / 16) + k * 4 + half * 2 + (r >> 1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][mt], va, pb[nt][0], pb[nt][1]);
                            }
                        }
                    }
                }
            };
            if (tok0 + CH <= minlim) {
#pragma unroll
                for (int kt = 0; kt < S::kTiles; ++kt) tile(kt, std::false_type{});
            } else {
#pragma unroll 1
                for (int kt = 0; kt < S::kTiles; ++kt)
                    if (tok0 + 16 * kt < len) tile(kt, std::true_type{});
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
                for (int mt = 0; mt < kKC; ++mt) {
                    const int gam = mt / (GRP / 16), in = mt % (GRP / 16);
                    // values 2 (in % 2 or 4) of this lane row's run of GRP / 8 values of the group
                    const int val = gam * GRP + gr * (GRP / 8) + 2 * in;
                    dst[val] = fmaf(o[nt][mt][0] + o[nt][mt][1], kTwo24, oz[nt][gam]);
                    dst[val + 1] = fmaf(o[nt][mt][2] + o[nt][mt][3], kTwo24 / 16.f, oz[nt][gam]);
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
    if (a.chained) {
        e = launch_pdl(tq_int4_attend_kernel<D, GRP, NT, DT>, dim3(ctas), dim3(S::kNW * 32), S::kSmem, s, a);
    } else {
        tq_int4_attend_kernel<D, GRP, NT, DT><<<ctas, S::kNW * 32, S::kSmem, s>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    return launch_int4_combine<D, DT>(a, S::kRows, false, ctas, s);
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
