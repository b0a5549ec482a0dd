// Encode and expand of the 4-bit cache (format in tq_int4.h), for sm_100a.
//
// Encode, per group of values x:  zero = fp16(min x), scale = fp16((max x - zero)
// * fp32(1/15)), c = clamp(rint((x - zero) * (1 / scale)), 0, 15), every step one
// correctly rounded fp32 operation, so the codes are defined to the bit.  x is
// taken within +-65504 (the range of fp16); a group with a NaN stores NaN for
// both.  A thread owns 16 consecutive values, i.e. two 32-bit words of codes, and
// the group's minimum and maximum are shuffled over group/16 lanes.
//
// Both kernels read and write each byte once; HBM bounds them once there are few
// enough instructions per value (about 9 fit into its time; the encode below has 15.8, by the
// count of warp instructions).  So (x - z) r with its
// clamp to [0, 32] is one saturating multiply by r / 32, rounding to an integer one
// addition of 1.5 2^18 (where an fp32 ulp is 1/32), the clamp to 15 one packed
// minimum per two values, and 16-bit inputs take their minimum and maximum two
// values at a time.  Measured on 262144 vectors of 128 bf16 values (floor 13 us):
// encode 54 us with 8 values per thread and separate steps, 21 to 23 us this way (issue slots
// 72 % used, ALU 62 %), expand 22 to 23 us.  fp32 (floor 23): encode 27, expand 59 us, whose stores
// of 16 bytes a lane fill half a sector each.
#include "tq_int4.h"

namespace tqi {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kFifteenth = 0.06666667014360428f;     // fp32(1/15), a constant of the format
constexpr float kMax = 65504.f;
constexpr int kThreads = 256;
constexpr int kUnroll = 2;                              // items in flight per thread

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Where vector gv sits: input offset (elements), block and token; blk
// null where the token lies outside the cache or its table entry outside the pool.
struct Spot {
    int64_t xoff;
    uint8_t* blk;
    int tau;
};
template <int D, int GRP>
__device__ __forceinline__ Spot spot(const Int4CopyArgs& a, const Int4Side& sd, uint32_t gv) {
    Spot r;
    const uint32_t bh = fdiv(gv, a.fdT);
    const uint32_t tt = gv - bh * (uint32_t)a.T;
    const uint32_t b = fdiv(bh, a.fdH);
    const uint32_t hh = bh - b * (uint32_t)a.Hkv;
    r.xoff = (int64_t)b * a.sb + (int64_t)hh * a.sh + (int64_t)tt * a.st;
    const int64_t t = (a.pos ? (int64_t)a.pos[b] : a.t0) + tt;
    r.tau = (int)(t & 63);
    r.blk = nullptr;
    if (t < 0 || t >= a.Tcap) {
        atomicExch(a.err, 1);
    } else {
        const int64_t pb = cache_block(sd.table, sd.pool, a.NB, bh, t >> 6, a.err);
        if (pb >= 0) r.blk = sd.cache + pb * int4_block_bytes(D, GRP);
    }
    return r;
}

template <int DT>
struct Elem;
template <>
struct Elem<TQ_F32> {
    using T = float;
    static __device__ __forceinline__ float to(float x) { return x; }
    static __device__ __forceinline__ float from(float x) { return x; }
};
template <>
struct Elem<TQ_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float to(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ T from(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<TQ_F16> {
    using T = __half;
    static __device__ __forceinline__ float to(T x) { return __half2float(x); }
    static __device__ __forceinline__ T from(float x) { return __float2half_rn(x); }
};

// packed fp32 pairs
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float mul_sat(float a, float b) {
    float r;
    asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr int kVals = 16;                               // values per thread
template <int DT>
constexpr int kRaw = DT == TQ_F32 ? 16 : 8;             // 32-bit registers of a thread's input

// 16 consecutive elements, as stored
template <int DT>
__device__ __forceinline__ void load16(const void* x, int64_t off, bool vec, uint32_t (&w)[kRaw<DT>]) {
    using T = typename Elem<DT>::T;
    const T* p = static_cast<const T*>(x) + off;
    if (vec) {
#pragma unroll
        for (int i = 0; i < kRaw<DT> / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (DT == TQ_F32) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) w[i] = __float_as_uint(p[i]);
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
    }
}
// element pair i of the loaded registers as fp32
template <int DT>
__device__ __forceinline__ void pair_of(const uint32_t (&w)[kRaw<DT>], int i, float& x, float& y) {
    if constexpr (DT == TQ_F32) {
        x = __uint_as_float(w[2 * i]);
        y = __uint_as_float(w[2 * i + 1]);
    } else if constexpr (DT == TQ_BF16) {
        x = __uint_as_float(w[i] << 16);
        y = __uint_as_float(w[i] & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x = f.x;
        y = f.y;
    }
}
// packed minimum of 16-bit elements, NaN if either is
template <int DT>
__device__ __forceinline__ uint32_t min16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == TQ_BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// minimum and maximum over the group of this lane (kL lanes), NaN if it holds one
template <int DT, int kL>
__device__ __forceinline__ void group_range(const uint32_t (&w)[kRaw<DT>], float& lo, float& hi) {
    if constexpr (DT == TQ_F32) {
        lo = hi = __uint_as_float(w[0]);
#pragma unroll
        for (int i = 1; i < kVals; ++i) {
            lo = min_nan(lo, __uint_as_float(w[i]));
            hi = max_nan(hi, __uint_as_float(w[i]));
        }
#pragma unroll
        for (int o = 1; o < kL; o <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
        }
    } else {
        // (min, -max) as a pair: one packed minimum per step
        uint32_t mn = w[0], mx = w[0] ^ 0x80008000u;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            mn = min16x2<DT>(mn, w[i]);
            mx = min16x2<DT>(mx, w[i] ^ 0x80008000u);
        }
        uint32_t p = min16x2<DT>(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
        for (int o = 1; o < kL; o <<= 1) p = min16x2<DT>(p, __shfl_xor_sync(kFull, p, o));
        p ^= 0x80000000u;
        if constexpr (DT == TQ_BF16) {
            lo = __uint_as_float(p << 16);
            hi = __uint_as_float(p & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
            lo = f.x;
            hi = f.y;
        }
    }
}

template <int D, int GRP, int DT>
__global__ void __launch_bounds__(kThreads) tq_int4_encode_kernel(const Int4CopyArgs a, uint32_t nitems) {
    constexpr int kW = D / kVals;             // threads per vector
    constexpr int kL = GRP / kVals;           // lanes per group
    pdl_trigger();                            // the kernel behind this one may start its set-up
    pdl_wait();
    const Int4Side& sd = a.side[blockIdx.y];
    const uint32_t stride = gridDim.x * kThreads;
    // (a warp goes out of range as a whole vector at a time: nitems is a multiple of kW, and the
    // shuffles run over kL <= kW neighbours)
    for (uint32_t i0 = blockIdx.x * kThreads + threadIdx.x; i0 - (threadIdx.x & 31) < nitems; i0 += kUnroll * stride) {
        uint32_t w[kUnroll][kRaw<DT>];
        Spot sp[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t it = i0 + u * stride;
            sp[u].blk = nullptr;
            if (it < nitems) {
                sp[u] = spot<D, GRP>(a, sd, it / kW);
                load16<DT>(sd.x, sp[u].xoff + kVals * (it % kW), a.vec16, w[u]);
            } else {
#pragma unroll
                for (int i = 0; i < kRaw<DT>; ++i) w[u][i] = 0u;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int wi = (int)((i0 + u * stride) % kW);
            float lo, hi;
            group_range<DT, kL>(w[u], lo, hi);
            // clamping is monotone, so the range of the clamped values is the clamped range,
            // and a value outside it takes code 0 or 15 either way
            lo = max_nan(min_nan(lo, kMax), -kMax);
            hi = max_nan(min_nan(hi, kMax), -kMax);
            const __half zh = __float2half_rn(lo);
            const float z = __half2float(zh);
            const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(hi, z), kFifteenth));
            const float s = __half2float(sh);
            const float r32 = s > 0.f ? __frcp_rn(s) * 0.03125f : 0.f;      // r / 32, exact
            const uint64_t mz = pack2(-z, -z), magic = pack2(393216.f, 393216.f);
            uint32_t word[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // t / 32 = sat((x - z) r / 32); + 1.5 2^18 rounds t to the nearest integer (half to
                // even) in the low bits; values k and k + 4 of a word meet in one register
                uint32_t n[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x, y;
                    pair_of<DT>(w[u], 4 * h + k, x, y);
                    unpack2(add2(pack2(x, y), mz), x, y);
                    unpack2(add2(pack2(mul_sat(x, r32), mul_sat(y, r32)), magic), x, y);
                    n[2 * k] = __float_as_uint(x);
                    n[2 * k + 1] = __float_as_uint(y);
                }
                uint32_t v = 0;
#pragma unroll
                for (int k = 3; k >= 0; --k)
                    v = v * 16u + __vminu2(__byte_perm(n[k], n[k + 4], 0x5410), 0x000f000fu);
                word[h] = v;
            }
            if (sp[u].blk) {
                const int tau = sp[u].tau;
                *reinterpret_cast<uint2*>(sp[u].blk + tau * (D / 2) + ((8 * wi) ^ int4_swizzle(D, tau))) =
                    make_uint2(word[0], word[1]);
                if (wi % kL == 0)
                    *reinterpret_cast<__half2*>(sp[u].blk + kBlockT * (D / 2) + (tau * (D / GRP) + wi / kL) * 4) =
                        __halves2half2(sh, zh);
            }
        }
    }
}

template <int D, int GRP, int DT>
__global__ void __launch_bounds__(kThreads) tq_int4_expand_kernel(const Int4CopyArgs a, uint32_t nitems) {
    using E = Elem<DT>;
    constexpr int kW = D / kVals, kL = GRP / kVals;
    pdl_trigger();
    pdl_wait();
    const Int4Side& sd = a.side[blockIdx.y];
    const uint32_t stride = gridDim.x * kThreads;
    for (uint32_t i0 = blockIdx.x * kThreads + threadIdx.x; i0 < nitems; i0 += kUnroll * stride) {
        uint2 word[kUnroll];
        __half2 pair[kUnroll];
        Spot sp[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t it = i0 + u * stride;
            sp[u].blk = nullptr;
            if (it < nitems) {
                sp[u] = spot<D, GRP>(a, sd, it / kW);
                const int wi = (int)(it % kW), tau = sp[u].tau;
                if (sp[u].blk) {
                    word[u] = *reinterpret_cast<const uint2*>(sp[u].blk + tau * (D / 2) + ((8 * wi) ^ int4_swizzle(D, tau)));
                    pair[u] = *reinterpret_cast<const __half2*>(sp[u].blk + kBlockT * (D / 2) + (tau * (D / GRP) + wi / kL) * 4);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!sp[u].blk) continue;
            const float s = __low2float(pair[u]), z = __high2float(pair[u]);
            // a nibble in the low bits of 2^23 is 2^23 + c 16^k; less 2^23 it is exact, and so is
            // the scale over 16^k: one rounding of z + s c, as the format defines
            const uint64_t z2 = pack2(z, z), m23 = pack2(-8388608.f, -8388608.f);
            const uint64_t sA = pack2(s, s * 0.0625f), sB = pack2(s * 0.00390625f, s * 0.000244140625f);
            typename E::T* p = static_cast<typename E::T*>(sd.x) + sp[u].xoff + kVals * ((i0 + u * stride) % kW);
            __align__(16) typename E::T e[kVals];
#pragma unroll
            for (int q = 0; q < 4; ++q) {                      // halfwords of the two words: four values each
                const uint32_t h = ((q & 2) ? word[u].y : word[u].x) >> (16 * (q & 1));
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = __uint_as_float((h & (15u << (4 * k))) | 0x4b000000u);
                unpack2(fma2(add2(pack2(f[0], f[1]), m23), sA, z2), f[0], f[1]);
                unpack2(fma2(add2(pack2(f[2], f[3]), m23), sB, z2), f[2], f[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) e[4 * q + k] = E::from(f[k]);
            }
            if (a.vec16) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(e) / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(e)[i];
            } else {
#pragma unroll
                for (int i = 0; i < kVals; ++i) p[i] = e[i];
            }
        }
    }
}

template <int D, int GRP, int DT>
cudaError_t launch_copy(bool encode, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    const uint32_t nitems = (uint32_t)(a.B * a.Hkv * a.T * (D / kVals));    // below 2^31 (checked by the caller)
    const uint32_t need = (nitems + kThreads - 1) / kThreads;
    const uint32_t most = (uint32_t)num_sms * 8;
    const dim3 grid(need < most ? need : most, (unsigned)a.nsides);
    return launch_pdl(encode ? tq_int4_encode_kernel<D, GRP, DT> : tq_int4_expand_kernel<D, GRP, DT>, grid, dim3(kThreads), 0, s,
                      a, nitems);
}

template <int D, int GRP>
cudaError_t launch_copy_t(bool encode, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    return dt == TQ_F32    ? launch_copy<D, GRP, TQ_F32>(encode, a, num_sms, s)
           : dt == TQ_BF16 ? launch_copy<D, GRP, TQ_BF16>(encode, a, num_sms, s)
                           : launch_copy<D, GRP, TQ_F16>(encode, a, num_sms, s);
}
cudaError_t launch_copy_d(bool encode, int d, int group, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    if (d == 64 && group == 32) return launch_copy_t<64, 32>(encode, dt, a, num_sms, s);
    if (d == 64) return launch_copy_t<64, 64>(encode, dt, a, num_sms, s);
    if (d == 128 && group == 32) return launch_copy_t<128, 32>(encode, dt, a, num_sms, s);
    if (d == 128 && group == 64) return launch_copy_t<128, 64>(encode, dt, a, num_sms, s);
    if (d == 128) return launch_copy_t<128, 128>(encode, dt, a, num_sms, s);
    if (group == 32) return launch_copy_t<256, 32>(encode, dt, a, num_sms, s);
    if (group == 64) return launch_copy_t<256, 64>(encode, dt, a, num_sms, s);
    return launch_copy_t<256, 128>(encode, dt, a, num_sms, s);
}

}  // namespace

cudaError_t launch_int4_encode(int d, int group, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    return launch_copy_d(true, d, group, dt, a, num_sms, s);
}
cudaError_t launch_int4_expand(int d, int group, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    return launch_copy_d(false, d, group, dt, a, num_sms, s);
}

}  // namespace tqi
