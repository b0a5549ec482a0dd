// Encode and expand of the 4-bit cache (format in tq_int4.h), for sm_100a.
//
// Encode, per group of values x:  zero = fp16(min x), scale = fp16((max x - zero)
// * fp32(1/15)), c = clamp(rint((x - zero) * (1 / scale)), 0, 15), every step one
// correctly rounded fp32 operation, so the codes are defined to the bit.  x is
// taken within +-65504 (the range of fp16); a group with a NaN stores NaN for
// both.  A thread owns 8 consecutive values, i.e. one 32-bit word of codes: the
// load is one or two 16-byte accesses, the group's minimum and maximum are
// shuffled over group/8 lanes, and a warp's words of a token are contiguous.
// Both kernels read and write each byte once; they are bound by HBM.
#include "tq_int4.h"

namespace tqi {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kFifteenth = 0.06666667014360428f;     // fp32(1/15), a constant of the format
constexpr float kMax = 65504.f;
constexpr int kThreads = 256;
constexpr int kUnroll = 4;                              // words in flight per thread

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

// Where word w of vector gv sits: input offset (elements), block and token; blk
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
    const int64_t t = (a.pos ? (int64_t)__ldg(a.pos + b) : a.t0) + tt;
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

template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t off, bool vec, float (&v)[8]) {
    using T = typename Elem<DT>::T;
    const T* p = static_cast<const T*>(x) + off;
    if (vec) {
        __align__(16) T e[8];
#pragma unroll
        for (int i = 0; i < (int)sizeof(e) / 16; ++i)
            reinterpret_cast<uint4*>(e)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Elem<DT>::to(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Elem<DT>::to(p[i]);
    }
}

template <int D, int GRP, int DT>
__global__ void __launch_bounds__(kThreads) tq_int4_encode_kernel(const Int4CopyArgs a, uint32_t nwords) {
    constexpr int kW = D / 8;                 // words (threads) per vector
    constexpr int kL = GRP / 8;               // lanes per group
    pdl_trigger();                            // an attention chained to this encode may start its set-up
    const Int4Side& sd = a.side[blockIdx.y];
    const uint32_t stride = gridDim.x * kThreads;
    // (whole vectors of a warp go out of range together: nwords is a multiple of kW, and
    // the shuffles below run over kL <= kW neighbours)
    for (uint32_t w0 = blockIdx.x * kThreads + threadIdx.x; w0 - (threadIdx.x & 31) < nwords; w0 += kUnroll * stride) {
        float v[kUnroll][8];
        Spot sp[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t w = w0 + u * stride;
            sp[u].blk = nullptr;
            if (w < nwords) {
                sp[u] = spot<D, GRP>(a, sd, w / kW);
                load8<DT>(sd.x, sp[u].xoff + 8 * (w % kW), a.vec16, v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int wi = (int)((w0 + u * stride) % kW);
            float lo = v[u][0], hi = v[u][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                lo = min_nan(lo, v[u][i]);
                hi = max_nan(hi, v[u][i]);
            }
#pragma unroll
            for (int o = 1; o < kL; o <<= 1) {
                lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
                hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
            }
            // clamping is monotone, so the range of the clamped values is the clamped range,
            // and a value outside it takes code 0 or 15 either way
            lo = max_nan(min_nan(lo, kMax), -kMax);
            hi = max_nan(min_nan(hi, kMax), -kMax);
            const __half zh = __float2half_rn(lo);
            const float z = __half2float(zh);
            const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(hi, z), kFifteenth));
            const float s = __half2float(sh);
            const float r = s > 0.f ? __frcp_rn(s) : 0.f;
            uint32_t word = 0;
#pragma unroll
            for (int i = 7; i >= 0; --i) {
                float t = __fmul_rn(__fsub_rn(v[u][i], z), r);
                t = fminf(fmaxf(t, 0.f), 15.f);
                // 1.5 2^23 + t rounds t to the nearest integer (half to even) in the low bits
                word = (word << 4) + (__float_as_uint(__fadd_rn(t, 12582912.f)) & 15u);
            }
            if (sp[u].blk) {
                const int tau = sp[u].tau;
                *reinterpret_cast<uint32_t*>(sp[u].blk + tau * (D / 2) + ((4 * wi) ^ int4_swizzle(D, tau))) = word;
                if (wi % kL == 0)
                    *reinterpret_cast<__half2*>(sp[u].blk + kBlockT * (D / 2) + (tau * (D / GRP) + wi / kL) * 4) =
                        __halves2half2(sh, zh);
            }
        }
    }
}

template <int D, int GRP, int DT>
__global__ void __launch_bounds__(kThreads) tq_int4_expand_kernel(const Int4CopyArgs a, uint32_t nwords) {
    using E = Elem<DT>;
    constexpr int kW = D / 8, kL = GRP / 8;
    const Int4Side& sd = a.side[blockIdx.y];
    const uint32_t stride = gridDim.x * kThreads;
    for (uint32_t w0 = blockIdx.x * kThreads + threadIdx.x; w0 < nwords; w0 += kUnroll * stride) {
        uint32_t word[kUnroll];
        __half2 pair[kUnroll];
        Spot sp[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t w = w0 + u * stride;
            sp[u].blk = nullptr;
            if (w < nwords) {
                sp[u] = spot<D, GRP>(a, sd, w / kW);
                const int wi = (int)(w % kW), tau = sp[u].tau;
                if (sp[u].blk) {
                    word[u] = *reinterpret_cast<const uint32_t*>(sp[u].blk + tau * (D / 2) + ((4 * wi) ^ int4_swizzle(D, tau)));
                    pair[u] = *reinterpret_cast<const __half2*>(sp[u].blk + kBlockT * (D / 2) + (tau * (D / GRP) + wi / kL) * 4);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!sp[u].blk) continue;
            const float s = __low2float(pair[u]), z = __high2float(pair[u]);
            typename E::T* p = static_cast<typename E::T*>(sd.x) + sp[u].xoff + 8 * ((w0 + u * stride) % kW);
            __align__(16) typename E::T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = E::from(fmaf((float)((word[u] >> (4 * i)) & 15u), s, z));
            if (a.vec16) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(e) / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(e)[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = e[i];
            }
        }
    }
}

template <int D, int GRP, int DT>
cudaError_t launch_copy(bool encode, const Int4CopyArgs& a, int num_sms, cudaStream_t s) {
    const uint32_t nwords = (uint32_t)(a.B * a.Hkv * a.T * (D / 8));        // below 2^31 (checked by the caller)
    const uint32_t need = (nwords + kThreads - 1) / kThreads;
    const uint32_t most = (uint32_t)num_sms * 8;
    const dim3 grid(need < most ? need : most, (unsigned)a.nsides);
    if (encode)
        tq_int4_encode_kernel<D, GRP, DT><<<grid, kThreads, 0, s>>>(a, nwords);
    else
        tq_int4_expand_kernel<D, GRP, DT><<<grid, kThreads, 0, s>>>(a, nwords);
    return cudaGetLastError();
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
