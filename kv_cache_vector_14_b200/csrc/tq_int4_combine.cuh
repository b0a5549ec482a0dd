// Merge of the partials of units cut by CTA borders, for the two 4-bit attention
// kernels: one warp per query row, the partials' (reference, sum) pairs over the
// lanes, then their accumulators with D/32 coordinates per lane.
#pragma once

#include "tq_int4.h"

namespace tqi {
namespace {

constexpr int kCombineWarps = 4;

// Split kernel: slot_rows rows of a partial slot, [row][D].  Block (c, y): rows kCombineWarps y ..
// of the unit that begins in CTA c; the unit index is (kv head, row group).
template <int D, int DT>
__global__ void __launch_bounds__(32 * kCombineWarps) tq_int4_combine_kernel(const __grid_constant__ Int4AttendArgs a,
                                                                            int slot_rows) {
    constexpr int E = D / 32;
    const int c = blockIdx.x, r = blockIdx.y * kCombineWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const int4 s = a.split[c];
    if (!s.w) return;
    const int groups = (a.rows + slot_rows - 1) / slot_rows;
    const int kv = s.y / groups, rt = s.y % groups;
    const int64_t row = (int64_t)rt * slot_rows + r;
    if (row >= a.rows) return;
    // the unit's partials: slot 1 of CTA c, slot 0 of CTAs c + 1 .. s.z
    const int n = s.z - c + 1;
    auto at = [&](int k) -> int64_t { return (2 * ((int64_t)c + k) + (k == 0 ? 1 : 0)) * slot_rows + r; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, a.part_ml[2 * at(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, A[E];
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] = 0.f;
    if (M != -INFINITY) {
        for (int k0 = 0; k0 < n; k0 += 32) {
            float f = 0.f;
            if (k0 + lane < n) {
                const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * at(k0 + lane));
                if (ml.x != -INFINITY) {
                    f = exp2f(ml.x - M);
                    L = fmaf(f, ml.y, L);
                }
            }
            const int m = n - k0 < 32 ? n - k0 : 32;
#pragma unroll 8
            for (int k = 0; k < m; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const float* p = a.part_acc + at(k0 + k) * D + E * lane;
                float v[E];
                if constexpr (E == 2) {
                    const float2 t = *reinterpret_cast<const float2*>(p);
                    v[0] = t.x; v[1] = t.y;
                } else {
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(p + e);
                        v[e] = t.x; v[e + 1] = t.y; v[e + 2] = t.z; v[e + 3] = t.w;
                    }
                }
                // a partial without a visible token may hold anything
#pragma unroll
                for (int e = 0; e < E; ++e) A[e] = fk != 0.f ? fmaf(fk, v[e], A[e]) : A[e];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    }
    const int64_t qi = row / a.G, g = row - qi * a.G;
    const int64_t out = ((s.x * a.Lq + qi) * a.Hq + (int64_t)kv * a.G + g) * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = M == -INFINITY ? 0.f : A[e] / L;
        if constexpr (DT == TQ_F32) static_cast<float*>(a.out)[out + e] = y;
        else if constexpr (DT == TQ_BF16) static_cast<__nv_bfloat16*>(a.out)[out + e] = __float2bfloat16_rn(y);
        else static_cast<__half*>(a.out)[out + e] = __float2half_rn(y);
    }
}

// Chunk kernel: slots [D][128 MT], the unit index is (row tile, kv head).  Lane = row, so that the
// partials are read in runs; block (c, y, z): rows 32 y .. and values 32 z .., eight per warp.
template <int D, int DT, int MT>
__global__ void __launch_bounds__(128) tq_int4_combine_tiles_kernel(const __grid_constant__ Int4AttendArgs a) {
    constexpr int R = 128 * MT;
    const int c = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * 32 + lane;
    const int col = blockIdx.z * 32 + (threadIdx.x >> 5) * 8;
    pdl_trigger();
    pdl_wait();
    const int4 s = a.split[c];
    if (!s.w) return;
    const int kv = s.y % (int)a.Hkv, rt = s.y / (int)a.Hkv;
    const int64_t row = (int64_t)rt * R + r;
    if (row >= a.rows) return;
    const int n = s.z - c + 1;
    auto slot = [&](int k) -> int64_t { return 2 * ((int64_t)c + k) + (k == 0 ? 1 : 0); };
    float M = -INFINITY, L = 0.f, A[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < n; ++k) M = fmaxf(M, a.part_ml[2 * (slot(k) * R + r)]);
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (slot(k) * R + r));
        if (ml.x == -INFINITY) continue;               // (a partial without a visible token may hold anything)
        const float f = exp2f(ml.x - M);
        L = fmaf(f, ml.y, L);
        const float* p = a.part_acc + (slot(k) * D + col) * R + r;
#pragma unroll
        for (int e = 0; e < 8; ++e) A[e] = fmaf(f, p[(int64_t)e * R], A[e]);
    }
    const int64_t qi = row / a.G, g = row - qi * a.G;
    const int64_t out = ((s.x * a.Lq + qi) * a.Hq + (int64_t)kv * a.G + g) * D + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) A[e] = M == -INFINITY ? 0.f : A[e] / L;
    if constexpr (DT == TQ_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) static_cast<float*>(a.out)[out + e] = A[e];
    } else {
        __align__(16) uint16_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[e] = DT == TQ_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(A[e])) : __half_as_ushort(__float2half_rn(A[e]));
        uint16_t* o = static_cast<uint16_t*>(a.out) + out;
        if (a.vec16) {
            *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(h);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = h[e];
        }
    }
}

template <int D, int DT, int MT>
cudaError_t launch_int4_combine_tiles(const Int4AttendArgs& a, int ctas, cudaStream_t s) {
    const int rows = a.rows < 128 * MT ? a.rows : 128 * MT;
    return launch_pdl(tq_int4_combine_tiles_kernel<D, DT, MT>, dim3(ctas, (rows + 31) / 32, D / 32), dim3(128), 0, s, a);
}

template <int D, int DT>
cudaError_t launch_int4_combine(const Int4AttendArgs& a, int slot_rows, int ctas, cudaStream_t s) {
    const int rows = a.rows < slot_rows ? a.rows : slot_rows;
    return launch_pdl(tq_int4_combine_kernel<D, DT>, dim3(ctas, (rows + kCombineWarps - 1) / kCombineWarps),
                      dim3(32 * kCombineWarps), 0, s, a, slot_rows);
}

}  // namespace
}  // namespace tqi
