// Internal declarations of the 4-bit cache: the packed format, kernel arguments
// and launchers shared by the encode, attention and API translation units.
//
// A vector of d values is cut into groups of 32, 64 or 128; a group stores an
// fp16 scale and an fp16 zero (its minimum), a value stands for zero + scale c
// with a 4-bit code c.  A block holds 64 tokens: 64 x d/2 bytes of codes, then
// 64 x d/group (scale, zero) pairs.  Byte j of a token's codes holds values 2j
// (low nibble) and 2j + 1; it is stored at j ^ int4_swizzle(d, token), which
// moves whole 16-byte pieces so that the attention kernel's shared-memory reads
// (four or eight tokens at once, 4 to 16 bytes of each) hit different banks.
#pragma once

#include "tq_internal.h"

namespace tqi {

__host__ __device__ constexpr int int4_code_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int int4_pair_bytes(int d, int group) { return 4 * (d / group); }
__host__ __device__ constexpr int64_t int4_block_bytes(int d, int group) {
    return (int64_t)kBlockT * (int4_code_bytes(d) + int4_pair_bytes(d, group));
}
__host__ __device__ constexpr int int4_swizzle(int d, int token) {
    return ((d >= 128 ? (token & 2) : 0) | (d == 256 ? (token & 1) << 2 : 0)) * 16;
}
inline bool int4_group_ok(int d, int group) { return (group == 32 || group == 64 || group == 128) && group <= d; }

// One or two caches (a layer's K and V) written or read by one launch.
struct Int4Side {
    void* x;                  // the vectors: input of an encode, output of an expand
    uint8_t* cache;
    const int32_t* table;     // paged cache: [B*Hkv][NB] pool blocks, or null
    int64_t pool;
};
struct Int4CopyArgs {
    Int4Side side[2];
    int nsides;
    int64_t sb, sh, st;       // element strides of x
    int64_t B, Hkv, T;
    const int32_t* pos;       // device [B] first token of each sequence, or null: t0
    int64_t t0, Tcap, NB;
    int vec16;                // every vector of x starts on a 16-byte boundary
    int* err;
    FastDiv fdT, fdH;
};

// Attention of Lq queries a sequence, causal at the end, over 4-bit caches.
struct Int4AttendArgs {
    const void* q;            // [B][Lq][Hq][d]
    void* out;                // the same shape and type
    const uint8_t* kc;
    const uint8_t* vc;
    const int32_t* ktable;
    const int32_t* vtable;
    int64_t kpool, vpool;
    const int32_t* lens;      // device [B], or null: T
    int64_t T, add;           // tokens of sequence b: (lens ? lens[b] : T) + add
    int64_t Tcap, NB;
    int64_t B, Hq, Hkv, Lq;
    int G;                    // query heads per kv head
    int rows;                 // Lq G query rows per kv head
    float scale_log2;         // softmax scale * log2(e)
    float* part_ml;           // [CTA][2][rows of a slot][2] (reference exponent, sum)
    float* part_acc;          // [CTA][2][rows of a slot][d]
    int4* split;              // [CTA] a unit that begins in this CTA and goes on: {sequence, unit, last CTA, 1}
    int* err;
    int first_wait;
    int vec16;                // q and out start on 16-byte boundaries
};
constexpr int kInt4MaxCtas = 256;
// Rows of a partial slot, by which a call's kernel is known: 8 the split kernel
// (tq_int4_attend.cu), 128 and 256 the chunk kernel (tq_int4_chunk.cu).
int int4_slot_rows(int d, tq_dtype dt, int rows);

cudaError_t launch_int4_encode(int d, int group, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_int4_expand(int d, int group, tq_dtype dt, const Int4CopyArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_int4_attend(int d, int group, tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_int4_chunk(int d, int group, tq_dtype dt, const Int4AttendArgs& a, int num_sms, cudaStream_t s);

}  // namespace tqi
