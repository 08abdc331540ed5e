// moe_kv.cuh -- the quantised paged key/value cache: its layout, the kernel
// that quantises rows as they are written, and the one that reads them back.
//
// Layout. A page holds page_size tokens of one layer; per kv head it is
// page_size / 16 blocks of 16 tokens, and a block is contiguous:
//   K codes | K scales | V codes | V scales
// Every kernel that streams the cache moves whole blocks with one bulk copy
// and feeds them to warp-level matrix instructions, so the codes are stored
// in the order in which a warp's lanes take them: lane l owns the 16-byte
// pieces at (x / 16) * 512 + l * 16, x its byte count, and a 128-bit
// shared-memory load by 32 lanes is one conflict-free run. With t the token
// in the block, d the dimension, RB = codes bytes of a row:
//   K: lane = (t % 8) * 4 + d / (D / 4), then token half t / 8, then the rest
//      of d: a lane holds a quarter of a row for tokens t and t + 8;
//   V: lane = d / (D / 8) * 4 + (t % 8) / 2, then t / 8, t % 2, the rest of
//      d: a lane holds an eighth of a row for tokens 2 i, 2 i + 1, 2 i + 8,
//      2 i + 9.
// These are the B fragments of a 16x8x16 product under a permutation of the
// contracted index (K) and of the columns (V), which the query fragments and
// the output undo. 4-bit codes are packed eight to a 32-bit word, code i at
// bit 4 (i / 2) + 16 (i % 2), so that (w >> 4 j) & 0x000F000F are codes 2j, 2j + 1.
// Scales are f16, one (Q8) or a scale and a minimum (Q4) per 32 values:
// K [token][group][1 or 2], V [1 or 2][group][token].
#pragma once
#include "moe_common.cuh"

#define MOE_KV_GROUP 32
#define MOE_KV_BLOCK 16        // tokens of a block
#define MOE_KV_LIMIT 60000.0f  // largest magnitude held (f16 operands with room for the rounding of the scale)

namespace moe {

struct KvDims {
    int dim, heads, page, fmt;  // page: tokens of a page
    __host__ __device__ int row_bytes() const { return fmt == MOE_KV_Q8 ? dim : dim / 2; }
    __host__ __device__ int groups() const { return dim / MOE_KV_GROUP; }
    __host__ __device__ int per() const { return fmt == MOE_KV_Q8 ? 1 : 2; }  // f16 words of a group
    __host__ __device__ int scale_bytes() const { return 16 * groups() * per() * 2; }
    __host__ __device__ int half_bytes() const { return 16 * row_bytes() + scale_bytes(); }  // K or V of a block
    __host__ __device__ int block_bytes() const { return 2 * half_bytes(); }
    __host__ __device__ size_t page_bytes() const { return (size_t)heads * (page / 16) * block_bytes(); }
};

// byte offset in a block's K (V) codes of code byte i (0 <= i < RB) of token t
__device__ __forceinline__ int kv_code_at(const KvDims &k, bool value, int t, int i)
{
    const int rb = k.row_bytes(), piece = value ? rb / 8 : rb / 4;
    const int lane = value ? i / piece * 4 + (t & 7) / 2 : (t & 7) * 4 + i / piece;
    const int x = (value ? (t / 8) * 2 + (t & 1) : t / 8) * piece + i % piece;
    return (x >> 4) * 512 + lane * 16 + (x & 15);
}

// index of the f16 word z (0: scale, 1: minimum) of group g of token t
__device__ __forceinline__ int kv_scale_at(const KvDims &k, bool value, int t, int g, int z)
{
    return value ? (z * k.groups() + g) * 16 + t : (t * k.groups() + g) * k.per() + z;
}

struct KvArgs {
    KvDims k;
    uint8_t *pages;
    long long n_slots;  // n_pages * page
    const uint16_t *src[2];
    long long tok_stride[2], head_stride[2];  // elements
    const int32_t *slots;
    void *out[2];
    int out_f32;
    int tokens;
    uint32_t *status;
};

__device__ __forceinline__ uint8_t *kv_half(const KvArgs &a, int slot, int head, int value)
{
    const int page = slot / a.k.page, in = slot % a.k.page;
    const size_t block = ((size_t)page * a.k.heads + head) * (a.k.page / 16) + in / 16;
    return a.pages + block * a.k.block_bytes() + (value ? a.k.half_bytes() : 0);
}

// Quantises and writes rows. Eight values a thread, D / 8 threads a row (a
// row: K or V of one token and head), four neighbouring lanes a group. The
// scale is rounded up and the minimum down to f16, so that no code is
// clipped: |x - value| <= scale / 2 for the whole range. VEC: rows that a
// 16-byte load can take (16-byte aligned with strides of 8 elements).
template <bool VEC>
__global__ void __launch_bounds__(256) moe_kv_append_kernel(const KvArgs a)
{
    const int per_row = a.k.dim / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = id / per_row;
    const int part = (int)(id % per_row);
    const bool live = row < 2ll * a.tokens * a.k.heads;
    int slot = -1, head = 0, value = 0;
    long long token = 0;
    if (live) {
        head = (int)(row % a.k.heads);
        token = row / a.k.heads;
        value = token >= a.tokens;
        token -= value ? a.tokens : 0;
        slot = a.slots[token];
        if (slot >= a.n_slots || slot < -1) {
            if (a.status)
                atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
            slot = -1;
        }
    }
    float v[8];
    bool odd = false;
    if (slot >= 0) {
        const uint16_t *p = a.src[value] + token * a.tok_stride[value] + head * a.head_stride[value] + part * 8;
        uint32_t w[4];
        if (VEC) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
            odd |= !(fabsf(f) <= 3.402823466e38f);
            f = f == f ? f : 0.0f;
            v[i] = fminf(fmaxf(f, -MOE_KV_LIMIT), MOE_KV_LIMIT);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.0f;
    }
    if (odd && a.status)
        atomicOr(a.status, (uint32_t)MOE_WS_NONFINITE);
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int m = 1; m < 4; m *= 2) {  // all 32 lanes take part: rows are whole groups of four lanes
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    if (slot < 0)
        return;
    uint8_t *half = kv_half(a, slot, head, value);
    const int t = slot % 16, g = part / 4;
    __half *scales = reinterpret_cast<__half *>(half + 16 * a.k.row_bytes());
    if (a.k.fmt == MOE_KV_Q8) {
        const __half d = __float2half_ru(__fdiv_rn(fmaxf(hi, -lo), 127.0f));
        const float f = __half2float(d);
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = f > 0.0f ? rintf(__fdiv_rn(v[i], f)) : 0.0f;
            c[i >> 2] |= (uint32_t)((int)fminf(fmaxf(r, -127.0f), 127.0f) + 128) << (8 * (i & 3));
        }
        *reinterpret_cast<uint2 *>(half + kv_code_at(a.k, value, t, part * 8)) = make_uint2(c[0], c[1]);
        if ((part & 3) == 0)
            scales[kv_scale_at(a.k, value, t, g, 0)] = d;
    } else {
        const __half m = __float2half_rd(lo);
        const float fm = __half2float(m);
        const __half d = __float2half_ru(__fdiv_rn(__fsub_rn(hi, fm), 15.0f));
        const float f = __half2float(d);
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = f > 0.0f ? rintf(__fdiv_rn(__fsub_rn(v[i], fm), f)) : 0.0f;
            c |= (uint32_t)(int)fminf(fmaxf(r, 0.0f), 15.0f) << (4 * (i >> 1) + 16 * (i & 1));
        }
        *reinterpret_cast<uint32_t *>(half + kv_code_at(a.k, value, t, part * 4)) = c;
        if ((part & 3) == 0) {
            scales[kv_scale_at(a.k, value, t, g, 0)] = d;
            scales[kv_scale_at(a.k, value, t, g, 1)] = m;
        }
    }
}

// Eight values of a row of the cache in f32. c + 128 (Q8) and the 4-bit codes
// times the scale are exact in f32; Q4's sum is rounded once.
__device__ __forceinline__ void kv_values8(const KvDims &k, const uint8_t *half, bool value, int t, int part, float (&v)[8])
{
    const __half *scales = reinterpret_cast<const __half *>(half + 16 * k.row_bytes());
    const int g = part / 4;
    const float d = __half2float(scales[kv_scale_at(k, value, t, g, 0)]);
    if (k.fmt == MOE_KV_Q8) {
        const uint2 c = *reinterpret_cast<const uint2 *>(half + kv_code_at(k, value, t, part * 8));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (float)((int)((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 255u) - 128) * d;
    } else {
        const float m = __half2float(scales[kv_scale_at(k, value, t, g, 1)]);
        const uint32_t c = *reinterpret_cast<const uint32_t *>(half + kv_code_at(k, value, t, part * 4));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fmaf((float)(c >> (4 * (i >> 1) + 16 * (i & 1)) & 15u), d, m);
    }
}

// Reads rows back: eight values a thread, rounded once to bf16 or kept in f32.
__global__ void __launch_bounds__(256) moe_kv_read_kernel(const KvArgs a)
{
    const int per_row = a.k.dim / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = id / per_row;
    const int part = (int)(id % per_row);
    if (row >= 2ll * a.tokens * a.k.heads)
        return;
    const int head = (int)(row % a.k.heads);
    long long token = row / a.k.heads;
    const int value = token >= a.tokens;
    token -= value ? a.tokens : 0;
    int slot = a.slots[token];
    if (slot >= a.n_slots || slot < -1) {
        if (a.status)
            atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
        slot = -1;
    }
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (slot >= 0)
        kv_values8(a.k, kv_half(a, slot, head, value), value, slot % 16, part, v);
    const long long at = (token * a.k.heads + head) * a.k.dim + part * 8;
    if (a.out_f32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out[value]) + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out[value]) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace moe
