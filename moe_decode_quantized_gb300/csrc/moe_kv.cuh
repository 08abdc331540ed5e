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
#include <cuda_bf16.h>

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

struct KvArgs {
    KvDims k;
    uint8_t *pages;
    long long n_slots;  // n_pages * page
    const uint16_t *src[2];
    long long tok_stride[2], head_stride[2];  // elements
    const int32_t *slots;
    void *out[2];
    int tokens;
    uint32_t *status;
};

// A warp of both kernels works on consecutive tokens of one head the way the
// cache stores them, so that where the tokens' slots are consecutive and
// aligned -- a prompt, a long context -- its accesses are whole lines: lanes
// are (token, piece of the row) for K, (eighth of the row, pair of tokens)
// for V. Any slots are right.

// the token of eight that this lane works on; which: V's token of the pair
__device__ __forceinline__ int kv_tile_token(bool value, int lane, int which)
{
    return value ? (lane & 3) * 2 + which : lane >> 2;
}

// checked slot of a token of the call: -1 where there is nothing to do
__device__ __forceinline__ int kv_slot(const KvArgs &a, int token)
{
    if (token >= a.tokens)
        return -1;
    const int slot = a.slots[token];
    if (slot >= a.n_slots || slot < -1) {
        if (a.status)
            atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
        return -1;
    }
    return slot;
}

template <int FMT, int D>
__device__ __forceinline__ uint8_t *kv_half(const KvArgs &a, int slot, int head, int value)
{
    constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2;
    constexpr int HALF = 16 * RB + 16 * (D / MOE_KV_GROUP) * (FMT == MOE_KV_Q8 ? 2 : 4);
    const unsigned page = (unsigned)slot / (unsigned)a.k.page, in = (unsigned)slot - page * a.k.page;
    const size_t block = ((size_t)page * a.k.heads + head) * (a.k.page / 16) + in / 16;
    return a.pages + block * (2 * HALF) + (value ? HALF : 0);
}

// rint(y / f) of a lane's group values, f > 0 (inv = 1 / f, or both 0), as
// 1.5 2^23 + code: the product with the reciprocal is within 2^-16 of the
// quotient (codes up to 127), so its rounding is the quotient's unless it
// lies within 2^-15 of the middle between two codes; `near` then says that
// the quotients have to be divided out (ties, and what rounds to one).
__device__ __forceinline__ float kv_round(float y, float inv, bool &near)
{
    const float q = __fmul_rn(y, inv), t = __fadd_rn(q, 12582912.0f);
    near |= fabsf(__fsub_rn(q, __fadd_rn(t, -12582912.0f))) >= 0.5f - 3.0517578e-5f;
    return t;
}

// the same by the division itself
__device__ __forceinline__ float kv_divide(float y, float f)
{
    return __fadd_rn(f > 0.0f ? rintf(__fdiv_rn(y, f)) : 0.0f, 12582912.0f);
}

__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162 *>(&v); }

// 32 bytes at once (8 words); p 32-byte aligned
__device__ __forceinline__ void ld_global_32(const void *p, uint32_t *w)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// Quantises and writes one lane's piece of a row: N values from dimension
// piece N. A group of 32 is the lane's own (N = 32) or shared with the lanes
// of the row's neighbouring pieces, 1 (K) or 4 (V) apart. The scale is rounded
// up and the minimum down to f16, so that no code is clipped: |x - value| <=
// scale / 2 over the whole range. ALIGN: 32, 16 or 2, what rows and strides
// are multiples of in bytes.
template <int FMT, int D, int N, bool VALUE, int ALIGN>
__device__ __forceinline__ void kv_append_piece(const KvArgs &a, int token, int head, int lane, int piece)
{
    constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2, GR = D / MOE_KV_GROUP, BYTES = N * RB / D;
    uint32_t in[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        in[i] = 0;
    if (token < a.tokens) {  // also a skipped token's: the load does not wait for the slot
        const uint16_t *p = a.src[VALUE] + token * a.tok_stride[VALUE] + head * a.head_stride[VALUE] + piece * N;
        if constexpr (ALIGN == 32 && N >= 16) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 8)
                ld_global_32(p + 2 * i, in + i);
        } else if constexpr (ALIGN >= 16) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(p + 2 * i);
                in[i] = q.x;
                in[i + 1] = q.y;
                in[i + 2] = q.z;
                in[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                in[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
    }
    const int slot = kv_slot(a, token);
    // the extremes, two values at a time; NaN stays, and with what is out of range leads to the slow way
    __nv_bfloat162 least = bf2(in[0]), most = least;
#pragma unroll
    for (int i = 1; i < N / 2; ++i) {
        least = __hmin2_nan(least, bf2(in[i]));
        most = __hmax2_nan(most, bf2(in[i]));
    }
    float lo = __low2float(__hmin2_nan(least, __lowhigh2highlow(least)));
    float hi = __low2float(__hmax2_nan(most, __lowhigh2highlow(most)));
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = i & 1 ? bf16_hi(in[i >> 1]) : bf16_lo(in[i >> 1]);
    if (!(lo >= -MOE_KV_LIMIT && hi <= MOE_KV_LIMIT)) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            odd |= !(fabsf(v[i]) <= 3.402823466e38f);
            v[i] = fminf(fmaxf(v[i] == v[i] ? v[i] : 0.0f, -MOE_KV_LIMIT), MOE_KV_LIMIT);
            lo = i ? fminf(lo, v[i]) : v[i];
            hi = i ? fmaxf(hi, v[i]) : v[i];
        }
        if (odd && slot >= 0 && a.status)
            atomicOr(a.status, (uint32_t)MOE_WS_NONFINITE);
    }
#pragma unroll
    for (int m = 1; m < MOE_KV_GROUP / N; m *= 2) {  // every lane of the warp is here
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m * (VALUE ? 4 : 1)));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m * (VALUE ? 4 : 1)));
    }
    if (slot < 0)
        return;
    uint8_t *half = kv_half<FMT, D>(a, slot, head, VALUE);
    const int t = slot & 15, g = piece * N / MOE_KV_GROUP;
    const bool first = piece * N % MOE_KV_GROUP == 0;  // of the group's lanes
    __half *s = reinterpret_cast<__half *>(half + 16 * RB);
    uint32_t w[BYTES / 4];
    float code[N];
    bool near = false;
    if (FMT == MOE_KV_Q8) {
        const __half d = __float2half_ru(__fdiv_rn(fmaxf(hi, -lo), 127.0f));
        const float f = __half2float(d), inv = f > 0.0f ? __fdiv_rn(1.0f, f) : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            code[i] = kv_round(v[i], inv, near);
        if (near) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                code[i] = kv_divide(v[i], f);
        }
#pragma unroll
        for (int i = 0; i < N; i += 4) {  // the codes' low bytes, and 128 added
            const uint32_t x = __byte_perm(__float_as_uint(code[i]), __float_as_uint(code[i + 1]), 0x0040);
            const uint32_t y = __byte_perm(__float_as_uint(code[i + 2]), __float_as_uint(code[i + 3]), 0x0040);
            w[i / 4] = __byte_perm(x, y, 0x5410) ^ 0x80808080u;
        }
        if (first)
            s[VALUE ? g * 16 + t : t * GR + g] = d;
    } else {
        const __half m = __float2half_rd(lo);
        const float fm = __half2float(m);
        const __half d = __float2half_ru(__fdiv_rn(__fsub_rn(hi, fm), 15.0f));
        const float f = __half2float(d), inv = f > 0.0f ? __fdiv_rn(1.0f, f) : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            code[i] = kv_round(__fsub_rn(v[i], fm), inv, near);
        if (near) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                code[i] = kv_divide(__fsub_rn(v[i], fm), f);
        }
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            w[i / 8] = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[i / 8] |= (__float_as_uint(code[i + k]) & 15u) << (4 * (k / 2) + 16 * (k & 1));
        }
        if (first) {
            s[VALUE ? g * 16 + t : (t * GR + g) * 2] = d;
            s[VALUE ? (GR + g) * 16 + t : (t * GR + g) * 2 + 1] = m;
        }
    }
    constexpr int PIECE = VALUE ? RB / 8 : RB / 4;  // bytes of a lane of the layout
    const int i = piece * BYTES, x = (VALUE ? (t >> 3) * 2 + (t & 1) : t >> 3) * PIECE + i % PIECE;
    const int at = VALUE ? i / PIECE * 4 + ((t & 7) >> 1) : (t & 7) * 4 + i / PIECE;
    uint8_t *p = half + (x >> 4) * 512 + at * 16 + (x & 15);
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int k = 0; k < BYTES / 16; ++k)
            *reinterpret_cast<uint4 *>(p + k * 512) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else if constexpr (BYTES == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

#define MOE_KV_THREADS 256

// tokens of a warp: K's pieces are 16 values, V's an eighth of a row
template <int D, bool VALUE>
__host__ __device__ constexpr int kv_append_tokens() { return VALUE ? 4 : 512 / D; }

// Quantises and writes rows: blockIdx.y = head x 2 + {K, V}. Bound by the
// reads and writes for a prompt, by latency for a decode step.
template <int FMT, int D, int ALIGN>
__global__ void __launch_bounds__(MOE_KV_THREADS) moe_kv_append_kernel(const KvArgs a)
{
    const int lane = threadIdx.x & 31, head = blockIdx.y >> 1;
    const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if ((blockIdx.y & 1) == 0) {
        const int token = warp * kv_append_tokens<D, false>();
        if (token < a.tokens)
            kv_append_piece<FMT, D, 16, false, ALIGN>(a, token + lane / (D / 16), head, lane, lane % (D / 16));
    } else {
        const int token = (warp >> 1) * 8;  // two warps eight tokens
        if (token < a.tokens)
            kv_append_piece<FMT, D, D / 8, true, ALIGN>(a, token + kv_tile_token(true, lane, warp & 1), head, lane,
                                                        lane >> 2);
    }
}

// 32 bytes at once (8 words); p 32-byte aligned
__device__ __forceinline__ void st_global_32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// one thread's piece of a row (BYTES of codes) as numbers
template <int FMT, int D, bool VALUE, bool F32, bool WIDE>
__device__ __forceinline__ void kv_read_piece(const KvArgs &a, int token, int head, int lane, int chunk)
{
    constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2, GR = D / MOE_KV_GROUP;
    constexpr int PIECE = VALUE ? RB / 8 : RB / 4, BYTES = PIECE < 16 ? PIECE : 16;
    constexpr int N = BYTES * D / RB, WORDS = BYTES / 4;
    if (token >= a.tokens)
        return;
    const int slot = kv_slot(a, token);
    const int d0 = (VALUE ? lane >> 2 : lane & 3) * (PIECE * D / RB) + chunk * N;  // first dimension
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = 0.0f;
    if (slot >= 0) {
        const uint8_t *half = kv_half<FMT, D>(a, slot, head, VALUE);
        const int t = slot & 15, g = d0 / MOE_KV_GROUP;
        const int x = (VALUE ? (t >> 3) * 2 + (t & 1) : t >> 3) * PIECE + chunk * 16;
        const int at = VALUE ? (lane & ~3) + ((t & 7) >> 1) : (t & 7) * 4 + (lane & 3);  // the slot's lane
        const uint8_t *p = half + (x >> 4) * 512 + at * 16 + (x & 15);
        uint32_t w[WORDS];
        if constexpr (BYTES == 16) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            w[0] = q.x;
            w[1] = q.y;
            w[2] = q.z;
            w[3] = q.w;
        } else if constexpr (BYTES == 8) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            w[0] = q.x;
            w[1] = q.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
        const __half *s = reinterpret_cast<const __half *>(half + 16 * RB);
        // a code in the low bits of 2^23 is 2^23 + code: exact, as is its product with the f16 scale
        if (FMT == MOE_KV_Q8) {
            const float d = __half2float(s[VALUE ? g * 16 + t : t * GR + g]);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = (__uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7440 | (i & 3))) - 8388736.0f) * d;
        } else {
            const float d = __half2float(s[VALUE ? g * 16 + t : (t * GR + g) * 2]);
            const float m = __half2float(s[VALUE ? (GR + g) * 16 + t : (t * GR + g) * 2 + 1]);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t c = w[i / 8] >> (4 * (i % 8 / 2) + 16 * (i & 1)) & 15u;
                v[i] = fmaf(__uint_as_float(c | 0x4B000000u) - 8388608.0f, d, m);
            }
        }
    }
    constexpr int OUT = F32 ? N : N / 2;  // words
    uint32_t o[OUT];
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
        if (F32) {
            o[i] = __float_as_uint(v[i]);
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    uint8_t *q = static_cast<uint8_t *>(a.out[VALUE]) + (((size_t)token * a.k.heads + head) * D + d0) * (F32 ? 4 : 2);
    if constexpr (OUT >= 8 && WIDE) {
#pragma unroll
        for (int i = 0; i < OUT; i += 8)
            st_global_32(q + 4 * i, o + i);
    } else {
#pragma unroll
        for (int i = 0; i < OUT; i += 4)
            *reinterpret_cast<uint4 *>(q + 4 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
}

// threads of a tile of eight tokens of one head: 16-byte (or smaller) pieces of codes
template <int FMT, int D, bool VALUE>
__host__ __device__ constexpr int kv_read_threads()
{
    constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2, PIECE = VALUE ? RB / 8 : RB / 4;
    return 8 * RB / (PIECE < 16 ? PIECE : 16);
}

// Reads rows back: blockIdx.y = head x 2 + {K, V}; a thread one piece of codes
// as 8, 16 or 32 numbers, rounded once to bf16 or kept in f32. WIDE: outputs
// on 32-byte boundaries (the stores are then whole sectors). Bound by the
// reads and writes.
template <int FMT, int D, bool F32, bool WIDE>
__global__ void __launch_bounds__(MOE_KV_THREADS) moe_kv_read_kernel(const KvArgs a)
{
    constexpr int NK = kv_read_threads<FMT, D, false>(), NV = kv_read_threads<FMT, D, true>();
    const int head = blockIdx.y >> 1;
    const int lane = threadIdx.x & 31;
    if ((blockIdx.y & 1) == 0) {
        const int tile = blockIdx.x * (MOE_KV_THREADS / NK) + threadIdx.x / NK;
        kv_read_piece<FMT, D, false, F32, WIDE>(a, tile * 8 + kv_tile_token(false, lane, 0), head, lane,
                                                threadIdx.x % NK / 32);
    } else {
        const int tile = blockIdx.x * (MOE_KV_THREADS / NV) + threadIdx.x / NV, x = threadIdx.x % NV / 32;
        kv_read_piece<FMT, D, true, F32, WIDE>(a, tile * 8 + kv_tile_token(true, lane, x & 1), head, lane, x >> 1);
    }
}

}  // namespace moe
