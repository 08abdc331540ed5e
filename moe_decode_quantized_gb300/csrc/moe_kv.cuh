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
    unsigned long long per_page;  // ceil(2^36 / (page / 16)): block / (page / 16) = block * per_page >> 36, block < 2^27
    uint32_t *status;
};

// A warp of both kernels works on consecutive tokens of one head, so that where
// the tokens' slots are consecutive and aligned -- a prompt, a long context --
// its accesses are whole sectors. The writer's lanes are (token, piece of the
// row), whose loads are whole rows; the reader's the cache's own (token, piece)
// for K, (eighth of the row, pair of tokens) for V. Any slots are right.

// the token of eight that a reading lane works on; which: V's token of the pair
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
    const unsigned at = (unsigned)slot / 16, page = (unsigned)(at * a.per_page >> 36), per = a.k.page / 16;
    const size_t block = ((size_t)page * a.k.heads + head) * per + (at - page * per);
    return a.pages + block * (2 * HALF) + (value ? HALF : 0);
}

// The codes rint(RN(y / f)) of a pair of values as 1.5 2^23 (Q8: + 128) +
// code, f a scale in f16 and inv = RN(1 / f) (both 0: codes of 0). The quotient
// by one step of correction (Markstein 1990): q = RN(y inv) is within 1.5 ulp,
// its remainder y - f q is exact, and q + remainder inv is within 2^-23 ulp of
// y / f before it is rounded; f's 11 bits keep y / f 2^-12 ulp or more from
// the middle between two floats, so the result is RN(y / f). (Numbers of few
// bits make ties between codes common; a product with inv alone, the rare
// doubtful ones divided out, sent 40 % of the warps to that branch.)
template <int FMT>
__device__ __forceinline__ void kv_codes(const F2 &y, const F2 &inv, const F2 &minus_f, float *code)
{
    constexpr float MAGIC = FMT == MOE_KV_Q8 ? 12583040.0f : 12582912.0f;
    const F2 q = mul2(y, inv);
    add2(fma2(fma2(minus_f, q, y), inv, q), F2(MAGIC, MAGIC)).get(code[0], code[1]);
}

__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162 *>(&v); }

// 32 bytes at once (8 words); p 32-byte aligned
__device__ __forceinline__ void ld_global_32(const void *p, uint32_t *w)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// value i of a row's words; as it is held; values i and i + 1
__device__ __forceinline__ float kv_value(const uint32_t *in, int i) { return i & 1 ? bf16_hi(in[i >> 1]) : bf16_lo(in[i >> 1]); }

__device__ __forceinline__ float kv_held(const uint32_t *in, int i)
{
    const float v = kv_value(in, i);
    return fminf(fmaxf(v == v ? v : 0.0f, -MOE_KV_LIMIT), MOE_KV_LIMIT);
}

template <bool SLOW>
__device__ __forceinline__ F2 kv_pair(const uint32_t *in, int i)
{
    return SLOW ? F2(kv_held(in, i), kv_held(in, i + 1)) : F2(kv_value(in, i), kv_value(in, i + 1));
}

// Values of a lane: a group, whose scale it then works out alone (65536 tokens of 8 heads of 128 in Q8: 64 us, with
// half a group 70), but half of one where rows are loaded two bytes at a time (157 and 117 us) or are of 64
template <int D, int ALIGN>
__host__ __device__ constexpr int kv_append_values() { return D >= 128 && ALIGN > 2 ? 32 : 16; }

// tokens of a warp
template <int D, int ALIGN>
__host__ __device__ constexpr int kv_append_tokens() { return 32 * kv_append_values<D, ALIGN>() / D; }

// Quantises and writes one lane's piece of a row: N values from dimension
// piece N. The scale is rounded up and the minimum down to f16, so that no
// code is clipped: |x - value| <= scale / 2 over the whole range. ALIGN: 32,
// 16 or 2, what rows and strides are multiples of in bytes (65536 tokens in Q8:
// 64, 69 and 117 us; views at odd boundaries are rare, so no wider loads are
// shifted for them).
template <int FMT, int D, bool VALUE, int ALIGN>
__device__ __forceinline__ void kv_append_piece(const KvArgs &a, int token, int head, int piece)
{
    constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2, GR = D / MOE_KV_GROUP, N = kv_append_values<D, ALIGN>(), BYTES = N * RB / D;
    uint32_t in[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        in[i] = 0;
    if (token < a.tokens) {  // also a skipped token's: the load does not wait for the slot
        const uint16_t *p = a.src[VALUE] + token * a.tok_stride[VALUE] + head * a.head_stride[VALUE] + piece * N;
        if constexpr (ALIGN == 32) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 8)
                ld_global_32(p + 2 * i, in + i);
        } else if constexpr (ALIGN == 16) {
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
    // the extremes (Q8: of the magnitudes), two values at a time; NaN stays, and with what is out of range leads to
    // the slow way
    __nv_bfloat162 least = bf2(in[0]), most = FMT == MOE_KV_Q8 ? __habs2(least) : least;
#pragma unroll
    for (int i = 1; i < N / 2; ++i) {
        if (FMT == MOE_KV_Q4)
            least = __hmin2_nan(least, bf2(in[i]));
        most = __hmax2_nan(most, FMT == MOE_KV_Q8 ? __habs2(bf2(in[i])) : bf2(in[i]));
    }
    float hi = __low2float(__hmax2_nan(most, __lowhigh2highlow(most)));
    float lo = FMT == MOE_KV_Q8 ? -hi : __low2float(__hmin2_nan(least, __lowhigh2highlow(least)));
    const bool slow = !(lo >= -MOE_KV_LIMIT && hi <= MOE_KV_LIMIT);
    if (slow) {
        bool odd = false;
        lo = MOE_KV_LIMIT;
        hi = -MOE_KV_LIMIT;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            odd |= !(fabsf(kv_value(in, i)) <= 3.402823466e38f);
            lo = fminf(lo, kv_held(in, i));
            hi = fmaxf(hi, kv_held(in, i));
        }
        if (FMT == MOE_KV_Q8)
            hi = fmaxf(hi, -lo);
        if (odd && slot >= 0 && a.status)
            atomicOr(a.status, (uint32_t)MOE_WS_NONFINITE);
    }
#pragma unroll
    for (int m = 1; m < MOE_KV_GROUP / N; m *= 2) {  // every lane of the warp is here
        if (FMT == MOE_KV_Q4)
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    if (slot < 0)
        return;
    uint8_t *half = kv_half<FMT, D>(a, slot, head, VALUE);
    const int t = slot & 15, g = piece * N / MOE_KV_GROUP;
    const bool first = piece * N % MOE_KV_GROUP == 0;  // of the group's lanes
    __half *s = reinterpret_cast<__half *>(half + 16 * RB);
    uint32_t w[BYTES / 4];
    const float m = FMT == MOE_KV_Q8 ? 0.0f : __half2float(__float2half_rd(lo));
    const __half d = __float2half_ru(__fdiv_rn(FMT == MOE_KV_Q8 ? hi : __fsub_rn(hi, m), FMT == MOE_KV_Q8 ? 127.0f : 15.0f));
    const float f = __half2float(d), inv = f > 0.0f ? __fdiv_rn(1.0f, f) : 0.0f;
    const F2 inv2(inv, inv), minus_f(-f, -f), minus_m(-m, -m);
    auto words = [&](auto held) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            float c[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                F2 y = kv_pair<decltype(held)::value>(in, i + k);
                if (FMT == MOE_KV_Q4)
                    y = add2(y, minus_m);
                kv_codes<FMT>(y, inv2, minus_f, c + k);
            }
            if (FMT == MOE_KV_Q8) {  // the low bytes: codes, 128 added
                w[i / 4] = __byte_perm(__byte_perm(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x0040),
                                       __byte_perm(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x0040), 0x5410);
            } else {  // the low halves: codes
                const uint32_t u = __byte_perm(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x5410) +
                                   (__byte_perm(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x5410) << 4);
                w[i / 8] = i & 4 ? w[i / 8] + (u << 8) : u;
            }
        }
    };
    if (slow)
        words(IntC<1>{});
    else
        words(IntC<0>{});
    if (first && FMT == MOE_KV_Q8) {
        s[VALUE ? g * 16 + t : t * GR + g] = d;
    } else if (first) {
        s[VALUE ? g * 16 + t : (t * GR + g) * 2] = d;
        s[VALUE ? (GR + g) * 16 + t : (t * GR + g) * 2 + 1] = __float2half_rn(m);  // exact
    }
    constexpr int PIECE = VALUE ? RB / 8 : RB / 4;  // bytes of a lane of the layout
    constexpr int C = BYTES < PIECE ? (BYTES < 16 ? BYTES : 16) : (PIECE < 16 ? PIECE : 16);  // stored at once
#pragma unroll
    for (int k = 0; k < BYTES / C; ++k) {
        const int i = piece * BYTES + k * C, x = (VALUE ? (t >> 3) * 2 + (t & 1) : t >> 3) * PIECE + i % PIECE;
        const int at = VALUE ? i / PIECE * 4 + ((t & 7) >> 1) : (t & 7) * 4 + i / PIECE;
        uint8_t *p = half + (x >> 4) * 512 + at * 16 + (x & 15);
        if constexpr (C == 16)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        else if constexpr (C == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[2 * k], w[2 * k + 1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[k];
    }
}

#define MOE_KV_THREADS 256

// Quantises and writes rows: blockIdx.y = head x 2 + {K, V}. Bound by the
// reads and writes for a prompt (65536 tokens of 8 heads of 128: 64 us in Q8,
// 96 % of the copy rate, 58 us in Q4, 89 %; 8192 tokens, from L2: 8 us), by
// latency for a decode step (8 tokens: 1.8 us).
template <int FMT, int D, int ALIGN>
__global__ void __launch_bounds__(MOE_KV_THREADS) moe_kv_append_kernel(const KvArgs a)
{
    constexpr int PIECES = D / kv_append_values<D, ALIGN>();
    pdl_wait();
    const int lane = threadIdx.x & 31, head = blockIdx.y >> 1;
    const int token = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kv_append_tokens<D, ALIGN>() +
                      lane / PIECES;
    if (blockIdx.y & 1)
        kv_append_piece<FMT, D, true, ALIGN>(a, token, head, lane % PIECES);
    else
        kv_append_piece<FMT, D, false, ALIGN>(a, token, head, lane % PIECES);
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
// on 32-byte boundaries: the stores are then whole sectors (65536 tokens of 8
// heads of 128 in Q8 as bf16: 68 us, with 16-byte stores 106; as f32 112 and
// 291). Bound by the reads and writes: 68 us is 90 % of the copy rate.
template <int FMT, int D, bool F32, bool WIDE>
__global__ void __launch_bounds__(MOE_KV_THREADS) moe_kv_read_kernel(const KvArgs a)
{
    constexpr int NK = kv_read_threads<FMT, D, false>(), NV = kv_read_threads<FMT, D, true>();
    const int head = blockIdx.y >> 1;
    const int lane = threadIdx.x & 31;
    pdl_wait();
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
