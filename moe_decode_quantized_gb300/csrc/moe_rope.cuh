// moe_rope.cuh -- rotary positions on part of each head.
//
// A pair (a, b) turns by the angle t = 2 pi p f: a' = m (a cos t - b sin t),
// b' = m (a sin t + b cos t). The table holds f, the part of a turn a position
// adds, times 2^64, so that p f modulo whole turns is the low half of one 64-bit
// product: exact for every position, where a product in f32 would be off by
// radians from position 10^6 on. The turn is rounded to 2^-32, then to f32 (by
// 2^-26 at most, near half a turn), and goes through sincospif. (With whole quarter
// turns taken off before, 2^-28 at most: 65536 rows written and read back 55.7 us
// for 55.1.)
//
// A CTA takes a few tokens: the sines and cosines of its (token, pair)s once into
// shared memory, then every head's rows, in pieces of 16 bytes where alignment
// allows. Bound by bytes: 16384 tokens of 32 heads of 192 values, bf16, 64 of
// them turned: 67.2 us, 90 % of the copy rate; all of them turned 62.9 to 66.4;
// half and half 76, a part of the threads having two pieces to move. Value by
// value (f32, 90 of 96 at odd places, 4099 tokens of 12 heads) 11 us, half of it.
#pragma once
#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {

#define MOE_ROPE_THREADS 256
#define MOE_ROPE_HEADS 64  // heads of a CTA at most
#define MOE_ROPE_SMEM 32768

struct RopeArgs {
    const void *x;
    void *out;
    long long x_tok, x_head, o_tok, o_head;  // strides, elements
    int tokens, heads, heads_cta, tokens_cta;
    int dim, offset, rope;
    const int32_t *positions;
    const unsigned long long *table;
    float magnitude, sign;
    int turned, items;  // pieces (values) of a row that turn, and all that are moved
};

// cosine and sine (times the magnitude) of position p and a table entry
__device__ __forceinline__ float2 rope_turn(int p, unsigned long long f, float magnitude, float sign)
{
    const unsigned long long t = (unsigned long long)(long long)p * f;
    const float half_turns = (float)(int)((t + 0x80000000ull) >> 32) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * magnitude, s * magnitude * sign);
}

__device__ __forceinline__ void rope_apply(float &a, float &b, float2 cs)
{
    const float x = a * cs.x - b * cs.y;
    b = a * cs.y + b * cs.x;
    a = x;
}

__device__ __forceinline__ uint32_t pack_bf2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// a 16-byte piece as numbers, and back
template <bool F32>
__device__ __forceinline__ void piece_get(const uint4 &w, float (&v)[F32 ? 4 : 8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (F32) {
            v[i] = __uint_as_float(u[i]);
        } else {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ uint4 piece_put(const float (&v)[F32 ? 4 : 8])
{
    if (F32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    return make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[F32 ? 0 : 4], v[F32 ? 0 : 5]),
                      pack_bf2(v[F32 ? 0 : 6], v[F32 ? 0 : 7]));
}

template <bool F32, bool WIDE, bool INTER>
__global__ void __launch_bounds__(MOE_ROPE_THREADS) moe_rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int V = WIDE ? (F32 ? 4 : 8) : 1;  // values of a piece
    constexpr int U = WIDE ? 2 : 4;              // pieces in flight (the calls above with 4 and 8: 72.5 us, 14.6)
    extern __shared__ __align__(16) float2 turns[];
    pdl_wait();
    const int t0 = blockIdx.x * a.tokens_cta, nt = min(a.tokens_cta, a.tokens - t0);
    const int h0 = blockIdx.y * a.heads_cta, nh = min(a.heads_cta, a.heads - h0);
    const int half = a.rope / 2;
    // (the P pairs of a piece lie `turned` apart, so that a warp's pieces read side by side: 16384 tokens of 32 heads of 192
    // values, all turned, 62.9 us, with the pairs in order 86.9)
    constexpr int P = !WIDE ? 1 : INTER ? V / 2 : V;
    for (int i = threadIdx.x; i < nt * half; i += MOE_ROPE_THREADS) {
        const int token = i / half, at = i - token * half, k = at / a.turned;
        turns[i] = rope_turn(a.positions[t0 + token], a.table[(at - k * a.turned) * P + k], a.magnitude, a.sign);
    }
    __syncthreads();
    const FastDiv by_items((uint32_t)a.items), by_heads((uint32_t)nh);
    const int n = nt * nh * a.items;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * MOE_ROPE_THREADS) {
        uint4 v[U], w[U];
        float x[U], y[U];
        int item[U], token[U], d[U], d2[U];
        long long to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * MOE_ROPE_THREADS;
            if (i >= n)
                break;
            const uint32_t row = by_items.div(i);
            item[u] = i - row * a.items;
            token[u] = by_heads.div(row);
            const int head = h0 + row - token[u] * nh;
            // dimension of the piece, and of the other of a pair
            const int c = item[u] - a.turned;
            d[u] = c < 0 ? a.offset + item[u] * (INTER && !WIDE ? 2 : V) : c * V < a.offset ? c * V : c * V + a.rope;
            d2[u] = INTER ? d[u] + 1 : d[u] + half;
            const long long from = (t0 + token[u]) * a.x_tok + head * a.x_head;
            to[u] = (t0 + token[u]) * a.o_tok + head * a.o_head;
            if (WIDE) {
                const char *p = static_cast<const char *>(a.x) + from * (F32 ? 4 : 2);
                v[u] = *reinterpret_cast<const uint4 *>(p + d[u] * (F32 ? 4 : 2));
                if (!INTER && c < 0)
                    w[u] = *reinterpret_cast<const uint4 *>(p + d2[u] * (F32 ? 4 : 2));
            } else if (F32) {
                const float *p = static_cast<const float *>(a.x) + from;
                x[u] = p[d[u]];
                y[u] = c < 0 ? p[d2[u]] : 0.0f;
            } else {
                const uint16_t *p = static_cast<const uint16_t *>(a.x) + from;
                x[u] = bf16_to_f32(p[d[u]]);
                y[u] = c < 0 ? bf16_to_f32(p[d2[u]]) : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * MOE_ROPE_THREADS >= n)
                break;
            const bool turns_here = item[u] < a.turned;
            const float2 *cs = turns + token[u] * half + item[u];
            if (WIDE) {
                char *p = static_cast<char *>(a.out) + to[u] * (F32 ? 4 : 2);
                if (turns_here) {
                    float f[F32 ? 4 : 8], g[F32 ? 4 : 8];
                    piece_get<F32>(v[u], f);
                    if (INTER) {
#pragma unroll
                        for (int k = 0; k < V; k += 2)
                            rope_apply(f[k], f[k + 1], cs[k / 2 * a.turned]);
                    } else {
                        piece_get<F32>(w[u], g);
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            rope_apply(f[k], g[k], cs[k * a.turned]);
                        *reinterpret_cast<uint4 *>(p + d2[u] * (F32 ? 4 : 2)) = piece_put<F32>(g);
                    }
                    v[u] = piece_put<F32>(f);
                }
                *reinterpret_cast<uint4 *>(p + d[u] * (F32 ? 4 : 2)) = v[u];
            } else {
                float f = x[u], g = y[u];
                if (turns_here)
                    rope_apply(f, g, *cs);
                if (F32) {
                    float *p = static_cast<float *>(a.out) + to[u];
                    p[d[u]] = f;
                    if (turns_here)
                        p[d2[u]] = g;
                } else {
                    // (a value that only moves keeps its bits, a NaN's too)
                    uint16_t *p = static_cast<uint16_t *>(a.out) + to[u];
                    p[d[u]] = turns_here ? (uint16_t)pack_bf2(f, f) : (uint16_t)(__float_as_uint(f) >> 16);
                    if (turns_here)
                        p[d2[u]] = (uint16_t)pack_bf2(g, g);
                }
            }
        }
    }
}

}  // namespace moe
