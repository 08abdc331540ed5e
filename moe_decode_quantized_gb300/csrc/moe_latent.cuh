// moe_latent.cuh -- the paged cache of latent vectors: rows written (the key's
// turning part rotated on its way) and read back. A row is latent_dim + rope_dim
// bf16 values, moved in pieces of 16 bytes: bound by bytes, and by the wait for
// a slot before a row can be moved: 65536 rows of 512 + 64 values are written and
// read back in 54.3 us, 45 at the copy rate.
#pragma once
#include "moe_rope.cuh"

namespace moe {

#define MOE_LATENT_THREADS 256

struct LatentRows {
    uint16_t *pages;
    long long n_slots;
    int latent, rope, layout;
    const int32_t *slots;
    int tokens;
    unsigned c_blocks;  // CTAs of the latent vectors
    uint16_t *c, *kr;  // sources of a write, destinations of a read
    long long c_stride, kr_stride;
    int c_wide, kr_wide;  // 16 bytes at a time
    const int32_t *positions;  // NULL: the key part is written as it is
    const unsigned long long *table;
    float magnitude;
    uint32_t *status;
};

// eight values at p
__device__ __forceinline__ uint4 latent_get(const uint16_t *p, bool wide)
{
    if (wide)
        return *reinterpret_cast<const uint4 *>(p);
    return make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                      p[6] | (uint32_t)p[7] << 16);
}

__device__ __forceinline__ void latent_put(uint16_t *p, const uint4 &v, bool wide)
{
    if (wide) {
        *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[2 * i] = (uint16_t)w[i];
        p[2 * i + 1] = (uint16_t)(w[i] >> 16);
    }
}

// bf16 values whose exponent is all ones (NaN, infinities) to 0
__device__ __forceinline__ uint32_t finite_bf2(uint32_t w)
{
    return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}

// the row of the token's slot; nullptr where there is none
__device__ __forceinline__ uint16_t *latent_row(const LatentRows &a, int token)
{
    const int slot = a.slots[token];
    if (slot >= 0 && slot < a.n_slots)
        return a.pages + (long long)slot * (a.latent + a.rope);
    if (slot != -1 && a.status)
        atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
    return nullptr;
}

#define MOE_LATENT_PIECES 2  // of a thread, in flight together (the calls above with 1: 60.9 us, 4: 55.8, 8: 72.4)

// One piece of a key part on its way into the cache: turned
__device__ __forceinline__ uint4 latent_turned(const LatentRows &a, int token, int piece, const uint16_t *row, uint4 v)
{
    const int p = a.positions[token];
    float f[8];
    piece_get<false>(v, f);
    if (a.layout == MOE_ROPE_INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            rope_apply(f[2 * k], f[2 * k + 1], rope_turn(p, a.table[piece * 4 + k], a.magnitude, 1.0f));
    } else {  // the other of each pair, which another thread writes, is read too
        const int half = a.rope / 2;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int d = piece * 8 + k, i2 = d < half ? d : d - half;
            const float2 cs = rope_turn(p, a.table[i2], a.magnitude, 1.0f);
            const float o = bf16_to_f32(row[d < half ? d + half : i2]);
            f[k] = d < half ? f[k] * cs.x - o * cs.y : o * cs.y + f[k] * cs.x;
        }
    }
    return piece_put<false>(f);
}

// the first c_blocks CTAs: the latent vectors' pieces; the others: the key parts'
template <bool READ>
__global__ void __launch_bounds__(MOE_LATENT_THREADS) moe_latent_rows_kernel(const __grid_constant__ LatentRows a)
{
    constexpr int U = MOE_LATENT_PIECES;
    pdl_wait();
    const bool key = blockIdx.x >= a.c_blocks;
    const int shift = key ? 0 : 31 - __clz(a.latent / 8), per = key ? a.rope / 8 : a.latent / 8;  // latent_dim is a power of two
    const bool wide = key ? a.kr_wide : a.c_wide;
    const long long stride = key ? a.kr_stride : a.c_stride;
    const long long first = (long long)(blockIdx.x - (key ? a.c_blocks : 0)) * (U * MOE_LATENT_THREADS) + threadIdx.x;
    uint16_t *rows[U], *others[U];
    uint4 v[U];
    int tokens[U], pieces[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long i = first + u * MOE_LATENT_THREADS;
        tokens[u] = (int)(key ? i / per : i >> shift);
        pieces[u] = (int)(i - (long long)tokens[u] * per);
        rows[u] = nullptr;
        if (i < (long long)a.tokens * per)
            rows[u] = latent_row(a, tokens[u]);
        else
            tokens[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        others[u] = (key ? a.kr : a.c) + max(tokens[u], 0) * stride;
        v[u] = make_uint4(0, 0, 0, 0);
        if (rows[u]) {
            rows[u] += (key ? a.latent : 0) + pieces[u] * 8;
            v[u] = READ ? *reinterpret_cast<const uint4 *>(rows[u]) : latent_get(others[u] + pieces[u] * 8, wide);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (READ) {
            if (tokens[u] >= 0)
                latent_put(others[u] + pieces[u] * 8, v[u], wide);
        } else if (rows[u]) {
            if (key && a.positions)
                v[u] = latent_turned(a, tokens[u], pieces[u], others[u], v[u]);
            *reinterpret_cast<uint4 *>(rows[u]) = v[u];
        }
    }
}

}  // namespace moe
