// moe_latent.cuh -- the paged cache of latent vectors: rows written (the key's
// turning part rotated on its way) and read back. A row is latent_dim + rope_dim
// bf16 values, moved in pieces of 16 bytes: bound by bytes.
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

// blockIdx.y 0: the latent vectors' pieces; 1: the key parts'
template <bool READ>
__global__ void __launch_bounds__(MOE_LATENT_THREADS) moe_latent_rows_kernel(const __grid_constant__ LatentRows a)
{
    pdl_wait();
    const long long i = (long long)blockIdx.x * MOE_LATENT_THREADS + threadIdx.x;
    const bool key = blockIdx.y != 0;
    const int per = (key ? a.rope : a.latent) / 8;
    const int token = (int)(i / per), piece = (int)(i - (long long)token * per);
    if (token >= a.tokens)
        return;
    uint16_t *row = latent_row(a, token);
    uint16_t *other = key ? a.kr + token * a.kr_stride : a.c + token * a.c_stride;
    const bool wide = key ? a.kr_wide : a.c_wide;
    if (READ) {
        const uint4 v = row ? *reinterpret_cast<const uint4 *>(row + (key ? a.latent : 0) + piece * 8) : make_uint4(0, 0, 0, 0);
        latent_put(other + piece * 8, v, wide);
        return;
    }
    if (!row)
        return;
    uint4 v = latent_get(other + piece * 8, wide);
    if (key && a.positions) {
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
                const float o = bf16_to_f32(other[d < half ? d + half : i2]);
                f[k] = d < half ? f[k] * cs.x - o * cs.y : o * cs.y + f[k] * cs.x;
            }
        }
        v = piece_put<false>(f);
    }
    *reinterpret_cast<uint4 *>(row + (key ? a.latent : 0) + piece * 8) = v;
}

}  // namespace moe
