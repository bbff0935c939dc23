// What the two 8-bit product kernels share (rb_gemm8.cu, rb_gemm8_mx.cu).
#pragma once

#include "rb_tc.cuh"

#include <cuda_bf16.h>

namespace rb {
namespace g8 {

using namespace tc;

constexpr int TM = 128;                 // tokens per CTA
constexpr uint32_t KB = 128;            // bytes of K per stage: one scale block, one swizzle row
enum : int { G8_ONE = 0, G8_SPLIT = 1, G8_PAIR = 2 };       // forms, see the kernels

struct G8Args {
    uint32_t* err;
    const float* xs;
    const float* ws;
    void* y;
    int64_t M, ldy;
    int T, G;               // tokens, K / 128
    int m_tiles, n_tiles;   // token tiles, weight tiles
    int bn;                 // weight rows per tile (PAIR: of both CTAs)
    int box;                // rows of the X box
    int stages;
    int y_dt;
    bool y_vec;             // y takes stores of 4 values at a time
    bool y_tma;             // y takes TMA stores (PAIR)
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t local, uint32_t rank) {
    const uint32_t addr = cluster_addr(local, rank);
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// 4 consecutive outputs of token t from column m on
__device__ __forceinline__ void store4(const G8Args& a, int64_t t, int64_t m, float4 v) {
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (a.y_vec && m + 4 <= a.M) {
        if (a.y_dt == B8_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + t * a.ldy + m) = v;
        } else if (a.y_dt == B8_F16) {
            const __half2 h[2] = {__floats2half2_rn(f[0], f[1]), __floats2half2_rn(f[2], f[3])};
            *reinterpret_cast<uint2*>(static_cast<__half*>(a.y) + t * a.ldy + m) = *reinterpret_cast<const uint2*>(h);
        } else {
            const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(f[0], f[1]), __floats2bfloat162_rn(f[2], f[3])};
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + t * a.ldy + m) = *reinterpret_cast<const uint2*>(h);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (m + i < a.M) {
            if (a.y_dt == B8_F32) static_cast<float*>(a.y)[t * a.ldy + m + i] = f[i];
            else if (a.y_dt == B8_F16) static_cast<__half*>(a.y)[t * a.ldy + m + i] = __float2half_rn(f[i]);
            else static_cast<__nv_bfloat16*>(a.y)[t * a.ldy + m + i] = __float2bfloat16_rn(f[i]);
        }
    }
}

// two outputs as 32 bits of a 16-bit type
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int dt) {
    if (dt == B8_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One lane: 32 rows of 128 staged bytes to Y (what lies past its rows or columns is not written).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

inline G8Args g8_args(const float* w_scales, const float* x_scales, int64_t M, int64_t K, int T, void* Y, int y_dt,
                      int64_t ldy, uint32_t* err) {
    G8Args a{};
    a.err = err;
    a.xs = x_scales;
    a.ws = w_scales;
    a.y = Y;
    a.M = M;
    a.ldy = ldy;
    a.T = T;
    a.G = static_cast<int>(K / 128);
    a.y_dt = y_dt;
    const int es = y_dt == B8_F32 ? 4 : 2;
    a.y_vec = reinterpret_cast<uintptr_t>(Y) % (4 * es) == 0 && ldy % 4 == 0;
    // a TMA store clips a box to the map's rows in pieces of 16 bytes: where M ends inside
    // a piece it would write the values after it, too
    a.y_tma = reinterpret_cast<uintptr_t>(Y) % 16 == 0 && (ldy * es) % 16 == 0 && (M * es) % 16 == 0;
    return a;
}

}  // namespace g8
}  // namespace rb
