// rb_pack8 / rb_unpack8: e4m3 codes with one power-of-two scale per block of
// 1 x 128 values (activations) or 128 x 128 values (weights).
//
// With A the largest finite magnitude of a block, the scale is s = 2^n with
// the smallest n >= -126 for which A <= 448 s (448 is e4m3's largest value;
// n = 0 for a block of zeros), and a code is the e4m3 value nearest to x / s
// (ties to even). A power of two makes x / s and code * s exact, so a code
// carries one rounding (half a step, 2^-4 of the value, or 2^-10 s where x / s
// is below e4m3's normal range), and a 16-bit float holds code * s exactly. It
// costs at most one binade of e4m3's range against s = A / 448, none of its
// precision. In the top binade of x's own type the codes stop at 240: 256 s
// would overflow that type.
// A value that is not finite becomes the NaN code and does not enter A.
//
// Both kernels are bound by HBM: 2 (or 4) bytes in and 1 byte out for each
// value, 1/32 byte of scales, and the reverse. Measured, with a copy's 6539
// GB/s as the peak: pack8 of 11008 x 4096 fp32 in 128 x 128 blocks 35.2 us
// (98 %), of 2048 x 14336 bf16 15.8 us (86 %; 13.6 us are one pass, the rest
// the launch and the last wave); unpack8 of 8192 x 11008 to bf16 44.2 us
// (95 %). One row of 4096: 2.0 us, nearly all of it the launch.
#include "rb_internal.cuh"

#include <cuda_bf16.h>

namespace rb {
namespace {

constexpr int THREADS = 256;
constexpr int UNITS = 4;        // blocks (of 16 lanes) a half warp has in flight

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// 8 consecutive values of one row
template <int DT>
struct Raw8;
template <>
struct Raw8<B8_F16> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p) { v = __ldg(static_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    // largest magnitude as fp32 bits; NaN and infinities come out >= 0x7f800000
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(max(m & 0xffffu, m >> 16)))));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
};
template <>
struct Raw8<B8_BF16> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p) { v = __ldg(static_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<B8_F32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p) {
        a = __ldg(static_cast<const uint4*>(p));
        b = __ldg(static_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t S = 0x7fffffffu;
        return max(max(max(a.x & S, a.y & S), max(a.z & S, a.w & S)), max(max(b.x & S, b.y & S), max(b.z & S, b.w & S)));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
};

template <int DT>
__host__ __device__ constexpr int elt_bytes() { return DT == B8_F32 ? 4 : 2; }

constexpr uint32_t INF_BITS = 0x7f800000u;

// largest finite magnitude of 8 values, as fp32 bits (the rare block that
// holds a value that is not finite)
template <int DT>
__device__ __forceinline__ uint32_t finite_top(const Raw8<DT>& r) {
    float f[8];
    r.get(f);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
        if (u < INF_BITS) m = max(m, u);
    }
    return m;
}

// exponent n of the block's scale from its largest finite magnitude
__device__ __forceinline__ int scale_exp(uint32_t top) {
    const int n = static_cast<int>(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top == 0u ? 0 : max(n, -126);
}

__device__ __forceinline__ float pow2f(int n) { return __int_as_float((n + 127) << 23); }   // -126 <= n <= 127

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// the 8 codes of one lane; n is the block's exponent, odd: the block holds a
// value that is not finite
template <int DT>
__device__ __forceinline__ uint2 encode(const Raw8<DT>& r, int n, bool odd) {
    constexpr int TOP = DT == B8_F16 ? 8 : 120;
    float f[8];
    r.get(f);
    const float inv = pow2f(-n);
    if (odd || n == TOP) {
        const float cap = n == TOP ? 240.0f : 448.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool fin = (__float_as_uint(f[i]) & 0x7fffffffu) < INF_BITS;
            f[i] = fin ? fminf(fmaxf(f[i] * inv, -cap), cap) : __uint_as_float(0x7fffffffu);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
    }
    return make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16), e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
}

// One scale per 128 columns of a row: a half warp per block, UNITS blocks of
// each half warp loaded before the first is used.
// DENSE: rows follow one another without a gap, so a block's place needs no
// division.
template <int DT, bool DENSE>
__global__ void __launch_bounds__(THREADS)
pack8_rows_kernel(const char* X, int64_t ldx, uint32_t blocks, uint32_t G, uint8_t* codes, float* scales) {
    const uint32_t lane = threadIdx.x & 15u;
    const uint32_t b0 = blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4);
    const uint32_t stride = gridDim.x * (THREADS / 16);
    Raw8<DT> r[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const uint32_t b = b0 + u * stride;
        if (b < blocks) {
            int64_t at = static_cast<int64_t>(b) * 128;
            if constexpr (!DENSE) {
                const uint32_t row = b / G;
                at = static_cast<int64_t>(row) * ldx + (b - row * G) * 128u;
            }
            r[u].load(X + (at + lane * 8u) * elt_bytes<DT>());
        } else {
            r[u].zero();
        }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const uint32_t b = b0 + u * stride;
        uint32_t top = r[u].top();
#pragma unroll
        for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(FULL_MASK, top, o));
        const bool odd = top >= INF_BITS;
        if (__any_sync(FULL_MASK, odd)) {
            uint32_t t = finite_top<DT>(r[u]);
#pragma unroll
            for (int o = 8; o; o >>= 1) t = max(t, __shfl_xor_sync(FULL_MASK, t, o));
            top = t;
        }
        const int n = scale_exp(top);
        if (b < blocks) {
            *reinterpret_cast<uint2*>(codes + static_cast<size_t>(b) * 128 + lane * 8) = encode<DT>(r[u], n, odd);
            if (lane == 0) scales[b] = pow2f(n);
        }
    }
}

// One scale per 128 x 128 block: one CTA per block, 8 rows of 8 columns in
// the registers of each thread between the maximum and the codes.
template <int DT>
__global__ void __launch_bounds__(THREADS)
pack8_tile_kernel(const char* X, int64_t ldx, int64_t rows, uint32_t G, uint8_t* codes, float* scales) {
    __shared__ uint32_t part[THREADS / 32];
    const uint32_t rb = blockIdx.x / G, g = blockIdx.x - rb * G;
    const uint32_t lane = threadIdx.x & 15u, r0 = threadIdx.x >> 4;
    const int64_t K = static_cast<int64_t>(G) * 128;
    Raw8<DT> r[8];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = static_cast<int64_t>(rb) * 128 + r0 + 16 * i;
        if (row < rows) r[i].load(X + (row * ldx + g * 128u + lane * 8u) * elt_bytes<DT>());
        else r[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, r[i].top());
    auto block_max = [&](uint32_t v) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(FULL_MASK, v, o));
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0u;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) v = max(v, part[i]);
        __syncthreads();
        return v;
    };
    top = block_max(top);
    const bool odd = top >= INF_BITS;        // the same in every thread
    if (odd) {
        uint32_t t = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, finite_top<DT>(r[i]));
        top = block_max(t);
    }
    const int n = scale_exp(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = static_cast<int64_t>(rb) * 128 + r0 + 16 * i;
        if (row < rows) *reinterpret_cast<uint2*>(codes + row * K + g * 128u + lane * 8u) = encode<DT>(r[i], n, odd);
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = pow2f(n);
}

__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int DT>
__device__ __forceinline__ void store8(char* p, const float (&f)[8]) {
    if constexpr (DT == B8_F32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == B8_F16) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// 8 codes of a thread, UNITS times; rbs = log2 of the rows that share a scale
template <int DT>
__global__ void __launch_bounds__(THREADS)
unpack8_kernel(const uint8_t* codes, const float* scales, uint32_t blocks, uint32_t G, int rbs, char* X, int64_t ldx) {
    const uint32_t lane = threadIdx.x & 15u;
    const uint32_t b0 = blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4);
    const uint32_t stride = gridDim.x * (THREADS / 16);
    uint2 c[UNITS];
    float s[UNITS];
    uint32_t row[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const uint32_t b = b0 + u * stride;
        row[u] = b / G;
        if (b < blocks) {
            c[u] = __ldg(reinterpret_cast<const uint2*>(codes + static_cast<size_t>(b) * 128 + lane * 8));
            s[u] = __ldg(scales + (rbs ? static_cast<size_t>(row[u] >> rbs) * G + (b - row[u] * G) : b));
        }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const uint32_t b = b0 + u * stride;
        if (b < blocks) {
            float f[8];
            const uint32_t w[4] = {c[u].x & 0xffffu, c[u].x >> 16, c[u].y & 0xffffu, c[u].y >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = e4m3x2_f32(w[i]);
                f[2 * i] = t.x * s[u];
                f[2 * i + 1] = t.y * s[u];
            }
            store8<DT>(X + (static_cast<int64_t>(row[u]) * ldx + (b - row[u] * G) * 128u + lane * 8u) * elt_bytes<DT>(), f);
        }
    }
}

unsigned grid_for(uint32_t blocks) {
    const uint32_t per = (THREADS / 16) * UNITS;
    return (blocks + per - 1) / per;
}

}  // namespace

cudaError_t launch_pack8(const void* X, int dt, int64_t ldx, int64_t rows, int64_t K, int block_rows, uint8_t* codes,
                         float* scales, cudaStream_t s) {
    const uint32_t G = static_cast<uint32_t>(K / 128);
    const char* x = static_cast<const char*>(X);
    if (block_rows == 1) {
        const uint32_t blocks = static_cast<uint32_t>(rows) * G;
        const unsigned grid = grid_for(blocks);
        auto go = [&](auto dense_kernel, auto kernel) {
            if (ldx == K) dense_kernel<<<grid, THREADS, 0, s>>>(x, ldx, blocks, G, codes, scales);
            else kernel<<<grid, THREADS, 0, s>>>(x, ldx, blocks, G, codes, scales);
        };
        if (dt == B8_F16) go(pack8_rows_kernel<B8_F16, true>, pack8_rows_kernel<B8_F16, false>);
        else if (dt == B8_BF16) go(pack8_rows_kernel<B8_BF16, true>, pack8_rows_kernel<B8_BF16, false>);
        else go(pack8_rows_kernel<B8_F32, true>, pack8_rows_kernel<B8_F32, false>);
    } else {
        const unsigned grid = static_cast<unsigned>((rows + 127) / 128) * G;
        if (dt == B8_F16) pack8_tile_kernel<B8_F16><<<grid, THREADS, 0, s>>>(x, ldx, rows, G, codes, scales);
        else if (dt == B8_BF16) pack8_tile_kernel<B8_BF16><<<grid, THREADS, 0, s>>>(x, ldx, rows, G, codes, scales);
        else pack8_tile_kernel<B8_F32><<<grid, THREADS, 0, s>>>(x, ldx, rows, G, codes, scales);
    }
    return cudaGetLastError();
}

cudaError_t launch_unpack8(const uint8_t* codes, const float* scales, int64_t rows, int64_t K, int block_rows, void* X,
                           int dt, int64_t ldx, cudaStream_t s) {
    const uint32_t G = static_cast<uint32_t>(K / 128), blocks = static_cast<uint32_t>(rows) * G;
    const int rbs = block_rows == 1 ? 0 : 7;
    char* x = static_cast<char*>(X);
    const unsigned grid = grid_for(blocks);
    if (dt == B8_F16) unpack8_kernel<B8_F16><<<grid, THREADS, 0, s>>>(codes, scales, blocks, G, rbs, x, ldx);
    else if (dt == B8_BF16) unpack8_kernel<B8_BF16><<<grid, THREADS, 0, s>>>(codes, scales, blocks, G, rbs, x, ldx);
    else unpack8_kernel<B8_F32><<<grid, THREADS, 0, s>>>(codes, scales, blocks, G, rbs, x, ldx);
    return cudaGetLastError();
}

}  // namespace rb
