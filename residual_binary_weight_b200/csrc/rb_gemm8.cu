// rb_gemm8: Y = X W^T from e4m3 codes, with one scale per 128 columns of a
// row of X and per 128 x 128 block of W, on the tcgen05 tensor cores.
//
//   y[t][m] = sum_g sx[t][g] sw[m / 128][g] (sum_{j in block g} cx[t][j] cw[m][j])
//
// The scales change with every 128 columns of K, so the tensor memory only
// holds one block's product at a time: per 128 columns the MMAs write a fresh
// 128-token x BN accumulator (two buffers in turn), and the epilogue warps
// add sx sw times it to fp32 sums in their registers. Tokens are the MMA's M
// (one tensor-memory lane = one thread = one token) and 128-row weight blocks
// its N, so the factor sx sw is one register for all columns of a thread:
// one packed fp32 FMA for two sums and no shared-memory reads.
//
// Roles (320 threads): warps 0-7 epilogue (warp w reads the lanes of quarter
// w % 4 and the column half w / 4), warp 8 TMA loads, warp 9 MMAs.
#include "rb_tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace rb {
namespace {

using namespace tc;

constexpr int THREADS = 320;
constexpr int EPI_WARPS = 8, TMA_WARP = 8, MMA_WARP = 9;
constexpr int TM = 128;                 // tokens per tile
constexpr uint32_t KB = 128;            // bytes of K per stage: one scale block, one swizzle row
constexpr int MAX_STAGES = 8;

struct G8Args {
    uint32_t* err;
    const float* xs;
    const float* ws;
    void* y;
    int64_t M, ldy;
    int T, G;               // tokens, K / 128
    int m_tiles, n_tiles;   // token tiles, weight tiles
    int box;                // rows of the X box
    int stages;
    int y_dt;
    bool y_vec;             // y rows take 16-byte stores
};

// error word of the calls without a workspace: nobody reads it
__device__ uint32_t unrecorded;

__device__ __forceinline__ float4 ld_cluster4(uint32_t local, uint32_t rank) {
    const uint32_t addr = cluster_addr(local, rank);
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// D (+)= A x B, fp8 operands from shared memory, one elected lane of a converged warp
__device__ __forceinline__ void umma_f8_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// both operands e4m3, K-major, fp32 accumulator, M = 128, N = n
__host__ __device__ constexpr uint32_t idesc_e4m3(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(TM >> 4) << 24);
}

__device__ __forceinline__ void fma2(float2& acc, float a, float b, uint64_t ss) {
    uint64_t c, v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(acc.x), "f"(acc.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(v), "l"(ss));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc.x), "=f"(acc.y) : "l"(c));
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

// BN: weight rows per tile (256: two scale blocks, one per column half).
// SPLIT: the K blocks of a tile are divided among the CTAs of a cluster,
// which add their sums through distributed shared memory; one tile per
// cluster. Otherwise every CTA walks the tiles by the grid's size.
template <int BN, bool SPLIT>
__global__ void __launch_bounds__(THREADS, BN == 128 ? 2 : 1)
gemm8_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, G8Args a) {
    constexpr int HALF = BN / 2;                       // columns of one epilogue thread
    constexpr uint32_t B_BYTES = BN * KB;
    extern __shared__ __align__(1024) unsigned char dsm[];
    __shared__ __align__(8) uint64_t bars[2 * MAX_STAGES + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;
    const uint32_t tiles = (smem_addr(dsm) + 1023u) & ~1023u;
    const int stages = a.stages;
    const uint32_t a_bytes = static_cast<uint32_t>(a.box) * KB;
    // the X boxes first: an MMA reads 128 rows of A; those past the box are
    // bytes of the next tiles and only reach accumulator rows of no token
    auto a_tile = [&](int s) { return tiles + static_cast<uint32_t>(s) * a_bytes; };
    auto b_tile = [&](int s) { return tiles + static_cast<uint32_t>(stages) * a_bytes + static_cast<uint32_t>(s) * B_BYTES; };
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + 2 + b); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* err = a.err ? a.err : &unrecorded;
    if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0u;      // flags are raised only by waits that ran out
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), EPI_WARPS);
        }
        abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) tmem_alloc(smem_addr(&tmem_slot), 2 * BN);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    const uint32_t rank = SPLIT ? cluster_rank() : 0u, size = SPLIT ? cluster_size() : 1u;
    const int g_lo = static_cast<int>(static_cast<int64_t>(a.G) * rank / size);
    const int g_hi = static_cast<int>(static_cast<int64_t>(a.G) * (rank + 1) / size);
    const int units = a.m_tiles * a.n_tiles;
    const int u0 = SPLIT ? blockIdx.x / size : blockIdx.x;
    const int u_step = SPLIT ? units : gridDim.x;

    if (warp == TMA_WARP) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int u = u0; u < units && ok; u += u_step) {
                const int mt = u % a.m_tiles, nt = u / a.m_tiles;
                for (int g = g_lo; g < g_hi; ++g, ++it) {
                    const int s = it % stages;
                    if (!mbar_wait(empty_bar(s), (static_cast<uint32_t>(it / stages) & 1u) ^ 1u, abort_flag, err, 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full_bar(s), a_bytes + B_BYTES);
                    tma_load_3d(b_tile(s), &wmap, g * static_cast<int>(KB), nt * BN, 0, full_bar(s));
                    tma_load_3d(a_tile(s), &xmap, g * static_cast<int>(KB), mt * TM, 0, full_bar(s));
                }
            }
            // after an abort the loads in flight land before the CTA gives up its shared memory
            if (*abort_flag)
                for (int i = it - 1; i >= 0 && i >= it - stages; --i)
                    mbar_drain(full_bar(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        }
    } else if (warp == MMA_WARP) {
        constexpr uint32_t idesc = idesc_e4m3(BN);
        int it = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += u_step) {
            for (int g = g_lo; g < g_hi; ++g, ++it) {
                const int s = it % stages, b = it & 1;
                if (!__all_sync(FULL_MASK, mbar_wait(acc_empty(b), (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u,
                                                     abort_flag, err, 2u) &&
                                               mbar_wait(full_bar(s), static_cast<uint32_t>(it / stages) & 1u,
                                                         abort_flag, err, 2u))) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint64_t ad = smem_desc(a_tile(s)), bd = smem_desc(b_tile(s));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f8_elect(tmem + static_cast<uint32_t>(b * BN), ad + 2u * kk, bd + 2u * kk, idesc, kk > 0);
                umma_commit_elect(empty_bar(s));
                umma_commit_elect(acc_full(b));
            }
        }
        // every MMA issued has completed before the tensor memory is given up
        // (each buffer's last commit; the epilogue may have left early)
        if (!ok)
            for (int i = it - 1; i >= 0 && i >= it - 2; --i) mbar_drain(acc_full(i & 1), static_cast<uint32_t>(i >> 1) & 1u);
    } else {
        const int q = warp & 3, h = warp >> 2;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * HALF);
        const int w_blocks = static_cast<int>((a.M + 127) / 128);
        int it = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += u_step) {
            const int mt = u % a.m_tiles, nt = u / a.m_tiles;
            const int t = mt * TM + q * 32 + lane;
            const bool live = mt * TM + q * 32 < a.T;         // some token of this warp's lanes exists
            const float* xs = a.xs + static_cast<int64_t>(min(t, a.T - 1)) * a.G;
            const int wb = min(BN == 256 ? 2 * nt + h : nt, w_blocks - 1);
            const float* ws = a.ws + static_cast<int64_t>(wb) * a.G;
            float2 acc[HALF / 2];
#pragma unroll
            for (int i = 0; i < HALF / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            float f = (live && g_lo < g_hi) ? __ldg(xs + g_lo) * __ldg(ws + g_lo) : 0.0f;
            for (int g = g_lo; g < g_hi; ++g, ++it) {
                const int b = it & 1;
                const float f_now = f;
                if (live && g + 1 < g_hi) f = __ldg(xs + g + 1) * __ldg(ws + g + 1);
                if (!__all_sync(FULL_MASK, mbar_wait(acc_full(b), static_cast<uint32_t>(it >> 1) & 1u, abort_flag, err, 8u))) {
                    ok = false;
                    break;
                }
                if (live) {
                    fence_after();
                    uint64_t ff;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(ff) : "f"(f_now));
#pragma unroll
                    for (int c = 0; c < HALF / 32; ++c) {
                        uint32_t v[32];
                        tmem_load<32>(taddr + static_cast<uint32_t>(b * BN + c * 32), v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            fma2(acc[c * 16 + i], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), ff);
                    }
                    fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty(b));
            }
            if (!ok) break;
            const int64_t m0 = static_cast<int64_t>(nt) * BN + h * HALF;
            if constexpr (SPLIT) {
                // this CTA's sums, one row per token (132 floats apart: the
                // lanes of a 16-byte store fall on distinct banks)
                if (t < a.T) {
                    float* row = reinterpret_cast<float*>(dsm + (tiles - smem_addr(dsm))) + (q * 32 + lane) * (BN + 4) + h * HALF;
#pragma unroll
                    for (int i = 0; i < HALF / 4; ++i)
                        reinterpret_cast<float4*>(row)[i] =
                            make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
                }
            } else if (t < a.T) {
#pragma unroll
                for (int i = 0; i < HALF / 4; ++i)
                    store4(a, t, m0 + 4 * i, make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y));
            }
        }
    }
    __syncwarp();
    fence_before();
    if constexpr (SPLIT) {
        cluster_sync();
        // the cluster's CTAs take the 4-column groups of the tile in turn and
        // add the ranks' sums in rank order
        const int mt = u0 % a.m_tiles, nt = u0 / a.m_tiles;
        const int rows = min(TM, a.T - mt * TM);
        if (*abort_flag == 0u) {
            for (int e = static_cast<int>(rank) * THREADS + threadIdx.x; e < rows * (BN / 4); e += static_cast<int>(size) * THREADS) {
                const int r = e / (BN / 4), c = e % (BN / 4);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t k = 0; k < size; ++k) {
                    const float4 p = ld_cluster4(tiles + static_cast<uint32_t>((r * (BN + 4) + 4 * c) * 4), k);
                    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
                }
                store4(a, mt * TM + r, static_cast<int64_t>(nt) * BN + 4 * c, v);
            }
        }
        cluster_sync();      // no CTA leaves while another reads its sums
    } else {
        __syncthreads();
    }
    fence_after();
    if (warp == MMA_WARP) tmem_dealloc(tmem, 2 * BN);
}

template <int BN, bool SPLIT>
cudaError_t launch(const CUtensorMap& xm, const CUtensorMap& wm, const G8Args& a, unsigned grid, unsigned cluster,
                   size_t smem, cudaStream_t s) {
    auto kern = gemm8_kernel<BN, SPLIT>;
    static SmemMark mark;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, mark);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, xm, wm, a);
}

}  // namespace

cudaError_t launch_gemm8(const uint8_t* W, const float* w_scales, const uint8_t* X, const float* x_scales, int64_t M,
                         int64_t K, int T, void* Y, int y_dt, int64_t ldy, uint32_t* err, cudaStream_t s) {
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
    a.m_tiles = (T + TM - 1) / TM;
    const int sms = device_sm_count();
    const int64_t tiles256 = static_cast<int64_t>(a.m_tiles) * ((M + 255) / 256);
    const bool wide = tiles256 >= sms;
    const int bn = wide ? 256 : 128;
    a.n_tiles = static_cast<int>((M + bn - 1) / bn);
    const int64_t units = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    a.box = T >= TM ? TM : (T + 7) / 8 * 8;
    CUtensorMap xm, wm;
    cudaError_t e = make_x8_map(&xm, X, K, T, 1, a.box);
    if (e == cudaSuccess) e = make_x8_map(&wm, W, K, M, 1, bn);
    if (e != cudaSuccess) return e;
    const size_t stage = (static_cast<size_t>(a.box) + bn) * KB;
    if (wide) {
        a.stages = 4;
        // every MMA of the last stage reads 128 rows of A
        return launch<256, false>(xm, wm, a, static_cast<unsigned>(std::min<int64_t>(units, sms)), 1,
                                  1024 + a.stages * stage, s);
    }
    // two CTAs share an SM: what fits in half of its shared memory
    a.stages = static_cast<int>(std::min<size_t>(MAX_STAGES, (108 * 1024) / stage));
    int split = 1;
    while (split < 8 && units * (split + 1) <= 2 * sms && split < a.G) ++split;
    const size_t smem = 1024 + std::max<size_t>(a.stages * stage, split > 1 ? static_cast<size_t>(std::min(T, TM)) * 132 * 4 : 0);
    if (split > 1) return launch<128, true>(xm, wm, a, static_cast<unsigned>(units * split), split, smem, s);
    return launch<128, false>(xm, wm, a, static_cast<unsigned>(std::min<int64_t>(units, 2 * sms)), 1, smem, s);
}

}  // namespace rb
