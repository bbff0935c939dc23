// rb_gemm8 where every scale is a power of two, as rb_pack8 writes them, and
// outputs have 16 bits: the tensor cores apply the scales.
//
//   y[t][m] = sum_g 2^(ex[t][g] + ew[m / 128][g]) (sum_{j in block g} cx[t][j] cw[m][j])
//
// A block-scaled MMA (kind::mxf8f6f4) multiplies each 32 values of a row of A
// and of B by an 8-bit exponent of that row, kept in tensor memory, so sums
// run through all of K in the fp32 accumulator and the epilogue only sees the
// finished tile. (The kernel of rb_gemm8.cu adds every 128 columns' product to
// sums in registers, 1300 cycles of each block where the MMAs take 450.) The
// accumulator cuts low bits off towards zero at every MMA, about 5e-10 of the
// terms' magnitudes a column (7e-5 after 131072 columns of one sign), so fp32
// outputs stay with that kernel; 16-bit outputs round far more away at any K in use.
//
// An exponent byte e stands for 2^(e - 127): the exponent field of the fp32
// scale. Row r's byte lies in tensor-memory lane r % 32 (of each quarter),
// column r / 32; a 128-column block needs it four times, in the four bytes of
// the 32-bit column. Four warps, one for each lane quarter, write the columns
// of a block (4 of A, one per 32 rows of B) with tcgen05.st as the block's
// tiles arrive by TMA. A scale that is no power of two gets the byte 255
// (NaN): every output that it enters is NaN, and the error word says why.
//
// Measured: 2048 tokens x 14336 x 4096 to bf16 112 us, 2150 TFLOP/s (96 us in
// short bursts; under load the power cap holds the SMs near 1.3 GHz; the kernel
// with sums in registers takes 190 us); 16 tokens x 28672 x 8192 45.1 us, 5.2 TB/s of
// the weight's bytes (80 % of a copy's rate: the first and last loads of one wave
// of tiles are not overlapped); one token x 4096 x 4096 8.3 us, of which HBM takes
// 2.6 (launch, fill of the rings, sum over the cluster).
//
// Forms as in rb_gemm8.cu: PAIR (two accumulators of up to 224 columns, TMA
// stores), SPLIT and ONE (128 x 128 tiles, two CTAs on each SM). Roles: the epilogue
// warps (8 in a pair's CTA, else 4), 4 scale warps, one TMA and one MMA warp.
#include "rb_gemm8.cuh"

#include <algorithm>

namespace rb {
namespace {

using namespace g8;

constexpr int MAX_STAGES = 8;
constexpr int SG = 8;                   // K blocks whose scales are read together
enum : int { ONE = G8_ONE, SPLIT = G8_SPLIT, PAIR = G8_PAIR };

template <int FORM>
struct MxCfg {
    static constexpr int EPI_WARPS = FORM == PAIR ? 8 : 4;
    static constexpr int SF_WARP0 = EPI_WARPS, TMA_WARP = EPI_WARPS + 4, MMA_WARP = EPI_WARPS + 5;
    static constexpr int THREADS = 32 * (EPI_WARPS + 6);
    static constexpr int BN = FORM == PAIR ? 224 : 128;         // most weight rows of a tile
    static constexpr int BUFS = FORM == PAIR ? 2 : 1;
    static constexpr int SFB = FORM == PAIR ? 8 : 4;            // columns of B's exponents
    static constexpr int SF0 = BUFS * BN, SF_COLS = 4 + SFB;    // a stage's exponents: 4 columns of A's, then B's
    static constexpr uint32_t TMEM_COLS = FORM == PAIR ? 512 : 256;
    static constexpr int STAGES = FORM == PAIR ? 5 : 8;         // at most
    static constexpr uint32_t B_BYTES = (FORM == PAIR ? BN / 2 : BN) * KB;
    // a pair's staged outputs: 2 x 32 rows of 64 bytes for each epilogue warp
    static constexpr uint32_t OUT_BYTES = FORM == PAIR ? EPI_WARPS * 4096 : 0;
    static_assert(SF0 + STAGES * SF_COLS <= static_cast<int>(TMEM_COLS), "exponents exceed tensor memory");
    static_assert(B_BYTES % 1024 == 0, "B tile must keep the 1024-byte swizzle alignment");
};

constexpr uint32_t BAD_SCALE = 16u;

// error word of the calls without a workspace: nobody reads it
__device__ uint32_t unrecorded;

// D (+)= A x B with the exponents of A's and B's rows, fp8 operands from shared memory
template <bool PAIRED>
__device__ __forceinline__ void umma_mx(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                                        uint32_t sfa, uint32_t sfb) {
    if constexpr (PAIRED)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
}

// both operands e4m3, K-major, byte 0 of the exponent columns, 8-bit exponents without mantissa
__host__ __device__ constexpr uint32_t idesc_mx(int m, int n) {
    return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_store4(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// the exponent byte of a scale, four times
__device__ __forceinline__ uint32_t exponent4(float s, bool& bad) {
    const uint32_t b = __float_as_uint(s);
    const bool ok = (b & 0x807fffffu) == 0u && b != 0u && b != 0x7f800000u;
    bad |= !ok;
    return (ok ? b >> 23 : 255u) * 0x01010101u;
}

template <int FORM>
__global__ void __launch_bounds__(MxCfg<FORM>::THREADS, FORM == PAIR ? 1 : 2)
gemm8_mx_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap ymap, G8Args a) {
    using C = MxCfg<FORM>;
    constexpr int EPI_WARPS = C::EPI_WARPS, SF_WARP0 = C::SF_WARP0, TMA_WARP = C::TMA_WARP, MMA_WARP = C::MMA_WARP, SFB = C::SFB;
    extern __shared__ __align__(1024) unsigned char dsm[];
    __shared__ __align__(8) uint64_t bars[2 * MAX_STAGES + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;
    const uint32_t base = (smem_addr(dsm) + 1023u) & ~1023u;
    const uint32_t tiles = base + C::OUT_BYTES;
    const int stages = a.stages;
    const int bnc = FORM == PAIR ? a.bn / 2 : 128;        // weight rows in this CTA
    const uint32_t a_bytes = static_cast<uint32_t>(a.box) * KB, b_bytes = static_cast<uint32_t>(bnc) * KB;
    // the X boxes first: an MMA reads 128 rows of A; those past the box are
    // bytes of the next tiles and only reach accumulator rows of no token
    auto a_tile = [&](int s) { return tiles + static_cast<uint32_t>(s) * a_bytes; };
    auto b_tile = [&](int s) { return tiles + static_cast<uint32_t>(stages) * a_bytes + static_cast<uint32_t>(s) * C::B_BYTES; };
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + 2 + b); };

    const uint32_t rank = FORM == ONE ? 0u : cluster_rank(), size = FORM == ONE ? 1u : cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* err = a.err ? a.err : &unrecorded;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            // the tiles' bytes, four scale warps, and in a pair's even CTA the other's word
            mbar_init(full_bar(s), FORM == PAIR && rank == 0 ? 6 : 5);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), FORM == PAIR ? 2 * EPI_WARPS : EPI_WARPS);
        }
        abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) {
        if constexpr (FORM == PAIR) tmem_alloc2(smem_addr(&tmem_slot), C::TMEM_COLS);
        else tmem_alloc(smem_addr(&tmem_slot), C::TMEM_COLS);
    }
    fence_before();
    if constexpr (FORM == PAIR) cluster_sync();      // the peer's barriers are ready, too
    else __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    const int g_lo = FORM == SPLIT ? static_cast<int>(static_cast<int64_t>(a.G) * rank / size) : 0;
    const int g_hi = FORM == SPLIT ? static_cast<int>(static_cast<int64_t>(a.G) * (rank + 1) / size) : a.G;
    const int units = a.m_tiles * a.n_tiles;
    const int u0 = static_cast<int>(blockIdx.x / size);
    const int u_step = FORM == SPLIT ? units : static_cast<int>(gridDim.x / size);
    // first token of this CTA and first weight row of the tile
    auto token0 = [&](int u) { return (u % a.m_tiles) * (FORM == PAIR ? 2 * TM : TM) + (FORM == PAIR ? static_cast<int>(rank) * TM : 0); };
    auto row0 = [&](int u) { return (u / a.m_tiles) * a.bn; };

    if (warp == TMA_WARP) {
        if (lane == 0) {
            int it = 0, s = 0;
            uint32_t ph = 1u;
            bool ok = true;
            for (int u = u0; u < units && ok; u += u_step) {
                const int t0 = token0(u), m0 = row0(u) + (FORM == PAIR ? static_cast<int>(rank) * bnc : 0);
                for (int g = g_lo; g < g_hi; ++g, ++it) {
                    if (!mbar_wait(empty_bar(s), ph, abort_flag, err, 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full_bar(s), a_bytes + b_bytes);
                    tma_load_3d(b_tile(s), &wmap, g * static_cast<int>(KB), m0, 0, full_bar(s));
                    tma_load_3d(a_tile(s), &xmap, g * static_cast<int>(KB), t0, 0, full_bar(s));
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // after an abort the loads in flight land before the CTA gives up its shared
            // memory (the scale warps may have left: a barrier's phase may stay open)
            if (*abort_flag)
                for (int i = it - 1; i >= 0 && i >= it - stages; --i)
                    mbar_drain(full_bar(i % stages), static_cast<uint32_t>(i / stages) & 1u);
            // the even CTA's commits also arrive here: all of them, before the CTA may go
            else if (FORM == PAIR)
                for (int i = it - 1; i >= 0 && i >= it - stages; --i)
                    mbar_drain(empty_bar(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        }
    } else if (FORM == PAIR && warp == MMA_WARP && rank == 1) {
        // the pair's MMAs are issued by the even CTA: tell it, stage by stage,
        // that this CTA's half of the operands and its exponents are there
        int s = 0;
        uint32_t ph = 0u;
        bool ok = true;
        for (int u = u0; u < units && ok; u += u_step) {
            for (int g = g_lo; g < g_hi; ++g) {
                if (!__all_sync(FULL_MASK, mbar_wait(full_bar(s), ph, abort_flag, err, 2u))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_remote(full_bar(s), 0);
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == MMA_WARP) {
        const uint32_t idesc = idesc_mx(FORM == PAIR ? 2 * TM : TM, a.bn);
        const uint64_t ad0 = smem_desc(a_tile(0)), bd0 = smem_desc(b_tile(0));
        int s = 0, tile = 0;
        uint32_t ph = 0u;
        bool ok = true, ready = false;
        auto commit = [](uint32_t bar) {
            if constexpr (FORM == PAIR) umma2_commit(bar);
            else umma_commit(bar);
        };
        for (int u = u0; u < units && ok; u += u_step, ++tile) {
            const int b = C::BUFS == 2 ? tile & 1 : 0;
            const uint32_t aph = (static_cast<uint32_t>(tile / C::BUFS) & 1u) ^ 1u;
            const uint32_t d = tmem + static_cast<uint32_t>(b * C::BN);
            ok = __all_sync(FULL_MASK, mbar_wait(acc_empty(b), aph, abort_flag, err, 2u));
            for (int g = g_lo; g < g_hi && ok; ++g) {
                if (!__all_sync(FULL_MASK, ready || mbar_wait(full_bar(s), ph, abort_flag, err, 2u))) {
                    ok = false;
                    break;
                }
                const int now = s;
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
                // the next stage's barrier is looked at while this one's MMAs are issued
                ready = mbar_test(full_bar(s), ph);
                fence_after();
                const uint64_t ad = ad0 + static_cast<uint32_t>(now) * (a_bytes >> 4);
                const uint64_t bd = bd0 + static_cast<uint32_t>(now) * (C::B_BYTES >> 4);
                const uint32_t sf = tmem + static_cast<uint32_t>(C::SF0 + now * C::SF_COLS);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_mx<FORM == PAIR>(d, ad + 2u * kk, bd + 2u * kk, idesc, (g > g_lo || kk > 0) ? 1u : 0u, sf, sf + 4u);
                    commit(empty_bar(now));
                    if (g + 1 == g_hi) commit(acc_full(b));
                }
                __syncwarp();
            }
            // after an abort the teardown waits for it
            if (!ok && elect_one()) commit(acc_full(b));
            __syncwarp();
        }
        // every MMA issued has completed before the tensor memory is given up
        if (!ok)
            for (int i = tile - 1; i >= 0 && i >= tile - C::BUFS; --i)
                mbar_drain(acc_full(C::BUFS == 2 ? i & 1 : 0), static_cast<uint32_t>(i / C::BUFS) & 1u);
    } else if (warp >= SF_WARP0) {
        // exponents: row 32 i + lane of A, rows 32 i .. 32 i + 31 of B (in one
        // weight block: bn is a multiple of 32), for each lane quarter alike
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int w_blocks = static_cast<int>((a.M + 127) / 128);
        const bool vec = (a.G & 3) == 0 && (g_lo & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0;
        int s = 0;
        uint32_t ph = 1u;
        bool ok = true, bad = false;
        for (int u = u0; u < units && ok; u += u_step) {
            const int t0 = token0(u), blk0 = row0(u) >> 7;
            for (int gs = g_lo; gs < g_hi && ok; gs += SG) {
                const int n = min(SG, g_hi - gs);
                float x[4][SG];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = t0 + 32 * i + lane;
                    const float* p = a.xs + static_cast<int64_t>(t) * a.G + gs;
                    if (t < a.T && vec && n == SG) {
                        const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
                        x[i][0] = lo.x, x[i][1] = lo.y, x[i][2] = lo.z, x[i][3] = lo.w;
                        x[i][4] = hi.x, x[i][5] = hi.y, x[i][6] = hi.z, x[i][7] = hi.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < SG; ++k) x[i][k] = t < a.T && k < n ? __ldg(p + k) : 1.0f;
                    }
                }
                // lane 4 k + j: weight block blk0 + j at K block gs + k
                const float w = (lane >> 2) < n ? __ldg(a.ws + static_cast<int64_t>(min(blk0 + (lane & 3), w_blocks - 1)) * a.G + gs + (lane >> 2)) : 1.0f;
                const uint32_t we = exponent4(w, bad);
#pragma unroll
                for (int k = 0; k < SG; ++k) {
                    if (k < n && ok) {
                        uint32_t va[4], vb[SFB];
#pragma unroll
                        for (int i = 0; i < 4; ++i) va[i] = exponent4(x[i][k], bad);
#pragma unroll
                        for (int i = 0; i < SFB; ++i) vb[i] = __shfl_sync(FULL_MASK, we, 4 * k + (((row0(u) + 32 * i) >> 7) - blk0 & 3));
                        if (!__all_sync(FULL_MASK, mbar_wait(empty_bar(s), ph, abort_flag, err, 4u))) {
                            ok = false;
                        } else {
                            fence_after();
                            const uint32_t sf = tmem + quarter + static_cast<uint32_t>(C::SF0 + s * C::SF_COLS);
                            tmem_store4(sf, va);
                            if constexpr (SFB == 8) tmem_store8(sf + 4u, vb);
                            else tmem_store4(sf + 4u, vb);
                            tmem_store_wait();
                            fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(full_bar(s));
                            if (++s == stages) {
                                s = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                }
            }
        }
        if (bad) atomicOr(err, BAD_SCALE);
    } else {
        const int q = warp & 3, half = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int tile = 0, turn = 0;
        for (int u = u0; u < units; u += u_step, ++tile) {
            const int b = C::BUFS == 2 ? tile & 1 : 0;
            if (!__all_sync(FULL_MASK, mbar_wait(acc_full(b), static_cast<uint32_t>(tile / C::BUFS) & 1u, abort_flag, err, 8u)) ||
                *abort_flag)
                break;
            fence_after();
            const int t = token0(u) + q * 32 + lane;
            const bool live = token0(u) + q * 32 < a.T;
            if (live) {
#pragma unroll 1
                for (int c0 = half * 32; c0 < a.bn; c0 += 32 * (EPI_WARPS / 4)) {
                    uint32_t v[32];
                    tmem_load<32>(tmem + lanes + static_cast<uint32_t>(b * C::BN + c0), v);
                    auto four = [&](int i) {
                        return make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                                           __uint_as_float(v[4 * i + 3]));
                    };
                    if constexpr (FORM == SPLIT) {
                        // this CTA's sums, one row per token (132 floats apart: the
                        // lanes of a 16-byte store fall on distinct banks)
                        if (t < a.T) {
                            float* row = reinterpret_cast<float*>(dsm + (base - smem_addr(dsm))) + (q * 32 + lane) * 132 + c0;
#pragma unroll
                            for (int i = 0; i < 8; ++i) reinterpret_cast<float4*>(row)[i] = four(i);
                        }
                    } else if (FORM == PAIR && a.y_tma) {
                        // through one of this warp's two pieces of 32 rows x 64 bytes, 64-byte swizzled
                        const uint32_t out = base + static_cast<uint32_t>(warp) * 4096u + static_cast<uint32_t>(turn & 1) * 2048u;
                        const uint32_t sw = static_cast<uint32_t>(lane >> 1) & 3u;
                        ++turn;
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");      // the store before last has read it
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t h[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                h[i] = pack_out(__uint_as_float(v[8 * c + 2 * i]), __uint_as_float(v[8 * c + 2 * i + 1]), a.y_dt);
                            sts128(out + static_cast<uint32_t>(lane) * 64u + ((static_cast<uint32_t>(c) ^ sw) << 4), h[0], h[1], h[2], h[3]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&ymap, out, row0(u) + c0, token0(u) + q * 32);
                    } else if (t < a.T) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) store4(a, t, static_cast<int64_t>(row0(u)) + c0 + 4 * i, four(i));
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (FORM == PAIR) mbar_arrive_remote(acc_empty(b), 0);
                else mbar_arrive(acc_empty(b));
            }
        }
        // the staged outputs have been read before the CTA gives up its shared memory
        if (FORM == PAIR && lane == 0) tma_store_wait_read();
    }
    __syncwarp();
    fence_before();
    if constexpr (FORM == SPLIT) {
        cluster_sync();
        // the cluster's CTAs take the 4-column groups of the tile in turn and
        // add the ranks' sums in rank order
        const int t0 = token0(u0), rows = min(TM, a.T - t0);
        if (*abort_flag == 0u) {
            for (int e = static_cast<int>(rank) * C::THREADS + threadIdx.x; e < rows * 32; e += static_cast<int>(size) * C::THREADS) {
                const int r = e / 32, c = e % 32;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t k = 0; k < size; ++k) {
                    const float4 p = ld_cluster4(base + static_cast<uint32_t>((r * 132 + 4 * c) * 4), k);
                    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
                }
                store4(a, t0 + r, static_cast<int64_t>(row0(u0)) + 4 * c, v);
            }
        }
        cluster_sync();      // no CTA leaves while another reads its sums
    } else if constexpr (FORM == PAIR) {
        cluster_sync();      // no CTA leaves while the pair's MMAs or arrivals may reach it
    } else {
        __syncthreads();
    }
    fence_after();
    if (warp == MMA_WARP) {
        if constexpr (FORM == PAIR) tmem_dealloc2(tmem, C::TMEM_COLS);
        else tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int FORM>
cudaError_t launch(const CUtensorMap& xm, const CUtensorMap& wm, const CUtensorMap& ym, const G8Args& a, unsigned grid,
                   unsigned cluster, size_t smem, cudaStream_t s) {
    auto kern = gemm8_mx_kernel<FORM>;
    static SmemLimit limit;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(MxCfg<FORM>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = FORM == ONE ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, xm, wm, ym, a);
}

// Y [T][M] of a 16-bit type in boxes of 32 columns x 32 rows, 64-byte swizzled
cudaError_t make_y_map(CUtensorMap* map, const G8Args& a) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.M), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldy) * 2};
    const cuuint32_t box[2] = {32u, 32u};
    const cuuint32_t estr[2] = {1, 1};
    if (enc(map, a.y_dt == B8_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_gemm8_mx(const uint8_t* W, const float* w_scales, const uint8_t* X, const float* x_scales, int64_t M,
                            int64_t K, int T, void* Y, int y_dt, int64_t ldy, uint32_t* err, cudaStream_t s) {
    G8Args a = g8_args(w_scales, x_scales, M, K, T, Y, y_dt, ldy, err);
    const int sms = device_sm_count();
    // the scale warps flag bad scales while the kernel runs, so the error word
    // is cleared before it and not by one of its blocks
    if (err) {
        const cudaError_t e = cudaMemsetAsync(err, 0, sizeof(uint32_t), s);
        if (e != cudaSuccess) return e;
    }
    CUtensorMap xm, wm, ym{};
    // a pair's tiles pay from one 256 x 224 tile per pair of SMs on
    const int64_t pairs = sms / 2, t256 = (T + 255) / 256;
    if (T > TM && t256 * ((M + 223) / 224) >= pairs) {
        // weight rows per tile: the least time over all waves of tiles; a
        // block's MMAs take 2 bn cycles, and issuing them about 300
        int64_t best = 0;
        for (int bn = 224; bn >= 128; bn -= 32) {
            const int64_t waves = (t256 * ((M + bn - 1) / bn) + pairs - 1) / pairs, cost = waves * std::max(2 * bn, 300);
            if (best == 0 || cost < best) {
                best = cost;
                a.bn = bn;
            }
        }
        a.m_tiles = static_cast<int>(t256);
        a.n_tiles = static_cast<int>((M + a.bn - 1) / a.bn);
        a.box = TM;
        a.stages = MxCfg<PAIR>::STAGES;
        cudaError_t e = make_x8_map(&xm, X, K, T, 1, TM);
        if (e == cudaSuccess) e = make_x8_map(&wm, W, K, M, 1, a.bn / 2);
        if (e == cudaSuccess && a.y_tma) e = make_y_map(&ym, a);
        if (e != cudaSuccess) return e;
        using C = MxCfg<PAIR>;
        const size_t smem = 1024 + C::OUT_BYTES + static_cast<size_t>(a.stages) * (TM * KB + C::B_BYTES);
        return launch<PAIR>(xm, wm, ym, a, static_cast<unsigned>(2 * std::min<int64_t>(pairs, t256 * a.n_tiles)), 2, smem, s);
    }
    a.bn = 128;
    a.m_tiles = (T + TM - 1) / TM;
    a.n_tiles = static_cast<int>((M + 127) / 128);
    a.box = T >= TM ? TM : (T + 7) / 8 * 8;
    cudaError_t e = make_x8_map(&xm, X, K, T, 1, a.box);
    if (e == cudaSuccess) e = make_x8_map(&wm, W, K, M, 1, 128);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    // two CTAs share an SM: what fits in half of its shared memory
    const size_t stage = static_cast<size_t>(a.box) * KB + 128 * KB;
    a.stages = static_cast<int>(std::min<size_t>(MxCfg<ONE>::STAGES, (110 * 1024) / stage));
    int split = 1;
    while (split < 8 && units * (split + 1) <= 2 * sms && split < a.G) ++split;
    const size_t smem = 1024 + std::max<size_t>(a.stages * stage, split > 1 ? static_cast<size_t>(std::min(T, TM)) * 132 * 4 : 0);
    if (split > 1) return launch<SPLIT>(xm, wm, ym, a, static_cast<unsigned>(units * split), split, smem, s);
    return launch<ONE>(xm, wm, ym, a, static_cast<unsigned>(std::min<int64_t>(units, 2 * sms)), 1, smem, s);
}

}  // namespace rb
