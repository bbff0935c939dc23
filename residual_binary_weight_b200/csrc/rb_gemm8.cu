// rb_gemm8: Y = X W^T from e4m3 codes, with one scale per 128 columns of a
// row of X and per 128 x 128 block of W, on the tcgen05 tensor cores.
//
//   y[t][m] = sum_g sx[t][g] sw[m / 128][g] (sum_{j in block g} cx[t][j] cw[m][j])
//
// The scales change with every 128 columns of K, so the tensor memory only
// holds one block's product at a time: per 128 columns the MMAs write a fresh
// accumulator (two buffers in turn), and the epilogue warps add sx sw times it
// to fp32 sums in their registers. Tokens are the MMA's M (one tensor-memory
// lane = one thread = one token) and weight rows its N, so the factor sx sw
// is one register for 32 columns of a thread: one FMA for a sum and no
// shared-memory reads. An epilogue warp has 32 tokens x 64
// columns: 64 sums a thread leave room for the loads in flight, and the buffer is
// given back as soon as the last of them has arrived, before the FMAs.
//
// Three forms:
//   PAIR   many tokens: two CTAs share a tile of 256 tokens x bn weight rows
//          (cta_group::2). Each loads its 128 tokens and half of the weight
//          rows: 32 KB written to and read from shared memory for the 512
//          cycles of MMAs of a 128-column block, where one CTA alone
//          would move 48 KB each way, more than its 128 bytes a cycle allow.
//          bn is the multiple of 32 that leaves the least work in the last
//          wave of tiles. Outputs leave through shared memory and TMA stores;
//   SPLIT  few tiles: the K blocks of a 128 x 128 tile are divided among the
//          CTAs of a cluster, which add their sums through distributed shared
//          memory in rank order (two CTAs on each SM);
//   ONE    tiles of 128 x 128 in between, two CTAs on each SM.
//
// The scales come through shared memory, too, eight blocks at a time: the TMA
// warp loads a token's eight (one 32-byte sector of its row) while the eight
// before are in use. Read by the epilogue threads themselves, block by
// block, they cost a sector for every 4 bytes and each of the 4 column slices,
// which took four times as long as the MMAs.
//
// Measured (fp32 outputs): 2048 tokens x 14336 x 4096 190 us, 1265 TFLOP/s: 1300
// cycles of each block, whose MMAs take 450. The promotion bounds it, by latency:
// its about 100 instructions a warp and block are 400 issue cycles of 16 warps on
// four schedulers, the rest four loads from tensor memory, each waited for before
// the next, and the buffer's way back to the CTA that issues the MMAs.
//
// Roles: the epilogue warps (16 in a pair's CTA, else 8; warp w reads the
// lanes of quarter w % 4 and the columns from 64 (w / 4) on), one TMA and
// scale warp, one MMA warp.
#include "rb_gemm8.cuh"

#include <algorithm>
#include <type_traits>

namespace rb {
namespace {

using namespace g8;

constexpr int MAX_STAGES = 8;
constexpr int SG = 8;                   // K blocks whose scales are staged together
constexpr int SLOTS = 2;
constexpr uint32_t SLOT_FLOATS = SG * (TM + 4);      // [SG][128 tokens], then [SG][4 weight blocks]
enum : int { ONE = G8_ONE, SPLIT = G8_SPLIT, PAIR = G8_PAIR };

template <int FORM>
struct G8Cfg {
    static constexpr int EPI_WARPS = FORM == PAIR ? 16 : 8;
    static constexpr int TMA_WARP = EPI_WARPS, MMA_WARP = EPI_WARPS + 1;
    static constexpr int THREADS = 32 * (EPI_WARPS + 2);
    static constexpr int BUF = FORM == PAIR ? 256 : 128;        // tensor-memory columns of a buffer
    static constexpr uint32_t B_BYTES = 128 * KB;               // most weight rows of a CTA
    static constexpr int CW = 16;                               // columns per tensor-memory load (registers)
    // a pair's staged outputs: 32 rows of 128 bytes for each epilogue warp
    static constexpr uint32_t OUT_BYTES = FORM == PAIR ? EPI_WARPS * 4096 : 0;
};

// error word of the calls without a workspace: nobody reads it
__device__ uint32_t unrecorded;

// D (+)= A x B, fp8 operands from shared memory (of one CTA, or of a pair)
template <bool PAIRED>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIRED)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// both operands e4m3, K-major, fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ bool normal(float f) {
    return (__float_as_uint(f) & 0x7fffffffu) - 0x00800000u < 0x7f000000u;
}

// Whether a product of two scales may not be a normal fp32 value: from the
// smallest and largest magnitudes (as bits) of either
__device__ __forceinline__ bool products_leave_range(uint32_t x_lo, uint32_t x_hi, uint32_t w_lo, uint32_t w_hi) {
    return min(x_lo, w_lo) < 0x00800000u || max(x_hi, w_hi) >= 0x7f800000u || (x_lo >> 23) + (w_lo >> 23) < 128u ||
           (x_hi >> 23) + (w_hi >> 23) > 380u;
}

// A block's factor f = sx sw where it is not a normal value although both scales
// are finite and not zero, in two steps, f after `first` (else first stays 1):
// where it is too large, the smaller scale comes first (it is at least 1 then, so a
// step that overflows has a result that does), where it is too small, the
// larger one (below 2^23 then).
__device__ __forceinline__ void two_factors(float sx, float sw, float& f, float& first) {
    const float lo = fminf(fabsf(sx), fabsf(sw)), hi = fmaxf(fabsf(sx), fabsf(sw));
    if (normal(f) || !(lo > 0.0f) || !(hi < INFINITY) || sx != sx || sw != sw) return;
    const bool x_first = (fabsf(sx) == lo) == (fabsf(f) > 1.0f);
    first = x_first ? sx : sw;
    f = x_first ? sw : sx;
}

template <int FORM>
__global__ void __launch_bounds__(G8Cfg<FORM>::THREADS, FORM == PAIR ? 1 : 2)
gemm8_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
             const __grid_constant__ CUtensorMap ymap, G8Args a) {
    using C = G8Cfg<FORM>;
    constexpr int EPI_WARPS = C::EPI_WARPS, TMA_WARP = C::TMA_WARP, MMA_WARP = C::MMA_WARP, CW = C::CW;
    extern __shared__ __align__(1024) unsigned char dsm[];
    __shared__ __align__(8) uint64_t bars[2 * MAX_STAGES + 4 + 2 * SLOTS];
    __shared__ float staged[SLOTS][SLOT_FLOATS];
    __shared__ uint32_t staged_apart[SLOTS];
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
    auto sc_full = [&](int n) { return bar0 + 8u * (2 * MAX_STAGES + 4 + n); };
    auto sc_empty = [&](int n) { return bar0 + 8u * (2 * MAX_STAGES + 4 + SLOTS + n); };

    const uint32_t rank = FORM == ONE ? 0u : cluster_rank(), size = FORM == ONE ? 1u : cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* err = a.err ? a.err : &unrecorded;
    if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0u;      // flags are raised only by waits that ran out
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), FORM == PAIR && rank == 0 ? 2 : 1);      // in a pair's even CTA, the other's word, too
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), FORM == PAIR ? 2 * EPI_WARPS : EPI_WARPS);
        }
        for (int n = 0; n < SLOTS; ++n) {
            mbar_init(sc_full(n), 1);
            mbar_init(sc_empty(n), EPI_WARPS);
        }
        abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) {
        if constexpr (FORM == PAIR) tmem_alloc2(smem_addr(&tmem_slot), 2 * C::BUF);
        else tmem_alloc(smem_addr(&tmem_slot), 2 * C::BUF);
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

    const int w_blocks = static_cast<int>((a.M + 127) / 128);
    if (warp == TMA_WARP) {
        // tiles: block by block, `issued` of them so far
        int u = u0, g = g_lo, issued = 0, s = 0;
        uint32_t ph = 1u;
        bool ok = true;
        auto issue_to = [&](int upto) {
            for (; issued < upto && u < units && ok; ++issued) {
                if (!__all_sync(FULL_MASK, mbar_wait(empty_bar(s), ph, abort_flag, err, 1u))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(full_bar(s), a_bytes + b_bytes);
                    tma_load_3d(b_tile(s), &wmap, g * static_cast<int>(KB), row0(u) + (FORM == PAIR ? static_cast<int>(rank) * bnc : 0),
                                0, full_bar(s));
                    tma_load_3d(a_tile(s), &xmap, g * static_cast<int>(KB), token0(u), 0, full_bar(s));
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++g == g_hi) {
                    g = g_lo;
                    u += u_step;
                }
            }
        };
        // scales of one group of up to SG blocks: 4 tokens a lane, and a
        // weight block's value of one K block (4 weight blocks)
        float xr[4][SG], wr = 0.0f;
        const bool vec = (a.G & 3) == 0 && (g_lo & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0;
        auto load = [&](int us, int gs) {
            const int t0 = token0(us), n = min(SG, g_hi - gs);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + lane + 32 * k;
                const float* p = a.xs + static_cast<int64_t>(t) * a.G + gs;
                if (t < a.T && vec && n == SG) {
                    const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
                    xr[k][0] = lo.x, xr[k][1] = lo.y, xr[k][2] = lo.z, xr[k][3] = lo.w;
                    xr[k][4] = hi.x, xr[k][5] = hi.y, xr[k][6] = hi.z, xr[k][7] = hi.w;
                } else {
#pragma unroll
                    for (int i = 0; i < SG; ++i) xr[k][i] = t < a.T && i < n ? __ldg(p + i) : 1.0f;
                }
            }
            const int wb = min((row0(us) >> 7) + (lane & 3), w_blocks - 1);
            wr = (lane >> 2) < n ? __ldg(a.ws + static_cast<int64_t>(wb) * a.G + gs + (lane >> 2)) : 1.0f;
        };
        int done = 0, slot = 0;
        uint32_t sph = 1u;
        if (u0 < units) load(u0, g_lo);
        issue_to(stages);
        for (int us = u0; us < units && ok; us += u_step) {
            for (int gs = g_lo; gs < g_hi && ok; gs += SG) {
                if (!__all_sync(FULL_MASK, mbar_wait(sc_empty(slot), sph, abort_flag, err, 1u))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < SG; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) staged[slot][i * TM + 32 * k + lane] = xr[k][i];
                staged[slot][SG * TM + lane] = wr;
                uint32_t x_lo = 0xffffffffu, x_hi = 0u;
#pragma unroll
                for (int i = 0; i < SG; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t e = __float_as_uint(xr[k][i]) & 0x7fffffffu;
                        x_lo = min(x_lo, e), x_hi = max(x_hi, e);
                    }
                const uint32_t w_e = __float_as_uint(wr) & 0x7fffffffu;
                const bool apart = products_leave_range(__reduce_min_sync(FULL_MASK, x_lo), __reduce_max_sync(FULL_MASK, x_hi),
                                                        __reduce_min_sync(FULL_MASK, w_e), __reduce_max_sync(FULL_MASK, w_e));
                if (lane == 0) staged_apart[slot] = apart;
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full(slot));
                if (++slot == SLOTS) {
                    slot = 0;
                    sph ^= 1u;
                }
                if (gs + SG < g_hi) load(us, gs + SG);
                else if (us + u_step < units) load(us + u_step, g_lo);
                // a block's tiles may be awaited once the scales of all blocks that its
                // slot's last user needs are out
                done += min(SG, g_hi - gs);
                issue_to(done + stages);
            }
        }
        // after an abort the loads in flight land before the CTA gives up its shared memory
        if (*abort_flag) {
            for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
                mbar_drain(full_bar(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        } else if (FORM == PAIR) {
            // the even CTA's commits also arrive here: all of them, before the CTA may go
            for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
                mbar_drain(empty_bar(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        }
    } else if (FORM == PAIR && warp == MMA_WARP && rank == 1) {
        // the pair's MMAs are issued by the even CTA: tell it, stage by stage,
        // that this CTA's half of the operands is there
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
        const uint32_t idesc = idesc_e4m3(FORM == PAIR ? 2 * TM : TM, a.bn);
        const uint64_t ad0 = smem_desc(a_tile(0)), bd0 = smem_desc(b_tile(0));
        int it = 0, s = 0;
        uint32_t ph = 0u;
        bool ok = true;
        for (int u = u0; u < units && ok; u += u_step) {
            for (int g = g_lo; g < g_hi; ++g, ++it) {
                const int b = it & 1;
                if (!__all_sync(FULL_MASK, mbar_wait(full_bar(s), ph, abort_flag, err, 2u) &&
                                               mbar_wait(acc_empty(b), (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag,
                                                         err, 2u))) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint64_t ad = ad0 + static_cast<uint32_t>(s) * (a_bytes >> 4), bd = bd0 + static_cast<uint32_t>(s) * (C::B_BYTES >> 4);
                const uint32_t d = tmem + static_cast<uint32_t>(b * C::BUF);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_f8<FORM == PAIR>(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0);
                    if constexpr (FORM == PAIR) {
                        umma2_commit(acc_full(b));
                        umma2_commit(empty_bar(s));
                    } else {
                        umma_commit(acc_full(b));
                        umma_commit(empty_bar(s));
                    }
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // every MMA issued has completed before the tensor memory is given up
        // (each buffer's last commit; the epilogue may have left early)
        if (!ok)
            for (int i = it - 1; i >= 0 && i >= it - 2; --i) mbar_drain(acc_full(i & 1), static_cast<uint32_t>(i >> 1) & 1u);
    } else {
        const int q = warp & 3, slice = warp >> 2;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(slice * 64);
        int b = 0, slot = 0;
        uint32_t bph = 0u, sph = 0u;
        bool ok = true;
        // the buffer's values are in this warp's registers
        const uint32_t to = FORM == PAIR ? cluster_addr(acc_empty(0), 0) : acc_empty(0);
        auto give_back = [&](int buf) {
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (FORM == PAIR) mbar_arrive_cluster(to + 8u * buf);
                else mbar_arrive(to + 8u * buf);
            }
        };
        for (int u = u0; u < units && ok; u += u_step) {
            const int t = token0(u) + q * 32 + lane;
            const int m0 = row0(u) + slice * 64;              // first column of this thread
            // columns 0-31 and 32-63 of the thread lie in one weight block each (bn is a multiple of 32)
            const int cols = min(64, a.bn - slice * 64);       // 64, 32, or none
            const bool live = token0(u) + q * 32 < a.T && cols > 0;
            const int w0 = (m0 >> 7) - (row0(u) >> 7), w1 = ((m0 + 32) >> 7) - (row0(u) >> 7);
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            for (int gs = g_lo; gs < g_hi; gs += SG) {
                if (!__all_sync(FULL_MASK, mbar_wait(sc_full(slot), sph, abort_flag, err, 8u))) {
                    ok = false;
                    break;
                }
                const float* sx = staged[slot] + q * 32 + lane;
                const float* sw = staged[slot] + SG * TM;
                const int n = min(SG, g_hi - gs);
                float fx = sx[0], fw0 = sw[w0], fw1 = FORM == PAIR ? sw[w1] : fw0;
                // apart: some factor sx sw of these blocks may not be a normal value
                // (the scale warp has looked at all of the tile's; a look at each block's
                // here would cost 4 to 8 %)
                auto blocks = [&](auto apart) {
                    for (int gi = 0; gi < n; ++gi) {
                        if (!__all_sync(FULL_MASK, mbar_wait(acc_full(b), bph, abort_flag, err, 8u))) {
                            ok = false;
                            break;
                        }
                        float f0 = fx * fw0, f1 = FORM == PAIR ? fx * fw1 : f0, first0 = 1.0f, first1 = 1.0f;
                        if constexpr (apart) {
                            two_factors(fx, fw0, f0, first0);
                            if (FORM == PAIR) two_factors(fx, fw1, f1, first1);
                            else f1 = f0, first1 = first0;
                        }
                        if (gi + 1 < n) {       // the next block's, on their way meanwhile
                            fx = sx[(gi + 1) * TM];
                            fw0 = sw[(gi + 1) * 4 + w0];
                            fw1 = FORM == PAIR ? sw[(gi + 1) * 4 + w1] : fw0;
                        }
                        if (live) {
                            fence_after();
                            const uint32_t from = taddr + static_cast<uint32_t>(b * C::BUF);
#pragma unroll
                            for (int c = 0; c < 64 / CW; ++c) {
                                if (c * CW < cols) {
                                    uint32_t v[CW];
                                    tmem_load<CW>(from + static_cast<uint32_t>(c * CW), v);
                                    if ((c + 1) * CW == cols) give_back(b);
#pragma unroll
                                    for (int i = 0; i < CW; ++i) {
                                        const float p = __uint_as_float(v[i]) * (!apart ? 1.0f : c * CW < 32 ? first0 : first1);
                                        acc[c * CW + i] = fmaf(p, c * CW < 32 ? f0 : f1, acc[c * CW + i]);
                                    }
                                }
                            }
                        } else {
                            give_back(b);
                        }
                        b ^= 1;
                        if (b == 0) bph ^= 1u;
                    }
                };
                if (staged_apart[slot]) blocks(std::true_type{});
                else blocks(std::false_type{});
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_empty(slot));
                if (++slot == SLOTS) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
            if (!ok) break;
            auto four = [&](int i) {      // columns 4 i .. 4 i + 3
                return make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            };
            if constexpr (FORM == SPLIT) {
                // this CTA's sums, one row per token (132 floats apart: the
                // lanes of a 16-byte store fall on distinct banks)
                if (t < a.T) {
                    float* row = reinterpret_cast<float*>(dsm + (base - smem_addr(dsm))) + (q * 32 + lane) * 132 + slice * 64;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        reinterpret_cast<float4*>(row)[i] = four(i);
                }
            } else if (FORM == PAIR && a.y_tma) {
                if (live) {
                    // through this warp's 32 x 128 bytes, 128-byte swizzled: 64
                    // columns of a 16-bit type, or twice 32 of fp32
                    const uint32_t out = base + static_cast<uint32_t>(warp) * 4096u;
                    const uint32_t row = out + static_cast<uint32_t>(lane) * 128u, sw = static_cast<uint32_t>(lane & 7);
                    const int t_row = token0(u) + q * 32;
                    const bool f32 = a.y_dt == B8_F32;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (r == 0 || (f32 && cols > 32)) {
                            if (lane == 0) tma_store_wait_read();      // the store before has read the buffer
                            __syncwarp();
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const uint32_t at = row + ((static_cast<uint32_t>(c) ^ sw) << 4);
                                if (f32) {
                                    const float4 v = four(r * 8 + c);
                                    sts128(at, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
                                } else if (r == 0) {
                                    sts128(at, pack_out(acc[8 * c], acc[8 * c + 1], a.y_dt), pack_out(acc[8 * c + 2], acc[8 * c + 3], a.y_dt),
                                           pack_out(acc[8 * c + 4], acc[8 * c + 5], a.y_dt),
                                           pack_out(acc[8 * c + 6], acc[8 * c + 7], a.y_dt));
                                }
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            // half a box where the slice has 32 columns of a 16-bit type
                            if (lane == 0) {
                                if (f32 || cols == 64) tma_store_2d(&ymap, out, m0 + r * 32, t_row);
                            }
                        }
                    }
                    if (!f32 && cols == 32 && t < a.T) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            store4(a, t, m0 + 4 * i, four(i));
                    }
                }
            } else if (t < a.T) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (4 * i < cols)
                        store4(a, t, m0 + 4 * i, four(i));
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
        if constexpr (FORM == PAIR) tmem_dealloc2(tmem, 2 * C::BUF);
        else tmem_dealloc(tmem, 2 * C::BUF);
    }
}

template <int FORM>
cudaError_t launch(const CUtensorMap& xm, const CUtensorMap& wm, const CUtensorMap& ym, const G8Args& a, unsigned grid,
                   unsigned cluster, size_t smem, cudaStream_t s) {
    auto kern = gemm8_kernel<FORM>;
    static SmemLimit limit;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(G8Cfg<FORM>::THREADS);
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

// Y [T][M] in boxes of 128 bytes x 32 rows, 128-byte swizzled
cudaError_t make_y_map(CUtensorMap* map, const G8Args& a) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const int es = a.y_dt == B8_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.M), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldy) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / es), 32u};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType ty = a.y_dt == B8_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : a.y_dt == B8_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (enc(map, ty, 2, a.y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_gemm8(const uint8_t* W, const float* w_scales, const uint8_t* X, const float* x_scales, int64_t M,
                         int64_t K, int T, void* Y, int y_dt, int64_t ldy, uint32_t* err, cudaStream_t s) {
    G8Args a = g8_args(w_scales, x_scales, M, K, T, Y, y_dt, ldy, err);
    const int sms = device_sm_count();
    CUtensorMap xm, wm, ym{};
    // a pair's tiles pay from one 256 x 256 tile per pair of SMs on
    const int64_t pairs = sms / 2, t256 = (T + 255) / 256;
    if (T > TM && t256 * ((M + 255) / 256) >= pairs) {
        // weight rows per tile: the least time over all waves of tiles; a
        // block's MMAs take 2 bn cycles, and the hand-over of a buffer about 400
        int64_t best = 0;
        for (int bn = 256; bn >= 128; bn -= 32) {
            const int64_t waves = (t256 * ((M + bn - 1) / bn) + pairs - 1) / pairs, cost = waves * std::max(2 * bn, 400);
            if (best == 0 || cost < best) {
                best = cost;
                a.bn = bn;
            }
        }
        a.m_tiles = static_cast<int>(t256);
        a.n_tiles = static_cast<int>((M + a.bn - 1) / a.bn);
        a.box = TM;
        a.stages = 4;
        cudaError_t e = make_x8_map(&xm, X, K, T, 1, TM);
        if (e == cudaSuccess) e = make_x8_map(&wm, W, K, M, 1, a.bn / 2);
        if (e == cudaSuccess && a.y_tma) e = make_y_map(&ym, a);
        if (e != cudaSuccess) return e;
        using C = G8Cfg<PAIR>;
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
    a.stages = static_cast<int>(std::min<size_t>(MAX_STAGES, (102 * 1024) / stage));
    int split = 1;
    while (split < 8 && units * (split + 1) <= 2 * sms && split < a.G) ++split;
    const size_t smem = 1024 + std::max<size_t>(a.stages * stage, split > 1 ? static_cast<size_t>(std::min(T, TM)) * 132 * 4 : 0);
    if (split > 1) return launch<SPLIT>(xm, wm, ym, a, static_cast<unsigned>(units * split), split, smem, s);
    return launch<ONE>(xm, wm, ym, a, static_cast<unsigned>(std::min<int64_t>(units, 2 * sms)), 1, smem, s);
}

}  // namespace rb
