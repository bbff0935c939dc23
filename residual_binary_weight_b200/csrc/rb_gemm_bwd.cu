// Backward pass of the layer on the tcgen05 tensor cores:
//
//   rb_gemm_dgrad   dX[t][j] = sum_i dY[t][i] W^[i][j],  W^ = sum_k alpha_k (.) B_k
//   rb_gemm_wgrad   dW[m][j] = add[m][j] + sum_t dY[t][m] s[t][j / 128] c[t][j]
//
// Both are products P[n][j] = sum_r B[n][r] A[r][j] in which one operand
// comes from HBM in a compressed form (sign planes and scales, or e4m3 codes
// and scales) whose rows run along the columns j, and the other is dY in 16
// bits. A 128-column tile of the compressed operand is expanded, 64 rows r at
// a time, into shared memory as the MMA's A (columns j = MMA rows, stored
// "M-major": 64 columns of one r per 128-byte swizzled row), so neither a
// transposed nor an expanded copy of it ever reaches HBM. dY tiles arrive by TMA:
// K-major for dgrad (a row of dY runs along r = i), N-major for wgrad (it
// runs along n = m).
//
// Two rings: C, the compressed operand as it lies in HBM (64 rows of 128 codes,
// or of 4 plane words per path) with its rows' scales, and the stages, its expansion A beside
// the dY tile B (TMA). A stage has one full barrier, for the expansion's
// arrivals and B's bytes, and one empty barrier: the MMA warp issues a stage's
// MMAs in about 300 cycles when it waits once and commits once, and took
// 550 with separate barriers for A and B, more than the 512 that the MMAs
// of a 256-wide tile last.
//
// Roles: warp 0 MMAs, 1 B loads, 2-3 C copies, 4-7 epilogue, then groups of four
// expansion warps that take the stages in turn.
// Three forms:
//   ONE    a CTA walks its 128 x BN tiles with two accumulators, so the
//          epilogue of a tile overlaps the next tile's MMAs;
//   SPLIT  few tiles: a cluster of CTAs shares a tile, each takes part of the
//          rows r, and the sums meet in distributed shared memory in rank
//          order;
//   PAIR   256-wide n tiles: two CTAs share a 256 x 256 tile (cta_group::2);
//          each expands its own 128 columns j and loads half of the dY tile.
//          One CTA with a 256-wide tile is bound by shared memory's 128 bytes
//          per cycle: it writes and reads 16 KB of A and 32 KB of B (and the
//          compressed operand) for 512 cycles of MMAs, which took 860 cycles a
//          stage (dgrad, two paths) and 1000 (wgrad). The pair moves 16 KB of
//          B in each CTA, and a stage takes about 600 cycles.
//
// Measured (2048 tokens x 14336 x 4096, bf16; 1628 TFLOP/s is the measured bf16
// peak in bursts, 1361 under the power cap, which both kernels reach, at 1.45 GHz):
// dgrad, two paths, 198 us, 1214 TFLOP/s (to fp32 dX 214 us; four paths with fp16
// scales per 128 columns 323 us: the expansion's work); wgrad to fp32 without
// `add` 231 us, 1040 TFLOP/s, to bf16 223 us; with an fp32 `add`, whose bytes
// take 36 us of HBM's time, 273 us.
// dgrad of 16 tokens through 8192 x 8192: 24.4 us (stage cycle, see STAGE_CYCLES);
// wgrad of 777 tokens x 256 x 256: 8.5 us (launch, fill and the ranks' sum).
//
// Rounding: dgrad's operand W^[i][j] is the exact sum of the scales (to fp32)
// rounded once to dY's 16-bit type; wgrad's operand s c is exact in that type
// for scales that are powers of two in its range, as rb_pack8 writes them,
// and rounded to it otherwise. Products are exact, sums fp32, in segments (see
// SEGMENT_F16).
#include "rb_tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace rb {
namespace {

using namespace tc;

constexpr int EPI_WARPS = 4, GROUP_WARPS = 4;
constexpr int BR = 64;                          // rows r per stage
constexpr uint32_t A_BYTES = 128 * BR * 2;      // two chunks of [64 r][64 j]
constexpr uint32_t CHUNK = 64 * BR * 2;         // 8 KB
enum : int { DGRAD = 0, WGRAD = 1 };
enum : int { ONE = 0, SPLIT = 1, PAIR = 2 };
// The tensor core cuts an accumulator's low bits off at every MMA, towards
// zero, so the error grows with the number of terms: of fp16 terms of one sign
// it is 5.4e-6 of the sum after 1024 terms, 9.6e-5 after 16384 and 1.5e-3 after 262144
// (bf16: 1.3e-6, 6.7e-5, 1.5e-3), of random signs 1.0e-6, 1.8e-5 and 3e-4 (2-norm).
// A long contraction is therefore summed in segments, each from an accumulator
// of its own, added to the sum so far with one rounding to nearest by the epilogue:
// fp32 outputs in segments of 1024 (fp16) or 2048 terms (bf16), 16-bit outputs
// of 16384, whose 1e-4 is a fifth of fp16's half step.
// The sum so far stays in tensor memory (2048 tokens x 14336 x 4096 to fp32 dX from
// bf16 201 -> 213 us, from fp16 210 -> 248 us: a pair's tile leaves room for one
// accumulator beside it, so its MMAs wait for the epilogue at a segment's end). Of an fp32
// weight gradient it is the output itself, which lies in L2 then, and a split
// one takes a launch for each segment.
constexpr int SEGMENT_F16 = 16, SEGMENT_BF16 = 32, SEGMENT_OUT16 = 256;     // stages
// How a stage's scales (of all paths) reach shared memory:
//   ASYNC  4-byte asynchronous copies (of fp32 values, or of pairs of fp16
//          values that hold the wanted ones);
//   LOADED fp16 scales whose pairs straddle rows or paths: loaded and stored.
// They, and the 16 bytes of plane words of each row and path, are not fetched
// by TMA: a box whose rows are 16 bytes takes it about 4 cycles a row, so
// that the 128 rows of two paths alone took longer (590 cycles a stage) than the
// MMAs of a 256-wide tile. Two warps copy stages in turn.
enum : int { ASYNC = 0, LOADED = 1 };

template <int MODE, int NP, int BN, int FORM>
struct BwCfg {
    static constexpr int BNC = FORM == PAIR ? BN / 2 : BN;      // rows of the dY tile in this CTA
    static constexpr uint32_t B_BYTES = BNC * BR * 2;
    static constexpr uint32_t C_BYTES = MODE == WGRAD ? 128 * BR : NP * 16 * BR;
    static constexpr uint32_t S_BYTES = NP * 4 * BR;       // most bytes of a stage's scales
    // Expansion groups of four warps (a group's stage takes about 1700 cycles)
    // and copying warps.
    // A split dgrad tile of few tokens has shared memory for a fourth group and
    // deeper rings: 16 tokens x 8192 x 8192 25.25 -> 24.5 us (six groups 24.4,
    // but 4096 x 4096 11.14 -> 11.4, with four 11.0).
    static constexpr bool DEEP = MODE == DGRAD && FORM == SPLIT && BN <= 64 && NP <= 2;
    static constexpr int GROUPS = DEEP ? 4 : 3, C_WARPS = MODE == WGRAD ? 1 : 2;
    static constexpr int MMA_WARP = 0, B_WARP = 1, C_WARP = 2, EPI_WARP0 = 4, EXP_WARP0 = EPI_WARP0 + EPI_WARPS;
    static constexpr int THREADS = 32 * (EXP_WARP0 + GROUPS * GROUP_WARPS);
    // Slots are a multiple of the groups (and copying warps) that take them in
    // turn, so that a slot always belongs to the same one, which then waits
    // for every phase of its barriers. Otherwise a group could wait for a
    // slot's use while the use before, another group's, was still being
    // filled (copies land in any order), and a parity wait for the phase
    // after an open one returns at once.
    static constexpr int ST = DEEP ? 8 : 6, CS = MODE == WGRAD ? 3 : DEEP ? 12 : 6;
    static_assert(ST % GROUPS == 0 && CS % GROUPS == 0 && CS % C_WARPS == 0, "a waiter would miss phases of its barriers");
    static constexpr uint32_t STAGE = A_BYTES + B_BYTES, TILES = ST * STAGE + CS * (C_BYTES + S_BYTES);
    static constexpr int BARS = 2 * (ST + CS) + 4;
    // at least 120 KB, so that two CTAs never share an SM's tensor memory
    static constexpr uint32_t SMEM = (TILES < 119u * 1024u ? 119u * 1024u : TILES) + 1024u;
    // two accumulators and, from column SUM_COL on, a sum of segments (in a
    // pair in the place of the second accumulator)
    static constexpr uint32_t TMEM_COLS = 2 * BN, SUM_COL = FORM == PAIR ? BN : 2 * BN, SUM_TMEM_COLS = FORM == PAIR ? 2 * BN : 4 * BN;
    static_assert(SUM_TMEM_COLS <= 512, "tensor memory");
    static_assert(SMEM + 512 <= 227 * 1024, "shared memory");
    // The CTAs of a cluster wait for one another while they hold tensor memory.
    // Beside one of these no CTA of another such kernel (rb_gemm8's take 97 KB
    // or more) finds room on an SM: if together they wanted more than 512 columns,
    // two clusters on two streams could each hold what the other waits for.
    static_assert(FORM == ONE || SMEM >= 132u * 1024u, "another cluster's CTA may share the SM's tensor memory");
    static_assert(FORM != SPLIT || BN * 512u <= TILES, "a split tile's sums do not fit the rings");
};

struct BwArgs {
    uint32_t* err;
    const uint32_t* planes;     // dgrad
    const void* alpha;
    const uint8_t* codes;       // wgrad
    const float* scales;
    const void* add;            // wgrad, may be null
    bool add_ahead;             // its rows take bulk prefetches
    void* out;
    int64_t R, N, J, ldo;       // contraction, output rows, output columns (K)
    int bn;                     // output rows per tile (BN, or less in a pair of dgrad)
    int j_tiles, n_tiles;
    bool first;                 // of the call's launches: clears the error word
    int segment;                // stages summed in one accumulator, see SEGMENT_F16
    bool sum_in_tmem;           // where the segments before are summed: tensor memory, or the output
    int out_dt;
    bool sliced, alpha_f16, g128;
    int scales_by;
    bool scales_f16;            // as they lie in shared memory
    uint32_t scale_row, scale_path;     // bytes from one row's and from one path's to the next there
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// error word of the calls without a workspace: nobody reads it
__device__ uint32_t unrecorded;

__device__ __forceinline__ float ld_cluster(uint32_t local, uint32_t rank) {
    const uint32_t addr = cluster_addr(local, rank);
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// Descriptor of an M-major (N-major) tile in the 128-byte swizzle layout:
// 64 columns of one row r per 128 bytes, 8 rows per 1024-byte atom (stride
// offset 1024), the next 64 columns one chunk on (leading offset CHUNK).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(CHUNK >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// fp32 accumulator, A and B both fp16 or both bf16, A M-major, B K- or N-major
__host__ __device__ constexpr uint32_t idesc_bw(int n, bool bf16, bool b_mn, int m) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (1u << 15) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// two floats in the 16-bit type of dY
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// 32 weights from the 32 bits of w[p]: path 0 gives the sign, the paths that
// agree or disagree with it choose one of 2^(NP-1) magnitudes.
// h[i] holds columns i and i + 16 of the word: a left shift by 15 - i puts both
// sign bits in place, and a byte's top bit spread over 16 bits by PRMT gives
// both choices at once. The columns of a tile are thus permuted within 32
// (position 2i: column i, 2i + 1: column i + 16), which the epilogue undoes.
template <int NP, bool BF16>
__device__ __forceinline__ void expand_planes(const uint32_t (&w)[NP], const float (&al)[NP], uint32_t (&h)[16]) {
    // of bit p - 1 of m: path p agrees with path 0 (the sum of up to four
    // scales is rounded to fp32, then once to dY's type)
    constexpr int NM = 1 << (NP - 1);
    uint32_t mag[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        float v = al[0];
#pragma unroll
        for (int p = 1; p < NP; ++p) v += (m >> (p - 1)) & 1 ? al[p] : -al[p];
        mag[m] = pack2<BF16>(v, v);
    }
    const uint32_t minus = ~w[0];
    uint32_t s[NP][8];
#pragma unroll
    for (int p = 1; p < NP; ++p) {
        const uint32_t x = minus ^ w[p];       // set: the path agrees with path 0
#pragma unroll
        for (int k = 0; k < 8; ++k) s[p][k] = x << (7 - k);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t v[NM];
#pragma unroll
        for (int k = 0; k < NM; ++k) v[k] = mag[k];
#pragma unroll
        for (int p = 1; p < NP; ++p) {
            // bits i and i + 16: the top bits of bytes i / 8 and i / 8 + 2 of s[i % 8]
            const uint32_t lo = 8u | (i >> 3), hi = 8u | ((i >> 3) + 2);
            const uint32_t mask = prmt(s[p][i & 7], 0u, lo | (lo << 4) | (hi << 8) | (hi << 12));
#pragma unroll
            for (int k = 0; k < (NM >> p); ++k) v[k] = (mask & v[2 * k + 1]) | (~mask & v[2 * k]);
        }
        h[i] = v[0] ^ ((minus << (15 - i)) & 0x80008000u);
    }
}

// 32 codes times the row's scale
template <bool BF16>
__device__ __forceinline__ void expand_codes(const uint32_t (&c)[8], float s, uint32_t (&h)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
            : "r"(c[i]));
    }
    // a scale that fp16 holds exactly: one fp16 product rounds s c once
    const __half sh = __float2half_rn(s);
    if (!BF16 && __half2float(sh) == s) {
        const __half2 s2 = __half2half2(sh);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), s2);
            h[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            h[i] = pack2<BF16>(f.x * s, f.y * s);
        }
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds_scale(uint32_t addr, bool f16) {
    if (f16) {
        uint16_t h;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
        return __half2float(__ushort_as_half(h));
    }
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// A ring position: slot and phase parity, advanced by one stage.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int by = 1) {
        slot += by;
        if (slot >= N) {
            slot -= N;
            ph ^= 1u;
        }
    }
};

__device__ __forceinline__ float load_out(const void* p, int dt, int64_t i) {
    if (dt == B8_F32) return static_cast<const float*>(p)[i];
    if (dt == B8_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_out(void* p, int dt, int64_t i, float v) {
    if (dt == B8_F32) static_cast<float*>(p)[i] = v;
    else if (dt == B8_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// asynchronous copies global -> shared; cp_async4 reads the first `bytes` of 4 and
// fills the rest with zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void to_out(float v, float* p) { *p = v; }
__device__ __forceinline__ void to_out(float v, __half* p) { *p = __float2half_rn(v); }
__device__ __forceinline__ void to_out(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// One column of up to 32 output rows (add + v), all loads before the first
// store. What is added to the fp32 output itself (a gradient summed in place, the
// later segments) is added in L2, with nothing to wait for: 8192 tokens x
// 14336 x 4096 from fp16 1108 -> 982 us. One thread makes all updates of an
// element, in order, so the result does not change from run to run; sums below
// 2^-126 become zero there.
template <typename T>
__device__ __forceinline__ void store_rows(void* out, const void* add, int64_t at, int64_t ldo, int left,
                                           const uint32_t (&v)[32]) {
    T* o = static_cast<T*>(out) + at;
    const T* ad = static_cast<const T*>(add) + at;
    T r[32];
    if (sizeof(T) == 4 && left >= 32 && add == out) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(o + i * ldo), "f"(__uint_as_float(v[i])) : "memory");
    } else if (left >= 32) {
        if (add) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = ad[i * ldo];
#pragma unroll
            for (int i = 0; i < 32; ++i) to_out(__uint_as_float(v[i]) + static_cast<float>(r[i]), o + i * ldo);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) to_out(__uint_as_float(v[i]), o + i * ldo);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < left) to_out(__uint_as_float(v[i]) + (add ? static_cast<float>(ad[i * ldo]) : 0.0f), o + i * ldo);
    }
}

template <int MODE, int NP, int BN, bool BF16, int FORM>
__global__ void __launch_bounds__(BwCfg<MODE, NP, BN, FORM>::THREADS, 1)
gemm_bwd_kernel(const __grid_constant__ CUtensorMap dmap, const __grid_constant__ CUtensorMap cmap, BwArgs a) {
    using C = BwCfg<MODE, NP, BN, FORM>;
    constexpr int ST = C::ST, CS = C::CS, GROUPS = C::GROUPS;
    constexpr int EPI_WARP0 = C::EPI_WARP0, EXP_WARP0 = C::EXP_WARP0, B_WARP = C::B_WARP, MMA_WARP = C::MMA_WARP, C_WARP = C::C_WARP;
    constexpr int C_WARPS = C::C_WARPS;
    extern __shared__ __align__(1024) unsigned char dsm[];
    __shared__ __align__(8) uint64_t bars[C::BARS];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;
    const uint32_t tiles = (smem_addr(dsm) + 1023u) & ~1023u;
    auto a_tile = [&](int s) { return tiles + static_cast<uint32_t>(s) * C::STAGE; };
    auto b_tile = [&](int s) { return a_tile(s) + A_BYTES; };
    auto c_tile = [&](int s) { return tiles + ST * C::STAGE + static_cast<uint32_t>(s) * C::C_BYTES; };
    auto s_tile = [&](int s) { return tiles + ST * C::STAGE + CS * C::C_BYTES + static_cast<uint32_t>(s) * C::S_BYTES; };
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (ST + s); };
    auto full_c = [&](int s) { return bar0 + 8u * (2 * ST + s); };
    auto empty_c = [&](int s) { return bar0 + 8u * (2 * ST + CS + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * (ST + CS) + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * (ST + CS) + 2 + b); };

    const uint32_t rank = FORM == ONE ? 0u : cluster_rank(), size = FORM == ONE ? 1u : cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* err = a.err ? a.err : &unrecorded;
    if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *err = 0u;      // flags are raised only by waits that ran out
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            // four expansion warps, the B loads, and in a pair's even CTA the other's word
            mbar_init(full_bar(s), GROUP_WARPS + 1 + (FORM == PAIR && rank == 0 ? 1 : 0));
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < CS; ++s) {
            // a copying warp's lanes, and wgrad's codes (TMA)
            mbar_init(full_c(s), 32 + (MODE == WGRAD ? 1 : 0));
            mbar_init(empty_c(s), GROUP_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), FORM == PAIR ? 2 * EPI_WARPS : EPI_WARPS);
        }
        abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem_cols = a.sum_in_tmem ? C::SUM_TMEM_COLS : C::TMEM_COLS;
    if (warp == MMA_WARP) {
        if constexpr (FORM == PAIR) tmem_alloc2(smem_addr(&tmem_slot), tmem_cols);
        else tmem_alloc(smem_addr(&tmem_slot), tmem_cols);
    }
    fence_before();
    if constexpr (FORM == PAIR) cluster_sync();      // the peer's barriers are ready, too
    else __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    const int bn = FORM == PAIR ? a.bn : BN;
    const int64_t nr = (a.R + BR - 1) / BR;
    const int r_lo = FORM == SPLIT ? static_cast<int>(nr * rank / size) : 0;
    const int r_hi = FORM == SPLIT ? static_cast<int>(nr * (rank + 1) / size) : static_cast<int>(nr);
    // a pair's CTAs take adjacent column tiles (of an odd number, the last
    // pair's second CTA works on zeros and stores nothing)
    const int jw = FORM == PAIR ? (a.j_tiles + 1) / 2 : a.j_tiles;
    const int units = jw * a.n_tiles;
    const int u0 = static_cast<int>(blockIdx.x / size);
    const int u_step = FORM == SPLIT ? units : static_cast<int>(gridDim.x / size);
    auto j_tile = [&](int u) { return FORM == PAIR ? 2 * (u % jw) + static_cast<int>(rank) : u % jw; };
    auto n_tile = [&](int u) { return u / jw; };
    // accumulators in turn: two, but one where a pair's other one holds the sum
    const int flip = FORM == PAIR && a.sum_in_tmem ? 0 : 1;

    auto epilogue = [&] {
        const int q = warp - EPI_WARP0;          // lane quarter
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const int column = MODE == DGRAD ? (lane >> 1) + (lane & 1) * 16 : lane;      // of this tensor-memory lane
        int tile = 0;
        // `add` is fetched into L2 a tile ahead (64 of a tile's rows of 128 values
        // by each warp): 32 loads in flight a warp hide L2's latency, not HBM's
        auto prefetch_add = [&](int u) {
            if (MODE != WGRAD || !a.add_ahead || u >= units || static_cast<int64_t>(j_tile(u)) * 128 >= a.J) return;
            const int64_t es = a.out_dt == B8_F32 ? 4 : 2;
            for (int c = q * 32 + lane; c < bn; c += 128) {
                const int64_t n = static_cast<int64_t>(n_tile(u)) * bn + c;
                if (n < a.N)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.add) +
                                                                                   (n * a.ldo + static_cast<int64_t>(j_tile(u)) * 128) * es),
                                 "r"(static_cast<uint32_t>(128 * es))
                                 : "memory");
            }
        };
        prefetch_add(u0);
        for (int u = u0, lo = r_lo; u < units; ++tile) {
            const int b = tile & flip;
            const bool keep = a.sum_in_tmem && lo + a.segment < r_hi;
            // to a later segment, the sums so far
            const void* add = MODE != WGRAD ? nullptr : lo > r_lo && !a.sum_in_tmem ? a.out : a.add;
            if (lo == r_lo) prefetch_add(u + u_step);
            const int64_t j = static_cast<int64_t>(j_tile(u)) * 128 + q * 32 + column;
            const int64_t n0 = static_cast<int64_t>(n_tile(u)) * bn;
            const bool mine = FORM != PAIR || j < a.J;
            if (!__all_sync(FULL_MASK, mbar_wait(acc_full(b), static_cast<uint32_t>(tile >> flip) & 1u, abort_flag, err, 8u)) ||
                *abort_flag)
                break;
            fence_after();
            // a segment joins the sum so far: there, or the last one in its accumulator
            if (a.sum_in_tmem) {
#pragma unroll 1
                for (int c0 = 0; c0 < bn; c0 += 16) {
                    const uint32_t acc = tmem + lanes + static_cast<uint32_t>(b * BN + c0), sum = tmem + lanes + C::SUM_COL + static_cast<uint32_t>(c0);
                    uint32_t v[16], w[16];
                    tmem_load<16>(acc, v);
                    if (lo > r_lo) {
                        tmem_load<16>(sum, w);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
                    }
                    tmem_store16(keep ? sum : acc, v);
                }
                tmem_store_wait();
            }
#pragma unroll 1
            for (int c0 = 0; c0 < bn && !keep; c0 += 32) {
                uint32_t v[32];
                tmem_load<32>(tmem + lanes + static_cast<uint32_t>(b * BN + c0), v);
                if constexpr (FORM == SPLIT) {
                    float* buf = reinterpret_cast<float*>(dsm + (tiles - smem_addr(dsm))) + c0 * 128 + q * 32 + column;
#pragma unroll
                    for (int i = 0; i < 32; ++i) buf[i * 128] = __uint_as_float(v[i]);
                } else {
                    const int left = mine ? static_cast<int>(min(static_cast<int64_t>(min(32, bn - c0)), a.N - n0 - c0)) : 0;
                    const int64_t at = (n0 + c0) * a.ldo + j;
                    if (a.out_dt == B8_F32) store_rows<float>(a.out, add, at, a.ldo, left, v);
                    else if (a.out_dt == B8_F16) store_rows<__half>(a.out, add, at, a.ldo, left, v);
                    else store_rows<__nv_bfloat16>(a.out, add, at, a.ldo, left, v);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (FORM == PAIR && rank == 1) mbar_arrive_remote(acc_empty(b), 0);
                else mbar_arrive(acc_empty(b));
            }
            lo += a.segment;
            if (lo >= r_hi) {
                lo = r_lo;
                u += u_step;
            }
        }
    };
    if (warp == B_WARP) {
        if (lane == 0) {
            Ring<ST> q;
            int it = 0;
            bool ok = true;
            for (int u = u0; u < units && ok; u += u_step) {
                const int n0 = n_tile(u) * bn + (FORM == PAIR ? static_cast<int>(rank) * (bn / 2) : 0);
                for (int rb = r_lo; rb < r_hi; ++rb, ++it, q.next()) {
                    if (!mbar_wait(empty_bar(q.slot), q.ph ^ 1u, abort_flag, err, 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full_bar(q.slot), static_cast<uint32_t>(FORM == PAIR ? bn / 2 : bn) * (BR * 2));
                    if constexpr (MODE == DGRAD) {
                        tma_load_2d(b_tile(q.slot), &dmap, rb * BR, n0, full_bar(q.slot));
                    } else {
#pragma unroll
                        for (int c = 0; c < C::BNC / 64; ++c)
                            tma_load_2d(b_tile(q.slot) + c * CHUNK, &dmap, n0 + c * 64, rb * BR, full_bar(q.slot));
                    }
                }
            }
            // after an abort the loads in flight land before the CTA gives up its shared memory
            // (the expansion may have left: the barrier's phase may stay open)
            if (*abort_flag)
                for (int i = it - 1; i >= 0 && i >= it - ST; --i)
                    mbar_drain(full_bar(i % ST), static_cast<uint32_t>(i / ST) & 1u);
            // the even CTA's commits also arrive here: all of them, before the CTA may go
            else if (FORM == PAIR)
                for (int i = it - 1; i >= 0 && i >= it - ST; --i)
                    mbar_drain(empty_bar(i % ST), static_cast<uint32_t>(i / ST) & 1u);
        }
    } else if (warp >= C_WARP && warp < C_WARP + C_WARPS) {
        const int mine = warp - C_WARP;
        Ring<CS> q;
        q.next(mine);
        int issued = 0, it = 0;          // stages of this warp; stages before this tile, modulo C_WARPS
        bool ok = true;
        const bool loaded = a.scales_by == LOADED;
        const bool per_block = MODE == WGRAD || a.g128;
        // two rows a lane, lane and lane + 32: bytes of a row of words, of a
        // path of words, of a row and a path of scales
        const int64_t w_row = a.sliced ? 64 : a.J >> 3, w_path = a.R * w_row * (a.sliced ? (a.J + 511) >> 9 : 1);
        const int es = MODE == DGRAD && a.alpha_f16 ? 2 : 4;
        const int64_t s_row = (per_block ? a.J >> 7 : 1) * es, s_path = a.R * s_row;
        const bool pairs = es == 2 && !per_block && !loaded;          // 32 copies bring 64 rows' fp16 scales
        const char* planes = reinterpret_cast<const char*>(a.planes);
        const char* scales = static_cast<const char*>(MODE == WGRAD ? static_cast<const void*>(a.scales) : a.alpha);
        for (int u = u0; u < units && ok; u += u_step, it = (it + r_hi - r_lo) % C_WARPS) {
            const int jt = min(j_tile(u), a.j_tiles - 1);
            int rb = r_lo + (mine - it + C_WARPS) % C_WARPS;
            int left = static_cast<int>(a.R - (static_cast<int64_t>(rb) * BR + (pairs ? 2 * lane : lane)));     // rows from this lane's first
            const char* wp = planes + (a.sliced ? static_cast<int64_t>(jt >> 2) * a.R * 64 + (jt & 3) * 16 : static_cast<int64_t>(jt) * 16) +
                             (static_cast<int64_t>(rb) * BR + lane) * w_row;
            const char* sp = scales + (per_block ? (static_cast<int64_t>(jt) * es & (loaded ? ~1ll : ~3ll)) : 0) +
                             (static_cast<int64_t>(rb) * BR + (pairs ? 2 * lane : lane)) * s_row;
            for (; rb < r_hi; rb += C_WARPS, q.next(C_WARPS), ++issued) {
                if (!__all_sync(FULL_MASK, mbar_wait(empty_c(q.slot), q.ph ^ 1u, abort_flag, err, 1u))) {
                    ok = false;
                    break;
                }
                if (MODE == WGRAD && lane == 0) {
                    mbar_arrive_expect_tx(full_c(q.slot), C::C_BYTES);
                    tma_load_3d(c_tile(q.slot), &cmap, j_tile(u) * 128, rb * BR, 0, full_c(q.slot));
                }
                const int rows_left = pairs ? left + lane : left;      // from row lane of the stage
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (MODE == DGRAD) {
                        const bool in = rows_left > 32 * k;
                        const char* src = in ? wp + 32 * k * w_row : planes;
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            cp_async16(c_tile(q.slot) + p * 16u * BR + (lane + 32 * k) * 16u, src + (in ? p * w_path : 0));
                    }
                    if (!pairs && !loaded) {
                        const bool in = left > 32 * k;
                        const char* src = in ? sp + 32 * k * s_row : scales;
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            cp_async4(s_tile(q.slot) + p * a.scale_path + (lane + 32 * k) * 4u, src + (in ? p * s_path : 0), in ? 4u : 0u);
                    }
                }
                if (MODE == DGRAD && pairs) {
                    const char* src = left > 0 ? sp : scales;               // rows 2 lane and 2 lane + 1
                    // of an odd number of rows, the last has nothing after it: what lies there
                    // is not the array's, and as a scale of row M it would turn dY's
                    // zeros into NaN if it were infinite
                    const uint32_t bytes = static_cast<uint32_t>(2 * max(min(left, 2), 0));
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        cp_async4(s_tile(q.slot) + p * a.scale_path + lane * 4u, src + (left > 0 ? p * s_path : 0), bytes);
                }
                if (MODE == DGRAD && loaded) {
                    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            const float v = left > 32 * k
                                                ? __half2float(__ldg(reinterpret_cast<const __half*>(sp + 32 * k * s_row + p * s_path)))
                                                : 0.0f;
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_tile(q.slot) + p * a.scale_path + (lane + 32 * k) * 4u), "f"(v)
                                         : "memory");
                        }
                    mbar_arrive(full_c(q.slot));
                } else {
                    // arrives once this lane's copies have landed
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full_c(q.slot)) : "memory");
                }
                left -= C_WARPS * BR;
                wp += C_WARPS * BR * w_row;
                sp += C_WARPS * BR * s_row;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // after an abort the codes in flight land before the CTA gives up its shared memory
        // (the other warp may have left: a barrier's phase may stay open)
        if (MODE == WGRAD && *abort_flag)
            for (int i = issued - 1; i >= 0 && i >= issued - CS; --i) {
                const int n = mine + i * C_WARPS;
                mbar_drain(full_c(n % CS), static_cast<uint32_t>(n / CS) & 1u);
            }
    } else if (FORM == PAIR && warp == MMA_WARP && rank == 1) {
        // the pair's MMAs are issued by the even CTA: tell it, stage by stage,
        // that this CTA's half of the operands is there
        if (lane == 0) {
            Ring<ST> q;
            bool ok = true;
            for (int u = u0; u < units && ok; u += u_step) {
                for (int rb = r_lo; rb < r_hi; ++rb, q.next()) {
                    if (!mbar_wait(full_bar(q.slot), q.ph, abort_flag, err, 2u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote(full_bar(q.slot), 0);
                }
            }
        }
    } else if (warp == MMA_WARP) {
        const uint32_t idesc = idesc_bw(bn, BF16, MODE == WGRAD, FORM == PAIR ? 256 : BM);
        auto commit = [](uint32_t bar) {
            if constexpr (FORM == PAIR) umma2_commit(bar);
            else umma_commit(bar);
        };
        Ring<ST> q;
        int tile = 0;
        bool ok = true, ready = false;
        // the low words of the descriptors of slot 0 (the high words do not change)
        const uint64_t ad0 = smem_desc_mn(a_tile(0)), bd0 = MODE == DGRAD ? smem_desc(b_tile(0)) : smem_desc_mn(b_tile(0));
        // 16 rows r on: two 1024-byte atoms (M- or N-major), 32 bytes (K-major)
        constexpr uint32_t A_STEP = 128u, B_STEP = MODE == DGRAD ? 2u : 128u;
        // One lane runs the loop: with a stage's votes, election and
        // reconvergence a warp was 1 to 3 % slower (dgrad, 64 tokens x 8192 x
        // 8192 28.2 -> 27.4 us).
        if (elect_one()) {
            for (int u = u0, lo = r_lo; u < units && ok; ++tile) {
                const int b = tile & flip, hi = min(lo + a.segment, r_hi);
                const uint32_t aph = (static_cast<uint32_t>(tile >> flip) & 1u) ^ 1u, d = tmem + static_cast<uint32_t>(b * BN);
                ok = mbar_wait(acc_empty(b), aph, abort_flag, err, 2u);
                for (int rb = lo; rb < hi && ok; ++rb) {
                    if (!ready && !mbar_wait(full_bar(q.slot), q.ph, abort_flag, err, 2u)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const int slot = q.slot;
                    const uint32_t off = static_cast<uint32_t>(slot) * (C::STAGE >> 4);
#pragma unroll
                    for (int kk = 0; kk < BR / 16; ++kk) {
                        const uint64_t ad = ad0 + off + A_STEP * kk, bd = bd0 + off + B_STEP * kk;
                        const uint32_t more = (rb > lo || kk > 0) ? 1u : 0u;
                        if constexpr (FORM == PAIR) umma2_f16(d, ad, bd, idesc, more);
                        else umma_f16(d, ad, bd, idesc, more);
                    }
                    commit(empty_bar(slot));
                    if (rb + 1 == hi) commit(acc_full(b));
                    q.next();
                    ready = mbar_test(full_bar(q.slot), q.ph);
                }
                // after an abort the teardown waits for it
                if (!ok) commit(acc_full(b));
                lo = hi;
                if (lo >= r_hi) {
                    lo = r_lo;
                    u += u_step;
                }
            }
            // every MMA issued has completed before the tensor memory is given up
            if (!ok)
                for (int i = tile - 1; i >= 0 && i >= tile - 1 - flip; --i)
                    mbar_drain(acc_full(i & flip), static_cast<uint32_t>(i >> flip) & 1u);
        }
    } else if (warp >= EXP_WARP0) {
        // A thread expands two rows of a stage, 32 columns of each. wgrad: warp wq
        // takes columns 32 wq.. of rows lane and lane + 32. dgrad: 4 lanes
        // share a row (its 4 words, one LDS of 128 contiguous bytes per 8
        // rows); the words 2 and 3 go to the other 64-column chunk, whose
        // rows lie on the same banks, so their lanes store the 16-byte
        // pieces in the order 2, 3, 0, 1 (bytes of the word swapped to match).
        // Either way the 8 lanes of a store phase cover all banks once.
        constexpr int UROWS = MODE == WGRAD ? 32 : 8;
        const int grp = (warp - EXP_WARP0) / GROUP_WARPS, wq = (warp - EXP_WARP0) % GROUP_WARPS;
        const int wd = MODE == WGRAD ? wq : lane & 3;
        const uint32_t row = MODE == WGRAD ? lane : wq * 16 + (lane >> 2);
        const uint32_t sw = row & 7u;
        const uint32_t at = static_cast<uint32_t>(wd >> 1) * CHUNK + row * 128u;
        const uint32_t c0 = static_cast<uint32_t>(wd & 1) * 4u;
        const uint32_t cx = MODE == DGRAD && wd >= 2 ? 2u : 0u;
        const uint32_t bytes = cx ? 0x2301u : 0x3210u;
        Ring<ST> qa;
        Ring<CS> qc;
        bool ok = true;
        int it = 0;                      // stages before this tile, modulo GROUPS
        qa.next(grp);
        qc.next(grp);
        for (int u = u0; u < units && ok; u += u_step, it = (it + r_hi - r_lo) % GROUPS) {
            int rb = r_lo + (grp - it + GROUPS) % GROUPS;          // the group's first stage of this tile
            // of a pair of fp16 group scales, the tile's
            const uint32_t scale_at = a.scales_f16 && a.g128 ? (j_tile(u) & 1) * 2u : 0u;
            for (; rb < r_hi; rb += GROUPS, qa.next(GROUPS), qc.next(GROUPS)) {
                if (!__all_sync(FULL_MASK, mbar_wait(full_c(qc.slot), qc.ph, abort_flag, err, 4u))) {
                    ok = false;
                    break;
                }
                uint32_t h[2][16];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t r = row + k * UROWS;
                    float sc[NP];
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        sc[p] = lds_scale(s_tile(qc.slot) + p * a.scale_path + r * a.scale_row + scale_at, a.scales_f16);
                    if constexpr (MODE == WGRAD) {
                        const uint32_t base = c_tile(qc.slot) + r * 128u;
                        const uint4 x = lds128(base + (((2u * wd) ^ sw) << 4)), y = lds128(base + (((2u * wd + 1u) ^ sw) << 4));
                        const uint32_t c[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                        expand_codes<BF16>(c, sc[0], h[k]);
                    } else {
                        uint32_t w[NP];
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            w[p] = prmt(lds32(c_tile(qc.slot) + p * 16u * BR + r * 16u + 4u * wd), 0u, bytes);
                        expand_planes<NP, BF16>(w, sc, h[k]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_c(qc.slot));
                if (!__all_sync(FULL_MASK, mbar_wait(empty_bar(qa.slot), qa.ph ^ 1u, abort_flag, err, 4u))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t base = a_tile(qa.slot) + at + static_cast<uint32_t>(k * UROWS) * 128u;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        sts128(base + (((c0 + (c ^ cx)) ^ sw) << 4), h[k][4 * c], h[k][4 * c + 1], h[k][4 * c + 2], h[k][4 * c + 3]);
                }
                fence_proxy_async_smem();   // make the generic-proxy stores visible to the tensor core
                __syncwarp();
                if (lane == 0) mbar_arrive(full_bar(qa.slot));
            }
        }
    } else if (warp >= EPI_WARP0) {
        epilogue();
    }
    __syncwarp();
    fence_before();
    if constexpr (FORM == SPLIT) {
        cluster_sync();
        // the CTAs of the cluster take the output rows in turn and add the ranks' sums in rank order
        const int64_t j = static_cast<int64_t>(j_tile(u0)) * 128 + (threadIdx.x & 127);
        const int64_t n0 = static_cast<int64_t>(n_tile(u0)) * bn;
        const int rows = static_cast<int>(min(static_cast<int64_t>(BN), a.N - n0));
        if (*abort_flag == 0u && threadIdx.x < 384) {
            for (int c = static_cast<int>(rank) * 3 + (threadIdx.x >> 7); c < rows; c += static_cast<int>(size) * 3) {
                float v = 0.0f;
                for (uint32_t k = 0; k < size; ++k) v += ld_cluster(tiles + static_cast<uint32_t>(c * 128 + (threadIdx.x & 127)) * 4u, k);
                const int64_t o = (n0 + c) * a.ldo + j;
                if (MODE == WGRAD && a.add) v += load_out(a.add, a.out_dt, o);
                store_out(a.out, a.out_dt, o, v);
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
        if constexpr (FORM == PAIR) tmem_dealloc2(tmem, tmem_cols);
        else tmem_dealloc(tmem, tmem_cols);
    }
}

struct BwMaps {
    CUtensorMap dy, c;      // dY, and wgrad's codes
};

// How the scales [n][R] or [n][R][J / 128] come to shared memory.
void plan_scales(BwArgs& a, int n) {
    const bool per_block = a.g128 || a.codes;
    const bool pairs = a.alpha_f16 && !per_block;
    a.scales_by = a.alpha_f16 && ((per_block ? a.J / 128 : n > 1 ? a.R : 0) % 2 != 0 || reinterpret_cast<uintptr_t>(a.alpha) % 4 != 0)
                      ? LOADED
                      : ASYNC;
    a.scales_f16 = a.alpha_f16 && a.scales_by == ASYNC;
    a.scale_row = pairs && a.scales_by == ASYNC ? 2 : 4;
    a.scale_path = a.scale_row * BR;
}

template <int MODE, int NP, int BN, bool BF16, int FORM>
cudaError_t launch(const BwMaps& m, BwArgs& a, int cluster, cudaStream_t s) {
    constexpr size_t smem = BwCfg<MODE, NP, BN, FORM>::SMEM;
    auto kern = gemm_bwd_kernel<MODE, NP, BN, BF16, FORM>;
    static SmemLimit limit;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, limit);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(FORM == PAIR ? (a.j_tiles + 1) / 2 : a.j_tiles) * a.n_tiles;
    const int64_t sms = device_sm_count();
    // segments, where a CTA has more stages than one holds (launch_gemm_wgrad
    // sees to it that a split fp32 weight gradient has not)
    const bool fp32 = a.out_dt == B8_F32;
    const int64_t ctas = FORM == SPLIT ? cluster : 1, stages = ((a.R + BR - 1) / BR + ctas - 1) / ctas;
    const int segment = !fp32 ? SEGMENT_OUT16 : BF16 ? SEGMENT_BF16 : SEGMENT_F16;
    a.segment = stages > segment ? segment : 1 << 30;
    a.sum_in_tmem = stages > segment && (MODE == DGRAD || !fp32);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(FORM == SPLIT ? units * cluster : FORM == PAIR ? 2 * std::min(units, sms / 2)
                                                                                             : std::min(units, sms)));
    cfg.blockDim = dim3(BwCfg<MODE, NP, BN, FORM>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = FORM == ONE ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, m.dy, m.c, a);
}

// A stage takes about 600 cycles (the MMA warp's waits, issue and commit; the
// expansion: 1700 cycles of each group) or its MMAs' 2 bn in a pair, whichever is more. Time in stages of
// the two ways to cover N rows of dY of more than 64:
constexpr int64_t STAGE_CYCLES = 600;

// 256-wide tiles of CTA pairs, of which a dgrad tile may use only bn rows (128
// to 256 by 16): the bn with the least time over all waves of tiles
int64_t pair_cycles(const BwArgs& a, int* bn, bool narrow) {
    const int64_t pairs = device_sm_count() / 2, jw = (a.j_tiles + 1) / 2, nr = (a.R + BR - 1) / BR;
    int64_t best = 0;
    for (int n = 256; n >= (narrow ? 128 : 256); n -= 16) {
        const int64_t waves = (jw * ((a.N + n - 1) / n) + pairs - 1) / pairs;
        const int64_t cycles = waves * nr * std::max<int64_t>(2 * n, STAGE_CYCLES);
        if (best == 0 || cycles < best) {
            best = cycles;
            *bn = n;
        }
    }
    return best;
}

// CTAs that share a tile's rows r
int split_of(int64_t units, int64_t nr) {
    int split = 1;
    while (split < 8 && units * (split + 1) <= device_sm_count() && split < nr) ++split;
    return split;
}

// 128-wide tiles, of one CTA or split
int64_t one_cycles(const BwArgs& a) {
    const int64_t units = a.j_tiles * ((a.N + 127) / 128), nr = (a.R + BR - 1) / BR, sms = device_sm_count();
    const int split = split_of(units, nr);
    return split > 1 ? (nr + split - 1) / split * STAGE_CYCLES : (units + sms - 1) / sms * nr * STAGE_CYCLES;
}

// Rows of the dY tile: the narrowest that covers N; 256 is a CTA pair's. (600
// tokens x 14336 x 4096, dgrad: 160 tiles of 128, two waves of 148, take 148 us; 64
// pairs' tiles of 160 one wave.)
int bwd_tile(BwArgs& a, bool narrow) {
    a.bn = a.N <= 32 ? 32 : a.N <= 64 ? 64 : 128;
    int bn = 0;
    if (a.N > 128 && pair_cycles(a, &bn, narrow) < one_cycles(a)) {
        a.bn = bn;
        return 256;
    }
    return a.bn;
}

template <int MODE, int NP, int BN>
cudaError_t launch_bn(const BwMaps& m, BwArgs& a, bool bf16, cudaStream_t s) {
    a.n_tiles = static_cast<int>((a.N + BN - 1) / BN);
    const int64_t units = static_cast<int64_t>(a.j_tiles) * a.n_tiles, nr = (a.R + BR - 1) / BR;
    const int split = split_of(units, nr);
    if (split > 1)
        return bf16 ? launch<MODE, NP, BN, true, SPLIT>(m, a, split, s) : launch<MODE, NP, BN, false, SPLIT>(m, a, split, s);
    return bf16 ? launch<MODE, NP, BN, true, ONE>(m, a, 1, s) : launch<MODE, NP, BN, false, ONE>(m, a, 1, s);
}

template <int NP>
cudaError_t launch_dgrad_np(BwArgs& a, const void* dY, int64_t ldd, bool bf16, cudaStream_t s) {
    BwMaps m{};
    const int bn = bwd_tile(a, true);
    plan_scales(a, NP);
    a.first = true;
    cudaError_t e = make_x_map(&m.dy, dY, a.R, a.N, ldd, bn == 256 ? a.bn / 2 : bn);
    if (e != cudaSuccess) return e;
    switch (bn) {
        case 32: return launch_bn<DGRAD, NP, 32>(m, a, bf16, s);
        case 64: return launch_bn<DGRAD, NP, 64>(m, a, bf16, s);
        case 128: return launch_bn<DGRAD, NP, 128>(m, a, bf16, s);
        default: break;
    }
    a.n_tiles = static_cast<int>((a.N + a.bn - 1) / a.bn);
    return bf16 ? launch<DGRAD, NP, 256, true, PAIR>(m, a, 2, s) : launch<DGRAD, NP, 256, false, PAIR>(m, a, 2, s);
}

}  // namespace

cudaError_t launch_gemm_dgrad(const uint32_t* planes, const void* alpha, bool alpha_f16, int64_t M, int64_t K,
                              int n_paths, int group, bool sliced, const void* dY, bool bf16, int64_t ldd, int T,
                              void* dX, int dx_dt, int64_t ldx, uint32_t* err, cudaStream_t s) {
    BwArgs a{};
    a.err = err;
    a.planes = planes;
    a.alpha = alpha;
    a.out = dX;
    a.R = M;
    a.N = T;
    a.J = K;
    a.ldo = ldx;
    a.j_tiles = static_cast<int>(K / 128);
    a.out_dt = dx_dt;
    a.sliced = sliced;
    a.alpha_f16 = alpha_f16;
    a.g128 = group == 128;
    switch (n_paths) {
        case 1: return launch_dgrad_np<1>(a, dY, ldd, bf16, s);
        case 2: return launch_dgrad_np<2>(a, dY, ldd, bf16, s);
        case 3: return launch_dgrad_np<3>(a, dY, ldd, bf16, s);
        case 4: return launch_dgrad_np<4>(a, dY, ldd, bf16, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_gemm_wgrad(const void* dY, bool bf16, int64_t ldd, int64_t M, const uint8_t* codes,
                              const float* scales, int64_t K, int T, const void* add, void* dW, int dw_dt, int64_t ldw,
                              uint32_t* err, cudaStream_t s) {
    BwArgs a{};
    a.err = err;
    a.out = dW;
    a.N = M;
    a.J = K;
    a.ldo = ldw;
    a.j_tiles = static_cast<int>(K / 128);
    a.out_dt = dw_dt;
    a.R = T;
    const int tile = bwd_tile(a, false);
    a.n_tiles = static_cast<int>((M + (tile == 256 ? 256 : std::max(tile, 64)) - 1) / (tile == 256 ? 256 : std::max(tile, 64)));
    // a split tile is summed in shared memory that its rings use before, so its
    // segments are launches of their own: as many tokens as `segment` stages of each CTA
    const int64_t nr = (static_cast<int64_t>(T) + BR - 1) / BR;
    const int split = tile == 256 ? 1 : split_of(static_cast<int64_t>(a.j_tiles) * a.n_tiles, nr);
    const bool fp32 = dw_dt == B8_F32;
    const int step = fp32 && split > 1 ? std::min(T, (bf16 ? SEGMENT_BF16 : SEGMENT_F16) * BR * split) : T;
    for (int64_t t0 = 0; t0 < T; t0 += step) {
        const int rows = static_cast<int>(std::min<int64_t>(step, T - t0));
        a.codes = codes + t0 * K;
        a.scales = scales + t0 * (K / 128);
        a.add = t0 ? dW : add;
        a.add_ahead = a.add && reinterpret_cast<uintptr_t>(a.add) % 16 == 0 && ldw * (fp32 ? 4 : 2) % 16 == 0;
        a.R = rows;
        a.first = t0 == 0;
        BwMaps m;
        // boxes of 64 m x 64 t
        cudaError_t e = make_x_map(&m.dy, static_cast<const char*>(dY) + t0 * ldd * 2, M, rows, ldd, BR);
        if (e == cudaSuccess) e = make_x8_map(&m.c, a.codes, K, rows, 1, BR);
        if (e != cudaSuccess) return e;
        plan_scales(a, 1);
        if (tile == 256) e = bf16 ? launch<WGRAD, 1, 256, true, PAIR>(m, a, 2, s) : launch<WGRAD, 1, 256, false, PAIR>(m, a, 2, s);
        else if (tile == 128) e = launch_bn<WGRAD, 1, 128>(m, a, bf16, s);
        else e = launch_bn<WGRAD, 1, 64>(m, a, bf16, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace rb
