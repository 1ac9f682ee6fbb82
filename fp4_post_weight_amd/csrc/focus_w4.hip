// focus_w4.hip -- linear layers with 4-bit weights and 8- or 16-bit
// activations on gfx950 matrix cores:
//     Y[t, o] = sum_k X[t, k] * W'[o, k]
// with X in MXFP8 (E4M3 codes, one E8M0 scale per 32) or BF16 and W' the
// value of MXFP4 codes (E2M1, one E8M0 scale per 32) or NVFP4 codes (E2M1,
// one E4M3 scale per 16, one FP32 scale per tensor, applied to the sum).
//
// How it maps onto CDNA4:
//  * MXFP8 x MXFP4 is the hardware's own block-scaled product
//    (v_mfma_scale_f32_16x16x128_f8f6f4): codes and scale bytes go in as they
//    are stored.  A lane holds one 32-block of a W row and its scale byte, and
//    two 16-element halves of the X row.  The instruction aligns the products
//    of each 8 consecutive k to the largest exponent among them and truncates
//    to 2^-13 of it (measured); the sums of those groups are binary32.
//  * BF16 activations: every c * S is exact in BF16 (at most 6 significant
//    bits), so weights are widened in registers and the product runs on
//    v_mfma_f32_16x16x32_bf16 with binary32 sums.  MXFP4's power-of-two scale
//    is an operand of the conversion (v_cvt_scalef32_pk_bf16_fp4); NVFP4's
//    takes one multiplication per weight and a packed rounding that is exact.
//
// With few tokens the layer streams W.  A workgroup owns 16 T output columns;
// its wavefronts take 512-wide k-steps in turn, each keeps the next step's W
// in registers while it multiplies the present one, and one reduction in LDS
// adds their partial tiles in order.  W is loaded in whole 128-byte lines
// (16 lanes cover one row's 256 bytes) and passes through an LDS area of the
// wavefront to reach the matrix layout, whose 16 neighbouring lanes hold 16
// different rows.  Within a step the sum is order-free: lane group g takes
// the blocks 4g..4g+3, so that its four scale bytes are one dword, selected
// by the instruction.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "focus_launch.h"
#include "focus_numerics.h"
#include "focus_w4.h"

namespace focus {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// rows of K/2 code bytes start at multiples of 8 (NVFP4) and rows of scale
// bytes at any byte
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

constexpr int kStep = 512;         // k per wavefront step
constexpr int kStageRow = 256 + 16;  // LDS bytes per staged W row

__device__ __forceinline__ uint4 ld16_a8(const uint8_t* p) {
    const u32x4 v = *reinterpret_cast<const u32x4_a8*>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint32_t ld4_a1(const uint8_t* p) { return *reinterpret_cast<const u32_a1*>(p); }

// 16 code bytes whose first code is k, of a row that ends at K (K % 16 == 0):
// absent codes are zeros.
__device__ __forceinline__ uint4 codes_until(const uint8_t* p, int64_t k, int64_t K) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k + 32 <= K) {
        v = ld16_a8(p);
    } else if (k < K) {
        const uint2 h = *reinterpret_cast<const uint2*>(p);
        v.x = h.x;
        v.y = h.y;
    }
    return v;
}

// Four scale bytes of blocks b, b+1, ... of a row of nb: absent ones are
// `one`, the byte of scale 1.
__device__ __forceinline__ uint32_t scales_until(const uint8_t* p, int64_t b, int64_t nb, uint32_t one) {
    if (b + 4 <= nb) return ld4_a1(p);
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) v |= (b + i < nb ? (uint32_t)p[i] : one) << (8 * i);
    return v;
}

template <int J>
__device__ __forceinline__ f32x4 mfma_mx(const uint4& lo, const uint4& hi, const uint4& w, uint32_t xs, uint32_t ws,
                                         f32x4 acc) {
    const i32x8 a = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    const i32x8 b = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 4, J, (int)xs, J, (int)ws);
}

__device__ __forceinline__ uint32_t pick(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Eight MXFP4 codes times the scale S (a power of two), in BF16.
__device__ __forceinline__ bf16x8 widen_mx(uint32_t c, float S) {
    const bf16x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, S, 0);
    const bf16x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, S, 1);
    const bf16x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, S, 2);
    const bf16x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, S, 3);
    return (bf16x8){a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
}

// Eight NVFP4 codes times their block's E4M3 scale, in BF16 (exact).
__device__ __forceinline__ bf16x8 widen_nv(uint32_t c, float S) {
    const f32x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f32x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    const uint4 v = make_uint4(bf16_pair(a0[0] * S, a0[1] * S), bf16_pair(a1[0] * S, a1[1] * S),
                               bf16_pair(a2[0] * S, a2[1] * S), bf16_pair(a3[0] * S, a3[1] * S));
    return __builtin_bit_cast(bf16x8, v);
}

// One wavefront step's W: 4 T row pieces as loaded, and the scale bytes of
// the lane's blocks (4 of 32 elements, or 8 of 16).
template <int KIND, int T>
struct StepW {
    uint4 c[4 * T];
    uint32_t s[T][KIND == kW4Bf16Nvfp4 ? 2 : 1];
};

template <int KIND, int T>
__device__ __forceinline__ void load_w(StepW<KIND, T>& o, const W4Args& a, int64_t n0, int64_t k0, int lane) {
    constexpr bool kNv = KIND == kW4Bf16Nvfp4;
    const int c16 = lane & 15, g = lane >> 4;
    const bool whole = k0 + kStep <= a.K;
#pragma unroll
    for (int r = 0; r < 4 * T; ++r) {
        const int64_t row = n0 + 4 * r + g;
        const int64_t k = k0 + 32 * c16;
        const uint8_t* p = a.wc + (row < a.N ? row : a.N - 1) * (a.K / 2) + k / 2;
        o.c[r] = whole ? ld16_a8(p) : codes_until(p, k, a.K);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int64_t row = n0 + 16 * t + c16;
        const int64_t rr = row < a.N ? row : a.N - 1;
        constexpr int kPer = kNv ? 8 : 4;  // scale bytes per lane
        const int64_t nb = a.K / (kNv ? 16 : 32), b = k0 / (kNv ? 16 : 32) + kPer * g;
        const uint8_t* p = a.ws + rr * nb + b;
#pragma unroll
        for (int i = 0; i < (kNv ? 2 : 1); ++i)
            o.s[t][i] = whole ? ld4_a1(p + 4 * i) : scales_until(p + 4 * i, b + 4 * i, nb, kNv ? 0x38u : 127u);
    }
}

template <int KIND, bool BF16_OUT, int WAVES, int T, int MT>
__global__ __launch_bounds__(64 * WAVES) void k_w4_decode(W4Args a, int64_t tiles_n) {
    constexpr bool kMx = KIND == kW4Mx, kNv = KIND == kW4Bf16Nvfp4;
    constexpr int kStage = WAVES * 16 * T * kStageRow;
    constexpr int kRed = WAVES * MT * T * 256 * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRed > kStage ? kRed : kStage];
    float(*red)[MT * T * 256] = reinterpret_cast<float(*)[MT * T * 256]>(lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c16 = lane & 15, g = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.x % tiles_n) * (16 * T);
    const int64_t m0 = ((int64_t)blockIdx.x / tiles_n) * (16 * MT);
    const int64_t nsteps = (a.K + kStep - 1) / kStep;

    f32x4 acc[MT][T];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[m][t] = (f32x4){};

    int64_t xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t row = m0 + 16 * m + c16;
        xrow[m] = row < a.M ? row : a.M - 1;  // such rows feed outputs that are never stored
    }
    uint8_t* st = lds + wave * (16 * T * kStageRow);
    StepW<KIND, T> w;
    if (wave < nsteps) load_w<KIND, T>(w, a, n0, (int64_t)wave * kStep, lane);
    for (int64_t s = wave; s < nsteps; s += WAVES) {
        const int64_t k0 = s * kStep;
        const bool whole = k0 + kStep <= a.K;
        uint32_t sc[T][kNv ? 2 : 1];
#pragma unroll
        for (int r = 0; r < 4 * T; ++r)
            *reinterpret_cast<uint4*>(st + (4 * r + g) * kStageRow + 16 * c16) = w.c[r];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < (kNv ? 2 : 1); ++i) sc[t][i] = w.s[t][i];
        __builtin_amdgcn_wave_barrier();
        if (s + WAVES < nsteps) load_w<KIND, T>(w, a, n0, (s + WAVES) * kStep, lane);
        if constexpr (kMx) {
            uint32_t xsc[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int64_t nb = a.K / 32, b = k0 / 32 + 4 * g;
                const uint8_t* p = a.xs + xrow[m] * nb + b;
                xsc[m] = whole ? ld4_a1(p) : scales_until(p, b, nb, 127u);
            }
            // Logical block b of product j is block 4 b + j of the step.  A
            // lane's X halves: logical k 16 g.. and 64 + 16 g.., i.e. half
            // g % 2 of logical blocks g / 2 and 2 + g / 2.
            auto product = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                uint4 wf[T];
#pragma unroll
                for (int t = 0; t < T; ++t)
                    wf[t] = *reinterpret_cast<const uint4*>(st + (16 * t + c16) * kStageRow + 64 * g + 16 * j);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int64_t k = k0 + 32 * (4 * (g >> 1) + j) + 16 * (g & 1);
                    const uint8_t* p = a.x + xrow[m] * a.K + k;
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (whole || k < a.K) lo = *reinterpret_cast<const uint4*>(p);
                    if (whole || k + 256 < a.K) hi = *reinterpret_cast<const uint4*>(p + 256);
#pragma unroll
                    for (int t = 0; t < T; ++t) acc[m][t] = mfma_mx<j>(lo, hi, wf[t], xsc[m], sc[t][0], acc[m][t]);
                }
            };
            product(std::integral_constant<int, 0>{});
            product(std::integral_constant<int, 1>{});
            product(std::integral_constant<int, 2>{});
            product(std::integral_constant<int, 3>{});
        } else {
            // product i takes k = 128 g + 8 i .. + 7 of the step in lane group g
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 wf[T];
#pragma unroll
                for (int t = 0; t < T; ++t)
                    wf[t] = *reinterpret_cast<const uint4*>(st + (16 * t + c16) * kStageRow + 64 * g + 16 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t k = k0 + 128 * g + 32 * j + 8 * i;
                    bf16x8 wb[T];
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        if (kNv) {
                            const int b = 2 * j + (i >> 1);  // the lane's 16-block
                            wb[t] = widen_nv(pick(wf[t], i), e4m3_any_value((sc[t][b >> 2 & (kNv ? 1 : 0)] >> (8 * (b & 3))) & 0xFFu));
                        } else {
                            wb[t] = widen_mx(pick(wf[t], i), e8m0_value((sc[t][0] >> (8 * j)) & 0xFFu));
                        }
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint4 xv = make_uint4(0, 0, 0, 0);
                        if (whole || k < a.K) xv = *reinterpret_cast<const uint4*>(a.x + 2 * (xrow[m] * a.K + k));
                        const bf16x8 xb = __builtin_bit_cast(bf16x8, xv);
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, wb[t], acc[m][t], 0, 0, 0);
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }

    // register r of lane l in tile (m, t): token 16 m + 4 (l / 16) + r, column
    // 16 t + l % 16.  The reduction shares LDS with the staging areas.
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][((m * T + t) * 16 + 4 * g + r) * 16 + c16] = acc[m][t][r];
    __syncthreads();
    const float s2 = kNv ? a.ws2[0] : 1.0f;
    for (int e = tid; e < MT * T * 256; e += 64 * WAVES) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += red[i][e];
        const int mt = e >> 8;
        const int64_t row = m0 + 16 * (mt / T) + ((e >> 4) & 15), col = n0 + 16 * (mt % T) + (e & 15);
        if (row < a.M && col < a.N) {
            if (kNv) v *= s2;
            if (BF16_OUT) reinterpret_cast<uint16_t*>(a.y)[row * a.N + col] = (uint16_t)(bf16_pair(v, 0.0f) & 0xFFFFu);
            else reinterpret_cast<float*>(a.y)[row * a.N + col] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// MXFP8 x MXFP4 with many tokens: tiles of BM tokens x BN columns, k in steps
// of 128, three stages in LDS.  Codes go from memory to LDS without passing
// through registers (16 bytes per lane).  Rows are stored unpadded (the
// transfer writes lane after lane) and their 16-byte pieces permuted by the
// row, so that the fragment reads of 8 rows cover all banks: X row r holds
// piece p at p ^ (r & 7) of 8, W row r at p ^ ((r >> 1) & 3) of 4; the
// transferring lane picks its global address accordingly.  The scale bytes of
// a row's step are one dword, loaded a step ahead into a register of the
// thread that owns the row.
//
// A step has two halves around its one barrier, which says that every
// wavefront has left step s - 1 and that the data of step s + 1 are in LDS.
// After it the transfer of step s + 2 starts, into the stage of s - 1, and has
// a whole step to land; the W fragments of step s + 1 and its first X
// fragments are read while the second half's products run, and X fragments
// come `kAhead` subtiles ahead of their products throughout.
//
// W is the first operand of the product, so that a lane's four accumulators
// are four neighbouring columns of one token.
// ---------------------------------------------------------------------------

constexpr int kTileK = 128;
constexpr int64_t kMaxTileK = (int64_t)1 << 23;  // a tile's offsets fit 32 bits

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
    return (uint32_t)(uintptr_t)(const lds_byte*)p;
}

// 16 bytes per lane from base + offset to LDS at `dst` + 16 * lane (dst and
// base uniform).  The instruction has no register result; it is complete
// after wait_transfers().  Written out because the compiler, which cannot tell
// the stages apart, would wait for every transfer before any LDS read.  m0
// holds nothing of the compiler's here: no other instruction of these kernels
// reads it.
__device__ __forceinline__ void to_lds16(const uint8_t* base, uint32_t offset, uint32_t dst) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2"
        :
        : "s"(dst), "v"(offset), "s"(base)
        : "memory");
}

__device__ __forceinline__ void wait_transfers() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The product of W subtile j and X subtile i, whose scales are bytes j % 4 and
// i % 4 of ws and xs.
template <int SW, int SX>
__device__ __forceinline__ f32x4 mfma_tile(const uint4& w, const uint4& lo, const uint4& hi, uint32_t ws, uint32_t xs,
                                           f32x4 acc) {
    const i32x8 a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8 b = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 0, SW, (int)ws, SX, (int)xs);
}

template <int SX>
__device__ __forceinline__ f32x4 mfma_tile(int sw, const uint4& w, const uint4& lo, const uint4& hi, uint32_t ws,
                                           uint32_t xs, f32x4 acc) {
    switch (sw & 3) {
        case 0: return mfma_tile<0, SX>(w, lo, hi, ws, xs, acc);
        case 1: return mfma_tile<1, SX>(w, lo, hi, ws, xs, acc);
        case 2: return mfma_tile<2, SX>(w, lo, hi, ws, xs, acc);
        default: return mfma_tile<3, SX>(w, lo, hi, ws, xs, acc);
    }
}

__device__ __forceinline__ f32x4 mfma_tile(int sw, int sx, const uint4& w, const uint4& lo, const uint4& hi,
                                           uint32_t ws, uint32_t xs, f32x4 acc) {
    switch (sx & 3) {
        case 0: return mfma_tile<0>(sw, w, lo, hi, ws, xs, acc);
        case 1: return mfma_tile<1>(sw, w, lo, hi, ws, xs, acc);
        case 2: return mfma_tile<2>(sw, w, lo, hi, ws, xs, acc);
        default: return mfma_tile<3>(sw, w, lo, hi, ws, xs, acc);
    }
}

// Scale byte of block g of a step, row r of an operand tile, in LDS: the bytes
// of SUB rows 16 apart (SUB subtiles of one wavefront) are neighbours, so that
// a lane reads them at once and the instruction selects one.
template <int SUB>
__device__ __forceinline__ int scale_at(int r, int g) {
    return SUB * (((r / (16 * SUB)) * 16 + (r & 15)) * 4 + g) + (r >> 4) % SUB;
}

template <int SUB>
__device__ __forceinline__ uint32_t read_scales(const uint8_t* base, int r, int g) {
    const uint8_t* p = base + scale_at<SUB>(r, g);
    if (SUB == 4) return *reinterpret_cast<const uint32_t*>(p);
    if (SUB == 2) return *reinterpret_cast<const uint16_t*>(p);
    return *p;
}

// Workgroup -> tile: workgroups are dealt to the 8 XCDs in turn, so each XCD
// takes a contiguous range of tiles, in columns of `kGroupM` token tiles, and
// its L2 holds few rows of both operands at a time.
constexpr int64_t kXcds = 8, kGroupM = 4;

struct TilePos {
    int64_t m, n;
};

__device__ __forceinline__ TilePos tile_of(int64_t bid, int64_t tiles_m, int64_t tiles_n) {
    const int64_t total = tiles_m * tiles_n;
    const int64_t q = total / kXcds, r = total % kXcds, xcd = bid % kXcds;
    const int64_t tile = xcd * q + (xcd < r ? xcd : r) + bid / kXcds;
    const int64_t group = tile / (kGroupM * tiles_n), in = tile % (kGroupM * tiles_n);
    const int64_t first = group * kGroupM;
    const int64_t gm = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
    return {first + in % gm, in / gm};
}

template <int BM, int BN, int WM, int WN, bool BF16_OUT>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_tiled(W4Args a, int64_t tiles_m, int64_t tiles_n) {
    constexpr int kThreads = 64 * WM * WN;
    constexpr int kXPieces = BM * 8 / kThreads, kWPieces = BN * 4 / kThreads;  // 16-byte pieces per thread and step
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kSubM = TM < 4 ? TM : 4, kSubN = TN < 4 ? TN : 4;
    constexpr int kAhead = TM >= 4 ? 2 : 1, kRing = 2 * kAhead;
    constexpr int kXBytes = BM * kTileK, kWBytes = BN * kTileK / 2, kSBytes = (BM + BN) * 4;
    constexpr int kStageBytes = kXBytes + kWBytes + kSBytes;
    constexpr int kScaleRows = (BM + BN + kThreads - 1) / kThreads;
    static_assert(kXPieces >= 1 && kWPieces >= 1, "every thread transfers both operands");
    static_assert(TM % kRing == 0 && TN % kSubN == 0, "fragment ring and scale groups");
    __shared__ __attribute__((aligned(128))) uint8_t lds[3 * kStageBytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g = lane >> 4;
    const TilePos pos = tile_of(blockIdx.x, tiles_m, tiles_n);
    const int64_t m0 = pos.m * BM, n0 = pos.n * BN;
    const int nsteps = (int)((a.K + kTileK - 1) / kTileK), full = (int)(a.K / kTileK);
    const int64_t nb = a.K / 32;

    // Piece i of this thread: rows in order of waves, then i.  Rows past the
    // operand's end read its last row and feed outputs that are never stored.
    // Offsets from the tile's first row fit 32 bits (K <= kMaxTileK).
    const uint8_t* xbase = a.x + m0 * a.K;
    const uint8_t* wbase = a.wc + n0 * (a.K / 2);
    uint32_t xoff[kXPieces], woff[kWPieces];
    constexpr int kXWave = kXPieces * 8, kWWave = kWPieces * 16;  // rows per wavefront
    const uint32_t K32 = (uint32_t)a.K;
    const int mlast = (int)(a.M - 1 - m0 < BM ? a.M - 1 - m0 : BM), nlast = (int)(a.N - 1 - n0 < BN ? a.N - 1 - n0 : BN);
    const int xpiece = (lane & 7) ^ (lane >> 3), wpiece = (lane & 3) ^ ((lane >> 3) & 3);
#pragma unroll
    for (int i = 0; i < kXPieces; ++i)
        xoff[i] = (uint32_t)min(wave * kXWave + 8 * i + (lane >> 3), mlast) * K32 + 16 * xpiece;
#pragma unroll
    for (int i = 0; i < kWPieces; ++i)
        woff[i] = (uint32_t)min(wave * kWWave + 16 * i + (lane >> 2), nlast) * (K32 / 2) + 16 * wpiece;
    const uint8_t* ssrc[kScaleRows];
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
        const int r = tid + kThreads * i;
        ssrc[i] = r < BM ? a.xs + (m0 + min(r, mlast)) * nb : a.ws + (n0 + min(r - BM, nlast)) * nb;
    }

    auto load_codes = [&](int s, uint8_t* st) {
        uint8_t* xd = st + wave * kXWave * kTileK;
        uint8_t* wd = st + kXBytes + wave * kWWave * (kTileK / 2);
        const uint8_t* xb = xbase + (int64_t)s * kTileK;
        const uint8_t* wb = wbase + (int64_t)s * (kTileK / 2);
        if (s < full) {
#pragma unroll
            for (int i = 0; i < kXPieces; ++i) to_lds16(xb, xoff[i], lds_address(xd + i * 8 * kTileK));
#pragma unroll
            for (int i = 0; i < kWPieces; ++i) to_lds16(wb, woff[i], lds_address(wd + i * 16 * (kTileK / 2)));
        } else {
            // the last, partial step: pieces past K are zeros
            const int left = (int)(a.K - (int64_t)s * kTileK);
#pragma unroll
            for (int i = 0; i < kXPieces; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (16 * xpiece < left) v = *reinterpret_cast<const uint4*>(xb + xoff[i]);
                *reinterpret_cast<uint4*>(xd + i * 8 * kTileK + 16 * lane) = v;
            }
#pragma unroll
            for (int i = 0; i < kWPieces; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (32 * wpiece < left) v = *reinterpret_cast<const uint4*>(wb + woff[i]);
                *reinterpret_cast<uint4*>(wd + i * 16 * (kTileK / 2) + 16 * lane) = v;
            }
        }
    };
    uint32_t sreg[kScaleRows];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < kScaleRows; ++i)
            if (kScaleRows * kThreads == BM + BN || tid + kThreads * i < BM + BN)
                sreg[i] = scales_until(ssrc[i] + 4 * s, 4 * s, nb, 127u);
    };
    auto store_scales = [&](uint8_t* st) {
#pragma unroll
        for (int i = 0; i < kScaleRows; ++i)
            if (kScaleRows * kThreads == BM + BN || tid + kThreads * i < BM + BN) {
                const int r = tid + kThreads * i;
                uint8_t* p = st + kXBytes + kWBytes;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    p[r < BM ? scale_at<kSubM>(r, b) : 4 * BM + scale_at<kSubN>(r - BM, b)] = (uint8_t)(sreg[i] >> (8 * b));
            }
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[j][i] = (f32x4){};
    const int mrow = (wave / WN) * (BM / WM), nrow = (wave % WN) * (BN / WN);
    // fragment addresses within a stage; the permutation depends on c16 alone
    const int xlo = (mrow + c16) * kTileK + 16 * (g ^ (c16 & 7)), xhi = xlo ^ 64;
    const int wat = kXBytes + (nrow + c16) * (kTileK / 2) + 16 * (g ^ ((c16 >> 1) & 3));

    struct Frags {  // of one step: W and all scales
        uint4 w[TN];
        uint32_t ws[TN / kSubN], xs[TM / kSubM];
    };
    uint4 xl[kRing], xh[kRing];
    auto read_x = [&](const uint8_t* st, int i) {
        xl[i % kRing] = *reinterpret_cast<const uint4*>(st + xlo + i * 16 * kTileK);
        xh[i % kRing] = *reinterpret_cast<const uint4*>(st + xhi + i * 16 * kTileK);
    };
    auto read_w = [&](const uint8_t* st, Frags& f) {
        const uint8_t* sc = st + kXBytes + kWBytes;
#pragma unroll
        for (int j = 0; j < TN; ++j) f.w[j] = *reinterpret_cast<const uint4*>(st + wat + j * 16 * (kTileK / 2));
#pragma unroll
        for (int j = 0; j < TN; j += kSubN) f.ws[j / kSubN] = read_scales<kSubN>(sc + 4 * BM, nrow + 16 * j + c16, g);
#pragma unroll
        for (int i = 0; i < TM; i += kSubM) f.xs[i / kSubM] = read_scales<kSubM>(sc, mrow + 16 * i + c16, g);
    };
    auto products = [&](int i, const Frags& f) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[j][i] = mfma_tile(j % kSubN, i % kSubM, f.w[j], xl[i % kRing], xh[i % kRing], f.ws[j / kSubN],
                                  f.xs[i / kSubM], acc[j][i]);
    };
    // step s with its fragments f, in stage `cur`; reads the next step's
    // fragments into n
    auto step = [&](int s, const uint8_t* cur, uint8_t* next, uint8_t* after, const Frags& f, Frags& n) {
#pragma unroll
        for (int i = 0; i < TM / 2; ++i) {
            read_x(cur, i + kAhead);
            products(i, f);
        }
        if (s + 1 < nsteps) store_scales(next);
        wait_transfers();
        __syncthreads();
        if (s + 2 < nsteps) {
            load_scales(s + 2);
            load_codes(s + 2, after);
        }
        read_w(next, n);  // past the last step: a stage's leftovers, not used
#pragma unroll
        for (int i = TM / 2; i < TM; ++i) {
            read_x(i + kAhead < TM ? cur : next, (i + kAhead) % TM);
            products(i, f);
        }
    };
    Frags f0, f1;
    uint8_t *s0 = lds, *s1 = lds + kStageBytes, *s2 = lds + 2 * kStageBytes;
    if (nsteps > 0) {
        load_scales(0);
        load_codes(0, s0);
        store_scales(s0);
        if (nsteps > 1) {
            load_scales(1);
            load_codes(1, s1);
        }
        wait_transfers();
        __syncthreads();
        read_w(s0, f0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) read_x(s0, i);
    }
    for (int s = 0; s < nsteps; s += 2) {
        step(s, s0, s1, s2, f0, f1);
        if (s + 1 < nsteps) step(s + 1, s1, s2, s0, f1, f0);
        uint8_t* t = s0;  // two steps on
        s0 = s2;
        s2 = s1;
        s1 = t;
    }

    // register r of lane l in tile (j, i): column 16 j + 4 (l / 16) + r, token
    // 16 i + l % 16
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t row = m0 + mrow + 16 * i + c16;
        if (row >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t col = n0 + nrow + 16 * j + 4 * g;
            const f32x4 v = acc[j][i];
            if (col + 3 < a.N && a.N % 4 == 0) {
                if (BF16_OUT)
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + row * a.N + col) =
                        make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
                else
                    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.y) + row * a.N + col) = v;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (col + r >= a.N) break;
                    if (BF16_OUT)
                        reinterpret_cast<uint16_t*>(a.y)[row * a.N + col + r] = (uint16_t)(bf16_pair(v[r], 0.0f) & 0xFFFFu);
                    else
                        reinterpret_cast<float*>(a.y)[row * a.N + col + r] = v[r];
                }
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, bool BF16_OUT>
hipError_t run_tiled(const W4Args& a, hipStream_t stream) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    return launch(&k_mx_tiled<BM, BN, WM, WN, BF16_OUT>, dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WM * WN), stream, a,
                  tiles_m, tiles_n);
}

template <int KIND, bool BF16_OUT, int MT>
hipError_t run_decode(const W4Args& args, hipStream_t stream) {
    constexpr int kWaves = 8, kT = 1;
    const int64_t tiles_n = (args.N + 16 * kT - 1) / (16 * kT);
    // runs of token tiles whose grid stays within 2^31 threads
    const int64_t most = (((int64_t)1 << 31) / (64 * kWaves)) / tiles_n;
    if (most < 1) return hipErrorInvalidValue;
    for (int64_t row = 0; row < args.M; row += most * 16 * MT) {
        W4Args a = args;
        a.M = args.M - row < most * 16 * MT ? args.M - row : most * 16 * MT;
        a.x += row * a.K * (KIND == kW4Mx ? 1 : 2);
        if (KIND == kW4Mx) a.xs += row * (a.K / 32);
        a.y = reinterpret_cast<uint8_t*>(a.y) + row * a.N * (BF16_OUT ? 2 : 4);
        const int64_t tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
        const hipError_t e = launch(&k_w4_decode<KIND, BF16_OUT, kWaves, kT, MT>, dim3((unsigned)(tiles_m * tiles_n)),
                                    dim3(64 * kWaves), stream, a, tiles_n);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int KIND, bool BF16_OUT>
hipError_t pick_decode(const W4Args& a, hipStream_t stream) {
    if (a.M <= 16) return run_decode<KIND, BF16_OUT, 1>(a, stream);
    if (KIND == kW4Mx && a.M > 64 && a.K <= kMaxTileK) return run_tiled<256, 256, 2, 4, BF16_OUT>(a, stream);
    return run_decode<KIND, BF16_OUT, 2>(a, stream);
}

}  // namespace

hipError_t launch_w4_linear(const W4Args& a, W4Kind kind, bool bf16_out, hipStream_t stream) {
    switch (kind) {
        case kW4Mx: return bf16_out ? pick_decode<kW4Mx, true>(a, stream) : pick_decode<kW4Mx, false>(a, stream);
        case kW4Bf16Nvfp4:
            return bf16_out ? pick_decode<kW4Bf16Nvfp4, true>(a, stream) : pick_decode<kW4Bf16Nvfp4, false>(a, stream);
        case kW4Bf16Mxfp4:
            return bf16_out ? pick_decode<kW4Bf16Mxfp4, true>(a, stream) : pick_decode<kW4Bf16Mxfp4, false>(a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace focus
