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
//    to 2^-13 of it (measured); the sums of those groups are binary32.  A BF16
//    result takes that: on ordinary activations it is 1.2e-5 of the result, and
//    the rounding to BF16 1.7e-3.  For an FP32 result the X codes go through the
//    instruction in two parts (codes_part) and no product loses a bit: 2e-8 of
//    the result, that of a binary32 sum.  Measured for FP32 results, two parts
//    against one, us: 1 x 4096 x 14336 9.1 and 8.9, 8 x 14336 x 4096 10.5 and 8.4,
//    100 x 14336 x 4096 21.6 and 15.0, 8192 x 14336 x 4096 708 and 407.
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
// by the instruction.  Measured: 1 x 4096 x 14336 of NVFP4 9.6 us (3.5 TB/s; a large
// copy reaches 4.9), 1 x 4096 x 4096 of MXFP8 x MXFP4 3.4-4.0 (a launch and two
// memory latencies).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "focus_gemm.h"
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
__device__ __forceinline__ uint4 codes_until(const uint8_t* p, int k, int K) {
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
__device__ __forceinline__ uint32_t scales_until(const uint8_t* p, int b, int nb, uint32_t one) {
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

// Part P of 16 E4M3 codes in PARTS: of 2, part 0 keeps those of magnitude 2 and
// above (bit 6; NaN among them) and part 1 the rest, with zeros elsewhere.  The
// exponents are then at most 8 and at least 1, or at most 0 with a last bit of
// at least 2^-9; E2M1's are at most 2 with a last bit of at least 2^-1.  So every
// product is a multiple of 2^-3 where the exponent sums are at most 10, and of
// 2^-10 where they are at most 2: nothing lies below 2^-13 of the largest.
template <int PARTS, int P>
__device__ __forceinline__ uint4 codes_part(const uint4& v) {
    if constexpr (PARTS == 1) {
        return v;
    } else {
        auto one = [](uint32_t c) {
            const uint32_t b = (c >> 6) & 0x01010101u, m = (b << 8) - b;
            return P == 0 ? c & m : c & ~m;
        };
        return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
    }
}

// Calls f(part number) for each of PARTS.
template <int PARTS, typename F>
__device__ __forceinline__ void for_parts(F f) {
    f(std::integral_constant<int, 0>{});
    if constexpr (PARTS == 2) f(std::integral_constant<int, 1>{});
}

__device__ __forceinline__ uint32_t pick(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// E4M3 and E8M0 (0..254) scale values of the low byte of v.
__device__ __forceinline__ float e4m3_f32(uint32_t v) { return __builtin_amdgcn_cvt_f32_fp8((int)v, 0); }
__device__ __forceinline__ float e8m0_f32(uint32_t v) { return __uint_as_float(max((v & 0xFFu) << 23, 0x00400000u)); }

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

// Loads take a uniform address and a 32-bit offset of the lane (K <= kMaxW4K,
// and a workgroup has at most 32 tokens and 64 columns).  MASK: the last step, of which only
// the first `left` < kStep values of k exist.

// One wavefront step's W: 4 T row pieces as loaded, and the scale bytes of
// the lane's blocks (4 of 32 elements, or 8 of 16).
template <int KIND, int T>
struct StepW {
    static constexpr bool kNv = KIND == kW4Bf16Nvfp4;
    static constexpr int kDwords = kNv ? 2 : 1;  // of scale bytes per lane
    uint4 c[4 * T];
    uint32_t s[T][kDwords];

    template <bool MASK>
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, const uint32_t (&coff)[4 * T],
                                         const uint32_t (&soff)[T], int left, int lane) {
#pragma unroll
        for (int r = 0; r < 4 * T; ++r) c[r] = MASK ? codes_until(codes + coff[r], 32 * (lane & 15), left) : ld16_a8(codes + coff[r]);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < kDwords; ++i)
                s[t][i] = MASK ? scales_until(scales + soff[t] + 4 * i, 4 * (kDwords * (lane >> 4) + i), left / (kNv ? 16 : 32),
                                              kNv ? 0x38u : 127u)
                               : ld4_a1(scales + soff[t] + 4 * i);
    }
};

// X fragments of a quarter step (quarter j: the lane's W piece j, 32 codes):
// 2 pieces of 16 bytes per token tile for MXFP8, 4 for BF16.
//
// MXFP8: logical block b of product j is block 4 b + j of the step.  A lane's
// halves of the X row are logical k 16 g.. and 64 + 16 g.., i.e. half g % 2 of
// logical blocks g / 2 and 2 + g / 2.  BF16: product 4 j + i takes
// k = 128 g + 32 j + 8 i .. + 7 in lane group g.
template <int KIND, int MT>
struct QuarterX {
    static constexpr bool kMx = KIND == kW4Mx;
    static constexpr int kPieces = kMx ? 2 : 4, kEach = kMx ? 256 : 8;  // k from piece to piece
    uint4 v[MT][kPieces];

    // the lane's first k within a step
    static __device__ __forceinline__ int first(int g) { return kMx ? 128 * (g >> 1) + 16 * (g & 1) : 128 * g; }

    // off: of the row, plus the lane's first k, in bytes
    template <bool MASK>
    __device__ __forceinline__ void load(const uint8_t* x, const uint32_t (&off)[MT], int j, int left, int g) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (MASK) v[m][i] = make_uint4(0, 0, 0, 0);
                if (!MASK || first(g) + 32 * j + kEach * i < left)
                    v[m][i] = *reinterpret_cast<const uint4*>(x + off[m] + (kMx ? 1 : 2) * (32 * j + kEach * i));
            }
    }
};

template <int KIND, bool BF16_OUT, int WAVES, int T, int MT>
__global__ __launch_bounds__(64 * WAVES) void k_w4_decode(W4Args a, int64_t tiles_n) {
    constexpr bool kMx = KIND == kW4Mx, kNv = KIND == kW4Bf16Nvfp4;
    constexpr int kParts = BF16_OUT ? 1 : 2;
    constexpr int kScaleDwords = StepW<KIND, T>::kDwords;
    constexpr int kStage = WAVES * 16 * T * kStageRow;
    constexpr int kRed = WAVES * MT * T * 256 * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRed > kStage ? kRed : kStage];
    float(*red)[MT * T * 256] = reinterpret_cast<float(*)[MT * T * 256]>(lds);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.x % tiles_n) * (16 * T);
    const int64_t m0 = ((int64_t)blockIdx.x / tiles_n) * (16 * MT);
    const int K = (int)a.K, full = K / kStep;

    f32x4 acc[MT][T];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[m][t] = (f32x4){};

    // Rows past an operand's end read its last row and feed outputs that are
    // never stored.
    const int mlast = (int)(a.M - 1 - m0 < 16 * MT ? a.M - 1 - m0 : 16 * MT);
    const int nlast = (int)(a.N - 1 - n0 < 16 * T ? a.N - 1 - n0 : 16 * T);
    const int nb = K / (kNv ? 16 : 32);
    const uint8_t* xb = a.x + m0 * K * (kMx ? 1 : 2);
    const uint8_t* xsb = a.xs + m0 * nb;
    const uint8_t* wb = a.wc + n0 * (K / 2);
    const uint8_t* wsb = a.ws + n0 * nb;
    uint32_t xoff[MT], xsoff[MT], coff[4 * T], soff[T];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const uint32_t row = (uint32_t)min(16 * m + c16, mlast);
        xoff[m] = (row * (uint32_t)K + QuarterX<KIND, MT>::first(g)) * (kMx ? 1 : 2);
        xsoff[m] = row * (uint32_t)nb + 4 * g;
    }
#pragma unroll
    for (int r = 0; r < 4 * T; ++r) coff[r] = (uint32_t)min(4 * r + g, nlast) * (uint32_t)(K / 2) + 16 * c16;
#pragma unroll
    for (int t = 0; t < T; ++t) soff[t] = (uint32_t)min(16 * t + c16, nlast) * (uint32_t)nb + (kNv ? 8 : 4) * g;

    uint8_t* st = lds + wave * (16 * T * kStageRow);
    StepW<KIND, T> w;
    QuarterX<KIND, MT> x0, x1;
    uint32_t sc[T][kScaleDwords], xsc[MT], xsn[MT];

    auto load_w = [&](int s) {
        w.template load<false>(wb + (int64_t)s * (kStep / 2), wsb + s * (kStep / (kNv ? 16 : 32)), coff, soff, 0, lane);
        if (kMx) {
#pragma unroll
            for (int m = 0; m < MT; ++m) xsn[m] = ld4_a1(xsb + s * (kStep / 32) + xsoff[m]);
        }
    };
    auto xat = [&](int s) { return xb + (int64_t)s * kStep * (kMx ? 1 : 2); };
    // W in registers -> the wavefront's LDS area, scales -> sc, xsc
    auto stage_w = [&]() {
#pragma unroll
        for (int r = 0; r < 4 * T; ++r) *reinterpret_cast<uint4*>(st + (4 * r + g) * kStageRow + 16 * c16) = w.c[r];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < kScaleDwords; ++i) sc[t][i] = w.s[t][i];
#pragma unroll
        for (int m = 0; m < MT; ++m) xsc[m] = xsn[m];
        __builtin_amdgcn_wave_barrier();
    };
    auto products = [&](auto jc, const QuarterX<KIND, MT>& x) {
        constexpr int j = decltype(jc)::value;
        uint4 wf[T];
#pragma unroll
        for (int t = 0; t < T; ++t)
            wf[t] = *reinterpret_cast<const uint4*>(st + (16 * t + c16) * kStageRow + 64 * g + 16 * j);
        if constexpr (kMx) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                for_parts<kParts>([&](auto pc) {
                    constexpr int p = decltype(pc)::value;
                    const uint4 lo = codes_part<kParts, p>(x.v[m][0]), hi = codes_part<kParts, p>(x.v[m][1]);
#pragma unroll
                    for (int t = 0; t < T; ++t) acc[m][t] = mfma_mx<j>(lo, hi, wf[t], xsc[m], sc[t][0], acc[m][t]);
                });
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    // the lane's 16-block 2 j + i / 2, or 32-block j
                    const uint32_t byte = kNv ? sc[t][kNv ? j >> 1 : 0] >> (8 * (2 * (j & 1) + (i >> 1))) : sc[t][0] >> (8 * j);
                    const bf16x8 wv = kNv ? widen_nv(pick(wf[t], i), e4m3_f32(byte))
                                          : widen_mx(pick(wf[t], i), e8m0_f32(byte));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, x.v[m][kMx ? 0 : i]), wv, acc[m][t], 0, 0, 0);
                }
        }
    };
    constexpr std::integral_constant<int, 0> q0{};
    constexpr std::integral_constant<int, 1> q1{};
    constexpr std::integral_constant<int, 2> q2{};
    constexpr std::integral_constant<int, 3> q3{};

    if (wave < full) {
        load_w(wave);
        x0.template load<false>(xat(wave), xoff, 0, 0, g);
    }
    for (int s = wave; s < full; s += WAVES) {
        const int sn = s + WAVES < full ? s + WAVES : s;  // the last step loads itself again
        stage_w();
        load_w(sn);
        x1.template load<false>(xat(s), xoff, 1, 0, g);
        products(q0, x0);
        x0.template load<false>(xat(s), xoff, 2, 0, g);
        products(q1, x1);
        x1.template load<false>(xat(s), xoff, 3, 0, g);
        products(q2, x0);
        x0.template load<false>(xat(sn), xoff, 0, 0, g);
        products(q3, x1);
        __builtin_amdgcn_wave_barrier();
    }
    const int left = K - full * kStep;
    if (left > 0 && wave == full % WAVES) {
        w.template load<true>(wb + (int64_t)full * (kStep / 2), wsb + full * (kStep / (kNv ? 16 : 32)), coff, soff, left, lane);
        if (kMx) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                xsn[m] = scales_until(xsb + full * (kStep / 32) + xsoff[m], 4 * g, left / 32, 127u);
        }
        stage_w();
        x0.template load<true>(xat(full), xoff, 0, left, g);
        products(q0, x0);
        x0.template load<true>(xat(full), xoff, 1, left, g);
        products(q1, x0);
        x0.template load<true>(xat(full), xoff, 2, left, g);
        products(q2, x0);
        x0.template load<true>(xat(full), xoff, 3, left, g);
        products(q3, x0);
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

// The call restricted to at most `most` token rows from `row` on.
template <int KIND, bool BF16_OUT>
W4Args rows_from(const W4Args& args, int64_t row, int64_t most) {
    W4Args a = args;
    a.M = args.M - row < most ? args.M - row : most;
    a.x += row * a.K * (KIND == kW4Mx ? 1 : 2);
    if (KIND == kW4Mx) a.xs += row * (a.K / 32);
    a.y = reinterpret_cast<uint8_t*>(a.y) + row * a.N * (BF16_OUT ? 2 : 4);
    return a;
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of BM tokens x BN columns, k in steps of KS, a ring of
// stages in LDS.  Codes go from memory to LDS without passing through registers
// (16 bytes per lane).  Rows are stored unpadded (the transfer writes lane after
// lane) and their 16-byte pieces permuted by the row, so that the fragment
// reads of neighbouring rows cover all banks: piece p of row r lies at
// p ^ (r mod the row's pieces, at most 16), in a 64-byte W row at
// p ^ ((r >> 1) & 3); the transferring lane picks its global address
// accordingly.
//
// STAGES > 0: K is a multiple of KS, the scale bytes are transferred likewise, 4
// per lane, and a wavefront waits by count, so that STAGES - 2 steps are under
// way.  STAGES = 0: any K; three stages, the scale bytes of a row's step loaded a
// step ahead into a register of the thread that owns the row, and a last step
// begun only is filled up with zeros.  W_REG (NVFP4 with K % 32 == 16, whose rows
// of codes start at multiples of 8 bytes): W comes by registers too, a step ahead.
//
// A step has two halves around its one barrier, which says that every
// wavefront has left step s - 1 and that the data of step s + 1 are in LDS.
// After it the next transfer starts, into the stage of s - 1; the W fragments of
// step s + 1 and its first X fragments are read while the second half's products
// run, and X fragments come `kAhead` subtiles ahead of their products throughout.
//
// Small tiles give each SIMD too little to hide those reads behind.  They take
// long steps, and WK wavefronts share an output tile: each multiplies 1 / WK of
// every step, and at the end the first adds the others' sums in order.
//
// W is the first operand of the product, so that a lane's four accumulators
// are four neighbouring columns of one token.
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
    return (uint32_t)(uintptr_t)(const lds_byte*)p;
}

// 16 bytes per lane from base + offset to LDS at `dst` + 16 * lane (dst and
// base uniform).  The instruction has no register result, and its address
// registers are read when it issues; it is complete after wait_transfers<0>().
// Written out because the compiler, which cannot tell the stages apart, would
// wait for every transfer before any LDS read.  m0 is named as overwritten: the
// compiler reserves it, sets it where an instruction of its own reads it, and so
// never has such a pair around this one (it warns of any reserved register here).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds16(const uint8_t* base, uint32_t offset, uint32_t dst) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2"
        :
        : "s"(dst), "v"(offset), "s"(base)
        : "memory", "m0");
}

// 4 bytes per lane, likewise; to `dst` + 4 * lane.
__device__ __forceinline__ void to_lds4(const uint8_t* base, uint32_t offset, uint32_t dst) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, %2"
        :
        : "s"(dst), "v"(offset), "s"(base)
        : "memory", "m0");
}

#pragma clang diagnostic pop

// All but this wavefront's last N have landed (they do so in order).
template <int N>
__device__ __forceinline__ void wait_transfers() {
    static_assert(N <= 63, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The block-scaled product of W subtile j and X subtile i, whose scales are
// bytes SW and SX of ws and xs.
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
    switch (sw) {
        case 0: return mfma_tile<0, SX>(w, lo, hi, ws, xs, acc);
        case 1: return mfma_tile<1, SX>(w, lo, hi, ws, xs, acc);
        case 2: return mfma_tile<2, SX>(w, lo, hi, ws, xs, acc);
        default: return mfma_tile<3, SX>(w, lo, hi, ws, xs, acc);
    }
}

__device__ __forceinline__ f32x4 mfma_tile(int sw, int sx, const uint4& w, const uint4& lo, const uint4& hi,
                                           uint32_t ws, uint32_t xs, f32x4 acc) {
    switch (sx) {
        case 0: return mfma_tile<0>(sw, w, lo, hi, ws, xs, acc);
        case 1: return mfma_tile<1>(sw, w, lo, hi, ws, xs, acc);
        case 2: return mfma_tile<2>(sw, w, lo, hi, ws, xs, acc);
        default: return mfma_tile<3>(sw, w, lo, hi, ws, xs, acc);
    }
}

// Where the scale bytes of a step lie, KS == 128 and MXFP8 with wavefront tiles
// of whole groups of 4 subtiles: block g of row r.  The bytes of 4 rows 16
// apart are neighbours, so that a lane reads 4 subtiles' scales at once and
// the instruction selects one.  (Otherwise a row's bytes stay together.)
__device__ __forceinline__ int scale_at(int r, int g) { return 4 * (((r >> 6) * 16 + (r & 15)) * 4 + g) + ((r >> 4) & 3); }

// Workgroup -> tile: workgroups are dealt to the 8 XCDs in turn, so each XCD
// takes a contiguous range of tiles, in columns of `kGroupM` token tiles, and
// its L2 holds few rows of both operands at a time.
constexpr uint32_t kXcds = 8, kGroupM = 4;

struct TilePos {
    int64_t m, n;
};

__device__ __forceinline__ TilePos tile_of(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n) {
    const uint32_t total = tiles_m * tiles_n;
    const uint32_t q = total / kXcds, r = total % kXcds, xcd = bid % kXcds;
    const uint32_t tile = xcd * q + (xcd < r ? xcd : r) + bid / kXcds;
    const uint32_t full = tiles_m / kGroupM * tiles_n;  // columns of kGroupM tiles
    if (tile / kGroupM < full) {
        const uint32_t c = tile / kGroupM;
        return {(int64_t)(c / tiles_n) * kGroupM + tile % kGroupM, c % tiles_n};
    }
    const uint32_t in = tile - full * kGroupM, gm = tiles_m % kGroupM;
    return {(int64_t)(tiles_m - gm) + in % gm, in / gm};
}

// The W row of a wavefront's columns that lies at position t of them.  For BF16
// results (PAIR) a lane's accumulators of two subtiles are then 8 neighbouring
// columns, and 4 lanes write 64 bytes in a row; 32-bit results do that as it is.
template <bool PAIR>
__device__ __forceinline__ int w_row(int t) {
    return PAIR ? (t & ~31) | (t & 12) << 1 | (t >> 2 & 4) | (t & 3) : t;
}

// Stores a wavefront's accumulators: register r of lane (c16, g) in acc[j][i] is
// column n0 + 16 j + 4 g + r of token m0 + 16 i (m0 includes c16), or with PAIR
// column n0 + 32 (j / 2) + 8 g + 4 (j % 2) + r.  wide: a lane's columns are
// aligned in y and all present or all absent; whole: all of it is in range.  The
// stores are ordinary ones: the L2 joins lines that a wavefront writes in parts
// (rows of 18000 bytes, 5000 x 9000 x 640 of MXFP8: 39 us against 72 with stores
// past the caches; rows of 28672 bytes, 8192 x 14336 x 4096, the same within 1 %).
template <int TM, int TN, bool BF16_OUT, bool PAIR>
__device__ __forceinline__ void store_tile(f32x4 (&acc)[TN][TM], const W4Args& a, int64_t m0, int64_t n0, int g, float s2,
                                           bool wide, bool whole) {
    constexpr int C = PAIR ? 2 : 1;  // subtiles per store
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t row = m0 + 16 * i;
        if (!whole && row >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TN; j += C) {
            const int64_t col = n0 + 16 * j + 4 * C * g;
            f32x4 v[C];
#pragma unroll
            for (int b = 0; b < C; ++b) v[b] = acc[j + b][i] * s2;
            if (whole || (wide && col < a.N)) {
                uint16_t* const h = reinterpret_cast<uint16_t*>(a.y) + row * a.N + col;
                if constexpr (PAIR) {
                    const u32x4 p = {bf16_pair(v[0][0], v[0][1]), bf16_pair(v[0][2], v[0][3]),
                                     bf16_pair(v[C - 1][0], v[C - 1][1]), bf16_pair(v[C - 1][2], v[C - 1][3])};
                    *reinterpret_cast<u32x4*>(h) = p;
                } else if constexpr (BF16_OUT) {
                    *reinterpret_cast<uint2*>(h) = make_uint2(bf16_pair(v[0][0], v[0][1]), bf16_pair(v[0][2], v[0][3]));
                } else {
                    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.y) + row * a.N + col) = v[0];
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4 * C; ++r) {
                    if (col + r >= a.N) break;
                    if constexpr (BF16_OUT)
                        reinterpret_cast<uint16_t*>(a.y)[row * a.N + col + r] =
                            (uint16_t)(bf16_pair(v[r / 4][r % 4], 0.0f) & 0xFFFFu);
                    else
                        reinterpret_cast<float*>(a.y)[row * a.N + col + r] = v[0][r];
                }
            }
        }
    }
}

// store_tile's `wide`
template <bool BF16_OUT, bool PAIR>
__device__ __forceinline__ bool wide_rows(const W4Args& a) {
    return a.N % (PAIR ? 8 : 4) == 0 && ((uintptr_t)a.y & (BF16_OUT && !PAIR ? 7 : 15)) == 0;
}

template <int KIND, int KS, int BM, int BN, int WM, int WN, int WK, int STAGES, bool BF16_OUT, bool W_REG>
__global__ __launch_bounds__(64 * WM * WN * WK) void k_w4_tiled(W4Args a, uint32_t tiles_m, uint32_t tiles_n) {
    constexpr bool kMx = KIND == kW4Mx, kNv = KIND == kW4Bf16Nvfp4;
    constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
    constexpr int kParts = BF16_OUT ? 1 : 2;                                      // of X, for MXFP8
    constexpr bool kDirect = STAGES > 0;                                          // whole steps; scales transferred too
    constexpr int kStages = kDirect ? STAGES : 3;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;                          // 16 x 16 subtiles per wavefront
    constexpr int kXRow = kMx ? KS : 2 * KS, kWRow = KS / 2;                     // bytes of a row's step
    constexpr int kXPer = kXRow / 16, kWPer = kWRow / 16;                        // 16-byte pieces of it
    constexpr int kXMask = kXPer < 16 ? kXPer - 1 : 15, kWMask = kWPer < 16 ? kWPer - 1 : 15;
    constexpr int kXInst = BM * kXRow / 1024 / kWaves, kWInst = BN * kWRow / 1024 / kWaves;  // transfers per wavefront
    constexpr int kBlock = kNv ? 16 : 32, kSb = KS / kBlock;                     // scale bytes of a row's step
    constexpr int kSRows = (kMx ? BM : 0) + BN;                                  // rows that have scales
    constexpr int kXBytes = BM * kXRow, kWBytes = BN * kWRow, kSInst = kDirect ? (kSRows * kSb + 256 * kWaves - 1) / (256 * kWaves) : 0;
    constexpr int kStageBytes = kXBytes + kWBytes + (kDirect ? kSInst * kWaves * 256 : kSRows * kSb);
    constexpr int KW = KS / WK;                                                  // k of a step per wavefront
    constexpr int NJ = KW >= 128 ? KW / 128 : 1;                                 // W pieces per lane and subtile
    constexpr int NP = kMx ? 2 * NJ : KW / 32;                                   // X pieces per lane and subtile
    constexpr bool kGroup = !kDirect && kMx && KS == 128 && TM % 4 == 0 && TN % 4 == 0;      // scale_at
    constexpr int kLaneSb = kMx ? NJ : (kSb / WK >= 4 ? kSb / WK / 4 : 1);                 // scale bytes per lane and subtile
    constexpr bool kPair = BF16_OUT && TN % 2 == 0;
    constexpr int kAhead = NP <= 4 && TM >= 4 ? 2 : 1, kRing = 2 * kAhead;
    static_assert(kMx ? KW % 128 == 0 && KW <= 512 : KW == 64 || KW == 128 || KW == 256, "k per step");
    static_assert(BM * kXRow % (1024 * kWaves) == 0 && BN * kWRow % (1024 * kWaves) == 0, "every wavefront transfers alike");
    static_assert((kDirect || kSRows <= kThreads) && TM % kRing == 0, "one row's scales per thread; fragment ring");
    static_assert(!kDirect || ((!kMx || BM * kSb % 256 == 0) && kStages >= 3), "a transfer of scales is of one operand");
    static_assert(WK == 1 || (kDirect && KW >= 128), "a wavefront's part of a step");
    static_assert(!W_REG || (kNv && !kDirect), "codes in registers");
    static_assert((WK - 1) * BM * BN * 4 <= kStages * kStageBytes, "room for partial sums");
    constexpr int kInst = kXInst + kWInst + kSInst;
    __shared__ __attribute__((aligned(256))) uint8_t lds[kStages * kStageBytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g = lane >> 4;
    const TilePos pos = tile_of(blockIdx.x, tiles_m, tiles_n);
    const int64_t m0 = pos.m * BM, n0 = pos.n * BN;
    const int K = (int)a.K, full = K / KS, nsteps = (K + KS - 1) / KS;
    const int nb = K / kBlock;

    // Sources of this lane's transfers, as offsets from the tile's first row
    // (32 bits: K <= kMaxW4K).  Rows past the operand's end read its last row
    // and feed outputs that are never stored.
    const uint8_t* xbase = a.x + m0 * K * (kMx ? 1 : 2);
    const uint8_t* wbase = a.wc + n0 * (K / 2);
    const int mlast = (int)(a.M - 1 - m0 < BM ? a.M - 1 - m0 : BM), nlast = (int)(a.N - 1 - n0 < BN ? a.N - 1 - n0 : BN);
    uint32_t xoff[kXInst], woff[kWInst];
    int xpiece[kXInst], wpiece[kWInst];
#pragma unroll
    for (int i = 0; i < kXInst; ++i) {
        const int row = (wave * kXInst + i) * 64 / kXPer + lane / kXPer;
        xpiece[i] = (lane % kXPer) ^ (row & kXMask);
        xoff[i] = (uint32_t)min(row, mlast) * (uint32_t)(K * (kMx ? 1 : 2)) + 16 * xpiece[i];
    }
    // Direct: transfers whose rows are all behind the last token are left out;
    // what LDS holds there feeds outputs that are never stored.
    int nx = kXInst;
    if (kDirect) {
        const int rows = 64 / kXPer > 0 ? 64 / kXPer : 1;
        nx = min(max((mlast / rows + 1) - wave * kXInst, 0), kXInst);
    }
    auto wperm = [](int r) { return kWPer == 2 ? 0 : kWPer == 4 ? (r >> 1) & 3 : r & kWMask; };
#pragma unroll
    for (int i = 0; i < kWInst; ++i) {
        const int row = (wave * kWInst + i) * 64 / kWPer + lane / kWPer;
        wpiece[i] = (lane % kWPer) ^ wperm(row);
        woff[i] = (uint32_t)min(w_row<kPair>(row), nlast) * (uint32_t)(K / 2) + 16 * wpiece[i];
    }
    // Scales, X rows first.  Transferred 4 bytes per lane (K % KS == 0, so that a
    // row's bytes start at multiples of 4), lanes behind the last row as the last;
    uint32_t soff[kSInst > 0 ? kSInst : 1];
    if (kDirect) {
#pragma unroll
        for (int i = 0; i < kSInst; ++i) {
            const int at = ((wave * kSInst + i) * 64 + lane) * 4, row = at / kSb;
            soff[i] = (uint32_t)(kMx && row < BM ? min(row, mlast) : min(w_row<kPair>(min(row - (kMx ? BM : 0), BN - 1)), nlast)) * (uint32_t)nb + at % kSb;
        }
    }
    // or loaded by the thread that owns the row
    const int srow = kMx && tid < BM ? min(tid, mlast) : min(w_row<kPair>(tid - (kMx ? BM : 0)), nlast);
    const uint8_t* ssrc = kMx && tid < BM ? a.xs + (m0 + srow) * nb : a.ws + (n0 + srow) * nb;
    constexpr int kSDwords = (kSb + 3) / 4;
    uint32_t sreg[kSDwords];
    uint4 wreg[W_REG ? kWInst : 1];

    auto load = [&](int s, uint8_t* st) {
        if (!kDirect && (kSRows == kThreads || tid < kSRows)) {
            const uint8_t* p = ssrc + s * kSb;
#pragma unroll
            for (int i = 0; i < kSDwords; ++i) {
                if (kSb >= 4) {
                    sreg[i] = s < full ? ld4_a1(p + 4 * i) : scales_until(p + 4 * i, s * kSb + 4 * i, nb, kNv ? 0x38u : 127u);
                } else {  // two blocks; K % 32 == 0, so an absent one is the second
                    sreg[i] = p[0] | (uint32_t)(s < full || s * kSb + 1 < nb ? p[1] : 127) << 8;
                }
            }
        }
        uint8_t* xd = st + wave * kXInst * 1024;
        uint8_t* wd = st + kXBytes + wave * kWInst * 1024;
        const uint8_t* xb = xbase + (int64_t)s * kXRow;
        const uint8_t* wb = wbase + (int64_t)s * kWRow;
        if (kDirect) {
#pragma unroll
            for (int i = 0; i < kSInst; ++i) {
                const int at = (wave * kSInst + i) * 256;
                const uint8_t* sb = kMx && at < BM * kSb ? a.xs + m0 * nb : a.ws + n0 * nb;
                to_lds4(sb + (int64_t)s * kSb, soff[i], lds_address(st + kXBytes + kWBytes + at));
            }
        }
        if constexpr (W_REG) {
#pragma unroll
            for (int i = 0; i < kWInst; ++i)
                wreg[i] = s < full ? ld16_a8(wb + woff[i]) : codes_until(wb + woff[i], 32 * wpiece[i], K - s * KS);
        }
        if (kDirect || s < full) {
#pragma unroll
            for (int i = 0; i < kXInst; ++i)
                if (i < nx) to_lds16(xb, xoff[i], lds_address(xd + i * 1024));
#pragma unroll
            for (int i = 0; i < (W_REG ? 0 : kWInst); ++i) to_lds16(wb, woff[i], lds_address(wd + i * 1024));
        } else {
            // the last, partial step: pieces past K are zeros
            const int left = K - s * KS;
#pragma unroll
            for (int i = 0; i < kXInst; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if ((kMx ? 16 : 8) * xpiece[i] < left) v = *reinterpret_cast<const uint4*>(xb + xoff[i]);
                *reinterpret_cast<uint4*>(xd + i * 1024 + 16 * lane) = v;
            }
#pragma unroll
            for (int i = 0; i < (W_REG ? 0 : kWInst); ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (32 * wpiece[i] < left) v = *reinterpret_cast<const uint4*>(wb + woff[i]);
                *reinterpret_cast<uint4*>(wd + i * 1024 + 16 * lane) = v;
            }
        }
    };
    // what `load` left in registers
    auto store_regs = [&](uint8_t* st) {
        uint8_t* p = st + kXBytes + kWBytes;
        if (kDirect) return;
        if constexpr (W_REG) {
#pragma unroll
            for (int i = 0; i < kWInst; ++i)
                *reinterpret_cast<uint4*>(st + kXBytes + (wave * kWInst + i) * 1024 + 16 * lane) = wreg[i];
        }
        if (kSRows == kThreads || tid < kSRows) {
            if (kGroup) {  // BM % 64 == 0
#pragma unroll
                for (int b = 0; b < 4; ++b) p[scale_at(tid, b)] = (uint8_t)(sreg[0] >> (8 * b));
            } else if (kSb >= 4) {
#pragma unroll
                for (int i = 0; i < kSDwords; ++i) reinterpret_cast<uint32_t*>(p + tid * kSb)[i] = sreg[i];
            } else {
                *reinterpret_cast<uint16_t*>(p + tid * kSb) = (uint16_t)sreg[0];
            }
        }
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[j][i] = (f32x4){};
    const int kz = WK == 1 ? 0 : wave / (WM * WN), tile_wave = WK == 1 ? wave : wave % (WM * WN);
    const int mrow = (tile_wave / WN) * (BM / WM), nrow = (tile_wave % WN) * (BN / WN);
    // Fragment addresses within a stage; the permutations depend on c16 alone.
    // MXFP8, product j of NJ: logical block b is block NJ b + j of the step; the
    // lane's W piece is that of logical block g, its X halves are half g % 2 of
    // logical blocks g / 2 and 2 + g / 2.  BF16: the lane takes k = KS/4 g ..
    // of the step, 8 per product.  Every index below is an XOR of disjoint bits.
    const int xat = (mrow + c16) * kXRow + 16 * ((kz * (kXPer / WK) + (kMx ? 2 * NJ * (g >> 1) + (g & 1) : NP * g)) ^ (c16 & kXMask));
    const int wat = kXBytes + (nrow + c16) * kWRow + (kWPer == 2 ? 8 * g : 16 * ((kz * (kWPer / WK) + NJ * g) ^ wperm(c16)));
    auto xpart = [](int q) { return kMx ? 32 * (q >> 1) ^ (q & 1) * 64 * NJ : 16 * q; };  // MXFP8: q = 2 j + half

    struct Frags {  // of one step: W as stored, and all scales
        uint4 w[TN][NJ];
        uint32_t ws[kGroup ? TN / 4 : TN], xs[kGroup ? TM / 4 : kMx ? TM : 1];
    };
    uint4 xf[kRing][NP];
    auto read_x = [&](const uint8_t* st, int i) {
#pragma unroll
        for (int q = 0; q < NP; ++q)
            xf[i % kRing][q] = *reinterpret_cast<const uint4*>(st + (xat ^ xpart(q)) + i * 16 * kXRow);
    };
    auto lane_scales = [&](const uint8_t* row) -> uint32_t {  // the lane's bytes of a row's step
        if (kSb == 2) return row[g >> 1];
        const uint8_t* p = row + kz * (kSb / WK) + kLaneSb * g;
        return kLaneSb == 4 ? *reinterpret_cast<const uint32_t*>(p) : kLaneSb == 2 ? *reinterpret_cast<const uint16_t*>(p) : *p;
    };
    auto read_w = [&](const uint8_t* st, Frags& f) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const uint8_t* p = st + j * 16 * kWRow;
            if (kWPer == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(p + wat);
                f.w[j][0] = make_uint4(v.x, v.y, 0, 0);
            } else {
#pragma unroll
                for (int q = 0; q < NJ; ++q) f.w[j][q] = *reinterpret_cast<const uint4*>(p + (wat ^ (16 * q)));
            }
        }
        const uint8_t* sc = st + kXBytes + kWBytes;
        if (kGroup) {
#pragma unroll
            for (int j = 0; j < TN; j += 4)
                f.ws[kGroup ? j / 4 : 0] = *reinterpret_cast<const uint32_t*>(sc + 4 * BM + scale_at(nrow + 16 * j + c16, g));
#pragma unroll
            for (int i = 0; i < TM; i += 4)
                f.xs[kGroup ? i / 4 : 0] = *reinterpret_cast<const uint32_t*>(sc + scale_at(mrow + 16 * i + c16, g));
        } else {
#pragma unroll
            for (int j = 0; j < TN; ++j)
                f.ws[kGroup ? 0 : j] = lane_scales(sc + ((kMx ? BM : 0) + nrow + 16 * j + c16) * kSb);
            if (kMx) {
#pragma unroll
                for (int i = 0; i < TM; ++i) f.xs[kGroup ? 0 : i] = lane_scales(sc + (mrow + 16 * i + c16) * kSb);
            }
        }
    };
    // BF16 activations: a step's W in BF16, product q of NP
    bf16x8 wv[kMx ? 1 : TN][NP];
    auto widen = [&](const Frags& f) {
        if constexpr (!kMx) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    const uint32_t c = pick(f.w[j][q >> 2], q & 3);  // 8 codes, k = 8 q of the lane's
                    wv[j][q] = kNv ? widen_nv(c, e4m3_f32(f.ws[j] >> (8 * (q >> 1)))) : widen_mx(c, e8m0_f32(f.ws[j] >> (8 * (q >> 2))));
                }
        }
    };
    auto products = [&](int i, const Frags& f) {
#pragma unroll
        for (int q = 0; q < (kMx ? NJ : NP); ++q) {
            if constexpr (kMx) {
                for_parts<kParts>([&](auto pc) {
                    constexpr int p = decltype(pc)::value;
                    const uint4 lo = codes_part<kParts, p>(xf[i % kRing][kMx ? 2 * q : 0]);
                    const uint4 hi = codes_part<kParts, p>(xf[i % kRing][kMx ? 2 * q + 1 : 0]);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[j][i] = mfma_tile(kGroup ? j % 4 : q, kGroup ? i % 4 : q, f.w[j][q], lo, hi, f.ws[kGroup ? j / 4 : j],
                                              f.xs[kGroup ? i / 4 : i], acc[j][i]);
                });
            } else {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        wv[j][q], __builtin_bit_cast(bf16x8, xf[i % kRing][q]), acc[j][i], 0, 0, 0);
            }
        }
    };
    // all but this wavefront's last steps' transfers (with left-out ones among
    // them at least those)
    auto wait_steps = [&](auto steps) {
        constexpr int n = decltype(steps)::value;
        if (nx == kXInst)
            wait_transfers<n * kInst>();
        else
            wait_transfers<n * (kInst - kXInst)>();
    };
    // step s with its fragments f, in stage `cur`; reads the next step's
    // fragments into n.  The transfer that starts goes into the stage of s - 1.
    auto step = [&](int s, const uint8_t* cur, uint8_t* next, uint8_t* last, const Frags& f, Frags& n) {
        widen(f);
#pragma unroll
        for (int i = 0; i < TM / 2; ++i) {
            read_x(cur, i + kAhead);
            products(i, f);
        }
        if (s + 1 < nsteps) store_regs(next);
        // s + 1 has landed, s + 2 .. s + kStages - 2 are under way
        if (kStages > 3 && s + kStages - 2 < nsteps)
            wait_steps(std::integral_constant<int, kStages - 3>{});
        else
            wait_transfers<0>();
        __syncthreads();
        if (s + kStages - 1 < nsteps) load(s + kStages - 1, last);
        read_w(next, n);  // past the last step: a stage's leftovers, not used
#pragma unroll
        for (int i = TM / 2; i < TM; ++i) {
            read_x(i + kAhead < TM ? cur : next, (i + kAhead) % TM);
            products(i, f);
        }
    };
    Frags f0, f1;
    if (nsteps > 0) {
        load(0, lds);
        store_regs(lds);
#pragma unroll
        for (int i = 1; i < kStages - 1; ++i)
            if (i < nsteps) load(i, lds + i * kStageBytes);
        if (kStages > 3 && kStages - 2 < nsteps)
            wait_steps(std::integral_constant<int, kStages - 2>{});
        else
            wait_transfers<0>();
        __syncthreads();
        read_w(lds, f0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) read_x(lds, i);
    }
    auto after = [&](int o) { return o == (kStages - 1) * kStageBytes ? 0 : o + kStageBytes; };
    int cur = 0, last = (kStages - 1) * kStageBytes;  // stages of steps s and s - 1
    for (int s = 0; s < nsteps; s += 2) {
        const int next = after(cur);
        step(s, lds + cur, lds + next, lds + last, f0, f1);
        if (s + 1 < nsteps) step(s + 1, lds + next, lds + after(next), lds + cur, f1, f0);
        last = next;
        cur = after(next);
    }

    if (WK > 1) {  // partial sums of the wavefronts that share a tile, added in order
        constexpr int kTile = WM * WN * TN * TM * 64;
        f32x4* const part = reinterpret_cast<f32x4*>(lds) + (tile_wave * TN * TM * 64 + lane);
        __syncthreads();
        if (kz > 0) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) part[(kz - 1) * kTile + (j * TM + i) * 64] = acc[j][i];
        }
        __syncthreads();
        if (kz > 0) return;
#pragma unroll
        for (int z = 0; z < WK - 1; ++z)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[j][i] = acc[j][i] + part[z * kTile + (j * TM + i) * 64];
    }
    const int64_t mw = m0 + mrow, nw = n0 + nrow;
    const bool wide = wide_rows<BF16_OUT, kPair>(a);
    store_tile<TM, TN, BF16_OUT, kPair>(acc, a, mw + c16, nw, g, kNv ? a.ws2[0] : 1.0f, wide,
                                        wide && mw + 16 * TM <= a.M && nw + 16 * TN <= a.N);
}

// ---------------------------------------------------------------------------
// Many tokens and columns, K % KS == 0: tiles of 256 x 256, one workgroup of
// eight wavefronts per CU, which takes tile after tile without a pause.
//
// Wavefronts w and w + 4 share a SIMD.  A wavefront alternates between reading
// all fragments of a step (and starting transfers) and multiplying them, with a
// barrier after each; wavefronts 4..7 run one barrier behind, so that on every
// SIMD one wavefront multiplies while the other reads.  The steps of all tiles
// of a workgroup are one sequence: a tile's results are stored, and its first
// transfers started, in reading phases under the other half's products.
//
//   phase      2s - 1      2s          2s + 1      2s + 2
//   w 0..3     read s      multiply s  read s + 1  multiply s + 1
//   w 4..7     multiply .  read s      multiply s  read s + 1
//
// Transfers of step s + 2 start in the reading phase of step s, into the stage
// of s - 1, which the other half has read a phase before; they have landed when
// the reading phase of step s + 1 ends, which is before either half reads them.
// Scales come 16 bytes per row, that is 4 or 8 steps at a time (a row's bytes
// of one step would cost a cache line each time), by way of a register.  BF16
// activations: of the W fragments only the first 16 columns are widened in the
// reading phase, the rest between the products that do not need them yet.
//
// Measured against the same tile with one barrier per step and fragments read
// under a wavefront's own products (k_w4_tiled), us: MXFP8 8192 x 14336 x 4096 358
// against 434, 2.69 PFLOP/s; BF16 4096 x 14336 x 4096 405 against 471 (NVFP4, 1.19
// PFLOP/s), 361 against 446 (MXFP4, 1.33).  With a byte read per subtile's scales
// instead of one dword for four the MXFP8 layer took 366, and 331 of these if
// nothing was stored; the products alone take 243 (the clock falls under them:
// 4.9 PFLOP/s on zeros, 4.0 on random codes).  An FP32 result, whose X codes go
// through in two parts, takes 700-708.
// ---------------------------------------------------------------------------

// A barrier alone (the waits stand before it); nothing moves across it.
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Byte i of the result in lanes 16 g .. 16 g + 15: byte g of v in the lane 16 i
// + (this lane mod 16).
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t v, int g) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));        // lanes 0..31, 32..63
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false));  // of 0, 1
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false));  // of 2, 3
    // bytes 0..3 of a selector name the second operand's, 4..7 the first's, 12 is 0
    const uint32_t l = __builtin_amdgcn_perm(lo[1], lo[0], 0x0C0C0400u + 0x0101u * g);
    const uint32_t h = __builtin_amdgcn_perm(hi[1], hi[0], 0x04000C0Cu + 0x01010000u * g);
    return l | h;
}

template <int KIND, bool BF16_OUT>
__global__ __launch_bounds__(512) void k_w4_big(W4Args a, uint32_t tiles_m, uint32_t tiles_n) {
    constexpr bool kMx = KIND == kW4Mx, kNv = KIND == kW4Bf16Nvfp4;
    constexpr int BM = 256, BN = 256, TM = 8, TN = 4;  // subtiles of 16 x 16 per wavefront
    constexpr int kParts = BF16_OUT ? 1 : 2;           // of X, for MXFP8
    constexpr int KS = kMx ? 128 : 64, kXRow = 128, kWRow = KS / 2;
    constexpr int kXInst = BM * kXRow / 8192, kWInst = BN * kWRow / 8192;  // transfers per wavefront and step
    constexpr int kWPer = kWRow / 16;
    constexpr int kXBytes = BM * kXRow, kStage = kXBytes + BN * kWRow;
    constexpr int kSb = kNv ? KS / 16 : KS / 32, kChunk = 16 / kSb;  // a row's scale bytes of a step; steps in 16 bytes
    constexpr int kSRows = (kMx ? BM : 0) + BN, kSBytes = kSRows * 16;
    constexpr int kStores = BF16_OUT ? TM * TN / 2 : TM * TN;
    typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
    __shared__ __attribute__((aligned(256))) uint8_t lds[3 * kStage + 2 * kSBytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = wave >> 2;
    const int c16 = lane & 15, g = lane >> 4;
    const uint32_t total = tiles_m * tiles_n;
    const int K = (int)a.K, n = K / KS, nb = K / (kNv ? 16 : 32);

    // What is transferred next: step ls of tile lt.  Offsets are from the tile's
    // first row (32 bits: K <= kMaxW4K).  Rows past the operand's end read its
    // last row and feed outputs that are never stored.
    uint32_t lt = blockIdx.x;
    int ls = 0;
    const uint8_t *xbase, *wbase, *sbase;
    uint32_t xoff[kXInst], woff[kWInst], soff;
    auto source = [&]() {
        const TilePos pos = tile_of(lt, tiles_m, tiles_n);
        const int64_t m0 = pos.m * BM, n0 = pos.n * BN;
        const int mlast = (int)(a.M - 1 - m0 < BM ? a.M - 1 - m0 : BM), nlast = (int)(a.N - 1 - n0 < BN ? a.N - 1 - n0 : BN);
        xbase = a.x + m0 * K * (kMx ? 1 : 2);
        wbase = a.wc + n0 * (K / 2);
#pragma unroll
        for (int i = 0; i < kXInst; ++i) {
            const int row = (wave * kXInst + i) * 8 + lane / 8;
            xoff[i] = (uint32_t)min(row, mlast) * (uint32_t)(K * (kMx ? 1 : 2)) + 16 * ((lane & 7) ^ (row & 7));
        }
#pragma unroll
        for (int i = 0; i < kWInst; ++i) {
            const int t = (wave * kWInst + i) * (64 / kWPer) + lane / kWPer;
            woff[i] = (uint32_t)min(w_row<BF16_OUT>(t), nlast) * (uint32_t)(K / 2) +
                      16 * ((lane % kWPer) ^ (kMx ? (t >> 1) & 3 : 0));
        }
        const bool sx = kMx && wave < 4;
        sbase = sx ? a.xs + m0 * nb : a.ws + n0 * nb;
        soff = (uint32_t)(sx ? min(tid, mlast) : min(w_row<BF16_OUT>(tid & 255), nlast)) * (uint32_t)nb;
    };
    // 16 scale bytes of the thread's row, of step ls and those behind it (the
    // row's last 16 where fewer are left)
    u32x4 sreg = {};
    auto load_scales = [&]() { sreg = *reinterpret_cast<const u32x4_a1*>(sbase + min(ls * kSb, nb - 16) + soff); };
    auto transfer = [&](uint32_t stage) {
        const uint8_t* xb = xbase + (int64_t)ls * kXRow;
        const uint8_t* wb = wbase + (int64_t)ls * kWRow;
#pragma unroll
        for (int i = 0; i < kXInst; ++i) to_lds16(xb, xoff[i], stage + (wave * kXInst + i) * 1024);
#pragma unroll
        for (int i = 0; i < kWInst; ++i) to_lds16(wb, woff[i], stage + kXBytes + (wave * kWInst + i) * 1024);
        if (++ls == n) {
            ls = 0;
            lt += gridDim.x;
            if (lt < total) source();
        }
    };
    // Chunks of scales alternate between two areas.  MXFP8: by step, then 64 rows
    // at a time a dword of lane (c16, g): block g of the rows c16 + 16 i, so that
    // one read gives a lane its scales of 4 subtiles and the instruction selects
    // one.  Else 16 bytes per row.
    uint8_t* const scales = lds + 3 * kStage;
    int filled = 0;
    auto store_scales = [&]() {
        uint8_t* const area = scales + filled * kSBytes;
        if constexpr (kMx) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                *reinterpret_cast<uint32_t*>(area + b * kSRows * 4 + tid * 4) = transpose_bytes(sreg[b], g);
        } else if (tid < kSRows) {
            *reinterpret_cast<u32x4*>(area + tid * 16) = sreg;
        }
        filled ^= 1;
    };

    // Fragments of a step.  MXFP8: the lane's W piece is logical block g, its X
    // halves are pieces g and 4 + g.  BF16: k = 16 g .. of the step.
    const int mrow = half * 128, nrow = (wave & 3) * 64;
    const int xat = (mrow + c16) * kXRow + 16 * ((kMx ? g : 2 * g) ^ (c16 & 7)), xother = kMx ? 64 : 16;
    const int wat = kXBytes + (nrow + c16) * kWRow + (kMx ? 16 * (g ^ ((c16 >> 1) & 3)) : 8 * g);
    const int sg = kSb == 2 ? g >> 1 : g;
    const int sxat = (mrow + lane) * 4, swat = kMx ? (BM + nrow + lane) * 4 : (nrow + c16) * 16 + sg;
    uint4 w[kMx ? TN : 1], x[TM][2];
    uint32_t ws[kMx ? TN / 4 : TN], xs[TM / 4];
    bf16x8 wv[kMx ? 1 : TN][2];
    auto read_x = [&](const uint8_t* st, const uint8_t* sc) {
        if constexpr (kMx) {
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) xs[i] = *reinterpret_cast<const uint32_t*>(sc + sxat + i * 256);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            x[i][0] = *reinterpret_cast<const uint4*>(st + xat + i * 16 * kXRow);
            x[i][1] = *reinterpret_cast<const uint4*>(st + (xat ^ xother) + i * 16 * kXRow);
        }
    };
    uint2 wc[kMx ? 1 : TN];
    auto read_w = [&](const uint8_t* st, const uint8_t* sc) {
        if constexpr (kMx) ws[0] = *reinterpret_cast<const uint32_t*>(sc + swat);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (kMx)
                w[j] = *reinterpret_cast<const uint4*>(st + wat + j * 16 * kWRow);
            else
                wc[j] = *reinterpret_cast<const uint2*>(st + wat + j * 16 * kWRow);
            if constexpr (!kMx) ws[j] = sc[swat + j * 256];
        }
    };
    auto widen = [&](int from, int to) {
        if constexpr (!kMx) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if (j < from || j >= to) continue;
                const float s = kNv ? e4m3_f32(ws[j]) : e8m0_f32(ws[j]);
                wv[j][0] = kNv ? widen_nv(wc[j].x, s) : widen_mx(wc[j].x, s);
                wv[j][1] = kNv ? widen_nv(wc[j].y, s) : widen_mx(wc[j].y, s);
            }
        }
    };
    f32x4 acc[TN][TM];
    auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[j][i] = (f32x4){};
    };
    auto products = [&]() {
        if constexpr (kMx) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                for_parts<kParts>([&](auto pc) {
                    constexpr int p = decltype(pc)::value;
                    const uint4 lo = codes_part<kParts, p>(x[i][0]), hi = codes_part<kParts, p>(x[i][1]);
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[j][i] = mfma_tile(j, i % 4, w[j], lo, hi, ws[0], xs[i / 4], acc[j][i]);
                });
        } else {
            // columns 16 .. 63 are widened under the first columns' products
            widen(1, TN);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j][q], __builtin_bit_cast(bf16x8, x[i][q]),
                                                                            acc[j][i], 0, 0, 0);
        }
    };
    // Stores tile t; whether exactly kStores instructions did it.
    const float s2w = kNv ? a.ws2[0] : 1.0f;
    const bool wide = wide_rows<BF16_OUT, BF16_OUT>(a);
    auto store = [&](uint32_t t) {
        const TilePos pos = tile_of(t, tiles_m, tiles_n);
        const int64_t m0 = pos.m * BM + mrow, n0 = pos.n * BN + nrow;
        const bool whole = wide && m0 + 128 <= a.M && n0 + 64 <= a.N;
        store_tile<TM, TN, BF16_OUT, BF16_OUT>(acc, a, m0 + c16, n0, g, s2w, wide, whole);
        return whole;
    };

    uint8_t *s0 = lds, *s1 = lds + kStage, *s2 = lds + 2 * kStage;
    source();
    load_scales();
    transfer(lds_address(s0));
    store_scales();
    bool chunk = false;  // a chunk of scales is in registers
    if (lt < total) {
        if (ls % kChunk == 0) {
            load_scales();
            chunk = true;
        }
        transfer(lds_address(s1));
    }
    wait_transfers<0>();
    clear();
    __syncthreads();
    if (half) phase_barrier();
    int used = 1;  // the area of the present chunk
    uint32_t before = blockIdx.x;
    for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
        for (int s = 0; s < n; ++s) {
            bool counted = false;
            if (s == 0 && t != before) {
                counted = store(before);
                clear();
            }
            if (s % kChunk == 0) used ^= 1;
            if (chunk) store_scales();
            chunk = false;
            const bool more = lt < total;
            if (more && ls % kChunk == 0) {
                load_scales();
                chunk = true;
            }
            const int at = s * kSb - min((s - s % kChunk) * kSb, nb - 16);  // in the chunk's 16 bytes
            const uint8_t* const sc = scales + used * kSBytes + (kMx ? at * kSRows : at);
            __builtin_amdgcn_sched_barrier(0);
            if (!kMx) read_w(s0, sc);  // widened while the rest comes
            __builtin_amdgcn_sched_barrier(0);
            if (more) transfer(lds_address(s2));
            __builtin_amdgcn_sched_barrier(0);
            if (kMx) read_w(s0, sc);
            read_x(s0, sc);
            widen(0, 1);
            __builtin_amdgcn_sched_barrier(0);
            // step s + 1 has landed; what came after it may be under way
            if (!more)
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            else if (counted)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kXInst + kWInst + kStores) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kXInst + kWInst) : "memory");
            phase_barrier();
            __builtin_amdgcn_s_setprio(1);
            products();
            __builtin_amdgcn_s_setprio(0);
            phase_barrier();
            uint8_t* const free = s0;
            s0 = s1;
            s1 = s2;
            s2 = free;
        }
        before = t;
    }
    if (!half) phase_barrier();
    store(before);
}

// Whole steps, and 16 scale bytes per row.
template <int KIND>
bool big_fits(int64_t K) {
    return K % (KIND == kW4Mx ? 128 : 64) == 0 && K >= (KIND == kW4Bf16Nvfp4 ? 256 : 512);
}

template <int KIND, bool BF16_OUT>
hipError_t run_big(const W4Args& args, int64_t cus, hipStream_t stream) {
    const int64_t tiles_n = (args.N + 255) / 256;
    const int64_t most = ((int64_t)1 << 30) / tiles_n;  // token tiles of a launch: 32-bit tile numbers
    for (int64_t row = 0; row < args.M; row += most * 256) {
        const W4Args a = rows_from<KIND, BF16_OUT>(args, row, most * 256);
        const int64_t tiles_m = (a.M + 255) / 256;
        const int64_t grid = tiles_m * tiles_n < cus ? tiles_m * tiles_n : cus;
        const hipError_t e = launch(&k_w4_big<KIND, BF16_OUT>, dim3((unsigned)grid), dim3(512), stream, a,
                                    (uint32_t)tiles_m, (uint32_t)tiles_n);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int KIND, int KS, int BM, int BN, int WM, int WN, int WK, int STAGES, bool BF16_OUT, bool W_REG = false>
hipError_t run_tiled(const W4Args& args, hipStream_t stream) {
    const int64_t tiles_n = (args.N + BN - 1) / BN;
    // runs of token tiles whose grid stays within 2^31 threads
    const int64_t most = (((int64_t)1 << 31) / (64 * WM * WN * WK)) / tiles_n;
    if (most < 1) return hipErrorInvalidValue;
    for (int64_t row = 0; row < args.M; row += most * BM) {
        const W4Args a = rows_from<KIND, BF16_OUT>(args, row, most * BM);
        const int64_t tiles_m = (a.M + BM - 1) / BM;
        const hipError_t e = launch(&k_w4_tiled<KIND, KS, BM, BN, WM, WN, WK, STAGES, BF16_OUT, W_REG>,
                                    dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WM * WN * WK), stream, a, (uint32_t)tiles_m,
                                    (uint32_t)tiles_n);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int KIND, bool BF16_OUT, int WAVES, int T, int MT>
hipError_t run_decode(const W4Args& args, hipStream_t stream) {
    const int64_t tiles_n = (args.N + 16 * T - 1) / (16 * T);
    // runs of token tiles whose grid stays within 2^31 threads
    const int64_t most = (((int64_t)1 << 31) / (64 * WAVES)) / tiles_n;
    if (most < 1) return hipErrorInvalidValue;
    for (int64_t row = 0; row < args.M; row += most * 16 * MT) {
        const W4Args a = rows_from<KIND, BF16_OUT>(args, row, most * 16 * MT);
        const int64_t tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
        const hipError_t e = launch(&k_w4_decode<KIND, BF16_OUT, WAVES, T, MT>, dim3((unsigned)(tiles_m * tiles_n)),
                                    dim3(64 * WAVES), stream, a, tiles_n);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Which kernel, by length, tokens and how many workgroups a tile gives.  The
// times are microseconds, medians of several buffers in turn.
//
// Decode (wavefronts share a column tile and split k): `t` 16-column tiles per
// workgroup, as few as let every workgroup be resident at once -- X is then read
// once per 16 t columns, and fewer, wider workgroups leave CUs idle (MXFP8 x
// MXFP4 at t = 1, 2, 4: 8 x 4096 x 4096 4.5, 5.4, -; 8 x 6144 x 4096 7.1, 6.0, 7.4;
// 8 x 28672 x 8192 39, 35.2, 32.1).  With up to 4 tokens X costs little and t
// stays at 2 at most (1 x 14336 x 4096 8.4 against 9.7 with 4).  Four
// wavefronts; eight where such a small batch meets a long K (1 x 8192 x 28672
// 23.9 against 27.3; at 4096 they are 10 % slower).
int decode_columns(int64_t tiles_m, int64_t M, int64_t N, int64_t cus) {
    int t = 1;
    while (t < (M <= 4 ? 2 : 4) && tiles_m * ((N + 16 * t - 1) / (16 * t)) > cus) t *= 2;
    return t;
}

constexpr int64_t kDecodeLongK = 8192;

template <int KIND, bool BF16_OUT>
hipError_t decode_16(const W4Args& a, int64_t cus, hipStream_t stream) {
    const int t = decode_columns(1, a.M, a.N, cus);
    if (a.M <= 4 && a.K > kDecodeLongK)
        return t == 1 ? run_decode<KIND, BF16_OUT, 8, 1, 1>(a, stream) : run_decode<KIND, BF16_OUT, 8, 2, 1>(a, stream);
    if (t == 1) return run_decode<KIND, BF16_OUT, 4, 1, 1>(a, stream);
    if (t == 2) return run_decode<KIND, BF16_OUT, 4, 2, 1>(a, stream);
    return run_decode<KIND, BF16_OUT, 4, 4, 1>(a, stream);
}

inline int64_t tiles(const W4Args& a, int bm, int bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); }

// Up to 4 tokens always, up to 8 where tiles of 32 x 32 would all be resident:
// 8 x 4096 x 4096 5.1 against 5.5 (MXFP8), 6.3 against 8.0 (BF16 x NVFP4); but
// 8 x 14336 x 4096 10.6 against 8.4, and 13.1 against 11.9; 16 x 4096 x 4096 6.1
// against 5.5, 16 x 4096 x 14336 21.6 against 21.4 (NVFP4).
bool decode_fits(const W4Args& a, int64_t cus) { return a.M <= 4 || (a.M <= 8 && tiles(a, 32, 32) <= cus); }

// Whole steps of at least one of the tiles below, scales that 4-byte transfers
// can take.
bool direct_fits(const W4Args& a) {
    return a.K % 256 == 0 && ((uintptr_t)a.ws & 3) == 0 && ((uintptr_t)a.xs & 3) == 0;
}

// Tiles: the smallest whose workgroups are all resident at once (a second round
// of few workgroups costs as much as a full one), else the largest, which moves
// the fewest bytes per product.  Small tiles have several wavefronts per output
// that split the step (61 x 6144 x 4096 of NVFP4: 11.8 with four, 13.0 with two,
// 15.7 with one; 1024 x 4096 x 4096 of MXFP8 in 128 x 128: 22.4 with two, 26.5 with
// one) and up to four stages (100 x 4096 x 4096 of MXFP8 8.5 with four, 9.3 with
// three).
// MXFP8, tiles of 32 x 32, 32 x 64, 64 x 64, 64 x 128: 32 x 4096 x 4096 5.8, 6.7,
// 8.6, -; 100 x 4096 x 4096 -, 7.7, 10.3, -; 100 x 14336 x 4096 -, -, 15.1, 13.6;
// 64 x 128, 128 x 128, 256 x 128, 256 x 256: 512 x 4096 x 4096 15.3, 20.3, 36, 46;
// 512 x 6144 x 4096 25.3, 20.8, 36, 47; 512 x 14336 x 4096 49, 39.5, 37, 47;
// 1024 x 14336 x 4096 82, 75, 77, 53.  (BF16 results; FP32 results follow the same
// rule.)
template <bool BF16_OUT>
hipError_t direct_mx(const W4Args& a, int64_t cus, hipStream_t stream) {
    if (a.K % 512 == 0) {
        if (tiles(a, 32, 32) <= cus) return run_tiled<kW4Mx, 512, 32, 32, 1, 2, 4, 4, BF16_OUT>(a, stream);
        if (tiles(a, 32, 64) <= cus) return run_tiled<kW4Mx, 512, 32, 64, 1, 2, 4, 4, BF16_OUT>(a, stream);
    }
    if (tiles(a, 64, 64) <= cus) return run_tiled<kW4Mx, 256, 64, 64, 2, 2, 2, 4, BF16_OUT>(a, stream);
    if (tiles(a, 64, 128) <= cus) return run_tiled<kW4Mx, 256, 64, 128, 2, 2, 2, 4, BF16_OUT>(a, stream);
    if (tiles(a, 128, 128) <= cus) return run_tiled<kW4Mx, 256, 128, 128, 2, 2, 2, 3, BF16_OUT>(a, stream);
    if (tiles(a, 256, 128) <= cus) return run_tiled<kW4Mx, 128, 256, 128, 4, 2, 1, 3, BF16_OUT>(a, stream);
    if (big_fits<kW4Mx>(a.K)) return run_big<kW4Mx, BF16_OUT>(a, cus, stream);
    return run_tiled<kW4Mx, 128, 256, 256, 2, 4, 1, 0, BF16_OUT>(a, stream);
}

// BF16 activations likewise, but with two workgroups per CU where their stages
// leave room (64 x 64 for NVFP4, whose widening costs more, and 128 x 128).
// NVFP4, tiles of 32 x 32, 32 x 64 in steps of 512 and of 256, 64 x 64, 32 x 128,
// 64 x 128: 61 x 4096 x 4096 10.3, 11.9, 13.0, 17, -, -; 61 x 6144 x 4096 17.1, 11.8,
// 13.0, 16.5, -, -; 61 x 14336 x 4096 31, 21.5, 19.1, 17.6, 18.3, 23;
// 8 x 28672 x 8192 55, 39, 36, 64, 34.2, 42; 64 x 28672 x 8192 -, -, 75, 70, 64, 48;
// 64 x 128, 128 x 128, 256 x 256: 512 x 4096 x 4096 24.9, 40, 89;
// 256 x 14336 x 4096 45.9, 42.0, 90; 512 x 14336 x 4096 89, 82, 90;
// 1024 x 14336 x 4096 154, -, 106.
template <int KIND, bool BF16_OUT>
hipError_t direct_bf16(const W4Args& a, int64_t cus, hipStream_t stream) {
    if (a.K % 512 == 0) {
        if (tiles(a, 32, 32) <= cus) return run_tiled<KIND, 512, 32, 32, 1, 2, 4, 3, BF16_OUT>(a, stream);
        if (tiles(a, 32, 64) <= cus) return run_tiled<KIND, 512, 32, 64, 1, 4, 4, 3, BF16_OUT>(a, stream);
    }
    if (tiles(a, 32, 64) <= cus) return run_tiled<KIND, 256, 32, 64, 1, 4, 2, 4, BF16_OUT>(a, stream);
    if constexpr (KIND == kW4Bf16Nvfp4) {
        if (a.M > 32 && tiles(a, 64, 64) <= cus) return run_tiled<KIND, 256, 64, 64, 1, 4, 2, 3, BF16_OUT>(a, stream);
    }
    if (tiles(a, 32, 128) <= cus) return run_tiled<KIND, 256, 32, 128, 1, 4, 2, 4, BF16_OUT>(a, stream);
    if (tiles(a, 64, 128) <= cus) return run_tiled<KIND, 256, 64, 128, 1, 4, 2, 3, BF16_OUT>(a, stream);
    if (tiles(a, 128, 128) <= 2 * cus) return run_tiled<KIND, 128, 128, 128, 2, 4, 1, 3, BF16_OUT>(a, stream);
    if (big_fits<KIND>(a.K)) return run_big<KIND, BF16_OUT>(a, cus, stream);
    return run_tiled<KIND, 64, 256, 256, 2, 4, 1, 0, BF16_OUT>(a, stream);
}

// BF16 activations, tiles for other lengths.  W_REG: K % 32 == 16, for which
// 16-byte transfers of W are not aligned.  K = 4112 and 4128: 61 x 14336 27.9 and
// 25.3, 128 x 14336 37.8 and 35.2, 1024 x 4096 53 and 53, 8192 x 14336 980 and 890
// (with the decode kernel 43.7, 80, 148, 4300 at K = 4112).
template <int KIND, bool BF16_OUT, bool W_REG>
hipError_t any_bf16(const W4Args& a, int64_t cus, hipStream_t stream) {
    if (tiles(a, 32, 64) <= 2 * cus) return run_tiled<KIND, 256, 32, 64, 1, 4, 1, 0, BF16_OUT, W_REG>(a, stream);
    if (tiles(a, 64, 128) <= 4 * cus) return run_tiled<KIND, 128, 64, 128, 1, 4, 1, 0, BF16_OUT, W_REG>(a, stream);
    if (!W_REG && big_fits<KIND>(a.K)) return run_big<KIND, BF16_OUT>(a, cus, stream);
    return run_tiled<KIND, 64, 256, 256, 2, 4, 1, 0, BF16_OUT, W_REG>(a, stream);
}

// Other lengths: decode up to 64 tokens, with two token tiles per wavefront from
// 17, while at most 32 columns per workgroup fill the device (32 x 4096 x 14336
// 20.7 against 27.5 with tiles of 32 x 64, but 32 x 14336 x 4096 13.5 against 11.3);
// then few tiles by the same rule, which bear a partial step (100 x 14336 x 4096
// of MXFP8: 64 x 64 17.3, 128 x 128 27.9; 128 x 14336 x 4096 of NVFP4: 32 x 64 41,
// 64 x 128 31.5).
template <int KIND, bool BF16_OUT>
hipError_t pick_any(const W4Args& a, int64_t cus, hipStream_t stream) {
    if (a.M <= 16) return decode_16<KIND, BF16_OUT>(a, cus, stream);
    const int64_t pairs = (a.M + 31) / 32;
    if (a.M <= 64 && pairs * ((a.N + 31) / 32) <= cus)
        return decode_columns(pairs, a.M, a.N, cus) == 1 ? run_decode<KIND, BF16_OUT, 4, 1, 2>(a, stream)
                                                         : run_decode<KIND, BF16_OUT, 4, 2, 2>(a, stream);
    if constexpr (KIND == kW4Mx) {
        if (tiles(a, 64, 64) <= 2 * cus) return run_tiled<KIND, 256, 64, 64, 2, 2, 1, 0, BF16_OUT>(a, stream);
        if (tiles(a, 128, 128) <= cus) return run_tiled<KIND, 128, 128, 128, 2, 2, 1, 0, BF16_OUT>(a, stream);
        if (big_fits<KIND>(a.K)) return run_big<KIND, BF16_OUT>(a, cus, stream);
        return run_tiled<KIND, 128, 256, 256, 2, 4, 1, 0, BF16_OUT>(a, stream);
    } else {
        if constexpr (KIND == kW4Bf16Nvfp4) {
            if (a.K % 32 != 0) return any_bf16<KIND, BF16_OUT, true>(a, cus, stream);
        }
        return any_bf16<KIND, BF16_OUT, false>(a, cus, stream);
    }
}

template <int KIND, bool BF16_OUT>
hipError_t pick_kind(const W4Args& a, int64_t cus, hipStream_t stream) {
    if (!direct_fits(a)) return pick_any<KIND, BF16_OUT>(a, cus, stream);
    if (decode_fits(a, cus)) return decode_16<KIND, BF16_OUT>(a, cus, stream);
    if constexpr (KIND == kW4Mx)
        return direct_mx<BF16_OUT>(a, cus, stream);
    else
        return direct_bf16<KIND, BF16_OUT>(a, cus, stream);
}

template <bool BF16_OUT>
hipError_t pick(const W4Args& a, W4Kind kind, int64_t cus, hipStream_t stream) {
    switch (kind) {
        case kW4Mx: return pick_kind<kW4Mx, BF16_OUT>(a, cus, stream);
        case kW4Bf16Nvfp4: return pick_kind<kW4Bf16Nvfp4, BF16_OUT>(a, cus, stream);
        case kW4Bf16Mxfp4: return pick_kind<kW4Bf16Mxfp4, BF16_OUT>(a, cus, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_w4_linear(const W4Args& a, W4Kind kind, bool bf16_out, hipStream_t stream) {
    int64_t cus = 0;
    const hipError_t e = nvfp4_linear_cus(cus);
    if (e != hipSuccess) return e;
    return bf16_out ? pick<true>(a, kind, cus, stream) : pick<false>(a, kind, cus, stream);
}

}  // namespace focus
