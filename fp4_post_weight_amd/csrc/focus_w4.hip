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
