// focus_rows.hip -- gfx950 kernels of the operators between a decoder layer's
// linear layers: the root-mean-square norm with the residual's addition and
// the gated activation, each with a BF16, NVFP4 or MXFP8 result, and the
// MXFP8 quantizer.
//
//   norm:   h = BF16(x + r);  y_i = (h_i * rs) * w_i,
//           rs = RN32(1 / sqrt(sum_i h_i^2 / n + eps))
//   gated:  y_i = (g_i * sigmoid(g_i)) * u_i
//   NVFP4:  s2 = max|y| / 2688 per row, then the weight quantizer's block
//           scale and codes with m = 1 and sigmoid = 1
//   MXFP8:  S = 2^(floor(log2 max|y_b|) - 8) per 32-block,
//           c = E4M3(clamp(y / S, -448, 448))
// Every operation is one binary32 operation, except that the sum of squares,
// its mean and the reciprocal root are binary64 (the square of a BF16 is
// exact there, and the order of the additions moves the sum by at most
// n * 2^-53, so the binary32 rs does not depend on the split of the row over
// lanes, short of a rounding border) and that exp in the sigmoid is correctly
// rounded to binary32.  y is quantized from binary32: no BF16 value lies
// between the norm or the activation and the codes.
//
// How it maps onto CDNA4 (wave64): a lane owns vectors of 8 consecutive
// elements (one 16-byte load), so every load and store instruction of a
// wavefront covers contiguous memory, and a 16- or 32-element block is 2 or 4
// neighbouring lanes, whose maximum is exchanged by DPP.  All of it is bound
// by HBM for large batches and by the launch and two dependent memory
// latencies for a single token.  Measured: norm to MXFP8 of [8192, 4096] 41 us
// (5.7 TB/s), norm to BF16 of [1003, 8192] 10.8 (6.1 TB/s, the last-level cache),
// gated activation to MXFP8 of [333, 28672] 10.6 (4.5 TB/s), to NVFP4 with values
// of [8192, 14336] 153-172 (4.5-5.0 TB/s, the exact exponential and the codes keep
// the vector units as busy), one row 2.5-2.9.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "focus_launch.h"
#include "focus_numerics.h"
#include "focus_rows.h"

namespace focus {

namespace {

constexpr int kFlatThreads = 256;
constexpr int64_t kMaxRowGrid = 1 << 20;

// ---------------------------------------------------------------------------
// lane exchanges
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

// Maximum of non-negative binary32 values (integer order) over the 2 or 4
// lanes of a block.
template <int LANES>
__device__ __forceinline__ float block_max(float v) {
    uint32_t u = __float_as_uint(v);
    u = max(u, dpp_u32<kDppXor1>(u));
    if (LANES == 4) u = max(u, dpp_u32<kDppXor2>(u));
    return __uint_as_float(u);
}

__device__ __forceinline__ float wave_max(float v) {
    uint32_t u = __float_as_uint(v);
    u = max(u, dpp_u32<kDppXor1>(u));
    u = max(u, dpp_u32<kDppXor2>(u));
    u = max(u, dpp_u32<kDppHalfMirror>(u));
    u = max(u, dpp_u32<kDppMirror>(u));
    uint32_t m = (uint32_t)__builtin_amdgcn_readlane((int)u, 0);
#pragma unroll
    for (int l = 16; l < 64; l += 16) m = max(m, (uint32_t)__builtin_amdgcn_readlane((int)u, l));
    return __uint_as_float(m);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp_u32<CTRL>((uint32_t)b), hi = dpp_u32<CTRL>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, lo | (hi << 32));
}

__device__ __forceinline__ double lane_f64(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, lo | (hi << 32));
}

// Sum over the wavefront, the same value in every lane.
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_f64<kDppXor1>(v);
    v += dpp_f64<kDppXor2>(v);
    v += dpp_f64<kDppHalfMirror>(v);
    v += dpp_f64<kDppMirror>(v);
    return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// ---------------------------------------------------------------------------
// eight elements
// ---------------------------------------------------------------------------

struct Vec8 {
    float f[8];
};

__device__ __forceinline__ Vec8 unpack8(uint4 v) {
    Vec8 o;
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.f[2 * i] = bf16_lo(d[i]);
        o.f[2 * i + 1] = bf16_hi(d[i]);
    }
    return o;
}

__device__ __forceinline__ uint4 pack_bf16(const Vec8& v) {
    return make_uint4(bf16_pair(v.f[0], v.f[1]), bf16_pair(v.f[2], v.f[3]), bf16_pair(v.f[4], v.f[5]),
                      bf16_pair(v.f[6], v.f[7]));
}

// A NaN wins every maximum below (here by the instruction, between lanes by the
// integer order of the bits).
__device__ __forceinline__ float max_abs8(const Vec8& v) {
    float m = __builtin_fabsf(v.f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __builtin_elementwise_maximum(m, __builtin_fabsf(v.f[i]));
    return m;
}

// BF16(x + r), the stored residual.
__device__ __forceinline__ uint4 add_bf16(uint4 a, uint4 b) {
    Vec8 x = unpack8(a);
    const Vec8 y = unpack8(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = x.f[i] + y.f[i];
    return pack_bf16(x);
}

__device__ __forceinline__ double sum_squares8(uint4 v) {
    const Vec8 x = unpack8(v);
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        s0 = __builtin_fma((double)x.f[i], (double)x.f[i], s0);
        s1 = __builtin_fma((double)x.f[i + 1], (double)x.f[i + 1], s1);
    }
    return s0 + s1;
}

__device__ __forceinline__ Vec8 norm8(uint4 h, uint4 w, float rs) {
    Vec8 x = unpack8(h);
    const Vec8 g = unpack8(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = (x.f[i] * rs) * g.f[i];
    return x;
}

// expf(-g) for a BF16 g, correctly rounded where it is at least 2^-126 (below,
// 1 + expf(-g) is 1 whatever its last bits): 2^t = 2^n P(f), t = -g log2(e),
// n = rint(t) by the addition of 1.5 * 2^52, whose sum holds n in its low word;
// P the degree-7 polynomial whose (P(f) - 1)/f meets (2^f - 1)/f at the
// Chebyshev nodes of [-1/2, 1/2] (60-digit decimal arithmetic), 2^-33 from 2^f
// -- which decides the binary32 rounding of every one of the 65280 finite g
// (checked on all of them).  Beyond +-105 the result is 0 or infinity.
__device__ __forceinline__ float exp_neg_bf16(float g) {
    constexpr double kLog2e = 0x1.71547652b82fep+0, kRound = 0x1.8p+52;
    const double x = (double)__builtin_amdgcn_fmed3f(-g, -105.0f, 105.0f);
    const double m = __builtin_fma(x, kLog2e, kRound);
    const double f = __builtin_fma(x, kLog2e, -(m - kRound));
    double p = __builtin_fma(0x1.00a58159a6cc2p-16, f, 0x1.443fffc90db59p-13);
    p = __builtin_fma(p, f, 0x1.5d879ead06012p-10);
    p = __builtin_fma(p, f, 0x1.3b2a1b7152befp-7);
    p = __builtin_fma(p, f, 0x1.c6b08d883dcabp-5);
    p = __builtin_fma(p, f, 0x1.ebfbe045f4d3cp-3);
    p = __builtin_fma(p, f, 0x1.62e42fefa39efp-1);
    p = __builtin_fma(p, f, 1.0);
    return __builtin_ldexpf((float)p, (int)(uint32_t)__builtin_bit_cast(uint64_t, m));
}

// (g * sigmoid(g)) * u, sigmoid(g) = 1 / (1 + expf(-g)), each a binary32
// rounding.  The quotient is the corrected hardware reciprocal, which equals
// it for every divisor in [1, 2^126) (recip_rn_ge1); larger ones need a gate
// below -87 and take the division.
__device__ __forceinline__ Vec8 silu8(uint4 g, uint4 u) {
    Vec8 x = unpack8(g);
    const Vec8 y = unpack8(u);
    float s[8], q[8], least = x.f[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s[i] = 1.0f + exp_neg_bf16(x.f[i]);
        const float r = __builtin_amdgcn_rcpf(s[i]);
        q[i] = __builtin_fmaf(__builtin_fmaf(-s[i], r, 1.0f), r, r);
        least = fminf(least, x.f[i]);
    }
    if (least < -87.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (x.f[i] < -87.0f) q[i] = 1.0f / s[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = (x.f[i] * q[i]) * y.f[i];
    return x;
}

// Outputs are written once and not read back by the kernel: nontemporal
// stores, measured against ordinary ones 42.0 and 45.1 us for the norm to MXFP8
// of [8192, 4096], 99 and 107 us for the norm to NVFP4 with values of
// [8192, 8192], 17.6 and 21.2 us for the MXFP8 quantizer of [8192, 4096].
__device__ __forceinline__ void store(uint4* p, uint4 v) {
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void store(uint2* p, uint2 v) {
    __builtin_nontemporal_store(u32x2{v.x, v.y}, reinterpret_cast<u32x2*>(p));
}
__device__ __forceinline__ void store(uint32_t* p, uint32_t v) { __builtin_nontemporal_store(v, p); }

// ---------------------------------------------------------------------------
// outputs: eight elements at vector index v (element 8 v of the dense output)
// ---------------------------------------------------------------------------

// Exponent of the MXFP8 block scale, clamped to E8M0's range (an all-zero
// block: 0, scale 1; a block with an infinity or NaN: 128, whose byte is E8M0's
// NaN), and four E4M3 codes per dword.  y * 2^-e is exact unless it falls below
// 2^-126, which rounds to the code of zero either way; the conversion gives NaN
// beyond 464, so the clamp to 448 stands before it.
__device__ __forceinline__ int mxfp8_exponent(float amax) {
    if (amax == 0.0f) return 0;
    if (!(amax < __builtin_inff())) return 128;
    const int e = __builtin_amdgcn_frexp_expf(amax) - 1 - 8;
    return e < -127 ? -127 : e;
}

__device__ __forceinline__ uint2 mxfp8_codes(const Vec8& y, int e) {
    float x[8];
    const float inv = __builtin_ldexpf(1.0f, -e);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(y.f[i] * inv, -448.0f, 448.0f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// c * 2^e as BF16 (exact: 4 significant bits, unless it leaves BF16's range).
__device__ __forceinline__ uint4 mxfp8_values(uint2 c, int e) {
    const float S = e == 128 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, e);
    uint32_t o[4];
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
    const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), f = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
    o[0] = bf16_pair(a[0] * S, a[1] * S);
    o[1] = bf16_pair(b[0] * S, b[1] * S);
    o[2] = bf16_pair(d[0] * S, d[1] * S);
    o[3] = bf16_pair(f[0] * S, f[1] * S);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool DEQ>
__device__ __forceinline__ void put_mxfp8(const RowArgs& a, int64_t v, const Vec8& y) {
    const int e = mxfp8_exponent(block_max<4>(max_abs8(y)));
    const uint2 c = mxfp8_codes(y, e);
    store(reinterpret_cast<uint2*>(a.codes) + v, c);
    if ((v & 3) == 0) a.scales[v >> 2] = (uint8_t)(e + 127);
    if (DEQ) store(reinterpret_cast<uint4*>(a.y) + v, mxfp8_values(c, e));
}

template <bool DEQ>
__device__ __forceinline__ void put_nvfp4(const RowArgs& a, int64_t v, const Vec8& y, float s2, double rden) {
    if (s2 == 0.0f) {
        // a zero row: scale 1, signed-zero codes, +-0
        uint32_t c = 0;
        Vec8 z;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t s = __float_as_uint(y.f[i]) >> 31;
            c |= s << (4 * i + 3);
            z.f[i] = __uint_as_float(s << 31);
        }
        store(reinterpret_cast<uint32_t*>(a.codes) + v, c);
        if ((v & 1) == 0) a.scales[v >> 1] = 0x38;
        if (DEQ) store(reinterpret_cast<uint4*>(a.y) + v, pack_bf16(z));
        return;
    }
    const uint32_t sb = e4m3_byte_normal(block_t(block_max<2>(max_abs8(y)), 1.0f, rden));
    const float S = e4m3_normal_value(sb);
    const uint32_t c = encode8(y.f, S * s2);
    store(reinterpret_cast<uint32_t*>(a.codes) + v, c);
    if ((v & 1) == 0) a.scales[v >> 1] = (uint8_t)sb;
    if (DEQ) store(reinterpret_cast<uint4*>(a.y) + v, dequant8(c, S, s2));
}

// ---------------------------------------------------------------------------
// rows: WAVES wavefronts share a row, each lane holds CH vectors of it in
// registers (CH == 0: a row of any length, read again in each pass -- the
// lane that wrote an element is the one that reads it back)
// ---------------------------------------------------------------------------

template <int SRC, int OUT, bool DEQ, int WAVES, int CH>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_rows(RowArgs a) {
    constexpr int kThreads = 64 * WAVES;
    constexpr int kRowsPerGroup = WAVES == 1 ? 4 : 1;
    constexpr int R = CH > 0 ? CH : 1;
    __shared__ double red_sum[2][WAVES];
    __shared__ float red_max[2][WAVES];
    const int tid = WAVES == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int wave = threadIdx.x >> 6;
    const int nv = (int)(a.hidden >> 3);
    const int wave0 = __builtin_amdgcn_readfirstlane(tid & ~63);
    const uint4* w = reinterpret_cast<const uint4*>(a.w);
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRowsPerGroup + (WAVES == 1 ? wave : 0); row < a.tokens;
         row += (int64_t)gridDim.x * kRowsPerGroup, parity ^= 1) {
        const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.x_stride);
        const uint4* r = reinterpret_cast<const uint4*>(a.r + (a.r ? row * a.r_stride : 0));
        uint4* res_out = reinterpret_cast<uint4*>(a.res_out + (a.res_out ? row * a.hidden : 0));
        // per lane and vector: the norm's row (then the sum h), residual and
        // weight, or gate and up
        uint4 p[R], q[R], wr[SRC == kRowNorm ? R : 1];
        Vec8 y[OUT == kRowNvfp4 ? R : 1];
        if (CH > 0) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int v = tid + kThreads * k;
                p[k] = q[k] = make_uint4(0, 0, 0, 0);
                if (SRC == kRowNorm) wr[SRC == kRowNorm ? k : 0] = make_uint4(0, 0, 0, 0);
                if (v < nv) {
                    p[k] = x[v];
                    if (SRC == kRowSilu || a.r) q[k] = r[v];
                    if (SRC == kRowNorm) wr[SRC == kRowNorm ? k : 0] = w[v];
                }
            }
        }
        // CH == 0: vector v of the row; SECOND: a later pass, in which the
        // residual may already hold the sum
        auto load = [&](int v, uint4& s, uint4& t, bool second) {
            if (SRC == kRowNorm) {
                t = w[v];
                if (second && a.res_out) {
                    s = res_out[v];
                } else {
                    s = x[v];
                    if (a.r) {
                        s = add_bf16(s, r[v]);
                        if (a.res_out) res_out[v] = s;
                    }
                }
            } else {
                s = x[v];
                t = r[v];
            }
        };
        auto value = [&](uint4 s, uint4 t, float rs) { return SRC == kRowNorm ? norm8(s, t, rs) : silu8(s, t); };

        float rs = 0.0f;
        if (SRC == kRowNorm) {
            double ss = 0.0;
            if (CH > 0) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int v = tid + kThreads * k;
                    if (a.r) {
                        p[k] = add_bf16(p[k], q[k]);
                        if (a.res_out && v < nv) store(res_out + v, p[k]);
                    }
                    ss += sum_squares8(p[k]);  // absent vectors are zeros
                }
            } else {
                for (int v = tid; v < nv; v += kThreads) {
                    load(v, p[0], q[0], false);
                    ss += sum_squares8(p[0]);
                }
            }
            ss = wave_sum(ss);
            if (WAVES > 1) {
                if ((tid & 63) == 0) red_sum[parity][wave] = ss;
                __syncthreads();
                ss = 0.0;
#pragma unroll
                for (int i = 0; i < WAVES; ++i) ss += red_sum[parity][i];
            }
            rs = (float)(1.0 / __builtin_sqrt(ss / (double)a.hidden + (double)a.eps));
        }

        float s2 = 0.0f;
        double rden = 0.0;
        if (OUT == kRowNvfp4) {
            float amax = 0.0f;
            if (CH > 0) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    y[k] = Vec8{};
                    if (wave0 + kThreads * k >= nv) continue;  // no lane of the wavefront has this vector
                    y[k] = SRC == kRowNorm ? norm8(p[k], wr[SRC == kRowNorm ? k : 0], rs) : silu8(p[k], q[k]);
                    amax = __builtin_elementwise_maximum(amax, max_abs8(y[k]));
                }
            } else {
                for (int v = tid; v < nv; v += kThreads) {
                    load(v, p[0], q[0], true);
                    amax = __builtin_elementwise_maximum(amax, max_abs8(value(p[0], q[0], rs)));
                }
            }
            amax = wave_max(amax);
            if (WAVES > 1) {
                if ((tid & 63) == 0) red_max[parity][wave] = amax;
                __syncthreads();
                amax = red_max[parity][0];
#pragma unroll
                for (int i = 1; i < WAVES; ++i) amax = __builtin_elementwise_maximum(amax, red_max[parity][i]);
            }
            s2 = amax / 2688.0f;
            if (tid == 0) a.s2[row] = s2;
            rden = 1.0 / (double)(6.0f * s2);
        }

        auto put = [&](int v, const Vec8& e) {
            const int64_t o = row * nv + v;
            if (OUT == kRowBf16) store(reinterpret_cast<uint4*>(a.y) + o, pack_bf16(e));
            else if (OUT == kRowNvfp4) put_nvfp4<DEQ>(a, o, e, s2, rden);
            else put_mxfp8<DEQ>(a, o, e);
        };
        if (CH > 0) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int v = tid + kThreads * k;
                if (v < nv)
                    put(v, OUT == kRowNvfp4 ? y[OUT == kRowNvfp4 ? k : 0]
                                            : norm8(p[k], wr[SRC == kRowNorm ? k : 0], rs));
            }
        } else {
            for (int v = tid; v < nv; v += kThreads) {
                load(v, p[0], q[0], true);
                put(v, value(p[0], q[0], rs));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// no reduction: vectors in any order
// ---------------------------------------------------------------------------

// Vector index -> row and column of a row of `nv` vectors (n < 2^31), by the
// multiplier of div_magic.
struct FlatShape {
    uint32_t total, nv, mul, shift;
};

template <int SRC, int OUT, bool DEQ>
__global__ __launch_bounds__(kFlatThreads) void k_flat(RowArgs a, FlatShape s) {
    for (uint32_t v = blockIdx.x * kFlatThreads + threadIdx.x; v < s.total; v += gridDim.x * kFlatThreads) {
        const uint32_t row = div_magic(v, s.mul, s.shift);
        const uint32_t col = v - row * s.nv;
        const uint4 p = *reinterpret_cast<const uint4*>(a.x + (int64_t)row * a.x_stride + 8 * (int64_t)col);
        Vec8 y;
        if (SRC == kRowSilu) {
            const uint4 q = *reinterpret_cast<const uint4*>(a.r + (int64_t)row * a.r_stride + 8 * (int64_t)col);
            y = silu8(p, q);
        } else {
            y = unpack8(p);
        }
        if (OUT == kRowBf16) store(reinterpret_cast<uint4*>(a.y) + v, pack_bf16(y));
        else put_mxfp8<DEQ>(a, v, y);
    }
}

template <int SRC, int OUT, bool DEQ, int WAVES, int CH>
hipError_t run_rows(const RowArgs& a, hipStream_t stream) {
    constexpr int per = WAVES == 1 ? 4 : 1;
    int64_t g = (a.tokens + per - 1) / per;
    if (g > kMaxRowGrid) g = kMaxRowGrid;
    return launch(&k_rows<SRC, OUT, DEQ, WAVES, CH>, dim3((unsigned)g), dim3(WAVES == 1 ? 256 : 64 * WAVES), stream, a);
}

// The form whose registers hold the row, with as few vectors per lane as leave
// the workgroup at 8 wavefronts: a lane's vectors are requested together, and
// more, smaller workgroups per CU overlap one row's arithmetic with another's
// loads.  Measured (us, lanes' vectors in brackets): norm to MXFP8 of
// [8192, 4096], 8 (1) and 4 wavefronts (2) 42.4, 42.9, 16 wavefronts 48; norm to
// BF16 of [8192, 8192], 8 (2), 4 (4) and 16 (1) 90.9, 92.7, 92.5; gated
// activation to NVFP4 with values of [8192, 14336], 8 (4), 4 (7) and 16 (2) 153,
// 179, 178; at one row the same choices are within 0.2 us of the best.
template <int SRC, int OUT, bool DEQ>
hipError_t pick_rows(const RowArgs& a, hipStream_t stream) {
    const int64_t nv = a.hidden / 8;
    if (nv <= 64) return run_rows<SRC, OUT, DEQ, 1, 1>(a, stream);
    if (nv <= 256) return run_rows<SRC, OUT, DEQ, 4, 1>(a, stream);
    if (nv <= 512) return run_rows<SRC, OUT, DEQ, 8, 1>(a, stream);
    if (nv <= 1024) return run_rows<SRC, OUT, DEQ, 8, 2>(a, stream);
    if (nv <= 2048) return run_rows<SRC, OUT, DEQ, 8, 4>(a, stream);
    if (nv <= 4096) return run_rows<SRC, OUT, DEQ, 16, 4>(a, stream);
    return run_rows<SRC, OUT, DEQ, 16, 0>(a, stream);
}

template <int SRC, int OUT, bool DEQ>
hipError_t run_flat(const RowArgs& args, hipStream_t stream) {
    // runs of rows of fewer than 2^31 vectors
    const int64_t nv = args.hidden / 8;
    const int64_t most = (((int64_t)1 << 31) - 1) / nv;
    FlatShape s;
    s.nv = (uint32_t)nv;
    uint32_t l = 0;
    while (((uint64_t)1 << l) < (uint64_t)nv) ++l;
    s.shift = 31 + l;
    s.mul = (uint32_t)((((uint64_t)1 << s.shift) + (uint64_t)nv - 1) / (uint64_t)nv);
    for (int64_t row = 0; row < args.tokens; row += most) {
        RowArgs a = args;
        a.tokens = args.tokens - row < most ? args.tokens - row : most;
        a.x += row * a.x_stride;
        if (a.r) a.r += row * a.r_stride;
        if (a.codes) a.codes += row * a.hidden;
        if (a.scales) a.scales += row * (a.hidden / 32);
        if (a.y) a.y += row * a.hidden;
        s.total = (uint32_t)(a.tokens * nv);
        int64_t g = ((int64_t)s.total + kFlatThreads - 1) / kFlatThreads;
        if (g > kMaxRowGrid) g = kMaxRowGrid;
        const hipError_t e = launch(&k_flat<SRC, OUT, DEQ>, dim3((unsigned)g), dim3(kFlatThreads), stream, a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rows(const RowArgs& a, RowSource src, RowOutput out, hipStream_t stream) {
    if (src == kRowNorm) {
        if (out == kRowBf16) return pick_rows<kRowNorm, kRowBf16, false>(a, stream);
        if (out == kRowNvfp4)
            return a.y ? pick_rows<kRowNorm, kRowNvfp4, true>(a, stream) : pick_rows<kRowNorm, kRowNvfp4, false>(a, stream);
        return a.y ? pick_rows<kRowNorm, kRowMxfp8, true>(a, stream) : pick_rows<kRowNorm, kRowMxfp8, false>(a, stream);
    }
    if (src == kRowSilu && out == kRowNvfp4)
        return a.y ? pick_rows<kRowSilu, kRowNvfp4, true>(a, stream) : pick_rows<kRowSilu, kRowNvfp4, false>(a, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_flat(const RowArgs& a, RowSource src, RowOutput out, hipStream_t stream) {
    if (src == kRowSilu) {
        if (out == kRowBf16) return run_flat<kRowSilu, kRowBf16, false>(a, stream);
        if (out == kRowMxfp8)
            return a.y ? run_flat<kRowSilu, kRowMxfp8, true>(a, stream) : run_flat<kRowSilu, kRowMxfp8, false>(a, stream);
    }
    if (src == kRowPlain && out == kRowMxfp8)
        return a.y ? run_flat<kRowPlain, kRowMxfp8, true>(a, stream) : run_flat<kRowPlain, kRowMxfp8, false>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace focus
