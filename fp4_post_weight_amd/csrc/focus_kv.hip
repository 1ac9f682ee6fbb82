// focus_kv.hip -- the paged 8-bit cache of keys and values: writing a step's
// keys and values, reading them back, and the table of the rotation's angles.
//
// A page holds 2^p consecutive tokens of one sequence.  Per page and key/value
// head it has the keys' E4M3 codes [page, dim], the values' E4M3 codes
// transposed [dim, page], and one E8M0 scale byte for each:
//     S = 2^e, e the least integer with max|x| <= 448 * 2^e, -127 <= e <= 119
//     code = E4M3(clamp(x / S, -448, 448))
// A power of two costs E4M3 nothing (its relative step is the same everywhere
// above 2^-6), makes x / S exact, and lets a page that gains a larger token
// move its older codes by a change of exponent, exactly wherever the result is
// above 2^-6.  The values lie transposed because the attention's second
// product contracts over tokens: its operand is then 16 consecutive bytes.
//
// Keys turn by their position's angle in binary32 on the way in:
//     k'[i] = k[i] c - k[i + dim/2] s,  k'[i + dim/2] = k[i + dim/2] c + k[i] s.
//
// Both kernels stream: a workgroup takes one page's part of one head, so that it
// alone decides the page's scale and owns its bytes.  Measured: prompts of up to
// 8191 tokens, 8 heads of 128, written in 42-44 us (3.9 TB/s; bound by dependent
// loads -- offsets, table, rows -- in 2.5 rounds of workgroups; loads where they
// are used 46.6 where this took 44.2), 128 single tokens
// in 5-6 us; 16 sequences of up to 16384 tokens read in 161-163 us (5.0 TB/s of a
// copy's 5.2).  Keys and values in workgroups of their own: 45.6 and 8.5 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "focus_kv.h"
#include "focus_launch.h"
#include "focus_numerics.h"

namespace focus {

namespace {

constexpr int kThreads = 256;

// Exponent of a page whose largest finite magnitude is amax.
__device__ __forceinline__ int kv_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, -127), 119);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

// x / 2^e before its rounding to E4M3; an infinity has no code and becomes NaN
__device__ __forceinline__ float scaled(float x, float inv) {
    const float r = __builtin_amdgcn_fmed3f(x * inv, -448.0f, 448.0f);
    return fabsf(x) < __builtin_inff() ? r : __builtin_nanf("");
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return (uint32_t)v;
}

// Four codes moved to another exponent: E4M3(code * f), f <= 1 a power of two.
__device__ __forceinline__ uint32_t moved4(uint32_t c, float f) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    return codes4(a[0] * f, a[1] * f, b[0] * f, b[1] * f);
}

// 4 x 4 bytes transposed: byte j of out[i] is byte i of in[j].
__device__ __forceinline__ void transpose4(const uint32_t (&in)[4], uint32_t (&out)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400), b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602);
    const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400), d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602);
    out[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
    out[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
    out[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
    out[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = scaled(x[i], inv);
    return make_uint2(codes4(r[0], r[1], r[2], r[3]), codes4(r[4], r[5], r[6], r[7]));
}

// One page of one sequence and head: the tokens lo .. hi-1 of its new ones.
struct PagePart {
    int64_t base;    // position of the page's first token
    int lo, hi;      // tokens of the page, 0 .. 2^log_page
    int row;         // row of the token at lo
    int physical;
};

// False: the item has no tokens, or they have no place (a negative position, a
// position past the table's row, an entry that is no page of the cache).
__device__ __forceinline__ bool page_part(const KvCacheArgs& c, const KvBatchArgs& b, int item, PagePart& p) {
    int number;
    const int i = kv_find(b, c.log_page, item, number);
    const KvSequence s = kv_sequence(b, i);
    const int64_t first = s.first();
    const int64_t page = (first >> c.log_page) + number;
    p.base = page << c.log_page;
    const int64_t lo = max(first, p.base), hi = min(s.length, p.base + ((int64_t)1 << c.log_page));
    if (number < 0 || lo >= hi) return false;
    p.lo = (int)(lo - p.base);
    p.hi = (int)(hi - p.base);
    p.row = s.row0 + (int)(lo - first);
    p.physical = -1;
    if (page >= 0 && page < b.max_pages) {
        const int e = b.table[(int64_t)i * b.table_stride + page];
        if (e >= 0 && e < c.pages) p.physical = e;
    }
    return true;
}

// A workgroup writes one page's part of one head, keys and values.  dim/16
// lanes hold a token, each the elements 8 l .. and dim/2 + 8 l .., the two
// halves of its rotation's pairs.  NP: passes of the workgroup over the page.
template <int D, int NP>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvCacheArgs c, KvBatchArgs b, RopeArgs rope, const uint16_t* k,
                                                       int64_t k_stride, const uint16_t* v, int64_t v_stride) {
    constexpr int kLanes = D / 16, kPass = kThreads / kLanes, kHalf = D / 2;
    constexpr int kRow = D + 4;  // LDS bytes of a token's codes
    __shared__ __attribute__((aligned(16))) uint8_t tile[NP * kPass * kRow];
    __shared__ float red[2][kThreads / 64];
    const int tid = threadIdx.x, sub = tid % kLanes, tok = tid / kLanes;
    const int head = (int)(blockIdx.x % (uint32_t)c.kv_heads), item = (int)(blockIdx.x / (uint32_t)c.kv_heads);
    PagePart p;
    if (!page_part(c, b, item, p) || p.physical < 0) return;
    const int log_page = c.log_page, page = 1 << log_page;

    // all loads of a thread first
    uint4 kr[NP][2], vr[NP][2];  // keys, values
    float4 angle[NP][4];         // cosines, sines
    bool known[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int t = p.lo + n * kPass + tok;
        if (t < p.hi) {
            const int64_t row = p.row + (t - p.lo);
            const uint16_t* kp = k + row * k_stride + head * D + 8 * sub;
            const uint16_t* vp = v + row * v_stride + head * D + 8 * sub;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kr[n][i] = *reinterpret_cast<const uint4*>(kp + i * kHalf);
                vr[n][i] = *reinterpret_cast<const uint4*>(vp + i * kHalf);
            }
            if (rope.table) {
                const int64_t pos = p.base + t;
                known[n] = pos < rope.positions;
                const float4* a = reinterpret_cast<const float4*>(rope.table + (known[n] ? pos : 0) * D + 8 * sub);
                angle[n][0] = a[0], angle[n][1] = a[1], angle[n][2] = a[kHalf / 4], angle[n][3] = a[kHalf / 4 + 1];
            }
        }
    }
    float x[NP][2][8];  // keys
    float ka = 0.0f, va = 0.0f;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int t = p.lo + n * kPass + tok;
        if (t < p.hi) {
            float y[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                unpack8(kr[n][i], x[n][i]);
                unpack8(vr[n][i], y[i]);
            }
            if (rope.table) {
                const float4 a = angle[n][0], b = angle[n][1], c = angle[n][2], d = angle[n][3];
                const float cs[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, sn[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = x[n][0][i], g = x[n][1][i];
                    x[n][0][i] = known[n] ? f * cs[i] - g * sn[i] : __builtin_nanf("");
                    x[n][1][i] = known[n] ? g * cs[i] + f * sn[i] : __builtin_nanf("");
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ka = fmaxf(ka, fmaxf(finite_abs(x[n][0][i]), finite_abs(x[n][1][i])));
                va = fmaxf(va, fmaxf(finite_abs(y[0][i]), finite_abs(y[1][i])));
            }
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        ka = fmaxf(ka, __shfl_xor(ka, m));
        va = fmaxf(va, __shfl_xor(va, m));
    }
    if ((tid & 63) == 0) red[0][tid >> 6] = ka, red[1][tid >> 6] = va;
    __syncthreads();
    ka = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    va = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));

    const int64_t at = (int64_t)p.physical * c.kv_heads + head;
    uint8_t* kc = c.kc + (at << log_page) * D;
    uint8_t* vc = c.vc + (at << log_page) * D;
    int ke = kv_exponent(ka), ve = kv_exponent(va);
    float kmove = 1.0f, vmove = 1.0f;  // of the tokens that the page held before
    if (p.lo > 0) {
        const int ko = (int)c.ks[at] - 127, vo = (int)c.vs[at] - 127;
        ke = max(ke, ko);
        ve = max(ve, vo);
        kmove = __builtin_ldexpf(1.0f, ko - ke);
        vmove = __builtin_ldexpf(1.0f, vo - ve);
    }
    const float kinv = __builtin_ldexpf(1.0f, -ke), vinv = __builtin_ldexpf(1.0f, -ve);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int t = p.lo + n * kPass + tok;
        if (t < p.hi) {
            *reinterpret_cast<uint2*>(kc + t * D + 8 * sub) = codes8(x[n][0], kinv);
            *reinterpret_cast<uint2*>(kc + t * D + kHalf + 8 * sub) = codes8(x[n][1], kinv);
            float y[2][8];
            unpack8(vr[n][0], y[0]);
            unpack8(vr[n][1], y[1]);
            const uint2 a = codes8(y[0], vinv), d = codes8(y[1], vinv);
            uint32_t* o = reinterpret_cast<uint32_t*>(tile + (t - p.lo) * kRow + 8 * sub);
            o[0] = a.x, o[1] = a.y;
            o[kHalf / 4] = d.x, o[kHalf / 4 + 1] = d.y;
        }
    }
    if (kmove != 1.0f) {
        uint32_t* o = reinterpret_cast<uint32_t*>(kc);
        for (int i = tid; i < p.lo * (D / 4); i += kThreads) o[i] = moved4(o[i], kmove);
    }
    __syncthreads();  // also: every thread has read the page's old scale bytes
    if (tid == 0) {
        c.ks[at] = (uint8_t)(ke + 127);
        c.vs[at] = (uint8_t)(ve + 127);
    }
    if (p.hi - p.lo == 1 && vmove == 1.0f) {
        // one token: a byte in each of the values' rows
        if (tid < D) vc[(tid << log_page) + p.lo] = tile[tid];
        return;
    }
    // The values go out four tokens at a time; a piece with tokens that are not
    // new keeps their bytes.
    const int quads = page / 4;
    const int q0 = vmove != 1.0f ? 0 : p.lo / 4, q1 = (p.hi + 3) / 4;
    for (int i = tid; i < (D / 4) * quads; i += kThreads) {
        const int q = i % quads, d = 4 * (i / quads);
        if (q < q0 || q >= q1) continue;
        uint32_t in[4], out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * q + j;
            in[j] = t >= p.lo && t < p.hi ? *reinterpret_cast<const uint32_t*>(tile + (t - p.lo) * kRow + d) : 0;
        }
        transpose4(in, out);
        // bytes of the new tokens, and of those that the page held before
        uint32_t fresh = 0, held = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * q + j;
            if (t >= p.lo && t < p.hi) fresh |= 0xFFu << (8 * j);
            if (t < p.lo) held |= 0xFFu << (8 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t* o = reinterpret_cast<uint32_t*>(vc + ((int64_t)(d + j) << log_page)) + q;
            if (fresh != 0xFFFFFFFFu) {
                const uint32_t old = *o;
                const uint32_t kept = vmove != 1.0f ? (moved4(old, vmove) & held) | (old & ~held) : old;
                *o = (out[j] & fresh) | (kept & ~fresh);
            } else {
                *o = out[j];
            }
        }
    }
}

// Eight codes times 2^e, in BF16, stored past the caches (a wavefront's stores
// cover whole lines).
__device__ __forceinline__ void put8(uint16_t* o, uint2 c, float S) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
    const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
    const u32x4 r = {bf16_pair(a[0] * S, a[1] * S), bf16_pair(b[0] * S, b[1] * S), bf16_pair(d[0] * S, d[1] * S), bf16_pair(e[0] * S, e[1] * S)};
    __builtin_nontemporal_store(r, reinterpret_cast<u32x4*>(o));
}

// A workgroup reads one page's part of one head, keys and values.  (Loads where
// they are used, and 32 bytes per lane stored: 194 us where this takes 163; the
// same stores past the caches 204.)
template <int D>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvCacheArgs c, KvBatchArgs b, uint16_t* k, uint16_t* v) {
    constexpr int kRow = D + 8;
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kRow];
    const int tid = threadIdx.x;
    const int head = (int)(blockIdx.x % (uint32_t)c.kv_heads), item = (int)(blockIdx.x / (uint32_t)c.kv_heads);
    PagePart p;
    if (!page_part(c, b, item, p)) return;
    const int log_page = c.log_page, page = 1 << log_page, n = p.hi - p.lo;
    const int64_t out_row = (int64_t)c.kv_heads * D;
    uint16_t* ko = k + p.row * out_row + head * D;
    uint16_t* vo = v + p.row * out_row + head * D;
    if (p.physical < 0) {
        // no such token (zeros) or no such page (NaN)
        const uint32_t w = p.base < 0 ? 0u : 0x7FC07FC0u;
        for (int i = tid; i < n * (D / 8); i += kThreads) {
            const int64_t o = (i / (D / 8)) * out_row + 8 * (i % (D / 8));
            *reinterpret_cast<uint4*>(ko + o) = make_uint4(w, w, w, w);
            *reinterpret_cast<uint4*>(vo + o) = make_uint4(w, w, w, w);
        }
        return;
    }
    const int64_t at = (int64_t)p.physical * c.kv_heads + head;
    const uint8_t* kc = c.kc + (at << log_page) * D;
    const uint8_t* vc = c.vc + (at << log_page) * D;
    const float ks = __builtin_ldexpf(1.0f, (int)c.ks[at] - 127), vs = __builtin_ldexpf(1.0f, (int)c.vs[at] - 127);
    // all loads of a thread first
    constexpr int kKeys = 128 * (D / 8) / kThreads, kQuads = (D / 4) * 32 / kThreads;
    const int quads = page / 4;
    uint2 keys[kKeys];
    uint32_t in[kQuads][4];
#pragma unroll
    for (int m = 0; m < kQuads; ++m) {
        const int i = tid + m * kThreads, q = i & (quads - 1), d = 4 * (i >> (log_page - 2));
        if (d >= D || 4 * q + 4 <= p.lo || 4 * q >= p.hi) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) in[m][j] = reinterpret_cast<const uint32_t*>(vc + ((int64_t)(d + j) << log_page))[q];
    }
#pragma unroll
    for (int m = 0; m < kKeys; ++m) {
        const int i = tid + m * kThreads;
        if (i < n * (D / 8)) keys[m] = *reinterpret_cast<const uint2*>(kc + p.lo * D + 8 * i);
    }
#pragma unroll
    for (int m = 0; m < kQuads; ++m) {
        const int i = tid + m * kThreads, q = i & (quads - 1), d = 4 * (i >> (log_page - 2));
        if (d >= D || 4 * q + 4 <= p.lo || 4 * q >= p.hi) continue;
        uint32_t out[4];
        transpose4(in[m], out);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(tile + (4 * q + j) * kRow + d) = out[j];
    }
#pragma unroll
    for (int m = 0; m < kKeys; ++m) {
        const int i = tid + m * kThreads, t = i / (D / 8), d = 8 * (i % (D / 8));
        if (i < n * (D / 8)) put8(ko + t * out_row + d, keys[m], ks);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kKeys; ++m) {
        const int i = tid + m * kThreads, t = i / (D / 8), d = 8 * (i % (D / 8));
        if (i < n * (D / 8)) put8(vo + t * out_row + d, *reinterpret_cast<const uint2*>(tile + (p.lo + t) * kRow + d), vs);
    }
}

__global__ __launch_bounds__(kThreads) void k_rope_table(const double* inv_freq, int64_t n, int half, float* table) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t pos = i / half;
    const int j = (int)(i - pos * half);
    double s, c;
    sincos((double)pos * inv_freq[j], &s, &c);
    table[pos * 2 * half + j] = (float)c;
    table[pos * 2 * half + half + j] = (float)s;
}

}  // namespace

hipError_t launch_rope_table(const double* inv_freq, int64_t positions, int64_t dim, float* table, hipStream_t stream) {
    const int64_t n = positions * (dim / 2);
    return launch(k_rope_table, dim3((uint32_t)((n + kThreads - 1) / kThreads)), dim3(kThreads), stream, inv_freq, n,
                  (int)(dim / 2), table);
}

bool kv_pages_fit(const KvCacheArgs& c, const KvBatchArgs& b) {
    return kv_items(b, c.log_page) * c.kv_heads <= 0xFFFFFFFFll / kThreads;
}

hipError_t launch_kv_write(const KvCacheArgs& c, const KvBatchArgs& b, const RopeArgs& r, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride, hipStream_t stream) {
    const dim3 grid((uint32_t)(kv_items(b, c.log_page) * c.kv_heads));
    const int page = 1 << c.log_page;
    auto run = [&](auto kernel) { return launch(kernel, grid, dim3(kThreads), stream, c, b, r, k, k_stride, v, v_stride); };
    if (c.dim == 128) return page <= 32 ? run(k_kv_write<128, 1>) : page == 64 ? run(k_kv_write<128, 2>) : run(k_kv_write<128, 4>);
    return page <= 64 ? run(k_kv_write<64, 1>) : run(k_kv_write<64, 2>);
}

hipError_t launch_kv_read(const KvCacheArgs& c, const KvBatchArgs& b, uint16_t* k, uint16_t* v, hipStream_t stream) {
    const dim3 grid((uint32_t)(kv_items(b, c.log_page) * c.kv_heads));
    if (c.dim == 128) return launch(k_kv_read<128>, grid, dim3(kThreads), stream, c, b, k, v);
    return launch(k_kv_read<64>, grid, dim3(kThreads), stream, c, b, k, v);
}

}  // namespace focus
