// focus_attention.hip -- attention over the paged 8-bit cache of keys and
// values (focus_kv.hip) on gfx950 matrix cores:
//     y_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(cap(scale q_i . k_j) - m_i)
// over the tokens j of row i's sequence with pos_i - window < j <= pos_i, in
// one pass with a running maximum m and sum.  Heads of the queries that share
// a head of the cache are rows of one tile: row r of a sequence is its token
// r / group and head r % group, so the cache is read once for all of them.
//
// Numbers.  Keys enter as FP16, which holds every E4M3 code exactly; their
// page's power of two goes into the factor that takes a score to base 2
// (16 tokens of a page share it).  Queries enter as FP16 too, times a power of
// two per row that brings the row's largest element to 2^14..2^15: a BF16 query
// loses nothing that is above 2^-28 of that largest one; a turned one keeps 22
// bits in two parts where a sequence has few rows, and 11 otherwise.  Scores,
// maxima, sums and results are binary32.  Probabilities
// meet the values in BF16: values are exact in it with their page's scale
// (an operand of the conversion) down to BF16's least, 2^-133, where FP16 would
// not hold them.
//
// Both products are formed transposed, S^T = K Q^T and Y^T = V^T P^T: a lane
// then holds scores of one query row (its column), and the four or eight
// tokens that it holds are those that the second product wants from it, so P
// goes from one product to the next in registers.
//
// Measured: one token over 131072, 64/8 heads of 128: 59-63 us with the join (4.4
// TB/s); 64 tokens over up to 16384, 32/8 heads of 128: 210-244 us (4.7-5.4 TB/s;
// HBM); a prompt of 8192 tokens, 32/8 heads of 128: 576-616 us (0.89-0.95
// PFLOP/s; matrix units 43 % and vector units 53 % busy).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "focus_kv.h"
#include "focus_launch.h"
#include "focus_numerics.h"

namespace focus {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kShortRows = 64;  // rows (tokens x group) up to which a sequence is split over its keys

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Eight E4M3 codes in FP16 (exact).
__device__ __forceinline__ f16x8 widen_f16(uint32_t lo, uint32_t hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return (f16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight E4M3 codes times S, a power of two, in BF16.
__device__ __forceinline__ bf16x8 widen_bf16(uint32_t lo, uint32_t hi, float S) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, S, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, S, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, S, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, S, true);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float e8m0_f32(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// Bytes of a dword whose E4M3 code is NaN (0x7F or 0xFF): their bit 7, moved to bit 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t c) {
    const uint32_t m = c & 0x7F7F7F7Fu;
    return ((m + 0x01010101u) >> 7) & 0x01010101u;
}

__device__ __forceinline__ bool any_nan(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t m = 0x7F7F7F7Fu, o = 0x01010101u;
    return ((((a & m) + o) | ((b & m) + o) | ((c & m) + o) | ((d & m) + o)) & 0x80808080u) != 0;
}

// The larger of a lane's value and that of the lane 32 from it (the exchange of
// a register with itself gives the lower lanes' values and the upper ones').
__device__ __forceinline__ float max_halves(float x) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// acc + the two BF16 values of a pair.
__device__ __forceinline__ float sum_pair(uint32_t pair, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x3F803F80u), acc, false);
}

// The first n (0..4, or beyond) bytes of a dword.
__device__ __forceinline__ uint32_t first_bytes(int n) { return n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u; }

// A query row's elements d .. d+7 and their partners d + dim/2 .., turned.
__device__ __forceinline__ void turn8(float (&lo)[8], float (&hi)[8], const RopeArgs& rope, int dim, int pos, int d) {
    const int half = dim / 2;
    const bool known = pos >= 0 && pos < rope.positions;
    const float* t = rope.table + (known ? (int64_t)pos * dim + d : 0);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 c = *reinterpret_cast<const float4*>(t + i), s = *reinterpret_cast<const float4*>(t + half + i);
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = lo[i + j], b = hi[i + j];
            lo[i + j] = known ? a * cs[j] - b * sn[j] : __builtin_nanf("");
            hi[i + j] = known ? b * cs[j] + a * sn[j] : __builtin_nanf("");
        }
    }
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), f); }

// The exponent that brings a row of largest magnitude amax to 2^14..2^15.
__device__ __forceinline__ int query_shift(float amax) {
    if (!(amax > 0.0f) || !(amax < __builtin_inff())) return 0;
    return 15 - __builtin_amdgcn_frexp_expf(amax);
}

// The products with exponents up to 2^15 and 2^8 over 128 elements stay far
// within binary32.
__device__ __forceinline__ f16x8 narrow(const float (&f)[8], int shift, float sign) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (_Float16)(sign * __builtin_ldexpf(f[i], shift));
    return r;
}

// What the scores' factor and cap need of the call.
struct Scoring {
    float c0;    // to base 2; not negative
    float sign;  // of the scale, given to the queries
    float cap2;  // the cap to base 2, 0 without one
    float inv;   // 1 / cap2
};

// Score times this is to base 2: c0 * 2^(e - shift), e the exponent of the
// key's page.  Kept normal and finite, so that a score of minus
// infinity, a hidden one's, stays it and 0 stays 0.
__device__ __forceinline__ float score_factor(float c0, int e, int shift) {
    return __builtin_amdgcn_fmed3f(__builtin_ldexpf(c0, e - shift), 1.1754944e-38f, 3.4028235e38f);
}

// A maximum is replaced only by one that is 2^kSlack above it (base 2), so that a
// result is rescaled a few times instead of at every new maximum.
// Probabilities are taken 2^kSlack smaller, which the quotient does not see: they
// stay at most 1, so that the values' sums leave binary32 no sooner than with an
// exact maximum (at 2^kSlack, values from 2^112 on could reach infinity).
constexpr float kSlack = 8.0f;

// What the exponents are taken from, of a running maximum.
__device__ __forceinline__ float exponent_base(float m) { return m == -__builtin_inff() ? 0.0f : m + kSlack; }

// N scores to cap tanh(s / cap), all to base 2, with an error relative to the
// result (26 u by its roundings, u = 2^-24) whatever the cap.  tanh(x) =
// 1 - 2 / (exp(2 x) + 1) cancels near 0, by 1 / x.  Below 0.75 an odd polynomial
// (x to x^11, the best on that range: 0.55 u off) stands beside s itself, so
// that a cap far above every score leaves the score as it is.  A wavefront whose
// scores are all there, as they mostly are, saves the exponential and the
// reciprocal of each (prompt of 8192, cap 30, 32/8 heads of 128: 751 us; the
// exponential for every score 780, both for every score 962).
constexpr float kCapNear = 0.75f;

__device__ __forceinline__ float capped_near(float s, float x) {
    const float z = x * x;
    float p = __builtin_fmaf(z, -0.0047694305f, 0.019664839f);
    p = __builtin_fmaf(p, z, -0.053390227f);
    p = __builtin_fmaf(p, z, 0.13326521f);
    p = __builtin_fmaf(p, z, -0.33333069f);
    return __builtin_fmaf(s * z, p, s);
}

template <int N>
__device__ __forceinline__ void cap_scores(float (&s)[N], const Scoring& sc) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(s[i]));
    if (__any(top * sc.inv >= kCapNear)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = s[i] * sc.inv, near = capped_near(s[i], x);
            const float far = sc.cap2 * (1.0f - 2.0f * __builtin_amdgcn_rcpf(exp2_hw(x * (2.0f * kLog2e)) + 1.0f));
            s[i] = fabsf(x) >= kCapNear ? far : near;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = capped_near(s[i], s[i] * sc.inv);
    }
}

inline Scoring scoring(const KvAttentionArgs& a) {
    const float mag = a.scale < 0.0f ? -a.scale : a.scale, sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;
    Scoring sc = {mag * kLog2e, sign, 0.0f, 0.0f};
    if (a.softcap > 0.0f) {
        // kept finite: of larger caps nothing to base 2 is left to cap, and no
        // score moves a weight under smaller ones
        const double most = 3.4028234e38, cap2 = (double)a.softcap * 1.4426950408889634;
        sc.cap2 = (float)(cap2 < most ? cap2 : most);
        sc.inv = (float)(1.0 / cap2 < most ? 1.0 / cap2 : most);
    }
    return sc;
}

// ---------------------------------------------------------------------------
// few rows per sequence: split over the keys
// ---------------------------------------------------------------------------
//
// A sequence's rows are taken 16 at a time (a tile).  Where the tiles' keys are
// many, they are cut, one tile after the other, into ranges of equal length, one
// for each workgroup of a head that the GPU holds at once, so that all of them
// end together whatever the sequences' lengths; a workgroup goes through the
// pieces of the tiles in its range.  Where they are few, a workgroup takes a
// tile's piece of at most the least length, which a range of several tiles would
// take one after the other.  The lengths are device memory: every workgroup adds
// them up and finds its own.  A tile of several pieces leaves unnormalised sums,
// and their maximum, in the workspace, and a second kernel joins them in order.
// (Measured, us: 64 sequences up to 16384 with chunks of equal length handed out
// in turn 251, with ranges 240; 40 up to 2000 with ranges 29, with pieces 18.)

struct ShortPlan {
    int ranges;  // per head; 0: no split, tiles are handed out in turn
    int slots;   // pieces per head, at most
    int waves;   // of a workgroup
    int resident;  // workgroups that the GPU holds at once
};

constexpr int kShortStep = 64;    // keys of a wavefront's step, the unit of the lengths here

// Steps that a range is a multiple of, and the least: shorter ones cost more in
// the join (4 us) than they save.
constexpr int kRangeUnit = 8, kLeastRange = 24;

struct ShortSequence {
    KvSequence s;
    int begin, end;  // keys that some row sees, begin a multiple of 64
    int tiles;       // 0: no rows, or too many
    __device__ __forceinline__ int span() const { return max((end - begin + kShortStep - 1) / kShortStep, 1); }  // steps
};

__device__ __forceinline__ bool is_short(int rows, int group) { return rows == 1 || (int64_t)rows * group <= kShortRows; }

__device__ __forceinline__ ShortSequence short_sequence(const KvAttentionArgs& a, int group, int i) {
    ShortSequence q;
    q.s = kv_sequence(a.batch, i);
    const int64_t room = (int64_t)a.batch.max_pages << a.cache.log_page;
    const int64_t first = q.s.first();
    q.end = (int)(q.s.length < room ? q.s.length : room);
    q.begin = 0;
    if (a.window > 0 && first >= a.window) q.begin = (int)min((first - a.window + 1) & ~(int64_t)(kShortStep - 1), (int64_t)q.end);
    q.tiles = q.s.rows > 0 && is_short(q.s.rows, group) ? (q.s.rows * group + 15) / 16 : 0;
    return q;
}

// Tiles of a sequence, and what each of them counts.
struct Weighed {
    int tiles, weight;
};

// What a tile counts here: one, its steps, or its pieces of the least length.
enum Count { kTiles, kSteps, kPieces };

__device__ __forceinline__ int weight(const ShortSequence& q, Count of) {
    return of == kTiles ? 1 : of == kSteps ? q.span() : (q.span() + kLeastRange - 1) / kLeastRange;
}

__device__ __forceinline__ auto weigh_short(const KvAttentionArgs& a, int group, Count of) {
    return [&a, group, of](int i) {
        const ShortSequence q = short_sequence(a, group, i);
        return Weighed{q.tiles, weight(q, of)};
    };
}

// Over the sequences before `seq`; the host has seen to it that 32 bits hold it
// where every row is of one sequence.  Offsets that count rows many times can wrap
// it: find_tile then finds nothing before the first tile, and a slot that is none
// of the workspace's, negative ones too, is not used.
struct Sum {
    int weight, tiles;
};

template <typename F>
__device__ __forceinline__ Sum sum_before(int seq, F weigh) {
    const int lane = threadIdx.x & 63;
    Sum n = {0, 0};
    for (int base = 0; base < seq; base += 64)
        if (base + lane < seq) {
            const Weighed w = weigh(base + lane);
            n.weight += w.weight * w.tiles;
            n.tiles += w.tiles;
        }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        n.weight += __shfl_xor(n.weight, m);
        n.tiles += __shfl_xor(n.tiles, m);
    }
    return n;
}

// The tile that holds a place in the row of all tiles, its number, its weight
// and the place within it.
struct Tile {
    int seq, tile, number, weight, rest;
};

template <typename F>
__device__ __forceinline__ bool find_tile(int sequences, int place, Tile& out, F weigh) {
    const int lane = threadIdx.x & 63;
    int before = 0, tiles_before = 0;
    for (int base = 0; base < sequences; base += 64) {
        const Weighed w = base + lane < sequences ? weigh(base + lane) : Weighed{0, 1};
        int upto = w.tiles * w.weight, tiles_upto = w.tiles;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int n = __shfl_up(upto, m), k = __shfl_up(tiles_upto, m);
            upto += lane >= m ? n : 0;
            tiles_upto += lane >= m ? k : 0;
        }
        const uint64_t past = __ballot(place < before + upto);
        if (past) {
            const int at = __builtin_ctzll(past);
            out.seq = base + at;
            out.weight = __builtin_amdgcn_readlane(w.weight, at);
            const int rel = place - (before + __builtin_amdgcn_readlane(upto - w.tiles * w.weight, at));
            if (rel < 0) return false;
            out.tile = rel / out.weight;
            out.rest = rel - out.tile * out.weight;
            out.number = tiles_before + __builtin_amdgcn_readlane(tiles_upto - w.tiles, at) + out.tile;
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
        tiles_before += __builtin_amdgcn_readlane(tiles_upto, 63);
    }
    return false;
}

// Steps of a range, or 0 where pieces are taken instead.
__device__ __forceinline__ int range_length(const KvAttentionArgs& a, const ShortPlan& pl, int group) {
    const int steps = sum_before(a.batch.sequences, weigh_short(a, group, kSteps)).weight;
    const int each = (steps + pl.ranges - 1) / pl.ranges;
    return each > kLeastRange ? (each + kRangeUnit - 1) / kRangeUnit * kRangeUnit : 0;
}

// Whether a tile's pieces have places in the workspace: always, but for rows that
// cu_tokens counts twice.
__device__ __forceinline__ bool has_slots(int slot0, int count, int slots) {
    return slot0 >= 0 && count >= 0 && (int64_t)slot0 + count <= slots;
}

// Workspace: per slot, head and row of 16 the sums [dim], then per slot, head
// and row the maximum (base 2) and the sum of the probabilities.  The piece of
// tile i in range k has slot i + k: going from piece to piece one of them grows.
// Pieces of the least length have their number.
__device__ __forceinline__ float* part_at(const KvAttentionArgs& a, int slot, int head, int row) {
    return a.workspace + (((int64_t)slot * a.cache.kv_heads + head) * 16 + row) * a.cache.dim;
}
__device__ __forceinline__ float2* part_stat(const KvAttentionArgs& a, int slots, int slot, int head, int row) {
    float* p = a.workspace + (int64_t)slots * a.cache.kv_heads * 16 * a.cache.dim;
    return reinterpret_cast<float2*>(p) + ((int64_t)slot * a.cache.kv_heads + head) * 16 + row;
}

// A piece of a tile: its steps from .. from + length - 1, slot -1: all of them.
struct Piece {
    int seq, tile, slot, from, length;
};

// What a row's sum becomes: no key (zeros), keys that have no page (NaN).
__device__ __forceinline__ float row_result(float sum, float total, int64_t pos, int64_t room) {
    if (pos < 0) return 0.0f;
    return pos < room ? sum / total : __builtin_nanf("");
}

template <int D, int WAVES>
struct ShortLds {
    static constexpr int kRow = D + 4;
    __attribute__((aligned(16))) float out[WAVES][16 * kRow];
    float2 stat[WAVES][16];
};

// One piece, by WAVES wavefronts.
template <int D, int WAVES>
__device__ __forceinline__ void short_piece(const KvAttentionArgs& a, const ShortPlan& pl, const Scoring& sc, const Piece& sh,
                                            int head, ShortLds<D, WAVES>& lds) {
    constexpr int kQ = D / 32;       // products per 16 tokens
    constexpr int kV = D / 16;       // tiles of the result
    constexpr int kOutRow = ShortLds<D, WAVES>::kRow, kStride = WAVES * kShortStep;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int x = lane & 15, c = lane >> 4;
    const int kvh = a.cache.kv_heads, group = a.heads / kvh;
    ShortSequence sq = short_sequence(a, group, sh.seq);
    sq.s.row0 = __builtin_amdgcn_readfirstlane(sq.s.row0);
    sq.s.rows = __builtin_amdgcn_readfirstlane(sq.s.rows);
    sq.begin = __builtin_amdgcn_readfirstlane(sq.begin);
    sq.end = __builtin_amdgcn_readfirstlane(sq.end);
    const int rows = sq.s.rows * group;
    const int log_page = a.cache.log_page, page = 1 << log_page;
    const int first = __builtin_amdgcn_readfirstlane((int)sq.s.first());

    // the lane's query row
    const int r = 16 * sh.tile + x, token = min(r, rows - 1) / group, member = min(r, rows - 1) - token * group;
    const int pos = r < rows ? first + token : -1;
    const int pos_lo = first + 16 * sh.tile / group, pos_hi = first + min(16 * sh.tile + 15, rows - 1) / group;

    const int jlo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    const int begin = min(sq.begin + sh.from * kShortStep, sq.end);
    const int end = min(sq.end, begin + sh.length * kShortStep);
    const int jhi = min(pos, end - 1);
    // keys that every row of the tile sees, and that any sees
    const int all_lo = a.window > 0 ? max(pos_hi - a.window + 1, 0) : 0, all_hi = min(pos_lo, end - 1);
    const int any_lo = a.window > 0 ? max(pos_lo - a.window + 1, 0) : 0, any_hi = min(pos_hi, end - 1);

    const int* table = a.batch.table + (int64_t)sh.seq * a.batch.table_stride;
    const int kgroup = 16 * (x >> 2);  // tokens that the lane's keys are of, within a step; its scores and values: 16 c

    uint4 kb[4][D / 64];
    uint4 vb[kV];
    bool has_page = false;
    uint32_t ks = 0, vs = 0;

    // The table's entries are read two steps ahead and looked at only where
    // they are used; behind the last key that of the last one, whose page the
    // masks hide.
    auto entry_of = [&](int t) { return table[min(t, end - 1) >> log_page]; };
    auto is_page = [&](int e) { return e >= 0 && e < a.cache.pages; };
    auto load_k = [&](int t, int e) {
        const int j = t + kgroup;
        const uint8_t* p = a.cache.kc + (((int64_t)(is_page(e) ? e : 0) * kvh + head) * page + (j & (page - 1)) + (x & 3)) * D + c * (D / 4);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) kb[g][i] = *reinterpret_cast<const uint4*>(p + 4 * g * D + 16 * i);
    };
    auto load_v = [&](int t, int e) {
        const int j = t + 16 * c;
        const uint8_t* p = a.cache.vc + (((int64_t)(is_page(e) ? e : 0) * kvh + head) * D + x) * page + (j & (page - 1));
#pragma unroll
        for (int i = 0; i < kV; ++i) vb[i] = *reinterpret_cast<const uint4*>(p + (int64_t)16 * i * page);
    };
    auto load_s = [&](int e) {
        has_page = is_page(e);
        const int64_t at = (int64_t)(has_page ? e : 0) * kvh + head;
        ks = a.cache.ks[at];
        vs = a.cache.vs[at];
    };

    f32x4 acc[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = (f32x4){};
    float m = -__builtin_inff(), l = 0.0f;

    // Loads that wait for nothing first: the table's entries, the query and its angles.
    int t = begin + kShortStep * wave;
    int k0 = 0, v0 = 0, ke = 0, ve = 0;  // entries of this step and the next
    if (t < end) {
        k0 = entry_of(t + kgroup);
        v0 = entry_of(t + 16 * c);
        ke = entry_of(t + kStride + kgroup);
        ve = entry_of(t + kStride + 16 * c);
    }
    // The queries, and what their rounding leaves of turned ones, whose products
    // cost 0 to 4 % where the cache is streamed and 0.3 to 0.7 us of 8.3 and 11.4
    // for one token over 333.  That is in registers (dim 64: 124 us for 64 tokens
    // over up to 16384, in LDS 127) or in LDS, where the wavefront's result goes in
    // the end and each lane reads what it wrote (dim 128: 1 x 131072 62.5 us, with
    // registers that spill 69).
    constexpr bool kInLds = D == 128;
    static_assert(sizeof(f16x8) * 64 * kQ <= sizeof(lds.out[0]), "room for the rest of the queries");
    f16x8 q[kQ], left[kInLds ? 1 : kQ];
    auto* kept = (__attribute__((address_space(3))) f16x8*)lds.out[wave] + lane;
    int shift;
    {
        const uint16_t* qp = a.q + (int64_t)(sq.s.row0 + token) * a.q_stride + (int64_t)(head * group + member) * D + c * (D / 4);
        float f[kQ][8];
        uint4 raw[kQ];
#pragma unroll
        for (int k = 0; k < kQ; ++k) raw[k] = *reinterpret_cast<const uint4*>(qp + 8 * k);
        float4 cs[kQ][2], sn[kQ][2];
        const int place = first + token;
        const bool known = place >= 0 && place < a.rope.positions;
        if (a.rope.table) {
            const float* angle = a.rope.table + (known ? (int64_t)place * D : 0) + (c & 1) * (D / 4);
#pragma unroll
            for (int k = 0; k < kQ; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    cs[k][i] = *reinterpret_cast<const float4*>(angle + 8 * k + 4 * i);
                    sn[k][i] = *reinterpret_cast<const float4*>(angle + D / 2 + 8 * k + 4 * i);
                }
        }
        if (t < end) {
            load_k(t, k0);
            load_s(v0);
            load_v(t, v0);
        }
#pragma unroll
        for (int k = 0; k < kQ; ++k) unpack8(raw[k], f[k]);
        if (a.rope.table) {
            // lanes 32 apart hold a pair's halves: a c - b s on the first, b c + a s on the second
#pragma unroll
            for (int k = 0; k < kQ; ++k) {
                const float co[8] = {cs[k][0].x, cs[k][0].y, cs[k][0].z, cs[k][0].w, cs[k][1].x, cs[k][1].y, cs[k][1].z, cs[k][1].w};
                const float si[8] = {sn[k][0].x, sn[k][0].y, sn[k][0].z, sn[k][0].w, sn[k][1].x, sn[k][1].y, sn[k][1].z, sn[k][1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const u32x2 both = __builtin_amdgcn_permlane32_swap(__float_as_uint(f[k][i]), __float_as_uint(f[k][i]), false, false);
                    const float mine = f[k][i] * co[i], other = __uint_as_float(c < 2 ? both[1] : both[0]) * si[i];
                    const float turned = c < 2 ? mine - other : mine + other;
                    f[k][i] = known ? turned : __builtin_nanf("");
                }
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < kQ; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[k][i]));
        amax = fmaxf(amax, __shfl_xor(amax, 16));
        amax = max_halves(amax);
        shift = query_shift(amax);
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            q[k] = narrow(f[k], shift, sc.sign);
#pragma unroll
            for (int i = 0; i < 8; ++i) left[kInLds ? 0 : k][i] = (_Float16)(sc.sign * __builtin_ldexpf(f[k][i], shift) - (float)q[k][i]);
            if (kInLds) kept[64 * k] = left[0];
        }
    }

    while (t < end) {
        const int tn = t + kStride;
        const int ke_n = entry_of(tn + kStride + kgroup), ve_n = entry_of(tn + kStride + 16 * c);
        // scores: s[g][i] is of token t + 16 c + 4 g + i
        f32x4 s[4];
        f16x8 rest[kQ];
        if (kInLds) asm volatile("" : "+v"(kept));  // or the loads would move out of the loop, into registers
#pragma unroll
        for (int k = 0; k < kQ; ++k) rest[k] = kInLds ? kept[64 * k] : left[kInLds ? 0 : k];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            s[g] = (f32x4){};
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const f16x8 k0 = widen_f16(kb[g][i].x, kb[g][i].y), k1 = widen_f16(kb[g][i].z, kb[g][i].w);
                s[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[2 * i], s[g], 0, 0, 0);
                s[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[2 * i + 1], s[g], 0, 0, 0);
                s[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, rest[2 * i], s[g], 0, 0, 0);
                s[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, rest[2 * i + 1], s[g], 0, 0, 0);
            }
        }
        const bool here = has_page;
        const float factor = here ? score_factor(sc.c0, (int)ks - 127, shift) : __builtin_nanf("");
        const float vscale = e8m0_f32(vs);
        if (tn < end) {
            load_k(tn, ke);
            load_s(ve);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[g][i] *= factor;
        if (sc.cap2 > 0.0f) {
            float e[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = s[i / 4][i % 4];
            cap_scores(e, sc);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i / 4][i % 4] = e[i];
        }
        const bool whole = t >= all_lo && t + kShortStep - 1 <= all_hi;
        if (!whole) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = t + 16 * c + 4 * g + i;
                    s[g][i] = j >= jlo && j <= jhi ? s[g][i] : -__builtin_inff();
                }
        }
        float mt = -__builtin_inff();
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) mt = fmaxf(mt, s[g][i]);
        mt = fmaxf(mt, __shfl_xor(mt, 16));
        mt = max_halves(mt);
        if (__any(mt > m + kSlack)) {
            const float mn = fmaxf(m, mt);
            const float alpha = mn > m ? exp2_hw(m - mn) : 1.0f;
            m = mn;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] *= alpha;
        }
        const float mu = exponent_base(m);
        // P in two BF16 parts, so that its rounding does not show in the result
        bf16x8 ph[2], pr[2];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = exp2_hw(s[g][i] - mu);
                l += p;
                const __bf16 h = (__bf16)p;
                ph[g >> 1][4 * (g & 1) + i] = h;
                pr[g >> 1][4 * (g & 1) + i] = (__bf16)(p - (float)h);
            }
        bool odd = false;
        if (!whole) {
            // values of tokens that no row sees are whatever the page holds
            uint32_t keep[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = t + 16 * c + 4 * k;
                keep[k] = here ? first_bytes(any_hi + 1 - j) & ~first_bytes(any_lo - j) : 0u;
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                vb[i].x &= keep[0];
                vb[i].y &= keep[1];
                vb[i].z &= keep[2];
                vb[i].w &= keep[3];
                odd = odd || any_nan(vb[i].x, vb[i].y, vb[i].z, vb[i].w);
            }
        }
        if (!whole && __any(odd)) {
            // A NaN value reaches exactly the rows that see its token: count
            // such tokens per row by a product of ones.
            bf16x8 seen[2];
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = t + 16 * c + 4 * g + i;
                    seen[g >> 1][4 * (g & 1) + i] = (__bf16)(j >= jlo && j <= jhi ? 1.0f : 0.0f);
                }
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                uint32_t w[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w}, n[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t b = nan_bytes(w[k]);
                    n[k] = b * 0x38u;  // the code of 1
                    w[k] &= ~(b * 0xFFu);
                }
                vb[i] = make_uint4(w[0], w[1], w[2], w[3]);
                f32x4 cnt = {};
                cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_bf16(n[0], n[1], 1.0f), seen[0], cnt, 0, 0, 0);
                cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_bf16(n[2], n[3], 1.0f), seen[1], cnt, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][k] = cnt[k] > 0.0f ? __builtin_nanf("") : acc[i][k];
            }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bf16x8 v0 = widen_bf16(vb[i].x, vb[i].y, vscale), v1 = widen_bf16(vb[i].z, vb[i].w, vscale);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, ph[0], acc[i], 0, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, ph[1], acc[i], 0, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pr[0], acc[i], 0, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pr[1], acc[i], 0, 0, 0);
        }
        if (tn < end) load_v(tn, ve);
        ke = ke_n;
        ve = ve_n;
        t = tn;
    }

    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (c == 0) lds.stat[wave][x] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < kV; ++i) *reinterpret_cast<f32x4*>(&lds.out[wave][x * kOutRow + 16 * i + 4 * c]) = acc[i];
    __syncthreads();
    const int64_t room = (int64_t)a.batch.max_pages << log_page;
    for (int i = tid; i < 16 * (D / 4); i += 64 * WAVES) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4)), rr = 16 * sh.tile + row;
        if (rr >= rows) continue;
        float mx = lds.stat[0][row].x;
#pragma unroll
        for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, lds.stat[w][row].x);
        float total = 0.0f;
        f32x4 o = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = mx == -__builtin_inff() ? 0.0f : exp2_hw(lds.stat[w][row].x - mx);
            total += f * lds.stat[w][row].y;
            o += f * *reinterpret_cast<const f32x4*>(&lds.out[w][row * kOutRow + d]);
        }
        if (sh.slot < 0) {
            const int tok = rr / group, mem = rr - tok * group;
            const int64_t p = (int64_t)first + tok;
            uint2 v;
            v.x = bf16_pair(row_result(o[0], total, p, room), row_result(o[1], total, p, room));
            v.y = bf16_pair(row_result(o[2], total, p, room), row_result(o[3], total, p, room));
            *reinterpret_cast<uint2*>(a.y + ((int64_t)(sq.s.row0 + tok) * a.heads + head * group + mem) * D + d) = v;
        } else {
            *reinterpret_cast<f32x4*>(part_at(a, sh.slot, head, row) + d) = o;
            if (d == 0) *part_stat(a, pl.slots, sh.slot, head, row) = make_float2(mx, total);
        }
    }
}

// The pieces of range w / kv_heads of a head, or every stride-th piece or tile
// of all heads.
template <int D, int WAVES>
__device__ __forceinline__ void short_pieces(const KvAttentionArgs& a, const ShortPlan& pl, const Scoring& sc, int w, int stride,
                                             ShortLds<D, WAVES>& lds) {
    const int kvh = a.cache.kv_heads, group = a.heads / kvh;
    const int length = pl.ranges > 0 ? range_length(a, pl, group) : 0;
    const Count of = length > 0 ? kSteps : pl.ranges > 0 ? kPieces : kTiles;
    int range = w / kvh, place = length > 0 ? range * length : range;
    const int head = w % kvh, stop = place + length;
    for (;;) {
        Tile t;
        if (of == kTiles && !a.batch.cu) {
            // as many tiles of every sequence: no length is waited for (1 x 333
            // 11.7 us, searched 13.1, with turned queries in one part)
            const int per = (group + 15) / 16;
            t.seq = __builtin_amdgcn_readfirstlane(place / per);
            if (t.seq >= a.batch.sequences) return;
            t.tile = place - t.seq * per;
        } else if (!find_tile(a.batch.sequences, place, t, weigh_short(a, group, of))) {
            return;
        }
        Piece p = {__builtin_amdgcn_readfirstlane(t.seq), __builtin_amdgcn_readfirstlane(t.tile), -1, 0, 1 << 24};
        if (length > 0) {
            p.from = __builtin_amdgcn_readfirstlane(t.rest);
            p.length = __builtin_amdgcn_readfirstlane(min(t.weight - t.rest, stop - place));
            if (p.length < t.weight) p.slot = t.number + range;
            place += p.length;
        } else if (of == kPieces && t.weight > 1) {
            p.from = t.rest * kLeastRange;
            p.length = kLeastRange;
            p.slot = place;
        }
        // rows that cu_tokens counts twice have no slot
        if (p.slot >= pl.slots || p.slot < -1) return;
        short_piece<D, WAVES>(a, pl, sc, p, length > 0 ? head : w % kvh, lds);
        if (length > 0) {
            if (place >= stop) return;
        } else {
            w += stride;
            place = w / kvh;
        }
        __syncthreads();  // the next piece writes where this one has read
    }
}

template <int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void k_attention_short(KvAttentionArgs a, ShortPlan pl, Scoring sc) {
    __shared__ ShortLds<D, WAVES> lds;
    short_pieces<D, WAVES>(a, pl, sc, (int)blockIdx.x, (int)gridDim.x, lds);
}

// A workgroup joins the pieces of rows of one sequence and head, in order:
// `each` workgroups share a sequence's rows, four wavefronts the pieces.
template <int D>
__global__ __launch_bounds__(256) void k_attention_join(KvAttentionArgs a, ShortPlan pl, int each) {
    constexpr int kPer = D / 64;  // elements of a lane
    __shared__ float part[4][D];
    __shared__ float2 sums[4];
    const int kvh = a.cache.kv_heads, group = a.heads / kvh;
    const int head = (int)(blockIdx.x % (uint32_t)kvh), seq = (int)(blockIdx.x / (uint32_t)kvh / (uint32_t)each);
    const ShortSequence sq = short_sequence(a, group, seq);
    if (sq.tiles == 0) return;
    const int length = range_length(a, pl, group);
    const Sum before = sum_before(seq, weigh_short(a, group, length > 0 ? kSteps : kPieces));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int row = (int)(blockIdx.x / (uint32_t)kvh % (uint32_t)each); row < sq.s.rows * group; row += each) {
        const int tile = row / 16, r = row % 16;
        int slot0, count;
        if (length > 0) {
            const int start = before.weight + tile * sq.span(), first = start / length;
            count = (start + sq.span() - 1) / length - first + 1;
            slot0 = before.tiles + tile + first;
        } else {
            count = weight(sq, kPieces);
            slot0 = before.weight + tile * count;
        }
        if (count == 1 || !has_slots(slot0, count, pl.slots)) continue;
        // eight pieces at a time, so that their loads are in flight together
        constexpr int kBatch = 8;
        float m = -__builtin_inff(), total = 0.0f, o[kPer] = {};
        for (int i = wave; i < count; i += 4 * kBatch) {
            float2 st[kBatch];
            float p[kBatch][kPer];
#pragma unroll
            for (int n = 0; n < kBatch; ++n) {
                const int slot = slot0 + min(i + 4 * n, count - 1);
                st[n] = *part_stat(a, pl.slots, slot, head, r);
                const float* from = part_at(a, slot, head, r) + kPer * lane;
#pragma unroll
                for (int k = 0; k < kPer; ++k) p[n][k] = from[k];
                if (i + 4 * n >= count) st[n] = make_float2(-__builtin_inff(), 0.0f);
            }
            float mn = m;
#pragma unroll
            for (int n = 0; n < kBatch; ++n) mn = fmaxf(mn, st[n].x);
            const float keep = m == -__builtin_inff() ? (total == 0.0f ? 0.0f : 1.0f) : exp2_hw(m - mn);
            total *= keep;
#pragma unroll
            for (int k = 0; k < kPer; ++k) o[k] *= keep;
            m = mn;
#pragma unroll
            for (int n = 0; n < kBatch; ++n) {
                if (i + 4 * n >= count) break;
                const float f = mn == -__builtin_inff() ? 0.0f : exp2_hw(st[n].x - mn);
                total += f * st[n].y;
#pragma unroll
                for (int k = 0; k < kPer; ++k) o[k] += f * p[n][k];
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) part[wave][kPer * lane + k] = o[k];
        if (lane == 0) sums[wave] = make_float2(m, total);
        __syncthreads();
        if (threadIdx.x < D) {
            const int d = threadIdx.x, token = row / group, member = row - token * group;
            float mx = sums[0].x;
#pragma unroll
            for (int w = 1; w < 4; ++w) mx = fmaxf(mx, sums[w].x);
            float sum = 0.0f, all = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = mx == -__builtin_inff() ? 0.0f : exp2_hw(sums[w].x - mx);
                all += f * sums[w].y;
                sum += f * part[w][d];
            }
            const float res = row_result(sum, all, sq.s.first() + token, (int64_t)a.batch.max_pages << a.cache.log_page);
            a.y[((int64_t)(sq.s.row0 + token) * a.heads + head * group + member) * D + d] = (uint16_t)bf16_pair(res, 0.0f);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// many rows per sequence
// ---------------------------------------------------------------------------
//
// A workgroup owns 256 rows of one sequence and head (128 where that leaves
// compute units idle) and goes over their keys in tiles of 64.  Keys and values
// are widened once per workgroup on their way to LDS, so that the conversions
// cost a wavefront little beside its products, and each of 8 (4) wavefronts
// multiplies them with its 32 rows.  A tile's global
// loads are in flight while the tile before is multiplied.  250 registers leave
// two wavefronts per SIMD.  What bounds it: 32 products and 240 vector
// instructions per 64 keys and wavefront, which take turns (matrix units 43 %
// and vector units 53 % busy add up to the whole time: a barrier per step keeps
// both wavefronts in the same part of it), and the clock, which falls to about
// 2.1 GHz.  Steps, us for a prompt
// of 8192 tokens, 32/8 heads of 128: table's entry loaded and looked at in each
// step, branch for NaN values in the loop 1050; entries and scales from lanes,
// NaN counted after the loop 612; lanes' equal values scalar 588.  Wavefront
// groups half a step apart: no gain.

// masks of the scheduler's groups
constexpr int kProducts = 0x008, kReads = 0x100;

constexpr int kWaveRows = 32, kLongKeys = 64;

struct LongPlan {
    int target;  // pieces per head to aim at; 0: no split
    int slots;   // pieces per head, at most
    int tiles;   // at most
    int waves;   // of a workgroup, each with kWaveRows rows of a tile
};

// Steps of a piece, at least, and the keys up to which nothing is split (64 tiles
// of 512 keys, us split and whole: 25 and 18 at dim 64, 31 and 24 at 128).
constexpr int kLeastPiece = 8, kLeastSplit = 1024;

// A sequence's tiles of R rows (0: few rows, or none), and the steps of
// the one that sees the most keys.
template <int R>
__device__ __forceinline__ Weighed long_sequence(const KvAttentionArgs& a, int group, int i) {
    const KvSequence s = kv_sequence(a.batch, i);
    const int64_t room = (int64_t)a.batch.max_pages << a.cache.log_page;
    int64_t keys = min(s.length, room);
    if (a.window > 0) keys = min(keys, (int64_t)a.window + R + kLongKeys);
    const bool is_long = s.rows > 0 && !is_short(s.rows, group);
    return {is_long ? (s.rows * group + R - 1) / R : 0, (int)((keys + kLongKeys - 1) / kLongKeys)};
}

// Steps of a piece: as many as give the pieces aimed at.
template <int R>
__device__ __forceinline__ int piece_length(const KvAttentionArgs& a, const LongPlan& pl, int group) {
    if (pl.target == 0) return 1 << 24;
    const int steps = sum_before(a.batch.sequences, [&](int i) { return long_sequence<R>(a, group, i); }).weight;
    return max((steps + pl.target - 1) / pl.target, kLeastPiece);
}

// Pieces that every tile of a sequence has places for.
template <int R>
__device__ __forceinline__ auto weigh_long(const KvAttentionArgs& a, int group, int length) {
    return [&a, group, length](int i) {
        const Weighed w = long_sequence<R>(a, group, i);
        return Weighed{w.tiles, max((w.weight + length - 1) / length, 1)};
    };
}

// Keys that some row of a tile sees, and the pieces that these are.
struct LongTile {
    int begin, end, pieces;
};

template <int R>
__device__ __forceinline__ LongTile long_tile(const KvAttentionArgs& a, int group, const KvSequence& s, int tile, int length) {
    const int rows = s.rows * group, row0 = tile * R, first = (int)s.first();
    const int g_lo = first + row0 / group, g_hi = first + min(row0 + R - 1, rows - 1) / group;
    const int64_t room = (int64_t)a.batch.max_pages << a.cache.log_page;
    LongTile t;
    t.end = (int)min((int64_t)g_hi + 1, min(s.length, room));
    t.begin = a.window > 0 ? max(g_lo - a.window + 1, 0) & ~(kLongKeys - 1) : 0;
    const int steps = max(t.end - t.begin + kLongKeys - 1, 0) / kLongKeys;
    t.pieces = max((steps + length - 1) / length, 1);
    return t;
}

// Workspace: per slot, head and row of a tile the sums [dim], then the maximum
// (base 2) and the sum of the probabilities.
template <int R>
__device__ __forceinline__ float* long_part(const KvAttentionArgs& a, int slot, int head, int row) {
    return a.workspace + (((int64_t)slot * a.cache.kv_heads + head) * R + row) * a.cache.dim;
}
template <int R>
__device__ __forceinline__ float2* long_stat(const KvAttentionArgs& a, int slots, int slot, int head, int row) {
    float* p = a.workspace + (int64_t)slots * a.cache.kv_heads * R * a.cache.dim;
    return reinterpret_cast<float2*>(p) + ((int64_t)slot * a.cache.kv_heads + head) * R + row;
}

// LDS places, in 16-byte pieces whose order within a row is exchanged so that
// 16 lanes that read one piece of 16 rows meet every bank once.
template <int D>
__device__ __forceinline__ int key_place(int token, int piece) {
    return D == 128 ? token * 16 + (piece ^ (token & 15)) : token * 8 + (piece ^ ((token >> 1) & 7));
}
__device__ __forceinline__ int value_place(int d, int piece) { return d * 8 + (piece ^ ((d >> 1) & 7)); }

template <int D>
struct LongLds {
    uint4 keys[2][kLongKeys * D / 8];
    uint4 values[2][kLongKeys * D / 8];
    int nan_seen;  // whether a value is NaN
};

// Piece `item / kv_heads` from behind of a head.
template <int D, bool CAP, int WAVES>
__device__ __forceinline__ void long_piece(const KvAttentionArgs& a, const LongPlan& pl, const Scoring& sc, uint32_t item, LongLds<D>& lds) {
    constexpr int kQ = D / 16;  // products per 32 keys
    constexpr int kV = D / 32;  // tiles of the result
    constexpr int R = kWaveRows * WAVES;
    auto& keys = lds.keys;
    auto& values = lds.values;
    int& nan_seen = lds.nan_seen;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int kvh = a.cache.kv_heads, group = a.heads / kvh;
    const int head = (int)(item % (uint32_t)kvh);
    // The last tiles of a sequence see the most keys: they go first.  What the
    // lanes have found alike is made scalar, or it would take vector registers.
    const int piece_steps = __builtin_amdgcn_readfirstlane(piece_length<R>(a, pl, group));
    const auto weigh = weigh_long<R>(a, group, piece_steps);
    const int count = min(__builtin_amdgcn_readfirstlane(sum_before(a.batch.sequences, weigh).weight), pl.slots);
    const int place = count - 1 - (int)(item / (uint32_t)kvh);
    Tile found;
    if (place < 0 || !find_tile(a.batch.sequences, place, found, weigh)) return;
    const int seq = __builtin_amdgcn_readfirstlane(found.seq);
    KvSequence s = kv_sequence(a.batch, seq);
    s.rows = __builtin_amdgcn_readfirstlane(s.rows);
    s.row0 = __builtin_amdgcn_readfirstlane(s.row0);
    LongTile tile = long_tile<R>(a, group, s, found.tile, piece_steps);
    tile.begin = __builtin_amdgcn_readfirstlane(tile.begin);
    tile.end = __builtin_amdgcn_readfirstlane(tile.end);
    tile.pieces = __builtin_amdgcn_readfirstlane(tile.pieces);
    if (found.rest >= tile.pieces) return;
    const int rows = s.rows * group, row0 = found.tile * R;
    const int log_page = a.cache.log_page, page = 1 << log_page;
    const int first = (int)s.first();
    const int64_t room = (int64_t)a.batch.max_pages << log_page;
    const int length = (int)min(s.length, room);

    const int r = row0 + 32 * wave + n;
    const int token = min(r, rows - 1) / group, member = min(r, rows - 1) - token * group;
    const int pos = first + token;
    // positions of the wavefront's first and last rows
    const int w_lo = first + min(row0 + 32 * wave, rows - 1) / group, w_hi = first + min(row0 + 32 * wave + 31, rows - 1) / group;

    f16x8 q[kQ];
    int shift;
    {
        const uint16_t* qp = a.q + (int64_t)(s.row0 + token) * a.q_stride + (int64_t)(head * group + member) * D + 8 * hf;
        float f[kQ][8];
#pragma unroll
        for (int k = 0; k < kQ; ++k) load8(qp + 16 * k, f[k]);
        if (a.rope.table) {
#pragma unroll
            for (int k = 0; k < kQ / 2; ++k) turn8(f[k], f[k + kQ / 2], a.rope, D, pos, 16 * k + 8 * hf);
        }
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < kQ; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[k][i]));
        amax = fmaxf(amax, __shfl_xor(amax, 32));
        shift = query_shift(amax);
#pragma unroll
        for (int k = 0; k < kQ; ++k) q[k] = narrow(f[k], shift, sc.sign);
    }
    const int jlo = a.window > 0 ? max(pos - a.window + 1, 0) : 0, jhi = min(pos, length - 1);
    const int all_lo = a.window > 0 ? max(w_hi - a.window + 1, 0) : 0, all_hi = min(w_lo, length - 1);
    // the piece's keys; every piece but the last ends with a step
    const int begin = tile.begin + (int)min((int64_t)found.rest * piece_steps * kLongKeys, (int64_t)1 << 30);
    const int end = (int)min((int64_t)tile.end, (int64_t)begin + (int64_t)piece_steps * kLongKeys);

    // What a wavefront loads of a tile: kParts times 16 bytes of a key per lane,
    // all of one 16-key group, and as many times 16 tokens of a row of values, of
    // one group too (8 wavefronts, dim 64: the first half of them the keys, the
    // other the values).  Page and address are then scalars, beside a lane's
    // constant offset.
    constexpr bool kBoth = D / WAVES >= 16;
    constexpr int kParts = kBoth ? D / WAVES / 16 : 1;
    const bool of_k = kBoth || wave < 4, of_v = kBoth || wave >= 4;
    constexpr int kGroupWaves = kBoth ? WAVES / 4 : 1;  // wavefronts of a group
    const int k_group = (kBoth ? wave : wave & 3) / kGroupWaves, v_group = wave & 3;
    constexpr int kPieces = D / 16;  // of a key
    const int k_token = 16 * k_group + 64 / kPieces * (kGroupWaves > 1 ? wave & 1 : 0) + lane / kPieces, k_piece = lane % kPieces;
    const int v_d = kGroupWaves > 1 ? 64 * (wave >> 2) + lane : lane;
    const uint32_t k_lane = (uint32_t)((k_token & (page - 1)) * D + 16 * k_piece), v_lane = (uint32_t)(v_d * page);
    const uint8_t* kc = a.cache.kc + (int64_t)head * page * D;
    const uint8_t* vc = a.cache.vc + (int64_t)head * page * D;
    const int64_t page_bytes = (int64_t)kvh * page * D;
    const int* table = a.batch.table + (int64_t)seq * a.batch.table_stride;

    // The table is read 1024 keys at a time, lane i the entry of the 16-key
    // group i (behind the last key that of the last one, whose page the masks
    // hide), and the groups' scales with it, well before they are used: a tile
    // then takes its pages and exponents from a lane, as scalars.
    struct Block {
        int page;  // -1: none
        int ke, ve;  // scale bytes
    };
    auto entries = [&](int t) __attribute__((always_inline)) { return table[min(t + 16 * lane, end - 1) >> log_page]; };
    auto block = [&](int e) __attribute__((always_inline)) {
        Block r;
        r.page = e >= 0 && e < a.cache.pages ? e : -1;
        const int64_t at = (int64_t)max(r.page, 0) * kvh + head;
        r.ke = a.cache.ks[at];
        r.ve = a.cache.vs[at];
        return r;
    };
    auto lane_of = [&](int v, int i) __attribute__((always_inline)) { return __builtin_amdgcn_readlane(v, i); };

    uint4 kl[kParts] = {}, vl[kParts] = {};
    int kp = 0, vp = 0;  // pages of kl and vl, -1: none
    uint32_t vs = 0;
    auto load_k = [&](int t, int physical) __attribute__((always_inline)) {
        if (!of_k) return;
        kp = physical;
        // a page of 128 tokens has two tiles
        const uint8_t* from = kc + max(physical, 0) * page_bytes + (t & (page - 1) & 64) * D + k_lane;
#pragma unroll
        for (int i = 0; i < kParts; ++i) kl[i] = *reinterpret_cast<const uint4*>(from + 1024 * i);
    };
    auto load_v = [&](int t, int physical, uint32_t scale) __attribute__((always_inline)) {
        if (!of_v) return;
        vp = physical;
        vs = scale;
        const uint8_t* from = vc + max(physical, 0) * page_bytes + ((t + 16 * v_group) & (page - 1)) + v_lane;
#pragma unroll
        for (int i = 0; i < kParts; ++i) vl[i] = *reinterpret_cast<const uint4*>(from + 64 * i * page);
    };
    auto store_k = [&](int buf) __attribute__((always_inline)) {
        if (!of_k) return;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int token = k_token + 64 / kPieces * i;
            uint4 lo = __builtin_bit_cast(uint4, widen_f16(kl[i].x, kl[i].y)), hi = __builtin_bit_cast(uint4, widen_f16(kl[i].z, kl[i].w));
            // a key without a page: NaN
            if (kp < 0) lo = hi = make_uint4(0x7E007E00, 0x7E007E00, 0x7E007E00, 0x7E007E00);
            keys[buf][key_place<D>(token, 2 * k_piece)] = lo;
            keys[buf][key_place<D>(token, 2 * k_piece + 1)] = hi;
        }
    };
    auto store_v = [&](int buf, int t) __attribute__((always_inline)) {
        if (!of_v) return;
        const float S = e8m0_f32(vs);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            uint32_t w[4] = {vl[i].x, vl[i].y, vl[i].z, vl[i].w};
            if (vp < 0 || t + kLongKeys > end) {
                // values without a page or behind the last token are whatever lies there
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] &= vp >= 0 ? first_bytes(end - (t + 16 * v_group + 4 * k)) : 0u;
            }
            if (any_nan(w[0], w[1], w[2], w[3])) {
                // see below
                nan_seen = 1;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] &= ~(nan_bytes(w[k]) * 0xFFu);
            }
            // a lane of the second product wants tokens 4 h .. and 8 + 4 h .. of 16
            const int d = v_d + 64 * i;
            values[buf][value_place(d, 2 * v_group)] = __builtin_bit_cast(uint4, widen_bf16(w[0], w[2], S));
            values[buf][value_place(d, 2 * v_group + 1)] = __builtin_bit_cast(uint4, widen_bf16(w[1], w[3], S));
        }
    };

    f32x16 acc[kV], score[2];
    float f[4];  // the scores' factors
    uint4 p[4];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = (f32x16){};
    float m = -__builtin_inff(), l = 0.0f, l2 = 0.0f;

    // Fragments from LDS, in eight groups: the values' 16-key groups 0..3, then
    // a quarter of the keys' products each.  Two groups are read ahead of the
    // one that is multiplied.
    constexpr int kRing = 3;
    static_assert(kQ == 2 * kV, "a group holds kV fragments of either kind");
    uint4 frag[kRing][kV];
    auto read = [&](auto index, int buf) __attribute__((always_inline)) {
        constexpr int g = decltype(index)::value;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (g < 4) {
                frag[g % kRing][i] = values[buf][value_place(32 * i + n, 2 * g + hf)];
            } else {
                const int k = (g - 4) * (kQ / 4) + i / 2;
                frag[g % kRing][i] = keys[buf ^ 1][key_place<D>(32 * (i & 1) + n, 2 * k + hf)];
            }
        }
    };
    // Register i of score[st] is of the tile's token 32 st + 8 (i / 4) + 4 hf + i % 4.
    auto multiply = [&](auto index) __attribute__((always_inline)) {
        constexpr int g = decltype(index)::value;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (g < 4) {
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, frag[g % kRing][i]),
                                                                 __builtin_bit_cast(bf16x8, p[g & 3]), acc[i], 0, 0, 0);
            } else {
                const int k = (g - 4) * (kQ / 4) + i / 2;
                score[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, frag[g % kRing][i]), q[k],
                                                                      k == 0 ? (f32x16){} : score[i & 1], 0, 0, 0);
            }
        }
    };
    constexpr std::integral_constant<int, 0> g0{};
    constexpr std::integral_constant<int, 1> g1{};
    constexpr std::integral_constant<int, 2> g2{};
    constexpr std::integral_constant<int, 3> g3{};
    constexpr std::integral_constant<int, 4> g4{};
    constexpr std::integral_constant<int, 5> g5{};
    constexpr std::integral_constant<int, 6> g6{};
    constexpr std::integral_constant<int, 7> g7{};
    const int shift127 = shift + 127;
    auto factors = [&](int ke, int first) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) f[u] = score_factor(sc.c0, lane_of(ke, first + u), shift127);
    };
    // whether the lane's row sees the key that register i of group u holds: one
    // comparison of the distance from the row's first key with its span
    const bool sees = jhi >= jlo;
    const int from = 4 * hf - (sees ? jlo : 1 << 30);
    const uint32_t span = sees ? (uint32_t)(jhi - jlo) : 0;
    auto seen = [&](int t, int u, int i) __attribute__((always_inline)) {
        return (uint32_t)(t + from) + (uint32_t)(16 * u + 8 * (i >> 2) + (i & 3)) <= span;
    };
    // score -> p, with the running maximum and sum
    auto soften = [&](int t) __attribute__((always_inline)) {
        if (CAP) {
            float e[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) e[i] = score[i / 16][i % 16] * f[i / 8];
            cap_scores(e, sc);
#pragma unroll
            for (int i = 0; i < 32; ++i) score[i / 16][i % 16] = e[i];
        }
        if (t < all_lo || t + kLongKeys - 1 > all_hi) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    score[u >> 1][8 * (u & 1) + i] = seen(t, u, i) ? score[u >> 1][8 * (u & 1) + i] : -__builtin_inff();
        }
        float mt = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float g = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 8; ++i) g = fmaxf(g, score[u >> 1][8 * (u & 1) + i]);
            mt = fmaxf(mt, CAP ? g : g * f[u]);
        }
        mt = max_halves(mt);
        if (__any(mt > m + kSlack)) {
            const float mn = fmaxf(m, mt);
            const float alpha = mn > m ? exp2_hw(m - mn) : 1.0f;
            m = mn;
            l *= alpha;
            l2 *= alpha;
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] *= alpha;
        }
        const float mu = exponent_base(m);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = score[u >> 1][8 * (u & 1) + i];
                e[i] = exp2_hw(CAP ? x - mu : __builtin_fmaf(x, f[u], -mu));
            }
            // One part of BF16: with the result's own rounding it is 2.1 to 2.3e-3
            // off (relative norm) where two parts give 1.7e-3, which cost a third
            // of the time: a prompt of 8192 782 us where this takes 594, chunks 776
            // and 582, a mixed batch 55 and 47.  A matter of the products, which
            // few rows have free: those take two.
            p[u] = make_uint4(bf16_pair(e[0], e[1]), bf16_pair(e[2], e[3]), bf16_pair(e[4], e[5]), bf16_pair(e[6], e[7]));
            // the sum of what the second product takes, two at a time
            l = sum_pair(p[u].x, l);
            l2 = sum_pair(p[u].y, l2);
            l = sum_pair(p[u].z, l);
            l2 = sum_pair(p[u].w, l2);
        }
    };
    if (tid == 0) nan_seen = 0;
    __syncthreads();
    if (begin < end) {
        Block now = block(entries(begin)), next = block(entries(begin + 1024));
        int after = entries(begin + 2048), base = begin;
        load_k(begin, lane_of(now.page, k_group));
        load_v(begin, lane_of(now.page, v_group), lane_of(now.ve, v_group));
        store_k(0);
        store_v(0, begin);
        load_k(begin + kLongKeys, lane_of(now.page, 4 + k_group));
        store_k(1);
        __syncthreads();
        factors(now.ke, 0);
        read(g4, 1);
        read(g5, 1);
        multiply(g4);
        read(g6, 1);
        multiply(g5);
        read(g7, 1);
        multiply(g6);
        multiply(g7);
        // the first step stores over these keys
        __syncthreads();
        // A step forms tile t's probabilities, then multiplies: values of t, keys
        // of t + 1.  What it stores at its end, keys of t + 2 and values of t + 1,
        // goes where the step before has read its last, so one barrier a step
        // is enough.  The last step loads, stores and multiplies keys that no
        // row sees: without a branch around them the results stay in their
        // registers.
        auto fetch = [&](int t) __attribute__((always_inline)) {
            if (t + kLongKeys - base == 1024) {
                base += 1024;
                now = next;
                next = block(after);
                after = entries(base + 2048);
            }
            const int first = (t + kLongKeys - base) >> 4;  // 16-key group of tile t + 1
            load_k(t + 2 * kLongKeys, first < 60 ? lane_of(now.page, first + 4 + k_group) : lane_of(next.page, k_group));
            load_v(t + kLongKeys, lane_of(now.page, first + v_group), lane_of(now.ve, first + v_group));
            return first;
        };
        int buf = 0;
        // a wavefront without rows only brings its part of the keys and values
        for (int t = begin; t < end && row0 + 32 * wave >= rows; t += kLongKeys, buf ^= 1) {
            fetch(t);
            store_k(buf);
            store_v(buf ^ 1, t + kLongKeys);
            __syncthreads();
        }
        for (int t = begin; t < end && row0 + 32 * wave < rows; t += kLongKeys, buf ^= 1) {
            const int first_group = fetch(t);
            soften(t);
            __builtin_amdgcn_sched_barrier(0);
            read(g0, buf);
            read(g1, buf);
            read(g2, buf);
            multiply(g0);
            read(g3, buf);
            multiply(g1);
            read(g4, buf);
            multiply(g2);
            read(g5, buf);
            multiply(g3);
            factors(now.ke, first_group);
            read(g6, buf);
            multiply(g4);
            read(g7, buf);
            multiply(g5);
            multiply(g6);
            multiply(g7);
            // in this order: three groups read, then one multiplied, one read ..
            __builtin_amdgcn_sched_group_barrier(kReads, 3 * kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kReads, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kReads, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kReads, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kReads, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kReads, kV, 0);
            __builtin_amdgcn_sched_group_barrier(kProducts, 3 * kV, 0);
            store_k(buf);
            store_v(buf ^ 1, t + kLongKeys);
            __syncthreads();
        }
        // the last tile's values were stored before a barrier that every
        // wavefront has passed
        if (__builtin_amdgcn_readfirstlane(nan_seen)) {
            // A NaN value reaches exactly the rows that see its token, which p
            // cannot say (0 times NaN is NaN): it was stored as 0, and here such
            // tokens are counted per row by products of ones.
            for (int t = begin; t < end; t += 16) {
                const int physical = table[t >> log_page];
                if (physical < 0 || physical >= a.cache.pages) continue;
                const uint8_t* row = vc + physical * page_bytes + n * page + (t & (page - 1));
                bf16x8 one;
#pragma unroll
                for (int k = 0; k < 8; ++k) one[k] = (__bf16)(seen(t, 0, k) ? 1.0f : 0.0f);
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4*>(row + 32 * i * page);
                    const uint32_t w0 = nan_bytes(hf ? w.y : w.x), w1 = nan_bytes(hf ? w.w : w.z);
                    if (!__any((w0 | w1) != 0)) continue;
                    // 0x38: the code of 1
                    const f32x16 cnt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16(w0 * 0x38u, w1 * 0x38u, 1.0f), one, (f32x16){}, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < 16; ++k) acc[i][k] += cnt[k] > 0.0f ? __builtin_nanf("") : 0.0f;
                }
            }
        }
    }

    l += l2;
    l += __shfl_xor(l, 32);
    if (r >= rows) return;
    if (tile.pieces > 1) {
        float* o = long_part<R>(a, place, head, 32 * wave + n);
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<f32x4*>(o + 32 * i + 2 * k + 4 * hf) = (f32x4){acc[i][k], acc[i][k + 1], acc[i][k + 2], acc[i][k + 3]};
        if (hf == 0) *long_stat<R>(a, pl.slots, place, head, 32 * wave + n) = make_float2(m, l);
        return;
    }
    uint16_t* y = a.y + ((int64_t)(s.row0 + token) * a.heads + head * group + member) * D;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            uint2 v;
            v.x = bf16_pair(row_result(acc[i][k], l, pos, room), row_result(acc[i][k + 1], l, pos, room));
            v.y = bf16_pair(row_result(acc[i][k + 2], l, pos, room), row_result(acc[i][k + 3], l, pos, room));
            *reinterpret_cast<uint2*>(y + 32 * i + 2 * k + 4 * hf) = v;
        }
}

// A batch that may hold sequences with many rows: the first workgroups take
// their pieces, the others those of the sequences with few rows, with a
// workspace of their own, so that the compute units that the ones leave idle
// stream the cache for the others (3 x 500 rows and 40 single ones over up to
// 2000 tokens, 32/8 heads of 64: 64 us, one launch after the other 82, and with
// tiles of 128 rows 49; a prompt alone takes as long either way).
template <int D, bool CAP, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void k_attention_mixed(KvAttentionArgs a, LongPlan lp, uint32_t long_items,
                                                                     ShortPlan pl, float* short_workspace, Scoring sc) {
    union Lds {
        LongLds<D> many;
        ShortLds<D, WAVES> few;
    };
    __shared__ __attribute__((aligned(16))) uint8_t lds[sizeof(Lds)];
    if (blockIdx.x < long_items) {
        long_piece<D, CAP, WAVES>(a, lp, sc, blockIdx.x, *reinterpret_cast<LongLds<D>*>(lds));
    } else {
        a.workspace = short_workspace;
        short_pieces<D, WAVES>(a, pl, sc, (int)(blockIdx.x - long_items), (int)(gridDim.x - long_items),
                                    *reinterpret_cast<ShortLds<D, WAVES>*>(lds));
    }
}

// A workgroup joins the pieces of 32 rows of a tile, in order, eight lanes a row.
constexpr int kJoinRows = 32, kSplitRows = 8 * kWaveRows;

template <int D>
__global__ __launch_bounds__(256) void k_attention_join_long(KvAttentionArgs a, LongPlan pl) {
    constexpr int R = kSplitRows;
    constexpr int kPer = D / 32;  // 4-element pieces of a lane, 32 elements apart
    const int kvh = a.cache.kv_heads, group = a.heads / kvh;
    const int head = (int)(blockIdx.x % (uint32_t)kvh), rest = (int)(blockIdx.x / (uint32_t)kvh);
    Tile found;
    const bool is = find_tile(a.batch.sequences, rest / (R / kJoinRows), found, [&](int i) { return Weighed{long_sequence<R>(a, group, i).tiles, 1}; });
    if (!is) return;
    const KvSequence s = kv_sequence(a.batch, found.seq);
    const int length = piece_length<R>(a, pl, group);
    const LongTile tile = long_tile<R>(a, group, s, found.tile, length);
    if (tile.pieces == 1) return;
    const Sum before = sum_before(found.seq, weigh_long<R>(a, group, length));
    const int slot0 = before.weight + found.tile * weigh_long<R>(a, group, length)(found.seq).weight;
    if (!has_slots(slot0, tile.pieces, pl.slots)) return;
    const int64_t room = (int64_t)a.batch.max_pages << a.cache.log_page;
    const int row = rest % (R / kJoinRows) * kJoinRows + threadIdx.x / 8, r = found.tile * R + row, d = 4 * (threadIdx.x & 7);
    if (r >= s.rows * group) return;
    constexpr int kBatch = 4;
    float m = -__builtin_inff(), total = 0.0f;
    f32x4 o[kPer] = {};
    for (int k = 0; k < tile.pieces; k += kBatch) {
        float2 st[kBatch];
        f32x4 p[kBatch][kPer];
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int slot = slot0 + min(k + n, tile.pieces - 1);
            st[n] = *long_stat<R>(a, pl.slots, slot, head, row);
#pragma unroll
            for (int e = 0; e < kPer; ++e) p[n][e] = *reinterpret_cast<const f32x4*>(long_part<R>(a, slot, head, row) + d + 32 * e);
        }
        float mn = m;
#pragma unroll
        for (int n = 0; n < kBatch; ++n) mn = fmaxf(mn, st[n].x);
        const float keep = m == -__builtin_inff() ? (total == 0.0f ? 0.0f : 1.0f) : exp2_hw(m - mn);
        total *= keep;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] *= keep;
        m = mn;
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            if (k + n >= tile.pieces) break;
            const float f = mn == -__builtin_inff() ? 0.0f : exp2_hw(st[n].x - mn);
            total += f * st[n].y;
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] += f * p[n][e];
        }
    }
    const int token = r / group, member = r - token * group;
    const int64_t pos = s.first() + token;
    uint16_t* y = a.y + ((int64_t)(s.row0 + token) * a.heads + head * group + member) * D + d;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        uint2 v;
        v.x = bf16_pair(row_result(o[e][0], total, pos, room), row_result(o[e][1], total, pos, room));
        v.y = bf16_pair(row_result(o[e][2], total, pos, room), row_result(o[e][3], total, pos, room));
        *reinterpret_cast<uint2*>(y + 32 * e) = v;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Workspace bytes per slot of all heads.
int64_t slot_bytes(const KvCacheArgs& c) { return (int64_t)c.kv_heads * 16 * (c.dim + 2) * 4; }

// 16-row tiles of all sequences, at most.
int64_t short_tiles(const KvBatchArgs& b, int group) {
    if (!b.cu) return (int64_t)b.sequences * ((group + 15) / 16);
    const int64_t most = (group > kShortRows ? group : kShortRows) / 16 + 1, by_rows = (int64_t)b.tokens * group / 16 + b.sequences;
    return by_rows < b.sequences * most ? by_rows : b.sequences * most;
}

// `waves`: of the launch of sequences with many rows, 0 where there are none.
ShortPlan short_plan(const KvCacheArgs& c, const KvBatchArgs& b, int heads, int window, int64_t workspace_bytes, int waves) {
    ShortPlan pl;
    const int64_t tiles = short_tiles(b, heads / c.kv_heads);
    // A compute unit holds eight wavefronts: of one workgroup where there are
    // no more tiles than compute units (1 x 131072 62 us, with four 67), else of two.
    pl.waves = waves > 0 ? waves : tiles * c.kv_heads <= 256 ? 8 : 4;
    pl.resident = pl.waves == 8 ? 256 : 512;
    // nothing to split where no sequence has more keys to see than the least range
    int64_t keys = (int64_t)b.max_pages << c.log_page;
    const int64_t seen = (int64_t)window + kShortStep + (b.cu ? kShortRows : 1);
    if (window > 0 && seen < keys) keys = seen;
    const int64_t fit = workspace_bytes / slot_bytes(c) - tiles, want = (pl.resident + c.kv_heads - 1) / c.kv_heads;
    const int64_t ranges = fit < want ? fit : want;
    // the steps of all tiles are counted in 32 bits
    const int64_t steps = (keys + kShortStep - 1) / kShortStep + 1;
    pl.ranges = keys > kLeastRange * kShortStep && ranges > 0 && tiles * steps < (int64_t)1 << 30 ? (int)ranges : 0;
    pl.slots = (int)(pl.ranges + tiles);
    return pl;
}

int64_t long_slot_bytes(const KvCacheArgs& c) { return (int64_t)c.kv_heads * kSplitRows * (c.dim + 2) * 4; }

LongPlan long_plan(const KvCacheArgs& c, const KvBatchArgs& b, int heads, int window, int64_t workspace_bytes) {
    LongPlan pl = {0, 0, 0, 0};
    const int64_t rows = b.cu ? (int64_t)b.tokens * (heads / c.kv_heads) : 0;
    if (rows <= kShortRows) return pl;
    // a sequence with many rows has more than kShortRows of them
    const int64_t most = rows / (kShortRows + 1), sequences = most < b.sequences ? most : b.sequences;
    int64_t tiles = rows / kSplitRows + sequences;
    int64_t keys = (int64_t)b.max_pages << c.log_page;
    if (window > 0 && (int64_t)window + kSplitRows + kLongKeys < keys) keys = (int64_t)window + kSplitRows + kLongKeys;
    const int64_t steps = (keys + kLongKeys - 1) / kLongKeys + 1;
    // A piece per compute unit where the rows give tiles for a quarter of them, or
    // for half of them and their keys are many; with more tiles the join takes
    // what the split saves.  us split and whole, dim 64 and 128, 32/8 heads: 64
    // tiles of 1500 keys 30 and 34, 40 and 47, of 8000 73 and 130, 96 and 200;
    // 96 of 4000 73 and 72, 98 and 108; 125 of 8000 113 and 133, 151 and 200;
    // 187 of 16000 548 and 346, 717 and 467.
    const int64_t high = rows / kSplitRows * c.kv_heads;
    const int64_t want = high <= 64 || (high < 128 && keys > 4096) ? (256 + c.kv_heads - 1) / c.kv_heads : 0;
    const int64_t fit = workspace_bytes / long_slot_bytes(c) - tiles, target = fit < want ? fit : want;
    pl.target = keys > kLeastSplit && target > 0 && tiles * steps < (int64_t)1 << 30 ? (int)target : 0;
    // Tiles of half the rows where those of 256 leave compute units idle, one
    // wavefront on each SIMD: us with four and eight wavefronts, 32/8 heads, dim 64
    // and 128, a prompt of 512 18 and 22, 24 and 27, of 1500 35 and 43, 52 and 57.  With two such workgroups on most units the
    // keys are widened twice as often for the same products: 1500 rows behind 6500
    // tokens 195 and 198, 264 and 243.  Past one tile of 256 for every unit: a
    // prompt of 4000 118 and 115, 183 and 156.
    pl.waves = 8;
    if (pl.target == 0 && high < (c.dim == 128 && keys > 4096 ? 128 : 256)) {
        pl.waves = 4;
        tiles = rows / (4 * kWaveRows) + sequences;
    }
    pl.tiles = (int)tiles;
    pl.slots = (int)(pl.target + tiles);
    return pl;
}

// Workspace bytes of a plan's pieces.
int64_t plan_bytes(const KvCacheArgs& c, const ShortPlan& pl) { return pl.ranges == 0 ? 0 : pl.slots * slot_bytes(c); }
int64_t plan_bytes(const KvCacheArgs& c, const LongPlan& pl) { return pl.target == 0 ? 0 : pl.slots * long_slot_bytes(c); }

template <int D>
hipError_t launch_attention(const KvAttentionArgs& a, hipStream_t stream) {
    const KvCacheArgs& c = a.cache;
    const KvBatchArgs& b = a.batch;
    const int group = a.heads / c.kv_heads;
    const Scoring sc = scoring(a);
    const LongPlan lp = long_plan(c, b, a.heads, a.window, a.workspace_bytes);
    const int64_t many_bytes = plan_bytes(c, lp);
    KvAttentionArgs few = a;
    if (few.workspace) few.workspace += many_bytes / 4;
    const ShortPlan pl = short_plan(c, b, a.heads, a.window, a.workspace_bytes - many_bytes, lp.waves);
    const int64_t tiles = (int64_t)pl.slots * c.kv_heads;
    // a range for each workgroup, or pieces and tiles in turn
    const uint32_t grid = pl.ranges > 0 ? (uint32_t)(pl.ranges * c.kv_heads) : (uint32_t)(tiles < 2 * pl.resident ? tiles : 2 * pl.resident);
    hipError_t e;
    if (lp.tiles > 0) {
        const uint32_t items = (uint32_t)((int64_t)lp.slots * c.kv_heads);
        auto run = [&](auto kernel) { return launch(kernel, dim3(items + grid), dim3(64 * lp.waves), stream, a, lp, items, pl, few.workspace, sc); };
        if (lp.waves == 8) e = a.softcap > 0.0f ? run(k_attention_mixed<D, true, 8>) : run(k_attention_mixed<D, false, 8>);
        else e = a.softcap > 0.0f ? run(k_attention_mixed<D, true, 4>) : run(k_attention_mixed<D, false, 4>);
        if (e == hipSuccess && lp.target > 0)
            e = launch(k_attention_join_long<D>, dim3((uint32_t)((int64_t)lp.tiles * (kSplitRows / kJoinRows) * c.kv_heads)), dim3(256), stream, a, lp);
    } else {
        e = launch(pl.waves == 8 ? k_attention_short<D, 8> : k_attention_short<D, 4>, dim3(grid), dim3(64 * pl.waves), stream, a, pl, sc);
    }
    if (e != hipSuccess || pl.ranges == 0) return e;
    const int each = group;
    return launch(k_attention_join<D>, dim3((uint32_t)((int64_t)b.sequences * each * c.kv_heads)), dim3(256), stream, few, pl, each);
}

}  // namespace

// Whether the launches stay within 2^32 threads and every count within 32 bits.
bool kv_attention_fits(const KvCacheArgs& c, const KvBatchArgs& b, int heads) {
    const int64_t most = 0xFFFFFFFFll, rows = (int64_t)b.tokens * (heads / c.kv_heads);
    if (rows >= ((int64_t)1 << 31) - kSplitRows || (int64_t)b.sequences * heads > most / 256) return false;
    // the plans add at most 512 ranges or pieces of all heads to the tiles
    const int64_t few = short_tiles(b, heads / c.kv_heads) * c.kv_heads + 1024;
    const int64_t many = b.cu ? (rows / kSplitRows + b.sequences) * c.kv_heads + 1024 : 0;
    return few < (int64_t)1 << 31 && many + 1024 <= most / 512 && many <= most / 256 / (kSplitRows / kJoinRows);
}

int64_t kv_attention_workspace_bytes(const KvCacheArgs& c, const KvBatchArgs& b, int heads) {
    if (!kv_attention_fits(c, b, heads)) return 0;
    const LongPlan lp = long_plan(c, b, heads, 0, (int64_t)1 << 60);
    return plan_bytes(c, lp) + plan_bytes(c, short_plan(c, b, heads, 0, (int64_t)1 << 60, lp.waves));
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream) {
    return a.cache.dim == 128 ? launch_attention<128>(a, stream) : launch_attention<64>(a, stream);
}

}  // namespace focus
