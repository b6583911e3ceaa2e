// Causal grouped-query attention over the FP8 key/value cache.
#include <float.h>
#include <math.h>

#include "jetfp8_common.h"
#include "jetfp8_kv.h"
#include "jetfp8_launch.h"
#include "jetfp8_mfma.h"

namespace jetfp8 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;          // waves of a thread block; they share nothing but caches
// Cache blocks of a span, the unit of summation, and spans of a run, the unit of joining.  Spans of 4 blocks measured
// 4 % slower where the cache is long (256 requests up to 8192 tokens 421 against 405 us: twice the partial results)
// and 6 % in the tile kernel (twice the joining), and 4 % faster for 32 requests up to 4096 tokens.
constexpr int kSpan = kKvSpan;
constexpr int kRun = kKvRun;
constexpr int kRunBlocks = kRun * kSpan;
// The cache's probabilities enter the second product as fp16, in which the values' codes are exact, each times its block's
// scale and relative to a reference of its own, near the row's largest such product in the span: what a block adds to the
// row decides about its bits, not its probability or its values alone.  This reference, and the denominator's, follow the
// running maxima only when those have grown by more than 2^8 (in 16 rows of fresh spans some maximum grows with nearly
// every block, and following each would rescale the whole accumulator each time).  A lead of 2^6 (up to 2^7 where the reference is rounded
// down to a whole number) keeps the largest at 2^15, below the type's 65504, and all above 2^-20 of the largest at 11
// significant bits; below that the error is 2^-31 of the largest.
// Where a whole block lies so low that fp16 has only zeros for it (below 2^-25), its exponentials are raised to 2^-kDeep,
// still zeros in fp16, so that in fp32 the denominator gets its terms however small the values are.  The reference is held
// no further than 2^-kLow (and the slack) below the denominator's, so that the power of two between them is in fp32's
// range: what is lost of values near 2^-126 and below is less than their own rounding to bf16.
constexpr float kLead = 6.0f, kSlack = 8.0f, kDeep = 30.0f, kLow = 130.0f;

struct AttnArgs {
    const uint16_t* q;
    const KvUnit* units;
    const int4* prefix;            // of attention_prefix: each unit's group and the blocks that it shares
    const int* table;
    const uint8_t* codes;
    const float* scales;
    const uint16_t* recent;
    uint16_t* o;                   // may be null
    uint8_t* oq;                   // may be null
    float* os;
    float* part_o;                 // partial results, [unit][kv head][part][row]
    float2* part_ml;
    int64_t ldq;
    float scale_log2;              // softmax scale * log2(e)
    int tokens, requests, width, num_blocks, recent_blocks, num_units, max_blocks;
    int q_heads, kv_heads, group;  // group: query heads of a kv head
    int max_rows;                  // rows (token, query head) that a unit may have
    int row_groups;                // row groups, each a wave's, that cover them
    int parts;                     // partial results that a row may have, its own block's among them
    int runs;                      // tile kernel: runs, a thread block each
    int ordered;                   // tile kernel: units taken by length
};

// Eight E4M3 codes -> bf16, exact.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ f16x8 widen_f16(uint32_t lo, uint32_t hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ v4f mfma(const bf16x8& a, const bf16x8& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(const f16x8& a, const f16x8& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v16f mfma(const bf16x8& a, const bf16x8& b, const v16f& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma(const f16x8& a, const f16x8& b, const v16f& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Maximum that keeps a NaN (one instruction for three operands, no quieting of its inputs).
__device__ __forceinline__ float max_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Maximum and sum over the lanes that hold one query's column: l and l + 32, or l, l + 16, l + 32 and l + 48.
__device__ __forceinline__ float pair_max(float x) {
    const u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_of(__uint_as_float(s.x), __uint_as_float(s.y));
}
__device__ __forceinline__ float pair_sum(float x) {
    const u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}
__device__ __forceinline__ float column_max(float x) {
    x = pair_max(x);
    const u32x2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_of(__uint_as_float(s.x), __uint_as_float(s.y));
}
__device__ __forceinline__ float column_sum(float x) {
    x = pair_sum(x);
    const u32x2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}

template <int R>
struct AccOf {
    typedef v4f type;
};
template <>
struct AccOf<32> {
    typedef v16f type;
};

// Running softmax state of R query rows: 16, for products of 16x16x32, or 32, for products of 32x32x16.  Lane l, with
// g = l / R, holds query l % R: top, the reference of its denominator (near its largest score, in log2), and m, that of
// the cache's exponentials times the values' scales; of a block's keys and of each R channels those at 8 j + 4 g .. + 3
// (R = 32, j < 4; R = 16: j = 0); its shares l of the denominator.  With R = 32 these are two, those that lanes g and
// g + 2 hold with R = 16, and two products in ascending order of the contraction give what one of 16x16x32 gives, bit for
// bit: a row's results are the same in both.
template <int D, int R>
struct State {
    typedef typename AccOf<R>::type Acc;
    static constexpr int kShares = R / 16;             // operands of a 32-long contraction
    static constexpr int kTiles = kKvBlock / R;        // of a block's keys
    static constexpr int kOut = D / R;                 // of the channels
    static constexpr int kSteps = D / 32 * kShares;    // of the score product
    typedef Acc Scores[kTiles];
    typedef bf16x8 Queries[kSteps];
    float m, top, l[kShares];
    Acc o[kOut];
    __device__ __forceinline__ void empty() {
#pragma unroll
        for (int g = 0; g < kShares; ++g) l[g] = 0.0f;
    }
    __device__ __forceinline__ void clear() {
        m = top = -INFINITY;
        empty();
#pragma unroll
        for (int t = 0; t < kOut; ++t) o[t] = Acc{};
    }
    __device__ __forceinline__ float sum() const {
        return R == 32 ? pair_sum(l[0] + l[kShares - 1]) : column_sum(l[0]);
    }
    // What takes o from units of 2^m to those of 2^top, a power of two (exp2f: it may be subnormal; 0 where there were no
    // keys).
    __device__ __forceinline__ float factor() const { return exp2f(m - (top == -INFINITY ? 0.0f : top)); }
    // Score j of share g of half h of a block's keys, and the key that it belongs to.
    static __device__ __forceinline__ float score(const Scores& s, int h, int g, int j) {
        return R == 32 ? s[h][j / 4 * 8 + g * 4 + j % 4] : s[h * (kTiles / 2) + j / 4][j % 4];
    }
    static __device__ __forceinline__ void set_score(Scores& s, int h, int g, int j, float x) {
        if (R == 32) s[h][j / 4 * 8 + g * 4 + j % 4] = x;
        else s[h * (kTiles / 2) + j / 4][j % 4] = x;
    }
    static __device__ __forceinline__ int key(int h, int g, int j, int lane) {
        return h * 32 + j / 4 * 16 + g * 8 + lane / R * 4 + j % 4;
    }
    // Largest of the 64 scores that a query has in a block.
    static __device__ __forceinline__ float top_score(const Scores& s) {
        constexpr int n = 16 * kShares;                // of a lane
        auto at = [&](int i) { return R == 32 ? s[i / 16][i % 16] : s[i / 4 % kTiles][i % 4]; };
        float top = max_of(max_of(at(0), at(1)), at(2));
#pragma unroll
        for (int i = 3; i < n - 1; i += 2) top = max_of(max_of(top, at(i)), at(i + 1));
        top = max_of(top, at(n - 1));
        return R == 32 ? pair_max(top) : column_max(top);
    }
};

// Joins the state of the next summation unit (its l already summed over the column) to that of those before it.
// A unit that has no keys at all (every block id out of range) has m = -inf and adds nothing.
__device__ __forceinline__ void join_factors(float& M, float m, float& a, float& b) {
    const float top = fmaxf(M, m);
    const float ref = top == -INFINITY ? 0.0f : top;
    a = __builtin_amdgcn_exp2f(M - ref);
    b = __builtin_amdgcn_exp2f(m - ref);
    M = top;
}

// Where a lane's 8 elements (16 bytes) of operand `step` of tile `tile` lie in a fragment of memory's order, which is that
// of 16x16x32 products: fragments of 16 rows and 32 of the contraction, `steps` of them after another for the same rows.
// With R = 32 a tile's rows are those of two fragments, and a step is half of one.
template <int R>
__device__ __forceinline__ int operand_at(int tile, int step, int steps, int lane) {
    if (R == 16) return (tile * steps + step) * 64 + lane;
    return ((2 * tile + lane % 32 / 16) * steps + step / 2) * 64 + (step % 2 * 2 + lane / 32) * 16 + lane % 16;
}

// A block's keys or values as a wave loads them: 16 codes, of two fragments after another.
template <int D>
struct Raw {
    uint4 w[D / 16];
};
template <int R, bool VALUES, bool KEEP, int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const uint8_t* block, int lane) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    constexpr int steps = VALUES ? 1 : D / 64, shares = R / 16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int at = operand_at<R>(i / (steps * shares), i % (steps * shares), steps, lane);
        const u32x4* p = reinterpret_cast<const u32x4*>(block) + at;
        const u32x4 x = KEEP ? *p : __builtin_nontemporal_load(p);
        r.w[i] = make_uint4(x.x, x.y, x.z, x.w);
    }
}

// Joins a state (m, l, o; l summed over the column, o in units of factor) to that of the units before it.
template <int NT>
__device__ __forceinline__ void join_state(float& M, float& L, v16f (&O)[NT], float m, float l, const v16f (&o)[NT],
                                           float factor) {
    float x, y;
    join_factors(M, m, x, y);
    L = fmaf(L, x, l * y);
    y *= factor;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[t][i] = fmaf(O[t][i], x, o[t][i] * y);
}

// One query row's results: bf16 channels, and their 1x128 codes where they are wanted.  The two lanes of a row exchange
// groups of 4 channels, so that each stores 8 in a row.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, int token, int head, int lane, const v16f (&o)[D / 32],
                                          float inv, bool live) {
    uint4 y[D / 16];
    uint32_t most = 0;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 b = {(__bf16)(o[n / 2][n % 2 * 8 + 2 * i] * inv), (__bf16)(o[n / 2][n % 2 * 8 + 2 * i + 1] * inv)};
            w[i] = __builtin_bit_cast(uint32_t, b);
        }
        const u32x2 u = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const u32x2 v = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        y[n] = make_uint4(u.x, v.x, u.y, v.y);
        most = pkmax16(most, pkmax16(max_mag2(w[0], w[1]), max_mag2(w[2], w[3])));
    }
    const int64_t at = ((int64_t)token * a.q_heads + head) * D + lane / 32 * 8;
    if (a.o && live) {
#pragma unroll
        for (int n = 0; n < D / 16; ++n) *reinterpret_cast<uint4*>(a.o + at + n * 16) = y[n];
    }
    if (D == 128 && a.oq) {
        most = max(most & 0xFFFFu, most >> 16);
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const GroupScale g = make_group_scale(bf16_to_f32(most));
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            const uint32_t w[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = j % 2 ? __uint_as_float(w[j / 2] & 0xFFFF0000u) : bf16_to_f32(w[j / 2] & 0xFFFFu);
            const uint2 codes = encode8(x, g);
            if (live) *reinterpret_cast<uint2*>(a.oq + at + n * 16) = codes;
        }
        if (live && lane < 32) a.os[(int64_t)head * a.tokens + token] = g.s;
    }
}

// The scalars of a run, block i in lane i.  The values' scale enters the exponential's argument as its log2 (-infinity for
// a block of zeros).  A block id out of range has no keys: its bit of use is 0.
struct Run {
    int at;            // physical block
    float c, log_v;    // the keys' scale * softmax scale * log2(e); log2 of the values' scale
    uint64_t use;
};

// Blocks first .. first + 63 of a request, of which those before `last` are used and those before `end` (no less) are
// loaded.
__device__ __forceinline__ Run load_run(const AttnArgs& a, int request, int head, int first, int last, int end, int lane) {
    Run s;
    const int id = a.table[(int64_t)request * a.width + max(min(first + lane, end - 1), 0)];
    s.at = min(max(id, 0), a.num_blocks - 1);
    const float2 scale = *reinterpret_cast<const float2*>(a.scales + ((int64_t)s.at * a.kv_heads + head) * 2);
    const bool here = first + lane < last && id == s.at;
    static_assert(kRunBlocks == 64, "a run's blocks are the lanes");
    s.use = __ballot(here);
    s.c = scale.x * a.scale_log2;
    s.log_v = log2f(scale.y);
    return s;
}

__device__ __forceinline__ float lane_value(float x, int i) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), i));
}

// The queries of a wave's rows, (token, query head of the group) from row0 on; rows behind the last are 0.
template <int D, int R>
__device__ __forceinline__ void load_queries(bf16x8 (&q)[D / 32 * (R / 16)], const AttnArgs& a, const KvUnit& u, int head,
                                             int row0, int rows, int lane) {
    const int row = row0 + lane % R, tok = row / a.group;
    const uint16_t* p = a.q + (u.row + tok) * a.ldq + ((int64_t)head * a.group + row % a.group) * D + lane / R * 8;
#pragma unroll
    for (int k = 0; k < D / 32 * (R / 16); ++k) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < rows) x = *reinterpret_cast<const uint4*>(p + k * (512 / R));
        q[k] = __builtin_bit_cast(bf16x8, x);
    }
}

// Takes the largest scores of a cache block's 64 keys (s, in units of c; log_v: of its values' scale) into the rows'
// references.  START: the first block of a span, whose state is empty (whatever the registers hold) and takes its maxima as
// they are.  References are whole numbers, so that what they rescale keeps its bits, in whatever order a form of the call
// does it.  base: what is added to a score in its exponential; den: takes such exponentials to the denominator's units.
template <bool START, int D, int R>
__device__ __forceinline__ void take_top(State<D, R>& st, const typename State<D, R>::Scores& s, float c, float log_v,
                                         float& base, float& den) {
    const float most = max_of(State<D, R>::top_score(s) * c, -FLT_MAX);      // scores of -infinity: a block without weight
    const float top = __builtin_ceilf(most);
    const float m = max_of(__builtin_floorf(most + log_v) - kLead, top - kLow);
    if (START) {
        st.m = m;
        st.top = top;
        st.empty();
    } else {
        const bool grown = m > st.m + kSlack, ahead = top > st.top + kSlack;
        if (__any(grown || ahead)) {
            const float to = grown ? m : st.m, up = ahead ? top : st.top;
            const float f = __builtin_amdgcn_exp2f(st.m - to), less = __builtin_amdgcn_exp2f(st.top - up);   // 1 if kept
#pragma unroll
            for (int g = 0; g < R / 16; ++g) st.l[g] *= less;
#pragma unroll
            for (int t = 0; t < D / R; ++t) st.o[t] *= f;
            st.m = to;
            st.top = up;
        }
    }
    base = max_of(log_v - st.m, -kDeep - most);
    den = __builtin_amdgcn_exp2f(-base - st.top);
}

// The probabilities of half a block's keys (32 h .. 32 h + 31), times the values' scale, as operands of the second
// product; their sum goes into the denominator.
template <int D, int R>
__device__ __forceinline__ void take_half(State<D, R>& st, const typename State<D, R>::Scores& s, float c, float base,
                                          float den, int h, f16x8 (&p)[2][R / 16]) {
#pragma unroll
    for (int g = 0; g < R / 16; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = __builtin_amdgcn_exp2f(fmaf(st.score(s, h, g, j), c, base));
            sum += e;
            p[h][g][j] = (_Float16)e;
        }
        st.l[g] = fmaf(sum, den, st.l[g]);
    }
}

// Whether some of a value operand's exponents are all ones (infinities, NaN): then bit 15 or 31 of the result is set.
__device__ __forceinline__ uint32_t all_ones(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) odd |= (w[i] & 0x7F807F80u) + 0x00800080u;
    return odd & 0x80008000u;
}

// Takes such values out of an operand; mark: 1 in their places.
__device__ __forceinline__ bf16x8 part_odd(const uint4& v, bf16x8& mark) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = ((w[i] & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) | ((w[i] & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
        w[i] &= ~((m[i] & 0xFFFFu ? 0xFFFFu : 0u) | (m[i] >> 16 ? 0xFFFF0000u : 0u));
    }
    mark = __builtin_bit_cast(bf16x8, make_uint4(m[0], m[1], m[2], m[3]));
    return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// The unit's own block, bf16 with the causal mask, into an empty state (whatever the registers hold).  key(tile, step),
// value(tile, half, share): the block's operands; odd(): whether there are infinities or NaN among the values.  Keys
// behind the last row's own come in halves of the block: the second is left out where no row reaches it (it would add
// zeros).
template <int D, int R, class Key, class Value, class Odd>
__device__ __forceinline__ void own_block(State<D, R>& st, const bf16x8 (&q)[D / 32 * (R / 16)], float scale_log2, int offset,
                                          int group, int row0, int lane, const Key& key, const Value& value,
                                          const Odd& odd) {
    typedef State<D, R> S;
    typedef typename S::Acc Acc;
    const bool both = offset + (row0 + R - 1) / group >= 32;
    const int place = offset + (row0 + lane % R) / group;        // of the query in the block
    typename S::Scores s;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && !both) {
#pragma unroll
            for (int t = S::kTiles / 2; t < S::kTiles; ++t) s[t] = Acc{} - INFINITY;
            break;
        }
#pragma unroll
        for (int t = h * (S::kTiles / 2); t < (h + 1) * (S::kTiles / 2); ++t)
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k) s[t] = mfma(key(t, k), q[k], k ? s[t] : Acc{});
#pragma unroll
        for (int g = 0; g < S::kShares; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (S::key(h, g, j, lane) > place) S::set_score(s, h, g, j, -INFINITY);
    }
    st.top = max_of(S::top_score(s) * scale_log2, -FLT_MAX);     // scores of -infinity: no weight
    st.empty();
    // The values are bf16 here, and so are the probabilities, each as a sum of two (16 significant bits).
    bf16x8 p[2][S::kShares], rest[2][S::kShares];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && !both) {
#pragma unroll
            for (int g = 0; g < S::kShares; ++g) p[h][g] = rest[h][g] = bf16x8{};
            break;
        }
#pragma unroll
        for (int g = 0; g < S::kShares; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = __builtin_amdgcn_exp2f(fmaf(S::score(s, h, g, j), scale_log2, -st.top));
                st.l[g] += e;
                p[h][g][j] = (__bf16)e;
                rest[h][g][j] = (__bf16)(e - (float)(__bf16)e);
            }
    }
    auto add = [&](int t, int h, const bf16x8 (&x)[S::kShares]) {
#pragma unroll
        for (int g = 0; g < S::kShares; ++g) st.o[t] = mfma(x[g], rest[h][g], h || g ? st.o[t] : Acc{});
#pragma unroll
        for (int g = 0; g < S::kShares; ++g) st.o[t] = mfma(x[g], p[h][g], st.o[t]);
    };
    if (__builtin_expect(!odd(), 1)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h && !both) break;
#pragma unroll
            for (int t = 0; t < S::kOut; ++t) {
                bf16x8 x[S::kShares];
#pragma unroll
                for (int g = 0; g < S::kShares; ++g) x[g] = __builtin_bit_cast(bf16x8, value(t, h, g));
                add(t, h, x);
            }
        }
        return;
    }
    // 0 * infinity and 0 * NaN would carry a masked key's values into the rows before it: such values count as 0 in
    // the product, and the channels of the rows that see one become NaN.
#pragma unroll
    for (int t = 0; t < S::kOut; ++t) {
        Acc bad = {};                 // above 0: the row sees such a value in this channel
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 x[S::kShares];
#pragma unroll
            for (int g = 0; g < S::kShares; ++g) {
                bf16x8 mark, seen;
                x[g] = part_odd(value(t, h, g), mark);
#pragma unroll
                for (int j = 0; j < 8; ++j) seen[j] = (__bf16)(S::key(h, g, j, lane) <= place ? 1.0f : 0.0f);
                bad = mfma(mark, seen, bad);
            }
            add(t, h, x);
        }
#pragma unroll
        for (int i = 0; i < R * R / 64; ++i) st.o[t][i] = bad[i] > 0.0f ? NAN : st.o[t][i];
    }
}

// A state as one of the partial results of its rows (l summed over the column, o in units of factor).
template <int D, int R>
__device__ __forceinline__ void store_part(float m, float l, const typename State<D, R>::Acc (&o)[D / R], float factor,
                                           const AttnArgs& a, int unit, int head, int part, int row, int rows, int lane) {
    if (row >= rows) return;
    const int64_t at = (((int64_t)unit * a.kv_heads + head) * a.parts + part) * a.max_rows + row;
#pragma unroll
    for (int t = 0; t < D / R; ++t)
#pragma unroll
        for (int j = 0; j < R * R / 256; ++j)
            *reinterpret_cast<v4f*>(a.part_o + at * D + t * R + j * 8 + lane / R * 4) =
                v4f{o[t][4 * j], o[t][4 * j + 1], o[t][4 * j + 2], o[t][4 * j + 3]} * factor;
    if (lane < R) a.part_ml[at] = make_float2(m, l);
}

// The operands of a recent block: its keys, and behind them (64 D elements on) its values.
template <int D>
__device__ __forceinline__ const uint4* recent_block(const AttnArgs& a, int recent, int head) {
    return reinterpret_cast<const uint4*>(a.recent + ((int64_t)recent * a.kv_heads + head) * 2 * (kKvBlock * D));
}

// Takes cache blocks first .. last - 1 of a request, at most a span and at least one, into the rows' state, which is empty
// before the first (whatever the registers hold).  The next block's codes are loaded while this one's are used; KEEP: they
// are to be kept in the caches, since others read them too.
template <int D, int R, bool KEEP>
__device__ __forceinline__ void walk_span(State<D, R>& st, const typename State<D, R>::Queries& q, const AttnArgs& a,
                                          int request, int head, int first, int last, int lane) {
    typedef State<D, R> S;
    const int64_t block_bytes = (int64_t)a.kv_heads * 2 * kKvBlock * D;
    const uint8_t* codes = a.codes + (int64_t)head * 2 * kKvBlock * D;
    const Run run = load_run(a, request, head, first, last, last, lane);
    if (!(run.use & 1)) st.clear();
    Raw<D> kr, vr;
    const uint8_t* here = codes + __builtin_amdgcn_readlane(run.at, 0) * block_bytes;
    load_raw<R, false, KEEP>(kr, here, lane);
    load_raw<R, true, KEEP>(vr, here + kKvBlock * D, lane);
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        if (first + i >= last) break;
        const uint8_t* next = codes + __builtin_amdgcn_readlane(run.at, i + 1) * block_bytes;
        typename S::Scores s;
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k) {
                // a load holds two fragments' codes: halves of two times kShares steps
                const uint4 w = kr.w[(t * (D / 64) + k / (2 * S::kShares)) * S::kShares + k % S::kShares];
                const bool second = k / S::kShares % 2;
                const bf16x8 x = second ? widen(w.z, w.w) : widen(w.x, w.y);
                s[t] = mfma(x, q[k], k ? s[t] : typename S::Acc{});
            }
        const bool more = i + 1 < kSpan && first + i + 1 < last;
        if (more) load_raw<R, false, KEEP>(kr, next, lane);
        if (run.use >> i & 1) {
            f16x8 p[2][S::kShares];
            const float c = lane_value(run.c, i), log_v = lane_value(run.log_v, i);
            float base, den;
            if (i == 0) take_top<true>(st, s, c, log_v, base, den);
            else take_top<false>(st, s, c, log_v, base, den);
            take_half(st, s, c, base, den, 0, p);
            take_half(st, s, c, base, den, 1, p);
#pragma unroll
            for (int t = 0; t < S::kOut; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < S::kShares; ++g) {
                        const uint4 w = vr.w[t * S::kShares + g];
                        const f16x8 x = h ? widen_f16(w.z, w.w) : widen_f16(w.x, w.y);
                        st.o[t] = mfma(x, p[h][g], i == 0 && h + g == 0 ? typename S::Acc{} : st.o[t]);
                    }
        }
        if (more) load_raw<R, true, KEEP>(vr, next + kKvBlock * D, lane);
    }
}

// Attention of the query rows of one unit's kv head.  Rows are (new token, query head of the group), R = 16 or 32 of them
// to a wave.  Scores are formed transposed, S^T = K Q^T, so that a lane holds R scores of one query per block: maximum
// and sum need two exchanges between lanes, or one, the factors of a row are plain lane values, and the probabilities
// are the second product's operand as they are (O^T = V^T P^T; the cache keeps the values in that key order).  Codes
// are widened to the queries' bf16 and the probabilities' fp16 (both exact) and multiplied by
// v_mfma_f32_16x16x32 or 32x32x16; the scales enter in fp32, in the exponentials' arguments.  Rounded below fp32 are
// only the probabilities (over the cache by at most 2^-12 of each whose product with its block's scale is above 2^-20 of
// the row's largest in the span, and by 2^-31 of that largest otherwise; an eighth of what bf16 would cost, whose error
// alone equals that of the results' own rounding), and the results.
//
// Blocks before the unit's own are complete and precede every query of the unit: no mask.  A row's sums have one order.
// Its blocks are taken in spans of 8, each from an empty state; the spans are joined in ascending order in runs of 8,
// each run from an empty state; the runs are joined in ascending order, and the own block last.  Two kernels do this,
// with the same operations on a row whatever rows share the call, so that a token's result is bitwise the same decoded
// alone, in a batch, or within a prompt:
//
// attention_span_kernel gives every span of a row group a wave of its own and leaves the joining to
// attention_join_kernel: for few rows, where the time is that of reading the cache and every wave must read.  Codes go
// from memory to registers in whole lines (1 KB per load of a wave) and the next block's are loaded while this one's
// are used; there is no LDS.  With R = 16 all rows are one wave's and nobody else reads its codes: the loads are marked
// as not to be kept, which leaves the caches to the partial results (256 requests up to 8192 tokens: 477 -> 422 us).
//
// PREFIX: the spans that the unit's group shares are attention_prefix_kernel's, and how many are left is known on the device
// only.  So they are taken from the last on (the own block), all units' last ones first: the thread blocks without work come
// at the end.  Two waves to a thread block, since what is left is seldom even (256 requests of 16 prompts with up to 1024
// tokens of their own, us: 4 waves and a unit's spans next to one another 78, 2 waves 71, 1 wave 71; 64 prompts of 8 samples 95, 92
// and 91); four with 64 channels, where starting them takes its share (12.7 against 15.6 and 16.6).
template <int D>
constexpr int kTailWaves = D == 64 ? 4 : 2;

template <int D, int R, bool PREFIX>
__global__ __launch_bounds__((PREFIX ? kTailWaves<D> : kWaves) * 64, R == 16 ? 3 : 2) void attention_span_kernel(AttnArgs a) {
    typedef State<D, R> S;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int head = blockIdx.x % a.kv_heads;
    const int jobs = a.parts * a.row_groups, chunks = (jobs + kWaves - 1) / kWaves;
    const int unit = PREFIX ? blockIdx.x / a.kv_heads % a.num_units : blockIdx.x / a.kv_heads / chunks;
    const int job = PREFIX ? blockIdx.x / a.kv_heads / a.num_units * kTailWaves<D> + wave
                           : blockIdx.x / a.kv_heads % chunks * kWaves + wave;
    if (job >= jobs) return;
    const int row0 = job % a.row_groups * R;
    const KvUnit u = a.units[unit];
    if (!unit_fits(u, a.requests, a.tokens, a.recent_blocks, a.num_blocks)) return;
    const int rows = u.rows * a.group, own = join_spans(u.block);
    if (row0 >= rows || rows > a.max_rows || u.block > a.max_blocks) return;
    const int from = PREFIX ? join_shared(u.block, a.prefix[unit].z) : 0;
    const int span = PREFIX ? own - job / a.row_groups : job / a.row_groups;
    if (span < from || span > own) return;

    typename S::Queries q;
    load_queries<D, R>(q, a, u, head, row0, rows, lane);
    S st;
    float factor = 1.0f;
    if (span == own) {
        const uint4* mem = recent_block<D>(a, u.recent, head);
        // loaded before the scores are formed; the second half of the keys only if a row reaches it, as own_block has it
        const bool both = u.offset + (row0 + R - 1) / a.group >= 32;
        uint4 v[S::kOut][2][S::kShares];
#pragma unroll
        for (int t = 0; t < S::kOut; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < S::kShares; ++g) {
                    v[t][h][g] = make_uint4(0, 0, 0, 0);
                    if (!h || both) v[t][h][g] = mem[kKvBlock * D / 8 + operand_at<R>(t, h * S::kShares + g, 2, lane)];
                }
        own_block<D, R>(
            st, q, a.scale_log2, u.offset, a.group, row0, lane,
            [&](int t, int k) { return __builtin_bit_cast(bf16x8, mem[operand_at<R>(t, k, D / 32, lane)]); },
            [&](int t, int h, int g) { return v[t][h][g]; },
            [&]() {
                uint32_t odd = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    odd |= all_ones(v[i / 2 / S::kShares][i / S::kShares % 2][i % S::kShares]);
                return __any(odd != 0);
            });
    } else {
        const int first = span * kSpan;
        // 16 rows: marked as not to be kept, but with 64 channels and shared prompts, where the blocks of a prompt that do not
        // fill a span are much of what is read (us, kept against not: 256 requests of 16 prompts 141 / 128, 128 channels; 124 of 3
        // prompts 37 / 40, 256 of 4 39 / 41, 64 channels; there too it loses where most of the blocks are a request's own: 256 of 16
        // prompts of 4500 with up to 2000 tokens of their own 92 / 82)
        constexpr bool keep = R == 32 || (PREFIX && D == 64);
        walk_span<D, R, keep>(st, q, a, u.request, head, first, min(first + kSpan, u.block), lane);
        factor = st.factor();
    }
    store_part<D, R>(st.top, st.sum(), st.o, factor, a, unit, head, span, row0 + lane % R, rows, lane);
}

// attention_prefix_kernel takes the blocks that the requests of a group share, in the rows of all its units at once: row g
// of the group is row g % max_rows of its unit g / max_rows, and 32 of them are a wave's, whatever units they belong to.
// A piece of work is such a tile of rows and a run of 8 spans: eight waves take a span each and join them in order as the other
// kernels do, so that one partial result of a run is written instead of eight, in the place of the run's last shared span.  Of
// the last run, where only s spans are shared, a piece is as many tiles as eight waves hold, 8 / s.
//
// How many pieces there are is known from the units' records only, so a fixed number of thread blocks, as many as fit the
// chip, count them and take them in turn.  (With a thread block for every piece that the sizes allow, most of which find
// nothing to do, the empty ones delayed the others: 16 samples of 16 prompts up to 8192 89 us instead of 59.)
//
// Bound by the arithmetic of 32 rows to a wave once a group has more rows than that, by HBM below (us for 8 kv heads of 128,
// 4 query heads each, and prompts of 4096 to 8192 tokens: 16 prompts of 8 samples 41, which is 4.9 TB/s of codes; of 16
// samples 59; of 32 samples 96; all with four waves that take two spans each, 3 to 10 % slower than eight).  What was tried
// instead, at 16 samples: the next blocks' codes by way of LDS, so that two blocks are on the way, 59; a stage in LDS that two
// waves share, 115; 64 rows to a wave, 108.
constexpr int kPrefixWaves = kRun;
struct PrefixUnit {
    int4 group;                // its record
    int full, rest, pack;      // runs that are shared whole, spans of the one behind them, tiles in a piece of that
    int tile, tiles;           // pieces of a whole run that begin in this unit's rows: the first, and how many
    int part, parts;           // the same for those of the last run
    __device__ __forceinline__ int pieces() const { return full * tiles + parts; }
};

__device__ __forceinline__ PrefixUnit prefix_unit(const AttnArgs& a, int unit) {
    PrefixUnit p;
    p.group = a.prefix[unit];
    const int rank = unit - p.group.x;
    const bool fits = p.group.x >= 0 && rank >= 0 && rank < p.group.y && p.group.y <= a.num_units - p.group.x &&
                      p.group.z > 0 && p.group.z <= a.max_blocks;
    const int spans = fits ? p.group.z / kSpan : 0;
    p.full = spans / kRun;
    p.rest = spans % kRun;
    p.pack = p.rest ? kPrefixWaves / p.rest : 1;
    const int begin = fits ? rank * a.max_rows : 0, end = fits ? begin + a.max_rows : 0;
    p.tile = (begin + 31) / 32;
    p.tiles = p.full ? (end + 31) / 32 - p.tile : 0;
    p.part = (begin + 32 * p.pack - 1) / (32 * p.pack);
    p.parts = p.rest ? (end + 32 * p.pack - 1) / (32 * p.pack) - p.part : 0;
    return p;
}

template <int D>
__global__ __launch_bounds__(kPrefixWaves * 64, 2) void attention_prefix_kernel(AttnArgs a) {
    typedef State<D, 32> S;
    constexpr int kQuads = D / 4, kMine = kQuads / 2 / kPrefixWaves;       // 4 channels each: of a row, and of a lane to join
    __shared__ v4f part_o[kPrefixWaves][kQuads][32];
    __shared__ float2 part_ml[kPrefixWaves][32];
    __shared__ int64_t place[kPrefixWaves][32];                      // of the rows' partial results; -1: none
    __shared__ int upto[kPrefixWaves * 64], found[6];                // pieces of the units up to a thread's last
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int each = (a.num_units + kPrefixWaves * 64 - 1) / (kPrefixWaves * 64), from = threadIdx.x * each;
    const int end = min(from + each, a.num_units);
    int pieces = 0;
    for (int i = from; i < end; ++i) pieces += prefix_unit(a, i).pieces();
    int sum = pieces;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(sum, d);
        if (lane >= d) sum += y;
    }
    upto[threadIdx.x] = sum;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPrefixWaves; ++w) {
        if (w < wave) base += upto[w * 64 + 63];
        total += upto[w * 64 + 63];
    }
    const int64_t all = (int64_t)total * a.kv_heads;
    for (int64_t job = blockIdx.x; job < all; job += gridDim.x) {
        const int head = job % a.kv_heads;
        int left = (int)(job / a.kv_heads) - (base + sum - pieces);
        __syncthreads();
        // the thread whose units have the piece tells the others
        if (left >= 0 && left < pieces) {
            found[5] = 0;
            for (int i = from; i < end; ++i) {
                const PrefixUnit p = prefix_unit(a, i);
                if (left < p.pieces()) {
                    const bool last = left >= p.full * p.tiles;
                    found[0] = p.group.x;
                    found[1] = p.group.y;
                    found[2] = p.group.z;
                    found[3] = last ? (p.part + left - p.full * p.tiles) * p.pack : p.tile + left / p.full;
                    found[4] = last ? p.full : left % p.full;
                    found[5] = last ? p.rest : kRun;
                    break;
                }
                left -= p.pieces();
            }
        }
        __syncthreads();
        const int first_unit = __builtin_amdgcn_readfirstlane(found[0]), units = __builtin_amdgcn_readfirstlane(found[1]);
        const int shared = __builtin_amdgcn_readfirstlane(found[2]);
        const int first_tile = __builtin_amdgcn_readfirstlane(found[3]), run = __builtin_amdgcn_readfirstlane(found[4]);
        const int spans = __builtin_amdgcn_readfirstlane(found[5]);
        if (spans == 0) continue;                        // the records have changed since they were counted
        const int request = a.units[first_unit].request, pack = kPrefixWaves / spans;
        if (request < 0 || request >= a.requests) continue;
        const int tile = wave / spans, span = wave % spans;              // of this wave; tiles from pack on: none

        // this lane's row, and where its result goes
        const int row = (first_tile + tile) * 32 + lane % 32, member = row / a.max_rows, local = row % a.max_rows;
        const int mine = first_unit + min(member, units - 1);
        const KvUnit u = a.units[mine];
        const int rows = u.rows * a.group;
        const bool live = tile < pack && member < units &&
                          unit_fits(u, a.requests, a.tokens, a.recent_blocks, a.num_blocks) && local < rows &&
                          rows <= a.max_rows && u.block <= a.max_blocks && u.block >= shared;
        if (span == 0 && lane < 32)
            place[tile][lane] =
                live ? (((int64_t)mine * a.kv_heads + head) * a.parts + run * kRun + spans - 1) * a.max_rows + local : -1;
        typename S::Queries q;
        const uint16_t* p =
            a.q + (live ? (u.row + local / a.group) * a.ldq + ((int64_t)head * a.group + local % a.group) * D : 0) + lane / 32 * 8;
#pragma unroll
        for (int k = 0; k < S::kSteps; ++k) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4*>(p + k * 16);
            q[k] = __builtin_bit_cast(bf16x8, x);
        }

        if (tile < pack && __any(live)) {
            S st;
            const int first = (run * kRun + span) * kSpan;
            walk_span<D, 32, true>(st, q, a, request, head, first, first + kSpan, lane);
            const float factor = st.factor(), l = st.sum();
#pragma unroll
            for (int t = 0; t < S::kOut; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part_o[wave][t * 8 + j * 2 + lane / 32][lane % 32] =
                        v4f{st.o[t][4 * j], st.o[t][4 * j + 1], st.o[t][4 * j + 2], st.o[t][4 * j + 3]} * factor;
            if (lane < 32) part_ml[wave][lane] = make_float2(st.top, l);
        }
        __syncthreads();
        for (int t = 0; t < pack; ++t) {
            const int64_t at = place[t][lane % 32];
            if (at < 0) continue;
            float M = -INFINITY, L = 0.0f;
            v4f o[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) o[i] = v4f{};
            for (int s = t * spans; s < (t + 1) * spans; ++s) {
                const float2 ml = part_ml[s][lane % 32];
                float x, y;
                join_factors(M, ml.x, x, y);
                L = fmaf(L, x, ml.y * y);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const v4f v = part_o[s][(wave * kMine + i) * 2 + lane / 32][lane % 32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][c] = fmaf(o[i][c], x, v[c] * y);
                }
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                *reinterpret_cast<v4f*>(a.part_o + at * D + (wave * kMine + i) * 8 + lane / 32 * 4) = o[i];
            if (wave == 0 && lane < 32) a.part_ml[at] = make_float2(M, L);
        }
    }
}

// The pair of units that stands at place x if all are ordered by the blocks that precede them, most first (64 classes;
// one class in any order, unused units last).  A counting sort that every thread block does for itself, about 1 us of
// latency: against that, thread blocks of long requests that start last and then run on alone, with ragged requests
// up to a quarter of the time.  x is below pairs, and pairs no more than 256 kOrder.
constexpr int kOrder = 4;              // pairs of a thread
__device__ __forceinline__ int ordered_pair(const AttnArgs& a, int pairs, int x) {
    __shared__ int count[64], sums[kWaves], found;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    if (threadIdx.x < 64) count[lane] = 0;
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    int key[kOrder];
#pragma unroll
    for (int i = 0; i < kOrder; ++i) {
        const int p = threadIdx.x * kOrder + i;
        key[i] = -1;
        if (p >= pairs) continue;
        const int most = min(max(max(a.units[2 * p].block, a.units[min(2 * p + 1, a.num_units - 1)].block), 0), a.max_blocks);
        key[i] = 63 - (int)((uint32_t)most * 63u / (uint32_t)max(a.max_blocks, 1));
        atomicAdd(&count[key[i]], 1);
    }
    __syncthreads();
    const int mine = count[lane];
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
    const int b = __builtin_ctzll(__ballot(upto > x) | 1ull << 63);
    int y = x - __builtin_amdgcn_readlane(upto - mine, b);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kOrder; ++i) n += key[i] == b;
    int before = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int z = __shfl_up(before, d);
        if (lane >= d) before += z;
    }
    if (lane == 63) sums[wave] = before;
    before -= n;
    __syncthreads();
    for (int w = 0; w < wave; ++w) before += sums[w];
    y -= before;
    if (y >= 0 && y < n) {
#pragma unroll
        for (int i = 0; i < kOrder; ++i) {
            if (key[i] == b && y-- == 0) found = threadIdx.x * kOrder + i;
        }
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(found);
}

// attention_tile_kernel walks a run of 128 rows in one block of four waves, and where that is all (up to 4096 tokens
// before the own block) finishes the rows, else leaves the joining of the runs to attention_join_kernel: for prompts,
// where the time is that of the arithmetic.  Each wave widens a quarter of a block's codes into LDS, as operands, and
// all four read them there, so that a code is widened once per 128 rows instead of once per 32 (the conversions would
// otherwise take a third of the vector unit's time).  Two buffers, one barrier per block; a block's codes are loaded
// from memory two blocks ahead.  A wave forming scores has priority over its SIMD's other wave (a chunk of 2048 at
// 14336: 777 -> 724 us; giving it to the second product as well changes nothing).
//
// A wave multiplies by v_mfma_f32_32x32x16: a lane then holds half of a query's scores instead of a quarter of two
// queries', and a block takes 300 instructions instead of 375, 11 % fewer cycles (64 ragged requests up to 4000: 210 ->
// 191 us; 64 channels, 4 prompts of 2048: 105 -> 97).  Long prompts of 128 channels gain nothing (a chunk of 2048 at 14336:
// 698 -> 700 us, 8 prompts of 2048: 330 -> 335): the card lowers its clock there, from 2.1 to 1.9 GHz.  Two such products
// in ascending order of the contraction give bit for bit what one 16x16x32 product gives (the tests compare the forms).
//
// Units are taken in pairs: two of one request share thread blocks, the waves of the first leaving out the last block or
// so, since a unit's rows (64 query heads per kv head) need not be a multiple of 128.  With D = 64 a third thread block
// fits a CU if a wave is held to 168 registers (4 prompts of 2048, 16 kv heads: 129 -> 113 us; a chunk of 300 at 30000:
// 481 -> 450 us; held to 128 for a fourth it spills).
template <int D>
__global__ __launch_bounds__(kWaves * 64, D == 64 ? 3 : 2) void attention_tile_kernel(AttnArgs a) {
    constexpr int NT = D / 32, NK = D / 16;     // output tiles, contraction steps of the score product
    constexpr int NL = D / 16 / kWaves;         // loads of a block's keys, and of its values, per wave
    constexpr int NO = kKvBlock * D / 8 / 64;   // operands of a block's keys, and of its values
    __shared__ bf16x8 kt[2][NO][64];
    __shared__ f16x8 vt[2][NO][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int head = blockIdx.x % a.kv_heads, chunks = (a.row_groups + kWaves - 1) / kWaves;
    const int pairs = (a.num_units + 1) / 2;
    const int place = blockIdx.x / a.kv_heads / (2 * chunks * a.runs);         // the longest rows first, also without order
    const int first_unit = 2 * (a.ordered ? ordered_pair(a, pairs, place) : pairs - 1 - place);
    const int chunk = blockIdx.x / a.kv_heads % (2 * chunks), run = blockIdx.x / a.kv_heads / (2 * chunks) % a.runs;
    KvUnit us[2];
    int tiles[2];                          // row tiles of 32 that the two units have
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        us[i] = a.units[min(first_unit + i, a.num_units - 1)];
        const int rows = us[i].rows * a.group;
        const bool fits = first_unit + i < a.num_units &&
                          unit_fits(us[i], a.requests, a.tokens, a.recent_blocks, a.num_blocks) &&
                          rows <= a.max_rows && us[i].block <= a.max_blocks;
        tiles[i] = fits ? (rows + 31) / 32 : 0;
    }
    const bool shared = tiles[0] && tiles[1] && us[0].request == us[1].request;
    const int own_chunks = (tiles[0] + kWaves - 1) / kWaves;      // of the first unit, where the two do not share
    int tile = chunk * kWaves + wave, which = 0, end;             // end: blocks that the thread block walks
    bool two = false;                                             // it has rows of both units
    if (shared) {
        if (chunk * kWaves >= tiles[0] + tiles[1]) return;
        which = tile >= tiles[0];
        two = chunk * kWaves < tiles[0] && chunk * kWaves + kWaves > tiles[0];
        end = two ? max(us[0].block, us[1].block) : us[chunk * kWaves >= tiles[0]].block;      // units come in any order
        if (which) tile -= tiles[0];
    } else {
        which = chunk >= own_chunks;
        if (which) tile -= own_chunks * kWaves;
        if (chunk - (which ? own_chunks : 0) >= (tiles[which] + kWaves - 1) / kWaves) return;
        end = us[which].block;
    }
    const int begin = run * kRunBlocks;
    if (run && begin >= end) return;
    // Whether a unit's own block may be due here: with the run that ends before it.
    const bool tail = max((two ? min(us[0].block, us[1].block) : end) - 1, 0) / kRunBlocks <= run;
    end = min(end, begin + kRunBlocks);
    const KvUnit u = us[which];
    const int own_run = max(u.block - 1, 0) / kRunBlocks;         // the run whose thread block takes the own block too
    const bool busy = tile < tiles[which] && run <= own_run;
    const int row0 = tile * 32, rows = busy ? u.rows * a.group : 0, last = busy ? min(u.block, end) : 0;

    bf16x8 q[NK];
    load_queries<D, 32>(q, a, u, head, row0, rows, lane);
    State<D, 32> st;
    float all_m = -INFINITY, all_l = 0.0f;      // the units joined so far
    v16f all_o[NT] = {};
    auto join = [&](float factor) { join_state(all_m, all_l, all_o, st.top, st.sum(), st.o, factor); };

    const int64_t block_bytes = (int64_t)a.kv_heads * 2 * kKvBlock * D;
    const uint8_t* codes = a.codes + (int64_t)head * 2 * kKvBlock * D + lane * 16 + wave * (NL * 1024);
    uint4 raw[2 * NL];               // a wave's share of a block: lines of the keys, then of the values
    auto load = [&](int at) {
        const uint8_t* p = codes + at * block_bytes;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            raw[i] = *reinterpret_cast<const uint4*>(p + i * 1024);
            raw[NL + i] = *reinterpret_cast<const uint4*>(p + kKvBlock * D + i * 1024);
        }
    };
    // Where a lane's 8 elements of operand k of 16 keys or channels t, in the order of 16x16x32 products as memory has it,
    // belong in that of 32x32x16 products: two t make a tile, and half of the lanes hold each of the two steps that k is.
    auto place_at = [&](int t, int steps, int k) {
        return (t / 2 * steps + 2 * k + lane / 32) * 64 + lane / 16 % 2 * 32 + t % 2 * 16 + lane % 16;
    };
    auto store = [&](int buf, int i) {
        const int n = wave * NL + i % NL;       // line of a block's keys or values
        if (i < NL) {
            const int t = n / (NK / 4), k = n % (NK / 4) * 2;
            (&kt[buf][0][0])[place_at(t, NK, k)] = widen(raw[i].x, raw[i].y);
            (&kt[buf][0][0])[place_at(t, NK, k + 1)] = widen(raw[i].z, raw[i].w);
        } else {
            (&vt[buf][0][0])[place_at(n, 4, 0)] = widen_f16(raw[i].x, raw[i].y);
            (&vt[buf][0][0])[place_at(n, 4, 1)] = widen_f16(raw[i].z, raw[i].w);
        }
    };
    if (begin < end) {
        const Run sc = load_run(a, u.request, head, begin, last, end, lane);
        load(__builtin_amdgcn_readlane(sc.at, 0));
#pragma unroll
        for (int i = 0; i < 2 * NL; ++i) store(0, i);
        load(__builtin_amdgcn_readlane(sc.at, 1));
        __syncthreads();
        for (int first = 0; first < end - begin; first += kSpan) {
            if (!(sc.use >> first & 1)) st.clear();
#pragma unroll
            for (int i = 0; i < kSpan; ++i) {
                const int b = first + i;
                if (begin + b >= end) break;
                const int buf = i % 2;
                // Operands come from LDS in a ring, kAhead reads under way before the first is used (left to itself
                // the compiler reads each just before its use, and every read's latency is waited for; 3 and 4 ahead
                // measure the same and spill); the next block's codes are widened and stored between the products.
                constexpr int kAhead = 2, kGroup = NO / 4;
                bf16x8 kf[kAhead];
                __builtin_amdgcn_s_setprio(1);                  // the other wave's vector work fits between these
                v16f s[2];
                auto read_k = [&](int f) { kf[f % kAhead] = kt[buf][f % 2 * NK + f / 2][lane]; };
#pragma unroll
                for (int f = 0; f < kAhead; ++f) read_k(f);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int f = h * kGroup; f < (h + 1) * kGroup; ++f) {
                        s[f % 2] = mfma(kf[f % kAhead], q[f / 2], f / 2 ? s[f % 2] : v16f{});
                        if (f + kAhead < NO) read_k(f + kAhead);
                    }
                    if (h < 2 * NL) store(buf ^ 1, h);          // block b + 1; nobody reads that buffer before the barrier
                }
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(0);
                load(__builtin_amdgcn_readlane(sc.at, min(b + 2, 63)));
                if (sc.use >> b & 1) {
                    f16x8 p[2][2], vf[kAhead];
                    const float c = lane_value(sc.c, b), log_v = lane_value(sc.log_v, b);
                    float base, den;
                    if (i == 0) take_top<true>(st, s, c, log_v, base, den);
                    else take_top<false>(st, s, c, log_v, base, den);
                    take_half(st, s, c, base, den, 0, p);
                    auto read_v = [&](int f) { vf[f % kAhead] = vt[buf][f % NT * 4 + f / NT][lane]; };
#pragma unroll
                    for (int f = 0; f < kAhead; ++f) read_v(f);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        // the second half's exponentials between the first half's products
                        if (h != 1) __builtin_amdgcn_sched_barrier(0);
                        if (h == 0) take_half(st, s, c, base, den, 1, p);
#pragma unroll
                        for (int f = h * kGroup; f < (h + 1) * kGroup; ++f) {
                            st.o[f % NT] = mfma(vf[f % kAhead], p[f / NT / 2][f / NT % 2],
                                                  i == 0 && f / NT == 0 ? v16f{} : st.o[f % NT]);
                            if (f + kAhead < NO) read_v(f + kAhead);
                        }
                        if (h == 1) {
#pragma unroll
                            for (int g = 0; g < NO / 2; ++g) {       // a product, a read from LDS, 6 vector instructions
                                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                                __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);
                            }
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                __syncthreads();
            }
            if (begin + first < last) join(st.factor());
        }
    }
    // The own blocks, as they are, through the same buffers: the first unit's (or the only one's) and the second's.
    uint32_t found = 0;               // infinities or NaN among their values
    const int owns[2] = {two ? us[0].recent : u.recent, us[1].recent};
#pragma unroll
    for (int buf = 0; buf < 2; ++buf) {
        if (!tail || (buf && !two)) break;
        const uint4* mem = recent_block<D>(a, owns[buf], head) + lane;
#pragma unroll
        for (int i = 0; i < NO / kWaves; ++i) {
            const int n = wave * (NO / kWaves) + i;
            const uint4 v = mem[kKvBlock * D / 8 + n * 64];
            (&kt[buf][0][0])[place_at(n / (NK / 2), NK, n % (NK / 2))] = __builtin_bit_cast(bf16x8, mem[n * 64]);
            (&vt[buf][0][0])[place_at(n / 2, 4, n % 2)] = __builtin_bit_cast(f16x8, v);
            found |= all_ones(v);
        }
    }
    const bool odd = __syncthreads_or(found != 0);
    if (!busy) return;
    const int unit = first_unit + which, own_part = (u.block + kRunBlocks - 1) / kRunBlocks;
    const int row = row0 + lane % 32;
    if (a.parts && run < own_part) store_part<D, 32>(all_m, all_l, all_o, 1.0f, a, unit, head, run, row, rows, lane);
    if (run < own_run) return;
    const int buf = two ? which : 0;
    own_block<D, 32>(
        st, q, a.scale_log2, u.offset, a.group, row0, lane, [&](int t, int k) { return kt[buf][t * NK + k][lane]; },
        [&](int t, int h, int g) { return __builtin_bit_cast(uint4, vt[buf][t * 4 + h * 2 + g][lane]); },
        [&]() { return odd; });
    if (a.parts) {
        store_part<D, 32>(st.top, st.sum(), st.o, 1.0f, a, unit, head, own_part, row, rows, lane);
        return;
    }
    join(1.0f);
    store_row<D>(a, u.row + row / a.group, head * a.group + row % a.group, lane, all_o, 1.0f / all_l, row < rows);
}

// Joins n <= N consecutive partial results of a row to the state (M, L, o) of those before them.  Lane s forms the
// factors of the s-th from the running maximum before it (a maximum has no rounding, so the prefix maxima may be formed
// in any order); then they are added one after the other, as the tile kernel does.  ml: lane s's (m, l).
constexpr int kJoin = kRun + 1;
template <int W>
__device__ __forceinline__ void join_parts(const float2& ml, const float* from, int64_t step, int n, int lane, float& M,
                                           float& L, float (&o)[W]) {
    float v[kJoin][W];
#pragma unroll
    for (int s = 0; s < kJoin; ++s)
        if (s < n) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[s][i] = from[s * step + i];
        }
    float top = lane < n ? ml.x : -INFINITY;         // maximum of the parts up to this lane's
#pragma unroll
    for (int d = 1; d < kJoin; d *= 2) {
        const float y = __shfl_up(top, d);
        if (lane >= d) top = fmaxf(top, y);
    }
    top = fmaxf(top, M);
    float before = __shfl_up(top, 1), x, y;
    if (lane == 0) before = M;
    join_factors(before, ml.x, x, y);
    const float ly = ml.y * y;
    M = lane_value(top, kJoin - 1);
#pragma unroll
    for (int s = 0; s < kJoin; ++s)
        if (s < n) {
            const float fx = lane_value(x, s), fy = lane_value(y, s);
            L = fmaf(L, fx, lane_value(ly, s));
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = fmaf(o[i], fx, v[s][i] * fy);
        }
}

// Joins the partial results of a row: those of its spans (SPANS) to runs, the runs, and the own block's.  (One run's
// spans and then the own block are one sequence: joining a state to an empty one changes nothing.)  Bound by the
// latency of a few dependent loads, so all of a run's parts are loaded at once and, where rows are few and may have
// several runs, WAVES waves form them at the same time.  (Loads of parts that are not there, of the last one again, cost
// 1 % of a chunk of 2048 at 14336 and 2 % of 16 chunks up to 12000.)
//
// PREFIX: a run's shared spans are one partial result, that of the last of them.
template <int D, bool SPANS, int WAVES, bool PREFIX>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    constexpr int W = D / 64;       // channels of a lane
    __shared__ float run_o[WAVES > 1 ? kRun : 1][D];
    __shared__ float2 run_ml[WAVES > 1 ? kRun : 1];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int64_t job = WAVES > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
    const int row = job % a.max_rows;
    job /= a.max_rows;
    const int head = job % a.kv_heads;
    const int unit = job / a.kv_heads;
    if (unit >= a.num_units) return;
    const KvUnit u = a.units[unit];
    if (!unit_fits(u, a.requests, a.tokens, a.recent_blocks, a.num_blocks)) return;
    const int rows = u.rows * a.group;
    if (row >= rows || rows > a.max_rows || u.block > a.max_blocks) return;
    const int runs = join_runs(u.block), parts = SPANS ? join_spans(u.block) : runs;
    const int64_t base = ((int64_t)unit * a.kv_heads + head) * a.parts * a.max_rows + row;
    const int64_t step = (int64_t)a.max_rows * D;
    const float* po = a.part_o + base * D + lane * W;
    const float2* pml = a.part_ml + base;
    auto load_ml = [&](int first, int n) {
        return lane < n ? pml[(int64_t)(first + lane) * a.max_rows] : make_float2(-INFINITY, 0.0f);
    };
    const int shared = PREFIX ? join_shared(u.block, a.prefix[unit].z) : 0;
    // First partial result of the run that begins at span s.
    auto run_begin = [&](int s) { return PREFIX ? join_run_begin(s, shared) : s; };
    float M = -INFINITY, L = 0.0f, o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = 0.0f;
    // With shared spans a row may have few parts in several runs.  Then they are all loaded at once, lane s knowing where the
    // s-th lies, and joined in the same order: a run's from an empty state, the runs, the own block's.
    // Join, us, run by run and at once: 256 requests of 16 prompts 9.4 / 8.4, with up to 1024 tokens of their own 10.3 / 8.9, of 4
    // prompts 9.3 / 7.9.  Counted before, so that rows with more parts do not go through their runs for nothing (64 samples of one
    // prompt of 30000: 7.2 -> 6.6).
    int few = 0, slot = 0;                 // parts, if they are few
    uint32_t last = 0;                     // bit s: the s-th is the last of its run
    if (PREFIX && runs > 1 && join_parts_of(u.block, shared) < kJoin) {
        for (int r = 0; r < runs; ++r) {
            const int begin = run_begin(r * kRun), n = min((r + 1) * kRun, parts) - begin;
            if (lane >= few && lane < few + n) slot = begin + lane - few;
            few += n;
            last |= 1u << (few - 1);
        }
        if (lane == few) slot = parts;
        ++few;
    }
    if (PREFIX && few) {
        if (WAVES > 1 && wave) return;
        const float2 ml = lane < few ? pml[(int64_t)slot * a.max_rows] : make_float2(-INFINITY, 0.0f);
        float v[kJoin][W];
#pragma unroll
        for (int s = 0; s < kJoin; ++s)
            if (s < few) {
                const float* from = po + __builtin_amdgcn_readlane(slot, s) * step;
#pragma unroll
                for (int i = 0; i < W; ++i) v[s][i] = from[i];
            }
        float rm = -INFINITY, rl = 0.0f, ro[W], x, y;
#pragma unroll
        for (int i = 0; i < W; ++i) ro[i] = 0.0f;
#pragma unroll
        for (int s = 0; s < kJoin; ++s)
            if (s < few) {
                join_factors(rm, lane_value(ml.x, s), x, y);
                rl = fmaf(rl, x, lane_value(ml.y, s) * y);
#pragma unroll
                for (int i = 0; i < W; ++i) ro[i] = fmaf(ro[i], x, v[s][i] * y);
                if (last >> s & 1 || s + 1 == few) {
                    join_factors(M, rm, x, y);
                    L = fmaf(L, x, rl * y);
                    rm = -INFINITY;
                    rl = 0.0f;
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        o[i] = fmaf(o[i], x, ro[i] * y);
                        ro[i] = 0.0f;
                    }
                }
            }
    } else if (!SPANS || runs <= 1) {
        if (WAVES > 1 && wave) return;
        for (int s0 = run_begin(0); s0 <= parts; s0 += kJoin) {
            const int n = min(kJoin, parts + 1 - s0);
            join_parts<W>(load_ml(s0, n), po + s0 * step, step, n, lane, M, L, o);
        }
    } else {
        int first_run = 0;
        if (PREFIX) {                    // the runs that are one partial result each
            first_run = join_whole_runs(shared);
            for (int r0 = 0; r0 < first_run; r0 += kJoin) {
                const int n = min(kJoin, first_run - r0), s0 = r0 * kRun + kRun - 1;
                const float2 ml = lane < n ? pml[(int64_t)(s0 + lane * kRun) * a.max_rows] : make_float2(-INFINITY, 0.0f);
                join_parts<W>(ml, po + s0 * step, kRun * step, n, lane, M, L, o);
            }
        }
        for (int r0 = first_run; r0 < runs; r0 += kRun) {
            const int n = min(kRun, runs - r0);
            for (int r = wave % WAVES; r < n; r += WAVES) {
                const int s0 = run_begin((r0 + r) * kRun), m = min((r0 + r + 1) * kRun, parts) - s0;
                float rm = -INFINITY, rl = 0.0f, ro[W];
#pragma unroll
                for (int i = 0; i < W; ++i) ro[i] = 0.0f;
                join_parts<W>(load_ml(s0, m), po + s0 * step, step, m, lane, rm, rl, ro);
                if (WAVES == 1) {
                    float x, y;
                    join_factors(M, rm, x, y);
                    L = fmaf(L, x, rl * y);
#pragma unroll
                    for (int i = 0; i < W; ++i) o[i] = fmaf(o[i], x, ro[i] * y);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) run_o[WAVES > 1 ? r : 0][lane * W + i] = ro[i];
                    if (lane == 0) run_ml[WAVES > 1 ? r : 0] = make_float2(rm, rl);
                }
            }
            if (WAVES > 1) {
                __syncthreads();
                if (wave == 0)
                    join_parts<W>(lane < n ? run_ml[WAVES > 1 ? lane : 0] : make_float2(-INFINITY, 0.0f),
                                  &run_o[0][lane * W], D, n, lane, M, L, o);
                __syncthreads();
            }
        }
        if (WAVES > 1 && wave) return;
        join_parts<W>(load_ml(parts, 1), po + parts * step, step, 1, lane, M, L, o);
    }
    const float inv = 1.0f / L;
    const int token = u.row + row / a.group, qh = head * a.group + row % a.group;
    uint32_t y[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const bf16x2 b = {(__bf16)(o[i] * inv), (__bf16)0.0f};
        y[i] = __builtin_bit_cast(uint32_t, b) & 0xFFFFu;
    }
    const int64_t at = ((int64_t)token * a.q_heads + qh) * D + lane * W;
    if (a.o) {
        if (W == 2) *reinterpret_cast<uint32_t*>(a.o + at) = y[0] | y[W - 1] << 16;
        else a.o[at] = (uint16_t)y[0];
    }
    if (D == 128 && a.oq) {
        uint32_t most = row16_max_u32(max(y[0] & 0x7FFFu, y[W - 1] & 0x7FFFu));
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const GroupScale g = make_group_scale(bf16_to_f32(most));
        // four lanes' channels make one group of eight for the encoder
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_to_f32(__shfl((int)y[0], lane / 4 * 4 + j));
            v[2 * j + 1] = bf16_to_f32(__shfl((int)y[W - 1], lane / 4 * 4 + j));
        }
        const uint2 codes = encode8(v, g);
        if (lane % 4 == 0) *reinterpret_cast<uint2*>(a.oq + at) = codes;
        if (lane == 0) a.os[(int64_t)qh * a.tokens + token] = g.s;
    }
}

// The form of a call, from what the host knows of it.
struct AttnShape {
    int64_t max_rows, row_groups, runs, parts, max_blocks;
    int rows;                       // of a wave
    bool split, prefix;
};

// Waves of 32 rows.
double attn_waves(const AttnShape& s, int64_t num_units, int64_t kv_heads) {
    return (double)num_units * kv_heads * ((s.max_rows + 31) / 32);
}

// Whether blocks that units share are taken apart, which costs about 40 us for its launches and their chains of loads, 30 with 64
// channels, however little there is to do.  Without, a call finds shared blocks in the last level of cache, so what decides
// is how much it may read in all.  Below, us apart against not, 8 kv heads, all but 50 to 200 tokens of the contexts shared,
// means over groups from two requests to all.
//   Up to 16 rows a unit, 128 channels (4 rows): 32 requests at 4060 (256 MiB) 41 / 27, at 5148 (324) 42 / 34, at 6620 (416) 45 / 47,
// at 8860 (556) 45 / 64; 64 requests at 3228 (408) 41 / 43, at 4380 (552) 47 / 58; 256 at 9200 146 / 421.  Long rows cost more to
// join otherwise: 2 requests at 66460 (260 MiB) 50 / 59, 4 at 42140 (330) 50 / 58, 8 at 16540 (259) 43 / 44, but 16 at 8220
// (258) 42 / 38.  64 channels (2 rows): 16 requests at 16540 (259) 30 / 33, 64 at 4060 (256) 32 / 28, at 5148 (324) 32 / 35.
//   Contexts of few spans have little to share: 256 requests at 988 (512 MiB) 65 / 56, at 1500 (768) 69 / 73; 512 at 668 (704) 94 / 85.
//   17 to 32 rows fill a wave by themselves, and few units of those are read as fast without (32 rows, 32 requests at 5148 (658 MiB)
// 67 / 54, at 20000 (2540) 153 / 159; 48 at 6000 (1140) 86 / 92).  More units would take the tile kernel, which is slower than
// spans are here: 64 requests at 1500 59 / 61, at 2524 71 / 94, 256 at 4400 300 / 690; with 64 channels not before 3000: 256 requests
// at 2000 142 / 105, 64 at 3100 62 / 64, at 5148 70 / 144.  Beyond 32 rows the partial results are several times as many
// (measured once: 2 prompts of 16 samples, 16 tokens of 8 query heads 132 / 156).
//   What is shared is known on the device only.  Where that is one span of a long context, a call loses by its records: 128
// requests with 8000 tokens of their own 225 / 210, with 64 channels 131 / 105.
bool takes_apart(const AttnShape& s, int64_t num_units, int64_t kv_heads, int64_t D) {
    if (s.max_rows > 32 || s.max_blocks < 24) return false;
    const double mib = (double)num_units * kv_heads * s.max_blocks * (2 * kKvBlock) * D / (1 << 20);
    if (s.max_rows <= 16) return mib >= (D == 64 || s.max_blocks >= 256 ? 256 : 384);
    return attn_waves(s, num_units, kv_heads) >= 1024 ? D == 128 || s.max_blocks >= 48 : mib >= 1024;
}

AttnShape attn_shape(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t D,
                     bool prefix) {
    AttnShape s;
    s.max_rows = (max_new < kKvBlock ? max_new : kKvBlock) * (q_heads / kv_heads);
    s.max_blocks = (max_seq - 1) / kKvBlock;
    const int64_t spans = (s.max_blocks + kSpan - 1) / kSpan;
    s.runs = (spans + kRun - 1) / kRun;
    // Rows that one wave holds read the cache once either way, and a wave per span reads it sooner.  More rows go to
    // the tile kernel if that has enough waves (32 rows each) for the chip's 1024 SIMDs: below, spans in parallel win (256
    // tokens at 4096, 320 waves: 54 against 106 us), at 1072 and 1472 waves the two are within 5 %, above the
    // partial results cost more than they bring (16 times 64 tokens at 4096, 3008 waves: 157 against 109 us).
    s.prefix = prefix && takes_apart(s, num_units, kv_heads, D);
    s.split = spans > 0 && (s.prefix || s.max_rows <= 16 || attn_waves(s, num_units, kv_heads) < 1024);
    s.rows = s.split && s.max_rows <= 16 ? 16 : 32;
    s.row_groups = (s.max_rows + s.rows - 1) / s.rows;
    s.parts = s.split ? spans + 1 : s.runs > 1 ? s.runs + 1 : 0;
    if (s.runs < 1) s.runs = 1;
    return s;
}

int64_t partial_rows(const AttnShape& s, int64_t num_units, int64_t kv_heads) {
    return num_units * kv_heads * s.parts * s.max_rows;
}

// Thread blocks of the first kernel.  In double: sizes at their limits would overflow 64 bits.
double attn_blocks(const AttnShape& s, int64_t num_units, int64_t kv_heads) {
    if (s.split) return (double)num_units * kv_heads * ((s.parts * s.row_groups + kWaves - 1) / kWaves);
    return (double)((num_units + 1) / 2 * 2) * kv_heads * ((s.row_groups + kWaves - 1) / kWaves) * s.runs;
}

template <int D, bool PREFIX>
hipError_t launch(const AttnArgs& a, const AttnShape& s, unsigned grid, hipStream_t st) {
    if (PREFIX) {
        attention_prefix_kernel<D><<<(unsigned)device_cu_count(), kPrefixWaves * 64, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned threads = (PREFIX ? kTailWaves<D> : kWaves) * 64;
    if (PREFIX) {       // no more threads than with four waves to a thread block, which attention_fits looks at
        const int64_t jobs = s.parts * s.row_groups, chunks = (jobs + kTailWaves<D> - 1) / kTailWaves<D>;
        grid = (unsigned)((int64_t)a.num_units * a.kv_heads * chunks);
    }
    if (!s.split) attention_tile_kernel<D><<<grid, kWaves * 64, 0, st>>>(a);
    else if (s.rows == 16) attention_span_kernel<D, 16, PREFIX><<<grid, threads, 0, st>>>(a);
    else attention_span_kernel<D, 32, PREFIX><<<grid, threads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.parts == 0) return e;
    const int64_t rows = (int64_t)a.num_units * a.kv_heads * a.max_rows;
    if (!s.split) attention_join_kernel<D, false, 1, false><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(a);
    // Four waves form a row's runs at once where there are several and rows are too few to fill the chip (one wave a row
    // against four, us: 4 runs 6.3 / 4.6 for 128 rows, 7.4 / 7.2 for 1024, 8.7 / 10.5 for 2048; 16 runs 17.5 / 8.8,
    // 20.8 / 16.2 and 23.2 / 25.9; 2 runs 4.0 / 4.5, 4.7 / 5.5, 5.4 / 8.7).
    else if (s.runs <= 2 || rows >= 2048) attention_join_kernel<D, true, 1, PREFIX><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(a);
    else attention_join_kernel<D, true, 4, PREFIX><<<(unsigned)rows, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t D, bool prefix) {
    return partial_rows(attn_shape(num_units, max_new, max_seq, q_heads, kv_heads, D, prefix), num_units, kv_heads) * (D + 2) *
           (int64_t)sizeof(float);
}

bool attention_fits(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t D,
                    bool prefix) {
    const AttnShape s = attn_shape(num_units, max_new, max_seq, q_heads, kv_heads, D, prefix);
    const double join = s.parts ? (double)num_units * kv_heads * s.max_rows / 4 : 0.0;      // its thread blocks, nearly
    return attn_blocks(s, num_units, kv_heads) < kKvMaxGrid && join < kKvMaxGrid - 1 &&
           (double)num_units * kv_heads * s.max_rows <= INT32_MAX;
}

hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                            const int32_t* prefix, const int32_t* table, int64_t requests, int64_t width,
                            const uint8_t* codes, const float* scales, int64_t num_blocks, const uint16_t* recent,
                            int64_t recent_blocks, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t D, float softmax_scale, uint16_t* o, uint8_t* oq, float* os, float* workspace,
                            hipStream_t st) {
    const AttnShape s = attn_shape(num_units, max_new, max_seq, q_heads, kv_heads, D, prefix != nullptr);
    AttnArgs a;
    a.q = q;
    a.units = reinterpret_cast<const KvUnit*>(units);
    a.prefix = reinterpret_cast<const int4*>(prefix);
    a.table = table;
    a.codes = codes;
    a.scales = scales;
    a.recent = recent;
    a.o = o;
    a.oq = oq;
    a.os = os;
    a.part_o = workspace;
    a.part_ml = reinterpret_cast<float2*>(workspace + partial_rows(s, num_units, kv_heads) * D);
    a.ldq = ldq;
    a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
    a.tokens = (int)tokens;
    a.requests = (int)requests;
    a.width = (int)width;
    a.num_blocks = (int)num_blocks;
    a.recent_blocks = (int)recent_blocks;
    a.num_units = (int)num_units;
    a.max_blocks = (int)(s.max_blocks < width ? s.max_blocks : width);
    a.q_heads = (int)q_heads;
    a.kv_heads = (int)kv_heads;
    a.group = (int)(q_heads / kv_heads);
    a.max_rows = (int)s.max_rows;
    a.row_groups = (int)s.row_groups;
    a.parts = (int)s.parts;
    a.runs = (int)s.runs;
    // Units of one request come in the order of their lengths already.  With several, ordering them shortens the end of
    // the call and costs each thread block its sort: at 3232 waves 79 -> 65 us, at 10048 238 -> 218, at 9040 within 2 %,
    // at 17344 344 -> 360, at 31840 405 -> 428.
    a.ordered = requests > 1 && s.max_blocks > 0 && num_units <= 2 * 256 * kOrder && attn_waves(s, num_units, kv_heads) < 12288;
    const unsigned grid = (unsigned)attn_blocks(s, num_units, kv_heads);
    if (s.prefix) return D == 64 ? launch<64, true>(a, s, grid, st) : launch<128, true>(a, s, grid, st);
    return D == 64 ? launch<64, false>(a, s, grid, st) : launch<128, false>(a, s, grid, st);
}

}  // namespace jetfp8
