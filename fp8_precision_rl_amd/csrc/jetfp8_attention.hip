// Causal grouped-query attention over the FP8 key/value cache.
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
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;          // waves of a thread block; they share nothing but caches
constexpr int kSpan = 4;           // cache blocks of a span, the unit of summation
// The cache's probabilities enter the second product as fp16 (the values' codes are exact in it), scaled by 2^14: the
// largest is 2^14, below the type's 65504, and all above 2^-28 of the largest keep 11 significant bits.
constexpr float kLead = 14.0f;

struct AttnArgs {
    const uint16_t* q;
    const KvUnit* units;
    const int* table;
    const uint8_t* codes;
    const float* scales;
    const uint16_t* recent;
    uint16_t* o;                   // may be null
    uint8_t* oq;                   // may be null
    float* os;
    float* part_o;                 // split form: partial results of the spans
    float2* part_ml;
    int64_t ldq;
    float scale_log2;              // softmax scale * log2(e)
    int tokens, requests, width, num_blocks, recent_blocks, num_units, max_blocks;
    int q_heads, kv_heads, group;  // group: query heads of a kv head
    int max_rows;                  // rows (token, query head) that a unit may have
    int row_groups;                // row groups of 16 RT rows that cover them
    int spans;                     // split form: partial results per row, the own block's among them
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

__device__ __forceinline__ v4f mfma16(const bf16x8& a, const bf16x8& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma16(const f16x8& a, const f16x8& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Maximum and sum over the four lanes that hold one query's column (lanes l, l + 16, l + 32, l + 48).
__device__ __forceinline__ float column_max(float x) {
    u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
    s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
}
__device__ __forceinline__ float column_sum(float x) {
    u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s.x) + __uint_as_float(s.y);
    s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}

// Running softmax state of 16 RT query rows.  Lane l holds query l % 16 of each tile: the reference m of its
// exponentials (the running maximum of the scores times log2 e, less a lead), its own share of the denominator, and
// the 4 channels 16 t + 4 (l / 16) .. + 3 of every t.
template <int D, int RT>
struct Softmax {
    float m[RT], l[RT];
    v4f o[RT][D / 16];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = -INFINITY;
            l[rt] = 0.0f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[rt][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
};

// Takes the next 64 scores of a query row (s, in units of c) into its state and leaves exp2(s c - m) in s.
template <int D, int RT>
__device__ __forceinline__ void take_scores(Softmax<D, RT>& st, int rt, v4f (&s)[4], float c, float lead) {
    float top = fmaxf(fmaxf(s[0].x, s[0].y), fmaxf(s[0].z, s[0].w));
#pragma unroll
    for (int t = 1; t < 4; ++t) top = fmaxf(top, fmaxf(fmaxf(s[t].x, s[t].y), fmaxf(s[t].z, s[t].w)));
    const float m = fmaxf(st.m[rt], fmaf(column_max(top), c, -lead));
    if (__any(m > st.m[rt])) {          // otherwise every factor is exp2(0) = 1
        const float a = __builtin_amdgcn_exp2f(st.m[rt] - m);
        st.l[rt] *= a;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) st.o[rt][t] *= a;
        st.m[rt] = m;
    }
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -m));
            sum += s[t][i];
        }
    st.l[rt] += sum;
}

// Joins the state of the next summation unit (its l already summed over the column) to that of those before it.
// A unit that has no keys at all (every block id out of range) has m = -inf and adds nothing.
__device__ __forceinline__ void join_factors(float& M, float m, float& a, float& b) {
    const float top = fmaxf(M, m);
    const float ref = top == -INFINITY ? 0.0f : top;
    a = __builtin_amdgcn_exp2f(M - ref);
    b = __builtin_amdgcn_exp2f(m - ref);
    M = top;
}

// Sixteen codes of every operand row: a block's keys or values as a wave loads them.
template <int D>
struct Raw {
    uint4 w[D / 16];
};
template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const uint8_t* block, int lane) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) r.w[i] = *reinterpret_cast<const uint4*>(block + i * 1024 + lane * 16);
}

// One query row's results: bf16 channels, and their 1x128 codes where they are wanted.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, int token, int head, int lane, const v4f (&o)[D / 16],
                                          float inv, bool live) {
    uint2 y[D / 16];
    uint32_t most = 0;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
        const bf16x2 lo = {(__bf16)(o[t].x * inv), (__bf16)(o[t].y * inv)};
        const bf16x2 hi = {(__bf16)(o[t].z * inv), (__bf16)(o[t].w * inv)};
        y[t] = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
        most = pkmax16(most, max_mag2(y[t].x, y[t].y));
    }
    const int64_t at = ((int64_t)token * a.q_heads + head) * D + lane / 16 * 4;
    if (a.o && live) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t) *reinterpret_cast<uint2*>(a.o + at + t * 16) = y[t];
    }
    if (D == 128 && a.oq) {
        most = max(most & 0xFFFFu, most >> 16);
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const GroupScale g = make_group_scale(bf16_to_f32(most));
#pragma unroll
        for (int t = 0; t < D / 16; t += 2) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t w = j % 4 < 2 ? y[t + j / 4].x : y[t + j / 4].y;
                x[j] = j % 2 ? __uint_as_float(w & 0xFFFF0000u) : bf16_to_f32(w & 0xFFFFu);
            }
            const uint2 codes = encode8(x, g);
            if (live) {
                *reinterpret_cast<uint32_t*>(a.oq + at + t * 16) = codes.x;
                *reinterpret_cast<uint32_t*>(a.oq + at + t * 16 + 16) = codes.y;
            }
        }
        if (live && lane < 16) a.os[(int64_t)head * a.tokens + token] = g.s;
    }
}

// Attention of the query rows of one unit's kv head: rows are (new token, query head of the group), 16 RT of them to
// a wave.  Scores are formed transposed, S^T = K Q^T, so that a lane holds 16 scores of one query per block: maximum
// and sum need two exchanges between lanes, the factors of a row are plain lane values, and the probabilities
// are the second product's operand as they are (O^T = V^T P^T; the cache keeps the values in that key order).  Codes
// go from memory to registers in whole lines, are widened to the queries' bf16 and the probabilities' fp16 (both exact)
// and multiplied by v_mfma_f32_16x16x32; the scales enter in fp32, the keys' in the exponent's argument, the values' on
// a block's product.  Rounded below fp32 are only the probabilities (at most 2^-12 of each, an eighth of what
// bf16 would cost, whose error alone equals that of the results' own rounding), and the results.
//
// Blocks before the unit's own are complete and precede every query of the unit: no mask.  The own block is read as
// bf16 with the causal mask.  A row's sums run over its blocks in ascending order in spans of 4 blocks, each span
// from its own zero state, the spans joined in ascending order and the own block last.  The split form gives every
// span a wave of its own and joins the partial results in a second kernel; the serial form walks them in one wave.
// Both perform the same operations on a row, whatever rows share the call: a token's result is bitwise the same
// decoded alone, in a batch, or within a prompt.
template <int D, int RT, bool SPLIT>
__global__ __launch_bounds__(kWaves * 64, RT == 1 ? 2 : 1) void attention_kernel(AttnArgs a) {
    constexpr int NT = D / 16;      // output tiles, and loads of a block's keys or values
    constexpr int NK = D / 32;      // contraction steps of the score product
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, col = lane % 16;
    int job = blockIdx.x;
    const int head = job % a.kv_heads;
    job /= a.kv_heads;
    int unit, rg, span = 0;
    if (SPLIT) {
        const int jobs = a.spans * a.row_groups, chunks = (jobs + kWaves - 1) / kWaves;
        unit = job / chunks;
        const int i = job % chunks * kWaves + wave;
        if (i >= jobs) return;
        span = i / a.row_groups;
        rg = i % a.row_groups;
    } else {
        const int chunks = (a.row_groups + kWaves - 1) / kWaves;
        unit = a.num_units - 1 - job / chunks;       // the longest rows of a request first
        rg = job % chunks * kWaves + wave;
    }
    const KvUnit u = a.units[unit];
    if (!unit_fits(u, a.requests, a.tokens, a.recent_blocks, a.num_blocks)) return;
    const int rows = u.rows * a.group, row0 = rg * (16 * RT);
    if (row0 >= rows || rows > a.max_rows || u.block > a.max_blocks) return;
    const int total_spans = (u.block + kSpan - 1) / kSpan;
    if (SPLIT && span > total_spans) return;
    const int first = SPLIT ? span * kSpan : 0;
    const int last = SPLIT ? min(first + kSpan, u.block) : u.block;      // first > last only for the own block's wave

    bf16x8 q[RT][NK];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + rt * 16 + col, tok = row / a.group;
        const uint16_t* p = a.q + (u.row + tok) * a.ldq + ((int64_t)head * a.group + row % a.group) * D + g * 8;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (row < rows) x = *reinterpret_cast<const uint4*>(p + k * 32);
            q[rt][k] = __builtin_bit_cast(bf16x8, x);
        }
    }

    Softmax<D, RT> st, all;
    st.clear();
    if (!SPLIT) all.clear();

    auto join = [&]() {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x, y;
            join_factors(all.m[rt], st.m[rt], x, y);
            all.l[rt] = fmaf(all.l[rt], x, column_sum(st.l[rt]) * y);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) all.o[rt][t][i] = fmaf(all.o[rt][t][i], x, st.o[rt][t][i] * y);
        }
        st.clear();
    };

    if (first < last) {
        const int* entries = a.table + (int64_t)u.request * a.width;
        const int64_t block_bytes = (int64_t)a.kv_heads * 2 * kKvBlock * D;
        const uint8_t* codes = a.codes + (int64_t)head * 2 * kKvBlock * D;
        const float* scales = a.scales + head * 2;
        Raw<D> kr, vr;
        int id = entries[first];
        int at = min(max(id, 0), a.num_blocks - 1);
        float ks = scales[(int64_t)at * a.kv_heads * 2], vs = scales[(int64_t)at * a.kv_heads * 2 + 1];
        load_raw(kr, codes + at * block_bytes, lane);
        load_raw(vr, codes + at * block_bytes + kKvBlock * D, lane);
        int next_id = entries[min(first + 1, last - 1)];
        for (int b = first; b < last; ++b) {
            const bool here = id == at;
            const float c = ks * a.scale_log2, vscale = vs;
            id = next_id;
            at = min(max(id, 0), a.num_blocks - 1);
            const uint8_t* next = codes + at * block_bytes;
            next_id = entries[min(b + 2, last - 1)];
            ks = scales[(int64_t)at * a.kv_heads * 2];
            vs = scales[(int64_t)at * a.kv_heads * 2 + 1];
            v4f s[RT][4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int k = 0; k < NK; k += 2) {
                    const uint4 w = kr.w[t * (NK / 2) + k / 2];
                    const bf16x8 k0 = widen(w.x, w.y), k1 = widen(w.z, w.w);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                        s[rt][t] = mfma16(k0, q[rt][k], k ? s[rt][t] : z);
                        s[rt][t] = mfma16(k1, q[rt][k + 1], s[rt][t]);
                    }
                }
            load_raw(kr, next, lane);
            if (here) {
                f16x8 p[RT][2];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    take_scores(st, rt, s[rt], c, kLead);
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[rt][i / 8][i % 8] = (_Float16)s[rt][i / 4][i % 4];
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const f16x8 v0 = widen_f16(vr.w[t].x, vr.w[t].y), v1 = widen_f16(vr.w[t].z, vr.w[t].w);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                        const v4f pv = mfma16(v1, p[rt][1], mfma16(v0, p[rt][0], z));
#pragma unroll
                        for (int i = 0; i < 4; ++i) st.o[rt][t][i] = fmaf(pv[i], vscale, st.o[rt][t][i]);
                    }
                }
            }
            load_raw(vr, next + kKvBlock * D, lane);
            if (!SPLIT && (b % kSpan == kSpan - 1 || b + 1 == last)) join();
        }
    }

    if (!SPLIT || span == total_spans) {
        // the own block: bf16, keys after the query masked
        const uint16_t* mem = a.recent + ((int64_t)u.recent * a.kv_heads + head) * 2 * (kKvBlock * D);
        v4f s[RT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(mem + ((t * NK + k) * 64 + lane) * 8);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                    s[rt][t] = mfma16(x, q[rt][k], k ? s[rt][t] : z);
                }
            }
        uint4 v[NT][2];
        uint32_t odd = 0;             // bit 15 of a half: some value's exponent is all ones (infinity or NaN)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[t][k] = *reinterpret_cast<const uint4*>(mem + kKvBlock * D + ((t * 2 + k) * 64 + lane) * 8);
                const uint32_t w[4] = {v[t][k].x, v[t][k].y, v[t][k].z, v[t][k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) odd |= (w[i] & 0x7F807F80u) + 0x00800080u;
            }
        const bool poisoned = __any((odd & 0x80008000u) != 0);
        // The values are bf16 here, and so are the probabilities, each as a sum of two (16 significant bits).
        bf16x8 p[RT][2], rest[RT][2], seen[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int place = u.offset + (row0 + rt * 16 + col) / a.group;      // of the query in the block
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool see = t * 16 + g * 4 + i <= place;
                    if (!see) s[rt][t][i] = -INFINITY;
                    seen[rt][t / 2][t % 2 * 4 + i] = see ? (__bf16)1.0f : (__bf16)0.0f;
                }
            take_scores(st, rt, s[rt], a.scale_log2, 0.0f);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = s[rt][i / 4][i % 4];
                p[rt][i / 8][i % 8] = (__bf16)x;
                rest[rt][i / 8][i % 8] = (__bf16)(x - (float)(__bf16)x);
            }
        }
        // 0 * infinity and 0 * NaN would carry a masked key's values into the rows before it.  Where the block holds
        // any, they count as 0 in the product, and the channels of the rows that see one become NaN.
        v4f bad[RT][NT];
        if (poisoned) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t w[4] = {v[t][k].x, v[t][k].y, v[t][k].z, v[t][k].w}, mark[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mark[i] = ((w[i] & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) |
                                  ((w[i] & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
                        if (mark[i] & 0xFFFFu) w[i] &= 0xFFFF0000u;
                        if (mark[i] >> 16) w[i] &= 0xFFFFu;
                    }
                    v[t][k] = make_uint4(w[0], w[1], w[2], w[3]);
                    const bf16x8 x = __builtin_bit_cast(bf16x8, make_uint4(mark[0], mark[1], mark[2], mark[3]));
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                        bad[rt][t] = mfma16(x, seen[rt][k], k ? bad[rt][t] : z);
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bf16x8 x = __builtin_bit_cast(bf16x8, v[t][k]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) st.o[rt][t] = mfma16(x, p[rt][k], mfma16(x, rest[rt][k], st.o[rt][t]));
            }
        if (poisoned) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (bad[rt][t][i] > 0.0f) st.o[rt][t][i] = NAN;
        }
        if (!SPLIT) join();
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + rt * 16 + col;
        const bool live = row < rows;
        if (SPLIT) {
            const float l = column_sum(st.l[rt]);
            if (live) {
                const int64_t at = (((int64_t)unit * a.kv_heads + head) * a.spans + span) * a.max_rows + row;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    *reinterpret_cast<v4f*>(a.part_o + at * D + t * 16 + g * 4) = st.o[rt][t];
                if (g == 0) a.part_ml[at] = make_float2(st.m[rt], l);
            }
        } else {
            store_row<D>(a, u.row + row / a.group, head * a.group + row % a.group, lane, all.o[rt], 1.0f / all.l[rt],
                         live);
        }
    }
}

// Joins the spans of one row (a wave each): 64 spans at a time, lane s forms the factors of span s from the running
// maximum before it (a maximum has no rounding, so the prefix maxima may be formed in any order), then the spans'
// results are added one after the other, as the serial form does.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    constexpr int W = D / 64;       // channels of a lane
    const int lane = threadIdx.x % 64;
    int64_t job = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int row = job % a.max_rows;
    job /= a.max_rows;
    const int head = job % a.kv_heads;
    const int unit = job / a.kv_heads;
    if (unit >= a.num_units) return;
    const KvUnit u = a.units[unit];
    if (!unit_fits(u, a.requests, a.tokens, a.recent_blocks, a.num_blocks)) return;
    const int rows = u.rows * a.group;
    if (row >= rows || rows > a.max_rows || u.block > a.max_blocks) return;
    const int n = (u.block + kSpan - 1) / kSpan + 1;
    const int64_t base = ((int64_t)unit * a.kv_heads + head) * a.spans * a.max_rows + row;
    const float* po = a.part_o + base * D + lane * W;
    const int64_t step = (int64_t)a.max_rows * D;
    float M = -INFINITY, L = 0.0f, o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = 0.0f;
    for (int s0 = 0; s0 < n; s0 += 64) {
        const int m_n = min(64, n - s0);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < m_n) ml = a.part_ml[base + (int64_t)(s0 + lane) * a.max_rows];
        float top = ml.x;             // maximum of the spans up to this lane's
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const float y = __shfl_up(top, d);
            if (lane >= d) top = fmaxf(top, y);
        }
        top = fmaxf(top, M);
        float before = __shfl_up(top, 1);
        if (lane == 0) before = M;
        float x, y;
        join_factors(before, ml.x, x, y);
        const float ly = ml.y * y;
        M = __shfl(top, 63);
        for (int s = 0; s < m_n; s += 8) {
            float from[8][W];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < W; ++i) from[j][i] = po[(s0 + min(s + j, m_n - 1)) * step + i];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (s + j >= m_n) break;
                const float fx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), s + j));
                const float fy = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(y), s + j));
                L = fmaf(L, fx, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ly), s + j)));
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = fmaf(o[i], fx, from[j][i] * fy);
            }
        }
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
    int64_t max_rows, row_groups, spans, max_blocks;
    int rt;
    bool split;
};

AttnShape attn_shape(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads) {
    AttnShape s;
    s.max_rows = (max_new < kKvBlock ? max_new : kKvBlock) * (q_heads / kv_heads);
    s.rt = s.max_rows <= 16 ? 1 : 2;
    s.row_groups = (s.max_rows + 16 * s.rt - 1) / (16 * s.rt);
    s.max_blocks = (max_seq - 1) / kKvBlock;
    s.spans = (s.max_blocks + kSpan - 1) / kSpan + 1;
    // Waves of the serial form; four per compute unit keep the memory and the matrix units busy.
    const int64_t waves = num_units * kv_heads * s.row_groups;
    s.split = s.spans > 1 && (s.max_rows <= 16 || waves < 1024);
    return s;
}

int64_t partial_rows(const AttnShape& s, int64_t num_units, int64_t kv_heads) {
    return s.split ? num_units * kv_heads * s.spans * s.max_rows : 0;
}

int64_t attn_blocks(const AttnShape& s, int64_t num_units, int64_t kv_heads) {
    const int64_t jobs = s.split ? s.spans * s.row_groups : s.row_groups;
    return num_units * kv_heads * ((jobs + kWaves - 1) / kWaves);
}

template <int D>
hipError_t launch(const AttnArgs& a, const AttnShape& s, unsigned grid, hipStream_t st) {
    if (!s.split) {
        if (s.rt == 1) attention_kernel<D, 1, false><<<grid, kWaves * 64, 0, st>>>(a);
        else attention_kernel<D, 2, false><<<grid, kWaves * 64, 0, st>>>(a);
        return hipGetLastError();
    }
    if (s.rt == 1) attention_kernel<D, 1, true><<<grid, kWaves * 64, 0, st>>>(a);
    else attention_kernel<D, 2, true><<<grid, kWaves * 64, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)a.num_units * a.kv_heads * a.max_rows;
    attention_join_kernel<D><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t D) {
    return partial_rows(attn_shape(num_units, max_new, max_seq, q_heads, kv_heads), num_units, kv_heads) * (D + 2) *
           (int64_t)sizeof(float);
}

bool attention_fits(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads) {
    const AttnShape s = attn_shape(num_units, max_new, max_seq, q_heads, kv_heads);
    return attn_blocks(s, num_units, kv_heads) <= INT32_MAX && num_units * kv_heads * s.max_rows <= INT32_MAX;
}

hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                            const int32_t* table, int64_t requests, int64_t width, const uint8_t* codes,
                            const float* scales, int64_t num_blocks, const uint16_t* recent, int64_t recent_blocks,
                            int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t D,
                            float softmax_scale, uint16_t* o, uint8_t* oq, float* os, float* workspace,
                            hipStream_t st) {
    const AttnShape s = attn_shape(num_units, max_new, max_seq, q_heads, kv_heads);
    AttnArgs a;
    a.q = q;
    a.units = reinterpret_cast<const KvUnit*>(units);
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
    a.spans = (int)s.spans;
    const unsigned grid = (unsigned)attn_blocks(s, num_units, kv_heads);
    return D == 64 ? launch<64>(a, s, grid, st) : launch<128>(a, s, grid, st);
}

}  // namespace jetfp8
