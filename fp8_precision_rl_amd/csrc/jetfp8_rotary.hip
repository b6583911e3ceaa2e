// Rotary positions for gfx950.
//
// Pair i < P of a head, channels (i, P + i) or (2 i, 2 i + 1), turns by the angle t = position * freqs[i]:
//   a' = A (a cos t - b sin t),  b' = A (b cos t + a sin t),
// A an amplitude that scaled frequencies may ask for; channels from 2 P on stay as they are.  The inverse turns by -t
// with the same A, which is the transposed map and so the backward pass.
#include "jetfp8_common.h"
#include "jetfp8_launch.h"

namespace jetfp8 {

namespace {

constexpr int kRotaryThreads = 256;

struct RotaryArgs {
    const uint16_t* x;
    uint16_t* out;
    const int* positions;
    const double* freqs;
    int64_t ldx, ldo;
    float amplitude;
    int tokens, heads, items, pairs;     // items: pieces of 16 channels of a head
    int block_tokens, splits;            // tokens of a thread block; thread blocks that share a token's heads
    int per_split;                       // heads of one of them
    bool inverse, copy;                  // copy: out is not x, so the other channels are written too
};

// A thread block takes a few tokens: first the cosines and sines of their angles into LDS, each formed once for all
// heads, then the heads in pieces of 16 channels, two 16-byte loads each.  The angle is reduced to a part of a turn in
// fp64 (a position of 2^20 leaves fp32 no more than three digits of it) and its cosine and sine are taken in fp32.
template <bool INTERLEAVED>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a) {
    __shared__ float2 turn[kRotaryThreads];          // (cos, sin), [token][pair]
    __shared__ int place[kRotaryThreads / 8];
    const int t0 = blockIdx.x / a.splits * a.block_tokens, h0 = blockIdx.x % a.splits * a.per_split;
    const int tokens = min(a.block_tokens, a.tokens - t0), heads = min(a.per_split, a.heads - h0);
    if (threadIdx.x < tokens * a.pairs) {
        const int t = threadIdx.x / a.pairs, i = threadIdx.x % a.pairs;
        const int position = a.positions[t0 + t];
        const double turns = (double)position * a.freqs[i] * 0.15915494309189533577;     // 1 / (2 pi)
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        turn[threadIdx.x] = make_float2(c * a.amplitude, (a.inverse ? -s : s) * a.amplitude);
        if (i == 0) place[t] = position;
    }
    __syncthreads();
    const int step = kRotaryThreads / a.items;       // heads that the thread block takes at a time
    const int piece = threadIdx.x % a.items;
    if (threadIdx.x >= step * a.items) return;
    const bool turned = piece * 8 < a.pairs;         // else: 16 of the channels behind the pairs
    if (!turned && !a.copy) return;
    const int first = INTERLEAVED || !turned ? piece * 16 : piece * 8, second = first + (INTERLEAVED || !turned ? 8 : a.pairs);
    int head = threadIdx.x / a.items, t = 0;
    const int jump = step / heads, rest = step % heads;
    t = head / heads;
    head %= heads;
    for (; t < tokens;) {
        if (place[t] >= 0) {
            const int64_t at = (int64_t)(h0 + head) * a.items * 16;
            const uint16_t* from = a.x + (t0 + t) * a.ldx + at;
            uint16_t* to = a.out + (t0 + t) * a.ldo + at;
            uint4 u = ld16(from + first), v = ld16(from + second);
            if (turned) {
                float p[8], q[8];
                const float2* cs = turn + t * a.pairs + piece * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 z = cs[i];
                    const float f = INTERLEAVED ? elem_of(i < 4 ? u : v, 2 * i % 8) : elem_of(u, i);
                    const float g = INTERLEAVED ? elem_of(i < 4 ? u : v, 2 * i % 8 + 1) : elem_of(v, i);
                    const float l = fmaf(f, z.x, -(g * z.y)), r = fmaf(g, z.x, f * z.y);
                    if (INTERLEAVED) {
                        (i < 4 ? p : q)[2 * i % 8] = l;
                        (i < 4 ? p : q)[2 * i % 8 + 1] = r;
                    } else {
                        p[i] = l;
                        q[i] = r;
                    }
                }
                u = bf16x8_rne(p);
                v = bf16x8_rne(q);
            }
            *reinterpret_cast<uint4*>(to + first) = u;
            *reinterpret_cast<uint4*>(to + second) = v;
        }
        head += rest;
        t += jump;
        if (head >= heads) {
            head -= heads;
            ++t;
        }
    }
}

// A thread block takes as many tokens as its threads have pairs for, if that leaves enough thread blocks; where tokens are
// few, several share a token's heads.
struct RotaryShape {
    int64_t block_tokens, splits, per_split, blocks;
};

RotaryShape rotary_shape(int64_t tokens, int64_t heads, int64_t D, int64_t pairs) {
    RotaryShape s;
    s.block_tokens = 1;
    while (2 * s.block_tokens * pairs <= kRotaryThreads && tokens / (2 * s.block_tokens) >= 4096) s.block_tokens *= 2;
    const int64_t most = (heads * (D / 16) + kRotaryThreads - 1) / kRotaryThreads;     // one piece for each thread
    s.splits = 1;
    while (2 * s.splits <= most && s.splits * tokens < 1024) s.splits *= 2;
    s.per_split = (heads + s.splits - 1) / s.splits;
    s.splits = (heads + s.per_split - 1) / s.per_split;
    s.blocks = (tokens + s.block_tokens - 1) / s.block_tokens * s.splits;
    return s;
}

}  // namespace

// A launch holds fewer than 2^32 threads; splits are only where tokens are few.
bool rotary_fits(int64_t tokens, int64_t heads) { return tokens < (1 << 24) - 1024 && heads < (1 << 20); }

hipError_t launch_rotary(const uint16_t* x, int64_t ldx, int64_t tokens, int64_t heads, int64_t D, const int32_t* positions,
                         const double* freqs, int64_t pairs, bool interleaved, float amplitude, bool inverse,
                         uint16_t* out, int64_t ldo, hipStream_t st) {
    RotaryArgs a;
    a.x = x;
    a.out = out;
    a.positions = positions;
    a.freqs = freqs;
    a.ldx = ldx;
    a.ldo = ldo;
    a.amplitude = amplitude;
    a.tokens = (int)tokens;
    a.heads = (int)heads;
    a.items = (int)(D / 16);
    a.pairs = (int)pairs;
    a.inverse = inverse;
    a.copy = x != out;
    const RotaryShape s = rotary_shape(tokens, heads, D, pairs);
    a.block_tokens = (int)s.block_tokens;
    a.splits = (int)s.splits;
    a.per_split = (int)s.per_split;
    const unsigned grid = (unsigned)s.blocks;
    if (interleaved) rotary_kernel<true><<<grid, kRotaryThreads, 0, st>>>(a);
    else rotary_kernel<false><<<grid, kRotaryThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace jetfp8
