// Page operations of the key/value cache, between the steps of a rollout: which units share a prompt's blocks, forks of
// requests, the sweep of blocks that nobody holds any more, and the compaction of the rest.
//
// Who holds a block is read from the block tables: a request of n tokens holds the first n / 64 entries of its row.  So
// blocks may be shared by any number of requests without counts to keep, and a fork is a copied row.
#include "jetfp8_common.h"
#include "jetfp8_kv.h"
#include "jetfp8_launch.h"

namespace jetfp8 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x = min(x, __shfl_xor(x, d));
    return x;
}

// Smallest x over the thread block.
__device__ __forceinline__ int block_min(int x, int* waves) {
    x = wave_min(x);
    if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = x;
    __syncthreads();
    x = waves[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) x = min(x, waves[w]);
    __syncthreads();
    return x;
}

// Inclusive sums over a thread block of N.
template <int N>
__device__ __forceinline__ uint32_t block_sum_upto(uint32_t x, uint32_t* waves) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) waves[wave] = x;
    __syncthreads();
    for (int w = 0; w < wave; ++w) x += waves[w];
    __syncthreads();
    return x;
}

// ------------------------------------------------------------------------------------------------ positions
// Units in the plan's order have ascending rows: each token looks its own up.
__global__ __launch_bounds__(kThreads) void kv_positions_kernel(const KvUnit* __restrict__ units, int num_units, int tokens,
                                                                int* __restrict__ positions) {
    const int t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= tokens) return;
    int lo = 0, n = num_units;       // units before lo: used, first row at or before t
    while (n > 0) {
        const int half = n / 2;
        const KvUnit u = units[lo + half];
        if (u.request >= 0 && u.row <= t) {
            lo += half + 1;
            n -= half + 1;
        } else {
            n = half;
        }
    }
    int at = -1;
    if (lo > 0) {
        const KvUnit u = units[lo - 1];
        if (t - u.row < u.rows) at = u.block * kKvBlock + u.offset + t - u.row;
    }
    positions[t] = at;
}

// ------------------------------------------------------------------------------------------------ shared prompts
constexpr int kPrefixRows = 8, kFewRows = 2, kWaves = kThreads / 64;      // rows that a wave compares at once

struct PrefixArgs {
    const KvUnit* units;
    const int* table;
    const int* groups;
    int4* prefix;
    int num_units, requests, width;
};

// First unit whose request is r or later; unused units count as behind every request.
__device__ __forceinline__ int first_unit(const PrefixArgs& a, int r) {
    int lo = 0, n = a.num_units;
    while (n > 0) {
        const int half = n / 2;
        const int q = a.units[lo + half].request;
        if (q >= 0 && q < r) {
            lo += half + 1;
            n -= half + 1;
        } else {
            n = half;
        }
    }
    return lo;
}

// How many entries the tables of units u0 + 1 .. used - 1 have in common with `first`, of its first `limit` (and no more than
// *common): a wave compares N rows at once.
template <int N>
__device__ __forceinline__ void compare_rows(const PrefixArgs& a, int u0, int used, int limit, const int* first, int* common) {
    const int lane = threadIdx.x % 64;
    for (int k0 = u0 + 1 + threadIdx.x / 64; k0 < used; k0 += N * kWaves) {
        const int* row[N];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = a.units[min(k0 + i * kWaves, used - 1)].request;
            const bool fits = q >= 0 && q < a.requests;
            bad |= !fits;
            row[i] = fits ? a.table + (int64_t)q * a.width : first;
        }
        int same = bad ? 0 : limit;
        for (int j = 0; j < same; j += 64) {
            const int at = min(j + lane, limit - 1), id = first[at];
            bool other = false;
#pragma unroll
            for (int i = 0; i < N; ++i) other |= row[i][at] != id;
            const uint64_t differ = __ballot(j + lane < limit && other);
            if (differ) same = j + __builtin_ctzll(differ);
        }
        if (lane == 0 && same < limit) atomicMin(common, same);
    }
}

// A thread block for each request; that of a group's first request (or of one without a group) takes the group: its units,
// the earliest of their blocks, and how many entries of their tables agree before that.  The time is that of chains of two
// dependent loads, so a wave compares several rows at once (us, a row against eight, 128 blocks: a group of 64 requests 12.6 /
// 6.0, of 512 80 / 29, of 4096 635 / 208; 16 groups of 16 6.7 / 5.8), but two where that takes them all, up to 9 units, instead of
// loading the last one several times (two against eight: 4 groups of 8 with 32 blocks 4.0 / 4.6, with 128 blocks 4.1 / 4.8;
// 32 groups of 2 4.1 / 4.7).
__global__ __launch_bounds__(kThreads) void kv_prefix_kernel(PrefixArgs a) {
    __shared__ int waves[kThreads / 64], common;
    const int r = blockIdx.x, id = a.groups[r];
    if (id >= 0 && r > 0 && a.groups[r - 1] == id) return;
    int end = r + 1;
    if (id >= 0) {
        for (;;) {        // first request from `end` on with another id
            const int q = end + threadIdx.x;
            const int other = block_min(q >= a.requests || a.groups[q] != id ? q : INT32_MAX, waves);
            if (other != INT32_MAX) {
                end = min(other, a.requests);
                break;
            }
            end += kThreads;
        }
    }
    const int u0 = r == 0 ? 0 : first_unit(a, r), u1 = end == a.requests ? a.num_units : first_unit(a, end);
    const int used = end == a.requests ? first_unit(a, end) : u1;       // behind it only unused units
    int shared = 0;
    if (id >= 0 && u0 < used && a.units[u0].request != a.units[used - 1].request) {
        int limit = a.width;
        for (int k = u0 + threadIdx.x; k < used; k += kThreads) limit = min(limit, a.units[k].block);
        limit = max(block_min(limit, waves), 0);
        if (threadIdx.x == 0) common = limit;
        __syncthreads();
        const int lead = a.units[u0].request;
        const bool known = lead >= 0 && lead < a.requests;
        const int* first = a.table + (int64_t)(known ? lead : 0) * a.width;
        if (known && used - u0 - 1 <= kFewRows * kWaves) compare_rows<kFewRows>(a, u0, used, limit, first, &common);
        else if (known) compare_rows<kPrefixRows>(a, u0, used, limit, first, &common);
        if (!known && threadIdx.x == 0) common = 0;          // units of another call
        __syncthreads();
        shared = common / kKvSpan * kKvSpan;
    }
    for (int k = u0 + threadIdx.x; k < u1; k += kThreads)
        a.prefix[k] = k >= used ? make_int4(-1, 0, 0, 0) : shared ? make_int4(u0, used - u0, shared, 0) : make_int4(k, 1, 0, 0);
}

// ------------------------------------------------------------------------------------------------ fork
// The request that r takes over, or r itself.
__device__ __forceinline__ int parent_of(const int* parents, const int2* state, int requests, int r) {
    const int p = parents[r];
    if (p < 0 || p >= requests || p == r) return r;
    const int a = state[r].y, b = state[p].y;
    return (a == 0 || a == 1) && (b == 0 || b == 1) ? p : r;
}

// Everything goes to other buffers than it comes from, so any map of requests will do.
__global__ __launch_bounds__(kThreads) void kv_fork_kernel(const int2* __restrict__ state, const int* __restrict__ table,
                                                           const int* __restrict__ parents, int requests, int width,
                                                           int2* __restrict__ next_state, int* __restrict__ next_table) {
    const int r = blockIdx.x, p = parent_of(parents, state, requests, r);
    const int2 s = state[p];
    const int held = max(s.x, 0) / kKvBlock;
    for (int j = threadIdx.x; j < width; j += kThreads)
        next_table[(int64_t)r * width + j] = j < held ? table[(int64_t)p * width + j] : -1;
    if (threadIdx.x == 0) next_state[r] = make_int2(s.x, p == r ? s.y : 1 - state[r].y);
}

// A request writes the one of its two recent blocks that it is not filling, and reads one that its parent is filling: no
// block is both, so the copies need no order.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_fork_recent_kernel(const int* __restrict__ parents,
                                                                  const int2* __restrict__ state, int requests, int heads,
                                                                  uint16_t* recent) {
    const int r = blockIdx.x / heads, head = blockIdx.x % heads, p = parent_of(parents, state, requests, r);
    if (p == r) return;
    constexpr int kPieces = 2 * kKvBlock * D / 8 / kThreads;
    const uint4* from = reinterpret_cast<const uint4*>(recent) + ((int64_t)(2 * p + state[p].y) * heads + head) * (kPieces * kThreads);
    uint4* to = reinterpret_cast<uint4*>(recent) + ((int64_t)(2 * r + 1 - state[r].y) * heads + head) * (kPieces * kThreads);
    uint4 x[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) x[i] = from[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) to[i * kThreads + threadIdx.x] = x[i];
}

// ------------------------------------------------------------------------------------------------ sweep
constexpr int kSweepThreads = 1024;
constexpr int kMarkBatch = 8;                        // table entries that a thread has on the way

struct SweepArgs {
    const int2* state;
    const int* table;
    uint64_t* marks;               // [copies][words], one bit for each block: held
    int* free_blocks;
    int* free_head;
    int* live;
    int* next_table;               // compaction; may be null
    int2* moves;
    int requests, width, num_blocks, words, copies;
    uint32_t entries, share;       // table entries; those that one copy of the marks covers
};

__device__ __forceinline__ int held_by(const SweepArgs& a, int r) { return min(max(a.state[r].x, 0) / kKvBlock, a.width); }

// Marks (in LDS) what the table entries from `first` on, `share` of them, hold.
__device__ __forceinline__ void mark(const SweepArgs& a, uint32_t first, uint64_t* bits) {
    for (int i = threadIdx.x; i < a.words; i += kSweepThreads) bits[i] = 0;
    __syncthreads();
    const uint32_t last = min(first + a.share, a.entries);
    for (uint32_t e0 = first + threadIdx.x; e0 < last; e0 += kMarkBatch * kSweepThreads) {
        int id[kMarkBatch];
#pragma unroll
        for (int i = 0; i < kMarkBatch; ++i) {
            const uint32_t e = e0 + i * kSweepThreads;
            id[i] = -1;
            if (e < last && (int)(e % a.width) < held_by(a, e / a.width)) id[i] = a.table[e];
        }
#pragma unroll
        for (int i = 0; i < kMarkBatch; ++i)
            if (id[i] >= 0 && id[i] < a.num_blocks)
                atomicOr(reinterpret_cast<uint32_t*>(bits) + id[i] / 32, 1u << id[i] % 32);
    }
    __syncthreads();
}

// Each thread block marks its share of the tables in a copy of its own, so that nothing has to be cleared first.
__global__ __launch_bounds__(kSweepThreads) void kv_sweep_mark_kernel(SweepArgs a) {
    extern __shared__ uint64_t bits[];
    mark(a, blockIdx.x * a.share, bits);
    for (int i = threadIdx.x; i < a.words; i += kSweepThreads) a.marks[(int64_t)blockIdx.x * a.words + i] = bits[i];
}

// The lists from the marks.  Every thread block forms the number of held blocks before each word in LDS, from which each
// of its items follows by itself: a free block's place in the list, a moving block's target, a table entry's new id.
__global__ __launch_bounds__(kSweepThreads) void kv_sweep_kernel(SweepArgs a) {
    extern __shared__ uint64_t bits[];               // [words], and behind them the held blocks before each word, [words + 1]
    __shared__ uint32_t waves[kSweepThreads / 64];
    uint32_t* before = reinterpret_cast<uint32_t*>(bits + a.words);
    if (a.copies == 1) {
        mark(a, 0, bits);
    } else {
        for (int i = threadIdx.x; i < a.words; i += kSweepThreads) {
            uint64_t x = 0;
#pragma unroll 8
            for (int c = 0; c < a.copies; ++c) x |= a.marks[(int64_t)c * a.words + i];
            bits[i] = x;
        }
        __syncthreads();
    }
    const int per = (a.words + kSweepThreads - 1) / kSweepThreads, w0 = threadIdx.x * per, w1 = min(w0 + per, a.words);
    uint32_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popcll(bits[w]);
    uint32_t sum = block_sum_upto<kSweepThreads>(mine, waves);
    if (threadIdx.x == kSweepThreads - 1) before[a.words] = sum;
    sum -= mine;
    for (int w = w0; w < w1; ++w) {
        before[w] = sum;
        sum += __popcll(bits[w]);
    }
    __syncthreads();
    const int live = before[a.words];
    // (for id = num_blocks the word behind the marks may be read, and is masked out)
    auto held_before = [&](int id) { return (int)before[id / 64] + __popcll(bits[id / 64] & ((1ull << id % 64) - 1)); };
    auto is_held = [&](int id) { return (bits[id / 64] >> id % 64 & 1) != 0; };
    // the k-th free block
    auto free_block = [&](int k) {
        int lo = 0, n = a.words;                     // the word is one of n from lo on
        while (n > 1) {
            const int half = n / 2;
            if ((lo + half) * 64 - (int)before[lo + half] <= k) {
                lo += half;
                n -= half;
            } else {
                n = half;
            }
        }
        uint64_t w = ~bits[lo];
        for (k -= lo * 64 - (int)before[lo]; k > 0; --k) w &= w - 1;
        return lo * 64 + __builtin_ctzll(w);
    };
    const bool compact = a.next_table != nullptr;
    const int stay = compact ? held_before(live) : 0;          // held blocks below `live`: they keep their ids
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.free_head = 0;
        *a.live = live;
    }
    const uint32_t stride = gridDim.x * kSweepThreads, start = blockIdx.x * kSweepThreads + threadIdx.x;
    for (int id = start; id < a.num_blocks; id += stride) {
        if (compact) {
            a.free_blocks[id] = id < a.num_blocks - live ? live + id : -1;
            if (id >= live && is_held(id)) {
                const int k = held_before(id) - stay;
                a.moves[k] = make_int2(id, free_block(k));
            }
            if (id >= live - stay && id < max(a.num_blocks / 2, 1)) a.moves[id] = make_int2(-1, -1);
        } else {
            if (!is_held(id)) a.free_blocks[id - held_before(id)] = id;
            if (id >= a.num_blocks - live) a.free_blocks[id] = -1;
        }
    }
    if (!compact) return;
    for (uint32_t e = start; e < a.entries; e += stride) {
        int id = -1;
        if ((int)(e % a.width) < held_by(a, e / a.width)) {
            id = a.table[e];
            if (id < 0 || id >= a.num_blocks) id = -1;
            else if (id >= live) id = free_block(held_before(id) - stay);
        }
        a.next_table[e] = id;
    }
}

// ------------------------------------------------------------------------------------------------ moves
template <int D>
__global__ __launch_bounds__(kThreads) void kv_move_kernel(const int2* __restrict__ moves, int heads, int num_blocks,
                                                           uint8_t* codes, float* scales) {
    const int2 m = moves[blockIdx.x / heads];
    if (m.x < 0 || m.x >= num_blocks || m.y < 0 || m.y >= num_blocks || m.x == m.y) return;
    constexpr int kPieces = 2 * kKvBlock * D / 16 / kThreads;
    const int head = blockIdx.x % heads;
    const int64_t s = (int64_t)m.x * heads + head, t = (int64_t)m.y * heads + head;
    const uint4* from = reinterpret_cast<const uint4*>(codes) + s * (kPieces * kThreads);
    uint4* to = reinterpret_cast<uint4*>(codes) + t * (kPieces * kThreads);
    uint4 x[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) x[i] = from[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) to[i * kThreads + threadIdx.x] = x[i];
    if (threadIdx.x < 2) scales[2 * t + threadIdx.x] = scales[2 * s + threadIdx.x];
}

// Copies of the marks: one for as many table entries as a thread block has on the way at once.  With one, every thread block
// of the second kernel marks the tables for itself and there is no first.
int64_t sweep_copies(int64_t requests, int64_t width) {
    constexpr int64_t share = kMarkBatch * kSweepThreads;
    const int64_t n = (requests * width + share - 1) / share;
    return n < 64 ? n : 64;
}

}  // namespace

hipError_t launch_kv_positions(const int32_t* units, int64_t num_units, int64_t tokens, int32_t* positions, hipStream_t st) {
    kv_positions_kernel<<<(unsigned)((tokens + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        reinterpret_cast<const KvUnit*>(units), (int)num_units, (int)tokens, positions);
    return hipGetLastError();
}

hipError_t launch_kv_prefix(const int32_t* units, int64_t num_units, const int32_t* table, int64_t requests, int64_t width,
                            const int32_t* groups, int32_t* prefix, hipStream_t st) {
    const PrefixArgs a{reinterpret_cast<const KvUnit*>(units), table, groups, reinterpret_cast<int4*>(prefix),
                       (int)num_units, (int)requests, (int)width};
    kv_prefix_kernel<<<(unsigned)requests, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const int32_t* state, const int32_t* table, int64_t width, int64_t requests,
                          const int32_t* parents, int32_t* next_state, int32_t* next_table, hipStream_t st) {
    kv_fork_kernel<<<(unsigned)requests, kThreads, 0, st>>>(reinterpret_cast<const int2*>(state), table, parents, (int)requests,
                                                          (int)width, reinterpret_cast<int2*>(next_state), next_table);
    return hipGetLastError();
}

hipError_t launch_kv_fork_recent(const int32_t* parents, const int32_t* state, int64_t requests, int64_t heads, int64_t D,
                                 uint16_t* recent, hipStream_t st) {
    const unsigned grid = (unsigned)(requests * heads);
    const int2* s = reinterpret_cast<const int2*>(state);
    if (D == 64) kv_fork_recent_kernel<64><<<grid, kThreads, 0, st>>>(parents, s, (int)requests, (int)heads, recent);
    else kv_fork_recent_kernel<128><<<grid, kThreads, 0, st>>>(parents, s, (int)requests, (int)heads, recent);
    return hipGetLastError();
}

int64_t kv_sweep_workspace(int64_t requests, int64_t width, int64_t num_blocks) {
    const int64_t copies = sweep_copies(requests, width);
    return copies > 1 ? copies * ((num_blocks + 63) / 64) * (int64_t)sizeof(uint64_t) : 0;
}

hipError_t launch_kv_sweep(const int32_t* state, const int32_t* table, int64_t width, int64_t requests, int64_t num_blocks,
                           int32_t* free_blocks, int32_t* free_head, int32_t* live, int32_t* next_table, int32_t* moves,
                           uint64_t* workspace, hipStream_t st) {
    SweepArgs a;
    a.state = reinterpret_cast<const int2*>(state);
    a.table = table;
    a.marks = workspace;
    a.free_blocks = free_blocks;
    a.free_head = free_head;
    a.live = live;
    a.next_table = next_table;
    a.moves = reinterpret_cast<int2*>(moves);
    a.requests = (int)requests;
    a.width = (int)width;
    a.num_blocks = (int)num_blocks;
    a.words = (int)((num_blocks + 63) / 64);
    a.copies = (int)sweep_copies(requests, width);
    a.entries = (uint32_t)(requests * width);
    a.share = (a.entries + a.copies - 1) / a.copies;
    if (a.copies > 1) {
        kv_sweep_mark_kernel<<<(unsigned)a.copies, kSweepThreads, (unsigned)(a.words * sizeof(uint64_t)), st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t items = next_table && a.entries > num_blocks ? a.entries : num_blocks;
    const int64_t blocks = (items + kSweepThreads - 1) / kSweepThreads;
    kv_sweep_kernel<<<(unsigned)(blocks < 256 ? blocks : 256), kSweepThreads,
                      (unsigned)(a.words * (sizeof(uint64_t) + sizeof(uint32_t)) + sizeof(uint32_t)), st>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_move(const int32_t* moves, int64_t num_moves, int64_t heads, int64_t D, uint8_t* codes, float* scales,
                          int64_t num_blocks, hipStream_t st) {
    const unsigned grid = (unsigned)(num_moves * heads);
    const int2* m = reinterpret_cast<const int2*>(moves);
    if (D == 64) kv_move_kernel<64><<<grid, kThreads, 0, st>>>(m, (int)heads, (int)num_blocks, codes, scales);
    else kv_move_kernel<128><<<grid, kThreads, 0, st>>>(m, (int)heads, (int)num_blocks, codes, scales);
    return hipGetLastError();
}

}  // namespace jetfp8
