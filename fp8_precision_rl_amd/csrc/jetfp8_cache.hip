// Writing the key/value cache of rollout: the plan of a step (block tables, slot maps and work units from request
// lengths) and the append of its new keys and values.
#include "../../include/jetfp8.h"
#include "jetfp8_common.h"
#include "jetfp8_kv.h"
#include "jetfp8_launch.h"

namespace jetfp8 {

namespace {

// ------------------------------------------------------------------------------------------------ plan
constexpr int kPlanThreads = 256;
constexpr int kPlanItems = 256;    // units and rows written by a block: one of each per thread

struct PlanArgs {
    const int2* state;
    const int* new_lens;
    const int* free_blocks;
    const int* free_head;
    int* table;
    int2* next_state;
    int* next_free;
    int* status;
    int4* units;
    int64_t* slots;   // may be null
    int requests, tokens, max_new, width, num_free, num_units;
    int num_blocks, max_ids;   // ids of the cache are below num_blocks; a step takes no more than max_ids
};

// Inclusive sums over the block of one 64-bit value per thread (two 32-bit sums side by side).
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* wave_sums) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) wave_sums[wave] = x;
    __syncthreads();
    for (int w = 0; w < wave; ++w) x += wave_sums[w];
    __syncthreads();
    return x;
}

// First r with ends[r] > x (ends ascending); n if there is none.
__device__ __forceinline__ int first_above(const uint32_t* ends, int n, uint32_t x) {
    int lo = 0;
    while (n > 0) {
        const int half = n / 2;
        if (ends[lo + half] > x) n = half;
        else { lo += half + 1; n -= half + 1; }
    }
    return lo;
}

// The step's layout from the requests' lengths: prefix sums over the requests of their new tokens, of the blocks they
// complete, of their units and of the blocks between their first and last.  Bound by latency (a few KB of data and
// two dependent sums), so one launch does it all: every block forms the same sums in LDS from the lengths, at
// most 4096 requests, and then writes one unit and one row per thread.  Nothing is passed between blocks.  A thread
// takes PER consecutive requests, whose lengths it loads at once and keeps (1000 requests with 64440 new tokens: 9.3 us
// against 17 when a thread loaded one request after the other).  With the check of the free list's ids that call takes
// 10.2 us, one of 32 single tokens 4.2 (3.7 without).
template <int PER>
__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(PlanArgs a) {
    extern __shared__ uint32_t sums[];              // [3][requests]
    __shared__ uint64_t wave_sums[kPlanThreads / 64];
    __shared__ int used, avail;
    uint32_t* row_end = sums;
    uint32_t* unit_end = sums + a.requests;
    uint32_t* seal_mid = unit_end + a.requests;     // completed blocks before the request << 16 | middle blocks before it
    const int r0 = threadIdx.x * PER;
    const int head = min(max(*a.free_head, 0), a.num_free);
    if (threadIdx.x == 0) {
        used = 0;
        avail = a.num_free - head;
    }
    __syncthreads();
    // The list ends at its first id that is no block of the cache: a unit with such an id would be left out later.
    for (int i = threadIdx.x; i < min(a.num_free - head, a.max_ids); i += kPlanThreads) {
        const int id = a.free_blocks[head + i];
        if (id < 0 || id >= a.num_blocks) {
            atomicMin(&avail, i);
            break;
        }
    }
    int2 s[PER];
    int n[PER], st[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = min(r0 + i, a.requests - 1);
        s[i] = a.state[r];
        n[i] = a.new_lens[r];
    }

    // A request's lengths are in order if they are no less than 0, fit the call's bound and its row of the table.
    // Rows count for every request, so that the others' rows stay where the caller has put them; rows behind the
    // call's end all saturate there.  (4096 requests of at most 2^19 + 1 rows stay below 2^32.)
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in_order = s[i].x >= 0 && n[i] >= 0 && n[i] <= a.max_new &&
                              (int64_t)s[i].x + n[i] <= (int64_t)kKvBlock * a.width && (s[i].y == 0 || s[i].y == 1);
        st[i] = in_order ? JETFP8_KV_OK : JETFP8_KV_BAD_LENGTH;
        const uint32_t seals = in_order && n[i] <= a.tokens ? (s[i].x + n[i]) / kKvBlock - s[i].x / kKvBlock : 0;
        if (r0 + i < a.requests) mine += ((uint64_t)min(max(n[i], 0), a.tokens + 1) << 32) | seals;
    }
    uint64_t before = block_scan(mine, wave_sums) - mine;
    uint64_t units_mids = 0;
    uint32_t rows = before >> 32, seals = (uint32_t)before;
    int most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (r0 + i >= a.requests) break;
        rows += min(max(n[i], 0), a.tokens + 1);
        row_end[r0 + i] = rows;
        seal_mid[r0 + i] = seals << 16;
        if (st[i] != JETFP8_KV_OK) continue;
        if (rows > (uint32_t)a.tokens) {
            st[i] = JETFP8_KV_NO_ROWS;
        } else if (n[i] > 0) {
            const uint32_t need = (s[i].x + n[i]) / kKvBlock - s[i].x / kKvBlock;
            seals += need;
            if (need > 0 && seals > (uint32_t)avail) {
                st[i] = JETFP8_KV_NO_BLOCK;
            } else {
                const int units = (s[i].x + n[i] - 1) / kKvBlock - s[i].x / kKvBlock + 1;
                units_mids += ((uint64_t)units << 32) | (uint32_t)max(units - 2, 0);
                if (need > 0) most = (int)seals;
            }
        }
    }
    if (most > 0) atomicMax(&used, most);
    before = block_scan(units_mids, wave_sums) - units_mids;
    uint32_t unit = before >> 32, mid = (uint32_t)before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (r0 + i >= a.requests) break;
        const bool live = st[i] == JETFP8_KV_OK && n[i] > 0;
        const int units = live ? (s[i].x + n[i] - 1) / kKvBlock - s[i].x / kKvBlock + 1 : 0;
        seal_mid[r0 + i] |= mid;
        unit += units;
        mid += max(units - 2, 0);
        unit_end[r0 + i] = unit;
        if (blockIdx.x == 0) {
            a.status[r0 + i] = st[i];
            a.next_state[r0 + i] = live ? make_int2(s[i].x + n[i], units > 1 ? 1 - s[i].y : s[i].y) : s[i];
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.next_free = head + used;

    const int item = blockIdx.x * kPlanItems + threadIdx.x;
    if (item < a.num_units) {
        const int u = item;
        const int r = first_above(unit_end, a.requests, u);
        int4 lo = make_int4(-1, -1, -1, -1), hi = lo;
        if (r < a.requests) {
            const int2 s = a.state[r];
            const int n = a.new_lens[r];
            const int first = s.x / kKvBlock, last = (s.x + n - 1) / kKvBlock;
            const int i = u - (int)unit_end[r] + last - first + 1, j = first + i;
            const int offset = i == 0 ? s.x % kKvBlock : 0;
            const int recent = i == 0 ? 2 * r + s.y
                               : j == last ? 2 * r + 1 - s.y
                                           : 2 * a.requests + (int)(seal_mid[r] & 0xFFFF) + i - 1;
            int physical = -1;
            if ((j + 1) * kKvBlock <= s.x + n) {
                physical = a.free_blocks[head + (int)(seal_mid[r] >> 16) + i];
                a.table[(int64_t)r * a.width + j] = physical;
            }
            lo = make_int4(r, j, recent, (int)row_end[r] - n + max(j * kKvBlock - s.x, 0));
            hi = make_int4(min(s.x + n - j * kKvBlock, kKvBlock) - offset, offset, physical, 0);
        }
        a.units[2 * u] = lo;
        a.units[2 * u + 1] = hi;
    }
    if (a.slots && item < a.tokens) {
        const int t = item;
        const int r = first_above(row_end, a.requests, t);
        int64_t slot = -1;
        if (r < a.requests && unit_end[r] > (r ? unit_end[r - 1] : 0)) {
            const int2 s = a.state[r];
            const int n = a.new_lens[r];
            const int pos = s.x + t - ((int)row_end[r] - n);
            if ((pos / kKvBlock + 1) * kKvBlock <= s.x + n)
                slot = (int64_t)a.free_blocks[head + (int)(seal_mid[r] >> 16) + pos / kKvBlock - s.x / kKvBlock] * kKvBlock +
                       pos % kKvBlock;
        }
        a.slots[t] = slot;
    }
}

// ------------------------------------------------------------------------------------------------ append
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const uint16_t* k;
    const uint16_t* v;
    const KvUnit* units;
    uint8_t* codes;
    float* scales;
    uint16_t* recent;
    int64_t ldk, ldv;
    int tokens, heads, num_blocks, recent_blocks;
};

// Largest magnitude pattern over the block.
__device__ __forceinline__ uint32_t block_max(uint32_t a, uint32_t* wave_max) {
    a = row16_max_u32(a);
#pragma unroll
    for (int d = 16; d < 64; d *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, d));
    if (threadIdx.x % 64 == 0) wave_max[threadIdx.x / 64] = a;
    __syncthreads();
    a = wave_max[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 64; ++w) a = max(a, wave_max[w]);
    return a;
}

__device__ __forceinline__ uint2 encode_chunk(const uint4& c, const GroupScale& g) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return encode8(x, g);
}

// One block of threads takes the keys or the values of one unit and kv head.  While the block fills, only the new
// tokens are written, into the unit's bf16 block; a block's first token also clears the rest of it, so that the
// attention may read it whole.  When the block completes, all its 64 tokens (those of earlier calls from the bf16
// block, the new ones from the call) are quantized at once: amax over 64 x D, scale = fl32(amax / 448), codes
// rounded to nearest even as everywhere in this library.  The codes therefore depend on the 64 tokens alone, not on
// how many came with which call.  Bound by HBM for prompts, by latency for single tokens (8 kv heads, D = 128:
// 16384 tokens 43-45 us, 3.7-3.9 TB/s of reads and writes together; 32 single tokens 5.0 us).
template <int D>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
    constexpr int kChunks = kKvBlock * D / 8 / kAppendThreads;   // 16-byte pieces of a block per thread
    constexpr int kPitch = D + 8;                                // row pitch of the values' LDS tile, in elements
    __shared__ __attribute__((aligned(16))) uint16_t tile[kKvBlock * kPitch];
    __shared__ uint32_t wave_max[kAppendThreads / 64];
    const int which = blockIdx.x % 2, head = blockIdx.x / 2 % a.heads, unit = blockIdx.x / (2 * a.heads);
    const KvUnit u = a.units[unit];
    if (!unit_fits(u, INT32_MAX, a.tokens, a.recent_blocks, a.num_blocks)) return;
    const uint16_t* src = (which ? a.v + (int64_t)u.row * a.ldv : a.k + (int64_t)u.row * a.ldk) + (int64_t)head * D;
    const int64_t ld = which ? a.ldv : a.ldk;
    uint16_t* mem = a.recent + (((int64_t)u.recent * a.heads + head) * 2 + which) * (kKvBlock * D);
    const bool whole = u.offset == 0 || u.physical >= 0;

    if (!whole) {
        for (int q = threadIdx.x; q < u.rows * (D / 8); q += kAppendThreads) {
            const int row = q / (D / 8), c = q % (D / 8), n = u.offset + row;
            const uint4 x = *reinterpret_cast<const uint4*>(src + row * ld + c * 8);
            if (which == 0) {
                *reinterpret_cast<uint4*>(mem + ((n / 16 * (D / 32) + c / 4) * 64 + c % 4 * 16 + n % 16) * 8) = x;
            } else {
                uint16_t* to = mem + ((c / 2 * 2 + n / 32) * 64 + n % 16 / 4 * 16 + c % 2 * 8) * 8 + n % 32 / 16 * 4 + n % 4;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) to[8 * i] = (uint16_t)(w[i / 2] >> (i % 2 * 16));
            }
        }
        return;
    }

    uint4 c[kChunks];
    if (which == 0) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int q = i * kAppendThreads + threadIdx.x;
            const int ks = q / 64, n = ks / (D / 32) * 16 + q % 16, d = ks % (D / 32) * 32 + q % 64 / 16 * 8;
            const int row = n - u.offset;
            c[i] = make_uint4(0, 0, 0, 0);
            if (row >= 0 && row < u.rows) c[i] = *reinterpret_cast<const uint4*>(src + row * ld + d);
            else if (row < 0) c[i] = *reinterpret_cast<const uint4*>(mem + q * 8);
        }
    } else {
        for (int q = threadIdx.x; q < u.rows * (D / 8); q += kAppendThreads) {
            const int row = q / (D / 8), d = q % (D / 8) * 8;
            *reinterpret_cast<uint4*>(tile + (u.offset + row) * kPitch + d) =
                *reinterpret_cast<const uint4*>(src + row * ld + d);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int q = i * kAppendThreads + threadIdx.x;
            const int d = q / 128 * 16 + q % 16, n0 = q / 64 % 2 * 32 + q % 64 / 16 * 4;
            uint4 old = make_uint4(0, 0, 0, 0);
            if (u.offset > n0) old = *reinterpret_cast<const uint4*>(mem + q * 8);
            uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int n = n0 + j / 4 * 16 + j % 4, row = n - u.offset;
                uint32_t x = row >= u.rows ? 0u : w[j / 2] >> (j % 2 * 16) & 0xFFFFu;
                if (row >= 0 && row < u.rows) x = tile[n * kPitch + d];
                w[j / 2] = j % 2 ? (w[j / 2] & 0xFFFFu) | x << 16 : (w[j / 2] & 0xFFFF0000u) | x;
            }
            c[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) *reinterpret_cast<uint4*>(mem + (i * kAppendThreads + threadIdx.x) * 8) = c[i];
    if (u.physical < 0) return;

    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) most = max(most, amax8_bits(c[i]));
    most = block_max(most, wave_max);
    const GroupScale g = make_group_scale(bf16_to_f32(most));
    const int64_t at = ((int64_t)u.physical * a.heads + head) * 2 + which;
    uint8_t* out = a.codes + at * (kKvBlock * D);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int q = i * kAppendThreads + threadIdx.x;
        // chunk q of the bf16 order: half q / 64 % 2 of a lane's 16 codes (two contraction steps of 32)
        *reinterpret_cast<uint2*>(out + (q / 128 * 64 + q % 64) * 16 + q / 64 % 2 * 8) = encode_chunk(c[i], g);
    }
    if (threadIdx.x == 0) a.scales[at] = g.s;
}

}  // namespace

int64_t kv_max_units(int64_t tokens, int64_t requests) {
    const int64_t n = (tokens + 62 * requests) / kKvBlock + requests;
    return n < tokens ? n : tokens;
}

hipError_t launch_kv_plan(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                          const int32_t* free_head, int32_t* table, int64_t width, int64_t requests, int64_t tokens,
                          int64_t max_new, int32_t* next_state, int32_t* next_free, int32_t* status, int32_t* units,
                          int64_t* slots, int64_t num_blocks, hipStream_t st) {
    PlanArgs a;
    a.state = reinterpret_cast<const int2*>(state);
    a.new_lens = new_lens;
    a.free_blocks = free_blocks;
    a.free_head = free_head;
    a.table = table;
    a.next_state = reinterpret_cast<int2*>(next_state);
    a.next_free = next_free;
    a.status = status;
    a.units = reinterpret_cast<int4*>(units);
    a.slots = slots;
    a.requests = (int)requests;
    a.tokens = (int)tokens;
    a.max_new = (int)max_new;
    a.width = (int)width;
    a.num_free = (int)num_free;
    a.num_units = (int)kv_max_units(tokens, requests);
    a.num_blocks = (int)num_blocks;
    a.max_ids = (int)((tokens + (kKvBlock - 1) * requests) / kKvBlock);
    const int items = slots ? a.tokens : a.num_units;    // never fewer rows than units
    const unsigned grid = (unsigned)((items + kPlanItems - 1) / kPlanItems), lds = (unsigned)(3 * requests * sizeof(uint32_t));
    if (requests <= kPlanThreads) kv_plan_kernel<1><<<grid, kPlanThreads, lds, st>>>(a);
    else if (requests <= 4 * kPlanThreads) kv_plan_kernel<4><<<grid, kPlanThreads, lds, st>>>(a);
    else kv_plan_kernel<16><<<grid, kPlanThreads, lds, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, int64_t tokens,
                            const int32_t* units, int64_t num_units, int64_t heads, int64_t D, uint8_t* codes,
                            float* scales, int64_t num_blocks, uint16_t* recent, int64_t recent_blocks, hipStream_t st) {
    AppendArgs a{k, v, reinterpret_cast<const KvUnit*>(units), codes, scales, recent, ldk, ldv,
                 (int)tokens, (int)heads, (int)num_blocks, (int)recent_blocks};
    const unsigned grid = (unsigned)(2 * heads * num_units);
    if (D == 64) kv_append_kernel<64><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<128><<<grid, kAppendThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace jetfp8
