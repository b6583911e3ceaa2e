// Walks the partial results that the attention's join reads, in its order, for every length of a row and every number of
// shared blocks that a record may hold, with the functions that the kernel uses.  With -DUNBOUNDED the record's number is
// taken as it is: the check must find that out.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <vector>

#include "jetfp8_join.h"

using namespace jetfp8;

static int shared_of(int block, int recorded) {
#ifdef UNBOUNDED
    return recorded / kKvSpan;
#else
    return join_shared(block, recorded);
#endif
}

static int whole_of(int shared, int runs) {
#ifdef UNBOUNDED
    return shared / kKvRun < 2 ? 0 : std::min(shared / kKvRun, runs);
#else
    (void)runs;
    return join_whole_runs(shared);
#endif
}

static bool few_parts(int block, int shared) {
    const int runs = join_runs(block);
#ifdef UNBOUNDED
    if (runs > kKvRun) return false;               // (the number of parts means nothing)
#endif
    return runs > 1 && join_parts_of(block, shared) < kKvRun + 1;
}

// The three ways of attention_join_kernel: few parts at once, one sequence, run by run.
static std::vector<int> walk(int block, int recorded) {
    const int runs = join_runs(block), spans = join_spans(block), shared = shared_of(block, recorded);
    std::vector<int> at;
    auto take = [&](int first, int n, int step) {
        for (int s = 0; s < n; ++s) at.push_back(first + s * step);
    };
    if (few_parts(block, shared)) {
        for (int r = 0; r < runs; ++r) {
            const int begin = join_run_begin(r * kKvRun, shared);
            take(begin, std::min((r + 1) * kKvRun, spans) - begin, 1);
        }
    } else if (runs <= 1) {
        for (int s0 = join_run_begin(0, shared); s0 <= spans; s0 += kKvRun + 1)
            take(s0, std::min(kKvRun + 1, spans + 1 - s0), 1);
        return at;
    } else {
        const int whole = whole_of(shared, runs);
        take(kKvRun - 1, whole, kKvRun);
        for (int r = whole; r < runs; ++r) {
            const int s0 = join_run_begin(r * kKvRun, shared);
            take(s0, std::min((r + 1) * kKvRun, spans) - s0, 1);
        }
    }
    at.push_back(spans);
    return at;
}

// What the other kernels have written: a run's shared spans in the place of the last of them, the others one by one, the own
// block's behind them.
static std::vector<int> written(int block, int shared_blocks) {
    std::vector<int> at;
    const int spans = (block + 7) / 8, shared = shared_blocks / 8;
    for (int s = 0; s < spans; ++s)
        if (s >= shared || s % 8 == 7 || s == shared - 1) at.push_back(s);
    at.push_back(spans);
    return at;
}

int main() {
    const int odd[] = {INT_MIN, -64, -1, 1 << 16, 1 << 30, INT_MAX};
    int bad = 0, rows = 0;
    for (int block = 0; block <= 64 * 20; ++block) {
        const int spans = join_spans(block);
        auto check = [&](int recorded) {
            ++rows;
            for (int i : walk(block, recorded))
                if (i < 0 || i > spans) {
                    if (bad++ < 5) std::printf("%d blocks, %d recorded: part %d of %d\n", block, recorded, i, spans + 1);
                    break;
                }
        };
        for (int recorded = 0; recorded <= 64 * 22; ++recorded) check(recorded);
        for (int recorded : odd) check(recorded);
        for (int recorded = 0; recorded <= block; recorded += 8)
            if (walk(block, recorded) != written(block, recorded) ||
                join_parts_of(block, recorded / 8) + 1 != (int)written(block, recorded).size()) {
                if (bad++ < 5) std::printf("%d blocks, %d shared: other parts than those written\n", block, recorded);
            }
    }
    std::printf("%d rows, %d wrong\n", rows, bad);
    return bad != 0;
}
