// Which partial results a row of the attention has, and which of them its join reads: index arithmetic alone, so that host
// code can walk the same indices.
//
// A unit with `block` cache blocks before its own has ceil(block / 8) spans of 8 and, behind their partial results, its own
// block's: a row holds no more than those.  8 spans make a run.  Of spans that the unit's group shares, a run has one partial
// result, in the place of the last of them.
#pragma once

namespace jetfp8 {

constexpr int kKvSpan = 8;         // blocks of a span, the attention's unit of summation
constexpr int kKvRun = 8;          // spans of a run, its unit of joining

constexpr int join_spans(int block) { return (block + kKvSpan - 1) / kKvSpan; }
constexpr int join_runs(int block) { return (block + kKvRun * kKvSpan - 1) / (kKvRun * kKvSpan); }

// Shared spans of a unit, from the blocks that its record says are shared.  A record of other units may say anything; only
// complete spans before the unit's own block can be.
constexpr int join_shared(int block, int recorded) {
    const int most = recorded < block ? recorded : block;
    return most < 0 ? 0 : most / kKvSpan;
}

// Where the run that begins at a span has its first partial result.
constexpr int join_run_begin(int span, int shared) {
    const int end = span + kKvRun;
    return shared <= span ? span : (shared < end ? shared : end) - 1;
}

// Partial results of a row but its own block's.
constexpr int join_parts_of(int block, int shared) {
    return join_spans(block) - shared + (shared + kKvRun - 1) / kKvRun;
}

// Leading runs that are taken as one partial result each, the last of their spans'; below two they are as quick one by one.
constexpr int join_whole_runs(int shared) { return shared / kKvRun < 2 ? 0 : shared / kKvRun; }

}  // namespace jetfp8
