// lm_packed.h - sequences that lie packed one after another, their cache entries, and how their tokens are dealt to
// workgroups without a pass over the lengths: what the sources of libselscan_lm that take packed prompts share.
#pragma once

#include "lm_common.h"

namespace {

// Tokens or rows of a call: tokens are counted in 32 bits, and a count may pass the last by two blocks of the scan or by
// the rows that a thread of a step takes (65,536 at most).
constexpr int64_t kMaxTokens = (INT64_C(1) << 31) - (1 << 17);

struct Seqs {
    const int32_t *cu;     // [nseq + 1]
    const int32_t *slots;  // [nseq], or NULL: slot s
    const uint8_t *carry;  // [nseq], or NULL: none
    int64_t nslots;
    int tokens, nseq;
};

struct Range {
    int t0, len;
};

__device__ __forceinline__ int cu_at(const Seqs &q, int i) {
    const int v = q.cu[i];
    return v < 0 ? 0 : v > q.tokens ? q.tokens : v;
}
__device__ __forceinline__ Range range_of(const Seqs &q, int s) {
    const int a = cu_at(q, s), b = cu_at(q, s + 1);
    return {a, b > a ? b - a : 0};
}
// cache entry of sequence s, or -1
__device__ __forceinline__ int64_t slot_of(const Seqs &q, int s) {
    const int64_t v = q.slots ? q.slots[s] : s;
    return v >= 0 && v < q.nslots ? v : -1;
}

// Segments of z tokens, without a pass over the lengths: sequence s owns the segment numbers
// from floor(cu[s] / z) + s to the next sequence's first, exclusively.  They are at least
// ceil(len / z) and at least one (floor(a + b) + 1 >= ceil(b) + floor(a)), and all of them together at
// most floor(tokens / z) + nseq, which the host knows; those past a sequence's end have nothing to do.
struct Segment {
    int s, t0, len;  // its sequence
    int j;           // its number within the sequence (negative: none)
    int slot;        // the sequence's cache entry, or negative
    bool carry;
};
// entries past 2^31 are none: slots are int32
__device__ __forceinline__ int slot_in(const Seqs &q, int v) { return v >= 0 && v < q.nslots ? v : -1; }

// What is kept of a segment until the next one starts from it has a place of its own, its entry: floor(cu[s] / z) + j for
// segment j of sequence s.  A segment that is not its sequence's last ends at j z + z < len, so that entries of different
// sequences differ and all of them lie below floor(tokens / z): none is set aside for a sequence of one segment.
//
// The sequence of a segment is the last one whose first segment is not after it: a search 64 positions wide,
// whose last round also brings the offsets, slots and carries (one trip to memory in all for up to 64 sequences).
// Every lane of the wave takes part.  div_z: division by z.
//
// BY_ENTRY: the segment that starts from entry `seg` (the last sequence whose first entry is not after it is the entry's, or it
// is no one's and the segment found lies past that sequence's end).
template <bool BY_ENTRY = false, class F>
__device__ __forceinline__ Segment find_segment(const Seqs &q, int seg, F div_z, int lane) {
    constexpr int OWN = BY_ENTRY ? 0 : 1;  // numbers that a sequence has beyond its entries
    int lo = 0, n = q.nseq;
    while (n > 64) {
        const int step = (n + 63) >> 6, i = lane * step;
        const bool at_or_before = i < n && div_z(cu_at(q, lo + i)) + OWN * (lo + i) <= seg;
        int c = __popcll(__ballot(at_or_before));
        c = c < 1 ? 1 : c;
        lo += (c - 1) * step;
        n -= (c - 1) * step;
        n = n < step ? n : step;
    }
    const int i = lo + (lane < n ? lane : n - 1);
    const int a = cu_at(q, i), b = cu_at(q, i + 1);
    const int sl = q.slots ? q.slots[i] : i, ca = q.carry ? q.carry[i] : 0;
    int c = __popcll(__ballot(lane < n && div_z(a) + OWN * (lo + lane) <= seg));
    c = __builtin_amdgcn_readfirstlane(c < 1 ? 0 : c - 1);
    const int s = lo + c, t0 = __builtin_amdgcn_readlane(a, c), t1 = __builtin_amdgcn_readlane(b, c);
    return {__builtin_amdgcn_readfirstlane(s), t0, t1 > t0 ? t1 - t0 : 0,
            seg - __builtin_amdgcn_readfirstlane(div_z(t0)) + (BY_ENTRY ? 1 : -s), slot_in(q, __builtin_amdgcn_readlane(sl, c)),
            __builtin_amdgcn_readlane(ca, c) != 0};
}
// a sequence as one segment
__device__ __forceinline__ Segment whole_sequence(const Seqs &q, int s) {
    const Range r = range_of(q, s);
    const int sl = q.slots ? q.slots[s] : s, ca = q.carry ? q.carry[s] : 0;
    return {s, __builtin_amdgcn_readfirstlane(r.t0), __builtin_amdgcn_readfirstlane(r.len), 0,
            slot_in(q, __builtin_amdgcn_readfirstlane(sl)), __builtin_amdgcn_readfirstlane(ca) != 0};
}

// The sequence that stands at place `place` when whole sequences are dealt to the chip (up to 64 of them): longest first, and
// every second round of `round` sequences (those whose workgroups fill the compute units once) in rising order, so that the
// units that got a round's longest get the next one's shortest; `round` of 64 or more: longest first. Twenty-four prompts of 1 to 4,096 tokens, 27,591 in all, x 4,096
// channels: 636 us against 675 as they come, and 532 to 566 against 600 to 708 in four other orders of the same prompts.
__device__ __forceinline__ Segment dealt_sequence(const Seqs &q, int place, int round, int lane) {
    const int n = q.nseq, i = lane < n ? lane : n - 1;
    const int a = cu_at(q, i), b = cu_at(q, i + 1), len = b > a ? b - a : 0;
    const int sl = q.slots ? q.slots[i] : i, ca = q.carry ? q.carry[i] : 0;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane) ? 1 : 0;
    }
    const int k = place / round, first = k * round, m = n - first < round ? n - first : round;
    const int want = k & 1 ? first + m - 1 - (place - first) : place;
    const int s = __builtin_amdgcn_readfirstlane(__builtin_ctzll(__ballot(lane < n && rank == want)));
    return {s, __builtin_amdgcn_readlane(a, s), __builtin_amdgcn_readlane(len, s), 0,
            slot_in(q, __builtin_amdgcn_readlane(sl, s)), __builtin_amdgcn_readlane(ca, s) != 0};
}

}  // namespace
