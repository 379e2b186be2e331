// libselscan_lm - the short causal convolution and the selective scan on packed prompts and on
// single tokens, with states in a cache (causal_conv1d_packed_fwd, selscan_packed_fwd,
// causal_conv1d_step, selscan_step of include/selscan_lm.h).  MI355X (gfx950).
#include "lm_common.h"

#include <float.h>

#include <type_traits>

namespace selscan_rt {
thread_local char g_last_hip_error[160] = "no error";
}  // namespace selscan_rt

namespace {

// ------------------------------------------------------------------------------------
// packed sequences
// ------------------------------------------------------------------------------------

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
// units that got a round's longest get the next one's shortest. Twenty-four prompts of 1 to 4,096 tokens, 27,591 in all, x 4,096
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

// ------------------------------------------------------------------------------------
// convolution
// ------------------------------------------------------------------------------------

struct ConvParams {
    const void *x;
    const float *w, *bias;
    void *state, *out;
    Seqs q;
    int64_t x_stride, dim;
    int shift, silu, vec, wvec;
    int rows_per;  // step: rows a thread takes one after another
};

// filters of 8 channels, tap-major
template <int K>
__device__ __forceinline__ void load_filters(const ConvParams &p, int64_t c0, int nv, float (&f)[K][8], float (&b)[8]) {
    const float *w = p.w + c0 * K;
    if (nv >= 8) {
        float flat[8 * K];
#pragma unroll
        for (int i = 0; i < 8 * K; i += 4) {
            const float4 v = load_f4(w + i);
            flat[i] = v.x, flat[i + 1] = v.y, flat[i + 2] = v.z, flat[i + 3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int i = 0; i < K; ++i) f[i][e] = flat[e * K + i];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int i = 0; i < K; ++i) f[i][e] = e < nv ? w[e * K + i] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = p.bias && e < nv ? p.bias[c0 + e] : 0.f;
}

template <typename T, int K>
__device__ __forceinline__ void conv_row(const float (&f)[K][8], const float (&b)[8], const Raw8<T> *win, int silu_on,
                                         float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float a = b[e];
#pragma unroll
        for (int i = 0; i < K; ++i) a = fmaf(f[i][e], raw_f32(win[i], e), a);
        v[e] = silu_on ? silu(a) : a;
    }
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *p, int n, bool vec, const Raw8<T> &r) {
    if (vec && n >= 8) {
        *(uint4 *)p = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        if constexpr (sizeof(T) == 4) *(uint4 *)(p + 4) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= n) continue;
        if constexpr (sizeof(T) == 4) p[e] = __uint_as_float(r.w[e]);
        else p[e] = (T)(e & 1 ? r.w[e >> 1] >> 16 : r.w[e >> 1] & 0xFFFFu);
    }
}

// A thread takes 2^SHIFT tokens of 8 channels: 16, or 4 where runs of 16 would leave most of the chip without a
// wave (a thread's run of 16 is 1,400 instructions).
constexpr int kConvLong = 4, kConvShort = 2;

// One workgroup: a segment of one sequence, 8 channels per thread.  HBM bound on
// long batches (27,591 tokens x 4,096 channels bf16: 99 us, 4.6 TB/s); on short ones the chain of loads counts, so the
// first rows come before the cache's.  Every row of the segment and the width-1 rows before it are read once by the thread (its neighbours in
// time read those again, from L2).  A sequence's first segment holds at least its first width-1 tokens,
// so its threads alone need the cached rows: they read them, and then write the sequence's last
// rows to the cache, in program order on the same addresses.
template <typename T, int K, int SHIFT>
__global__ __launch_bounds__(256) void conv_packed(ConvParams p) {
    constexpr int R = 1 << SHIFT, B = 4;  // B: rows in flight at a time (8: a wave less per SIMD, 103 us for the 99 above)
    static_assert(R >= K - 1, "a sequence's first segment holds its first width - 1 tokens");
    const int seg = blockIdx.x;
    const int64_t c0 = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 8;
    const bool live = c0 < p.dim;
    const int nv = !live ? 0 : (int)(p.dim - c0 < 8 ? p.dim - c0 : 8);
    const bool vec = p.vec != 0;
    const Segment g = find_segment(p.q, seg, [](int v) { return v >> SHIFT; }, threadIdx.x & 63);
    const int first = g.j << SHIFT;
    if (!live || g.j < 0 || (g.j > 0 && first >= g.len)) return;
    const T *x = (const T *)p.x + (int64_t)g.t0 * p.x_stride + c0;
    T *out = (T *)p.out + (int64_t)g.t0 * p.dim + c0;
    T *st = K > 1 && p.state && g.slot >= 0 ? (T *)p.state + (int64_t)g.slot * (K - 1) * p.dim + c0 : nullptr;
    const int n = g.len - first < R ? g.len - first : R;
    Raw8<T> win[B + K - 1];  // the rows before the current block, then the block
    auto load_block = [&](int u0) {
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const int t = first + u0 + u < g.len ? first + u0 + u : g.len - 1;
            win[K - 1 + u] = load_raw8(x + (int64_t)t * p.x_stride, nv, vec);
        }
    };
    if (n > 0) load_block(0);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        win[i] = Raw8<T>{};
        if (first > 0) win[i] = load_raw8(x + (int64_t)(first - (K - 1) + i) * p.x_stride, nv, vec);
        else if (st && g.carry) win[i] = load_raw8(st + i * p.dim, nv, vec);
    }
    float f[K][8], b[8];
    load_filters<K>(p, c0, nv, f, b);
    if constexpr (K > 1) {
        if (first == 0 && st) {
#pragma unroll
            for (int i = 0; i < K - 1; ++i) {
                const int at = g.len - (K - 1) + i;  // row of the sequence, or a cached one where negative
                Raw8<T> r{};
                if (at >= 0) r = load_raw8(x + (int64_t)at * p.x_stride, nv, vec);
#pragma unroll
                for (int o = 0; o < K - 1; ++o)
                    if (at < 0 && o == at + K - 1) r = win[o];
                store_raw8(st + i * p.dim, nv, vec, r);
            }
        }
    }
#pragma unroll
    for (int u0 = 0; u0 < R; u0 += B) {
        if (u0 >= n) break;
        if (u0 > 0) load_block(u0);
#pragma unroll
        for (int u = 0; u < B; ++u) {
            if (u0 + u < n) {
                float v[8];
                conv_row<T, K>(f, b, win + u, p.silu, v);
                T *o = out + (int64_t)(first + u0 + u) * p.dim;
                // with the streaming hint 4,097 x 1,536 fp32 15.4 us instead of 16.4, bf16 rows 101 instead of 99
                if constexpr (sizeof(T) == 4) store8_stream(o, nv, vec, v);
                else store8(o, nv, vec, v);
            }
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) win[i] = win[B + i];
    }
}

// One token per sequence: 8 channels per thread, rows_per rows one after another with the filters
// held.  Per row and channel the cache's width-1 values move in and out, shifted by one.  256 rows x 4,096 channels bf16: 7.8
// us, of which the bytes at the rate of a large copy are 3.2 and an empty launch about 2.5; one row 2.8.
template <typename T, int K>
__global__ __launch_bounds__(64) void conv_step(ConvParams p) {
    const int64_t c0 = ((int64_t)blockIdx.x * 64 + threadIdx.x) * 8;
    if (c0 >= p.dim) return;
    const int nv = (int)(p.dim - c0 < 8 ? p.dim - c0 : 8);
    const bool vec = p.vec != 0;
    float f[K][8], b[8];
    load_filters<K>(p, c0, nv, f, b);
    const int r0 = blockIdx.y * p.rows_per;
    for (int i = 0; i < p.rows_per; ++i) {
        const int r = r0 + i;
        if (r >= p.q.tokens) break;
        const int64_t slot = slot_of(p.q, r);
        Raw8<T> win[K];
        win[K - 1] = load_raw8((const T *)p.x + r * p.x_stride + c0, nv, vec);
        T *st = K > 1 ? (T *)p.state + (slot < 0 ? 0 : slot) * (K - 1) * p.dim + c0 : nullptr;
#pragma unroll
        for (int t = 0; t < K - 1; ++t) {
            win[t] = Raw8<T>{};
            if (slot >= 0) win[t] = load_raw8(st + t * p.dim, nv, vec);
        }
        float v[8];
        conv_row<T, K>(f, b, win, p.silu, v);
        store8((T *)p.out + r * p.dim + c0, nv, vec, v);
        if (slot >= 0) {
#pragma unroll
            for (int t = 0; t < K - 1; ++t) store_raw8(st + t * p.dim, nv, vec, win[t + 1]);
        }
    }
}

int conv_check(const void *x, int64_t x_stride, const float *weight, const float *bias, const void *state, bool packed,
               unsigned flags, const void *out, int64_t rows, int64_t nseq, int64_t nslots, int64_t dim, int64_t width,
               int io_dtype, const int32_t *cu, const int32_t *slots, const uint8_t *carry, bool *nothing) {
    *nothing = false;
    if (rows < 0 || nseq < 0 || nslots < 0 || dim < 0) return SELSCAN_E_SHAPE;
    if (!io_known(io_dtype) || (flags & ~SELSCAN_FLAG_SILU) || width < 1 || width > 4) return SELSCAN_E_UNSUPPORTED;
    if (rows > kMaxTokens || nseq > INT32_MAX / 2 || dim > INT32_MAX) return SELSCAN_E_UNSUPPORTED;
    if (dim == 0 || nseq == 0) {
        *nothing = true;
        return nseq == 0 && rows > 0 && dim > 0 ? SELSCAN_E_SHAPE : SELSCAN_OK;
    }
    if (x_stride < dim) return SELSCAN_E_SHAPE;
    if (state && !slots && nslots < nseq) return SELSCAN_E_SHAPE;
    const int64_t tok = mul_size(rows, x_stride), cache = mul_size(mul_size(nslots, dim), width);
    if (tok < 0 || mul_size(rows, dim) < 0 || cache < 0 || mul_size(nslots, dim) < 0) return SELSCAN_E_SHAPE;
    if ((rows > 0 && (!x || !out)) || !weight || (packed && !cu) || (!packed && width > 1 && !state)) return SELSCAN_E_NULL;
    const size_t s = io_bytes(io_dtype);
    if (!span_aligned(x, s) || !span_aligned(out, s) || !span_aligned(state, s) || !span_aligned(weight, 4) ||
        !span_aligned(bias, 4) || !span_aligned(cu, 4) || !span_aligned(slots, 4))
        return SELSCAN_E_ALIGN;
    const Span in[] = {{x, strided_bytes(rows, dim, x_stride, s)},
                       {weight, (size_t)dim * width * 4},
                       {bias, (size_t)dim * 4},
                       {cu, (size_t)(nseq + 1) * 4},
                       {slots, (size_t)nseq * 4},
                       {carry, (size_t)nseq}};
    const Span outs[] = {{out, (size_t)rows * dim * s}, {state, (size_t)nslots * (width - 1) * dim * s}};
    return any_alias(in, 6, outs, 2) ? SELSCAN_E_ALIAS : SELSCAN_OK;
}

ConvParams conv_params(const void *x, int64_t x_stride, const float *weight, const float *bias, const int32_t *cu,
                       const int32_t *slots, const uint8_t *carry, void *state, unsigned flags, void *out, int64_t rows,
                       int64_t nseq, int64_t nslots, int64_t dim, int io_dtype) {
    ConvParams p{};
    p.x = x, p.w = weight, p.bias = bias, p.state = state, p.out = out;
    p.q = {cu, slots, carry, nslots, (int)rows, (int)nseq};
    p.x_stride = x_stride, p.dim = dim;
    p.silu = (flags & SELSCAN_FLAG_SILU) ? 1 : 0;
    const size_t s = io_bytes(io_dtype);
    p.vec = dim % 8 == 0 && x_stride * s % 16 == 0 && span_aligned(x, 16) && span_aligned(out, 16) && span_aligned(state, 16);
    return p;
}

// ------------------------------------------------------------------------------------
// scan
// ------------------------------------------------------------------------------------

struct ScanParams {
    const void *x, *delta, *z, *B, *C;
    const float *A, *D, *bias;
    void *y;
    float *h;     // cache, or NULL
    float *seg;   // split: [entries][dim][16] end state of a segment, from zero but for a sequence's first
    float *sdt;   // split: [entries][dim] sum of delta over the segment
    Seqs q;
    int64_t dim, bc_stride, z_stride;
    int softplus;
    int size;      // split: tokens of a segment, and division by it
    FastDiv dsize;
    int ntiles;    // blocks of 64 channels
    int round;     // whole sequences: how many fill the compute units once (0: taken as they come)
    int joined;    // split: scan_join runs between the launches
    int entries;   // split: of seg and sdt
    int rows_per;  // step: rows a thread takes one after another
};

// a value of another lane of the group of four: lane CTRL & 3, CTRL >> 2 & 3, ... of lanes 0, 1, 2, 3
template <int CTRL>
__device__ __forceinline__ float quad(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int I>
__device__ __forceinline__ float quad_lane(float v) {
    return quad<I * 0x55>(v);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;

// The scan, one wave per 16 channels of a sequence or segment: the four lanes of a channel hold four of
// its 16 states each and walk its tokens in order.
//
//  - Per (token, channel, state): mul, exp, mul, fma, fma.  What is done per token and channel (softplus, the
//    gate, conversions, the store) is shared out: lane q of a channel does it for token q of every four, and
//    the others read delta and delta x from it with DPP, as an operand of the products that use them.  The
//    sums over states of four tokens are transposed and added across the four lanes at once.
//  - B and C are the same for all channels: a block of 16 tokens of them is converted once per wave to fp32
//    in LDS, and read back as one 16-byte broadcast each per token.  The wave reads only what it wrote itself,
//    in order: no barrier.
//  - The next block's x, delta, z, B and C are in flight during a block's arithmetic.
//
// Bound by instruction issue (34 VALU instructions and 2 LDS accesses per token of a wave, with gate and softplus; 27,591 tokens
// in 24 sequences x 4,096 channels bf16: 550 to 605 us, about four fifths of it VALU issue).  A lane per
// channel with all 16 states and B and C as scalar operands needs a tenth less issue per element, but a
// quarter of the waves, each token taking four times as long: measured slower wherever the chip was not full
// of long sequences of equal length.
//
// The four waves of a workgroup take neighbouring channels, 128 bytes of a bf16 row together.
//
// Segments of a sequence run side by side in two launches.  The first takes segment 0 from the sequence's true
// start, y and all, and of the others but the last only the end state from a zero start and the sum of delta, which
// make the segment a map h -> exp(A sum delta) h + end.  The second takes all but segment 0, each from the
// state that the maps before it lead to.  Whole sequences are the first launch alone, one segment each.
constexpr int kBlk = 16;  // tokens per block

// A as an exponent of 2.  An infinite one (a state that forgets at once) becomes the largest number, whose product with any
// delta that is not 0 is as good, and with the 0 of a token past the end is 0.
__device__ __forceinline__ float rate(float A) {
    const float a = A * kLog2e;
    return fabsf(a) == INFINITY ? copysignf(FLT_MAX, a) : a;
}

// The state after a segment, a map h -> 2^x h + end.  A negative delta can let x pass fp32's exponents (as a decay can on
// the other side) over a segment whose own states do not, and a state of 0 has to stay 0: the power goes in as two finite
// ones of half the exponent.  (Past 2 * 127 only a state below 2^-126 would not be infinite.)
__device__ __forceinline__ float through_map(float h, float x, float end) {
    const float e = __builtin_amdgcn_exp2f(__builtin_amdgcn_fmed3f(0.5f * x, -126.f, 127.f));
    return fmaf(e, e * h, end);
}

struct Piece {
    int t0, len;          // tokens
    const float *h_in;    // [dim][16] start state, or NULL: zero
    float *h_out, *sdt;   // [dim][16], or NULL: not kept; [dim], of a map only
};

// FULL: y and the last state.  Else the map.
template <typename T, bool ZOH, bool FULL, bool GATE>
__device__ __forceinline__ void scan_piece(const ScanParams &p, const Piece &w, float (*bc)[2 * kN], int64_t c0, int lane,
                                           const float (&a2)[4], float (&h)[4]) {
    const int cl = lane >> 2, q = lane & 3;
    const int64_t dim = p.dim;
    const bool live = c0 + cl < dim;
    const int64_t ch = live ? c0 + cl : dim - 1;  // lanes past the last channel repeat it
    const int len = w.len;
    const float Dd = FULL && p.D ? p.D[ch] : 0.f, bias = p.bias ? p.bias[ch] : 0.f;
    // Bytes: a row's start is uniform, and what a lane adds to it for the tokens of a block are four constants (the host
    // admits strides whose 16 rows lie within 32 bits), cut off at the last token's
    const uint32_t row = (uint32_t)dim * sizeof(T), zrow = (uint32_t)p.z_stride * sizeof(T), bcrow = (uint32_t)p.bc_stride * sizeof(T);
    const uint32_t chb = (uint32_t)ch * sizeof(T);
    uint32_t at[4], zat[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = (4 * j + q) * row + chb, zat[j] = (4 * j + q) * zrow + chb;
    auto row_of = [&](const void *a, int t, uint32_t bytes) { return (const char *)a + (int64_t)(w.t0 + t) * bytes; };
    // this lane's eighth of a token's B (q < 2) and C
    const char *src = (const char *)(q < 2 ? (const T *)p.B + 8 * q : (const T *)p.C + 8 * (q - 2));

    struct Block {
        uint32_t x[4], d[4], z[4];  // tokens 4 j + q (as 32-bit words: 16-bit pairs would tie two loads together)
        Raw8<T> bc;                 // token lane / 4
    };
    auto raw = [](const char *a) -> uint32_t {
        if constexpr (sizeof(T) == 4) return __float_as_uint(*(const T *)a);
        else return *(const T *)a;
    };
    auto val = [](uint32_t w) { return __uint_as_float(sizeof(T) == 4 ? w : w << 16); };
    auto load = [&](int t, Block &b) {
        const int ts = t < len ? t : len - 1;
        const uint32_t left = len - 1 - ts < kBlk - 1 ? len - 1 - ts : kBlk - 1;
        const uint32_t end = left * row + chb, zend = left * zrow + chb, bcat = (cl < (int)left ? cl : left) * bcrow;
        const char *x = row_of(p.x, ts, row), *dl = row_of(p.delta, ts, row), *z = row_of(p.z, ts, zrow);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t o = at[j] < end ? at[j] : end, oz = zat[j] < zend ? zat[j] : zend;
            b.x[j] = raw(x + o);
            b.d[j] = raw(dl + o);
            b.z[j] = GATE ? raw(z + oz) : 0u;
        }
        if (FULL || q < 2) b.bc = load_any8((const T *)(row_of(src, ts, bcrow) + bcat));
    };
    float sum = 0.f;
    auto compute = [&](int t, const Block &b) {
        if (FULL || q < 2) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = raw_f32(b.bc, e);
            if (t + kBlk > len && t + cl >= len) {  // (the last token's again, and 0 times an infinity is not 0)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
            }
            *(float4 *)&bc[cl][8 * q] = make_float4(v[0], v[1], v[2], v[3]);
            *(float4 *)&bc[cl][8 * q + 4] = make_float4(v[4], v[5], v[6], v[7]);
        }
        float d[4], dx[4], gate[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = val(b.d[j]) + bias;
        if (p.softplus) {
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = softplus(d[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dx[j] = d[j] * val(b.x[j]);
            gate[j] = GATE ? silu(val(b.z[j])) : 1.f;
        }
        if (t + kBlk > len) {  // past the end: the identity step
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + 4 * j + q >= len) d[j] = dx[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += d[j];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t + 4 * j >= len) break;
            float yt[4];
            // what does not wait for the state first, for four tokens: e = exp(delta A) and u = delta B x
            float4 Bq[4], Cq[4];
            float e[4][4], u[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Bq[i] = *(const float4 *)&bc[4 * j + i][4 * q];
                if constexpr (FULL) Cq[i] = *(const float4 *)&bc[4 * j + i][kN + 4 * q];
            }
            auto coef = [&](auto ic) {
                constexpr int I = decltype(ic)::value;
                const float bv[4] = {Bq[I].x, Bq[I].y, Bq[I].z, Bq[I].w};
#pragma unroll
                for (int n = 0; n < 4; ++n) e[I][n] = quad_lane<I>(d[j]) * a2[n];
#pragma unroll
                for (int n = 0; n < 4; ++n) u[I][n] = quad_lane<I>(dx[j]) * bv[n];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float arg = e[I][n];
                    e[I][n] = __builtin_amdgcn_exp2f(arg);
                    if constexpr (ZOH) u[I][n] *= zoh_phi(e[I][n], arg);
                }
            };
            coef(std::integral_constant<int, 0>{});
            coef(std::integral_constant<int, 1>{});
            coef(std::integral_constant<int, 2>{});
            coef(std::integral_constant<int, 3>{});
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int n = 0; n < 4; ++n) h[n] = fmaf(e[i][n], h[n], u[i][n]);
                if constexpr (FULL) yt[i] = fmaf(Cq[i].w, h[3], fmaf(Cq[i].z, h[2], fmaf(Cq[i].y, h[1], Cq[i].x * h[0])));
            }
            if constexpr (FULL) {
                // lane q gets the sum of yt[q] over the four lanes
                const bool b0 = q & 1, b1 = q & 2;
                const float r0 = (b0 ? yt[1] : yt[0]) + quad<kQuadXor1>(b0 ? yt[0] : yt[1]);
                const float r1 = (b0 ? yt[3] : yt[2]) + quad<kQuadXor1>(b0 ? yt[2] : yt[3]);
                const float r = (b1 ? r1 : r0) + quad<kQuadXor2>(b1 ? r0 : r1);
                const float v = fmaf(Dd, val(b.x[j]), r) * gate[j];
                if (live && t + 4 * j + q < len) *(T *)((char *)row_of(p.y, t, row) + at[j]) = Io<T>::to(v);
            }
        }
    };
    // two buffers named in turn: copying one to the other would wait for every load and store in flight
    Block even, odd;
    if (len > 0) load(0, even);
    // (a block past the end loads the last token again: where a load depended on a condition, the wait before
    // the next use would be for all of them)
    for (int t = 0; t < len; t += 2 * kBlk) {
        load(t + kBlk, odd);
        compute(t, even);
        if (t + kBlk >= len) break;
        load(t + 2 * kBlk, even);
        compute(t + kBlk, odd);
    }
    if (!live) return;
    if (w.h_out) *(float4 *)(w.h_out + ch * kN + 4 * q) = make_float4(h[0], h[1], h[2], h[3]);
    if constexpr (!FULL) {
        sum += quad<kQuadXor1>(sum);
        sum += quad<kQuadXor2>(sum);
        if (q == 0) w.sdt[ch] = sum;
    }
}

// LAUNCH 0, 1: the first and the second launch above.
template <typename T, bool ZOH, bool GATE, int LAUNCH>
__global__ __launch_bounds__(256) void scan_packed(ScanParams p) {
    __shared__ __attribute__((aligned(16))) float bc_lds[4][kBlk][2 * kN];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & 3;
    // channel blocks of a segment follow one another: they go to different XCDs, so that a long
    // sequence does not load one of them
    const int seg = blockIdx.x / p.ntiles, tile = blockIdx.x - seg * p.ntiles;
    const int64_t dim = p.dim, c0 = (int64_t)tile * 64 + wave * 16;
    if (c0 >= dim) return;
    const int64_t ch = c0 + (lane >> 2) < dim ? c0 + (lane >> 2) : dim - 1;
    const float4 av = load_f4(p.A + ch * kN + 4 * q);
    const bool split = p.seg != nullptr;
    const auto div = [&](int v) { return (int)fdiv((uint32_t)v, p.dsize); };
    const Segment g = LAUNCH == 1 ? find_segment<true>(p.q, seg, div, lane)
                      : split     ? find_segment(p.q, seg, div, lane)
                      : p.round ? dealt_sequence(p.q, seg, p.round, lane)
                                : whole_sequence(p.q, seg);
    const int first = split ? g.j * p.size : 0, size = split ? p.size : g.len;
    if (g.j < LAUNCH || (g.j > 0 && first >= g.len)) return;
    const bool last = g.len - first <= size;
    if (LAUNCH == 0 && g.j > 0 && last) return;
    const int64_t st = dim * kN;
    float *cache = p.h && g.slot >= 0 ? p.h + g.slot * st : nullptr;
    Piece w{g.t0 + first, last ? g.len - first : size, nullptr, nullptr, nullptr};
    if (last) w.h_out = cache;
    else if (LAUNCH == 0) w.h_out = p.seg + (int64_t)(seg - g.s) * st;
    if (LAUNCH == 0) w.sdt = split ? p.sdt + (int64_t)(seg - g.s) * dim : nullptr;

    const float a2[4] = {rate(av.x), rate(av.y), rate(av.z), rate(av.w)};
    float h[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (LAUNCH == 0) {
        if (g.j == 0 && cache && g.carry) {
            const float4 v = *(const float4 *)(cache + ch * kN + 4 * q);
            h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        }
        if (g.j == 0) scan_piece<T, ZOH, true, GATE>(p, w, bc_lds[wave], c0, lane, a2, h);
        else scan_piece<T, ZOH, false, false>(p, w, bc_lds[wave], c0, lane, a2, h);
    } else {
        // the state this segment starts from: the maps of those before it, in order, or what scan_join left
        const int entry0 = seg - (g.j - 1);  // of the sequence
        const float *e = p.seg + entry0 * st + ch * kN + 4 * q;
        const float *d = p.sdt + entry0 * dim + ch;
        const int n = p.joined ? 1 : g.j;
        if (p.joined) e += (g.j - 1) * st;
        constexpr int U = 4;  // maps loaded ahead
        for (int i0 = 0; i0 < n; i0 += U) {
            float4 ev[U];
            float dv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u < n ? i0 + u : n - 1;
                ev[u] = *(const float4 *)(e + i * st);
                dv[u] = i > 0 ? d[i * dim] : 0.f;  // (segment 0 is a state, not a map)
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u >= n) break;
                h[0] = through_map(h[0], a2[0] * dv[u], ev[u].x);
                h[1] = through_map(h[1], a2[1] * dv[u], ev[u].y);
                h[2] = through_map(h[2], a2[2] * dv[u], ev[u].z);
                h[3] = through_map(h[3], a2[3] * dv[u], ev[u].w);
            }
        }
        scan_piece<T, ZOH, true, GATE>(p, w, bc_lds[wave], c0, lane, a2, h);
    }
}

// Joins the segments of long sequences between the launches: one thread per (sequence, channel, state) walks the
// maps in order and leaves the state at the end of each segment in its place.  Sequences are dealt out by their numbers, or,
// where there are more sequences than entries, by those entries that are their first.
__global__ __launch_bounds__(64) void scan_join(ScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x, st = p.dim * kN, ch = i / kN < p.dim ? i / kN : p.dim - 1;
    const bool live = i < st, by_entry = p.q.nseq > p.entries;
    const float a2 = rate(p.A[live ? i : 0]);
    const auto div = [&](int v) { return (int)fdiv((uint32_t)v, p.dsize); };
    for (int b = blockIdx.y; b < (by_entry ? p.entries : p.q.nseq); b += gridDim.y) {
        Range rg;
        if (by_entry) {
            const Segment g = find_segment<true>(p.q, b, div, threadIdx.x);
            if (g.j != 1) continue;  // not its sequence's first
            rg = {g.t0, g.len};
        } else {
            rg = range_of(p.q, b);
        }
        const int first = div(rg.t0);
        const int n = rg.len > 0 ? div(rg.len - 1) : 0;  // all but the last
        if (n >= 2 && live) {
            float *e = p.seg + (int64_t)first * st + i;
            const float *d = p.sdt + (int64_t)first * p.dim + ch;
            float h = e[0];
            constexpr int U = 16;  // segments loaded ahead
            for (int j0 = 1; j0 < n; j0 += U) {
                float ev[U], dv[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t j = j0 + u < n ? j0 + u : n - 1;
                    ev[u] = e[j * st];
                    dv[u] = d[j * p.dim];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (j0 + u >= n) break;
                    h = through_map(h, a2 * dv[u], ev[u]);
                    e[(j0 + u) * st] = h;
                }
            }
        }
    }
}

typedef float NtF4 __attribute__((ext_vector_type(4), aligned(4)));
// 4 values from any address aligned to one
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Four {
    T v[4];
};

// One token per sequence.  Four lanes per channel hold four states each, so that a wave moves 16 channels' states as
// 1 KB of adjacent memory in and out; y is summed over the four lanes.  HBM bound by the states (128
// bytes per row and channel of fp32 state in and out) where there are many rows: 256 rows x 4,096 channels bf16 29.6 us, 4.8
// TB/s, from states that are in no cache; one row x 1,536 3.3 us.  A, D and bias are held
// over the rows_per rows that a thread takes.
//
// The next row's loads are in flight during a row's arithmetic, none of them under a condition (that would make the wait
// for one a wait for all): a row without an entry of the cache reads A in its place, which has an entry's layout, and
// takes zero.
//
// NT: the states without a place in the caches.
template <typename T, bool ZOH, bool NT>
__global__ __launch_bounds__(256) void scan_step(ScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, ch = i >> 2;
    if (ch >= p.dim) return;  // whole groups of four lanes leave
    const int n0 = (int)(i & 3) * 4;
    const float4 a = load_f4(p.A + ch * kN + n0);
    const float a2[4] = {rate(a.x), rate(a.y), rate(a.z), rate(a.w)};
    const float Dd = p.D ? p.D[ch] : 0.f, bias = p.bias ? p.bias[ch] : 0.f;
    struct Row {
        int64_t slot;
        float4 h;
        Four<T> B, C;
        T d, x, z;
    };
    auto fetch = [&](int r) {
        Row w;
        w.slot = slot_of(p.q, r);
        const float *hp = (w.slot >= 0 ? p.h + w.slot * p.dim * kN : p.A) + ch * kN + n0;
        if constexpr (NT) w.h = __builtin_bit_cast(float4, __builtin_nontemporal_load((const NtF4 *)hp));
        else w.h = load_f4(hp);
        w.B = *(const Four<T> *)((const T *)p.B + r * p.bc_stride + n0);
        w.C = *(const Four<T> *)((const T *)p.C + r * p.bc_stride + n0);
        w.d = ((const T *)p.delta)[r * p.dim + ch];
        w.x = ((const T *)p.x)[r * p.dim + ch];
        w.z = (p.z ? (const T *)p.z + r * p.z_stride : (const T *)p.x + r * p.dim)[ch];
        return w;
    };
    auto step = [&](int r, const Row &w) {
        float h[4] = {w.h.x, w.h.y, w.h.z, w.h.w};
        float d = Io<T>::f32(w.d) + bias;
        if (p.softplus) d = softplus(d);
        const float xv = Io<T>::f32(w.x), dx = d * xv;
        float acc = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float arg = d * a2[n], e = __builtin_amdgcn_exp2f(arg);
            float g = dx;
            if constexpr (ZOH) g = dx * zoh_phi(e, arg);
            h[n] = fmaf(e, w.slot >= 0 ? h[n] : 0.f, g * Io<T>::f32(w.B.v[n]));
            acc = fmaf(Io<T>::f32(w.C.v[n]), h[n], acc);
        }
        if (w.slot >= 0) {
            NtF4 *hp = (NtF4 *)(p.h + (w.slot * p.dim + ch) * kN + n0);
            const NtF4 v = {h[0], h[1], h[2], h[3]};
            if constexpr (NT) __builtin_nontemporal_store(v, hp);
            else *hp = v;
        }
        acc += quad<kQuadXor1>(acc);
        acc += quad<kQuadXor2>(acc);
        if (n0 == 0) {
            float v = fmaf(Dd, xv, acc);
            if (p.z) v *= silu(Io<T>::f32(w.z));
            ((T *)p.y)[r * p.dim + ch] = Io<T>::to(v);
        }
    };
    const int r0 = blockIdx.y * p.rows_per, r1 = p.rows_per < p.q.tokens - r0 ? r0 + p.rows_per : p.q.tokens;
    Row w = fetch(r0), next;
    for (int r = r0; r < r1; r += 2) {
        next = fetch(r + 1 < r1 ? r + 1 : r);
        step(r, w);
        if (r + 1 >= r1) break;
        w = fetch(r + 2 < r1 ? r + 2 : r + 1);
        step(r + 1, next);
    }
}

// Tokens per segment, or 0: whole sequences.
//  - In clocks of a SIMD a wave's token was measured at 245 alone and 150 beside others, a map's at 115.  Whole sequences take
//    the longest alone, or all evenly plus a quarter for lengths that do not even out; segments take both passes, and 25,000
//    for the second launch and the join.
//  - Segments of multiples of 16 (a block) that give each compute unit four workgroups: measured, 4,097 tokens x 1,536
//    channels fp32 67 us at 96 tokens (4.0 workgroups per unit), 69 at 64, 75 at 112, 85 at 176 and 372 whole; 505 tokens in 8
//    sequences x 1,536 bf16 17.6 us at 16, 18.4 at 32, 21 at 64 and 28.5 whole; 27,591 tokens in 24 sequences x 4,096 746 us
//    at 256, and 537 whole.
constexpr int kSimds = 1024, kUnits = 256;  // MI355X: 256 compute units of 4
// Segments of the longest sequence up to which the second launch walks the maps itself, without a join (the scan's time in
// us, walked and joined, bf16: 256 tokens x 1,536 in 16 segments 12.3 and 15.2, 512 in 32 18.2 and 20.1, 4,097 in 42 61.3 and
// 62.7; 800 x 512 in 50 16.5 and 17.6; 1,000 x 768 in 62 23.6 and 21.9; 1,300 x 512 in 81 23.9 and 23.1; 2,048 x 512 in 128 36
// and 30)
constexpr int kWalk = 48;

int64_t segments(int64_t tokens, int64_t nseq, int64_t size) { return tokens / size + nseq; }

int split_size(int64_t tokens, int64_t max_seqlen, int64_t dim) {
    const int64_t tiles = (dim + 15) / 16, blocks = (dim + 63) / 64;
    const int64_t longest = max_seqlen < tokens ? max_seqlen : tokens;
    const int64_t share = (tokens * tiles + kSimds - 1) / kSimds;  // token times of a SIMD if all is even
    const int64_t whole = longest * 245 > share * 188 ? longest * 245 : share * 188;
    if (whole <= share * 265 + 25000) return 0;
    const int64_t even = (tokens * blocks / (4 * kUnits) + 8) / 16 * 16;
    const int size = (int)(even < 16 ? 16 : even > 4096 ? 4096 : even);
    return 2 * size <= longest ? size : 0;
}

size_t packed_workspace(int64_t tokens, int64_t max_seqlen, int64_t dim) {
    const int size = split_size(tokens, max_seqlen, dim);
    return size ? (size_t)(tokens / size) * (size_t)dim * (kN + 1) * sizeof(float) : 0;
}

struct ScanArgs {
    const void *x, *delta;
    const float *A;
    const void *B, *C;
    int64_t bc_stride;
    const float *D;
    const void *z;
    int64_t z_stride;
    const float *bias;
    unsigned flags;
    const int32_t *cu, *slots;
    const uint8_t *carry;
    float *h;
    void *y;
    int64_t rows, nseq, nslots, dim, dstate;
    int dtype;
    void *ws;
    size_t ws_need, ws_bytes;
    bool packed;
};

constexpr int64_t kMaxStride = INT64_C(1) << 26;

int scan_check(const ScanArgs &a, bool *nothing) {
    *nothing = false;
    if (a.rows < 0 || a.nseq < 0 || a.nslots < 0 || a.dim < 0 || a.dstate < 0) return SELSCAN_E_SHAPE;
    if (!io_known(a.dtype) || (a.flags & ~(SELSCAN_FLAG_DELTA_SOFTPLUS | SELSCAN_FLAG_ZOH)) || a.dstate != kN)
        return SELSCAN_E_UNSUPPORTED;
    if (a.rows > kMaxTokens || a.nseq > INT32_MAX / 2 || a.dim > INT32_MAX) return SELSCAN_E_UNSUPPORTED;
    if (a.dim == 0 || a.nseq == 0) {
        *nothing = true;
        return a.nseq == 0 && a.rows > 0 && a.dim > 0 ? SELSCAN_E_SHAPE : SELSCAN_OK;
    }
    if (a.bc_stride < kN || (a.z && a.z_stride < a.dim)) return SELSCAN_E_SHAPE;
    // 16 rows of any array within 32 bits
    if (a.packed && (a.dim > kMaxStride || a.bc_stride > kMaxStride || (a.z && a.z_stride > kMaxStride))) return SELSCAN_E_UNSUPPORTED;
    if (a.h && !a.slots && a.nslots < a.nseq) return SELSCAN_E_SHAPE;
    if (mul_size(a.rows, a.bc_stride) < 0 || (a.z && mul_size(a.rows, a.z_stride) < 0) || mul_size(a.rows, a.dim) < 0 ||
        mul_size(a.nslots, a.dim * kN) < 0)
        return SELSCAN_E_SHAPE;
    if ((a.rows > 0 && (!a.x || !a.delta || !a.B || !a.C || !a.y)) || !a.A || (a.packed && !a.cu) || (!a.packed && !a.h))
        return SELSCAN_E_NULL;
    const size_t s = io_bytes(a.dtype);
    const void *io[] = {a.x, a.delta, a.B, a.C, a.z, a.y};
    for (const void *q : io)
        if (!span_aligned(q, s)) return SELSCAN_E_ALIGN;
    if (!span_aligned(a.A, 4) || !span_aligned(a.D, 4) || !span_aligned(a.bias, 4) || !span_aligned(a.cu, 4) ||
        !span_aligned(a.slots, 4) || !span_aligned(a.h, 16) || (a.ws_need && !span_aligned(a.ws, 16)))
        return SELSCAN_E_ALIGN;
    if (a.ws_need && (!a.ws || a.ws_bytes < a.ws_need)) return SELSCAN_E_WORKSPACE;
    const size_t tok = (size_t)a.rows * a.dim * s, bc = strided_bytes(a.rows, kN, a.bc_stride, s);
    const Span in[] = {{a.x, tok},
                       {a.delta, tok},
                       {a.B, bc},
                       {a.C, bc},
                       {a.z, strided_bytes(a.rows, a.dim, a.z_stride, s)},
                       {a.A, (size_t)a.dim * kN * 4},
                       {a.D, (size_t)a.dim * 4},
                       {a.bias, (size_t)a.dim * 4},
                       {a.cu, (size_t)(a.nseq + 1) * 4},
                       {a.slots, (size_t)a.nseq * 4},
                       {a.carry, (size_t)a.nseq}};
    const Span out[] = {{a.y, tok}, {a.h, (size_t)a.nslots * a.dim * kN * 4}, {a.ws_need ? a.ws : nullptr, a.ws_need}};
    return any_alias(in, 11, out, 3) ? SELSCAN_E_ALIAS : SELSCAN_OK;
}

ScanParams scan_params(const ScanArgs &a) {
    ScanParams p{};
    p.x = a.x, p.delta = a.delta, p.z = a.z, p.B = a.B, p.C = a.C, p.A = a.A, p.D = a.D, p.bias = a.bias;
    p.y = a.y, p.h = a.h;
    p.q = {a.cu, a.slots, a.carry, a.nslots, (int)a.rows, (int)a.nseq};
    p.dim = a.dim, p.bc_stride = a.bc_stride, p.z_stride = a.z_stride;
    p.softplus = (a.flags & SELSCAN_FLAG_DELTA_SOFTPLUS) ? 1 : 0;
    return p;
}

constexpr int64_t kGridY = 65535;

template <typename T, bool ZOH, bool GATE>
int launch_scan(const ScanParams &p, int64_t blocks, void *stream) {
    int rc = enqueue(scan_packed<T, ZOH, GATE, 0>, dim3((unsigned)blocks), dim3(256), p, stream);
    if (rc == SELSCAN_OK && p.joined) {
        const int64_t y = p.q.nseq < p.entries ? p.q.nseq : p.entries;
        rc = enqueue(scan_join, dim3((unsigned)((p.dim * kN + 63) / 64), (unsigned)(y < kGridY ? y : kGridY)), dim3(64), p, stream);
    }
    if (rc == SELSCAN_OK && p.seg)
        rc = enqueue(scan_packed<T, ZOH, GATE, 1>, dim3((unsigned)((int64_t)p.entries * p.ntiles)), dim3(256), p, stream);
    return rc;
}

template <typename T>
int launch_scan_io(const ScanParams &p, int64_t blocks, bool zoh, void *stream) {
    if (zoh) return p.z ? launch_scan<T, true, true>(p, blocks, stream) : launch_scan<T, true, false>(p, blocks, stream);
    return p.z ? launch_scan<T, false, true>(p, blocks, stream) : launch_scan<T, false, false>(p, blocks, stream);
}

// rows that a thread of a step kernel takes one after another: one while the launch has fewer than
// four workgroups of 256 threads per compute unit, up to 8 (then A and the filters are read an eighth as often)
int step_rows(int64_t rows, int64_t threads_per_row) {
    const int64_t full = 256 * 4 * 256;
    int64_t n = rows * threads_per_row / full;
    return n < 1 ? 1 : n > 8 ? 8 : (int)n;
}

// States of this many bytes go without a place in the caches.  By the time a model's next token comes to a layer again the
// other layers' states have passed, 256 MB of them from 32 layers on.  Measured with states that are in no cache, with a
// place and without: 100 rows x 1,536 channels 8.2 and 7.3 us, 64 x 4,096 11.7 and 10.5, 256 x 4,096 32.7 and 29.6,
// 2,000 x 4,096 231 and 214; with one layer alone, from the caches, 64 x 4,096 8.9 and 10.0.  8 rows x 1,536 no difference.
constexpr int64_t kStatesPast = INT64_C(8) << 20;

}  // namespace

extern "C" {

int selscan_lm_abi_version(void) { return SELSCAN_LM_ABI_VERSION; }
const char *selscan_lm_last_hip_error(void) { return g_last_hip_error; }

int causal_conv1d_packed_fwd(const void *x, int64_t x_stride, const float *weight, const float *bias,
                             const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry, void *conv_state,
                             unsigned flags, void *out, int64_t tokens, int64_t nseq, int64_t nslots, int64_t dim,
                             int64_t width, int io_dtype, void *stream) {
    bool nothing;
    int rc = conv_check(x, x_stride, weight, bias, conv_state, true, flags, out, tokens, nseq, nslots, dim, width, io_dtype,
                        cu_seqlens, slots, carry, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    ConvParams p = conv_params(x, x_stride, weight, bias, cu_seqlens, slots, carry, conv_state, flags, out, tokens, nseq,
                               nslots, dim, io_dtype);
    // threads per workgroup: the channel groups of a row, at most 256, in whole waves
    const int64_t groups = (dim + 7) / 8;
    const unsigned block = groups >= 256 ? 256 : (unsigned)((groups + 63) / 64 * 64);
    // (4,097 tokens x 1,536 channels fp32, 771 waves of runs of 16: 15.7 us with them, 19.6 with runs of 4; 505 tokens in 8
    // sequences, 117 waves: 9.4 and 5.8)
    const int shift = segments(tokens, nseq, 1 << kConvLong) * ((groups + 63) / 64) >= kSimds / 2 ? kConvLong : kConvShort;
    const dim3 grid((unsigned)segments(tokens, nseq, 1 << shift), (unsigned)((groups + block - 1) / block));
    if (grid.y > kGridY || !grid_fits(segments(tokens, nseq, 1 << shift), block)) return SELSCAN_E_UNSUPPORTED;
    void (*k)(ConvParams) = nullptr;
#define PICK(T, S) (width == 1 ? conv_packed<T, 1, S> : width == 2 ? conv_packed<T, 2, S> : width == 3 ? conv_packed<T, 3, S> : conv_packed<T, 4, S>)
#define PICK_T(S) (io_dtype == SELSCAN_BF16 ? PICK(uint16_t, S) : PICK(float, S))
    k = shift == kConvLong ? PICK_T(kConvLong) : PICK_T(kConvShort);
#undef PICK_T
#undef PICK
    return enqueue(k, grid, dim3(block), p, stream);
}

int causal_conv1d_step(const void *x, int64_t x_stride, const float *weight, const float *bias, const int32_t *slots,
                       void *conv_state, unsigned flags, void *out, int64_t rows, int64_t nslots, int64_t dim,
                       int64_t width, int io_dtype, void *stream) {
    bool nothing;
    int rc = conv_check(x, x_stride, weight, bias, conv_state, false, flags, out, rows, rows, nslots, dim, width, io_dtype,
                        nullptr, slots, nullptr, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    ConvParams p = conv_params(x, x_stride, weight, bias, nullptr, slots, nullptr, conv_state, flags, out, rows, rows,
                               nslots, dim, io_dtype);
    p.rows_per = step_rows(rows, (dim + 7) / 8);
    while ((rows + p.rows_per - 1) / p.rows_per > kGridY) p.rows_per *= 2;
    const dim3 grid((unsigned)((dim + 511) / 512), (unsigned)((rows + p.rows_per - 1) / p.rows_per));
    void (*k)(ConvParams) = nullptr;
#define PICK(T) (width == 1 ? conv_step<T, 1> : width == 2 ? conv_step<T, 2> : width == 3 ? conv_step<T, 3> : conv_step<T, 4>)
    k = io_dtype == SELSCAN_BF16 ? PICK(uint16_t) : PICK(float);
#undef PICK
    return enqueue(k, grid, dim3(64), p, stream);
}

size_t selscan_packed_workspace_bytes(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t dim, int64_t dstate) {
    if (tokens <= 0 || nseq <= 0 || max_seqlen <= 0 || dim <= 0 || dstate != kN || tokens > kMaxTokens || nseq > INT32_MAX / 2 ||
        dim > INT32_MAX)
        return 0;
    return packed_workspace(tokens, max_seqlen, dim);
}

int selscan_packed_fwd(const void *x, const void *delta, const float *A, const void *B, const void *C,
                       int64_t bc_stride, const float *D, const void *z, int64_t z_stride, const float *delta_bias,
                       unsigned flags, const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry,
                       float *h_state, void *y, int64_t tokens, int64_t nseq, int64_t nslots, int64_t max_seqlen,
                       int64_t dim, int64_t dstate, int io_dtype, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (max_seqlen < 0) return SELSCAN_E_SHAPE;
    const size_t need = selscan_packed_workspace_bytes(tokens, nseq, max_seqlen, dim, dstate);
    const ScanArgs a{x,     delta, A,       B,    C,      bc_stride, D,        z,        z_stride, delta_bias, flags,
                     cu_seqlens, slots, carry, h_state, y, tokens, nseq, nslots, dim, dstate, io_dtype, workspace, need,
                     workspace_bytes, true};
    bool nothing;
    const int rc = scan_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    ScanParams p = scan_params(a);
    p.ntiles = (int)((dim + 63) / 64);
    int64_t pieces = nseq;
    if (!need) {
        const int round = p.ntiles < kUnits ? kUnits / p.ntiles : 1;
        p.round = nseq <= 64 && nseq > round ? round : 0;
    } else {
        p.size = split_size(tokens, max_seqlen, dim);
        p.dsize = make_div((uint32_t)p.size);
        pieces = segments(tokens, nseq, p.size);
        p.seg = (float *)workspace;
        p.entries = (int)(tokens / p.size);
        p.sdt = p.seg + (int64_t)p.entries * dim * kN;
        p.joined = max_seqlen / p.size > kWalk ? 1 : 0;
    }
    if (!grid_fits(pieces * p.ntiles, 256)) return SELSCAN_E_UNSUPPORTED;
    const bool zoh = (flags & SELSCAN_FLAG_ZOH) != 0;
    return io_dtype == SELSCAN_BF16 ? launch_scan_io<uint16_t>(p, pieces * p.ntiles, zoh, stream)
                                    : launch_scan_io<float>(p, pieces * p.ntiles, zoh, stream);
}

int selscan_step(const void *x, const void *delta, const float *A, const void *B, const void *C, int64_t bc_stride,
                 const float *D, const void *z, int64_t z_stride, const float *delta_bias, unsigned flags,
                 const int32_t *slots, float *h_state, void *y, int64_t rows, int64_t nslots, int64_t dim,
                 int64_t dstate, int io_dtype, void *stream) {
    const ScanArgs a{x,       delta, A,     B,       C, bc_stride, D,    z,      z_stride, delta_bias, flags,
                     nullptr, slots, nullptr, h_state, y, rows,      rows, nslots, dim,      dstate,     io_dtype, nullptr, 0, 0,
                     false};
    bool nothing;
    const int rc = scan_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    ScanParams p = scan_params(a);
    p.rows_per = step_rows(rows, dim * 4);
    while ((rows + p.rows_per - 1) / p.rows_per > kGridY) p.rows_per *= 2;
    const dim3 grid((unsigned)((dim * 4 + 255) / 256), (unsigned)((rows + p.rows_per - 1) / p.rows_per));
    if (!grid_fits(grid.x, 256)) return SELSCAN_E_UNSUPPORTED;
    const bool zoh = (flags & SELSCAN_FLAG_ZOH) != 0;
    const bool nt = rows * dim * kN * 4 >= kStatesPast;
#define PICK(T) (zoh ? nt ? scan_step<T, true, true> : scan_step<T, true, false> : nt ? scan_step<T, false, true> : scan_step<T, false, false>)
    return enqueue(io_dtype == SELSCAN_BF16 ? PICK(uint16_t) : PICK(float), grid, dim3(256), p, stream);
#undef PICK
}

}  // extern "C"
