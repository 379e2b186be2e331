// libselscan_lm - log probability of a token, entropy and top alternatives from logits, and the
// gradient of the first two (token_logprobs_fwd, token_logprobs_bwd of include/selscan_lm.h).
// MI355X (gfx950).
//
// With c = scale log2 e, m the largest logit of a row and a = c (x - m):
//     s = sum 2^a,  t = sum 2^a a,  logprob = scale (x[target] - m) - ln s,  entropy = ln 2 (log2 s - t / s).
// a is c x - fl(c m) in one fma where c m is below 2^24; else x - m comes before the product, so that a row of the
// type's lowest value, whose c x overflows, is a row of equal logits.
// A row is cut into slices that a workgroup holds in registers, so the logits are read once; the
// slices' (m, s, t) and their best alternatives are joined by a second, small kernel.  HBM bound: 2,048 x 50,280 bf16 with
// five alternatives 48 us (4.3 TB/s of reads; a plain reduction of a large array reaches 4.05) and 5 for the join.  Few rows
// are two launches and two trips to memory: 7 x 50,280 with eight alternatives 5.2 + 4.8 us.
#include "lm_common.h"

#include <float.h>

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = 32;
constexpr int kMaxVocab = 1 << 21;
constexpr int kCand = 512;  // candidates a slice ranks directly

struct LpParams {
    const void *x;
    const int64_t *targets;
    float *logprob, *entropy, *stats, *top_logprob;
    int64_t *top_index;
    float4 *part;               // [rows][nsl]: m, s, t
    unsigned long long *cand;   // [rows][nsl][top]: order of the logit above, complement of its index below; 0: none
    const float *in_stats, *in_entropy, *dlogprob, *dentropy;
    void *dx;
    int64_t rows, stride;
    int vocab, nsl, top;
    float c, scale;
};

// elements [at, at + 8) of a row of n; those past its end are -inf
template <bool NT, typename T>
__device__ __forceinline__ Raw8<T> load_logits(const T *row, int at, int n) {
    if (at + 8 <= n) return load_stream8<NT>(row + at);
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.w[e] = at + e < n ? __float_as_uint(row[at + e]) : 0xFF800000u;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = at + 2 * e < n ? row[at + 2 * e] : 0xFF80u, hi = at + 2 * e + 1 < n ? row[at + 2 * e + 1] : 0xFF80u;
            r.w[e] = lo | hi << 16;
        }
    }
    return r;
}

// floats in the order of their values as unsigned numbers (both zeros alike), and back
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ unsigned long long entry(float x, int index) {
    return (unsigned long long)order_of(x) << 32 | (uint32_t)~index;
}

// The k-th largest of the 64 lanes' values (k <= 64), bit by bit from the top; bf16 values differ in
// their upper 16 bits only.
template <typename T>
__device__ __forceinline__ float kth_of_wave(float v, int k) {
    const uint32_t o = sizeof(T) == 2 ? order_of(v) >> 16 : order_of(v);
    uint32_t best = 0;
#pragma unroll
    for (int b = sizeof(T) == 2 ? 15 : 31; b >= 0; --b) {
        const uint32_t cand = best | 1u << b;
        if (__popcll(__ballot(o >= cand)) >= k) best = cand;
    }
    // (of a negative number's bits below, all are set in the order)
    return value_of(sizeof(T) == 2 ? (best << 16) | (best & 0x8000u ? 0u : 0xFFFFu) : best);
}

// How a largest logit m is taken off: c x - fl(c m) in one fma, whose terms all carry the factor 2^(c m - fl(c m)), taken out
// again at the end; or, where c m is so large that its rounding would be more than half a step of the exponent (a factor
// that can itself overflow, and at the far end a c x that does), c (x - m).
constexpr float kPlainBase = 16777216.f;  // 2^24: fl(c m) is off by 1/2 at most
struct Base {
    float mc;
    bool plain;
    float rest;  // plain: c m - fl(c m)
};
__device__ __forceinline__ Base base_of(float m, float c) {
    const float mc = m * c;
    const bool plain = fabsf(mc) < kPlainBase;
    return {mc, plain, plain ? fmaf(m, c, -mc) : 0.f};
}

// what a row comes to: from its largest logit m and s, t as they were taken with base_of(m)
template <typename T, bool WRITE>
struct RowEnd {
    float m, scale, ls;  // ls: log of sum exp(scale (x - m))
    bool empty, nan;

    // (lead: one thread of those that call this writes)
    __device__ __forceinline__ RowEnd(const LpParams &p, int row, float m_, float s, float t, bool lead) : m(m_), scale(p.scale) {
        const float l = __builtin_amdgcn_logf(s);
        ls = (l - base_of(m, p.c).rest) * kLn2;
        empty = s == 0.f, nan = s != s;
        if (!WRITE || !lead) return;
        p.stats[2 * (int64_t)row] = m;
        p.stats[2 * (int64_t)row + 1] = ls;
        p.entropy[row] = empty ? 0.f : (l - t / s) * kLn2;
        const int64_t y = p.targets[row];
        float lp = 0.f;
        if (y >= 0 && y < p.vocab) lp = empty ? -INFINITY : logp(Io<T>::f32(((const T *)p.x)[row * p.stride + y]));
        p.logprob[row] = lp;
    }
    // exactly as far as x - m is; by the scale itself, since c (x - m) of a masked logit of the type's lowest value overflows
    __device__ __forceinline__ float logp(float x) const { return fmaf(x - m, scale, -ls); }
    __device__ __forceinline__ void put(const LpParams &p, int row, unsigned long long k, int rank) const {
        if (rank >= p.top) return;
        p.top_logprob[(int64_t)row * p.top + rank] = logp(value_of((uint32_t)(k >> 32)));
        p.top_index[(int64_t)row * p.top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
    }
    // places from `have` on: fewer logits with a probability than asked for, or (NaN) no order at all
    __device__ __forceinline__ void pad(const LpParams &p, int row, int have, int tid, int threads) const {
        for (int i = (nan ? 0 : have) + tid; i < p.top; i += threads) {
            p.top_logprob[(int64_t)row * p.top + i] = nan ? NAN : -INFINITY;
            p.top_index[(int64_t)row * p.top + i] = -1;
        }
    }
};

// One workgroup: PIECES x 256 x 8 logits of one row, in registers.  WHOLE: that is all of the row, and the
// workgroup finishes it; else a slice for logprobs_join.
//
// a = c x - fl(c m) takes one fma per logit instead of c (x - m)'s two operations; the rounding of c m is the same
// for all logits and so a factor of s and t, which the join takes out again (from the exact residue of c m).  base_of says
// where the subtraction has to come first.
//
// Alternatives: the `top`-th largest of a wave's 64 per-lane maxima is no larger than the slice's `top`-th
// largest logit, so every logit of the slice that can be among the best is at or above the largest of the
// waves' bounds.  Those few (some hundred for top = 32) are found by the maxima of pieces of 8, gathered in LDS
// and ranked by counting.  If equal values make them too many, the best are taken out one after another.
template <typename T, int PIECES, bool WHOLE, bool NT>
__global__ __launch_bounds__(kThreads) void logprobs_slice(LpParams p) {
    constexpr int NW = kThreads / 64;
    __shared__ float red[NW], red2[NW][2], bound[NW];
    __shared__ unsigned long long cand[kCand], pick[NW];
    __shared__ int ncand;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int row = WHOLE ? blockIdx.x : blockIdx.x / p.nsl, sl = WHOLE ? 0 : blockIdx.x - row * p.nsl;
    const int base = sl * (PIECES * kThreads * 8);
    const T *x = (const T *)p.x + row * p.stride;
    Raw8<T> r[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) r[i] = load_logits<NT>(x, base + (i * kThreads + tid) * 8, p.vocab);
    if (tid == 0) ncand = 0;
    float pm[PIECES], mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        pm[i] = raw_f32(r[i], 0);
#pragma unroll
        for (int e = 1; e < 8; ++e) pm[i] = fmaxf(pm[i], raw_f32(r[i], e));
        mine = fmaxf(mine, pm[i]);
    }
    float m = wave_max(mine);
    if (lane == 0) red[wave] = m;
    if (p.top) {
        const float b = kth_of_wave<T>(mine, p.top);
        if (lane == 0) bound[wave] = b;
    }
    lds_barrier();
    m = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) m = fmaxf(m, red[i]);
    const Base off = base_of(m, p.c);
    const float mc = off.mc;
    float s = 0.f, t = 0.f;
    if (off.plain) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = fmaf(raw_f32(r[i], e), p.c, -mc), w = __builtin_amdgcn_exp2f(a);
                s += w;
                t = fmaf(w, fmaxf(a, -200.f), t);  // 2^-200 is 0: no 0 * inf for a logit of -inf
            }
    } else {
        const float mm = m == -INFINITY ? 0.f : m;  // (nothing but -inf)
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = (raw_f32(r[i], e) - mm) * p.c, w = __builtin_amdgcn_exp2f(a);
                s += w;
                t = fmaf(w, fmaxf(a, -200.f), t);
            }
    }
    s = wave_sum(s), t = wave_sum(t);
    if (lane == 0) red2[wave][0] = s, red2[wave][1] = t;
    if (p.top) {
        float b = -FLT_MAX;  // a logit of -inf is no alternative
#pragma unroll
        for (int i = 0; i < NW; ++i) b = fmaxf(b, bound[i]);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (pm[i] >= b) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = raw_f32(r[i], e);
                    if (v >= b) {
                        const int at = atomicAdd(&ncand, 1);
                        if (at < kCand) cand[at] = entry(v, base + (i * kThreads + tid) * 8 + e);
                    }
                }
            }
        }
    }
    lds_barrier();
    s = red2[0][0], t = red2[0][1];
#pragma unroll
    for (int i = 1; i < NW; ++i) s += red2[i][0], t += red2[i][1];
    unsigned long long *out = p.cand + (int64_t)blockIdx.x * p.top;  // (a slice's)
    if constexpr (!WHOLE) {
        if (tid == 0) p.part[blockIdx.x] = make_float4(m, s, t, 0.f);
    }
    const RowEnd<T, WHOLE> end(p, row, m, s, t, tid == 0);
    if (!p.top) return;
    if (WHOLE && end.nan) {
        end.pad(p, row, 0, tid, kThreads);
        return;
    }
    auto put = [&](unsigned long long k, int rank) {
        if constexpr (WHOLE) end.put(p, row, k, rank);
        else if (rank < p.top) out[rank] = k;
    };
    const int n = ncand;
    if (n <= kCand) {
        for (int i = tid; i < n; i += kThreads) {
            const unsigned long long k = cand[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += cand[j] > k ? 1 : 0;
            put(k, rank);
        }
        if constexpr (WHOLE) {
            end.pad(p, row, n, tid, kThreads);
        } else {
            for (int i = n + tid; i < p.top; i += kThreads) out[i] = 0;
        }
        return;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < p.top; ++k) {
        unsigned long long best = 0;
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
            // (from memory again: this rare loop then costs the kernel no registers)
            const Raw8<T> q8 = load_logits<NT>(x, base + (i * kThreads + tid) * 8, p.vocab);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = raw_f32(q8, e);
                const unsigned long long q = entry(v, base + (i * kThreads + tid) * 8 + e);
                if (v > -INFINITY && q < last && q > best) best = q;
            }
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const unsigned long long q = __shfl_xor(best, o);
            best = q > best ? q : best;
        }
        if (lane == 0) pick[wave] = best;
        lds_barrier();
        best = pick[0];
        for (int i = 1; i < NW; ++i) best = pick[i] > best ? pick[i] : best;
        if (tid == 0) put(best, k);  // (more than kCand candidates: every round finds one)
        last = best;
        lds_barrier();  // every wave has read the picks before the next round writes them
    }
}

// One workgroup per row: joins the slices.  Alternatives: with `low` the worst over the slices of their place-th entries,
// place = ceil(top / slices), at least top entries are at or above it, so only those can be among the
// best.  They are gathered in LDS and ranked by counting.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_join(LpParams p) {
    __shared__ unsigned long long list[kCand], lows[4];
    __shared__ int count;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const float4 *part = p.part + (int64_t)row * p.nsl;
    const unsigned long long *cand = p.cand + (int64_t)row * p.nsl * p.top;
    const int n = p.nsl * p.top;
    const unsigned long long first = p.top && tid < n ? cand[tid] : 0;  // (all of them, mostly)
    unsigned long long low = ~0ull;
    if (p.top) {
        const int place = (p.top + p.nsl - 1) / p.nsl - 1;
        for (int i = tid; i < p.nsl; i += blockDim.x) {
            const unsigned long long k = cand[i * p.top + place];
            low = k < low ? k : low;
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const unsigned long long k = __shfl_xor(low, o);
            low = k < low ? k : low;
        }
        if (lane == 0) lows[tid >> 6] = low;
        if (tid == 0) count = 0;
    }
    float M = -INFINITY;
    for (int i = lane; i < p.nsl; i += 64) M = fmaxf(M, part[i].x);
    M = wave_max(M);
    const Base B = base_of(M, p.c);
    float s = 0.f, t = 0.f;
    for (int i = lane; i < p.nsl; i += 64) {
        const float4 q = part[i];
        // a slice of nothing but -inf has s = t = 0, or NaN where it holds one: taken as it is
        const bool none = q.x == -INFINITY;
        // how far the slice's base lies below the row's, as both were taken off
        const float d = none ? 0.f : fmaf(q.x - M, p.c, B.rest - base_of(q.x, p.c).rest);
        const float f = none ? 1.f : __builtin_amdgcn_exp2f(d);
        s = fmaf(q.y, f, s);
        t = fmaf(f, fmaf(q.y, fmaxf(d, -200.f), q.z), t);
    }
    s = wave_sum(s), t = wave_sum(t);
    const RowEnd<T, true> end(p, row, M, s, t, tid == 0);
    if (!p.top) return;
    if (end.nan) {
        end.pad(p, row, 0, tid, blockDim.x);
        return;
    }
    __syncthreads();
    low = lows[0];
    for (int i = 1; i < (int)(blockDim.x >> 6); ++i) low = lows[i] < low ? lows[i] : low;
    low = low == 0 ? 1 : low;  // a slice with fewer: every entry there is
    for (int i = tid; i < n; i += blockDim.x) {
        const unsigned long long k = i < (int)blockDim.x ? first : cand[i];
        if (k >= low) {
            const int at = atomicAdd(&count, 1);
            if (at < kCand) list[at] = k;
        }
    }
    __syncthreads();
    const int have = count;
    if (have <= kCand) {
        for (int i = tid; i < have; i += blockDim.x) {
            const unsigned long long k = list[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += list[j] > k ? 1 : 0;
            end.put(p, row, k, rank);
        }
    } else {
        // the best sit together in a few of very many slices
        for (int i = tid; i < n; i += blockDim.x) {
            const unsigned long long k = cand[i];
            int rank = k >= low ? 0 : p.top;
            for (int j = 0; j < n && rank < p.top; ++j) rank += cand[j] > k ? 1 : 0;
            end.put(p, row, k, rank);
        }
    }
    end.pad(p, row, have, tid, blockDim.x);
}

constexpr int kBwdPieces = 4;

// gradient: reads a logit, writes its gradient; HBM bound (1,000 x 32,001 fp32: 43 us, 5.9 TB/s of what it reads and writes,
// where a copy of 1 GiB reaches 5.2)
template <typename T, bool NT>
__global__ __launch_bounds__(kThreads) void logprobs_bwd(LpParams p) {
    const int row = blockIdx.x / p.nsl, sl = blockIdx.x - row * p.nsl;
    const int base = sl * (kBwdPieces * kThreads * 8);
    const T *x = (const T *)p.x + row * p.stride;
    T *dx = (T *)p.dx + (int64_t)row * p.vocab;
    const int64_t y = p.targets[row];
    const bool valid = y >= 0 && y < p.vocab;
    const float gl = p.dlogprob && valid ? p.dlogprob[row] * p.scale : 0.f;
    const float gh = p.dentropy ? p.dentropy[row] * p.scale : 0.f;
    const float m = p.in_stats[2 * (int64_t)row], ls = p.in_stats[2 * (int64_t)row + 1] * kLog2e;
    const bool empty = m == -INFINITY && !(ls != ls);
    // -gl p - gh p (ln 2 a + H) = p (k0 + k1 a), a = log2 p
    const float k0 = -fmaf(gh, p.in_entropy[row], gl), k1 = -gh * kLn2;
    Raw8<T> r[kBwdPieces];
#pragma unroll
    for (int i = 0; i < kBwdPieces; ++i) r[i] = load_logits<NT>(x, base + (i * kThreads + (int)threadIdx.x) * 8, p.vocab);
#pragma unroll
    for (int i = 0; i < kBwdPieces; ++i) {
        const int at = base + (i * kThreads + (int)threadIdx.x) * 8;
        if (at >= p.vocab) break;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fmaf(raw_f32(r[i], e) - m, p.c, -ls);
            v[e] = empty ? 0.f : __builtin_amdgcn_exp2f(a) * fmaf(k1, fmaxf(a, -200.f), k0);
        }
        const int64_t hot = y - at;
        if (valid && !empty && hot >= 0 && hot < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += e == hot ? gl : 0.f;
        }
        if (at + 8 <= p.vocab) {
            store_any8(dx + at, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e < p.vocab) dx[at + e] = Io<T>::to(v[e]);
        }
    }
}

// (A vocabulary well under 8,192 costs as much as that: 100,000 rows of 256 bf16 logits 198 us, of 1,024 195 us, 1.05 TB/s, against
// 20,000 of 8,192 in 50 us, 6.5 TB/s.)
//
// 8-logit pieces per thread of a slice: 4 (8,192 logits; 8 pieces measured 52 us where 4 take 49, 2,048 x 50,280 bf16), or 2
// where slices that long would leave the chip's compute units without four workgroups each
int pieces_for(int64_t rows, int64_t vocab) {
    const int64_t big = 4 * kThreads * 8;
    return rows * ((vocab + big - 1) / big) >= 1024 || vocab > kMaxVocab / 2 ? 4 : 2;
}
// rows of a slice's length need no join.  (Longer ones by a workgroup of 16 waves measured slower than slices and a join: 7 x
// 50,280 bf16 with eight alternatives 11.0 us against 9.3.)
bool whole_row(int64_t vocab) { return vocab <= 4 * kThreads * 8; }
int64_t slices_for(int64_t rows, int64_t vocab) {
    const int64_t n = (int64_t)pieces_for(rows, vocab) * kThreads * 8;
    return (vocab + n - 1) / n;
}

// Logits of this many bytes are read without a place in the caches: forward, those that a gradient right after it would find
// there are no more than what they push out (forward and gradient, us, with a place and without: 600 x 50,280 bf16, 60 MB, 37
// and 38; 1,000, 101 MB, 57 and 59; 1,400, 141 MB, 88 and 76; 4,096 x 32,001, 262 MB, 168 and 160; 1,400 x 32,001 fp32, 179 MB,
// 111 and 105); gradient, what the forward left is gone by then (2,048 x 50,280, 206 MB, 113 and 102; 4,096 x 32,001 160 and
// 142; 1,400 x 32,001 fp32 no difference; 128 MB 72 and 78).
constexpr int64_t kForwardPast = INT64_C(112) << 20, kBackwardPast = INT64_C(160) << 20;

int lp_check(const void *logits, int64_t stride, const int64_t *targets, float scale, int64_t rows, int64_t vocab, int dtype) {
    if (rows < 0 || vocab < 0) return SELSCAN_E_SHAPE;
    if (!io_known(dtype) || !(scale > 0.f) || !(scale * kLog2e < INFINITY) || vocab > kMaxVocab) return SELSCAN_E_UNSUPPORTED;
    if (rows == 0 || vocab == 0) return SELSCAN_OK;
    if (stride < vocab || mul_size(rows, stride) < 0) return SELSCAN_E_SHAPE;
    if (!logits || !targets) return SELSCAN_E_NULL;
    if (!span_aligned(logits, io_bytes(dtype)) || !span_aligned(targets, 8)) return SELSCAN_E_ALIGN;
    return SELSCAN_OK;
}

}  // namespace

extern "C" {

size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top) {
    if (rows <= 0 || vocab <= 0 || vocab > kMaxVocab || top < 0 || top > kMaxTop) return 0;
    if (whole_row(vocab)) return 0;
    const size_t n = (size_t)rows * (size_t)slices_for(rows, vocab);
    return n * (sizeof(float4) + (size_t)top * 8);
}

int token_logprobs_fwd(const void *logits, int64_t logits_stride, const int64_t *targets, float scale, int top,
                       float *logprob, float *entropy, float *stats, float *top_logprob, int64_t *top_index, int64_t rows,
                       int64_t vocab, int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = lp_check(logits, logits_stride, targets, scale, rows, vocab, io_dtype);
    if (rc != SELSCAN_OK) return rc;
    if (top < 0 || top > kMaxTop) return SELSCAN_E_UNSUPPORTED;
    if (rows == 0) return SELSCAN_OK;
    if (vocab == 0 || top > vocab) return SELSCAN_E_SHAPE;
    const size_t need = token_logprobs_workspace_bytes(rows, vocab, top);
    if (!logprob || !entropy || !stats || (top && (!top_logprob || !top_index))) return SELSCAN_E_NULL;
    if (!span_aligned(logprob, 4) || !span_aligned(entropy, 4) || !span_aligned(stats, 4) ||
        (top && (!span_aligned(top_logprob, 4) || !span_aligned(top_index, 8))) || (need && !span_aligned(workspace, 16)))
        return SELSCAN_E_ALIGN;
    if (need && (!workspace || workspace_bytes < need)) return SELSCAN_E_WORKSPACE;
    const Span in[] = {{logits, strided_bytes(rows, vocab, logits_stride, io_bytes(io_dtype))}, {targets, (size_t)rows * 8}};
    const Span out[] = {{logprob, (size_t)rows * 4},
                        {entropy, (size_t)rows * 4},
                        {stats, (size_t)rows * 8},
                        {top ? top_logprob : nullptr, (size_t)rows * top * 4},
                        {top ? top_index : nullptr, (size_t)rows * top * 8},
                        {need ? workspace : nullptr, need}};
    if (any_alias(in, 2, out, 6)) return SELSCAN_E_ALIAS;
    LpParams p{};
    p.x = logits, p.targets = targets, p.logprob = logprob, p.entropy = entropy, p.stats = stats;
    p.top_logprob = top_logprob, p.top_index = top_index;
    p.rows = rows, p.stride = logits_stride, p.vocab = (int)vocab, p.top = top;
    p.scale = scale, p.c = scale * kLog2e;
    const bool bf = io_dtype == SELSCAN_BF16, nt = rows * vocab * (int64_t)io_bytes(io_dtype) >= kForwardPast;
#define PICK(PIECES, WHOLE)                                                                                       \
    (bf ? nt ? logprobs_slice<uint16_t, PIECES, WHOLE, true> : logprobs_slice<uint16_t, PIECES, WHOLE, false>     \
        : nt ? logprobs_slice<float, PIECES, WHOLE, true> : logprobs_slice<float, PIECES, WHOLE, false>)
    if (whole_row(vocab)) {
        if (!grid_fits(rows, kThreads)) return SELSCAN_E_UNSUPPORTED;
        return enqueue(PICK(4, true), dim3((unsigned)rows), dim3(kThreads), p, stream);
    }
    const int pieces = pieces_for(rows, vocab);
    p.nsl = (int)slices_for(rows, vocab);
    const int64_t blocks = rows * p.nsl;
    if (!grid_fits(blocks, kThreads)) return SELSCAN_E_UNSUPPORTED;
    p.part = (float4 *)workspace;
    p.cand = (unsigned long long *)(p.part + blocks);
    // (slices of 2 pieces are of a few rows)
    rc = enqueue(pieces == 4 ? PICK(4, false) : bf ? logprobs_slice<uint16_t, 2, false, false> : logprobs_slice<float, 2, false, false>,
                 dim3((unsigned)blocks), dim3(kThreads), p, stream);
#undef PICK
    if (rc != SELSCAN_OK) return rc;
    return enqueue(bf ? logprobs_join<uint16_t> : logprobs_join<float>, dim3((unsigned)rows),
                   dim3(top && p.nsl * top > 64 ? kThreads : 64), p, stream);
}

int token_logprobs_bwd(const void *logits, int64_t logits_stride, const int64_t *targets, const float *stats,
                       const float *entropy, const float *dlogprob, const float *dentropy, float scale, void *dlogits,
                       int64_t rows, int64_t vocab, int io_dtype, void *stream) {
    const int rc = lp_check(logits, logits_stride, targets, scale, rows, vocab, io_dtype);
    if (rc != SELSCAN_OK) return rc;
    if (rows == 0 || vocab == 0) return SELSCAN_OK;
    if (!stats || !entropy || (!dlogprob && !dentropy) || !dlogits) return SELSCAN_E_NULL;
    const size_t s = io_bytes(io_dtype);
    if (!span_aligned(stats, 4) || !span_aligned(entropy, 4) || !span_aligned(dlogprob, 4) || !span_aligned(dentropy, 4) ||
        !span_aligned(dlogits, s))
        return SELSCAN_E_ALIGN;
    const Span in[] = {{logits, strided_bytes(rows, vocab, logits_stride, s)},
                       {targets, (size_t)rows * 8},
                       {stats, (size_t)rows * 8},
                       {entropy, (size_t)rows * 4},
                       {dlogprob, (size_t)rows * 4},
                       {dentropy, (size_t)rows * 4}};
    const Span out[] = {{dlogits, (size_t)rows * vocab * s}};
    if (any_alias(in, 6, out, 1)) return SELSCAN_E_ALIAS;
    LpParams p{};
    p.x = logits, p.targets = targets, p.in_stats = stats, p.in_entropy = entropy, p.dlogprob = dlogprob, p.dentropy = dentropy;
    p.dx = dlogits, p.rows = rows, p.stride = logits_stride, p.vocab = (int)vocab;
    p.scale = scale, p.c = scale * kLog2e;
    const int64_t per = kBwdPieces * kThreads * 8;
    p.nsl = (int)((vocab + per - 1) / per);
    const int64_t blocks = rows * p.nsl;
    if (!grid_fits(blocks, kThreads)) return SELSCAN_E_UNSUPPORTED;
    const bool nt = rows * vocab * (int64_t)s >= kBackwardPast;
    return enqueue(io_dtype == SELSCAN_BF16 ? nt ? logprobs_bwd<uint16_t, true> : logprobs_bwd<uint16_t, false>
                                            : nt ? logprobs_bwd<float, true> : logprobs_bwd<float, false>,
                   dim3((unsigned)blocks), dim3(kThreads), p, stream);
}

}  // extern "C"
