// libselscan_lm - the next token drawn from logits (token_sample of include/selscan_lm.h).  MI355X (gfx950).
//
// With T the temperature and m a row's largest logit, token i has weight 2^t, t = (x_i - m) log2(e) / T, as a whole multiple of
// 2^-shift.  Whole numbers add up to the same sum in any order, so that which tokens stay and which one is drawn does not depend
// on how a row is split; they are 64 bits wide, and t and its power are formed in 64 bits, since both turn on sums of up to
// 2^21 weights next to a border.
//
// Tokens are ranked by their logit and then by their index, as one number of 64 bits (entry_of); top-k, top-p and min-p
// leave those from a bound on.  A workgroup has a row and finds a bound without sorting: it adds up counts or weights in
// bins that follow the order, takes the bin in which the sum passes what is wanted, and looks into that bin alone, with bins as
// much finer, until it holds few enough tokens to rank each among them.
#include "lm_common.h"

#include <float.h>

namespace {

constexpr int kMaxVocab = 1 << 21;
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kRound = kThreads * 8;  // logits of a round: 8 adjacent ones of each thread
constexpr int kMaxSums = kMaxVocab / kRound * kWaves;
constexpr int kBins = 2048, kList = 256, kSteps = 256;
typedef unsigned long long u64;

struct SampleParams {
    const void *x;
    const float *uniform, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logprob;
    int32_t *kept;
    int64_t stride;
    int vocab, rounds, shift, top_k_all;
    float temperature_all, top_p_all, min_p_all;
};

// elements [at, at + 8) of a row of n; those past its end are -inf
template <typename T>
__device__ __forceinline__ Raw8<T> load_logits(const T *row, int at, int n) {
    if (at + 8 <= n) return load_any8(row + at);
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
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ u64 entry_of(float x, int index) { return (u64)order_of(x) << 32 | (uint32_t)~index; }

// Over the 64 lanes, with DPP: the sums up to each lane (the last lane's is the whole), and the largest.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp_u64(u64 v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
    return (u64)hi << 32 | lo;
}
template <class F>
__device__ __forceinline__ u64 wave_scan(u64 v, F f) {
    v = f(v, dpp_u64<0x111, 0xF>(v));
    v = f(v, dpp_u64<0x112, 0xF>(v));
    v = f(v, dpp_u64<0x114, 0xF>(v));
    v = f(v, dpp_u64<0x118, 0xF>(v));
    v = f(v, dpp_u64<0x142, 0xA>(v));
    return f(v, dpp_u64<0x143, 0xC>(v));
}
__device__ __forceinline__ u64 lane_of(u64 v, int lane) {
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
struct Add {
    __device__ u64 operator()(u64 a, u64 b) const { return a + b; }
};
struct Larger {
    __device__ u64 operator()(u64 a, u64 b) const { return a > b ? a : b; }
};

struct SampleLds {
    u64 bins[kMaxSums > kBins ? kMaxSums : kBins];  // (of the draw: sums of each round and wave)
    u64 entries[kList], weights[kList];
    double step[kSteps];  // 2^(i / 256)
    u64 part[2][kWaves];
    u64 found[2];
    int count;
};

// over the workgroup; buf: 0 or 1, not that of the reduction just before
template <class F>
__device__ __forceinline__ u64 block_reduce(SampleLds &m, u64 v, int buf, F f) {
    v = lane_of(wave_scan(v, f), 63);
    if ((threadIdx.x & 63) == 0) m.part[buf][threadIdx.x >> 6] = v;
    lds_barrier();
    u64 a = m.part[buf][threadIdx.x & (kWaves - 1)];
    a = f(a, dpp_u64<0x111, 0xF>(a));
    a = f(a, dpp_u64<0x112, 0xF>(a));
    a = f(a, dpp_u64<0x114, 0xF>(a));
    a = f(a, dpp_u64<0x118, 0xF>(a));
    return lane_of(a, 15);
}

// 2^t as a multiple of 2^-shift, t = (x - m) c / 256 <= 0: 2^(i / 256) from a table and the Taylor sum of 2^(r / 256), |r| <=
// 1/2, whose rest is below 2^-54.
__device__ __forceinline__ u64 weight_of(const SampleLds &m, float x, double top, double c256, int shift) {
    constexpr double magic = 6755399441055744., l = 0.693147180559945309417232121458 / 256.;
    double y = ((double)x - top) * c256;
    y = y > -80. * 256. ? y : -80. * 256.;
    const double z = y + magic, r = y - (z - magic);
    const int k = (int)(uint32_t)__double_as_longlong(z);
    double e = l * l * l * l / 24.;
    e = fma(e, r, l * l * l / 6.);
    e = fma(e, r, l * l / 2.);
    e = fma(e, r, l);
    e = fma(e, r, 1.);
    e = ldexp(e * m.step[k & (kSteps - 1)], (k >> 8) + shift) + 4503599627370496.;  // 2^52: the sum is a whole number
    return (u64)__double_as_longlong(e) & ((1ull << 52) - 1);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_row(SampleParams p) {
    __shared__ __attribute__((aligned(16))) SampleLds m;
    const int64_t row = blockIdx.x;
    const T *x = (const T *)p.x + row * p.stride;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const auto each = [&](auto f) {  // f(first index, 8 logits); the next round's are in flight
        Raw8<T> next = load_logits(x, tid * 8, p.vocab);
        for (int v = 0; v < p.rounds; ++v) {
            const Raw8<T> r = next;
            const int i = v * kRound + tid * 8;
            next = load_logits(x, i + kRound, p.vocab);
            f(i, r);
        }
    };
    if (tid < kSteps) m.step[tid] = exp2(tid * (1. / kSteps));
    if (tid == 0) m.count = 0;

    // the largest logit; whether a NaN or an infinity is among them; how many have a weight at all
    float best = -INFINITY;
    uint32_t live = 0;
    bool bad = false;
    each([&](int, const Raw8<T> &r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = raw_f32(r, e);
            bad |= !(v < INFINITY);
            live += v > -INFINITY;
            best = fmaxf(best, v);
        }
    });
    const float mine = best;
    // (order in the upper half of one, count and the mark in the other)
    const float top = value_of((uint32_t)block_reduce(m, order_of(bad ? -INFINITY : best), 0, Larger()));
    const u64 seen = block_reduce(m, (u64)(bad ? 1 : 0) << 32 | live, 1, Add());
    const uint32_t all = (uint32_t)seen;
    if (seen >> 32 || !all) {
        if (tid == 0) p.token[row] = -1, p.logprob[row] = seen >> 32 ? NAN : -INFINITY, p.kept[row] = 0;
        return;
    }
    const float temperature = p.temperature ? p.temperature[row] : p.temperature_all;
    const int k = p.top_k ? p.top_k[row] : p.top_k_all;
    const float top_p = p.top_p ? p.top_p[row] : p.top_p_all, min_p = p.min_p ? p.min_p[row] : p.min_p_all;
    if (!(temperature > 0.f) || k == 1 || top_p <= 0.f) {
        uint32_t at = 0;  // the complement of the first index
        each([&](int i, const Raw8<T> &r) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (raw_f32(r, e) == top && (uint32_t)~(i + e) > at) at = (uint32_t)~(i + e);
        });
        const u64 first = block_reduce(m, at, 0, Larger());
        if (tid == 0) p.token[row] = (int64_t)(uint32_t)~(uint32_t)first, p.logprob[row] = 0.f, p.kept[row] = 1;
        return;
    }
    const double m64 = top, c = 1.44269504088896340735992468100 / (double)temperature, c256 = c * 256.;
    const auto weight = [&](float v) { return weight_of(m, v, m64, c256, p.shift); };

    // tokens stay from this one on
    float bv = -FLT_MAX;
    int bi = INT32_MAX;
    const auto stays = [&](float v, int i) { return v > bv || (v == bv && i <= bi); };

    // The token, of those that stay, at which the sum of `what` (from the largest on) reaches `want`, 1 <= want <= the whole: the
    // bound becomes that token.  edge: tokens below it cannot be it; per: bins per unit of a logit.  WANT gives `want` from the
    // whole (the sums of the first bins).
    const auto select = [&](auto what, auto want_of, float edge, float per) {
        u64 want = 0, base = 0, hi = 0, lo = 0;
        int sh = -1;  // bins of the logit; else of entry numbers, 2^sh of them from hi down to lo
        for (;;) {
            const auto bin_of = [&](float v, int i) {
                if (sh < 0) {
                    const float d = (top - v) * per;
                    return (int)(d < (float)(kBins - 1) ? d : (float)(kBins - 1));
                }
                return (int)((hi - entry_of(v, i)) >> sh);
            };
            const auto inside = [&](float v, int i) {
                if (!(v >= edge) || !stays(v, i)) return false;
                if (sh < 0) return true;
                const u64 e = entry_of(v, i);
                return e <= hi && e >= lo;
            };
            lds_barrier();
            for (int b = tid; b < kBins; b += kThreads) m.bins[b] = 0;
            if (tid == 0) m.count = 0;
            lds_barrier();
            each([&](int i, const Raw8<T> &r) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = raw_f32(r, e);
                    if (inside(v, i + e)) atomicAdd(&m.bins[bin_of(v, i + e)], what(v));
                }
            });
            lds_barrier();
            // two bins of each thread; the sum up to them
            const u64 b0 = m.bins[2 * tid], b1 = m.bins[2 * tid + 1];
            const u64 up = wave_scan(b0 + b1, Add());
            if (lane == 63) m.part[0][wave] = up;
            lds_barrier();
            u64 before = 0, whole = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const u64 s = m.part[0][w];
                before += w < wave ? s : 0;
                whole += s;
            }
            if (sh < 0) want = want_of(whole);
            const u64 s0 = base + before + up - b0 - b1, s1 = s0 + b0, s2 = s1 + b1;
            if (s0 < want && s1 >= want) m.found[0] = 2 * tid, m.found[1] = s0;
            else if (s1 < want && s2 >= want) m.found[0] = 2 * tid + 1, m.found[1] = s1;
            lds_barrier();
            const int bin = (int)m.found[0];
            base = m.found[1];
            // that bin's tokens
            u64 most = 0, least = 0;  // (least: the largest complement)
            each([&](int i, const Raw8<T> &r) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = raw_f32(r, e);
                    if (inside(v, i + e) && bin_of(v, i + e) == bin) {
                        const u64 en = entry_of(v, i + e);
                        most = most > en ? most : en;
                        least = least > ~en ? least : ~en;
                        const int at = atomicAdd(&m.count, 1);
                        if (at < kList) m.entries[at] = en, m.weights[at] = what(v);
                    }
                }
            });
            lds_barrier();
            const int count = m.count;
            if (count <= kList) {
                if (tid < count) {
                    const u64 en = m.entries[tid];
                    u64 above = base;
                    for (int j = 0; j < count; ++j) above += m.entries[j] > en ? m.weights[j] : 0;
                    if (above < want && above + m.weights[tid] >= want) m.found[0] = en;
                }
                lds_barrier();
                bv = value_of((uint32_t)(m.found[0] >> 32));
                bi = (int)~(uint32_t)m.found[0];
                return;
            }
            hi = block_reduce(m, most, 0, Larger());
            lo = ~block_reduce(m, least, 1, Larger());
            sh = 64 - __builtin_clzll((hi - lo) | 1) - 11;
            sh = sh < 0 ? 0 : sh;
        }
    };

    if (k > 0 && (uint32_t)k < all) {
        float edge = -FLT_MAX, per = 0.f;
        // the k-th largest of the threads' largest is no larger than the k-th of all; where it lies is found among those
        const float far = value_of(~(uint32_t)block_reduce(m, (uint32_t)~order_of(mine < -FLT_MAX ? -FLT_MAX : mine), 0, Larger()));
        per = (float)kBins / (top - far);
        per = per < FLT_MAX ? per : FLT_MAX;
        if (k <= kThreads / 2) {
            lds_barrier();
            for (int b = tid; b < kBins; b += kThreads) m.bins[b] = 0;
            if (tid == 0) m.found[0] = 0;
            lds_barrier();
            const float d = (top - mine) * per;
            const int bin = d < (float)(kBins - 1) ? (int)d : kBins - 1;
            atomicAdd(&m.bins[bin], (u64)1);
            lds_barrier();
            const u64 b0 = m.bins[2 * tid], b1 = m.bins[2 * tid + 1];
            const u64 up = wave_scan(b0 + b1, Add());
            if (lane == 63) m.part[1][wave] = up;
            lds_barrier();
            u64 before = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) before += w < wave ? m.part[1][w] : 0;
            const u64 s0 = before + up - b0 - b1;
            if (s0 < (u64)k && s0 + b0 >= (u64)k) m.found[0] = 2 * tid;
            else if (s0 + b0 < (u64)k && s0 + b0 + b1 >= (u64)k) m.found[0] = 2 * tid + 1;
            lds_barrier();
            // the smallest of the threads' largest that lie in this bin or before it
            const uint32_t low = bin <= (int)m.found[0] ? ~order_of(mine) : 0;
            edge = value_of(~(uint32_t)block_reduce(m, low, 0, Larger()));
        }
        select([&](float) { return (u64)1; }, [&](u64) { return (u64)k; }, edge, per);
    }
    if (top_p < 1.f) {
        const float per = (float)((double)kBins * c / (p.shift + 2));
        select(weight, [&](u64 whole) {
            const u64 want = (u64)ceil((double)top_p * (double)whole);
            return want < 1 ? 1 : want < whole ? want : whole;
        }, -FLT_MAX, per < FLT_MAX ? per : FLT_MAX);
    }
    if (min_p > 0.f) {
        // the smallest logit of weight min_p and more
        const double low = log2((double)(min_p < 1.f ? min_p : 1.f)), v0 = m64 + low / c;
        float v = v0 > -FLT_MAX ? (float)v0 : -FLT_MAX;
        v = v < top ? v : top;
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = order_of(v);
            if (!(((double)v - m64) * c >= low)) v = value_of(o + 1);
            else if (v > -FLT_MAX && ((double)value_of(o - 1) - m64) * c >= low) v = value_of(o - 1);
        }
        if (v > bv) bv = v, bi = INT32_MAX;
    }

    // The draw: weights of each wave's part of each round, in the order of the indices
    u64 *sums = m.bins;  // [rounds][kWaves]
    uint32_t kept = 0;
    lds_barrier();
    {
        int at = wave;
        each([&](int i, const Raw8<T> &r) {
            u64 s = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = raw_f32(r, e);
                if (stays(v, i + e)) s += weight(v), ++kept;
            }
            s = __any(s != 0) ? lane_of(wave_scan(s, Add()), 63) : 0;
            if (lane == 0) m.bins[at] = s;
            at += kWaves;
        });
    }
    const uint32_t stay = (uint32_t)block_reduce(m, kept, 0, Add());  // (its barrier is the sums' too)
    if (wave != 0) return;
    // the first wave: a share of the sums in each lane, in order
    const int n = p.rounds * kWaves, each_n = (n + 63) / 64;
    u64 s = 0;
    for (int i = lane * each_n; i < n && i < (lane + 1) * each_n; ++i) s += sums[i];
    const u64 up = wave_scan(s, Add()), total = lane_of(up, 63);
    const float u = p.uniform[row];
    u64 at = u > 0.f ? (u64)((double)(u < 1.f ? u : 1.f) * (double)total) : 0;
    at = at < total ? at : total - 1;
    const int l1 = __builtin_ctzll(__ballot(up > at));
    u64 base = lane_of(up - s, l1);
    int part = l1 * each_n;
    while (base + sums[part] <= at) base += sums[part++];
    // the 64 lanes of that wave and round
    const int i0 = (part / kWaves) * kRound + (part % kWaves) * 512 + lane * 8;
    const Raw8<T> r = load_logits(x, i0, p.vocab);
    u64 w[8], sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = raw_f32(r, e);
        w[e] = stays(v, i0 + e) ? weight(v) : 0;
        sum += w[e];
    }
    const u64 up2 = base + wave_scan(sum, Add());
    if (lane != (int)__builtin_ctzll(__ballot(up2 > at))) return;
    u64 run = up2 - sum;
    int e = 0;
    float v = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        u64 upto = run;
#pragma unroll
        for (int i = 0; i <= j; ++i) upto += w[i];
        if (upto > at) e = j, v = raw_f32(r, j);
    }
    p.token[row] = i0 + e;
    p.logprob[row] = (float)((((double)v - m64) * c + p.shift - log2((double)total)) * 0.693147180559945309417232121458);
    p.kept[row] = (int32_t)stay;
}

}  // namespace

extern "C" int token_sample(const void *logits, int64_t logits_stride, const float *uniform, const float *temperature,
                            float temperature_all, const int32_t *top_k, int top_k_all, const float *top_p, float top_p_all,
                            const float *min_p, float min_p_all, int64_t *token, float *logprob, int32_t *kept, int64_t rows,
                            int64_t vocab, int io_dtype, void *stream) {
    if (rows < 0 || vocab < 0) return SELSCAN_E_SHAPE;
    if (!io_known(io_dtype) || vocab > kMaxVocab) return SELSCAN_E_UNSUPPORTED;
    if (!temperature && !(temperature_all >= 0.f && temperature_all < INFINITY)) return SELSCAN_E_UNSUPPORTED;
    if ((!top_k && top_k_all < 0) || (!top_p && !(top_p_all >= 0.f && top_p_all <= 1.f)) ||
        (!min_p && !(min_p_all >= 0.f && min_p_all <= 1.f)))
        return SELSCAN_E_UNSUPPORTED;
    if (rows == 0) return SELSCAN_OK;
    if (vocab == 0 || logits_stride < vocab || mul_size(rows, logits_stride) < 0) return SELSCAN_E_SHAPE;
    if (!logits || !uniform || !token || !logprob || !kept) return SELSCAN_E_NULL;
    const size_t s = io_bytes(io_dtype);
    const void *words[] = {uniform, temperature, top_k, top_p, min_p, logprob, kept};
    for (const void *w : words)
        if (!span_aligned(w, 4)) return SELSCAN_E_ALIGN;
    if (!span_aligned(logits, s) || !span_aligned(token, 8)) return SELSCAN_E_ALIGN;
    const size_t n = (size_t)rows * 4;
    const Span in[] = {{logits, strided_bytes(rows, vocab, logits_stride, s)}, {uniform, n}, {temperature, n}, {top_k, n}, {top_p, n}, {min_p, n}};
    const Span out[] = {{token, 2 * n}, {logprob, n}, {kept, n}};
    if (any_alias(in, 6, out, 3)) return SELSCAN_E_ALIAS;
    if (!grid_fits(rows, kThreads)) return SELSCAN_E_UNSUPPORTED;
    SampleParams p{};
    p.x = logits, p.uniform = uniform, p.temperature = temperature, p.top_p = top_p, p.min_p = min_p, p.top_k = top_k;
    p.token = token, p.logprob = logprob, p.kept = kept, p.stride = logits_stride, p.vocab = (int)vocab;
    p.temperature_all = temperature_all, p.top_k_all = top_k_all, p.top_p_all = top_p_all, p.min_p_all = min_p_all;
    int bits = 0;
    while ((INT64_C(1) << bits) < vocab) ++bits;
    p.shift = 62 - bits < 51 ? 62 - bits : 51;  // sums stay below 2^63, weights below 2^52
    p.rounds = (int)((vocab + kRound - 1) / kRound);
    return enqueue(io_dtype == SELSCAN_BF16 ? sample_row<uint16_t> : sample_row<float>, dim3((unsigned)rows), dim3(kThreads), p, stream);
}
