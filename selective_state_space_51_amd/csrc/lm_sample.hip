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
constexpr int kPart = 512;  // logits of a round of a wave: 8 adjacent ones of each lane
constexpr int kBins = 2048, kList = 256, kSteps = 256, kMaxThreads = 1024;
constexpr size_t kLds = 160 << 10;
typedef unsigned long long u64;

struct SampleParams {
    const void *x;
    const float *uniform, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logprob;
    int32_t *kept;
    int64_t stride;
    int vocab, shift, top_k_all;
    int rounds, join;  // of a wave, which has a stretch of the row; rounds whose weights are added up together
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

// 2^(i / 256)
struct Steps {
    double v[kSteps];
    constexpr Steps() : v() {
        for (int i = 0; i < kSteps; ++i) {
            const double f = i * (0.693147180559945309417232121458 / kSteps);
            double e = 1.;
            for (int n = 24; n > 0; --n) e = 1. + e * f / n;
            v[i] = e;
        }
    }
};
__constant__ const Steps kStepTable;

struct SampleLds {
    u64 bins[kBins];  // (of the draw: sums over parts of the row; of few tokens: entries and weights of a bin)
    double step[kSteps];
    u64 entries[kList], weights[kList];
    u64 part[2][16];
    u64 found[2];
    int listed[kList];
    float few[kMaxThreads];  // tokens taken out of the row, in the order of their indices
    int few_at[kMaxThreads];
    int count;
};

// over the workgroup; buf: 0 or 1, not that of the reduction just before
template <int kWaves, class F>
__device__ __forceinline__ u64 block_reduce(SampleLds &m, u64 v, int buf, F f) {
    v = lane_of(wave_scan(v, f), 63);
    if ((threadIdx.x & 63) == 0) m.part[buf][threadIdx.x >> 6] = v;
    lds_barrier();
    u64 a = m.part[buf][threadIdx.x & (kWaves - 1)];
    a = f(a, dpp_u64<0x111, 0xF>(a));
    a = f(a, dpp_u64<0x112, 0xF>(a));
    a = f(a, dpp_u64<0x114, 0xF>(a));
    if constexpr (kWaves > 8) a = f(a, dpp_u64<0x118, 0xF>(a));
    return lane_of(a, kWaves - 1);
}
// The sum over the threads before this one, and the whole.
template <int kWaves>
__device__ __forceinline__ u64 block_scan(SampleLds &m, u64 v, int buf, u64 &whole) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const u64 up = wave_scan(v, Add());
    if (lane == 63) m.part[buf][wave] = up;
    lds_barrier();
    u64 before = up - v;
    whole = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const u64 s = m.part[buf][w];
        before += w < wave ? s : 0;
        whole += s;
    }
    return before;
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

// HELD: the row lies in LDS after its first reading.
//
// Where top-k or min_p leave few tokens, those and all larger than the smallest of them are taken out of the row in the order of
// their indices, from an edge on that is found among the threads' largest logits (or follows from min_p), and the rest is about
// them, one in each thread.  Else the same is done on the row itself; top-p on bf16 logits by counting equal ones first, so that a
// weight is formed for each value and not for each token.
//
// Instructions bound it: each logit passes three to six passes, 4 instructions in the first and about 30 where its weight is formed.
// 1,000 rows of 32,001 fp32 logits without limits take 59 us (vector units busy for 70 %, 2.2 TB/s), 64 of 131,072 bf16 with top-p 67
// (80 % of 64 compute units), 256 of 50,280 with mixed settings 36, three of them 21 (the chain of passes of one row).  A pass over a
// row costs a compute unit an instruction's issue for every 64 logits' step, and most of the code runs once or twice for a row and has to be
// fetched for that: loops are not unrolled over rounds.  Weights of eight logits are formed
// side by side, without a branch between them, or not at all where no lane of the wave has one that counts (one after another for
// those that count: 64 rows 66 us for 67, 256 rows 39 for 36).
template <typename T, int kWaves, bool HELD>
__global__ __launch_bounds__(64 * kWaves, 4) void sample_row(SampleParams p) {
    constexpr int kThreads = 64 * kWaves, kOwn = kBins / kThreads, kFew = kThreads;
    __shared__ __attribute__((aligned(16))) SampleLds m;
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    T *held = (T *)dynamic;
    const int64_t row = blockIdx.x;
    const T *x = (const T *)p.x + row * p.stride;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int start = wave * p.rounds * kPart + lane * 8;
    const auto each = [&](auto f) {  // f(first index, 8 logits)
        if constexpr (HELD) {
#pragma unroll 1
            for (int v = 0; v < p.rounds; ++v) f(start + v * kPart, load_raw8(held + start + v * kPart, 8, true));
        } else {
            Raw8<T> next = load_logits(x, start, p.vocab);
#pragma unroll 1
            for (int v = 0; v < p.rounds; ++v) {
                const Raw8<T> r = next;
                next = load_logits(x, start + (v + 1) * kPart, p.vocab);
                f(start + v * kPart, r);
            }
        }
    };
    if (tid < kSteps) m.step[tid] = kStepTable.v[tid];

    // the largest logit, and whether a NaN or an infinity is among them
    float best = -INFINITY;
    bool bad = false;
    constexpr int A = 4;  // rounds in flight
#pragma unroll 1
    for (int v = 0; v < p.rounds; v += A) {
        Raw8<T> r[A];
#pragma unroll
        for (int a = 0; a < A; ++a) r[a] = load_logits(x, start + (v + a) * kPart, v + a < p.rounds ? p.vocab : 0);
#pragma unroll
        for (int a = 0; a < A; ++a) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = raw_f32(r[a], e);
                bad |= !(f < INFINITY);
                best = fmaxf(best, f);
            }
            if constexpr (HELD) {
                if (v + a < p.rounds) {
                    uint4 *to = (uint4 *)(held + start + (v + a) * kPart);
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                        to[i] = make_uint4(r[a].w[4 * i], r[a].w[4 * i + 1], r[a].w[4 * i + 2], r[a].w[4 * i + 3]);
                }
            }
        }
    }
    const u64 most = block_reduce<kWaves>(m, __any(bad) ? ~(u64)0 : order_of(best), 0, Larger());
    const float top = value_of((uint32_t)most);
    if (most == ~(u64)0 || top == -INFINITY) {
        if (tid == 0) p.token[row] = -1, p.logprob[row] = most == ~(u64)0 ? NAN : -INFINITY, p.kept[row] = 0;
        return;
    }
    const float temperature = p.temperature ? p.temperature[row] : p.temperature_all;
    const int k = p.top_k ? p.top_k[row] : p.top_k_all;
    const float top_p = p.top_p ? p.top_p[row] : p.top_p_all, min_p = p.min_p ? p.min_p[row] : p.min_p_all;
    const bool one = !(temperature > 0.f) || k == 1 || top_p <= 0.f;  // the first of the largest
    const bool by_k = k > 0 && k < p.vocab, by_p = top_p < 1.f;
    const double m64 = top, c = 1.44269504088896340735992468100 / (temperature > 0.f ? (double)temperature : 1.), c256 = c * 256.;
    const auto weight = [&](float v) { return weight_of(m, v, m64, c256, p.shift); };
    // min_p is held against the weights; logits clearly below it are left out beforehand
    const u64 least = min_p > 0.f ? (u64)ceil(ldexp((double)(min_p < 1.f ? min_p : 1.f), p.shift)) : 0;
    float pre = -FLT_MAX;
    if (min_p > 0.f) {
        const float f = (float)(m64 + ((double)__builtin_amdgcn_logf(min_p < 1.f ? min_p : 1.f) * 1.001 - 0.001) / c);
        pre = f - fabsf(f) * 1e-6f;
        pre = pre > -FLT_MAX ? pre : -FLT_MAX;
    }
    const float u = p.uniform[row];
    const auto place_of = [&](u64 total) {  // the sum that the drawn token is the first to pass
        const u64 at = u > 0.f ? (u64)((double)(u < 1.f ? u : 1.f) * (double)total) : 0;
        return at < total ? at : total - 1;
    };
    const auto mass_wanted = [&](u64 whole) {
        const u64 want = (u64)ceil((double)top_p * (double)whole);
        return want < 1 ? 1 : want < whole ? want : whole;
    };
    const auto write = [&](int i, float v, u64 total, uint32_t kept) {
        p.token[row] = i;
        p.logprob[row] = (float)((((double)v - m64) * c + p.shift - log2((double)total)) * 0.693147180559945309417232121458);
        p.kept[row] = (int32_t)kept;
    };

    // bins of the logit, `per` of them to a unit, from the largest on
    float per = 0.f;
    const auto wide_bin = [&](float v) {
        const float d = (top - v) * per;
        return (int)(d < (float)(kBins - 1) ? d : (float)(kBins - 1));
    };
    const auto set_bins = [&](float n) { per = n < FLT_MAX ? n : FLT_MAX; };
    const auto clear = [&] {
        lds_barrier();
#pragma unroll
        for (int b = 0; b < kOwn; ++b) m.bins[tid + b * kThreads] = 0;
        if (tid == 0) m.found[0] = kBins, m.count = 0;
        lds_barrier();
    };
    // The bin in which the sum over the bins, from the first on and from base, reaches want_of(whole), and the sum before it;
    // kBins where the whole does not reach it.
    const auto crossing = [&](u64 base, auto want_of, u64 &want, u64 &before) {
        lds_barrier();
        u64 own[kOwn], s = 0, whole;
#pragma unroll
        for (int b = 0; b < kOwn; ++b) own[b] = m.bins[kOwn * tid + b], s += own[b];
        u64 at = base + block_scan<kWaves>(m, s, 0, whole);
        want = want_of(whole);
#pragma unroll
        for (int b = 0; b < kOwn; ++b) {
            if (at < want && at + own[b] >= want) m.found[0] = kOwn * tid + b, m.found[1] = at;
            at += own[b];
        }
        lds_barrier();
        before = m.found[1];
        return (int)m.found[0];
    };

    // Takes out the tokens whose logit pick() picks, in the order of their indices; returns their number, of which kFew at most
    // are there.
    const auto take = [&](auto pick) {
        const auto picked = [&](const Raw8<T> &r) {
            uint32_t some = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) some |= (uint32_t)pick(raw_f32(r, e)) << e;
            return some;
        };
        uint32_t mine = 0;
        each([&](int, const Raw8<T> &r) { mine += __popc(picked(r)); });
        u64 n;
        lds_barrier();
        uint32_t place = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)block_scan<kWaves>(m, mine, 1, n));
        each([&](int i, const Raw8<T> &r) {
            const uint32_t some = picked(r);
            if (!__any(some != 0) || place >= kFew) return;
            const uint32_t up = (uint32_t)wave_scan(__popc(some), Add());
            uint32_t at = place + up - __popc(some);
            place += (uint32_t)__builtin_amdgcn_readlane((int)up, 63);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (some >> e & 1) {
                    if (at < kFew) m.few[at] = raw_f32(r, e), m.few_at[at] = i + e;
                    ++at;
                }
            }
        });
        lds_barrier();
        return (int)n;
    };

    // ---- few tokens
    float edge = -FLT_MAX;  // no token that stays is below it
    if (one) {
        edge = top;
    } else if (by_k && k <= kThreads / 2) {
        // The n-th largest of all is no smaller than the n-th of the threads' largest, nor so than the smallest of those in
        // that one's bin or before it.  (Threads past the end of the row, and those whose logits are all masked, have none.)
        const bool none = best < -FLT_MAX;
        const float far = value_of(~(uint32_t)block_reduce<kWaves>(m, (uint32_t)~order_of(none ? top : best), 1, Larger()));
        set_bins((float)kBins / (top - far));
        const int bin = wide_bin(best);
        clear();
        if (!none) atomicAdd(&m.bins[bin], (u64)1);
        u64 want, before;
        const int at = crossing(0, [&](u64 whole) { return (u64)k < whole ? (u64)k : whole; }, want, before);
        edge = value_of(~(uint32_t)block_reduce<kWaves>(m, !none && bin <= at ? ~order_of(best) : 0, 1, Larger()));
        // (fewer of the threads than wanted have one: all that there are)
        if (want < (u64)k) edge = -FLT_MAX;
    }
    edge = edge < pre && !by_p ? pre : edge;
    if (one || edge > -FLT_MAX) {
        const int n = take([&](float v) { return v >= edge; });
        if (n <= kFew || one) {
            if (one) {
                if (tid == 0) p.token[row] = m.few_at[0], p.logprob[row] = 0.f, p.kept[row] = 1;
                return;
            }
            const bool on = tid < n;
            const float v = on ? m.few[tid] : top;
            const int i = on ? m.few_at[tid] : 0;
            const u64 en = on ? entry_of(v, i) : 0, w = on ? weight(v) : 0;
            u64 bound = 1;
            set_bins((float)kBins / (top - edge));
            const int bin = wide_bin(v);
#pragma unroll 1
            for (int step = by_k ? 0 : 1; step < (by_p ? 2 : 1); ++step) {  // 0: top-k, 1: top-p
                const bool in = en >= bound;
                const u64 what = step ? w : 1;
                clear();
                if (in) atomicAdd(&m.bins[bin], what);
                u64 want, base;
                const int at = crossing(0, [&](u64 whole) { return step ? mass_wanted(whole) : (u64)k; }, want, base);
                if (at == kBins) continue;  // fewer than k: all stay
                // (its tokens, where the bins were)
                if (in && bin == at) {
                    const int to = atomicAdd(&m.count, 1);
                    m.bins[to] = en, m.bins[kFew + to] = what;
                }
                lds_barrier();
                const int count = m.count;
                if (in && bin == at) {
                    u64 above = base;
#pragma unroll 4
                    for (int j = 0; j < count; ++j) above += m.bins[j] > en ? m.bins[kFew + j] : 0;
                    if (above < want && above + what >= want) m.found[0] = en;
                }
                lds_barrier();
                bound = m.found[0];
            }
            const bool stay = en >= bound && w >= least;
            u64 total;
            lds_barrier();
            const u64 before = block_scan<kWaves>(m, stay ? w : 0, 0, total), kept = block_reduce<kWaves>(m, stay ? 1 : 0, 1, Add());
            const u64 at = place_of(total);
            if (stay && before <= at && at < before + w) write(i, v, total, (uint32_t)kept);
            return;
        }
    }

    // ---- the row itself
    float bv = -FLT_MAX;  // tokens stay from this one on
    int bi = INT32_MAX;
    const auto stays = [&](float v, int i) { return (v > bv) | ((v == bv) & (i <= bi)); };
    // Bounds: at the token at which the sum of 1 for each (top-k) or of weights (top-p), from the largest logit on, reaches what is
    // wanted.  Nothing changes where the whole does not reach it.
    if (by_k) set_bins((float)kBins / (top - (edge > -FLT_MAX ? edge : top - 64.f)));
    u64 want = 0, base = 0, hi = 0, lo = 0;
    int sh = -1;  // bins of the logit; else of entry numbers, 2^sh of them from hi down to lo
    bool weigh = !by_k, more = by_k || by_p;
    const float weight_bins = (float)((double)kBins * c / (p.shift + 2));
    if (weigh) set_bins(weight_bins);
    if constexpr (sizeof(T) == 2) {
        if (by_p && !by_k) {
            // How many tokens have each value, largest value first: both signs of 16 octaves, which hold every logit that has a
            // weight but those near 0.  These lie between the positive and the negative ones; if the sum is reached among them
            // the row is not done this way, nor if they are many.
            uint32_t *counts = (uint32_t *)m.bins;
            const double reach = (p.shift + 3) / c;  // (at this distance from the largest: no weight)
            const float far = m64 - reach > -FLT_MAX ? (float)(m64 - reach) : -FLT_MAX;
            const int lowest = (int)(__float_as_uint(fmaxf(fabsf(top), fabsf(far))) >> 23) * 128 - 15 * 128;
            clear();
            if (tid == 0) m.found[0] = ~(u64)0;
            each([&](int i, const Raw8<T> &r) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int b = (int)(r.w[e >> 1] << (e & 1 ? 0 : 16)) >> 16;
                    const int at = (b & 0x7FFF) - lowest;
                    if ((uint32_t)at < 2048u) {
                        atomicAdd(&counts[2048 + (at ^ ~(b >> 31))], 1u);
                    } else if (raw_f32(r, e) >= far) {
                        const int to = atomicAdd(&m.count, 1);
                        if (to < kList) m.listed[to] = i + e;
                    }
                }
            });
            lds_barrier();
            const int odd = m.count;
            if (odd <= kList && lowest > 0) {
                constexpr int kMine = 2 * kBins / kThreads;
                u64 w[kMine], s = 0, mid = 0, whole;
#pragma unroll
                for (int b = 0; b < kMine; ++b) {
                    const int at = tid * kMine + b - 2048;
                    const uint32_t n = counts[tid * kMine + b];
                    w[b] = n ? weight(__uint_as_float((uint32_t)((at >= 0 ? at : ~at) + lowest) << 16 | (at >= 0 ? 0x80000000u : 0u))) : 0;
                    s += w[b] * n;
                }
                if (tid < odd) {
                    const int i = m.listed[tid];
                    mid = weight(Io<T>::f32(HELD ? held[i] : x[i]));
                }
                const u64 before = block_scan<kWaves>(m, s, 0, whole);
                mid = block_reduce<kWaves>(m, mid, 1, Add());
                want = mass_wanted(whole + mid);
                u64 at = before + (tid >= kThreads / 2 ? mid : 0);
#pragma unroll
                for (int b = 0; b < kMine; ++b) {
                    const u64 to = at + w[b] * counts[tid * kMine + b];
                    if (at < want && to >= want) m.found[0] = tid * kMine + b, m.found[1] = (want - at + w[b] - 1) / w[b];
                    at = to;
                }
                lds_barrier();
                if (m.found[0] != ~(u64)0) {
                    // of the tokens with that value so many stay, by their indices
                    const int bin = (int)m.found[0], to = bin - 2048;
                    const uint32_t some = (uint32_t)m.found[1], n = counts[bin];
                    const float v = __uint_as_float((uint32_t)((to >= 0 ? to : ~to) + lowest) << 16 | (to >= 0 ? 0x80000000u : 0u));
                    if (some < n) {
                        const auto picked = [&](const Raw8<T> &r) {
                            uint32_t bits = 0;
#pragma unroll
                            for (int e = 0; e < 8; ++e) bits |= (uint32_t)(raw_f32(r, e) == v) << e;
                            return bits;
                        };
                        uint32_t mine = 0;
                        each([&](int, const Raw8<T> &r) { mine += __popc(picked(r)); });
                        u64 all;
                        const uint32_t first = (uint32_t)block_scan<kWaves>(m, mine, 1, all);
                        uint32_t place = (uint32_t)__builtin_amdgcn_readfirstlane((int)first);
                        // (the wave that has the last one that stays)
                        if (place < some && some <= (uint32_t)__builtin_amdgcn_readlane((int)(first + mine), 63)) {
                            each([&](int i, const Raw8<T> &r) {
                                uint32_t bits = picked(r);
                                if (!__any(bits != 0) || place >= some) return;
                                const uint32_t own = __popc(bits), up = place + (uint32_t)wave_scan(own, Add());
                                if (up - own < some && some <= up) {
                                    for (uint32_t j = up - own + 1; j < some; ++j) bits &= bits - 1;
                                    m.found[0] = (u64)(i + __builtin_ctz(bits));
                                }
                                place = (uint32_t)__builtin_amdgcn_readlane((int)up, 63);
                            });
                        }
                        lds_barrier();
                        bi = (int)m.found[0];
                    }
                    bv = v;
                    more = false;
                }
            }
        }
    }
#pragma unroll 1
    while (more) {
        clear();
        int bin = -1;
        float most_v = -FLT_MAX, least_v = top;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {  // 0: the sums; 1: a list of the tokens of the bin that they lead to
            each([&](int i, const Raw8<T> &r) {
                int at[8];
                bool in[8], some = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = raw_f32(r, e);
                    in[e] = (v >= edge) & stays(v, i + e);
                    at[e] = wide_bin(v);
                }
                if (sh >= 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const u64 en = entry_of(raw_f32(r, e), i + e);
                        in[e] &= (en <= hi) & (en >= lo);
                        at[e] = (int)((hi - en) >> sh);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) in[e] &= (pass == 0) | (at[e] == bin), some |= in[e];
                if (!__any(some)) return;
                if (pass == 0) {
                    u64 w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 1;
                    if (weigh) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = weight(raw_f32(r, e));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (in[e]) atomicAdd(&m.bins[at[e]], w[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (!in[e]) continue;
                        const float v = raw_f32(r, e);
                        most_v = fmaxf(most_v, v), least_v = fminf(least_v, v);
                        const int to = atomicAdd(&m.count, 1);
                        if (to < kList) m.listed[to] = i + e;
                    }
                }
            });
            if (pass == 1) break;
            const u64 known = want;
            u64 before;
            bin = crossing(base, [&](u64 whole) { return sh >= 0 ? known : weigh ? mass_wanted(whole) : (u64)k; }, want, before);
            if (bin == kBins) break;
            base = before;
        }
        lds_barrier();
        const int count = m.count;
        if (bin < kBins && count > kList) {
            // The entry numbers of the bin: those of the values in it and, where it was one of entry numbers, no others than
            // its own (what lies before it is in the base; a value of more than 2^19 tokens takes two such rounds).  Each of
            // these leaves a 2,048th of the numbers, so that six of them end the search.
            u64 first = block_reduce<kWaves>(m, order_of(most_v), 0, Larger()) << 32 | 0xFFFFFFFFu;
            u64 last = (u64)(~(uint32_t)block_reduce<kWaves>(m, (uint32_t)~order_of(least_v), 1, Larger())) << 32 | (uint32_t)~(p.vocab - 1);
            if (sh >= 0) {
                const u64 from = hi - ((u64)bin << sh), to = from - ((1ull << sh) - 1);
                first = first < from ? first : from, last = last > to ? last : to;
            }
            hi = first, lo = last;
            sh = 64 - __builtin_clzll((hi - lo) | 1) - 11;
            sh = sh < 0 ? 0 : sh;
            continue;
        }
        if (bin < kBins) {
            u64 en = 0, w = 1;
            if (tid < count) {
                const int i = m.listed[tid];
                const float v = Io<T>::f32(HELD ? held[i] : x[i]);
                en = entry_of(v, i);
                if (weigh) w = weight(v);
                m.entries[tid] = en, m.weights[tid] = w;
            }
            lds_barrier();
            if (tid < count) {
                u64 above = base;
#pragma unroll 4
                for (int j = 0; j < count; ++j) above += m.entries[j] > en ? m.weights[j] : 0;
                if (above < want && above + w >= want) m.found[0] = en;
            }
            lds_barrier();
            bv = value_of((uint32_t)(m.found[0] >> 32));
            bi = (int)~(uint32_t)m.found[0];
        }
        more = by_p && !weigh;
        weigh = true, base = 0, edge = -FLT_MAX, sh = -1;
        set_bins(weight_bins);
    }

    // The draw: the weights of each wave's rounds, `join` of them together, in the order of the indices
    pre = pre < bv ? bv : pre;
    const auto weights = [&](int i, const Raw8<T> &r, u64 (&w)[8]) {
        uint32_t kept = 0;
        bool in[8], some = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) in[e] = stays(raw_f32(r, e), i + e) & (raw_f32(r, e) >= pre), some |= in[e], w[e] = 0;
        if (__any(some)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = weight(raw_f32(r, e));
                in[e] &= w[e] >= least;
                w[e] = in[e] ? w[e] : 0;
                kept += in[e];
            }
        }
        return kept;
    };
    const auto sum_of = [](const u64 (&w)[8]) { return (w[0] + w[1] + w[2] + w[3]) + (w[4] + w[5] + w[6] + w[7]); };
    const int units = (p.rounds + p.join - 1) / p.join;  // of a wave
    uint32_t kept = 0;
    lds_barrier();
    {
        u64 sum = 0;
        int left = p.join, unit = wave * units, v = p.rounds;
        each([&](int i, const Raw8<T> &r) {
            u64 w[8];
            kept += weights(i, r, w);
            sum += sum_of(w);
            --v;
            if (--left == 0 || v == 0) {
                const u64 s = __any(sum != 0) ? lane_of(wave_scan(sum, Add()), 63) : 0;
                if (lane == 0) m.bins[unit] = s;
                ++unit, left = p.join, sum = 0;
            }
        });
    }
    const uint32_t stay = (uint32_t)block_reduce<kWaves>(m, kept, 0, Add());  // (its barrier is the sums' too)
    if (wave != 0) return;
    // the first wave: a share of the sums in each lane, in order
    const int n = units * kWaves, share = (n + 63) / 64;
    u64 s = 0;
    for (int i = lane * share; i < n && i < (lane + 1) * share; ++i) s += m.bins[i];
    const u64 up = wave_scan(s, Add()), total = lane_of(up, 63), at = place_of(total);
    const int l1 = __builtin_ctzll(__ballot(up > at));
    u64 before = lane_of(up - s, l1);
    int unit = l1 * share;
    while (before + m.bins[unit] <= at) before += m.bins[unit++];
    // the rounds of that wave and unit
#pragma unroll 1
    for (int v = unit % units * p.join; v < p.rounds; ++v) {
        const int i0 = (unit / units * p.rounds + v) * kPart + lane * 8;
        const Raw8<T> r = load_logits(x, i0, p.vocab);
        u64 w[8];
        weights(i0, r, w);
        const u64 sum = sum_of(w), upto = before + wave_scan(sum, Add()), whole = lane_of(upto, 63);
        if (whole <= at) {
            before = whole;
            continue;
        }
        if (lane == (int)__builtin_ctzll(__ballot(upto > at))) {
            int e = 0;
            float f = 0.f;
            u64 to = upto;
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                if (to > at) e = j, f = raw_f32(r, j);
                to -= w[j];
            }
            write(i0 + e, f, total, stay);
        }
        return;
    }
}

template <typename T, int WAVES>
int launch_sample(SampleParams p, int64_t rows, void *stream) {
    const dim3 grid((unsigned)rows), block(64 * WAVES);
    p.rounds = (p.vocab + WAVES * kPart - 1) / (WAVES * kPart);
    p.join = (p.rounds * WAVES + kBins - 1) / kBins;
    const size_t bytes = (size_t)p.rounds * WAVES * kPart * sizeof(T);
    if (WAVES == 16 && bytes + (sizeof(SampleLds) + 15) / 16 * 16 <= kLds) return enqueue(sample_row<T, 16, true>, grid, block, p, stream, (unsigned)bytes);
    return enqueue(sample_row<T, WAVES, false>, grid, block, p, stream);
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
    if (!grid_fits(rows, kMaxThreads)) return SELSCAN_E_UNSUPPORTED;
    SampleParams p{};
    p.x = logits, p.uniform = uniform, p.temperature = temperature, p.top_p = top_p, p.min_p = min_p, p.top_k = top_k;
    p.token = token, p.logprob = logprob, p.kept = kept, p.stride = logits_stride, p.vocab = (int)vocab;
    p.temperature_all = temperature_all, p.top_k_all = top_k_all, p.top_p_all = top_p_all, p.min_p_all = min_p_all;
    int bits = 0;
    while ((INT64_C(1) << bits) < vocab) ++bits;
    p.shift = 62 - bits < 51 ? 62 - bits : 51;  // sums stay below 2^63, weights below 2^52
    // Up to 256 rows each has a compute unit, 16 waves and, if it fits, a place in LDS (200 rows of 32,001 bf16 17.3 us, with 8 waves that
    // read it again 19.5).  More have 8 waves, several to a compute unit, so that one's barriers pass while another works (512 rows 30.5
    // us for 33, 1,024 53 for 62, with top-p 88 for 95, fp32 122 for 139; 400 rows of 131,072 bf16 149 for 156).
    const bool two = rows > 256;
    if (io_dtype == SELSCAN_BF16) return two ? launch_sample<uint16_t, 8>(p, rows, stream) : launch_sample<uint16_t, 16>(p, rows, stream);
    return two ? launch_sample<float, 8>(p, rows, stream) : launch_sample<float, 16>(p, rows, stream);
}
