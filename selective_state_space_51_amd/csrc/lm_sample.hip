// libselscan_lm - the next token drawn from logits (token_sample of include/selscan_lm.h).  MI355X (gfx950).
//
// With T the temperature and m a row's largest logit, token i has weight 2^t, t = (x_i - m) log2(e) / T, as a whole multiple of
// 2^-shift.  Whole numbers add up to the same sum in any order, so that which tokens stay and which one is drawn does not depend
// on how a row is split; they are 64 bits wide, and t and its power are formed in 64 bits, since both turn on sums of up to
// 2^21 weights next to a border.
//
// Tokens are ranked by their logit and then by their index, as one number of 64 bits (entry); top-k and top-p
// leave those from a bound on.
#include "lm_common.h"

#include <float.h>

namespace {

constexpr int kMaxVocab = 1 << 21;
constexpr int kThreads = 1024, kWaves = kThreads / 64;
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
    float temperature_all, top_p_all, min_p_all;
};

// floats in the order of their values as unsigned numbers (both zeros alike)
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 entry(float x, int index) { return (u64)order_of(x) << 32 | (uint32_t)~index; }

// 2^t as a multiple of 2^-shift, t <= 0: the Taylor sum of 2^f for |f| <= 1/2 (its rest is below 2^-56)
__device__ __forceinline__ u64 weight(double t, int shift) {
    const double n = rint(t), f = (t - n) * 0.693147180559945309417232121458;
    double e = 1. / 479001600.;
    e = fma(e, f, 1. / 39916800.);
    e = fma(e, f, 1. / 3628800.);
    e = fma(e, f, 1. / 362880.);
    e = fma(e, f, 1. / 40320.);
    e = fma(e, f, 1. / 5040.);
    e = fma(e, f, 1. / 720.);
    e = fma(e, f, 1. / 120.);
    e = fma(e, f, 1. / 24.);
    e = fma(e, f, 1. / 6.);
    e = fma(e, f, 0.5);
    e = fma(e, f, 1.);
    e = fma(e, f, 1.);
    return n < -64. ? 0 : (u64)rint(ldexp(e, (int)n + shift));
}

template <class V, class F>
__device__ __forceinline__ V block_reduce(V v, V *sh, F f) {
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v = f(v, __shfl_xor(v, m));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < kWaves; ++i) v = f(v, sh[i]);
    return v;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_row(SampleParams p) {
    __shared__ u64 sh[kWaves];
    const int64_t row = blockIdx.x;
    const T *x = (const T *)p.x + row * p.stride;
    const int n = p.vocab, tid = threadIdx.x;
    const auto add = [](u64 a, u64 b) { return a + b; };
    const auto larger = [](u64 a, u64 b) { return a > b ? a : b; };
    const auto sum = [&](auto f) {
        u64 s = 0;
        for (int i = tid; i < n; i += kThreads) s += f(i, Io<T>::f32(x[i]));
        return block_reduce(s, sh, add);
    };
    // the best token; whether a NaN or an infinity is among them; how many have a weight at all
    u64 best = 0;
    uint32_t bad = 0, live = 0;
    for (int i = tid; i < n; i += kThreads) {
        const float v = Io<T>::f32(x[i]);
        bad |= !(v < INFINITY);
        live += v > -INFINITY;
        best = larger(best, entry(v, i));
    }
    best = block_reduce(best, sh, larger);
    const u64 seen = block_reduce((u64)bad << 32 | live, sh, [](u64 a, u64 b) { return ((a | b) >> 32 << 32) | (uint32_t)((uint32_t)a + (uint32_t)b); });
    bad = (uint32_t)(seen >> 32), live = (uint32_t)seen;
    if (bad || !live) {
        if (tid == 0) p.token[row] = -1, p.logprob[row] = bad ? NAN : -INFINITY, p.kept[row] = 0;
        return;
    }
    const int first = (int)~(uint32_t)best;
    const float T_ = p.temperature ? p.temperature[row] : p.temperature_all;
    const int k = p.top_k ? p.top_k[row] : p.top_k_all;
    const float tp = p.top_p ? p.top_p[row] : p.top_p_all, mp = p.min_p ? p.min_p[row] : p.min_p_all;
    if (!(T_ > 0.f)) {
        if (tid == 0) p.token[row] = first, p.logprob[row] = 0.f, p.kept[row] = 1;
        return;
    }
    const double m = (double)Io<T>::f32(x[first]), c = 1.44269504088896340735992468100 / (double)T_;
    const auto exponent = [&](float v) { return ((double)v - m) * c; };
    // the bound: the k-th best entry, then the one at which the sum reaches top_p of the whole; found bit by bit
    u64 bound = entry(-FLT_MAX, kMaxVocab);
    const auto search = [&](auto reaches) {
        u64 b = 0;
        for (int bit = 63; bit >= 0; --bit)
            if (reaches(b | (u64)1 << bit)) b |= (u64)1 << bit;
        return b;
    };
    if (k > 0 && (uint32_t)k < live)
        bound = search([&](u64 b) { return sum([&](int i, float v) { return (u64)(entry(v, i) >= b); }) >= (u64)k; });
    const auto mass = [&](u64 b) {
        return sum([&](int i, float v) { return entry(v, i) >= b && v > -INFINITY ? weight(exponent(v), p.shift) : 0; });
    };
    if (tp < 1.f) {
        const double want = (double)(tp > 0.f ? tp : 0.f) * (double)mass(bound);
        const u64 b0 = bound;
        const u64 b = search([&](u64 b) { return (double)mass(b > b0 ? b : b0) >= want; });
        bound = b < b0 ? b0 : b > best ? best : b;
    }
    const double low = log2((double)(mp > 1.f ? 1.f : mp > 0.f ? mp : 0.f));
    const auto stays = [&](int i, float v) { return entry(v, i) >= bound && v > -INFINITY && exponent(v) >= low; };
    const u64 total = sum([&](int i, float v) { return stays(i, v) ? weight(exponent(v), p.shift) : 0; });
    const u64 kept = sum([&](int i, float v) { return (u64)stays(i, v); });
    const float u = p.uniform[row];
    u64 at = u > 0.f ? (u64)((double)u * (double)total) : 0;
    at = at < total ? at : total - 1;
    int lo = 0, hi = n - 1;
    while (lo < hi) {  // the first token at which the sum passes `at`
        const int mid = (lo + hi) >> 1;
        if (sum([&](int i, float v) { return i <= mid && stays(i, v) ? weight(exponent(v), p.shift) : 0; }) > at) hi = mid;
        else lo = mid + 1;
    }
    if (tid == 0) {
        p.token[row] = lo;
        p.logprob[row] = (float)((exponent(Io<T>::f32(x[lo])) + p.shift - log2((double)total)) * 0.693147180559945309417232121458);
        p.kept[row] = (int32_t)kept;
    }
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
    p.shift = 62 - bits < 52 ? 62 - bits : 52;  // sums stay below 2^63
    return enqueue(io_dtype == SELSCAN_BF16 ? sample_row<uint16_t> : sample_row<float>, dim3((unsigned)rows), dim3(kThreads), p, stream);
}
