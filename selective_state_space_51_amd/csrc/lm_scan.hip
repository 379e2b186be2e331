// libselscan_lm - the short causal convolution and the selective scan on packed prompts and on
// single tokens, with states in a cache (causal_conv1d_packed_fwd, selscan_packed_fwd,
// causal_conv1d_step, selscan_step of include/selscan_lm.h).  MI355X (gfx950).
#include "lm_common.h"

namespace selscan_rt {
thread_local char g_last_hip_error[160] = "no error";
}  // namespace selscan_rt

namespace {

// ------------------------------------------------------------------------------------
// packed sequences
// ------------------------------------------------------------------------------------

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

// Segments of 2^shift tokens, without a pass over the lengths: sequence s owns the segment numbers
// from (cu[s] >> shift) + s to the next sequence's first, exclusively.  They are at least
// ceil(len / 2^shift) and at least one (floor(a + b) + 1 >= ceil(b) + floor(a)), and all of them together at
// most (tokens >> shift) + nseq, which the host knows; those past a sequence's end have nothing to do.
// The sequence of a segment: the last one whose first segment is not after it, by a search 64
// positions wide (one load for up to 64 sequences).  Every lane of the wave takes part.
__device__ __forceinline__ int seq_of_segment(const Seqs &q, int seg, int shift, int lane) {
    int lo = 0, n = q.nseq;
    while (n > 1) {
        const int step = (n + 63) >> 6, i = lane * step;
        const bool at_or_before = i < n && (cu_at(q, lo + i) >> shift) + lo + i <= seg;
        int c = __popcll(__ballot(at_or_before));
        c = c < 1 ? 1 : c;
        lo += (c - 1) * step;
        n -= (c - 1) * step;
        n = n < step ? n : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
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

constexpr int kConvShift = 4;  // a thread takes 16 tokens of 8 channels

// One workgroup: a segment of 16 tokens of one sequence, a block of 8 channels per thread.  Every
// row of the segment and the width-1 rows before it are read once by the thread (its neighbours in
// time read those again, from L2).  A sequence's first segment holds at least its first width-1 tokens,
// so its threads alone need the cached rows: they read them, and then write the sequence's last
// rows to the cache, in program order on the same addresses.
template <typename T, int K>
__global__ __launch_bounds__(256) void conv_packed(ConvParams p) {
    constexpr int R = 1 << kConvShift, B = sizeof(T) == 2 ? 8 : 4;  // B: rows in flight at a time
    const int seg = blockIdx.x;
    const int s = seq_of_segment(p.q, seg, kConvShift, threadIdx.x & 63);
    const Range rg = range_of(p.q, s);
    const int j = seg - (rg.t0 >> kConvShift) - s;
    const int first = j << kConvShift;
    if (j < 0 || (j > 0 && first >= rg.len)) return;
    const int64_t c0 = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (c0 >= p.dim) return;
    const int nv = (int)(p.dim - c0 < 8 ? p.dim - c0 : 8);
    const bool vec = p.vec != 0;
    const T *x = (const T *)p.x + (int64_t)rg.t0 * p.x_stride + c0;
    T *out = (T *)p.out + (int64_t)rg.t0 * p.dim + c0;
    Raw8<T> win[B + K - 1];  // the rows before the current block, then the block
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        win[i] = Raw8<T>{};
        if (first > 0) win[i] = load_raw8(x + (int64_t)(first - (K - 1) + i) * p.x_stride, nv, vec);
    }
    if constexpr (K > 1) {
        const int64_t slot = p.state ? slot_of(p.q, s) : -1;
        if (first == 0 && slot >= 0) {
            T *st = (T *)p.state + slot * (K - 1) * p.dim + c0;
            if (p.q.carry && p.q.carry[s]) {
#pragma unroll
                for (int i = 0; i < K - 1; ++i) win[i] = load_raw8(st + i * p.dim, nv, vec);
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i) {
                const int at = rg.len - (K - 1) + i;  // row of the sequence, or a cached one where negative
                Raw8<T> r{};
                if (at >= 0) r = load_raw8(x + (int64_t)at * p.x_stride, nv, vec);
#pragma unroll
                for (int o = 0; o < K - 1; ++o)
                    if (at < 0 && o == at + K - 1) r = win[o];
                store_raw8(st + i * p.dim, nv, vec, r);
            }
        }
    }
    const int n = rg.len - first < R ? rg.len - first : R;
    float f[K][8], b[8];
    load_filters<K>(p, c0, nv, f, b);
#pragma unroll
    for (int u0 = 0; u0 < R; u0 += B) {
        if (u0 >= n) break;
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const int t = first + u0 + u < rg.len ? first + u0 + u : rg.len - 1;
            win[K - 1 + u] = load_raw8(x + (int64_t)t * p.x_stride, nv, vec);
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
            if (u0 + u < n) {
                float v[8];
                conv_row<T, K>(f, b, win + u, p.silu, v);
                store8(out + (int64_t)(first + u0 + u) * p.dim, nv, vec, v);
            }
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) win[i] = win[B + i];
    }
}

// One token per sequence: 8 channels per thread, rows_per rows one after another with the filters
// held.  Per row and channel the cache's width-1 values move in and out, shifted by one.
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
        T *st = K > 1 ? (T *)p.state + (slot < 0 ? 0 : slot) * (K - 1) * p.dim + c0 : nullptr;
#pragma unroll
        for (int t = 0; t < K - 1; ++t) {
            win[t] = Raw8<T>{};
            if (slot >= 0) win[t] = load_raw8(st + t * p.dim, nv, vec);
        }
        win[K - 1] = load_raw8((const T *)p.x + r * p.x_stride + c0, nv, vec);
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
    if (rows > INT32_MAX || nseq > INT32_MAX / 2 || dim > INT32_MAX) return SELSCAN_E_UNSUPPORTED;
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
    float *seg;   // split: [nsegs][dim][16] end state of a segment from zero, then the state it starts from
    float *sdt;   // split: [nsegs][dim] sum of delta over the segment
    Seqs q;
    int64_t dim, bc_stride, z_stride;
    int softplus, shift;
    int rows_per;  // step: rows a thread takes one after another
};

// B and C of one step as raw words, wave-uniform.  Scalar loads bring them to scalar registers (rows on 4-byte
// boundaries); otherwise lanes 0-31 load one value each and they are read lane by lane.
template <typename T>
struct BcRaw {
    static constexpr int NW = kN * (int)sizeof(T) / 4;
    uint32_t b[NW], c[NW];
};

template <typename T, bool SC, bool WITH_C>
__device__ __forceinline__ BcRaw<T> load_bc(const T *B, const T *C, int64_t off, int lane) {
    BcRaw<T> r;
    constexpr int NW = BcRaw<T>::NW;
    if constexpr (SC) {
        using W = const __attribute__((address_space(4))) uint32_t;
        W *b = (W *)(uintptr_t)(B + off), *c = (W *)(uintptr_t)(C + off);
#pragma unroll
        for (int i = 0; i < NW; ++i) r.b[i] = b[i];
        if constexpr (WITH_C) {
#pragma unroll
            for (int i = 0; i < NW; ++i) r.c[i] = c[i];
        }
    } else {
        uint32_t v = 0;
        if (lane < kN || (WITH_C && lane < 2 * kN)) {
            const T *src = lane < kN ? B + off + lane : C + off + lane - kN;
            if constexpr (sizeof(T) == 4) v = __float_as_uint(*src);
            else v = *src;
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if constexpr (sizeof(T) == 4) {
                r.b[i] = __builtin_amdgcn_readlane(v, i);
                if constexpr (WITH_C) r.c[i] = __builtin_amdgcn_readlane(v, kN + i);
            } else {
                r.b[i] = __builtin_amdgcn_readlane(v, 2 * i) | (__builtin_amdgcn_readlane(v, 2 * i + 1) << 16);
                if constexpr (WITH_C)
                    r.c[i] = __builtin_amdgcn_readlane(v, kN + 2 * i) | (__builtin_amdgcn_readlane(v, kN + 2 * i + 1) << 16);
            }
        }
    }
    return r;
}
template <typename T>
__device__ __forceinline__ float bc_f32(const uint32_t *w, int n) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[n]);
    else return __uint_as_float(n & 1 ? w[n >> 1] & 0xFFFF0000u : w[n >> 1] << 16);
}

// The scan, one wave per 64 channels of a sequence or segment: a lane walks its channel's tokens in
// order with the 16 states in registers.
//
// Per (token, channel, state) this is mul, exp, mul, fma, fma and nothing else: B and C are the same for every lane
// and come as scalar operands, x, delta, z and y are one coalesced row piece per token, and no state
// passes between lanes.  (A scan whose lanes share a channel needs 2.5 more instructions per element for the maps
// between lanes and the LDS reads of B and C.)  Bound by instruction issue; the price is that only
// sequences x channels / 64 waves exist, so where those do not fill the chip the sequence is cut
// into segments (FULL = false is their first pass, see split_shift).
//
// FULL: y and the last state.  Else a segment's end state from zero and the sum of its delta: the
// segment as a map h -> exp(A sum delta) h + end.
template <typename T, bool ZOH, bool FULL, bool SC>
__global__ __launch_bounds__(64) void scan_packed(ScanParams p) {
    constexpr int U = 4;  // tokens whose x, delta and z are loaded ahead
    const int lane = threadIdx.x;
    const bool split = p.seg != nullptr;
    int s = blockIdx.x, t0, len;
    int64_t slot = -1;
    if (split) {
        s = seq_of_segment(p.q, blockIdx.x, p.shift, lane);
        const Range rg = range_of(p.q, s);
        const int first = ((int)blockIdx.x - (rg.t0 >> p.shift) - s) << p.shift;
        if (first < 0 || first >= rg.len) return;
        t0 = rg.t0 + first;
        len = rg.len - first < (1 << p.shift) ? rg.len - first : 1 << p.shift;
    } else {
        const Range rg = range_of(p.q, s);
        t0 = rg.t0, len = rg.len;
        slot = p.h ? slot_of(p.q, s) : -1;
    }
    t0 = __builtin_amdgcn_readfirstlane(t0), len = __builtin_amdgcn_readfirstlane(len);
    const int64_t dim = p.dim, c0 = (int64_t)blockIdx.y * 64;
    const int lc = (int)(c0 + lane < dim ? lane : dim - 1 - c0);  // lanes past the last channel repeat it
    const bool live = c0 + lane < dim;
    const int64_t ch = c0 + lc;

    float a2[kN], h[kN];
#pragma unroll
    for (int n = 0; n < kN; n += 4) {
        const float4 v = load_f4(p.A + ch * kN + n);
        a2[n] = v.x * kLog2e, a2[n + 1] = v.y * kLog2e, a2[n + 2] = v.z * kLog2e, a2[n + 3] = v.w * kLog2e;
    }
    const float *h_in = nullptr;
    if (FULL && split) h_in = p.seg + ((int64_t)blockIdx.x * dim + ch) * kN;
    else if (FULL && slot >= 0 && p.q.carry && p.q.carry[s]) h_in = p.h + (slot * dim + ch) * kN;
#pragma unroll
    for (int n = 0; n < kN; n += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h_in) v = *(const float4 *)(h_in + n);
        h[n] = v.x, h[n + 1] = v.y, h[n + 2] = v.z, h[n + 3] = v.w;
    }
    const float Dd = FULL && p.D ? p.D[ch] : 0.f, bias = p.bias ? p.bias[ch] : 0.f;
    const T *x = (const T *)p.x + (int64_t)t0 * dim + c0;
    const T *dl = (const T *)p.delta + (int64_t)t0 * dim + c0;
    const T *z = FULL && p.z ? (const T *)p.z + (int64_t)t0 * p.z_stride + c0 : nullptr;
    T *y = (T *)p.y + (int64_t)t0 * dim + c0;
    const T *B = (const T *)p.B + (int64_t)t0 * p.bc_stride, *C = (const T *)p.C + (int64_t)t0 * p.bc_stride;
    float sum = 0.f;

    T xr[U], dr[U], zr[U];
    auto load_block = [&](int t, T (&xb)[U], T (&db)[U], T (&zb)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u < len ? t + u : len - 1;
            xb[u] = (x + (int64_t)tt * dim)[lc];
            db[u] = (dl + (int64_t)tt * dim)[lc];
            if constexpr (FULL) {
                if (z) zb[u] = (z + (int64_t)tt * p.z_stride)[lc];
            }
        }
    };
    BcRaw<T> bc;
    if (len > 0) {
        load_block(0, xr, dr, zr);
        bc = load_bc<T, SC, FULL>(B, C, 0, lane);
    }
    for (int t = 0; t < len; t += U) {
        T xn[U], dn[U], zn[U];
        load_block(t + U, xn, dn, zn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= len) break;
            // the next token's B and C, in flight during this one's arithmetic
            const int tn = t + u + 1 < len ? t + u + 1 : len - 1;
            const BcRaw<T> next = load_bc<T, SC, FULL>(B, C, (int64_t)tn * p.bc_stride, lane);
            float d = Io<T>::f32(dr[u]) + bias;
            if (p.softplus) d = softplus(d);
            const float xv = Io<T>::f32(xr[u]), dx = d * xv;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const float arg = d * a2[n], e = __builtin_amdgcn_exp2f(arg);
                float g = dx;
                if constexpr (ZOH) g = dx * zoh_phi(e, arg);
                h[n] = fmaf(e, h[n], g * bc_f32<T>(bc.b, n));
                if constexpr (FULL) acc[n & 3] = fmaf(bc_f32<T>(bc.c, n), h[n], acc[n & 3]);
            }
            if constexpr (FULL) {
                float v = fmaf(Dd, xv, (acc[0] + acc[1]) + (acc[2] + acc[3]));
                if (z) v *= silu(Io<T>::f32(zr[u]));
                if (live) (y + (int64_t)(t + u) * dim)[lane] = Io<T>::to(v);
            } else {
                sum += d;
            }
            bc = next;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) xr[u] = xn[u], dr[u] = dn[u], zr[u] = zn[u];
    }
    if (!live) return;
    float *h_out = nullptr;
    if (!FULL) h_out = p.seg + ((int64_t)blockIdx.x * dim + ch) * kN;
    else if (slot >= 0) h_out = p.h + (slot * dim + ch) * kN;
    if (h_out) {
#pragma unroll
        for (int n = 0; n < kN; n += 4) *(float4 *)(h_out + n) = make_float4(h[n], h[n + 1], h[n + 2], h[n + 3]);
    }
    if (!FULL) p.sdt[(int64_t)blockIdx.x * dim + ch] = sum;
}

// Joins the segments of a sequence: one thread per (sequence, channel, state) walks its segments in
// order, replaces each end state from zero by the state the segment starts from, and leaves the last in the cache.
__global__ __launch_bounds__(256) void scan_join(ScanParams p) {
    const int s = blockIdx.x;
    const Range rg = range_of(p.q, s);
    const int64_t i = (int64_t)blockIdx.y * 256 + threadIdx.x, ch = i / kN;
    if (ch >= p.dim) return;
    const int64_t slot = p.h ? slot_of(p.q, s) : -1;
    const float a2 = p.A[i] * kLog2e;
    const int first = (rg.t0 >> p.shift) + s, n = (rg.len + (1 << p.shift) - 1) >> p.shift;
    float h = 0.f;
    if (slot >= 0 && p.q.carry && p.q.carry[s]) h = p.h[slot * p.dim * kN + i];
    constexpr int U = 8;  // segments loaded ahead
    for (int j0 = 0; j0 < n; j0 += U) {
        float e[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = first + (j0 + u < n ? j0 + u : n - 1);
            e[u] = p.seg[j * p.dim * kN + i];
            d[u] = p.sdt[j * p.dim + ch];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= n) break;
            p.seg[(int64_t)(first + j0 + u) * p.dim * kN + i] = h;
            h = fmaf(__builtin_amdgcn_exp2f(a2 * d[u]), h, e[u]);
        }
    }
    if (slot >= 0) p.h[slot * p.dim * kN + i] = h;
}

// One token per sequence.  Four lanes per channel hold four states each, so that a wave moves 16 channels' states as
// 1 KB of adjacent memory in and out; y is summed over the four lanes.  HBM bound by the states (128
// bytes per row and channel of fp32 state in and out) where there are many rows; A, D and bias are held
// over the rows_per rows that a thread takes.
template <typename T, bool ZOH>
__global__ __launch_bounds__(256) void scan_step(ScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, ch = i >> 2;
    if (ch >= p.dim) return;  // whole groups of four lanes leave
    const int n0 = (int)(i & 3) * 4;
    const float4 a = load_f4(p.A + ch * kN + n0);
    const float a2[4] = {a.x * kLog2e, a.y * kLog2e, a.z * kLog2e, a.w * kLog2e};
    const float Dd = p.D ? p.D[ch] : 0.f, bias = p.bias ? p.bias[ch] : 0.f;
    const int r0 = blockIdx.y * p.rows_per;
    for (int k = 0; k < p.rows_per; ++k) {
        const int r = r0 + k;
        if (r >= p.q.tokens) break;
        const int64_t slot = slot_of(p.q, r);
        float *hp = p.h + ((slot < 0 ? 0 : slot) * p.dim + ch) * kN + n0;
        float4 hv = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= 0) hv = *(const float4 *)hp;
        float h[4] = {hv.x, hv.y, hv.z, hv.w};
        const T *B = (const T *)p.B + r * p.bc_stride + n0, *C = (const T *)p.C + r * p.bc_stride + n0;
        float d = Io<T>::f32(((const T *)p.delta)[r * p.dim + ch]) + bias;
        if (p.softplus) d = softplus(d);
        const float xv = Io<T>::f32(((const T *)p.x)[r * p.dim + ch]), dx = d * xv;
        float acc = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float arg = d * a2[n], e = __builtin_amdgcn_exp2f(arg);
            float g = dx;
            if constexpr (ZOH) g = dx * zoh_phi(e, arg);
            h[n] = fmaf(e, h[n], g * Io<T>::f32(B[n]));
            acc = fmaf(Io<T>::f32(C[n]), h[n], acc);
        }
        if (slot >= 0) *(float4 *)hp = make_float4(h[0], h[1], h[2], h[3]);
        acc += __shfl_xor(acc, 1);
        acc += __shfl_xor(acc, 2);
        if (n0 == 0) {
            float v = fmaf(Dd, xv, acc);
            if (p.z) v *= silu(Io<T>::f32(((const T *)p.z)[r * p.z_stride + ch]));
            ((T *)p.y)[r * p.dim + ch] = Io<T>::to(v);
        }
    }
}

// Tokens per segment as a power of two, or 0: whole sequences.  A sequence walks alone at the rate of
// its longest, so whole sequences take max(longest, tokens x tiles / SIMDs) token times; segments cost the
// first pass on top (mul, exp, mul, fma of the five: 1.55 times the work) and the join.
constexpr int kSimds = 1024;  // MI355X: 256 compute units of 4

int split_shift(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t dim) {
    const int64_t tiles = (dim + 63) / 64;
    const int64_t longest = max_seqlen < tokens ? max_seqlen : tokens;
    const int64_t share = (tokens * tiles + kSimds - 1) / kSimds;  // token times of a SIMD if all is even
    const int64_t whole = longest > share ? longest : share;
    if (whole <= share + share / 2 + 64) return 0;
    // two waves per SIMD, segments of 32 to 4096 tokens
    int shift = 5;
    while (shift < 12 && (tokens >> shift) * tiles > 2 * kSimds) ++shift;
    if ((INT64_C(2) << shift) > longest) return 0;
    (void)nseq;
    return shift;
}

int64_t segments(int64_t tokens, int64_t nseq, int shift) { return (tokens >> shift) + nseq; }

size_t packed_workspace(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t dim) {
    const int shift = split_shift(tokens, nseq, max_seqlen, dim);
    return shift ? (size_t)segments(tokens, nseq, shift) * (size_t)dim * (kN + 1) * sizeof(float) : 0;
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

int scan_check(const ScanArgs &a, bool *nothing) {
    *nothing = false;
    if (a.rows < 0 || a.nseq < 0 || a.nslots < 0 || a.dim < 0 || a.dstate < 0) return SELSCAN_E_SHAPE;
    if (!io_known(a.dtype) || (a.flags & ~(SELSCAN_FLAG_DELTA_SOFTPLUS | SELSCAN_FLAG_ZOH)) || a.dstate != kN)
        return SELSCAN_E_UNSUPPORTED;
    if (a.rows > INT32_MAX || a.nseq > INT32_MAX / 2 || a.dim > INT32_MAX) return SELSCAN_E_UNSUPPORTED;
    if (a.dim == 0 || a.nseq == 0) {
        *nothing = true;
        return a.nseq == 0 && a.rows > 0 && a.dim > 0 ? SELSCAN_E_SHAPE : SELSCAN_OK;
    }
    if (a.bc_stride < kN || (a.z && a.z_stride < a.dim)) return SELSCAN_E_SHAPE;
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

template <typename T, bool ZOH, bool SC>
int launch_scan(const ScanParams &p, int64_t blocks, void *stream) {
    const dim3 grid((unsigned)blocks, (unsigned)((p.dim + 63) / 64));
    if (p.seg) {
        int rc = enqueue(scan_packed<T, ZOH, false, SC>, grid, dim3(64), p, stream);
        if (rc == SELSCAN_OK)
            rc = enqueue(scan_join, dim3((unsigned)p.q.nseq, (unsigned)((p.dim * kN + 255) / 256)), dim3(256), p, stream);
        if (rc != SELSCAN_OK) return rc;
    }
    return enqueue(scan_packed<T, ZOH, true, SC>, grid, dim3(64), p, stream);
}

template <typename T>
int launch_scan_io(const ScanParams &p, int64_t blocks, bool zoh, void *stream) {
    // scalar loads of B and C need their rows on 4-byte boundaries
    const bool sc = sizeof(T) == 4 || (p.bc_stride % 2 == 0 && aligned(p.B, 4) && aligned(p.C, 4));
    if (zoh) return sc ? launch_scan<T, true, true>(p, blocks, stream) : launch_scan<T, true, false>(p, blocks, stream);
    return sc ? launch_scan<T, false, true>(p, blocks, stream) : launch_scan<T, false, false>(p, blocks, stream);
}

// rows that a thread of a step kernel takes one after another: one while the launch has fewer than
// four workgroups of 256 threads per compute unit, up to 8 (then A and the filters are read an eighth as often)
int step_rows(int64_t rows, int64_t threads_per_row) {
    const int64_t full = 256 * 4 * 256;
    int64_t n = rows * threads_per_row / full;
    return n < 1 ? 1 : n > 8 ? 8 : (int)n;
}

constexpr int64_t kGridY = 65535;

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
    const dim3 grid((unsigned)segments(tokens, nseq, kConvShift), (unsigned)((groups + block - 1) / block));
    if (grid.y > kGridY) return SELSCAN_E_UNSUPPORTED;
    void (*k)(ConvParams) = nullptr;
#define PICK(T) (width == 1 ? conv_packed<T, 1> : width == 2 ? conv_packed<T, 2> : width == 3 ? conv_packed<T, 3> : conv_packed<T, 4>)
    k = io_dtype == SELSCAN_BF16 ? PICK(uint16_t) : PICK(float);
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
    if (tokens <= 0 || nseq <= 0 || max_seqlen <= 0 || dim <= 0 || dstate != kN || tokens > INT32_MAX || nseq > INT32_MAX / 2 ||
        dim > INT32_MAX)
        return 0;
    return packed_workspace(tokens, nseq, max_seqlen, dim);
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
    int64_t blocks = nseq;
    if (need) {
        p.shift = split_shift(tokens, nseq, max_seqlen, dim);
        blocks = segments(tokens, nseq, p.shift);
        p.seg = (float *)workspace;
        p.sdt = p.seg + blocks * dim * kN;
    }
    if ((dim * kN + 255) / 256 > kGridY) return SELSCAN_E_UNSUPPORTED;
    const bool zoh = (flags & SELSCAN_FLAG_ZOH) != 0;
    return io_dtype == SELSCAN_BF16 ? launch_scan_io<uint16_t>(p, blocks, zoh, stream)
                                    : launch_scan_io<float>(p, blocks, zoh, stream);
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
    const bool zoh = (flags & SELSCAN_FLAG_ZOH) != 0;
    void (*k)(ScanParams) = nullptr;
    if (io_dtype == SELSCAN_BF16) k = zoh ? scan_step<uint16_t, true> : scan_step<uint16_t, false>;
    else k = zoh ? scan_step<float, true> : scan_step<float, false>;
    return enqueue(k, grid, dim3(256), p, stream);
}

}  // extern "C"
