// libselscan_lm - linear attention with a decay for each head, on packed prompts and on single tokens, with states in a
// cache (linear_attn_packed_fwd, linear_attn_step of include/selscan_lm.h).  MI355X (gfx950).
#include "lm_packed.h"

namespace {

constexpr int kMaxKeys = 256, kMaxValues = 1024;

// 2^x for what multiplies the state before a segment: (hi + lo) 2^n, n of 0 unless x is above kWhole
struct alignas(16) Factor {
    float hi, lo;
    int n;
};

struct LaParams {
    const void *q, *k, *v;
    const float *decay;
    float *state;
    void *out;
    Seqs s;
    int64_t q_stride, k_stride, v_stride, decay_stride;
    int heads, share, dk, dv, vblocks;  // share: heads of a group
    int round;  // whole sequences are dealt out longest first (64: a round of all), or (0) as they come
    float scale;
    // sequences in segments of `size` tokens: what each entry holds (the state at the end of a segment that another
    // follows, from zero but for a sequence's first), and what its decays make of a state before it
    float *seg;    // [entries][heads][dk][dv]
    Factor *factor; // [entries][heads]
    int size, entries;
    FastDiv dsize;
};

// A log decay as it is used: one of -infinity, or below any whose exponential is not 0 in fp32, is a number of which a
// chunk's worth can be added and subtracted again; so is one of infinity.
__device__ __forceinline__ float finite_decay(float g) { return g < -16384.f ? -16384.f : g > 16384.f ? 16384.f : g; }

// Exponents (base 2) up to which a power is formed whole.  Powers beyond are 2^(x - n) 2^n with n = floor(x), and what is multiplied
// takes the two one after another: a state of zero stays zero, and a small one comes out as the number that it grows to.  (Half of
// what fp32 holds: the power is multiplied by values and keys before the sums.)
constexpr float kWhole = 64.f;
constexpr double kLog2e64 = 1.44269504088896340735992468100;
// the power of a segment's sum (one past 2^20 counts as 2^20: zero alone survives it)
__device__ __forceinline__ Factor factor_of(double x) {
    const int n = x > (double)kWhole ? __double2int_rd(x < 1048576. ? x : 1048576.) : 0;
    const double f = exp2(n ? x < 1048576. ? x - n : 0. : x);
    const float hi = (float)f;
    return {hi, (float)(f - (double)hi), n};
}

typedef float F4 __attribute__((ext_vector_type(4)));
typedef __bf16 B8 __attribute__((ext_vector_type(8)));
typedef short I4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ F4 mma(B8 a, B8 b, F4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ F4 mma(float a, float b, F4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// Waits out the longest of these products (16 passes of 4 clocks at most), for results that another block reads: the compiler
// counts the clocks between a product and its reader along one path of those that join, not along the shortest.
__device__ __forceinline__ void results_ready() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15");
    __builtin_amdgcn_sched_barrier(0);
}

// 4 x 16 bf16 of LDS, one row of 4 adjacent columns from each lane's address (16 lanes: 4 rows of 4 such pieces), transposed:
// lane i of 16 gets column i's 4 rows
__device__ __forceinline__ I4 read_transposed(const uint16_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) I4 *)p);
}
__device__ __forceinline__ B8 join8(I4 a, I4 b) {
    struct {
        I4 a, b;
    } u = {a, b};
    return __builtin_bit_cast(B8, u);
}
__device__ __forceinline__ B8 pack8(const F4 &a, const F4 &b) {
    const uint4 w = {Io<uint16_t>::to2(a[0], a[1]), Io<uint16_t>::to2(a[2], a[3]), Io<uint16_t>::to2(b[0], b[1]), Io<uint16_t>::to2(b[2], b[3])};
    return __builtin_bit_cast(B8, w);
}

// Eight numbers as bf16 that are exact in their bits (rounded towards zero, so that none becomes infinite) and bf16 of what is left:
// together they are off by 2^-15 of a number at most, where bf16 alone is by 2^-8.
struct Parts {
    B8 hi, lo;
};
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float left_over(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ Parts split8(const F4 &a, const F4 &b) {
    const uint4 w = {high_halves(a[0], a[1]), high_halves(a[2], a[3]), high_halves(b[0], b[1]), high_halves(b[2], b[3])};
    const F4 la = {left_over(a[0]), left_over(a[1]), left_over(a[2]), left_over(a[3])};
    const F4 lb = {left_over(b[0]), left_over(b[1]), left_over(b[2]), left_over(b[3])};
    return {__builtin_bit_cast(B8, w), pack8(la, lb)};
}

// A chunk of C tokens of one head, with G_t the sum of the log decays up to token t and S the state before it:
//     out_t = scale (e^{G_t} q_t S + sum_{j <= t} e^{G_t - G_j} (q_t . k_j) v_j),
//     S' = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// as products of matrices on the matrix cores.  A workgroup of four waves has 64 columns of the head's values; a wave keeps the 16
// columns of S that are its own in registers from chunk to chunk, in the places in which the matrix cores leave a result.
// bf16: these places are also those of an operand, if of the 32 rows of a step two tiles hold rows 8 g .. 8 g + 3 and 8 g + 4 .. 8 g +
// 7 in lanes 16 g .. 16 g + 15.  So S never leaves the registers: row_of says which row a place is.
// bf16: q, k and v go in as they are; scores and S, which are sums in 32 bits, in two parts, and what is added to S in three (the
// outputs of one 24-prompt batch were 0.0023 of their size off with scores and S rounded to one, where rounding the output alone is 0.0017).
template <typename T, int KB>
struct Chunk {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int C = BF ? 64 : 32, NT = C / 16;  // tokens, and tiles of 16 of them
    static constexpr int D = 32 * KB;                               // rows of the state, padded
    static constexpr int E = 16 / sizeof(T);                        // elements of 16 bytes
    // Row strides in LDS: rows start at different banks, for 16 rows of 16 bytes and (bf16) for 4 rows of 4 pieces 16 bytes apart
    static constexpr int LQ = BF ? D + (KB >= 4 ? 40 : 8) : D + 4, LV = 64 + E, LP = C + E;
    static constexpr int NQ = C * D / E / 256, NV = C * 64 / E / 256;  // 16-byte pieces of a thread
    T q[C * LQ], k[C * LQ], v[C * LV], p[C * LP], pl[BF ? C * LP : 1];  // (pl: the second parts of p)
    struct alignas(16) Decay {
        float gh[C], gl[C], w[C];  // G_t (base 2) in two parts; 2^(G_C - G_t)
        float fh, fl;              // 2^G_C in two parts
        int grows;                 // decays above 0 add up to more than kWhole: token t's power is gh[t] 2^gl[t]
    } decay[2];                    // of this chunk and the next
    // row of the state that register r of tile d has in lanes 16 g .. 16 g + 15
    static __device__ __forceinline__ int row_of(int d, int g, int r) {
        return BF ? 32 * (d >> 1) + 8 * g + 4 * (d & 1) + r : 16 * d + 4 * g + r;
    }
};

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Piece16 {
    uint32_t w[4];
};
// elements [at, at + E) of a row of n, zeros past its end
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T *row, int at, int n) {
    constexpr int E = 16 / sizeof(T);
    if (at + E <= n) {
        const Piece16<T> a = *(const Piece16<T> *)(row + at);
        return make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (at + e >= n) continue;
        if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(row[at + e]);
        else w[e >> 1] |= (uint32_t)row[at + e] << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Reads and writes of up to 64 rows through a buffer descriptor: what lies past the end of the last row reads as zeros and is not
// written, so that the rows of a short chunk need no branch.  kNowhere: an offset that no buffer reaches.
constexpr uint32_t kNowhere = 0x80000000u;
typedef unsigned int U4 __attribute__((ext_vector_type(4)));
typedef unsigned int U2 __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const T *at, int rows, int64_t stride, int width) {
    const uint32_t bytes = rows > 0 ? (uint32_t)(((rows - 1) * stride + width) * sizeof(T)) : 0u;
    return __builtin_amdgcn_make_buffer_rsrc((void *)at, 0, bytes, 0x00027000);
}

// What a workgroup does: `n` tokens from row t0 on, outputs or only the state.
struct LaPiece {
    int t0, n;
    bool outputs;
};

// VEC: the heads' rows are whole 16-byte pieces that start at words.
template <typename T, int KB, bool VEC>
__device__ __forceinline__ void la_piece(const LaParams &p, const LaPiece &w, Chunk<T, KB> &m, int h, int c0, F4 (&S)[2 * KB],
                                         double *total) {
    typedef Chunk<T, KB> M;
    constexpr int C = M::C, NT = M::NT, E = M::E, PQ = M::D / E, PV = 64 / E, PAIRS = (NT * (NT + 1) / 2 + 3) / 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane & 15, g = lane >> 4;
    const int group = h / p.share;
    const float scale = p.scale;  // (read in the loop, the compiler keeps it and its neighbours in memory)
    const T *q = (const T *)p.q + w.t0 * p.q_stride + (int64_t)group * p.dk;
    const T *k = (const T *)p.k + w.t0 * p.k_stride + (int64_t)group * p.dk;
    const T *v = (const T *)p.v + w.t0 * p.v_stride + (int64_t)h * p.dv + c0;
    const float *decay = p.decay + w.t0 * p.decay_stride + h;
    const int64_t out_stride = (int64_t)p.heads * p.dv;
    T *out = (T *)p.out + w.t0 * out_stride + (int64_t)h * p.dv + c0;
    const int nv = p.dv - c0 < 64 ? p.dv - c0 : 64;
    uint4 qr[M::NQ], kr[M::NQ], vr[M::NV];
    float gr = 0.f;
    const auto fetch = [&](int first) {
        const int rows = w.n - first < C ? w.n - first : C;
        const T *q1 = q + first * p.q_stride, *k1 = k + first * p.k_stride, *v1 = v + first * p.v_stride;
        if constexpr (VEC) {
            const __amdgpu_buffer_rsrc_t qb = rows_buffer(q1, rows, p.q_stride, p.dk), kb = rows_buffer(k1, rows, p.k_stride, p.dk),
                                         vb = rows_buffer(v1, rows, p.v_stride, nv);
#pragma unroll
            for (int i = 0; i < M::NQ; ++i) {
                const int r = (tid + 256 * i) / PQ, c = tid % PQ * E;  // (256 is whole rows)
                const uint32_t qa = c < p.dk ? (uint32_t)(r * (int)p.q_stride + c) * sizeof(T) : kNowhere;
                const uint32_t ka = c < p.dk ? (uint32_t)(r * (int)p.k_stride + c) * sizeof(T) : kNowhere;
                if (w.outputs) qr[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(qb, qa, 0, 0));
                kr[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(kb, ka, 0, 0));
            }
#pragma unroll
            for (int i = 0; i < M::NV; ++i) {
                const int r = (tid + 256 * i) / PV, c = tid % PV * E;
                const uint32_t va = c < nv ? (uint32_t)(r * (int)p.v_stride + c) * sizeof(T) : kNowhere;
                vr[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(vb, va, 0, 0));
            }
        } else {
#pragma unroll
            for (int i = 0; i < M::NQ; ++i) {
                const int r = (tid + 256 * i) / PQ, c = tid % PQ * E;
                const bool on = r < rows && c < p.dk;
                if (w.outputs) qr[i] = on ? load_piece(q1 + r * p.q_stride, c, p.dk) : make_uint4(0, 0, 0, 0);
                kr[i] = on ? load_piece(k1 + r * p.k_stride, c, p.dk) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < M::NV; ++i) {
                const int r = (tid + 256 * i) / PV, c = tid % PV * E;
                vr[i] = r < rows && c < nv ? load_piece(v1 + r * p.v_stride, c, nv) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    // The last wave, which has the fewest tiles of the scores, sums the decays, a chunk ahead.
    const bool sums = wave == 3;
    const auto fetch_decay = [&](int first) { gr = lane < C && first + lane < w.n ? decay[(first + lane) * p.decay_stride] : 0.f; };
    double sum = 0.;
    const auto sum_decays = [&](typename M::Decay &to) {
        // sums of up to 64 x 16384 whose differences count: 64 bits, then two parts of 32
        double G = (double)finite_decay(gr) * kLog2e64;
        G += dpp_or_zero<0x111, 0xF>(G);
        G += dpp_or_zero<0x112, 0xF>(G);
        G += dpp_or_zero<0x114, 0xF>(G);
        G += dpp_or_zero<0x118, 0xF>(G);
        G += dpp_or_zero<0x142, 0xA>(G);
        G += dpp_or_zero<0x143, 0xC>(G);
        const int64_t b = __double_as_longlong(G);
        const double all = __longlong_as_double((int64_t)__builtin_amdgcn_readlane((int)(b >> 32), 63) << 32 |
                                                (uint32_t)__builtin_amdgcn_readlane((int)b, 63));
        sum += all;
        bool grows = false;
        if (__any(gr > 0.f)) {
            float up = gr > 0.f ? finite_decay(gr) * kLog2e : 0.f;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) up += __shfl_xor(up, d);
            grows = up > kWhole;
        }
        if (lane == 0) to.grows = grows;
        if (grows) {
            const double one = (double)finite_decay(gr) * kLog2e64;
            const int n = __double2int_rd(one);
            if (lane < C) to.gh[lane] = __builtin_amdgcn_exp2f((float)(one - n)), to.gl[lane] = (float)n;
            return;
        }
        if (lane < C) {
            const float hi = (float)G;
            to.gh[lane] = hi, to.gl[lane] = (float)(G - (double)hi);
            to.w[lane] = __builtin_amdgcn_exp2f((float)(all - G));
        }
        const double f = exp2(all);
        if (lane == 0) to.fh = (float)f, to.fl = (float)(f - (double)(float)f);
    };
    // tiles of the scores that are this wave's: pair i is key tile jt and query tile tt, jt <= tt
    const auto pair_of = [&](int i, int &jt, int &tt) {
        const int at = wave + 4 * i;
        tt = 0;
#pragma unroll
        for (int t = 1; t < NT; ++t) tt = at >= t * (t + 1) / 2 ? t : tt;
        jt = at - tt * (tt + 1) / 2;
        return at < NT * (NT + 1) / 2;
    };
    const int vrow = 8 * g + (l >> 2), vcol = 16 * wave + 4 * (l & 3);  // of a transposed read
    if (w.n > 0) {
        fetch(0);
        if (sums) {
            fetch_decay(0);
            sum_decays(m.decay[0]);
            fetch_decay(C);
        }
    }
    int now = 0;  // which of the two decays
    for (int first = 0; first < w.n; first += C, now ^= 1) {
        const typename M::Decay &dc = m.decay[now];
        lds_barrier();  // the chunk before is no longer read
        const int grows = dc.grows;
        T *to = m.k + tid / PQ * M::LQ + tid % PQ * E, *qto = m.q + tid / PQ * M::LQ + tid % PQ * E;
#pragma unroll
        for (int i = 0; i < M::NQ; ++i) {
            if (w.outputs) *(uint4 *)(qto + i * (256 / PQ) * M::LQ) = qr[i];
            *(uint4 *)(to + i * (256 / PQ) * M::LQ) = kr[i];
        }
#pragma unroll
        for (int i = 0; i < M::NV; ++i) *(uint4 *)(m.v + (tid / PV + i * (256 / PV)) * M::LV + tid % PV * E) = vr[i];
        if (first + C < w.n) fetch(first + C);
        lds_barrier();
        if (sums && first + C < w.n) {
            sum_decays(m.decay[now ^ 1]);
            fetch_decay(first + 2 * C);
        }
        if (__builtin_amdgcn_readfirstlane(grows)) {
            // Powers that products would not take: the recurrence, a token after another.  A lane has its column's rows, the four
            // lanes of a column add up their parts of the output.
            int self = lane;  // (known here alone: what is formed from it would take registers of the other path)
            asm volatile("" : "+v"(self));
            const int rows = w.n - first < C ? w.n - first : C, c = 16 * wave + (self & 15), g = self >> 4;
            T *oto = out + first * out_stride + c;
#pragma unroll 1
            for (int t = 0; t < rows; ++t) {
                const float e = dc.gh[t], x = Io<T>::f32(m.v[t * M::LV + c]);
                const int n = (int)dc.gl[t];
                float o = 0.f;
#pragma unroll
                for (int d = 0; d < 2 * KB; ++d) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = M::row_of(d, g, r);
                        S[d][r] = fmaf(ldexpf(S[d][r], n), e, Io<T>::f32(m.k[t * M::LQ + row]) * x);
                        if (w.outputs) o = fmaf(Io<T>::f32(m.q[t * M::LQ + row]), S[d][r], o);
                    }
                    // (four rows at a time, each kept where it was: the other registers hold the next chunk; without it up to 47 of a
                    // wave's went to memory at every chunk of the other path)
                    if constexpr (KB == 8) asm volatile("" : "+a"(S[d]));
                    else asm volatile("" : "+v"(S[d]));
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (!w.outputs) continue;
                o += __shfl_xor(o, 16);
                o += __shfl_xor(o, 32);
                if (g == 0 && c < nv) oto[t * out_stride] = Io<T>::to(o * scale);
            }
            continue;
        }
        if (w.outputs) {
            // scores, keys down, so that a lane's four are adjacent in a row of p
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                int jt, tt;
                if (pair_of(i, jt, tt) || 4 * (i + 1) <= NT * (NT + 1) / 2) {
                    const T *kp = m.k + (16 * jt + l) * M::LQ, *qp = m.q + (16 * tt + l) * M::LQ;
                    F4 acc = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (M::BF) {
#pragma unroll
                        for (int s = 0; s < KB; ++s) acc = mma(*(const B8 *)(kp + 32 * s + 8 * g), *(const B8 *)(qp + 32 * s + 8 * g), acc);
                    } else {
#pragma unroll
                        for (int d = 0; d < 2 * KB; ++d) {
                            const F4 a = *(const F4 *)(kp + 16 * d + 4 * g), b = *(const F4 *)(qp + 16 * d + 4 * g);
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc = mma(a[r], b[r], acc);
                        }
                    }
                    const int t = 16 * tt + l, j = 16 * jt + 4 * g;
                    const float th = dc.gh[t], tl = dc.gl[t];
                    const F4 jh = *(const F4 *)(dc.gh + j), jl = *(const F4 *)(dc.gl + j);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = __builtin_amdgcn_exp2f((th - jh[r]) + (tl - jl[r]));
                        acc[r] = j + r <= t ? acc[r] * e : 0.f;
                    }
                    T *pto = m.p + t * M::LP + j;
                    if constexpr (M::BF) {
                        T *plto = m.pl + t * M::LP + j;
                        *(uint2 *)pto = make_uint2(high_halves(acc[0], acc[1]), high_halves(acc[2], acc[3]));
                        *(uint2 *)plto = make_uint2(Io<T>::to2(left_over(acc[0]), left_over(acc[1])), Io<T>::to2(left_over(acc[2]), left_over(acc[3])));
                        if (jt == tt && !(tt & 1)) *(uint2 *)(pto + 16) = *(uint2 *)(plto + 16) = make_uint2(0, 0);  // the other half of a step of 32
                    } else {
                        *(F4 *)pto = acc;
                    }
                }
            }
        }
        // this wave's columns of the values: lane l has column l; bf16: 8 rows (tokens) of each step of 32, fp32: 4 of each 16
        B8 vf[M::BF ? C / 32 : 1];
        float vx[M::BF ? 1 : NT][4];
        const auto read_values = [&] {
            if constexpr (M::BF) {
#pragma unroll
                for (int s = 0; s < C / 32; ++s)
                    vf[s] = join8(read_transposed(m.v + (32 * s + vrow) * M::LV + vcol), read_transposed(m.v + (32 * s + vrow + 4) * M::LV + vcol));
            } else {
#pragma unroll
                for (int s = 0; s < NT; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) vx[s][r] = m.v[(16 * s + 4 * g + r) * M::LV + 16 * wave + l];
            }
        };
        if (w.outputs) {
            read_values();
            // A score of 0 (a later token's) times a value that is no number would reach the tokens before it: such values
            // are taken out of the product and added one by one.
            bool odd;
            if constexpr (M::BF) {
                typedef unsigned short H2 __attribute__((ext_vector_type(2)));
                H2 most = {0, 0};
#pragma unroll
                for (int s = 0; s < C / 32; ++s) {
                    const U4 b = __builtin_bit_cast(U4, vf[s]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(H2, b[i] & 0x7FFF7FFFu));
                }
                odd = __any(most.x >= 0x7F80 || most.y >= 0x7F80);
            } else {
                float z = 0.f;
#pragma unroll
                for (int i = 0; i < C / 4; ++i) z = fmaf(vx[i >> 2][i & 3], 0.f, z);
                odd = __any(z != z);
            }
            if (odd) {
                if constexpr (M::BF) {
#pragma unroll
                    for (int i = 0; i < C / 4; ++i)
                        if (!(fabsf((float)vf[i >> 3][i & 7]) < INFINITY)) vf[i >> 3][i & 7] = (__bf16)0.f;
                } else {
#pragma unroll
                    for (int i = 0; i < C / 4; ++i)
                        if (!(fabsf(vx[i >> 2][i & 3]) < INFINITY)) vx[i >> 2][i & 3] = 0.f;
                }
            }
            // (all tiles side by side and before the next branch: their products do not wait for one another, and a result of the
            // matrix cores is read in the block that makes it.  bf16: what a step's products read is on its way during the last
            // step's, which the compiler does not do by itself: four prompts of 1,024 tokens x 24 heads of 64 x 64 44 us for 51.)
            F4 o[NT];
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) o[tt] = (F4){0.f, 0.f, 0.f, 0.f};
            if constexpr (M::BF) {
                B8 qb[2][NT];
                const auto read_q = [&](int s) {
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt) qb[s & 1][tt] = *(const B8 *)(m.q + (16 * tt + l) * M::LQ + 32 * s + 8 * g);
                };
                read_q(0);
#pragma unroll
                for (int s = 0; s < KB; ++s) {
                    if (s + 1 < KB) read_q(s + 1);
                    const Parts a = split8(S[2 * s], S[2 * s + 1]);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt) o[tt] = mma(a.lo, qb[s & 1][tt], o[tt]);
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt) o[tt] = mma(a.hi, qb[s & 1][tt], o[tt]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            lds_barrier();  // the scores are there
            const int rows = w.n - first < C ? w.n - first : C, left = nv - 16 * wave - 4 * g;
            T *out1 = out + first * out_stride;
            const __amdgpu_buffer_rsrc_t ob = rows_buffer(out1, rows, out_stride, nv);
            if constexpr (M::BF) {
                B8 pb[2][NT];
                const auto read_p = [&](int s) {
#pragma unroll
                    for (int tt = 2 * s; tt < NT; ++tt) {
                        pb[0][tt] = *(const B8 *)(m.pl + (16 * tt + l) * M::LP + 32 * s + 8 * g);
                        pb[1][tt] = *(const B8 *)(m.p + (16 * tt + l) * M::LP + 32 * s + 8 * g);
                    }
                };
                read_p(0);
#pragma unroll
                for (int tt = 0; tt < NT; ++tt) o[tt] *= __builtin_amdgcn_exp2f(dc.gh[16 * tt + l] + dc.gl[16 * tt + l]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < C / 32; ++s) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int tt = 2 * s; tt < NT; ++tt) o[tt] = mma(vf[s], pb[i][tt], o[tt]);
                    if (s + 1 < C / 32) read_p(s + 1);
                }
            }
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                if constexpr (!M::BF) {
                    const int t = 16 * tt + l;
                    const T *pp = m.p + t * M::LP;
#pragma unroll
                    for (int d = 0; d < 2 * KB; ++d) {
                        const F4 b = *(const F4 *)(m.q + t * M::LQ + 16 * d + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[tt] = mma(S[d][r], b[r], o[tt]);
                    }
                    o[tt] *= __builtin_amdgcn_exp2f(dc.gh[t] + dc.gl[t]);
#pragma unroll
                    for (int s = 0; s <= tt; ++s) {
                        const F4 b = *(const F4 *)(pp + 16 * s + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[tt] = mma(vx[s][r], b[r], o[tt]);
                    }
                }
                o[tt] *= scale;
            }
            if (odd) {
#pragma unroll
                for (int tt = 0; tt < NT; ++tt) {
                    const int t = 16 * tt + l;
#pragma unroll 1
                    for (int j = 0; j <= t; ++j) {
                        float score = Io<T>::f32(m.p[t * M::LP + j]);
                        if constexpr (M::BF) score += Io<T>::f32(m.pl[t * M::LP + j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float x = Io<T>::f32(m.v[j * M::LV + 16 * wave + 4 * g + r]);
                            if (!(fabsf(x) < INFINITY)) o[tt][r] = fmaf(score * scale, x, o[tt][r]);
                        }
                    }
                }
            }
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                const int t = 16 * tt + l;
                if constexpr (VEC) {
                    const uint32_t at = left > 0 ? (uint32_t)(t * (int)out_stride + 16 * wave + 4 * g) * sizeof(T) : kNowhere;
                    if constexpr (M::BF)
                        __builtin_amdgcn_raw_buffer_store_b64((U2){Io<T>::to2(o[tt][0], o[tt][1]), Io<T>::to2(o[tt][2], o[tt][3])}, ob, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(U4, o[tt]), ob, at, 0, 0);
                } else if (t < rows) {
                    T *oto = out1 + t * out_stride + 16 * wave + 4 * g;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r < left) oto[r] = Io<T>::to(o[tt][r]);
                }
            }
        }
        // the state
        read_values();
        const float fh = dc.fh, fl = dc.fl;
        if constexpr (M::BF) {
            // (the rounding of a chunk's factor, 2^-25 of a state, is far below a sum's with k and v in bf16)
#pragma unroll
            for (int d = 0; d < 2 * KB; ++d) S[d] *= fh;
            // k is exact, a weighted value goes in as three bf16 parts whose sum it is
            B8 part[C / 32][3];
#pragma unroll
            for (int s = 0; s < C / 32; ++s) {
                F4 x[2] = {*(const F4 *)(dc.w + 32 * s + 8 * g), *(const F4 *)(dc.w + 32 * s + 8 * g + 4)};
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e >> 2][e & 3] *= (float)vf[s][e];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    part[s][i] = pack8(x[0], x[1]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e >> 2][e & 3] -= (float)part[s][i][e];
                }
            }
            B8 kb[2][2][C / 32];
            const auto read_k = [&](int e) {  // of tiles 2 e and 2 e + 1
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int s = 0; s < C / 32; ++s) {
                        const T *kp = m.k + (32 * s + vrow) * M::LQ + 8 * (l & 3) + 32 * e + 4 * d;
                        kb[e & 1][d][s] = join8(read_transposed(kp), read_transposed(kp + 4 * M::LQ));
                    }
            };
            read_k(0);
#pragma unroll
            for (int e = 0; e < KB; ++e) {
                if (e + 1 < KB) read_k(e + 1);
#pragma unroll
                for (int s = 0; s < C / 32; ++s)
#pragma unroll
                    for (int i = 2; i >= 0; --i)
#pragma unroll
                        for (int d = 0; d < 2; ++d) S[2 * e + d] = mma(kb[e & 1][d][s], part[s][i], S[2 * e + d]);
            }
        } else {
#pragma unroll
            for (int d = 0; d < 2 * KB; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[d][r] = fmaf(S[d][r], fh, S[d][r] * fl);
#pragma unroll
            for (int s = 0; s < NT; ++s) {
                const F4 x = *(const F4 *)(dc.w + 16 * s + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) vx[s][r] *= x[r];
            }
#pragma unroll
            for (int d = 0; d < 2 * KB; ++d)
#pragma unroll
                for (int s = 0; s < NT; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[d] = mma(m.k[(16 * s + 4 * g + r) * M::LQ + 16 * d + l], vx[s][r], S[d]);
        }
        results_ready();
    }
    *total = sum;
}

// Packed prompts.  A workgroup has 64 columns of a head's values and a whole sequence or one of its segments.  Segments take
// two launches: the first (LAUNCH 0) reads sequences of one segment for good, and of the others what each segment that a further
// one follows makes of the sequence's first state or of a state of zero; the states are joined; the second (LAUNCH 1) reads
// the others' segments from the states that they start from.  (Outputs of every first segment in the first launch make that
// launch as long as the second: 4,097 tokens x 24 heads of 64 x 64 fp32 take 60 us, and took 70.)
// What bounds it: where sequences are few, the chunks of the longest one after another, 64 tokens in 2.6 us (bf16, 64 x 64; four
// waves in one compute unit, each with its own chain of reads, products and exponentials) or 3.4 us (128 x 64).  Where they fill the
// chip, what a chunk costs: 27,591 tokens of 24 prompts x 64 heads of 128 x 64 bf16 are 28,224 chunks, two at a time on each of 256 compute
// units and 5.0 us then, so 277 us if they are even; 271 to 286 are measured, 2.0 TB/s of what has to pass.  A wave has some 520
// vector instructions, 102 products and 120 accesses of LDS to a chunk; LDS is busy for 58 % of the clocks, the vector units for 46 %.
// Other paddings of LDS and priorities of waves change nothing (270 to 275).  Before scores and states had two parts (258): two
// 64-column pieces or two heads in a workgroup of eight waves 302 us, 32 columns per wave 409 (fewer waves, each with longer
// chains), chunks of 32 tokens 281, and segments of 512, 1,024 or 2,048 tokens slower than whole sequences longest first.  fp32
// chunks are of 32 tokens: 31 KB of LDS at 64 keys, five workgroups to a compute unit, where 64 tokens take 70 KB and allow two.
template <typename T, int KB, bool VEC, int LAUNCH>
__global__ __launch_bounds__(256, KB <= 4 ? 2 : 1) void la_packed(LaParams p) {
    typedef Chunk<T, KB> M;
    __shared__ __attribute__((aligned(16))) M m;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15, gq = lane >> 4;
    const int vb = blockIdx.x % p.vblocks, hs = blockIdx.x / p.vblocks, h = hs % p.heads, seg = hs / p.heads;
    const bool split = p.seg != nullptr;
    const Segment g = split ? find_segment(p.s, seg, [&](int v) { return (int)fdiv((uint32_t)v, p.dsize); }, lane) : p.round ? dealt_sequence(p.s, seg, p.round, lane) : whole_sequence(p.s, seg);
    const int first = split ? g.j * p.size : 0;
    if (g.j < 0 || (g.j > 0 && first >= g.len)) return;
    const bool last = !split || g.len - first <= p.size, only = last && g.j == 0;
    const int c0 = vb * 64, c = c0 + 16 * wave + l;
    const int64_t head = (int64_t)p.dk * p.dv;
    float *cache = p.state && g.slot >= 0 ? p.state + ((int64_t)g.slot * p.heads + h) * head : nullptr;
    const int64_t entry = (int64_t)(seg - g.s) * p.heads + h;  // of this segment
    const float *from = g.j == 0 ? g.carry ? cache : nullptr : LAUNCH == 1 ? p.seg + (entry - p.heads) * head : nullptr;
    // (a first segment that starts from the cache is read for good before the launch whose last segment writes there)
    const bool early = only || (g.j == 0 && from);
    if (LAUNCH == 0 ? last && !only : early) return;
    F4 S[2 * KB];
#pragma unroll
    for (int d = 0; d < 2 * KB; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = M::row_of(d, gq, r);
            S[d][r] = from && c < p.dv && row < p.dk ? from[row * p.dv + c] : 0.f;
        }
    double total;
    // (the same in all lanes, for the buffers' descriptors)
    const int t0 = __builtin_amdgcn_readfirstlane(g.t0 + first), n = __builtin_amdgcn_readfirstlane(last ? g.len - first : p.size);
    la_piece<T, KB, VEC>(p, {t0, n, LAUNCH == 1 || early}, m, h, c0, S, &total);
    float *to = last ? cache : nullptr;
    if (LAUNCH == 0 && !last) {
        to = p.seg + entry * head;
        if (threadIdx.x == 192 && vb == 0) p.factor[entry] = factor_of(total);  // (of the wave that sums the decays)
    }
    if (!to || c >= p.dv) return;
#pragma unroll
    for (int d = 0; d < 2 * KB; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = M::row_of(d, gq, r);
            if (row < p.dk) to[row * p.dv + c] = S[d][r];
        }
}

// Between the launches: a thread per number of a head's state walks the entries of a sequence in order and leaves the state at
// the end of each segment in its place.  Sequences are dealt out by their numbers, or, where there are more of them than
// entries, by those entries that are their first.
__global__ __launch_bounds__(64) void la_join(LaParams p) {
    const int64_t head = (int64_t)p.dk * p.dv, entry = p.heads * head, i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const bool live = i < entry, by_entry = p.s.nseq > p.entries;
    const int h = (int)((live ? i : 0) / head);
    const auto div = [&](int v) { return (int)fdiv((uint32_t)v, p.dsize); };
    for (int b = blockIdx.y; b < (by_entry ? p.entries : p.s.nseq); b += gridDim.y) {
        Range rg;
        if (by_entry) {
            const Segment g = find_segment<true>(p.s, b, div, threadIdx.x);
            if (g.j != 1) continue;  // not its sequence's first
            rg = {g.t0, g.len};
        } else {
            rg = range_of(p.s, b);
        }
        const int n = rg.len > 0 ? div(rg.len - 1) : 0;  // all but the last
        if (n < 2 || !live) continue;
        const int64_t first = div(rg.t0);
        float *e = p.seg + first * entry + i;
        const Factor *t = p.factor + first * p.heads + h;
        float S = e[0];
        constexpr int U = 16;  // loaded ahead
        for (int j0 = 1; j0 < n; j0 += U) {
            float ev[U];
            Factor tv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t j = j0 + u < n ? j0 + u : n - 1;
                ev[u] = e[j * entry], tv[u] = t[j * p.heads];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j0 + u >= n) break;
                S = ldexpf(S, tv[u].n);
                S = fmaf(S, tv[u].hi, fmaf(S, tv[u].lo, ev[u]));
                e[(j0 + u) * entry] = S;
            }
        }
    }
}

// One token per sequence: S' = e^g S + k v^T, out = scale q^T S'.  The state is read and written once, and that bounds it: 4 x CG
// columns of a head's state in a workgroup, CG lanes side by side in a row of it, ND rows in each thread, all of them in flight at
// once.  128 rows x 64 heads of 128 x 64 (fp32 states of 268 MB): 96 us in a trace, 5.6 TB/s, where a copy of 1 GiB reaches 5.1; 110
// between calls on other states, 88 on the same ones again and again.  A decay near 1 is taken
// as S + (e^g - 1) S: rounded to 24 bits itself, it would be off in the same direction at every step.
template <typename T, int CG, int ND, bool VEC, bool PAST>
__global__ __launch_bounds__(256) void la_step(LaParams p) {
    __shared__ float4 part[4][CG];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cg = lane % CG;
    const int vb = blockIdx.x % p.vblocks, hs = blockIdx.x / p.vblocks, h = hs % p.heads;
    const int row = hs / p.heads;
    const int64_t slot = slot_of(p.s, row);
    const int c = (vb * CG + cg) * 4, nc = p.dv - c < 4 ? p.dv - c : 4;
    const int d0 = (threadIdx.x / CG) * ND;
    float *cache = p.state + ((slot < 0 ? 0 : slot) * p.heads + h) * p.dk * p.dv + c;
    const T *q = (const T *)p.q + row * p.q_stride + (int64_t)(h / p.share) * p.dk;
    const T *k = (const T *)p.k + row * p.k_stride + (int64_t)(h / p.share) * p.dk;
    const T *v = (const T *)p.v + row * p.v_stride + (int64_t)h * p.dv + c;
    float S[ND][4], kv[ND], qv[ND], x[4];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        const bool on = d0 + i < p.dk && slot >= 0;
        const float *at = cache + (int64_t)(d0 + i) * p.dv;
        if constexpr (VEC) {
            F4 w = {0.f, 0.f, 0.f, 0.f};
            if (on && nc > 0) w = *(const F4 *)at;
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = on && j < nc ? at[j] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        kv[i] = d0 + i < p.dk ? Io<T>::f32(k[d0 + i]) : 0.f;
        qv[i] = d0 + i < p.dk ? Io<T>::f32(q[d0 + i]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = j < nc ? Io<T>::f32(v[j]) : 0.f;
    const float decay = finite_decay(p.decay[row * p.decay_stride + h]);
    const bool slow = fabsf(decay) < 0.5f;
    float e = slow ? expm1f(decay) : __builtin_amdgcn_exp2f(decay * kLog2e);
    if (decay >= 0.5f) {  // growth: the power in two parts, as in a chunk that grows
        const double G = (double)decay * kLog2e64;
        const int n = __double2int_rd(G);
        e = __builtin_amdgcn_exp2f((float)(G - n));
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = ldexpf(S[i][j], n);
    }
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ND; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float kx = slow ? fmaf(kv[i], x[j], S[i][j]) : kv[i] * x[j];
            S[i][j] = fmaf(e, S[i][j], kx);
            o[j] = fmaf(qv[i], S[i][j], o[j]);
        }
        if (d0 + i < p.dk && slot >= 0) {
            float *at = cache + (int64_t)(d0 + i) * p.dv;
            if constexpr (VEC) {
                const F4 w = {S[i][0], S[i][1], S[i][2], S[i][3]};
                if (nc > 0) {
                    if constexpr (PAST) __builtin_nontemporal_store(w, (F4 *)at);
                    else *(F4 *)at = w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nc) at[j] = S[i][j];
            }
        }
    }
#pragma unroll
    for (int m = CG; m < 64; m *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], m);
    if (lane < CG) part[wave][cg] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (threadIdx.x >= CG) return;
    T *out = (T *)p.out + ((int64_t)row * p.heads + h) * p.dv + c;
    const float4 a = part[0][cg], b = part[1][cg], e2 = part[2][cg], f = part[3][cg];
    const float s[4] = {a.x + b.x + e2.x + f.x, a.y + b.y + e2.y + f.y, a.z + b.z + e2.z + f.z, a.w + b.w + e2.w + f.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nc) out[j] = Io<T>::to(p.scale * s[j]);
}

constexpr int64_t kMaxStride = INT64_C(1) << 23;  // 64 rows within 31 bits

struct LaArgs {
    const void *q;
    int64_t q_stride;
    const void *k;
    int64_t k_stride;
    const void *v;
    int64_t v_stride;
    const float *decay;
    int64_t decay_stride;
    float scale;
    const int32_t *cu, *slots;
    const uint8_t *carry;
    float *state;
    void *out;
    int64_t rows, nseq, nslots, heads, groups, dk, dv;
    int dtype;
    void *ws;
    size_t ws_need, ws_bytes;
    bool packed;
};

int la_check(const LaArgs &a, bool *nothing) {
    *nothing = false;
    if (a.rows < 0 || a.nseq < 0 || a.nslots < 0 || a.heads < 0 || a.groups < 0 || a.dk < 0 || a.dv < 0) return SELSCAN_E_SHAPE;
    if (!io_known(a.dtype) || !(a.scale - a.scale == 0.f)) return SELSCAN_E_UNSUPPORTED;
    if (a.rows > kMaxTokens || a.nseq > INT32_MAX / 2) return SELSCAN_E_UNSUPPORTED;
    if (a.heads == 0 || a.dv == 0 || a.nseq == 0) {
        *nothing = true;
        return a.nseq == 0 && a.rows > 0 && a.heads > 0 && a.dv > 0 ? SELSCAN_E_SHAPE : SELSCAN_OK;
    }
    if (a.groups == 0 || a.dk == 0 || a.heads % a.groups) return SELSCAN_E_SHAPE;
    if (a.dk > kMaxKeys || a.dv > kMaxValues || a.heads > kMaxStride) return SELSCAN_E_UNSUPPORTED;
    const int64_t qk = a.groups * a.dk, vw = a.heads * a.dv;
    if (a.q_stride < qk || a.k_stride < qk || a.v_stride < vw || (a.decay_stride != 0 && a.decay_stride < a.heads)) return SELSCAN_E_SHAPE;
    if (a.q_stride > kMaxStride || a.k_stride > kMaxStride || a.v_stride > kMaxStride || a.decay_stride > kMaxStride)
        return SELSCAN_E_UNSUPPORTED;
    if (a.state && !a.slots && a.nslots < a.nseq) return SELSCAN_E_SHAPE;
    const int64_t entry = vw * a.dk;  // below 2^26 * 2^8
    if (mul_size(a.nslots, entry) < 0) return SELSCAN_E_SHAPE;
    if ((a.rows > 0 && (!a.q || !a.k || !a.v || !a.decay || !a.out)) || (a.packed && !a.cu) || (!a.packed && !a.state)) return SELSCAN_E_NULL;
    const size_t s = io_bytes(a.dtype);
    const void *io[] = {a.q, a.k, a.v, a.out};
    for (const void *x : io)
        if (!span_aligned(x, s)) return SELSCAN_E_ALIGN;
    if (!span_aligned(a.decay, 4) || !span_aligned(a.cu, 4) || !span_aligned(a.slots, 4) || !span_aligned(a.state, 16) ||
        (a.ws_need && !span_aligned(a.ws, 16)))
        return SELSCAN_E_ALIGN;
    if (a.ws_need && (!a.ws || a.ws_bytes < a.ws_need)) return SELSCAN_E_WORKSPACE;
    const Span in[] = {{a.q, strided_bytes(a.rows, qk, a.q_stride, s)},
                       {a.k, strided_bytes(a.rows, qk, a.k_stride, s)},
                       {a.v, strided_bytes(a.rows, vw, a.v_stride, s)},
                       {a.decay, strided_bytes(a.rows, a.heads, a.decay_stride, 4)},
                       {a.cu, (size_t)(a.nseq + 1) * 4},
                       {a.slots, (size_t)a.nseq * 4},
                       {a.carry, (size_t)a.nseq}};
    const Span out[] = {{a.out, (size_t)a.rows * vw * s}, {a.state, (size_t)a.nslots * entry * 4}, {a.ws_need ? a.ws : nullptr, a.ws_need}};
    return any_alias(in, 7, out, 3) ? SELSCAN_E_ALIAS : SELSCAN_OK;
}

LaParams la_params(const LaArgs &a, int columns) {
    LaParams p{};
    p.q = a.q, p.k = a.k, p.v = a.v, p.decay = a.decay, p.state = a.state, p.out = a.out;
    p.s = {a.cu, a.slots, a.carry, a.nslots, (int)a.rows, (int)a.nseq};
    p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.v_stride = a.v_stride, p.decay_stride = a.decay_stride;
    p.heads = (int)a.heads, p.share = (int)(a.heads / a.groups), p.dk = (int)a.dk, p.dv = (int)a.dv;
    p.vblocks = (int)((a.dv + columns - 1) / columns), p.scale = a.scale;
    return p;
}

// Tokens per segment, or 0: whole sequences.  In chunks of 64 tokens, the longest sequence takes `whole` of them one after another,
// and all take `share` if they are even.  Measured, whole and in segments (us): bf16, 24 heads of 64 x 64, 512 tokens 24 and 24,
// 768 34 and 22, 2,048 85 and 29, four of 1,024 45 and 46, eight of 2,048 84 and 99; 64 heads of 128 x 64, 1,024 tokens 58 and
// 42, two of 2,048 113 and 109, four of 4,096 222 and 262; 16 heads of 256 x 64, 512 tokens 47 and 38, four of 1,024 91 and 84, 64 heads,
// four of 2,048 175 and 318; 24 heads of 32 x 64, four of 1,024 38 and 36, eight of 2,048 72 and 80; of 16 x 16, 768 tokens 28 and 17.
// fp32, whose chunks take longer, 24 heads of 64 x 64, 768 tokens 62 and 29, four of 1,024 82 and 56, eight of 2,048 160 and 145; 64
// heads of 128 x 64, two of 2,048 270 and 227, four of 4,096 536 and 612; 16 heads of 256 x 64, 512 tokens 126 and 67, four of
// 1,024 253 and 141, 64 heads, four of 2,048 502 and 755.  The three constants below and kSlots are fits to these.  Segments of 192
// tokens of one of 4,097 fp32: 63 us, of 128 70, of 256 70, of 384 76.
constexpr int64_t kSlots = 768;  // workgroups, three to each of 256 compute units: between what 128 keys (two) and 64 in fp32 (five) allow

int split_size(int64_t tokens, int64_t max_seqlen, int64_t heads, int64_t dv, int io) {
    const int64_t lanes = heads * ((dv + 63) / 64), longest = max_seqlen < tokens ? max_seqlen : tokens;
    const int64_t whole = (longest + 63) / 64, times = io == SELSCAN_BF16 ? 5 : 3;
    const double share = (double)tokens * (double)lanes / (double)(kSlots * 64);
    if ((double)whole <= share * times + 7.) return 0;
    const int64_t even = (int64_t)ceil(share), size = even < 2 ? 2 : even > 64 ? 64 : even;
    return 2 * size <= whole ? (int)size * 64 : 0;
}
bool la_sizes(int64_t heads, int64_t dk, int64_t dv) {
    return heads > 0 && dk > 0 && dv > 0 && dk <= kMaxKeys && dv <= kMaxValues && heads <= kMaxStride;
}
size_t factors_bytes(int64_t entries, int64_t heads) { return ((size_t)entries * heads * sizeof(Factor) + 15) / 16 * 16; }

constexpr int64_t kGridY = 65535;

template <typename T, int KB, bool VEC>
int launch_packed(const LaParams &p, int64_t blocks, void *stream) {
    int rc = enqueue(la_packed<T, KB, VEC, 0>, dim3((unsigned)blocks), dim3(256), p, stream);
    if (rc != SELSCAN_OK || !p.seg) return rc;
    const int64_t entry = (int64_t)p.heads * p.dk * p.dv, y = p.s.nseq < p.entries ? p.s.nseq : p.entries;
    rc = enqueue(la_join, dim3((unsigned)((entry + 63) / 64), (unsigned)(y < kGridY ? y : kGridY)), dim3(64), p, stream);
    if (rc != SELSCAN_OK) return rc;
    return enqueue(la_packed<T, KB, VEC, 1>, dim3((unsigned)blocks), dim3(256), p, stream);
}
template <typename T, bool VEC>
int launch_packed_keys(const LaParams &p, int64_t blocks, void *stream) {
    return p.dk <= 32    ? launch_packed<T, 1, VEC>(p, blocks, stream)
           : p.dk <= 64  ? launch_packed<T, 2, VEC>(p, blocks, stream)
           : p.dk <= 128 ? launch_packed<T, 4, VEC>(p, blocks, stream)
                         : launch_packed<T, 8, VEC>(p, blocks, stream);
}

// Bytes of states from which on they are written past the caches, of which the last holds as many: 256 MB of them are 89 us either way
// (114 and 110 where other work comes between), 400 MB 133 us for 165, 800 MB 289 for 327; 192 MB 69 for 68.  (Read past
// them too: 150 and 303.)
constexpr int64_t kPast = INT64_C(256) << 20;

template <typename T, int CG, int ND>
int launch_step(const LaParams &p, int64_t blocks, bool vec, void *stream) {
    const bool past = blocks * 4 * CG * p.dk * 4 >= kPast;
    return enqueue(!vec ? la_step<T, CG, ND, false, false> : past ? la_step<T, CG, ND, true, true> : la_step<T, CG, ND, true, false>,
                   dim3((unsigned)blocks), dim3(256), p, stream);
}

}  // namespace

extern "C" {

size_t linear_attn_packed_workspace_bytes(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t heads, int64_t dk, int64_t dv,
                                          int io_dtype) {
    if (tokens <= 0 || nseq <= 0 || max_seqlen <= 0 || tokens > kMaxTokens || nseq > INT32_MAX / 2 || !la_sizes(heads, dk, dv) || !io_known(io_dtype)) return 0;
    const int size = split_size(tokens, max_seqlen, heads, dv, io_dtype);
    if (!size) return 0;
    const int64_t entries = tokens / size;
    return factors_bytes(entries, heads) + (size_t)entries * heads * dk * dv * 4;
}

int linear_attn_packed_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const float *log_decay, int64_t decay_stride, float scale,
                           const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry, float *state, void *out,
                           int64_t tokens, int64_t nseq, int64_t nslots, int64_t max_seqlen, int64_t heads, int64_t groups,
                           int64_t dk, int64_t dv, int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (max_seqlen < 0) return SELSCAN_E_SHAPE;
    const size_t need = linear_attn_packed_workspace_bytes(tokens, nseq, max_seqlen, heads, dk, dv, io_dtype);
    const LaArgs a{q, q_stride, k, k_stride, v, v_stride, log_decay, decay_stride, scale, cu_seqlens, slots, carry, state, out,
                   tokens, nseq, nslots, heads, groups, dk, dv, io_dtype, workspace, need, workspace_bytes, true};
    bool nothing;
    const int rc = la_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    LaParams p = la_params(a, 64);
    const int64_t per = heads * p.vblocks;
    int64_t pieces = nseq;
    if (need) {
        p.size = split_size(tokens, max_seqlen, heads, dv, io_dtype);
        p.dsize = make_div((uint32_t)p.size);
        p.entries = (int)(tokens / p.size);
        pieces = tokens / p.size + nseq;
        p.factor = (Factor *)workspace;
        p.seg = (float *)((char *)workspace + factors_bytes(p.entries, heads));
    }
    // Whole sequences longest first where they take more workgroups than there are compute units (24 prompts, 27,591 tokens x 64
    // heads of 128 x 64 bf16 in rising order 388 us as they come and 282 dealt out, in three other orders 351..393 and 282; fp32 in rising
    // order 992 and 700.  With every second round of sequences in rising order, as the scan has them, 2 % slower.)
    else if (nseq > 1 && nseq <= 64 && nseq * per > 256) p.round = 64;
    if (mul_size(pieces, per) < 0 || !grid_fits(pieces * per, 256) || (need && !grid_fits(heads * dk * dv / 64 + 1, 64))) return SELSCAN_E_UNSUPPORTED;
    const int64_t e = io_dtype == SELSCAN_BF16 ? 8 : 4, word = io_dtype == SELSCAN_BF16 ? 2 : 1;
    const bool vec = dk % e == 0 && dv % e == 0 && q_stride % word == 0 && k_stride % word == 0 && v_stride % word == 0 &&
                     span_aligned(q, 4) && span_aligned(k, 4) && span_aligned(v, 4) && span_aligned(out, 4);
    if (io_dtype == SELSCAN_BF16)
        return vec ? launch_packed_keys<uint16_t, true>(p, pieces * per, stream) : launch_packed_keys<uint16_t, false>(p, pieces * per, stream);
    return vec ? launch_packed_keys<float, true>(p, pieces * per, stream) : launch_packed_keys<float, false>(p, pieces * per, stream);
}

int linear_attn_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const float *log_decay, int64_t decay_stride, float scale, const int32_t *slots, float *state,
                     void *out, int64_t rows, int64_t nslots, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                     int io_dtype, void *stream) {
    const LaArgs a{q,    q_stride, k,      k_stride, v,      v_stride, log_decay, decay_stride, scale, nullptr, slots, nullptr,
                   state, out,      rows,   rows,     nslots, heads,    groups,    dk,           dv,    io_dtype, nullptr, 0,
                   0,    false};
    bool nothing;
    const int rc = la_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    const int cg = dv > 32 ? 16 : dv > 16 ? 8 : 4;
    const LaParams p = la_params(a, 4 * cg);
    const int64_t per = heads * p.vblocks;
    if (mul_size(rows, per) < 0 || !grid_fits(rows * per, 256)) return SELSCAN_E_UNSUPPORTED;
    const int64_t blocks = rows * per;
    const bool vec = dv % 4 == 0;
    const int rowlanes = 256 / cg, nd = (int)((dk + rowlanes - 1) / rowlanes);
#define GO(CG, ND)                                                                                   \
    if (cg == CG && nd <= ND)                                                                        \
        return io_dtype == SELSCAN_BF16 ? launch_step<uint16_t, CG, ND>(p, blocks, vec, stream) : launch_step<float, CG, ND>(p, blocks, vec, stream);
    GO(16, 4) GO(16, 8) GO(16, 16) GO(8, 2) GO(8, 4) GO(8, 8) GO(4, 1) GO(4, 2) GO(4, 4)
#undef GO
    return SELSCAN_E_UNSUPPORTED;
}

}  // extern "C"
