// libselscan_lm - entries of a model's cache copied, moved and freed (cache_entries_copy of include/selscan_lm.h).
// MI355X (gfx950).
//
// A workgroup takes CW pieces of 16 bytes of an entry of one cache, and all n pairs of entries: it reads those pieces of
// every source, waits, and writes them to every destination.  No other workgroup touches these pieces, so that any set of
// moves, rings among them, needs neither an order nor a second copy of the data.  Bytes bound it: every entry is read and written once,
// 60 pairs of 2 MB in each of four layers at 5.4 TB/s (a copy of 1 GiB: 5.1); 10,000 pairs of 8 KB, whose strips are 16 bytes wide, at 1.0.
#include "lm_common.h"

namespace {

constexpr int kCaches = 128;  // caches of a launch (their addresses are kernel arguments)
constexpr int64_t kMaxPairs = 16384, kMaxEntry = INT64_C(1) << 32;

struct Cache {
    char *p;
    int64_t bytes;  // of an entry
};
struct CopyParams {
    const int32_t *src, *dst;
    int64_t nslots;
    int n, ncaches;
    uint32_t first[kCaches];  // workgroup
    Cache c[kCaches];
};

typedef uint32_t Any4 __attribute__((ext_vector_type(4), aligned(1)));

// 16 bytes or, at an entry's end, the nb < 16 that are left
__device__ __forceinline__ uint4 load_piece(const char *p, int nb) {
    if (nb >= 16) {
        const Any4 a = *(const Any4 *)p;
        return make_uint4(a[0], a[1], a[2], a[3]);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < nb) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool NT>
__device__ __forceinline__ void store_piece(char *p, int nb, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (nb >= 16) {
        const Any4 a = {w[0], w[1], w[2], w[3]};
        if constexpr (NT) __builtin_nontemporal_store(a, (Any4 *)p);
        else *(Any4 *)p = a;
        return;
    }
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < nb) p[i] = (char)(w[i >> 2] >> (8 * (i & 3)));
}

// CW pieces wide, THREADS / CW pairs side by side, NR of them in each thread; NT: written past the caches
template <int THREADS, int CW, int NR, bool NT>
__global__ __launch_bounds__(THREADS) void copy_entries(CopyParams p) {
    int lo = 0, n = p.ncaches;  // the last cache whose first workgroup is not after this one
    while (n > 1) {
        const int half = n >> 1;
        if (p.first[lo + half] <= blockIdx.x) lo += half, n -= half;
        else n = half;
    }
    const Cache c = p.c[lo];
    const int64_t at = ((int64_t)(blockIdx.x - p.first[lo]) * CW + threadIdx.x % CW) * 16;
    const int64_t left = c.bytes - at;
    const int nb = left < 0 ? 0 : left < 16 ? (int)left : 16, pair = threadIdx.x / CW;
    constexpr int PL = THREADS / CW;
    uint4 v[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int i = r * PL + pair;
        const int64_t s = i < p.n ? p.src[i] : -1;
        v[r] = s >= 0 && s < p.nslots && nb > 0 ? load_piece(c.p + s * c.bytes + at, nb) : make_uint4(0, 0, 0, 0);
    }
    // every read of the workgroup has come back before any of its writes
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int i = r * PL + pair;
        const int64_t d = i < p.n ? p.dst[i] : -1;
        if (d >= 0 && d < p.nslots && nb > 0) store_piece<NT>(c.p + d * c.bytes + at, nb, v[r]);
    }
}

}  // namespace

extern "C" int cache_entries_copy(void *const *caches, const int64_t *entry_bytes, int64_t ncaches, const int32_t *src,
                                  const int32_t *dst, int64_t n, int64_t nslots, void *stream) {
    if (ncaches < 0 || n < 0 || nslots < 0) return SELSCAN_E_SHAPE;
    if (n > kMaxPairs) return SELSCAN_E_UNSUPPORTED;
    if (ncaches == 0 || n == 0 || nslots == 0) return SELSCAN_OK;
    if (!caches || !entry_bytes || !src || !dst) return SELSCAN_E_NULL;
    if (!span_aligned(src, 4) || !span_aligned(dst, 4)) return SELSCAN_E_ALIGN;
    for (int64_t i = 0; i < ncaches; ++i) {
        if (entry_bytes[i] < 0 || mul_size(nslots, entry_bytes[i]) < 0) return SELSCAN_E_SHAPE;
        if (entry_bytes[i] > kMaxEntry) return SELSCAN_E_UNSUPPORTED;
        if (entry_bytes[i] > 0 && !caches[i]) return SELSCAN_E_NULL;
    }
    const auto span = [&](int64_t i) { return Span{caches[i], (size_t)(nslots * entry_bytes[i])}; };
    const Span s{src, (size_t)n * 4}, d{dst, (size_t)n * 4};
    for (int64_t i = 0; i < ncaches; ++i) {
        if (overlap(span(i), s) || overlap(span(i), d)) return SELSCAN_E_ALIAS;
        for (int64_t j = 0; j < i; ++j)
            if (overlap(span(i), span(j))) return SELSCAN_E_ALIAS;
    }
    // As wide as 1,024 threads leave it: 1 KB next to each other, while 4 or 8 pairs in a thread are enough.  (60 pairs of entries of 2
    // MB in 4 layers: 1,024 threads with 4 pairs each 161 us, 512 with 8 167, 256 with 16 192, 16 pieces wide and 16 pairs 221; 7 pairs
    // of small ones in 24 layers: 256 threads 8.3, 1,024 14.  Times are of the same moves again and again: the first one takes 169
    // where others come between.)  More than 16 pairs are written past the caches: what is read stays there (161 us for 181; in one
    // cache, 250 pairs of 1 MB 87 for 112, 500 of 256 KB 39 for 37); not where a row of pieces is less than a cache line (4,000 pairs
    // of 32 KB 57 us, past the caches 66, 10,000 of 8 KB 164 and 279).
    void (*kernel)(CopyParams) = copy_entries<1024, 1, 16, false>;
    int threads = 1024, cw = 1;
    if (n <= 4) kernel = copy_entries<256, 64, 1, false>, threads = 256, cw = 64;
    else if (n <= 16) kernel = copy_entries<256, 64, 4, false>, threads = 256, cw = 64;
    else if (n <= 64) kernel = copy_entries<1024, 64, 4, true>, cw = 64;
    else if (n <= 128) kernel = copy_entries<1024, 64, 8, true>, cw = 64;
    else if (n <= 256) kernel = copy_entries<1024, 32, 8, true>, cw = 32;
    else if (n <= 512) kernel = copy_entries<1024, 16, 8, true>, cw = 16;
    else if (n <= 1024) kernel = copy_entries<1024, 16, 16, true>, cw = 16;
    else if (n <= 2048) kernel = copy_entries<1024, 8, 16, true>, cw = 8;
    else if (n <= 4096) kernel = copy_entries<1024, 4, 16, false>, cw = 4;
    int64_t all = 0;
    for (int64_t i = 0; i < ncaches; ++i) all += (entry_bytes[i] + 16 * cw - 1) / (16 * cw);
    if (!grid_fits(all, threads)) return SELSCAN_E_UNSUPPORTED;
    CopyParams p;
    p.src = src, p.dst = dst, p.nslots = nslots, p.n = (int)n;
    for (int64_t i0 = 0; i0 < ncaches; i0 += kCaches) {
        int64_t blocks = 0;
        p.ncaches = 0;
        for (int64_t i = i0; i < ncaches && i < i0 + kCaches; ++i) {
            if (entry_bytes[i] == 0) continue;
            p.first[p.ncaches] = (uint32_t)blocks;
            p.c[p.ncaches++] = {(char *)caches[i], entry_bytes[i]};
            blocks += (entry_bytes[i] + 16 * cw - 1) / (16 * cw);
        }
        if (blocks == 0) continue;
        const int rc = enqueue(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), p, stream);
        if (rc != SELSCAN_OK) return rc;
    }
    return SELSCAN_OK;
}
