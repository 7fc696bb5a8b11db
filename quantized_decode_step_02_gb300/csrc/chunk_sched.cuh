// chunk_sched.cuh -- how the chunk attention cuts its work: host and device
// code, exact integer arithmetic.
//
// A request's new tokens are taken TP at a time, TP tokens x G query heads of
// one kv head = up to 256 rows (128 where requests are short: the launcher's
// choice): an item (request, kv head, row block).  An item's keys are cut into chunks of 128 (two pages) at multiples
// of 128; its weight is its number of chunks, at least 1.  The items in order
// (request, kv head, row block) lie on a line of W units, and CTA i of P takes
// the units [i W / P, (i + 1) W / P): every CTA gets the same number of chunks
// whatever the lengths are, items are cut where the line is.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define ZHD __host__ __device__ __forceinline__
#define ZHD_CALL __host__ __device__ __noinline__   // code that runs once is fetched once
#else
#define ZHD inline
#define ZHD_CALL inline
#endif

namespace zdec {

constexpr int CA_ROWS = 256, CA_KEYS = 128;   // most rows of an item, keys of a chunk

// sum over i in [0, n) of floor((a i + b) / m); a n + b < 2^32, m > 0.  The
// division steps of Euclid's algorithm on (m, a); 32-bit divisions.
ZHD long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long s = 0;
    while (n > 0) {
        if (a >= m) { s += (long long)(n - 1) * n / 2 * (a / m); a %= m; }
        if (b >= m) { s += (long long)n * (b / m); b %= m; }
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return s;
}

// One request: new tokens t0 .. t0 + n - 1 (rows of them in q: neff <= n),
// key j is seen by token i if j <= a + i (causal; a = kv - n) and, with a
// window, j > a + i - window.
struct ChunkReq {
    int t0, neff, kv, causal, window, TP;
    long long a;

    ZHD int blocks() const { return kv >= 0 ? (neff + TP - 1) / TP : 0; }
    // keys [lo, hi) that some row of block j sees
    ZHD long long hi(int j) const {
        if (!causal) return kv;
        const long long e = a + ((long long)(j + 1) * TP < neff ? (long long)(j + 1) * TP : neff);
        return e > 0 ? e : 0;
    }
    ZHD long long lo(int j) const {
        if (!window) return 0;
        const long long s = a + (long long)j * TP + 1 - window;
        return s > 0 ? s : 0;
    }
    ZHD int c_lo(int j) const { return (int)(lo(j) >> 7); }
    ZHD int chunks(int j) const {
        const long long h = hi(j);
        return h > 0 ? (int)((h + 127) >> 7) - c_lo(j) : 0;
    }
    ZHD int weight(int j) const { const int c = chunks(j); return c > 0 ? c : 1; }
    // sum of the weights of blocks 0 .. j-1 (j <= blocks())
    ZHD_CALL long long before(int j) const {
        if (j <= 0) return 0;
        if (!causal) return (long long)j * weight(0);
        const int J = blocks();
        if (J == 1) return weight(0);
        long long s = 0;
        int k = j;
        if (k == J) { s += weight(J - 1); k--; }   // the last block may be short
        // blocks whose keys end at or before 0: a + (i + 1) TP <= 0
        long long z = a < 0 ? -a / TP : 0;
        if (z > k) z = k;
        s += z;
        if (k > z) s += floor_sum((uint32_t)(k - z), 128u, (uint32_t)TP, (uint32_t)(a + (z + 1) * TP + 127));
        if (window) {
            const long long w = window - 1 - a;             // lo(i) > 0 from i TP > w on
            long long i0 = w >= 0 ? w / TP + 1 : 0;
            if (i0 < z) i0 = z;
            if (i0 < k) s -= floor_sum((uint32_t)(k - i0), 128u, (uint32_t)TP, (uint32_t)(i0 * TP - w));
        }
        return s;
    }
};

}  // namespace zdec
