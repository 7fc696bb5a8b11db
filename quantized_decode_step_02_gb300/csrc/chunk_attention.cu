// chunk_attention.cu -- attention of a chunk of new tokens over the paged
// cache, on the tensor cores.
//
// Per item (chunk_sched.cuh: up to 256 rows of (token, query head) that share
// a kv head) the keys pass once, 128 at a time, with the running maximum and
// sum of a softmax:
//   S = Q K^T          tcgen05, Q and K in shared memory, S (fp32) in TMEM
//   P = exp2(c S - m)  in registers, one row per thread; m lags the maximum by
//                      at most 2^8 so that O is rarely rescaled
//   O += P V           tcgen05, P (fp16) in TMEM over S, V in shared memory
// A CTA (one per SM, persistent) works on two buffers (S/P and O of 128 rows
// each, all 512 columns of TMEM): the two tiles of 128 rows of an item, or, for
// an item of at most 128 rows, its even and its odd chunks, joined at the end.
// So a softmax runs while the tensor core works on the other buffer.
//
// Warps: 0 copies (TMA), 1 issues the MMAs (one thread), 2 walks the line, 4-7
// and 8-11 are the softmax of buffer 0 and 1 (a row per thread), 12-15 prepare
// K and V.
//
// The page layout is what the MMA reads: V^T rows of 32 tokens, 64 bytes,
// swizzled as the 64-byte K-major operand; K rows of 256 bytes, whose two
// halves are each swizzled as the 128-byte K-major operand, so a tensor-map
// copy that splits the rows lands them as operands.  An fp16 cache needs no
// arithmetic between HBM and the tensor core; Q8_0 and FP8 chunks land raw and
// the preparing warps write them as fp16 operands (FP8 exactly; a Q8_0 code
// times its scale is rounded to fp16 once, 2^-12 of it on average, as P is:
// the tensor core takes no scale per key and 32 dims).  Values past the last
// key and of missing pages are set to 0 there (0 * NaN is NaN).
//
// Items cut between CTAs leave (m, l, O) in the workspace; a second kernel
// joins them in key order, so the result does not depend on timing.
//
// What bounds it (GB300, graph replays, both kernels):
// - 2048 tokens behind 30000 cached ones, fp16, 32 query and 8 kv heads: 700 us,
//   1490 TFLOP/s (77 % of cuBLAS's burst bf16 rate).  A chunk of two tiles takes
//   about 3300 cycles: its 32 MMAs 2048 of them, the softmax of its 256 rows on the
//   other side 1024 for the exp2 alone (4 cycles per warp and SM quarter) beside
//   packed fp32 arithmetic and TMEM reads; the two overlap, hand-overs do not.
// - the same from an FP8 cache: 850 us.  Eight bytes of a raw page become
//   sixteen, in and out of shared memory, on four warps with 96 registers; they
//   need as long as the softmax.  More warps would take the softmax's registers.
// - a step of 8 sequences, 800 to 30000 tokens, Q8_0: 76 us where the bytes
//   take 24; the conversion again, and 4 us of start, 5 us of joining.
// - one token over 2048, fp16: 14.7 us: launches, the walk to the first chunk, one
//   chunk, the epilogue and the join, each a microsecond or two of latency.
// Not kept, all slower: the conversions rolled up or further unrolled, K and V on
// warps of their own, the softmax of 256 quantised rows in two passes over S, one
// rolled loop for both buffers' MMAs, waiting for P V before the next Q K^T (the
// tensor core runs them in the order of issue).
#include <cuda.h>

#include <atomic>

#include "chunk.cuh"
#include "chunk_sched.cuh"
#include "tcgen05.cuh"

namespace zdec {

constexpr uint32_t CAF = 0xFFFFFFFFu;
constexpr int CA_THREADS = 512, CA_MAX_CTAS = 160;
constexpr int CA_SLOT = 32768;                     // bytes of a K or V operand chunk
constexpr int CA_RAW = 8704;                       // bytes of a raw one-byte region (one page's K or V)
constexpr int CA_MAX_SLOTS = 6, CA_MAX_RAW = 7;
// Shared memory: Q (rows x 256 bytes), operand slots, raw slots.  An fp16 cache
// needs no raw slots; a one-byte chunk in flight is half an operand.
template <int ROWS, bool ALL_F16>
struct CaLayout {
    static constexpr int Q_BYTES = ROWS * 256;
    static constexpr int SLOTS = ALL_F16 ? (ROWS > 128 ? 5 : 6) : (ROWS > 128 ? 3 : 4);
    static constexpr int RAWS = ALL_F16 ? 0 : (ROWS > 128 ? 6 : 7);
    static constexpr int BYTES = Q_BYTES + SLOTS * CA_SLOT + RAWS * CA_RAW;
};
constexpr uint32_t CA_WAIT_LIMIT = 1u << 31;       // clock cycles (~1 s)
constexpr float CA_LAG = 8.0f;                     // log2 units that m may lag behind the maximum
constexpr int PART_LD = HD + 4;                    // floats of a partial row: m, l, -, -, o[128]
constexpr int CA_COMBINE_Y = 8;
constexpr int CA_SEGS = 4, CA_SEG_READERS = 14;   // segments on their way; warps that read each

// Workspace: one descriptor per CTA, then two partial items per CTA (0: the
// end of an item that an earlier CTA began, 1: the begin of one that a later
// CTA ends).
struct CaDesc {
    int valid, t0, h, row0, rows, last;            // rows of the item begun, last: the CTA that ends it
    int pad[10];
};
size_t chunk_attention_workspace(int, int) {
    return CA_MAX_CTAS * sizeof(CaDesc) + (size_t)CA_MAX_CTAS * 2 * CA_ROWS * PART_LD * sizeof(float);
}
__device__ __forceinline__ float *part_row(uint8_t *ws, int cta, int which, int row) {
    return reinterpret_cast<float *>(ws + CA_MAX_CTAS * sizeof(CaDesc)) + ((size_t)(cta * 2 + which) * CA_ROWS + row) * PART_LD;
}

// ---------------------------------------------------------------- segments ---
// A CTA's piece of the line as (item, chunk range) segments.  Warp 2 walks it
// and passes the segments on through shared memory, so that no other warp
// holds the walk's state or waits for the lengths.
struct Segment {
    int h, row0, rows;        // kv head; first row and rows of the item within (request, head)
    int t0, r, kv;            // first token, index and keys of the request
    int c0, n_c;              // first chunk and chunks of this piece; n_c < 0: the walk's end
    long long a;              // last key of token 0 of the request
    int begins, ends;         // the piece holds the item's first / last chunk
    int last;                 // begins, but does not end: the CTA that ends the item
};
struct Walk {
    ChunkReq q;
    int r, h, j, J;
    int ov;                   // units of an item's fixed cost
    int off;                  // units of the item before this CTA's
    long long left;           // units left to this CTA
};
__device__ __forceinline__ ChunkReq load_req(const ChunkAttnParams &p, int r) {
    ChunkReq q;
    const int a = __ldg(p.cu + r), b = __ldg(p.cu + r + 1);
    const long long cap = (long long)p.kv.max_pages * 64;
    q.kv = (int)min(cap, (long long)max(0, __ldg(p.kv_len + r)));
    q.t0 = a;
    q.neff = a >= 0 ? max(0, min(b, p.T) - a) : 0;
    q.causal = p.causal;
    q.window = p.window;
    q.TP = p.rows / p.G;
    q.a = (long long)q.kv - ((long long)b - a);
    return q;
}
__device__ __forceinline__ bool next_segment(const ChunkAttnParams &p, Walk &w, long long u1, long long W, int P, Segment &s) {
    if (w.left <= 0) return false;
    while (w.j >= w.J) {
        if (w.J > 0 && w.h + 1 < p.kv.n_kv) {
            w.h++;
        } else {
            if (++w.r >= p.R) return false;
            w.q = load_req(p, w.r);
            w.J = w.q.blocks();
            w.h = 0;
        }
        w.j = 0;
    }
    const int chunks = w.q.chunks(w.j), weight = max(1, chunks) + w.ov;
    const int take = (int)min((long long)(weight - w.off), w.left);
    const int a = max(0, w.off - w.ov), b = max(0, w.off + take - w.ov);   // of its chunks (or of the one unit of an item without)
    s.h = w.h;
    s.r = w.r;
    s.row0 = w.j * w.q.TP * p.G;
    s.rows = min(w.q.TP, w.q.neff - w.j * w.q.TP) * p.G;
    s.t0 = w.q.t0;
    s.a = w.q.a;
    s.kv = w.q.kv;
    s.c0 = w.q.c_lo(w.j) + a;
    s.n_c = chunks > 0 ? b - a : 0;
    s.begins = a == 0;
    s.ends = w.off + take == weight;
    w.left -= take;
    w.off += take;
    // this CTA's range ends here: the item's last unit is at u1 + what is left of it
    s.last = s.ends ? 0 : (int)(((u1 + weight - w.off) * P + W - 1) / W) - 1;
    if (s.ends) {
        w.off = 0;
        w.j++;
    }
    return b > a;   // false: only the item's fixed cost lies in this CTA's range, which ends there
}

// Keys [lo, hi) that some row, and [all_lo, all_hi) that every row of the item sees.
struct Seen {
    long long lo, hi, all_lo, all_hi;
};
__device__ __forceinline__ Seen seen_by(const ChunkAttnParams &p, const Segment &s) {
    const long long first = s.a + s.row0 / p.G, last = s.a + (s.row0 + s.rows - 1) / p.G;
    Seen k;
    k.hi = p.causal ? min((long long)s.kv, last + 1) : s.kv;
    k.all_hi = p.causal ? min((long long)s.kv, first + 1) : s.kv;
    k.lo = p.window ? max(0LL, first + 1 - p.window) : 0;
    k.all_lo = p.window ? max(0LL, last + 1 - p.window) : 0;
    return k;
}
// Whether some key of the chunk at key0 is seen by some rows of the item, not by all.
__device__ __forceinline__ bool partly_seen(const Seen &k, long long key0) {
    return min(key0 + CA_KEYS, k.hi) > k.all_hi || max(key0, k.lo) < k.all_lo;
}

// ---------------------------------------------------------------- shared ---
constexpr int CA_BARS_1 = 2 * CA_MAX_SLOTS + CA_MAX_RAW + 5 + 8 + CA_SEGS, CA_BARS_4 = CA_MAX_SLOTS + CA_MAX_RAW + 6;
constexpr int CA_BARS = CA_BARS_1 + CA_BARS_4 + CA_SEGS;
__device__ __forceinline__ int bar_count(int i) { return i < CA_BARS_1 ? 1 : (i < CA_BARS_1 + CA_BARS_4 ? 4 : CA_SEG_READERS); }
struct CaShared {
    float2 odd[128];               // (m, l) of each row over the odd chunks of an item with one tile
    union {
        uint64_t bars[CA_BARS];
        struct {
            // one arrival each
            uint64_t full[CA_MAX_SLOTS], empty[CA_MAX_SLOTS], raw_full[CA_MAX_RAW], s_full[2], o_done[2], drain;
            uint64_t odd_full[4], odd_read[4];   // per softmax warp: `odd` written, and O of the odd chunks read
            uint64_t seg_full[CA_SEGS];
            // four warps
            uint64_t ready[CA_MAX_SLOTS], raw_empty[CA_MAX_RAW], q_ready[2], p_ready[2][2];   // p_ready: keys 0-63, 64-127
            uint64_t seg_empty[CA_SEGS];
        };
    };
    Segment seg[CA_SEGS];
    ChunkReq w_q;             // the request that holds this CTA's first unit, its index, its weight per kv head,
    int w_r;                  // and which of its units that is
    long long w_per, w_x;
    long long scan[2][CA_THREADS / 32];
    uint32_t tmem;
    int abort;
    int pages_ok[8];          // chunk i (mod 8): bit k, page k of it is in the pool
    uint32_t bad[8];          // one byte per preparing warp: a value that only some rows see is not finite
};
constexpr int CA_SHARED_BYTES = (int)((sizeof(CaShared) + 15) / 16 * 16);

// K and V of an item's chunks in the order they are used: with two tiles
// K0 V0 K1 V1 ..., with one K0 K1 V0 K2 V1 ... (its scores run a chunk ahead).
__device__ __forceinline__ int k_item(int c, bool two) { return two ? 2 * c : (c == 0 ? 0 : 2 * c - 1); }
__device__ __forceinline__ int v_item(int c, int n_c, bool two) { return two ? 2 * c + 1 : min(2 * c + 2, 2 * n_c - 1); }
__device__ __forceinline__ void item_at(int i, int n_c, bool two, int &kv, int &c) {
    if (two) {
        kv = i & 1;
        c = i >> 1;
    } else if (i == 0 || i == 2 * n_c - 1) {
        kv = i != 0;
        c = kv ? n_c - 1 : 0;
    } else {
        kv = !(i & 1);
        c = kv ? i / 2 - 1 : (i + 1) / 2;
    }
}

// Bounded waits (the 32-bit clock wraps after about 2 s; the bound is half of that).
struct Waiter {
    volatile int *abort;
    uint32_t *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const uint32_t t0 = (uint32_t)clock();
        bool late = false;
        do {
            if (mbar_try_wait(bar, parity)) return true;
            late = (uint32_t)clock() - t0 > CA_WAIT_LIMIT;
        } while (!late && !*abort);
        *abort = 1;
        if (late && status) atomicOr(status, (uint32_t)ZDEC_CHUNK_TIMEOUT);
        return false;
    }
    // the same answer on every lane of a warp
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
        return __all_sync(CAF, (*this)(bar, parity));
    }
};
__device__ __forceinline__ void mbar_arrive1(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One box of 64 elements x 64 keys of a K region (row half `half`).
__device__ __forceinline__ void tma_k_half(void *dst, const CUtensorMap *map, int half, int chunk, int page, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(0), "r"(half), "r"(0), "r"(chunk), "r"(page), "r"(smem_u32(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------ preparing K, V ---
// Sixteen one-byte codes -> sixteen fp16 (two 16-byte groups).
template <bool Q8>
__device__ __forceinline__ void codes16(uint4 c, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (Q8) {
            const __half2 bias = __float2half2_rn(1152.0f);   // 1024 + the stored offset of 128
            o[2 * i] = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(w[i], 0x64646464u, 0x4140)), bias));
            o[2 * i + 1] = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(w[i], 0x64646464u, 0x4342)), bias));
        } else {
            o[2 * i] = e4m3x2_to_h2((uint16_t)w[i]);
            o[2 * i + 1] = e4m3x2_to_h2((uint16_t)(w[i] >> 16));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }
// Two Q8_0 scales, at most 515.5: 127 x 516, which only a block that reaches
// 65,488 has, is past fp16.  A NaN stays one.
__device__ __forceinline__ uint32_t q8_scales(uint32_t s) {
    return h2_as_u32(__hmin2_nan(u32_as_h2(s), __float2half2_rn(515.5f)));
}
__device__ __forceinline__ uint4 hmul8(uint4 a, uint4 b) {
    return make_uint4(hmul2_u(a.x, b.x), hmul2_u(a.y, b.y), hmul2_u(a.z, b.z), hmul2_u(a.w, b.w));
}
// Keeps elements [lo, hi) of eight fp16 (group element indices), zeroes the rest.
__device__ __forceinline__ uint4 keep8(uint4 v, int lo, int hi) {
    if (lo <= 0 && hi >= 8) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (2 * i < lo || 2 * i >= hi) w[i] &= 0xFFFF0000u;
        if (2 * i + 1 < lo || 2 * i + 1 >= hi) w[i] &= 0x0000FFFFu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// K of one page: thread = (key, half of the dims) -> [half][keys][128 bytes], SW128; `page`: the chunk's page.
template <bool Q8>
__device__ __forceinline__ void prepare_k(const uint8_t *reg, uint8_t *slot, int th, int page) {
    const int t = th & 63, half = th >> 6;
    uint32_t sc = 0;
    if (Q8) sc = q8_scales(*reinterpret_cast<const uint32_t *>(reg + ks_off(t, 2 * half)));
    uint8_t *row = slot + half * 16384 + (page * 64 + t) * 128;
    uint4 c[4];
#pragma unroll
    for (int s = 0; s < 4; s++) c[s] = *reinterpret_cast<const uint4 *>(reg + k8_off(t, 64 * half + 16 * s));
#pragma unroll
    for (int s = 0; s < 4; s++) {   // 16 dims
        uint4 lo, hi;
        codes16<Q8>(c[s], lo, hi);
        if (Q8) {
            const uint32_t d = s < 2 ? __byte_perm(sc, sc, 0x1010) : __byte_perm(sc, sc, 0x3232);
            const uint4 d4 = make_uint4(d, d, d, d);
            lo = hmul8(lo, d4);
            hi = hmul8(hi, d4);
        }
        *reinterpret_cast<uint4 *>(row + (((2 * s) ^ (t & 7)) << 4)) = lo;
        *reinterpret_cast<uint4 *>(row + (((2 * s + 1) ^ (t & 7)) << 4)) = hi;
    }
}
// V of one page: thread = dim -> [unit of 32 tokens][128 dims][64 bytes], SW64.
template <bool Q8>
__device__ __forceinline__ void prepare_v(const uint8_t *reg, uint8_t *slot, int d, int page) {
    uint4 c[4];
#pragma unroll
    for (int i = 0; i < 4; i++) c[i] = *reinterpret_cast<const uint4 *>(reg + v8_off(16 * i, d));
#pragma unroll
    for (int i = 0; i < 4; i++) {   // 16 tokens
        uint4 a, b;
        codes16<Q8>(c[i], a, b);
        if (Q8) {
            const uint4 s0 = *reinterpret_cast<const uint4 *>(reg + vs_off(16 * i, d >> 5));
            const uint4 s1 = *reinterpret_cast<const uint4 *>(reg + vs_off(16 * i + 8, d >> 5));
            a = hmul8(a, make_uint4(q8_scales(s0.x), q8_scales(s0.y), q8_scales(s0.z), q8_scales(s0.w)));
            b = hmul8(b, make_uint4(q8_scales(s1.x), q8_scales(s1.y), q8_scales(s1.z), q8_scales(s1.w)));
        }
        uint8_t *row = slot + (2 * page + (i >> 1)) * 8192 + d * 64;
        const int g = 2 * (i & 1);
        *reinterpret_cast<uint4 *>(row + ((g ^ ((d >> 1) & 3)) << 4)) = a;
        *reinterpret_cast<uint4 *>(row + (((g + 1) ^ ((d >> 1) & 3)) << 4)) = b;
    }
}
// V values outside tokens [lo, hi) of the chunk, or of a missing page, to 0.
__device__ __forceinline__ void clean_v(uint8_t *slot, int d, int lo, int hi, int pages_ok) {
    if (!(pages_ok & 1)) lo = max(lo, 64);
    if (!(pages_ok & 2)) hi = min(hi, 64);
#pragma unroll 1
    for (int c0 = 0; c0 < CA_KEYS; c0 += 8) {
        if (c0 >= lo && c0 + 8 <= hi) continue;
        uint4 *at = reinterpret_cast<uint4 *>(slot + (c0 >> 5) * 8192 + d * 64 + ((((c0 >> 3) & 3) ^ ((d >> 1) & 3)) << 4));
        *at = keep8(*at, lo - c0, hi - c0);
    }
}

// Whether dim d of a V operand chunk holds an infinity or a NaN.
__device__ __forceinline__ bool v_not_finite(const uint8_t *slot, int d) {
    uint32_t bad = 0;   // an exponent of all ones plus one carries into the bit above it
#pragma unroll 1
    for (int g = 0; g < 16; g++) {
        const uint4 v = *reinterpret_cast<const uint4 *>(slot + (g >> 2) * 8192 + d * 64 + ((g & 3) << 4));
        bad |= ((v.x & 0x7C007C00u) + 0x04000400u) | ((v.y & 0x7C007C00u) + 0x04000400u) | ((v.z & 0x7C007C00u) + 0x04000400u) |
               ((v.w & 0x7C007C00u) + 0x04000400u);
    }
    return (bad & 0x80008000u) != 0;
}
__device__ __forceinline__ float v_at(const uint8_t *slot, int j, int d) {
    return __half2float(*reinterpret_cast<const __half *>(slot + (j >> 5) * 8192 + d * 64 +
                                                          ((((j & 31) >> 3) ^ ((d >> 1) & 3)) << 4) + (j & 7) * 2));
}

// The 32 rows of a warp into its part of a Q operand tile (`src`: this lane's
// row), copied two rows of 16 lanes x 16 bytes at a time, BATCH of them in
// flight (8 for the prompts of one-byte caches: 2048 tokens over 6000 FP8 keys
// 251 to 238 us; 4 else: over fp16 ones 189 and 191, a step of 8 76 and 78).  fp16 stays as it
// is.  A bf16 row is multiplied in place by 2^-e, which brings its largest
// element below fp16's top (exact but for elements below 2^-28 of it): by the
// lane that owns it (sixteen conflict-free 16-byte accesses, no exchange between
// lanes: prompts of a mixed batch 120 to 114 us), or where warps hold FEW rows by
// the 16 lanes that copied it (a step of 8: 77 us, with the other form 83).
// Returns e of this lane's row.  Rows from n_rows on stay as
// they are: a row of the MMA touches no other.
template <bool FEW, int BATCH>
__device__ __forceinline__ int load_q(const uint16_t *src, int io_type, bool store, uint8_t *tile, int row0, int n_rows) {
    const int lane = threadIdx.x & 31, c = lane & 15, up = lane >> 4;
    uint8_t *to = tile + (c >> 3) * 16384 + (row0 + up) * 128;
    if (store) {
#pragma unroll 1
        for (int i0 = 0; 2 * i0 < n_rows; i0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; i++) {
                const uint16_t *from = (const uint16_t *)__shfl_sync(CAF, (unsigned long long)src, 2 * (i0 + i) + up);
                v[i] = __ldg(reinterpret_cast<const uint4 *>(from) + c);
            }
#pragma unroll
            for (int i = 0; i < BATCH; i++)
                *reinterpret_cast<uint4 *>(to + (i0 + i) * 256 + (((c ^ (2 * (i0 + i) + up)) & 7) << 4)) = v[i];
        }
    }
    if (io_type == ZDEC_F16) return 0;
    __syncwarp();
    if (FEW) {
        int mine = 0;
#pragma unroll 1
        for (int i = 0; 2 * i < n_rows; i++) {
            uint4 *at = reinterpret_cast<uint4 *>(to + i * 256 + (((c ^ (2 * i + up)) & 7) << 4));
            const uint16_t *from = (const uint16_t *)__shfl_sync(CAF, (unsigned long long)src, 2 * i + up);
            const uint4 x = store ? *at : __ldg(reinterpret_cast<const uint4 *>(from) + c);
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, top = 0;   // largest magnitude bits of the row
#pragma unroll
            for (int k = 0; k < 4; k++) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(CAF, top, o));
            const int ex = (int)(top >> 7);                  // biased exponent
            const int e = ex == 0 || ex == 255 ? 0 : ex - 127 - 14;
            const int both = __shfl_sync(CAF, e, (lane & 1) * 16);
            if ((lane >> 1) == i) mine = both;
            // 2^-e, e in [-140, 113]: 2^140 in two steps
            const float f1 = __int_as_float((127 + min(-e, 100)) << 23), f2 = __int_as_float((127 + max(-e - 100, 0)) << 23);
#pragma unroll
            for (int k = 0; k < 4; k++)
                w[k] = h2_as_u32(__floats2half2_rn(__uint_as_float(w[k] << 16) * f1 * f2, __uint_as_float(w[k] & 0xFFFF0000u) * f1 * f2));
            if (store) *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return mine;
    }
    uint8_t *row = tile + (row0 + lane) * 128;
    auto at = [&](int k) { return reinterpret_cast<uint4 *>(row + (k >> 3) * 16384 + (((k ^ lane) & 7) << 4)); };
    uint32_t top2 = 0;                                   // largest magnitude bits, of even and odd elements
#pragma unroll 4
    for (int k = 0; k < 16; k++) {
        const uint4 x = store ? *at(k) : __ldg(reinterpret_cast<const uint4 *>(src) + k);
        top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
    const int ex = (int)(max(top2 & 0xFFFFu, top2 >> 16) >> 7);   // biased exponent
    const int e = ex == 0 || ex == 255 ? 0 : ex - 127 - 14;
    if (!store) return e;
    // 2^-e, e in [-140, 113]: 2^140 in two steps
    const float f1 = __int_as_float((127 + min(-e, 100)) << 23), f2 = __int_as_float((127 + max(-e - 100, 0)) << 23);
#pragma unroll 4
    for (int k = 0; k < 16; k++) {
        const uint4 x = *at(k);
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = h2_as_u32(__floats2half2_rn(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2));
        *at(k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return e;
}
// 256 bytes of each of a warp's 32 rows, staged in shared memory in the same
// arrangement, to `dst` (this lane's row; null: not written).
__device__ __forceinline__ void flush_rows(const uint8_t *tile, int row0, int n_rows, uint8_t *dst) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < 16; i++) {
        if (2 * i >= n_rows) break;
        const int row = row0 + 2 * i + (lane >> 4);
        uint8_t *to = (uint8_t *)__shfl_sync(CAF, (unsigned long long)dst, 2 * i + (lane >> 4));
        const uint4 x = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        if (to) *reinterpret_cast<uint4 *>(to + 16 * c) = x;
    }
    __syncwarp();
}
__device__ __forceinline__ void stage(uint8_t *tile, int row, int c, uint32_t a, uint32_t b, uint32_t d, uint32_t e) {
    *reinterpret_cast<uint4 *>(tile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(a, b, d, e);
}
__device__ __forceinline__ uint32_t pack_out(float x, float y, int io_type) {
    if (io_type == ZDEC_F16) return h2_as_u32(__floats2half2_rn(x, y));
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
// Scores outside [lo, hi) of 32 to -inf.
__device__ __forceinline__ void hide(uint32_t (&v)[32], int lo, int hi) {
    const int a = max(lo, 0), b = min(hi, 32);
    const uint32_t sees = b > a ? (0xFFFFFFFFu >> (32 - (b - a))) << a : 0u;
    if (sees == 0xFFFFFFFFu) return;
#pragma unroll
    for (int k = 0; k < 32; k++)
        if (!((sees >> k) & 1)) v[k] = 0xFF800000u;
}
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
    float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]);
#pragma unroll
    for (int k = 2; k < 32; k += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(v[k])), __uint_as_float(v[k + 1]));
        if (k + 3 < 32) b = fmaxf(fmaxf(b, __uint_as_float(v[k + 2])), __uint_as_float(v[k + 3]));
    }
    return fmaxf(a, b);
}
// Two fp32 at a time.
__device__ __forceinline__ void fma_pair(float &x, float &y, float a, float b) {   // x, y = x a + b, y a + b
    asm("{\n .reg .b64 v, m, c;\n mov.b64 v, {%0, %1};\n mov.b64 m, {%2, %2};\n mov.b64 c, {%3, %3};\n"
        " fma.rn.f32x2 v, v, m, c;\n mov.b64 {%0, %1}, v;\n}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void add_pair(float &x, float &y, float a, float b) {
    asm("{\n .reg .b64 v, c;\n mov.b64 v, {%0, %1};\n mov.b64 c, {%2, %3};\n add.rn.f32x2 v, v, c;\n mov.b64 {%0, %1}, v;\n}"
        : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
// ------------------------------------------------------------------ kernel ---
__device__ __noinline__ long long div_any(long long a, long long b) {   // a >= 0, b > 0
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int ROWS, bool ALL_F16>
__global__ __launch_bounds__(CA_THREADS, 1) void chunk_attention_kernel(const __grid_constant__ ChunkAttnParams p,
                                                                        const __grid_constant__ CUtensorMap k_map) {
    extern __shared__ __align__(1024) uint8_t dyn[];   // no static shared memory: starts on a 1024-byte boundary
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    const bool k16 = ALL_F16 || p.kv.k_type == KV_T_F16, v16 = ALL_F16 || p.kv.v_type == KV_T_F16;
    using Lay = CaLayout<ROWS, ALL_F16>;
    constexpr uint32_t NS = Lay::SLOTS, NR = Lay::RAWS > 0 ? Lay::RAWS : 1;
    uint8_t *q_smem = dyn, *slots = dyn + Lay::Q_BYTES, *raws = slots + NS * CA_SLOT;
    CaShared &sh = *reinterpret_cast<CaShared *>(dyn + Lay::BYTES);
    CaDesc *desc = reinterpret_cast<CaDesc *>(p.ws) + cta;

    // ---- this CTA's piece of the line: a prefix sum over the requests' weights, 512 at a time (the last strip's
    // weights stay in registers: with up to 512 requests they are read once)
    const int n_kv = p.kv.n_kv;
    ChunkReq my_q;
    long long W = -1, run = 0, u0 = 0, u1 = 0;
    int P = 0;
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    for (int i = tid; i < CA_BARS; i += CA_THREADS) mbar_init(&sh.bars[i], bar_count(i));
    if (tid == 0) sh.abort = 0;
    mbar_fence_init();
    tc_fence_before();
    if (ROWS == 128) pdl_wait();   // short items: started while the kernel before ends; it wrote the inputs, or reads the workspace
    if (tid == 0) desc->valid = 0;
    long long run_items = 0;   // an item costs ov units beside its chunks
    int ov = 0;
    // With more than two chunks per CTA an item's start and end (its Q, its O, an empty pipeline) are worth about three
    // chunks of 256 rows or four of 128; with fewer every chunk gets a CTA of its own.
    auto cut = [&]() {
        ov = run > 2LL * gridDim.x ? (ROWS > 128 ? 3 : 4) : 0;
        W = run + ov * run_items;
        P = (int)min((long long)gridDim.x, W);   // every CTA of the first P has units: pieces follow each other
        if (cta >= P) return;
        u0 = div_any(W * cta, P);
        u1 = div_any(W * (cta + 1), P);
    };
    if (p.R <= 32) {   // every warp by itself
        long long my_per = 0, my_w = 0, my_i = 0;
        if (lane < p.R) {
            my_q = load_req(p, lane);
            my_per = my_q.before(my_q.blocks());
            my_w = my_per * n_kv;
            my_i = (long long)my_q.blocks() * n_kv;
        }
        run = my_w;
        run_items = my_i;
#pragma unroll 1
        for (int o = 1; o < p.R; o <<= 1) {
            const long long v = __shfl_up_sync(CAF, run, o), vi = __shfl_up_sync(CAF, run_items, o);
            if (lane >= o) {
                run += v;
                run_items += vi;
            }
        }
        const long long incl = run, incl_i = run_items;
        run = __shfl_sync(CAF, run, p.R - 1);
        run_items = __shfl_sync(CAF, run_items, p.R - 1);
        cut();
        const long long mine = my_w + ov * my_i, excl = incl + ov * incl_i - mine;
        if (warp == 2 && mine > 0 && excl <= u0 && u0 < excl + mine) {
            sh.w_q = my_q;
            sh.w_r = lane;
            sh.w_per = my_per + (long long)ov * my_q.blocks();
            sh.w_x = u0 - excl;
        }
    }
#pragma unroll 1
    for (int r0 = 0; p.R > 32;) {
        long long my_per = 0, my_w = 0, my_i = 0;
        if (r0 + tid < p.R) {
            my_q = load_req(p, r0 + tid);
            my_per = my_q.before(my_q.blocks());
            my_w = my_per * n_kv;
            my_i = (long long)my_q.blocks() * n_kv;
        }
        long long incl = my_w, incl_i = my_i;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(CAF, incl, o), vi = __shfl_up_sync(CAF, incl_i, o);
            if (lane >= o) {
                incl += v;
                incl_i += vi;
            }
        }
        if (lane == 31) {
            sh.scan[0][warp] = incl;
            sh.scan[1][warp] = incl_i;
        }
        __syncthreads();
        incl += run;
        incl_i += run_items;
#pragma unroll 1
        for (int i = 0; i < CA_THREADS / 32; i++) {
            const long long v = sh.scan[0][i], vi = sh.scan[1][i];
            if (i < warp) {
                incl += v;
                incl_i += vi;
            }
            run += v;
            run_items += vi;
        }
        __syncthreads();
        if (W < 0) {                               // first time: up to all requests' weight
            r0 += CA_THREADS;
            if (r0 < p.R) continue;
            cut();
            if (cta >= P) break;
            r0 = 0;
            if (p.R > CA_THREADS) {                // second time: up to this CTA's first unit
                run = 0;
                run_items = 0;
                continue;
            }
        }
        const long long mine = my_w + ov * my_i, excl = incl + ov * incl_i - mine;
        if (mine > 0 && excl <= u0 && u0 < excl + mine) {
            sh.w_q = my_q;
            sh.w_r = r0 + tid;
            sh.w_per = my_per + (long long)ov * my_q.blocks();
            sh.w_x = u0 - excl;
        }
        if (run + ov * run_items > u0) break;
        r0 += CA_THREADS;
    }
    __syncthreads();
    tc_fence_after();
    if (cta >= P) {
        if (warp == 1) tmem_dealloc(sh.tmem, 512);
        pdl_launch_dependents();
        return;
    }
    const uint32_t tmem = __shfl_sync(CAF, sh.tmem, 0);
    pdl_launch_dependents();

    const Waiter wait{&sh.abort, p.status};
    const int group = warp >> 2;
    uint32_t si = 0;          // segments read so far
    // the next segment (by reference: fields are read where they are used); false at the end
    auto next = [&]() -> bool {
        return wait.warp(&sh.seg_full[si % CA_SEGS], (si / CA_SEGS) & 1) && sh.seg[si % CA_SEGS].n_c >= 0;
    };
    auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive1(&sh.seg_empty[si % CA_SEGS]);
        si++;
    };

    // registers: 4 warpgroups x 128 at launch = 64 + 80 + 2 x 184, or 64 + 96 + 2 x 176; short items need no other split
    if (group == 0) {
        if (ROWS > 128) reg_dec<64>();
        if (warp == 0) {
            // ---------------------------------------------------------- copies ---
            const uint32_t kb = kv_region_bytes(p.kv.k_type), vb = kv_region_bytes(p.kv.v_type);
            const size_t coff = kv_chunk_off(p.kv, p.layer, 0);
            uint32_t it = 0, dir = 0, raw = 0, ci = 0;   // operands, those landing as such, raw pages; chunks
            bool ok = true;
            for (; ok && next(); done()) {
                const Segment s = sh.seg[si % CA_SEGS];
                const bool two = ROWS > 128 && s.rows > 128;
                const int32_t *row = p.kv.table + (size_t)s.r * p.kv.max_pages;
                const size_t off = coff + (size_t)s.h * (kb + vb);
                // pages of 16 chunks, one per lane; V lags K by up to two chunks, so the 16 before are kept
                auto pages_of = [&](int c16) {
                    const long long pg = ((long long)s.c0 + 16 * c16) * 2 + lane;
                    return pg < p.kv.max_pages && pg * 64 < s.kv ? __ldg(row + pg) : -2;   // -2: no key there
                };
                int now = pages_of(0), before = -2, now_i = 0;
                for (int i = 0; ok && i < 2 * s.n_c; i++, it++) {
                    int kv, c;
                    item_at(i, s.n_c, two, kv, c);
                    if (kv == 0 && (c >> 4) != now_i) {
                        before = now;
                        now_i = c >> 4;
                        now = pages_of(now_i);
                    }
                    const int from = (c >> 4) == now_i ? now : before;
                    const int pa = __shfl_sync(CAF, from, 2 * (c & 15)), pb = __shfl_sync(CAF, from, 2 * (c & 15) + 1);
                    const int okm = (kv_page_ok(p.kv, pa) ? 1 : 0) | (kv_page_ok(p.kv, pb) ? 2 : 0);
                    if (lane == 0) {
                        const uint32_t bytes = kv ? vb : kb;
                        const size_t at = off + (kv ? kb : 0);
                        if (kv ? v16 : k16) {
                            const uint32_t sl = it % NS;
                            ok = it < NS || wait(&sh.empty[sl], (it / NS - 1) & 1);
                            if (ok) {
                                // chunk ci + c's entry was last read for chunk ci + c - 8, whose operands have left their slots
                                if (kv == 0) sh.pages_ok[(ci + c) & 7] = okm;
                                uint8_t *dst = slots + sl * CA_SLOT;
                                uint64_t *bar = &sh.full[dir % CA_MAX_SLOTS];
                                dir++;
                                if (okm) mbar_expect_tx(bar, __popc(okm) * bytes);
                                else mbar_arrive1(bar);
#pragma unroll 1
                                for (int k = 0; k < 2; k++) {
                                    if (!((okm >> k) & 1)) continue;
                                    const int page = k ? pb : pa;
                                    if (kv) bulk_g2s(dst + k * 16384, p.kv.base + (size_t)page * p.kv.page_bytes + at, bytes, bar);
                                    else
                                        for (int half = 0; half < 2; half++)
                                            tma_k_half(dst + half * 16384 + k * 8192, &k_map, half, p.layer * n_kv + s.h, page, bar);
                                }
                            }
                        } else {
#pragma unroll 1
                            for (int k = 0; ok && k < 2; k++) {
                                const uint32_t sl = raw % NR;
                                ok = raw < NR || wait(&sh.raw_empty[sl], (raw / NR - 1) & 1);
                                if (!ok) break;
                                if (kv == 0 && k == 0) sh.pages_ok[(ci + c) & 7] = okm;
                                uint64_t *bar = &sh.raw_full[sl];
                                raw++;
                                if ((okm >> k) & 1) {
                                    mbar_expect_tx(bar, bytes);
                                    bulk_g2s(raws + sl * CA_RAW, p.kv.base + (size_t)(k ? pb : pa) * p.kv.page_bytes + at, bytes, bar);
                                } else {
                                    mbar_arrive1(bar);
                                }
                            }
                        }
                        if (p.status && kv == 0 && ((!(okm & 1) && pa != -2) || (!(okm & 2) && pb != -2)))
                            atomicOr(p.status, (uint32_t)ZDEC_CHUNK_NO_PAGE);
                    }
                    ok = __shfl_sync(CAF, (int)ok, 0);
                }
                ci += s.n_c;
            }
            // copies in flight land before the CTA leaves, also where a wait gave up
            if (lane == 0 && sh.abort) {
                const uint32_t t0 = (uint32_t)clock();
                for (uint32_t i = dir > CA_MAX_SLOTS ? dir - CA_MAX_SLOTS : 0; i < dir; i++)
                    while (!mbar_try_wait(&sh.full[i % CA_MAX_SLOTS], (i / CA_MAX_SLOTS) & 1) && (uint32_t)clock() - t0 < CA_WAIT_LIMIT) {}
                for (uint32_t i = raw > NR ? raw - NR : 0; !ALL_F16 && i < raw; i++)
                    while (!mbar_try_wait(&sh.raw_full[i % NR], (i / NR) & 1) && (uint32_t)clock() - t0 < CA_WAIT_LIMIT) {}
            }
        } else if (warp == 1) {
            // -------------------------------------------------------------- MMA ---
            if (elect_one()) {
                constexpr uint32_t IDESC = MMA_IDESC_F16<128, 128>;
                const uint64_t q_desc = mma_desc_sw128(smem_u32(q_smem)), k_desc = mma_desc_sw128(smem_u32(slots)),
                               v_desc = mma_desc_sw64(smem_u32(slots));
                uint32_t it0 = 0, ci = 0, segs[2] = {0, 0}, n_p[2] = {0, 0};   // operands, chunks before; segments, steps per buffer
                bool ok = true;
                auto ready = [&](uint32_t item) { return wait(&sh.ready[item % NS], (item / NS) & 1); };
                for (; ok; si++) {
                    ok = wait(&sh.seg_full[si % CA_SEGS], (si / CA_SEGS) & 1);
                    const int n_c = sh.seg[si % CA_SEGS].n_c;
                    const bool two = ROWS > 128 && sh.seg[si % CA_SEGS].rows > 128;
                    if (!ok || n_c < 0) break;
                    mbar_arrive1(&sh.seg_empty[si % CA_SEGS]);
                    if (n_c == 0) continue;
                    const int steps = two ? 2 * n_c : n_c;
                    for (int t = 0; t < (two ? 2 : 1); t++) ok = ok && wait(&sh.q_ready[t], segs[t]++ & 1);
                    // step i: chunk i / 2 of tile i % 2, or chunk i of the one tile, in buffer i % 2; its S two steps ahead
#pragma unroll 1
                    for (int i = -2; i < steps; i++) {
                        const int u = i & 1;
                        if (i >= 0) {
                            const int c = two ? i >> 1 : i;
                            const uint32_t item = it0 + v_item(c, n_c, two);
                            if (!two || u == 0) ok = ok && ready(item);
                            ok = ok && wait(&sh.p_ready[u][0], n_p[u] & 1);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t vd = v_desc + (item % NS) * (CA_SLOT >> 4);
                            const uint32_t od = tmem + 256 + u * 128;
                            // a chunk whose product the softmax threads make themselves only reports
                            const bool bad = sh.bad[(ci + c) & 7] != 0;
                            if (!bad)
#pragma unroll
                                for (int k = 0; k < 4; k++)    // keys 0-63
                                    mma_ts(od, tmem + u * 128 + k * 8, vd + (((k >> 1) * 8192 + (k & 1) * 32) >> 4), IDESC, i > 1 || k > 0);
                            ok = wait(&sh.p_ready[u][1], n_p[u] & 1);
                            if (!ok) break;
                            tc_fence_after();
                            if (!bad)
#pragma unroll
                                for (int k = 4; k < 8; k++)
                                    mma_ts(od, tmem + u * 128 + k * 8, vd + (((k >> 1) * 8192 + (k & 1) * 32) >> 4), IDESC, true);
                            mma_commit(&sh.o_done[u]);
                            if (!two || u == 1) mma_commit(&sh.empty[item % NS]);
                            n_p[u]++;
                        }
                        if (i + 2 < steps) {
                            const uint32_t item = it0 + k_item(two ? (i + 2) >> 1 : i + 2, two);
                            if (!two || u == 0) ok = ok && ready(item);
                            if (!ok) break;
                            tc_fence_after();
                            tc_fence_order();   // S overwrites the P that the PV before reads
                            const uint64_t qd = q_desc + (two ? u * (32768 >> 4) : 0), kd = k_desc + (item % NS) * (CA_SLOT >> 4);
#pragma unroll
                            for (int k = 0; k < 8; k++) {
                                const uint32_t o = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                                mma_ss(tmem + u * 128, qd + o, kd + o, IDESC, k > 0);
                            }
                            mma_commit(&sh.s_full[u]);
                            if (!two || u == 1) mma_commit(&sh.empty[item % NS]);
                        }
                    }
                    it0 += 2 * n_c;
                    ci += n_c;
                }
                if (!ok) {   // a wait gave up: MMAs in flight end before the CTA leaves
                    mma_commit(&sh.drain);
                    const uint32_t t0 = (uint32_t)clock();
                    while (!mbar_try_wait(&sh.drain, 0) && (uint32_t)clock() - t0 < CA_WAIT_LIMIT) {}
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // --------------------------------------------------------- the walk ---
            Walk w;
            w.r = sh.w_r;
            w.q = sh.w_q;
            w.J = w.q.blocks();
            {
                const long long x = sh.w_x, per = sh.w_per;
                w.h = (int)div_any(x, per);
                const long long y = x - w.h * per;
                int a = 0, b = w.J;   // the block that holds unit y: 32 lanes try as many places at once
                while (b - a > 1) {
                    const int step = (b - a + 31) / 32, at = a + lane * step;
                    const unsigned le = __ballot_sync(CAF, at < b && w.q.before(at) + (long long)ov * at <= y);
                    const int k = 31 - __clz(le);   // lane 0 always holds
                    a += k * step;
                    b = min(b, a + step);
                }
                w.j = a;
                w.off = (int)(y - (a > 0 ? w.q.before(a) + (long long)ov * a : 0));
                w.ov = ov;
                w.left = u1 - u0;
            }
            if (lane == 0) {
                bool more = true;
                for (uint32_t i = 0; more; i++) {
                    Segment s;
                    more = next_segment(p, w, u1, W, P, s);
                    if (!more) s.n_c = -1;
                    if (i >= CA_SEGS && !wait(&sh.seg_empty[i % CA_SEGS], (i / CA_SEGS - 1) & 1)) break;
                    sh.seg[i % CA_SEGS] = s;
                    mbar_arrive1(&sh.seg_full[i % CA_SEGS]);
                }
            }
        }
    } else if (group == 3) {
        // ------------------------------------------------------- preparing ---
        if (ROWS > 128) reg_dec<ALL_F16 ? 80 : 96>();
        const int th = tid - 384;
        uint32_t it = 0, dir = 0, raw = 0, ci = 0;   // operands, those landing as such, raw pages; chunks
        bool ok = true;
        for (; ok && next(); done()) {
            const Segment s = sh.seg[si % CA_SEGS];
            const bool two = ROWS > 128 && s.rows > 128;
            const Seen seen = seen_by(p, s);
            // chunks in [c_a, c_b) are seen whole by every row
            const int c_a = (int)((seen.all_lo + CA_KEYS - 1) / CA_KEYS) - s.c0, c_b = (int)(seen.all_hi / CA_KEYS) - s.c0;
            for (int i = 0; ok && i < 2 * s.n_c; i++, it++) {
                int kv, c;
                item_at(i, s.n_c, two, kv, c);
                const uint32_t sl = it % NS;
                uint8_t *slot = slots + sl * CA_SLOT;
                if (kv ? v16 : k16) {
                    ok = wait.warp(&sh.full[dir % CA_MAX_SLOTS], (dir / CA_MAX_SLOTS) & 1);
                    if (!ok) break;
                    dir++;
                } else {
                    // three waits at once: the slot (lane 0), the raw pages (lanes 1, 2)
                    const uint32_t mine = raw + (lane == 2), rs = mine % NR;
                    bool there = true;
                    if (lane == 0) there = it < NS || wait(&sh.empty[sl], (it / NS - 1) & 1);
                    else if (lane < 3) there = wait(&sh.raw_full[rs], (mine / NR) & 1);
                    ok = __all_sync(CAF, there);
                    __syncwarp();
                    if (!ok) break;
#pragma unroll 1
                    for (int k = 0; k < 2; k++) {
                        const uint8_t *r = raws + ((raw + k) % NR) * CA_RAW;
                        if (kv) {
                            if (p.kv.v_type == KV_T_Q8) prepare_v<true>(r, slot, th, k);
                            else prepare_v<false>(r, slot, th, k);
                        } else {
                            if (p.kv.k_type == KV_T_Q8) prepare_k<true>(r, slot, th, k);
                            else prepare_k<false>(r, slot, th, k);
                        }
                    }
                    __syncwarp();
                    if (lane == 1 || lane == 2) mbar_arrive1(&sh.raw_empty[rs]);
                    raw += 2;
                }
                if (kv) {
                    const int pok = sh.pages_ok[(ci + c) & 7];
                    bool bad = false;
                    if (c < c_a || c >= c_b || pok != 3) {
                        const long long key0 = (long long)(s.c0 + c) * CA_KEYS;
                        const int lo = (int)max(0LL, seen.lo - key0), hi = (int)min((long long)CA_KEYS, seen.hi - key0);
                        clean_v(slot, th, lo, hi, pok);
                        bad = __any_sync(CAF, partly_seen(seen, key0) && v_not_finite(slot, th));
                    }
                    if (lane == 0) reinterpret_cast<uint8_t *>(&sh.bad[(ci + c) & 7])[warp & 3] = bad;
                }
                async_proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sh.ready[sl]);
            }
            ci += s.n_c;
        }
    } else {
        // --------------------------------------------------------- softmax ---
        if (ROWS > 128) reg_inc<ALL_F16 ? 184 : 176>();
        const int u = group - 1, w4 = warp & 3, row = w4 * 32 + lane;     // buffer; TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)w4 << 21);           // lanes 32 (warp % 4) ..
        const uint32_t s_addr = lane_base + u * 128, o_addr = lane_base + 256 + u * 128;
        uint32_t n_s = 0, n_odd = 0, it0 = 0, ci = 0;   // steps of this buffer, joins; operands, chunks before
        bool ok = true;
        for (; ok && next(); done()) {
            const Segment &s = sh.seg[si % CA_SEGS];
            const int n_c = s.n_c, rows = s.rows;
            const bool two = ROWS > 128 && rows > 128;
            const int first = two ? u * 128 : 0;           // this buffer's tile begins at this row of the item
            if (n_c == 0) {                                // nothing is seen
                const int my = u * 128 + row;
                if (my < rows) {
                    const int flat = s.row0 + my, tok = flat / p.G, head = s.h * p.G + flat - tok * p.G;
                    uint4 *out = reinterpret_cast<uint4 *>(p.o + (long long)(s.t0 + tok) * p.o_ld + (long long)head * HD);
                    for (int d = 0; d < 16; d++) out[d] = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
                continue;
            }
            const bool act = first + w4 * 32 < rows;       // a warp without a row only takes part in the barriers
            const int flat = s.row0 + min(first + row, rows - 1);   // rows past the last repeat it
            const int tok = flat / p.G, head = s.h * p.G + flat - tok * p.G;
            const long long pos = s.a + tok;
            float scale = 0.0f;                            // log2 units per score
            if (act) {
                const uint16_t *src = p.q + (long long)(s.t0 + tok) * p.q_ld + (long long)head * HD;
                const bool mine = two || u == 0;
                const int e = mine || p.io_type != ZDEC_F16 ? load_q<ROWS == 128, (ROWS > 128 && !ALL_F16) ? 8 : 4>(src, p.io_type, mine, q_smem + first * 256, w4 * 32, min(32, rows - first - w4 * 32)) : 0;
                scale = fmaxf(ldexpf(p.scale_log2, e), 7.9e-31f);   // never 0 (0 * -inf)
            }
            if (two || u == 0) {
                async_proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sh.q_ready[u]);
            }
            const Seen seen = seen_by(p, s);
            // chunks in [c_a, c_b) are seen whole by every row
            const int c_a = (int)((seen.all_lo + CA_KEYS - 1) / CA_KEYS) - s.c0, c_b = (int)(seen.all_hi / CA_KEYS) - s.c0;
            float m = -INFINITY, ms = 0.0f, l = 0.0f;      // running maximum (raw), m * scale, sum
            const int c_first = two ? 0 : u, c_step = two ? 1 : 2;
            for (int c = c_first; c < n_c; c += c_step, n_s++) {
                ok = wait.warp(&sh.s_full[u], n_s & 1);
                if (!ok) break;
                tc_fence_after();
                if (act) {
                    // S is read once into 128 registers where the tensor core's rate counts; short items, which wait for
                    // memory, read it twice, 64 and 32 columns at a time: a quarter of the code, fewer registers
                    constexpr bool ONCE = ROWS > 128;
                    uint32_t v[ONCE ? 4 : 2][32];
                    if (ONCE) {
#pragma unroll
                        for (int g = 0; g < 4; g++) tmem_ld32(s_addr + 32 * g, v[ONCE ? g : 0]);
                    }
                    const int pok = sh.pages_ok[(ci + c) & 7];
                    int lo = 0, hi = CA_KEYS;              // keys of the chunk that this row sees
                    uint32_t bad = 0;
                    const bool edge = c < c_a || c >= c_b || pok != 3;
                    if (edge) {
                        const long long key0 = (long long)(s.c0 + c) * CA_KEYS;
                        const long long khi = p.causal ? min((long long)s.kv, pos + 1) : s.kv, klo = p.window ? pos + 1 - p.window : 0;
                        lo = (int)max(0LL, min((long long)CA_KEYS, klo - key0));
                        hi = (int)max(0LL, min((long long)CA_KEYS, khi - key0));
                        if (!(pok & 1)) lo = max(lo, 64);
                        if (!(pok & 2)) hi = min(hi, 64);
                        if (partly_seen(seen, key0)) {     // V has been looked through by now
                            const uint32_t vi = it0 + v_item(c, n_c, two);
                            ok = wait.warp(&sh.ready[vi % NS], (vi / NS) & 1);
                            bad = sh.bad[(ci + c) & 7];
                        }
                    }
                    if (ONCE) {
#pragma unroll
                        for (int g = 0; g < 4; g++) tmem_wait_ld(v[ONCE ? g : 0]);
                    }
                    if (!ok) break;
                    float top = -INFINITY;
                    if (ONCE) {
                        if (edge) {
#pragma unroll
                            for (int g = 0; g < 4; g++) hide(v[ONCE ? g : 0], lo - 32 * g, hi - 32 * g);
                        }
                        const float a = max32(v[0]), b = max32(v[1]);
                        top = fmaxf(fmaxf(a, b), fmaxf(max32(v[ONCE ? 2 : 0]), max32(v[ONCE ? 3 : 0])));
                    } else {
#pragma unroll 1
                        for (int g = 0; g < 4; g += 2) {
                            tmem_ld32(s_addr + 32 * g, v[0]);
                            tmem_ld32(s_addr + 32 * g + 32, v[1]);
                            tmem_wait_ld(v[0]);
                            tmem_wait_ld(v[1]);
                            if (edge) {
                                hide(v[0], lo - 32 * g, hi - 32 * g);
                                hide(v[1], lo - 32 * g - 32, hi - 32 * g - 32);
                            }
                            top = fmaxf(top, fmaxf(max32(v[0]), max32(v[1])));
                        }
                    }
                    const bool grow = (top - m) * scale > CA_LAG || (m == -INFINITY && top > m);
                    if (__any_sync(CAF, grow)) {
                        const float m_new = grow ? top : m, ms_new = grow ? top * scale : ms;
                        if (c > c_first) {
                            const float f = grow ? (m == -INFINITY ? 0.0f : exp2_approx(ms - ms_new)) : 1.0f;
                            l *= f;
                            ok = wait.warp(&sh.o_done[u], (n_s - 1) & 1);   // the PV before has finished
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int g = 0; g < 8; g++) {
                                uint32_t x[16];
                                tmem_ld16(o_addr + 16 * g, x);
#pragma unroll
                                for (int k = 0; k < 16; k++) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                                tmem_st16(o_addr + 16 * g, x);
                            }
                        }
                        m = m_new;
                        ms = ms_new;
                    }
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll(ONCE ? 4 : 1)
                    for (int g = 0; g < 4; g++) {
                        if (!ONCE) {                       // P of this group lies over scores that have been read
                            tmem_ld32(s_addr + 32 * g, v[0]);
                            tmem_wait_ld(v[0]);
                            if (edge) hide(v[0], lo - 32 * g, hi - 32 * g);
                        }
                        const uint32_t(&x)[32] = v[ONCE ? g : 0];
                        uint32_t h[16];
#pragma unroll
                        for (int k = 0; k < 16; k++) {
                            float a = __uint_as_float(x[2 * k]), b = __uint_as_float(x[2 * k + 1]);
                            fma_pair(a, b, scale, -ms);
                            a = exp2_approx(a);
                            b = exp2_approx(b);
                            add_pair(sum[2 * (k & 1)], sum[2 * (k & 1) + 1], a, b);
                            h[k] = h2_as_u32(__floats2half2_rn(a, b));
                        }
                        tmem_st16(s_addr + 16 * g, h);
                        if (g == 1 && !bad) {              // the product of the first 64 keys may start
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive1(&sh.p_ready[u][0]);
                        }
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                    if (bad) {
                        // a value that is not finite lies in the chunk and some rows do not see it: 0 times it would be
                        // NaN, so each row adds up what it sees by itself (rare, and slow)
                        if (c > c_first) {
                            ok = wait.warp(&sh.o_done[u], (n_s - 1) & 1);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        const uint8_t *vs = slots + ((it0 + v_item(c, n_c, two)) % NS) * CA_SLOT;
#pragma unroll 1
                        for (int g = 0; g < 8; g++) {
                            uint32_t x[16];
                            tmem_ld16(o_addr + 16 * g, x);
                            if (c == c_first)
#pragma unroll
                                for (int k = 0; k < 16; k++) x[k] = 0u;
#pragma unroll 1
                            for (int j = 0; j < CA_KEYS; j++) {
                                const float2 pp = __half22float2(u32_as_h2(tmem_ld1(s_addr + (j >> 1))));
                                const float pj = j & 1 ? pp.y : pp.x;
                                const bool sees = j >= lo && j < hi;
#pragma unroll
                                for (int k = 0; k < 16; k++)
                                    x[k] = sees ? __float_as_uint(fmaf(pj, v_at(vs, j, 16 * g + k), __uint_as_float(x[k]))) : x[k];
                            }
                            tmem_st16(o_addr + 16 * g, x);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive1(&sh.p_ready[u][0]);
                    }
                } else if (lane == 0) {
                    mbar_arrive1(&sh.p_ready[u][0]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sh.p_ready[u][1]);
            }
            if (!ok) break;
            const bool join = !two && n_c > 1;             // both buffers hold a part of the one tile
            if (act && c_first < n_c) {
                ok = wait.warp(&sh.o_done[u], (n_s - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                float f0 = 1.0f, f1 = 0.0f;
                if (join && u == 1) {
                    sh.odd[row] = make_float2(m == -INFINITY ? m : ms, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(&sh.odd_full[w4]);
                    ok = wait.warp(&sh.odd_read[w4], n_odd & 1);
                    if (!ok) break;
                } else {
                    float mf = m == -INFINITY ? m : ms;
                    if (join) {
                        ok = wait.warp(&sh.odd_full[w4], n_odd & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const float2 o = sh.odd[row];
                        const float top = fmaxf(mf, o.x);
                        f0 = mf == -INFINITY ? 0.0f : exp2f(mf - top);
                        f1 = o.x == -INFINITY ? 0.0f : exp2f(o.x - top);
                        l = f0 * l + f1 * o.y;
                        mf = top;
                    }
                    // rows leave through this warp's part of the Q tile, which no MMA reads any more, in whole lines
                    const bool whole = s.begins && s.ends, valid = first + row < rows;
                    uint8_t *tile = q_smem + first * 256;
                    float *part = part_row(p.ws, cta, s.begins ? 1 : 0, first + row);
                    if (!whole && valid) *reinterpret_cast<float2 *>(part) = make_float2(mf, l);
                    uint8_t *dst = nullptr;
                    if (valid) dst = whole ? (uint8_t *)(p.o + (long long)(s.t0 + tok) * p.o_ld + (long long)head * HD) : (uint8_t *)(part + 4);
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    if (whole) { f0 *= inv; f1 *= inv; }
#pragma unroll 1
                    for (int g = 0; g < 4; g++) {
                        uint32_t x[32], y[32];
                        tmem_ld32(o_addr + 32 * g, x);
                        tmem_ld32(o_addr + (join ? 128 : 0) + 32 * g, y);   // x again where nothing is joined: f1 is 0 then
                        tmem_wait_ld(x);
                        tmem_wait_ld(y);
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            x[k] = __float_as_uint(join ? fmaf(f1, __uint_as_float(y[k]), f0 * __uint_as_float(x[k])) : f0 * __uint_as_float(x[k]));
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < 16; k++) x[k] = pack_out(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]), p.io_type);
#pragma unroll
                            for (int k = 0; k < 4; k++) stage(tile, row, 4 * g + k, x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; k++)
                                stage(tile, row, 8 * (g & 1) + k, x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                        }
                        if (whole ? g == 3 : g & 1) flush_rows(tile, w4 * 32, min(32, rows - first - w4 * 32), !dst || whole ? dst : dst + 256 * (g >> 1));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (join && lane == 0) mbar_arrive1(&sh.odd_read[w4]);
                }
                if (join) n_odd++;
            }
            if (s.begins && !s.ends && u == 0 && row == 0) {
                desc->t0 = s.t0;
                desc->h = s.h;
                desc->row0 = s.row0;
                desc->rows = s.rows;
                desc->last = s.last;
                desc->valid = 1;
            }
            it0 += 2 * n_c;
            ci += n_c;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the item that CTA blockIdx.x began and a later one
// ended, in key order, a row per half warp, eight dims per lane.  Items of 256
// rows have few pieces: one pass with the running maximum and many warps per
// SM.  Items of 128 rows (MANY) may have a piece of every CTA and few rows:
// sixteen pieces at a time, lane i the statistics of the i-th, the sums behind
// them with eight rows in flight (one sequence's token over 2048: 18.4 us with
// the other form, 14.7 with this; prompts over a mixed batch 119 and 123).
template <bool MANY>
__global__ __launch_bounds__(256) void chunk_combine_kernel(const __grid_constant__ ChunkAttnParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const CaDesc *d = reinterpret_cast<const CaDesc *>(p.ws) + blockIdx.x;
    if (!d->valid) return;
    const int lane = threadIdx.x & 15, up = (threadIdx.x >> 4) & 1, first = blockIdx.x, last = d->last, rows = d->rows;
    for (int base = blockIdx.y * 16 + (threadIdx.x >> 5) * 2; base < rows; base += CA_COMBINE_Y * 16) {
        const int row = min(base + up, rows - 1);
        float m = -INFINITY, l = 0.0f, y[8] = {};
        if (MANY) {
            for (int c0 = first; c0 <= last; c0 += 16) {
                const int n = min(16, last + 1 - c0);
                float4 v[8][2];
                auto fetch = [&](int i0) {   // up to eight pieces' rows in flight
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        v[i][0] = v[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (i0 + i < n) {
                            const float4 *r = reinterpret_cast<const float4 *>(part_row(p.ws, c0 + i0 + i, c0 + i0 + i == first ? 1 : 0, row) + 4) + 2 * lane;
                            v[i][0] = r[0];
                            v[i][1] = r[1];
                        }
                    }
                };
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (lane < n) ml = *reinterpret_cast<const float2 *>(part_row(p.ws, c0 + lane, c0 + lane == first ? 1 : 0, row));
                fetch(0);
                float top = ml.x;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(CAF, top, o));
                top = fmaxf(top, m);
                const float f0 = m == -INFINITY ? 0.0f : exp2_approx(m - top), f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
                float sum = f * ml.y;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(CAF, sum, o);
                m = top;
                l = f0 * l + sum;
#pragma unroll
                for (int k = 0; k < 8; k++) y[k] *= f0;
#pragma unroll 1
                for (int i0 = 0;;) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float fi = __shfl_sync(CAF, f, i0 + i, 16);
                        y[0] = fmaf(fi, v[i][0].x, y[0]); y[1] = fmaf(fi, v[i][0].y, y[1]);
                        y[2] = fmaf(fi, v[i][0].z, y[2]); y[3] = fmaf(fi, v[i][0].w, y[3]);
                        y[4] = fmaf(fi, v[i][1].x, y[4]); y[5] = fmaf(fi, v[i][1].y, y[5]);
                        y[6] = fmaf(fi, v[i][1].z, y[6]); y[7] = fmaf(fi, v[i][1].w, y[7]);
                    }
                    i0 += 8;
                    if (i0 >= n) break;
                    fetch(i0);
                }
            }
        } else {
#pragma unroll 4
            for (int c = first; c <= last; c++) {
                const float *r = part_row(p.ws, c, c == first ? 1 : 0, row);
                const float2 ml = *reinterpret_cast<const float2 *>(r);
                const float4 a = *reinterpret_cast<const float4 *>(r + 4 + 8 * lane), b = *reinterpret_cast<const float4 *>(r + 8 + 8 * lane);
                const float top = fmaxf(m, ml.x);
                const float f0 = m == -INFINITY ? 0.0f : exp2_approx(m - top), f1 = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
                m = top;
                l = f0 * l + f1 * ml.y;
                y[0] = f0 * y[0] + f1 * a.x; y[1] = f0 * y[1] + f1 * a.y; y[2] = f0 * y[2] + f1 * a.z; y[3] = f0 * y[3] + f1 * a.w;
                y[4] = f0 * y[4] + f1 * b.x; y[5] = f0 * y[5] + f1 * b.y; y[6] = f0 * y[6] + f1 * b.z; y[7] = f0 * y[7] + f1 * b.w;
            }
        }
        if (base + up >= rows) continue;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int flat = d->row0 + row, tok = flat / p.G, head = d->h * p.G + flat - tok * p.G;
        uint16_t *out = p.o + (long long)(d->t0 + tok) * p.o_ld + (long long)head * HD + 8 * lane;
        *reinterpret_cast<uint4 *>(out) =
            make_uint4(pack_out(y[0] * inv, y[1] * inv, p.io_type), pack_out(y[2] * inv, y[3] * inv, p.io_type),
                       pack_out(y[4] * inv, y[5] * inv, p.io_type), pack_out(y[6] * inv, y[7] * inv, p.io_type));
    }
}

// ------------------------------------------------------------------ launch ---
// K regions of an fp16 pool as a tensor: (64 elements, 2 row halves, 64 keys,
// (layer, head) chunks of a page, pages); a box is one row half of one region.
static cudaError_t make_k_map(const ChunkAttnParams &p, CUtensorMap *map) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (Encode)fn;
    }();
    if (!encode) return cudaErrorNotSupported;
    const uint32_t chunk = kv_region_bytes(p.kv.k_type) + kv_region_bytes(p.kv.v_type);
    const cuuint64_t dims[5] = {64, 2, 64, (cuuint64_t)p.kv.n_layers * p.kv.n_kv, (cuuint64_t)p.kv.n_pages};
    const cuuint64_t strides[4] = {128, 256, chunk, p.kv.page_bytes};
    const cuuint32_t box[5] = {64, 1, 64, 1, 1}, step[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, p.kv.base, dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int ROWS, bool ALL_F16>
constexpr int ca_smem = CaLayout<ROWS, ALL_F16>::BYTES + CA_SHARED_BYTES;
template <int ROWS, bool ALL_F16>
static cudaError_t allow_smem() {
    static_assert(ca_smem<ROWS, ALL_F16> <= 232448, "shared memory of an SM");
    return cudaFuncSetAttribute(chunk_attention_kernel<ROWS, ALL_F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, ca_smem<ROWS, ALL_F16>);
}
template <int ROWS, bool ALL_F16>
static cudaError_t run(const ChunkAttnParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream) {
    return launch_k(chunk_attention_kernel<ROWS, ALL_F16>, dim3(ctas), dim3(CA_THREADS), ca_smem<ROWS, ALL_F16>, ROWS == 128, 1, stream, p, map);
}

cudaError_t launch_chunk_attention(const ChunkAttnParams &p0, cudaStream_t stream) {
    ChunkAttnParams p = p0;
    // Items of 256 rows share each chunk of keys between two tiles; where requests have few tokens (as single-token
    // steps do) most would hold one tile, whose shared memory then serves better for chunks on their way.
    p.rows = (long long)p.T * p.G > 128LL * p.R ? 256 : 128;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> known[64];   // SMs of a device whose kernel attributes are set
    int sms = dev < 64 ? known[dev].load() : 0;
    if (sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = allow_smem<256, true>();
        if (e == cudaSuccess) e = allow_smem<256, false>();
        if (e == cudaSuccess) e = allow_smem<128, true>();
        if (e == cudaSuccess) e = allow_smem<128, false>();
        if (e != cudaSuccess) return e;
        if (dev < 64) known[dev].store(sms);
    }
    CUtensorMap map = {};
    if (p.kv.k_type == KV_T_F16 && (e = make_k_map(p, &map)) != cudaSuccess) return e;
    const int ctas = std::min(sms, CA_MAX_CTAS);
    const bool f16 = p.kv.k_type == KV_T_F16 && p.kv.v_type == KV_T_F16;
    if (p.rows > 128) e = f16 ? run<256, true>(p, map, ctas, stream) : run<256, false>(p, map, ctas, stream);
    else e = f16 ? run<128, true>(p, map, ctas, stream) : run<128, false>(p, map, ctas, stream);
    if (e != cudaSuccess) return e;
    return launch_k(p.rows > 128 ? chunk_combine_kernel<false> : chunk_combine_kernel<true>, dim3(ctas, CA_COMBINE_Y), dim3(256), 0, true, 1, stream, p);
}

}  // namespace zdec
