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
// A CTA (one per SM, persistent) holds two tiles of 128 rows, so that one
// tile's softmax runs while the tensor core works on the other.  TMEM: S/P of
// both tiles 2 x 128 columns, O of both 2 x 128: all 512.
//
// Warps: 0 copies (TMA), 1 issues the MMAs, 2 walks the line, 4-7 and 8-11 are the softmax of
// tile 0 and 1, 12-15 prepare K and V.
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
#include <cuda.h>

#include "chunk.cuh"
#include "chunk_sched.cuh"
#include "tcgen05.cuh"

namespace zdec {

constexpr uint32_t CAF = 0xFFFFFFFFu;
constexpr int CA_THREADS = 512, CA_MAX_CTAS = 160;
constexpr int CA_SLOT = 32768;                     // bytes of a K or V operand chunk
constexpr int CA_RAW = 2 * 8704;                   // bytes of two raw one-byte regions
constexpr int CA_MAX_SLOTS = 5, CA_MAX_RAW = 3;    // fp16 cache: 5 operand slots; else 3 and 3 raw ones
constexpr int CA_Q_BYTES = 2 * 32768;
constexpr int CA_SMEM = 1024 + CA_Q_BYTES + CA_MAX_SLOTS * CA_SLOT;
constexpr long long CA_WAIT_LIMIT = 1LL << 32;     // clock cycles (~2 s)
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
    q.TP = CA_ROWS / p.G;
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
    const int chunks = w.q.chunks(w.j), weight = max(1, chunks);
    const int take = (int)min((long long)(weight - w.off), w.left);
    s.h = w.h;
    s.r = w.r;
    s.row0 = w.j * w.q.TP * p.G;
    s.rows = min(w.q.TP, w.q.neff - w.j * w.q.TP) * p.G;
    s.t0 = w.q.t0;
    s.a = w.q.a;
    s.kv = w.q.kv;
    s.c0 = w.q.c_lo(w.j) + w.off;
    s.n_c = chunks > 0 ? take : 0;
    s.begins = w.off == 0;
    s.ends = w.off + take == weight;
    w.left -= take;
    w.off += take;
    // this CTA's range ends here: the item's last unit is at u1 + what is left of it
    s.last = s.ends ? 0 : (int)(((u1 + weight - w.off) * P + W - 1) / W) - 1;
    if (s.ends) {
        w.off = 0;
        w.j++;
    }
    return true;
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
struct CaShared {
    uint64_t full[CA_MAX_SLOTS], ready[CA_MAX_SLOTS], empty[CA_MAX_SLOTS];
    uint64_t raw_full[CA_MAX_RAW], raw_empty[CA_MAX_RAW];
    uint64_t q_ready[2], s_full[2], p_ready[2], o_done[2], drain;
    uint64_t seg_full[CA_SEGS], seg_empty[CA_SEGS];
    Segment seg[CA_SEGS];
    uint32_t tmem;
    int abort;
    int pages_ok[8];          // chunk i (mod 8): bit k, page k of it is in the pool
    uint32_t bad[8];          // one byte per preparing warp: a value that only some rows see is not finite
    int w_r, w_h, w_j, w_off;
    long long scan[CA_THREADS / 32], total;
};

struct Waiter {
    volatile int *abort;
    uint32_t *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*abort) return false;
            if (clock64() - t0 > CA_WAIT_LIMIT) {
                *abort = 1;
                if (status) atomicOr(status, (uint32_t)ZDEC_CHUNK_TIMEOUT);
                return false;
            }
        }
        return true;
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
// code * scale, at most fp16's largest value (127 x a scale of 516 rounds past it); a NaN stays one
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
    const __half2 top = __float2half2_rn(65504.0f);
    return h2_as_u32(__hmin2_nan(__hmax2_nan(__hmul2(u32_as_h2(a), u32_as_h2(b)), __hneg2(top)), top));
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

// K: thread = key of the chunk (0..127); both raw pages -> [half][128 keys][128 bytes], SW128.
template <bool Q8>
__device__ __forceinline__ void prepare_k(const uint8_t *raw, uint8_t *slot, int key) {
    const int t = key & 63;
    const uint8_t *reg = raw + (key >> 6) * kv_region_bytes(Q8 ? KV_T_Q8 : KV_T_FP8);
    uint2 sc = make_uint2(0u, 0u);
    if (Q8) sc = *reinterpret_cast<const uint2 *>(reg + ks_off(t, 0));
#pragma unroll
    for (int s = 0; s < 8; s++) {   // 16 dims
        uint4 lo, hi;
        codes16<Q8>(*reinterpret_cast<const uint4 *>(reg + k8_off(t, 16 * s)), lo, hi);
        if (Q8) {
            const uint32_t two = s < 4 ? sc.x : sc.y, d = (s >> 1) & 1 ? (two >> 16) : (two & 0xFFFFu), dd = d | (d << 16);
            const uint4 d4 = make_uint4(dd, dd, dd, dd);
            lo = hmul8(lo, d4);
            hi = hmul8(hi, d4);
        }
        uint8_t *row = slot + (s >> 2) * 16384 + key * 128;
        const int g = 2 * (s & 3);
        *reinterpret_cast<uint4 *>(row + ((g ^ (t & 7)) << 4)) = lo;
        *reinterpret_cast<uint4 *>(row + (((g + 1) ^ (t & 7)) << 4)) = hi;
    }
}
// V: thread = dim; both raw pages -> [unit of 32 tokens][128 dims][64 bytes],
// SW64, tokens outside [lo, hi) of the chunk or of a missing page zero.
template <bool Q8>
__device__ __forceinline__ void prepare_v(const uint8_t *raw, uint8_t *slot, int d, int lo, int hi, int pages_ok) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const uint8_t *reg = raw + (u >> 1) * kv_region_bytes(Q8 ? KV_T_Q8 : KV_T_FP8);
        const bool there = (pages_ok >> (u >> 1)) & 1;
#pragma unroll
        for (int s = 0; s < 2; s++) {   // 16 tokens
            const int t = 32 * (u & 1) + 16 * s, c0 = 32 * u + 16 * s;   // within the page, within the chunk
            uint4 a, b;
            codes16<Q8>(*reinterpret_cast<const uint4 *>(reg + v8_off(t, d)), a, b);
            if (Q8) {
                a = hmul8(a, *reinterpret_cast<const uint4 *>(reg + vs_off(t, d >> 5)));
                b = hmul8(b, *reinterpret_cast<const uint4 *>(reg + vs_off(t + 8, d >> 5)));
            }
            a = there ? keep8(a, lo - c0, hi - c0) : make_uint4(0u, 0u, 0u, 0u);
            b = there ? keep8(b, lo - c0 - 8, hi - c0 - 8) : make_uint4(0u, 0u, 0u, 0u);
            uint8_t *row = slot + u * 8192 + d * 64;
            *reinterpret_cast<uint4 *>(row + (((2 * s) ^ ((d >> 1) & 3)) << 4)) = a;
            *reinterpret_cast<uint4 *>(row + (((2 * s + 1) ^ ((d >> 1) & 3)) << 4)) = b;
        }
    }
}
// fp16 V that landed as an operand: the same zeroing in place.
__device__ __forceinline__ void clean_v(uint8_t *slot, int d, int lo, int hi, int pages_ok) {
    for (int u = 0; u < 4; u++) {
        const bool there = (pages_ok >> (u >> 1)) & 1;
        if (there && 32 * u >= lo && 32 * u + 32 <= hi) continue;
        for (int g = 0; g < 4; g++) {
            uint4 *at = reinterpret_cast<uint4 *>(slot + u * 8192 + d * 64 + ((g ^ ((d >> 1) & 3)) << 4));
            const int c0 = 32 * u + 8 * g;
            *at = there ? keep8(*at, lo - c0, hi - c0) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// Whether dim d of a V operand chunk holds an infinity or a NaN.
__device__ __forceinline__ bool v_not_finite(const uint8_t *slot, int d) {
    bool bad = false;
    for (int u = 0; u < 4; u++)
        for (int g = 0; g < 4; g++) {
            const uint4 v = *reinterpret_cast<const uint4 *>(slot + u * 8192 + d * 64 + (g << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            for (int i = 0; i < 4; i++) bad = bad || (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
        }
    return bad;
}
__device__ __forceinline__ float v_at(const uint8_t *slot, int j, int d) {
    return __half2float(*reinterpret_cast<const __half *>(slot + (j >> 5) * 8192 + d * 64 +
                                                          ((((j & 31) >> 3) ^ ((d >> 1) & 3)) << 4) + (j & 7) * 2));
}

// One row of Q: fp16 as it is, bf16 scaled by a power of two into fp16's range
// (exact but for elements below 2^-28 of the row's largest).  Returns the
// exponent taken out.
__device__ __forceinline__ int load_q_row(const ChunkAttnParams &p, const uint16_t *src, bool valid, uint8_t *tile, int row) {
    uint8_t *dst = tile + row * 128;
    auto put = [&](int c, uint4 v) {
        *reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4)) = v;
    };
    if (!valid) {
#pragma unroll
        for (int c = 0; c < 16; c++) put(c, make_uint4(0u, 0u, 0u, 0u));
        return 0;
    }
    const uint4 *s4 = reinterpret_cast<const uint4 *>(src);
    if (p.io_type == ZDEC_F16) {
#pragma unroll
        for (int c = 0; c < 16; c++) put(c, __ldg(s4 + c));
        return 0;
    }
    uint32_t top = 0;   // largest magnitude bits of the row
#pragma unroll
    for (int c = 0; c < 16; c++) {
        const uint4 v = __ldg(s4 + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    }
    const int ex = (int)(top >> 7);   // biased exponent
    const int e = ex == 0 || ex == 255 ? 0 : ex - 127 - 14;
    const float f = exp2f((float)-e);   // e in [-140, 113]; 2^140 is past fp32: two steps below
    const float f1 = e < -100 ? exp2f(100.0f) : f, f2 = e < -100 ? exp2f((float)(-e - 100)) : 1.0f;
#pragma unroll
    for (int c = 0; c < 16; c++) {
        const uint4 v = __ldg(s4 + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            o[i] = h2_as_u32(__floats2half2_rn(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2));
        put(c, make_uint4(o[0], o[1], o[2], o[3]));
    }
    return e;
}

// 32 fp32 values of a row, times inv, as fp16 or bf16.
__device__ __forceinline__ void store_o32(uint16_t *dst, const float *v, float inv, int io_type) {
#pragma unroll
    for (int c = 0; c < 4; c++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float x = v[8 * c + 2 * i] * inv, y = v[8 * c + 2 * i + 1] * inv;
            if (io_type == ZDEC_F16) w[i] = h2_as_u32(__floats2half2_rn(x, y));
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y), "f"(x));
        }
        reinterpret_cast<uint4 *>(dst)[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ kernel ---
__global__ __launch_bounds__(CA_THREADS, 1) void chunk_attention_kernel(const __grid_constant__ ChunkAttnParams p,
                                                                        const __grid_constant__ CUtensorMap k_map) {
    extern __shared__ uint8_t dyn[];
    __shared__ CaShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    const bool k16 = p.kv.k_type == KV_T_F16, v16 = p.kv.v_type == KV_T_F16;
    const int NS = k16 && v16 ? CA_MAX_SLOTS : 3;
    uint8_t *q_smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    uint8_t *slots = q_smem + CA_Q_BYTES, *raws = slots + 3 * CA_SLOT;
    CaDesc *desc = reinterpret_cast<CaDesc *>(p.ws) + cta;

    // ---- this CTA's piece of the line
    long long W = 0;
    for (int r0 = 0; r0 < p.R; r0 += CA_THREADS) {
        long long w = 0;
        if (r0 + tid < p.R) {
            const ChunkReq q = load_req(p, r0 + tid);
            w = q.before(q.blocks());
        }
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(CAF, w, o);
        if (lane == 0) sh.scan[warp] = w;
        __syncthreads();
        for (int i = 0; i < CA_THREADS / 32; i++) W += sh.scan[i];
        __syncthreads();
    }
    W *= p.kv.n_kv;
    const int P = (int)min((long long)gridDim.x, W);   // every CTA of the first P has work: pieces follow each other
    const long long u0 = cta < P ? W * cta / P : 0, u1 = cta < P ? W * (cta + 1) / P : 0;
    if (tid == 0) {
        desc->valid = 0;
        sh.abort = 0;
    }
    if (u0 >= u1) {
        pdl_launch_dependents();
        return;
    }
    long long base = 0;
    for (int r0 = 0; r0 < p.R; r0 += CA_THREADS) {
        ChunkReq q;
        long long w = 0;
        if (r0 + tid < p.R) {
            q = load_req(p, r0 + tid);
            w = q.before(q.blocks()) * p.kv.n_kv;
        }
        long long incl = w;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(CAF, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        long long excl = base + incl - w;
        for (int i = 0; i < warp; i++) excl += sh.scan[i];
        if (w > 0 && excl <= u0 && u0 < excl + w) {
            const long long per = w / p.kv.n_kv, x = u0 - excl;
            sh.w_r = r0 + tid;
            sh.w_h = (int)(x / per);
            sh.w_j = q.block_at(x % per);
            sh.w_off = (int)(x % per - q.before(sh.w_j));
        }
        for (int i = 0; i < CA_THREADS / 32; i++) base += sh.scan[i];
        __syncthreads();
        if (base > u0) break;
    }
    if (tid == 0) {
        for (int i = 0; i < CA_MAX_SLOTS; i++) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.ready[i], 4);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < CA_MAX_RAW; i++) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        for (int t = 0; t < 2; t++) {
            mbar_init(&sh.q_ready[t], 4);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_ready[t], 4);
            mbar_init(&sh.o_done[t], 1);
        }
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < CA_SEGS; i++) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], CA_SEG_READERS);
        }
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
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

    if (group == 0) {
        reg_dec<64>();
        if (warp == 0) {
            // ------------------------------------------------------ copies ---
            const uint32_t kb = kv_region_bytes(p.kv.k_type), vb = kv_region_bytes(p.kv.v_type);
            const size_t coff = kv_chunk_off(p.kv, p.layer, 0);
            uint32_t it = 0, dir = 0, raw = 0, ci = 0;   // operands, those landing as such, raw ones; chunks
            bool ok = true;
            for (; ok && next(); done()) {
                const Segment s = sh.seg[si % CA_SEGS];
                const int32_t *row = p.kv.table + (size_t)s.r * p.kv.max_pages;
                const size_t off = coff + (size_t)s.h * (kb + vb);
                int mine = -1;
                for (int c = 0; ok && c < s.n_c; c++, ci++) {
                    if ((c & 15) == 0) {   // the pages of the next 16 chunks, one per lane
                        const long long pg = (long long)(s.c0 + c) * 2 + lane;
                        mine = pg < p.kv.max_pages && pg * 64 < s.kv ? __ldg(row + pg) : -2;   // -2: no key there
                    }
                    const int pa = __shfl_sync(CAF, mine, 2 * (c & 15)), pb = __shfl_sync(CAF, mine, 2 * (c & 15) + 1);
                    const int okm = (kv_page_ok(p.kv, pa) ? 1 : 0) | (kv_page_ok(p.kv, pb) ? 2 : 0);
                    if (lane == 0) {
                        if (p.status && ((!(okm & 1) && pa != -2) || (!(okm & 2) && pb != -2)))
                            atomicOr(p.status, (uint32_t)ZDEC_CHUNK_NO_PAGE);
                        for (int kv = 0; ok && kv < 2; kv++, it++) {   // K, then V
                            const bool direct = kv ? v16 : k16;
                            const uint32_t bytes = kv ? vb : kb;
                            uint8_t *dst;
                            uint64_t *bar;
                            if (direct) {
                                const uint32_t sl = it % NS;
                                ok = it < (uint32_t)NS || wait(&sh.empty[sl], (it / NS - 1) & 1);
                                dst = slots + sl * CA_SLOT;
                                bar = &sh.full[dir % CA_MAX_SLOTS];
                                dir++;
                            } else {
                                const uint32_t sl = raw % CA_MAX_RAW;
                                ok = raw < (uint32_t)CA_MAX_RAW || wait(&sh.raw_empty[sl], (raw / CA_MAX_RAW - 1) & 1);
                                dst = raws + sl * CA_RAW;
                                bar = &sh.raw_full[sl];
                                raw++;
                            }
                            if (!ok) break;
                            // chunk ci's entry was last read for chunk ci - 8, whose operands have left their slots
                            if (kv == 0) sh.pages_ok[ci & 7] = okm;
                            const int n = __popc(okm);
                            if (n) mbar_expect_tx(bar, n * bytes);
                            else mbar_arrive1(bar);
                            for (int k = 0; k < 2; k++) {
                                if (!((okm >> k) & 1)) continue;
                                const int page = k ? pb : pa;
                                const uint8_t *src = p.kv.base + (size_t)page * p.kv.page_bytes + off + (kv ? kb : 0);
                                if (!direct) bulk_g2s(dst + k * bytes, src, bytes, bar);
                                else if (kv) bulk_g2s(dst + k * 16384, src, bytes, bar);
                                else
                                    for (int half = 0; half < 2; half++)
                                        tma_k_half(dst + half * 16384 + k * 8192, &k_map, half, p.layer * p.kv.n_kv + s.h, page, bar);
                            }
                        }
                    }
                    ok = __shfl_sync(CAF, (int)ok, 0);
                }
            }
            // copies in flight land before the CTA leaves, also where a wait gave up
            if (lane == 0 && sh.abort) {
                const long long t0 = clock64();
                for (uint32_t i = dir > (uint32_t)CA_MAX_SLOTS ? dir - CA_MAX_SLOTS : 0; i < dir; i++)
                    while (!mbar_try_wait(&sh.full[i % CA_MAX_SLOTS], (i / CA_MAX_SLOTS) & 1) && clock64() - t0 < CA_WAIT_LIMIT) {}
                for (uint32_t i = raw > (uint32_t)CA_MAX_RAW ? raw - CA_MAX_RAW : 0; i < raw; i++)
                    while (!mbar_try_wait(&sh.raw_full[i % CA_MAX_RAW], (i / CA_MAX_RAW) & 1) && clock64() - t0 < CA_WAIT_LIMIT) {}
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------- MMA ---
            constexpr uint32_t IDESC = MMA_IDESC_F16<128, 128>;
            const uint32_t q_addr = smem_u32(q_smem), slot_addr = smem_u32(slots);
            const bool leader = lane == 0;
            uint32_t it = 0, ci = 0, segs[2] = {0, 0}, n_p[2] = {0, 0};   // operands, chunks; segments and PVs per tile
            bool ok = true;
            auto qk = [&](int t, uint32_t sl) {
                const uint32_t qa = q_addr + t * 32768, ka = slot_addr + sl * CA_SLOT;
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const uint32_t o = (k >> 2) * 16384 + (k & 3) * 32;
                    mma_ss(tmem + t * 128, mma_desc_sw128(qa + o), mma_desc_sw128(ka + o), IDESC, k > 0);
                }
                mma_commit(&sh.s_full[t]);
            };
            auto pv = [&](int t, uint32_t sl, bool first, bool bad) {
                // a chunk whose product the softmax threads make themselves only reports
                if (bad) { mma_commit(&sh.o_done[t]); return; }
                const uint32_t va = slot_addr + sl * CA_SLOT;
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, mma_desc_sw64(va + (k >> 1) * 8192 + (k & 1) * 32), IDESC,
                           !first || k > 0);
                mma_commit(&sh.o_done[t]);
            };
            for (; ok && next(); done()) {
                const int n_c = sh.seg[si % CA_SEGS].n_c, nt = sh.seg[si % CA_SEGS].rows > 128 ? 2 : 1;
                if (n_c == 0) continue;
                for (int t = 0; t < nt; t++) ok = ok && wait.warp(&sh.q_ready[t], segs[t]++ & 1);
                uint32_t ks = it % NS;
                ok = ok && wait.warp(&sh.ready[ks], (it / NS) & 1);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    for (int t = 0; t < nt; t++) qk(t, ks);
                    mma_commit(&sh.empty[ks]);
                }
                it++;
                for (int c = 0; ok && c < n_c; c++, ci++) {
                    const uint32_t vi = it, ki = it + 1;   // V of this chunk, K of the next
                    const bool more = c + 1 < n_c;
                    ok = wait.warp(&sh.ready[vi % NS], (vi / NS) & 1);
                    for (int t = 0; ok && t < nt; t++) {
                        ok = wait.warp(&sh.p_ready[t], n_p[t] & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            pv(t, vi % NS, c == 0, sh.bad[ci & 7] != 0);
                            if (t == nt - 1) mma_commit(&sh.empty[vi % NS]);
                        }
                        if (more) {
                            if (t == 0) ok = wait.warp(&sh.ready[ki % NS], (ki / NS) & 1);
                            // the next S overwrites the P that this PV reads
                            ok = ok && wait.warp(&sh.o_done[t], n_p[t] & 1);
                            if (!ok) break;
                            tc_fence_after();
                            if (leader) {
                                qk(t, ki % NS);
                                if (t == nt - 1) mma_commit(&sh.empty[ki % NS]);
                            }
                        }
                        n_p[t]++;
                    }
                    it += more ? 2 : 1;
                }
            }
            if (!ok) {   // a wait gave up: MMAs in flight end before the CTA leaves
                if (leader) mma_commit(&sh.drain);
                const long long t0 = clock64();
                while (!mbar_try_wait(&sh.drain, 0) && clock64() - t0 < CA_WAIT_LIMIT) {}
            }
        } else if (warp == 2) {
            // ----------------------------------------------------- the walk ---
            if (lane == 0) {
                Walk w;
                w.r = sh.w_r;
                w.h = sh.w_h;
                w.j = sh.w_j;
                w.off = sh.w_off;
                w.left = u1 - u0;
                w.q = load_req(p, w.r);
                w.J = w.q.blocks();
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
        reg_dec<64>();
        const int th = tid - 384;
        uint32_t it = 0, dir = 0, raw = 0, ci = 0;
        bool ok = true;
        for (; ok && next(); done()) {
            const Segment s = sh.seg[si % CA_SEGS];
            const Seen seen = seen_by(p, s);
            for (int c = 0; ok && c < s.n_c; c++, ci++) {
                const long long key0 = (long long)(s.c0 + c) * CA_KEYS;
                const int vlo = (int)max(0LL, seen.lo - key0), vhi = (int)min((long long)CA_KEYS, seen.hi - key0);
                const bool part = partly_seen(seen, key0);
                for (int kv = 0; ok && kv < 2; kv++, it++) {
                    const uint32_t sl = it % NS;
                    uint8_t *slot = slots + sl * CA_SLOT;
                    if (kv ? v16 : k16) {
                        ok = wait.warp(&sh.full[dir % CA_MAX_SLOTS], (dir / CA_MAX_SLOTS) & 1);
                        if (!ok) break;
                        dir++;
                        const int pok = sh.pages_ok[ci & 7];
                        if (kv && (vlo > 0 || vhi < CA_KEYS || pok != 3)) {
                            clean_v(slot, th, vlo, vhi, pok);
                            async_proxy_fence();
                        }
                    } else {
                        const uint32_t rs = raw % CA_MAX_RAW;
                        ok = wait.warp(&sh.raw_full[rs], (raw / CA_MAX_RAW) & 1) &&
                             (it < (uint32_t)NS || wait.warp(&sh.empty[sl], (it / NS - 1) & 1));
                        if (!ok) break;
                        const uint8_t *src = raws + rs * CA_RAW;
                        if (kv) {
                            const int pok = sh.pages_ok[ci & 7];
                            if (p.kv.v_type == KV_T_Q8) prepare_v<true>(src, slot, th, vlo, vhi, pok);
                            else prepare_v<false>(src, slot, th, vlo, vhi, pok);
                        } else {
                            if (p.kv.k_type == KV_T_Q8) prepare_k<true>(src, slot, th);
                            else prepare_k<false>(src, slot, th);
                        }
                        async_proxy_fence();
                        __syncwarp();
                        if (lane == 0) mbar_arrive1(&sh.raw_empty[rs]);
                        raw++;
                    }
                    if (kv) {
                        const bool bad = __any_sync(CAF, part && v_not_finite(slot, th));
                        if (lane == 0) reinterpret_cast<uint8_t *>(&sh.bad[ci & 7])[warp & 3] = bad;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(&sh.ready[sl]);
                }
            }
        }
    } else {
        // --------------------------------------------------------- softmax ---
        reg_inc<192>();
        const int t = group - 1;                       // tile
        const int row = tid - 128 - 128 * t;           // row of the tile = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);   // lanes 32 (warp % 4) ..
        const uint32_t s_addr = lane_base + t * 128, o_addr = lane_base + 256 + t * 128;
        uint32_t n_s = 0, ci = 0;                      // chunks of this tile, of the CTA
        bool ok = true;
        for (; ok && next(); done()) {
            const Segment &s = sh.seg[si % CA_SEGS];
            const int n_c = s.n_c;
            const int first_row = t * 128, my = first_row + row;
            if (first_row >= s.rows) {                 // no row of this tile in the item
                ci += n_c;
                continue;
            }
            const bool valid = my < s.rows;
            const int flat = s.row0 + min(my, s.rows - 1);
            const int tok = flat / p.G, head = s.h * p.G + flat % p.G;
            uint16_t *out = p.o + (long long)(s.t0 + tok) * p.o_ld + (long long)head * HD;
            if (n_c == 0) {                            // nothing is seen
                if (valid) {
                    const float zero[32] = {};
                    for (int d = 0; d < 4; d++) store_o32(out + 32 * d, zero, 0.0f, p.io_type);
                }
                __syncwarp();
                continue;
            }
            const int e = load_q_row(p, p.q + (long long)(s.t0 + tok) * p.q_ld + (long long)head * HD, valid,
                                     q_smem + t * 32768, row);
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive1(&sh.q_ready[t]);
            const float sc = fmaxf(ldexpf(p.scale_log2, e), 7.9e-31f);   // log2 units per score; never 0 (0 * -inf)
            const float lag = CA_LAG / sc;
            const long long pos = s.a + tok;              // keys [klo, khi) of this row
            const long long khi = p.causal ? min((long long)s.kv, pos + 1) : s.kv;
            const long long klo = p.window ? pos + 1 - p.window : 0;
            const Seen seen = seen_by(p, s);
            float m = -INFINITY, msc = 0.0f, l = 0.0f;   // running maximum (raw), m * sc, sum
            for (int c = 0; ok && c < n_c; c++, ci++, n_s++) {
                ok = wait.warp(&sh.s_full[t], n_s & 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int g = 0; g < 4; g++) tmem_ld32(s_addr + 32 * g, v[g]);
#pragma unroll
                for (int g = 0; g < 4; g++) tmem_wait_ld(v[g]);
                const long long key0 = (long long)(s.c0 + c) * CA_KEYS;
                const int pok = sh.pages_ok[ci & 7];
                int lo2 = 0, hi2 = CA_KEYS;
                uint32_t bad = 0;
                if (key0 + CA_KEYS > seen.all_hi || key0 < seen.all_lo || pok != 3) {
                    lo2 = (int)max(0LL, min((long long)CA_KEYS, klo - key0));
                    hi2 = (int)max(0LL, min((long long)CA_KEYS, khi - key0));
                    if (!(pok & 1)) lo2 = max(lo2, 64);
                    if (!(pok & 2)) hi2 = min(hi2, 64);
                    if (partly_seen(seen, key0)) {       // V has been looked through by now
                        const uint32_t vi = 2 * ci + 1;
                        ok = wait.warp(&sh.ready[vi % NS], (vi / NS) & 1);
                        if (!ok) break;
                        bad = sh.bad[ci & 7];
                    }
#pragma unroll
                    for (int g = 0; g < 4; g++)
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            if (32 * g + i < lo2 || 32 * g + i >= hi2) v[g][i] = 0xFF800000u;   // -inf
                }
                float mx[4];
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    mx[g] = __uint_as_float(v[g][0]);
#pragma unroll
                    for (int i = 1; i < 32; i++) mx[g] = fmaxf(mx[g], __uint_as_float(v[g][i]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool grow = top > m + lag || (m == -INFINITY && top > m);
                if (__any_sync(CAF, grow)) {
                    const float m_new = grow ? top : m, msc_new = grow ? top * sc : msc;
                    if (c > 0) {
                        const float f = grow ? (m == -INFINITY ? 0.0f : exp2_approx(msc - msc_new)) : 1.0f;
                        l *= f;
                        ok = wait.warp(&sh.o_done[t], (n_s - 1) & 1);   // the PV before has finished
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int g = 0; g < 4; g++) {
                            uint32_t x[32];
                            tmem_ld32(o_addr + 32 * g, x);
                            tmem_wait_ld(x);
#pragma unroll
                            for (int i = 0; i < 32; i++) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            tmem_st32(o_addr + 32 * g, x);
                        }
                    }
                    m = m_new;
                    msc = msc_new;
                }
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const float a = exp2_approx(fmaf(__uint_as_float(v[g][2 * i]), sc, -msc));
                        const float b = exp2_approx(fmaf(__uint_as_float(v[g][2 * i + 1]), sc, -msc));
                        sum[i & 3] += a + b;
                        h[i] = h2_as_u32(__floats2half2_rn(a, b));
                    }
                    tmem_st16(s_addr + 16 * g, h);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                if (bad) {
                    // a value that is not finite lies in the chunk and some rows do not see it: 0 times it would be
                    // NaN, so each row adds up what it sees by itself (rare, and slow)
                    if (c > 0) {
                        ok = wait.warp(&sh.o_done[t], (n_s - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    const uint8_t *vs = slots + ((2 * ci + 1) % NS) * CA_SLOT;
#pragma unroll 1
                    for (int g = 0; g < 4; g++) {
                        uint32_t x[32];
                        tmem_ld32(o_addr + 32 * g, x);
                        tmem_wait_ld(x);
                        if (c == 0)
#pragma unroll
                            for (int i = 0; i < 32; i++) x[i] = 0u;
#pragma unroll 1
                        for (int j = 0; j < CA_KEYS; j++) {
                            const float2 pp = __half22float2(u32_as_h2(tmem_ld1(s_addr + (j >> 1))));
                            const float pj = j & 1 ? pp.y : pp.x;
                            const bool mine = j >= lo2 && j < hi2;
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                x[i] = mine ? __float_as_uint(fmaf(pj, v_at(vs, j, 32 * g + i), __uint_as_float(x[i]))) : x[i];
                        }
                        tmem_st32(o_addr + 32 * g, x);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sh.p_ready[t]);
            }
            if (!ok) break;
            ok = wait.warp(&sh.o_done[t], (n_s - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const bool whole = s.begins && s.ends;
            float *part = part_row(p.ws, cta, s.begins ? 1 : 0, my);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (!whole && valid) *reinterpret_cast<float2 *>(part) = make_float2(m == -INFINITY ? m : msc, l);
#pragma unroll 1
            for (int g = 0; g < 4; g++) {
                __syncwarp();
                uint32_t x[32];
                tmem_ld32(o_addr + 32 * g, x);
                tmem_wait_ld(x);
                if (valid && whole) {
                    store_o32(out + 32 * g, reinterpret_cast<const float *>(x), inv, p.io_type);
                } else if (valid) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        *reinterpret_cast<uint4 *>(part + 4 + 32 * g + 4 * i) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
            }
            __syncwarp();
            tc_fence_before();
            if (s.begins && !s.ends && t == 0 && row == 0) {
                desc->t0 = s.t0;
                desc->h = s.h;
                desc->row0 = s.row0;
                desc->rows = s.rows;
                desc->last = s.last;
                desc->valid = 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the item that CTA blockIdx.x began and a later one
// ended, in key order: one warp per row, four dims per lane.
__global__ __launch_bounds__(256) void chunk_combine_kernel(const __grid_constant__ ChunkAttnParams p) {
    pdl_wait();
    const CaDesc *d = reinterpret_cast<const CaDesc *>(p.ws) + blockIdx.x;
    if (!d->valid) return;
    const int lane = threadIdx.x & 31, first = blockIdx.x, last = d->last, rows = d->rows;
    for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < rows; row += CA_COMBINE_Y * 8) {
        float m = -INFINITY;
        for (int c = first + lane; c <= last; c += 32) m = fmaxf(m, *part_row(p.ws, c, c == first ? 1 : 0, row));
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(CAF, m, o));
        float l = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int c = first; c <= last; c++) {
            const float *r = part_row(p.ws, c, c == first ? 1 : 0, row);
            const float2 ml = *reinterpret_cast<const float2 *>(r);
            const float4 x = *reinterpret_cast<const float4 *>(r + 4 + 4 * lane);
            const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - m);
            l += f * ml.y;
            y.x += f * x.x; y.y += f * x.y; y.z += f * x.z; y.w += f * x.w;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int flat = d->row0 + row, tok = flat / p.G, head = d->h * p.G + flat % p.G;
        uint16_t *out = p.o + (long long)(d->t0 + tok) * p.o_ld + (long long)head * HD + 4 * lane;
        uint2 o2;
        if (p.io_type == ZDEC_F16) {
            o2.x = h2_as_u32(__floats2half2_rn(y.x * inv, y.y * inv));
            o2.y = h2_as_u32(__floats2half2_rn(y.z * inv, y.w * inv));
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o2.x) : "f"(y.y * inv), "f"(y.x * inv));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o2.y) : "f"(y.w * inv), "f"(y.z * inv));
        }
        *reinterpret_cast<uint2 *>(out) = o2;
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

cudaError_t launch_chunk_attention(const ChunkAttnParams &p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(chunk_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CA_SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap map = {};
    if (p.kv.k_type == KV_T_F16 && (e = make_k_map(p, &map)) != cudaSuccess) return e;
    const int ctas = std::min(sms, CA_MAX_CTAS);
    e = launch_k(chunk_attention_kernel, dim3(ctas), dim3(CA_THREADS), CA_SMEM, false, 1, stream, p, map);
    if (e != cudaSuccess) return e;
    return launch_k(chunk_combine_kernel, dim3(ctas, CA_COMBINE_Y), dim3(256), 0, true, 1, stream, p);
}

}  // namespace zdec
