// paged.cuh -- attention over a paged key-value cache: the arguments, the split of a call's work over
// the grid, and the buffers through which parts of one row meet (GPU side only).
//
// Work.  A request j with n_j new tokens gives, for each kv head, G n_j rows (G = Hq / Hk query heads
// share a kv head; row r is token r / G, head r % G), cut into row tiles; each (request, kv head, row
// tile) is an item, and an item is a run of key tiles over the cache.  All items' key tiles, in order
// (request, kv head, row tile, key tile), form one list of units that is cut into equal contiguous
// ranges, one a block.  The lengths are on the device only, so every block adds them up itself (a
// block-wide prefix sum over the requests) and finds its own range; nothing is planned on the host
// and a call can be replayed from a graph with other lengths.  An item's beginning and end (its queries,
// the meeting of the warps, its rows written) cost about as much as a few key tiles, so each item
// counts `extra` units before its first tile; without them the block that met a run of one-tile items took
// a third longer than the others.
//
// Join.  A range may begin or end inside an item.  Such a segment's (maximum, sum, unnormalised output)
// goes to one of the block's two partial buffers -- kTail when the segment does not begin the item,
// kHead when it does but does not end it -- with a description of the item.  A second kernel joins the
// parts in a fixed order, so results do not depend on timing; the rows of an item are dealt out over
// as many of its blocks as it has parts.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {

struct AttnArgs {
    int T, B, Hq, Hk, G, D;
    uint32_t g_mul, g_shift;  // row / G = umulhi(2 row, g_mul) >> g_shift for rows below 2^31 (group_division)
    int page_shift, num_pages, max_blocks;
    int causal, window;
    float sum_scale;  // ProbScale's inverse, for lse
    int q_vec;        // rows of q start on 16-byte boundaries
    float scale, softcap;
    const unsigned char* q;
    long long q_token, q_head;  // strides, elements
    const unsigned char* k_pages;
    const unsigned char* v_pages;
    long long page, token, head;  // strides of the pools, bytes
    const int32_t* block_table;
    const int32_t* seq_len;
    const int32_t* offsets;  // or null: one token a request
    const float* k_scale;
    const float* v_scale;
    unsigned char* out;  // [T, Hq, D]
    float* lse;          // [T, Hq] or null
    // workspace
    int32_t* status;
    int32_t* error;  // the caller's word for the first error, or null
    struct PartItem* items;  // [parts]
    float2* part_ml;         // [2 parts][rows of a tile]: (maximum, log2 domain; sum)
    float* part_o;           // [2 parts][rows of a tile][D]
};

// An item spread over blocks, as each of them describes it (first < 0: none).
struct PartDesc {
    int first, last;  // blocks that begin and end it
    int row0, rows;   // first row of the tile within the request and kv head, its real rows
    int token0;       // row of q and out of the request's first token
    int head;         // kv head
    int pad[2];
};
struct PartItem {
    PartDesc d[2];    // of the block's kTail and kHead segment
    int err, pad[7];  // DSPARK_* recorded by the block
};

enum { kTail = 0, kHead = 1 };
constexpr int kMaxParts = 480;    // blocks of the largest grid with row tiles of 16 (three a multiprocessor)
constexpr int kMaxTcParts = 160;  // and of 128 (one)

// One request as the kernels see it: every number clamped to the buffers (bad: it was not).  Keys before lo,
// the first that any row sees, have no pages any more as far as a call is concerned.
struct AttnReq {
    int token0, n, seq, lo;
    bool bad;
};
__device__ __forceinline__ AttnReq attn_request(const AttnArgs& a, int j) {
    AttnReq r;
    int o0 = j, o1 = j + 1;
    if (a.offsets) {
        o0 = __ldg(a.offsets + j);
        o1 = __ldg(a.offsets + j + 1);
    }
    const int t0 = min(max(o0, 0), a.T), t1 = min(max(o1, t0), a.T);
    const int len = __ldg(a.seq_len + j);
    const long long cap = min((long long)a.max_blocks << a.page_shift, (long long)INT32_MAX - 4096);  // (tiles end past seq)
    r.token0 = t0;
    r.n = t1 - t0;
    r.seq = (int)min((long long)max(len, 0), cap);
    r.bad = t0 != o0 || t1 != o1 || len != r.seq;
    r.lo = a.window > 0 ? (int)max((long long)r.seq - r.n - a.window + 1, 0ll) : 0;
    return r;
}
// Row tiles and key tiles of a request's items (an item has at least one key tile, so that rows that
// see nothing are written too).
__device__ __forceinline__ int row_tiles(const AttnArgs& a, int n, int row_tile) {
    return (int)(((long long)n * a.G + row_tile - 1) / row_tile);
}
__device__ __forceinline__ int key_tiles(const AttnReq& r, int key_tile) {
    const int first = r.lo / key_tile;
    return max((r.seq + key_tile - 1) / key_tile - first, 1);
}

// Where a block's range begins: request, unit within the request.
struct AttnStart {
    long long begin, end, per, total;  // this block's units, units a block, all units
    int j;
    long long at;
};

struct AttnScratch {  // in shared memory, for attn_start
    long long warp_sum[16], at;
    int j;
};

// Adds up all requests' units and finds the range of block `part` of `parts`.  All threads of the block.
// min_units: a block takes no fewer (a short range would cost more to join than it saves).
template <int THREADS>
__device__ AttnStart attn_start(const AttnArgs& a, int row_tile, int key_tile, int extra, int parts, int part, int min_units,
                                AttnScratch* scratch, bool* bad) {
    static_assert(THREADS / 32 <= 16, "scratch");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m = (a.B + THREADS - 1) / THREADS;
    const int j0 = min(tid * m, a.B), j1 = min(j0 + m, a.B);
    long long u = 0;
    bool b = false;
    for (int j = j0; j < j1; ++j) {
        const AttnReq r = attn_request(a, j);
        b |= r.bad;
        u += (long long)row_tiles(a, r.n, row_tile) * a.Hk * (key_tiles(r, key_tile) + extra);
    }
    long long inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) scratch->warp_sum[warp] = inc;
    if (tid == 0) scratch->j = a.B;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w == warp) before = total;
        total += scratch->warp_sum[w];
    }
    AttnStart s;
    s.total = total;
    s.per = max((total + parts - 1) / parts, (long long)min_units);
    s.begin = min((long long)part * s.per, total);
    s.end = min(s.begin + s.per, total);
    long long at = before + inc - u;  // units before this thread's requests
    if (s.begin < s.end && at <= s.begin && s.begin < at + u) {
        int j = j0;
        for (; j < j1; ++j) {
            const AttnReq r = attn_request(a, j);
            const long long x = (long long)row_tiles(a, r.n, row_tile) * a.Hk * (key_tiles(r, key_tile) + extra);
            if (s.begin < at + x) break;
            at += x;
        }
        scratch->j = j;
        scratch->at = s.begin - at;
    }
    *bad = __syncthreads_or(b) != 0;
    s.j = scratch->j;
    s.at = scratch->at;
    return s;
}

// A walk over a block's range, one key tile at a time.
struct AttnWalk {
    AttnReq r;
    int j, item, items, kt, kts, rts, kt_first, extra;
    long long left;  // units left in the block's range, this tile's included
    __device__ __forceinline__ bool done() const { return left <= 0; }
};
__device__ __forceinline__ void walk_request(const AttnArgs& a, AttnWalk& w, int row_tile, int key_tile) {
    w.r = attn_request(a, w.j);
    w.rts = row_tiles(a, w.r.n, row_tile);
    w.items = w.rts * a.Hk;
    w.kts = key_tiles(w.r, key_tile);
    w.kt_first = w.r.lo / key_tile;
}
__device__ __forceinline__ AttnWalk walk_begin(const AttnArgs& a, const AttnStart& s, int row_tile, int key_tile, int extra) {
    AttnWalk w;
    w.left = s.end - s.begin;
    w.j = s.j;
    w.item = w.kt = 0;
    w.items = w.kts = w.rts = 1;
    w.kt_first = 0;
    w.extra = extra;
    w.r = AttnReq{0, 0, 0, 0, false};
    if (w.left > 0) {
        walk_request(a, w, row_tile, key_tile);
        w.item = (int)(s.at / (w.kts + extra));
        w.kt = (int)(s.at - (long long)w.item * (w.kts + extra)) - extra;
        if (w.kt < 0) {  // the range begins before the item's first tile
            w.left += w.kt;
            w.kt = 0;
        }
    }
    return w;
}
__device__ __forceinline__ void walk_next(const AttnArgs& a, AttnWalk& w, int row_tile, int key_tile) {
    --w.left;
    if (++w.kt < w.kts || w.left <= 0) return;
    w.kt = 0;
    w.left -= w.extra;
    if (++w.item < w.items || w.left <= 0) return;
    w.item = 0;
    do {  // requests without new tokens have no units
        ++w.j;
        walk_request(a, w, row_tile, key_tile);
    } while (w.items == 0 && w.j + 1 < a.B);
}

// The first key that a request's token sees, and the end of those it sees.
__device__ __forceinline__ int attn_see_lo(const AttnArgs& a, const AttnReq& r, int token) {
    return a.window > 0 ? (int)max((long long)r.seq - r.n + token - a.window + 1, 0ll) : 0;
}
__device__ __forceinline__ int attn_see_hi(const AttnArgs& a, const AttnReq& r, int token) {
    return a.causal ? min(r.seq - r.n + token + 1, r.seq) : r.seq;
}

// Rows of out (and lse) past the last request's tokens: no request owns them.  i0: this thread of n.
__device__ __forceinline__ void attn_tail_rows(const AttnArgs& a, size_t i0, size_t n) {
    const int end = a.offsets ? min(max(__ldg(a.offsets + a.B), 0), a.T) : a.B;
    const size_t row = (size_t)a.Hq * a.D * 2 / 16;  // 16-byte groups of a token
    for (size_t i = end * row + i0; i < a.T * row; i += n) reinterpret_cast<uint4*>(a.out)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
        for (size_t i = (size_t)end * a.Hq + i0; i < (size_t)a.T * a.Hq; i += n) a.lse[i] = -CUDART_INF_F;
}

// Token of a row of a request and kv head.
__device__ __forceinline__ int attn_token(const AttnArgs& a, int row) {
    return (int)(__umulhi(2u * (uint32_t)row, a.g_mul) >> a.g_shift);
}

// Row of [T Hq] of row `row` of a request and kv head.
__device__ __forceinline__ long long attn_out_row(const AttnArgs& a, int token0, int head, int row) {
    const int token = attn_token(a, row);
    return (long long)(token0 + token) * a.Hq + head * a.G + (row - token * a.G);
}

// 16 bytes, or 16 zero bytes where !real (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
    const int n = real ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// The description of a segment that is not a whole item.
__device__ __forceinline__ PartDesc part_desc(const AttnStart& s, const AttnWalk& w, int row0, int rows, int head) {
    const long long unit = s.end - w.left;
    PartDesc d;
    d.first = (int)((unit - w.kt) / s.per);
    d.last = (int)((unit + (w.kts - 1 - w.kt)) / s.per);
    d.row0 = row0;
    d.rows = rows;
    d.token0 = w.r.token0;
    d.head = head;
    d.pad[0] = d.pad[1] = 0;
    return d;
}

// c tanh(s / c) log2 e of two scores, in = 2 log2 e scale / c of the unscaled ones, out = c log2 e; without a branch.
// With y = 2 log2 e s / c: 1 - 2 / (1 + 2^y), whose error of some 3e-7 is 1.3e-6 of tanh where s / c is 1/4 and less
// above, and below that, where the difference would cancel, the odd Taylor series t - t^3/3 + 2 t^5/15 - 17 t^7/315 of
// t = y ln 2 / 2, whose next term is below 4e-7 of t there.  So a score is off by 2e-6 of itself, however large the cap.
// Two at a time by packed arithmetic: three requests of 200000 tokens, heads of 256, 129 us (143 one by one, 121 without
// the series; a branch around the far side for warps all below a quarter of the cap: 138).
__device__ __forceinline__ float2 softcap2(float x0, float x1, float in, float out) {
    constexpr float kT = 0.5f * kLn2, kT2 = kT * kT;
    constexpr float k3 = -1.f / 3.f * kT2, k5 = 2.f / 15.f * kT2 * kT2, k7 = -17.f / 315.f * kT2 * kT2 * kT2;
    const uint64_t y2 = mul2(pk2(x0, x1), pk2(in, in)), u = mul2(y2, y2);
    const float2 y = up2(y2);
    const float2 d = up2(add2(pk2(ex2(y.x), ex2(y.y)), pk2(1.f, 1.f)));
    float r0, r1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d.y));
    const float2 far = up2(fma2(pk2(r0, r1), pk2(-2.f * out, -2.f * out), pk2(out, out)));
    const uint64_t series = fma2(u, fma2(u, fma2(u, pk2(k7, k7), pk2(k5, k5)), pk2(k3, k3)), pk2(1.f, 1.f));
    const float2 near = up2(mul2(mul2(y2, pk2(out * kT, out * kT)), series));
    return make_float2(fabsf(y.x) < 0.25f / kT ? near.x : far.x, fabsf(y.y) < 0.25f / kT ? near.y : far.y);
}

// Whether one of a word's values is NaN or inf, gathered over words: note(w, acc), then found(acc).
template <bool F8, bool BF16>
__device__ __forceinline__ void odd_note(uint32_t w, uint32_t& acc) {
    if (F8)  // e4m3 has no inf: NaN is 0x7f but for the sign
        acc |= (w & 0x7f7f7f7fu) + 0x01010101u;
    else  // the largest magnitude of either half
        acc = __vmaxu2(acc, w & 0x7fff7fffu);
}
template <bool F8, bool BF16>
__device__ __forceinline__ bool odd_found(uint32_t acc) {
    if (F8) return (acc & 0x80808080u) != 0;
    constexpr uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
    return (acc & 0xffffu) >= inf || (acc >> 16) >= inf;
}

// Probabilities as halves are taken against a reference 2^7 below the running maximum's (which follows within 2^8, so
// they stay below 2^15): halves lose bits below 2^-14, which is then 2^-21 of the largest.  bf16 has fp32's exponents.
// Sums carry the same factor; it cancels in the output and is taken out of lse.
template <bool BF16>
struct ProbScale {
    static constexpr float kBits = BF16 ? 0.f : 7.f;
    static constexpr float kInverse = BF16 ? 1.f : 0x1p-7f;
};

// Two floats rounded to the 16-bit type, first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}


// Row tiles of 128 on the fifth-generation tensor cores (paged_attn_tc.cu); needs 16-byte
// aligned query rows.
dspark_status launch_attn_tc(const AttnArgs& a, bool bf16, bool e4m3, int sms, cudaStream_t s, int* parts);

}  // namespace dspark
