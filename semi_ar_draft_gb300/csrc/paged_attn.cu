// paged_attn.cu -- dspark_paged_attention: attention of each request's new tokens over its paged
// key-value cache (paged.cuh has the split of the work and the join).
//
//   s_l = scale q . k_l,  capped c tanh(s_l / c);  m, sum: running maximum and sum of 2^(s_l log2 e);
//   o = sum_l 2^(s_l log2 e - m) v_l / sum
//
// attn_rows16_kernel: row tiles of 16 (one token of up to 16 query heads a kv head, or a few tokens of
// fewer; up to some 48 rows of an 8-bit cache: wide_rows).  A cache row of D 16-bit values is used for 4 D
// operations a row, so at 16 rows the kernel is bound by the cache's bytes: 16 operations a byte against the
// card's several hundred.  What it needs is loads in flight, so each warp streams key slices of its own (16
// keys, or 32 of an 8-bit cache) through a ring of its own in shared memory, 16 bytes a copy, with no barrier
// between warps; the page numbers of a slice are fetched a step before its copies are issued.  The warps'
// statistics and outputs meet once per segment, in the stages just consumed (a stage is as large as a warp's
// output: 64 D bytes).  Two blocks a multiprocessor or more, so that one streams while another joins.
// Measured: 32 requests of up to 8192 tokens, 8 kv heads of 128, bf16: 95 us = 5.9 TB/s (0.87 of the measured copy
// rate), of which 5 us are the join; 128 requests over an e4m3 cache 209 us = 5.4 TB/s (0.79), where the
// conversions keep the issue slots busy; one request of 1024 tokens 12 us, latency.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "host_util.h"
#include "paged.cuh"
#include "pdl.cuh"
#include "tc05.cuh"

namespace dspark {
namespace {

constexpr int kRows = 16;
constexpr int kTcRows = 128;  // rows of a tile of launch_attn_tc

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 values (low 16 bits) as two halves.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w) {
    uint32_t r;
    asm("{ .reg .b16 x; cvt.u16.u32 x, %1; cvt.rn.f16x2.e4m3x2 %0, x; }" : "=r"(r) : "r"(w));
    return r;
}

// The half in the low 16 bits.
__device__ __forceinline__ float half_bits_to_f32(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)w));
}

template <bool F8, int DP>
struct Rows16 {
    static constexpr int kEsz = F8 ? 1 : 2;
    static constexpr int kKeys = F8 ? 32 : 16;           // keys of a warp's slice
    // (heads of 256, one block a multiprocessor: six warps of two stages, 204 us for 16 kv heads of 192 over 32
    // requests of up to 5625 tokens, against 244 us with four of three)
    static constexpr int kWarps = DP == 256 ? 6 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kKeyTile = kWarps * kKeys;      // keys of a unit
    static constexpr int kRowBytes = DP * kEsz;
    static constexpr int kChunks = kRowBytes / 16;       // 16-byte groups of a row
    static constexpr int kHalf = kKeys * kRowBytes;      // K (or V) of a slice
    static constexpr int kStage = 2 * kHalf;             // = 64 DP: also a warp's output in fp32
    // Blocks a multiprocessor and stages a warp, measured: 16-bit heads of 128 want two blocks of three (95
    // us for 32 requests up to 8192 tokens, 97 us with three of two); heads of 64 three of four (60 us for the same
    // requests, 66 with two of four); 8-bit heads of 128, bound by their conversions, three of two (208 us for 128
    // requests up to 8000 tokens, 210 with two of three).
    static constexpr bool kThree = DP == 64 || (F8 && DP == 128);
    static constexpr int kStages = DP == 64 ? 4 : (kThree || DP == 256 ? 2 : 3);
    static constexpr int kExtra = DP == 64 ? 4 : 2;      // what an item costs beside its key tiles
    static constexpr int kBlocksPerSm = DP == 256 ? 1 : (kThree ? 3 : 2);
    // Registers: 64 of q beside 128 of output do not fit a thread, nor 32 beside 64 three blocks; the MMAs
    // then take q from shared memory every time.
    static constexpr bool kQInSmem = DP == 256 || (kThree && DP == 128);
    static constexpr int kQBytes = kRows * DP * 2;
    static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage + kQBytes;
    static_assert(kStage == kRows * DP * 4, "a stage holds a warp's output");
    // Rows are a multiple of 128 bytes apart (or 64): the swizzle spreads eight rows' same 16-byte group
    // over all banks.
    static __device__ __forceinline__ uint32_t at(int row, int chunk) {
        const int x = kChunks >= 8 ? (row & 7) : ((row >> 1) & 3);
        return (uint32_t)(row * kRowBytes + ((chunk ^ x) << 4));
    }
    static __device__ __forceinline__ uint32_t q_at(int row, int chunk) {  // 16-bit rows of q
        return (uint32_t)(row * (DP * 2) + ((chunk ^ (row & 7)) << 4));
    }
};

template <bool BF16>
__device__ __forceinline__ void store_out4(const AttnArgs& a, long long row, int col, float4 v) {
    uint2 w = make_uint2(pack16<BF16>(v.x, v.y), pack16<BF16>(v.z, v.w));
    *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.D + col) * 2) = w;
}

template <bool BF16, bool F8, int DP>
__global__ void __launch_bounds__(Rows16<F8, DP>::kThreads, Rows16<F8, DP>::kBlocksPerSm) attn_rows16_kernel(AttnArgs a) {
    using C = Rows16<F8, DP>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps;
    constexpr bool MB = BF16 && !F8;  // an 8-bit cache is multiplied as halves, which hold e4m3 exactly
    constexpr int KT = C::kKeys / 8;  // key n-tiles of a slice
    constexpr int DT = DP / 8;        // output n-tiles
    constexpr int KS = DP / 16;       // k-steps over the head dimension
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 s_ml[kWarps][kRows];
    __shared__ int s_err;
    __shared__ AttnScratch s_start;
    __shared__ uint32_t s_qmax[kRows];  // largest |q| of each row (its bits)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int part = blockIdx.x, parts = gridDim.x;
    wait_primary();
    launch_dependents();
    if (tid == 0) s_err = 0;
    bool bad;
    const AttnStart start = attn_start<kThreads>(a, kRows, C::kKeyTile, C::kExtra, parts, part, 2 + C::kExtra, &s_start, &bad);

    attn_tail_rows(a, (size_t)part * kThreads + tid, (size_t)parts * kThreads);
    unsigned char* ring = smem + (size_t)warp * C::kStages * C::kStage;
    const uint32_t ring_addr = smem_addr(ring);
    unsigned char* qs = smem + (size_t)kWarps * C::kStages * C::kStage;
    const uint32_t qs_addr = smem_addr(qs);
    int err = bad ? DSPARK_ERR_CACHE : 0;

    // ---- loads: `ld` walks ahead of the arithmetic; `pid` is the page of this lane's key of its slice
    AttnWalk ld = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    auto slice_key = [&](const AttnWalk& w) { return (w.kt_first + w.kt) * C::kKeyTile + warp * C::kKeys; };
    auto fetch_page = [&]() -> int {
        const int key = slice_key(ld) + lane;
        if (ld.done() || lane >= C::kKeys || key >= ld.r.seq) return -1;
        return __ldg(a.block_table + (size_t)ld.j * a.max_blocks + (key >> a.page_shift));
    };
    int pid = fetch_page();
    int ld_stage = 0;
    // An item's queries, asked for (into L1) when its first keys are: 16 rows of up to four 128-byte lines.
    auto touch_queries = [&]() {
        const int head = ld.item / ld.rts, first = (ld.item - head * ld.rts) * kRows;
        const int last = min(ld.r.n * a.G, first + kRows);
        for (int i = lane; i < kRows * (DP / 64); i += 32) {
            const int row = first + i / (DP / 64), token = attn_token(a, row), d = 64 * (i % (DP / 64));
            if (row < last && d < a.D)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + 2 * ((ld.r.token0 + token) * a.q_token +
                                                                        (head * a.G + row - token * a.G) * a.q_head + d)));
        }
    };
    if (warp == 0 && !ld.done()) touch_queries();
    auto load_step = [&]() {
        if (!ld.done() && slice_key(ld) < ld.r.seq) {
            const int key = slice_key(ld) + lane;
            const bool live = lane < C::kKeys && key < ld.r.seq && key >= ld.r.lo;
            const bool found = live && pid >= 0 && pid < a.num_pages;
            if (live && !found) err = DSPARK_ERR_CACHE;
            const long long off = found ? pid * a.page + (key & ((1 << a.page_shift) - 1)) * a.token +
                                              (ld.item / ld.rts) * a.head
                                        : -1;
            const uint32_t dst = ring_addr + ld_stage * C::kStage;
            constexpr int kPer = 32 / C::kChunks;  // rows a warp copies at a time
            const int chunk = lane % C::kChunks;
            const bool inside = chunk * 16 < a.D * C::kEsz;
#pragma unroll
            for (int i = 0; i < C::kKeys / kPer; ++i) {
                const int row = i * kPer + lane / C::kChunks;
                const long long o = __shfl_sync(0xffffffffu, off, row);
                const bool real = inside && o >= 0;
                const long long src = real ? o + chunk * 16 : 0;
                copy16(dst + C::at(row, chunk), a.k_pages + src, real);
                copy16(dst + C::kHalf + C::at(row, chunk), a.v_pages + src, real);
            }
        }
        cp_async_commit();
        if (++ld_stage == C::kStages) ld_stage = 0;
        if (!ld.done()) {
            walk_next(a, ld, kRows, C::kKeyTile);
            pid = fetch_page();
            if (warp == 0 && ld.kt == 0 && !ld.done()) touch_queries();
        }
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load_step();

    // ---- arithmetic
    AttnWalk w = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    PartItem* mine = a.items + part;  // written by thread 0
    if (tid == 0) mine->d[kTail].first = mine->d[kHead].first = -1;
    float o[DT][4];
    uint32_t qf[C::kQInSmem ? 1 : KS][4];
    const float cap_out = a.softcap * kLog2e;
    float m[2], l[2], row_scale[2];
    int see_lo[2], see_hi[2], all_lo = 0, all_hi = 0, rows = 0, head = 0, row0 = 0, seg_first = 0;
    bool fresh = true;
    int st = 0;
    while (!w.done()) {
        if (fresh) {  // a new segment: its rows, their queries and what each may see
            fresh = false;
            seg_first = w.kt;
            head = w.item / w.rts;
            row0 = (w.item % w.rts) * kRows;
            rows = min(w.r.n * a.G - row0, kRows);
            all_lo = attn_see_lo(a, w.r, attn_token(a, row0 + rows - 1));
            all_hi = attn_see_hi(a, w.r, attn_token(a, row0));
            // The queries, through shared memory: 16 bytes a thread, then the MMA's fragments by ldmatrix.  (The
            // previous segment's readers are past its last barrier.)
            constexpr int kQc = DP / 8;
            constexpr int kQSteps = (kRows * kQc + kThreads - 1) / kThreads;
            uint4 qv[kQSteps];
            constexpr bool kRescale = F8 && BF16;
            if (kRescale) {
                if (tid < kRows) s_qmax[tid] = 0;
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < kQSteps; ++u) {
                const int row = (tid + u * kThreads) / kQc, c = (tid + u * kThreads) % kQc, token = attn_token(a, row0 + row);
                qv[u] = make_uint4(0, 0, 0, 0);
                if (kRows * kQc % kThreads && row >= kRows) continue;
                if (row < rows && 8 * c < a.D) {
                    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (w.r.token0 + token) * a.q_token +
                                          (head * a.G + row0 + row - token * a.G) * a.q_head + 8 * c;
                    if (a.q_vec) {
                        qv[u] = __ldg(reinterpret_cast<const uint4*>(src));
                    } else {  // rows may start at any element
                        uint32_t* y = reinterpret_cast<uint32_t*>(&qv[u]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = (uint32_t)__ldg(src + 2 * e) | ((uint32_t)__ldg(src + 2 * e + 1) << 16);
                    }
                }
                if (kRescale) {
                    float big = 0.f;
                    const uint32_t* y = reinterpret_cast<const uint32_t*>(&qv[u]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) big = fmaxf(big, fmaxf(fabsf(bf16_lo(y[e])), fabsf(bf16_hi(y[e]))));
                    atomicMax(&s_qmax[row], __float_as_uint(big));
                }
            }
            // bf16 queries as halves (an 8-bit cache): each row times the power of two that brings its largest
            // value to 2^14, taken back in the scores' scale; what a half then cannot hold is below 2^-38 of the
            // row's largest, less than fp32 keeps of the sum.
            auto raise = [&](int row) {
                const int e = (int)(s_qmax[row] >> 23) - 127;  // floor(log2) of a normal number
                return e > -127 && e < 128 ? min(max(14 - e, -120), 120) : 0;
            };
            if (kRescale) __syncthreads();
#pragma unroll
            for (int u = 0; u < kQSteps; ++u) {
                const int row = (tid + u * kThreads) / kQc, c = (tid + u * kThreads) % kQc;
                if (kRows * kQc % kThreads && row >= kRows) continue;
                if (!F8) {
                    *reinterpret_cast<uint4*>(qs + C::q_at(row, c)) = qv[u];
                } else {
                    // 8-bit keys arrive four k a lane: the MMA's k slots (2t, 2t + 1 | 2t + 8, 2t + 9) hold k = 4t .. 4t + 3,
                    // so pair p of 16 values goes to pair p / 2 + 4 (p % 2)
                    const uint32_t* y = reinterpret_cast<const uint32_t*>(&qv[u]);
                    const float up = kRescale ? __uint_as_float((uint32_t)(127 + raise(row)) << 23) : 1.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int p = 4 * (c & 1) + e, to = (p >> 1) + 4 * (p & 1);
                        const uint32_t x = kRescale ? pack16<false>(bf16_lo(y[e]) * up, bf16_hi(y[e]) * up) : y[e];
                        *reinterpret_cast<uint32_t*>(qs + C::q_at(row, (c & ~1) + (to >> 2)) + 4 * (to & 3)) = x;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r, token = attn_token(a, row0 + row);
                const bool real = row < rows;
                see_lo[r] = real ? attn_see_lo(a, w.r, token) : 0;
                see_hi[r] = real ? attn_see_hi(a, w.r, token) : 0;
                m[r] = -CUDART_INF_F;
                l[r] = 0.f;
                // to the log2 domain, or to the cap's exponent
                row_scale[r] = (a.softcap > 0.f ? 2.f * kLog2e / a.softcap : kLog2e) * a.scale *
                               (F8 && a.k_scale ? __ldg(a.k_scale + head) : 1.f);
                if (kRescale) row_scale[r] *= __uint_as_float((uint32_t)(127 - raise(row)) << 23);
            }
            if (!C::kQInSmem) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    ldsm4(qf[C::kQInSmem ? 0 : ks], qs_addr + C::q_at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * ks + (lane >> 4)));
            }
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
        }
        load_step();
        cp_async_wait_group<C::kStages - 1>();
        __syncwarp();
        const int key0 = slice_key(w);
        if (key0 < w.r.seq) {
            const uint32_t kb = ring_addr + st * C::kStage, vb = kb + C::kHalf;
            float s[KT][4];
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t q4[4];
                if (C::kQInSmem) {
                    ldsm4(q4, qs_addr + C::q_at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * ks + (lane >> 4)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) q4[i] = qf[C::kQInSmem ? 0 : ks][i];
                }
                uint32_t b[4];
                if (F8) {
                    ldsm4(b, kb + C::at(lane, ks));  // matrix i: keys 8 i .. 8 i + 7, k = 16 ks .. + 15
#pragma unroll
                    for (int i = 0; i < KT; ++i)
                        mma16<MB>(s[i], q4, e4m3x2_to_half2(b[i]), e4m3x2_to_half2(b[i] >> 16));
                } else {
                    const int row = (lane & 7) + ((lane >> 4) << 3);
                    ldsm4(b, kb + C::at(row, 2 * ks + ((lane >> 3) & 1)));
                    mma16<MB>(s[0], q4, b[0], b[1]);
                    mma16<MB>(s[1], q4, b[2], b[3]);
                }
            }
            // scores in the log2 domain, hidden ones -inf
            const bool edge = key0 < all_lo || key0 + C::kKeys > all_hi;
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2 x = make_float2(s[i][2 * r] * row_scale[r], s[i][2 * r + 1] * row_scale[r]);
                    if (a.softcap > 0.f) x = softcap2(s[i][2 * r], s[i][2 * r + 1], row_scale[r], cap_out);
                    if (edge) {
                        const int key = key0 + 8 * i + 2 * t;
                        if (key < see_lo[r] || key >= see_hi[r]) x.x = -CUDART_INF_F;
                        if (key + 1 < see_lo[r] || key + 1 >= see_hi[r]) x.y = -CUDART_INF_F;
                    }
                    s[i][2 * r] = x.x;
                    s[i][2 * r + 1] = x.y;
                    mx[r] = fmaxf(mx[r], fmaxf(x.x, x.y));
                }
            bool grow = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                grow |= mx[r] > m[r] + 8.f;
            }
            // The reference of the exponents follows the maximum only when it is 2^8 behind (values up
            // to 2^8 lose nothing), so most slices do not touch the output.
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float mn = fmaxf(m[r], mx[r]);
                    const float f = mn == m[r] ? 1.f : ex2(m[r] - mn);  // m = -inf: 0
                    m[r] = mn;
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < DT; ++i) {
                        o[i][2 * r] *= f;
                        o[i][2 * r + 1] *= f;
                    }
                }
            }
            constexpr float kUp = ProbScale<MB>::kBits;
            const float ref[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0] - kUp, m[1] == -CUDART_INF_F ? 0.f : m[1] - kUp};
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[i][c] = ex2(s[i][c] - ref[c >> 1]);
                    l[c >> 1] += s[i][c];
                }
            // A hidden key's value must not reach a row that does not see it, even as 0 x inf.  Values of
            // an edge slice that are not finite (never, in a healthy cache) take the long way: products key by
            // key, over the rows that see it.
            bool odd = false;
            if (edge) {
                uint32_t acc = 0;
                const uint4* vs = reinterpret_cast<const uint4*>(ring + st * C::kStage + C::kHalf);
                for (int i = lane; i < C::kHalf / 16; i += 32) {
                    const uint4 y = vs[i];
                    odd_note<F8, BF16>(y.x, acc);
                    odd_note<F8, BF16>(y.y, acc);
                    odd_note<F8, BF16>(y.z, acc);
                    odd_note<F8, BF16>(y.w, acc);
                }
                odd = __any_sync(0xffffffffu, odd_found<F8, BF16>(acc));
            }
            if (!odd) {
                // Probabilities are rounded to the cache's 16-bit type (halves for an 8-bit cache) for
                // the second product; their sum is kept unrounded in fp32.
#pragma unroll
                for (int h = 0; h < KT / 2; ++h) {
                    const uint32_t p[4] = {pack16<MB>(s[2 * h][0], s[2 * h][1]), pack16<MB>(s[2 * h][2], s[2 * h][3]),
                                           pack16<MB>(s[2 * h + 1][0], s[2 * h + 1][1]),
                                           pack16<MB>(s[2 * h + 1][2], s[2 * h + 1][3])};
                    if (F8) {
#pragma unroll
                        for (int c = 0; c < DP / 16; c += 2) {  // two 16-value groups, keys 16 h .. 16 h + 15
                            uint32_t b[4];
                            const int row = 16 * h + (lane & 7) + ((lane >> 3) & 1) * 8;
                            ldsm4_trans(b, vb + C::at(row, c + (lane >> 4)));
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                // bytes (k0 d0, k0 d1, k1 d0, k1 d1) -> (k0 d0, k1 d0 | k0 d1, k1 d1)
                                const uint32_t x = __byte_perm(b[2 * u], 0, 0x3120);
                                const uint32_t y = __byte_perm(b[2 * u + 1], 0, 0x3120);
                                mma16<MB>(o[2 * (c + u)], p, e4m3x2_to_half2(x), e4m3x2_to_half2(y));
                                mma16<MB>(o[2 * (c + u) + 1], p, e4m3x2_to_half2(x >> 16), e4m3x2_to_half2(y >> 16));
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < DP / 16; ++c) {
                            uint32_t b[4];
                            const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
                            ldsm4_trans(b, vb + C::at(row, 2 * c + (lane >> 4)));
                            mma16<MB>(o[2 * c], p, b[0], b[1]);
                            mma16<MB>(o[2 * c + 1], p, b[2], b[3]);
                        }
                    }
                }
            } else {
                const unsigned char* vs = ring + st * C::kStage + C::kHalf;
#pragma unroll
                for (int i = 0; i < KT; ++i)
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        const int key = key0 + 8 * i + k, from = (lane & ~3) | (k >> 1);
                        float p[2];
                        p[0] = __shfl_sync(0xffffffffu, (k & 1) ? s[i][1] : s[i][0], from);
                        p[1] = __shfl_sync(0xffffffffu, (k & 1) ? s[i][3] : s[i][2], from);
                        const bool in0 = key >= see_lo[0] && key < see_hi[0], in1 = key >= see_lo[1] && key < see_hi[1];
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int col = F8 ? 16 * (d >> 1) + 4 * t + 2 * c + (d & 1) : 8 * d + 2 * t + c;
                                const uint32_t at = C::at(8 * i + k, col * C::kEsz / 16) + (col * C::kEsz) % 16;
                                float v;
                                if (F8)
                                    v = half_bits_to_f32(e4m3x2_to_half2(vs[at]));
                                else if (BF16)
                                    v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(vs + at));
                                else
                                    v = half_bits_to_f32(*reinterpret_cast<const uint16_t*>(vs + at));
                                if (in0) o[d][c] = fmaf(p[0], v, o[d][c]);
                                if (in1) o[d][2 + c] = fmaf(p[1], v, o[d][2 + c]);
                            }
                    }
            }
        }
        __syncwarp();  // the slice has been read by every lane

        const bool last_of_item = w.kt + 1 == w.kts;
        if (last_of_item || w.left == 1) {
            // ---- the four warps' parts of the segment meet
            float* mine_o = reinterpret_cast<float*>(ring + st * C::kStage);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                const int row = g + 8 * r, x = (row & 3) << 3;
                if (t == 0) s_ml[warp][row] = make_float2(m[r], l[r]);
                if (F8) {
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c)
                        *reinterpret_cast<float4*>(mine_o + row * DP + ((16 * c + 4 * t) ^ x)) =
                            make_float4(o[2 * c][2 * r], o[2 * c + 1][2 * r], o[2 * c][2 * r + 1], o[2 * c + 1][2 * r + 1]);
                } else {
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        *reinterpret_cast<float2*>(mine_o + row * DP + ((8 * d + 2 * t) ^ x)) =
                            make_float2(o[d][2 * r], o[d][2 * r + 1]);
                }
            }
            __syncthreads();
            const bool whole = last_of_item && seg_first == 0;
            const int slot = 2 * part + (seg_first == 0 ? kHead : kTail);
            const float vscale = F8 && a.v_scale ? __ldg(a.v_scale + head) : 1.f;
            for (int i = tid; i < rows * (DP / 4); i += kThreads) {
                const int row = i / (DP / 4), col = 4 * (i % (DP / 4));
                float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, s_ml[x][row].x);
                const float ref = mm == -CUDART_INF_F ? 0.f : mm;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float2 ml = s_ml[x][row];
                    const float f = ex2(ml.x - ref);
                    if (ml.y == 0.f) continue;  // saw nothing
                    ll = fmaf(ml.y, f, ll);
                    const float4 y = *reinterpret_cast<const float4*>(
                        smem + (size_t)(x * C::kStages + st) * C::kStage + 4 * (row * DP + (col ^ ((row & 3) << 3))));
                    v.x = fmaf(y.x, f, v.x);
                    v.y = fmaf(y.y, f, v.y);
                    v.z = fmaf(y.z, f, v.z);
                    v.w = fmaf(y.w, f, v.w);
                }
                if (whole) {
                    const long long at = attn_out_row(a, w.r.token0, head, row0 + row);
                    if (col < a.D) {
                        const float inv = ll == 0.f ? 0.f : vscale / ll;
                        store_out4<BF16>(a, at, col, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                    }
                    if (a.lse && col == 0)
                        a.lse[at] = ll == 0.f ? -CUDART_INF_F : (mm + lg2(ll * ProbScale<MB>::kInverse)) * kLn2;
                } else {
                    if (col < a.D)
                        *reinterpret_cast<float4*>(a.part_o + ((size_t)slot * kRows + row) * a.D + col) = v;
                    if (col == 0) a.part_ml[(size_t)slot * kRows + row] = make_float2(mm, ll);
                }
            }
            if (!whole && tid == 0) mine->d[seg_first == 0 ? kHead : kTail] = part_desc(start, w, row0, rows, head);
            __syncthreads();
            fresh = true;
        }
        if (++st == C::kStages) st = 0;
        walk_next(a, w, kRows, C::kKeyTile);
    }
    cp_async_wait_group<0>();
    if (err) s_err = err;  // any of the block's errors: all are the same code
    __syncthreads();
    if (tid == 0) mine->err = s_err;
}

// Joins the parts of the items that are spread over blocks.  Block (p, y) takes rows of the items that
// part p belongs to: of an item of n parts, rows k, k + n Y, ... with k = Y (p - first) + y, so that few
// items of many parts keep as many blocks busy as many items of few.  The four warps share a row's parts,
// or, where the parts are few, take rows of their own; either way the first parts are asked for before the
// weights are known.
constexpr int kJoinWarps = 4;
constexpr int kJoinAhead = 4;
constexpr int kJoinFew = 8;  // up to so many parts, a warp joins a row by itself (20 -> 8 us for 64 rows of 2 parts)
template <bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(AttnArgs a, int row_tile, int parts) {
    __shared__ float s_f[kMaxParts];
    __shared__ float4 s_acc[kJoinWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_primary();
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
        int err = 0;
        for (int p = lane; p < parts; p += 32) err = max(err, a.items[p].err);
        err = __reduce_max_sync(0xffffffffu, err);
        if (lane == 0) {
            *a.status = err;
            if (err && a.error) record_status(a.error, err);
        }
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const PartDesc it = a.items[blockIdx.x].d[side];
        if (it.first < 0) continue;
        const int n = it.last - it.first + 1;  // parts: the first block's head, then tails
        auto slot_of = [&](int i) { return (size_t)(2 * (it.first + i) + (i == 0 ? kHead : kTail)); };
        if (n <= kJoinFew) {
            const int worker = (((int)blockIdx.x - it.first) * gridDim.y + blockIdx.y) * kJoinWarps + warp;
#pragma unroll 1
            for (int row = worker; row < it.rows; row += n * gridDim.y * kJoinWarps) {
                const float2 ml = lane < n ? a.part_ml[slot_of(lane) * row_tile + row] : make_float2(-CUDART_INF_F, 0.f);
                const float vscale = a.v_scale ? __ldg(a.v_scale + it.head) : 1.f;
                const long long at = attn_out_row(a, it.token0, it.head, it.row0 + row);
#pragma unroll 1
                for (int col = 4 * lane; col - 4 * lane < a.D; col += 128) {
                    const bool in = col < a.D;
                    float4 y[kJoinFew];
#pragma unroll
                    for (int i = 0; i < kJoinFew; ++i)
                        if (i < n && in)
                            y[i] = *reinterpret_cast<const float4*>(a.part_o + (slot_of(i) * row_tile + row) * a.D + col);
                    const float mm = warp_max(ml.x);
                    const float f = ml.y == 0.f ? 0.f : ex2(ml.x - (mm == -CUDART_INF_F ? 0.f : mm));
                    const float ll = warp_sum(ml.y * f);
                    const float inv = ll == 0.f ? 0.f : vscale / ll;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < kJoinFew; ++i) {
                        const float fi = __shfl_sync(0xffffffffu, f, i);
                        if (i < n && in) {
                            v.x = fmaf(y[i].x, fi, v.x);
                            v.y = fmaf(y[i].y, fi, v.y);
                            v.z = fmaf(y[i].z, fi, v.z);
                            v.w = fmaf(y[i].w, fi, v.w);
                        }
                    }
                    if (in) store_out4<BF16>(a, at, col, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                    if (a.lse && col == 0) a.lse[at] = ll == 0.f ? -CUDART_INF_F : (mm + lg2(ll * a.sum_scale)) * kLn2;
                }
            }
            continue;
        }
#pragma unroll 1
        for (int row = ((int)blockIdx.x - it.first) * gridDim.y + blockIdx.y; row < it.rows; row += n * gridDim.y) {
            const float vscale = a.v_scale ? __ldg(a.v_scale + it.head) : 1.f;
            float ll = 0.f, mm = -CUDART_INF_F;
#pragma unroll 1
            for (int col = 4 * lane; col - 4 * lane < a.D; col += 128) {
                const bool in = col < a.D;
                auto part = [&](int i) {
                    return *reinterpret_cast<const float4*>(a.part_o + (slot_of(i) * row_tile + row) * a.D + col);
                };
                float4 y[kJoinAhead];
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u) {
                    const int i = warp + u * kJoinWarps;
                    y[u] = in && i < n ? part(i) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (col < 128) {  // the parts' weights, once a row
                    for (int i = tid; i < n; i += 32 * kJoinWarps) s_f[i] = a.part_ml[slot_of(i) * row_tile + row].x;
                    __syncthreads();
                    for (int i = lane; i < n; i += 32) mm = fmaxf(mm, s_f[i]);
                    mm = warp_max(mm);
                    const float ref = mm == -CUDART_INF_F ? 0.f : mm;
                    __syncthreads();
                    for (int i = lane; i < n; i += 32) {  // (every warp: the same sum in the same order)
                        const float2 ml = a.part_ml[slot_of(i) * row_tile + row];
                        const float f = ml.y == 0.f ? 0.f : ex2(ml.x - ref);
                        ll = fmaf(ml.y, f, ll);
                        if (warp == 0) s_f[i] = f;
                    }
                    ll = warp_sum(ll);
                    __syncthreads();
                }
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                auto add = [&](float f, const float4& x) {
                    v.x = fmaf(x.x, f, v.x);
                    v.y = fmaf(x.y, f, v.y);
                    v.z = fmaf(x.z, f, v.z);
                    v.w = fmaf(x.w, f, v.w);
                };
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u) {
                    const int i = warp + u * kJoinWarps;
                    if (i < n) add(s_f[i], y[u]);
                }
                if (in)
#pragma unroll 4
                    for (int i = warp + kJoinAhead * kJoinWarps; i < n; i += kJoinWarps) add(s_f[i], part(i));
                s_acc[warp][lane] = v;
                __syncthreads();
                if (warp == 0 && in) {
                    const float inv = ll == 0.f ? 0.f : vscale / ll;
                    float4 t = s_acc[0][lane];
#pragma unroll
                    for (int x = 1; x < kJoinWarps; ++x) {
                        const float4 z = s_acc[x][lane];
                        t.x += z.x;
                        t.y += z.y;
                        t.z += z.z;
                        t.w += z.w;
                    }
                    const long long at = attn_out_row(a, it.token0, it.head, it.row0 + row);
                    store_out4<BF16>(a, at, col, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
                    if (a.lse && col == 0) a.lse[at] = ll == 0.f ? -CUDART_INF_F : (mm + lg2(ll * a.sum_scale)) * kLn2;
                }
                __syncthreads();
            }
        }
    }
}

template <bool BF16, bool F8, int DP>
dspark_status launch_rows16(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    using C = Rows16<F8, DP>;
    int per_sm = 0;
    auto fn = attn_rows16_kernel<BF16, F8, DP>;
    if (prepare_kernel((const void*)fn, C::kSmem, C::kThreads, &per_sm) != cudaSuccess || per_sm < 1)
        return DSPARK_ERR_CUDA;
    int n = sms * (per_sm < C::kBlocksPerSm ? per_sm : C::kBlocksPerSm);
    if (n > kMaxParts) n = kMaxParts;
    *parts = n;
    return launch_overlapped(fn, n, C::kThreads, C::kSmem, s, a) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

template <bool BF16, bool F8>
dspark_status launch_rows16_d(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    if (a.D <= 64) return launch_rows16<BF16, F8, 64>(a, sms, s, parts);
    if (a.D <= 128) return launch_rows16<BF16, F8, 128>(a, sms, s, parts);
    return launch_rows16<BF16, F8, 256>(a, sms, s, parts);
}

struct AttnWs {
    size_t items, ml, o, bytes;
};
// Whether a call takes row tiles of 128: when a request has more rows a kv head than the limit, on average
// (T / B tokens) and at most (max_new, if given).  Measured, tiles of 16 against tiles of 128, us:
//   16-bit   mean 11 rows 117 / 115 (long contexts) and 63 / 84 (short); mean 14: 130 / 109 and 71 / 83;
//            mean 24: 88 / 67; heads of 256, mean 11: 214 / 255, mean 24: 159 / 139
//   e4m3     mean 35 rows 69 / 85 and 36 / 42; 68 rows: 80 / 58; mean 70: 159 / 101; 119 rows: 254 / 92
// (an 8-bit tile has to be widened for the wide kernel, so it needs more rows to pay).
bool wide_rows(const dspark_attention_params* p) {
    const long long G = p->Hq / p->Hk, limit = p->kv_dtype == p->dtype ? kRows : 48;
    return G * p->T > limit * p->B && (p->max_new <= 0 || G * p->max_new > limit);
}
AttnWs attn_ws(const dspark_attention_params* p) {
    const size_t rows = wide_rows(p) ? (size_t)2 * kMaxTcParts * kTcRows : (size_t)2 * kMaxParts * kRows;
    AttnWs w;
    w.items = kHeaderBytes;
    w.ml = align_up(w.items + sizeof(PartItem) * kMaxParts, 256);
    w.o = align_up(w.ml + sizeof(float2) * rows, 256);
    w.bytes = align_up(w.o + sizeof(float) * rows * (size_t)p->D, 256);
    return w;
}

dspark_status check_attention_params(const dspark_attention_params* p) {
    if (!p || p->T < 0 || p->B < 1 || p->Hk < 1 || p->Hq < 1 || p->D < 1 || p->num_pages < 1 || p->max_blocks < 1 ||
        page_shift_of(p->page_size) < 0 || p->window < 0 || ((uintptr_t)p->error & 3u))
        return DSPARK_ERR_INVALID_ARG;
    if (p->Hq % p->Hk || !(p->softcap >= 0.f) || isinf(p->softcap) || !isfinite(p->scale)) return DSPARK_ERR_INVALID_ARG;
    if (p->dtype != DSPARK_BF16 && p->dtype != DSPARK_F16) return DSPARK_ERR_INVALID_ARG;
    if (p->kv_dtype != p->dtype && p->kv_dtype != DSPARK_E4M3) return DSPARK_ERR_INVALID_ARG;
    if (p->D % 16 || p->D > 256 || (long long)p->T * p->Hq > INT32_MAX) return DSPARK_ERR_UNSUPPORTED;
    return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_paged_attention_workspace_size(const dspark_attention_params* p) {
    return check_attention_params(p) == DSPARK_OK ? attn_ws(p).bytes : 0;
}

extern "C" dspark_status dspark_paged_attention(const dspark_attention_params* p, const void* q, const void* k_pages,
                                                const void* v_pages, const int32_t* block_table, const int32_t* seq_len,
                                                const int32_t* offsets, const float* k_scale, const float* v_scale,
                                                void* out, float* lse, void* workspace, size_t ws_bytes,
                                                dspark_stream_t stream) {
    const dspark_status st = check_attention_params(p);
    if (st != DSPARK_OK) return st;
    if (!k_pages || !v_pages || !block_table || !seq_len || (p->T && (!q || !out))) return DSPARK_ERR_INVALID_ARG;
    if (!offsets && p->T < p->B) return DSPARK_ERR_INVALID_ARG;
    const bool e4m3 = p->kv_dtype == DSPARK_E4M3;
    const long long esz = e4m3 ? 1 : 2;
    if ((((uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)out) & 15u) || ((uintptr_t)q & 1u) ||
        (p->kv_page_stride * esz) % 16 || (p->kv_token_stride * esz) % 16 || (p->kv_head_stride * esz) % 16)
        return DSPARK_ERR_INVALID_ARG;
    const AttnWs w = attn_ws(p);
    if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < w.bytes) return DSPARK_ERR_WORKSPACE;
    for (const long long x : {p->kv_page_stride, p->kv_token_stride, p->kv_head_stride})  // 32 bits of 16 bytes
        if (x < 0 || x * esz / 16 > INT32_MAX) return DSPARK_ERR_INVALID_ARG;
    int sms = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    AttnArgs a;
    a.T = p->T;
    a.B = p->B;
    a.Hq = p->Hq;
    a.Hk = p->Hk;
    a.G = p->Hq / p->Hk;
    // Division by G: with 2^(s-1) < G <= 2^s and m = floor(2^(31+s) / G) + 1, m G exceeds 2^(31+s) by at most G
    // <= 2^s, so floor(row m / 2^(31+s)) = floor(row / G) for row < 2^31.
    a.g_shift = 0;
    while ((1ll << a.g_shift) < a.G) ++a.g_shift;
    a.g_mul = (uint32_t)((1ull << (31 + a.g_shift)) / (uint64_t)a.G + 1);
    a.D = p->D;
    a.page_shift = page_shift_of(p->page_size);
    a.num_pages = p->num_pages;
    a.max_blocks = p->max_blocks;
    a.causal = p->causal != 0;
    a.window = p->window;
    a.scale = p->scale;
    // A cap past 2^100 leaves every score as it is (s^2 / 3 c^2 is below 2^-24 for |s| up to 2^88); 1 / c would come near
    // the smallest normal number.
    a.softcap = p->softcap > 0x1p100f ? 0.f : p->softcap;
    a.q = static_cast<const unsigned char*>(q);
    a.q_token = p->q_token_stride;
    a.q_head = p->q_head_stride;
    a.q_vec = !((uintptr_t)q & 15u) && p->q_token_stride % 8 == 0 && p->q_head_stride % 8 == 0;
    a.k_pages = static_cast<const unsigned char*>(k_pages);
    a.v_pages = static_cast<const unsigned char*>(v_pages);
    a.page = p->kv_page_stride * esz;
    a.token = p->kv_token_stride * esz;
    a.head = p->kv_head_stride * esz;
    a.block_table = block_table;
    a.seq_len = seq_len;
    a.offsets = offsets;
    a.k_scale = e4m3 ? k_scale : nullptr;
    a.v_scale = e4m3 ? v_scale : nullptr;
    a.out = static_cast<unsigned char*>(out);
    a.lse = lse;
    a.status = &reinterpret_cast<WsHeader*>(ws)->status;
    a.error = p->error;
    a.items = reinterpret_cast<PartItem*>(ws + w.items);
    a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    a.part_o = reinterpret_cast<float*>(ws + w.o);
    const bool bf16 = p->dtype == DSPARK_BF16;
    a.sum_scale = bf16 && !e4m3 ? ProbScale<true>::kInverse : ProbScale<false>::kInverse;
    int parts = 0;
    const bool tc = wide_rows(p) && a.q_vec;
    const dspark_status ls = tc     ? launch_attn_tc(a, bf16, e4m3, sms, s, &parts)
                             : bf16 ? (e4m3 ? launch_rows16_d<true, true>(a, sms, s, &parts)
                                          : launch_rows16_d<true, false>(a, sms, s, &parts))
                                  : (e4m3 ? launch_rows16_d<false, true>(a, sms, s, &parts)
                                          : launch_rows16_d<false, false>(a, sms, s, &parts));
    if (ls != DSPARK_OK) return ls;
    note_launch();
    const int row_tile = tc ? kTcRows : kRows;
    // The join's blocks become resident as the attention kernel's leave.
    const dim3 grid(parts, 8), block(32 * kJoinWarps);
    const cudaError_t e = bf16 ? launch_overlapped(attn_join_kernel<true>, grid, block, 0, s, a, row_tile, parts)
                               : launch_overlapped(attn_join_kernel<false>, grid, block, 0, s, a, row_tile, parts);
    if (e != cudaSuccess) return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}
