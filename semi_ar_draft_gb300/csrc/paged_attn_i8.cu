// paged_attn_i8.cu -- dspark_paged_attention_i8 for up to eight rows a kv head, a decoding step's (paged.cuh has the split
// of the work and the join, paged_attn_i8_rows.cu more rows, paged_attn_tc.cu many).
//
// With k_l = c_l 2^(e_l) and v_l = d_l 2^(f_l), c and d the codes:
//   s_l = scale (q . c_l) 2^(e_l), capped;  sum = sum_l 2^(s_l log2 e - m)
//   o = sum_l 2^(s_l log2 e - m + f_l - u) d_l;  out = o 2^u / sum
// m follows the largest score of a row and m + u the largest s_l log2 e + f_l, each by itself: a value's weight keeps its bits
// as a half whatever the scales of the blocks before it, and blocks of zeros (whose scale is the smallest there is) do not
// move the sum's reference.  u is held as such: f_l added to a score of 10^7 would be rounded away, and s_l log2 e - m is
// the same number in both sums, so that a row of one key is its value however large the score.  Codes are halves exactly, and so is a query times a power of two; nothing else is rounded
// before the products but the weights.
//
// What bounds it is issue slots as much as the cache's bytes, so everything beside the products has to be little.  Keys and
// values are therefore the products' A operand (16 keys, 16 values of a head), and the rows are B, eight at a time:
// S^T = K Q^T and O^T = V^T P^T.  With the rows in A, as the other caches have them, a decoding step of eight heads a kv
// head computes 16 rows of everything, scores, exponentials and output registers alike.  P^T is S^T's fragment transposed
// (movmatrix).  A warp streams slices of its own through a ring of its own in shared memory, as in paged_attn.cu.
//
// Measured: 32 requests of up to 8192 tokens, 8 kv heads of 128, 57 us = 5.0 TB/s (0.74 of the measured copy rate; the rows
// in A 73 us); 128 requests of up to 8000 tokens 191 us = 5.9 TB/s (0.87; 237 us); heads of 64, 128 requests, 121 us (183
// before the block's warps took a head each); 48 requests of 1000 tokens' window, five rows of 96, 29 us; one request of
// up to 1024 tokens 10.5 us, latency.
#include "host_util.h"
#include "mma16.cuh"
#include "paged.cuh"
#include "pdl.cuh"
#include "tc05.cuh"

namespace dspark {
namespace {

template <int DP, int HG>
struct SliceI8 {
    static constexpr int kKeys = DP == 256 ? 16 : 32;  // keys of a warp's slice
    static constexpr int kMt = kKeys / 16;
    static constexpr int kWarps = 4, kThreads = 32 * kWarps;
    static constexpr int kKeyWarps = kWarps / HG;       // warps of a head, each with slices of its own
    static constexpr int kKeyTile = kKeyWarps * kKeys;  // keys of a unit
    static constexpr int kChunks = DP / 16;          // 16-byte groups of a row
    static constexpr int kHalf = kKeys * DP;         // K (or V) of a slice
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = DP == 64 ? 4 : 2;
    static constexpr int kExtra = 2;  // what an item costs beside its key tiles
    static constexpr int kBlocksPerSm = 3;
    static constexpr bool kQInSmem = DP > 128;    // (else in registers)
    static constexpr int kQBytes = 8 * DP * 2;    // of a head
    static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage + HG * kQBytes;
    static_assert(kStage >= 8 * DP * 4, "a stage holds a warp's output");
    // Rows are a multiple of 128 bytes apart (or 64): the swizzle spreads eight rows' same 16-byte group over all banks.
    static __device__ __forceinline__ uint32_t at(int row, int chunk) {
        const int x = kChunks >= 8 ? (row & 7) : ((row >> 1) & 3);
        return (uint32_t)(row * DP + ((chunk ^ x) << 4));
    }
    static __device__ __forceinline__ uint32_t q_at(int row, int chunk) {  // rows of q as halves
        return (uint32_t)(row * (DP * 2) + ((chunk ^ (row & 7)) << 4));
    }
};


__device__ __forceinline__ void copy16_all(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void store_out4(const AttnArgs& a, long long row, int col, float4 v) {
    uint2 w = make_uint2(pack16<BF16>(v.x, v.y), pack16<BF16>(v.z, v.w));
    *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.D + col) * 2) = w;
}

// a.Hk counts groups of HG heads here.  DU: the values of a head that are worked on, of the DP that a row has room for.
template <bool BF16, int DP, int HG, int DU>
__global__ void __launch_bounds__(SliceI8<DP, HG>::kThreads, SliceI8<DP, HG>::kBlocksPerSm) attn_i8_kernel(AttnArgs a) {
    using C = SliceI8<DP, HG>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kRows = 8, MT = C::kMt;
    constexpr int KS = DU / 16;  // k-steps over the head dimension, and m-tiles of the output
    static_assert(KS % 2 == 0 && DU <= DP, "k-steps come in pairs");
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 s_ml[kWarps][kRows];
    __shared__ int s_err;
    __shared__ AttnScratch s_start;
    // where a row's products begin, its scores' factor in two (score_factor): rows of the first head, of the second, ...
    __shared__ __align__(8) float s_base[HG * kRows], s_scale[HG * kRows], s_far[HG * kRows];
    __shared__ AttnStart s_range;                    // the block's units
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int my_head = warp % HG, my_keys = warp / HG;  // of the group's heads, of the unit's slices
    const int part = blockIdx.x, parts = gridDim.x;
    wait_primary();
    launch_dependents();
    if (tid == 0) s_err = 0;
    bool bad;
    const AttnStart start = attn_start<kThreads>(a, kRows, C::kKeyTile, C::kExtra, parts, part, 1, &s_start, &bad);

    attn_tail_rows(a, (size_t)part * kThreads + tid, (size_t)parts * kThreads);
    unsigned char* ring = smem + (size_t)warp * C::kStages * C::kStage;
    const uint32_t ring_addr = smem_addr(ring);
    unsigned char* qs = smem + (size_t)kWarps * C::kStages * C::kStage;
    const uint32_t qs_addr = smem_addr(qs) + my_head * C::kQBytes;
    int err = bad ? DSPARK_ERR_CACHE : 0;
    if (tid == 0) s_range = start;  // (read by this thread)

    // ---- loads: `ld` walks ahead of the arithmetic; `pid` is the page of this lane's key of its slice
    AttnWalk ld = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    int ld_group = ld.done() ? 0 : ld.item / ld.rts;
    auto slice_key = [&](const AttnWalk& w) { return (w.kt_first + w.kt) * C::kKeyTile + my_keys * C::kKeys; };
    auto fetch_page = [&]() -> int {
        const int key = slice_key(ld) + lane;
        if (ld.done() || lane >= C::kKeys || key >= ld.r.seq) return -1;
        return __ldg(a.block_table + (size_t)ld.j * a.max_blocks + (key >> a.page_shift));
    };
    int pid = fetch_page();
    int ld_stage = 0;
    // An item's queries, asked for (into L1) when its first keys are.
    auto touch_queries = [&]() {
        const int first = (ld.item - ld_group * ld.rts) * kRows;
        const int last = min(ld.r.n * a.G, first + kRows);
        for (int i = lane; i < HG * kRows * (DP / 64); i += 32) {
            const int head = ld_group * HG + i / (kRows * (DP / 64)), row = first + i / (DP / 64) % kRows;
            const int token = attn_token(a, row), d = 64 * (i % (DP / 64));
            if (row < last && d < a.D)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + 2 * ((ld.r.token0 + token) * a.q_token +
                                                                        (head * a.G + row - token * a.G) * a.q_head + d)));
        }
    };
    if (warp == 0 && !ld.done()) touch_queries();
    // The exponents of this lane's key of the slices on their way, as they arrive; [0] are those of the slice in hand.
    uint32_t k_exp[C::kStages], v_exp[C::kStages];
    auto load_step = [&](int queue) {
        k_exp[queue] = v_exp[queue] = 0;
        if (!ld.done() && slice_key(ld) < ld.r.seq) {
            const int key = slice_key(ld) + lane, place = key & ((1 << a.page_shift) - 1), head = ld_group * HG + my_head;
            const bool live = lane < C::kKeys && key < ld.r.seq && key >= ld.r.lo;
            const bool found = live && pid >= 0 && pid < a.num_pages;
            if (live && !found) err = DSPARK_ERR_CACHE;
            const Steps32& by = a.steps;
            if (found) {
                const uint32_t e = pid * by.e_page + (place >> a.exp.shift) * by.e_block + head * by.e_head;
                k_exp[queue] = __ldg(a.exp.k + e);
                v_exp[queue] = __ldg(a.exp.v + e);
            }
            const uint32_t off = found ? pid * by.page + place * by.token + head * by.head : kNoKey;
            const uint32_t dst = ring_addr + ld_stage * C::kStage;
            constexpr int kPer = 32 / C::kChunks;  // rows a warp copies at a time
            const int chunk = lane % C::kChunks;
            const unsigned char *k_from = a.k_pages + chunk * 16, *v_from = a.v_pages + chunk * 16;
            // What is not there is not copied: the bytes that a stage still holds are codes too, and finite ones, which meet
            // queries of zero, weights of zero or values that nobody stores.
#pragma unroll
            for (int i = 0; i < C::kKeys / kPer; ++i) {
                const int row = i * kPer + lane / C::kChunks;
                const uint32_t o = __shfl_sync(0xffffffffu, off, row);
                if (chunk * 16 < a.D && o != kNoKey) {
                    copy16_all(dst + C::at(row, chunk), k_from + (uint64_t)o * by.unit);
                    copy16_all(dst + C::kHalf + C::at(row, chunk), v_from + (uint64_t)o * by.unit);
                }
            }
        }
        cp_async_commit();
        if (++ld_stage == C::kStages) ld_stage = 0;
        if (!ld.done()) {
            walk_next(a, ld, kRows, C::kKeyTile);
            pid = fetch_page();
            if (ld.kt == 0 && !ld.done()) {
                ld_group = ld.item / ld.rts;
                if (warp == 0) touch_queries();
            }
        }
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load_step(i + 1);

    // ---- arithmetic
    AttnWalk w = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    PartItem* mine = a.items + part;  // written by thread 0
    if (tid == 0) mine->d[kTail].first = mine->d[kHead].first = -1;
    float o[KS][4];  // of 16 values of the head: values 2 g (rows 2 t, 2 t + 1), 2 g + 1
    uint32_t qf[C::kQInSmem ? 1 : KS][2];
    const float cap_out = a.softcap * kLog2e;
    constexpr float kUp = ProbScale<false>::kBits;
    // What is taken off the scores for the sums, kUp less than the largest that a row followed, and off their differences and
    // the values' exponents for the weights (kNone: the row has seen nothing); and the sums.
    constexpr float kNone = -3.4028234e38f;
    float ref[2], ref_u[2];
    uint64_t sums;
    int all_lo = 0, all_hi = 0, rows = 0, group = 0, row0 = 0, seg_first = 0;
    bool fresh = true, far = false;  // far: some row's second factor counts
    int st = 0;
    // The queries' fragments of k-steps ks and ks + 1.
    auto load_q = [&](uint32_t (&b)[4], int ks) { ldsm4(b, qs_addr + C::q_at(lane & 7, 2 * ks + (lane >> 3))); };
    while (!w.done()) {
        if (fresh) {  // a new segment: its rows, their queries and what each may see
            fresh = false;
            seg_first = w.kt;
            group = w.item / w.rts;
            row0 = (w.item - group * w.rts) * kRows;
            rows = min(w.r.n * a.G - row0, kRows);
            all_lo = attn_see_lo(a, w.r, attn_token(a, row0 + rows - 1));
            all_hi = attn_see_hi(a, w.r, attn_token(a, row0));
            // The queries, through shared memory: 16 bytes a thread, then fragments by ldmatrix.  (The previous segment's
            // readers are past its last barrier.)
            constexpr int kQc = DP / 8;  // threads of a row
            bool row_far = false;
            constexpr int kQRows = HG * kRows, kQSteps = (kQRows * kQc + kThreads - 1) / kThreads;
#pragma unroll
            for (int u = 0; u < kQSteps; ++u) {
                const int qrow = (tid + u * kThreads) / kQc, c = (tid + u * kThreads) % kQc;
                if (kQRows * kQc % kThreads && qrow >= kQRows) break;  // (whole warps)
                const int row = qrow % kRows, head = group * HG + qrow / kRows, token = attn_token(a, row0 + row);
                uint32_t y[4] = {0, 0, 0, 0};
                if (row < rows && 8 * c < a.D) {
                    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (w.r.token0 + token) * a.q_token +
                                          (head * a.G + row0 + row - token * a.G) * a.q_head + 8 * c;
                    if (a.q_vec) {
                        const uint4 q = __ldg(reinterpret_cast<const uint4*>(src));
                        y[0] = q.x, y[1] = q.y, y[2] = q.z, y[3] = q.w;
                    } else {  // rows may start at any element
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = (uint32_t)__ldg(src + 2 * e) | ((uint32_t)__ldg(src + 2 * e + 1) << 16);
                    }
                }
                float sum;
                const int raise = query_halves<BF16, kQc>(y, sum);
                // Codes arrive four k a lane and are taken apart by even and odd bytes: the MMA's k slots 2t, 2t + 1 hold
                // k = 4t, 4t + 2 and its slots 2t + 8, 2t + 9 hold k = 4t + 1, 4t + 3.
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int at = 4 * (e + 2 * (c & 1));
                    *reinterpret_cast<uint32_t*>(qs + C::q_at(qrow, c & ~1) + at) = __byte_perm(y[2 * e], y[2 * e + 1], 0x5410);
                    *reinterpret_cast<uint32_t*>(qs + C::q_at(qrow, c | 1) + at) = __byte_perm(y[2 * e], y[2 * e + 1], 0x7632);
                }
                if (c == 0) {
                    const ScoreFactor f = score_factor(a, raise);
                    s_base[qrow] = -128.f * 0x1p-24f * sum;
                    s_scale[qrow] = f.near;
                    s_far[qrow] = f.far;
                    row_far |= f.far != 1.f;
                }
            }
            far = __syncthreads_or(row_far);
            ref[0] = ref[1] = 0.f;
            ref_u[0] = ref_u[1] = kNone;
            sums = 0;
            if (!C::kQInSmem) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t b[4];
                    load_q(b, ks);
#pragma unroll
                    for (int e = 0; e < 4; ++e) qf[C::kQInSmem ? 0 : ks + (e >> 1)][e & 1] = b[e];
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i + 1 < C::kStages; ++i) {
            k_exp[i] = k_exp[i + 1];
            v_exp[i] = v_exp[i + 1];
        }
        load_step(C::kStages - 1);
        cp_async_wait_group<C::kStages - 1>();
        __syncwarp();
        const int key0 = slice_key(w);
        if (key0 < w.r.seq) {
            const uint32_t kb = ring_addr + st * C::kStage, vb = kb + C::kHalf;
            // ---- S^T: lane (g, t) gets keys 16 i + g (h = 0) and + 8, of rows 2 t and 2 t + 1
            float s[MT][4];
            const float2 base = *reinterpret_cast<const float2*>(&s_base[my_head * kRows + 2 * t]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                s[i][0] = s[i][2] = base.x;
                s[i][1] = s[i][3] = base.y;
            }
            // Four k of keys g and g + 8.  A byte alone in a half is the subnormal number byte 2^-24, so a key's code needs
            // no arithmetic: code + 128 goes in, and the products begin at - 128 times the sum of the row's query instead
            // of zero.  (What fp32 loses by that is 2^-24 of 128 sum |q|, the error of 2^-16 of a code.)
            auto codes_a = [](uint32_t (&f)[4], uint32_t lo, uint32_t hi) {
                f[0] = (lo & 0x00ff00ffu) ^ 0x00800080u;
                f[1] = (hi & 0x00ff00ffu) ^ 0x00800080u;
                f[2] = ((lo >> 8) & 0x00ff00ffu) ^ 0x00800080u;
                f[3] = ((hi >> 8) & 0x00ff00ffu) ^ 0x00800080u;
            };
#pragma unroll
            for (int ks = 0; ks < KS; ks += 2) {
                uint32_t q[4];
                if (C::kQInSmem) {
                    load_q(q, ks);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = qf[C::kQInSmem ? 0 : ks + (e >> 1)][e & 1];
                }
                uint32_t b[2][4];
                if (MT == 2) {  // matrix i: keys 8 i .. 8 i + 7
                    ldsm4(b[0], kb + C::at(lane, ks));
                    ldsm4(b[1], kb + C::at(lane, ks + 1));
                } else {  // keys 0 .. 7, 8 .. 15 of both k-steps
                    ldsm4(b[0], kb + C::at(lane & 15, ks + (lane >> 4)));
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t f[4];
                        if (MT == 2)
                            codes_a(f, b[u][2 * i], b[u][2 * i + 1]);
                        else
                            codes_a(f, b[0][2 * u], b[0][2 * u + 1]);
                        mma16<false>(s[i], f, q[2 * u], q[2 * u + 1]);
                    }
            }
            // each key's 2^e (as bf16, in the low half) and its values' e (as bf16), from the lane of the key's number
            const uint32_t both = (uint32_t)(exponent_of<BF16>(k_exp[0]) + 127) << 7 |
                                  (__float_as_uint((float)exponent_of<BF16>(v_exp[0])) & 0xffff0000u);
            float key_scale[MT][2], value_exp[MT][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = __shfl_sync(0xffffffffu, both, 16 * i + 8 * h + g);
                    key_scale[i][h] = __uint_as_float(x << 16);
                    value_exp[i][h] = __uint_as_float(x & 0xffff0000u);
                }
            // scores in the log2 domain, hidden ones -inf
            const float2 row_scale = *reinterpret_cast<const float2*>(&s_scale[my_head * kRows + 2 * t]);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = up2(mul2(mul2(pk2(s[i][2 * h], s[i][2 * h + 1]), pk2(row_scale.x, row_scale.y)),
                                              pk2(key_scale[i][h], key_scale[i][h])));
                    s[i][2 * h] = x.x;
                    s[i][2 * h + 1] = x.y;
                }
            if (far) {
                const float2 f = *reinterpret_cast<const float2*>(&s_far[my_head * kRows + 2 * t]);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[i][2 * h] *= f.x;
                        s[i][2 * h + 1] *= f.y;
                    }
            }
            if (a.softcap > 0.f) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 x = softcap2(s[i][2 * h], s[i][2 * h + 1], 1.f, cap_out);
                        s[i][2 * h] = x.x;
                        s[i][2 * h + 1] = x.y;
                    }
            }
            if (key0 < all_lo || key0 + C::kKeys > all_hi) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int token = attn_token(a, row0 + 2 * t + r);
                    const int lo = attn_see_lo(a, w.r, token), hi = 2 * t + r < rows ? attn_see_hi(a, w.r, token) : 0;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + 16 * i + 8 * h + g;
                            if (key < lo || key >= hi) s[i][2 * h + r] = -CUDART_INF_F;
                        }
                }
            }
            // s becomes the differences from the row's reference.  The references follow a row's maxima only when these are 2^8
            // ahead (values up to 2^8 lose nothing), so most slices need no maximum over the lanes and do not touch the
            // output.  Each row's by itself: what another row sees must not decide how this one's weights are rounded.
            float mx[2], mz[2];
            bool grow = false;
            auto take = [&](float x, float y) {  // off the differences
                const uint64_t both = pk2(-x, -y);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 e = up2(add2(pk2(s[i][2 * h], s[i][2 * h + 1]), both));
                        s[i][2 * h] = e.x;
                        s[i][2 * h + 1] = e.y;
                    }
            };
            auto largest = [&](int r) {  // of the lane's differences of a row, and with the values' exponents
                mx[r] = mz[r] = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    mx[r] = fmax3(mx[r], s[i][r], s[i][2 + r]);
                    mz[r] = fmax3(mz[r], s[i][r] + value_exp[i][0], s[i][2 + r] + value_exp[i][1]);
                }
            };
            take(ref[0], ref[1]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                largest(r);
                grow |= mx[r] > kUp + 8.f || mz[r] > ref_u[r] + (kUp + 8.f);
            }
            if (__any_sync(0xffffffffu, grow)) {
                float by[2], down[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], d));
                    const bool first = ref_u[r] == kNone && mx[r] > -CUDART_INF_F;  // (scores, not differences yet)
                    by[r] = first || mx[r] > kUp + 8.f ? mx[r] - kUp : 0.f;
                    down[r] = first ? 1.f : ex2(-by[r]);  // (the first time the sum is 0)
                    ref[r] += by[r];
                }
                take(by[0], by[1]);
                sums = mul2(sums, pk2(down[0], down[1]));
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    largest(r);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mz[r] = fmaxf(mz[r], __shfl_xor_sync(0xffffffffu, mz[r], d));
                    const float was = ref_u[r] == kNone ? kNone : ref_u[r] - by[r];
                    ref_u[r] = mz[r] > was + (kUp + 8.f) ? mz[r] - kUp : was;
                    const float f = ex2(was - ref_u[r]);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[i][r] *= f;
                        o[i][2 + r] *= f;
                    }
                }
            }
            // ---- P^T as halves, fragments of the second product's B
            uint32_t p[MT][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t e = pk2(s[i][2 * h], s[i][2 * h + 1]);
                    const float2 z = up2(add2(add2(e, pk2(value_exp[i][h], value_exp[i][h])), pk2(-ref_u[0], -ref_u[1])));
                    sums = add2(sums, pk2(ex2(s[i][2 * h]), ex2(s[i][2 * h + 1])));
                    p[i][h] = transpose8x8(pack16<false>(ex2(z.x), ex2(z.y)));
                }
            // ---- O^T += V^T P^T: bytes (k0 d0, k0 d1, k1 d0, k1 d1) are rows 2 g and 2 g + 1 of the m-tile, which are
            // its rows g and g + 8 to the MMA.  (What nobody sees needs no care: codes are finite.)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int c = 0; c < KS; c += 2) {
                    uint32_t b[4];
                    ldsm4_trans(b, vb + C::at(16 * i + (lane & 15), c + (lane >> 4)));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t x = b[2 * u] ^ 0x80808080u, y = b[2 * u + 1] ^ 0x80808080u;
                        const uint32_t f[4] = {i8x2_to_half2<kBytes02>(x), i8x2_to_half2<kBytes13>(x), i8x2_to_half2<kBytes02>(y),
                                               i8x2_to_half2<kBytes13>(y)};
                        mma16<false>(o[c + u], f, p[i][0], p[i][1]);
                    }
                }
        }
        __syncwarp();  // the slice has been read by every lane

        const bool last_of_item = w.kt + 1 == w.kts;
        if (last_of_item || w.left == 1) {
            // ---- the warps' parts of the segment meet, in the stages just consumed
            float* mine_o = reinterpret_cast<float*>(ring + st * C::kStage);
            auto o_at = [](int row, int col) { return row * DP + (col ^ (((row >> 1) & 3) << 4)); };
            const float2 both = up2(sums);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = r ? both.y : both.x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (g == 0) s_ml[warp][2 * t + r] = make_float2(ref_u[r] == kNone ? -CUDART_INF_F : ref[r] + kUp, l);
                // Averages, which are no larger than the values (127 2^121 is nearly fp32's largest number); to the
                // reference of the sums in two steps, since 2^f may be as large as that too.
                const float f = ex2(0.5f * ref_u[r]), inv = l == 0.f ? 0.f : __fdividef(1.f, l);
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    *reinterpret_cast<float2*>(mine_o + o_at(2 * t + r, 16 * i + 2 * g)) =
                        make_float2(o[i][r] * inv * f * f, o[i][2 + r] * inv * f * f);
            }
            __syncthreads();
            const bool whole = last_of_item && seg_first == 0;
            const int slot = 2 * part + (seg_first == 0 ? kHead : kTail);
            for (int i = tid; i < HG * kRows * (DP / 4); i += kThreads) {
                const int hd = i / (kRows * (DP / 4)), head = group * HG + hd;
                const int row = i / (DP / 4) % kRows, col = 4 * (i % (DP / 4));
                if (row >= rows) continue;
                float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
                for (int x = hd; x < kWarps; x += HG) mm = fmaxf(mm, s_ml[x][row].x);
                const float ref = mm == -CUDART_INF_F ? 0.f : mm;
                float weight[C::kKeyWarps];
#pragma unroll
                for (int x = 0; x < C::kKeyWarps; ++x) {
                    const float2 ml = s_ml[hd + x * HG][row];
                    weight[x] = ml.y == 0.f ? 0.f : ml.y * ex2(ml.x - ref);  // (0: saw nothing)
                    ll += weight[x];
                }
                const float inv = ll == 0.f ? 0.f : __fdividef(1.f, ll);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < C::kKeyWarps; ++x) {
                    const float f = weight[x] * inv;
                    const float4 y = *reinterpret_cast<const float4*>(
                        smem + (size_t)((hd + x * HG) * C::kStages + st) * C::kStage + 4 * o_at(row, col));
                    v.x = fmaf(y.x, f, v.x);
                    v.y = fmaf(y.y, f, v.y);
                    v.z = fmaf(y.z, f, v.z);
                    v.w = fmaf(y.w, f, v.w);
                }
                if (whole) {
                    const long long at = attn_out_row(a, w.r.token0, head, row0 + row);
                    if (col < a.D) store_out4<BF16>(a, at, col, v);
                    if (a.lse && col == 0)
                        a.lse[at] = ll == 0.f ? -CUDART_INF_F : (mm + lg2(ll * ProbScale<false>::kInverse)) * kLn2;
                } else {
                    const size_t at = (size_t)slot * (HG * kRows) + hd * kRows + row;
                    if (col < a.D) *reinterpret_cast<float4*>(a.part_o + at * a.D + col) = v;
                    if (col == 0) a.part_ml[at] = make_float2(mm, ll);
                }
            }
            if (!whole && tid == 0) mine->d[seg_first == 0 ? kHead : kTail] = part_desc(s_range, w, row0, rows, group);
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

template <bool BF16, int DP, int HG, int DU = DP>
dspark_status launch_slices(AttnArgs a, int sms, cudaStream_t s, int* parts) {
    using C = SliceI8<DP, HG>;
    int per_sm = 0;
    auto fn = attn_i8_kernel<BF16, DP, HG, DU>;
    if (prepare_kernel((const void*)fn, C::kSmem, C::kThreads, &per_sm) != cudaSuccess || per_sm < 1) return DSPARK_ERR_CUDA;
    int n = sms * (per_sm < C::kBlocksPerSm ? per_sm : C::kBlocksPerSm);
    if (n > kMaxParts) n = kMaxParts;
    *parts = n;
    a.Hk /= HG;
    return launch_overlapped(fn, n, C::kThreads, C::kSmem, s, a) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
template <bool BF16>
dspark_status launch_slices_d(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    const int heads = i8_head_group(a.D, a.Hk);
    if (a.D <= 64) {
        if (heads == 4) return launch_slices<BF16, 64, 4>(a, sms, s, parts);
        return heads == 2 ? launch_slices<BF16, 64, 2>(a, sms, s, parts) : launch_slices<BF16, 64, 1>(a, sms, s, parts);
    }
    // Three quarters of the room, where that is enough: heads of 96, 32 requests up to 8192 tokens, 51 against 56 us; of 80,
    // 370 requests up to 1508, 205 against 221; of 192, 300 requests up to 596, 154 against 176.
    if (a.D <= 96) return heads == 2 ? launch_slices<BF16, 128, 2, 96>(a, sms, s, parts) : launch_slices<BF16, 128, 1, 96>(a, sms, s, parts);
    if (a.D <= 128) return heads == 2 ? launch_slices<BF16, 128, 2>(a, sms, s, parts) : launch_slices<BF16, 128, 1>(a, sms, s, parts);
    return a.D <= 192 ? launch_slices<BF16, 256, 1, 192>(a, sms, s, parts) : launch_slices<BF16, 256, 1>(a, sms, s, parts);
}

}  // namespace

// Heads that lie side by side are read together where one head's row is less than a 128-byte line or not many: the warps
// of a block take a head each.  (Otherwise the lines that two heads share are read twice, by blocks far apart in time: 128
// requests up to 3000 tokens, 8 heads of 64: 445 MB read for 223.)
int i8_head_group(int D, int Hk) {
    if (D <= 64 && Hk % 4 == 0) return 4;
    return D <= 128 && Hk % 2 == 0 ? 2 : 1;
}

dspark_status launch_attn_i8(const AttnArgs& a, bool bf16, int sms, cudaStream_t s, int* parts) {
    return bf16 ? launch_slices_d<true>(a, sms, s, parts) : launch_slices_d<false>(a, sms, s, parts);
}

}  // namespace dspark
