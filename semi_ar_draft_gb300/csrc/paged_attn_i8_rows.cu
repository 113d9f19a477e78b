// paged_attn_i8_rows.cu -- dspark_paged_attention_i8 for 9 to some 32 rows a kv head (several new tokens a request, or many
// query heads a kv head): row tiles of 16.  paged_attn_i8.cu has the arithmetic, paged.cuh the split of the work and the
// join.
//
// A block's four warps share a tile of 128 keys (64 with heads past 128), and every code is widened once: for S^T = K Q^T a
// warp takes a quarter of the keys, for O^T = V^T P^T a quarter of the head's values.  P^T goes from one to the other
// through shared memory.  A row's references are the block's: whether one has to follow is asked of all warps at a
// barrier that a tile needs anyway.  Outputs need no meeting of the warps, each has all keys of its values; only sums do.
//
// Bound by issue slots (about half of them are used by twelve warps a multiprocessor).  Measured, against the 8-row
// kernel's layout with two row tiles a warp: 32 requests of up to 8192 tokens, 16 rows, 8 kv heads of 128: 73 us (82);
// 64 requests, 23 rows, 4 kv heads: 65 us (79).  Three contexts of up to 200000 tokens, two or three tiles of 16
// rows of 256, softcap: 164 us, each tile reading the cache for itself (752 MB for 264, 4.6 TB/s).  Row tiles of 32 and 64
// need more registers or shared memory than three blocks a multiprocessor leave: 105 and 207 us for the first case.
#include "host_util.h"
#include "mma16.cuh"
#include "paged.cuh"
#include "pdl.cuh"
#include "tc05.cuh"

namespace dspark {
namespace {

constexpr int kRows = 16;
constexpr int NT = kRows / 8;  // n-tiles of rows

template <int DP>
struct RowsI8 {
    static constexpr int kWarps = 4, kThreads = 32 * kWarps;
    static constexpr int kMt = DP == 256 ? 1 : 2;    // m-tiles of a warp's keys
    static constexpr int kKeys = 16 * kMt;           // keys of a tile that a warp takes
    static constexpr int kKeyTile = kKeys * kWarps;  // keys of a unit
    static constexpr int kChunks = DP / 16;       // 16-byte groups of a row
    static constexpr int kHalf = kKeyTile * DP;   // K (or V) of a tile
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = DP == 64 ? 3 : 2;
    static constexpr int kExtra = 1;     // what an item costs beside its key tiles
    static constexpr int kBlocksPerSm = 3;
    static constexpr int kQBytes = kRows * DP * 2;
    // The weights of a tile lie over its keys, which every warp has done with by then.
    static_assert(kRows * kKeyTile * 2 <= kHalf, "room for the weights");
    static constexpr size_t kSmem = (size_t)kStages * kStage + kQBytes;
    static __device__ __forceinline__ uint32_t at(int row, int chunk) {  // of codes
        const int x = kChunks >= 8 ? (row & 7) : ((row >> 1) & 3);
        return (uint32_t)(row * DP + ((chunk ^ x) << 4));
    }
    static __device__ __forceinline__ uint32_t q_at(int row, int chunk) {  // rows of q as halves
        return (uint32_t)(row * (DP * 2) + ((chunk ^ (row & 7)) << 4));
    }
    static __device__ __forceinline__ uint32_t p_at(int row, int chunk) {  // eight keys' weights of a row
        return (uint32_t)(row * (kKeyTile * 2) + ((chunk ^ (row & 7)) << 4));
    }
};


__device__ __forceinline__ void copy16_all(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Four 8 x 8 matrices of 16-bit values, each transposed on its way to shared memory.
__device__ __forceinline__ void stsm4_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}

// DU: the values of a head that are worked on, of the DP that a row has room for.
template <bool BF16, int DP, int DU>
__global__ void __launch_bounds__(RowsI8<DP>::kThreads, RowsI8<DP>::kBlocksPerSm) attn_i8_rows_kernel(AttnArgs a) {
    using C = RowsI8<DP>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps, MT = C::kMt;
    constexpr int KS = DU / 16;  // k-steps over the head dimension
    constexpr int DM = DU / 64;  // 16-value groups of a warp's quarter of a head
    constexpr int R = 2 * NT;    // rows of a lane: 8 j + 2 t + (0, 1)
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_max[2][kWarps][kRows];  // a tile's largest scores, and weights' exponents
    __shared__ float s_sum[kWarps][kRows];
    __shared__ int s_err;
    __shared__ AttnScratch s_start;
    // where a row's products begin, its scores' factor in two (score_factor)
    __shared__ __align__(8) float s_base[kRows], s_scale[kRows], s_far[kRows];
    __shared__ AttnStart s_range;                     // the block's units
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int part = blockIdx.x, parts = gridDim.x;
    wait_primary();
    launch_dependents();
    if (tid == 0) s_err = 0;
    bool bad;
    const AttnStart start = attn_start<kThreads>(a, kRows, C::kKeyTile, C::kExtra, parts, part, 1, &s_start, &bad);

    attn_tail_rows(a, (size_t)part * kThreads + tid, (size_t)parts * kThreads);
    const uint32_t ring = smem_addr(smem);
    unsigned char* qs = smem + (size_t)C::kStages * C::kStage;
    const uint32_t qs_addr = smem_addr(qs);
    int err = bad ? DSPARK_ERR_CACHE : 0;
    if (tid == 0) s_range = start;  // (read by this thread)

    // ---- loads: `ld` walks ahead of the arithmetic; a lane looks up one of the warp's keys
    AttnWalk ld = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    int ld_head = ld.done() ? 0 : ld.item / ld.rts;
    auto tile_key = [&](const AttnWalk& w) { return (w.kt_first + w.kt) * C::kKeyTile + C::kKeys * warp; };
    auto fetch_page = [&]() -> int {
        const int key = tile_key(ld) + lane;
        if (ld.done() || lane >= C::kKeys || key >= ld.r.seq) return -1;
        return __ldg(a.block_table + (size_t)ld.j * a.max_blocks + (key >> a.page_shift));
    };
    int pid = fetch_page();
    int ld_stage = 0;
    // The exponents of this lane's key of the tiles on their way, as they arrive; [0] are those of the tile in hand.
    uint32_t k_exp[C::kStages], v_exp[C::kStages];
    auto load_step = [&](int queue) {
        k_exp[queue] = v_exp[queue] = 0;
        if (!ld.done() && tile_key(ld) < ld.r.seq) {
            const int key = tile_key(ld) + lane, place = key & ((1 << a.page_shift) - 1);
            const bool live = lane < C::kKeys && key < ld.r.seq && key >= ld.r.lo;
            const bool found = live && pid >= 0 && pid < a.num_pages;
            if (live && !found) err = DSPARK_ERR_CACHE;
            const Steps32& by = a.steps;
            if (found) {
                const uint32_t e = pid * by.e_page + (place >> a.exp.shift) * by.e_block + ld_head * by.e_head;
                k_exp[queue] = __ldg(a.exp.k + e);
                v_exp[queue] = __ldg(a.exp.v + e);
            }
            const uint32_t off = found ? pid * by.page + place * by.token + ld_head * by.head : kNoKey;
            const uint32_t dst = ring + ld_stage * C::kStage;
            constexpr int kPer = 32 / C::kChunks;  // rows a warp copies at a time
            const int chunk = lane % C::kChunks;
            const unsigned char *k_from = a.k_pages + chunk * 16, *v_from = a.v_pages + chunk * 16;
            // (What is not there is not copied: see paged_attn_i8.cu.)
#pragma unroll
            for (int i = 0; i < C::kKeys / kPer; ++i) {
                const int row = i * kPer + lane / C::kChunks;
                const uint32_t o = __shfl_sync(0xffffffffu, off, row);
                if (chunk * 16 < a.D && o != kNoKey) {
                    copy16_all(dst + C::at(C::kKeys * warp + row, chunk), k_from + (uint64_t)o * by.unit);
                    copy16_all(dst + C::kHalf + C::at(C::kKeys * warp + row, chunk), v_from + (uint64_t)o * by.unit);
                }
            }
        }
        cp_async_commit();
        if (++ld_stage == C::kStages) ld_stage = 0;
        if (!ld.done()) {
            walk_next(a, ld, kRows, C::kKeyTile);
            pid = fetch_page();
            if (ld.kt == 0 && !ld.done()) ld_head = ld.item / ld.rts;
        }
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load_step(i + 1);

    // ---- arithmetic
    AttnWalk w = walk_begin(a, start, kRows, C::kKeyTile, C::kExtra);
    PartItem* mine = a.items + part;  // written by thread 0
    if (tid == 0) mine->d[kTail].first = mine->d[kHead].first = -1;
    float o[DM][NT][4];  // [16 of the warp's values][8 rows]: values 2 g (rows 2 t, 2 t + 1), 2 g + 1
    const float cap_out = a.softcap * kLog2e;
    constexpr float kUp = ProbScale<false>::kBits, kNone = -3.4028234e38f;  // (as in paged_attn_i8.cu)
    float ref[R], ref_u[R];
    uint64_t sums[NT];  // of rows 8 j + 2 t and the next
    int all_lo = 0, all_hi = 0, rows = 0, head = 0, row0 = 0, seg_first = 0;
    bool fresh = true, far = false;  // far: some row's second factor counts
    int st = 0;
    auto row_of = [&](int r) { return 8 * (r >> 1) + 2 * t + (r & 1); };
    while (!w.done()) {
        if (fresh) {  // a new segment: its rows, their queries and what each may see
            fresh = false;
            seg_first = w.kt;
            head = w.item / w.rts;
            row0 = (w.item - head * w.rts) * kRows;
            rows = min(w.r.n * a.G - row0, kRows);
            all_lo = attn_see_lo(a, w.r, attn_token(a, row0 + rows - 1));
            all_hi = attn_see_hi(a, w.r, attn_token(a, row0));
            // The queries, through shared memory: 16 bytes a thread, then fragments by ldmatrix.  (The previous segment's
            // readers are past its last barrier.)
            constexpr int kQc = DP / 8;  // threads of a row
            constexpr int kQSteps = kRows * kQc / kThreads;
            static_assert(kRows * kQc % kThreads == 0, "whole steps");
            bool row_far = false;
#pragma unroll
            for (int u = 0; u < kQSteps; ++u) {
                const int row = (tid + u * kThreads) / kQc, c = (tid + u * kThreads) % kQc, token = attn_token(a, row0 + row);
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
                // the MMA's k slots 2t, 2t + 1 hold k = 4t, 4t + 2 and its slots 2t + 8, 2t + 9 hold k = 4t + 1, 4t + 3
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int at = 4 * (e + 2 * (c & 1));
                    *reinterpret_cast<uint32_t*>(qs + C::q_at(row, c & ~1) + at) = __byte_perm(y[2 * e], y[2 * e + 1], 0x5410);
                    *reinterpret_cast<uint32_t*>(qs + C::q_at(row, c | 1) + at) = __byte_perm(y[2 * e], y[2 * e + 1], 0x7632);
                }
                if (c == 0) {
                    const ScoreFactor f = score_factor(a, raise);
                    s_base[row] = -128.f * 0x1p-24f * sum;
                    s_scale[row] = f.near;
                    s_far[row] = f.far;
                    row_far |= f.far != 1.f;
                }
            }
            far = __syncthreads_or(row_far);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ref[r] = 0.f;
                ref_u[r] = kNone;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[j] = 0;
#pragma unroll
            for (int i = 0; i < DM; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i + 1 < C::kStages; ++i) {
            k_exp[i] = k_exp[i + 1];
            v_exp[i] = v_exp[i + 1];
        }
        cp_async_wait_group<C::kStages - 2>();
        __syncwarp();
        const int key0 = tile_key(w);
        const uint32_t kb = ring + st * C::kStage, vb = kb + C::kHalf;
        // ---- S^T: lane (g, t) gets keys 16 i + g (h = 0) and + 8 of the warp's, of rows 8 j + 2 t and the next
        float s[MT][NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 base = *reinterpret_cast<const float2*>(&s_base[8 * j + 2 * t]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                s[i][j][0] = s[i][j][2] = base.x;
                s[i][j][1] = s[i][j][3] = base.y;
            }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
            uint32_t b[2][4];
            if (MT == 2) {  // matrix i: keys 8 i .. 8 i + 7
                ldsm4(b[0], kb + C::at(C::kKeys * warp + lane, ks));
                ldsm4(b[1], kb + C::at(C::kKeys * warp + lane, ks + 1));
            } else {  // keys 0 .. 7, 8 .. 15 of both k-steps
                ldsm4(b[0], kb + C::at(C::kKeys * warp + (lane & 15), ks + (lane >> 4)));
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t f[MT][4];  // four k of keys g and g + 8, as subnormal halves
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t lo = MT == 2 ? b[u][2 * i] : b[0][2 * u], hi = MT == 2 ? b[u][2 * i + 1] : b[0][2 * u + 1];
                    f[i][0] = (lo & 0x00ff00ffu) ^ 0x00800080u;
                    f[i][1] = (hi & 0x00ff00ffu) ^ 0x00800080u;
                    f[i][2] = ((lo >> 8) & 0x00ff00ffu) ^ 0x00800080u;
                    f[i][3] = ((hi >> 8) & 0x00ff00ffu) ^ 0x00800080u;
                }
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t q[4];
                    ldsm4(q, qs_addr + C::q_at(8 * j + (lane & 7) + (lane >> 4) * 8, 2 * (ks + u) + ((lane >> 3) & 1)));
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        mma16<false>(s[i][j], f[i], q[0], q[1]);
                        mma16<false>(s[i][j + 1], f[i], q[2], q[3]);
                    }
                }
            }
        }
        // scores in the log2 domain, hidden ones -inf
        float key_scale[MT][2], value_exp[MT][2];
        {
            const uint32_t both = (uint32_t)(exponent_of<BF16>(k_exp[0]) + 127) << 7 |
                                  (__float_as_uint((float)exponent_of<BF16>(v_exp[0])) & 0xffff0000u);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = __shfl_sync(0xffffffffu, both, 16 * i + 8 * h + g);
                    key_scale[i][h] = __uint_as_float(x << 16);
                    value_exp[i][h] = __uint_as_float(x & 0xffff0000u);
                }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 f = *reinterpret_cast<const float2*>(&s_scale[8 * j + 2 * t]);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = up2(mul2(mul2(pk2(s[i][j][2 * h], s[i][j][2 * h + 1]), pk2(f.x, f.y)),
                                              pk2(key_scale[i][h], key_scale[i][h])));
                    s[i][j][2 * h] = x.x;
                    s[i][j][2 * h + 1] = x.y;
                }
        }
        if (far) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float2 f = *reinterpret_cast<const float2*>(&s_far[8 * j + 2 * t]);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[i][j][2 * h] *= f.x;
                        s[i][j][2 * h + 1] *= f.y;
                    }
            }
        }
        if (a.softcap > 0.f) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 x = softcap2(s[i][j][2 * h], s[i][j][2 * h + 1], 1.f, cap_out);
                        s[i][j][2 * h] = x.x;
                        s[i][j][2 * h + 1] = x.y;
                    }
        }
        if (key0 < all_lo || key0 + C::kKeys > all_hi) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = row_of(r), token = attn_token(a, row0 + row);
                const int lo = attn_see_lo(a, w.r, token), hi = row < rows ? attn_see_hi(a, w.r, token) : 0;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = key0 + 16 * i + 8 * h + g;
                        if (key < lo || key >= hi) s[i][r >> 1][2 * h + (r & 1)] = -CUDART_INF_F;
                    }
            }
        }
        // s becomes the differences from the rows' references, which follow a row's maxima only when these are 2^8 ahead, in
        // all warps alike.
        auto take = [&](const float (&x)[R]) {  // off the differences
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint64_t both = pk2(-x[2 * j], -x[2 * j + 1]);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 e = up2(add2(pk2(s[i][j][2 * h], s[i][j][2 * h + 1]), both));
                        s[i][j][2 * h] = e.x;
                        s[i][j][2 * h + 1] = e.y;
                    }
            }
        };
        auto largest = [&](int r, float& mx, float& mz) {  // of the lane's differences of a row, and with the values' exponents
            mx = mz = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float x = s[i][r >> 1][r & 1], y = s[i][r >> 1][2 + (r & 1)];
                mx = fmax3(mx, x, y);
                mz = fmax3(mz, x + value_exp[i][0], y + value_exp[i][1]);
            }
        };
        take(ref);
        bool grow = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx, mz;
            largest(r, mx, mz);
            grow |= mx > kUp + 8.f || mz > ref_u[r] + (kUp + 8.f);
        }
        grow = __syncthreads_or(grow);  // (and every warp is done with the tile before this one)
        load_step(C::kStages - 1);
        if (grow) {
            // The largest of a row in all warps: of the differences, then, from their new reference, with the exponents.
            auto meet = [&](bool exponents, float (&top)[R]) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float mx, mz;
                    largest(r, mx, mz);
                    float x = exponents ? mz : mx;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    if (g == 0) s_max[exponents][warp][row_of(r)] = x;
                }
                __syncthreads();
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    top[r] = s_max[exponents][0][row_of(r)];
#pragma unroll
                    for (int x = 1; x < kWarps; ++x) top[r] = fmaxf(top[r], s_max[exponents][x][row_of(r)]);
                }
            };
            float top[R], by[R];
            meet(false, top);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool first = ref_u[r] == kNone && top[r] > -CUDART_INF_F;  // (scores, not differences yet)
                by[r] = first || top[r] > kUp + 8.f ? top[r] - kUp : 0.f;
                const float down = first ? 1.f : ex2(-by[r]);  // (the first time the sum is 0)
                const float2 l = up2(sums[r >> 1]);
                sums[r >> 1] = r & 1 ? pk2(l.x, l.y * down) : pk2(l.x * down, l.y);
                ref[r] += by[r];
            }
            take(by);
            meet(true, top);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float was = ref_u[r] == kNone ? kNone : ref_u[r] - by[r];
                ref_u[r] = top[r] > was + (kUp + 8.f) ? top[r] - kUp : was;
                const float f = ex2(was - ref_u[r]);
#pragma unroll
                for (int i = 0; i < DM; ++i) {
                    o[i][r >> 1][r & 1] *= f;
                    o[i][r >> 1][2 + (r & 1)] *= f;
                }
            }
        }
        // ---- P^T as halves, rows of P over the tile's keys
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t p[4];  // keys 16 i .. + 7, + 8 .. of rows 8 j .., of rows 8 j + 8 ..
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint64_t less_u = pk2(-ref_u[2 * (j + u)], -ref_u[2 * (j + u) + 1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = s[i][j + u][2 * h], y = s[i][j + u][2 * h + 1];
                        const float2 z = up2(add2(add2(pk2(x, y), pk2(value_exp[i][h], value_exp[i][h])), less_u));
                        sums[j + u] = add2(sums[j + u], pk2(ex2(x), ex2(y)));
                        p[2 * u + h] = pack16<false>(ex2(z.x), ex2(z.y));
                    }
                }
                stsm4_trans(kb + C::p_at(8 * j + (lane & 7) + (lane >> 4) * 8, 2 * (MT * warp + i) + ((lane >> 3) & 1)), p);
            }
        }
        __syncthreads();
        // ---- O^T += V^T P^T, the warp's quarter of the values
#pragma unroll
        for (int kk = 0; kk < kWarps * MT; ++kk) {
            uint32_t p[NT][2];
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                uint32_t b[4];
                ldsm4(b, kb + C::p_at(8 * j + (lane & 7) + (lane >> 4) * 8, 2 * kk + ((lane >> 3) & 1)));
                p[j][0] = b[0];
                p[j][1] = b[1];
                p[j + 1][0] = b[2];
                p[j + 1][1] = b[3];
            }
#pragma unroll
            for (int i = 0; i < DM; i += 2) {
                uint32_t b[4];  // 16 keys of two 16-value groups (heads of 64: one group, the same twice)
                ldsm4_trans(b, vb + C::at(16 * kk + (lane & 15), DM * warp + i + (DM > 1 ? lane >> 4 : 0)));
#pragma unroll
                for (int u = 0; u < 2 && i + u < DM; ++u) {
                    const uint32_t x = b[2 * u] ^ 0x80808080u, y = b[2 * u + 1] ^ 0x80808080u;
                    const uint32_t f[4] = {i8x2_to_half2<kBytes02>(x), i8x2_to_half2<kBytes13>(x), i8x2_to_half2<kBytes02>(y),
                                           i8x2_to_half2<kBytes13>(y)};
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma16<false>(o[i + u][j], f, p[j][0], p[j][1]);
                }
            }
        }

        const bool last_of_item = w.kt + 1 == w.kts;
        if (last_of_item || w.left == 1) {
            // ---- the warps' sums meet
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 both = up2(sums[r >> 1]);
                float l = r & 1 ? both.y : both.x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (g == 0) s_sum[warp][row_of(r)] = l;
            }
            __syncthreads();
            const bool whole = last_of_item && seg_first == 0;
            const int slot = 2 * part + (seg_first == 0 ? kHead : kTail);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = row_of(r);
                if (row >= rows) continue;
                float ll = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) ll += s_sum[x][row];
                const float m = ref_u[r] == kNone ? -CUDART_INF_F : ref[r] + kUp;
                // (averages, and in two steps: see paged_attn_i8.cu)
                const float f = ex2(0.5f * ref_u[r]), inv = ll == 0.f ? 0.f : __fdividef(1.f, ll);
                const long long at = attn_out_row(a, w.r.token0, head, row0 + row);
                const size_t part_at = (size_t)slot * kRows + row;
#pragma unroll
                for (int i = 0; i < DM; ++i) {
                    const int col = 16 * (DM * warp + i) + 2 * g;
                    const float x = o[i][r >> 1][r & 1] * inv * f * f, y = o[i][r >> 1][2 + (r & 1)] * inv * f * f;
                    if (col >= a.D) continue;
                    if (whole)
                        *reinterpret_cast<uint32_t*>(a.out + ((size_t)at * a.D + col) * 2) = pack16<BF16>(x, y);
                    else
                        *reinterpret_cast<float2*>(a.part_o + part_at * a.D + col) = make_float2(x, y);
                }
                if (warp == 0 && g == 0) {
                    if (!whole)
                        a.part_ml[part_at] = make_float2(m, ll);
                    else if (a.lse)
                        a.lse[at] = ll == 0.f ? -CUDART_INF_F : (m + lg2(ll * ProbScale<false>::kInverse)) * kLn2;
                }
            }
            if (!whole && tid == 0) mine->d[seg_first == 0 ? kHead : kTail] = part_desc(s_range, w, row0, rows, head);
            fresh = true;  // (the next segment's first barrier comes before its sums)
        }
        if (++st == C::kStages) st = 0;
        walk_next(a, w, kRows, C::kKeyTile);
    }
    cp_async_wait_group<0>();
    if (err) s_err = err;  // any of the block's errors: all are the same code
    __syncthreads();
    if (tid == 0) mine->err = s_err;
}

template <bool BF16, int DP, int DU = DP>
dspark_status launch_rows(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    using C = RowsI8<DP>;
    int per_sm = 0;
    auto fn = attn_i8_rows_kernel<BF16, DP, DU>;
    if (prepare_kernel((const void*)fn, C::kSmem, C::kThreads, &per_sm) != cudaSuccess || per_sm < 1) return DSPARK_ERR_CUDA;
    int n = sms * (per_sm < C::kBlocksPerSm ? per_sm : C::kBlocksPerSm);
    if (n > kMaxParts) n = kMaxParts;
    *parts = n;
    return launch_overlapped(fn, n, C::kThreads, C::kSmem, s, a) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
template <bool BF16>
dspark_status launch_rows_d(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    if (a.D <= 64) return launch_rows<BF16, 64>(a, sms, s, parts);
    if (a.D <= 128) return launch_rows<BF16, 128>(a, sms, s, parts);
    // (192 values of the room for 256: 64 requests up to 8000 tokens, 16 rows of 192, 147 against 164 us)
    return a.D <= 192 ? launch_rows<BF16, 256, 192>(a, sms, s, parts) : launch_rows<BF16, 256>(a, sms, s, parts);
}

}  // namespace

dspark_status launch_attn_i8_rows(const AttnArgs& a, bool bf16, int sms, cudaStream_t s, int* parts) {
    return bf16 ? launch_rows_d<true>(a, sms, s, parts) : launch_rows_d<false>(a, sms, s, parts);
}

}  // namespace dspark
