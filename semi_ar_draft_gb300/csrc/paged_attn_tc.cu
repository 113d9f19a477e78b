// paged_attn_tc.cu -- dspark_paged_attention on the fifth-generation tensor cores: row tiles of 128 for
// requests whose new tokens give more than 16 rows a kv head, 48 with an 8-bit cache (the flattened verify, draft
// blocks).
//
// One persistent CTA a multiprocessor walks its range of units (paged.cuh).  Roles:
//   loaders (4 warps)    copy the item's queries and, tile by tile, KT keys and values into a ring in
//                        shared memory, 16 bytes a thread and copy, in the 128-byte-swizzled layout the MMA
//                        reads; several tiles in flight, across items; tiles of an 8-bit cache arrive as they are
//                        and are widened into the ring by the lanes that copied them
//   MMA (1 warp a stream) S = Q K^T into tensor memory, and O += P V with P from tensor memory
//   softmax (4 warps a   thread = row: takes S, writes P (16 bits) back to tensor memory, keeps the row's
//     stream)            maximum and sum; at an item's end joins the streams and writes the output
// A unit's key tiles go to kStreams streams in turn, each with its own S, P, O and statistics (heads up to
// 128): while one stream's softmax runs, the tensor cores have the other's products.  With heads of
// 256 the output alone takes half of tensor memory, and one stream with tiles of 32 keys is used.
//
// Values are the second product's B operand as they lie in the cache (one row a key, so N-major).
// An output starts at zero, so every product accumulates; it is scaled when a row's maximum has grown by
// 2^8, which needs the stream's earlier products done.
//
// Bound by the cache's bytes where a unit's softmax (about 2000 cycles for a stream's tile of 64 keys) is
// shorter than its loads: 512 requests of up to 4096 tokens, 8 query heads of 128 a kv head, 5 new tokens on
// average: 417 us = 6.0 TB/s (0.88 of the measured copy rate).  With heads of 64 a tile is half the bytes and the
// softmax decides: 32 draft blocks of 16 over up to 4100 tokens 52.5 us = 2.8 TB/s (0.42).
// Over an 8-bit cache the loaders' widening decides at few rows (32 requests, 35 rows on average: 85 us, of row
// tiles of 16: 69) and pays at many (145 requests, 119 rows of 192 over 200 keys: 92 us against 254).
#include "host_util.h"
#include "paged.cuh"
#include "pdl.cuh"
#include "tc05.cuh"

namespace dspark {
namespace {

constexpr int kTcRowTile = 128;

template <bool F8, int DP>
struct TcAttn {
    static constexpr int kStreams = DP == 256 ? 1 : 2;
    static constexpr int kKt = DP == 256 ? 32 : 64;  // keys of a tile
    static constexpr int kUnit = kStreams * kKt;
    static constexpr int kExtra = DP == 128 ? 2 : 4;  // what an item costs beside its key tiles
    static constexpr int kSoftmaxWarps = 4 * kStreams;
    // Four loader warps, two a stream: a warp that copied a part of every tile spent more time between tiles
    // (waits, page numbers, the walk) than on its copies.
    static constexpr int kLoaders = 4;
    static constexpr int kTileLoaders = kLoaders / kStreams;
    // Warps after the softmax's: multiprocessor quarter (warp % 4) 0 has none of them and quarter 1 the MMA
    // warps, one a stream; the loaders are in quarters 2 and 3.  Short row tiles keep quarter 0 busiest.
    static constexpr int kWarps = kSoftmaxWarps + 8;
    static __device__ __forceinline__ int loader_of(int warp) {  // 0 .. 3, or -1
        const int h = warp - kSoftmaxWarps;
        return h >= 0 && (h & 2) ? (h >> 2) * 2 + (h & 1) : -1;
    }
    static __device__ __forceinline__ int mma_of(int warp) {  // the stream, or -1
        const int h = warp - kSoftmaxWarps;
        return h == 1 ? 0 : (h == 5 && kStreams == 2 ? 1 : -1);
    }
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSub = DP / 64;                  // 64-value groups of a row
    static constexpr int kTile = kKt * DP * 2;            // bytes of a tile's K (or V)
    static constexpr int kQ = kTcRowTile * DP * 2;
    static constexpr int kQBufs = DP == 64 ? 2 : 1;
    static constexpr int kSlots = F8 ? (DP == 64 ? 6 : (DP == 128 ? 4 : 3)) : (DP == 64 ? 10 : (DP == 128 ? 6 : 4));
    // 8-bit caches: raw tiles a loader keeps on their way, 16 bytes a lane and copy, K and V of its rows
    static constexpr int kRawSlots = F8 ? (DP == 128 ? 2 : 4) : 0;
    static constexpr int kRawTile = 2 * (kKt / kTileLoaders) * DP;  // bytes of a loader's part of one
    static_assert(kSlots % kStreams == 0, "a slot belongs to one stream, whose loaders wait for no other's turn");
    static constexpr int kRing = kQBufs * kQ;
    static constexpr int kRaw = kRing + kSlots * 2 * kTile;
    static constexpr int kMeta = kRaw + kLoaders * kRawSlots * kRawTile;
    static constexpr size_t kSmem = (size_t)kMeta + 2 * kTcRowTile * 8 + 512;
    // tensor memory columns
    static constexpr int kColS = kStreams * DP, kColP = kColS + kStreams * kKt;
    static_assert(kColP + kStreams * kKt <= 512, "tensor memory");  // (two buffers of P a stream)
    static_assert(kSmem <= kMaxSmem, "shared memory");
};

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(v)::"memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {  // (as tmem_wait_ld: tied to the registers)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
// Descriptor of an N-major (values as they lie: N adjacent, one 128-byte row a K index) operand with the
// 128-byte swizzle: the leading offset goes from one group of 64 N to the next, the stride offset from
// eight K rows to the next eight.
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t saddr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lead >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// kind::f16 with fp32 accumulation, A and B of one 16-bit type; bit 16: B is N-major.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool b_mn) {
    return (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
template <bool BF16>
__device__ __forceinline__ bool is_odd16(uint32_t half) {  // NaN or inf in the low 16 bits
    const uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
    return (half & e) == e;
}
template <bool BF16>
__device__ __forceinline__ float from16(uint32_t half) {
    return BF16 ? bf16_bits_to_f32(half & 0xffffu) : __half2float(__ushort_as_half((unsigned short)half));
}

// Sixteen e4m3 values as bf16 or fp16 values (both hold them exactly), in order.
template <bool BF16>
__device__ __forceinline__ void widen16(const uint4 v, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        const uint32_t pair = i & 1 ? w[i >> 1] >> 16 : w[i >> 1];
        asm("{ .reg .b16 x; cvt.u16.u32 x, %1; cvt.rn.f16x2.e4m3x2 %0, x; }" : "=r"(h) : "r"(pair));
        if (BF16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            r[i] = pack16<true>(f.x, f.y);
        } else {
            r[i] = h;
        }
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// MMAs and commits by one elected lane of a converged warp (always the same one).  Descriptors come in
// halves; kind::f16, fp32 accumulation; accumulate = 0 overwrites D.
__device__ __forceinline__ void mma_elect_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 x, y;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n"
        " setp.ne.b32 p, %6, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_elect_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 y;\n mov.b64 y, {%2, %3};\n"
        " setp.ne.b32 p, %5, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(bar))
        : "memory");
}

// One arrival on `bar` (counted in its expected arrivals) once this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

struct TcBars {
    uint64_t full[10], empty[10], qfull[2], qempty[2], sfull[2], sfree[2], pfull[2], pvdone[2], smeet[2], drain[2], meet;
    uint32_t tmem;
    int abort, status, misaligned;
    int odd[2][2];
    AttnScratch scratch;
};
static_assert(sizeof(TcBars) <= 512, "barriers");

template <bool BF16, bool F8, int DP>
__global__ void __launch_bounds__(TcAttn<F8, DP>::kThreads, 1) attn_tc_kernel(AttnArgs a, uint64_t limit_ns) {
    using C = TcAttn<F8, DP>;
    constexpr bool VB = BF16 && !F8;  // type of P and V: an 8-bit cache's values meet the probabilities as halves
    constexpr int KT = C::kKt, NS = C::kStreams;
    extern __shared__ __align__(1024) unsigned char smem[];
    float2* s_ml = reinterpret_cast<float2*>(smem + C::kMeta);  // [kStreams][128]
    TcBars* bars = reinterpret_cast<TcBars*>(smem + C::kMeta + 2 * kTcRowTile * 8);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x, parts = gridDim.x;
    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&bars->full[i], 32 * C::kTileLoaders);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->qempty[i], NS);
            mbar_init(&bars->qfull[i], 32 * C::kLoaders);
            mbar_init(&bars->sfull[i], 1);
            mbar_init(&bars->sfree[i], 4);
            mbar_init(&bars->pfull[i], 4);
            mbar_init(&bars->pvdone[i], 1);
            mbar_init(&bars->smeet[i], 4);
            bars->odd[i][0] = bars->odd[i][1] = 0;
        }
        mbar_init(&bars->meet, C::kSoftmaxWarps);
        mbar_init(&bars->drain[0], 1);
        mbar_init(&bars->drain[1], 1);
        bars->abort = 0;
        // the swizzled tiles need 1024-byte alignment; where it is not given nothing is computed
        bars->misaligned = (smem_addr(smem) & 1023u) != 0;
        bars->status = bars->misaligned ? DSPARK_ERR_UNSUPPORTED : 0;
        mbar_init_fence();
    }
    constexpr int kAllocWarp = C::kSoftmaxWarps + 1;
    if (warp == kAllocWarp) {
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    wait_primary();
    launch_dependents();
    bool bad;
    AttnStart start = attn_start<C::kThreads>(a, kTcRowTile, C::kUnit, C::kExtra, parts, part, 2 + C::kExtra, &bars->scratch, &bad);  // (barriers inside)
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    if (bars->misaligned) start.end = start.begin;
    volatile int* abort = &bars->abort;
    int32_t* status = &bars->status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_hint_or_abort(bar, parity, abort, status, limit_ns); };
    // by a whole warp, with one answer for all lanes
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    attn_tail_rows(a, (size_t)part * C::kThreads + tid, (size_t)parts * C::kThreads);
    PartItem* mine = a.items + part;  // written by thread 0
    if (tid == 0) mine->d[kTail].first = mine->d[kHead].first = -1;

    if (C::loader_of(warp) >= 0) {
        // ---------------------------------------------------------------- loaders
        constexpr int kChunks = DP / (F8 ? 16 : 8);  // 16-byte groups of a row in the cache
        constexpr int kPer = 32 / kChunks;           // rows a warp copies at a time
        const int lw = C::loader_of(warp);
        const int chunk = lane % kChunks, sub_row = lane / kChunks;
        const bool inside = chunk * (F8 ? 16 : 8) < a.D;
        const uint32_t base = smem_addr(smem);
        const uint32_t mask = (1u << a.page_shift) - 1;
        const uint32_t page16 = (uint32_t)(a.page >> 4), token16 = (uint32_t)(a.token >> 4);
        const unsigned char* k_at = a.k_pages + chunk * 16;
        const long long v_after_k = a.v_pages - a.k_pages;
        AttnWalk w = walk_begin(a, start, kTcRowTile, C::kUnit, C::kExtra);
        int err = 0, seg = 0;
        // This warp's keys of its stream's tiles.
        constexpr int kKeys = KT / C::kTileLoaders;
        const int first_key = (lw / C::kTileLoaders) * KT + (lw % C::kTileLoaders) * kKeys;
        auto tile_key = [&]() { return (w.kt_first + w.kt) * C::kUnit + first_key; };
        // Page of this lane's key of the next tile, asked for a tile ahead.  The load is unconditional (entry 0
        // where there is no key) and looked at when the copies are issued, so that nothing waits for it here.
        int pid;
        auto fetch_pages = [&]() {
            const int key = min(tile_key() + lane, w.r.seq - 1);
            const size_t at = w.done() || key < 0 ? 0 : (size_t)w.j * a.max_blocks + (key >> a.page_shift);
            pid = __ldg(a.block_table + at);
        };
        fetch_pages();
        bool fresh = true;
        int head = 0, slot = lw / C::kTileLoaders, round = 0;
        const int tile_row = (lw % C::kTileLoaders) * kKeys + sub_row;
        // 8-bit caches: a tile arrives as it is, each lane's pieces in places of its own, `ahead` tiles at a time; the
        // lane that copied a piece widens it into the slot, keys to q's type, values to halves (both exact).
        constexpr int kSteps = kKeys / kPer;
        int raw_slot = 0, raw_old = 0, ahead = 0;
        unsigned char* raw = smem + C::kRaw + lw * (C::kRawSlots * C::kRawTile) + lane * 16;
        auto widen = [&]() {
            if (round > 0 && !warp_wait(&bars->empty[slot], (uint32_t)((round - 1) & 1))) return false;
            unsigned char* to = smem + C::kRing + slot * (2 * C::kTile) + ((2 * chunk) >> 3) * (KT * 128);
            const unsigned char* from = raw + raw_old * C::kRawTile;
#pragma unroll 2
            for (int u = 0; u < kSteps; ++u) {
                const uint32_t at0 = sw128_offset(tile_row + u * kPer, (2 * chunk) & 7);
                const uint32_t at1 = sw128_offset(tile_row + u * kPer, (2 * chunk + 1) & 7);
                const uint4 k = *reinterpret_cast<const uint4*>(from + 2 * u * 512);
                const uint4 v = *reinterpret_cast<const uint4*>(from + (2 * u + 1) * 512);
                uint4 x, y;
                widen16<BF16>(k, x, y);
                *reinterpret_cast<uint4*>(to + at0) = x;
                *reinterpret_cast<uint4*>(to + at1) = y;
                widen16<false>(v, x, y);
                *reinterpret_cast<uint4*>(to + at0 + C::kTile) = x;
                *reinterpret_cast<uint4*>(to + at1 + C::kTile) = y;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive_local(&bars->full[slot]);
            slot += NS;
            if (slot >= C::kSlots) {
                slot -= C::kSlots;
                ++round;
            }
            if (++raw_old == C::kRawSlots) raw_old = 0;
            return true;
        };
        // An item's queries: with two streams after its first keys, since their buffer is free later than a
        // slot (421 against 426 us for the 512-request verify); with heads of 256, where they are as large as two
        // tiles, before (122 against 131 us for three long contexts, with a softcap 8 us cheaper than now).
        constexpr bool kQueriesFirst = NS == 1;
        auto queries = [&]() {
            const int qb = seg % C::kQBufs, use = seg / C::kQBufs;
            if (F8 && use > 0 && !__all_sync(0xffffffffu, mbar_try_wait(&bars->qempty[qb], (uint32_t)((use - 1) & 1)))) {
                // the products that still read it may be waiting for raw tiles
                asm volatile("cp.async.wait_all;" ::: "memory");
                while (ahead > 0 && widen()) --ahead;
            }
            if (use > 0 && !warp_wait(&bars->qempty[qb], (uint32_t)((use - 1) & 1))) return false;
            ++seg;
            const int row0 = (w.item - head * w.rts) * kTcRowTile;
            const int rows = min(w.r.n * a.G - row0, kTcRowTile);
            constexpr int kQPer = 256 / DP;  // rows a warp copies at a time
            const int qc = lane % (DP / 8);
            const uint32_t qbase = base + (uint32_t)qb * C::kQ + (uint32_t)(qc >> 3) * (kTcRowTile * 128);
            for (int r = lw * kQPer + lane / (DP / 8); r < ((rows + 31) & ~31); r += C::kLoaders * kQPer) {
                const bool real = qc * 8 < a.D && r < rows;
                const int row = row0 + r;
                const int token = attn_token(a, row);
                const long long src = real ? (w.r.token0 + token) * a.q_token +
                                                 (head * a.G + row - token * a.G) * a.q_head + qc * 8
                                           : 0;
                copy16(qbase + sw128_offset(r, qc & 7), a.q + 2 * src, real);
            }
            copy_arrive(&bars->qfull[qb]);
            return true;
        };
        while (!w.done()) {
            if (fresh) {
                head = w.item / w.rts;
                if (kQueriesFirst && !queries()) break;
            }
            if (!F8 && round > 0 && !warp_wait(&bars->empty[slot], (uint32_t)((round - 1) & 1))) break;
            const int key0 = tile_key();
            const unsigned char* head_at = k_at + head * a.head;
            const bool none = key0 + lane >= w.r.seq || key0 + lane < w.r.lo;
            if ((uint32_t)pid >= (uint32_t)a.num_pages) {
                if (!none && lane < kKeys) err = DSPARK_ERR_CACHE;
                pid = -1;
            }
            if (none) pid = -1;
            const uint32_t kb = base + C::kRing + (uint32_t)slot * (2 * C::kTile) + (uint32_t)(chunk >> 3) * (KT * 128);
            const uint32_t rb = smem_addr(raw) + (uint32_t)(raw_slot * C::kRawTile);
#pragma unroll 8
            for (int i = 0; i < kKeys; i += kPer) {
                const int p = __shfl_sync(0xffffffffu, pid, i + sub_row);
                const bool real = inside && p >= 0;
                const uint64_t at16 = (uint64_t)(uint32_t)max(p, 0) * page16 +
                                      (uint64_t)((uint32_t)(key0 + i + sub_row) & mask) * token16;
                const unsigned char* src = real ? head_at + 16 * at16 : a.k_pages;
                const uint32_t dst = F8 ? rb + (uint32_t)(i / kPer) * 1024u : kb + sw128_offset(tile_row + i, chunk & 7);
                copy16(dst, src, real);
                copy16(dst + (F8 ? 512 : C::kTile), src + v_after_k, real);
            }
            if constexpr (F8) {
                cp_async_commit();
                if (++raw_slot == C::kRawSlots) raw_slot = 0;
                if (++ahead == C::kRawSlots) {  // the oldest has landed once the others alone are in flight
                    cp_async_wait_group<C::kRawSlots - 1>();
                    --ahead;
                    if (!widen()) break;
                }
            } else {
                // The slot is full once its loaders' copies so far have landed; nobody waits for that here, so
                // the whole ring can be in flight.
                copy_arrive(&bars->full[slot]);
                slot += NS;
                if (slot >= C::kSlots) {
                    slot -= C::kSlots;
                    ++round;
                }
            }
            if (fresh && !kQueriesFirst && !queries()) break;
            fresh = w.kt + 1 == w.kts;
            walk_next(a, w, kTcRowTile, C::kUnit);
            fetch_pages();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (F8)
            while (ahead > 0 && widen()) --ahead;
        if (err) bars->status = err;
    } else if (C::mma_of(warp) >= 0) {
        // ---------------------------------------------------------------- MMA issue
        // The whole warp runs this with equal values and one elected lane issues: descriptors then stay in
        // uniform registers (from one divergent lane each MMA cost 90 to 160 cycles to issue).
        constexpr uint32_t idesc_s = idesc16<BF16>(kTcRowTile, KT, false);
        constexpr uint32_t idesc_o = idesc16<VB>(kTcRowTile, DP, true);
        const uint32_t base = smem_addr(smem);
        // The upper halves of the descriptors hold layout and stride only (and the leading offset, V's, sits in
        // the lower half's upper bits; with one group of 64 values it is not used).
        const uint64_t k_desc = umma_desc_sw128(base, 1024);
        const uint64_t v_desc = umma_desc_sw128_mn(base, C::kSub > 1 ? KT * 128 : 1024, 1024);
        const uint32_t k_hi = (uint32_t)(k_desc >> 32), k_lo = (uint32_t)k_desc & 0xffff0000u;
        const uint32_t v_hi = (uint32_t)(v_desc >> 32), v_lo = (uint32_t)v_desc & 0xffff0000u;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        AttnWalk w = walk_begin(a, start, kTcRowTile, C::kUnit, C::kExtra);
        const int s = C::mma_of(warp);
        int seg = 0, slot = s, turn = 0, held = 0;  // turn: parity of the ring's round; held: the slot whose values
        bool ok = true, behind = false;             // are still to come, if behind
        auto values = [&](int n) {  // O_s += P_s V of the stream's n-th tile
            if (!warp_wait(&bars->pfull[s], (uint32_t)(n & 1))) return false;
            tc_fence_after();
            const uint32_t vd = v_lo + ((base + C::kRing + (uint32_t)held * (2 * C::kTile) + C::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < KT / 16; ++k)
                mma_elect_ts(tm + s * DP, tm + C::kColP + (2 * s + (n & 1)) * (KT / 2) + 8 * k, vd + k * (2048 >> 4), v_hi, idesc_o,
                             1u);
            commit_elect(&bars->empty[held]);
            commit_elect(&bars->pvdone[s]);
            return true;
        };
        for (int unit = 0; ok && __shfl_sync(0xffffffffu, !w.done(), 0); ++unit) {
            const int qb = seg % C::kQBufs;
            if ((!behind && !warp_wait(&bars->qfull[qb], (uint32_t)((seg / C::kQBufs) & 1))) ||  // an item's first tile
                !warp_wait(&bars->full[slot], (uint32_t)turn) ||
                (unit > 0 && !warp_wait(&bars->sfree[s], (uint32_t)((unit - 1) & 1))))
                break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the loaders' copies, to the MMA
            tc_fence_after();
            const uint32_t qd = k_lo + ((base + (uint32_t)qb * C::kQ) >> 4);
            const uint32_t kd = k_lo + ((base + C::kRing + (uint32_t)slot * (2 * C::kTile)) >> 4);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                mma_elect_ss(tm + C::kColS + s * KT, qd + (k >> 2) * (kTcRowTile * 128 >> 4) + 2 * (k & 3), k_hi,
                             kd + (k >> 2) * (KT * 128 >> 4) + 2 * (k & 3), k_hi, idesc_s, k > 0 ? 1u : 0u);
            commit_elect(&bars->sfull[s]);
            if (behind && !values(unit - 1)) break;
            held = slot;
            slot += NS;
            if (slot >= C::kSlots) {
                slot -= C::kSlots;
                turn ^= 1;
            }
            // An item's last values do not wait for the next item's keys.
            const bool end = __shfl_sync(0xffffffffu, w.kt + 1 == w.kts || w.left == 1, 0);
            if (end) {
                commit_elect(&bars->qempty[qb]);
                ++seg;
                ok = values(unit);
            }
            behind = !end;
            walk_next(a, w, kTcRowTile, C::kUnit);
        }
        commit_elect(&bars->drain[s]);  // everything issued has completed before tensor memory is freed
        mbar_wait_bounded(&bars->drain[s], 0, status, limit_ns);
        __syncwarp();
    } else if (warp < C::kSoftmaxWarps) {
        // ---------------------------------------------------------------- softmax
        const int s = warp >> 2, row = tid & 127, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t ts = tmem + lanes + C::kColS + s * KT;
        float c = a.scale * kLog2e;  // (times the head's key scale)
        bool plain = a.softcap == 0.f && c > 0.f;
        float cap_in = a.softcap > 0.f ? 2.f * c / a.softcap : 0.f;
        const float cap_out = a.softcap * kLog2e;
        uint32_t zero[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) zero[i] = 0u;
        if (s == 0)
#pragma unroll 1
            for (int i = 0; i < NS * DP; i += 16) tmem_st16(tmem + lanes + i, zero);
        tmem_wait_st();
        tc_fence_before();
        uint32_t meets = 0, smeets = 0;
        auto meet = [&]() {  // all softmax warps
            __syncwarp();
            if (lane == 0) mbar_arrive_local(&bars->meet);
            return warp_wait(&bars->meet, meets++ & 1);
        };
        auto stream_meet = [&]() {  // the stream's
            __syncwarp();
            if (lane == 0) mbar_arrive_local(&bars->smeet[s]);
            return warp_wait(&bars->smeet[s], smeets++ & 1);
        };
        AttnWalk w = walk_begin(a, start, kTcRowTile, C::kUnit, C::kExtra);
        float m = -CUDART_INF_F, l = 0.f;
        int n = 0, seg_first = 0, row0 = 0, rows = 0, head = 0, see_lo = 0, see_hi = 0, all_lo = 0, all_hi = 0;
        bool fresh = true, ok = meet();
        while (ok && !w.done()) {
            if (fresh) {
                fresh = false;
                seg_first = w.kt;
                head = w.item / w.rts;
                row0 = (w.item % w.rts) * kTcRowTile;
                rows = min(w.r.n * a.G - row0, kTcRowTile);
                all_lo = attn_see_lo(a, w.r, attn_token(a, row0 + rows - 1));
                all_hi = attn_see_hi(a, w.r, attn_token(a, row0));
                const int token = attn_token(a, row0 + row);
                see_lo = row < rows ? attn_see_lo(a, w.r, token) : 0;
                see_hi = row < rows ? attn_see_hi(a, w.r, token) : 0;
                m = -CUDART_INF_F;
                l = 0.f;
                if (F8 && a.k_scale) {
                    c = a.scale * kLog2e * __ldg(a.k_scale + head);
                    plain = a.softcap == 0.f && c > 0.f;
                    cap_in = a.softcap > 0.f ? 2.f * c / a.softcap : 0.f;
                }
            }
            const int key0 = (w.kt_first + w.kt) * C::kUnit + s * KT;
            const bool edge = key0 < all_lo || key0 + KT > all_hi;  // some row does not see all of the tile
            const bool live = 32 * quarter < rows;
            if (!warp_wait(&bars->sfull[s], (uint32_t)(n & 1))) break;
            tc_fence_after();
            // P has two buffers: the MMA warp issues S of this tile after the values of the last but one, so the
            // buffer they read is free once S is here.
            const uint32_t tp = tmem + lanes + C::kColP + (2 * s + (n & 1)) * (KT / 2);
            // The output stands still once the stream's earlier products are done: awaited before it is touched,
            // and in any case before this tile's P is announced, so that no phase of the barrier is skipped.
            bool stands = n == 0;
            auto still = [&]() {
                if (stands) return true;
                stands = warp_wait(&bars->pvdone[s], (uint32_t)((n - 1) & 1));
                tc_fence_after();
                return stands;
            };
            if (live) {
                // What is not a plain scaled score is prepared in tensor memory first, 32 columns at a time in a
                // rolled loop: unrolled beside the common path its code cost more in instruction fetches.
                if (!plain || edge) {
#pragma unroll 1
                    for (int h = 0; h < KT; h += 32) {
                        uint32_t x[32];
                        tmem_ld32(ts + h, x);
                        tmem_wait_ld(x);
                        if (a.softcap > 0.f) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 y = softcap2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), cap_in, cap_out);
                                x[i] = __float_as_uint(y.x);
                                x[i + 1] = __float_as_uint(y.y);
                            }
                        } else if (!plain) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * c);
                        }
                        if (edge) {
                            const int from = see_lo - key0 - h;
                            const uint32_t count = (uint32_t)max(see_hi - see_lo, 0);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if ((uint32_t)(i - from) >= count) x[i] = 0xff800000u;  // -inf
                        }
                        tmem_st32(ts + h, x);
                    }
                    tmem_wait_st();
                }
                const float f = plain ? c : 1.f;  // (f > 0)
                uint32_t x[KT / 32][32];
#pragma unroll
                for (int h = 0; h < KT / 32; ++h) tmem_ld32(ts + 32 * h, x[h]);
#pragma unroll
                for (int h = 0; h < KT / 32; ++h) tmem_wait_ld(x[h]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_local(&bars->sfree[s]);
                float t4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) t4[i] = fmaxf(__uint_as_float(x[0][i]), __uint_as_float(x[0][4 + i]));
#pragma unroll
                for (int i = 8; i < KT; i += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        t4[q] = fmax3(t4[q], __uint_as_float(x[i >> 5][(i & 31) + q]), __uint_as_float(x[i >> 5][(i & 31) + 4 + q]));
                const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * f;
                float grow = 1.f;
                if (top > m + 8.f) {
                    if (m != -CUDART_INF_F) grow = ex2(m - top);  // (else sum and output are still zero)
                    m = top;
                    l *= grow;
                }
                if (__any_sync(0xffffffffu, grow != 1.f)) {
                    if (!still()) break;
#pragma unroll 1
                    for (int i = 0; i < DP; i += 16) {
                        uint32_t o[16];
                        tmem_ld16(tmem + lanes + s * DP + i, o);
                        tmem_wait_ld16(o);
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * grow);
                        tmem_st16(tmem + lanes + s * DP + i, o);
                    }
                }
                const float ref = m == -CUDART_INF_F ? 0.f : m - ProbScale<VB>::kBits;
                const uint64_t f2 = pk2(f, f), r2 = pk2(-ref, -ref);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < KT; h += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 e = up2(fma2(pk2(__uint_as_float(x[h >> 5][i]), __uint_as_float(x[h >> 5][i + 1])), f2, r2));
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], pk2(p0, p1));
                        p[i / 2] = pack16<VB>(p0, p1);
                    }
                    tmem_st16(tp + h / 2, p);
                }
                const float2 total = up2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                l += total.x + total.y;
                tmem_wait_st();
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive_local(&bars->sfree[s]);
            }
            // A hidden key's value must not reach a row that does not see it, even as 0 x inf: values of an
            // edge tile that are not finite (never, in a healthy cache) are added by hand to the rows that
            // see them, and taken out of the tile.
            if (edge) {
                const int tile = n * NS + s, slot = tile % C::kSlots;
                if (!warp_wait(&bars->full[slot], (uint32_t)((tile / C::kSlots) & 1))) break;
                unsigned char* v = smem + C::kRing + slot * (2 * C::kTile) + C::kTile;
                uint32_t acc = 0;
                for (int i = row; i < C::kTile / 16; i += 128) {
                    const uint4 y = reinterpret_cast<const uint4*>(v)[i];
                    odd_note<false, VB>(y.x, acc);
                    odd_note<false, VB>(y.y, acc);
                    odd_note<false, VB>(y.z, acc);
                    odd_note<false, VB>(y.w, acc);
                }
                int* odd = &bars->odd[s][n & 1];  // (cleared before the tile after next can set it)
                if (odd_found<false, VB>(acc)) *odd = 1;
                if (!stream_meet()) break;
                const bool found = *reinterpret_cast<volatile int*>(odd) != 0;
                if (found) {
                    if (!still()) break;
#pragma unroll 1
                    for (int k = 0; k < KT; ++k) {
                        uint32_t pk = 0;
                        if (live) tmem_ld1(tp + (k >> 1), pk);
                        const float pv = from16<VB>((k & 1) ? pk >> 16 : pk);
                        const bool see = key0 + k >= see_lo && key0 + k < see_hi;
#pragma unroll 1
                        for (int d = 0; d < DP; ++d) {
                            const uint32_t bits = *reinterpret_cast<const uint16_t*>(
                                v + (d >> 6) * (KT * 128) + sw128_offset(k, (d & 63) >> 3) + 2 * (d & 7));
                            if (live && is_odd16<VB>(bits)) {
                                uint32_t o;
                                tmem_ld1(tmem + lanes + s * DP + d, o);
                                if (see) o = __float_as_uint(fmaf(pv, from16<VB>(bits), __uint_as_float(o)));
                                tmem_st1(tmem + lanes + s * DP + d, o);
                                tmem_wait_st();
                            }
                        }
                    }
                    if (!stream_meet()) break;
                    for (int i = row; i < C::kTile / 2; i += 128) {
                        uint16_t* y = reinterpret_cast<uint16_t*>(v) + i;
                        if (is_odd16<VB>(*y)) *y = 0;
                    }
                    if (row == 0) *odd = 0;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
            }
            if (!still()) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_local(&bars->pfull[s]);

            const bool last_of_item = w.kt + 1 == w.kts;
            if (last_of_item || w.left == 1) {
                // ---- the streams' parts of the segment meet: WG s takes the s-th half of the columns
                if (!warp_wait(&bars->pvdone[s], (uint32_t)(n & 1))) break;
                tc_fence_after();
                s_ml[s * kTcRowTile + row] = make_float2(m, l);
                tc_fence_before();
                if (!meet()) break;  // (every stream has seen its own products done)
                tc_fence_after();
                float f[NS], mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
                for (int q = 0; q < NS; ++q) mm = fmaxf(mm, s_ml[q * kTcRowTile + row].x);
                const float ref = mm == -CUDART_INF_F ? 0.f : mm;
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const float2 ml = s_ml[q * kTcRowTile + row];
                    f[q] = ml.y == 0.f ? 0.f : ex2(ml.x - ref);
                    ll = fmaf(ml.y, f[q], ll);
                }
                const bool whole = last_of_item && seg_first == 0;
                const size_t slot = 2 * (size_t)part + (seg_first == 0 ? kHead : kTail);
                const float inv = !whole ? 1.f : (ll == 0.f ? 0.f : (F8 && a.v_scale ? __ldg(a.v_scale + head) : 1.f) / ll);
                const long long at = attn_out_row(a, w.r.token0, head, row0 + row);
                unsigned char* dst = a.out + (size_t)at * a.D * 2;
                float* part_dst = a.part_o + (slot * kTcRowTile + row) * a.D;
#pragma unroll 1
                for (int i = s * (DP / NS); i < (s + 1) * (DP / NS); i += 16) {
                    if (live) {
                        uint32_t o[NS][16];
#pragma unroll
                        for (int q = 0; q < NS; ++q) tmem_ld16(tmem + lanes + q * DP + i, o[q]);
#pragma unroll
                        for (int q = 0; q < NS; ++q) tmem_wait_ld16(o[q]);
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            v[e] = __uint_as_float(o[0][e]) * f[0];
                            if (NS == 2) v[e] = fmaf(__uint_as_float(o[NS - 1][e]), f[NS - 1], v[e]);
                        }
                        if (row < rows && i < a.D) {
                            if (whole) {
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = pack16<BF16>(v[2 * e] * inv, v[2 * e + 1] * inv);
                                uint4* to = reinterpret_cast<uint4*>(dst + 2 * i);
                                to[0] = make_uint4(y[0], y[1], y[2], y[3]);
                                to[1] = make_uint4(y[4], y[5], y[6], y[7]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<float4*>(part_dst + i + e) =
                                        make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                            }
                        }
                    }  // (rows of nobody have gathered whatever lay in P)
#pragma unroll
                    for (int q = 0; q < NS; ++q) tmem_st16(tmem + lanes + q * DP + i, zero);
                }
                tmem_wait_st();
                if (s == 0 && row < rows) {
                    if (!whole)
                        a.part_ml[slot * kTcRowTile + row] = make_float2(mm, ll);
                    else if (a.lse)
                        a.lse[at] = ll == 0.f ? -CUDART_INF_F : (mm + lg2(ll * ProbScale<VB>::kInverse)) * kLn2;
                }
                if (!whole && tid == 0) mine->d[seg_first == 0 ? kHead : kTail] = part_desc(start, w, row0, rows, head);
                tc_fence_before();
                if (!meet()) break;  // the outputs are zero again, and the statistics have been read
                tc_fence_after();
                fresh = true;
            }
            ++n;
            walk_next(a, w, kTcRowTile, C::kUnit);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAllocWarp) tmem_dealloc(tmem, 512);
    if (tid == 0) mine->err = bars->status ? bars->status : (bad ? DSPARK_ERR_CACHE : 0);
}

template <bool BF16, bool F8, int DP>
dspark_status launch_tc(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    using C = TcAttn<F8, DP>;
    int per_sm = 0;
    auto fn = attn_tc_kernel<BF16, F8, DP>;
    if (prepare_kernel((const void*)fn, C::kSmem, C::kThreads, &per_sm) != cudaSuccess || per_sm < 1)
        return DSPARK_ERR_CUDA;
    const int n = sms < kMaxTcParts ? sms : kMaxTcParts;
    *parts = n;
    return launch_overlapped(fn, n, C::kThreads, C::kSmem, s, a, wait_limit_ns()) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

template <bool BF16, bool F8>
dspark_status launch_tc_d(const AttnArgs& a, int sms, cudaStream_t s, int* parts) {
    if (a.D <= 64) return launch_tc<BF16, F8, 64>(a, sms, s, parts);
    if (a.D <= 128) return launch_tc<BF16, F8, 128>(a, sms, s, parts);
    return launch_tc<BF16, F8, 256>(a, sms, s, parts);
}

}  // namespace

dspark_status launch_attn_tc(const AttnArgs& a, bool bf16, bool e4m3, int sms, cudaStream_t s, int* parts) {
    if (e4m3) return bf16 ? launch_tc_d<true, true>(a, sms, s, parts) : launch_tc_d<false, true>(a, sms, s, parts);
    return bf16 ? launch_tc_d<true, false>(a, sms, s, parts) : launch_tc_d<false, false>(a, sms, s, parts);
}

}  // namespace dspark
