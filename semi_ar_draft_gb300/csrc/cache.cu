// cache.cu -- bookkeeping of the paged key-value cache: dspark_cache_plan (block tables, slots and
// positions of a step's new tokens), dspark_cache_commit (lengths after the verification, pages
// given back) and dspark_cache_append (new keys and values written into their pages).
//
// plan and commit are prefix sums over the requests followed by one independent action per new
// token or page.  Each block repeats the prefix sum over all B requests (two 4-byte reads a request,
// from L2) and keeps it in shared memory, so that tokens and pages can be dealt out over any number
// of blocks with no second launch and no grid-wide wait.  Both are bound by the latency of one launch
// with three dependent rounds of memory (lengths, stack or table, result), not by their bytes: 3.6 us for a
// step of 32 requests, 5.8 us for the 200000 tokens of 48 prompts, 6.1 us to take back the pages of 50 finished
// requests of 512.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "host_util.h"
#include "pdl.cuh"

namespace dspark {
namespace {
namespace cg = cooperative_groups;

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxRequests = 8192;  // two 32 KB prefix arrays in shared memory
constexpr int kItemsPerBlock = 2 * kPlanThreads;

// Exclusive prefix sums over the block of two non-negative 64-bit values per thread, and their totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb) {
    __shared__ long long sa[kPlanWarps], sb[kPlanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += x;
            ib += y;
        }
    }
    if (lane == 31) {
        sa[warp] = ia;
        sb[warp] = ib;
    }
    __syncthreads();
    long long pa = 0, pb = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w == warp) {
            pa = ta;
            pb = tb;
        }
        ta += sa[w];
        tb += sb[w];
    }
    a = pa + ia - a;
    b = pb + ib - b;
}

// The request whose range [pre[j], pre[j + 1]) holds x (pre ascending, pre[0] = 0 <= x < pre[B]).
__device__ __forceinline__ int find_range(const int32_t* pre, int B, int x) {
    int lo = 0, hi = B;  // pre[lo] <= x < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t sat32(long long x) { return (int32_t)(x > INT32_MAX ? INT32_MAX : x); }

struct PlanArgs {
    int B, page_shift, num_pages, max_blocks, max_tokens, extra;
    const int32_t* cache_len;
    const int32_t* new_len;  // or null: no tokens but the extra ones
    int32_t* block_table;
    const int32_t* n_blocks;
    const int32_t* free_pages;
    const int32_t* n_free;
    int32_t* seq_len;
    int32_t* offsets;
    int64_t* slots;
    int32_t* positions;  // or null
    int32_t* n_blocks_out;
    int32_t* n_free_out;
    int32_t* status;
    int32_t* error;  // or null
};

// One request's numbers, with every input clamped to what the other inputs allow (bad: it was not).
struct PlanReq {
    long long seq;
    int old, n, have, need;
    bool bad;
};
__device__ __forceinline__ PlanReq plan_request(const PlanArgs& a, int j) {
    PlanReq r;
    const int len = a.cache_len[j], add = a.new_len ? a.new_len[j] : 0, have = a.n_blocks[j];
    const long long n = (long long)add + a.extra;
    r.old = max(len, 0);
    r.n = (int)min(max(n, 0ll), (long long)INT32_MAX);
    r.have = min(max(have, 0), a.max_blocks);
    r.seq = (long long)r.old + r.n;
    const long long blocks = (r.seq + (1ll << a.page_shift) - 1) >> a.page_shift;
    r.need = (int)max(min(blocks, (long long)a.max_blocks) - r.have, 0ll);
    r.bad = len < 0 || n < 0 || have != r.have || blocks > a.max_blocks || r.seq > INT32_MAX;
    return r;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(PlanArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* off = sm;               // [B + 1] first token of each request
    int32_t* page0 = sm + a.B + 1;   // [B + 1] first new page of each request (those the stack holds)
    const int tid = threadIdx.x;
    const int m = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int j0 = min(tid * m, a.B), j1 = min(j0 + m, a.B);
    wait_primary();
    launch_dependents();
    const int n_free_in = *a.n_free;
    const int n_free = min(max(n_free_in, 0), a.num_pages);
    long long tok = 0, pg = 0, T, P;
    bool bad = n_free != n_free_in;
    for (int j = j0; j < j1; ++j) {
        const PlanReq r = plan_request(a, j);
        tok += r.n;
        pg += r.need;
        bad |= r.bad;
    }
    block_scan2(tok, pg, T, P);
    bad |= T > a.max_tokens || P > n_free;
    const int given = (int)min(P, (long long)n_free);
    const bool first = blockIdx.x == 0;
    for (int j = j0; j < j1; ++j) {
        const PlanReq r = plan_request(a, j);
        const int p = (int)min(pg, (long long)given);
        off[j] = sat32(tok);
        page0[j] = p;
        if (first) {
            a.offsets[j] = sat32(tok);
            a.seq_len[j] = sat32(r.seq);
            a.n_blocks_out[j] = r.have + (int)min((long long)r.need, (long long)given - p);
        }
        tok += r.n;
        pg += r.need;
    }
    if (tid == 0) {
        off[a.B] = sat32(T);
        page0[a.B] = given;
    }
    const int any_bad = __syncthreads_or(bad);
    if (first && tid == 0) {
        a.offsets[a.B] = sat32(T);
        *a.n_free_out = n_free - given;
        *a.status = any_bad ? DSPARK_ERR_CACHE : DSPARK_OK;
        if (any_bad && a.error) record_status(a.error, DSPARK_ERR_CACHE);
    }
    const int stride = gridDim.x * kPlanThreads;
    // The new pages' table entries.  A page is known from the stack alone, so the tokens below look
    // it up there too and nothing waits for these writes.
    for (int k = blockIdx.x * kPlanThreads + tid; k < given; k += stride) {
        const int j = find_range(page0, a.B, k);
        const int have = min(max(a.n_blocks[j], 0), a.max_blocks);
        a.block_table[(size_t)j * a.max_blocks + have + (k - page0[j])] = a.free_pages[n_free - 1 - k];
    }
    // Blocks for which the stack had no page: their entries must not go on naming pages of earlier rounds, which
    // are other requests' by now.
    if (P > given)
        for (int j = blockIdx.x * kPlanWarps + (tid >> 5); j < a.B; j += gridDim.x * kPlanWarps) {
            const PlanReq r = plan_request(a, j);
            for (int b = page0[j + 1] - page0[j] + (tid & 31); b < r.need; b += 32)
                a.block_table[(size_t)j * a.max_blocks + r.have + b] = -1;
        }
    const int live = off[a.B];
    for (long long t = blockIdx.x * kPlanThreads + tid; t < a.max_tokens; t += stride) {
        long long slot = -1;
        int pos = -1;
        if (t < live) {
            const int j = find_range(off, a.B, (int)t);
            const long long at = (long long)max(a.cache_len[j], 0) + (t - off[j]);
            pos = sat32(at);
            const int have = min(max(a.n_blocks[j], 0), a.max_blocks);
            const long long blk = at >> a.page_shift;
            int page = -1;
            if (blk < have)
                page = a.block_table[(size_t)j * a.max_blocks + blk];
            else if (blk - have < page0[j + 1] - page0[j])
                page = a.free_pages[n_free - 1 - (page0[j] + (int)(blk - have))];
            if (page >= 0 && page < a.num_pages)
                slot = ((long long)page << a.page_shift) | (at & ((1 << a.page_shift) - 1));
        }
        a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
    }
}

struct CommitArgs {
    int B, page_shift, num_pages, max_blocks, extra;
    const int32_t* cache_len;
    const int32_t* add_len;  // or null
    const uint8_t* done;     // or null
    const int32_t* block_table;
    const int32_t* n_blocks;
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* cache_len_out;
    int32_t* n_blocks_out;
    int32_t* n_free_out;
    int32_t* status;
    int32_t* error;    // or null
    int32_t* settled;  // or null; may be cache_len, n_blocks and n_free
};

struct CommitReq {
    int len, have, keep;
    bool bad;
};
__device__ __forceinline__ CommitReq commit_request(const CommitArgs& a, int j) {
    CommitReq r;
    const int have = a.n_blocks[j];
    long long len = (long long)a.cache_len[j] + (a.add_len ? a.add_len[j] : 0) + a.extra;
    r.have = min(max(have, 0), a.max_blocks);
    r.bad = have != r.have;
    if (a.done && a.done[j]) len = 0;
    const long long most = (long long)r.have << a.page_shift;
    r.bad |= len < 0 || len > most;
    len = min(max(len, 0ll), min(most, (long long)INT32_MAX));
    r.len = (int)len;
    r.keep = (int)((len + (1ll << a.page_shift) - 1) >> a.page_shift);
    return r;
}

// The entries of the blocks past each request's length, requests and blocks in order, form one list, of which
// every warp of the cluster takes a run; entries that name a page go to the stack.  A request whose first pages were
// given back before (a sliding window) has entries that name none, so where a page goes depends on all entries
// before it: the warps count theirs, the blocks of the cluster (eight at most) send each other their counts, and
// each warp writes its own, from registers where its run is kHeldSteps steps at most (32768 entries over eight blocks).
// Measured: 32 requests, few pages: 3.5 us, one block and no cluster; 512 requests of up to 500 pages, a tenth of them
// finished: 6.1 us, of which the exchange takes 1.
constexpr int kCommitBlocks = 8;
constexpr int kHeldSteps = 8;
template <bool ALONE>  // one block, without a cluster
__global__ void __launch_bounds__(kPlanThreads) cache_commit_kernel(CommitArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* entry0 = sm;           // [B + 1] first entry of each request
    int32_t* keep = sm + a.B + 1;   // [B] blocks kept
    __shared__ int s_count[kPlanWarps];
    __shared__ int2 s_blocks[kCommitBlocks];  // of each block: pages that its entries name; whether anything is wrong
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int j0 = min(tid * m, a.B), j1 = min(j0 + m, a.B);
    cg::cluster_group cluster = cg::this_cluster();
    if (!ALONE) cluster.barrier_arrive();  // (a block is written to only once it runs)
    wait_primary();
    launch_dependents();
    const int n_free_in = *a.n_free;
    const int n_free = min(max(n_free_in, 0), a.num_pages);
    long long at = 0, none = 0, E, unused;
    bool bad = n_free != n_free_in;
    for (int j = j0; j < j1; ++j) {
        const CommitReq r = commit_request(a, j);
        at += r.have - r.keep;
        bad |= r.bad;
    }
    block_scan2(at, none, E, unused);
    bad |= E > INT32_MAX;
    const int entries = sat32(E);
    const bool first = blockIdx.x == 0;
    for (int j = j0; j < j1; ++j) {
        const CommitReq r = commit_request(a, j);
        entry0[j] = sat32(at);
        keep[j] = r.keep;
        if (first) {
            a.cache_len_out[j] = r.len;
            a.n_blocks_out[j] = r.keep;
        }
        at += r.have - r.keep;
    }
    if (tid == 0) entry0[a.B] = entries;
    __syncthreads();

    const long long warps = (long long)gridDim.x * kPlanWarps;
    const long long run = ((entries + warps - 1) / warps + 31) & ~31ll;
    const long long begin = (blockIdx.x * kPlanWarps + warp) * run, end = min(begin + run, (long long)entries);
    int page[kHeldSteps];
    auto load = [&](long long from) {
#pragma unroll
        for (int u = 0; u < kHeldSteps; ++u) {
            const long long k = from + 32 * u + lane;
            page[u] = -1;
            if (k >= end) continue;
            const int j = find_range(entry0, a.B, (int)k);
            page[u] = a.block_table[(size_t)j * a.max_blocks + keep[j] + ((int)k - entry0[j])];
        }
    };
    int count = 0;
#pragma unroll 1
    for (long long from = begin; from < end; from += 32 * kHeldSteps) {
        load(from);
#pragma unroll
        for (int u = 0; u < kHeldSteps; ++u) {
            bad |= page[u] >= a.num_pages;
            count += __popc(__ballot_sync(0xffffffffu, page[u] >= 0 && page[u] < a.num_pages));
        }
    }
    if (lane == 0) s_count[warp] = count;
    bool any_bad = __syncthreads_or(bad) != 0;
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w == warp) before = total;
        total += s_count[w];
    }
    if (!ALONE) {
        cluster.barrier_wait();
        if (tid < (int)gridDim.x) *cluster.map_shared_rank(&s_blocks[blockIdx.x], tid) = make_int2(total, any_bad);
        cluster.sync();
        total = 0;
        for (int r = 0; r < (int)gridDim.x; ++r) {
            if (r < (int)blockIdx.x) before += s_blocks[r].x;
            total += s_blocks[r].x;
            any_bad |= s_blocks[r].y != 0;
        }
    }
    const int room = a.num_pages - n_free;
    any_bad |= total > room;
    // Every block has read its inputs: settled may lie over them.
    if (first && a.settled) {
        for (int j = j0; j < j1; ++j) {
            a.settled[j] = a.cache_len_out[j];  // (written by this thread)
            a.settled[a.B + j] = keep[j];
        }
        if (tid == 0) a.settled[2 * a.B] = n_free + min(total, room);
    }
    if (first && tid == 0) {
        *a.n_free_out = n_free + min(total, room);
        *a.status = any_bad ? DSPARK_ERR_CACHE : DSPARK_OK;
        if (any_bad && a.error) record_status(a.error, DSPARK_ERR_CACHE);
    }
#pragma unroll 1
    for (long long from = begin; from < end; from += 32 * kHeldSteps) {
        if (run > 32 * kHeldSteps) load(from);
#pragma unroll
        for (int u = 0; u < kHeldSteps; ++u) {
            const bool real = page[u] >= 0 && page[u] < a.num_pages;
            const uint32_t lanes = __ballot_sync(0xffffffffu, real);
            const int i = before + __popc(lanes & ((1u << lane) - 1));
            if (real && i < room) a.free_pages[n_free + i] = page[u];
            before += __popc(lanes);
        }
    }
}

// ---------------------------------------------------------------- append
struct AppendArgs {
    int T, chunks, page_shift;  // chunks: 8-element groups of one head's row
    uint32_t per_token;         // Hk * chunks
    long long slots_end;        // num_pages * page_size
    const uint16_t* k;
    const uint16_t* v;
    long long k_token, k_head, v_token, v_head;  // strides, elements
    unsigned char* k_pages;
    unsigned char* v_pages;
    long long page, token, head;  // strides of the pools, elements
    const int64_t* slots;
    const float* k_scale;
    const float* v_scale;
};

constexpr int kAppendThreads = 256;

template <bool ALIGNED>
__device__ __forceinline__ uint4 load_row8(const uint16_t* p) {
    if constexpr (ALIGNED) {
        return *reinterpret_cast<const uint4*>(p);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if (BF16) return make_float2(bf16_lo(w), bf16_hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Eight values divided by the head's scale in fp32 (IEEE division) and rounded to e4m3, to nearest even,
// finite values clamped to +-448.  The product with the reciprocal r is within two units of the last place
// of the quotient, so it rounds to the same e4m3 value unless a border between two of them is as near: for
// |q| >= 2^-6 a border is where the 20 bits below e4m3's three are 0x80000.  Groups of eight with a value within
// eight units of one, or below 2^-6, are divided after all.  (A prompt of 16384 tokens, 8 heads of 128: 24 us
// with every value divided, 21 so.)
template <bool BF16>
__device__ __forceinline__ uint2 quantize8(uint4 x, float scale, float r, bool divide) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8], q[8];
    uint32_t border = 0xffffffffu;
    float least = CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack16<BF16>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = f[i] * r;
        border = min(border, (__float_as_uint(q[i]) << 12) + 0x80008000u);
        least = fminf(least, fabsf(q[i]));
    }
    if (border <= 0x10000u || least < 0x1p-6f || divide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(f[i], scale);
    }
    uint32_t y[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        y[i >> 1] |= b << (16 * (i & 1));
    }
    return make_uint2(y[0], y[1]);
}

// One thread moves a few 8-element groups of K and the same ones of V, all loads first: two of 16-bit
// pages (21 us for a prompt of 16384 tokens against 24 with one), one of e4m3 pages, where the arithmetic
// wants the warps.  Bound by HBM for prompts, by the launch for a decoding step.
__host__ __device__ constexpr int append_items(bool cache8) { return cache8 ? 1 : 2; }
template <bool CACHE8, bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendArgs a) {
    constexpr int kAppendItems = append_items(CACHE8);
    wait_primary();
    launch_dependents();
    const long long total = (long long)a.T * a.per_token;
    const long long stride = (long long)gridDim.x * kAppendThreads * kAppendItems;
    for (long long i0 = (long long)blockIdx.x * kAppendThreads * kAppendItems + threadIdx.x; i0 < total; i0 += stride) {
        uint4 kx[kAppendItems], vx[kAppendItems];
        long long at[kAppendItems];
        int head[kAppendItems];
#pragma unroll
        for (int u = 0; u < kAppendItems; ++u) {
            const long long i = i0 + u * kAppendThreads;
            at[u] = -1;
            if (i >= total) continue;
            const long long t = total <= UINT32_MAX ? (long long)((uint32_t)i / a.per_token) : i / a.per_token;
            const uint32_t rest = (uint32_t)(i - t * a.per_token);
            const int h = (int)(rest / (uint32_t)a.chunks), c = (int)(rest - (uint32_t)h * (uint32_t)a.chunks);
            const long long slot = a.slots[t];
            kx[u] = load_row8<ALIGNED>(a.k + t * a.k_token + h * a.k_head + 8 * c);
            vx[u] = load_row8<ALIGNED>(a.v + t * a.v_token + h * a.v_head + 8 * c);
            head[u] = h;
            if (slot >= 0 && slot < a.slots_end)
                at[u] = (slot >> a.page_shift) * a.page + (slot & ((1 << a.page_shift) - 1)) * a.token + h * a.head + 8 * c;
        }
#pragma unroll
        for (int u = 0; u < kAppendItems; ++u) {
            if (at[u] < 0) continue;
            if (CACHE8) {
                const float ks = a.k_scale ? a.k_scale[head[u]] : 1.f, vs = a.v_scale ? a.v_scale[head[u]] : 1.f;
                // (reciprocals that would be subnormal or infinite: divide)
                const bool kd = !(fabsf(ks) > 0x1p-120f && fabsf(ks) < 0x1p120f);
                const bool vd = !(fabsf(vs) > 0x1p-120f && fabsf(vs) < 0x1p120f);
                *reinterpret_cast<uint2*>(a.k_pages + at[u]) = quantize8<BF16>(kx[u], ks, __frcp_rn(ks), kd);
                *reinterpret_cast<uint2*>(a.v_pages + at[u]) = quantize8<BF16>(vx[u], vs, __frcp_rn(vs), vd);
            } else {
                *reinterpret_cast<uint4*>(a.k_pages + 2 * at[u]) = kx[u];
                *reinterpret_cast<uint4*>(a.v_pages + 2 * at[u]) = vx[u];
            }
        }
    }
}

template <bool CACHE8, bool BF16>
cudaError_t launch_append(const AppendArgs& a, bool aligned, int blocks, cudaStream_t s) {
    return launch_overlapped(aligned ? cache_append_kernel<CACHE8, BF16, true> : cache_append_kernel<CACHE8, BF16, false>,
                             blocks, kAppendThreads, 0, s, a);
}

struct Span {
    const void* at;
    size_t bytes;
};
// Whether something that is written lies over anything else (reads may share).
template <int W, int R>
bool clash(const Span (&written)[W], const Span (&read)[R]) {
    auto over = [](const Span& a, const Span& b) {
        const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
        return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
    };
    for (int i = 0; i < W; ++i) {
        for (const Span& r : read)
            if (over(written[i], r)) return true;
        for (int o = 0; o < i; ++o)
            if (over(written[i], written[o])) return true;
    }
    return false;
}

dspark_status check_cache_params(const dspark_cache_params* p) {
    if (!p || p->B < 1 || p->num_pages < 1 || p->max_blocks < 1 || page_shift_of(p->page_size) < 0 ||
        (((uintptr_t)p->error | (uintptr_t)p->settled) & 3u))
        return DSPARK_ERR_INVALID_ARG;
    if (p->B > kMaxRequests) return DSPARK_ERR_UNSUPPORTED;
    return DSPARK_OK;
}

int blocks_for(long long items, int sms) {
    const long long b = (items + kItemsPerBlock - 1) / kItemsPerBlock;
    return (int)(b < 1 ? 1 : (b > sms ? sms : b));
}

}  // namespace

int page_shift_of(int page_size) {
    if (page_size < 1 || page_size > 4096 || (page_size & (page_size - 1))) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_cache_workspace_size(const dspark_cache_params* p) {
    return check_cache_params(p) == DSPARK_OK ? kHeaderBytes : 0;
}

extern "C" dspark_status dspark_cache_plan(const dspark_cache_params* p, const int32_t* cache_len,
                                           const int32_t* new_len, int32_t* block_table, const int32_t* n_blocks,
                                           const int32_t* free_pages, const int32_t* n_free, int32_t* seq_len,
                                           int32_t* offsets, int64_t* slots, int32_t* positions, int32_t* n_blocks_out,
                                           int32_t* n_free_out, void* workspace, size_t ws_bytes,
                                           dspark_stream_t stream) {
    dspark_status st = check_cache_params(p);
    if (st != DSPARK_OK) return st;
    if (p->max_tokens < 0 || p->extra < 0) return DSPARK_ERR_INVALID_ARG;
    if (!cache_len || !block_table || !n_blocks || !free_pages || !n_free || !seq_len || !offsets ||
        (!slots && p->max_tokens) || !n_blocks_out || !n_free_out)
        return DSPARK_ERR_INVALID_ARG;
    // Every block reads all of the inputs while the first one writes the outputs.
    const size_t nb = sizeof(int32_t) * (size_t)p->B, nt = (size_t)p->max_tokens;
    const Span ins[] = {{cache_len, nb}, {new_len, nb}, {n_blocks, nb}, {n_free, sizeof(int32_t)},
                        {free_pages, sizeof(int32_t) * (size_t)p->num_pages}};
    const Span outs[] = {{seq_len, nb}, {offsets, nb + sizeof(int32_t)}, {n_blocks_out, nb}, {n_free_out, sizeof(int32_t)},
                         {slots, sizeof(int64_t) * nt}, {positions, sizeof(int32_t) * nt}, {block_table, nb * (size_t)p->max_blocks}};
    if (clash(outs, ins)) return DSPARK_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < kHeaderBytes) return DSPARK_ERR_WORKSPACE;
    int sms = 0, per_sm = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    const size_t smem = sizeof(int32_t) * 2 * ((size_t)p->B + 1);
    if (prepare_kernel((const void*)cache_plan_kernel, smem, kPlanThreads, &per_sm) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    PlanArgs a{p->B, page_shift_of(p->page_size), p->num_pages, p->max_blocks, p->max_tokens, p->extra, cache_len,
               new_len, block_table, n_blocks, free_pages, n_free, seq_len, offsets, slots, positions, n_blocks_out,
               n_free_out, &static_cast<WsHeader*>(workspace)->status, p->error};
    if (launch_overlapped(cache_plan_kernel, blocks_for(p->max_tokens, sms), kPlanThreads, smem,
                          reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_commit(const dspark_cache_params* p, const int32_t* cache_len,
                                             const int32_t* add_len, const uint8_t* done, const int32_t* block_table,
                                             const int32_t* n_blocks, int32_t* free_pages, const int32_t* n_free,
                                             int32_t* cache_len_out, int32_t* n_blocks_out, int32_t* n_free_out,
                                             void* workspace, size_t ws_bytes, dspark_stream_t stream) {
    dspark_status st = check_cache_params(p);
    if (st != DSPARK_OK) return st;
    if (p->extra < 0) return DSPARK_ERR_INVALID_ARG;
    if (!cache_len || !block_table || !n_blocks || !free_pages || !n_free || !cache_len_out || !n_blocks_out ||
        !n_free_out)
        return DSPARK_ERR_INVALID_ARG;
    const size_t nb = sizeof(int32_t) * (size_t)p->B;
    const Span ins[] = {{cache_len, nb}, {add_len, nb}, {n_blocks, nb}, {n_free, sizeof(int32_t)}, {done, (size_t)p->B},
                        {block_table, nb * (size_t)p->max_blocks}};
    const Span outs[] = {{cache_len_out, nb}, {n_blocks_out, nb}, {n_free_out, sizeof(int32_t)},
                         {free_pages, sizeof(int32_t) * (size_t)p->num_pages}};
    const Span settled[] = {{p->settled, 2 * nb + sizeof(int32_t)}}, kept[] = {ins[1], ins[4], ins[5], outs[0], outs[1], outs[2], outs[3]};
    if (clash(outs, ins) || clash(settled, kept)) return DSPARK_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < kHeaderBytes) return DSPARK_ERR_WORKSPACE;
    int sms = 0, per_sm = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    const size_t smem = sizeof(int32_t) * 2 * ((size_t)p->B + 1);
    // The pages that come back are known on the device only: a block for every 64 requests, up to eight, spreads
    // those of finished requests, and one block does for the usual few.
    const int want = (p->B + 63) / 64, blocks = want < kCommitBlocks ? want : kCommitBlocks;
    const auto kernel = blocks == 1 ? cache_commit_kernel<true> : cache_commit_kernel<false>;
    if (prepare_kernel((const void*)kernel, smem, kPlanThreads, &per_sm) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    CommitArgs a{p->B, page_shift_of(p->page_size), p->num_pages, p->max_blocks, p->extra, cache_len, add_len, done,
                 block_table, n_blocks, free_pages, n_free, cache_len_out, n_blocks_out, n_free_out,
                 &static_cast<WsHeader*>(workspace)->status, p->error, p->settled};
    if (launch_overlapped_clusters(kernel, blocks, blocks, kPlanThreads, smem,
                                   reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_append(const dspark_append_params* p, const void* k, const void* v, void* k_pages,
                                             void* v_pages, const int64_t* slots, const float* k_scale,
                                             const float* v_scale, dspark_stream_t stream) {
    if (!p || p->T < 0 || p->Hk < 1 || p->D < 1 || p->num_pages < 1 || page_shift_of(p->page_size) < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (p->dtype != DSPARK_BF16 && p->dtype != DSPARK_F16) return DSPARK_ERR_INVALID_ARG;
    const bool e4m3 = p->kv_dtype == DSPARK_E4M3;
    if (!e4m3 && p->kv_dtype != p->dtype) return DSPARK_ERR_INVALID_ARG;
    if (!k_pages || !v_pages || (p->T && (!k || !v || !slots))) return DSPARK_ERR_INVALID_ARG;
    if (p->D % 16 || p->D > 4096 || (long long)p->Hk * p->D > (1 << 22)) return DSPARK_ERR_UNSUPPORTED;
    const size_t esz = e4m3 ? 1 : 2;
    if ((((uintptr_t)k_pages | (uintptr_t)v_pages) & 15u) || (p->kv_page_stride * esz) % 16 ||
        (p->kv_token_stride * esz) % 16 || (p->kv_head_stride * esz) % 16)
        return DSPARK_ERR_INVALID_ARG;
    if (p->T == 0) return DSPARK_OK;
    int sms = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    AppendArgs a;
    a.T = p->T;
    a.chunks = p->D / 8;
    a.page_shift = page_shift_of(p->page_size);
    a.per_token = (uint32_t)p->Hk * (uint32_t)a.chunks;
    a.slots_end = (long long)p->num_pages * p->page_size;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_token = p->k_token_stride;
    a.k_head = p->k_head_stride;
    a.v_token = p->v_token_stride;
    a.v_head = p->v_head_stride;
    a.k_pages = static_cast<unsigned char*>(k_pages);
    a.v_pages = static_cast<unsigned char*>(v_pages);
    a.page = p->kv_page_stride;
    a.token = p->kv_token_stride;
    a.head = p->kv_head_stride;
    a.slots = slots;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    const bool aligned = !((((uintptr_t)k | (uintptr_t)v) & 15u) || (a.k_token | a.k_head | a.v_token | a.v_head) % 8);
    const long long total = (long long)a.T * a.per_token;
    const long long per_block = kAppendThreads * append_items(e4m3);
    const long long want = (total + per_block - 1) / per_block, most = (long long)sms * 16;
    const int blocks = (int)(want < most ? want : most);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = p->dtype == DSPARK_BF16;
    // (without e4m3 a copy of the bits, whichever 16-bit type)
    const cudaError_t e = !e4m3  ? launch_append<false, true>(a, aligned, blocks, s)
                          : bf16 ? launch_append<true, true>(a, aligned, blocks, s)
                                 : launch_append<true, false>(a, aligned, blocks, s);
    if (e != cudaSuccess) return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}
