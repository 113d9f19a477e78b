// cache_i8.cu -- dspark_cache_append_i8 (keys and values quantised to int8 as they are written into their pages,
// with a scale for each block of tokens and kv head) and dspark_cache_read_i8 (the way back).  block_scale.cuh has
// the number format.
//
//   append   e = the smallest exponent with max |x| <= 127 2^e over the block's tokens of the call, no smaller than the
//            block's own unless its first token is among them; code = x 2^-e to nearest even; where e grew by n, the
//            block's other codes are rounded once more, code 2^-n.
//
// A power of two: the product with 2^-e is exact, so a code is one rounding of the value whoever computes it; a scale
// that grows again and again costs an old code at most 1/2 + 1/4 + ... < 1 step of the last one (a scale free to grow by
// any factor could cost a half step each time); and what is read back is a number of the 16-bit type.  The price is a
// step up to twice as wide as max / 127.
#include "block_scale.cuh"
#include "host_util.h"
#include "pdl.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct I8Args {
    int T, Hk, D, page_shift, block_shift;
    int chunks;          // D / 8
    uint32_t chunk_mul;  // i / chunks = i chunk_mul >> 16 for i < 32 chunks
    int window_shift;    // entries of slots a warp looks after
    long long slots_end, items;
    const uint16_t* x[2];             // keys, values: [T, Hk, D]
    long long x_token[2], x_head[2];  // strides, elements
    signed char* pages[2];
    long long page, token, head;  // strides of the pools
    unsigned char* exps[2];
    long long e_page, e_block, e_head;
    const int64_t* slots;
    int32_t* error;
};

template <bool ALIGNED>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
    if constexpr (ALIGNED) {
        return __ldg(reinterpret_cast<const uint4*>(p));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(p + 2 * i) | ((uint32_t)__ldg(p + 2 * i + 1) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (BF16) return make_float2(bf16_lo(w), bf16_hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ float mag_to_float(uint32_t bits) {  // of a 16-bit magnitude
    return BF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
}
__device__ __forceinline__ uint32_t mag_max(uint32_t acc, const uint4& x) {
    acc = __vmaxu2(acc, x.x & 0x7fff7fffu);
    acc = __vmaxu2(acc, x.y & 0x7fff7fffu);
    acc = __vmaxu2(acc, x.z & 0x7fff7fffu);
    return __vmaxu2(acc, x.w & 0x7fff7fffu);
}
// The largest magnitude below `inf` of either half of each word.
__device__ __forceinline__ uint32_t finite_max(uint32_t acc, const uint4& x, uint32_t inf) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (lo < inf) acc = max(acc, lo);
        if (hi < inf) acc = max(acc, hi);
    }
    return acc;
}

// Eight values times inv = 2^-e, rounded to whole numbers: 1.5 2^23 added, the low byte is the code.  CLAMP: where the
// scale could not grow to the largest value, or something is not finite (NaN becomes 0).
template <bool BF16, bool CLAMP>
__device__ __forceinline__ uint2 quantize8(const uint4& x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v = unpack2<BF16>(w[i]);
        if (CLAMP) {
            v.x = v.x != v.x ? 0.f : fminf(fmaxf(v.x * inv, -127.f), 127.f);
            v.y = v.y != v.y ? 0.f : fminf(fmaxf(v.y * inv, -127.f), 127.f);
        }
        r[2 * i] = __float_as_uint(fmaf(v.x, CLAMP ? 1.f : inv, 12582912.f));
        r[2 * i + 1] = __float_as_uint(fmaf(v.y, CLAMP ? 1.f : inv, 12582912.f));
    }
    auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    };
    return make_uint2(four(r[0], r[1], r[2], r[3]), four(r[4], r[5], r[6], r[7]));
}

// Four codes times 2^-n, n >= 1, to nearest even.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, int n) {
    if (n > 8) return 0;
    uint32_t y = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = (int)(signed char)(w >> (8 * i));
        const int q = (c + (1 << (n - 1)) - 1 + ((c >> n) & 1)) >> n;
        y |= (uint32_t)(q & 0xff) << (8 * i);
    }
    return y;
}

// The tokens of one block among the 32 entries of slots from `base` on: n of them, in order, in `list` (entry - base, and
// the place in the block << 8; bit 31 where a later one of these entries has the same place).  A run of a block's tokens
// ends where another block's begins.
struct Members {
    int n, last;        // last: entry - base of the last one
    uint32_t place[4];  // places in the block
    bool more;          // the run may go on behind these entries
};
__device__ __forceinline__ Members members(const I8Args& a, long long block, long long base, int before, uint32_t* list) {
    const int lane = threadIdx.x & 31;
    const long long slot = base + lane < a.T ? __ldg(a.slots + base + lane) : -1;
    const bool valid = slot >= 0 && slot < a.slots_end;
    const uint32_t vm = __ballot_sync(0xffffffffu, valid);
    uint32_t mm = __ballot_sync(0xffffffffu, valid && (slot >> a.block_shift) == block);
    const uint32_t other = vm & ~mm;
    if (other) mm &= (other & (0u - other)) - 1u;
    if (mm && __ffs(mm) - 1 > before) mm = 0;  // 32 skipped entries or more: another run
    const bool in = (mm >> lane) & 1u;
    const int place = (int)(slot & ((1 << a.block_shift) - 1));
    const uint32_t same = __match_any_sync(0xffffffffu, in ? place : -1 - lane);
    Members r;
    r.n = __popc(mm);
    r.last = 31 - __clz(mm);
    r.more = !other && mm && base + 32 < a.T;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.place[i] = i == 0 || a.block_shift > 5 ? __reduce_or_sync(0xffffffffu, in && (place >> 5) == i ? 1u << (place & 31) : 0u) : 0u;
    __syncwarp();
    if (in)
        list[__popc(mm & ((1u << lane) - 1u))] = (uint32_t)lane | (uint32_t)place << 8 | (31 - __clz(same) != lane ? 0x80000000u : 0u);
    __syncwarp();
    return r;
}

// A warp takes keys or values of one kv head of a run: the tokens of a block that follow one another in slots.  It is
// the warp whose window of slots holds the run's first entry.  The values are read once where the run fits the
// registers (4 KB: 16 tokens of 128), and a second time, from L2, where it does not.
constexpr int kHold = 8;
template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) cache_append_i8_kernel(I8Args a) {
    __shared__ uint32_t s_list[kWarps][32];
    const int lane = threadIdx.x & 31;
    uint32_t* list = s_list[threadIdx.x >> 5];
    wait_primary();
    launch_dependents();
    const uint32_t per_window = 2u * (uint32_t)a.Hk;
    for (long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); item < a.items; item += (long long)gridDim.x * kWarps) {
        const long long window = item / per_window;
        const int rest = (int)(item - window * per_window), kv = rest & 1, head = rest >> 1;
        const long long t0 = window << a.window_shift;
        // The window's entries that begin a run: no token of the same block stands before them, but for fewer than 32
        // skipped entries.
        auto block_at = [&](long long t) -> long long {
            if (t < 0 || t >= a.T) return -1;
            const long long slot = __ldg(a.slots + t);
            return slot >= 0 && slot < a.slots_end ? slot >> a.block_shift : -1;
        };
        const long long bp = block_at(t0 - 32 + lane), bc = block_at(t0 + lane);
        const uint32_t pm = __ballot_sync(0xffffffffu, bp >= 0), below = __ballot_sync(0xffffffffu, bc >= 0) & ((1u << lane) - 1u);
        const int far = pm ? 31 - __clz(pm) : -1;
        const long long near_block = __shfl_sync(0xffffffffu, bc, below ? 31 - __clz(below) : 0);
        const long long far_block = __shfl_sync(0xffffffffu, bp, max(far, 0));
        const long long prev = below ? near_block : (far >= lane ? far_block : -1);
        uint32_t first = __ballot_sync(0xffffffffu, bc >= 0 && bc != prev && lane < (1 << a.window_shift));
#pragma unroll 1
        for (; first; first &= first - 1) {
            const int at = __ffs(first) - 1;
            const long long block = __shfl_sync(0xffffffffu, bc, at);
            const uint16_t* x = a.x[kv] + head * a.x_head[kv];
            auto vec = [&](long long base, int i) {  // of the listed tokens' i-th eight values
                const int m = (int)((uint32_t)i * a.chunk_mul >> 16);
                return load8<ALIGNED>(x + (base + (list[m] & 31u)) * a.x_token[kv] + 8 * (i - m * a.chunks));
            };
            // ---- the largest magnitude
            long long base = t0 + at;
            Members r = members(a, block, base, 32, list);
            const int n0 = r.n * a.chunks;
            const bool held = !r.more && n0 <= 32 * kHold;
            uint4 h[kHold];
            uint32_t acc = 0, place[4] = {r.place[0], r.place[1], r.place[2], r.place[3]};
#pragma unroll
            for (int u = 0; u < kHold; ++u)
                h[u] = lane + 32 * u < n0 ? vec(base, lane + 32 * u) : make_uint4(0, 0, 0, 0);
            unsigned char* exp_at;
            signed char* row0;  // the block's first token
            {
                const long long slot = block << a.block_shift, page = slot >> a.page_shift;
                const int i = (int)(slot & ((1 << a.page_shift) - 1));
                exp_at = a.exps[kv] + page * a.e_page + (i >> a.block_shift) * a.e_block + head * a.e_head;
                row0 = a.pages[kv] + page * a.page + i * a.token + head * a.head;
            }
            const uint32_t old_byte = *exp_at;
#pragma unroll
            for (int u = 0; u < kHold; ++u) acc = mag_max(acc, h[u]);
            auto rest_of = [&](auto&& f) {  // every listed value past the held ones, chunk of entries by chunk
                for (int i = lane + 32 * kHold; i < n0; i += 32) f(vec(base, i));
                for (Members y = r; y.more;) {
                    base += 32;
                    y = members(a, block, base, y.last, list);
#pragma unroll
                    for (int j = 0; j < 4; ++j) place[j] |= y.place[j];
                    for (int i = lane; i < y.n * a.chunks; i += 32) f(vec(base, i));
                }
                if (r.more) {
                    base = t0 + at;
                    members(a, block, base, 32, list);
                }
            };
            if (!held) rest_of([&](const uint4& v) { acc = mag_max(acc, v); });
            constexpr uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
            uint32_t top = __reduce_max_sync(0xffffffffu, max(acc & 0xffffu, acc >> 16));
            const bool odd = top >= inf;
            if (odd) {  // of the finite ones
                acc = 0;
#pragma unroll
                for (int u = 0; u < kHold; ++u) acc = finite_max(acc, h[u], inf);
                if (!held) rest_of([&](const uint4& v) { acc = finite_max(acc, v, inf); });
                top = __reduce_max_sync(0xffffffffu, acc);
                if (lane == 0 && a.error) record_status(a.error, DSPARK_ERR_NOT_FINITE);
            }
            // ---- the scale.  127 / 64 is 1.984375: a mantissa up to that stays in its binade's steps, a larger one
            // carries into the exponent.
            const int wanted = (int)((__float_as_uint(mag_to_float<BF16>(top)) + 0x1ffffu) >> 23) - 127 - 6;
            int e = min(max(wanted, ExpRange<BF16>::kLo), ExpRange<BF16>::kHi);
            const int old = exponent_of<BF16>(old_byte);
            const bool begun = place[0] & 1u;
            if (!begun) e = max(e, old);
            if (!begun && e > old) {  // the block's other tokens
                const int per = a.D / 16;
                for (int i = lane; i < per << a.block_shift; i += 32) {
                    const int p = i / per;
                    uint32_t word = place[0];  // (by selects: an indexed register array would go to local memory)
                    if (p >= 32) word = p >= 96 ? place[3] : (p >= 64 ? place[2] : place[1]);
                    if ((word >> (p & 31)) & 1u) continue;
                    uint4* y = reinterpret_cast<uint4*>(row0 + p * a.token + 16 * (i - p * per));
                    uint4 v = *y;
                    v.x = shrink4(v.x, e - old);
                    v.y = shrink4(v.y, e - old);
                    v.z = shrink4(v.z, e - old);
                    v.w = shrink4(v.w, e - old);
                    *y = v;
                }
            }
            __syncwarp();  // (every lane has read the old exponent)
            if (lane == 0) *exp_at = (unsigned char)(e + 127);
            // ---- the codes
            const float inv = two_to(-e);
            const bool clamp = odd || wanted > ExpRange<BF16>::kHi;
            auto put = [&](int i, const uint4& v) {
                const int m = (int)((uint32_t)i * a.chunk_mul >> 16);
                const uint32_t it = list[m];
                const uint2 y = clamp ? quantize8<BF16, true>(v, inv) : quantize8<BF16, false>(v, inv);
                if (!(it >> 31)) *reinterpret_cast<uint2*>(row0 + (long long)((it >> 8) & 127u) * a.token + 8 * (i - m * a.chunks)) = y;
            };
#pragma unroll
            for (int u = 0; u < kHold; ++u)
                if (lane + 32 * u < n0) put(lane + 32 * u, h[u]);
            if (!held) {
                for (int i = lane + 32 * kHold; i < n0; i += 32) put(i, vec(base, i));
                for (Members y = r; y.more;) {
                    base += 32;
                    y = members(a, block, base, y.last, list);  // (a warp's barrier: later tokens of a slot land later)
                    for (int i = lane; i < y.n * a.chunks; i += 32) put(i, vec(base, i));
                }
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- read back
struct ReadArgs {
    int page_shift;
    uint32_t per_token, chunks;  // 16-value groups of a token, of a head's row
    long long total, slots_end;
    const signed char* pages[2];
    long long page, token, head;
    BlockExp exp;
    const int64_t* slots;
    uint4* out[2];
};

template <bool BF16>
__device__ __forceinline__ void widen16(const uint4& w, float s, uint4* out) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
        widen4(x[i], f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (BF16)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[2 * i + j]) : "f"(f[2 * j + 1] * s), "f"(f[2 * j] * s));
            else
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y[2 * i + j]) : "f"(f[2 * j + 1] * s), "f"(f[2 * j] * s));
        }
    }
    out[0] = make_uint4(y[0], y[1], y[2], y[3]);
    out[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

// One thread widens 16 adjacent codes of K and the same ones of V.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) cache_read_i8_kernel(ReadArgs a) {
    wait_primary();
    launch_dependents();
    const long long stride = (long long)gridDim.x * kThreads;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < a.total; i += stride) {
        const long long t = a.total <= UINT32_MAX ? (long long)((uint32_t)i / a.per_token) : i / a.per_token;
        const uint32_t rest = (uint32_t)(i - t * a.per_token), h = rest / a.chunks, c = rest - h * a.chunks;
        const long long slot = __ldg(a.slots + t);
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        uint32_t ke = 0, ve = 0;
        if (slot >= 0 && slot < a.slots_end) {
            const long long page = slot >> a.page_shift;
            const int at = (int)(slot & ((1 << a.page_shift) - 1));
            const long long from = page * a.page + at * a.token + h * a.head + 16 * c;
            const long long e = page * a.exp.page + (at >> a.exp.shift) * a.exp.block + h * a.exp.head;
            k = __ldg(reinterpret_cast<const uint4*>(a.pages[0] + from));
            v = __ldg(reinterpret_cast<const uint4*>(a.pages[1] + from));
            ke = __ldg(a.exp.k + e);
            ve = __ldg(a.exp.v + e);
        }
        widen16<BF16>(k, two_to(exponent_of<BF16>(ke)), a.out[0] + 2 * i);
        widen16<BF16>(v, two_to(exponent_of<BF16>(ve)), a.out[1] + 2 * i);
    }
}

dspark_status check_i8(const dspark_append_params* p, const dspark_block_exponents* x, const void* k_pages, const void* v_pages) {
    if (!p || !x || p->T < 0 || p->Hk < 1 || p->D < 1 || p->num_pages < 1 || page_shift_of(p->page_size) < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (p->dtype != DSPARK_BF16 && p->dtype != DSPARK_F16) return DSPARK_ERR_INVALID_ARG;
    if (p->kv_dtype != DSPARK_I8 || !k_pages || !v_pages || !valid_block_exponents(x, p->page_size)) return DSPARK_ERR_INVALID_ARG;
    if (p->D % 16 || p->D > 256 || p->Hk > (1 << 20)) return DSPARK_ERR_UNSUPPORTED;
    if ((((uintptr_t)k_pages | (uintptr_t)v_pages) & 15u) || p->kv_page_stride % 16 || p->kv_token_stride % 16 ||
        p->kv_head_stride % 16)
        return DSPARK_ERR_INVALID_ARG;
    return DSPARK_OK;
}
int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

bool valid_block_exponents(const dspark_block_exponents* x, int page_size) {
    return x->k && x->v && x->block >= 1 && x->block <= 128 && x->block <= page_size && !(x->block & (x->block - 1)) &&
           x->page_stride >= 0 && x->block_stride >= 0 && x->head_stride >= 0;
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_cache_append_i8(const dspark_append_params* p, const dspark_block_exponents* x, const void* k,
                                                const void* v, void* k_pages, void* v_pages, const int64_t* slots,
                                                int32_t* error, dspark_stream_t stream) {
    const dspark_status st = check_i8(p, x, k_pages, v_pages);
    if (st != DSPARK_OK) return st;
    if ((p->T && (!k || !v || !slots)) || (((uintptr_t)k | (uintptr_t)v) & 1u) || ((uintptr_t)error & 3u)) return DSPARK_ERR_INVALID_ARG;
    if (k_pages == v_pages || x->k == x->v) return DSPARK_ERR_INVALID_ARG;
    if (p->T == 0) return DSPARK_OK;
    int sms = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    I8Args a;
    a.T = p->T;
    a.Hk = p->Hk;
    a.D = p->D;
    a.page_shift = page_shift_of(p->page_size);
    a.block_shift = log2_of(x->block);
    a.chunks = p->D / 8;
    a.chunk_mul = (65536u + a.chunks - 1) / a.chunks;
    a.slots_end = (long long)p->num_pages * p->page_size;
    a.x[0] = static_cast<const uint16_t*>(k);
    a.x[1] = static_cast<const uint16_t*>(v);
    a.x_token[0] = p->k_token_stride;
    a.x_token[1] = p->v_token_stride;
    a.x_head[0] = p->k_head_stride;
    a.x_head[1] = p->v_head_stride;
    a.pages[0] = static_cast<signed char*>(k_pages);
    a.pages[1] = static_cast<signed char*>(v_pages);
    a.page = p->kv_page_stride;
    a.token = p->kv_token_stride;
    a.head = p->kv_head_stride;
    a.exps[0] = x->k;
    a.exps[1] = x->v;
    a.e_page = x->page_stride;
    a.e_block = x->block_stride;
    a.e_head = x->head_stride;
    a.slots = slots;
    a.error = error;
    // A warp looks after one entry of slots, or, where that would be more warps than are resident at once, after up to a
    // block's worth (most of a prompt's entries begin no run).
    a.window_shift = 0;
    auto items = [&] { return ((long long)a.T + (1 << a.window_shift) - 1 >> a.window_shift) * 2 * a.Hk; };
    while (a.window_shift < 5 && a.window_shift < a.block_shift && items() > (long long)sms * 32) ++a.window_shift;
    a.items = items();
    const bool aligned = !((((uintptr_t)k | (uintptr_t)v) & 15u) || (a.x_token[0] | a.x_token[1] | a.x_head[0] | a.x_head[1]) % 8);
    const long long want = (a.items + kWarps - 1) / kWarps, most = (long long)sms * 16;
    const int blocks = (int)(want < most ? want : most);
    const bool bf16 = p->dtype == DSPARK_BF16;
    const auto kernel = bf16 ? (aligned ? cache_append_i8_kernel<true, true> : cache_append_i8_kernel<true, false>)
                             : (aligned ? cache_append_i8_kernel<false, true> : cache_append_i8_kernel<false, false>);
    if (launch_overlapped(kernel, blocks, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess) return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_read_i8(const dspark_append_params* p, const dspark_block_exponents* x,
                                              const void* k_pages, const void* v_pages, const int64_t* slots, void* k, void* v,
                                              dspark_stream_t stream) {
    const dspark_status st = check_i8(p, x, k_pages, v_pages);
    if (st != DSPARK_OK) return st;
    if ((p->T && (!k || !v || !slots)) || (((uintptr_t)k | (uintptr_t)v) & 15u)) return DSPARK_ERR_INVALID_ARG;
    const long long row = (long long)p->Hk * p->D;
    if (p->k_token_stride != row || p->v_token_stride != row || p->k_head_stride != p->D || p->v_head_stride != p->D)
        return DSPARK_ERR_INVALID_ARG;
    if (p->T == 0) return DSPARK_OK;
    int sms = 0;
    if (device_sm_count(&sms) != cudaSuccess) return DSPARK_ERR_CUDA;
    ReadArgs a;
    a.page_shift = page_shift_of(p->page_size);
    a.chunks = (uint32_t)p->D / 16;
    a.per_token = (uint32_t)p->Hk * a.chunks;
    a.total = (long long)p->T * a.per_token;
    a.slots_end = (long long)p->num_pages * p->page_size;
    a.pages[0] = static_cast<const signed char*>(k_pages);
    a.pages[1] = static_cast<const signed char*>(v_pages);
    a.page = p->kv_page_stride;
    a.token = p->kv_token_stride;
    a.head = p->kv_head_stride;
    a.exp = {x->k, x->v, x->page_stride, x->block_stride, x->head_stride, log2_of(x->block)};
    a.slots = slots;
    a.out[0] = static_cast<uint4*>(k);
    a.out[1] = static_cast<uint4*>(v);
    const long long want = (a.total + kThreads - 1) / kThreads, most = (long long)sms * 32;
    const int blocks = (int)(want < most ? want : most);
    const auto kernel = p->dtype == DSPARK_BF16 ? cache_read_i8_kernel<true> : cache_read_i8_kernel<false>;
    if (launch_overlapped(kernel, blocks, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess) return DSPARK_ERR_CUDA;
    note_launch();
    return DSPARK_OK;
}
