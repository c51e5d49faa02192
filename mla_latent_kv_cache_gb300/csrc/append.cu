// From a projection's output to cached rows (mla_cache_append): a token's
// latent c[0:D] and rotary key k[0:64] become the row
//   c * rsqrt(mean(c^2) + eps) * w   and   k turned by its position,
// computed in 32 bits and written where the request's block table puts the
// token, each value rounded once.
//
// Bound: HBM for prompts (1152 bytes read, 576 to 1152 written a token),
// latency for steps: the loads of a row depend on nothing but its index, so they
// go out before the request, its length and its page are looked up.
//
// Prompts are near the rate at which instructions issue as well (unpacking, the
// norm, the rotation and the rounding are some 240 of them a token), hence packed
// fp32 instructions, a reduction for several tokens at once, one sine and cosine
// for four positions, and tokens that wait in shared memory instead of registers.
// Measured: 98,304 tokens into 656-byte rows 31 to 32 us (5.6 TB/s, 0.81 to 0.84 of the copy
// rate), into bf16 rows 41 us (0.81), 52,106 tokens of 16 prompts into page rows, with dense rows
// besides, 33 us (0.67, issue slots 55% busy), 64 requests with a token each 3.7 us (7 as a call).
//
// bf16 and fp8_ds_mla rows: a warp a token, or for prompts a stream of them. Page rows (one scale for all rows of
// a page): the warps of a page hold its new tokens in registers, meet for the
// largest value, and write when the scale is known, so a token's input is read
// once. The scale is a power of two: e4m3 values keep their 4 significant bits
// whatever it is, and when a later token makes it grow, the codes before it are
// divided by a power of two, which changes only those that become subnormal.
#include <climits>

#include "launch.cuh"
#include "mla.h"
#include "mla_common.cuh"
#include "rope.cuh"

namespace mla {

namespace {

constexpr int kAppendWarps = 8;

__device__ __forceinline__ int a_cu(const AppendParams& p, int b) {
    return static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.cu + b), 0)), p.total));
}

using F2 = packed2;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& u, F2 (&f)[4]) {
    f[0] = f2(bf16_lo(u.x), bf16_hi(u.x));
    f[1] = f2(bf16_lo(u.y), bf16_hi(u.y));
    f[2] = f2(bf16_lo(u.z), bf16_hi(u.z));
    f[3] = f2(bf16_lo(u.w), bf16_hi(u.w));
}

__device__ __forceinline__ uint32_t bf16x2(F2 v) {
    const float2 f = un2(v);
    return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
    return make_uint4(bf16x2(f[0]), bf16x2(f[1]), bf16x2(f[2]), bf16x2(f[3]));
}

__device__ __forceinline__ float most_abs(float a, const F2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = un2(f[i]);
        a = fmaxf(a, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    return a;
}

// The sum of squares of 8 values, by pairs.
__device__ __forceinline__ F2 squares(F2 s, const F2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(f[i], f[i], s);
    return s;
}

// One step of a sum of several numbers over a warp at once: a lane keeps half of its
// N numbers and hands the other half to the lane `bit` away, so that all of them
// together take N - 1 shuffles until a lane has one, where one by one they take five each.
template <int N>
__device__ __forceinline__ void halve(float (&v)[N], int bit, int lane) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = up ? v[i + N / 2] : v[i], give = up ? v[i] : v[i + N / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
    }
}

// The sums over a warp of eight numbers: lane L gets number L / 4's.
__device__ __forceinline__ float sums_of(float (&v)[8], int lane) {
    halve(v, 16, lane);
    float a[4] = {v[0], v[1], v[2], v[3]};
    halve(a, 8, lane);
    float b[2] = {a[0], a[1]};
    halve(b, 4, lane);
    float r = b[0] + __shfl_xor_sync(0xffffffffu, b[0], 2);
    return r + __shfl_xor_sync(0xffffffffu, r, 1);
}

// 1 / rms from a lane's sum of squares; a whole warp.
__device__ __forceinline__ float norm_factor(F2 squares, float per, float eps) {
    const float2 v = un2(squares);
    float s = v.x + v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return rsqrtf(fmaf(s, per, eps));
}

// A lane's norm weights of the 16-byte unit u (1 without a norm).
__device__ __forceinline__ void weights8(const AppendParams& p, int u, F2 (&w)[4]) {
    if (p.norm) unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm) + u), w);
    else w[0] = w[1] = w[2] = w[3] = f2(1.f, 1.f);
}

// Pair `lane` of the rotary key at pe, as two bf16 values, the first in the low
// half. (Plain loads: the dense rows may be written over the input they came from.)
__device__ __forceinline__ uint32_t load_pair(const void* pe, int interleaved, int lane) {
    if (interleaved) return static_cast<const uint32_t*>(pe)[lane];
    const uint32_t a = static_cast<const unsigned short*>(pe)[lane], b = static_cast<const unsigned short*>(pe)[lane + 32];
    return a | b << 16;
}

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -__fmul_rn(b, cs.y)), fmaf(a, cs.y, __fmul_rn(b, cs.x)));
}

// The angles of a warp's tokens, every DELTA-th, for the lane's pair. Most
// positions follow each other, and a turn by DELTA positions more is four
// instructions instead of another sine and cosine. It is off by some 2^-22 each
// time, so every fourth is formed anew.
// (The fused steps are written out, so that every kernel rounds alike.)
template <int DELTA>
struct Angle {
    int pos;
    float2 cs, step;
    int left = -1;  // turns before the next one is formed anew
    __device__ __forceinline__ float2 turn(const AppendParams& p, uint32_t pe, int at, int lane) {
        const float a = bf16_lo(pe), b = bf16_hi(pe);
        if (!p.steps) return make_float2(a, b);
        if (left > 0 && at == pos + DELTA) {
            cs = turned(cs.x, cs.y, step);
            --left;
        } else {
            const int64_t f = __ldg(p.steps + lane);
            cs = rope_cos_sin(at, f, p.mscale);
            if (left < 0) step = rope_cos_sin(DELTA, f, 1.f);
            left = 3;
        }
        pos = at;
        return turned(a, b, cs);
    }
};

// The turned pair as bf16 into the 64 values at dst.
__device__ __forceinline__ void store_pe(const AppendParams& p, void* dst, float2 r, int lane) {
    const uint32_t v = pack_bf16x2(r.x, r.y);
    if (p.interleaved) {
        static_cast<uint32_t*>(dst)[lane] = v;
    } else {
        static_cast<unsigned short*>(dst)[lane] = static_cast<unsigned short>(v);
        static_cast<unsigned short*>(dst)[lane + 32] = static_cast<unsigned short>(v >> 16);
    }
}

// Four values as e4m3 codes, saturated.
__device__ __forceinline__ uint32_t codes4(F2 a, F2 b) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(un2(a), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(un2(b), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// x / s correctly rounded for s within 2^-89 .. 2^82, with y = 1 / s correctly
// rounded, by Markstein's correction (P. Markstein, Computation of elementary
// functions on the IBM RISC System/6000 processor, 1990): the remainder of
// x y is exact in one fused step. It is taken as q s - x, so that a zero keeps its
// sign. (Where x is so small that the remainder is not exact, below 2^-10 s, the code is 0 anyway.)
__device__ __forceinline__ F2 div2(F2 x, F2 minus_x, F2 s, F2 y, F2 minus_y) {
    const F2 q = mul2(x, y);
    return fma2(fma2(q, s, minus_x), minus_y, q);
}

// The page of table column pi of request b, or -1 (outside the pool or the row).
__device__ __forceinline__ int64_t a_page(const AppendParams& p, int b, int64_t pi) {
    if (pi < 0 || pi >= p.bt_cols) return -1;
    const int64_t page = __ldg(p.block_table + static_cast<int64_t>(b) * p.bt_stride + pi);
    return page >= 0 && (page + 1) * p.page_size <= p.num_slots ? page : -1;
}

__device__ __forceinline__ void a_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Where a token goes: the first byte of its row in the pool (-1: nowhere) and its
// position; named: a request names it.
struct Where {
    int64_t row;
    int pos;
    int named;
};
template <int KIND, int D>
__device__ __forceinline__ Where locate(const AppendParams& p, int64_t t) {
    constexpr int row_bytes = KIND == MLA_CACHE_FP8_DS_MLA_656 ? kRowFp8 : 2 * (D + kP);
    // the last b with cu[b] <= t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a_cu(p, mid) <= t) lo = mid;
        else hi = mid;
    }
    const int c0 = a_cu(p, lo), c1 = a_cu(p, lo + 1);
    Where w;
    w.named = t >= c0 && t < c1;
    const int place = max(__ldg(p.seq_lens + lo), 0) - c1 + static_cast<int>(t);
    const int64_t page = w.named && place >= 0 ? a_page(p, lo, place / p.page_size) : -1;
    w.row = page >= 0 ? (page * p.page_size + place % p.page_size) * row_bytes : -1;
    w.pos = p.positions && w.named ? __ldg(p.positions + t) : place;
    return w;
}

// A lane's 16-byte units of the latent: lane, lane + 32, ..; of fp8_ds_mla rows
// 2 lane and 2 lane + 1, so that it has one block's scale to find, with seven
// other lanes.
template <int KIND>
__device__ __forceinline__ int a_unit(int lane, int k) {
    return KIND == MLA_CACHE_FP8_DS_MLA_656 ? 2 * lane + k : lane + 32 * k;
}

// Token t from its units and its turned pair to its row and its dense row.
template <int KIND, int D>
__device__ __forceinline__ void put_token(const AppendParams& p, int64_t t, const Where& at, const uint4 (&lat)[D / 256],
                                          const F2 (&w)[D / 256][4], float2 pe, int lane) {
    constexpr bool kFp8 = KIND == MLA_CACHE_FP8_DS_MLA_656;
    constexpr int U = D / 256;
    F2 f[U][4];
    F2 sq = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        unpack8(lat[k], f[k]);
        sq = squares(sq, f[k]);
    }
    float c = 1.f;  // f times c are the normalised values
    if (p.norm) {
        c = norm_factor(sq, 1.f / D, p.eps);
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[k][i] = mul2(f[k][i], w[k][i]);
    }
    uint8_t* row = p.cache + at.row;
    const bool put = at.row >= 0;
    if (p.rows || !kFp8) {
        uint4* dense = p.rows ? reinterpret_cast<uint4*>(p.rows + t * p.rows_st) : nullptr;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            F2 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul2(f[k][i], f2(c, c));
            const uint4 v = pack8(y);
            if (dense) dense[a_unit<KIND>(lane, k)] = v;
            if (!kFp8 && put) reinterpret_cast<uint4*>(row)[a_unit<KIND>(lane, k)] = v;
        }
        if (dense) store_pe(p, dense + D / 8, pe, lane);
    }
    if constexpr (kFp8) {
        float top = most_abs(most_abs(0.f, f[0]), f[U - 1]) * c;  // (rounding keeps the order)
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float scale;
        uint32_t code[4];
        if (top > 0x1p-80f && top < 0x1p90f) {
            const float q = top * (1.f / 448.f);
            scale = fmaf(fmaf(q, 448.f, -top), -1.f / 448.f, q);  // top / 448, correctly rounded (see div2)
            if (p.norm) {
                // values and factor in one: a quotient within two units of its last place
                const float r = __fdividef(c, scale);
                const F2 r2 = f2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    code[i] = codes4(mul2(f[i >> 1][2 * (i & 1)], r2), mul2(f[i >> 1][2 * (i & 1) + 1], r2));
            } else {
                // the codes of mla_cache_write, bit for bit
                const float y = __frcp_rn(scale);
                const F2 s2 = f2(scale, scale), y2 = f2(y, y), my2 = f2(-y, -y), m1 = f2(-1.f, -1.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 a = f[i >> 1][2 * (i & 1)], b = f[i >> 1][2 * (i & 1) + 1];
                    code[i] = codes4(div2(a, mul2(a, m1), s2, y2, my2), div2(b, mul2(b, m1), s2, y2, my2));
                }
            }
        } else {
            scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = un2(f[i >> 1][2 * (i & 1)]), b = un2(f[i >> 1][2 * (i & 1) + 1]);
                code[i] = codes4(f2(__fdiv_rn(a.x * c, scale), __fdiv_rn(a.y * c, scale)),
                                 f2(__fdiv_rn(b.x * c, scale), __fdiv_rn(b.y * c, scale)));
            }
        }
        if (put) {
            reinterpret_cast<uint4*>(row)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
            if ((lane & 7) == 0) reinterpret_cast<float*>(row + kD)[lane >> 3] = scale;
        }
    }
    if (put) store_pe(p, row + (kFp8 ? kD + 16 : 2 * D), pe, lane);
}

// A warp a token.
template <int KIND, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
    constexpr int U = D / 256;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= p.total) return;
    uint4 lat[U];
    const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * p.lat_st);
#pragma unroll
    for (int k = 0; k < U; ++k) lat[k] = src[a_unit<KIND>(lane, k)];
    const uint32_t pair = load_pair(p.k_pe + t * p.pe_st, p.interleaved, lane);
    F2 w[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) weights8(p, a_unit<KIND>(lane, k), w[k]);
    const Where at = locate<KIND, D>(p, t);
    if (!at.named) return;
    if (at.row < 0 && lane == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    Angle<1> angle;
    put_token<KIND, D>(p, t, at, lat, w, angle.turn(p, pair, at.pos, lane), lane);
}

// Prompts: a CTA a run of tokens, as long as lets all CTAs run at once, its warps
// every eighth of it. Each has kMany on their way to shared memory, and looks 32 up at
// once, a lane each. (98,304 tokens into 656-byte rows: 31.1 us; with a run a warp
// 31.7; runs for twice as many CTAs 37 against 35.4; kMany 2 31.1, 4 31.9; four CTAs
// an SM, whose 64 registers a thread spill, 34.8; a CTA for every 32 tokens, all of
// them asked for at once, 36.)
constexpr int kMany = 3;
template <int D>
constexpr int many_smem() {
    return kAppendWarps * kMany * 2 * (D + kP);
}
constexpr int kManyCtas = 3;  // CTAs an SM holds

template <int KIND, int D>
__global__ void __launch_bounds__(32 * kAppendWarps, kManyCtas) append_many_kernel(const AppendParams p, int per) {
    constexpr int U = D / 256, held_row = 2 * (D + kP);
    extern __shared__ uint8_t held_raw[];
    __shared__ Where ways[kAppendWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    // token n of the warp is t0 + n kAppendWarps
    const int64_t first = static_cast<int64_t>(blockIdx.x) * per, t0 = first + (threadIdx.x >> 5);
    const int m = static_cast<int>((min(first + per, p.total) - t0 + kAppendWarps - 1) / kAppendWarps);
    if (m <= 0) return;
    const uint8_t* held = held_raw + (threadIdx.x >> 5) * kMany * held_row;
    const uint32_t to = smem_u32(held) + lane * 16;
    const __nv_bfloat16 *lat_at = p.latent + t0 * p.lat_st + lane * 8, *pe_at = p.k_pe + t0 * p.pe_st + lane * 8;
    int fetched = 0;
    auto fetch = [&]() {  // the next token, if any
        if (fetched < m) {
            const uint32_t dst = to + (fetched % kMany) * held_row;
#pragma unroll
            for (int k = 0; k < U; ++k) a_cp16(dst + 512 * k, lat_at + 256 * k);
            if (lane < 8) a_cp16(dst + 2 * D, pe_at);
            lat_at += kAppendWarps * p.lat_st;
            pe_at += kAppendWarps * p.pe_st;
            ++fetched;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int n = 0; n < kMany; ++n) fetch();
    F2 w[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) weights8(p, a_unit<KIND>(lane, k), w[k]);
    Where* way = ways[threadIdx.x >> 5];
    Angle<kAppendWarps> angle;
#pragma unroll 1
    for (int n = 0; n < m; ++n) {
        if ((n & 31) == 0) {
            const Where mine = locate<KIND, D>(p, t0 + min(n + lane, m - 1) * kAppendWarps);
            way[lane] = mine;
            if (__any_sync(0xffffffffu, mine.named && mine.row < 0) && lane == 0 && p.status) atomicOr(p.status, kErrBadBlock);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kMany - 1) : "memory");
        __syncwarp();
        const Where at = way[n & 31];
        const uint4* src = reinterpret_cast<const uint4*>(held + (n % kMany) * held_row);
        uint4 lat[U];
#pragma unroll
        for (int k = 0; k < U; ++k) lat[k] = src[a_unit<KIND>(lane, k)];
        const uint32_t pair = load_pair(src + D / 8, p.interleaved, lane);
        __syncwarp();
        fetch();
        if (!at.named) continue;
        put_token<KIND, D>(p, t0 + n * kAppendWarps, at, lat, w, angle.turn(p, pair, at.pos, lane), lane);
    }
}

// ------------------------------------------------------------------ page rows

constexpr int kHold = 8;                    // new tokens of a page that a warp keeps
constexpr int kHeldRow = 2 * (kD + kP);     // bytes of one
constexpr int kPageSmem = kAppendWarps * kHold * kHeldRow;

// The least power of two s with top <= 448 s, within 2^-40 .. 2^40: top =
// m 2^e with m in [1, 2), and 448 = 1.75 * 2^8.
__device__ __forceinline__ float page_scale(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(-40, min(40, e)) + 127) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;  // NaN too
}

// W warps a page. Page items: request b has (cu[b+1] - cu[b]) / page_size + 2
// or more of them, from item cu[b] / page_size + 2 b on, which is as many as
// the pages its tokens can touch; those past its last page have nothing to do.
template <int W>
__global__ void __launch_bounds__(32 * kAppendWarps, 3) append_page_kernel(const AppendParams p) {
    constexpr int kItems = kAppendWarps / W;  // pages a CTA
    extern __shared__ uint8_t held_raw[];
    __shared__ float tops[kAppendWarps];
    __shared__ alignas(16) float factors[kAppendWarps][kHold];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % W, grp = warp / W;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kItems + grp;
    const int ps = p.page_size;
    auto first_item = [&](int b) { return static_cast<int64_t>(a_cu(p, b) / ps) + 2 * static_cast<int64_t>(b); };
    // the last b with first_item(b) <= item, 32 probes at a time
    int b = 0;
    for (int left = p.B; left > 1;) {
        const int step = (left + 31) / 32, off = lane * step;
        const int hits = __popc(__ballot_sync(0xffffffffu, off < left && first_item(b + off) <= item));
        const int at = max(hits - 1, 0) * step;
        b += at;
        left = min(step, left - at);
    }
    const int c0 = a_cu(p, b), n = a_cu(p, b + 1) - c0;
    if (n <= 0) return;  // (the whole group leaves)
    // places p0 .. p1 - 1 are new; those below 0 have none
    const int64_t p1 = max(__ldg(p.seq_lens + b), 0), p0 = p1 - n;
    const int64_t pi = static_cast<int>(max(p0, static_cast<int64_t>(0))) / ps + (item - first_item(b));
    const bool none = p0 < 0 && item == first_item(b);  // this item also sees to the tokens without a place
    if (none && lane == 0 && wi == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    int64_t j0 = max(pi * ps, max(p0, static_cast<int64_t>(0)));
    const int64_t j1 = min((pi + 1) * ps, p1);
    if (none) j0 = p0;
    if (j0 >= j1) return;
    const int64_t t0 = c0 + (j0 - p0);  // the first token's row
    const int m = static_cast<int>(j1 - j0);
    // the token at index x of the item, 0 <= x < m, is warp x % W's. The first
    // kHold of each are on their way to shared memory while the page is looked up.
    uint8_t* held = held_raw + warp * kHold * kHeldRow;
    {
        const __nv_bfloat16 *src = p.latent + (t0 + wi) * p.lat_st + lane * 8, *pe = p.k_pe + (t0 + wi) * p.pe_st + lane * 8;
        uint32_t dst = smem_u32(held) + lane * 16;
        for (int x = wi; x < min(m, kHold * W); x += W, src += W * p.lat_st, pe += W * p.pe_st, dst += kHeldRow) {
            a_cp16(dst, src);
            a_cp16(dst + 512, src + 256);
            if (lane < 8) a_cp16(dst + 1024, pe);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // Tokens without a place touch no page: of a request without any (its length 0 in a padded
    // batch) the table's first entry is no page of its own, and its scale another request's.
    const bool placed = j1 > max(j0, static_cast<int64_t>(0));
    const int64_t page = placed ? a_page(p, b, pi) : -1;
    const bool bad = placed && page < 0;
    if (bad && lane == 0 && wi == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    const int64_t off = max(p0, static_cast<int64_t>(0)) - pi * ps;  // rows of the page that were there before (if > 0)
    const float old = page >= 0 && off > 0 ? __ldcg(p.scales + page) : 0.f;
    F2 w[2][4];
    weights8(p, lane, w[0]);
    weights8(p, lane + 32, w[1]);
    float top = 0.f;
    Angle<W> angle;
    auto position = [&](int x) { return p.positions ? __ldg(p.positions + t0 + x) : static_cast<int>(j0) + x; };
    // a token's values times the weights (times its factor they are normalised);
    // returns the factor
    auto weighed = [&](uint4 a, uint4 c, F2 (&f)[2][4], bool want) {
        unpack8(a, f[0]);
        unpack8(c, f[1]);
        if (!p.norm) return 1.f;
        const float fac = want ? norm_factor(squares(squares(f2(0.f, 0.f), f[0]), f[1]), 1.f / kD, p.eps) : 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[u][i] = mul2(f[u][i], w[u][i]);
        return fac;
    };
    // the largest magnitude of a token's finite values
    const int skip = static_cast<int>(max(-j0, static_cast<int64_t>(0)));  // tokens of the item without a place
    auto largest = [&](const F2 (&f)[2][4], float fac, float2 e, int x) {
        if (x < skip) return;
        float a = most_abs(most_abs(0.f, f[0]), f[1]) * fac;  // (rounding keeps the order)
        a = fmaxf(a, fmaxf(fabsf(e.x), fabsf(e.y)));
        if (!(a < INFINITY)) {
            a = fmaxf(finite_abs(e.x), finite_abs(e.y));
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = un2(f[u][i]);
                    a = fmaxf(a, fmaxf(finite_abs(v.x * fac), finite_abs(v.y * fac)));
                }
        }
        top = fmaxf(top, a);
    };
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // Sums of squares and largest magnitudes of the held tokens: one pass, and one
    // reduction for all of them.
    float sq[kHold], mx[kHold];
    float2 es[kHold];  // the turned pairs (16 prompts 32.6 us; turned again when they are written 34.2)
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int x = wi + k * W;
        sq[k] = mx[k] = 0.f;
        if (x >= m) continue;
        const uint4* lat = reinterpret_cast<const uint4*>(held + k * kHeldRow);
        F2 f[2][4];
        unpack8(lat[lane], f[0]);
        unpack8(lat[lane + 32], f[1]);
        if (p.norm) {
            const float2 v = un2(squares(squares(f2(0.f, 0.f), f[0]), f[1]));
            sq[k] = v.x + v.y;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) f[u][i] = mul2(f[u][i], w[u][i]);
        }
        const float2 e = es[k] = angle.turn(p, load_pair(lat + 64, p.interleaved, lane), position(x), lane);
        if (x < skip) continue;
        mx[k] = most_abs(most_abs(0.f, f[0]), f[1]);
        top = fmaxf(top, fmaxf(fabsf(e.x), fabsf(e.y)));
    }
    {
        const float total = sums_of(sq, lane);  // lane L: token L / 4's
        if ((lane & 3) == 0) factors[warp][lane >> 2] = p.norm ? rsqrtf(fmaf(total, 1.f / kD, p.eps)) : 1.f;
        __syncwarp();
        const float4 a = *reinterpret_cast<const float4*>(factors[warp]), c = *reinterpret_cast<const float4*>(factors[warp] + 4);
        const float fac[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < kHold; ++k) top = fmaxf(top, mx[k] * fac[k]);  // (rounding keeps the order; NaN is left out)
        if (__any_sync(0xffffffffu, !(top < INFINITY))) {
            // an infinity among them: the largest of the finite ones, value by value
            top = 0.f;
            for (int k = 0, x = wi; k < kHold && x < m; ++k, x += W) {
                const uint4* lat = reinterpret_cast<const uint4*>(held + k * kHeldRow);
                F2 f[2][4];
                weighed(lat[lane], lat[lane + 32], f, false);
                largest(f, factors[warp][k], angle.turn(p, load_pair(lat + 64, p.interleaved, lane), position(x), lane), x);
            }
        }
    }
    angle.left = min(angle.left, 0);
    for (int x = wi + kHold * W; x < m; x += W) {  // pages of more rows than the warps hold: read twice
        const uint4* lat = reinterpret_cast<const uint4*>(p.latent + (t0 + x) * p.lat_st);
        F2 f[2][4];
        const float fac = weighed(lat[lane], lat[lane + 32], f, true);
        largest(f, fac, angle.turn(p, load_pair(p.k_pe + (t0 + x) * p.pe_st, p.interleaved, lane), position(x), lane), x);
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // (not negative: ordered as its bits)
    if constexpr (W > 1) {
        if (lane == 0) tops[warp] = top;
        named_bar_sync(1 + grp, 32 * W);
#pragma unroll
        for (int i = 0; i < W; ++i) top = fmaxf(top, tops[grp * W + i]);
    }
    float scale = page_scale(top);
    if (page >= 0) {
        if (off > 0 && old >= scale) scale = old;
        else if (off > 0 && old > 0.f) {
            // the rows before, in units of the new scale
            const float ratio = old / scale;
            uint8_t* rows = p.cache + page * ps * static_cast<int64_t>(kRowPage);
            for (int64_t u = wi * 32 + lane; u < off * (kRowPage / 16); u += 32 * W) {
                uint4 v = reinterpret_cast<const uint4*>(rows)[u];
                uint32_t* v4 = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw h01 = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v4[i] & 0xFFFFu), __NV_E4M3);
                    const __half2_raw h23 = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v4[i] >> 16), __NV_E4M3);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h23));
                    v4[i] = codes4(f2(a.x * ratio, a.y * ratio), f2(c.x * ratio, c.y * ratio));
                }
                reinterpret_cast<uint4*>(rows)[u] = v;
            }
        }
        if (lane == 0 && wi == 0 && scale != old) p.scales[page] = scale;
    }
    const float inv = 1.f / scale;  // exact: a power of two
    // the dense row and the cached row of token wi; those of the warp's next are W rows further
    __nv_bfloat16* dense = p.rows ? p.rows + (t0 + wi) * p.rows_st : nullptr;
    uint8_t* row = p.cache + (page * ps + (j0 + wi - pi * ps)) * static_cast<int64_t>(kRowPage);
    const int from = page >= 0 ? skip : INT_MAX;  // tokens below this are not cached
    auto write = [&](const F2 (&f)[2][4], float fac, float2 e, int x) {
        if (dense) {
            uint4* d = reinterpret_cast<uint4*>(dense);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                F2 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = mul2(f[u][i], f2(fac, fac));
                d[lane + 32 * u] = pack8(y);
            }
            store_pe(p, d + kD / 8, e, lane);
            dense += W * p.rows_st;
        }
        if (x >= from) {
            const F2 c = f2(fac * inv, fac * inv);  // (inv is a power of two: the same as two multiplications)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                reinterpret_cast<uint2*>(row)[lane + 32 * u] =
                    make_uint2(codes4(mul2(f[u][0], c), mul2(f[u][1], c)), codes4(mul2(f[u][2], c), mul2(f[u][3], c)));
            const uint32_t v = __nv_cvt_float2_to_fp8x2(make_float2(e.x * inv, e.y * inv), __NV_SATFINITE, __NV_E4M3);
            if (p.interleaved) {
                reinterpret_cast<unsigned short*>(row + kD)[lane] = static_cast<unsigned short>(v);
            } else {
                row[kD + lane] = static_cast<uint8_t>(v);
                row[kD + 32 + lane] = static_cast<uint8_t>(v >> 8);
            }
        }
        row += W * kRowPage;
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int x = wi + k * W;
        if (x >= m) break;
        const uint4* lat = reinterpret_cast<const uint4*>(held + k * kHeldRow);
        F2 f[2][4];
        weighed(lat[lane], lat[lane + 32], f, false);
        write(f, factors[warp][k], es[k], x);
    }
    angle.left = min(angle.left, 0);  // (as the first time: the largest value is among these)
    for (int x = wi + kHold * W; x < m; x += W) {
        const uint4* lat = reinterpret_cast<const uint4*>(p.latent + (t0 + x) * p.lat_st);
        F2 f[2][4];
        const float fac = weighed(lat[lane], lat[lane + 32], f, true);
        write(f, fac, angle.turn(p, load_pair(p.k_pe + (t0 + x) * p.pe_st, p.interleaved, lane), position(x), lane), x);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int kind, int lat_dim, int sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    if (kind == MLA_CACHE_FP8_PAGE_576) {
        const int W = p.page_size <= 8 ? 1 : p.page_size <= 16 ? 2 : p.page_size <= 32 ? 4 : 8;
        const int64_t items = p.total / p.page_size + 2 * static_cast<int64_t>(p.B);
        const int64_t blocks = (items + kAppendWarps / W - 1) / (kAppendWarps / W);
        static std::atomic<uint64_t> done[4];
        auto go = [&](auto* k, int i) {
            const cudaError_t e = attribute_once(done[i], reinterpret_cast<const void*>(k),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kPageSmem);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), 32 * kAppendWarps, kPageSmem, stream, attr);
            return cudaLaunchKernelEx(&cfg, k, p);
        };
        return W == 1   ? go(append_page_kernel<1>, 0)
               : W == 2 ? go(append_page_kernel<2>, 1)
               : W == 4 ? go(append_page_kernel<4>, 2)
                        : go(append_page_kernel<8>, 3);
    }
    // Runs where every warp that fits gets kMany tokens or more (11,008 tokens into
    // 656-byte rows: 5.9 us, 6.1 with a warp a token; 4,096: 4.0 and 3.7)
    const int64_t held = static_cast<int64_t>(sms) * kManyCtas, share = (p.total + held - 1) / held;
    const bool many = share >= kAppendWarps * kMany && lat_dim <= 768;
    const int64_t each = many ? share : kAppendWarps, blocks = (p.total + each - 1) / each;
    static std::atomic<uint64_t> done[4];
    auto go = [&](auto* k, int smem, int i, auto... more) {
        if (smem > 0) {
            const cudaError_t e = attribute_once(done[i], reinterpret_cast<const void*>(k),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), 32 * kAppendWarps, smem, stream, attr);
        return cudaLaunchKernelEx(&cfg, k, p, more...);
    };
#define MLA_APPEND(K, DV, I) \
    (many ? go(append_many_kernel<K, DV>, many_smem<DV>(), I, static_cast<int>(share)) : go(append_kernel<K, DV>, 0, I))
    if (kind == MLA_CACHE_FP8_DS_MLA_656) return MLA_APPEND(MLA_CACHE_FP8_DS_MLA_656, 512, 0);
    return lat_dim == 256   ? MLA_APPEND(MLA_CACHE_BF16_576, 256, 1)
           : lat_dim == 512 ? MLA_APPEND(MLA_CACHE_BF16_576, 512, 2)
           : lat_dim == 768 ? MLA_APPEND(MLA_CACHE_BF16_576, 768, 3)
                            : go(append_kernel<MLA_CACHE_BF16_576, 1792>, 0, 0);
#undef MLA_APPEND
}

}  // namespace mla
