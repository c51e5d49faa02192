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
// bf16 and fp8_ds_mla rows: a warp a token. Page rows (one scale for all rows of
// a page): the warps of a page hold its new tokens in registers, meet for the
// largest value, and write when the scale is known, so a token's input is read
// once. The scale is a power of two: e4m3 values keep their 4 significant bits
// whatever it is, and when a later token makes it grow, the codes before it are
// divided by a power of two, which changes only those that become subnormal.
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

// (Plain loads: the dense rows may be written over the input they came from.)
// A token's input as a lane holds it: 16-byte units lane, lane + 32, .. of the
// latent, and pair `lane` of the rotary key.
template <int D>
struct Raw {
    static constexpr int kU = D / 256;
    uint4 lat[kU];
    uint32_t pe;  // two bf16 values, the pair's first in the low half
};

template <int D>
__device__ __forceinline__ void load_raw(const AppendParams& p, int64_t t, int lane, Raw<D>& r) {
    const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * p.lat_st);
#pragma unroll
    for (int k = 0; k < Raw<D>::kU; ++k) r.lat[k] = src[lane + 32 * k];
    const __nv_bfloat16* pe = p.k_pe + t * p.pe_st;
    if (p.interleaved) {
        r.pe = reinterpret_cast<const uint32_t*>(pe)[lane];
    } else {
        const uint32_t a = reinterpret_cast<const unsigned short*>(pe)[lane];
        const uint32_t b = reinterpret_cast<const unsigned short*>(pe)[lane + 32];
        r.pe = a | b << 16;
    }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// 1 / rms of the token's latent (1 without a norm); a whole warp.
template <int D>
__device__ __forceinline__ float norm_factor(const AppendParams& p, const Raw<D>& r) {
    if (!p.norm) return 1.f;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < Raw<D>::kU; ++k) {
        float f[8];
        unpack8(r.lat[k], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return rsqrtf(s * (1.f / D) + p.eps);
}

// Unit k of the lane's latent values, normalised.
template <int D>
__device__ __forceinline__ void latent8(const AppendParams& p, const Raw<D>& r, int k, int lane, float factor, float (&f)[8]) {
    unpack8(r.lat[k], f);
    if (!p.norm) return;
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm) + lane + 32 * k), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * factor * w[i];
}

// The lane's pair of the rotary key, turned.
__device__ __forceinline__ float2 turned(const AppendParams& p, uint32_t pe, int64_t pos, int lane) {
    const float a = bf16_lo(pe), b = bf16_hi(pe);
    if (!p.steps) return make_float2(a, b);
    const float2 cs = rope_cos_sin(pos, __ldg(p.steps + lane), p.mscale);
    return make_float2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

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
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// The page of table column pi of request b, or -1 (outside the pool or the row).
__device__ __forceinline__ int64_t a_page(const AppendParams& p, int b, int64_t pi) {
    if (pi < 0 || pi >= p.bt_cols) return -1;
    const int64_t page = __ldg(p.block_table + static_cast<int64_t>(b) * p.bt_stride + pi);
    return page >= 0 && (page + 1) * p.page_size <= p.num_slots ? page : -1;
}

template <int KIND, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= p.total) return;
    Raw<D> raw;
    load_raw<D>(p, t, lane, raw);
    // the request: the last b with cu[b] <= t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a_cu(p, mid) <= t) lo = mid;
        else hi = mid;
    }
    const int b = lo, c0 = a_cu(p, b), c1 = a_cu(p, b + 1);
    if (t < c0 || t >= c1) return;  // a row that no request names
    const int64_t place = static_cast<int64_t>(max(__ldg(p.seq_lens + b), 0)) - c1 + t;
    const int64_t page = place >= 0 ? a_page(p, b, place / p.page_size) : -1;
    const int64_t pos = p.positions ? __ldg(p.positions + t) : place;
    if (page < 0 && lane == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    const float factor = norm_factor<D>(p, raw);
    const float2 pe = turned(p, raw.pe, pos, lane);
    constexpr int row_bytes = KIND == MLA_CACHE_FP8_DS_MLA_656 ? kRowFp8 : 2 * (D + kP);
    uint8_t* row = p.cache + (page * p.page_size + place % p.page_size) * row_bytes;
    __nv_bfloat16* dense = p.rows ? p.rows + t * p.rows_st : nullptr;
#pragma unroll
    for (int k = 0; k < Raw<D>::kU; ++k) {
        float f[8];
        latent8<D>(p, raw, k, lane, factor, f);
        if (dense || KIND == MLA_CACHE_BF16_576) {
            const uint4 v = pack8(f);
            if (dense) reinterpret_cast<uint4*>(dense)[lane + 32 * k] = v;
            if (KIND == MLA_CACHE_BF16_576 && page >= 0) reinterpret_cast<uint4*>(row)[lane + 32 * k] = v;
        }
        if constexpr (KIND == MLA_CACHE_FP8_DS_MLA_656) {
            // lanes 0..15 hold block 2k, 16..31 block 2k + 1
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], scale);
            if (page >= 0) {
                reinterpret_cast<uint2*>(row)[lane + 32 * k] =
                    make_uint2(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]));
                if ((lane & 15) == 0) reinterpret_cast<float*>(row + kD)[2 * k + (lane >> 4)] = scale;
            }
        }
    }
    if (dense) store_pe(p, dense + D, pe, lane);
    if (page >= 0) store_pe(p, row + (KIND == MLA_CACHE_FP8_DS_MLA_656 ? kD + 16 : 2 * D), pe, lane);
}

// ------------------------------------------------------------------ page rows

constexpr int kHold = 8;  // new tokens of a page that a warp keeps in registers

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
__global__ void __launch_bounds__(32 * kAppendWarps) append_page_kernel(const AppendParams p) {
    constexpr int kItems = kAppendWarps / W;  // pages a CTA
    __shared__ float tops[kAppendWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % W, grp = warp / W;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kItems + grp;
    const int ps = p.page_size;
    auto first_item = [&](int b) { return static_cast<int64_t>(a_cu(p, b) / ps) + 2 * static_cast<int64_t>(b); };
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_item(mid) <= item) lo = mid;
        else hi = mid;
    }
    const int b = lo, c0 = a_cu(p, b), n = a_cu(p, b + 1) - c0;
    if (n <= 0) return;  // (the whole group leaves)
    // places p0 .. p1 - 1 are new; those below 0 have none
    const int64_t p1 = max(__ldg(p.seq_lens + b), 0), p0 = p1 - n;
    const int64_t pi = max(p0, static_cast<int64_t>(0)) / ps + (item - first_item(b));
    const bool none = p0 < 0 && item == first_item(b);  // this item also sees to the tokens without a place
    if (none && lane == 0 && wi == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    int64_t j0 = max(pi * ps, max(p0, static_cast<int64_t>(0)));
    const int64_t j1 = min((pi + 1) * ps, p1);
    if (none) j0 = p0;
    if (j0 >= j1) return;
    const int64_t t0 = c0 + (j0 - p0);  // the first token's row
    const int m = static_cast<int>(j1 - j0);
    // the token at index x of the item, 0 <= x < m, is warp x % W's
    Raw<kD> raw[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k)
        if (wi + k * W < m) load_raw<kD>(p, t0 + wi + k * W, lane, raw[k]);
    const int64_t page = a_page(p, b, pi);
    const bool bad = page < 0 && j1 > max(pi * ps, static_cast<int64_t>(0));
    if (bad && lane == 0 && wi == 0 && p.status) atomicOr(p.status, kErrBadBlock);
    const int64_t off = max(p0, static_cast<int64_t>(0)) - pi * ps;  // rows of the page that were there before (if > 0)
    const float old = page >= 0 && off > 0 ? __ldcg(p.scales + page) : 0.f;
    float factor[kHold];
    float2 pe[kHold];
    float top = 0.f;
    auto position = [&](int x) -> int64_t { return p.positions ? __ldg(p.positions + t0 + x) : j0 + x; };
    auto largest = [&](const Raw<kD>& r, float fac, float2 e, int x) {
        if (j0 + x < 0) return;
        top = fmaxf(top, fmaxf(finite_abs(e.x), finite_abs(e.y)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float f[8];
            latent8<kD>(p, r, u, lane, fac, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(f[i]));
        }
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int x = wi + k * W;
        if (x < m) {
            factor[k] = norm_factor<kD>(p, raw[k]);
            pe[k] = turned(p, raw[k].pe, position(x), lane);
            largest(raw[k], factor[k], pe[k], x);
        }
    }
    for (int x = wi + kHold * W; x < m; x += W) {  // pages of more rows than the warps hold: read twice
        Raw<kD> r;
        load_raw<kD>(p, t0 + x, lane, r);
        largest(r, norm_factor<kD>(p, r), turned(p, r.pe, position(x), lane), x);
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
                uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw h01 = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xFFFFu), __NV_E4M3);
                    const __half2_raw h23 = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h23));
                    w[i] = codes4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
                }
                reinterpret_cast<uint4*>(rows)[u] = v;
            }
        }
        if (lane == 0 && wi == 0 && scale != old) p.scales[page] = scale;
    }
    const float inv = 1.f / scale;  // exact: a power of two
    auto write = [&](const Raw<kD>& r, float fac, float2 e, int x) {
        const bool put = page >= 0 && j0 + x >= 0;
        __nv_bfloat16* dense = p.rows ? p.rows + (t0 + x) * p.rows_st : nullptr;
        uint8_t* row = p.cache + (page * ps + (j0 + x - pi * ps)) * static_cast<int64_t>(kRowPage);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float f[8];
            latent8<kD>(p, r, u, lane, fac, f);
            if (dense) reinterpret_cast<uint4*>(dense)[lane + 32 * u] = pack8(f);
            if (put)
                reinterpret_cast<uint2*>(row)[lane + 32 * u] =
                    make_uint2(codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                               codes4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
        }
        if (dense) store_pe(p, dense + kD, e, lane);
        if (put) {
            const uint32_t v = codes4(e.x * inv, e.y * inv, 0.f, 0.f);
            if (p.interleaved) {
                reinterpret_cast<unsigned short*>(row + kD)[lane] = static_cast<unsigned short>(v);
            } else {
                row[kD + lane] = static_cast<uint8_t>(v);
                row[kD + 32 + lane] = static_cast<uint8_t>(v >> 8);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int x = wi + k * W;
        if (x < m) write(raw[k], factor[k], pe[k], x);
    }
    for (int x = wi + kHold * W; x < m; x += W) {
        Raw<kD> r;
        load_raw<kD>(p, t0 + x, lane, r);
        write(r, norm_factor<kD>(p, r), turned(p, r.pe, position(x), lane), x);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int kind, int lat_dim, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    if (kind == MLA_CACHE_FP8_PAGE_576) {
        const int W = p.page_size <= 8 ? 1 : p.page_size <= 16 ? 2 : p.page_size <= 32 ? 4 : 8;
        const int64_t items = p.total / p.page_size + 2 * static_cast<int64_t>(p.B);
        const int64_t blocks = (items + kAppendWarps / W - 1) / (kAppendWarps / W);
        cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), 32 * kAppendWarps, 0, stream, attr);
        return W == 1   ? cudaLaunchKernelEx(&cfg, append_page_kernel<1>, p)
               : W == 2 ? cudaLaunchKernelEx(&cfg, append_page_kernel<2>, p)
               : W == 4 ? cudaLaunchKernelEx(&cfg, append_page_kernel<4>, p)
                        : cudaLaunchKernelEx(&cfg, append_page_kernel<8>, p);
    }
    const int64_t blocks = (p.total + kAppendWarps - 1) / kAppendWarps;
    cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), 32 * kAppendWarps, 0, stream, attr);
    if (kind == MLA_CACHE_FP8_DS_MLA_656) return cudaLaunchKernelEx(&cfg, append_kernel<MLA_CACHE_FP8_DS_MLA_656, 512>, p);
    return lat_dim == 256   ? cudaLaunchKernelEx(&cfg, append_kernel<MLA_CACHE_BF16_576, 256>, p)
           : lat_dim == 512 ? cudaLaunchKernelEx(&cfg, append_kernel<MLA_CACHE_BF16_576, 512>, p)
           : lat_dim == 768 ? cudaLaunchKernelEx(&cfg, append_kernel<MLA_CACHE_BF16_576, 768>, p)
                            : cudaLaunchKernelEx(&cfg, append_kernel<MLA_CACHE_BF16_576, 1792>, p);
}

}  // namespace mla
