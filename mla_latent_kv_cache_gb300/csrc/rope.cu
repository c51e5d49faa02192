// Rotary positions (mla_rope): every pair (a, b) of a head's rotary part
// becomes (a cos - b sin, a sin + b cos) * mscale, in 32 bits, rounded once.
//
// Bound: HBM for prompts (each value is read and written once), launch latency
// for steps. A cosine and sine cost as much as rotating eight pairs, so a warp
// takes one token and some of its heads, its lanes form each angle once, and
// the values go through shared memory. A lane holds 16 values of a head in
// 16-byte vectors placed so that neighbouring lanes read neighbouring vectors
// (of both halves, or of the interleaved pairs).
// Measured: 64 of 192 values of 16 heads for 32,768 tokens 24.8 us (5.4 TB/s, 0.80 of
// the copy rate; 0.86 where the heads lie packed), 4,099 tokens of 20 fp32 heads 8.5 us
// (0.73), 64 tokens 1.7 us. Value by value (rope_any_kernel), 32,768 tokens of 16 heads:
// 24 values a head 29 us (floor 7.4), 64 values of 193-wide heads 81 us (floor 19.8).
#include <algorithm>

#include "launch.cuh"
#include "mla_common.cuh"
#include "rope.cuh"

namespace mla {

namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeMostPairs = 128;  // of the vector kernel's table

template <typename E>
struct Vec {  // 16 bytes
    static constexpr int kN = 16 / sizeof(E);
    uint4 raw;
    __device__ __forceinline__ void unpack(float (&f)[kN]) const {
        if constexpr (kN == 4) {
            f[0] = __uint_as_float(raw.x);
            f[1] = __uint_as_float(raw.y);
            f[2] = __uint_as_float(raw.z);
            f[3] = __uint_as_float(raw.w);
        } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[kN]) {
        if constexpr (kN == 4) {
            raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        } else {
            raw = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                             pack_bf16x2(f[6], f[7]));
        }
    }
};

// R a multiple of 16, at most 256; 16-byte aligned bases and strides. Warp
// w of token t takes heads of chunk w % chunks, `per` lanes' worth at a time.
template <typename E, bool INTER>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeParams p) {
    constexpr int N = Vec<E>::kN, NV = 16 / N;  // values a vector, vectors a lane
    __shared__ alignas(16) float2 table[kRopeWarps][kRopeMostPairs];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, wl = threadIdx.x >> 5;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + wl;
    const int64_t t = w / p.chunks;
    if (t >= p.T) return;
    const int chunk = static_cast<int>(w - t * p.chunks);
    const int lph = p.R / 16;  // lanes a head
    const int items = p.H * lph;
    const int i0 = static_cast<int>(static_cast<int64_t>(chunk) * p.items_chunk);
    const int i1 = min(items, i0 + p.items_chunk);
    const E* xt = static_cast<const E*>(p.x) + t * p.x_t;
    E* ot = static_cast<E*>(p.out) + t * p.o_t;
    // the head's unit of 16 bytes that is lane o's vector v; half layout: the
    // first NV / 2 are of the first half, the others their partners
    const int half_units = p.R / (2 * N);
    auto unit = [&](int o, int v) {
        if (INTER) return o + v * lph;
        return NV == 2 ? o + v * half_units : o + (v & 1) * lph + (v >> 1) * half_units;
    };
    Vec<E> a[NV];
    // item it is lane o of head h; the warp's next 32 items on
    const int first = i0 + lane, step_h = 32 / lph, step_o = 32 - step_h * lph;
    auto next = [&](int& h, int& o) {
        h += step_h;
        o += step_o;
        if (o >= lph) {
            o -= lph;
            ++h;
        }
    };
    auto load = [&](int h, int o) {
        const E* src = xt + static_cast<int64_t>(h) * p.x_h;
#pragma unroll
        for (int v = 0; v < NV; ++v) a[v].raw = reinterpret_cast<const uint4*>(src)[unit(o, v)];
    };
    int h = first / lph, o = first - h * lph;
    if (first < i1) load(h, o);
    const int64_t pos = __ldg(p.positions + t);
    for (int i = lane; i < p.R / 2; i += 32) table[wl][i] = rope_cos_sin(pos, __ldg(p.steps + i), p.mscale);
    __syncwarp();
    for (int it = first; it < i1; it += 32) {
        E* dst = ot + static_cast<int64_t>(h) * p.o_h;
        Vec<E> y[NV];
        if constexpr (INTER) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[N];
                a[v].unpack(f);
                const float2* cs = &table[wl][unit(o, v) * (N / 2)];
#pragma unroll
                for (int k = 0; k < N / 2; ++k) {
                    const float2 r = cs[k];
                    const float u = f[2 * k], q = f[2 * k + 1];
                    f[2 * k] = u * r.x - q * r.y;
                    f[2 * k + 1] = u * r.y + q * r.x;
                }
                y[v].pack(f);
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV / 2; ++v) {
                float f[N], g[N];
                a[v].unpack(f);
                a[v + NV / 2].unpack(g);
                const float2* cs = &table[wl][unit(o, v) * N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float2 r = cs[k];
                    const float u = f[k], q = g[k];
                    f[k] = u * r.x - q * r.y;
                    g[k] = u * r.y + q * r.x;
                }
                y[v].pack(f);
                y[v + NV / 2].pack(g);
            }
        }
        const int o_now = o;
        next(h, o);
        if (it + 32 < i1) load(h, o);
#pragma unroll
        for (int v = 0; v < NV; ++v) reinterpret_cast<uint4*>(dst)[unit(o_now, v)] = y[v].raw;
    }
}

// Any even R and any alignment: a lane a pair at a time, value by value.
template <typename E>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_any_kernel(const RopeParams p) {
    __shared__ float2 table[kRopeWarps][kRopeMostPairs];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, wl = threadIdx.x >> 5, half = p.R / 2;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + wl;
    const int64_t t = w / p.chunks;
    if (t >= p.T) return;
    const int i0 = static_cast<int>(w - t * p.chunks) * p.items_chunk, i1 = min(p.H * half, i0 + p.items_chunk);
    const int64_t pos = __ldg(p.positions + t);
    for (int k = lane; k < min(half, kRopeMostPairs); k += 32) table[wl][k] = rope_cos_sin(pos, __ldg(p.steps + k), p.mscale);
    __syncwarp();
    const E* xt = static_cast<const E*>(p.x) + t * p.x_t;
    E* yt = static_cast<E*>(p.out) + t * p.o_t;
    for (int i = i0 + lane; i < i1; i += 32) {
        const int h = i / half, k = i - h * half;
        const float2 cs = k < kRopeMostPairs ? table[wl][k] : rope_cos_sin(pos, __ldg(p.steps + k), p.mscale);
        const E* x = xt + static_cast<int64_t>(h) * p.x_h;
        E* y = yt + static_cast<int64_t>(h) * p.o_h;
        const int ia = p.interleaved ? 2 * k : k, ib = p.interleaved ? 2 * k + 1 : k + half;
        const float a = static_cast<float>(x[ia]), b = static_cast<float>(x[ib]);
        y[ia] = static_cast<E>(a * cs.x - b * cs.y);
        y[ib] = static_cast<E>(a * cs.y + b * cs.x);
    }
}

template <typename E>
cudaError_t launch(RopeParams& p, int sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    const int64_t n = 16 / sizeof(E);
    auto aligned = [&](const void* base, int64_t st, int64_t sh) {
        return reinterpret_cast<uintptr_t>(base) % 16 == 0 && st % n == 0 && sh % n == 0;
    };
    const bool any = p.R % 16 || p.R > 2 * kRopeMostPairs || !aligned(p.x, p.x_t, p.x_h) || !aligned(p.out, p.o_t, p.o_h);
    // a token's heads are shared out between as many warps as fill the GPU twice
    const int64_t items = static_cast<int64_t>(p.H) * (any ? p.R / 2 : p.R / 16);
    const int64_t turns = (items + 31) / 32;
    const int64_t want = std::min((static_cast<int64_t>(sms) * 32 + p.T - 1) / p.T, turns);
    const int64_t per = (turns + want - 1) / want;
    p.items_chunk = static_cast<int>(per * 32);
    p.chunks = static_cast<int>((turns + per - 1) / per);
    const int64_t blocks = (p.T * p.chunks + kRopeWarps - 1) / kRopeWarps;
    cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), 32 * kRopeWarps, 0, stream, attr);
    if (any) return cudaLaunchKernelEx(&cfg, rope_any_kernel<E>, p);
    return p.interleaved ? cudaLaunchKernelEx(&cfg, rope_kernel<E, true>, p)
                         : cudaLaunchKernelEx(&cfg, rope_kernel<E, false>, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int f32, int sms, cudaStream_t stream) {
    return f32 ? launch<float>(p, sms, stream) : launch<__nv_bfloat16>(p, sms, stream);
}

}  // namespace mla
