// Attention over whole prompts (mla_prefill): packed sequences of different
// lengths, causal, grouped heads, one rotary key shared by all heads, with
// tcgen05 products on sm_103a.
//
// Mathematics. Query t of a sequence (one head) sees keys 0 .. Lk - Lq + t:
//   s_j = scale * (q[0:128] . k_nope_j + q[128:192] . k_pe_j)
//   out = sum_j softmax_j(s) v_j,   lse = ln sum_j exp(s_j)
// in one pass over the keys with a running maximum m and sum l. m moves only
// when a score passes it by more than 2^8, so rescaling O is rare and the
// probabilities stay below 2^8; they are rounded to bf16 for the product with
// V (relative 2^-8 each, the same as the output's own rounding), while l sums
// them unrounded in fp32.
//
// Bound: the tensor cores. 640 flop per query, key and head against 2 (192 +
// 128) bytes per key and head shared by 256 queries: far past the ridge for
// prompts. A CTA takes 256 queries of one head as two tiles of 128 rows, each
// with its own warpgroup of softmax threads, so that one tile's products run
// while the other's probabilities are formed:
//   S_i = Q_i K^T   128 x 128 x 192, Q and K from shared memory, into TMEM
//   P_i             thread = row: no exchange between threads; bf16, written
//                   over S_i in TMEM, where it is the next product's A operand
//   O_i += P_i V    128 x 128 x 128, into TMEM
// TMEM: S_0, S_1, O_0, O_1 of 128 columns each = all 512. Shared memory: Q
// 96 KB, and a ring of eight 16-KB blocks (64 dims of 128 tokens) through which
// K (two blocks of k_nope, one of k_pe) and V (two) stream by TMA.
//
// Keys past a sequence's end and masked ones have probability 0, which keeps
// finite values of theirs out of the sums. A NaN or infinity there would still
// spread (0 times it is NaN), so a row whose O comes out non-finite is formed
// again by its warp from the keys that it sees alone.
#include <climits>

#include "launch.cuh"
#include "mla_common.cuh"

namespace mla {

namespace {

constexpr int kQT = 128;                  // rows of a query tile
constexpr int kKT = 128;                  // keys of a tile
constexpr int kBlkP = 128 * 128;          // a block: 64 dims of 128 tokens
constexpr int kSlots = 8;
constexpr int kDv = 128;
constexpr int kThreadsP = 320;            // 8 softmax warps, the MMA issuer, the loader
constexpr int kQBytesP = 2 * 3 * kBlkP;
constexpr int kSmemP = 1024 + 1024 + kQBytesP + kSlots * kBlkP;
constexpr float kRaise = 8.f;             // log2 units

struct PCtrl {
    uint64_t q_full[2], blk_full[kSlots], blk_empty[kSlots];
    uint64_t s_full[2], p_full[2], o_full[2], fin;
    uint32_t tmem_base;
    int abort;
    int b, qt;  // this CTA's sequence (-1: none) and pair of query tiles
};
static_assert(sizeof(PCtrl) <= 1024, "control block");

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}

__device__ __forceinline__ void p_fail(const PrefillParams& p, PCtrl* c) {
    if (p.status) atomicOr(p.status, kErrWaitTimeout);
    *const_cast<volatile int*>(&c->abort) = 1;
}

// A sequence's first row and its rows, of prefix sums clamped to [0, total].
__device__ __forceinline__ int2 p_span(const int32_t* cu, int b, int total) {
    const int a = min(max(__ldg(cu + b), 0), total), e = min(max(__ldg(cu + b + 1), 0), total);
    return make_int2(a, max(e - a, 0));
}

// The s-th pair of query tiles of all sequences, the last pairs (which see the
// most keys) first: a whole warp. b = -1 if there are fewer.
__device__ __forceinline__ void p_locate(const PrefillParams& p, int64_t s, int lane, int& b, int& qt) {
    auto pairs = [&](int i) { return i < p.B ? (p_span(p.cu_q, i, p.total_q).y + 2 * kQT - 1) / (2 * kQT) : 0; };
    const int mine = pairs(lane);  // of the first 32 sequences
    int top = 0;
    for (int base = 0; base < p.B; base += 32) top = max(top, base == 0 ? mine : pairs(base + lane));
    top = __reduce_max_sync(0xffffffffu, top);
    auto from = [&](int q) -> int64_t {  // pairs with index >= q
        int64_t n = 0;
        for (int base = 0; base < p.B; base += 32)
            n += __reduce_add_sync(0xffffffffu, max(0, (base == 0 ? mine : pairs(base + lane)) - q));
        return n;
    };
    b = -1;
    qt = 0;
    if (from(0) <= s) return;
    int lo = 0, hi = top;  // from(lo) > s, from(hi) = 0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from(mid) > s) lo = mid;
        else hi = mid;
    }
    int64_t r = s - from(lo + 1);
    for (int base = 0; base < p.B; base += 32) {
        unsigned m = __ballot_sync(0xffffffffu, (base == 0 ? mine : pairs(base + lane)) > lo);
        const int n = __popc(m);
        if (r < n) {
            for (; r > 0; --r) m &= m - 1;
            b = base + __ffs(m) - 1;
            break;
        }
        r -= n;
    }
    qt = lo;
}

// A row again from the keys that it sees alone, by its whole warp (q of the
// row and V of a visible key may be non-finite, and then so is the row).
__device__ __noinline__ void p_row_again(const PrefillParams& p, int64_t qrow, int h, int hk, int64_t k0, int vis,
                                         float m2, float inv_l, int lane) {
    const __nv_bfloat16* q = p.q + qrow * p.q_st + h * p.q_sh;
    float qv[6], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 6; ++i) qv[i] = __bfloat162float(q[lane + 32 * i]);
    for (int j = 0; j < vis; ++j) {
        const int64_t kr = k0 + j;
        const __nv_bfloat16* kn = p.k_nope + kr * p.k_st + hk * p.k_sh;
        const __nv_bfloat16* kp = p.k_pe + kr * p.kp_st;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(qv[i], __bfloat162float(kn[lane + 32 * i]), s);
#pragma unroll
        for (int i = 0; i < 2; ++i) s = fmaf(qv[4 + i], __bfloat162float(kp[lane + 32 * i]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float w = ex2(fmaf(s, p.scale_log2, -m2)) * inv_l;
        const __nv_bfloat16* v = p.v + kr * p.v_st + hk * p.v_sh;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(w, __bfloat162float(v[lane + 32 * i]), acc[i]);
    }
    __nv_bfloat16* o = p.out + (qrow * p.Hq + h) * kDv;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[lane + 32 * i] = __float2bfloat16(acc[i]);
}

__global__ void __launch_bounds__(kThreadsP, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps maps, const __grid_constant__ PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    PCtrl* ctrl = reinterpret_cast<PCtrl*>(smem);
    uint8_t* qs = smem + 1024;
    uint8_t* ring = qs + kQBytesP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.Hq, hk = h / (p.Hq / p.Hkv);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->q_full[i], 1);
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->p_full[i], 4);
            mbar_init(&ctrl->o_full[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ctrl->blk_full[i], 1);
            mbar_init(&ctrl->blk_empty[i], 1);
        }
        mbar_init(&ctrl->fin, 1);
        ctrl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == 9) {
        int b, qt;
        p_locate(p, blockIdx.x / p.Hq, lane, b, qt);
        if (lane == 0) {
            ctrl->b = b;
            ctrl->qt = qt;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    volatile int* abort = &ctrl->abort;
    const int b = ctrl->b;
    if (b >= 0) {
        const int2 sq = p_span(p.cu_q, b, p.total_q), sk = p_span(p.cu_k, b, p.total_k);
        const int t0 = ctrl->qt * 2 * kQT;
        // keys that row t sees, and a tile's number of key tiles
        auto seen = [&](int t) { return p.causal ? min(sk.y, max(0, sk.y - sq.y + t + 1)) : sk.y; };
        int n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rows = min(kQT, sq.y - t0 - i * kQT);
            n[i] = rows > 0 ? (seen(t0 + i * kQT + rows - 1) + kKT - 1) / kKT : 0;
        }
        const int nk = max(n[0], n[1]);

        if (warp == 9) {
            if (lane == 0) {
                // ---------------------------------------------------- loader
                uint32_t u = 0;
                bool ok = true;
                auto load_q = [&](int i) {
                    if (n[i] == 0) return;
                    mbar_arrive_expect_tx(&ctrl->q_full[i], 3 * kBlkP);
                    for (int c = 0; c < 3; ++c)
                        tma_load_3d(qs + (i * 3 + c) * kBlkP, &maps.q, &ctrl->q_full[i], 64 * c, h, sq.x + t0 + i * kQT);
                };
                load_q(0);
                for (int j = 0; j < nk && ok; ++j) {
                    for (int x = 0; x < 5; ++x, ++u) {
                        const uint32_t slot = u % kSlots;
                        if (u >= kSlots && !mbar_wait(&ctrl->blk_empty[slot], ((u / kSlots) - 1) & 1, abort)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&ctrl->blk_full[slot], kBlkP);
                        uint8_t* dst = ring + slot * kBlkP;
                        const int kr = sk.x + j * kKT;
                        if (x < 2) tma_load_3d(dst, &maps.k_nope, &ctrl->blk_full[slot], 64 * x, hk, kr);
                        else if (x == 2) tma_load_3d(dst, &maps.k_pe, &ctrl->blk_full[slot], 0, 0, kr);
                        else tma_load_3d(dst, &maps.v, &ctrl->blk_full[slot], 64 * (x - 3), hk, kr);
                        if (u == 2) load_q(1);
                    }
                }
                if (!ok) {
                    p_fail(p, ctrl);
                    // no copy may arrive after the CTA is gone
                    volatile int never = 0;
                    for (uint32_t v = u < kSlots ? 0 : u - kSlots; v < u; ++v)
                        mbar_wait(&ctrl->blk_full[v % kSlots], (v / kSlots) & 1, &never);
                    for (int i = 0; i < 2; ++i)
                        if (n[i]) mbar_wait(&ctrl->q_full[i], 0, &never);
                }
            }
        } else if (warp == 8) {
            // ---------------------------------------------------- MMA issuer
            // The whole warp walks the loop and one lane issues: descriptors are
            // then warp-uniform values, which the instruction takes from uniform
            // registers (formed by a single lane they cost a move each per product).
            const bool leader = elect_lane();
            const uint32_t idS = idesc_bf16(128, 128, false, false), idPV = idesc_bf16(128, 128, false, true),
                           idPVh = idesc_bf16(128, 64, false, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const int n0 = __shfl_sync(0xffffffffu, n[0], 0), n1 = __shfl_sync(0xffffffffu, n[1], 0);
            const uint64_t dQ = smem_desc(smem_u32(qs), 16, 1024, kSw128);
            const uint64_t dK = smem_desc(smem_u32(ring), 16, 1024, kSw128);
            const uint64_t dV = smem_desc(smem_u32(ring), kBlkP, 1024, kSw128);
            constexpr uint32_t kBlkD = kBlkP >> 4;
            bool ok = true;
            auto wait_blk = [&](uint32_t u) {
                if (ok && !mbar_wait(&ctrl->blk_full[u % kSlots], (u / kSlots) & 1, abort)) ok = false;
            };
            auto scores = [&](int i, int j) {
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const uint32_t u = 5 * j + c;
                    wait_blk(u);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t da = dQ + (i * 3 + c) * kBlkD, db = dK + (u % kSlots) * kBlkD;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) umma_bf16(tm + i * 128, da + 2 * kk, db + 2 * kk, idS, (c | kk) != 0);
                    }
                }
                if (leader) {
                    umma_commit(&ctrl->s_full[i]);
                    if (i == 1 || j >= n1)
                        for (int c = 0; c < 3; ++c) umma_commit(&ctrl->blk_empty[(5 * j + c) % kSlots]);
                }
            };
            auto values = [&](int i, int j) {
                const uint32_t u = 5 * j + 3;
                wait_blk(u);
                wait_blk(u + 1);
                if (!ok) return;
                tc_fence_after();
                const uint32_t s0 = u % kSlots, s1 = (u + 1) % kSlots;
                const uint64_t d0 = dV + s0 * kBlkD, d1 = dV + s1 * kBlkD;
                const uint32_t tO = tm + 256 + i * 128, tP = tm + i * 128;
                if (leader) {
                    if (s1 == s0 + 1) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16_ta(tO, tP + 8 * kk, d0 + kk * (2048 >> 4), idPV, (j | kk) != 0);
                    } else {  // the two blocks are the ring's last and first
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            umma_bf16_ta(tO, tP + 8 * kk, d0 + kk * (2048 >> 4), idPVh, (j | kk) != 0);
                            umma_bf16_ta(tO + 64, tP + 8 * kk, d1 + kk * (2048 >> 4), idPVh, (j | kk) != 0);
                        }
                    }
                    if (i == 1 || j >= n1) {
                        umma_commit(&ctrl->blk_empty[s0]);
                        umma_commit(&ctrl->blk_empty[s1]);
                    }
                }
            };
            auto step = [&](int i, int j, int ni) {  // P_i(j) V, then the scores of the next key tile
                if (!ok || j >= ni) return;
                if (!mbar_wait(&ctrl->p_full[i], j & 1, abort)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                values(i, j);
                if (!ok) return;
                // in order behind the product that reads P_i from the same columns
                if (j + 1 < ni) scores(i, j + 1);
                else if (leader) umma_commit(&ctrl->o_full[i]);
            };
            if (n0 && !mbar_wait(&ctrl->q_full[0], 0, abort)) ok = false;
            if (ok && n0) scores(0, 0);
            if (ok && n1 && !mbar_wait(&ctrl->q_full[1], 0, abort)) ok = false;
            if (ok && n1) scores(1, 0);
            const int most = max(n0, n1);
            for (int j = 0; j < most && ok; ++j) {
                step(0, j, n0);
                step(1, j, n1);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (leader) {
                if (!ok) p_fail(p, ctrl);
                drain_mma(&ctrl->fin);
            }
        } else {
            // ------------------------------------------------------- softmax
            const int i = warp >> 2;
            const int row = (warp & 3) * 32 + lane, t = t0 + i * kQT + row;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + i * 128 + lanes, tO = tmem + 256 + i * 128 + lanes;
            const int vis = seen(t);  // keys 0 .. vis - 1
            float m = -INFINITY, l = 0.f;  // m in log2 units
            bool ok = true;
            const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
            for (int j = 0; j < n[i] && ok; ++j) {
                if (!__all_sync(0xffffffffu, mbar_wait(&ctrl->s_full[i], j & 1, abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[128];
                tmem_ld_x64(tS, *reinterpret_cast<uint32_t(*)[64]>(s));
                tmem_ld_x64(tS + 64, *reinterpret_cast<uint32_t(*)[64]>(s + 64));
                const int left = vis - j * kKT;  // visible keys of this tile
                if (__any_sync(0xffffffffu, left < kKT)) {
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k >= left) s[k] = 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 128; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(s[k]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                const bool raise = top > m + kRaise || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, raise)) {
                    const float to = raise ? top : m;
                    const float a = raise ? (m > -INFINITY ? ex2(m - to) : 0.f) : 1.f;
                    l *= a;
                    m = to;
                    if (j > 0) {
                        // S_i(j) follows the product with P_i(j - 1), so O_i is at rest
#pragma unroll
                        for (int c = 0; c < 128; c += 32) {
                            uint32_t o[32];
                            tmem_ld_x32(tO + c, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                            tmem_st_x32(tO + c, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t nb = pack2(-base, -base);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t x = fma2(pack2(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1])), c2, nb);
                        float x0, x1;
                        unpack2(x, x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum[k & 1] = add2(sum[k & 1], pack2(x0, x1));
                        pk[k] = pack_bf16x2(x0, x1);
                    }
                    tmem_st_x16(tS + 16 * c, pk);
                }
                float a0, a1;
                unpack2(add2(sum[0], sum[1]), a0, a1);
                l += a0 + a1;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctrl->p_full[i]);
            }
            // ------------------------------------------------------ epilogue
            if (ok && n[i] > 0 && !__all_sync(0xffffffffu, mbar_wait(&ctrl->o_full[i], 0, abort))) ok = false;
            if (!ok && lane == 0) p_fail(p, ctrl);
            if (ok) {
                tc_fence_after();
                const bool mine = t < sq.y;
                const int64_t qrow = sq.x + t;
                const float inv = l > 0.f ? 1.f / l : l;  // l = 0: nothing seen; NaN: the row is NaN
                __nv_bfloat16* o = p.out + (qrow * p.Hq + h) * kDv;
                bool fine = true;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t v[32];
                    if (n[i] > 0) {
                        tmem_ld_x32(tO + c, v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0u;
                    }
                    if (vis <= 0) {  // sees nothing, beside rows that do
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            f[e] = __uint_as_float(v[k + e]) * inv;
                            fine = fine && fabsf(f[e]) <= 3.0e38f;
                        }
                        if (mine)
                            *reinterpret_cast<uint4*>(o + c + k) =
                                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                           pack_bf16x2(f[6], f[7]));
                    }
                }
                if (mine) p.lse[qrow * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
                // rows to form again: O is not finite though the sums are
                unsigned again = __ballot_sync(0xffffffffu, mine && !fine && l > 0.f && l < INFINITY && fabsf(m) < INFINITY);
                while (again) {
                    const int r = __ffs(again) - 1;
                    again &= again - 1;
                    __syncwarp();
                    p_row_again(p, __shfl_sync(0xffffffffu, qrow, r), h, hk, sk.x, __shfl_sync(0xffffffffu, vis, r),
                                __shfl_sync(0xffffffffu, m, r), __shfl_sync(0xffffffffu, inv, r), lane);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_prefill(const PrefillMaps& maps, const PrefillParams& p, cudaStream_t stream) {
    // sum of ceil(len / 256) <= total / 256 + B
    const int64_t pairs = static_cast<int64_t>(p.total_q) / (2 * kQT) + p.B;
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemP);
    if (e != cudaSuccess) return e;
    prefill_kernel<<<dim3(static_cast<unsigned>(pairs * p.Hq)), kThreadsP, kSmemP, stream>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace mla
