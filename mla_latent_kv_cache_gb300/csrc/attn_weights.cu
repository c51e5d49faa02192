// Attention received per cached token (mla_attn_weights), for a step's queries
// over the paged latent cache, with tcgen05 score products.
//
// Mathematics. With the log-sum-exp L_r that the step's decode left for query
// row r, the probability of token j is exp(s_rj - L_r), so one product and one
// exponential per pair give it without a second softmax pass:
//   w[b][j] = decay * w[b][j] + sum_r exp(scale * q_r . row_j - L_r)
// over the rows r of request b that see token j.
//
// Bound: HBM. Each cached row is read once (1152 or 656 bytes; up to 128 query
// rows share the read), 4 bytes are read and written per token, and the product
// is 1,152 flop per row and token: 16 to 128 rows are 16 to 128 flop/B, under
// the ridge of about 290. So the kernel is a stream: 128-token tiles arrive by
// TMA as 16-KB blocks (64 dims, or 128 fp8 codes, of 128 tokens) in one ring
// of all the shared memory that the queries leave, one warp issues the score
// products (tokens are the 128 rows of the A operand, query rows the columns),
// and four warps turn the scores into weights: a thread holds a token, so the
// sum over query rows stays in its registers, needs no atomics, and has one
// order whatever the grid.
//
// fp8_ds_mla rows are not widened. A bf16 query value has 8 significant bits:
// scaled by a power of two per row (so that the row's largest lies in
// [128, 256)) it is the sum of an e4m3 value (4 bits) and an e5m2 value (the
// rest, at most 8 units of its last place, so 3 bits), and the tensor cores
// multiply the e4m3 codes with both: each 128-code block has its own
// accumulator, and its fp32 scale is applied to the finished sum. Only
// elements below 2^-13 of their row's largest are rounded, by at most 2^-21 of
// it: scaled, they lie below 2^-6, where e4m3's step stays at 2^-9 and the rest
// may have more bits than e5m2. The codes go from HBM to the tensor core untouched: no conversion
// instructions, and half the shared-memory traffic of widened rows.
//
// Warp roles: 0 issues the products (and allocates TMEM), 1 and 2 load blocks
// (row by row: 3 and 12 too), 4..7 weights, 8..11 queries (shared-memory layout, and
// the split for fp8 rows) and, from 32 query rows on, the second half of the columns. With more query rows than fit beside the ring they
// are taken in groups over chunks of kChunk tiles, so that the groups after
// the first find the rows in L2.
#include <climits>
#include <type_traits>

#include "launch.cuh"
#include "mla_common.cuh"

namespace mla {

namespace {

constexpr int kTok = 128;          // tokens per tile
constexpr int kBlk = 128 * 128;    // bytes of a ring block
constexpr int kMaxSlots = 12;
constexpr int kScSlots = 4;        // fp8: tiles' block scales
constexpr int kQBufs = 4;          // generations of lse / query scales that may be in use at once
constexpr int kParts = 4;          // tiles whose second halves may be on their way
constexpr int kChunk = 8;          // tiles per turn when the query rows take several groups
constexpr int kThreads = 416;
constexpr int kLse = 128;
constexpr int kSmemLimit = 232448;
constexpr float kLog2e = 1.4426950408889634f;

struct WCtrl {
    uint64_t blk_full[kMaxSlots], blk_empty[kMaxSlots];
    uint64_t s_full[2], s_free[2];
    uint64_t q_full[kQBufs], q_empty;
    uint64_t sc_full[kScSlots], sc_empty[kScSlots];
    uint64_t part_full[kParts];
    uint64_t fin;
    uint32_t tmem_base;
    int abort;
    int n_items, b0, j0;
    alignas(16) float lse2[kQBufs][kLse];  // log-sum-exp in log2 units; +inf where a row adds nothing
    alignas(16) float qs[kQBufs][kLse];    // fp8: what undoes the row's power of two
    float part[kParts][kTok];              // sums over the second half of the columns
};
constexpr int kCtrlBytes = (sizeof(WCtrl) + 1023) / 1024 * 1024;

__device__ __forceinline__ int w_tokens(const WeightsParams& p, int b) { return max(__ldg(p.seq_lens + b), 0); }
// Tiles of the tokens whose weights are kept.
__device__ __forceinline__ int w_tiles(const WeightsParams& p, int b) {
    return static_cast<int>((static_cast<uint32_t>(min(w_tokens(p, b), p.max_len)) + kTok - 1) / kTok);
}

// The order in which every role walks this CTA's tiles: `rem` tiles from tile
// j of request b on, in chunks inside a request, each chunk once per row group.
struct Walk {
    int b, T, tiles, c0, c1, g, j, rem, q, B, groups;
    bool newq;
    __device__ __forceinline__ void chunk() {
        const int most = groups > 1 ? min(rem, kChunk) : rem;
        c1 = c0 + min(tiles - c0, most);
        j = c0;
    }
    __device__ __forceinline__ void init(const WeightsParams& p, const WCtrl* c) {
        b = c->b0;
        c0 = c->j0;
        rem = c->n_items;
        groups = p.groups;
        B = p.B;
        g = 0;
        q = 0;
        newq = true;
        T = tiles = 0;
        if (rem > 0) {
            T = w_tokens(p, b);
            tiles = w_tiles(p, b);
            chunk();
        }
    }
    __device__ __forceinline__ bool done() const { return rem <= 0; }
    __device__ __forceinline__ bool last_of_q() const {  // the queries change after this tile
        return j + 1 >= c1 && (groups > 1 || rem - (c1 - c0) <= 0 || c1 >= tiles);
    }
    __device__ __forceinline__ void next(const WeightsParams& p) {
        newq = false;
        if (++j < c1) return;
        newq = groups > 1;
        if (++g < groups) {
            j = c0;
            ++q;
            return;
        }
        g = 0;
        rem -= c1 - c0;
        c0 = c1;
        if (rem > 0 && c0 >= tiles) {
            newq = true;
            c0 = 0;
            do {
                if (++b >= B) {  // cannot happen while rem > 0 matches the lengths
                    rem = 0;
                    return;
                }
                T = w_tokens(p, b);
                tiles = w_tiles(p, b);
            } while (tiles == 0);
        }
        if (newq) ++q;
        if (rem > 0) chunk();
    }
};

__device__ __forceinline__ void w_fail(const WeightsParams& p, WCtrl* c) {
    if (p.status) atomicOr(p.status, kErrWaitTimeout);
    *const_cast<volatile int*>(&c->abort) = 1;
}

__device__ __forceinline__ int w_slot(const WeightsParams& p, int b, int tok, bool& bad) {
    const int pi = tok / p.page_size;
    int64_t page = pi < p.bt_stride ? __ldg(p.block_table + static_cast<int64_t>(b) * p.bt_stride + pi) : -1;
    if (page < 0 || (page + 1) * p.page_size > p.num_slots) {
        bad = true;
        page = 0;
    }
    const int64_t s = page * p.page_size + tok % p.page_size;
    return static_cast<int>(s < p.num_slots ? s : 0);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// bytes = 0 writes 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The request and tile of the x-th tile of all (x below the total); a whole warp.
__device__ __forceinline__ void w_locate(const WeightsParams& p, long long x, int lane, int& b, int& j) {
    long long acc = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int tl = base + lane < p.B ? w_tiles(p, base + lane) : 0;
        long long it = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) it += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, acc + it > x);
        if (hit) {
            const int L = __ffs(hit) - 1;
            b = base + L;
            j = static_cast<int>(x - (acc + __shfl_sync(0xffffffffu, it, L) - __shfl_sync(0xffffffffu, tl, L)));
            return;
        }
        acc += __shfl_sync(0xffffffffu, it, 31);
    }
    b = j = 0;
}

// KIND 0: bf16 rows of any width, 1: fp8_ds_mla. LSU: pages that are not a
// multiple of 8 rows, read row by row with cp.async.
template <int KIND, bool LSU>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_kernel(const __grid_constant__ WeightsMaps maps, const WeightsParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    WCtrl* ctrl = reinterpret_cast<WCtrl*>(smem);
    const int NP = p.np, NB = p.lat_dim / (KIND == 1 ? 128 : 64) + 1;  // the last block is the rope
    const int qblk = NP * 128;                                         // bytes of a query block
    const int n_qblk = KIND == 1 ? 2 * (NB - 1) + 1 : NB;
    uint8_t* qbuf = smem + kCtrlBytes;
    uint8_t* sc_ring = qbuf + n_qblk * qblk;
    uint8_t* ring = sc_ring + (KIND == 1 ? kScSlots * kTok * 16 : 0);
    const int NS = p.slots;
    // columns of an S buffer: fp8 rows hold five sums (four blocks and the rope);
    // two buffers where TMEM holds them (fp8: up to 48 query rows). bf16 rows: the
    // products are summed in up to four parts, which fp32 additions join, since
    // the tensor core's running sum truncates (one part was off by 2e-6 in the
    // weights; four parts 4.5e-7 to 5.1e-7 at 16 and 64 rows, and the two that
    // TMEM holds above 64 rows 5.7e-7 to 5.9e-7 at 96 and 128)
    const int sums = KIND == 1 ? 5 : NP <= 64 ? 4 : 2;
    const int buf_cols = sums * NP;
    const int nbuf = 2 * buf_cols <= 512 ? 2 : 1;
    const bool two = NP >= 32;  // two groups of warps share a tile's columns
    const int used = nbuf * buf_cols;
    const uint32_t tmem_cols = used <= 32 ? 32 : used <= 64 ? 64 : used <= 128 ? 128 : used <= 256 ? 256 : 512;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&ctrl->blk_full[i], 1);
            mbar_init(&ctrl->blk_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->s_free[i], two ? 8 : 4);
        }
        for (int i = 0; i < kQBufs; ++i) mbar_init(&ctrl->q_full[i], 4);
        mbar_init(&ctrl->q_empty, 1);
        for (int i = 0; i < kScSlots; ++i) {
            mbar_init(&ctrl->sc_full[i], 1);
            mbar_init(&ctrl->sc_empty[i], two ? 8 : 4);
        }
        for (int i = 0; i < kParts; ++i) mbar_init(&ctrl->part_full[i], 4);
        mbar_init(&ctrl->fin, 1);
        ctrl->abort = 0;
        fence_mbar_init();
    }
    if (!LSU && warp == 1 && lane == 0) {
        prefetch_tensormap(&maps.rows);
        if (KIND == 1) {
            prefetch_tensormap(&maps.rope);
            prefetch_tensormap(&maps.scales);
        }
    }
    if (warp == 0) {
        tmem_alloc(&ctrl->tmem_base, tmem_cols);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == 3) {
        // equal contiguous ranges of all requests' tiles
        long long total = 0;
        for (int base = 0; base < p.B; base += 32) total += base + lane < p.B ? w_tiles(p, base + lane) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const long long t0 = total * blockIdx.x / gridDim.x, t1 = total * (blockIdx.x + 1) / gridDim.x;
        int b = 0, j = 0;
        if (t1 > t0) w_locate(p, t0, lane, b, j);
        if (lane == 0) {
            ctrl->n_items = static_cast<int>(t1 - t0);
            ctrl->b0 = b;
            ctrl->j0 = j;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    Walk wk;
    wk.init(p, ctrl);
    volatile int* abort = &ctrl->abort;

    if (warp == 0) {
        // ------------------------------------------------------ score products
        // The whole warp walks the tiles and one lane issues: descriptors are then
        // warp-uniform values, which the instruction takes from uniform registers.
        const bool leader = elect_lane();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int buf = 0, turn = 0;            // S buffer of the next tile, and its uses before
        uint32_t slot = 0, phase = 0;     // the next block's
        bool ok = true;
        const uint32_t id_b = (1u << 7) | (1u << 10) | idesc_f8(kTok, NP, 0, 0);
        const uint32_t id_h = idesc_f8(kTok, NP, 0, 0), id_l = idesc_f8(kTok, NP, 0, 1);
        const uint64_t dR = smem_desc(smem_u32(ring), 16, 1024, kSw128), dQ = smem_desc(smem_u32(qbuf), 16, 1024, kSw128);
        const uint32_t q_step = static_cast<uint32_t>(qblk) >> 4;
        while (ok && !wk.done()) {
            if (wk.newq && !mbar_wait(&ctrl->q_full[wk.q % kQBufs], (wk.q / kQBufs) & 1, abort)) ok = false;
            if (ok && turn > 0 && !mbar_wait(&ctrl->s_free[buf], (turn - 1) & 1, abort)) ok = false;
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tm + buf * buf_cols;
            uint64_t dq = dQ;
            for (int kb = 0; kb < NB; ++kb) {
                if (!mbar_wait(&ctrl->blk_full[slot], phase, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = dR + slot * static_cast<uint32_t>(kBlk >> 4);
                const int part = KIND == 1 ? kb : kb * sums / NB;  // the sum that this block goes into
                const bool first = KIND == 1 || kb == 0 || part != (kb - 1) * sums / NB;
                if (leader) {
                    if (KIND == 1 && kb < NB - 1) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            umma_f8(tS + kb * NP, da + 2 * kk, dq + 2 * kk, id_h, kk != 0);
                            umma_f8(tS + kb * NP, da + 2 * kk, dq + q_step + 2 * kk, id_l, 1u);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tS + part * NP, da + 2 * kk, dq + 2 * kk, id_b, kk != 0 || !first);
                    }
                    umma_commit(&ctrl->blk_empty[slot]);
                }
                dq += KIND == 1 ? 2 * q_step : q_step;
                if (++slot == static_cast<uint32_t>(NS)) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (leader) {
                umma_commit(&ctrl->s_full[buf]);
                if (wk.last_of_q()) umma_commit(&ctrl->q_empty);
            }
            if (++buf == nbuf) {
                buf = 0;
                ++turn;
            }
            wk.next(p);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (leader) {
            if (!ok) w_fail(p, ctrl);
            drain_mma(&ctrl->fin);
        }
    } else if (warp == 1 || warp == 2 || (LSU && (warp == 3 || warp == 12))) {
        // ---------------------------------------------------------- blocks
        // Loader w takes every kLoaders-th block (TMA: the ring has an even number of
        // slots, so a slot always has the same loader).
        constexpr uint32_t kLoaders = LSU ? 4 : 2;
        const uint32_t me = warp == 12 ? 3 : warp - 1;
        const int BR = p.run_rows;
        const uint64_t pol = l2_policy_evict_first();
        bool ok = true, bad = false;
        uint32_t u = 0;
        int i = 0;
        uint32_t armed = 0;                  // TMA: ring slots (by bit) whose barrier this warp has armed
        uint32_t parity = 0;                 // and the parity of the last fill of each
        int sc_armed = 0;                    // TMA: tiles whose scales this warp has asked for
        uint32_t pend_slot = 0;              // LSU: the fill before, not yet handed over
        int pend = 0, pend_sc = -1, sc_new = -1;
        auto hand_over = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && pend) {
                mbar_arrive(&ctrl->blk_full[pend_slot]);
                if (pend_sc >= 0) mbar_arrive(&ctrl->sc_full[pend_sc]);
            }
            pend = 0;
        };
        // waits for a barrier; LSU: what waits behind it may need this warp's last fill first
        auto wait_empty = [&](uint64_t* bar, uint32_t parity) -> bool {
            if (LSU && pend && !__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
                cp_async_wait<0>();
                hand_over();
            }
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
        };
        int y_next = 0;
        auto run_slot = [&]() -> int {
            if (wk.done()) return 0;
            const int valid = min(kTok, min(wk.T, p.max_len) - wk.j * kTok);
            return lane * BR < valid ? w_slot(p, wk.b, wk.j * kTok + lane * BR, bad) : 0;
        };
        if (!LSU) y_next = run_slot();
        while (ok && !wk.done()) {
            const int valid = min(kTok, min(wk.T, p.max_len) - wk.j * kTok);
            const int nruns = LSU ? 0 : (valid + BR - 1) / BR;
            const int y = y_next;
            int slot4[4] = {0, 0, 0, 0}, row_slot[LSU ? 32 : 1];
            if (LSU) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (lane + 32 * q < valid) slot4[q] = w_slot(p, wk.b, wk.j * kTok + lane + 32 * q, bad);
#pragma unroll
                for (int it = 0; it < (LSU ? 32 : 1); ++it)
                    row_slot[it] = __shfl_sync(0xffffffffu, slot4[it >> 3], (it & 7) * 4 + (lane >> 3));
            }
            // this tile's block scales
            if (KIND == 1 && me == 0) {
                const int sl = i % kScSlots;
                if (i >= kScSlots && !wait_empty(&ctrl->sc_empty[sl], ((i / kScSlots) - 1) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t* dst = sc_ring + sl * kTok * 16;
                if (!LSU) {
                    if (lane == 0) mbar_arrive_expect_tx(&ctrl->sc_full[sl], nruns * BR * 16);
                    __syncwarp();
                    sc_armed = i + 1;
                    if (lane < nruns) tma_load_2d(dst + lane * BR * 16, &maps.scales, &ctrl->sc_full[sl], 512, y, pol);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (lane + 32 * q < valid)
                            cp_async16(smem_u32(dst + (lane + 32 * q) * 16),
                                       p.cache + static_cast<int64_t>(slot4[q]) * p.row_bytes + 512);
                    sc_new = sl;
                }
            }
            for (int kb = 0; kb < NB; ++kb) {
                const uint32_t v = u + kb;
                if (v % kLoaders != me) continue;
                const uint32_t slot = v % NS;
                if (v >= static_cast<uint32_t>(NS) && !wait_empty(&ctrl->blk_empty[slot], ((v / NS) - 1) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t* dst = ring + slot * kBlk;
                const bool rope = kb == NB - 1;
                if (!LSU) {
                    if (lane == 0) mbar_arrive_expect_tx(&ctrl->blk_full[slot], nruns * BR * 128);
                    __syncwarp();
                    armed |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | (((v / NS) & 1u) << slot);
                    if (lane < nruns) {
                        if (KIND == 1 && rope) tma_load_2d(dst + lane * BR * 128, &maps.rope, &ctrl->blk_full[slot], 264, y, pol);
                        else tma_load_2d(dst + lane * BR * 128, &maps.rows, &ctrl->blk_full[slot], kb * (KIND == 1 ? 128 : 64), y, pol);
                    }
                } else {
                    const int off = KIND == 1 && rope ? 528 : kb * 128;
#pragma unroll
                    for (int it = 0; it < (LSU ? 32 : 1); ++it) {
                        const int r = it * 4 + (lane >> 3), un = lane & 7;
                        if (r < valid)
                            cp_async16(smem_u32(dst + r * 128 + ((un ^ (r & 7)) << 4)),
                                       p.cache + static_cast<int64_t>(row_slot[it]) * p.row_bytes + off + un * 16);
                    }
                    cp_async_commit();
                    // the fill before this one has landed: hand it over
                    cp_async_wait<1>();
                    hand_over();
                    pend = 1;
                    pend_slot = slot;
                    // loader 0's first fill of a tile carries the tile's scales
                    pend_sc = sc_new;
                    sc_new = -1;
                }
            }
            if (!ok) break;
            u += NB;
            ++i;
            wk.next(p);
            if (!LSU) y_next = run_slot();
        }
        if (!ok && lane == 0) w_fail(p, ctrl);
        if (LSU) {
            cp_async_wait<0>();
            hand_over();
        } else {
            // no copy may arrive after the CTA is gone: wait (bounded, whatever the
            // abort flag says) for the last fill of every barrier this warp armed
            volatile int never = 0;
            for (int s = 0; s < NS; ++s)
                if (armed >> s & 1) mbar_wait(&ctrl->blk_full[s], parity >> s & 1, &never);
            for (int k = max(0, sc_armed - kScSlots); k < sc_armed; ++k)
                mbar_wait(&ctrl->sc_full[k % kScSlots], (k / kScSlots) & 1, &never);
        }
        if (bad && p.status) atomicOr(p.status, kErrBadBlock);
    } else if (warp >= 4 && warp < 12) {
        // --------------------------------------------- weights; 8..11: queries
        const int grp = warp >> 3;  // 0: warps 4..7
        const int wq = warp & 3, tk = wq * 32 + lane, D = p.lat_dim;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        // this group's columns: the first half (all, with one group) or the second
        const int half = two ? (NP / 16 + 1) / 2 * 16 : NP;
        const int cb = grp ? half : 0, ce = grp ? NP : half;
        auto load_q = [&]() {
            const int gen = wk.q % kQBufs;
            const int r0 = wk.g * NP, rows = min(NP, p.HQ - r0);
            const int64_t row0 = static_cast<int64_t>(wk.b) * p.HQ + r0;
            // everything in flight at once: a request's queries are one latency
            const uint32_t q0 = smem_u32(qbuf);
            if (KIND == 0) {
                for (int r = wq; r < NP; r += 4) {
                    const int64_t row = row0 + (r < rows ? r : 0);
                    const __nv_bfloat16 *ql = p.q_lat + row * D, *qp = p.q_pe + row * kP;
                    for (int un = lane; un < (D + kP) / 8; un += 32)
                        cp_async16_or_zero(q0 + (un >> 3) * qblk + r * 128 + (((un & 7) ^ (r & 7)) << 4),
                                           un < D / 8 ? ql + un * 8 : qp + (un * 8 - D), r < rows ? 16 : 0);
                }
            } else {
                if (lane < 8)
                    for (int r = wq; r < NP; r += 4)
                        cp_async16_or_zero(q0 + 8 * qblk + r * 128 + ((lane ^ (r & 7)) << 4),
                                           p.q_pe + (row0 + (r < rows ? r : 0)) * kP + lane * 8, r < rows ? 16 : 0);
                for (int r4 = wq; r4 < NP; r4 += 16) {  // four rows at a time; NP is a multiple of 16
                    uint4 x[4][2];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int r = r4 + 4 * n;
                        // lane holds values 16 lane .. 16 lane + 15: unit lane % 8 of block lane / 8
                        const uint4* ql = reinterpret_cast<const uint4*>(p.q_lat + (row0 + r) * D) + 2 * lane;
                        x[n][0] = r < rows ? __ldg(ql) : make_uint4(0u, 0u, 0u, 0u);
                        x[n][1] = r < rows ? __ldg(ql + 1) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int r = r4 + 4 * n;
                        const __nv_bfloat162* xb = reinterpret_cast<const __nv_bfloat162*>(x[n]);
                        float mx = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 f = __bfloat1622float2(xb[k]);
                            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                        // (non-negative floats are ordered as their bits)
                        mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
                        // the power of two that brings the largest into [128, 256)
                        const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
                        const int k2 = max(-120, min(120, 7 - e));
                        const float up = __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 f = __bfloat1622float2(xb[k]);
                            // (x - x is 0, and NaN for an infinity, which 8 bits do not hold)
                            const float2 s = make_float2(fmaf(f.x, up, f.x - f.x), fmaf(f.y, up, f.y - f.y));
                            const uint32_t hc = __nv_cvt_float2_to_fp8x2(s, __NV_SATFINITE, __NV_E4M3);
                            const __half2_raw hr =
                                __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hc), __NV_E4M3);
                            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                            const float2 d = make_float2(s.x - hf.x, s.y - hf.y);
                            const uint32_t lc = __nv_cvt_float2_to_fp8x2(d, __NV_SATFINITE, __NV_E5M2);
                            if (k & 1) {
                                h[k >> 1] |= hc << 16;
                                l[k >> 1] |= lc << 16;
                            } else {
                                h[k >> 1] = hc & 0xFFFFu;
                                l[k >> 1] = lc & 0xFFFFu;
                            }
                        }
                        uint8_t* at = qbuf + (lane >> 3) * 2 * qblk + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(at + qblk) = make_uint4(l[0], l[1], l[2], l[3]);
                        if (lane == 0) ctrl->qs[gen][r] = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23);
                    }
                }
            }
            const int own = wq * 32 + lane;
            if (own < NP) {
                const float L = own < rows ? __ldg(p.lse + row0 + own) : INFINITY;
                ctrl->lse2[gen][own] = L == -INFINITY ? INFINITY : L * kLog2e;
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctrl->q_full[gen]);
        };
        int n = 0, buf = 0, turn = 0;  // tiles, S buffer and its uses before
        bool ok = true;
        while (ok && !wk.done()) {
            if (grp == 1 && wk.newq) {
                if (wk.q > 0) {
                    // (the last queries may be in use for long: as long as the products, whose
                    // own waits end)
                    bool there;
                    do there = mbar_wait(&ctrl->q_empty, (wk.q - 1) & 1, abort);
                    while (!there && !*abort);
                    if (!__all_sync(0xffffffffu, there)) {
                        ok = false;
                        break;
                    }
                }
                load_q();
            }
            if (grp == 1 && !two) {
                wk.next(p);
                continue;
            }
            const int tok = wk.j * kTok + tk;
            const bool mine = tok < wk.T && tok < p.max_len;
            float* wp = p.weights + wk.b * p.w_stride + tok;
            const bool keep = wk.g > 0 || p.decay != 0.f;
            const float old = grp == 0 && mine && keep ? *wp : 0.f;
            if (wk.newq && !__all_sync(0xffffffffu, mbar_wait(&ctrl->q_full[wk.q % kQBufs], (wk.q / kQBufs) & 1, abort))) {
                ok = false;
                break;
            }
            const float* lse2 = ctrl->lse2[wk.q % kQBufs];
            const float* qs = ctrl->qs[wk.q % kQBufs];
            // columns from c0 on see the token: query t sees tokens up to T - Qt + t
            const int c0 = mine ? max(0, max(0, tok - (wk.T - p.Qt)) * p.Hq - wk.g * NP) : 0;
            float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (KIND == 1) {
                const int sl = n % kScSlots;
                if (!__all_sync(0xffffffffu, mbar_wait(&ctrl->sc_full[sl], (n / kScSlots) & 1, abort))) {
                    ok = false;
                    break;
                }
                sc = *reinterpret_cast<const float4*>(sc_ring + sl * kTok * 16 + tk * 16);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctrl->sc_empty[sl]);
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&ctrl->s_full[buf], turn & 1, abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tS = tmem + buf * buf_cols + lane_base;
            float acc = 0.f;
            // W columns from cc on: their sums first (the buffer is free when the last
            // are read), then the exponentials
            auto columns = [&](auto width, int cc) {
                constexpr int W = decltype(width)::value;
                float x[W];  // scores; fp8: the four block sums, each times its scale
                uint32_t a[W];
                auto load = [&](int part) {
                    if constexpr (W == 32) tmem_ld_x32(tS + part * NP + cc, a);
                    else tmem_ld_x16(tS + part * NP + cc, a);
                };
                load(0);
#pragma unroll
                for (int k = 0; k < W; ++k) x[k] = KIND == 1 ? __uint_as_float(a[k]) * sc.x : __uint_as_float(a[k]);
                load(1);
#pragma unroll
                for (int k = 0; k < W; ++k) x[k] = KIND == 1 ? fmaf(__uint_as_float(a[k]), sc.y, x[k]) : x[k] + __uint_as_float(a[k]);
                if (sums > 2) {
                    load(2);
#pragma unroll
                    for (int k = 0; k < W; ++k) x[k] = KIND == 1 ? fmaf(__uint_as_float(a[k]), sc.z, x[k]) : x[k] + __uint_as_float(a[k]);
                    load(3);
#pragma unroll
                    for (int k = 0; k < W; ++k) x[k] = KIND == 1 ? fmaf(__uint_as_float(a[k]), sc.w, x[k]) : x[k] + __uint_as_float(a[k]);
                }
                if (KIND == 1) load(4);  // the rotary part
                if (cc + W >= ce) {      // this group's share of the buffer is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctrl->s_free[buf]);
                }
                // columns that see the token and whose rows add (a NaN in the token stays
                // out of the others)
                uint32_t add = __ballot_sync(0xffffffffu, lane < W && !(lse2[cc + lane % W] == INFINITY));
                add &= c0 - cc >= 32 ? 0u : 0xffffffffu << max(c0 - cc, 0);
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    const int c = cc + k;
                    const float v = KIND == 1 ? fmaf(x[k], qs[c], __uint_as_float(a[k])) : x[k];
                    const float e = ex2(fmaf(v, p.scale_log2, -lse2[c]));
                    acc += add >> k & 1u ? e : 0.f;
                }
            };
            int cc = cb;
            for (; cc + 32 <= ce; cc += 32) columns(std::integral_constant<int, 32>{}, cc);
            if (cc < ce) columns(std::integral_constant<int, 16>{}, cc);
            if (++buf == nbuf) {
                buf = 0;
                ++turn;
            }
            // the halves meet (a tile's S waits for both groups' reads of an earlier
            // one, so the second group is never kParts tiles ahead of the first)
            if (two && grp == 1) {
                ctrl->part[n % kParts][tk] = acc;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctrl->part_full[n % kParts]);
            } else {
                if (two) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&ctrl->part_full[n % kParts], (n / kParts) & 1, abort))) {
                        ok = false;
                        break;
                    }
                    acc += ctrl->part[n % kParts][tk];
                }
                if (mine) *wp = wk.g > 0 ? old + acc : keep ? fmaf(p.decay, old, acc) : acc;
            }
            ++n;
            wk.next(p);
        }
        if (!ok && lane == 0) w_fail(p, ctrl);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }
}

}  // namespace

// Shared memory and row groups of a call; false if even 16 query rows do not fit.
bool weights_plan(int HQ, int lat_dim, int kind, WeightsParams& p, int* smem_bytes) {
    const int qrow = (lat_dim + kP) * 2;
    const int fixed = 1024 + kCtrlBytes + (kind == 1 ? kScSlots * kTok * 16 : 0);
    const int avail = kSmemLimit - fixed;
    // query rows that leave four blocks; fp8: and whose five sums fit TMEM
    int most = (avail - 4 * kBlk) / qrow / 16 * 16;
    const int cap = kind == 1 ? 96 : kLse;
    most = most > cap ? cap : most;
    if (most < 16) return false;
    const int groups = (HQ + most - 1) / most;
    const int per = (HQ + groups - 1) / groups;
    p.np = (per + 15) / 16 * 16;
    p.groups = (HQ + p.np - 1) / p.np;
    p.slots = (avail - p.np * qrow) / kBlk;
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    p.slots &= ~1;  // even, so that each slot always has the same loader
    *smem_bytes = fixed + p.np * qrow + p.slots * kBlk;
    return true;
}

cudaError_t launch_attn_weights(const WeightsMaps& maps, const WeightsParams& p, int kind, bool lsu, int ctas,
                                int smem_bytes, cudaStream_t stream) {
    static std::atomic<uint64_t> done[4];
    auto go = [&](auto* k) {
        const cudaError_t e = attribute_once(done[(kind == 1 ? 2 : 0) + (lsu ? 1 : 0)], reinterpret_cast<const void*>(k),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        k<<<dim3(ctas), kThreads, smem_bytes, stream>>>(maps, p);
        return cudaGetLastError();
    };
    return kind == 1 ? (lsu ? go(attn_weights_kernel<1, true>) : go(attn_weights_kernel<1, false>))
                     : (lsu ? go(attn_weights_kernel<0, true>) : go(attn_weights_kernel<0, false>));
}

}  // namespace mla
