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
// 128) bytes per key and head shared by 256 rows: far past the ridge for
// prompts. An item is two tiles of 128 rows, each with its own warpgroup of
// softmax threads, so that one tile's products run while the other's
// probabilities are formed. The query heads that share a key head lie in one
// tile (row = token x heads + head), which fills tiles for short sequences, wastes
// less of the causal diagonal and reads the keys once for all of them:
//   S_i = Q_i K^T   128 x 128 x 192, Q and K from shared memory, into TMEM
//   P_i             thread = row: no exchange between threads; bf16, written
//                   over S_i in TMEM, where it is the next product's A operand
//   O_i += P_i V    128 x 128 x 128, into TMEM
// The grid has a CTA for every item, longest first; a running CTA takes over
// pending ones (cluster launch control) until there are none, so that SMs share
// the items evenly, and the next item's Q, keys and scores are on their way
// while the last one's output is written.
// TMEM: S_0, S_1, O_0, O_1 of 128 columns each = all 512. Shared memory: Q
// 96 KB, and a ring of eight 16-KB blocks through which K (two blocks of k_nope
// and one of k_pe, 64 dims of 128 tokens) and V (two of 128 dims of 64 tokens)
// stream by TMA. Eight blocks are 1.6 key tiles, so a block is given back when
// its own last product is done: with V cut by dims and K given back by the tile
// the issuer waited 945 of 3,700 cycles a key tile for blocks.
//
// Keys past a sequence's end and masked ones have probability 0, which keeps
// finite values of theirs out of the sums. A NaN or infinity there would still
// spread (0 times it is NaN). So V past the sequence's end is cleared in shared
// memory (a buffer longer than its sequences holds anything there), and a row
// whose O comes out non-finite though the cause may lie behind what it sees is
// formed again by its warp from the keys that it sees alone.
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
constexpr int kThreadsP = 352;            // 8 softmax warps, the MMA issuer, the loader, the scheduler
constexpr int kItems = 4;                 // items between the scheduler and the slowest role
constexpr int kAhead = 4;                 // key tiles before an item's last load at which the next is asked for
constexpr int kAliveTiles = 4096;         // key tiles (about 7 ms) after which the loader shows that it goes on
constexpr int kQBytesP = 2 * 3 * kBlkP;
constexpr int kSmemP = 1024 + 1024 + kQBytesP + kSlots * kBlkP;
constexpr float kRaise = 8.f;             // log2 units

// Two tiles of queries of heads h .. h + pack - 1: query rows q_row .. of a
// sequence of q_len and k_len tokens, from its query t0 on, and the key tiles
// that each tile sees.
struct PItem {
    int h, q_row, k_row, q_len, k_len, t0, n0, n1;
};

struct PCtrl {
    uint64_t q_full[2], q_empty[2], blk_full[kSlots], blk_empty[kSlots];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], fin;
    uint64_t item_full[kItems], item_empty[kItems], more_full, want;
    uint32_t tmem_base;
    int stop[2];             // abort flag, and a count that goes up while long work goes on
    PItem item[kItems];  // h < 0: no more
    alignas(16) uint4 more;  // what a request for a pending CTA answered
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

// 32 columns of TMEM on their way into r, which holds them after tmem_ld_end
// (of every load begun before).
__device__ __forceinline__ void tmem_ld_x32_begin(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
                 "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_end(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void p_fail(const PrefillParams& p, PCtrl* c) {
    if (p.status) atomicOr(p.status, kErrWaitTimeout);
    *const_cast<volatile int*>(&c->stop[0]) = 1;
}

// mbar_wait that gives up only when nothing goes on: rows formed again over a
// long context take longer than a wait's limit, and so does an item of 80 million
// keys, during which a tile without queries waits for the next one.
__device__ __forceinline__ bool p_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_slow<false, true>(bar, parity, stop);
}

// A sequence's first row and its rows, of prefix sums clamped to [0, total].
__device__ __forceinline__ int2 p_span(const int32_t* cu, int b, int total) {
    const int a = min(max(__ldg(cu + b), 0), total), e = min(max(__ldg(cu + b + 1), 0), total);
    return make_int2(a, max(e - a, 0));
}

// Keys that query t of a sequence sees.
__device__ __forceinline__ int p_seen(int causal, int q_len, int k_len, int t) {
    return causal ? min(k_len, max(0, k_len - q_len + t + 1)) : k_len;
}

// Finds pairs of query tiles by their number in descending order of the key
// tiles that they see; used by a whole warp, mostly with ascending numbers.
struct PFinder {
    int lq, lk;            // lane's lengths of the first 32 sequences
    int tokens;            // of a pair
    int top, level;        // the most key tiles that a pair sees, and those of the last one found
    int64_t above, upto;   // pairs that see more, and at least, level key tiles
    __device__ __forceinline__ void lens(const PrefillParams& p, int i, int lane, int& q, int& k) const {
        if (i < 32) {
            q = lq;
            k = lk;
        } else {
            q = i + lane < p.B ? p_span(p.cu_q, i + lane, p.total_q).y : 0;
            k = i + lane < p.B ? p_span(p.cu_k, i + lane, p.total_k).y : 0;
        }
    }
    __device__ __forceinline__ void init(const PrefillParams& p, int lane) {
        tokens = 2 * p.tile_tokens;
        lq = lane < p.B ? p_span(p.cu_q, lane, p.total_q).y : 0;
        lk = lane < p.B ? p_span(p.cu_k, lane, p.total_k).y : 0;
        top = 0;
        for (int i = 0; i < p.B; i += 32) {
            int q, k;
            lens(p, i, lane, q, k);
            top = max(top, q > 0 ? (k + kKT - 1) / kKT : 0);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        level = top + 1;
        above = upto = 0;
    }
    // Pairs of a sequence that see at least x key tiles: the last ones, and the
    // very last sees all keys.
    __device__ __forceinline__ int count(const PrefillParams& p, int q, int k, int x) const {
        const int pairs = (q + tokens - 1) / tokens;
        if (x == 0 || pairs == 0) return pairs;
        if (x > (k + kKT - 1) / kKT) return 0;
        if (!p.causal) return pairs;
        const int y = (x - 1) * kKT - k + q;  // a pair ends past y; (x - 1) kKT < k, so y < q
        return y < 0 ? pairs : max(1, pairs - y / tokens);
    }
    __device__ __forceinline__ int64_t from(const PrefillParams& p, int x, int lane) const {
        int64_t n = 0;
        for (int i = 0; i < p.B; i += 32) {
            int q, k;
            lens(p, i, lane, q, k);
            n += __reduce_add_sync(0xffffffffu, count(p, q, k, x));
        }
        return n;
    }
    // Sequence b and pair qt of the s-th; false if there are fewer.
    __device__ __forceinline__ bool find(const PrefillParams& p, int64_t s, int lane, int& b, int& qt) {
        if (s < above || s >= upto) {  // another level: the highest whose pairs and those above pass s
            int lo = 0, hi = s < above ? top + 1 : level;
            int64_t n_lo = from(p, 0, lane), n_hi = s < above ? 0 : upto;  // n_lo > s >= n_hi
            if (n_lo <= s) return false;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                const int64_t n = from(p, mid, lane);
                if (n > s) {
                    lo = mid;
                    n_lo = n;
                } else {
                    hi = mid;
                    n_hi = n;
                }
            }
            level = lo;
            above = n_hi;
            upto = n_lo;
        }
        int64_t r = s - above;  // among the pairs that see exactly `level`
        for (int i = 0; i < p.B; i += 32) {
            int q, k;
            lens(p, i, lane, q, k);
            const int all = count(p, q, k, level), c = all - count(p, q, k, level + 1);
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, sum > r);
            if (hit) {
                const int L = __ffs(hit) - 1;
                const int first = (q + tokens - 1) / tokens - all - (sum - c);
                b = i + L;
                qt = static_cast<int>(__shfl_sync(0xffffffffu, first, L) + r);
                return true;
            }
            r -= __shfl_sync(0xffffffffu, sum, 31);
        }
        return false;
    }
};

// Asks for a pending CTA of this grid in this one's place; the answer lands at
// `dst` (16 bytes) and completes on `bar`.
__device__ __forceinline__ void ask_for_cta(uint4* dst, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(dst)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The block index that an answer gives, or -1 if none was pending.
__device__ __forceinline__ int64_t answered_cta(const uint4* src) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(src))
        : "memory");
    return got ? static_cast<int64_t>(x) : -1;
}

// The first (or last) of keys from .. to - 1 whose V is not finite, or INT_MAX
// (-1); by a whole warp, 16 keys at a time.
__device__ __noinline__ int p_bad_value(const PrefillParams& p, int hk, int64_t k0, int from, int to, bool last, int lane,
                                        int* alive) {
    const __nv_bfloat16* v = p.v + k0 * p.v_st + hk * p.v_sh + (lane & 15) * 8;
    auto bad = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
    const int none = last ? -1 : INT_MAX;
    for (int c = 0; c < to - from; c += 16) {
        if (lane == 0 && c % 32768 == 0) atomicAdd(alive, 1);
        const int j0 = last ? to - 16 - c : from + c;
        int at = none;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + 2 * i + (lane >> 4);
            const uint4 x = *reinterpret_cast<const uint4*>(v + min(max(j, from), to - 1) * p.v_st);
            if (j >= from && j < to && (bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w))) at = last ? max(at, j) : min(at, j);
        }
        at = last ? __reduce_max_sync(0xffffffffu, at) : __reduce_min_sync(0xffffffffu, at);
        if (at != none) return at;
    }
    return none;
}

// A row again from the keys that it sees alone, by its whole warp (V of a
// visible key may be non-finite, and then so is the row): 32 keys at a time.
// Eight lanes form the score of one of four keys, each over 24 of its dims, and
// a lane forms four of the 128 sums.
__device__ __noinline__ void p_row_again(const PrefillParams& p, int64_t qrow, int h, int hk, int64_t k0, int vis,
                                         float m2, float inv_l, int lane, int* alive) {
    const __nv_bfloat16* q = p.q + qrow * p.q_st + h * p.q_sh;
    auto unit = [](const __nv_bfloat16* a) { return *reinterpret_cast<const uint4*>(a); };
    auto dot8 = [](const uint4& x, const uint4& y, float s) {
        const __nv_bfloat162 *xa = reinterpret_cast<const __nv_bfloat162*>(&x), *yb = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(xa[i]), g = __bfloat1622float2(yb[i]);
            s = fmaf(f.x, g.x, s);
            s = fmaf(f.y, g.y, s);
        }
        return s;
    };
    const int u8 = (lane & 7) * 8;
    const uint4 q0 = unit(q + u8), q1 = unit(q + 64 + u8), q2 = unit(q + 128 + u8);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < vis; j0 += 32) {
        if (lane == 0 && j0 % 32768 == 0) atomicAdd(alive, 1);
        float s = 0.f;  // of key j0 + lane
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // keys j0 + 4 i .. j0 + 4 i + 3
            const int64_t kr = k0 + min(j0 + 4 * i + (lane >> 3), vis - 1);
            const __nv_bfloat16 *kn = p.k_nope + kr * p.k_st + hk * p.k_sh + u8, *kp = p.k_pe + kr * p.kp_st + u8;
            float d = dot8(q2, unit(kp), dot8(q1, unit(kn + 64), dot8(q0, unit(kn), 0.f)));
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            d += __shfl_xor_sync(0xffffffffu, d, 4);
            const float t = __shfl_sync(0xffffffffu, d, (lane & 3) * 8);
            if (lane >> 2 == i) s = t;
        }
        const float w = ex2(fmaf(s, p.scale_log2, -m2)) * inv_l;
        const int n = min(32, vis - j0);
        const __nv_bfloat16* v = p.v + (k0 + j0) * p.v_st + hk * p.v_sh + 4 * lane;
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const uint2 x = *reinterpret_cast<const uint2*>(v + j * p.v_st);
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.x)),
                         g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.y));
            acc[0] = fmaf(wj, f.x, acc[0]);
            acc[1] = fmaf(wj, f.y, acc[1]);
            acc[2] = fmaf(wj, g.x, acc[2]);
            acc[3] = fmaf(wj, g.y, acc[3]);
        }
    }
    *reinterpret_cast<uint2*>(p.out + (qrow * p.Hq + h) * kDv + 4 * lane) =
        make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
}

__global__ void __launch_bounds__(kThreadsP, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps maps, const __grid_constant__ PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    PCtrl* ctrl = reinterpret_cast<PCtrl*>(smem);
    uint8_t* qs = smem + 1024;
    uint8_t* ring = qs + kQBytesP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->q_full[i], 1);
            mbar_init(&ctrl->q_empty[i], 1);
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->p_half[i], 4);
            mbar_init(&ctrl->p_full[i], 4);
            mbar_init(&ctrl->o_full[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ctrl->blk_full[i], 1);
            mbar_init(&ctrl->blk_empty[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ctrl->item_full[i], 1);
            mbar_init(&ctrl->item_empty[i], 10);  // every warp but the scheduler
        }
        mbar_init(&ctrl->more_full, 1);
        mbar_init(&ctrl->want, 1);
        mbar_init(&ctrl->fin, 1);
        ctrl->stop[0] = ctrl->stop[1] = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k_nope);
        prefetch_tensormap(&maps.k_pe);
        prefetch_tensormap(&maps.v);
    }
    const int units = p.Hq / p.pack;  // head groups
    int64_t idx = blockIdx.x;         // item: head group idx % units of pair idx / units
    PFinder f;
    PItem next = {-1, 0, 0, 0, 0, 0, 0, 0};
    // item idx in `next` (h < 0: there is none), by the scheduler's whole warp
    auto look_up = [&]() {
        int b = 0, qt = 0;
        next.h = -1;
        if (!f.find(p, idx / units, lane, b, qt)) return;
        const int2 sq = p_span(p.cu_q, b, p.total_q), sk = p_span(p.cu_k, b, p.total_k);
        next.h = static_cast<int>(idx % units) * p.pack;
        next.q_row = sq.x;
        next.k_row = sk.x;
        next.q_len = sq.y;
        next.k_len = sk.y;
        next.t0 = qt * 2 * p.tile_tokens;
        auto tiles = [&](int t) {
            const int n = min(p.tile_tokens, sq.y - t);
            return n > 0 ? (p_seen(p.causal, sq.y, sk.y, t + n - 1) + kKT - 1) / kKT : 0;
        };
        next.n0 = tiles(next.t0);
        next.n1 = tiles(next.t0 + p.tile_tokens);
    };
    if (warp == 10) {
        f.init(p, lane);
        look_up();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    volatile int* abort = ctrl->stop;

    // The next item of this CTA, held by a whole warp until it gives it back;
    // null at the end (or on failure).
    int taken = 0;
    bool ok = true;
    auto take = [&]() -> const PItem* {
        const int k = taken % kItems;
        if (!__all_sync(0xffffffffu, p_wait(&ctrl->item_full[k], (taken / kItems) & 1, abort))) {
            ok = false;
            return nullptr;
        }
        return ctrl->item[k].h >= 0 ? &ctrl->item[k] : nullptr;
    };
    auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->item_empty[taken % kItems]);
        ++taken;
    };
    const int group = p.Hq / p.Hkv;

    if (warp == 10) {
        // ------------------------------------------------------------ scheduler
        // Finding an item takes a few microseconds (the code is cold each time), so
        // it is done aside; but a CTA asks for the next one only a few key tiles
        // before the loader is through with this one, so that it does not hold
        // items that another could begin.
        uint32_t asked = 0;  // answers taken
        bool on_its_way = false;
        auto next_cta = [&]() {
            if (lane == 0) {
                mbar_arrive_expect_tx(&ctrl->more_full, 16);
                ask_for_cta(&ctrl->more, &ctrl->more_full);
            }
            on_its_way = true;
            if (!__all_sync(0xffffffffu, p_wait(&ctrl->more_full, asked & 1, abort))) {
                ok = false;
                return;
            }
            on_its_way = false;
            ++asked;
            idx = answered_cta(&ctrl->more);
            fence_proxy_async_smem();  // read before the next answer is written
            __syncwarp();
        };
        while (ok) {
            const int k = taken % kItems;
            if (taken >= kItems &&
                !__all_sync(0xffffffffu, p_wait(&ctrl->item_empty[k], static_cast<uint32_t>(taken / kItems - 1) & 1, abort))) {
                ok = false;
                break;
            }
            if (lane == 0) {
                ctrl->item[k] = next;
                mbar_arrive(&ctrl->item_full[k]);
            }
            if (next.h < 0) break;
            // (an item may take long: as long as the loader, whose own waits end)
            bool there;
            do there = p_wait(&ctrl->want, taken & 1, abort);
            while (!there && !*abort);
            if (!__all_sync(0xffffffffu, there)) {
                ok = false;
                break;
            }
            ++taken;
            next_cta();
            if (!ok) break;
            next.h = -1;
            if (idx >= 0) look_up();
        }
        // past the last item the grid may hold CTAs that would find nothing (it is
        // sized by a bound): taken here they need not start
        while (ok && idx >= 0) next_cta();
        if (!ok && lane == 0) {
            p_fail(p, ctrl);
            volatile int never = 0;
            if (on_its_way) mbar_wait(&ctrl->more_full, asked & 1, &never);
        }
    } else if (warp == 9) {
        // --------------------------------------------------------------- loader
        uint32_t u = 0;         // blocks loaded
        int nq[2] = {0, 0};     // items whose tile i was loaded
        while (const PItem* item = take()) {
            const PItem it = *item;
            const int hk = it.h / group, nk = max(it.n0, it.n1);
            if (lane == 0) {
                auto load_q = [&](int i, int n) {
                    if (n == 0 || !ok) return;
                    if (nq[i] > 0 && !p_wait(&ctrl->q_empty[i], (nq[i] - 1) & 1, abort)) {
                        ok = false;
                        return;
                    }
                    mbar_arrive_expect_tx(&ctrl->q_full[i], 3 * p.pack * p.tile_tokens * 128);
                    for (int c = 0; c < 3; ++c)
                        tma_load_3d(qs + (i * 3 + c) * kBlkP, &maps.q, &ctrl->q_full[i], 64 * c, it.h,
                                    it.q_row + it.t0 + i * p.tile_tokens);
                    ++nq[i];
                };
                load_q(0, it.n0);
                if (nk == 0) mbar_arrive(&ctrl->want);
                for (int j = 0; j < nk && ok; ++j) {
                    if (j == max(nk - kAhead, 0)) mbar_arrive(&ctrl->want);
                    if (j % kAliveTiles == kAliveTiles - 1) atomicAdd(&ctrl->stop[1], 1);
                    for (int x = 0; x < 5; ++x, ++u) {
                        const uint32_t slot = u % kSlots;
                        if (u >= kSlots && !p_wait(&ctrl->blk_empty[slot], ((u / kSlots) - 1) & 1, abort)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&ctrl->blk_full[slot], kBlkP);
                        uint8_t* dst = ring + slot * kBlkP;
                        const int kr = it.k_row + j * kKT;
                        if (x < 2) tma_load_3d(dst, &maps.k_nope, &ctrl->blk_full[slot], 64 * x, hk, kr);
                        else if (x == 2) tma_load_3d(dst, &maps.k_pe, &ctrl->blk_full[slot], 0, 0, kr);
                        else
                            for (int d = 0; d < 2; ++d)
                                tma_load_3d(dst + d * (kBlkP / 2), &maps.v, &ctrl->blk_full[slot], 64 * d, hk, kr + 64 * (x - 3));
                        if (j == 0 && x == 2) load_q(1, it.n1);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            give_back();
        }
        if (!ok && lane == 0) {
            p_fail(p, ctrl);
            // no copy may arrive after the CTA is gone
            volatile int never = 0;
            for (uint32_t v = u < kSlots ? 0 : u - kSlots; v < u; ++v)
                mbar_wait(&ctrl->blk_full[v % kSlots], (v / kSlots) & 1, &never);
            for (int i = 0; i < 2; ++i)
                if (nq[i]) mbar_wait(&ctrl->q_full[i], (nq[i] - 1) & 1, &never);
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------- MMA issuer
        // The whole warp walks the loop and one lane issues: descriptors are then
        // warp-uniform values, which the instruction takes from uniform registers
        // (formed by a single lane they cost a move each per product: 4.6 against
        // 3.4 ms for a causal prompt of 32,768 tokens and 16 heads).
        const bool leader = elect_lane();
        const uint32_t idS = idesc_bf16(128, 128, false, false), idPV = idesc_bf16(128, 128, false, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dQ = smem_desc(smem_u32(qs), 16, 1024, kSw128);
        const uint64_t dK = smem_desc(smem_u32(ring), 16, 1024, kSw128);
        const uint64_t dV = smem_desc(smem_u32(ring), kBlkP / 2, 1024, kSw128);
        constexpr uint32_t kBlkD = kBlkP >> 4;
        uint32_t u0 = 0;                 // the item's first block
        uint32_t nq0 = 0, nq1 = 0;       // items with a tile 0, 1
        uint32_t np0 = 0, np1 = 0;       // probabilities taken of each
        int n0 = 0, n1 = 0;              // the item's key tiles
        auto wait_blk = [&](uint32_t u) {
            if (ok && !p_wait(&ctrl->blk_full[u % kSlots], (u / kSlots) & 1, abort)) ok = false;
        };
        auto scores = [&](int i, int j, int ni) {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const uint32_t u = u0 + 5 * j + c;
                wait_blk(u);
                if (!ok) return;
                tc_fence_after();
                const uint64_t da = dQ + (i * 3 + c) * kBlkD, db = dK + (u % kSlots) * kBlkD;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_bf16(tm + i * 128, da + 2 * kk, db + 2 * kk, idS, (c | kk) != 0);
                    // a block is free as soon as its last product is done, not the tile's
                    if (i == 1 || j >= n1) umma_commit(&ctrl->blk_empty[u % kSlots]);
                }
            }
            if (leader) {
                umma_commit(&ctrl->s_full[i]);
                if (j + 1 == ni) umma_commit(&ctrl->q_empty[i]);
            }
        };
        // P_i(j) V over keys 64 half .. 64 half + 63 of the tile
        auto values = [&](int i, int j, int half) {
            const uint32_t slot = (u0 + 5 * j + 3 + half) % kSlots;
            const uint64_t dv = dV + slot * kBlkD;
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16_ta(tm + 256 + i * 128, tm + i * 128 + half * 32 + 8 * kk, dv + kk * (2048 >> 4), idPV,
                                 (j | half | kk) != 0);
                if (i == 1 || j >= n1) umma_commit(&ctrl->blk_empty[slot]);
            }
        };
        auto step = [&](int i, int j, int ni, uint32_t& np) {  // P_i(j) V, then the scores of the next key tile
            if (!ok || j >= ni) return;
            // (the item's first P_i comes after the last one's O_i was read)
            if (!p_wait(&ctrl->p_half[i], np & 1, abort)) ok = false;
            wait_blk(u0 + 5 * j + 3);
            if (!ok) return;
            tc_fence_after();
            values(i, j, 0);
            wait_blk(u0 + 5 * j + 4);
            if (!p_wait(&ctrl->p_full[i], np & 1, abort)) {
                ok = false;
                return;
            }
            ++np;
            tc_fence_after();
            values(i, j, 1);
            // in order behind the product that reads P_i from the same columns
            if (j + 1 < ni) scores(i, j + 1, ni);
            else if (leader) umma_commit(&ctrl->o_full[i]);
        };
        auto start = [&](int i, int ni, uint32_t& nq) {
            if (!ok || ni == 0) return;
            if (!p_wait(&ctrl->q_full[i], nq & 1, abort)) {
                ok = false;
                return;
            }
            ++nq;
            scores(i, 0, ni);
        };
        while (const PItem* item = take()) {
            n0 = __shfl_sync(0xffffffffu, item->n0, 0);
            n1 = __shfl_sync(0xffffffffu, item->n1, 0);
            const int nk = max(n0, n1);
            start(0, n0, nq0);
            start(1, n1, nq1);
            for (int j = 0; j < nk && ok; ++j) {
                step(0, j, n0, np0);
                step(1, j, n1, np1);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            u0 += 5 * nk;
            give_back();
        }
        if (leader) {
            if (!ok) p_fail(p, ctrl);
            drain_mma(&ctrl->fin);
        }
    } else {
        // -------------------------------------------------------------- softmax
        const int i = warp >> 2;
        // row of the tile: token row / pack, head row % pack (rows past the last token's are not used)
        const int row = (warp & 3) * 32 + lane;
        const int tok = i * p.tile_tokens + row / p.pack, head = row % p.pack;
        const bool used = row < p.tile_tokens * p.pack;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + i * 128 + lanes, tO = tmem + 256 + i * 128 + lanes;
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        uint32_t ns = 0, no = 0;  // score tiles and outputs taken
        uint32_t u0 = 0;          // the item's first block
        while (const PItem* item = take()) {
            const int n = i == 0 ? item->n0 : item->n1;
            const int vis = p_seen(p.causal, item->q_len, item->k_len, item->t0 + tok);  // keys 0 .. vis - 1
            float m = -INFINITY, l = 0.f;                             // m in log2 units
            for (int j = 0; j < n && ok; ++j, ++ns) {
                if (!__all_sync(0xffffffffu, p_wait(&ctrl->s_full[i], ns & 1, abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int left = vis - j * kKT;  // visible keys of this tile
                const bool cut = __any_sync(0xffffffffu, left < kKT);
                // the scores twice, 32 at a time and the next ones on their way: for
                // the maximum and for the probabilities (128 at once would spill)
                uint32_t s[2][32];
                auto mask = [&](uint32_t(&x)[32], int c) {
                    if (cut) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k >= left) x[k] = 0xff800000u;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tmem_ld_x32_begin(tS, s[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld_end(s[c & 1]);
                    if (c < 3) tmem_ld_x32_begin(tS + (c + 1) * 32, s[~c & 1]);
                    mask(s[c & 1], c);
#pragma unroll
                    for (int k = 0; k < 32; k += 2)
                        mx[k / 2 & 3] = fmaxf(mx[k / 2 & 3], fmaxf(__uint_as_float(s[c & 1][k]), __uint_as_float(s[c & 1][k + 1])));
                }
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
                if (cut && item->k_len < (j + 1) * kKT) {
                    // V past the sequence's end: zeros (both tiles' threads write them)
                    const uint32_t uv = u0 + 5 * j + 3;
                    for (int h = 0; h < 2; ++h)
                        if (!__all_sync(0xffffffffu, p_wait(&ctrl->blk_full[(uv + h) % kSlots], ((uv + h) / kSlots) & 1, abort)))
                            ok = false;
                    if (!ok) break;
                    const int end = item->k_len - j * kKT;
                    for (int x = row; x < (kKT - end) * 16; x += kQT) {
                        const int r = end + x / 16;
                        *reinterpret_cast<uint4*>(ring + (uv + r / 64) % kSlots * kBlkP + (x / 8 & 1) * (kBlkP / 2) +
                                                  r % 64 * 128 + x % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t nb = pack2(-base, -base);
                tmem_ld_x32_begin(tS, s[0]);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
                    tmem_ld_end(s[c & 1]);
                    if (c < 3) tmem_ld_x32_begin(tS + (c + 1) * 32, s[~c & 1]);
                    mask(s[c & 1], c);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t x = fma2(pack2(__uint_as_float(s[c & 1][2 * k]), __uint_as_float(s[c & 1][2 * k + 1])), c2, nb);
                        float x0, x1;
                        unpack2(x, x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum[k & 1] = add2(sum[k & 1], pack2(x0, x1));
                        pk[k] = pack_bf16x2(x0, x1);
                    }
                    // (over scores that have been read)
                    tmem_st_x16(tS + 16 * c, pk);
                    if (c == 1) {  // the product with the first half of the keys may begin
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctrl->p_half[i]);
                    }
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
            if (ok && n > 0) {
                if (!__all_sync(0xffffffffu, p_wait(&ctrl->o_full[i], no & 1, abort))) ok = false;
                ++no;
            }
            if (!ok) break;
            tc_fence_after();
            const int t = item->t0 + tok, h = item->h + head;
            const bool mine = used && t < item->q_len;
            const int64_t at = (static_cast<int64_t>(item->q_row) + t) * p.Hq + h;
            const float inv = l > 0.f ? __fdividef(1.f, l) : l;  // l = 0: nothing seen; NaN: the row is NaN
            bool fine = true;
            // Four lanes trade 16-byte units, so that lane j of them holds unit j of four
            // rows and a store writes whole sectors. A loop, not unrolled: the code is
            // cold at every item, and its length costs more than its steps.
            const int64_t at_ = mine ? at : -1;
            int64_t rows[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) rows[k] = __shfl_sync(0xffffffffu, at_, (lane & 28) + k);
            __nv_bfloat16* out = p.out + (lane & 3) * 8;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                uint32_t v[32], x[4][4];
                if (n > 0) tmem_ld_x32(tO + c, v);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    // (a row that sees nothing may lie beside rows that do)
                    const float f = vis > 0 ? __uint_as_float(v[k]) * inv : 0.f, g = vis > 0 ? __uint_as_float(v[k + 1]) * inv : 0.f;
                    fine = fine && fabsf(f) <= 3.0e38f && fabsf(g) <= 3.0e38f;
                    x[k / 8][k % 8 / 2] = pack_bf16x2(f, g);
                }
#pragma unroll
                for (int b = 2; b > 0; b >>= 1)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if ((q & b) == 0) {
                            const bool up = (lane & b) != 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[q][e] : x[q | b][e], b);
                                x[q][e] = up ? got : x[q][e];
                                x[q | b][e] = up ? x[q | b][e] : got;
                            }
                        }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (rows[k] >= 0)
                        *reinterpret_cast<uint4*>(out + rows[k] * kDv + c) = make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
            }
            if (mine) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
            // O is not finite though the sums are: form the row again if a value that is
            // not lies in its last tile behind what it sees, or if none does that it sees
            // (large values whose weighted sum passes fp32's range, though not their mean)
            unsigned again = __ballot_sync(0xffffffffu, mine && !fine && l > 0.f && l < INFINITY && fabsf(m) < INFINITY);
            if (again) {
                const int hk = item->h / group, end = min(n * kKT, item->k_len);
                const bool these = again >> lane & 1u;
                const int low = __reduce_min_sync(0xffffffffu, these ? vis : INT_MAX);
                const int behind = p_bad_value(p, hk, item->k_row, low, end, true, lane, &ctrl->stop[1]);
                const int first = p_bad_value(p, hk, item->k_row, 0, end, false, lane, &ctrl->stop[1]);
                again = __ballot_sync(0xffffffffu, these && (behind >= vis || first >= vis));
            }
            while (again) {
                const int r = __ffs(again) - 1;
                again &= again - 1;
                __syncwarp();
                const int hr = __shfl_sync(0xffffffffu, h, r);
                p_row_again(p, item->q_row + __shfl_sync(0xffffffffu, t, r), hr, hr / group, item->k_row,
                            __shfl_sync(0xffffffffu, vis, r), __shfl_sync(0xffffffffu, m, r),
                            __shfl_sync(0xffffffffu, inv, r), lane, &ctrl->stop[1]);
            }
            // O_i has been read before this warp's next P_i is handed over
            tc_fence_before();
            u0 += 5 * max(item->n0, item->n1);
            give_back();
        }
        if (!ok && lane == 0) p_fail(p, ctrl);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

// Query heads of a group that lie in one tile: the largest divisor of the group
// whose whole tokens fill at least 124 of a tile's 128 rows.
int prefill_pack(int group) {
    for (int d = group < kQT ? group : kQT; d > 1; --d)
        if (group % d == 0 && kQT / d * d >= 124) return d;
    return 1;
}

// A bound of the pairs of tiles that all sequences have.
int64_t prefill_pairs(int64_t total_q, int B, int max_q_len, int tile_tokens) {
    const int64_t t = 2 * tile_tokens, each = (static_cast<int64_t>(max_q_len) + t - 1) / t;
    // sum of ceil(len / t) <= total / t + B, and B times the longest's
    return each <= (total_q / t + B) / B ? each * B : total_q / t + B;
}

cudaError_t launch_prefill(const PrefillMaps& maps, const PrefillParams& p, int max_q_len, cudaStream_t stream) {
    const int64_t items = prefill_pairs(p.total_q, p.B, max_q_len, p.tile_tokens) * (p.Hq / p.pack);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attribute_once(done, reinterpret_cast<const void*>(prefill_kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemP);
    if (e != cudaSuccess) return e;
    prefill_kernel<<<dim3(static_cast<unsigned>(items)), kThreadsP, kSmemP, stream>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace mla
