// Paged MLA decode over 8-bit rows with one scale for each page
// (mla_decode_fp8_page): tcgen05 products on the codes as they are.
//
// Mathematics. With code_j the 576 e4m3 codes of token j and s_j = s(page of j):
//   score_j = scale s_j (q . code_j),   out = sum_j p_j s_j code_j / sum_j p_j.
// The scale is the same for all of a row, so it never meets a code: it is one
// factor on the finished score, and it goes into the weight of the value
// product. In log2 units, x_j = log2(e) score_j + log2(s_j) and a running
// maximum m over x (not over the scores) give
//   P_j = 2^(x_j - m),   O += P_j code_j,   l += P_j / s_j,
//   out = O / l,   lse = (m + log2 l) ln 2,
// and P_j lies in a known range whatever the scales are, as 8 bits need it.
//
// 8-bit operands. A bf16 query value, scaled by a power of two per row to have
// the row's largest in [128, 256), is h + l / 32: h the nearest e4m3 value, l the
// nearest to 32 times the rest (the rest is at most 8, and has at most 3 more
// bits). h and l are two columns of the B operand, so the score product reads
// the tile once, and the two sums meet in fp32. P in (0, 256] is split the same
// way. Up to 32 query rows its two parts are columns too, with accumulators of
// their own; at 64 rows TMEM has no room for them, and the parts (l not scaled and
// e5m2 there) go into the same accumulator one after the other.
//
// Small weights. Under 2^-6, where h is at its finest step, l is a rounding up or down by
// the token's number in the golden-section sequence, up as often as the part of a step that
// is rounded: many weights of a long tail, each less than a step, add up to their sum
// (l's own sum takes them unrounded, so a tail rounded to nothing would be missing from
// the output). Up to 32 rows a fraction of l's one step there is added before it is rounded to
// the nearest, at 64 rows to the bits of f16 below those of e5m2 before they are cut off.
// 65,536 tokens alike 12.5 nats below one of them: these roundings put the tail's part of the output
// off by 2^-11, to the nearest by 2%, and with the largest weight at 2^3 all of it was missing. Time with
// both: 4 x 262,144 tokens at 32 rows 106.2 -> 107.0 us, 64 requests 39.3 -> 39.7, 64 rows 107.9 -> 108.6.
//
// Bound: HBM, 576 bytes a token; at 16 query rows the products take a third of
// the time the bytes do, at 64 rows about as long (S 1,150 cycles a tile, the value
// product 1,640; the bytes 2,940). Measured (among others in a graph): 4 x 262,144 tokens at 32 rows 106 us (5.7
// TB/s, 0.84 of the copy rate), 64 requests of 1k to 8k at 16 rows 38.5 us (0.68: some 10
// us are start-up, output and merge; pages read row by row 61 to 74 us), 786k tokens at 64 rows
// 105 us (0.63: two tiles of shared memory, each block held some 6,000 cycles from its load to
// its value product), 32 requests at 128 rows 123 us. So the kernel is a stream:
// 128-token tiles arrive by TMA as four blocks of 128 dims (16 KB, one 128-byte
// swizzle row a token) and the rotary part (8 KB). A block is the K-major A
// operand of S = C Q^T (thread = token = TMEM lane) and the MN-major A operand of
// O^T += C^T P, and its ring slot is free when its own value product is done.
//
// Warps: 0 issues S, 3 the value product, 1 and 2 load (at 16 rows 8 and 9 too); 4..7
// (and 8..11 from 32 rows on, each group half of the columns) turn a request's queries
// into h and l, then softmax, P and output. Pages that are not a multiple of 8 rows are
// read row by row by four warps behind those. The split of the work between CTAs, the
// partial results and their merge are those of the other decode kernels.
#include <climits>

#include "decode_split.cuh"
#include "launch.cuh"
#include "mla_common.cuh"

namespace mla {

namespace {

using F2 = packed2;

constexpr int kTok = 128;             // tokens a tile
constexpr int kBlk = kTok * 128;      // bytes of a latent block
constexpr int kRopeBlk = kTok * 64;   // and of the rotary part
constexpr int kQGens = 4;             // generations of query scales (three may be in use: a group is at most two tiles behind)
constexpr int kScs = 4;               // tiles' scales
constexpr float kNoMax = -1e30f;
constexpr float kLn2f = 0.69314718055994530942f;

// Shared memory decides the rate: a block is held from its load to its value
// product, so the ring's slots are what is in flight. At 64 rows the last block
// of a tile would wait for the value product of the tile before with seven slots
// (a chain of 4,700 cycles a tile); with eight it does not, and they fit beside
// one rotary slot (free again after the first two products of a tile).
template <int NP, bool LSU>
struct P8Cfg {
    static constexpr bool kStack = NP <= 32;            // P's parts in columns of their own
    static constexpr int kSlots = NP == 16 ? 11 : NP == 32 ? 9 : LSU ? 7 : 8;
    static constexpr int kRopes = NP == 64 && !LSU ? 1 : 2;
    static constexpr int kScW = LSU ? kTok : 16;        // scales of a tile: one for each row, or run of rows
    static constexpr int kPBufs = NP == 64 ? 1 : 2;
    // P of the maximum itself is 2^kTop, and a score may pass it by 2^kSlack before the
    // maximum is raised (O rescaled, a few thousand cycles). What a weight is rounded by, of
    // the largest: half of l's finest step and as much for the evenly spread part, 2^-14 / 2^kTop =
    // 2^-20; at 64 rows a step of e5m2 below 2^-10, 2^-13 / 2^kTop = 2^-16. (Raised
    // rarely, 2^3, up to 32 rows: 2^-17, and 0.5% less time at 32 rows, 0.4% at 16; 2^6
    // at 64 rows raises it in every other of the first dozen tiles of a request.)
    static constexpr float kTop = kStack ? 6.f : 3.f, kSlack = 8.f - kTop;
    static constexpr int kGroups = NP == 16 ? 1 : 2;    // softmax groups of four warps
    static constexpr int kCW = NP / kGroups;            // columns of a group
    static constexpr int kQBlk = 2 * NP * 128;          // a 128-dim block of the queries: h rows, then l rows
    static constexpr int kQBytes = 4 * kQBlk + 2 * NP * 64;
    static constexpr int kPRow = kStack ? 2 * NP : NP;  // bytes of a token's row of P (one swizzle row)
    static constexpr int kPBytes = 2 * NP * kTok;
    static constexpr uint32_t kPSw = kPRow == 32 ? kSw32 : kSw64;
    static constexpr int kOffRope = kSlots * kBlk;
    static constexpr int kOffQ = kOffRope + kRopes * kRopeBlk;  // (swizzle atoms: all of these lie at multiples of 1024)
    static constexpr int kOffP = kOffQ + kQBytes;
    static constexpr int kOffCtrl = kOffP + kPBufs * kPBytes;
    static constexpr int kMore = 4 + 4 * kGroups;       // first of the warps behind the softmax
    // loading warps: 1 and 2, and at 16 rows, where there are registers for it, two more
    // (a tile of 16-token pages is 40 boxes, about 75 cycles each to the warp that issues
    // them); LSU: four behind the softmax
    static constexpr int kLoaders = LSU ? 0 : NP == 16 ? 4 : 2;
    static constexpr int kThreads = 32 * (kMore + (LSU ? 4 : kLoaders - 2));
    static constexpr int kOCols = 4 * (kStack ? 2 * NP : NP);
    static constexpr int kColS = kOCols;                // two S buffers of 2 NP columns
    static_assert(kPRow == 32 || kPRow == 64, "one swizzle row");
    static_assert(kColS + 4 * NP <= 512, "tmem");
    static_assert(kQBlk % 1024 == 0 && (2 * NP * 64) % 1024 == 0 && kPBytes % 1024 == 0, "alignment of the swizzle atoms");
};

template <class C>
struct P8Ctrl {
    uint64_t blk_full[C::kSlots], blk_empty[C::kSlots];
    uint64_t rope_full[C::kRopes], rope_empty[C::kRopes];
    uint64_t s_full[2], s_free[2];
    // tile t's hand-off is p_full[t & 1], its products' end o_done[t & 1]: the
    // softmax may be a tile ahead of a slow issuer, which a single barrier's
    // parity could not tell
    uint64_t p_full[2], o_done[2];
    uint64_t q_full;
    uint64_t sc_full[kScs];
    uint64_t fin[2];
    uint32_t tmem_base;
    int abort;
    int t_begin, t_end, b0, j0;
    int unset[2];                         // a softmax group has columns without a maximum
    alignas(16) float sc[kScs][C::kScW];  // scales of a tile
    alignas(16) float kq[kQGens][64];     // what turns a column's sum into log2 units (without the token's scale)
    alignas(16) float m[64];              // running maximum (kNoMax: nothing seen yet)
    alignas(16) float nm[64];             // kTop - m (0 where m is kNoMax)
    alignas(16) float dy[64];             // how much nm changed; at a segment's end 1 / sum
    alignas(16) int most[64];             // largest of a tile, as an ordered whole number (INT_MIN: not raised)
};

// (no slack for alignment: dynamic shared memory begins at a multiple of 1024,
// which the kernel checks)
template <int NP, bool LSU>
constexpr int p8_smem() {
    return P8Cfg<NP, LSU>::kOffCtrl + (static_cast<int>(sizeof(P8Ctrl<P8Cfg<NP, LSU>>)) + 15) / 16 * 16;
}
static_assert(p8_smem<16, false>() <= 232448 && p8_smem<32, false>() <= 232448 && p8_smem<64, false>() <= 232448 &&
                  p8_smem<16, true>() <= 232448 && p8_smem<32, true>() <= 232448 && p8_smem<64, true>() <= 232448,
              "shared memory");

// Page and slot of token tok of the request with this table row; page 0 and a
// flag for an entry outside the pool or the row.
__device__ __forceinline__ int p8_slot(const DecodeParams& p, const int32_t* btr, int tok, int& page, bool& bad) {
    const int pi = tok / p.page_size;
    int64_t pg = pi < p.bt_cols ? __ldg(btr + pi) : -1;
    if (pg < 0 || (pg + 1) * p.page_size > p.num_slots) {
        bad = true;
        pg = 0;
    }
    page = static_cast<int>(pg);
    const int64_t s = pg * p.page_size + tok % p.page_size;
    return static_cast<int>(s < p.num_slots ? s : 0);
}

// L2 prefetch of request b's query rows of row group gy.
__device__ __forceinline__ void prefetch_queries(const DecodeParams& p, int b, int gy) {
    const int rows = req_rows_in_group(p, b, gy);
    const int64_t row0 = req_row0(p, b) + gy * 64;
    if (rows > 0) {
        prefetch_l2_bulk(p.q_lat + row0 * kD, static_cast<uint32_t>(rows * kD * 2));
        prefetch_l2_bulk(p.q_pe + row0 * kP, static_cast<uint32_t>(rows * kP * 2));
    }
}

// A page's scale. A pool smaller than a page has no scales (and no rows that count).
__device__ __forceinline__ float p8_scale(const DecodeParams& p, int page) {
    if (p.num_slots < p.page_size) return 1.f;
    const float s = __ldg(p.scales + page);
    return s < 0x1p-40f ? 0x1p-40f : s > 0x1p40f ? 0x1p40f : s;  // (NaN stays)
}

__device__ __forceinline__ void p8_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// N columns (16 or 32) of 32 lanes to one number each: lane c gets column c's (16
// columns: lanes c and c + 16). Each step hands half of what a lane holds to
// its partner, N - 1 or N shuffles in all; a redux for each column took some 100 cycles.
template <int N, class Op>
__device__ __forceinline__ float across_lanes(const F2 (&y)[N / 2], int lane, Op op) {
    float v[N / 2];
    {
        constexpr int h = N / 2;
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int c = 0; c < h; c += 2) {
            const float2 lo = un2(y[c / 2]), hi = un2(y[(c + h) / 2]);
            v[c] = op(up ? hi.x : lo.x, __shfl_xor_sync(0xffffffffu, up ? lo.x : hi.x, h));
            v[c + 1] = op(up ? hi.y : lo.y, __shfl_xor_sync(0xffffffffu, up ? lo.y : hi.y, h));
        }
    }
#pragma unroll
    for (int h = N / 4; h > 0; h >>= 1) {
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int c = 0; c < h; ++c) {
            const float lo = v[c], hi = v[c + h];
            v[c] = op(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, h));
        }
    }
    return N == 16 ? op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16)) : v[0];
}

// 16 columns from each of two places in TMEM, one wait for both.
__device__ __forceinline__ void p8_ld_pair(uint32_t at0, uint32_t at1, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
          "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]), "=r"(b[1]),
          "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]),
          "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
        : "r"(at0), "r"(at1)
        : "memory");
}

__device__ __forceinline__ void p8_store(float* to, float v) { *to = v; }
__device__ __forceinline__ void p8_store(__nv_bfloat16* to, float v) { *to = __float2bfloat16_rn(v); }

// Two values in f16 as e4m3 codes (the first in the low byte), and what is left of them.
__device__ __forceinline__ uint32_t p8_high(__half2 v, __half2& rest) {
    const uint32_t h = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&v), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h), __NV_E4M3);
    rest = __hsub2(v, *reinterpret_cast<const __half2*>(&hr));
    return h & 0xFFFFu;
}
// rest times 32 plus `more` as e4m3 codes.
__device__ __forceinline__ uint32_t p8_low(__half2 rest, __half2 more) {
    rest = __hfma2(rest, __float2half2_rn(32.f), more);
    return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&rest), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
}

template <int NP, bool LSU>
__global__ void __launch_bounds__(P8Cfg<NP, LSU>::kThreads, 1)
    mla_decode_page8_kernel(const __grid_constant__ DecodeMaps maps, const DecodeParams p) {
    using C = P8Cfg<NP, LSU>;
    using Ctrl = P8Ctrl<C>;
    using It = TileItT<7>;
    constexpr int CW = C::kCW, kRopes = C::kRopes;
    constexpr float kTop = C::kTop, kSlack = C::kSlack;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem;
    uint8_t* rope_ring = smem + C::kOffRope;
    uint8_t* qs = smem + C::kOffQ;
    uint8_t* pbufs = smem + C::kOffP;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + C::kOffCtrl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x, G = gridDim.x, gy = blockIdx.y;
    volatile int* abort = &ctrl->abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&ctrl->blk_full[i], LSU ? 4 : 1);
            mbar_init(&ctrl->blk_empty[i], 1);
        }
        for (int i = 0; i < kRopes; ++i) {
            mbar_init(&ctrl->rope_full[i], LSU ? 4 : C::kLoaders);
            mbar_init(&ctrl->rope_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->s_free[i], 4 * C::kGroups);
            mbar_init(&ctrl->p_full[i], 4 * C::kGroups);
            mbar_init(&ctrl->o_done[i], 1);
            mbar_init(&ctrl->fin[i], 1);
        }
        mbar_init(&ctrl->q_full, 4 * C::kGroups);
        for (int i = 0; i < kScs; ++i) mbar_init(&ctrl->sc_full[i], LSU ? 4 : 1);
        ctrl->abort = 0;
        fence_mbar_init();
    }
    if (!LSU && warp == 1 && lane == 0) {
        prefetch_tensormap(&maps.lat);
        prefetch_tensormap(&maps.rope);
    }
    // the previous kernel in the stream may still be writing the inputs or
    // reading the workspace
    griddep_wait();
    if (threadIdx.x == 0) {
        int4* r = reinterpret_cast<int4*>(status_rec(p));
#pragma unroll
        for (int k = 0; k < kStatusRecWords / 4; ++k) r[k] = make_int4(0, 0, 0, 0);
    }
    if (warp == 0) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    bool split = false;
    if (p.B <= C::kThreads) {
        // A thread a request: prefix sums of cost and tiles (the split of scan_range, in the
        // latency of one load instead of several passes over the lengths; lengths whose sums
        // might pass 32 bits are left to that).
        const int t = threadIdx.x;
        const uint32_t tl = t < p.B ? (static_cast<uint32_t>(max(__ldg(p.seq_lens + t), 0)) + kTok - 1) / kTok : 0u;
        const uint32_t cost = tl > 0 ? tl + p.wseg : 0u;
        uint32_t ic = cost, tt = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t vc = __shfl_up_sync(0xffffffffu, ic, o), vt = __shfl_up_sync(0xffffffffu, tt, o);
            if (lane >= o) {
                ic += vc;
                tt += vt;
            }
        }
        uint2* part = reinterpret_cast<uint2*>(pbufs);  // (not in use yet)
        if (lane == 31) part[warp] = make_uint2(ic, tt);
        if (t == 0) ctrl->t_begin = ctrl->t_end = ctrl->b0 = ctrl->j0 = 0;
        split = __syncthreads_or(tl > (1u << 21)) == 0;
        if (split) {
            uint32_t all_c = 0, all_t = 0, c0 = ic - cost, t0 = tt - tl;
#pragma unroll
            for (int w = 0; w < C::kThreads / 32; ++w) {
                const uint2 v = part[w];
                if (w < warp) {
                    c0 += v.x;
                    t0 += v.y;
                }
                all_c += v.x;
                all_t += v.y;
            }
            auto bound = [&](int k) -> uint32_t {  // k all_c / G
                return all_c < (1u << 31) / (G + 1) ? k * all_c / static_cast<uint32_t>(G)
                                                    : static_cast<uint32_t>(static_cast<unsigned long long>(k) * all_c / G);
            };
            const uint32_t x0 = bound(g), x1 = bound(g + 1), wseg = p.wseg;
            if (cost > 0 && c0 <= x0 && x0 < c0 + cost) {
                const uint32_t j = x0 - c0 > wseg ? x0 - c0 - wseg : 0u;
                ctrl->t_begin = static_cast<int>(t0 + j);
                ctrl->b0 = t;
                ctrl->j0 = static_cast<int>(j);
            }
            if (cost > 0 && c0 <= x1 && x1 < c0 + cost)
                ctrl->t_end = static_cast<int>(t0 + (x1 - c0 > wseg ? x1 - c0 - wseg : 0u));
            if (t == 0 && g == G - 1) ctrl->t_end = static_cast<int>(all_t);
        }
    }
    if (!split && warp == 2) {
        const TileRange r = scan_range<7>(p, g, G, lane);
        if (lane == 0) {
            ctrl->t_begin = r.tb;
            ctrl->t_end = r.te;
            ctrl->b0 = r.b0;
            ctrl->j0 = r.j0;
        }
    }
    if (threadIdx.x >= 128 && threadIdx.x < 192) {
        ctrl->nm[threadIdx.x - 128] = 0.f;
        ctrl->most[threadIdx.x - 128] = INT_MIN;
    }
    const bool misplaced = (smem_u32(smem) & 1023u) != 0;  // (cannot happen)
    if (misplaced && threadIdx.x == 0) atomicOr(status_rec(p), kErrWaitTimeout);
    __syncthreads();
    if (threadIdx.x == 0) griddep_launch_dependents();  // the merge grid may be scheduled as CTAs retire
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const int ntiles = misplaced ? 0 : ctrl->t_end - ctrl->t_begin;
    if (ntiles == 0 && ctrl->j0 > 0 && threadIdx.x < 64) {
        // an empty range strictly inside request b0 (more workers than tiles):
        // the merge of b0 counts this worker's slot, so mark it empty
        p.part_lse[(static_cast<int64_t>(gy) * p.SPG + g + ctrl->b0) * 64 + threadIdx.x] = -INFINITY;
    }
    It it;
    if (ntiles > 0) it.init(p.seq_lens, ctrl->b0, ctrl->j0);

    // The query rows of request b in this row group as h and l codes, and what undoes
    // their powers of two: rows w, w + W, .. are this warp's.
    auto load_q = [&](int b, int gen, int w, int W) {
        const int rows = req_rows_in_group(p, b, gy);
        const int64_t row0 = req_row0(p, b) + gy * 64;
        uint8_t* qr = qs + 4 * C::kQBlk;
        constexpr int kAt = 4;  // rows at a time, loads first
#pragma unroll 1
        for (int r4 = w; r4 < NP; r4 += kAt * W) {
            uint4 x[kAt][2];
            uint32_t e[kAt];
#pragma unroll
            for (int n = 0; n < kAt; ++n) {
                const int r = r4 + W * n;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                // lane holds latent values 16 lane .. 16 lane + 15 and rotary values 2 lane, 2 lane + 1
                const uint4* ql = reinterpret_cast<const uint4*>(p.q_lat + (row0 + r) * kD) + 2 * lane;
                x[n][0] = r < rows ? __ldg(ql) : z;
                x[n][1] = r < rows ? __ldg(ql + 1) : z;
                e[n] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(p.q_pe + (row0 + r) * kP) + lane) : 0u;
            }
#pragma unroll
            for (int n = 0; n < kAt; ++n) {
                const int r = r4 + W * n;
                if (r >= NP) break;
                const uint32_t v[9] = {x[n][0].x, x[n][0].y, x[n][0].z, x[n][0].w, x[n][1].x,
                                       x[n][1].y, x[n][1].z, x[n][1].w, e[n]};
                // the largest magnitude (non-negative floats are ordered as their bits)
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 9; ++k) {
                    // (a NaN is not the largest: its bits would be)
                    const uint32_t a = v[k] << 16 & 0x7FFFFFFFu, c = v[k] & 0x7FFF0000u;
                    top = max(top, max(a > 0x7F800000u ? 0u : a, c > 0x7F800000u ? 0u : c));
                }
                top = __reduce_max_sync(0xffffffffu, top);
                // the power of two that brings it into [128, 256); a row with an infinity, which
                // 8 bits do not hold, becomes NaN
                const int ex = static_cast<int>(top >> 23) - 127;
                const int k2 = max(-120, min(120, 7 - ex));
                const float up = top == 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
                // in f16, which holds 8 bits of every value that counts: the rest is one subtraction
                uint32_t h[9], l[9];
#pragma unroll
                for (int k = 0; k < 9; ++k) {
                    const float2 f = un2(mul2(f2(__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xFFFF0000u)), f2(up, up)));
                    __half2 rest;
                    h[k] = p8_high(__floats2half2_rn(f.x, f.y), rest);
                    l[k] = p8_low(rest, __float2half2_rn(0.f));
                }
                // unit lane % 8 of row r, block lane / 8 (NP is a multiple of 8: rows NP + r swizzle alike)
                uint8_t* at = qs + (lane >> 3) * C::kQBlk + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                auto pair = [](const uint32_t (&c)[9], int k) { return c[k] | c[k + 1] << 16; };
                *reinterpret_cast<uint4*>(at) = make_uint4(pair(h, 0), pair(h, 2), pair(h, 4), pair(h, 6));
                *reinterpret_cast<uint4*>(at + NP * 128) = make_uint4(pair(l, 0), pair(l, 2), pair(l, 4), pair(l, 6));
                uint8_t* ar = qr + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2;
                *reinterpret_cast<uint16_t*>(ar) = static_cast<uint16_t>(h[8]);
                *reinterpret_cast<uint16_t*>(ar + NP * 64) = static_cast<uint16_t>(l[8]);
                if (lane == 0)
                    ctrl->kq[gen][r] = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23) * p.scale_log2;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->q_full);
    };

    if (ntiles > 0) {
        if (warp == 0) {
            // ---------------------------------------------------------- scores
            // The whole warp walks the tiles and one lane issues, so descriptors are
            // warp-uniform values. The rotary part first: its slot is free soonest.
            const bool leader = elect_lane();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t id = idesc_f8(kTok, 2 * NP, 0, 0);
            const uint64_t dq = smem_desc(smem_u32(qs), 16, 1024, kSw128);
            const uint64_t dqr = smem_desc(smem_u32(qs) + 4 * C::kQBlk, 16, 512, kSw64);
            const uint64_t dring = smem_desc(smem_u32(ring), 16, 1024, kSw128);
            const uint64_t drope = smem_desc(smem_u32(rope_ring), 16, 512, kSw64);
            uint32_t slot = 0, phase = 0;
            int seg = -1, site = 0, i = 0;
            for (; i < ntiles; ++i) {
                if (i == 0 || it.j == 0) {
                    ++seg;
                    if (!mbar_wait(&ctrl->q_full, seg & 1, abort)) {
                        site = kSiteQFull;
                        break;
                    }
                }
                if (i >= 2 && !mbar_wait(&ctrl->s_free[i & 1], ((i >> 1) - 1) & 1, abort)) {
                    site = kSiteSFree;
                    break;
                }
                const int rr = i % kRopes;
                if (!mbar_wait(&ctrl->rope_full[rr], (i / kRopes) & 1, abort)) {
                    site = kSiteRopeFull;
                    break;
                }
                tc_fence_after();
                const uint32_t tS = tm + C::kColS + (i & 1) * 2 * NP;
                if (leader) {
                    const uint64_t da = drope + rr * static_cast<uint32_t>(kRopeBlk >> 4);
                    umma_f8(tS, da, dqr, id, 0u);
                    umma_f8(tS, da + 2, dqr + 2, id, 1u);
                    umma_commit(&ctrl->rope_empty[rr]);
                }
                for (int kb = 0; kb < 4; ++kb) {
                    if (!mbar_wait(&ctrl->blk_full[slot], phase, abort)) {
                        site = kSitePairFull;
                        break;
                    }
                    tc_fence_after();
                    if (leader) {
                        const uint64_t da = dring + slot * static_cast<uint32_t>(kBlk >> 4);
                        const uint64_t db = dq + kb * static_cast<uint32_t>(C::kQBlk >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) umma_f8(tS, da + 2 * kk, db + 2 * kk, id, 1u);
                    }
                    if (++slot == static_cast<uint32_t>(C::kSlots)) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (site) break;
                if (leader) umma_commit(&ctrl->s_full[i & 1]);
                it.next(p.seq_lens, p.B);
            }
            __syncwarp();
            if (leader) {
                if (site) {
                    fail(p, ctrl, kErrWaitTimeout, site, i);
                    report(p, kRoleS, site, i);
                }
                // every product issued here completes before the CTA may release TMEM or exit
                drain_mma(&ctrl->fin[0]);
            }
        } else if (warp == 3) {
            // --------------------------------------------------- value product
            const bool leader = elect_lane();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t id = idesc_f8(128, C::kPRow, 0, 0, true), id_l = idesc_f8(128, C::kPRow, 0, 1, true);
            const uint64_t dring = smem_desc(smem_u32(ring), kBlk, 1024, kSw128);
            const uint64_t dp0 = smem_desc(smem_u32(pbufs), C::kPBytes, 8 * C::kPRow, C::kPSw);
            uint32_t slot = 0;
            int site = 0, i = 0;
            for (; i < ntiles; ++i) {
                const bool fresh = i == 0 || it.j == 0;
                if (!mbar_wait(&ctrl->p_full[i & 1], (i >> 1) & 1, abort)) {
                    site = kSitePFull;
                    break;
                }
                tc_fence_after();
                const uint64_t dp = dp0 + (i % C::kPBufs) * static_cast<uint32_t>(C::kPBytes >> 4);
                for (int kb = 0; kb < 4; ++kb) {
                    if (leader) {
                        const uint64_t da = dring + slot * static_cast<uint32_t>(kBlk >> 4);
                        const uint32_t tO = tm + kb * C::kPRow;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            // tokens 32 kk .. 32 kk + 31
                            umma_f8(tO, da + kk * (32 * 128 >> 4), dp + kk * (32 * C::kPRow >> 4), id, !(fresh && kk == 0));
                            if (!C::kStack)
                                umma_f8(tO, da + kk * (32 * 128 >> 4), dp + ((NP * kTok + kk * 32 * C::kPRow) >> 4), id_l, 1u);
                        }
                        umma_commit(&ctrl->blk_empty[slot]);
                    }
                    if (++slot == static_cast<uint32_t>(C::kSlots)) slot = 0;
                }
                if (leader) umma_commit(&ctrl->o_done[i & 1]);
                it.next(p.seq_lens, p.B);
            }
            __syncwarp();
            if (leader) {
                if (site) {
                    fail(p, ctrl, kErrWaitTimeout, site, i);
                    report(p, kRolePV, site, i);
                }
                drain_mma(&ctrl->fin[1]);
            }
        } else if (!LSU && (warp == 1 || warp == 2 || warp >= C::kMore)) {
            // ------------------------------------------------------------ loads
            // Lane r owns run r of a tile: BR rows that lie next to each other in a page.
            // Each loading warp has its blocks of every tile and a share of the rotary part's
            // runs. A refill waits for the block 1 ring before by its parity, which could not
            // tell it from the one 2 rings before; but the warp's last wait was for a block
            // at most 4 earlier, and products end in order, so that one is long done.
            constexpr int kMine = LSU ? 4 : 4 / C::kLoaders;  // blocks of a warp
            const int me = warp < 4 ? warp - 1 : 2 + warp - C::kMore, kb0 = me * kMine;
            const int BR = p.run_rows;
            const uint64_t pol = gridDim.y > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
            bool bad = false, ok = true;
            int site = 0, i = 0;
            // the table is read two tiles ahead and the scales one, so that neither load is
            // waited for where it is made
            auto entry = [&](const It& t) -> int {
                const int tok = t.j * kTok + lane * BR, pi = tok / p.page_size;
                return tok < t.T && lane * BR < kTok && pi < p.bt_cols
                           ? __ldg(p.block_table + static_cast<int64_t>(t.b) * p.bt_stride + pi) : -1;
            };
            auto run_of = [&](const It& t, int pg, int& page) -> int {
                page = 0;
                const int tok = t.j * kTok + lane * BR;
                if (lane * BR >= min(kTok, t.T - t.j * kTok)) return 0;
                if (pg < 0 || (static_cast<int64_t>(pg) + 1) * p.page_size > p.num_slots) bad = true;
                else page = pg;
                const int64_t s = static_cast<int64_t>(page) * p.page_size + tok % p.page_size;
                return static_cast<int>(s < p.num_slots ? s : 0);
            };
            const int e_first = entry(it);
            It it1 = it;  // the tile after the one that is loaded
            if (ntiles > 1) it1.next(p.seq_lens, p.B);
            int e_next = ntiles > 1 ? entry(it1) : -1;
            int page_next, y_next = run_of(it, e_first, page_next);
            float s_next = warp == 1 ? p8_scale(p, page_next) : 1.f;
            uint32_t armed = 0;  // blocks whose barrier this warp has armed
            int rope_armed = 0;
            for (; i < ntiles && ok; ++i) {
                const int valid = min(kTok, it.T - it.j * kTok);
                const int nruns = (valid + BR - 1) / BR;
                const int y = y_next;
                const float s_now = s_next;
                it = it1;
                if (i + 1 < ntiles) {
                    const int e = e_next;
                    if (i + 2 < ntiles) {
                        it1.next(p.seq_lens, p.B);
                        e_next = entry(it1);
                        // (a new request: its queries are wanted as soon as the last one's are done with)
                        if (it1.j == 0 && warp == 2 && lane == 0) prefetch_queries(p, it1.b, gy);
                    }
                    y_next = run_of(it, e, page_next);
                    if (warp == 1) s_next = p8_scale(p, page_next);
                }
                {
                    const int rr = i % kRopes;
                    if (i >= kRopes && !__all_sync(0xffffffffu, mbar_wait(&ctrl->rope_empty[rr], ((i / kRopes) - 1) & 1, abort))) {
                        ok = false;
                        site = kSiteTmaRopeEmpty;
                        break;
                    }
                    // the runs of lanes me, me + kLoaders, ..
                    constexpr int kL = C::kLoaders > 0 ? C::kLoaders : 1;
                    const int share = (nruns - me + kL - 1) / kL;
                    if (lane == 0) mbar_arrive_expect_tx(&ctrl->rope_full[rr], static_cast<uint32_t>(share * BR * 64));
                    __syncwarp();
                    rope_armed = i + 1;
                    if (lane < nruns && lane % kL == me)
                        tma_load_2d(rope_ring + rr * kRopeBlk + lane * BR * 64, &maps.rope, &ctrl->rope_full[rr], kD, y, pol);
                }
                for (int kb = kb0; kb < kb0 + kMine; ++kb) {
                    const uint32_t u = 4u * i + kb, slot = u % C::kSlots, fill = u / C::kSlots;
                    if (fill > 0 && !__all_sync(0xffffffffu, mbar_wait(&ctrl->blk_empty[slot], (fill - 1) & 1, abort))) {
                        ok = false;
                        site = kSiteTmaPairEmpty;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&ctrl->blk_full[slot], static_cast<uint32_t>(nruns * BR * 128));
                    __syncwarp();
                    armed = u + 1;
                    if (lane < nruns)
                        tma_load_2d(ring + slot * kBlk + lane * BR * 128, &maps.lat, &ctrl->blk_full[slot], kb * 128, y, pol);
                }
                if (warp == 1) {
                    // (its slot: the loads of tile i are behind the value product of tile i - 3,
                    // which read nothing later than the scales of tile i - 3 did)
                    if (lane < nruns) ctrl->sc[i % kScs][lane] = s_now;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctrl->sc_full[i % kScs]);
                }
            }
            if (!ok && lane == 0) {
                fail(p, ctrl, kErrWaitTimeout, site, i);
                report(p, kRoleTma, site, i);
            }
            if (lane == 0 && *abort) {
                // Copies armed here may still be on their way: let them land before the CTA
                // leaves (otherwise the score product has waited for every one). A slot that
                // the other loader filled since cannot be told by its parity and waits out
                // the deadline, one for all.
                const unsigned long long t0 = globaltimer_ns();
                auto land = [&](uint64_t* bar, uint32_t par) {
                    while (!mbar_try_wait(bar, par) && globaltimer_ns() - t0 < kWaitLimitNs) {
                    }
                };
                const uint32_t from = armed > static_cast<uint32_t>(C::kSlots) ? armed - C::kSlots : 0;
                for (uint32_t u = from; u < armed; ++u)
                    if ((u & 3) / kMine == static_cast<uint32_t>(me)) land(&ctrl->blk_full[u % C::kSlots], (u / C::kSlots) & 1);
                for (int k = max(0, rope_armed - kRopes); k < rope_armed; ++k) land(&ctrl->rope_full[k % kRopes], (k / kRopes) & 1);
            }
            if (bad) atomicOr(status_rec(p), kErrBadBlock);
        } else if (warp >= C::kMore) {
            // -------------------------------------------- loads, row by row (LSU)
            // Warp w's rows of a tile are 32 w .. 32 w + 31.
            bool bad = false;
            int site = 0, i = 0;
            const int w = warp - C::kMore;
            uint64_t *pend = nullptr, *pend2 = nullptr;  // barriers of the fill before, not yet handed over
            uint32_t u = 0;
            auto hand_over = [&]() {
                if (!pend) return;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(pend);
                    if (pend2) mbar_arrive(pend2);
                }
                pend = pend2 = nullptr;
            };
            // what waits behind a barrier may need this warp's last fill first
            auto wait = [&](uint64_t* bar, uint32_t par, int where) {
                if (pend && !__all_sync(0xffffffffu, mbar_try_wait(bar, par))) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    hand_over();
                }
                if (__all_sync(0xffffffffu, mbar_wait(bar, par, abort))) return true;
                site = where;
                return false;
            };
            auto filled = [&](uint64_t* bar, uint64_t* bar2) {  // the fill before this one has landed: hand it over
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                hand_over();
                pend = bar;
                pend2 = bar2;
            };
            for (; i < ntiles; ++i) {
                if constexpr (LSU) {
                    const int valid = min(kTok, it.T - it.j * kTok);
                    const int row = w * 32 + lane;
                    const int32_t* btr = p.block_table + static_cast<int64_t>(it.b) * p.bt_stride;
                    int page = 0, slot_of = 0;
                    if (row < valid) slot_of = p8_slot(p, btr, it.j * kTok + row, page, bad);
                    ctrl->sc[i % kScs][row] = row < valid ? p8_scale(p, page) : 1.f;
                    const int rr = i % kRopes;
                    if (i >= kRopes && !wait(&ctrl->rope_empty[rr], ((i / kRopes) - 1) & 1, kSiteLsuRopeEmpty)) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // 8 rows of four 16-byte units at a time
                        const int r = w * 32 + 8 * k + (lane >> 2), un = lane & 3;
                        const int s = __shfl_sync(0xffffffffu, slot_of, 8 * k + (lane >> 2));
                        if (r < valid)
                            p8_cp16(smem_u32(rope_ring + rr * kRopeBlk + r * 64 + ((un ^ ((r >> 1) & 3)) << 4)),
                                    p.cache + static_cast<int64_t>(s) * kRowPage + kD + un * 16);
                    }
                    filled(&ctrl->rope_full[rr], &ctrl->sc_full[i % kScs]);
                    bool stop = false;
                    for (int kb = 0; kb < 4; ++kb, ++u) {
                        const uint32_t slot = u % C::kSlots, fill = u / C::kSlots;
                        if (fill > 0 && !wait(&ctrl->blk_empty[slot], (fill - 1) & 1, kSiteLsuPairEmpty)) {
                            stop = true;
                            break;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {  // 4 rows of eight units at a time
                            const int r = w * 32 + 4 * k + (lane >> 3), un = lane & 7;
                            const int s = __shfl_sync(0xffffffffu, slot_of, 4 * k + (lane >> 3));
                            if (r < valid)
                                p8_cp16(smem_u32(ring + slot * kBlk + r * 128 + ((un ^ (r & 7)) << 4)),
                                        p.cache + static_cast<int64_t>(s) * kRowPage + kb * 128 + un * 16);
                        }
                        filled(&ctrl->blk_full[slot], nullptr);
                    }
                    if (stop) break;
                }
                it.next(p.seq_lens, p.B);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            hand_over();
            if (site && lane == 0) {
                fail(p, ctrl, kErrWaitTimeout, site, i);
                report(p, kRoleLsu0, site, i);
            }
            if (bad) atomicOr(status_rec(p), kErrBadBlock);
        } else if (warp >= 4) {
            // ------------------------------------------ softmax, P and output
            // Thread tk holds token tk of the tile (TMEM lane tk), for the group's columns cb .. cb + CW.
            const int grp = (warp - 4) >> 2, wq = warp & 3, tk = wq * 32 + lane;
            const int cb = grp * CW;
            const int bar = 1 + grp;
            const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
            const int run_shift = LSU ? 0 : 31 - __clz(p.run_rows);  // (a power of two)
            load_q(it.b, 0, warp - 4, 4 * C::kGroups);
            F2 l[CW / 2];          // this token's share of the columns' sums
            bool unset = false;
            int seg = -1, start_j = 0, T = 0, qt = 0, rows = 0;
            bool failed = false;
            int site = 0, i = 0;
            auto wait = [&](uint64_t* b, uint32_t par, int where) {
                if (!mbar_wait(b, par, abort)) {
                    if (!failed) site = where;
                    failed = true;
                }
            };
            for (; i < ntiles; ++i) {
                const bool fresh = i == 0 || it.j == 0;
                if (fresh) {
                    ++seg;
                    start_j = it.j;
                    T = it.T;
                    qt = req_qt(p, it.b);
                    rows = req_rows_in_group(p, it.b, gy);
#pragma unroll
                    for (int c = 0; c < CW / 2; ++c) l[c] = 0ull;
                    wait(&ctrl->q_full, seg & 1, kSiteQFull);
                }
                const float* kq = ctrl->kq[seg % kQGens] + cb;
                const int tok = it.j * kTok + tk, valid = min(kTok, T - it.j * kTok);
                wait(&ctrl->sc_full[i % kScs], (i / kScs) & 1, kSiteSFull);
                const float vs = tk < valid ? ctrl->sc[i % kScs][tk >> run_shift] : 1.f;
                // (a scale that is NaN makes NaN of the weights that count, and must not of a weight of 0)
                const float lv = log2f(vs), inv_vs = vs == vs ? 1.f / vs : 1.f;
                wait(&ctrl->s_full[i & 1], (i >> 1) & 1, kSiteSFull);
                tc_fence_after();
                // y = log2 of P before any limit: score and scale in log2 units, less the maximum, and kTop
                F2 y[CW / 2];
                {
                    const uint32_t tS = tmem + C::kColS + (i & 1) * 2 * NP + lane_base + cb;
                    const F2 vs2 = f2(vs, vs), lv2 = f2(lv, lv), old2 = fresh ? 0ull : f2(1.f, 1.f);
#pragma unroll
                    for (int c0 = 0; c0 < CW; c0 += 16) {
                        uint32_t h[16], lo[16];
                        p8_ld_pair(tS + c0, tS + NP + c0, h, lo);
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 k = *reinterpret_cast<const float4*>(kq + c0 + c);
                            const float4 nm = *reinterpret_cast<const float4*>(ctrl->nm + cb + c0 + c);
                            const F2 a = fma2(f2(__uint_as_float(lo[c]), __uint_as_float(lo[c + 1])), f2(0x1p-5f, 0x1p-5f),
                                              f2(__uint_as_float(h[c]), __uint_as_float(h[c + 1])));
                            const F2 b = fma2(f2(__uint_as_float(lo[c + 2]), __uint_as_float(lo[c + 3])), f2(0x1p-5f, 0x1p-5f),
                                              f2(__uint_as_float(h[c + 2]), __uint_as_float(h[c + 3])));
                            y[(c0 + c) / 2] = fma2(mul2(a, vs2), f2(k.x, k.y), fma2(f2(nm.x, nm.y), old2, lv2));
                            y[(c0 + c) / 2 + 1] = fma2(mul2(b, vs2), f2(k.z, k.w), fma2(f2(nm.z, nm.w), old2, lv2));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctrl->s_free[i & 1]);
                bool clear = tk >= valid;  // the row's codes must not meet the value product
                if (it.j * kTok + valid > T - qt || valid < kTok) {
                    // columns from c0 on see the token: query t sees tokens up to T - qt + t
                    const int c0 = tk < valid ? max(0, tok - (T - qt)) * p.Hq - gy * 64 - cb : INT_MAX;
                    bool nan = true;
#pragma unroll
                    for (int c = 0; c < CW; c += 2) {
                        float2 v = un2(y[c / 2]);
                        nan = nan && v.x != v.x && v.y != v.y;
                        if (c < c0) v.x = -INFINITY;
                        if (c + 1 < c0) v.y = -INFINITY;
                        y[c / 2] = f2(v.x, v.y);
                    }
                    // a NaN code would pass a weight of 0: rows that some queries do not see are
                    // cleared if they hold one (those that do see it have NaN for a weight)
                    if (tk < valid && c0 > -cb && nan && tok > T - qt) {
                        const uint32_t s0 = (4u * i) % C::kSlots;
                        for (int kb = 0; kb < 4 && !clear; ++kb) {
                            const uint8_t* blk = ring + (s0 + kb) % C::kSlots * kBlk + tk * 128;
                            for (int un = 0; un < 32; ++un) {
                                const uint32_t v = reinterpret_cast<const uint32_t*>(blk)[un] & 0x7F7F7F7Fu;
                                if (((v + 0x01010101u) & 0x80808080u) != 0) clear = true;
                            }
                        }
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < CW / 2; ++c) {
                    const float2 v = un2(y[c]);
                    top = fmaxf(top, fmaxf(v.x, v.y));
                }
                if (named_bar_or(bar, 128, fresh || failed || unset || top > kTop + kSlack)) {
                    // maxima move: of a fresh segment all columns', otherwise of those that a
                    // score passes by more than kSlack. Lane c finds its warp's largest of
                    // column c (as an ordered whole number; NaN counts as nothing).
                    const float best = across_lanes<CW>(y, lane, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < CW && (fresh || unset || best > kTop + kSlack)) {
                        const int k = __float_as_int(fmaxf(best, kNoMax));
                        atomicMax(&ctrl->most[cb + lane], k < 0 ? k ^ 0x7FFFFFFF : k);
                    }
                    named_bar_sync(bar, 128);
                    if (tk < CW) {
                        const int c = cb + tk, k = ctrl->most[c];
                        ctrl->most[c] = INT_MIN;
                        const float old = fresh ? kNoMax : ctrl->m[c], shift = fresh ? 0.f : ctrl->nm[c];
                        const float t = k == INT_MIN ? kNoMax : __int_as_float(k < 0 ? k ^ 0x7FFFFFFF : k);
                        const float m = t > kNoMax ? fmaxf(old, t - shift) : old;
                        const float nm = m > kNoMax ? kTop - m : 0.f;
                        ctrl->m[c] = m;
                        ctrl->nm[c] = nm;
                        ctrl->dy[c] = nm - shift;
                        const unsigned none = __ballot_sync(CW == 32 ? 0xffffffffu : 0xffffu, !(m > kNoMax));
                        if (tk == 0) ctrl->unset[grp] = none != 0;
                    }
                    if (named_bar_or(bar, 128, failed)) break;
                    unset = ctrl->unset[grp] != 0;
                    if (!fresh) {
                        wait(&ctrl->o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, kSiteORescale);
                        tc_fence_after();
                        __syncwarp();
                    }
#pragma unroll
                    for (int c0 = 0; c0 < CW; c0 += 16) {
                        float a[16];
                        bool moved = false;
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 d = *reinterpret_cast<const float4*>(ctrl->dy + cb + c0 + c);
                            y[(c0 + c) / 2] = add2(y[(c0 + c) / 2], f2(d.x, d.y));
                            y[(c0 + c) / 2 + 1] = add2(y[(c0 + c) / 2 + 1], f2(d.z, d.w));
                            a[c] = d.x;
                            a[c + 1] = d.y;
                            a[c + 2] = d.z;
                            a[c + 3] = d.w;
                            moved = moved || fminf(fminf(d.x, d.y), fminf(d.z, d.w)) < 0.f;
                        }
                        if (fresh || !moved) continue;
                        // (a column that had nothing yet may go up; there is nothing to scale)
#pragma unroll
                        for (int c = 0; c < 16; ++c) a[c] = ex2(fminf(a[c], 0.f));
#pragma unroll
                        for (int c = 0; c < 16; c += 2) l[(c0 + c) / 2] = mul2(l[(c0 + c) / 2], f2(a[c], a[c + 1]));
                        if constexpr (NP == 16) {
                            // all of O is the group's: 128 columns, h and l of each M-tile side by side
#pragma unroll 1
                            for (int half = 0; half < 2; ++half) {
                                uint32_t o[64];
                                tmem_ld_x64(tmem + lane_base + half * 64, o);
#pragma unroll
                                for (int c = 0; c < 64; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a[c & 15]);
                                tmem_st_x64(tmem + lane_base + half * 64, o);
                            }
                        } else {
#pragma unroll 1
                            for (int mt = 0; mt < 4; ++mt) {
                                const uint32_t at = tmem + lane_base + mt * C::kPRow + cb + c0;
                                uint32_t o[16], u[16];
                                if constexpr (C::kStack) p8_ld_pair(at, at + NP, o, u);
                                else tmem_ld_x16(at, o);
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    o[c] = __float_as_uint(__uint_as_float(o[c]) * a[c]);
                                    if (C::kStack) u[c] = __float_as_uint(__uint_as_float(u[c]) * a[c]);
                                }
                                tmem_st_x16(at, o);
                                if (C::kStack) tmem_st_x16(at + NP, u);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                uint32_t hc[CW / 4], lc[CW / 4];
                const F2 inv2 = f2(inv_vs, inv_vs);
                // where this token's roundings of small weights lie: the golden section's multiples,
                // which any run of tokens covers evenly
                const uint32_t turn = static_cast<uint32_t>(tok) * 2654435769u;
                const __half2 dither = __float2half2_rn(static_cast<float>(static_cast<int32_t>(turn)) * 0x1p-41f);
                const uint32_t up = (turn >> 24) * 0x10001u;
                uint32_t rests[2];
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    const float2 v = un2(y[c / 2]);
                    const float a = ex2(v.x), b = ex2(v.y);
                    l[c / 2] = fma2(f2(a, b), inv2, l[c / 2]);
                    // (f16 holds 11 bits, the two codes 8 of them)
                    const __half2 weights = __floats2half2_rn(a, b);
                    __half2 rest;
                    const uint32_t h = p8_high(weights, rest);
                    hc[c >> 2] = c & 2 ? hc[c >> 2] | h << 16 : h;
                    if constexpr (C::kStack) {
                        const uint32_t lo = p8_low(rest, dither);
                        lc[c >> 2] = c & 2 ? lc[c >> 2] | lo << 16 : lo;
                    } else {
                        // e5m2 is the upper byte of f16: half a step added and cut off rounds to the
                        // nearest, any part of a step rounds up that often
                        const uint32_t small = __hlt2_mask(weights, __float2half2_rn(0x1p-6f));
                        rests[(c >> 1) & 1] = *reinterpret_cast<const uint32_t*>(&rest) + ((up & small) | (0x00800080u & ~small));
                        if (c & 2) lc[c >> 2] = __byte_perm(rests[0], rests[1], 0x7531);
                    }
                }
                // P's place is free when the value product that read it last is done
                if (i >= C::kPBufs)
                    wait(&ctrl->o_done[(i - C::kPBufs) & 1], ((i - C::kPBufs) >> 1) & 1, kSiteOPbuf);
                uint8_t* prow = pbufs + (i % C::kPBufs) * C::kPBytes + tk * C::kPRow;
                const int sw = swz_p(tk, C::kPSw);
#pragma unroll
                for (int n = 0; n < CW / 16; ++n) {
                    const int un = cb / 16 + n;
                    *reinterpret_cast<uint4*>(prow + ((un ^ sw) << 4)) =
                        make_uint4(hc[4 * n], hc[4 * n + 1], hc[4 * n + 2], hc[4 * n + 3]);
                    uint8_t* lrow = C::kStack ? prow + (((NP / 16 + un) ^ sw) << 4) : prow + NP * kTok + ((un ^ sw) << 4);
                    *reinterpret_cast<uint4*>(lrow) = make_uint4(lc[4 * n], lc[4 * n + 1], lc[4 * n + 2], lc[4 * n + 3]);
                }
                if (clear) {
                    const uint32_t s0 = (4u * i) % C::kSlots;
                    for (int kb = grp; kb < 4; kb += C::kGroups) {
                        uint4* row = reinterpret_cast<uint4*>(ring + (s0 + kb) % C::kSlots * kBlk + tk * 128);
#pragma unroll
                        for (int un = 0; un < 8; ++un) row[un ^ (tk & 7)] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && (p.test_hold != 1 || i > 0)) mbar_arrive(&ctrl->p_full[i & 1]);  // (test hook: a hand-off that never comes)
                const int b = it.b, tiles = it.tiles, j = it.j;
                it.next(p.seq_lens, p.B);
                if (i + 1 < ntiles && j + 1 < tiles) continue;
                // ------------------------------------------- the segment's end
                // The next request's queries first: the score product has read these, and while
                // the last value product runs there is nothing else to do.
                if (i + 1 < ntiles) load_q(it.b, (seg + 1) % kQGens, warp - 4, 4 * C::kGroups);
                // The warps' sums meet in the group's own part of P, which the last value
                // product has read: CW / 4 numbers in each row.
                wait(&ctrl->o_done[i & 1], (i >> 1) & 1, kSiteOFinal);
                auto sums = [&](int w, int c) -> float* {
                    const int idx = w * CW + c, row = idx / (CW / 4), at = idx % (CW / 4);
                    return reinterpret_cast<float*>(pbufs + (i % C::kPBufs) * C::kPBytes + row * C::kPRow +
                                                    (((cb / 16 + at / 4) ^ swz_p(row, C::kPSw)) << 4)) + at % 4;
                };
                const float sum = across_lanes<CW>(l, lane, [](float a, float b) { return a + b; });
                if (lane < CW) *sums(wq, lane) = sum;
                named_bar_sync(bar, 128);
                const bool whole = start_j == 0 && j + 1 == tiles;
                const int64_t row0 = req_row0(p, b) + gy * 64;
                const int64_t slot0 = (static_cast<int64_t>(gy) * p.SPG + g + b) * 64;
                if (tk < CW) {
                    const int c = cb + tk;
                    const float s = *sums(0, tk) + *sums(1, tk) + *sums(2, tk) + *sums(3, tk);
                    // (a NaN sum is not nothing)
                    ctrl->dy[c] = s == 0.f ? 0.f : 1.f / s;
                    const float L = s == 0.f ? -INFINITY : (ctrl->m[c] - kTop + log2f(s)) * kLn2f;
                    if (c < rows) {
                        if (whole) p.lse[row0 + c] = L;
                        // (the merge leaves a NaN out of its maximum, and of an infinity it makes NaN)
                        else p.part_lse[slot0 + c] = L != L ? INFINITY : L;
                    }
                }
                named_bar_sync(bar, 128);
                tc_fence_after();
                __syncwarp();
                // lane tk holds dim 128 mt + tk here, of 16 rows at a time
                auto put = [&](auto* base) {  // row cb of this segment, dim tk
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += 16) {
                        const int n = rows - cb - c0;  // rows of these 16 that there are
                        if (n <= 0) break;
                        float inv[16];
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(ctrl->dy + cb + c0 + c);
                            inv[c] = v.x;
                            inv[c + 1] = v.y;
                            inv[c + 2] = v.z;
                            inv[c + 3] = v.w;
                        }
#pragma unroll 1
                        for (int mt = 0; mt < 4; ++mt) {
                            const uint32_t at = tmem + lane_base + mt * C::kPRow + cb + c0;
                            uint32_t o[16];
                            if constexpr (C::kStack) {
                                uint32_t lo[16];
                                p8_ld_pair(at, at + NP, o, lo);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    o[c] = __float_as_uint(fmaf(__uint_as_float(lo[c]), 0x1p-5f, __uint_as_float(o[c])));
                            } else {
                                tmem_ld_x16(at, o);
                            }
                            auto* to = base + c0 * kD + mt * 128;
                            if (n >= 16) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) p8_store(to + c * kD, __uint_as_float(o[c]) * inv[c]);
                            } else {
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    if (c < n) p8_store(to + c * kD, __uint_as_float(o[c]) * inv[c]);
                            }
                        }
                    }
                };
                if (!whole) put(p.part_o + (slot0 + cb) * kD + tk);
                else if (p.out_f32) put(static_cast<float*>(p.out) + (row0 + cb) * kD + tk);
                else put(static_cast<__nv_bfloat16*>(p.out) + (row0 + cb) * kD + tk);
                tc_fence_before();
            }
            if (failed) {
                fail(p, ctrl, kErrWaitTimeout, site, i);
                report(p, kRoleSoftmax, site, i);
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int NP, bool LSU>
cudaError_t go(const DecodeMaps& maps, const DecodeParams& p, int W, int GY, cudaStream_t stream) {
    static std::atomic<uint64_t> done;
    const auto k = mla_decode_page8_kernel<NP, LSU>;
    const cudaError_t e = attribute_once(done, reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         p8_smem<NP, LSU>());
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(W, GY), P8Cfg<NP, LSU>::kThreads, p8_smem<NP, LSU>(), stream, attr);
    return cudaLaunchKernelEx(&cfg, k, maps, p);
}

}  // namespace

cudaError_t launch_decode_page8(const DecodeMaps& maps, const DecodeParams& p, int NP, bool lsu, int W, int GY,
                                cudaStream_t stream) {
    const cudaError_t e = NP == 16   ? (lsu ? go<16, true>(maps, p, W, GY, stream) : go<16, false>(maps, p, W, GY, stream))
                          : NP == 32 ? (lsu ? go<32, true>(maps, p, W, GY, stream) : go<32, false>(maps, p, W, GY, stream))
                                     : (lsu ? go<64, true>(maps, p, W, GY, stream) : go<64, false>(maps, p, W, GY, stream));
    return e == cudaSuccess ? launch_decode_merge(p, W, W * GY, GY, stream) : e;
}

}  // namespace mla
