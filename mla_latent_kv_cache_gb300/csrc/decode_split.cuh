// What the decode kernels and their merge share: the walk over the requests'
// tiles, the split of the work between CTAs, query rows of a request, status
// records and paged addressing.
#pragma once
#include <climits>

#include "launch.cuh"
#include "mla_common.cuh"

namespace mla {

__device__ __forceinline__ int swz_p(int row, uint32_t mode) {
    return mode == kSw128 ? (row & 7) : mode == kSw64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
}

// Walks the tiles (1 << SH tokens each) of consecutive requests.
template <int SH>
struct TileItT {
    int b, j, tiles, T;
    __device__ __forceinline__ void init(const int32_t* sl, int b0, int j0) {
        b = b0;
        j = j0;
        T = max(__ldg(sl + b), 0);
        tiles = (T + (1 << SH) - 1) >> SH;
    }
    __device__ __forceinline__ void next(const int32_t* sl, int B) {
        if (++j >= tiles) {
            j = 0;
            do {
                ++b;
                if (b >= B) { T = 0; tiles = 1; break; }
                T = max(__ldg(sl + b), 0);
                tiles = (T + (1 << SH) - 1) >> SH;
            } while (tiles == 0);
        }
    }
};
using TileIt = TileItT<7>;

// Query rows of request b: the first row of its verify step and the step's
// length in tokens (Qt for every request unless per-request lengths are given),
// and how many of its rows fall in row group gy (0 .. 64). Per-request prefix
// sums are clamped to [0, total_q], so whatever they hold no row past the
// query, output and LSE buffers is touched (a request whose sums run past
// total_q keeps its tokens below it).
__device__ __forceinline__ int cu_clamped(const DecodeParams& p, int b) {
    return min(max(__ldg(p.cu_q + b), 0), p.total_q);
}
__device__ __forceinline__ int64_t req_row0(const DecodeParams& p, int b) {
    return p.cu_q ? static_cast<int64_t>(cu_clamped(p, b)) * p.Hq : static_cast<int64_t>(b) * p.HQ;
}
__device__ __forceinline__ int req_qt(const DecodeParams& p, int b) {
    return p.cu_q ? cu_clamped(p, b + 1) - cu_clamped(p, b) : p.Qt;
}
__device__ __forceinline__ int req_rows_in_group(const DecodeParams& p, int b, int gy) {
    return min(64, max(0, req_qt(p, b) * p.Hq - gy * 64));
}

// L2 prefetch of what the first tiles of request b read besides the cache:
// its query rows of row group gy and its block-table row (whole 16-byte
// units inside the row only).
__device__ __forceinline__ void prefetch_request(const DecodeParams& p, int b, int gy) {
    const int HQg = req_rows_in_group(p, b, gy);
    const int64_t row0 = req_row0(p, b) + gy * 64;
    if (HQg > 0) {
        prefetch_l2_bulk(p.q_lat + row0 * p.lat_dim, static_cast<uint32_t>(HQg * p.lat_dim * 2));
        prefetch_l2_bulk(p.q_pe + row0 * p.rope_dim, static_cast<uint32_t>(HQg * p.rope_dim * 2));
    }
    const int T = max(__ldg(p.seq_lens + b), 0);
    const int64_t pages = min((static_cast<int64_t>(T) + p.page_size - 1) / p.page_size, p.bt_stride);
    uintptr_t a0 = reinterpret_cast<uintptr_t>(p.block_table + static_cast<int64_t>(b) * p.bt_stride);
    uintptr_t a1 = a0 + static_cast<uintptr_t>(pages) * 4;
    a0 = (a0 + 15) & ~static_cast<uintptr_t>(15);
    a1 &= ~static_cast<uintptr_t>(15);
    if (a1 > a0) {
        const uintptr_t n = a1 - a0;
        prefetch_l2_bulk(reinterpret_cast<const void*>(a0), static_cast<uint32_t>(n < (1u << 20) ? n : (1u << 20)));
    }
}

// Work split. Tiles of all requests in order form one sequence; a non-empty
// request also carries wseg units of cost before its first tile (what a
// request boundary costs a cluster: the next request's queries, the drain of
// the previous output). Cluster g of G takes the tiles whose cost coordinate
// lies in [g*C/G, (g+1)*C/G), C the total cost. Both functions are called by
// a whole warp and return the same value in every lane.

// Total tiles and total cost over all requests.
template <int SH>
__device__ __forceinline__ void work_totals(const int32_t* sl, int B, int wseg, int lane, long long& tiles,
                                            long long& cost) {
    long long t = 0, c = 0;
    for (int base = 0; base < B; base += 32) {
        const int b = base + lane;
        const int tl = b < B ? (max(__ldg(sl + b), 0) + (1 << SH) - 1) >> SH : 0;
        int st = tl, sc = tl > 0 ? tl + wseg : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            st += __shfl_xor_sync(0xffffffffu, st, o);
            sc += __shfl_xor_sync(0xffffffffu, sc, o);
        }
        t += st;
        c += sc;
    }
    tiles = t;
    cost = c;
}

// Number of tiles whose cost coordinate is below x.
template <int SH>
__device__ __forceinline__ long long tiles_before_cost(const int32_t* sl, int B, int wseg, long long x, int lane) {
    long long acc_c = 0, acc_t = 0;
    for (int base = 0; base < B; base += 32) {
        const int b = base + lane;
        const int tl = b < B ? (max(__ldg(sl + b), 0) + (1 << SH) - 1) >> SH : 0;
        const int cb = tl > 0 ? tl + wseg : 0;
        int ic = cb, it = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int vc = __shfl_up_sync(0xffffffffu, ic, o);
            const int vt = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) {
                ic += vc;
                it += vt;
            }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, b < B && acc_c + ic > x);
        if (hit) {
            const int L = __ffs(hit) - 1;
            const long long cs = acc_c + __shfl_sync(0xffffffffu, ic, L) - __shfl_sync(0xffffffffu, cb, L);
            const long long ts = acc_t + __shfl_sync(0xffffffffu, it, L) - __shfl_sync(0xffffffffu, tl, L);
            const long long in = x - cs - wseg;  // tiles of request L below x
            return ts + (in > 0 ? in : 0);
        }
        acc_c += __shfl_sync(0xffffffffu, ic, 31);
        acc_t += __shfl_sync(0xffffffffu, it, 31);
    }
    return acc_t;
}

// Tile range [tb, te) of worker g of G and the request / tile it starts at.
// Called by a whole warp; every lane returns the same values.
struct TileRange {
    int tb, te, b0, j0;
};
template <int SH>
__device__ __forceinline__ TileRange scan_range(const DecodeParams& p, int g, int G, int lane) {
    long long total = 0, cost = 0;
    work_totals<SH>(p.seq_lens, p.B, p.wseg, lane, total, cost);
    const int tb = static_cast<int>(tiles_before_cost<SH>(p.seq_lens, p.B, p.wseg, g * cost / G, lane));
    const int te = static_cast<int>(tiles_before_cost<SH>(p.seq_lens, p.B, p.wseg, (g + 1) * cost / G, lane));
    int b0 = 0, j0 = 0;
    long long acc = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const int tl = b < p.B ? (max(__ldg(p.seq_lens + b), 0) + (1 << SH) - 1) >> SH : 0;
        int incl = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const long long gi = acc + incl;
        const unsigned hit = __ballot_sync(0xffffffffu, b < p.B && tl > 0 && gi > tb);
        if (hit) {
            const int L = __ffs(hit) - 1;
            const long long gl = __shfl_sync(0xffffffffu, gi, L);
            const int tll = __shfl_sync(0xffffffffu, tl, L);
            b0 = base + L;
            j0 = static_cast<int>(tb - (gl - tll));
            break;
        }
        acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    TileRange r;
    r.tb = tb;
    r.te = te;
    r.b0 = b0;
    r.j0 = j0;
    return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int NP>
__device__ __forceinline__ void tmem_ld_np(uint32_t taddr, uint32_t (&r)[NP]) {
    if constexpr (NP == 8) tmem_ld_x8(taddr, r);
    else if constexpr (NP == 16) tmem_ld_x16(taddr, r);
    else if constexpr (NP == 32) tmem_ld_x32(taddr, r);
    else tmem_ld_x64(taddr, r);
}

// Wait sites, recorded with the first failure (workspace header words 1..3:
// site, tile index within the CTA's range, linear block index).
enum WaitSite : int {
    kSiteQFull = 1, kSiteSFree, kSitePairFull, kSiteRopeFull, kSitePFull, kSiteTmaPairEmpty, kSiteTmaRopeEmpty,
    kSiteLsuPairEmpty, kSiteLsuRopeEmpty, kSiteSFull, kSiteXFree, kSiteXFull, kSiteOEpi, kSiteORescale, kSiteOPbuf,
    kSiteOFinal, kSiteRawFull, kSiteDFull, kSitePIn, kSiteRpFree
};

// This CTA's status record; zeroed by the CTA itself at launch and folded
// into the workspace header by the merge step.
__device__ __forceinline__ int* status_rec(const DecodeParams& p) {
    return p.rec + static_cast<int64_t>(blockIdx.y * gridDim.x + blockIdx.x) * kStatusRecWords;
}

template <class CT>
__device__ __forceinline__ void fail(const DecodeParams& p, CT* ctrl, int code, int site = 0, int tile = 0) {
    int* r = status_rec(p);
    atomicOr(r, code);
    if (site && atomicCAS(r + 1, 0, site) == 0) r[2] = tile;
    ctrl->abort = 1;
}

// Every softmax thread waits, then the 128 threads agree on the outcome, so a
// timeout seen by some of them cannot strand the rest at a named barrier.
// When a role leaves its loop on a failed wait it records where it was
// waiting: record word 4 + role = (site << 24) | tile.
enum Role : int { kRoleS = 0, kRolePV, kRoleSoftmax, kRoleTma, kRoleLsu0 };

__device__ __forceinline__ void report(const DecodeParams& p, int role, int site, int idx) {
    status_rec(p)[4 + role] = (site << 24) | (idx & 0xFFFFFF);
}

// Softmax-group wait. A thread whose wait fails raises the abort flag and
// carries on (its results no longer matter); the group leaves its tile loop
// together after the tile's last barrier, where every thread reads the flag.
template <class CT>
__device__ __forceinline__ bool group_wait(uint64_t* bar, uint32_t parity, const DecodeParams& p, CT* ctrl,
                                           int site, int tile, bool cluster_scope = false) {
    const bool ok = cluster_scope ? mbar_wait_cluster(bar, parity, &ctrl->abort) : mbar_wait(bar, parity, &ctrl->abort);
    if (!ok) {
        fail(p, ctrl, kErrWaitTimeout, site, tile);
        report(p, kRoleSoftmax, site, tile);
    }
    return ok;
}

// 64-bit slot of token `tok` of the request whose block-table row is `btr`.
__device__ __forceinline__ int64_t token_slot(const DecodeParams& p, const int32_t* btr, int tok, bool& bad) {
    const int pi = tok / p.page_size;
    // a page index past the block-table row (a sequence longer than the table)
    // counts as an entry outside the pool
    const int64_t page = pi < p.bt_stride ? __ldg(btr + pi) : -1;
    const int64_t ps = p.page_size;
    if (page < 0 || (page + 1) * ps > p.num_slots) {
        bad = true;
        return tok % p.page_size;  // page 0: in bounds, flagged
    }
    return page * ps + tok % p.page_size;
}

}  // namespace mla
