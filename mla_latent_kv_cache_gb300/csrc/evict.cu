// Eviction from the paged latent cache by score (mla_cache_evict): of each
// request's T cached tokens the K best stay, and the K rows are closed up in
// the request's first K places.
//
// Mathematics. A token's key is its score as an order-preserving 32-bit
// number (protected tokens above everything, NaN below everything); the kept
// set is the K largest keys, equal keys by lower place. The threshold is found
// by a radix select from the top (11, 11 and 10 bits): a histogram of the keys
// that agree with the digits found so far, the bin in which the K-th largest
// falls, and the next digit inside it.
//
// Why the gaps are filled instead of the rows shifted: a token that stays and
// already lies in the first K places does not move; every place below K whose
// token goes is filled by a kept token from above K (both in ascending order).
// Attention does not depend on the order of cached rows (the rotary part is
// baked into a row), the sources (>= K) and the targets (< K) are disjoint, so
// the copies need no order among themselves and the call can be repeated with
// the same result, and the rows moved are the fewest that any closing-up must
// move: one per step in the steady state, where a shift would move them all.
//
// Two kernels. evict_select_kernel: a cluster of CL CTAs per request, each with
// a contiguous part of the tokens whose keys stay in shared memory over all
// passes; histograms and counts are combined through distributed shared
// memory. evict_move_kernel: all SMs copy the listed rows, whatever request
// they belong to.
#include <climits>

#include <cooperative_groups.h>

#include "launch.cuh"
#include "mla_common.cuh"

namespace mla {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
// keys a CTA keeps in shared memory; the rest are formed again from the scores on every pass
constexpr int kSelCap = 49152;

struct SelectShared {
    uint32_t hist[kSelBins];      // this CTA's counts of the current digit, read by the cluster
    uint32_t scan[kSelWarps + 1];
    int newest;                   // largest position in this CTA's part
    uint32_t ties, holes, srcs;   // this CTA's counts, read by the cluster
    uint32_t bin, above;          // the chosen bin and the keys above it
};

__device__ __forceinline__ uint32_t evict_key(float w, bool safe) {
    if (safe) return 0xFFFFFFFFu;
    if (!(w == w)) return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 and 0 are one score
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Scan over the block of one value per thread: returns the exclusive value,
// and the block's total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* scan, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const uint32_t s = scan[lane];
        uint32_t z = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        scan[lane] = z - s;
        if (lane == 31) scan[kSelWarps] = z;
    }
    __syncthreads();
    total = scan[kSelWarps];
    const uint32_t r = scan[warp] + x - v;
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p, int cap) {
    extern __shared__ uint32_t keys[];
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = static_cast<int>(blockIdx.x) / CL;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) griddep_launch_dependents();

    const int T0 = max(__ldg(p.seq_lens + b), 0);
    // tokens that neither the score rows nor the table row hold are not there
    const int64_t held = min(static_cast<int64_t>(p.max_len), p.bt_stride * p.page_size);
    const int T = static_cast<int>(min(static_cast<int64_t>(T0), held));
    const int K = min(max(__ldg(p.budgets + b), 0), T);
    const float* w = p.weights + b * p.stride;
    const int32_t* pos = p.positions + b * p.stride;
    float* nw = p.new_weights + b * p.stride;
    int32_t* np = p.new_positions + b * p.stride;
    int32_t* moves = p.moves + b * p.moves_stride;
    const bool copy = nw != w, copyp = np != pos;

    // this CTA's tokens [t0, t1), a warp's [s0, s1): spans of a multiple of 32
    const int per = ((T + CL - 1) / CL + kSelThreads - 1) / kSelThreads * kSelThreads;
    const int t0 = static_cast<int>(min(static_cast<int64_t>(rank) * per, static_cast<int64_t>(T)));
    const int t1 = min(t0 + per, T);
    const int span = per / kSelWarps;
    const int s0 = min(t0 + warp * span, t1), s1 = min(s0 + span, t1);

    if (T <= K) {
        // nothing goes
        for (int i = t0 + tid; i < t1; i += kSelThreads) {
            if (copy) nw[i] = w[i];
            if (copyp) np[i] = pos[i];
        }
        cluster.sync();  // every part has read its length
        if (rank == 0 && tid == 0) {
            moves[0] = 0;
            moves[1] = K;
            p.new_lens[b] = K;
            if (T0 > T && p.status) atomicOr(p.status, kErrBadBlock);
        }
        return;
    }

    // ---- the newest position, which the protected recent ones are counted from
    int mx = INT_MIN;
    for (int i = s0 + lane; i < s1; i += 32) mx = max(mx, pos[i]);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) sh.scan[warp] = static_cast<uint32_t>(mx);
    for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    if (warp == 0) {
        mx = __reduce_max_sync(0xffffffffu, static_cast<int>(sh.scan[lane]));
        if (lane == 0) sh.newest = mx;
    }
    cluster.sync();
    int newest = INT_MIN;
    for (int c = 0; c < CL; ++c) newest = max(newest, *cluster.map_shared_rank(&sh.newest, c));
    const int64_t recent_from = static_cast<int64_t>(newest) + 1 - p.n_recent;

    auto make_key = [&](int i) -> uint32_t {
        const int ps = pos[i];
        return evict_key(w[i], ps < p.n_sink || ps >= recent_from);
    };
    auto key_at = [&](int i) -> uint32_t { return i - t0 < cap ? keys[i - t0] : make_key(i); };

    // ---- radix select of the K-th largest key
    uint32_t prefix = 0, want = static_cast<uint32_t>(K);  // the `want`-th largest among keys that start with prefix
    uint32_t kth = 0, ties_kept = 0;
    const bool have = K > 0;
    if (have) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            const uint32_t mask = (1u << bits) - 1u;
            for (int i0 = s0; i0 < s1; i0 += 32) {
                const int i = i0 + lane;
                const bool in = i < s1;
                uint32_t k = 0;
                if (in) {
                    if (pass == 0) {
                        k = make_key(i);
                        if (i - t0 < cap) keys[i - t0] = k;
                    } else {
                        k = key_at(i);
                    }
                }
                const bool hit = in && (pass == 0 || (k >> (shift + bits)) == prefix);
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                if (m == 0) continue;
                const uint32_t d = (k >> shift) & mask;
                // equal digits all through the warp (decayed scores are often all
                // zero) would queue up on one counter: count them at once
                const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
                if (__all_sync(0xffffffffu, !hit || d == d0)) {
                    if (lane == 0) atomicAdd(&sh.hist[d0], static_cast<uint32_t>(__popc(m)));
                } else if (hit) {
                    atomicAdd(&sh.hist[d], 1u);
                }
            }
            cluster.sync();
            // thread t holds the bins 2047 - 2t and 2046 - 2t, so that an ascending
            // scan over threads counts keys from the top
            const int hb = kSelBins - 1 - 2 * tid;
            uint32_t c_hi = 0, c_lo = 0;
            for (int c = 0; c < CL; ++c) {
                const uint32_t* h = cluster.map_shared_rank(sh.hist, c);
                c_hi += h[hb];
                c_lo += h[hb - 1];
            }
            uint32_t total;
            const uint32_t above = block_scan(c_hi + c_lo, sh.scan, total);
            if (above < want && want <= above + c_hi) {
                sh.bin = hb;
                sh.above = above;
            } else if (above + c_hi < want && want <= above + c_hi + c_lo) {
                sh.bin = hb - 1;
                sh.above = above + c_hi;
            }
            cluster.sync();  // all histograms read, and the bin is there
            prefix = (prefix << bits) | sh.bin;
            want -= sh.above;
            for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[i] = 0;
            __syncthreads();
        }
        kth = prefix;
        ties_kept = want;  // of the keys equal to kth, the first `want` in order of place stay
    }

    // ---- ties before this warp's span
    uint32_t n_tie = 0;
    if (have)
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane;
            n_tie += __popc(__ballot_sync(0xffffffffu, i < s1 && key_at(i) == kth));
        }
    uint32_t total;
    uint32_t tie_base = block_scan(lane == 0 ? n_tie : 0u, sh.scan, total);
    tie_base = __shfl_sync(0xffffffffu, tie_base, 0);
    if (tid == 0) sh.ties = total;
    cluster.sync();
    for (int c = 0; c < rank; ++c) tie_base += *cluster.map_shared_rank(&sh.ties, c);

    // ---- what stays: count the free places below K and the kept tokens above
    uint32_t n_hole = 0, n_src = 0, tie = tie_base;
    auto kept_at = [&](int i, uint32_t& run) -> bool {  // run: ties before this group of 32
        const uint32_t k = (have && i < s1) ? key_at(i) : 0u;
        const bool is_tie = have && i < s1 && k == kth;
        const unsigned m = __ballot_sync(0xffffffffu, is_tie);
        const uint32_t before = run + __popc(m & ((1u << lane) - 1u));
        run += __popc(m);
        return have && i < s1 && (k > kth || (is_tie && before < ties_kept));
    };
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const bool kp = kept_at(i, tie);
        n_hole += __popc(__ballot_sync(0xffffffffu, i < s1 && i < K && !kp));
        n_src += __popc(__ballot_sync(0xffffffffu, i < s1 && i >= K && kp));
    }
    uint32_t th, ts;
    uint32_t hole = block_scan(lane == 0 ? n_hole : 0u, sh.scan, th);
    uint32_t src = block_scan(lane == 0 ? n_src : 0u, sh.scan, ts);
    hole = __shfl_sync(0xffffffffu, hole, 0);
    src = __shfl_sync(0xffffffffu, src, 0);
    if (tid == 0) {
        sh.holes = th;
        sh.srcs = ts;
    }
    cluster.sync();
    uint32_t n_moves = 0;
    for (int c = 0; c < CL; ++c) {
        const uint32_t hc = *cluster.map_shared_rank(&sh.holes, c), sc = *cluster.map_shared_rank(&sh.srcs, c);
        if (c < rank) {
            hole += hc;
            src += sc;
        }
        n_moves += hc;
    }

    // ---- the lists: move r takes the token at moves[2 + 2r] to place moves[3 + 2r]
    tie = tie_base;
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const bool kp = kept_at(i, tie);
        const bool is_hole = i < s1 && i < K && !kp, is_src = i < s1 && i >= K && kp;
        const unsigned mh = __ballot_sync(0xffffffffu, is_hole), ms = __ballot_sync(0xffffffffu, is_src);
        const unsigned below = (1u << lane) - 1u;
        if (is_src) moves[2 + 2 * static_cast<int64_t>(src + __popc(ms & below))] = i;
        if (is_hole) moves[3 + 2 * static_cast<int64_t>(hole + __popc(mh & below))] = i;
        src += __popc(ms);
        hole += __popc(mh);
        if (kp && i < K) {
            if (copy) nw[i] = w[i];
            if (copyp) np[i] = pos[i];
        }
    }
    if (rank == 0 && tid == 0) {
        moves[0] = static_cast<int32_t>(n_moves);
        moves[1] = K;
        p.new_lens[b] = K;  // after the cluster barriers above, so every part has read its length
        if (T0 > T && p.status) atomicOr(p.status, kErrBadBlock);
    }
    cluster.sync();  // no CTA leaves while another reads its counts
}

// Copies the listed rows. The moves of all requests form one sequence, dealt
// out to warps four rows at a time; a warp has all its loads in flight before
// the first store. UNITS: 16-byte units of a row (0: given at run time).
constexpr int kMoveRows = 4;
constexpr int kMoveThreads = 256;
constexpr int kMoveReqs = 1024;  // requests whose counts a CTA holds at once

template <int UNITS>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    __shared__ uint32_t first[kMoveReqs + 1];
    __shared__ uint32_t wsum[kMoveThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = UNITS > 0 ? UNITS : p.row_bytes / 16;
    constexpr int kMaxPer = UNITS > 0 ? (kMoveRows * UNITS + 31) / 32 : 8;
    constexpr int kPer = kMoveReqs / kMoveThreads;
    griddep_wait();
    bool bad = false;
    for (int b0 = 0; b0 < p.B; b0 += kMoveReqs) {
        const int nb = min(kMoveReqs, p.B - b0);
        // prefix sums of the counts of requests b0 .. b0 + nb (kPer a thread)
        uint32_t c[kPer], sum = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int b = tid * kPer + k;
            c[k] = b < nb ? static_cast<uint32_t>(p.moves[(b0 + b) * p.moves_stride]) : 0u;
            sum += c[k];
        }
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        uint32_t run = x - sum;
        for (int k = 0; k < warp; ++k) run += wsum[k];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            first[tid * kPer + k] = run;
            run += c[k];
        }
        if (tid == kMoveThreads - 1) first[kMoveReqs] = run;
        __syncthreads();
        const uint32_t total = first[kMoveReqs];
        const uint64_t step = static_cast<uint64_t>(gridDim.x) * (kMoveThreads / 32) * kMoveRows;
        for (uint64_t m0 = static_cast<uint64_t>(blockIdx.x * (kMoveThreads / 32) + warp) * kMoveRows; m0 < total; m0 += step) {
            const int n = static_cast<int>(min(static_cast<uint64_t>(kMoveRows), total - m0));
            // lane r < n looks up move m0 + r
            int64_t s_slot = -1, d_slot = -1;
            if (lane < n) {
                const uint32_t m = static_cast<uint32_t>(m0) + lane;
                int lo = 0, hi = nb;  // the last request whose first move is <= m
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (first[mid] <= m) lo = mid;
                    else hi = mid;
                }
                const int64_t b = b0 + lo;
                const int32_t* mv = p.moves + b * p.moves_stride + 2 + 2 * static_cast<int64_t>(m - first[lo]);
                const int s = mv[0], d = mv[1];
                p.new_weights[b * p.stride + d] = p.weights[b * p.stride + s];
                p.new_positions[b * p.stride + d] = p.positions[b * p.stride + s];
                const int32_t* bt = p.block_table + b * p.bt_stride;
                const int64_t sp = __ldg(bt + s / p.page_size), dp = __ldg(bt + d / p.page_size);
                s_slot = sp * p.page_size + s % p.page_size;
                d_slot = dp * p.page_size + d % p.page_size;
                // a page outside the pool: the row is not moved
                if (sp < 0 || dp < 0 || s_slot >= p.num_slots || d_slot >= p.num_slots) {
                    bad = true;
                    s_slot = d_slot = -1;
                }
            }
            const int all = n * units;
            for (int u0 = 0; u0 < all; u0 += 32 * kMaxPer) {
                uint4 v[kMaxPer];
#pragma unroll
                for (int k = 0; k < kMaxPer; ++k) {
                    const int u = u0 + k * 32 + lane;
                    const int r = min(u / units, kMoveRows - 1);
                    const int64_t s = __shfl_sync(0xffffffffu, s_slot, r);
                    if (u < all && s >= 0)
                        v[k] = *reinterpret_cast<const uint4*>(p.cache + s * p.row_bytes + (u - r * units) * 16);
                }
#pragma unroll
                for (int k = 0; k < kMaxPer; ++k) {
                    const int u = u0 + k * 32 + lane;
                    const int r = min(u / units, kMoveRows - 1);
                    const int64_t d = __shfl_sync(0xffffffffu, d_slot, r);
                    if (u < all && d >= 0)
                        *reinterpret_cast<uint4*>(p.cache + d * p.row_bytes + (u - r * units) * 16) = v[k];
                }
            }
        }
        __syncthreads();
    }
    if (bad && p.status) atomicOr(p.status, kErrBadBlock);
}

// CTAs that share a request's tokens.
int select_cluster(int max_len) { return max_len <= 8192 ? 1 : max_len <= 16384 ? 2 : max_len <= 32768 ? 4 : 8; }

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    const int CL = select_cluster(p.max_len);
    const int per = ((p.max_len + CL - 1) / CL + kSelThreads - 1) / kSelThreads * kSelThreads;
    const int cap = per < kSelCap ? per : kSelCap;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(CL) * p.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(cap) * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cap);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t mc = {};
    cudaLaunchAttribute ma[1];
    ma[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ma[0].val.programmaticStreamSerializationAllowed = 1;
    mc.gridDim = dim3(static_cast<unsigned>(4 * sms));
    mc.blockDim = dim3(kMoveThreads);
    mc.stream = stream;
    mc.attrs = ma;
    mc.numAttrs = 1;
    return p.row_bytes == kRowBf16  ? cudaLaunchKernelEx(&mc, evict_move_kernel<kRowBf16 / 16>, p)
           : p.row_bytes == kRowFp8 ? cudaLaunchKernelEx(&mc, evict_move_kernel<kRowFp8 / 16>, p)
                                    : cudaLaunchKernelEx(&mc, evict_move_kernel<0>, p);
}

}  // namespace mla
