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
// Two kernels. The select kernel: a cluster of up to 16 CTAs per request, each
// with a contiguous part of the tokens whose keys stay in the threads'
// registers over all passes (evict_select_kernel; up to 524,288 tokens), or in
// shared memory as far as they fit (evict_select_long_kernel); histograms and
// counts are combined through distributed shared memory. evict_move_kernel:
// all SMs copy the listed rows, whatever request they belong to, by bulk
// copies through shared memory, with two batches of rows a warp in flight.
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

// Any number of tokens: keys in shared memory, formed again past `cap`.
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_long_kernel(const EvictParams p, int cap) {
    extern __shared__ uint32_t keys[];
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = static_cast<int>(blockIdx.x) / CL;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();  // the kernel before may still be writing the inputs
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

// Sum over the warps before this one, and over all, of one value per warp
// (given by every lane). One barrier; buf holds kSelWarps values.
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t* buf, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    const uint32_t mine = buf[lane];
    total = __reduce_add_sync(0xffffffffu, mine);
    return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u);
}

struct SelectRegShared {
    uint32_t hist[3][kSelBins];        // this CTA's counts of each digit
    uint32_t slice[3][kSelBins / 2];   // the cluster's counts of this CTA's slice of the bins
    uint32_t slice_total[3];
    uint32_t warp[6][kSelWarps];  // per-warp values of the passes
    int newest;
    uint32_t ties, moves;         // this CTA's counts, read by the cluster
    uint32_t bin[3], above[3], count[3];  // the chosen bin of each digit, the keys above it, and in it
};

// Up to KPT keys a thread, in registers: warp w of the CTA holds the span of
// 32 kn consecutive tokens at t0 + 32 kn w, lane l its tokens l, l + 32, ...
template <int KPT>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p) {
    __shared__ __align__(16) SelectRegShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = static_cast<int>(blockIdx.x) / CL;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto meet = [&]() {
        if (CL > 1) cluster.sync();
        else __syncthreads();
    };
    griddep_wait();  // the kernel before may still be writing the inputs
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

    const int kn = ((T + CL - 1) / CL + kSelThreads - 1) / kSelThreads;  // keys a thread, <= KPT
    const int t0 = min(rank * kn * kSelThreads, T), t1 = min(t0 + kn * kSelThreads, T);
    const int at0 = t0 + warp * kn * 32 + lane;  // this thread's tokens: at0 + 32 k < t1

    if (T <= K) {
        // nothing goes
        for (int i = t0 + tid; i < t1; i += kSelThreads) {
            if (copy) nw[i] = w[i];
            if (copyp) np[i] = pos[i];
        }
        meet();  // every part has read its length
        if (rank == 0 && tid == 0) {
            moves[0] = 0;
            moves[1] = K;
            p.new_lens[b] = K;
            if (T0 > T && p.status) atomicOr(p.status, kErrBadBlock);
        }
        return;
    }

    // ---- the newest position, which the protected recent ones are counted from
    // (up to 16 tokens a thread: their scores are asked for at once and both are held;
    // else eight of each at a time)
    constexpr bool kHold = KPT <= 16;
    constexpr int kIn = kHold ? KPT : 8;
    uint32_t key[KPT];  // a score's bits at first
    int ps[kIn];
    auto read = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kIn; ++k) {
            const int i = at0 + 32 * (k0 + k);
            const bool in = k0 + k < kn && i < t1;
            key[k0 + k] = in ? __float_as_uint(w[i]) : 0u;
            ps[k] = in ? pos[i] : INT_MIN;
        }
    };
    int mx = INT_MIN;
    if (kHold) {
        read(0);
#pragma unroll
        for (int k = 0; k < kIn; ++k) mx = max(mx, ps[k]);
    } else {
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
            const int i = at0 + 32 * k;
            mx = max(mx, k < kn && i < t1 ? pos[i] : INT_MIN);
        }
    }
    for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    if (CL > 1)
        for (int i = tid; i < 3 * (kSelBins / 2) + 3; i += kSelThreads) (&sh.slice[0][0])[i] = 0;  // and the totals
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) sh.warp[0][warp] = static_cast<uint32_t>(mx);
    __syncthreads();
    int newest = __reduce_max_sync(0xffffffffu, static_cast<int>(sh.warp[0][lane]));
    if (CL > 1) {
        if (tid == 0) sh.newest = newest;
        cluster.sync();
        newest = __reduce_max_sync(0xffffffffu, lane < CL ? *cluster.map_shared_rank(&sh.newest, lane) : INT_MIN);
    }
    const int64_t recent_from = static_cast<int64_t>(newest) + 1 - p.n_recent;
    // keys. Entries below K go to the new arrays as they are: the places whose token
    // goes are written again when their new token moves in.
#pragma unroll
    for (int k0 = 0; k0 < KPT; k0 += kIn) {
        if (k0 >= kn) break;
        if (!kHold) read(k0);
#pragma unroll
        for (int k = 0; k < kIn; ++k) {
            const int i = at0 + 32 * (k0 + k);
            const float wk = __uint_as_float(key[k0 + k]);
            key[k0 + k] = evict_key(wk, ps[k] < p.n_sink || ps[k] >= recent_from);
            if (k0 + k < kn && i < min(t1, K)) {
                if (copy) nw[i] = wk;
                if (copyp) np[i] = ps[k];
            }
        }
    }

    // ---- radix select of the K-th largest key; it ends early where all keys of a bin stay
    uint32_t prefix = 0, want = static_cast<uint32_t>(K);  // the `want`-th largest among keys that start with prefix
    int low = 32;                                          // bits not yet decided
    bool rank_ties = false;                                // of the keys equal to the threshold only the first `want` stay
    if (K > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass == 2 ? 10 : 11, shift = low - bits;
            const uint32_t mask = (1u << bits) - 1u;
            uint32_t* hist = sh.hist[pass];
#pragma unroll
            for (int k = 0; k < KPT; ++k) {
                if (k >= kn) break;
                const bool hit = at0 + 32 * k < t1 && (pass == 0 || (key[k] >> low) == prefix);
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                if (m == 0) continue;
                const uint32_t d = (key[k] >> shift) & mask;
                // equal digits all through the warp (decayed scores are often all
                // zero) would queue up on one counter: count them at once
                const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
                if (__all_sync(0xffffffffu, !hit || d == d0)) {
                    if (lane == 0) atomicAdd(hist + d0, static_cast<uint32_t>(__popc(m)));
                } else if (hit) {
                    atomicAdd(hist + d, 1u);
                }
            }
            // the bin in which the want-th largest falls: threads hold bins from the top
            // down, so that a scan over threads counts keys from the top
            uint32_t c_hi, c_lo = 0, above0 = 0;
            int top;  // this thread's upper bin
            if (CL > 1) {
                // each CTA holds the cluster's sums of a slice of the bins, into which the
                // others add theirs (every CTA reading all bins of all others is 16
                // times the traffic: 9 us a digit); the slices' totals then say which
                // slice to look into
                __syncthreads();
                const int S = kSelBins / CL;
                uint32_t* slice = sh.slice[pass];
                const int bin = 2 * tid, to = bin / S;  // (a warp's 64 bins lie in one slice)
                const uint2 h = *reinterpret_cast<const uint2*>(hist + bin);
                uint32_t* sums = cluster.map_shared_rank(slice + bin % S, to);
                if (h.x) atomicAdd(sums, h.x);
                if (h.y) atomicAdd(sums + 1, h.y);
                const uint32_t sum = __reduce_add_sync(0xffffffffu, h.x + h.y);
                if (lane == 0 && sum) atomicAdd(cluster.map_shared_rank(&sh.slice_total[pass], to), sum);
                cluster.sync();
                const uint32_t mine = lane < CL ? *cluster.map_shared_rank(&sh.slice_total[pass], lane) : 0u;
                uint32_t up = mine;  // keys in this slice and those above it
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const uint32_t y = __shfl_down_sync(0xffffffffu, up, o);
                    if (lane + o < 32) up += y;
                }
                const int owner = __ffs(__ballot_sync(0xffffffffu, up - mine < want && want <= up)) - 1;
                above0 = __shfl_sync(0xffffffffu, up - mine, owner);
                top = owner * S + S - 1 - tid;
                c_hi = tid < S ? *cluster.map_shared_rank(slice + S - 1 - tid, owner) : 0u;
            } else {
                __syncthreads();
                top = kSelBins - 1 - 2 * tid;
                c_hi = hist[top];
                c_lo = hist[top - 1];
            }
            uint32_t x = c_hi + c_lo;  // inclusive scan over the warp
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            uint32_t total;
            const uint32_t base = warps_before(__shfl_sync(0xffffffffu, x, 31), sh.warp[1 + pass], total);
            const uint32_t above = above0 + base + x - c_hi - c_lo;
            if (above < want && want <= above + c_hi) {
                sh.bin[pass] = top;
                sh.above[pass] = above;
                sh.count[pass] = c_hi;
            } else if (above + c_hi < want && want <= above + c_hi + c_lo) {
                sh.bin[pass] = top - 1;
                sh.above[pass] = above + c_hi;
                sh.count[pass] = c_lo;
            }
            __syncthreads();
            prefix = (prefix << bits) | sh.bin[pass];
            want -= sh.above[pass];
            low = shift;
            if (sh.count[pass] == want) break;
            rank_ties = pass == 2;
        }
    }
    const uint32_t thr = K > 0 ? prefix << low : 0u;

    // ---- what stays, as bits: k of this thread
    uint32_t keep = 0, tie = 0;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const bool in = k < kn && at0 + 32 * k < t1 && K > 0;
        keep |= (in && (rank_ties ? key[k] > thr : key[k] >= thr) ? 1u : 0u) << k;
        tie |= (in && rank_ties && key[k] == thr ? 1u : 0u) << k;
    }
    if (rank_ties) {  // by place: ties in the CTAs, the warps and the groups of 32 before
        uint32_t total;
        uint32_t before = warps_before(__reduce_add_sync(0xffffffffu, __popc(tie)), sh.warp[4], total);
        if (CL > 1) {
            if (tid == 0) sh.ties = total;
            cluster.sync();
            const uint32_t t = lane < rank ? *cluster.map_shared_rank(&sh.ties, lane) : 0u;
            before += __reduce_add_sync(0xffffffffu, t);
        }
        for (int k = 0; k < kn; ++k) {
            const unsigned m = __ballot_sync(0xffffffffu, tie >> k & 1u);
            if ((tie >> k & 1u) && before + __popc(m & ((1u << lane) - 1u)) < want) keep |= 1u << k;
            before += __popc(m);
        }
    }

    // ---- the free places below K, the kept tokens above, and how many lie before
    uint32_t in_bits = 0, below = 0;  // this thread's tokens, and those at places below K
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = at0 + 32 * k;
        in_bits |= (k < kn && i < t1 ? 1u : 0u) << k;
        below |= (k < kn && i < min(t1, K) ? 1u : 0u) << k;
    }
    const uint32_t holes = ~keep & below, srcs = keep & in_bits & ~below;
    // (a CTA has at most 32,768 of either: two counts in one sum)
    uint32_t total;
    uint32_t n = warps_before(__reduce_add_sync(0xffffffffu, __popc(holes) | __popc(srcs) << 16), sh.warp[5], total);
    uint32_t hole = n & 0xFFFFu, src = n >> 16, n_moves = total & 0xFFFFu;
    if (CL > 1) {
        if (tid == 0) sh.moves = total;
        cluster.sync();
        const uint32_t t = lane < CL ? *cluster.map_shared_rank(&sh.moves, lane) : 0u;
        hole += __reduce_add_sync(0xffffffffu, lane < rank ? t & 0xFFFFu : 0u);
        src += __reduce_add_sync(0xffffffffu, lane < rank ? t >> 16 : 0u);
        n_moves = __reduce_add_sync(0xffffffffu, t & 0xFFFFu);
    }

    // ---- the lists: move r takes the token at moves[2 + 2r] to place moves[3 + 2r]
    const unsigned lower = (1u << lane) - 1u;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        if (k >= kn) break;
        const int i = at0 + 32 * k;
        const bool is_hole = holes >> k & 1u, is_src = srcs >> k & 1u;
        const unsigned mh = __ballot_sync(0xffffffffu, is_hole), ms = __ballot_sync(0xffffffffu, is_src);
        if (is_src) moves[2 + 2 * static_cast<int64_t>(src + __popc(ms & lower))] = i;
        if (is_hole) moves[3 + 2 * static_cast<int64_t>(hole + __popc(mh & lower))] = i;
        src += __popc(ms);
        hole += __popc(mh);
    }
    meet();  // every part has read its length and the others' counts
    if (rank == 0 && tid == 0) {
        moves[0] = static_cast<int32_t>(n_moves);
        moves[1] = K;
        p.new_lens[b] = K;
        if (T0 > T && p.status) atomicOr(p.status, kErrBadBlock);
    }
}

// Copies the listed rows. The moves of all requests form one sequence (of rows,
// or of kStage-byte pieces of longer rows), dealt out to warps in batches of
// what a stage holds: a lane looks one row up and copies it into shared memory
// and out again by bulk copies. A warp loads a batch while the one before is
// written.
constexpr int kMoveThreads = 384;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kStage = 9216;     // bytes of a batch: eight 1,152-byte rows

struct MoveShared {
    uint64_t full[kMoveWarps][2];
    uint32_t first[kMoveReqs + 1];
    uint32_t wsum[kMoveWarps];
    int abort;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's stores have read their shared memory.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int reqs) {
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ MoveShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = kMoveReqs / kMoveThreads;
    if (tid == 0) {
        for (int i = 0; i < kMoveWarps; ++i)
            for (int k = 0; k < 2; ++k) mbar_init(&sh.full[i][k], 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    // pieces a row has, and rows or pieces of a batch (at most a warp's lanes)
    const int pieces = (p.row_bytes + kStage - 1) / kStage;
    const int batch = pieces > 1 ? 1 : min(32, kStage / p.row_bytes);
    uint8_t* stage = stages + warp * 2 * kStage;
    bool bad = false, ok = true;
    uint32_t loads = 0;  // batches this warp has asked for
    // the batch on its way: this lane's target and bytes
    uint8_t* out = nullptr;
    uint32_t out_bytes = 0;
    auto write_last = [&]() {  // writes batch loads - 1 once it has landed
        const uint32_t k = loads - 1;
        if (ok && !__all_sync(0xffffffffu, mbar_wait(&sh.full[warp][k & 1], (k >> 1) & 1, &sh.abort))) ok = false;
        if (ok && out_bytes) bulk_store(out, stage + (k & 1) * kStage + lane * (pieces > 1 ? 0 : p.row_bytes), out_bytes);
        bulk_commit();
    };
    griddep_wait();
    if (tid == 0) griddep_launch_dependents();
    for (int b0 = 0; b0 < p.B; b0 += reqs) {
        const int nb = min(reqs, p.B - b0);
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
        if (lane == 31) sh.wsum[warp] = x;
        __syncthreads();
        uint32_t run = x - sum;
        for (int k = 0; k < warp; ++k) run += sh.wsum[k];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            sh.first[tid * kPer + k] = run;
            run += c[k];
        }
        if (tid == kMoveThreads - 1) sh.first[kMoveReqs] = run;
        __syncthreads();
        const uint64_t total = static_cast<uint64_t>(sh.first[kMoveReqs]) * pieces;
        const uint64_t step = static_cast<uint64_t>(gridDim.x) * kMoveWarps * batch;
        // this lane's row (or piece) of the batch at m0: looked up while the batch
        // before is on its way
        const uint8_t* from = nullptr;
        uint8_t* to = nullptr;
        uint32_t bytes = 0;
        auto look_up = [&](uint64_t m0) {
            const uint64_t item = m0 + lane;
            bytes = 0;
            if (lane >= batch || item >= total) return;
            const uint32_t m = static_cast<uint32_t>(pieces > 1 ? item / pieces : item);
            const uint32_t piece = static_cast<uint32_t>(item - static_cast<uint64_t>(m) * pieces);
            int lo = 0, hi = nb;  // the last request whose first move is <= m
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sh.first[mid] <= m) lo = mid;
                else hi = mid;
            }
            const int64_t b = b0 + lo;
            const int32_t* mv = p.moves + b * p.moves_stride + 2 + 2 * static_cast<int64_t>(m - sh.first[lo]);
            const int s = mv[0], d = mv[1];
            if (piece == 0) {
                p.new_weights[b * p.stride + d] = p.weights[b * p.stride + s];
                p.new_positions[b * p.stride + d] = p.positions[b * p.stride + s];
            }
            const int32_t* bt = p.block_table + b * p.bt_stride;
            const int64_t sp = __ldg(bt + s / p.page_size), dp = __ldg(bt + d / p.page_size);
            const int64_t ss = sp * p.page_size + s % p.page_size, ds = dp * p.page_size + d % p.page_size;
            // a page outside the pool: the row is not moved
            if (sp < 0 || dp < 0 || ss >= p.num_slots || ds >= p.num_slots) {
                bad = true;
                return;
            }
            const int64_t off = static_cast<int64_t>(piece) * kStage;
            from = p.cache + ss * p.row_bytes + off;
            to = p.cache + ds * p.row_bytes + off;
            bytes = static_cast<uint32_t>(min(static_cast<int64_t>(kStage), p.row_bytes - off));
        };
        uint64_t m0 = (static_cast<uint64_t>(warp) * gridDim.x + blockIdx.x) * batch;
        if (m0 < total) look_up(m0);
        for (; m0 < total && ok; m0 += step) {
            // the stores of batch loads - 2 have left its stage
            bulk_wait_read();
            __syncwarp();
            const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
            uint64_t* bar = &sh.full[warp][loads & 1];
            if (lane == 0) mbar_arrive_expect_tx(bar, all);
            __syncwarp();
            if (bytes) bulk_load(stage + (loads & 1) * kStage + lane * (pieces > 1 ? 0 : p.row_bytes), from, bytes, bar);
            if (loads > 0) write_last();
            ++loads;
            out = to;
            out_bytes = bytes;
            if (m0 + step < total) look_up(m0 + step);
        }
        if (loads > 0) {
            write_last();
            // the next requests' batches count on: none is on its way
            out_bytes = 0;
        }
        __syncthreads();
    }
    bulk_wait_read();
    if (!ok) {
        // no copy may arrive after the CTA is gone
        volatile int never = 0;
        for (uint32_t k = loads < 2 ? 0 : loads - 2; k < loads; ++k) mbar_wait(&sh.full[warp][k & 1], (k >> 1) & 1, &never);
        if (lane == 0) {
            sh.abort = 1;
            if (p.status) atomicOr(p.status, kErrWaitTimeout);
        }
    }
    if (bad && p.status) atomicOr(p.status, kErrBadBlock);
}

template <int KPT>
cudaError_t launch_select(const cudaLaunchConfig_t& cfg, const EvictParams& p) {
    // clusters of 16
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attribute_once(done, reinterpret_cast<const void*>(evict_select_kernel<KPT>),
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<KPT>, p);
}

// CTAs of the largest cluster of the select kernels that the current device can
// run: 16 (which is not portable) on a whole GPU, fewer on a part of one. The
// kernels' threads and registers leave one CTA to an SM, so one answers for all.
int largest_cluster() {
    static std::atomic<int> largest[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    if (const int n = largest[dev].load(std::memory_order_relaxed)) return n;
    auto* k = evict_select_kernel<32>;
    int CL = 16;
    // (a size that does not fit is no error of a later launch)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        CL = 8;
    }
    for (; CL > 1; CL /= 2) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CL;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(CL);
        cfg.blockDim = dim3(kSelThreads);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
        if (e == cudaSuccess && n > 0) break;
        if (e != cudaSuccess) (void)cudaGetLastError();
    }
    largest[dev].store(CL, std::memory_order_relaxed);
    return CL;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int sms, int most_ctas, cudaStream_t stream) {
    int most = largest_cluster();
    while (most > 1 && most_ctas > 0 && most > most_ctas) most /= 2;
    // CTAs that share a request's tokens: 8 keys a thread where there are SMs for
    // it, up to 32 otherwise
    int CL = 1;
    while (CL < most && p.max_len > CL * 8 * kSelThreads) CL *= 2;
    auto keys = [&](int cl) { return ((p.max_len + cl - 1) / cl + kSelThreads - 1) / kSelThreads; };
    while (CL > 1 && static_cast<int64_t>(CL) * p.B > sms && keys(CL / 2) <= 32) CL /= 2;
    const int kpt = keys(CL);
    if (kpt > 32) CL = most < 8 ? most : 8;  // evict_select_long_kernel
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(CL) * p.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e;
    if (kpt <= 4) {
        e = launch_select<4>(cfg, p);
    } else if (kpt <= 8) {
        e = launch_select<8>(cfg, p);
    } else if (kpt <= 16) {
        e = launch_select<16>(cfg, p);
    } else if (kpt <= 32) {
        e = launch_select<32>(cfg, p);
    } else {
        static std::atomic<uint64_t> done{0};
        e = attribute_once(done, reinterpret_cast<const void*>(evict_select_long_kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
        if (e != cudaSuccess) return e;
        cfg.dynamicSmemBytes = kSelCap * 4;
        e = cudaLaunchKernelEx(&cfg, evict_select_long_kernel, p, kSelCap);
    }
    if (e != cudaSuccess) return e;
    constexpr int kMoveSmem = kMoveWarps * 2 * kStage;
    static std::atomic<uint64_t> move_done{0};
    e = attribute_once(move_done, reinterpret_cast<const void*>(evict_move_kernel),
                       cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t mc = {};
    cudaLaunchAttribute ma[1];
    ma[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ma[0].val.programmaticStreamSerializationAllowed = 1;
    mc.gridDim = dim3(static_cast<unsigned>(sms));
    mc.blockDim = dim3(kMoveThreads);
    mc.dynamicSmemBytes = kMoveSmem;
    mc.stream = stream;
    mc.attrs = ma;
    mc.numAttrs = 1;
    return cudaLaunchKernelEx(&mc, evict_move_kernel, p, evict_requests_at_once(p.max_len));
}

}  // namespace mla
