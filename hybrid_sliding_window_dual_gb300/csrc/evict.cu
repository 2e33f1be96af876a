// Which pages of a sequence stay when its Full cache is cut to a budget.
//
// The heaviest pages stay (the attention weight that hswa_decode_weights
// accumulated), beside the first pages and everything within the last
// `recent` tokens. One CTA per sequence holds a row's weights in registers as
// ordered integers, neighbours in a thread, and bisects between the smallest
// and the largest: how many are at or above the middle? Once no more
// candidates are left in between than threads, each takes one. It ends as
// soon as the answer is the number that stays, or at a single weight, of
// whose pages the lower ones stay. One scan in page order places the pages.
//
// Bound by latency: a row is a few KB, and the loads, 10 to 20 rounds of a
// barrier each and the scan follow one another. 64 rows of up to 512 pages
// take 4.2 us on the device, 128 of 2048 6.1, 5 of 16384 20. A radix
// selection, 8 bits a pass, took 7.2, 11 and 50 (the weights' first bits are
// nearly all alike, so that its counters collide); one warp per row 5.9 on
// the first; the row in shared memory instead of registers 8.0, 10 and 23.
#include "common.cuh"
#include "internal.h"

namespace hswa {
namespace {

// Weights in order as unsigned integers; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (w != w) return 0;
    const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelectArgs {
    const int32_t *seq_len;
    const float *w_in;
    const int32_t *budget;
    int32_t sink, recent, page, max_pages;
    int32_t *keep, *n_keep;
    float *w_out;
};

// kItems pages a thread in registers. kLong: rows longer than kThreads *
// kItems; the bisection then reads the row again each time (it lies in L2),
// and the pages are placed one stretch of that many after the other.
template <int kItems, int kThreads, bool kLong>
__global__ void __launch_bounds__(kThreads) evict_select(const SelectArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ int32_t s_count[2][kWarps], s_sure[kWarps], s_tied[kWarps];
    __shared__ uint32_t s_min[kWarps], s_max[kWarps], s_few[kThreads];
    __shared__ int32_t s_few_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t s = blockIdx.x;
    const float *w = a.w_in + s * a.max_pages;
    int32_t *keep = a.keep + s * a.max_pages;
    float *w_out = a.w_out + s * a.max_pages;
    // this thread's pages of a stretch, and their order
    float x[kItems];
    uint32_t key[kItems];
    int32_t first = tid * kItems;
    const bool wide = ((uintptr_t)w & 15) == 0;
    const auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kItems; k += 4) {
            if (wide && first + k + 4 <= a.max_pages) {
                const float4 y = *reinterpret_cast<const float4 *>(w + first + k);
                x[k] = y.x, x[k + 1] = y.y, x[k + 2] = y.z, x[k + 3] = y.w;
            } else {
#pragma unroll
                for (int i = k; i < k + 4; ++i) x[i] = first + i < a.max_pages ? w[first + i] : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) key[k] = order_of(x[k]);
    };
    load();
    const int64_t L = max(a.seq_len[s], 0);
    const int32_t pages = (int32_t)min((L + a.page - 1) / a.page, (int64_t)a.max_pages);
    // pages [c0, c1) may go
    const int32_t c0 = min(a.sink, pages);
    const int32_t c1 = max(c0, L > a.recent ? (int32_t)min((L - a.recent) / a.page, (int64_t)pages) : 0);
    const int32_t fixed = pages - (c1 - c0);
    const int32_t n_keep = min(pages, max(a.budget[s], fixed));
    const int32_t left = n_keep - fixed;  // candidates that stay
    const auto may_go = [&](int32_t p) { return p >= c0 && p < c1; };
    // f(order) of this thread's candidates
    const auto each_candidate = [&](auto f) {
        if constexpr (kLong) {
            for (int32_t p = c0 + tid; p < c1; p += kThreads) f(order_of(w[p]));
        } else {
#pragma unroll
            for (int k = 0; k < kItems; ++k)
                if (may_go(first + k)) f(key[k]);
        }
    };
    // Candidates above `bound` in order of weight stay, and `quota` at most of
    // those at it, the lower pages.
    uint32_t bound = 0xffffffffu;  // no weight's order
    int32_t quota = 0;
    if (left == c1 - c0) {
        bound = 0;
        quota = INT32_MAX;
    } else if (left > 0) {
        uint32_t lo = 0xffffffffu, hi = 0;
        each_candidate([&](uint32_t o) { lo = min(lo, o), hi = max(hi, o); });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) s_min[warp] = lo, s_max[warp] = hi;
        if (tid == 0) s_few_n = 0;
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? s_min[lane] : 0xffffffffu);
        hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? s_max[lane] : 0u);
        // `upto` >= left candidates are at or above lo, `above` < left above hi
        int32_t above = 0, upto = c1 - c0;
        bool exact = false, few = false;
        uint32_t mine = 0;      // few: one of the candidates in [lo, hi] of then, or 0,
        int32_t few_above = 0;  // and how many were above them
        for (int round = 0; lo < hi && !exact; round ^= 1) {
            if (kItems > 4 && !few && upto - above <= kThreads) {
                // a thread each for those still in question
                few = true;
                few_above = above;
                each_candidate([&](uint32_t o) {
                    if (o >= lo && o <= hi) s_few[atomicAdd(&s_few_n, 1)] = o;
                });
                __syncthreads();
                if (tid < upto - above) mine = s_few[tid];
            }
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int32_t n = 0;
            if (few)
                n = mine >= mid;
            else
                each_candidate([&](uint32_t o) { n += o >= mid; });
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) s_count[round][warp] = n;
            __syncthreads();
            n = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_count[round][lane] : 0) + few_above;
            exact = n == left;
            if (n >= left)
                lo = mid, upto = n;
            else
                hi = mid - 1, above = n;
        }
        bound = lo;
        quota = exact ? INT32_MAX : left - above;
    }
    // In page order: how many stay for sure before this thread's pages, and
    // how many at the bound come before them. w_out may be w_in: a page goes
    // to its own place or a lower one, after its stretch has been read.
    int32_t sure_before = 0, tied_before = 0;  // in the stretches before
    for (int32_t base = 0; base < pages; base += kThreads * kItems) {
        if (kLong) {
            first = base + tid * kItems;
            load();
        }
        int32_t sure = 0, tied = 0;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const bool there = first + k < pages, may = may_go(first + k);
            sure += there && (!may || key[k] > bound);
            tied += there && may && key[k] == bound;
        }
        int32_t sure_upto = sure, tied_upto = tied;
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, sure_upto, off), z = __shfl_up_sync(0xffffffffu, tied_upto, off);
            if (lane >= off) sure_upto += y, tied_upto += z;
        }
        if (lane == 31) s_sure[warp] = sure_upto, s_tied[warp] = tied_upto;
        __syncthreads();
        const int32_t y = lane < kWarps ? s_sure[lane] : 0, z = lane < kWarps ? s_tied[lane] : 0;
        int32_t t = tied_before + __reduce_add_sync(0xffffffffu, lane < warp ? z : 0) + tied_upto - tied;
        int32_t at = sure_before + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + sure_upto - sure + min(t, quota);
        if (kLong) {
            sure_before += __reduce_add_sync(0xffffffffu, y);
            tied_before += __reduce_add_sync(0xffffffffu, z);
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (first + k >= pages) continue;
            const bool tie = may_go(first + k) && key[k] == bound;
            if (!may_go(first + k) || key[k] > bound || (tie && t < quota)) {
                keep[at] = first + k;
                w_out[at] = x[k];
                ++at;
            }
            t += tie;
        }
        if (!kLong) break;
        __syncthreads();  // before the next stretch is read over the same sums
    }
    if (pages == 0) __syncthreads();  // every thread has read its pages
    for (int32_t p = n_keep + tid; p < a.max_pages; p += kThreads) {
        keep[p] = -1;
        w_out[p] = 0.f;
    }
    if (tid == 0) a.n_keep[s] = n_keep;
}

template <int kItems, int kThreads, bool kLong = false>
cudaError_t launch_select(const SelectArgs &a, int n_seqs, cudaStream_t st) {
    return launch_pdl(evict_select<kItems, kThreads, kLong>, dim3(n_seqs), dim3(kThreads), 0, st, a);
}

}  // namespace
}  // namespace hswa

using namespace hswa;

extern "C" int hswa_evict_select(const hswa_pool *pool, const int32_t *d_seq_len, const float *w_in,
                                 const int32_t *d_budget, int n_seqs, int sink_pages, int recent_tokens,
                                 int32_t *keep, int32_t *n_keep, float *w_out, hswa_stream_t stream) {
    HSWA_NVTX("hswa_evict_select");
    if (!pool || n_seqs < 0 || n_seqs > pool->cfg.max_seqs || sink_pages < 0 || recent_tokens < pool->cfg.window)
        return HSWA_ERR_INVALID_ARG;
    if (n_seqs == 0) return HSWA_OK;
    if (!d_seq_len || !w_in || !d_budget || !keep || !n_keep || !w_out) return HSWA_ERR_INVALID_ARG;
    if (overlap_but_differ(w_in, w_out, (size_t)n_seqs * pool->cfg.max_pages_per_seq * sizeof(float)))
        return HSWA_ERR_INVALID_ARG;
    const SelectArgs a = {d_seq_len, w_in, d_budget, sink_pages, recent_tokens, pool->cfg.page_size,
                          pool->cfg.max_pages_per_seq, keep, n_keep, w_out};
    set_last_kernel("evict_select");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int32_t n = a.max_pages;
    // threads for the row: fewer make cheaper barriers (a round takes 230
    // cycles with 128, 330 with 512 and 610 with 1024)
    const cudaError_t rc = n <= 512     ? launch_select<4, 128>(a, n_seqs, st)
                           : n <= 1024  ? launch_select<4, 256>(a, n_seqs, st)
                           : n <= 2048  ? launch_select<4, 512>(a, n_seqs, st)
                           : n <= 8192  ? launch_select<16, 512>(a, n_seqs, st)
                           : n <= 16384 ? launch_select<16, 1024>(a, n_seqs, st)
                                        : launch_select<16, 1024, true>(a, n_seqs, st);
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_evict_select");
}
