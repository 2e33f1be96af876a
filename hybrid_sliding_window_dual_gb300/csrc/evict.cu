// Which pages of a sequence stay when its Full cache is cut to a budget.
//
// The heaviest pages stay (the attention weight that hswa_decode_weights
// accumulated), beside the first pages and everything within the last
// `recent` tokens. One CTA per sequence holds a row's weights in registers as
// ordered integers. It counts the candidates in bins that cut the range from
// the smallest to the largest into equal parts, takes the bin that the answer
// lies in for the next range, and ends when that holds as many candidates as
// still stay, or one weight, of whose pages the lower ones stay, or so few
// candidates that each can count those above it. One scan in page order
// places the pages.
//
// Bound by latency: a row is a few KB, and the loads, the steps with a barrier
// each and the scan follow one another, much of it by instructions that run
// for the first time. On the device 64 rows of 512 pages take 3.3 us, 152 of
// 2048 4.4, 8 of 16384, split, 8.1; rows beyond that 32 to 37 (32768 pages, one
// CTA that reads the row from L2 for every count).
//
// (A bisection of the range, one barrier a bit, took 4.2 us on 64 rows of up
// to 512 pages, 6.1 on 128 of 2048 and 20 on 5 of 16384, now 3.3, 4.2 and 7.1; a
// radix selection, 8 bits a pass, 7.2, 11 and 50: the weights' first bits are
// nearly all alike, so that its counters collide. A thread's pages next to
// each other made placing them 1.6 times as long: its loads and stores are
// 64 bytes apart over a warp.)
#include <algorithm>

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
    int32_t row_keys;  // keys of a table row, INT32_MAX at most
    int *err;
    int32_t ctas;  // of a row
};

constexpr int kMaxCtas = 8;

// kItems pages a thread in registers, 32 neighbours in a warp's lanes.
// kSplit: a cluster of a.ctas CTAs takes a row, each its stretch of kThreads *
// kItems pages; they read each other's counts through distributed shared
// memory, and each of them finds the answer. kLong: longer rows, by one CTA;
// the counts then read the row again each time (it lies in L2), and the pages
// are placed one stretch after the other.
template <int kItems, int kThreads, bool kSplit, bool kLong>
__global__ void __launch_bounds__(kThreads) evict_select(const SelectArgs a) {
    constexpr int kWarps = kThreads / 32, kBinBits = kThreads <= 256 || kSplit ? 9 : kThreads == 512 ? 10 : 11, kBins = 1 << kBinBits;
    constexpr int kPer = kBins / kThreads, kStretch = kThreads * kItems;
    constexpr int kFew = 128;  // candidates that count each other
    constexpr int kMost = kSplit ? kMaxCtas : 1;
    static_assert(!kSplit || (kPer == 1 && kWarps >= kMaxCtas), "a bin a thread, a warp a CTA");
    __shared__ int32_t s_bin[1 + kSplit][kBins], s_sum[kWarps], s_tied[kWarps], s_found[3], s_few_n, s_few[kFew], s_all[kFew];
    __shared__ uint32_t s_min[kWarps], s_max[kWarps];
    __shared__ uint64_t s_range[kMost], s_place[kMost];  // from each CTA
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned before_me = (1u << lane) - 1;
    const int ctas = kSplit ? a.ctas : 1, rank = kSplit ? blockIdx.x % ctas : 0;
    if constexpr (kSplit) cluster_arrive();  // awaited before the first store into another CTA's shared memory
    pdl_wait();
    pdl_launch_dependents();
    const int64_t s = kSplit ? blockIdx.x / ctas : blockIdx.x;
    const float *w = a.w_in + s * a.max_pages;
    int32_t *keep = a.keep + s * a.max_pages;
    float *w_out = a.w_out + s * a.max_pages;
    // this thread's pages of a stretch, and their order
    float x[kItems];
    uint32_t key[kItems];
    int32_t first = rank * kStretch + warp * kItems * 32 + lane;  // the k-th is 32 k further
    const auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kItems; ++k) x[k] = first + 32 * k < a.max_pages ? w[first + 32 * k] : 0.f;
#pragma unroll
        for (int k = 0; k < kItems; ++k) key[k] = order_of(x[k]);
    };
    load();
    // a length ends where its table row does, as in decode with page weights
    const int32_t asked = a.seq_len[s], L = min(max(asked, 0), a.row_keys);
    const int32_t pages = (int32_t)(((uint32_t)L + (uint32_t)a.page - 1) / (uint32_t)a.page);
    // pages [c0, c1) may go
    const int32_t c0 = min(a.sink, pages);
    const int32_t c1 = max(c0, L > a.recent ? (L - a.recent) / a.page : 0);
    const int32_t fixed = pages - (c1 - c0);
    const int32_t n_keep = min(pages, max(a.budget[s], fixed));
    const int32_t left = n_keep - fixed;  // candidates that stay
    for (int32_t p = n_keep + rank * kThreads + tid; p < a.max_pages; p += ctas * kThreads) keep[p] = -1;
    if (rank == 0 && tid == 0) {
        a.n_keep[s] = n_keep;
        if (asked > L) set_error(a.err, HSWA_ERR_BOUNDS);
    }
    if constexpr (kSplit) cluster_wait();  // every CTA of the cluster has started
    const auto may_go = [&](int32_t p) { return p >= c0 && p < c1; };
    // f(is a candidate, its order), by whole warps
    const auto each_page = [&](auto f) {
        if constexpr (kLong) {
            for (int32_t p = c0 + tid; p - lane < c1; p += kThreads) f(p < c1, p < c1 ? order_of(w[p]) : 0u);
        } else {
#pragma unroll
            for (int k = 0; k < kItems; ++k) f(may_go(first + 32 * k), key[k]);
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
        each_page([&](bool may, uint32_t o) {
            if (may) lo = min(lo, o), hi = max(hi, o);
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) s_min[warp] = lo, s_max[warp] = hi;
        if (tid == 0) s_few_n = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) s_bin[0][tid * kPer + k] = 0;
        if (kSplit) s_bin[kSplit][tid] = 0;
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? s_min[lane] : 0xffffffffu);
        hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? s_max[lane] : 0u);
        if constexpr (kSplit) {
            if (tid < ctas) st_cluster_u64(&s_range[rank], tid, (uint64_t)hi << 32 | lo);
            cluster_arrive();
            cluster_wait();
            for (int i = 0; i < ctas; ++i) lo = min(lo, (uint32_t)s_range[i]), hi = max(hi, (uint32_t)(s_range[i] >> 32));
        }
        // `above` < left candidates are above hi, `here` in [lo, hi], and with
        // those at least `left`
        int32_t above = 0, here = c1 - c0;
        bool all = false;  // all of [lo, hi] stay
        // each time the range loses kBinBits of its at most 32 bits
        for (int pass = 0; pass < (32 + kBinBits - 1) / kBinBits && lo < hi && !all && here > kFew; ++pass) {
            const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
            int32_t *bin = s_bin[kSplit ? pass & 1 : 0];
            each_page([&](bool may, uint32_t o) {
                const bool in = may && o >= lo && o <= hi;
                const uint32_t b = (hi - o) >> shift;  // heavier bins first
                const unsigned mask = __ballot_sync(0xffffffffu, in);
                if (mask == 0) return;
                // many weights may be alike: one count for those in the first one's bin
                const int one = __ffs(mask) - 1;
                const uint32_t of_one = __shfl_sync(0xffffffffu, b, one);  // by every lane
                const bool same = in && b == of_one;
                const unsigned with = __ballot_sync(0xffffffffu, same);
                if (in && (!same || lane == one)) atomicAdd(&bin[b], same ? __popc(with) : 1);
            });
            int32_t n[kPer] = {}, sum = 0;
            if constexpr (kSplit) {
                cluster_arrive();
                cluster_wait();
#pragma unroll
                for (int i = 0; i < kMaxCtas; ++i)
                    if (i < ctas) sum += ld_cluster_i32(&bin[tid], i);
                n[0] = sum;
                // the other bins have been read by all; the sums' barriers come before they are counted in again
                s_bin[(pass & 1) ^ 1][tid] = 0;
            } else {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    sum += n[k] = bin[tid * kPer + k];
                    bin[tid * kPer + k] = 0;
                }
            }
            int32_t upto = sum;
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            if (lane == 31) s_sum[warp] = upto;
            __syncthreads();
            int32_t at = above + upto - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (at < left && at + n[k] >= left) s_found[0] = tid * kPer + k, s_found[1] = at, s_found[2] = n[k];
                at += n[k];
            }
            __syncthreads();
            const uint32_t width = (1u << shift) - 1;
            hi -= (uint32_t)s_found[0] << shift;
            if (hi - lo > width) lo = hi - width;
            above = s_found[1];
            here = s_found[2];
            all = above + here == left;
        }
        if (lo < hi && !all) {  // `here` is at most kFew now
            each_page([&](bool may, uint32_t o) {
                if (may && o >= lo && o <= hi) {
                    const int32_t i = atomicAdd(&s_few_n, 1);
                    if (i < kFew) s_few[i] = (int32_t)o;  // more only if another stream changes the weights meanwhile
                }
            });
            const int32_t *few = s_few;
            if constexpr (kSplit) {  // everyone's, a warp for each CTA
                cluster_arrive();
                cluster_wait();
                const int32_t n = lane < ctas ? ld_cluster_i32(&s_few_n, lane) : 0;
                const int32_t from = __reduce_add_sync(0xffffffffu, lane < warp ? n : 0), its = __shfl_sync(0xffffffffu, n, warp);
                for (int32_t i = lane; i < its && from + i < kFew; i += 32) s_all[from + i] = ld_cluster_i32(&s_few[i], warp);
                few = s_all;
            }
            __syncthreads();
            here = min(here, kFew);
            if (tid < here) {
                const uint32_t mine = (uint32_t)few[tid];
                int32_t over = above, upto = above;
#pragma unroll 8
                for (int i = 0; i < here; ++i) over += (uint32_t)few[i] > mine, upto += (uint32_t)few[i] >= mine;
                if (over < left && upto >= left) s_found[0] = (int32_t)mine, s_found[1] = over;  // equal ones write the same
            }
            __syncthreads();
            lo = (uint32_t)s_found[0];
            above = s_found[1];
        }
        bound = lo;
        quota = all ? INT32_MAX : max(left - above, 0);
    }
    // In page order: how many stay before this warp's pages, and up to which
    // page those at the bound do. w_out may be w_in: a page goes to its own
    // place or a lower one, after its stretch has been read (kSplit: all).
    int32_t before = 0, tied_before = 0;  // sure and tied ones in the stretches before
    for (int32_t base = 0; base < pages; base += kStretch) {
        if (kLong) {
            first = base + warp * kItems * 32 + lane;
            load();
        }
        uint32_t sure = 0, tied = 0;  // bit k: this thread's k-th page
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int32_t p = first + 32 * k;
            sure |= p < pages && (!may_go(p) || key[k] > bound) ? 1u << k : 0u;
            tied |= may_go(p) && key[k] == bound ? 1u << k : 0u;
        }
        const int32_t n_sure = __reduce_add_sync(0xffffffffu, __popc(sure));
        const int32_t n_tied = __reduce_add_sync(0xffffffffu, __popc(tied));
        if (lane == 0) s_sum[warp] = n_sure, s_tied[warp] = n_tied;
        __syncthreads();
        const int32_t y = lane < kWarps ? s_sum[lane] : 0, z = lane < kWarps ? s_tied[lane] : 0;
        if constexpr (kSplit) {
            const uint64_t sums = (uint64_t)__reduce_add_sync(0xffffffffu, z) << 32 | (uint32_t)__reduce_add_sync(0xffffffffu, y);
            if (tid < ctas) st_cluster_u64(&s_place[rank], tid, sums);
            cluster_arrive();
            cluster_wait();
            for (int i = 0; i < rank; ++i) before += (int32_t)s_place[i], tied_before += (int32_t)(s_place[i] >> 32);
        }
        const int32_t ties = tied_before + __reduce_add_sync(0xffffffffu, lane < warp ? z : 0);  // before this warp's
        int32_t n = before + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + min(ties, quota);
        if (kLong) {
            before += __reduce_add_sync(0xffffffffu, y);
            tied_before += __reduce_add_sync(0xffffffffu, z);
        }
        uint32_t stay = sure | tied;
        if (ties + n_tied > quota) {  // by whole warps: some of its ties go
            stay = sure;
            int32_t t = ties;
            for (int k = 0; k < kItems; ++k) {
                const unsigned m = __ballot_sync(0xffffffffu, tied >> k & 1);
                if ((tied >> k & 1) && t + __popc(m & before_me) < quota) stay |= 1u << k;
                t += __popc(m);
            }
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const unsigned m = __ballot_sync(0xffffffffu, stay >> k & 1);
            if (stay >> k & 1) {
                const int32_t at = n + __popc(m & before_me);
                keep[at] = first + 32 * k;
                w_out[at] = x[k];
            }
            n += __popc(m);
        }
        if (!kLong) break;
        __syncthreads();  // before the next stretch is read over the same sums
    }
    if (pages == 0) __syncthreads();  // every thread has read its pages
    for (int32_t p = n_keep + rank * kThreads + tid; p < a.max_pages; p += ctas * kThreads) w_out[p] = 0.f;
}

// CTAs of 2048 pages to a row.
int split_ctas(int32_t max_pages) {
    int n = 2;
    while (n * 2048 < max_pages) n *= 2;
    return n;
}

template <int kItems, int kThreads, bool kSplit = false, bool kLong = false>
cudaError_t launch_select(SelectArgs a, int n_seqs, cudaStream_t st) {
    if constexpr (kSplit) {
        a.ctas = split_ctas(a.max_pages);
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = a.ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)n_seqs * a.ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, evict_select<kItems, kThreads, kSplit, kLong>, a);
    } else {
        return launch_pdl(evict_select<kItems, kThreads, kSplit, kLong>, dim3(n_seqs), dim3(kThreads), 0, st, a);
    }
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
                          pool->cfg.max_pages_per_seq, keep, n_keep, w_out,
                          (int32_t)std::min((int64_t)pool->cfg.max_pages_per_seq * pool->cfg.page_size, (int64_t)INT32_MAX),
                          error_word(), 1};
    set_last_kernel("evict_select");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int32_t n = a.max_pages;
    // Threads for the row: fewer make cheaper barriers. Long rows are split as
    // long as every CTA has an SM of its own (8 rows of 16384 pages 8.1 us, by
    // one CTA each 13.7; 64 of 4096 6.7 and 9.1, but 64 of 8192 11.9 and 9.1,
    // 64 of 16384 22 and 14).
    const int sms = sm_count();
    if (sms <= 0) return HSWA_ERR_CUDA;
    const bool split = n > 2048 && n <= 2048 * kMaxCtas && (int64_t)n_seqs * split_ctas(n) <= sms;
    const cudaError_t rc = n <= 512     ? launch_select<4, 128>(a, n_seqs, st)
                           : n <= 1024  ? launch_select<4, 256>(a, n_seqs, st)
                           : n <= 2048  ? launch_select<4, 512>(a, n_seqs, st)
                           : split      ? launch_select<4, 512, true>(a, n_seqs, st)
                           : n <= 8192  ? launch_select<16, 512>(a, n_seqs, st)
                           : n <= 16384 ? launch_select<16, 1024>(a, n_seqs, st)
                                        : launch_select<16, 1024, false, true>(a, n_seqs, st);
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_evict_select");
}
