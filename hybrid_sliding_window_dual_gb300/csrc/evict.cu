// Which pages of a sequence stay when its Full cache is cut to a budget.
//
// The heaviest pages stay (the attention weight that hswa_decode_weights
// accumulated), beside the first pages and everything within the last
// `recent` tokens. One CTA per sequence: a radix selection on the weights'
// ordered bits finds the weight of the last page that stays and how many
// pages of exactly that weight do (the lower ones), and a second pass over
// the pages in order writes the list and closes up the weights.
#include "common.cuh"
#include "internal.h"

namespace hswa {
namespace {

constexpr int kThreads = 1024;

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

__global__ void __launch_bounds__(kThreads) evict_select(const SelectArgs a) {
    __shared__ int32_t hist[256];
    __shared__ int32_t s_digit, s_left;
    __shared__ int32_t warp_kept[32], warp_tied[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t s = blockIdx.x;
    const float *w = a.w_in + s * a.max_pages;
    int32_t *keep = a.keep + s * a.max_pages;
    float *w_out = a.w_out + s * a.max_pages;
    const int64_t L = max(a.seq_len[s], 0);
    const int32_t pages = (int32_t)min((L + a.page - 1) / a.page, (int64_t)a.max_pages);
    // pages [c0, c1) may go
    const int32_t c0 = min(a.sink, pages);
    const int32_t c1 = max(c0, L > a.recent ? (int32_t)min((L - a.recent) / a.page, (int64_t)pages) : 0);
    const int32_t fixed = pages - (c1 - c0);
    const int32_t n_keep = min(pages, max(a.budget[s], fixed));
    int32_t left = n_keep - fixed;  // candidates that stay
    // the order of the last candidate that stays, digit by digit
    uint32_t bound = 0;
    if (left > 0 && left < c1 - c0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int32_t p = c0 + tid; p < c1; p += kThreads) {
                const uint32_t o = order_of(w[p]);
                if (shift == 24 || (o >> (shift + 8)) == (bound >> (shift + 8))) atomicAdd(&hist[(o >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {  // from the largest digit down, 8 digits a lane
                int32_t mine = 0;
                for (int i = 0; i < 8; ++i) mine += hist[255 - (lane * 8 + i)];
                int32_t upto = mine;
                for (int off = 1; off < 32; off <<= 1) {
                    const int32_t y = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += y;
                }
                if (upto >= left && upto - mine < left) {
                    int32_t rest = left - (upto - mine);
                    int i = 0;
                    while (hist[255 - (lane * 8 + i)] < rest) rest -= hist[255 - (lane * 8 + i++)];
                    s_digit = 255 - (lane * 8 + i);
                    s_left = rest;
                }
            }
            __syncthreads();
            bound |= (uint32_t)s_digit << shift;
            left = s_left;  // of the pages that agree so far, how many stay
            __syncthreads();
        }
    } else if (left > 0) {
        left = 0;  // every candidate stays: all are above the bound or equal to it
        bound = 0;
    }
    const bool all = n_keep - fixed == c1 - c0, none = n_keep == fixed;
    // in page order: the list, and the weights closed up
    int32_t kept = 0, tied = 0;  // so far
    for (int32_t base = 0; base < pages; base += kThreads) {
        const int32_t p = base + tid;
        const bool there = p < pages;
        const float x = there ? w[p] : 0.f;
        const uint32_t o = order_of(x);
        const bool may_go = p >= c0 && p < c1;
        const bool tie = there && may_go && !all && !none && o == bound;
        const unsigned tie_mask = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) warp_tied[warp] = __popc(tie_mask);
        __syncthreads();
        int32_t t = tied, t_all = tied;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) t += warp_tied[i];
            t_all += warp_tied[i];
        }
        t += __popc(tie_mask & ((1u << lane) - 1));
        tied = t_all;
        const bool stays = there && (!may_go || all || (!none && (o > bound || (tie && t < left))));
        const unsigned mask = __ballot_sync(0xffffffffu, stays);
        if (lane == 0) warp_kept[warp] = __popc(mask);
        __syncthreads();
        int32_t at = kept, k_all = kept;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) at += warp_kept[i];
            k_all += warp_kept[i];
        }
        at += __popc(mask & ((1u << lane) - 1));
        kept = k_all;
        if (stays) {  // at <= p: w_out may be w_in, whose pages up to base + 1023 every thread has read
            keep[at] = p;
            w_out[at] = x;
        }
        __syncthreads();
    }
    for (int32_t p = n_keep + tid; p < a.max_pages; p += kThreads) {
        keep[p] = -1;
        w_out[p] = 0.f;
    }
    if (tid == 0) a.n_keep[s] = n_keep;
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
    const SelectArgs a = {d_seq_len, w_in, d_budget, sink_pages, recent_tokens, pool->cfg.page_size,
                          pool->cfg.max_pages_per_seq, keep, n_keep, w_out};
    set_last_kernel("evict_select");
    evict_select<<<n_seqs, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t rc = cudaGetLastError();
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_evict_select");
}
