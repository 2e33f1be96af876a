// From a step's logits to the probabilities that verification takes: penalties
// for tokens that occurred, biases, grammar masks, temperature and softmax in
// one pass; and the token counts that the penalties read.
//
// Row r = i n_tok + w of sequence i. With c the times that token v has been
// generated (its count and its occurrences among the drafts before w):
//     z = logit; if v occurred (c > 0 or in the prompt): z > 0 ? z / rep : z rep
//     if c > 0: z -= frequency c, then z -= presence
//     z += bias; not allowed by the mask: z = -inf; NaN: z = -inf
//     p = softmax(z / T), or for T <= 0 one at the first largest z.
// Every step is rounded to fp32 as written, in this order.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace hswa {
namespace {

constexpr int kMaxCluster = 8;     // CTAs per row
constexpr int kBiasSlots = 2048;   // hash slots for at most half as many biases
constexpr int kMaxSlice = HSWA_VERIFY_MAX_VOCAB / kMaxCluster;

struct ProbsArgs {
    const void *logits;
    void *p;
    int64_t logits_stride, p_stride, count_stride, mask_stride;
    const float *params;      // [n_seqs][4]: temperature, repetition, frequency, presence
    const uint16_t *counts;
    const int32_t *draft;     // [n_seqs][n_tok - 1]
    const int32_t *bias_token;
    const float *bias;        // [n_seqs][n_bias]
    const uint32_t *mask;
    int32_t n_bias, n_tok, vocab, cluster, slice;  // slice: elements per CTA, a multiple of 8
    int *err;
};

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

struct ProbsSmem {
    int32_t key[kBiasSlots];  // token of a slot, -1: free
    int32_t at[kBiasSlots];   // the last entry of the bias list with that token
    uint32_t special[kMaxSlice / 8 / 32];  // groups of 8 tokens with a bias or a draft among them
    int32_t draft[HSWA_DECODE_MAX_TOKENS];
    float warp[32];
    uint64_t part[kMaxCluster];  // every CTA's (maximum, sum or first index)
};

__device__ __forceinline__ uint32_t bias_slot(int32_t token) { return (uint32_t)token * 0x9E3779B1u >> 21; }
static_assert(kBiasSlots == 1 << 11, "the hash keeps 11 bits");

// The row of a CTA, and what happens to its logits.
template <typename TL, bool kVec>
struct ProbsRow {
    const ProbsArgs &a;
    const ProbsSmem &sm;
    const TL *logits;
    const uint16_t *counts;
    const uint32_t *mask;
    const float *bias;
    int32_t lo, hi;  // this CTA's tokens
    int32_t w;
    bool specials;
    float rep, inv_rep, freq, pres;  // inv_rep 0: divide

    // Token of element e of group k of this thread (kVec: 8 neighbours, else 8
    // as far apart as the CTA has threads).
    __device__ __forceinline__ int32_t token(int32_t k, int e) const {
        return kVec ? lo + 8 * (k * (int32_t)blockDim.x + (int32_t)threadIdx.x) + e : lo + (8 * k + e) * (int32_t)blockDim.x + (int32_t)threadIdx.x;
    }

    __device__ __forceinline__ float penalized(float z, uint32_t c, int extra) const {
        const int32_t n = (int32_t)(c & 0x7fff) + extra;
        if (n > 0 || c >> 15) {
            if (inv_rep > 0.f) {
                // z / rep: the product with 1 / rep, corrected by its remainder
                float q = __fmul_rn(z, inv_rep);
                q = __fmaf_rn(__fmaf_rn(-rep, q, z), inv_rep, q);
                z = z > 0.f ? (z <= FLT_MAX ? q : z) : __fmul_rn(z, rep);
            } else {
                z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
            }
        }
        if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)n)), pres);
        return z;
    }

    __device__ __noinline__ float special(float z, uint32_t c, int32_t v) const {
        int extra = 0;
        if (counts)
            for (int j = 0; j < w; ++j) extra += sm.draft[j] == v;
        if (counts) z = penalized(z, c, extra);
        if (a.n_bias) {
            uint32_t s = bias_slot(v);
            while (sm.key[s] != -1 && sm.key[s] != v) s = (s + 1) & (kBiasSlots - 1);
            if (sm.key[s] == v) z = __fadd_rn(z, bias[sm.at[s]]);
        }
        return z;
    }

    // Group k: its 8 values of z, -inf behind the CTA's last token.
    __device__ __forceinline__ void load(int32_t k, float (&z)[8]) const {
        uint32_t c[8];
        uint32_t allowed = 0xff;
        const int32_t v0 = token(k, 0);
        if (kVec && v0 + 8 <= hi) {
            if constexpr (sizeof(TL) == 4) {
                const float4 x = reinterpret_cast<const float4 *>(logits + v0)[0], y = reinterpret_cast<const float4 *>(logits + v0)[1];
                z[0] = x.x, z[1] = x.y, z[2] = x.z, z[3] = x.w, z[4] = y.x, z[5] = y.y, z[6] = y.z, z[7] = y.w;
            } else {
                const uint4 x = *reinterpret_cast<const uint4 *>(logits + v0);
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) z[2 * e] = __uint_as_float(u[e] << 16), z[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
            uint4 n = make_uint4(0, 0, 0, 0);
            if (counts) n = *reinterpret_cast<const uint4 *>(counts + v0);
            const uint32_t u[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) c[2 * e] = u[e] & 0xffff, c[2 * e + 1] = u[e] >> 16;
            if (mask) allowed = reinterpret_cast<const uint8_t *>(mask)[v0 >> 3];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, e);
                z[e] = v < hi ? as_float(logits[v]) : -INFINITY;
                c[e] = counts && v < hi ? counts[v] : 0;
                if (mask && !(v < hi && mask[v >> 5] >> (v & 31) & 1)) allowed &= ~(1u << e);
            }
        }
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) any |= c[e];
        uint32_t spec = 0;
        if (specials) {
#pragma unroll
            for (int e = 0; e < 8; e += kVec ? 8 : 1) {
                const int32_t r = (token(k, e) - lo) >> 3;
                if (token(k, e) < hi) spec |= (sm.special[r >> 5] >> (r & 31) & 1) << e;
            }
        }
        if (spec) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, e);
                if (v < hi) z[e] = special(z[e], c[e], v);
            }
        } else if (any) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = penalized(z[e], c[e], 0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!(allowed >> e & 1) || z[e] != z[e]) z[e] = -INFINITY;
    }
};

template <typename TP, bool kVec>
__device__ __forceinline__ void store_probs(TP *p, int32_t v0, int32_t step, int32_t hi, const float (&x)[8]) {
    if (kVec && v0 + 8 <= hi) {
        if constexpr (sizeof(TP) == 4) {
            reinterpret_cast<float4 *>(p + v0)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4 *>(p + v0)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4 *>(p + v0) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int32_t v = v0 + e * step;
            if (v < hi) {
                if constexpr (sizeof(TP) == 4)
                    p[v] = x[e];
                else
                    p[v] = __float2bfloat16_rn(x[e]);
            }
        }
    }
}

__device__ __forceinline__ float block_max(float x, float *warp) {
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = x;
    __syncthreads();
    const int n = blockDim.x >> 5, lane = threadIdx.x & 31;
    x = lane < n ? warp[lane] : -INFINITY;
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();
    return x;
}

__device__ __forceinline__ float block_sum(float x, float *warp) {
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = x;
    __syncthreads();
    const int n = blockDim.x >> 5, lane = threadIdx.x & 31;
    x = lane < n ? warp[lane] : 0.f;
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    return x;
}

__device__ __forceinline__ int32_t block_min(int32_t x, float *warp) {
    x = __reduce_min_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = __int_as_float(x);
    __syncthreads();
    const int n = blockDim.x >> 5, lane = threadIdx.x & 31;
    x = __reduce_min_sync(0xffffffffu, lane < n ? __float_as_int(warp[lane]) : INT32_MAX);
    __syncthreads();
    return x;
}

// exp((z - top) / T) of a row's value: k is log2 e / T. A top of +inf shares
// the probability among the infinite values.
__device__ __forceinline__ float weight(float z, float top, float k) {
    if (z == -INFINITY) return 0.f;
    if (top == INFINITY) return z == INFINITY ? 1.f : 0.f;
    return fast_exp2((z - top) * k);
}

// A cluster per row, kGroups groups of 8 values per thread in registers between
// the one read and the one write; rows longer than that (kLoop) are read three
// times, for the maximum, the sum and the result.
template <typename TL, typename TP, bool kVec, int kThreads, int kGroups, bool kLoop>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logits_probs(const ProbsArgs a) {
    __shared__ ProbsSmem sm;
    const int tid = threadIdx.x;
    cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    const int32_t rank = blockIdx.x % a.cluster;
    const int64_t row = blockIdx.x / a.cluster;
    const int32_t seq = (int32_t)(row / a.n_tok), w = (int32_t)(row % a.n_tok);
    float temperature = 1.f, rep = 1.f, freq = 0.f, pres = 0.f;
    if (a.params) {
        const float *x = a.params + (int64_t)seq * 4;
        temperature = x[0], rep = x[1] > 0.f ? x[1] : 1.f, freq = x[2], pres = x[3];
    }
    const bool penalties = a.counts && !(rep == 1.f && freq == 0.f && pres == 0.f);
    const int32_t lo = min(rank * a.slice, a.vocab), hi = min(lo + a.slice, a.vocab);
    const bool drafts = penalties && a.draft && w > 0;
    ProbsRow<TL, kVec> r{a, sm, static_cast<const TL *>(a.logits) + row * a.logits_stride,
                         penalties ? a.counts + seq * a.count_stride : nullptr,
                         a.mask ? a.mask + row * a.mask_stride : nullptr,
                         a.bias + (int64_t)seq * a.n_bias, lo, hi, drafts ? w : 0, a.n_bias > 0 || drafts,
                         rep, rep >= 0x1p-64f && rep <= 0x1p64f ? __frcp_rn(rep) : 0.f, freq, pres};
    if (r.specials) {
        for (int i = tid; i < kBiasSlots; i += kThreads) sm.key[i] = sm.at[i] = -1;
        for (int i = tid; i < (a.slice / 8 + 31) / 32; i += kThreads) sm.special[i] = 0;
        __syncthreads();
        for (int i = tid; i < a.n_bias; i += kThreads) {
            const int32_t v = a.bias_token[(int64_t)seq * a.n_bias + i];
            if (v >= a.vocab) set_error(a.err, HSWA_ERR_BOUNDS);
            if (v < lo || v >= hi) continue;
            atomicOr(&sm.special[(v - lo) >> 8], 1u << ((v - lo) >> 3 & 31));
            uint32_t s = bias_slot(v);
            for (;;) {  // at most half of the slots are taken
                const int32_t was = atomicCAS(&sm.key[s], -1, v);
                if (was == -1 || was == v) break;
                s = (s + 1) & (kBiasSlots - 1);
            }
            atomicMax(&sm.at[s], i);
        }
        if (drafts && tid < w) {
            const int32_t v = a.draft[(int64_t)seq * (a.n_tok - 1) + tid];
            sm.draft[tid] = v;
            if (v >= lo && v < hi) atomicOr(&sm.special[(v - lo) >> 8], 1u << ((v - lo) >> 3 & 31));
        }
        __syncthreads();
    }
    const int32_t groups = kLoop ? (a.slice / 8 + kThreads - 1) / kThreads : kGroups;
    const bool greedy = !(temperature > 0.f);
    const float k = greedy ? 0.f : fminf(1.4426950408889634f / temperature, FLT_MAX);

    float z[kGroups][8];
    float top = -INFINITY;
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.load(g, z[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, z[0][e]);
        }
    } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            r.load(g, z[g]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, z[g][e]);
        }
    }
    top = block_max(top, sm.warp);  // of this CTA's tokens
    // this CTA's sum relative to it, or the first token that has it
    float sum = 0.f;
    int32_t first = INT32_MAX;
    const auto take = [&](int32_t g, float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (greedy) {
                if (x[e] == top && x[e] > -INFINITY) first = min(first, r.token(g, e));
            } else {
                x[e] = weight(x[e], top, k);
                sum += x[e];
            }
        }
    };
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.load(g, z[0]);
            take(g, z[0]);
        }
    } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) take(g, z[g]);
    }
    if (greedy)
        first = block_min(first, sm.warp);
    else
        sum = block_sum(sum, sm.warp);
    float all = top, total = sum, mine = 1.f;
    if (a.cluster > 1) {
        cluster_wait();  // every CTA of the cluster has started
        if (tid < a.cluster)
            st_cluster_u64(&sm.part[rank], tid, (uint64_t)__float_as_uint(top) << 32 | (greedy ? (uint32_t)first : __float_as_uint(sum)));
        cluster_arrive();
        cluster_wait();
        for (int i = 0; i < a.cluster; ++i) all = fmaxf(all, __uint_as_float((uint32_t)(sm.part[i] >> 32)));
        total = 0.f;
        first = INT32_MAX;
        for (int i = 0; i < a.cluster; ++i) {
            const float t = __uint_as_float((uint32_t)(sm.part[i] >> 32));
            if (greedy)
                first = t == all ? min(first, (int32_t)(uint32_t)sm.part[i]) : first;
            else
                total += __uint_as_float((uint32_t)sm.part[i]) * weight(t, all, k);
        }
        mine = weight(top, all, k);
    } else {
        cluster_wait();
    }
    // nothing allowed: no probability at all
    const float f = total > 0.f ? mine / total : 0.f;
    TP *p = static_cast<TP *>(a.p) + row * a.p_stride;
    const auto put = [&](int32_t g, float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = greedy ? (r.token(g, e) == first ? 1.f : 0.f) : x[e] * f;
        store_probs<TP, kVec>(p, r.token(g, 0), kVec ? 1 : kThreads, hi, x);
    };
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.load(g, z[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[0][e] = greedy ? 0.f : weight(z[0][e], top, k);
            put(g, z[0]);
        }
    } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) put(g, z[g]);
    }
}

// --------------------------------------------------------------- counting
struct CountArgs {
    uint16_t *counts;
    int64_t count_stride, token_stride;
    const int32_t *tokens, *n_prompt;
    int32_t n_seqs, n_tokens, vocab, slices, clear;
    int *err;
};

constexpr int kCountSlice = 8192, kCountThreads = 512;

// A CTA per sequence and slice of the vocabulary: it goes through the
// sequence's tokens, counts its own in shared memory (bit 31: in the prompt)
// and writes the slice. No order of the additions shows in the result.
__global__ void __launch_bounds__(kCountThreads) count_slices(const CountArgs a) {
    __shared__ uint32_t n[kCountSlice];
    pdl_wait();
    pdl_launch_dependents();
    const int32_t s = blockIdx.x / a.slices, lo = blockIdx.x % a.slices * kCountSlice, size = min(kCountSlice, a.vocab - lo);
    for (int i = threadIdx.x; i < size; i += kCountThreads) n[i] = 0;
    __syncthreads();
    const int32_t *tokens = a.tokens + s * a.token_stride;
    const int32_t prompt = a.n_prompt ? a.n_prompt[s] : 0;
    constexpr int kAhead = 8;
    for (int32_t i0 = threadIdx.x; i0 < a.n_tokens; i0 += kCountThreads * kAhead) {
        int32_t v[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int32_t i = i0 + e * kCountThreads;
            v[e] = i < a.n_tokens ? tokens[i] : -1;
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int32_t i = i0 + e * kCountThreads;
            if (v[e] >= a.vocab && lo == 0) set_error(a.err, HSWA_ERR_BOUNDS);
            if (v[e] < lo || v[e] - lo >= size) continue;
            if (i < prompt)
                atomicOr(&n[v[e] - lo], 1u << 31);
            else
                atomicAdd(&n[v[e] - lo], 1u);
        }
    }
    __syncthreads();
    uint16_t *out = a.counts + s * a.count_stride + lo;
    for (int i = threadIdx.x; i < size; i += kCountThreads) {
        uint32_t x = n[i];
        if (!a.clear) {
            if (x == 0) continue;
            const uint32_t was = out[i];
            x = ((x | was << 16) & 1u << 31) | min((x & 0x7fffffff) + (was & 0x7fff), 0x7fffu);
        }
        out[i] = (uint16_t)(min(x & 0x7fffffff, 0x7fffu) | x >> 31 << 15);
    }
}

// A few tokens added to counts that stay: a thread each.
__global__ void __launch_bounds__(256) count_few(const CountArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t at = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (at >= (int64_t)a.n_seqs * a.n_tokens) return;
    const int32_t s = (int32_t)(at / a.n_tokens), i = (int32_t)(at % a.n_tokens);
    const int32_t v = a.tokens[s * a.token_stride + i];
    if (v >= a.vocab) set_error(a.err, HSWA_ERR_BOUNDS);
    if (v < 0 || v >= a.vocab) return;
    const bool prompt = a.n_prompt && i < a.n_prompt[s];
    unsigned short *n = a.counts + s * a.count_stride + v, was = *n;
    for (;;) {
        const unsigned short next = prompt ? was | 0x8000 : (was & 0x7fff) == 0x7fff ? was : was + 1;
        if (next == was) return;
        const unsigned short seen = atomicCAS(n, was, next);
        if (seen == was) return;
        was = seen;
    }
}

constexpr int kFewTokens = 64;  // of a sequence

template <typename TL, typename TP, bool kVec, int kThreads, int kGroups, bool kLoop>
cudaError_t launch(const ProbsArgs &a, int64_t rows, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logits_probs<TL, TP, kVec, kThreads, kGroups, kLoop>, a);
}

template <typename TL, typename TP, bool kVec>
cudaError_t launch_row(const ProbsArgs &a, int64_t rows, cudaStream_t st) {
    const int32_t groups = (a.slice / 8 + 511) / 512;  // of 512 threads
    if (groups <= 2) return launch<TL, TP, kVec, 512, 2, false>(a, rows, st);
    if (groups <= 5) return launch<TL, TP, kVec, 512, 5, false>(a, rows, st);
    if (groups <= 10) return launch<TL, TP, kVec, 1024, 5, false>(a, rows, st);
    return launch<TL, TP, kVec, 1024, 1, true>(a, rows, st);
}

template <typename TL, typename TP>
cudaError_t launch_types(const ProbsArgs &a, bool vec, int64_t rows, cudaStream_t st) {
    return vec ? launch_row<TL, TP, true>(a, rows, st) : launch_row<TL, TP, false>(a, rows, st);
}

}  // namespace
}  // namespace hswa

using namespace hswa;

extern "C" int hswa_logits_probs(int logits_dtype, const void *logits, int64_t logits_stride, int p_dtype, void *p,
                                 int64_t p_stride, const float *params, const uint16_t *counts, int64_t count_stride,
                                 const int32_t *d_draft, const int32_t *bias_token, const float *bias, int n_bias,
                                 const uint32_t *mask, int64_t mask_stride, int n_seqs, int n_tok, int vocab,
                                 hswa_stream_t stream) {
    HSWA_NVTX("hswa_logits_probs");
    if (n_seqs < 0 || n_tok < 1 || n_tok > HSWA_DECODE_MAX_TOKENS || vocab < 1 || n_bias < 0) return HSWA_ERR_INVALID_ARG;
    for (const int dt : {logits_dtype, p_dtype})
        if (dt != HSWA_DTYPE_F32 && dt != HSWA_DTYPE_BF16) return HSWA_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)n_seqs * n_tok;
    if (vocab > HSWA_VERIFY_MAX_VOCAB || n_bias > HSWA_LOGITS_MAX_BIAS || rows > INT32_MAX / kMaxCluster) return HSWA_ERR_UNSUPPORTED;
    if (n_seqs == 0) return HSWA_OK;
    const int64_t el = logits_dtype == HSWA_DTYPE_F32 ? 4 : 2, ep = p_dtype == HSWA_DTYPE_F32 ? 4 : 2;
    const int64_t words = (vocab + 31) / 32;
    if (!logits || !p || logits_stride < vocab || p_stride < vocab || (counts && count_stride < vocab) ||
        (n_bias > 0 && (!bias_token || !bias)) || (mask && mask_stride < words))
        return HSWA_ERR_INVALID_ARG;
    if (((uintptr_t)logits & (el - 1)) || ((uintptr_t)p & (ep - 1)) || ((uintptr_t)counts & 1) ||
        (((uintptr_t)params | (uintptr_t)d_draft | (uintptr_t)bias_token | (uintptr_t)bias | (uintptr_t)mask) & 3))
        return HSWA_ERR_INVALID_ARG;
    // p apart from the logits, or the logits themselves, each value in its place
    const uintptr_t x0 = (uintptr_t)logits, x1 = x0 + (uintptr_t)(((rows - 1) * logits_stride + vocab) * el);
    const uintptr_t y0 = (uintptr_t)p, y1 = y0 + (uintptr_t)(((rows - 1) * p_stride + vocab) * ep);
    if (x0 < y1 && y0 < x1 && !(x0 == y0 && el == ep && (logits_stride == p_stride || rows == 1))) return HSWA_ERR_INVALID_ARG;
    ProbsArgs a;
    a.logits = logits, a.p = p;
    a.logits_stride = logits_stride, a.p_stride = p_stride, a.count_stride = count_stride, a.mask_stride = mask_stride;
    a.params = params;
    a.counts = counts;
    a.draft = n_tok > 1 ? d_draft : nullptr;
    a.bias_token = bias_token, a.bias = bias;
    a.mask = mask;
    a.n_bias = n_bias, a.n_tok = n_tok, a.vocab = vocab;
    a.err = error_word();
    // CTAs per row: few rows spread over the GPU, in slices of at least 1024
    // values; many rows take as many as keep a thread's values in registers.
    const int sms = sm_count();
    if (sms <= 0) return HSWA_ERR_CUDA;
    const auto slice_of = [&](int c) { return ((vocab + 8 * c - 1) / (8 * c)) * 8; };
    a.cluster = 1;
    while (a.cluster < kMaxCluster &&
           (slice_of(a.cluster) > 512 * 8 * 5 || (rows * a.cluster * 2 <= 2 * sms && slice_of(a.cluster) >= 2048)))
        a.cluster *= 2;
    a.slice = slice_of(a.cluster);
    const bool vec = (x0 & 15) == 0 && (y0 & 15) == 0 && logits_stride * el % 16 == 0 && p_stride * ep % 16 == 0 &&
                     (!counts || (((uintptr_t)counts & 15) == 0 && count_stride % 8 == 0));
    set_last_kernel(vec ? "logits_probs" : "logits_probs_any");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (el == 4)
        e = ep == 4 ? launch_types<float, float>(a, vec, rows, st) : launch_types<float, __nv_bfloat16>(a, vec, rows, st);
    else
        e = ep == 4 ? launch_types<__nv_bfloat16, float>(a, vec, rows, st)
                    : launch_types<__nv_bfloat16, __nv_bfloat16>(a, vec, rows, st);
    return e == cudaSuccess ? HSWA_OK : cuda_fail(e, "hswa_logits_probs");
}

extern "C" int hswa_count_tokens(uint16_t *counts, int64_t count_stride, const int32_t *tokens, int64_t token_stride,
                                 const int32_t *d_n_prompt, int n_seqs, int n_tokens, int vocab, int clear,
                                 hswa_stream_t stream) {
    HSWA_NVTX("hswa_count_tokens");
    if (n_seqs < 0 || n_tokens < 0 || vocab < 1) return HSWA_ERR_INVALID_ARG;
    const int32_t slices = (vocab + kCountSlice - 1) / kCountSlice;
    if (vocab > HSWA_VERIFY_MAX_VOCAB || (int64_t)n_seqs * slices > INT32_MAX ||
        (int64_t)n_seqs * n_tokens > (int64_t)INT32_MAX * 128)
        return HSWA_ERR_UNSUPPORTED;
    if (n_seqs == 0 || (n_tokens == 0 && !clear)) return HSWA_OK;
    if (!counts || count_stride < vocab || (n_tokens > 0 && (!tokens || token_stride < n_tokens)) ||
        ((uintptr_t)counts & 1) || (((uintptr_t)tokens | (uintptr_t)d_n_prompt) & 3))
        return HSWA_ERR_INVALID_ARG;
    CountArgs a;
    a.counts = counts;
    a.count_stride = count_stride, a.token_stride = token_stride;
    a.tokens = tokens, a.n_prompt = d_n_prompt;
    a.n_seqs = n_seqs, a.n_tokens = n_tokens, a.vocab = vocab, a.slices = slices, a.clear = clear != 0;
    a.err = error_word();
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!clear && n_tokens <= kFewTokens) {
        set_last_kernel("count_few");
        e = launch_pdl(count_few, dim3((unsigned)(((int64_t)n_seqs * n_tokens + 255) / 256)), dim3(256), 0, st, a);
    } else {
        set_last_kernel("count_slices");
        e = launch_pdl(count_slices, dim3((unsigned)(n_seqs * slices)), dim3(kCountThreads), 0, st, a);
    }
    return e == cudaSuccess ? HSWA_OK : cuda_fail(e, "hswa_count_tokens");
}
