// Verification of drafted tokens against the target's probabilities.
//
// Rejection sampling of a draft chain (Leviathan, Kalman, Matias, "Fast
// Inference from Transformers via Speculative Decoding"): draft w of a
// sequence stays while u_w q_w(x_w) < p_w(x_w); at the first refusal a the
// next token is drawn from max(p_a - q_a, 0), after n drafts that all stay
// from p_n, by inverse CDF with one more given number.
//
// Everything that decides is exact. The acceptance test compares a product
// of two fp32 values with a third in 64-bit floating point, where the
// product is exact. For the draw, probabilities are turned into integers
// (2^50 steps to 1) and their differences summed in 64 and 96 bits, so the
// sums, and with them the token, do not depend on how the row is split.
#include "common.cuh"
#include "internal.h"

namespace hswa {
namespace {

constexpr int kWarps = 16;
constexpr int kCluster = 8;                  // CTAs per sequence
constexpr int kParts = kCluster * kWarps;    // a row is cut into that many slices, one per warp

typedef unsigned __int128 u128;

struct VerifyArgs {
    const void *p, *q;
    int64_t p_stride, q_stride;
    const int32_t *draft, *n_draft;
    const float *u;
    int32_t n_tok, vocab;
    int32_t *n_accept, *tokens;
    int *err;
};

template <typename T>
__device__ __forceinline__ float prob(const T *row, int64_t i);
template <>
__device__ __forceinline__ float prob<float>(const float *row, int64_t i) { return row[i]; }
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(const __nv_bfloat16 *row, int64_t i) {
    return __bfloat162float(row[i]);
}

// A probability in steps of 2^-50: [0, 1] clamped, NaN as 0.
__device__ __forceinline__ uint64_t steps(float x) {
    return __float2ull_rn(fminf(fmaxf(x, 0.f), 1.f) * 0x1p50f);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int m) {
    return __shfl_xor_sync(0xffffffffu, (unsigned long long)x, m);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Store to the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(const uint64_t *mine, int rank, uint64_t x) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}

// floor(u x) for u in [0, 1)
__device__ u128 times_fraction(u128 x, float u) {
    const uint32_t b = __float_as_uint(u);
    const int e = (int)(b >> 23);
    const uint32_t m = e ? (b & 0x7fffff) | 0x800000 : b & 0x7fffff;
    const int shift = 150 - (e ? e : 1);  // u = m 2^-shift, shift in [24, 149]
    return shift < 128 ? (x * m) >> shift : 0;
}

// What the draw at row position i weighs: the target's probability less the
// draft's (less everything at the drafted token when the draft is greedy).
template <typename T>
__device__ __forceinline__ uint64_t weight(const T *p, const T *q, int64_t i, int64_t gone) {
    const uint64_t x = steps(prob(p, i));
    if (q) {
        const uint64_t y = steps(prob(q, i));
        return x > y ? x - y : 0;
    }
    return i == gone ? 0 : x;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) verify_draft(const __grid_constant__ VerifyArgs a) {
    __shared__ uint64_t sums[2][kParts];  // slice sums of both passes, in every CTA of the cluster
    __shared__ int32_t s_accept;
    __shared__ int32_t s_token;
    __shared__ uint64_t s_warp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % kCluster;
    const int64_t s = blockIdx.x / kCluster;
    const int n_rows = a.n_tok - 1;  // drafts a sequence can have
    cluster_arrive();  // awaited before the first store into another CTA's shared memory
    if (warp == 0) {
        int32_t n = a.n_draft ? a.n_draft[s] : n_rows;
        bool bad = n < 0 || n > n_rows;
        n = max(0, min(n, n_rows));
        bool stays = false;
        if (lane < n) {
            const int32_t x = a.draft[s * n_rows + lane];
            if (x < 0 || x >= a.vocab) {
                bad = true;
            } else {
                const double px = prob((const T *)a.p + (s * a.n_tok + lane) * a.p_stride, x);
                const double qx = a.q ? (double)prob((const T *)a.q + (s * n_rows + lane) * a.q_stride, x) : 1.0;
                stays = (double)a.u[s * a.n_tok + lane] * qx < px;
            }
        }
        if (bad && rank == 0) set_error(a.err, HSWA_ERR_BOUNDS);
        const unsigned gone = __ballot_sync(0xffffffffu, !stays);  // lanes past the drafts are in it
        if (lane == 0) {
            s_accept = __ffs(gone) - 1;
            s_token = n;
        }
    }
    __syncthreads();
    const int32_t acc = s_accept;
    const bool refused = acc < s_token;
    __syncthreads();
    const T *p = (const T *)a.p + (s * a.n_tok + acc) * a.p_stride;
    const T *q = refused && a.q ? (const T *)a.q + (s * n_rows + acc) * a.q_stride : nullptr;
    int64_t gone = refused && !a.q ? a.draft[s * n_rows + acc] : -1;
    const int32_t part = (a.vocab + kParts - 1) / kParts;

    u128 total = 0;
    int pass = 0;
    for (; pass < 2; ++pass) {
        const int64_t lo = (int64_t)(rank * kWarps + warp) * part;
        const int64_t hi = lo + part < a.vocab ? lo + part : a.vocab;
        uint64_t sum = 0;
        for (int64_t i = lo + lane; i < hi; i += 32) sum += weight(p, q, i, gone);
        for (int m = 16; m > 0; m >>= 1) sum += shfl_xor64(sum, m);
        if (pass == 0) cluster_wait();  // every CTA of the cluster has started
        if (lane < kCluster) st_cluster_u64(&sums[pass][rank * kWarps + warp], lane, sum);
        cluster_arrive();
        cluster_wait();
        total = 0;
        for (int i = 0; i < kParts; ++i) total += sums[pass][i];
        if (total != 0 || (!q && gone < 0)) break;
        q = nullptr;  // nothing is left of the target where the draft was: draw from the target itself
        gone = -1;
    }
    if (rank != 0) return;  // every store into this CTA's shared memory came before the barrier
    pass = min(pass, 1);
    // the first position whose cumulative weight passes u times the total
    if (threadIdx.x == 0) s_token = -1;
    __syncthreads();
    if (total != 0) {
        const float u = fminf(fmaxf(a.u[s * a.n_tok + a.n_tok - 1], 0.f), 0x1.fffffep-1f);
        u128 left = times_fraction(total, u);
        int slice = 0;
        for (; slice < kParts - 1; ++slice) {
            const uint64_t x = sums[pass][slice];
            if (left < x) break;
            left -= x;
        }
        uint64_t t = (uint64_t)left;
        const int64_t lo = (int64_t)slice * part;
        const int64_t hi = lo + part < a.vocab ? lo + part : a.vocab;
        for (int64_t base = lo; base < hi; base += blockDim.x) {
            const int64_t i = base + threadIdx.x;
            const uint64_t x = i < hi ? weight(p, q, i, gone) : 0;
            uint64_t upto = x;  // inclusive sums over the warp, then over the warps before it
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, (unsigned long long)upto, off);
                if (lane >= off) upto += y;
            }
            if (lane == 31) s_warp[warp] = upto;
            __syncthreads();
            uint64_t before = 0, all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s_warp[w];
                all += s_warp[w];
            }
            upto += before;
            if (upto > t && upto - x <= t) s_token = (int32_t)i;  // one thread at most
            __syncthreads();
            if (all > t) break;
            t -= all;
        }
    }
    if (threadIdx.x == 0) a.n_accept[s] = acc;
    if (threadIdx.x < a.n_tok)
        a.tokens[s * a.n_tok + threadIdx.x] =
            threadIdx.x < acc ? a.draft[s * n_rows + threadIdx.x] : threadIdx.x == acc ? s_token : -1;
}

}  // namespace
}  // namespace hswa

using namespace hswa;

extern "C" int hswa_verify_draft(int dtype, const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                                 const int32_t *d_draft, const int32_t *d_n_draft, const float *u, int n_seqs,
                                 int n_tok, int vocab, int32_t *n_accept, int32_t *tokens, hswa_stream_t stream) {
    HSWA_NVTX("hswa_verify_draft");
    if (n_seqs < 0 || n_tok < 1 || n_tok > HSWA_DECODE_MAX_TOKENS || vocab < 1) return HSWA_ERR_INVALID_ARG;
    if (dtype != HSWA_DTYPE_F32 && dtype != HSWA_DTYPE_BF16) return HSWA_ERR_UNSUPPORTED;
    if (vocab > HSWA_VERIFY_MAX_VOCAB || n_seqs > INT32_MAX / kCluster) return HSWA_ERR_UNSUPPORTED;
    if (n_seqs == 0) return HSWA_OK;
    const int64_t e = dtype == HSWA_DTYPE_F32 ? 4 : 2;
    if (!p || !u || !n_accept || !tokens || (n_tok > 1 && !d_draft) || p_stride < vocab ||
        (q && n_tok > 1 && q_stride < vocab) || ((uintptr_t)p & (e - 1)) || ((uintptr_t)q & (e - 1)))
        return HSWA_ERR_INVALID_ARG;
    VerifyArgs a;
    a.p = p, a.q = n_tok > 1 ? q : nullptr;
    a.p_stride = p_stride, a.q_stride = q_stride;
    a.draft = d_draft, a.n_draft = n_tok > 1 ? d_n_draft : nullptr;
    a.u = u;
    a.n_tok = n_tok, a.vocab = vocab;
    a.n_accept = n_accept, a.tokens = tokens;
    a.err = error_word();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_seqs * kCluster);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    set_last_kernel(e == 4 ? "verify_draft_f32" : "verify_draft_bf16");
    const cudaError_t rc = e == 4 ? cudaLaunchKernelEx(&cfg, verify_draft<float>, a)
                                  : cudaLaunchKernelEx(&cfg, verify_draft<__nv_bfloat16>, a);
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_verify_draft");
}
