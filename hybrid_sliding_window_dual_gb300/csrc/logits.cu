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
    bool wide;                // fp32 rows start on 32 bytes
    int32_t n_bias, n_tok, vocab, cluster, slice;  // slice: elements per CTA, a multiple of 8
    int32_t rows, ahead;  // ahead: rows that run at once, 0 if all do
    int *err;
};

// 8 neighbouring fp32 values: in one access where they start on 32 bytes (two of
// 16 bytes from each lane touch every sector of the warp's kilobyte twice).
__device__ __forceinline__ void load8(const float *p, bool wide, float (&x)[8]) {
    if (wide) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                     : "l"(p)
                     : "memory");
    } else {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
__device__ __forceinline__ void store8(float *p, bool wide, const float (&x)[8]) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
                     "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// Loads where `on` says so, x as it was otherwise. Without branches, so that a
// thread has those of all its groups in flight.
__device__ __forceinline__ void load8_if(bool on, const float *p, bool wide, float (&x)[8]) {
    asm volatile("{\n\t.reg .pred w, n;\n\t.reg .b32 f;\n\t"
                 "and.b32 f, %9, %10;\n\tsetp.ne.u32 w, f, 0;\n\t"
                 "not.b32 f, %10;\n\tand.b32 f, f, %9;\n\tand.b32 f, f, 1;\n\tsetp.ne.u32 n, f, 0;\n\t"
                 "@w ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "@n ld.global.v4.f32 {%0, %1, %2, %3}, [%8];\n\t"
                 "@n ld.global.v4.f32 {%4, %5, %6, %7}, [%8 + 16];\n\t}"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7])
                 : "l"(p), "r"((uint32_t)on), "r"((uint32_t)wide));
}
__device__ __forceinline__ void load_if(bool on, const float *p, float &x) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.f32 %0, [%1];\n\t}" : "+f"(x) : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void load_if(bool on, const void *p, uint16_t &x) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}" : "+h"(x) : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void load16b_if(bool on, const void *p, uint32_t (&x)[4]) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3])
                 : "l"(p), "r"((uint32_t)on));
}

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Bytes (less a last partial 16) from a 16-byte boundary on into L2.
__device__ __forceinline__ void prefetch_l2(const void *p, int32_t bytes) {
    if (bytes >= 16) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes & ~15));
}

struct ProbsSmem {
    int32_t key[kBiasSlots];  // token of a slot, -1: free
    int32_t at[kBiasSlots];   // the last entry of the bias list with that token
    uint32_t special[kMaxSlice / 32];  // the CTA's tokens with a bias or a draft
    int32_t draft[HSWA_DECODE_MAX_TOKENS];
    uint64_t row;                     // those of all
    uint64_t part[kMaxCluster * 32];  // every warp's of the cluster: maximum, sum or first index
};

__device__ __forceinline__ uint32_t bias_slot(int32_t token) { return (uint32_t)token * 0x9E3779B1u >> 21; }
static_assert(kBiasSlots == 1 << 11, "the hash keeps 11 bits");

// The row of a CTA, and what happens to its logits.
template <typename TL, bool kVec, int kThreads>
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
    float rep, freq, pres;

    // Element e of group k, counted from a thread's first (kVec: 8 neighbours, else
    // 8 as far apart as the CTA has threads).
    static __device__ __forceinline__ constexpr int32_t offset(int32_t k, int e) {
        return kVec ? 8 * k * kThreads + e : (8 * k + e) * kThreads;
    }
    // Its token in thread t.
    __device__ __forceinline__ int32_t token(int32_t k, int32_t t, int e) const {
        return lo + (kVec ? 8 * t : t) + offset(k, e);
    }

    __device__ __forceinline__ float penalized(float z, uint32_t c, int extra) const {
        const int32_t n = (int32_t)(c & 0x7fff) + extra;
        if (n > 0 || c >> 15) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
        if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)n)), pres);
        return z;
    }

    // z of any token but for the mask, from its logit and its count.
    __device__ __forceinline__ float value(int32_t v, float z, uint32_t c) const {
        int extra = 0;
        if (counts) {
            for (int j = 0; j < w; ++j) extra += sm.draft[j] == v;
            z = penalized(z, c, extra);
        }
        if (a.n_bias) {
            uint32_t s = bias_slot(v);
            while (sm.key[s] != -1 && sm.key[s] != v) s = (s + 1) & (kBiasSlots - 1);
            if (sm.key[s] == v) z = __fadd_rn(z, bias[sm.at[s]]);
        }
        return z;
    }
    // 8 neighbouring logits.
    __device__ __forceinline__ void read8(int32_t v0, float (&z)[8]) const {
        if constexpr (sizeof(TL) == 4) {
            load8(reinterpret_cast<const float *>(logits + v0), a.wide, z);
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(logits + v0);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) z[2 * e] = __uint_as_float(u[e] << 16), z[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
    }

    // Group k of this thread: its 8 logits as z, and whether a token of it may
    // need more (one that occurred, a draft, one with a bias).
    __device__ __forceinline__ bool load(int32_t k, float (&z)[8]) const {
        const int32_t v0 = token(k, threadIdx.x, 0);
        uint32_t any = 0;
        if (kVec && v0 >= hi) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = -INFINITY;
        } else if (kVec && v0 + 8 <= hi) {
            uint4 n = make_uint4(0, 0, 0, 0);
            if (counts) n = *reinterpret_cast<const uint4 *>(counts + v0);
            read8(v0, z);
            any = n.x | n.y | n.z | n.w;
            if (specials) any |= sm.special[(v0 - lo) >> 5] >> ((v0 - lo) & 31) & 0xff;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, threadIdx.x, e);
                z[e] = -INFINITY;
                if (v < hi) {
                    z[e] = as_float(logits[v]);
                    if (counts) any |= counts[v];
                    if (specials) any |= sm.special[(v - lo) >> 5] >> ((v - lo) & 31) & 1;
                }
            }
        }
        return any != 0;
    }

    // load() for all groups of the thread whose bits (8 a group) are not all 0, the
    // others' z being -inf: bit k of the result is group k's.
    template <int kGroups>
    __device__ __forceinline__ uint32_t load_all(uint64_t bits, float (&z)[kGroups][8]) const {
        uint32_t own = 0;
        const int32_t first = token(0, threadIdx.x, 0), left = hi - first;
        const TL *const from = logits + first;
        const uint16_t *const counted = counts + first;  // not read without counts
        if constexpr (kVec) {
            uint32_t on = 0;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                on |= (offset(g, 8) <= left && (bits >> (8 * g) & 0xff) ? 1u : 0u) << g;
            const auto occurred = [&] {
                if (!counts) return;
                uint32_t n[kGroups][4];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    n[g][0] = n[g][1] = n[g][2] = n[g][3] = 0;
                    load16b_if(on >> g & 1, counted + offset(g, 0), n[g]);
                }
#pragma unroll
                for (int g = 0; g < kGroups; ++g) own |= (n[g][0] | n[g][1] | n[g][2] | n[g][3] ? 1u : 0u) << g;
            };
            if constexpr (sizeof(TL) == 4) {
                occurred();  // first: registers for both are not there
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[g][e] = -INFINITY;
                    load8_if(on >> g & 1, reinterpret_cast<const float *>(from + offset(g, 0)), a.wide, z[g]);
                }
            } else {
                uint32_t x[kGroups][4];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    x[g][0] = x[g][1] = x[g][2] = x[g][3] = 0xff80ff80;  // -inf
                    load16b_if(on >> g & 1, from + offset(g, 0), x[g]);
                }
                occurred();
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[g][2 * e] = __uint_as_float(x[g][e] << 16), z[g][2 * e + 1] = __uint_as_float(x[g][e] & 0xffff0000u);
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int32_t at = first - lo + offset(g, 0);
                if (specials && (on >> g & 1)) own |= (sm.special[at >> 5] >> (at & 31) & 0xff ? 1u : 0u) << g;
                if (offset(g, 0) < left && offset(g, 8) > left && (bits >> (8 * g) & 0xff)) own |= (load(g, z[g]) ? 1u : 0u) << g;  // the row's last
            }
        } else {
            const auto on = [&](int g, int e) { return offset(g, e) < left && (bits >> (8 * g + e) & 1); };
            if (counts) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    uint16_t n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] = 0, load_if(on(g, e), counted + offset(g, e), n[e]);
                    own |= (n[0] | n[1] | n[2] | n[3] | n[4] | n[5] | n[6] | n[7] ? 1u : 0u) << g;
                }
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    z[g][e] = -INFINITY;
                    if constexpr (sizeof(TL) == 4) {
                        load_if(on(g, e), reinterpret_cast<const float *>(from + offset(g, e)), z[g][e]);
                    } else {
                        uint16_t x = 0xff80;
                        load_if(on(g, e), from + offset(g, e), x);
                        z[g][e] = __uint_as_float((uint32_t)x << 16);
                    }
                }
            if (specials) {
                // a warp's tokens of one (group, element) are a word of the bits; mostly none is set
                constexpr int kWords = kThreads / 32;
                const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
                uint32_t some = 0;
                for (int i = lane; i < 8 * kGroups; i += 32)
                    if (lo + i * kThreads < hi) some |= sm.special[i * kWords + warp];
                if (__any_sync(0xffffffffu, some != 0)) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (on(g, e)) own |= (sm.special[(8 * g + e) * kWords + warp] >> lane & 1) << g;
                }
            }
        }
        return own;
    }

    // z of group k of thread t into z8 (shared memory), each token with what it needs.
    __device__ __forceinline__ void fetch(int32_t k, int32_t t, float *z8) const {
        const int32_t v0 = token(k, t, 0);
        uint32_t own = 0;
        if (kVec && v0 + 8 <= hi) {
            float z[8];
            read8(v0, z);
            if (counts) {
                const uint4 n = *reinterpret_cast<const uint4 *>(counts + v0);
                const uint32_t u[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) own |= (u[e] & 0xffff ? 1u : 0u) << (2 * e) | (u[e] >> 16 ? 2u : 0u) << (2 * e);
            }
            if (specials) own |= sm.special[(v0 - lo) >> 5] >> ((v0 - lo) & 31) & 0xff;
#pragma unroll
            for (int e = 0; e < 8; ++e) z8[e] = z[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, t, e);
                float z = -INFINITY;
                if (v < hi) {
                    z = as_float(logits[v]);
                    if ((counts && counts[v]) || (specials && (sm.special[(v - lo) >> 5] >> ((v - lo) & 31) & 1))) own |= 1u << e;
                }
                z8[e] = z;
            }
        }
        while (own) {
            const int e = __ffs((int)own) - 1;
            own &= own - 1;
            const int32_t v = token(k, t, e);
            z8[e] = value(v, z8[e], counts ? counts[v] : 0);
        }
    }

    // Group k's 8 bits of the mask.
    __device__ __forceinline__ uint32_t allowed(int32_t k) const {
        uint32_t bits = 0;
        if constexpr (kVec) {
            const int32_t v0 = token(k, threadIdx.x, 0);
            if (v0 < hi) bits = reinterpret_cast<const uint8_t *>(mask)[v0 >> 3];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, threadIdx.x, e);
                if (v < hi) bits |= (mask[v >> 5] >> (v & 31) & 1) << e;
            }
        }
        return bits;
    }

    // All of it, where nothing is kept between.
    __device__ __forceinline__ void whole(int32_t k, float (&z)[8]) const {
        if (load(k, z)) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const int32_t v = token(k, threadIdx.x, e);
                const float x = v < hi ? value(v, as_float(logits[v]), counts ? counts[v] : 0) : -INFINITY;
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    if (y == e) z[y] = x;
            }
        }
        const uint32_t bits = mask ? allowed(k) : 0xff;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = bits >> e & 1 ? fmaxf(z[e], -INFINITY) : -INFINITY;  // NaN too
    }
};

// A group of results from p on, `left` of the row's values from there; step
// apart where they are not neighbours.
template <typename TP, bool kVec>
__device__ __forceinline__ void store_probs(TP *p, int32_t step, int32_t left, bool wide, const float (&x)[8]) {
    if (kVec && left <= 0) return;
    if (kVec && left >= 8) {
        if constexpr (sizeof(TP) == 4) {
            store8(reinterpret_cast<float *>(p), wide, x);
        } else {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e * step < left) {
                if constexpr (sizeof(TP) == 4)
                    p[e * step] = x[e];
                else
                    p[e * step] = __float2bfloat16_rn(x[e]);
            }
        }
    }
}

__device__ __forceinline__ float warp_max(float x) {  // passes NaN over
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_sum(float x) {
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// exp((z - top) / T): k is log2 e / T, finite and above 0. A top of +inf
// shares the probability among the infinite values; -inf is that of no value at all.
__device__ __forceinline__ float weight(float z, float top, float k) {
    if (top == INFINITY) return z == INFINITY ? 1.f : 0.f;
    return fast_exp2((z - (top == -INFINITY ? 0.f : top)) * k);
}

// A cluster per row, kGroups groups of 8 values per thread in registers between
// the one read and the one write; rows longer than that (kLoop) are read three
// times, for the maximum, the sum and the result. Warps work on their own (their
// maximum, the sum relative to it) and meet once, at the cluster's barrier, with
// every warp's pair in every CTA.
//
// What few tokens need (penalties, drafts, biases) is not done where they lie,
// where a warp would do it for all its values: groups with such a token go on the
// warp's list, its lanes take one each, and the owners fetch the results.
//
// 256 rows of 150000, bf16 to fp32: 79 us with penalties, 57 without, 35 at a
// plain copy's rate. An SM holds two CTAs (a thread's 40 values are registers), and
// loads, list, exponentials, the cluster's barrier and stores follow each other
// in both: issue slots and memory are each busy for less than half of the
// time (34 instructions a value, 20 without penalties). What it took: loads of all
// groups in flight at once (without counts 74 us before, 63 after), fp32 rows 32
// bytes a lane, redux for the maximum, lists by groups (tokens by themselves 101,
// groups 96), constant offsets between groups (93 to 81), the next rows on their
// way to L2 (81 to 79). Rows streamed twice through shared memory instead of kept
// took 115, three reads (kLoop) 585, clusters of 16 CTAs of 256 threads 85.
template <typename TL, typename TP, bool kVec, int kThreads, int kGroups, bool kLoop>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logits_probs(const __grid_constant__ ProbsArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ ProbsSmem sm;
    constexpr int kList = 32;  // groups at once, one a lane
    __shared__ uint8_t list[kLoop ? 1 : kWarps][kList];  // group k of lane t: 32 k + t
    __shared__ __align__(16) float fetched[kLoop ? 1 : kWarps][kList][8];
    static_assert(kGroups <= 8, "an entry of the list is a byte");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t row = blockIdx.x / (uint32_t)a.cluster, rank = blockIdx.x - row * a.cluster;
    const uint32_t seq = row / (uint32_t)a.n_tok;
    const int32_t w = (int32_t)(row - seq * a.n_tok);
    float temperature = 1.f, rep = 1.f, freq = 0.f, pres = 0.f;
    if (a.params) {
        const float *x = a.params + (size_t)seq * 4;
        temperature = x[0], rep = x[1] > 0.f ? x[1] : 1.f, freq = x[2], pres = x[3];
    }
    const bool penalties = a.counts && !(rep == 1.f && freq == 0.f && pres == 0.f);
    const int32_t lo = min((int32_t)rank * a.slice, a.vocab), hi = min(lo + a.slice, a.vocab);
    const bool drafts = penalties && a.draft && w > 0;
    const ProbsRow<TL, kVec, kThreads> r{a, sm, static_cast<const TL *>(a.logits) + row * a.logits_stride,
                               penalties ? a.counts + seq * a.count_stride : nullptr,
                               a.mask ? a.mask + row * a.mask_stride : nullptr,
                               a.bias + (size_t)seq * a.n_bias, lo, hi, drafts ? w : 0, a.n_bias > 0 || drafts,
                               rep, freq, pres};
    if (r.specials) {
        if (a.n_bias)
            for (int i = tid; i < kBiasSlots; i += kThreads) sm.key[i] = sm.at[i] = -1;
        for (int i = tid; i < (a.slice + 31) / 32; i += kThreads) sm.special[i] = 0;
        __syncthreads();
        for (int i = tid; i < a.n_bias; i += kThreads) {
            const int32_t v = a.bias_token[(int64_t)seq * a.n_bias + i];
            if (v >= a.vocab) set_error(a.err, HSWA_ERR_BOUNDS);
            if (v < lo || v >= hi) continue;
            atomicOr(&sm.special[(v - lo) >> 5], 1u << ((v - lo) & 31));
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
            if (v >= lo && v < hi) atomicOr(&sm.special[(v - lo) >> 5], 1u << ((v - lo) & 31));
        }
        __syncthreads();
    }
    const int32_t groups = kLoop ? (a.slice / 8 + kThreads - 1) / kThreads : kGroups;
    const bool greedy = !(temperature > 0.f);
    const float k = greedy ? 1.f : fminf(fmaxf(1.4426950408889634f / temperature, 0x1p-149f), FLT_MAX);

    float z[kGroups][8];
    float top = -INFINITY;
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.whole(g, z[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, z[0][e]);
        }
    } else {
        uint64_t bits = ~0ull;
        if (r.mask) {
            bits = 0;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) bits |= (uint64_t)r.allowed(g) << (8 * g);
        }
        const uint32_t own = r.load_all(bits, z);  // bit g: group g goes on the list
        if constexpr (kVec) {
            // what a CTA in this one's place will read, under a mask whole slices all the
            // same: on its way to L2 while this one computes
            if (tid == 0 && a.ahead > 0 && (int64_t)row + a.ahead < a.rows) {
                const int64_t next = (int64_t)row + a.ahead;
                prefetch_l2(r.logits + a.ahead * a.logits_stride + lo, (hi - lo) * (int32_t)sizeof(TL));
                if (r.counts) prefetch_l2(a.counts + next / a.n_tok * a.count_stride + lo, (hi - lo) * 2);
            }
        }
        if (__any_sync(0xffffffffu, own != 0)) {
            int place[kGroups], n_list = 0;  // of this lane's groups on the list
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const uint32_t takers = __ballot_sync(0xffffffffu, own >> g & 1);
                place[g] = n_list + __popc(takers & ((1u << lane) - 1));
                n_list += __popc(takers);
            }
            for (int from = 0; from < n_list; from += kList) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int at = place[g] - from;
                    if ((own >> g & 1) && (uint32_t)at < kList) list[warp][at] = (uint8_t)(32 * g + lane);
                }
                __syncwarp();
                if (from + lane < n_list) {
                    const int id = list[warp][lane];
                    r.fetch(id >> 5, 32 * warp + (id & 31), fetched[warp][lane]);
                }
                __syncwarp();
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int at = place[g] - from;
                    if ((own >> g & 1) && (uint32_t)at < kList) {
                        const float4 x0 = *reinterpret_cast<const float4 *>(&fetched[warp][at][0]), x1 = *reinterpret_cast<const float4 *>(&fetched[warp][at][4]);
                        z[g][0] = x0.x, z[g][1] = x0.y, z[g][2] = x0.z, z[g][3] = x0.w, z[g][4] = x1.x, z[g][5] = x1.y, z[g][6] = x1.z, z[g][7] = x1.w;
                    }
                }
                __syncwarp();
            }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            if (r.mask) {
                const uint32_t b = (uint32_t)(bits >> (8 * g));
#pragma unroll
                for (int e = 0; e < 8; ++e) z[g][e] = b >> e & 1 ? z[g][e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) top = fmaxf(fmaxf(top, z[g][e]), z[g][e + 1]);  // passes NaN over
        }
    }
    top = warp_max(top);
    // the warp's sum relative to it, or the first token that has it
    float sum = 0.f;
    int32_t first = INT32_MAX;
    const bool plain = top < INFINITY;
    const float ref = top == -INFINITY ? 0.f : -top;
    const auto take = [&](int32_t g, float (&x)[8]) {
        if (greedy) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (x[e] == top && x[e] > -INFINITY) first = min(first, r.token(g, tid, e));
        } else if (plain) {
            float2 part = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[e], x[e + 1]), make_float2(ref, ref)), make_float2(k, k));
                x[e] = fmaxf(fast_exp2(y.x), 0.f), x[e + 1] = fmaxf(fast_exp2(y.y), 0.f);  // NaN becomes 0
                part = __fadd2_rn(part, make_float2(x[e], x[e + 1]));
            }
            sum += part.x + part.y;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = weight(x[e], top, k);
                sum += x[e];
            }
        }
    };
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.whole(g, z[0]);
            take(g, z[0]);
        }
    } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) take(g, z[g]);
    }
    if (greedy)
        first = __reduce_min_sync(0xffffffffu, first);
    else
        sum = warp_sum(sum);
    cluster_wait();  // every CTA of the cluster has started
    const uint64_t pair = (uint64_t)__float_as_uint(top) << 32 | (greedy ? (uint32_t)first : __float_as_uint(sum));
    if (lane < a.cluster) st_cluster_u64(&sm.part[rank * kWarps + warp], lane, pair);
    cluster_arrive();
    cluster_wait();
    // all warps' pairs, kPer of them a lane of one warp
    if (warp == 0) {
        constexpr int kPer = kMaxCluster * kWarps / 32;
        const int n_parts = a.cluster * kWarps;
        uint64_t parts[kPer];
        float all = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            parts[i] = lane + 32 * i < n_parts ? sm.part[lane + 32 * i] : (uint64_t)0xff800000u << 32;
            all = fmaxf(all, __uint_as_float((uint32_t)(parts[i] >> 32)));
        }
        all = warp_max(all);
        uint32_t x = (uint32_t)INT32_MAX;
        if (greedy) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (__uint_as_float((uint32_t)(parts[i] >> 32)) == all) x = min(x, (uint32_t)parts[i]);
            x = __reduce_min_sync(0xffffffffu, x);
            if (all == -INFINITY) x = (uint32_t)INT32_MAX;
        } else {
            float total = 0.f;
            if (all > -INFINITY) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) total += __uint_as_float((uint32_t)parts[i]) * weight(__uint_as_float((uint32_t)(parts[i] >> 32)), all, k);
                total = warp_sum(total);
            }
            x = __float_as_uint(total);
        }
        if (lane == 0) sm.row = (uint64_t)__float_as_uint(all) << 32 | x;
    }
    __syncthreads();
    const float all = __uint_as_float((uint32_t)(sm.row >> 32)), total = greedy ? 0.f : __uint_as_float((uint32_t)sm.row);
    first = (int32_t)(uint32_t)sm.row;
    // nothing allowed: no probability at all
    const float f = total > 0.f && top > -INFINITY ? weight(top, all, k) / total : 0.f;
    const int32_t at = r.token(0, tid, 0), left = hi - at;
    TP *p = static_cast<TP *>(a.p) + row * a.p_stride + at;
    const auto put = [&](int32_t g, float (&x)[8]) {
        if (greedy) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = r.token(g, tid, e) == first ? 1.f : 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 y = __fmul2_rn(make_float2(x[e], x[e + 1]), make_float2(f, f));
                x[e] = y.x, x[e + 1] = y.y;
            }
        }
        store_probs<TP, kVec>(p + r.offset(g, 0), kVec ? 1 : kThreads, left - r.offset(g, 0), a.wide, x);
    };
    if constexpr (kLoop) {
        for (int32_t g = 0; g < groups; ++g) {
            r.whole(g, z[0]);
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
constexpr int kCountAhead = 8;  // tokens of a thread in flight

// Many tokens: a CTA per sequence and slice of the vocabulary goes through the
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
    for (int32_t i0 = threadIdx.x; i0 < a.n_tokens; i0 += kCountThreads * kCountAhead) {
        int32_t v[kCountAhead];
#pragma unroll
        for (int e = 0; e < kCountAhead; ++e) {
            const int32_t i = i0 + e * kCountThreads;
            v[e] = i < a.n_tokens ? tokens[i] : -1;
        }
#pragma unroll
        for (int e = 0; e < kCountAhead; ++e) {
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

// Rows of counts from nothing.
__global__ void __launch_bounds__(256) count_clear(const CountArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kPer = 256 * 8 * 2;  // counts of a CTA
    const int32_t parts = (a.vocab + kPer - 1) / kPer, v0 = blockIdx.x % parts * kPer;
    uint16_t *row = a.counts + (int64_t)(blockIdx.x / parts) * a.count_stride;
    const bool vec = ((uintptr_t)a.counts & 15) == 0 && a.count_stride % 8 == 0;
    for (int i = threadIdx.x; i < kPer / 8; i += 256) {
        const int32_t v = v0 + 8 * i;
        if (vec && v + 8 <= a.vocab) {
            *reinterpret_cast<uint4 *>(row + v) = make_uint4(0, 0, 0, 0);
        } else {
            for (int e = 0; e < 8; ++e)
                if (v + e < a.vocab) row[v + e] = 0;
        }
    }
}

// One count, 16 bits by themselves: the array's first or last, where its word is not all the array's.
__device__ void count_alone(uint16_t *count, bool prompt) {
    uint16_t was = *(volatile uint16_t *)count;
    for (;;) {
        const uint16_t next = prompt ? was | 0x8000 : (was & 0x7fff) == 0x7fff ? was : was + 1;
        if (next == was) return;
        const uint16_t seen = atomicCAS(reinterpret_cast<unsigned short *>(count), was, next);
        if (seen == was) return;
        was = seen;
    }
}

// Tokens [from, to) of every sequence added to counts that are there: a thread
// each. Additions and ors that need no answer, unless a count could pass 32767.
__global__ void __launch_bounds__(256) count_each(const CountArgs a, int32_t from, int32_t to) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t at = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (at >= (int64_t)a.n_seqs * (to - from)) return;
    const int32_t s = (int32_t)(at / (to - from)), i = from + (int32_t)(at % (to - from));
    const int32_t v = a.tokens[s * a.token_stride + i];
    if (v >= a.vocab) set_error(a.err, HSWA_ERR_BOUNDS);
    if (v < 0 || v >= a.vocab) return;
    const int32_t prompt = a.n_prompt ? a.n_prompt[s] : 0;
    // the word that the count is half of (the other half stays as it is)
    uint16_t *const count = a.counts + s * a.count_stride + v;
    const uintptr_t n = reinterpret_cast<uintptr_t>(count);
    uint32_t *word = reinterpret_cast<uint32_t *>(n & ~(uintptr_t)3);
    if (reinterpret_cast<uint16_t *>(word) < a.counts ||
        reinterpret_cast<uint16_t *>(word + 1) > a.counts + (a.n_seqs - 1) * a.count_stride + a.vocab) {
        count_alone(count, i < prompt);
        return;
    }
    const int shift = n & 2 ? 16 : 0;
    if (i < prompt) {
        atomicOr(word, 0x8000u << shift);
        return;
    }
    uint32_t was = *(volatile uint32_t *)word;
    if ((int32_t)(was >> shift & 0x7fff) + to - max(from, prompt) <= 0x7fff) {
        atomicAdd(word, 1u << shift);  // all that this launch adds cannot take it past 32767
    } else {
        while ((was >> shift & 0x7fff) != 0x7fff) {
            const uint32_t seen = atomicCAS(word, was, was + (1u << shift));
            if (seen == was) break;
            was = seen;
        }
    }
}

// Atomics on the counts themselves (64 sequences of 4096 tokens added 6.1 us, all
// the same token 12; a cluster that counts in its shared memory and adds to the
// rows 15 and 17, slices 20 and 10). One launch takes up to 2^15 tokens, which cannot
// overflow a count from nothing (one of so many being a prompt's); of more, each
// takes so many that few counts come near it: those need a compare-and-swap, 0.9
// us for each of the same token. Above kEachTokens tokens slices.
constexpr int kEachTokens = 65536, kEachOnce = 1 << 15, kEachPart = 16384;

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

// The groups that a thread of a CTA of 512 has registers for, where a slice needs n.
constexpr int kRowGroups = 5;
int row_groups(int n) { return n <= 2 ? 2 : n <= 4 ? 4 : n; }

// Registers for as few groups as hold a slice: an idle group costs its
// instructions (256 rows of 131000 fp32 under grammars 82 us with 4, 89 with 5). Few
// rows take 1024 threads with half the groups (4 rows of 100003 9.2 us against 9.6);
// many are faster with CTAs of 512, two an SM (256 rows of 150000 79 us, with 1024
// threads of 3 groups 128).
template <typename TL, typename TP, bool kVec>
cudaError_t launch_row(const ProbsArgs &a, int64_t rows, cudaStream_t st) {
    const int32_t groups = (a.slice / 8 + 511) / 512;  // of 512 threads
    if (groups <= 2) return launch<TL, TP, kVec, 512, 2, false>(a, rows, st);
    if (groups <= 4 && rows * a.cluster <= sm_count()) return launch<TL, TP, kVec, 1024, 2, false>(a, rows, st);
    if (groups <= 4) return launch<TL, TP, kVec, 512, 4, false>(a, rows, st);
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
    a.rows = (int32_t)rows;
    a.err = error_word();
    // CTAs per row: few rows spread over the GPU, in slices of at least 1024
    // values; many rows take as many as keep a thread's values in registers (256 rows of
    // 100000, bf16 to fp32, on 5 CTAs of 5 groups 53.5 us, on 8 of 4 63.4; of 50000 on 3 of
    // 5 35.4, on 7 of 2 44). Not the best everywhere: 8 of 2 groups take 34.5 for those
    // 50000, and 37.5 in place of 39.8 where the logits are fp32.
    const int sms = sm_count();
    if (sms <= 0) return HSWA_ERR_CUDA;
    const auto slice_of = [&](int c) { return ((vocab + 8 * c - 1) / (8 * c)) * 8; };
    a.cluster = 1;
    if (rows * 4 <= 2 * sms) {
        while (a.cluster < kMaxCluster &&
               (slice_of(a.cluster) > kRowGroups * 4096 || (rows * a.cluster * 2 <= 2 * sms && slice_of(a.cluster) >= 2048)))
            a.cluster *= 2;
    } else {  // of those that hold the row, where a CTA costs its groups and about three more
        int best = INT32_MAX;
        for (int c = kMaxCluster; c >= 1; --c) {
            const int groups = row_groups((slice_of(c) + 4095) / 4096);
            if (groups > kRowGroups && c < kMaxCluster) break;
            if (c * (groups + 3) < best) best = c * (groups + 3), a.cluster = c;
        }
    }
    a.slice = slice_of(a.cluster);
    a.ahead = rows * a.cluster > 2 * sms ? 2 * sms / a.cluster : 0;
    const bool vec = (x0 & 15) == 0 && (y0 & 15) == 0 && logits_stride * el % 16 == 0 && p_stride * ep % 16 == 0 &&
                     (!counts || (((uintptr_t)counts & 15) == 0 && count_stride % 8 == 0));
    a.wide = (el == 2 || ((x0 & 31) == 0 && logits_stride % 8 == 0)) && (ep == 2 || ((y0 & 31) == 0 && p_stride % 8 == 0));
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
    cudaError_t e = cudaSuccess;
    const int64_t clears = (int64_t)n_seqs * ((vocab + 4095) / 4096);
    if (n_tokens <= kEachTokens && clears <= INT32_MAX) {
        set_last_kernel(n_tokens ? clear ? "count_clear+count_each" : "count_each" : "count_clear");
        if (clear) e = launch_pdl(count_clear, dim3((unsigned)clears), dim3(256), 0, st, a);
        const int32_t part = n_tokens <= kEachOnce ? kEachOnce : kEachPart;
        for (int32_t from = 0; from < n_tokens && e == cudaSuccess; from += part) {
            const int32_t to = std::min(from + part, n_tokens);
            e = launch_pdl(count_each, dim3((unsigned)(((int64_t)n_seqs * (to - from) + 255) / 256)), dim3(256), 0, st, a, from, to);
        }
    } else {
        set_last_kernel("count_slices");
        e = launch_pdl(count_slices, dim3((unsigned)(n_seqs * slices)), dim3(kCountThreads), 0, st, a);
    }
    return e == cudaSuccess ? HSWA_OK : cuda_fail(e, "hswa_count_tokens");
}
