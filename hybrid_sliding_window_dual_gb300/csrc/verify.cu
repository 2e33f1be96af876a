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
// product is exact. For the draw, probabilities are counted in whole steps
// and their differences summed as integers of up to 96 bits, so the sums, and
// with them the token, do not depend on how the row is split.
#include "common.cuh"
#include "internal.h"

namespace hswa {
namespace {

constexpr int kWarps = 16;
constexpr int kMaxCluster = 8;  // CTAs per sequence
constexpr int kMaxPart = 8192;  // positions of a warp

typedef unsigned __int128 u128;

struct VerifyArgs {
    const void *p, *q;
    int64_t p_stride, q_stride;
    const int32_t *draft, *n_draft;
    const float *u;
    int32_t n_tok, vocab, cluster, part;  // part: positions of a warp's slice
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

// Two fp32 values in a register pair, which one instruction adds to another
// pair. Each operation is rounded as on single values. Worth it where
// instructions bound the kernel: 256 rows of bf16 18.2 us against 19.1; fp32
// rows of both models, which memory bounds, 18.4 against 18.5, and 19.2 with
// the subtractions in pairs too.
struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ uint32_t lo() const { return (uint32_t)v; }
    __device__ __forceinline__ uint32_t hi() const { return (uint32_t)(v >> 32); }
};
__device__ __forceinline__ Pair operator+(Pair x, Pair y) {
    Pair z;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z.v) : "l"(x.v), "l"(y.v));
    return z;
}
__device__ __forceinline__ Pair operator-(Pair x, Pair y) {  // x + (-1) y is rounded once
    Pair z;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z.v) : "l"(y.v), "l"(Pair(-1.f, -1.f).v), "l"(x.v));
    return z;
}
__device__ __forceinline__ Pair minus_each(Pair x, Pair y) {
    return Pair(__fsub_rn(__uint_as_float(x.lo()), __uint_as_float(y.lo())),
                __fsub_rn(__uint_as_float(x.hi()), __uint_as_float(y.hi())));
}

// A sum of probabilities in whole steps: 2^-50 for fp32, 2^-45 for bf16,
// whose 8 significant bits that holds down to 2^-37. A value is cut into
// digits of 16 or 22 bits by adding a power of two whose last place is the
// digit's: the low bits of the sum are the digit, rounded to nearest, and
// what is left over is exact. That is 4 or 7 additions, of two values at
// once; a conversion to a 64-bit integer took 20 times as long. 32-bit digits
// hold 2^9 values, and are emptied into 64 bits before that.
template <typename T>
struct Steps;

template <>
struct Steps<float> {
    uint32_t a = 0, b = 0, c = 0;  // units of 2^-16, 2^-33, 2^-50; signed, modulo 2^32

    struct Digits {
        Pair a, b, c;  // off by the constants' bits
    };
    static __device__ __forceinline__ Digits digits(Pair x) {
        const Pair one(128.f, 128.f), two(0x1.8p-10f, 0x1.8p-10f), three(0x1.8p-27f, 0x1.8p-27f);
        const Pair t = x + one, r = minus_each(x, minus_each(t, one));
        const Pair u = r + two, q = minus_each(r, minus_each(u, two));
        return {t, u, q + three};
    }
    // add_raw leaves the constants in; drop takes n values' out
    __device__ __forceinline__ void add_raw(Pair x) {
        const Digits d = digits(x);
        a += d.a.lo() + d.a.hi(), b += d.b.lo() + d.b.hi(), c += d.c.lo() + d.c.hi();
    }
    __device__ __forceinline__ void drop(int n) {
        a -= n * 0x43000000, b -= n * 0x3ac00000, c -= n * 0x32400000;  // 128, 1.5 2^-10, 1.5 2^-27
    }
    __device__ __forceinline__ void add_difference(Pair x, Pair y) {
        const Digits d = digits(x), z = digits(y);
        a += d.a.lo() + d.a.hi(), b += d.b.lo() + d.b.hi(), c += d.c.lo() + d.c.hi();
        a -= z.a.lo() + z.a.hi(), b -= z.b.lo() + z.b.hi(), c -= z.c.lo() + z.c.hi();
    }
    __device__ __forceinline__ uint64_t total() const {
        return (uint64_t)(((int64_t)(int32_t)a << 34) + ((int64_t)(int32_t)b << 17) + (int32_t)c);
    }
};

template <>
struct Steps<__nv_bfloat16> {
    uint32_t a = 0, b = 0;  // units of 2^-22, 2^-45; signed, modulo 2^32

    struct Digits {
        Pair a, b;
    };
    static __device__ __forceinline__ Digits digits(Pair x) {
        const Pair t = x + Pair(2.f, 2.f), r = x - (t + Pair(-2.f, -2.f));
        return {t, r + Pair(0x1.8p-22f, 0x1.8p-22f)};
    }
    __device__ __forceinline__ void add_raw(Pair x) {
        const Digits d = digits(x);
        a += d.a.lo() + d.a.hi(), b += d.b.lo() + d.b.hi();
    }
    __device__ __forceinline__ void drop(int n) {
        a -= n * 0x40000000, b -= n * 0x34c00000;  // 2, 1.5 2^-22
    }
    __device__ __forceinline__ void add_difference(Pair x, Pair y) {
        const Digits d = digits(x), z = digits(y);
        a += d.a.lo() + d.a.hi(), b += d.b.lo() + d.b.hi();
        a -= z.a.lo() + z.a.hi(), b -= z.b.lo() + z.b.hi();
    }
    __device__ __forceinline__ uint64_t total() const { return (uint64_t)(((int64_t)(int32_t)a << 23) + (int32_t)b); }
};

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int m) {
    return __shfl_xor_sync(0xffffffffu, (unsigned long long)x, m);
}

// floor(u x) for u in [0, 1)
__device__ u128 times_fraction(u128 x, float u) {
    const uint32_t b = __float_as_uint(u);
    const int e = (int)(b >> 23);
    const uint32_t m = e ? (b & 0x7fffff) | 0x800000 : b & 0x7fffff;
    const int shift = 150 - (e ? e : 1);  // u = m 2^-shift, shift in [24, 149]
    return shift < 128 ? (x * m) >> shift : 0;
}

// Elements of a 16-byte load, and loads of a row in flight per thread (with
// two rows 8 in all; fewer, or twice the threads with half of them, were 3 to
// 30 % slower on 64 sequences, 8 in place of 4 of each row 12 %).
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
// Rows off a 16-byte boundary take one element a load, and twice as many loads
// (183 sequences of 100003 fp32 values 41 us, with as many 50; 64 of bf16 12.3,
// with as many 14.3, with four times as many 15.2; one row alone: 256 of 32001
// bf16 9.6, with as many 10.6).
template <bool kBoth, int kWide>
constexpr int kUnroll = (kBoth ? 4 : 8) * (kWide == 1 ? 2 : 1);

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &c, float (&x)[kVec<T>]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(c.x), x[1] = __uint_as_float(c.y);
        x[2] = __uint_as_float(c.z), x[3] = __uint_as_float(c.w);
    } else {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// What a sequence draws from: the target's row less the draft's (less
// everything at `gone`, the drafted token, when the draft was greedy).
template <typename T>
struct Weights {
    const T *p, *q;
    int32_t gone;

    // Add two positions' weights, but for `gone`. __saturatef: [0, 1], NaN as
    // 0. With one row the constants stay in (Steps::drop).
    template <bool kBoth>
    static __device__ __forceinline__ void add(Steps<T> &sum, float px, float qx, float px1 = 0.f, float qx1 = 0.f) {
        const float x = __saturatef(px), x1 = __saturatef(px1);
        if constexpr (kBoth)
            sum.add_difference({x, x1}, {fminf(x, __saturatef(qx)), fminf(x1, __saturatef(qx1))});
        else
            sum.add_raw({x, x1});
    }
    __device__ __forceinline__ uint64_t at(int32_t i) const {
        if (i == gone) return 0;
        Steps<T> sum;
        if (q) {
            add<true>(sum, prob(p, i), prob(q, i));
        } else {
            add<false>(sum, prob(p, i), 0.f);
            sum.drop(2);
        }
        return sum.total();
    }

    // Sum of this lane's share of positions [i0, i0 + kUnroll * 32 * kWide) of
    // a row that ends at hi: kUnroll loads of each row in flight, of 16 bytes
    // where both rows are aligned (positions count from a vector's first).
    template <int kWide, bool kBoth>
    __device__ __forceinline__ uint64_t chunk(int32_t i0, int32_t hi) const {
        const int lane = threadIdx.x & 31;
        constexpr int kUnroll = hswa::kUnroll<kBoth, kWide>;
        Steps<T> sum;
        if constexpr (kWide > 1) {
            uint4 a[kUnroll], b[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int32_t i = i0 + (k * 32 + lane) * kWide;
                a[k] = b[k] = make_uint4(0, 0, 0, 0);
                if (i + kWide <= hi) {
                    a[k] = *reinterpret_cast<const uint4 *>(p + i);
                    if constexpr (kBoth) b[k] = *reinterpret_cast<const uint4 *>(q + i);
                }
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                float x[kWide], y[kWide];
                unpack<T>(a[k], x);
                unpack<T>(b[k], y);
#pragma unroll
                for (int e = 0; e < kWide; e += 2) add<kBoth>(sum, x[e], y[e], x[e + 1], y[e + 1]);
            }
            // the row's last elements, short of a vector
            const int32_t i = hi / kWide * kWide + lane;
            if (i < hi && i >= i0 && i < i0 + kUnroll * 32 * kWide) {
                add<kBoth>(sum, prob(p, i), kBoth ? prob(q, i) : 0.f);
                if (!kBoth) sum.drop(2);
            }
        } else {
            float x[kUnroll], y[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int32_t i = i0 + k * 32 + lane;
                x[k] = i < hi ? prob(p, i) : 0.f;
                y[k] = kBoth && i < hi ? prob(q, i) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kUnroll; k += 2) add<kBoth>(sum, x[k], y[k], x[k + 1], y[k + 1]);
        }
        if (!kBoth) sum.drop(kUnroll * kWide);
        uint64_t total = sum.total();
        if (!kBoth && lane == 0 && gone >= i0 && gone < min(i0 + kUnroll * 32 * kWide, hi)) {
            Steps<T> x;
            add<false>(x, prob(p, gone), 0.f);
            x.drop(2);
            total -= x.total();  // the warp's sum stays at or above 0
        }
        return total;
    }

    // The warp's slice [lo, hi), a chunk at a time: lane k keeps the sums of
    // chunks k and 32 + k. The slice's sum.
    template <int kWide, bool kBoth>
    __device__ __forceinline__ uint64_t slice(int32_t lo, int32_t hi, uint64_t (&chunks)[2]) const {
        const int lane = threadIdx.x & 31;
        uint64_t total = 0;
        chunks[0] = chunks[1] = 0;
        int c = 0;
        for (int32_t i0 = lo; i0 < hi; i0 += kUnroll<kBoth, kWide> * 32 * kWide, ++c) {
            uint64_t x = chunk<kWide, kBoth>(i0, hi);
            for (int m = 16; m > 0; m >>= 1) x += shfl_xor64(x, m);
            if (lane == c) chunks[0] = x;
            if (lane + 32 == c) chunks[1] = x;
            total += x;
        }
        return total;
    }
};

// Slices of rows off a 16-byte boundary: of fp32 rows out of line, since the
// registers of their loads cost the 16-byte path more (64 sequences of 150000
// values 17.8 us, in line 19.0) than the call costs them (of 100003 14.5, in line
// 13.2); of bf16 rows in line (18.2 and 19.0 on the greedy rows).
template <typename T, bool kBoth>
__device__ __noinline__ uint64_t narrow_call(const Weights<T> &w, int32_t lo, int32_t hi, uint64_t (&chunks)[2]) {
    return w.template slice<1, kBoth>(lo, hi, chunks);
}
template <typename T, bool kBoth>
__device__ __forceinline__ uint64_t narrow_slice(const Weights<T> &w, int32_t lo, int32_t hi, uint64_t (&chunks)[2]) {
    if constexpr (sizeof(T) == 4)
        return narrow_call<T, kBoth>(w, lo, hi, chunks);
    else
        return w.template slice<1, kBoth>(lo, hi, chunks);
}

// One cluster of a.cluster CTAs per sequence. Every CTA settles the
// acceptance tests for itself (two rounds of loads); each warp sums its slice
// of the row; the CTAs tell each other their sums through distributed shared
// memory; the warp whose slice the draw falls into finds its chunk, by the
// sums that its lanes kept; and its CTA finds the token there. (One warp
// alone takes 5 us longer for that: its instructions wait on each other.)
//
// Bound by memory while a row is read (64 sequences, 150000 fp32 values: 10
// us of 17.8, for 11.3 of bytes at the copy rate less what L2 holds; 256 of
// 131000 bf16 values, greedy: 10 to 11 of 18.3, for 9.9); before and after
// comes a fixed 5 to 6 us of dependent loads and barriers: the launch 2, the
// tests 1, the CTAs' sums 1.5, the token 2. One sequence of 100003 takes 6.1
// us on the device.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps, 2) verify_draft(const __grid_constant__ VerifyArgs a) {
    __shared__ uint64_t s_cta[2][kMaxCluster][2];  // sums of the cluster's CTAs (low, high), both passes
    __shared__ uint64_t s_warp[kWarps];
    __shared__ uint64_t s_left;
    __shared__ int32_t s_accept, s_last, s_from, s_end;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % a.cluster;
    const int64_t s = blockIdx.x / a.cluster;
    const int n_rows = a.n_tok - 1;  // drafts a sequence can have
    cluster_arrive();  // awaited before the first store into another CTA's shared memory
    pdl_wait();
    pdl_launch_dependents();
    const float u_draw = a.u[s * a.n_tok + n_rows];
    if (warp == 0) {
        const bool row = lane < n_rows;
        int32_t n = a.n_draft ? a.n_draft[s] : n_rows;
        const int32_t x = row ? a.draft[s * n_rows + lane] : 0;
        const float u = row ? a.u[s * a.n_tok + lane] : 0.f;
        const bool inside = x >= 0 && x < a.vocab;
        double px = 0.0, qx = 1.0;
        if (row && inside) {
            px = prob((const T *)a.p + (s * a.n_tok + lane) * a.p_stride, x);
            if (a.q) qx = prob((const T *)a.q + (s * n_rows + lane) * a.q_stride, x);
        }
        bool bad = n < 0 || n > n_rows;
        n = max(0, min(n, n_rows));
        bad |= lane < n && !inside;
        const bool stays = lane < n && inside && (double)u * qx < px;
        if (bad && rank == 0) set_error(a.err, HSWA_ERR_BOUNDS);
        const unsigned gone = __ballot_sync(0xffffffffu, !stays);  // lanes past the drafts are in it
        const int32_t acc = __ffs(gone) - 1;
        if (lane == 0) {
            s_accept = acc;
            s_last = n;
        }
        if (rank == 0) {
            if (lane == 0) a.n_accept[s] = acc;
            if (lane < a.n_tok && lane != acc) a.tokens[s * a.n_tok + lane] = lane < acc ? x : -1;
        }
    }
    __syncthreads();
    const int32_t acc = s_accept;
    const bool refused = acc < s_last;
    Weights<T> w;
    w.p = (const T *)a.p + (s * a.n_tok + acc) * a.p_stride;
    w.q = refused && a.q ? (const T *)a.q + (s * n_rows + acc) * a.q_stride : nullptr;
    w.gone = refused && !a.q ? a.draft[s * n_rows + acc] : -1;
    constexpr int V = kVec<T>;
    const int32_t lo = (int32_t)min((int64_t)(rank * kWarps + warp) * a.part, (int64_t)a.vocab);
    const int32_t hi = min(lo + a.part, a.vocab);
    u128 total = 0;
    uint64_t chunks[2], sum;
    bool wide;
    int pass = 0;
    while (true) {
        wide = (((uintptr_t)w.p | (uintptr_t)w.q) & 15) == 0;
        if (w.q)
            sum = wide ? w.template slice<V, true>(lo, hi, chunks) : narrow_slice<T, true>(w, lo, hi, chunks);
        else
            sum = wide ? w.template slice<V, false>(lo, hi, chunks) : narrow_slice<T, false>(w, lo, hi, chunks);
        if (lane == 0) s_warp[warp] = sum;
        if (pass == 0) cluster_wait();  // every CTA of the cluster has started
        __syncthreads();
        if (threadIdx.x < a.cluster) {
            u128 x = 0;
            for (int i = 0; i < kWarps; ++i) x += s_warp[i];
            st_cluster_u64(&s_cta[pass][rank][0], threadIdx.x, (uint64_t)x);
            st_cluster_u64(&s_cta[pass][rank][1], threadIdx.x, (uint64_t)(x >> 64));
        }
        cluster_arrive();
        cluster_wait();
        total = 0;
        for (int i = 0; i < a.cluster; ++i) total += ((u128)s_cta[pass][i][1] << 64) + s_cta[pass][i][0];
        if (total != 0 || pass == 1 || (!w.q && w.gone < 0)) break;
        w.q = nullptr;  // nothing is left of the target where the draft was: draw from the target itself
        w.gone = -1;
        pass = 1;
    }
    if (total == 0) {  // a row without a positive value
        if (rank == 0 && threadIdx.x == 0) a.tokens[s * a.n_tok + acc] = -1;
        return;
    }
    // whose slice does u times the total fall into?
    u128 left = times_fraction(total, fminf(fmaxf(u_draw, 0.f), 0x1.fffffep-1f));
    for (int i = 0; i < rank; ++i) left -= ((u128)s_cta[pass][i][1] << 64) + s_cta[pass][i][0];
    const u128 mine = ((u128)s_cta[pass][rank][1] << 64) + s_cta[pass][rank][0];
    if (left >= mine) return;  // another CTA's; wrapped round if it came before
    for (int i = 0; i < warp; ++i) left -= s_warp[i];
    if (left < sum) {
        uint64_t t = (uint64_t)left;
        const int32_t step = wide ? (w.q ? kUnroll<true, V> : kUnroll<false, V>) * 32 * V
                                  : (w.q ? kUnroll<true, 1> : kUnroll<false, 1>) * 32;
        int32_t c = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the chunk, among 32 at a time
            uint64_t upto = chunks[half];
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, (unsigned long long)upto, off);
                if (lane >= off) upto += y;
            }
            const unsigned mask = __ballot_sync(0xffffffffu, upto > t);
            const int at = mask ? __ffs(mask) - 1 : 31;
            t -= __shfl_sync(0xffffffffu, (unsigned long long)(mask ? upto - chunks[half] : upto), at);
            if (mask) {
                c = half * 32 + at;
                break;
            }
        }
        if (lane == 0) {
            s_from = lo + c * step;
            s_end = min(lo + (c + 1) * step, hi);
            s_left = t;
        }
    }
    __syncthreads();
    // the token in the chunk (256 to 2048 positions): neighbours in a thread
    const int32_t each = (s_end - s_from + 32 * kWarps - 1) / (32 * kWarps);  // at most 4
    const int32_t i0 = s_from + threadIdx.x * each, end = min(i0 + each, s_end);
    uint64_t x[4], here = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = i0 + k < end ? w.at(i0 + k) : 0;
        here += x[k];
    }
    uint64_t upto = here;  // inclusive sums over the warp, then over the warps before it
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, (unsigned long long)upto, off);
        if (lane >= off) upto += y;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
        if (i < warp) upto += s_warp[i];
    const uint64_t t = s_left;
    if (upto > t && upto - here <= t) {  // one thread
        uint64_t rest = t - (upto - here);
        int32_t at = i0;
        bool open = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            open = open && rest >= x[k];
            if (open) rest -= x[k], ++at;
        }
        a.tokens[s * a.n_tok + acc] = at;
    }
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
    if (vocab > HSWA_VERIFY_MAX_VOCAB || n_seqs > INT32_MAX / kMaxCluster) return HSWA_ERR_UNSUPPORTED;
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
    // As many CTAs per sequence as fit the GPU at once (2 per SM), so that a
    // few sequences spread over it and many keep to one CTA each; enough of
    // them that a slice's sum of ones, 2^50 steps each, stays below 2^64 and
    // a slice has at most 64 chunks.
    const int sms = sm_count();
    if (sms <= 0) return HSWA_ERR_CUDA;
    const auto part_of = [&](int c) { return ((vocab + c * kWarps - 1) / (c * kWarps) + 7) / 8 * 8; };
    a.cluster = 1;
    while (a.cluster < kMaxCluster && (n_seqs * (int64_t)a.cluster * 2 <= 2 * sms || part_of(a.cluster) > kMaxPart))
        a.cluster *= 2;
    a.part = part_of(a.cluster);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_seqs * a.cluster);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    set_last_kernel(e == 4 ? "verify_draft_f32" : "verify_draft_bf16");
    const cudaError_t rc = e == 4 ? cudaLaunchKernelEx(&cfg, verify_draft<float>, a)
                                  : cudaLaunchKernelEx(&cfg, verify_draft<__nv_bfloat16>, a);
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_verify_draft");
}
