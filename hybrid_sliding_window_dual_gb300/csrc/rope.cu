// Rotary positions with several axes, fused with the KV append.
//
// A head's first R elements form R / 2 pairs; pair i turns by the angle
// pos[axis(i)][t] * f_i. One pass over a token's projections writes the
// rotated q rows where the attention calls read them, the rotated K row and
// the V row into their pool slots (quantized for FP8 pools), so neither q
// nor K makes the extra trip through memory that a rotary pass before
// hswa_append_kv costs.
//
// Angles. f_i / 2 pi is kept as a 64-bit fraction of a turn (made on the
// host in 64-bit floating point), so pos * fraction mod 2^64 is the exact
// phase of that fraction at any int32 position: no range reduction. The
// phase's upper 32 bits give the angle to 2^-25 of a half turn (it is rounded
// to fp32 for sincospif), 1e-7 radians; the fraction's own rounding adds 4e-7
// at position 2^31 (2^-53 of f / 2 pi a position, f = 1).
#include <cmath>
#include <new>

#include <cuda_fp8.h>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"

struct hswa_rope {
    int32_t rotary_dim, n_axes, pairing;
    uint64_t turn[HSWA_ROPE_MAX_DIM / 2];  // f_i / 2 pi, a fraction of 2^64
    uint8_t axis[HSWA_ROPE_MAX_DIM / 2];
};

namespace hswa {
namespace {

struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    void *q_out;                           // [n_tokens][Hq][d]
    void *kp, *vp;
    float *ks, *vs;
    const int32_t *pos;    // [n_axes][n_tokens]
    const int32_t *slots;  // [n_tokens]
    int32_t n_tokens, hq, hkv, d, page, half, adjacent;
    int64_t pool_slots;
    int *err;
    uint64_t turn[HSWA_ROPE_MAX_DIM / 2];
    uint8_t axis[HSWA_ROPE_MAX_DIM / 2];
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// (cos, sin) of pair i for token t
__device__ __forceinline__ float2 rope_turn(const RopeArgs &a, int i, int64_t t) {
    const int32_t p = a.pos[(int64_t)a.axis[i] * a.n_tokens + t];
    const uint64_t phase = (uint64_t)(int64_t)p * a.turn[i];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

// Element e of a head after the rotation; x is the head's row.
template <typename T>
__device__ __forceinline__ float rotated(const T *x, int e, const RopeArgs &a, const float2 *cs) {
    const float xe = to_f(x[e]);
    if (e >= 2 * a.half) return xe;
    const int i = a.adjacent ? e >> 1 : (e < a.half ? e : e - a.half);
    const bool first = a.adjacent ? !(e & 1) : e < a.half;
    const float y = to_f(x[a.adjacent ? e ^ 1 : (first ? e + a.half : e - a.half)]);
    return first ? xe * cs[i].x - y * cs[i].y : xe * cs[i].x + y * cs[i].y;
}

// Any head_dim, rotary dim and alignment: one CTA per token, one warp per
// row, a lane per element. A row is read before any of it is written, so q
// may be rotated in place. Bound by loads and instructions of one element each:
// 4096 bf16 tokens of 64 / 8 heads, 100 of 128 elements turned, take 146 us, 25
// for the bytes at the copy rate; 64 tokens 14.
// kQuant: 0 for pools of T, 8 and 4 for FP8 and FP4 pools.
template <typename T, int kQuant>
__global__ void __launch_bounds__(256) rope_append_any(const __grid_constant__ RopeArgs a) {
    constexpr int kMaxE = HSWA_ROPE_MAX_HEAD / 32;
    __shared__ float2 cs[HSWA_ROPE_MAX_DIM / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    for (int i = threadIdx.x; i < a.half; i += blockDim.x) cs[i] = rope_turn(a, i, t);
    __syncthreads();
    const int32_t slot = a.slots[t];
    const bool kv = slot >= 0 && slot < a.pool_slots;
    if (slot >= a.pool_slots && threadIdx.x == 0) set_error(a.err, HSWA_ERR_BOUNDS);
    const int rows = a.hq + (kv ? 2 * a.hkv : 0);
    for (int r = warp; r < rows; r += 8) {
        const int kind = r < a.hq ? 0 : r < a.hq + a.hkv ? 1 : 2;
        const int h = kind == 0 ? r : kind == 1 ? r - a.hq : r - a.hq - a.hkv;
        const T *x = (kind == 0   ? (const T *)a.q + t * a.q_stride
                      : kind == 1 ? (const T *)a.k + t * a.k_stride
                                  : (const T *)a.v + t * a.v_stride) +
                     (int64_t)h * a.d;
        float y[kMaxE];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxE; ++j) {
            const int e = lane + 32 * j;
            y[j] = e >= a.d ? 0.f : kind == 2 ? to_f(x[e]) : rotated(x, e, a, cs);
            amax = fmaxf(amax, fabsf(y[j]));
        }
        __syncwarp();
        if (kind == 0) {
            T *o = (T *)a.q_out + (t * a.hq + h) * a.d;
            for (int j = 0; j < kMaxE; ++j)
                if (lane + 32 * j < a.d) o[lane + 32 * j] = from_f<T>(y[j]);
            continue;
        }
        const int64_t blk = (int64_t)(slot / a.page) * a.hkv + h;  // (page, kv head) block
        const int32_t row = slot % a.page;
        if constexpr (kQuant == 4) {  // a block is half a warp's elements, a byte two lanes'
            uint8_t *p = (uint8_t *)(kind == 1 ? a.kp : a.vp) + (blk * a.page + row) * (a.d / 2);
            uint8_t *sp = (uint8_t *)(kind == 1 ? a.ks : a.vs) + (blk * a.page + row) * (a.d / kFp4Block);
#pragma unroll
            for (int j = 0; j < kMaxE; ++j) {
                const int e = lane + 32 * j;
                float top = fabsf(y[j]);
                for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const uint32_t scale = fp4_scale(top), code = fp4_code(y[j], scale);
                const uint32_t next = __shfl_xor_sync(0xffffffffu, code, 1);
                if (e < a.d && !(lane & 1)) p[e / 2] = (uint8_t)(code | next << 4);
                if (e < a.d && !(lane & 15)) sp[e / kFp4Block] = (uint8_t)scale;
            }
        } else if constexpr (kQuant == 8) {
            for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
            uint8_t *p = (uint8_t *)(kind == 1 ? a.kp : a.vp) + blk * a.page * a.d;
            for (int j = 0; j < kMaxE; ++j) {
                const int e = lane + 32 * j;
                if (e < a.d)
                    p[kind == 1 ? (int64_t)row * a.d + e : (int64_t)e * a.page + row] =
                        (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(y[j], scale), __NV_SATFINITE, __NV_E4M3);
            }
            if (lane == 0) (kind == 1 ? a.ks : a.vs)[blk * a.page + row] = scale;
        } else {
            T *p = (T *)(kind == 1 ? a.kp : a.vp) + (blk * a.page + row) * a.d;
            for (int j = 0; j < kMaxE; ++j)
                if (lane + 32 * j < a.d) p[lane + 32 * j] = from_f<T>(y[j]);
        }
    }
}

// The usual shapes: 16-byte chunks, two of a row per thread. A thread's two
// chunks are the two halves of 8 (fp32: 4) pairs, or two neighbours where
// pairs are adjacent or nothing turns. blockDim.x threads make a row,
// blockDim.y rows go at a time, kItems of them in flight per thread.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

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

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[kVec<T>]) {
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    else
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Turn pairs: V of them across chunks a and b (halves), or the V / 2 inside
// chunk a (adjacent). cs, sn: from the first of them on.
template <typename T>
__device__ __forceinline__ void turn_across(float (&a)[kVec<T>], float (&b)[kVec<T>], const float *cs, const float *sn) {
#pragma unroll
    for (int i = 0; i < kVec<T>; i += 4) {
        const float4 c = *reinterpret_cast<const float4 *>(cs + i), s = *reinterpret_cast<const float4 *>(sn + i);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = a[i + k], y = b[i + k];
            a[i + k] = x * cc[k] - y * ss[k];
            b[i + k] = x * ss[k] + y * cc[k];
        }
    }
}
template <typename T>
__device__ __forceinline__ void turn_inside(float (&a)[kVec<T>], const float *cs, const float *sn) {
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; i += 2) {
        const float2 c = *reinterpret_cast<const float2 *>(cs + i), s = *reinterpret_cast<const float2 *>(sn + i);
        const float cc[2] = {c.x, c.y}, ss[2] = {s.x, s.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = a[2 * (i + k)], y = a[2 * (i + k) + 1];
            a[2 * (i + k)] = x * cc[k] - y * ss[k];
            a[2 * (i + k) + 1] = x * ss[k] + y * cc[k];
        }
    }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// 8 elements over a scale, as codes: the quotients are correctly rounded
// before they become codes, as in hswa_append_kv. With y the correctly
// rounded 1 / b and q within a step of x / b, q + (x - b q) y rounds to the
// correctly rounded quotient (Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990): the second correction is
// that one, the first makes q near enough. Scales so small or large that the
// remainder is not exact are divided by. (67.6 against 69.7 us on 9999 tokens
// with divisions alone.)
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float scale) {
    float y[8];
    if (scale > 0x1p-90f && scale < 0x1p90f) {
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float q = x[i] * r;
            q = fmaf(fmaf(-scale, q, x[i]), r, q);
            y[i] = copysignf(fmaf(fmaf(-scale, q, x[i]), r, q), x[i]);  // -0 / b is -0
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
    }
    return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}

// The scale of a row of 128 elements, 16 of them in each of 8 neighbouring lanes.
__device__ __forceinline__ float row_scale(const float (&a)[8], const float (&b)[8]) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(a[i]), fabsf(b[i])));
    const uint32_t mates = 0xffu << (threadIdx.y * 8 & 24);  // blockDim.x is 8
    for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mates, amax, off));
    return amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
}

constexpr int kMaxTile = 4;  // tokens per CTA
constexpr int kVTile = 64;   // tokens per CTA of FP8 V rows

// FP8 V: a page keeps V transposed ([d][rows]), so the codes of a tile of
// tokens of one kv head turn around in shared memory and go out token by
// lane: tokens of one sequence are neighbours there, and a warp's bytes for
// one d fill whole sectors. (hswa_append_kv writes them one by one.)
template <int kTokens>
__device__ void rope_v_fp8(const RopeArgs &a, int32_t block) {
    __shared__ uint8_t tile[128][kTokens + 1];  // an odd number of bytes: 8 rows of codes fall into 8 banks
    __shared__ int64_t at[kTokens];  // element (0, row) of the token's page, or -1
    const int tid = threadIdx.y * 8 + threadIdx.x;
    const int64_t t0 = (int64_t)(block / a.hkv) * kTokens;
    const int32_t h = block % a.hkv;
    const int32_t n = (int32_t)min((int64_t)kTokens, a.n_tokens - t0);
    for (int r = threadIdx.y; r < kTokens; r += 32) {
        const bool there = r < n;
        const int64_t t = t0 + (there ? r : 0);
        const int32_t slot = a.slots[t];
        const bool ok = there && slot >= 0 && slot < a.pool_slots;
        const uint4 *x = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.v + t * a.v_stride + h * 128);
        float lo[8], hi[8];
        unpack<__nv_bfloat16>(x[2 * threadIdx.x], lo);
        unpack<__nv_bfloat16>(x[2 * threadIdx.x + 1], hi);
        const float scale = row_scale(lo, hi);
        const uint2 c0 = e4m3x8(lo, scale), c1 = e4m3x8(hi, scale);
        const uint32_t w[4] = {c0.x, c0.y, c1.x, c1.y};
#pragma unroll
        for (int i = 0; i < 16; ++i) tile[threadIdx.x * 16 + i][r] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        if (threadIdx.x == 0) {
            const int64_t blk = ok ? (int64_t)(slot / a.page) * a.hkv + h : 0;
            at[r] = ok ? blk * 128 * a.page + slot % a.page : -1;
            if (ok) a.vs[blk * a.page + slot % a.page] = scale;
        }
    }
    __syncthreads();
    uint8_t *vp = (uint8_t *)a.vp;
    const int r = tid % kTokens;
    if (r < n && at[r] >= 0)
        for (int d = tid / kTokens; d < 128; d += 256 / kTokens) vp[at[r] + (int64_t)d * a.page] = tile[d][r];
}

// kTile tokens per CTA: their q and K rows and, but for FP8 pools, V rows;
// for FP8 pools the CTAs from n_q_blocks on take the V rows.
//
// Bound by memory: a token reads and writes (Hq + 2 Hkv) d elements and does
// three flops for each. What that takes is enough loads in flight, that is
// CTAs per SM more than items per thread: capped at 48 registers (5 CTAs, 2
// items of two 16-byte loads each) 32768 bf16 tokens of 64 / 8 heads take 201
// us, 98 % of the copy bandwidth; at 74 registers with 4 items 268 us. FP8
// codes need more registers (4 CTAs, 3 items): 9999 tokens in 68 us, 85 %;
// 8 us of it is V's turning round, which the tiles at the end of the grid do
// (put first or spread among the others they cost 2 and 7 us more; four
// tokens' codes stored as a word where they make one, 9 more). A
// decode step of 64 tokens takes 3.5 us on the device.
template <typename T, int kQuant, bool kAdjacent, int kTile, int kItems, int kMinCtas>
__global__ void __launch_bounds__(256, kMinCtas) rope_append_vec(const __grid_constant__ RopeArgs a, int32_t n_q_blocks) {
    constexpr int V = kVec<T>;
    __shared__ __align__(16) float cs[kTile][HSWA_ROPE_MAX_DIM / 2], sn[kTile][HSWA_ROPE_MAX_DIM / 2];
    __shared__ int32_t slot_of[kTile];
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (kQuant == 8) {
        if ((int32_t)blockIdx.x >= n_q_blocks) {
            rope_v_fp8<kTile == 1 ? 8 : kVTile>(a, blockIdx.x - n_q_blocks);
            return;
        }
    }
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
    const int nt = (int)min((int64_t)kTile, a.n_tokens - t0);
    const int rows = a.hq + (kQuant == 8 ? 1 : 2) * a.hkv;  // of a token: q, K, V
    const int n = nt * rows, chunks = a.d / V;
    // this thread's two chunks of a row: j-th of the first halves and its
    // partner, or j and j + half the row; neighbours in a warp are neighbours
    // in the row either way, so loads and stores cover whole sectors
    const int j = threadIdx.x, rc = 2 * a.half / V, hc = kAdjacent ? 0 : rc / 2;
    const bool across = j < hc;
    const int rest = chunks - 2 * hc;  // chunks outside pairs of chunks
    const int c0 = across ? j : hc + j, c1 = across ? j + hc : c0 + (rest + 1) / 2;
    const bool two = c1 < chunks;
    uint4 xa[kItems], xb[kItems];
    const auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int r = r0 + i * blockDim.y;
            xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
            if (r >= n) continue;
            const int t = r / rows, h = r - t * rows;
            const T *x = h < a.hq           ? (const T *)a.q + (t0 + t) * a.q_stride + (int64_t)h * a.d
                         : h < a.hq + a.hkv ? (const T *)a.k + (t0 + t) * a.k_stride + (int64_t)(h - a.hq) * a.d
                                            : (const T *)a.v + (t0 + t) * a.v_stride + (int64_t)(h - a.hq - a.hkv) * a.d;
            xa[i] = reinterpret_cast<const uint4 *>(x)[c0];
            if (two) xb[i] = reinterpret_cast<const uint4 *>(x)[c1];
        }
    };
    load(threadIdx.y);  // on their way while the angles are made
    for (int i = tid; i < nt * a.half; i += threads) {
        const int t = i / a.half, p = i - t * a.half;
        const float2 x = rope_turn(a, p, t0 + t);
        cs[t][p] = x.x;
        sn[t][p] = x.y;
    }
    if (tid < nt) {
        const int32_t slot = a.slots[t0 + tid];
        if (slot >= a.pool_slots) set_error(a.err, HSWA_ERR_BOUNDS);
        slot_of[tid] = slot < a.pool_slots ? slot : -1;
    }
    __syncthreads();
    for (int r0 = threadIdx.y; r0 < n; r0 += blockDim.y * kItems) {
        if (r0 != (int)threadIdx.y) load(r0);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int r = r0 + i * blockDim.y;
            if (r >= n) continue;
            const int t = r / rows, h = r - t * rows;
            float lo[V], hi[V];
            unpack<T>(xa[i], lo);
            unpack<T>(xb[i], hi);
            if (h < a.hq + a.hkv) {
                if (!kAdjacent && across) turn_across<T>(lo, hi, &cs[t][c0 * V], &sn[t][c0 * V]);
                if (kAdjacent && c0 < rc) turn_inside<T>(lo, &cs[t][c0 * (V / 2)], &sn[t][c0 * (V / 2)]);
                if (kAdjacent && c1 < rc) turn_inside<T>(hi, &cs[t][c1 * (V / 2)], &sn[t][c1 * (V / 2)]);
            }
            if (h < a.hq) {
                uint4 *o = reinterpret_cast<uint4 *>((T *)a.q_out + ((t0 + t) * a.hq + h) * a.d);
                o[c0] = pack<T>(lo);
                if (two) o[c1] = pack<T>(hi);
                continue;
            }
            const int32_t slot = slot_of[t];
            if (slot < 0) continue;
            const bool is_k = h < a.hq + a.hkv;
            const int64_t blk = (int64_t)(slot / a.page) * a.hkv + (h - a.hq - (is_k ? 0 : a.hkv));
            const int64_t row = blk * a.page + slot % a.page;
            if constexpr (kQuant == 4) {
                // a block is this thread's chunk and its neighbour's (c0 and c1
                // have j's parity: hswa_rope_append sees to it)
                float m0 = 0.f, m1 = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) m0 = fmaxf(m0, fabsf(lo[e])), m1 = fmaxf(m1, fabsf(hi[e]));
                const uint32_t mates = 3u << (tid & 30);
                const uint32_t s0 = fp4_scale(fmaxf(m0, __shfl_xor_sync(mates, m0, 1)));
                const uint32_t s1 = fp4_scale(fmaxf(m1, __shfl_xor_sync(mates, m1, 1)));
                uint32_t *o = reinterpret_cast<uint32_t *>((uint8_t *)(is_k ? a.kp : a.vp) + row * (a.d / 2));
                o[c0] = fp4_codes8(lo, s0);
                o[c1] = fp4_codes8(hi, s1);
                if (!(j & 1)) {
                    uint8_t *sp = (uint8_t *)(is_k ? a.ks : a.vs) + row * (a.d / kFp4Block);
                    sp[c0 / 2] = (uint8_t)s0;
                    sp[c1 / 2] = (uint8_t)s1;
                }
            } else if constexpr (kQuant == 8) {
                const float scale = row_scale(lo, hi);
                uint2 *o = reinterpret_cast<uint2 *>((uint8_t *)a.kp + row * 128);
                o[c0] = e4m3x8(lo, scale);
                o[c1] = e4m3x8(hi, scale);
                if (j == 0) a.ks[row] = scale;
            } else {
                uint4 *o = reinterpret_cast<uint4 *>((T *)(is_k ? a.kp : a.vp) + row * a.d);
                o[c0] = pack<T>(lo);
                if (two) o[c1] = pack<T>(hi);
            }
        }
    }
}

// Tokens from which a CTA takes kMaxTile of them. One token per CTA ends
// soonest while the grid is a few waves; with more, the angles and the start
// of a CTA are paid for too often, the sooner the less there is to do for a
// token: `threads` is its rows times the threads of a row. One token a CTA
// against four, us: 80 threads (8 / 1 heads, d = 128, bf16) 256 tokens 2.8 / 3.3,
// 1024 5.2 / 3.9, 4096 15.7 / 9.3; 160 (16 / 2) 256 2.9 / 4.0, 1024 5.5 / 4.8; 320 (32
// / 4) 1024 6.7 / 6.6, 2048 12.2 / 11.5; 640 (64 / 8) 2048 15.9 / 19.8, 4096 36.9 /
// 32.2; fp32 32 / 4 heads 2048 13.3 / 16.8, 4096 32.4 / 32.0, 64 / 8 4096 52 / 58,
// 16384 equal; FP8 32 / 4 1024 9.2 / 9.4, 2048 16.0 / 11.2, 64 / 8 1280 14.5 / 16.0, 1536
// 17.1 / 16.4; FP4 64 / 8 2560 25.7 / 26.0, 4096 40.5 / 33.7, 32 / 4 4096 27.0 /
// 18.0. (Up to 16 tokens a CTA for few heads gained nothing.)
template <typename T, int kQuant>
int tile_from(int threads) {
    if (threads <= 160) return 640;
    if (threads <= 320) return 1024;
    if (kQuant == 8) return 1440;
    return threads > 640 ? 8192 : sizeof(T) == 2 ? 2560 : 4096;
}

template <typename T, int kQuant, bool kAdjacent>
cudaError_t launch_rope_vec(const RopeArgs &a, cudaStream_t st) {
    const int units = (a.d / kVec<T> + 1) / 2;  // threads of a row
    const int rows = a.hq + (kQuant == 8 ? 1 : 2) * a.hkv;
    const bool tiled = a.n_tokens >= tile_from<T, kQuant>(rows * units);
    const int64_t nq = tiled ? ((int64_t)a.n_tokens + kMaxTile - 1) / kMaxTile : a.n_tokens;
    const int64_t vt = tiled ? kVTile : 8;
    const int64_t nv = kQuant == 8 ? (a.n_tokens + vt - 1) / vt * a.hkv : 0;
    const dim3 grid((unsigned)(nq + nv)), block(units, 256 / units);
    // FP4, 32768 tokens of 64 / 8 heads: 216 us with 2 items, 224 with 3; 188 at a plain
    // copy's rate, the quantizer's instructions between
    constexpr int kItems = kQuant == 8 || kAdjacent ? 3 : 2, kMinCtas = kQuant || kAdjacent ? 4 : 5;
    return tiled ? launch_pdl(rope_append_vec<T, kQuant, kAdjacent, kMaxTile, kItems, kMinCtas>, grid, block, 0, st, a, (int32_t)nq)
                 : launch_pdl(rope_append_vec<T, kQuant, kAdjacent, 1, 3, 4>, grid, block, 0, st, a, (int32_t)nq);
}

}  // namespace
}  // namespace hswa

using namespace hswa;

extern "C" int hswa_rope_create(const hswa_rope_config *cfg, hswa_rope **out) {
    if (!cfg || !out || cfg->rotary_dim < 2 || cfg->rotary_dim > HSWA_ROPE_MAX_DIM || cfg->rotary_dim % 2 ||
        cfg->n_axes < 1 || cfg->n_axes > HSWA_ROPE_MAX_AXES ||
        (cfg->pairing != HSWA_ROPE_HALVES && cfg->pairing != HSWA_ROPE_ADJACENT) ||
        (cfg->order != HSWA_ROPE_SECTIONS && cfg->order != HSWA_ROPE_INTERLEAVED))
        return HSWA_ERR_INVALID_ARG;
    const int half = cfg->rotary_dim / 2, n = cfg->n_axes;
    int64_t total = 0;
    for (int x = 0; x < n; ++x) {
        if (cfg->section[x] < 0) return HSWA_ERR_INVALID_ARG;
        total += cfg->section[x];
    }
    if (total != half) return HSWA_ERR_INVALID_ARG;
    if (!cfg->inv_freq && !(cfg->theta > 0.0 && std::isfinite(cfg->theta))) return HSWA_ERR_INVALID_ARG;
    hswa_rope *r = new (std::nothrow) hswa_rope();
    if (!r) return HSWA_ERR_INVALID_ARG;
    r->rotary_dim = cfg->rotary_dim;
    r->n_axes = n;
    r->pairing = cfg->pairing;
    int count[HSWA_ROPE_MAX_AXES] = {};
    for (int i = 0; i < half; ++i) {
        int x = 0;
        if (cfg->order == HSWA_ROPE_SECTIONS) {
            for (int at = cfg->section[0]; i >= at; at += cfg->section[x]) ++x;
        } else {
            x = i % n;
            if (i / n >= cfg->section[x]) x = 0;
        }
        r->axis[i] = (uint8_t)x;
        ++count[x];
        const double f = cfg->inv_freq ? cfg->inv_freq[i] : std::pow(cfg->theta, -2.0 * i / cfg->rotary_dim);
        if (!std::isfinite(f)) {
            delete r;
            return HSWA_ERR_INVALID_ARG;
        }
        double turn = f * 0.15915494309189533577;  // 1 / (2 pi)
        turn -= std::floor(turn);                  // positions are whole numbers: whole turns drop out
        r->turn[i] = turn < 1.0 ? (uint64_t)std::ldexp(turn, 64) : 0;
    }
    for (int x = 0; x < n; ++x)
        if (count[x] != cfg->section[x]) {  // interleaved sections that do not fit their turns
            delete r;
            return HSWA_ERR_INVALID_ARG;
        }
    *out = r;
    return HSWA_OK;
}

extern "C" int hswa_rope_destroy(hswa_rope *rope) {
    if (!rope) return HSWA_ERR_INVALID_ARG;
    delete rope;
    return HSWA_OK;
}

extern "C" int hswa_rope_append(const hswa_pool *pool, const hswa_layer *layer, const hswa_rope *rope, const void *q,
                                int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                const int32_t *d_pos, const int32_t *d_slots, void *q_out, int n_tokens,
                                hswa_stream_t stream) {
    HSWA_NVTX("hswa_rope_append");
    if (!pool || !layer || !rope || n_tokens < 0 || !layer->k_pool || !layer->v_pool ||
        (layer->kind != HSWA_KIND_FULL && layer->kind != HSWA_KIND_SWA))
        return HSWA_ERR_INVALID_ARG;
    const hswa_config &c = pool->cfg;
    const bool fp8 = c.dtype == HSWA_DTYPE_FP8_E4M3, fp4 = c.dtype == HSWA_DTYPE_FP4;
    if (rope->rotary_dim > c.head_dim) return HSWA_ERR_INVALID_ARG;
    if (c.head_dim > HSWA_ROPE_MAX_HEAD || (fp8 && c.head_dim != 128) || (fp4 && c.head_dim % kFp4Block))
        return HSWA_ERR_UNSUPPORTED;
    if ((fp8 || fp4) && (!layer->k_scale || !layer->v_scale)) return HSWA_ERR_INVALID_ARG;
    if (n_tokens == 0) return HSWA_OK;
    const int64_t q_row = (int64_t)c.n_q_heads * c.head_dim, kv_row = (int64_t)c.n_kv_heads * c.head_dim;
    if (!q || !k || !v || !d_pos || !d_slots || !q_out || q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
        return HSWA_ERR_INVALID_ARG;
    const int64_t e = c.dtype == HSWA_DTYPE_F32 ? 4 : 2;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & (e - 1)) return HSWA_ERR_INVALID_ARG;
    // q_out apart from q, k and v, or q itself when q is packed already
    const uintptr_t o0 = (uintptr_t)q_out, o1 = o0 + (uintptr_t)(n_tokens * q_row * e);
    const auto meets = [&](const void *x, int64_t stride, int64_t row) {
        const uintptr_t x0 = (uintptr_t)x, x1 = x0 + (uintptr_t)(((n_tokens - 1) * stride + row) * e);
        return x0 < o1 && o0 < x1;
    };
    if (meets(k, k_stride, kv_row) || meets(v, v_stride, kv_row) ||
        (meets(q, q_stride, q_row) && !(q == q_out && q_stride == q_row)))
        return HSWA_ERR_INVALID_ARG;
    RopeArgs a;
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.q_out = q_out;
    a.kp = layer->k_pool, a.vp = layer->v_pool;
    a.ks = layer->k_scale, a.vs = layer->v_scale;
    a.pos = d_pos, a.slots = d_slots;
    a.n_tokens = n_tokens, a.hq = c.n_q_heads, a.hkv = c.n_kv_heads, a.d = c.head_dim, a.page = c.page_size;
    a.half = rope->rotary_dim / 2;
    a.adjacent = rope->pairing == HSWA_ROPE_ADJACENT;
    a.pool_slots = (int64_t)(layer->kind == HSWA_KIND_SWA ? c.swa_pages : c.full_pages) * c.page_size;
    a.err = error_word();
    std::copy(rope->turn, rope->turn + a.half, a.turn);
    std::copy(rope->axis, rope->axis + a.half, a.axis);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // 16-byte chunks need every row on a 16-byte boundary and the turning part
    // in whole pairs of chunks; the plain kernel takes the rest
    const int64_t w = 16 / e;
    const uintptr_t bases = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)a.kp | (uintptr_t)a.vp;
    const bool vec = rope->rotary_dim % (a.adjacent ? w : 2 * w) == 0 && c.head_dim % w == 0 && (q_stride | k_stride | v_stride) % w == 0 &&
                     (bases & 15) == 0 &&
                     // FP4: the two chunks of a block belong to neighbouring threads
                     (!fp4 || (c.head_dim % 32 == 0 && (a.adjacent || rope->rotary_dim % 32 == 0))) &&
                     n_tokens + (fp8 ? (n_tokens + INT64_C(7)) / 8 * c.n_kv_heads : 0) <= INT32_MAX;
    cudaError_t rc;
    if (vec) {
        set_last_kernel(fp8 ? "rope_append_fp8" : fp4 ? "rope_append_fp4" : e == 4 ? "rope_append_f32" : "rope_append_bf16");
        if (fp8)
            rc = a.adjacent ? launch_rope_vec<__nv_bfloat16, 8, true>(a, st) : launch_rope_vec<__nv_bfloat16, 8, false>(a, st);
        else if (fp4)
            rc = a.adjacent ? launch_rope_vec<__nv_bfloat16, 4, true>(a, st) : launch_rope_vec<__nv_bfloat16, 4, false>(a, st);
        else if (e == 4)
            rc = a.adjacent ? launch_rope_vec<float, 0, true>(a, st) : launch_rope_vec<float, 0, false>(a, st);
        else
            rc = a.adjacent ? launch_rope_vec<__nv_bfloat16, 0, true>(a, st) : launch_rope_vec<__nv_bfloat16, 0, false>(a, st);
    } else {
        set_last_kernel(fp8 ? "rope_append_any_fp8" : fp4 ? "rope_append_any_fp4" : e == 4 ? "rope_append_any_f32" : "rope_append_any_bf16");
        if (fp8)
            rope_append_any<__nv_bfloat16, 8><<<n_tokens, 256, 0, st>>>(a);
        else if (fp4)
            rope_append_any<__nv_bfloat16, 4><<<n_tokens, 256, 0, st>>>(a);
        else if (e == 4)
            rope_append_any<float, 0><<<n_tokens, 256, 0, st>>>(a);
        else
            rope_append_any<__nv_bfloat16, 0><<<n_tokens, 256, 0, st>>>(a);
        rc = cudaGetLastError();
    }
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_rope_append");
}
