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
// phase of any int32 position: no range reduction, and far positions lose
// nothing. The phase's upper 32 bits give the angle to 2^-25 of a half turn
// (it is rounded to fp32 for sincospif): 1e-7 radians.
#include <cmath>
#include <new>

#include <cuda_fp8.h>

#include "common.cuh"
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
// may be rotated in place.
template <typename T, bool kFP8>
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
        if constexpr (kFP8) {
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
    const bool fp8 = c.dtype == HSWA_DTYPE_FP8_E4M3;
    if (rope->rotary_dim > c.head_dim) return HSWA_ERR_INVALID_ARG;
    if (c.head_dim > HSWA_ROPE_MAX_HEAD || (fp8 && c.head_dim != 128)) return HSWA_ERR_UNSUPPORTED;
    if (fp8 && (!layer->k_scale || !layer->v_scale)) return HSWA_ERR_INVALID_ARG;
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
    set_last_kernel(fp8 ? "rope_append_any_fp8" : e == 4 ? "rope_append_any_f32" : "rope_append_any_bf16");
    if (fp8)
        rope_append_any<__nv_bfloat16, true><<<n_tokens, 256, 0, st>>>(a);
    else if (e == 4)
        rope_append_any<float, false><<<n_tokens, 256, 0, st>>>(a);
    else
        rope_append_any<__nv_bfloat16, false><<<n_tokens, 256, 0, st>>>(a);
    const cudaError_t rc = cudaGetLastError();
    return rc == cudaSuccess ? HSWA_OK : cuda_fail(rc, "hswa_rope_append");
}
