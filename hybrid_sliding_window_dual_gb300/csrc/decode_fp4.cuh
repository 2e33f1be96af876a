// Decode over FP4 pools (d = 128, 8 query heads per kv head, page 64): part of
// decode.cu, whose plan, partial records and merge it shares.
//
// The bytes of a page and kv head are 9 KB, 1.83 times fewer than in FP8, and
// the work to turn codes into MMA operands is the same, so that here the
// instructions of an element, not the loads, decide how near the kernel comes
// to the memory's rate. Every choice below saves some:
//   * A warp is a worker of its own. It takes an equal share of the units (a
//     page of a kv head), streams them through its own ring of kFp4Stages
//     stages and leaves its own partial records: no barriers between warps,
//     no producer, one wait for 64 keys.
//   * Codes become f16 pairs by the conversion instruction, two at a time, and
//     are multiplied by their block's scale as pairs, which is exact (see
//     fp4.cuh). No layout change follows: both pools keep a token's codes in a
//     row, and the MMAs are arranged so that those pairs are operands as they
//     stand.
//   * S = Q K^T: keys are the columns of B. Lane (g, t) holds 32 d's of one
//     key per 8-key tile (one 16-byte load, two scales); the contraction takes
//     d = 32 t + 4 s + 0..3 in step s from lane t, and Q's fragments follow.
//   * O += P V, one token: a pair holds two d's of one key where B wants two
//     rows of the contraction. So the contraction runs over (key, parity of
//     d): 8 keys a step, and the rows of the tile are (head, parity): the
//     A operand is P where the parities agree and 0 elsewhere, which makes the
//     MMA's 16 rows useful with 8 heads. Lane (g, t) then holds head g and
//     d = 32 t .. 32 t + 31 of O.
//   * Two tokens: the 16 rows are (token, head), and the pairs of two keys are
//     turned round by two byte permutes.
//   * S leaves each lane two keys of a tile, and the same two are the keys of
//     its A and B fragments of PV: P needs no shuffle. Which two is chosen so
//     that the 8-byte loads of V (64-byte swizzle) meet different banks.
#pragma once

constexpr int kFp4Warps = 4;    // workers per CTA
constexpr int kFp4Stages = 2;   // units in flight per worker
struct Fp4Unit {
    uint8_t k[kK4Bytes];   // [64 keys][64 B]
    uint8_t v[kK4Bytes];   // [64 keys][64 B], 64-byte swizzle
    uint8_t ks[kS4Bytes];  // [64 keys][8]
    uint8_t vs[kS4Bytes];
};
static_assert(sizeof(Fp4Unit) % 1024 == 0, "swizzled tiles stay aligned");

struct DecodeSmem4 {
    Fp4Unit unit[kFp4Warps][kFp4Stages];
    StageDesc desc[kFp4Warps][kFp4Stages];
    uint64_t full[kFp4Warps][kFp4Stages];
};
constexpr size_t kDecodeSmem4Bytes = sizeof(DecodeSmem4) + 1024;

// The MMAs here are not volatile: the compiler may move them among the
// conversions of other tiles.
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The units [u, u1) of a worker, one after the other (uniform over the warp).
struct Fp4Walk {
    int64_t u, u1, u0;
    int64_t piece_end;
    int32_t s, g, p, npg, pf, lo, hi;
    int32_t batch, mine;  // table entries of pages 32 batch .. 32 batch + 31 of the sequence, one per lane
    int32_t flags, slot;
    int4 d, dn;

    __device__ Fp4Walk(const DecodeArgs &a, int64_t u0_, int64_t u1_) : u(u0_), u1(u1_), u0(u0_), piece_end(u0_) {
        s = 0, batch = -1, mine = -1;
        d = dn = make_int4(0, 0, 0, 0);
        if (u0 < u1) {
            s = find_seq(a.sdesc, a.n_seqs, u0);
            d = a.sdesc[s];
            dn = a.sdesc[s + 1];
        }
    }
    __device__ bool more() const { return u < u1; }

    // The next unit: its descriptor and page.
    __device__ int32_t next(const DecodeArgs &a, StageDesc &out) {
        int32_t first = 0;
        if (u == piece_end) {
            first = kFirst;
            while (u >= (int64_t)d.x + d.w) {  // next sequence with units
                ++s;
                d = dn;
                dn = a.sdesc[s + 1];
                batch = -1;
            }
            lo = d.y, hi = d.z;
            pf = lo / kP;
            npg = d.w / a.hkv;
            const int32_t at = (int32_t)(u - d.x);
            g = at / npg;
            p = at - g * npg;
            const int64_t seg_end = u - p + npg;
            piece_end = seg_end < u1 ? seg_end : u1;
            flags = p == 0 && piece_end == seg_end ? kDirect : 0;
            slot = u == u0 ? 0 : 1;
        }
        if ((p >> 5) != batch) {
            batch = p >> 5;
            const int32_t q = (p & ~31) + (threadIdx.x & 31);
            mine = q < npg && pf + q < a.bt_stride ? a.bt[(int64_t)s * a.bt_stride + pf + q] : -1;
        }
        const int32_t page = __shfl_sync(0xffffffffu, mine, p & 31);
        const int32_t key0 = (pf + p) * kP;
        const bool valid = page >= 0 && page < a.num_pages;
        out.seq = s;
        out.kvh = g;
        out.lo = lo - key0 > 0 ? lo - key0 : 0;
        out.hi = hi - key0 < kP ? hi - key0 : kP;
        out.slot = slot;
        out.key0 = key0;
        out.len = hi;
        out.flags = flags | first | (u + 1 == piece_end ? kLast : 0) | (valid ? 0 : kSkip);
        ++u;
        ++p;
        return valid ? page : -1;
    }
};

// One worker. kTok = 1 or 2 query tokens, from token a.tok0 of each sequence.
template <int kTok>
__device__ void decode_fp4_worker(DecodeSmem4 &sm, const CUtensorMap *tv, const DecodeArgs &a, int64_t u0, int64_t u1,
                                  int32_t worker) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int gr = lane >> 2, t = lane & 3;
    Fp4Walk walk(a, u0, u1);
    const uint8_t *kp = reinterpret_cast<const uint8_t *>(a.k_pool);
    const uint8_t *ksp = reinterpret_cast<const uint8_t *>(a.k_scale), *vsp = reinterpret_cast<const uint8_t *>(a.v_scale);
    const int64_t n = u1 - u0;
    int64_t issued = 0;
    const auto issue = [&] {
        const int st = (int)(issued % kFp4Stages);
        StageDesc d;
        const int32_t page = walk.next(a, d);
        if (lane == 0) {
            sm.desc[w][st] = d;
            uint64_t *full = &sm.full[w][st];
            if (page >= 0) {
                Fp4Unit &x = sm.unit[w][st];
                const int64_t blk = (int64_t)page * a.hkv + d.kvh;  // (page, kv head) block
                mbar_arrive_expect_tx(full, kUnit4Bytes);
                bulk_g2s(x.k, kp + blk * kK4Bytes, kK4Bytes, full);
                tma_load_2d(x.v, tv, 0, (int32_t)(blk * kP), full);
                bulk_g2s(x.ks, ksp + blk * kS4Bytes, kS4Bytes, full);
                bulk_g2s(x.vs, vsp + blk * kS4Bytes, kS4Bytes, full);
            } else {
                set_error(a.err, HSWA_ERR_BOUNDS);
                mbar_arrive(full);
            }
        }
        __syncwarp();
        ++issued;
    };
    while (issued < n && issued < kFp4Stages) issue();

    uint32_t qf[kTok][8][2];  // this lane's 32 d's of head gr as f16 pairs
    float o[2][8][4];         // kTok 1: o[0] only; else [parity of d][pair of d's]
    float m[kTok], l[kTok];   // this lane's head: reference (log2 units) and sum of P
#pragma unroll
    for (int j = 0; j < kTok; ++j) m[j] = -INFINITY, l[j] = 0.f;
    // the key of a tile in column gr of S; this lane's two keys of a tile are
    // 2 t + b and 2 t + 1 - b
    const int b = t & 1, krow = (gr & ~1) + ((gr ^ (gr >> 1)) & 1);

    for (int64_t i = 0; i < n; ++i) {
        const int st = (int)(i % kFp4Stages);
        const StageDesc d = sm.desc[w][st];
        if (d.flags & kFirst) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const int tok = a.tok0 + j;
                const uint4 *q = reinterpret_cast<const uint4 *>(
                    a.q + (q_row(a, d.seq, tok) * a.hq + (int64_t)d.kvh * kG + gr) * kD + 32 * t);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 f = bf16x8_to_f16x8(q[x]);
                    qf[j][2 * x][0] = f.x, qf[j][2 * x][1] = f.y, qf[j][2 * x + 1][0] = f.z, qf[j][2 * x + 1][1] = f.w;
                }
                m[j] = -INFINITY, l[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[0][j][e] = o[1][j][e] = 0.f;
        }
        bool ok = mbar_wait(&sm.full[w][st], (uint32_t)(i / kFp4Stages) & 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!(d.flags & kSkip)) {
            const Fp4Unit &x = sm.unit[w][st];
            float s[8][2 * kTok];  // [tile][token's two keys]
#pragma unroll
            for (int tile = 0; tile < 8; ++tile) {
                const int key = 8 * tile + krow;
                const uint4 c = *reinterpret_cast<const uint4 *>(x.k + key * 64 + t * 16);
                const uint32_t sc = *reinterpret_cast<const uint16_t *>(x.ks + key * 8 + 2 * t);
                const uint32_t s0 = scale_f16x2(sc & 0xff), s1 = scale_f16x2(sc >> 8);
                const uint32_t words[4] = {c.x, c.y, c.z, c.w};
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint32_t p0, p1, p2, p3;
                    e2m1x8_f16(words[y], p0, p1, p2, p3);
                    const uint32_t sy = y < 2 ? s0 : s1;
                    p0 = hmul2_bits(p0, sy), p1 = hmul2_bits(p1, sy), p2 = hmul2_bits(p2, sy), p3 = hmul2_bits(p3, sy);
                    if constexpr (kTok == 1) {
                        mma4(acc, qf[0][2 * y][0], 0u, qf[0][2 * y][1], 0u, p0, p1);
                        mma4(acc, qf[0][2 * y + 1][0], 0u, qf[0][2 * y + 1][1], 0u, p2, p3);
                    } else {
                        mma4(acc, qf[0][2 * y][0], qf[1][2 * y][0], qf[0][2 * y][1], qf[1][2 * y][1], p0, p1);
                        mma4(acc, qf[0][2 * y + 1][0], qf[1][2 * y + 1][0], qf[0][2 * y + 1][1], qf[1][2 * y + 1][1], p2, p3);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2 * kTok; ++e) s[tile][e] = acc[e] * a.scale_log2;
            }
            uint32_t pk[8][kTok];  // P of this lane's two keys of a tile, an f16 pair
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                int32_t lo = d.lo, hi = d.hi;  // one token: the stage's range is its own
                if (a.n_tok > 1) {
                    const int32_t at = d.len - a.n_tok + a.tok0 + j;
                    hi = min(d.hi, at - d.key0 + 1);
                    if (a.window > 0) lo = max(d.lo, at - a.window + 1 - d.key0);
                }
                if (lo > 0 || hi < kP) {
#pragma unroll
                    for (int tile = 0; tile < 8; ++tile)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = 8 * tile + 2 * t + (e ^ b);
                            if (key < lo || key >= hi) s[tile][2 * j + e] = -INFINITY;
                        }
                }
                float top = fmaxf(s[0][2 * j], s[0][2 * j + 1]);
#pragma unroll
                for (int tile = 1; tile < 8; ++tile) top = max3(top, s[tile][2 * j], s[tile][2 * j + 1]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // P carries 2^14, in the middle of f16's range, and so does its
                // sum: the reference is 14 below the largest score
                const float next = fmaxf(m[j], top - 14.f);
                const float ref = next == -INFINITY ? 0.f : next;
                if (__any_sync(0xffffffffu, next > m[j])) {
                    const float al = next == -INFINITY ? 1.f : fast_exp2(m[j] - next);
                    l[j] *= al;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        if constexpr (kTok == 1) {
                            o[0][y][0] *= al, o[0][y][1] *= al, o[0][y][2] *= al, o[0][y][3] *= al;
                        } else {
                            o[0][y][2 * j] *= al, o[0][y][2 * j + 1] *= al, o[1][y][2 * j] *= al, o[1][y][2 * j + 1] *= al;
                        }
                    }
                    m[j] = next;
                }
#pragma unroll
                for (int tile = 0; tile < 8; ++tile) {
                    const float p0 = fast_exp2(s[tile][2 * j] - ref), p1 = fast_exp2(s[tile][2 * j + 1] - ref);
                    l[j] += p0 + p1;
                    pk[tile][j] = pack_f16(p0, p1);
                }
            }
            // V of the lane's keys of a tile, block gr: 8 f16 pairs (d, d + 1) each
            const auto values = [&](int tile, int e, uint32_t (&v)[8]) {
                const int key = 8 * tile + 2 * t + (e ^ b);  // (key >> 1) & 3 is t
                const uint2 c = *reinterpret_cast<const uint2 *>(x.v + key * 64 + (((gr >> 1) ^ t) << 4) + (gr & 1) * 8);
                const uint32_t sv = scale_f16x2(x.vs[key * 8 + gr]);
                e2m1x8_f16(c.x, v[0], v[1], v[2], v[3]);
                e2m1x8_f16(c.y, v[4], v[5], v[6], v[7]);
#pragma unroll
                for (int y = 0; y < 8; ++y) v[y] = hmul2_bits(v[y], sv);
            };
            if constexpr (kTok == 1) {
#pragma unroll
                for (int tile = 0; tile < 8; ++tile) {
                    uint32_t v0[8], v1[8];
                    values(tile, 0, v0);
                    values(tile, 1, v1);
                    const uint32_t p = pk[tile][0];
#pragma unroll
                    for (int y = 0; y < 8; ++y) mma4(o[0][y], p & 0xffff, p << 16, p >> 16, p & 0xffff0000u, v0[y], v1[y]);
                }
            } else {
#pragma unroll
                for (int tile = 0; tile < 8; tile += 2) {
                    uint32_t v0[8], v1[8], v2[8], v3[8];
                    values(tile, 0, v0);
                    values(tile, 1, v1);
                    values(tile + 1, 0, v2);
                    values(tile + 1, 1, v3);
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        mma4(o[0][y], pk[tile][0], pk[tile][1], pk[tile + 1][0], pk[tile + 1][1],
                             __byte_perm(v0[y], v1[y], 0x5410), __byte_perm(v2[y], v3[y], 0x5410));
                        mma4(o[1][y], pk[tile][0], pk[tile][1], pk[tile + 1][0], pk[tile + 1][1],
                             __byte_perm(v0[y], v1[y], 0x7632), __byte_perm(v2[y], v3[y], 0x7632));
                    }
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (issued < n) issue();

        if (d.flags & kLast) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                float L = l[j];
                L += __shfl_xor_sync(0xffffffffu, L, 1);
                L += __shfl_xor_sync(0xffffffffu, L, 2);
                float f[32];  // d = 32 t .. 32 t + 31
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    if constexpr (kTok == 1) {
                        f[2 * y] = o[0][y][0], f[2 * y + 1] = o[0][y][2];
                        f[16 + 2 * y] = o[0][y][1], f[17 + 2 * y] = o[0][y][3];
                    } else {
                        f[2 * y] = o[0][y][2 * j], f[2 * y + 1] = o[1][y][2 * j];
                        f[16 + 2 * y] = o[0][y][2 * j + 1], f[17 + 2 * y] = o[1][y][2 * j + 1];
                    }
                }
                const int tok = a.tok0 + j;
                if (d.flags & kDirect) {
                    const float inv = L > 0.f ? 1.f / L : 0.f;
                    uint4 *out = reinterpret_cast<uint4 *>(a.o + (q_row(a, d.seq, tok) * a.hq + (int64_t)d.kvh * kG + gr) * kD + 32 * t);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        out[y] = make_uint4(pack_bf16(f[8 * y] * inv, f[8 * y + 1] * inv), pack_bf16(f[8 * y + 2] * inv, f[8 * y + 3] * inv),
                                            pack_bf16(f[8 * y + 4] * inv, f[8 * y + 5] * inv), pack_bf16(f[8 * y + 6] * inv, f[8 * y + 7] * inv));
                } else {
                    Partial &p = a.part[((int64_t)worker * 2 + d.slot) * a.n_tok + tok];
                    if (t == 0) p.m[gr] = m[j], p.l[gr] = L;
                    float4 *out = reinterpret_cast<float4 *>(p.o[gr] + 32 * t);
#pragma unroll
                    for (int y = 0; y < 8; ++y) out[y] = make_float4(f[4 * y], f[4 * y + 1], f[4 * y + 2], f[4 * y + 3]);
                }
            }
        }
    }
    // a wait gave up: never leave with copies still landing in shared memory
    // (stages that were waited for already return at once)
    if (lane == 0)
        for (int64_t i = issued > kFp4Stages ? issued - kFp4Stages : 0; i < issued; ++i)
            mbar_wait(&sm.full[w][i % kFp4Stages], (uint32_t)(i / kFp4Stages) & 1, a.err);
}

template <int kTok>
__global__ void __launch_bounds__(32 * kFp4Warps, 3) decode_mma_fp4_d128(const __grid_constant__ CUtensorMap tv, DecodeArgs a) {
    extern __shared__ uint8_t raw[];
    DecodeSmem4 &sm = *reinterpret_cast<DecodeSmem4 *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    if (threadIdx.x < kFp4Warps * kFp4Stages) mbar_init(&sm.full[0][0] + threadIdx.x, 1);
    fence_barrier_init();
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const int64_t U = a.sdesc[a.n_seqs].x, N = (int64_t)gridDim.x * kFp4Warps;
    if (U == 0) return;
    const int32_t worker = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
    const int64_t u0 = cta_start(worker, U, N), u1 = cta_start(worker + 1, U, N);
    decode_fp4_worker<kTok>(sm, &tv, a, u0, u1, worker);
}
