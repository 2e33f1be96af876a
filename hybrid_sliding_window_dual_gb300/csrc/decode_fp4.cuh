// Decode of 1 to 4 tokens over FP4 pools (d = 128, 8 query heads per kv head,
// page 64): part of decode.cu, whose plan, partial records and merge it shares.
//
// A page and kv head are 9 KB, 1.83 times less than in FP8, and the work to
// turn codes into MMA operands is the same, so that here the instructions of an
// element, not the loads, decide how near the kernel comes to the memory's rate:
// conversions, their products with scales, and the MMAs, which an SM's quarter
// issues one after the other (64 sequences of 1K to 32K tokens, one token each:
// 210 us, 0.9 of a plain copy's rate; two each 306; four each 555 to 564, where the
// MMAs alone are 240). Every choice below saves some; times are that first case's.
//   * A warp is a worker of its own. It takes an equal share of the units (a
//     page of a kv head), streams them through its own ring of kParts parts
//     and leaves its own partial records: no barriers between warps, no
//     producer. 12 workers on an SM are best; with 8 an exposed latency shows,
//     16 spill.
//   * Parts come by cp.async of all lanes, 16 bytes each, waited for by count
//     (an elected lane's bulk copies and a barrier per part: 247 us against
//     236). A unit's descriptor is made once, 8 units at a time, a lane each.
//   * Codes become f16 pairs by the conversion instruction, two at a time, and
//     are multiplied by their block's scale as pairs, which is exact (see
//     fp4.cuh).
//   * Both pools keep a token's codes in a row. S: lane (g, t) holds 32 d's of
//     one key per 8 keys (one 16-byte load, two scales); the contraction takes
//     d = 32 t + 4 s + 0..3 in step s from lane t, and Q's fragments follow.
//   * One token: keys are the 16 rows of S^T = K Q^T and d's those of
//     O^T += V^T P^T, with the 8 heads as columns: no row is idle (heads as
//     rows: 271 us against 238). S^T leaves a lane one key of two heads; the
//     transpose of an 8 x 8 tile of pairs gives it P^T's fragment.
//   * Two to four: (token, head) are the rows. S leaves each lane two keys of a
//     tile, and the same two are those of its fragments of PV: P needs no
//     shuffle. Q's fragments lie in shared memory.
//   * PV wants pairs of two keys where the pool has pairs of two d's: the codes
//     of two keys are paired before the conversion, four logic operations for
//     16 elements (253 us -> 247).
//   * Which keys of a tile a lane holds is chosen so that the 8-byte loads of V
//     (its 16-byte chunks turned round by the row) meet different banks.
#pragma once

// kTok query tokens per launch (1, 2 or 4), kKeys keys taken at once, kWarps
// workers per CTA, kParts parts in flight per worker, kCtas CTAs per SM.
template <int kTok_, int kKeys_, int kWarps_, int kParts_, int kCtas_>
struct Fp4Shape {
    static constexpr int kTok = kTok_, kKeys = kKeys_, kWarps = kWarps_, kParts = kParts_, kCtas = kCtas_;
    static constexpr int kSteps = kP / kKeys;      // of a unit
    static constexpr int kTiles = kKeys / 8;       // of 8 keys
    static constexpr int kPairs = (kTok + 1) / 2;  // tokens share the 16 rows of a tile two by two
};
using Fp4One = Fp4Shape<1, 64, 4, 4, 3>;
using Fp4Two = Fp4Shape<2, 64, 4, 4, 2>;
using Fp4Four = Fp4Shape<4, 32, 4, 6, 2>;
constexpr int kFp4Ahead = 8;          // units whose descriptors are made at once
constexpr int kFp4PlanSeqs = 32;      // sequences whose descriptors every CTA makes for itself

// K or V of kKeys keys.
template <int kKeys>
struct alignas(128) Fp4Part {
    static constexpr uint32_t kCodeBytes = kKeys * kD / 2, kScaleBytes = kKeys * kD / kFp4Block;
    uint8_t codes[kCodeBytes];    // [keys][64 B]; V with the 64-byte swizzle
    uint8_t scales[kScaleBytes];  // [keys][8]
};

struct Fp4Desc {
    int32_t row;    // first row of the page and kv head in the pool, -1: nothing to load
    int32_t range;  // keys of the page in the sequence's range: first | last + 1 << 8 | flags << 16
    int32_t seq;    // sequence | kv head << 16
    int32_t rel;    // the sequence's length from the page's first key on
};

template <class Shape>
struct DecodeSmem4 {
    Fp4Part<Shape::kKeys> part[Shape::kWarps][Shape::kParts];
    // Q's fragments, where registers do not hold them
    uint4 q[Shape::kTok > 1 ? Shape::kWarps : 1][Shape::kPairs][8][Shape::kTok > 1 ? 32 : 1];
    Fp4Desc desc[Shape::kWarps][2 * kFp4Ahead];
    int4 plan[kFp4PlanSeqs + 1];
};
template <class Shape>
constexpr size_t decode_smem4_bytes() { return sizeof(DecodeSmem4<Shape>) + 128; }

// The MMAs here are not volatile: the compiler may move them among the
// conversions of other tiles.
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes global -> shared, without a register between.
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Makes the descriptors of a worker's units [u0, u1), 8 at a time, a lane
// each. A unit's table entry is loaded when those before it are written down.
struct Fp4Units {
    const int4 *sdesc;
    int32_t u0, u1, base, s;  // the next 8 units are base ..; s: the sequence of an earlier one
    int32_t page;
    Fp4Desc x;

    __device__ __forceinline__ void fetch(const DecodeArgs &a) {
        const int lane = threadIdx.x & 31;
        const int32_t u = base + lane;
        int32_t mine = s;
        if (lane < kFp4Ahead && u < u1) {
            int4 d = sdesc[mine];
            while (u >= d.x + d.w) d = sdesc[++mine];
            const int32_t npg = d.w / a.hkv, pf = d.y / kP;
            const int32_t g = (u - d.x) / npg, p = u - d.x - g * npg;
            const int32_t seg = u - p;  // the segment's first unit
            const int32_t key0 = (pf + p) * kP;
            page = pf + p < a.bt_stride ? a.bt[(int64_t)mine * a.bt_stride + pf + p] : -1;
            const int32_t flags = (u == seg || u == u0 ? kFirst : 0) | (p == npg - 1 || u == u1 - 1 ? kLast : 0) |
                                  (seg >= u0 && seg + npg <= u1 ? kDirect : 0) | (seg > u0 ? kSecond : 0);
            x.range = max(d.y - key0, 0) | min(d.z - key0, kP) << 8 | flags << 16;
            x.seq = mine | g << 16;
            x.rel = d.z - key0;
        }
        s = __shfl_sync(0xffffffffu, mine, max(min(kFp4Ahead, u1 - base) - 1, 0));
    }
    __device__ __forceinline__ Fp4Units(const DecodeArgs &a, const int4 *sdesc_, int32_t u0_, int32_t u1_)
        : sdesc(sdesc_), u0(u0_), u1(u1_), base(u0_) {
        s = find_seq(sdesc, a.n_seqs, u0);
        fetch(a);
    }
    // Write the next 8 down.
    __device__ __forceinline__ void put(const DecodeArgs &a, Fp4Desc *desc) {
        const int lane = threadIdx.x & 31;
        if (lane < kFp4Ahead && base + lane < u1) {
            const bool valid = page >= 0 && page < a.num_pages;
            if (!valid) set_error(a.err, HSWA_ERR_BOUNDS);
            x.row = valid ? (page * a.hkv + (x.seq >> 16)) * kP : -1;
            if (!valid) x.range |= kSkip << 16;
            desc[(base - u0 + lane) % (2 * kFp4Ahead)] = x;
        }
        base += kFp4Ahead;
        fetch(a);
        __syncwarp();
    }
};

// 16 elements of o, over the sum of P.
__device__ __forceinline__ void fp4_store(__nv_bfloat16 *to, const float (&f)[16], float L) {
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int y = 0; y < 2; ++y)
        reinterpret_cast<uint4 *>(to)[y] =
            make_uint4(pack_bf16(f[8 * y] * inv, f[8 * y + 1] * inv), pack_bf16(f[8 * y + 2] * inv, f[8 * y + 3] * inv),
                       pack_bf16(f[8 * y + 4] * inv, f[8 * y + 5] * inv), pack_bf16(f[8 * y + 6] * inv, f[8 * y + 7] * inv));
}

// One worker.
template <class Shape>
__device__ void decode_fp4_worker(DecodeSmem4<Shape> &sm, const DecodeArgs &a, const int4 *sdesc, int32_t u0,
                                  int32_t u1, int32_t worker) {
    constexpr int kTok = Shape::kTok, kPairs = Shape::kPairs, kParts = Shape::kParts, kTiles = Shape::kTiles;
    constexpr int kSteps = Shape::kSteps, kKeys = Shape::kKeys;
    using Part = Fp4Part<kKeys>;
    if (u0 >= u1) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int gr = lane >> 2, t = lane & 3;
    // this lane's 16 bytes of a run of 8 rows of codes, in the pool and in a
    // part (V: its 16-byte chunks turned round by the row's bits 1 and 2), and of scales
    const uint8_t *const kp = reinterpret_cast<const uint8_t *>(a.k_pool) + lane * 16, *const vp = reinterpret_cast<const uint8_t *>(a.v_pool) + lane * 16;
    const uint8_t *const ksp = reinterpret_cast<const uint8_t *>(a.k_scale) + lane * 16, *const vsp = reinterpret_cast<const uint8_t *>(a.v_scale) + lane * 16;
    const uint32_t parts0 = smem_u32(sm.part[w]);
    const int32_t parts = 2 * kSteps * (u1 - u0);
    Fp4Units units(a, sdesc, u0, u1);
    Fp4Desc *const desc = sm.desc[w];
    int32_t described = 0;
    // Part c: K (c even) or V of step c / 2, into buffer st; a group of copies of its own.
    const auto issue = [&](int32_t c, int st, bool is_v) {
        const int32_t i = (c >> 1) / kSteps;
        if (c < parts) {
            if (i == described) {
                units.put(a, desc);
                described += kFp4Ahead;
            }
            const int32_t first = desc[i % (2 * kFp4Ahead)].row, row = first + (c >> 1) % kSteps * kKeys;
            if (first >= 0) {
                const uint8_t *from = (is_v ? vp : kp) + (int64_t)row * (kD / 2);
                const uint32_t to = parts0 + st * (uint32_t)sizeof(Part) + (is_v ? (lane & ~3) << 4 | ((lane ^ lane >> 3) & 3) << 4 : lane << 4);
#pragma unroll
                for (int x = 0; x < kTiles; ++x) copy16(to + x * 512, from + x * 512);
                if (kKeys == 64 || lane < kKeys / 2)
                    copy16(parts0 + st * (uint32_t)sizeof(Part) + Part::kCodeBytes + lane * 16, (is_v ? vsp : ksp) + (int64_t)row * (kD / kFp4Block));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    static_assert(kParts % 2 == 0, "K and V in turn");
#pragma unroll
    for (int st = 0; st < kParts; ++st) issue(st, st, st & 1);

    uint32_t qf[8][2];         // kTok 1: this lane's 32 d's of head gr as f16 pairs
    float o[kPairs][2][8][4];  // kTok 1: o[0][0] only; else [pair of tokens][parity of d][pair of d's]
    float m[kTok];             // this lane's head: reference (log2 units),
    float2 l[kTok];            // sums of P over its keys (two sums; kTok 1: of heads 2 t, 2 t + 1);
    float2 m2 = make_float2(-INFINITY, -INFINITY);  // kTok 1: references of heads 2 t, 2 t + 1
#pragma unroll
    for (int j = 0; j < kTok; ++j) m[j] = -INFINITY, l[j] = make_float2(0.f, 0.f);
    const float scale = a.scale_log2;  // above 0
    const uint32_t flip = a.q_flip;
    // the key of a tile in column gr of S; this lane's two keys of a tile are
    // 2 t + b and 2 t + 1 - b
    const int b = t & 1, krow = (gr & ~1) + ((gr ^ (gr >> 1)) & 1);

    int st = 0;
    // the part in buffer st is there once at most kParts - 1 younger ones are not
    const auto arrived = [&] {
        asm volatile("cp.async.wait_group %0;" ::"n"(kParts - 1) : "memory");
        __syncwarp();
    };
    // every lane has read the buffer: it is filled again, on to the next
    const auto release = [&](int32_t c, bool is_v) {
        __syncwarp();
        issue(c + kParts, st, is_v);
        if (++st == kParts) st = 0;
    };
    for (int32_t i = 0; i < parts / 2; ++i) {
        const Fp4Desc d = desc[i / kSteps % (2 * kFp4Ahead)];
        const int32_t from = i % kSteps * kKeys;  // the step's first key of the page
        const int32_t flags = (d.range >> 16) & (kSteps == 1 ? ~0 : i % kSteps == 0 ? ~kLast : i % kSteps == kSteps - 1 ? ~kFirst : ~(kFirst | kLast));
        if (flags & kFirst) {
            m2 = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const int tok = min(j, a.n_tok - 1);  // a row too many is computed and not stored
                const uint4 *q = reinterpret_cast<const uint4 *>(
                    a.q + (q_row(a, d.seq & 0xffff, tok) * a.hq + (int64_t)(d.seq >> 16) * kG + gr) * kD + 32 * t);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 f = bf16x8_to_f16x8(q[x], flip);
                    if constexpr (kTok > 1) {
                        // A operand: .x, .z the pair's first token, .y, .w its second
                        uint32_t *to = reinterpret_cast<uint32_t *>(&sm.q[w][j / 2][2 * x][lane]) + (j & 1);
                        to[0] = f.x, to[2] = f.y;
                        to += 32 * 4;
                        to[0] = f.z, to[2] = f.w;
                    } else {
                        qf[2 * x][0] = f.x, qf[2 * x][1] = f.y;
                        qf[2 * x + 1][0] = f.z, qf[2 * x + 1][1] = f.w;
                    }
                }
                m[j] = -INFINITY, l[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int pr = 0; pr < kPairs; ++pr)
#pragma unroll
                for (int y = 0; y < 8; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[pr][0][y][e] = o[pr][1][y][e] = 0.f;
        }
        arrived();
        uint32_t pk[kTok][kTiles];  // P of this lane's two keys of a tile, an f16 pair
        if (!(flags & kSkip)) {
            const Part &x = sm.part[w][st];
            if constexpr (kTok == 1) {
                float s[kTiles / 2][4];  // keys of two tiles as rows: heads 2 t, 2 t + 1 of one key, of the other
                constexpr int kGroup = 2;
#pragma unroll
                for (int r0 = 0; r0 < kTiles / 2; r0 += kGroup) {
                    uint4 c[2 * kGroup];
                    uint32_t sc[2 * kGroup];
#pragma unroll
                    for (int z = 0; z < 2 * kGroup; ++z) {
                        const int key = 8 * (2 * r0 + z) + krow;
                        c[z] = *reinterpret_cast<const uint4 *>(x.codes + key * 64 + t * 16);
                        sc[z] = *reinterpret_cast<const uint16_t *>(x.scales + key * 8 + 2 * t);
                    }
#pragma unroll
                    for (int z = 0; z < kGroup; ++z) s[r0 + z][0] = s[r0 + z][1] = s[r0 + z][2] = s[r0 + z][3] = 0.f;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int z = 0; z < kGroup; ++z) {
                            uint32_t k[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 &cz = c[2 * z + h];
                                const uint32_t sy = scale_f16x2(y < 2 ? sc[2 * z + h] & 0xff : sc[2 * z + h] >> 8);
                                e2m1x8_f16(y == 0 ? cz.x : y == 1 ? cz.y : y == 2 ? cz.z : cz.w, k[h][0], k[h][1], k[h][2], k[h][3]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) k[h][e] = hmul2_bits(k[h][e], sy);
                            }
                            mma4(s[r0 + z], k[0][0], k[1][0], k[0][1], k[1][1], qf[2 * y][0], qf[2 * y][1]);
                            mma4(s[r0 + z], k[0][2], k[1][2], k[0][3], k[1][3], qf[2 * y + 1][0], qf[2 * y + 1][1]);
                        }
                }
                const int32_t lo = (d.range & 0xff) - from, hi = (d.range >> 8 & 0xff) - from;
                if (lo > 0 || hi < kKeys) {
#pragma unroll
                    for (int z = 0; z < kTiles; ++z) {
                        const int key = 8 * z + krow;
                        if (key < lo || key >= hi) s[z / 2][2 * (z & 1)] = s[z / 2][2 * (z & 1) + 1] = -INFINITY;
                    }
                }
                float top0 = fmaxf(s[0][0], s[0][2]), top1 = fmaxf(s[0][1], s[0][3]);
#pragma unroll
                for (int z = 1; z < kTiles / 2; ++z) top0 = max3(top0, s[z][0], s[z][2]), top1 = max3(top1, s[z][1], s[z][3]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, off));
                    top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, off));
                }
                // P carries 2^14, in the middle of f16's range, and so does its
                // sum: the reference is 14 below the largest score
                const float n0 = fmaxf(m2.x, fmaf(top0, scale, -14.f)), n1 = fmaxf(m2.y, fmaf(top1, scale, -14.f));
                if (__any_sync(0xffffffffu, n0 > m2.x || n1 > m2.y)) {
                    const float al0 = n0 == -INFINITY ? 1.f : fast_exp2(m2.x - n0), al1 = n1 == -INFINITY ? 1.f : fast_exp2(m2.y - n1);
                    l[0].x *= al0, l[0].y *= al1;
#pragma unroll
                    for (int y = 0; y < 8; ++y) o[0][0][y][0] *= al0, o[0][0][y][1] *= al1, o[0][0][y][2] *= al0, o[0][0][y][3] *= al1;
                    m2 = make_float2(n0, n1);
                }
                const float2 scale2 = make_float2(scale, scale);
                const float2 ref2 = make_float2(n0 == -INFINITY ? 0.f : -n0, n1 == -INFINITY ? 0.f : -n1);
#pragma unroll
                for (int z = 0; z < kTiles; ++z) {
                    const float2 y = __ffma2_rn(make_float2(s[z / 2][2 * (z & 1)], s[z / 2][2 * (z & 1) + 1]), scale2, ref2);
                    const float2 pp = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    l[0] = __fadd2_rn(l[0], pp);
                    pk[0][z] = movmatrix_t(pack_f16(pp.x, pp.y));  // head gr, keys of columns 2 t, 2 t + 1
                }
            } else {
                float s[kPairs][kTiles][4];  // rows: the pair's first token (two keys), its second
                constexpr int kGroup = 4;       // tiles whose MMAs go side by side
#pragma unroll
                for (int t0 = 0; t0 < kTiles; t0 += kGroup) {
                    uint4 c[kGroup];
                    uint32_t sc[kGroup];
#pragma unroll
                    for (int z = 0; z < kGroup; ++z) {
                        const int key = 8 * (t0 + z) + krow;
                        c[z] = *reinterpret_cast<const uint4 *>(x.codes + key * 64 + t * 16);
                        sc[z] = *reinterpret_cast<const uint16_t *>(x.scales + key * 8 + 2 * t);
#pragma unroll
                        for (int pr = 0; pr < kPairs; ++pr) s[pr][t0 + z][0] = s[pr][t0 + z][1] = s[pr][t0 + z][2] = s[pr][t0 + z][3] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint4 qa[kPairs][2];  // steps 2 y and 2 y + 1
#pragma unroll
                        for (int pr = 0; pr < kPairs; ++pr)
#pragma unroll
                            for (int h = 0; h < 2; ++h) qa[pr][h] = sm.q[w][pr][2 * y + h][lane];
#pragma unroll
                        for (int z = 0; z < kGroup; ++z) {
                            const uint32_t word = y == 0 ? c[z].x : y == 1 ? c[z].y : y == 2 ? c[z].z : c[z].w;
                            const uint32_t sy = scale_f16x2(y < 2 ? sc[z] & 0xff : sc[z] >> 8);
                            uint32_t p0, p1, p2, p3;
                            e2m1x8_f16(word, p0, p1, p2, p3);
                            p0 = hmul2_bits(p0, sy), p1 = hmul2_bits(p1, sy), p2 = hmul2_bits(p2, sy), p3 = hmul2_bits(p3, sy);
#pragma unroll
                            for (int pr = 0; pr < kPairs; ++pr) {
                                mma4(s[pr][t0 + z], qa[pr][0].x, qa[pr][0].y, qa[pr][0].z, qa[pr][0].w, p0, p1);
                                mma4(s[pr][t0 + z], qa[pr][1].x, qa[pr][1].y, qa[pr][1].z, qa[pr][1].w, p2, p3);
                            }
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    float(&sj)[kTiles][4] = s[j / 2];
                    const int e0 = 2 * (j & 1);
                    int32_t lo = (d.range & 0xff) - from, hi = (d.range >> 8 & 0xff) - from;
                    const int32_t at = d.rel - a.n_tok + j - from;  // its position
                    hi = min(hi, at + 1);
                    if (a.window > 0) lo = max(lo, at - a.window + 1);
                    if (lo > 0 || hi < kKeys) {
#pragma unroll
                        for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = 8 * tile + 2 * t + (e ^ b);
                                if (key < lo || key >= hi) sj[tile][e0 + e] = -INFINITY;
                            }
                    }
                    float top = fmaxf(sj[0][e0], sj[0][e0 + 1]);
#pragma unroll
                    for (int tile = 1; tile < kTiles; ++tile) top = max3(top, sj[tile][e0], sj[tile][e0 + 1]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // P carries 2^14, in the middle of f16's range, and so does its
                    // sum: the reference is 14 below the largest score
                    const float next = fmaxf(m[j], fmaf(top, scale, -14.f));
                    if (__any_sync(0xffffffffu, next > m[j])) {
                        const float al = next == -INFINITY ? 1.f : fast_exp2(m[j] - next);
                        l[j].x *= al, l[j].y *= al;
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            float(&oj)[2][8][4] = o[j / 2];
                            oj[0][y][e0] *= al, oj[0][y][e0 + 1] *= al, oj[1][y][e0] *= al, oj[1][y][e0 + 1] *= al;
                        }
                        m[j] = next;
                    }
                    const float ref = next == -INFINITY ? 0.f : -next;
                    const float2 scale2 = make_float2(scale, scale), ref2 = make_float2(ref, ref);
#pragma unroll
                    for (int tile = 0; tile < kTiles; ++tile) {
                        const float2 y = __ffma2_rn(make_float2(sj[tile][e0], sj[tile][e0 + 1]), scale2, ref2);
                        const float2 pp = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                        l[j] = __fadd2_rn(l[j], pp);
                        pk[j][tile] = pack_f16(pp.x, pp.y);
                    }
                }
            }
        }
        release(2 * i, false);
        arrived();
        if (!(flags & kSkip)) {
            const Part &x = sm.part[w][st];
            // V of the lane's two keys of a tile, block gr: f16 pairs of both
            // keys' even d's (ve) and odd d's (vo). The codes are paired before they
            // are converted, a byte taking one code of each key.
            const uint8_t *const at0 = x.codes + (2 * t + b) * 64 + (((gr >> 1) ^ t) << 4) + (gr & 1) * 8;  // (key >> 1) & 3 is t
            const uint8_t *const at1 = at0 + (b ? -64 : 64);
            const uint8_t *const sc0 = x.scales + (2 * t + b) * 8 + gr, *const sc1 = sc0 + (b ? -8 : 8);
            const auto values = [&](int tile, uint32_t (&ve)[8], uint32_t (&vo)[8]) {
                const uint2 c0 = *reinterpret_cast<const uint2 *>(at0 + tile * 512), c1 = *reinterpret_cast<const uint2 *>(at1 + tile * 512);
                const uint32_t sv = (uint32_t)sc0[tile * 64] << 7 | (uint32_t)sc1[tile * 64] << 23;
                constexpr uint32_t kLow = 0x0f0f0f0f;
                e2m1x8_f16((c0.x & kLow) | (c1.x << 4 & ~kLow), ve[0], ve[1], ve[2], ve[3]);
                e2m1x8_f16((c0.y & kLow) | (c1.y << 4 & ~kLow), ve[4], ve[5], ve[6], ve[7]);
                e2m1x8_f16((c0.x >> 4 & kLow) | (c1.x & ~kLow), vo[0], vo[1], vo[2], vo[3]);
                e2m1x8_f16((c0.y >> 4 & kLow) | (c1.y & ~kLow), vo[4], vo[5], vo[6], vo[7]);
#pragma unroll
                for (int y = 0; y < 8; ++y) ve[y] = hmul2_bits(ve[y], sv), vo[y] = hmul2_bits(vo[y], sv);
            };
#pragma unroll
            for (int tile = 0; tile < kTiles; tile += 2) {
                uint32_t a0[8], a1[8], a2[8], a3[8];
                values(tile, a0, a1);
                values(tile + 1, a2, a3);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    if constexpr (kTok == 1) {
                        mma4(o[0][0][y], a0[y], a1[y], a2[y], a3[y], pk[0][tile], pk[0][tile + 1]);
                    } else {
#pragma unroll
                        for (int pr = 0; pr < kPairs; ++pr) {
                            mma4(o[pr][0][y], pk[2 * pr][tile], pk[2 * pr + 1][tile], pk[2 * pr][tile + 1], pk[2 * pr + 1][tile + 1], a0[y], a2[y]);
                            mma4(o[pr][1][y], pk[2 * pr][tile], pk[2 * pr + 1][tile], pk[2 * pr][tile + 1], pk[2 * pr + 1][tile + 1], a1[y], a3[y]);
                        }
                    }
                }
            }
        }
        release(2 * i + 1, true);

        if (flags & kLast) {
            if constexpr (kTok == 1) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[0].x += __shfl_xor_sync(0xffffffffu, l[0].x, off);
                    l[0].y += __shfl_xor_sync(0xffffffffu, l[0].y, off);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // head 2 t + e, d = 16 gr .. 16 gr + 15
                    const int h = 2 * t + e;
                    const float L = e ? l[0].y : l[0].x;
                    float f[16];
#pragma unroll
                    for (int y = 0; y < 8; ++y) f[2 * y] = o[0][0][y][e], f[2 * y + 1] = o[0][0][y][2 + e];
                    if (flags & kDirect) {
                        fp4_store(a.o + ((int64_t)(d.seq & 0xffff) * a.hq + (int64_t)(d.seq >> 16) * kG + h) * kD + 16 * gr, f, L);
                    } else {
                        Partial &p = a.part[(int64_t)worker * 2 + (flags & kSecond ? 1 : 0)];
                        if (gr == 0) p.m[h] = e ? m2.y : m2.x, p.l[h] = L;
                        float4 *out = reinterpret_cast<float4 *>(p.o[h] + 16 * gr);
#pragma unroll
                        for (int y = 0; y < 4; ++y) out[y] = make_float4(f[4 * y], f[4 * y + 1], f[4 * y + 2], f[4 * y + 3]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    if (j >= a.n_tok) break;
                    float L = l[j].x + l[j].y;
                    L += __shfl_xor_sync(0xffffffffu, L, 1);
                    L += __shfl_xor_sync(0xffffffffu, L, 2);
                    float(&oj)[2][8][4] = o[j / 2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {  // head gr, d = 32 t + 16 c ..
                        float f[16];
#pragma unroll
                        for (int y = 0; y < 8; ++y) f[2 * y] = oj[0][y][2 * (j & 1) + c], f[2 * y + 1] = oj[1][y][2 * (j & 1) + c];
                        if (flags & kDirect) {
                            fp4_store(a.o + (q_row(a, d.seq & 0xffff, j) * a.hq + (int64_t)(d.seq >> 16) * kG + gr) * kD + 32 * t + 16 * c, f, L);
                        } else {
                            Partial &p = a.part[((int64_t)worker * 2 + (flags & kSecond ? 1 : 0)) * a.n_tok + j];
                            if (t == 0 && c == 0) p.m[gr] = m[j], p.l[gr] = L;
                            float4 *out = reinterpret_cast<float4 *>(p.o[gr] + 32 * t + 16 * c);
#pragma unroll
                            for (int y = 0; y < 4; ++y) out[y] = make_float4(f[4 * y], f[4 * y + 1], f[4 * y + 2], f[4 * y + 3]);
                        }
                    }
                }
            }
        }
    }
}

// decode_plan by one warp, for at most kFp4PlanSeqs sequences: descriptors into
// plan, and from the first CTA into the workspace, for the merge.
__device__ __forceinline__ void fp4_plan(const DecodeArgs &a, int4 *plan) {
    const int lane = threadIdx.x & 31;
    int32_t u = 0, lo = 0, hi = 0;
    if (lane < a.n_seqs) key_range(a.seq_len[lane], a.window, a.n_tok, lo, hi);
    if (hi > lo) u = a.hkv * ((hi - 1) / kP - lo / kP + 1);
    int32_t x = u;
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    const int32_t all = __shfl_sync(0xffffffffu, x, 31);
    for (int4 *out : {plan, blockIdx.x == 0 ? const_cast<int4 *>(a.sdesc) : nullptr}) {
        if (!out) continue;
        if (lane < a.n_seqs) out[lane] = make_int4(x - u, lo, hi, u);
        if (lane == 0) out[a.n_seqs] = make_int4(all, 0, 0, 0);
    }
}
static_assert(kFp4PlanSeqs <= 32, "a lane each");

// kPlan: without decode_plan before it, one launch less (3 sequences of 700 to
// 2500 tokens 12.5 us against 13.3). With 64 sequences it was 1 us slower, and with
// Fp4Four's registers 10.
template <class Shape>
bool fp4_plans(int n_seqs) { return Shape::kTok <= 2 && n_seqs <= kFp4PlanSeqs; }
template <class Shape, bool kPlan>
__global__ void __launch_bounds__(32 * Shape::kWarps, Shape::kCtas) decode_mma_fp4_d128(const __grid_constant__ DecodeArgs a) {
    extern __shared__ uint8_t raw[];
    using Smem = DecodeSmem4<Shape>;
    static_assert(Shape::kCtas * (decode_smem4_bytes<Shape>() + 1024) <= 228 << 10, "kCtas CTAs on an SM");
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (kPlan) {
        if (threadIdx.x < 32) fp4_plan(a, sm.plan);
        __syncthreads();
    }
    const int4 *const sdesc = kPlan ? sm.plan : a.sdesc;
    const int64_t U = sdesc[a.n_seqs].x, N = (int64_t)gridDim.x * Shape::kWarps;
    const int32_t worker = blockIdx.x * Shape::kWarps + (threadIdx.x >> 5);
    decode_fp4_worker<Shape>(sm, a, sdesc, (int32_t)cta_start(worker, U, N), (int32_t)cta_start(worker + 1, U, N), worker);
}

// Other shapes (any head size in blocks, head ratio and page): a cluster per
// query row, kv head and up to four of its query heads, whose warps take tiles of
// 32 keys in turn. Scores: a lane has a key, q comes from shared memory; a block's
// sum of q times codes is multiplied by its scale. Output: a lane has bytes of
// the row, pairs of elements. All in fp32. Bound by a few dependent steps where there
// are few keys, by instructions otherwise (each element of K and V is converted for
// four heads). d = 64, 4 heads on one: 16 sequences of 1000 to 2000 tokens 17 us (one
// CTA a row 41, a warp a row and head 2440); d = 128, 32 heads on 8: 64 of 1K to 8K
// 604 (with registers for one CTA an SM 866; a warp a row and head 16900), one of
// 30000 135. 8 warps a CTA: 14, 1022 and 214.
struct Fp4AnyArgs {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    const uint8_t *k, *v, *ks, *vs;
    const int32_t *bt, *seq_len;
    int32_t n_tok, bt_stride, hq, hkv, d, page, window, num_pages, cluster;
    float scale_log2;
    int *err;
};

constexpr int kFp4AnyHeads = 4, kFp4AnyWarps = 16, kFp4AnyMaxD = 256, kFp4AnyCluster = 8;

// kE: bytes of a row that a lane has.
template <int kE>
__global__ void __launch_bounds__(32 * kFp4AnyWarps, kE <= 2 ? 2 : 1) decode_fp4_any(const Fp4AnyArgs a) {
    constexpr int kH = kFp4AnyHeads, kW = kFp4AnyWarps;
    __shared__ __align__(16) float q[kH][kFp4AnyMaxD];  // then the CTA's output
    __shared__ __align__(16) float4 ps[kW][32];   // P of the four heads
    __shared__ int64_t rows[kW][32];              // rows of V
    __shared__ float2 ml[kW][kH];                 // a warp's reference and sum
    __shared__ float2 cta_ml[kH];                 // those of the CTA
    __shared__ __align__(16) float sum[kH][2 * 32 * kE][4];  // four warps' outputs
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int32_t group = a.hq / a.hkv, chunks = (group + kH - 1) / kH;
    const int32_t rank = blockIdx.x % a.cluster;
    const int64_t row = blockIdx.x / a.cluster;  // sequence n_tok + query token
    const int32_t s = (int32_t)(row / a.n_tok), g = blockIdx.y / chunks, h0 = blockIdx.y % chunks * kH;
    const int32_t heads = min(kH, group - h0);
    const int64_t head0 = row * a.hq + g * group + h0;  // first of the CTA's in q and o
    const int32_t t = a.seq_len[s] - a.n_tok + (int32_t)(row - (int64_t)s * a.n_tok);
    const int32_t hi = t + 1, lo = a.window > 0 ? max(0, hi - a.window) : 0;
    for (int i = threadIdx.x; i < kH * a.d; i += 32 * kW) {
        const int h = i / a.d, c = i - h * a.d;
        q[h][c] = h < heads ? __bfloat162float(a.q[(head0 + h) * a.d + c]) * a.scale_log2 : 0.f;
    }
    __syncthreads();
    float m[kH], l[kH], acc[kH][kE][2];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[h][e][0] = acc[h][e][1] = 0.f;
    }
    const int32_t bytes = a.d / 2, blocks = a.d / kFp4Block;
    // positions past the table's last page are reported and left out (a length may be any int32)
    const int32_t end = (int32_t)min((int64_t)hi, (int64_t)a.bt_stride * a.page);
    if (hi > end && threadIdx.x == 0) set_error(a.err, HSWA_ERR_BOUNDS);
    for (int64_t at = lo + 32 * (int64_t)(rank * kW + w); at < end; at += 32 * kW * a.cluster) {
        int64_t key = -1;
        if (at + lane < end) {
            const int32_t j = (int32_t)at + lane, lp = j / a.page, pg = a.bt[(int64_t)s * a.bt_stride + lp];
            if (pg >= 0 && pg < a.num_pages)
                key = ((int64_t)pg * a.hkv + g) * a.page + (j - lp * a.page);
            else
                set_error(a.err, HSWA_ERR_BOUNDS);
        }
        float x[kH] = {};
        if (key >= 0) {
            const uint2 *codes = reinterpret_cast<const uint2 *>(a.k + key * bytes);
            const uint8_t *scales = a.ks + key * blocks;
#pragma unroll 4
            for (int32_t b = 0; b < blocks; ++b) {
                const uint2 c = codes[b];
                const float scale = scale_value(scales[b]);
                uint32_t p[8];
                e2m1x8_f16(c.x, p[0], p[1], p[2], p[3]);
                e2m1x8_f16(c.y, p[4], p[5], p[6], p[7]);
                float part[kH] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&p[2 * i])), v = __half22float2(*reinterpret_cast<const __half2 *>(&p[2 * i + 1]));
#pragma unroll
                    for (int h = 0; h < kH; ++h) {
                        const float4 y = *reinterpret_cast<const float4 *>(&q[h][16 * b + 4 * i]);
                        part[h] = fmaf(y.w, v.y, fmaf(y.z, v.x, fmaf(y.y, u.y, fmaf(y.x, u.x, part[h]))));
                    }
                }
#pragma unroll
                for (int h = 0; h < kH; ++h) x[h] = fmaf(part[h], scale, x[h]);
            }
        }
        float p[kH];
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            if (key < 0) x[h] = -INFINITY;
            float top = x[h];
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float next = fmaxf(m[h], top);
            const float alpha = next == -INFINITY ? 1.f : fast_exp2(m[h] - next);
            p[h] = x[h] == -INFINITY ? 0.f : fast_exp2(x[h] - (next == -INFINITY ? 0.f : next));  // a NaN stays one
            l[h] = l[h] * alpha + p[h];
            m[h] = next;
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[h][e][0] *= alpha, acc[h][e][1] *= alpha;
        }
        ps[w][lane] = make_float4(p[0], p[1], p[2], p[3]);
        rows[w][lane] = key < 0 ? 0 : key;  // a row that P takes 0 times
        __syncwarp();
        const int32_t n = (int32_t)min((int64_t)32, end - at);
#pragma unroll 8
        for (int32_t i = 0; i < n; ++i) {
            const float4 pi = ps[w][i];
            const int64_t r = rows[w][i];
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const int32_t c = lane + 32 * e;
                if (c >= bytes) continue;
                const float scale = scale_value(a.vs[r * blocks + c / 8]);
                uint32_t f;
                asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(f) : "r"((uint32_t)a.v[r * bytes + c]));
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
                const float v0 = v.x * scale, v1 = v.y * scale;
                acc[0][e][0] = fmaf(pi.x, v0, acc[0][e][0]), acc[0][e][1] = fmaf(pi.x, v1, acc[0][e][1]);
                acc[1][e][0] = fmaf(pi.y, v0, acc[1][e][0]), acc[1][e][1] = fmaf(pi.y, v1, acc[1][e][1]);
                acc[2][e][0] = fmaf(pi.z, v0, acc[2][e][0]), acc[2][e][1] = fmaf(pi.z, v1, acc[2][e][1]);
                acc[3][e][0] = fmaf(pi.w, v0, acc[3][e][0]), acc[3][e][1] = fmaf(pi.w, v1, acc[3][e][1]);
            }
        }
        __syncwarp();
    }
    // the warps' outputs relative to the CTA's largest reference, four warps at a time
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        for (int off = 16; off > 0; off >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
        if (lane == 0) ml[w][h] = make_float2(m[h], l[h]);
    }
    __syncthreads();
    float f[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        const float2 x = ml[lane % kW][h];
        float top = x.x;
        for (int off = kW / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float L = x.y * (x.x > -INFINITY ? fast_exp2(x.x - top) : 0.f);
        for (int off = kW / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        f[h] = m[h] > -INFINITY ? fast_exp2(m[h] - top) : 0.f;
        if (threadIdx.x == 0) cta_ml[h] = make_float2(top, L);
    }
    for (int from = 0; from < kW; from += 4) {
        if (w >= from && w < from + 4) {
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int e = 0; e < kE; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &to = sum[h][2 * (lane + 32 * e) + i][w - from];
                        to = (from ? to : 0.f) + acc[h][e][i] * f[h];
                    }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < heads * a.d; i += 32 * kW) {
        const int h = i / a.d, c = i - h * a.d;
        const float4 x = *reinterpret_cast<const float4 *>(sum[h][c]);
        q[h][c] = (x.x + x.y) + (x.z + x.w);
    }
    // and the CTAs', each of them joining a share of the elements
    cluster_arrive();
    cluster_wait();
    for (int i = rank * 32 * kW + threadIdx.x; i < heads * a.d; i += a.cluster * 32 * kW) {
        const int h = i / a.d, c = i - h * a.d;
        float ref[kFp4AnyCluster], part_l[kFp4AnyCluster], part[kFp4AnyCluster];
#pragma unroll
        for (int r = 0; r < kFp4AnyCluster; ++r) {
            const int from = min(r, a.cluster - 1);  // all loads at once, some for nothing
            ref[r] = ld_cluster_f32(&cta_ml[h].x, from);
            part_l[r] = ld_cluster_f32(&cta_ml[h].y, from);
            part[r] = ld_cluster_f32(&q[h][c], from);
        }
        float top = -INFINITY, L = 0.f, x = 0.f;
#pragma unroll
        for (int r = 0; r < kFp4AnyCluster; ++r) top = fmaxf(top, ref[r]);
#pragma unroll
        for (int r = 0; r < kFp4AnyCluster; ++r) {
            const float weight = r < a.cluster && ref[r] > -INFINITY ? fast_exp2(ref[r] - top) : 0.f;
            L = fmaf(weight, part_l[r], L);
            x = fmaf(weight, part[r], x);
        }
        a.o[(head0 + h) * a.d + c] = __float2bfloat16_rn(L == 0.f ? 0.f : x / L);
    }
    cluster_arrive();
    cluster_wait();  // nobody leaves while its results are read
}
