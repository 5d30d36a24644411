// cache_attn.cu -- attention of a few query tokens of each sequence over the paged 8-bit cache
// (dr.h, dr_cache_attn): one pass over the codes with running softmax statistics.
//
// The rows of a sequence and cache head are its query tokens times the G query heads that share
// the cache head, row = t * G + g.  A block works on a tile of 8 NT rows of one (sequence, cache
// head) over a stretch of its positions, in stages of 128; warp w takes positions 32 w .. 32 w + 31
// of each stage on its own, through a ring in shared memory that it fills with asynchronous copies
// a stage ahead, so that warps never wait for one another before the rows are joined.
//
// Matrix products (m16n8k16, 16-bit operands, fp32 accumulation), with 16 positions as rows:
//   S^T = K Q^T    A = K codes (16 positions x d), B = Q^T (d x 8 rows)
//   O^T += V^T P^T A = V^T codes (16 channels x 16 positions), B = P^T (16 positions x 8 rows)
// Which channels a thread supplies is free as long as both operands agree, so every thread loads
// 16 consecutive bytes at a time, and a code is exact in 16 bits.  16-byte chunk j of row r sits at
// chunk j ^ swizzle(r) of the row in the ring, which spreads the reads of both products over the banks.
//
// Softmax in base 2.  The page scales enter in fp32: the key scale multiplies S, the value scale
// vs multiplies the weights.  Both references are whole numbers, so that every rescaling is exact:
//   m >= max s, weights p = 2^(s - m), l = sum p;
//   M >= max (s + log2 vs), w = p vs 2^(m - M + 14) <= 2^14 is the 16-bit operand.
// Where vs 2^(m - M + 14) passes 2^100 w is taken as one power of two, 2^(s - M + 14 + log2 vs): the test for it takes
// 1 us of 58 (64 ragged sequences of 17 to 8191 positions), in a branch for each of the two rows 2 us.
// With PREC (fp32 queries or outputs) queries and weights are split into two 16-bit terms.
//
// Work is divided evenly: the stages of all tiles, each tile with a few more for its start and end,
// form one line, block i of n takes the i-th part of it.  A tile that lies in one block is finished
// there; of the others each block leaves its rows (sums, l, m, M) in the workspace, and a second
// kernel joins them, a block or a warp to a row.  It is launched early and waits on the device for the first.
//
// Bound by HBM where the cache is long: two sequences of 200001 to 262143 positions, four cache heads of 128,
// 84.5 us for 474 MB (82 % of the copy rate, join and launches within it); 64 ragged sequences of 17 to 8191
// positions 58 us for 270 MB (69 %: a tile's start and end cost as much as four stages).
#include "attn_util.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStep = 32, kStage = kStep * kWarps;  // positions of a warp's step, of a stage
constexpr int kOver = 4;  // what a tile costs beside its stages, in stages (64 ragged sequences: 57.6 us; 61.1 with 2, 59.0 with 6)

// ------------------------------------------------------------------ the line of stages
// Stages of sequence b that its tokens see, tiles of rows, and their product with the heads.
struct Seq {
    int len, n;         // positions before the call's tokens, tokens (0: nothing to do)
    int s0, stages;     // first stage, stages
    int tiles;          // tiles of rows
};
template <int ROWS>
__device__ __forceinline__ Seq make_seq(const AttnParams& p, int b) {
    Seq s;
    if (!cache_seq(p.c, b, s.len, s.n)) s.n = 0;
    s.s0 = s.stages = s.tiles = 0;
    if (s.n > 0) {
        const int lo = p.window > 0 ? max(0, s.len - p.window + 1) : 0;
        s.s0 = lo / kStage;
        s.stages = (s.len + s.n + kStage - 1) / kStage - s.s0;
        s.tiles = (s.n * p.G + ROWS - 1) / ROWS;
    }
    return s;
}
__device__ __forceinline__ long long work_of(const AttnParams& p, const Seq& s) {
    return s.n > 0 ? (long long)s.tiles * (s.stages + kOver) * p.c.H : 0;
}
// The whole line (every lane gets it).
template <int ROWS>
__device__ __forceinline__ long long line_length(const AttnParams& p, int lane) {
    long long total = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        if (b0 + lane < p.c.B) total += work_of(p, make_seq<ROWS>(p, b0 + lane));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
}
// The sequence that holds place `at` of the line, and where its own stretch begins.
template <int ROWS>
__device__ __forceinline__ int find_seq(const AttnParams& p, int lane, long long at, long long& begin) {
    long long before = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const long long x = b0 + lane < p.c.B ? work_of(p, make_seq<ROWS>(p, b0 + lane)) : 0;
        const long long upto = before + warp_scan(x, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, upto > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            begin = __shfl_sync(0xffffffffu, upto - x, l);
            return b0 + l;
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    begin = before;
    return p.c.B;
}
// ------------------------------------------------------------------ operands
// Bytes 0, 1 (HI: 2, 3) of the words of two positions, so that codes_to_half pairs the positions.
template <bool E4M3, bool HI> __device__ __forceinline__ uint32_t pair_up(uint32_t x, uint32_t y) {
    return __byte_perm(x, y, E4M3 ? (HI ? 0x7362 : 0x5140) : (HI ? 0x7632 : 0x5410));
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 16 positions in the ring.  Thread (g, c) = (lane / 4, lane % 4) takes of the keys positions g and
// g + 8, 16-byte chunks c d/64 .. + d/64 - 1 of the row; of the values positions 2c, 2c + 1, 2c + 8,
// 2c + 9, channels g d/8 .. + d/8 - 1.
template <int D> __device__ __forceinline__ int swizzle(int row) { return D == 128 ? row & 7 : (row >> 1) & 3; }
template <int D>
__device__ __forceinline__ void copy_codes(uint32_t ring, const uint8_t* src, int lane) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const int at = 32 * j + lane, row = at / (D / 16), chunk = at % (D / 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + row * D +
                                                                        ((chunk ^ swizzle<D>(row)) << 4)),
                     "l"(src + 16 * at)
                     : "memory");
    }
}
template <int D>
__device__ __forceinline__ void load_keys(uint32_t (&k)[2][D / 16], const uint8_t* kp, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int row = g + 8 * r, chunk = c * (D / 64) + i;
            const uint4 u = *reinterpret_cast<const uint4*>(kp + row * D + ((chunk ^ swizzle<D>(row)) << 4));
            k[r][4 * i] = u.x; k[r][4 * i + 1] = u.y; k[r][4 * i + 2] = u.z; k[r][4 * i + 3] = u.w;
        }
}
template <int D>
__device__ __forceinline__ void load_values(uint32_t (&v)[4][D / 32], const uint8_t* vp, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * c + (r & 1) + 8 * (r >> 1);
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(vp + row * D + ((g ^ swizzle<D>(row)) << 4));
            v[r][0] = u.x; v[r][1] = u.y; v[r][2] = u.z; v[r][3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vp + row * D + (((g >> 1) ^ swizzle<D>(row)) << 4) +
                                                            8 * (g & 1));
            v[r][0] = u.x; v[r][1] = u.y;
        }
    }
}

template <int D, int NT, bool PREC>
struct Tile {
    uint32_t q[NT][D / 16][2], ql[NT][PREC ? D / 16 : 1][2];  // Q^T as B operands
    float qs[NT][2];       // factor of S for rows 2c, 2c + 1
    int pos[NT][2];        // their positions (-1: no such row)
    float o[NT][D / 16][4], l[NT][2], m[NT][2], M[NT][2];
    float f[NT][2];        // 2^(m - M + 14)
};

// Queries as loaded: the thread's channels c d/4 .. + d/4 - 1 of row g of each 8.
template <int D, int NT> struct RawQ {
    uint4 b[NT][D / 32];  // bf16
    float x[D / 4];       // fp32, one group of 8 rows at a time
};
__device__ __forceinline__ long long q_at(const AttnParams& p, int b, int h, int row, const Seq& s, int d, int c) {
    const int tok = row / p.G, head = h * p.G + row % p.G;
    return ((long long)b * p.c.T + tok) * p.ld_q + (long long)head * d + c * (d / 4);
}
template <int D, int NT>
__device__ __forceinline__ void fetch_q(RawQ<D, NT>& r, const AttnParams& p, int b, int h, int row0, const Seq& s,
                                        int lane) {
    if (p.io == DR_F32) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = row0 + 8 * n + (lane >> 2);
        const bool on = row < s.n * p.G;
        const uint4* at = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         (on ? q_at(p, b, h, row, s, D, lane & 3) : 0));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) r.b[n][i] = on ? __ldg(at + i) : make_uint4(0, 0, 0, 0);
    }
}

// The queries of rows row0 .. row0 + 8 NT - 1 as operands, their factors, and empty sums.
template <int D, int NT, bool E4M3, bool PREC>
__device__ __forceinline__ void load_tile(Tile<D, NT, PREC>& t, RawQ<D, NT>& raw, const AttnParams& p, int b, int h,
                                          int row0, const Seq& s, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = row0 + 8 * n + g;
        const bool on = row < s.n * p.G;
        float (&x)[D / 4] = raw.x;
        if (p.io == DR_F32) {
            const float4* at = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                                               (on ? q_at(p, b, h, row, s, D, c) : 0));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float4 u = on ? __ldg(at + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {raw.b[n][i].x, raw.b[n][i].y, raw.b[n][i].z, raw.b[n][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                    x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e;
        float up, rest;
        query_scale(top, e, up, rest);
#pragma unroll
        for (int w = 0; w < D / 16; ++w)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // the channels of the pairs that codes_to_half makes
                const float a = x[4 * w + (E4M3 ? 2 * r : r)] * up * rest;
                const float d = x[4 * w + (E4M3 ? 2 * r + 1 : r + 2)] * up * rest;
                const uint32_t hi = pack_half(a, d);
                t.q[n][w][r] = hi;
                if constexpr (PREC) {
                    const float2 f = unpack_half(hi);
                    // an infinity or NaN stays in the first term
                    t.ql[n][w][r] = pack_half(isfinite(f.x) ? a - f.x : 0.f, isfinite(f.y) ? d - f.y : 0.f);
                }
            }
        // factors and positions belong to rows 2c, 2c + 1: held by the lanes with g = 2c, 2c + 1
        const float f = ldexpf(p.scale * kLog2e, e);
        const int ps = on ? s.len + row / p.G : -1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            t.qs[n][j] = __shfl_sync(0xffffffffu, f, (2 * c + j) * 4);
            t.pos[n][j] = __shfl_sync(0xffffffffu, ps, (2 * c + j) * 4);
            t.l[n][j] = t.f[n][j] = 0.f;
            t.m[n][j] = t.M[n][j] = kNegInf;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) t.o[n][j][i] = 0.f;
    }
}

// A page's weights as 2^(s - x) y: w = 2^(s - M + 14 + ve) (vs 2^-ve), where s - M + ve <= 0.
__device__ __forceinline__ float2 weight_parts(float M, const Meta& page) {
    int e;
    const float y = frexpf(page.vs, &e);  // ve = e; -inf where vs = 0
    return make_float2((M == kNegInf ? 0.f : M) - kBias - page.ve, y);
}

// One step: 32 positions from `first` on, as two halves of 16 with their pages' scales.
// Positions from `end` on hold no value (EDGE: some are hidden from some row).  `same`: both halves
// lie in one page.
template <int D, int NT, bool E4M3, bool PREC, bool EDGE>
__device__ __forceinline__ void step(Tile<D, NT, PREC>& t, const uint8_t* slot, const AttnParams& p, int first,
                                     int end, const Meta& m0, const Meta& m1, bool same, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float sc[NT][2][4];
    {
        uint32_t k0[2][D / 16], k1[2][D / 16];
        load_keys<D>(k0, slot, lane);
        load_keys<D>(k1, slot + 16 * D, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[n][0][i] = sc[n][1][i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {  // the two halves' sums side by side
            uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
            codes_to_half<E4M3>(k0[0][j], a0, a2);
            codes_to_half<E4M3>(k0[1][j], a1, a3);
            codes_to_half<E4M3>(k1[0][j], b0, b2);
            codes_to_half<E4M3>(k1[1][j], b1, b3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(sc[n][0], a0, a1, a2, a3, t.q[n][j][0], t.q[n][j][1]);
                mma(sc[n][1], b0, b1, b2, b3, t.q[n][j][0], t.q[n][j][1]);
                if constexpr (PREC) {
                    mma(sc[n][0], a0, a1, a2, a3, t.ql[n][j][0], t.ql[n][j][1]);
                    mma(sc[n][1], b0, b1, b2, b3, t.ql[n][j][0], t.ql[n][j][1]);
                }
            }
        }
    }
    uint32_t pb[NT][2][2], pl[NT][2][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float top[2], topv[2];  // largest s; largest whole number s + log2 vs
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float k0 = t.qs[n][j] * m0.ks, k1 = t.qs[n][j] * m1.ks;
            sc[n][0][j] *= k0;
            sc[n][0][2 + j] *= k0;
            sc[n][1][j] *= k1;
            sc[n][1][2 + j] *= k1;
            if constexpr (EDGE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // positions first + g + 8 i
                    const int back = t.pos[n][j] - (first + g + 8 * i);
                    if (back < 0 || (p.window > 0 && back >= p.window)) sc[n][i >> 1][2 * (i & 1) + j] = kNegInf;
                }
            }
            const float h0 = fmaxf(sc[n][0][j], sc[n][0][2 + j]), h1 = fmaxf(sc[n][1][j], sc[n][1][2 + j]);
            top[j] = fmaxf(h0, h1);
            topv[j] = fmaxf(ceilf(h0) + m0.ve, ceilf(h1) + m1.ve);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
            top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
        }
        if (same) {
            const float ve = fmaxf(m0.ve, m1.ve);  // a half that no row sees has none
            topv[0] = ceilf(top[0]) + ve;
            topv[1] = ceilf(top[1]) + ve;
        } else {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                topv[0] = fmaxf(topv[0], __shfl_xor_sync(0xffffffffu, topv[0], o));
                topv[1] = fmaxf(topv[1], __shfl_xor_sync(0xffffffffu, topv[1], o));
            }
        }
        const bool grew = top[0] > t.m[n][0] || top[1] > t.m[n][1] || topv[0] > t.M[n][0] || topv[1] > t.M[n][1];
        if (__any_sync(0xffffffffu, grew)) {
            float oscale[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m = fmaxf(t.m[n][j], ceilf(top[j])), M = fmaxf(t.M[n][j], topv[j]);
                t.l[n][j] *= pow2i(t.m[n][j] - m);
                oscale[j] = pow2i(t.M[n][j] - M);
                t.m[n][j] = m;
                t.M[n][j] = M;
                t.f[n][j] = m - M + kBias < 128.f ? pow2i(m - M + kBias) : INFINITY;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                t.o[n][i][0] *= oscale[0];
                t.o[n][i][1] *= oscale[1];
                t.o[n][i][2] *= oscale[0];
                t.o[n][i][3] *= oscale[1];
            }
        }
        float w[2][4];
        bool apart = false;  // (an infinite factor and a scale of zero make a NaN)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float mref = t.m[n][j] == kNegInf ? 0.f : t.m[n][j];
            const float f0 = t.f[n][j] * m0.vs, f1 = t.f[n][j] * m1.vs;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e0 = ex2(sc[n][0][2 * i + j] - mref), e1 = ex2(sc[n][1][2 * i + j] - mref);
                t.l[n][j] += e0 + e1;
                w[0][2 * i + j] = e0 * f0;
                w[1][2 * i + j] = e1 * f1;
            }
            apart |= !(fmaxf(f0, f1) <= pow2i(kMaxFactor));
        }
        if (apart) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (fmaxf(t.f[n][j] * m0.vs, t.f[n][j] * m1.vs) <= pow2i(kMaxFactor)) continue;
                const float2 v0 = weight_parts(t.M[n][j], m0), v1 = weight_parts(t.M[n][j], m1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[0][2 * i + j] = ex2(sc[n][0][2 * i + j] - v0.x) * v0.y;
                    w[1][2 * i + j] = ex2(sc[n][1][2 * i + j] - v1.x) * v1.y;
                }
            }
        }
        if constexpr (EDGE) {  // a hidden position weighs nothing even where the page's value scale is NaN
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sc[n][0][i] == kNegInf) w[0][i] = 0.f;
                if (sc[n][1][i] == kNegInf) w[1][i] = 0.f;
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t hi = pack_half(w[hf][2 * r], w[hf][2 * r + 1]);
                pb[n][hf][r] = transpose8x8(hi);
                if constexpr (PREC) {
                    const float2 x = unpack_half(hi);
                    pl[n][hf][r] = transpose8x8(pack_half(w[hf][2 * r] - x.x, w[hf][2 * r + 1] - x.y));
                }
            }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t v[4][D / 32];
        load_values<D>(v, slot + (2 + hf) * 16 * D, lane);
        if constexpr (EDGE) {
            // what lies in the ring there may be anything: as values it counts as zero
            const bool none = (hf ? m1.id : m0.id) < 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (none || first + 16 * hf + 2 * c + (r & 1) + 8 * (r >> 1) >= end) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) v[r][i] = 0;
                }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            uint32_t a[2][4];  // channels 4j, 4j + 1 and 4j + 2, 4j + 3 of the thread's D / 8
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t x = v[2 * r][j], y = v[2 * r + 1][j];
                codes_to_half<E4M3>(pair_up<E4M3, false>(x, y), a[0][2 * r], a[0][2 * r + 1]);
                codes_to_half<E4M3>(pair_up<E4M3, true>(x, y), a[1][2 * r], a[1][2 * r + 1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma(t.o[n][2 * j + i], a[i][0], a[i][1], a[i][2], a[i][3], pb[n][hf][0], pb[n][hf][1]);
                    if constexpr (PREC)
                        mma(t.o[n][2 * j + i], a[i][0], a[i][1], a[i][2], a[i][3], pl[n][hf][0], pl[n][hf][1]);
                }
        }
    }
}

// ------------------------------------------------------------------ the kernel
constexpr int kRing = 2;  // steps of a warp's ring
template <int D> __host__ __device__ constexpr int ring_bytes() { return kRing * 2 * kStep * D; }
constexpr int kMetas = 64;  // of 16 positions each, a power of two
// The rows of the warps, when they are joined, take the place of the rings.
template <int D, int NT> struct Joined {
    float o[kWarps][8 * NT][D + 4];
    float l[kWarps][8 * NT], m[kWarps][8 * NT], M[kWarps][8 * NT];
};
template <int D, int NT> __host__ __device__ constexpr int rows_or_rings() {
    return kWarps * ring_bytes<D>() > (int)sizeof(Joined<D, NT>) ? kWarps * ring_bytes<D>()
                                                                 : (int)sizeof(Joined<D, NT>);
}
template <int D, int NT> __host__ __device__ constexpr int smem_bytes() {
    return rows_or_rings<D, NT>() + kWarps * kMetas * (int)sizeof(Meta);
}

template <int D, int NT, bool E4M3, bool PREC>
__global__ void __launch_bounds__(kThreads, NT == 1 && !PREC ? 3 : 2) cache_attn_kernel(const AttnParams p) {
    constexpr int ROWS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    Joined<D, NT>& joined = *reinterpret_cast<Joined<D, NT>*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * ring_bytes<D>();
    const uint32_t ring32 = (uint32_t)__cvta_generic_to_shared(ring);
    Meta* metas = reinterpret_cast<Meta*>(smem + rows_or_rings<D, NT>()) + warp * kMetas;
    const bool same = p.c.page > 16;

    chain_wait();
    chain_release();
    const long long total = line_length<ROWS>(p, lane);
    const int used = blocks_used(total, gridDim.x);
    if ((int)blockIdx.x >= used) return;
    const long long begin = share(total, blockIdx.x, used);
    const long long end = share(total, blockIdx.x + 1, used);
    long long at = begin, seq_begin;
    int b = find_seq<ROWS>(p, lane, at, seq_begin);
    bool first_part = true;  // of the block: the part that may continue another block's
    while (at < end) {
        Seq s = make_seq<ROWS>(p, b);
        while (work_of(p, s) == 0 || at >= seq_begin + work_of(p, s)) {
            seq_begin += work_of(p, s);
            if (++b >= p.c.B) return;
            s = make_seq<ROWS>(p, b);
        }
        // stretches of one sequence: head by head, tile by tile, stage by stage
        const long long in = at - seq_begin;
        const int cost = s.stages + kOver, unit = (int)(in / cost), place = (int)(in - (long long)unit * cost);
        const int h = unit / s.tiles, row0 = (unit % s.tiles) * ROWS;
        const int span = (int)min((long long)cost - place, end - at);  // of the line
        const int from = max(0, place - kOver), upto = place + span - kOver;
        if (upto <= from) {  // the tile's start alone
            at += span;
            continue;
        }
        // positions that the tile's rows see
        const int t0 = row0 / p.G, t1 = min(s.n - 1, (row0 + ROWS - 1) / p.G);
        const int hi = s.len + t1 + 1, lo = p.window > 0 ? max(0, s.len + t0 - p.window + 1) : 0;
        // positions that every row sees need no mask
        const int all_hi = s.len + t0 + 1, all_lo = p.window > 0 ? max(0, s.len + t1 - p.window + 1) : 0;

        // Step k = 0 .. n - 1 of the stretch is its stage from + k; the meta of its halves are entries 2k
        // and 2k + 1 modulo kMetas.  A batch of 32 entries is written while the one before is in use.
        const int n = upto - from, base = (s.s0 + from) * kStage + kStep * warp;
        auto page_of = [&](int entry) {
            const int first = base + (entry >> 1) * kStage + (entry & 1) * 16;
            const bool seen = entry < 2 * n && first < hi && first + 16 > lo;
            return seen ? cache_page(p.c, b, first / p.c.page) : -2;
        };
        auto note = [&](int entry, int id) {
            Meta x;
            x.id = id;
            x.ks = x.vs = 0.f;
            x.ve = kNegInf;
            if (id >= 0) {
                const size_t ph = (size_t)id * p.c.H + h;
                x.ks = p.c.k_scale[ph];
                x.vs = p.c.v_scale[ph];
                x.ve = scale_exponent(x.vs);
            } else if (id == -1) {
                flag_index_error(p.c);
                x.ks = x.vs = __uint_as_float(0x7fc00000u);
                x.ve = 0.f;
            }
            metas[entry & (kMetas - 1)] = x;
        };
        auto fetch = [&](int k) {
            if (k < n) {
                const uint32_t slot = ring32 + (k % kRing) * 2 * kStep * D;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int id = metas[(2 * k + hf) & (kMetas - 1)].id;
                    if (id < 0) continue;
                    const int first = base + k * kStage + 16 * hf;
                    const size_t off = (((size_t)id * p.c.H + h) * p.c.page + (first & (p.c.page - 1))) * D;
                    copy_codes<D>(slot + hf * 16 * D, p.c.k + off, lane);
                    copy_codes<D>(slot + (2 + hf) * 16 * D, p.c.v + off, lane);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        RawQ<D, NT> raw;
        fetch_q<D, NT>(raw, p, b, h, row0, s, lane);
        // the first pages are on their way before their scales are asked for
        const int id0 = page_of(lane), id1 = page_of(32 + lane);
        metas[lane].id = id0;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kRing - 1; ++k) fetch(k);
        __syncwarp();
        note(lane, id0);
        note(32 + lane, id1);
        Tile<D, NT, PREC> t;
        load_tile<D, NT, E4M3, PREC>(t, raw, p, b, h, row0, s, lane);
        for (int k = 0; k < n; ++k) {
            __syncwarp();  // step k - 1 is read
            fetch(k + kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();  // every lane's copies of step k are there
            const Meta m0 = metas[(2 * k) & (kMetas - 1)], m1 = metas[(2 * k + 1) & (kMetas - 1)];
            if (m0.id != -2 || m1.id != -2) {
                const int first = base + k * kStage;
                const bool edge = first + kStep > all_hi || first < all_lo || m0.id < 0 || m1.id < 0;
                const uint8_t* slot = ring + (k % kRing) * 2 * kStep * D;
                if (edge) step<D, NT, E4M3, PREC, true>(t, slot, p, first, s.len + s.n, m0, m1, same, lane);
                else step<D, NT, E4M3, PREC, false>(t, slot, p, first, s.len + s.n, m0, m1, same, lane);
            }
            if ((k & 15) == 15) {  // entries 2k - 30 .. 2k + 1 are used up
                __syncwarp();
                note(2 * k + 34 + lane, page_of(2 * k + 34 + lane));
            }
        }

        // join the warps: rows 2c, 2c + 1 of each 8, channels g d/8 ..
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // the rings are free
#pragma unroll
        for (int n8 = 0; n8 < NT; ++n8)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = t.l[n8][j];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int row = 8 * n8 + 2 * c + j;
                if (g == 0) {
                    joined.l[warp][row] = l;
                    joined.m[warp][row] = t.m[n8][j];
                    joined.M[warp][row] = t.M[n8][j];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(&joined.o[warp][row][g * (D / 8) + 2 * i]) =
                        make_float2(t.o[n8][i][j], t.o[n8][i][2 + j]);
            }
        __syncthreads();
        const bool whole = n == s.stages;
        float* out = p.part + ((size_t)blockIdx.x * 2 + (first_part ? 0 : 1)) * tile_floats(D, ROWS);
        first_part = false;
        for (int i = threadIdx.x; i < ROWS * D; i += kThreads) {
            const int r = i / D, ch = i % D, row = row0 + r;
            if (row >= s.n * p.G) break;
            float m = kNegInf, M = kNegInf, l = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) { m = fmaxf(m, joined.m[w][r]); M = fmaxf(M, joined.M[w][r]); }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a warp without weight adds nothing, one that met a NaN hands it on
                const float wl = joined.l[w][r], wo = joined.o[w][r][ch];
                l += wl * (wl == wl ? pow2i(joined.m[w][r] - m) : 1.f);
                sum += wo * (wo == wo ? pow2i(joined.M[w][r] - M) : 1.f);
            }
            if (whole) {
                write_row(p, b, h, row, ch, D, sum, l, m, M);
            } else {
                out[(size_t)r * D + ch] = sum;
                if (ch == 0) {
                    out[ROWS * D + r] = l;
                    out[ROWS * D + ROWS + r] = m;
                    out[ROWS * D + 2 * ROWS + r] = M;
                }
            }
        }
        __syncthreads();  // the rings are filled again
        at += span;
    }
}

// Joins the parts of a tile that several blocks worked on.  Block x: the tile.  A row is a block's
// (DEEP: many parts; y: the row) or a warp's (y: 8 rows).  Rows of no query get zeros (behind a
// sequence's tokens) or NaN (a sequence out of range).
constexpr int kJoinWarps = 8;
template <int D, int NT, bool DEEP>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_attn_join_kernel(const AttnParams p, int blocks,
                                                                          int max_tiles) {
    constexpr int ROWS = 8 * NT, V = D / 32;
    __shared__ float sums[DEEP ? kJoinWarps : 1][D], ls[kJoinWarps], ms[kJoinWarps], Ms[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / (p.c.H * max_tiles), rest = blockIdx.x % (p.c.H * max_tiles);
    const int h = rest / max_tiles, tile = rest % max_tiles;
    const int r = DEEP ? blockIdx.y : blockIdx.y * kJoinWarps + warp, row = tile * ROWS + r;
    // The first kernel's blocks released this one after their own wait: what they read may be read.  Its
    // parts are there after chain_wait(), which every thread comes to, so that the end of this kernel is
    // also the end of the first.
    const Seq s = make_seq<ROWS>(p, b);
    if (row >= s.n * p.G) {
        int len, n;
        const bool ok = cache_seq(p.c, b, len, n);
        if (!ok && lane == 0) flag_index_error(p.c);
        if (row < p.c.T * p.G) {
            const size_t at = ((size_t)b * p.c.T + row / p.G) * p.Hq + h * p.G + row % p.G;
            const float bad = __uint_as_float(0x7fc00000u);
            for (int ch = DEEP ? threadIdx.x : lane; ch < D; ch += DEEP ? 32 * kJoinWarps : 32)
                st_any(p.o, at * D + ch, p.out, ok ? 0.f : bad);
            if (lane == 0 && p.lse) p.lse[at] = ok ? kNegInf : bad;
        }
        chain_wait();
        chain_release();
        return;
    }
    long long total = 0, before = 0;  // the line, and up to this sequence
    for (int i = lane; i < p.c.B; i += 32) {
        const long long x = work_of(p, make_seq<ROWS>(p, i));
        total += x;
        if (i < b) before += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    // the tile's stages on the line, and the blocks that hold them
    const long long a = before + ((long long)h * s.tiles + tile) * (s.stages + kOver) + kOver;
    const int used = blocks_used(total, blocks);
    const int first = holder(total, a, used), last = holder(total, a + s.stages - 1, used);
    // the tile is the first part of a block with stages of it that begins in it or in its start
    const float* head = p.part + ((size_t)first * 2 + (share(total, first, used) >= a - kOver ? 0 : 1)) * tile_floats(D, ROWS);
    chain_wait();
    chain_release();
    if (first == last) return;  // finished by its block
    // A warp takes parts i0, i0 + step, .., kAtOnce of them in flight.  A part without weight adds nothing,
    // one that met a NaN hands it on.
    constexpr int kAtOnce = DEEP ? 8 : 4, step = DEEP ? kJoinWarps : 1;
    float m = kNegInf, M = kNegInf, l = 0.f, sum[V] = {};
    for (int i0 = first + (DEEP ? warp : 0); i0 <= last; i0 += kAtOnce * step) {
        float pl[kAtOnce], pm[kAtOnce], pM[kAtOnce], x[kAtOnce][V];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + k * step;
            const float* in = i == first ? head : p.part + (size_t)i * 2 * tile_floats(D, ROWS);
            const bool on = i <= last;
            pl[k] = on ? in[ROWS * D + r] : 0.f;
            pm[k] = on ? in[ROWS * D + ROWS + r] : kNegInf;
            pM[k] = on ? in[ROWS * D + 2 * ROWS + r] : kNegInf;
#pragma unroll
            for (int j = 0; j < V; ++j) x[k][j] = on ? in[(size_t)r * D + 32 * j + lane] : 0.f;
        }
        float m2 = m, M2 = M;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) { m2 = fmaxf(m2, pm[k]); M2 = fmaxf(M2, pM[k]); }
        l = l == l ? l * pow2i(m - m2) : l;
        const float fs = pow2i(M - M2);
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = sum[j] == sum[j] ? sum[j] * fs : sum[j];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (i0 + k * step > last) break;  // uniform
            const float f = pow2i(pM[k] - M2);
            l += pl[k] == pl[k] ? pl[k] * pow2i(pm[k] - m2) : pl[k];
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += x[k][j] == x[k][j] ? x[k][j] * f : x[k][j];
        }
        m = m2;
        M = M2;
    }
    if constexpr (!DEEP) {
#pragma unroll
        for (int j = 0; j < V; ++j) write_row(p, b, h, row, 32 * j + lane, D, sum[j], l, m, M);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[warp][32 * j + lane] = sum[j];
        if (lane == 0) { ls[warp] = l; ms[warp] = m; Ms[warp] = M; }
        __syncthreads();
        if (threadIdx.x >= D) return;
        float x = 0.f, tot = 0.f, mm = kNegInf, MM = kNegInf;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) { mm = fmaxf(mm, ms[i]); MM = fmaxf(MM, Ms[i]); }
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
            const float y = sums[i][threadIdx.x];
            x += y == y ? y * pow2i(Ms[i] - MM) : y;
            tot += ls[i] == ls[i] ? ls[i] * pow2i(ms[i] - mm) : ls[i];
        }
        write_row(p, b, h, row, threadIdx.x, D, x, tot, mm, MM);
    }
}

constexpr int kMaxBlocks = 152 * 8;

template <int D, int NT, bool E4M3, bool PREC>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    constexpr int smem = smem_bytes<D, NT>();
    if (cudaError_t e = set_smem_once(cache_attn_kernel<D, NT, E4M3, PREC>, smem, ready); e != cudaSuccess) return e;
    static const int resident = resident_blocks(cache_attn_kernel<D, NT, E4M3, PREC>, kThreads, smem);
    if (resident <= 0) return cudaErrorUnknown;
    const int blocks = resident < kMaxBlocks ? resident : kMaxBlocks;
    {
        TraceScope ts("cache_attn", st);
        if (cudaError_t e = launch_chained(cache_attn_kernel<D, NT, E4M3, PREC>, dim3(blocks), kThreads, smem, st, p);
            e != cudaSuccess)
            return e;
    }
    const int max_tiles = (p.c.T * p.G + 8 * NT - 1) / (8 * NT);
    TraceScope ts("cache_attn_join", st);
    // a block for each row where a tile has 8 parts or more on average: 114 parts take 5 us (a warp: 12 us);
    // a warp where it has fewer: 1024 rows of one or two parts take 7 us (a block: 11 us)
    const unsigned tiles = (unsigned)p.c.B * p.c.H * max_tiles;
    const int rows = max_tiles > 1 ? 8 * NT : p.c.T * p.G;
    return tiles * 8 <= (unsigned)blocks
               ? launch_chained(cache_attn_join_kernel<D, NT, true>, dim3(tiles, rows), 32 * kJoinWarps, 0, st, p, blocks, max_tiles)
               : launch_chained(cache_attn_join_kernel<D, NT, false>, dim3(tiles, (rows + kJoinWarps - 1) / kJoinWarps),
                                32 * kJoinWarps, 0, st, p, blocks, max_tiles);
}

// Rows of a tile: 16 halve the reads of the cache where a sequence and head have more than 8.  The
// split operands of 16 rows do not fit the registers, there the tiles stay at 8.
template <int D, bool E4M3>
cudaError_t by_rows(const AttnParams& p, cudaStream_t st) {
    if (p.io == DR_F32 || p.out == DR_F32) return launch<D, 1, E4M3, true>(p, st);
    return p.c.T * p.G > 8 ? launch<D, 2, E4M3, false>(p, st) : launch<D, 1, E4M3, false>(p, st);
}

}  // namespace

size_t cache_attn_rows_bytes(int d) { return (size_t)kMaxBlocks * 2 * tile_floats(d, 16) * sizeof(float); }

cudaError_t cache_attn_rows(const AttnParams& p, cudaStream_t st) {
    if (p.c.code == DR_CODE_E4M3) return p.c.d == 128 ? by_rows<128, true>(p, st) : by_rows<64, true>(p, st);
    return p.c.d == 128 ? by_rows<128, false>(p, st) : by_rows<64, false>(p, st);
}

}  // namespace dr
