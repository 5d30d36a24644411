// linear_attn_tc.cu -- linear attention with a decay for each head, bf16: the chunked scan of linear_attn.cuh on
// the fifth-generation tensor cores.  Chunks of C = 128 tokens, i and j within the chunk, X the state before it,
// a = e^g, n the chunk's tokens:
//   A = Q K^T;  P_ij = beta a^{|i-j|} A_ij (j <= i, reverse j >= i);  out = alpha (P V + diag(a^{out(i)}) Q X)
//   X' = a^n X + K'^T V,  K'_j = beta a^{in(j)} k_j
//   forward: out(i) = i + 1, in(j) = n - 1 - j;  reverse: out(i) = n - 1 - i, in(j) = j + 1
// so no power of a is ever above one, however strong the decay.
//
// A block has a sequence, or a segment of one, and a head.  The state stays in fp32 registers, a row of it in each
// thread of eight warps, half each; what a chunk adds comes from tensor memory, and a bf16 image of the state goes to
// shared memory for the next chunk's queries.  K' is a sum of two bf16 parts (2^-16 of it is lost), so that what the states add up over
// a sequence is not bf16; P, and the state as an operand, are rounded once (2^-8 at most).
// Tensor memory: A with P over it, Q X, P V, K'^T V: 4 x 128 columns.
// Warps 0-3: P.  4-7: K' (its high part over K, once A is there).  8-11: output rows.  12-19: state.  20: products,
// 21: copies, through a ring of five tiles in the order Q, K, V.
//
// The products of a chunk are issued as P V (n), Q X (n), A (n + 1), K'V (n), each when what it needs is there.  So the
// tile of a chunk's queries is the first to be free, for the values of the next chunk, which are on their way while A
// and K'V run (with Q X last the loop waited for them: 133 us for b8 t4096 h16 d128 instead of 119).
// 8 x 4096 tokens, 16 heads of 128: 110 us (537 MB, 4.9 TB/s), the gradient's three scans 295 us.  Bound by how little is
// in flight: of 227 KB, low parts and state hold 64 KB and a chunk's own tiles most of the ring (with nothing but the
// copies the same kernel takes 61 us).  What moved it: short code for each task (unrolled to the end, five instruction
// streams missed the instruction cache: 170 us), K' and P by warps of their own, the order of the products, rows by tensor
// stores.  Slower: prefetches of the next chunks to L2 (158 us where it was 144), K' V before P V (173).
#include "f32x2.cuh"
#include "linear_work.cuh"
#include "tc_block.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kC = kScanChunk, kThreads = 768, kSlots = 5;
// Registers of a thread: as launched, then of the six groups of four warps (two of them the state's).  What is compiled for
// 80 spills 24 bytes (64 channels), 56 (128) or 80 (64 and 128), 8 where only states are formed.
constexpr int kRegs = 80, kWeightRegs = 88, kKeyRegs = 72, kOutRegs = 96, kStateRegs = 88, kOtherRegs = 48;
static_assert(kWeightRegs >= kRegs && kOutRegs >= kRegs && kStateRegs >= kRegs && kKeyRegs <= kRegs && kOtherRegs <= kRegs,
              "each takes or gives, as its instruction says");
static_assert(kWeightRegs + kKeyRegs + kOutRegs + 2 * kStateRegs + kOtherRegs <= 6 * kRegs, "more than the block has");
constexpr uint32_t kA = 0, kQX = 128, kPV = 256, kKV = 384;  // columns of tensor memory

struct Control {
    uint64_t full[kSlots], empty[kSlots], landed, afull, akeys, pfull, kfull, dfull, dread, xfull, xempty, ofull, oempty, drained;
    uint32_t tmem;
    volatile int dead;
    __align__(16) float power[32 + kC];  // beta a^n from place 32 on, zeros before
    __align__(16) float column[32];  // a^{31 - j}, reverse a^j
};
template <int DK, int DV> struct Smem {
    // K'^T is read as 128 rows, for 64 channels 64 rows past them (at most of x) that nobody looks at; x: the image of the
    // state, and 128 output rows
    static constexpr int slot = kC * (DK > DV ? DK : DV) * 2, low = kSlots * slot, x = low + kC * DK * 2,
                         control = x + kC * DV * 2, bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};

// What goes through the ring for a chunk: Q, K, V, or K, V where only states are formed.
template <bool ONLY> constexpr int kTiles = ONLY ? 2 : 3;
template <bool ONLY> constexpr int kKeyTile = ONLY ? 0 : 1;

template <int DK, int DV, bool ONLY>
__device__ __forceinline__ void copy_tiles(const ScanParams& p, const Work& w, int head, const CUtensorMap* mq,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t landings = 0;
    Ring<kSlots> ring;
    [&] {
        for (int n = 0; n < w.chunks; ++n) {
            const int first = w.at(p, n), row = w.row0 + first, rows = w.tokens(first);
#pragma unroll
            for (int i = 0; i < kTiles<ONLY>; ++i) {
                constexpr int V = kTiles<ONLY> - 1;
                if (!wait(ct.dead, &ct.empty[ring.at], ring.phase ^ 1)) return;
                uint8_t* tile = smem + ring.at * Smem<DK, DV>::slot;
                // values behind the sequence are summed with weights of zero: they have to be numbers
                const bool cut = i == V && rows < kC;
                uint64_t* bar = cut ? &ct.landed : &ct.full[ring.at];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, kC * (i == V ? DV : DK) * 2);
                    if (i == V) load_rows<kC, DV>(tile, mv, bar, head, row);
                    else load_rows<kC, DK>(tile, i == kKeyTile<ONLY> ? mk : mq, bar, head, row);
                }
                __syncwarp();
                if (cut) {
                    if (!wait(ct.dead, &ct.landed, landings++ & 1)) return;
                    clear_rows<kC, DV>(tile, rows);
                    if (lane == 0) mbar_arrive(&ct.full[ring.at]);
                    __syncwarp();
                }
                ring.step();
            }
        }
    }();
    settle(&ct.landed, landings);
    settle(ring, ct.full);
}

template <int DK, int DV, bool ONLY> struct Issuer {
    using S = Smem<DK, DV>;
    static constexpr int N = kTiles<ONLY>, K = kKeyTile<ONLY>, Q = 0, V = N - 1;
    Control& ct;
    uint32_t tm;
    uint64_t row0, col0, low0, x0;  // descriptors: of slot 0, by rows and by columns; of the low parts; of the state
    __device__ __forceinline__ Issuer(uint8_t* smem, Control& c) : ct(c), tm(c.tmem) {
        const uint32_t base = smem_u32(smem);
        row0 = desc_kmajor(Tile{base, kC}, 0);
        col0 = desc_mnmajor(Tile{base, kC}, 0);
        low0 = desc_mnmajor(Tile{base + S::low, kC}, 0);
        x0 = desc_mnmajor(Tile{base + S::x, DK}, 0);
    }
    static __device__ __forceinline__ uint32_t slot(int n, int i) { return (uint32_t)(N * n + i) % kSlots; }
    static __device__ __forceinline__ uint64_t at(int n, int i) { return slot(n, i) * (uint64_t)(S::slot >> 4); }
    __device__ __forceinline__ bool arrived(int n, int i) {
        return wait(ct.dead, &ct.full[slot(n, i)], ((uint32_t)(N * n + i) / kSlots) & 1);
    }
    __device__ __forceinline__ bool scores(int n) {  // A
        if (!arrived(n, Q) || !arrived(n, K)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK; kk += 16)  // 16 channels: 32 bytes of a 128-byte row
                mma_bf16(tm + kA, row0 + at(n, Q) + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8,
                         row0 + at(n, K) + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8, idesc_bf16(kC, kC), kk > 0);
            mma_commit(&ct.afull);
            mma_commit(&ct.akeys);
        }
        __syncwarp();
        return true;
    }
    __device__ __forceinline__ bool values(int n) {  // P V
        if (!wait(ct.dead, &ct.pfull, n & 1) || !wait(ct.dead, &ct.oempty, (n & 1) ^ 1)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kC; kk += 16)  // 16 tokens: 16 rows of 128 bytes
                mma_ts(tm + kPV, tm + kA + kk / 2, col0 + at(n, V) + kk * 8, idesc_bf16(kC, DV, false, true), kk > 0);
        }
        __syncwarp();
        return true;
    }
    __device__ __forceinline__ bool added(int n) {  // K'V
        if (!wait(ct.dead, &ct.kfull, n & 1) || !wait(ct.dead, &ct.dread, (n & 1) ^ 1)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < kC; kk += 16)
                    mma_bf16(tm + kKV, (part ? low0 : col0 + at(n, K)) + kk * 8, col0 + at(n, V) + kk * 8,
                             idesc_bf16(128, DV, true, true), part + kk > 0);
            mma_commit(&ct.dfull);
            mma_commit(&ct.empty[slot(n, K)]);
            mma_commit(&ct.empty[slot(n, V)]);  // after P V too
        }
        __syncwarp();
        return true;
    }
    __device__ __forceinline__ bool reads(int n) {  // Q X
        if (!wait(ct.dead, &ct.xfull, n & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK; kk += 16)
                mma_bf16(tm + kQX, row0 + at(n, Q) + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8, x0 + kk * 8,
                         idesc_bf16(kC, DV, false, true), kk > 0);
            mma_commit(&ct.ofull);
            mma_commit(&ct.empty[slot(n, Q)]);
        }
        __syncwarp();
        return true;
    }
    __device__ __forceinline__ void run(int chunks) {
        if (ONLY) {
            for (int n = 0; n < chunks; ++n)
                if (!arrived(n, V) || !added(n)) return;
            return;
        }
        if (chunks > 0 && !scores(0)) return;
        for (int n = 0; n < chunks; ++n) {
            if (!arrived(n, V) || !values(n) || !reads(n)) return;
            if (n + 1 < chunks && !scores(n + 1)) return;
            if (!added(n)) return;
        }
    }
};

// The parts hi + lo of f times two bf16 values: what hi, rounded, leaves of a value is rounded to lo.
__device__ __forceinline__ void split2(uint32_t u, float f, uint32_t& hi, uint32_t& lo) {
    const float2 x = mul2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), both(f));
    hi = pack_bf16(x.x, x.y);
    lo = pack_bf16(x.x - __uint_as_float(hi << 16), x.y - __uint_as_float(hi & 0xffff0000u));
}
// Warps 4-7, a token per thread: K', channels c0 .. c1 - 1 (all; where there is no P to form warps 0-3 have half of them).
template <int DK, int DV, bool ONLY>
__device__ __forceinline__ void keys(const ScanParams& p, const Work& w, int head, int c0, int c1, uint8_t* smem, Control& ct) {
    const int j = threadIdx.x & (kC - 1);
    const float g = p.g[head], f_in = p.reverse ? p.scale : 1.f;
    for (int n = 0; n < w.chunks; ++n) {
        const uint32_t u = kTiles<ONLY> * n + kKeyTile<ONLY>;
        const int tokens = w.tokens(w.at(p, n));
        const float f = j < tokens ? f_in * decay(g, (float)(p.reverse ? j + 1 : tokens - 1 - j)) : 0.f;
        uint8_t* tile = smem + u % kSlots * Smem<DK, DV>::slot;
        if (!wait(ct.dead, &ct.full[u % kSlots], (u / kSlots) & 1)) return;
        if (!ONLY) {  // A needs the keys as they came; it is formed up to a chunk ahead of this, so its phases count both
            warp_arrive(&ct.akeys);
            if (!wait(ct.dead, &ct.akeys, n & 1)) return;
        }
        if (n && !wait(ct.dead, &ct.dfull, (n - 1) & 1)) return;       // low parts of the chunk before are in use
        const bool none = tokens < kC && j >= tokens;  // behind the sequence: may be no numbers
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {  // four pieces are read before the first is written
            const uint32_t row = c / 64 * kC * 128 + j * 128;
            uint4 x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const uint4*>(tile + row + (((c / 8 + q) & 7 ^ (j & 7)) << 4));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t off = row + (((c / 8 + q) & 7 ^ (j & 7)) << 4);
                uint4 hi, lo;
                if (none) x[q] = make_uint4(0, 0, 0, 0);
                split2(x[q].x, f, hi.x, lo.x);
                split2(x[q].y, f, hi.y, lo.y);
                split2(x[q].z, f, hi.z, lo.z);
                split2(x[q].w, f, hi.w, lo.w);
                *reinterpret_cast<uint4*>(tile + off) = hi;
                *reinterpret_cast<uint4*>(smem + Smem<DK, DV>::low + off) = lo;
            }
        }
        fence_async_smem();
        warp_arrive(&ct.kfull);
    }
}

// Warps 0-3, a token per thread: P, 32 columns at a time.  Those that all the warp's rows see take a^{|i-j|} as a row's
// and a column's factor, both at most one; those on the diagonal one of the powers each; the others are zero.
__device__ __forceinline__ void weights(const ScanParams& p, const Work& w, Control& ct) {
    const int i = threadIdx.x, warp = i >> 5;
    const uint32_t tm = warp_lane_base(ct.tmem);
    for (int n = 0; n < w.chunks; ++n) {
        const int tokens = w.tokens(w.at(p, n));
        if (!wait(ct.dead, &ct.afull, n & 1)) return;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            float s[32];
            uint32_t z[16];
            const int c = 32 * b;
            if (p.reverse ? b < warp : b > warp) {
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = 0;
            } else {
                tmem_ld32(tm + kA + c, s);
                tmem_ld_wait();
                if (tokens < kC) {  // scores behind the sequence may be no numbers
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j >= tokens) s[j] = 0.f;
                }
                if (b == warp) {
                    // power[n] is zero for n < 0
                    const float* f = ct.power + 32 + (p.reverse ? c - i : i - c);
                    const int step = p.reverse ? 1 : -1;
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[j] *= f[step * j];
                } else {
                    const float2 fr = both(ct.power[32 + (p.reverse ? c - i : i - c - 31)]);
                    const float4* fc = reinterpret_cast<const float4*>(ct.column);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 y = fc[j / 4];
                        const float2 t0 = mul2(make_float2(s[j], s[j + 1]), mul2(fr, make_float2(y.x, y.y)));
                        const float2 t1 = mul2(make_float2(s[j + 2], s[j + 3]), mul2(fr, make_float2(y.z, y.w)));
                        s[j] = t0.x; s[j + 1] = t0.y; s[j + 2] = t1.x; s[j + 3] = t1.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
            }
            tmem_st16(tm + kA + c / 2, z);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&ct.pfull);
    }
}

// Warps 8-11, a token per thread.  The rows of a whole chunk leave as tensor stores, 32 by each warp, from the place of the
// state's image, which nobody needs between Q X and the next state: a lane has a row of its own, and its pieces in
// memory would be a transaction each (122 us for b8 t4096 h16 d128 that way, 97 without stores).
template <int DK, int DV>
__device__ __forceinline__ void outputs(const ScanParams& p, const Work& w, int head, const CUtensorMap* mo, uint8_t* smem, Control& ct) {
    const int i = threadIdx.x & (kC - 1), lane = threadIdx.x & 31;
    const uint32_t tm = warp_lane_base(ct.tmem);
    const float g = p.g[head], f_out = p.reverse ? 1.f : p.scale;
    uint8_t* tile = smem + Smem<DK, DV>::x;
    for (int n = 0; n < w.chunks; ++n) {
        const int first = w.at(p, n), tokens = w.tokens(first);
        const float2 fx = both(f_out * decay(g, (float)(p.reverse ? tokens - 1 - i : i + 1))), fy = both(f_out);
        if (!wait(ct.dead, &ct.ofull, n & 1)) break;
        tc_fence_after();
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (w.row0 + first + i) * p.ld_o + (long long)head * DV;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
            float x[32], y[32];
            tmem_ld32(tm + kQX + c, x);
            tmem_ld32(tm + kPV + c, y);
            tmem_ld_wait();
            uint32_t z[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 o = fma2(fx, make_float2(x[2 * j], x[2 * j + 1]), mul2(fy, make_float2(y[2 * j], y[2 * j + 1])));
                z[j] = pack_bf16(o.x, o.y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 u = make_uint4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
                if (tokens == kC) *reinterpret_cast<uint4*>(tile + sw128_offset(i, c + 8 * j, kC)) = u;
                else if (i < tokens) reinterpret_cast<uint4*>(to + c)[j] = u;
            }
        }
        tc_fence_before();
        warp_arrive(&ct.oempty);
        if (tokens == kC) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int c = 0; c < DV; c += 64)
                    tma_store_3d(mo, tile + (c / 64) * kC * 128 + i * 128, c, head, w.row0 + first + i);
                bulk_commit();
                bulk_wait_read();
            }
        }
        warp_arrive(&ct.xempty);
    }
    if (lane == 0) bulk_wait_all();
}

// Warps 12-19: half a row of the state per thread (of the first DK rows; warps 12-15 the first half of the columns).
template <int DK, int DV, bool ONLY>
__device__ __forceinline__ void states(const ScanParams& p, const Work& w, int head, uint8_t* smem, Control& ct) {
    constexpr int N = DV / 2;  // columns of a thread
    const int r = threadIdx.x & 127, c0 = threadIdx.x >= 16 * 32 ? N : 0;
    const bool on = r < DK;
    const uint32_t td = warp_lane_base(ct.tmem) + kKV + c0;
    const float g = p.g[head];
    const size_t unit = (size_t)w.seq * p.H + head;
    float x[N];
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = 0.f;
    const float* from = w.before ? w.before : p.x0 ? p.x0 + unit * DK * DV : nullptr;
    if (!ONLY && from && on) {
        if (!w.before && p.x0_transposed) {
#pragma unroll
            for (int c = 0; c < N; ++c) x[c] = from[(c0 + c) * DK + r];
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
                const float4 y = load4(from + r * DV + c0 + c);
                x[c] = y.x; x[c + 1] = y.y; x[c + 2] = y.z; x[c + 3] = y.w;
            }
        }
    }
    for (int n = 0; n <= w.chunks; ++n) {
        if (n > 0) {
            if (!wait(ct.dead, &ct.dfull, (n - 1) & 1)) return;
            tc_fence_after();
            const float a = decay(g, (float)w.tokens(w.at(p, n - 1)));
#pragma unroll
            for (int c = 0; c < N; c += 16) {
                float y[16];
                tmem_ld16(td + c, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 z = fma2(both(a), make_float2(x[c + j], x[c + j + 1]), make_float2(y[j], y[j + 1]));
                    x[c + j] = z.x;
                    x[c + j + 1] = z.y;
                }
            }
            tc_fence_before();
            warp_arrive(&ct.dread);
            if (!ONLY && !wait(ct.dead, &ct.xempty, (n - 1) & 1)) return;  // its image, and then the rows there, have been read
        }
        if (!ONLY && n < w.chunks) {
            if (on)
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = x[c + j];
                    tile_store16(smem + Smem<DK, DV>::x, r, c0 + c, DK, y);
                }
            fence_async_smem();
            warp_arrive(&ct.xfull);
        }
    }
    float* to = ONLY ? const_cast<float*>(w.before) : w.last && p.xT ? p.xT + unit * DK * DV : nullptr;
    if (to && on)
#pragma unroll
        for (int c = 0; c < N; c += 4) store4(to + r * DV + c0 + c, make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]));
}

// n scans of the same sequences side by side: what they share is read at about the same time, and a block that is
// through with one takes what comes next of all.
struct ScanSet {
    CUtensorMap m[kMostScans][4];  // of q, k, v, out
    ScanParams p[kMostScans];
};
template <int DK, int DV, bool ONLY>
__device__ __forceinline__ void scan_block(const ScanParams& p, const CUtensorMap* m, const Work& w, int head, uint8_t* smem) {
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<DK, DV>::control);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ct.full[i], 1);
            mbar_init(&ct.empty[i], 1);
        }
        for (uint64_t* one : {&ct.landed, &ct.afull, &ct.dfull, &ct.ofull, &ct.drained}) mbar_init(one, 1);
        mbar_init(&ct.akeys, 1 + 4);
        for (uint64_t* four : {&ct.pfull, &ct.xempty, &ct.oempty}) mbar_init(four, 4);
        mbar_init(&ct.kfull, ONLY ? 8 : 4);
        for (uint64_t* eight : {&ct.dread, &ct.xfull}) mbar_init(eight, 8);
        ct.dead = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < 32 + kC)
        ct.power[threadIdx.x] = threadIdx.x < 32 ? 0.f : (p.reverse ? p.scale : 1.f) * decay(p.g[head], (float)threadIdx.x - 32.f);
    if (threadIdx.x < 32) ct.column[threadIdx.x] = decay(p.g[head], (float)(p.reverse ? threadIdx.x : 31 - threadIdx.x));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWeightRegs));
        if (ONLY) keys<DK, DV, ONLY>(p, w, head, DK / 2, DK, smem, ct);
        else weights(p, w, ct);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kKeyRegs));
        keys<DK, DV, ONLY>(p, w, head, 0, ONLY ? DK / 2 : DK, smem, ct);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
        if (!ONLY) outputs<DK, DV>(p, w, head, m + 3, smem, ct);
    } else if (warp < 20) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        states<DK, DV, ONLY>(p, w, head, smem, ct);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 20) Issuer<DK, DV, ONLY>(smem, ct).run(w.chunks), drain(&ct.drained);
        else if (warp == 21) copy_tiles<DK, DV, ONLY>(p, w, head, m, m + 1, m + 2, smem, ct);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.status) *reinterpret_cast<volatile int32_t*>(p.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}
// Scans with DA channels of queries and DB of values, or the other way round.  ONLY: the segments' own states, from nothing.
template <int DA, int DB, bool ONLY>
__global__ void __launch_bounds__(kThreads, 1) linear_scan_tc_kernel(const __grid_constant__ ScanSet set, int n) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const ScanParams& p = set.p[blockIdx.x % n];
    const CUtensorMap* m = set.m[blockIdx.x % n];
    const int item = blockIdx.x / n, head = item % p.H;
    Work w;
    if (!make_work(p, item / p.H, head, w) || (ONLY && (!w.before || w.last))) return;
    if (DA == DB || p.dk == DA) scan_block<DA, DB, ONLY>(p, m, w, head, smem);
    else scan_block<DB, DA, ONLY>(p, m, w, head, smem);
}

template <int DA, int DB, bool ONLY> cudaError_t launch(const ScanSet& set, int n, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    constexpr int smem = Smem<DA, DB>::bytes > Smem<DB, DA>::bytes ? Smem<DA, DB>::bytes : Smem<DB, DA>::bytes;
    // the split of the registers must not ask for more than the block is launched with: it would wait for them
    static const bool fits = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, linear_scan_tc_kernel<DA, DB, ONLY>) == cudaSuccess && a.numRegs == kRegs;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = set_smem_once(linear_scan_tc_kernel<DA, DB, ONLY>, smem, ready); e != cudaSuccess) return e;
    TraceScope ts(ONLY ? "linear_segments_tc" : "linear_scan_tc", st);
    const long long blocks = scan_items(set.p[0]) * set.p[0].H * n;
    if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
    linear_scan_tc_kernel<DA, DB, ONLY><<<(unsigned)blocks, kThreads, smem, st>>>(set, n);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linear_scans_tc(const ScanParams* p, int n, bool only, cudaStream_t st) {
    ScanSet set;
    for (int i = 0; i < n; ++i) {
        set.p[i] = p[i];
        if (!head_rows_map(&set.m[i][0], p[i].q, p[i].dk, p[i].H, p[i].rows, p[i].ld_q, kC) ||
            !head_rows_map(&set.m[i][1], p[i].k, p[i].dk, p[i].H, p[i].rows, p[i].ld_k, kC) ||
            !head_rows_map(&set.m[i][2], p[i].v, p[i].dv, p[i].H, p[i].rows, p[i].ld_v, kC) ||
            !head_rows_map(&set.m[i][3], p[i].out, p[i].dv, p[i].H, p[i].rows, p[i].ld_o, 32))
            return cudaErrorInvalidValue;
    }
    if (p->dk != p->dv) return only ? launch<64, 128, true>(set, n, st) : launch<64, 128, false>(set, n, st);
    if (p->dk == 128) return only ? launch<128, 128, true>(set, n, st) : launch<128, 128, false>(set, n, st);
    return only ? launch<64, 64, true>(set, n, st) : launch<64, 64, false>(set, n, st);
}

}  // namespace dr
