// cache_attn_tc.cu -- attention of many query tokens of each sequence over the paged 8-bit cache
// (dr.h, dr_cache_attn; bf16 queries and outputs): the products on the fifth-generation tensor cores.
//
// A block works on a tile of 256 rows (query tokens times the G query heads that share a cache head,
// row = t * G + g), two halves of 128, over a stretch of positions, in stages of 64:
//   S = Q K^T   128 x 64 for each half, contraction d
//   O += P V    128 x d for each half, contraction 64
// Tensor memory, all 512 columns of it, holds O and two S of each half, used in turn; P takes the
// columns of its S.  So S of the next stage is formed before the weights of this one are there, and a
// half waits for nobody (with one S it waited for the exchange with the issuing thread and for two
// products every stage: 2950 cycles for both halves, where the products take 1140).  Shared memory
// holds Q, and K and V as 16-bit floats (exact), three stages of K and four of V.
// Warps 0-3 and 4-7 hold a row of their half per thread: they read S, keep the softmax statistics and
// write P.  Warps 8-15 turn codes into the operand tiles (four of them were slower than the rows: a
// stage took 2400 cycles instead of 2100); warps 16 and 18 issue the products; warp 17 has the codes
// copied to a ring in shared memory.
//
// Softmax in base 2 with whole-number references, as in cache_attn.cu: p = 2^(s - m), l = sum p,
// operand w = p vs 2^(m - M + 13).  The accumulator is rescaled (exactly, by a power of two) only when
// a row's largest s + log2 vs passes M by more than 2.9: a row's largest operand is never below 2^12
// nor above 2^15.9, and with scores of unit size few stages rescale (8 % of them, 63 % where M
// follows by whole numbers).  Where vs 2^(m - M + 13) could pass 2^100, w is a power of two
// of its own, in a copy of the loop: without the test for it 124 us instead of 126.5.
//
// The stages of all tiles form one line that is divided evenly among the blocks (one per SM); a tile
// that several blocks worked on is joined by a second kernel from their rows in the workspace.
//
// Chunks of 512 tokens of four sequences of 4000 to 8191 positions, 16 query heads on 4 of 128: 126 to 127 us for
// 107 GFLOP (0.85 PFLOP/s; tensor pipe 38 % active).  The rows' threads bound it: they work 1650 of a stage's
// 2100 cycles (350 instructions a warp, two warps a scheduler), and the products take 1140.
#include "attn_util.cuh"
#include "f32x2.cuh"
#include "tc.cuh"
#include "trace.cuh"

namespace dr {
namespace {

using namespace tc;

constexpr int kHalf = 128, kRows = 2 * kHalf, kStage = 64;
constexpr int kTcThreads = 640;  // warps 0-7 rows, 8-15 codes, 16-18 products and copies (19: none)
// Registers of a thread: as launched, then of the rows' threads and of the others, which give theirs up.
constexpr int kRegs = 96, kRowRegs = 152, kOtherRegs = 56;  // 130 us; 132 with 144 and 64, 137 with 128 and 72
static_assert(256 * kRowRegs + (kTcThreads - 256) * kOtherRegs <= kTcThreads * kRegs, "more than the block has");
constexpr int kCodeThread0 = 256;
constexpr int kKBuffers = 3, kVBuffers = 4;  // stages of K and V as operands: V is needed for longer
constexpr int kRaw = 3;                      // as codes
constexpr int kTcBias = 13;       // weights as 16-bit operands: 2^12 .. 2^15.9 for a row's largest
constexpr float kSlack = 2.9f;
constexpr int kTcOver = 8;       // what a tile costs beside its stages, in stages (126 us with 8, 127 with 6 and 12, 130 with 4)
constexpr int kMetas = 8;        // stages whose scales are kept: more than the warps can be apart
constexpr int kMaxTcBlocks = 152;
// columns of tensor memory of half i
__device__ __forceinline__ uint32_t s_col(int i, uint32_t b) { return 128 * i + 64 * b; }  // S, and P over it
__device__ __forceinline__ uint32_t o_col(int i) { return 256 + 128 * i; }

// ------------------------------------------------------------------ the line of stages
struct TcTile {
    int row0, t0, t1;    // first row; tokens of the first and last row
    int lo, hi;          // positions that its rows see
    int s0, stages;
};
__device__ __forceinline__ int tiles_of(const AttnParams& p, int n) { return (n * p.G + kRows - 1) / kRows; }
__device__ __forceinline__ TcTile make_tile(const AttnParams& p, int len, int n, int tile) {
    TcTile t;
    t.row0 = tile * kRows;
    t.t0 = t.row0 / p.G;
    t.t1 = min(n - 1, (t.row0 + kRows - 1) / p.G);
    t.hi = len + t.t1 + 1;
    t.lo = p.window > 0 ? max(0, len + t.t0 - p.window + 1) : 0;
    t.s0 = t.lo / kStage;
    t.stages = (t.hi + kStage - 1) / kStage - t.s0;
    return t;
}
// Places on the line of one head of sequence b (0: nothing to do).
__device__ __forceinline__ long long head_work(const AttnParams& p, int b) {
    int len, n;
    if (!cache_seq(p.c, b, len, n)) return 0;
    long long w = 0;
    for (int i = 0, tiles = tiles_of(p, n); i < tiles; ++i) w += make_tile(p, len, n, i).stages + kTcOver;
    return w;
}

// A block's stretch of a tile: stages from .. upto - 1.
struct Stretch {
    int b, h, len, n, from, upto;
    bool whole, first;   // the whole tile; the block's first stretch
    TcTile t;
};
// The whole line (every lane gets it).
__device__ __forceinline__ long long line_length(const AttnParams& p, int lane) {
    long long total = 0;
    for (int i = lane; i < p.c.B; i += 32) total += head_work(p, i) * p.c.H;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
}
// Walks through a block's part of the line; every warp does so for itself, with the same result.
struct Walk {
    long long at, end;
    int b, h, tile, place, len, n;
    bool first;

    __device__ __forceinline__ void start(const AttnParams& p, int lane) {
        const long long total = line_length(p, lane);
        const int used = blocks_used(total, gridDim.x);
        at = end = 0;
        first = true;
        if ((int)blockIdx.x >= used) return;
        at = share(total, blockIdx.x, used);
        end = share(total, blockIdx.x + 1, used);
        find(p, lane);
    }
    // The tile that holds place `at`, and the place within it; b < 0 where there is none.
    __device__ __forceinline__ void find(const AttnParams& p, int lane) {
        long long before = 0, mine = 0;
        b = -1;
        for (int b0 = 0; b0 < p.c.B && b < 0; b0 += 32) {
            const long long w = b0 + lane < p.c.B ? head_work(p, b0 + lane) : 0;
            const long long upto = before + warp_scan(w * p.c.H, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, upto > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                before = __shfl_sync(0xffffffffu, upto - w * p.c.H, l);
                mine = __shfl_sync(0xffffffffu, w, l);
                b = b0 + l;
            } else {
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (b < 0) {  // the lengths changed under the call
            at = end;
            return;
        }
        cache_seq(p.c, b, len, n);
        h = (int)((at - before) / mine);
        long long rest = (at - before) % mine;
        tile = 0;
        for (int tiles = tiles_of(p, n); tile < tiles; ++tile) {
            const int cost = make_tile(p, len, n, tile).stages + kTcOver;
            if (rest < cost) break;
            rest -= cost;
        }
        place = (int)rest;
    }
    __device__ __forceinline__ bool next(const AttnParams& p, Stretch& s) {
        while (at < end) {
            s.t = make_tile(p, len, n, tile);
            s.b = b;
            s.h = h;
            s.len = len;
            s.n = n;
            const int cost = s.t.stages + kTcOver, span = (int)min((long long)cost - place, end - at);
            if (span <= 0) break;  // the lengths changed under the call
            s.from = max(0, place - kTcOver);
            s.upto = place + span - kTcOver;
            at += span;
            place += span;
            if (place >= cost) {
                place = 0;
                if (++tile >= tiles_of(p, n)) {
                    tile = 0;
                    if (++h >= p.c.H) {
                        h = 0;
                        do {
                            if (++b >= p.c.B) { at = end; break; }
                        } while (!cache_seq(p.c, b, len, n) || n == 0);
                    }
                }
            }
            if (s.upto > s.from) {
                s.whole = s.upto - s.from == s.t.stages;
                s.first = first;
                first = false;
                return true;
            }
        }
        return false;
    }
};

// A tile that several blocks worked on, as its first block leaves it for the second kernel: its rows, the last of the
// blocks (none: -1) and which of the first block's two parts it is.
struct __align__(16) Joint {
    int b, h, n, row0, last, slot, unused[2];
};
__device__ __forceinline__ Joint* joints(const AttnParams& p, int d) {
    return reinterpret_cast<Joint*>(p.part + (size_t)kMaxTcBlocks * 2 * tile_floats(d, kRows));
}

// ------------------------------------------------------------------ shared memory
struct __align__(16) StageMeta {  // read as 16-byte words
    float ks[4], vs[4], lv[4];  // of the four 16-position parts: scales, log2 vs
    int id[4];                  // their pages: -1 out of range, -2 seen by no row
    float top;                  // largest of lv and 0
};
struct Control {
    uint64_t rfull[kRaw], rempty[kRaw], kfull[kKBuffers], kempty[kKBuffers], vfull[kVBuffers], vempty[kVBuffers];
    uint64_t sfull[2], pfull[2], odone[2], qfull, drain[2];
    uint32_t tmem;
    volatile int dead;
    StageMeta meta[kMetas];
};
template <int D> struct Smem {
    static constexpr int tile = kStage * D * 2, codes = kStage * D, k = 0, v = kKBuffers * tile,
                         raw = v + kVBuffers * tile, q = raw + 2 * kRaw * codes,
                         qtile = kHalf * D * 2, control = q + 2 * qtile, bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bytes that the phase waits for, beside its arrivals.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Once for a whole warp, after what its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Bounded wait of a thread; false once it or any other of the block's waits has run out.
__device__ __forceinline__ bool wait_one(Control& ct, uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t k = 1;; ++k) {
        if (mbar_try_wait(bar, parity)) return true;
        if (k & 63) continue;
        if (ct.dead) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > kWaitLimitNs) {
            ct.dead = 1;
            return false;
        }
    }
}
// Of a whole warp.
__device__ __forceinline__ bool wait(Control& ct, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_one(ct, bar, parity));
}
// One lane of a converged warp: the compiler then keeps descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// D[tmem] (+)= A[tmem] B[smem], 16-bit floats (A: a row per lane, two values a column), fp32 accumulator.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 codes as 16-bit floats: two 16-byte chunks.  The four channels of a word come in the order of
// codes_to_half: 0, 2, 1, 3 for int8 codes (queries and outputs follow), 0, 1, 2, 3 for e4m3.
template <bool E4M3>
__device__ __forceinline__ void convert16(const uint4& u, uint4& x, uint4& y) {
    codes_to_half<E4M3>(u.x, x.x, x.y);
    codes_to_half<E4M3>(u.y, x.z, x.w);
    codes_to_half<E4M3>(u.z, y.x, y.y);
    codes_to_half<E4M3>(u.w, y.z, y.w);
}

// ------------------------------------------------------------------ warp 17: copies
// Lane 4 j + g holds page and scales of part g of the j-th of eight stages; the next eight stages'
// are read while these are in use.
template <int D>
__device__ __forceinline__ void copy_pages(const AttnParams& p, uint8_t* smem, Control& ct, Walk walk) {
    const int lane = threadIdx.x & 31, g = lane & 3;
    const int rows = min(p.c.page, kStage), copies = kStage / rows;  // of a stage
    uint32_t n = 0;
    Stretch s;
    s.from = s.upto = s.t.stages = 0;
    if (lane == 0) joints(p, D)[blockIdx.x].last = -1;
    bool ok = true;
    while (ok && walk.next(p, s)) {
        const int stages = s.upto - s.from, base = (s.t.s0 + s.from) * kStage;
        struct Part { int id; float ks, vs; };
        auto lookup = [&](int i) {
            Part x;
            const int part = base + i * kStage + 16 * g;
            x.id = i < stages && part < s.t.hi && part + 16 > s.t.lo ? cache_page(p.c, s.b, part / p.c.page) : -2;
            x.ks = x.vs = x.id == -1 ? __uint_as_float(0x7fc00000u) : 0.f;
            if (x.id >= 0) {
                const size_t ph = (size_t)x.id * p.c.H + s.h;
                x.ks = p.c.k_scale[ph];
                x.vs = p.c.v_scale[ph];
            }
            return x;
        };
        Part now, next = lookup(lane >> 2);
        for (int i = 0; i < stages; ++i, ++n) {
            if ((i & 7) == 0) {
                now = next;
                next = lookup(i + 8 + (lane >> 2));
            }
            const uint32_t buf = n % kRaw, parity = (n / kRaw) & 1;
            ok = wait(ct, &ct.rempty[buf], parity ^ 1);
            if (!ok) break;
            // copy c takes the page of its first part that is seen
            int id = __shfl_sync(0xffffffffu, now.id, 4 * (i & 7) + g);
            if (rows > 16) id = max(id, __shfl_xor_sync(0xffffffffu, id, 1));
            if (rows > 32) id = max(id, __shfl_xor_sync(0xffffffffu, id, 2));
            const int c = lane;  // lane c < copies issues copy c, of parts c * rows / 16 ..
            id = __shfl_sync(0xffffffffu, id, min(c * (rows / 16), 3));
            const bool mine = c < copies && id >= 0;
            const int total = __popc(__ballot_sync(0xffffffffu, mine)) * 2 * rows * D;
            if (lane == 0) mbar_expect_tx(&ct.rfull[buf], total);
            __syncwarp();
            if (mine) {
                const int first = base + i * kStage + c * rows;
                const size_t off = (((size_t)id * p.c.H + s.h) * p.c.page + (first & (p.c.page - 1))) * D;
                uint8_t* to = smem + Smem<D>::raw + buf * 2 * Smem<D>::codes + c * rows * D;
                bulk_g2s(to, p.c.k + off, rows * D, &ct.rfull[buf]);
                bulk_g2s(to + Smem<D>::codes, p.c.v + off, rows * D, &ct.rfull[buf]);
            }
            // the copies are on their way: now the scales
            if ((lane >> 2) == (i & 7)) {
                StageMeta& m = ct.meta[n % kMetas];
                m.ks[g] = now.ks;
                m.vs[g] = now.vs;
                m.lv[g] = now.vs == now.vs ? log2f(now.vs) : 0.f;
                m.id[g] = now.id;
                float top = fmaxf(m.lv[g], 0.f);
                const unsigned four = 15u << (lane & 28);
                top = fmaxf(top, __shfl_xor_sync(four, top, 1));
                m.top = fmaxf(top, __shfl_xor_sync(four, top, 2));
                if (now.id == -1) flag_index_error(p.c);
            }
            warp_arrive(&ct.rfull[buf]);
        }
    }
    // the block's last tile goes on in the next ones
    if (s.from == 0 && s.upto > 0 && s.upto < s.t.stages) {
        const long long total = line_length(p, lane);
        const int used = blocks_used(total, gridDim.x), i = blockIdx.x;
        const long long after = share(total, i + 1, used) - s.upto + s.t.stages;  // the tile's last place + 1
        if (lane == 0 && after <= total)  // (the lengths may have changed under the call)
            joints(p, D)[i] = {s.b, s.h, s.n, s.t.row0, min(holder(total, after - 1, used), used - 1), s.first ? 0 : 1};
    }
    // no copy outlives the block, whatever became of the other warps
    for (uint32_t m = n > kRaw ? n - kRaw : 0; m < n; ++m) mbar_wait(&ct.rfull[m % kRaw], (m / kRaw) & 1, kWaitLimitNs);
}

// ------------------------------------------------------------------ warps 8-15: codes to operand tiles
// Warps 8-11 convert keys, 12-15 values, each a part of 16 positions: 8 rows and a 64-byte
// half row of each at a time; even and odd rows take the other half (d = 128), which keeps reads and
// writes off each other's banks.
template <int D, bool E4M3>
__device__ __forceinline__ void convert_codes(const AttnParams& p, uint8_t* smem, Control& ct, Walk walk) {
    constexpr int IT = D / 64;  // half rows of a row
    const int lane = threadIdx.x & 31, w = (threadIdx.x - kCodeThread0) >> 5;
    const int r8 = lane >> 2, q = lane & 3, part = w & 3;
    const bool keys = w < 4;
    uint64_t* full = keys ? ct.kfull : ct.vfull;
    uint64_t* empty = keys ? ct.kempty : ct.vempty;
    const uint32_t buffers = keys ? kKBuffers : kVBuffers;
    uint8_t* tiles = smem + (keys ? Smem<D>::k : Smem<D>::v);
    const uint8_t* raws = smem + Smem<D>::raw + (keys ? 0 : Smem<D>::codes);
    uint32_t n = 0, buf = 0, parity = 0, rb = 0, rparity = 0;  // stages so far; buffers and their phases
    Stretch s;
    while (walk.next(p, s)) {
        const int end = s.len + s.n, stages = s.upto - s.from, base = (s.t.s0 + s.from) * kStage;
        for (int i = 0; i < stages; ++i, ++n) {
            if (!wait(ct, &ct.rfull[rb], rparity)) return;
            if (!wait(ct, &empty[buf], parity ^ 1)) return;
            const uint8_t* raw = raws + rb * 2 * Smem<D>::codes;
            uint8_t* tile = tiles + buf * Smem<D>::tile;
            // values that hide behind the last position, or were not copied, may be anything: zeros
            // (as keys they make scores that are hidden)
            const int keep = keys ? 16 : ct.meta[n % kMetas].id[part] < 0 ? 0 : end - (base + i * kStage + 16 * part);
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int row = 16 * part + 8 * o + r8, half = IT == 2 ? (row ^ it) & 1 : 0;
                    uint4 u = *reinterpret_cast<const uint4*>(raw + row * D + half * 64 + q * 16);
                    if (8 * o + r8 >= keep) u = make_uint4(0, 0, 0, 0);
                    uint4 x, y;
                    convert16<E4M3>(u, x, y);
                    uint8_t* at = tile + half * kStage * 128 + row * 128;
                    *reinterpret_cast<uint4*>(at + (((2 * q) ^ (row & 7)) << 4)) = x;
                    *reinterpret_cast<uint4*>(at + (((2 * q + 1) ^ (row & 7)) << 4)) = y;
                }
            fence_async_smem();
            warp_arrive(&full[buf]);
            if (lane == 0) mbar_arrive(&ct.rempty[rb]);
            if (++buf == buffers) { buf = 0; parity ^= 1; }
            if (++rb == kRaw) { rb = 0; rparity ^= 1; }
        }
    }
}

// ------------------------------------------------------------------ warps 16 and 18: the products
// A wait, a commit and a switch from one product to the other cost the issuing warp 100 to 250 cycles
// each, so S and O have a warp each, which issues both halves together.
// S = Q K^T of stage n, over the columns of P of stage n - 2: after that P's products.
template <int D>
__device__ __forceinline__ void issue_scores(const AttnParams& p, uint8_t* smem, Control& ct, Walk walk) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    // descriptors of the first buffers; an address step of 16 bytes is 1 in their lowest field
    const uint64_t k0 = desc_kmajor(Tile{base + Smem<D>::k, kStage}, 0);
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kHalf}, 0);
    uint32_t buf = 0, parity = 0, n = 0, tiles = 0;
    Stretch s;
    while (walk.next(p, s)) {
        const int stages = s.upto - s.from;
        if (!wait(ct, &ct.qfull, tiles & 1)) return;
        ++tiles;
        for (int i = 0; i < stages; ++i, ++n) {
            if (!wait(ct, &ct.kfull[buf], parity)) return;
            if (n >= 2 && !wait(ct, &ct.odone[n & 1], ((n - 2) >> 1) & 1)) return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t kd = k0 + buf * (Smem<D>::tile >> 4);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int kk = 0; kk < D; kk += 16)  // 16 channels: 32 bytes of a 128-byte row
                        mma_bf16(tm + s_col(hf, n & 1),
                                 q0 + hf * (Smem<D>::qtile >> 4) + (kk >> 6) * (kHalf * 128 / 16) + (kk & 63) / 8,
                                 kd + (kk >> 6) * (kStage * 128 / 16) + (kk & 63) / 8, idesc_f16(kHalf, kStage, false),
                                 kk > 0);
                mma_commit(&ct.sfull[n & 1]);
                mbar_arrive(&ct.sfull[n & 1]);  // hands on the scales, which came with kfull
                mma_commit(&ct.kempty[buf]);
            }
            __syncwarp();
            if (++buf == kKBuffers) { buf = 0; parity ^= 1; }
        }
    }
}
// O += P V.
template <int D>
__device__ __forceinline__ void issue_values(const AttnParams& p, uint8_t* smem, Control& ct, Walk walk) {
    const uint32_t tm = ct.tmem;
    const uint64_t v0 = desc_mnmajor(Tile{smem_u32(smem) + Smem<D>::v, kStage}, 0);
    uint32_t buf = 0, parity = 0, n = 0;
    Stretch s;
    while (walk.next(p, s)) {
        const int stages = s.upto - s.from;
        for (int i = 0; i < stages; ++i, ++n) {
            if (!wait(ct, &ct.vfull[buf], parity) || !wait(ct, &ct.pfull[n & 1], (n >> 1) & 1)) return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t vd = v0 + buf * (Smem<D>::tile >> 4);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int kk = 0; kk < kStage; kk += 16)  // 16 positions: 16 rows of 128 bytes
                        mma_ts(tm + o_col(hf), tm + s_col(hf, n & 1) + kk / 2, vd + kk * 8, idesc_f16(kHalf, D, true),
                               i > 0 || kk > 0);
                mma_commit(&ct.odone[n & 1]);
                mma_commit(&ct.vempty[buf]);
            }
            __syncwarp();
            if (++buf == kVBuffers) { buf = 0; parity ^= 1; }
        }
    }
}
// Lets what a warp has in flight end before the tensor memory goes.
__device__ __forceinline__ void drain(Control& ct, uint64_t* bar) {
    __syncwarp();
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    mbar_wait(bar, 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ warps 0-7: a row per thread
// Keeps the instructions before and after it apart: a pair's chain of product, powers, sum and conversion is
// long, and two warps a scheduler hide it only where eight pairs take each of its steps together (17 cycles a
// pair and scheduler otherwise, 10 so).
__device__ __forceinline__ void in_order(float2 (&z)[8]) {
    asm volatile("" : "+f"(z[0].x), "+f"(z[0].y), "+f"(z[1].x), "+f"(z[1].y), "+f"(z[2].x), "+f"(z[2].y), "+f"(z[3].x), "+f"(z[3].y),
                 "+f"(z[4].x), "+f"(z[4].y), "+f"(z[5].x), "+f"(z[5].y), "+f"(z[6].x), "+f"(z[6].y), "+f"(z[7].x), "+f"(z[7].y));
}
// The weights of the 64 positions of a stage, to tensor memory as 16-bit operands, and their sum:
// p = 2^(x kf - mref), w = p (2^(m - M + 13) vs).  APART: the rows that
// are `mine` take w as a power of two of its own, 2^(x kf - M + 13 + log2 vs).
template <bool APART>
__device__ __forceinline__ void weigh(uint32_t ts, const float (&x)[4][16], const float (&kf)[4], const float (&vs)[4],
                                      const StageMeta& mt, float mref, float m, float M, bool mine, float2& l2, float2& l3) {
    const float fm = pow2i(m - M + kTcBias), up = M == kNegInf ? 0.f : kTcBias - M;
    const float2 nm = make_float2(-mref, -mref);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float2 f = make_float2(fm * vs[g], fm * vs[g]), k2 = make_float2(kf[g], kf[g]);
        float2 z[8];
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = fma2(make_float2(x[g][2 * j], x[g][2 * j + 1]), k2, nm);
        in_order(z);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = make_float2(ex2(z[j].x), ex2(z[j].y));
        in_order(z);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            l2 = add2(l2, z[j]);
            z[j] = mul2(z[j], f);
            l3 = add2(l3, z[j + 1]);
            z[j + 1] = mul2(z[j + 1], f);
        }
        in_order(z);
        if (APART && mine) {
            const float one = vs[g] == vs[g] ? 1.f : vs[g];  // a NaN marks the page
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[j] = make_float2(ex2(fmaf(x[g][2 * j], kf[g], up + mt.lv[g])) * one,
                                   ex2(fmaf(x[g][2 * j + 1], kf[g], up + mt.lv[g])) * one);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(pack_half(z[j].x, z[j].y));
        __syncwarp();
        tmem_st8(ts + 8 * g, w);
    }
}
// A row's result is its sum times 2^f / l: as two factors, which stay normal numbers where the result is not.
__device__ __forceinline__ float2 row_factors(float f, float l, float M) {
    if (M == kNegInf) return make_float2(l > 0.f ? 0.f : 0.f / l, 1.f);  // no value scale but zeros; no weights
    f = fminf(fmaxf(f, -250.f), 250.f);
    const float half = truncf(0.5f * f);
    return make_float2(pow2i(half) / l, pow2i(f - half));
}
template <int D, bool E4M3>
__device__ __forceinline__ void soften_rows(const AttnParams& p, uint8_t* smem, Control& ct, Walk walk) {
    const int hf = threadIdx.x / kHalf, r = threadIdx.x % kHalf, lane = threadIdx.x & 31;
    const uint32_t tm = warp_lane_base(ct.tmem), to = tm + o_col(hf);
    uint32_t n = 0;  // stages so far
    Stretch s;
    while (walk.next(p, s)) {
        const int stages = s.upto - s.from, row = s.t.row0 + hf * kHalf + r;
        const bool on = row < s.n * p.G;
        const bool some = s.t.row0 + hf * kHalf < s.n * p.G;  // the half has rows
        const int tok = on ? row / p.G : 0, head = s.h * p.G + (on ? row % p.G : 0), pos = on ? s.len + tok : -1;
        // The warp's queries as operand: whole rows at a time, 16 bytes a lane, each row scaled (with the sign
        // of the softmax scale, so that the factors of S are positive).
        const long long at0 = on ? ((long long)s.b * p.c.T + tok) * p.ld_q + (long long)head * D : -1;
        int e = 0;
        {
            constexpr int L = D / 8, R = 32 / L;  // lanes of a row, rows at a time
            const int lr = lane / L, chunk = lane % L;
            uint4 raw[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const long long from = __shfl_sync(0xffffffffu, at0, R * i + lr);
                raw[i] = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + from) + chunk)
                                   : make_uint4(0, 0, 0, 0);
            }
            // Magnitudes of bf16 values order as their bits: the largest of two rows at once, and of this lane's own.
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < L; i += 2) {
                uint32_t top[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 u = raw[i + j];
                    const uint32_t t = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                                __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
                    top[j] = __vmaxu2(t, t >> 16);
                }
                uint32_t two = __byte_perm(top[0], top[1], 0x5410);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
                two = __shfl_sync(0xffffffffu, two, (lane % R) * L);
                if (lane / R == i) mine = two & 0xffffu;
                if (lane / R == i + 1) mine = two >> 16;
            }
            // a power of two to a largest magnitude of 2^9 .. 2^10: a bf16 value stays exact unless it is below
            // 2^-24 of the row's largest
            e = mine > 0 && mine < 0x7f80u ? max((int)(mine >> 7) - 136, -126) : 0;
            const float f = p.scale < 0.f ? -pow2i(-(float)e) : pow2i(-(float)e);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                float x[8];
                const float fi = __shfl_sync(0xffffffffu, f, R * i + lr);
                unpack8(raw[i], x);
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] *= fi;
                constexpr int a = E4M3 ? 1 : 2, b = 3 - a;  // the order of convert16
                const int rr = (threadIdx.x & 96) + R * i + lr;
                *reinterpret_cast<uint4*>(smem + Smem<D>::q + hf * Smem<D>::qtile + (chunk >> 3) * kHalf * 128 + rr * 128 +
                                          (((chunk & 7) ^ (rr & 7)) << 4)) =
                    make_uint4(pack_half(x[0], x[a]), pack_half(x[b], x[3]), pack_half(x[4], x[4 + a]),
                               pack_half(x[4 + b], x[7]));
            }
        }
        fence_async_smem();
        warp_arrive(&ct.qfull);
        const float qs = ldexpf(fabsf(p.scale) * kLog2e, e);
        // positions that every row of the half sees need no mask
        const int t0 = (s.t.row0 + hf * kHalf) / p.G, t1 = min(s.n - 1, (s.t.row0 + hf * kHalf + kHalf - 1) / p.G);
        const int all_hi = s.len + t0 + 1, all_lo = p.window > 0 ? max(0, s.len + t1 - p.window + 1) : 0;
        float l = 0.f, m = kNegInf, M = kNegInf;
        for (int i = 0; i < stages; ++i, ++n) {
            const int first = (s.t.s0 + s.from + i) * kStage;
            const uint32_t ts = tm + s_col(hf, n & 1);
            if (!wait(ct, &ct.sfull[n & 1], (n >> 1) & 1)) return;
            if (!some) {
                warp_arrive(&ct.pfull[n & 1]);
                continue;
            }
            tc_fence_after();
            const StageMeta& mt = ct.meta[n % kMetas];
            const float4 ks4 = *reinterpret_cast<const float4*>(mt.ks), vs4 = *reinterpret_cast<const float4*>(mt.vs);
            const float4 lv4 = *reinterpret_cast<const float4*>(mt.lv);
            float kf[4] = {qs * ks4.x, qs * ks4.y, qs * ks4.z, qs * ks4.w}, vs[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
            const float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w};
            const float sum = (ks4.x + ks4.y) + (ks4.z + ks4.w);
            if (first + kStage > all_hi || first < all_lo || sum != sum) {
                // Hidden positions become -inf in tensor memory, so that the code below knows no mask.  A part
                // whose key scale is NaN makes what it shows NaN; a part that shows nothing weighs nothing, even
                // where its value scale is NaN (in a row that sees some of it everything is NaN anyway).
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float x[16];
                    __syncwarp();
                    tmem_ld16(ts + 16 * g, x);
                    tmem_ld_wait();
                    const bool bad = kf[g] != kf[g];
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int back = pos - (first + 16 * g + j);
                        const bool see = back >= 0 && (p.window == 0 || back < p.window);
                        any |= see;
                        x[j] = see ? (bad ? kf[g] : x[j]) : kNegInf;
                    }
                    if (bad) kf[g] = 1.f;
                    if (!any) vs[g] = 0.f;
                    float a[8], b[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) { a[q] = x[q]; b[q] = x[8 + q]; }
                    tmem_st8(ts + 16 * g, a);
                    tmem_st8(ts + 16 * g + 8, b);
                }
                tmem_st_wait();
            }
            __syncwarp();
            float x[4][16];
#pragma unroll
            for (int g = 0; g < 4; ++g) tmem_ld16(ts + 16 * g, x[g]);
            tmem_ld_wait();
            float mx = kNegInf, need = kNegInf;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float gm = fmaxf(x[g][0], x[g][1]);
#pragma unroll
                for (int j = 2; j < 16; j += 2) gm = fmaxf(gm, fmaxf(x[g][j], x[g][j + 1]));
                kf[g] = fmaxf(kf[g], 1e-37f);  // a zero factor and -inf make no NaN
                gm *= kf[g];
                mx = fmaxf(mx, gm);
                need = fmaxf(need, gm + lv[g]);
            }
            const float m2 = fmaxf(m, ceilf(mx));
            l *= pow2i(m - m2);
            m = m2;
            const bool grow = need > M + kSlack;
            // 2^(m - M + 13) vs of the stage's largest vs (or of 1): too large before M grows, and after it?
            const float most = kMaxFactor - kTcBias - mt.top;
            bool apart = false;
            if (__any_sync(0xffffffffu, grow || m - M > most)) {
                const float up2 = ceilf(need), f = grow ? pow2i(M - up2) : 1.f;
                if (grow) M = up2;
                apart = __any_sync(0xffffffffu, m - M > most);
                if (i > 0) {
                    // O has the product of the stage before
                    if (!wait(ct, &ct.odone[(n - 1) & 1], ((n - 1) >> 1) & 1)) return;
                    tc_fence_after();
#pragma unroll 1
                    for (int j = 0; j < D; j += 32) {
                        float y[2][16];
                        __syncwarp();
                        tmem_ld16(to + j, y[0]);
                        tmem_ld16(to + j + 16, y[1]);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            float a[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) a[q] = y[h >> 1][8 * (h & 1) + q] * f;
                            tmem_st8(to + j + 8 * h, a);
                        }
                    }
                }
            }
            const float mref = m == kNegInf ? 0.f : m;
            float2 l2 = make_float2(0.f, 0.f), l3 = l2;
            if (!apart) weigh<false>(ts, x, kf, vs, mt, mref, m, M, false, l2, l3);
            else weigh<true>(ts, x, kf, vs, mt, mref, m, M, m - M > most, l2, l3);
            l2 = add2(l2, l3);
            l += l2.x + l2.y;
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&ct.pfull[n & 1]);
        }
        // the row leaves
        if (!wait(ct, &ct.odone[(n - 1) & 1], ((n - 1) >> 1) & 1)) return;
        tc_fence_after();
        const int rr = hf * kHalf + r;
        float* part = p.part + ((size_t)blockIdx.x * 2 + (s.first ? 0 : 1)) * tile_floats(D, kRows);
        const size_t at = ((size_t)s.b * p.c.T + tok) * p.Hq + head;
        // sums are in units of 2^(M - 13), l in units of 2^m
        const float2 inv = row_factors(M - m - kTcBias, l, M);
#pragma unroll 2
        for (int j = 0; j < D; j += 16) {
            float y[16];
            __syncwarp();
            tmem_ld16(to + j, y);
            tmem_ld_wait();
            if (!E4M3) {  // back to the order of the channels
#pragma unroll
                for (int q = 0; q < 16; q += 4) {
                    const float z = y[q + 1];
                    y[q + 1] = y[q + 2];
                    y[q + 2] = z;
                }
            }
            if (on && s.whole) {
#pragma unroll
                for (int q = 0; q < 16; ++q) y[q] = y[q] * inv.x * inv.y;
                uint4 u[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    u[q] = make_uint4(pack_bf16(y[8 * q], y[8 * q + 1]), pack_bf16(y[8 * q + 2], y[8 * q + 3]),
                                      pack_bf16(y[8 * q + 4], y[8 * q + 5]), pack_bf16(y[8 * q + 6], y[8 * q + 7]));
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at * D + j);
                o[0] = u[0];
                o[1] = u[1];
            } else if (on) {
                // four channels of all rows side by side, then the next four
                float4* o = reinterpret_cast<float4*>(part) + (j / 4) * kRows + rr;
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q * kRows] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
            }
        }
        tc_fence_before();
        if (on) {
            if (!s.whole) {
                part[kRows * D + rr] = l;
                part[kRows * D + kRows + rr] = m;
                part[kRows * D + 2 * kRows + rr] = M + (kBias - kTcBias);
            } else if (p.lse) {
                p.lse[at] = (m + log2f(l)) * kLn2;
            }
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTcThreads, 1) cache_attn_tc_kernel(const AttnParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<D>::control);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&ct.rfull[i], 1);
            mbar_init(&ct.rempty[i], 8);
        }
        for (int i = 0; i < kKBuffers; ++i) {
            mbar_init(&ct.kfull[i], 4);
            mbar_init(&ct.kempty[i], 1);
        }
        for (int i = 0; i < kVBuffers; ++i) {
            mbar_init(&ct.vfull[i], 4);
            mbar_init(&ct.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.sfull[i], 2);
            mbar_init(&ct.pfull[i], 8);
            mbar_init(&ct.odone[i], 1);
            mbar_init(&ct.drain[i], 1);
        }
        mbar_init(&ct.qfull, 8);
        ct.dead = 0;
        fence_barrier_init();
    }
    chain_wait();
    chain_release();
    Walk walk;
    walk.start(p, threadIdx.x & 31);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        soften_rows<D, E4M3>(p, smem, ct, walk);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < 16) convert_codes<D, E4M3>(p, smem, ct, walk);
        else if (warp == 16) issue_scores<D>(p, smem, ct, walk), drain(ct, &ct.drain[0]);
        else if (warp == 17) copy_pages<D>(p, smem, ct, walk);
        else if (warp == 18) issue_values<D>(p, smem, ct, walk), drain(ct, &ct.drain[1]);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.c.status) *reinterpret_cast<volatile int32_t*>(p.c.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}

// Joins the parts of the tiles that several blocks worked on.  Block x: the tile that the first kernel's block x
// began and others went on with, if any, so that the number of tiles does not matter (a search for it on the
// line took 10 us); y: 32 of its rows, a lane each; warp w takes channels w d/8 .. + d/8 - 1.  Rows of no
// query get zeros (behind a sequence's tokens) or NaN (a sequence out of range).
template <int D>
__global__ void __launch_bounds__(256) cache_attn_tc_join_kernel(const AttnParams p) {
    constexpr int V = D / 32;  // float4s of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch0 = warp * (D / 8);
    // The first kernel's blocks released this one after their own wait: what they read may be read.  Its
    // parts are there after chain_wait(), which every thread comes to, so that the end of this kernel is
    // also the end of the first.
    const long long tokens = (long long)p.c.B * p.c.T;
    for (long long t = (blockIdx.y * gridDim.x + blockIdx.x) * 8 + warp; t < tokens; t += gridDim.x * gridDim.y * 8) {
        int len, n;
        const bool ok = cache_seq(p.c, (int)(t / p.c.T), len, n);
        if (!ok && lane == 0) flag_index_error(p.c);
        if (ok && t % p.c.T < n) continue;
        const uint32_t bad = ok ? 0u : 0x7fc07fc0u;
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + t * p.Hq * D);
        for (int j = lane; j < p.Hq * D / 8; j += 32) o[j] = make_uint4(bad, bad, bad, bad);
        if (p.lse)
            for (int j = lane; j < p.Hq; j += 32) p.lse[t * p.Hq + j] = ok ? kNegInf : __uint_as_float(0x7fc00000u);
    }
    chain_wait();
    chain_release();
    const int first = blockIdx.x;
    const Joint j0 = joints(p, D)[first];
    if (j0.last <= first) return;  // its last tile was finished by it, or is another's to join
    const int b = j0.b, h = j0.h, n = j0.n, last = j0.last, slot = j0.slot;
    const int r = blockIdx.y * 32 + lane, row = j0.row0 + r;
    if (row >= n * p.G) return;
    float m = kNegInf, M = kNegInf, l = 0.f;
    float4 sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    // a part without weight adds nothing, one that met a NaN hands it on
    auto add = [](float& x, float fx, float y, float fy) { x = (x == x ? x * fx : x) + (y == y ? y * fy : y); };
#pragma unroll 2
    for (int i = first; i <= last; ++i) {
        const float* in = p.part + ((size_t)i * 2 + (i == first ? slot : 0)) * tile_floats(D, kRows);
        float4 y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = reinterpret_cast<const float4*>(in)[(ch0 / 4 + j) * kRows + r];
        const float pl = in[kRows * D + r], pm = in[kRows * D + kRows + r], pM = in[kRows * D + 2 * kRows + r];
        const float m2 = fmaxf(m, pm), M2 = fmaxf(M, pM);
        const float s1 = pow2i(M - M2), s2 = pow2i(pM - M2);
        add(l, pow2i(m - m2), pl, pow2i(pm - m2));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            add(sum[j].x, s1, y[j].x, s2);
            add(sum[j].y, s1, y[j].y, s2);
            add(sum[j].z, s1, y[j].z, s2);
            add(sum[j].w, s1, y[j].w, s2);
        }
        m = m2;
        M = M2;
    }
    const float2 inv = row_factors(M - m - kBias, l, M);
    const size_t at = ((size_t)b * p.c.T + row / p.G) * p.Hq + h * p.G + row % p.G;
    uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + ch0);
#pragma unroll
    for (int j = 0; j < V; ++j)
        sum[j] = make_float4(sum[j].x * inv.x * inv.y, sum[j].y * inv.x * inv.y, sum[j].z * inv.x * inv.y, sum[j].w * inv.x * inv.y);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const uint4 u = make_uint4(pack_bf16(sum[j].x, sum[j].y), pack_bf16(sum[j].z, sum[j].w),
                                   pack_bf16(sum[j + 1].x, sum[j + 1].y),
                                   pack_bf16(sum[j + 1].z, sum[j + 1].w));
        *reinterpret_cast<uint4*>(o + j) = u;
    }
    if (warp == 0 && p.lse) p.lse[at] = (m + log2f(l)) * kLn2;
}

template <int D, bool E4M3>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    constexpr int smem = Smem<D>::bytes;
    // the split of the registers must not ask for more than the block is launched with: it would wait for them
    static const bool fits = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, cache_attn_tc_kernel<D, E4M3>) == cudaSuccess && a.numRegs == kRegs;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = set_smem_once(cache_attn_tc_kernel<D, E4M3>, smem, ready); e != cudaSuccess) return e;
    const int blocks = kMaxTcBlocks;
    {
        TraceScope ts("cache_attn_tc", st);
        if (cudaError_t e = launch_chained(cache_attn_tc_kernel<D, E4M3>, dim3(blocks), kTcThreads, smem, st, p);
            e != cudaSuccess)
            return e;
    }
    TraceScope ts("cache_attn_tc_join", st);
    return launch_chained(cache_attn_tc_join_kernel<D>, dim3(blocks, kRows / 32), 256, 0, st, p);
}

}  // namespace

size_t cache_attn_tc_bytes(int d) { return (size_t)kMaxTcBlocks * (2 * tile_floats(d, kRows) * sizeof(float) + sizeof(Joint)); }

cudaError_t cache_attn_tc(const AttnParams& p, cudaStream_t st) {
    if (p.c.code == DR_CODE_E4M3) return p.c.d == 128 ? launch<128, true>(p, st) : launch<64, true>(p, st);
    return p.c.d == 128 ? launch<128, false>(p, st) : launch<64, false>(p, st);
}

}  // namespace dr
