// tc_block.cuh -- what the tensor-core kernels over whole prompts share: bounded waits of a block whose warps
// have different tasks, operand products from tensor memory, 32-column accesses of tensor memory, and tensor
// maps of rows of heads.
#pragma once
#include <cudaTypedefs.h>

#include "common.cuh"
#include "tc.cuh"

namespace dr {
namespace {

using namespace tc;

// ------------------------------------------------------------------ barriers
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Once for a whole warp, after what its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Bounded wait of a thread; false once it or any other of the block's waits has run out.
__device__ __forceinline__ bool wait_one(volatile int& dead, uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t k = 1;; ++k) {
        if (mbar_try_wait(bar, parity)) return true;
        if (k & 63) continue;
        if (dead) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > kWaitLimitNs) {
            dead = 1;
            return false;
        }
    }
}
// Of a whole warp.
__device__ __forceinline__ bool wait(volatile int& dead, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_one(dead, bar, parity));
}
// One lane of a converged warp: the compiler then keeps descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// Lets what a warp has in flight on the tensor cores end before the tensor memory goes.
__device__ __forceinline__ void drain(uint64_t* bar) {
    __syncwarp();
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    mbar_wait(bar, 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ tensor memory
// D[tmem] (+)= A[tmem] B[smem], bf16 (A: a row per lane, two values a column), fp32 accumulator.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 consecutive columns of the warp's 32 lanes (thread t: lane warp_base + t).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ------------------------------------------------------------------ tiles
// R rows of a head as an SW128 tile: a box for each 64 channels.
template <int R, int D>
__device__ __forceinline__ void load_rows(uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int head, int row) {
#pragma unroll
    for (int c = 0; c < D; c += 64) tma_load_3d(tile + (c / 64) * R * 128, map, bar, c, head, row);
}
// Zeros in the rows n .. R - 1 of such a tile; a whole warp, ordered before what it signals next.
template <int R, int D> __device__ __forceinline__ void clear_rows(uint8_t* tile, int n) {
    const int lane = threadIdx.x & 31;
    for (int c = 0; c < D / 64; ++c)
        for (int i = n * 8 + lane; i < R * 8; i += 32)
            *reinterpret_cast<uint4*>(tile + c * R * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
}

// Counts through the phases of a ring of buffers.
template <int N> struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) { at = 0; phase ^= 1; }
    }
};
// Before a block ends no copy of it may be on its way, whatever became of its warps: waits, with a limit, for the last
// phase of each buffer that was filled (what was never filled is not waited for).
template <int N> __device__ __forceinline__ void settle(const Ring<N>& ring, uint64_t (&full)[N]) {
    for (uint32_t b = 0; b < N; ++b) mbar_wait(&full[b], b < ring.at ? ring.phase : ring.phase ^ 1, kWaitLimitNs);
}
// The same for a barrier that `n` copies went through one after another.
__device__ __forceinline__ void settle(uint64_t* full, long long n) { mbar_wait(full, (uint32_t)(n & 1) ^ 1, kWaitLimitNs); }

// ------------------------------------------------------------------ host
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}
// The encoder is a call of the driver and wants a current context, which a host thread has from its first call of the
// runtime that needs one: once for each thread and device.
inline bool thread_context() {
    static thread_local int bound = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev != bound && cudaSetDevice(dev) != cudaSuccess) return false;
    bound = dev;
    return true;
}
// `rows` token rows of H heads of D bf16 values, ld elements apart; boxes of 64 channels of one head of R rows.
inline bool head_rows_map(CUtensorMap* m, const void* ptr, int D, int H, long long rows, long long ld, int R) {
    auto enc = tensor_map_encoder();
    if (!enc || !thread_context()) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)R};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

}  // namespace
}  // namespace dr
