// sm100.cuh -- thin inline-PTX wrappers for the Blackwell (sm_100 family)
// features the kernels use: mbarriers, TMA tensor copies, tcgen05 tensor-core
// MMAs with tensor-memory accumulators, and bounded waits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dspark {

// Host side: a tiled tensor map of rank 1 to 3 (draft_tc.cu); false if the
// driver refuses it.
bool make_tensor_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
                     const cuuint64_t* strides_bytes, const cuuint32_t* box,
                     CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B);

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// True for one lane of the (converged) warp, the same one every time.  The
// compiler knows the branch to be taken by a single thread; behind a plain
// comparison of the lane number it loops over the active lanes for every
// instruction that takes uniform registers (TMA copies, tensor-core MMAs and
// their commits), about 70 cycles each.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// SM cycle counter: monotonic on the SM that reads it, unlike the global
// nanosecond timer, which the driver may adjust (a forward step during a
// wait would end it early).  Every wait limit below is in these cycles.
__device__ __forceinline__ uint64_t sm_cycles() { return clock64(); }

__device__ __forceinline__ uint32_t ld_relaxed_gpu(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Packed pairs of float32 (one instruction for two values).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2x(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Per-CTA state of the bounded waits, in shared memory: the limit (SM
// cycles; from the workspace header, 2^32 = 2 to 4 s at 2 to 1 GHz unless a
// caller set another) and the abort flag that the first thread whose wait ran
// out raises, so that every later wait of the CTA gives up at once.
struct WaitState {
    int abort;
    int pad;
    uint64_t limit;
};
constexpr uint64_t kWaitLimitCycles = 1ull << 32;   // the default limit

// Wait for the phase of `bar` with the given parity to complete.  Gives up
// after w->limit SM cycles (or at once when another thread of the CTA
// already gave up) and returns false; the caller then winds down without
// touching the pipeline.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile WaitState* w) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = sm_cycles();
    const uint64_t limit = w->limit;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0) {
            if (w->abort) return false;
            if (sm_cycles() - t0 > limit) {
                w->abort = 1;
                return false;
            }
        }
    }
}

// mbar_wait in few instructions, of which there are many: the first try in
// place, the rest in one function.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile WaitState* w) {
    const uint64_t t0 = sm_cycles();
    do {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
    } while (!w->abort && sm_cycles() - t0 <= w->limit);
    w->abort = 1;
    return false;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile WaitState* w) {
    return mbar_test(bar, parity) || wait_on(smem_u32(bar), parity, w);
}

// Sums over the 32 lanes of the first N = 8, 16 or 32 values per lane; lane i
// gets the sum of value i % N.  (Each exchange halves the values; what is left
// of the lanes is summed for one value.)
template <int N>
__device__ __forceinline__ float lane_sums(float* x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
#pragma unroll
    for (int o = N; o < 32; o <<= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    return x[0];
}

// The same all in place and with a first try that may suspend the thread: about
// 110 cycles from arrival to return, against 270 through the function, and no
// call (registers cannot be moved between warpgroups around one).
__device__ __forceinline__ bool wait_bar_here(uint64_t* bar, uint32_t parity, volatile WaitState* w) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = sm_cycles();
    do {
        if (mbar_try_wait(bar, parity)) return true;
    } while (!w->abort && sm_cycles() - t0 <= w->limit);
    w->abort = 1;
    return false;
}

// Bounded wait that ignores the abort flag (used to drain copies in flight
// after an abort).
__device__ __forceinline__ bool mbar_wait_for(uint64_t* bar, uint32_t parity, uint64_t limit_cycles) {
    const uint64_t t0 = sm_cycles();
    while (!mbar_try_wait(bar, parity))
        if (sm_cycles() - t0 > limit_cycles) return false;
    return true;
}

// Spin for about a millisecond (2^21 SM cycles).
__device__ __forceinline__ void spin_about_1ms() {
    const uint64_t t0 = sm_cycles();
    while (sm_cycles() - t0 < (1ull << 21)) {
    }
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t policy_evict_last() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}

// 2-d tile copy delivered to the same shared-memory offset of every CTA in
// `cta_mask` (this cluster); each destination's mbarrier at the offset of
// `bar` receives the bytes that land in that CTA.
// The CTA mask is narrowed to .b16 inside the asm; callers pass a
// compile-time constant (see umma_commit_mc).
__device__ __forceinline__ void tma_load_2d_mc(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                               uint32_t cta_mask, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .b16 msk;\n\tcvt.u16.u32 msk, %5;\n\t"
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], msk, %6;\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(cta_mask), "l"(policy)
        : "memory");
}

// Order this thread's generic shared-memory accesses before later accesses
// of the asynchronous proxy (TMA, tcgen05 operands).
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barrier of `threads` threads (whole warps) of the CTA, numbered 1..15.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, returning whether any of them brings a true `pred`.
__device__ __forceinline__ bool named_any(int id, int threads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(pred ? 1u : 0u)
        : "memory");
    return r != 0;
}
// Largest value of the warp's lanes (NaN only if every lane's is).
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// ---------------------------------------------------------------- cp.async
// 16-byte global -> shared copy that reads `src_bytes` (16 or 0) bytes and
// fills the rest of the 16 with zeros (0: nothing is read, src may be any
// valid address), with an L2 cache policy (createpolicy).
__device__ __forceinline__ void cp_async16_zf(void* dst, const void* src, uint32_t src_bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(src_bytes), "l"(policy)
                 : "memory");
}
// The same without a cache policy.
__device__ __forceinline__ void cp_async16_zf(void* dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(src_bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrive on `bar` once every cp.async this thread issued so far has landed
// (the barrier's count includes this arrival).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t* holder, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory matrix descriptor (tcgen05 format): start address, leading
// and stride byte offsets (16-byte units), descriptor version 1 (bits 46-47),
// base offset 0, layout 128-byte swizzle (value 2 in bits 61-63).
__device__ __forceinline__ uint64_t smem_desc_sw128(const void* p, uint32_t lbo, uint32_t sbo) {
    const uint64_t addr = smem_u32(p);
    return ((addr >> 4) & 0x3FFFull) | (((uint64_t)(lbo >> 4) & 0x3FFFull) << 16) |
           (((uint64_t)(sbo >> 4) & 0x3FFFull) << 32) | (1ull << 46) | (2ull << 61);
}

// The same without swizzle (layout value 0): 8 x 16-byte core matrices of 128
// contiguous bytes.  For an MN-major operand (16-bit values) a core matrix is
// 8 MN values by 8 K; lbo is the distance from one 8-row K group to the next,
// sbo from one group of 8 MN values to the next.
__device__ __forceinline__ uint64_t smem_desc_plain(const void* p, uint32_t lbo, uint32_t sbo) {
    const uint64_t addr = smem_u32(p);
    return ((addr >> 4) & 0x3FFFull) | (((uint64_t)(lbo >> 4) & 0x3FFFull) << 16) |
           (((uint64_t)(sbo >> 4) & 0x3FFFull) << 32) | (1ull << 46);
}

// The same for rows of 64 bytes (64-byte swizzle, layout value 4).
__device__ __forceinline__ uint64_t smem_desc_sw64(const void* p, uint32_t lbo, uint32_t sbo) {
    return smem_desc_plain(p, lbo, sbo) | (4ull << 61);
}

// Instruction descriptor of kind::f16: f32 accumulate, bf16 A and B,
// A K-major, B given by b_mn_major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// Same with A's major-ness in bit 15 (1: MN-major).
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return idesc_bf16_f32(M, N, b_mn_major) | ((a_mn_major ? 1u : 0u) << 15);
}

__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same for fp16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}
// kind::f8f6f4: e4m3 A and B (format value 0), both K-major, f32 accumulate;
// one MMA takes K = 32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Same with the A operand in tensor memory: `a_tmem` addresses 128 lanes
// (row m in lane m) by 8 columns of K = 16 bf16 values, two per column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Arrive once on the mbarrier at the offset of `bar` in every CTA of
// `cta_mask` when this thread's tensor-core operations issued so far complete.
// Callers pass a compile-time constant mask (the cluster size is a template
// parameter of every kernel that multicasts).  In one build of the draft sweep
// whose MMA loop had a run-time trip count, a mask computed at run time (its
// value checked in the kernel: all CTAs of the cluster) left the issuing CTA's
// own barrier without its arrival on every stage, while its peer received
// one; the same kernel with a constant mask completed.
__device__ __forceinline__ void umma_commit_mc(uint64_t* bar, uint32_t cta_mask) {
    asm volatile(
        "{\n\t.reg .b16 msk;\n\tcvt.u16.u32 msk, %1;\n\t"
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], msk;\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(cta_mask)
        : "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA in the cluster (a plain block barrier as well).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 32 lanes x 32 consecutive 32-bit columns: thread i of the warp gets the
// 32 columns of TMEM lane (warp quarter * 32 + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Store 8 consecutive 32-bit columns of this thread's TMEM lane (warp
// quarter * 32 + lane); complete with tmem_st_wait().
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Store 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// N = 4, 8, 16 or 32 consecutive 32-bit columns of this thread's lane, usable on
// return: the registers are operands of the wait, so that no use of them can
// be scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float (&v)[N]) {
    static_assert(N == 4 || N == 8 || N == 16 || N == 32, "column counts in use");
    if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]) ::"memory");
    }
    if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0 % N]), "=f"(v[1 % N]), "=f"(v[2 % N]), "=f"(v[3 % N]), "=f"(v[4 %
                       N]), "=f"(v[5 % N]), "=f"(v[6 % N]), "=f"(v[7 % N])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0 % N]), "+f"(v[1 % N]), "+f"(v[2 % N]), "+f"(v[3 % N]), "+f"(v[4 %
                       N]), "+f"(v[5 % N]), "+f"(v[6 % N]), "+f"(v[7 % N]) ::"memory");
    }
    if constexpr (N == 16) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=f"(v[0 % N]), "=f"(v[1 % N]), "=f"(v[2 % N]), "=f"(v[3 % N]), "=f"(v[4 %
                       N]), "=f"(v[5 % N]), "=f"(v[6 % N]), "=f"(v[7 % N]), "=f"(v[8 % N]), "=f"(v[9
                       % N]), "=f"(v[10 % N]), "=f"(v[11 % N]), "=f"(v[12 % N]), "=f"(v[13 % N]),
                       "=f"(v[14 % N]), "=f"(v[15 % N])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0 % N]), "+f"(v[1 % N]), "+f"(v[2 % N]), "+f"(v[3 % N]), "+f"(v[4 %
                       N]), "+f"(v[5 % N]), "+f"(v[6 % N]), "+f"(v[7 % N]), "+f"(v[8 % N]), "+f"(v[9
                       % N]), "+f"(v[10 % N]), "+f"(v[11 % N]), "+f"(v[12 % N]), "+f"(v[13 % N]),
                       "+f"(v[14 % N]), "+f"(v[15 % N]) ::"memory");
    }
    if constexpr (N == 32) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                     : "=f"(v[0 % N]), "=f"(v[1 % N]), "=f"(v[2 % N]), "=f"(v[3 % N]), "=f"(v[4 %
                       N]), "=f"(v[5 % N]), "=f"(v[6 % N]), "=f"(v[7 % N]), "=f"(v[8 % N]), "=f"(v[9
                       % N]), "=f"(v[10 % N]), "=f"(v[11 % N]), "=f"(v[12 % N]), "=f"(v[13 % N]),
                       "=f"(v[14 % N]), "=f"(v[15 % N]), "=f"(v[16 % N]), "=f"(v[17 % N]), "=f"(v[18
                       % N]), "=f"(v[19 % N]), "=f"(v[20 % N]), "=f"(v[21 % N]), "=f"(v[22 % N]),
                       "=f"(v[23 % N]), "=f"(v[24 % N]), "=f"(v[25 % N]), "=f"(v[26 % N]), "=f"(v[27
                       % N]), "=f"(v[28 % N]), "=f"(v[29 % N]), "=f"(v[30 % N]), "=f"(v[31 % N])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0 % N]), "+f"(v[1 % N]), "+f"(v[2 % N]), "+f"(v[3 % N]), "+f"(v[4 %
                       N]), "+f"(v[5 % N]), "+f"(v[6 % N]), "+f"(v[7 % N]), "+f"(v[8 % N]), "+f"(v[9
                       % N]), "+f"(v[10 % N]), "+f"(v[11 % N]), "+f"(v[12 % N]), "+f"(v[13 % N]),
                       "+f"(v[14 % N]), "+f"(v[15 % N]), "+f"(v[16 % N]), "+f"(v[17 % N]), "+f"(v[18
                       % N]), "+f"(v[19 % N]), "+f"(v[20 % N]), "+f"(v[21 % N]), "+f"(v[22 % N]),
                       "+f"(v[23 % N]), "+f"(v[24 % N]), "+f"(v[25 % N]), "+f"(v[26 % N]), "+f"(v[27
                       % N]), "+f"(v[28 % N]), "+f"(v[29 % N]), "+f"(v[30 % N]), "+f"(v[31 % N]) ::"memory");
    }
}

// Registers per thread of the calling warpgroup (all its warps make the call).
// A launch has its threads times its registers in all; shares that add up to
// no more than that never wait.
template <int N>
__device__ __forceinline__ void regs_raise() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_lower() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace dspark
