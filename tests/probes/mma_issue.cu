// Probe of how the code that issues tcgen05.mma bounds its rate (measurement,
// not a test of the method): one thread per SM issues 32 back-to-back GEMMs of 8
// 128 x 128 x 16 bf16 instructions.  The thread is picked by a comparison of its
// number or by elect.sync in a whole warp, and the form is an argument of the
// kernel, as in mma_rate.cu, or fixed when it is compiled.  Forms: both operands
// in shared memory (SS), A in tensor memory (TS), and the two in turn.  Operands in shared memory are zeros (64 KB of a 120 KB
// buffer, so one CTA per SM), A in tensor memory and all results are not read;
// D takes columns 0-127 and 256-383, A in tensor memory 384-447 of the 512
// allocated.  The one wait is bounded.
#include <cstdio>
#include <cstdint>
#include <cuda_runtime.h>
#include "../../nystr_coreset_approximate_b200/csrc/tc_common.cuh"
using namespace wildcat::tc;

constexpr int G = 32;
__device__ long long g_cycles[148];
__device__ int g_ok[148];

__device__ __forceinline__ void gemm(int form, int g, unsigned tm, uint32_t a_lo, uint32_t b_lo, uint32_t hi) {
    const bool ss = form == 0 || (form == 2 && (g & 1) == 0);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        const uint32_t o = (uint32_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
        if (ss) mma_bf16_w(tm + 256, a_lo + o, hi, b_lo + o, hi, idesc_bf16(128, 128), kk > 0);
        else mma_bf16_ts_w(tm, tm + 384 + kk * 8, b_lo + o, hi, idesc_bf16(128, 128), kk > 0);
    }
}

template <bool ELECT, int FIXED>
__global__ void __launch_bounds__(128, 1) probe(int argument) {
    const int form = FIXED >= 0 ? FIXED : argument;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ uint64_t bar;
    __shared__ unsigned tbase;
    const int tid = threadIdx.x, warp = tid >> 5;
    unsigned char* op = sm + ((1024u - (smem_u32(sm) & 1023u)) & 1023u);
    for (int i = tid; i < 65536 / 16; i += 128) reinterpret_cast<int4*>(op)[i] = make_int4(0, 0, 0, 0);
    if (tid == 0) {
        mbar_init(&bar, 1);
        g_ok[blockIdx.x] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tbase)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tm = tbase;
    const uint64_t da = umma_desc(smem_u32(op)), db = umma_desc(smem_u32(op) + 32768);
    const uint32_t hi = (uint32_t)(da >> 32);
    const long long t0 = clock64();
    if constexpr (ELECT) {
        if (warp == 0) {
            if (elect_one()) {
                for (int g = 0; g < G; ++g) gemm(form, g, tm, (uint32_t)da, (uint32_t)db, hi);
                mma_commit(&bar);
            }
            __syncwarp();
        }
    } else if (tid == 0) {
        for (int g = 0; g < G; ++g) gemm(form, g, tm, (uint32_t)da, (uint32_t)db, hi);
        mma_commit(&bar);
    }
    if (tid == 0) {
        g_ok[blockIdx.x] = mbar_wait(&bar, 0, 100000000ull) ? 1 : 0;
        g_cycles[blockIdx.x] = clock64() - t0;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
    }
}

template <bool ELECT, int FIXED>
bool run(int form) {
    static const char* names[3] = {"SS", "TS", "alternating"};
    cudaError_t e = cudaFuncSetAttribute(probe<ELECT, FIXED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 120 * 1024);
    for (int rep = 0; rep < 2 && e == cudaSuccess; ++rep) {
        probe<ELECT, FIXED><<<148, 128, 120 * 1024>>>(form);
        e = cudaDeviceSynchronize();
    }
    if (e != cudaSuccess) {
        printf("error %s\n", cudaGetErrorString(e));
        return false;
    }
    long long cycles[148];
    int ok[148], n = 0;
    cudaMemcpyFromSymbol(cycles, g_cycles, sizeof(cycles));
    cudaMemcpyFromSymbol(ok, g_ok, sizeof(ok));
    for (int i = 0; i < 148; ++i) n += ok[i];
    printf("%-10s form %-8s %-12s ok=%d %.1f cycles per MMA\n", ELECT ? "elect.sync" : "tid == 0", FIXED >= 0 ? "fixed" : "argument",
           names[form], n, (double)cycles[0] / (G * 8));
    return true;
}

template <bool ELECT>
bool all() {
    for (int form = 0; form < 3; ++form)
        if (!run<ELECT, -1>(form)) return false;
    return run<ELECT, 0>(0) && run<ELECT, 1>(1) && run<ELECT, 2>(2);
}

int main() { return all<false>() && all<true>() ? 0 : 1; }
