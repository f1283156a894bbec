// paged_join.cu -- joins the partial sums of the units that the paged
// attention cut between blocks (paged.cuh).
//
// The pieces of a unit, in the order of its keys, hold m_k (the running maximum
// in powers of two), l_k and A_k = sum_j 2^(s_j - m_k) v_j; with m = max m_k
//   O = sum_k 2^(m_k - m) A_k / sum_k 2^(m_k - m) l_k,
// in float32, rounded once.  Of the unit that ends in block c and begins in c0,
// block c0 holds the first piece (its slot 1: it begins the unit), blocks c0 +
// 1 .. c the others (slot 0).  At most one unit ends so in each block.  A warp
// takes a row or two.  Bounded by the latency of its reads, one after the other
// (the unit, its rows, the pieces' sums, the pieces, which are in L2): with eight
// rows to a warp it took 20 us for 148 units of 256 rows.  A unit of which a block
// gave up is not joined: what that block left in the workspace is not its piece.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace wildcat {

namespace {

using namespace paged;
constexpr int kJoinThreads = 256, kJoinRows = 2;  // rows of a warp

template <typename E, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedJoin a, int M) {
    using T = typename E::T;
    // the attention's grid has finished, and its writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const int4 j = a.p.joins[c];
    if (j.w < 0) return;  // kNoJoin or kGaveUp
    const int c0 = j.w, pieces = c - c0 + 1;
    const int n = a.s.new_tokens(j.x), first = a.s.first_row(j.x);
    const int64_t row0 = (int64_t)j.z * a.s.M;
    const int rows = (int)min((int64_t)a.s.M, (int64_t)n * a.s.g - row0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int W = D / 32;
    for (int r = blockIdx.y * (kJoinThreads / 32) + warp; r < rows; r += gridDim.y * (kJoinThreads / 32)) {
        float m = -INFINITY;
        float2 mine = make_float2(-INFINITY, 0.f);  // of piece `lane`
        bool lost = false;
        for (int k = lane; k < pieces; k += 32) {
            const float2 ml = a.p.ml[((int64_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * M + r];
            lost = lost || a.p.joins[c0 + k].w == kGaveUp;
            if (k < 32) mine = ml;
            m = fmaxf(m, ml.x);
        }
        if (__any_sync(0xffffffffu, lost)) return;
        m = warp_max(m);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc[W];
#pragma unroll
        for (int x = 0; x < W; ++x) acc[x] = 0.f;
#pragma unroll 4
        for (int k = 0; k < pieces; ++k) {
            const int64_t at = ((int64_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * M + r;
            float2 ml = make_float2(__shfl_sync(0xffffffffu, mine.x, k & 31), __shfl_sync(0xffffffffu, mine.y, k & 31));
            if (k >= 32) ml = a.p.ml[at];
            const float f = exp2f(ml.x - base);
            l = fmaf(f, ml.y, l);
            const float* src = a.p.part + at * D + lane * W;
            float v[W];
            if constexpr (W == 4) {
                const float4 u = *reinterpret_cast<const float4*>(src);
                v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
            } else if constexpr (W == 2) {
                const float2 u = *reinterpret_cast<const float2*>(src);
                v[0] = u.x; v[1] = u.y;
            } else {
                v[0] = *src;
            }
#pragma unroll
            for (int x = 0; x < W; ++x) acc[x] = fmaf(f, v[x], acc[x]);
        }
        const int i = (int)((row0 + r) / a.s.g), hq = j.y * a.s.g + (int)(row0 + r - (int64_t)i * a.s.g);
        const float rcp = l > 0.f || l != l ? 1.f / l : 0.f;
        T* o = static_cast<T*>(a.O) + (int64_t)(first + i) * a.o_t + (int64_t)hq * a.o_h + lane * W;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            if constexpr (sizeof(T) == 4) o[x] = acc[x] * rcp;
            else o[x] = __float2bfloat16_rn(acc[x] * rcp);
        }
        if (a.lse && lane == 0)
            a.lse[(int64_t)(first + i) * (a.s.Hkv * a.s.g) + hq] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <typename E, int D>
Status run_join(const PagedJoin& a, int M, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.G, (unsigned)(M / (kJoinRows * kJoinThreads / 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, paged_join_kernel<E, D>, a, M);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend: join launch");
    return Status::ok();
}

}  // namespace

Status launch_paged_join(const PagedJoin& a, int dtype, int d, int M, cudaStream_t st) {
    const bool bf = dtype == 1;
    switch (d) {
        case 32: return bf ? run_join<BF16, 32>(a, M, st) : run_join<F32, 32>(a, M, st);
        case 64: return bf ? run_join<BF16, 64>(a, M, st) : run_join<F32, 64>(a, M, st);
        case 128: return bf ? run_join<BF16, 128>(a, M, st) : run_join<F32, 128>(a, M, st);
    }
    return Status::fail(2, "paged_attend: unsupported head dim");
}

}  // namespace wildcat
