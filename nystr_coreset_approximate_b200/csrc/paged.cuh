// paged.cuh -- how the paged attention's work is cut, shared by its kernels.
//
// A unit is (request b, key head h, row tile t): `rows` consecutive rows of
// the request's n * g query rows of that key head (row r = token r / g, query
// head h * g + r % g), M at most.  Its keys come in tiles of N.  All units'
// key tiles stand in one line, requests first, then heads, row tiles and keys;
// block c of G takes the tiles [c T / G, (c + 1) T / G) of the T in all.  Every
// block so has the same number of key tiles whatever the lengths are: one long
// request is spread over the GPU, and many short ones are packed.  A unit that
// lies whole in one block is finished there; of one that is cut, each block
// leaves a partial sum, and join_kernel joins them in the order of the keys,
// the same in every run.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace wildcat {
namespace paged {

struct Plan {
    int64_t* prefix;    // [B + 1] key tiles before request b
    int64_t* per_head;  // [B] key tiles of one key head of request b
    int4* joins;        // [G] the cut unit that ends in block c: (b, h, t, first block), first block -1 for none
    float* part;        // [2 G][M][D] partial sums of the exponentials times V
    float2* ml;         // [2 G][M] their maximum (of beta s, in powers of two) and sum
};

inline size_t carve_plan(Carve& cv, Plan* p, int64_t B, int G, int M, int D) {
    p->prefix = static_cast<int64_t*>(cv.take(sizeof(int64_t) * (B + 1)));
    p->per_head = static_cast<int64_t*>(cv.take(sizeof(int64_t) * (B + 1)));
    p->joins = static_cast<int4*>(cv.take(sizeof(int4) * G));
    p->ml = static_cast<float2*>(cv.take(sizeof(float2) * 2 * G * M));
    p->part = static_cast<float*>(cv.take(sizeof(float) * 2 * G * (size_t)M * D));
    return cv.used;
}

// What the kernels know of the call.
struct Shape {
    const int32_t* table;
    int64_t table_stride, W;
    const int32_t* seq_lens;
    const int32_t* cu_new;
    int64_t T, pages;
    int B, Hkv, g, page_size, M;
    bool causal;

    __device__ __forceinline__ int first_row(int b) const {
        return (int)min(max((int64_t)cu_new[b], (int64_t)0), T);
    }
    __device__ __forceinline__ int new_tokens(int b) const { return max(first_row(b + 1) - first_row(b), 0); }
    // a length past the table's pages is cut to them (and reported by the plan); so is one
    // whose last key tile would end past 2^31
    __device__ __forceinline__ int64_t most() const { return min(W * page_size, (int64_t)0x7fffff00); }
    __device__ __forceinline__ int length(int b) const { return (int)min((int64_t)max(seq_lens[b], 0), most()); }
};

// Key tiles of row tile t (at least one: rows that see nothing are written too).
template <int N>
__device__ __forceinline__ int unit_tiles(int M, int n, int L, int g, bool causal, int64_t t) {
    int end = L;
    if (causal) {
        const int64_t last = min((t * M + M - 1) / g, (int64_t)n - 1);  // the tile's last token
        end = (int)max((int64_t)L - n + last + 1, (int64_t)0);
    }
    return max((end + N - 1) / N, 1);
}

struct Seg {
    int b, h, n, L, row0, rows;  // row0: first row of the unit among the request's n * g
    int t, nt, t0, t1;           // key tiles [t0, t1) of the unit's nt
    int64_t unit_start;          // place of the unit's first tile in the line
};

// The segments of one block, in order.
template <int N>
struct Walk {
    int64_t pos, hi;
    int b, h, n, L, tiles, off;
    int64_t t;

    // places [lo, hi_) of the line; lo < hi_ <= prefix[B]
    __device__ void start(const Shape& s, const Plan& p, int64_t lo, int64_t hi_) {
        pos = lo;
        hi = hi_;
        if (pos >= hi) return;
        int x = 0, y = s.B - 1;
        while (x < y) {
            const int mid = (x + y + 1) >> 1;
            if (p.prefix[mid] <= lo) x = mid;
            else y = mid - 1;
        }
        b = x;
        load(s);
        const int64_t ph = p.per_head[b];
        int64_t rem = lo - p.prefix[b];
        h = (int)(rem / ph);
        rem -= (int64_t)h * ph;
        t = 0;
        int nt = unit_tiles<N>(s.M, n, L, s.g, s.causal, 0);
        while (rem >= nt) {
            rem -= nt;
            ++t;
            nt = unit_tiles<N>(s.M, n, L, s.g, s.causal, t);
        }
        off = (int)rem;
    }
    __device__ __forceinline__ void load(const Shape& s) {
        n = s.new_tokens(b);
        L = s.length(b);
        tiles = (int)(((int64_t)n * s.g + s.M - 1) / s.M);
    }
    __device__ bool next(const Shape& s, Seg& o) {
        if (pos >= hi) return false;
        o.b = b;
        o.h = h;
        o.n = n;
        o.L = L;
        o.t = (int)t;
        o.row0 = (int)(t * s.M);
        o.rows = (int)min((int64_t)s.M, (int64_t)n * s.g - t * s.M);
        o.nt = unit_tiles<N>(s.M, n, L, s.g, s.causal, t);
        o.t0 = off;
        o.unit_start = pos - off;
        o.t1 = (int)min((int64_t)o.nt, off + (hi - pos));
        pos += o.t1 - o.t0;
        off = 0;
        if (pos < hi && ++t >= tiles) {
            t = 0;
            if (++h >= s.Hkv) {
                h = 0;
                do ++b;
                while (b < s.B - 1 && s.new_tokens(b) == 0);
                load(s);
            }
        }
        return true;
    }
};

// Blocks that have work, and the first place of block c (total < 2^48 by the host's checks, so the
// products fit).
__device__ __forceinline__ int active_blocks(int64_t total, int G) { return (int)min(total, (int64_t)G); }
__device__ __forceinline__ int64_t block_start(int64_t total, int active, int c) {
    return active > 0 ? total * c / active : 0;
}
// The block whose range holds place x.
__device__ __forceinline__ int block_of(int64_t total, int active, int64_t x) {
    int c = (int)(x * active / total);
    while (c + 1 < active && block_start(total, active, c + 1) <= x) ++c;
    while (c > 0 && block_start(total, active, c) > x) --c;
    return c;
}

// prefix and per_head from the lengths: one block.
template <int N>
__device__ void plan_block(const Shape& s, const Plan& p, int* status) {
    __shared__ int64_t warp_sums[32];
    __shared__ int64_t carry;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int base = 0; base < s.B; base += blockDim.x) {
        const int b = base + tid;
        int64_t tiles = 0;
        if (b < s.B) {
            const int n = s.new_tokens(b), L = s.length(b);
            if ((int64_t)s.seq_lens[b] > s.most() || s.seq_lens[b] < 0 || s.cu_new[b] < 0 ||
                s.cu_new[b + 1] < s.cu_new[b] || s.cu_new[b + 1] > s.T)
                atomicMax(status, 1);
            const int64_t row_tiles = ((int64_t)n * s.g + s.M - 1) / s.M;
            if (s.causal)
                for (int64_t t = 0; t < row_tiles; ++t) tiles += unit_tiles<N>(s.M, n, L, s.g, true, t);
            else if (row_tiles > 0)
                tiles = row_tiles * unit_tiles<N>(s.M, n, L, s.g, false, 0);
            p.per_head[b] = tiles;
        }
        int64_t x = tiles * s.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += a;
        }
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        int64_t before = carry;
        for (int w = 0; w < warp; ++w) before += warp_sums[w];
        if (b < s.B) p.prefix[b + 1] = before + x;
        if (b == 0) p.prefix[0] = 0;
        __syncthreads();
        if (tid == 0)
            for (int w = 0; w < nw; ++w) carry += warp_sums[w];
        __syncthreads();
    }
}

}  // namespace paged

constexpr int kPagedTcRows = 256;  // rows of a unit of the tensor-core kernel, at most

struct PagedJoin {
    paged::Shape s;
    paged::Plan p;
    void* O;
    int64_t o_t, o_h;
    float* lse;
    int G;
};
// M: rows of a piece
Status launch_paged_join(const PagedJoin& a, int dtype, int d, int M, cudaStream_t stream);

}  // namespace wildcat
