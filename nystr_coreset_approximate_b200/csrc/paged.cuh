// paged.cuh -- how the paged attention's work is cut, shared by its kernels.
//
// A unit is (request b, key head h, row tile t): `rows` consecutive rows of
// the request's n * g query rows of that key head (row r = token r / g, query
// head h * g + r % g), M at most.  Its keys come in tiles of N.  All units
// stand in one line, requests first, then heads and row tiles; a unit takes
// kUnitCost places for its beginning and end and then 2^wide places for each key
// tile (one where it has R rows at most: less work).  Block c of G takes the
// next T / G of the T places in all, and of each unit the key tiles that end
// there.  Every block so has about the same work whatever the lengths
// are: one long request is spread over the GPU, and many short ones are packed.
// A unit that lies whole in one block is finished there; of one that is cut, each
// block leaves a partial sum, and paged_join_kernel joins them in the order of the
// keys, the same in every run.  Each block finds its place in the line for itself.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace wildcat {
namespace paged {

struct Plan {
    int4* joins;        // [G] the cut unit that ends in block c: (b, h, t, first block), first block kNoJoin for none
    float* part;        // [2 G][M][D] partial sums of the exponentials times V
    float2* ml;         // [2 G][M] their maximum (of beta s, in powers of two) and sum
};

constexpr int kNoJoin = -1;   // no cut unit ends in the block
constexpr int kGaveUp = -2;   // the block gave up (an expired wait): its pieces may be missing

inline size_t carve_plan(Carve& cv, Plan* p, int G, int M, int D) {
    p->joins = static_cast<int4*>(cv.take(sizeof(int4) * G));
    p->ml = static_cast<float2*>(cv.take(sizeof(float2) * 2 * G * M));
    p->part = static_cast<float*>(cv.take(sizeof(float) * 2 * G * (size_t)M * D));
    return cv.used;
}

// Opts kernel F into `bytes` of dynamic shared memory, once for each device.
template <auto F>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};  // devices 0 to 63
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(F, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// What the kernels know of the call.
struct Shape {
    const int32_t* table;
    int64_t table_stride, W;
    const int32_t* seq_lens;
    const int32_t* cu_new;
    int64_t T, pages;
    int B, Hkv, g, page_size;
    int M, R, wide;  // rows of a unit; up to R of them a key tile takes one place, else 2^wide
    bool causal;

    __device__ __forceinline__ int first_row(int b) const {
        return (int)min(max((int64_t)cu_new[b], (int64_t)0), T);
    }
    __device__ __forceinline__ int new_tokens(int b) const { return max(first_row(b + 1) - first_row(b), 0); }
    // a length past the table's pages is cut to them (find_share reports it); so is one
    // whose last key tile would end past 2^31
    __device__ __forceinline__ int64_t most() const { return min(W * page_size, (int64_t)0x7fffff00); }
    __device__ __forceinline__ int length(int b) const { return (int)min((int64_t)max(seq_lens[b], 0), most()); }
};

// With 1, 2 and 4 (us, bf16): 2,000 decoded tokens over one key tile 586, 600, 597, over
// two 717, 748, 750; 64 over 900 keys 79, 80, 80, three of them 17.3, 17.0, 16.0; 16 prompts
// of 300 tokens 62.7, 63.9, 61.0; 200 tokens over 600 keys with heads of 64 275, 267, 259.
constexpr int kUnitCost = 2;

// x / y of what nearly always fits in 32 bits: a division of 64 bits takes some hundred
// instructions, and these stand before a block's first copy.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if (((uint64_t)x | (uint64_t)y) >> 32) return x / y;
    return (int64_t)((uint32_t)x / (uint32_t)y);
}

// A request's units of one key head.
template <int N>
struct Units {
    int n, L, tiles;  // new tokens, positions, row tiles

    __device__ __forceinline__ void of(const Shape& s, int b) {
        n = s.new_tokens(b);
        L = s.length(b);
        tiles = (int)(((unsigned)n * (unsigned)s.g + (unsigned)s.M - 1u) / (unsigned)s.M);  // n g < 2^31
    }
    __device__ __forceinline__ int rows(const Shape& s, int t) const {
        return min(s.M, n * s.g - t * s.M);
    }
    // log2 of the places of a key tile
    __device__ __forceinline__ int width(const Shape& s, int t) const { return rows(s, t) > s.R ? s.wide : 0; }
    // key tiles of row tile t (at least one: rows that see nothing are written too)
    __device__ __forceinline__ int keys(const Shape& s, int t) const {
        int end = L;
        if (s.causal) {
            const int last = min((int)(((unsigned)t * s.M + s.M - 1u) / (unsigned)s.g), n - 1);  // the tile's last token
            end = max(L - n + last + 1, 0);
        }
        return max((end + N - 1) / N, 1);
    }
    __device__ __forceinline__ int64_t places(const Shape& s, int t) const {
        return kUnitCost + ((int64_t)keys(s, t) << width(s, t));
    }
    // places of all row tiles
    __device__ int64_t all(const Shape& s) const {
        if (tiles == 0) return 0;
        const int64_t last = places(s, tiles - 1);
        const int head = tiles - 1;
        if (head == 0) return last;
        if (!s.causal) return last + head * places(s, 0);  // these tiles are full
        if (s.M % s.g || N & (N - 1)) {
            int64_t sum = last;
            for (int t = 0; t < head; ++t) sum += places(s, t);
            return sum;
        }
        // tile t ends at a + q t, q = M / g: sum of max(ceil((a + q t) / N), 1) over t < head
        const int q = s.M / s.g, a = L - n + q;
        const int below = a > 0 ? 0 : min((unsigned)-a / (unsigned)q + 1u, (unsigned)head);  // tiles that see no key
        return last + (int64_t)head * kUnitCost + ((below + floor_sum(head - below, q, (int64_t)a + q * below + N - 1)) << width(s, 0));
    }
    // sum over i < count of floor((q i + b) / N), 0 < q <= 2 N, b >= 0, N a power of two: the
    // steps of Euclid's algorithm, each of which turns the sum's triangle of points over
    __device__ static int64_t floor_sum(unsigned count, unsigned q, int64_t b) {
        int64_t sum = (int64_t)count * (b / N);
        unsigned m = N, r = (unsigned)(b % N);
        bool plus = true;
        while (count > 0) {  // of floor((q i + r) / m), m and q at most 2 N: 32 bits hold q count + r
            int64_t part = (int64_t)count * (count - 1) / 2 * (q / m) + (int64_t)count * (r / m);
            q %= m;
            r %= m;
            const unsigned high = (q * count + r) / m;
            // points (i, y), 1 <= y <= floor((q i + r) / m), i < count: of the count in row y <= high
            // those below i = ceil((m y - r) / q) are missing
            part += (int64_t)count * high;
            sum += plus ? part : -part;
            if (high == 0) break;
            plus = !plus;
            // sum over y = 1 .. high of ceil((m y - r) / q) = sum over j < high of floor((m j + m - r + q - 1) / q)
            const unsigned nr = m - r + q - 1u;
            count = high;
            r = nr;
            const unsigned old = m;
            m = q;
            q = old;
        }
        return sum;
    }
};

struct Seg {
    int b, h, n, L, row0, rows;  // row0: first row of the unit among the request's n * g
    int t, nt, t0, t1;           // key tiles [t0, t1) of the unit's nt
    int64_t first_end;           // the last place of the unit's first key tile
};

// The T places in all and the blocks that share them.  Each block has at least the 2^wide
// places of a key tile, so that one that lies wholly within a unit's key tiles finishes
// one: the join takes a piece from every block between the first piece's and the last's.
// (Where a unit begins, a block may have no more than its kUnitCost places, and no piece.)
struct Line {
    int64_t total, each;  // places of a block, and one more for the first `rest` of them
    int active, rest;

    __device__ __forceinline__ void of(const Shape& s, int64_t t, int G) {
        total = t;
        active = (int)min(max(t >> s.wide, (int64_t)(t > 0)), (int64_t)G);
        each = active > 0 ? quotient(t, active) : 0;
        rest = (int)(t - each * active);
    }
    __device__ __forceinline__ int64_t start(int c) const { return each * c + min(c, rest); }
    // the block whose range holds place x
    __device__ __forceinline__ int block(int64_t x) const {
        const int64_t y = x - (each + 1) * rest;
        return y < 0 ? (int)quotient(x, each + 1) : rest + (int)quotient(y, each);
    }
};

// A block's share of the line.
struct Share {
    Line line;
    int64_t lo, hi;
    int64_t before;    // places before request b, that of place lo
    int64_t per_head;  // places of one of its key heads
    int b;
};
struct ShareScratch {
    int64_t warp_sums[32];
    Share share;
};
// All threads of the block; `scratch` in shared memory, the caller synchronises after it.
template <int N>
__device__ void find_share(const Shape& s, int G, ShareScratch* scratch, int* status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    // consecutive requests to each thread; first their places, then the request that holds lo
    const int each = ((unsigned)s.B + blockDim.x - 1u) / blockDim.x;
    const int b0 = min(tid * each, s.B), b1 = min(b0 + each, s.B);
    int64_t lo = 0, end = 0;
    Share* o = &scratch->share;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const int64_t before = end;  // places before this thread's requests
        if (pass == 1 && !(before <= lo && lo < scratch->share.hi)) break;
        int64_t sum = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            Units<N> u;
            u.of(s, b);
            const int64_t ph = u.all(s), next = sum + ph * s.Hkv;
            if (pass == 1 && before + sum <= lo && lo < before + next) {
                o->b = b;
                o->before = before + sum;
                o->per_head = ph;
                break;
            }
            if (pass == 0 && blockIdx.x == 0 &&
                ((int64_t)s.seq_lens[b] > s.most() || s.seq_lens[b] < 0 || s.cu_new[b] < 0 ||
                 s.cu_new[b + 1] < s.cu_new[b] || s.cu_new[b + 1] > s.T))
                atomicMax(status, 1);
            sum = next;
        }
        if (pass == 1) break;
        int64_t x = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += a;
        }
        if (lane == 31) scratch->warp_sums[warp] = x;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < nw; ++w) {
            const int64_t a = scratch->warp_sums[w];
            if (w < warp) x += a;
            total += a;
        }
        end = x - sum;
        if (tid == 0) {
            Line line;
            line.of(s, total, G);
            const int c = blockIdx.x;
            o->line = line;
            o->lo = c < line.active ? line.start(c) : 0;
            o->hi = c < line.active ? line.start(c + 1) : 0;
        }
        __syncthreads();
        lo = o->lo;
        if (x <= lo) end = lo + 1;  // not among this thread's
    }
}

// The segments of one block, in order.  Called by whole warps.
template <int N>
struct Walk {
    Units<N> u;
    int64_t pos, hi, off;
    int b, h, t;

    __device__ void start(const Shape& s, const Share& o) {
        pos = o.lo;
        hi = o.hi;
        if (pos >= hi) return;
        b = o.b;
        u.of(s, b);
        int64_t rem = o.lo - o.before;
        h = (int)quotient(rem, o.per_head);
        rem -= (int64_t)h * o.per_head;
        // the row tile, 32 at a time
        const int lane = threadIdx.x & 31;
        for (int base = 0;; base += 32) {
            const int64_t mine = base + lane < u.tiles ? u.places(s, base + lane) : (int64_t)1 << 50;
            int64_t x = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t a = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += a;
            }
            const unsigned past = __ballot_sync(0xffffffffu, x > rem);
            if (past) {
                const int f = __ffs(past) - 1;
                t = base + f;
                off = rem - __shfl_sync(0xffffffffu, x - mine, f);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __device__ bool next(const Shape& s, Seg& o) {
        while (pos < hi) {
            const int nt = u.keys(s, t), w = u.width(s, t);
            const int64_t size = kUnitCost + ((int64_t)nt << w), end = min(size, off + (hi - pos));
            o.b = b;
            o.h = h;
            o.n = u.n;
            o.L = u.L;
            o.t = t;
            o.row0 = t * s.M;
            o.rows = u.rows(s, t);
            o.nt = nt;
            o.t0 = (int)(max(off - kUnitCost, (int64_t)0) >> w);
            o.t1 = (int)(max(end - kUnitCost, (int64_t)0) >> w);
            o.first_end = pos - off + kUnitCost + (1 << w) - 1;
            pos += end - off;
            off = 0;
            if (pos < hi && ++t >= u.tiles) {
                t = 0;
                if (++h >= s.Hkv) {
                    h = 0;
                    do ++b;
                    while (b < s.B - 1 && s.new_tokens(b) == 0);
                    u.of(s, b);
                }
            }
            if (o.t1 > o.t0) return true;
        }
        return false;
    }
};

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
