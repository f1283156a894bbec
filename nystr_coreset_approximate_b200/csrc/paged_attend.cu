// paged_attend.cu -- exact attention of new tokens over a paged cache.
//
//   O_i = sum_{j < e_i} exp(beta <q_i, k_j>) v_j / sum_{j < e_i} exp(beta <q_i, k_j>),
// e_i = L - n + i + 1 for token i of a request's n new ones (causal) or L; key
// j lies in page table[j / page] at row j % page.  A row that sees no key is
// zero (its log-sum -inf).  One pass over the keys with the running maximum m
// and sum l of each row: when m grows to m', l and the accumulated values are
// multiplied by 2^(m - m') (m in powers of two, beta log2(e) folded into the
// scores).
//
// Here: the dispatch, and the CUDA-core kernel, for
// float32 and for bf16 in shapes that the tensor cores' copies do not take
// (d = 32, pages that neither divide 128 rows in whole groups of 8 nor are a
// multiple of 128, strides that are no multiple of 16 bytes).  It works in float32
// throughout: one row tile is 64 rows, or 16 where the unit has no more, against
// 64 keys (units of up to four rows go without tiles); a thread holds 4 x 4 (1 x 4)
// scores and 4 (1) rows of D / 16 accumulators, in packed pairs.  A tile of 64 rows
// takes 8,000 cycles of an SM that has two blocks (4,096 of them multiply-adds,
// 3,000 reads of shared memory).  In float32, two requests of 2,000 tokens, 900 of
// them new, with 8/2 heads of 128: 405 us (28 TFLOP/s); 32 decoded tokens over 4,000
// keys each, 8 key heads of 128 with one query head 299 us (3.5 TB/s), with four 385,
// with five to sixteen 747 (1.4 TB/s, in tiles).  bf16 there: 32 over 4,000 with
// 32/8 heads of 32 166 us (0.8 TB/s), with heads of 128 in pages of 48 rows 654 us,
// where the tensor cores take 102 with pages of 16.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc_common.cuh"

namespace wildcat {

__device__ int g_paged_attend_status = 0;  // WILDCAT_ERR_INVALID_ARG: lengths or page ids out of range

namespace {

using namespace paged;

constexpr int kM = 64, kN = 64, kThreads = 256;
constexpr int kPad = 4;

int paged_sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    return n;
}

struct SimtArgs {
    Shape s;
    Plan p;
    const void* Q;
    const void* K;
    const void* V;
    int64_t q_t, q_h, k_p, k_h, k_r, v_p, v_h, v_r, o_t, o_h;
    void* O;
    float* lse;
    float scale;  // beta log2(e)
    bool wide;    // 16-byte loads of Q, K and V
    int G;
};

// Four values, widened.  The pools are read through the read-only path (RO); Q is not: O
// may be Q itself, and what that path reads must not be written while the kernel runs.
template <bool RO, typename V>
__device__ __forceinline__ V load_as(const void* p) {
    if constexpr (RO) return __ldg(static_cast<const V*>(p));
    else return *static_cast<const V*>(p);
}
template <bool RO>
__device__ __forceinline__ void load4(const float* p, bool wide, float (&v)[4]) {
    if (wide) {
        const float4 a = load_as<RO, float4>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = load_as<RO, float>(p + k);
    }
}
template <bool RO>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, bool wide, float (&v)[4]) {
    if (wide) {
        const uint2 u = load_as<RO, uint2>(p);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __bfloat162float(p[k]);
    }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 64 key (or value) rows from key k0 on: into registers (widened; rows at or past
// the length, or in a page outside the pool, as zeros), and from there into shared
// memory.  All page ids are read before the first row, and the rows are fetched
// while the tile before is worked on: one after the other the reads took 13,000
// cycles for a tile of a decoded token.
template <typename E, int D>
struct Rows {
    static constexpr int kCount = kN * (D / 4) / kThreads;
    float v[kCount][4];

    __device__ __forceinline__ void fetch(const SimtArgs& a, const Seg& g, const void* pool, int64_t sp, int64_t sh, int64_t sr,
                                          int k0) {
        using T = typename E::T;
        const T* base = static_cast<const T*>(pool) + (int64_t)g.h * sh;
        const int32_t* tab = a.s.table + (int64_t)g.b * a.s.table_stride;
        int id[kCount], at[kCount];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int j = k0 + (threadIdx.x + i * kThreads) / (D / 4);
            const int p = (unsigned)j / (unsigned)a.s.page_size;
            at[i] = j - p * a.s.page_size;
            id[i] = j < g.L ? __ldg(tab + p) : -1;
            bad = bad || (j < g.L && (id[i] < 0 || id[i] >= a.s.pages));
        }
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int c = (threadIdx.x + i * kThreads) % (D / 4) * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = 0.f;
            if (id[i] >= 0 && id[i] < a.s.pages) load4<true>(base + (int64_t)id[i] * sp + (int64_t)at[i] * sr + c, a.wide, v[i]);
        }
        if (bad) atomicMax(&g_paged_attend_status, 1);
    }
    __device__ __forceinline__ void store(float* dst) const {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int e = threadIdx.x + i * kThreads;
            *reinterpret_cast<float4*>(dst + e / (D / 4) * (D + kPad) + e % (D / 4) * 4) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        }
    }
};

// One segment with row tiles of 16 RT rows.
template <typename E, int D, int RT>
__device__ void simt_segment(const SimtArgs& a, const Seg& g, float* Qs, float* KVs, float* Ps) {
    using T = typename E::T;
    constexpr int MR = 16 * RT, CH = D / 64 > 0 ? D / 64 : 1, CW = D >= 64 ? 4 : 2;
    constexpr int QS = D + kPad, PS = kN + kPad;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int first = a.s.first_row(g.b);
    __syncthreads();  // the previous segment's reads are done
    for (int e = tid; e < MR * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = (e - r * (D / 4)) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < g.rows) {
            const int x = g.row0 + r, i = x / a.s.g;
            load4<false>(static_cast<const T*>(a.Q) + (int64_t)(first + i) * a.q_t +
                         (int64_t)(g.h * a.s.g + x - i * a.s.g) * a.q_h + c,
                     a.wide, v);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= a.scale;
        *reinterpret_cast<float4*>(Qs + r * QS + c) = make_float4(v[0], v[1], v[2], v[3]);
    }
    float2 acc[RT][CH][CW / 2];
    float m[RT], l[RT];
    int end[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int x = ty * RT + r;
        end[r] = x >= g.rows ? 0 : (a.s.causal ? g.L - g.n + (g.row0 + x) / a.s.g + 1 : g.L);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < CW / 2; ++k) acc[r][c][k] = make_float2(0.f, 0.f);
    }
    Rows<E, D> rows;
    rows.fetch(a, g, a.K, a.k_p, a.k_h, a.k_r, g.t0 * kN);
    for (int kt = g.t0; kt < g.t1; ++kt) {
        const int k0 = kt * kN;
        __syncthreads();
        rows.store(KVs);
        rows.fetch(a, g, a.V, a.v_p, a.v_h, a.v_r, k0);
        __syncthreads();
        float s[RT][4];
        float2 s2[RT][4];  // over even and odd columns: packed multiply-adds
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k) s2[r][k] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 kv[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) kv[k] = *reinterpret_cast<const float4*>(KVs + (tx + 16 * k) * QS + c);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float4 q = *reinterpret_cast<const float4*>(Qs + (ty * RT + r) * QS + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s2[r][k] = tc::ffma2(make_float2(q.x, q.y), make_float2(kv[k].x, kv[k].y), s2[r][k]);
                    s2[r][k] = tc::ffma2(make_float2(q.z, q.w), make_float2(kv[k].z, kv[k].w), s2[r][k]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[r][k] = s2[r][k].x + s2[r][k].y;
        __syncthreads();  // K has been read: V takes its place
        rows.store(KVs);
        if (kt + 1 < g.t1) rows.fetch(a, g, a.K, a.k_p, a.k_h, a.k_r, k0 + kN);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float best = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + tx + 16 * k >= end[r]) s[r][k] = -INFINITY;
                best = fmaxf(best, s[r][k]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
            const float mn = fmaxf(m[r], best), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[r] - base);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float p = exp2f(s[r][k] - base);
                Ps[(ty * RT + r) * PS + tx + 16 * k] = p;
                sum += p;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[r] = l[r] * f + sum;
            m[r] = mn;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < CW / 2; ++k) {
                    acc[r][c][k].x *= f;
                    acc[r][c][k].y *= f;
                }
        }
        __syncthreads();
#pragma unroll 2
        for (int j = 0; j < kN; j += 4) {
            float4 p[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) p[r] = *reinterpret_cast<const float4*>(Ps + (ty * RT + r) * PS + j);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float2 v[CW / 2];
                    const float* src = KVs + (j + jj) * QS + c * 64 + tx * CW;
                    if constexpr (CW == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        v[0] = make_float2(x.x, x.y);
                        v[1] = make_float2(x.z, x.w);
                    } else {
                        v[0] = *reinterpret_cast<const float2*>(src);
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float pr = jj == 0 ? p[r].x : jj == 1 ? p[r].y : jj == 2 ? p[r].z : p[r].w;
#pragma unroll
                        for (int k = 0; k < CW / 2; ++k) acc[r][c][k] = tc::ffma2(make_float2(pr, pr), v[k], acc[r][c][k]);
                    }
                }
            }
        }
    }
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    const int64_t piece = ((int64_t)blockIdx.x * 2 + (g.t0 > 0 ? 0 : 1)) * kM;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int x = ty * RT + r;
        if (x >= g.rows) continue;
        if (whole) {
            const int i = (g.row0 + x) / a.s.g, hq = g.h * a.s.g + g.row0 + x - i * a.s.g;
            const float rcp = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
            T* o = static_cast<T*>(a.O) + (int64_t)(first + i) * a.o_t + (int64_t)hq * a.o_h;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < CW / 2; ++k) {
                    put(o + c * 64 + tx * CW + 2 * k, acc[r][c][k].x * rcp);
                    put(o + c * 64 + tx * CW + 2 * k + 1, acc[r][c][k].y * rcp);
                }
            if (a.lse && tx == 0)
                a.lse[(int64_t)(first + i) * (a.s.Hkv * a.s.g) + hq] =
                    l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * 0.6931471805599453f;
        } else {
            float* o = a.p.part + (piece + x) * D;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < CW / 2; ++k) *reinterpret_cast<float2*>(o + c * 64 + tx * CW + 2 * k) = acc[r][c][k];
            if (tx == 0) a.p.ml[piece + x] = make_float2(m[r], l[r]);
        }
    }
}

// One segment of a unit of up to kFew rows (a decoded token of a few query heads): no
// tiles, since 16 rows of threads would idle behind as many reads of shared memory
// (11,600 cycles for 64 keys).  D / 4 lanes make a stream that takes every kStreams-th
// key, straight from memory to registers, four keys at a time, with a running maximum,
// sum and accumulators of its own; the streams are joined in shared memory, in order.
// Why four: 32 x 4,000 keys, 8 key heads of 64, float32, take 155, 167, 181, 195 us with
// one to four rows, and 404 in tiles with any number.  A build for up to eight rows
// takes 276, 301, 328, 366 with five to eight, but 179 to 252 with one to four: its
// registers cost the common cases a sixth to a third.
constexpr int kFew = 4;
template <typename E, int D>
__device__ void simt_few(const SimtArgs& a, const Seg& g, float* sm) {
    using T = typename E::T;
    constexpr int LN = D / 4, kStreams = kThreads / LN, U = 4;
    const int tid = threadIdx.x, col = tid % LN * 4, stream = tid / LN;
    const int first = a.s.first_row(g.b);
    float q[kFew][4], acc[kFew][4], m[kFew], l[kFew];
    int end[kFew];
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
        const int x = g.row0 + r, i = x / a.s.g;
        end[r] = r >= g.rows ? 0 : (a.s.causal ? g.L - g.n + i + 1 : g.L);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) q[r][k] = acc[r][k] = 0.f;
        if (r < g.rows)
            load4<false>(static_cast<const T*>(a.Q) + (int64_t)(first + i) * a.q_t + (int64_t)(g.h * a.s.g + x - i * a.s.g) * a.q_h + col,
                     a.wide, q[r]);
#pragma unroll
        for (int k = 0; k < 4; ++k) q[r][k] *= a.scale;
    }
    const T* K = static_cast<const T*>(a.K) + (int64_t)g.h * a.k_h + col;
    const T* V = static_cast<const T*>(a.V) + (int64_t)g.h * a.v_h + col;
    const int32_t* tab = a.s.table + (int64_t)g.b * a.s.table_stride;
    const int hi = min(g.t1 * kN, g.L);
    bool bad = false;
    for (int j0 = g.t0 * kN + stream; j0 - stream < hi; j0 += U * kStreams) {  // the same number of turns for all
        int id[U];
        float k4[U][4], v4[U][4], s[kFew][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kStreams;
            id[u] = j < hi ? __ldg(tab + (unsigned)j / (unsigned)a.s.page_size) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kStreams, at = (unsigned)j % (unsigned)a.s.page_size;
#pragma unroll
            for (int k = 0; k < 4; ++k) k4[u][k] = v4[u][k] = 0.f;
            if (j < hi) {
                if (id[u] >= 0 && id[u] < a.s.pages) {
                    load4<true>(K + (int64_t)id[u] * a.k_p + (int64_t)at * a.k_r, a.wide, k4[u]);
                    load4<true>(V + (int64_t)id[u] * a.v_p + (int64_t)at * a.v_r, a.wide, v4[u]);
                } else {
                    bad = true;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            if (r >= g.rows) break;
            float best = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x = q[r][0] * k4[u][0];
#pragma unroll
                for (int k = 1; k < 4; ++k) x = fmaf(q[r][k], k4[u][k], x);
#pragma unroll
                for (int o = LN / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                s[r][u] = j0 + u * kStreams < min(end[r], hi) ? x : -INFINITY;
                best = fmaxf(best, s[r][u]);
            }
            const float mn = fmaxf(m[r], best), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[r] - base);
            m[r] = mn;
            l[r] *= f;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[r][k] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = exp2f(s[r][u] - base);
                l[r] += p;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[r][k] = fmaf(p, v4[u][k], acc[r][k]);
            }
        }
    }
    if (bad) atomicMax(&g_paged_attend_status, 1);
    float2* ml = reinterpret_cast<float2*>(sm + kStreams * kFew * D);
    __syncthreads();  // the previous segment's reads are done
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
        *reinterpret_cast<float4*>(sm + (stream * kFew + r) * D + col) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
        if (col == 0) ml[stream * kFew + r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    const int64_t piece = ((int64_t)blockIdx.x * 2 + (g.t0 > 0 ? 0 : 1)) * kM;
    for (int e = tid; e < g.rows * D; e += kThreads) {
        const int r = e / D, c = e - r * D;
        float top = -INFINITY;
        for (int x = 0; x < kStreams; ++x) top = fmaxf(top, ml[x * kFew + r].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, out = 0.f;
        for (int x = 0; x < kStreams; ++x) {
            const float2 w = ml[x * kFew + r];
            const float f = exp2f(w.x - base);
            sum = fmaf(f, w.y, sum);
            out = fmaf(f, sm[(x * kFew + r) * D + c], out);
        }
        if (whole) {
            const int i = (g.row0 + r) / a.s.g, hq = g.h * a.s.g + g.row0 + r - i * a.s.g;
            put(static_cast<T*>(a.O) + (int64_t)(first + i) * a.o_t + (int64_t)hq * a.o_h + c,
                sum > 0.f || sum != sum ? out / sum : 0.f);
            if (a.lse && c == 0)
                a.lse[(int64_t)(first + i) * (a.s.Hkv * a.s.g) + hq] =
                    sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        } else {
            a.p.part[(piece + r) * D + c] = out;
            if (c == 0) a.p.ml[piece + r] = make_float2(top, sum);
        }
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 2) paged_simt_kernel(SimtArgs a) {
    extern __shared__ __align__(16) float simt_sm[];
    float* Qs = simt_sm;
    float* KVs = Qs + kM * (D + kPad);
    float* Ps = KVs + kN * (D + kPad);
    __shared__ ShareScratch scratch;
    find_share<kN>(a.s, a.G, &scratch, &g_paged_attend_status);
    __syncthreads();
    int4 join = make_int4(0, 0, 0, kNoJoin);
    {
        Walk<kN> w;
        w.start(a.s, scratch.share);
        Seg g;
        while (w.next(a.s, g)) {
            if (g.rows <= kFew) simt_few<E, D>(a, g, simt_sm);
            else if (g.rows <= 16) simt_segment<E, D, 1>(a, g, Qs, KVs, Ps);
            else simt_segment<E, D, 4>(a, g, Qs, KVs, Ps);
            if (g.t0 > 0 && g.t1 == g.nt) join = make_int4(g.b, g.h, g.t, scratch.share.line.block(g.first_end));
        }
    }
    if (threadIdx.x == 0) a.p.joins[blockIdx.x] = join;
}

template <typename E, int D>
Status run_simt(const PagedAttendRequest& q, cudaStream_t st) {
    using T = typename E::T;
    const int G = 2 * paged_sm_count();
    Carve cv(q.ws, q.ws_bytes);
    SimtArgs a{};
    carve_plan(cv, &a.p, G, kM, D);
    if (!cv.fits()) return Status::fail(4, "paged_attend: workspace too small");
    a.s = Shape{q.table, q.table_stride, q.W, q.seq_lens, q.cu_new, q.T, q.pages, (int)q.B, q.Hkv, q.Hq / q.Hkv,
                q.page_size, kM, kFew, 2, q.causal};
    a.Q = q.Q; a.K = q.K; a.V = q.V;
    a.q_t = q.q_t; a.q_h = q.q_h;
    a.k_p = q.k_p; a.k_h = q.k_h; a.k_r = q.k_r;
    a.v_p = q.v_p; a.v_h = q.v_h; a.v_r = q.v_r;
    a.O = q.O; a.o_t = q.o_t; a.o_h = q.o_h;
    a.lse = q.lse;
    a.scale = q.beta * 1.4426950408889634f;
    a.G = G;
    const int64_t all = q.q_t | q.q_h | q.k_p | q.k_h | q.k_r | q.v_p | q.v_h | q.v_r;
    const uintptr_t ptrs = reinterpret_cast<uintptr_t>(q.Q) | reinterpret_cast<uintptr_t>(q.K) | reinterpret_cast<uintptr_t>(q.V);
    a.wide = all % 4 == 0 && ptrs % (4 * sizeof(T)) == 0;
    const size_t smem = sizeof(float) * ((size_t)(kM + kN) * (D + kPad) + (size_t)kM * (kN + kPad));
    cudaError_t e = allow_smem<paged_simt_kernel<E, D>>((int)smem);
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend: shared memory attribute");
    paged_simt_kernel<E, D><<<G, kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend launch");
    return launch_paged_join(PagedJoin{a.s, a.p, q.O, q.o_t, q.o_h, q.lse, G}, q.dtype, D, kM, st);
}

}  // namespace

size_t paged_attend_workspace_bytes(int d) {
    const int sms = paged_sm_count();
    Plan p;
    Carve a(nullptr, 0), b(nullptr, 0);
    const size_t simt = carve_plan(a, &p, 2 * sms, kM, d), tc = carve_plan(b, &p, sms, kPagedTcRows, d);
    return std::max(simt, tc) + 256;
}

Status launch_paged_attend(const PagedAttendRequest& q, cudaStream_t st) {
    const bool bf = q.dtype == 1;
    if (paged_attend_tc_supported(q)) return launch_paged_attend_tc(q, st);
    switch (q.d) {
        case 32: return bf ? run_simt<BF16, 32>(q, st) : run_simt<F32, 32>(q, st);
        case 64: return bf ? run_simt<BF16, 64>(q, st) : run_simt<F32, 64>(q, st);
        case 128: return bf ? run_simt<BF16, 128>(q, st) : run_simt<F32, 128>(q, st);
    }
    return Status::fail(2, "paged_attend: unsupported head dim");
}

int read_paged_attend_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_attend_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_paged_attend_status, &z, sizeof(int));
    }
    return v;
}

}  // namespace wildcat
