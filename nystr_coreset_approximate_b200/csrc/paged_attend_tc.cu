// paged_attend_tc.cu -- exact attention over a paged cache on the tensor cores
// (bf16, d in {64, 128}); the formulas are those of paged_attend.cu.
//
// One persistent block per SM walks its share of the key tiles (paged.cuh).  A
// row tile is R <= 128 query rows of one key head, whole tokens of g rows each
// (R = floor(128 / g) g), loaded by one TMA box that gathers the g heads; a
// unit has up to two of them.  The work is a sequence of operations, numbered
// k = 0, 1, ...; operation k takes one row tile and one tile of 128 keys in slot
// k & 1 of the tensor memory (scores S, accumulator O):
//     S = Q K^T          (tcgen05.mma, both operands in shared memory)
//     P = 2^(beta log2e S - m), rounded to bf16, written over S
//     O += P V           (A from tensor memory, V as it lies: keys by columns)
// A unit with two row tiles runs both against each key tile (one slot each, one
// load of K and V for 2 R rows: the tensor cores bound it); a unit with one, a
// decoded token's or a short chunk's, runs successive key tiles in the two slots
// with a running maximum and sum of its own for each (HBM bounds it), which the
// epilogue adds up.  The issue order is S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...,
// across units: while one slot's scores are exponentiated the other's products
// run.  K and V tiles pass through one ring of stages in the order of first use.
// Warp roles:
//   warp 0      producer: block-table lookups (one lane per page) and TMA
//   warp 1      tensor cores (one thread issues)
//   warp 2      zeroes the rows of V at or past the request's length in its last
//               key tile: what the page holds there may be NaN, and 0 NaN is NaN
//   warps 4-7   softmax of slot 0, warps 8-11 of slot 1, one row per thread.  The
//               maximum is raised only when a row's grows by more than 2^8 (sums
//               in float32 hold that; a bf16 P is as exact at 2^8 as at 1), so
//               the accumulator is hardly ever rescaled
//   warps 12-15 epilogue: O / l as bf16, or a partial sum of a unit that is cut
// P is rounded to bf16 for the product (the operand type of V); the sum l is
// float32 of the unrounded P.
//
// Every wait is bounded (2 s) and gives up when another role has given up; an
// expired wait records WILDCAT_ERR_TIMEOUT in the device status word, the block
// drains its copies and products (bounded), frees its tensor memory and returns.
// No load uses cluster multicast.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc_common.cuh"
#include "tmap.h"

namespace wildcat {

__device__ int g_paged_tc_status = 0;  // WILDCAT_ERR_TIMEOUT or WILDCAT_ERR_INVALID_ARG

namespace {

using namespace tc;
using namespace paged;

constexpr int kRows = 128, kKeys = 128;
constexpr int kThreads = 512;
constexpr int kPlanThreads = 512;
// registers per thread after the split: 96 + 2 * 168 + 80 = 512 per lane of a
// sub-partition, the 4 * 128 it was launched with
constexpr int kRegsLow = 96, kRegsSoftmax = 168, kRegsEpilogue = 80;
static_assert(kRegsLow + 2 * kRegsSoftmax + kRegsEpilogue == 512, "register split");
constexpr unsigned long long kDrainNs = 100000000ull;
constexpr float kRaise = 8.0f;  // the maximum is raised when a row's grows by more (powers of two)

template <int NS>
struct Bars {
    uint64_t q_full[2], q_free[2];
    uint64_t full[NS], fixed[NS], empty[NS];
    uint64_t s_full[2], p_full[2], pv_done[2], o_full[2], o_free[2], den_full[2];
    uint64_t drain;
    unsigned tmem_base;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr int KB = D / 64;                   // 128-byte blocks of a row
    static constexpr int NS = D == 128 ? 5 : 12;        // stages of the ring of K and V tiles
    static constexpr uint32_t q_bytes = kRows * D * 2;  // one row tile
    static constexpr uint32_t t_bytes = kKeys * D * 2;  // one tile of K or V
    static constexpr uint32_t blk = kKeys * 128;        // one 128-byte block of a tile
    static constexpr uint32_t off_q = 0;
    static constexpr uint32_t off_t = off_q + 2 * q_bytes;
    static constexpr uint32_t off_ml = off_t + NS * t_bytes;  // (m, l) of each slot's rows
    static constexpr uint32_t off_bar = off_ml + 2 * kRows * 8;
    static constexpr uint32_t total = off_bar + (uint32_t)sizeof(Bars<NS>);
    static constexpr unsigned tmem_cols = 512;
    static constexpr unsigned col_O = 0;      // O of slot t at t * D
    static constexpr unsigned col_S = 2 * D;  // S of slot t at 2 D + 128 t
    static_assert(total <= 232448, "shared memory");
};

struct TcArgs {
    Shape s;
    Plan p;
    __nv_bfloat16* O;
    int64_t o_t, o_h;
    float* lse;
    float scale;  // beta log2(e)
    int G, R;     // blocks; rows of a row tile
    int box;      // rows of a page in one copy: min(page_size, 128)
};

// The operations of one block, in order.
struct Ops {
    Walk<kKeys> w;
    Seg g;
    int i, n;      // operation of the segment, and how many it has
    unsigned k0;   // number of its first operation
    unsigned q0;   // row tiles loaded before it
    bool two;      // two row tiles
    bool valid;

    __device__ __forceinline__ void load(int R) {
        two = g.rows > R;
        n = (g.t1 - g.t0) << (two ? 1 : 0);
        i = 0;
    }
    __device__ __forceinline__ void start(const TcArgs& a, int64_t lo, int64_t hi) {
        w.start(a.s, a.p, lo, hi);
        k0 = q0 = 0;
        valid = w.next(a.s, g);
        if (valid) load(a.R);
    }
    __device__ __forceinline__ void next_seg(const TcArgs& a) {
        k0 += n;
        q0 += two ? 2 : 1;
        valid = w.next(a.s, g);
        if (valid) load(a.R);
    }
    __device__ __forceinline__ void next(const TcArgs& a) {
        if (++i == n) next_seg(a);
    }
    __device__ __forceinline__ int slot() const { return (int)((k0 + i) & 1u); }
    __device__ __forceinline__ int tile() const { return two ? i & 1 : 0; }  // row tile
    __device__ __forceinline__ int key_tile() const { return g.t0 + (two ? i >> 1 : i); }
    __device__ __forceinline__ bool first() const { return i < 2; }  // of its slot in the segment
    __device__ __forceinline__ bool last() const { return i >= n - 2; }
    __device__ __forceinline__ bool opens() const { return !two || !(i & 1); }  // first use of the key tile
    __device__ __forceinline__ bool closes() const { return !two || (i & 1); }  // last use
    __device__ __forceinline__ int q_buf() const { return (int)((q0 + tile()) & 1u); }
    __device__ __forceinline__ bool q_opens() const { return i < (two ? 2 : 1); }
    __device__ __forceinline__ bool q_closes() const { return i >= n - (two ? 2 : 1); }
    // rows of V past the length in this key tile
    __device__ __forceinline__ bool tail() const { return (key_tile() + 1) * kKeys > g.L; }
};

template <int D>
struct Ctx {
    unsigned char* sm;
    unsigned sbase, tmem;
    Bars<Cfg<D>::NS>* bars;
    volatile int* abort_flag;
    int64_t lo, hi;
    __device__ void give_up() const {
        *abort_flag = 1;
        atomicMax(&g_paged_tc_status, 5);
    }
};

// Warp 0.  All lanes walk alike; lane p looks up and copies page p of a tile.
template <int D>
__device__ __forceinline__ void role_producer(const Ctx<D>& x, const TcArgs& a, const CUtensorMap* tmQ,
                                              const CUtensorMap* tmK, const CUtensorMap* tmV, int lane) {
    using C = Cfg<D>;
    constexpr int NS = C::NS;
    auto* bars = x.bars;
    if (lane == 0) {
        prefetch_tmap(tmQ);
        prefetch_tmap(tmK);
        prefetch_tmap(tmV);
    }
    unsigned n = 0, qn = 0;  // tiles and row tiles issued
    bool ok = true;
    auto put_tile = [&](const Ops& o, const CUtensorMap* tm) {
        const int s = (int)(n % NS);
        if (n >= NS) {
            ok = __all_sync(0xffffffffu, mbar_wait_suspend(&bars->empty[s], (n / NS - 1) & 1u, x.abort_flag));
            if (!ok) return;
        }
        if (lane == 0) mbar_expect_tx(&bars->full[s], C::t_bytes);
        __syncwarp();
        const int boxes = kKeys / a.box;
        if (lane < boxes) {
            const int j = o.key_tile() * kKeys + lane * a.box, p = j / a.s.page_size;
            int id = (int)a.s.pages;  // past the pool: the copy fills zeros
            if (j < o.g.L) {
                const int v = a.s.table[(int64_t)o.g.b * a.s.table_stride + p];
                if (v >= 0 && v < a.s.pages) id = v;
                else atomicMax(&g_paged_tc_status, 1);
            }
            const unsigned dst = x.sbase + C::off_t + (unsigned)s * C::t_bytes + (unsigned)(lane * a.box) * 128u;
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
                tma_load_4d(dst + kb * C::blk, tm, kb * 64, j - p * a.s.page_size, o.g.h, id, &bars->full[s]);
        }
        ++n;
    };
    auto put_k = [&](const Ops& o) {
        if (o.q_opens()) {
            const int qb = (int)(qn & 1u);
            if (qn >= 2) {
                ok = __all_sync(0xffffffffu, mbar_wait_suspend(&bars->q_free[qb], (qn / 2 - 1) & 1u, x.abort_flag));
                if (!ok) return;
            }
            if (lane == 0) {
                mbar_expect_tx(&bars->q_full[qb], (unsigned)a.R * 128u * C::KB);
                const int token = a.s.first_row(o.g.b) + (o.g.row0 + o.tile() * a.R) / a.s.g;
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb)
                    tma_load_4d(x.sbase + C::off_q + (unsigned)qb * C::q_bytes + kb * (kRows * 128), tmQ, kb * 64, 0,
                                o.g.h, token, &bars->q_full[qb]);
            }
            ++qn;
        }
        if (o.opens()) put_tile(o, tmK);
    };
    Ops k, v;
    k.start(a, x.lo, x.hi);
    v = k;
    for (int e = 0; e < 2 && k.valid && ok; ++e) {
        put_k(k);
        k.next(a);
    }
    while (v.valid && ok) {
        if (v.opens()) put_tile(v, tmV);
        v.next(a);
        if (!ok) break;
        if (k.valid) {
            put_k(k);
            k.next(a);
        }
    }
    if (!ok && lane == 0) x.give_up();
    __syncwarp();
    if (*x.abort_flag) {
        // copies still in flight land before the block's shared memory is released
        if (qn > 0) mbar_wait(&bars->q_full[(qn - 1) & 1u], ((qn - 1) / 2) & 1u, kDrainNs);
        if (qn > 1) mbar_wait(&bars->q_full[(qn - 2) & 1u], ((qn - 2) / 2) & 1u, kDrainNs);
        for (unsigned c = n > NS ? n - NS : 0; c < n; ++c) mbar_wait(&bars->full[c % NS], (c / NS) & 1u, kDrainNs);
    }
}

// Warp 2: takes every tile of the ring in the producer's order, so that it is
// never more than the ring's length away from the other roles, and zeroes the
// rows of V past the length before it hands a tile on.
template <int D>
__device__ __forceinline__ void role_fix(const Ctx<D>& x, const TcArgs& a, int lane) {
    using C = Cfg<D>;
    constexpr int NS = C::NS;
    unsigned n = 0;
    bool ok = true;
    auto take = [&](int keep) {  // rows of the tile that stay as they are
        const int s = (int)(n % NS);
        ok = __all_sync(0xffffffffu, mbar_wait_suspend(&x.bars->full[s], (n / NS) & 1u, x.abort_flag));
        if (!ok) return;
        if (keep < kKeys) {
            unsigned char* tile = x.sm + C::off_t + (unsigned)s * C::t_bytes;
            for (int e = lane; e < (kKeys - keep) * 8; e += 32)
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb)
                    *reinterpret_cast<uint4*>(tile + kb * C::blk + keep * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&x.bars->fixed[s]);
            mbar_arrive(&x.bars->empty[s]);
        }
        ++n;
    };
    Ops k, v;
    k.start(a, x.lo, x.hi);
    v = k;
    for (int e = 0; e < 2 && k.valid && ok; ++e) {
        if (k.opens()) take(kKeys);
        k.next(a);
    }
    while (v.valid && ok) {
        if (v.opens()) take(v.tail() ? max(v.g.L - v.key_tile() * kKeys, 0) : kKeys);
        v.next(a);
        if (!ok) break;
        if (k.valid) {
            if (k.opens()) take(kKeys);
            k.next(a);
        }
    }
    if (!ok && lane == 0) x.give_up();
}

template <int D>
__device__ __forceinline__ void gemm_s(const Ctx<D>& x, int qb, unsigned stage, int t) {  // S_t = Q K^T
    using C = Cfg<D>;
    const uint64_t da = umma_desc(x.sbase + C::off_q + (unsigned)qb * C::q_bytes);
    const uint64_t db = umma_desc(x.sbase + C::off_t + stage * C::t_bytes);
    const uint32_t hi = (uint32_t)(da >> 32), a_lo = (uint32_t)da, b_lo = (uint32_t)db;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (uint32_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
        mma_bf16_w(x.tmem + C::col_S + t * kKeys, a_lo + o, hi, b_lo + o, hi, idesc_bf16(128, kKeys), kk > 0);
    }
}
template <int D>
__device__ __forceinline__ void gemm_pv(const Ctx<D>& x, unsigned stage, int t, bool first) {  // O_t (+)= P_t V
    using C = Cfg<D>;
    const uint64_t db = umma_desc_mn(x.sbase + C::off_t + stage * C::t_bytes, C::blk);
    const uint32_t hi = (uint32_t)(db >> 32), b_lo = (uint32_t)db;
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_bf16_ts_w(x.tmem + C::col_O + t * D, x.tmem + C::col_S + t * kKeys + kk * 8, b_lo + (uint32_t)((kk * 2048) >> 4),
                      hi, idesc_bf16_bmn(128, D), (!first || kk > 0) ? 1 : 0);
}

// Warp 1, one thread.
template <int D>
__device__ __forceinline__ void role_mma(const Ctx<D>& x, const TcArgs& a) {
    using C = Cfg<D>;
    constexpr int NS = C::NS;
    auto* bars = x.bars;
    unsigned n = 0;               // tiles taken from the ring
    unsigned ks = 0, vs = 0;      // the ring's index of the current K and V tile
    unsigned qn = 0;              // row tiles taken
    unsigned pn[2] = {0, 0};      // operations of each slot
    unsigned on[2] = {0, 0};      // segments of each slot
    bool ok = true;
    auto wait = [&](uint64_t* b, unsigned parity) { return mbar_wait_suspend(b, parity & 1u, x.abort_flag); };
    auto scores = [&](const Ops& o) {
        if (o.opens()) ks = n++;
        if (!wait(&bars->full[ks % NS], ks / NS)) return false;
        if (o.q_opens()) {
            if (!wait(&bars->q_full[qn & 1u], qn / 2)) return false;
            ++qn;
        }
        tc_fence_after();
        const int t = o.slot();
        gemm_s<D>(x, o.q_buf(), ks % NS, t);
        mma_commit(&bars->s_full[t]);
        if (o.closes()) mma_commit(&bars->empty[ks % NS]);
        if (o.q_closes()) mma_commit(&bars->q_free[o.q_buf()]);
        return true;
    };
    Ops k, v;
    k.start(a, x.lo, x.hi);
    v = k;
    for (int e = 0; e < 2 && k.valid && ok; ++e) {
        ok = scores(k);
        k.next(a);
    }
    while (v.valid && ok) {
        const int t = v.slot();
        if (v.opens()) vs = n++;
        ok = wait(&bars->full[vs % NS], vs / NS);
        if (ok && v.opens() && v.tail()) ok = wait(&bars->fixed[vs % NS], vs / NS);
        ok = ok && wait(&bars->p_full[t], pn[t]++);
        // the epilogue has taken the slot's previous O
        if (ok && v.first()) {
            if (on[t] > 0) ok = wait(&bars->o_free[t], on[t] - 1);
            ++on[t];
        }
        if (!ok) break;
        tc_fence_after();
        gemm_pv<D>(x, vs % NS, t, v.first());
        mma_commit(&bars->pv_done[t]);
        if (v.last()) mma_commit(&bars->o_full[t]);
        if (v.closes()) mma_commit(&bars->empty[vs % NS]);
        v.next(a);
        if (k.valid) {
            // issued after the slot's product with V, which has read P out of these
            // columns by the time this one writes them (products run in issue order)
            ok = scores(k);
            k.next(a);
        }
    }
    if (!ok) x.give_up();
    mma_commit(&bars->drain);
    mbar_wait(&bars->drain, 0, kDrainNs);
}

// Softmax of slot t: thread `row` owns row `row` of the slot's row tile.
template <int D>
__device__ __forceinline__ void role_softmax(const Ctx<D>& x, const TcArgs& a, int t, int quad, int lane) {
    using C = Cfg<D>;
    auto* bars = x.bars;
    const int row = quad * 32 + lane;
    const unsigned tS = x.tmem + C::col_S + t * kKeys + ((unsigned)(quad * 32) << 16);
    const unsigned tO = x.tmem + C::col_O + t * D + ((unsigned)(quad * 32) << 16);
    float2* ml = reinterpret_cast<float2*>(x.sm + C::off_ml) + t * kRows;
    const float2 a2 = make_float2(a.scale, a.scale);
    unsigned cs = 0, on = 0;  // operations and segments of this slot
    float m = -INFINITY, l = 0.f;
    int end = 0;
    bool active = false, ok = true;
    Ops o;
    o.start(a, x.lo, x.hi);
    for (; o.valid && ok; o.next(a)) {
        if (o.slot() != t) continue;
        if (o.first()) {
            const int r = o.tile() * a.R + row;  // row of the unit
            const int rows = min(o.g.rows - o.tile() * a.R, a.R);
            active = quad * 32 < rows;
            end = row < rows ? (a.s.causal ? o.g.L - o.g.n + (o.g.row0 + r) / a.s.g + 1 : o.g.L) : 0;
            m = -INFINITY;
            l = 0.f;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_suspend(&bars->s_full[t], cs & 1u, x.abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (active) {  // the same for all lanes of a warp
            const int lim = end - o.key_tile() * kKeys;  // keys of this tile that the row sees
            const bool edge = __any_sync(0xffffffffu, lim < kKeys);
            uint32_t v[4][32];
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_ld32_nowait(tS + 32 * j, v[j]);
            tmem_wait_ld();
            if (edge) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * j + e >= lim) v[j][e] = 0xff800000u;
            }
            float best[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                best[j] = __uint_as_float(v[j][0]);
#pragma unroll
                for (int e = 1; e < 32; ++e) best[j] = fmaxf(best[j], __uint_as_float(v[j][e]));
            }
            const float mt = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])) * a.scale;
            if (o.first()) {
                m = mt;
            } else {
                const bool raise = mt > m + kRaise || (m == -INFINITY && mt > m);
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? ex2_approx(m - mt) : 1.f;
                    if (raise) m = mt;
                    l *= f;
                    // the slot's previous product has been added to O
                    ok = __all_sync(0xffffffffu, mbar_wait_suspend(&bars->pv_done[t], (cs - 1) & 1u, x.abort_flag));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float acc[16];
                        uint32_t w[16];
                        tmem_ld16(tO + c, acc);
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(acc[e] * f);
                        tmem_st16(tO + c, w);
                    }
                    tmem_wait_st();
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const float2 nb = make_float2(-base, -base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 y =
                        ffma2(make_float2(__uint_as_float(v[j][2 * e]), __uint_as_float(v[j][2 * e + 1])), a2, nb);
                    const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                    pk[e] = pack_bf16x2(p0, p1);
                    sum[e & 1] = fadd2(sum[e & 1], make_float2(p0, p1));
                }
                tmem_st16(tS + 16 * j, pk);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_wait_st();
        }
        ++cs;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
        if (o.last()) {
            // the epilogue has read the slot's previous (m, l)
            if (on > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_suspend(&bars->o_free[t], (on - 1) & 1u, x.abort_flag));
                if (!ok) break;
            }
            ++on;
            ml[row] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->den_full[t]);
        }
    }
    if (!ok && lane == 0) x.give_up();
}

// One row tile out: acc = f0 O_s0 + f1 O_s1 (the second slot only with `both`).
template <int D>
__device__ __forceinline__ bool put_tile(const Ctx<D>& x, const TcArgs& a, const Seg& g, int tile, int s0, bool both,
                                         unsigned (&on)[2], int quad, int lane) {
    using C = Cfg<D>;
    auto* bars = x.bars;
    const int row = quad * 32 + lane;
    const float2* ml = reinterpret_cast<const float2*>(x.sm + C::off_ml);
    for (int e = 0; e <= (both ? 1 : 0); ++e) {
        const int t = s0 ^ e;
        const bool got = mbar_wait_suspend(&bars->o_full[t], on[t] & 1u, x.abort_flag) &&
                         mbar_wait_suspend(&bars->den_full[t], on[t] & 1u, x.abort_flag);
        if (!__all_sync(0xffffffffu, got)) return false;
        ++on[t];
    }
    tc_fence_after();
    const float2 x0 = ml[s0 * kRows + row];
    const float2 x1 = both ? ml[(s0 ^ 1) * kRows + row] : make_float2(-INFINITY, 0.f);
    const float m = fmaxf(x0.x, x1.x), base = m == -INFINITY ? 0.f : m;
    float f0 = ex2_approx(x0.x - base), f1 = ex2_approx(x1.x - base);
    const float l = f0 * x0.y + f1 * x1.y;
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    const int rows = min(g.rows - tile * a.R, a.R), r = tile * a.R + row;
    const bool mine = row < rows;
    __nv_bfloat16* out = nullptr;
    float* part = nullptr;
    if (whole) {
        const float rcp = l > 0.f || l != l ? 1.f / l : 0.f;
        f0 *= rcp;
        f1 *= rcp;
        if (mine) {
            const int i = (g.row0 + r) / a.s.g, hq = g.h * a.s.g + (g.row0 + r - i * a.s.g);
            const int64_t tok = a.s.first_row(g.b) + i;
            out = a.O + tok * a.o_t + (int64_t)hq * a.o_h;
            if (a.lse) a.lse[tok * (a.s.Hkv * a.s.g) + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
    } else if (mine) {
        const int64_t at = ((int64_t)blockIdx.x * 2 + (g.t0 > 0 ? 0 : 1)) * kPagedTcRows + r;
        part = a.p.part + at * D;
        a.p.ml[at] = make_float2(m, l);
    }
    const unsigned lanes = (unsigned)(quad * 32) << 16;
    const bool live = quad * 32 < rows;  // the same for all lanes of a warp
    if (live) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            float u[16], w[16];
            tmem_ld16(x.tmem + C::col_O + s0 * D + c + lanes, u);
            if (both) tmem_ld16(x.tmem + C::col_O + (s0 ^ 1) * D + c + lanes, w);
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = both ? fmaf(f0, u[e], f1 * w[e]) : f0 * u[e];
            if (out) {
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(u[2 * e], u[2 * e + 1]);
                *reinterpret_cast<uint4*>(out + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            } else if (part) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float4*>(part + c + 4 * e) =
                        make_float4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(&bars->o_free[s0]);
        if (both) mbar_arrive(&bars->o_free[s0 ^ 1]);
    }
    return true;
}

template <int D>
__device__ __forceinline__ void role_epilogue(const Ctx<D>& x, const TcArgs& a, int quad, int lane, int64_t total,
                                              int active) {
    unsigned on[2] = {0, 0};
    bool ok = true;
    int4 join = make_int4(0, 0, 0, -1);
    Ops o;
    o.start(a, x.lo, x.hi);
    for (; o.valid && ok; o.next_seg(a)) {
        const int s0 = (int)(o.k0 & 1u);
        if (o.two)
            ok = put_tile<D>(x, a, o.g, 0, s0, false, on, quad, lane) &&
                 put_tile<D>(x, a, o.g, 1, s0 ^ 1, false, on, quad, lane);
        else
            ok = put_tile<D>(x, a, o.g, 0, s0, o.n > 1, on, quad, lane);
        if (o.g.t0 > 0 && o.g.t1 == o.g.nt) join = make_int4(o.g.b, o.g.h, o.g.t, block_of(total, active, o.g.unit_start));
    }
    if (!ok && lane == 0) x.give_up();
    if (quad == 0 && lane == 0) a.p.joins[blockIdx.x] = join;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcArgs a) {
    using C = Cfg<D>;
    constexpr int NS = C::NS;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Ctx<D> x;
    x.sm = sm;
    x.sbase = smem_u32(sm);
    x.bars = reinterpret_cast<Bars<NS>*>(sm + C::off_bar);
    x.abort_flag = &x.bars->abort;
    auto* bars = x.bars;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->q_free[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 4);  // one arrival per warp of the softmax group
            mbar_init(&bars->pv_done[t], 1);
            mbar_init(&bars->o_full[t], 1);
            mbar_init(&bars->o_free[t], 4);  // one arrival per warp of the epilogue group
            mbar_init(&bars->den_full[t], 4);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->fixed[s], 1);
            mbar_init(&bars->empty[s], 2);  // the tensor cores' last use, and warp 2
        }
        mbar_init(&bars->drain, 1);
        // the operand layouts need a 1024-byte aligned base
        bars->abort = (x.sbase & 1023u) ? 1 : 0;
        if (x.sbase & 1023u) atomicMax(&g_paged_tc_status, 3);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(C::tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    x.tmem = bars->tmem_base;
    const bool go = *x.abort_flag == 0;
    // the plan has been made
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t total = a.p.prefix[a.s.B];
    const int active = active_blocks(total, a.G), c = blockIdx.x;
    x.lo = c < active ? block_start(total, active, c) : 0;
    x.hi = c < active ? block_start(total, active, c + 1) : 0;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (go) {
            if (warp == 0) role_producer<D>(x, a, &tmQ, &tmK, &tmV, lane);
            else if (warp == 1 && lane == 0) role_mma<D>(x, a);
            else if (warp == 2) role_fix<D>(x, a, lane);
        }
        __syncwarp();
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        if (go) role_softmax<D>(x, a, (warp - 4) >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
        if (go) role_epilogue<D>(x, a, warp & 3, lane, total, active);
        else if (warp == 12 && lane == 0) a.p.joins[c] = make_int4(0, 0, 0, -1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(x.tmem), "r"(C::tmem_cols)
                     : "memory");
    }
}

__global__ void __launch_bounds__(kPlanThreads) paged_tc_plan_kernel(Shape s, Plan p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    plan_block<kKeys>(s, p, &g_paged_tc_status);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    return n;
}

template <int D>
Status run_tc(const PagedAttendRequest& q, cudaStream_t st) {
    using C = Cfg<D>;
    const int G = sm_count(), g = q.Hq / q.Hkv, R = kRows / g * g;
    Carve cv(q.ws, q.ws_bytes);
    TcArgs a{};
    carve_plan(cv, &a.p, q.B, G, kPagedTcRows, D);
    if (!cv.fits()) return Status::fail(4, "paged_attend: workspace too small");
    a.s = Shape{q.table, q.table_stride, q.W, q.seq_lens, q.cu_new, q.T, q.pages, (int)q.B, q.Hkv, g,
                q.page_size, 2 * R, q.causal};
    a.O = static_cast<__nv_bfloat16*>(q.O);
    a.o_t = q.o_t;
    a.o_h = q.o_h;
    a.lse = q.lse;
    a.scale = q.beta * 1.4426950408889634f;
    a.G = G;
    a.R = R;
    a.box = std::min(q.page_size, kKeys);
    CUtensorMap tmQ, tmK, tmV;
    const uint64_t Du = D, ps = (uint64_t)q.page_size, H = (uint64_t)q.Hkv, P = (uint64_t)q.pages;
    const uint32_t box = (uint32_t)a.box;
    const bool ok =
        make_tmap_4d(&tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q.Q, {Du, (uint64_t)g, H, (uint64_t)q.T},
                     {(uint64_t)q.q_h * 2, (uint64_t)q.q_h * 2 * g, (uint64_t)q.q_t * 2},
                     {64u, (uint32_t)g, 1u, (uint32_t)(R / g)}) &&
        make_tmap_4d(&tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q.K, {Du, ps, H, P},
                     {(uint64_t)q.k_r * 2, (uint64_t)q.k_h * 2, (uint64_t)q.k_p * 2}, {64u, box, 1u, 1u}) &&
        make_tmap_4d(&tmV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q.V, {Du, ps, H, P},
                     {(uint64_t)q.v_r * 2, (uint64_t)q.v_h * 2, (uint64_t)q.v_p * 2}, {64u, box, 1u, 1u});
    if (!ok) return Status::fail(3, "paged_attend: tensor map encoding failed");
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend: shared memory attribute");
    paged_tc_plan_kernel<<<1, kPlanThreads, 0, st>>>(a.s, a.p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend: plan launch");
    // a programmatic dependent of the plan: its prologue overlaps it
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)G);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::total;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_tc_kernel<D>, tmQ, tmK, tmV, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend launch");
    return launch_paged_join(PagedJoin{a.s, a.p, q.O, q.o_t, q.o_h, q.lse, G}, q.dtype, D, kPagedTcRows, st);
}

// A stride that a tensor map takes: a positive multiple of 16 bytes below 2^40,
// where the dimension has more than one entry.
bool map_stride(int64_t extent, int64_t stride) {
    return extent <= 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t(1) << 39));
}

}  // namespace

// bf16 with d in {64, 128}; pages that tile 128 keys in whole 8-row groups (or
// are tiled by them); pointers and strides that the copies and the 16-byte
// stores take; at most 128 query heads to a key head.  The rest runs on CUDA cores.
bool paged_attend_tc_supported(const PagedAttendRequest& q) {
    const int g = q.Hq / q.Hkv, ps = q.page_size;
    const uintptr_t ptrs = reinterpret_cast<uintptr_t>(q.Q) | reinterpret_cast<uintptr_t>(q.K) |
                           reinterpret_cast<uintptr_t>(q.V) | reinterpret_cast<uintptr_t>(q.O);
    return q.dtype == 1 && (q.d == 64 || q.d == 128) && q.pages > 0 && g <= kRows &&
           (ps % kKeys == 0 || (kKeys % ps == 0 && ps % 8 == 0)) && (ptrs & 15u) == 0 && map_stride(q.T, q.q_t) &&
           map_stride(q.Hq, q.q_h) && q.q_h < (int64_t(1) << 32) && map_stride(ps, q.k_r) && map_stride(q.Hkv, q.k_h) &&
           map_stride(q.pages, q.k_p) && map_stride(ps, q.v_r) && map_stride(q.Hkv, q.v_h) && map_stride(q.pages, q.v_p) &&
           (q.T <= 1 || q.o_t % 8 == 0) && (q.Hq <= 1 || q.o_h % 8 == 0);
}

Status launch_paged_attend_tc(const PagedAttendRequest& q, cudaStream_t st) {
    return q.d == 64 ? run_tc<64>(q, st) : run_tc<128>(q, st);
}

int read_paged_attend_tc_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_tc_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_paged_tc_status, &z, sizeof(int));
    }
    return v;
}

}  // namespace wildcat
