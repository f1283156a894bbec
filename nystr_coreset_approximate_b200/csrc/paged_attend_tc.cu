// paged_attend_tc.cu -- exact attention over a paged cache on the tensor cores
// (bf16, d in {64, 128}); the formulas are those of paged_attend.cu.
//
// One persistent block per SM walks its share of the key tiles (paged.cuh).  A
// row tile is R <= 128 query rows of one key head, whole tokens of g rows each
// (R = floor(128 / g) g), loaded by one TMA box that gathers the g heads; a
// unit has up to two of them.  The work is a sequence of operations, numbered
// k = 0, 1, ...; operation k takes one row tile and one tile of 128 keys in slot
// k & 1 (a softmax group, and P and O in tensor memory):
//     S = Q K^T          (tcgen05.mma, both operands in shared memory)
//     P = 2^(beta log2e S - m), rounded to bf16
//     O += P V           (A from tensor memory, V as it lies: keys by columns)
// A unit with two row tiles runs both against each key tile (one slot each, one
// load of K and V for 2 R rows: the tensor cores bound it); a unit with one, a
// decoded token's or a short chunk's, runs successive key tiles in the two slots
// with a running maximum and sum of its own for each (HBM bounds it), which the
// epilogue adds up.  S(k) waits for the scores of k - 1 to be taken, PV(k) for P(k),
// across units.  The slots share one place for scores: a group takes its scores
// into registers at once (128 of a thread's), which frees it for the other
// slot's next product, so that S(k + 2) does not wait for P(k) and both groups
// exponentiate without a pause.  Warp roles:
//   warp 0      cuts the block's share into segments (one unit's key tiles), hands
//               them to the other roles through a ring, and copies K tiles: page
//               lookups (one lane per page) and TMA
//   warp 1      tensor cores, one thread: S(k + 2), then PV(k).  The tensor pipe
//               holds only a few products and runs dry when the code between two
//               issues is long; two issuing warps are no way out, products of both
//               kinds in turn run at half the rate
//   warp 2      follows the V tiles and zeroes their rows at or past the request's
//               length: what the page holds there may be NaN, and 0 NaN is NaN
//   warp 3      copies Q and V tiles
//   warps 4-7   softmax of slot 0, warps 8-11 of slot 1, one row per thread.  The
//               exponentials are formed with the maximum of the tiles before;
//               only when a row's sum over the tile says that it has grown far is
//               the maximum raised, O rescaled and the tile done again (float32
//               sums hold 2^16, and a bf16 P is as exact there as at 1), so that
//               the tile's maximum is not on the path from S to P
//   warps 12-15 epilogue: O / l as bf16, or a partial sum of a unit that is cut
// P is rounded to bf16 for the product (the operand type of V); the sum l is
// float32 of the unrounded P.
//
// Every wait is bounded (2 s) and gives up when another role has given up; an
// expired wait records WILDCAT_ERR_TIMEOUT in the device status word, the block
// drains its copies and products (bounded), marks its pieces as missing, frees its
// tensor memory and returns.  No load uses cluster multicast.
//
// Measured: 2,048 new tokens behind 30,001 (32/8 heads of 128) 0.91 to 1.05 ms, 1.0 to
// 1.15 PFLOP/s in 1.32 M cycles, under the power cap; one token each of 32 requests of
// 20,000 to 32,768 0.55 to 0.60 ms, 5.5 to 6.0 TB/s of a copy's 6.6; short units (1 to 6
// key tiles, d = 64) 2,900 cycles an operation instead of 1,450, waiting for instructions.
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
// registers per thread after the split: 96 + 2 * 168 + 80 = 512 per lane of a
// sub-partition, the 4 * 128 it was launched with
constexpr int kRegsLow = 96, kRegsSoftmax = 168, kRegsEpilogue = 80;
static_assert(kRegsLow + 2 * kRegsSoftmax + kRegsEpilogue == 512, "register split");
constexpr unsigned long long kDrainNs = 100000000ull;
constexpr int kItems = 8;  // segments in the ring
constexpr int kLead = 5;   // segments that warp 2 hands out ahead of its own
constexpr float kRaise = 65536.f;  // a row's sum of one tile above which its maximum is raised
constexpr int kAhead = 3;  // key tiles between the first touch of their page ids and their use
constexpr int kPagesOfTile = kKeys / 8;

// One segment: key tiles [t0, t1) of a unit; t1 == t0 ends the ring.
struct Item {
    int b, h, t, n, L, row0, rows, t0, t1, nt, first, join;
};

template <int NK, int NV>
struct Bars {
    uint64_t q_full[2], q_free[2];
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_fixed[NV], v_empty[NV];
    uint64_t s_go, s_full[2], p_full[2], pv_done[2], o_full[2], o_free[2], den_full[2];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain, never;
    unsigned tmem_base;
    int abort;
};

template <int D>
struct Cfg {
    static constexpr int KB = D / 64;                   // 128-byte blocks of a row
    static constexpr int NK = D == 128 ? 3 : 6;         // stages of K tiles: two operations more are on their way
    static constexpr int NV = D == 128 ? 2 : 5;         // stages of V tiles
    static constexpr uint32_t q_bytes = kRows * D * 2;  // one row tile
    static constexpr uint32_t t_bytes = kKeys * D * 2;  // one tile of K or V
    static constexpr uint32_t blk = kKeys * 128;        // one 128-byte block of a tile
    static constexpr uint32_t off_q = 0;
    static constexpr uint32_t off_k = off_q + 2 * q_bytes;
    static constexpr uint32_t off_v = off_k + NK * t_bytes;
    static constexpr uint32_t off_ml = off_v + NV * t_bytes;  // (m, l) of each slot's rows
    static constexpr uint32_t off_items = off_ml + 2 * kRows * 8;
    static constexpr uint32_t off_ids = off_items + kItems * (uint32_t)sizeof(Item);  // a tile's pages: K, V
    static constexpr uint32_t off_bar = off_ids + 2 * kPagesOfTile * 4;
    static constexpr uint32_t total = off_bar + (uint32_t)sizeof(Bars<NK, NV>);
    static constexpr unsigned tmem_cols = 512;
    static constexpr unsigned col_O = 0;      // O of slot t at t * D
    static constexpr unsigned col_S = 2 * D;  // S
    static constexpr unsigned col_P = 2 * D + kKeys;  // P of slot t, two bf16 to a column, at col_P + 64 t
    static_assert(col_P + kKeys <= tmem_cols, "tensor memory");
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
    unsigned long long stall_ns;  // test hook, 0 = off: warp 2 of block 0 waits this long on `never`
};

template <int D>
struct Ctx {
    unsigned char* sm;
    unsigned sbase, tmem;
    Bars<Cfg<D>::NK, Cfg<D>::NV>* bars;
    volatile int* abort_flag;
    __device__ void give_up() const {
        *abort_flag = 1;
        atomicMax(&g_paged_tc_status, 5);
    }
    // a wait of a whole warp
    __device__ __forceinline__ bool wait(uint64_t* b, unsigned parity) const {
        return __all_sync(0xffffffffu, mbar_wait_suspend(b, parity & 1u, abort_flag));
    }
    __device__ __forceinline__ bool wait_one(uint64_t* b, unsigned parity) const {
        return mbar_wait_suspend(b, parity & 1u, abort_flag);
    }
    __device__ __forceinline__ Item* item(unsigned s) const {
        return reinterpret_cast<Item*>(sm + Cfg<D>::off_items) + s % kItems;
    }
    // segment s once it is in the ring
    __device__ __forceinline__ bool item_wait(unsigned s) const { return wait(&bars->item_full[s % kItems], s / kItems); }
    // this warp has read segment s
    __device__ __forceinline__ void item_done(unsigned s, int lane) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[s % kItems]);
    }
};
constexpr int kItemReaders = 4 + 8 + 4;  // warps 0 to 3, the softmax groups, the epilogue

// A place in a ring of N stages and the parity of its use.
template <int N>
struct Ring {
    int s = 0;
    unsigned ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// The page ids of a segment's key tiles, one tile after the other: lane p has page p
// of a tile.
struct Pages {
    const int32_t* row;  // the request's row of the table
    int count;           // its pages
    int ix, sub;         // the entry of the tile read next, and which tile of its page that is
    int boxes, tiles;    // pages of a tile; tiles of a page
    int last;            // the entry read last, -1 for none

    __device__ __forceinline__ void of(const TcArgs& a, const Item& g, int lane) {
        row = a.s.table + (int64_t)g.b * a.s.table_stride;
        count = ((unsigned)g.L + (unsigned)a.s.page_size - 1u) / (unsigned)a.s.page_size;
        boxes = kKeys / a.box;
        tiles = (unsigned)a.s.page_size / (unsigned)a.box;
        ix = boxes > 1 ? g.t0 * boxes + lane : (unsigned)g.t0 / (unsigned)tiles;
        sub = boxes > 1 ? 0 : g.t0 - ix * tiles;
        if (lane >= boxes) count = 0;
        if (lane == 0)
            for (int e = 0; e < kAhead; ++e) touch(e);
    }
    // the next tile's entry (not looked at yet: it may be on its way)
    __device__ __forceinline__ int read() {
        const bool there = ix < count;
        const int id = there ? __ldg(row + ix) : 0;
        last = there ? ix : -1;
        if (boxes > 1) {
            ix += boxes;
        } else if (++sub == tiles) {
            sub = 0;
            ++ix;
        }
        return id;
    }
    // what the copy takes for an entry that was read at `at`: past the pool it fills zeros
    __device__ __forceinline__ int check(const TcArgs& a, int id, int at) const {
        if (at < 0) return (int)a.s.pages;
        if (id >= 0 && id < a.s.pages) return id;
        atomicMax(&g_paged_tc_status, 1);
        return (int)a.s.pages;
    }
    // bring the entries of a later tile into L2: a read from HBM takes as long as a tile's copy
    __device__ __forceinline__ void touch(int ahead) const {
        const int at = ix + ahead * boxes;
        if (at < count) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
    }
};

// One tile of K or V, page by page, by one lane; `ids` holds the pages in shared memory.
template <int D>
__device__ __forceinline__ void copy_pages(const CUtensorMap* tm, unsigned dst, unsigned page_bytes, int row, int h, int boxes,
                                           const int* ids, uint64_t* full) {
    using C = Cfg<D>;
    mbar_expect_tx(full, C::t_bytes);
    if (boxes >= 4) {
#pragma unroll 1
        for (int p = 0; p < boxes; p += 4, dst += 4 * page_bytes) {
            const int4 id = *reinterpret_cast<const int4*>(ids + p);
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb) {
                tma_load_4d(dst + kb * C::blk, tm, kb * 64, row, h, id.x, full);
                tma_load_4d(dst + page_bytes + kb * C::blk, tm, kb * 64, row, h, id.y, full);
                tma_load_4d(dst + 2 * page_bytes + kb * C::blk, tm, kb * 64, row, h, id.z, full);
                tma_load_4d(dst + 3 * page_bytes + kb * C::blk, tm, kb * 64, row, h, id.w, full);
            }
        }
    } else {
#pragma unroll 1
        for (int p = 0; p < boxes; ++p, dst += page_bytes)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb) tma_load_4d(dst + kb * C::blk, tm, kb * 64, row, h, ids[p], full);
    }
}

// Warps 0 and 3: the segments and the K tiles (V false), or each segment's Q tiles
// and its V tiles.
template <int D, bool V>
__device__ __forceinline__ void role_copy(const Ctx<D>& x, const TcArgs& a, const CUtensorMap* tmQ, const CUtensorMap* tm,
                                          int lane, const Share& share) {
    using C = Cfg<D>;
    constexpr int N = V ? C::NV : C::NK;
    auto* bars = x.bars;
    uint64_t* full = V ? bars->v_full : bars->k_full;
    uint64_t* empty = V ? bars->v_empty : bars->k_empty;
    const unsigned base = x.sbase + (V ? C::off_v : C::off_k);
    if (lane == 0) {
        prefetch_tmap(tm);
        if (V) prefetch_tmap(tmQ);
    }
    Ring<N> r;
    unsigned n = 0, qn = 0;  // tiles and row tiles issued
    bool ok = true;
    Walk<kKeys> w;
    unsigned pushed = 0;
    bool more = !V;
    if (!V) w.start(a.s, share);
    auto push = [&]() {  // one more segment into the ring
        if (pushed >= kItems && !x.wait(&bars->item_empty[pushed % kItems], pushed / kItems - 1)) return false;
        Seg g;
        more = w.next(a.s, g);
        if (lane == 0) {
            Item* it = x.item(pushed);
            if (more) {
                const bool ends = g.t0 > 0 && g.t1 == g.nt;  // the last piece of a cut unit
                *it = Item{g.b, g.h, g.t, g.n, g.L, g.row0, g.rows, g.t0, g.t1, g.nt, a.s.first_row(g.b),
                           ends ? share.line.block(g.first_end) : -1};
            } else {
                it->t0 = it->t1 = 0;
            }
            mbar_arrive(&bars->item_full[pushed % kItems]);
        }
        __syncwarp();
        ++pushed;
        return true;
    };
    Item g;
    g.t1 = 0;
    Pages pages;
    int kt = 0, next = 0;
    int* ids = reinterpret_cast<int*>(x.sm + C::off_ids) + (V ? kPagesOfTile : 0);
    for (unsigned s = 0;;) {
#pragma unroll 1
        for (int e = 0; e < 2 && more && pushed < s + kLead && ok; ++e) ok = push();
        if (!ok) break;
        if (kt == g.t1) {  // the next segment
            ok = x.item_wait(s);
            if (!ok) break;
            g = *x.item(s);
            x.item_done(s, lane);
            if (g.t1 == g.t0) break;
            ++s;
            kt = g.t0;
            pages.of(a, g, lane);
            if (V) {
                const int tiles = g.rows > a.R ? 2 : 1;
#pragma unroll 1
                for (int e = 0; e < tiles && ok; ++e, ++qn) {
                    const unsigned qb = qn & 1u;
                    if (qn >= 2) ok = x.wait(&bars->q_free[qb], qn / 2 - 1);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect_tx(&bars->q_full[qb], (unsigned)a.R * 128u * C::KB);
                        const int token = g.first + (g.row0 + e * a.R) / a.s.g;
#pragma unroll
                        for (int kb = 0; kb < C::KB; ++kb)
                            tma_load_4d(x.sbase + C::off_q + qb * C::q_bytes + kb * (kRows * 128), tmQ, kb * 64, 0, g.h, token,
                                        &bars->q_full[qb]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            next = pages.read();
        }
        if (lane == 0) pages.touch(kAhead);
        const int id = pages.check(a, next, pages.last);
        const int row = pages.boxes > 1 ? 0 : (kt - (pages.ix - (pages.sub == 0 ? 1 : 0)) * pages.tiles) * kKeys;
        if (lane < kPagesOfTile) ids[lane] = id;
        next = pages.read();
        if (n >= N) ok = x.wait(&empty[r.s], r.ph ^ 1u);
        if (!ok) break;
        __syncwarp();
        if (elect_one())
            copy_pages<D>(tm, base + (unsigned)r.s * C::t_bytes, (unsigned)a.box * 128u, row, g.h, pages.boxes, ids, &full[r.s]);
        __syncwarp();
        r.next();
        ++n;
        ++kt;
    }
    if (!ok && lane == 0) x.give_up();
    __syncwarp();
    if (*x.abort_flag) {
        // copies still in flight land before the block's shared memory is released
        for (unsigned c = n > N ? n - N : 0; c < n; ++c) mbar_wait(&full[c % N], (c / N) & 1u, kDrainNs);
        if (V)
            for (unsigned c = qn > 2 ? qn - 2 : 0; c < qn; ++c) mbar_wait(&bars->q_full[c & 1u], (c / 2) & 1u, kDrainNs);
    }
}

// S_t = Q K^T and O_t (+)= P_t V, one thread.
template <int D>
__device__ __forceinline__ void gemm_s(unsigned tmem_s, uint32_t q_lo, uint32_t k_lo, uint32_t hi) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (uint32_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
        mma_bf16_w(tmem_s, q_lo + o, hi, k_lo + o, hi, idesc_bf16(128, kKeys), kk > 0);
    }
}
template <int D>
__device__ __forceinline__ void gemm_pv(unsigned tmem_o, unsigned tmem_p, uint32_t v_lo, uint32_t hi, bool first) {
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_bf16_ts_w(tmem_o, tmem_p + kk * 8, v_lo + (uint32_t)((kk * 2048) >> 4), hi, idesc_bf16_bmn(128, D),
                      (!first || kk > 0) ? 1 : 0);
}

// The operations of a segment as warp 1 sees them.
struct OpCursor {
    unsigned s = 0;  // segment
    int i, n;        // operation of n
    bool two;
    __device__ __forceinline__ bool opens() const { return !two || !(i & 1); }  // first use of the key tile
    __device__ __forceinline__ bool closes() const { return !two || (i & 1); }  // last use
    __device__ __forceinline__ bool q_opens() const { return i < (two ? 2 : 1); }
    __device__ __forceinline__ bool q_closes() const { return i >= n - (two ? 2 : 1); }
    __device__ __forceinline__ bool first() const { return i < 2; }  // of its slot in the segment
    __device__ __forceinline__ bool last() const { return i >= n - 2; }
    // the segment s; n = 0 after the last
    template <int D>
    __device__ __forceinline__ bool load(const Ctx<D>& x, int R) {
        if (!x.wait_one(&x.bars->item_full[s % kItems], s / kItems)) return false;
        const Item* it = x.item(s);
        two = it->rows > R;
        n = (it->t1 - it->t0) << (two ? 1 : 0);
        i = 0;
        return true;
    }
};

// Warp 1, one thread.
template <int D>
__device__ __forceinline__ void role_mma(const Ctx<D>& x, const TcArgs& a) {
    using C = Cfg<D>;
    auto* bars = x.bars;
    const uint64_t dk = umma_desc(x.sbase + C::off_k), dv = umma_desc_mn(x.sbase + C::off_v, C::blk);
    const uint32_t q_lo = (uint32_t)umma_desc(x.sbase + C::off_q), k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
    const uint32_t k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
    Ring<C::NK> kr;
    Ring<C::NV> vr;
    int ks = 0, vs = 0;         // stages of the current K and V tile
    unsigned sn = 0, pn = 0;    // operations whose S, whose PV was issued
    unsigned qn = 0, q0 = 0;    // row tiles taken; row tiles before the S cursor's segment
    unsigned on[2] = {0, 0};    // accumulations of each slot
    OpCursor k, v;
    bool ok = k.load(x, a.R);
    v = k;
    auto scores = [&]() {
        if (k.opens()) {
            ks = kr.s;
            if (!x.wait_one(&bars->k_full[kr.s], kr.ph)) return false;
            kr.next();
        }
        if (k.q_opens()) {
            if (!x.wait_one(&bars->q_full[qn & 1u], qn / 2)) return false;
            ++qn;
        }
        // the scores before are in registers
        if (sn > 0 && !x.wait_one(&bars->s_go, sn - 1)) return false;
        const unsigned qb = (q0 + (k.two ? k.i & 1 : 0)) & 1u;
        tc_fence_after();
        gemm_s<D>(x.tmem + C::col_S, q_lo + qb * (C::q_bytes >> 4), k_lo + (uint32_t)ks * (C::t_bytes >> 4), k_hi);
        mma_commit(&bars->s_full[sn & 1u]);
        if (k.closes()) mma_commit(&bars->k_empty[ks]);
        if (k.q_closes()) mma_commit(&bars->q_free[qb]);
        ++sn;
        if (++k.i == k.n) {
            q0 += k.two ? 2 : 1;
            ++k.s;
            return k.load(x, a.R);
        }
        return true;
    };
    // Both cursors inside one segment of two row tiles: the same without its conditions, a
    // key tile at a time.  The code of the general form between two products takes longer
    // than they do.
    auto pairs = [&]() {
        const unsigned t0 = pn & 1u;
        const uint32_t qa = q_lo + (q0 & 1u) * (C::q_bytes >> 4), qb = q_lo + (~q0 & 1u) * (C::q_bytes >> 4);
        const unsigned o0 = x.tmem + C::col_O + t0 * D, o1 = x.tmem + C::col_O + (t0 ^ 1u) * D;
        const unsigned p0 = x.tmem + C::col_P + t0 * (kKeys / 2), p1 = x.tmem + C::col_P + (t0 ^ 1u) * (kKeys / 2);
        uint64_t *s_full0 = &bars->s_full[t0], *s_full1 = &bars->s_full[t0 ^ 1u];
        uint64_t *p_full0 = &bars->p_full[t0], *p_full1 = &bars->p_full[t0 ^ 1u];
        uint64_t *pv_done0 = &bars->pv_done[t0], *pv_done1 = &bars->pv_done[t0 ^ 1u];
        unsigned par0 = pn / 2, par1 = (pn + 1) / 2;
        unsigned go = sn - 1;
        const int m = (k.n - 2 - k.i) / 2;
#pragma unroll 1
        for (int e = 0; e < m; ++e) {
            const uint32_t kd = k_lo + (uint32_t)kr.s * (C::t_bytes >> 4), vd = v_lo + (uint32_t)vr.s * (C::t_bytes >> 4);
            if (!x.wait_one(&bars->k_full[kr.s], kr.ph) || !x.wait_one(&bars->s_go, go)) return false;
            tc_fence_after();
            gemm_s<D>(x.tmem + C::col_S, qa, kd, k_hi);
            mma_commit(s_full0);
            if (!x.wait_one(&bars->v_fixed[vr.s], vr.ph) || !x.wait_one(p_full0, par0)) return false;
            tc_fence_after();
            gemm_pv<D>(o0, p0, vd, v_hi, false);
            mma_commit(pv_done0);
            if (!x.wait_one(&bars->s_go, go + 1)) return false;
            tc_fence_after();
            gemm_s<D>(x.tmem + C::col_S, qb, kd, k_hi);
            mma_commit(s_full1);
            mma_commit(&bars->k_empty[kr.s]);
            if (!x.wait_one(p_full1, par1)) return false;
            tc_fence_after();
            gemm_pv<D>(o1, p1, vd, v_hi, false);
            mma_commit(pv_done1);
            mma_commit(&bars->v_empty[vr.s]);
            kr.next();
            vr.next();
            go += 2;
            ++par0;
            ++par1;
        }
        k.i += 2 * m;
        v.i += 2 * m;
        sn += 2 * m;
        pn += 2 * m;
        return true;
    };
#pragma unroll 1
    for (int step = 0; ok && v.n > 0; ++step) {
        if (v.two && v.i == 2 && k.s == v.s && k.n - k.i > 2) {
            ok = pairs();
            if (!ok) break;
        }
        if (k.n > 0) ok = scores();
        if (step < 2) continue;
        const unsigned t = pn & 1u;
        if (ok && v.opens()) {
            vs = vr.s;
            ok = x.wait_one(&bars->v_fixed[vr.s], vr.ph);
            vr.next();
        }
        if (ok && v.first()) {  // the epilogue has taken the slot's previous O
            if (on[t] > 0) ok = x.wait_one(&bars->o_free[t], on[t] - 1);
            ++on[t];
        }
        if (!ok || !x.wait_one(&bars->p_full[t], pn / 2)) {
            ok = false;
            break;
        }
        tc_fence_after();
        gemm_pv<D>(x.tmem + C::col_O + t * D, x.tmem + C::col_P + t * (kKeys / 2), v_lo + (uint32_t)vs * (C::t_bytes >> 4), v_hi,
                   v.first());
        mma_commit(&bars->pv_done[t]);
        if (v.last()) mma_commit(&bars->o_full[t]);
        if (v.closes()) mma_commit(&bars->v_empty[vs]);
        ++pn;
        if (++v.i == v.n) {
            mbar_arrive(&bars->item_empty[v.s % kItems]);
            ++v.s;
            ok = v.load(x, a.R);
        }
    }
    if (!ok) x.give_up();
    mma_commit(&bars->drain);
    mbar_wait(&bars->drain, 0, kDrainNs);
}

// Warp 2.
template <int D>
__device__ __forceinline__ void role_tail(const Ctx<D>& x, const TcArgs& a, int lane) {
    using C = Cfg<D>;
    Ring<C::NV> r;
    bool ok = true;
    for (unsigned s = 0; ok; ++s) {
        ok = x.item_wait(s);
        if (!ok) break;
        const int t0 = x.item(s)->t0, t1 = x.item(s)->t1, L = x.item(s)->L;
        x.item_done(s, lane);
        if (t0 == t1) break;
        if (a.stall_ns && s == 0 && blockIdx.x == 0) {  // copies and products of other roles are on their way
            ok = __all_sync(0xffffffffu, mbar_wait(&x.bars->never, 0, a.stall_ns));
            if (!ok) break;
        }
        for (int kt = t0; kt < t1; ++kt, r.next()) {
            ok = x.wait(&x.bars->v_full[r.s], r.ph);
            if (!ok) break;
            if ((kt + 1) * kKeys > L) {
                const int keep = max(L - kt * kKeys, 0);
                unsigned char* tile = x.sm + C::off_v + (unsigned)r.s * C::t_bytes;
                for (int e = lane; e < (kKeys - keep) * 8; e += 32)
#pragma unroll
                    for (int kb = 0; kb < C::KB; ++kb)
                        *reinterpret_cast<uint4*>(tile + kb * C::blk + keep * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&x.bars->v_fixed[r.s]);
        }
    }
    if (!ok && lane == 0) x.give_up();
}

// Softmax of slot t: thread `row` owns row `row` of the slot's row tile.
template <int D>
__device__ __forceinline__ void role_softmax(const Ctx<D>& x, const TcArgs& a, unsigned t, int quad, int lane) {
    using C = Cfg<D>;
    auto* bars = x.bars;
    const int row = quad * 32 + lane;
    const unsigned tS = x.tmem + C::col_S + ((unsigned)(quad * 32) << 16);
    const unsigned tP = x.tmem + C::col_P + t * (kKeys / 2) + ((unsigned)(quad * 32) << 16);
    const unsigned tO = x.tmem + C::col_O + t * D + ((unsigned)(quad * 32) << 16);
    float2* ml = reinterpret_cast<float2*>(x.sm + C::off_ml) + t * kRows;
    const float2 a2 = make_float2(a.scale, a.scale);
    unsigned cs = 0, on = 0;  // operations and segments of this slot
    unsigned k0 = 0;          // operations before the segment
    bool ok = true;
    for (unsigned s = 0; ok; ++s) {
        ok = x.item_wait(s);
        if (!ok) break;
        int lim, step, ops, rows;
        bool mine;
        {
            const Item g = *x.item(s);
            x.item_done(s, lane);
            if (g.t1 == g.t0) break;
            const bool two = g.rows > a.R;
            const int n = (g.t1 - g.t0) << (two ? 1 : 0), i0 = (int)((t ^ k0) & 1u);
            k0 += n;
            ops = (n - i0 + 1) >> 1;
            const int tile = two ? i0 : 0, r = tile * a.R + row;
            rows = min(g.rows - tile * a.R, a.R);
            // rows past the unit's are formed like the others and not used
            const int end = a.s.causal && row < rows ? g.L - g.n + (g.row0 + r) / a.s.g + 1 : g.L;
            mine = row < rows;
            lim = end - (g.t0 + (two ? 0 : i0)) * kKeys;  // keys of the tile that the row sees
            step = two ? kKeys : 2 * kKeys;
        }
        if (ops <= 0) continue;
        const bool active = quad * 32 < rows;  // the same for all lanes of a warp
        float m = -INFINITY, l = 0.f;
        for (int c = 0; c < ops; ++c, lim -= step) {
            ok = x.wait(&bars->s_full[t], cs);
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
            if (active) {
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld32_nowait(tS + 32 * j, v[j]);
                tmem_wait_ld();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_go);
            // the slot's product before has read P, and been added to O
            if (cs > 0) {
                ok = x.wait(&bars->pv_done[t], cs - 1);
                if (!ok) break;
                tc_fence_after();
            }
            ++cs;
            if (active) {
                if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int left = lim - 32 * j;
                        const uint32_t seen = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen >> e & 1u)) v[j][e] = 0xff800000u;
                    }
                }
                float sum;
                // Once with the maximum so far, and once more where it has to be raised; the first
                // tile begins with its maximum.  (One copy of this code: the roles' loops together
                // have to stay in the instruction cache.)
                bool raise = c == 0;
#pragma unroll 1
                for (;;) {
                    if (raise) {
                        float best[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            best[j] = __uint_as_float(v[j][0]);
#pragma unroll
                            for (int e = 1; e < 32; ++e) best[j] = fmaxf(best[j], __uint_as_float(v[j][e]));
                        }
                        const float mt = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])) * a.scale;
                        const float mn = fmaxf(m, mt);
                        if (c > 0) {
                            const float f = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
                            l *= f;
#pragma unroll 1
                            for (int cc = 0; cc < D; cc += 16) {
                                float acc[16];
                                uint32_t w[16];
                                tmem_ld16(tO + cc, acc);
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(acc[e] * f);
                                tmem_st16(tO + cc, w);
                            }
                        }
                        m = mn;
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    const float2 nb = make_float2(-base, -base);
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // P, and its sum
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y =
                                ffma2(make_float2(__uint_as_float(v[j][2 * e]), __uint_as_float(v[j][2 * e + 1])), a2, nb);
                            const float2 pr = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                            pk[e] = pack_bf16x2(pr.x, pr.y);
                            part[e & 1] = fadd2(part[e & 1], pr);
                        }
                        tmem_st16(tP + 16 * j, pk);
                    }
                    sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    if (raise) break;
                    raise = __any_sync(0xffffffffu, mine && (sum > kRaise || (m == -INFINITY && lim > 0)));
                    if (!raise) break;
                }
                l += sum;
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[t]);
        }
        if (!ok) break;
        // the epilogue has read the slot's previous (m, l)
        if (on > 0) {
            ok = x.wait(&bars->o_free[t], on - 1);
            if (!ok) break;
        }
        ++on;
        ml[row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->den_full[t]);
    }
    if (!ok && lane == 0) x.give_up();
}

// One row tile out: acc = f0 O_s0 + f1 O_s1 (the second slot only with `both`).
template <int D>
__device__ __forceinline__ bool put_tile(const Ctx<D>& x, const TcArgs& a, const Item& g, int tile, int s0, bool both,
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
            const int64_t tok = g.first + i;
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
__device__ __forceinline__ void role_epilogue(const Ctx<D>& x, const TcArgs& a, int quad, int lane) {
    unsigned on[2] = {0, 0};
    unsigned k0 = 0;
    bool ok = true;
    int4 join = make_int4(0, 0, 0, kNoJoin);
    for (unsigned s = 0; ok; ++s) {
        ok = x.item_wait(s);
        if (!ok) break;
        const Item g = *x.item(s);
        x.item_done(s, lane);
        if (g.t1 == g.t0) break;
        const int s0 = (int)(k0 & 1u), n = g.t1 - g.t0;
        const int tiles = g.rows > a.R ? 2 : 1;
#pragma unroll 1
        for (int e = 0; e < tiles && ok; ++e) ok = put_tile<D>(x, a, g, e, s0 ^ e, tiles == 1 && n > 1, on, quad, lane);
        if (tiles == 1) k0 += n;
        if (g.join >= 0) join = make_int4(g.b, g.h, g.t, g.join);
    }
    if (!ok && lane == 0) x.give_up();
    if (quad == 0 && lane == 0) a.p.joins[blockIdx.x] = ok ? join : make_int4(0, 0, 0, kGaveUp);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Ctx<D> x;
    x.sm = sm;
    x.sbase = smem_u32(sm);
    x.bars = reinterpret_cast<Bars<C::NK, C::NV>*>(sm + C::off_bar);
    x.abort_flag = &x.bars->abort;
    auto* bars = x.bars;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join's prologue
    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->q_free[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->pv_done[t], 1);
            mbar_init(&bars->p_full[t], 4);  // the warps of the softmax group
            mbar_init(&bars->o_full[t], 1);
            mbar_init(&bars->o_free[t], 4);  // one arrival per warp of the epilogue group
            mbar_init(&bars->den_full[t], 4);
        }
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_fixed[s], 1);
            mbar_init(&bars->v_empty[s], 1);
        }
        for (int s = 0; s < kItems; ++s) {
            mbar_init(&bars->item_full[s], 1);
            mbar_init(&bars->item_empty[s], kItemReaders);
        }
        mbar_init(&bars->s_go, 4);  // the warps that took the scores
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->never, 1);
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
    ShareScratch* scratch = reinterpret_cast<ShareScratch*>(sm + C::off_ml);
    find_share<kKeys>(a.s, a.G, scratch, &g_paged_tc_status);
    __syncthreads();
    const Share share = scratch->share;
    __syncthreads();  // the softmax groups write there

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (go) {
            if (warp == 0) role_copy<D, false>(x, a, &tmQ, &tmK, lane, share);
            else if (warp == 1) {
                if (elect_one()) role_mma<D>(x, a);
                __syncwarp();
            }
            else if (warp == 2) role_tail<D>(x, a, lane);
            else role_copy<D, true>(x, a, &tmQ, &tmV, lane, share);
        }
        __syncwarp();
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        if (go) role_softmax<D>(x, a, (unsigned)(warp - 4) >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
        if (go) role_epilogue<D>(x, a, warp & 3, lane);
        else if (warp == 12 && lane == 0) a.p.joins[blockIdx.x] = make_int4(0, 0, 0, kGaveUp);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(x.tmem), "r"(C::tmem_cols)
                     : "memory");
    }
}

std::atomic<unsigned long long> g_stall_ns{0};  // test hook

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
    carve_plan(cv, &a.p, G, kPagedTcRows, D);
    if (!cv.fits()) return Status::fail(4, "paged_attend: workspace too small");
    a.s = Shape{q.table, q.table_stride, q.W, q.seq_lens, q.cu_new, q.T, q.pages, (int)q.B, q.Hkv, g,
                q.page_size, 2 * R, R, 1, q.causal};
    a.O = static_cast<__nv_bfloat16*>(q.O);
    a.o_t = q.o_t;
    a.o_h = q.o_h;
    a.lse = q.lse;
    a.scale = q.beta * 1.4426950408889634f;
    a.G = G;
    a.R = R;
    a.box = std::min(q.page_size, kKeys);
    a.stall_ns = g_stall_ns.load(std::memory_order_relaxed);
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
    cudaError_t e = allow_smem<paged_tc_kernel<D>>((int)C::total);
    if (e != cudaSuccess) return Status::cuda(e, "paged_attend: shared memory attribute");
    paged_tc_kernel<D><<<G, kThreads, C::total, st>>>(tmQ, tmK, tmV, a);
    e = cudaGetLastError();
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
           map_stride(q.Hq, q.q_h) && q.q_h < (int64_t(1) << 31) && map_stride(ps, q.k_r) && map_stride(q.Hkv, q.k_h) &&
           map_stride(q.pages, q.k_p) && map_stride(ps, q.v_r) && map_stride(q.Hkv, q.v_h) && map_stride(q.pages, q.v_p) &&
           (q.T <= 1 || q.o_t % 8 == 0) && (q.Hq <= 1 || q.o_h % 8 == 0);
}

Status launch_paged_attend_tc(const PagedAttendRequest& q, cudaStream_t st) {
    return q.d == 64 ? run_tc<64>(q, st) : run_tc<128>(q, st);
}

void set_paged_attend_force_timeout(unsigned long long ns) { g_stall_ns.store(ns, std::memory_order_relaxed); }

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
