// paged_cache.cu -- an exact key / value cache in pages: its tables, the rotary
// positions of what goes into it, and the writes.
//
// page_tables_kernel  from the requests' cached and new lengths: the pages that
//   each request needs (off a ring of free pages), the pages of requests that
//   end (back to the ring), and position and slot of every new token.  With
//   have = ceil(ctx / page), want = ceil((ctx + new) / page), the k-th page
//   needed (request order) is ring[(head + k) mod P].  Everything is whole
//   numbers, and every value has one writer, so results do not depend on any
//   order.  The kernel is latency: three prefix sums over the requests, which
//   every block forms for itself (no block waits for another), then each block
//   writes its share of tokens and pages.  6.0 us for 64 requests, 8.8 us for 1,000
//   with 90 prompts (graph replays); a call costs the host 14 us.
// turn_kernel  rotary positions with several axes, and the cache writes fused
//   with them: pair i of axis a turns by the angle p_a f_i,
//     (u, v) = (x cos - y sin, y cos + x sin).
//   Bounded by HBM: each row is read once and written once, 16 bytes per load.
//   A block takes a few tokens and forms their cosines and sines once in shared
//   memory for all heads; the angle is reduced to a fraction of a turn in
//   double (positions run far: in float32 a position of 10^5 would leave the
//   angle off by 10^-2), the rest is float32, rounded once at the end.  31,104 x 16
//   rows of 128 float32 take 82 us (6.2 TB/s, 0.95 of a copy's rate); keys, values
//   and queries of a 16,383-token prompt into random slots 60 us (5.0 TB/s: rows of
//   256 bytes; two units in flight per thread instead of one cost 3 us more).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace wildcat {

__device__ int g_paged_status = 0;  // WILDCAT_ERR_INVALID_ARG: a slot, page id, length or ring state out of range

namespace {

// ---------------------------------------------------------------- page tables
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 16384;  // three prefix arrays of B + 1 ints in shared memory

struct Sums {
    int64_t tokens;
    int need, gives;
};

// Inclusive prefix sums over the block's threads of three values at once.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, v.tokens, o);
        const int b = __shfl_up_sync(0xffffffffu, v.need, o), c = __shfl_up_sync(0xffffffffu, v.gives, o);
        if (lane >= o) {
            v.tokens += a;
            v.need += b;
            v.gives += c;
        }
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < kTabThreads / 32 ? warp_sums[lane] : Sums{0, 0, 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, w.tokens, o);
            const int b = __shfl_up_sync(0xffffffffu, w.need, o), c = __shfl_up_sync(0xffffffffu, w.gives, o);
            if (lane >= o) {
                w.tokens += a;
                w.need += b;
                w.gives += c;
            }
        }
        if (lane < kTabThreads / 32) warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        v.tokens += warp_sums[warp - 1].tokens;
        v.need += warp_sums[warp - 1].need;
        v.gives += warp_sums[warp - 1].gives;
    }
    return v;
}

// The request whose range of the prefix array (n + 1 entries) holds x.
__device__ __forceinline__ int range_of(const int* prefix, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(TablesRequest q) {
    extern __shared__ int tab_sm[];
    const int B = (int)q.B;
    int* cu = tab_sm;              // [B + 1] tokens before request b
    int* first = cu + B + 1;       // [B + 1] pages needed before it
    int* gfirst = first + B + 1;   // [B + 1] pages given back before it
    __shared__ Sums warp_sums[kTabThreads / 32];
    __shared__ int totals[2];      // pages taken, requests that do not advance
    const int tid = threadIdx.x;
    const int64_t page = q.page_size;
    const int P = (int)q.P;
    // A page's slots are id page .. id page + page - 1, and fit in 32 bits up to this id: a
    // larger one (or one below zero) is no page of any pool, and in 32 bits its slots would be
    // another page's.
    const int most_id = (int)(0x80000000u / (unsigned)q.page_size - 1u);
    auto no_page = [&](int id) { return id < 0 || id > most_id; };
    bool bad = false;  // an id, a length or the ring's state is out of range
    int head = 0, count = 0;
    if (P > 0) {
        head = q.ring_state[0] % P;
        if (head < 0) head += P;
        count = min(max(q.ring_state[1], 0), P);
        bad = head != q.ring_state[0] || count != q.ring_state[1];
    }
    if (tid < 2) totals[tid] = 0;
    // prefix sums over the requests, kTabThreads of them at a time
    Sums carry{0, 0, 0};
    for (int base = 0; base < B; base += kTabThreads) {
        const int b = base + tid;
        int64_t ctx = 0, fresh = 0;
        bool ends = false;
        if (b < B) {
            ctx = max(q.ctx_lens[b], 0);
            const int n = q.new_lens[b];
            ends = n < 0;
            fresh = max(n, 0);
        }
        const int64_t have = (ctx + page - 1) / page, want = (ctx + fresh + page - 1) / page;
        __syncthreads();  // warp_sums of the previous round have been read
        // tokens first: whether a request's tokens fit in the outputs decides its need
        Sums s = block_scan(Sums{fresh, 0, ends ? (int)min(have, q.W) : 0}, warp_sums);
        const int64_t cu_end = carry.tokens + s.tokens;
        const bool fits = b < B && !ends && want <= q.W && cu_end <= q.max_tokens && ctx + fresh <= 0x7fffffffLL;
        __syncthreads();
        const Sums t = block_scan(Sums{0, fits ? (int)(want - have) : 0, 0}, warp_sums);
        if (b < B) {
            cu[b] = (int)min(cu_end - fresh, (int64_t)0x7fffffff);
            first[b] = carry.need + t.need - (fits ? (int)(want - have) : 0);
            gfirst[b] = carry.gives + s.gives - (ends ? (int)min(have, q.W) : 0);
        }
        const Sums last{warp_sums[kTabThreads / 32 - 1].tokens, warp_sums[kTabThreads / 32 - 1].need, 0};
        carry.need += last.need;
        // the token and give totals of the first scan: from the last thread
        __shared__ int64_t tok_total;
        __shared__ int give_total;
        if (tid == kTabThreads - 1) {
            tok_total = s.tokens;
            give_total = s.gives;
        }
        __syncthreads();
        carry.tokens += tok_total;
        carry.gives += give_total;
    }
    if (tid == 0) {
        cu[B] = (int)min(carry.tokens, (int64_t)0x7fffffff);
        first[B] = carry.need;
        gfirst[B] = carry.gives;
    }
    __syncthreads();

    // whether request b gets what it needs (its own range of `first` ends within the ring's count)
    auto advances = [&](int b, int64_t ctx, int n) {
        const int64_t want = (ctx + max(n, 0) + page - 1) / page;
        const bool fits = n >= 0 && want <= q.W && (int64_t)cu[b] + max(n, 0) <= q.max_tokens &&
                          ctx + max(n, 0) <= 0x7fffffffLL;
        return fits && (first[b + 1] == first[b] || first[b + 1] <= count);
    };
    if (blockIdx.x == 0) {
        int taken = 0, refused = 0;
        for (int b = tid; b <= B; b += kTabThreads) {
            q.cu_new[b] = cu[b];
            if (b == B) break;
            const int64_t ctx = max(q.ctx_lens[b], 0);
            const int n = q.new_lens[b];
            bad = bad || q.ctx_lens[b] < 0 || (ctx + page - 1) / page > q.W;
            const bool adv = advances(b, ctx, n);
            q.seq_lens[b] = n < 0 ? 0 : (int)(adv ? ctx + n : ctx);
            if (adv && first[b + 1] > first[b]) taken = max(taken, first[b + 1]);
            refused += n >= 0 && !adv;
        }
        // pages taken: the needs that fit are a prefix of all needs
        atomicMax(&totals[0], taken);
        atomicAdd(&totals[1], refused);
        __syncthreads();
        if (tid == 0) {
            const int give = min(gfirst[B], P - count);
            bad = bad || give < gfirst[B];
            q.ring_out[0] = P > 0 ? (int)(((int64_t)head + totals[0]) % P) : 0;
            q.ring_out[1] = count - totals[0] + give;
            q.ring_out[2] = first[B] - totals[0];
            q.ring_out[3] = totals[1];
        }
    }
    const int stride = gridDim.x * kTabThreads, at = blockIdx.x * kTabThreads + tid;
    // the tokens
    for (int64_t t = at; t < q.max_tokens; t += stride) {
        int pos = 0, slot = -1;
        if (t < cu[B]) {
            const int b = range_of(cu, B, (int)t);
            const int64_t ctx = max(q.ctx_lens[b], 0);
            const int64_t x = ctx + (t - cu[b]);
            pos = (int)min(x, (int64_t)0x7fffffff);
            if (advances(b, ctx, q.new_lens[b])) {
                const int64_t have = (ctx + page - 1) / page, p = x / page;
                // a page that this call hands out is read off the ring: its table entry is
                // written by another thread
                const int id = p < have ? q.table[b * q.table_stride + p]
                                        : q.ring[((int64_t)head + first[b] + (p - have)) % P];
                if (no_page(id)) bad = true;
                else slot = (int)((int64_t)id * page + x % page);
            }
        }
        q.positions[t] = pos;
        q.slots[t] = slot;
    }
    // pages handed out (64 bits: the step past the last of up to 2^31 - 1 of them)
    for (int64_t k = at; k < min(first[B], count); k += stride) {
        const int b = range_of(first, B, (int)k);
        const int64_t ctx = max(q.ctx_lens[b], 0);
        if (first[b + 1] > count) continue;
        const int64_t have = (ctx + page - 1) / page;
        const int id = q.ring[((int64_t)head + k) % P];
        bad = bad || no_page(id);
        q.table[b * q.table_stride + have + (k - first[b])] = id;
    }
    // pages given back: never onto the entries read above (those are the ring's filled part)
    for (int64_t k = at; k < min(gfirst[B], P - count); k += stride) {
        const int b = range_of(gfirst, B, (int)k);
        const int id = q.table[b * q.table_stride + (k - gfirst[b])];
        bad = bad || no_page(id);
        q.ring[((int64_t)head + count + k) % P] = id;
    }
    if (bad) atomicMax(&g_paged_status, 1);
}

// ------------------------------------------------------------ rotary and writes
constexpr int kTurnThreads = 128;

template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(x[k] << 16);
            v[2 * k + 1] = __uint_as_float(x[k] & 0xffff0000u);
        }
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            x[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

// The pair (a, b) turned by (cos, sin).  Which product is rounded on its own is said here
// and not left to the compiler, so that the loads' width (the strides and alignment of any
// tensor of the call) does not change a result.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pair(float& a, float& b, float2 cs) {
    const float u = fmaf(a, cs.x, -__fmul_rn(b, cs.y));
    b = INTERLEAVED ? fmaf(b, cs.x, __fmul_rn(a, cs.y)) : fmaf(a, cs.y, __fmul_rn(b, cs.x));
    a = u;
}

// One block: `tokens_per_block` tokens, all heads of all parts.  Work comes in
// units of 2 VEC elements of one head: VEC pairs where the part is rotated
// (elements c and c + half, or 2 VEC neighbours for interleaved pairs), else
// 2 VEC neighbours copied.
template <typename E, int VEC>
__global__ void __launch_bounds__(kTurnThreads) turn_kernel(TurnRequest q, int tokens_per_block) {
    using T = typename E::T;
    extern __shared__ float2 turn_sm[];  // [tokens_per_block][half] (cos, sin)
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
    const int nt = (int)min((int64_t)tokens_per_block, q.T - t0);
    const int half = q.half;
    for (int e = tid; e < nt * half; e += kTurnThreads) {
        const int tt = e / half, i = e - tt * half;
        int a = 0;
        while (a < 3 && i >= q.ends[a]) ++a;
        const double turns = (double)q.positions[a * q.pos_stride + t0 + tt] * q.inv_freq[i] * 0.15915494309189533577;
        const float f = (float)(turns - rint(turns));  // the angle as a fraction of a turn, |f| <= 1/2
        float s, c;
        sincospif(2.0f * f, &s, &c);
        turn_sm[e] = make_float2(c, q.back ? -s : s);
    }
    __syncthreads();
    const int uph = q.d / (2 * VEC);  // units of one head
    const int heads = q.part[0].heads + q.part[1].heads + q.part[2].heads;
    const int upt = heads * uph;  // units of one token
    const int rot_units = half / VEC;
    for (int u = tid; u < nt * upt; u += kTurnThreads) {
        const int tt = u / upt;
        int w = u - tt * upt;
        int h = w / uph;
        const int c = w - h * uph;
        int pi = 0;
        while (pi < 2 && h >= q.part[pi].heads) {
            h -= q.part[pi].heads;
            ++pi;
        }
        const TurnPart& p = q.part[pi];
        const int64_t t = t0 + tt;
        const T* src = static_cast<const T*>(p.src) + t * p.src_t + h * p.src_h;
        T* dst = static_cast<T*>(p.dst);
        if (p.pool) {
            const int slot = q.slots[t];
            if (slot < 0) continue;
            const int page = slot / q.page_size;
            if (page >= q.pages) {
                atomicMax(&g_paged_status, 1);
                continue;
            }
            dst += (int64_t)page * p.dst_t + (int64_t)h * p.dst_h + (int64_t)(slot - page * q.page_size) * p.dst_r;
        } else {
            dst += t * p.dst_t + h * p.dst_h;
        }
        const bool turn = p.turn && c < rot_units;
        int i0, i1;  // first elements of the unit's two vectors
        if (turn && !q.interleaved) {
            i0 = c * VEC;
            i1 = half + c * VEC;
        } else {
            i0 = c * 2 * VEC;
            i1 = i0 + VEC;
        }
        float x[VEC], y[VEC];
        load_vec<VEC>(src + i0, x);
        load_vec<VEC>(src + i1, y);
        if (turn) {
            const float2* cs = turn_sm + tt * half + c * VEC;
            if (!q.interleaved) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) turn_pair<false>(x[k], y[k], cs[k]);
            } else if constexpr (VEC == 1) {
                turn_pair<true>(x[0], y[0], cs[0]);
            } else {
#pragma unroll
                for (int k = 0; k < VEC / 2; ++k) {
                    turn_pair<true>(x[2 * k], x[2 * k + 1], cs[k]);
                    turn_pair<true>(y[2 * k], y[2 * k + 1], cs[VEC / 2 + k]);
                }
            }
        }
        store_vec<VEC>(dst + i0, x);
        store_vec<VEC>(dst + i1, y);
    }
}

template <typename E, int VEC>
Status run_turn(const TurnRequest& q, cudaStream_t st) {
    // tokens of a block: about 32 KB of rows, so that the angles are formed once for
    // many heads, but at least two blocks for each SM where there are tokens enough (a
    // 16,383-token prompt's write 60 us; 64 KB in blocks of 256 threads 63, 24 KB 61)
    const int64_t heads = q.part[0].heads + q.part[1].heads + q.part[2].heads;
    const int64_t row = heads * q.d * (int64_t)sizeof(typename E::T);
    int64_t tpb = std::max<int64_t>(1, std::min<int64_t>(32768 / std::max<int64_t>(row, 1), q.T / 296));
    if (q.half > 0) tpb = std::min<int64_t>(tpb, std::max<int64_t>(1, 4096 / q.half));
    const size_t smem = sizeof(float2) * (size_t)tpb * q.half;
    const int64_t grid = ceil_div(q.T, tpb);
    if (grid > 0x7fffffffLL) return Status::fail(2, "rotary: more than 2^31 blocks of tokens");
    turn_kernel<E, VEC><<<(unsigned)grid, kTurnThreads, smem, st>>>(q, (int)tpb);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "rotary launch");
    return Status::ok();
}

}  // namespace

Status launch_page_tables(const TablesRequest& q, cudaStream_t st) {
    if (q.B > kTabMaxB) return Status::fail(2, "page_tables: more than 16384 requests");
    const size_t smem = sizeof(int) * 3 * (size_t)(q.B + 1);
    // for the most requests at once, whatever this call needs: the attribute belongs to the
    // function, and 48 KB without it cover the kernel's static shared memory too
    const cudaError_t a = paged::allow_smem<page_tables_kernel>((int)sizeof(int) * 3 * (kTabMaxB + 1));
    if (a != cudaSuccess) return Status::cuda(a, "page_tables: shared memory attribute");
    const int64_t work = std::max<int64_t>(q.max_tokens, 1);
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(work, kTabThreads), 148);
    page_tables_kernel<<<grid, kTabThreads, smem, st>>>(q);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return Status::cuda(e, "page_tables launch");
    return Status::ok();
}

// 16 bytes per load where all strides, offsets and section lengths allow it.
Status launch_turn(const TurnRequest& q, cudaStream_t st) {
    const int vec = q.dtype == 1 ? 8 : 4;
    const size_t es = q.dtype == 1 ? 2 : 4;
    bool wide = q.half % vec == 0 && (q.d - 2 * q.half) % (2 * vec) == 0;
    for (const TurnPart& p : q.part) {
        if (p.heads == 0) continue;
        // a part that is not rotated is copied in whole units of a head
        wide = wide && q.d % (2 * vec) == 0 && p.src_t % vec == 0 && p.src_h % vec == 0 && p.dst_t % vec == 0 &&
               p.dst_h % vec == 0 && (!p.pool || p.dst_r % vec == 0) &&
               (reinterpret_cast<uintptr_t>(p.src) | reinterpret_cast<uintptr_t>(p.dst)) % (vec * es) == 0;
    }
    if (q.dtype == 1) return wide ? run_turn<BF16, 8>(q, st) : run_turn<BF16, 1>(q, st);
    return wide ? run_turn<F32, 4>(q, st) : run_turn<F32, 1>(q, st);
}

int read_paged_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_paged_status, &z, sizeof(int));
    }
    return v;
}

}  // namespace wildcat
