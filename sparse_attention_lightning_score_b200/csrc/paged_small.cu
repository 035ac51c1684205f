// The bookkeeping between a new token and its attention over a paged latent
// cache: block tables and slot maps, rotary positions, rows into and out of the
// 4-bit cache.
#include <cuda_fp16.h>

#include "li_common.cuh"
#include "li_kernels.cuh"

namespace li {

namespace {

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
// Request r holds ceil((seq - new) / P) pages and takes the next ones of the pool,
// in request order, up to ceil(seq / P).  Both the pages' and the tokens' offsets
// are prefix sums over the requests.  Every CTA computes all of them (in shared
// memory, two 64-bit sums a run of requests) rather than waiting for another CTA: the
// lengths are a few KB that come from L2.  After that CTAs share the tokens and the
// new pages; a token in a new page takes the page from the pool, so nothing reads
// a table entry that this launch writes.  Latency bound: one launch, and a chain of
// three loads (length, table or pool, and the lookup of the owner in shared memory).
constexpr int BT_THREADS = 512;

struct BtSum {
    long long tokens, pages;
};
__device__ __forceinline__ BtSum bt_add(BtSum a, BtSum b) { return {a.tokens + b.tokens, a.pages + b.pages}; }

// Pages of n positions.
__device__ __forceinline__ int bt_pages(const BlockTableArgs& a, int n) {
    return n > 0 ? divided(n - 1, a.by_page) + 1 : 0;
}

// Last index i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int bt_find(const int32_t* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(BT_THREADS) block_table_kernel(const BlockTableArgs a) {
    extern __shared__ int32_t sm[];
    const int R = a.requests;
    int32_t* starts = sm;                  // [R + 1] new tokens, then the first token of each request (saturated)
    int32_t* first = sm + R + 1;           // [R + 1] pages to take, then the first page of each request (saturated)
    int32_t* old = first + R + 1;          // [R] positions before the step
    __shared__ BtSum wsum[BT_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    bool bad = false;
    for (int r = tid; r < R; r += BT_THREADS) {
        const int seq = __ldg(a.seq + r);
        int add = __ldg(a.add + r);
        int before = seq - add;
        // an impossible request counts as having no new token
        if (add < 0 || seq < add || (long long)seq > (long long)a.max_blocks * a.page_size) {
            bad = true;
            add = before = 0;
            first[r] = 0;
        } else {
            first[r] = bt_pages(a, seq) - bt_pages(a, before);
        }
        starts[r] = add;
        old[r] = before;
    }
    __syncthreads();
    // each thread sums a run of requests (of odd length: no two threads of a warp on one bank), then the block's
    // prefix gives its start
    const int per = ((R + BT_THREADS - 1) / BT_THREADS) | 1;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    BtSum mine{0, 0};
    for (int r = r0; r < r1; ++r) mine = bt_add(mine, {starts[r], first[r]});
    BtSum inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const BtSum up{__shfl_up_sync(0xffffffffu, inc.tokens, o), __shfl_up_sync(0xffffffffu, inc.pages, o)};
        if (lane >= o) inc = bt_add(inc, up);
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    BtSum at{inc.tokens - mine.tokens, inc.pages - mine.pages}, all{0, 0};
#pragma unroll
    for (int w = 0; w < BT_THREADS / 32; ++w) {
        if (w < warp) at = bt_add(at, wsum[w]);
        all = bt_add(all, wsum[w]);
    }
    const long long top = 0x7fffffffll;
    for (int r = r0; r < r1; ++r) {
        const BtSum next = bt_add(at, {starts[r], first[r]});
        starts[r] = (int32_t)min(at.tokens, top);
        first[r] = (int32_t)min(at.pages, top);
        at = next;
    }
    const int total = (int32_t)min(all.tokens, top), taken = (int32_t)min(all.pages, top);
    if (tid == 0) {
        starts[R] = total;
        first[R] = taken;
    }
    __syncthreads();

    int pool0 = a.pool_at ? __ldg(a.pool_at) : 0;
    const bool pool_ok = pool0 >= 0 && pool0 <= a.pool_len;
    if (!pool_ok) pool0 = a.pool_len;          // nothing to take
    const int left = a.pool_len - pool0;
    if (blockIdx.x == 0) {
        if (tid == 0) {
            a.pool_next[0] = pool0 + min(taken, left);
            if (!pool_ok || taken > left || total > a.max_tokens) bad = true;
        }
        if (bad) record_error(a.err, ERRBIT_BOUNDS);
        for (int r = tid; r <= R; r += BT_THREADS) a.starts[r] = starts[r];
    }
    const int gid = blockIdx.x * BT_THREADS + tid, step = gridDim.x * BT_THREADS;
    // page j of the ones taken goes to the request whose run holds j
    auto pool_page = [&](long long j) {
        if (j >= left) return -1;
        const int page = __ldg(a.pool + pool0 + j);
        if ((unsigned)page >= (unsigned)a.num_pages) {
            record_error(a.err, ERRBIT_BOUNDS);
            return -1;
        }
        return page;
    };
    for (long long i = gid; i < a.max_tokens; i += step) {
        const int t = (int)i;
        int64_t slot = -1;
        int pos = -1, owner = -1;
        if (t < total) {
            owner = bt_find(starts, R, t);
            pos = old[owner] + (t - starts[owner]);
            const int block = divided(pos, a.by_page), held = bt_pages(a, old[owner]);
            int page;
            if (block < held) {
                page = a.table[(size_t)owner * a.max_blocks + block];
                if ((unsigned)page >= (unsigned)a.num_pages) {
                    record_error(a.err, ERRBIT_BOUNDS);
                    page = -1;
                }
            } else {
                page = pool_page((long long)first[owner] + (block - held));
            }
            if (page >= 0) slot = (int64_t)page * a.page_size + (pos - block * a.page_size);
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
        a.owner[t] = owner;
    }
    for (long long j = gid; j < taken; j += step) {
        const int r = bt_find(first, R, (int)j);
        a.table[(size_t)r * a.max_blocks + bt_pages(a, old[r]) + ((int)j - first[r])] = pool_page(j);
    }
}

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
// (a, b) -> m (a cos - b sin, a sin + b cos) with the angle pos * f_i.  A far position
// times a frequency loses its fraction in fp32, so the frequency comes in turns as a
// 64-bit fixed-point fraction: the product wraps modulo one turn by itself.  The table
// is within 2^-63 turns of the frequency, so the angle is within pos * 2^-63 turns, and
// the top 32 bits are a signed fraction for sincospi (2^-33 turns, and the fp32 rounding
// of an angle within half a turn: 2^-26 turns).
// Two forms.  Few tokens, rows rotated in place, or heads spread out: a CTA takes one tensor's
// run of heads of one token (or a few tokens with few heads); a thread keeps one place of a
// head (an item: a 16-byte vector, or with the half layout two) and walks the rows (token,
// head) with it, four loads in flight, while the angles are made in shared memory.  Latency
// bound for a decode step, whose heads are spread over more CTAs.
// Many tokens out of place, where most of the bytes are only moved: the copy engine moves
// them.  A persistent CTA brings a token's heads into a ring of stages by bulk copies, turns
// the rotated part where it lies, and sends the stage to its place.  HBM bound: each element
// read once and written once (8192 tokens of 64 heads x 128: 43 us, 6.2 TB/s).
constexpr int RP_THREADS = 256;
constexpr int RP_UNROLL = 4;
constexpr int RP_BLOCK = 16;       // most tokens of a CTA
constexpr int RP_PAIRS = 1024;     // most angles of a CTA
constexpr int RP_ANGLES = 256;     // most angles of a share of several tokens
constexpr int RP_STAGES = 3;       // (3 stages and 4 CTAs an SM: 43 us for 8192 x 64 x 128, 4 and 3: 47)
constexpr int RP_STAGE = 16384;    // bytes of a stage
// Bytes of a call from which it goes by bulk copies (by the threads' own loads: 2.1 MB 3.6 us against 3.0, 8.4 MB 6.1
// against 4.6, 134 MB 51 against 43; 1 MB 2.6 against 2.9).
constexpr long long RP_BULK = 2 << 20;

// (written out, so that every form of the call rounds alike)
__device__ __forceinline__ void rope_pair(float& x, float& y, float c, float s) {
    const float u = __fmaf_rn(x, c, -__fmul_rn(y, s));
    y = __fmaf_rn(x, s, __fmul_rn(y, c));
    x = u;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}

// One 16-byte vector with its pairs inside it; cs: their cosines and sines (16-byte aligned).
__device__ __forceinline__ uint4 rope_inside(uint4 v, bool bf16, const float2* cs) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 a = *reinterpret_cast<const float4*>(cs + i);
            float x0 = bf_lo(w[i]), y0 = bf_hi(w[i]), x1 = bf_lo(w[i + 1]), y1 = bf_hi(w[i + 1]);
            rope_pair(x0, y0, a.x, a.y);
            rope_pair(x1, y1, a.z, a.w);
            w[i] = bf_pack(x0, y0);
            w[i + 1] = bf_pack(x1, y1);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(cs);
        float x0 = __uint_as_float(w[0]), y0 = __uint_as_float(w[1]);
        float x1 = __uint_as_float(w[2]), y1 = __uint_as_float(w[3]);
        rope_pair(x0, y0, a.x, a.y);
        rope_pair(x1, y1, a.z, a.w);
        w[0] = __float_as_uint(x0);
        w[1] = __float_as_uint(y0);
        w[2] = __float_as_uint(x1);
        w[3] = __float_as_uint(y1);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Two vectors, each element of the first with the same one of the second.
__device__ __forceinline__ void rope_across(uint4& p, uint4& q, bool bf16, const float2* cs) {
    uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(cs + 2 * i);
            float x0 = bf_lo(a[i]), y0 = bf_lo(b[i]), x1 = bf_hi(a[i]), y1 = bf_hi(b[i]);
            rope_pair(x0, y0, w.x, w.y);
            rope_pair(x1, y1, w.z, w.w);
            a[i] = bf_pack(x0, x1);
            b[i] = bf_pack(y0, y1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 w = *reinterpret_cast<const float4*>(cs + i);
            float x0 = __uint_as_float(a[i]), y0 = __uint_as_float(b[i]);
            float x1 = __uint_as_float(a[i + 1]), y1 = __uint_as_float(b[i + 1]);
            rope_pair(x0, y0, w.x, w.y);
            rope_pair(x1, y1, w.z, w.w);
            a[i] = __float_as_uint(x0);
            b[i] = __float_as_uint(y0);
            a[i + 1] = __float_as_uint(x1);
            b[i + 1] = __float_as_uint(y1);
        }
    }
    p = make_uint4(a[0], a[1], a[2], a[3]);
    q = make_uint4(b[0], b[1], b[2], b[3]);
}

// Share `at` of a launch: its tensor, tokens and heads.
struct RopePart {
    int token0, tokens, head0, heads;
};
__device__ __forceinline__ const RopeTensor& rope_part(const RopeArgs& a, int at, RopePart& c) {
    int k = 0;
#pragma unroll
    for (int j = 0; j + 1 < LI_ROPE_TENSORS; ++j)
        if (j + 1 < a.n && at >= a.t[j].end) k = j + 1;
    const RopeTensor& t = a.t[k];
    if (k > 0) at -= a.t[k - 1].end;
    const int tb = at / t.chunks;
    c.token0 = tb * t.block;
    c.tokens = min(t.block, a.tokens - c.token0);
    c.head0 = (at - tb * t.chunks) * t.run;
    c.heads = min(t.run, t.heads - c.head0);
    return t;
}

// Cosine and sine of pair j at a position, times mscale.
__device__ __forceinline__ float2 rope_angle(const RopeArgs& a, int pos, int j) {
    const uint64_t turn = (uint64_t)(int64_t)pos * __ldg(a.turns + j);
    const int32_t frac = (int32_t)((turn + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)frac * 0x1p-31f, &s, &c);
    return make_float2(c * a.mscale, s * a.mscale);
}
// Those of the CTA's tokens; live[k]: token k is no padding.
__device__ __forceinline__ void rope_angles(const RopeArgs& a, const RopePart& c, float2* cs, int* live) {
    const int n = a.rot_dim / 2;
    for (int i = threadIdx.x; i < c.tokens * n; i += RP_THREADS) {
        const int k = i / n, j = i - k * n, pos = __ldg(a.positions + c.token0 + k);
        if (j == 0) live[k] = pos >= 0;
        cs[i] = rope_angle(a, pos, j);
    }
}

template <bool BF16, bool HALF>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, const RopeTensor& t, const RopePart& c, float2* cs,
                                          int* live) {
    constexpr int V = BF16 ? 8 : 4, SIZE = 16 / V;
    const int step = RP_THREADS / t.per_head;          // rows of a pass
    const int slot = threadIdx.x / t.per_head, i = threadIdx.x - slot * t.per_head;
    const int all = c.tokens * t.run, rows = slot < step ? all : 0;  // (the last threads have no place)
    const bool turns = i < t.rotated;
    int e = turns ? t.offset + i * V : (i - t.rotated) * V;
    if (!turns && e >= t.offset) e += a.rot_dim;
    const int pair = HALF ? i * V : i * V / 2;
    const bool two = HALF && turns;
    const int far = a.rot_dim / 2 * SIZE;
    const uint8_t* x = static_cast<const uint8_t*>(t.x) + (c.token0 * t.x_token + c.head0 * t.x_head + e) * SIZE;
    uint8_t* out = static_cast<uint8_t*>(t.out) + (c.token0 * t.out_token + c.head0 * t.out_head + e) * SIZE;
    for (int base = 0; base < all; base += step * RP_UNROLL) {  // (the same for every thread)
        uint4 p[RP_UNROLL], q[RP_UNROLL];
#pragma unroll
        for (int j = 0; j < RP_UNROLL; ++j) {
            const int row = base + j * step + slot, k = divided(row, t.by_run), h = row - k * t.run;
            if (row < rows && h < c.heads) {
                const uint8_t* src = x + (k * t.x_token + h * t.x_head) * SIZE;
                p[j] = *reinterpret_cast<const uint4*>(src);
                if (two) q[j] = *reinterpret_cast<const uint4*>(src + far);
            }
        }
        if (base == 0) {
            rope_angles(a, c, cs, live);
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < RP_UNROLL; ++j) {
            const int row = base + j * step + slot, k = divided(row, t.by_run), h = row - k * t.run;
            if (row < rows && h < c.heads && live[k]) {  // (padding: the row stays as it was)
                uint8_t* dst = out + (k * t.out_token + h * t.out_head) * SIZE;
                if (turns) {
                    const float2* w = cs + k * (a.rot_dim / 2) + pair;
                    if (HALF) rope_across(p[j], q[j], BF16, w);
                    else p[j] = rope_inside(p[j], BF16, w);
                }
                *reinterpret_cast<uint4*>(dst) = p[j];
                if (two) *reinterpret_cast<uint4*>(dst + far) = q[j];
            }
        }
    }
}

__global__ void __launch_bounds__(RP_THREADS) rope_wide_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float2 cs[RP_PAIRS];  // [tokens of the CTA][rot_dim / 2] m cos, m sin
    __shared__ int live[RP_BLOCK];
    RopePart c;
    const RopeTensor& t = rope_part(a, blockIdx.x, c);
    pdl_wait();
    if (t.bf16) {
        if (t.half) rope_rows<true, true>(a, t, c, cs, live);
        else rope_rows<true, false>(a, t, c, cs, live);
    } else {
        if (t.half) rope_rows<false, true>(a, t, c, cs, live);
        else rope_rows<false, false>(a, t, c, cs, live);
    }
}

// The bulk form.  Shares (some heads of a token, or several tokens of few heads whose rows lie side by side) go
// round robin over the CTAs; a CTA's k-th share uses stage k % RP_STAGES, and is loaded RP_STAGES - 1 shares ahead, when
// the store of the share that had the stage before has been read out.
__global__ void __launch_bounds__(RP_THREADS) rope_bulk_kernel(const __grid_constant__ RopeArgs a, const int shares,
                                                              const int angles_max, const DevErr err) {
    extern __shared__ __align__(128) uint8_t stages[];  // [RP_STAGES][RP_STAGE], then the angles [2][angles_max]
    __shared__ uint64_t full[RP_STAGES];
    float2* cs = reinterpret_cast<float2*>(stages + RP_STAGES * RP_STAGE);
    const int n = a.rot_dim / 2, tid = threadIdx.x;
    if (tid == 0) {
        for (int s = 0; s < RP_STAGES; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    auto load = [&](int k) {                                       // (one thread) the CTA's k-th share
        const long long at = blockIdx.x + (long long)k * gridDim.x;
        if (at >= shares) return;
        RopePart c;
        const RopeTensor& t = rope_part(a, (int)at, c);
        const int size = t.bf16 ? 2 : 4;
        const uint32_t bytes = (uint32_t)(c.tokens * c.heads * t.dim * size);
        uint64_t* bar = &full[k % RP_STAGES];
        mbar_arrive_expect_tx(bar, bytes);
        bulk_load(stages + (k % RP_STAGES) * RP_STAGE,
                  static_cast<const uint8_t*>(t.x) + (c.token0 * t.x_token + (long long)c.head0 * t.dim) * size, bytes, bar);
    };
    auto angles = [&](int k) {
        const long long at = blockIdx.x + (long long)k * gridDim.x;
        if (at >= shares) return;
        RopePart c;
        rope_part(a, (int)at, c);
        for (int i = tid; i < c.tokens * n; i += RP_THREADS) {
            const int tok = i / n, j = i - tok * n;
            cs[(k & 1) * angles_max + i] = rope_angle(a, __ldg(a.positions + c.token0 + tok), j);
        }
    };
    if (tid == 0)
        for (int k = 0; k < RP_STAGES - 1; ++k) load(k);
    angles(0);
    __syncthreads();
    int k = 0;
    bool ok = true;
    for (long long at = blockIdx.x; at < shares; at += gridDim.x, ++k) {
        RopePart c;
        const RopeTensor& t = rope_part(a, (int)at, c);
        uint8_t* stage = stages + (k % RP_STAGES) * RP_STAGE;
        const int size = t.bf16 ? 2 : 4, far = n * size, head = t.dim * size, v = t.bf16 ? 8 : 4;
        ok = ok && mbar_wait(&full[k % RP_STAGES], (k / RP_STAGES) & 1, err);
        angles(k + 1);
        const float2* w = cs + (k & 1) * angles_max;
        for (int i = tid; i < c.tokens * c.heads * t.rotated; i += RP_THREADS) {
            const int row = divided(i, t.by_rotated), j = i - row * t.rotated;
            const float2* f = w + divided(row, t.by_run) * n + (t.half ? j * v : j * v / 2);  // (a token has run rows)
            uint4* p = reinterpret_cast<uint4*>(stage + row * head + t.offset * size + j * 16);
            if (t.half) {
                uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) + far);
                uint4 x = *p, y = *q;
                rope_across(x, y, t.bf16, f);
                *p = x;
                *q = y;
            } else {
                *p = rope_inside(*p, t.bf16, f);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            uint8_t* dst = static_cast<uint8_t*>(t.out) + (c.token0 * t.out_token + (long long)c.head0 * t.dim) * size;
            const uint32_t row = (uint32_t)(c.heads * head);       // bytes of a token
            for (int i = 0; ok && i < c.tokens;) {                 // runs of tokens that are no padding
                int m = i;
                while (m < c.tokens && __ldg(a.positions + c.token0 + m) >= 0) ++m;
                if (m > i)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                     reinterpret_cast<uint64_t>(dst + (size_t)i * row)),
                                 "r"(smem_u32(stage + i * row)), "r"((m - i) * row)
                                 : "memory");
                i = m + 1;
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the share before has left its stage
            if (ok) load(k + RP_STAGES - 1);
        }
    }
    // every load has been waited for (or, after a wait that ran out, is given one more), every store is finished
    if (tid == 0) {
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok)
            for (int s = 0; s < RP_STAGES; ++s) mbar_wait(&full[s], (k / RP_STAGES) & 1, err);
    }
}

// Any alignment and strides, and heads of more than 256 items: a pair, or one copied element, at a time.
__global__ void __launch_bounds__(RP_THREADS) rope_single_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float2 cs[RP_PAIRS];
    __shared__ int live[RP_BLOCK];
    RopePart c;
    const RopeTensor& t = rope_part(a, blockIdx.x, c);
    pdl_wait();
    rope_angles(a, c, cs, live);
    __syncthreads();
    const int work = c.tokens * c.heads * t.per_head;
    for (int w = threadIdx.x; w < work; w += RP_THREADS) {
        const int row = w / t.per_head, i = w - row * t.per_head;
        const int k = row / c.heads, h = row - k * c.heads;
        if (!live[k]) continue;
        const bool turns = i < t.rotated;
        int e = !turns ? i - t.rotated : t.offset + (t.half ? i : 2 * i);
        if (!turns && e >= t.offset) e += a.rot_dim;
        const int far = t.half ? a.rot_dim / 2 : 1;
        const long long from = (c.token0 + k) * t.x_token + (c.head0 + h) * t.x_head + e;
        const long long to = (c.token0 + k) * t.out_token + (c.head0 + h) * t.out_head + e;
        const float2 f = turns ? cs[k * (a.rot_dim / 2) + i] : make_float2(1.f, 0.f);
        if (t.bf16) {
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(t.x) + from;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out) + to;
            if (!turns) {
                o[0] = x[0];
            } else {
                float u = __bfloat162float(x[0]), v = __bfloat162float(x[far]);
                rope_pair(u, v, f.x, f.y);
                o[0] = __float2bfloat16_rn(u);
                o[far] = __float2bfloat16_rn(v);
            }
        } else {
            const float* x = static_cast<const float*>(t.x) + from;
            float* o = static_cast<float*>(t.out) + to;
            if (!turns) {
                o[0] = x[0];
            } else {
                float u = x[0], v = x[far];
                rope_pair(u, v, f.x, f.y);
                o[0] = u;
                o[far] = v;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The 4-bit cache
// ---------------------------------------------------------------------------
// A row: 512 e2m1 codes (element i in byte i / 2, even elements in the low half),
// 32 e4m3 scales (one per 16 elements), 64 bf16 unchanged.  A warp takes a row, a
// lane one block of 16.  HBM bound: 1152 B in and 416 B out a row.
constexpr int K4_THREADS = 256;

__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

// A lane's 16 latent elements (w) as codes and scale.
__device__ __forceinline__ void kv4_block(const uint32_t (&w)[8], uint2& code, uint32_t& sbyte) {
    // largest magnitude, as bits: a NaN is above infinity and so becomes the scale (and the whole block)
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
    sbyte = e4m3x2(__fdiv_rn(__uint_as_float(top), 6.f), 0.f) & 0xffu;
    uint32_t sh;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"((unsigned short)sbyte));
    const float s = __low2float(*reinterpret_cast<__half2*>(&sh));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // x / s: the product with the reciprocal, then Markstein's correction by the exact residual (IBM J. Res.
            // Dev. 34, 1990), which makes a quotient that fp32 can hold exact, so ties between two codes are seen
            // as ties; the conversion saturates beyond 6.  An infinity stands for the largest float.
            float x = k & 1 ? bf_hi(w[4 * j + (k >> 1)]) : bf_lo(w[4 * j + (k >> 1)]);
            if (top >= 0x7f800000u) x = fminf(fmaxf(x, -3.3e38f), 3.3e38f);
            const float q = x * r;
            y[k] = copysignf(__fmaf_rn(__fmaf_rn(-q, s, x), r, q), x);  // (the sum would lose the sign of -0)
        }
        c[j] = e2m1x8(y);
    }
    code = make_uint2(c[0], c[1]);
}

// ROWS rows a warp, their loads all in flight: 2 once there are enough of them to fill the GPU, else 1 (a short chain).
// Rows are read past the caches (__ldcs): nothing reads them again.
template <bool WIDE, int ROWS>
__global__ void __launch_bounds__(K4_THREADS) kv4_write_kernel(const Kv4Args a) {
    const int lane = threadIdx.x & 31;
    const long long i0 = ((long long)blockIdx.x * (K4_THREADS / 32) + (threadIdx.x >> 5)) * ROWS;
    pdl_wait();
    long long slot[ROWS];
    uint32_t w[ROWS][8], rot[ROWS];  // the lane's 16 latent elements, two of the rotary ones
#pragma unroll
    for (int k = 0; k < ROWS; ++k) slot[k] = i0 + k < a.n ? __ldg(a.slots + i0 + k) : -1;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        if (i0 + k >= a.n) continue;
        const uint16_t* src = a.rows + (i0 + k) * a.row_stride;
        if constexpr (WIDE) {
            const uint4 lo = __ldcs(reinterpret_cast<const uint4*>(src + lane * 16));
            const uint4 hi = __ldcs(reinterpret_cast<const uint4*>(src + lane * 16) + 1);
            w[k][0] = lo.x; w[k][1] = lo.y; w[k][2] = lo.z; w[k][3] = lo.w;
            w[k][4] = hi.x; w[k][5] = hi.y; w[k][6] = hi.z; w[k][7] = hi.w;
            rot[k] = __ldg(reinterpret_cast<const uint32_t*>(src + 512 + lane * 2));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[k][j] = __ldg(src + lane * 16 + 2 * j) | ((uint32_t)__ldg(src + lane * 16 + 2 * j + 1) << 16);
            rot[k] = __ldg(src + 512 + lane * 2) | ((uint32_t)__ldg(src + 512 + lane * 2 + 1) << 16);
        }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        if (slot[k] < 0) continue;  // padding, or past the end
        if (slot[k] >= a.num_slots) {
            if (lane == 0) record_error(a.err, ERRBIT_BOUNDS);
            continue;
        }
        uint2 code;
        uint32_t sbyte;
        kv4_block(w[k], code, sbyte);
        uint8_t* dst = a.cache + slot[k] * LI_KV4_ROW_BYTES;
        *reinterpret_cast<uint2*>(dst + lane * 8) = code;
        dst[256 + lane] = (uint8_t)sbyte;
        *reinterpret_cast<uint32_t*>(dst + 288 + lane * 4) = rot[k];
    }
}

// e2m1 x e4m3 has 6 significant bits, so the bf16 row is exact.  A slot < 0 reads as zeros.  (65537 rows 19 us, 5.4 TB/s;
// four rows a warp: the same, and 32768 rows 10.8 against 9.3.)
__global__ void __launch_bounds__(K4_THREADS) kv4_read_kernel(const Kv4Args a) {
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * (K4_THREADS / 32) + (threadIdx.x >> 5);
    pdl_wait();
    if (i >= a.n) return;
    const long long slot = __ldg(a.slots + i);
    uint2 code = make_uint2(0, 0);
    uint32_t sbyte = 0, rot = 0;
    if (slot >= a.num_slots) {
        if (lane == 0) record_error(a.err, ERRBIT_BOUNDS);
    } else if (slot >= 0) {
        const uint8_t* src = a.cache + slot * LI_KV4_ROW_BYTES;
        code = *reinterpret_cast<const uint2*>(src + lane * 8);
        sbyte = src[256 + lane];
        rot = *reinterpret_cast<const uint32_t*>(src + 288 + lane * 4);
    }
    uint32_t sh;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"((unsigned short)sbyte));
    const __half2 s2 = __low2half2(*reinterpret_cast<__half2*>(&sh));
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = ((j < 4 ? code.x : code.y) >> (8 * (j & 3))) & 0xffu;
        uint32_t h;
        asm("{\n\t.reg .b8 b, z0, z1, z2;\n\tmov.b32 {b, z0, z1, z2}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
            : "=r"(h)
            : "r"(byte));
        // at most 6 x 448 and at least 2^-10: exact in fp16 too
        const float2 f = __half22float2(__hmul2(*reinterpret_cast<__half2*>(&h), s2));
        o[j] = bf_pack(f.x, f.y);
    }
    uint16_t* dst = a.out + i * 576;
    *reinterpret_cast<uint4*>(dst + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    *(reinterpret_cast<uint4*>(dst + lane * 16) + 1) = make_uint4(o[4], o[5], o[6], o[7]);
    *reinterpret_cast<uint32_t*>(dst + 512 + lane * 2) = rot;
}

// From this many rows on a warp takes two (1, 2 and 4 rows a warp: 8192 rows 3.7, 4.2 and 4.4 us, 16384 5.9, 5.9 and
// 6.8, 65537 21.2, 19.4 and 20.2, 131072 42.1, 36.7 and 37.6: 5.6 TB/s).
constexpr long long K4_MANY = 16384;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace

li_status launch_block_tables(BlockTableArgs a, cudaStream_t st) {
    a.by_page = divisor_of(a.page_size);
    const size_t smem = (size_t)3 * (a.requests + 1) * sizeof(int32_t);
    if (smem > 48 * 1024) {
        // set on every such call: the attribute belongs to the current device
        if (cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess) {
            cudaGetLastError();
            return LI_ERR_CUDA;
        }
    }
    int grid = ceil_div(a.max_tokens, BT_THREADS);
    grid = grid < 1 ? 1 : grid > host_num_sms() ? host_num_sms() : grid;
    if (launch_pdl(block_table_kernel, dim3(grid), dim3(BT_THREADS), smem, st, 1, a) != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return host_check_launch();
}

li_status launch_rope(RopeArgs a, cudaStream_t st) {
    const int sms = host_num_sms(), pairs = a.rot_dim / 2;
    long long bytes = 0;
    for (int i = 0; i < a.n; ++i) {
        const RopeTensor& t = a.t[i];
        const int v = t.bf16 ? 8 : 4, size = t.bf16 ? 2 : 4;
        if ((t.half ? pairs / v : a.rot_dim / v) + (t.in_place ? 0 : (t.dim - a.rot_dim) / v) > RP_THREADS) a.wide = 0;
        if (t.dim * size > RP_STAGE) a.dense = 0;
        bytes += (long long)a.tokens * t.heads * t.dim * size;
    }
    const bool bulk = a.wide && a.dense && bytes >= RP_BULK;
    long long shares = 0;
    int angles_max = 0;
    for (int i = 0; i < a.n; ++i) {
        RopeTensor& t = a.t[i];
        const int v = a.wide ? (t.bf16 ? 8 : 4) : 1;
        t.rotated = t.half ? pairs / v : a.wide ? a.rot_dim / v : pairs;
        t.per_head = t.rotated + (t.in_place ? 0 : (t.dim - a.rot_dim) / v);
        t.block = 1;
        const long long items = (long long)t.heads * t.per_head;
        if (bulk) {
            const int size = t.bf16 ? 2 : 4;
            t.chunks = ceil_div(t.heads, RP_STAGE / (t.dim * size));
            // (positions' order is the rows': tokens side by side in both tensors can share a copy)
            if (t.chunks == 1 && t.x_token == (long long)t.heads * t.dim && t.out_token == t.x_token)
                while (t.block < RP_BLOCK && 2 * t.block * t.heads * t.dim * size <= RP_STAGE &&
                       2 * t.block * pairs <= RP_ANGLES)
                    t.block *= 2;
            if (angles_max < t.block * pairs) angles_max = t.block * pairs;
        } else {
            // four items a thread when the tokens fill the GPU that way (several tokens a CTA where one has fewer),
            // else fewer heads a CTA, down to an item a thread
            const int full = RP_THREADS * RP_UNROLL;
            t.chunks = ceil_div(items, full);
            if ((long long)a.tokens * t.chunks < 4LL * sms) {
                const int most = ceil_div(items, RP_THREADS), wanted = ceil_div(4LL * sms, a.tokens);
                if (t.chunks < most) t.chunks = wanted < most ? (wanted > t.chunks ? wanted : t.chunks) : most;
            } else {
                while (t.block < RP_BLOCK && 2 * t.block * items <= full && 2 * t.block * pairs <= RP_PAIRS &&
                       a.tokens >= 8LL * t.block * sms)
                    t.block *= 2;
            }
        }
        if (t.chunks > t.heads) t.chunks = t.heads;
        t.run = ceil_div(t.heads, t.chunks);
        t.chunks = ceil_div(t.heads, t.run);
        t.by_run = divisor_of(t.run);
        t.by_rotated = divisor_of(t.rotated);
        shares += (long long)ceil_div(a.tokens, t.block) * t.chunks;
        if (shares >= (1ll << 31)) return LI_ERR_UNSUPPORTED;
        t.end = (int)shares;
    }
    cudaError_t e;
    if (bulk) {
        const size_t smem = RP_STAGES * RP_STAGE + 2 * angles_max * sizeof(float2);
        // (set on every call: the attribute belongs to the current device)
        e = cudaFuncSetAttribute(rope_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 RP_STAGES * RP_STAGE + RP_PAIRS * (int)sizeof(float2));
        const long long most = (long long)(227 * 1024 / (smem + 1536)) * sms;  // as many CTAs as fit the SMs at a time
        const DevErr err = host_dev_err();
        if (e == cudaSuccess)
            e = launch_pdl(rope_bulk_kernel, dim3((unsigned)(shares < most ? shares : most)), dim3(RP_THREADS), smem, st, 1,
                           a, (int)shares, angles_max, err);
    } else {
        e = a.wide ? launch_pdl(rope_wide_kernel, dim3((unsigned)shares), dim3(RP_THREADS), 0, st, 1, a)
                   : launch_pdl(rope_single_kernel, dim3((unsigned)shares), dim3(RP_THREADS), 0, st, 1, a);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return host_check_launch();
}

li_status launch_kv4_write(const Kv4Args& a, cudaStream_t st) {
    const int rows = a.wide && a.n >= K4_MANY ? 2 : 1;
    const dim3 grid(ceil_div(a.n, K4_THREADS / 32 * rows)), block(K4_THREADS);
    const cudaError_t e = !a.wide     ? launch_pdl(kv4_write_kernel<false, 1>, grid, block, 0, st, 1, a)
                          : rows == 1 ? launch_pdl(kv4_write_kernel<true, 1>, grid, block, 0, st, 1, a)
                                      : launch_pdl(kv4_write_kernel<true, 2>, grid, block, 0, st, 1, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return host_check_launch();
}

li_status launch_kv4_read(const Kv4Args& a, cudaStream_t st) {
    if (launch_pdl(kv4_read_kernel, dim3(ceil_div(a.n, K4_THREADS / 32)), dim3(K4_THREADS), 0, st, 1, a) != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return host_check_launch();
}

}  // namespace li
