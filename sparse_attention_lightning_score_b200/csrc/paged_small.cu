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
// are prefix sums over the requests.  Every CTA computes all of them (two 64-bit
// sums a request, in shared memory) rather than waiting for another CTA: the
// lengths are a few KB that come from L2.  After that CTAs share the tokens and the
// new pages; a token in a new page takes the page from the pool, so nothing reads
// a table entry that this launch writes.  Latency bound: one launch, three
// dependent loads (length, table or pool, store).
constexpr int BT_THREADS = 256;

struct BtSum {
    long long tokens, pages;
};
__device__ __forceinline__ BtSum bt_add(BtSum a, BtSum b) { return {a.tokens + b.tokens, a.pages + b.pages}; }

// (new tokens, held pages, needed pages) of one request; an impossible one counts as having no new token.
__device__ __forceinline__ bool bt_request(const BlockTableArgs& a, int r, int* add, int* held, int* need) {
    const int seq = __ldg(a.seq + r);
    *add = __ldg(a.add + r);
    const bool ok = *add >= 0 && seq >= *add && (long long)seq <= (long long)a.max_blocks * a.page_size;
    if (!ok) {
        *add = *held = *need = 0;
        return false;
    }
    const int old = seq - *add;
    *held = old > 0 ? (int)((unsigned)(old - 1) / (unsigned)a.page_size) + 1 : 0;
    *need = (seq > 0 ? (int)((unsigned)(seq - 1) / (unsigned)a.page_size) + 1 : 0) - *held;
    return true;
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
    int32_t* starts = sm;                      // [requests + 1] first token of each request (saturated)
    int32_t* first = sm + a.requests + 1;      // [requests + 1] first page of each request (saturated)
    __shared__ BtSum wsum[BT_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    // each thread sums a run of requests, then the block's prefix gives its start
    const int per = (a.requests + BT_THREADS - 1) / BT_THREADS;
    const int r0 = min(a.requests, tid * per), r1 = min(a.requests, r0 + per);
    BtSum mine{0, 0};
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        int add, held, need;
        bad |= !bt_request(a, r, &add, &held, &need);
        mine = bt_add(mine, {add, need});
    }
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
        int add, held, need;
        bt_request(a, r, &add, &held, &need);
        starts[r] = (int32_t)min(at.tokens, top);
        first[r] = (int32_t)min(at.pages, top);
        at = bt_add(at, {add, need});
    }
    if (tid == 0) {
        starts[a.requests] = (int32_t)min(all.tokens, top);
        first[a.requests] = (int32_t)min(all.pages, top);
    }
    __syncthreads();

    int pool0 = a.pool_at ? __ldg(a.pool_at) : 0;
    const bool pool_ok = pool0 >= 0 && pool0 <= a.pool_len;
    if (!pool_ok) pool0 = a.pool_len;          // nothing to take
    const int left = a.pool_len - pool0;
    const int total = starts[a.requests], taken = first[a.requests];
    if (blockIdx.x == 0) {
        if (tid == 0) {
            a.pool_next[0] = pool0 + min(taken, left);
            if (!pool_ok || taken > left || total > a.max_tokens) bad = true;
        }
        if (bad) record_error(a.err, ERRBIT_BOUNDS);
        for (int r = tid; r <= a.requests; r += BT_THREADS) a.starts[r] = starts[r];
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
    for (int t = gid; t < a.max_tokens; t += step) {
        int64_t slot = -1;
        int pos = -1, owner = -1;
        if (t < total) {
            owner = bt_find(starts, a.requests, t);
            int add, held, need;
            bt_request(a, owner, &add, &held, &need);
            pos = __ldg(a.seq + owner) - add + (t - starts[owner]);
            const int block = (int)((unsigned)pos / (unsigned)a.page_size);
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
        const int r = bt_find(first, a.requests, (int)j);
        int add, held, need;
        bt_request(a, r, &add, &held, &need);
        a.table[(size_t)r * a.max_blocks + held + ((int)j - first[r])] = pool_page(j);
    }
}

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
// (a, b) -> m (a cos - b sin, a sin + b cos) with the angle pos * f_i.  A far position
// times a frequency loses its fraction in fp32, so the frequency comes in turns as a
// 64-bit fixed-point fraction: the product wraps modulo one turn by itself, exactly up
// to pos * 2^-65 turns, and the top 32 bits are a signed fraction for sincospi (fp32
// rounding of an angle within half a turn: 2^-25 turns).
// A CTA takes one token and a run of its items: it loads them, computes the token's
// cosines and sines once in shared memory while the loads are in flight, and stores.
// HBM bound for many tokens (each element read once and written once), latency
// bound for a decode step, where the items of a token are spread over several CTAs.
constexpr int RP_THREADS = 256;
constexpr int RP_UNROLL = 2;

struct RopeItem {
    const RopeTensor* t;
    long long x, out;   // element offsets of the item's first vector
    int pair;           // first pair of a rotated item, -1 for a copied one
    int far;            // half layout: elements from the first vector to its partner, else 0
};

// Items of a head: the rotated part (half layout: two vectors an item), then the rest.
template <int V>
__device__ __forceinline__ RopeItem rope_item(const RopeArgs& a, int token, int i) {
    int k = 0;
#pragma unroll
    for (int j = 0; j + 1 < LI_ROPE_TENSORS; ++j)
        if (j + 1 < a.n && i >= a.t[j].end) k = j + 1;
    const RopeTensor& t = a.t[k];
    if (k > 0) i -= a.t[k - 1].end;
    const int head = i / t.per_head;
    i -= head * t.per_head;
    RopeItem r;
    r.t = &t;
    int e;
    // V elements of the tensor's own type make an item's vector; a single-element item is one pair
    const int v = V == 1 ? 1 : t.bf16 ? 8 : 4;
    const int nrot = t.half ? a.rot_dim / 2 / v : (V == 1 ? a.rot_dim / 2 : a.rot_dim / v);
    if (i < nrot) {
        if (t.half) {
            e = t.offset + i * v;
            r.pair = i * v;
            r.far = a.rot_dim / 2;
        } else {
            e = t.offset + i * (V == 1 ? 2 : v);
            r.pair = V == 1 ? i : i * v / 2;
            r.far = V == 1 ? 1 : 0;
        }
    } else {
        e = (i - nrot) * v;
        if (e >= t.offset) e += a.rot_dim;
        r.pair = -1;
        r.far = 0;
    }
    r.x = token * t.x_token + head * t.x_head + e;
    r.out = token * t.out_token + head * t.out_head + e;
    return r;
}

__device__ __forceinline__ void rope_pair(float& x, float& y, float2 cs) {
    const float u = x * cs.x - y * cs.y;
    y = x * cs.y + y * cs.x;
    x = u;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}

// One 16-byte vector with its pairs inside it.
__device__ __forceinline__ uint4 rope_inside(uint4 v, bool bf16, const float2* cs) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = bf_lo(w[i]), y = bf_hi(w[i]);
            rope_pair(x, y, cs[i]);
            w[i] = bf_pack(x, y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x = __uint_as_float(w[2 * i]), y = __uint_as_float(w[2 * i + 1]);
            rope_pair(x, y, cs[i]);
            w[2 * i] = __float_as_uint(x);
            w[2 * i + 1] = __float_as_uint(y);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Two vectors, each element of the first with the same one of the second.
__device__ __forceinline__ void rope_across(uint4& p, uint4& q, bool bf16, const float2* cs) {
    uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            float x0 = bf_lo(a[i]), y0 = bf_lo(b[i]), x1 = bf_hi(a[i]), y1 = bf_hi(b[i]);
            rope_pair(x0, y0, cs[2 * i]);
            rope_pair(x1, y1, cs[2 * i + 1]);
            a[i] = bf_pack(x0, x1);
            b[i] = bf_pack(y0, y1);
        } else {
            float x = __uint_as_float(a[i]), y = __uint_as_float(b[i]);
            rope_pair(x, y, cs[i]);
            a[i] = __float_as_uint(x);
            b[i] = __float_as_uint(y);
        }
    }
    p = make_uint4(a[0], a[1], a[2], a[3]);
    q = make_uint4(b[0], b[1], b[2], b[3]);
}

__global__ void __launch_bounds__(RP_THREADS) rope_wide_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 cs[];  // [rot_dim / 2] m cos, m sin
    const int token = blockIdx.x;
    const int lo = blockIdx.y * a.chunk, hi = min(a.items, lo + a.chunk);
    pdl_wait();
    const int pos = __ldg(a.positions + token);
    if (pos < 0) return;  // padding: the row stays as it was
    for (int base = lo; base < hi; base += RP_THREADS * RP_UNROLL) {
        RopeItem it[RP_UNROLL];
        uint4 p[RP_UNROLL], q[RP_UNROLL];
#pragma unroll
        for (int j = 0; j < RP_UNROLL; ++j) {
            const int i = base + j * RP_THREADS + threadIdx.x;
            if (i < hi) {
                it[j] = rope_item<0>(a, token, i);
                const int size = it[j].t->bf16 ? 2 : 4;
                const uint8_t* src = static_cast<const uint8_t*>(it[j].t->x) + it[j].x * size;
                p[j] = *reinterpret_cast<const uint4*>(src);
                if (it[j].far) q[j] = *reinterpret_cast<const uint4*>(src + it[j].far * size);
            }
        }
        if (base == lo) {
            for (int i = threadIdx.x; i < a.rot_dim / 2; i += RP_THREADS) {
                const uint64_t turn = (uint64_t)(int64_t)pos * __ldg(a.turns + i);
                const int32_t frac = (int32_t)((turn + 0x80000000ull) >> 32);
                float s, c;
                sincospif((float)frac * 0x1p-31f, &s, &c);
                cs[i] = make_float2(c * a.mscale, s * a.mscale);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < RP_UNROLL; ++j) {
            const int i = base + j * RP_THREADS + threadIdx.x;
            if (i < hi) {
                const bool bf16 = it[j].t->bf16;
                const int size = bf16 ? 2 : 4;
                uint8_t* dst = static_cast<uint8_t*>(it[j].t->out) + it[j].out * size;
                if (it[j].pair >= 0) {
                    if (it[j].far) rope_across(p[j], q[j], bf16, cs + it[j].pair);
                    else p[j] = rope_inside(p[j], bf16, cs + it[j].pair);
                }
                *reinterpret_cast<uint4*>(dst) = p[j];
                if (it[j].far) *reinterpret_cast<uint4*>(dst + it[j].far * size) = q[j];
            }
        }
    }
}

// Any alignment and strides: a pair, or one copied element, per item.
__global__ void __launch_bounds__(RP_THREADS) rope_single_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 cs[];
    const int token = blockIdx.x;
    const int lo = blockIdx.y * a.chunk, hi = min(a.items, lo + a.chunk);
    pdl_wait();
    const int pos = __ldg(a.positions + token);
    if (pos < 0) return;
    for (int i = threadIdx.x; i < a.rot_dim / 2; i += RP_THREADS) {
        const uint64_t turn = (uint64_t)(int64_t)pos * __ldg(a.turns + i);
        const int32_t frac = (int32_t)((turn + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)frac * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += RP_THREADS) {
        const RopeItem it = rope_item<1>(a, token, i);
        if (it.t->bf16) {
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(it.t->x) + it.x;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(it.t->out) + it.out;
            if (it.pair < 0) {
                o[0] = x[0];
            } else {
                float u = __bfloat162float(x[0]), v = __bfloat162float(x[it.far]);
                rope_pair(u, v, cs[it.pair]);
                o[0] = __float2bfloat16_rn(u);
                o[it.far] = __float2bfloat16_rn(v);
            }
        } else {
            const float* x = static_cast<const float*>(it.t->x) + it.x;
            float* o = static_cast<float*>(it.t->out) + it.out;
            if (it.pair < 0) {
                o[0] = x[0];
            } else {
                float u = x[0], v = x[it.far];
                rope_pair(u, v, cs[it.pair]);
                o[0] = u;
                o[it.far] = v;
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

template <bool WIDE>
__global__ void __launch_bounds__(K4_THREADS) kv4_write_kernel(const Kv4Args a) {
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * (K4_THREADS / 32) + (threadIdx.x >> 5);
    pdl_wait();
    if (i >= a.n) return;
    const long long slot = __ldg(a.slots + i);
    if (slot < 0) return;  // padding
    if (slot >= a.num_slots) {
        if (lane == 0) record_error(a.err, ERRBIT_BOUNDS);
        return;
    }
    const uint16_t* src = a.rows + i * a.row_stride;
    uint32_t w[8], rot;  // the lane's 16 latent elements, two of the rotary ones
    if constexpr (WIDE) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src + lane * 16));
        const uint4 hi = __ldg(reinterpret_cast<const uint4*>(src + lane * 16) + 1);
        w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
        w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
        rot = __ldg(reinterpret_cast<const uint32_t*>(src + 512 + lane * 2));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = __ldg(src + lane * 16 + 2 * j) | ((uint32_t)__ldg(src + lane * 16 + 2 * j + 1) << 16);
        rot = __ldg(src + 512 + lane * 2) | ((uint32_t)__ldg(src + 512 + lane * 2 + 1) << 16);
    }
    // largest magnitude, as bits: a NaN is above infinity and so becomes the scale (and the whole block)
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
    const float amax = __uint_as_float(top);
    const uint32_t sbyte = e4m3x2(__fdiv_rn(amax, 6.f), 0.f) & 0xffu;
    uint32_t sh;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"((unsigned short)sbyte));
    const float s = __low2float(*reinterpret_cast<__half2*>(&sh));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t code[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // x / s: one correction makes a quotient that fp32 can hold exact, so ties between two codes
            // are seen as ties.  Beyond 6 s every x takes the largest code; clamping keeps infinity finite.
            float x = k & 1 ? bf_hi(w[4 * j + (k >> 1)]) : bf_lo(w[4 * j + (k >> 1)]);
            x = fminf(fmaxf(x, -4096.f), 4096.f);
            const float q = x * r;
            y[k] = copysignf(__fmaf_rn(__fmaf_rn(-q, s, x), r, q), x);  // (the sum would lose the sign of -0)
        }
        code[j] = e2m1x8(y);
    }
    uint8_t* dst = a.cache + slot * LI_KV4_ROW_BYTES;
    *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(code[0], code[1]);
    dst[256 + lane] = (uint8_t)sbyte;
    *reinterpret_cast<uint32_t*>(dst + 288 + lane * 4) = rot;
}

// e2m1 x e4m3 has 6 significant bits, so the bf16 row is exact.  A slot < 0 reads as zeros.
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

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace

li_status launch_block_tables(const BlockTableArgs& a, cudaStream_t st) {
    const size_t smem = (size_t)2 * (a.requests + 1) * sizeof(int32_t);
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
    int items = 0;
    for (int i = 0; i < a.n; ++i) {
        RopeTensor& t = a.t[i];
        const int v = a.wide ? (t.bf16 ? 8 : 4) : 1;
        const int rot = t.half ? a.rot_dim / 2 / v : a.wide ? a.rot_dim / v : a.rot_dim / 2;
        t.per_head = rot + (t.in_place ? 0 : (t.dim - a.rot_dim) / v);
        items += t.heads * t.per_head;
        t.end = items;
    }
    a.items = items;
    // a CTA's run: two items a thread, more when the tokens alone fill the GPU several times over
    const int run = RP_THREADS * RP_UNROLL;
    int chunks = ceil_div(items, run);
    const int wanted = ceil_div(16LL * host_num_sms(), a.tokens);
    if (chunks > wanted) chunks = wanted;
    a.chunk = ceil_div(items, chunks);
    chunks = ceil_div(items, a.chunk);
    const size_t smem = (size_t)(a.rot_dim / 2) * sizeof(float2);
    const dim3 grid(a.tokens, chunks);
    const cudaError_t e = a.wide ? launch_pdl(rope_wide_kernel, grid, dim3(RP_THREADS), smem, st, 1, a)
                                 : launch_pdl(rope_single_kernel, grid, dim3(RP_THREADS), smem, st, 1, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return host_check_launch();
}

li_status launch_kv4_write(const Kv4Args& a, cudaStream_t st) {
    const dim3 grid(ceil_div(a.n, K4_THREADS / 32));
    const cudaError_t e = a.wide ? launch_pdl(kv4_write_kernel<true>, grid, dim3(K4_THREADS), 0, st, 1, a)
                                 : launch_pdl(kv4_write_kernel<false>, grid, dim3(K4_THREADS), 0, st, 1, a);
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
