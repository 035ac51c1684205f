// Attention over a paged latent cache, for a token's selected positions or for
// a sliding window with first positions that stay visible (sinks):
//
//   o[t,h,:] = sum_s p_s c[s, :512],   p = softmax over the visible s of scale * (q[t,h,:] . c[s,:])
//
// in the absorbed-MLA form (a cache row is 512 latent + 64 rotary elements,
// shared by every head).  A row is held in 4 bits (LI_KV4_ROW_BYTES: 512 e2m1
// codes, one e4m3 scale per 16 of them, 64 bf16) or as 576 bf16.  e2m1 x e4m3
// has 6 significant bits, so a 4-bit row is expanded to bf16 exactly and the
// two formats share everything behind the rows' expansion.
//
// One CTA (one per SM, persistent) takes units of one token, 64, 32 or 16 heads and
// a share of the token's visible positions, 128 positions (a tile) at a time.
// Sixteen warps do all that is not a matrix product, in turn: they bring a tile's
// rows into shared memory, and when its scores are done they make its weights.
//   - Rows: each tile's rows lie once in shared memory, as bf16 in nine 16 KB chunks
//     of 64 elements x 128 positions (128-byte swizzle), handed over in pairs.
//     bf16 rows and the rotary part of 4-bit rows come by gathers of the copy engine,
//     four rows of a chunk each (16-byte cp.async by the threads kept the load-store
//     unit busy for 4000 cycles a tile: the window below took 385 us).  The 4-bit
//     codes of a row belong to four threads: each holds its quarter in registers a
//     whole tile ahead (the row's page two and its position three tiles ahead, one
//     dependent load each) and expands it pair by pair.
//   - Weights: one position per TMEM lane, a quarter of the heads per group of four
//     warps.  The running maximum of a head is raised only when a tile exceeds it by
//     more than 2^8 (p stays below 2^8, which bf16 and the fp32 sums hold as exactly
//     as p <= 1), so after a unit's first tile no maximum is exchanged and O is
//     rescaled in TMEM almost never.  p is rounded to bf16 for the product (at most 2^-8
//     of it, the same step as the bf16 output's); the fp32 sums are of the rounded p, so
//     the weights that the rows get sum to one, and what the rows have in common comes
//     through unchanged.
//   - Warp 16 issues S^T = K Q^T (M = 128 positions, N = the unit's heads, K = 576) and
//     O^T += V^T P^T (M = 128 latent elements, four blocks, K = 128), both
//     from the same chunks: K is read K-major, V^T MN-major, so nothing is loaded
//     or transposed a second time.  P takes the rotary chunk's place, which V does
//     not need and whose scores are done by then.
// A pair is released as soon as its value product is done, so the next tile's rows
// come in under this tile's value product.
// What bounds it is the chain of a tile, since a tile's rows fill shared memory: its
// 68 products take 48 cycles each at 64 heads (40 at 32 or 16; at 128 heads 64, but
// TMEM has no room for their O), the weights between them about 1000, and the rows
// of a pair (540 to 700 cycles to expand, about 1000 to gather) are hidden only
// under the value products of the pairs behind it.  Measured: 2.8 us a tile of 64
// heads in 4 bits with few CTAs, 3.5 with all SMs busy (128 heads over a window of
// 131071: 67 us, 0.54 PFLOP/s); bf16 2.7 and 3.4 (1024 tokens x 128 heads, window
// 512: 281 us, 0.54 PFLOP/s).
// With few units the visible tiles are split over several CTAs; a second kernel
// merges the parts (see paged_attn_plan for the rule).
#include <cuda_fp16.h>

#include "li_common.cuh"
#include "li_kernels.cuh"

namespace li {

namespace {

constexpr int PA_D = 576;
constexpr int PA_DV = 512;
constexpr int PA_M = 128;                  // positions per tile
constexpr int PA_CH = PA_D / 64;           // 9 chunks of 64 elements
constexpr int PA_VCH = PA_DV / 64;         // 8 of them hold the value
constexpr int PA_PAIRS = PA_VCH / 2 + 1;   // chunks are handed over in twos (one block of V^T), the rotary one alone
constexpr int PA_CHUNK = PA_M * 128;       // 16 KB
constexpr int PA_WORKERS = 512;            // warps 0-15
constexpr int PA_THREADS = PA_WORKERS + 32;
constexpr float PA_RAISE = 8.f;            // log2: a head's maximum is raised when exceeded by more
constexpr float PA_NOTHING = -3e38f;       // the reference of a head without a logit yet: any is more than PA_RAISE above

// What depends on NH, the heads of a unit (MMA N): 64, 32 or 16.
template <int NH>
struct Pa {
    static constexpr int GH = NH / 4;                     // heads per softmax group of four warps
    static constexpr int QCHUNK = NH * 128;               // the query's 64 elements of every head
    static constexpr int O_COL = NH;                      // TMEM: S^T in NH columns, O^T in 4 x NH
    static constexpr int TMEM_COLS = NH == 64 ? 512 : NH == 32 ? 256 : 128;
    static constexpr int K = PA_CH * QCHUNK;              // shared memory: query, rows, then
    static constexpr int RED = K + PA_CH * PA_CHUNK;      // [4 groups][4 warps][GH] fp32
    static constexpr int MAXI = RED + 16 * GH * 4;        // [16 warps][GH] fp32: maxima in use; factors
    static constexpr int VALID = MAXI + 16 * GH * 4;      // [2][128] bytes
    static constexpr int STAGE = VALID + 2 * PA_M;        // [4 groups] 2 KB: output on its way to whole lines
    static constexpr int BAR = STAGE + 4 * 2048;          // full[5], empty[5], qfull, sdone, pready, odone
    static constexpr int NBAR = 2 * PA_PAIRS + 4;
    static constexpr int TMEM = BAR + NBAR * 8;
    static constexpr int SMEM = TMEM + 16;                // the base is 1024-byte aligned (checked)
};
static_assert(Pa<64>::SMEM <= 232448, "shared memory per CTA");
static_assert(Pa<16>::SMEM + kScorerSmem > kSmemPerSm, "no scorer beside it (see pdl_wait)");
static_assert(Pa<16>::K % 1024 == 0, "the rows' swizzle atoms");

// 64 bf16 elements (from x) of four rows of the cache, 128 bytes each, side by side at dst in the swizzled layout;
// a row past the end reads as zeros.  The map's box is one row high.
__device__ __forceinline__ void pa_gather4(uint32_t dst, const void* map, int x, const int (&row)[4], uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float pa_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A thread's part of a row, read a tile ahead of its use.  Zeros where there is no row.
__device__ __forceinline__ uint4 early16(const uint8_t* p) {
    return p ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint2 early8(const uint8_t* p) {
    return p ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
}

// 3-D tiled load (see tma_load_2d).
__device__ __forceinline__ void pa_tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar,
                                               uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// 32 lanes x 4, 8 or 16 columns (see tmem_ld32), and back.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Barrier over a group's 128 threads; group_any also returns whether any of them said yes.
__device__ __forceinline__ void group_sync(int bar) { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); }
__device__ __forceinline__ bool group_any(int bar, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(bar), "r"((uint32_t)yes)
        : "memory");
    return r != 0;
}

// Reduction of N values over the warp: lane l ends with v[0] reduced for index l % N (log2 N steps keep
// the half selected by one lane bit, the others join lanes that hold the same index).
template <bool MAX, int N>
__device__ __forceinline__ void warp_reduce_scatter(float (&v)[N], int lane) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = upper ? v[i] : v[i + o];
            const float keep = upper ? v[i + o] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = MAX ? fmaxf(keep, recv) : keep + recv;
        }
    }
#pragma unroll
    for (int o = N; o < 32; o <<= 1) {
        const float recv = __shfl_xor_sync(0xffffffffu, v[0], o);
        v[0] = MAX ? fmaxf(v[0], recv) : v[0] + recv;
    }
}

// What a unit works on.  Entry j of a token's visible list is position j for
// j < nsink and first + j after that.
struct PaUnit {
    int row, hg, req;
    int n;              // length of the visible list (selection slots or window positions)
    int nsink;
    int first;          // window: position of list entry j >= nsink is first + j
    int t0, t1;         // tiles of the list this unit takes
    bool live;          // the token is no padding (and its request and position are in range)
};

// A token's row is left as it was when it is padding (request or position < 0) or names a request or a
// position out of range (reported).
__device__ __forceinline__ bool token_of(const PagedAttnArgs& a, int row, int* req, int* pos, bool report) {
    const int r = a.req ? __ldg(a.req + row) : row;
    int p = 0;
    if (a.pos) p = __ldg(a.pos + row);
    *req = r;
    *pos = p;
    if (r < 0 || p < 0) return false;
    if (r >= a.requests || (a.pos && p >= a.max_len)) {
        if (report) record_error(a.err, ERRBIT_BOUNDS);
        return false;
    }
    return true;
}

__device__ __forceinline__ PaUnit unit_of(const PagedAttnArgs& a, int u, bool report) {
    PaUnit x;
    const unsigned v = (unsigned)u / (unsigned)a.hgroups, split = v % (unsigned)a.splits;
    x.hg = (int)((unsigned)u - v * (unsigned)a.hgroups);
    x.row = (int)(v / (unsigned)a.splits);
    int p;
    x.live = token_of(a, x.row, &x.req, &p, report);
    x.nsink = 0;
    x.first = 0;
    x.n = a.k;
    if (a.pos) {
        const int w0 = p + 1 > a.window ? p + 1 - a.window : 0;   // first position of the window
        x.nsink = min(a.sinks, w0);
        x.first = w0 - x.nsink;
        x.n = x.nsink + (p + 1 - w0);
    }
    if (!x.live) x.n = 0;
    // (at most 2^21 tiles, and no more splits than units of four waves: 32 bits hold the product, and a 64-bit
    // division would take longer than a load)
    const unsigned nt = (unsigned)(x.n + PA_M - 1) / PA_M;
    x.t0 = (int)(nt * split / (unsigned)a.splits);
    x.t1 = (int)(nt * (split + 1) / (unsigned)a.splits);
    return x;
}

// A tile entry on its way to a row address, one dependent load a step.
constexpr int PA_BEYOND = 0x7fffffff;  // (no request: those are below the number of requests)
struct PaEntry {
    int s;              // position in the request, < 0: none
    int req;            // PA_BEYOND: the list has ended before the warp's rows
    int page;           // of the cache, < 0: none
};
// Step 1: entry j of the unit's list.
__device__ __forceinline__ void entry_position(const PagedAttnArgs& a, const PaUnit& x, int j, PaEntry& e) {
    e.req = x.req;
    e.s = -1;
    if (j < x.n) e.s = a.pos ? (j < x.nsink ? j : x.first + j) : __ldg(a.sel + (size_t)x.row * a.k + j);
}
// Step 2: its page.
__device__ __forceinline__ void entry_page(const PagedAttnArgs& a, PaEntry& e) {
    e.page = -1;
    if (e.s < 0) {
        if (e.s < -1) record_error(a.err, ERRBIT_BOUNDS);
        return;
    }
    if ((long long)e.s >= (long long)a.max_blocks * a.page_size) {
        record_error(a.err, ERRBIT_BOUNDS);
        e.s = -1;
        return;
    }
    const long long at = (long long)e.req * a.max_blocks + divided(e.s, a.by_page);
    e.page = a.table ? __ldg(a.table + at) : (int)at;
}
// Step 3: its slot of the cache, < 0 for none.
__device__ __forceinline__ long long entry_slot(const PagedAttnArgs& a, const PaEntry& e) {
    if (e.s < 0) return -1;
    if ((unsigned)e.page >= (unsigned)a.num_pages) {
        record_error(a.err, ERRBIT_BOUNDS);
        return -1;
    }
    return (long long)e.page * a.page_size + (e.s - divided(e.s, a.by_page) * a.page_size);
}

// A walk over the CTA's tiles.
struct PaWalk {
    PaUnit x;
    int u, t;
    bool more;
    __device__ __forceinline__ void start(const PagedAttnArgs& a) {
        u = blockIdx.x;
        seek(a);
    }
    __device__ __forceinline__ void seek(const PagedAttnArgs& a) {
        for (more = false; u < a.units; u += gridDim.x) {
            x = unit_of(a, u, false);
            if (x.t0 < x.t1) {
                t = x.t0;
                more = true;
                return;
            }
        }
    }
    __device__ __forceinline__ void next(const PagedAttnArgs& a) {
        if (++t == x.t1) {
            u += gridDim.x;
            seek(a);
        }
    }
};

// Eight e2m1 codes (element i in bits 4i..4i+3) times their block's scale, as four bf16 pairs.  The
// product has 6 significant bits and lies between 2^-10 and 2688: exact in fp16 and in bf16.  (Placing the
// codes' bits in bf16 with shifts and masks takes five integer instructions a pair, and the integer pipe
// runs at half rate: 620 cycles a pair of chunks against 540 this way.)
__device__ __forceinline__ void expand8(uint32_t w, __half2 scale, uint32_t (&o)[4]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(*reinterpret_cast<__half2*>(&h[i]), scale));
        __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
        o[i] = *reinterpret_cast<uint32_t*>(&p);
    }
}
// Two e4m3 scales.
__device__ __forceinline__ __half2 scales2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    return *reinterpret_cast<__half2*>(&h);
}

// A warp's N values of shared memory (16-byte aligned) in every lane.
template <int N>
__device__ __forceinline__ void read_factors(const float* m, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(m + i);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
    }
}

template <bool FP4, int NH>
__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const PagedAttnArgs a) {
    using L = Pa<NH>;
    constexpr int GH = L::GH, HB = GH < 8 ? GH : 8, PASSES = GH / HB;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* qs = smem;
    uint8_t* ks = smem + L::K;
    uint8_t* ps = ks + (PA_CH - 1) * PA_CHUNK;  // P over the rotary chunk
    float* red = reinterpret_cast<float*>(smem + L::RED);
    float* msm = reinterpret_cast<float*>(smem + L::MAXI);
    uint8_t* vflag = smem + L::VALID;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR);
    uint64_t* empty = full + PA_PAIRS;
    uint64_t* qfull = empty + PA_PAIRS;
    uint64_t* sdone = qfull + 1;
    uint64_t* pready = sdone + 1;
    uint64_t* odone = pready + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::TMEM);

    if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it; every thread sees the same address
        if (threadIdx.x == 0) record_error(a.err, ERRBIT_BOUNDS);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < PA_PAIRS; ++i) {
            mbar_init(&full[i], PA_WORKERS / 32);
            mbar_init(&empty[i], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(sdone, 1);
        mbar_init(pready, PA_WORKERS / 32);
        mbar_init(odone, 1);
        fence_mbar_init();
    }
    if (warp == 16 && lane == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
    }
    pdl_wait();  // the query, the selection and the cache may come from the previous kernel of the stream
    if (warp == 16) {  // (behind the wait: see pdl_wait)
        tmem_alloc(tmem_slot, L::TMEM_COLS);
        tmem_relinquish();
    }
    // No early trigger for the merge or the stream's next kernel: their waiting blocks cost more than they gain (one at
    // the head of the kernel: 8 x 128 heads over 2048 rows 22.3 us against 19.8, 128 heads over 131071 71.0 against
    // 66.8, 1 x 64 11.8 against 11.7; a two-stream step of 8 layers, 8 x 128 heads, 350 against 316).
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 16) {
        // ---------------------------------------------------------------- query loads and MMA issue
        // The whole warp walks and waits (so that the operands stay in uniform registers); one lane issues.
        constexpr uint32_t IDESC_S = idesc_f32acc(PA_M, NH, kFmtBF16);
        constexpr uint32_t IDESC_O = idesc_f32acc(128, NH, kFmtBF16) | (1u << 15) | (1u << 16);
        // start addresses are in units of 16 bytes in the low 14 bits and stay below 2^14: plain additions
        const uint64_t k_desc = sw128_kmajor_desc(smem_u32(ks)), q_desc = sw128_kmajor_desc(smem_u32(qs));
        const uint64_t v_desc = sw128_mnmajor_desc(smem_u32(ks), PA_CHUNK, 1024);
        const uint64_t p_desc = sw128_mnmajor_desc(smem_u32(ps), PA_CHUNK, 1024);
        const bool one = elect_one();
        auto load_q = [&](const PaUnit& x) {
            if (one) {
                mbar_arrive_expect_tx(qfull, PA_CH * L::QCHUNK);
                for (int c = 0; c < PA_CH; ++c)
                    pa_tma_load_3d(qs + c * L::QCHUNK, &qmap, c * 64, x.hg * NH, x.row, qfull,
                                   l2_policy_evict_last());
            }
        };
        PaWalk w;
        w.start(a);
        uint32_t n = 0, units = 0, loads = 0;
        bool ok = true;
        if (w.more) {
            load_q(w.x);
            ++loads;
        }
        while (w.more && ok) {
            ok = mbar_wait(qfull, units & 1, a.err);
            const int tiles = w.x.t1 - w.x.t0;
            for (int t = 0; ok && t < tiles; ++t, ++n) {
                const uint32_t par = n & 1;
                // The last tile's value product ends with the 16 positions that hold the list's last entry, and bf16
                // rows behind them are not fetched (window 512 after 16 first positions, 1024 x 128 heads: 299 ->
                // 292 us; the same skip in the expansion of 4-bit rows cost registers: 69.4 -> 72.5 us over 131071).
                const int steps = (min(w.x.n - (w.x.t0 + t) * PA_M, PA_M) + 15) / 16;
#pragma unroll
                for (int p = 0; p < PA_PAIRS; ++p) {
                    ok = ok && mbar_wait(&full[p], par, a.err);
                    if (ok && one) {
#pragma unroll
                        for (int kk = 0; kk < (p < PA_PAIRS - 1 ? 8 : 4); ++kk)
                            mma_bf16(tmem_base, k_desc + (2 * p + kk / 4) * (PA_CHUNK >> 4) + (kk & 3) * 2,
                                     q_desc + (2 * p + kk / 4) * (L::QCHUNK >> 4) + (kk & 3) * 2, IDESC_S,
                                     (p | kk) != 0);
                    }
                }
                if (!ok) break;
                if (one) tc_commit(sdone);
                if (!mbar_wait(pready, par, a.err)) { ok = false; break; }  // (and the unit before has read its O)
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int blk = 0; blk < PA_VCH / 2; ++blk) {
#pragma unroll
                        for (int s = 0; s < PA_M / 16; ++s)
                            if (s < steps) mma_bf16(tmem_base + (uint32_t)(L::O_COL + blk * NH),
                                     v_desc + (2 * blk * PA_CHUNK + s * 2048) / 16, p_desc + s * 2048 / 16, IDESC_O,
                                     (t | s) != 0);
                        tc_commit(&empty[blk]);
                    }
                    tc_commit(&empty[PA_PAIRS - 1]);
                    if (t == tiles - 1) tc_commit(odone);
                }
            }
            if (!ok) break;
            ++units;
            w.t = w.x.t1 - 1;
            w.next(a);
            if (w.more) {  // the scores of this unit are done (its last P has been made from them)
                load_q(w.x);
                ++loads;
            }
        }
        if (loads > units) mbar_wait(qfull, (loads - 1) & 1, a.err);  // leave no copy in flight
    } else {
        // ---------------------------------------------------------------- rows, softmax and output
        // rows: a thread's half of one chunk of each pair; eight neighbouring threads of a store share a chunk and
        // differ in their swizzled 16-byte unit, so stores meet no bank twice
        const int r = warp * 8 + ((lane >> 1) & 7), hi = lane >> 4, half = lane & 1;
        // (unit 4 half + i of the row lies at dst0 ^ 16 i: the swizzle is an exclusive or of the unit)
        const uint32_t dst0 = smem_u32(ks) + hi * PA_CHUNK + sw128_offset(r, 4 * half);
        const uint32_t rdst = smem_u32(ks) + (PA_CH - 1) * PA_CHUNK + warp * 8 * 128;
        // softmax: GH heads of group g; q4 is the warp's quarter of the TMEM lanes
        const int g = warp >> 2, q4 = warp & 3;
        const int row = q4 * 32 + lane;            // position of the tile; latent element of an O block
        const uint32_t s_at = tmem_base + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(g * GH);
        const float c2 = a.scale * 1.4426950408889634f;  // exp(x) = exp2(x log2 e)
        float* gred = red + g * 4 * GH;
        float* wm = msm + warp * GH;
        const int bar = 1 + g;

        // Lookups run ahead of the rows, one dependent load a tile, under the score products: behind tile np the
        // thread's part of tile np + 1 is read (4 bits), the page of np + 2 and the position of np + 3.
        PaWalk w;
        w.start(a);
        // Tiles of a unit, < 0 for padding: looked up while the unit before still has its value product to wait for (at
        // the head of each unit the loads and divisions took 1700 cycles: 292 -> 281 us for 1024 tokens x 128 heads).
        const auto tiles_of = [&](int u) {
            if (u >= a.units) return -1;
            const PaUnit x = unit_of(a, u, threadIdx.x == 0);
            return x.live ? x.t1 - x.t0 : -1;
        };
        int tiles = tiles_of(blockIdx.x);
        PaEntry e1{-1, -1, -1}, e2{-1, -1, -1};
        uint4 code[FP4 ? 4 : 1];
        uint2 sc = make_uint2(0, 0);                // 4 bits: pair 2 hi + half's eight scales
        int src = 0;                                // the slot of the thread's row of tile np
        bool here = false;                          // it exists
        bool more = false;                          // tile np exists
        uint32_t np = 0;                            // tiles brought in
        bool ok = true;
        const auto position = [&](PaEntry& e) {     // of the next tile of the walk
            e.s = -1;
            e.req = w.more ? 0 : -1;                // (-1: no such tile)
            if (w.more) {
                entry_position(a, w.x, w.t * PA_M + r, e);
                if (!FP4 && w.t * PA_M + (warp & ~1) * 8 >= w.x.n) e.req = PA_BEYOND;  // (16 rows of two warps)
                w.next(a);
            }
        };
        auto look_ahead = [&]() {
            more = e1.req >= 0;
            const long long slot = entry_slot(a, e1);
            here = slot >= 0;
            // (no row: past every end, where a gather fills in zeros; -1: not even that)
            src = here ? (int)slot : !FP4 && e1.req == PA_BEYOND ? -1 : 0x7fffffff;
            if constexpr (FP4) {
                const uint8_t* from = here ? static_cast<const uint8_t*>(a.cache) + slot * LI_KV4_ROW_BYTES : nullptr;
#pragma unroll
                for (int p = 0; p < 3; ++p) code[p] = early16(from ? from + p * 64 + hi * 32 + half * 16 : nullptr);
                sc = early8(from ? from + 256 + (2 * hi + half) * 8 : nullptr);
            }
            e1 = e2;
            entry_page(a, e1);
            position(e2);
        };
        // Brings tile np in, pair by pair as the tile before releases them.
        auto bring = [&]() {
            const uint32_t free_parity = (np & 1) ^ 1;
            if (hi == 0 && half == 0) vflag[(np & 1) * PA_M + r] = here ? 1 : 0;  // (last read two tiles ago)
            if (!FP4 && src == -1) {  // (the whole warp) the value product ends before these rows: they stay as they are
                __syncwarp();
                if (lane == 0)
                    for (int p = 0; p < PA_PAIRS; ++p) mbar_arrive(&full[p]);
                ++np;
                look_ahead();
                return;
            }
            // the warp's eight rows make two gathers of four
            const int group = FP4 ? lane & 1 : lane >= 9;
            int four[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) four[i] = __shfl_sync(0xffffffffu, src, 2 * (4 * group + i));
            if constexpr (FP4) {
                // (the last pair's codes, a tile's time late: they are wanted last, and registers are short)
                const uint8_t* from =
                    here ? static_cast<const uint8_t*>(a.cache) + (long long)src * LI_KV4_ROW_BYTES : nullptr;
                code[3] = early16(from ? from + 3 * 64 + hi * 32 + half * 16 : nullptr);
                uint32_t sw[4];
#pragma unroll
                for (int p = 0; p < PA_PAIRS - 1; ++p) {
                    const int from = (lane & 14) | (p & 1) | ((p & 2) << 3);
                    const uint32_t w0 = __shfl_sync(0xffffffffu, sc.x, from), w1 = __shfl_sync(0xffffffffu, sc.y, from);
                    sw[p] = hi ? w1 : w0;
                }
                uint32_t o[2][4];
                const __half2 sA = scales2((sw[0] >> (16 * half)) & 0xffffu);
                expand8(code[0].x, __low2half2(sA), o[0]);
                expand8(code[0].y, __low2half2(sA), o[1]);
#pragma unroll
                for (int p = 0; p < PA_PAIRS - 1; ++p) {
                    const __half2 s = scales2((sw[p] >> (16 * half)) & 0xffffu);
                    const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
                    ok = ok && mbar_wait(&empty[p], free_parity, a.err);
                    const uint32_t at = dst0 + 2 * p * PA_CHUNK;
                    st_shared16(at, o[0][0], o[0][1], o[0][2], o[0][3]);
                    st_shared16(at ^ 16, o[1][0], o[1][1], o[1][2], o[1][3]);
                    expand8(code[p].z, s1, o[0]);
                    st_shared16(at ^ 32, o[0][0], o[0][1], o[0][2], o[0][3]);
                    expand8(code[p].w, s1, o[0]);
                    st_shared16(at ^ 48, o[0][0], o[0][1], o[0][2], o[0][3]);
                    if (p < PA_PAIRS - 2) {  // the next pair's first words, while the stores drain before the fence
                        const __half2 sn = scales2((sw[p + 1] >> (16 * half)) & 0xffffu);
                        expand8(code[p + 1].x, __low2half2(sn), o[0]);
                        expand8(code[p + 1].y, __low2half2(sn), o[1]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[p]);
                    if (p == PA_PAIRS - 3) {  // the rotary part (free by now) comes in under the last pair's expansion
                        ok = ok && mbar_wait(&empty[PA_PAIRS - 1], free_parity, a.err);
                        if (lane == 0) mbar_arrive_expect_tx(&full[PA_PAIRS - 1], 8 * 128);
                        __syncwarp();
                        if (lane < 2)  // (it lies behind the codes and scales)
                            pa_gather4(rdst + lane * 512, &kmap, (PA_DV / 2 + PA_DV / 16) / 2, four,
                                       &full[PA_PAIRS - 1]);
                    }
                }
            } else {
                const int chunk = lane - 9 * group;  // lanes 0-8 take the first one's chunks, 9-17 the second's
                const uint32_t to = smem_u32(ks) + chunk * PA_CHUNK + (warp * 8 + 4 * group) * 128;
#pragma unroll
                for (int p = 0; p < PA_PAIRS; ++p) {
                    ok = ok && mbar_wait(&empty[p], free_parity, a.err);
                    if (lane == 0) mbar_arrive_expect_tx(&full[p], (p < PA_PAIRS - 1 ? 2 : 1) * 8 * 128);
                    __syncwarp();
                    if (lane < 18 && chunk >> 1 == p) pa_gather4(to, &kmap, chunk * 64, four, &full[p]);
                }
            }
            ++np;
            look_ahead();
        };
        if (w.more) {
            position(e1);
            entry_page(a, e1);
            position(e2);
            look_ahead();
            bring();
        }

        uint32_t n = 0, units = 0;
        for (int u = blockIdx.x, next; ok && u < a.units; u += gridDim.x, tiles = next) {
            if (tiles <= 0) next = tiles_of(u + gridDim.x);
            if (tiles < 0) continue;
            // where the unit's output goes (worked out again at its end: registers are short)
            const int h0 = (u % a.hgroups) * NH + g * GH;
            const int nh = min(GH, a.heads - h0);   // heads of this group that exist (may be <= 0)
            if (tiles == 0) {  // nothing visible in this share
                const size_t part = (size_t)(u / a.hgroups) * a.heads + h0;
                if (a.splits > 1) {
                    if (q4 == 0 && lane < nh) {
                        a.mpart[part + lane] = -INFINITY;
                        a.lpart[part + lane] = 0.f;
                    }
                } else {
                    for (int i = row; i < nh * (PA_DV / 2); i += 128)
                        reinterpret_cast<uint32_t*>(a.out + part * PA_DV)[i] = 0u;  // (one part per token)
                }
                continue;
            }
            const bool whole = a.splits == 1;
            const size_t part = (size_t)(u / a.hgroups) * a.heads + h0;  // [row][split][head]
            float m_run[PASSES];      // of head h0 + HB pass + lane % HB, the same in the group's four warps
            float l[GH];              // sums over this thread's positions, per head
#pragma unroll
            for (int i = 0; i < PASSES; ++i) m_run[i] = -INFINITY;
#pragma unroll
            for (int i = 0; i < GH; ++i) l[i] = 0.f;
            for (int t = 0; t < tiles; ++t, ++n) {
                // full[0] orders the other threads' flags before this read; it stays in this phase until the
                // tile's value product has released the pair
                if (!mbar_wait(&full[0], n & 1, a.err) || !mbar_wait(sdone, n & 1, a.err)) { ok = false; break; }
                tc_fence_after();
                const bool valid = vflag[(n & 1) * PA_M + row] != 0;
#pragma unroll
                for (int pass = 0; pass < PASSES; ++pass) {  // HB heads at a time: registers are short
                    const uint32_t at = s_at + pass * HB;
                    float* w8 = wm + pass * HB;
                    uint32_t s[HB];
                    bool high = t == 0;  // no maximum yet
                    if (!high) {
                        float m[HB], top = -INFINITY;
                        tmem_ld(at, s);
                        read_factors(w8, m);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < HB; ++i) {
                            const float x = __fmaf_rn(__uint_as_float(s[i]), c2, -m[i]);
                            top = fmaxf(top, x);
                            s[i] = __float_as_uint(pa_ex2(x));
                        }
                        // a position over some head's maximum by more than PA_RAISE: the group takes new ones
                        high = group_any(bar, valid && top > PA_RAISE);
                    }
                    if (high) {
                        float v[HB];
                        tmem_ld(at, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < HB; ++i) v[i] = valid ? __uint_as_float(s[i]) * c2 : -INFINITY;
                        warp_reduce_scatter<true>(v, lane);
                        float* r8 = gred + pass * 4 * HB;
                        if (lane < HB) r8[q4 * HB + lane] = v[0];
                        group_sync(bar);
                        const int k = lane % HB;
                        const float mx = fmaxf(fmaxf(r8[k], r8[HB + k]), fmaxf(r8[2 * HB + k], r8[3 * HB + k]));
                        const bool raise = mx > m_run[pass] + PA_RAISE;
                        const float m_use = raise ? mx : m_run[pass];
                        const float f = raise && m_run[pass] != -INFINITY ? pa_ex2(m_run[pass] - m_use) : 1.f;
                        const bool rescale = __any_sync(0xffffffffu, f != 1.f);  // the same in the group's four warps
                        m_run[pass] = m_use;
                        if (rescale) {  // O of the tiles before is complete: its commit came before sdone's
                            __syncwarp();
                            if (lane < HB) w8[lane] = f;
                            __syncwarp();
                            read_factors(w8, v);
#pragma unroll
                            for (int i = 0; i < HB; ++i) l[pass * HB + i] *= v[i];
#pragma unroll 1
                            for (int blk = 0; blk < PA_DV / 128; ++blk) {
                                const uint32_t o_at = at + (uint32_t)(L::O_COL + blk * NH);
                                tmem_ld(o_at, s);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < HB; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * v[i]);
                                tmem_st(o_at, s);
                            }
                            tmem_st_wait();
                        }
                        tmem_ld(at, s);  // (read again rather than held: registers are short)
                        tmem_ld_wait();
                        __syncwarp();
                        if (lane < HB) w8[lane] = m_use == -INFINITY ? PA_NOTHING : m_use;
                        __syncwarp();
                        read_factors(w8, v);
#pragma unroll
                        for (int i = 0; i < HB; ++i)
                            s[i] = __float_as_uint(pa_ex2(__fmaf_rn(__uint_as_float(s[i]), c2, -v[i])));
                    }
                    if (!__all_sync(0xffffffffu, valid)) {
#pragma unroll
                        for (int i = 0; i < HB; ++i) s[i] = valid ? s[i] : 0u;
                    }
                    uint32_t pk[HB / 2];
#pragma unroll
                    for (int j = 0; j < HB / 2; ++j) {
                        __nv_bfloat162 pp =
                            __floats2bfloat162_rn(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                        pk[j] = *reinterpret_cast<uint32_t*>(&pp);
                    }
                    if constexpr (HB == 8)
                        *reinterpret_cast<uint4*>(ps + sw128_offset(row, PASSES * g + pass)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    else
                        *reinterpret_cast<uint2*>(ps + sw128_offset(row, g >> 1) + 8 * (g & 1)) =
                            make_uint2(pk[0], pk[1]);
#pragma unroll
                    for (int j = 0; j < HB / 2; ++j) {  // (what the product takes, not what was rounded to it)
                        l[pass * HB + 2 * j] += __uint_as_float(pk[j] << 16);
                        l[pass * HB + 2 * j + 1] += __uint_as_float(pk[j] & 0xffff0000u);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready);
                if (t == tiles - 1) {  // the sums, while the value product runs
                    warp_reduce_scatter<false>(l, lane);
                    if (lane < GH) wm[lane] = l[0];  // (another warp may still read the maxima in red)
                    group_sync(bar);
                    const float* parts = msm + g * 4 * GH + lane % GH;
                    const float sum = (parts[0] + parts[GH]) + (parts[2 * GH] + parts[3 * GH]);
                    group_sync(bar);
                    if (!whole && q4 == 0 && lane < nh) {
                        // (m_run is of head lane % HB)
                        const float m = PASSES == 1 || lane < HB ? m_run[0] : m_run[PASSES - 1];
                        // without a maximum the sum is 0 (nothing visible) or NaN, which the merge does not drop
                        a.mpart[part + lane] = m == -INFINITY && sum != 0.f ? 0.f : m;
                        a.lpart[part + lane] = sum;
                    }
                    if (lane < GH) wm[lane] = sum == 0.f ? 0.f : 1.f / sum;
                    __syncwarp();
                }
                if (more) bring();
                if (!ok) break;
            }
            if (!ok) break;
            next = tiles_of(u + gridDim.x);
            if (!mbar_wait(odone, units & 1, a.err)) { ok = false; break; }
            tc_fence_after();
            ++units;
            float fac[GH];
            read_factors(wm, fac);
#pragma unroll 1
            for (int blk = 0; blk < PA_DV / 128; ++blk) {
                uint32_t s[GH];
                tmem_ld(s_at + (uint32_t)(L::O_COL + blk * NH), s);
                tmem_ld_wait();
                if (whole) {
                    // Each lane holds one latent element of GH heads; the group's stage, [8 heads][128 elements] in
                    // bf16, turns that into 16 bytes of a head's 256-byte run per thread.
                    __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem + L::STAGE + g * 2048);
#pragma unroll
                    for (int b8 = 0; b8 < (GH + 7) / 8; ++b8) {
#pragma unroll
                        for (int i = 0; i < (GH < 8 ? GH : 8); ++i)
                            stage[i * 128 + row] = __float2bfloat16_rn(__uint_as_float(s[8 * b8 + i]) * fac[8 * b8 + i]);
                        group_sync(bar);
                        const int hd = row >> 4, el = (row & 15) * 8, k = 8 * b8 + hd;  // (row: the thread of the group)
                        if (k < nh)
                            *reinterpret_cast<uint4*>(a.out + (part + k) * PA_DV + blk * 128 + el) =
                                *reinterpret_cast<const uint4*>(stage + hd * 128 + el);
                        group_sync(bar);
                    }
                } else {
                    float* o = a.opart + part * PA_DV + blk * 128 + row;  // whole lines: 32 elements of a head a warp
#pragma unroll
                    for (int i = 0; i < GH; ++i)
                        if (i < nh) o[(size_t)i * PA_DV] = __uint_as_float(s[i]);
                }
            }
            tc_fence_before();  // the next unit's pready hands O on
        }
        // (after a wait that ran out: leave no copy in flight)
        if (!ok)
            for (int p = 0; p < PA_PAIRS; ++p) mbar_wait(&full[p], (np & 1) ^ 1, a.err);
    }
    __syncwarp();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
}

// Merge of a token's splits: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M the
// largest m_s (maxima are in the log2 domain).  A CTA takes 512 / ST latent elements of one (head, token), four
// to a thread, the parts dealt over its ST stripes of threads, eight in flight in each; the weights are made once in
// shared memory.  Latency bound: an L2 read of the maxima, then the parts.  ST = 1 keeps the CTAs few (a whole call
// of 24 tokens x 128 heads over 2048 rows in 3 parts: 36.5 us, 43.0 with ST = 4; 8 x 128 in 8: 20.0 and 22.0), ST = 4
// shortens the walk over more than eight parts (1 x 64 in 16 parts: 11.5 us, 11.9 with ST = 1; 1 x 128 over 131071 in
// 74: 63.5 and 68.7).
constexpr int PA_MERGE = 128;
constexpr float PA_UNWRITTEN = -1.f;  // weight of a part without a visible position: it has not been written
template <int ST>
__global__ void __launch_bounds__(PA_MERGE) paged_attn_merge_kernel(const PagedAttnArgs a) {
    constexpr int LANES = PA_MERGE / ST;
    extern __shared__ float weight[];  // [splits]
    __shared__ float wred[2][PA_MERGE / 32];
    __shared__ float4 wsum[ST > 1 ? PA_MERGE : 1];
    const int h = blockIdx.x, row = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stripe = tid / LANES, d = blockIdx.y * (PA_DV / ST) + tid % LANES * 4;
    pdl_wait();
    int r, p;
    if (!token_of(a, row, &r, &p, false)) return;
    const size_t at = (size_t)row * a.splits * a.heads + h;
    float top = -INFINITY;
    for (int s = tid; s < a.splits; s += PA_MERGE) {
        const float m = a.mpart[at + (size_t)s * a.heads];
        weight[s] = m;
        top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) wred[0][warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wred[0][0], wred[0][1]), fmaxf(wred[0][2], wred[0][3]));
    float sum = 0.f;
    for (int s = tid; s < a.splits; s += PA_MERGE) {
        // (a weight that underflows still counts: a NaN in its sum or values comes through, as it does without parts)
        const float f = weight[s] == -INFINITY ? PA_UNWRITTEN : pa_ex2(weight[s] - top);
        weight[s] = f;
        if (f != PA_UNWRITTEN) sum += f * a.lpart[at + (size_t)s * a.heads];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) wred[1][warp] = sum;
    __syncthreads();
    sum = (wred[1][0] + wred[1][1]) + (wred[1][2] + wred[1][3]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = a.opart + at * PA_DV + d;
#pragma unroll 8
    for (int s = stripe; s < a.splits; s += ST) {
        const float f = weight[s];
        if (f == PA_UNWRITTEN) continue;
        const float4 o = *reinterpret_cast<const float4*>(src + (size_t)s * a.heads * PA_DV);
        acc.x += f * o.x;
        acc.y += f * o.y;
        acc.z += f * o.z;
        acc.w += f * o.w;
    }
    if constexpr (ST > 1) {
        wsum[tid] = acc;
        __syncthreads();
        if (stripe > 0) return;
#pragma unroll
        for (int i = 1; i < ST; ++i) {
            const float4 o = wsum[i * LANES + tid];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.heads + h) * PA_DV + d) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}

constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <bool FP4, int NH>
li_status launch_units(const CUtensorMap& qmap, const CUtensorMap& kmap, const PagedAttnArgs& a, cudaStream_t st) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_done[dev]) {
        if (cudaFuncSetAttribute(paged_attn_kernel<FP4, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Pa<NH>::SMEM) != cudaSuccess) {
            cudaGetLastError();
            return LI_ERR_CUDA;
        }
        if (dev < 64) attr_done[dev] = true;
    }
    const int grid = a.units < host_num_sms() ? a.units : host_num_sms();
    if (launch_pdl(paged_attn_kernel<FP4, NH>, dim3(grid), dim3(PA_THREADS), Pa<NH>::SMEM, st, 1, qmap, kmap, a) !=
        cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    return LI_OK;
}

}  // namespace

// How many heads a unit takes and how many CTAs share a token's tiles: the pair with the least estimated time,
// in microseconds.  Units run in waves of one per SM; a unit costs its tiles and a start and end that grow with
// its heads (the end writes them); parts cost a merge, and their fp32 sums are written and read once more.  For
// each number of waves the largest count of splits that fits is tried, lowered as far as the longest share stays
// the same.  The constants are fitted to whole calls; a further tile alone takes 2.8 / 2.2 / 2.0 us at 64 / 32 / 16
// heads a unit with 4-bit rows (bf16: 2.7 / 2.2 / 2.1), near enough for one set to choose well for both.  What the rule
// decides between, as measured in a graph (4 bits; bf16), its choice first: 1 token x 64 heads, 2048 rows: 16 heads in 16
// splits 11.3; 10.8, 64 heads in 16 14.6; 13.2.  8 x 128, 2048 rows: 64 in 8 19.8; 18.0, 32 in 4 21.8; 21.2, 16 in 2 30.5;
// 29.9.  32 x 128, 516 rows: 32 unsplit 20.4; 19.7, 64 in 2 25.1; 23.3, 64 unsplit 25.0; 23.0.  32 x 128, 2048 rows: 64 in 2
// 44.3; 45.4, 32 unsplit 51.5; 54.5.  74 x 16, 1000 rows: 16 in 2 20.2; 21.4, unsplit 27.6; 29.5.  1 x 128, 131071 rows: 64
// in 74 63.8; 69.3, 32 in 37 88.8; 97.5, 64 in 148 75.3; 80.3.  (4 x 128, 2048 rows: its 64 in 16 takes 16.0; 14.7, 32 in 8
// 15.5; 15.0.)  The rule knows the longest list alone: a batch of one long list and many short ones is split for the long
// one, whose units then share few SMs (32 x 128, one of 131071 and 31 of 1000 positions: 447 us, most of it on 18 SMs).
PagedAttnPlan paged_attn_plan(int rows, int heads, int positions, int sms) {
    const int tiles = (positions + PA_M - 1) / PA_M;
    static const struct {
        int nh;
        double tile, unit;
    } kind[3] = {{64, 3.05, 4.2}, {32, 2.4, 3.0}, {16, 2.35, 2.4}};
    PagedAttnPlan best{64, 1};
    double least = 1e30;
    for (const auto& k : kind) {
        const long long base = (long long)rows * ((heads + k.nh - 1) / k.nh);
        for (int waves = 0; waves <= 4; ++waves) {  // 0: no split
            int s = 1, share = tiles;
            long long w = (base + sms - 1) / sms;
            if (waves > 0) {
                const long long fit = waves * (long long)sms / base;
                if (fit < 2 || tiles < 2) continue;
                s = fit < tiles ? (int)fit : tiles;
                share = (tiles + s - 1) / s;
                s = (tiles + share - 1) / share;
                if (s < 2) continue;
                w = (base * s + sms - 1) / sms;
            }
            const double merge = s > 1 ? 3.0 + w + (double)rows * heads * s * (2 * PA_DV * sizeof(float)) / 8e6 : 0.0;
            const double cost = w * (share * k.tile + k.unit) + merge;
            if (cost < least) {
                least = cost;
                best = PagedAttnPlan{k.nh, s};
            }
        }
    }
    return best;
}

size_t paged_attn_workspace_bytes(int rows, int heads, int splits) {
    if (splits <= 1) return 0;
    const size_t parts = (size_t)rows * splits * heads;
    return up256(parts * PA_DV * 4) + 2 * up256(parts * 4);
}

li_status launch_paged_attn(const CUtensorMap& qmap, const CUtensorMap& kmap, PagedAttnArgs a, int heads_per_unit,
                            bool fp4, void* workspace, cudaStream_t st) {
    a.by_page = divisor_of(a.page_size);
    if (a.splits > 1) {
        const size_t parts = (size_t)a.rows * a.splits * a.heads;
        uint8_t* w = static_cast<uint8_t*>(workspace);
        a.opart = reinterpret_cast<float*>(w);
        a.mpart = reinterpret_cast<float*>(w + up256(parts * PA_DV * 4));
        a.lpart = reinterpret_cast<float*>(w + up256(parts * PA_DV * 4) + up256(parts * 4));
    }
    li_status s;
    if (fp4)
        s = heads_per_unit == 64   ? launch_units<true, 64>(qmap, kmap, a, st)
            : heads_per_unit == 32 ? launch_units<true, 32>(qmap, kmap, a, st)
                                   : launch_units<true, 16>(qmap, kmap, a, st);
    else
        s = heads_per_unit == 64   ? launch_units<false, 64>(qmap, kmap, a, st)
            : heads_per_unit == 32 ? launch_units<false, 32>(qmap, kmap, a, st)
                                   : launch_units<false, 16>(qmap, kmap, a, st);
    if (s != LI_OK) return s;
    if (a.splits > 1) {
        const size_t smem = a.splits * sizeof(float);
        const dim3 block(PA_MERGE);
        const cudaError_t e =
            a.splits > 8 ? launch_pdl(paged_attn_merge_kernel<4>, dim3(a.heads, 4, a.rows), block, smem, st, 1, a)
                         : launch_pdl(paged_attn_merge_kernel<1>, dim3(a.heads, 1, a.rows), block, smem, st, 1, a);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return LI_ERR_CUDA;
        }
    }
    return host_check_launch();
}

}  // namespace li
