// Attention over a paged latent cache, for a token's selected positions or for
// a sliding window with first positions that stay visible (sinks):
//
//   o[t,h,:] = sum_s p_s c[s, :512],   p = softmax over the visible s of scale * (q[t,h,:] . c[s,:])
//
// in the absorbed-MLA form (a cache row is 512 latent + 64 rotary elements,
// shared by every head).  A row is held in 4 bits (LI_KV4_ROW_BYTES: 512 e2m1
// codes, one e4m3 scale per 16 of them, 64 bf16) or as 576 bf16.  e2m1 x e4m3
// has 6 significant bits, so a 4-bit row is expanded to bf16 exactly and the
// two formats share everything behind the producer warps.
//
// One CTA (one per SM, persistent) takes units of one token, 64 heads and a
// share of the token's visible positions, 128 positions (a tile) at a time:
//   - warps 0-7 (producers) hold each tile's rows once in shared memory, as bf16
//     in nine 16 KB chunks of 64 elements x 128 positions (128-byte swizzle).
//     A row belongs to two threads.  4 bits: a thread loads its half of the row
//     into registers one whole tile ahead and expands it chunk by chunk; bf16:
//     16-byte cp.async straight into the chunks.
//   - warp 16 issues S^T = K Q^T (M = 128 positions, N = 64 heads, K = 576) and
//     O^T += V^T P^T (M = 128 latent elements, four blocks, N = 64, K = 128),
//     both from the same chunks: K is read K-major, V^T MN-major, so nothing is
//     loaded or transposed a second time.  P takes the rotary chunk's place,
//     which V does not need and whose scores are done by then.
//   - warps 8-15 (softmax): one position per TMEM lane, 32 heads per group of four
//     warps.  The running maximum of a head is raised only when a tile exceeds
//     it by more than 2^8 (p stays below 2^8, which bf16 and the fp32 sums hold
//     as exactly as p <= 1), so O is rescaled in TMEM almost never after the
//     first tile.  Sums are kept in fp32; p is rounded to bf16 for the product
//     (2^-9 each, the same step as the bf16 output).
// A chunk is released as soon as its value product is done, so the next tile's
// expansion runs under this tile's value product.
// With few units the visible tiles are split over several CTAs; a second kernel
// merges the parts (see attn_splits for the rule).
#include <cuda_fp16.h>

#include "li_common.cuh"
#include "li_kernels.cuh"

namespace li {

namespace {

constexpr int PA_D = 576;
constexpr int PA_DV = 512;
constexpr int PA_NH = 64;                  // heads per unit (MMA N)
constexpr int PA_M = 128;                  // positions per tile
constexpr int PA_CH = PA_D / 64;           // 9 chunks of 64 elements
constexpr int PA_VCH = PA_DV / 64;         // 8 of them hold the value
constexpr int PA_CHUNK = PA_M * 128;       // 16 KB
constexpr int PA_QCHUNK = PA_NH * 128;     // 8 KB
constexpr int PA_PRODUCERS = 256;
constexpr int PA_SOFTMAX = 256;
constexpr int PA_THREADS = PA_PRODUCERS + PA_SOFTMAX + 32;
constexpr int PA_TMEM_COLS = 512;          // S^T: 64 columns, O^T: 4 x 64
constexpr int PA_O_COL = 64;
constexpr int PA_DEPTH = 4;                // bf16: chunks in flight per producer thread
constexpr float PA_RAISE = 8.f;            // log2: a head's maximum is raised when exceeded by more

constexpr int PO_Q = 0;
constexpr int PO_K = PO_Q + PA_CH * PA_QCHUNK;
constexpr int PO_RED = PO_K + PA_CH * PA_CHUNK;        // [2 groups][4 warps][32] fp32
constexpr int PO_M = PO_RED + 2 * 4 * 32 * 4;          // [8 warps][32] fp32: maxima in use, later factors
constexpr int PO_VALID = PO_M + 8 * 32 * 4;            // [2][128] bytes
constexpr int PO_BAR = PO_VALID + 2 * PA_M;            // full[9], empty[9], qfull, sdone, pready, odone, oempty
constexpr int PA_NBAR = 2 * PA_CH + 5;
constexpr int PO_TMEM = PO_BAR + PA_NBAR * 8;
constexpr int PA_SMEM = PO_TMEM + 16 + 1024;           // + slack to align the base to 1024
static_assert(PA_SMEM <= 232448, "shared memory per CTA");

__device__ __forceinline__ void pa_cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ float pa_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MN-major operand with the 128-byte swizzle: each 128-byte row holds 64
// consecutive M (or N) elements of one K index; atoms of 8 rows follow each other
// along K every `sbo` bytes, blocks of 64 M elements every `lbo` bytes.
__device__ __forceinline__ uint64_t pa_mnmajor_desc(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
    d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
    d |= uint64_t((sbo >> 4) & 0x3FFFu) << 32;
    d |= uint64_t(1u) << 46;
    d |= uint64_t(2u) << 61;
    return d;
}

// Reduce-scatter of 32 values over the warp: lane l ends with v[0] reduced for
// index l (each step keeps the half selected by one lane bit: 31 shuffles).
template <bool MAX>
__device__ __forceinline__ void warp_reduce_scatter32(float (&v)[32], int lane) {
#pragma unroll
    for (int step = 0; step < 5; ++step) {
        const int o = 16 >> step;
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = upper ? v[i] : v[i + o];
            const float keep = upper ? v[i + o] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = MAX ? fmaxf(keep, recv) : keep + recv;
        }
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
    x.hg = u % a.hgroups;
    const int v = u / a.hgroups;
    const int split = v % a.splits;
    x.row = v / a.splits;
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
    const int nt = (x.n + PA_M - 1) / PA_M;
    x.t0 = (int)((long long)nt * split / a.splits);
    x.t1 = (int)((long long)nt * (split + 1) / a.splits);
    return x;
}

// Cache row of entry j of the unit's list, or null (padding, past the end, out of range).
__device__ __forceinline__ const uint8_t* row_of(const PagedAttnArgs& a, const PaUnit& x, int j, uint32_t row_bytes) {
    if (j >= x.n) return nullptr;
    int s;
    if (a.pos) {
        s = j < x.nsink ? j : x.first + j;
    } else {
        s = __ldg(a.sel + (size_t)x.row * a.k + j);
        if (s < 0) return nullptr;
        if ((long long)s >= (long long)a.max_blocks * a.page_size) {
            record_error(a.err, ERRBIT_BOUNDS);
            return nullptr;
        }
    }
    const int block = (int)((unsigned)s / (unsigned)a.page_size);
    const int off = s - block * a.page_size;
    const long long at = (long long)x.req * a.max_blocks + block;
    const long long page = a.table ? (long long)__ldg(a.table + at) : at;
    if (page < 0 || page >= a.num_pages) {
        record_error(a.err, ERRBIT_BOUNDS);
        return nullptr;
    }
    return static_cast<const uint8_t*>(a.cache) + (page * a.page_size + off) * (long long)row_bytes;
}

// The producers' walk over the CTA's tiles.
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

// Eight e2m1 codes (element i in bits 4i..4i+3) times the block's scale, as four
// bf16 pairs.  A code s.ee.m moved to bits 15 and 8..6 of a bf16 is its value
// times 2^-126 (ee = 0 lands on the bf16 subnormals, which the multiply takes), and
// `scale` carries the factor back up, so each product is exact: two instructions
// to place a pair, three to mask and multiply it.
__device__ __forceinline__ void expand8(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
    const uint32_t lo = w << 4;  // the even codes move to the high half of their byte
    const uint32_t sel[4] = {0x4000u, 0x5010u, 0x6020u, 0x7030u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = __byte_perm(lo, w, sel[i]);                   // bits 15..12: even code, 31..28: odd code
        const uint32_t z = (y & 0x80008000u) | ((y >> 6) & 0x01C001C0u);
        __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&z),
                                   *reinterpret_cast<const __nv_bfloat162*>(&scale));
        o[i] = *reinterpret_cast<uint32_t*>(&p);
    }
}

// e4m3 scales (two bytes) to expand8's multipliers: the scale times 2^117 in both
// halves of a bf16 pair (448 x 2^117 is still below bf16's largest value).  The
// missing 2^9 stays on the whole row (the rotary part is multiplied by 2^-9, exact
// down to bf16's subnormals) and is put back in fp32: kUp4.
constexpr float kUp4 = 512.f;
__device__ __forceinline__ void scales2(uint32_t two, uint32_t& s0, uint32_t& s1) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
    const __nv_bfloat162 a = __float2bfloat162_rn(f.x * 0x1p117f), b = __float2bfloat162_rn(f.y * 0x1p117f);
    s0 = *reinterpret_cast<const uint32_t*>(&a);
    s1 = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t down4(uint32_t w) {
    const __nv_bfloat162 k = __float2bfloat162_rn(1.f / kUp4);
    __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), k);
    return *reinterpret_cast<uint32_t*>(&p);
}

template <bool FP4>
__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const PagedAttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* qs = smem + PO_Q;
    uint8_t* ks = smem + PO_K;
    uint8_t* ps = ks + (PA_CH - 1) * PA_CHUNK;  // P over the rotary chunk
    float* red = reinterpret_cast<float*>(smem + PO_RED);
    float* msm = reinterpret_cast<float*>(smem + PO_M);
    uint8_t* vflag = smem + PO_VALID;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + PO_BAR);
    uint64_t* empty = full + PA_CH;
    uint64_t* qfull = empty + PA_CH;
    uint64_t* sdone = qfull + 1;
    uint64_t* pready = sdone + 1;
    uint64_t* odone = pready + 1;
    uint64_t* oempty = odone + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PO_TMEM);

    if (threadIdx.x == 0) {
        for (int i = 0; i < PA_CH; ++i) {
            mbar_init(&full[i], PA_PRODUCERS / 32);
            mbar_init(&empty[i], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(sdone, 1);
        mbar_init(pready, PA_SOFTMAX / 32);
        mbar_init(odone, 1);
        mbar_init(oempty, PA_SOFTMAX / 32);
        fence_mbar_init();
    }
    if (warp == 16) {
        if (lane == 0) tma_prefetch_desc(&qmap);
        tmem_alloc(tmem_slot, PA_TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();  // the query, the selection and the cache may come from the previous kernel of the stream
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < PA_PRODUCERS / 32) {
        // ---------------------------------------------------------------- producers
        const int r = threadIdx.x >> 1, h = threadIdx.x & 1;  // position of the tile, half of each chunk's row
        const uint32_t k_s = smem_u32(ks);
        uint32_t dst[4];  // the thread's four 16-byte units of a chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = k_s + sw128_offset(r, 4 * h + i);
        PaWalk w;
        w.start(a);
        if constexpr (FP4) {
            uint4 code[PA_VCH], sc[2], rot[4];
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint8_t* src = w.more ? row_of(a, w.x, w.t * PA_M + r, LI_KV4_ROW_BYTES) : nullptr;
#pragma unroll
            for (int c = 0; c < PA_VCH; ++c)
                code[c] = src ? __ldg(reinterpret_cast<const uint4*>(src + c * 32 + h * 16)) : z;
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[i] = src ? __ldg(reinterpret_cast<const uint4*>(src + 256 + i * 16)) : z;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rot[i] = src ? __ldg(reinterpret_cast<const uint4*>(src + 288 + h * 64 + i * 16)) : z;
            for (uint32_t n = 0; w.more; ++n) {
                const bool valid = src != nullptr;
                w.next(a);
                src = w.more ? row_of(a, w.x, w.t * PA_M + r, LI_KV4_ROW_BYTES) : nullptr;
                const uint32_t scw[8] = {sc[0].x, sc[0].y, sc[0].z, sc[0].w, sc[1].x, sc[1].y, sc[1].z, sc[1].w};
                const uint32_t free_parity = (n & 1) ^ 1;
                bool ok = true;
#pragma unroll
                for (int c = 0; c < PA_VCH; ++c) {
                    uint32_t s0, s1;
                    scales2((scw[c] >> (16 * h)) & 0xffffu, s0, s1);
                    uint32_t o[4][4];
                    expand8(code[c].x, s0, o[0]);
                    expand8(code[c].y, s0, o[1]);
                    expand8(code[c].z, s1, o[2]);
                    expand8(code[c].w, s1, o[3]);
                    code[c] = src ? __ldg(reinterpret_cast<const uint4*>(src + c * 32 + h * 16)) : z;
                    ok = ok && mbar_wait(&empty[c], free_parity, a.err);
                    if (c == 0 && h == 0) vflag[(n & 1) * PA_M + r] = valid ? 1 : 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_shared16(dst[i] + c * PA_CHUNK, o[i][0], o[i][1], o[i][2], o[i][3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[c]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[i] = src ? __ldg(reinterpret_cast<const uint4*>(src + 256 + i * 16)) : z;
                ok = ok && mbar_wait(&empty[PA_CH - 1], free_parity, a.err);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st_shared16(dst[i] + (PA_CH - 1) * PA_CHUNK, down4(rot[i].x), down4(rot[i].y), down4(rot[i].z),
                                down4(rot[i].w));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[PA_CH - 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rot[i] = src ? __ldg(reinterpret_cast<const uint4*>(src + 288 + h * 64 + i * 16)) : z;
                if (!__all_sync(0xffffffffu, ok)) break;  // a wait ran out: the other roles' waits run out too
            }
        } else {
            const uint8_t* src = w.more ? row_of(a, w.x, w.t * PA_M + r, PA_D * 2) : nullptr;
            for (uint32_t n = 0; w.more; ++n) {
                const uint8_t* at = src ? src + h * 64 : static_cast<const uint8_t*>(a.cache);
                const uint32_t bytes = src ? 16u : 0u;  // 0: the unit is filled with zeros, nothing is read
                const bool valid = src != nullptr;
                const uint32_t free_parity = (n & 1) ^ 1;
                bool ok = true;
#pragma unroll
                for (int c = 0; c < PA_CH; ++c) {
                    ok = ok && mbar_wait(&empty[c], free_parity, a.err);
                    if (c == 0 && h == 0) vflag[(n & 1) * PA_M + r] = valid ? 1 : 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pa_cp_async16(dst[i] + c * PA_CHUNK, at + (src ? c * 128 + i * 16 : 0), bytes);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (c >= PA_DEPTH) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(PA_DEPTH) : "memory");
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[c - PA_DEPTH]);
                    }
                }
                // the next tile waits for this one's products, so its last chunks are handed over first
                w.next(a);
                src = w.more ? row_of(a, w.x, w.t * PA_M + r, PA_D * 2) : nullptr;
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int c = PA_CH - PA_DEPTH; c < PA_CH; ++c) mbar_arrive(&full[c]);
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            }
        }
    } else if (warp == 16) {
        // ---------------------------------------------------------------- query loads and MMA issue
        if (lane == 0) {
            const uint32_t k_s = smem_u32(ks), q_s = smem_u32(qs), p_s = smem_u32(ps);
            constexpr uint32_t IDESC_S = idesc_f32acc(PA_M, PA_NH, kFmtBF16);
            constexpr uint32_t IDESC_O = idesc_f32acc(128, PA_NH, kFmtBF16) | (1u << 15) | (1u << 16);
            const uint64_t keep = l2_policy_evict_last();
            auto load_q = [&](const PaUnit& x) {
                mbar_arrive_expect_tx(qfull, PA_CH * PA_QCHUNK);
                for (int c = 0; c < PA_CH; ++c)
                    pa_tma_load_3d(qs + c * PA_QCHUNK, &qmap, c * 64, x.hg * PA_NH, x.row, qfull, keep);
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
                    for (int c = 0; c < PA_CH; ++c) {
                        if (!mbar_wait(&full[c], par, a.err)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16(tmem_base, sw128_kmajor_desc(k_s + c * PA_CHUNK + kk * 32),
                                     sw128_kmajor_desc(q_s + c * PA_QCHUNK + kk * 32), IDESC_S, (c | kk) != 0);
                    }
                    if (!ok) break;
                    tc_commit(sdone);
                    if (t == 0 && !mbar_wait(oempty, (units & 1) ^ 1, a.err)) { ok = false; break; }
                    if (!mbar_wait(pready, par, a.err)) { ok = false; break; }
                    tc_fence_after();
                    for (int blk = 0; blk < PA_VCH / 2; ++blk) {
#pragma unroll
                        for (int s = 0; s < PA_M / 16; ++s)
                            mma_bf16(tmem_base + (uint32_t)(PA_O_COL + blk * PA_NH),
                                     pa_mnmajor_desc(k_s + 2 * blk * PA_CHUNK + s * 2048, PA_CHUNK, 1024),
                                     pa_mnmajor_desc(p_s + s * 2048, PA_CHUNK, 1024), IDESC_O, (t | s) != 0);
                        tc_commit(&empty[2 * blk]);
                        tc_commit(&empty[2 * blk + 1]);
                    }
                    tc_commit(&empty[PA_CH - 1]);
                    if (t == tiles - 1) tc_commit(odone);
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
        }
    } else {
        // ---------------------------------------------------------------- softmax and output
        const int sw = warp - PA_PRODUCERS / 32;   // 0..7
        const int g = sw >> 2, q4 = warp & 3;      // heads 32g..32g+31; TMEM lane quarter
        const int row = q4 * 32 + lane;            // position of the tile; latent element of an O block
        const uint32_t lane_base = tmem_base + ((uint32_t)(q4 * 32) << 16);
        const float up = FP4 ? kUp4 : 1.f;
        const float c2 = a.scale * up * 1.4426950408889634f;  // exp(x) = exp2(x log2 e)
        float* gred = red + g * 128;
        float* wm = msm + sw * 32;
        const int bar = 1 + g;
        uint32_t n = 0, units = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const PaUnit x = unit_of(a, u, sw == 0 && lane == 0);
            if (!x.live) continue;
            const int split = (u / a.hgroups) % a.splits;
            const int h0 = x.hg * PA_NH + g * 32;
            const int nh = min(32, a.heads - h0);   // heads of this group that exist (may be <= 0)
            const size_t part = ((size_t)x.row * a.splits + split) * a.heads + h0;
            if (x.t0 == x.t1) {  // nothing visible in this share
                if (a.splits > 1) {
                    if (q4 == 0 && lane < nh) {
                        a.mpart[part + lane] = -INFINITY;
                        a.lpart[part + lane] = 0.f;
                    }
                } else {
                    for (int i = q4 * 32 + lane; i < nh * (PA_DV / 2); i += 128)
                        reinterpret_cast<uint32_t*>(a.out + ((size_t)x.row * a.heads + h0) * PA_DV)[i] = 0u;
                }
                continue;
            }
            float m_run = -INFINITY, l_run = 0.f;  // of head h0 + lane; l_run over this warp's positions
            for (int t = x.t0; t < x.t1; ++t, ++n) {
                // full[0] orders the producers' flags before this read; it stays in this phase until the
                // tile's value product has released the chunk
                if (!mbar_wait(&full[0], n & 1, a.err) || !mbar_wait(sdone, n & 1, a.err)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[32];
                tmem_ld32(lane_base + g * 32, s);
                tmem_ld_wait();
                const bool valid = vflag[(n & 1) * PA_M + row] != 0;
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = valid ? __uint_as_float(s[i]) * c2 : -INFINITY;
                warp_reduce_scatter32<true>(v, lane);
                gred[q4 * 32 + lane] = v[0];
                asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
                const float mx = fmaxf(fmaxf(gred[lane], gred[32 + lane]), fmaxf(gred[64 + lane], gred[96 + lane]));
                const bool raise = mx > m_run + PA_RAISE;
                const float m_use = raise ? mx : m_run;
                const float f = raise && m_run != -INFINITY ? pa_ex2(m_run - m_use) : 1.f;
                const bool rescale = __any_sync(0xffffffffu, f != 1.f);  // the same for the group's four warps
                m_run = m_use;
                wm[lane] = m_use == -INFINITY ? 0.f : m_use;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 m4 = *reinterpret_cast<const float4*>(wm + i);
                    v[i] = valid ? pa_ex2(__fmaf_rn(__uint_as_float(s[i]), c2, -m4.x)) : 0.f;
                    v[i + 1] = valid ? pa_ex2(__fmaf_rn(__uint_as_float(s[i + 1]), c2, -m4.y)) : 0.f;
                    v[i + 2] = valid ? pa_ex2(__fmaf_rn(__uint_as_float(s[i + 2]), c2, -m4.z)) : 0.f;
                    v[i + 3] = valid ? pa_ex2(__fmaf_rn(__uint_as_float(s[i + 3]), c2, -m4.w)) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t pk[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        __nv_bfloat162 pp = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                        pk[j] = *reinterpret_cast<uint32_t*>(&pp);
                    }
                    *reinterpret_cast<uint4*>(ps + sw128_offset(row, 4 * g + i)) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                if (rescale) {  // O of the tiles before is complete: its commit came before sdone's
                    __syncwarp();
                    wm[lane] = f;
                    __syncwarp();
#pragma unroll 1
                    for (int blk = 0; blk < PA_DV / 128; ++blk) {
                        const uint32_t at = lane_base + (uint32_t)(PA_O_COL + blk * PA_NH + g * 32);
                        tmem_ld32(at, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * wm[i]);
                        tmem_st32(at, s);
                    }
                    tmem_st_wait();
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready);
                warp_reduce_scatter32<false>(v, lane);
                l_run = l_run * f + v[0];
            }
            if (!ok) break;
            if (!mbar_wait(odone, units & 1, a.err)) { ok = false; break; }
            tc_fence_after();
            ++units;
            gred[q4 * 32 + lane] = l_run;
            asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
            const float l = (gred[lane] + gred[32 + lane]) + (gred[64 + lane] + gred[96 + lane]);
            asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");  // red is written again by the next unit
            const bool whole = a.splits == 1;
            if (!whole && q4 == 0 && lane < nh) {
                a.mpart[part + lane] = m_run;
                a.lpart[part + lane] = l;
            }
            wm[lane] = !whole ? up : l == 0.f ? 0.f : up / l;
            __syncwarp();
#pragma unroll 1
            for (int blk = 0; blk < PA_DV / 128; ++blk) {
                uint32_t s[32];
                tmem_ld32(lane_base + (uint32_t)(PA_O_COL + blk * PA_NH + g * 32), s);
                tmem_ld_wait();
                const int d = blk * 128 + row;
                if (whole) {
                    __nv_bfloat16* o = a.out + ((size_t)x.row * a.heads + h0) * PA_DV + d;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < nh) o[(size_t)i * PA_DV] = __float2bfloat16_rn(__uint_as_float(s[i]) * wm[i]);
                } else {
                    float* o = a.opart + part * PA_DV + d;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < nh) o[(size_t)i * PA_DV] = __uint_as_float(s[i]) * wm[i];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem_base, PA_TMEM_COLS);
    }
}

// Merge of a token's splits: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M the
// largest m_s (maxima are in the log2 domain).  One CTA per (head, token).
__global__ void __launch_bounds__(128) paged_attn_merge_kernel(const PagedAttnArgs a) {
    const int h = blockIdx.x, row = blockIdx.y;
    const int d = threadIdx.x * 4;
    int r, p;
    if (!token_of(a, row, &r, &p, false)) return;
    const size_t at = (size_t)row * a.splits * a.heads + h;
    float M = -INFINITY;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, a.mpart[at + (size_t)s * a.heads]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    if (M != -INFINITY) {
        for (int s = 0; s < a.splits; ++s) {
            const size_t part = at + (size_t)s * a.heads;
            const float m = a.mpart[part];
            if (m == -INFINITY) continue;
            const float f = pa_ex2(m - M);
            L += f * a.lpart[part];
            const float4 o = *reinterpret_cast<const float4*>(a.opart + part * PA_DV + d);
            acc.x += f * o.x;
            acc.y += f * o.y;
            acc.z += f * o.z;
            acc.w += f * o.w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.heads + h) * PA_DV + d) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}

constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// How many CTAs share a token's tiles: the count with the least estimated time, in
// tiles, over the waves of units the GPU runs one after another.  A unit costs its
// tiles and about one more to fill and drain; parts cost a merge.
int paged_attn_splits(int rows, int heads, int positions, int sms) {
    const long long base = (long long)rows * ((heads + PA_NH - 1) / PA_NH);
    const int tiles = (positions + PA_M - 1) / PA_M;
    int best = 1;
    double least = 0;
    for (int s = 1; s <= tiles && s <= 2 * sms; ++s) {
        const long long waves = (base * s + sms - 1) / sms;
        const double cost = (double)waves * ((tiles + s - 1) / s + 1.0) + (s > 1 ? 1.5 + 0.02 * s : 0.0);
        if (s == 1 || cost < least) {
            best = s;
            least = cost;
        }
        if (base * s >= 4LL * sms) break;
    }
    return best;
}

size_t paged_attn_workspace_bytes(int rows, int heads, int splits) {
    if (splits <= 1) return 0;
    const size_t parts = (size_t)rows * splits * heads;
    return up256(parts * PA_DV * 4) + 2 * up256(parts * 4);
}

li_status launch_paged_attn(const CUtensorMap& qmap, PagedAttnArgs a, bool fp4, void* workspace, cudaStream_t st) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_done[dev]) {
        if (cudaFuncSetAttribute(paged_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, PA_SMEM) !=
                cudaSuccess ||
            cudaFuncSetAttribute(paged_attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, PA_SMEM) !=
                cudaSuccess) {
            cudaGetLastError();
            return LI_ERR_CUDA;
        }
        if (dev < 64) attr_done[dev] = true;
    }
    if (a.splits > 1) {
        const size_t parts = (size_t)a.rows * a.splits * a.heads;
        uint8_t* w = static_cast<uint8_t*>(workspace);
        a.opart = reinterpret_cast<float*>(w);
        a.mpart = reinterpret_cast<float*>(w + up256(parts * PA_DV * 4));
        a.lpart = reinterpret_cast<float*>(w + up256(parts * PA_DV * 4) + up256(parts * 4));
    }
    const int grid = a.units < host_num_sms() ? a.units : host_num_sms();
    const cudaError_t e = fp4 ? launch_pdl(paged_attn_kernel<true>, dim3(grid), dim3(PA_THREADS), PA_SMEM, st, 1, qmap, a)
                              : launch_pdl(paged_attn_kernel<false>, dim3(grid), dim3(PA_THREADS), PA_SMEM, st, 1, qmap, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return LI_ERR_CUDA;
    }
    if (a.splits > 1) paged_attn_merge_kernel<<<dim3(a.heads, a.rows), 128, 0, st>>>(a);
    return host_check_launch();
}

}  // namespace li
