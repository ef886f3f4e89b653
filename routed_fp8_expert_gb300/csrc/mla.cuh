// Building blocks shared by the latent-attention kernels: the two 16-bit element
// types, tcgen05 forms beyond those of ptx.cuh, and the launchers' argument blocks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace moe {

// The latent-attention shapes the tensor-core kernels are built for: a latent of 512
// columns and a shared rotary key of 64 per token; heads of 128 + 64 (query, key) and
// 128 (value) columns in the expanded form.
constexpr int kMlaLatent = 512;
constexpr int kMlaRope = 64;
constexpr int kMlaWidth = kMlaLatent + kMlaRope;
constexpr int kMlaNope = 128;
constexpr int kMlaV = 128;

// kLift: the softmax weights are 2^(score - reference), the reference kLift below the running
// maximum. fp16 weights start at 2^7: below 2^-14 their rounding is absolute and below 2^-25
// nothing is left, which many far keys beside one that dominates would notice (131,072 keys
// of 2^-25 of the largest weight are 0.4% of the sum; 2^-7 of that step is below the rounding
// of the result). With the lag of 2^8 a weight reaches 2^15 of the 65,504 that fit.
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr uint32_t kFmt = 1;   // kind::f16 operand format
    static constexpr float kLift = 0.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
    static constexpr uint32_t kFmt = 0;
    static constexpr float kLift = 7.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

// Instruction descriptor of kind::f16 with fp32 accumulation; a_mn / b_mn: the operand
// is stored with its M (N) dimension contiguous instead of K.
__host__ __device__ constexpr uint32_t idesc16(uint32_t fmt, int M, int N, bool a_mn = false, bool b_mn = false) {
    return idesc_make(fmt, fmt, M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

// Descriptor of an operand whose M (N) dimension is contiguous, stored as tiles of 64
// columns: each K row is 128 bytes of one tile (128-byte swizzle, 8-row groups 1024
// bytes apart) and consecutive tiles lie `tile_bytes` apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t tile_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((tile_bytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// D[tmem] (+)= A[smem] B[smem] and D[tmem] (+)= A[tmem] B[smem], kind::f16.
__device__ __forceinline__ void mma_16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    mma_bf16(d_tmem, a, b, idesc, accumulate);   // the element type is in the descriptor
}
__device__ __forceinline__ void mma_16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

#define MLA_R8(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), "=r"(r[b + 5]), "=r"(r[b + 6]), "=r"(r[b + 7])
#define MLA_W8(b) "r"(r[b]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), "r"(r[b + 5]), "r"(r[b + 6]), "r"(r[b + 7])
#define MLA_LIST32                                                                                                   \
    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29," \
    "%30,%31}"
#define MLA_LIST32_1                                                                                               \
    "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29," \
    "%30,%31,%32}"

// 32 lanes x 32 consecutive columns: thread i gets lane (base + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " MLA_LIST32 ", [%32];"
                 : MLA_R8(0), MLA_R8(8), MLA_R8(16), MLA_R8(24)
                 : "r"(taddr));
}

// 16 lanes x 32 columns in the 16x256b shape: thread t gets, for every 8-column group g,
// columns 8g + 2(t % 4) + {0, 1} of lane t / 4 (r[4g], r[4g + 1]) and of lane t / 4 + 8
// (r[4g + 2], r[4g + 3]).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : MLA_R8(0), MLA_R8(8)
        : "r"(taddr));
}

// Four 8x8 matrices of 16-bit values, stored transposed: lane 8i + j names the row that
// receives column j of matrix i.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t src) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
    return v;
}

// The store counterpart of tmem_ld32.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], " MLA_LIST32_1 ";" ::"r"(taddr), MLA_W8(0), MLA_W8(8),
                 MLA_W8(16), MLA_W8(24)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Order this thread's generic-proxy shared-memory writes before later async-proxy
// accesses (MMA operand reads, TMA) that are synchronised after it.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// True for every thread of the named barrier when `p` holds for any of them.
__device__ __forceinline__ bool named_bar_or(int id, int nthreads, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p)), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// CTA pairs (clusters of two): this CTA's rank; a barrier over both CTAs' threads; tensor
// memory of both at once; MMAs over both, issued by rank 0, with one half of the rows of
// A, of B and of D in each CTA at the same shared-memory and tensor-memory addresses;
// a commit that arrives at the same barrier of both; and a load into this CTA's shared
// memory that counts on rank 0's barrier.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int NCOLS> __device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "n"(NCOLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <int NCOLS> __device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(NCOLS) : "memory");
}
__device__ __forceinline__ void pair_mma_16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ uint32_t rank0_address(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t rank0_bar, int x, int y, int z,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(rank0_bar), "l"(policy)
        : "memory");
}

// Store a box of shared memory through a 3D tensor map (rows and columns past the
// tensor's end are not written), and the issuing thread's waits: until its stores have
// read shared memory, and until they are done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Two fp32 values in one 64-bit register pair: the packed fp32 instructions take one
// issue slot for both.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// sum += x with what rounding loses kept in `lost` and added to the next x (Kahan, 1965). A
// softmax's sum takes a tile's weights at a time: beside one weight of 1, 131,072 keys of 2^-24
// each would otherwise be rounded at half their size (lse off by 3e-4).
__device__ __forceinline__ void add_compensated(float &sum, float &lost, float x) {
    const float y = x + lost, t = sum + y;
    lost = y - (t - sum);
    sum = t;
}

// Move registers between the launch's warpgroups (all 128 threads of one execute it).
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void st_shared_v4(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void st_shared_u32(uint32_t dst, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}

// One lane of the (converged) warp. The compiler knows that a single lane runs what is
// guarded by it: an MMA then issues in 27 cycles instead of the 48 it takes behind
// `lane == 0` (64 x 64 x 16, measured), which decides whether small MMAs reach the
// tensor rate.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Whether the phase with the given parity has completed, without suspending.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait of a whole role: false once any role of the CTA has given up.
struct Waiter {
    uint32_t abort_addr;
    unsigned int *err;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, uint32_t bit) const {
        return mbar_wait(bar, parity, abort_addr, err, bit);
    }
};

// The same for issuing loops: the path that has to wait stays out of line, so that many
// waits leave the loop small enough for the instruction cache.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort_addr, unsigned int *err,
                                              uint32_t bit) {
    return mbar_wait(bar, parity, abort_addr, err, bit);
}
struct IssueWaiter {
    uint32_t abort_addr;
    unsigned int *err;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, uint32_t bit) const {
        return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_addr, err, bit);
    }
};

// ---------------------------------------------------------------- argument blocks

// Division of 0 <= x < 2^31 by a divisor known on the host, in three instructions instead of
// twenty (Granlund and Montgomery, 1994): with 2^s >= d, m = floor(2^32 (2^s - d) / d) + 1,
// x / d = (hi(x m) + x) >> s.
struct Divisor {
    uint32_t mul, shift;
    Divisor() = default;
    explicit Divisor(uint32_t d) : shift(0) {
        while ((uint64_t{1} << shift) < d) ++shift;
        mul = static_cast<uint32_t>((((uint64_t{1} << shift) - d) << 32) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int x) const {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(x), mul) + static_cast<uint32_t>(x)) >> shift);
    }
#endif
};

struct RopeArgs {
    const void *q;            // [T, H, dim], strides below (elements)
    int64_t q_st, q_sh;
    void *q_out;
    int64_t qo_st, qo_sh;
    const void *kv;           // [T, latent + dim]
    int64_t kv_st;
    const void *gamma;        // [latent] or NULL
    void *kv_out;             // or NULL
    int64_t kvo_st;
    void *cache;              // or NULL
    int64_t page_st, row_st;
    int64_t num_pages;
    int page_size;
    Divisor by_page;          // (launch_t)
    const int32_t *slots;
    const int32_t *positions;
    const uint64_t *freq;
    int T, H, dim, latent, layout;
    float amplitude, eps;
    unsigned int *err;
};

struct PagedArgs {
    int64_t Tq;
    const int32_t *table;     // [B, table_st]
    int64_t table_st;
    const int32_t *ctx;       // [B]
    const int32_t *cu_q;      // [B + 1] or NULL (one row each)
    void *out;
    int64_t o_st, o_sh;
    float *lse;               // [Tq, H] or NULL
    int64_t num_pages;
    int max_pages, page_size, box_rows;
    int q_box;                // heads of one query load
    int B, H;
    Divisor by_H, by_page;    // (launch_paged)
    float scale_log2;         // scale * log2(e)
    int few_joins;            // joins whose rows are few (launch_paged)
    float *part_o;            // [2 * grid][64][512]
    float2 *part_ml;          // [2 * grid][64]
    int4 *joins;              // [grid]
    unsigned int *err;
};

struct RaggedArgs {
    const int32_t *cu_q, *cu_k;
    int64_t Tq, Tk;
    void *out;
    int64_t o_st, o_sh;
    float *lse;
    int B, H, max_q, causal;
    float scale_log2;
    unsigned int *err;
};

struct ProjArgs {
    int T, H, K, N;
    int shared_x;             // x has one head that every output head reads
    int x_rows;               // rows of one load of x
    // (launch_t) weight blocks of a head, token tiles, and a worker's tiles: each, one more
    // for the first `longer`
    int ntiles, ttiles, each, longer;
    Divisor by_ntiles, by_ttiles;
    unsigned int *err;
};

cudaError_t launch_rope(const RopeArgs &a, bool bf16, cudaStream_t stream);
// Tensor maps of mla_attn_paged: the queries; the cache in loads of two column groups
// and of one.
struct PagedMaps {
    CUtensorMap q, pair, group;
};

cudaError_t launch_paged(const PagedMaps &m, const PagedArgs &a, bool bf16, int grid, cudaStream_t stream);
cudaError_t launch_ragged(const CUtensorMap &q, const CUtensorMap &k_nope, const CUtensorMap &k_pe,
                          const CUtensorMap &v, const RaggedArgs &a, bool bf16, cudaStream_t stream);
bool proj_uses_pairs(int T, int H, int K, int N, bool shared_x);
cudaError_t launch_proj(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &out, const ProjArgs &a, bool bf16,
                        bool w_kn, int num_sms, cudaStream_t stream);

}  // namespace moe
