// Per-head projections of the latent attention (mla_head_proj).
#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

// out[t, h] = x[t, h] W_h in 128 x 128 output tiles (tokens x features of one head), K in
// chunks of 64. The tiles form one line, token tiles fastest, cut evenly over the CTAs:
// a CTA meets runs of token tiles of one weight block [128 features, K] and loads the
// block once per run (K up to 512 stays in its ring of eight 16 KB chunks; longer
// blocks pass through it for every tile). x passes through a ring of four. Streaming
// both operands for every tile would take 124 bytes per cycle and SM from L2 at the
// tensor rate, twice what it delivers; x alone takes 62.
// The accumulator is doubled in tensor memory, so that one tile's results leave (shared
// memory, then TMA, which clips rows past T and columns past N) while the next one's
// products run. W is read as it is stored, K or N contiguous: the descriptor, not a
// copy, transposes it. Chunks past K, rows past T and columns past N arrive as zeros.
constexpr int kTile = 128;
constexpr int kChunk = kTile * 128;      // 16 KB: 128 rows of 64 values
constexpr int kXSlots = 4;
constexpr int kWSlots = 8;
constexpr int kOffX = kWSlots * kChunk;
constexpr int kOffOut = kOffX + kXSlots * kChunk;
constexpr int kOffMisc = kOffOut + 2 * kChunk;
constexpr int kSmem = kOffMisc + 1024;
constexpr int kThreads = 192;            // four result warps, loads, MMA
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct Shared {
    uint64_t x_full[kXSlots], x_empty[kXSlots], w_full[kWSlots], w_empty[kWSlots], acc_full[2], acc_empty[2], mma_done;
    uint32_t tmem;
    int abort;
};

// A CTA's part of the line, tile by tile.
struct Line {
    int at, end, ntiles, ttiles;   // output tiles; feature tiles of a head; token tiles
    int tt, n0, h;
    bool first, last;              // of the run on one weight block
    bool keep;                     // the block stays in shared memory over a run

    __device__ Line(const ProjArgs &a, int chunks) {
        ntiles = (a.N + kTile - 1) / kTile;
        ttiles = (a.T + kTile - 1) / kTile;
        const int64_t total = static_cast<int64_t>(ttiles) * a.H * ntiles;
        at = static_cast<int>(total * blockIdx.x / gridDim.x);
        end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
        keep = chunks <= kWSlots;
        const int block = at / ttiles;
        tt = at - block * ttiles;
        h = block / ntiles;
        n0 = (block - h * ntiles) * kTile;
        first = true;
        last = !keep || at + 1 == end || tt + 1 == ttiles;
    }
    __device__ bool more() const { return at < end; }
    __device__ void next(const ProjArgs &a) {
        ++at;
        first = !keep;
        if (++tt == ttiles) {
            tt = 0;
            first = true;
            if ((n0 += kTile) >= a.N) n0 = 0, ++h;
        }
        last = !keep || at + 1 == end || tt + 1 == ttiles;
    }
};

template <typename T, bool KN>
__global__ void __launch_bounds__(kThreads, 1)
    head_proj_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_out, const ProjArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using E = Elem<T>;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kXSlots; ++i) mbar_init(smem_u32(&sh.x_full[i]), 1), mbar_init(smem_u32(&sh.x_empty[i]), 1);
        for (int i = 0; i < kWSlots; ++i) mbar_init(smem_u32(&sh.w_full[i]), 1), mbar_init(smem_u32(&sh.w_empty[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), 128);
        mbar_init(smem_u32(&sh.mma_done), 1);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_out);
    }
    if (warp == 5) tmem_alloc<256>(smem_u32(&sh.tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const Waiter wait{smem_u32(&sh.abort), a.err};
    const int chunks = (a.K + 63) / 64;
    pdl_wait();

    if (warp == 4) {
        // -------------------------------------------------------- loads
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            uint32_t xi = 0, wi = 0;   // chunks loaded
            bool ok = true;
            for (Line l(a, chunks); l.more() && ok; l.next(a)) {
                for (int c = 0; c < chunks; ++c) {
                    if (l.first) {
                        const int st = wi % kWSlots;
                        if (!wait(smem_u32(&sh.w_empty[st]), ((wi / kWSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                        const uint32_t full = smem_u32(&sh.w_full[st]), dst = sbase + st * kChunk;
                        mbar_arrive_expect_tx(full, kChunk);
                        if (KN) {
                            // two boxes of 64 features x 64 K rows
                            tma_load_3d(dst, &map_w, full, l.n0, c * 64, l.h, pol);
                            tma_load_3d(dst + kChunk / 2, &map_w, full, l.n0 + 64, c * 64, l.h, pol);
                        } else {
                            tma_load_3d(dst, &map_w, full, c * 64, l.n0, l.h, pol);
                        }
                        ++wi;
                    }
                    const int st = xi % kXSlots;
                    if (!wait(smem_u32(&sh.x_empty[st]), ((xi / kXSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                    const uint32_t full = smem_u32(&sh.x_full[st]);
                    mbar_arrive_expect_tx(full, kChunk);
                    tma_load_3d(sbase + kOffX + st * kChunk, &map_x, full, c * 64, a.shared_x ? 0 : l.h, l.tt * kTile, pol);
                    ++xi;
                }
            }
            // the last loads must land before the CTA may exit
            for (uint32_t i = xi < kXSlots ? 0 : xi - kXSlots; i < xi; ++i)
                mbar_wait_drain(smem_u32(&sh.x_full[i % kXSlots]), (i / kXSlots) & 1, a.err);
            for (uint32_t i = wi < kWSlots ? 0 : wi - kWSlots; i < wi; ++i)
                mbar_wait_drain(smem_u32(&sh.w_full[i % kWSlots]), (i / kWSlots) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 5) {
        // -------------------------------------------------------- MMA issue
        if (elect_one()) {
            const IssueWaiter wait{smem_u32(&sh.abort), a.err};
            constexpr uint32_t id = idesc16(E::kFmt, kTile, kTile, false, KN);
            const uint64_t dx = sdesc_sw128(sbase + kOffX);
            const uint64_t dw = KN ? sdesc_mn_sw128(sbase, kChunk / 2) : sdesc_sw128(sbase);
            uint32_t xi = 0, w0 = 0, n = 0;   // x chunks used; the block's first chunk; tiles
            bool ok = true;
            for (Line l(a, chunks); l.more() && ok; l.next(a), ++n) {
                const uint32_t buf = n & 1;
                if (!wait(smem_u32(&sh.acc_empty[buf]), ((n >> 1) & 1) ^ 1, ERR_WAIT_PART_EMPTY)) break;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c, ++xi) {
                    const uint32_t wi = w0 + c, ws = wi % kWSlots, xs = xi % kXSlots;
                    if (l.first && !wait(smem_u32(&sh.w_full[ws]), (wi / kWSlots) & 1, ERR_WAIT_TMA_FULL)) { ok = false; break; }
                    if (!wait(smem_u32(&sh.x_full[xs]), (xi / kXSlots) & 1, ERR_WAIT_TMA_FULL)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t xd = dx + (xs * kChunk >> 4), wd = dw + (ws * kChunk >> 4);
                    const uint32_t acc0 = c > 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_16_ss(tmem + buf * kTile, xd + (k * 32 >> 4), wd + (KN ? k * 2048 >> 4 : k * 32 >> 4), id, k > 0 ? 1 : acc0);
                    mma_commit(smem_u32(&sh.x_empty[xs]));
                    if (l.last) mma_commit(smem_u32(&sh.w_empty[ws]));
                }
                if (!ok) break;
                mma_commit(smem_u32(&sh.acc_full[buf]));
                if (l.last) w0 += chunks;
            }
            mma_commit(smem_u32(&sh.mma_done));
            mbar_wait_drain(smem_u32(&sh.mma_done), 0, a.err);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- results
        // A warp's 32 rows x 128 features: two boxes of 64 features with the 128-byte
        // swizzle, in its own 8 KB.
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16, stage = sbase + kOffOut + warp * (kChunk / 2);
        uint32_t n = 0;
        bool ok = true;
        for (Line l(a, chunks); l.more(); l.next(a), ++n) {
            const uint32_t buf = n & 1;
            if (ok) ok = wait(smem_u32(&sh.acc_full[buf]), (n >> 1) & 1, ERR_WAIT_PART_FULL);
            __syncwarp();
            tc_fence_after();
            if (lane == 0) tma_store_wait_read();   // the last tile's boxes have left
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kTile; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + buf * kTile + lanes + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = E::pack(__uint_as_float(r[k + 2 * q]), __uint_as_float(r[k + 2 * q + 1]));
                    const int u = ((c & 32) + k) / 8;
                    st_shared_v4(stage + (c / 64) * 4096 + lane * 128 + ((u ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.acc_empty[buf]));
            fence_async_smem();
            __syncwarp();
            const int t = l.tt * kTile + warp * 32;
            if (lane == 0 && ok && t < a.T) {
                tma_store_3d(&map_out, stage, l.n0, l.h, t);
                if (l.n0 + 64 < a.N) tma_store_3d(&map_out, stage + 4096, l.n0 + 64, l.h, t);
            }
            if (lane == 0) tma_store_commit();
        }
        if (lane == 0) tma_store_wait();
    }
    __syncthreads();
    if (warp == 5) tmem_dealloc<256>(tmem);
}

template <typename T, bool KN>
cudaError_t launch_t(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &out, const ProjArgs &a, int num_sms,
                     cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(head_proj_kernel<T, KN>, kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t total = static_cast<int64_t>((a.T + kTile - 1) / kTile) * a.H * ((a.N + kTile - 1) / kTile);
    const int grid = total < num_sms ? static_cast<int>(total) : num_sms;
    return launch_pdl(head_proj_kernel<T, KN>, dim3(grid), dim3(kThreads), kSmem, stream, x, w, out, a);
}

}  // namespace

cudaError_t launch_proj(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &out, const ProjArgs &a, bool bf16,
                        bool w_kn, int num_sms, cudaStream_t stream) {
    if (bf16)
        return w_kn ? launch_t<__nv_bfloat16, true>(x, w, out, a, num_sms, stream)
                    : launch_t<__nv_bfloat16, false>(x, w, out, a, num_sms, stream);
    return w_kn ? launch_t<__half, true>(x, w, out, a, num_sms, stream)
                : launch_t<__half, false>(x, w, out, a, num_sms, stream);
}

}  // namespace moe
