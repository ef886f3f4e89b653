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
// blocks pass through it for every tile). x passes through a ring of five. Streaming
// both operands for every tile would take 124 bytes per cycle and SM from L2 at the
// tensor rate, twice what it delivers; x alone takes 62.
// The accumulator is doubled in tensor memory, so that one tile's results leave (shared
// memory, then TMA, which clips rows past T and columns past N) while the next one's
// products run. W is read as it is stored, K or N contiguous: the descriptor, not a
// copy, transposes it. Chunks past K, rows past T and columns past N arrive as zeros.
// 256 tokens of 64 heads, 128 -> 512: 6.6 us, of which the first loads (2 us) and the last
// stores overlap nothing: 29 MB are 4.3 us of HBM. 512 tiles are three or four per CTA.
constexpr int kTile = 128;
constexpr int kChunk = kTile * 128;      // 16 KB: 128 rows of 64 values
constexpr int kXSlots = 5;
constexpr int kWSlots = 8;
constexpr int kOffX = kWSlots * kChunk;
constexpr int kOffOut = kOffX + kXSlots * kChunk;
constexpr int kOffMisc = kOffOut + kChunk;
constexpr int kSmem = kOffMisc + 1024;
constexpr int kThreads = 192;            // four result warps, loads, MMA
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct Shared {
    uint64_t x_full[kXSlots], x_empty[kXSlots], w_full[kWSlots], w_empty[kWSlots], acc_full[2], acc_empty[2], mma_done;
    uint32_t tmem;
    int abort;
};

// A worker's (CTA's or pair's) part of the line, tile by tile. A tile is `rows` tokens of
// `blocks` neighbouring weight blocks.
struct Line {
    int at, end, ttiles;   // tiles of the line; token tiles
    int tt, block;         // the present tile: token tile, first weight block
    bool first, last;      // of the run on one set of weight blocks
    bool keep;             // the blocks stay in shared memory over a run
    int blocks;

    __device__ Line(const ProjArgs &a, int chunks, int worker, int blocks_) : ttiles(a.ttiles), blocks(blocks_) {
        at = a.each * worker + min(worker, a.longer);
        end = at + a.each + (worker < a.longer);
        keep = chunks <= kWSlots;
        const int g = a.by_ttiles.div(at);
        tt = at - g * ttiles;
        block = g * blocks;
        first = true;
        last = !keep || at + 1 == end || tt + 1 == ttiles;
    }
    __device__ bool more() const { return at < end; }
    __device__ void next() {
        ++at;
        first = !keep;
        if (++tt == ttiles) {
            tt = 0;
            first = true;
            block += blocks;
        }
        last = !keep || at + 1 == end || tt + 1 == ttiles;
    }
};

// One warp's 32 rows x 128 features of a tile, from the accumulator at `acc` through the
// warp's 4 KB at `stage`: boxes of 64 features with the 128-byte swizzle. TMA clips rows
// past T and features past N.
template <typename T>
__device__ __forceinline__ void store_tile(const ProjArgs &a, const CUtensorMap *map_out, uint32_t acc, uint32_t stage,
                                           int lane, int t, int block, bool ok) {
    using E = Elem<T>;
    const int h = a.by_ntiles.div(block), n0 = (block - h * a.ntiles) * kTile;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
            tmem_ld32(acc + half * 64 + c * 32, r);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) w[c * 16 + k] = E::pack(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
        }
        if (lane == 0) tma_store_wait_read();   // the last box has left
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u)
            st_shared_v4(stage + lane * 128 + ((u ^ (lane & 7)) << 4), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (ok && t < a.T && n0 + half * 64 < a.N) tma_store_3d(map_out, stage, n0 + half * 64, h, t);
            tma_store_commit();
        }
    }
}

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
            for (Line l(a, chunks, blockIdx.x, 1); l.more() && ok; l.next()) {
                const int h = a.by_ntiles.div(l.block), n0 = (l.block - h * a.ntiles) * kTile;
                for (int c = 0; c < chunks; ++c) {
                    if (l.first) {
                        const int st = wi % kWSlots;
                        if (!wait(smem_u32(&sh.w_empty[st]), ((wi / kWSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                        const uint32_t full = smem_u32(&sh.w_full[st]), dst = sbase + st * kChunk;
                        mbar_arrive_expect_tx(full, kChunk);
                        if (KN) {
                            // two boxes of 64 features x 64 K rows
                            tma_load_3d(dst, &map_w, full, n0, c * 64, h, pol);
                            tma_load_3d(dst + kChunk / 2, &map_w, full, n0 + 64, c * 64, h, pol);
                        } else {
                            tma_load_3d(dst, &map_w, full, c * 64, n0, h, pol);
                        }
                        ++wi;
                    }
                    const int st = xi % kXSlots;
                    if (!wait(smem_u32(&sh.x_empty[st]), ((xi / kXSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                    const uint32_t full = smem_u32(&sh.x_full[st]);
                    // (a short call loads only its rows: what the rest of the tile holds
                    // reaches only results that are not stored)
                    mbar_arrive_expect_tx(full, a.x_rows * 128);
                    tma_load_3d(sbase + kOffX + st * kChunk, &map_x, full, c * 64, a.shared_x ? 0 : h, l.tt * kTile, pol);
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
            for (Line l(a, chunks, blockIdx.x, 1); l.more() && ok; l.next(), ++n) {
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
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16, stage = sbase + kOffOut + warp * (kChunk / 4);
        uint32_t n = 0;
        bool ok = true;
        for (Line l(a, chunks, blockIdx.x, 1); l.more(); l.next(), ++n) {
            const uint32_t buf = n & 1;
            if (ok) ok = wait(smem_u32(&sh.acc_full[buf]), (n >> 1) & 1, ERR_WAIT_PART_FULL);
            __syncwarp();
            tc_fence_after();
            store_tile<T>(a, &map_out, tmem + buf * kTile + lanes, stage, lane, l.tt * kTile + warp * 32, l.block, ok);
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.acc_empty[buf]));
        }
        if (lane == 0) tma_store_wait();
    }
    __syncthreads();
    if (warp == 5) tmem_dealloc<256>(tmem);
}

// The same over CTA pairs for long inputs: tiles of 256 tokens x 256 features, of which
// each CTA holds half of the tokens' rows, one of the two weight blocks and the results
// of its rows. A CTA's chunk of x then feeds MMAs of twice the width, so that its ring of
// five covers the loads' latency (1,700 cycles) at the tensor rate.
// 4,096 latents of 512 to 64 heads of 256: 50 us, 1.4 PFLOP/s. Of 81,000 cycles the MMA warp
// waits 25,000 for an accumulator whose results are on their way out (a warp's eight boxes
// per tile share one staging buffer), 16,000 for x and 10,000 for weights.
template <typename T, bool KN>
__global__ void __launch_bounds__(kThreads, 1)
    head_proj_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ CUtensorMap map_out, const ProjArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    using E = Elem<T>;

    pdl_trigger();
    if (threadIdx.x == 0) {
        // Full barriers are used at rank 0: its own arrival and both CTAs' bytes. Empty
        // ones are used in each CTA, and a commit arrives at both. acc_empty, at rank 0,
        // takes the result warps of both.
        for (int i = 0; i < kXSlots; ++i) mbar_init(smem_u32(&sh.x_full[i]), 1), mbar_init(smem_u32(&sh.x_empty[i]), 1);
        for (int i = 0; i < kWSlots; ++i) mbar_init(smem_u32(&sh.w_full[i]), 1), mbar_init(smem_u32(&sh.w_empty[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), 8);
        mbar_init(smem_u32(&sh.mma_done), 1);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_out);
    }
    if (warp == 5) pair_tmem_alloc<512>(smem_u32(&sh.tmem));
    tc_fence_before();
    cluster_sync();   // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // all 512 columns of both CTAs
    const Waiter wait{smem_u32(&sh.abort), a.err};
    const int chunks = (a.K + 63) / 64;
    auto line = [&] { return Line(a, chunks, blockIdx.x / 2, 2); };
    pdl_wait();

    if (warp == 4) {
        // -------------------------------------------------------- loads (each CTA its own half)
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            uint32_t xi = 0, wi = 0;   // chunks loaded
            bool ok = true;
            for (Line l = line(); l.more() && ok; l.next()) {
                const int block = l.block + rank, h = a.by_ntiles.div(block), n0 = (block - h * a.ntiles) * kTile;
                for (int c = 0; c < chunks; ++c) {
                    if (l.first) {
                        const int st = wi % kWSlots;
                        if (!wait(smem_u32(&sh.w_empty[st]), ((wi / kWSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                        const uint32_t full = rank0_address(smem_u32(&sh.w_full[st])), dst = sbase + st * kChunk;
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.w_full[st]), 2 * kChunk);
                        if (KN) {
                            pair_load_3d(dst, &map_w, full, n0, c * 64, h, pol);
                            pair_load_3d(dst + kChunk / 2, &map_w, full, n0 + 64, c * 64, h, pol);
                        } else {
                            pair_load_3d(dst, &map_w, full, c * 64, n0, h, pol);
                        }
                        ++wi;
                    }
                    const int st = xi % kXSlots;
                    if (!wait(smem_u32(&sh.x_empty[st]), ((xi / kXSlots) & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.x_full[st]), 2 * kChunk);
                    pair_load_3d(sbase + kOffX + st * kChunk, &map_x, rank0_address(smem_u32(&sh.x_full[st])), c * 64,
                                 a.shared_x ? 0 : h, (2 * l.tt + static_cast<int>(rank)) * kTile, pol);
                    ++xi;
                }
            }
            // the last loads of both must land before either may exit
            if (rank == 0) {
                for (uint32_t i = xi < kXSlots ? 0 : xi - kXSlots; i < xi; ++i)
                    mbar_wait_drain(smem_u32(&sh.x_full[i % kXSlots]), (i / kXSlots) & 1, a.err);
                for (uint32_t i = wi < kWSlots ? 0 : wi - kWSlots; i < wi; ++i)
                    mbar_wait_drain(smem_u32(&sh.w_full[i % kWSlots]), (i / kWSlots) & 1, a.err);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // -------------------------------------------------------- MMA issue (rank 0, for both)
        if (rank == 0 && elect_one()) {
            const IssueWaiter wait{smem_u32(&sh.abort), a.err};
            constexpr uint32_t id = idesc16(E::kFmt, 2 * kTile, 2 * kTile, false, KN);
            const uint64_t dx = sdesc_sw128(sbase + kOffX);
            const uint64_t dw = KN ? sdesc_mn_sw128(sbase, kChunk / 2) : sdesc_sw128(sbase);
            uint32_t xi = 0, w0 = 0, n = 0;   // x chunks used; the blocks' first chunk; tiles
            bool ok = true;
            for (Line l = line(); l.more() && ok; l.next(), ++n) {
                const uint32_t buf = n & 1;
                if (!wait(smem_u32(&sh.acc_empty[buf]), ((n >> 1) & 1) ^ 1, ERR_WAIT_PART_EMPTY)) break;
                tc_fence_after();
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
                        pair_mma_16_ss(tmem + buf * 2 * kTile, xd + (k * 32 >> 4), wd + (KN ? k * 2048 >> 4 : k * 32 >> 4), id,
                                       k > 0 ? 1 : acc0);
                    pair_commit(smem_u32(&sh.x_empty[xs]));
                    if (l.last) pair_commit(smem_u32(&sh.w_empty[ws]));
                }
                if (!ok) break;
                pair_commit(smem_u32(&sh.acc_full[buf]));
                if (l.last) w0 += chunks;
            }
            pair_commit(smem_u32(&sh.mma_done));
            mbar_wait_drain(smem_u32(&sh.mma_done), 0, a.err);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- results (each CTA its rows)
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16, stage = sbase + kOffOut + warp * (kChunk / 4);
        uint32_t n = 0;
        bool ok = true;
        for (Line l = line(); l.more(); l.next(), ++n) {
            const uint32_t buf = n & 1;
            if (ok) ok = wait(smem_u32(&sh.acc_full[buf]), (n >> 1) & 1, ERR_WAIT_PART_FULL);
            __syncwarp();
            tc_fence_after();
            const int t = (2 * l.tt + static_cast<int>(rank)) * kTile + warp * 32;
            for (int b = 0; b < 2; ++b)
                store_tile<T>(a, &map_out, tmem + (2 * buf + b) * kTile + lanes, stage, lane, t, l.block + b, ok);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = rank0_address(smem_u32(&sh.acc_empty[buf]));
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
            }
        }
        if (lane == 0) tma_store_wait();
    }
    __syncwarp();
    cluster_sync();   // neither CTA leaves while the other may reach its memory
    if (warp == 5) pair_tmem_dealloc<512>(sh.tmem);
}

template <typename T, bool KN>
cudaError_t launch_t(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &out, ProjArgs a, int num_sms,
                     cudaStream_t stream) {
    a.ntiles = (a.N + kTile - 1) / kTile;
    const bool pairs = proj_uses_pairs(a.T, a.H, a.K, a.N, a.shared_x);
    auto kernel = pairs ? head_proj_pair_kernel<T, KN> : head_proj_kernel<T, KN>;
    static std::atomic<uint64_t> done[2];
    cudaError_t e = allow_smem(kernel, kSmem, done[pairs]);
    if (e != cudaSuccess) return e;
    const int per = pairs ? 2 : 1, workers = num_sms / per;
    a.ttiles = (a.T + per * kTile - 1) / (per * kTile);
    const int64_t total = static_cast<int64_t>(a.ttiles) * (a.H * a.ntiles / per);
    const int parts = total < workers ? static_cast<int>(total) : workers;
    a.each = static_cast<int>(total / parts), a.longer = static_cast<int>(total % parts);
    a.by_ntiles = Divisor(a.ntiles), a.by_ttiles = Divisor(a.ttiles);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(per * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = per;
    return cudaLaunchKernelEx(&cfg, kernel, x, w, out, a);
}

}  // namespace

// Pairs take two weight blocks that read the same x: an even number of a head's, or of all
// when the heads share x. They win where the tensor rate bounds the call (from 350 flops
// per byte; the GPU's own ratio is 270): 4096 tokens of 512 -> 64 x 256, shared, 66 -> 51
// us. Where memory bounds it they lose to the 128-token tiles, which spread over twice as
// many workers: 4096 tokens of 64 heads, 128 -> 512, 95 against 83 us.
bool proj_uses_pairs(int T, int H, int K, int N, bool shared_x) {
    const double t = T, h = H, k = K, n = N;
    const double bytes = 2.0 * (t * k * (shared_x ? 1.0 : h) + h * k * n + t * h * n);
    const int ntiles = (N + kTile - 1) / kTile;
    return (shared_x ? H * ntiles : ntiles) % 2 == 0 && 2.0 * t * h * k * n > 350.0 * bytes;
}

cudaError_t launch_proj(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &out, const ProjArgs &a, bool bf16,
                        bool w_kn, int num_sms, cudaStream_t stream) {
    if (bf16)
        return w_kn ? launch_t<__nv_bfloat16, true>(x, w, out, a, num_sms, stream)
                    : launch_t<__nv_bfloat16, false>(x, w, out, a, num_sms, stream);
    return w_kn ? launch_t<__half, true>(x, w, out, a, num_sms, stream)
                : launch_t<__half, false>(x, w, out, a, num_sms, stream);
}

}  // namespace moe
