// Per-head projections of the latent attention (mla_head_proj).
#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

// out[t, h] = x[t, h] W_h: one 128 x 128 output tile (tokens x features of one head) at
// a time per CTA, K in chunks of 64 through a ring of six (16 KB of x, 16 KB of W), the
// accumulator doubled in tensor memory so that one tile's results are written while the
// next one's products run. W is read as it is stored, K or N contiguous: the
// descriptor, not a copy, transposes it. Chunks past K, rows past T and columns past N
// arrive as zeros.
// A decode step reads 8.4 MB of W for 64 heads; a prompt's absorb and value products
// are bound by x and out, the expansion (K = 512, N = 256) by the tensor rate.
constexpr int kTile = 128;
constexpr int kStages = 6;
constexpr int kABytes = kTile * 128;
constexpr int kBBytes = kTile * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kOffMisc = kStages * kStageBytes;
constexpr int kSmem = kOffMisc + 1024;
constexpr int kThreads = 192;   // four result warps, loads, MMA

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], mma_done;
    uint32_t tmem;
    int abort;
};

// Output tile `i` of the line: column tiles of a head fastest, then the heads, then the
// tokens, so that tiles running together share rows of x (and all of W stays in L2).
struct TileAt {
    int t0, h, n0;
};
__device__ __forceinline__ TileAt tile_at(const ProjArgs &a, int64_t i, int ntiles) {
    TileAt p;
    const int64_t per = static_cast<int64_t>(a.H) * ntiles;
    const int tt = static_cast<int>(i / per);
    const int r = static_cast<int>(i - tt * per);
    p.t0 = tt * kTile;
    p.h = r / ntiles;
    p.n0 = (r - p.h * ntiles) * kTile;
    return p;
}

template <typename T, bool KN>
__global__ void __launch_bounds__(kThreads, 1)
    head_proj_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const ProjArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using E = Elem<T>;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1), mbar_init(smem_u32(&sh.empty[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), 128);
        mbar_init(smem_u32(&sh.mma_done), 1);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
    }
    if (warp == 5) tmem_alloc<256>(smem_u32(&sh.tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const Waiter wait{smem_u32(&sh.abort), a.err};
    const int ntiles = (a.N + kTile - 1) / kTile;
    const int64_t total = static_cast<int64_t>((a.T + kTile - 1) / kTile) * a.H * ntiles;
    const int chunks = (a.K + 63) / 64;
    pdl_wait();

    if (warp == 4) {
        // -------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            uint32_t it = 0, used = 0, parity = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
                const TileAt p = tile_at(a, i, ntiles);
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int st = it % kStages;
                    const uint32_t ph = (it / kStages) & 1;
                    if (!wait(smem_u32(&sh.empty[st]), ph ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                    const uint32_t full = smem_u32(&sh.full[st]), dst = sbase + st * kStageBytes;
                    mbar_arrive_expect_tx(full, kStageBytes);
                    tma_load_3d(dst, &map_x, full, c * 64, a.shared_x ? 0 : p.h, p.t0, pol);
                    if (KN) {
                        // two boxes of 64 features x 64 K rows
                        tma_load_3d(dst + kABytes, &map_w, full, p.n0, c * 64, p.h, pol);
                        tma_load_3d(dst + kABytes + kBBytes / 2, &map_w, full, p.n0 + 64, c * 64, p.h, pol);
                    } else {
                        tma_load_3d(dst + kABytes, &map_w, full, c * 64, p.n0, p.h, pol);
                    }
                    used |= 1u << st;
                    parity = (parity & ~(1u << st)) | (ph << st);
                }
            }
            // the last loads must land before the CTA may exit
            for (int s = 0; s < kStages; ++s)
                if (used >> s & 1) mbar_wait_drain(smem_u32(&sh.full[s]), parity >> s & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 5) {
        // -------------------------------------------------------- MMA issue
        if (elect_one()) {
            constexpr uint32_t id = idesc16(E::kFmt, kTile, kTile, false, KN);
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x, ++n) {
                const uint32_t buf = n & 1;
                if (!wait(smem_u32(&sh.acc_empty[buf]), ((n >> 1) & 1) ^ 1, ERR_WAIT_PART_EMPTY)) break;
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int st = it % kStages;
                    if (!wait(smem_u32(&sh.full[st]), (it / kStages) & 1, ERR_WAIT_TMA_FULL)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t xa = sbase + st * kStageBytes, wb = xa + kABytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_16_ss(tmem + buf * kTile, sdesc_sw128(xa + k * 32),
                                 KN ? sdesc_mn_sw128(wb + k * 2048, kBBytes / 2) : sdesc_sw128(wb + k * 32), id,
                                 c > 0 || k > 0);
                    mma_commit(smem_u32(&sh.empty[st]));
                }
                if (ok) mma_commit(smem_u32(&sh.acc_full[buf]));
            }
            mma_commit(smem_u32(&sh.mma_done));
            mbar_wait_drain(smem_u32(&sh.mma_done), 0, a.err);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- results
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        uint32_t n = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total; i += gridDim.x, ++n) {
            const TileAt p = tile_at(a, i, ntiles);
            const uint32_t buf = n & 1;
            if (ok) ok = wait(smem_u32(&sh.acc_full[buf]), (n >> 1) & 1, ERR_WAIT_PART_FULL);
            __syncwarp();
            tc_fence_after();
            const int t = p.t0 + warp * 32 + lane;
            T *dst = static_cast<T *>(a.out) + static_cast<int64_t>(t) * a.o_st + static_cast<int64_t>(p.h) * a.o_sh + p.n0;
#pragma unroll
            for (int c = 0; c < kTile; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + buf * kTile + lanes + c, r);
                tmem_wait_ld();
                if (t < a.T && ok) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        if (p.n0 + c + k >= a.N) break;
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = E::pack(__uint_as_float(r[k + 2 * q]), __uint_as_float(r[k + 2 * q + 1]));
                        *reinterpret_cast<uint4 *>(dst + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.acc_empty[buf]));
        }
    }
    __syncthreads();
    if (warp == 5) tmem_dealloc<256>(tmem);
}

template <typename T, bool KN>
cudaError_t launch_t(const CUtensorMap &x, const CUtensorMap &w, const ProjArgs &a, int num_sms, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(head_proj_kernel<T, KN>, kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t total = static_cast<int64_t>((a.T + kTile - 1) / kTile) * a.H * ((a.N + kTile - 1) / kTile);
    const int grid = total < num_sms ? static_cast<int>(total) : num_sms;
    return launch_pdl(head_proj_kernel<T, KN>, dim3(grid), dim3(kThreads), kSmem, stream, x, w, a);
}

}  // namespace

cudaError_t launch_proj(const CUtensorMap &x, const CUtensorMap &w, const ProjArgs &a, bool bf16, bool w_kn,
                        int num_sms, cudaStream_t stream) {
    if (bf16)
        return w_kn ? launch_t<__nv_bfloat16, true>(x, w, a, num_sms, stream)
                    : launch_t<__nv_bfloat16, false>(x, w, a, num_sms, stream);
    return w_kn ? launch_t<__half, true>(x, w, a, num_sms, stream) : launch_t<__half, false>(x, w, a, num_sms, stream);
}

}  // namespace moe
