// Expanded latent attention of a ragged batch (mla_attn_ragged).
#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

// One CTA takes 256 query rows of one head as two tiles of 128 and walks the sequence's
// keys in tiles of 128 with the running maximum and sum of a softmax:
//   S_t [128, 128]  = Q_t K^T      M = 128, N = 128, 192 columns (128 + the shared 64)
//   P_t = 2^(S_t scale - m)         m: the row's reference (its maximum, less Elem::kLift)
//   O_t [128, 128] += P_t V        P_t in tensor memory, V with its columns contiguous
// The two tiles alternate: while one's scores pass through the exponentials, the other's
// products run. Both read one copy of the keys and values. K and V arrive in 16 KB
// pieces (128 keys x 64 columns) through a ring of eight; the rotary piece is shared
// by all heads, so the [k_nope | k_pe] concatenation is never stored.
// Tensor memory: S_0, S_1, O_0, O_1 of 128 columns each; P_t lies over the first half
// of S_t (two 16-bit values per column). 2,560 tensor cycles per 256 x 128 scores bound a
// long prompt, and the 336 KB that pass through shared memory for them take as long:
// 8,192 tokens of 64 heads 856 us, 1.6 PFLOP/s (2,690 cycles at 128 bytes each; 931 us at
// the 1,830 MHz of the power limit). Short
// prompts pay 8,000 cycles of start and end per CTA and the empty part of a sequence's
// last 256 rows.
constexpr int kTile = 128;
constexpr int kQRows = 2 * kTile;
constexpr int kPiece = kTile * 128;              // 16 KB
constexpr int kQPieces = 3;                      // per row tile
constexpr int kSlots = 8;
constexpr int kPerTile = 5;                      // 3 pieces of K, 2 of V
constexpr int kOffRing = 2 * kQPieces * kPiece;
constexpr int kOffMisc = kOffRing + kSlots * kPiece;
constexpr int kSmem = kOffMisc + 1024;
constexpr int kThreads = 3 * kTile;              // a warpgroup per row tile; loads and MMA (two warps idle)
constexpr float kLag = 8.0f;                     // see mla_paged.cu
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // of every other key tile
    uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], mma_done;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Shared) <= 1024, "");

__device__ __forceinline__ bool offsets_ok(const RaggedArgs &a, int64_t q0, int64_t q1, int64_t k0, int64_t k1) {
    return !(q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk || q1 - q0 > a.max_q);
}
__device__ __forceinline__ bool offsets_ok(const RaggedArgs &a, int b) {
    return offsets_ok(a, a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]);
}

// The grid has max_q's tiles for every sequence, of which each finds its own, or, where
// those are kSlotRatio times as many, Tq / 256 + B slots: sequence b's tiles start at slot
// cu_q[b] / 256 + b, which leaves room for its last, partial one. A CTA without a tile
// costs 0.7 us of an SM, the search for a slot's sequence as much. 3,000 tokens beside 31
// prompts of 10: 306 us with max_q's tiles (384 a head), 241 with slots (43); 200 tokens
// under a bound of 65,536: 81 and 9.6; but nine prompts of 3 to 1,900: 319 (72) and 328
// (35).
constexpr int kSlotRatio = 3;
static_assert(kQRows == 256, "");
__device__ __forceinline__ int first_slot(const RaggedArgs &a, int b) { return (a.cu_q[b] >> 8) + b; }

// The last sequence that starts at slot x or before (a search by the whole warp).
__device__ __forceinline__ int sequence_of(const RaggedArgs &a, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = a.B;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < n && first_slot(a, lo + i) <= x);
        const int k = le ? (31 - __clz(le)) * step : 0;
        lo += k;
        n = min(step, n - k);
    }
    return lo;
}

template <typename T, bool SLOTS>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kn,
                       const __grid_constant__ CUtensorMap map_kp, const __grid_constant__ CUtensorMap map_v,
                       const RaggedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using E = Elem<T>;

    pdl_trigger();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_kn);
        tma_prefetch_desc(&map_kp);
        tma_prefetch_desc(&map_v);
    }
    pdl_wait();
    // the longest rows first: they see the most keys
    int qt = gridDim.x - 1 - blockIdx.x;
    const int h = blockIdx.y, b = SLOTS ? sequence_of(a, blockIdx.x) : blockIdx.z;
    if (SLOTS && h == 0 && threadIdx.x == 0 && blockIdx.x < static_cast<unsigned>(a.B) && !offsets_ok(a, blockIdx.x))
        record_error(a.err, ERR_BAD_INDEX);   // each of the first B slots looks after one sequence's offsets
    const int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1], kk0 = a.cu_k[b], kk1 = a.cu_k[b + 1];
    if (!offsets_ok(a, q0, q1, kk0, kk1)) {
        if (!SLOTS && threadIdx.x == 0 && qt == 0 && h == 0) record_error(a.err, ERR_BAD_INDEX);
        return;
    }
    const int nq = static_cast<int>(q1 - q0), nk = static_cast<int>(kk1 - kk0);
    if (SLOTS) qt = (nq + kQRows - 1) / kQRows - 1 - (static_cast<int>(blockIdx.x) - first_slot(a, b));
    const int r0 = qt * kQRows;
    if ((SLOTS && qt < 0) || r0 >= nq) return;
    const int rows = min(kQRows, nq - r0);
    const bool two = rows > kTile;
    // keys the CTA's last row sees
    auto visible = [&](int row) {
        if (!a.causal) return nk;
        const int v = nk - nq + row + 1;
        return v < 0 ? 0 : v;
    };
    const int keys = visible(r0 + rows - 1);
    const int tiles = (keys + kTile - 1) / kTile;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sh.k_full[t]), 1), mbar_init(smem_u32(&sh.k_empty[t]), 1);
            mbar_init(smem_u32(&sh.v_full[t]), 1), mbar_init(smem_u32(&sh.v_empty[t]), 1);
            mbar_init(smem_u32(&sh.q_full[t]), 1), mbar_init(smem_u32(&sh.s_full[t]), 1);
            mbar_init(smem_u32(&sh.p_full[t][0]), kTile), mbar_init(smem_u32(&sh.p_full[t][1]), kTile);
            mbar_init(smem_u32(&sh.o_full[t]), 1);
        }
        mbar_init(smem_u32(&sh.mma_done), 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc<512>(smem_u32(&sh.tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are this CTA's, so its tensor memory starts at address 0: a
    // constant costs the MMA issue nothing
    constexpr uint32_t tmem = 0;
    const Waiter wait{smem_u32(&sh.abort), a.err};

    // 384 threads x 168 registers are the launch's; the third warpgroup gives 80 of its
    // 168 to the other two, which hold a row's 128 scores (2 x 208 + 88 = 3 x 168). The
    // instructions stand inside the branches: the compiler takes each as the budget of
    // what it dominates.
    if (warp >= 8) regs_down<88>();
    if (warp == 8) {
        // -------------------------------------------------------- loads
        if (lane == 0 && tiles > 0) {
            const uint64_t pol = policy_evict_normal();
            auto load_q = [&](int t) {
                mbar_arrive_expect_tx(smem_u32(&sh.q_full[t]), kQPieces * kPiece);
                for (int c = 0; c < kQPieces; ++c)
                    tma_load_3d(sbase + (t * kQPieces + c) * kPiece, &map_q, smem_u32(&sh.q_full[t]), c * 64, h,
                                static_cast<int>(q0) + r0 + t * kTile, pol);
            };
            load_q(0);
            int g = 0;
            for (; g < tiles; ++g) {
                const int key = static_cast<int>(kk0) + g * kTile;
                // The pieces take the slots of those eight before them: the third of K and
                // the two of V of two tiles ago, and the first two of the last K.
                const uint32_t two_ago = ((g >> 1) & 1) ^ 1, one_ago = ((g - 1) >> 1) & 1;
                const uint32_t kf = smem_u32(&sh.k_full[g & 1]), vf = smem_u32(&sh.v_full[g & 1]);
                auto dst = [&](int c) { return sbase + kOffRing + ((g * kPerTile + c) % kSlots) * kPiece; };
                if (!wait(smem_u32(&sh.k_empty[g & 1]), two_ago, ERR_WAIT_SMEM_EMPTY)) break;
                mbar_arrive_expect_tx(kf, 3 * kPiece);
                tma_load_3d(dst(0), &map_kn, kf, 0, h, key, pol);
                if (!wait(smem_u32(&sh.v_empty[g & 1]), two_ago, ERR_WAIT_SMEM_EMPTY)) break;
                tma_load_3d(dst(1), &map_kn, kf, 64, h, key, pol);
                tma_load_2d(dst(2), &map_kp, kf, 0, key, pol);
                if (g == 0 && two) load_q(1);
                if (g > 0 && !wait(smem_u32(&sh.k_empty[(g - 1) & 1]), one_ago, ERR_WAIT_SMEM_EMPTY)) break;
                mbar_arrive_expect_tx(vf, 2 * kPiece);
                tma_load_3d(dst(3), &map_v, vf, 0, h, key, pol);
                tma_load_3d(dst(4), &map_v, vf, 64, h, key, pol);
            }
            // the last loads must land before the CTA may exit
            for (int t = 0; t < (two && g > 0 ? 2 : 1); ++t) mbar_wait_drain(smem_u32(&sh.q_full[t]), 0, a.err);
            for (int i = g < 2 ? 0 : g - 2; i < g; ++i) {
                mbar_wait_drain(smem_u32(&sh.k_full[i & 1]), (i >> 1) & 1, a.err);
                mbar_wait_drain(smem_u32(&sh.v_full[i & 1]), (i >> 1) & 1, a.err);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        // -------------------------------------------------------- MMA issue
        if (tiles > 0 && elect_one()) {
            const IssueWaiter wait{smem_u32(&sh.abort), a.err};
            constexpr uint32_t id_s = idesc16(E::kFmt, kTile, kTile);
            constexpr uint32_t id_o = idesc16(E::kFmt, kTile, kMlaV, false, true);
            constexpr uint32_t id_o64 = idesc16(E::kFmt, kTile, 64, false, true);
            const int nt = two ? 2 : 1;
            const uint64_t dq = sdesc_sw128(sbase), dk = sdesc_sw128(sbase + kOffRing);
            const uint64_t dv = sdesc_mn_sw128(sbase + kOffRing, kPiece);
            // A third of S_t of key tile g. MMAs run in issue order: S_t overwrites P_t after
            // the product before has read it.
            auto scores = [&](int t, uint32_t g, int c) {
                const uint64_t q = dq + ((t * kQPieces + c) * kPiece >> 4);
                const uint64_t kd = dk + (((g * kPerTile + c) % kSlots) * kPiece >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_16_ss(tmem + t * kTile, q + (k * 32 >> 4), kd + (k * 32 >> 4), id_s, c > 0 || k > 0);
            };
            auto k_test = [&](uint32_t g) { return mbar_test(smem_u32(&sh.k_full[g & 1]), (g >> 1) & 1); };
            auto k_wait = [&](uint32_t g) { return wait(smem_u32(&sh.k_full[g & 1]), (g >> 1) & 1, ERR_WAIT_TMA_FULL); };
            auto v_test = [&](uint32_t g) { return mbar_test(smem_u32(&sh.v_full[g & 1]), (g >> 1) & 1); };
            auto v_wait = [&](uint32_t g) { return wait(smem_u32(&sh.v_full[g & 1]), (g >> 1) & 1, ERR_WAIT_TMA_FULL); };
            // One loop body issues a row tile's product with V and then its next scores; row
            // tiles take turns, one at its exponentials while the other multiplies. The body
            // stays small on purpose: unrolled over the row tiles it outgrew the instruction
            // cache beside the softmax's code, and every turn of the loop cost 900 cycles.
            // A barrier test takes about 100 cycles and few MMAs are queued: the tests for
            // the next step are made between the present one's MMAs.
            bool ok = true, ready = false;
            const int steps = tiles * nt;
#pragma unroll 1
            for (int i = -nt; i < steps && ok; ++i) {
                const int t = two ? i & 1 : 0, j = two ? i >> 1 : i;   // j = -1: the first scores
                const bool last_t = t == nt - 1;
                if (j >= 0) {
                    // the product's V and the first half of its weights
                    if (!ready && !(v_wait(j) && wait(smem_u32(&sh.p_full[t][0]), j & 1, ERR_WAIT_PART_FULL))) break;
                    const uint32_t s0 = (j * kPerTile + 3) % kSlots, s1 = (j * kPerTile + 4) % kSlots;
                    const uint32_t p = tmem + t * kTile, o = tmem + 2 * kTile + t * kMlaV;
                    const uint64_t b0 = dv + (s0 * kPiece >> 4);
                    const uint32_t acc0 = j > 0;
                    tc_fence_after();
                    if (s1 == s0 + 1) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (k == 4) {
                                if (!wait(smem_u32(&sh.p_full[t][1]), j & 1, ERR_WAIT_PART_FULL)) { ok = false; break; }
                                tc_fence_after();
                            }
                            mma_16_ts(o, p + k * 8, b0 + (k * 2048 >> 4), id_o, k > 0 ? 1 : acc0);
                        }
                    } else {   // the two pieces lie at the ring's end and start
                        const uint64_t b1 = dv + (s1 * kPiece >> 4);
                        ok = wait(smem_u32(&sh.p_full[t][1]), j & 1, ERR_WAIT_PART_FULL);
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < 8 && ok; ++k) {
                            mma_16_ts(o, p + k * 8, b0 + (k * 2048 >> 4), id_o64, k > 0 ? 1 : acc0);
                            mma_16_ts(o + 64, p + k * 8, b1 + (k * 2048 >> 4), id_o64, k > 0 ? 1 : acc0);
                        }
                    }
                    if (!ok) break;
                    if (last_t) mma_commit(smem_u32(&sh.v_empty[j & 1]));   // the last row tile frees V
                    if (j == tiles - 1) mma_commit(smem_u32(&sh.o_full[t]));
                }
                const int g = j + 1;   // the key tile of the next scores
                ready = false;
                if (g < tiles) {
                    if (j < 0 && !wait(smem_u32(&sh.q_full[t]), 0, ERR_WAIT_TMA_FULL)) break;
                    if (t == 0 && !k_test(g) && !k_wait(g)) break;
                    tc_fence_after();
                    // the step after this one
                    const int t1 = last_t ? 0 : 1, j1 = last_t ? g : j;
                    scores(t, g, 0);
                    const bool v_ready = j1 >= 0 && v_test(j1);
                    scores(t, g, 1);
                    ready = v_ready && mbar_test(smem_u32(&sh.p_full[t1][0]), j1 & 1);
                    scores(t, g, 2);
                    mma_commit(smem_u32(&sh.s_full[t]));
                    if (last_t) mma_commit(smem_u32(&sh.k_empty[g & 1]));   // the last row tile frees K
                }
            }
            mma_commit(smem_u32(&sh.mma_done));
            mbar_wait_drain(smem_u32(&sh.mma_done), 0, a.err);
        }
        __syncwarp();
    } else if (warp < 8) {
        // -------------------------------------------------------- softmax and results
        regs_up<208>();
        const int t = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + t * kTile + lanes, to = tmem + 2 * kTile + t * kMlaV + lanes;
        const int row = r0 + t * kTile + (warp & 3) * 32 + lane;
        const bool valid = row < nq;
        const int vis = valid ? visible(row) : 0;
        // tiles that every row of the warp sees whole need no mask
        const int vis_min = __reduce_min_sync(0xffffffffu, vis);
        float m = -INFINITY, l = 0.f, lost = 0.f;
        bool ok = true;
        auto hold = [&](uint64_t *bar, uint32_t parity, uint32_t bit) {
            if (ok) ok = wait(smem_u32(bar), parity, bit);
        };
        if (t == 0 || two) {
            for (int j = 0; j < tiles; ++j) {
                hold(&sh.s_full[t], j & 1, ERR_WAIT_PART_FULL);
                __syncwarp();
                tc_fence_after();
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, r[c]);
                tmem_wait_ld();
                const int kb = j * kTile;
                if (kb + kTile > vis_min) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (kb + c * 32 + i >= vis) r[c][i] = __float_as_uint(-INFINITY);
                }
                if (t == 0 && nk - kb < kTile) {
                    // value rows past the sequence's end: their weights are zero, but
                    // zero times a NaN is not. The rows are the next sequence's.
                    hold(&sh.v_full[j & 1], (j >> 1) & 1, ERR_WAIT_TMA_FULL);
                    const int left = nk - kb, per = (kTile - left) * 8;
                    for (int i = threadIdx.x; i < 2 * per; i += kTile) {
                        const int c = i >= per;
                        st_shared_v4(sbase + kOffRing + ((j * kPerTile + 3 + c) % kSlots) * kPiece + left * 128 + (i - c * per) * 16,
                                     make_uint4(0, 0, 0, 0));
                    }
                    fence_async_smem();
                }
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    top[c] = __uint_as_float(r[c][0]);
#pragma unroll
                    for (int i = 1; i < 31; i += 2)
                        top[c] = fmaxf(top[c], fmaxf(__uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1])));
                    top[c] = fmaxf(top[c], __uint_as_float(r[c][31]));
                }
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
                const bool behind = mx - m > E::kLift + kLag;
                if (__any_sync(0xffffffffu, behind)) {
                    const float mn = fmaxf(m, mx - E::kLift);
                    const float f = m == -INFINITY ? 0.f : ex2(m - mn);
                    l *= f, lost *= f;
                    m = mn;
                    if (j > 0) {
                        // S_t of this tile was issued after P_t V of the one before, and
                        // its completion covers both: O_t is at rest
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[32];
                            tmem_ld32(to + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(to + c * 32, o);
                        }
                    }
                }
                const float e = m == -INFINITY ? 0.f : m;
                const uint64_t scale2 = pack_f32x2(a.scale_log2, a.scale_log2), neg2 = pack_f32x2(-e, -e);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    // 64 keys: the product starts on them while the rest is computed
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const uint64_t s2 = pack_f32x2(__uint_as_float(r[2 * hh + c][i]), __uint_as_float(r[2 * hh + c][i + 1]));
                            const float2 x = unpack_f32x2(fma_f32x2(s2, scale2, neg2));
                            const float p0 = ex2(x.x), p1 = ex2(x.y);
                            sum[(i / 2) & 3] = add_f32x2(sum[(i / 2) & 3], pack_f32x2(p0, p1));
                            // the weights enter the second product in the tensors' 16-bit
                            // type: half an ulp each, averaged over the keys (fp16: down to
                            // 2^-21 of the largest, from there an absolute 2^-32 of it)
                            p[c * 16 + i / 2] = E::pack(p0, p1);
                        }
                    tmem_st32(ts + hh * 32, p);
                    if (hh == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(smem_u32(&sh.p_full[t][0]));
                    }
                }
                const float2 both = unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])));
                add_compensated(l, lost, both.x + both.y);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[t][1]));
            }
            if (tiles > 0) {
                hold(&sh.o_full[t], 0, ERR_WAIT_PART_FULL);
                __syncwarp();
                tc_fence_after();
            }
            l += lost;
            const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
            // Results leave through the row tile's query buffer (its scores are done): a
            // thread holds a row, and rows are far apart in memory, so that 16-byte stores
            // from registers would touch 32 lines each (4,000 cycles for the tile). From the
            // buffer 16 lanes store a row's 256 bytes. Rows of 256 bytes, the 16-byte unit
            // swizzled by the row; a warp keeps to its own 32 rows.
            const uint32_t stage = sbase + t * kQPieces * kPiece + (warp & 3) * 32 * 256;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                if (tiles > 0) {
                    tmem_ld32(to + c * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = E::pack(__uint_as_float(o[i + 2 * k]) * inv, __uint_as_float(o[i + 2 * k + 1]) * inv);
                    st_shared_v4(stage + lane * 256 + (((c * 4 + i / 8) ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
            __syncwarp();
            T *dst = static_cast<T *>(a.out) + (q0 + row - lane) * a.o_st + h * a.o_sh + (lane & 15) * 8;
            const int left = nq - (row - lane);   // rows of the warp that exist
#pragma unroll 4
            for (int i = 0; i < 32; i += 2) {
                const int r = i + (lane >> 4);
                const uint4 v = ld_shared_v4(stage + r * 256 + (((lane & 15) ^ (r & 7)) << 4));
                if (r < left) *reinterpret_cast<uint4 *>(dst + r * a.o_st) = v;
            }
            if (valid && a.lse)
                a.lse[(q0 + row) * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 9) tmem_dealloc<512>(sh.tmem);
}

template <typename T, bool SLOTS>
cudaError_t launch_t(const CUtensorMap &q, const CUtensorMap &kn, const CUtensorMap &kp, const CUtensorMap &v,
                     const RaggedArgs &a, dim3 grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(ragged_attn_kernel<T, SLOTS>, kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(ragged_attn_kernel<T, SLOTS>, grid, dim3(kThreads), kSmem, stream, q, kn, kp, v, a);
}

}  // namespace

cudaError_t launch_ragged(const CUtensorMap &q, const CUtensorMap &k_nope, const CUtensorMap &k_pe,
                          const CUtensorMap &v, const RaggedArgs &a, bool bf16, cudaStream_t stream) {
    // (max_q = 0: one tile, which reports the sequences that have queries all the same)
    const int64_t tiles = a.max_q > 0 ? (a.max_q + kQRows - 1) / kQRows : 1, slots = a.Tq / kQRows + a.B;
    if (tiles * a.B >= kSlotRatio * slots) {
        const dim3 grid(static_cast<unsigned>(slots), a.H);
        return bf16 ? launch_t<__nv_bfloat16, true>(q, k_nope, k_pe, v, a, grid, stream)
                    : launch_t<__half, true>(q, k_nope, k_pe, v, a, grid, stream);
    }
    const dim3 grid(static_cast<unsigned>(tiles), a.H, a.B);
    return bf16 ? launch_t<__nv_bfloat16, false>(q, k_nope, k_pe, v, a, grid, stream)
                : launch_t<__half, false>(q, k_nope, k_pe, v, a, grid, stream);
}

}  // namespace moe
