// Absorbed latent attention over the paged cache (mla_attn_paged).
#include <algorithm>

#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

// The (token, head) rows of a sequence are flattened (row = token * H + head) and cut
// into tiles of 64; keys come in tiles of 64. For one pair of tiles
//   S [64 rows, 64 keys]  = Q K^T          9 column groups of 64, M = 64, N = 64
//   P = 2^(S scale - m)                     m: the row's reference (its maximum, less Elem::kLift)
//   O^T [512, 64 rows]   += C^T P^T        4 blocks of 128 latent columns, M = 128, N = 64
// The latent columns of the key tile serve both products from one copy in shared
// memory: as B of the first (keys x columns, columns contiguous) and, transposed, as A
// of the second. Holding O transposed keeps the accumulator at 256 of the 512 tensor
// memory columns and lets every MMA of the larger product fill its 128 lanes, although
// there are only 64 rows (one token of 64 heads). Q stays in shared memory (72 KB);
// the key tiles pass through a ring of two (144 KB).
//
// One token of 64 heads does 121 flops per byte of cache: the HBM rate bounds it. A tile's
// MMAs run 1,970 cycles (33 and 49 each, the time to read 4 and 6 KB of operands at 128
// bytes per cycle) of the 3,410 in which HBM delivers one to every SM (2,070 MHz). A ring
// of two tiles covers that if a tile's way through it stays short: arrival (2,800 cycles
// from HBM under load), scores, softmax, first products. For the same reason the two
// products have their issuing warps, and eight warps share a tile's softmax. 256 sequences
// of 4,246 keys on average: 217 us, 5.9 TB/s of what has to be read and written. The row
// tiles of a sequence follow one another: where L2 still holds its keys by then (a chunk of
// new tokens), shared memory is the bound; in a batch it does not, and HBM delivers them
// once per row tile (64 sequences of 4,000 tokens, 128 heads: 579 MB read for a cache of
// 295; 256 sequences 431 us for a floor of 207). Shared memory: 240 KB that a tile's
// MMAs read and 80 KB that are written for them take 2,560 cycles of the 2,760 per tile
// (2 x 512 new tokens over 7,000 keys: 950 us, 0.96 PFLOP/s).
//
// The work is split evenly by key tiles over the CTAs, whatever the sequences' lengths:
// the tiles of all (sequence, row tile) items form one line, CTA c takes the c-th part
// of it, and an item that several CTAs share leaves partial sums that a second kernel
// joins in a fixed order.
constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kGroups = 4;                       // pairs of 64-column groups of the latent
constexpr int kPairBytes = 2 * kKeys * 128;      // 16 KB
constexpr int kGroupBytes = kKeys * 128;         // 8 KB
constexpr int kPairSlots = 2 * kGroups;
constexpr int kRopeSlots = 2;
constexpr int kMaxSubs = 8;                      // boxes per key tile: pages of 8 rows
constexpr int kQBytes = (kMlaWidth / 64) * kRows * 128;
constexpr int kOffP = kQBytes;
constexpr int kOffPairs = kOffP + kRows * 128;
constexpr int kOffRope = kOffPairs + kPairSlots * kPairBytes;
constexpr int kOffMisc = kOffRope + kRopeSlots * kGroupBytes;
constexpr int kMisc = 2560;
constexpr int kSmem = kOffMisc + kMisc;
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kThreads = kSoftThreads + 128;     // + loads of keys and of queries, two MMA warps
constexpr int kTmemO = 0;                        // 4 x 64 columns
constexpr int kTmemS = 256;                      // 2 x 64 columns
// A row's reference follows its running maximum only when that has risen by more than
// 2^8: the sums then stay below 2^8 times their true scale, far from overflow, and O is
// rescaled a few times per item instead of once per tile. (Differences are compared: at
// references where 8 is less than the spacing of fp32 a sum would round past it.)
constexpr float kLag = 8.0f;
// Fewest key tiles a CTA is given: one, or, where that cuts no CTA's part between two items,
// two, which make half as many partial sums. A CTA with pieces of two items has two results
// and two sets of queries.
// - No more tiles than CTAs: two if every item has an even number of them (one sequence of
//   960 tokens and 128 heads, two items of 15 tiles: with two 16.2 us, with one 12.9; two
//   sequences of 4,000, 63 tiles: 19.3 and 16.4; 60 of 128: 12.6 and 16.4; 8 of 1,000: 17.4
//   and 18.7; one of 1,000: 13.7 and 13.1).
// - Up to twice as many: one would leave some CTAs two all the same. Two if every sequence's
//   items together have an even number (one of 8,000 tokens and 128 heads, two items of 125
//   tiles: with two 19.2 us, with one 21.2; sequences of 100, 700 and 5,000 tokens in one
//   call: 21.2 and 19.5).
constexpr int kEvenTiles = 2;

static_assert(kQBytes >= 8192 * 8, "the start-up scan keeps one 8-byte prefix per sequence in the query buffer");
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kSoftWarps == 2 * kGroups, "a softmax warp clears a column group");

struct Seq {
    int row0, n, ctx;
};

struct Shared {
    uint64_t pair_full[kPairSlots], pair_empty[kPairSlots];
    uint64_t rope_full[kRopeSlots], rope_empty[kRopeSlots];
    uint64_t s_full[2], s_empty[2];
    uint64_t p_full, pv_done, q_full, q_empty, mma_done[2];
    uint32_t tmem;
    int abort;
    float factor[kRows];
    // the two halves' maxima of a tile, and their sums of a segment: a segment of one tile has
    // no barrier between a warp's read of its partner's maxima and the partner's sums
    float half_of[2][kRows], sum_of[2][kRows];
    int64_t row_off[kRows];
    int64_t warp_sum[kThreads / 32];
    // the line of key tiles: CTA c's part starts at each * c + min(c, rem)
    int64_t each, lo, hi, start_off;
    int rem, start_b, start_rt;
    Seq start;
};
static_assert(sizeof(Shared) <= kMisc, "");

// Queries and visible keys of sequence b. A length or offset outside its buffer is
// recorded once and leaves the sequence without rows.
__device__ __forceinline__ Seq read_seq(const PagedArgs &a, int b, bool report) {
    Seq s;
    s.ctx = a.ctx[b];
    int64_t r0 = b, r1 = b + 1;
    if (a.cu_q) r0 = a.cu_q[b], r1 = a.cu_q[b + 1];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.Tq && s.ctx >= 0 &&
                    s.ctx <= static_cast<int64_t>(a.max_pages) * a.page_size;
    if (!ok && report) record_error(a.err, ERR_BAD_INDEX);
    s.row0 = ok ? static_cast<int>(r0) : 0;
    s.n = ok ? static_cast<int>(r1 - r0) : 0;
    if (!ok) s.ctx = 0;
    return s;
}

// (The rows of a call fit 31 bits: checked on the host.)
__device__ __forceinline__ int row_tiles(const Seq &s, int H) { return (s.n * H + kRows - 1) / kRows; }

// Keys that the last row of a row tile sees, and the key tiles that cover them (at
// least one unit of work, so that rows without keys get their zeros).
__device__ __forceinline__ int tile_keys(const PagedArgs &a, const Seq &s, int rt) {
    const int last = min((rt + 1) * kRows, s.n * a.H) - 1;
    return max(0, s.ctx - s.n + a.by_H.div(last) + 1);
}
__device__ __forceinline__ int units_of(int keys) { return keys <= kKeys ? 1 : (keys - 1) / kKeys + 1; }

// Walks a CTA's part [lo, hi) of the line of key tiles, item by item.
struct Walk {
    int b, rt, rts;
    int64_t at, hi, off;   // off: units of item (b, rt) before `at`
    Seq s;
    // the current segment: key tiles [k0, k1) of `kt` of row tile rt of sequence b
    int k0, k1, kt, keys;

    __device__ void start(const PagedArgs &a, const Shared &sh) {
        b = sh.start_b, rt = sh.start_rt, at = sh.lo, hi = sh.hi, off = sh.start_off;
        s = sh.start;
        rts = row_tiles(s, a.H);
    }
    __device__ bool next(const PagedArgs &a) {
        if (at >= hi) return false;
        while (true) {
            if (rt >= rts) {
                ++b;
                if (b >= a.B) return false;
                rt = 0;
                s = read_seq(a, b, false);
                rts = row_tiles(s, a.H);
                continue;
            }
            keys = tile_keys(a, s, rt);
            const int u = units_of(keys);
            if (off >= u) {
                off -= u;
                ++rt;
                continue;
            }
            kt = u;
            k0 = static_cast<int>(off);
            const int64_t take = min(static_cast<int64_t>(u) - off, hi - at);
            k1 = k0 + static_cast<int>(take);
            return true;
        }
    }
    __device__ void advance() {
        at += k1 - k0;
        off = 0;
        ++rt;
    }
    // key tiles of the segment that hold keys
    __device__ int tiles() const { return keys > 0 ? k1 - k0 : 0; }
};

// Walks the same part key tile by key tile and reads the page table one tile ahead of
// its user: page[i], row[i] of the boxes of the present tile, of which `boxes` hold keys.
struct Cursor {
    Walk w;
    const int32_t *tab;
    int j, n, key, at, end;
    int boxes, page[kMaxSubs], row[kMaxSubs];

    __device__ void start(const PagedArgs &a, const Shared &sh) {
        w.start(a, sh);
        j = n = 0;
    }
    __device__ bool step(const PagedArgs &a) {
        if (j == n) {
            do {
                if (n > 0) w.advance();
                n = 0;
                if (!w.next(a)) return false;
                n = w.tiles();
                if (n == 0) w.advance();
            } while (n == 0);
            j = 0;
            key = w.k0 * kKeys;
            const int first = a.by_page.div(key);
            at = key - first * a.page_size;
            end = min(w.keys, w.k1 * kKeys);
            tab = a.table + static_cast<int64_t>(w.b) * a.table_st + first;
        }
        ++j;
#pragma unroll
        for (int i = 0; i < kMaxSubs; ++i) {
            if (i * a.box_rows >= kKeys) break;
            row[i] = at;
            if (key < end) page[i] = *tab, boxes = i + 1;
            key += a.box_rows;
            at += a.box_rows;
            if (at == a.page_size) at = 0, ++tab;
        }
        return true;
    }
};

__device__ __forceinline__ int64_t part_lo(int64_t each, int rem, int c) { return each * c + min(c, rem); }

// The CTA whose part holds unit u.
__device__ __forceinline__ int part_of(int64_t each, int rem, int64_t u) {
    const int64_t longer = (each + 1) * rem;
    return static_cast<int>(u < longer ? u / (each + 1) : rem + (u - longer) / each);
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Every thread: the line's length, this CTA's part of it, and the sequence it starts in.
__device__ void plan(const PagedArgs &a, Shared &sh, int64_t *prefix) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t base = 0;
    bool odd_items = false, odd_sums = false;   // of an item; of a sequence's items together
    if (tid == 0) sh.start_b = 0, sh.start_rt = 0, sh.start_off = 0, sh.start = Seq{0, 0, 0};   // a CTA without a part
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Seq s{0, 0, 0};
        if (b < a.B) s = read_seq(a, b, blockIdx.x == 0);
        int64_t u = 0;
        int any = 0;   // the items' lengths
        const int rts = row_tiles(s, a.H);
        // few row tiles: one thread per sequence; many: the warp takes them together
        if (rts <= 8)
            for (int r = 0; r < rts; ++r) {
                const int n = units_of(tile_keys(a, s, r));
                u += n, any |= n;
            }
        unsigned many = __ballot_sync(0xffffffffu, rts > 8);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            Seq o;
            o.row0 = 0;
            o.n = __shfl_sync(0xffffffffu, s.n, src);
            o.ctx = __shfl_sync(0xffffffffu, s.ctx, src);
            const int orts = __shfl_sync(0xffffffffu, rts, src);
            int64_t v = 0;
            for (int r = lane; r < orts; r += 32) {
                const int n = units_of(tile_keys(a, o, r));
                v += n, any |= n;
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            if (lane == src) u = v;
        }
        const int64_t inc = warp_scan(u, lane);
        if (lane == 31) sh.warp_sum[warp] = inc;
        odd_items |= __syncthreads_or(any & 1);
        int64_t before = base, all = 0;
#pragma unroll 1
        for (int w = 0; w < min(kThreads, a.B - b0 + 31) / 32; ++w) {   // (short code: it runs once)
            if (w < warp) before += sh.warp_sum[w];
            all += sh.warp_sum[w];
        }
        if (b < a.B) prefix[b] = before + inc - u;
        base += all;
        odd_sums |= __syncthreads_or(u & 1);
    }
    const bool odd = base <= gridDim.x ? odd_items : odd_sums;
    const int64_t most = odd ? base : base / kEvenTiles;
    const unsigned parts = most < 1 ? 1u : most < gridDim.x ? static_cast<unsigned>(most) : gridDim.x;
    int64_t each;
    int rem;
    if (most > 0 && most <= gridDim.x) {
        each = odd ? 1 : kEvenTiles, rem = 0;
    } else if (base < (int64_t{1} << 32)) {   // 32-bit division takes a quarter of the time
        const unsigned t = static_cast<unsigned>(base);
        each = t / parts, rem = static_cast<int>(t % parts);
    } else {
        each = base / parts, rem = static_cast<int>(base % parts);
    }
    const unsigned c = blockIdx.x;
    const int64_t lo = c < parts ? part_lo(each, rem, c) : base, hi = c < parts ? part_lo(each, rem, c + 1) : base;
    if (tid == 0) sh.each = each, sh.rem = rem, sh.lo = lo, sh.hi = hi;
    for (int b = tid; b < a.B; b += kThreads) {
        const int64_t p = prefix[b], e = b + 1 < a.B ? prefix[b + 1] : base;
        if (p <= lo && lo < e) {
            sh.start_b = b;
            sh.start_rt = 0;
            sh.start_off = lo - p;
            sh.start = read_seq(a, b, false);
        }
    }
    fence_async_smem();   // the prefixes' buffer is filled by TMA next
    __syncthreads();
    const Seq s = sh.start;
    const int rts = row_tiles(s, a.H);
    if (warp == 0 && rts > 1) {
        // the row tile of that sequence: 32 at a time
        int64_t off = sh.start_off;
        for (int r0 = 0; r0 < rts; r0 += 32) {
            const int64_t u = r0 + lane < rts ? units_of(tile_keys(a, s, r0 + lane)) : 0;
            const int64_t inc = warp_scan(u, lane);
            if (inc - u <= off && off < inc) {
                sh.start_rt = r0 + lane;
                sh.start_off = off - (inc - u);
            }
            const int64_t all = __shfl_sync(0xffffffffu, inc, 31);
            if (off < all) break;
            off -= all;
        }
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using E = Elem<T>;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairSlots; ++i) mbar_init(smem_u32(&sh.pair_full[i]), 1), mbar_init(smem_u32(&sh.pair_empty[i]), 1);
        for (int i = 0; i < kRopeSlots; ++i) mbar_init(smem_u32(&sh.rope_full[i]), 1), mbar_init(smem_u32(&sh.rope_empty[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.s_full[i]), 1), mbar_init(smem_u32(&sh.s_empty[i]), kSoftThreads);
        mbar_init(smem_u32(&sh.p_full), kSoftThreads);
        mbar_init(smem_u32(&sh.pv_done), 1);
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.mma_done[0]), 1), mbar_init(smem_u32(&sh.mma_done[1]), 1);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.pair);
        tma_prefetch_desc(&maps.group);
    }
    if (warp == kSoftWarps + 1) tmem_alloc<512>(smem_u32(&sh.tmem));
    pdl_wait();
    plan(a, sh, reinterpret_cast<int64_t *>(smem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const Waiter wait{smem_u32(&sh.abort), a.err};

    if (warp == kSoftWarps) {
        // -------------------------------------------------------- loads
        if (elect_one()) {
            const uint64_t pol = policy_evict_first();
            const int box = a.box_rows, subs = kKeys / box;
            Cursor cur;
            cur.start(a, sh);
            bool more = cur.step(a);
            uint32_t tile = 0;
            uint32_t used = 0, parity = 0;   // per slot (pairs, then rotary): loaded at all; last load's phase
            bool ok = true;
            while (ok && more) {
                int z[kMaxSubs], y[kMaxSubs];
#pragma unroll
                for (int i = 0; i < kMaxSubs; ++i) {
                    if (i >= subs) break;
                    // A box past the last key repeats the tile's first: its scores are masked and
                    // its values cleared, whereas a box outside the cache would cost a request
                    // per row, all CTAs' at one place. A page that is not one reads zeros.
                    const bool none = i > 0 && i >= cur.boxes;
                    const bool bad = !none && static_cast<uint32_t>(cur.page[i]) >= static_cast<uint32_t>(a.num_pages);
                    if (bad) record_error(a.err, ERR_BAD_INDEX);
                    z[i] = none ? z[0] : bad ? static_cast<int>(a.num_pages) : cur.page[i];
                    y[i] = none ? y[0] : cur.row[i];
                }
                more = cur.step(a);
                const uint32_t turn = tile >> 1;   // earlier uses of this half of the ring
#pragma unroll
                for (int g = 0; g <= kGroups; ++g) {
                    const bool is_rope = g == kGroups;
                    const int slot = is_rope ? tile & 1 : (tile & 1) * kGroups + g;
                    const uint32_t full = smem_u32(is_rope ? &sh.rope_full[slot] : &sh.pair_full[slot]);
                    const uint32_t empty = smem_u32(is_rope ? &sh.rope_empty[slot] : &sh.pair_empty[slot]);
                    if (!wait(empty, (turn & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) { ok = false; break; }
                    mbar_arrive_expect_tx(full, is_rope ? kGroupBytes : kPairBytes);
                    const int bit = is_rope ? kPairSlots + slot : slot;
                    used |= 1u << bit;
                    parity = (parity & ~(1u << bit)) | ((turn & 1) << bit);
                    const uint32_t dst = sbase + (is_rope ? kOffRope + slot * kGroupBytes : kOffPairs + slot * kPairBytes);
                    if (subs == 1) {
                        tma_load_4d(dst, is_rope ? &maps.group : &maps.pair, full, 0, y[0], 2 * g, z[0], pol);
                    } else {
#pragma unroll
                        for (int i = 0; i < kMaxSubs; ++i) {
                            if (i >= subs) break;
                            tma_load_4d(dst + i * box * 128, &maps.group, full, 0, y[i], 2 * g, z[i], pol);
                            if (!is_rope)
                                tma_load_4d(dst + kGroupBytes + i * box * 128, &maps.group, full, 0, y[i], 2 * g + 1, z[i], pol);
                        }
                    }
                }
                ++tile;
            }
            // the ring's last loads must land before the CTA may exit
            for (int i = 0; i < kPairSlots + kRopeSlots; ++i)
                if (used >> i & 1)
                    mbar_wait_drain(smem_u32(i < kPairSlots ? &sh.pair_full[i] : &sh.rope_full[i - kPairSlots]),
                                    parity >> i & 1, a.err);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 3) {
        // -------------------------------------------------------- queries
        // Apart from the keys, which run ahead of the segment: the next segment's rows
        // replace this one's as soon as its last scores are done.
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            Walk w;
            w.start(a, sh);
            uint32_t seg = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                if (w.tiles() > 0) {
                    const uint32_t full = smem_u32(&sh.q_full);
                    if (!wait(smem_u32(&sh.q_empty), (seg & 1) ^ 1, ERR_WAIT_SMEM_EMPTY)) break;
                    // rows past the sequence keep what the buffer held: their weights are zero
                    const int r0 = w.rt * kRows, rows = min(kRows, w.s.n * a.H - r0);
                    mbar_arrive_expect_tx(full, rows * kMlaWidth * 2);
                    int t = a.by_H.div(r0), h = r0 - t * a.H;
                    for (int r = 0; r < rows; r += a.q_box) {
                        if (a.q_box == kRows) {
                            tma_load_4d(sbase, &maps.q, full, 0, h, 0, w.s.row0 + t, pol);
                        } else {
                            for (int c = 0; c < kMlaWidth / 64; ++c)
                                tma_load_4d(sbase + (c * kRows + r) * 128, &maps.q, full, 0, h, c, w.s.row0 + t, pol);
                        }
                        h += a.q_box;
                        if (h >= a.H) h = 0, ++t;
                    }
                    ++seg;
                }
                w.advance();
            }
            if (seg > 0) mbar_wait_drain(smem_u32(&sh.q_full), (seg - 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 1) {
        // -------------------------------------------------------- score MMAs
        // The two products are issued by two warps that wait apart: one thread that
        // blocked on a key tile would keep back the second product whose end lets that
        // tile be loaded, and one that polled for either would spend 100 cycles, three
        // small MMAs' time, on every test.
        if (elect_one()) {
            constexpr uint32_t id_s = idesc16(E::kFmt, kRows, kKeys);
            const uint64_t dq = sdesc_sw128(sbase), dk = sdesc_sw128(sbase + kOffPairs), dr = sdesc_sw128(sbase + kOffRope);
            Walk w;
            w.start(a, sh);
            uint32_t tile = 0, seg = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                const int n = w.tiles();
                if (n > 0) {
                    ok = wait(smem_u32(&sh.q_full), seg & 1, ERR_WAIT_TMA_FULL);
                    ++seg;
                }
                for (int j = 0; j < n && ok; ++j, ++tile) {
                    const uint32_t buf = tile & 1, ph = (tile >> 1) & 1, d = tmem + kTmemS + buf * kKeys;
                    if (!wait(smem_u32(&sh.s_empty[buf]), ph ^ 1, ERR_WAIT_PART_EMPTY)) { ok = false; break; }
#pragma unroll
                    for (int g = 0; g <= kGroups; ++g) {
                        const bool is_rope = g == kGroups;
                        if (!wait(smem_u32(is_rope ? &sh.rope_full[buf] : &sh.pair_full[buf * kGroups + g]), ph, ERR_WAIT_TMA_FULL)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t q = dq + (g * 2 * kRows * 128 >> 4);
                        const uint64_t k0 = is_rope ? dr + (buf * kGroupBytes >> 4) : dk + ((buf * kGroups + g) * kPairBytes >> 4);
#pragma unroll
                        for (int k = 0; k < (is_rope ? 4 : 8); ++k)
                            mma_16_ss(d, q + ((k >> 2) * kRows * 128 + (k & 3) * 32 >> 4),
                                      k0 + ((k >> 2) * kGroupBytes + (k & 3) * 32 >> 4), id_s, g > 0 || k > 0);
                    }
                    if (!ok) break;
                    mma_commit(smem_u32(&sh.s_full[buf]));
                    mma_commit(smem_u32(&sh.rope_empty[buf]));
                    if (j + 1 == n) mma_commit(smem_u32(&sh.q_empty));
                }
                w.advance();
            }
            mma_commit(smem_u32(&sh.mma_done[0]));
            mbar_wait_drain(smem_u32(&sh.mma_done[0]), 0, a.err);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 2) {
        // -------------------------------------------------------- weight x latent MMAs
        if (elect_one()) {
            constexpr uint32_t id_o = idesc16(E::kFmt, 128, kRows, true, false);
            const uint64_t dp = sdesc_sw128(sbase + kOffP), dv = sdesc_mn_sw128(sbase + kOffPairs, kGroupBytes);
            Walk w;
            w.start(a, sh);
            uint32_t tile = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                const int n = w.tiles();
                for (int j = 0; j < n && ok; ++j, ++tile) {
                    if (!wait(smem_u32(&sh.p_full), tile & 1, ERR_WAIT_PART_FULL)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t half = tile & 1, acc0 = j > 0;
#pragma unroll
                    for (int m = 0; m < kGroups; ++m) {
                        const uint64_t v = dv + ((half * kGroups + m) * kPairBytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_16_ss(tmem + kTmemO + m * kRows, v + (k * 2048 >> 4), dp + (k * 32 >> 4), id_o, k > 0 ? 1 : acc0);
                        mma_commit(smem_u32(&sh.pair_empty[half * kGroups + m]));
                    }
                    mma_commit(smem_u32(&sh.pv_done));
                }
                w.advance();
            }
            mma_commit(smem_u32(&sh.mma_done[1]));
            mbar_wait_drain(smem_u32(&sh.mma_done[1]), 0, a.err);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- softmax and results
        // Eight warps: warps w and w + 4 hold the same 16 rows (a warp reaches the tensor
        // memory lanes of its number modulo 4) and half of the tile's keys each, later
        // half of the latent columns each.
        const int tid = threadIdx.x, quad = warp & 3, half = warp >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        // this thread's two rows of the tile and its 8 key columns (pairs of two)
        const int ra = quad * 16 + lane / 4, rb = ra + 8;
        const int c0 = 2 * (lane & 3);
        Walk w;
        w.start(a, sh);
        uint32_t tile = 0;
        int4 join = make_int4(0, 0, 0, 0);
        // after a wait that gave up a thread waits no more but keeps to the loops, so
        // that every named barrier still gets all of its threads
        bool ok = true;
        auto hold = [&](uint64_t *bar, uint32_t parity, uint32_t bit) {
            if (ok) ok = wait(smem_u32(bar), parity, bit);
        };
        while (w.next(a)) {
            const int n = w.tiles();
            const int r0 = w.rt * kRows;
            const int rows = min(kRows, w.s.n * a.H - r0);
            const bool whole = w.k0 == 0 && w.k1 == w.kt;
            auto visible = [&](int r) {
                return r >= rows ? 0 : max(0, w.s.ctx - w.s.n + a.by_H.div(r0 + r) + 1);
            };
            const int vis_a = visible(ra), vis_b = visible(rb);
            float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f, lost_a = 0.f, lost_b = 0.f;
            for (int j = 0; j < n; ++j, ++tile) {
                const uint32_t buf = tile & 1, ph = (tile >> 1) & 1;
                hold(&sh.s_full[buf], ph, ERR_WAIT_PART_FULL);
                tc_fence_after();
                uint32_t r[16];
                tmem_ld_16x32(tmem + kTmemS + buf * kKeys + half * 32 + lane_base, r);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.s_empty[buf]));
                const int kb = (w.k0 + j) * kKeys;
                if (kb + kKeys > min(vis_a, vis_b)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = kb + half * 32 + 8 * g + c0 + e;
                            if (key >= vis_a) r[4 * g + e] = __float_as_uint(-INFINITY);
                            if (key >= vis_b) r[4 * g + 2 + e] = __float_as_uint(-INFINITY);
                        }
                }
                float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    mx_a = fmaxf(mx_a, fmaxf(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1])));
                    mx_b = fmaxf(mx_b, fmaxf(__uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3])));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
                    mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
                }
                mx_a *= a.scale_log2, mx_b *= a.scale_log2;
                const bool behind = mx_a - m_a > E::kLift + kLag || mx_b - m_b > E::kLift + kLag;
                if (named_bar_or(1, kSoftThreads, behind)) {
                    if ((lane & 3) == 0) sh.half_of[half][ra] = mx_a, sh.half_of[half][rb] = mx_b;
                    named_bar_sync(1, kSoftThreads);
                    const float na = fmaxf(m_a, fmaxf(mx_a, sh.half_of[half ^ 1][ra]) - E::kLift);
                    const float nb = fmaxf(m_b, fmaxf(mx_b, sh.half_of[half ^ 1][rb]) - E::kLift);
                    const float fa = m_a == -INFINITY ? 0.f : ex2(m_a - na), fb = m_b == -INFINITY ? 0.f : ex2(m_b - nb);
                    l_a *= fa, l_b *= fb, lost_a *= fa, lost_b *= fb;
                    m_a = na, m_b = nb;
                    if (j > 0) {
                        if (half == 0 && (lane & 3) == 0) sh.factor[ra] = fa, sh.factor[rb] = fb;
                        hold(&sh.pv_done, (tile - 1) & 1, ERR_WAIT_PART_FULL);
                        tc_fence_after();
                        named_bar_sync(1, kSoftThreads);
#pragma unroll 1
                        for (int c = half * 2 * kRows; c < (half + 1) * 2 * kRows; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(tmem + kTmemO + c + lane_base, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.factor[(c & 32) + i]);
                            tmem_st32(tmem + kTmemO + c + lane_base, o);
                        }
                        tmem_wait_st();
                    }
                }
                const float ea = m_a == -INFINITY ? 0.f : m_a, eb = m_b == -INFINITY ? 0.f : m_b;
                uint32_t pa[4], pb[4];
                float s_a = 0.f, s_b = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float a0 = ex2(fmaf(__uint_as_float(r[4 * g]), a.scale_log2, -ea));
                    const float a1 = ex2(fmaf(__uint_as_float(r[4 * g + 1]), a.scale_log2, -ea));
                    const float b0 = ex2(fmaf(__uint_as_float(r[4 * g + 2]), a.scale_log2, -eb));
                    const float b1 = ex2(fmaf(__uint_as_float(r[4 * g + 3]), a.scale_log2, -eb));
                    s_a += a0 + a1;
                    s_b += b0 + b1;
                    // the weights enter the second product in the tensors' 16-bit type:
                    // half an ulp each, averaged over the keys (fp16: down to 2^-21 of
                    // the largest, from there an absolute 2^-32 of it)
                    pa[g] = E::pack(a0, a1);
                    pb[g] = E::pack(b0, b1);
                }
                add_compensated(l_a, lost_a, s_a);
                add_compensated(l_b, lost_b, s_b);
                if (tile > 0) hold(&sh.pv_done, (tile - 1) & 1, ERR_WAIT_PART_FULL);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int u = half * 4 + g;
                    st_shared_u32(sbase + kOffP + ra * 128 + ((u ^ (ra & 7)) << 4) + c0 * 2, pa[g]);
                    st_shared_u32(sbase + kOffP + rb * 128 + ((u ^ (rb & 7)) << 4) + c0 * 2, pb[g]);
                }
                // rows past the last key hold whatever the page held: their weights are
                // zero, but zero times a NaN is not
                const int left = w.keys - kb;
                if (left < kKeys) {
                    // (a warp per group of 64 columns)
                    const uint32_t end = sbase + kOffPairs + ((tile & 1) * kSoftWarps + warp + 1) * kGroupBytes;
                    for (int i = lane; i < (kKeys - left) * 8; i += 32) st_shared_v4(end - 16 - i * 16, make_uint4(0, 0, 0, 0));
                }
                tc_fence_before();
                fence_async_smem();
                mbar_arrive(smem_u32(&sh.p_full));
            }
            // -------------------------------------------------- the segment's result
            l_a += lost_a, l_b += lost_b;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                l_a += __shfl_xor_sync(0xffffffffu, l_a, o);
                l_b += __shfl_xor_sync(0xffffffffu, l_b, o);
            }
            const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
            if ((lane & 3) == 0) sh.sum_of[half][ra] = l_a, sh.sum_of[half][rb] = l_b;
            named_bar_sync(1, kSoftThreads);   // factor and row_off are free again, too
            if ((lane & 3) == 0) {
                // the two warps of 16 rows take eight each
                const int r = half ? rb : ra;
                const float l = sh.sum_of[0][r] + sh.sum_of[1][r], m = half ? m_b : m_a;
                const int t = a.by_H.div(r0 + r), h = r0 + r - t * a.H;
                if (whole) {
                    sh.factor[r] = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
                    sh.row_off[r] = r < rows ? (w.s.row0 + t) * a.o_st + h * a.o_sh : -1;
                    if (a.lse && r < rows)
                        a.lse[static_cast<int64_t>(w.s.row0 + t) * a.H + h] =
                            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                } else if (r < rows) {
                    a.part_ml[static_cast<int64_t>(slot) * kRows + r] = make_float2(m, l);
                }
            }
            named_bar_sync(1, kSoftThreads);
            if (n > 0) {
                hold(&sh.pv_done, (tile - 1) & 1, ERR_WAIT_PART_FULL);
                tc_fence_after();
            }
            if (whole) {
                // O^T (lanes: columns of the latent; columns: rows) leaves transposed, 16
                // rows x 32 latent columns of a warp at a time, through the warp's 1 KB of
                // the weights' buffer: 16-byte stores, 64 bytes of a row per four lanes.
                // (The next weights are written behind the next tile's named barrier.)
                const uint32_t stage = sbase + kOffP + warp * 1024;
                const uint32_t st_row = lane & 7, st_chunk = lane >> 3;
                T *out = static_cast<T *>(a.out) + quad * 32 + (lane & 3) * 8;
#pragma unroll 1
                for (int c = 0; c < 2 * kRows; c += 32) {
                    if ((c & 32) >= rows) continue;
                    uint32_t o0[16], o1[16];
                    if (n > 0) {
                        const uint32_t src = tmem + kTmemO + half * 2 * kRows + c + lane_base;
                        tmem_ld_16x32(src, o0);
                        tmem_ld_16x32(src + (16u << 16), o1);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o0[i] = o1[i] = 0;
                    }
                    T *dst = out + (half * 2 + c / kRows) * 128;
#pragma unroll
                    for (int g0 = 0; g0 < 4; g0 += 2) {
                        const int rbase = (c & 32) + 8 * g0;
                        __syncwarp();   // the last 16 rows have been read
#pragma unroll
                        for (int g = g0; g < g0 + 2; ++g) {
                            const float2 f = *reinterpret_cast<const float2 *>(&sh.factor[(c & 32) + 8 * g + c0]);
                            auto two = [&](const uint32_t *o) {
                                return E::pack(__uint_as_float(o[0]) * f.x, __uint_as_float(o[1]) * f.y);
                            };
                            // rows of 64 bytes; the 16-byte unit is swizzled by the row pair
                            stmatrix_x4_trans(stage + (8 * (g - g0) + st_row) * 64 + ((st_chunk ^ (st_row >> 1)) << 4),
                                              two(o0 + 4 * g), two(o0 + 4 * g + 2), two(o1 + 4 * g), two(o1 + 4 * g + 2));
                        }
                        __syncwarp();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const int r = 8 * g + (lane >> 2);
                            const int64_t off = sh.row_off[rbase + r];
                            const uint4 v = ld_shared_v4(stage + r * 64 + (((lane & 3) ^ ((r & 7) >> 1)) << 4));
                            if (off >= 0) *reinterpret_cast<uint4 *>(dst + off) = v;
                        }
                    }
                }
            } else {
                float *part = a.part_o + static_cast<int64_t>(slot) * kRows * kMlaLatent + quad * 32 + lane;
#pragma unroll 1
                for (int c = 0; c < 2 * kRows; c += 32) {
                    if ((c & 32) >= rows) continue;
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(tmem + kTmemO + half * 2 * kRows + c + lane_base, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
                    const int rbase = c & 32;
                    float *dst = part + rbase * kMlaLatent + (half * 2 + c / kRows) * 128;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (rbase + i < rows) dst[i * kMlaLatent] = __uint_as_float(o[i]);
                }
            }
            tc_fence_before();
            if (!whole && w.k0 == 0) {
                // this CTA holds the item's first key tiles: it names the item to the join
                const int c_end = part_of(sh.each, sh.rem, w.at + (w.kt - 1));
                join = make_int4(w.s.row0, r0, rows, c_end);
            }
            w.advance();
        }
        if (tid == 0) a.joins[blockIdx.x] = join;
    }
    __syncthreads();
    if (warp == kSoftWarps + 1) tmem_dealloc<512>(tmem);
}

// Joins the partial results of the items that several CTAs shared: row by row
//   M = max m_s,  O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s
// over the item's parts in order. joins[c] = (the sequence's first query, first row of
// the tile, rows, last CTA) of the item whose first part CTA c holds (rows 0: none).
// A large batch has two parts of each of 10,000 rows, a single long sequence up to 150 of
// each of 64. More than kFewRows rows: a warp takes a whole row of up to 32 parts (33
// sequences' 64 rows of 6 to 10 parts 14 -> 9 us). Fewer, or rows of more parts: a CTA takes
// a row, or half of one. (128 rows of 16 parts 13.2 us a call, with a warp each 16.8; 320
// rows of 11 parts 18.4 and 16.3, of 25 parts 19.6 and 21.4. Both kinds in one call cost
// the sum: 12 sequences of 16 heads and 5 to 11 parts 16.5, either kind 15.)
// Two CTAs of 256 threads per SM with 128 registers each: with 512 threads the 64 registers
// spilled (33 sequences 42.1 -> 38.0 us, one of 1,000 tokens 16.9 -> 13.5); one CTA of 512
// had to take 150 to 300 rows in two turns (4 x 1,000 tokens 16.6 -> 14.9 us).
constexpr int kJoinThreads = 256;
constexpr int kMaxCtas = 256;
constexpr int kFewRows = 300;
constexpr int kAhead = 16;   // parts whose sums are on their way together

// Sum of parts [s0, s1) of a row for four columns, relative to their largest reference
// maximum M, and the sum L of their exponentials (s1 - s0 <= 128).
template <typename SlotOf>
__device__ __forceinline__ float4 join_parts(const PagedArgs &a, SlotOf slot_of, int s0, int s1, int col, float &M, float &L) {
    const int lane = threadIdx.x & 31;
    float4 v[kAhead];
    // the first sums are on their way while the weights are formed
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (s0 + k < s1) v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot_of(s0 + k) * kMlaLatent + col));
    static_assert(kMaxCtas <= 2 * 128, "two shares of an item's parts");
    float2 ml[4];
    M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        ml[k] = s0 + 32 * k + lane < s1 ? a.part_ml[slot_of(s0 + 32 * k + lane)] : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // a part without visible keys has weight zero and sums of zero
        ml[k].x = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
        L += ml[k].x * ml[k].y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < s1 - s0; k0 += kAhead) {
        const float w = k0 < 32 ? ml[0].x : k0 < 64 ? ml[1].x : k0 < 96 ? ml[2].x : ml[3].x;   // (kAhead divides 32)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s0 + k0 + k < s1) {
                const float f = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                acc.x += f * v[k].x, acc.y += f * v[k].y, acc.z += f * v[k].z, acc.w += f * v[k].w;
                if (s0 + k0 + kAhead + k < s1)
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot_of(s0 + k0 + kAhead + k) * kMlaLatent + col));
            }
        }
    }
    return acc;
}

template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 2) paged_join_kernel(const PagedArgs a, int ctas) {
    // rows before join c, of the joins of few parts and of many
    __shared__ int s_rows[2][kMaxCtas + 1];
    __shared__ unsigned s_sum[kMaxCtas / 32];
    __shared__ int4 s_join[kMaxCtas];
    __shared__ float4 s_acc[kJoinThreads / 32 - 1][32];
    __shared__ float2 s_ml[kJoinThreads / 32];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    static_assert(kJoinThreads == kMaxCtas && kMaxCtas * kRows < 1 << 16, "a thread's join; both counts in one word");
    {
        const int4 j = tid < ctas ? a.joins[tid] : make_int4(0, 0, 0, 0);
        s_join[tid] = j;
        const int joins = __syncthreads_count(j.z > 0);
        if (joins == 0) return;
        const bool many = j.w - tid + 1 > (joins > a.few_joins ? 32 : 0);
        unsigned inc = static_cast<unsigned>(j.z) << (many ? 16 : 0);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        for (int i = 0; i < warp; ++i) inc += s_sum[i];
        s_rows[0][tid + 1] = inc & 0xffff, s_rows[1][tid + 1] = inc >> 16;
        if (tid == 0) s_rows[0][0] = s_rows[1][0] = 0;
    }
    __syncthreads();
    auto find = [&](int kind, int i) {   // the join with s_rows[c] <= i < s_rows[c + 1]
        int lo = 0, hi = kMaxCtas;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (s_rows[kind][mid] <= i ? lo : hi) = mid;
        }
        return lo;
    };
    auto store = [&](const int4 &j, int r, int col, float4 acc, float M, float L) {
        const float inv = L > 0.f ? 1.0f / L : (L == 0.f ? 0.f : L);
        const int t = a.by_H.div(j.y + r), h = j.y + r - t * a.H;
        const int64_t q = j.x + t;
        T *dst = static_cast<T *>(a.out) + q * a.o_st + h * a.o_sh + col;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(Elem<T>::pack(acc.x * inv, acc.y * inv), Elem<T>::pack(acc.z * inv, acc.w * inv));
        if (a.lse && col == 0) a.lse[q * a.H + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    };
    for (int i = (kJoinThreads / 32) * blockIdx.x + warp; i < s_rows[0][kMaxCtas]; i += (kJoinThreads / 32) * gridDim.x) {
        const int c = find(0, i), r = i - s_rows[0][c];
        const int4 j = s_join[c];
        const int parts = j.w - c + 1;
        auto slot_of = [&](int s) { return static_cast<int64_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)) * kRows + r; };
        auto sums_of = [&](int s, int k) {
            return __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot_of(s) * kMlaLatent + k * 128 + lane * 4));
        };
        float4 v[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[s][k] = sums_of(s, k);
        const float2 ml = lane < parts ? a.part_ml[slot_of(lane)] : make_float2(-INFINITY, 0.f);
        float M = ml.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        M = __shfl_sync(0xffffffffu, M, 0);
        // a part without visible keys has weight zero and sums of zero
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        float L = w * ml.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        L = __shfl_sync(0xffffffffu, L, 0);
        float4 acc[4] = {};
        for (int s0 = 0; s0 < parts; s0 += 2)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s0 + s >= parts) break;
                const float f = __shfl_sync(0xffffffffu, w, s0 + s);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[k].x += f * v[s][k].x, acc[k].y += f * v[s][k].y, acc[k].z += f * v[s][k].z, acc[k].w += f * v[s][k].w;
                    if (s0 + s + 2 < parts) v[s][k] = sums_of(s0 + s + 2, k);
                }
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) store(j, r, k * 128 + lane * 4, acc[k], M, L);
    }
    // Rows of many parts: a CTA takes all of a row's columns in four slices, the parts in
    // two shares, or, if there are CTAs enough, half of the columns and four shares, or a
    // quarter and eight (one sequence of 20,000 tokens, 152 parts: 20.1 us with eight shares,
    // 25.0 with four).
    const int rows = s_rows[1][kMaxCtas], ctas_free = gridDim.x;
    const int split = 4 * rows <= ctas_free ? 2 : 2 * rows <= ctas_free ? 1 : 0;
    const int slices = 4 >> split, shares = 2 << split, slice = warp & (slices - 1), grp = warp >> (2 - split);
    for (int i = blockIdx.x; i < rows << split; i += gridDim.x) {
        const int row = i >> split, col = ((i & ((1 << split) - 1)) * slices + slice) * 128 + lane * 4;
        const int c = find(1, row), r = row - s_rows[1][c];
        const int4 j = s_join[c];
        const int parts = j.w - c + 1, per = (parts + shares - 1) >> (1 + split);
        auto slot_of = [&](int s) { return static_cast<int64_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)) * kRows + r; };
        float M, L;
        float4 acc = join_parts(a, slot_of, min(parts, grp * per), min(parts, (grp + 1) * per), col, M, L);
        __syncthreads();   // the last row's sums have been read
        if (grp > 0) s_acc[warp - slices][lane] = acc;
        if (slice == 0 && lane == 0) s_ml[grp] = make_float2(M, L);
        __syncthreads();
        if (grp == 0) {
            float m = M;
            for (int g = 1; g < shares; ++g) m = fmaxf(m, s_ml[g].x);
            float f = M == -INFINITY ? 0.f : ex2(M - m);
            L *= f;
            acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll 1
            for (int g = 1; g < shares; ++g) {
                f = s_ml[g].x == -INFINITY ? 0.f : ex2(s_ml[g].x - m);
                L += f * s_ml[g].y;
                const float4 x = s_acc[(g - 1) * slices + slice][lane];
                acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
            }
            store(j, r, col, acc, m, L);
        }
    }
}

template <typename T>
cudaError_t launch_t(const PagedMaps &m, const PagedArgs &a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(paged_attn_kernel<T>, kSmem, done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(paged_attn_kernel<T>, dim3(grid), dim3(kThreads), kSmem, stream, m, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_join_kernel<T>, dim3(2 * grid), dim3(kJoinThreads), 0, stream, a, grid);
}

}  // namespace

cudaError_t launch_paged(const PagedMaps &m, const PagedArgs &a, bool bf16, int grid, cudaStream_t stream) {
    if (grid > kMaxCtas) return cudaErrorInvalidValue;
    PagedArgs args = a;
    args.by_H = Divisor(a.H), args.by_page = Divisor(a.page_size);
    const int64_t item_rows = std::min<int64_t>(kRows, (a.Tq * a.H + a.B - 1) / a.B);
    args.few_joins = static_cast<int>(kFewRows / std::max<int64_t>(item_rows, 1));
    return bf16 ? launch_t<__nv_bfloat16>(m, args, grid, stream) : launch_t<__half>(m, args, grid, stream);
}

}  // namespace moe
