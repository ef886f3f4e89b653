// Rotary positions, latent RMSNorm and cache append of the latent attention.
#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

// One CTA per token. With f_i the pair's frequency in turns per position,
//   (a, b) -> amplitude * (a cos - b sin, b cos + a sin),  angle = 2 pi frac(pos * f_i).
// The frequency is a 64-bit fixed-point fraction of a turn, so pos * f_i wraps modulo
// one turn in integer arithmetic. Its upper 32 bits, as a signed number of half turns in
// fp32, feed sincospi: the angle is off by up to 2^-26 turns (24 bits of a number below
// half a turn; 2^-32 for the bits that are dropped), at every position. The frequency's
// own error, 2^-50 of it for the host's roundings in 64 bits, adds pos times that: 2^-32
// turns at position 2^20. An fp32 product of position and frequency would be off by 2^-7
// there. All arithmetic is fp32, rounded once when stored.
//
// A prompt is bound by memory, and nearly as much by the issue rate. 32 bytes per thread
// are on their way before the angles are known; what only the key's warps need is theirs
// alone, and with DIM, the rotary dimension when it is known at compile time (64, else 0),
// the divisions by a head's vectors are shifts. 32 registers and CTAs of 128 threads keep
// sixteen tokens on an SM: 8192 tokens of 64 heads 27.8 us, 5.5 TB/s (with 256 threads
// 31.3, without the two before 34.3; 27.3 for a dense copy of the queries' 134 MB alone),
// of 16 heads 11.7 (16.5). Where an SM has no more than eight tokens, 256 threads have
// each done sooner (1024 tokens of 16 heads 3.5 us, with 128 threads 4.1).
template <typename T, bool HALF, int DIM, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) rope_append_kernel(const RopeArgs a) {
    __shared__ __align__(16) float2 s_cs[128];
    __shared__ float s_part[THREADS / 32];
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const int dim = DIM ? DIM : a.dim, half = dim / 2;
    using E = Elem<T>;

    if (tid < half) {
        const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t])) * a.freq[tid];
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * (1.0f / 2147483648.0f);
        float s, c;
        sincospif(half_turns, &s, &c);
        s_cs[tid] = make_float2(c * a.amplitude, s * a.amplitude);
    }

    // the latent's vector (8 elements per thread) and its sum of squares
    const T *kv = a.kv ? static_cast<const T *>(a.kv) + t * a.kv_st : nullptr;
    const bool has_c = kv && tid < a.latent / 8;
    uint4 cv = make_uint4(0, 0, 0, 0);
    if (has_c) cv = *reinterpret_cast<const uint4 *>(kv + tid * 8);
    const int c_warps = kv ? (a.latent / 8 + 31) / 32 : 0;   // warps that hold parts of the latent
    if ((tid >> 5) < c_warps) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&cv);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = E::unpack(w[i]);
            ss += f.x * f.x + f.y * f.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((tid & 31) == 0) s_part[tid >> 5] = ss;
    }

    // a rotated vector: 8 interleaved elements, or 8 + 8 of the two halves
    const unsigned nvec = HALF ? dim / 16 : dim / 8;
    struct Pair {
        uint4 lo, hi;   // (interleaved: only lo)
    };
    constexpr int kEarly = HALF ? 1 : 2;
    auto fetch = [&](const T *src, int v) {
        Pair p;
        p.lo = *reinterpret_cast<const uint4 *>(src + v * 8);
        p.hi = HALF ? *reinterpret_cast<const uint4 *>(src + half + v * 8) : make_uint4(0, 0, 0, 0);
        return p;
    };
    auto rotate = [&](const Pair &p, T *d0, T *d1, int v) {
        const uint32_t *wl = reinterpret_cast<const uint32_t *>(&p.lo), *wh = reinterpret_cast<const uint32_t *>(&p.hi);
        uint32_t ol[4], oh[4];
        if (!HALF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = E::unpack(wl[i]), cs = s_cs[v * 4 + i];
                ol[i] = E::pack(f.x * cs.x - f.y * cs.y, f.y * cs.x + f.x * cs.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = E::unpack(wl[i]), y = E::unpack(wh[i]);
                const float4 c = *reinterpret_cast<const float4 *>(&s_cs[v * 8 + 2 * i]);   // two pairs
                ol[i] = E::pack(x.x * c.x - y.x * c.y, x.y * c.z - y.y * c.w);
                oh[i] = E::pack(y.x * c.x + x.x * c.y, y.y * c.z + x.y * c.w);
            }
        }
        const uint4 rl = make_uint4(ol[0], ol[1], ol[2], ol[3]);
        if (d0) *reinterpret_cast<uint4 *>(d0 + v * 8) = rl;
        if (d1) *reinterpret_cast<uint4 *>(d1 + v * 8) = rl;
        if (HALF) {
            const uint4 rh = make_uint4(oh[0], oh[1], oh[2], oh[3]);
            if (d0) *reinterpret_cast<uint4 *>(d0 + half + v * 8) = rh;
            if (d1) *reinterpret_cast<uint4 *>(d1 + half + v * 8) = rh;
        }
    };

    // this thread's first query vectors are on their way before the angles
    const T *q = a.q ? static_cast<const T *>(a.q) + t * a.q_st : nullptr;
    const unsigned items = a.q ? a.H * nvec : 0;
    Pair early[kEarly];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) {
        const unsigned i = tid + k * THREADS;
        if (i < items) early[k] = fetch(q + i / nvec * a.q_sh, i % nvec);
    }
    // the rotary key: the last threads, which hold no part of a 512-column latent
    const unsigned kvec = THREADS - 1 - tid;
    Pair key;
    if (kv && kvec < nvec) key = fetch(kv + a.latent, kvec);
    __syncthreads();

    if (kv && (has_c || kvec < nvec)) {
        T *row_out = a.kv_out ? static_cast<T *>(a.kv_out) + t * a.kvo_st : nullptr;
        T *row_cache = nullptr;
        if (a.cache) {
            const int slot = a.slots[t];   // negative: this token is not cached
            if (slot >= 0) {
                const unsigned page = a.by_page.div(slot);
                if (page < a.num_pages)
                    row_cache = static_cast<T *>(a.cache) + page * a.page_st + (slot - page * a.page_size) * a.row_st;
                else if (kvec == 0)
                    record_error(a.err, ERR_BAD_INDEX);
            }
        }
        if (has_c) {
            uint32_t o[4];
            if (a.gamma) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < THREADS / 32; ++i) ss += i < c_warps ? s_part[i] : 0.f;
                const float inv = 1.0f / sqrtf(ss / static_cast<float>(a.latent) + a.eps);
                const uint4 gv = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.gamma) + tid * 8);
                const uint32_t *g = reinterpret_cast<const uint32_t *>(&gv), *w = reinterpret_cast<const uint32_t *>(&cv);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = E::unpack(w[i]), f = E::unpack(g[i]);
                    o[i] = E::pack(x.x * inv * f.x, x.y * inv * f.y);
                }
            } else {
                o[0] = cv.x, o[1] = cv.y, o[2] = cv.z, o[3] = cv.w;
            }
            const uint4 r = make_uint4(o[0], o[1], o[2], o[3]);
            if (row_out) *reinterpret_cast<uint4 *>(row_out + tid * 8) = r;
            if (row_cache) *reinterpret_cast<uint4 *>(row_cache + tid * 8) = r;
        }
        if (kvec < nvec)
            rotate(key, row_out ? row_out + a.latent : nullptr, row_cache ? row_cache + a.latent : nullptr, kvec);
    }

    if (a.q) {
        T *qo = static_cast<T *>(a.q_out) + t * a.qo_st;
#pragma unroll
        for (int k = 0; k < kEarly; ++k) {
            const unsigned i = tid + k * THREADS;
            if (i < items) rotate(early[k], qo + i / nvec * a.qo_sh, nullptr, i % nvec);
        }
        for (unsigned i = tid + kEarly * THREADS; i < items; i += THREADS)
            rotate(fetch(q + i / nvec * a.q_sh, i % nvec), qo + i / nvec * a.qo_sh, nullptr, i % nvec);
    }
}

}  // namespace

template <typename T>
static cudaError_t launch_t(RopeArgs a, cudaStream_t stream) {
    a.by_page = Divisor(a.cache ? a.page_size : 1);   // (without a cache it may be anything)
    if (a.dim == 64 && a.latent <= 8 * 128 && a.T > 8 * num_sms()) {
        auto kernel = a.layout ? rope_append_kernel<T, true, 64, 128> : rope_append_kernel<T, false, 64, 128>;
        return launch_pdl(kernel, dim3(a.T), dim3(128), 0, stream, a);
    }
    auto kernel = a.dim == 64 ? (a.layout ? rope_append_kernel<T, true, 64, 256> : rope_append_kernel<T, false, 64, 256>)
                              : (a.layout ? rope_append_kernel<T, true, 0, 256> : rope_append_kernel<T, false, 0, 256>);
    return launch_pdl(kernel, dim3(a.T), dim3(256), 0, stream, a);
}

cudaError_t launch_rope(const RopeArgs &a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<__half>(a, stream);
}

}  // namespace moe
