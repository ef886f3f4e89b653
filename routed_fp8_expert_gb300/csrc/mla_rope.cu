// Rotary positions, latent RMSNorm and cache append of the latent attention.
#include <cuda_runtime.h>

#include "internal.h"
#include "mla.cuh"

namespace moe {

namespace {

constexpr int kRopeThreads = 256;

// One CTA per token. With f_i the pair's frequency in turns per position,
//   (a, b) -> amplitude * (a cos - b sin, b cos + a sin),  angle = 2 pi frac(pos * f_i).
// The frequency is a 64-bit fixed-point fraction of a turn, so pos * f_i wraps modulo
// one turn in integer arithmetic: at position 2^20 the phase is off by at most 2^-36
// turns (the frequency's own rounding to 53 bits), where an fp32 product of position
// and frequency would be off by 2^-7.
// Its upper 32 bits, as a signed number of half turns, feed sincospi. All arithmetic is
// fp32, rounded once when stored.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
    __shared__ float2 s_cs[128];
    __shared__ float s_part[kRopeThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const int half = a.dim / 2;
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
    uint4 cv = make_uint4(0, 0, 0, 0), gv = cv;
    float x[8];
    if (has_c) {
        cv = *reinterpret_cast<const uint4 *>(kv + tid * 8);
        if (a.gamma) gv = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.gamma) + tid * 8);
    }
    {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&cv);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = E::unpack(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
            ss += f.x * f.x + f.y * f.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((tid & 31) == 0) s_part[tid >> 5] = ss;
    }
    __syncthreads();

    // a rotated vector: 8 interleaved elements, or 8 + 8 of the two halves
    const int nvec = a.layout == 0 ? a.dim / 8 : a.dim / 16;
    auto rotate = [&](const T *src, T *d0, T *d1, int v) {
        if (a.layout == 0) {
            const uint4 in = *reinterpret_cast<const uint4 *>(src + v * 8);
            const uint32_t *w = reinterpret_cast<const uint32_t *>(&in);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = E::unpack(w[i]);
                const float2 cs = s_cs[v * 4 + i];
                o[i] = E::pack(f.x * cs.x - f.y * cs.y, f.y * cs.x + f.x * cs.y);
            }
            const uint4 r = make_uint4(o[0], o[1], o[2], o[3]);
            if (d0) *reinterpret_cast<uint4 *>(d0 + v * 8) = r;
            if (d1) *reinterpret_cast<uint4 *>(d1 + v * 8) = r;
        } else {
            const uint4 lo = *reinterpret_cast<const uint4 *>(src + v * 8);
            const uint4 hi = *reinterpret_cast<const uint4 *>(src + half + v * 8);
            const uint32_t *wl = reinterpret_cast<const uint32_t *>(&lo), *wh = reinterpret_cast<const uint32_t *>(&hi);
            uint32_t ol[4], oh[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = E::unpack(wl[i]), q = E::unpack(wh[i]);
                const float2 c0 = s_cs[v * 8 + 2 * i], c1 = s_cs[v * 8 + 2 * i + 1];
                ol[i] = E::pack(p.x * c0.x - q.x * c0.y, p.y * c1.x - q.y * c1.y);
                oh[i] = E::pack(q.x * c0.x + p.x * c0.y, q.y * c1.x + p.y * c1.y);
            }
            const uint4 rl = make_uint4(ol[0], ol[1], ol[2], ol[3]), rh = make_uint4(oh[0], oh[1], oh[2], oh[3]);
            if (d0) {
                *reinterpret_cast<uint4 *>(d0 + v * 8) = rl;
                *reinterpret_cast<uint4 *>(d0 + half + v * 8) = rh;
            }
            if (d1) {
                *reinterpret_cast<uint4 *>(d1 + v * 8) = rl;
                *reinterpret_cast<uint4 *>(d1 + half + v * 8) = rh;
            }
        }
    };

    if (kv) {
        T *row_out = a.kv_out ? static_cast<T *>(a.kv_out) + t * a.kvo_st : nullptr;
        T *row_cache = nullptr;
        if (a.cache) {
            const int64_t slot = a.slots[t];   // negative: this token is not cached
            if (slot >= 0) {
                const int64_t page = slot / a.page_size;
                if (page < a.num_pages)
                    row_cache = static_cast<T *>(a.cache) + page * a.page_st + (slot - page * a.page_size) * a.row_st;
                else if (tid == 0)
                    record_error(a.err, ERR_BAD_INDEX);
            }
        }
        if (has_c) {
            uint32_t o[4];
            if (a.gamma) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < kRopeThreads / 32; ++i) ss += s_part[i];
                const float inv = 1.0f / sqrtf(ss / static_cast<float>(a.latent) + a.eps);
                const uint32_t *g = reinterpret_cast<const uint32_t *>(&gv);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = E::unpack(g[i]);
                    o[i] = E::pack(x[2 * i] * inv * f.x, x[2 * i + 1] * inv * f.y);
                }
            } else {
                o[0] = cv.x, o[1] = cv.y, o[2] = cv.z, o[3] = cv.w;
            }
            const uint4 r = make_uint4(o[0], o[1], o[2], o[3]);
            if (row_out) *reinterpret_cast<uint4 *>(row_out + tid * 8) = r;
            if (row_cache) *reinterpret_cast<uint4 *>(row_cache + tid * 8) = r;
        }
        // the rotary key: the last threads, which hold no part of a 512-column latent
        const int v = kRopeThreads - 1 - tid;
        if (v < nvec)
            rotate(kv + a.latent, row_out ? row_out + a.latent : nullptr, row_cache ? row_cache + a.latent : nullptr, v);
    }

    if (a.q) {
        const T *q = static_cast<const T *>(a.q) + t * a.q_st;
        T *qo = static_cast<T *>(a.q_out) + t * a.qo_st;
        for (int i = tid; i < a.H * nvec; i += kRopeThreads) {
            const int h = i / nvec, v = i - h * nvec;
            rotate(q + h * a.q_sh, qo + h * a.qo_sh, nullptr, v);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool bf16, int, cudaStream_t stream) {
    if (bf16) return launch_pdl(rope_append_kernel<__nv_bfloat16>, dim3(a.T), dim3(kRopeThreads), 0, stream, a);
    return launch_pdl(rope_append_kernel<__half>, dim3(a.T), dim3(kRopeThreads), 0, stream, a);
}

}  // namespace moe
