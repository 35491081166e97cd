// cache_write_kernel / cache_read_kernel: states into and out of a cache that
// holds them in 8 or 4 bits.
//
// Groups of 32 consecutive values along dv share one bf16 scale,
//     scale = bf16(fp32(max|x| / m)), m = 127 or 7,   code = nearest(x / scale),
// ties to even by the exact quotient, and the value held is code * scale.
// Eight lanes hold a group (4 values, one 16-byte load each); its largest
// magnitude is taken on the bit patterns, so a NaN or an infinity wins.
//
// The exact quotient without a division per value: q = rint(x * (1 / scale)) is
// off by at most one, and r = x - q scale is exact in one fused multiply-add
// (|r| is about scale at most, and both products' last bits lie above 2^-32 of
// it), so |r| against scale / 2 decides, and a tie goes to the even code.
//
// What bounds them: the bytes, 4 + bits/8 + 1/16 a value, one pass.  537 MB of
// state at 8 bits: save 113 us, restore 114 us (floor 104 us at the measured copy
// rate); at 4 bits 111 and 102 us (floor 93 us), the save's integer work then
// being next.  A CTA takes up to four chunks and fetches one ahead: one chunk a
// CTA spent its time on the slot's latency (147 us each way).
#include "ss_common.cuh"
#include "ss_many.h"

namespace ss {
namespace {

constexpr int CT = 256;                    // threads of a CTA
constexpr int CI = 4;                      // 16-byte pieces of the state a thread takes at a time
constexpr int CHUNK = CT * CI * 4;         // values a CTA takes at a time: n is a multiple of 64 * 64 = CHUNK
constexpr int TAKE = 4;                    // and so many of them

// The slot of sequence b, or -1 where the sequence takes no part.
__device__ __forceinline__ int slot_of(const CacheParams& p, int b, bool first) {
    const int s = p.slot[b];
    if (s >= p.slots) {
        if (first && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, SS_DEVICE_BAD_SLOT);
        return -1;
    }
    return s < 0 ? -1 : s;
}

// Nearest code (ties to even by the exact quotient) of x for a scale > 0, |code| <= m.
__device__ __forceinline__ int code_of(float x, float scale, float inv, float m) {
    float q = rintf(x * inv);
    q = fminf(fmaxf(q, -m), m);
    const float r = fmaf(-q, scale, x);
    const float half = 0.5f * scale, ar = fabsf(r);
    const float step = copysignf(1.f, r);
    const bool odd = __float2int_rn(q) & 1;
    if (ar > half || (ar == half && odd)) q += step;
    return __float2int_rn(fminf(fmaxf(q, -m), m));
}

// Codes of four values of one group whose largest magnitude has the bits `a`,
// the low bits of c; returns the scale.
template <int BITS>
__device__ __forceinline__ uint16_t quantise4(const float (&f)[4], unsigned a, unsigned (&c)[4]) {
    constexpr float M = BITS == 8 ? 127.f : 7.f;
    constexpr float MAGIC = 12582912.f;                    // 1.5 * 2^23: x + MAGIC holds rint(x) in its low bits
    const bool finite = a < 0x7f800000u;
    // top / M rounded to fp32: one step of correction after the product with
    // 1 / M, right for all 2^23 mantissas (tried one by one) wherever the
    // remainder, 2^-24 of top, is a normal number
    const float top = __uint_as_float(a);
    float d = top * (1.f / M);
    d = fmaf(fmaf(-d, M, top), 1.f / M, d);
    if (top < 7.9e-31f) d = __fdiv_rn(top, M);
    const uint16_t sb = finite ? f2bf(d) : uint16_t(0x7fc0);
    const float scale = bf2f(sb);
    float inv;                                             // within two units in the last place
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = fmaf(f[e], inv, MAGIC);
        worst = fmaxf(worst, fabsf(fmaf(MAGIC - t, scale, f[e])));
        c[e] = __float_as_uint(t);
    }
    // Next to a border between two codes (the product with 1 / scale is off by
    // less than 2^-16), and for a scale that is subnormal, zero or no number,
    // each value is looked at again.
    if (!(worst <= 0.49998f * scale) || !(scale >= 1.2e-38f)) {
        // 1 / scale would overflow for a subnormal scale: there both are raised by 2^64, which is exact
        const float up = scale < 1.2e-38f ? 18446744073709551616.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c[e] = finite && scale > 0.f ? unsigned(code_of(f[e] * up, scale * up, __frcp_rn(scale * up), M)) : 0u;
    }
    return sb;
}

template <int BITS>
__global__ void __launch_bounds__(CT) cache_write_kernel(const __grid_constant__ CacheParams p, int per, int take) {
    const int b = int(blockIdx.x / unsigned(per));
    const int c0 = int(blockIdx.x % unsigned(per)) * take;
    griddep_wait();
    griddep_launch_next();
    const float4* src = reinterpret_cast<const float4*>(p.state + b * p.n + (long long)c0 * CHUNK) + threadIdx.x;
    float4 x[CI];
#pragma unroll
    for (int i = 0; i < CI; ++i) x[i] = __ldcs(src + i * CT);
    const int slot = slot_of(p, b, c0 == 0);
    if (slot < 0) return;
    // the last of the sequences that name this slot keeps it
    bool later = false;
    for (int i = b + 1 + int(threadIdx.x); i < p.B; i += CT) later |= p.slot[i] == slot;
    if (__syncthreads_or(later)) return;
    long long v = slot * p.n + (long long)c0 * CHUNK + threadIdx.x * 4;
    for (int k = 0; k < take; ++k) {
        float4 y[CI];
        const bool more = k + 1 < take;
        src += CI * CT;
#pragma unroll
        for (int i = 0; i < CI; ++i)
            if (more) y[i] = __ldcs(src + i * CT);
#pragma unroll
        for (int i = 0; i < CI; ++i) {
            const float f[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            unsigned a = 0, c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) a = max(a, __float_as_uint(f[e]) & 0x7fffffffu);
#pragma unroll
            for (int m = 4; m >= 1; m >>= 1) a = max(a, __shfl_xor_sync(FULL, a, m));
            const uint16_t sb = quantise4<BITS>(f, a, c);
            if (BITS == 8) {
                const unsigned w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
                *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(p.codes) + v) = w;
            } else {
                unsigned w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410) & 0x0f0f0f0fu;
                w = (w | (w >> 4));                        // bytes 0 and 2: codes 1 | 0 and 3 | 2
                w = (w & 0xffu) | ((w >> 8) & 0xff00u);
                *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.codes) + v / 2) = uint16_t(w);
            }
            if ((threadIdx.x & 7) == 0) p.scales[v / 32] = sb;
            v += CT * 4;
        }
#pragma unroll
        for (int i = 0; i < CI; ++i) x[i] = y[i];
    }
}

template <int BITS>
__global__ void __launch_bounds__(CT) cache_read_kernel(const __grid_constant__ CacheParams p, int per, int take) {
    const int b = int(blockIdx.x / unsigned(per));
    const int c0 = int(blockIdx.x % unsigned(per)) * take;
    griddep_wait();
    griddep_launch_next();
    const int slot = slot_of(p, b, c0 == 0);
    if (slot < 0) return;
    long long v = slot * p.n + (long long)c0 * CHUNK + threadIdx.x * 4;
    float4* dst = reinterpret_cast<float4*>(p.state + b * p.n + (long long)c0 * CHUNK) + threadIdx.x;
    unsigned w[CI];
    uint16_t sc[CI];
    auto fetch = [&](unsigned (&w)[CI], uint16_t (&sc)[CI]) {
#pragma unroll
        for (int i = 0; i < CI; ++i, v += CT * 4) {
            w[i] = BITS == 8 ? *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(p.codes) + v)
                             : *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.codes) + v / 2);
            sc[i] = p.scales[v / 32];
        }
    };
    fetch(w, sc);
    for (int k = 0; k < take; ++k) {
        unsigned wn[CI];
        uint16_t sn[CI];
        if (k + 1 < take) fetch(wn, sn);
#pragma unroll
        for (int i = 0; i < CI; ++i) {
            float f[4];
            const float scale = bf2f(sc[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = BITS == 8 ? int(w[i] << (24 - 8 * e)) >> 24 : int(w[i] << (28 - 4 * e)) >> 28;
                f[e] = float(c) * scale;
            }
            __stcs(dst + i * CT, make_float4(f[0], f[1], f[2], f[3]));
        }
        dst += CI * CT;
#pragma unroll
        for (int i = 0; i < CI; ++i) {
            w[i] = wn[i];
            sc[i] = sn[i];
        }
    }
}

// Chunks a CTA takes: TAKE where that leaves at least two CTAs for every place
// on the device, else fewer (a power of two: n is a multiple of it).
template <typename F>
cudaError_t cache_launch(F kern, const CacheParams& p, cudaStream_t stream) {
    const long long chunks = p.n / CHUNK;
    int take = 1;
    while (take < TAKE && chunks % (2 * take) == 0 && p.B * chunks / (2 * take) >= 2LL * 8 * sm_count()) take *= 2;
    const long long ctas = p.B * (chunks / take);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(kern, dim3(unsigned(ctas)), dim3(CT), 0, stream, p, int(chunks / take), take);
}

}  // namespace

cudaError_t launch_cache_write(int bits, const CacheParams& p, cudaStream_t stream) {
    return bits == 8 ? cache_launch(cache_write_kernel<8>, p, stream) : cache_launch(cache_write_kernel<4>, p, stream);
}

cudaError_t launch_cache_read(int bits, const CacheParams& p, cudaStream_t stream) {
    return bits == 8 ? cache_launch(cache_read_kernel<8>, p, stream) : cache_launch(cache_read_kernel<4>, p, stream);
}

}  // namespace ss
