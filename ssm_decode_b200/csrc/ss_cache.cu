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
// What bounds them: the bytes, 4 + bits/8 + 1/16 a value, one pass.
#include "ss_common.cuh"

namespace ss {
namespace {

constexpr int CT = 256;                    // threads of a CTA
constexpr int CI = 4;                      // 16-byte pieces of the state per thread
constexpr int CHUNK = CT * CI * 4;         // values a CTA takes: n is a multiple of 64 * 64 = CHUNK

// The slot of sequence b, or -1 where the sequence takes no part.
__device__ __forceinline__ int slot_of(const CacheParams& p, int b) {
    const int s = p.slot[b];
    if (s >= p.slots) {
        if (blockIdx.x % unsigned(p.n / CHUNK) == 0 && threadIdx.x == 0 && p.status != nullptr)
            atomicOr(p.status, SS_DEVICE_BAD_SLOT);
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

template <int BITS>
__global__ void __launch_bounds__(CT) cache_write_kernel(const __grid_constant__ CacheParams p) {
    const unsigned per = unsigned(p.n / CHUNK);
    const int b = int(blockIdx.x / per);
    const long long base = (long long)(blockIdx.x % per) * CHUNK;
    griddep_wait();
    griddep_launch_next();
    const int slot = slot_of(p, b);
    if (slot < 0) return;
    // the last of the sequences that name this slot keeps it
    bool later = false;
    for (int i = b + 1 + int(threadIdx.x); i < p.B; i += CT) later |= p.slot[i] == slot;
    if (__syncthreads_or(later)) return;
    const float4* src = reinterpret_cast<const float4*>(p.state + b * p.n + base) + threadIdx.x;
    const long long dst = slot * p.n + base;
    constexpr float M = BITS == 8 ? 127.f : 7.f;
    float4 x[CI];
#pragma unroll
    for (int i = 0; i < CI; ++i) x[i] = __ldcs(src + i * CT);
#pragma unroll
    for (int i = 0; i < CI; ++i) {
        const float f[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        unsigned a = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) a = max(a, __float_as_uint(f[e]) & 0x7fffffffu);
#pragma unroll
        for (int m = 4; m >= 1; m >>= 1) a = max(a, __shfl_xor_sync(FULL, a, m));
        const bool finite = a < 0x7f800000u;
        const uint16_t sb = finite ? f2bf(__fdiv_rn(__uint_as_float(a), M)) : uint16_t(0x7fc0);
        const float scale = bf2f(sb);
        int c[4] = {0, 0, 0, 0};
        if (finite && scale > 0.f) {
            // 1 / scale would overflow for a subnormal scale: there both are raised by 2^64, which is exact
            const float up = scale < 1.2e-38f ? 18446744073709551616.f : 1.f;
            const float inv = __frcp_rn(scale * up);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = code_of(f[e] * up, scale * up, inv, M);
        }
        const long long v = dst + (long long)(threadIdx.x + i * CT) * 4;
        if (BITS == 8) {
            const unsigned w = (c[0] & 255) | ((c[1] & 255) << 8) | ((c[2] & 255) << 16) | (unsigned(c[3]) << 24);
            *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(p.codes) + v) = w;
        } else {
            const unsigned w = (c[0] & 15) | ((c[1] & 15) << 4) | ((c[2] & 15) << 8) | ((c[3] & 15) << 12);
            *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.codes) + v / 2) = uint16_t(w);
        }
        if ((threadIdx.x & 7) == 0) p.scales[v / 32] = sb;
    }
}

template <int BITS>
__global__ void __launch_bounds__(CT) cache_read_kernel(const __grid_constant__ CacheParams p) {
    const unsigned per = unsigned(p.n / CHUNK);
    const int b = int(blockIdx.x / per);
    const long long base = (long long)(blockIdx.x % per) * CHUNK;
    griddep_wait();
    griddep_launch_next();
    const int slot = slot_of(p, b);
    if (slot < 0) return;
    const long long src = slot * p.n + base;
    float4* dst = reinterpret_cast<float4*>(p.state + b * p.n + base) + threadIdx.x;
    unsigned w[CI];
    float scale[CI];
#pragma unroll
    for (int i = 0; i < CI; ++i) {
        const long long v = src + (long long)(threadIdx.x + i * CT) * 4;
        w[i] = BITS == 8 ? *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(p.codes) + v)
                         : *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.codes) + v / 2);
        scale[i] = bf2f(p.scales[v / 32]);
    }
#pragma unroll
    for (int i = 0; i < CI; ++i) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = BITS == 8 ? int(w[i] << (24 - 8 * e)) >> 24 : int(w[i] << (28 - 4 * e)) >> 28;
            f[e] = float(c) * scale[i];
        }
        __stcs(dst + i * CT, make_float4(f[0], f[1], f[2], f[3]));
    }
}

template <typename F>
cudaError_t cache_launch(F kern, const CacheParams& p, cudaStream_t stream) {
    const long long ctas = p.B * (p.n / CHUNK);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(kern, dim3(unsigned(ctas)), dim3(CT), 0, stream, p);
}

}  // namespace

cudaError_t launch_cache_write(int bits, const CacheParams& p, cudaStream_t stream) {
    return bits == 8 ? cache_launch(cache_write_kernel<8>, p, stream) : cache_launch(cache_write_kernel<4>, p, stream);
}

cudaError_t launch_cache_read(int bits, const CacheParams& p, cudaStream_t stream) {
    return bits == 8 ? cache_launch(cache_read_kernel<8>, p, stream) : cache_launch(cache_read_kernel<4>, p, stream);
}

}  // namespace ss
