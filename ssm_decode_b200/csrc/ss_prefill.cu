// prefill_tokens_kernel: many tokens per sequence, token by token, with the
// fp32 state in registers.
//
// Per (sequence, head), for each of the sequence's tokens in order,
//     S <- M S + b k v^T,   o = S^T q,
// Mamba-2 M = a (a = exp(dt A), b = dt), GDN M = a (I - beta k k^T), KDA
// M = (I - beta k k^T) Diag(a), b = beta.  With S' = the decayed state,
//     u = b (v - S'^T k)  (Mamba-2: u = dt v),   S = S' + k u^T,
//     o = S'^T q + (k . q) u,
// so one pass over the registers gives both contractions (S'^T k and S'^T q)
// and a second one adds the update; k . q, which no state enters, is formed
// once per token for the whole CTA when the tokens are staged.
//
// Split.  State columns are independent of one another, so a warp owns 16
// columns of one head and never waits for another warp between tokens: lane
// (g, c) = (lane / 4, lane % 4) holds columns 4c .. 4c+3 of rows 4g .. 4g+3
// of every 32 (dk / 2 floats).  The eight sums of a token (4 columns, two
// contractions) are reduced over the 8 row groups by 7 shuffles that halve the
// number of values each time, and u comes back by 4.  A CTA is 64 columns of a
// head, four warps: whole heads (eight warps) left the loads, the tokens and the
// stores of fewer CTAs to overlap (GDN, 256 x 32 heads, 4 tokens: 248 us against
// 203), two warps staged k and q too often (KDA prompts 485 against 453 us).
//
// What bounds it: for a few tokens the state, read and written once (128 KB a
// head at 128 x 128); beyond about ten tokens the fp32 pipe and its issue
// slots: a state value takes one multiply (its decay) and three multiply-adds a
// token, Mamba-2's two.  256 x 32 heads, 128 x 128, bf16 out, calls back to back,
// in us by tokens: GDN 1 165, 4 195, 8 269, 16 455, 24 661, 31 819; KDA 172, 205,
// 289, 480, 690, 858 (floors 165 and 166 for one token, 195 and 210 for 24).
#include "ss_prefill.cuh"

namespace ss {
namespace {

constexpr int TOK = 16;                     // tokens staged at a time
constexpr int VC = 64;                      // state columns of a CTA

// One stage of TOK tokens (bytes): k, q rows, the CTA's columns of v, decays
// (per channel for KDA), then per token a, b and k . q.
struct TokLayout {
    int k, q, v, gate, a, b, kq, total;
};
__host__ __device__ constexpr TokLayout tok_layout(int fam, int K) {
    TokLayout L{};
    int o = 0;
    L.k = o; o += TOK * K * 2;
    L.q = o; o += TOK * K * 2;
    L.v = o; o += TOK * VC * 2;
    L.gate = o; o += fam == KDA ? TOK * K * 4 : 0;
    L.a = o; o += TOK * 4;
    L.b = o; o += TOK * 4;
    L.kq = o; o += TOK * 4;
    L.total = o;
    return L;
}

template <int FAM, int K>
__global__ void __launch_bounds__(2 * VC, K == 128 ? 4 : 6) prefill_tokens_kernel(const __grid_constant__ PrefillParams p,
                                                                              int V) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int NR = K / 8;                             // state rows of a lane
    constexpr int threads = 2 * VC;
    constexpr TokLayout L = tok_layout(FAM, K);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const unsigned splits = unsigned(V) / VC;
    const long long u = blockIdx.x / splits;
    const int col0 = int(blockIdx.x % splits) * VC;
    const int b = int(u / p.H), h = int(u % p.H);
    griddep_wait();
    int first, count;
    if (!seq_rows<true>(p, b, first, count)) return;
    const bool fresh = p.fresh != nullptr && p.fresh[b] != 0;
    if (count == 0 && !fresh) return;
    // The next launch starts early over a few tokens.  Over a prompt its CTAs would
    // settle unevenly on the SMs that fall idle first and keep those places: KDA
    // prompts of 300 to 512 tokens, calls back to back, 508 us with it, 457
    // without; 4 tokens 208 and 212.
    if (count <= TOK) griddep_launch_next();

    const int rg = lane >> 2, cg = lane & 3;
    const int wc = warp * 16 + cg * 4;                    // the lane's first column within the CTA
    float* sp = p.state + u * (long long)K * V + (long long)(rg * 4) * V + col0 + wc;
    auto row = [&](int i) { return (long long)((i >> 2) * 32 + (i & 3)) * V; };
    float2 S[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!fresh) x = __ldcs(reinterpret_cast<const float4*>(sp + row(i)));
        S[i][0] = make_float2(x.x, x.y);
        S[i][1] = make_float2(x.z, x.w);
    }

    const float A = FAM == MAMBA2 ? p.A[h] : 0.f;
    const uint16_t* gk = p.k + (long long)(h / p.group) * K;
    const uint16_t* gq = p.q + (long long)(h / p.group) * K;
    const uint16_t* gv = p.v + (long long)h * V + col0;
    const float* gg = p.gate + (FAM == KDA ? (long long)h * K : h);
    const float* gb = p.beta + h;
    // Stage tokens at .. at + n - 1 of the sequence into buffer `s`.
    auto fetch = [&](int at, int s) {
        unsigned char* sm = smem + s * L.total;
        const int n = min(TOK, count - at);
        const long long r0 = first + at;
        constexpr int KC = K / 8;                         // 16-byte pieces of a row
        for (int i = t; i < n * KC; i += threads) {
            const long long r = r0 + i / KC;
            const int c = i % KC;
            cp_async16(sm + L.k + i * 16, gk + r * p.ks + c * 8);
            cp_async16(sm + L.q + i * 16, gq + r * p.qs + c * 8);
        }
        constexpr int vc = VC / 8;
        for (int i = t; i < n * vc; i += threads)
            cp_async16(sm + L.v + i * 16, gv + (r0 + i / vc) * p.vs + (i % vc) * 8);
        if (FAM == KDA) {
            constexpr int GC = K / 4;
            for (int i = t; i < n * GC; i += threads)
                cp_async16(sm + L.gate + i * 16, gg + (r0 + i / GC) * p.gs + (i % GC) * 4);
        }
        if (t < n) {
            if (FAM != KDA) cp_async4(sm + L.a + t * 4, gg + (r0 + t) * p.gs);
            if (FAM != MAMBA2) cp_async4(sm + L.b + t * 4, gb + (r0 + t) * p.bs);
        }
        cp_async_commit();
    };

    if (count > 0) fetch(0, 0);
    for (int at = 0, s = 0; at < count; at += TOK, s ^= 1) {
        unsigned char* sm = smem + s * L.total;
        const int n = min(TOK, count - at);
        cp_async_wait_all();
        __syncthreads();                                  // this stage is in; the other one is no longer read
        if (at + TOK < count) fetch(at + TOK, s ^ 1);
        float* sa = reinterpret_cast<float*>(sm + L.a);
        float* sb = reinterpret_cast<float*>(sm + L.b);
        float* skq = reinterpret_cast<float*>(sm + L.kq);
        for (int i = warp; i < n; i += threads >> 5) {    // k . q, and Mamba-2's decay
            const uint32_t* kr = reinterpret_cast<const uint32_t*>(sm + L.k + i * K * 2);
            const uint32_t* qr = reinterpret_cast<const uint32_t*>(sm + L.q + i * K * 2);
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < K / 64; ++j) {
                const uint32_t kw = kr[lane + 32 * j], qw = qr[lane + 32 * j];
                x = fmaf(bf2f_lo(kw), bf2f_lo(qw), x);
                x = fmaf(bf2f_hi(kw), bf2f_hi(qw), x);
            }
            x = warp_sum(x);
            if (lane == 0) {
                skq[i] = x;
                if (FAM == MAMBA2) {
                    const float dt = sa[i];
                    sb[i] = dt;
                    sa[i] = expf(dt * A);
                }
            }
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const uint2* kr = reinterpret_cast<const uint2*>(sm + L.k + i * K * 2) + rg;
            const uint2* qr = reinterpret_cast<const uint2*>(sm + L.q + i * K * 2) + rg;
            const float4* ar = reinterpret_cast<const float4*>(sm + L.gate + i * K * 4) + rg;
            const float2 a2 = FAM == KDA ? dup2(1.f) : dup2(sa[i]);
            const float bt = sb[i], kq = skq[i];
            float kf[NR];
            float2 y[2] = {dup2(0.f), dup2(0.f)}, o[2] = {dup2(0.f), dup2(0.f)};
#pragma unroll
            for (int j = 0; j < NR / 4; ++j) {
                const uint2 kw = kr[j * 8], qw = qr[j * 8];
                const float qf[4] = {bf2f_lo(qw.x), bf2f_hi(qw.x), bf2f_lo(qw.y), bf2f_hi(qw.y)};
                kf[4 * j] = bf2f_lo(kw.x); kf[4 * j + 1] = bf2f_hi(kw.x);
                kf[4 * j + 2] = bf2f_lo(kw.y); kf[4 * j + 3] = bf2f_hi(kw.y);
                float4 ga = make_float4(1.f, 1.f, 1.f, 1.f);
                if (FAM == KDA) ga = ar[j * 8];
                const float gf[4] = {ga.x, ga.y, ga.z, ga.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float2& x = S[4 * j + e][c];
                        x = fmul2(x, FAM == KDA ? dup2(gf[e]) : a2);
                        if (FAM != MAMBA2) y[c] = ffma2(dup2(kf[4 * j + e]), x, y[c]);
                        o[c] = ffma2(dup2(qf[e]), x, o[c]);
                    }
                }
            }
            // Reduce over the row groups (lane bits 2-4): bit 4 picks S'^T k or
            // S'^T q, bits 3 and 2 one of the four columns.
            const bool hi = lane & 16;
            float z0, z1, z2, z3;
            {
                const float a0 = hi ? y[0].x : o[0].x, a1 = hi ? y[0].y : o[0].y, a2_ = hi ? y[1].x : o[1].x,
                            a3 = hi ? y[1].y : o[1].y;
                z0 = (hi ? o[0].x : y[0].x) + __shfl_xor_sync(FULL, a0, 16);
                z1 = (hi ? o[0].y : y[0].y) + __shfl_xor_sync(FULL, a1, 16);
                z2 = (hi ? o[1].x : y[1].x) + __shfl_xor_sync(FULL, a2_, 16);
                z3 = (hi ? o[1].y : y[1].y) + __shfl_xor_sync(FULL, a3, 16);
            }
            const bool h8 = lane & 8, h4 = lane & 4;
            const float w0 = (h8 ? z2 : z0) + __shfl_xor_sync(FULL, h8 ? z0 : z2, 8);
            const float w1 = (h8 ? z3 : z1) + __shfl_xor_sync(FULL, h8 ? z1 : z3, 8);
            const float w = (h4 ? w1 : w0) + __shfl_xor_sync(FULL, h4 ? w0 : w1, 4);
            const int ci = (h8 ? 2 : 0) + (h4 ? 1 : 0);   // the lane's column of its four
            const float vv = bf2f(reinterpret_cast<const uint16_t*>(sm + L.v)[i * VC + wc + ci]);
            const float un = bt * (FAM == MAMBA2 ? vv : vv - w);   // valid where bit 4 is clear (every lane: Mamba-2)
            float uc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) uc[c] = __shfl_sync(FULL, un, cg | ((c & 1) << 2) | ((c >> 1) << 3));
            if (hi) {
                const float mine = ci == 0 ? uc[0] : ci == 1 ? uc[1] : ci == 2 ? uc[2] : uc[3];
                const float x = fmaf(kq, mine, w);
                const long long at_o = (first + at + i) * p.os + (long long)h * V + col0 + wc + ci;
                if (p.out_bf16) static_cast<uint16_t*>(p.out)[at_o] = f2bf(x);
                else static_cast<float*>(p.out)[at_o] = x;
            }
            const float2 u0 = make_float2(uc[0], uc[1]), u1 = make_float2(uc[2], uc[3]);
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                S[j][0] = ffma2(dup2(kf[j]), u0, S[j][0]);
                S[j][1] = ffma2(dup2(kf[j]), u1, S[j][1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
        __stcs(reinterpret_cast<float4*>(sp + row(i)), make_float4(S[i][0].x, S[i][0].y, S[i][1].x, S[i][1].y));
}

template <int FAM, int K>
cudaError_t tokens_launch(const PrefillParams& p, int V, cudaStream_t stream) {
    const long long ctas = (long long)p.B * p.H * (V / VC);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(prefill_tokens_kernel<FAM, K>, dim3(unsigned(ctas)), dim3(2 * VC), 2 * tok_layout(FAM, K).total, stream,
                      p, V);
}

}  // namespace

cudaError_t launch_prefill_tokens(int family, int dk, int dv, const PrefillParams& p, cudaStream_t stream) {
    switch (family * 1000 + dk) {
        case MAMBA2 * 1000 + 64: return tokens_launch<MAMBA2, 64>(p, dv, stream);
        case MAMBA2 * 1000 + 128: return tokens_launch<MAMBA2, 128>(p, dv, stream);
        case GDN * 1000 + 64: return tokens_launch<GDN, 64>(p, dv, stream);
        case GDN * 1000 + 128: return tokens_launch<GDN, 128>(p, dv, stream);
        case KDA * 1000 + 64: return tokens_launch<KDA, 64>(p, dv, stream);
        case KDA * 1000 + 128: return tokens_launch<KDA, 128>(p, dv, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ss
