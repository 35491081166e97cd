// prefill_chunks_kernel: prompts through the Mamba-2 and GDN recurrences in
// chunks of 64 tokens on the fifth-generation tensor cores.
//
// Chunked gated delta rule.  Within a chunk, with D_ij = a_{j+1} ... a_i (1 for
// j = i), g_i = a_0 ... a_i, t_j = a_{j+1} ... a_63 and S the state before it,
//     A_ij = b_i D_ij (k_i . k_j) for j < i,     R_i = b_i (v_i - g_i S^T k_i),
//     U = (I + A)^-1 R,
//     o_i = g_i S^T q_i + sum_{j<=i} D_ij (q_i . k_j) u_j,
//     S  <- g_63 S + sum_j k_j (t_j u_j)^T.
// Mamba-2 has no erase term: A = 0, u_i = dt_i v_i.  With P_ij = D_ij (q_i . k_j),
// U = T R and P U = (P T) R for T = (I + A)^-1, so once S^T k is known one
// product with the stacked [P T; T] gives the outputs' part and U together.
// Decays are products of the given a, never ratios or exponentials of sums:
// an a of 0 or a product that underflows needs no care.
//
// Everything that meets the state lives transposed, state column v = TMEM lane:
//     D1  = S^T [Q; K]^T              128 x 128, K = dk     (A = S^T in TMEM)
//     X   = R^T [P T; T]^T            128 x 128, K = 64     (A = R^T in TMEM)
//     X   = (t o U)^T K               128 x dk,  K = 64     (A in TMEM, K rows MN-major)
//     G   = [Q; K] K^T                128 x 64,  K = dk     (both from shared memory)
// so the B operands are the token rows as they lie in memory, and A operands
// are written by the threads that own a state column.
//
// fp32 arithmetic from bf16 operands.  q and k are bf16 already.  An fp32
// operand is cut into three bf16 parts of eight bits each, x = x0 + x1 + x2
// exactly; against an exact operand that is three products, between two cut
// ones (R with [P T; T]) the six with i + j <= 2, whose dropped rest is below
// 2^-21 of a product.  Accumulators, the state, the decays and the inverse are
// fp32; out is rounded once.
//
// Work split: one CTA per (sequence, head), one per SM (all of TMEM).
//   8 worker warps   hold S in registers, two threads a state column, half of
//                    the dk rows each; they make the A operands and the output;
//   4 staging warps  run a chunk ahead: bring q, k, v (cp.async into the
//                    tensor cores' swizzle, zeros behind the last token), the
//                    Gram products G, then solve X (I + A) = [P; I] from the
//                    last column back, one row of [P T; T] a thread;
//   1 issuing warp   one lane issues the state's MMAs.
// Roles are paced by mbarriers only.  Every wait is bounded: when one runs out
// the kernel sets SS_DEVICE_TIMEOUT, waits (bounded) for its MMAs in flight,
// releases its tensor memory and returns.
#include "ss_tc.cuh"

namespace ss {
namespace {

constexpr int C = 64;                    // tokens a chunk
constexpr int NP = 3;                    // bf16 parts of an fp32 operand
constexpr int NWK = 256;                 // worker threads
constexpr int NST = 128;                 // staging threads
constexpr int NT = NWK + NST + 32;
constexpr int AP = C + 4;                // row pitch of A (floats): float4 rows without bank conflicts

// TMEM columns (all 512).
constexpr uint32_t T_X = 0;              // [P T; T] R: outputs' part, U; then the state's update (128)
constexpr uint32_t T_SP = 128;           // S^T in parts (dk / 2 columns each); then R and t o U in parts (32 each)
constexpr uint32_t T_RP = T_SP, T_UP = T_SP + 32 * NP;
constexpr uint32_t T_D1 = 320;           // S^T q (64), S^T k (64); Mamba-2: the outputs' part in place of S^T k
constexpr uint32_t T_G = 448;            // Gram products (64)
static_assert(T_SP + 64 * NP <= T_D1 && T_UP + 32 * NP <= T_D1, "operand parts overlap D1");

struct PfLayout {
    int qk[2], tp[2], v[2], a, vec[2], bars, total;
};
// Floats of vec: decays a, b, g, t of the chunk's tokens.
__host__ __device__ constexpr PfLayout pf_layout(int K, int V) {
    PfLayout L{};
    int o = 0;
    for (int s = 0; s < 2; ++s) { L.qk[s] = o; o += 2 * C * K * 2; }          // q rows, k rows: dk / 64 blocks of 128 rows
    for (int s = 0; s < 2; ++s) { L.tp[s] = o; o += NP * 2 * C * C * 2; }     // [P T; T], a 128-row block per part
    for (int s = 0; s < 2; ++s) { L.v[s] = o; o += C * V * 2; }
    L.a = o; o += C * AP * 4;
    for (int s = 0; s < 2; ++s) { L.vec[s] = o; o += 4 * C * 4; }
    L.bars = o; o += 128;
    L.total = o + 1024;
    return L;
}

// 16 bytes global -> shared, or zeros (nothing is read) where !live.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void st_bar() { asm volatile("bar.sync 2, 128;\n" ::: "memory"); }    // staging threads

// x0, x1 cut into parts, packed two to a register (x0 in the low half).  The
// first parts are the leading 16 bits of what is left (8 significant ones), so
// every difference is exact, and so is the last part.
__device__ __forceinline__ void cut(float x0, float x1, uint32_t (&w)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
        w[i] = __byte_perm(b0, b1, 0x7632);
        x0 -= __uint_as_float(b0 & 0xffff0000u);
        x1 -= __uint_as_float(b1 & 0xffff0000u);
    }
}

// N (a multiple of 32) fp32 values of this thread's lane cut into parts and
// stored as columns of NP A operands: `base` is the first part's column for
// the thread's first value, parts `pitch` columns apart.
template <int N>
__device__ __forceinline__ void put_parts(uint32_t base, uint32_t pitch, const float* x) {
#pragma unroll
    for (int k = 0; k < N; k += 32) {
        uint32_t w[NP][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            uint32_t c[NP];
            cut(x[k + 2 * i], x[k + 2 * i + 1], c);
#pragma unroll
            for (int p = 0; p < NP; ++p) w[p][i] = c[p];
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) tc::st16(base + p * pitch + k / 2, w[p]);
    }
}

// N columns (a multiple of 16) of this thread's lane; the caller waits.
template <int N>
__device__ __forceinline__ void get(uint32_t a, uint32_t* r) {
#pragma unroll
    for (int k = 0; k < N; k += 16) {
        uint32_t(&x)[16] = *reinterpret_cast<uint32_t(*)[16]>(r + k);
        tc::ld16(a + k, x);
    }
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned phase) {
    return __all_sync(FULL, mbar_wait(bar, phase));
}

template <int FAM, int K, int V>
__global__ void __launch_bounds__(NT, 1) prefill_chunks_kernel(const __grid_constant__ PrefillParams p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr PfLayout L = pf_layout(K, V);
    constexpr int NA = 2 * V;                                  // worker threads with a state column
    constexpr bool ERASE = FAM == GDN;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const long long u = blockIdx.x;
    const int b = int(u / p.H), h = int(u % p.H);
    griddep_wait();
    griddep_launch_next();
    const int first = p.seq_start[b], end = p.seq_start[b + 1];
    if (first < 0 || end < first || end > p.rows) {
        if (t == 0 && p.status != nullptr) atomicOr(p.status, SS_DEVICE_BAD_ROWS);
        return;
    }
    const int count = end - first;
    const bool fresh = p.fresh != nullptr && p.fresh[b] != 0;
    float* const state = p.state + u * (long long)(K * V);
    if (count == 0) {
        if (fresh)
            for (int i = t; i < K * V / 4; i += NT) reinterpret_cast<float4*>(state)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const int chunks = (count + C - 1) / C;

    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L.bars);
    uint64_t* full = bars + 0;                                 // [2] q, k rows staged
    uint64_t* ready = bars + 2;                                // [2] [P T; T], v and the decays staged
    uint64_t* freed = bars + 4;                                // [2] the stage is no longer read (workers, last MMA)
    uint64_t* gbar = bars + 6;                                 // Gram products done
    uint64_t* sbar = bars + 7;                                 // S^T's parts written (workers)
    uint64_t* rbar = bars + 8;                                 // R's parts written (workers)
    uint64_t* ubar = bars + 9;                                 // t o U's parts written (workers)
    uint64_t* d1bar = bars + 10;                               // D1 done
    uint64_t* d2bar = bars + 11;                               // [P T; T] R done
    uint64_t* xbar = bars + 12;                                // the state's update done
    uint64_t* drain = bars + 13;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
    if (t == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bars + i, 1);
        mbar_init(freed, NA + 1);
        mbar_init(freed + 1, NA + 1);
        mbar_init(gbar, 1);
        mbar_init(sbar, NA);
        mbar_init(rbar, NA);
        mbar_init(ubar, NA);
        mbar_init(d1bar, 1);
        mbar_init(d2bar, 1);
        mbar_init(xbar, 1);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::alloc(tmem_slot, 512);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tq = tmem + (uint32_t(32 * (warp & 3)) << 16);    // this warp's TMEM lane quarter
    bool failed = false;

    if (warp < NWK / 32) {
        // ------------------------------------------------------------ workers
        const int d = (warp & 3) * 32 + lane, half = warp >> 2;
        constexpr int KH = K / 2;                              // state rows of a thread
        if ((warp & 3) * 32 < V) {
            float S[KH];
            float* const sp = state + (long long)(half * KH) * V + d;
#pragma unroll
            for (int i = 0; i < KH; ++i) S[i] = fresh ? 0.f : __ldcs(sp + i * V);
            for (int c = 0; c < chunks; ++c) {
                const int s = c & 1;
                const unsigned ph = c & 1, ph2 = (c >> 1) & 1;
                const float* vec = reinterpret_cast<const float*>(sm + L.vec[s]);
                const float4* vb = reinterpret_cast<const float4*>(vec + C + half * 32);
                const float4* vg = reinterpret_cast<const float4*>(vec + 2 * C + half * 32);
                const float4* vt = reinterpret_cast<const float4*>(vec + 3 * C + half * 32);
                const uint16_t* sv = reinterpret_cast<const uint16_t*>(sm + L.v[s]) + half * 32 * V + d;
                put_parts<KH>(tq + T_SP + half * (KH / 2), K / 2, S);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(sbar);

                if (!warp_wait(d1bar, ph) || !warp_wait(ready + s, ph2)) { failed = true; break; }
                tc::fence_after();
                float y[32], o[32];                            // tokens half * 32 .. + 31 of this state column
                if (ERASE) {
                    get<32>(tq + T_D1 + C + half * 32, reinterpret_cast<uint32_t*>(y));
                    tc::wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 bt = vb[i], g = ERASE ? vg[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                    const float be[4] = {bt.x, bt.y, bt.z, bt.w}, ge[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = bf2f(sv[(4 * i + e) * V]);
                        y[4 * i + e] = be[e] * (ERASE ? fmaf(-ge[e], y[4 * i + e], v) : v);
                    }
                }
                put_parts<32>(tq + T_RP + half * 16, 32, y);
                if (ERASE) {
                    tc::wait_st();
                    tc::fence_before();
                    mbar_arrive(rbar);
                    if (!warp_wait(d2bar, ph)) { failed = true; break; }
                    tc::fence_after();
                    get<32>(tq + T_X + C + half * 32, reinterpret_cast<uint32_t*>(y));
                    get<32>(tq + T_X + half * 32, reinterpret_cast<uint32_t*>(o));
                    tc::wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 tl = vt[i];
                    y[4 * i] *= tl.x; y[4 * i + 1] *= tl.y; y[4 * i + 2] *= tl.z; y[4 * i + 3] *= tl.w;
                }
                put_parts<32>(tq + T_UP + half * 16, 32, y);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(ubar);

                // the output, beside the update's MMAs
                if (!ERASE) {
                    if (!warp_wait(d2bar, ph)) { failed = true; break; }
                    tc::fence_after();
                    get<32>(tq + T_D1 + C + half * 32, reinterpret_cast<uint32_t*>(o));
                }
                get<32>(tq + T_D1 + half * 32, reinterpret_cast<uint32_t*>(y));
                tc::wait_ld();
                const int live = min(C, count - c * C) - half * 32;
                const long long at = (long long)(first + c * C + half * 32) * p.os + (long long)h * V + d;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 g = vg[i];
                    const float ge[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 4 * i + e;
                        const float x = fmaf(ge[e], y[r], o[r]);
                        if (r < live) {
                            if (p.out_bf16) static_cast<uint16_t*>(p.out)[at + r * p.os] = f2bf(x);
                            else static_cast<float*>(p.out)[at + r * p.os] = x;
                        }
                    }
                }
                const float whole = vec[2 * C + C - 1];
                mbar_arrive(freed + s);

                if (!warp_wait(xbar, ph)) { failed = true; break; }
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < KH; k += 32) {
                    get<32>(tq + T_X + half * KH + k, reinterpret_cast<uint32_t*>(y));
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[k + i] = fmaf(whole, S[k + i], y[i]);
                }
            }
            if (!failed)
#pragma unroll
                for (int i = 0; i < KH; ++i) __stcs(sp + i * V, S[i]);
        }
    } else if (warp < (NWK + NST) / 32) {
        // ------------------------------------------------------------ staging
        const int st = t - NWK;                                // row of [Q; K] and of [P T; T]
        const float A = FAM == MAMBA2 ? p.A[h] : 0.f;
        const uint16_t* gq = p.q + (long long)(h / p.group) * K;
        const uint16_t* gk = p.k + (long long)(h / p.group) * K;
        const uint16_t* gv = p.v + (long long)h * V;
        auto load = [&](int c) {
            const int s = c & 1, n = min(C, count - c * C);
            const long long r0 = first + c * C;
            float ga = FAM == MAMBA2 ? 0.f : 1.f, be = 0.f;
            if (st < n) {
                ga = p.gate[(r0 + st) * p.gs + h];
                if (ERASE) be = p.beta[(r0 + st) * p.bs + h];
            }
            const uint32_t qk = smem_u32(sm + L.qk[s]), vv = smem_u32(sm + L.v[s]);
            constexpr int KC = K / 8, VC = V / 8;              // 16-byte pieces of a row
#pragma unroll 4
            for (int i = st; i < C * KC; i += NST) {
                const int r = i / KC, x = (i % KC) * 8;
                const bool live = r < n;
                const long long row = live ? r0 + r : r0;
                cp_async16_or_zero(qk + tc::sw128h_off(2 * C, r, x), gq + row * p.qs + x, live);
                cp_async16_or_zero(qk + tc::sw128h_off(2 * C, C + r, x), gk + row * p.ks + x, live);
            }
#pragma unroll 4
            for (int i = st; i < C * VC; i += NST) {
                const int r = i / VC, x = (i % VC) * 8;
                const bool live = r < n;
                cp_async16_or_zero(vv + (r * V + x) * 2, gv + (live ? r0 + r : r0) * p.vs + x, live);
            }
            cp_async_commit();
            if (st < C) {
                float* vec = reinterpret_cast<float*>(sm + L.vec[s]);
                if (FAM == MAMBA2) {
                    be = ga;
                    ga = st < n ? expf(ga * A) : 1.f;
                }
                vec[st] = ga;
                vec[C + st] = be;
            }
        };
        load(0);
        if (chunks > 1) load(1);
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const unsigned ph = c & 1;
            if (c >= 2) {
                if (!warp_wait(freed + s, ((c >> 1) - 1) & 1)) { failed = true; break; }
                load(c);
            }
            if (c == 0 && chunks > 1) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
            else cp_async_wait_all();
            tc::fence_proxy_async();
            tc::fence_before();
            st_bar();
            const uint32_t qk = smem_u32(sm + L.qk[s]);
            if (st == 0) {
                mbar_arrive(full + s);
                tc::fence_after();
                constexpr uint32_t id = tc::idesc_bf16(128, C);
#pragma unroll
                for (int k = 0; k < K / 16; ++k) {
                    const uint32_t o = (k >> 2) * (2 * C * 128) + (k & 3) * 32;
                    tc::mma_ss_bf16(tmem + T_G, tc::sdesc(qk + o, 16, 1024, tc::LAYOUT_SW128),
                                    tc::sdesc(qk + C * 128 + o, 16, 1024, tc::LAYOUT_SW128), id, k > 0);
                }
                tc::commit(gbar);
            }
            float* vec = reinterpret_cast<float*>(sm + L.vec[s]);
            if (warp == NWK / 32) {                            // g and t: products from the front and from the back
                const float2 a = reinterpret_cast<const float2*>(vec)[lane];
                float f = a.x * a.y, r = f;
#pragma unroll
                for (int m = 1; m < 32; m *= 2) {
                    const float x = __shfl_up_sync(FULL, f, m), y = __shfl_down_sync(FULL, r, m);
                    if (lane >= m) f *= x;
                    if (lane + m < 32) r *= y;
                }
                float fe = __shfl_up_sync(FULL, f, 1), re = __shfl_down_sync(FULL, r, 1);
                if (lane == 0) fe = 1.f;
                if (lane == 31) re = 1.f;
                reinterpret_cast<float2*>(vec + 2 * C)[lane] = make_float2(fe * a.x, f);
                reinterpret_cast<float2*>(vec + 3 * C)[lane] = make_float2(re * a.y, re);
            }
            if (!warp_wait(gbar, ph)) { failed = true; break; }
            tc::fence_after();
            float x[C];                                        // a row of [P; -A], then of [P T; T]
            get<C>(tq + T_G, reinterpret_cast<uint32_t*>(x));
            tc::wait_ld();
            const int row = st & (C - 1);                      // token of this row
            const bool krow = st >= C;
            {
                const float scale = krow ? vec[C + row] : 1.f;
                float dij = scale;
#pragma unroll
                for (int j = C - 1; j >= 0; --j) {             // D_ij from j = i down
                    if (j < row) dij *= vec[j + 1];
                    x[j] = j <= row ? dij * x[j] : 0.f;
                }
            }
            if (ERASE) {
                if (krow) {
                    float* sa = reinterpret_cast<float*>(sm + L.a) + row * AP;
#pragma unroll
                    for (int j = 0; j < C; j += 4)
                        *reinterpret_cast<float4*>(sa + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
#pragma unroll
                    for (int j = 0; j < C; ++j) x[j] = j == row ? 1.f : 0.f;
                }
                st_bar();
                // X (I + A) = [P; I]: x_m is final once every later one has been
                // taken out; then x_j -= x_m A_mj for the j before it.
                const float* sa = reinterpret_cast<const float*>(sm + L.a);
#pragma unroll
                for (int m = C - 1; m > 0; --m) {
                    const float2 xm = dup2(-x[m]);
#pragma unroll
                    for (int j = ((m - 1) & ~3); j >= 0; j -= 4) {
                        const float4 a = *reinterpret_cast<const float4*>(sa + m * AP + j);
                        if (j + 3 < m) {
                            const float2 hi = ffma2(xm, make_float2(a.z, a.w), make_float2(x[j + 2], x[j + 3]));
                            const float2 lo = ffma2(xm, make_float2(a.x, a.y), make_float2(x[j], x[j + 1]));
                            x[j] = lo.x; x[j + 1] = lo.y; x[j + 2] = hi.x; x[j + 3] = hi.y;
                        } else {
                            if (j + 2 < m) x[j + 2] = fmaf(xm.x, a.z, x[j + 2]);
                            if (j + 1 < m) x[j + 1] = fmaf(xm.x, a.y, x[j + 1]);
                            x[j] = fmaf(xm.x, a.x, x[j]);
                        }
                    }
                }
            }
            if (ERASE || !krow) {
                unsigned char* tp = sm + L.tp[s] + st * 128;
#pragma unroll
                for (int j = 0; j < C; j += 8) {
                    uint32_t w[4][NP];
#pragma unroll
                    for (int e = 0; e < 4; ++e) cut(x[j + 2 * e], x[j + 2 * e + 1], w[e]);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        *reinterpret_cast<uint4*>(tp + q * (2 * C * C * 2) + (((j >> 3) ^ (st & 7)) << 4)) =
                            make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
                }
            }
            tc::fence_proxy_async();
            tc::fence_before();
            st_bar();
            if (st == 0) mbar_arrive(ready + s);
        }
        cp_async_wait_all();
    } else if (lane == 0) {
        // ------------------------------------------------------------ MMAs
        constexpr int N1 = ERASE ? 2 * C : C;
        constexpr uint32_t id1 = tc::idesc_bf16(128, N1), id3 = tc::idesc_bf16_bmn(128, K);
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const unsigned ph = c & 1, ph2 = (c >> 1) & 1;
            const uint32_t qk = smem_u32(sm + L.qk[s]), tp = smem_u32(sm + L.tp[s]);
            if (!mbar_wait(full + s, ph2) || !mbar_wait(sbar, ph)) { failed = true; break; }
            tc::fence_after();
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int k = 0; k < K / 16; ++k)
                    tc::mma_ts_bf16(tmem + T_D1, tmem + T_SP + i * (K / 2) + k * 8,
                                    tc::sdesc(qk + (k >> 2) * (2 * C * 128) + (k & 3) * 32, 16, 1024, tc::LAYOUT_SW128),
                                    id1, i + k > 0);
            tc::commit(d1bar);
            // [P T; T] R, or Mamba-2's P R beside S^T q
            auto products = [&](uint32_t dst) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; i + j < NP; ++j)
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            tc::mma_ts_bf16(dst, tmem + T_RP + i * 32 + k * 8,
                                            tc::sdesc(tp + j * (2 * C * C * 2) + k * 32, 16, 1024, tc::LAYOUT_SW128), id1,
                                            i + j + k > 0);
                tc::commit(d2bar);
            };
            if (ERASE) {
                if (!mbar_wait(ready + s, ph2) || !mbar_wait(rbar, ph)) { failed = true; break; }
                tc::fence_after();
                products(tmem + T_X);
            }
            if (!mbar_wait(ready + s, ph2) || !mbar_wait(ubar, ph)) { failed = true; break; }
            tc::fence_after();
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    tc::mma_ts_bf16(tmem + T_X, tmem + T_UP + i * 32 + k * 8,
                                    tc::sdesc(qk + C * 128 + k * 2048, 2 * C * 128, 1024, tc::LAYOUT_SW128), id3, i + k > 0);
            tc::commit(xbar);
            if (!ERASE) products(tmem + T_D1 + C);
            tc::commit(freed + s);
        }
        // every MMA of this thread has completed before the memory is released
        tc::commit(drain);
        if (!mbar_wait(drain, 0)) failed = true;
    }
    if (failed && lane == 0) report_timeout(p.status);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, 512);
}

template <int FAM, int K, int V>
cudaError_t chunks_launch(const PrefillParams& p, cudaStream_t stream) {
    static KernelCache kc;
    constexpr int need = pf_layout(K, V).total;
    static_assert(need <= SMEM_LIMIT, "shared memory");
    // more than half an SM's shared memory: one CTA an SM (each takes all of TMEM)
    constexpr int bytes = need > SMEM_SM / 2 + 4096 ? need : SMEM_SM / 2 + 4096;
    auto kern = prefill_chunks_kernel<FAM, K, V>;
    const cudaError_t e = ensure_smem(kern, kc, bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned(p.B) * unsigned(p.H)), dim3(NT), bytes, stream, p);
}

template <int FAM>
cudaError_t chunks_dispatch(int dk, int dv, const PrefillParams& p, cudaStream_t stream) {
    if (dk == 128 && dv == 128) return chunks_launch<FAM, 128, 128>(p, stream);
    if (dk == 128 && dv == 64) return chunks_launch<FAM, 128, 64>(p, stream);
    if (dk == 64 && dv == 128) return chunks_launch<FAM, 64, 128>(p, stream);
    if (dk == 64 && dv == 64) return chunks_launch<FAM, 64, 64>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefill_chunks(int family, int dk, int dv, const PrefillParams& p, cudaStream_t stream) {
    if (family == GDN) return chunks_dispatch<GDN>(dk, dv, p, stream);
    if (family == MAMBA2) return chunks_dispatch<MAMBA2>(dk, dv, p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace ss
