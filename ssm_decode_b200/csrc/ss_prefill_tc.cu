// prefill_chunks_kernel: prompts through the Mamba-2 and GDN recurrences in
// chunks of 64 tokens on the fifth-generation tensor cores.
//
// Chunked gated delta rule.  Within a chunk, with D_ij = a_{j+1} ... a_i (1 for
// j = i), g_i = a_0 ... a_i, t_j = a_{j+1} ... a_63 and S the state before it,
//     A_ij = b_i D_ij (k_i . k_j) for j < i,     R_i = b_i (v_i - g_i S^T k_i),
//     U = (I + A)^-1 R,
//     o_i = g_i S^T q_i + sum_{j<=i} D_ij (q_i . k_j) u_j,
//     S  <- g_63 S + sum_j k_j (t_j u_j)^T.
// Mamba-2 has no erase term: A = 0, u_i = dt_i v_i, and the outputs' part is
// (P o dt) V, whose V is exact in bf16 and known from the start.  With P_ij = D_ij (q_i . k_j),
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
//   8 worker warps    hold S in registers, two threads a state column, half of
//                     the dk rows each; they make the A operands and write out;
//   4 staging warps   run ahead: from the Gram products G they solve
//                     X (I + A) = [P; I] from the last column back, one row of
//                     [P T; T] a thread;
//   4 service warps   one lane each: the state's MMAs; the TMA loads of q, k, v
//                     (three chunks deep); the Gram MMAs, a chunk ahead of the
//                     staging warps (that warp also zeroes the rows behind a
//                     sequence's last token, whatever memory holds there).
// The output of a chunk is stored while the next chunk's first product runs.
// Registers move from the service warps to the workers (168 + 168 + 136 + 40
// a thread of the four warpgroups = the 4 x 128 of the launch).  Roles are
// paced by mbarriers only.  Every wait is bounded: when one runs out the
// kernel sets SS_DEVICE_TIMEOUT, waits (bounded) for its MMAs and copies in
// flight, releases its tensor memory and returns.
//
// What bounds it (measured, GDN 128 x 128): a chunk takes 10.2 k cycles, and two
// chains of about that length run side by side: the workers' (S into parts 1.5 k,
// D1 2.2 k, R 1.1 k, X 2.1 k, t o U 1.2 k, update and sum 1.4 k) and the staging
// warps' (decays 1.7 k, the solve 5.5 k, parts 1.8 k).  Each warp runs its
// straight-line code at about four cycles an instruction, instruction fetches
// being the largest stall after the waits; the tensor pipe works for 4.6 k of the
// 10.2 k (60 MMAs of 77 cycles, whatever N up to 128) and the 8 Gram MMAs; 30 % is
// its share of a whole cold launch of 16 chunks, with its start and state loads.
// 8192 tokens x 32 heads take 703 us (32 of 148 SMs), 16 x 1024 tokens 422 to 446 us
// by the GPU.
// Measured and left out: the inverse by 16 x 16 blocks (fp32 tiles 400 against
// 350 us for 4096 tokens x 32 heads; warp-level tf32 or bf16 MMAs wait for the
// tcgen05 ones, 400 cycles and more a block), 8 staging or 16 worker warps
// (fewer registers a thread: spills, and with the SM's shared memory in use they
// miss L1), persistent CTAs (391 us), S handed over in two steps (373 us).
#include "ss_mma.cuh"
#include "ss_prefill.cuh"
#include "ss_tc.cuh"

namespace ss {
namespace {

constexpr int C = 64;                    // tokens a chunk
constexpr int NP = 3;                    // bf16 parts of an fp32 operand
constexpr int NWK = 256;                 // worker threads
constexpr int NST = 128;                 // staging threads
constexpr int NT = NWK + NST + 128;
constexpr int NS = 3;                    // stages of q, k, v
constexpr int AP = C + 4;                // row pitch of A (floats): float4 rows without bank conflicts

// TMEM columns (all 512).
constexpr uint32_t T_X = 0;              // [P T; T] R: outputs' part, U; then the state's update (128)
constexpr uint32_t T_SP = 128;           // S^T in parts (dk / 2 columns each); then R and t o U in parts (32 each)
constexpr uint32_t T_VP = T_X;           // Mamba-2: v^T in bf16, 16 columns in each half of X (a worker writes
                                         // where it alone read the last update)
constexpr uint32_t T_RP = T_SP, T_UP = T_SP + 32 * NP;
constexpr uint32_t T_D1 = 320;           // S^T q (64), S^T k (64); Mamba-2: the outputs' part in place of S^T k
constexpr uint32_t T_G = 448;            // Gram products (64)
static_assert(T_SP + 64 * NP <= T_D1 && T_UP + 32 * NP <= T_D1, "operand parts overlap D1");

struct PfLayout {
    int qk[NS], v[NS], tp, a, vec[NS], bars, total;
};
// Floats of vec: decays a, b, g, t of the chunk's tokens.
__host__ __device__ constexpr PfLayout pf_layout(int K, int V) {
    PfLayout L{};
    int o = 0;
    for (int s = 0; s < NS; ++s) { L.qk[s] = o; o += 2 * C * K * 2; }         // dk / 64 blocks of 128 rows: q, k
    L.tp = o; o += NP * 2 * C * C * 2;                                        // [P T; T], a 128-row block per part
    for (int s = 0; s < NS; ++s) { L.v[s] = o; o += C * V * 2; }
    L.a = o; o += C * AP * 4;
    for (int s = 0; s < NS; ++s) { L.vec[s] = o; o += 4 * C * 4; }
    L.bars = o; o += 256;
    L.total = o + 1024;
    return L;
}

// Box of 64 token rows of one head: x = channel, y = head, z = row.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
// Named barrier of the staging threads, and the same returning whether any of
// them passed `x` true: they leave together.
__device__ __forceinline__ bool st_any(bool x) {
    unsigned r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(unsigned(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void st_bar() { asm volatile("bar.sync 2, 128;\n" ::: "memory"); }

// x0, x1 cut into parts, packed two to a register (x0 in the low half).  The
// first parts are the leading 16 bits of what is left (8 significant ones), so
// every difference is exact, and so is the last part.
__device__ __forceinline__ void cut(float x0, float x1, uint32_t (&w)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
        w[i] = __byte_perm(b0, b1, 0x7632);
        const float2 r = ffma2(make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)),
                               dup2(-1.f), make_float2(x0, x1));
        x0 = r.x;
        x1 = r.y;
    }
}

// N (a multiple of 16) fp32 values of this thread's lane cut into parts and
// stored as columns of NP A operands: `base` is the first part's column for
// the thread's first value, parts `pitch` columns apart.
template <int N>
__device__ __forceinline__ void put_parts(uint32_t base, uint32_t pitch, const float* x) {
#pragma unroll
    for (int k = 0; k < N; k += 16) {
        uint32_t w[NP][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t c[NP];
            cut(x[k + 2 * i], x[k + 2 * i + 1], c);
#pragma unroll
            for (int p = 0; p < NP; ++p) w[p][i] = c[p];
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) tc::st8(base + p * pitch + k / 2, w[p]);
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

// Four MMAs: 64 elements of K of an A operand in TMEM and of a B operand whose
// K steps of 16 are `step` 16-byte units apart.  acc = 0: the first overwrites D.
__device__ __forceinline__ void mma_k64(uint32_t dst, uint32_t a, uint64_t b, uint32_t step, uint32_t id, uint32_t acc) {
#pragma unroll
    for (int k = 0; k < 4; ++k) tc::mma_ts_bf16(dst, a + 8 * k, b + step * k, id, k > 0 ? 1 : acc);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned phase) {
    return __all_sync(FULL, mbar_wait(bar, phase));
}

template <int FAM, int K, int V>
__global__ void __launch_bounds__(NT, 1) prefill_chunks_kernel(const __grid_constant__ PrefillParams p,
                                                               const __grid_constant__ CUtensorMap qmap,
                                                               const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr PfLayout L = pf_layout(K, V);
    constexpr int NA = 2 * V;                                  // worker threads with a state column
    constexpr bool ERASE = FAM == GDN;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    griddep_wait();
    // The next launch is let in when this one ends, not here: its blocks would
    // settle one by one on the SMs that fall idle first, long sequences beside
    // short ones, and the two SMs of a pair, which share instruction fetches, take
    // 5.5 to 6.9 us a chunk in step and 7 to 9 us apart.  16 ragged sequences x 32
    // heads, calls back to back: 512 us with the early start, 428 without it (432
    // with another kernel between); equal lengths lose nothing (237 and 237 us).
    const int h = int(blockIdx.x % unsigned(p.H));
    int b = int(blockIdx.x / unsigned(p.H)), first, count;
    const bool good = seq_rows<false>(p, b, first, count);
    if (!good && t == 0 && p.status != nullptr) atomicOr(p.status, SS_DEVICE_BAD_ROWS);
    bool fresh = p.fresh != nullptr && p.fresh[b] != 0;
    if (good && count == 0 && fresh) {                         // no token: the state only starts afresh
        float4* const s0 = reinterpret_cast<float4*>(p.state + ((long long)b * p.H + h) * (K * V));
        for (int i = t; i < K * V / 4; i += NT) s0[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (p.order) {
        b = sequence_at<NT>(p, b, reinterpret_cast<int*>(sm + L.a));     // (no copy lands in this scratch)
        if (b < 0 || !seq_rows<false>(p, b, first, count)) return;
        fresh = p.fresh != nullptr && p.fresh[b] != 0;
    } else if (!good) {
        return;
    }
    if (count == 0) return;
    float* const state = p.state + ((long long)b * p.H + h) * (K * V);
    const int chunks = (count + C - 1) / C;

    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L.bars);
    uint64_t* lbar = bars + 0;                                 // [3] a stage's copies have landed
    uint64_t* full = bars + 3;                                 // [3] and its rows behind the end are zero
    uint64_t* freed = bars + 6;                                // [3] the stage is no longer read (workers, last MMA)
    uint64_t* gbar = bars + 9;                                 // Gram products done
    uint64_t* gread = bars + 10;                               // and read (staging)
    uint64_t* ready = bars + 11;                               // [P T; T] and the decays staged
    uint64_t* sbar = bars + 12;                                // S^T's parts written (workers)
    uint64_t* rbar = bars + 13;                                // R's parts, or Mamba-2's v^T, written (workers)
    uint64_t* ubar = bars + 14;                                // t o U's parts written (workers)
    uint64_t* d1bar = bars + 15;                               // D1 done
    uint64_t* d2bar = bars + 16;                               // [P T; T] R, or Mamba-2's P v, done
    uint64_t* xbar = bars + 17;                                // the state's update done
    uint64_t* drain = bars + 18;                               // [2] the issuing threads' last MMAs done
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
    if (t == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(lbar + i, 1);
            mbar_init(full + i, 1);
            mbar_init(freed + i, NA + 1);
        }
        mbar_init(gbar, 1);
        mbar_init(gread, NST);
        mbar_init(ready, 1);
        mbar_init(sbar, NA);
        mbar_init(rbar, NA);
        mbar_init(ubar, NA);
        mbar_init(d1bar, 1);
        mbar_init(d2bar, 1);
        mbar_init(xbar, 1);
        mbar_init(drain, 1);
        mbar_init(drain + 1, 1);
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
        regs_inc<168>();
        const int d = (warp & 3) * 32 + lane, half = warp >> 2;
        constexpr int KH = K / 2;                              // state rows of a thread
        if ((warp & 3) * 32 < V) {
            float S[KH];
            float* const sp = state + (long long)(half * KH) * V + d;
#pragma unroll
            for (int i = 0; i < KH; ++i) S[i] = fresh ? 0.f : __ldcs(sp + i * V);
            float o[32];                                       // tokens half * 32 .. + 31 of this state column
            // o to the output rows of chunk c
            auto store = [&](int c) {
                const int live = min(C, count - c * C) - half * 32;
                const long long at = (long long)(first + c * C + half * 32) * p.os + (long long)h * V + d;
                if (p.out_bf16) {
                    uint16_t* w = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
                    for (int r = 0; r < 32; ++r, w += p.os)
                        if (r < live) *w = f2bf(o[r]);
                } else {
                    float* w = static_cast<float*>(p.out) + at;
#pragma unroll
                    for (int r = 0; r < 32; ++r, w += p.os)
                        if (r < live) *w = o[r];
                }
            };
            int s = 0;
            unsigned sph = 0;
            for (int c = 0; c < chunks; ++c) {
                const unsigned ph = c & 1;
                const float* vec = reinterpret_cast<const float*>(sm + L.vec[0] + s * (4 * C * 4));
                const float4* vb = reinterpret_cast<const float4*>(vec + C + half * 32);
                const float4* vg = reinterpret_cast<const float4*>(vec + 2 * C + half * 32);
                const float4* vt = reinterpret_cast<const float4*>(vec + 3 * C + half * 32);
                const uint16_t* sv = reinterpret_cast<const uint16_t*>(sm + L.v[0] + s * (C * V * 2)) + half * 32 * V + d;
                uint32_t vp[16];                               // Mamba-2: v of this thread's tokens, two a register
                if (!ERASE) {
                    // (ready first: once the product with v is issued, staging may complete
                    // the next chunk's, and this one's could no longer be waited for)
                    if (!warp_wait(lbar + s, sph) || !warp_wait(full + s, sph) || !warp_wait(ready, ph)) { failed = true; break; }
#pragma unroll
                    for (int i = 0; i < 16; ++i) vp[i] = uint32_t(sv[2 * i * V]) | (uint32_t(sv[(2 * i + 1) * V]) << 16);
                    tc::st16(tq + T_VP + half * KH, vp);
                    tc::wait_st();
                    tc::fence_before();
                    mbar_arrive(rbar);
                }
                put_parts<KH>(tq + T_SP + half * (KH / 2), K / 2, S);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(sbar);
                if (c > 0) store(c - 1);

                if (ERASE && (!warp_wait(lbar + s, sph) || !warp_wait(full + s, sph) || !warp_wait(ready, ph))) { failed = true; break; }
                if (!warp_wait(d1bar, ph)) { failed = true; break; }
                tc::fence_after();
                float y[32];
                if (ERASE) {
                    get<32>(tq + T_D1 + C + half * 32, reinterpret_cast<uint32_t*>(y));
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 bt = vb[i], g = vg[i];
                        const float be[4] = {bt.x, bt.y, bt.z, bt.w}, ge[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[4 * i + e] = be[e] * fmaf(-ge[e], y[4 * i + e], bf2f(sv[(4 * i + e) * V]));
                    }
                    put_parts<32>(tq + T_RP + half * 16, 32, y);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 bt = vb[i];
                        y[4 * i] = bt.x * bf2f_lo(vp[2 * i]); y[4 * i + 1] = bt.y * bf2f_hi(vp[2 * i]);
                        y[4 * i + 2] = bt.z * bf2f_lo(vp[2 * i + 1]); y[4 * i + 3] = bt.w * bf2f_hi(vp[2 * i + 1]);
                    }
                }
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
                if (!ERASE) get<32>(tq + T_D1 + C + half * 32, reinterpret_cast<uint32_t*>(o));
                get<32>(tq + T_D1 + half * 32, reinterpret_cast<uint32_t*>(y));
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 g = vg[i];
                    const float ge[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[4 * i + e] = fmaf(ge[e], y[4 * i + e], o[4 * i + e]);
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
                if (++s == NS) { s = 0; sph ^= 1u; }
            }
            if (!failed) {
                store(chunks - 1);
#pragma unroll
                for (int i = 0; i < KH; ++i) __stcs(sp + i * V, S[i]);
            }
        }
    } else if (warp < (NWK + NST) / 32) {
        // ------------------------------------------------------------ staging
        regs_inc<136>();
        const int st = t - NWK;                                // row of [Q; K] and of [P T; T]
        const int row = st & (C - 1);                          // its token
        const bool krow = st >= C;
        const float A = FAM == MAMBA2 ? p.A[h] : 0.f;
        float ga = 1.f, be = 0.f;                              // of token `row`, a chunk ahead
        auto fetch = [&](int c) {
            ga = FAM == MAMBA2 ? 0.f : 1.f;
            be = 0.f;
            if (c * C + row < count) {
                const long long r = first + c * C + row;
                ga = p.gate[r * p.gs + h];
                if (ERASE) be = p.beta[r * p.bs + h];
            }
        };
        fetch(0);
        int s = 0;
        for (int c = 0; c < chunks; ++c) {
            const unsigned ph = c & 1;
            float* vec = reinterpret_cast<float*>(sm + L.vec[0] + s * (4 * C * 4));
            // G of this chunk: its stage was free to load, so its vec is free too
            if (st_any(!warp_wait(gbar, ph))) { failed = true; break; }
            tc::fence_after();
            if (FAM == MAMBA2) {
                be = ga;
                ga = c * C + row < count ? expf(ga * A) : 1.f;
            }
            if (!krow) {
                vec[row] = ga;
                vec[C + row] = be;
            }
            const float scale = krow ? be : 1.f;
            float x[C];                                        // a row of [P; A], then of [P T; T]
            get<C>(tq + T_G, reinterpret_cast<uint32_t*>(x));
            tc::wait_ld();
            tc::fence_before();
            mbar_arrive(gread);
            st_bar();
            if (c + 1 < chunks) fetch(c + 1);
            if (warp == NWK / 32) {                            // g and t: products from the front and from the back
                const float2 a = reinterpret_cast<const float2*>(vec)[lane];
                float f = a.x * a.y, r = f;
#pragma unroll
                for (int m = 1; m < 32; m *= 2) {
                    const float fx = __shfl_up_sync(FULL, f, m), ry = __shfl_down_sync(FULL, r, m);
                    if (lane >= m) f *= fx;
                    if (lane + m < 32) r *= ry;
                }
                float fe = __shfl_up_sync(FULL, f, 1), re = __shfl_down_sync(FULL, r, 1);
                if (lane == 0) fe = 1.f;
                if (lane == 31) re = 1.f;
                reinterpret_cast<float2*>(vec + 2 * C)[lane] = make_float2(fe * a.x, f);
                reinterpret_cast<float2*>(vec + 3 * C)[lane] = make_float2(re * a.y, re);
            }
            {
                float dij = scale;
#pragma unroll
                for (int j = C - 4; j >= 0; j -= 4) {          // D_ij from j = i down
                    const float4 a = *reinterpret_cast<const float4*>(vec + j);
                    const float ae[4] = {a.x, a.y, a.z, a.w};
                    float be[4] = {1.f, 1.f, 1.f, 1.f};
                    if (!ERASE) {                              // u_j = dt_j v_j: dt goes with P
                        const float4 bt = *reinterpret_cast<const float4*>(vec + C + j);
                        be[0] = bt.x; be[1] = bt.y; be[2] = bt.z; be[3] = bt.w;
                    }
#pragma unroll
                    for (int e = 3; e >= 0; --e) {
                        x[j + e] = j + e <= row ? dij * x[j + e] : 0.f;
                        if (!ERASE) x[j + e] *= be[e];
                        if (j + e <= row) dij *= ae[e];
                    }
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
            // the product with the previous chunk's [P T; T] is done with the buffer
            if (st_any(c > 0 && !warp_wait(d2bar, ph ^ 1u))) { failed = true; break; }
            if (ERASE || !krow) {
                unsigned char* tp = sm + L.tp + st * 128;
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
            st_bar();
            if (st == 0) mbar_arrive(ready);
            if (++s == NS) s = 0;
        }
    } else {
        regs_dec<40>();
        if (warp == NWK / 32 + 4 && lane == 0) {
            // -------------------------------------------------------- the state's MMAs
            constexpr int N1 = ERASE ? 2 * C : C;
            constexpr uint32_t id1 = tc::idesc_bf16(128, N1), id3 = tc::idesc_bf16_bmn(128, K);
            const uint64_t dtp = tc::sdesc(smem_u32(sm + L.tp), 16, 1024, tc::LAYOUT_SW128);
            int s = 0;
            unsigned sph = 0;
            for (int c = 0; c < chunks; ++c) {
                const unsigned ph = c & 1;
                const uint32_t qk = smem_u32(sm + L.qk[0] + s * (2 * C * K * 2));
                // operands further on: the byte distance / 16 added to the address field
                const uint64_t dqk = tc::sdesc(qk, 16, 1024, tc::LAYOUT_SW128);
                const uint64_t dkt = tc::sdesc(qk + C * 128, 2 * C * 128, 1024, tc::LAYOUT_SW128);
                if (!mbar_wait(full + s, sph)) { failed = true; break; }
                // (rolled loops: unrolled ones keep every operand address in registers the warp does not have)
                if (!ERASE) {                                  // the outputs' part: v is exact, one part of it
                    if (!mbar_wait(ready, ph) || !mbar_wait(rbar, ph)) { failed = true; break; }
                    tc::fence_after();
#pragma unroll 1
                    for (int j = 0; j < NP; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_ts_bf16(tmem + T_D1 + C, tmem + T_VP + (k >> 1) * (K / 2) + (k & 1) * 8,
                                            dtp + uint32_t(j) * (2 * C * C * 2 >> 4) + 2 * k, id1, j + k > 0);
                    tc::commit(d2bar);
                }
                if (!mbar_wait(sbar, ph)) { failed = true; break; }
                tc::fence_after();
#pragma unroll 1
                for (int i = 0; i < NP * (K / 64); ++i)
                    mma_k64(tmem + T_D1, tmem + T_SP + 32 * i, dqk + uint32_t(i & (K / 64 - 1)) * (2 * C * 128 >> 4), 2, id1,
                            i > 0);
                tc::commit(d1bar);
                if (ERASE) {
                    if (!mbar_wait(ready, ph) || !mbar_wait(rbar, ph)) { failed = true; break; }
                    tc::fence_after();
#pragma unroll 1
                    for (int i = 0; i < NP; ++i)
#pragma unroll 1
                        for (int j = 0; i + j < NP; ++j)
                            mma_k64(tmem + T_X, tmem + T_RP + 32 * i, dtp + uint32_t(j) * (2 * C * C * 2 >> 4), 2, id1,
                                    i + j > 0);
                    tc::commit(d2bar);
                }
                if (!mbar_wait(ubar, ph)) { failed = true; break; }
                tc::fence_after();
#pragma unroll 1
                for (int i = 0; i < NP; ++i) mma_k64(tmem + T_X, tmem + T_UP + 32 * i, dkt, 2048 >> 4, id3, i > 0);
                tc::commit(xbar);
                tc::commit(freed + s);
                if (++s == NS) { s = 0; sph ^= 1u; }
            }
            // every MMA of this thread has completed before the memory is released
            tc::commit(drain);
            if (!mbar_wait(drain, 0)) failed = true;
        } else if (warp == NWK / 32 + 5 && lane == 0) {
            // -------------------------------------------------------- loads
            const int hq = h / p.group;
            int s = 0;
            unsigned sph = 1;
            int c = 0;
            for (; c < chunks; ++c) {
                if (c >= NS && !mbar_wait(freed + s, sph)) { failed = true; break; }
                const uint32_t qk = smem_u32(sm + L.qk[0] + s * (2 * C * K * 2));
                mbar_expect_tx(lbar + s, C * (2 * K + V) * 2 + (p.stall && blockIdx.x == 0 && c == 0 ? 16 : 0));
#pragma unroll
                for (int j = 0; j < K / 64; ++j) {
                    tma_load_3d(qk + j * (2 * C * 128), &qmap, 64 * j, hq, first + c * C, lbar + s);
                    tma_load_3d(qk + j * (2 * C * 128) + C * 128, &kmap, 64 * j, hq, first + c * C, lbar + s);
                }
                tma_load_3d(smem_u32(sm + L.v[0] + s * (C * V * 2)), &vmap, 0, h, first + c * C, lbar + s);
                if (++s == NS) { s = 0; sph ^= 1u; }
            }
            // nothing is in flight into this CTA's shared memory when it ends (they
            // have long been waited for, unless a wait ran out)
            for (int i = max(0, c - NS); i < c; ++i)
                if (!mbar_wait(lbar + i % NS, (i / NS) & 1)) failed = true;
        } else if (warp == NWK / 32 + 6) {
            // -------------------------------------------------------- Gram products
            constexpr uint32_t id = tc::idesc_bf16(128, C);
            int s = 0;
            unsigned sph = 0;
            for (int c = 0; c < chunks; ++c) {
                unsigned char* const qkp = sm + L.qk[0] + s * (2 * C * K * 2);
                if (!warp_wait(lbar + s, sph)) { failed = true; break; }
                const int n = count - c * C;
                if (n < C) {                                   // zeros behind the last token
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    for (int i = lane; i < (C - n) * 8; i += 32)
#pragma unroll
                        for (int j = 0; j < 2 * (K / 64); ++j)
                            *reinterpret_cast<uint4*>(qkp + j * (C * 128) + n * 128 + i * 16) = z;
                    uint4* const vp = reinterpret_cast<uint4*>(sm + L.v[0] + s * (C * V * 2) + n * V * 2);
                    for (int i = lane; i < (C - n) * V / 8; i += 32) vp[i] = z;
                    tc::fence_proxy_async();
                }
                __syncwarp();
                if (c > 0 && !warp_wait(gread, (c - 1) & 1)) { failed = true; break; }
                if (lane == 0) {
                    mbar_arrive(full + s);
                    tc::fence_after();
                    const uint32_t qk = smem_u32(qkp);
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) {
                        const uint32_t o = (k >> 2) * (2 * C * 128) + (k & 3) * 32;
                        tc::mma_ss_bf16(tmem + T_G, tc::sdesc(qk + o, 16, 1024, tc::LAYOUT_SW128),
                                        tc::sdesc(qk + C * 128 + o, 16, 1024, tc::LAYOUT_SW128), id, k > 0);
                    }
                    tc::commit(gbar);
                }
                __syncwarp();
                if (++s == NS) { s = 0; sph ^= 1u; }
            }
            if (lane == 0) tc::commit(drain + 1);
            if (!warp_wait(drain + 1, 0)) failed = true;
        }
    }
    if (failed && lane == 0) report_timeout(p.status);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, 512);
}

// Tensor map of [rows][heads][channels] bf16 token rows, boxes of 64 rows of
// `box` channels of one head; rows behind the last are zero.
cudaError_t token_map(const uint16_t* base, int channels, int heads, int rows, long long stride, int box, bool swizzle,
                      CUtensorMap* out) {
    const EncodeTiled enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {cuuint64_t(channels), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(channels) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t boxes[3] = {cuuint32_t(box), 1, C};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, boxes,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int FAM, int K, int V>
cudaError_t chunks_launch(const PrefillParams& p, cudaStream_t stream) {
    static KernelCache kc;
    constexpr int need = pf_layout(K, V).total;
    static_assert(need <= SMEM_LIMIT, "shared memory");
    // more than half an SM's shared memory: one CTA an SM (each takes all of TMEM)
    constexpr int bytes = need > SMEM_SM / 2 + 4096 ? need : SMEM_SM / 2 + 4096;
    auto kern = prefill_chunks_kernel<FAM, K, V>;
    cudaError_t e = ensure_smem(kern, kc, bytes);
    CUtensorMap qm, km, vm;
    if (e == cudaSuccess) e = token_map(p.q, K, p.H / p.group, p.rows, p.qs, 64, true, &qm);
    if (e == cudaSuccess) e = token_map(p.k, K, p.H / p.group, p.rows, p.ks, 64, true, &km);
    if (e == cudaSuccess) e = token_map(p.v, V, p.H, p.rows, p.vs, V, false, &vm);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned(p.B) * unsigned(p.H)), dim3(NT), bytes, stream, p, qm, km, vm);
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

// The chunked form's time goes by the chunks of 64 tokens, full or not, and by
// the waves of units over the SMs, one a CTA; the token form's by the tokens: a
// latency of half a microsecond each while its CTAs have SMs to themselves, dk dv
// multiply-adds each once they do not.  So the first chunk pays from a number of
// tokens that grows with the waves and with how small the state is, a later one
// from 3 / 8 of it more.  Measured on equal lengths, tokens / chunks in us:
//   one wave   GDN 1 x 32 heads, 128 x 128: 20 tokens 14.4 / 15.9, 24 16.4 / 15.7, 64 34 / 15.5;
//              64 x 64, 4 x 32 heads: 24 tokens 14.8 / 15.4, 28 15.9 / 15.2
//   to four    GDN 16 x 32 heads: 128 x 128, 24 tokens 50 / 54, 28 57 / 54; 64 x 128, 32 44 / 50, 40 53 / 51;
//              128 x 64, 40 48 / 53, 48 56 / 53; 64 x 64, 48 47 / 48.  8 x 32 heads, 128 x 64: 32 26 / 29, 40 31 / 29
//   more       GDN 256 x 32 heads: 128 x 128, 32 tokens 843 / 879, 40 1057 / 879; 64 x 128, 48 758 / 823, 56 884 / 824;
//              128 x 64, 56 739 / 847, 80 1035 / 1155, 96 1238 / 1159; 64 x 64, 112 884 / 1077, 160 1257 / 1364.
//              Mamba-2 64 x 32 heads: 128 x 128, 28 167 / 162; 64 x 128, 40 147 / 135; 128 x 64, 56 164 / 147,
//              65 189 / 196; 64 x 64, 64 119 / 125, 96 175 / 168, 112 203 / 169
bool prefill_chunks_pay(int dk, int dv, long long units, long long longest) {
    static constexpr int from[2][2][3] = {{{24, 44, 80}, {20, 30, 44}}, {{20, 38, 57}, {20, 24, 32}}};
    longest = longest < 0x7fffffffLL ? longest : 0x7fffffffLL;          // (a bound: any number may be given)
    const long long waves = (units + sm_count() - 1) / sm_count(), chunks = (longest + C - 1) / C;
    return longest * 8 >= from[dk == 128][dv == 128][waves <= 1 ? 0 : waves <= 4 ? 1 : 2] * (5 + 3 * chunks);
}

cudaError_t launch_prefill_chunks(int family, int dk, int dv, const PrefillParams& p, cudaStream_t stream) {
    if (family == GDN) return chunks_dispatch<GDN>(dk, dv, p, stream);
    if (family == MAMBA2) return chunks_dispatch<MAMBA2>(dk, dv, p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace ss
