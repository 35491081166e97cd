// Internal parameter structs and launchers of the calls beside decode: many
// tokens a sequence (ss_prefill) and the state cache.
#pragma once
#include "ss_internal.h"

namespace ss {

// Parameters of the many-token kernels (ss_prefill).  Strides are elements
// between token rows; head h reads q and k of head h / group.
struct PrefillParams {
    float* state;
    const float* A;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const float* gate;
    const float* beta;
    void* out;
    const int32_t* seq_start;
    const int32_t* fresh;
    int32_t* status;
    long long qs, ks, vs, gs, bs, os;
    int rows, B, H, group, out_bf16;
    int order;               // chunked form: the sequences longest first (B <= PREFILL_ORDER_MAX), those without
                             // tokens not at all
    int stall;               // testing hook: extra bytes expected by the first bulk wait (chunked form)
};

constexpr int PREFILL_ORDER_MAX = 512;     // largest batch with PrefillParams::order

// Parameters of the state cache kernels: `n` values per sequence (H * dk * dv).
struct CacheParams {
    float* state;
    void* codes;
    uint16_t* scales;
    const int32_t* slot;     // [B], < 0: the sequence is left out
    int32_t* status;
    long long n;
    int B, slots;
};

// Many tokens per sequence, token by token with the state in registers.
cudaError_t launch_prefill_tokens(int family, int dk, int dv, const PrefillParams& p, cudaStream_t stream);
// The same in chunks of 64 tokens on the tensor cores (Mamba-2, GDN).
cudaError_t launch_prefill_chunks(int family, int dk, int dv, const PrefillParams& p, cudaStream_t stream);
// Whether that is the faster one for `units` = batch * heads and a longest sequence of `longest` tokens.
bool prefill_chunks_pay(int dk, int dv, long long units, long long longest);
// States into / out of quantised slots.
cudaError_t launch_cache_write(int bits, const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_read(int bits, const CacheParams& p, cudaStream_t stream);

}  // namespace ss
