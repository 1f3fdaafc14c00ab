// Causal attention over whole sequences: arguments, sequence tiles and launchers (internal to libgdr2).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr2 {

struct PromptArgs {
    const void *q, *k, *v;               // [tokens][heads][D] with strides
    long long qs[2], ks[2], vs[2];       // token and head stride, elements
    void *o, *rest;                      // [tokens][Hq][D]; rest: what o's rounding left over, or null
    float* lse;                          // [tokens][Hq] or null
    const void* dout;                    // [tokens][Hq][D]
    void *dq, *dk, *dv;                  // [tokens][Hq][D], [tokens][Hkv][D]
    float *lse2, *delta;                 // workspace of the backward, [tokens][Hq] each
    const int* cu;                       // packed: [N + 1] on the device, else null
    int N, T;                            // sequences; tokens of each (packed: tokens in all)
    int Hq, Hkv, G, D;                   // G = Hq / Hkv query heads share a key head
    int window;                          // the last `window` tokens; at least T where all are seen
    int zero_rest;                       // packed: 1 sets the outputs' rows of no sequence to zero
    int neg;                             // 1: the scale is negative, and q enters with its sign turned
    float scale, scale2;                 // |scale| and |scale| log2(e), not zero
};

// Tiles of `tile` rows: tile slots of all sequences. Packed ones take slots from start / tile + s on, as many as
// they have tiles fit before the next one's first.
inline long long prompt_slots(int N, int T, bool packed, int tile) {
    return packed ? (long long)T / tile + N : (long long)N * (((long long)T + tile - 1) / tile);
}

hipError_t launch_prompt_fwd(const PromptArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_prompt_bwd(const PromptArgs& a, bool bf16, hipStream_t stream);

}  // namespace gdr2
