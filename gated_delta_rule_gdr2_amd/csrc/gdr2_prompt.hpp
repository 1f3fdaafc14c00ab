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
    float* part;                         // workspace: parts of dk, then of dv, [parts][tokens][Hkv][D] each
    int parts;                           // parts that a key head's query heads are cut in (dk, dv)
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

// Blocks of 32 rows, a wave's, of all sequences and one head; packed ones may be spare.
inline long long prompt_blocks(int N, int T, bool packed) { return prompt_slots(N, T, packed, 32); }
// Tokens of a sequence: of packed ones the mean, the lengths being the device's to know.
inline long long prompt_length(int N, int T, bool packed) { return packed ? ((long long)T + N - 1) / (N > 0 ? N : 1) : T; }

// Waves that share a block's other axis. None share where the longest walk is at most half of what each of the 1024 SIMDs
// has to do anyway; two where it is no longer than that; else four, which end soonest where all blocks are under way at
// once. More blocks than that (`once`: LDS holds the tiles of as many) take short walks alone, middle ones by twos and, up
// to 1024 of them, long ones by fours; in fp32, whose products are the longest, by twos. A sequence of one tile has nothing
// to share (in fp32 two share its rows). Of packed sequences the mean length has to do, the lengths being the device's to
// know: with one of 2000 tokens beside 23 of 5 - 28, 16 heads of 128, the backward takes 176 us alone and 135 by twos.
// `tasks`: walks of one head each; `heads`: heads that a walk goes through one after another; es: bytes of an element.
// Measured with S = 1, 2, 4, us, forward and backward, bf16, 128 channels:
//     2 x 4096 tokens, 16 heads 154, 183, 228 and 478, 533, 640     1 x 8192, 8 heads over 1 182, 163, 193 and 706, 572, 634
//     1 x 2048, 16 heads 43, 42, 36 and 140, 111, 105               1 x 1152, 16 heads 27, 27, 20 and 88, 72, 59
//     1 x 2048, 24 heads 48, 44, 56 and 155, 129, 163               1 x 1152, 32 heads 30, 29, 37 and 96, 76, 108
//     2 x 1024, 16 heads 26, 27, 27 and 83, 70, 79                  1 x 512, 16 heads 15, 17, 11 and 48, 42, 28
//     24 packed of 17 - 700 tokens, 16 heads over 4 48, 69, 105 and 183, 224, 360
//     5 x 168, 64 heads over 8 19, 29, 34 and 64, 84, 121           4 x 300, 32 heads 14, 22, 28 and 46, 59, 88
//     2 x 168, 48 heads 9.6, 12, 18 and 32, 32, 50                  2 x 512, 16 heads 16, 17, 14 and 50, 44, 39
//     16 x 60, 16 heads 8.0, 8.6, 7.9 and 22, 24, 31                64 x 20, 8 heads 7.6, 8.3, 7.6 and 20, 28, 42
// 64 channels: 4 x 300, 32 heads 10, 12, 14 and 29, 33, 49          1 x 1024, 32 heads 20, 20, 15 and 56, 46, 46
// fp32, 64:    4 x 300, 32 heads 38, 31, 46 and 107, 88, 137        1 x 130, 4 heads over 2 18, 12, 10 and 53, 36, 30
// fp32, 128:   2 x 168, 48 heads 33, 23, 35 and 107, 73, 116        1 x 2048, 16 heads over 4 271, 172, 205 and 924, 558, 663
//              16 x 64, 16 heads 16, 13, 25 and 51, 43, 80          1 x 60, 16 heads over 4 14, 12, 12 and 46, 38, 40
inline int prompt_sharing(const PromptArgs& a, long long tasks, int heads, int es) {
    const long long len = prompt_length(a.N, a.T, a.cu != nullptr), seen = len < a.window ? len : a.window;
    const long long walk = (seen + 63) / 64 * heads;  // tiles of the longest walk
    const long long once = es == 2 && a.D == 64 ? 1024 : 512;
    const double each = (double)tasks * walk * (seen < len ? 1.0 : 0.5) / 1024.0;
    if (a.T <= 64) return es == 2 ? 1 : 2;
    if (2.0 * walk <= each || (tasks >= 2048 && walk <= 8)) return 1;
    if (es == 2 && tasks > once && walk <= 8) return 1;
    return walk <= each || tasks > (es == 2 && walk > 16 ? 1024 : once) ? 2 : 4;
}

// Parts that the query heads of a key head are cut in for dK and dV, each walked by itself and added up by a further
// kernel: as many as make 4096 walks. The backward with 1, 2 and G parts, us: 1 x 4096 tokens, 32 heads over 8 505, 504, 492;
// 1 x 8192, 8 over 1 1155, 716, 499; 9 packed documents, 16 over 4 of 64 channels 205, 186, 180.
inline int prompt_parts(int N, int T, int Hq, int Hkv, bool packed) {
    const long long walks = prompt_blocks(N, T, packed) * Hkv, G = Hq / Hkv;
    const long long p = walks > 0 ? (4096 + walks - 1) / walks : 1;
    return (int)(p < G ? p : G);
}

// Queries that see few keys, the first 64 of a sequence (prompt_few), have their weights in two bf16 parts in the forward
// (bf16), whatever the call, so that a token's output does not lose precision by the batch it is in: the workgroups that hold
// such queries take a walk of their own. With it and without, us: 2 x 4096 tokens, 16 heads of 128 150.5 and 149.4, 1 x 16384
// 1003 and 1001, 24 packed of 17 - 700 tokens 29.8 and 29.1, 2 x 4096 of 64 channels with a window of 2048 76 and 74.4.
//
// Calls in which the backward does so too, for weights and their gradients: those of short sequences, and of few sequences and
// heads. Such queries hold the most of dq's and dk's size, and few roundings that balance one another: of 2 heads with one
// part, both were off by 1.5 times their own rounding on average and by up to 1.8 for 10 tokens, 1.6 for 40, 1.5 for 300, and
// with two parts by up to 1.2, 1.1 and 1.3; from some 8 heads on the average over a call's heads holds. For all calls, as in the
// forward, the backward takes 492 us for 471 (2 x 4096 tokens, 16 heads), 53 for 46 (4 x 300, 32 heads), and 200 for 176 (9
// packed documents of 64 channels): its registers hold two walks' operands only with spills.
inline bool prompt_exacts(const PromptArgs& a) {
    const long long len = prompt_length(a.N, a.T, a.cu != nullptr);
    return (len < a.window ? len : a.window) <= 128 || (long long)a.N * a.Hq <= 8;
}

hipError_t launch_prompt_fwd(const PromptArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_prompt_bwd(const PromptArgs& a, bool bf16, hipStream_t stream);

}  // namespace gdr2
