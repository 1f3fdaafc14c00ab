// Causal attention over whole sequences on gfx950, forward.
//
//     o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i.k_j - max),   lse_i = max + log sum_j p_ij
//
// over the keys j <= i of the token's sequence, the last `window` of them.
//
// A workgroup takes NW x 32 queries of one head, a wave 32 of them; keys and values pass through LDS in tiles of 64.
// The scores come out transposed, S^T = K Q^T, with a query in each column of lanes: its softmax runs in one lane and
// its partner in the other half wave, and the weights are the next product's operand where they stand
// (gdr2_prompt_device.hpp): O^T += V^T P^T, V^T by transposing LDS reads.
#include "gdr2_prompt_device.hpp"

namespace gdr2 {

constexpr int PKT = 64;  // keys of a tile

template <class OT, int D, int NW>
__global__ __launch_bounds__(64 * NW) void k_prompt_fwd(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int QT = 32 * NW, TB = PKT * TL::RB;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 4 * TB);
    poison_lds_done();
    PromptAt at;
    int slot;
    const int hp = prompt_at(a, blockIdx.x, QT, a.Hq, true, at, slot);
    const int hk = hp % a.Hkv, hq = hk * a.G + hp / a.Hkv;
    if (a.cu && a.zero_rest) {
        prompt_zero(a, slot, QT, (OT*)a.o, a.Hq, hq, D);
        if (a.rest) prompt_zero(a, slot, QT, (OT*)a.rest, a.Hq, hq, D);
        if (a.lse) prompt_zero(a, slot, QT, a.lse, a.Hq, hq, 1);
    }
    if (!at.any) return;
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q0 = at.tile * QT, last = at.len - 1;
    const int wq0 = q0 + 32 * w, qi = wq0 + (l & 31);
    const long long tok = at.tok0 + min(qi, last);
    FR qf[D / 16];
    load_own<OT, D>((const OT*)a.q + tok * a.qs[0] + hq * a.qs[1], a.neg, qf);
    const char* kb = (const char*)((const OT*)a.k + at.tok0 * a.ks[0] + hk * a.ks[1]);
    const char* vb = (const char*)((const OT*)a.v + at.tok0 * a.vs[0] + hk * a.vs[1]);
    const long long krs = a.ks[0] * (int)sizeof(OT), vrs = a.vs[0] * (int)sizeof(OT);
    // the tiles that any of the workgroup's queries sees
    const int t0 = max(0, q0 - a.window + 1) / PKT, t1 = min(q0 + QT - 1, last) / PKT;
    auto fetch = [&](int t) {
        lds_char* b = lds + (t & 1) * 2 * TB;
        TL::template load<PKT, NW>(kb, krs, t * PKT, last, b, w);
        TL::template load<PKT, NW>(vb, vrs, t * PKT, last, b + TB, w);
    };
    fetch(t0);
    f32x16 acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
    float m = -INFINITY, sum = 0.f;
    for (int t = t0; t <= t1; ++t) {
        wait_vm<0>();
        __syncthreads();  // the tile has landed, and everyone is done with the one before
        if (t < t1) fetch(t + 1);
        const int k0 = t * PKT;
        if (k0 > wq0 + 31 || k0 + PKT - 1 <= wq0 - a.window) continue;  // nothing of it is seen by this wave
        const lds_char* kt = lds + (t & 1) * 2 * TB;
        const lds_char* vt = kt + TB;
        f32x16 s[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n] = zero16();
#pragma unroll
            for (int b = 0; b < D / 16; ++b) mma32(s[n], TL::rows(kt, 32 * n, 16 * b), qf[b]);
        }
        if (k0 + PKT - 1 > wq0 || k0 <= wq0 + 31 - a.window) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = qi - (k0 + 32 * n + 8 * (r >> 2) + 4 * h + (r & 3));
                    s[n][r] = d >= 0 && d < a.window ? s[n][r] : -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[n][r]);
        mx = fmaxf(mx, other_half(mx)) * a.scale2;
        // the reference moves only where it would let a weight pass 2^8: sums and weights are relative to it
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            sum *= al;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * al;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        FR pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[n][r] = __builtin_amdgcn_exp2f(fmaf(s[n][r], a.scale2, -mu));
                sum += s[n][r];
            }
            pf[2 * n] = acc_frag<OT>(s[n], 0);
            pf[2 * n + 1] = acc_frag<OT>(s[n], 1);
        }
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int b = 0; b < 4; ++b) mma32(acc[dt], TL::cols(vt, 32 * dt, 16 * b), pf[b]);
    }
    sum += other_half(sum);
    if (qi > last) return;
    const float inv = 1.f / sum;
    const size_t row = (size_t)(at.tok0 + qi) * a.Hq + hq;
    if (sizeof(OT) == 2 && a.rest) {
        OT *po = (OT*)a.o + row * D, *pr = (OT*)a.rest + row * D;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = acc[dt][4 * j + i] * inv;
                    y[i] = x[i] - to_f(to_ot<OT>(x[i]));
                }
                st4(po + 32 * dt + 8 * j + 4 * h, x);
                st4(pr + 32 * dt + 8 * j + 4 * h, y);
            }
    } else {
        store_col<OT, D>((OT*)a.o + row * D, acc, inv);
    }
    if (a.lse && h == 0) a.lse[row] = (m + __log2f(sum)) * 0.6931471805599453f;
}

template <class OT, int D, int NW>
static hipError_t launch_fwd_t(const PromptArgs& a, hipStream_t stream) {
    constexpr int LDS = 4 * PKT * D * (int)sizeof(OT);
    const auto f = k_prompt_fwd<OT, D, NW>;
    if (LDS > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)f, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) return e;
    }
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 32 * NW) * a.Hq;
    hipLaunchKernelGGL(f, dim3((unsigned)n), dim3(64 * NW), LDS, stream, a);
    return hipGetLastError();
}

hipError_t launch_prompt_fwd(const PromptArgs& a, bool bf, hipStream_t stream) {
    if (bf) return a.D == 64 ? launch_fwd_t<bf16, 64, 8>(a, stream) : launch_fwd_t<bf16, 128, 8>(a, stream);
    return a.D == 64 ? launch_fwd_t<float, 64, 4>(a, stream) : launch_fwd_t<float, 128, 4>(a, stream);
}

}  // namespace gdr2
