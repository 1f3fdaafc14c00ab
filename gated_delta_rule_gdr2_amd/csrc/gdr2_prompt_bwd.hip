// Causal attention over whole sequences on gfx950, backward. With P_ij = exp(scale q_i.k_j - lse_i) on what i sees,
//
//     dV = P^T dO    dS_ij = P_ij (dO_i.v_j - delta_i),  delta_i = dO_i.o_i    dQ = scale dS K    dK = scale dS^T Q
//
// dK and dV summed over the query heads that share a key head. Two kernels, one for dQ (a wave owns 32 queries and
// walks their keys) and one for dK and dV (a wave owns 32 keys and walks the queries of all heads that see them), each
// with its sums in registers: every result is added up by one wave in a fixed order, without atomics, for the price of
// forming the scores twice. The first one leaves lse log2(e) and delta for the second.
#include "gdr2_prompt_device.hpp"

namespace gdr2 {

constexpr int BT = 64;  // rows of a tile

// waves a SIMD that a kernel's registers have to leave room for
template <class OT, int D>
constexpr int prompt_waves() { return sizeof(OT) == 4 && D == 128 ? 1 : 2; }

// ---------------------------------------------------------------- dQ: as the forward, keys in tiles
template <class OT, int D, int NW>
__global__ __launch_bounds__(64 * NW, (prompt_waves<OT, D>())) void k_prompt_dq(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int QT = 32 * NW, TB = BT * TL::RB;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 4 * TB);
    poison_lds_done();
    PromptAt at;
    int slot;
    const int hp = prompt_at(a, blockIdx.x, QT, a.Hq, true, at, slot);
    const int hk = hp % a.Hkv, hq = hk * a.G + hp / a.Hkv;
    if (a.cu && a.zero_rest) prompt_zero(a, slot, QT, (OT*)a.dq, a.Hq, hq, D);
    if (!at.any) return;
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q0 = at.tile * QT, last = at.len - 1;
    const int wq0 = q0 + 32 * w, qi = wq0 + (l & 31);
    const long long tok = at.tok0 + min(qi, last);
    const size_t row = (size_t)tok * a.Hq + hq;
    FR qf[D / 16], df[D / 16];
    load_own<OT, D>((const OT*)a.q + tok * a.qs[0] + hq * a.qs[1], a.neg, qf);
    load_own<OT, D>((const OT*)a.dout + row * D, false, df);
    const char* kb = (const char*)((const OT*)a.k + at.tok0 * a.ks[0] + hk * a.ks[1]);
    const char* vb = (const char*)((const OT*)a.v + at.tok0 * a.vs[0] + hk * a.vs[1]);
    const long long krs = a.ks[0] * (int)sizeof(OT), vrs = a.vs[0] * (int)sizeof(OT);
    const int t0 = max(0, q0 - a.window + 1) / BT, t1 = min(q0 + QT - 1, last) / BT;
    auto fetch = [&](int t) {
        lds_char* b = lds + (t & 1) * 2 * TB;
        TL::template load<BT, NW>(kb, krs, t * BT, last, b, w);
        TL::template load<BT, NW>(vb, vrs, t * BT, last, b + TB, w);
    };
    fetch(t0);
    // delta from o and what its rounding left over: of a row that sees few keys dP - delta is a small difference
    float delta = 0.f;
    {
        const OT* po = (const OT*)a.o + row * D + 8 * h;
        const OT* pr = a.rest ? (const OT*)a.rest + row * D + 8 * h : nullptr;
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {
            const FR x = *(const FR*)(po + 16 * b);
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = fmaf(to_f(x[e]), to_f(df[b][e]), delta);
            if (pr) {
                const FR y = *(const FR*)(pr + 16 * b);
#pragma unroll
                for (int e = 0; e < 8; ++e) delta = fmaf(to_f(y[e]), to_f(df[b][e]), delta);
            }
        }
        delta += other_half(delta);
    }
    const float lse2 = a.lse[row] * 1.4426950408889634f;
    if (qi <= last && h == 0) {
        a.lse2[row] = lse2;
        a.delta[row] = delta;
    }
    f32x16 acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
    for (int t = t0; t <= t1; ++t) {
        wait_vm<0>();
        __syncthreads();
        if (t < t1) fetch(t + 1);
        const int k0 = t * BT;
        if (k0 > wq0 + 31 || k0 + BT - 1 <= wq0 - a.window) continue;
        const lds_char* kt = lds + (t & 1) * 2 * TB;
        const lds_char* vt = kt + TB;
        const bool part = k0 + BT - 1 > wq0 || k0 <= wq0 + 31 - a.window;
#pragma unroll
        for (int n = 0; n < BT / 32; ++n) {
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int b = 0; b < D / 16; ++b) mma32(s, TL::rows(kt, 32 * n, 16 * b), qf[b]);
#pragma unroll
            for (int b = 0; b < D / 16; ++b) mma32(dp, TL::rows(vt, 32 * n, 16 * b), df[b]);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale2, -lse2));
                s[r] = p * (dp[r] - delta);
            }
            if (part) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = qi - (k0 + 32 * n + 8 * (r >> 2) + 4 * h + (r & 3));
                    s[r] = d >= 0 && d < a.window ? s[r] : 0.f;
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const FR f = acc_frag<OT>(s, b);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) mma32(acc[dt], TL::cols(kt, 32 * dt, 32 * n + 16 * b), f);
            }
        }
    }
    if (qi <= last) store_col<OT, D>((OT*)a.dq + row * D, acc, a.neg ? -a.scale : a.scale);
}

// ---------------------------------------------------------------- dK, dV: queries in tiles
template <class OT, int D, int NW>
__global__ __launch_bounds__(64 * NW, (prompt_waves<OT, D>())) void k_prompt_dkv(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int KT = 32 * NW, TB = BT * TL::RB, BUF = 2 * TB + 2 * BT * 4;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 2 * BUF);
    poison_lds_done();
    PromptAt at;
    int slot;
    const int hk = prompt_at(a, blockIdx.x, KT, a.Hkv, false, at, slot);
    if (a.cu && a.zero_rest) {
        prompt_zero(a, slot, KT, (OT*)a.dk, a.Hkv, hk, D);
        prompt_zero(a, slot, KT, (OT*)a.dv, a.Hkv, hk, D);
    }
    if (!at.any) return;
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k0 = at.tile * KT, last = at.len - 1;
    const int wk0 = k0 + 32 * w, ki = wk0 + (l & 31);
    const long long tok = at.tok0 + min(ki, last);
    FR kf[D / 16], vf[D / 16];
    load_own<OT, D>((const OT*)a.k + tok * a.ks[0] + hk * a.ks[1], a.neg, kf);
    load_own<OT, D>((const OT*)a.v + tok * a.vs[0] + hk * a.vs[1], false, vf);
    // the query tiles that see any of the workgroup's keys, for each head in turn
    const int t0 = k0 / BT, t1 = (int)min((long long)last, (long long)k0 + KT - 2 + a.window) / BT, nt = t1 - t0 + 1;
    const long long qrs = a.qs[0] * (int)sizeof(OT), drs = (long long)a.Hq * TL::RB;
    auto fetch = [&](int i) {
        const int hq = hk * a.G + i / nt, r0 = (t0 + i % nt) * BT;
        lds_char* b = lds + (i & 1) * BUF;
        TL::template load<BT, NW>((const char*)((const OT*)a.q + at.tok0 * a.qs[0] + hq * a.qs[1]), qrs, r0, last, b, w);
        TL::template load<BT, NW>((const char*)((const OT*)a.dout + (at.tok0 * a.Hq + hq) * D), drs, r0, last, b + TB, w);
        if (w < 2) {
            const float* src = (w ? a.delta : a.lse2) + (at.tok0 + min(r0 + l, last)) * a.Hq + hq;
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(b + 2 * TB + w * BT * 4), 4, 0, 0);
        }
    };
    fetch(0);
    f32x16 ak[D / 32], av[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) ak[i] = av[i] = zero16();
    const int all = nt * a.G;
    for (int i = 0; i < all; ++i) {
        wait_vm<0>();
        __syncthreads();
        if (i + 1 < all) fetch(i + 1);
        const lds_char* qt = lds + (i & 1) * BUF;
        const lds_char* dt_ = qt + TB;
        const lds_char* st = qt + 2 * TB;
#pragma unroll
        for (int n = 0; n < BT / 32; ++n) {
            const int r0 = (t0 + i % nt) * BT + 32 * n;
            if (r0 + 31 < wk0 || r0 > last || r0 - wk0 - 31 >= a.window) continue;
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int b = 0; b < D / 16; ++b) mma32(s, TL::rows(qt, 32 * n, 16 * b), kf[b]);
#pragma unroll
            for (int b = 0; b < D / 16; ++b) mma32(dp, TL::rows(dt_, 32 * n, 16 * b), vf[b]);
            const bool part = r0 < wk0 + 31 || r0 + 31 > last || r0 + 31 - wk0 >= a.window;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 ls = lds_load<f32x4>(st + (32 * n + 8 * j + 4 * h) * 4);
                const f32x4 de = lds_load<f32x4>(st + (BT + 32 * n + 8 * j + 4 * h) * 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float p = __builtin_amdgcn_exp2f(fmaf(s[4 * j + x], a.scale2, -ls[x]));
                    float g = p * (dp[4 * j + x] - de[x]);
                    if (part) {
                        const int r = r0 + 8 * j + 4 * h + x, d = r - ki;
                        const bool see = d >= 0 && d < a.window && r <= last;
                        p = see ? p : 0.f;
                        g = see ? g : 0.f;
                    }
                    s[4 * j + x] = p;
                    dp[4 * j + x] = g;
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const FR pf = acc_frag<OT>(s, b), gf = acc_frag<OT>(dp, b);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) {
                    mma32(av[dt], TL::cols(dt_, 32 * dt, 32 * n + 16 * b), pf);
                    mma32(ak[dt], TL::cols(qt, 32 * dt, 32 * n + 16 * b), gf);
                }
            }
        }
    }
    if (ki > last) return;
    const size_t row = (size_t)(at.tok0 + ki) * a.Hkv + hk;
    // the sign of a negative scale went into k for the scores; q itself entered dK
    store_col<OT, D>((OT*)a.dk + row * D, ak, a.neg ? -a.scale : a.scale);
    store_col<OT, D>((OT*)a.dv + row * D, av, 1.f);
}

template <class OT, int D, int NW>
static hipError_t launch_bwd_t(const PromptArgs& a, hipStream_t stream) {
    constexpr int TB = BT * D * (int)sizeof(OT), LQ = 4 * TB, LK = 4 * TB + 4 * BT * 4;
    const auto fq = k_prompt_dq<OT, D, NW>;
    const auto fk = k_prompt_dkv<OT, D, NW>;
    if (LK > 65536) {
        hipError_t e = hipFuncSetAttribute((const void*)fq, hipFuncAttributeMaxDynamicSharedMemorySize, LQ);
        if (e == hipSuccess) e = hipFuncSetAttribute((const void*)fk, hipFuncAttributeMaxDynamicSharedMemorySize, LK);
        if (e != hipSuccess) return e;
    }
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 32 * NW);
    hipLaunchKernelGGL(fq, dim3((unsigned)(n * a.Hq)), dim3(64 * NW), LQ, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fk, dim3((unsigned)(n * a.Hkv)), dim3(64 * NW), LK, stream, a);
    return hipGetLastError();
}

hipError_t launch_prompt_bwd(const PromptArgs& a, bool bf, hipStream_t stream) {
    if (bf) return a.D == 64 ? launch_bwd_t<bf16, 64, 4>(a, stream) : launch_bwd_t<bf16, 128, 4>(a, stream);
    return a.D == 64 ? launch_bwd_t<float, 64, 4>(a, stream) : launch_bwd_t<float, 128, 4>(a, stream);
}

}  // namespace gdr2
