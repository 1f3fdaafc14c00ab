// Causal attention over whole sequences on gfx950, backward. With P_ij = exp(scale q_i.k_j - lse_i) on what i sees,
//
//     dV = P^T dO    dS_ij = P_ij (dO_i.v_j - delta_i),  delta_i = dO_i.o_i    dQ = scale dS K    dK = scale dS^T Q
//
// dK and dV summed over the query heads that share a key head. Two kernels, one for dQ (a wave owns 32 queries and
// walks their keys) and one for dK and dV (a wave owns 32 keys and walks the queries of all heads that see them), each
// with its sums in registers: every result is added up by one wave in a fixed order, without atomics, for the price of
// forming the scores twice. The first one leaves lse log2(e) and -delta for the second.
//
// Matrix products bound both (seven of them where a single walk with atomics has five): 2 x 4096 tokens, 16 heads of 128
// channels, 465 us together, 1030 TFLOP/s counted as seven products, where a large product alone reaches 1198. Packed
// documents of 64 channels (9 of them, 16 query heads over 4, 2048-token window) 173 us with the sum of the parts: vector
// units busy for 50 % of dQ's cycles and 44 of dK/dV's, matrix cores for 37 and 39, and little of both at once. fp32, 128
// channels (2048 tokens, 8 heads over 2) 338 us: one wave a SIMD, whose tile takes 128 of 160 KB of LDS, with nothing beside
// it: matrix cores busy for 57 and 61 % of the cycles, vector units for 12, 15 and 13 % waited.
#include "gdr2_prompt_device.hpp"

namespace gdr2 {

// ---------------------------------------------------------------- dQ: as the forward, keys in tiles
// (RW x 32 queries a workgroup, S waves for each 32 of them, which share the keys)
template <class OT, int D, int RW, int S, bool EXACT>
__global__ __launch_bounds__(64 * RW * S, (prompt_waves<OT, D>())) void k_prompt_dq(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int NW = RW * S, QT = 32 * RW, BT = tile_rows(S), TB = BT * TL::RB, NB = BT / 32 / S;
    constexpr int BUFS = tile_bufs<OT, D>(S);
    constexpr int ACC = D / 32 * 4096, KB = D / 16, DT = D / 32, AHEAD = sizeof(OT) == 2 ? 4 : 1;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 2 * BUFS * TB);
    poison_lds_done();
    PromptAt at;
    int slot;
    const int hp = prompt_at(a, blockIdx.x, QT, a.Hq, true, at, slot);
    const int hk = hp % a.Hkv, hq = hk * a.G + hp / a.Hkv;
    if (a.cu && a.zero_rest) prompt_zero(a, slot, QT, (OT*)a.dq, a.Hq, hq, D);
    if (!at.any) return;
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = S == 1 ? w : w % RW, sp = S == 1 ? 0 : w / RW;
    const int q0 = at.tile * QT, last = at.len - 1;
    const int wq0 = q0 + 32 * rw, qi = wq0 + (l & 31);
    const long long tok = at.tok0 + min(qi, last);
    const size_t row = (size_t)tok * a.Hq + hq;
    FR qf[D / 16], df[D / 16];
    load_own<OT, D>((const OT*)a.q + tok * a.qs[0] + hq * a.qs[1], a.neg, qf);
    load_own<OT, D>((const OT*)a.dout + row * D, false, df);
    const char* kb = (const char*)((const OT*)a.k + at.tok0 * a.ks[0] + hk * a.ks[1]);
    const char* vb = (const char*)((const OT*)a.v + at.tok0 * a.vs[0] + hk * a.vs[1]);
    const TileLoad<OT, D, BT, NW> lk(a.ks[0] * (int)sizeof(OT), last, w), lv(a.vs[0] * (int)sizeof(OT), last, w);
    const int t0 = max(0, q0 - a.window + 1) / BT, t1 = min(q0 + QT - 1, last) / BT;
    auto fetch = [&](int t) {
        lds_char* b = lds + t % BUFS * 2 * TB;
        lk(kb, t * BT, b);
        lv(vb, t * BT, b + TB);
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
        delta = sum_halves(delta);
    }
    const float lse2 = a.lse[row] * 1.4426950408889634f;
    if (qi <= last && h == 0 && sp == 0) {
        a.lse2[row] = lse2;
        a.delta[row] = -delta;
    }
    f32x16 acc[D / 32], less;  // less: what dP starts from
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
#pragma unroll
    for (int r = 0; r < 16; ++r) less[r] = -delta;
    TL tl;
    for (int t = t0; t <= t1; ++t) {
        tl.fresh();
        if (BUFS == 1 && t > t0) {
            __syncthreads();
            fetch(t);
        }
        wait_vm<0>();
        __syncthreads();
        if (BUFS == 2 && t < t1) fetch(t + 1);
        const int b0 = 32 * NB * sp, k0 = t * BT + b0;
        if (k0 > wq0 + 31 || wq0 > last || k0 + 32 * NB - 1 <= wq0 - a.window) continue;
        const lds_char* kt = lds + t % BUFS * 2 * TB;
        const lds_char* vt = kt + TB;
        const bool part = k0 + 32 * NB - 1 > wq0 || k0 <= wq0 + 31 - a.window;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f32x16 s = zero16(), dp = less;
            auto row = [&](int i) __attribute__((always_inline)) {
                return i < KB ? tl.rows(kt, b0 + 32 * n, 16 * i) : tl.rows(vt, b0 + 32 * n, 16 * (i - KB));
            };
            Pipe<2 * KB, AHEAD, FR> scores;
            scores.start(row);
            scores.run(row, [&](int i, const FR& x) __attribute__((always_inline)) {
                if (i < KB) mma32(s, x, qf[i]);
                else mma32(dp, x, df[i - KB]);
            });
            auto col = [&](int i) __attribute__((always_inline)) {
                return tl.cols(kt, 32 * (i % DT), b0 + 32 * n + 16 * (i / DT));
            };
            Pipe<2 * DT, AHEAD, FR> sums;
            sums.start(col);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale2, -lse2));
                s[r] = p * dp[r];
            }
            if (part) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = qi - (k0 + 32 * n + 8 * (r >> 2) + 4 * h + (r & 3));
                    s[r] = d >= 0 && d < a.window ? s[r] : 0.f;
                }
            }
            FR f[2] = {acc_frag<OT>(s, 0), acc_frag<OT>(s, 1)};
            if constexpr (EXACT)
                if (prompt_few(a, wq0)) {
                    const FR y[2] = {rest_frag(s, 0, f[0]), rest_frag(s, 1, f[1])};
                    Pipe<2 * DT, 1, FR> rest;
                    rest.start(col);
                    rest.run(col, [&](int i, const FR& x) __attribute__((always_inline)) { mma32(acc[i % DT], x, y[i / DT]); });
                }
            sums.run(col, [&](int i, const FR& x) __attribute__((always_inline)) { mma32(acc[i % DT], x, f[i / DT]); });
        }
    }
    if constexpr (S > 1) {
        __syncthreads();
        if (sp > 0) put_acc(lds + ((sp - 1) * RW + rw) * ACC, acc);
        __syncthreads();
        if (sp > 0) return;
        for (int x = 0; x < S - 1; ++x) add_acc(lds + (x * RW + rw) * ACC, 1.f, acc);
    }
    if (qi <= last) store_col<OT, D>((OT*)a.dq + row * D, acc, a.neg ? -a.scale : a.scale);
}

// ---------------------------------------------------------------- dK, dV: queries in tiles
// (RW x 32 keys a workgroup, S waves for each 32 of them, which share the queries)
// Registers leave room for two waves a SIMD at 128 channels, 192 of a lane's 256 being sums and own rows, but for 1 to 3 that
// are spilled outside of the loop, and 5 to 8 that variants with two parts load again inside it (operands two ahead spilled
// more: 503 us for 480), and for three at 64 (packed documents: the backward 181 us with two, 172 with three). The
// scheduling barriers keep the compiler from drawing one phase's operands into the one before, which spilled 24.
template <class OT, int D>
constexpr int dkv_waves() { return sizeof(OT) == 2 && D == 64 ? 3 : prompt_waves<OT, D>(); }
template <class OT, int D, int RW, int S, bool EXACT>
__global__ __launch_bounds__(64 * RW * S, (dkv_waves<OT, D>())) void k_prompt_dkv(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int NW = RW * S, KT = 32 * RW, BT = tile_rows(S), TB = BT * TL::RB, BUF = 2 * TB + 2 * BT * 4, NB = BT / 32 / S;
    constexpr int BUFS = tile_bufs<OT, D>(S);
    constexpr int ACC = D / 32 * 4096, KB = D / 16, DT = D / 32, AHEAD = sizeof(OT) == 2 && D == 64 ? 2 : 1;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, BUFS * BUF);
    poison_lds_done();
    PromptAt at;
    int slot;
    const int hp = prompt_at(a, blockIdx.x, KT, a.Hkv * a.parts, false, at, slot);
    const int hk = hp % a.Hkv, part = hp / a.Hkv;
    const int g0 = a.G * part / a.parts, g1 = a.G * (part + 1) / a.parts;  // its query heads
    if (a.cu && a.zero_rest && a.parts == 1) {
        prompt_zero(a, slot, KT, (OT*)a.dk, a.Hkv, hk, D);
        prompt_zero(a, slot, KT, (OT*)a.dv, a.Hkv, hk, D);
    }
    if (!at.any) return;
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = S == 1 ? w : w % RW, sp = S == 1 ? 0 : w / RW;
    const int k0 = at.tile * KT, last = at.len - 1;
    const int wk0 = k0 + 32 * rw, ki = wk0 + (l & 31);
    const long long tok = at.tok0 + min(ki, last);
    FR kf[D / 16], vf[D / 16];
    load_own<OT, D>((const OT*)a.k + tok * a.ks[0] + hk * a.ks[1], a.neg, kf);
    load_own<OT, D>((const OT*)a.v + tok * a.vs[0] + hk * a.vs[1], false, vf);
    // the query tiles that see any of the workgroup's keys, for each head in turn
    const int t0 = k0 / BT, t1 = (int)min((long long)last, (long long)k0 + KT - 2 + a.window) / BT, nt = t1 - t0 + 1;
    const TileLoad<OT, D, BT, NW> lq(a.qs[0] * (int)sizeof(OT), last, w), ld((long long)a.Hq * TL::RB, last, w);
    int fh = hk * a.G + g0, ft = t0;  // what is read next: head and tile
    auto fetch = [&](int i) {
        const int hq = fh, r0 = ft * BT;
        if (++ft > t1) ft = t0, ++fh;
        lds_char* b = lds + i % BUFS * BUF;
        lq((const char*)((const OT*)a.q + at.tok0 * a.qs[0] + hq * a.qs[1]), r0, b);
        ld((const char*)((const OT*)a.dout + (at.tok0 * a.Hq + hq) * D), r0, b + TB);
#pragma unroll
        for (int x = 0; x < (2 * BT / 64 + NW - 1) / NW; ++x) {
            const int y = x * NW + w;  // which 64 of the 2 BT numbers
            if (y < 2 * BT / 64) {
                const int r = y % (BT / 64) * 64 + l;
                const float* src = (y / (BT / 64) ? a.delta : a.lse2) + (at.tok0 + r0) * a.Hq + hq;
                __builtin_amdgcn_global_load_lds(src + (unsigned)(min(r, last - r0) * a.Hq), (lds_void*)(b + 2 * TB + y * 256), 4, 0, 0);
            }
        }
    };
    fetch(0);
    f32x16 ak[D / 32], av[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) ak[i] = av[i] = zero16();
    const int all = nt * (g1 - g0);
    TL tl;
    for (int i = 0, t = t0; i < all; ++i, t = t == t1 ? t0 : t + 1) {
        tl.fresh();
        if (BUFS == 1 && i > 0) {
            __syncthreads();
            fetch(i);
        }
        wait_vm<0>();
        __syncthreads();
        if (BUFS == 2 && i + 1 < all) fetch(i + 1);
        const lds_char* qt = lds + i % BUFS * BUF;
        const lds_char* dt_ = qt + TB;
        const lds_char* st = qt + 2 * TB;
#pragma unroll
        for (int n_ = 0; n_ < NB; ++n_) {
            const int n = NB * sp + n_, r0 = t * BT + 32 * n;
            if (r0 + 31 < wk0 || r0 > last || r0 - wk0 - 31 >= a.window) continue;
            // (the second parts of queries that see few keys by doing all of it again: registers)
#pragma unroll 1
            for (int again = EXACT && prompt_few(a, r0); again >= 0; --again) {
                asm volatile("" : "+v"(tl.rb), "+v"(tl.cb));  // (addresses formed anew: registers)
                f32x16 s = zero16(), dp;  // dP - delta from the start
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 de = lds_load<f32x4>(st + (BT + 32 * n + 8 * j + 4 * h) * 4);
#pragma unroll
                    for (int x = 0; x < 4; ++x) dp[4 * j + x] = de[x];
                }
                auto row = [&](int i) __attribute__((always_inline)) {
                    return i < KB ? tl.rows(qt, 32 * n, 16 * i) : tl.rows(dt_, 32 * n, 16 * (i - KB));
                };
                Pipe<2 * KB, AHEAD, FR> scores;
                scores.start(row);
                scores.run(row, [&](int i, const FR& x) __attribute__((always_inline)) {
                    if (i < KB) mma32(s, x, kf[i]);
                    else mma32(dp, x, vf[i - KB]);
                });
                auto col = [&](int i) __attribute__((always_inline)) {
                    return tl.cols(i % 2 ? qt : dt_, 32 * (i / 2 % DT), 32 * n + 16 * (i / 2 / DT));
                };
                Pipe<4 * DT, AHEAD, FR> sums;
                sums.start(col);
                const bool mask = r0 < wk0 + 31 || r0 + 31 > last || r0 + 31 - wk0 >= a.window;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 ls = lds_load<f32x4>(st + (32 * n + 8 * j + 4 * h) * 4);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[4 * j + x] = __builtin_amdgcn_exp2f(fmaf(s[4 * j + x], a.scale2, -ls[x]));
                        dp[4 * j + x] *= s[4 * j + x];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (mask) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int q = r0 + 8 * (r >> 2) + 4 * h + (r & 3), d = q - ki;
                        const bool see = d >= 0 && d < a.window && q <= last;
                        s[r] = see ? s[r] : 0.f;
                        dp[r] = see ? dp[r] : 0.f;
                    }
                }
                FR pf[2], gf[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if constexpr (EXACT)
                        if (again) {
                            pf[b] = rest_frag(s, b, acc_frag<OT>(s, b));
                            gf[b] = rest_frag(dp, b, acc_frag<OT>(dp, b));
                            continue;
                        }
                    pf[b] = acc_frag<OT>(s, b);
                    gf[b] = acc_frag<OT>(dp, b);
                }
                sums.run(col, [&](int i, const FR& x) __attribute__((always_inline)) {
                    const int dt = i / 2 % DT, b = i / 2 / DT;
                    if (i % 2) mma32(ak[dt], x, gf[b]);
                    else mma32(av[dt], x, pf[b]);
                });
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if constexpr (S > 1) {
        // one of the two at a time: both together pass the LDS
        __syncthreads();
        if (sp > 0) put_acc(lds + ((sp - 1) * RW + rw) * ACC, ak);
        __syncthreads();
        if (sp == 0)
            for (int x = 0; x < S - 1; ++x) add_acc(lds + (x * RW + rw) * ACC, 1.f, ak);
        __syncthreads();
        if (sp > 0) put_acc(lds + ((sp - 1) * RW + rw) * ACC, av);
        __syncthreads();
        if (sp > 0) return;
        for (int x = 0; x < S - 1; ++x) add_acc(lds + (x * RW + rw) * ACC, 1.f, av);
    }
    if (ki > last) return;
    const size_t row = (size_t)(at.tok0 + ki) * a.Hkv + hk;
    if (a.parts > 1) {
        const size_t tokens = a.cu ? (size_t)a.T : (size_t)a.N * a.T;
        float* pk = a.part + ((size_t)part * tokens * a.Hkv + row) * D;
        store_col<float, D>(pk, ak, 1.f);
        store_col<float, D>(pk + (size_t)a.parts * tokens * a.Hkv * D, av, 1.f);
        return;
    }
    // the sign of a negative scale went into k for the scores; q itself entered dK
    store_col<OT, D>((OT*)a.dk + row * D, ak, a.neg ? -a.scale : a.scale);
    store_col<OT, D>((OT*)a.dv + row * D, av, 1.f);
}

// dK and dV from their parts, in order
template <class OT>
__global__ __launch_bounds__(256) void k_prompt_sum(PromptArgs a) {
    const size_t tokens = a.cu ? (size_t)a.T : (size_t)a.N * a.T, all = tokens * a.Hkv * a.D;
    const size_t e = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= all) return;
    bool rest = false;
    if (a.cu) {
        const int r = (int)(e / ((size_t)a.Hkv * a.D)), b = clamp_int(a.cu[0], 0, a.T);
        rest = r < b || r >= clamp_int(a.cu[a.N], b, a.T);
        if (rest && !a.zero_rest) return;
    }
    f32x4 k = {0.f, 0.f, 0.f, 0.f}, v = k;
    if (!rest)
        for (int p = 0; p < a.parts; ++p) {
            k += *(const f32x4*)(a.part + p * all + e);
            v += *(const f32x4*)(a.part + (a.parts + p) * all + e);
        }
    const float f = a.neg ? -a.scale : a.scale;
    const float x[4] = {k[0] * f, k[1] * f, k[2] * f, k[3] * f}, y[4] = {v[0], v[1], v[2], v[3]};
    st4((OT*)a.dk + e, x);
    st4((OT*)a.dv + e, y);
}

template <class F>
static hipError_t launch_one(F f, long long groups, int threads, int lds, const PromptArgs& a, hipStream_t stream) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(f, dim3((unsigned)groups), dim3((unsigned)threads), lds, stream, a);
    return hipGetLastError();
}
template <class OT, int D, int RW, int S>
static hipError_t launch_dq_t(const PromptArgs& a, hipStream_t stream) {
    constexpr int TILES = 2 * tile_bufs<OT, D>(S) * tile_rows(S) * D * (int)sizeof(OT), JOIN = (S - 1) * RW * (D / 32 * 4096);
    constexpr int LDS = TILES > JOIN ? TILES : JOIN;
    static_assert(LDS <= 160 * 1024, "a compute unit's LDS");
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 32 * RW) * a.Hq;
    constexpr bool BF = sizeof(OT) == 2;
    return launch_one(BF && prompt_exacts(a) ? k_prompt_dq<OT, D, RW, S, BF> : k_prompt_dq<OT, D, RW, S, false>, n, 64 * RW * S, LDS, a, stream);
}
template <class OT, int D, int RW, int S>
static hipError_t launch_dkv_t(const PromptArgs& a, hipStream_t stream) {
    constexpr int TILES = 2 * tile_bufs<OT, D>(S) * tile_rows(S) * (D * (int)sizeof(OT) + 4), JOIN = (S - 1) * RW * (D / 32 * 4096);
    constexpr int LDS = TILES > JOIN ? TILES : JOIN;
    static_assert(LDS <= 160 * 1024, "a compute unit's LDS");
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 32 * RW) * a.Hkv * a.parts;
    constexpr bool BF = sizeof(OT) == 2;
    const hipError_t e = launch_one(BF && prompt_exacts(a) ? k_prompt_dkv<OT, D, RW, S, BF> : k_prompt_dkv<OT, D, RW, S, false>, n, 64 * RW * S, LDS, a, stream);
    if (e != hipSuccess || a.parts == 1) return e;
    const long long all = (a.cu ? (long long)a.T : (long long)a.N * a.T) * a.Hkv * D;
    return launch_one(k_prompt_sum<OT>, (all / 4 + 255) / 256, 256, 0, a, stream);
}

template <class OT, int D>
static hipError_t launch_dq_d(const PromptArgs& a, hipStream_t stream) {
    const long long tasks = prompt_blocks(a.N, a.T, a.cu != nullptr) * a.Hq;
    const int S = prompt_sharing(a, tasks, 1, sizeof(OT));
    if constexpr (sizeof(OT) == 2) {
        // 256 queries a workgroup from two rounds of them on (2 x 4096 tokens, 16 heads 200 us, with 128 queries 214;
        // 64 channels, 9 packed documents, 92 and 73)
        if constexpr (D == 128)
            if (S == 1 && tasks >= 4096 && prompt_length(a.N, a.T, a.cu != nullptr) >= 1024)
                return launch_dq_t<OT, D, 8, 1>(a, stream);
        if (S == 1) return launch_dq_t<OT, D, 4, 1>(a, stream);
        if (S == 2) return launch_dq_t<OT, D, 4, 2>(a, stream);
        return tasks <= 256 ? launch_dq_t<OT, D, 1, 4>(a, stream) : launch_dq_t<OT, D, 2, 4>(a, stream);
    } else {
        if (S == 1) return launch_dq_t<OT, D, 4, 1>(a, stream);
        if (S == 4) return launch_dq_t<OT, D, 1, 4>(a, stream);
        return launch_dq_t<OT, D, 2, 2>(a, stream);
    }
}
template <class OT, int D>
static hipError_t launch_dkv_d(const PromptArgs& a, hipStream_t stream) {
    const long long tasks = prompt_blocks(a.N, a.T, a.cu != nullptr) * a.Hkv * a.parts;
    const int S = prompt_sharing(a, tasks, (a.G + a.parts - 1) / a.parts, sizeof(OT));
    if (S == 1) return launch_dkv_t<OT, D, 4, 1>(a, stream);
    if constexpr (sizeof(OT) == 2) {
        if (S == 2) return launch_dkv_t<OT, D, 2, 2>(a, stream);
        return tasks <= 256 ? launch_dkv_t<OT, D, 1, 4>(a, stream) : launch_dkv_t<OT, D, 2, 4>(a, stream);
    } else {
        if (S == 4) return launch_dkv_t<OT, D, 1, 4>(a, stream);
        return launch_dkv_t<OT, D, 2, 2>(a, stream);
    }
}
template <class OT, int D>
static hipError_t launch_bwd_d(const PromptArgs& a, hipStream_t stream) {
    const hipError_t e = launch_dq_d<OT, D>(a, stream);
    return e == hipSuccess ? launch_dkv_d<OT, D>(a, stream) : e;
}
hipError_t launch_prompt_bwd(const PromptArgs& a, bool bf, hipStream_t stream) {
    if (bf) return a.D == 64 ? launch_bwd_d<bf16, 64>(a, stream) : launch_bwd_d<bf16, 128>(a, stream);
    return a.D == 64 ? launch_bwd_d<float, 64>(a, stream) : launch_bwd_d<float, 128>(a, stream);
}

}  // namespace gdr2
