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
//
// Bound by the matrix products, and by the softmax between them (a wave's tile of 64 keys: 1024 clocks of products of 128
// channels, some 900 of vector work): 16384 tokens, 16 heads over 2 of 128 990 us, 1110 TFLOP/s; 2 x 4096, 16 heads 150 us, 916;
// 9 packed documents, 64 channels, 2048-token window 59 us: there the vector units are busy for 61 % of the cycles and the
// matrix cores for 28, and little of both at once. 24 packed prompts of 17 - 700 tokens 30 us: 784 workgroups where LDS holds
// 512, most of short prompts with waves to spare, and the longest walk 11 tiles one after another; 1.4 waves a SIMD on
// average, vector units busy for 30 % of the cycles and matrix cores for 16.
#include "gdr2_prompt_device.hpp"

namespace gdr2 {

// RW x 32 queries of head hq a workgroup, S waves for each 32 of them, which share the keys; EXACT: queries of few keys
// (prompt_few) in two parts
template <class OT, int D, int RW, int S, bool EXACT>
__device__ __forceinline__ void prompt_fwd(const PromptArgs& a, const PromptAt& at, int hq, int hk, lds_char* lds) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int NW = RW * S, QT = 32 * RW, KT = tile_rows(S), TB = KT * TL::RB, NB = KT / 32 / S;
    constexpr int ACC = D / 32 * 4096;  // bytes of a wave's accumulators
    constexpr int BUFS = tile_bufs<OT, D>(S);
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = S == 1 ? w : w % RW, sp = S == 1 ? 0 : w / RW;
    const int q0 = at.tile * QT, last = at.len - 1;
    const int wq0 = q0 + 32 * rw, qi = wq0 + (l & 31);
    const long long tok = at.tok0 + min(qi, last);
    FR qf[D / 16];
    load_own<OT, D>((const OT*)a.q + tok * a.qs[0] + hq * a.qs[1], a.neg, qf);
    const char* kb = (const char*)((const OT*)a.k + at.tok0 * a.ks[0] + hk * a.ks[1]);
    const char* vb = (const char*)((const OT*)a.v + at.tok0 * a.vs[0] + hk * a.vs[1]);
    const TileLoad<OT, D, KT, NW> lk(a.ks[0] * (int)sizeof(OT), last, w), lv(a.vs[0] * (int)sizeof(OT), last, w);
    // the tiles that any of the workgroup's queries sees
    const int t0 = max(0, q0 - a.window + 1) / KT, t1 = min(q0 + QT - 1, last) / KT;
    auto fetch = [&](int t) {
        lds_char* b = lds + t % BUFS * 2 * TB;
        lk(kb, t * KT, b);
        lv(vb, t * KT, b + TB);
    };
    fetch(t0);
    f32x16 acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
    float m = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};  // the lane's weights, in four chains
    TL tl;
    for (int t = t0; t <= t1; ++t) {
        tl.fresh();
        if (BUFS == 1 && t > t0) {
            __syncthreads();
            fetch(t);
        }
        wait_vm<0>();
        __syncthreads();  // the tile has landed, and everyone is done with the one before
        if (BUFS == 2 && t < t1) fetch(t + 1);
        const int r0 = 32 * NB * sp, k0 = t * KT + r0;  // the wave's keys of the tile
        if (k0 > wq0 + 31 || wq0 > last || k0 + 32 * NB - 1 <= wq0 - a.window) continue;  // it sees nothing of them
        const lds_char* kt = lds + t % BUFS * 2 * TB;
        const lds_char* vt = kt + TB;
        f32x16 s[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) s[n] = zero16();
#pragma unroll
        for (int b = 0; b < D / 16; ++b)
#pragma unroll
            for (int n = 0; n < NB; ++n) mma32(s[n], tl.rows(kt, r0 + 32 * n, 16 * b), qf[b]);
        if constexpr (sizeof(OT) == 2) reads_ahead<D / 16 * NB, 1, 4>();
        if (k0 + 32 * NB - 1 > wq0 || k0 <= wq0 + 31 - a.window) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = qi - (k0 + 32 * n + 8 * (r >> 2) + 4 * h + (r & 3));
                    s[n][r] = d >= 0 && d < a.window ? s[n][r] : -INFINITY;
                }
        }
        const float mx = max_halves(max_acc(s)) * a.scale2;
        // the reference moves only where it would let a weight pass 2^8: sums and weights are relative to it
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] *= al;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * al;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        FR pf[2 * NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[n][r] = __builtin_amdgcn_exp2f(fmaf(s[n][r], a.scale2, -mu));
                sum[r & 3] += s[n][r];
            }
            pf[2 * n] = acc_frag<OT>(s[n], 0);
            pf[2 * n + 1] = acc_frag<OT>(s[n], 1);
        }
        if constexpr (EXACT)
            if (prompt_few(a, wq0)) {
                FR f[2 * NB];
#pragma unroll
                for (int b = 0; b < 2 * NB; ++b) f[b] = rest_frag(s[b / 2], b % 2, pf[b]);
                Pipe<2 * NB * (D / 32), 1, FR> rest;
                auto col = [&](int i) __attribute__((always_inline)) {
                    return tl.cols(vt, 32 * (i % (D / 32)), r0 + 16 * (i / (D / 32)));
                };
                rest.start(col);
                rest.run(col, [&](int i, const FR& x) __attribute__((always_inline)) {
                    mma32(acc[i % (D / 32)], x, f[i / (D / 32)]);
                });
            }
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) mma32(acc[dt], tl.cols(vt, 32 * dt, r0 + 16 * b), pf[b]);
        if constexpr (sizeof(OT) == 2) reads_ahead<D / 16 * NB, 2, 4>();
    }
    float total = sum_halves((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if constexpr (S > 1) {
        // join the waves of the same queries, in their order
        __syncthreads();
        if (sp > 0) {
            lds_char* p = lds + ((sp - 1) * RW + rw) * (ACC + 512);
            put_acc(p, acc);
            lds_store<float>(p + ACC + l * 4, m);
            lds_store<float>(p + ACC + 256 + l * 4, total);
        }
        __syncthreads();
        if (sp > 0) return;
        for (int x = 0; x < S - 1; ++x) {
            const lds_char* p = lds + (x * RW + rw) * (ACC + 512);
            const float mo = lds_load<float>(p + ACC + l * 4), so = lds_load<float>(p + ACC + 256 + l * 4);
            const float mn = fmaxf(m, mo), mu = mn == -INFINITY ? 0.f : mn;
            const float fa = __builtin_amdgcn_exp2f(m - mu), fb = __builtin_amdgcn_exp2f(mo - mu);
            m = mn;
            total = total * fa + so * fb;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * fa;
            add_acc(p, fb, acc);
        }
    }
    if (qi > last) return;
    const float inv = 1.f / total;
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
    if (a.lse && h == 0) a.lse[row] = (m + __log2f(total)) * 0.6931471805599453f;
}

template <class OT, int D, int RW, int S>
__global__ __launch_bounds__(64 * RW * S, (prompt_waves<OT, D>())) void k_prompt_fwd(PromptArgs a) {
    constexpr int QT = 32 * RW;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 2 * tile_bufs<OT, D>(S) * tile_rows(S) * D * (int)sizeof(OT));
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
    if constexpr (sizeof(OT) == 2)
        if (prompt_few(a, at.tile * QT)) return prompt_fwd<OT, D, RW, S, true>(a, at, hq, hk, lds);
    prompt_fwd<OT, D, RW, S, false>(a, at, hq, hk, lds);
}

template <class OT, int D, int RW, int S>
static hipError_t launch_fwd_t(const PromptArgs& a, hipStream_t stream) {
    constexpr int TILES = 2 * tile_bufs<OT, D>(S) * tile_rows(S) * D * (int)sizeof(OT), JOIN = (S - 1) * RW * (D / 32 * 4096 + 512);
    constexpr int LDS = TILES > JOIN ? TILES : JOIN;
    static_assert(LDS <= 160 * 1024, "a compute unit's LDS");
    const auto f = k_prompt_fwd<OT, D, RW, S>;
    if (LDS > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)f, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) return e;
    }
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 32 * RW) * a.Hq;
    hipLaunchKernelGGL(f, dim3((unsigned)n), dim3(64 * RW * S), LDS, stream, a);
    return hipGetLastError();
}

// Long sequences: 256 queries a workgroup, two waves a SIMD that take turns. A wave's tile is a phase of matrix products
// (the weights of the tile before with its values, then this tile's scores) and one of vector work (its softmax), which
// take about as long; the waves 4 .. 7 are a phase behind the waves 0 .. 3, with a barrier between phases, so that on
// each SIMD one wave multiplies while the other is in its softmax. Phase 2 i is the products of tile i (first half), phase
// 2 i + 1 its softmax.
//
// Tiles are three deep in LDS. A load is held at its issue while the compute unit moves what was asked for before, some
// 400 clocks for a wave's share of a tile, so each half sends for its share in its softmax phase: keys of tile i + 2 and
// values of tile i + 1 from phase 2 i on, when what they replace has been read, for phase 2 i + 4.
template <class OT, int D>
__global__ __launch_bounds__(512, 2) void k_prompt_fwd2(PromptArgs a) {
    using FR = typename Frag<OT>::type;
    using TL = Tile32<OT, D>;
    constexpr int NW = 8, QT = 32 * NW, KT = 64, TB = KT * TL::RB;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, 6 * TB);
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
    // queries of few keys, whose walk is short (but for small windows): without turns, in two parts
    if (prompt_few(a, at.tile * QT)) return prompt_fwd<OT, D, 8, 1, true>(a, at, hq, hk, lds);
    const int l = lane_id(), h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q0 = at.tile * QT, last = at.len - 1;
    const int wq0 = q0 + 32 * w, qi = wq0 + (l & 31);
    const long long tok = at.tok0 + min(qi, last);
    FR qf[D / 16];
    load_own<OT, D>((const OT*)a.q + tok * a.qs[0] + hq * a.qs[1], a.neg, qf);
    const char* kb = (const char*)((const OT*)a.k + at.tok0 * a.ks[0] + hk * a.ks[1]);
    const char* vb = (const char*)((const OT*)a.v + at.tok0 * a.vs[0] + hk * a.vs[1]);
    const TileLoad<OT, D, KT, NW> lk(a.ks[0] * (int)sizeof(OT), last, w), lv(a.vs[0] * (int)sizeof(OT), last, w);
    constexpr int LOADS = 2 * decltype(lk)::N;  // of a wave, a tile's keys and values
    const int t0 = max(0, q0 - a.window + 1) / KT, n = min(q0 + QT - 1, last) / KT - t0 + 1;
    TL tl;
    tl.fresh();
    // (past the last tile the last one is sent for again, so that as many loads are under way at every wait)
    auto send_k = [&](int i, int buf) __attribute__((always_inline)) { lk(kb, (t0 + min(i, n - 1)) * KT, lds + buf * TB); };
    auto send_v = [&](int i, int buf) __attribute__((always_inline)) { lv(vb, (t0 + min(i, n - 1)) * KT, lds + (3 + buf) * TB); };
    send_k(0, 0);
    send_k(1, 1);
    send_v(0, 0);
    f32x16 acc[D / 32], s[2];
    FR pf[4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
    float m = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};  // the lane's weights, in four chains
    // tile i is seen by the wave
    auto sees = [&](int i) __attribute__((always_inline)) {
        const int k0 = (t0 + i) * KT;
        return k0 <= wq0 + 31 && wq0 <= last && k0 + KT - 1 > wq0 - a.window;
    };
    // b0: i mod 3, b1 and b2 the two buffers after it (the second is also the one before it)
    auto products = [&](int i, int b0, int b2) __attribute__((always_inline)) {
        const lds_char *kt = lds + b0 * TB, *vt = lds + (3 + b2) * TB;
        __builtin_amdgcn_s_setprio(1);
        if (i > 0 && sees(i - 1)) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) mma32(acc[dt], tl.cols(vt, 32 * dt, 16 * b), pf[b]);
            reads_ahead<D / 8, 2, 4>();
        }
        if (i < n && sees(i)) {
            s[0] = s[1] = zero16();
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
#pragma unroll
                for (int x = 0; x < 2; ++x) mma32(s[x], tl.rows(kt, 32 * x, 16 * b), qf[b]);
            reads_ahead<D / 8, 1, 4>();
        }
        __builtin_amdgcn_s_setprio(0);
    };
    auto softmax = [&](int i) __attribute__((always_inline)) {
        if (!sees(i)) return;
        const int k0 = (t0 + i) * KT;
        if (k0 + KT - 1 > wq0 || k0 <= wq0 + 31 - a.window) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = qi - (k0 + 32 * x + 8 * (r >> 2) + 4 * h + (r & 3));
                    s[x][r] = d >= 0 && d < a.window ? s[x][r] : -INFINITY;
                }
        }
        const float mx = max_halves(max_acc(s)) * a.scale2;
        // the reference moves only where it would let a weight pass 2^8: sums and weights are relative to it
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] *= al;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) acc[j] = acc[j] * al;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[x][r] = __builtin_amdgcn_exp2f(fmaf(s[x][r], a.scale2, -mu));
                sum[r & 3] += s[x][r];
            }
            pf[2 * x] = acc_frag<OT>(s[x], 0);
            pf[2 * x + 1] = acc_frag<OT>(s[x], 1);
        }
    };
    wait_vm<LOADS>();
    sync_lds();
    int b0 = 0, b1 = 1, b2 = 2;
    auto turn = [&]() __attribute__((always_inline)) {
        const int x = b0;
        b0 = b1;
        b1 = b2;
        b2 = x;
    };
    if (w < 4) {
        for (int i = 0; i <= n; ++i) {
            products(i, b0, b2);
            sync_lds();
            send_k(i + 2, b2);
            send_v(i + 1, b1);
            if (i < n) softmax(i);
            wait_vm<LOADS>();
            sync_lds();
            turn();
        }
    } else {
        send_k(2, 2);
        send_v(1, 1);
        sync_lds();
        for (int i = 0; i <= n; ++i) {
            products(i, b0, b2);
            wait_vm<LOADS>();
            sync_lds();
            turn();
            if (i == n) break;
            send_k(i + 3, b2);
            send_v(i + 2, b1);
            softmax(i);
            sync_lds();
        }
    }
    wait_vm<0>();  // no load outlives the workgroup's LDS
    float total = sum_halves((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (qi > last) return;
    const float inv = 1.f / total;
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
    if (a.lse && h == 0) a.lse[row] = (m + __log2f(total)) * 0.6931471805599453f;
}

template <class OT, int D>
static hipError_t launch_fwd2_t(const PromptArgs& a, hipStream_t stream) {
    const long long n = prompt_slots(a.N, a.T, a.cu != nullptr, 256) * a.Hq;
    constexpr int LDS = 6 * 64 * D * (int)sizeof(OT);
    const auto f = k_prompt_fwd2<OT, D>;
    if (LDS > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)f, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(f, dim3((unsigned)n), dim3(512), LDS, stream, a);
    return hipGetLastError();
}

template <class OT, int D>
static hipError_t launch_fwd_d(const PromptArgs& a, hipStream_t stream) {
    const long long blocks = prompt_blocks(a.N, a.T, a.cu != nullptr), tasks = blocks * a.Hq;
    const int S = prompt_sharing(a, tasks, 1, sizeof(OT));
    if constexpr (sizeof(OT) == 2) {
        // the turns of k_prompt_fwd2 from two rounds of its workgroups on (us against those of four waves: 2 x 4096
        // tokens, 16 heads 143 and 165; 16384 tokens 985 and 1048; 8 x 1024 58 and 58; with 64 channels, whose products
        // are half as long as their softmax, 79 and 56)
        if constexpr (D == 128)
            if (S == 1 && tasks >= 4096 && prompt_length(a.N, a.T, a.cu != nullptr) >= 1024)
                return launch_fwd2_t<OT, D>(a, stream);
        // sequences that one tile holds: 64 rows of it, while they are few (29 tokens, 16 heads: 6.5 us, of 128 rows 7.8;
        // 6 x 64 tokens, 64 heads 10.1 and, by waves that do not share, 9.5)
        if (a.T <= 64 && tasks <= 512) return launch_fwd_t<OT, D, 2, 2>(a, stream);
        if (S == 1) return launch_fwd_t<OT, D, 4, 1>(a, stream);
        if (S == 2) return launch_fwd_t<OT, D, 4, 2>(a, stream);
        return tasks <= 256 ? launch_fwd_t<OT, D, 1, 4>(a, stream) : launch_fwd_t<OT, D, 2, 4>(a, stream);
    } else {
        if (S == 1) return launch_fwd_t<OT, D, 4, 1>(a, stream);
        if (S == 4) return launch_fwd_t<OT, D, 1, 4>(a, stream);
        return launch_fwd_t<OT, D, 2, 2>(a, stream);
    }
}
hipError_t launch_prompt_fwd(const PromptArgs& a, bool bf, hipStream_t stream) {
    if (bf) return a.D == 64 ? launch_fwd_d<bf16, 64>(a, stream) : launch_fwd_d<bf16, 128>(a, stream);
    return a.D == 64 ? launch_fwd_d<float, 64>(a, stream) : launch_fwd_d<float, 128>(a, stream);
}

}  // namespace gdr2
