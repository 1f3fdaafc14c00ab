// Attention of a tree of drafted tokens over a paged cache on gfx950, where a key head has more than 32 (draft, head) rows:
// the cache in tiles in LDS, as whole sequences have it (gdr2_prompt.hip), for up to 256 rows at once.
//
// RW waves of 32 rows, S of them on the same rows, each with its 32 keys of a tile of 64 (RW = 2: of 128): a tile comes
// from memory once for all rows, by loads that go from the pages into LDS, sixteen tokens of a page at a time. Rows are
// split over workgroups as in gdr2_attn.hip, a unit of the line being a tile. From the rows' registers straight against
// the cache, four waves side by side (gdr2_tree.hip), 32 sequences of 200 to 16384 tokens with trees of 32, 32 heads over 8
// of 128, took 200 us: every wave loaded and turned all values by itself. So 112 us and 8.4 for the join, 3.6 TB/s of
// the cache. A workgroup's two tiles take 128 of a compute unit's 160 KB of LDS and a third does not fit, so that one tile at
// most is on its way, and none between a tile's arrival and the sending for the next: waves wait for 38 % of their time,
// matrix cores are busy for 22 % of the cycles and vector units for 29.
//
// Weights enter the second product as one bf16 (the step, and trees of up to 32 rows, take them in two parts): o is off by
// 2.3e-3 instead of its own rounding's 1.7e-3. Two parts took 127 us for 118 there, 16.6 for 15.9 (one sequence of 777
// tokens, 12 drafts, 16 heads over 2), 122 for 101 (16 of 4096, 64 drafts, 32 heads over 4), 54 for 44 (64 of 2000, 16 drafts, 32
// heads over 4 of 64): the products of a tile follow its loads.
#include "gdr2_prompt_device.hpp"
#include "gdr2_tree_device.hpp"

namespace gdr2 {

// The mask of 32 tokens from k0 on for one draft (bit e: it sees token k0 + e): context from `lo` on, then the drafts that
// `sees` names, of what `in` names (tokens held, on pages).
__device__ __forceinline__ unsigned tree_mask(int k0, int start, int lo, unsigned long long sees, unsigned in) {
    const int d = k0 - start;  // the draft at token k0; negative: in the context
    unsigned long long m = d >= 0 ? (d < 64 ? sees >> d : 0) : (d > -32 ? sees << -d : 0);
    if (d < 0) {
        unsigned ctx = d <= -32 ? ~0u : (1u << -d) - 1;
        const int skip = lo - k0;
        if (skip > 0) ctx = skip < 32 ? ctx & (~0u << skip) : 0;
        m |= ctx;
    }
    return (unsigned)m & in;
}

template <int D, int RW, int S, int KT>
struct TreeWide {
    using TL = Tile32<bf16, D>;
    static constexpr int KB = D / 16, DT = D / 32, NW = RW * S, TB = KT * TL::RB, NB = KT / 32 / S, GR = KT / 16;
    // tiles in LDS, all but one on their way: one ahead alone leaves the memory's latency longer than a tile's work
    static constexpr int NBUF = 8 * TB <= 131072 ? 4 : 2;
    // Half of the waves send for a tile after their scores: loads are held at their issue while the memory is busy with
    // earlier ones, and the other half multiplies meanwhile. 32 ragged trees of 32 drafts, 32 heads over 8: 126 us, 123 so;
    // but with 64 rows a key head (64 sequences of 2000, 16 drafts) 118, and 122 so, and tiles of 64 tokens gain nothing.
    static constexpr bool LATE = RW == 4 && KT == 128;
    static constexpr int ACC = D / 32 * 4096, TILES = NBUF * 2 * TB, JOIN = (S - 1) * RW * (ACC + 512);
    static constexpr int LDS = TILES > JOIN ? TILES : JOIN;

    static constexpr int ALL = TB / 1024, RPI = 64 / TL::NCH, N = (ALL + NW - 1) / NW;  // load instructions of 1 KB
    static constexpr int LOADS = 2 * N;
    static_assert(ALL % NW == 0, "as many loads for each wave");

    // The page of the sixteen tokens from tok on, negative where there is none; by a scalar load, which does not wait
    // behind the tiles on their way.
    static __device__ __forceinline__ int page_of(const TreeArgs& a, int b, int tok, const TreeSpan& sp) {
        typedef const __attribute__((address_space(4))) int cint;
        cint* row = (cint*)(uintptr_t)(a.c.table + (size_t)b * a.c.max_pages);
        const int p = row[min(tok, sp.hi - 1) >> a.c.shift];
        return tok < sp.hi && (unsigned)p < (unsigned)a.c.pages ? p : -1;
    }
    // Sends for tile t's keys and values. Returns which of its groups of sixteen tokens lie on pages.
    static __device__ __forceinline__ unsigned fetch(const TreeArgs& a, int b, int t, int hk, const TreeSpan& sp,
                                                     lds_char* buf, int w) {
        const int l = lane_id(), lr = l / TL::NCH;  // the lane's row of an instruction
        int pg[N];
        unsigned ok = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) pg[i] = page_of(a, b, t * KT + (i * NW + w) * RPI / 16 * 16, sp);
#pragma unroll
        for (int g = 0; g < GR; ++g) ok |= (page_of(a, b, t * KT + 16 * g, sp) >= 0 ? 1u : 0u) << g;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int n = i * NW + w, r = n * RPI, in = (t * KT + r) & (a.c.page - 1);
            const long long p = max(0, pg[i]);
            const unsigned piece = ((l % TL::NCH) ^ tile_f<TL::NCH>(r + lr)) * 16;
            const char* kp = (const char*)((const bf16*)a.c.k + p * a.c.ks[0] + in * a.c.ks[1] + hk * a.c.ks[2]);
            const char* vp = (const char*)((const bf16*)a.c.v + p * a.c.vs[0] + in * a.c.vs[1] + hk * a.c.vs[2]);
            __builtin_amdgcn_global_load_lds(kp + lr * a.c.ks[1] * 2 + piece, (lds_void*)(buf + n * 1024), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(vp + lr * a.c.vs[1] * 2 + piece, (lds_void*)(buf + TB + n * 1024), 16, 0, 0);
        }
        return ok;
    }

    // Tiles i0 .. i0 + n - 1 of a row; whole: all of it, finished here, else its sums go to `part`: the accumulators as
    // they are held, 16 bytes a lane, then maxima and weights.
    static __device__ __forceinline__ void run(const TreeArgs& a, int b, int hr, const TreeSpan& sp, int i0, int n,
                                               bool whole, float* part, lds_char* lds) {
        const int l = lane_id(), li = l & 31, h = l >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int rw = S == 1 ? w : w % RW, sh = S == 1 ? 0 : w / RW;
        const int hk = hr / a.nb, blk = hr % a.nb, rows = a.T * a.G;
        const int c = (blk * RW + rw) * 32 + li, cc = min(c, rows - 1), dr = cc / a.G;
        const int t0 = sp.u0 + i0, work = sp.hi > sp.lo ? n : 0;
        const TreeLane tl = tree_lane(a, b);
        const size_t row = ((size_t)b * a.T + dr) * a.Hq + hk * a.G + cc % a.G;
        bf16x8 qf[D / 16];
        load_own<bf16, D>((const bf16*)a.q + row * D, a.neg, qf);
        const bool one = (tl.all >> dr) & 1;
        const unsigned long long sees = __shfl(tl.sees, dr);
        const int depth = __shfl(tl.depth, dr);
        const int lo = !one ? 0x7fffffff : a.window > 0 ? (int)max(0ll, (long long)sp.start + depth + 1 - a.window) : 0;
        // first token that the deepest draft sees
        const int lo_in = a.window > 0 ? (int)max(0ll, (long long)sp.start + a.T - a.window) : 0;
        f32x16 acc[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = zero16();
        float m = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};
        unsigned okq = 0;  // which groups of the tiles under way lie on pages, a byte a buffer
        auto send = [&](int i) __attribute__((always_inline)) {
            const int x = i % NBUF;
            okq = (okq & ~(255u << (8 * x))) | (fetch(a, b, t0 + i, hk, sp, lds + x * 2 * TB, w) << (8 * x));
        };
        for (int i = 0; i < NBUF - 1 && i < work; ++i) send(i);
        TL tf;
        for (int i = 0; i < work; ++i) {
            tf.fresh();
            if (i + NBUF - 2 < work) wait_vm<(NBUF - 2) * LOADS>();
            else wait_vm<0>();
            __syncthreads();  // the tile has landed, and everyone is done with the one before
            const int k0 = (t0 + i) * KT;
            const unsigned okp = (okq >> (8 * (i % NBUF))) & 255u;
            const bool more = i + NBUF - 1 < work;
            if (more && !(LATE && w >= NW / 2)) send(i + NBUF - 1);
            lds_char* kt = lds + i % NBUF * 2 * TB;
            lds_char* vt = kt + TB;
            const bool mask = k0 < lo_in || k0 + KT > sp.start || okp != (1u << GR) - 1;
            if (mask) {
                // what no draft sees has a zero value, whatever the cache holds there
                for (int e = threadIdx.x; e < TB / 16; e += 64 * NW) {
                    const int r = e / TL::NCH, tok = k0 + r, d = tok - sp.start;
                    const bool any = tok >= sp.lo && tok < sp.hi && ((okp >> (r / 16)) & 1) &&
                                     (d < 0 || ((tl.all >> (d & 63)) & 1));
                    if (!any) lds_store<f32x4>(vt + e * 16, f32x4{0.f, 0.f, 0.f, 0.f});
                }
                __syncthreads();
            }
            const int r0 = 32 * NB * sh;
            f32x16 s[NB];
#pragma unroll
            for (int x = 0; x < NB; ++x) s[x] = zero16();
            auto row = [&](int i) __attribute__((always_inline)) { return tf.rows(kt, r0 + 32 * (i % NB), 16 * (i / NB)); };
            Pipe<KB * NB, 4, bf16x8> scores;
            scores.start(row);
            scores.run(row, [&](int i, const bf16x8& x) __attribute__((always_inline)) { mma32(s[i % NB], x, qf[i / NB]); });
            if constexpr (LATE) {
                __builtin_amdgcn_sched_barrier(0);
                if (more && w >= NW / 2) send(i + NBUF - 1);
            }
            if (mask) {
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    const int k = k0 + r0 + 32 * x, left = sp.hi - k, skip = sp.lo - k;
                    unsigned in = left <= 0 ? 0 : left < 32 ? (1u << left) - 1 : ~0u;
                    if (skip > 0) in = skip < 32 ? in & (~0u << skip) : 0;
                    const int g = (r0 + 32 * x) / 16;
                    if (!((okp >> g) & 1)) in &= 0xffff0000u;
                    if (!((okp >> (g + 1)) & 1)) in &= 0xffffu;
                    const unsigned v = tree_mask(k, sp.start, lo, sees, in) >> (4 * h);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[x][r] = (v >> (8 * (r >> 2) + (r & 3))) & 1 ? s[x][r] : -INFINITY;
                }
            }
            const float mx = max_halves(max_acc(s)) * a.scale2;
            // the reference moves only where it would let a weight pass 2^8
            if (__any(mx > m + 8.f)) {
                const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
                m = mn;
#pragma unroll
                for (int y = 0; y < 4; ++y) sum[y] *= al;
#pragma unroll
                for (int y = 0; y < D / 32; ++y) acc[y] = acc[y] * al;
            }
            const float mu = m == -INFINITY ? 0.f : m;
            bf16x8 pf[2 * NB];
#pragma unroll
            for (int x = 0; x < NB; ++x) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[x][r] = __builtin_amdgcn_exp2f(fmaf(s[x][r], a.scale2, -mu));
                    sum[r & 3] += s[x][r];
                }
                pf[2 * x] = acc_frag<bf16>(s[x], 0);
                pf[2 * x + 1] = acc_frag<bf16>(s[x], 1);
            }
            auto col = [&](int i) __attribute__((always_inline)) { return tf.cols(vt, 32 * (i % DT), r0 + 16 * (i / DT)); };
            Pipe<2 * NB * DT, 4, bf16x8> sums;
            sums.start(col);
            sums.run(col, [&](int i, const bf16x8& x) __attribute__((always_inline)) { mma32(acc[i % DT], x, pf[i / DT]); });
        }
        float total = one ? sum_halves((sum[0] + sum[1]) + (sum[2] + sum[3])) : 0.f;
        if (!one) m = -INFINITY;  // padding sees nothing
        if constexpr (S > 1) {
            __syncthreads();
            if (sh > 0) {
                lds_char* p = lds + ((sh - 1) * RW + rw) * (ACC + 512);
                put_acc(p, acc);
                lds_store<float>(p + ACC + l * 4, m);
                lds_store<float>(p + ACC + 256 + l * 4, total);
            }
            __syncthreads();
            if (sh > 0) return;
            for (int x = 0; x < S - 1; ++x) {
                const lds_char* p = lds + (x * RW + rw) * (ACC + 512);
                const float mo = lds_load<float>(p + ACC + l * 4), so = lds_load<float>(p + ACC + 256 + l * 4);
                const float mn = fmaxf(m, mo), mu = mn == -INFINITY ? 0.f : mn;
                const float fa = __builtin_amdgcn_exp2f(m - mu), fb = __builtin_amdgcn_exp2f(mo - mu);
                m = mn;
                total = total * fa + so * fb;
#pragma unroll
                for (int y = 0; y < D / 32; ++y) acc[y] = acc[y] * fa;
                add_acc(p, fb, acc);
            }
        }
        if (!whole) {
            float* p = part + (size_t)rw * (32 * D);
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(f32x4*)(p + ((dt * 4 + j) * 64 + l) * 4) =
                        f32x4{acc[dt][4 * j], acc[dt][4 * j + 1], acc[dt][4 * j + 2], acc[dt][4 * j + 3]};
            if (h == 0) {
                float* q = part + (size_t)RW * 32 * D + 2 * (rw * 32 + li);
                q[0] = m;
                q[1] = total;
            }
            return;
        }
        if (c >= rows) return;
        const float inv = total == 0.f ? 0.f : 1.f / total;  // nothing visible: a row of zeros
        if (!one) {
#pragma unroll
            for (int y = 0; y < D / 32; ++y) acc[y] = zero16();
        }
        store_col<bf16, D>((bf16*)a.o + row * D, acc, inv);
        if (a.lse && h == 0) a.lse[row] = total == 0.f ? -INFINITY : (m + __log2f(total)) * 0.6931471805599453f;
    }
};

template <int D, int RW, int S, int KT, bool SPLIT>
__global__ __launch_bounds__(64 * RW * S, 2) void k_tree_wide(TreeArgs a) {
    using TW = TreeWide<D, RW, S, KT>;
    extern __shared__ __align__(16) char smem[];
    lds_char* lds = (lds_char*)smem;
    poison_lds(lds, TW::LDS);
    poison_lds_done();
    const int HR = a.Hkv * a.nb;
    if constexpr (!SPLIT) {
        const int b = blockIdx.x / HR, hr = blockIdx.x % HR;
        const TreeSpan sp = tree_span<KT>(a, b);
        TW::run(a, b, hr, sp, 0, sp.units, true, nullptr, lds);
        return;
    }
    const TreeLine line = tree_line<KT>(a);
    unsigned t = blockIdx.x * line.share;
    int* head = tree_heads(a) + 4 * blockIdx.x;  // the row that begins here and goes on behind the run, for the join
    if (t >= line.total) {
        if (threadIdx.x == 0) head[2] = -1;
        return;
    }
    const unsigned tend = min(t + line.share, line.total);
    TreeAt f = tree_find<KT>(a, line, t);
    while (t < tend) {
        const int len = f.sp.units + a.cost;
        const int hr = (t - f.at) / len;
        const unsigned r0 = f.at + (unsigned)hr * len, r1 = min(r0 + len, tend);
        const int i0 = max(0, (int)(t - r0) - a.cost), i1 = max(0, (int)(r1 - r0) - a.cost);
        if (i1 > i0) {
            const bool whole = i1 - i0 == f.sp.units;
            float* part = a.part + (size_t)(2 * blockIdx.x + (i0 > 0 ? 0 : 1)) * ((size_t)32 * RW * (D + 4));
            TW::run(a, f.b, hr, f.sp, i0, i1 - i0, whole, part, lds);
            __syncthreads();
        }
        if (r1 == tend && threadIdx.x == 0) {
            const bool on = i1 > i0 && i0 == 0 && i1 < f.sp.units;
            head[0] = f.b;
            head[1] = hr;
            head[2] = on ? (int)((r0 + len - 1) / line.share) : -1;  // the last run that has a part of it
        }
        t = r1;
        if (t < tend && t == f.at + (unsigned)len * HR) {
            f.at = t;
            f.sp = tree_span<KT>(a, ++f.b);
        }
    }
}

// Joins the rows that cross workgroups (see k_tree_join), four channels of a row a thread, in the layout that the parts
// are left in; four parts' loads at a time.
template <int D, int RW>
__global__ __launch_bounds__(256) void k_tree_wide_join(TreeArgs a) {
    const unsigned w0 = blockIdx.x;
    const int* head = tree_heads(a) + 4 * w0;
    const int b = head[0], hr = head[1];
    if (head[2] < 0) return;
    const unsigned w1 = head[2];
    constexpr size_t stride = (size_t)32 * RW * (D + 4);
    const int e = blockIdx.y * 256 + threadIdx.x;  // (wave, piece, lane)
    const int l = e & 63, piece = (e >> 6) % (D / 8), rw = e / (8 * D), r = 32 * rw + (l & 31);
    const int c = hr % a.nb * (32 * RW) + r;
    if (c >= a.T * a.G) return;
    float M = -INFINITY, L = 0.f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    for (unsigned w = w0; w <= w1; w += 4) {
        float m[4], s[4];
        f32x4 y[4];
#pragma unroll
        for (unsigned i = 0; i < 4; ++i) {
            const unsigned z = min(w + i, w1);
            const float* p = a.part + (size_t)(2 * z + (z == w0 ? 1 : 0)) * stride;
            m[i] = p[(size_t)32 * RW * D + 2 * r];
            s[i] = p[(size_t)32 * RW * D + 2 * r + 1];
            y[i] = *(const f32x4*)(p + (size_t)4 * e);
        }
#pragma unroll
        for (unsigned i = 0; i < 4; ++i) {
            if (w + i > w1) break;
            const float mn = fmaxf(M, m[i]), mu = mn == -INFINITY ? 0.f : mn;
            const float fa = __builtin_amdgcn_exp2f(M - mu), fb = __builtin_amdgcn_exp2f(m[i] - mu);
            x = x * fa + y[i] * fb;
            L = L * fa + s[i] * fb;
            M = mn;
        }
    }
    const size_t row = ((size_t)b * a.T + c / a.G) * a.Hq + hr / a.nb * a.G + c % a.G;
    const float fl = L == 0.f ? 0.f : 1.f / L;
    const float ov[4] = {L == 0.f ? 0.f : x[0] * fl, L == 0.f ? 0.f : x[1] * fl, L == 0.f ? 0.f : x[2] * fl,
                         L == 0.f ? 0.f : x[3] * fl};
    st4((bf16*)a.o + row * D + 32 * (piece / 4) + 8 * (piece % 4) + 4 * (l >> 5), ov);
    if (a.lse && piece == 0 && l < 32) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
}

template <int D, int RW, int S, int KT>
static hipError_t launch_wide_t(const TreeArgs& a, hipStream_t stream) {
    using TW = TreeWide<D, RW, S, KT>;
    const auto one = k_tree_wide<D, RW, S, KT, false>, line = k_tree_wide<D, RW, S, KT, true>;
    // One row a workgroup, without a second kernel, where no row can pass 512 tokens. Few rows end sooner split, many whole; us,
    // whole and split, 12 drafts, 16 heads over 2 of 128: 1 x 400 tokens 18.6 and 15.0, 8 x 400 18.9 and 16.4, 64 x 400 19.7 and
    // 24.7; 1 x 777 28.4 and 16.1, 8 x 777 29.0 and 18.1, 64 x 777 27.3 and 31.2; 32 drafts, 32 heads over 8: 8 x 400 19.9 and
    // 22.9, 64 x 400 43 and 48, 64 x 777 60 and 65
    const long long rows = (long long)a.B * a.Hkv * a.nb;
    const bool whole = tree_max_units(a) <= 512 / KT && rows < (1LL << 32) / (64 * RW * S);
    if (TW::LDS > 65536) {
        const hipError_t e = hipFuncSetAttribute(whole ? (const void*)one : (const void*)line,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, TW::LDS);
        if (e != hipSuccess) return e;
    }
    if (whole) {
        hipLaunchKernelGGL(one, dim3((unsigned)rows), dim3(64 * RW * S), TW::LDS, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(line, dim3(a.wgs), dim3(64 * RW * S), TW::LDS, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_tree_wide_join<D, RW>), dim3((unsigned)(a.wgs - 1), RW * D / 32), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <int D>
static hipError_t launch_wide_d(const TreeArgs& a, hipStream_t stream) {
    if (a.rg == 2) return launch_wide_t<D, 2, 4, 128>(a, stream);
    if (a.rg == 8) return launch_wide_t<D, 8, 1, 64>(a, stream);
    return a.unit == 128 ? launch_wide_t<D, 4, 2, 128>(a, stream) : launch_wide_t<D, 4, 2, 64>(a, stream);
}
hipError_t launch_tree_wide(const TreeArgs& a, hipStream_t stream) {
    return a.D == 64 ? launch_wide_d<64>(a, stream) : launch_wide_d<128>(a, stream);
}

}  // namespace gdr2
