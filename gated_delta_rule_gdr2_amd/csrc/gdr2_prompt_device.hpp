// Device building blocks of attention over whole sequences: 32x32 matrix products and the tiles they read.
//
// Products are built from 32x32 output tiles with 16-deep K blocks: one v_mfma_f32_32x32x16_bf16, or eight
// v_mfma_f32_32x32x2_f32. Lane l = li + 32 h (li = l % 32, h = l / 32) holds 8 elements of an operand: row (A) or
// column (B) li, and K indices 8 h + e in the contiguous order, or 8 (e / 4) + 4 h + e % 4 in the accumulator's. An
// accumulator holds rows 8 (r / 4) + 4 h + r % 4, r = 0 .. 15, of column li; so registers 8 b .. 8 b + 7 are, in the
// accumulator's order, the B operand of the K block 16 b .. 16 b + 15: scores become weights and enter the next
// product where they stand.
//
// A 32x32 product takes 32 clocks for two operands of 16 bytes a lane, a 16x16x32 one 16 clocks: half the LDS
// traffic, which with 16x16 tiles would be what bounds these kernels.
#pragma once
#include "gdr2_device.hpp"
#include "gdr2_prompt.hpp"

namespace gdr2 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void mma32(f32x16& acc, const bf16x8& a, const bf16x8& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma32(f32x16& acc, const f32x8& a, const f32x8& b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    return x;
}

// Tiles in LDS: rows of D elements, their 16-byte chunks permuted by an XOR with tile_f(row). A 16-byte read is served
// in passes of 16 lanes, an 8-byte one of 32 (gdr2_device.hpp); the row reads of a 32x32 operand (row li, chunk
// c + h) have in a pass the rows whose bits 4..2 have even (odd) parity, and the transposing reads four rows and four
// chunks. Both cover distinct banks with
//   16 chunks a row: f(r) = 4 (r mod 4) + (r / 4 mod 4)     8 chunks: f(r) = 4 (r / 2 mod 2) + (r / 4 mod 4)
// (fp32, 32 chunks: as 16; its transposing reads are single floats and two lanes share a bank).
template <int NCH>
__device__ __forceinline__ int tile_f(int r) {
    static_assert(NCH == 8 || NCH == 16 || NCH == 32, "tiles have 8, 16 or 32 chunks a row");
    return NCH == 8 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : 4 * (r & 3) + ((r >> 2) & 3);
}
// A lane's addresses are an XOR of a part that belongs to the lane and one that belongs to the operand: left to itself
// the compiler keeps one address for each operand over the whole loop, some thirty registers; from lane parts that it
// cannot trace back to the thread index (fresh) it forms them where they are used, one instruction each.
template <class OT, int D>
struct Tile32 {
    static constexpr int ES = (int)sizeof(OT), EPC = 16 / ES, NCH = D / EPC, RB = D * ES;  // row bytes
    int rb, cb;  // lane parts of row and transposed reads

    __device__ __forceinline__ void fresh() {
        int l = lane_id();
        asm volatile("" : "+v"(l));
        const int li = l & 31, h = l >> 5;
        if constexpr (ES == 2) {
            const int r4 = (l & 15) >> 2;  // row of four
            rb = li * RB + ((h ^ tile_f<NCH>(li)) * 16);
            cb = (4 * h + r4) * RB + (((2 * ((l >> 4) & 1) + ((l & 3) >> 1)) ^ tile_f<NCH>(4 * h + r4)) * 16) + 8 * (l & 1);
        } else {
            rb = li * RB + (((2 * h) ^ tile_f<NCH>(li)) * 16);
            cb = 4 * h * RB + (((li >> 2) ^ h) * 16) + (li & 3) * 4;
        }
    }
    // A operand of the K block k0 .. k0 + 15, rows r0 + li (r0 a multiple of 32), contiguous K order
    __device__ __forceinline__ typename Frag<OT>::type rows(const lds_char* t, int r0, int k0) const {
        const lds_char* p = t + r0 * RB;
        if constexpr (ES == 2) {
            return lds_load<bf16x8>(p + (rb ^ (k0 * ES)));
        } else {
            const f32x4 x0 = lds_load<f32x4>(p + (rb ^ (k0 * ES))), x1 = lds_load<f32x4>(p + (rb ^ (k0 * ES + 16)));
            return __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // A operand of the transposed tile: rows are the tile's columns c0 + li (c0 a multiple of 32), the K block its rows
    // k0 .. k0 + 15 in the accumulator's order
    __device__ __forceinline__ typename Frag<OT>::type cols(const lds_char* t, int c0, int k0) const {
        const lds_char* p = t + k0 * RB;
        if constexpr (ES == 2) {
            const bf16x4 v0 = lds_read_tr16_now(p + (cb ^ (c0 * ES))), v1 = lds_read_tr16_now(p + (cb ^ (c0 * ES + 32)) + 8 * RB);
            return __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typename Frag<OT>::type f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = lds_load<float>(p + (cb ^ (c0 * ES) ^ ((4 * (e & 3) + 2 * (e >> 2)) * 16)) + (8 * (e >> 2) + (e & 3)) * RB);
            return f;
        }
    }
};

// Rows of a matrix (row stride rs bytes, rows 0 .. last) in tiles of R into LDS by NW waves, this one being wave w: 1 KB an
// instruction. An instruction's first row is the wave's to know, and the permutation of its chunks repeats after PER
// instructions: the lane's share of the address is formed once. (Formed at each instruction, a 64-row tile of queries and
// of their gradients kept each wave of the backward 1280 clocks.) A tile that reaches past the last row forms all anew, and
// so does any of rows so far apart that the lane's share would pass 32 bits.
template <class OT, int D, int R, int NW>
struct TileLoad {
    using TL = Tile32<OT, D>;
    static constexpr int ALL = R * TL::RB / 1024, N = (ALL + NW - 1) / NW, RPI = 64 / TL::NCH;
    static constexpr int PER = NW * RPI % 16 == 0 ? 1 : 2;  // tile_f goes by the row modulo 16
    static_assert(R * TL::RB % 1024 == 0 && 2 * NW * RPI % 16 == 0, "whole rows an instruction");
    long long rs;
    int last, quick, w;  // quick: the last row of tiles that are not formed anew
    unsigned off[PER];

    __device__ __forceinline__ int row(int l, int i) const { return (i * NW + w) * RPI + l / TL::NCH; }
    __device__ __forceinline__ unsigned piece(int l, int i) const { return ((l % TL::NCH) ^ tile_f<TL::NCH>(row(l, i))) * 16; }
    __device__ __forceinline__ TileLoad(long long rs_, int last_, int w_) : rs(rs_), last(last_), w(w_) {
        quick = rs < (1 << 29) ? last : -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) off[i] = lane_id() / TL::NCH * (unsigned)rs + piece(lane_id(), i);
    }
    __device__ __forceinline__ void operator()(const char* base, int row0, lds_char* t) const {
        auto send = [&](const char* src, int i) __attribute__((always_inline)) {
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(t + (i * NW + w) * 1024), 16, 0, 0);
        };
        if (row0 + R - 1 <= quick) {
            const char* b = base + ((long long)row0 + w * RPI) * rs;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (ALL % NW == 0 || i * NW + w < ALL) send(b + (long long)(i * NW * RPI) * rs + off[i % PER], i);
        } else {
            int l = lane_id();
            asm volatile("" : "+v"(l));  // or these addresses take registers from the whole walk
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (ALL % NW == 0 || i * NW + w < ALL)
                    send(base + (long long)max(0, min(row0 + row(l, i), last)) * rs + piece(l, i), i);
        }
    }
};

// Order of a block of STEPS matrix products with R LDS reads each: the reads run AHEAD products before their use. Left
// to itself the compiler reads each operand just before its product and waits for it.
template <int STEPS, int R, int AHEAD>
__device__ __forceinline__ void reads_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, R * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < STEPS - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

// STEPS matrix products whose A operands are read from LDS AHEAD of them, in the order that is written here: asked for by
// groups of kinds alone (reads_ahead), the compiler takes the product whose operand it has just read, where there are
// two chains of them or registers are short, and waits for it (training step's backward 487 us so, 480 in order). Vector
// and scalar work may move across. start: the first reads, for vector work to cover.
template <int STEPS, int AHEAD, class FR>
struct Pipe {
    FR x[AHEAD + 1];
    template <class R>
    __device__ __forceinline__ void start(R read) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = read(i);
        __builtin_amdgcn_sched_barrier(0x6);
    }
    template <class R, class M>
    __device__ __forceinline__ void run(R read, M mul) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (i + AHEAD < STEPS) x[(i + AHEAD) % (AHEAD + 1)] = read(i + AHEAD);
            __builtin_amdgcn_sched_barrier(0x6);
            mul(i, x[i % (AHEAD + 1)]);
            __builtin_amdgcn_sched_barrier(0x6);
        }
    }
};

// B operands of a wave's own 32 rows, all K blocks, straight from memory: row p (this lane's), contiguous K order.
template <class OT, int D>
__device__ __forceinline__ void load_own(const OT* p, bool neg, typename Frag<OT>::type (&f)[D / 16]) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int kb = 0; kb < D / 16; ++kb) {
        f[kb] = *(const typename Frag<OT>::type*)(p + 16 * kb + 8 * h);
        if (neg) f[kb] = -f[kb];
    }
}
// registers 8 b .. 8 b + 7 of an accumulator as the B operand of K block b
template <class OT>
__device__ __forceinline__ typename Frag<OT>::type acc_frag(const f32x16& x, int b) {
    typename Frag<OT>::type f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_ot<OT>(x[8 * b + e]);
    return f;
}
// what the rounding of f = acc_frag(x, b) left over, as an operand too
__device__ __forceinline__ bf16x8 rest_frag(const f32x16& x, int b, const bf16x8& f) {
    bf16x8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (bf16)(x[8 * b + e] - (float)f[e]);
    return y;
}
// Queries of few keys, from q0 on (prompt_exacts).
__device__ __forceinline__ bool prompt_few(const PromptArgs& a, int q0) { return q0 < 64 || a.window <= 64; }
// this lane's column of D rows, held in accumulators, times f: four consecutive elements at a time
template <class OT, int D>
__device__ __forceinline__ void store_col(OT* p, const f32x16 (&acc)[D / 32], float f) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x[4] = {acc[dt][4 * j] * f, acc[dt][4 * j + 1] * f, acc[dt][4 * j + 2] * f, acc[dt][4 * j + 3] * f};
            st4(p + 32 * dt + 8 * j + 4 * h, x);
        }
}
// waves a SIMD that a kernel's registers have to leave room for
template <class OT, int D>
constexpr int prompt_waves() { return sizeof(OT) == 4 && D == 128 ? 1 : 2; }

// Waves side by side (S of them) on the same rows, each with its part of the other axis: their sums come together
// through LDS, which everyone is done with. A wave's accumulators as 16 bytes a lane, one after another.
template <int N>
__device__ __forceinline__ void put_acc(lds_char* p, const f32x16 (&acc)[N]) {
    const int l = lane_id();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            lds_store<f32x4>(p + (4 * i + j) * 1024 + l * 16,
                             f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]});
}
template <int N>
__device__ __forceinline__ void add_acc(const lds_char* p, float f, f32x16 (&acc)[N]) {
    const int l = lane_id();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 x = lds_load<f32x4>(p + (4 * i + j) * 1024 + l * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][4 * j + e] += x[e] * f;
        }
}
// rows of a tile of the other axis: two blocks of 32 for a wave alone, one or two for each of several
constexpr int tile_rows(int S) { return S == 4 ? 128 : 64; }
// Tiles of each kind in LDS, the next one on its way while one is worked on; of 128 rows of 512 bytes there is room for one.
// (4 waves on 32 rows so, 2048 tokens, 8 heads over 2 of 128, fp32: 103 and 336 us forward and backward; 2 waves on 64
// rows with two tiles of 64 154 and 508.)
template <class OT, int D>
constexpr int tile_bufs(int S) { return sizeof(OT) == 4 && D == 128 && S == 4 ? 1 : 2; }
// the larger, or the sum, of this lane's value and the other half wave's of the same column, by an exchange of half waves
// in the vector unit
__device__ __forceinline__ float max_halves(float x) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// largest value of accumulators, in four chains: one chain of dependent instructions would take twice as long
template <int N>
__device__ __forceinline__ float max_acc(const f32x16 (&s)[N]) {
    float m[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        m[c] = fmaxf(s[0][c], s[0][4 + c]);
        m[c] = fmaxf(fmaxf(m[c], s[0][8 + c]), s[0][12 + c]);
#pragma unroll
        for (int n = 1; n < N; ++n) {
            m[c] = fmaxf(fmaxf(m[c], s[n][c]), s[n][4 + c]);
            m[c] = fmaxf(fmaxf(m[c], s[n][8 + c]), s[n][12 + c]);
        }
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The sequence tile a workgroup works on.
struct PromptAt {
    long long tok0;  // the sequence's first token
    int len, tile;   // its tokens; which of its tiles
    bool any;        // false: a spare slot
};
__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
// Packed sequence s: its first token and tokens. cu is data of the caller's that no host check can see, so its entries
// are held inside the tensors here.
__device__ __forceinline__ void prompt_seq(const PromptArgs& a, int s, int& tok0, int& len) {
    tok0 = clamp_int(a.cu[s], 0, a.T);
    len = clamp_int(a.cu[s + 1], tok0, a.T) - tok0;
}
// Packed, more sequences than lanes: the sequence whose tile a slot holds, the last one whose first slot is not behind
// it, found by 64 probes at a time.
__device__ __forceinline__ void prompt_slot(const PromptArgs& a, int slot, int tile, PromptAt& p) {
    int lo = 0, hi = a.N;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, s = lo + lane_id() * step;
        const bool in = s < hi && clamp_int(a.cu[s < hi ? s : lo], 0, a.T) / tile + s <= slot;
        const unsigned long long out = ~__ballot(in);
        const int n = out ? __builtin_ctzll(out) : 64;  // probes before the first that is behind the slot
        lo += max(n - 1, 0) * step;
        hi = min(hi, lo + step);
    }
    int tok0;
    prompt_seq(a, lo, tok0, p.len);
    p.tok0 = tok0;
    p.tile = slot - (tok0 / tile + lo);
    p.any = p.tile >= 0 && (long long)p.tile * tile < p.len;
}
// sum over the wave, by moves between lanes in the vector unit
__device__ __forceinline__ int wave_sum(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);  // lane 15 of a row: the row's sum
    return __builtin_amdgcn_readlane(x, 15) + __builtin_amdgcn_readlane(x, 31) + __builtin_amdgcn_readlane(x, 47) +
           __builtin_amdgcn_readlane(x, 63);
}
// Packed, a sequence to a lane: the r-th tile of all in the order of their distance from the sequence's other end,
// longest first, so that no long tile begins late. `last_first`: that distance is the tile's number (it sees all tiles
// before it), else the tiles behind it (which see it).
__device__ __forceinline__ void prompt_rank(const PromptArgs& a, int r, int tile, bool last_first, PromptAt& p) {
    const int l = lane_id();
    int tok0 = 0, len = 0;
    if (l < a.N) prompt_seq(a, l, tok0, len);
    const int nt = (len + tile - 1) / tile;
    // tiles with more than L tiles on their side
    auto above = [&](int L) {
        return wave_sum(max(nt - 1 - L, 0));
    };
    p.any = r < above(-1);
    if (!p.any) return;
    int lo = 0, hi = (a.T + tile - 1) / tile;  // the smallest L with above(L) <= r
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (above(mid) <= r) hi = mid;
        else lo = mid + 1;
    }
    unsigned long long who = __ballot(nt > lo);
    for (int n = r - above(lo); n > 0; --n) who &= who - 1;
    const int s = __builtin_ctzll(who);
    p.tok0 = __builtin_amdgcn_readlane(tok0, s);
    p.len = __builtin_amdgcn_readlane(len, s);
    p.tile = last_first ? lo : __builtin_amdgcn_readlane(nt, s) - 1 - lo;
}
// Tiles in the order of the launch: the last tile of every sequence first (`last_first`), which sees the most keys, or
// the first one first, which is seen most. `heads` workgroups a tile; heads that share keys lie a multiple of the
// key heads apart, mostly on one XCD. Returns the head's place 0 .. heads - 1, key heads innermost.
__device__ __forceinline__ int prompt_at(const PromptArgs& a, int bid, int tile, int heads, bool last_first, PromptAt& p,
                                         int& slot) {
    if (a.cu) {
        slot = bid / heads;
        if (a.N <= 64) prompt_rank(a, slot, tile, last_first, p);
        else prompt_slot(a, slot, tile, p);
        return bid % heads;
    }
    const int nt = (a.T + tile - 1) / tile, cols = a.N * heads, t = bid / cols, c = bid % cols;
    // c: group of heads outermost, then sequences, then key heads
    const int per = a.N * a.Hkv, g = c / per, s = c % per / a.Hkv, hk = c % a.Hkv;
    p.tile = last_first ? nt - 1 - t : t;
    p.tok0 = (long long)s * a.T;
    p.len = a.T;
    p.any = true;
    slot = 0;
    return g * a.Hkv + hk;
}
// Packed, zero_rest: rows of no sequence among rows tile * slot .. of a [tokens][heads][D] output, one head, set to zero.
template <class OT>
__device__ __forceinline__ void prompt_zero(const PromptArgs& a, int slot, int tile, OT* p, int heads, int head, int D) {
    const int b = clamp_int(a.cu[0], 0, a.T), e = clamp_int(a.cu[a.N], b, a.T);
    const int r0 = min((long long)tile * slot, (long long)a.T), r1 = min(r0 + tile, a.T);
    if (r0 >= b && r1 <= e) return;
    for (int i = threadIdx.x; i < (r1 - r0) * D; i += blockDim.x) {
        const int r = r0 + i / D;
        if (r < b || r >= e) p[((long long)r * heads + head) * D + i % D] = to_ot<OT>(0.f);
    }
}

}  // namespace gdr2
