// Recurrent (token-by-token) form of the gated delta rule with scalar gates, for decoding on states
// that live in a pool and are picked by index. With S the state before a token, u = S^T k and
// p = S^T q,
//     delta = beta (v - e^g u),   S' = e^g S + k delta^T,   o = S'^T q = e^g p + (k.q) delta,
// so one pass over the old state gives both sums over the key axis, and the update needs no second
// reduction. Bound by HBM: the state is read and written once a call.
//
// k_sc_step: one workgroup of two waves per (row, value head, 64 columns), a wave on 32 columns. Lane l
// holds columns 4 (l % 8) .. + 3 of rows l / 8 + 8 i, so each row segment a wave moves is one 128-byte
// line, and the sums over the key axis stay inside a wave. The state stays in registers for all tokens
// of the call. Measured at d = 128, 16 value heads: 512 rows (1.08 GB) in 222 us, 4.8 TB/s, where each call has
// another pool (214 us with the states in order), and in 184 us, 5.8 TB/s, on one pool again and again, part of
// which the Infinity Cache still holds from the call before (written there with ordinary stores: 225 and 226 us);
// one row (2.1 MB) in 5.0 us, a launch and the latency of one read, and no less with the key axis split
// over four waves that join their sums in LDS (5.1 us).
#include "gdr2_device.hpp"
#include "gdr2_scalar.hpp"

namespace gdr2 {

__device__ __forceinline__ f32x4 sum_row_groups(f32x4 x) {  // over lanes l ^ 8, 16, 32
#pragma unroll
    for (int m = 8; m < 64; m <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], m, 64);
    return x;
}

template <class OT, int DK, int DV, bool NT>
__global__ __launch_bounds__(128) void k_sc_step(ScStepArgs a) {
    constexpr int NTHR = 128, NI = DK / 8, NJ = DV / 64;
    __shared__ float sk[DK], sq[DK], sv[64];
    poison_lds((lds_char*)sk, sizeof(sk));
    poison_lds((lds_char*)sq, sizeof(sq));
    poison_lds((lds_char*)sv, sizeof(sv));
    poison_lds_done();
    const int tid = threadIdx.x, wv = tid >> 6, l = tid & 63, cq = l & 7, rg = l >> 3;
    const int jb = blockIdx.x % NJ, hb = blockIdx.x / NJ;
    const int h = hb % a.Hv, b0 = hb / a.Hv, hk = h / a.R;
    const int slot = a.slots ? a.slots[b0] : b0;
    const int col0 = 64 * jb, col = col0 + 32 * wv + 4 * cq;
    if (slot < 0 || slot >= a.states) {  // a padding row: no state, zero output
        for (int t = 0; t < a.T; ++t)
            if (tid < 64) ((OT*)a.o)[(((size_t)b0 * a.T + t) * a.Hv + h) * DV + col0 + tid] = to_ot<OT>(0.f);
        return;
    }
    float* hs = a.state + ((size_t)slot * a.Hv + h) * DK * DV + col;
    f32x4 S[NI];  // S[i]: row rg + 8 i
#pragma unroll
    for (int i = 0; i < NI; ++i) S[i] = *(const f32x4*)(hs + (size_t)(rg + 8 * i) * DV);
    // Rows that name the same state are one sequence, in the order of the rows: the first of them
    // does the work of all. Every workgroup looks through all slots: 1 us of 214 for 512 rows of 16 heads of
    // 128, 43 of 150 for 4096 rows of 4 heads of 64, 208 of 314 for 16384 rows of one.
    int more = 0;
    if (a.slots) {
        int seen = 0;  // 1: an earlier row has this state; 2: a later one
        for (int i = tid; i < a.B; i += NTHR)
            if (i != b0 && a.slots[i] == slot) seen |= i < b0 ? 1 : 2;
        if (__syncthreads_or(seen & 1)) return;
        more = __syncthreads_or(seen & 2);
    }
#pragma unroll 1
    for (int b = b0; b < a.B; ++b) {
        if (b != b0 && a.slots[b] != slot) continue;
#pragma unroll 1
        for (int t = 0; t < a.T; ++t) {
            const size_t tok = (size_t)b * a.T + t;
            const size_t kr = (tok * a.Hk + hk) * DK, vr = (tok * a.Hv + h) * DV;
            for (int i = tid; i < DK; i += NTHR) {
                sk[i] = to_f(((const OT*)a.k)[kr + i]);
                sq[i] = to_f(((const OT*)a.q)[kr + i]);
            }
            if (tid < 64) sv[tid] = to_f(((const OT*)a.v)[vr + col0 + tid]);
            const float e = expf(to_f(((const OT*)a.g)[tok * a.Hv + h]));
            const float beta = to_f(((const OT*)a.beta)[tok * a.Hv + h]);
            __syncthreads();
            f32x4 u = {0.f, 0.f, 0.f, 0.f}, p = u;
            float kq = 0.f;  // k.q, the same in all lanes of a row group
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = rg + 8 * i;
                const float k = sk[r], q = sq[r];
                u += k * S[i];
                p += q * S[i];
                kq += k * q;
            }
            u = sum_row_groups(u);
            p = sum_row_groups(p);
#pragma unroll
            for (int m = 8; m < 64; m <<= 1) kq += __shfl_xor(kq, m, 64);
            f32x4 d;
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = beta * (sv[32 * wv + 4 * cq + j] - e * u[j]);
#pragma unroll
            for (int i = 0; i < NI; ++i) S[i] = e * S[i] + sk[rg + 8 * i] * d;
            if (rg == 0) {
                const f32x4 o = e * p + kq * d;
                const float ov[4] = {o[0], o[1], o[2], o[3]};
                st4((OT*)a.o + vr + col, ov);
            }
            __syncthreads();  // the token's vectors are free
        }
        if (!more) break;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
        store_out<NT>((f32x4*)(hs + (size_t)(rg + 8 * i) * DV), S[i]);
}

template <class OT, int DK, int DV>
static hipError_t launch_sc_step_t(const ScStepArgs& a, hipStream_t stream) {
    const unsigned groups = (unsigned)a.B * a.Hv * (DV / 64);
    if (a.nt_out)
        hipLaunchKernelGGL((k_sc_step<OT, DK, DV, true>), dim3(groups), dim3(128), 0, stream, a);
    else
        hipLaunchKernelGGL((k_sc_step<OT, DK, DV, false>), dim3(groups), dim3(128), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_sc_step(const ScStepArgs& a, bool bf16_, hipStream_t stream) {
    if (bf16_) {
        if (a.DK == 64 && a.DV == 64) return launch_sc_step_t<bf16, 64, 64>(a, stream);
        if (a.DK == 64 && a.DV == 128) return launch_sc_step_t<bf16, 64, 128>(a, stream);
        if (a.DK == 128 && a.DV == 64) return launch_sc_step_t<bf16, 128, 64>(a, stream);
        if (a.DK == 128 && a.DV == 128) return launch_sc_step_t<bf16, 128, 128>(a, stream);
    } else if (a.DK == 64 && a.DV == 64) {
        return launch_sc_step_t<float, 64, 64>(a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace gdr2
