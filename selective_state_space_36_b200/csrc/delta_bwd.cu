// delta_bwd.cu -- the chunked gated delta rule's gradient on the tensor cores.
//
// With dS1 the gradient of the state leaving a chunk (notation of
// delta_chunk.cuh, gam = exp G, w = exp(G_C - G)):
//   z   = Pb^T dO + w beta K dS1^T,   dV = z - M^T z
//   dS0 = gam_C dS1 + (scale gam dO)^T Q - (gam dV)^T K
// runs backwards over the chunks (delta_reverse_kernel, the mirror image of
// delta_chain.cu: one warp per 16 state rows, everything transposed).  It needs
// no state; it leaves dS1 and dV of each chunk in the workspace.  Then, for all
// chunks at once (delta_grad_kernel), with S0 and r from the forward's
// recomputation and x = scale lower(Gam o (dO r^T)), y = -strict_lower(Gam o (dV r^T)),
// X = x beta, E = y beta (columns scaled):
//   dQ = scale gam dO S0 + X K
//   dK = L + R,  L = E K - gam dV S0,  R = X^T Q + E^T K + w beta r dS1
//   dbeta_s = sum_t x_ts q_t . k_s + sum_t y_ts k_t . k_s + w_s (r dS1)_s . k_s
// (beta enters R alone, as a factor of its row s: dbeta_s = k_s . R_s / beta_s,
// without the division),
//   dG_t = q_t . dq_t + k_t . (L_t - R_t),  dG_C += <S1, dS1>
//   dg_t = sum of dG over the chunk's tokens from t on
// dG needs no difference of large sums: its terms are row products that exist
// anyway, and <S1, dS1> = gam_C <S0, dS1> + sum_t w beta (r dS1)_t . k_t.
#include "delta_chunk.cuh"
#include "kernel_setup.cuh"

namespace ssm {
namespace delta {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ------------------------------------------------------- backwards in time
template <int NP>
constexpr int stage_bytes(int w) {
    return (2 * kC * (NP + 8) + kC * (16 * w + 8) + kMats * kC * kMatLd) * 2 + kDec * kC * 4;
}

template <int NP, bool VECQK, bool VECV>
__global__ void __launch_bounds__(256) delta_reverse_kernel(DeltaBwdArgs p, DeltaChunkWs ws, int vtiles) {
    extern __shared__ __align__(16) unsigned char raw[];
    const DeltaArgs &a = p.f;
    const int nthreads = blockDim.x, nwarps = nthreads >> 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ldk = NP + 8, ldv = 16 * nwarps + 8;
    const int64_t bh = blockIdx.x / vtiles;
    const int v0 = (int)(blockIdx.x - bh * vtiles) * 16 * nwarps;
    const int64_t b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int64_t nch = (a.seqlen + kC - 1) / kC;
    const int bytes = stage_bytes<NP>(nwarps);
    const int pp = (a.headdim + 15) / 16 * 16;

    const int64_t qk_ld = (int64_t)a.groups * a.dstate, v_ld = (int64_t)a.heads * a.headdim;
    const bf16 *gq = static_cast<const bf16 *>(a.q) + (b * a.seqlen * a.groups + gr) * a.dstate;
    const bf16 *gk = static_cast<const bf16 *>(a.k) + (b * a.seqlen * a.groups + gr) * a.dstate;
    const bf16 *go = static_cast<const bf16 *>(p.dout) + (b * a.seqlen * a.heads + h) * a.headdim + v0;
    bf16 *gv = static_cast<bf16 *>(p.dv) + (b * a.seqlen * a.heads + h) * a.headdim + v0;

    // step i is chunk nch - 1 - i
    auto issue = [&](int64_t i) {
        if (i < nch) {
            const int64_t ch = nch - 1 - i;
            unsigned char *st = raw + (i & 1) * bytes;
            bf16 *sk = reinterpret_cast<bf16 *>(st), *sq = sk + kC * ldk, *so = sq + kC * ldk, *sm = so + kC * ldv;
            float *sd = reinterpret_cast<float *>(sm + kMats * kC * kMatLd);
            const int64_t t0 = ch * kC, unit = bh * nch + ch;
            const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
            load_tile<VECQK>(sk, ldk, gk + t0 * qk_ld, qk_ld, kC, NP, live, a.dstate, tid, nthreads);
            load_tile<VECQK>(sq, ldk, gq + t0 * qk_ld, qk_ld, kC, NP, live, a.dstate, tid, nthreads);
            load_tile<VECV>(so, ldv, go + t0 * v_ld, v_ld, kC, 16 * nwarps, live, a.headdim - v0, tid, nthreads);
            load_tile<true>(sm, kMatLd, ws.mats + unit * (kMats * kC * kC), kC, kMats * kC, kC, kMats * kC, kC, tid,
                            nthreads);
            const float *gd = ws.dec + unit * (kDec * kC);
            for (int j = tid; j < kDec * kC / 4; j += nthreads) cp_async16(sd + 4 * j, gd + 4 * j, true);
        }
        cp_async_commit();
    };

    float s[NP / 8][4];  // dS
    const int row = v0 + 16 * warp + (lane >> 2);
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row + (e >> 1) * 8, c = 8 * j + 2 * (lane & 3) + (e & 1);
            s[j][e] = p.dend && r < a.headdim && c < a.dstate ? p.dend[(bh * a.headdim + r) * (int64_t)a.dstate + c] : 0.f;
        }
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int cf_row = cols_first_row(lane), cf_col = cols_first_col(lane);

    issue(0);
    for (int64_t i = 0; i < nch; ++i) {
        issue(i + 1);
        cp_async_wait<1>();
        __syncthreads();
        const int64_t ch = nch - 1 - i, unit = bh * nch + ch, t0 = ch * kC;
        const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
        unsigned char *st = raw + (i & 1) * bytes;
        bf16 *sk = reinterpret_cast<bf16 *>(st), *sq = sk + kC * ldk, *so = sq + kC * ldk, *sm = so + kC * ldv;
        const float *gam = reinterpret_cast<const float *>(sm + kMats * kC * kMatLd), *wend = gam + kC,
                    *beta = wend + kC;
        const bf16 *sn = sm, *sp = sm + kC * kMatLd;
        constexpr int kLow = 2 * kC * kMatLd;
        bf16 *mine = so + 16 * warp;  // this warp's columns of dO, later of its results

        store_state<NP>(ws.ds1 + unit * 2 * pp * NP, pp, s, v0 + 16 * warp, lane);
        // x = z^T = w beta (dS K^T) + dO^T Pb
        float x[kC / 8][4];
#pragma unroll
        for (int j = 0; j < kC / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NP / 16; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                split(s[2 * kk + (q >> 1)][2 * (q & 1)], s[2 * kk + (q >> 1)][2 * (q & 1) + 1], hi[q], lo[q]);
#pragma unroll
            for (int jj = 0; jj < kC / 16; ++jj) {
                uint32_t f[4];
                ldm4(f, sk + (16 * jj + cf_row) * ldk + 16 * kk + cf_col);
                mma(x[2 * jj], hi, f[0], f[1]);
                mma(x[2 * jj + 1], hi, f[2], f[3]);
                mma(x[2 * jj], lo, f[0], f[1]);
                mma(x[2 * jj + 1], lo, f[2], f[3]);
            }
        }
#pragma unroll
        for (int j = 0; j < kC / 8; ++j) {
            const float2 w2 = *reinterpret_cast<const float2 *>(wend + 8 * j + 2 * (lane & 3));
            const float2 b2 = *reinterpret_cast<const float2 *>(beta + 8 * j + 2 * (lane & 3));
            const float f0 = w2.x * b2.x, f1 = w2.y * b2.y;
            x[j][0] *= f0; x[j][1] *= f1; x[j][2] *= f0; x[j][3] *= f1;
        }
        uint32_t dof[kC / 16][4];
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk) {
            ldm4t(dof[kk], mine + (16 * kk + cf_row) * ldv + cf_col);
#pragma unroll
            for (int jj = 0; jj <= kk; ++jj) {
                uint32_t f[4], fl[4];
                ldm4t(f, sp + (16 * kk + rf_row) * kMatLd + 16 * jj + rf_col);
                ldm4t(fl, sp + kLow + (16 * kk + rf_row) * kMatLd + 16 * jj + rf_col);
                mma(x[2 * jj], dof[kk], f[0], f[1]);
                mma(x[2 * jj + 1], dof[kk], f[2], f[3]);
                mma(x[2 * jj], dof[kk], fl[0], fl[1]);
                mma(x[2 * jj + 1], dof[kk], fl[2], fl[3]);
            }
        }
        // dV^T = x - x M, in place: blocks of 16 tokens from the first (M is strictly
        // lower: a block changes itself and those before it)
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 2 * kk + (q >> 1);
                split(-x[j][2 * (q & 1)], -x[j][2 * (q & 1) + 1], hi[q], lo[q]);
            }
#pragma unroll
            for (int jj = 0; jj <= kk; ++jj) {
                uint32_t f[4], fl[4];
                ldm4t(f, sn + (16 * kk + rf_row) * kMatLd + 16 * jj + rf_col);
                ldm4t(fl, sn + kLow + (16 * kk + rf_row) * kMatLd + 16 * jj + rf_col);
                mma(x[2 * jj], hi, f[0], f[1]);
                mma(x[2 * jj + 1], hi, f[2], f[3]);
                mma(x[2 * jj], lo, f[0], f[1]);
                mma(x[2 * jj + 1], lo, f[2], f[3]);
                mma(x[2 * jj], hi, fl[0], fl[1]);
                mma(x[2 * jj + 1], hi, fl[2], fl[3]);
            }
        }
        // dV to the workspace and to memory
        __syncwarp();
        store_rows(ws.dv + unit * 2 * kC * pp, pp, x, mine, ldv, v0 + 16 * warp, lane);
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj) {
            uint32_t f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 2 * jj + (q >> 1);
                f[q] = pack(x[j][2 * (q & 1)], x[j][2 * (q & 1) + 1]);
            }
            stm4t(mine + (16 * jj + cf_row) * ldv + cf_col, f[0], f[1], f[2], f[3]);
        }
        __syncwarp();
        const int have = a.headdim - v0 - 16 * warp;
        bf16 *dst = gv + t0 * v_ld + 16 * warp;
        if (VECV) {
#pragma unroll
            for (int it = 0; it < kC / 16; ++it) {
                const int t = 16 * it + (lane >> 1), c = 8 * (lane & 1);
                if (t < live && c < have)
                    *reinterpret_cast<uint4 *>(dst + t * v_ld + c) = *reinterpret_cast<const uint4 *>(mine + t * ldv + c);
            }
        } else {
            for (int k = lane; k < kC * 16; k += 32) {
                const int t = k >> 4, c = k & 15;
                if (t < live && c < have) dst[t * v_ld + c] = mine[t * ldv + c];
            }
        }
        // dS0 = gam_C dS1 + (scale gam dO)^T Q - (gam dV)^T K
        const float whole = gam[kC - 1];
#pragma unroll
        for (int j = 0; j < NP / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] *= whole;
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk) {
            uint32_t ohi[4], olo[4], hi[4], lo[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 2 * kk + (q >> 1);
                const float2 g2 = *reinterpret_cast<const float2 *>(gam + 8 * j + 2 * (lane & 3));
                split(a.scale * g2.x * low_of(dof[kk][q]), a.scale * g2.y * high_of(dof[kk][q]), ohi[q], olo[q]);
                split(-g2.x * x[j][2 * (q & 1)], -g2.y * x[j][2 * (q & 1) + 1], hi[q], lo[q]);
            }
#pragma unroll
            for (int nn = 0; nn < NP / 16; ++nn) {
                uint32_t f[4];
                ldm4t(f, sq + (16 * kk + rf_row) * ldk + 16 * nn + rf_col);
                mma(s[2 * nn], ohi, f[0], f[1]);
                mma(s[2 * nn + 1], ohi, f[2], f[3]);
                mma(s[2 * nn], olo, f[0], f[1]);
                mma(s[2 * nn + 1], olo, f[2], f[3]);
                ldm4t(f, sk + (16 * kk + rf_row) * ldk + 16 * nn + rf_col);
                mma(s[2 * nn], hi, f[0], f[1]);
                mma(s[2 * nn + 1], hi, f[2], f[3]);
                mma(s[2 * nn], lo, f[0], f[1]);
                mma(s[2 * nn + 1], lo, f[2], f[3]);
            }
        }
        __syncthreads();
    }
    if (!p.dh0) return;
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row + (e >> 1) * 8, c = 8 * j + 2 * (lane & 3) + (e & 1);
            if (r < a.headdim && c < a.dstate) p.dh0[(bh * a.headdim + r) * (int64_t)a.dstate + c] = s[j][e];
        }
}

template <int NP, bool VECQK, bool VECV>
cudaError_t launch_reverse_t(const DeltaBwdArgs &p, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    const DeltaArgs &a = p.f;
    int w = (a.headdim + 15) / 16;
    if (w > 8) w = 8;
    while (w > 1 && a.batch * a.heads * ((a.headdim + 16 * w - 1) / (16 * w)) < sms) w = (w + 1) / 2;
    const int vtiles = (a.headdim + 16 * w - 1) / (16 * w);
    const int bytes = 2 * stage_bytes<NP>(w);
    cudaError_t e = allow_smem<delta_reverse_kernel<NP, VECQK, VECV>, 2 * stage_bytes<NP>(8)>();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.batch * a.heads * vtiles));
    delta_reverse_kernel<NP, VECQK, VECV><<<grid, 32 * w, bytes, st>>>(p, ws, vtiles);
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

cudaError_t launch_delta_reverse(const DeltaBwdArgs &p, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    using namespace delta;
    const bool qk = p.f.dstate % 8 == 0 && aligned16(p.f.q) && aligned16(p.f.k);
    const bool v = p.f.headdim % 8 == 0 && aligned16(p.dout) && aligned16(p.dv);
    if (p.f.dstate <= 64) {
        if (qk) return v ? launch_reverse_t<64, true, true>(p, ws, sms, st) : launch_reverse_t<64, true, false>(p, ws, sms, st);
        return v ? launch_reverse_t<64, false, true>(p, ws, sms, st) : launch_reverse_t<64, false, false>(p, ws, sms, st);
    }
    if (qk) return v ? launch_reverse_t<128, true, true>(p, ws, sms, st) : launch_reverse_t<128, true, false>(p, ws, sms, st);
    return v ? launch_reverse_t<128, false, true>(p, ws, sms, st) : launch_reverse_t<128, false, false>(p, ws, sms, st);
}

}  // namespace ssm
