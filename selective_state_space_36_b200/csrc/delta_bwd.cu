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

// ------------------------------------------------------- all chunks at once
constexpr int kGradThreads = 256;

template <int NP>
struct GradSmem {  // headdim rounded up to 16 (pp) decides the sizes of the rest
    bf16 k[kC][NP + 8], q[kC][NP + 8];
    bf16 x[2][kC][kMatLd], e[2][kC][kMatLd];  // X and E, high and low terms
    double cum[kC];
    float dec[kDec][kC];
    float dg[2][kC], kr[2][kC];               // row sums of the two halves of dstate: dG, k . (r dS1)
    float db[4][kC];                          // column sums of the four row blocks: dbeta's first terms
    float part[kGradThreads / 32];
};
template <int NP>
constexpr size_t grad_smem_bytes(int pp) {
    return sizeof(GradSmem<NP>) + (size_t)(5 * kC * (pp + 8) + 2 * pp * (NP + 8)) * sizeof(bf16);
}

template <int NP, bool VECQK, bool VECV>
__global__ void __launch_bounds__(kGradThreads) delta_grad_kernel(DeltaBwdArgs p, DeltaChunkWs ws) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<NP> &sm = *reinterpret_cast<GradSmem<NP> *>(raw);
    constexpr int NT = NP / 16;  // column tiles of 8 per warp: half of dstate
    const DeltaArgs &a = p.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tb = warp & 3, half = warp >> 2;
    const int pp = (a.headdim + 15) / 16 * 16, ldp = pp + 8, lds = NP + 8;
    bf16 *so = reinterpret_cast<bf16 *>(raw + sizeof(GradSmem<NP>));  // dO
    bf16 *sr = so + kC * ldp, *se = sr + 2 * kC * ldp;               // r, dV: high and low terms
    bf16 *ss = se + 2 * kC * ldp;                                    // S0, then dS1: high and low terms
    const int64_t nch = (a.seqlen + kC - 1) / kC;
    const int64_t bg = blockIdx.x / nch, ch = blockIdx.x - bg * nch;
    const int64_t b = bg / a.groups;
    const int gr = (int)(bg - b * a.groups), rep = a.heads / a.groups;
    const int64_t t0 = ch * kC;
    const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
    const int64_t qk0 = ((b * a.seqlen + t0) * a.groups + gr) * a.dstate, qk_ld = (int64_t)a.groups * a.dstate;
    const int64_t v_ld = (int64_t)a.heads * a.headdim;
    load_tile<VECQK>(&sm.k[0][0], NP + 8, static_cast<const bf16 *>(a.k) + qk0, qk_ld, kC, NP, live, a.dstate, tid,
                     kGradThreads);
    load_tile<VECQK>(&sm.q[0][0], NP + 8, static_cast<const bf16 *>(a.q) + qk0, qk_ld, kC, NP, live, a.dstate, tid,
                     kGradThreads);
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int cf_row = cols_first_row(lane), cf_col = cols_first_col(lane);
    const int n0 = half * (NP / 2);
    const int ta = 16 * tb + (lane >> 2);  // this thread's rows: ta, ta + 8

    float tq[NT][4], tk[NT][4];  // sums over the group's heads
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) tq[j][i] = tk[j][i] = 0.f;

    for (int hh = 0; hh < rep; ++hh) {
        const int h = gr * rep + hh;
        const int64_t unit = (b * a.heads + h) * nch + ch;
        __syncthreads();  // the last head's tiles are read
        load_tile<VECV>(so, ldp, static_cast<const bf16 *>(p.dout) + ((b * a.seqlen + t0) * a.heads + h) * a.headdim,
                        v_ld, kC, pp, live, a.headdim, tid, kGradThreads);
        load_tile<true>(sr, ldp, ws.r + unit * 2 * kC * pp, pp, 2 * kC, pp, 2 * kC, pp, tid, kGradThreads);
        load_tile<true>(se, ldp, ws.dv + unit * 2 * kC * pp, pp, 2 * kC, pp, 2 * kC, pp, tid, kGradThreads);
        cp_async_commit();
        {
            const bf16 *src = ws.s0 + unit * 2 * pp * NP;
            for (int i = tid; i < 2 * pp * (NP / 8); i += kGradThreads) {  // 16 bytes each, in their order in memory
                const int g = i / pp, row = i - g * pp, term = g / (NP / 8);
                cp_async16(ss + (term * pp + row) * lds + (g - term * (NP / 8)) * 8, src + (int64_t)i * 8, true);
            }
        }
        cp_async_commit();
        if (tid < kDec * kC) sm.dec[tid / kC][tid % kC] = ws.dec[unit * (kDec * kC) + tid];
        if (warp == 7) {
            const float *g = a.g + (b * a.seqlen + t0) * a.heads + h;
            const int t = 2 * lane;
            const double g0 = t < live ? fmax((double)g[(int64_t)t * a.heads], -1e4) : 0.0;
            const double g1 = t + 1 < live ? fmax((double)g[(int64_t)(t + 1) * a.heads], -1e4) : 0.0;
            double sum = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            sm.cum[t] = sum - g1;
            sm.cum[t + 1] = sum;
        }
        cp_async_wait<1>();
        __syncthreads();
        // x = scale Gam (dO_t . r_s), y = -Gam (dV_t . r_s): this warp's 16 rows and
        // its half of the columns, blocks up to the diagonal; q_t . k_s and k_t . k_s
        // beside them for dbeta
        {
            float cx[4][4], ce[4][4], cqk[4][4], ckk[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) cx[j][i] = ce[j][i] = cqk[j][i] = ckk[j][i] = 0.f;
            if (2 * half <= tb)
                for (int kk = 0; kk < pp / 16; ++kk) {
                    uint32_t ao[4], ah[4], al[4];
                    const int at = (16 * tb + rf_row) * ldp + 16 * kk + rf_col;
                    ldm4(ao, so + at);
                    ldm4(ah, se + at);
                    ldm4(al, se + kC * ldp + at);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        if (2 * half + jj > tb) continue;
                        uint32_t fh[4], fl[4];
                        const int bt = (16 * (2 * half + jj) + cf_row) * ldp + 16 * kk + cf_col;
                        ldm4(fh, sr + bt);
                        ldm4(fl, sr + kC * ldp + bt);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mma(cx[2 * jj + i], ao, fh[2 * i], fh[2 * i + 1]);
                            mma(ce[2 * jj + i], ah, fh[2 * i], fh[2 * i + 1]);
                            mma(cx[2 * jj + i], ao, fl[2 * i], fl[2 * i + 1]);
                            mma(ce[2 * jj + i], ah, fl[2 * i], fl[2 * i + 1]);
                            mma(ce[2 * jj + i], al, fh[2 * i], fh[2 * i + 1]);
                        }
                    }
                }
            if (2 * half <= tb)
#pragma unroll 2
                for (int kk = 0; kk < NP / 16; ++kk) {
                    uint32_t aq[4], ak[4];
                    ldm4(aq, &sm.q[16 * tb + rf_row][16 * kk + rf_col]);
                    ldm4(ak, &sm.k[16 * tb + rf_row][16 * kk + rf_col]);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        if (2 * half + jj > tb) continue;
                        uint32_t f[4];
                        ldm4(f, &sm.k[16 * (2 * half + jj) + cf_row][16 * kk + cf_col]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mma(cqk[2 * jj + i], aq, f[2 * i], f[2 * i + 1]);
                            mma(ckk[2 * jj + i], ak, f[2 * i], f[2 * i + 1]);
                        }
                    }
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = 32 * half + 8 * j + 2 * (lane & 3);
                float cols[2] = {0.f, 0.f};
                if (2 * half + (j >> 1) <= tb) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = ta + 8 * i;
                        float xv[2], ev[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float gam = s + c <= t ? expf((float)(sm.cum[t] - sm.cum[s + c])) : 0.f;
                            const float x = s + c <= t ? a.scale * gam * cx[j][2 * i + c] : 0.f;
                            const float y = s + c < t ? -gam * ce[j][2 * i + c] : 0.f;
                            if (s + c <= t) cols[c] += x * cqk[j][2 * i + c] + y * ckk[j][2 * i + c];
                            xv[c] = x * sm.dec[2][s + c];
                            ev[c] = y * sm.dec[2][s + c];
                        }
                        uint32_t hi, lo;
                        split(xv[0], xv[1], hi, lo);
                        *reinterpret_cast<uint32_t *>(&sm.x[0][t][s]) = hi;
                        *reinterpret_cast<uint32_t *>(&sm.x[1][t][s]) = lo;
                        split(ev[0], ev[1], hi, lo);
                        *reinterpret_cast<uint32_t *>(&sm.e[0][t][s]) = hi;
                        *reinterpret_cast<uint32_t *>(&sm.e[1][t][s]) = lo;
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) cols[c] += __shfl_xor_sync(0xffffffffu, cols[c], o);
                    if (lane < 4) sm.db[tb][s + c] = cols[c];
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        // q = scale gam dO S0 + X K,  l = E K - gam dV S0
        float cq[NT][4], cl[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) cq[j][i] = cl[j][i] = 0.f;
        for (int kk = 0; kk < pp / 16; ++kk) {
            uint32_t ao[4], ah[4], al[4];
            const int at = (16 * tb + rf_row) * ldp + 16 * kk + rf_col;
            ldm4(ao, so + at);
            ldm4(ah, se + at);
            ldm4(al, se + kC * ldp + at);
#pragma unroll
            for (int nn = 0; nn < NT / 2; ++nn) {
                uint32_t fh[4], fl[4];
                const int bt = (16 * kk + rf_row) * lds + n0 + 16 * nn + rf_col;
                ldm4t(fh, ss + bt);
                ldm4t(fl, ss + pp * lds + bt);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma(cq[2 * nn + i], ao, fh[2 * i], fh[2 * i + 1]);
                    mma(cl[2 * nn + i], ah, fh[2 * i], fh[2 * i + 1]);
                    mma(cq[2 * nn + i], ao, fl[2 * i], fl[2 * i + 1]);
                    mma(cl[2 * nn + i], ah, fl[2 * i], fl[2 * i + 1]);
                    mma(cl[2 * nn + i], al, fh[2 * i], fh[2 * i + 1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float g = sm.dec[0][ta + 8 * i], fq = a.scale * g, fl = -g;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                cq[j][2 * i] *= fq; cq[j][2 * i + 1] *= fq;
                cl[j][2 * i] *= fl; cl[j][2 * i + 1] *= fl;
            }
        }
        for (int kk = 0; kk <= tb; ++kk) {
            uint32_t xh[4], xl[4], eh[4], el[4];
            ldm4(xh, &sm.x[0][16 * tb + rf_row][16 * kk + rf_col]);
            ldm4(xl, &sm.x[1][16 * tb + rf_row][16 * kk + rf_col]);
            ldm4(eh, &sm.e[0][16 * tb + rf_row][16 * kk + rf_col]);
            ldm4(el, &sm.e[1][16 * tb + rf_row][16 * kk + rf_col]);
#pragma unroll
            for (int nn = 0; nn < NT / 2; ++nn) {
                uint32_t f[4];
                ldm4t(f, &sm.k[16 * kk + rf_row][n0 + 16 * nn + rf_col]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma(cq[2 * nn + i], xh, f[2 * i], f[2 * i + 1]);
                    mma(cl[2 * nn + i], eh, f[2 * i], f[2 * i + 1]);
                    mma(cq[2 * nn + i], xl, f[2 * i], f[2 * i + 1]);
                    mma(cl[2 * nn + i], el, f[2 * i], f[2 * i + 1]);
                }
            }
        }
        // q . dq + k . l of this warp's rows; the sums over heads
        float dot[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = n0 + 8 * j + 2 * (lane & 3);
                const uint32_t qv = *reinterpret_cast<const uint32_t *>(&sm.q[ta + 8 * i][n]);
                const uint32_t kv = *reinterpret_cast<const uint32_t *>(&sm.k[ta + 8 * i][n]);
                dot[i] += low_of(qv) * cq[j][2 * i] + high_of(qv) * cq[j][2 * i + 1] + low_of(kv) * cl[j][2 * i] +
                          high_of(kv) * cl[j][2 * i + 1];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tq[j][2 * i + c] += cq[j][2 * i + c];
                    tk[j][2 * i + c] += cl[j][2 * i + c];
                }
            }
        __syncthreads();  // S0 is read by the products
        // dS1 takes its place; <S0, dS1> on the way
        float inner = 0.f;
        {
            const bf16 *src = ws.ds1 + unit * 2 * pp * NP;
            for (int i = tid; i < pp * (NP / 8); i += kGradThreads) {
                const int g = i / pp;
                bf16 *at = ss + (i - g * pp) * lds + g * 8;
                const uint4 nh = *reinterpret_cast<const uint4 *>(src + (int64_t)i * 8);
                const uint4 nl = *reinterpret_cast<const uint4 *>(src + (int64_t)pp * NP + (int64_t)i * 8);
                const uint4 oh = *reinterpret_cast<const uint4 *>(at), ol = *reinterpret_cast<const uint4 *>(at + pp * lds);
                const uint32_t w0[4] = {nh.x, nh.y, nh.z, nh.w}, w1[4] = {nl.x, nl.y, nl.z, nl.w};
                const uint32_t w2[4] = {oh.x, oh.y, oh.z, oh.w}, w3[4] = {ol.x, ol.y, ol.z, ol.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    inner = fmaf(low_of(w0[e]) + low_of(w1[e]), low_of(w2[e]) + low_of(w3[e]), inner);
                    inner = fmaf(high_of(w0[e]) + high_of(w1[e]), high_of(w2[e]) + high_of(w3[e]), inner);
                }
                *reinterpret_cast<uint4 *>(at) = nh;
                *reinterpret_cast<uint4 *>(at + pp * lds) = nl;
            }
        }
        inner *= sm.dec[0][kC - 1];
        __syncthreads();
        // R = w beta r dS1 + X^T Q + E^T K
        float(&cr)[NT][4] = cq;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) cr[j][i] = 0.f;
        for (int kk = 0; kk < pp / 16; ++kk) {
            uint32_t ah[4], al[4];
            const int at = (16 * tb + rf_row) * ldp + 16 * kk + rf_col;
            ldm4(ah, sr + at);
            ldm4(al, sr + kC * ldp + at);
#pragma unroll
            for (int nn = 0; nn < NT / 2; ++nn) {
                uint32_t fh[4], fl[4];
                const int bt = (16 * kk + rf_row) * lds + n0 + 16 * nn + rf_col;
                ldm4t(fh, ss + bt);
                ldm4t(fl, ss + pp * lds + bt);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma(cr[2 * nn + i], ah, fh[2 * i], fh[2 * i + 1]);
                    mma(cr[2 * nn + i], ah, fl[2 * i], fl[2 * i + 1]);
                    mma(cr[2 * nn + i], al, fh[2 * i], fh[2 * i + 1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = sm.dec[1][ta + 8 * i] * sm.dec[2][ta + 8 * i];
            float kr = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = n0 + 8 * j + 2 * (lane & 3);
                const uint32_t kv = *reinterpret_cast<const uint32_t *>(&sm.k[ta + 8 * i][n]);
                kr += low_of(kv) * cr[j][2 * i] + high_of(kv) * cr[j][2 * i + 1];
                cr[j][2 * i] *= f;
                cr[j][2 * i + 1] *= f;
            }
            inner = fmaf(f, kr, inner);
            kr += __shfl_xor_sync(0xffffffffu, kr, 1);
            kr += __shfl_xor_sync(0xffffffffu, kr, 2);
            if ((lane & 3) == 0) sm.kr[half][ta + 8 * i] = kr;
        }
        for (int kk = tb; kk < kC / 16; ++kk) {
            uint32_t xh[4], xl[4], eh[4], el[4];
            ldm4t(xh, &sm.x[0][16 * kk + cf_row][16 * tb + cf_col]);
            ldm4t(xl, &sm.x[1][16 * kk + cf_row][16 * tb + cf_col]);
            ldm4t(eh, &sm.e[0][16 * kk + cf_row][16 * tb + cf_col]);
            ldm4t(el, &sm.e[1][16 * kk + cf_row][16 * tb + cf_col]);
#pragma unroll
            for (int nn = 0; nn < NT / 2; ++nn) {
                uint32_t fq[4], fk[4];
                ldm4t(fq, &sm.q[16 * kk + rf_row][n0 + 16 * nn + rf_col]);
                ldm4t(fk, &sm.k[16 * kk + rf_row][n0 + 16 * nn + rf_col]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma(cr[2 * nn + i], xh, fq[2 * i], fq[2 * i + 1]);
                    mma(cr[2 * nn + i], xl, fq[2 * i], fq[2 * i + 1]);
                    mma(cr[2 * nn + i], eh, fk[2 * i], fk[2 * i + 1]);
                    mma(cr[2 * nn + i], el, fk[2 * i], fk[2 * i + 1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = n0 + 8 * j + 2 * (lane & 3);
                const uint32_t kv = *reinterpret_cast<const uint32_t *>(&sm.k[ta + 8 * i][n]);
                dot[i] -= low_of(kv) * cr[j][2 * i] + high_of(kv) * cr[j][2 * i + 1];
                tk[j][2 * i] += cr[j][2 * i];
                tk[j][2 * i + 1] += cr[j][2 * i + 1];
            }
        // dg and dbeta of this head
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 1);
            dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 2);
            if ((lane & 3) == 0) sm.dg[half][ta + 8 * i] = dot[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
        if (lane == 0) sm.part[warp] = inner;
        __syncthreads();
        if (warp == 0) {
            float whole = 0.f;
#pragma unroll
            for (int w = 0; w < kGradThreads / 32; ++w) whole += sm.part[w];
            // lane i: tokens 63 - 2 i and 62 - 2 i; a prefix sum over lanes is a sum from the end
            const int t = kC - 1 - 2 * lane;
            const float d1 = sm.dg[0][t] + sm.dg[1][t], d0 = sm.dg[0][t - 1] + sm.dg[1][t - 1];
            float sum = d1 + d0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const int64_t at = (b * a.seqlen + t0) * a.heads + h;
            if (t < live) p.dg[at + (int64_t)t * a.heads] = whole + (sum - d0);
            if (t - 1 < live) p.dg[at + (int64_t)(t - 1) * a.heads] = whole + sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = t - i;
                const float db = (sm.db[0][s] + sm.db[1][s]) + (sm.db[2][s] + sm.db[3][s]);
                if (s < live) p.dbeta[at + (int64_t)s * a.heads] = db + sm.dec[1][s] * (sm.kr[0][s] + sm.kr[1][s]);
            }
        }
    }
    bf16 *dq = static_cast<bf16 *>(p.dq) + qk0, *dk = static_cast<bf16 *>(p.dk) + qk0;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = ta + 8 * i, n = n0 + 8 * j + 2 * (lane & 3);
            if (t >= live) continue;
            if (VECQK) {
                if (n < a.dstate) {
                    *reinterpret_cast<uint32_t *>(dq + t * qk_ld + n) = pack(tq[j][2 * i], tq[j][2 * i + 1]);
                    *reinterpret_cast<uint32_t *>(dk + t * qk_ld + n) = pack(tk[j][2 * i], tk[j][2 * i + 1]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (n + c < a.dstate) {
                        dq[t * qk_ld + n + c] = __float2bfloat16_rn(tq[j][2 * i + c]);
                        dk[t * qk_ld + n + c] = __float2bfloat16_rn(tk[j][2 * i + c]);
                    }
            }
        }
}

template <int NP, bool VECQK, bool VECV>
cudaError_t launch_grad_t(const DeltaBwdArgs &p, const DeltaChunkWs &ws, cudaStream_t st) {
    const DeltaArgs &a = p.f;
    const size_t bytes = grad_smem_bytes<NP>((a.headdim + 15) / 16 * 16);
    cudaError_t e = allow_smem<delta_grad_kernel<NP, VECQK, VECV>, (int)grad_smem_bytes<NP>(kDeltaMaxDstate)>();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.batch * a.groups * ((a.seqlen + kC - 1) / kC)));
    delta_grad_kernel<NP, VECQK, VECV><<<grid, kGradThreads, bytes, st>>>(p, ws);
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

cudaError_t launch_delta_grad(const DeltaBwdArgs &p, const DeltaChunkWs &ws, cudaStream_t st) {
    using namespace delta;
    const bool qk = p.f.dstate % 8 == 0 && aligned16(p.f.q) && aligned16(p.f.k) && aligned16(p.dq) && aligned16(p.dk);
    const bool v = p.f.headdim % 8 == 0 && aligned16(p.dout);
    if (p.f.dstate <= 64) {
        if (qk) return v ? launch_grad_t<64, true, true>(p, ws, st) : launch_grad_t<64, true, false>(p, ws, st);
        return v ? launch_grad_t<64, false, true>(p, ws, st) : launch_grad_t<64, false, false>(p, ws, st);
    }
    if (qk) return v ? launch_grad_t<128, true, true>(p, ws, st) : launch_grad_t<128, true, false>(p, ws, st);
    return v ? launch_grad_t<128, false, true>(p, ws, st) : launch_grad_t<128, false, false>(p, ws, st);
}

}  // namespace ssm
