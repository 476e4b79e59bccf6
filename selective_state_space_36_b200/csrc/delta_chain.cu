// delta_chain.cu -- the chunked gated delta rule's pass over the chunks of a
// sequence, after delta_prep.cu.
//
// The columns of V (rows of the state) are independent given K, Q, M and Pb,
// so one warp owns 16 of them for the whole sequence and keeps its slice of
// the state, 16 x dstate, in the accumulator registers of the matrix
// instructions.  Everything is computed transposed (state rows as the
// instruction's rows), so that an accumulator is, without any exchange, the
// left operand of the next product:
//   X^T = S K^T -> r^T = (V^T - X^T gam)(I - M)^T -> S += (r beta w)^T K,
//   O^T = S Q^T gam scale + r^T Pb^T.
// No block-wide exchange exists in a chunk; the block shares only the tiles of
// K, Q, V, M and Pb, which cp.async brings one chunk ahead (two stages).
// Products of the state or of r take two bf16 terms of each (delta_chunk.cuh).
#include "delta_chunk.cuh"
#include "kernel_setup.cuh"

namespace ssm {
namespace delta {
namespace {

// Shared memory of one stage, in bytes, for W warps (16 W columns of V).
template <int NP>
constexpr int stage_bytes(int w) {
    return (2 * kC * (NP + 8) + kC * (16 * w + 8) + kMats * kC * kMatLd) * 2 + kDec * kC * 4;
}

// STORE: the backward pass's first half -- no output, but the state entering
// each chunk and r, as two bf16 terms each, go to the workspace.
template <int NP, bool VECQK, bool VECV, bool STORE>
__global__ void __launch_bounds__(256) delta_chain_kernel(DeltaArgs a, DeltaChunkWs ws, int vtiles) {
    extern __shared__ __align__(16) unsigned char raw[];
    const int nthreads = blockDim.x, nwarps = nthreads >> 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ldk = NP + 8, ldv = 16 * nwarps + 8;
    const int64_t bh = blockIdx.x / vtiles;
    const int v0 = (int)(blockIdx.x - bh * vtiles) * 16 * nwarps;
    const int64_t b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int64_t nch = (a.seqlen + kC - 1) / kC;
    const int bytes = stage_bytes<NP>(nwarps);

    const int64_t qk_ld = (int64_t)a.groups * a.dstate, v_ld = (int64_t)a.heads * a.headdim;
    const bf16 *gq = static_cast<const bf16 *>(a.q) + (b * a.seqlen * a.groups + gr) * a.dstate;
    const bf16 *gk = static_cast<const bf16 *>(a.k) + (b * a.seqlen * a.groups + gr) * a.dstate;
    const bf16 *gv = static_cast<const bf16 *>(a.v) + (b * a.seqlen * a.heads + h) * a.headdim + v0;
    bf16 *go = STORE ? nullptr : static_cast<bf16 *>(a.out) + (b * a.seqlen * a.heads + h) * a.headdim + v0;
    const int pp = (a.headdim + 15) / 16 * 16;  // rows of a stored state, columns of a stored r

    auto issue = [&](int64_t ch) {
        if (ch < nch) {
            unsigned char *st = raw + (ch & 1) * bytes;
            bf16 *sk = reinterpret_cast<bf16 *>(st), *sq = sk + kC * ldk, *sv = sq + kC * ldk, *sm = sv + kC * ldv;
            float *sd = reinterpret_cast<float *>(sm + kMats * kC * kMatLd);
            const int64_t t0 = ch * kC, unit = bh * nch + ch;
            const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
            load_tile<VECQK>(sk, ldk, gk + t0 * qk_ld, qk_ld, kC, NP, live, a.dstate, tid, nthreads);
            if (!STORE)
                load_tile<VECQK>(sq, ldk, gq + t0 * qk_ld, qk_ld, kC, NP, live, a.dstate, tid, nthreads);
            load_tile<VECV>(sv, ldv, gv + t0 * v_ld, v_ld, kC, 16 * nwarps, live, a.headdim - v0, tid, nthreads);
            load_tile<true>(sm, kMatLd, ws.mats + unit * (kMats * kC * kC), kC, kMats * kC, kC, kMats * kC, kC, tid,
                            nthreads);
            const float *gd = ws.dec + unit * (kDec * kC);
            for (int i = tid; i < kDec * kC / 4; i += nthreads) cp_async16(sd + 4 * i, gd + 4 * i, true);
        }
        cp_async_commit();
    };

    // the state slice: rows v = v0 + 16 warp + lane / 4 (+ 8), columns 8 j + 2 (lane % 4) (+ 1)
    float s[NP / 8][4];
    const int row = v0 + 16 * warp + (lane >> 2);
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row + (e >> 1) * 8, c = 8 * j + 2 * (lane & 3) + (e & 1);
            s[j][e] = a.h0 && r < a.headdim && c < a.dstate ? a.h0[(bh * a.headdim + r) * (int64_t)a.dstate + c] : 0.f;
        }
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int cf_row = cols_first_row(lane), cf_col = cols_first_col(lane);

    issue(0);
    for (int64_t ch = 0; ch < nch; ++ch) {
        issue(ch + 1);
        cp_async_wait<1>();
        __syncthreads();
        unsigned char *st = raw + (ch & 1) * bytes;
        bf16 *sk = reinterpret_cast<bf16 *>(st), *sq = sk + kC * ldk, *sv = sq + kC * ldk, *sm = sv + kC * ldv;
        const float *gam = reinterpret_cast<const float *>(sm + kMats * kC * kMatLd), *wend = gam + kC,
                    *beta = wend + kC;
        const bf16 *sn = sm, *sp = sm + kC * kMatLd;
        constexpr int kLow = 2 * kC * kMatLd;  // from a high term's tile to the low term's
        bf16 *mine = sv + 16 * warp;       // this warp's columns of V, later of the output

        if constexpr (STORE) store_state<NP>(ws.s0 + (bh * nch + ch) * 2 * pp * NP, pp, s, v0 + 16 * warp, lane);
        float x[kC / 8][4], o[kC / 8][4];
#pragma unroll
        for (int j = 0; j < kC / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = o[j][e] = 0.f;
        // X^T = S K^T, O^T = S Q^T
#pragma unroll
        for (int kk = 0; kk < NP / 16; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split(s[2 * kk + (i >> 1)][2 * (i & 1)], s[2 * kk + (i >> 1)][2 * (i & 1) + 1], hi[i], lo[i]);
#pragma unroll
            for (int jj = 0; jj < kC / 16; ++jj) {
                uint32_t f[4];
                ldm4(f, sk + (16 * jj + cf_row) * ldk + 16 * kk + cf_col);
                mma(x[2 * jj], hi, f[0], f[1]);
                mma(x[2 * jj + 1], hi, f[2], f[3]);
                mma(x[2 * jj], lo, f[0], f[1]);
                mma(x[2 * jj + 1], lo, f[2], f[3]);
                if constexpr (STORE) continue;
                ldm4(f, sq + (16 * jj + cf_row) * ldk + 16 * kk + cf_col);
                mma(o[2 * jj], hi, f[0], f[1]);
                mma(o[2 * jj + 1], hi, f[2], f[3]);
                mma(o[2 * jj], lo, f[0], f[1]);
                mma(o[2 * jj + 1], lo, f[2], f[3]);
            }
        }
        // x = V^T - gam X^T;  o = scale gam O^T
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj) {
            uint32_t f[4];
            ldm4t(f, mine + (16 * jj + cf_row) * ldv + cf_col);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 2 * jj + i;
                const float2 g2 = *reinterpret_cast<const float2 *>(gam + 8 * j + 2 * (lane & 3));
                x[j][0] = fmaf(-g2.x, x[j][0], low_of(f[2 * i]));
                x[j][1] = fmaf(-g2.y, x[j][1], high_of(f[2 * i]));
                x[j][2] = fmaf(-g2.x, x[j][2], low_of(f[2 * i + 1]));
                x[j][3] = fmaf(-g2.y, x[j][3], high_of(f[2 * i + 1]));
                o[j][0] *= a.scale * g2.x;
                o[j][1] *= a.scale * g2.y;
                o[j][2] *= a.scale * g2.x;
                o[j][3] *= a.scale * g2.y;
            }
        }
        // r^T = x - x M^T, in place: blocks of 16 tokens from the last, whose own
        // values no earlier step has changed yet (M is strictly lower)
#pragma unroll
        for (int kk = kC / 16 - 1; kk >= 0; --kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 2 * kk + (i >> 1);
                split(-x[j][2 * (i & 1)], -x[j][2 * (i & 1) + 1], hi[i], lo[i]);
            }
#pragma unroll
            for (int jj = kk; jj < kC / 16; ++jj) {
                uint32_t f[4], fl[4];
                ldm4(f, sn + (16 * jj + cf_row) * kMatLd + 16 * kk + cf_col);
                ldm4(fl, sn + kLow + (16 * jj + cf_row) * kMatLd + 16 * kk + cf_col);
                mma(x[2 * jj], hi, f[0], f[1]);
                mma(x[2 * jj + 1], hi, f[2], f[3]);
                mma(x[2 * jj], lo, f[0], f[1]);
                mma(x[2 * jj + 1], lo, f[2], f[3]);
                mma(x[2 * jj], hi, fl[0], fl[1]);
                mma(x[2 * jj + 1], hi, fl[2], fl[3]);
            }
        }
        if constexpr (STORE) {
            store_rows(ws.r + (bh * nch + ch) * 2 * kC * pp, pp, x, mine, ldv, v0 + 16 * warp, lane);
        }
        // O^T += r^T Pb^T;  S = exp(G_C) S + (r beta w)^T K
        const float whole = gam[kC - 1];
#pragma unroll
        for (int j = 0; j < NP / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] *= whole;
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk) {
            uint32_t hi[4], lo[4], whi[4], wlo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 2 * kk + (i >> 1);
                const float2 b2 = *reinterpret_cast<const float2 *>(beta + 8 * j + 2 * (lane & 3));
                const float2 w2 = *reinterpret_cast<const float2 *>(wend + 8 * j + 2 * (lane & 3));
                const float r0 = x[j][2 * (i & 1)], r1 = x[j][2 * (i & 1) + 1];
                split(r0, r1, hi[i], lo[i]);
                split(w2.x * b2.x * r0, w2.y * b2.y * r1, whi[i], wlo[i]);
            }
#pragma unroll
            for (int jj = kk; jj < kC / 16; ++jj) {
                if constexpr (STORE) continue;
                uint32_t f[4], fl[4];
                ldm4(f, sp + (16 * jj + cf_row) * kMatLd + 16 * kk + cf_col);
                ldm4(fl, sp + kLow + (16 * jj + cf_row) * kMatLd + 16 * kk + cf_col);
                mma(o[2 * jj], hi, f[0], f[1]);
                mma(o[2 * jj + 1], hi, f[2], f[3]);
                mma(o[2 * jj], lo, f[0], f[1]);
                mma(o[2 * jj + 1], lo, f[2], f[3]);
                mma(o[2 * jj], hi, fl[0], fl[1]);
                mma(o[2 * jj + 1], hi, fl[2], fl[3]);
            }
#pragma unroll
            for (int nn = 0; nn < NP / 16; ++nn) {
                uint32_t f[4];
                ldm4t(f, sk + (16 * kk + rf_row) * ldk + 16 * nn + rf_col);
                mma(s[2 * nn], whi, f[0], f[1]);
                mma(s[2 * nn + 1], whi, f[2], f[3]);
                mma(s[2 * nn], wlo, f[0], f[1]);
                mma(s[2 * nn + 1], wlo, f[2], f[3]);
            }
        }
        if constexpr (STORE) {
            __syncthreads();
            continue;
        }
        // the output over this warp's columns of V, then to memory
        __syncwarp();
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj)
            stm4t(mine + (16 * jj + cf_row) * ldv + cf_col, pack(o[2 * jj][0], o[2 * jj][1]),
                  pack(o[2 * jj][2], o[2 * jj][3]), pack(o[2 * jj + 1][0], o[2 * jj + 1][1]),
                  pack(o[2 * jj + 1][2], o[2 * jj + 1][3]));
        __syncwarp();
        const int64_t t0 = ch * kC;
        const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
        const int have = a.headdim - v0 - 16 * warp;  // columns of the output in this warp's 16
        bf16 *dst = go + t0 * v_ld + 16 * warp;
        if (VECV) {
#pragma unroll
            for (int it = 0; it < kC / 16; ++it) {
                const int t = 16 * it + (lane >> 1), c = 8 * (lane & 1);
                if (t < live && c < have)
                    *reinterpret_cast<uint4 *>(dst + t * v_ld + c) = *reinterpret_cast<const uint4 *>(mine + t * ldv + c);
            }
        } else {
            for (int i = lane; i < kC * 16; i += 32) {
                const int t = i >> 4, c = i & 15;
                if (t < live && c < have) dst[t * v_ld + c] = mine[t * ldv + c];
            }
        }
        __syncthreads();
    }
    if (!a.state) return;
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row + (e >> 1) * 8, c = 8 * j + 2 * (lane & 3) + (e & 1);
            if (r < a.headdim && c < a.dstate) a.state[(bh * a.headdim + r) * (int64_t)a.dstate + c] = s[j][e];
        }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int NP, bool VECQK, bool VECV, bool STORE>
cudaError_t launch_t(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    // as many warps to a block as share its tiles of K, Q, N and P (eight
    // cover 128 columns), fewer while the grid would leave SMs empty
    int w = (a.headdim + 15) / 16;
    if (w > 8) w = 8;
    while (w > 1 && a.batch * a.heads * ((a.headdim + 16 * w - 1) / (16 * w)) < sms) w = (w + 1) / 2;
    const int vtiles = (a.headdim + 16 * w - 1) / (16 * w);
    const int bytes = 2 * stage_bytes<NP>(w);
    cudaError_t e = allow_smem<delta_chain_kernel<NP, VECQK, VECV, STORE>, 2 * stage_bytes<NP>(8)>();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.batch * a.heads * vtiles));
    delta_chain_kernel<NP, VECQK, VECV, STORE><<<grid, 32 * w, bytes, st>>>(a, ws, vtiles);
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

template <bool STORE>
static cudaError_t launch_chain(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    using namespace delta;
    const bool qk = a.dstate % 8 == 0 && aligned16(a.q) && aligned16(a.k);
    const bool v = a.headdim % 8 == 0 && aligned16(a.v) && aligned16(a.out);
    if (a.dstate <= 64) {
        if (qk) return v ? launch_t<64, true, true, STORE>(a, ws, sms, st) : launch_t<64, true, false, STORE>(a, ws, sms, st);
        return v ? launch_t<64, false, true, STORE>(a, ws, sms, st) : launch_t<64, false, false, STORE>(a, ws, sms, st);
    }
    if (qk) return v ? launch_t<128, true, true, STORE>(a, ws, sms, st) : launch_t<128, true, false, STORE>(a, ws, sms, st);
    return v ? launch_t<128, false, true, STORE>(a, ws, sms, st) : launch_t<128, false, false, STORE>(a, ws, sms, st);
}

cudaError_t launch_delta_chain(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    return launch_chain<false>(a, ws, sms, st);
}
cudaError_t launch_delta_chain_store(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    return launch_chain<true>(a, ws, sms, st);
}

}  // namespace ssm
