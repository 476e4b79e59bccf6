// delta_grad.cu -- the chunked gated delta rule's gradient, second half: dq, dk,
// dg and dbeta of all chunks at once (formulas at delta_bwd.cu), from what the
// forward's recomputation left (S0, r) and the pass backwards in time (dS1, dV).
//
// A block keeps a chunk's K and Q and sums dq and dk over the heads that share
// them (in registers, in the order of the heads); blocks take chunks in turn.
// The two states are the bulk of what is read: 128 of a unit's 208 KB at 128 x 128.
// They come 32 rows of S0 and of dS1 at a time, the next piece on its way while
// this one is multiplied, and the next head's other tiles while X and E are.
#include "delta_chunk.cuh"
#include "kernel_setup.cuh"

namespace ssm {
namespace delta {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// 16 warps: one has 16 of the chunk's tokens and a quarter of dstate.  (With 8
// warps and half of dstate each, a block stands still at every wait: two warps
// a scheduler.)
constexpr int kGradThreads = 512;
constexpr int kPiece = 32;  // rows of S0 and dS1 in shared memory at a time, twice

struct Place {     // one head of a chunk
    int64_t token;  // the chunk's first, counted over the batch
    int64_t unit;   // in the workspace
    unsigned w;     // chunk; the number of chunks or more: none
    int gr, h, hh, live;
};

template <int NP>
struct GradSmem {  // headdim rounded up to 16 (pp) decides the sizes of the rest
    bf16 k[kC][NP + 8], q[kC][NP + 8];
    bf16 x[2][kC][kMatLd], e[2][kC][kMatLd];       // X and E, high and low terms
    bf16 s[2][4][kPiece][NP + 8];                  // S0 high, low, dS1 high, low
    double cum[2][kC];
    float dec[2][kDec][kC];
    float db[4][kC];                               // column sums of the row blocks: dbeta's first terms
    float part[kGradThreads / 32];
    Place place[4];  // this head's, the next two's

    // Row sums of the quarters of dstate (dG, k . (r dS1)) have their place in the
    // corner of X's arrays above the diagonal, which no product reads: rows 0 to
    // 31, columns from 32 on.
    __device__ __forceinline__ float &dg(int quarter, int t) { return corner(x[0], quarter, t); }
    __device__ __forceinline__ float &kr(int quarter, int t) { return corner(x[1], quarter, t); }
    __device__ __forceinline__ static float &corner(bf16 (&m)[kC][kMatLd], int quarter, int t) {
        return reinterpret_cast<float *>(&m[t >> 1][32])[4 * (t & 1) + quarter];
    }
};
static_assert(sizeof(GradSmem<128>) + 5 * kC * (kDeltaMaxDstate + 8) * sizeof(bf16) <= 227 * 1024, "fits an SM");
template <int NP>
constexpr size_t grad_smem_bytes(int pp) {
    return sizeof(GradSmem<NP>) + (size_t)(5 * kC * (pp + 8)) * sizeof(bf16);
}

template <int NP, bool VECQK, bool VECV>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(DeltaBwdArgs p, DeltaChunkWs ws, unsigned chunks) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<NP> &sm = *reinterpret_cast<GradSmem<NP> *>(raw);
    constexpr int NT = NP / 32;  // column tiles of 8 per warp
    const DeltaArgs &a = p.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, qt = warp >> 2;
    // The row block: every scheduler (warp % 4) gets 2 or 3 of the 10 blocks on
    // and below the diagonal of a 64 x 64 product whose columns are split by qt.
    const int tb = (0x2130'3102'3210'3210ull >> (16 * qt + 4 * (warp & 3))) & 3;
    const int pp = (a.headdim + 15) / 16 * 16, ldp = pp + 8, pieces = (pp + kPiece - 1) / kPiece;
    constexpr int lds = NP + 8;
    bf16 *so = reinterpret_cast<bf16 *>(raw + sizeof(GradSmem<NP>));  // dO
    bf16 *sr = so + kC * ldp, *se = sr + 2 * kC * ldp;               // r, dV: high and low terms
    const unsigned nch = (unsigned)((a.seqlen + kC - 1) / kC);
    const int rep = a.heads / a.groups;
    const int64_t qk_ld = (int64_t)a.groups * a.dstate, v_ld = (int64_t)a.heads * a.headdim;
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int cf_row = cols_first_row(lane), cf_col = cols_first_col(lane);
    const int n0 = qt * (NP / 4);
    const int ta = 16 * tb + (lane >> 2);  // this thread's rows: ta, ta + 8

    auto place = [&](unsigned w) {  // a chunk's first head
        Place u;
        const unsigned bg = w / nch, ch = w - bg * nch, b = bg / (unsigned)a.groups;
        const int64_t left = a.seqlen - (int64_t)ch * kC;
        u.w = w;
        u.gr = (int)(bg - b * (unsigned)a.groups);
        u.h = u.gr * rep;
        u.hh = 0;
        u.live = (int)(left < kC ? left : kC);
        u.token = b * a.seqlen + (int64_t)ch * kC;
        u.unit = ((int64_t)b * a.heads + u.h) * nch + ch;
        return u;
    };
    auto after = [&](Place u) {
        if (u.hh + 1 == rep || u.w >= chunks) return place(u.w < chunks ? u.w + gridDim.x : u.w);
        ++u.hh;
        ++u.h;
        u.unit += nch;
        return u;
    };
    auto load_qk = [&](const Place &u) {
        const int64_t at = (u.token * a.groups + u.gr) * a.dstate;
        load_tile<VECQK>(&sm.k[0][0], lds, static_cast<const bf16 *>(a.k) + at, qk_ld, kC, NP, u.live, a.dstate, tid,
                         kGradThreads);
        load_tile<VECQK>(&sm.q[0][0], lds, static_cast<const bf16 *>(a.q) + at, qk_ld, kC, NP, u.live, a.dstate, tid,
                         kGradThreads);
    };
    auto load_head = [&](const Place &u) {
        const bf16 *go = static_cast<const bf16 *>(p.dout) + (u.token * a.heads + u.h) * a.headdim;
        const bf16 *r = ws.r + u.unit * 2 * kC * pp, *dv = ws.dv + u.unit * 2 * kC * pp;
        if (!VECV) load_tile<false>(so, ldp, go, v_ld, kC, pp, u.live, a.headdim, tid, kGradThreads);
        const int c = (tid & 15) * 8;  // no row has more than 16 pieces of 16 bytes
        if (c < pp) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (tid >> 4) + 32 * i;
                cp_async16(sr + row * ldp + c, r + row * pp + c, true);
                cp_async16(se + row * ldp + c, dv + row * pp + c, true);
                if (VECV && i < 2) {
                    const bool in = row < u.live && c < a.headdim;
                    cp_async16(so + row * ldp + c, in ? go + row * v_ld + c : go, in);
                }
            }
        }
    };
    auto load_piece = [&](const Place &u, int piece, int slot) {
        const int64_t at = u.unit * 2 * pp * NP;
#pragma unroll
        for (int i = tid; i < 4 * (NP / 8) * kPiece; i += kGradThreads) {
            const int row = i % kPiece, g = i / kPiece % (NP / 8), which = i / kPiece / (NP / 8);
            const bf16 *src = (which < 2 ? ws.s0 : ws.ds1) + at + state_at<NP>(pp, which & 1, piece * kPiece + row, 8 * g);
            if (piece * kPiece + row < pp) cp_async16(&sm.s[slot][which][row][8 * g], src, true);
        }
    };
    // the decays of a head, fetched by thread (token) and put into the buffer of its turn
    auto fetch_decays = [&](const Place &u, float &d, float2 &g01) {
        if (tid < kDec * kC) d = ws.dec[u.unit * (kDec * kC) + tid];
        if (warp == 15) {
            const float *g = a.g + u.token * a.heads + u.h;
            const int t = 2 * lane;
            g01.x = t < u.live ? g[(int64_t)t * a.heads] : 0.f;
            g01.y = t + 1 < u.live ? g[(int64_t)(t + 1) * a.heads] : 0.f;
        }
    };
    auto put_decays = [&](int turn, float d, float2 g01) {
        if (tid < kDec * kC) (&sm.dec[turn][0][0])[tid] = d;
        if (warp == 15) {
            const int t = 2 * lane;
            const double g0 = fmax((double)g01.x, -1e4), g1 = fmax((double)g01.y, -1e4);
            double sum = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            sm.cum[turn][t] = sum - g1;
            sm.cum[turn][t + 1] = sum;
        }
    };

    int slot = 0;
    {
        const Place u = place(blockIdx.x);
        if (tid == 0) {
            sm.place[0] = u;
            sm.place[1] = after(u);
        }
        float d = 0.f;
        float2 g01 = make_float2(0.f, 0.f);
        fetch_decays(u, d, g01);
        load_qk(u);
        load_head(u);
        load_piece(u, 0, 0);
        cp_async_commit();
        put_decays(0, d, g01);
    }
    float tq[NT][4], tk[NT][4];  // sums over the group's heads
    for (unsigned head = 0;; ++head) {
        cp_async_wait<0>();
        __syncthreads();  // this head's tiles and first piece; the last one's sums are read
        const int turn = head & 1;
        const float(&dec)[kDec][kC] = sm.dec[turn];
        const Place &u = sm.place[head & 3], &next = sm.place[(head + 1) & 3];
        const bool more = next.w < chunks;
        if (tid == 0) sm.place[(head + 2) & 3] = after(next);
        if (u.hh == 0)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) tq[j][i] = tk[j][i] = 0.f;
        // x = scale Gam (dO_t . r_s), y = -Gam (dV_t . r_s): 16 rows and 16 columns
        // a warp, up to the diagonal; q_t . k_s and k_t . k_s beside them for dbeta
        {
            float cx[2][4], ce[2][4], cqk[2][4], ckk[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) cx[j][i] = ce[j][i] = cqk[j][i] = ckk[j][i] = 0.f;
            if (qt <= tb) {
#pragma unroll 2
                for (int kk = 0; kk < pp / 16; ++kk) {
                    uint32_t ao[4], ah[4], al[4], fh[4], fl[4];
                    const int at = (16 * tb + rf_row) * ldp + 16 * kk + rf_col;
                    const int bt = (16 * qt + cf_row) * ldp + 16 * kk + cf_col;
                    ldm4(ao, so + at);
                    ldm4(ah, se + at);
                    ldm4(al, se + kC * ldp + at);
                    ldm4(fh, sr + bt);
                    ldm4(fl, sr + kC * ldp + bt);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma(cx[i], ao, fh[2 * i], fh[2 * i + 1]);
                        mma(ce[i], ah, fh[2 * i], fh[2 * i + 1]);
                        mma(cx[i], ao, fl[2 * i], fl[2 * i + 1]);
                        mma(ce[i], ah, fl[2 * i], fl[2 * i + 1]);
                        mma(ce[i], al, fh[2 * i], fh[2 * i + 1]);
                    }
                }
#pragma unroll 2
                for (int kk = 0; kk < NP / 16; ++kk) {
                    uint32_t aq[4], ak[4], f[4];
                    ldm4(aq, &sm.q[16 * tb + rf_row][16 * kk + rf_col]);
                    ldm4(ak, &sm.k[16 * tb + rf_row][16 * kk + rf_col]);
                    ldm4(f, &sm.k[16 * qt + cf_row][16 * kk + cf_col]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma(cqk[i], aq, f[2 * i], f[2 * i + 1]);
                        mma(ckk[i], ak, f[2 * i], f[2 * i + 1]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int s = 16 * qt + 8 * j + 2 * (lane & 3);
                float cols[2] = {0.f, 0.f};
                if (qt <= tb) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = ta + 8 * i;
                        float xv[2], ev[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float gam = s + c <= t ? expf((float)(sm.cum[turn][t] - sm.cum[turn][s + c])) : 0.f;
                            const float x = s + c <= t ? a.scale * gam * cx[j][2 * i + c] : 0.f;
                            const float y = s + c < t ? -gam * ce[j][2 * i + c] : 0.f;
                            if (s + c <= t) cols[c] += x * cqk[j][2 * i + c] + y * ckk[j][2 * i + c];
                            xv[c] = x * dec[2][s + c];
                            ev[c] = y * dec[2][s + c];
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
        // dO S0, dV S0, r dS1; <S0, dS1> on the way
        float cq[NT][4], cl[NT][4], cr[NT][4], inner = 0.f, nd = 0.f;
        float2 ng = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) cq[j][i] = cl[j][i] = cr[j][i] = 0.f;
        for (int piece = 0; piece < pieces; ++piece) {
            if (piece > 0) {
                cp_async_wait<0>();
                __syncthreads();  // this piece is here, and the one before it is read
            }
            if (piece + 1 < pieces)
                load_piece(u, piece + 1, slot ^ 1);
            else if (more)
                load_piece(next, 0, slot ^ 1);
            cp_async_commit();
            const bf16 *ss = &sm.s[slot][0][0][0];
            const int rows = pp - piece * kPiece < kPiece ? pp - piece * kPiece : kPiece;
            for (int kk = 0; kk < rows / 16; ++kk) {
                uint32_t ao[4], ah[4], al[4], rh[4], rl[4];
                const int at = (16 * tb + rf_row) * ldp + piece * kPiece + 16 * kk + rf_col;
                ldm4(ao, so + at);
                ldm4(ah, se + at);
                ldm4(al, se + kC * ldp + at);
                ldm4(rh, sr + at);
                ldm4(rl, sr + kC * ldp + at);
#pragma unroll
                for (int nn = 0; nn < NT / 2; ++nn) {
                    uint32_t fh[4], fl[4];
                    const bf16 *bt = ss + (16 * kk + rf_row) * lds + n0 + 16 * nn + rf_col;
                    ldm4t(fh, bt);
                    ldm4t(fl, bt + kPiece * lds);
                    uint32_t dh[4], dl[4];
                    ldm4t(dh, bt + 2 * kPiece * lds);
                    ldm4t(dl, bt + 3 * kPiece * lds);
                    // an accumulator's next product comes six products later
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma(cq[2 * nn + i], ao, fh[2 * i], fh[2 * i + 1]);
                        mma(cl[2 * nn + i], ah, fh[2 * i], fh[2 * i + 1]);
                        mma(cr[2 * nn + i], rh, dh[2 * i], dh[2 * i + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma(cq[2 * nn + i], ao, fl[2 * i], fl[2 * i + 1]);
                        mma(cl[2 * nn + i], ah, fl[2 * i], fl[2 * i + 1]);
                        mma(cr[2 * nn + i], rh, dl[2 * i], dl[2 * i + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma(cl[2 * nn + i], al, fh[2 * i], fh[2 * i + 1]);
                        mma(cr[2 * nn + i], rl, dh[2 * i], dh[2 * i + 1]);
                    }
                }
            }
            for (int i = tid; i < kPiece * (NP / 8); i += kGradThreads) {
                const int row = i % kPiece, c = i / kPiece * 8;
                if (row < rows) {
                    uint4 v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4 *>(ss + (q * kPiece + row) * lds + c);
                    const uint32_t *w0 = &v[0].x, *w1 = &v[1].x, *w2 = &v[2].x, *w3 = &v[3].x;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        inner = fmaf(low_of(w0[q]) + low_of(w1[q]), low_of(w2[q]) + low_of(w3[q]), inner);
                        inner = fmaf(high_of(w0[q]) + high_of(w1[q]), high_of(w2[q]) + high_of(w3[q]), inner);
                    }
                }
            }
            slot ^= 1;
        }
        inner *= dec[0][kC - 1];
        __syncthreads();  // dO, dV and r are read; X and E are written
        if (more) {
            load_head(next);
            fetch_decays(next, nd, ng);
        }
        cp_async_commit();
        // q = scale gam dO S0 + X K,  l = E K - gam dV S0,  r = w beta r dS1 + X^T Q + E^T K
        float dot[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float g = dec[0][ta + 8 * i], fq = a.scale * g, fl = -g;
            const float f = dec[1][ta + 8 * i] * dec[2][ta + 8 * i];
            float kr = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = n0 + 8 * j + 2 * (lane & 3);
                const uint32_t kv = *reinterpret_cast<const uint32_t *>(&sm.k[ta + 8 * i][n]);
                kr += low_of(kv) * cr[j][2 * i] + high_of(kv) * cr[j][2 * i + 1];
                cq[j][2 * i] *= fq; cq[j][2 * i + 1] *= fq;
                cl[j][2 * i] *= fl; cl[j][2 * i + 1] *= fl;
                cr[j][2 * i] *= f; cr[j][2 * i + 1] *= f;
            }
            inner = fmaf(f, kr, inner);
            kr += __shfl_xor_sync(0xffffffffu, kr, 1);
            kr += __shfl_xor_sync(0xffffffffu, kr, 2);
            if ((lane & 3) == 0) sm.kr(qt, ta + 8 * i) = kr;
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
        // q . dq + k . (l - r) of this warp's rows; the sums over heads
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = n0 + 8 * j + 2 * (lane & 3);
                const uint32_t qv = *reinterpret_cast<const uint32_t *>(&sm.q[ta + 8 * i][n]);
                const uint32_t kv = *reinterpret_cast<const uint32_t *>(&sm.k[ta + 8 * i][n]);
                dot[i] += low_of(qv) * cq[j][2 * i] + high_of(qv) * cq[j][2 * i + 1] +
                          low_of(kv) * (cl[j][2 * i] - cr[j][2 * i]) +
                          high_of(kv) * (cl[j][2 * i + 1] - cr[j][2 * i + 1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tq[j][2 * i + c] += cq[j][2 * i + c];
                    tk[j][2 * i + c] += cl[j][2 * i + c] + cr[j][2 * i + c];
                }
            }
        // dg and dbeta of this head
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 1);
            dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 2);
            if ((lane & 3) == 0) sm.dg(qt, ta + 8 * i) = dot[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
        if (lane == 0) sm.part[warp] = inner;
        if (more) put_decays(turn ^ 1, nd, ng);
        __syncthreads();  // the sums are there; K and Q are read
        if (u.hh + 1 == rep && more) load_qk(next);
        cp_async_commit();
        if (warp == 0) {
            float whole = 0.f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i) whole += sm.part[i];
            // lane i: tokens 63 - 2 i and 62 - 2 i; a prefix sum over lanes is a sum from the end
            const int t = kC - 1 - 2 * lane;
            const float d1 = (sm.dg(0, t) + sm.dg(1, t)) + (sm.dg(2, t) + sm.dg(3, t));
            const float d0 = (sm.dg(0, t - 1) + sm.dg(1, t - 1)) + (sm.dg(2, t - 1) + sm.dg(3, t - 1));
            float sum = d1 + d0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const int64_t at = u.token * a.heads + u.h;
            if (t < u.live) p.dg[at + (int64_t)t * a.heads] = whole + (sum - d0);
            if (t - 1 < u.live) p.dg[at + (int64_t)(t - 1) * a.heads] = whole + sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = t - i;
                const float db = (sm.db[0][s] + sm.db[1][s]) + (sm.db[2][s] + sm.db[3][s]);
                const float kr = (sm.kr(0, s) + sm.kr(1, s)) + (sm.kr(2, s) + sm.kr(3, s));
                if (s < u.live) p.dbeta[at + (int64_t)s * a.heads] = db + dec[1][s] * kr;
            }
        }
        if (u.hh + 1 == rep) {
            const int64_t at = (u.token * a.groups + u.gr) * a.dstate;
            bf16 *dq = static_cast<bf16 *>(p.dq) + at, *dk = static_cast<bf16 *>(p.dk) + at;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = ta + 8 * i, n = n0 + 8 * j + 2 * (lane & 3);
                    if (t >= u.live) continue;
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
        if (!more) break;
    }
}

template <int NP, bool VECQK, bool VECV>
cudaError_t launch_grad_t(const DeltaBwdArgs &p, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    const DeltaArgs &a = p.f;
    const size_t bytes = grad_smem_bytes<NP>((a.headdim + 15) / 16 * 16);
    cudaError_t e = allow_smem<delta_grad_kernel<NP, VECQK, VECV>, (int)grad_smem_bytes<NP>(kDeltaMaxDstate)>();
    if (e != cudaSuccess) return e;
    const int64_t chunks = a.batch * a.groups * ((a.seqlen + kC - 1) / kC);
    const dim3 grid((unsigned)(chunks < sms ? chunks : sms));
    delta_grad_kernel<NP, VECQK, VECV><<<grid, kGradThreads, bytes, st>>>(p, ws, (unsigned)chunks);
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

cudaError_t launch_delta_grad(const DeltaBwdArgs &p, const DeltaChunkWs &ws, int sms, cudaStream_t st) {
    using namespace delta;
    const bool qk = p.f.dstate % 8 == 0 && aligned16(p.f.q) && aligned16(p.f.k) && aligned16(p.dq) && aligned16(p.dk);
    const bool v = p.f.headdim % 8 == 0 && aligned16(p.dout);
    if (p.f.dstate <= 64) {
        if (qk) return v ? launch_grad_t<64, true, true>(p, ws, sms, st) : launch_grad_t<64, true, false>(p, ws, sms, st);
        return v ? launch_grad_t<64, false, true>(p, ws, sms, st) : launch_grad_t<64, false, false>(p, ws, sms, st);
    }
    if (qk) return v ? launch_grad_t<128, true, true>(p, ws, sms, st) : launch_grad_t<128, true, false>(p, ws, sms, st);
    return v ? launch_grad_t<128, false, true>(p, ws, sms, st) : launch_grad_t<128, false, false>(p, ws, sms, st);
}

}  // namespace ssm
