// delta_fused.cu -- the chunked gated delta rule on the sm_100a tensor cores,
// one kernel (notation of delta_chunk.cuh).
//
// One CTA owns 128 state rows of a head (the columns of V) for the whole
// sequence and walks over its chunks of 64 tokens.  Everything is computed
// transposed, with the state rows as the 128 lanes of tensor memory: then the
// state, beta R and w u -- each an accumulator of one product and the left
// operand of the next -- never leave tensor memory, and the row-wise work is
// one thread per lane.  Per chunk, three tcgen05 products:
//   [X | O1]^T = S [K; Q]^T                       (128 x 128, K = dstate)
//   [Y | O2]^T = (beta R)^T [N; P - P beta N]^T   (128 x 128, K = 64),  R = V - gam X
//   S          = gam_C S + (w beta r)^T K         (128 x dstate, K = 64),  r = R - Y
//   out        = scale gam O1 + O2
// O2 reads beta R instead of u = beta r (P u = (P - P beta N) beta R), so the
// output needs no product behind r.  Operands that are not bf16 already take
// two bf16 terms (state: 2 products instead of 1; beta R with N, P: 3).
//
// N and P - P beta N of the next chunk are made meanwhile by four warps of
// their own (mma.sync, float32 and float64 arithmetic): K K^T and Q K^T, the
// decays, then N by 32 x 32 blocks -- N11 and N22 by substitution, one column
// per thread, N21 = (I - N22 beta) Abar21 (I - beta N11) by products of
// two-term operands.  A kernel of their own would have to write and read 64 KB
// per chunk and head, as much as q, k, v and out together.
//
// Warps: 0-7 row-wise work (two per lane quarter, each half of the columns),
// 8-11 the chunk matrices, 12 issues the products, 13 the TMA copies.  They
// meet at mbarriers only; every wait is bounded and reports through the device
// status word.
#include "delta_chunk.cuh"
#include "scan_kernels.cuh"
#include "tma_maps.cuh"
#include "umma.cuh"

namespace ssm {
namespace delta {
namespace {

using namespace umma;

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait
constexpr int kRowWarps = 8, kMatWarps = 4;
constexpr int kThreadsF = (kRowWarps + kMatWarps + 2) * 32;
constexpr uint32_t kHalfTile = kC * 128;  // 64 rows x 128 bytes
constexpr int kALd = kC + 4, kNLd = 36;

// tensor memory columns
constexpr uint32_t kTX = 0, kTO1 = 64, kTY = 128, kTO2 = 192, kTS = 256, kTSh = 384, kTSl = 448;
// beta R (where X was) and w u (where Y was): tokens 32 wg .. 32 wg + 31 of
// both terms stay within the columns that their warps have read themselves
__host__ __device__ constexpr uint32_t operand_col(uint32_t base, int kstep, int term) {
    return base + 32 * (kstep >> 1) + 16 * term + 8 * (kstep & 1);
}

struct __align__(16) Dec {         // per chunk, float32
    float gam[kC], gs[kC], beta[kC], wb[kC];  // exp G, scale exp G, beta, exp(G_C - G) beta
    float whole, pad[3];           // exp G_C
};

template <int NT>
struct FusedSmem {
    unsigned char kq[2][NT][2 * kHalfTile];  // per stage and 64 columns: K rows, then Q rows
    unsigned char v[2][2][kHalfTile];        // V, later the output
    unsigned char np[2][2][2 * kHalfTile];   // [N; P - P beta N]: high, low term
    float a[kC][kALd];                       // Abar
    float n[2][32][kNLd];                    // N11, N22
    float t1[32][kNLd];
    double cum[kC];
    Dec dec[2];
    // Barriers whose waiters may fall a chunk behind have one per stage, so that
    // a phase cannot be overtaken.
    uint64_t ld[2], prep[2];                 // copies landed; chunk matrices ready
    uint64_t x, y, s[2];                     // products complete
    uint64_t s_ready, r_ready, u_ready, o_ready[2];  // row-wise results written
    uint64_t fin;
    uint32_t tmem;
};

struct FusedArgs {
    const float *g, *beta, *h0;
    float *state;
    float scale;
    int64_t seqlen;
    int heads, rep, headdim, dstate, vtiles;
    unsigned int *status;
};

__device__ __forceinline__ void mats_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The same barrier; true where `ok` holds in all four warps.
__device__ __forceinline__ bool mats_all(bool ok) {
    uint32_t all;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbar.red.and.pred p, 1, 128, q;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(all) : "r"((uint32_t)ok) : "memory");
    return all != 0;
}

__device__ __forceinline__ bf16 *tile_at(unsigned char *tile, int row, int col) {
    return reinterpret_cast<bf16 *>(tile + sw128_offset(row, col >> 3) + (col & 7) * 2);
}

// ------------------------------------------------------- the chunk matrices
// acc (16 x 16, two n-tiles) -= A (16 x 32) B (32 x 16) with two-term operands;
// a(i, k), b(k, j) give float32 values.
template <typename FA, typename FB>
__device__ __forceinline__ void product32(float (&acc)[2][4], int lane, FA a, FB b) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (lane >> 2) + 8 * (i & 1), k = 16 * kk + 2 * (lane & 3) + 8 * (i >> 1);
            split(-a(r, k), -a(r, k + 1), hi[i], lo[i]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = 8 * j + (lane >> 2), k = 16 * kk + 2 * (lane & 3);
            uint32_t bh0, bl0, bh1, bl1;
            split(b(k, n), b(k + 1, n), bh0, bl0);
            split(b(k + 8, n), b(k + 9, n), bh1, bl1);
            mma(acc[j], hi, bh0, bh1);
            mma(acc[j], lo, bh0, bh1);
            mma(acc[j], hi, bl0, bl1);
        }
    }
}

template <int NT>
__device__ __forceinline__ void chunk_matrices(FusedSmem<NT> &sm, const FusedArgs &a, int64_t c, int live, int w,
                                               int lane, float g0, float g1, float b0, float b1) {
    Dec &dec = sm.dec[c & 1];
    unsigned char *kq[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) kq[i] = sm.kq[c & 1][i];
    if (w == 0) {
        double d0 = 2 * lane < live ? fmax((double)g0, -1e4) : 0.0, d1 = 2 * lane + 1 < live ? fmax((double)g1, -1e4) : 0.0;
        double sum = d0 + d1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const double end = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const double cum = i ? sum : sum - d1;
            const float be = t < live ? (i ? b1 : b0) : 0.f, gam = expf((float)cum);
            sm.cum[t] = cum;
            dec.gam[t] = gam;
            dec.gs[t] = a.scale * gam;
            dec.beta[t] = be;
            dec.wb[t] = expf((float)(end - cum)) * be;
        }
        if (lane == 31) dec.whole = expf((float)end);
    }
    // K K^T and Q K^T, rows 16 w .. 16 w + 15, blocks up to the diagonal
    float ck[kC / 8][4], cq[kC / 8][4];
#pragma unroll
    for (int j = 0; j < kC / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[j][e] = cq[j][e] = 0.f;
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int cf_row = cols_first_row(lane), cf_col = cols_first_col(lane);
#pragma unroll
    for (int kk = 0; kk < 4 * NT; ++kk) {
        unsigned char *t = kq[kk / 4];
        const int col = 16 * (kk % 4);
        uint32_t ak[4], aq[4];
        ldm4(ak, tile_at(t, 16 * w + rf_row, col + rf_col));
        ldm4(aq, tile_at(t, kC + 16 * w + rf_row, col + rf_col));
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj) {
            if (jj > w) continue;
            uint32_t bk[4];
            ldm4(bk, tile_at(t, 16 * jj + cf_row, col + cf_col));
            mma(ck[2 * jj], ak, bk[0], bk[1]);
            mma(ck[2 * jj + 1], ak, bk[2], bk[3]);
            mma(cq[2 * jj], aq, bk[0], bk[1]);
            mma(cq[2 * jj + 1], aq, bk[2], bk[3]);
        }
    }
    mats_sync();  // cum
#pragma unroll
    for (int j = 0; j < kC / 8; ++j) {
        if (j > 2 * w + 1) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 16 * w + (lane >> 2) + 8 * (e >> 1), s = 8 * j + 2 * (lane & 3) + (e & 1);
            const float gam = s <= t ? expf((float)(sm.cum[t] - sm.cum[s])) : 0.f;
            cq[j][e] = s <= t ? a.scale * gam * cq[j][e] : 0.f;
            sm.a[t][s] = s < t ? gam * ck[j][e] : 0.f;
        }
    }
    mats_sync();  // Abar
    unsigned char *nh = sm.np[c & 1][0], *nl = sm.np[c & 1][1];
    if (w < 2) {
        // N11 (w = 0), N22 (w = 1): column `lane`, row after row; y = beta N
        const int o = 32 * w;
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float acc[4] = {i > lane ? sm.a[o + i][o + lane] : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s4 = 0; s4 < i; s4 += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&sm.a[o + i][o + s4]);
                acc[0] = fmaf(-m.x, y[s4], acc[0]);
                if (s4 + 1 < i) acc[1] = fmaf(-m.y, y[s4 + 1], acc[1]);
                if (s4 + 2 < i) acc[2] = fmaf(-m.z, y[s4 + 2], acc[2]);
                if (s4 + 3 < i) acc[3] = fmaf(-m.w, y[s4 + 3], acc[3]);
            }
            const float x = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            y[i] = dec.beta[o + i] * x;
            sm.n[w][i][lane] = x;
            const bf16 hi = __float2bfloat16_rn(x);
            *tile_at(nh, o + i, o + lane) = hi;
            *tile_at(nl, o + i, o + lane) = __float2bfloat16_rn(x - __bfloat162float(hi));
        }
    }
    mats_sync();  // N11, N22
    const int qi = 16 * (w >> 1), qj = 16 * (w & 1);  // this warp's 16 x 16 of the 32 x 32 block N21
    float acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[j][e] = sm.a[32 + qi + (lane >> 2) + 8 * (e >> 1)][qj + 8 * j + 2 * (lane & 3) + (e & 1)];
    product32(acc, lane, [&](int i, int k) { return sm.a[32 + qi + i][k] * dec.beta[k]; },
              [&](int k, int j) { return sm.n[0][k][qj + j]; });
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sm.t1[qi + (lane >> 2) + 8 * (e >> 1)][qj + 8 * j + 2 * (lane & 3) + (e & 1)] = acc[j][e];
    mats_sync();  // Abar21 (I - beta N11)
    product32(acc, lane, [&](int i, int k) { return sm.n[1][qi + i][k] * dec.beta[32 + k]; },
              [&](int k, int j) { return sm.t1[k][qj + j]; });
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t hi, lo;
            split(acc[j][2 * half], acc[j][2 * half + 1], hi, lo);
            const int row = 32 + qi + (lane >> 2) + 8 * half, col = qj + 8 * j + 2 * (lane & 3);
            *reinterpret_cast<uint32_t *>(tile_at(nh, row, col)) = hi;
            *reinterpret_cast<uint32_t *>(tile_at(nl, row, col)) = lo;
        }
    mats_sync();  // N
    // P - (P beta) N: blocks of 16 columns from the last, whose left operand no
    // earlier step has changed (N is strictly lower)
#pragma unroll
    for (int kk = 0; kk < kC / 16; ++kk) {
        if (kk > w) continue;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * kk + (i >> 1);
            const float2 b2 = *reinterpret_cast<const float2 *>(&dec.beta[8 * j + 2 * (lane & 3)]);
            split(-b2.x * cq[j][2 * (i & 1)], -b2.y * cq[j][2 * (i & 1) + 1], hi[i], lo[i]);
        }
#pragma unroll
        for (int jj = 0; jj <= kk; ++jj) {
            uint32_t f[4], fl[4];
            ldm4t(f, tile_at(nh, 16 * kk + rf_row, 16 * jj + rf_col));
            ldm4t(fl, tile_at(nl, 16 * kk + rf_row, 16 * jj + rf_col));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma(cq[2 * jj + i], hi, f[2 * i], f[2 * i + 1]);
                mma(cq[2 * jj + i], lo, f[2 * i], f[2 * i + 1]);
                mma(cq[2 * jj + i], hi, fl[2 * i], fl[2 * i + 1]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kC / 8; ++j) {
        if (j > 2 * w + 1) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t hi, lo;
            split(cq[j][2 * half], cq[j][2 * half + 1], hi, lo);
            const int row = kC + 16 * w + (lane >> 2) + 8 * half, col = 8 * j + 2 * (lane & 3);
            *reinterpret_cast<uint32_t *>(tile_at(nh, row, col)) = hi;
            *reinterpret_cast<uint32_t *>(tile_at(nl, row, col)) = lo;
        }
    }
}

// ------------------------------------------------------------- row-wise work
// 32 columns as two bf16 terms, 16 tensor memory columns each.
__device__ __forceinline__ void put_terms(uint32_t hi_col, uint32_t lo_col, const float (&v)[32]) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) split(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
    tmem_st16(hi_col, hi);
    tmem_st16(lo_col, lo);
}

// 32 columns of the state: its two terms, and gam_C of the next chunk times it
// where the next chunk's product accumulates.
__device__ __forceinline__ void put_state(uint32_t tl, int col, const float (&s)[32], float whole) {
    put_terms(tl + kTSh + col / 2, tl + kTSl + col / 2, s);
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(whole * s[i]);
    tmem_st32(tl + kTS + col, r);
}

template <int NT>
__global__ void __launch_bounds__(kThreadsF, 1)
delta_fused_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapO,
                   const FusedArgs a) {
    extern __shared__ unsigned char raw[];
    FusedSmem<NT> &sm = *reinterpret_cast<FusedSmem<NT> *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t bh = blockIdx.x / a.vtiles;
    const int v0 = (int)(blockIdx.x - bh * a.vtiles) * 128;
    const int64_t b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / a.rep;
    const int nch = (int)((a.seqlen + kC - 1) / kC);
    const int halves = a.headdim - v0 > 64 ? 2 : 1;  // 64-column halves of V in this CTA

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.ld[i], 1);
            mbar_init(&sm.prep[i], kMatWarps);
            mbar_init(&sm.s[i], 1);
            mbar_init(&sm.o_ready[i], kRowWarps);
        }
        mbar_init(&sm.x, 1);
        mbar_init(&sm.y, 1);
        mbar_init(&sm.s_ready, kRowWarps);
        mbar_init(&sm.r_ready, kRowWarps);
        mbar_init(&sm.u_ready, kRowWarps);
        mbar_init(&sm.fin, 1);
        mbar_fence_init();
    }
    // the parts of [N; P] above the diagonal are written here only
    for (int i = tid; i < (int)sizeof(sm.np) / 16; i += kThreadsF)
        reinterpret_cast<uint4 *>(sm.np)[i] = make_uint4(0, 0, 0, 0);
    if (warp == 0) tmem_alloc(&sm.tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = sm.tmem;
    auto wait = [&](uint64_t *bar, uint32_t par) {
        if (!mbar_wait(bar, par & 1u, kWaitNs)) {
            atomicOr(a.status, 4u);
            return false;
        }
        return true;
    };
    auto signal = [&](uint64_t *bar) {  // one arrival per warp, after the warp's writes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp == kRowWarps + kMatWarps) {
        // ------------------------------------------------ the products
        const uint32_t el = elect_one();
        auto wait_w = [&](uint64_t *bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)) != 0; };
        constexpr uint32_t id_k = idesc_bf16(128, 128, kMajorK, kMajorK);
        constexpr uint32_t id_s = idesc_bf16(128, 64 * NT, kMajorK, kMajorMN);
        bool ok = true;
        for (int c = 0; ok && c < nch; ++c) {
            const int st = c & 1;
            if (!(ok = wait_w(&sm.ld[st], c >> 1)) || !(ok = wait_w(&sm.s_ready, c))) break;
            fence_after_sync();
            const uint64_t dkq = desc_sw128(smem_u32(sm.kq[st][0]), 16, 1024);
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int k = 0; k < 4 * NT; ++k)
                    mma_bf16_ts_if(el, tm + kTX, tm + (term ? kTSl : kTSh) + 8 * k,
                                   dkq + (((k / 4) * 2 * kHalfTile + (k % 4) * 32) >> 4), id_k, term > 0 || k > 0);
            mma_commit_if(el, &sm.x);
            if (!(ok = wait_w(&sm.prep[st], c >> 1)) || !(ok = wait_w(&sm.r_ready, c))) break;
            fence_after_sync();
            const uint64_t dnh = desc_sw128(smem_u32(sm.np[st][0]), 16, 1024);
            const uint64_t dnl = desc_sw128(smem_u32(sm.np[st][1]), 16, 1024);
#pragma unroll
            for (int term = 0; term < 3; ++term)  // high high, low high, high low
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_ts_if(el, tm + kTY, tm + operand_col(kTX, k, term == 1),
                                   (term == 2 ? dnl : dnh) + ((k * 32) >> 4), id_k, term > 0 || k > 0);
            mma_commit_if(el, &sm.y);
            if (!(ok = wait_w(&sm.u_ready, c))) break;
            fence_after_sync();
            // K as the right operand with tokens as the summed index: rows of 64
            // state columns, the second 64 in the next tile
            const uint64_t dk = desc_sw128(smem_u32(sm.kq[st][0]), 2 * kHalfTile, 1024);
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_ts_if(el, tm + kTS, tm + operand_col(kTY, k, term), dk + ((k * 2048) >> 4), id_s, true);
            mma_commit_if(el, &sm.s[st]);
        }
        mma_commit_if(el, &sm.fin);  // whatever was issued completes before tensor memory goes away
        (void)mbar_wait(&sm.fin, 0u, kWaitNs);
        __syncwarp();
    } else if (warp == kRowWarps + kMatWarps + 1) {
        // -------------------------------------------------- the copies
        const uint32_t el = elect_one();
        auto wait_w = [&](uint64_t *bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)) != 0; };
        int issued[2] = {0, 0};
        auto load = [&](int c) {
            const int st = c & 1;
            if (el) {
                mbar_expect_tx(&sm.ld[st], (uint32_t)(2 * NT + halves) * kHalfTile);
                const int32_t t0 = c * kC;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    tma_load_3d(sm.kq[st][i], &mapK, gr * a.dstate + 64 * i, t0, (int32_t)b, &sm.ld[st]);
                    tma_load_3d(sm.kq[st][i] + kHalfTile, &mapQ, gr * a.dstate + 64 * i, t0, (int32_t)b, &sm.ld[st]);
                }
                for (int i = 0; i < halves; ++i)
                    tma_load_3d(sm.v[st][i], &mapV, h * a.headdim + v0 + 64 * i, t0, (int32_t)b, &sm.ld[st]);
            }
            if (st) ++issued[1]; else ++issued[0];
        };
        load(0);
        if (nch > 1) load(1);
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1;
            if (!wait_w(&sm.o_ready[st], c >> 1)) break;
            if (el) {
                for (int i = 0; i < halves; ++i)
                    tma_store_3d(&mapO, h * a.headdim + v0 + 64 * i, c * kC, (int32_t)b, sm.v[st][i]);
                tma_store_commit();
                tma_store_wait_read<0>();
            }
            __syncwarp();
            if (c + 2 >= nch) continue;
            if (!wait_w(&sm.s[st], c >> 1)) break;  // K and Q are read
            load(c + 2);
        }
        if (el) tma_store_wait_all<0>();
        if (issued[0] > 0) (void)mbar_wait(&sm.ld[0], (uint32_t)(issued[0] - 1) & 1u, kWaitNs);
        if (issued[1] > 0) (void)mbar_wait(&sm.ld[1], (uint32_t)(issued[1] - 1) & 1u, kWaitNs);
        __syncwarp();
    } else if (warp >= kRowWarps) {
        // ------------------------------------------- the chunk matrices
        const int w = warp - kRowWarps;
        const float *g = a.g + b * a.seqlen * a.heads + h, *be = a.beta + b * a.seqlen * a.heads + h;
        float g0 = 0.f, g1 = 0.f, b0 = 0.f, b1 = 0.f;
        auto fetch = [&](int64_t c) {
            const int64_t t = c * kC + 2 * lane;
            if (w != 0) return;
            if (t < a.seqlen) { g0 = __ldg(g + t * a.heads); b0 = __ldg(be + t * a.heads); }
            if (t + 1 < a.seqlen) { g1 = __ldg(g + (t + 1) * a.heads); b1 = __ldg(be + (t + 1) * a.heads); }
        };
        fetch(0);
        for (int c = 0; c < nch; ++c) {
            bool ok = wait(&sm.ld[c & 1], c >> 1);
            if (c >= 2) ok = wait(&sm.o_ready[c & 1], (c - 2) >> 1) && ok;  // chunk c - 2 is done with its matrices
            if (!mats_all(ok)) break;
            const int64_t left = a.seqlen - (int64_t)c * kC;
            const float c0 = g0, c1 = g1, d0 = b0, d1 = b1;
            if (c + 1 < nch) fetch(c + 1);
            chunk_matrices<NT>(sm, a, c, (int)(left < kC ? left : kC), w, lane, c0, c1, d0, d1);
            fence_proxy_async();
            signal(&sm.prep[c & 1]);
        }
    } else {
        // --------------------------------------------- the row-wise work
        const int quad = warp & 3, wg = warp >> 2, r = 32 * quad + lane;
        const bool active = 32 * quad < 64 * halves;  // the warp's lanes hold rows of the state
        const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
        const int64_t row = bh * a.headdim + v0 + r;
        bool ok = wait(&sm.prep[0], 0);
        if (active) {
            const float whole = sm.dec[0].whole;
#pragma unroll
            for (int p = 0; p < NT; ++p) {
                const int col = 32 * (NT * wg + p);
                float s[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (a.h0) {
                        const float *src = a.h0 + row * a.dstate + col + i;
                        x = make_float4(src[0], src[1], src[2], src[3]);
                    }
                    s[i] = x.x; s[i + 1] = x.y; s[i + 2] = x.z; s[i + 3] = x.w;
                }
                put_state(tl, col, s, whole);
            }
            tmem_wait_st();
        }
        fence_before_sync();
        signal(&sm.s_ready);
        for (int c = 0; ok && c < nch; ++c) {
            const int st = c & 1;
            const Dec &dec = sm.dec[st];
            unsigned char *vt = sm.v[st][r >> 6];
            const int vp = (r & 63) >> 3, vo = (r & 7) * 2;
            float res[32];
            // R = V - gam X, and beta R as an operand
            if (!(ok = wait(&sm.ld[st], c >> 1)) || !(ok = wait(&sm.x, c))) break;
            fence_after_sync();
            if (active) {
                tmem_ld32(tl + kTX + 32 * wg, res);
                tmem_wait_ld();
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int t = 32 * wg + i;
                    const float4 g4 = *reinterpret_cast<const float4 *>(&dec.gam[t]);
                    const float4 b4 = *reinterpret_cast<const float4 *>(&dec.beta[t]);
                    const float gg[4] = {g4.x, g4.y, g4.z, g4.w}, bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const unsigned short u = *reinterpret_cast<const unsigned short *>(vt + sw128_offset(t + e, vp) + vo);
                        res[i + e] = fmaf(-gg[e], res[i + e], __uint_as_float((uint32_t)u << 16));
                        v[i + e] = bb[e] * res[i + e];
                    }
                }
                put_terms(tl + kTX + 32 * wg, tl + kTX + 32 * wg + 16, v);
                tmem_wait_st();
            }
            fence_before_sync();
            signal(&sm.r_ready);
            // r = R - Y, and w beta r as an operand
            if (!(ok = wait(&sm.y, c))) break;
            fence_after_sync();
            if (active) {
                float y[32];
                tmem_ld32(tl + kTY + 32 * wg, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(&dec.wb[32 * wg + i]);
                    y[i] = w4.x * (res[i] - y[i]);
                    y[i + 1] = w4.y * (res[i + 1] - y[i + 1]);
                    y[i + 2] = w4.z * (res[i + 2] - y[i + 2]);
                    y[i + 3] = w4.w * (res[i + 3] - y[i + 3]);
                }
                put_terms(tl + kTY + 32 * wg, tl + kTY + 32 * wg + 16, y);
                tmem_wait_st();
            }
            fence_before_sync();
            signal(&sm.u_ready);
            // the output over V
            if (active) {
                float o1[32], o2[32];
                tmem_ld32(tl + kTO1 + 32 * wg, o1);
                tmem_ld32(tl + kTO2 + 32 * wg, o2);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int t = 32 * wg + i;
                    const float4 g4 = *reinterpret_cast<const float4 *>(&dec.gs[t]);
                    const float gg[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<bf16 *>(vt + sw128_offset(t + e, vp) + vo) =
                            __float2bfloat16_rn(fmaf(gg[e], o1[i + e], o2[i + e]));
                }
            }
            fence_proxy_async();
            fence_before_sync();
            signal(&sm.o_ready[st]);
            // the state
            const bool last = c + 1 == nch;
            if (!last && !(ok = wait(&sm.prep[st ^ 1], (c + 1) >> 1))) break;
            if (!(ok = wait(&sm.s[st], c >> 1))) break;
            fence_after_sync();
            if (active) {
                const float whole = sm.dec[st ^ 1].whole;
#pragma unroll
                for (int p = 0; p < NT; ++p) {
                    const int col = 32 * (NT * wg + p);
                    float s[32];
                    tmem_ld32(tl + kTS + col, s);
                    tmem_wait_ld();
                    if (!last) {
                        put_state(tl, col, s, whole);
                    } else if (a.state) {
                        float *dst = a.state + row * a.dstate + col;
#pragma unroll
                        for (int i = 0; i < 32; ++i) dst[i] = s[i];
                    }
                }
                if (!last) tmem_wait_st();
            }
            fence_before_sync();
            if (!last) signal(&sm.s_ready);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 512);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int NT>
cudaError_t launch_t(const DeltaArgs &a, cudaStream_t st) {
    CUtensorMap mq, mk, mv, mo;
    const int64_t gn = (int64_t)a.groups * a.dstate, hp = (int64_t)a.heads * a.headdim;
    if (!encode_btw(&mq, a.q, a.batch, a.seqlen, gn, kC) || !encode_btw(&mk, a.k, a.batch, a.seqlen, gn, kC) ||
        !encode_btw(&mv, a.v, a.batch, a.seqlen, hp, kC) || !encode_btw(&mo, a.out, a.batch, a.seqlen, hp, kC))
        return cudaErrorInvalidValue;
    FusedArgs f{};
    f.g = a.g; f.beta = a.beta; f.h0 = a.h0; f.state = a.state; f.scale = a.scale;
    f.seqlen = a.seqlen; f.heads = a.heads; f.rep = a.heads / a.groups; f.headdim = a.headdim; f.dstate = a.dstate;
    f.vtiles = (a.headdim + 127) / 128;
    cudaError_t e = device_status_address(&f.status);
    if (e != cudaSuccess) return e;
    constexpr int bytes = (int)sizeof(FusedSmem<NT>) + 1024;
    e = cudaFuncSetAttribute(delta_fused_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    delta_fused_kernel<NT><<<(unsigned)(a.batch * a.heads * f.vtiles), kThreadsF, bytes, st>>>(mq, mk, mv, mo, f);
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

bool delta_fused_eligible(const DeltaArgs &a) {
    using namespace delta;
    return (a.dstate == 64 || a.dstate == 128) && a.headdim % 64 == 0 && a.seqlen < (int64_t)1 << 30 &&
           a.batch < (int64_t)1 << 30 && (int64_t)a.heads * a.headdim < (int64_t)1 << 30 && aligned16(a.q) &&
           aligned16(a.k) && aligned16(a.v) && aligned16(a.out) && encode_tiled_fn() != nullptr;
}

cudaError_t launch_delta_fused(const DeltaArgs &a, cudaStream_t st) {
    return a.dstate == 64 ? delta::launch_t<1>(a, st) : delta::launch_t<2>(a, st);
}

}  // namespace ssm
