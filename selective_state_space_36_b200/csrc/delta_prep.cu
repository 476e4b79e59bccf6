// delta_prep.cu -- what the chunked gated delta rule needs of each chunk before
// any state enters: the triangular matrices M and Pb (see delta_chunk.cuh) as
// two bf16 terms each, and the decays.
//
// One block per (batch row, head, chunk): K K^T and Q K^T (64 x 64, exact bf16
// operands) on the tensor cores, four warps of 16 rows each and only the
// blocks on and below the diagonal; the decays between tokens from sums in
// float64, because a difference of two float32 sums of a strong decay loses
// the digits of the small difference; then one thread per column solves
// M = L - L M downwards in float32, 16 rows at a time: the rows above enter as a
// product with broadcast reads, the 16 x 16 block on the diagonal is unrolled.
#include "delta_chunk.cuh"
#include "kernel_setup.cuh"

namespace ssm {
namespace delta {
namespace {

constexpr int kPrepThreads = 128;
constexpr int kAtLd = kC + 4;  // row stride of the transposed L: 16-byte rows, conflict-free column reads

template <int NP>
struct PrepSmem {
    bf16 k[kC][NP + 8], q[kC][NP + 8];
    float at[kC][kAtLd];  // at[s][t] = L[t][s]
    float xs[kC][kC];     // xs[t][j] = M[t][j]
    double cum[kC];
    float beta[kC];
};

template <int NP, bool VEC>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(DeltaArgs a, DeltaChunkWs ws) {
    extern __shared__ __align__(16) unsigned char raw[];
    PrepSmem<NP> &sm = *reinterpret_cast<PrepSmem<NP> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t nch = (a.seqlen + kC - 1) / kC;
    const int64_t unit = blockIdx.x, bh = unit / nch, ch = unit - bh * nch;
    const int64_t b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int64_t t0 = ch * kC;
    const int live = (int)(a.seqlen - t0 < kC ? a.seqlen - t0 : kC);
    const int64_t qk0 = ((b * a.seqlen + t0) * a.groups + gr) * a.dstate, qk_ld = (int64_t)a.groups * a.dstate;
    load_tile<VEC>(&sm.k[0][0], NP + 8, static_cast<const bf16 *>(a.k) + qk0, qk_ld, kC, NP, live, a.dstate, tid,
                   kPrepThreads);
    load_tile<VEC>(&sm.q[0][0], NP + 8, static_cast<const bf16 *>(a.q) + qk0, qk_ld, kC, NP, live, a.dstate, tid,
                   kPrepThreads);
    cp_async_commit();
    if (warp == 0) {
        const float *g = a.g + (b * a.seqlen + t0) * a.heads + h, *be = a.beta + (b * a.seqlen + t0) * a.heads + h;
        const int t = 2 * lane;
        // below -1e4 a decay is zero in float32 either way; the clamp keeps
        // differences of two such sums finite
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
        sm.beta[t] = t < live ? be[(int64_t)t * a.heads] : 0.f;
        sm.beta[t + 1] = t + 1 < live ? be[(int64_t)(t + 1) * a.heads] : 0.f;
    }
    cp_async_wait<0>();
    __syncthreads();
    if (tid < kC) {
        float *dec = ws.dec + unit * (kDec * kC);
        dec[tid] = expf((float)sm.cum[tid]);
        dec[kC + tid] = expf((float)(sm.cum[kC - 1] - sm.cum[tid]));
        dec[2 * kC + tid] = sm.beta[tid];
    }
    // K K^T and Q K^T, rows 16 warp .. 16 warp + 15, column blocks up to the diagonal
    float ck[kC / 8][4], cq[kC / 8][4];
#pragma unroll
    for (int j = 0; j < kC / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[j][e] = cq[j][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < NP / 16; ++kk) {
        uint32_t ak[4], aq[4];
        ldm4(ak, &sm.k[16 * warp + rows_first_row(lane)][16 * kk + rows_first_col(lane)]);
        ldm4(aq, &sm.q[16 * warp + rows_first_row(lane)][16 * kk + rows_first_col(lane)]);
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj) {
            if (jj > warp) continue;
            uint32_t bk[4];
            ldm4(bk, &sm.k[16 * jj + cols_first_row(lane)][16 * kk + cols_first_col(lane)]);
            mma(ck[2 * jj], ak, bk[0], bk[1]);
            mma(ck[2 * jj + 1], ak, bk[2], bk[3]);
            mma(cq[2 * jj], aq, bk[0], bk[1]);
            mma(cq[2 * jj + 1], aq, bk[2], bk[3]);
        }
    }
    bf16 *mats = ws.mats + unit * (kMats * kC * kC);
#pragma unroll
    for (int j = 0; j < kC / 8; ++j) {
        if (j > 2 * warp + 1) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 16 * warp + (lane >> 2) + 8 * half, s = 8 * j + 2 * (lane & 3);
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float gam = s + e <= t ? expf((float)(sm.cum[t] - sm.cum[s + e])) * sm.beta[s + e] : 0.f;
                p[e] = s + e <= t ? a.scale * gam * cq[j][2 * half + e] : 0.f;
                sm.at[s + e][t] = s + e < t ? gam * ck[j][2 * half + e] : 0.f;
            }
            uint32_t hi, lo;
            split(p[0], p[1], hi, lo);
            *reinterpret_cast<uint32_t *>(mats + kC * kC + t * kC + s) = hi;
            *reinterpret_cast<uint32_t *>(mats + 3 * kC * kC + t * kC + s) = lo;
        }
    }
    __syncthreads();
    if (tid >= kC) return;
    const int j = tid, first = j & 32;  // the warp's first column: rows above it are zero
    for (int blk = 0; blk < kC / 16; ++blk) {
        const int t0b = 16 * blk;
        float acc[16];
        if (t0b < first) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&sm.at[j][t0b + i]);
                acc[i] = t0b + i > j ? x.x : 0.f;
                acc[i + 1] = t0b + i + 1 > j ? x.y : 0.f;
                acc[i + 2] = t0b + i + 2 > j ? x.z : 0.f;
                acc[i + 3] = t0b + i + 3 > j ? x.w : 0.f;
            }
#pragma unroll 2
            for (int s = first; s < t0b; ++s) {
                const float x = sm.xs[s][j];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(&sm.at[s][t0b + i]);
                    acc[i] = fmaf(-m.x, x, acc[i]);
                    acc[i + 1] = fmaf(-m.y, x, acc[i + 1]);
                    acc[i + 2] = fmaf(-m.z, x, acc[i + 2]);
                    acc[i + 3] = fmaf(-m.w, x, acc[i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = acc[i];
                sm.xs[t0b + i][j] = x;
#pragma unroll
                for (int i2 = i + 1; i2 < 16; ++i2) acc[i2] = fmaf(-sm.at[t0b + i][t0b + i2], x, acc[i2]);
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const bf16 hi = __float2bfloat16_rn(acc[i]);
            mats[(t0b + i) * kC + j] = hi;
            mats[2 * kC * kC + (t0b + i) * kC + j] = __float2bfloat16_rn(acc[i] - __bfloat162float(hi));
        }
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int NP, bool VEC>
cudaError_t launch_t(const DeltaArgs &a, const DeltaChunkWs &ws, cudaStream_t st) {
    const int64_t units = a.batch * a.heads * ((a.seqlen + kC - 1) / kC);
    const size_t bytes = sizeof(PrepSmem<NP>);
    cudaError_t e = allow_smem<delta_prep_kernel<NP, VEC>, (int)sizeof(PrepSmem<NP>)>();
    if (e != cudaSuccess) return e;
    delta_prep_kernel<NP, VEC><<<(unsigned)units, kPrepThreads, bytes, st>>>(a, ws);
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

cudaError_t launch_delta_prep(const DeltaArgs &a, const DeltaChunkWs &ws, cudaStream_t st) {
    using namespace delta;
    const bool vec = a.dstate % 8 == 0 && aligned16(a.q) && aligned16(a.k);
    if (a.dstate <= 64) return vec ? launch_t<64, true>(a, ws, st) : launch_t<64, false>(a, ws, st);
    return vec ? launch_t<128, true>(a, ws, st) : launch_t<128, false>(a, ws, st);
}

}  // namespace ssm
