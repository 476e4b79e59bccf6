// delta_recurrent.cu -- the gated delta rule token by token (the decode step
// is one token), in fp32 for both element types.
//
// Eight lanes share one row of the state S (headdim x dstate): a row's
// dstate values are dealt out in pieces of four, piece i to lane i mod 8, so
// that the eight lanes read and write 128 contiguous bytes at a time.  A
// warp holds 4 rows at once and kRows sets of them, all in registers for the
// whole sequence; rows are independent, so no block-wide synchronisation
// exists.  Per token a row needs two dot products over dstate (S k and S q),
// each reduced over its eight lanes by three shuffles.
//
// One token moves 8 headdim dstate bytes of state per head and computes 8
// flops per state value, so the step is bound by HBM: the loads of all
// kRows sets are issued before the first is used.
#include "delta_rule.cuh"
#include "ssm_device.cuh"

namespace ssm {
namespace {

constexpr int kLanes = 8;             // lanes that share a state row
constexpr int kWarps = 4;             // warps per block
constexpr int kRows = 2;              // row sets per warp

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}

// Four values of a row of n at column c; zeros behind its end.
template <typename T, bool VEC>
__device__ __forceinline__ void row4(const T *row, int c, int n, float *v) {
    if (VEC) {
        if (c < n) io_traits<T>::load4(row + c, v);
        else v[0] = v[1] = v[2] = v[3] = 0.f;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < n ? io_traits<T>::load(row + c + e) : 0.f;
    }
}

template <int PIECES, bool VEC>
__device__ __forceinline__ void put_row(float *dst, const float (&s)[PIECES][4], int sub, int n) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int c = 4 * (sub + kLanes * p);
        if (VEC) {
            if (c < n) *reinterpret_cast<float4 *>(dst + c) = make_float4(s[p][0], s[p][1], s[p][2], s[p][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < n) dst[c + e] = s[p][e];
        }
    }
}

// PIECES pieces of four values per lane: dstate <= 32 PIECES.  VEC: dstate is
// a multiple of 4 and q, k, the states are aligned to four elements.  STORE:
// the backward pass's first half (DeltaArgs::marks, r; no output).
template <typename T, int PIECES, bool VEC, bool STORE>
__global__ void __launch_bounds__(kWarps * 32) delta_recurrent_kernel(DeltaArgs a) {
    const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
    constexpr int kRowsPerWarp = 4 * kRows;
    const int tiles = (a.headdim + kWarps * kRowsPerWarp - 1) / (kWarps * kRowsPerWarp);
    const int64_t bh = blockIdx.x / tiles;
    const int tile = (int)(blockIdx.x % tiles);
    const int64_t b = bh / a.heads;
    const int h = (int)(bh % a.heads), gr = h / (a.heads / a.groups);
    const int row0 = (tile * kWarps + (threadIdx.x >> 5)) * kRowsPerWarp + (lane >> 3);
    const int n = a.dstate;
    const T *q = static_cast<const T *>(a.q) + ((b * a.seqlen) * a.groups + gr) * n;
    const T *k = static_cast<const T *>(a.k) + ((b * a.seqlen) * a.groups + gr) * n;
    const T *v = static_cast<const T *>(a.v) + ((b * a.seqlen) * a.heads + h) * a.headdim;
    T *out = STORE ? nullptr : static_cast<T *>(a.out) + ((b * a.seqlen) * a.heads + h) * a.headdim;
    const float *g = a.g + (b * a.seqlen) * a.heads + h, *beta = a.beta + (b * a.seqlen) * a.heads + h;

    float s[kRows][PIECES][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = row0 + 4 * r;
        const float *src = a.h0 ? a.h0 + (bh * a.headdim + row) * (int64_t)n : nullptr;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int c = 4 * (sub + kLanes * p);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r][p][e] = 0.f;
            if (!src || row >= a.headdim) continue;
            // plain loads: the state may be written back to the same place
            if (VEC) {
                if (c < n) {
                    const float4 x = *reinterpret_cast<const float4 *>(src + c);
                    s[r][p][0] = x.x; s[r][p][1] = x.y; s[r][p][2] = x.z; s[r][p][3] = x.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < n) s[r][p][e] = src[c + e];
            }
        }
    }
    for (int64_t t = 0; t < a.seqlen; ++t) {
        if (STORE && t % kDeltaStep == 0) {
            const int64_t every = (a.seqlen + kDeltaStep - 1) / kDeltaStep;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int row = row0 + 4 * r;
                if (row < a.headdim)
                    put_row<PIECES, VEC>(a.marks + ((bh * every + t / kDeltaStep) * a.headdim + row) * n, s[r], sub, n);
            }
        }
        float kk[PIECES][4], qq[PIECES][4];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int c = 4 * (sub + kLanes * p);
            row4<T, VEC>(k, c, n, kk[p]);
            row4<T, VEC>(q, c, n, qq[p]);
        }
        const float decay = expf(__ldg(g)), bt = __ldg(beta);
        float vv[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int row = row0 + 4 * r;
            vv[r] = row < a.headdim ? io_traits<T>::load(v + row) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float dot = 0.f;
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][p][e] *= decay;
                    dot = fmaf(s[r][p][e], kk[p][e], dot);
                }
            const float res = vv[r] - sum8(dot), u = bt * res;
            if (STORE && sub == 0 && row0 + 4 * r < a.headdim)
                a.r[((b * a.seqlen + t) * a.heads + h) * a.headdim + row0 + 4 * r] = res;
            float o = 0.f;
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][p][e] = fmaf(u, kk[p][e], s[r][p][e]);
                    o = fmaf(s[r][p][e], qq[p][e], o);
                }
            o = sum8(o);
            const int row = row0 + 4 * r;
            if (!STORE && sub == 0 && row < a.headdim) io_traits<T>::store(out + row, a.scale * o);
        }
        q += (int64_t)a.groups * n;
        k += (int64_t)a.groups * n;
        v += (int64_t)a.heads * a.headdim;
        if (!STORE) out += (int64_t)a.heads * a.headdim;
        g += a.heads;
        beta += a.heads;
    }
    if (!a.state) return;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = row0 + 4 * r;
        if (row >= a.headdim) continue;
        put_row<PIECES, VEC>(a.state + (bh * a.headdim + row) * (int64_t)n, s[r], sub, n);
    }
}

bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T, bool STORE>
cudaError_t launch_t(const DeltaArgs &a, cudaStream_t st) {
    const int tiles = (a.headdim + kWarps * 4 * kRows - 1) / (kWarps * 4 * kRows);
    const int64_t blocks = a.batch * a.heads * tiles;
    const bool vec = a.dstate % 4 == 0 && aligned_to(a.q, 4 * sizeof(T)) && aligned_to(a.k, 4 * sizeof(T)) &&
                     aligned_to(a.h0, 16) && aligned_to(a.state, 16);
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    if (a.dstate <= 32) {
        if (vec) delta_recurrent_kernel<T, 1, true, STORE><<<grid, block, 0, st>>>(a);
        else delta_recurrent_kernel<T, 1, false, STORE><<<grid, block, 0, st>>>(a);
    } else if (a.dstate <= 64) {
        if (vec) delta_recurrent_kernel<T, 2, true, STORE><<<grid, block, 0, st>>>(a);
        else delta_recurrent_kernel<T, 2, false, STORE><<<grid, block, 0, st>>>(a);
    } else {
        if (vec) delta_recurrent_kernel<T, 4, true, STORE><<<grid, block, 0, st>>>(a);
        else delta_recurrent_kernel<T, 4, false, STORE><<<grid, block, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool bf16, cudaStream_t st) {
    if (a.marks) return bf16 ? launch_t<__nv_bfloat16, true>(a, st) : launch_t<float, true>(a, st);
    return bf16 ? launch_t<__nv_bfloat16, false>(a, st) : launch_t<float, false>(a, st);
}

}  // namespace ssm
