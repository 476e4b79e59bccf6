// delta_chunk.cuh -- device helpers shared by the chunked kernels of the gated
// delta rule: the chunk workspace, warp-level bf16 matrix products with
// operands split into two bf16 terms, and the loads of a chunk's tiles.
//
// Chunks of C = 64 tokens.  With G_t the sum of the log decays of the chunk's
// tokens up to t and Gam_ts = exp(G_t - G_s) for s <= t, the definition's
// recurrence inside a chunk that starts from the state S0 is
//   r = (I - M) (V - diag(exp G) K S0^T)
//   O = scale diag(exp G) Q S0^T + Pb r,    Pb = scale lower(Gam o Q K^T) diag(beta)
//   S1 = exp(G_C) S0 + (beta r)^T diag(exp(G_C - G)) K
// where I - M is the inverse of I + L, L = strict_lower(Gam o K K^T) diag(beta).
// Nothing is divided by beta, which may be zero.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cp_async.cuh"
#include "delta_rule.cuh"

namespace ssm {
namespace delta {

constexpr int kC = 64;        // tokens per chunk
constexpr int kMatLd = 72;    // row stride of a 64 x 64 bf16 tile in shared memory (conflict-free ldmatrix)
constexpr int kMats = 4;      // per chunk and head: M, Pb (high terms), M, Pb (low terms), each 64 x 64
constexpr int kDec = 3;       // per chunk and head: exp(G_t), exp(G_C - G_t), beta_t (zero behind the end)

typedef __nv_bfloat16 bf16;

// ------------------------------------------------------ matrix instructions
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], const bf16 *p) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], const bf16 *p) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void stm4t(bf16 *p, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n"
                 ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
__device__ __forceinline__ void stm4(bf16 *p, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n"
                 ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
// an 8 x 8 block of 16-bit values, transposed within the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// c (16 x 8) += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float low_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// x, y as two bf16 terms each: x = hi + lo up to 2^-17 of |x| (the low term is
// the bf16 rounding of the remainder, which float32 holds exactly).  Products
// of two such operands drop low x low, 2^-16 of the product at most: the
// accuracy of a state or gradient sum stays near float32's while the matrix
// instructions run on bf16.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack(x, y);
    lo = pack(x - low_of(hi), y - high_of(hi));
}

// Row and column this lane addresses in a 16 x 16 block of ldmatrix.x4:
// "rows first" gives registers (rows 0-7, 8-15) x (columns 0-7) then columns
// 8-15; "columns first" the columns of rows 0-7, then those of rows 8-15.
__device__ __forceinline__ int rows_first_row(int lane) { return (lane & 7) + ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int rows_first_col(int lane) { return (lane >> 4) * 8; }
__device__ __forceinline__ int cols_first_row(int lane) { return (lane & 7) + (lane >> 4) * 8; }
__device__ __forceinline__ int cols_first_col(int lane) { return ((lane >> 3) & 1) * 8; }

// ------------------------------------------------------------- tile loads
// rows x cols of a row-major global matrix (row stride gld elements) into
// shared memory (row stride sld), zeros outside [0, have_rows) x [0, have_cols).
// VEC: rows start 16-byte aligned and have_cols is a multiple of 8 (an
// asynchronous copy of 16 bytes at a time); otherwise element by element.
template <bool VEC>
__device__ __forceinline__ void load_tile(bf16 *s, int sld, const bf16 *g, int64_t gld, int rows, int cols,
                                          int have_rows, int have_cols, int tid, int nthreads) {
    if (VEC) {
        const int per = cols / 8;
        for (int i = tid; i < rows * per; i += nthreads) {
            const int r = i / per, c = (i - r * per) * 8;
            const bool in = r < have_rows && c < have_cols;
            cp_async16(s + r * sld + c, in ? g + r * gld + c : g, in);
        }
    } else {
        for (int i = tid; i < rows * cols; i += nthreads) {
            const int r = i / cols, c = i - r * cols;
            s[r * sld + c] = r < have_rows && c < have_cols ? g[r * gld + c] : __float2bfloat16_rn(0.f);
        }
    }
}

// A stored state: two bf16 terms, each as (NP / 8, pp, 8) -- the eight columns of
// a group row after row, so that neither a thread per row nor a quad per row
// spreads a store over more lines than its bytes fill (row-major, the forward's
// recomputation spent two thirds of its time in these stores).
template <int NP>
__device__ __forceinline__ int64_t state_at(int pp, int term, int row, int col) {
    return ((int64_t)(term * (NP / 8) + (col >> 3)) * pp + row) * 8 + (col & 7);
}

// A warp's 16 x NP slice of a state (accumulators: rows row0 + lane / 4 (+ 8),
// columns 8 j + 2 (lane % 4) (+ 1)).
template <int NP>
__device__ __forceinline__ void store_state(bf16 *dst, int pp, const float (&s)[NP / 8][4], int row0, int lane) {
    if (row0 >= pp) return;
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t hi, lo;
            split(s[j][2 * half], s[j][2 * half + 1], hi, lo);
            const int row = row0 + (lane >> 2) + 8 * half, col = 8 * j + 2 * (lane & 3);
            *reinterpret_cast<uint32_t *>(dst + state_at<NP>(pp, 0, row, col)) = hi;
            *reinterpret_cast<uint32_t *>(dst + state_at<NP>(pp, 1, row, col)) = lo;
        }
}

// A warp's 16 columns of a (64, pp) matrix held transposed in accumulators
// (x[j]: columns col0 + lane / 4 (+ 8), rows 8 j + 2 (lane % 4) (+ 1)) as two
// bf16 terms: high (64, pp), then low.  `stage`: this warp's 16 columns of a
// shared tile of 64 rows.
__device__ __forceinline__ void store_rows(bf16 *dst, int pp, const float (&x)[kC / 8][4], bf16 *stage, int ld,
                                           int col0, int lane) {
    if (col0 >= pp) return;
    __syncwarp();
#pragma unroll
    for (int term = 0; term < 2; ++term) {
#pragma unroll
        for (int jj = 0; jj < kC / 16; ++jj) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi, lo;
                split(x[2 * jj + (i >> 1)][2 * (i & 1)], x[2 * jj + (i >> 1)][2 * (i & 1) + 1], hi, lo);
                f[i] = term ? lo : hi;
            }
            stm4t(stage + (16 * jj + cols_first_row(lane)) * ld + cols_first_col(lane), f[0], f[1], f[2], f[3]);
        }
        __syncwarp();
#pragma unroll
        for (int it = 0; it < kC / 16; ++it) {
            const int t = 16 * it + (lane >> 1), c = 8 * (lane & 1);
            *reinterpret_cast<uint4 *>(dst + (int64_t)(term * kC + t) * pp + col0 + c) =
                *reinterpret_cast<const uint4 *>(stage + t * ld + c);
        }
        __syncwarp();
    }
}

}  // namespace delta

// Workspace of the chunked kernels; sizes in elements.
struct DeltaChunkWs {
    __nv_bfloat16 *mats;  // (batch, heads, chunks, kMats, 64, 64)
    float *dec;           // (batch, heads, chunks, kDec, 64)
    // backward only; headdim rounded up to 16 (pp), dstate to 64 or 128 (np)
    __nv_bfloat16 *s0;    // (batch, heads, chunks, 2, np / 8, pp, 8): the state entering each chunk
    __nv_bfloat16 *ds1;   // the same: the gradient of the state leaving it
    __nv_bfloat16 *r, *dv; // (batch, heads, chunks, 2, 64, pp): r, the gradient of V
};

// The forward on the tcgen05 tensor cores: dstate 64 or
// 128, headdim a multiple of 64, 16-byte aligned tensors.
// With few heads the sequence is split into segments that run side by side
// (delta_fused_segments > 1: needs workspace).
bool delta_fused_eligible(const DeltaArgs &a);
int delta_fused_segments(const DeltaArgs &a, int sms);
int64_t delta_fused_workspace(const DeltaArgs &a, int nseg);  // bytes
cudaError_t launch_delta_fused(const DeltaArgs &a, int nseg, float *ws, cudaStream_t st);
// The gradient's first half on the same kernel (out is not read): everything of
// the workspace but ds1 and dv.
cudaError_t launch_delta_fused_store(const DeltaArgs &a, const DeltaChunkWs &ws, cudaStream_t st);

// The pass backwards in time on tcgen05: what delta_fused_eligible asks, headdim <=
// 128, dout and dv aligned too.
bool delta_fused_reverse_eligible(const DeltaBwdArgs &a);
cudaError_t launch_delta_fused_reverse(const DeltaBwdArgs &a, const DeltaChunkWs &ws, cudaStream_t st);
// dq, dk, dg and dbeta on tcgen05: that, and dq and dk aligned.
bool delta_fused_grad_eligible(const DeltaBwdArgs &a);
cudaError_t launch_delta_fused_grad(const DeltaBwdArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st);

cudaError_t launch_delta_prep(const DeltaArgs &a, const DeltaChunkWs &ws, cudaStream_t st);
cudaError_t launch_delta_chain(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st);
cudaError_t launch_delta_chain_store(const DeltaArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st);
cudaError_t launch_delta_reverse(const DeltaBwdArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st);
cudaError_t launch_delta_grad(const DeltaBwdArgs &a, const DeltaChunkWs &ws, int sms, cudaStream_t st);

}  // namespace ssm
