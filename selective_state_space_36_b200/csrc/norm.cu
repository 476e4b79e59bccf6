// norm.cu -- layer and RMS normalisation of rows with weight, bias and a
// silu(z) gate, and its gradient.
//
// Forward, one pass over HBM: the threads of a row keep it in registers, take
// the mean, then the mean of the squared deviations from it (no difference of
// large squares), then write.  Backward, with dy = dout silu(z) and
// dxhat = dy weight:
//   dx = rstd (dxhat - mean(dxhat) - xhat mean(dxhat xhat))   (RMS: no mean(dxhat))
//   dz = dout (xhat weight + bias) silu'(z)
//   dweight = sum_rows dy xhat,  dbias = sum_rows dy.
// Both are bound by HBM: x, z (and dout) read once, out (dx, dz) written once.
//
// The column sums: a thread always holds the same columns, so a block that
// walks over its rows adds dy xhat and dy in registers and writes one partial
// row at its end; a second kernel adds the partial rows in a fixed order.  No
// atomics: the same inputs give the same bits.
//
// TPR threads share a row, each holding NV vectors of VEC values (16 bytes
// where dim and the pointers allow, else single values).  Rows too long for
// the registers are walked twice (forward, dx), and their column sums come
// from a kernel of their own over tiles of columns.
#include "norm.cuh"
#include "ssm_device.cuh"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerBlock = kThreads / 32;

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *v) {
    if constexpr (VEC == 1) {
        v[0] = io_traits<T>::load(p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4) *p = v[0];
        else *p = __float2bfloat16_rn(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int VEC>
__device__ __forceinline__ void load_param(const float *p, float *v, float none) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = none;
    if (!p) return;
    if constexpr (VEC == 1) {
        v[0] = __ldg(p);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = __ldg(p + e);
    }
}

// sigmoid(z): fp32 I/O with the full-precision exponential, bf16 I/O with the
// SFU's (a few fp32 ulps, far below the output's rounding)
template <bool PRECISE>
__device__ __forceinline__ float sigmoid(float z) {
    if (PRECISE) return 1.f / (1.f + expf(-z));
    return 1.f / (1.f + __expf(-z));
}

// Sum over the TPR threads of a row, in every one of them.  `red`: two floats
// per warp of scratch for rows wider than a warp; `flip` alternates between
// two buffers, so that one barrier per sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*red)[kWarpsPerBlock][2], int &flip) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[flip][warp][i] = x[i];
        __syncthreads();
        const int first = warp / W * W;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) x[i] += red[flip][first + w][i];
        }
        flip ^= 1;
    }
}

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(NormArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ float red[2][kWarpsPerBlock][2];
    int flip = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + row * a.dim;
    const T *z = a.z ? static_cast<const T *>(a.z) + row * a.dim : nullptr;
    const float inv = 1.f / a.dim;
    float v[NV][VEC], zv[NV][VEC];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * TPR) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = zv[i][e] = 0.f;
        if (live && c < a.dim) {
            load_vec<T, VEC>(x + c, v[i]);
            if (z) load_vec<T, VEC>(z + c, zv[i]);
        }
    }
    float mean = 0.f;
    if (a.center) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[0] += v[i][e];
        row_sum<TPR>(sum, red, flip);
        mean = sum[0] * inv;
        sum[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((lane + i * TPR) * VEC < a.dim)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] -= mean;
                sum[0] = fmaf(v[i][e], v[i][e], sum[0]);
            }
    row_sum<TPR>(sum, red, flip);
    const float rstd = 1.f / sqrtf(sum[0] * inv + a.eps);
    if (!live) return;
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T *out = static_cast<T *>(a.out) + row * a.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * TPR) * VEC;
        if (c >= a.dim) continue;
        float w[VEC], bias[VEC];
        load_param<VEC>(a.weight ? a.weight + c : nullptr, w, 1.f);
        load_param<VEC>(a.bias ? a.bias + c : nullptr, bias, 0.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float y = fmaf(v[i][e] * rstd, w[e], bias[e]);
            if (z) y *= zv[i][e] * sigmoid<PRECISE>(zv[i][e]);
            v[i][e] = y;
        }
        store_vec<T, VEC>(out + c, v[i]);
    }
}

// Rows of any length: one block per row, the row read three times (its second
// and third reading come from the L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_long_kernel(NormArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ float red[2][kWarpsPerBlock][2];
    int flip = 0;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.dim;
    const T *z = a.z ? static_cast<const T *>(a.z) + row * a.dim : nullptr;
    float mean = 0.f, sum[1] = {0.f};
    if (a.center) {
        for (int c = threadIdx.x; c < a.dim; c += kThreads) sum[0] += io_traits<T>::load(x + c);
        row_sum<kThreads>(sum, red, flip);
        mean = sum[0] / a.dim;
        sum[0] = 0.f;
    }
    for (int c = threadIdx.x; c < a.dim; c += kThreads) {
        const float d = io_traits<T>::load(x + c) - mean;
        sum[0] = fmaf(d, d, sum[0]);
    }
    row_sum<kThreads>(sum, red, flip);
    const float rstd = 1.f / sqrtf(sum[0] / a.dim + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T *out = static_cast<T *>(a.out) + row * a.dim;
    for (int c = threadIdx.x; c < a.dim; c += kThreads) {
        float y = fmaf((io_traits<T>::load(x + c) - mean) * rstd, a.weight ? __ldg(a.weight + c) : 1.f,
                       a.bias ? __ldg(a.bias + c) : 0.f);
        if (z) {
            const float zc = io_traits<T>::load(z + c);
            y *= zc * sigmoid<PRECISE>(zc);
        }
        store_vec<T, 1>(out + c, &y);
    }
}

// One element's dy and dz.
template <bool PRECISE>
__device__ __forceinline__ void gate_grad(float dout, float y, float z, float &dy, float &dz) {
    const float s = sigmoid<PRECISE>(z);
    dy = dout * z * s;
    dz = dout * y * s * fmaf(z, 1.f - s, 1.f);
}

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(NormArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    constexpr int RPB = kThreads / TPR;  // rows per block and step
    __shared__ float red[2][kWarpsPerBlock][2];
    int flip = 0;
    const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const float inv = 1.f / a.dim;
    float w[NV][VEC], bias[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * TPR) * VEC;
        const bool in = c < a.dim;
        load_param<VEC>(in && a.weight ? a.weight + c : nullptr, w[i], in ? 1.f : 0.f);
        load_param<VEC>(in && a.bias ? a.bias + c : nullptr, bias[i], 0.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += (int64_t)gridDim.x * RPB) {
        const int64_t row = base + slot;
        const bool live = row < a.rows;
        const int64_t at = row * a.dim;
        const float mean = live && a.mean_in ? __ldg(a.mean_in + row) : 0.f;
        const float rstd = live ? __ldg(a.rstd_in + row) : 0.f;
        float xh[NV][VEC], dy[NV][VEC], zv[NV][VEC], sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * TPR) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) xh[i][e] = dy[i][e] = zv[i][e] = 0.f;
            if (live && c < a.dim) {
                load_vec<T, VEC>(static_cast<const T *>(a.x) + at + c, xh[i]);
                load_vec<T, VEC>(static_cast<const T *>(a.dout) + at + c, dy[i]);
                if (a.z) load_vec<T, VEC>(static_cast<const T *>(a.z) + at + c, zv[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * TPR) * VEC;
            if (!live || c >= a.dim) continue;
            float dz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[i][e] = (xh[i][e] - mean) * rstd;
                if (a.z) {
                    float d;
                    gate_grad<PRECISE>(dy[i][e], fmaf(xh[i][e], w[i][e], bias[i][e]), zv[i][e], d, dz[e]);
                    dy[i][e] = d;
                }
                dw[i][e] = fmaf(dy[i][e], xh[i][e], dw[i][e]);
                db[i][e] += dy[i][e];
                dy[i][e] *= w[i][e];
                sums[0] += dy[i][e];
                sums[1] = fmaf(dy[i][e], xh[i][e], sums[1]);
            }
            if (a.z) store_vec<T, VEC>(static_cast<T *>(a.dz) + at + c, dz);
        }
        row_sum<TPR>(sums, red, flip);
        const float m1 = a.center ? sums[0] * inv : 0.f, m2 = sums[1] * inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * TPR) * VEC;
            if (c >= a.dim) continue;
            float dx[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) dx[e] = (dy[i][e] - m1 - xh[i][e] * m2) * rstd;
            store_vec<T, VEC>(static_cast<T *>(a.dx) + at + c, dx);
        }
    }
    if (!a.partial) return;
    // the block's rows of one column set, then one partial row
    __shared__ float part[RPB > 1 ? kThreads * VEC : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (which ? !a.dbias : !a.dweight) continue;
            float(&s)[VEC] = which ? db[i] : dw[i];
            const int c = (lane + i * TPR) * VEC;
            if constexpr (RPB > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < VEC; ++e) part[e * kThreads + threadIdx.x] = s[e];
                __syncthreads();
                if (slot == 0)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        for (int o = 1; o < RPB; ++o) s[e] += part[e * kThreads + o * TPR + lane];
            }
            if (slot == 0 && c < a.dim)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    a.partial[((int64_t)which * gridDim.x + blockIdx.x) * a.dim + c + e] = s[e];
        }
}

// dx and dz of rows of any length, one block per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_long_kernel(NormArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ float red[2][kWarpsPerBlock][2];
    int flip = 0;
    const int64_t row = blockIdx.x, at = row * a.dim;
    const float mean = a.mean_in ? __ldg(a.mean_in + row) : 0.f, rstd = __ldg(a.rstd_in + row);
    const T *x = static_cast<const T *>(a.x) + at, *dout = static_cast<const T *>(a.dout) + at;
    const T *z = a.z ? static_cast<const T *>(a.z) + at : nullptr;
    float sums[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.dim; c += kThreads) {
        const float xh = (io_traits<T>::load(x + c) - mean) * rstd, w = a.weight ? __ldg(a.weight + c) : 1.f;
        float dy = io_traits<T>::load(dout + c);
        if (z) {
            float d, dz;
            gate_grad<PRECISE>(dy, fmaf(xh, w, a.bias ? __ldg(a.bias + c) : 0.f), io_traits<T>::load(z + c), d, dz);
            dy = d;
            store_vec<T, 1>(static_cast<T *>(a.dz) + at + c, &dz);
        }
        sums[0] = fmaf(dy, w, sums[0]);
        sums[1] = fmaf(dy * w, xh, sums[1]);
    }
    row_sum<kThreads>(sums, red, flip);
    const float m1 = a.center ? sums[0] / a.dim : 0.f, m2 = sums[1] / a.dim;
    for (int c = threadIdx.x; c < a.dim; c += kThreads) {
        const float xh = (io_traits<T>::load(x + c) - mean) * rstd, w = a.weight ? __ldg(a.weight + c) : 1.f;
        float dy = io_traits<T>::load(dout + c);
        if (z) {
            const float zc = io_traits<T>::load(z + c);
            dy *= zc * sigmoid<PRECISE>(zc);
        }
        const float dx = (dy * w - m1 - xh * m2) * rstd;
        store_vec<T, 1>(static_cast<T *>(a.dx) + at + c, &dx);
    }
}

// Partial column sums for rows of any length: block (x: 256 columns, y: every
// gridDim.y-th row).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_columns_kernel(NormArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const int64_t at = row * a.dim + c;
        const float mean = a.mean_in ? __ldg(a.mean_in + row) : 0.f;
        const float xh = (io_traits<T>::load(static_cast<const T *>(a.x) + at) - mean) * __ldg(a.rstd_in + row);
        float dy = io_traits<T>::load(static_cast<const T *>(a.dout) + at);
        if (a.z) {
            const float zc = io_traits<T>::load(static_cast<const T *>(a.z) + at);
            dy *= zc * sigmoid<PRECISE>(zc);
        }
        dw = fmaf(dy, xh, dw);
        db += dy;
    }
    if (a.dweight) a.partial[(int64_t)blockIdx.y * a.dim + c] = dw;
    if (a.dbias) a.partial[((int64_t)gridDim.y + blockIdx.y) * a.dim + c] = db;
}

// Adds the partial rows in a fixed order: 32 columns per block, 8 threads per
// column, each over every 8th partial row.
__global__ void __launch_bounds__(kThreads) norm_bwd_reduce_kernel(const float *partial, int parts, int dim,
                                                                  float *dweight, float *dbias) {
    __shared__ float s[kWarpsPerBlock][32];
    float *dst = blockIdx.y ? dbias : dweight;
    if (!dst) return;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float sum = 0.f;
    if (col < dim)
        for (int p = part; p < parts; p += kWarpsPerBlock)
            sum += partial[((int64_t)blockIdx.y * parts + p) * dim + col];
    s[part][threadIdx.x & 31] = sum;
    __syncthreads();
    if (part == 0 && col < dim) {
#pragma unroll
        for (int p = 1; p < kWarpsPerBlock; ++p) sum += s[p][threadIdx.x & 31];
        dst[col] = sum;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Threads per row and vectors per thread for `pieces` vectors in a row; false:
// the row does not fit the registers.
struct Shape { int tpr, nv; };
bool shape_of(int64_t pieces, Shape *s) {
    static constexpr Shape shapes[] = {{8, 1}, {16, 1}, {32, 1}, {32, 2}, {32, 4}, {256, 1}, {256, 2}, {256, 4}};
    for (const Shape &x : shapes)
        if (pieces <= (int64_t)x.tpr * x.nv) {
            *s = x;
            return true;
        }
    return false;
}

template <typename T>
bool vectors(const NormArgs &a) {
    return a.dim % (16 / sizeof(T)) == 0 && aligned16(a.x) && aligned16(a.z) && aligned16(a.dout) &&
           aligned16(a.out) && aligned16(a.dx) && aligned16(a.dz);
}

template <typename T, int VEC, typename F>
cudaError_t with_shape(Shape s, F f) {
    if (s.tpr == 8) return f.template run<T, VEC, 8, 1>();
    if (s.tpr == 16) return f.template run<T, VEC, 16, 1>();
    if (s.tpr == 32) {
        if (s.nv == 1) return f.template run<T, VEC, 32, 1>();
        if (s.nv == 2) return f.template run<T, VEC, 32, 2>();
        return f.template run<T, VEC, 32, 4>();
    }
    if (s.nv == 1) return f.template run<T, VEC, 256, 1>();
    if (s.nv == 2) return f.template run<T, VEC, 256, 2>();
    return f.template run<T, VEC, 256, 4>();
}

struct Fwd {
    const NormArgs &a;
    cudaStream_t st;
    template <typename T, int VEC, int TPR, int NV>
    cudaError_t run() const {
        constexpr int RPB = kThreads / TPR;
        norm_fwd_kernel<T, VEC, TPR, NV><<<(unsigned)((a.rows + RPB - 1) / RPB), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
};

// Blocks of the backward pass: each leaves one partial row of column sums.
constexpr int kBwdBlocksPerSm = 4;
int64_t bwd_blocks(int64_t rows, int rows_per_block, int sms) {
    const int64_t all = (rows + rows_per_block - 1) / rows_per_block, most = (int64_t)kBwdBlocksPerSm * sms;
    return all < most ? all : most;
}

struct Bwd {
    const NormArgs &a;
    int64_t blocks;
    cudaStream_t st;
    template <typename T, int VEC, int TPR, int NV>
    cudaError_t run() const {
        norm_bwd_kernel<T, VEC, TPR, NV><<<(unsigned)blocks, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
};

template <typename T>
struct BwdPlan {
    bool vec, fits;
    Shape s;
    int64_t parts;
    BwdPlan(const NormArgs &a, int sms) {
        vec = vectors<T>(a);
        fits = shape_of(vec ? a.dim / (16 / sizeof(T)) : a.dim, &s);
        if (fits) {
            parts = bwd_blocks(a.rows, kThreads / s.tpr, sms);
        } else {
            const int64_t tiles = (a.dim + kThreads - 1) / kThreads;
            const int64_t most = (8 * (int64_t)sms + tiles - 1) / tiles;
            parts = a.rows < most ? a.rows : most;
        }
    }
};

template <typename T>
cudaError_t fwd_t(const NormArgs &a, cudaStream_t st) {
    const bool vec = vectors<T>(a);
    Shape s;
    if (shape_of(vec ? a.dim / (16 / sizeof(T)) : a.dim, &s))
        return vec ? with_shape<T, 16 / sizeof(T)>(s, Fwd{a, st}) : with_shape<T, 1>(s, Fwd{a, st});
    norm_fwd_long_kernel<T><<<(unsigned)a.rows, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const NormArgs &a, int sms, cudaStream_t st) {
    const BwdPlan<T> p(a, sms);
    cudaError_t e;
    if (p.fits) {
        const Bwd f{a, p.parts, st};
        e = p.vec ? with_shape<T, 16 / sizeof(T)>(p.s, f) : with_shape<T, 1>(p.s, f);
    } else {
        norm_bwd_long_kernel<T><<<(unsigned)a.rows, kThreads, 0, st>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess && a.partial) {
            const dim3 grid((unsigned)((a.dim + kThreads - 1) / kThreads), (unsigned)p.parts);
            norm_bwd_columns_kernel<T><<<grid, kThreads, 0, st>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e != cudaSuccess || !a.partial) return e;
    const dim3 grid((unsigned)((a.dim + 31) / 32), 2);
    norm_bwd_reduce_kernel<<<grid, kThreads, 0, st>>>(a.partial, (int)p.parts, a.dim, a.dweight, a.dbias);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int sms, cudaStream_t st) {
    return bf16 ? bwd_t<__nv_bfloat16>(a, sms, st) : bwd_t<float>(a, sms, st);
}

size_t norm_bwd_partial_bytes(const NormArgs &a, bool bf16, int sms) {
    const int64_t parts = bf16 ? BwdPlan<__nv_bfloat16>(a, sms).parts : BwdPlan<float>(a, sms).parts;
    return (size_t)2 * parts * a.dim * sizeof(float);
}

}  // namespace ssm
