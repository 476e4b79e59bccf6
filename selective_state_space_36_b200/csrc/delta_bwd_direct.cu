// delta_bwd_direct.cu -- the gated delta rule's gradient in float32 throughout,
// for float32 tensors (the formulas of delta_fused_bwd.cu on chunks of kDeltaStep
// tokens, with a state per chunk from launch_delta_recurrent).
//
// One block per (batch row, head) walks backwards over the chunks; dS and S0
// live in shared memory, everything of a chunk is a small dense product that
// the block's threads divide by output element.  The equations couple all of
// headdim (in dq, dk, dg, dbeta) and all of dstate (in e), so a head is not
// divided over blocks.  e solves e = dU - Abar^T (beta e) by substitution from
// the last token, one thread per column of V.
//
// Measured: 3 sequences of 600 tokens, 16 heads of 100 x 80: 2050 us, 54 us per 16
// tokens; bound by the latency of the products' shared-memory loops (48 blocks).
#include "delta_rule.cuh"
#include "kernel_setup.cuh"
#include "ssm_device.cuh"

namespace ssm {
namespace {

constexpr int kT = kDeltaStep, kThreadsD = 256;

struct Layout {  // float offsets in shared memory
    int ldn, ldp, ds, s0, q, k, o, r, e, l, kk, pm, x, em, cum, total;
    __host__ __device__ constexpr Layout(int P, int N) : ldn(N | 1), ldp(P | 1), ds(0), s0(0), q(0), k(0), o(0), r(0), e(0), l(0), kk(0), pm(0), x(0), em(0), cum(0), total(0) {
        // odd strides: a column read by a warp falls into different banks
        int at = 0;
        cum = at; at += 2 * (kT + 2);  // doubles first
        ds = at; at += P * ldn;
        s0 = at; at += P * ldn;
        q = at; at += kT * ldn;
        k = at; at += kT * ldn;
        l = at; at += kT * ldn;
        o = at; at += kT * ldp;
        r = at; at += kT * ldp;
        e = at; at += kT * ldp;
        kk = at; at += kT * (kT + 1);
        pm = at; at += kT * (kT + 1);
        x = at; at += kT * (kT + 1);
        em = at; at += kT * (kT + 1);
        total = at + 5 * kT + kThreadsD / 32;
    }
};

__global__ void __launch_bounds__(kThreadsD) delta_bwd_direct_kernel(DeltaBwdArgs p) {
    extern __shared__ __align__(16) float sh[];
    const DeltaArgs &a = p.f;
    const int P = a.headdim, N = a.dstate, tid = threadIdx.x;
    const Layout L(P, N);
    double *cum = reinterpret_cast<double *>(sh + L.cum);
    float *ds = sh + L.ds, *s0 = sh + L.s0, *q = sh + L.q, *k = sh + L.k, *o = sh + L.o, *r = sh + L.r, *e = sh + L.e;
    float *left = sh + L.l, *kk = sh + L.kk, *pm = sh + L.pm, *x = sh + L.x, *em = sh + L.em;
    float *gam = em + kT * (kT + 1), *wend = gam + kT, *beta = wend + kT, *dot = beta + kT, *dbeta = dot + kT;
    float *part = dbeta + kT;
    constexpr int ldt = kT + 1;
    const int64_t bh = blockIdx.x, b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int64_t nch = (a.seqlen + kT - 1) / kT;
    for (int i = tid; i < P * N; i += kThreadsD)
        ds[i / N * L.ldn + i % N] = p.dend ? p.dend[bh * P * (int64_t)N + i] : 0.f;
    for (int64_t ch = nch - 1; ch >= 0; --ch) {
        const int64_t t0 = ch * kT;
        const int live = (int)(a.seqlen - t0 < kT ? a.seqlen - t0 : kT);
        __syncthreads();
        for (int i = tid; i < P * N; i += kThreadsD)
            s0[i / N * L.ldn + i % N] = a.marks[(bh * nch + ch) * P * N + i];
        for (int i = tid; i < kT * N; i += kThreadsD) {
            const int t = i / N, c = i % N;
            const int64_t at = ((b * a.seqlen + t0 + t) * a.groups + gr) * N + c;
            q[t * L.ldn + c] = t < live ? io_traits<float>::load(static_cast<const float *>(a.q) + at) : 0.f;
            k[t * L.ldn + c] = t < live ? io_traits<float>::load(static_cast<const float *>(a.k) + at) : 0.f;
        }
        for (int i = tid; i < kT * P; i += kThreadsD) {
            const int t = i / P, c = i % P;
            const int64_t at = ((b * a.seqlen + t0 + t) * a.heads + h) * P + c;
            o[t * L.ldp + c] = t < live ? io_traits<float>::load(static_cast<const float *>(p.dout) + at) : 0.f;
            r[t * L.ldp + c] = t < live ? a.r[at] : 0.f;
        }
        if (tid == 0) {
            double sum = 0.0;
            for (int t = 0; t < kT; ++t) {
                if (t < live) sum += fmax((double)a.g[(b * a.seqlen + t0 + t) * a.heads + h], -1e4);
                cum[t] = sum;
            }
        }
        __syncthreads();
        if (tid < kT) {
            gam[tid] = expf((float)cum[tid]);
            wend[tid] = expf((float)(cum[kT - 1] - cum[tid]));
            beta[tid] = tid < live ? a.beta[(b * a.seqlen + t0 + tid) * a.heads + h] : 0.f;
            dot[tid] = 0.f;
        }
        // Abar (without the diagonal) and P
        for (int i = tid; i < kT * kT; i += kThreadsD) {
            const int t = i / kT, s = i % kT;
            float ck = 0.f, cq = 0.f;
            if (s <= t)
                for (int c = 0; c < N; ++c) {
                    ck = fmaf(k[t * L.ldn + c], k[s * L.ldn + c], ck);
                    cq = fmaf(q[t * L.ldn + c], k[s * L.ldn + c], cq);
                }
            const float f = s <= t ? expf((float)(cum[t] - cum[s])) : 0.f;
            kk[t * ldt + s] = s < t ? f * ck : 0.f;
            pm[t * ldt + s] = s <= t ? a.scale * f * cq : 0.f;
        }
        __syncthreads();
        // dU, then e in its place, one column of V per thread; dV = beta e
        for (int v = tid; v < P; v += kThreadsD) {
            float du[kT];
#pragma unroll
            for (int t = 0; t < kT; ++t) du[t] = 0.f;
            for (int c = 0; c < N; ++c) {
                const float d = ds[v * L.ldn + c];
#pragma unroll
                for (int t = 0; t < kT; ++t) du[t] = fmaf(d, k[t * L.ldn + c], du[t]);
            }
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                du[t] *= wend[t];
#pragma unroll
                for (int t2 = 0; t2 < kT; ++t2)
                    if (t2 >= t) du[t] = fmaf(pm[t2 * ldt + t], o[t2 * L.ldp + v], du[t]);
            }
#pragma unroll
            for (int t = kT - 1; t >= 0; --t) {
#pragma unroll
                for (int t2 = 0; t2 < kT; ++t2)
                    if (t2 > t) du[t] = fmaf(-kk[t2 * ldt + t] * beta[t2], du[t2], du[t]);
                e[t * L.ldp + v] = du[t];
                if (t < live) {
                    float *dst = static_cast<float *>(p.dv) + ((b * a.seqlen + t0 + t) * a.heads + h) * P + v;
                    io_traits<float>::store(dst, beta[t] * du[t]);
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < kT * kT; i += kThreadsD) {
            const int t = i / kT, s = i % kT;
            float cx = 0.f, ce = 0.f;
            if (s <= t)
                for (int v = 0; v < P; ++v) {
                    cx = fmaf(o[t * L.ldp + v], r[s * L.ldp + v], cx);
                    ce = fmaf(e[t * L.ldp + v], r[s * L.ldp + v], ce);
                }
            const float f = s <= t ? expf((float)(cum[t] - cum[s])) * beta[s] : 0.f;
            x[t * ldt + s] = s <= t ? a.scale * f * cx : 0.f;
            em[t * ldt + s] = s < t ? -f * beta[t] * ce : 0.f;
            if (s == t) dbeta[t] = ce;
        }
        __syncthreads();
        // dq, dk; the row products of dg: eight lanes per token and pass over dstate
        float inner = 0.f;
        const float whole = gam[kT - 1];
        for (int i = tid; i < kT * N; i += kThreadsD) {
            const int t = i / N, c = i % N;
            float cq = 0.f, cl = 0.f, cr = 0.f;
            for (int v = 0; v < P; ++v) {
                const float s = s0[v * L.ldn + c];
                cq = fmaf(o[t * L.ldp + v], s, cq);
                cl = fmaf(e[t * L.ldp + v], s, cl);
                cr = fmaf(r[t * L.ldp + v], ds[v * L.ldn + c], cr);
            }
            cq *= a.scale * gam[t];
            cl *= -gam[t] * beta[t];
            cr *= wend[t] * beta[t];
            inner = fmaf(k[t * L.ldn + c], cr, inner);
            for (int s = 0; s < kT; ++s) {
                if (s <= t) {
                    cq = fmaf(x[t * ldt + s], k[s * L.ldn + c], cq);
                    cl = fmaf(em[t * ldt + s], k[s * L.ldn + c], cl);
                }
                if (s >= t) {
                    cr = fmaf(x[s * ldt + t], q[s * L.ldn + c], cr);
                    cr = fmaf(em[s * ldt + t], k[s * L.ldn + c], cr);
                }
            }
            left[t * L.ldn + c] = q[t * L.ldn + c] * cq + k[t * L.ldn + c] * (cl - cr);
            if (t < live) {
                const int64_t at = ((b * a.seqlen + t0 + t) * a.heads + h) * N + c;
                p.dq_heads[at] = cq;
                p.dk_heads[at] = cl + cr;
            }
        }
        // dS0, and <S0, dS1> on the way
        for (int i = tid; i < P * N; i += kThreadsD) {
            const int v = i / N, c = i % N;
            inner = fmaf(whole * s0[v * L.ldn + c], ds[v * L.ldn + c], inner);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, off);
        if ((tid & 31) == 0) part[tid >> 5] = inner;
        __syncthreads();
        for (int i = tid; i < P * N; i += kThreadsD) {
            const int v = i / N, c = i % N;
            float d = whole * ds[v * L.ldn + c];
            for (int t = 0; t < kT; ++t)
                d = fmaf(gam[t], a.scale * o[t * L.ldp + v] * q[t * L.ldn + c] -
                                     beta[t] * e[t * L.ldp + v] * k[t * L.ldn + c], d);
            ds[v * L.ldn + c] = d;
        }
        {
            const int t = tid / 16, part16 = tid % 16;  // 256 threads: 16 tokens x 16
            float sum = 0.f;
            for (int c = part16; c < N; c += 16) sum += left[t * L.ldn + c];
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (part16 == 0) dot[t] = sum;
        }
        __syncthreads();
        if (tid < live) {
            float sum = 0.f;
            for (int w = 0; w < kThreadsD / 32; ++w) sum += part[w];
            for (int t = kT - 1; t >= tid; --t) sum += dot[t];
            const int64_t at = (b * a.seqlen + t0 + tid) * a.heads + h;
            p.dg[at] = sum;
            p.dbeta[at] = dbeta[tid];
        }
    }
    if (!p.dh0) return;
    __syncthreads();
    for (int i = tid; i < P * N; i += kThreadsD) p.dh0[bh * P * (int64_t)N + i] = ds[i / N * L.ldn + i % N];
}

// dq, dk of a group: the sum over its heads, in their order
__global__ void __launch_bounds__(256) delta_group_sum_kernel(const float *dq_heads, const float *dk_heads, float *dq,
                                                              float *dk, int64_t tokens, int groups, int rep, int n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = tokens * groups * n;
    if (i >= total) return;
    const int64_t tg = i / n, c = i - tg * n;  // (token, group): heads tg rep .. tg rep + rep - 1
    float sq = 0.f, sk = 0.f;
    for (int r = 0; r < rep; ++r) {
        sq += dq_heads[(tg * rep + r) * n + c];
        sk += dk_heads[(tg * rep + r) * n + c];
    }
    io_traits<float>::store(dq + i, sq);
    io_traits<float>::store(dk + i, sk);
}

}  // namespace

cudaError_t launch_delta_bwd_direct(const DeltaBwdArgs &p, cudaStream_t st) {
    const DeltaArgs &a = p.f;
    const int bytes = Layout(a.headdim, a.dstate).total * (int)sizeof(float);
    cudaError_t e = allow_smem<delta_bwd_direct_kernel, 4 * Layout(kDeltaMaxDstate, kDeltaMaxDstate).total>();
    if (e != cudaSuccess) return e;
    delta_bwd_direct_kernel<<<(unsigned)(a.batch * a.heads), kThreadsD, bytes, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t tokens = a.batch * a.seqlen, total = tokens * a.groups * a.dstate;
    delta_group_sum_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
        p.dq_heads, p.dk_heads, static_cast<float *>(p.dq), static_cast<float *>(p.dk), tokens, a.groups, a.heads / a.groups,
        a.dstate);
    return cudaGetLastError();
}

}  // namespace ssm
