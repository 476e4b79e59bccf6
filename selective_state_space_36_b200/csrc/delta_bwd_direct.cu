// delta_bwd_direct.cu -- the gated delta rule's gradient in float32 throughout,
// for float32 tensors, on chunks of kDeltaStep tokens with a state per chunk from
// launch_delta_recurrent.  The formulas of delta_fused_bwd.cu in another form:
//   dU = Pm^T dO + w K dS1^T,   e = dU - Abar^T (beta e),   dV = beta e,
//   dS0 = gam_C dS1 + (scale gam dO)^T Q - (gam dV)^T K,
//   dbeta_t = e_t . r_t,   X, E, L and R as there
// with Abar = strict_lower(Gam o K K^T) and Pm = scale lower(Gam o Q K^T).
//
// The pass backwards in time couples only dstate: a row of the state (a column
// of V) goes through it by itself, so eight lanes take one each, their part of
// dS1 in registers, and 16 rows are a block.  Everything else, which couples
// headdim too, is left to a second kernel over all chunks at once.
//
// Measured: 3 sequences of 600 tokens, 16 heads of 100 x 80: 372 us backwards (9.8 us
// per 16 tokens, bound by their chain of steps) and 177 us for the rest (bound by
// shared-memory reads, 5 per 12 products); one kernel that walked over the chunks
// with a head per block took 2050 us.
#include "delta_rule.cuh"
#include "kernel_setup.cuh"
#include "ssm_device.cuh"

namespace ssm {
namespace {

constexpr int kT = kDeltaStep, kLdT = kT + 1;

// Row stride of kT rows of dstate values: 16-byte pieces, an odd number of them.
__host__ __device__ constexpr int row_stride(int n) { return 4 * (((n + 3) / 4) | 1); }

__device__ __forceinline__ void copy4(float *smem, const float *gmem, bool have) {
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(smem));
    const int n = have ? 4 : 0;  // 0: no global read, destination zero-filled
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(s), "l"(gmem), "r"(n) : "memory");
}

// A lane's token of a chunk: log decay and beta, zero behind the chunk's end.
__device__ __forceinline__ float2 token_decay(const DeltaArgs &a, int64_t token, int h, int live, int lane) {
    const int64_t at = (token + lane) * a.heads + h;
    return lane < live ? make_float2(a.g[at], a.beta[at]) : make_float2(0.f, 0.f);
}

// A chunk's decays from its tokens', warp-wide (lanes 0 to kT - 1).
__device__ __forceinline__ void chunk_decays(float2 gb, int lane, double *cum, float *gam, float *wend, float *beta) {
    double sum = log_decay(gb.x);
#pragma unroll
    for (int o = 1; o < kT; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
    }
    const double end = __shfl_sync(0xffffffffu, sum, kT - 1);
    if (lane < kT) {
        cum[lane] = sum;
        gam[lane] = expf((float)sum);
        wend[lane] = expf((float)(end - sum));
        beta[lane] = gb.y;
    }
}

// Entry (t, s), s <= t, of a triangle in rows: entry i.
__device__ __forceinline__ void triangle(int i, int &t, int &s) {
    t = 0;
    while ((t + 1) * (t + 2) / 2 <= i) ++t;
    s = i - t * (t + 1) / 2;
}
constexpr int kTriangle = kT * (kT + 1) / 2;

// ------------------------------------------------------- backwards in time
constexpr int kRowsR = 16, kThreadsR = 8 * kRowsR;

struct ReverseSmem {  // float offsets; ld: row_stride(dstate)
    int stage, total;
    __host__ __device__ constexpr explicit ReverseSmem(int ld) : stage(2 * kT * ld + kT * kRowsR), total(2 * stage) {}
};

__global__ void __launch_bounds__(kThreadsR) delta_reverse_direct_kernel(DeltaBwdArgs p, float *ds1, float *es) {
    extern __shared__ __align__(16) float sh[];
    __shared__ double cum[kT];
    __shared__ __align__(16) float kkb[kT][kT];
    __shared__ float gam[kT], wend[kT], beta[kT], pm[kT][kLdT], e[kT][kRowsR + 1];
    const DeltaArgs &a = p.f;
    const int P = a.headdim, N = a.dstate, tid = threadIdx.x, lane = tid & 31, sub = tid & 7, mine = tid >> 3;
    const int ld = row_stride(N);
    const ReverseSmem L(ld);
    const int tiles = (P + kRowsR - 1) / kRowsR;
    const int64_t bh = blockIdx.x / tiles, b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int v0 = (int)(blockIdx.x - bh * tiles) * kRowsR, row = v0 + mine;
    const int64_t nch = (a.seqlen + kT - 1) / kT;
    const float *gq = static_cast<const float *>(a.q), *gk = static_cast<const float *>(a.k);
    const float *go = static_cast<const float *>(p.dout);
    int ti[2], si[2];
    triangle(tid, ti[0], si[0]);
    triangle(tid + kThreadsR, ti[1], si[1]);

    auto issue = [&](int64_t ch) {  // chunk ch's tiles into stage ch & 1
        if (ch >= 0) {
            float *k = sh + (ch & 1) * L.stage, *q = k + kT * ld, *o = q + kT * ld;
            const int64_t t0 = ch * kT;
            static_assert(kThreadsR == 8 * kT, "eight threads a token");
            const bool row_in = t0 + mine < a.seqlen;
            const int64_t at = row_in ? ((b * a.seqlen + t0 + mine) * a.groups + gr) * N : 0;
#pragma unroll 4
            for (int c = sub; c < ld; c += 8) {
                const bool in = row_in && c < N;
                copy4(k + mine * ld + c, gk + (in ? at + c : 0), in);
                copy4(q + mine * ld + c, gq + (in ? at + c : 0), in);
            }
            for (int i = tid; i < kT * kRowsR; i += kThreadsR) {
                const int t = i / kRowsR, c = i % kRowsR;
                const bool in = t0 + t < a.seqlen && v0 + c < P;
                copy4(o + i, in ? go + ((b * a.seqlen + t0 + t) * a.heads + h) * P + v0 + c : go, in);
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    float d[4][4];  // columns 4 (sub + 8 i) ..
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 4 * (sub + 8 * i) + j;
            d[i][j] = p.dend && row < P && c < N ? p.dend[(bh * P + row) * (int64_t)N + c] : 0.f;
        }
    auto fetch = [&](int64_t ch) {
        const int64_t left = a.seqlen - ch * kT;
        return ch >= 0 && tid < 32 ? token_decay(a, b * a.seqlen + ch * kT, h, (int)(left < kT ? left : kT), lane)
                                   : make_float2(0.f, 0.f);
    };
    issue(nch - 1);
    float2 gb = fetch(nch - 1);
    for (int64_t ch = nch - 1; ch >= 0; --ch) {
        const int64_t t0 = ch * kT, token = b * a.seqlen + t0;
        const int live = (int)(a.seqlen - t0 < kT ? a.seqlen - t0 : kT);
        const float *k = sh + (ch & 1) * L.stage, *q = k + kT * ld, *o = q + kT * ld;
        issue(ch - 1);
        if (row < P) {
            float *to = ds1 + ((bh * nch + ch) * P + row) * (int64_t)N;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * (sub + 8 * i) + j < N) to[4 * (sub + 8 * i) + j] = d[i][j];
        }
        if (tid < 32) chunk_decays(gb, lane, cum, gam, wend, beta);
        gb = fetch(ch - 1);
        asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        __syncthreads();
        // Abar_ts beta_t and Pm_ts
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (tid + u * kThreadsR >= kTriangle) continue;
            const int t = ti[u], s = si[u];
            float ck[2] = {0.f, 0.f}, cq[2] = {0.f, 0.f};
#pragma unroll 4
            for (int c = 0; c < N; c += 4) {  // (zeros behind the row)
                const float4 ks = *reinterpret_cast<const float4 *>(k + s * ld + c);
                const float4 kt = *reinterpret_cast<const float4 *>(k + t * ld + c);
                const float4 qt = *reinterpret_cast<const float4 *>(q + t * ld + c);
                ck[0] = fmaf(kt.x, ks.x, ck[0]); ck[1] = fmaf(kt.y, ks.y, ck[1]);
                ck[0] = fmaf(kt.z, ks.z, ck[0]); ck[1] = fmaf(kt.w, ks.w, ck[1]);
                cq[0] = fmaf(qt.x, ks.x, cq[0]); cq[1] = fmaf(qt.y, ks.y, cq[1]);
                cq[0] = fmaf(qt.z, ks.z, cq[0]); cq[1] = fmaf(qt.w, ks.w, cq[1]);
            }
            const float f = expf((float)(cum[t] - cum[s]));
            kkb[t][s] = s < t ? f * (ck[0] + ck[1]) * beta[t] : 0.f;
            pm[t][s] = a.scale * f * (cq[0] + cq[1]);
        }
        // dS1 K^T of this row: the lanes' parts, then sums over lanes; a lane ends with tokens 2 sub, 2 sub + 1
        float du[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (32 * i >= N) break;
                const int c = 4 * (sub + 8 * i);
                const float4 kv = c < ld ? *reinterpret_cast<const float4 *>(k + t * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                s[0] = fmaf(d[i][0], kv.x, s[0]); s[1] = fmaf(d[i][1], kv.y, s[1]);
                s[0] = fmaf(d[i][2], kv.z, s[0]); s[1] = fmaf(d[i][3], kv.w, s[1]);
            }
            du[t] = s[0] + s[1];
        }
#pragma unroll
        for (int o8 = 4; o8 > 0; o8 >>= 1)
#pragma unroll
            for (int i = 0; i < 2 * o8; ++i) {
                const bool up = (sub & o8) != 0;
                const float keep = up ? du[i + 2 * o8] : du[i], send = up ? du[i] : du[i + 2 * o8];
                du[i] = keep + __shfl_xor_sync(0xffffffffu, send, o8);
            }
        __syncthreads();  // kkb, pm
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * sub + i;
            x[i] = wend[t] * du[i];
#pragma unroll
            for (int t2 = 0; t2 < kT; ++t2)
                if (t2 >= t) x[i] = fmaf(pm[t2][t], o[t2 * kRowsR + mine], x[i]);
        }
        // e from the last token: what a token's e takes from those before it
#pragma unroll
        for (int t = kT - 1; t > 0; --t) {
            const float et = __shfl_sync(0xffffffffu, x[t & 1], (lane & 24) + (t >> 1));
            const float2 w = *reinterpret_cast<const float2 *>(&kkb[t][2 * sub]);
            if (2 * sub < t) x[0] = fmaf(-w.x, et, x[0]);
            if (2 * sub + 1 < t) x[1] = fmaf(-w.y, et, x[1]);
        }
        e[2 * sub][mine] = x[0];
        e[2 * sub + 1][mine] = x[1];
        __syncwarp();
        const float whole = gam[kT - 1];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] *= whole;
#pragma unroll 4
        for (int t = 0; t < kT; ++t) {
            const float cq = gam[t] * a.scale * o[t * kRowsR + mine], ck = -gam[t] * beta[t] * e[t][mine];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 4 * (sub + 8 * i);
                if (c >= ld) break;
                const float4 qv = *reinterpret_cast<const float4 *>(q + t * ld + c);
                const float4 kv = *reinterpret_cast<const float4 *>(k + t * ld + c);
                d[i][0] = fmaf(cq, qv.x, fmaf(ck, kv.x, d[i][0]));
                d[i][1] = fmaf(cq, qv.y, fmaf(ck, kv.y, d[i][1]));
                d[i][2] = fmaf(cq, qv.z, fmaf(ck, kv.z, d[i][2]));
                d[i][3] = fmaf(cq, qv.w, fmaf(ck, kv.w, d[i][3]));
            }
        }
        __syncthreads();  // all rows' e; the tiles are read
        for (int i = tid; i < kT * kRowsR; i += kThreadsR) {
            const int t = i / kRowsR, c = i % kRowsR;
            if (t < live && v0 + c < P) {
                const int64_t at = ((token + t) * a.heads + h) * P + v0 + c;
                es[at] = e[t][c];
                static_cast<float *>(p.dv)[at] = beta[t] * e[t][c];
            }
        }
        __syncthreads();  // e, the decays and the matrices are read
    }
    if (!p.dh0 || row >= P) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * (sub + 8 * i) + j < N) p.dh0[(bh * P + row) * (int64_t)N + 4 * (sub + 8 * i) + j] = d[i][j];
}

// ------------------------------------------------------- all chunks at once
constexpr int kThreadsD = 256, kLdV = kT + 4;  // tokens of a column of V, 16-byte pieces

struct GradSmem {  // float offsets in shared memory
    int ldn, ds, s0, q, k, l, o, r, e, total;
    __host__ __device__ constexpr GradSmem(int P, int N)
        : ldn(N | 1), ds(0), s0(P * ldn), q(2 * P * ldn), k(q + kT * ldn), l(k + kT * ldn),
          o((l + kT * ldn + 3) / 4 * 4), r(o + P * kLdV), e(r + P * kLdV), total(e + P * kLdV) {}
};

__global__ void __launch_bounds__(kThreadsD) delta_grad_direct_kernel(DeltaBwdArgs p, const float *ds1, const float *es) {
    extern __shared__ __align__(16) float sh[];
    __shared__ double cum[kT];
    __shared__ float gam[kT], wend[kT], beta[kT], dbeta[kT], dot[kT], part[kThreadsD / 32], x[kT][kLdT], em[kT][kLdT];
    const DeltaArgs &a = p.f;
    const int P = a.headdim, N = a.dstate, tid = threadIdx.x;
    const GradSmem L(P, N);
    float *ds = sh + L.ds, *s0 = sh + L.s0, *q = sh + L.q, *k = sh + L.k, *left = sh + L.l;
    float *o = sh + L.o, *r = sh + L.r, *e = sh + L.e;  // [headdim][kLdV]
    const int64_t nch = (a.seqlen + kT - 1) / kT, unit = blockIdx.x, bh = unit / nch, ch = unit - bh * nch, b = bh / a.heads;
    const int h = (int)(bh - b * a.heads), gr = h / (a.heads / a.groups);
    const int64_t t0 = ch * kT, token = b * a.seqlen + t0;
    const int live = (int)(a.seqlen - t0 < kT ? a.seqlen - t0 : kT);
#pragma unroll 4
    for (int i = tid; i < P * N; i += kThreadsD) {
        const int at = i / N * L.ldn + i % N;
        copy4(s0 + at, a.marks + unit * P * N + i, true);
        copy4(ds + at, ds1 + unit * P * N + i, true);
    }
    for (int i = tid; i < kT * N; i += kThreadsD) {
        const int t = i / N, c = i % N;
        const int64_t at = t < live ? ((token + t) * a.groups + gr) * N + c : 0;
        copy4(q + t * L.ldn + c, static_cast<const float *>(a.q) + at, t < live);
        copy4(k + t * L.ldn + c, static_cast<const float *>(a.k) + at, t < live);
    }
    for (int i = tid; i < kT * P; i += kThreadsD) {
        const int t = i / P, c = i % P;
        const int64_t at = t < live ? ((token + t) * a.heads + h) * P + c : 0;
        copy4(o + c * kLdV + t, static_cast<const float *>(p.dout) + at, t < live);
        copy4(r + c * kLdV + t, a.r + at, t < live);
        copy4(e + c * kLdV + t, es + at, t < live);
    }
    if (tid < 32) chunk_decays(token_decay(a, token, h, live, tid), tid, cum, gam, wend, beta);
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
    if (tid < kTriangle) {
        int t, s;
        triangle(tid, t, s);
        float cx[2] = {0.f, 0.f}, ce[2] = {0.f, 0.f};
#pragma unroll 4
        for (int v = 0; v < P; ++v) {
            cx[v & 1] = fmaf(o[v * kLdV + t], r[v * kLdV + s], cx[v & 1]);
            ce[v & 1] = fmaf(e[v * kLdV + t], r[v * kLdV + s], ce[v & 1]);
        }
        const float f = expf((float)(cum[t] - cum[s])) * beta[s], ee = ce[0] + ce[1];
        x[t][s] = a.scale * f * (cx[0] + cx[1]);
        em[t][s] = s < t ? -f * beta[t] * ee : 0.f;
        if (s == t) dbeta[t] = ee;
    }
    __syncthreads();
    // dq, dk: four tokens and a column of dstate at a time; the row products of dg
    float inner = 0.f;
    for (int i = tid; i < kT / 4 * N; i += kThreadsD) {
        const int tt = i / N * 4, c = i % N;
        float cq[4] = {}, cl[4] = {}, cr[4] = {};
#pragma unroll 4
        for (int v = 0; v < P; ++v) {
            const float s = s0[v * L.ldn + c], d = ds[v * L.ldn + c];
            const float4 ov = *reinterpret_cast<const float4 *>(o + v * kLdV + tt);
            const float4 ev = *reinterpret_cast<const float4 *>(e + v * kLdV + tt);
            const float4 rv = *reinterpret_cast<const float4 *>(r + v * kLdV + tt);
            cq[0] = fmaf(ov.x, s, cq[0]); cq[1] = fmaf(ov.y, s, cq[1]); cq[2] = fmaf(ov.z, s, cq[2]); cq[3] = fmaf(ov.w, s, cq[3]);
            cl[0] = fmaf(ev.x, s, cl[0]); cl[1] = fmaf(ev.y, s, cl[1]); cl[2] = fmaf(ev.z, s, cl[2]); cl[3] = fmaf(ev.w, s, cl[3]);
            cr[0] = fmaf(rv.x, d, cr[0]); cr[1] = fmaf(rv.y, d, cr[1]); cr[2] = fmaf(rv.z, d, cr[2]); cr[3] = fmaf(rv.w, d, cr[3]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = tt + u;
            cq[u] *= a.scale * gam[t];
            cl[u] *= -gam[t] * beta[t];
            cr[u] *= wend[t] * beta[t];
            inner = fmaf(k[t * L.ldn + c], cr[u], inner);
        }
        for (int s = 0; s < kT; ++s) {
            const float ks = k[s * L.ldn + c], qs = q[s * L.ldn + c];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = tt + u;
                if (s <= t) {
                    cq[u] = fmaf(x[t][s], ks, cq[u]);
                    cl[u] = fmaf(em[t][s], ks, cl[u]);
                }
                if (s >= t) cr[u] = fmaf(x[s][t], qs, fmaf(em[s][t], ks, cr[u]));
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = tt + u;
            left[t * L.ldn + c] = q[t * L.ldn + c] * cq[u] + k[t * L.ldn + c] * (cl[u] - cr[u]);
            if (t < live) {
                const int64_t at = ((token + t) * a.heads + h) * N + c;
                p.dq_heads[at] = cq[u];
                p.dk_heads[at] = cl[u] + cr[u];
            }
        }
    }
    float states = 0.f;
    for (int i = tid; i < P * N; i += kThreadsD) {
        const int at = i / N * L.ldn + i % N;
        states = fmaf(s0[at], ds[at], states);
    }
    inner = fmaf(gam[kT - 1], states, inner);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, off);
    if ((tid & 31) == 0) part[tid >> 5] = inner;
    __syncthreads();
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
        const int64_t at = (token + tid) * a.heads + h;
        p.dg[at] = sum;
        p.dbeta[at] = dbeta[tid];
    }
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

cudaError_t launch_delta_bwd_direct(const DeltaBwdArgs &p, float *ds1, float *es, cudaStream_t st) {
    const DeltaArgs &a = p.f;
    constexpr int most = kDeltaMaxDstate;
    const int64_t heads = a.batch * a.heads, chunks = (a.seqlen + kT - 1) / kT;
    cudaError_t e = allow_smem<delta_reverse_direct_kernel, 4 * ReverseSmem(row_stride(most)).total>();
    if (e != cudaSuccess) return e;
    e = allow_smem<delta_grad_direct_kernel, 4 * GradSmem(most, most).total>();
    if (e != cudaSuccess) return e;
    const int64_t blocks = heads * ((a.headdim + kRowsR - 1) / kRowsR);
    delta_reverse_direct_kernel<<<(unsigned)blocks, kThreadsR, 4 * ReverseSmem(row_stride(a.dstate)).total, st>>>(p, ds1, es);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    delta_grad_direct_kernel<<<(unsigned)(heads * chunks), kThreadsD, 4 * GradSmem(a.headdim, a.dstate).total, st>>>(p, ds1, es);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t tokens = a.batch * a.seqlen, total = tokens * a.groups * a.dstate;
    delta_group_sum_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
        p.dq_heads, p.dk_heads, static_cast<float *>(p.dq), static_cast<float *>(p.dk), tokens, a.groups, a.heads / a.groups,
        a.dstate);
    return cudaGetLastError();
}

}  // namespace ssm
