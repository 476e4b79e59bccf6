// delta_recurrent.cu -- the gated delta rule token by token, in fp32 for both
// element types: the decode step, and whole sequences where the chunked kernels
// do not apply (float32 tensors) or do not pay (a few dozen tokens).
//
// Eight lanes share one row of the state S (headdim x dstate): a row's
// dstate values are dealt out in pieces of four, piece i to lane i mod 8, so
// that the eight lanes read and write 128 contiguous bytes at a time.  A
// warp holds 4 rows at once and kRows sets of them, all in registers for the
// whole sequence; rows are independent.  Per token a row needs two dot products
// over dstate (S k and S q), each reduced over its eight lanes by three shuffles.
//
// One token moves 8 headdim dstate bytes of state per head and computes 8
// flops per state value, so the step is bound by HBM: the loads of all
// kRows sets are issued before the first is used (256 sequences x 32 heads of
// 128 x 128: 165 us, the measured copy rate).  Over a sequence the state stays
// in registers and the chain of dot products bounds the kernel, two tokens a
// link; k, q, v, g and beta come a stage of kTok tokens ahead through shared memory.
#include "cp_async.cuh"
#include "delta_rule.cuh"
#include "ssm_device.cuh"

#include <type_traits>

namespace ssm {
namespace {

constexpr int kLanes = 8;             // lanes that share a state row
constexpr int kWarps = 4;             // warps per block
constexpr int kRows = 2;              // row sets per warp
constexpr int kRowsPerBlock = kWarps * 4 * kRows;

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}

template <int N>
__device__ __forceinline__ void sum8(float *x) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
}

// A lane's part of a row's dot product, as four short chains.
template <int PIECES>
__device__ __forceinline__ float row_dot(const float (&s)[PIECES][4], const float (&x)[PIECES][4]) {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = fmaf(s[p][e], x[p][e], d[e]);
    return (d[0] + d[1]) + (d[2] + d[3]);
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

// The state rows of this lane, kRows sets; plain loads: the state may be
// written back to the same place.
template <int PIECES, bool VEC, int ROWS>
__device__ __forceinline__ void get_rows(float (&s)[ROWS][PIECES][4], const float *h0, int64_t bh, int row0,
                                         int headdim, int sub, int n) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = row0 + 4 * r;
        const float *src = h0 ? h0 + (bh * headdim + row) * (int64_t)n : nullptr;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int c = 4 * (sub + kLanes * p);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r][p][e] = 0.f;
            if (!src || row >= headdim) continue;
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
}

// One token (decode) or a few: the tokens' operands straight from global
// memory.  PIECES pieces of four values per lane: dstate <= 32 PIECES.  VEC:
// dstate is a multiple of 4 and q, k, the states are aligned to four elements.
// For 256 sequences x 32 heads of 128 x 128 the order of a warp's accesses
// decides: 166 us with the state's loads before, and its stores after, a token
// loop that fetches its own operands; 186 to 206 us with everything fetched
// ahead or a loop of one token unrolled away.
template <typename T, int PIECES, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) delta_step_kernel(DeltaArgs a) {
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
    T *out = static_cast<T *>(a.out) + ((b * a.seqlen) * a.heads + h) * a.headdim;
    const float *g = a.g + (b * a.seqlen) * a.heads + h, *beta = a.beta + (b * a.seqlen) * a.heads + h;

    float s[kRows][PIECES][4];
    get_rows<PIECES, VEC>(s, a.h0, bh, row0, a.headdim, sub, n);
    for (int64_t t = 0; t < a.seqlen; ++t) {
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
            const float u = bt * (vv[r] - sum8(dot));
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
            if (sub == 0 && row < a.headdim) io_traits<T>::store(out + row, a.scale * o);
        }
        q += (int64_t)a.groups * n;
        k += (int64_t)a.groups * n;
        v += (int64_t)a.heads * a.headdim;
        out += (int64_t)a.heads * a.headdim;
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

constexpr int kFewTokens = 4;  // up to this many go to delta_step_kernel
constexpr int kTok = 16;       // tokens per stage of a sequence

template <typename T, int PIECES, int ROWS>
struct TokenStage {
    T k[kTok][32 * PIECES], q[kTok][32 * PIECES];
    T v[kTok][kWarps * 4 * ROWS];
    float decay[kTok], beta[kTok];
    float4 pair[kTok / 2];  // of tokens 1, 2: k1 . k2, k1 . q1, k1 . q2, k2 . q2
};

// A sequence.  VEC: as above, and rows of q and k are multiples of 16 bytes and
// start aligned (copied asynchronously).  STORE: the backward pass's first half
// (DeltaArgs::marks, r; no output).
template <typename T, int PIECES, int ROWS, bool VEC, bool STORE>
__global__ void __launch_bounds__(kWarps * 32) delta_tokens_kernel(DeltaArgs a) {
    __shared__ __align__(16) TokenStage<T, PIECES, ROWS> stages[2];
    constexpr int kThreads = kWarps * 32, kBlockRows = kWarps * 4 * ROWS;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane & (kLanes - 1), n = a.dstate;
    const int tiles = (a.headdim + kBlockRows - 1) / kBlockRows;
    const int64_t bh = blockIdx.x / tiles, b = bh / a.heads;
    const int tile = (int)(blockIdx.x % tiles), h = (int)(bh % a.heads), gr = h / (a.heads / a.groups);
    const int first = tile * kBlockRows, mine = (tid >> 5) * 4 * ROWS + (lane >> 3), row0 = first + mine;
    const int64_t qk_ld = (int64_t)a.groups * n, v_ld = (int64_t)a.heads * a.headdim;
    const T *q = static_cast<const T *>(a.q) + (b * a.seqlen * a.groups + gr) * n;
    const T *k = static_cast<const T *>(a.k) + (b * a.seqlen * a.groups + gr) * n;
    const T *v = static_cast<const T *>(a.v) + (b * a.seqlen * a.heads + h) * a.headdim + first;
    const float *g = a.g + b * a.seqlen * a.heads + h, *beta = a.beta + b * a.seqlen * a.heads + h;
    const int have = a.headdim - first < kBlockRows ? a.headdim - first : kBlockRows;

    auto issue = [&](int64_t t0) {
        if (t0 < a.seqlen) {
            TokenStage<T, PIECES, ROWS> &st = stages[(t0 / kTok) & 1];
            const int live = (int)(a.seqlen - t0 < kTok ? a.seqlen - t0 : kTok);
            if (VEC) {
                constexpr int E = 16 / sizeof(T), PER = 32 * PIECES / E;
                for (int i = tid; i < kTok * PER; i += kThreads) {
                    const int t = i / PER, c = (i % PER) * E;
                    const bool in = t < live && c < n;
                    const int64_t at = (t0 + t) * qk_ld + c;
                    cp_async16(&st.k[t][c], in ? k + at : k, in);
                    cp_async16(&st.q[t][c], in ? q + at : q, in);
                }
            } else {
                for (int i = tid; i < kTok * 32 * PIECES; i += kThreads) {
                    const int t = i / (32 * PIECES), c = i % (32 * PIECES);
                    const bool in = t < live && c < n;
                    st.k[t][c] = in ? k[(t0 + t) * qk_ld + c] : T(0.f);
                    st.q[t][c] = in ? q[(t0 + t) * qk_ld + c] : T(0.f);
                }
            }
        }
        cp_async_commit();
    };
    // v, g and beta have rows too short for asynchronous copies: loaded into
    // registers when a stage begins, put into the next stage's tile at its end
    constexpr int kV = kTok * kBlockRows / kThreads;
    T rv[kV];
    float rg = 0.f, rb = 0.f;
    auto small_loads = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int t = (tid + i * kThreads) / kBlockRows, c = tid % kBlockRows;
            rv[i] = t0 + t < a.seqlen && c < have ? v[(t0 + t) * v_ld + c] : T(0.f);
        }
        if (tid < kTok) {  // behind the end: tokens that leave the state as it is
            const bool in = t0 + tid < a.seqlen;
            rg = in ? g[(t0 + tid) * a.heads] : 0.f;
            rb = in ? beta[(t0 + tid) * a.heads] : 0.f;
        }
    };
    auto small_stores = [&](int64_t t0) {
        TokenStage<T, PIECES, ROWS> &st = stages[(t0 / kTok) & 1];
#pragma unroll
        for (int i = 0; i < kV; ++i) st.v[(tid + i * kThreads) / kBlockRows][tid % kBlockRows] = rv[i];
        if (tid < kTok) {
            st.decay[tid] = expf(rg);
            st.beta[tid] = rb;
        }
    };

    static_assert(kThreads % kBlockRows == 0, "a thread stays in its column of v");
    float s[ROWS][PIECES][4];
    auto put_out = [&](int64_t t, int r, float o) {
        if (!STORE && sub == 0 && row0 + 4 * r < a.headdim)
            io_traits<T>::store(static_cast<T *>(a.out) + ((b * a.seqlen + t) * a.heads + h) * a.headdim + row0 + 4 * r,
                                a.scale * o);
    };
    auto put_r = [&](int64_t t, int r, float res) {
        if (STORE && sub == 0 && row0 + 4 * r < a.headdim)
            a.r[((b * a.seqlen + t) * a.heads + h) * a.headdim + row0 + 4 * r] = res;
    };
    issue(0);
    small_loads(0);
    small_stores(0);
    get_rows<PIECES, VEC>(s, a.h0, bh, row0, a.headdim, sub, n);
    for (int64_t t0 = 0; t0 < a.seqlen; t0 += kTok) {
        issue(t0 + kTok);
        small_loads(t0 + kTok);
        cp_async_wait<1>();
        __syncthreads();
        if (STORE) {
            static_assert(kTok == kDeltaStep, "a stored state per stage");
            const int64_t marks = (a.seqlen + kTok - 1) / kTok;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int row = row0 + 4 * r;
                if (row < a.headdim)
                    put_row<PIECES, VEC>(a.marks + ((bh * marks + t0 / kTok) * a.headdim + row) * n, s[r], sub, n);
            }
        }
        TokenStage<T, PIECES, ROWS> &st = stages[(t0 / kTok) & 1];
        const int live = (int)(a.seqlen - t0 < kTok ? a.seqlen - t0 : kTok);
        {  // the pairs' products: 8 x 4 of them, four threads each
            const int pair = tid >> 4, which = (tid >> 2) & 3, from = tid & 3;
            const T *x = which == 3 ? st.k[2 * pair + 1] : st.k[2 * pair];
            const T *y = which == 0 ? st.k[2 * pair + 1] : st.q[2 * pair + (which > 1)];
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 2 * PIECES; ++i) {
                float xv[4], yv[4];
                io_traits<T>::load4_smem(x + 4 * (from + 4 * i), xv);
                io_traits<T>::load4_smem(y + 4 * (from + 4 * i), yv);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = fmaf(xv[e], yv[e], d[e]);
            }
            float sum = (d[0] + d[1]) + (d[2] + d[3]);
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            static_assert(kThreads == kTok / 2 * 16, "four threads a product");
            if (from == 0) (&st.pair[pair].x)[which] = sum;
        }
        __syncthreads();
        float k1[PIECES][4], k2[PIECES][4], q1[PIECES][4], q2[PIECES][4];
        auto row_of = [&](const T *x, float (&v)[PIECES][4]) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p) io_traits<T>::load4_smem(x + 4 * (sub + kLanes * p), v[p]);
        };
        row_of(st.k[0], k1);
        row_of(st.k[1], k2);
        row_of(st.q[0], q1);
        row_of(st.q[1], q2);
        // Two tokens at a time: the state's products with both tokens' k and q go
        // through one set of shuffles, and the second token's come from the first's,
        //   S1 x = a1 S x + u1 (k1 . x),  S2 = a1 a2 S + a2 u1 k1 + u2 k2.
        // (18 heads of 40 x 48: 170 ns a token; one at a time 245 ns.)
#pragma unroll 1
        for (int t = 0; t < live; t += 2) {
            const float2 dec = *reinterpret_cast<const float2 *>(&st.decay[t]), be = *reinterpret_cast<const float2 *>(&st.beta[t]);
            const float4 c = st.pair[t / 2];
            float sums[4 * ROWS], vv[2][ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                vv[0][r] = io_traits<T>::load_smem(&st.v[t][mine + 4 * r]);
                vv[1][r] = io_traits<T>::load_smem(&st.v[t + 1][mine + 4 * r]);
                sums[4 * r] = row_dot<PIECES>(s[r], k1);
                sums[4 * r + 1] = row_dot<PIECES>(s[r], k2);
                if (!STORE) {
                    sums[4 * r + 2] = row_dot<PIECES>(s[r], q1);
                    sums[4 * r + 3] = row_dot<PIECES>(s[r], q2);
                } else {
                    sums[4 * r + 2] = sums[4 * r + 3] = 0.f;
                }
            }
            const int next = t + 2 < live ? t + 2 : t;
            if (!STORE) {
                row_of(st.q[next], q1);
                row_of(st.q[next + 1], q2);
            }
            sum8<4 * ROWS>(sums);
            const float both = dec.x * dec.y;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float *d = sums + 4 * r;
                const float r1 = fmaf(-dec.x, d[0], vv[0][r]), u1 = be.x * r1;
                const float r2 = fmaf(-dec.y, fmaf(u1, c.x, dec.x * d[1]), vv[1][r]), u2 = be.y * r2;
                const float w1 = dec.y * u1;
#pragma unroll
                for (int p = 0; p < PIECES; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][p][e] = fmaf(u2, k2[p][e], fmaf(w1, k1[p][e], both * s[r][p][e]));
                put_r(t0 + t, r, r1);
                put_out(t0 + t, r, fmaf(u1, c.y, dec.x * d[2]));
                if (t + 1 < live) {
                    put_r(t0 + t + 1, r, r2);
                    put_out(t0 + t + 1, r, fmaf(u2, c.w, dec.y * fmaf(u1, c.z, dec.x * d[3])));
                }
            }
            row_of(st.k[next], k1);
            row_of(st.k[next + 1], k2);
        }
        small_stores(t0 + kTok);
        __syncthreads();
    }
    if (!a.state) return;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = row0 + 4 * r;
        if (row < a.headdim) put_row<PIECES, VEC>(a.state + (bh * a.headdim + row) * (int64_t)n, s[r], sub, n);
    }
}

bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T, int PIECES, bool VEC, bool STORE>
cudaError_t launch_pieces(const DeltaArgs &a, bool async, int sms, cudaStream_t st) {
    const int tiles = (a.headdim + kRowsPerBlock - 1) / kRowsPerBlock;
    const dim3 grid((unsigned)(a.batch * a.heads * tiles)), block(kWarps * 32);
    if (a.seqlen <= kFewTokens && !STORE) {
        delta_step_kernel<T, PIECES, VEC><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    }
    // One row set per warp where that still leaves SMs free: a warp's chain is shorter
    // (18 heads of 40 x 48, 301 tokens: 52 us, two sets 56 us), the work of a row larger.
    const int64_t small = a.batch * a.heads * ((a.headdim + kRowsPerBlock / 2 - 1) / (kRowsPerBlock / 2));
    auto tokens = [&](auto fast) {
        constexpr bool FAST = decltype(fast)::value;
        if (small <= sms) delta_tokens_kernel<T, PIECES, 1, FAST, STORE><<<(unsigned)small, block, 0, st>>>(a);
        else delta_tokens_kernel<T, PIECES, kRows, FAST, STORE><<<grid, block, 0, st>>>(a);
    };
    if (VEC && async) tokens(std::true_type());
    else tokens(std::false_type());
    return cudaGetLastError();
}

template <typename T, bool STORE>
cudaError_t launch_t(const DeltaArgs &a, int sms, cudaStream_t st) {
    const bool vec = a.dstate % 4 == 0 && aligned_to(a.q, 4 * sizeof(T)) && aligned_to(a.k, 4 * sizeof(T)) &&
                     aligned_to(a.h0, 16) && aligned_to(a.state, 16);
    const bool async = a.dstate * sizeof(T) % 16 == 0 && aligned_to(a.q, 16) && aligned_to(a.k, 16);
    if (a.dstate <= 32)
        return vec ? launch_pieces<T, 1, true, STORE>(a, async, sms, st) : launch_pieces<T, 1, false, STORE>(a, async, sms, st);
    if (a.dstate <= 64)
        return vec ? launch_pieces<T, 2, true, STORE>(a, async, sms, st) : launch_pieces<T, 2, false, STORE>(a, async, sms, st);
    if (a.dstate <= 96)
        return vec ? launch_pieces<T, 3, true, STORE>(a, async, sms, st) : launch_pieces<T, 3, false, STORE>(a, async, sms, st);
    return vec ? launch_pieces<T, 4, true, STORE>(a, async, sms, st) : launch_pieces<T, 4, false, STORE>(a, async, sms, st);
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool bf16, int sms, cudaStream_t st) {
    if (a.marks) return launch_t<float, true>(a, sms, st);
    return bf16 ? launch_t<__nv_bfloat16, false>(a, sms, st) : launch_t<float, false>(a, sms, st);
}

}  // namespace ssm
