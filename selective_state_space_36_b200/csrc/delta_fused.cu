// delta_fused.cu -- the chunked gated delta rule on the sm_100a tensor cores,
// one kernel (notation of delta_chunk.cuh).
//
// One CTA owns 128 state rows of a head (the columns of V) for the whole
// sequence and walks over its chunks of 64 tokens.  Everything is computed
// transposed, with the state rows as the 128 lanes of tensor memory: then the
// state, R and w u -- each an accumulator of one product and the left
// operand of the next -- never leave tensor memory, and the row-wise work is
// one thread per lane.  Per chunk, three tcgen05 products:
//   [X | O1]^T = S [K; Q]^T                       (128 x 128, K = dstate)
//   [Y | O2]^T = R^T [M; Pb - Pb M]^T             (128 x 128, K = 64),  R = V - gam X
//   S          = gam_C S + (w beta r)^T K         (128 x dstate, K = 64),  r = R - Y
//   out        = scale gam O1 + O2
// with M = N beta = I - (I + L)^-1, L = Abar beta, and Pb = P beta.  O2 reads R
// instead of r (Pb r = (Pb - Pb M) R), so the output needs no product behind r.
// Operands that are not bf16 already take two bf16 terms (state: 2 products
// instead of 1; R with M, Pb: 3).
//
// M and Pb - Pb M of the next chunk are made meanwhile by four warps of their
// own: [K; Q] K^T (tcgen05), the decays, then, on mma.sync, M: its 16 x 16 diagonal
// blocks by substitution, one column per thread, and from them twice as large
// blocks, 16 to 32 to 64, by M21 = (I - M22) L21 (I - M11) with products of
// two-term operands.  (Every factor is part of an inverse whose entries stay
// bounded; powers of L would not.)  A kernel of their own would have to write
// and read 64 KB per chunk and head, as much as q, k, v and out together.
//
// Warps: 0-7 row-wise work (two per lane quarter, each half of the columns),
// 8-11 the chunk matrices, 12 issues the products, 13 the TMA copies, 14 the
// decays.  They meet at mbarriers only; every wait is bounded and reports
// through the device status word.
#include "delta_chunk.cuh"
#include "scan_kernels.cuh"
#include "ssm_device.cuh"
#include "tma_maps.cuh"
#include "umma.cuh"

namespace ssm {
namespace delta {
namespace {

using namespace umma;

constexpr int kRowWarps = 8, kMatWarps = 4;
constexpr int kThreadsF = (kRowWarps + kMatWarps + 4) * 32;  // 13-15: products, copies, decays; one idle
// Registers per thread: 128 at launch, then by group of four warps
constexpr int kRowRegs = 152, kMatRegs = 168, kRestRegs = 40;
static_assert(2 * kRowRegs + kMatRegs + kRestRegs <= 4 * 128, "no more than the block was launched with");
constexpr uint32_t kHalfTile = kC * 128;  // 64 rows x 128 bytes
constexpr int kDLd = 36;                 // row stride of a 32 x 32 float32 block: 16-byte rows

// tensor memory columns
constexpr uint32_t kTX = 0, kTO1 = 64, kTY = 128, kTO2 = 192, kTS = 256, kTSh = 384, kTSl = 448;
// R (where X was) and w u (where Y was): tokens 32 wg .. 32 wg + 31 of
// both terms stay within the columns that their warps have read themselves
__host__ __device__ constexpr uint32_t operand_col(uint32_t base, int kstep, int term) {
    return base + 32 * (kstep >> 1) + 16 * term + 8 * (kstep & 1);
}

struct __align__(16) Dec {         // per chunk, float32
    float gam[kC], gs[kC], wb[kC];  // exp G, scale exp G, exp(G_C - G) beta
    float beta[kC], sbeta[kC];      // beta, scale beta
    // G in units of ln 2 as two floats: the difference of two such sums keeps the
    // digits that a difference of two floats loses, without float64's cost
    float ch[kC], cl[kC];
    float whole, pad[3];           // exp G_C
};

template <int NT>
struct FusedSmem {
    unsigned char kq[2][NT][2 * kHalfTile];  // per stage and 64 columns: K rows, then Q rows
    unsigned char v[2][2][kHalfTile];        // V, later the output
    unsigned char np[2][2][2 * kHalfTile];   // [M; Pb - Pb M]: high, low term
    unsigned char l[2][kHalfTile];           // L: high, low term
    float ld32[kC][kDLd];                    // L's 32 x 32 diagonal blocks
    Dec dec[2];
    // Barriers whose waiters may fall a chunk behind have one per stage, so that
    // a phase cannot be overtaken.
    uint64_t ld[2], cum[2], prep[2];         // copies landed; decays, chunk matrices ready
    uint64_t kqd, x, y, s[2];                // products complete ([K; Q] K^T first)
    uint64_t s_ready, r_ready, u_ready, o_ready[2];  // row-wise results written
    uint64_t kq_read;                        // [K; Q] K^T is in registers
    uint64_t fin;
    uint32_t tmem;
};

struct FusedArgs {
    const float *g, *beta, *h0;
    float *state;
    float scale;
    int64_t seqlen;
    int heads, rep, headdim, dstate, vtiles;
    int vec_state;  // h0 and state start 16-byte aligned
    unsigned int *status;
};

template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
// acc (16 x 8) += A (16 x 16) B (16 x 8), two terms each.
__device__ __forceinline__ void product(float (&acc)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                        const uint32_t (&bh)[2], const uint32_t (&bl)[2]) {
    mma(acc, ah, bh[0], bh[1]);
    mma(acc, al, bh[0], bh[1]);
    mma(acc, ah, bl[0], bl[1]);
}

// Eight columns (col ..) of M21 = (I - M22) L21 (I - M11), the block of 16 R rows
// at row r0 and columns from c0, into M (high, low term).
template <int R>
__device__ __forceinline__ void block_columns(unsigned char *mh, unsigned char *ml, unsigned char *lh,
                                              unsigned char *ll, int r0, int c0, int col, int lane) {
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    float acc[R][4];  // -(L21 - L21 M11) = -T, then -(T - M22 T)
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = r0 + 16 * m + g + 8 * half;
            const uint32_t h = *reinterpret_cast<const uint32_t *>(tile_at(lh, row, col + c2));
            const uint32_t l = *reinterpret_cast<const uint32_t *>(tile_at(ll, row, col + c2));
            acc[m][2 * half] = -(low_of(h) + low_of(l));
            acc[m][2 * half + 1] = -(high_of(h) + high_of(l));
        }
#pragma unroll
    for (int kk = 0; kk < R; ++kk) {
        uint32_t b[4];  // M11: both terms of its eight columns
        ldm4t(b, tile_at(lane < 16 ? mh : ml, c0 + 16 * kk + rf_row, col));
        const uint32_t bh[2] = {b[0], b[1]}, bl[2] = {b[2], b[3]};
#pragma unroll
        for (int m = 0; m < R; ++m) {
            uint32_t ah[4], al[4];
            ldm4(ah, tile_at(lh, r0 + 16 * m + rf_row, c0 + 16 * kk + rf_col));
            ldm4(al, tile_at(ll, r0 + 16 * m + rf_row, c0 + 16 * kk + rf_col));
            product(acc[m], ah, al, bh, bl);
        }
    }
    uint32_t bh[R][2], bl[R][2];  // T as a right operand
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t h, l;
            split(-acc[m][2 * half], -acc[m][2 * half + 1], h, l);
            bh[m][half] = transpose8(h);
            bl[m][half] = transpose8(l);
        }
#pragma unroll
    for (int m = 0; m < R; ++m) {
#pragma unroll
        for (int kk = 0; kk <= m; ++kk) {  // M22 is lower triangular
            uint32_t ah[4], al[4];
            ldm4(ah, tile_at(mh, r0 + 16 * m + rf_row, r0 + 16 * kk + rf_col));
            ldm4(al, tile_at(ml, r0 + 16 * m + rf_row, r0 + 16 * kk + rf_col));
            product(acc[m], ah, al, bh[kk], bl[kk]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t h, l;
            split(-acc[m][2 * half], -acc[m][2 * half + 1], h, l);
            const int row = r0 + 16 * m + g + 8 * half;
            *reinterpret_cast<uint32_t *>(tile_at(mh, row, col + c2)) = h;
            *reinterpret_cast<uint32_t *>(tile_at(ml, row, col + c2)) = l;
        }
    }
}

// A 16 x 16 block (two accumulators side by side) in both terms.
__device__ __forceinline__ void put_block(unsigned char *high, unsigned char *low, int row, int col,
                                          const float (&x)[4], const float (&y)[4], int lane) {
    uint32_t h[4], l[4];
    split(x[0], x[1], h[0], l[0]);
    split(x[2], x[3], h[1], l[1]);
    split(y[0], y[1], h[2], l[2]);
    split(y[2], y[3], h[3], l[3]);
    row += rows_first_row(lane);
    col += rows_first_col(lane);
    stm4(tile_at(high, row, col), h[0], h[1], h[2], h[3]);
    stm4(tile_at(low, row, col), l[0], l[1], l[2], l[3]);
}

// This thread's row of K K^T (warps 0, 1: L) or Q K^T (warps 2, 3: Pb): the 32
// columns from s0 in x become exp(G_t - G_s) beta_s x (beta: scaled for Pb) for s + strict <= t and
// zero above, and go to row `row` of two tiles in both terms.
__device__ __forceinline__ void decay_row(float (&x)[32], const Dec &dec, const float *beta, int strict, int t, int s0,
                                          unsigned char *high, unsigned char *low, int row) {
    const float2 th = make_float2(dec.ch[t], dec.ch[t]), tl = make_float2(dec.cl[t], dec.cl[t]);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 h = *reinterpret_cast<const float4 *>(&dec.ch[s0 + i]);
        const float4 l = *reinterpret_cast<const float4 *>(&dec.cl[s0 + i]);
        const float4 b = *reinterpret_cast<const float4 *>(&beta[s0 + i]);
        const float2 d0 = add2(sub2(th, make_float2(h.x, h.y)), sub2(tl, make_float2(l.x, l.y)));
        const float2 d1 = add2(sub2(th, make_float2(h.z, h.w)), sub2(tl, make_float2(l.z, l.w)));
        const float2 e0 = mul2(make_float2(ex2_approx(d0.x), ex2_approx(d0.y)), make_float2(b.x, b.y));
        const float2 e1 = mul2(make_float2(ex2_approx(d1.x), ex2_approx(d1.y)), make_float2(b.z, b.w));
        const int at = s0 + i + strict;
        x[i] = at <= t ? x[i] * e0.x : 0.f;
        x[i + 1] = at + 1 <= t ? x[i + 1] * e0.y : 0.f;
        x[i + 2] = at + 2 <= t ? x[i + 2] * e1.x : 0.f;
        x[i + 3] = at + 3 <= t ? x[i + 3] * e1.y : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split(x[8 * p + 2 * i], x[8 * p + 2 * i + 1], hi[i], lo[i]);
        const uint32_t at = sw128_offset(row, (s0 >> 3) + p);
        *reinterpret_cast<uint4 *>(high + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(low + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// The matrices of chunk c from [K; Q] K^T in tensor memory (kq: this warp's 32
// lanes); `taken` is called when it has been read.
template <int NT, typename F>
__device__ __forceinline__ void chunk_matrices(FusedSmem<NT> &sm, int c, int w, int lane, uint32_t kq,
                                               F taken) {
    const Dec &dec = sm.dec[c & 1];
    unsigned char *mh = sm.np[c & 1][0], *ml = sm.np[c & 1][1];
    {
        // rows 32 (w % 2) ...: the columns of the first half, and for the lower rows
        // those of the second
        const int t = 32 * (w & 1) + lane, strict = w < 2;
        unsigned char *high = strict ? sm.l[0] : mh, *low = strict ? sm.l[1] : ml;
        const int row = strict ? t : kC + t;
        float x[32], y[32];
        tmem_ld32(kq + 32 * (w & 1), x);  // the columns of the block on the diagonal
        tmem_ld32(kq, y);
        tmem_wait_ld();
        taken();
        // one copy of the code for both halves: the kernel's instructions have to
        // stay in the instruction cache (at 95 KB it ran at a third of its speed)
#pragma unroll 1
        for (int half = w & 1; half >= 0; --half) {
            decay_row(x, dec, strict ? dec.beta : dec.sbeta, strict, t, 32 * half, high, low, row);
            if (half == (w & 1) && strict) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4 *>(&sm.ld32[t][i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = y[i];
        }
    }
    mats_sync();  // L and Pb
    // the diagonal blocks of M, column lane % 16 from its top
    {
        const int o = 16 * w, oc = 16 * (w & 1), j = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s[2] = {sm.ld32[o + i][oc + j], 0.f};  // zero for i <= j
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&sm.ld32[o + i][oc + k]);
                s[0] = fmaf(-m.x, x[k], s[0]);
                if (k + 1 < i) s[1] = fmaf(-m.y, x[k + 1], s[1]);
                if (k + 2 < i) s[0] = fmaf(-m.z, x[k + 2], s[0]);
                if (k + 3 < i) s[1] = fmaf(-m.w, x[k + 3], s[1]);
            }
            x[i] = s[0] + s[1];
        }
        // lanes 0-15 write the high terms, the others the low ones
        unsigned char *dst = lane < 16 ? mh : ml;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float hi = __bfloat162float(__float2bfloat16_rn(x[i]));
            *tile_at(dst, o + i, o + j) = __float2bfloat16_rn(lane < 16 ? hi : x[i] - hi);
        }
    }
    mats_sync();  // the diagonal blocks
    // 16 to 32: warps 0, 1 the block at (16, 0), warps 2, 3 that at (48, 32)
    block_columns<1>(mh, ml, sm.l[0], sm.l[1], 32 * (w >> 1) + 16, 32 * (w >> 1), 32 * (w >> 1) + 8 * (w & 1), lane);
    mats_sync();  // the 32 x 32 blocks on the diagonal
    block_columns<2>(mh, ml, sm.l[0], sm.l[1], 32, 0, 8 * w, lane);
    mats_sync();  // M
    // Pb - Pb M, rows 16 w ...: blocks of 16 columns, in place (M is strictly
    // lower: a block changes itself and those before it).  The zero blocks above
    // the diagonal are not left out: the last rows need as long without them.
    const int rf_row = rows_first_row(lane), rf_col = rows_first_col(lane);
    float acc[kC / 8][4];
#pragma unroll
    for (int kk = 0; kk < kC / 16; ++kk) {
        uint32_t hi[4], lo[4];  // as accumulators: negated Pb
        ldm4(hi, tile_at(mh, kC + 16 * w + rf_row, 16 * kk + rf_col));
        ldm4(lo, tile_at(ml, kC + 16 * w + rf_row, 16 * kk + rf_col));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float(&x)[4] = acc[2 * kk + (i >> 1)];
            x[2 * (i & 1)] = -(low_of(hi[i]) + low_of(lo[i]));
            x[2 * (i & 1) + 1] = -(high_of(hi[i]) + high_of(lo[i]));
        }
#pragma unroll
        for (int jj = 0; jj <= kk; ++jj) {
            uint32_t f[4], fl[4];
            ldm4t(f, tile_at(mh, 16 * kk + rf_row, 16 * jj + rf_col));
            ldm4t(fl, tile_at(ml, 16 * kk + rf_row, 16 * jj + rf_col));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma(acc[2 * jj + i], hi, f[2 * i], f[2 * i + 1]);
                mma(acc[2 * jj + i], lo, f[2 * i], f[2 * i + 1]);
                mma(acc[2 * jj + i], hi, fl[2 * i], fl[2 * i + 1]);
            }
        }
    }
    __syncwarp();  // (a warp reads and writes only its own rows of Pb)
#pragma unroll
    for (int j = 0; j < kC / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = -acc[j][e];
#pragma unroll
    for (int jj = 0; jj < kC / 16; ++jj) put_block(mh, ml, kC + 16 * w, 16 * jj, acc[2 * jj], acc[2 * jj + 1], lane);
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
            mbar_init(&sm.cum[i], 1);
            mbar_init(&sm.prep[i], kMatWarps);
            mbar_init(&sm.s[i], 1);
            mbar_init(&sm.o_ready[i], kRowWarps);
        }
        mbar_init(&sm.kqd, 1);
        mbar_init(&sm.kq_read, kMatWarps);
        mbar_init(&sm.x, 1);
        mbar_init(&sm.y, 1);
        mbar_init(&sm.s_ready, kRowWarps);
        mbar_init(&sm.r_ready, kRowWarps);
        mbar_init(&sm.u_ready, kRowWarps);
        mbar_init(&sm.fin, 1);
        mbar_fence_init();
    }
    // the parts of [M; Pb - Pb M] above the diagonal are written here only
    for (int i = tid; i < (int)sizeof(sm.np) / 16; i += kThreadsF)
        reinterpret_cast<uint4 *>(sm.np)[i] = make_uint4(0, 0, 0, 0);
    if (warp == 0) tmem_alloc(&sm.tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = sm.tmem;
    auto wait = [&](uint64_t *bar, uint32_t par) { return __all_sync(0xffffffffu, mbar_wait_2s(bar, par & 1u)) != 0; };
    bool ok = true;  // false: a wait of this warp ran out
    auto signal = [&](uint64_t *bar) {  // one arrival per warp, after the warp's writes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp >= kRowWarps + kMatWarps) {
      fewer_regs<kRestRegs>();
      if (warp == kRowWarps + kMatWarps) {
        // ------------------------------------------------ the products
        const uint32_t el = elect_one();
        constexpr uint32_t id_k = idesc_bf16(128, 128, kMajorK, kMajorK);
        constexpr uint32_t id_kq = idesc_bf16(128, 64, kMajorK, kMajorK);
        constexpr uint32_t id_s = idesc_bf16(128, 64 * NT, kMajorK, kMajorMN);
        // [K; Q] K^T of chunk c where O2 will be: the rows' read of the last O2 is
        // behind s_ready, the next M2 waits for kq_read
        auto kq_product = [&](int c) {
            if (!(ok = wait(&sm.ld[c & 1], c >> 1))) return;
            fence_after_sync();
            const uint64_t d = desc_sw128(smem_u32(sm.kq[c & 1][0]), 16, 1024);
#pragma unroll 1
            for (int k = 0; k < 4 * NT; ++k) {
                const uint64_t at = d + (((k / 4) * 2 * kHalfTile + (k % 4) * 32) >> 4);
                mma_bf16_if(el, tm + kTO2, at, at, id_kq, k > 0);
            }
            mma_commit_if(el, &sm.kqd);
        };
        // (step -1: the first chunk's [K; Q] K^T only)
        for (int c = -1; ok && c < nch; ++c) {
            const int st = c & 1;
            if (c >= 0) {
                if (!(ok = wait(&sm.s_ready, c))) break;
                fence_after_sync();
                const uint64_t dkq = desc_sw128(smem_u32(sm.kq[st][0]), 16, 1024);
#pragma unroll 1
                for (int k = 0; k < 8 * NT; ++k) {  // high terms, then low ones
                    const int kk = k & (4 * NT - 1);
                    mma_bf16_ts_if(el, tm + kTX, tm + (k < 4 * NT ? kTSh : kTSl) + 8 * kk,
                                   dkq + (((kk / 4) * 2 * kHalfTile + (kk % 4) * 32) >> 4), id_k, k > 0);
                }
                mma_commit_if(el, &sm.x);
                // (chunk 0's product has to be read before chunk 1's replaces it)
                if (c == 0 && !(ok = wait(&sm.kq_read, 0))) break;
            }
            if (c + 1 < nch) kq_product(c + 1);
            if (c < 0) continue;
            if (!ok || !(ok = wait(&sm.prep[st], c >> 1)) || !(ok = wait(&sm.r_ready, c))) break;
            if (c + 1 < nch && !(ok = wait(&sm.kq_read, c + 1))) break;
            fence_after_sync();
            const uint64_t dnh = desc_sw128(smem_u32(sm.np[st][0]), 16, 1024);
            const uint64_t dnl = desc_sw128(smem_u32(sm.np[st][1]), 16, 1024);
#pragma unroll 1
            for (int k = 0; k < 12; ++k) {  // R high with high terms, R low with high, R high with low
                const int kk = k & 3, term = k >> 2;
                mma_bf16_ts_if(el, tm + kTY, tm + operand_col(kTX, kk, term == 1),
                               (term == 2 ? dnl : dnh) + ((kk * 32) >> 4), id_k, k > 0);
            }
            mma_commit_if(el, &sm.y);
            if (!(ok = wait(&sm.u_ready, c))) break;
            fence_after_sync();
            // K as the right operand with tokens as the summed index: rows of 64
            // state columns, the second 64 in the next tile
            const uint64_t dk = desc_sw128(smem_u32(sm.kq[st][0]), 2 * kHalfTile, 1024);
#pragma unroll 1
            for (int k = 0; k < 8; ++k)
                mma_bf16_ts_if(el, tm + kTS, tm + operand_col(kTY, k & 3, k >> 2), dk + (((k & 3) * 2048) >> 4), id_s, true);
            mma_commit_if(el, &sm.s[st]);
        }
        mma_commit_if(el, &sm.fin);  // whatever was issued completes before tensor memory goes away
        (void)mbar_wait_2s(&sm.fin, 0u);
        __syncwarp();
      } else if (warp == kRowWarps + kMatWarps + 1) {
        // -------------------------------------------------- the copies
        const uint32_t el = elect_one();
        int issued[2] = {0, 0};
        // step c: chunk c's output leaves, chunk c + 2 comes (two steps ahead of the first chunk)
        for (int c = -2; c < nch; ++c) {
            const int st = c & 1;
            if (c >= 0) {
                if (!(ok = wait(&sm.o_ready[st], c >> 1))) break;
                if (el) {
#pragma unroll 1
                    for (int i = 0; i < halves; ++i)
                        tma_store_3d(&mapO, h * a.headdim + v0 + 64 * i, c * kC, (int32_t)b, sm.v[st][i]);
                    tma_store_commit();
                    tma_store_wait_read<0>();
                }
                __syncwarp();
            }
            if (c + 2 >= nch) continue;
            if (c >= 0 && !(ok = wait(&sm.s[st], c >> 1))) break;  // K and Q are read
            if (el) {
                mbar_expect_tx(&sm.ld[st], (uint32_t)(2 * NT + halves) * kHalfTile);
                const int32_t t0 = (c + 2) * kC;
#pragma unroll 1
                for (int i = 0; i < NT; ++i) {
                    tma_load_3d(sm.kq[st][i], &mapK, gr * a.dstate + 64 * i, t0, (int32_t)b, &sm.ld[st]);
                    tma_load_3d(sm.kq[st][i] + kHalfTile, &mapQ, gr * a.dstate + 64 * i, t0, (int32_t)b, &sm.ld[st]);
                }
#pragma unroll 1
                for (int i = 0; i < halves; ++i)
                    tma_load_3d(sm.v[st][i], &mapV, h * a.headdim + v0 + 64 * i, t0, (int32_t)b, &sm.ld[st]);
            }
            if (st) ++issued[1]; else ++issued[0];
        }
        if (el) tma_store_wait_all<0>();
        if (issued[0] > 0) (void)mbar_wait_2s(&sm.ld[0], (uint32_t)(issued[0] - 1) & 1u);
        if (issued[1] > 0) (void)mbar_wait_2s(&sm.ld[1], (uint32_t)(issued[1] - 1) & 1u);
        __syncwarp();
      } else if (warp == kRowWarps + kMatWarps + 2) {
        // -------------------------------------------------- the decays
        const float *g = a.g + b * a.seqlen * a.heads + h, *be = a.beta + b * a.seqlen * a.heads + h;
        float gv[2], bv[2];
        auto fetch = [&](int c) {  // this lane's two tokens; none behind the end
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t t = (int64_t)c * kC + 2 * lane + i;
                gv[i] = t < a.seqlen ? __ldg(g + t * a.heads) : 0.f;
                bv[i] = t < a.seqlen ? __ldg(be + t * a.heads) : 0.f;
            }
        };
        fetch(0);
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1;
            Dec &dec = sm.dec[st];
            // below -1e4 a decay is zero in float32 either way; the clamp keeps
            // differences of two such sums finite
            constexpr double kLog2 = 1.4426950408889634;
            const double d0 = kLog2 * fmax((double)gv[0], -1e4), d1 = kLog2 * fmax((double)gv[1], -1e4);
            const float be2[2] = {bv[0], bv[1]};
            double sum = d0 + d1;
            if (c + 1 < nch) fetch(c + 1);
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double end = __shfl_sync(0xffffffffu, sum, 31);
            // chunk c - 2 is done with its decays and matrices
            if (c >= 2 && !(ok = wait(&sm.o_ready[st], (c - 2) >> 1))) break;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const double cum = i ? sum : sum - d1;
                const float gam = ex2_approx((float)cum), be = i ? be2[1] : be2[0];
                dec.ch[t] = (float)cum;
                dec.cl[t] = (float)(cum - (double)(float)cum);
                dec.gam[t] = gam;
                dec.gs[t] = a.scale * gam;
                dec.beta[t] = be;
                dec.sbeta[t] = a.scale * be;
                dec.wb[t] = ex2_approx((float)(end - cum)) * be;
            }
            if (lane == 31) dec.whole = ex2_approx((float)end);
            signal(&sm.cum[st]);
        }
      }
    } else if (warp >= kRowWarps) {
        // ------------------------------------------- the chunk matrices
        more_regs<kMatRegs>();
        const int w = warp - kRowWarps;
        for (int c = 0; c < nch; ++c) {
            const int st = c & 1;
            // (cum comes after chunk c - 2 is done with its matrices)
            ok = wait(&sm.cum[st], c >> 1) && wait(&sm.kqd, c);
            if (!mats_all(ok)) break;
            fence_after_sync();
            chunk_matrices<NT>(sm, c, w, lane, tm + kTO2 + ((uint32_t)(32 * w) << 16), [&] {
                fence_before_sync();
                signal(&sm.kq_read);
            });
            fence_proxy_async();
            signal(&sm.prep[st]);
        }
    } else {
        // --------------------------------------------- the row-wise work
        more_regs<kRowRegs>();
        const int quad = warp & 3, wg = warp >> 2, r = 32 * quad + lane;
        const bool active = 32 * quad < 64 * halves;  // the warp's lanes hold rows of the state
        const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
        const int64_t row = bh * a.headdim + v0 + r;
        const int vp = (r & 63) >> 3, vo = (r & 7) * 2;  // this row's place in a row of the V tile
        // the start state, where the first chunk's "last product" would have left it
        if (active) {
#pragma unroll 1
            for (int p = 0; p < NT; ++p) {
                const int col = 32 * (NT * wg + p);
                uint32_t s[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = 0;
                if (a.h0) {
                    const float *src = a.h0 + row * a.dstate + col;
                    if (a.vec_state) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(src + i);
                            s[i] = __float_as_uint(x.x); s[i + 1] = __float_as_uint(x.y);
                            s[i + 2] = __float_as_uint(x.z); s[i + 3] = __float_as_uint(x.w);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(src[i]);
                    }
                }
                tmem_st32(tl + kTS + col, s);
            }
            tmem_wait_st();
        }
        uint32_t ov[16];  // the last chunk's output values, packed
        // chunk c's state is there when chunk c - 1's last product is done; the
        // step behind the last chunk only stores the state and the output
        for (int c = 0; c <= nch; ++c) {
            const int st = c & 1;
            const Dec &dec = sm.dec[st];
            if (c < nch && !(ok = wait(&sm.cum[st], c >> 1))) break;
            if (c > 0 && !(ok = wait(&sm.s[st ^ 1], (c - 1) >> 1))) break;
            fence_after_sync();
            if (active) {
#pragma unroll 1
                for (int p = 0; p < NT; ++p) {
                    const int col = 32 * (NT * wg + p);
                    float s[32];
                    tmem_ld32(tl + kTS + col, s);
                    tmem_wait_ld();
                    if (c < nch) {
                        put_state(tl, col, s, dec.whole);
                    } else if (a.state) {
                        float *dst = a.state + row * a.dstate + col;
                        if (a.vec_state) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4 *>(dst + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) dst[i] = s[i];
                        }
                    }
                }
                tmem_wait_st();
            }
            fence_before_sync();
            if (c < nch) signal(&sm.s_ready);
            // while the first product runs: the last chunk's output over its V
            if (c > 0) {
                if (active) {
                    unsigned char *vt = sm.v[st ^ 1][r >> 6];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int t = 32 * wg + 2 * i;
                        *reinterpret_cast<unsigned short *>(vt + sw128_offset(t, vp) + vo) = (unsigned short)(ov[i] & 0xffffu);
                        *reinterpret_cast<unsigned short *>(vt + sw128_offset(t + 1, vp) + vo) = (unsigned short)(ov[i] >> 16);
                    }
                }
                fence_proxy_async();
                signal(&sm.o_ready[st ^ 1]);
            }
            if (c == nch) break;
            // this row's 32 values of V, R = V - gam X, and R as an operand
            float res[32];
            if (!(ok = wait(&sm.ld[st], c >> 1))) break;
            if (active) {
                const unsigned char *vt = sm.v[st][r >> 6];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const unsigned short u =
                        *reinterpret_cast<const unsigned short *>(vt + sw128_offset(32 * wg + i, vp) + vo);
                    res[i] = __uint_as_float((uint32_t)u << 16);
                }
            }
            if (!(ok = wait(&sm.x, c))) break;
            fence_after_sync();
            if (active) {
                float x[32];
                tmem_ld32(tl + kTX + 32 * wg, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g4 = *reinterpret_cast<const float4 *>(&dec.gam[32 * wg + i]);
                    res[i] = fmaf(-g4.x, x[i], res[i]);
                    res[i + 1] = fmaf(-g4.y, x[i + 1], res[i + 1]);
                    res[i + 2] = fmaf(-g4.z, x[i + 2], res[i + 2]);
                    res[i + 3] = fmaf(-g4.w, x[i + 3], res[i + 3]);
                }
                put_terms(tl + kTX + 32 * wg, tl + kTX + 32 * wg + 16, res);
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
            // the output's values, while the state's product runs
            if (active) {
                float o1[32], o2[32];
                tmem_ld32(tl + kTO1 + 32 * wg, o1);
                tmem_ld32(tl + kTO2 + 32 * wg, o2);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g4 = *reinterpret_cast<const float4 *>(&dec.gs[32 * wg + i]);
                    ov[i / 2] = pack(fmaf(g4.x, o1[i], o2[i]), fmaf(g4.y, o1[i + 1], o2[i + 1]));
                    ov[i / 2 + 1] = pack(fmaf(g4.z, o1[i + 2], o2[i + 2]), fmaf(g4.w, o1[i + 3], o2[i + 3]));
                }
            }
        }
    }
    if (!ok && lane == 0) atomicOr(a.status, 4u);
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
    f.vec_state = aligned16(a.h0) && aligned16(a.state);
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
