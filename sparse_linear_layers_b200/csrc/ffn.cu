// The gated feed-forward block on prepared ternary weights:
//
//   g[t, f] = acc_g * scale_g[f] / s_t,  u[t, f] = acc_u * scale_u[f] / s_t,  h = act(g) * u
//
// with acc = x_q . W_t^T the integer products of the Sparse-BitNet Guide's
// linear-evaluation equation ("Mathematical Formulation of Sparse-BitLinear")
// for the gate and the up matrix, act SiLU (g * sigmoid(g)) or the squared
// ReLU, and its straight-through backward (the Guide's "Training Stability &
// The Straight-Through Estimator"):
//
//   dg = dh * u * act'(g),  du = dh * act(g)
//   dX = (dg * scale_g) . W_g + (du * scale_u) . W_u
//   dW_g = dg^T . (x_q / s),  dW_u = du^T . (x_q / s)
//
// Forward, up to 16 tokens: ffn_decode_kernel streams the 2-bit codes of both
// matrices once (bound by launch latency, then HBM).  A 16-row MMA tile holds
// 8 rows of each matrix, so one thread ends with g and u of the same element.
//
// Forward, more tokens: ffn_pair_kernel, the 2-SM int8 tensor-core GEMM with
// a 256-token x (128 gate + 128 up)-row tile.  CTA rank 0 expands the gate
// rows, rank 1 the up rows; both hold, for their 128 tokens, g in TMEM columns
// 0-127 and u in columns 128-255, and the epilogue multiplies them.  Neither g
// nor u is written.  Bound by the tensor cores at large K; at K = 896 by the
// epilogue's instructions.
//
// Backward: nothing is kept from the forward but x; the same kernel computes
// g and u again and its epilogue writes v = (dg | du) * scale / s_t in fp32 and
// each token's largest |v| (atomic maximum: no order to depend on).  Both
// gradients are then products of v with exact factors:
//   dX[t] = s_t * sum_f v[t, f] * W_t[f],  dW[f] = (1 / scale[f]) * sum_t v[t, f] * x_q[t].
// ffn_operands_kernel splits v, scaled by a power of two 2^-er[t] that brings
// the token's largest value to [2^14, 2^15), into two fp16 parts (11 + 11
// significant bits; what they drop is at most 2^-22 of v plus 2^-39 of the
// token's largest |v|), writes the codes as fp16, and x_q * 2^(er[t] - max er + 8) as fp16,
// normal numbers down to er = max er - 22.  Tokens below that (their largest |v| under
// 2^-22 of all tokens' largest) would be subnormal, whose products the tensor cores align
// as if they were larger (a hidden unit that only such tokens reach: off by 2^-17 at 2^-30),
// then lose bits of x_q, then all of it.  They are left out of dW's product and
// counted, and ffn_far_kernel adds their terms in fp32.  Two products of those in one launch (gemm_f16.cuh,
// fp16 operands, both parts summed, segments of 4 k-blocks promoted to
// round-to-nearest sums) give dX and dW: at 4096 x 2048 -> 7168 0.57 ms, the tensor
// pipe 95% busy (0.60 as two launches).  Two parts instead of three bf16 ones
// save a third of the tensor work that bounds this.
#include <cuda.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "gemm_f16.cuh"
#include "sbl_common.cuh"
#include "tc_util.cuh"

namespace sbl {

constexpr int kLayoutPairsFfn = 1;  // launch_quant's pairing order
cudaError_t launch_quant(const uint16_t* x, long long T, long long K, int8_t* xq, float* s_tok, int layout,
                         unsigned* status, cudaStream_t stream, void* zero16, long long nzero16);

namespace {

constexpr int kActSilu = 0;

__device__ __forceinline__ float2 exp_neg2(float2 g) {  // exp(-g)
    const float2 e = mul2(g, both(-1.4426950408889634f));
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
}
__device__ __forceinline__ float2 rcp2(float2 a) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(a.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(a.y));
    return r;
}

// act(g) * u, in this order: g * u may pass fp32's range where act(g) * u does not.
// A sigmoid below 2^-126 comes out as 0.
template <int ACT>
__device__ __forceinline__ float2 act_times(float2 g, float2 u) {
    if (ACT == kActSilu) return mul2(mul2(g, rcp2(add2(exp_neg2(g), both(1.0f)))), u);
    const float2 r = make_float2(fmaxf(g.x, 0.0f), fmaxf(g.y, 0.0f));
    return mul2(mul2(r, r), u);
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void act_both(float2 g, float2& a, float2& da) {
    if (ACT == kActSilu) {
        const float2 s = rcp2(add2(exp_neg2(g), both(1.0f)));
        a = mul2(g, s);
        da = fma2(a, fma2(s, both(-1.0f), both(1.0f)), s);  // s + g s (1 - s)
    } else {
        const float2 r = make_float2(fmaxf(g.x, 0.0f), fmaxf(g.y, 0.0f));
        a = mul2(r, r);
        da = add2(r, r);
    }
}

// acc * scale * inv_s of two integer sums
__device__ __forceinline__ float2 dequant2(uint32_t a0, uint32_t a1, float2 scale, float2 inv_s) {
    return mul2(mul2(make_float2(static_cast<float>(static_cast<int>(a0)), static_cast<float>(static_cast<int>(a1))), scale),
                inv_s);
}

// ---------------------------------------------------------------- a few tokens
namespace fd {
constexpr int MAX_TOKENS = 16;
// Up to 8 tokens: blocks of 8 warps, four to an SM; more: 16 warps, two.
constexpr int warps(int nt) { return nt == 1 ? 8 : 16; }
constexpr int SM_WARPS = 32;
__host__ __device__ inline int pad64(int K) { return (K + 63) / 64 * 64; }
// one token's activations: 64 mod 128 bytes apart, so two tokens of a
// quarter-warp read disjoint banks
__host__ __device__ inline int stride(int K) { return pad64(K) % 128 == 64 ? pad64(K) : pad64(K) + 64; }
inline size_t smem_bytes(int K, int tokens) {
    return static_cast<size_t>(tokens) * stride(K) + static_cast<size_t>(warps(tokens > 8 ? 2 : 1)) * 32 * 4 * (tokens > 8 ? 2 : 1) * 4;
}
}  // namespace fd

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// CW code words of a row from word w0 on, zeros past the row's end.
template <int CW>
__device__ __forceinline__ void load_codes(const uint8_t* row, int w0, int words, bool ok, uint32_t (&w)[CW]) {
    if (!ok || w0 >= words) {  // CW > 1 only where CW divides the row's words
#pragma unroll
        for (int i = 0; i < CW; ++i) w[i] = 0u;
        return;
    }
    const uint8_t* p = row + 4 * static_cast<size_t>(w0);
    if constexpr (CW == 4) {
        const uint4 v = ldg_stream(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (CW == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const unsigned int*>(p));
    }
}

// A warp owns 8 rows f of both matrices and a slice of their chunks (64 * CW
// weights); KS warps of a block share a tile and add their int32 partials in
// shared memory.  NT: tiles of 8 tokens.
template <int NT, int CW, int ACT>
__global__ void __launch_bounds__(fd::warps(NT) * 32, fd::SM_WARPS / fd::warps(NT))
    ffn_decode_kernel(const uint8_t* __restrict__ pg, const float* __restrict__ scale_g, const uint8_t* __restrict__ pu,
                      const float* __restrict__ scale_u, int F, int K, const uint16_t* __restrict__ x, int t0, int TP,
                      int KS, void* __restrict__ h, int h_bf16, unsigned* status) {
    constexpr int WARPS = fd::warps(NT);
    extern __shared__ __align__(16) uint8_t fd_smem[];
    __shared__ uint32_t red_max[WARPS];
    __shared__ float s_sh[fd::MAX_TOKENS];
    asm volatile("griddepcontrol.launch_dependents;");
    const int S = fd::stride(K);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tg = lane & 3;
    const int words = K >> 4;
    const int C = fd::pad64(K) / (64 * CW);
    const int ks = warp % KS;
    const int f = (blockIdx.x * (WARPS / KS) + warp / KS) * 8 + gq;
    const bool ok = f < F;
    const size_t rowb = static_cast<size_t>(K) >> 2;
    const uint8_t* const rg = pg + static_cast<size_t>(ok ? f : 0) * rowb;
    const uint8_t* const ru = pu + static_cast<size_t>(ok ? f : 0) * rowb;
    const int nck = ks < C ? (C - ks + KS - 1) / KS : 0;
    auto word0 = [&](int j) { return ((ks + j * KS) * 4 + tg) * CW; };  // first code word of this thread's chunk j

    // before the dependency wait: pull this warp's weights into L2
    for (int j = 0; j < nck; ++j)
        if (ok && word0(j) < words) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rg + 4 * static_cast<size_t>(word0(j))));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(ru + 4 * static_cast<size_t>(word0(j))));
        }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    constexpr int NB = CW == 4 ? 2 : 4;  // chunks loaded together
    uint32_t wg[NB][CW], wu[NB][CW];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        load_codes<CW>(rg, word0(b), words, ok && b < nck, wg[b]);
        load_codes<CW>(ru, word0(b), words, ok && b < nck, wu[b]);
    }
    const float sg = ok ? __ldg(scale_g + f) : 0.f, su = ok ? __ldg(scale_u + f) : 0.f;

    // quantise the pass's TP tokens, 16 / TP warps each, into the slots that
    // the B fragments are read from
    auto pos = [](int blk) {
        const int c = blk / (4 * CW), l = blk % (4 * CW);
        return c * 4 * CW + (l % CW) * 4 + l / CW;
    };
    {
        const int wpt = WARPS / TP;
        const int qt = warp / wpt;
        const bool qw = qt < TP;
        const int qj = (warp - qt * wpt) * 32 + lane, nthr = wpt * 32;
        const uint4* const xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t0 + (qw ? qt : 0)) * K);
        constexpr int XB = 2;  // 16-element blocks kept in registers
        uint4 xa[XB][2];
        uint32_t mx = 0;
        if (qw) {
#pragma unroll
            for (int i = 0; i < XB; ++i) {
                const int b = qj + i * nthr;
                if (b < words) {
                    xa[i][0] = ldg_nc(xr + 2 * b);
                    xa[i][1] = ldg_nc(xr + 2 * b + 1);
                    mx = absmax8(xa[i][1], absmax8(xa[i][0], mx));
                }
            }
            for (int b = qj + XB * nthr; b < words; b += nthr)
                mx = absmax8(ldg_nc(xr + 2 * b + 1), absmax8(ldg_nc(xr + 2 * b), mx));
        }
        mx = __reduce_max_sync(0xFFFFFFFFu, mx);
        if (lane == 0) red_max[warp] = mx;
        __syncthreads();
        if (threadIdx.x < TP) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                if (w / wpt == static_cast<int>(threadIdx.x)) m = max(m, red_max[w]);
            if (m >= 0x7F80u && blockIdx.x == 0) raise_status(status, kStatusNonfinite);
            s_sh[threadIdx.x] = __fdiv_rn(127.0f, fmaxf(__uint_as_float(m << 16), 1e-5f));
        }
        __syncthreads();
        if (qw) {
            const float st = s_sh[qt];
            uint4* const xt = reinterpret_cast<uint4*>(fd_smem + static_cast<size_t>(qt) * S);
#pragma unroll
            for (int i = 0; i < XB; ++i) {
                const int b = qj + i * nthr;
                if (b < words) xt[pos(b)] = quant_block16_pairs(xa[i][0], xa[i][1], st);
            }
            for (int b = qj + XB * nthr; b < words; b += nthr)
                xt[pos(b)] = quant_block16_pairs(ldg_nc(xr + 2 * b), ldg_nc(xr + 2 * b + 1), st);
        }
        __syncthreads();
    }

    int acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[nt][r] = 0;
    for (int j0 = 0; j0 < nck; j0 += NB) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (j0 + b >= nck) break;
            const int c = ks + (j0 + b) * KS;
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                uint32_t eg[4], eu[4];
                expand_pairs(wg[b][i], eg);
                expand_pairs(wu[b][i], eu);
                // slots past the row's end hold anything: their codes are zero
                const int unit = c * 4 * CW + i * 4 + tg;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int tok = nt * 8 + gq;
                    uint4 xv = make_uint4(0u, 0u, 0u, 0u);
                    if (tok < TP) xv = reinterpret_cast<const uint4*>(fd_smem + static_cast<size_t>(tok) * S)[unit];
                    mma_s8(acc[nt], eg[0], eu[0], eg[1], eu[1], xv.x, xv.y);
                    mma_s8(acc[nt], eg[2], eu[2], eg[3], eu[3], xv.z, xv.w);
                }
            }
        }
        if (j0 + NB < nck) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int j = j0 + NB + b;
                load_codes<CW>(rg, word0(j), words, ok && j < nck, wg[b]);
                load_codes<CW>(ru, word0(j), words, ok && j < nck, wu[b]);
            }
        }
    }
    if (KS > 1) {
        int* const red = reinterpret_cast<int*>(fd_smem + static_cast<size_t>(TP) * S);
        if (ks != 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) red[(warp * 4 * NT + nt * 4 + r) * 32 + lane] = acc[nt][r];
        }
        __syncthreads();
        if (ks == 0) {
            for (int k2 = 1; k2 < KS; ++k2)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[nt][r] += red[((warp + k2) * 4 * NT + nt * 4 + r) * 32 + lane];
        }
    }
    if (ks != 0 || !ok) return;
    // this thread: row f of both matrices, tokens 2 tg and 2 tg + 1 of each tile of 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = nt * 8 + 2 * tg + e;
            if (tok >= TP) continue;
            const float inv_s = __frcp_rn(s_sh[tok]);
            const float g = __fmul_rn(__fmul_rn(static_cast<float>(acc[nt][e]), sg), inv_s);
            const float u = __fmul_rn(__fmul_rn(static_cast<float>(acc[nt][2 + e]), su), inv_s);
            const float v = act_times<ACT>(both(g), both(u)).x;
            const size_t at = static_cast<size_t>(t0 + tok) * F + f;
            if (h_bf16) reinterpret_cast<__nv_bfloat16*>(h)[at] = __float2bfloat16_rn(v);
            else reinterpret_cast<float*>(h)[at] = v;
        }
    }
}

// ---------------------------------------------------------------- many tokens
namespace fp {
constexpr int BM = 128;              // tokens per CTA (pair: 256)
constexpr int BF = 128;              // hidden units per tile
constexpr int BN = 2 * BF;           // accumulator columns: gate, then up
constexpr int BK = 128;              // k per stage (bytes of int8)
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BF * BK;
constexpr int P_BYTES = BF * BK / 4;
constexpr int EPI_WARPS = 8;
constexpr int DEC_WARPS = BF / 32;
constexpr int WARP_TMA = EPI_WARPS + DEC_WARPS;
constexpr int WARP_MMA = WARP_TMA + 1;
constexpr int THREADS = (WARP_MMA + 1) * 32;
constexpr int BOX = 32 * 128;
constexpr int stages(bool bwd) { return bwd ? 4 : 5; }
constexpr int boxes(bool bwd) { return bwd ? 2 : 1; }
}  // namespace fp

template <bool BWD>
struct FfnSmem {
    uint8_t a[fp::stages(BWD)][fp::A_BYTES];  // 1024-byte aligned tiles
    uint8_t b[fp::stages(BWD)][fp::B_BYTES];
    uint8_t box[fp::EPI_WARPS][fp::boxes(BWD)][fp::BOX];
    uint8_t p[fp::stages(BWD)][fp::P_BYTES];
    alignas(16) float scale[fp::EPI_WARPS][2][fp::BF / 2];
    uint64_t full_a[fp::stages(BWD)];         // used in the even CTA
    uint64_t full_c[fp::stages(BWD)];
    uint64_t full_dec[fp::stages(BWD)];       // used in the even CTA
    uint64_t empty[fp::stages(BWD)];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];                   // used in the even CTA
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
template <bool BWD>
constexpr size_t ffn_smem_bytes() {
    return sizeof(FfnSmem<BWD>) + 1024;
}
static_assert(ffn_smem_bytes<false>() <= 232448 && ffn_smem_bytes<true>() <= 232448, "feed-forward tile does not fit");

// 16 bytes (unit c) of this lane's row in a 32-row x 128-byte staging box, 128B swizzle.
__device__ __forceinline__ void box_put(uint8_t* box, int lane, int c, uint32_t w0, uint32_t w1, uint32_t w2,
                                        uint32_t w3) {
    const uint32_t a = smem_u32(box + lane * 128 + ((c ^ (lane & 7)) << 4));
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w0), "r"(w1), "r"(w2), "r"(w3) : "memory");
}
__device__ __forceinline__ void box_wait(int lane) {  // the stores sent so far have read their boxes
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
}

struct FfnParams {
    CUtensorMap x, wg, wu;     // int8 activations [T, K]; 2-bit codes [F, K / 4]
    CUtensorMap out;           // h [T, F] (forward, when out_tma), v [T, 2 Fp] (backward)
    const float* scale_g;
    const float* scale_u;
    const float* s_tok;
    void* h;                   // forward
    const float* dh;           // backward
    unsigned* row_max;         // backward: [T] bits of the largest |v| of a token
    unsigned* all_max;         // backward: of all tokens
    int T, K, F, Fp;
    int h_bf16, out_tma;
};

template <bool BWD, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(fp::THREADS, 1)
    ffn_pair_kernel(const __grid_constant__ FfnParams q, unsigned* status) {
    constexpr int STAGES = fp::stages(BWD);
    extern __shared__ uint8_t smem_raw[];
    auto* sm = reinterpret_cast<FfnSmem<BWD>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int* abort_flag = &sm->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int T = q.T, F = q.F;
    const int MT = (T + 2 * fp::BM - 1) / (2 * fp::BM), NT = (F + fp::BF - 1) / fp::BF;
    const int tiles = MT * NT;
    const int KB = (q.K + fp::BK - 1) / fp::BK;

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 32) {
        prefetch_tmap(&q.x);
        prefetch_tmap(rank ? &q.wu : &q.wg);
        prefetch_tmap(&q.out);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm->full_a[s], 1);
            mbar_init(&sm->full_c[s], 1);
            mbar_init(&sm->full_dec[s], 2 * fp::DEC_WARPS);
            mbar_init(&sm->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->tmem_full[b], 1);
            mbar_init(&sm->tmem_empty[b], 2 * fp::EPI_WARPS);
        }
        mbar_init(&sm->mma_done, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == fp::WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                     "r"(2 * fp::BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = sm->tmem_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    auto give_up = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            raise_status(status, kStatusTimeout);
        }
    };
    auto arrive_leader = [&](uint64_t* bar) {
        if (leader) mbar_arrive(bar);
        else mbar_arrive_cluster(map_to_cta(smem_u32(bar), 0));
    };

    if (warp < fp::EPI_WARPS) {
        // ------------------------------------------------------------ epilogue
        // Warp w: tokens 32 (w % 4) .. + 31 of the CTA's half, hidden units
        // 64 (w / 4) .. + 63 of the tile, in two slices of 32.
        const int qd = warp & 3, half = warp >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(qd * 32) << 16;
        float* const sc_g = sm->scale[warp][0];
        float* const sc_u = sm->scale[warp][1];
        uint8_t* const box = sm->box[warp][0];
        int tc = 0;
        for (int tile = pair; tile < tiles; tile += npairs, ++tc) {
            const int mt = tile / NT, nt = tile % NT;  // hidden tiles fastest: a token tile is read once
            const int b = tc & 1;
            const int f0 = nt * fp::BF + half * 64;
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int f = f0 + 32 * k + lane;
                sc_g[32 * k + lane] = f < F ? __ldg(q.scale_g + f) : 0.f;
                sc_u[32 * k + lane] = f < F ? __ldg(q.scale_u + f) : 0.f;
            }
            const int trow0 = mt * 2 * fp::BM + static_cast<int>(rank) * fp::BM + qd * 32;
            const int t = trow0 + lane;
            const float inv_s = t < T ? __frcp_rn(__ldg(q.s_tok + t)) : 0.f;
            float top = 0.f;
            __syncwarp();
            if (!warp_wait(&sm->tmem_full[b], (tc >> 1) & 1, abort_flag)) { give_up(); break; }
            tc_fence_after();
            const uint32_t tbase = tmem_base + lane_addr + b * fp::BN + half * 64;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t g[32], u[32];
                tmem_ld32_nowait(tbase + 32 * k, g);
                tmem_ld32_nowait(tbase + fp::BF + 32 * k, u);
                const int fk = f0 + 32 * k;
                if (BWD) {
                    // dh of 32 tokens x 32 units, read along the rows and turned in
                    // the second box (word c of row r at c ^ r: no bank conflicts)
                    uint32_t* const tb = reinterpret_cast<uint32_t*>(sm->box[warp][1]);
                    float d[32];
                    const float* const dp = q.dh + static_cast<size_t>(trow0 < T ? trow0 : 0) * F + fk + lane;
                    const int rows = fk + lane < F ? T - trow0 : 0;  // rows of the warp to read
#pragma unroll
                    for (int r = 0; r < 32; ++r) d[r] = r < rows ? __ldg(dp + static_cast<long long>(r) * F) : 0.f;
                    box_wait(lane);  // both boxes' stores have been read
#pragma unroll
                    for (int r = 0; r < 32; ++r) tb[r * 32 + (lane ^ r)] = __float_as_uint(d[r]);
                    __syncwarp();
                    tmem_wait_into(g);
                    tmem_wait_into(u);
                    if (k == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader(&sm->tmem_empty[b]);
                    }
                    const float2 is = both(inv_s);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 dhv = make_float2(__uint_as_float(tb[lane * 32 + (i ^ lane)]),
                                                       __uint_as_float(tb[lane * 32 + ((i + 1) ^ lane)]));
                        const float2 sgi = *reinterpret_cast<const float2*>(sc_g + 32 * k + i);
                        const float2 sui = *reinterpret_cast<const float2*>(sc_u + 32 * k + i);
                        const float2 gv = dequant2(g[i], g[i + 1], sgi, is), uv = dequant2(u[i], u[i + 1], sui, is);
                        float2 a, da;
                        act_both<ACT>(gv, a, da);
                        // u * act'(g) first: dh * u may pass fp32's range where dh * u * act'(g) does not
                        const float2 vg = mul2(mul2(mul2(uv, da), dhv), mul2(sgi, is));
                        const float2 vu = mul2(mul2(dhv, a), mul2(sui, is));
                        // a token past the end has inv_s = 0, a unit past F a scale of 0
                        g[i] = __float_as_uint(vg.x);
                        g[i + 1] = __float_as_uint(vg.y);
                        u[i] = __float_as_uint(vu.x);
                        u[i + 1] = __float_as_uint(vu.y);
                        top = max3(top, fabsf(vg.x), fabsf(vg.y));
                        top = max3(top, fabsf(vu.x), fabsf(vu.y));
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        box_put(box, lane, c, g[4 * c], g[4 * c + 1], g[4 * c + 2], g[4 * c + 3]);
                        box_put(sm->box[warp][1], lane, c, u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&q.out, smem_u32(box), fk, trow0);
                        tma_store_2d(&q.out, smem_u32(sm->box[warp][1]), q.Fp + fk, trow0);
                    }
                } else {
                    tmem_wait_into(g);
                    tmem_wait_into(u);
                    if (k == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader(&sm->tmem_empty[b]);
                    }
                    float h[32];
                    const float2 is = both(inv_s);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 gv = dequant2(g[i], g[i + 1], *reinterpret_cast<const float2*>(sc_g + 32 * k + i), is);
                        const float2 uv = dequant2(u[i], u[i + 1], *reinterpret_cast<const float2*>(sc_u + 32 * k + i), is);
                        const float2 v = act_times<ACT>(gv, uv);
                        h[i] = v.x;
                        h[i + 1] = v.y;
                    }
                    if (q.out_tma) {
                        if (q.h_bf16) {
                            if (k == 0) box_wait(lane);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                box_put(box, lane, 4 * k + c, pack_bf16(h[8 * c], h[8 * c + 1]), pack_bf16(h[8 * c + 2], h[8 * c + 3]),
                                        pack_bf16(h[8 * c + 4], h[8 * c + 5]), pack_bf16(h[8 * c + 6], h[8 * c + 7]));
                        } else {
                            box_wait(lane);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                box_put(box, lane, c, __float_as_uint(h[4 * c]), __float_as_uint(h[4 * c + 1]),
                                        __float_as_uint(h[4 * c + 2]), __float_as_uint(h[4 * c + 3]));
                        }
                        if (!q.h_bf16 || k == 1) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) tma_store_2d(&q.out, smem_u32(box), q.h_bf16 ? f0 : fk, trow0);
                        }
                    } else {
                        // rows that TMA cannot address (pitch not a multiple of 16
                        // bytes): turned in the box, then written along the rows
                        uint32_t* const tb = reinterpret_cast<uint32_t*>(box);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 32; ++i) tb[lane * 32 + (i ^ lane)] = __float_as_uint(h[i]);
                        __syncwarp();
#pragma unroll 8
                        for (int r = 0; r < 32; ++r) {
                            const float v = __uint_as_float(tb[r * 32 + (lane ^ r)]);
                            if (trow0 + r < T && fk + lane < F) {
                                const size_t at = static_cast<size_t>(trow0 + r) * F + fk + lane;
                                if (q.h_bf16) reinterpret_cast<__nv_bfloat16*>(q.h)[at] = __float2bfloat16_rn(v);
                                else reinterpret_cast<float*>(q.h)[at] = v;
                            }
                        }
                    }
                }
            }
            if (BWD) {
                const unsigned bits = __float_as_uint(top);
                if (t < T && bits) atomicMax(q.row_max + t, bits);
                const unsigned m = __reduce_max_sync(0xFFFFFFFFu, bits);
                if (lane == 0 && m) atomicMax(q.all_max, m);
            }
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp < fp::WARP_TMA) {
        // ------------------------------------------------------------ weight expansion
        // Thread r expands row r of this CTA's matrix (rank 0: gate, rank 1: up).
        const int r = threadIdx.x - fp::EPI_WARPS * 32;
        uint32_t it = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += npairs) {
            for (int kb = 0; kb < KB; ++kb, ++it) {
                const int s = it % STAGES;
                // the producer loads codes only into a stage that the MMAs released
                if (!mbar_wait(&sm->full_c[s], (it / STAGES) & 1, abort_flag)) { give_up(); ok = false; break; }
                // 32-byte code rows, 32B-swizzled by TMA
                const uint8_t* src = sm->p[s] + r * 32;
                const int hs = (r >> 2) & 1;
                const uint4 p0 = *reinterpret_cast<const uint4*>(src + (hs << 4));
                const uint4 p1 = *reinterpret_cast<const uint4*>(src + ((hs ^ 1) << 4));
                uint8_t* dst = sm->b[s] + r * 128;
                const int sw = r & 7;
                const uint32_t w[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t e[4];
                    expand_pairs(w[c], e);
                    const uint32_t a = smem_u32(dst + ((c ^ sw) << 4));
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(e[0]), "r"(e[1]), "r"(e[2]),
                                 "r"(e[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if ((r & 31) == 0) arrive_leader(&sm->full_dec[s]);
            }
        }
    } else if (warp == fp::WARP_TMA) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const CUtensorMap* const wmap = rank ? &q.wu : &q.wg;
            uint32_t it = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += npairs) {
                const int trow = tile / NT * 2 * fp::BM + static_cast<int>(rank) * fp::BM;
                const int frow = tile % NT * fp::BF;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&sm->empty[s], ((it / STAGES) & 1) ^ 1, abort_flag)) { give_up(); ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(&sm->full_a[s], 2 * fp::A_BYTES);
                    mbar_arrive_expect_tx(&sm->full_c[s], fp::P_BYTES);
                    tma_load_2d_pair(smem_u32(sm->a[s]), &q.x, kb * fp::BK, trow, map_to_cta(smem_u32(&sm->full_a[s]), 0));
                    tma_load_2d(smem_u32(sm->p[s]), wmap, kb * (fp::BK / 4), frow, &sm->full_c[s]);
                }
            }
            // let the issued loads land before the CTA can exit
            const uint32_t first = it > STAGES ? it - STAGES : 0;
            volatile int never = 0;
            for (uint32_t j = first; j < it; ++j) {
                const int s = j % STAGES;
                const uint32_t ph = (j / STAGES) & 1;
                if (!mbar_wait(&sm->full_c[s], ph, &never)) give_up();
                if (leader && !mbar_wait(&sm->full_a[s], ph, &never)) give_up();
            }
        }
    } else {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        if (lane == 0) {
            if (leader) {
                const uint32_t idesc = i8_idesc<2 * fp::BM, fp::BN>();
                uint32_t it = 0;
                int tc = 0;
                bool ok = true;
                for (int tile = pair; tile < tiles && ok; tile += npairs, ++tc) {
                    const int b = tc & 1;
                    if (!mbar_wait(&sm->tmem_empty[b], ((tc >> 1) & 1) ^ 1, abort_flag)) { give_up(); break; }
                    tc_fence_after();
                    const uint32_t d = tmem_base + b * fp::BN;
                    for (int kb = 0; kb < KB; ++kb, ++it) {
                        const int s = it % STAGES;
                        const uint32_t ph = (it / STAGES) & 1;
                        if (!mbar_wait(&sm->full_a[s], ph, abort_flag) || !mbar_wait(&sm->full_dec[s], ph, abort_flag)) {
                            give_up(); ok = false; break;
                        }
                        tc_fence_after();
                        const uint32_t a0 = smem_u32(sm->a[s]), b0 = smem_u32(sm->b[s]);
#pragma unroll
                        for (int kk = 0; kk < fp::BK / 32; ++kk)
                            tc_mma_pair(d, sw128_desc(a0 + kk * 32), sw128_desc(b0 + kk * 32), idesc, (kb | kk) != 0);
                        tc_commit_pair_both(&sm->empty[s]);
                    }
                    if (ok) tc_commit_pair_both(&sm->tmem_full[b]);
                }
                tc_commit_pair_both(&sm->mma_done);
            }
            volatile int never = 0;
            if (!mbar_wait(&sm->mma_done, 0, &never)) give_up();
        }
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();
    if (warp == fp::WARP_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * fp::BN)
                     : "memory");
    }
}

// Codes of a matrix whose rows are not a multiple of 16 bytes (K % 64 != 0),
// copied to rows that are, zero codes at the end: TMA's row pitch.
__global__ void __launch_bounds__(256)
    ffn_pad_codes_kernel(const uint32_t* __restrict__ pg, const uint32_t* __restrict__ pu, long long F, int words,
                         int padded, uint32_t* __restrict__ og, uint32_t* __restrict__ ou) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long n = F * padded;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < 2 * n; i += gridDim.x * 256ll) {
        const bool up = i >= n;
        const long long j = up ? i - n : i, row = j / padded;
        const int c = static_cast<int>(j - row * padded);
        (up ? ou : og)[j] = c < words ? __ldg((up ? pu : pg) + row * words + c) : 0u;
    }
}

// ---------------------------------------------------------------- backward operands
// er: the power of two that a token's v is divided by.  Its largest |v|, with
// exponent e, lands in [2^14, 2^15) (a token below 2^-112 keeps what 2^126 gives it).
// An infinite v counts as 2^128: it stays infinite, and its token above all others.
__device__ __forceinline__ int row_exponent(unsigned bits) {
    const int e = static_cast<int>(bits >> 23) - 127;
    return max(e - 14, -126);
}
// Power of two that x_q of a token takes in dW's product.
__device__ __forceinline__ int token_shift(unsigned bits, int top) { return row_exponent(bits) - top + 8; }
// Whether x_q times that falls below fp16's normal numbers.
constexpr int kLeastShift = -14;
__device__ __forceinline__ bool token_far(unsigned bits, int top) { return bits != 0u && token_shift(bits, top) < kLeastShift; }
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }

struct FfnOperands {
    const float* v;            // [T, 2 Fp]
    const unsigned* row_max;
    const unsigned* all_max;
    const uint8_t* pg;
    const uint8_t* pu;
    const int8_t* xq;          // [T, K], pairing order
    __half* parts;             // [T, 2 * 2 Fp]: high parts, low parts
    __half* codes;             // [2 Fp, K] or NULL (no dX)
    __half* xs;                // [T, K] or NULL (no dW)
    unsigned* far;             // tokens left out of xs
    int T, K, F, Fp;
    int split_blocks, code_blocks, x_blocks;
};

// Up to three copies in one launch: blocks split into ranges, 256 threads, items of 8 or 16 elements.
__global__ void __launch_bounds__(256) ffn_operands_kernel(const FfnOperands q) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int block = blockIdx.x;
    if (block < q.split_blocks) {
        // 8 values of one token: v * 2^-er in two fp16 parts
        const int per_row = 2 * q.Fp / 8;
        const long long n = static_cast<long long>(q.T) * per_row;
        for (long long i = block * 256ll + threadIdx.x; i < n; i += q.split_blocks * 256ll) {
            const long long t = i / per_row;
            const int c = static_cast<int>(i - t * per_row) * 8;
            const float s = pow2f(-row_exponent(__ldg(q.row_max + t)));
            const float4* const p = reinterpret_cast<const float4*>(q.v + t * 2 * q.Fp + c);
            const float4 a = __ldg(p), b = __ldg(p + 1);
            const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v0 = f[2 * j] * s, v1 = f[2 * j + 1] * s;
                const __half2 h = __floats2half2_rn(v0, v1);
                const float2 hf = __half22float2(h);
                const __half2 l = __floats2half2_rn(v0 - hf.x, v1 - hf.y);  // the difference is exact
                hi[j] = *reinterpret_cast<const uint32_t*>(&h);
                lo[j] = *reinterpret_cast<const uint32_t*>(&l);
            }
            __half* const o = q.parts + t * 4 * q.Fp + c;
            *reinterpret_cast<uint4*>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(o + 2 * q.Fp) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        return;
    }
    block -= q.split_blocks;
    const int words = q.K / 16;
    if (block < q.code_blocks) {
        // 16 codes of one row: 0, +1, -1 in fp16; rows past F are zeros
        const long long n = 2ll * q.Fp * words;
        for (long long i = block * 256ll + threadIdx.x; i < n; i += q.code_blocks * 256ll) {
            const long long r = i / words;
            const int c = static_cast<int>(i - r * words);
            const bool up = r >= q.Fp;
            const long long f = up ? r - q.Fp : r;
            const uint32_t w = f < q.F ? __ldg(reinterpret_cast<const uint32_t*>(up ? q.pu : q.pg) + f * words + c) : 0u;
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t c0 = (w >> (4 * j)) & 3u, c1 = (w >> (4 * j + 2)) & 3u;
                // 01 -> 0x3C00, 10 -> 0xBC00
                o[j] = (c0 ? 0x3C00u | (c0 & 2u) << 14 : 0u) | (c1 ? 0x3C00u | (c1 & 2u) << 14 : 0u) << 16;
            }
            uint4* const p = reinterpret_cast<uint4*>(q.codes + r * q.K + 16 * c);
            p[0] = make_uint4(o[0], o[1], o[2], o[3]);
            p[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        return;
    }
    block -= q.code_blocks;
    // 16 activations of one token: x_q * 2^(er - max er + 8), back in column order; zeros
    // for a token without a gradient and for one that ffn_far_kernel adds
    const long long n = static_cast<long long>(q.T) * words;
    const int top = row_exponent(*q.all_max);
    for (long long i = block * 256ll + threadIdx.x; i < n; i += q.x_blocks * 256ll) {
        const long long t = i / words;
        const unsigned bits = __ldg(q.row_max + t);
        const int e = token_shift(bits, top);
        const float s = e < kLeastShift ? 0.f : pow2f(e);
        if (i == t * words && token_far(bits, top)) atomicAdd(q.far, 1u);
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(q.xq) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};  // even 0-6, odd 1-7, even 8-14, odd 9-15
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // elements 2 j and 2 j + 1
            const int g = (j >> 2) * 2, sh = 8 * (j & 3);
            const float a = static_cast<float>(static_cast<int8_t>(w[g] >> sh)) * s;
            const float b = static_cast<float>(static_cast<int8_t>(w[g + 1] >> sh)) * s;
            const __half2 h = __floats2half2_rn(a, b);
            o[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        uint4* const p = reinterpret_cast<uint4*>(q.xs) + 2 * i;
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// dX: the token's sums times 2^er * s_t.
struct FfnDx {
    struct Params {
        CUtensorMap out;
        const unsigned* row_max;
        const float* s_tok;
        int T, row_mask;  // 127 when rows 128 .. 255 are the low parts' sums of the same tokens, else -1
    };
    static __device__ __forceinline__ void prefetch(const Params& p) { prefetch_tmap(&p.out); }
    const Params& p;
    float e, s;
    __device__ __forceinline__ explicit FfnDx(const Params& r) : p(r), e(0.f), s(0.f) {}
    __device__ __forceinline__ void begin(const GemmTile& t) {
        const int token = t.row & p.row_mask;
        if (token < p.T) {
            e = pow2f(row_exponent(__ldg(p.row_max + token)));
            s = __ldg(p.s_tok + token);
        }
    }
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (v[i] * e) * s;
        if ((t.warp_row & p.row_mask) < p.T) put_f32(t, k, v, &p.out, 0, false);  // later rows are the next part's
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// The parts of a split reduction, added in order; 4 elements per thread.
__global__ void __launch_bounds__(256) ffn_sum_kernel(const float4* __restrict__ parts, int splits, long long stride4,
                                                      long long n4, float4* __restrict__ out) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
        float4 a = parts[i];
        for (int s = 1; s < splits; ++s) {
            const float4 b = parts[i + s * stride4];
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        out[i] = a;
    }
}

// dW's terms of the far tokens (token_far), added to the gradients that the product has
// written: dW[f, k] += (1 / scale[f]) * sum_t v[t, f] * x_q[t, k], v from fp32 memory.
// Most calls have none and the kernel ends at once.  Tiles of 128 units x 128 k, 8 x 8
// of them a thread; the tokens in order, added in groups of 32, 32 groups of 1024, the
// 1024s to dW: 32 + 32 + T / 1024 roundings of a sum at most.  The list of the far tokens
// stays in shared memory for all of a block's tiles unless it is longer than KEEP.  On
// CUDA cores: at 4096 tokens, 2048 -> 7168, the backward takes 0.85 ms with no far
// token, 1.02 with one, 1.15 with 64 and 10.3 with all but one.
struct FfnFar {
    const unsigned* far;
    const unsigned* row_max;
    const unsigned* all_max;
    const float* v;            // [T, 2 Fp]
    const int8_t* xq;          // [T, K], pairing order
    const float* scale_g;
    const float* scale_u;
    float* dwg;                // each [F, K] or NULL
    float* dwu;
    int T, K, F, Fp, ternary;
};
__global__ void __launch_bounds__(256) ffn_far_kernel(const FfnFar q) {
    constexpr int TILE = 128, GROUP = 32, CHUNK = 1024, KEEP = 2048;
    __shared__ int list[KEEP + CHUNK];
    __shared__ int warp_count[8];
    __shared__ __align__(16) float sv[GROUP][TILE];
    __shared__ __align__(16) float sx[GROUP][TILE];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (*q.far == 0u) return;
    const int top = row_exponent(*q.all_max), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // lists the far tokens from t0 on, in order, until it holds more than KEEP; moves t0 on
    auto fill = [&](int& t0) {
        int n = 0;
        while (t0 < q.T && n <= KEEP) {
            const int t = t0 + 4 * tid;
            unsigned mine = 0;
            if (t < q.T) {  // row_max ends on a 16-byte unit
                const uint4 b = __ldg(reinterpret_cast<const uint4*>(q.row_max + t));
                const unsigned bits[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) mine |= t + i < q.T && token_far(bits[i], top) ? 1u << i : 0u;
            }
            const int c = __popc(mine);
            int upto = c;  // of the warp's threads up to this one
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
                if (lane >= off) upto += o;
            }
            __syncthreads();  // the last counts, and the last list, have been read
            if (lane == 31) warp_count[warp] = upto;
            __syncthreads();
            int at = n + upto - c;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                at += w < warp ? warp_count[w] : 0;
                n += warp_count[w];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (mine >> i & 1u) list[at++] = t + i;
            t0 += CHUNK;
        }
        __syncthreads();
        return n;
    };
    int t0 = 0;
    int n = fill(t0);
    const bool whole = t0 >= q.T;
    const int ft = (q.F + TILE - 1) / TILE, kt = (q.K + TILE - 1) / TILE;
    const long long per_matrix = static_cast<long long>(ft) * kt;
    const long long tiles = per_matrix * ((q.dwg != nullptr) + (q.dwu != nullptr));
    const int fc = tid / 16 * 4, kc = tid % 16 * 4;  // this thread's units fc .. + 3 and 64 + fc .. + 3, k likewise
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const bool up = !q.dwg || tile >= per_matrix;
        const long long at = tile % per_matrix;
        const int f0 = static_cast<int>(at / kt) * TILE, k0 = static_cast<int>(at % kt) * TILE;
        const float* const vp = q.v + (up ? q.Fp : 0) + f0;
        float* const out = up ? q.dwu : q.dwg;
        const float* const scale = up ? q.scale_u : q.scale_g;
        float sum[8][8];
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 8; ++b) sum[a][b] = 0.f;
        auto flush = [&] {
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                const int f = f0 + fc + (a & 3) + (a >> 2) * 64;
                if (f >= q.F) continue;
                const float s = q.ternary ? 1.0f : __frcp_rn(__ldg(scale + f));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + kc + h * 64;
                    if (k >= q.K) continue;  // K % 16 == 0: four columns at once
                    float4* const d = reinterpret_cast<float4*>(out + static_cast<size_t>(f) * q.K + k);
                    float4 o = *d;
                    o.x += sum[a][4 * h] * s;
                    o.y += sum[a][4 * h + 1] * s;
                    o.z += sum[a][4 * h + 2] * s;
                    o.w += sum[a][4 * h + 3] * s;
                    *d = o;
                }
#pragma unroll
                for (int b = 0; b < 8; ++b) sum[a][b] = 0.f;
            }
        };
        int groups = 0;
        if (!whole) t0 = 0;
        do {
            if (!whole) n = fill(t0);
            for (int g0 = 0; g0 < n; g0 += GROUP) {
                const int m = n - g0 < GROUP ? n - g0 : GROUP;
                __syncthreads();  // the previous group has been read
                for (int i = tid; i < m * (TILE / 4); i += 256) {  // v's units past F, up to Fp, are zeros
                    const int j = i / (TILE / 4), c = i % (TILE / 4) * 4;
                    *reinterpret_cast<float4*>(&sv[j][c]) =
                        __ldg(reinterpret_cast<const float4*>(vp + static_cast<long long>(list[g0 + j]) * 2 * q.Fp + c));
                }
                if (const int j = tid / 8, c = tid % 8 * 16; j < m) {
                    uint4 u = make_uint4(0u, 0u, 0u, 0u);
                    if (k0 + c < q.K)
                        u = __ldg(reinterpret_cast<const uint4*>(q.xq + static_cast<long long>(list[g0 + j]) * q.K + k0 + c));
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};  // even 0-6, odd 1-7, even 8-14, odd 9-15
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sx[j][c + i] = static_cast<float>(static_cast<int8_t>(w[(i >> 3) * 2 + (i & 1)] >> (8 * ((i & 7) >> 1))));
                }
                __syncthreads();
                float part[8][8];
#pragma unroll
                for (int a = 0; a < 8; ++a)
#pragma unroll
                    for (int b = 0; b < 8; ++b) part[a][b] = 0.f;
                for (int j = 0; j < m; ++j) {
                    float va[8], xa[8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        *reinterpret_cast<float4*>(va + 4 * h) = *reinterpret_cast<const float4*>(&sv[j][fc + 64 * h]);
                        *reinterpret_cast<float4*>(xa + 4 * h) = *reinterpret_cast<const float4*>(&sx[j][kc + 64 * h]);
                    }
#pragma unroll
                    for (int a = 0; a < 8; ++a)
#pragma unroll
                        for (int b = 0; b < 8; ++b) part[a][b] = fmaf(va[a], xa[b], part[a][b]);
                }
#pragma unroll
                for (int a = 0; a < 8; ++a)
#pragma unroll
                    for (int b = 0; b < 8; ++b) sum[a][b] += part[a][b];
                if (++groups == 32) {
                    flush();
                    groups = 0;
                }
            }
        } while (!whole && t0 < q.T);
        if (groups) flush();
    }
}

// dW: rows 0 .. Fp - 1 to the gate's gradient, the next Fp to the up's, times
// 2^(max er - 8) / scale (ternary: without the division).
struct FfnDw {
    struct Params {
        CUtensorMap out_g, out_u;
        const unsigned* all_max;
        const float* scale_g;
        const float* scale_u;
        int F, Fp, up_row, want_g, want_u, ternary;  // up_row: row of the up's first in its output
    };
    static __device__ __forceinline__ void prefetch(const Params& p) {
        if (p.want_g) prefetch_tmap(&p.out_g);
        if (p.want_u) prefetch_tmap(&p.out_u);
    }
    const Params& p;
    float e, s;
    bool up;
    __device__ __forceinline__ explicit FfnDw(const Params& r) : p(r), e(pow2f(row_exponent(*r.all_max))), s(0.f), up(false) {}
    __device__ __forceinline__ void begin(const GemmTile& t) {
        up = t.warp_row >= p.Fp;  // Fp % 128 == 0: a warp's 32 rows are of one matrix
        const int f = t.row - (up ? p.Fp : 0);
        s = f < p.F ? (p.ternary ? 1.0f : __frcp_rn(__ldg((up ? p.scale_u : p.scale_g) + f))) : 0.f;
        s *= 0.00390625f;  // x_q came times 2^8
    }
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        if (up ? !p.want_u : !p.want_g) return;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (v[i] * e) * s;
        put_f32(t, k, v, up ? &p.out_u : &p.out_g, up ? p.up_row : 0, false);
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// ---------------------------------------------------------------- host side
size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

bool takes_decode(long long T, long long K) {
    return T <= fd::MAX_TOKENS && K <= (1 << 20) && fd::smem_bytes(static_cast<int>(K), 1) <= kMostShared;
}

// Quantised activations, their scales, and the padded codes of both matrices.
struct FfnSpace {
    size_t xq, s_tok, codes, end;
};
FfnSpace ffn_space(long long T, long long K, long long F) {
    FfnSpace s;
    s.xq = 0;
    s.s_tok = round256(static_cast<size_t>(T) * K);
    s.codes = s.s_tok + round256(static_cast<size_t>(T) * 4);
    s.end = s.codes + (K % 64 ? 2 * round256(static_cast<size_t>(F) * ((K + 63) / 64 * 16)) : 0);
    return s;
}

// Parts of the two gradients' reductions (over 2 Fp hidden units, over T).
// Up to 128 tokens v's two parts lie in the two CTAs' rows of one A (GemmShape::stack)
// instead of in two A of 256 rows: half the MMAs.
bool dx_stacks(long long T) { return T <= gm::BM; }
// (The plan is of both gradients also when one is wanted: the same bits.)
GemmPlan make_grad_plan(long long T, long long K, long long Fp) {
    const long long cols = (K + gm::BN - 1) / gm::BN;
    const GemmWork dx{(T + 255) / 256 * cols, 2 * Fp / gm::BK, dx_stacks(T) ? 0.45 : 0.8, 1.0,
                      (dx_stacks(T) ? 8.0 : 4.0) * T * K, 32};
    const GemmWork dw{(2 * Fp + 255) / 256 * cols, (T + gm::BK - 1) / gm::BK, 0.8, 1.0, 8.0 * Fp * K, 32};
    return gemm_plan(dx, dw);
}
// Asked for three times a call (workspace, its check, the launch) at 1 to 2 us: the
// thread's last sizes are remembered.
GemmPlan grad_plan(long long T, long long K, long long Fp) {
    thread_local long long sizes[3] = {};
    thread_local GemmPlan plan = {};
    if (sizes[0] != T || sizes[1] != K || sizes[2] != Fp) {
        plan = make_grad_plan(T, K, Fp);
        sizes[0] = T;
        sizes[1] = K;
        sizes[2] = Fp;
    }
    return plan;
}

struct FfnBwdSpace {
    FfnSpace fwd;
    size_t maxima, v, parts, codes, xs, dx_sums, dw_sums, end;
    long long Fp, nmax16, dx_rows;
    GemmPlan plan;  // of dX and dW
};
FfnBwdSpace ffn_bwd_space(long long T, long long K, long long F, int need_dx, int need_dw) {
    FfnBwdSpace s;
    s.fwd = ffn_space(T, K, F);
    s.Fp = (F + 127) / 128 * 128;
    s.nmax16 = (T + 2 + 3) / 4;  // row maxima, the maximum of all, the far tokens' count: 16-byte units
    s.maxima = s.fwd.end;
    s.v = s.maxima + round256(static_cast<size_t>(s.nmax16) * 16);
    s.parts = s.v + round256(static_cast<size_t>(T) * 2 * s.Fp * 4);
    s.codes = s.parts + round256(static_cast<size_t>(T) * 4 * s.Fp * 2);
    s.xs = s.codes + (need_dx ? round256(static_cast<size_t>(2) * s.Fp * K * 2) : 0);
    s.dx_sums = s.xs + (need_dw ? round256(static_cast<size_t>(T) * K * 2) : 0);
    s.dx_rows = dx_stacks(T) ? 2 * gm::BM : (T + 31) / 32 * 32;
    s.plan = grad_plan(T, K, s.Fp);
    const bool dx_parts = need_dx && (s.plan.splits1 > 1 || dx_stacks(T)), dw_parts = need_dw && s.plan.splits2 > 1;
    s.dw_sums = s.dx_sums + (dx_parts ? round256(static_cast<size_t>(s.plan.splits1) * s.dx_rows * K * 4) : 0);
    s.end = s.dw_sums + (dw_parts ? round256(static_cast<size_t>(s.plan.splits2) * 2 * s.Fp * K * 4) : 0);
    return s;
}

bool byte_map(CUtensorMap* map, const void* base, long long rows, long long row_bytes, int box_bytes, int box_rows,
              CUtensorMapSwizzle swizzle) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const cuuint32_t estr[2] = {1, 1};
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows)};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BWD, int ACT>
cudaError_t launch_pair(const FfnParams& q, unsigned* status, cudaStream_t st) {
    auto kern = ffn_pair_kernel<BWD, ACT>;
    static int clusters[64] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(fp::THREADS);
    cfg.dynamicSmemBytes = ffn_smem_bytes<BWD>();
    cfg.stream = st;
    if (clusters[dev] == 0) {
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(ffn_smem_bytes<BWD>())))
            return e;
        int n = 0;
        if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) return e;
        if (n <= 0) return cudaErrorNotSupported;
        clusters[dev] = n;
    }
    const long long tiles = ((q.T + 2ll * fp::BM - 1) / (2 * fp::BM)) * ((q.F + fp::BF - 1) / fp::BF);
    if (tiles > (1ll << 30)) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < clusters[dev] ? tiles : clusters[dev]));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, q, status);
}

// Activations quantised (and `nzero16` 16-byte units at zero16 cleared), codes
// padded where TMA needs it, and the tensor maps and scales that both
// directions share.
cudaError_t pair_inputs(FfnParams& q, const uint16_t* x, long long T, long long K, const uint8_t* pg,
                        const float* scale_g, const uint8_t* pu, const float* scale_u, long long F, uint8_t* ws,
                        void* zero16, long long nzero16, unsigned* status, int num_sms, cudaStream_t st) {
    const FfnSpace sp = ffn_space(T, K, F);
    int8_t* const xq = reinterpret_cast<int8_t*>(ws + sp.xq);
    float* const s_tok = reinterpret_cast<float*>(ws + sp.s_tok);
    if (cudaError_t e = launch_quant(x, T, K, xq, s_tok, kLayoutPairsFfn, status, st, zero16, nzero16)) return e;
    long long row_bytes = K / 4;
    if (K % 64) {
        const int words = static_cast<int>(K / 16), padded = (words + 3) / 4 * 4;
        uint8_t* const og = ws + sp.codes;
        uint8_t* const ou = og + round256(static_cast<size_t>(F) * padded * 4);
        const long long blocks = (2 * F * padded + 255) / 256, most = 8ll * num_sms;
        if (cudaError_t e = pdl_launch(ffn_pad_codes_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                       dim3(256), 0, st, reinterpret_cast<const uint32_t*>(pg),
                                       reinterpret_cast<const uint32_t*>(pu), F, words, padded,
                                       reinterpret_cast<uint32_t*>(og), reinterpret_cast<uint32_t*>(ou)))
            return e;
        pg = og;
        pu = ou;
        row_bytes = padded * 4ll;
    }
    if (!byte_map(&q.x, xq, T, K, fp::BK, fp::BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !byte_map(&q.wg, pg, F, row_bytes, fp::BK / 4, fp::BF, CU_TENSOR_MAP_SWIZZLE_32B) ||
        !byte_map(&q.wu, pu, F, row_bytes, fp::BK / 4, fp::BF, CU_TENSOR_MAP_SWIZZLE_32B))
        return cudaErrorInvalidValue;
    q.scale_g = scale_g;
    q.scale_u = scale_u;
    q.s_tok = s_tok;
    q.T = static_cast<int>(T);
    q.K = static_cast<int>(K);
    q.F = static_cast<int>(F);
    return cudaSuccess;
}

template <int NT, int CW, int ACT>
cudaError_t launch_decode_as(const uint8_t* pg, const float* sg, const uint8_t* pu, const float* su, int F, int K,
                             const uint16_t* x, int t0, int TP, int KS, void* h, int h_bf16, unsigned* status,
                             cudaStream_t st) {
    const size_t smem = fd::smem_bytes(K, TP);
    if (smem > 48 * 1024)
        if (cudaError_t e = allow_shared<ffn_decode_kernel<NT, CW, ACT>>()) return e;
    const int tiles = (F + 7) / 8, per_block = fd::warps(NT) / KS;
    return pdl_launch(ffn_decode_kernel<NT, CW, ACT>, dim3((tiles + per_block - 1) / per_block), dim3(fd::warps(NT) * 32), smem,
                      st, pg, sg, pu, su, F, K, x, t0, TP, KS, h, h_bf16, status);
}

template <int NT, int ACT>
cudaError_t launch_decode_cw(int CW, const uint8_t* pg, const float* sg, const uint8_t* pu, const float* su, int F, int K,
                             const uint16_t* x, int t0, int TP, int KS, void* h, int h_bf16, unsigned* status,
                             cudaStream_t st) {
    if (CW == 4) return launch_decode_as<NT, 4, ACT>(pg, sg, pu, su, F, K, x, t0, TP, KS, h, h_bf16, status, st);
    if (CW == 2) return launch_decode_as<NT, 2, ACT>(pg, sg, pu, su, F, K, x, t0, TP, KS, h, h_bf16, status, st);
    return launch_decode_as<NT, 1, ACT>(pg, sg, pu, su, F, K, x, t0, TP, KS, h, h_bf16, status, st);
}

template <int ACT>
cudaError_t run_decode(const uint16_t* x, long long T, int K, const uint8_t* pg, const float* sg, const uint8_t* pu,
                       const float* su, int F, void* h, int h_bf16, unsigned* status, int num_sms, cudaStream_t st) {
    const int CW = K % 256 == 0 ? 4 : K % 128 == 0 ? 2 : 1;
    const int C = fd::pad64(K) / (64 * CW), nb = CW == 4 ? 2 : 4, tiles = (F + 7) / 8;
    // warps per tile: the fewest whose slices fit one batch of loads, then more
    // while all of them still fit the SMs at once, never more than chunks or
    // than a block has
    const int most = fd::warps(T > 8 ? 2 : 1);
    int KS = 1;
    while (KS < most && KS < C && (C + KS - 1) / KS > nb) KS *= 2;
    while (KS < most && 2 * KS <= C && static_cast<long long>(tiles) * 2 * KS <= static_cast<long long>(num_sms) * fd::SM_WARPS)
        KS *= 2;
    int cap = fd::MAX_TOKENS;  // tokens of one pass
    while (cap > 1 && fd::smem_bytes(K, cap) > kMostShared) --cap;
    for (int t0 = 0; t0 < T; t0 += cap) {
        const int TP = static_cast<int>(T) - t0 < cap ? static_cast<int>(T) - t0 : cap;
        const int ks = KS < fd::warps(TP > 8 ? 2 : 1) ? KS : fd::warps(TP > 8 ? 2 : 1);
        const cudaError_t e = TP > 8 ? launch_decode_cw<2, ACT>(CW, pg, sg, pu, su, F, K, x, t0, TP, ks, h, h_bf16, status, st)
                                     : launch_decode_cw<1, ACT>(CW, pg, sg, pu, su, F, K, x, t0, TP, ks, h, h_bf16, status, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t ffn_workspace_bytes(long long T, long long K, long long F) { return takes_decode(T, K) ? 0 : ffn_space(T, K, F).end; }

size_t ffn_backward_workspace_bytes(long long T, long long K, long long F, int need_dx, int need_dw) {
    return ffn_bwd_space(T, K, F, need_dx, need_dw).end;
}

cudaError_t launch_ffn(const uint16_t* x, long long T, long long K, const uint8_t* pg, const float* scale_g,
                       const uint8_t* pu, const float* scale_u, long long F, int act, void* h, int h_bf16, void* ws,
                       unsigned* status, int num_sms, cudaStream_t st) {
    if (takes_decode(T, K))
        return act == kActSilu ? run_decode<0>(x, T, static_cast<int>(K), pg, scale_g, pu, scale_u, static_cast<int>(F), h,
                                               h_bf16, status, num_sms, st)
                               : run_decode<1>(x, T, static_cast<int>(K), pg, scale_g, pu, scale_u, static_cast<int>(F), h,
                                               h_bf16, status, num_sms, st);
    FfnParams q;
    memset(&q, 0, sizeof(q));
    if (cudaError_t e = pair_inputs(q, x, T, K, pg, scale_g, pu, scale_u, F, static_cast<uint8_t*>(ws), nullptr, 0, status,
                                    num_sms, st))
        return e;
    const int es = h_bf16 ? 2 : 4;
    q.h = h;
    q.h_bf16 = h_bf16;
    q.out_tma = F * es % 16 == 0;
    q.out = q.x;
    if (q.out_tma && !gemm_map(&q.out, h_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, h, T, F,
                               F * es, 128 / es, 32))
        return cudaErrorInvalidValue;
    return act == kActSilu ? launch_pair<false, 0>(q, status, st) : launch_pair<false, 1>(q, status, st);
}

cudaError_t launch_ffn_backward(const float* dh, const uint16_t* x, long long T, long long K, const uint8_t* pg,
                                const float* scale_g, const uint8_t* pu, const float* scale_u, long long F, int act,
                                float* dx, float* dwg, float* dwu, int ternary, void* ws, unsigned* status, int num_sms,
                                cudaStream_t st) {
    uint8_t* const base = static_cast<uint8_t*>(ws);
    const int need_dw = dwg || dwu;
    const FfnBwdSpace sp = ffn_bwd_space(T, K, F, dx != nullptr, need_dw);
    const int Ti = static_cast<int>(T), Ki = static_cast<int>(K), Fi = static_cast<int>(F), Fp = static_cast<int>(sp.Fp);
    FfnParams q;
    memset(&q, 0, sizeof(q));
    if (cudaError_t e = pair_inputs(q, x, T, K, pg, scale_g, pu, scale_u, F, base, base + sp.maxima, sp.nmax16, status,
                                    num_sms, st))
        return e;
    float* const v = reinterpret_cast<float*>(base + sp.v);
    unsigned* const row_max = reinterpret_cast<unsigned*>(base + sp.maxima);
    unsigned* const all_max = row_max + T;
    unsigned* const far = all_max + 1;
    const int8_t* const xq = reinterpret_cast<const int8_t*>(base + sp.fwd.xq);
    const float* const s_tok = q.s_tok;
    q.all_max = all_max;
    q.Fp = Fp;
    __half* const parts = reinterpret_cast<__half*>(base + sp.parts);
    __half* const codes = reinterpret_cast<__half*>(base + sp.codes);
    __half* const xs = reinterpret_cast<__half*>(base + sp.xs);
    auto blocks_for = [&](long long items, int per_sm) {
        const long long want = (items + 255) / 256, most = static_cast<long long>(per_sm) * num_sms;
        return static_cast<int>(want < most ? want : most);
    };
    FfnOperands o;
    o.v = v;
    o.all_max = all_max;
    o.pg = pg;
    o.pu = pu;
    o.xq = xq;
    o.codes = codes;
    o.xs = xs;
    o.far = far;
    o.K = Ki;
    o.F = Fi;
    o.Fp = Fp;
    q.dh = dh;
    q.row_max = row_max;
    if (!gemm_map(&q.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, v, T, 2 * sp.Fp, 2 * sp.Fp * 4, 32, 32)) return cudaErrorInvalidValue;
    if (cudaError_t e = act == kActSilu ? launch_pair<true, 0>(q, status, st) : launch_pair<true, 1>(q, status, st)) return e;
    o.row_max = row_max;
    o.parts = parts;
    o.T = Ti;
    o.split_blocks = blocks_for(T * (2 * sp.Fp / 8), 8);
    o.code_blocks = dx ? blocks_for(2 * sp.Fp * (K / 16), 4) : 0;
    o.x_blocks = need_dw ? blocks_for(T * (K / 16), 4) : 0;
    if (cudaError_t e = pdl_launch(ffn_operands_kernel, dim3(o.split_blocks + o.code_blocks + o.x_blocks), dim3(256), 0, st, o))
        return e;

    const int k_panel = (Ki + gm::BN - 1) / gm::BN;
    float* const dx_sums = reinterpret_cast<float*>(base + sp.dx_sums);
    float* const dw_sums = reinterpret_cast<float*>(base + sp.dw_sums);
    using DxJob = GemmJob<FfnDx, 2, false, true>;
    using DxStacked = GemmJob<FfnDx, 1, false, true>;
    using DwJob = GemmJob<FfnDw, 2, true, true>;
    const bool stack = dx_stacks(T);
    const int dx_splits = sp.plan.splits1, dw_splits = sp.plan.splits2;
    GemmArgs<DxJob> gx;
    GemmArgs<DwJob> gw;
    memset(&gx, 0, sizeof(gx));
    memset(&gw, 0, sizeof(gw));
    if (dx) {
        const int a_box = gemm_a_box(T);
        const bool parts_first = dx_splits > 1 || stack;
        if (!gemm_operand(&gx.a, true, false, parts, T, 4 * sp.Fp, 4 * sp.Fp, a_box) ||
            !gemm_operand(&gx.b, true, true, codes, 2 * sp.Fp, K, K) ||
            !gemm_result_f32(&gx.p.out, parts_first ? dx_sums : dx, parts_first ? dx_splits * sp.dx_rows : T, K))
            return cudaErrorInvalidValue;
        gx.p.row_max = row_max;
        gx.p.s_tok = s_tok;
        gx.p.T = Ti;
        gx.p.row_mask = stack ? gm::BM - 1 : -1;
        gx.shape = GemmShape{Ti, Ki, 2 * Fp, 2 * Fp, k_panel, dx_splits, static_cast<int>(sp.dx_rows), a_box, 0, stack ? 2 * Fp : 0};
    }
    if (need_dw) {
        FfnDw::Params& p = gw.p;
        if (!gemm_operand(&gw.a, true, true, parts, T, 4 * sp.Fp, 4 * sp.Fp) || !gemm_operand(&gw.b, true, true, xs, T, K, K))
            return cudaErrorInvalidValue;
        if (dw_splits > 1 ? !gemm_result_f32(&p.out_g, dw_sums, dw_splits * 2 * sp.Fp, K) ||
                                !gemm_result_f32(&p.out_u, dw_sums, dw_splits * 2 * sp.Fp, K)
                          : (dwg && !gemm_result_f32(&p.out_g, dwg, F, K)) || (dwu && !gemm_result_f32(&p.out_u, dwu, F, K)))
            return cudaErrorInvalidValue;
        p.all_max = all_max;
        p.scale_g = scale_g;
        p.scale_u = scale_u;
        p.F = Fi;
        p.Fp = Fp;
        p.up_row = dw_splits > 1 ? 0 : Fp;
        p.want_g = dwg != nullptr;
        p.want_u = dwu != nullptr;
        p.ternary = ternary;
        gw.shape = GemmShape{2 * Fp, Ki, Ti, 2 * Fp, k_panel, dw_splits, 2 * Fp, gm::BM, sp.plan.lead, 0};
    }
    const GemmArgs<DxStacked> gs{gx.a, gx.b, gx.p, gx.shape};
    const GemmArgs<GemmNoJob> none{};
    cudaError_t e;
    if (dx && need_dw)
        e = stack ? launch_gemm_jobs<DxStacked, DwJob, 1, true, 4>(gs, gw, status, st)
                  : launch_gemm_jobs<DxJob, DwJob, 1, true, 4>(gx, gw, status, st);
    else if (dx)
        e = stack ? launch_gemm_jobs<DxStacked, GemmNoJob, 1, true, 4>(gs, none, status, st)
                  : launch_gemm_jobs<DxJob, GemmNoJob, 1, true, 4>(gx, none, status, st);
    else
        e = launch_gemm_jobs<DwJob, GemmNoJob, 1, true, 4>(gw, none, status, st);
    // adds `splits` parts of `rows` rows, split_rows apart
    auto join = [&](const float* sums, int splits, long long split_rows, long long rows, float* out) {
        return pdl_launch(ffn_sum_kernel, dim3(blocks_for(rows * K / 4, 8)), dim3(256), 0, st,
                          reinterpret_cast<const float4*>(sums), splits, split_rows * K / 4, rows * K / 4,
                          reinterpret_cast<float4*>(out));
    };
    if (e == cudaSuccess && dx && (dx_splits > 1 || stack))
        e = stack ? join(dx_sums, 2 * dx_splits, gm::BM, T, dx) : join(dx_sums, dx_splits, sp.dx_rows, T, dx);
    if (e == cudaSuccess && dw_splits > 1 && dwg) e = join(dw_sums, dw_splits, 2 * sp.Fp, F, dwg);
    if (e == cudaSuccess && dw_splits > 1 && dwu) e = join(dw_sums + sp.Fp * K, dw_splits, 2 * sp.Fp, F, dwu);
    if (e == cudaSuccess && need_dw) {
        const FfnFar q_far{far, row_max, all_max, v, xq, scale_g, scale_u, dwg, dwu, Ti, Ki, Fi, Fp, ternary};
        const long long tiles = ((F + 127) / 128) * ((K + 127) / 128) * ((dwg != nullptr) + (dwu != nullptr)), most = num_sms;
        e = pdl_launch(ffn_far_kernel, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(256), 0, st, q_far);
    }
    return e;
}

}  // namespace sbl
