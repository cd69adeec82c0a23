// Softmax cross entropy of a vocabulary projection (the LM head's loss), with
// its gradients, without keeping the logits.
//
//   z[t, v] = x[t] . W[v],  lse[t] = log sum_v exp z[t, v],  loss[t] = lse[t] - z[t, target[t]]
//   G[t, v] = (exp(z[t, v] - lse[t]) - [v == target[t]]) * dloss[t]
//   dX = G . W,  dW = G^T . x
//
// (0 for a token whose target is the ignored index.)  The pages' repository
// layout names such a step for training (a fused LM-head matmul with a chunked
// cross entropy); here it is three uses of one tcgen05 GEMM (gemm_f16.cuh):
//
//   forward   z tiles of 256 x 256 whose epilogue keeps, per row and 128
//             columns, the maximum and the sum of exponentials below it, and
//             the target's logit; xent_merge_kernel joins the V / 128 parts of
//             a row.  Memory: x and W once, 8 bytes per row and 128 columns (32
//             for few tokens, whose tiles are turned: LseWords).
//   backward  per piece of the vocabulary: the z tiles again, their epilogue
//             writing G in bf16; dX += G . W[piece] and dW[piece] = G^T . x in
//             one launch or two (grad_plan).  G of
//             one piece is all that exists of the [T, V] matrix.
//
// What G's bf16 costs: dX and dW are bf16, rounded from fp32 sums; rounding
// each G adds an independent error of the same relative size (2^-8 at most) to each
// term, at most sqrt(2) times the output's own rounding in the 2-norm.  To keep
// the largest terms out of it, c = max_t |dloss[t]| is taken out of G and
// multiplied back into the fp32 results: under a mean or sum reduction G's
// entry at an unlikely target is then -1 exactly.  A few tokens, whose errors do
// not average out, take two bf16 parts (kFewTokens).
//
// Bound by what feeds the tensor cores (gemm_f16.cuh) and, over longer runs, by
// the power limit: 2 T V D operations forward, 6 T V D backward (a third of them
// the second time z is computed, the price of not keeping it).  At 8192 x
// 128000 x 896 the four products take 6.6 ms, 1140 TFLOP/s (a library bf16 product
// of 8192^3 sustains 1395); at 4096 x 32000 x 2048 1.84 ms, 1170 TFLOP/s.  The epilogues
// spend about three instructions per logit on pairs of values; an index into
// a row's registers anywhere in them would put the row into local memory.
#include <cuda.h>

#include <cstring>

#include "gemm_f16.cuh"
#include "sbl_common.cuh"

namespace sbl {

namespace {

// The forward's logits are summed in segments of 16 k-blocks (1024 terms): in
// one piece, D = 2048 left lse 1.5e-6 off (the tensor cores' rounding towards
// zero), three times what a sum rounded to nearest leaves.
constexpr int kLogitSegment = 16;
// Up to 256 tokens, whose MMAs leave the tensor pipe mostly idle, segments of 2: over few
// losses, some of them small, the sum's error shows (a token: 1e-6 of its loss).
constexpr int kFewSegment = 2;
// The backward's logits are summed in the same segments, so that they are the ones
// that lse is of, bit for bit.  With a sum of its own in one piece a likely word's
// G = p - 1, which may be 1e-6, was off by 2e-5 at D = 2048 and 3e-4 at 16384; so by
// 5e-7 at both (fp32 products and log-sum-exp: 4e-7).  It costs the tall tiles above
// D = 1024: loss and gradients of 4096 x 32000 x 2048 1.54 ms instead of 1.48.
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Forward epilogue: part[t][p] = (max, sum of exp(z - max)) over columns 128 p .. + 127.
struct LsePart {
    struct Params {
        float2* part;
        float* tlogit;
        const long long* target;
        int T, V, P;  // P: parts of a row
    };
    static __device__ __forceinline__ void prefetch(const Params&) {}
    const Params& p;
    float mx, sum;
    long long tcol;  // the target's column less col0
    __device__ __forceinline__ explicit LsePart(const Params& q) : p(q), mx(0.f), sum(0.f), tcol(-1) {}
    __device__ __forceinline__ void begin(const GemmTile& t) {
        mx = -INFINITY;
        sum = 0.f;
        tcol = t.row < p.T ? __ldg(p.target + t.row) - t.col0 : -1;
    }
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        const int valid = p.V - (t.col0 + 32 * k);
        if (valid <= 0) return;
        if (valid < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i >= valid) v[i] = -INFINITY;
        }
        const long long tc = tcol - 32 * k;
        if (tc >= 0 && tc < 32) {
            // by a bit, not by index: an index would put the row into local memory
            const uint32_t hot = 1u << tc;
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) z = (hot & (1u << i)) ? v[i] : z;
            p.tlogit[t.row] = z;
        }
        float m4[4] = {mx, v[0], v[1], v[2]};
#pragma unroll
        for (int i = 3; i < 31; i += 2) m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], v[i], v[i + 1]);
        const float m = fmaxf(max3(m4[0], m4[1], m4[2]), fmaxf(m4[3], v[31]));
        // (z - m) log2 e, not z log2 e - m log2 e in one step: the maximum's term has to
        // be exactly 1, or a likely word's small loss is the rounding of m log2 e
        const float2 l2 = both(kLog2e), less = both(-m);
        // by the sum, not by mx == -inf: 32 NaN logits leave mx there (max drops NaN) and a NaN sum
        float2 s2[2] = {make_float2(sum == 0.f ? 0.f : sum * exp2_fast((mx - m) * kLog2e), 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 e = mul2(add2(make_float2(v[2 * i], v[2 * i + 1]), less), l2);
            s2[i & 1] = add2(s2[i & 1], make_float2(exp2_fast(e.x), exp2_fast(e.y)));
        }
        s2[0] = add2(s2[0], s2[1]);
        sum = s2[0].x + s2[0].y;
        mx = m;
    }
    __device__ __forceinline__ void end(const GemmTile& t) {
        if (t.row < p.T && t.col0 < p.V) p.part[static_cast<size_t>(t.row) * p.P + (t.col0 >> 7)] = make_float2(mx, sum);
    }
};

// Backward epilogue of the logits: G / c in bf16, columns counted from the
// piece's first word v0.
struct GradInputs {
    const float* lse;
    const float* dloss;
    float* cmax;
    const long long* target;
    long long ignore, v0;
    int T, V, n;  // n: words of the piece
};
// -lse and dloss / c of a token; d stays 0 for one without a gradient.
__device__ __forceinline__ void token_factors(const GradInputs& q, float c, int token, long long y, float& less, float& d) {
    less = -__ldg(q.lse + token);
    if (y != q.ignore && y >= 0 && y < q.V && c != 0.f) d = __fdiv_rn(__ldg(q.dloss + token), c);
}

// |dloss| of a token that counts; magnitudes order like their bits, NaN above all.
__device__ __forceinline__ unsigned weight_bits(const float* dloss, const long long* target, long long ignore, int t) {
    return target[t] != ignore ? __float_as_uint(dloss[t]) & 0x7FFFFFFFu : 0u;
}

struct GradTile {
    struct Params {
        CUtensorMap g;
        GradInputs q;
    };
    static __device__ __forceinline__ void prefetch(const Params& p) { prefetch_tmap(&p.g); }
    const Params& p;
    float less, d;
    long long tcol;
    bool some_zero;  // a row of this warp has d = 0
    __device__ __forceinline__ explicit GradTile(const Params& r) : p(r), less(0.f), d(0.f), tcol(-1), some_zero(false) {}
    __device__ __forceinline__ void begin(const GemmTile& t) {
        d = 0.f;
        tcol = -1;
        if (t.row < p.q.T) {
            const long long y = __ldg(p.q.target + t.row);
            token_factors(p.q, *p.q.cmax, t.row, y, less, d);
            tcol = y - p.q.v0 - t.col0;
        }
        some_zero = __any_sync(0xFFFFFFFFu, d == 0.f);
    }
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        const float2 l2 = both(kLog2e), ls = both(less);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            // the difference first: for a likely word it is small and exact
            const float2 e = mul2(add2(make_float2(v[i], v[i + 1]), ls), l2);
            v[i] = exp2_fast(e.x);
            v[i + 1] = exp2_fast(e.y);
        }
        const long long tc = tcol - 32 * k;
        if (tc >= 0 && tc < 32) {
            const uint32_t hot = 1u << tc;  // by a bit: see LsePart
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] -= (hot & (1u << i)) ? 1.0f : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 g = mul2(make_float2(v[i], v[i + 1]), both(d));
            v[i] = g.x;
            v[i + 1] = g.y;
        }
        if (some_zero) {
            // not by 0 * exp: an ignored token's logits may be NaN or overflow
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = d == 0.f ? 0.f : v[i];
        }
        put_bf16(t, k, v, &p.g);
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// ---------------------------------------------------------------- a few tokens
// Up to kFewTokens the logits' tiles are turned: 256 words x 64 or 128 tokens
// instead of 256 tokens, most of them past the end, x 256 words.  A thread then
// holds one word's logits of 32 tokens, and a warp's 32 words are a part of the row.
// 64 x 128000 x 896: 53 us forward, 66% of the copy bandwidth (70 us not turned), 58 us
// for G (49 with the logits in one sum).  Neither memory nor L2 is at its limit there (52%
// of DRAM's peak, 36 bytes/ns to an SM); what sets the pace is not known.  One token x 15710 x 1440: 15.5 us (19), of which 5 are the launch.
constexpr int kFewTokens = 128;

// Reduces 32 values over the 32 lanes; lane l gets value l's result (norm.cu's
// warp_sums: each step halves the values a lane carries).
template <class Op>
__device__ __forceinline__ float reduce_to_lanes(float (&v)[32], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 32, off = 16; n > 1; n >>= 1, off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, off));
        }
    }
    return v[0];
}

// The lane (0..31) whose word is the target of each lane's token, or -1.
__device__ __forceinline__ int target_lane(long long y, long long first_word) {
    const long long d = y - first_word;
    return d >= 0 && d < 32 ? static_cast<int>(d) : -1;
}

// Forward: part[t][p] = (max, sum of exp(z - max)) over words 32 p .. + 31.
struct LseWords {
    using Params = LsePart::Params;
    static __device__ __forceinline__ void prefetch(const Params&) {}
    const Params& p;
    __device__ __forceinline__ explicit LseWords(const Params& q) : p(q) {}
    __device__ __forceinline__ void begin(const GemmTile&) {}
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        const int c0 = t.col0 + 32 * k, token = c0 + t.lane;
        if (c0 >= p.T || t.warp_row >= p.V) return;
        if (t.row >= p.V) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = -INFINITY;
        }
        const int at = token < p.T ? target_lane(__ldg(p.target + token), t.warp_row) : -1;
        if (__any_sync(0xFFFFFFFFu, at >= 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (__shfl_sync(0xFFFFFFFFu, at, i) == t.lane) p.tlogit[c0 + i] = v[i];
        }
        float w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = v[i];
        const float m = reduce_to_lanes(w, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = exp2_fast((v[i] - __shfl_sync(0xFFFFFFFFu, m, i)) * kLog2e);
        const float sum = reduce_to_lanes(v, [](float a, float b) { return a + b; });
        if (token < p.T) p.part[static_cast<size_t>(token) * p.P + (t.warp_row >> 5)] = make_float2(m, sum);
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// Backward: G / c as two bf16 values, the second what the first rounds off,
// written along the words like GradTile's.
struct GradWords {
    struct Params {
        CUtensorMap g, g_low;
        GradInputs q;
    };
    static __device__ __forceinline__ void prefetch(const Params& p) {
        prefetch_tmap(&p.g);
        prefetch_tmap(&p.g_low);
    }
    const Params& p;
    float c;
    // c of a few tokens by each warp itself (a kernel less); kept for the products
    __device__ __forceinline__ explicit GradWords(const Params& r) : p(r) {
        unsigned m = 0;
        for (int t = threadIdx.x & 31; t < p.q.T; t += 32) m = max(m, weight_bits(p.q.dloss, p.q.target, p.q.ignore, t));
        c = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m));
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.q.cmax = c;
    }
    __device__ __forceinline__ void begin(const GemmTile&) {}
    // 32 tokens x 32 words from tokens' pairs in registers (thread: one word)
    // through a box (64B swizzle) to column warp_row, row c0 of the map.
    __device__ __forceinline__ void put(GemmTile& t, int c0, const uint32_t (&h)[16], const CUtensorMap* map) {
        uint8_t* const box = t.box + (t.stores & 1) * gm::BOX;  // two boxes: MH = 1
        ++t.stores;
        if (t.lane == 0) bulk_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t a = smem_u32(box + i * 64 + (((t.lane >> 3) ^ ((i >> 1) & 3)) << 4) + (t.lane & 7) * 2);
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)))) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (t.lane == 0) tma_store_2d(map, smem_u32(box), t.warp_row, c0);
    }
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        const GradInputs& q = p.q;
        const int c0 = t.col0 + 32 * k, token = c0 + t.lane;
        if (c0 >= q.T) return;
        float less = 0.f, d = 0.f;
        int at = -1;
        if (token < q.T) {
            const long long y = __ldg(q.target + token);
            token_factors(q, c, token, y, less, d);
            at = target_lane(y, q.v0 + t.warp_row);
        }
        const bool hot = __any_sync(0xFFFFFFFFu, at >= 0), inside = t.row < q.n;
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = exp2_fast((v[i] + __shfl_sync(0xFFFFFFFFu, less, i)) * kLog2e);
            if (hot) v[i] -= __shfl_sync(0xFFFFFFFFu, at, i) == t.lane ? 1.0f : 0.0f;
            const float di = __shfl_sync(0xFFFFFFFFu, d, i);
            // words past the last, which the products read, and ignored tokens (see GradTile): zeros
            v[i] = inside && di != 0.f ? v[i] * di : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        put(t, c0, h, &p.g);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            h[i] = pack_bf16(v[2 * i] - __uint_as_float(h[i] << 16), v[2 * i + 1] - __uint_as_float(h[i] & 0xFFFF0000u));
        put(t, c0, h, &p.g_low);
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// fp32 tiles stored to, or added to, a matrix (dX over the pieces).
struct SumF32 {
    struct Params {
        CUtensorMap out;
        int add, rows, row_mask;  // row_mask: 127 when rows 128 .. 255 are the second part's sums, else -1
    };
    static __device__ __forceinline__ void prefetch(const Params& p) { prefetch_tmap(&p.out); }
    const Params& p;
    __device__ __forceinline__ explicit SumF32(const Params& q) : p(q) {}
    __device__ __forceinline__ void begin(const GemmTile&) {}
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
        if ((t.warp_row & p.row_mask) < p.rows) put_f32(t, k, v, &p.out, 0, p.add != 0);  // later rows are the next part's
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// c times the tile, in bf16 (dW of a piece).
struct ScaledBf16 {
    struct Params {
        CUtensorMap out;
        const float* cmax;
    };
    static __device__ __forceinline__ void prefetch(const Params& p) { prefetch_tmap(&p.out); }
    const Params& p;
    float c;
    __device__ __forceinline__ explicit ScaledBf16(const Params& q) : p(q), c(*q.cmax) {}
    __device__ __forceinline__ void begin(const GemmTile&) {}
    __device__ __forceinline__ void slice(GemmTile& t, int k, float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= c;
        put_bf16(t, k, v, &p.out);
    }
    __device__ __forceinline__ void end(const GemmTile&) {}
};

// Joins the P parts of a row, in a fixed order: WARPS warps per row.
template <int WARPS>
__global__ void __launch_bounds__(256)
    xent_merge_kernel(const float2* __restrict__ part, const float* __restrict__ tlogit,
                      const long long* __restrict__ target, long long ignore, int T, int V, int P,
                      float* __restrict__ loss, float* __restrict__ lse_out, unsigned* status) {
    constexpr int STEP = 32 * WARPS;
    __shared__ float2 joined[WARPS];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = blockIdx.x * static_cast<long long>(8 / WARPS) + warp / WARPS;
    if (t >= T) return;  // WARPS = 8: the whole block
    const float2* const row = part + static_cast<size_t>(t) * P;
    // every part has a column, so its sum has a term 1 (or is NaN); the empty
    // start of a lane past the last part has the sum 0
    float m = -INFINITY, sum = 0.f;
    auto join = [&](float qm, float qs) {
        const float n = fmaxf(m, qm);
        sum = (sum == 0.f ? 0.f : sum * exp2_fast((m - n) * kLog2e)) + (qs == 0.f ? 0.f : qs * exp2_fast((qm - n) * kLog2e));
        m = n;
    };
    int p = warp % WARPS * 32 + lane;
    for (; p + 3 * STEP < P; p += 4 * STEP) {  // four loads in flight
        const float2 a = __ldg(row + p), b = __ldg(row + p + STEP), c = __ldg(row + p + 2 * STEP), d = __ldg(row + p + 3 * STEP);
        const float n = fmaxf(fmaxf(m, fmaxf(a.x, b.x)), fmaxf(c.x, d.x));
        const float s0 = a.y * exp2_fast((a.x - n) * kLog2e) + b.y * exp2_fast((b.x - n) * kLog2e);
        const float s1 = c.y * exp2_fast((c.x - n) * kLog2e) + d.y * exp2_fast((d.x - n) * kLog2e);
        sum = (sum == 0.f ? 0.f : sum * exp2_fast((m - n) * kLog2e)) + (s0 + s1);
        m = n;
    }
    for (; p < P; p += STEP) {
        const float2 q = __ldg(row + p);
        join(q.x, q.y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        join(__shfl_xor_sync(0xFFFFFFFFu, m, off), __shfl_xor_sync(0xFFFFFFFFu, sum, off));
    if constexpr (WARPS > 1) {
        if (lane == 0) joined[warp] = make_float2(m, sum);
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) join(joined[w].x, joined[w].y);
    }
    if (lane != 0) return;
    const float log_sum = logf(sum);
    const long long y = target[t];
    float l = 0.f;
    if (y != ignore) {
        if (y >= 0 && y < V) {
            // not lse - z: for a likely word both are large and the loss is what their
            // rounding would leave
            l = (m - tlogit[t]) + log_sum;
        } else {
            raise_status(status, kStatusInvalid);
            l = NAN;
        }
    }
    loss[t] = l;
    lse_out[t] = m + log_sum;
}

// c = max |dloss[t]| over the tokens that count (NaN if one is NaN).
__global__ void __launch_bounds__(1024) xent_cmax_kernel(const float* __restrict__ dloss,
                                                         const long long* __restrict__ target, long long ignore,
                                                         int T, float* __restrict__ cmax) {
    __shared__ unsigned s[32];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    unsigned m = 0;
    for (int t = threadIdx.x; t < T; t += 1024) m = max(m, weight_bits(dloss, target, ignore, t));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = __reduce_max_sync(0xFFFFFFFFu, s[threadIdx.x]);
        if (threadIdx.x == 0) *cmax = __uint_as_float(m);
    }
}

// dX = c * (the parts' fp32 sums, added in a fixed order), in bf16; 8 elements per
// thread and slice of the parts.  Eight slices for many parts, which come from few
// rows: one thread adding 64 parts of them took 12 us.
template <int SLICES>
__global__ void __launch_bounds__(256) xent_dx_kernel(const float* __restrict__ sums, const float* __restrict__ cmax,
                                                      long long n8, int parts, long long part8,
                                                      uint16_t* __restrict__ dx) {
    constexpr int COLS = 256 / SLICES;
    __shared__ float4 slice_sum[SLICES > 1 ? SLICES : 1][2][COLS];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float c = *cmax;
    const int col = threadIdx.x % COLS, slice = threadIdx.x / COLS;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    auto add = [&](const float4& u, const float4& v) {
        a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
        b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w;
    };
    for (long long base = static_cast<long long>(blockIdx.x) * COLS; base < n8; base += static_cast<long long>(gridDim.x) * COLS) {
        const long long i = base + col;
        const float4* const p = reinterpret_cast<const float4*>(sums) + 2 * i;
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n8)
#pragma unroll 4
            for (int s = slice; s < parts; s += SLICES) add(p[2 * s * part8], p[2 * s * part8 + 1]);
        if constexpr (SLICES > 1) {
            slice_sum[slice][0][col] = a;
            slice_sum[slice][1][col] = b;
            __syncthreads();
            if (slice == 0)
#pragma unroll
                for (int s = 1; s < SLICES; ++s) add(slice_sum[s][0][col], slice_sum[s][1][col]);
            __syncthreads();
        }
        if (slice == 0 && i < n8)
            reinterpret_cast<uint4*>(dx)[i] = make_uint4(pack_bf16(a.x * c, a.y * c), pack_bf16(a.z * c, a.w * c),
                                                         pack_bf16(b.x * c, b.y * c), pack_bf16(b.z * c, b.w * c));
    }
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int parts(long long T, long long V) { return static_cast<int>(T <= kFewTokens ? (V + 31) / 32 : (V + 127) / 128); }

// One segment holds a logit's whole sum: tall tiles need none.
bool one_segment(long long D) { return D <= kLogitSegment * gm::BK; }

// Words per piece of the backward: at most 2^28 entries of G (512 MB).  Smaller
// pieces stay in L2 but cost more launches and more passes over dX's sums
// (8192 x 128000 x 896: 2^26 entries 7.96 ms, 2^28 6.93 ms, 2^29 6.70 ms).
long long piece_words(long long T, long long V) {
    const long long most = (1ll << 28) / (T < 256 ? 256 : T);
    long long w = most / 256 * 256;
    if (w < 2048) w = 2048;
    const long long all = (V + 255) / 256 * 256;
    return w < all ? w : all;
}

// Up to kFewTokens G goes as two bf16 parts: the rounding of a token's
// one large entry, its target's, moves a whole row of dX and dW together, and
// over a few tokens such errors do not average out (1 to 8 tokens: up to 1.75
// times the error that rounding the results alone leaves).  The second part's MMAs have
// room: the tensor pipe is 48% busy with both (64 x 128000 x 896).
bool g_parts(long long T) { return T <= kFewTokens; }

// With G in two parts they lie in the two CTAs' rows of one A (GemmShape::stack),
// each with sums of its own, instead of in two A of 256 rows: half the MMAs.
long long dx_rows(long long T) { return g_parts(T) ? 2 * gm::BM : (T + 31) / 32 * 32; }

// dX has few tiles (T / 512 x D / 256) and a long reduction over the words, so it
// may be cut into parts, each with its own fp32 sums over the pieces, which
// xent_dx_kernel adds in order.  dX and dW of a piece run as one launch where one
// height of tiles suits both (8192 x 128000 x 896: loss and gradients 6.43 ms
// together, 6.73 apart; 4112 x 2066 x 2944, tall dX tiles and flat dW ones: both
// products 99 us apart, 121 together).  (The plan is
// of both also when one is wanted: the same bits.)
struct GradPlan {
    int splits, lead;
    bool together, tall_x, tall_w;
};
GradPlan make_grad_plan(long long T, long long D, long long V) {
    const long long words = piece_words(T, V) < V ? piece_words(T, V) : V, cols = (D + gm::BN - 1) / gm::BN;
    const double bytes = (g_parts(T) ? 8.0 : 4.0) * T * D;
    const GemmWork none{0, 1, 0.0, 0.0, 0.0, 1};
    auto x = [&](bool tall) {
        return GemmWork{(T + (tall ? 511 : 255)) / (tall ? 512 : 256) * cols, (words + gm::BK - 1) / gm::BK,
                        tall ? 0.8 : g_parts(T) ? 0.52 : 0.55, tall ? 2.5 : 1.0, bytes, 64};
    };
    auto w = [&](bool tall) {
        return GemmWork{(words + (tall ? 511 : 255)) / (tall ? 512 : 256) * cols, (T + gm::BK - 1) / gm::BK,
                        tall || g_parts(T) ? 0.8 : 0.55, tall ? 2.5 : 1.0, 0.0, 1};
    };
    GemmPlan best = gemm_plan(x(false), w(false));
    GradPlan plan{best.splits1, best.lead, true, false, false};
    if (g_parts(T)) return plan;
    const GemmPlan tall = gemm_plan(x(true), w(true));
    if (tall.us < best.us) {
        best = tall;
        plan = GradPlan{best.splits1, best.lead, true, true, true};
    }
    const GemmPlan xs[2] = {gemm_plan(x(false), none), gemm_plan(x(true), none)};
    const GemmPlan ws[2] = {gemm_plan(w(false), none), gemm_plan(w(true), none)};
    const bool tx = xs[1].us < xs[0].us, tw = ws[1].us < ws[0].us;
    if (xs[tx].us + ws[tw].us + 3.0 < best.us) plan = GradPlan{xs[tx].splits1, 0, false, tx, tw};
    return plan;
}
// Asked for three times a call (workspace, its check, the launch) at 2 us: the
// thread's last sizes are remembered.
GradPlan grad_plan(long long T, long long D, long long V) {
    thread_local long long sizes[3] = {};
    thread_local GradPlan plan = {};
    if (sizes[0] != T || sizes[1] != D || sizes[2] != V) {
        plan = make_grad_plan(T, D, V);
        sizes[0] = T;
        sizes[1] = D;
        sizes[2] = V;
    }
    return plan;
}

}  // namespace

size_t xent_workspace_bytes(long long T, long long V) {
    return round256(static_cast<size_t>(parts(T, V)) * T * sizeof(float2)) + round256(static_cast<size_t>(T) * sizeof(float));
}

size_t xent_backward_workspace_bytes(long long T, long long D, long long V, int need_dx) {
    return 256 + (need_dx ? round256(static_cast<size_t>(grad_plan(T, D, V).splits) * dx_rows(T) * D * sizeof(float)) : 0) +
           round256(static_cast<size_t>(T) * piece_words(T, V) * (g_parts(T) ? 4 : 2));
}

cudaError_t launch_xent(const uint16_t* x, long long T, long long D, const uint16_t* w, long long V,
                        const long long* target, long long ignore, float* loss, float* lse, void* ws, unsigned* status,
                        cudaStream_t st) {
    float2* part = static_cast<float2*>(ws);
    float* tlogit = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                             round256(static_cast<size_t>(parts(T, V)) * T * sizeof(float2)));
    const int Ti = static_cast<int>(T), Vi = static_cast<int>(V), Di = static_cast<int>(D);
    const LsePart::Params p{part, tlogit, target, Ti, Vi, parts(T, V)};
    CUtensorMap a, b;
    cudaError_t e;
    if (T <= kFewTokens) {
        const int box = T <= 64 ? 32 : 64;
        if (!gemm_operand(&a, false, false, w, V, D, D, gemm_a_box(V)) || !gemm_operand(&b, false, false, x, T, D, D, box))
            return cudaErrorInvalidValue;
        const GemmShape shape{Vi, Ti, Di, 0, 1, 1, 0, gemm_a_box(V), 0, 0};
        e = T <= 64 ? launch_gemm_f16<LseWords, 1, 1, false, false, false, kFewSegment, 64>(a, b, p, shape, status, st)
                    : launch_gemm_f16<LseWords, 1, 1, false, false, false, kFewSegment, 128>(a, b, p, shape, status, st);
    } else {
        if (!gemm_operand(&a, false, false, x, T, D, D) || !gemm_operand(&b, false, false, w, V, D, D))
            return cudaErrorInvalidValue;
        const GemmShape shape{Ti, Vi, Di, 0, 8, 1, 0, gm::BM, 0, 0};
        const bool tall = one_segment(D) && gemm_tall(T, V, 1);
        e = T <= 256 ? launch_gemm_f16<LsePart, 1, 1, false, false, false, kFewSegment>(a, b, p, shape, status, st)
            : tall   ? launch_gemm_f16<LsePart, 1, 2, false, false, false, 0>(a, b, p, shape, status, st)
                     : launch_gemm_f16<LsePart, 1, 1, false, false, false, kLogitSegment>(a, b, p, shape, status, st);
    }
    if (e != cudaSuccess) return e;
    // a block per row for few rows (64 x 128000: 15 us with a warp each, 5 so; 333 x 50001: 3.3, 4.0)
    auto merge = [&](auto kern, int rows_per_block) {
        return pdl_launch(kern, dim3(static_cast<unsigned>((T + rows_per_block - 1) / rows_per_block)), dim3(256), 0, st,
                          static_cast<const float2*>(part), static_cast<const float*>(tlogit), target, ignore,
                          static_cast<int>(T), static_cast<int>(V), parts(T, V), loss, lse, status);
    };
    return T <= 256 ? merge(xent_merge_kernel<8>, 1) : merge(xent_merge_kernel<1>, 8);
}

cudaError_t launch_xent_backward(const float* dloss, const uint16_t* x, long long T, long long D, const uint16_t* w,
                                 long long V, const long long* target, long long ignore, const float* lse, uint16_t* dx,
                                 uint16_t* dw, void* ws, unsigned* status, int num_sms, cudaStream_t st) {
    const GradPlan plan = grad_plan(T, D, V);
    const int splits = plan.splits;
    const long long rows = dx_rows(T);
    uint8_t* at = static_cast<uint8_t*>(ws);
    float* cmax = reinterpret_cast<float*>(at);
    at += 256;
    float* dx32 = nullptr;
    if (dx) {
        dx32 = reinterpret_cast<float*>(at);
        at += round256(static_cast<size_t>(splits) * rows * D * sizeof(float));
    }
    uint16_t* g = reinterpret_cast<uint16_t*>(at);
    const long long piece = piece_words(T, V);
    const bool parts = g_parts(T);
    const long long pitch = parts ? 2 * piece : piece;
    cudaError_t e = cudaSuccess;
    if (!parts) e = pdl_launch(xent_cmax_kernel, dim3(1), dim3(1024), 0, st, dloss, target, ignore, static_cast<int>(T), cmax);
    const int Ti = static_cast<int>(T), Di = static_cast<int>(D);
    const int d_panel = (Di + gm::BN - 1) / gm::BN;
    for (long long v0 = 0; v0 < V && e == cudaSuccess; v0 += piece) {
        const long long n = V - v0 < piece ? V - v0 : piece;
        const int ni = static_cast<int>(n);
        const uint16_t* wp = w + v0 * D;
        const GradInputs in{lse, dloss, cmax, target, ignore, v0, Ti, static_cast<int>(V), ni};
        CUtensorMap xk, wk;
        if (parts) {
            const int box = T <= 64 ? 32 : 64;
            GradWords::Params p;
            p.q = in;
            if (!gemm_operand(&wk, false, false, wp, n, D, D, gemm_a_box(n)) || !gemm_operand(&xk, false, false, x, T, D, D, box) ||
                !gemm_result_bf16(&p.g, g, T, piece, pitch) || !gemm_result_bf16(&p.g_low, g + piece, T, piece, pitch))
                return cudaErrorInvalidValue;
            const GemmShape shape{ni, Ti, Di, 0, 1, 1, 0, gemm_a_box(n), 0, 0};
            e = T <= 64 ? launch_gemm_f16<GradWords, 1, 1, false, false, false, kFewSegment, 64>(wk, xk, p, shape, status, st)
                        : launch_gemm_f16<GradWords, 1, 1, false, false, false, kFewSegment, 128>(wk, xk, p, shape, status, st);
        } else {
            GradTile::Params p;
            p.q = in;
            if (!gemm_operand(&xk, false, false, x, T, D, D) || !gemm_operand(&wk, false, false, wp, n, D, D) ||
                !gemm_result_bf16(&p.g, g, T, n, pitch))
                return cudaErrorInvalidValue;
            const GemmShape shape{Ti, ni, Di, 0, 8, 1, 0, gm::BM, 0, 0};
            e = T <= 256 ? launch_gemm_f16<GradTile, 1, 1, false, false, false, kFewSegment>(xk, wk, p, shape, status, st)
                : one_segment(D) && gemm_tall(T, n, 1)
                    ? launch_gemm_f16<GradTile, 1, 2, false, false, false, 0>(xk, wk, p, shape, status, st)
                    : launch_gemm_f16<GradTile, 1, 1, false, false, false, kLogitSegment>(xk, wk, p, shape, status, st);
        }
        if (e != cudaSuccess) return e;
        const long long g_cols = parts ? piece + n : n;
        const int low = static_cast<int>(piece);  // columns from a part to the next
        using DxJob = GemmJob<SumF32, 1, false, true>;
        using DwJob = GemmJob<ScaledBf16, 1, true, true>;
        using DwParts = GemmJob<ScaledBf16, 2, true, true>;
        GemmArgs<DxJob> gx;
        GemmArgs<DwJob> gw;
        memset(&gx, 0, sizeof(gx));
        memset(&gw, 0, sizeof(gw));
        if (dx) {
            gx.p.add = v0 > 0;
            gx.p.rows = Ti;
            gx.p.row_mask = parts ? gm::BM - 1 : -1;
            if (!gemm_operand(&gx.a, false, false, g, T, g_cols, pitch, gemm_a_box(T)) ||
                !gemm_operand(&gx.b, false, true, wp, n, D, D) || !gemm_result_f32(&gx.p.out, dx32, splits * rows, D))
                return cudaErrorInvalidValue;
            gx.shape = GemmShape{Ti, Di, ni, 0, d_panel, splits, static_cast<int>(rows), gemm_a_box(T), 0, parts ? low : 0};
        }
        if (dw) {
            gw.p.cmax = cmax;
            if (!gemm_operand(&gw.a, false, true, g, T, g_cols, pitch) || !gemm_operand(&gw.b, false, true, x, T, D, D) ||
                !gemm_result_bf16(&gw.p.out, dw + v0 * D, n, D, D))
                return cudaErrorInvalidValue;
            gw.shape = GemmShape{ni, Di, Ti, low, d_panel, 1, 0, gm::BM, plan.lead, 0};
        }
        const GemmArgs<DwParts> gp{gw.a, gw.b, gw.p, gw.shape};
        const GemmArgs<GemmNoJob> none{};
        if (dx && dw && plan.together) {
            e = parts         ? launch_gemm_jobs<DxJob, DwParts, 1, false, 0>(gx, gp, status, st)
                : plan.tall_x ? launch_gemm_jobs<DxJob, DwJob, 2, false, 0>(gx, gw, status, st)
                              : launch_gemm_jobs<DxJob, DwJob, 1, false, 0>(gx, gw, status, st);
            continue;
        }
        if (dx)
            e = plan.tall_x ? launch_gemm_jobs<DxJob, GemmNoJob, 2, false, 0>(gx, none, status, st)
                            : launch_gemm_jobs<DxJob, GemmNoJob, 1, false, 0>(gx, none, status, st);
        if (dw && e == cudaSuccess)
            e = parts         ? launch_gemm_jobs<DwParts, GemmNoJob, 1, false, 0>(gp, none, status, st)
                : plan.tall_w ? launch_gemm_jobs<DwJob, GemmNoJob, 2, false, 0>(gw, none, status, st)
                              : launch_gemm_jobs<DwJob, GemmNoJob, 1, false, 0>(gw, none, status, st);
    }
    if (e == cudaSuccess && dx) {
        const int sums = parts ? 2 * splits : splits;
        const long long n8 = T * D / 8, part8 = (parts ? gm::BM : rows) * D / 8, most = 8ll * num_sms;
        auto sum_up = [&](auto kern, int cols) {
            const long long blocks = (n8 + cols - 1) / cols;
            return pdl_launch(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, st,
                              static_cast<const float*>(dx32), static_cast<const float*>(cmax), n8, sums, part8, dx);
        };
        e = sums > 8 ? sum_up(xent_dx_kernel<8>, 32) : sum_up(xent_dx_kernel<1>, 256);
    }
    return e;
}

}  // namespace sbl
