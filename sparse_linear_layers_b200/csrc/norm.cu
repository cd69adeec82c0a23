// Layer norm and RMS norm of rows, forward and backward.
//
//   forward   xhat = (x - mean) * rstd,  y = xhat * w + b
//             mean = sum_k x / K (0 for the RMS form), rstd = 1 / sqrt(sum_k (x - mean)^2 / K + eps)
//   backward  with q = dy * w:
//             dx = rstd * (q - sum_k q / K - xhat * sum_k (q * xhat) / K)   (RMS form: without the middle term)
//             dw = sum_t dy * xhat,  db = sum_t dy
//
// (The RMSNorm in front of the Sparse-BitNet Guide's layer, "Mathematical
// Formulation of Sparse-BitLinear"; the layer form is torch's LayerNorm.)
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and dy
// and writes dx.  What keeps a simple kernel from that bound is the instruction
// count (30 per element with 8 columns a thread, a quarter of them a sum's
// shuffles), so a thread takes up to 32 columns of two rows and the arithmetic
// runs on pairs of fp32 values.  All sums are fp32; the variance is the sum of
// squared differences from the mean, which is divided, not multiplied by 1 / K: a
// constant row, whose sum is exact in bf16, then has exactly its value as the mean
// (K = 896: 3.0 came out as 3 - 2^-22, which rstd = 316 makes 7e-5).
//
// Forward: a group of warps holds its rows in registers between the sums and
// the results; weights come from L1 once per two rows.  16384 x 4864 bf16:
// 61 us, 79% of the copy bandwidth (8 columns, one row: 108 us).
// Backward, many rows: one persistent block per
// SM whose column sums stay in registers.  A producer warp copies tiles of
// whole rows (contiguous in memory) into a ring in shared memory with bulk
// asynchronous copies, so loads are in flight whatever the sums wait for, and
// the consumer warps read each tile twice from shared memory.  16384 x 4864
// bf16: 92 us, 79%.
// Backward, few rows: a row per group at a time straight from global memory,
// without the ring's set-up (64 x 2048 bf16: 6.5 us, the ring 9.8 us).
// Longer rows than kMaxColumns: the wide kernels, which read a row again from L2
// in each pass.
//
// Column sums: a block adds its rows in order, norm_colsum_kernel adds the
// blocks' partial rows in order, so results do not depend on timing.
#include <cstdint>
#include <cuda_runtime.h>

#include "sbl_common.cuh"

namespace sbl {

namespace nrm {
constexpr int COLS = 8;              // columns of one read
constexpr int kMaxDirect = 8192;     // 1024 threads x 8
constexpr int kMaxColumns = 10240;   // 10 warps x 32 x 32
constexpr int WIDE_THREADS = 512;
constexpr int STREAM_WARPS = 11;     // consumer warps of a stream block, at most (168 registers a thread)
constexpr int STREAM_THREADS = (STREAM_WARPS + 1) * 32;
constexpr int MAX_STAGES = 8;
constexpr int RING_BYTES = 200 * 1024;
constexpr int FWD_THREADS = 320;     // 10 warps: a row of kMaxColumns
constexpr int FWD_BLOCKS = 2;        // of those per SM: 96 registers a thread
}  // namespace nrm

struct Bf16Row {
    using type = uint16_t;
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = ldg_stream(p); }
    __device__ __forceinline__ void load_shared(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the one rounding of the result: nearest even
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct F32Row {
    using type = float;
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ldg_stream(p);
        b = ldg_stream(p + 4);
    }
    __device__ __forceinline__ void load_shared(const float* p) {
        a = *reinterpret_cast<const uint4*>(p);
        b = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <class Row>
__device__ __forceinline__ void get_pairs(const Row& r, float2 (&f)[4]) {
    float v[8];
    r.get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}
template <class Row>
__device__ __forceinline__ void store_pairs(typename Row::type* p, const float2 (&f)[4]) {
    const float v[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    Row::store(p, v);
}
__device__ __forceinline__ void load_pairs(const float* p, float2 (&f)[4]) {
    float v[8];
    load8(p, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// Sums of N values over the 32 lanes: each step halves the values a lane
// carries and adds the other half's from its partner, so N values cost about
// N + 5 - log2(N) shuffles.  Lane l ends with the sum of value l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int off = 16;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[i + n / 2];
            const float keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, off);
        }
    }
#pragma unroll
    for (; off > 0; off >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], off);
    return v[0];
}

// Sums of N values over the warps of a row group (all 32 * wpr threads get
// all N).  `red`: this group's N * wpr floats for this call; callers alternate
// between two such areas, so one barrier per call is enough.  `barrier` joins
// the group's threads (or more of the block, which then call this together).
template <int N, class Barrier>
__device__ __forceinline__ void group_sums(float (&v)[N], int wpr, int warp_in_group, float* red, Barrier barrier) {
    const int lane = threadIdx.x & 31;
    float s = warp_sums<N>(v);
    if (wpr > 1) {
        if (lane % (32 / N) == 0) red[warp_in_group * N + lane / (32 / N)] = s;
        barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = red[i];
#pragma unroll 4
        for (int e = 1; e < wpr; ++e)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += red[e * N + i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i * (32 / N));
    }
}

// ---------------------------------------------------------------- forward
// R rows per group of wpr warps, NC * 8 columns of each per thread in
// registers.  R = 2 halves what the weights cost: they come from L1, whose
// bandwidth bounds the kernel with one row (80% busy at 42% of DRAM's).
template <typename Row, bool LAYER, int NC, int R>
__global__ void __launch_bounds__(NC == 1 && R == 1 ? 1024 : nrm::FWD_THREADS, NC == 1 && R == 1 ? 1 : nrm::FWD_BLOCKS)
    norm_fwd_kernel(const typename Row::type* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                    float eps, long long T, int K, int wpr, typename Row::type* __restrict__ y,
                    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float red[2][32 * R];
    asm volatile("griddepcontrol.launch_dependents;");
    const int wig = threadIdx.x >> 5, group = threadIdx.y;  // rows of one group per threadIdx.y
    const int col0 = threadIdx.x * nrm::COLS, span = wpr * 32 * nrm::COLS;
    const float inv_k = 1.0f / static_cast<float>(K);
    const long long t0 = (static_cast<long long>(blockIdx.x) * blockDim.y + group) * R;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto barrier = [] { __syncthreads(); };
    const typename Row::type* const xr = x + t0 * K + col0;
    auto in = [&](int r, int c) { return col0 + c * span < K && t0 + r < T; };
    float2 f[R][NC][4];
    {
        Row raw[R][NC];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (in(r, c)) raw[r][c].load(xr + r * K + c * span);
                else raw[r][c].zero();
            }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) get_pairs(raw[r][c], f[r][c]);
    }
    float mean[R], sq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = 0.f;
    if (LAYER) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                sum = add2(sum, add2(add2(f[r][c][0], f[r][c][1]), add2(f[r][c][2], f[r][c][3])));
            mean[r] = sum.x + sum.y;
        }
        group_sums<R>(mean, wpr, wig, red[0] + group * wpr * R, barrier);
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = __fdiv_rn(mean[r], static_cast<float>(K));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
        const float2 less = both(-mean[r]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (LAYER) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[r][c][i] = add2(f[r][c][i], less);
            }
            if (in(r, c)) {
                s0 = fma2(f[r][c][0], f[r][c][0], s0);
                s1 = fma2(f[r][c][1], f[r][c][1], s1);
                s0 = fma2(f[r][c][2], f[r][c][2], s0);
                s1 = fma2(f[r][c][3], f[r][c][3], s1);
            }
        }
        s0 = add2(s0, s1);
        sq[r] = s0.x + s0.y;
    }
    group_sums<R>(sq, wpr, wig, red[1] + group * wpr * R, barrier);
    float rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] = 1.0f / sqrtf(fmaf(sq[r], inv_k, eps));
    typename Row::type* const yr = y + t0 * K + col0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (!in(0, c)) continue;
        float2 wv[4], bv[4];
        load_pairs(w + col0 + c * span, wv);
        if (b) load_pairs(b + col0 + c * span, bv);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!in(r, c)) continue;
            const float2 r2 = both(rstd[r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 n = mul2(f[r][c][i], r2);
                f[r][c][i] = b ? fma2(n, wv[i], bv[i]) : mul2(n, wv[i]);
            }
            store_pairs<Row>(yr + r * K + c * span, f[r][c]);
        }
    }
    if (threadIdx.x == 0)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (t0 + r < T) {
                if (LAYER && mean_out) mean_out[t0 + r] = mean[r];
                if (rstd_out) rstd_out[t0 + r] = rstd[r];
            }
}

// ---------------------------------------------------------------- backward of few rows
// part: NULL (only dx is wanted) or [gridDim.x][2][K], the block's sums of
// dy * xhat and of dy.
template <typename Row, bool LAYER>
__global__ void __launch_bounds__(1024)
    norm_bwd_kernel(const typename Row::type* __restrict__ dy, const typename Row::type* __restrict__ x,
                    const float* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                    long long T, int K, int wpr, typename Row::type* __restrict__ dx, float* __restrict__ part) {
    constexpr int N = LAYER ? 2 : 1;
    __shared__ float red[2][32 * N];
    __shared__ float comb[8 * 32 * 16];  // column sums of the groups of a block (at most 8 warps share it)
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / wpr, wig = warp % wpr, groups = (blockDim.x >> 5) / wpr;
    const int col = (wig * 32 + lane) * nrm::COLS;
    const float inv_k = 1.0f / static_cast<float>(K);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto barrier = [] { __syncthreads(); };
    float wv[8], dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[i] = dw[i] = db[i] = 0.f;
    if (col < K) load8(w + col, wv);
    const long long step = static_cast<long long>(gridDim.x) * groups;
    int flip = 0;
    // the loop bound is the block's first row, so all its threads meet at the barriers
    for (long long base = static_cast<long long>(blockIdx.x) * groups; base < T; base += step, flip ^= 1) {
        const long long t = base + group;
        const bool active = col < K && t < T;
        Row rx, rdy;
        rx.zero();
        rdy.zero();
        float mean = 0.f, rstd = 0.f;
        if (active) {
            rx.load(x + t * K + col);
            rdy.load(dy + t * K + col);
            if (LAYER) mean = __ldg(mean_in + t);
            rstd = __ldg(rstd_in + t);
        }
        float xh[8], g[8], sums[N];
        rx.get(xh);
        rdy.get(g);
        float s = 0.f, q = 0.f;
        if (active) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[i] = (xh[i] - mean) * rstd;
                dw[i] = fmaf(g[i], xh[i], dw[i]);
                db[i] += g[i];
                g[i] *= wv[i];
                s = fmaf(g[i], xh[i], s);
                q += g[i];
            }
        }
        sums[0] = s;
        if (LAYER) sums[N - 1] = q;
        if (dx) {
            group_sums<N>(sums, wpr, wig, red[flip] + group * wpr * N, barrier);
            if (active) {
                const float c1 = sums[0] * inv_k, c0 = LAYER ? sums[N - 1] * inv_k : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = rstd * fmaf(-xh[i], c1, g[i] - c0);
                Row::store(dx + t * K + col, g);
            }
        }
    }
    if (!part) return;
    if (groups > 1) {
        float* const mine = comb + (warp * 32 + lane) * 16;
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mine[i] = dw[i];
                mine[8 + i] = db[i];
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int g = 1; g < groups; ++g) {
            const float* const other = comb + ((g * wpr + wig) * 32 + lane) * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] += other[i];
                db[i] += other[8 + i];
            }
        }
    }
    if (col < K) {
        float* const p = part + static_cast<size_t>(blockIdx.x) * 2 * K + col;
        F32Row::store(p, dw);
        F32Row::store(p + K, db);
    }
}

// ---------------------------------------------------------------- backward of many rows
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The ring of a stream block: tile i (rows i * rows .. + rows - 1 of every one
// of NSRC matrices) goes to stage i / gridDim.x mod stages.
struct StreamPlan {
    int wpr, groups;    // warps per row, rows side by side
    int rows;           // rows of a tile: groups * R
    int stages;
    int stage_bytes;    // of one matrix
};

struct StreamBars {
    uint64_t full[nrm::MAX_STAGES];
    uint64_t empty[nrm::MAX_STAGES];
    int abort_flag;
};

template <int NSRC>
__device__ __forceinline__ void stream_producer(const char* s0, const char* s1, long long T, int row_bytes,
                                                const StreamPlan& p, char* ring, StreamBars* bars, unsigned* status) {
    const long long tiles = (T + p.rows - 1) / p.rows;
    uint32_t it = 0;
    for (long long i = blockIdx.x; i < tiles; i += gridDim.x, ++it) {
        const int s = it % p.stages;
        if (!mbar_wait(&bars->empty[s], ((it / p.stages) & 1) ^ 1, &bars->abort_flag)) {
            bars->abort_flag = 1;
            raise_status(status, kStatusTimeout);
            break;
        }
        const long long row0 = i * p.rows;
        const uint32_t bytes = static_cast<uint32_t>((T - row0 < p.rows ? T - row0 : p.rows) * row_bytes);
        mbar_arrive_expect_tx(&bars->full[s], NSRC * bytes);
        char* const dst = ring + static_cast<size_t>(s) * NSRC * p.stage_bytes;
        bulk_load(dst, s0 + row0 * row_bytes, bytes, &bars->full[s]);
        if (NSRC == 2) bulk_load(dst + p.stage_bytes, s1 + row0 * row_bytes, bytes, &bars->full[s]);
    }
    // let the issued copies land before the block can exit
    volatile int never = 0;
    for (uint32_t j = it > static_cast<uint32_t>(p.stages) ? it - p.stages : 0; j < it; ++j)
        if (!mbar_wait(&bars->full[j % p.stages], (j / p.stages) & 1, &never)) raise_status(status, kStatusTimeout);
}

__device__ __forceinline__ void stream_init(StreamBars* bars, const StreamPlan& p) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], p.wpr * p.groups);
        }
        bars->abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
}

// Barrier 1 + group joins the warps of a row group.
__device__ __forceinline__ void group_barrier(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

// part: NULL or [gridDim.x][2][K], as in norm_bwd_kernel.
template <typename Row, bool LAYER, int NC, int R>
__global__ void __launch_bounds__(nrm::STREAM_THREADS, 1)
    norm_bwd_stream_kernel(const typename Row::type* __restrict__ dy, const typename Row::type* __restrict__ x,
                           const float* __restrict__ w, const float* __restrict__ mean_in,
                           const float* __restrict__ rstd_in, long long T, int K, const StreamPlan p,
                           typename Row::type* __restrict__ dx, float* __restrict__ part, unsigned* status) {
    using E = typename Row::type;
    constexpr int N = LAYER ? 2 * R : R;
    extern __shared__ __align__(128) char ring[];
    __shared__ StreamBars bars;
    __shared__ float red[2][nrm::STREAM_WARPS * N];
    asm volatile("griddepcontrol.launch_dependents;");
    stream_init(&bars, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int consumers = p.wpr * p.groups;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == consumers) {
        if (lane == 0)
            stream_producer<2>(reinterpret_cast<const char*>(x), reinterpret_cast<const char*>(dy), T,
                               K * static_cast<int>(sizeof(E)), p, ring, &bars, status);
        __syncwarp();
        if (part && p.groups > 1) __syncthreads();  // the consumers' hand-over below
        return;
    }
    const int group = warp / p.wpr, wig = warp % p.wpr, span = p.wpr * 32 * nrm::COLS;
    const int col0 = (wig * 32 + lane) * nrm::COLS;
    const float inv_k = 1.0f / static_cast<float>(K);
    auto barrier = [&] { group_barrier(group, p.wpr * 32); };
    float2 wv[NC][4], dw[NC][4], db[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[c][i] = dw[c][i] = db[c][i] = make_float2(0.f, 0.f);
        if (col0 + c * span < K) load_pairs(w + col0 + c * span, wv[c]);
    }
    const long long tiles = (T + p.rows - 1) / p.rows;
    uint32_t it = 0;
    bool ok = true;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++it) {
        const long long row0 = tile * p.rows + group * R;
        float mean[R], rstd[R], sums[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = row0 + r < T;
            mean[r] = LAYER && in ? __ldg(mean_in + row0 + r) : 0.f;
            rstd[r] = in ? __ldg(rstd_in + row0 + r) : 0.f;
        }
        const int s = it % p.stages;
        if (ok && !mbar_wait(&bars.full[s], (it / p.stages) & 1, &bars.abort_flag)) {
            bars.abort_flag = 1;
            raise_status(status, kStatusTimeout);
            ok = false;  // keep meeting at the barriers
        }
        const E* const sx = reinterpret_cast<const E*>(ring + static_cast<size_t>(s) * 2 * p.stage_bytes) +
                            static_cast<size_t>(group) * R * K + col0;
        const E* const sdy = reinterpret_cast<const E*>(reinterpret_cast<const char*>(sx) + p.stage_bytes);
        auto each = [&](int r, int c, float2 (&f)[4], float2 (&g)[4]) {
            Row a, d;
            a.load_shared(sx + r * K + c * span);
            d.load_shared(sdy + r * K + c * span);
            get_pairs(a, f);
            get_pairs(d, g);
        };
        // xhat = (x - mean) * rstd, as in the other kernels: of a mean far from 0,
        // x * rstd - mean * rstd would keep the rounding of mean * rstd, and its one
        // instruction less gains nothing (16384 x 4864 bf16: the same 92 us)
        float2 scale[R], less[R];
        auto xhat = [](float2 f, float2 less_r, float2 scale_r) { return mul2(LAYER ? add2(f, less_r) : f, scale_r); };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            scale[r] = both(rstd[r]);
            less[r] = both(-mean[r]);
            float2 s1 = make_float2(0.f, 0.f), s0 = s1;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (col0 + c * span < K && row0 + r < T) {
                    float2 f[4], g[4];
                    each(r, c, f, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 xh = xhat(f[i], less[r], scale[r]);
                        const float2 q = mul2(g[i], wv[c][i]);
                        s1 = fma2(q, xh, s1);
                        if (LAYER) s0 = add2(s0, q);
                        dw[c][i] = fma2(g[i], xh, dw[c][i]);
                        db[c][i] = add2(db[c][i], g[i]);
                    }
                }
            sums[r] = s1.x + s1.y;
            if (LAYER) sums[N - R + r] = s0.x + s0.y;
        }
        if (dx) {
            group_sums<N>(sums, p.wpr, wig, red[it & 1] + group * p.wpr * N, barrier);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (row0 + r >= T) continue;
                // dx = q * rstd - xhat * (rstd c1) - rstd c0
                const float2 c1 = both(-rstd[r] * (sums[r] * inv_k));
                const float2 c0 = LAYER ? both(-rstd[r] * (sums[N - R + r] * inv_k)) : make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (col0 + c * span < K) {
                        float2 f[4], g[4];
                        each(r, c, f, g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 xh = xhat(f[i], less[r], scale[r]);
                            const float2 q = mul2(g[i], wv[c][i]);
                            f[i] = fma2(xh, c1, LAYER ? fma2(q, scale[r], c0) : mul2(q, scale[r]));
                        }
                        store_pairs<Row>(dx + (row0 + r) * K + col0 + c * span, f);
                    }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.empty[s]);
    }
    if (!part) return;
    if (p.groups > 1) {
        // the groups' sums through shared memory (the ring is free: every copy
        // has landed and every tile has been read)
        float* const comb = reinterpret_cast<float*>(ring);
        __syncthreads();
        if (group > 0)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (col0 + c * span < K) {
                    float* const mine = comb + static_cast<size_t>(group - 1) * 2 * K + col0 + c * span;
                    store_pairs<F32Row>(mine, dw[c]);
                    store_pairs<F32Row>(mine + K, db[c]);
                }
        asm volatile("bar.sync 0, %0;" ::"r"(consumers * 32) : "memory");
        if (group > 0) return;
        for (int g = 1; g < p.groups; ++g)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (col0 + c * span < K) {
                    const float* const other = comb + static_cast<size_t>(g - 1) * 2 * K + col0 + c * span;
                    float2 ow[4], ob[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ow[i] = reinterpret_cast<const float2*>(other)[i];
                        ob[i] = reinterpret_cast<const float2*>(other + K)[i];
                        dw[c][i] = add2(dw[c][i], ow[i]);
                        db[c][i] = add2(db[c][i], ob[i]);
                    }
                }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (col0 + c * span < K) {
            float* const q = part + static_cast<size_t>(blockIdx.x) * 2 * K + col0 + c * span;
            store_pairs<F32Row>(q, dw[c]);
            store_pairs<F32Row>(q + K, db[c]);
        }
}

// dw, db: the sums of the P partial rows [P][2][K], in a fixed order: a thread
// takes every 32nd row of one column, then its block adds the 32 sums.
__global__ void __launch_bounds__(1024)
    norm_colsum_kernel(const float* __restrict__ part, int P, int K, float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;  // column of [2][K]
    float a = 0.f;
    if (c < 2ll * K)
        for (int p = slice; p < P; p += 32) a += __ldg(part + static_cast<size_t>(p) * 2 * K + c);
    s[slice][lane] = a;
    __syncthreads();
    if (slice != 0 || c >= 2ll * K) return;
    float t = 0.f;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    if (c < K) {
        if (dw) dw[c] = t;
    } else if (db) {
        db[c - K] = t;
    }
}

// ---------------------------------------------------------------- long rows
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < nrm::WIDE_THREADS / 32; ++i) s += red[i];
    return s;
}

template <typename Row, bool LAYER>
__global__ void __launch_bounds__(nrm::WIDE_THREADS)
    norm_fwd_wide_kernel(const typename Row::type* x, const float* __restrict__ w, const float* __restrict__ b, float eps,
                         long long T, int K, typename Row::type* y, float* __restrict__ mean_out,
                         float* __restrict__ rstd_out) {
    __shared__ float red[nrm::WIDE_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float inv_k = 1.0f / static_cast<float>(K);
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        const typename Row::type* const xr = x + t * K;
        Row raw;
        float f[8];
        float mean = 0.f;
        if (LAYER) {
            float s = 0.f;
            for (int c = threadIdx.x * 8; c < K; c += nrm::WIDE_THREADS * 8) {
                raw.load(xr + c);
                raw.get(f);
                s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            }
            mean = __fdiv_rn(block_sum(s, red), static_cast<float>(K));
        }
        float q = 0.f;
        for (int c = threadIdx.x * 8; c < K; c += nrm::WIDE_THREADS * 8) {
            raw.load(xr + c);
            raw.get(f);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(f[i] - mean, f[i] - mean, s);
            q += s;
        }
        const float rstd = 1.0f / sqrtf(fmaf(block_sum(q, red), inv_k, eps));
        for (int c = threadIdx.x * 8; c < K; c += nrm::WIDE_THREADS * 8) {
            float wv[8], bv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            raw.load(xr + c);
            raw.get(f);
            load8(w + c, wv);
            if (b) load8(b + c, bv);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf((f[i] - mean) * rstd, wv[i], bv[i]);
            Row::store(y + t * K + c, f);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[t] = mean;
            if (rstd_out) rstd_out[t] = rstd;
        }
    }
}

template <typename Row, bool LAYER>
__global__ void __launch_bounds__(nrm::WIDE_THREADS)
    norm_bwd_wide_kernel(const typename Row::type* dy, const typename Row::type* x, const float* __restrict__ w,
                         const float* __restrict__ mean_in, const float* __restrict__ rstd_in, long long T, int K,
                         typename Row::type* dx) {
    __shared__ float red[nrm::WIDE_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float inv_k = 1.0f / static_cast<float>(K);
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        const float mean = LAYER ? mean_in[t] : 0.f, rstd = rstd_in[t];
        Row rx, rdy;
        float f[8], g[8], wv[8];
        float s = 0.f, q = 0.f;
        for (int c = threadIdx.x * 8; c < K; c += nrm::WIDE_THREADS * 8) {
            rx.load(x + t * K + c);
            rdy.load(dy + t * K + c);
            rx.get(f);
            rdy.get(g);
            load8(w + c, wv);
            float s8 = 0.f, q8 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float qi = g[i] * wv[i];
                s8 = fmaf(qi, (f[i] - mean) * rstd, s8);
                q8 += qi;
            }
            s += s8;
            q += q8;
        }
        const float c1 = block_sum(s, red) * inv_k;
        const float c0 = LAYER ? block_sum(q, red) * inv_k : 0.f;
        for (int c = threadIdx.x * 8; c < K; c += nrm::WIDE_THREADS * 8) {
            rx.load(x + t * K + c);
            rdy.load(dy + t * K + c);
            rx.get(f);
            rdy.get(g);
            load8(w + c, wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (f[i] - mean) * rstd;
                f[i] = rstd * fmaf(-xh, c1, fmaf(g[i], wv[i], -c0));
            }
            Row::store(dx + t * K + c, f);
        }
    }
}

// Partial column sums of long rows: block (c, p) sums rows p, p + P, ... of
// 256 * 8 columns into part[p].
template <typename Row, bool LAYER>
__global__ void __launch_bounds__(256)
    norm_wide_part_kernel(const typename Row::type* __restrict__ dy, const typename Row::type* __restrict__ x,
                          const float* __restrict__ mean_in, const float* __restrict__ rstd_in, long long T, int K,
                          float* __restrict__ part) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= K) return;
    float dw[8], db[8], f[8], g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
    for (long long t = blockIdx.y; t < T; t += gridDim.y) {
        Row rx, rdy;
        rx.load(x + t * K + c);
        rdy.load(dy + t * K + c);
        rx.get(f);
        rdy.get(g);
        const float mean = LAYER ? __ldg(mean_in + t) : 0.f, rstd = __ldg(rstd_in + t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = fmaf(g[i], (f[i] - mean) * rstd, dw[i]);
            db[i] += g[i];
        }
    }
    float* const p = part + static_cast<size_t>(blockIdx.y) * 2 * K + c;
    F32Row::store(p, dw);
    F32Row::store(p + K, db);
}

// ---------------------------------------------------------------- host side
namespace {
// Warps per row with nc * 8 columns per thread, and rows side by side in
// blocks of up to `warps` warps.
struct RowPlan {
    int wpr, groups, threads;
};
RowPlan row_plan(long long K, int nc, int warps) {
    RowPlan p;
    p.wpr = static_cast<int>((K / nrm::COLS + 32 * nc - 1) / (32 * nc));
    p.groups = p.wpr >= warps ? 1 : warps / p.wpr;
    p.threads = p.wpr * p.groups * 32;
    return p;
}

// Columns per thread where there are rows for every warp: a sum's shuffles and
// barriers then serve 32 elements (with 8 the sums alone were half of 30
// instructions per element).
int columns_per_thread(long long K) { return K <= 256 ? 1 : K <= 512 ? 2 : 4; }

// The backward's ring: `es`-byte elements, rows that leave warps over side by
// side, R rows each; R = 1 where two tiles of R = 2 do not fit.
struct StreamChoice {
    StreamPlan plan;
    int nc, r, grid, smem;
};
bool stream_choice(long long T, long long K, int es, int num_sms, StreamChoice& c) {
    if (K > nrm::kMaxColumns) return false;
    c.nc = columns_per_thread(K);
    StreamPlan& p = c.plan;
    const RowPlan rows = row_plan(K, c.nc, nrm::STREAM_WARPS);
    p.wpr = rows.wpr;
    p.groups = rows.groups;
    for (c.r = 2; c.r >= 1; --c.r) {
        p.rows = p.groups * c.r;
        p.stage_bytes = static_cast<int>((p.rows * K * es + 127) / 128 * 128);
        p.stages = nrm::RING_BYTES / (2 * p.stage_bytes);
        if (p.stages >= 2 || c.r == 1) break;
    }
    if (p.stages > nrm::MAX_STAGES) p.stages = nrm::MAX_STAGES;
    if (p.stages < 2) return false;
    c.grid = num_sms;
    c.smem = p.stages * 2 * p.stage_bytes;
    // both kernels, us: 1021 x 896 fp32 direct 11.3, ring 11.5 (4096: 21.3, 18.1); 592 x 2048 bf16 9.0, 10.2
    // (1021: 12.1, 10.3); 64 x 4864 bf16 7.8, 10.5 (296: 13.1, 11.0)
    return T * K > 10000ll * num_sms;
}

// Blocks of the backward, each with a partial row of column sums.
int bwd_grid(long long T, long long K, int es, int num_sms) {
    StreamChoice c;
    if (stream_choice(T, K, es, num_sms, c)) return c.grid;
    if (K > nrm::kMaxDirect) return static_cast<int>(T < 32 ? T : 32);
    const RowPlan p = row_plan(K, 1, 8);
    const long long want = (T + p.groups - 1) / p.groups;
    const long long most = 2ll * num_sms;
    return static_cast<int>(want < most ? want : most);
}

// Opts a kernel in to the largest ring, once per device (`done`: its flags).
template <typename Kern>
cudaError_t allow_ring(Kern kern, bool (&done)[64]) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, nrm::RING_BYTES)) return e;
        done[dev] = true;
    }
    return cudaSuccess;
}

template <typename Row, bool LAYER>
cudaError_t fwd(const void* x, const float* w, const float* b, float eps, long long T, long long K, void* y,
                float* mean, float* rstd, int num_sms, cudaStream_t st) {
    using E = typename Row::type;
    const E* xp = static_cast<const E*>(x);
    E* yp = static_cast<E*>(y);
    if (K > nrm::kMaxColumns) {
        const long long most = 4ll * num_sms;
        return pdl_launch(norm_fwd_wide_kernel<Row, LAYER>, dim3(static_cast<unsigned>(T < most ? T : most)),
                          dim3(nrm::WIDE_THREADS), 0, st, xp, w, b, eps, T, static_cast<int>(K), yp, mean, rstd);
    }
    // few elements: more threads per row, each with less to do (us, 8 columns and one row against
    // 32 and two: 2048 x 896 fp32 6.2, 7.5; 4096 x 896 9.2, 8.4; 592 x 2048 bf16 4.2, 4.8; 2048 x 2048 8.0, 6.2;
    // 296 x 4864 bf16 4.3, 4.8; 592 x 4864 7.5, 5.8)
    const bool few = T * K < 14000ll * num_sms && K <= nrm::kMaxDirect;
    const int nc = few ? 1 : columns_per_thread(K), r = few ? 1 : 2;
    const RowPlan p = row_plan(K, nc, 8);
    auto kern = few       ? norm_fwd_kernel<Row, LAYER, 1, 1>
                : nc == 1 ? norm_fwd_kernel<Row, LAYER, 1, 2>
                : nc == 2 ? norm_fwd_kernel<Row, LAYER, 2, 2>
                          : norm_fwd_kernel<Row, LAYER, 4, 2>;
    return pdl_launch(kern, dim3(static_cast<unsigned>((T + p.groups * r - 1) / (p.groups * r))), dim3(p.wpr * 32, p.groups), 0,
                      st, xp, w, b, eps, T, static_cast<int>(K), p.wpr, yp, mean, rstd);
}

template <typename Row, bool LAYER>
cudaError_t bwd(const void* dy, const void* x, const float* w, const float* mean, const float* rstd, long long T,
                long long K, void* dx, float* dw, float* db, float* part, unsigned* status, int num_sms,
                cudaStream_t st) {
    using E = typename Row::type;
    const E* xp = static_cast<const E*>(x);
    const E* dyp = static_cast<const E*>(dy);
    E* dxp = static_cast<E*>(dx);
    const bool sums = dw || db;
    const int P = bwd_grid(T, K, sizeof(E), num_sms);
    const int Ki = static_cast<int>(K);
    float* const part_or_null = sums ? part : nullptr;
    cudaError_t e = cudaSuccess;
    StreamChoice c;
    if (stream_choice(T, K, sizeof(E), num_sms, c)) {
        // rows of up to 512 columns always fit two at a time
        auto kern = c.nc == 1   ? norm_bwd_stream_kernel<Row, LAYER, 1, 2>
                    : c.nc == 2 ? norm_bwd_stream_kernel<Row, LAYER, 2, 2>
                    : c.r == 2  ? norm_bwd_stream_kernel<Row, LAYER, 4, 2>
                                : norm_bwd_stream_kernel<Row, LAYER, 4, 1>;
        static bool allowed[4][64] = {};
        e = allow_ring(kern, allowed[c.nc < 4 ? c.nc - 1 : 1 + c.r]);
        if (e == cudaSuccess)
            e = pdl_launch(kern, dim3(P), dim3((c.plan.wpr * c.plan.groups + 1) * 32), c.smem, st, dyp, xp, w, mean, rstd, T, Ki,
                           c.plan, dxp, part_or_null, status);
    } else if (K > nrm::kMaxDirect) {
        if (sums)
            e = pdl_launch(norm_wide_part_kernel<Row, LAYER>, dim3(static_cast<unsigned>((K + 2047) / 2048), P),
                           dim3(256), 0, st, dyp, xp, mean, rstd, T, Ki, part);
        if (e == cudaSuccess && dx) {
            const long long most = 4ll * num_sms;
            e = pdl_launch(norm_bwd_wide_kernel<Row, LAYER>, dim3(static_cast<unsigned>(T < most ? T : most)),
                           dim3(nrm::WIDE_THREADS), 0, st, dyp, xp, w, mean, rstd, T, Ki, dxp);
        }
    } else {
        const RowPlan p = row_plan(K, 1, 8);
        e = pdl_launch(norm_bwd_kernel<Row, LAYER>, dim3(P), dim3(p.threads), 0, st, dyp, xp, w, mean, rstd, T, Ki, p.wpr, dxp,
                       part_or_null);
    }
    if (e == cudaSuccess && sums)
        e = pdl_launch(norm_colsum_kernel, dim3(static_cast<unsigned>((2 * K + 31) / 32)), dim3(1024), 0, st,
                       static_cast<const float*>(part), P, Ki, dw, db);
    return e;
}
}  // namespace

// Bytes of the partial column sums of launch_norm_bwd.
size_t norm_bwd_part_bytes(long long T, long long K, int bf16, int num_sms) {
    return static_cast<size_t>(bwd_grid(T, K, bf16 ? 2 : 4, num_sms)) * 2 * static_cast<size_t>(K) * sizeof(float);
}

cudaError_t launch_norm_fwd(const void* x, int bf16, int layer, const float* w, const float* b, float eps, long long T,
                            long long K, void* y, float* mean, float* rstd, int num_sms, cudaStream_t st) {
    if (bf16)
        return layer ? fwd<Bf16Row, true>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st)
                     : fwd<Bf16Row, false>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st);
    return layer ? fwd<F32Row, true>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st)
                 : fwd<F32Row, false>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st);
}

cudaError_t launch_norm_bwd(const void* dy, const void* x, int bf16, int layer, const float* w, const float* mean,
                            const float* rstd, long long T, long long K, void* dx, float* dw, float* db, float* part,
                            unsigned* status, int num_sms, cudaStream_t st) {
    if (bf16)
        return layer ? bwd<Bf16Row, true>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, status, num_sms, st)
                     : bwd<Bf16Row, false>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, status, num_sms, st);
    return layer ? bwd<F32Row, true>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, status, num_sms, st)
                 : bwd<F32Row, false>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, status, num_sms, st);
}

}  // namespace sbl
