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
// and writes dx.  A thread owns 8 columns for as many rows as its block takes
// (weights, and in the backward the column sums, stay in its registers); a
// group of ceil(K / 256) warps shares a row, and takes R rows at a time so
// that one barrier serves R rows and R rows of loads are in flight.  All sums
// are fp32; the variance is the sum of squared differences from the mean (two
// passes over registers, none over memory).  Column sums: each block adds its
// rows in order, norm_colsum_kernel adds the blocks' partial rows in order,
// so results do not depend on timing.  Rows longer than kMaxColumns take the
// wide kernels, which walk a row in shared blocks of threads and read it again
// from L2 in each pass.
#include <cstdint>
#include <cuda_runtime.h>

#include "sbl_common.cuh"

namespace sbl {

namespace nrm {
constexpr int COLS = 8;              // columns per thread
constexpr int kMaxColumns = 8192;    // 1024 threads x 8
constexpr int WIDE_THREADS = 512;
}  // namespace nrm

struct Bf16Row {
    using type = uint16_t;
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = ldg_stream(p); }
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
// all N).  `red`: this group's N * wpr floats for this call; a block alternates
// between two such areas, so one barrier per call is enough.  Every thread of
// the block calls this together.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int wpr, int warp_in_group, float* red) {
    const int lane = threadIdx.x & 31;
    float s = warp_sums<N>(v);
    if (wpr > 1) {
        if (lane % (32 / N) == 0) red[warp_in_group * N + lane / (32 / N)] = s;
        __syncthreads();
        s = 0.f;
        for (int e = lane / N; e < wpr; e += 32 / N) s += red[e * N + lane % N];
#pragma unroll
        for (int off = N; off < 32; off <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i * (32 / N));
    }
}

// MAXT: most threads a block of this instance has (its register budget).
template <typename Row, bool LAYER, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : (MAXT <= 512 ? 2 : 1))
    norm_fwd_kernel(const typename Row::type* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                    float eps, long long T, int K, int wpr, typename Row::type* __restrict__ y,
                    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float red[2][32 * R];
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / wpr, wig = warp % wpr, groups = (blockDim.x >> 5) / wpr;
    const int col = (wig * 32 + lane) * nrm::COLS;
    const bool active = col < K;
    const float inv_k = 1.0f / static_cast<float>(K);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float wv[8], bv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[i] = bv[i] = 0.f;
    if (active) {
        load8(w + col, wv);
        if (b) load8(b + col, bv);
    }
    const long long step = static_cast<long long>(gridDim.x) * groups * R;
    // the loop bound is the block's first row, so all its threads meet at the barriers
    for (long long base = static_cast<long long>(blockIdx.x) * groups * R; base < T; base += step) {
        const long long row0 = base + static_cast<long long>(group) * R;
        Row raw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (active && row0 + r < T) raw[r].load(x + (row0 + r) * K + col);
            else raw[r].zero();
        }
        float mean[R], sq[R];
        if (LAYER) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float f[8];
                raw[r].get(f);
                mean[r] = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            }
            group_sums<R>(mean, wpr, wig, red[0] + group * wpr * R);
#pragma unroll
            for (int r = 0; r < R; ++r) mean[r] *= inv_k;
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) mean[r] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float f[8];
            raw[r].get(f);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float d0 = f[i] - mean[r], d1 = f[i + 1] - mean[r];
                s0 = fmaf(d0, d0, s0);
                s1 = fmaf(d1, d1, s1);
            }
            sq[r] = active ? s0 + s1 : 0.f;
        }
        group_sums<R>(sq, wpr, wig, red[1] + group * wpr * R);
        // the RMS form has one barrier per trip: a second one keeps the next
        // trip's sums out of the area that slower warps still read
        if (!LAYER && wpr > 1) __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= T) continue;
            const float rstd = 1.0f / sqrtf(fmaf(sq[r], inv_k, eps));
            if (active) {
                float f[8];
                raw[r].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = fmaf((f[i] - mean[r]) * rstd, wv[i], bv[i]);
                Row::store(y + (row0 + r) * K + col, f);
            }
            if (wig == 0 && lane == 0) {
                if (mean_out) mean_out[row0 + r] = mean[r];
                if (rstd_out) rstd_out[row0 + r] = rstd;
            }
        }
    }
}

// part: NULL (only dx is wanted) or [gridDim.x][2][K], the block's sums of
// dy * xhat and of dy.
template <typename Row, bool LAYER, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 3 : 1)
    norm_bwd_kernel(const typename Row::type* __restrict__ dy, const typename Row::type* __restrict__ x,
                    const float* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                    long long T, int K, int wpr, typename Row::type* __restrict__ dx, float* __restrict__ part) {
    constexpr int N = LAYER ? 2 * R : R;
    __shared__ float red[2][32 * N];
    __shared__ float comb[8 * 32 * 16];  // column sums of the groups of a block (at most 8 warps share it)
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / wpr, wig = warp % wpr, groups = (blockDim.x >> 5) / wpr;
    const int col = (wig * 32 + lane) * nrm::COLS;
    const bool active = col < K;
    const float inv_k = 1.0f / static_cast<float>(K);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float wv[8], dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[i] = dw[i] = db[i] = 0.f;
    if (active) load8(w + col, wv);
    const long long step = static_cast<long long>(gridDim.x) * groups * R;
    int flip = 0;
    for (long long base = static_cast<long long>(blockIdx.x) * groups * R; base < T; base += step, flip ^= 1) {
        const long long row0 = base + static_cast<long long>(group) * R;
        Row rx[R], rdy[R];
        float mean[R], rstd[R], sums[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = row0 + r < T;
            if (active && in) {
                rx[r].load(x + (row0 + r) * K + col);
                rdy[r].load(dy + (row0 + r) * K + col);
            } else {
                rx[r].zero();
                rdy[r].zero();
            }
            mean[r] = LAYER && in ? __ldg(mean_in + row0 + r) : 0.f;
            rstd[r] = in ? __ldg(rstd_in + row0 + r) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float f[8], g[8];
            rx[r].get(f);
            rdy[r].get(g);
            float s = 0.f, q = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (f[i] - mean[r]) * rstd[r];
                const float qi = g[i] * wv[i];
                s = fmaf(qi, xh, s);
                q += qi;
                if (active) {
                    dw[i] = fmaf(g[i], xh, dw[i]);
                    db[i] += g[i];
                }
            }
            sums[r] = active ? s : 0.f;
            if (LAYER) sums[R + r] = q;
        }
        if (dx) {
            group_sums<N>(sums, wpr, wig, red[flip] + group * wpr * N);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!active || row0 + r >= T) continue;
                float f[8], g[8];
                rx[r].get(f);
                rdy[r].get(g);
                const float c1 = sums[r] * inv_k, c0 = LAYER ? sums[R + r] * inv_k : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (f[i] - mean[r]) * rstd[r];
                    f[i] = rstd[r] * fmaf(-xh, c1, fmaf(g[i], wv[i], -c0));
                }
                Row::store(dx + (row0 + r) * K + col, f);
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
    if (active) {
        float* const p = part + static_cast<size_t>(blockIdx.x) * 2 * K + col;
        F32Row::store(p, dw);
        F32Row::store(p + K, db);
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
            mean = block_sum(s, red) * inv_k;
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
struct RowPlan {
    int wpr, groups, threads;
};
// Warps per row, and rows side by side in blocks of up to 8 warps.
RowPlan row_plan(long long K) {
    RowPlan p;
    p.wpr = static_cast<int>((K / nrm::COLS + 31) / 32);
    p.groups = p.wpr >= 8 ? 1 : 8 / p.wpr;
    p.threads = p.wpr * p.groups * 32;
    return p;
}
// Rows per trip of the backward: 64 registers a thread (blocks over 640
// threads) hold half as many.
int bwd_rows(int bf16, int threads) { return (bf16 ? 4 : 2) / (threads > 640 ? 2 : 1); }
int bwd_blocks(long long T, long long K, int bf16, int num_sms) {
    if (K > nrm::kMaxColumns) return static_cast<int>(T < 32 ? T : 32);
    const RowPlan p = row_plan(K);
    const long long rows = static_cast<long long>(p.groups) * bwd_rows(bf16, p.threads);
    const long long want = (T + rows - 1) / rows;
    const long long most = static_cast<long long>(num_sms) * (p.threads <= 256 ? 3 : 1);
    return static_cast<int>(want < most ? want : most);
}

template <typename Row, bool LAYER, int R>
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
    const RowPlan p = row_plan(K);
    const long long want = (T + p.groups * R - 1) / (p.groups * R);
    const long long most = static_cast<long long>(num_sms) * (p.threads <= 256 ? 4 : (p.threads <= 512 ? 2 : 1));
    const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(p.threads);
    auto kern = p.threads <= 256 ? norm_fwd_kernel<Row, LAYER, R, 256>
                : p.threads <= 512 ? norm_fwd_kernel<Row, LAYER, R, 512>
                                   : norm_fwd_kernel<Row, LAYER, R, 1024>;
    return pdl_launch(kern, grid, block, 0, st, xp, w, b, eps, T, static_cast<int>(K), p.wpr, yp, mean, rstd);
}

template <typename Row, bool LAYER, int R>
cudaError_t bwd(const void* dy, const void* x, const float* w, const float* mean, const float* rstd, long long T,
                long long K, void* dx, float* dw, float* db, float* part, int bf16, int num_sms, cudaStream_t st) {
    using E = typename Row::type;
    const E* xp = static_cast<const E*>(x);
    const E* dyp = static_cast<const E*>(dy);
    E* dxp = static_cast<E*>(dx);
    const bool sums = dw || db;
    const int P = bwd_blocks(T, K, bf16, num_sms);
    const int Ki = static_cast<int>(K);
    cudaError_t e = cudaSuccess;
    if (K > nrm::kMaxColumns) {
        if (sums)
            e = pdl_launch(norm_wide_part_kernel<Row, LAYER>, dim3(static_cast<unsigned>((K + 2047) / 2048), P),
                           dim3(256), 0, st, dyp, xp, mean, rstd, T, Ki, part);
        if (e == cudaSuccess && sums)
            e = pdl_launch(norm_colsum_kernel, dim3(static_cast<unsigned>((2 * K + 31) / 32)), dim3(1024), 0, st,
                           static_cast<const float*>(part), P, Ki, dw, db);
        if (e == cudaSuccess && dx) {
            const long long most = 4ll * num_sms;
            e = pdl_launch(norm_bwd_wide_kernel<Row, LAYER>, dim3(static_cast<unsigned>(T < most ? T : most)),
                           dim3(nrm::WIDE_THREADS), 0, st, dyp, xp, w, mean, rstd, T, Ki, dxp);
        }
        return e;
    }
    const RowPlan p = row_plan(K);
    auto kern = p.threads <= 256 ? norm_bwd_kernel<Row, LAYER, R, 256>
                : p.threads <= 640 ? norm_bwd_kernel<Row, LAYER, R, 640>
                                   : norm_bwd_kernel<Row, LAYER, R / 2, 1024>;
    e = pdl_launch(kern, dim3(P), dim3(p.threads), 0, st, dyp, xp, w, mean, rstd, T, Ki, p.wpr, dxp,
                   sums ? part : static_cast<float*>(nullptr));
    if (e == cudaSuccess && sums)
        e = pdl_launch(norm_colsum_kernel, dim3(static_cast<unsigned>((2 * K + 31) / 32)), dim3(1024), 0, st,
                       static_cast<const float*>(part), P, Ki, dw, db);
    return e;
}
}  // namespace

// Bytes of the partial column sums of launch_norm_bwd.
size_t norm_bwd_part_bytes(long long T, long long K, int bf16, int num_sms) {
    return static_cast<size_t>(bwd_blocks(T, K, bf16, num_sms)) * 2 * static_cast<size_t>(K) * sizeof(float);
}

cudaError_t launch_norm_fwd(const void* x, int bf16, int layer, const float* w, const float* b, float eps, long long T,
                            long long K, void* y, float* mean, float* rstd, int num_sms, cudaStream_t st) {
    if (bf16)
        return layer ? fwd<Bf16Row, true, 4>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st)
                     : fwd<Bf16Row, false, 4>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st);
    return layer ? fwd<F32Row, true, 2>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st)
                 : fwd<F32Row, false, 2>(x, w, b, eps, T, K, y, mean, rstd, num_sms, st);
}

cudaError_t launch_norm_bwd(const void* dy, const void* x, int bf16, int layer, const float* w, const float* mean,
                            const float* rstd, long long T, long long K, void* dx, float* dw, float* db, float* part,
                            int num_sms, cudaStream_t st) {
    if (bf16)
        return layer ? bwd<Bf16Row, true, 4>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, bf16, num_sms, st)
                     : bwd<Bf16Row, false, 4>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, bf16, num_sms, st);
    return layer ? bwd<F32Row, true, 2>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, bf16, num_sms, st)
                 : bwd<F32Row, false, 2>(dy, x, w, mean, rstd, T, K, dx, dw, db, part, bf16, num_sms, st);
}

}  // namespace sbl
