// A persistent 2-SM tcgen05 GEMM on bf16 or fp16 operands (kind::f16, fp32
// accumulators) whose epilogue is a template parameter:
//
//   acc[m, n] = sum_j sum_k A_j[m, k] * B[n, k],  j < NA
//
// A cluster of two CTAs computes 256 x 256 tiles.  CTA rank r stages rows
// 128 r .. + 127 of each A_j and 128 r .. + 127 of B per 64-deep k-block (TMA,
// 128B swizzle) and holds the accumulators of its 128 rows in its own tensor
// memory; the even CTA issues the MMAs (M = 256, N = 256, K = 16).  Either
// operand may be stored with k along its rows (K-major: [m, k] row-major) or
// with m or n along its rows (MN-major: [k, m] row-major, two boxes of 64
// columns per stage), so no operand is transposed in memory.
//
// MH = 1: two accumulator buffers (all 512 TMEM columns) let the eight epilogue
// warps read one while the MMAs fill the other.
// MH = 2: tiles of 512 x 256, both buffers one tile's (its upper and lower 256
// rows), so B is loaded once for twice the rows.  What feeds the MMAs bounds
// this GEMM: L2 delivers about 9 TB/s to the SMs whatever the kernel (measured on
// four of them), 60 bytes/ns to one SM, also when 15 pairs run alone; a 256 x 256
// tile takes 7.8 KB per MFLOP and a 512 x 256 one 5.9 KB.  The MMAs of the next tile wait until the epilogue has read a half, while
// the loads run on for four stages; sixteen epilogue warps read both halves at
// once to keep that wait short.  (Letting the upper half's MMAs run ahead
// through those stages made the whole 3% slower: their stages come back later.)
//
// BN_ = 64 or 128: narrow tiles for a B of few rows (K-major, one A), eight stages.
//
// SEGMENT > 0: the tensor cores round every fp32 accumulation towards zero, an
// error that grows with the number of MMAs summed into one accumulator (a
// relative 1.4e-5 after 1344 of them, measured).  The reduction is then cut
// into segments of SEGMENT k-blocks; each segment starts from zero and the
// epilogue threads add it, rounding to nearest, to sums in registers.
// Costs one 128-column TMEM read and 128 additions per thread and segment,
// hidden behind the next segment's MMAs.  The sums beside a slice being read take
// all 168 registers: 64 to 88 bytes a thread spill in the epilogue warps, 244 in the
// kernel that holds both of the feed-forward block's epilogues (0.57 ms all the same,
// 0.60 as two launches).
//
// Warps: 8 MH epilogue (warp w: TMEM lanes 32 (w % 4) .. + 31, columns
// 128 (w / 4 % 2) .. + 127 of buffer w / 8), one TMA producer, one for TMEM
// allocation and, in the even CTA, MMA issue.  Every wait is bounded; a CTA that
// gives up records a timeout, lets its loads land and its MMAs finish (bounded) and
// exits.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "sbl_common.cuh"
#include "tc_util.cuh"

namespace sbl {

namespace gm {
constexpr int BM = 128;             // rows per CTA (pair: 256)
constexpr int BN = 256;             // columns per pair tile, unless the kernel's BN_ says fewer
constexpr int BK = 64;              // reduction elements per stage (128 bytes)
constexpr int TILE = BM * BK * 2;   // one operand tile of one CTA: 16 KB
constexpr int EPI_WARPS = 8;        // per accumulator half of a tall tile
constexpr int threads(int mh) { return (EPI_WARPS * mh + 2) * 32; }
constexpr int BOX = 32 * 64;        // a staging box: 32 rows x 64 bytes; 2 / MH per epilogue warp
constexpr int BOXES = 16;
constexpr int b_tile(int bn) { return bn / 2 * BK * 2; }  // B tile of one CTA
constexpr int stages(int tiles, int bn = BN) { return bn < BN ? 8 : tiles == 1 ? 6 : 4; }  // by A tiles of a stage
}  // namespace gm

template <int AT, int BN_ = gm::BN>
struct GemmSmem {
    uint8_t a[gm::stages(AT, BN_)][AT][gm::TILE];  // 1024-byte aligned tiles
    uint8_t b[gm::stages(AT, BN_)][gm::b_tile(BN_)];
    uint8_t box[gm::BOXES][gm::BOX];
    uint64_t full[gm::stages(AT, BN_)];            // used in the even CTA
    uint64_t empty[gm::stages(AT, BN_)];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];                   // used in the even CTA
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
template <int AT, int BN_ = gm::BN>
constexpr size_t gemm_smem_bytes() {
    return sizeof(GemmSmem<AT, BN_>) + 1024;
}
static_assert(gemm_smem_bytes<1>() <= 232448 && gemm_smem_bytes<2>() <= 232448 && gemm_smem_bytes<1, 128>() <= 232448,
              "GEMM stages do not fit");

// The sizes of one launch.  Rows of A beyond M, of B beyond N and k beyond K
// are zero-filled by TMA.  a_part: columns between the A_j, which lie side by
// side in one matrix (columns of k when K-major, of m when MN-major).
struct GemmShape {
    int M, N, K;
    int a_part;
    int panel;      // consecutive tiles walk across `panel` column tiles, then down M
    int splits;     // parts of the reduction, each a GEMM of its own into rows
    int split_rows; // split_rows further down (whole staging boxes: a multiple of 32)
    int a_box;      // rows of a box of K-major A (gemm_a_box)
    int lead;       // of a second product: tiles that a pair takes first if it has one less of the first
    int stack;      // 0, or: the odd CTA's A rows are the even one's again, `stack` columns further on
                    // (K-major A of at most 128 rows); their sums are rows 128 .. 255 of the result
};

struct GemmTile {
    int m0, n0;       // first row and column of the pair's tile
    int row;          // this thread's row
    int warp_row;     // first row of this warp
    int out_row;      // where that row goes: warp_row, further down for later splits
    int col0;         // first of this warp's 128 columns
    int lane;
    uint8_t* box;     // this warp's staging boxes
    int boxes;        // one or two
    int stores;       // stores sent so far
};

// MN-major, 128-byte swizzle: 64 columns x 8 k per 1024-byte atom, atoms along
// k 1024 bytes apart, the second 64 columns a whole box (64 k x 128 bytes) on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Wait for this thread's TMEM loads; the registers pass through, so that no
// use of them can be moved before the wait.
__device__ __forceinline__ void tmem_wait_into(uint32_t (&r)[32]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ void tc_mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

// Adds a staging box to fp32 memory (each element once: no order to depend on).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 bytes of a row (four 16-byte units: 32 bf16 or 16 fp32 columns) through one
// of the warp's boxes (64B swizzle) to column `col` of the output; a box is
// written again once its last store has read it.
template <bool ADD = false>
__device__ __forceinline__ void put_64(GemmTile& t, int col, int row0, const uint4 (&w)[4], const CUtensorMap* map) {
    uint8_t* const box = t.box + (t.boxes == 2 ? t.stores & 1 : 0) * gm::BOX;
    ++t.stores;
    if (t.lane == 0) {
        if (t.boxes == 2) bulk_wait_read<1>();
        else bulk_wait_read<0>();
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        // 16-byte unit c of row r at c ^ (r / 2 mod 4)
        const uint32_t a = smem_u32(box + t.lane * 64 + ((c ^ ((t.lane >> 1) & 3)) << 4));
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[c].x), "r"(w[c].y), "r"(w[c].z), "r"(w[c].w)
                     : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (t.lane == 0) {
        if (ADD) tma_add_2d(map, smem_u32(box), col, t.out_row - row0);
        else tma_store_2d(map, smem_u32(box), col, t.out_row - row0);
    }
}
__device__ __forceinline__ void to_bf16(const float (&v)[32], uint4 (&w)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        w[c] = make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                          pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
}
// Slice k (32 columns) of a row in bf16.
__device__ __forceinline__ void put_bf16(GemmTile& t, int k, const float (&v)[32], const CUtensorMap* map) {
    uint4 w[4];
    to_bf16(v, w);
    put_64(t, t.col0 + 32 * k, 0, w, map);
}
// Slice k of a row in fp32, to rows out_row - row0 of a matrix; added to what
// is there when `add`.
__device__ __forceinline__ void put_f32(GemmTile& t, int k, const float (&v)[32], const CUtensorMap* map, int row0,
                                        bool add) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 16 * h + 4 * c;
            w[c] = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                              __float_as_uint(v[i + 3]));
        }
        if (add) put_64<true>(t, t.col0 + 32 * k + 16 * h, row0, w, map);
        else put_64(t, t.col0 + 32 * k + 16 * h, row0, w, map);
    }
}

// Epi: a struct with
//   struct Params (a kernel argument, may hold tensor maps), static prefetch(const Params&),
//   Epi(const Params&), begin(const GemmTile&), slice(GemmTile&, int k, float (&v)[32])
//   for columns col0 + 32 k .. + 31 of the thread's row (k = 0 .. BN_ / 64 - 1 in order), end(const GemmTile&).

// A product of a launch.
template <class Epi_, int NA_, bool A_MN_, bool B_MN_>
struct GemmJob {
    using Epi = Epi_;
    static constexpr int NA = NA_;
    static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
};
struct GemmNoEpi {
    struct Params {};
    __device__ __forceinline__ explicit GemmNoEpi(const Params&) {}
};
using GemmNoJob = GemmJob<GemmNoEpi, 1, false, false>;
template <class Job>
struct GemmArgs {
    CUtensorMap a, b;
    typename Job::Epi::Params p;
    GemmShape shape;
};
template <>
struct GemmArgs<GemmNoJob> {
    GemmNoEpi::Params p;
};

template <bool SECOND, class A, class B>
__device__ __forceinline__ const std::conditional_t<SECOND, B, A>& gemm_pick(const A& a, const B& b) {
    if constexpr (SECOND) return b;
    else return a;
}

// J2: a second product that does not depend on the first, in the same launch;
// its tiles follow the first's on each pair (GemmShape::lead).
template <class J1, class J2, int MH, bool FP16, int SEGMENT, int BN_ = gm::BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(gm::threads(MH), 1)
    gemm_f16_kernel(const __grid_constant__ GemmArgs<J1> g1, const __grid_constant__ GemmArgs<J2> g2, unsigned* status) {
    constexpr bool TWO = !std::is_same_v<J2, GemmNoJob>;
    constexpr int NA = J1::NA > J2::NA ? J1::NA : J2::NA;
    static_assert(MH == 1 || (NA == 1 && SEGMENT == 0), "a tall tile has one A and one sum per row");
    constexpr int AT = NA * MH;  // A tiles of a stage
    static_assert(BN_ == gm::BN || (AT == 1 && !TWO && !J1::B_MN && (BN_ == 64 || BN_ == 128)), "narrow tiles: K-major B, one A");
    constexpr int SLICES = BN_ / 64;  // 32-column slices of a warp's half of the columns
    constexpr int STAGES = gm::stages(AT, BN_);
    constexpr int ROWS = 2 * gm::BM * MH;  // rows of a tile
    constexpr int EPI = gm::EPI_WARPS * MH, WARP_TMA = EPI, WARP_MMA = EPI + 1;
    extern __shared__ uint8_t smem_raw[];
    auto* sm = reinterpret_cast<GemmSmem<AT, BN_>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int* abort_flag = &sm->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    auto tiles_of = [](const GemmShape& shape) {
        return (shape.M + ROWS - 1) / ROWS * ((shape.N + BN_ - 1) / BN_) * shape.splits;
    };
    auto blocks_of = [](const GemmShape& shape) {  // k-blocks of a part; those past the end read zeros
        return ((shape.K + gm::BK - 1) / gm::BK + shape.splits - 1) / shape.splits;
    };
    // f(which product, tile) for this pair's tiles, until it returns false
    auto for_tiles = [&](auto&& f) {
        const int n1 = tiles_of(g1.shape);
        for (int t = pair; t < n1; t += npairs)
            if (!f(std::false_type{}, t)) return;
        if constexpr (TWO) {
            // pairs with a tile less of the first product begin with `lead` of the second
            const int n2 = tiles_of(g2.shape), extra = n1 % npairs, idle = npairs - extra;
            const int order = pair >= extra ? pair - extra : idle + pair, lead = extra ? g2.shape.lead : 0;
            if (pair >= extra)
                for (int i = 0, t = order; i < lead && t < n2; ++i, t += idle)
                    if (!f(std::true_type{}, t)) return;
            for (int t = idle * lead + order; t < n2; t += npairs)
                if (!f(std::true_type{}, t)) return;
        }
    };

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 32) {
        prefetch_tmap(&g1.a);
        prefetch_tmap(&g1.b);
        J1::Epi::prefetch(g1.p);
        if constexpr (TWO) {
            prefetch_tmap(&g2.a);
            prefetch_tmap(&g2.b);
            J2::Epi::prefetch(g2.p);
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->tmem_full[b], 1);
            mbar_init(&sm->tmem_empty[b], 2 * gm::EPI_WARPS);
        }
        mbar_init(&sm->mma_done, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                     "r"(2 * BN_)
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
    // tiles go panel by panel of column tiles, row by row of a panel: the
    // panel's B tiles stay in L2 while A streams past them once per panel
    auto tile_at = [](const GemmShape& shape, int tile, int& m0, int& n0, int& split) {
        const int MT = (shape.M + ROWS - 1) / ROWS, NT = (shape.N + BN_ - 1) / BN_;
        split = shape.splits > 1 ? tile / (MT * NT) : 0;
        tile -= split * MT * NT;
        const int first = tile / (MT * shape.panel) * shape.panel;
        const int rem = tile - first * MT;
        const int width = NT - first < shape.panel ? NT - first : shape.panel;
        m0 = rem / width * ROWS;
        n0 = (first + rem % width) * BN_;
    };

    if (warp < EPI) {
        // ------------------------------------------------------------ epilogue
        const int qd = warp & 3, half = (warp >> 2) & 1;
        const uint32_t lane_addr = static_cast<uint32_t>(qd * 32) << 16;
        GemmTile t;
        t.lane = lane;
        t.boxes = 2 / MH;
        t.stores = 0;
        t.box = sm->box[warp * t.boxes];
        uint32_t seg = 0;  // accumulator buffers taken so far
        auto release = [&](int b) {  // every load of the buffer has completed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(&sm->tmem_empty[b]);
                else mbar_arrive_cluster(map_to_cta(smem_u32(&sm->tmem_empty[b]), 0));
            }
        };
        auto store_tile = [&](auto second, int tile, auto& epi) {
            const GemmShape& shape = gemm_pick<second.value>(g1, g2).shape;
            const int KB = blocks_of(shape);
            int split;
            tile_at(shape, tile, t.m0, t.n0, split);
            t.col0 = t.n0 + half * (BN_ / 2);
            if (SEGMENT > 0) {
                t.warp_row = t.m0 + static_cast<int>(rank) * gm::BM + qd * 32;
                t.row = t.warp_row + lane;
                t.out_row = t.warp_row + split * shape.split_rows;
                epi.begin(t);
                float acc[SLICES][32];
#pragma unroll
                for (int k = 0; k < SLICES; ++k)
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[k][i] = 0.f;
                for (int kb = 0; kb < KB; kb += SEGMENT > 0 ? SEGMENT : 1, ++seg) {
                    const int b = seg & 1;
                    if (!warp_wait(&sm->tmem_full[b], (seg >> 1) & 1, abort_flag)) { give_up(); return false; }
                    tc_fence_after();
                    const uint32_t tbase = tmem_base + lane_addr + b * BN_ + half * (BN_ / 2);
#pragma unroll
                    for (int k = 0; k < SLICES; ++k) {
                        uint32_t r[32];
                        tmem_ld32_nowait(tbase + 32 * k, r);
                        tmem_wait_into(r);
                        if (k == SLICES - 1) release(b);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[k][i] += __uint_as_float(r[i]);
                    }
                }
#pragma unroll
                for (int k = 0; k < SLICES; ++k) epi.slice(t, k, acc[k]);
                epi.end(t);
            } else {
                // MH = 2: this warp's half of the tile is in buffer j
                const int j = MH == 2 ? warp >> 3 : 0, b = MH == 2 ? j : seg & 1;
                const uint32_t phase = MH == 2 ? seg & 1 : (seg >> 1) & 1;
                ++seg;
                t.warp_row = t.m0 + 2 * gm::BM * j + static_cast<int>(rank) * gm::BM + qd * 32;
                t.row = t.warp_row + lane;
                t.out_row = t.warp_row + split * shape.split_rows;
                epi.begin(t);
                if (!warp_wait(&sm->tmem_full[b], phase, abort_flag)) { give_up(); return false; }
                tc_fence_after();
                const uint32_t tbase = tmem_base + lane_addr + b * BN_ + half * (BN_ / 2);
                if constexpr (MH == 2) {
                    // sixteen warps hide each other's loads
#pragma unroll
                    for (int k = 0; k < SLICES; ++k) {
                        uint32_t r[32];
                        tmem_ld32_nowait(tbase + 32 * k, r);
                        tmem_wait_into(r);
                        if (k == SLICES - 1) release(b);
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                        epi.slice(t, k, v);
                    }
                } else {
                    uint32_t ra[32], rb[32];
                    tmem_ld32_nowait(tbase, ra);
                    tmem_wait_into(ra);
#pragma unroll
                    for (int k = 0; k < SLICES; ++k) {
                        uint32_t(&cur)[32] = k & 1 ? rb : ra;
                        uint32_t(&nxt)[32] = k & 1 ? ra : rb;
                        if (k < SLICES - 1) tmem_ld32_nowait(tbase + 32 * (k + 1), nxt);
                        else release(b);
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(cur[i]);
                        epi.slice(t, k, v);
                        if (k < SLICES - 1) tmem_wait_into(nxt);
                    }
                }
                epi.end(t);
            }
            return true;
        };
        if constexpr (TWO) {  // made for each tile: both at once cost registers
            for_tiles([&](auto second, int tile) {
                typename std::conditional_t<second.value, J2, J1>::Epi epi(gemm_pick<second.value>(g1, g2).p);
                return store_tile(second, tile, epi);
            });
        } else {
            typename J1::Epi epi(g1.p);
            for_tiles([&](auto second, int tile) { return store_tile(second, tile, epi); });
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp == WARP_TMA) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t it = 0;
            for_tiles([&](auto second, int tile) {
                using Job = std::conditional_t<second.value, J2, J1>;
                constexpr int JT = Job::NA * MH;
                const auto& g = gemm_pick<second.value>(g1, g2);
                const GemmShape& shape = g.shape;
                const int KB = blocks_of(shape);
                int m0, n0, split;
                tile_at(shape, tile, m0, n0, split);
                const int arow = m0 + (shape.stack ? 0 : static_cast<int>(rank) * gm::BM);
                const int acol = rank ? shape.stack : 0, brow = n0 + static_cast<int>(rank) * (BN_ / 2);
                // boxes of A without a row are left out: what the tile holds there
                // ends in rows that no epilogue stores
                int boxes = 0;
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const int r = m0 + (MH == 2 ? 2 * gm::BM * j : 0);
                    boxes += (r < shape.M) + (r + (shape.stack ? 0 : gm::BM) < shape.M);
                }
                const uint32_t bytes = static_cast<uint32_t>(boxes * (Job::A_MN ? gm::TILE : shape.a_box * 128) + 2 * gm::b_tile(BN_));
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&sm->empty[s], ((it / STAGES) & 1) ^ 1, abort_flag)) { give_up(); return false; }
                    // the even CTA expects the bytes of both CTAs
                    if (leader) mbar_arrive_expect_tx(&sm->full[s], bytes);
                    const uint32_t full = map_to_cta(smem_u32(&sm->full[s]), 0);
                    const int k0 = (split * KB + kb) * gm::BK;
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        const uint32_t dst = smem_u32(sm->a[s][j]);
                        const int part = MH == 2 ? 0 : j * shape.a_part, r = arow + (MH == 2 ? 2 * gm::BM * j : 0);
                        if (r >= shape.M) continue;
                        if (Job::A_MN) {
                            tma_load_2d_pair(dst, &g.a, part + r, k0, full);
                            tma_load_2d_pair(dst + gm::TILE / 2, &g.a, part + r + 64, k0, full);
                        } else {
                            tma_load_2d_pair(dst, &g.a, acol + part + k0, r, full);
                        }
                    }
                    const uint32_t dst = smem_u32(sm->b[s]);
                    if (Job::B_MN) {
                        tma_load_2d_pair(dst, &g.b, brow, k0, full);
                        tma_load_2d_pair(dst + gm::TILE / 2, &g.b, brow + 64, k0, full);
                    } else {
                        tma_load_2d_pair(dst, &g.b, k0, brow, full);
                    }
                }
                return true;
            });
            // let the issued loads land before either CTA can exit (the even
            // CTA's barriers count both CTAs' loads)
            if (leader) {
                const uint32_t first = it > STAGES ? it - STAGES : 0;
                volatile int never = 0;
                for (uint32_t j = first; j < it; ++j)
                    if (!mbar_wait(&sm->full[j % STAGES], (j / STAGES) & 1, &never)) give_up();
            }
        }
    } else {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        if (lane == 0) {
            if (leader) {
                uint32_t it = 0, seg = 0;
                // buffer of the seg-th accumulation, once the epilogue has read what it held
                auto take = [&](uint32_t sg) {
                    if (!mbar_wait(&sm->tmem_empty[sg & 1], ((sg >> 1) & 1) ^ 1, abort_flag)) return false;
                    tc_fence_after();
                    return true;
                };
                auto loaded = [&](uint32_t i) { return mbar_wait(&sm->full[i % STAGES], (i / STAGES) & 1, abort_flag); };
                for_tiles([&](auto second, int) {
                    using Job = std::conditional_t<second.value, J2, J1>;
                    constexpr uint32_t idesc = (1u << 4) | (FP16 ? 0u : (1u << 7) | (1u << 10)) | (Job::A_MN ? 1u << 15 : 0u) |
                                               (Job::B_MN ? 1u << 16 : 0u) | (static_cast<uint32_t>(BN_ >> 3) << 17) |
                                               (static_cast<uint32_t>((2 * gm::BM) >> 4) << 24);
                    const int KB = blocks_of(gemm_pick<second.value>(g1, g2).shape);
                    // the MMAs of one k-block (stage of iteration i) on A tile j
                    auto issue = [&](uint32_t i, int j, uint32_t d, bool fresh) {
                        const uint32_t a0 = smem_u32(sm->a[i % STAGES][j]), b0 = smem_u32(sm->b[i % STAGES]);
#pragma unroll
                        for (int kk = 0; kk < gm::BK / 16; ++kk)
                            tc_mma_pair_f16(d, Job::A_MN ? sw128_mn_desc(a0 + kk * 2048) : sw128_desc(a0 + kk * 32),
                                            Job::B_MN ? sw128_mn_desc(b0 + kk * 2048) : sw128_desc(b0 + kk * 32), idesc,
                                            !(fresh && kk == 0));
                    };
                    for (int kb = 0; kb < KB; ++kb, ++it) {
                        bool first = kb == 0, last = kb == KB - 1;
                        if constexpr (SEGMENT > 0) {
                            first = kb % SEGMENT == 0;
                            last = last || kb % SEGMENT == SEGMENT - 1;
                        }
                        if (first && !take(seg)) { give_up(); return false; }
                        if (!loaded(it)) { give_up(); return false; }
                        tc_fence_after();
                        if constexpr (MH == 2) {
                            // upper half, then lower half; the lower buffer comes back later
                            issue(it, 0, tmem_base + (seg & 1) * BN_, first);
                            if (last) tc_commit_pair_both(&sm->tmem_full[seg & 1]);
                            if (first && !take(seg + 1)) { give_up(); return false; }
                            issue(it, 1, tmem_base + ((seg + 1) & 1) * BN_, first);
                        } else {
#pragma unroll
                            for (int j = 0; j < Job::NA; ++j) issue(it, j, tmem_base + (seg & 1) * BN_, first && j == 0);
                        }
                        tc_commit_pair_both(&sm->empty[it % STAGES]);
                        if (last) {
                            tc_commit_pair_both(&sm->tmem_full[(seg + MH - 1) & 1]);
                            seg += MH;
                        }
                    }
                    return true;
                });
                // every MMA must be complete before either CTA frees tensor memory
                tc_commit_pair_both(&sm->mma_done);
            }
            volatile int never = 0;
            if (!mbar_wait(&sm->mma_done, 0, &never)) give_up();
        }
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
    if (warp == WARP_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * BN_)
                     : "memory");
    }
}

// ---------------------------------------------------------------- host side
// Tensor map of a row-major [rows, cols] matrix of 2- or 4-byte elements with
// a box of box_cols x box_rows (rows of 128 bytes with the 128B swizzle, or of
// 64 with the 64B one).
inline bool gemm_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, long long rows, long long cols,
                     long long pitch_bytes, int box_cols, int box_rows,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const cuuint32_t estr[2] = {1, 1};
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    return enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An fp32 result, stored by put_f32.
inline bool gemm_result_f32(CUtensorMap* map, void* base, long long rows, long long cols) {
    return gemm_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, rows, cols, cols * 4, 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// A bf16 result, stored by put_bf16.
inline bool gemm_result_bf16(CUtensorMap* map, void* base, long long rows, long long cols, long long pitch_elems) {
    return gemm_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rows, cols, pitch_elems * 2, 32, 32,
                    CU_TENSOR_MAP_SWIZZLE_64B);
}

// An operand of the GEMM: a 2-byte row-major matrix [rows, cols].  K-major
// operands are read in boxes of 64 k x box_rows rows, MN-major ones in boxes of
// 64 columns x 64 k.
inline bool gemm_operand(CUtensorMap* map, bool fp16, bool mn_major, const void* base, long long rows, long long cols,
                         long long pitch_elems, int box_rows = gm::BM) {
    return gemm_map(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rows, cols,
                    pitch_elems * 2, 64, mn_major ? 64 : box_rows);
}

// Rows of a box of K-major A with M rows: whole swizzle atoms, no more than
// there are rows (1 row x 1440 against 15710 columns: 21 us with boxes of 128, 19 so).
inline int gemm_a_box(long long M) { return M < gm::BM ? static_cast<int>((M + 7) / 8 * 8) : gm::BM; }

template <class J1, class J2, int MH, bool FP16, int SEGMENT, int BN_ = gm::BN>
cudaError_t launch_gemm_jobs(const GemmArgs<J1>& g1, const GemmArgs<J2>& g2, unsigned* status, cudaStream_t stream) {
    auto kern = gemm_f16_kernel<J1, J2, MH, FP16, SEGMENT, BN_>;
    constexpr size_t smem = gemm_smem_bytes<(J1::NA > J2::NA ? J1::NA : J2::NA) * MH, BN_>();
    constexpr int rows = 2 * gm::BM * MH;
    static int clusters[64] = {};  // pairs of this kernel that fit on each device at once
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(gm::threads(MH));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    if (clusters[dev] == 0) {
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)))
            return e;
        int n = 0;
        if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) return e;
        if (n <= 0) return cudaErrorNotSupported;
        clusters[dev] = n;
    }
    auto count = [&](const GemmShape& shape) {
        return static_cast<long long>((shape.M + rows - 1) / rows) * ((shape.N + BN_ - 1) / BN_) * shape.splits;
    };
    long long tiles = count(g1.shape);
    if constexpr (!std::is_same_v<J2, GemmNoJob>) tiles += count(g2.shape);
    if (tiles <= 0 || tiles > (1ll << 30)) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < clusters[dev] ? tiles : clusters[dev]));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, g1, g2, status);
}

// One product.
template <class Epi, int NA, int MH, bool A_MN, bool B_MN, bool FP16, int SEGMENT, int BN_ = gm::BN>
cudaError_t launch_gemm_f16(const CUtensorMap& a, const CUtensorMap& b, const typename Epi::Params& p,
                            const GemmShape& shape, unsigned* status, cudaStream_t stream) {
    using Job = GemmJob<Epi, NA, A_MN, B_MN>;
    return launch_gemm_jobs<Job, GemmNoJob, MH, FP16, SEGMENT, BN_>(GemmArgs<Job>{a, b, p, shape}, GemmArgs<GemmNoJob>{}, status,
                                                                   stream);
}

// What the parts that two products' reductions are cut into cost, when each
// part's fp32 result (part_bytes) is written and read back: the tiles of both in
// one launch (the first's the longer ones) take rounds of 74 pairs of SMs, a
// k-block of a tile about us_per_block (what L2 feeds a pair: 0.55 us for 256 rows
// and one A, 0.45 to 0.52 if half of them are past the end, 0.8 for 512 rows or two A), each
// tile us_tile more (1 us; 2.5 for 512 rows, whose epilogue no MMAs hide), the sum
// over the parts 3 us and its bytes at 6 TB/s.  Alone, 1 token, 2 tiles of 619 k-blocks: 200 us in one part, 37 in 37.
struct GemmWork {
    long long tiles, KB;
    double us_per_block, us_tile, part_bytes;
    int most;  // parts at most
};
struct GemmPlan {
    int splits1, splits2, lead;
    double us;
};
inline GemmPlan gemm_plan(const GemmWork& w1, const GemmWork& w2) {
    static constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16, 18, 20, 24, 28, 32, 37, 48, 64};
    auto tile_us = [](const GemmWork& w, int s) { return static_cast<double>((w.KB + s - 1) / s) * w.us_per_block + w.us_tile; };
    auto sum_us = [](const GemmWork& w, int s) { return s > 1 ? 3.0 + s * 2.0 * w.part_bytes / 6e6 : 0.0; };
    GemmPlan best{1, 1, 0, 0.0};
    for (int s1 : kParts) {
        if (s1 > 1 && (s1 > w1.most || s1 > w1.KB)) break;
        const double l1 = tile_us(w1, s1);
        const long long n1 = w1.tiles * s1, each = n1 / 74, extra = n1 % 74, idle = 74 - extra;
        for (int s2 : kParts) {
            if (s2 > 1 && (s2 > w2.most || s2 > w2.KB || w2.tiles * s2 > 148)) break;
            const double l2 = tile_us(w2, s2);
            const long long n2 = w2.tiles * s2;
            const int lead = extra && n2 ? static_cast<int>(l1 / l2 + 0.5) : 0;  // no second product: nothing to lead with
            const long long early = n2 < idle * lead ? n2 : idle * lead, rest = n2 - early, full = rest / 74, tail = rest % 74;
            const double a = each * l1 + static_cast<double>((early + idle - 1) / idle + full + (tail > 0)) * l2;
            const double b = extra ? (each + 1) * l1 + static_cast<double>(full + (tail > idle)) * l2 : 0.0;
            const double us = (a > b ? a : b) + sum_us(w1, s1) + sum_us(w2, s2);
            if ((s1 == 1 && s2 == 1) || us < best.us) best = GemmPlan{s1, s2, lead, us};
        }
    }
    return best;
}

// Whether 512-row tiles finish first: their rounds at 0.8 us per k-block against
// those of 256-row tiles at 0.55 us (gemm_plan).  8192 x 16384 x 896: 64 tall tiles
// 173 us, 128 flat ones 203 us.
inline bool gemm_tall(long long M, long long N, int splits) {
    const long long cols = (N + gm::BN - 1) / gm::BN * splits;
    const long long tall = ((M + 511) / 512 * cols + 73) / 74, flat = ((M + 255) / 256 * cols + 73) / 74;
    return 0.8 * static_cast<double>(tall) < 0.55 * static_cast<double>(flat);
}

}  // namespace sbl
