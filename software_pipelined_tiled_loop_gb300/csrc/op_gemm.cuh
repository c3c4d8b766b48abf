// Tensor-core product of the operators (linear, gated, cross entropy): the
// pipelined tcgen05 kernel of tc_gemm.cuh with what those products need on
// top of it -- operands in either major order, two operand pairs summed along
// K or set side by side along N, a K range split into parts, and an epilogue
// given as a type.
//
//   warp 0 (one lane)  producer: TMA copies of the A and B panels into an
//                      S-stage ring (full / empty mbarriers).
//   warp 1 (one lane)  MMA issuer: tcgen05.mma kind::f16 (bf16 operands, fp32
//                      accumulators in tensor memory, two of them, so that a
//                      unit's epilogue overlaps the next unit's main loop).
//   warps 2..9         epilogue: two warps for each TMEM lane quadrant, each
//                      half of the accumulator's columns.  A thread holds a
//                      whole row segment, so row statistics need no shuffles.
//
// Operand layouts in shared memory, all with TMA's 128-byte swizzle:
//   A K-major   (stored M x K): box 64 k x 128 rows; 8-row groups 1024 B
//               apart; K = 16 -> + 32 B.
//   A M-major   (stored K x M): two boxes of 64 m x 64 k-rows; 8-k-row groups
//               1024 B apart, the 64-column blocks 8192 B; K = 16 -> + 2048 B.
//   B N-major   (stored K x N): boxes of 64 n x 64 k-rows, as A M-major.
//   B K-major   (stored N x K): boxes of 64 k x 64 columns below one another,
//               as A K-major.
// With a CTA pair (CG = 2) each CTA holds its 128 rows of A and half of B's
// columns; the pair computes a 256-row tile with one M = 256 MMA.
//
// What bounds it: the tensor core for K beyond some 500 (a CTA pair's 256 x 256
// tile takes 0.32 us a 64-wide K step against 2 to 4 us of epilogue, which the
// second accumulator hides except behind a slot's last unit), the writing of the
// output below (write-only traffic peaks at 4.05 TB/s here, a memset's rate).
// Measured, one call from a graph: 4096 x 4096 x 2048 42.9 us (1.60 PFLOP/s,
// 85 % of the measured bf16 peak; 3.6 waves of tiles), with bias and gelu_tanh
// 45 us, 8192 x 8192 x 4096 312 us (94 %); 65536 x 2048 x 16 67 us (4.0 TB/s).
//
// DUAL: the accumulator's left half is A * B0 and its right half A * B1 for
// the same columns of two matrices, so that one epilogue thread holds both
// products of an output element (the gate and the value of a gated block).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "op_host.h"
#include "ptx.cuh"

namespace pg {

// Programmatic stream serialisation, the two ways a kernel here uses it.
// Ordinary: every thread waits for the kernel before it ahead of its first
// access to memory, so that only its prologue overlaps that kernel's tail.
// Overlapping (`overlap`): the kernel reads nothing that the kernel before it
// writes, nor writes what that one touches, but only what was complete when that
// one began (which let this one launch only after its own wait).  It starts
// as SMs fall free and waits at its end instead, so that its completion still
// implies everything before it.  The second of two gradient products runs so.
__device__ __forceinline__ void op_begin(int overlap) {
    if (!overlap) grid_dependency_wait();
    grid_launch_dependents();
}
__device__ __forceinline__ void op_end(int overlap) {
    if (overlap) grid_dependency_wait();
}

struct OpMaps {
    CUtensorMap a[2], b[2], c[3];
};

// The schedule of one launch.  Units are (part, tile) pairs, all tiles of
// part 0 first; part p of P covers K-tiles [p T / P, (p + 1) T / P).
struct OpArgs {
    int M, N;          // extents of one output (N: of one segment along N)
    int K;             // columns of one K segment
    int m_tiles;       // of BM * CG rows
    int n_tiles;       // over all N segments
    int n_seg;         // tiles of one N segment; tiles from n_seg on read b[1], write c[1]
    int k_tiles;       // over all K segments
    int k_seg;         // K-tiles of one K segment; from k_seg on a[1], b[1]
    int parts;
    int group_m;
    int half_tiles;    // leftover tiles that run as two half-width units each
    int overlap;       // see op_begin
};

// ROUND: K-tiles of one accumulation round (0: all of a unit's K range).  The
// accumulator is handed to the epilogue after every round and starts again at
// zero; the epilogue adds the rounds in fp32 registers.
// NBUF: staging buffers of an epilogue warp.
template <int BN_, int STAGES_, int KSUB_, int CG_, bool A_MN_, bool B_K_, bool DUAL_ = false,
          int ROUND_ = 0, int NBUF_ = 2>
struct OpCfg {
    static constexpr int BM = 128, BN = BN_, BK = 64, STAGES = STAGES_, KSUB = KSUB_, CG = CG_;
    static constexpr bool A_MN = A_MN_, B_K = B_K_, DUAL = DUAL_;
    static constexpr int ROUND = ROUND_;
    static constexpr int SBK = BK * KSUB;
    static constexpr int B_COLS = BN / CG;          // B columns this CTA loads and holds
    static constexpr int TILE_N = DUAL ? BN / 2 : BN;  // output columns of a tile
    static constexpr int A_SUB = BM * BK * 2, B_SUB = B_COLS * BK * 2;
    static constexpr int A_BYTES = A_SUB * KSUB, B_BYTES = B_SUB * KSUB;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int TX_BYTES = STAGE_BYTES * CG;
    static constexpr bool HALVES = BN == 256 && CG == 2;  // half-width units
    static constexpr int TX_BYTES_HALF = (A_BYTES + B_BYTES / 2) * CG;
    static constexpr int EPI = 8;
    static constexpr int EPI_COLS = BN / 2;         // accumulator columns of an epilogue warp
    static constexpr int NBUF = NBUF_;
    static constexpr int STAGING_BYTES = EPI * NBUF * 2048;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int STAGING_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFFSET = STAGING_OFFSET + STAGING_BYTES;
    static constexpr int USED = BAR_OFFSET + (2 * STAGES + 5) * 8 + 16;
    static constexpr int SMEM_BYTES = smem_request(USED + 1024, 1);  // one block per SM
    static_assert(USED + 1024 <= 232448, "shared memory");
    static_assert(BN == 128 || BN == 256, "BN");
    static_assert(CG == 1 || (CG == 2 && BN == 256), "a pair computes 256 x 256 tiles");
    static_assert(!DUAL || !B_K, "the two B matrices of a dual product are N-major");
};

// ------------------------------------------------------- epilogue helpers ---
// Where one epilogue warp works: 32 rows from m0, its NB 2 KB staging buffers
// (used in turn, so that stores are still being read by TMA while the next is
// staged), the extents it may touch.
template <int NB_>
struct EpiCtx {
    static constexpr int NB = NB_;
    uint8_t *bufs;  // 1024-byte aligned
    uint32_t n;     // blocks staged so far
    int m0;         // first of the warp's 32 rows (may lie beyond M)
    int M, N;
    uint32_t lane;
    __device__ __forceinline__ int row() const { return m0 + static_cast<int>(lane); }
    // The next buffer, once the store that last used it has been read.  Every
    // block staged commits one bulk group (empty when no TMA store was made),
    // so that all but the last NB - 1 groups being read means this buffer is
    // free.  free(B): the next B buffers are.
    template <int B>
    __device__ __forceinline__ void free() {
        if (lane == 0) bulk_wait_read<NB - B>();
        __syncwarp();
    }
    __device__ __forceinline__ uint32_t take_buf() {
        return smem_u32(bufs) + (n++ % NB) * 2048u;
    }
    __device__ __forceinline__ uint32_t next_buf() {
        free<1>();
        return take_buf();
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// A staged block is 32 rows of 64 bytes with TMA's 64-byte swizzle: 16-byte
// chunk j of row r lies at chunk j ^ (r / 2 % 4), so the 8 rows of a store
// phase cover all banks.
__device__ __forceinline__ uint32_t staged(uint32_t buf, uint32_t row, uint32_t chunk) {
    return buf + row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}
__device__ __forceinline__ uint16_t lds_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Store 32 rows x 32 columns of 16-bit values, lane t's row in p[16] (pairs).
// map != nullptr: one TMA store (clips at the edges); else coalesced stores of
// pairs, or of single elements where rows may start on odd ones, for pitches
// TMA cannot describe.
template <class Ctx>
__device__ __forceinline__ void put_rows32(Ctx &c, const CUtensorMap *map, uint16_t *out,
                                           long long ld, int col, const uint32_t *p) {
    if (c.m0 >= c.M || col >= c.N) return;
    const uint32_t buf = c.next_buf();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts128(staged(buf, c.lane, j), p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
    if (map != nullptr) {
        fence_proxy_async_smem();
        __syncwarp();
        if (c.lane == 0) tma_store_2d(map, c.bufs + (buf - smem_u32(c.bufs)), col, c.m0);
    } else {
        __syncwarp();
        const int rows = min(32, c.M - c.m0);
        uint16_t *o = out + static_cast<long long>(c.m0) * ld + col;
        if (((ld | (reinterpret_cast<uintptr_t>(out) >> 1)) & 1) == 0) {
            const uint32_t w = c.lane & 15u, h = c.lane >> 4;  // pair w of rows h, h + 2, ...
            if (col + 2 * static_cast<int>(w) < c.N) {  // N is even here
#pragma unroll 4
                for (int r = static_cast<int>(h); r < rows; r += 2)
                    *reinterpret_cast<uint32_t *>(o + r * ld + 2 * w) =
                        lds32(staged(buf, r, w >> 2) + (w & 3u) * 4u);
            }
        } else if (col + static_cast<int>(c.lane) < c.N) {
#pragma unroll 8
            for (int r = 0; r < rows; ++r)
                o[r * ld + c.lane] = lds_u16(staged(buf, r, c.lane >> 3) + (c.lane & 7u) * 2u);
        }
    }
    if (c.lane == 0) bulk_commit();
    __syncwarp();
}

// B such blocks side by side (p[16 B]) by TMA: one fence and one wait for all.
template <int B, class Ctx>
__device__ __forceinline__ void put_rows32_batch(Ctx &c, const CUtensorMap *map, int col,
                                                 const uint32_t *p) {
    static_assert(B <= Ctx::NB, "staging buffers");
    if (c.m0 >= c.M || col >= c.N) return;
    c.template free<B>();
    uint32_t buf[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        buf[b] = c.take_buf();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sts128(staged(buf[b], c.lane, j), p[16 * b + 4 * j], p[16 * b + 4 * j + 1],
                   p[16 * b + 4 * j + 2], p[16 * b + 4 * j + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (c.lane == 0) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (col + 32 * b < c.N)
                tma_store_2d(map, c.bufs + (buf[b] - smem_u32(c.bufs)), col + 32 * b, c.m0);
        }
        // one group holds all B stores; the others keep the count
#pragma unroll
        for (int b = 0; b < B; ++b) bulk_commit();
    }
    __syncwarp();
}

// The same for 32 rows x 16 columns of 32-bit values, v[16] lane t's row;
// row0: the output row of m0.
template <class Ctx>
__device__ __forceinline__ void put_words16(Ctx &c, const CUtensorMap *map, float *out,
                                            long long ld, int row0, int col, const uint32_t *v) {
    if (c.m0 >= c.M || col >= c.N) return;
    const uint32_t buf = c.next_buf();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts128(staged(buf, c.lane, j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    if (map != nullptr) {
        fence_proxy_async_smem();
        __syncwarp();
        if (c.lane == 0) tma_store_2d(map, c.bufs + (buf - smem_u32(c.bufs)), col, row0);
    } else {
        __syncwarp();
        const int rows = min(32, c.M - c.m0);
        const uint32_t w = c.lane & 15u, h = c.lane >> 4;
        if (col + static_cast<int>(w) < c.N) {
            float *o = out + static_cast<long long>(row0) * ld + col + w;
#pragma unroll 4
            for (int r = static_cast<int>(h); r < rows; r += 2)
                o[r * ld] = __uint_as_float(lds32(staged(buf, r, w >> 2) + (w & 3u) * 4u));
        }
    }
    if (c.lane == 0) bulk_commit();
    __syncwarp();
}

// Read 32 rows x 32 columns of bf16 in two steps, so that the loads travel
// while something else is done: load() issues them, take() leaves lane t's row
// in p[16] (zero outside).  Rows of 16-byte pitch: each lane reads 16-byte
// vectors of its own row.  Other pitches: a lane reads pairs (w = lane % 16) of
// rows lane / 16 + 2 i, as two single elements since rows may start on odd ones,
// and take() turns them through a staging buffer.
struct RowsIn {
    const uint16_t *in;
    long long ld;
    uint32_t x[16];

    __device__ __forceinline__ bool vec() const { return (ld & 7) == 0; }
    template <class Ctx>
    __device__ __forceinline__ void load(const Ctx &c, int col) {
        if (vec()) {
            const bool row_in = c.row() < c.M;
            const uint16_t *src = in + static_cast<long long>(c.row()) * ld + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                // a vector that starts inside a row lies inside the matrix: the
                // pitch is N, a multiple of 8, or a padded one
                if (row_in && col + 8 * j < c.N) q = *reinterpret_cast<const uint4 *>(src + 8 * j);
                x[4 * j] = q.x;
                x[4 * j + 1] = q.y;
                x[4 * j + 2] = q.z;
                x[4 * j + 3] = q.w;
            }
        } else {
            const int cc = col + 2 * static_cast<int>(c.lane & 15u);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = c.m0 + 2 * i + static_cast<int>(c.lane >> 4);
                const uint16_t *src = in + static_cast<long long>(r) * ld + cc;
                uint32_t lo = 0, hi = 0;
                if (r < c.M && cc < c.N) lo = src[0];
                if (r < c.M && cc + 1 < c.N) hi = src[1];
                x[i] = lo | (hi << 16);
            }
        }
    }
    template <class Ctx>
    __device__ __forceinline__ void take(Ctx &c, uint32_t (&p)[16]) const {
        if (vec()) {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = x[j];
        } else {
            const uint32_t buf = c.next_buf();
            const uint32_t w = c.lane & 15u;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sts32(staged(buf, 2 * i + (c.lane >> 4), w >> 2) + (w & 3u) * 4u, x[i]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 q = lds_u4(staged(buf, c.lane, j));
                p[4 * j] = q.x;
                p[4 * j + 1] = q.y;
                p[4 * j + 2] = q.z;
                p[4 * j + 3] = q.w;
            }
            if (c.lane == 0) bulk_commit();
            __syncwarp();
        }
    }
};

// 32 values of a bf16 vector from index col (zero beyond n), the same in
// every lane.  The vector's base is 16-byte aligned and col a multiple of 32.
__device__ __forceinline__ void get_vec32(const uint16_t *v, int n, int col, float (&f)[32]) {
    if (col + 32 <= n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + col) + j);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[8 * j + 2 * i] = bf16_lo(w[i]);
                f[8 * j + 2 * i + 1] = bf16_hi(w[i]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            f[j] = col + j < n ? __uint_as_float(static_cast<uint32_t>(v[col + j]) << 16) : 0.0f;
    }
}

// One unit as its epilogue sees it.
struct OpUnit {
    int tile, part, seg;  // seg: N segment (output c[seg])
    int m0, n0;           // of the cluster's tile (n0: of the unit's own columns)
    int kb, ke;
    bool half;            // a half-width unit: BN / 2 accumulator columns
};

// Unit u of slot's list: whole tiles slot, slot + slots, ... first, then, when
// the last wave's R leftover tiles fit twice on the slots, one half-width unit
// (column half u % 2 of leftover tile u / 2) on each of 2 R slots, so that the
// last wave is half as long, and so is its epilogue.
template <class Cfg>
struct OpWalk {
    int tiles, whole, slot, slots, units;

    __device__ __forceinline__ OpWalk(const OpArgs &a, int slot_, int slots_)
        : slot(slot_), slots(slots_) {
        tiles = a.m_tiles * a.n_tiles;
        whole = tiles * a.parts - a.half_tiles;
        units = (slot < whole ? (whole - slot + slots - 1) / slots : 0) +
                (slot < 2 * a.half_tiles ? 1 : 0);
    }
    __device__ __forceinline__ OpUnit unit(const OpArgs &a, int i) const {
        OpUnit w;
        int u = slot + i * slots;
        int h = 0;
        w.half = u >= whole;
        if (w.half) {
            u = whole + (slot >> 1);
            h = slot & 1;
        }
        w.part = u / tiles;
        w.tile = u - w.part * tiles;
        const int per_group = a.group_m * a.n_tiles;
        const int g = w.tile / per_group;
        const int first_m = g * a.group_m;
        const int gm = min(a.m_tiles - first_m, a.group_m);
        const int r = w.tile - g * per_group;
        const int nt = r / gm;
        w.m0 = (first_m + r % gm) * (Cfg::BM * Cfg::CG);
        w.seg = nt >= a.n_seg ? 1 : 0;
        w.n0 = (nt - w.seg * a.n_seg) * Cfg::TILE_N + h * (Cfg::TILE_N / 2);
        w.kb = static_cast<int>(static_cast<long long>(w.part) * a.k_tiles / a.parts);
        w.ke = static_cast<int>(static_cast<long long>(w.part + 1) * a.k_tiles / a.parts);
        return w;
    }
};

// The accumulator columns of a unit that epilogue warp e (of 8) takes:
// [col0, col0 + cols); cols is a multiple of 64.
template <class Cfg>
__device__ __forceinline__ void epi_cols(const OpUnit &w, uint32_t e, int &col0, int &cols) {
    cols = Cfg::EPI_COLS > 64 && w.half ? Cfg::EPI_COLS / 2 : Cfg::EPI_COLS;
    col0 = static_cast<int>(e >> 2) * cols;
}
// DUAL: 64 output columns a warp, [col0, col0 + 64) of both halves, the halves
// `width` apart; none for the second four warps of a tile that is no wider.
template <class Cfg>
__device__ __forceinline__ bool epi_cols_dual(const OpUnit &w, uint32_t e, int &col0, int &width) {
    width = w.half ? Cfg::TILE_N / 2 : Cfg::TILE_N;
    col0 = static_cast<int>(e >> 2) * 64;
    return col0 < width;
}

// The accumulators as an epilogue warp takes them, one round after another.
template <class Cfg>
struct OpAcc {
    uint64_t *full, *empty;
    uint32_t base;  // tensor memory, in the warp's lanes
    uint32_t lane;
    uint32_t gr;    // rounds taken so far: selects the accumulator and its phase
    int rounds;     // of the present unit
    const KernelCtx &ctx;

    __device__ __forceinline__ bool have() const { return rounds > 0; }
    __device__ __forceinline__ uint32_t row() const { return base + (gr & 1u) * Cfg::BN; }
    __device__ __forceinline__ bool wait() const {
        if (rounds == 0) return true;
        const bool ok = mbar_wait(&full[gr & 1u], (gr >> 1) & 1u, ctx, kSiteEpilogueFull);
        tc_fence_after();
        return ok;
    }
    __device__ __forceinline__ void release() {
        if (rounds == 0) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if constexpr (Cfg::CG == 2)
                mbar_arrive_cluster(mapa_shared(smem_u32(&empty[gr & 1u]), 0));
            else
                mbar_arrive(&empty[gr & 1u]);
        }
        ++gr;
    }
    // pass all of the unit's rounds on unread
    __device__ __forceinline__ bool skip() {
#pragma unroll 1
        for (int r = 0; r < rounds; ++r) {
            if (!wait()) return false;
            release();
        }
        return true;
    }
};

// Epi: a struct of kernel parameters with
//   template <class Cfg, class Acc> __device__ bool run(EpiCtx<Cfg::NBUF> &, const OpMaps &,
//        const OpArgs &, const OpUnit &, Acc &acc, int e) const
// (acc: OpAcc)
// called by warp e of the eight epilogue warps for its 32 rows and its columns
// (epi_cols, epi_cols_dual).  For each of the unit's `rounds` rounds,
// wait() blocks until the accumulator is complete (false: the wait ran out, run
// returns false at once), row() addresses its first column in the warp's lanes
// and release() hands it back, once each and in this order; without ROUND that
// is one round, or none (an empty K range: the accumulator counts as zero, and
// wait and release do nothing).
template <class Cfg, class Epi>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    op_gemm_kernel(const __grid_constant__ OpMaps maps, const OpArgs args,
                   const __grid_constant__ Epi epi, const KernelCtx ctx) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    uint8_t *sA = smem;
    uint8_t *sB = smem + STAGES * Cfg::A_BYTES;
    uint8_t *sStage = smem + Cfg::STAGING_OFFSET;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFFSET);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_empty = acc_full + 2;   // [2]
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);

    const uint32_t warp = warp_id_uniform();
    const uint32_t lane = lane_id();
    if (warp == 0 && lane == 0) {
        if (args.k_tiles > 0) {
            prefetch_tmap(&maps.a[0]);
            prefetch_tmap(&maps.b[0]);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI * Cfg::CG);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        if constexpr (Cfg::CG == 2) {
            tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (Cfg::CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // on-chip set-up is done; what follows may read what the kernel before wrote
    op_begin(args.overlap);

    const int crank = Cfg::CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const int slot = static_cast<int>(blockIdx.x) / Cfg::CG;
    const int slots = static_cast<int>(gridDim.x) / Cfg::CG;
    const OpWalk<Cfg> walk(args, slot, slots);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- producer ----------------
            uint32_t it = 0;
            bool ok = true;
            for (int u = 0; ok && u < walk.units; ++u) {
                const OpUnit w = walk.unit(args, u);
                const int m0 = w.m0 + crank * BM;
                for (int kt = w.kb; kt < w.ke; ++kt, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(&empty[s], ph ^ 1u, ctx, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    const int ks = kt >= args.k_seg ? 1 : 0;
                    const CUtensorMap *ma = &maps.a[ks];
                    const uint32_t full_lead =
                        Cfg::CG == 2 ? mapa_shared(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                    if (crank == 0)
                        mbar_arrive_expect_tx(&full[s], w.half ? Cfg::TX_BYTES_HALF : Cfg::TX_BYTES);
                    auto load = [&](uint8_t *dst, const CUtensorMap *map, int x, int y) {
                        if constexpr (Cfg::CG == 2)
                            tma_load_2d_pair(dst, map, full_lead, x, y);
                        else
                            tma_load_2d(dst, map, &full[s], x, y);
                    };
#pragma unroll
                    for (int q = 0; q < Cfg::KSUB; ++q) {
                        const int k0 = (kt - ks * args.k_seg) * Cfg::SBK + q * BK;
                        uint8_t *da = sA + s * Cfg::A_BYTES + q * Cfg::A_SUB;
                        uint8_t *db = sB + s * Cfg::B_BYTES + q * Cfg::B_SUB;
                        if constexpr (Cfg::A_MN) {
#pragma unroll
                            for (int j = 0; j < BM / 64; ++j)
                                load(da + j * (BK * 128), ma, m0 + 64 * j, k0);
                        } else {
                            load(da, ma, k0, m0);
                        }
                        const int bc = Cfg::HALVES && w.half ? Cfg::B_COLS / 2 : Cfg::B_COLS;
                        if constexpr (Cfg::DUAL) {
                            // half h of the accumulator reads columns of b[h]; a
                            // pair's CTA h holds exactly that half
#pragma unroll
                            for (int j = 0; j < Cfg::B_COLS / 64; ++j) {
                                if (64 * j >= bc) break;
                                const int h = Cfg::CG == 2 ? crank : j / (Cfg::TILE_N / 64);
                                const int x = Cfg::CG == 2 ? 64 * j : 64 * j - h * Cfg::TILE_N;
                                load(db + j * (BK * 128), &maps.b[h], w.n0 + x, k0);
                            }
                        } else {
                            const int nb = w.n0 + crank * bc;
                            const CUtensorMap *mb = &maps.b[ks | w.seg];
                            if constexpr (Cfg::B_K) {
                                // boxes of 64 rows (columns of B) below one another
#pragma unroll
                                for (int j = 0; j < Cfg::B_COLS / 64; ++j)
                                    if (64 * j < bc) load(db + j * 8192, mb, k0, nb + 64 * j);
                            } else {
#pragma unroll
                                for (int j = 0; j < Cfg::B_COLS / 64; ++j)
                                    if (64 * j < bc) load(db + j * (BK * 128), mb, nb + 64 * j, k0);
                            }
                        }
                    }
                }
            }
            if constexpr (Cfg::CG == 2) {
                // the pair's last multicast releases of this CTA's barriers must
                // have landed before the cluster is left
                for (int i = 0; ok && i < STAGES; ++i, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    ok = mbar_wait(&empty[s], ph ^ 1u, ctx, kSiteProducerEmpty);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && crank == 0) {
            // ---------------- MMA issuer ----------------
            constexpr uint32_t idesc_full = idesc_f16(BM * Cfg::CG, BN, 1, Cfg::A_MN ? 1 : 0,
                                                      Cfg::B_K ? 0 : 1);
            constexpr uint32_t idesc_half = idesc_f16(BM * Cfg::CG, BN / 2, 1, Cfg::A_MN ? 1 : 0,
                                                      Cfg::B_K ? 0 : 1);
            constexpr uint16_t kPair = 3;
            uint32_t it = 0, gr = 0;
            bool ok = true;
            for (int u = 0; ok && u < walk.units; ++u) {
                const OpUnit w = walk.unit(args, u);
                const uint32_t idesc = Cfg::HALVES && w.half ? idesc_half : idesc_full;
                for (int k_begin = w.kb; ok && k_begin < w.ke;) {
                const int k_end = Cfg::ROUND > 0 ? min(w.ke, k_begin + Cfg::ROUND) : w.ke;
                const uint32_t ab = gr & 1u, aph = (gr >> 1) & 1u;
                ++gr;
                if (!mbar_wait(&acc_empty[ab], aph ^ 1u, ctx, kSiteMmaAccEmpty)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + ab * BN;
                for (int kt = k_begin; kt < k_end; ++kt, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(&full[s], ph, ctx, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int kk = kt >= args.k_seg ? kt - args.k_seg : kt;
#pragma unroll
                    for (int q = 0; q < Cfg::KSUB; ++q) {
                        // a sub-tile wholly beyond K holds only zero fill
                        if (q > 0 && kk * Cfg::SBK + q * BK >= args.K) break;
                        const uint32_t a_addr = smem_u32(sA + s * Cfg::A_BYTES + q * Cfg::A_SUB);
                        const uint32_t b_addr = smem_u32(sB + s * Cfg::B_BYTES + q * Cfg::B_SUB);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k) {
                            const uint64_t ad =
                                Cfg::A_MN ? smem_desc_sw128(a_addr + k * 2048, BK * 128, 1024)
                                          : smem_desc_sw128(a_addr + k * 32, 16, 1024);
                            const uint64_t bd =
                                Cfg::B_K ? smem_desc_sw128(b_addr + k * 32, 16, 1024)
                                         : smem_desc_sw128(b_addr + k * 2048, BK * 128, 1024);
                            const uint32_t acc = (kt == k_begin && q == 0 && k == 0) ? 0u : 1u;
                            if constexpr (Cfg::CG == 2)
                                umma_f16_ss_pair(d_tmem, ad, bd, idesc, acc);
                            else
                                umma_f16_ss(d_tmem, ad, bd, idesc, acc);
                        }
                    }
                    if constexpr (Cfg::CG == 2)
                        umma_commit_pair_multicast(&empty[s], kPair);
                    else
                        umma_commit(&empty[s]);
                }
                if (ok) {
                    if constexpr (Cfg::CG == 2)
                        umma_commit_pair_multicast(&acc_full[ab], kPair);
                    else
                        umma_commit(&acc_full[ab]);
                }
                k_begin = k_end;
                }
            }
            if constexpr (Cfg::CG == 2)
                umma_commit_pair_multicast(mma_done, 1);
            else
                umma_commit(mma_done);
            mbar_wait(mma_done, 0, ctx, kSiteMmaDone);
        }
    } else {
        // ---------------- epilogue warps ----------------
        const uint32_t e = warp - 2;
        const uint32_t q = warp & 3u;  // the TMEM lane quadrant this warp may read
        EpiCtx<Cfg::NBUF> c;
        c.bufs = sStage + e * (Cfg::NBUF * 2048);
        c.n = 0;
        c.M = args.M;
        c.N = args.N;
        c.lane = lane;
        OpAcc<Cfg> acc{acc_full, acc_empty, tmem_base + ((q * 32u) << 16), lane, 0u, 0, ctx};
        for (int u = 0; u < walk.units; ++u) {
            const OpUnit w = walk.unit(args, u);
            c.m0 = w.m0 + crank * BM + static_cast<int>(q * 32);
            acc.rounds = w.ke <= w.kb     ? 0
                         : Cfg::ROUND > 0 ? (w.ke - w.kb + Cfg::ROUND - 1) / Cfg::ROUND
                                          : 1;
            if (!epi.template run<Cfg>(c, maps, args, w, acc, e)) break;
        }
        if (lane == 0) bulk_wait_all();  // this warp's stores have landed
        __syncwarp();
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncwarp();
    if constexpr (Cfg::CG == 2)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (Cfg::CG == 2)
            tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
    op_end(args.overlap);
}

// Read 32 accumulator columns (zeros when there is no accumulator).
__device__ __forceinline__ void acc_cols32(uint32_t taddr, bool have, uint32_t (&v)[32]) {
    if (have) {
        tmem_ld_32x32b_x32(taddr, v);
        tmem_ld_wait();
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0u;
    }
}

// v += N accumulator columns from taddr.
template <int N>
__device__ __forceinline__ void acc_add(uint32_t taddr, float *v) {
    if constexpr (N <= 64) {  // room in the register file for longer loads
#pragma unroll
        for (int c = 0; c < N; c += 32) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(taddr + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[c + j] += __uint_as_float(x[j]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 16) {
            uint32_t x[16];
            tmem_ld_32x32b_x16(taddr + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[c + j] += __uint_as_float(x[j]);
        }
    }
}

// All rounds of a unit, added in fp32 registers: N columns from col, and with
// N2 > 0 another N2 from col2.  false: a wait ran out.
template <int N, int N2, class Acc>
__device__ __forceinline__ bool acc_sum(Acc &acc, int col, float *v, int col2, float *v2) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < N2; ++j) v2[j] = 0.0f;
#pragma unroll 1
    for (int r = 0; r < acc.rounds; ++r) {
        if (!acc.wait()) return false;
        const uint32_t t = acc.row();
        acc_add<N>(t + col, v);
        if constexpr (N2 > 0) acc_add<N2>(t + col2, v2);
        acc.release();
    }
    return true;
}

// The same for the columns of epi_cols, fewer in a half-width unit.
template <class Cfg, class Acc>
__device__ __forceinline__ bool acc_sum_unit(Acc &acc, int col0, int cols, float *v) {
    if constexpr (Cfg::EPI_COLS > 64) {
        if (cols < Cfg::EPI_COLS)
            return acc_sum<Cfg::EPI_COLS / 2, 0>(acc, col0, v, 0, nullptr);
    }
    return acc_sum<Cfg::EPI_COLS, 0>(acc, col0, v, 0, nullptr);
}

// What a ReLU's derivative needs: it jumps at zero, and a pre-activation whose
// sign the rounding of its sum flips puts a whole dY in the wrong place.  The
// tensor core truncates its running sum every 16 products, toward zero: a chain
// of K = 8192 ends 4e-6 of itself short, an fp32 sum with rounding 1e-6.  Rounds of
// 512 products added in registers end at 5e-7.  So products whose Z decides a
// ReLU run in rounds when K is longer than one (of few rows: a CTA's share of K);
// smooth activations do not need it.
constexpr int kSignRound = 512;
inline bool op_sign_rounds(int act, int K) { return act == PGEMM_ACT_RELU && K > kSignRound; }
using SignPair = std::integral_constant<int, kSignRound / 128>;  // K-tiles a round
using SignOne = std::integral_constant<int, kSignRound / 64>;

// ------------------------------------------------------------------- host ---
// Schedule slots: one block (or pair) per SM.
template <class Cfg, class Epi>
static cudaError_t op_slots(const LaunchCommon &p, int *slots) {
    if constexpr (Cfg::CG == 1) {
        *slots = p.sm_count;
        return cudaSuccess;
    } else {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = Cfg::CG;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t lc{};
        lc.blockDim = dim3(Cfg::THREADS);
        lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
        lc.gridDim = dim3(Cfg::CG * p.sm_count);
        lc.attrs = attr;
        lc.numAttrs = 1;
        int clusters = 0;
        cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, op_gemm_kernel<Cfg, Epi>, &lc);
        if (e != cudaSuccess) return e;
        if (clusters < 1) return cudaErrorInvalidConfiguration;
        *slots = clusters;
        return cudaSuccess;
    }
}

template <class Cfg, class Epi>
static KernelInfo op_info() {
    KernelInfo k;
    k.threads = Cfg::THREADS;
    k.smem_bytes = Cfg::SMEM_BYTES;
    k.schedule_slots = op_slots<Cfg, Epi>;
    k.func = reinterpret_cast<const void *>(op_gemm_kernel<Cfg, Epi>);
    return k;
}

// Sets the kernel up on the device (once), then launches it on `stream` under
// programmatic stream serialisation: the kernel waits for the one before it ahead of its
// first access to memory, or with a.overlap at its end (op_begin).
template <class Cfg, class Epi>
static pgemm_status op_launch(const OpDevice &dev, const OpMaps &maps, OpArgs a, const Epi &epi,
                              cudaStream_t stream) {
    static const KernelInfo info = op_info<Cfg, Epi>();
    int slots = 0;
    const pgemm_status st = op_kernel_setup(dev, info, &slots);
    if (st != PGEMM_OK) return st;
    const long long units = static_cast<long long>(a.m_tiles) * a.n_tiles * a.parts;
    if (units < 1) return PGEMM_OK;
    if (units > 0x7fffffffll) return PGEMM_ERR_INVALID_VALUE;
    const long long left = units % slots;
    a.half_tiles = Cfg::HALVES && 2 * left <= slots ? static_cast<int>(left) : 0;
    // Raster groups: down group_m tile rows, then one tile column across, so
    // that the blocks running at once share panels of A and B through L2 (the
    // same widths as the plain products: 16 up to K = 4096, else 8).
    a.group_m = static_cast<long long>(a.k_tiles) * Cfg::SBK / a.parts <= 4096 ? 16 : 8;
    cudaLaunchAttribute attr[2];
    int nattr = 0;
    attr[nattr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[nattr].val.programmaticStreamSerializationAllowed = 1;
    ++nattr;
    if constexpr (Cfg::CG == 2) {
        attr[nattr].id = cudaLaunchAttributeClusterDimension;
        attr[nattr].val.clusterDim.x = Cfg::CG;
        attr[nattr].val.clusterDim.y = 1;
        attr[nattr].val.clusterDim.z = 1;
        ++nattr;
    }
    cudaLaunchConfig_t lc{};
    lc.blockDim = dim3(Cfg::THREADS);
    const long long most = units + a.half_tiles;
    lc.gridDim = dim3(Cfg::CG * static_cast<int>(most < slots ? most : slots));
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = nattr;
    return cudaLaunchKernelEx(&lc, op_gemm_kernel<Cfg, Epi>, maps, a, epi, dev.ctx) == cudaSuccess
               ? PGEMM_OK
               : PGEMM_ERR_CUDA;
}

// As op_launch launches: the kernel waits before it touches memory, or as op_begin says.
template <class... KArgs, class... Args>
static pgemm_status launch_small(void (*kernel)(KArgs...), dim3 grid, dim3 block,
                                 cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.stream = s;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...) == cudaSuccess ? PGEMM_OK : PGEMM_ERR_CUDA;
}

}  // namespace pg
