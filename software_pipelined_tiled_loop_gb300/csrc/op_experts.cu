// The experts' products: rows sorted by expert, expert e's rows [offsets[e], offsets[e + 1])
// times its own matrices.
//
//   experts_linear  Y[r] = X[r] W[e];  dX[r] = dY[r] W[e]^T, dW[e] = X_e^T dY_e
//   experts_gated   H[r] = act(X[r] Wg[e]) * (X[r] Wu[e]); dG = dH U act'(G), dU = dH act(G),
//                   dX = dG Wg^T + dU Wu^T, dWg[e] = X_e^T dG_e, dWu[e] = X_e^T dU_e
//
// The groups' sizes are known on the device alone: every CTA reads the offsets and works
// out the same list of units, so a call needs no host round trip and can be captured.
//
// Rows (forward and dX): experts_rows_kernel.  The weights take the tensor core's M side,
// D[n][t] = sum_k W[e][k][n] X[t][k]: A = W^T read M-major from the K x N rows (dX: the
// same rows K-major), B = a group's rows K-major, N = as many of them as there are, rounded
// up to 32 (16 on one CTA).  A group of 40 rows then costs 64 columns of products, where
// 256-row tiles on the M side would pay for 256; groups are ragged in one direction only,
// and the instruction's N follows them.  A group of more rows than a tile takes is dealt
// out evenly.  A thread owns one feature of the output: a warp's store covers 32 features
// of a row, 64 bytes, so rows need no staging, no alignment and no tensor map, and stop
// where the group does.  (Whole 32-byte sectors where rows are a multiple of 16 features
// long; elsewhere those at its two ends are written in part.)
//
// Gated: a CTA's 128 accumulator lanes are 64 features of Wg and the same 64 of Wu, so the
// two products of an element lie in lanes of different warps; each of the two warps hands
// the other half of its columns through shared memory and finishes the other half.
//
// The gated gradient's dG and dU are rounded to bf16, as the dense one's are: the products
// that follow take both operands in one type, and the other one is the bf16 weights or rows.
// In 32 bits they would be tf32 products at half of the rate, or a second bf16 product for
// what the rounding left.  dX, dWg and dWu are off by 2.35e-3 (2-norm) with it, of which
// their own rounding is 1.66e-3.
//
// Weights' gradients: experts_weights_kernel, the tiled TN product with a group's rows
// as its K range.  The range starts and ends anywhere; in its last K step the rows behind
// the group (the next group's, which may hold anything) are cleared in shared memory.
#include <algorithm>
#include <climits>

#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

constexpr int kExpertsMax = 1024;

enum class Exp {
    LINEAR,      // X W
    GATED,       // act(X Wg) * (X Wu)
    GATED_GRAD,  // dH U act'(G), dH act(G)
    TRANSPOSED,  // sum over segments of X W^T
};

struct ExpertsMaps {
    CUtensorMap x[2][3];     // rows, in boxes of three sizes
    CUtensorMap w[2];
};
struct ExpertsWeightsMaps {
    CUtensorMap x[4], z[2][4];  // boxes of 96, 64, 32 and 16 rows
    CUtensorMap c[2];
};

struct ExpertsArgs {
    int R, E;             // rows at most; experts
    int M;                // features of an output (gated: of one product)
    int K;                // reduction columns of one segment
    int k_tiles, k_seg;   // K steps over all segments, and of one
    int f_tiles;          // tiles of features
    const int32_t *offsets;
    uint16_t *out, *out2;
    long long ldo;        // row length of out and out2
    float *preact;        // gated: both products, R x M each
    const uint16_t *dy;   // gated gradient: R x M
    int act;
    int tma_out;          // weights' gradient: the outputs have tensor maps
    int n_seg;            // weights' gradient: tiles along N of one output
    int segments;         // and outputs
    int overlap;          // weights' gradient: see op_begin
};

// CG CTAs work on a tile of CG * 128 accumulator lanes x up to TOK rows, BK columns of the
// reduction a step.  What a step's copies cost is their number: one expert, 8192 x 8192 x
// 4096 on pairs, took 404 us with four boxes of 32 rows a step, 323 with one of 128, and
// 285 (1.93 PFLOP/s) since the warps that issue them run as one (warp_value).  A pair's ring
// holds six steps of 64 columns, so that loads from HBM have longer to arrive: 64 experts
// of some 512 rows, 2048 x 1024 gated, 187 us, with three steps of 128 197.  Such ragged
// groups (32 experts, 4096 x 2048: 1.48 PFLOP/s) pay for tiles of fewer than 256 rows, whose
// weights are as many bytes for fewer products.
template <int CG_, int TOK_, int BK_, int STAGES_, Exp MODE_>
struct ExpCfg {
    static constexpr int CG = CG_, TOK = TOK_, STAGES = STAGES_, BK = BK_, BM = 128;
    static constexpr Exp MODE = MODE_;
    static constexpr bool DUAL = MODE == Exp::GATED || MODE == Exp::GATED_GRAD;
    static constexpr bool W_K = MODE == Exp::TRANSPOSED;  // W's rows run along the reduction
    static constexpr int FEATS = DUAL ? 64 : 128;         // features of a CTA
    static constexpr int STEP = 16 * CG;                  // granularity of a tile's rows
    static constexpr int BOX = TOK / CG / 4;              // rows of the smallest TMA box
    static constexpr int B_SUB = TOK / CG * 128;          // 64 columns of all rows
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = TOK / CG * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI = 8;
    static constexpr int CHUNK = CG == 2 ? 32 : 16;       // columns an epilogue warp takes at once
    static constexpr int SWAP_BYTES = DUAL ? EPI * CHUNK / 2 * 128 : 0;
    static constexpr int SWAP_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFFSET = SWAP_OFFSET + SWAP_BYTES;
    static constexpr int TABLE_OFFSET = BAR_OFFSET + (2 * STAGES + 5) * 8 + 24;
    static constexpr int USED = TABLE_OFFSET + (3 * kExpertsMax + 1) * 4;
    static constexpr int TMEM_COLS = 2 * TOK;
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int SMEM_BYTES = smem_request(USED + 1024, 1);
    static_assert(USED + 1024 <= 232448, "shared memory");
    static_assert(BK == 64 || BK == 128, "BK");
    static_assert(BOX % 8 == 0 && TMEM_COLS >= 32 && TMEM_COLS <= 512, "TOK");
};

// The list of units, the same in every CTA: begin[e], end[e] (clamped to the rows there
// are) and first[e], the units before expert e's.
struct ExpertsTable {
    int32_t *begin, *end, *first;
    int E;
    __device__ __forceinline__ int units() const { return first[E]; }
    // the expert of unit u
    __device__ __forceinline__ int expert(int u) const {
        int lo = 0, hi = E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
};

// All threads; count(rows) gives an expert's units, fewer than kUnitsMost (as the host
// checks for all of a call's).  The sums stop there, so that offsets which decrease, and
// count rows twice, still make a list whose units lie within their experts' rows.
constexpr int kUnitsMost = INT_MAX / 2;
template <class Count>
__device__ __forceinline__ ExpertsTable experts_table(const ExpertsArgs &a, uint8_t *at,
                                                      Count &&count) {
    ExpertsTable t;
    t.begin = reinterpret_cast<int32_t *>(at);
    t.end = t.begin + kExpertsMax;
    t.first = t.end + kExpertsMax;
    t.E = a.E;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < a.E) {
                const int b = min(max(a.offsets[e], 0), a.R);
                const int d = min(max(a.offsets[e + 1], b), a.R);
                t.begin[e] = b;
                t.end[e] = d;
                n = count(d - b);
            }
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum = min(sum + o, kUnitsMost);
            }
            const int earlier = __shfl_up_sync(0xffffffffu, sum, 1);
            if (e < a.E) t.first[e] = min(before + (lane > 0 ? earlier : 0), kUnitsMost);
            before = min(before + __shfl_sync(0xffffffffu, sum, 31), kUnitsMost);
        }
        if (lane == 0) t.first[a.E] = before;
    }
    __syncthreads();
    return t;
}

// Where a ring of stages is: stage s, in its phase.
template <int STAGES>
struct Ring {
    uint32_t s = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
        }
    }
};

// One unit: rows [row0, row0 + rows) of an expert, `cols` accumulator columns, features
// from f0 (the whole tile's).
struct RowsUnit {
    int expert, row0, rows, cols, f0;
};

template <class Cfg>
__device__ __forceinline__ int row_tiles(int rows) {
    return rows > 0 ? (rows - 1) / Cfg::TOK + 1 : 0;  // (rows up to 2^31 - 1)
}

// Units of an expert: down its tiles of rows, up to sixteen of them, then one tile of
// features across, so that the CTAs running at once share panels of weights and of rows.
template <class Cfg>
__device__ __forceinline__ RowsUnit rows_unit(const ExpertsTable &t, const ExpertsArgs &a, int u) {
    RowsUnit w;
    w.expert = t.expert(u);
    const int begin = t.begin[w.expert], n = t.end[w.expert] - begin;
    const int r = u - t.first[w.expert];
    const int tiles = row_tiles<Cfg>(n);
    const int group = r / (16 * a.f_tiles), first = group * 16;
    const int g = min(tiles - first, 16), q = r - group * 16 * a.f_tiles;
    const int rt = first + q % g;
    w.f0 = q / g * (Cfg::FEATS * Cfg::CG);
    const int each = ((n - 1) / tiles + Cfg::STEP) / Cfg::STEP * Cfg::STEP;
    w.row0 = begin + rt * each;
    w.rows = min(each, n - rt * each);
    w.cols = (w.rows + Cfg::STEP - 1) / Cfg::STEP * Cfg::STEP;
    return w;
}

__device__ __forceinline__ RowsUnit warp_unit(const RowsUnit &w) {
    return RowsUnit{warp_value(w.expert), warp_value(w.row0), warp_value(w.rows),
                    warp_value(w.cols), warp_value(w.f0)};
}

__device__ __forceinline__ void put_bf16(uint16_t *p, float v) {
    *p = static_cast<uint16_t>(pack_bf16(v, 0.0f) & 0xffffu);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    experts_rows_kernel(const __grid_constant__ ExpertsMaps maps, const ExpertsArgs a,
                        const KernelCtx ctx) {
    constexpr int CG = Cfg::CG, STAGES = Cfg::STAGES, BK = Cfg::BK, TOK = Cfg::TOK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    uint8_t *sA = smem, *sB = smem + STAGES * Cfg::A_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFFSET);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_empty = acc_full + 2;   // [2]
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    const uint32_t warp = warp_id_uniform(), lane = lane_id();
    if (warp == 0 && lane == 0) {
        if (a.k_tiles > 0) {
            prefetch_tmap(&maps.x[0][0]);
            prefetch_tmap(&maps.w[0]);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI * CG);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    op_begin(0);
    const ExpertsTable table =
        experts_table(a, smem + Cfg::TABLE_OFFSET,
                      [&](int rows) { return row_tiles<Cfg>(rows) * a.f_tiles; });
    const int units = warp_value(table.units());
    const int crank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const int slot = static_cast<int>(blockIdx.x) / CG;
    const int slots = static_cast<int>(gridDim.x) / CG;

    // The first two warps run as one each, with one lane's instructions (see warp_value).
    const uint32_t lead = lane == 0 ? 1u : 0u;
    if (warp == 0) {
        // ---------------- producer ----------------
        Ring<STAGES> ring;
        bool ok = true;
        const uint32_t full0 = smem_u32(full);
        const uint32_t full_lead = CG == 2 ? warp_value(mapa_shared(full0, 0)) : full0;
        const uint32_t first = crank == 0 ? lead : 0u;
        const int segments = a.k_tiles > a.k_seg ? 2 : 1;
        RowsUnit next = warp_unit(slot < units ? rows_unit<Cfg>(table, a, slot) : RowsUnit{});
        for (int u = slot; u < units; u += slots) {
            const RowsUnit w = next;
            const int half = w.cols / CG;  // columns of B in this CTA
            const int boxes = (half + Cfg::BOX - 1) / Cfg::BOX;  // 1 .. 4
            const int box = boxes == 4 ? 0 : boxes >= 2 ? 1 : 2;
            // (may pass 2^31 where the rows have ended: zero fill either way)
            const int y0 = static_cast<int>(static_cast<uint32_t>(w.row0) + crank * half);
            const uint32_t tx = CG * (Cfg::A_BYTES + boxes * Cfg::BOX * BK * 2);
            const int f0 = w.f0 + crank * Cfg::FEATS;
            for (int sg = 0; sg < segments; ++sg) {
                const CUtensorMap *mx = &maps.x[sg][box], *mw = &maps.w[sg];
                for (int left = a.K; left > 0; left -= BK, ring.next()) {
                    const int k0 = a.K - left;
                    const uint32_t s = ring.s;
                    if (ok)
                        ok = warp_value(mbar_wait(&empty[s], ring.phase ^ 1u, ctx,
                                                  kSiteProducerEmpty)) != 0;
                    const uint32_t go = ok ? lead : 0u;  // (after a failure nothing is issued)
                    const uint32_t bar = full_lead + s * 8;
                    mbar_arrive_expect_tx_if(ok ? first : 0u, full0 + s * 8, tx);
                    const uint32_t da = smem_u32(sA) + s * Cfg::A_BYTES;
                    const uint32_t db = smem_u32(sB) + s * Cfg::B_BYTES;
                    if constexpr (Cfg::W_K) {
#pragma unroll
                        for (int q = 0; q < BK / 64; ++q)
                            tma_load_3d_if<CG>(go, da + q * 16384, mw, bar, k0 + 64 * q, f0,
                                               w.expert);
                    } else {
                        tma_load_3d_if<CG>(go, da, &maps.w[0], bar, f0, k0, w.expert);
                        tma_load_3d_if<CG>(go, da + BK * 128, &maps.w[Cfg::DUAL ? 1 : 0], bar,
                                           Cfg::DUAL ? f0 : f0 + 64, k0, w.expert);
                    }
#pragma unroll
                    for (int q = 0; q < BK / 64; ++q)
                        tma_load_2d_if<CG>(go, db + q * Cfg::B_SUB, mx, bar, k0 + 64 * q, y0);
                    if (boxes == 3) {
#pragma unroll
                        for (int q = 0; q < BK / 64; ++q)
                            tma_load_2d_if<CG>(go, db + q * Cfg::B_SUB + 2 * Cfg::BOX * 128,
                                               &maps.x[sg][2], bar, k0 + 64 * q,
                                               y0 + 2 * Cfg::BOX);
                    }
                }
                // (found while these copies travel)
                if (sg == 0 && u + slots < units)
                    next = warp_unit(rows_unit<Cfg>(table, a, u + slots));
            }
        }
        if constexpr (CG == 2) {
            // the pair's last multicast releases of this CTA's barriers must
            // have landed before the cluster is left
            for (int i = 0; ok && i < STAGES; ++i, ring.next())
                ok = warp_value(mbar_wait(&empty[ring.s], ring.phase ^ 1u, ctx,
                                          kSiteProducerEmpty)) != 0;
        }
    } else if (warp == 1) {
        if (crank == 0) {
            // ---------------- MMA issuer ----------------
            constexpr uint16_t kPair = 3;
            // descriptors of the first stage; addresses count in 16 bytes
            const uint64_t a0 = smem_desc_sw128(smem_u32(sA), Cfg::W_K ? 16 : BK * 128, 1024);
            const uint64_t b0 = smem_desc_sw128(smem_u32(sB), 16, 1024);
            const uint32_t tmem_w = warp_value(tmem);
            Ring<STAGES> ring;
            uint32_t n = 0;
            bool ok = true;
            int cols = warp_value(slot < units ? rows_unit<Cfg>(table, a, slot).cols : 0), next = 0;
            for (int u = slot; u < units && a.k_tiles > 0; u += slots, ++n, cols = next) {
                const uint32_t idesc =
                    idesc_f16(Cfg::BM * CG, cols, 1, Cfg::W_K ? 0 : 1, /*B K-major*/ 0);
                const uint32_t ab = n & 1u;
                if (ok)
                    ok = warp_value(mbar_wait(&acc_empty[ab], ((n >> 1) & 1u) ^ 1u, ctx,
                                              kSiteMmaAccEmpty)) != 0;
                tc_fence_after();
                const uint32_t d = tmem_w + ab * TOK;
                int left = a.K;  // of the segment
                uint32_t acc = 0;
                for (int kt = 0; kt < a.k_tiles; ++kt, ring.next()) {
                    const uint32_t s = ring.s;
                    if (ok)
                        ok = warp_value(mbar_wait(&full[s], ring.phase, ctx, kSiteMmaFull)) != 0;
                    const uint32_t go = ok ? lead : 0u;
                    tc_fence_after();
                    const uint64_t as = a0 + s * (Cfg::A_BYTES / 16), bs = b0 + s * (Cfg::B_BYTES / 16);
                    auto multiply = [&](int k) {
                        umma_f16_ss_if<CG>(
                            go, d,
                            as + (Cfg::W_K ? k / 4 * 16384 + k % 4 * 32 : k * 2048) / 16,
                            bs + (k / 4 * Cfg::B_SUB + k % 4 * 32) / 16, idesc, acc);
                        acc = 1;
                    };
                    if (left >= BK) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k) multiply(k);
                        left -= BK;
                    } else {  // what lies wholly beyond K is zero fill
#pragma unroll 1
                        for (int k = 0; 16 * k < left; ++k) multiply(k);
                        left = 0;
                    }
                    if (left == 0) left = a.K;
                    umma_commit_if<CG>(go, smem_u32(&empty[s]), kPair);
                    // (found while these products run)
                    if (kt == 0 && u + slots < units)
                        next = warp_value(rows_unit<Cfg>(table, a, u + slots).cols);
                }
                umma_commit_if<CG>(ok ? lead : 0u, smem_u32(&acc_full[ab]), kPair);
            }
            umma_commit_if<CG>(lead, smem_u32(mma_done), 1);
            mbar_wait(mma_done, 0, ctx, kSiteMmaDone);
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        // A quadrant's two warps take W accumulator columns (rows of the output) in turn;
        // the next ones are on their way from tensor memory while these are worked on.
        constexpr int W = Cfg::CHUNK, KEEP = W / 2;
        const int e = static_cast<int>(warp) - 2, h = e >> 2;
        const uint32_t q = warp & 3u;  // the TMEM lane quadrant this warp may read
        // gated: quadrants 0 and 1 hold Wg's 64 features, 2 and 3 Wu's
        const bool gate = q < 2;
        const int lane_feat = Cfg::DUAL ? static_cast<int>((q & 1u) * 32 + lane)
                                        : static_cast<int>(q * 32 + lane);
        const bool have = a.k_tiles > 0;
        uint32_t n = 0;
        bool ok = true;  // a wait that ran out: the rest goes by unread, barriers and all
        for (int u = slot; u < units; u += slots, ++n) {
            const RowsUnit w = rows_unit<Cfg>(table, a, u);
            const int feat = w.f0 + crank * Cfg::FEATS + lane_feat;
            const bool mine = feat < a.M;
            const uint32_t ab = n & 1u;
            const uint32_t t_row = tmem + ((q * 32u) << 16) + ab * TOK;
            const int chunks = (w.rows + W - 1) / W;
            uint32_t v[W];
            // gated gradient: dH of the columns that this warp finishes (the gate's warp a
            // chunk's first half, the other one the rest)
            const int c0 = gate ? 0 : KEEP;
            uint16_t dh[Cfg::MODE == Exp::GATED_GRAD ? KEEP : 1];
            auto fetch_dh = [&](int c) {
                if constexpr (Cfg::MODE == Exp::GATED_GRAD) {
                    const long long row = static_cast<long long>(w.row0) + c * W + c0;
                    const uint16_t *in = a.dy + row * a.M + feat;
#pragma unroll
                    for (int j = 0; j < KEEP; ++j) {
                        dh[j] = mine && c * W + c0 + j < w.rows ? *in : 0;
                        in += a.M;
                    }
                }
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[ab]), 0));
                    else
                        mbar_arrive(&acc_empty[ab]);
                }
            };
            auto fetch = [&](int c) {
                if (have && ok) {
                    if constexpr (W == 32)
                        tmem_ld_32x32b_x32(t_row + c * W, *reinterpret_cast<uint32_t(*)[32]>(v));
                    else
                        tmem_ld_32x32b_x16(t_row + c * W, v);
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = 0u;
                }
            };
            if (h < chunks) fetch_dh(h);
            if (have) {
                if (ok) ok = mbar_wait(&acc_full[ab], (n >> 1) & 1u, ctx, kSiteEpilogueFull);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            if (h < chunks)
                fetch(h);
            else if (have)
                release();
#pragma unroll 1
            for (int c = h; c < chunks; c += 2) {
                const int left = ok ? w.rows - c * W : 0;  // rows from this chunk on
                const long long row = w.row0 + static_cast<long long>(c) * W;
                const bool more = c + 2 < chunks;
                tmem_ld_wait();
                if (have && !more) release();
                if constexpr (!Cfg::DUAL) {
                    uint32_t r[W / 2];
#pragma unroll
                    for (int j = 0; j < W / 2; ++j)
                        r[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    if (more) fetch(c + 2);
                    uint16_t *o = a.out + row * a.ldo + feat;
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (j < left)
                                *o = static_cast<uint16_t>(j & 1 ? r[j / 2] >> 16 : r[j / 2]);
                            o += a.ldo;
                        }
                    }
                } else {
                    if (Cfg::MODE == Exp::GATED && a.preact != nullptr && mine) {
                        float *z = a.preact + (gate ? 0 : static_cast<long long>(a.R) * a.M) +
                                   row * a.M + feat;
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (j < left) *z = __uint_as_float(v[j]);
                            z += a.M;
                        }
                    }
                    // half of the columns to the other warp of the features, half from it
                    float *own = reinterpret_cast<float *>(smem + Cfg::SWAP_OFFSET) +
                                 e * (KEEP * 32) + lane;
                    const float *other = own + ((e ^ 2) - e) * (KEEP * 32);
                    const uint32_t bar = 1 + h * 2 + (q & 1u);
                    float g[KEEP], up[KEEP], d[KEEP];
#pragma unroll
                    for (int j = 0; j < KEEP; ++j) {
                        own[32 * j] = __uint_as_float(gate ? v[KEEP + j] : v[j]);
                        g[j] = __uint_as_float(gate ? v[j] : v[KEEP + j]);
                        if (Cfg::MODE == Exp::GATED_GRAD)
                            d[j] = __uint_as_float(
                                static_cast<uint32_t>(dh[Cfg::MODE == Exp::GATED_GRAD ? j : 0])
                                << 16);
                    }
                    if (more) {
                        fetch(c + 2);
                        fetch_dh(c + 2);
                    }
                    named_barrier(bar, 64);
#pragma unroll
                    for (int j = 0; j < KEEP; ++j) {
                        const float got = other[32 * j];
                        up[j] = gate ? got : g[j];
                        g[j] = gate ? g[j] : got;
                    }
                    named_barrier(bar, 64);  // both have read: the next chunk may be written
                    with_act(a.act, [&](auto A) {
                        constexpr int ACT = decltype(A)::value;
#pragma unroll
                        for (int j = 0; j < KEEP; ++j) {
                            if constexpr (Cfg::MODE == Exp::GATED_GRAD) {
                                float value;
                                const float slope = act_value_grad<ACT>(g[j], value);
                                g[j] = d[j] * up[j] * slope;
                                up[j] = d[j] * value;
                            } else {
                                g[j] = act_value<ACT>(g[j]) * up[j];
                            }
                        }
                    });
                    if (mine) {
                        const long long at = (row + c0) * a.ldo + feat;
                        uint16_t *o = a.out + at;
                        uint16_t *o2 = Cfg::MODE == Exp::GATED_GRAD ? a.out2 + at : nullptr;
#pragma unroll
                        for (int j = 0; j < KEEP; ++j) {
                            if (c0 + j < left) {
                                put_bf16(o, g[j]);
                                if constexpr (Cfg::MODE == Exp::GATED_GRAD) put_bf16(o2, up[j]);
                            }
                            o += a.ldo;
                            if constexpr (Cfg::MODE == Exp::GATED_GRAD) o2 += a.ldo;
                        }
                    }
                }
            }
        }
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncwarp();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (CG == 2)
            tmem_dealloc_pair(tmem, Cfg::TMEM_COLS);
        else
            tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------ weights' gradients ---
// dW[e] = X_e^T dZ_e in 256 x 256 tiles on a CTA pair, BK rows a step: A = X^T M-major,
// B = dZ N-major, both in boxes of 64 columns.
//
// A product of the tensor core takes 16 rows.  A group's rows in whole sixteens go through
// the ring; what is left of the sixteen that its last row lies in belongs to the next
// group, and may hold anything.  Those 16 rows have buffers of their own: they are fetched
// when the unit begins, a warp of each CTA clears what is not the group's, and they are
// multiplied last, so that neither the clearing nor the two CTAs' agreement on it is
// waited for.  (Cleared in the ring's last stage, groups of 520 rows took 258 us for 32
// experts' 2048 x 4096, 512 rows 182.)
//
// The tensor core truncates its sums, so an accumulator falls behind by up to 2^-23 of the
// magnitudes in it with every 16 rows.  A group's rows go by in rounds of kWeightsRound,
// each from zero, which the epilogue adds in fp32, rounded to nearest: the error
// of a dW is that of one round, however long its group, and no wait lasts longer than one.
//
// Few rows a group: a unit's output takes longer than its products.  Then a ring of three
// stages instead of four makes room to stage all of a warp's output at once, 64 columns
// wide (WIDE), whose rows of 128 bytes also write fewer 32-byte sectors in part where the
// matrix's rows start anywhere in one.  us with three and with four stages, sizes of groups
// that spread by half: 32 experts 2048 x 4096, 24 rows a group 123 and 127, 256 rows 153 and
// 170, 320 rows 165 and 172, 448 rows 192 and 187; 64 experts 1024 x 1368 8 rows 52 and 60,
// 256 rows 70 and 77, 448 rows 92 and 89 (all before sums went by rounds, which cost some
// 0.5 %).  (Where rows start on 128 bytes and experts are
// small four stages are the quicker below some 128 rows too: 1024 x 2048, 96 rows 82 and 79.)
// What is left is writing dW (8 rows each of 64 experts 1024 x 2048: 4.2 TB/s, a memset's
// rate) and, with more rows, the traffic of both directions beside the products (512 rows
// 183 us, 1.50 PFLOP/s; one expert of 8192 rows 1.95).
template <int BK_, int STAGES_, int NBUF_, bool WIDE_>
struct ExpWeightsCfg {
    static constexpr bool WIDE = WIDE_;
    static constexpr int BM = 128, BN = 256, BK = BK_, STAGES = STAGES_, NBUF = NBUF_;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN / 2 * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int TAIL_HALF = 128 * 16 * 2, TAIL_BYTES = 2 * TAIL_HALF;  // a buffer
    static constexpr int EPI = 8, EPI_COLS = BN / 2;
    static constexpr int TAIL_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int STAGING_OFFSET = TAIL_OFFSET + 2 * TAIL_BYTES;
    static constexpr int BAR_OFFSET = STAGING_OFFSET + EPI * NBUF * 2048;
    static constexpr int USED = BAR_OFFSET + (2 * STAGES + 13) * 8 + 16;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int THREADS = 64 + 32 * EPI + 32;
    static constexpr int SMEM_BYTES = smem_request(USED + 1024, 1);
    static_assert(USED + 1024 <= 232448, "shared memory");
    static_assert(WIDE ? NBUF == EPI_COLS / 32 : EPI_COLS / 32 % NBUF == 0, "whole batches");
    static_assert(BK == 96, "a step's rows are one box of 96, 64 or 32");
};

// Rows of a round: whole steps, and as many as a round's error of 516 truncations (2^-14 of
// the sum of magnitudes, a sixty-fourth of bf16's rounding) allows.
constexpr int kWeightsRound = 96 * 86;
// What a step may take at most where a wait spans a unit's steps: ten times what it takes.
constexpr uint64_t kWeightsStepNs = 4000;

struct WeightsUnit {
    int expert, begin, end, seg, m0, n0;
    __device__ __forceinline__ int whole() const { return begin + (end - begin) / 16 * 16; }
    // (one for a group of fewer than 16 rows; without rows there are none)
    __device__ __forceinline__ int rounds() const {
        const int rows = whole() - begin;
        return rows > 0 ? (rows - 1) / kWeightsRound + 1 : 1;
    }
};

template <class Cfg>
__device__ __forceinline__ WeightsUnit weights_unit(const ExpertsArgs &a, int u) {
    WeightsUnit w;
    const int n_tiles = a.n_seg * a.segments, per = a.f_tiles * n_tiles;
    w.expert = u / per;
    w.begin = warp_value(min(max(a.offsets[w.expert], 0), a.R));
    w.end = warp_value(min(max(a.offsets[w.expert + 1], w.begin), a.R));
    const int r = u - w.expert * per;
    const int group = r / (8 * n_tiles), first = group * 8;
    const int g = min(a.f_tiles - first, 8), q = r - group * 8 * n_tiles;
    const int nt = q / g;
    w.m0 = (first + q % g) * (Cfg::BM * 2);
    w.seg = nt >= a.n_seg ? 1 : 0;
    w.n0 = (nt - w.seg * a.n_seg) * Cfg::BN;
    return w;
}

// Zeros for an expert without rows: part `i` of `parts` of its matrix, `size` elements at p,
// by the pair's epilogue warps, `thread` of 512.  One contiguous run whatever the pitch (64
// experts 1024 x 2047, seven with rows: 55 us, 4.8 TB/s; as tiles 119).
__device__ __forceinline__ void put_zeros(uint16_t *p, long long size, int i, int parts,
                                          unsigned thread) {
    const long long share = ((size - 1) / parts + 8) / 8 * 8;
    const long long lo = min(size, i * share), hi = min(size, lo + share);
    uint16_t *begin = p + lo, *end = p + hi;
    // whole vectors from `a` to `z`
    const int head = static_cast<int>((0u - static_cast<unsigned>(
                                                reinterpret_cast<uintptr_t>(begin) >> 1)) & 7u);
    uint16_t *a = begin + min(hi - lo, static_cast<long long>(head));
    uint16_t *z = a + (end - a) / 8 * 8;
    for (uint16_t *at = a + 8ll * thread; at < z; at += 8 * 512)
        *reinterpret_cast<uint4 *>(at) = make_uint4(0u, 0u, 0u, 0u);
    if (begin + thread < a) begin[thread] = 0;
    if (z + thread < end) z[thread] = 0;
}

// put_rows32_batch for a matrix of a 3-D map.
template <int B, class Ctx>
__device__ __forceinline__ void put_rows32_batch_3d(Ctx &c, const CUtensorMap *map, int z, int col,
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
        for (int b = 0; b < B; ++b)
            if (col + 32 * b < c.N)
                tma_store_3d(map, c.bufs + (buf[b] - smem_u32(c.bufs)), col + 32 * b, c.m0, z);
        // one group holds all B stores; the others keep the count
#pragma unroll
        for (int b = 0; b < B; ++b) bulk_commit();
    }
    __syncwarp();
}

// 64-column blocks side by side, in 4 KB each with the 128-byte swizzle (16-byte chunk j of
// row r at j ^ (r % 8)), all of a warp's columns at once.
template <int BLOCKS, class Ctx>
__device__ __forceinline__ void put_rows64_3d(Ctx &c, const CUtensorMap *map, int z, int col,
                                              const uint32_t *p) {
    static_assert(2 * BLOCKS == Ctx::NB, "staging buffers");
    if (c.m0 >= c.M || col >= c.N) return;
    if (c.lane == 0) bulk_wait_read<0>();
    __syncwarp();
    const uint32_t base = smem_u32(c.bufs);
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            sts128(base + b * 4096 + c.lane * 128 + ((j ^ (c.lane & 7u)) << 4), p[32 * b + 4 * j],
                   p[32 * b + 4 * j + 1], p[32 * b + 4 * j + 2], p[32 * b + 4 * j + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (c.lane == 0) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
            if (col + 64 * b < c.N) tma_store_3d(map, c.bufs + b * 4096, col + 64 * b, c.m0, z);
        bulk_commit();
    }
    __syncwarp();
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    experts_weights_kernel(const __grid_constant__ ExpertsWeightsMaps maps, const ExpertsArgs a,
                           const KernelCtx ctx) {
    constexpr int STAGES = Cfg::STAGES, BK = Cfg::BK, BM = Cfg::BM, BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    uint8_t *sA = smem, *sB = smem + STAGES * Cfg::A_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFFSET);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_empty = acc_full + 2;   // [2]
    uint64_t *mma_done = acc_empty + 2;
    uint64_t *tail_full = mma_done + 1;   // [2] last rows fetched, in this CTA
    uint64_t *tail_peer = tail_full + 2;  // [2] the peer's are cleared
    uint64_t *tail_ready = tail_peer + 2; // [2] both are
    uint64_t *tail_empty = tail_ready + 2;  // [2] they have been multiplied
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail_empty + 2);
    const uint32_t warp = warp_id_uniform(), lane = lane_id();
    const int crank = static_cast<int>(cluster_ctarank());
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&maps.x[0]);
        prefetch_tmap(&maps.z[0][0]);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail_full[b], 1);
            mbar_init(&tail_peer[b], 1);
            mbar_init(&tail_ready[b], 1);
            mbar_init(&tail_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI * 2);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    op_begin(a.overlap);
    const int units = a.E * a.f_tiles * a.n_seg * a.segments;
    const int slot = static_cast<int>(blockIdx.x) / 2, slots = static_cast<int>(gridDim.x) / 2;

    // The first two warps run as one each, with one lane's instructions (see warp_value).
    const uint32_t lead = lane == 0 ? 1u : 0u;
    if (warp == 0) {
        // ---------------- producer ----------------
        Ring<STAGES> ring;
        uint32_t tails = 0;
        bool ok = true;
        const uint32_t full0 = smem_u32(full);
        const uint32_t full_lead = warp_value(mapa_shared(full0, 0));
        const uint32_t first = crank == 0 ? lead : 0u;
        for (int u = slot; u < units; u += slots) {
            const WeightsUnit w = weights_unit<Cfg>(a, u);
            const CUtensorMap *mx = maps.x, *mz = maps.z[w.seg];
            const int ma = w.m0 + crank * BM, nb = w.n0 + crank * (BN / 2);
            const int whole = w.whole();
            if (whole < w.end) {
                const uint32_t b = tails & 1u;
                if (ok)
                    ok = warp_value(mbar_wait(&tail_empty[b], ((tails >> 1) & 1u) ^ 1u, ctx,
                                              kSiteGroupTail)) != 0;
                ++tails;
                const uint32_t go = ok ? lead : 0u;  // (after a failure nothing is issued)
                const uint32_t d = smem_u32(smem + Cfg::TAIL_OFFSET) + b * Cfg::TAIL_BYTES;
                const uint32_t bar = smem_u32(&tail_full[b]);
                mbar_arrive_expect_tx_if(go, bar, Cfg::TAIL_BYTES);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tma_load_2d_if<1>(go, d + j * 2048, &mx[3], bar, ma + 64 * j, whole);
                    tma_load_2d_if<1>(go, d + Cfg::TAIL_HALF + j * 2048, &mz[3], bar, nb + 64 * j,
                                      whole);
                }
            }
            for (int left = whole - w.begin; left > 0; left -= BK, ring.next()) {
                const int y = whole - left;
                const uint32_t s = ring.s;
                if (ok)
                    ok = warp_value(mbar_wait(&empty[s], ring.phase ^ 1u, ctx,
                                              kSiteProducerEmpty)) != 0;
                const uint32_t go = ok ? lead : 0u;
                const uint32_t da = smem_u32(sA) + s * Cfg::A_BYTES;
                const uint32_t db = smem_u32(sB) + s * Cfg::B_BYTES;
                const uint32_t bar = full_lead + s * 8;
                // a box of 96 rows, in a last step perhaps of 64 or 32
                const int box = left > 64 ? 0 : left > 32 ? 1 : 2;
                mbar_arrive_expect_tx_if(ok ? first : 0u, full0 + s * 8,
                                         (96 - 32 * box) * (2 * Cfg::STAGE_BYTES / BK));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tma_load_2d_if<2>(go, da + j * (BK * 128), &mx[box], bar, ma + 64 * j, y);
                    tma_load_2d_if<2>(go, db + j * (BK * 128), &mz[box], bar, nb + 64 * j, y);
                }
            }
        }
        // the pair's last multicast releases of this CTA's barriers must have landed
        // before the cluster is left
        for (int i = 0; ok && i < STAGES; ++i, ring.next())
            ok = warp_value(mbar_wait(&empty[ring.s], ring.phase ^ 1u, ctx, kSiteProducerEmpty)) != 0;
        for (int i = 0; ok && i < 2; ++i, ++tails)
            ok = warp_value(mbar_wait(&tail_empty[tails & 1u], ((tails >> 1) & 1u) ^ 1u, ctx,
                                      kSiteGroupTail)) != 0;
    } else if (warp == Cfg::THREADS / 32 - 1) {
        // ---------------- the groups' last rows ----------------
        uint32_t tails = 0;
        uint64_t steps = 0;  // of the units since the last such rows
        for (int u = slot; u < units; u += slots) {
            const WeightsUnit w = weights_unit<Cfg>(a, u);
            const int rows = w.end - w.whole();
            const uint64_t waited = steps;
            steps = (rows == 0 ? steps : 0) + static_cast<uint64_t>((w.end - w.begin) / BK + 1);
            if (rows == 0) continue;
            const uint32_t b = tails & 1u, ph = (tails >> 1) & 1u;
            ++tails;
            // (every lane waits: it must see the copies before it overwrites them)
            if (!__all_sync(0xffffffffu,
                            mbar_wait_behind(&tail_full[b], ph, ctx, kSiteGroupTail,
                                             waited * kWeightsStepNs)))
                break;
            const uint32_t d = smem_u32(smem + Cfg::TAIL_OFFSET + b * Cfg::TAIL_BYTES);
            for (int r = rows * 8 + static_cast<int>(lane); r < 16 * 8; r += 32)
#pragma unroll
                for (int j = 0; j < 4; ++j) sts128(d + j * 2048 + r * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (crank == 1)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&tail_peer[b]), 0));
                else if (mbar_wait_cluster(&tail_peer[b], ph, ctx, kSiteGroupTail))
                    mbar_arrive(&tail_ready[b]);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        if (crank == 0) {
            // ---------------- MMA issuer ----------------
            constexpr uint16_t kPair = 3;
            constexpr uint32_t idesc = idesc_f16(BM * 2, BN, 1, 1, 1);
            const uint64_t a0 = smem_desc_sw128(smem_u32(sA), BK * 128, 1024);
            const uint64_t b0 = smem_desc_sw128(smem_u32(sB), BK * 128, 1024);
            const uint32_t tmem_w = warp_value(tmem);
            Ring<STAGES> ring;
            uint32_t n = 0, tails = 0;
            bool ok = true;
            for (int u = slot; u < units; u += slots) {
                const WeightsUnit w = weights_unit<Cfg>(a, u);
                if (w.end <= w.begin) continue;
                const int whole = w.whole();
                int left = whole - w.begin;
                do {  // a round
                    const uint32_t ab = n & 1u;
                    if (ok)
                        ok = warp_value(mbar_wait(&acc_empty[ab], ((n >> 1) & 1u) ^ 1u, ctx,
                                                  kSiteMmaAccEmpty)) != 0;
                    ++n;
                    tc_fence_after();
                    const uint32_t d = tmem_w + ab * BN;
                    const int rest = max(left - kWeightsRound, 0);  // of the rounds after
                    uint32_t acc = 0;
                    for (; left > rest; left -= BK, ring.next()) {
                        const uint32_t s = ring.s;
                        if (ok)
                            ok = warp_value(mbar_wait(&full[s], ring.phase, ctx,
                                                      kSiteMmaFull)) != 0;
                        const uint32_t go = ok ? lead : 0u;
                        tc_fence_after();
                        const uint64_t as = a0 + s * (Cfg::A_BYTES / 16);
                        const uint64_t bs = b0 + s * (Cfg::B_BYTES / 16);
                        auto multiply = [&](int k) {
                            umma_f16_ss_if<2>(go, d, as + k * 128, bs + k * 128, idesc, acc);
                            acc = 1;
                        };
                        if (left >= BK) {
#pragma unroll
                            for (int k = 0; k < BK / 16; ++k) multiply(k);
                        } else {
#pragma unroll 1
                            for (int k = 0; 16 * k < left; ++k) multiply(k);
                        }
                        umma_commit_if<2>(go, smem_u32(&empty[s]), kPair);
                    }
                    if (left <= 0 && whole < w.end) {
                        const uint32_t b = tails & 1u;
                        if (ok)
                            ok = warp_value(mbar_wait(&tail_ready[b], (tails >> 1) & 1u, ctx,
                                                      kSiteGroupTail)) != 0;
                        ++tails;
                        tc_fence_after();
                        const uint32_t st =
                            smem_u32(smem + Cfg::TAIL_OFFSET) + b * Cfg::TAIL_BYTES;
                        umma_f16_ss_if<2>(ok ? lead : 0u, d, smem_desc_sw128(st, 2048, 1024),
                                          smem_desc_sw128(st + Cfg::TAIL_HALF, 2048, 1024), idesc,
                                          acc);
                        umma_commit_if<2>(ok ? lead : 0u, smem_u32(&tail_empty[b]), kPair);
                    }
                    umma_commit_if<2>(ok ? lead : 0u, smem_u32(&acc_full[ab]), kPair);
                } while (left > 0);
            }
            umma_commit_if<2>(lead, smem_u32(mma_done), 1);
            mbar_wait(mma_done, 0, ctx, kSiteMmaDone);
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        const uint32_t e = warp - 2, q = warp & 3u;
        EpiCtx<Cfg::NBUF> c;
        c.bufs = smem + Cfg::STAGING_OFFSET + e * (Cfg::NBUF * 2048);
        c.n = 0;
        c.M = a.K;  // dW is K x M: the rows of X are its output's rows here
        c.N = a.M;
        c.lane = lane;
        const int col0 = static_cast<int>(e >> 2) * Cfg::EPI_COLS;
        uint32_t n = 0;
        for (int u = slot; u < units; u += slots) {
            const WeightsUnit w = weights_unit<Cfg>(a, u);
            c.m0 = w.m0 + crank * BM + static_cast<int>(q * 32);
            uint16_t *matrix = (w.seg ? a.out2 : a.out) +
                               static_cast<long long>(w.expert) * a.K * a.M;
            if (w.end <= w.begin) {
                put_zeros(matrix, static_cast<long long>(a.K) * a.M,
                          w.m0 / (BM * 2) * a.n_seg + w.n0 / BN, a.f_tiles * a.n_seg,
                          crank * 256 + e * 32 + lane);
                continue;
            }
            constexpr int C = Cfg::EPI_COLS / 32, B = C < Cfg::NBUF ? C : Cfg::NBUF;
            uint32_t v[32 * C];
            const bool several = w.whole() - w.begin > kWeightsRound;
            // The sum of the rounds before the last: in local memory, so that the groups of one
            // round, nearly all, keep their registers as they were (in registers: 1 % more time
            // for 32 experts of 512 rows).
            float sums[32 * C];
            if (several) {
                bool ok = true;
                const int before = w.rounds() - 1;
#pragma unroll 1
                for (int r = 0; r < before; ++r) {
                    const uint32_t ab = n & 1u;
                    ok = mbar_wait(&acc_full[ab], (n >> 1) & 1u, ctx, kSiteEpilogueFull);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem + ((q * 32u) << 16) + ab * BN + col0;
#pragma unroll 1
                    for (int b = 0; b < C; ++b) {
                        uint32_t x[32];
                        tmem_ld_32x32b_x32(t_row + 32 * b, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            sums[32 * b + j] =
                                __uint_as_float(x[j]) + (r > 0 ? sums[32 * b + j] : 0.0f);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[ab]), 0));
                    ++n;
                }
                if (!ok) break;
            }
            const uint32_t ab = n & 1u;
            const uint32_t t_row = tmem + ((q * 32u) << 16) + ab * BN + col0;
            if (!mbar_wait(&acc_full[ab], (n >> 1) & 1u, ctx, kSiteEpilogueFull)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < C; ++b)
                tmem_ld_32x32b_x32(t_row + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * b));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[ab]), 0));
            ++n;
            if (several) {
#pragma unroll
                for (int j = 0; j < 32 * C; ++j)
                    v[j] = __float_as_uint(__uint_as_float(v[j]) + sums[j]);
            }
#pragma unroll
            for (int j = 0; j < 16 * C; ++j)
                v[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            if (Cfg::WIDE && a.tma_out) {
                if constexpr (Cfg::WIDE)
                    put_rows64_3d<C / 2>(c, &maps.c[w.seg], w.expert, w.n0 + col0, v);
            } else if (a.tma_out) {
#pragma unroll
                for (int b = 0; b < C; b += B)
                    put_rows32_batch_3d<B>(c, &maps.c[w.seg], w.expert, w.n0 + col0 + 32 * b,
                                           v + 16 * b);
            } else {
#pragma unroll
                for (int b = 0; b < C; ++b)
                    put_rows32(c, nullptr, matrix, a.M, w.n0 + col0 + 32 * b, v + 16 * b);
            }
        }
        if (lane == 0) bulk_wait_all();  // this warp's stores have landed
        __syncwarp();
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, Cfg::TMEM_COLS);
    }
    op_end(a.overlap);
}

// A call's sizes: R rows, N outputs (gated: features), K reduction columns, E experts.
struct ExpSizes {
    int R, N, K, E;
    const int32_t *offsets;
};

// --------------------------------------------------------------- relayout ---
// Matrices whose rows are no multiples of 16 bytes, to a pitch that TMA reads: many short
// rows (an expert's weights), so a thread takes 16-byte vectors of the whole copy in turn,
// each shifted out of the two aligned ones that cover it.  blockIdx.y is the expert: those
// without rows are not copied.  Bound by HBM: 171 MB in rows of 1686 bytes in 55 us, 6.2 TB/s
// (a block a row at a time: 117).
struct RelayoutParams {
    const uint16_t *src;
    uint16_t *dst;
    unsigned long long rows, vecs;  // of a matrix's copy
    unsigned row_vecs, cols;
    long long ld, end;       // elements of a row of the copy, and of the source
    const int32_t *offsets;  // nullptr: one matrix
    int early;               // op_begin_early
};

__global__ void __launch_bounds__(256) relayout_kernel(const RelayoutParams p) {
    op_begin_early(p.early);
    const unsigned e = blockIdx.y;
    if (p.offsets != nullptr && p.offsets[e + 1] <= p.offsets[e]) return;
    constexpr int AHEAD = 4;
    const unsigned long long first = blockIdx.x * (256ull * AHEAD) + threadIdx.x;
    uint4 lo[AHEAD], hi[AHEAD];
    long long to[AHEAD];
    uint32_t off[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        const unsigned long long i = first + 256 * u;
        to[u] = -1;
        if (i >= p.vecs) continue;
        const unsigned long long row = p.vecs >> 32 == 0
                                           ? static_cast<unsigned>(i) / p.row_vecs
                                           : i / p.row_vecs;
        const unsigned c = 8 * static_cast<unsigned>(i - row * p.row_vecs);
        const unsigned long long all = e * p.rows + row;  // of all matrices' rows
        const long long from = static_cast<long long>(all * p.cols) + c;
        to[u] = static_cast<long long>(all) * p.ld + c;
        off[u] = static_cast<uint32_t>(from & 7) * 2u;
        const long long at = from & ~7ll;
        if (at + 16 <= p.end) {
            lo[u] = __ldg(reinterpret_cast<const uint4 *>(p.src + at));
            hi[u] = __ldg(reinterpret_cast<const uint4 *>(p.src + at) + 1);
        } else {  // the source's last elements, one by one
            uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (at + j < p.end)
                    w[j / 2] |= static_cast<uint32_t>(p.src[at + j]) << (j % 2 * 16);
            lo[u] = make_uint4(w[0], w[1], w[2], w[3]);
            hi[u] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        if (to[u] < 0) continue;
        uint32_t w[4];
        shift16(lo[u], hi[u], off[u], w);
        *reinterpret_cast<uint4 *>(p.dst + to[u]) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// As OpRelayout: the copies are planned, then made; a matrix that TMA reads stays.
class ExpRelayout {
  public:
    void add(OpMat *out, const uint16_t *src, long long rows, long long cols, OpArena &arena) {
        out->p = src;
        out->ld = cols;
        if (cols % 8 == 0 || rows == 0 || cols == 0) return;
        const long long ld = op_round_up(cols, 64);
        jobs_[n_++] = Job{out, src, rows, cols, ld, arena.add(rows * ld * 2), nullptr, 1};
    }
    // E matrices of K x N
    void add_weights(OpMat *out, const uint16_t *src, const ExpSizes &z, OpArena &arena) {
        const int before = n_;
        add(out, src, static_cast<long long>(z.E) * z.K, z.N, arena);
        if (n_ > before) {
            jobs_[before].offsets = z.offsets;
            jobs_[before].experts = z.E;
        }
    }
    pgemm_status run(const OpDevice &dev, OpArena &arena, cudaStream_t s) {
        for (int i = 0; i < n_; ++i) {
            const Job &j = jobs_[i];
            RelayoutParams p{};
            p.src = j.src;
            p.dst = arena.at<uint16_t>(j.at);
            p.row_vecs = static_cast<unsigned>((j.cols + 7) / 8);
            p.rows = static_cast<unsigned long long>(j.rows / j.experts);
            p.vecs = p.rows * p.row_vecs;
            p.cols = static_cast<unsigned>(j.cols);
            p.ld = j.ld;
            p.end = j.rows * j.cols;
            p.offsets = j.offsets;
            j.out->p = p.dst;
            j.out->ld = j.ld;
            const unsigned long long blocks = (p.vecs + 1023) / 1024;
            if (blocks > INT_MAX) return PGEMM_ERR_TOO_LARGE;
            const dim3 grid(static_cast<unsigned>(blocks), j.experts);
            p.early = blocks * j.experts <= static_cast<unsigned>(dev.sm_count);
            const pgemm_status st = launch_small(relayout_kernel, grid, dim3(256), s, p);
            if (st != PGEMM_OK) return st;
        }
        return PGEMM_OK;
    }

  private:
    struct Job {
        OpMat *out;
        const uint16_t *src;
        long long rows, cols, ld, at;
        const int32_t *offsets;
        int experts;
    };
    Job jobs_[4];
    int n_ = 0;
};

// ------------------------------------------------------------------- host ---
template <class Maps>
using ExpKernel = void (*)(const Maps, const ExpertsArgs, const KernelCtx);

template <int CG>
static cudaError_t exp_slots_of(const void *func, int threads, int smem, int sm_count, int *slots) {
    if constexpr (CG == 1) {
        *slots = sm_count;
        return cudaSuccess;
    } else {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CG;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t lc{};
        lc.blockDim = dim3(threads);
        lc.dynamicSmemBytes = smem;
        lc.gridDim = dim3(CG * sm_count);
        lc.attrs = attr;
        lc.numAttrs = 1;
        int clusters = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, func, &lc);
        if (e != cudaSuccess) return e;
        if (clusters < 1) return cudaErrorInvalidConfiguration;
        *slots = clusters;
        return cudaSuccess;
    }
}

// One launch on as many CTAs (pairs) as run at once, or as there can be units.
template <class Cfg, int CG, class Maps, ExpKernel<Maps> KERNEL>
static pgemm_status exp_launch(const OpDevice &dev, const Maps &maps, const ExpertsArgs &a,
                               long long most_units, cudaStream_t stream) {
    static const KernelInfo info = [] {
        KernelInfo k;
        k.threads = Cfg::THREADS;
        k.smem_bytes = Cfg::SMEM_BYTES;
        k.func = reinterpret_cast<const void *>(KERNEL);
        k.schedule_slots = [](const LaunchCommon &p, int *slots) {
            return exp_slots_of<CG>(reinterpret_cast<const void *>(KERNEL), Cfg::THREADS,
                                    Cfg::SMEM_BYTES, p.sm_count, slots);
        };
        return k;
    }();
    int slots = 0;
    const pgemm_status st = op_kernel_setup(dev, info, &slots);
    if (st != PGEMM_OK) return st;
    if (most_units > kUnitsMost) return PGEMM_ERR_TOO_LARGE;
    cudaLaunchAttribute attr[2];
    int nattr = 0;
    attr[nattr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[nattr].val.programmaticStreamSerializationAllowed = 1;
    ++nattr;
    if constexpr (CG == 2) {
        attr[nattr].id = cudaLaunchAttributeClusterDimension;
        attr[nattr].val.clusterDim.x = 2;
        attr[nattr].val.clusterDim.y = 1;
        attr[nattr].val.clusterDim.z = 1;
        ++nattr;
    }
    cudaLaunchConfig_t lc{};
    lc.blockDim = dim3(Cfg::THREADS);
    lc.gridDim = dim3(CG * static_cast<int>(most_units < slots ? most_units : slots));
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = nattr;
    return cudaLaunchKernelEx(&lc, KERNEL, maps, a, dev.ctx) == cudaSuccess ? PGEMM_OK
                                                                            : PGEMM_ERR_CUDA;
}

template <class Cfg>
static pgemm_status rows_launch(const OpDevice &dev, const ExpSizes &z, const OpMat *x,
                                const OpMat *w, int segments, ExpertsArgs a, cudaStream_t s) {
    // TRANSPOSED: z.N is the reduction, z.K the features
    constexpr bool T = Cfg::W_K;
    a.R = z.R;
    a.E = z.E;
    a.M = T ? z.K : z.N;
    a.K = T ? z.N : z.K;
    a.offsets = z.offsets;
    a.k_seg = op_blocks(a.K, Cfg::BK);
    a.k_tiles = a.k_seg * segments;
    a.f_tiles = op_blocks(a.M, Cfg::FEATS * Cfg::CG);
    ExpertsMaps maps{};
    const int ws = Cfg::DUAL ? 2 : segments;
    pgemm_status st = PGEMM_OK;
    for (int j = 0; a.K > 0 && j < segments; ++j)
        for (int b = 0; b < 3 && st == PGEMM_OK; ++b)
            st = op_encode(&maps.x[j][b], x[j].p, a.K, z.R, x[j].ld, Cfg::BOX * (4 >> b));
    for (int j = 0; a.K > 0 && j < ws && st == PGEMM_OK; ++j)
        st = op_encode_3d(&maps.w[j], w[j].p, z.N, z.K, z.E, w[j].ld, T ? 128 : Cfg::BK);
    if (st != PGEMM_OK) return st;
    // units at most: every tile of rows full, and a partial one more for each expert
    const long long live = z.R < z.E ? z.R : z.E;
    const long long most = (z.R / Cfg::TOK + live) * a.f_tiles;
    return exp_launch<Cfg, Cfg::CG, ExpertsMaps, experts_rows_kernel<Cfg>>(dev, maps, a, most, s);
}

template <Exp MODE>
static pgemm_status rows_product(const OpDevice &dev, const ExpSizes &z, const OpMat *x,
                                 const OpMat *w, int segments, const ExpertsArgs &a,
                                 cudaStream_t s) {
    // Few rows a group: the weights are all there is to read, and single CTAs with small
    // tiles of rows keep more of them on the way: 64 experts 2048 x 1024, 16 rows each, 45 us
    // (6.1 TB/s) against 48 on pairs, 40 rows 47 against 49.5.  Groups that pass a tile's 64
    // rows read them twice (96 rows: 63 against 52), and groups are uneven: 16 experts 1024 x
    // 4096 of sizes that spread by half, a mean of 40 rows 25.9 against 27.3, of 48 35.5
    // against 27.6.  And few tiles: smaller ones on more SMs (one expert, 512 rows 1024 x
    // 2048: 10 against 16).
    const long long live = z.R < z.E ? z.R : z.E;
    const long long pairs =
        (z.R / 256 + live) * op_blocks(MODE == Exp::TRANSPOSED ? z.K : z.N,
                                       MODE == Exp::LINEAR || MODE == Exp::TRANSPOSED ? 256 : 128);
    if (z.R <= 40ll * z.E || 4 * pairs <= dev.sm_count)
        return rows_launch<ExpCfg<1, 64, 128, 4, MODE>>(dev, z, x, w, segments, a, s);
    return rows_launch<ExpCfg<2, 256, 64, 6, MODE>>(dev, z, x, w, segments, a, s);
}

template <class Cfg>
static pgemm_status weights_launch(const OpDevice &dev, const ExpSizes &z, const OpMat &x,
                                   const OpMat *dz, int segments, uint16_t *const *out,
                                   bool overlap, cudaStream_t s) {
    ExpertsArgs a{};
    a.R = z.R;
    a.E = z.E;
    a.M = z.N;
    a.K = z.K;
    a.offsets = z.offsets;
    a.f_tiles = op_blocks(z.K, 256);
    a.n_seg = op_blocks(z.N, 256);
    a.segments = segments;
    a.out = out[0];
    a.out2 = segments > 1 ? out[1] : nullptr;
    a.tma_out = z.N % 8 == 0;
    a.overlap = overlap ? 1 : 0;
    ExpertsWeightsMaps maps{};
    constexpr int kBoxes[4] = {96, 64, 32, 16};
    pgemm_status st = PGEMM_OK;
    for (int b = 0; b < 4 && st == PGEMM_OK; ++b)
        st = op_encode(&maps.x[b], x.p, z.K, z.R, x.ld, kBoxes[b]);
    for (int j = 0; j < segments && st == PGEMM_OK; ++j) {
        for (int b = 0; b < 4 && st == PGEMM_OK; ++b)
            st = op_encode(&maps.z[j][b], dz[j].p, z.N, z.R, dz[j].ld, kBoxes[b]);
        if (st == PGEMM_OK && a.tma_out)
            st = Cfg::WIDE ? op_encode_3d(&maps.c[j], out[j], z.N, z.K, z.E, z.N, 32)
                           : op_encode_out_3d(&maps.c[j], out[j], z.N, z.K, z.E, z.N);
    }
    if (st != PGEMM_OK) return st;
    const long long units = static_cast<long long>(z.E) * a.f_tiles * a.n_seg * segments;
    return exp_launch<Cfg, 2, ExpertsWeightsMaps, experts_weights_kernel<Cfg>>(dev, maps, a, units, s);
}

// dW[j][e] = x_e^T dz[j]_e for each of `segments` outputs.  overlap: behind the product for
// dX, which reads what this one reads and writes nothing of it.
static pgemm_status weights_product(const OpDevice &dev, const ExpSizes &z, const OpMat &x,
                                    const OpMat *dz, int segments, uint16_t *const *out,
                                    bool overlap, cudaStream_t s) {
    if (z.R <= 320ll * z.E)  // (see ExpWeightsCfg)
        return weights_launch<ExpWeightsCfg<96, 3, 4, true>>(dev, z, x, dz, segments, out, overlap, s);
    return weights_launch<ExpWeightsCfg<96, 4, 1, false>>(dev, z, x, dz, segments, out, overlap, s);
}

static pgemm_status exp_check(const ExpSizes &z) {
    if (z.R < 0 || z.N < 0 || z.K < 0 || z.E < 1) return PGEMM_ERR_INVALID_VALUE;
    if (z.E > kExpertsMax || static_cast<long long>(z.E) * z.K > INT_MAX)
        return PGEMM_ERR_TOO_LARGE;
    return PGEMM_OK;
}

// Whether a tile's sum over so many columns is taken: every 16 of them truncate it by up to
// 2^-23 of the magnitudes in it, 2^19 by a bf16 rounding's 2^-8.  (A unit's main loop, which
// its epilogue waits for, is then some milliseconds long.)
constexpr long long kSumMost = 1 << 19;
static bool exp_sum_fits(long long columns) { return columns <= kSumMost; }

static pgemm_status zero_bf16(uint16_t *p, long long n, cudaStream_t s) {
    return n == 0 || cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 2, s) == cudaSuccess
               ? PGEMM_OK
               : PGEMM_ERR_CUDA;
}

static pgemm_status experts_linear_forward(const ExpSizes &z, const uint16_t *X, const uint16_t *W,
                                           uint16_t *Y, cudaStream_t s) {
    pgemm_status st = exp_check(z);
    if (st != PGEMM_OK) return st;
    if (!exp_sum_fits(z.K)) return PGEMM_ERR_TOO_LARGE;
    if (z.R == 0 || z.N == 0) return PGEMM_OK;
    if (!z.offsets || !Y || (z.K > 0 && (!X || !W))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(z.offsets) || !op_aligned16(X) || !op_aligned16(W) || !op_aligned16(Y))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    OpArena arena(dev, s);
    ExpRelayout rl;
    OpMat x, w;
    rl.add(&x, X, z.R, z.K, arena);
    rl.add_weights(&w, W, z, arena);
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if (z.K > 0 && (st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    ExpertsArgs a{};
    a.out = Y;
    a.ldo = z.N;
    return rows_product<Exp::LINEAR>(dev, z, &x, &w, 1, a, s);
}

static pgemm_status experts_linear_backward(const ExpSizes &z, const uint16_t *X,
                                            const uint16_t *W, const uint16_t *dY, uint16_t *dX,
                                            uint16_t *dW, cudaStream_t s) {
    pgemm_status st = exp_check(z);
    if (st != PGEMM_OK) return st;
    const bool want_x = dX && z.R > 0 && z.K > 0, want_w = dW && z.K > 0 && z.N > 0;
    if (!want_x && !want_w) return PGEMM_OK;
    if (want_x && !exp_sum_fits(z.N)) return PGEMM_ERR_TOO_LARGE;
    const bool some = z.R > 0 && z.N > 0;
    if (!z.offsets || (some && (!dY || (want_w && !X) || (want_x && !W))))
        return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(z.offsets) || !op_aligned16(X) || !op_aligned16(W) || !op_aligned16(dY) ||
        !op_aligned16(dX) || !op_aligned16(dW))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    if (z.R == 0) return zero_bf16(dW, static_cast<long long>(z.E) * z.K * z.N, s);
    OpArena arena(dev, s);
    ExpRelayout rl;
    OpMat x, w, dy;
    if (some) {
        rl.add(&dy, dY, z.R, z.N, arena);
        if (want_w) rl.add(&x, X, z.R, z.K, arena);
        if (want_x) rl.add_weights(&w, W, z, arena);
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    if (want_x) {
        ExpertsArgs a{};
        a.out = dX;
        a.ldo = z.K;
        st = rows_product<Exp::TRANSPOSED>(dev, z, &dy, &w, 1, a, s);
        if (st != PGEMM_OK) return st;
    }
    return want_w ? weights_product(dev, z, x, &dy, 1, &dW, want_x, s) : PGEMM_OK;
}

// A ReLU gate is not offered: its derivative hangs on the sign of a sum that the tensor
// core truncates (see op_sign_rounds), and the rounds that would mend it need registers
// that this epilogue does not have.
static bool exp_act_known(int act) { return op_act_known(act) && act != PGEMM_ACT_RELU; }

static pgemm_status experts_gated_forward(const ExpSizes &z, const uint16_t *X, const uint16_t *Wg,
                                          const uint16_t *Wu, int act, uint16_t *H, float *preact,
                                          cudaStream_t s) {
    pgemm_status st = exp_check(z);
    if (st != PGEMM_OK) return st;
    if (!exp_act_known(act)) return PGEMM_ERR_INVALID_VALUE;
    if (!exp_sum_fits(z.K)) return PGEMM_ERR_TOO_LARGE;
    if (z.R == 0 || z.N == 0) return PGEMM_OK;
    if (!z.offsets || !H || (z.K > 0 && (!X || !Wg || !Wu))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(z.offsets) || !op_aligned16(X) || !op_aligned16(Wg) || !op_aligned16(Wu) ||
        !op_aligned16(H) || !op_aligned16(preact))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    OpArena arena(dev, s);
    ExpRelayout rl;
    OpMat x, w[2];
    rl.add(&x, X, z.R, z.K, arena);
    rl.add_weights(&w[0], Wg, z, arena);
    rl.add_weights(&w[1], Wu, z, arena);
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if (z.K > 0 && (st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    ExpertsArgs a{};
    a.out = H;
    a.ldo = z.N;
    a.preact = preact;
    a.act = act;
    return rows_product<Exp::GATED>(dev, z, &x, w, 1, a, s);
}

static pgemm_status experts_gated_backward(const ExpSizes &z, const uint16_t *X,
                                           const uint16_t *Wg, const uint16_t *Wu, int act,
                                           const uint16_t *dH, const float *preact, uint16_t *dX,
                                           uint16_t *dWg, uint16_t *dWu, cudaStream_t s) {
    pgemm_status st = exp_check(z);
    if (st != PGEMM_OK) return st;
    if (!exp_act_known(act) || (!dWg) != (!dWu)) return PGEMM_ERR_INVALID_VALUE;
    const bool want_x = dX && z.R > 0 && z.K > 0, want_w = dWg && z.K > 0 && z.N > 0;
    if (!want_x && !want_w) return PGEMM_OK;
    const bool some = z.R > 0 && z.N > 0;
    const bool recompute = some && !preact;
    if ((want_x && !exp_sum_fits(2ll * z.N)) || (recompute && !exp_sum_fits(z.K)))
        return PGEMM_ERR_TOO_LARGE;
    if (!z.offsets || (some && (!dH || ((want_w || recompute) && !X) ||
                                ((want_x || recompute) && (!Wg || !Wu)))))
        return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(z.offsets) || !op_aligned16(X) || !op_aligned16(Wg) || !op_aligned16(Wu) ||
        !op_aligned16(dH) || !op_aligned16(preact) || !op_aligned16(dX) || !op_aligned16(dWg) ||
        !op_aligned16(dWu))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    const long long size = static_cast<long long>(z.E) * z.K * z.N;
    if (z.R == 0) {
        st = zero_bf16(dWg, size, s);
        return st == PGEMM_OK ? zero_bf16(dWu, size, s) : st;
    }
    OpArena arena(dev, s);
    ExpRelayout rl;
    OpMat x, w[2], dz[2];
    if (some) {
        if (want_w || recompute) rl.add(&x, X, z.R, z.K, arena);
        if (want_x || recompute) {
            rl.add_weights(&w[0], Wg, z, arena);
            rl.add_weights(&w[1], Wu, z, arena);
        }
    }
    const long long dz_ld = op_round_up(z.N, 64);
    const long long at0 = arena.add(dz_ld * z.R * 2), at1 = arena.add(dz_ld * z.R * 2);
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    for (int j = 0; j < 2; ++j) dz[j] = OpMat{arena.at<uint16_t>(j ? at1 : at0), dz_ld};
    if (some && preact) {
        OpActGrad g;
        g.M = z.R;
        g.N = z.N;
        g.act = act;
        g.z = preact;
        g.u = preact + static_cast<long long>(z.R) * z.N;
        g.dy = dH;
        g.dy_ld = z.N;
        g.dz = arena.at<uint16_t>(at0);
        g.du = arena.at<uint16_t>(at1);
        g.dz_ld = dz_ld;
        g.early = false;
        if ((st = op_act_grad(dev, g, arena, false, s)) != PGEMM_OK) return st;
    } else if (some) {
        ExpertsArgs a{};
        a.out = arena.at<uint16_t>(at0);
        a.out2 = arena.at<uint16_t>(at1);
        a.ldo = dz_ld;
        a.dy = dH;
        a.act = act;
        st = rows_product<Exp::GATED_GRAD>(dev, z, &x, w, 1, a, s);
        if (st != PGEMM_OK) return st;
    }
    if (want_x) {
        ExpertsArgs a{};
        a.out = dX;
        a.ldo = z.K;
        if ((st = rows_product<Exp::TRANSPOSED>(dev, z, dz, w, 2, a, s)) != PGEMM_OK) return st;
    }
    uint16_t *out[2] = {dWg, dWu};
    return want_w ? weights_product(dev, z, x, dz, 2, out, want_x, s) : PGEMM_OK;
}

}  // namespace pg

extern "C" {

pgemm_status experts_linear_bf16(int R, int N, int K, int E, const int32_t *offsets,
                                 const uint16_t *X, const uint16_t *W, uint16_t *Y,
                                 pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::experts_linear_forward(pg::ExpSizes{R, N, K, E, offsets}, X, W, Y, stream);
    });
}

pgemm_status experts_linear_bf16_backward(int R, int N, int K, int E, const int32_t *offsets,
                                          const uint16_t *X, const uint16_t *W, const uint16_t *dY,
                                          uint16_t *dX, uint16_t *dW, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::experts_linear_backward(pg::ExpSizes{R, N, K, E, offsets}, X, W, dY, dX, dW,
                                           stream);
    });
}

pgemm_status experts_gated_bf16(int R, int F, int K, int E, const int32_t *offsets,
                                const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu, int act,
                                uint16_t *H, float *preact, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::experts_gated_forward(pg::ExpSizes{R, F, K, E, offsets}, X, Wg, Wu, act, H,
                                         preact, stream);
    });
}

pgemm_status experts_gated_bf16_backward(int R, int F, int K, int E, const int32_t *offsets,
                                         const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
                                         int act, const uint16_t *dH, const float *preact,
                                         uint16_t *dX, uint16_t *dWg, uint16_t *dWu,
                                         pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::experts_gated_backward(pg::ExpSizes{R, F, K, E, offsets}, X, Wg, Wu, act, dH,
                                          preact, dX, dWg, dWu, stream);
    });
}

}  // extern "C"
