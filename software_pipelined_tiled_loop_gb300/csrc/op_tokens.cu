// Products of a few rows (up to 128 tokens, of a decoding step or a small batch; more
// where there are too few tiles for the GPU otherwise, tokens_beat):
// Y = act(X W + b) + R, H = act(X Wg) * (X Wu), what their backward passes
// recompute, and dX = dZ W^T; all bound by streaming the weights once.
//
// The weights take the tensor core's M side: D[n][t] = sum_k W[k][n] X[t][k],
// A = W^T read M-major straight from the K x N rows by TMA (64-column boxes of
// 64 k-rows), B = X K-major with N = 16 .. 128 tokens.  An SM's ring then holds
// weights, not padding of X: 128 x 128 tiles with a token a row would load as
// many bytes for one token as for 128.  A thread owns one output column, so
// bias, residual and stores run along n, coalesced for every token.  dX = dZ W^T
// reads the same rows as D[k][t] = sum_n W[k][n] dZ[t][n], A = W K-major.
//
// Long axis: a cluster of S CTAs shares a 128-column tile, CTA r taking K steps
// [r T / S, (r + 1) T / S).  The fp32 partial sums meet in the CTAs' own shared
// memory: after a cluster barrier each CTA adds, in rank order, the partials of
// its share of the tokens (a warp a token, a lane four columns, so that the
// peers' sums come as 16-byte loads) and writes those outputs.  No scratch, no
// second kernel, the same bits every time.
//
// Bound by HBM: a call from a graph over cold weights reads 134 MB (gated 1 x
// 8192 x 4096) in 22.3 us (6.0 TB/s of a measured 6.8), 67 MB (24 x 16384 x
// 2048) in 15.4, 33.5 MB (1 x 4096 x 4096) in 9.3 and nothing to speak of (1 x
// 512 x 512) in 4.1: some 4 us are launch, first loads, barriers and exit.
//
// Rings are sized for two CTAs an SM (S chosen for one such CTA an SM took 11.8 us
// for 1 x 4096 x 4096 and 30 for 24 x 16384 x 2048), and the next kernel in the stream may
// start its CTAs while this one drains: before they wait for it they ask L2 for
// their first weights.  That is safe whatever the kernel before writes, since
// a prefetch moves nothing past L2, where all writes meet.
//
// Weights whose rows TMA cannot read (no multiples of 16 bytes) come through the
// epilogue's warps, idle until the sums are complete (raw_weights).
#include <algorithm>

#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

struct TokensArgs {
    int M, N, K;            // outputs M x N; K: reduction columns of one segment
    int k_tiles, k_seg;     // K steps over all segments, and of one
    const uint16_t *bias, *residual;  // linear
    float *preact;          // gated: both products
    const uint16_t *dy;     // gradients: M x N
    const float *scale;     // one device value times the sums, or nullptr
    const uint16_t *w[2];   // RAW: the weights and their row length
    long long w_ld;
    uint16_t *out, *out2;   // out2: dU of a gated gradient
    long long ldo;          // row length of out and out2
    int act;
};

struct TokensMaps {
    CUtensorMap x[2], w[2];
};

enum class Tok {
    LINEAR,       // act(X W + b) + R
    GATED,        // act(X Wg) * (X Wu)
    LINEAR_GRAD,  // dY act'(X W + b)
    GATED_GRAD,   // dH U act'(G), dH act(G)
    TRANSPOSED,   // sum over segments of X W^T
};

// TOK: tokens of the MMA's N side.  DUAL: two weight matrices (gated), whose
// accumulators lie side by side in tensor memory.  RAW: weights whose rows are not
// multiples of 16 bytes, which TMA cannot read (raw_weights).  ROUND: K steps of an
// accumulation round (0: a CTA's whole share), whose sums the epilogue warps add in
// fp32 registers while the next round fills a second accumulator; for a Z that decides
// a ReLU (op_sign_rounds).  Hidden behind the weights' loads: 64 x 20000 x 8192 with Z
// kept 60.3 us, 59.8 as one chain.
template <int TOK_, Tok MODE_, bool RAW_ = false, int ROUND_ = 0>
struct TokCfg {
    static constexpr bool RAW = RAW_;
    static constexpr int ROUND = ROUND_;
    static constexpr int TOK = TOK_, BN = 128, BK = 64;
    static constexpr Tok MODE = MODE_;
    static constexpr bool DUAL = MODE == Tok::GATED || MODE == Tok::GATED_GRAD;
    static constexpr bool GRAD = MODE == Tok::LINEAR_GRAD || MODE == Tok::GATED_GRAD;
    static constexpr bool W_K = MODE == Tok::TRANSPOSED;  // W's rows run along the reduction
    static constexpr int NW = DUAL ? 2 : 1;
    static constexpr int W_SUB = BN * BK * 2;  // one matrix, 64 k-rows
    static constexpr int X_SUB = TOK * BK * 2;
    static constexpr int STAGE_BYTES = NW * W_SUB + X_SUB;
    static constexpr int SUM_BYTES = NW * TOK * BN * 4;  // partial sums, over the drained ring
    // RAW: weight rows of a K step, the aligned 16-byte chunks that cover a row, and
    // the steps on the way
    static constexpr int RAW_ALL = W_K ? BN : NW * BK;
    static constexpr int RAW_CHUNKS = (W_K ? BK : BN) / 8 + 1;
    static constexpr int RAW_STEPS = DUAL && TOK == 128 ? 2 : 3;  // (what fits)
    static constexpr int RAW_BYTES = RAW ? RAW_STEPS * RAW_ALL * RAW_CHUNKS * 16 : 0;
    // two CTAs an SM, unless the partial sums alone (RAW: with two stages' worth of
    // ring beside the fetched rows) are more than half of it
    static constexpr int HALF_SM = kSmemPerSm / 2 - kSmemReservedPerBlock - 2048;
    static constexpr int LEAST = RAW && SUM_BYTES < 2 * STAGE_BYTES ? 2 * STAGE_BYTES : SUM_BYTES;
    static constexpr int CTAS = LEAST + RAW_BYTES <= HALF_SM ? 2 : 1;
    static constexpr int STAGES =
        ((CTAS == 2 ? HALF_SM : 232448 - 2048) - RAW_BYTES) / STAGE_BYTES;
    static constexpr int RING = STAGES * STAGE_BYTES;
    static constexpr int RAW_OFFSET = RING;
    static constexpr int BAR_OFFSET = RING + RAW_BYTES;
    static constexpr int USED = BAR_OFFSET + (2 * STAGES + (ROUND > 0 ? 5 : 1)) * 8 + 16;
    static constexpr int SMEM_BYTES = smem_request(USED + 1024, CTAS);
    static constexpr int ACC = NW * TOK;
    static constexpr int ACCS = ACC * (ROUND > 0 ? 2 : 1);  // of two CTAs: 512 columns at most
    static constexpr int TMEM_COLS = ACCS <= 32    ? 32
                                     : ACCS <= 64  ? 64
                                     : ACCS <= 128 ? 128
                                     : ACCS <= 256 ? 256
                                                   : 512;
    // epilogue warps: two for each TMEM lane quadrant, or four where one CTA an SM has
    // to shift all weights, or to hold 256 columns of sums
    static constexpr int EPI = (RAW || ROUND > 0) && CTAS == 1 ? 16 : 8;
    static constexpr int CHUNKS = (ACC + 4 * EPI - 1) / (4 * EPI);  // 16 columns, a warp's
    static constexpr int RAW_ROWS = RAW_ALL / EPI;  // a warp's
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int PREFETCH = 4;  // K steps asked for ahead of the kernel before
    static_assert(STAGES >= 2 && SUM_BYTES <= RING && SMEM_BYTES <= 232448, "shared memory");
    static_assert(TOK % 16 == 0 && TOK <= 128, "TOK");
    static_assert(TMEM_COLS * CTAS <= 512, "accumulators");
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Ask L2 for a box of a tensor.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// Four bf16 values (8-byte aligned with vec), of which `cols` exist.
__device__ __forceinline__ void get4(const uint16_t *p, int cols, bool vec, float (&f)[4]) {
    if (vec) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        f[0] = bf16_lo(x.x);
        f[1] = bf16_hi(x.x);
        f[2] = bf16_lo(x.y);
        f[3] = bf16_hi(x.y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = j < cols ? __uint_as_float(static_cast<uint32_t>(p[j]) << 16) : 0.0f;
    }
}

__device__ __forceinline__ void put4(uint16_t *p, int cols, bool vec, const float (&f)[4]) {
    const uint32_t lo = pack_bf16(f[0], f[1]), hi = pack_bf16(f[2], f[3]);
    // (vec: rows padded to four columns at least)
    if (vec) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
        const uint32_t w[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < cols) p[j] = static_cast<uint16_t>(w[j]);
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// RAW: each epilogue warp w brings its rows of every K step into the ring.  Rows start on
// any even byte: the aligned 16-byte chunks that cover a row's part of the tile come
// by cp.async, RAW_STEPS ahead, into the warp's own buffers (zero beyond the row, so
// that nothing outside the matrix is read and the reduction's tail is zero), and are
// shifted from there into the layout that TMA would have written.  A K step moves every
// address by a multiple of 16 bytes (64 rows, or 64 columns), so a lane's chunks keep
// their alignment and their place, and are worked out once.
// after(i) is called when step i of the share has been handed over.
template <class Cfg, class After>
__device__ __forceinline__ void raw_weights(const TokensArgs &a, const KernelCtx &ctx,
                                            uint8_t *smem, uint64_t *full, uint64_t *empty,
                                            int n0, int kb, int ke, int w, int lane,
                                            After &&after) {
    constexpr int ROWS = Cfg::RAW_ROWS, CH = Cfg::RAW_CHUNKS, STEPS = Cfg::RAW_STEPS;
    constexpr int BK = Cfg::BK, STEP_BYTES = ROWS * CH * 16;
    constexpr int NF = (ROWS * CH + 31) / 32;   // chunks a lane fetches of a step
    constexpr int RPI = 32 / (CH - 1);          // rows that the warp shifts at a time
    const uint32_t raw = smem_u32(smem + Cfg::RAW_OFFSET) + w * (STEPS * STEP_BYTES);
    const long long move = Cfg::W_K ? BK * 2 : BK * 2 * a.w_ld;  // bytes from step to step

    // chunk lane + 32 i: where it starts, and the bytes from there to the row's end
    const uint8_t *src[NF];
    int left[NF];
    auto start = [&](int kt) {
        const int sg = kt >= a.k_seg ? 1 : 0, k0 = (kt - sg * a.k_seg) * BK;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            const int c = lane + 32 * i, row = c / CH, r = w * ROWS + row;
            const bool second = Cfg::W_K ? sg == 1 : r >= BK;
            const uint16_t *m = second ? a.w[1] : a.w[0];
            const long long g = Cfg::W_K ? n0 + r : k0 + r % BK;
            const long long col = Cfg::W_K ? k0 : n0;
            const long long at = ((g * a.w_ld + col) & ~7ll) + 8 * (c - row * CH);
            const long long l = (g * a.w_ld + (Cfg::W_K ? a.K : a.N) - at) * 2;
            const bool in = l > 0 && c < ROWS * CH && (!Cfg::W_K || g < a.N);
            src[i] = reinterpret_cast<const uint8_t *>(in ? m + at : m);
            left[i] = !in ? 0 : l < 0x40000000 ? static_cast<int>(l) : 0x40000000;
        }
    };
    auto fetch = [&](int kt) {
        if (kt < ke) {
            if (kt == kb || (Cfg::W_K && kt == a.k_seg)) start(kt);
            const uint32_t to = raw + (kt - kb) % STEPS * STEP_BYTES + lane * 16;
            const bool tail = !Cfg::W_K && (kt + 1) * static_cast<long long>(BK) > a.K;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int c = lane + 32 * i;
                int bytes = max(0, min(16, left[i]));
                if (tail && kt * BK + (w * ROWS + c / CH) % BK >= a.K) bytes = 0;
                const uint8_t *from =
                    bytes > 0 ? src[i] : reinterpret_cast<const uint8_t *>(a.w[0]);
                if (c < ROWS * CH) cp_async16(to + 512 * i, from, bytes);
                src[i] += move;
                if (Cfg::W_K) left[i] -= BK * 2;
            }
        }
        cp_async_commit();
    };
    // the 16 bytes that lane shifts of every RPI rows: row, chunk, place in the ring
    const int row = lane / (CH - 1), j = lane % (CH - 1), r = w * ROWS + row;
    const uint32_t at0 =
        static_cast<uint32_t>((Cfg::W_K ? n0 + r : r % BK) * a.w_ld) & 7u;  // (n0, k0: 0 mod 8)
    const uint32_t shift = static_cast<uint32_t>(RPI * a.w_ld) & 7u;
    // 128-byte rows, chunk j of row r at j ^ (r % 8)
    const uint32_t ring = Cfg::W_K ? r * 128 + ((j ^ (r & 7)) << 4)
                                   : r / BK * Cfg::W_SUB + (j >> 3) * (BK * 128) +
                                         r % BK * 128 + (((j ^ r) & 7) << 4);
#pragma unroll
    for (int i = 0; i < STEPS - 1; ++i) fetch(kb + i);
    int s = 0;
    uint32_t ph = 0, step = 0;
    for (int kt = kb; kt < ke; ++kt) {
        fetch(kt + STEPS - 1);
        if (!mbar_wait(&empty[s], ph ^ 1u, ctx, kSiteProducerEmpty)) break;
        cp_async_wait<STEPS - 1>();
        __syncwarp();
        const uint32_t from = raw + step * STEP_BYTES + (row * CH + j) * 16;
        const uint32_t to = smem_u32(smem) + s * Cfg::STAGE_BYTES + ring;
#pragma unroll
        for (int i = 0; i < ROWS / RPI; ++i) {
            const uint4 lo = lds_u4(from + i * RPI * CH * 16);
            const uint4 hi = lds_u4(from + i * RPI * CH * 16 + 16);
            uint32_t o[4];
            shift16(lo, hi, ((at0 + i * shift) & 7u) * 2u, o);
            sts128((to ^ ((RPI * i & 7) << 4)) + RPI * i * 128, o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == Cfg::STAGES) {
            s = 0;
            ph ^= 1u;
        }
        if (++step == STEPS) step = 0;
        after(kt - kb);
    }
    cp_async_wait<0>();
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    tokens_kernel(const __grid_constant__ TokensMaps maps, const TokensArgs a,
                  const KernelCtx ctx) {
    constexpr int TOK = Cfg::TOK, STAGES = Cfg::STAGES, BK = Cfg::BK, BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFFSET);
    uint64_t *empty = full + STAGES;
    uint64_t *done = empty + STAGES;
    uint64_t *acc_full = done + 1, *acc_empty = acc_full + 2;  // [2] each, with ROUND
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + (Cfg::ROUND > 0 ? 5 : 1));
    const uint32_t warp = warp_id_uniform(), lane = lane_id();
    uint32_t S;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    const int n0 = static_cast<int>(blockIdx.x / S) * BN;
    const int m0 = static_cast<int>(blockIdx.y) * TOK, rows = min(TOK, a.M - m0);
    const int kb = static_cast<int>(static_cast<long long>(rank) * a.k_tiles / S);
    const int ke = static_cast<int>(static_cast<long long>(rank + 1) * a.k_tiles / S);

    if (warp == 0 && lane == 0) {
        if (a.k_tiles > 0) {
            prefetch_tmap(&maps.x[0]);
            if (!Cfg::RAW) prefetch_tmap(&maps.w[0]);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], Cfg::RAW ? 1 + Cfg::EPI : 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        for (int b = 0; Cfg::ROUND > 0 && b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI);
        }
        fence_barrier_init();
    }
    if (!Cfg::RAW && warp == 2 && lane == 0) {
        for (int kt = kb; kt < min(ke, kb + Cfg::PREFETCH); ++kt)
        {
            const int sg = kt >= a.k_seg ? 1 : 0, k0 = (kt - sg * a.k_seg) * BK;
            if constexpr (Cfg::W_K) {
                tma_prefetch_2d(&maps.w[sg], k0, n0);
            } else {
#pragma unroll
                for (int d = 0; d < Cfg::NW; ++d)
#pragma unroll
                    for (int j = 0; j < BN / 64; ++j)
                        if (n0 + 64 * j < a.N) tma_prefetch_2d(&maps.w[d], n0 + 64 * j, k0);
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    // ROUND: the sums of a warp's columns, 16 from every 4 * EPI, and the rounds in them
    float acc[Cfg::ROUND > 0 ? Cfg::CHUNKS : 1][16];
    const int c0 = static_cast<int>((warp - 2) >> 2) * 16;
    const uint32_t t_row = tmem + (((warp & 3u) * 32u) << 16);
    const int rounds = Cfg::ROUND > 0 ? (ke - kb + Cfg::ROUND - 1) / Cfg::ROUND : 0;
    int taken = 0;
    auto take_round = [&] {
        const int r = taken++;
        if (!mbar_wait(&acc_full[r & 1], (r >> 1) & 1, ctx, kSiteEpilogueFull)) {
            taken = rounds;  // (the call has failed)
            return;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < Cfg::CHUNKS; ++i) {
            const int c = c0 + i * 4 * Cfg::EPI;
            if (c >= Cfg::ACC || c % TOK >= rows) continue;  // no tokens there
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_row + (r & 1) * Cfg::ACC + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][j] += __uint_as_float(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[r & 1]);
    };
    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int kt = kb; kt < ke; ++kt, ++it) {
                const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                if (!mbar_wait(&empty[s], ph ^ 1u, ctx, kSiteProducerEmpty)) break;
                uint8_t *st = smem + s * Cfg::STAGE_BYTES;
                mbar_arrive_expect_tx(&full[s], Cfg::RAW ? Cfg::X_SUB : Cfg::STAGE_BYTES);
                const int sg = kt >= a.k_seg ? 1 : 0, k0 = (kt - sg * a.k_seg) * BK;
                if constexpr (Cfg::RAW) {
                    // the epilogue's warps bring the weights
                } else if constexpr (Cfg::W_K) {
                    tma_load_2d(st, &maps.w[sg], &full[s], k0, n0);
                } else {
#pragma unroll
                    for (int d = 0; d < Cfg::NW; ++d)
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j)
                            tma_load_2d(st + d * Cfg::W_SUB + j * (BK * 128), &maps.w[d], &full[s],
                                        n0 + 64 * j, k0);
                }
                tma_load_2d(st + Cfg::NW * Cfg::W_SUB, &maps.x[sg], &full[s], k0, m0);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(BN, TOK, 1, /*A*/ Cfg::W_K ? 0 : 1, /*B K-major*/ 0);
            int it = 0;
            bool ok = true;
            uint32_t d_tmem = tmem;
            for (int kt = kb; kt < ke; ++kt, ++it) {
                bool first = kt == kb;
                if constexpr (Cfg::ROUND > 0) {
                    first = it % Cfg::ROUND == 0;
                    if (first) {
                        const uint32_t r = it / Cfg::ROUND;
                        if (r > 0) umma_commit(&acc_full[(r - 1) & 1u]);
                        if (!mbar_wait(&acc_empty[r & 1u], ((r >> 1) & 1u) ^ 1u, ctx,
                                       kSiteMmaAccEmpty)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        d_tmem = tmem + (r & 1u) * Cfg::ACC;
                    }
                }
                const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                if (!mbar_wait(&full[s], ph, ctx, kSiteMmaFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * Cfg::STAGE_BYTES);
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                    const uint64_t bd =
                        smem_desc_sw128(st + Cfg::NW * Cfg::W_SUB + k * 32, 16, 1024);
#pragma unroll
                    for (int d = 0; d < Cfg::NW; ++d) {
                        const uint64_t ad =
                            Cfg::W_K ? smem_desc_sw128(st + k * 32, 16, 1024)
                                     : smem_desc_sw128(st + d * Cfg::W_SUB + k * 2048, BK * 128,
                                                       1024);
                        umma_f16_ss(d_tmem + d * TOK, ad, bd, idesc, (first && k == 0) ? 0u : 1u);
                    }
                }
                umma_commit(&empty[s]);
            }
            if (Cfg::ROUND > 0 && ok && ke > kb)
                umma_commit(&acc_full[((ke - kb - 1) / Cfg::ROUND) & 1]);
            umma_commit(done);
        }
    } else {
        if constexpr (Cfg::ROUND > 0) {
#pragma unroll
            for (int i = 0; i < Cfg::CHUNKS; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[i][j] = 0.0f;
        }
        if constexpr (Cfg::RAW)
            raw_weights<Cfg>(a, ctx, smem, full, empty, n0, kb, ke, static_cast<int>(warp) - 2,
                             static_cast<int>(lane), [&](int i) {
                                 // half a round on, the last one's products have ended
                                 if constexpr (Cfg::ROUND > 0)
                                     if (i >= Cfg::ROUND && i % Cfg::ROUND == Cfg::ROUND / 2 &&
                                         taken < rounds)
                                         take_round();
                             });
        if constexpr (Cfg::ROUND > 0)
            while (taken < rounds) take_round();
    }
    // Every MMA of this CTA has completed: the ring is free, the sums final.
    // (With an empty K range the commit arrives at once.)
    const bool ok = mbar_wait(done, 0, ctx, kSiteEpilogueFull);
    tc_fence_after();
    __syncwarp();
    float *sums = reinterpret_cast<float *>(smem);  // [NW][TOK][128]
    if (warp >= 2) {
        const uint32_t q = warp & 3u;
        const int col = static_cast<int>(q * 32 + lane);
        // a quadrant's warps take 16 accumulator columns in turn
        if constexpr (Cfg::ROUND > 0) {
#pragma unroll
            for (int i = 0; i < Cfg::CHUNKS; ++i) {
                const int c = c0 + i * 4 * Cfg::EPI;
                if (c >= Cfg::ACC || c % TOK >= rows) continue;
#pragma unroll
                for (int j = 0; j < 16; ++j) sums[(c + j) * BN + col] = acc[i][j];
            }
        } else {
#pragma unroll 1
            for (int c = c0; c < Cfg::ACC; c += 4 * Cfg::EPI) {
                if (c % TOK >= rows) continue;  // no tokens there
                uint32_t v[16];
                if (ke > kb && ok) {
                    tmem_ld_32x32b_x16(t_row + c, v);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) sums[(c + j) * BN + col] = __uint_as_float(v[j]);
            }
        }
    }
    __syncwarp();
    if (S > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp >= 2 && ok) {
        // tokens rank, rank + S, ... are this CTA's; its warps take them in turn
        const int n = n0 + static_cast<int>(lane) * 4;
        const int cols = a.N - n;
        const bool vec = a.N % 4 == 0;  // the caller's rows on 8-byte boundaries
        const bool vec_out = a.ldo % 4 == 0;
        if (cols > 0) {
            float b[4] = {0.f, 0.f, 0.f, 0.f};
            if (a.bias) get4(a.bias + n, cols, vec, b);
            for (int t = static_cast<int>(rank + S * (warp - 2)); t < rows;
                 t += static_cast<int>(S) * Cfg::EPI) {
                const long long at = static_cast<long long>(m0 + t) * a.N + n;
                float r[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.residual) get4(a.residual + at, cols, vec, r);
                if (Cfg::GRAD) get4(a.dy + at, cols, vec, r);
                float4 part[Cfg::NW][8];
#pragma unroll
                for (int d = 0; d < Cfg::NW; ++d) {
                    const float *p = sums + (d * TOK + t) * BN + lane * 4;
                    const uint32_t local = smem_u32(p);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < static_cast<int>(S))
                            part[d][i] = S == 1 ? *reinterpret_cast<const float4 *>(p)
                                                : ld_cluster_f32x4(mapa_shared(local, i));
                }
                float z[Cfg::NW][4];
#pragma unroll
                for (int d = 0; d < Cfg::NW; ++d) {
                    z[d][0] = part[d][0].x;
                    z[d][1] = part[d][0].y;
                    z[d][2] = part[d][0].z;
                    z[d][3] = part[d][0].w;
#pragma unroll
                    for (int i = 1; i < 8; ++i)
                        if (i < static_cast<int>(S)) {
                            z[d][0] += part[d][i].x;
                            z[d][1] += part[d][i].y;
                            z[d][2] += part[d][i].z;
                            z[d][3] += part[d][i].w;
                        }
                }
                if (a.scale) {
                    const float f = *a.scale;
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[0][j] *= f;
                }
                if constexpr (!Cfg::DUAL) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[0][j] += b[j];
                }
                if (a.preact) {
#pragma unroll
                    for (int d = 0; d < Cfg::NW; ++d)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < cols)
                                a.preact[d * static_cast<long long>(a.M) * a.N + at + j] = z[d][j];
                }
                float y[4], y2[4] = {0.f, 0.f, 0.f, 0.f};
                with_act(a.act, [&](auto A) {
                    constexpr int ACT = decltype(A)::value;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (Cfg::GRAD) {
                            float value;
                            const float d = act_value_grad<ACT>(z[0][j], value);
                            y[j] = r[j] * d * (Cfg::DUAL ? z[Cfg::NW - 1][j] : 1.0f);
                            y2[j] = r[j] * value;
                        } else {
                            y[j] = act_value<ACT>(z[0][j]);
                            y[j] = Cfg::DUAL ? y[j] * z[Cfg::NW - 1][j] : y[j] + r[j];
                        }
                    }
                });
                const long long to = static_cast<long long>(m0 + t) * a.ldo + n;
                put4(a.out + to, cols, vec_out, y);
                if constexpr (Cfg::MODE == Tok::GATED_GRAD) put4(a.out2 + to, cols, vec_out, y2);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (S > 1)
        cluster_sync();  // the peers have read this CTA's sums
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// CTAs that share a tile along K: the S of 1, 2, 4, 8 whose waves (`slots` clusters
// at once, each CTA 1 / S of a tile's K steps) end soonest, with at least four
// steps a CTA, and half a step's worth for each doubling of the join.  A wave costs
// `wave` steps beside its own: its CTAs' set-up, first loads and join.  (Over 84 shapes
// from 1000 x 512 to 65536 x 2048 and up to 128 tokens that S is 0.9 % slower than the
// best of the four, 27 % at worst; without the term 11 %, and 1.9 times.  Rows that
// TMA cannot read take longer a step: 16 would cost 2.7 % there, 12 costs 0.8 %.)
constexpr int kWaveSteps = 16, kRawWaveSteps = 12;

// Clusters of 1, 2, 4 and 8 CTAs that run at once, `ctas` CTAs an SM.  A cluster stays
// within one of the GPU's own clusters of 16 to 20 SMs: of eight CTAs with an SM each
// only 15 fit on 152 SMs (gated 1 x 2033 x 2256, 16 tiles, as one wave of such: 20.5 us,
// as 4 CTAs a tile 14.4).  The other sizes lose one or two, which is not counted: a
// cluster left over by that costs less than a wave (37 tiles by eight, two CTAs an SM, 1 x
// 4619 x 7120: 29.4 us, by four 31.0).
struct ClusterSlots {
    int n[4];
};
static ClusterSlots cluster_slots(int sm_count, int ctas) {
    const int all = sm_count * ctas;
    return ClusterSlots{{all, all / 2, all / 4, ctas == 1 ? sm_count / 10 : all / 8}};
}

static int cluster_share(const ClusterSlots &slots, int n_tiles, int k_tiles, int wave) {
    int best = 1;
    double best_cost = 1e30, join = 0.0;
    for (int S = 1, i = 0; S <= 8; S *= 2, ++i, join += 0.5) {
        const int per_wave = slots.n[i];
        if ((S > 1 && k_tiles / S < 4) || per_wave < 1) break;
        const double waves = (n_tiles + per_wave - 1) / per_wave;
        const double cost = waves * ((k_tiles + S - 1) / S + wave) + join;
        if (cost < best_cost) {
            best_cost = cost;
            best = S;
        }
    }
    return best;
}

// More than 128 rows: tiles of 128 x 128 whose K a cluster shares, which saves the tiled
// product's parts and the kernel that joins them, while one wave holds them all.  Times
// fitted to 112 shapes of 136 to 1024 rows (us, one CTA an SM and two); a call from a
// graph by this and by tiles: 136 x 520 x 2736 7.6 / 10.4, 512 x 2048 x 2736 12.6 / 16.2,
// 300 x 520 x 1024 7.0 / 9.5; gated, whose tiles have no parts, 136 x 520 x 8192 15.5 /
// 34.2, 512 x 520 x 2736 13.1 / 15.0.
static bool tokens_beat(const OpDevice &dev, int M, long long N, long long K, int ctas, double us0,
                        double step0, double us1, double step1, double tiled_us) {
    const long long tiles = static_cast<long long>(op_blocks(M, 128)) * op_blocks(N, 128);
    if (tiles > ctas * dev.sm_count) return false;
    const int k_tiles = op_blocks(K, 64);
    const ClusterSlots slots = cluster_slots(dev.sm_count, ctas);
    const int S = cluster_share(slots, static_cast<int>(tiles), k_tiles, kWaveSteps);
    if (tiles > slots.n[S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3]) return false;
    const int steps = (k_tiles + S - 1) / S;
    const double us = tiles * S <= dev.sm_count ? us0 + step0 * steps : us1 + step1 * steps;
    return us < 0.93 * tiled_us;
}

bool op_tokens_fit(const OpDevice &dev, int M, long long N, long long K) {
    if (M > kTokensMax)
        return tokens_beat(dev, M, N, K, 2, 5.7, 0.32, 8.5, 0.47, op_product_us(dev, M, N, K));
    const int n_tiles = op_blocks(N, 128);
    const int k_tiles = op_blocks(K, 64);
    const int S = cluster_share(cluster_slots(dev.sm_count, 2), n_tiles, k_tiles, kWaveSteps);
    return n_tiles * S >= dev.sm_count || k_tiles / S <= 32;
}

bool op_tokens_gated_fit(const OpDevice &dev, int M, int F, int K) {
    if (M <= kTokensMax) return true;
    return tokens_beat(dev, M, F, K, 1, 8.8, 0.48, 8.8, 0.48, op_gated_us(dev, M, F, K));
}

// Measured, a call from a graph with the weights read in place / copied first / at a
// pitch of whole vectors: 1 x 16383 x 2048 20.6 / 33.0 / 13.1 us, 1 x 1001 x 1000 6.4 /
// 7.6 / 4.3, gated 1 x 8191 x 4096 38 / 64 / 22, 1 x 1001 x 1000 8.8 / 9.9 / 5.3; dX of
// 1 x 8191 x 4096 22.8 / 31.1 / 13.3, of 1 x 1537 x 512 8.7 / 7.9 / 4.6.  A step takes
// some 0.5 us more (gated 0.8, W^T 0.35), which few CTAs with many steps feel most.
double op_raw_us(const OpDevice &dev, int M, long long N, long long K, bool dual,
                 bool transposed) {
    const ClusterSlots slots = cluster_slots(dev.sm_count, M <= 64 && !dual ? 2 : 1);
    const int n_tiles = op_blocks(N, 128), k_tiles = op_blocks(K, 64);
    const int S = cluster_share(slots, n_tiles, k_tiles, kRawWaveSteps);
    const int per_wave = slots.n[S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3];
    const double waves = (n_tiles + per_wave - 1) / per_wave;
    return waves * ((k_tiles + S - 1) / S) * (transposed ? 0.35 : dual ? 0.8 : 0.5);
}

constexpr int kSignSteps = kSignRound / 64;  // K steps of a round

// sign: the call's Z decides a ReLU's derivative, here or in the backward pass.
template <class Cfg>
static pgemm_status launch_tokens(const OpDevice &dev, TokensArgs a, const OpMat *X,
                                  const OpMat *W, int segments, bool sign, cudaStream_t s) {
    a.k_seg = op_blocks(a.K, Cfg::BK);
    a.k_tiles = a.k_seg * segments;
    const int n_tiles = op_blocks(a.N, Cfg::BN);
    const int m_tiles = op_blocks(a.M, Cfg::TOK);
    const int S = cluster_share(cluster_slots(dev.sm_count, Cfg::CTAS), n_tiles * m_tiles, a.k_tiles,
                                Cfg::RAW ? kRawWaveSteps : kWaveSteps);
    if constexpr (!Cfg::W_K && Cfg::ROUND == 0) {
        if (sign && op_blocks(a.k_tiles, S) > kSignSteps)
            return launch_tokens<TokCfg<Cfg::TOK, Cfg::MODE, Cfg::RAW, kSignSteps>>(
                dev, a, X, W, segments, sign, s);
    }
    static const KernelInfo info = [] {
        KernelInfo k;
        k.threads = Cfg::THREADS;
        k.smem_bytes = Cfg::SMEM_BYTES;
        k.func = reinterpret_cast<const void *>(tokens_kernel<Cfg>);
        return k;
    }();
    int slots = 0;
    pgemm_status st = op_kernel_setup(dev, info, &slots);
    TokensMaps maps{};
    if (a.K > 0) {
        for (int d = 0; d < segments && st == PGEMM_OK; ++d)
            st = op_encode(&maps.x[d], X[d].p, a.K, a.M, X[d].ld, Cfg::TOK);
        const int matrices = Cfg::DUAL ? 2 : segments;
        for (int d = 0; d < matrices && st == PGEMM_OK && !Cfg::RAW; ++d)
            st = Cfg::W_K ? op_encode(&maps.w[d], W[d].p, a.K, a.N, W[d].ld, 128)
                          : op_encode(&maps.w[d], W[d].p, a.N, a.K, W[d].ld, 64);
    }
    if (st != PGEMM_OK) return st;
    a.w[0] = W[0].p;
    a.w[1] = W[Cfg::DUAL || segments == 2 ? 1 : 0].p;
    a.w_ld = W[0].ld;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(S);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(n_tiles) * S, static_cast<unsigned>(m_tiles));
    lc.blockDim = dim3(Cfg::THREADS);
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = s;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, tokens_kernel<Cfg>, maps, a, dev.ctx) == cudaSuccess
               ? PGEMM_OK
               : PGEMM_ERR_CUDA;
}

template <Tok MODE, bool RAW>
static pgemm_status launch_tokens_rows(const OpDevice &dev, const TokensArgs &a, const OpMat *X,
                                       const OpMat *W, int segments, bool sign, cudaStream_t s) {
    if (a.M <= 16) return launch_tokens<TokCfg<16, MODE, RAW>>(dev, a, X, W, segments, sign, s);
    if (a.M <= 32) return launch_tokens<TokCfg<32, MODE, RAW>>(dev, a, X, W, segments, sign, s);
    if (a.M <= 64) return launch_tokens<TokCfg<64, MODE, RAW>>(dev, a, X, W, segments, sign, s);
    return launch_tokens<TokCfg<128, MODE, RAW>>(dev, a, X, W, segments, sign, s);
}

template <Tok MODE>
static pgemm_status launch_tokens_size(const OpDevice &dev, const TokensArgs &a, const OpMat *X,
                                       const OpMat *W, int segments, bool sign, cudaStream_t s) {
    return W[0].ld % 8 == 0 ? launch_tokens_rows<MODE, false>(dev, a, X, W, segments, sign, s)
                            : launch_tokens_rows<MODE, true>(dev, a, X, W, segments, sign, s);
}

pgemm_status op_tokens_linear(const OpDevice &dev, int M, int N, int K, const OpMat &X,
                              const OpMat &W, const OpEpilogue &e, uint16_t *Y, cudaStream_t s) {
    TokensArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.bias = e.bias;
    a.residual = e.residual;
    a.preact = e.preact;
    a.scale = e.scale;
    a.act = e.act;
    a.out = Y;
    a.ldo = N;
    return launch_tokens_size<Tok::LINEAR>(dev, a, &X, &W, 1,
                                           e.preact && e.act == PGEMM_ACT_RELU, s);
}

pgemm_status op_tokens_gated(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                             const OpMat &Wg, const OpMat &Wu, int act, uint16_t *H,
                             float *preact, cudaStream_t s) {
    TokensArgs a{};
    a.M = M;
    a.N = F;
    a.K = K;
    a.preact = preact;
    a.act = act;
    a.out = H;
    a.ldo = F;
    const OpMat w[2] = {Wg, Wu};
    return launch_tokens_size<Tok::GATED>(dev, a, &X, w, 1, preact && act == PGEMM_ACT_RELU, s);
}

pgemm_status op_tokens_linear_grad(const OpDevice &dev, int M, int N, int K, const OpMat &X,
                                   const OpMat &W, const uint16_t *bias, int act,
                                   const uint16_t *dy, uint16_t *dz, long long dz_ld,
                                   cudaStream_t s) {
    TokensArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.bias = bias;
    a.dy = dy;
    a.act = act;
    a.out = dz;
    a.ldo = dz_ld;
    return launch_tokens_size<Tok::LINEAR_GRAD>(dev, a, &X, &W, 1, act == PGEMM_ACT_RELU, s);
}

pgemm_status op_tokens_gated_grad(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                                  const OpMat &Wg, const OpMat &Wu, int act, const uint16_t *dh,
                                  uint16_t *dg, uint16_t *du, long long dz_ld, cudaStream_t s) {
    TokensArgs a{};
    a.M = M;
    a.N = F;
    a.K = K;
    a.dy = dh;
    a.act = act;
    a.out = dg;
    a.out2 = du;
    a.ldo = dz_ld;
    const OpMat w[2] = {Wg, Wu};
    return launch_tokens_size<Tok::GATED_GRAD>(dev, a, &X, w, 1, act == PGEMM_ACT_RELU, s);
}

pgemm_status op_tokens_transposed(const OpDevice &dev, int M, int N, int K, const OpMat *X,
                                  const OpMat *W, int segments, uint16_t *out, cudaStream_t s) {
    TokensArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = PGEMM_ACT_NONE;
    a.out = out;
    a.ldo = N;
    return launch_tokens_size<Tok::TRANSPOSED>(dev, a, X, W, segments, false, s);
}

}  // namespace pg
