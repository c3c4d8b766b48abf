// xent_bf16: softmax cross entropy of logits L = X W^T over a vocabulary
// (W: one row of D for each of V tokens), and its gradients, without keeping L.
//
//   lse_t  = log sum_v exp L_tv          loss_t = lse_t - L_t,y(t)
//   P_tv   = (exp(L_tv - lse_t) - [v = y(t)]) dloss_t / c,  c = max_t |dloss_t|
//   dX     = c P W                       dW = c P^T X
//
// P is rounded to bf16 as an operand of the last two products; c is what keeps
// that rounding from adding up.  A row's entry at its target is nearly -dloss_t
// and outweighs the rest of the row; with dloss the same for all rows (a mean)
// every one of them would round by the same up to 2^-8 of itself, and the whole
// gradient with them.  Divided by c those entries start from exactly -1; c
// itself multiplies the sums in fp32.
//
// Forward: the product's epilogue folds every accumulator into a maximum m and
// sum s of exp(L - m) for each row and column block (a thread holds a whole row
// segment, so neither needs a shuffle).  A second kernel joins the blocks of a
// row, lse = M + log sum_b s_b exp(m_b - M), and multiplies out the row's own
// target logit.
// Gradient: where all of P fits the workspace the forward epilogue also keeps the
// exponentials, which one elementwise pass turns into P; else the vocabulary goes by
// in pieces, whose logits the same product computes a second time and whose epilogue
// writes P.
//
// Tensor-bound beyond some 300 tokens: 4096 x 131072 x 4096 with gradients takes
// 8.2 ms for three products of 4.4e12 operations each (1.61 PFLOP/s overall, 95 %
// of what plain products sustain under the power cap; 0.3 ms of it turns the
// exponentials into P at 7 TB/s).  Few tokens: bound by reading W (290 MB at
// 5.8 TB/s for 24 tokens) and writing dW (4.0 TB/s, a memset's rate).
//
// A row whose target lies outside [0, V) does not count: loss 0, gradient 0.
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>

#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Statistics take ex2_ftz: results below 2^-126 of the block's largest count as zero.
// Probabilities themselves take exp2f, which keeps subnormal results.

// Softmax statistics are kept to base 2: m is the largest L log2(e) of a row's
// column block (or 15 less, see KEEP), s the block's sum of 2^(L log2(e) - m).
//
// Accumulation rounds of 1024 products are added in fp32 registers.  The
// tensor core truncates its running sum at every step of 16 products, always
// toward zero: over the 256 steps of D = 4096 that shrinks every logit by some
// 1e-5 of its size, which the statistics of a whole vocabulary do not average
// out (lse off by 2e-6 of itself); four rounds of 64 steps and three rounded
// additions leave a quarter of it.
//
// KEEP: the exponentials themselves are stored as fp16, 2^(L log2(e) - m) with
// the block's own m, 15 below its largest, so that the gradient pass turns them into P without the
// logits' product a second time: 4 bytes of traffic a logit instead of 2 D
// operations (with gradients, kept against computed again: 4096 x 32768 x 128 294
// against 298 us, x 768 504 against 566, 3472 x 5843 x 336 82 against 94).  They lie
// in (0, 2^15], just within fp16, which carries them to 2^-11 of their size, an eighth
// of what rounding P to bf16 costs, down to 2^-29 of the block's largest, and to 2^-40
// of that largest below: an unlikely token beside a likely one keeps its gradient.
constexpr int kStatsRound = 1024;
constexpr float kKeepShift = 15.0f;
template <bool KEEP>
struct EpiXentStats {
    float *part_m, *part_s;  // [column block][rows]
    long long rows;

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        // whole column blocks: of a half-width unit the first four warps take
        // the one it has
        constexpr int COLS = Cfg::EPI_COLS;
        const int col0 = static_cast<int>(e >> 2) * COLS;
        if (Cfg::HALVES && w.half && e >= 4) return acc.skip();
        const int n0 = w.n0 + col0;
        float v[COLS];
        if (!acc_sum<COLS, 0>(acc, col0, v, 0, nullptr)) return false;
        const int left = c.N - n0;  // columns of the vocabulary in this block
        if (left <= 0) return true;
        if (left < COLS) {
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                if (j >= left) v[j] = -CUDART_INF_F;
        }
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < COLS; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // (KEEP: 2^-22 of itself more than its two roundings could take from it, so that the
        // exponentials of logits of millions stay within fp16 too)
        float m = top * kLog2e;
        if (KEEP && top != -CUDART_INF_F)
            m = fmaf(fabsf(top), kLog2e * 2.384185791015625e-7f, m) - kKeepShift;
        // nothing but -inf: any finite reference gives sums of zero
        const float ref = m == -CUDART_INF_F ? 0.0f : m;
        // +inf among them: less itself it is no number, but the sum is infinite, unless
        // one of them was none before
        float inf_sum = CUDART_INF_F;
        if (m == CUDART_INF_F) {
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                if (isnan(v[j])) inf_sum = v[j];
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int cc = 0; cc < COLS; cc += 32) {
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float a = ex2_ftz(fmaf(v[cc + 2 * j], kLog2e, -ref));
                const float b = ex2_ftz(fmaf(v[cc + 2 * j + 1], kLog2e, -ref));
                s[(2 * j) & 3] += a;
                s[(2 * j + 1) & 3] += b;
                if constexpr (KEEP)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p[j]) : "f"(b), "f"(a));
            }
            if constexpr (KEEP) put_rows32(c, &maps.c[0], nullptr, 0, n0 + cc, p);
        }
        if (c.row() < c.M) {
            const long long at = static_cast<long long>(n0 / COLS) * rows + c.row();
            part_m[at] = m;
            part_s[at] = m == CUDART_INF_F ? inf_sum : (s[0] + s[1]) + (s[2] + s[3]);
        }
        return true;
    }
};

// P of one piece of the vocabulary.  Its logits are summed in the same rounds as the
// statistics' (kStatsRound): from one long chain every exp(L - lse) of a row would be
// short by what the truncation takes from L: 7e-4 of itself for logits of 24 at D =
// 8192, products all positive.
struct EpiXentGrad {
    const int64_t *target;
    const float *lse, *dloss, *scale;  // dloss nullptr: 1, and no scale
    long long v0;              // the piece's first token
    long long V;

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        int col0, cols;
        epi_cols<Cfg>(w, e, col0, cols);
        const int n0 = w.n0 + col0;
        const bool have = acc.have();
        const bool in = c.row() < c.M;
        const int64_t y = in ? __ldg(target + c.row()) : -1;
        const bool counts = y >= 0 && y < V;
        const float l = counts ? lse[c.row()] * kLog2e : 0.0f;
        const float g = counts ? (dloss ? dloss[c.row()] / *scale : 1.0f) : 0.0f;
        const int64_t yc = y - v0 - n0;
        auto finish = [&](int cc, const uint32_t *v) {
            float x[32];
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                x[j] = exp2f(fmaf(__uint_as_float(v[j]), kLog2e, -l));
                if (yc == cc + j) x[j] -= 1.0f;
                x[j] = counts ? x[j] * g : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
            put_rows32(c, &maps.c[0], nullptr, 0, n0 + cc, p);
        };
        if constexpr (Cfg::ROUND > 0) {
            float f[Cfg::EPI_COLS];
            if (!acc_sum_unit<Cfg>(acc, col0, cols, f)) return false;
#pragma unroll
            for (int b = 0; b < Cfg::EPI_COLS / 32; ++b) {
                if (32 * b >= cols) break;
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(f[32 * b + j]);
                finish(32 * b, v);
            }
            return true;
        }
        if (!acc.wait()) return false;
        const uint32_t t_row = acc.row() + col0;
#pragma unroll 1
        for (int cc = 0; cc < cols; cc += 32) {
            uint32_t v[32];
            acc_cols32(t_row + cc, have, v);
            if (cc + 32 >= cols) acc.release();
            finish(cc, v);
        }
        return true;
    }
};

// lse and loss of a row from its column blocks' (m, s), and its target's logit
// as an fp32 dot product of its own (the epilogues would have to pick one of
// their registers by a runtime index).  A block takes ROWS rows: 256 / ROWS
// threads a row share its column blocks (8 adjacent rows make a 32-byte sector;
// with few rows there are not enough blocks of 8 to hide the loads' latency,
// and each row gets a block), then a warp a row multiplies X[t] by W[target].
__device__ __forceinline__ void join_ms(float &m, float &s, float m2, float s2) {
    const float n = fmaxf(m, m2);
    const float ref = fabsf(n) == CUDART_INF_F ? 0.0f : n;  // (+inf: an infinite sum)
    s = s * ex2_ftz(m - ref) + s2 * ex2_ftz(m2 - ref);
    m = n;
}

// A thread's part of the dot product of two rows (16-byte aligned): columns from
// k, eight at a time.
__device__ __forceinline__ float row_dot(const uint16_t *x, const uint16_t *e, int D, int k,
                                         int step) {
    float d = 0.0f;
    for (; k < D; k += step) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x + k);
        const uint4 b = *reinterpret_cast<const uint4 *>(e + k);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (k + 2 * i < D) d = fmaf(bf16_lo(aw[i]), bf16_lo(bw[i]), d);
            if (k + 2 * i + 1 < D) d = fmaf(bf16_hi(aw[i]), bf16_hi(bw[i]), d);
        }
    }
    return d;
}

// lse and the target's logit d are sums of their own, each rounded on its way: of a
// nearly certain token their difference may come out some 3e-6 of d below the zero that
// bounds it (a NaN stays one).
__device__ __forceinline__ float loss_of(float lse, float d) {
    const float x = lse - d;
    return x < 0.0f ? 0.0f : x;
}

template <int ROWS>
__global__ void __launch_bounds__(256)
    xent_join_kernel(const float *part_m, const float *part_s, long long rows, int blocks, int T,
                     long long V, int D, const OpMat X, const OpMat W, const int64_t *target,
                     float *loss, float *lse, const float *dloss, float *scale) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float sm[8][ROWS], ss[8][ROWS], dot[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int r = threadIdx.x % ROWS;
    const int t = blockIdx.x * ROWS + r;
    float m = -CUDART_INF_F, s = 0.0f;
    if (t < T) {
        constexpr int STEP = 256 / ROWS, AHEAD = 8;
        for (int b = threadIdx.x / ROWS; b < blocks; b += STEP * AHEAD) {
            float m2[AHEAD], s2[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const bool in = b + i * STEP < blocks;
                m2[i] = in ? part_m[(b + i * STEP) * rows + t] : -CUDART_INF_F;
                s2[i] = in ? part_s[(b + i * STEP) * rows + t] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) join_ms(m, s, m2[i], s2[i]);
        }
    }
#pragma unroll
    for (int o = ROWS; o <= 16; o *= 2) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join_ms(m, s, m2, s2);
    }
    if (lane < ROWS) {
        sm[w][lane] = m;
        ss[w][lane] = s;
    }
    // the target's logit: a warp a row, or all eight warps for the one row
    {
        const int tw = blockIdx.x * ROWS + (ROWS > 1 ? w : 0);
        const int64_t y = tw < T ? target[tw] : -1;
        float d = 0.0f;
        if (loss && y >= 0 && y < V)
            d = row_dot(X.p + tw * X.ld, W.p + y * W.ld, D,
                        (ROWS > 1 ? lane : static_cast<int>(threadIdx.x)) * 8,
                        ROWS > 1 ? 256 : 2048);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (lane == 0) dot[w] = d;
    }
    __syncthreads();
    if (threadIdx.x < ROWS && t < T) {
        m = sm[0][r];
        s = ss[0][r];
        float d = dot[r];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            join_ms(m, s, sm[i][r], ss[i][r]);
            if (ROWS == 1) d += dot[i];
        }
        const float l = kLn2 * (m + log2f(s));
        const int64_t y = target[t];
        if (lse) lse[t] = l;
        if (loss) loss[t] = y >= 0 && y < V ? loss_of(l, d) : 0.0f;
    }
    if (dloss != nullptr && blockIdx.x == 0) {
        // the common scale of P (xent): the largest |dloss| of a row that counts
        __syncthreads();
        float g = 0.0f;
#pragma unroll 8
        for (int i = static_cast<int>(threadIdx.x); i < T; i += 256) {
            const int64_t y = target[i];
            const float v = fabsf(dloss[i]);
            if (y >= 0 && y < V && v < CUDART_INF_F) g = fmaxf(g, v);
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (lane == 0) dot[w] = g;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 1; i < 8; ++i) g = fmaxf(g, dot[i]);
            *scale = g > 0.0f ? g : 1.0f;
        }
    }
}

// P from the kept exponentials, in place (fp16 to bf16):
//   P = (E 2^(m - lse log2(e)) - [v = target]) dloss.
// Memory-bound, 4 bytes an entry.  A block takes 32 rows x 1024 columns: the
// factors of its column blocks first (loads of 32 adjacent rows), then 16-byte
// vectors, a warp 512 adjacent bytes of a row.
template <int COLS>
__global__ void __launch_bounds__(256)
    xent_scale_kernel(uint16_t *P, long long ld, int T, int V, const float *part_m, long long rows,
                      const float *lse, const int64_t *target, const float *dloss,
                      const float *scale) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int NB = 1024 / COLS;
    __shared__ float f[NB][32], g[32];
    __shared__ int yc[32];  // the target's column within the block's 1024, or -1
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int across = (V - 1) / 1024 + 1;
    const int c0 = static_cast<int>(blockIdx.x % across) * 1024;
    const int row0 = static_cast<int>(blockIdx.x / across) * 32;
    const int t = row0 + lane;
    const int64_t y = t < T ? target[t] : -1;
    const bool counts = y >= 0 && y < V;
    const float gt = counts ? (dloss ? dloss[t] / *scale : 1.0f) : 0.0f;
    if (w == 0) {
        g[lane] = gt;
        yc[lane] = counts && y >= c0 && y < c0 + 1024 ? static_cast<int>(y - c0) : -1;
    }
    const float l = counts ? lse[t] * kLog2e : 0.0f;
    for (int b = w; b < NB; b += 8) {
        const int col = c0 + b * COLS;
        const float m =
            counts && col < V ? part_m[static_cast<long long>(col / COLS) * rows + t] : 0.0f;
        // (a block with a logit of +inf: its E are 0, or NaN for that logit)
        f[b][lane] = !counts || col >= V ? 0.0f : m == CUDART_INF_F ? gt : exp2f(m - l) * gt;
    }
    __syncthreads();
    // warp w: rows w, w + 8, ...; four vectors of 8 columns a lane and row
    for (int r = w; r < 32; r += 8) {
        if (row0 + r >= T) break;
        uint16_t *row = P + static_cast<long long>(row0 + r) * ld + c0;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i * 256 + lane * 8 < V)
                x[i] = *reinterpret_cast<const uint4 *>(row + i * 256 + lane * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = i * 256 + lane * 8;
            if (c0 + col >= V) continue;
            const float fr = f[col / COLS][r];
            const int hit = yc[r] - col;
            const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 e = __half22float2(*reinterpret_cast<const __half2 *>(&in[k]));
                float a = e.x * fr, b = e.y * fr;
                if (hit == 2 * k) a -= g[r];
                if (hit == 2 * k + 1) b -= g[r];
                // a row that does not count is zero whatever its logits were
                o[k] = g[r] == 0.0f ? 0u : pack_bf16(a, b);
            }
            *reinterpret_cast<uint4 *>(row + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ------------------------------------------------------------ few tokens ---
// Up to 64 tokens: the pass is bound by reading W once.  The rows of W take the
// tensor core's M side (up to 128 of the vocabulary a tile), the tokens its N side, so
// that a ring stage is 16 KB of W beside 2 to 8 KB of X; with a token a row it
// would be half padding (V = 98392, D = 1472, 24 tokens: 72 us so, 50 here, 5.8 TB/s
// of W).
// A thread holds one vocabulary entry's logits of 16 or 32 tokens and keeps
// running (m, s) for each through all of its CTA's tiles; lanes and warps are
// joined once at the end.  KEEP: the logits themselves are stored (fp32, T x V,
// coalesced along v) for the gradient's P, which for so few tokens costs less
// than anything read of W.
template <int TOK_>
struct FewCfg {
    static constexpr int TOK = TOK_, BK = 64;
    static constexpr int EPI = TOK == 16 ? 4 : 8;  // warps; two share a lane quadrant's tokens
    static constexpr int TT = TOK * 4 / EPI;       // tokens of a warp
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int CTAS = TOK <= 32 ? 2 : 1;
    static constexpr int W_BYTES = 128 * BK * 2, X_BYTES = TOK * BK * 2;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int ROOM =
        (CTAS == 2 ? kSmemPerSm / 2 - kSmemReservedPerBlock : 232448) - 3072;
    static constexpr int STAGES = ROOM / STAGE_BYTES;
    static constexpr int ROUND = kStatsRound / 64;  // K steps of a round
    static constexpr int BAR_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int SMEM_BYTES =
        smem_request(BAR_OFFSET + (2 * STAGES + 5) * 8 + 16 + 1024, CTAS);
    static constexpr int TMEM_COLS = 2 * TOK;
    static constexpr int BN = TOK;  // OpAcc: accumulator stride
    static constexpr int CG = 1;
};

struct FewArgs {
    int T, V, D, k_tiles, tiles;
    int tile_rows;           // rows of W a tile, at most 128
    float *part_m, *part_s;  // [CTA][rows]
    long long rows;
    float *logits;           // T x V, pitch ld; or nullptr
    long long ld;
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    xent_few_kernel(const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_x, const FewArgs a,
                    const KernelCtx ctx) {
    constexpr int TOK = Cfg::TOK, TT = Cfg::TT, STAGES = Cfg::STAGES, BK = Cfg::BK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFFSET);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    __shared__ float sm[4][TOK], ss[4][TOK];
    const uint32_t warp = warp_id_uniform(), lane = lane_id();
    if (warp == 0 && lane == 0) {
        if (a.k_tiles > 0) {
            prefetch_tmap(&map_w);
            prefetch_tmap(&map_x);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
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

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t stage_tx = a.tile_rows * BK * 2 + Cfg::X_BYTES;
            uint32_t it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < a.tiles; tile += gridDim.x) {
                for (int kt = 0; kt < a.k_tiles; ++kt, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(&empty[s], ph ^ 1u, ctx, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = smem + s * Cfg::STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[s], stage_tx);
                    tma_load_2d(st, &map_w, &full[s], kt * BK, tile * a.tile_rows);
                    tma_load_2d(st + Cfg::W_BYTES, &map_x, &full[s], kt * BK, 0);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(128, TOK, 1, 0, 0);
            uint32_t it = 0, gr = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < a.tiles; tile += gridDim.x) {
                for (int k0 = 0; ok && k0 < a.k_tiles; k0 += Cfg::ROUND, ++gr) {
                    const uint32_t ab = gr & 1u, aph = (gr >> 1) & 1u;
                    if (!mbar_wait(&acc_empty[ab], aph ^ 1u, ctx, kSiteMmaAccEmpty)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int k1 = min(a.k_tiles, k0 + Cfg::ROUND);
                    for (int kt = k0; kt < k1; ++kt, ++it) {
                        const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                        if (!mbar_wait(&full[s], ph, ctx, kSiteMmaFull)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = smem_u32(smem + s * Cfg::STAGE_BYTES);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            umma_f16_ss(tmem + ab * TOK, smem_desc_sw128(st + k * 32, 16, 1024),
                                        smem_desc_sw128(st + Cfg::W_BYTES + k * 32, 16, 1024),
                                        idesc, (kt == k0 && k == 0) ? 0u : 1u);
                        umma_commit(&empty[s]);
                    }
                    if (ok) umma_commit(&acc_full[ab]);
                }
            }
            umma_commit(mma_done);
            mbar_wait(mma_done, 0, ctx, kSiteMmaDone);
        }
    } else {
        const uint32_t q = warp & 3u;
        const int t0 = static_cast<int>((warp - 2) >> 2) * TT;  // this warp's tokens
        OpAcc<Cfg> acc{acc_full, acc_empty, tmem + ((q * 32u) << 16) + t0, lane, 0u,
                       (a.k_tiles + Cfg::ROUND - 1) / Cfg::ROUND, ctx};
        float m[TT], s[TT];
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            m[j] = -CUDART_INF_F;
            s[j] = 0.0f;
        }
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < a.tiles; tile += gridDim.x) {
            __syncwarp();
            float x[TT];
#pragma unroll
            for (int j = 0; j < TT; ++j) x[j] = 0.0f;
#pragma unroll 1
            for (int r = 0; r < acc.rounds; ++r) {
                if (!acc.wait()) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int c = 0; c < TT; c += 16) {
                    uint32_t y[16];
                    tmem_ld_32x32b_x16(acc.row() + c, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[c + j] += __uint_as_float(y[j]);
                }
                acc.release();
            }
            // the MMA's rows beyond the tile's hold what the stage held before
            const int row = static_cast<int>(q * 32 + lane);
            const long long v = static_cast<long long>(tile) * a.tile_rows + row;
            if (!ok || row >= a.tile_rows || v >= a.V) continue;
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                if (a.logits != nullptr && t0 + j < a.T)
                    a.logits[static_cast<long long>(t0 + j) * a.ld + v] = x[j];
                const float b = x[j] * kLog2e;
                const float n = fmaxf(m[j], b);
                const float ref = fabsf(n) == CUDART_INF_F ? 0.0f : n;
                s[j] = fmaf(s[j], ex2_ftz(m[j] - ref), ex2_ftz(b - ref));
                m[j] = n;
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < TT; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o /= 2) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m[j], o);
                const float s2 = __shfl_xor_sync(0xffffffffu, s[j], o);
                join_ms(m[j], s[j], m2, s2);
            }
            if (lane == 0) {
                sm[q][t0 + j] = m[j];
                ss[q][t0 + j] = s[j];
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    for (int t = static_cast<int>(threadIdx.x); t < a.T; t += Cfg::THREADS) {
        float m = sm[0][t], s = ss[0][t];
#pragma unroll
        for (int i = 1; i < 4; ++i) join_ms(m, s, sm[i][t], ss[i][t]);
        a.part_m[blockIdx.x * a.rows + t] = m;
        a.part_s[blockIdx.x * a.rows + t] = s;
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// P from kept logits, with what xent_join_kernel does for other gradients: a
// block takes kProbCols columns of a row, joins the row's (m, s) itself (a few hundred
// pairs from L2) and the weights' common scale, and leaves a launch out.  The first
// block of a row also writes its loss and lse.
constexpr int kProbCols = 2048;  // eight a thread
__global__ void __launch_bounds__(256)
    xent_probs_kernel(const float *part_m, const float *part_s, long long rows, int blocks,
                      const float *logits, uint16_t *P, long long ld, int T, int V, int D,
                      const OpMat X, const OpMat W, const int64_t *target, float *loss,
                      float *lse, const float *dloss, float *scale) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float sm[8], ss[8], dot[8], sc[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int across = (V - 1) / kProbCols + 1;
    const int t = blockIdx.x / across;
    const int c0 = (blockIdx.x - t * across) * kProbCols;
    const int64_t y = target[t];
    const bool counts = y >= 0 && y < V;
    float m = -CUDART_INF_F, s = 0.0f, d = 0.0f, g = 0.0f;
    for (int b = threadIdx.x; b < blocks; b += 256)
        join_ms(m, s, part_m[b * rows + t], part_s[b * rows + t]);
    if (dloss != nullptr && threadIdx.x < T) {  // T <= kFewMax threads
        const int64_t yi = target[threadIdx.x];
        const float v = fabsf(dloss[threadIdx.x]);
        if (yi >= 0 && yi < V && v < CUDART_INF_F) g = v;
    }
    if (c0 == 0 && loss != nullptr && counts)
        d = row_dot(X.p + t * X.ld, W.p + y * W.ld, D, static_cast<int>(threadIdx.x) * 8, 2048);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join_ms(m, s, m2, s2);
        d += __shfl_xor_sync(0xffffffffu, d, o);
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    }
    if (lane == 0) {
        sm[w] = m;
        ss[w] = s;
        dot[w] = d;
        sc[w] = g;
    }
    __syncthreads();
    m = sm[0];
    s = ss[0];
    d = dot[0];
    g = sc[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        join_ms(m, s, sm[i], ss[i]);
        d += dot[i];
        g = fmaxf(g, sc[i]);
    }
    const float c = dloss != nullptr && g > 0.0f ? g : 1.0f;
    const float l2 = m + log2f(s);
    if (threadIdx.x == 0 && c0 == 0) {
        if (lse) lse[t] = kLn2 * l2;
        if (loss) loss[t] = counts ? loss_of(kLn2 * l2, d) : 0.0f;
        if (dloss != nullptr && t == 0) *scale = c;
    }
    const float gt = counts ? (dloss ? dloss[t] / c : 1.0f) : 0.0f;
    const int k = c0 + static_cast<int>(threadIdx.x) * 8;
    if (k < V) {
        const float4 *src = reinterpret_cast<const float4 *>(logits + t * ld + k);
        const float4 p = src[0], q = src[1];
        const float x[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float e = exp2f(fmaf(x[j], kLog2e, -l2));
            if (y == k + j) e -= 1.0f;
            o[j] = counts ? e * gt : 0.0f;
        }
        *reinterpret_cast<uint4 *>(P + t * ld + k) =
            make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                       pack_bf16(o[6], o[7]));
    }
}

template <class Cfg>
static pgemm_status launch_few(const OpDevice &dev, FewArgs a, const OpMat &X, const OpMat &W,
                               int ctas, cudaStream_t s) {
    static const KernelInfo info = [] {
        KernelInfo k;
        k.threads = Cfg::THREADS;
        k.smem_bytes = Cfg::SMEM_BYTES;
        k.func = reinterpret_cast<const void *>(xent_few_kernel<Cfg>);
        return k;
    }();
    int slots = 0;
    pgemm_status st = op_kernel_setup(dev, info, &slots);
    CUtensorMap mw{}, mx{};
    if (a.D > 0) {
        if (st == PGEMM_OK) st = op_encode(&mw, W.p, a.D, a.V, W.ld, a.tile_rows);
        if (st == PGEMM_OK) st = op_encode(&mx, X.p, a.D, a.T, X.ld, Cfg::TOK);
    }
    if (st != PGEMM_OK) return st;
    a.k_tiles = op_blocks(a.D, Cfg::BK);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(ctas));
    lc.blockDim = dim3(Cfg::THREADS);
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = s;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, xent_few_kernel<Cfg>, mw, mx, a, dev.ctx) == cudaSuccess
               ? PGEMM_OK
               : PGEMM_ERR_CUDA;
}
constexpr int kFewMax = 64;
constexpr int kFewEvenD = 512;  // from here on every CTA gets the same number of tiles

// the statistics' tiles (rounds of kStatsRound products), and P's where D is no longer
// than a round
using StatsPair = OpCfg<256, 3, 2, 2, false, true, false, kStatsRound / 128>;
using StatsOne = OpCfg<128, 6, 1, 1, false, true, false, kStatsRound / 64>;
using XentPair = OpCfg<256, 3, 2, 2, false, true>;
using XentOne = OpCfg<128, 6, 1, 1, false, true>;

template <class Cfg, class Epi>
static pgemm_status launch_logits(const OpDevice &dev, int T, int cols, int D, const OpMat &X,
                                  const OpMat &W, long long v0, OpMaps &maps, const Epi &e,
                                  cudaStream_t s) {
    if (D > 0) {
        pgemm_status st = op_encode(&maps.a[0], X.p, D, T, X.ld, 128);
        if (st == PGEMM_OK)
            st = op_encode(&maps.b[0], W.p + v0 * W.ld, D, cols, W.ld, 64);
        if (st != PGEMM_OK) return st;
    }
    constexpr int TM = Cfg::BM * Cfg::CG;
    OpArgs a{};
    a.M = T;
    a.N = cols;
    a.K = D;
    a.m_tiles = op_blocks(T, TM);
    a.n_seg = a.n_tiles = op_blocks(cols, Cfg::TILE_N);
    a.k_seg = a.k_tiles = op_blocks(D, Cfg::SBK);
    a.parts = 1;
    return op_launch<Cfg, Epi>(dev, maps, a, e, s);
}

// Workspace of a gradient's P when the caller names none: 2 GiB (all of P up
// to 8192 tokens x 131072).
constexpr long long kDefaultWorkspace = 2ll << 30;

static pgemm_status xent(int T, int V, int D, const uint16_t *X, const uint16_t *W,
                         const int64_t *target, const float *dloss, float *loss, float *lse,
                         uint16_t *dX, uint16_t *dW, long long workspace, cudaStream_t s) {
    if (T < 0 || V < 1 || D < 0 || workspace < 0) return PGEMM_ERR_INVALID_VALUE;
    const bool want_x = dX && T > 0 && D > 0, want_w = dW && D > 0;
    if (T == 0 && !want_w) return PGEMM_OK;
    if (T > 0 && (!target || (D > 0 && (!X || !W)))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(W) || !op_aligned16(dX) || !op_aligned16(dW) ||
        !op_aligned16(target) || !op_aligned16(dloss) || !op_aligned16(loss) || !op_aligned16(lse))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    if (T == 0)
        return cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * D * 2, s) == cudaSuccess
                   ? PGEMM_OK
                   : PGEMM_ERR_CUDA;

    const bool few = T <= kFewMax;
    const bool pair = op_use_pair(dev, T, V, D, 256, 128);
    const int block_cols = pair ? StatsPair::EPI_COLS : StatsOne::EPI_COLS;
    // (m, s) of a row: one for each column block, or for each CTA
    int blocks = op_blocks(V, block_cols);
    int few_rows = 128, few_tiles = 0;
    if (few) {
        // 128 rows a tile, unless the CTAs take several each: then the same number for
        // every CTA, since a few left over would cost a wave of their own.  39928 x
        // 2048, one token: 38.7 us with whole tiles, 33.8 so; 50257 x 1024: 25.0 and
        // 23.5.  A short D pays more for the further tile than for the wave (39928 x
        // 160: 8.7 and 9.6 us), and CTAs with one tile each lose by shorter ones
        // (18488 x 1024: 12.3 and 13.7).
        const long long ctas = dev.sm_count * (T <= 32 ? 2 : 1);
        const long long waves = (V + 128 * ctas - 1) / (128 * ctas);
        if (waves > 1 && D >= kFewEvenD)
            few_rows = static_cast<int>(
                op_round_up((V + waves * ctas - 1) / (waves * ctas), 8));
        few_tiles = op_blocks(V, few_rows);
        blocks = static_cast<int>(few_tiles < ctas ? few_tiles : ctas);
    }
    const long long rows = op_round_up(T, 32);
    // vocabulary pieces, whole tiles wide
    const long long p_ld_all = op_round_up(V, 256);
    long long piece = 0;
    int pieces = 0;
    const long long cap = workspace > 0 ? workspace : kDefaultWorkspace;
    if (want_x || want_w) {
        // bytes an entry: P, and with few tokens its fp32 logits
        piece = cap / ((few ? 6ll : 2ll) * T) / 256 * 256;
        if (piece < 256) piece = 256;
        if (piece > p_ld_all) piece = p_ld_all;
        pieces = op_blocks(V, piece);
        // of equal width, so that none is a sliver
        piece = op_round_up(op_blocks(V, pieces), 256);
        pieces = op_blocks(V, piece);
    }

    OpArena arena(dev, s);
    OpRelayout rl;
    OpMat x, w;
    if (D > 0) {
        rl.add(&x, X, T, D, arena);
        rl.add(&w, W, V, D, arena);
    }
    const long long at_m = arena.add(blocks * rows * 4);
    const long long at_s = arena.add(blocks * rows * 4);
    const long long at_l = lse ? 0 : arena.add(rows * 4);
    if (pieces == 0) dloss = nullptr;
    const long long at_c = dloss ? arena.add(4) : 0;
    const long long at_p = pieces ? arena.add(piece * T * 2) : 0;
    const bool keep_logits = few && pieces == 1;
    const long long at_z = keep_logits ? arena.add(piece * T * 4) : 0;
    // dX of several pieces: fp32 partial sums, T x D each.  As many as the workspace
    // holds again, at least a running sum and one piece's parts; when they are full the
    // running sum takes them in (sums over more pieces in less memory).
    long long at_x = 0;
    int x_slots = 0;
    const long long x_slot = op_parts_ld(D) * op_parts_rows(T);
    const bool x_pieces = want_x && pieces > 1;
    if (x_pieces) {
        long long all = 0, most = 0;
        for (int i = 0; i < pieces; ++i) {
            const long long cols = V - i * piece < piece ? V - i * piece : piece;
            const int parts = op_product_parts(dev, T, D, static_cast<int>(cols), 1);
            all += parts;
            most = parts > most ? parts : most;
        }
        const long long fit = cap / (x_slot * 4), least = 1 + most;
        x_slots = static_cast<int>(std::min(all, std::max(least, fit)));
        at_x = arena.add(x_slot * 4 * x_slots);
    }
    // the products of a piece, planned for the first (the widest): the others'
    // parts need no more room
    // (more rows: dW starts beside the parts of a tiled dX, 352 x 7517 x 1456 54 us
    // against 58)
    const bool x_tokens = !x_pieces && T <= kTokensMax && op_tokens_fit(dev, T, D, V);
    OpProduct px, pw;
    const auto shape = [&](int cols) {
        px.form = OpForm::NN;
        px.M = T;
        px.N = D;
        px.K = cols;
        px.out[0] = dX;
        pw.form = OpForm::TN;
        pw.M = cols;
        pw.N = D;
        pw.K = T;
    };
    if (pieces) {
        shape(static_cast<int>(V < piece ? V : piece));
        if (want_x && !x_pieces && !x_tokens) op_product_plan(dev, px, arena);
        if (want_w) op_product_plan(dev, pw, arena);
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    float *lse_buf = lse ? lse : arena.at<float>(at_l);
    float *scale = dloss ? arena.at<float>(at_c) : nullptr;  // c
    px.epi.scale = pw.epi.scale = scale;

    // One piece: its exponentials are kept and P follows from them.
    const bool keep = pieces == 1 && !few;
    float *part_m = arena.at<float>(at_m), *part_s = arena.at<float>(at_s);
    uint16_t *P = pieces ? arena.at<uint16_t>(at_p) : nullptr;
    {
        OpMaps maps{};
        if (few) {
            const FewArgs a{T, V, D, 0, few_tiles, few_rows, part_m, part_s, rows,
                            keep_logits ? arena.at<float>(at_z) : nullptr, piece};
            st = T <= 16   ? launch_few<FewCfg<16>>(dev, a, x, w, blocks, s)
                 : T <= 32 ? launch_few<FewCfg<32>>(dev, a, x, w, blocks, s)
                           : launch_few<FewCfg<64>>(dev, a, x, w, blocks, s);
        } else if (keep) {
            st = op_encode_out(&maps.c[0], OpElem::BF16, P, V, T, piece);
            if (st != PGEMM_OK) return st;
            const EpiXentStats<true> e{part_m, part_s, rows};
            st = pair ? launch_logits<StatsPair>(dev, T, V, D, x, w, 0, maps, e, s)
                      : launch_logits<StatsOne>(dev, T, V, D, x, w, 0, maps, e, s);
        } else {
            const EpiXentStats<false> e{part_m, part_s, rows};
            st = pair ? launch_logits<StatsPair>(dev, T, V, D, x, w, 0, maps, e, s)
                      : launch_logits<StatsOne>(dev, T, V, D, x, w, 0, maps, e, s);
        }
        if (st != PGEMM_OK) return st;
        if (keep_logits) {
            const unsigned across = op_blocks(V, kProbCols);
            st = launch_small(xent_probs_kernel, dim3(across * T), dim3(256), s,
                              static_cast<const float *>(part_m),
                              static_cast<const float *>(part_s), rows, blocks,
                              static_cast<const float *>(arena.at<float>(at_z)), P, piece, T, V, D,
                              x, w, target, loss, lse, dloss, scale);
        } else {
            const bool by_row = T < 8 * dev.sm_count;  // fewer than a block of 8 rows an SM
            st = launch_small(by_row ? xent_join_kernel<1> : xent_join_kernel<8>,
                              dim3(by_row ? T : op_blocks(T, 8)), dim3(256), s,
                              static_cast<const float *>(part_m),
                              static_cast<const float *>(part_s), rows, blocks, T,
                              static_cast<long long>(V), D, x, w, target, loss, lse_buf, dloss,
                              scale);
        }
        if (st != PGEMM_OK) return st;
    }

    int x_done = 0;
    for (int i = 0; i < pieces; ++i) {
        const long long v0 = i * piece;
        const int cols = static_cast<int>(V - v0 < piece ? V - v0 : piece);
        if (keep_logits) {
            // P is there already
        } else if (keep) {
            const dim3 grid(static_cast<unsigned>(op_blocks(V, 1024)) * op_blocks(T, 32));
            st = launch_small(pair ? xent_scale_kernel<StatsPair::EPI_COLS>
                                   : xent_scale_kernel<StatsOne::EPI_COLS>,
                              grid, dim3(256), s, P, piece, T, V,
                              static_cast<const float *>(part_m), rows,
                              static_cast<const float *>(lse_buf), target, dloss,
                              static_cast<const float *>(scale));
        } else {
            OpMaps maps{};
            st = op_encode_out(&maps.c[0], OpElem::BF16, P, cols, T, piece);
            if (st != PGEMM_OK) return st;
            const EpiXentGrad e{target, lse_buf, dloss, scale, v0, V};
            const bool two = op_use_pair(dev, T, cols, D, 256, 128);
            if (D > kStatsRound)
                st = two ? launch_logits<StatsPair>(dev, T, cols, D, x, w, v0, maps, e, s)
                         : launch_logits<StatsOne>(dev, T, cols, D, x, w, v0, maps, e, s);
            else
                st = two ? launch_logits<XentPair>(dev, T, cols, D, x, w, v0, maps, e, s)
                         : launch_logits<XentOne>(dev, T, cols, D, x, w, v0, maps, e, s);
        }
        if (st != PGEMM_OK) return st;
        shape(cols);
        if (want_x) {
            px.A[0] = OpMat{P, piece};
            px.B[0] = OpMat{w.p + v0 * w.ld, w.ld};
            if (x_pieces) {
                float *sums = px.parts_area = arena.at<float>(at_x);
                op_product_plan(dev, px, arena);  // this piece's; reserves nothing
                if (x_done + px.plan.parts > x_slots) {
                    if ((st = op_fold_parts(dev, sums, x_done, T, D, s)) != PGEMM_OK) return st;
                    x_done = 1;
                }
                px.parts_area = sums + x_slot * x_done;
                x_done += px.plan.parts;
            }
            st = x_tokens ? op_tokens_linear(dev, T, D, cols, px.A[0], px.B[0], px.epi, dX, s)
                          : op_product(dev, px, arena, s);
            if (st != PGEMM_OK) return st;
        }
        if (want_w) {
            pw.A[0] = OpMat{P, piece};
            pw.B[0] = x;
            pw.out[0] = dW + v0 * D;
            pw.overlap = want_x;  // behind dX, which has waited for P
            if ((st = op_product(dev, pw, arena, s)) != PGEMM_OK) return st;
            if ((st = op_product_join(dev, pw, arena, s)) != PGEMM_OK) return st;
        }
        if (want_x && !x_pieces && (st = op_product_join(dev, px, arena, s)) != PGEMM_OK) return st;
    }
    if (x_pieces) {
        uint16_t *out[2] = {dX, nullptr};
        OpEpilogue scaled;
        scaled.scale = scale;
        st = op_join_parts(dev, arena.at<float>(at_x), x_done, 1, T, D, out, scaled, s);
    }
    return st;
}

}  // namespace pg

extern "C" {

pgemm_status xent_bf16(int T, int V, int D, const uint16_t *X, const uint16_t *W,
                       const int64_t *target, float *loss, float *lse, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::xent(T, V, D, X, W, target, nullptr, loss, lse, nullptr, nullptr, 0, stream);
    });
}

pgemm_status xent_bf16_grad(int T, int V, int D, const uint16_t *X, const uint16_t *W,
                            const int64_t *target, const float *dloss, float *loss, float *lse,
                            uint16_t *dX, uint16_t *dW, long long workspace_bytes,
                            pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::xent(T, V, D, X, W, target, dloss, loss, lse, dX, dW, workspace_bytes, stream);
    });
}

}  // extern "C"
