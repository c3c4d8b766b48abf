// xent_bf16: softmax cross entropy of logits L = X W^T over a vocabulary
// (W: one row of D for each of V tokens), and its gradients, without keeping L.
//
//   lse_t  = log sum_v exp L_tv          loss_t = lse_t - L_t,y(t)
//   P_tv   = (exp(L_tv - lse_t) - [v = y(t)]) dloss_t
//   dX     = P W                         dW = P^T X
//
// Forward: the product's epilogue folds every accumulator into a running
// maximum m and sum s of exp(L - m) for each row and column block (a thread
// holds a whole row segment, so neither needs a shuffle), and the logit of the
// row's own target is written by the thread that holds it.  A second kernel
// joins the blocks of a row: lse = M + log sum_b s_b exp(m_b - M).
// Gradient: the vocabulary goes by in pieces whose P fits the workspace; each
// piece's logits are recomputed by the same product, whose epilogue writes P
// (rounded to bf16 once, as an operand of the gradient products).
//
// A row whose target lies outside [0, V) does not count: loss 0, gradient 0.
#include <cuda_fp16.h>
#include <math_constants.h>

#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// For statistics: results below 2^-126 of the block's largest count as zero.
// Probabilities themselves take exp2f, which keeps subnormal results.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Softmax statistics are kept to base 2: m is the largest L log2(e) of a row's
// column block, s the block's sum of 2^(L log2(e) - m).
//
// Accumulation rounds of 1024 products are added in fp32 registers.  The
// tensor core truncates its running sum at every step of 16 products, always
// toward zero: over the 256 steps of D = 4096 that shrinks every logit by some
// 1e-5 of its size, which the statistics of a whole vocabulary do not average
// out (lse off by 2e-6 of itself); four rounds of 64 steps and three rounded
// additions leave a quarter of it.
//
// KEEP: the exponentials themselves are stored as fp16, 2^(L log2(e) - m) with
// the block's own m, so that the gradient pass turns them into P without the
// logits' product a second time.  They lie in (0, 1] and fp16 carries them to
// 2^-11 of their size, an eighth of what rounding P to bf16 costs.
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
        if (Cfg::HALVES && w.half && e >= 4) {
#pragma unroll 1
            for (int r = 0; r < acc.rounds; ++r) {
                if (!acc.wait()) return false;
                acc.release();
            }
            return true;
        }
        const int n0 = w.n0 + col0;
        float v[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) v[j] = 0.0f;
#pragma unroll 1
        for (int r = 0; r < acc.rounds; ++r) {
            if (!acc.wait()) return false;
            const uint32_t t_row = acc.row() + col0;
#pragma unroll
            for (int cc = 0; cc < COLS; cc += 16) {
                uint32_t x[16];
                tmem_ld_32x32b_x16(t_row + cc, x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[cc + j] += __uint_as_float(x[j]);
            }
            acc.release();
        }
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
        const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kLog2e;
        // nothing but -inf: any finite reference gives sums of zero
        const float ref = m == -CUDART_INF_F ? 0.0f : m;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int cc = 0; cc < COLS; cc += 32) {
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float a = ex2(fmaf(v[cc + 2 * j], kLog2e, -ref));
                const float b = ex2(fmaf(v[cc + 2 * j + 1], kLog2e, -ref));
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
            part_s[at] = (s[0] + s[1]) + (s[2] + s[3]);
        }
        return true;
    }
};

// P of one piece of the vocabulary.
struct EpiXentGrad {
    const int64_t *target;
    const float *lse, *dloss;  // dloss nullptr: 1
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
        const float g = counts ? (dloss ? dloss[c.row()] : 1.0f) : 0.0f;
        const int64_t yc = y - v0 - n0;
        if (!acc.wait()) return false;
        const uint32_t t_row = acc.row() + col0;
#pragma unroll 1
        for (int cc = 0; cc < cols; cc += 32) {
            uint32_t v[32], p[16];
            acc_cols32(t_row + cc, have, v);
            if (cc + 32 >= cols) acc.release();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                float x = exp2f(fmaf(__uint_as_float(v[j]), kLog2e, -l));
                if (yc == cc + j) x -= 1.0f;
                v[j] = __float_as_uint(counts ? x * g : 0.0f);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                p[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            put_rows32(c, &maps.c[0], nullptr, 0, n0 + cc, p);
        }
        return true;
    }
};

// lse and loss of a row from its column blocks' (m, s), and its target's logit
// as an fp32 dot product of its own (the epilogues would have to pick one of
// their registers by a runtime index).  A block takes eight rows: 32 threads a
// row join every 32nd column block (8 adjacent rows make a 32-byte sector),
// then a warp a row multiplies X[t] by W[target].
__device__ __forceinline__ void join_ms(float &m, float &s, float m2, float s2) {
    const float n = fmaxf(m, m2);
    const float ref = n == -CUDART_INF_F ? 0.0f : n;
    s = s * ex2(m - ref) + s2 * ex2(m2 - ref);
    m = n;
}

__global__ void __launch_bounds__(256)
    xent_join_kernel(const float *part_m, const float *part_s, long long rows, int blocks, int T,
                     long long V, int D, const OpMat X, const OpMat W, const int64_t *target,
                     float *loss, float *lse) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float sm[8][8], ss[8][8], dot[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int r = threadIdx.x & 7;
    const int t = blockIdx.x * 8 + r;
    float m = -CUDART_INF_F, s = 0.0f;
    if (t < T) {
#pragma unroll 8
        for (int b = threadIdx.x >> 3; b < blocks; b += 32)
            join_ms(m, s, part_m[b * rows + t], part_s[b * rows + t]);
    }
#pragma unroll
    for (int o = 8; o <= 16; o *= 2) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join_ms(m, s, m2, s2);
    }
    if (lane < 8) {
        sm[w][lane] = m;
        ss[w][lane] = s;
    }
    {
        const int tw = blockIdx.x * 8 + w;
        const int64_t y = tw < T ? target[tw] : -1;
        if (loss && y >= 0 && y < V) {
            const uint16_t *x = X.p + tw * X.ld, *e = W.p + y * W.ld;  // 16-byte-aligned rows
            float d = 0.0f;
            for (int k = lane * 8; k < D; k += 256) {
                const uint4 a = *reinterpret_cast<const uint4 *>(x + k);
                const uint4 b = *reinterpret_cast<const uint4 *>(e + k);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (k + 2 * i < D) d = fmaf(bf16_lo(aw[i]), bf16_lo(bw[i]), d);
                    if (k + 2 * i + 1 < D) d = fmaf(bf16_hi(aw[i]), bf16_hi(bw[i]), d);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
            if (lane == 0) dot[w] = d;
        }
    }
    __syncthreads();
    if (threadIdx.x < 8 && t < T) {
        m = sm[0][r];
        s = ss[0][r];
#pragma unroll
        for (int i = 1; i < 8; ++i) join_ms(m, s, sm[i][r], ss[i][r]);
        const float l = kLn2 * (m + log2f(s));
        const int64_t y = target[t];
        if (lse) lse[t] = l;
        if (loss) loss[t] = y >= 0 && y < V ? l - dot[r] : 0.0f;
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
                      const float *lse, const int64_t *target, const float *dloss) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int NB = 1024 / COLS;
    __shared__ float f[NB][32], g[32];
    __shared__ int yc[32];  // the target's column within the block's 1024, or -1
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int across = (V + 1023) / 1024;
    const int c0 = static_cast<int>(blockIdx.x % across) * 1024;
    const int row0 = static_cast<int>(blockIdx.x / across) * 32;
    const int t = row0 + lane;
    const int64_t y = t < T ? target[t] : -1;
    const bool counts = y >= 0 && y < V;
    const float gt = counts ? (dloss ? dloss[t] : 1.0f) : 0.0f;
    if (w == 0) {
        g[lane] = gt;
        yc[lane] = counts && y >= c0 && y < c0 + 1024 ? static_cast<int>(y - c0) : -1;
    }
    const float l = counts ? lse[t] * kLog2e : 0.0f;
    for (int b = w; b < NB; b += 8) {
        const int col = c0 + b * COLS;
        f[b][lane] = counts && col < V
                         ? exp2f(part_m[static_cast<long long>(col / COLS) * rows + t] - l) * gt
                         : 0.0f;
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

// rounds of 1024 products for the statistics
using StatsPair = OpCfg<256, 3, 2, 2, false, true, false, 8>;
using StatsOne = OpCfg<128, 6, 1, 1, false, true, false, 16>;
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
    a.m_tiles = (T + TM - 1) / TM;
    a.n_seg = a.n_tiles = (cols + Cfg::TILE_N - 1) / Cfg::TILE_N;
    a.k_seg = a.k_tiles = (D + Cfg::SBK - 1) / Cfg::SBK;
    a.parts = 1;
    return op_launch<Cfg, Epi>(dev, maps, a, e, s);
}

// Workspace of a gradient's P when the caller names none: 2 GiB (all of P up
// to 8192 tokens x 131072).
constexpr long long kDefaultWorkspace = 2ll << 30;

// Kept exponentials cost 4 bytes of traffic a logit, computing it again 2 D
// operations: even near D = 600 at the measured peaks.
constexpr int kKeepMinD = 640;

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

    const bool pair = op_use_pair(dev, T, V, 256, 128, 1);
    const int block_cols = pair ? StatsPair::EPI_COLS : StatsOne::EPI_COLS;
    const int blocks = (V + block_cols - 1) / block_cols;
    const long long rows = op_round_up(T, 32);
    // vocabulary pieces, whole tiles wide
    const long long p_ld_all = op_round_up(V, 256);
    long long piece = 0;
    int pieces = 0;
    if (want_x || want_w) {
        const long long cap = workspace > 0 ? workspace : kDefaultWorkspace;
        piece = cap / (2ll * T) / 256 * 256;
        if (piece < 256) piece = 256;
        if (piece > p_ld_all) piece = p_ld_all;
        pieces = static_cast<int>((V + piece - 1) / piece);
        // of equal width, so that none is a sliver
        piece = op_round_up((V + pieces - 1) / pieces, 256);
        pieces = static_cast<int>((V + piece - 1) / piece);
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
    const long long at_p = pieces ? arena.add(piece * T * 2) : 0;
    long long at_x = 0;
    int x_parts = 0;
    const bool x_pieces = want_x && pieces > 1;
    if (x_pieces) {
        for (int i = 0; i < pieces; ++i) {
            const long long cols = V - i * piece < piece ? V - i * piece : piece;
            x_parts += op_product_parts(dev, T, D, static_cast<int>(cols), 1);
        }
        at_x = arena.add(op_parts_ld(D) * op_parts_rows(T) * 4 * x_parts);
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    float *lse_buf = lse ? lse : arena.at<float>(at_l);

    // One piece: its exponentials are kept and P follows from them.
    const bool keep = pieces == 1 && D >= kKeepMinD;
    float *part_m = arena.at<float>(at_m), *part_s = arena.at<float>(at_s);
    uint16_t *P = pieces ? arena.at<uint16_t>(at_p) : nullptr;
    {
        OpMaps maps{};
        if (keep) {
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
        st = launch_small(xent_join_kernel, dim3((T + 7) / 8), dim3(256), s,
                          static_cast<const float *>(part_m), static_cast<const float *>(part_s),
                          rows, blocks, T, static_cast<long long>(V), D, x, w, target, loss,
                          lse_buf);
        if (st != PGEMM_OK) return st;
    }

    int x_done = 0;
    for (int i = 0; i < pieces; ++i) {
        const long long v0 = i * piece;
        const int cols = static_cast<int>(V - v0 < piece ? V - v0 : piece);
        if (keep) {
            const dim3 grid(static_cast<unsigned>((V + 1023) / 1024) * ((T + 31) / 32));
            st = launch_small(pair ? xent_scale_kernel<StatsPair::EPI_COLS>
                                   : xent_scale_kernel<StatsOne::EPI_COLS>,
                              grid, dim3(256), s, P, piece, T, V,
                              static_cast<const float *>(part_m), rows,
                              static_cast<const float *>(lse_buf), target, dloss);
        } else {
            OpMaps maps{};
            st = op_encode_out(&maps.c[0], OpElem::BF16, P, cols, T, piece);
            if (st != PGEMM_OK) return st;
            const EpiXentGrad e{target, lse_buf, dloss, v0, V};
            st = op_use_pair(dev, T, cols, 256, 128, 1)
                     ? launch_logits<XentPair>(dev, T, cols, D, x, w, v0, maps, e, s)
                     : launch_logits<XentOne>(dev, T, cols, D, x, w, v0, maps, e, s);
        }
        if (st != PGEMM_OK) return st;
        if (want_x) {
            OpProduct p;
            p.form = OpForm::NN;
            p.M = T;
            p.N = D;
            p.K = cols;
            p.A[0] = OpMat{P, piece};
            p.B[0] = OpMat{w.p + v0 * w.ld, w.ld};
            p.out[0] = dX;
            if (x_pieces) {
                p.parts_area = arena.at<float>(at_x) +
                               op_parts_ld(D) * op_parts_rows(T) * static_cast<long long>(x_done);
                x_done += op_product_parts(dev, T, D, cols, 1);
            }
            if ((st = op_product(dev, p, s)) != PGEMM_OK) return st;
        }
        if (want_w) {
            OpProduct p;
            p.form = OpForm::TN;
            p.M = cols;
            p.N = D;
            p.K = T;
            p.A[0] = OpMat{P, piece};
            p.B[0] = x;
            p.out[0] = dW + v0 * D;
            if ((st = op_product(dev, p, s)) != PGEMM_OK) return st;
        }
    }
    if (x_pieces) {
        uint16_t *out[2] = {dX, nullptr};
        st = op_join_parts(dev, arena.at<float>(at_x), x_parts, 1, T, D, out, OpEpilogue{}, s);
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
