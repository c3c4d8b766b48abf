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
#include <math_constants.h>

#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

constexpr float kLog2e = 1.4426950408889634f;

// Running maximum and sum of one row segment.
struct EpiXentStats {
    const int64_t *target;
    float *part_m, *part_s;  // [column block][rows]
    long long rows;
    float *target_logit;     // [rows]

    template <class Cfg, class Wait, class Rel>
    __device__ __forceinline__ bool run(const EpiCtx &c, const OpMaps &, const OpArgs &,
                                        const OpUnit &w, uint32_t t_row, int col0, bool have,
                                        Wait wait, Rel release) const {
        const int n0 = w.n0 + col0;
        const bool in = c.row() < c.M;
        // the target's column in this warp's segment (none: out of [0, EPI_COLS))
        const int64_t y = in ? __ldg(target + c.row()) : -1;
        const int64_t yc = y - n0;
        if (!wait()) return false;
        float m = -CUDART_INF_F, s = 0.0f;
#pragma unroll 1
        for (int cc = 0; cc < Cfg::EPI_COLS; cc += 32) {
            uint32_t v[32];
            acc_cols32(t_row + col0 + cc, have, v);
            if (cc + 32 >= Cfg::EPI_COLS) release();
            const int left = c.N - (n0 + cc);  // columns of the vocabulary in this chunk
            if (left <= 0) continue;
            if (left < 32) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= left) v[j] = __float_as_uint(-CUDART_INF_F);
            }
            float cm = m;
#pragma unroll
            for (int j = 0; j < 32; ++j) cm = fmaxf(cm, __uint_as_float(v[j]));
            // nothing but -inf so far: any finite reference gives exp(-inf) = 0
            const float ref = cm == -CUDART_INF_F ? 0.0f : cm;
            s *= exp2f((m - ref) * kLog2e);
            float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                t0 += exp2f((__uint_as_float(v[j]) - ref) * kLog2e);
                t1 += exp2f((__uint_as_float(v[j + 1]) - ref) * kLog2e);
            }
            s += t0 + t1;
            m = cm;
            if (yc >= cc && yc < cc + 32 && y < c.N) {
                float at = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j == static_cast<int>(yc) - cc) at = __uint_as_float(v[j]);
                target_logit[c.row()] = at;
            }
        }
        if (in && n0 < c.N) {
            const long long at = static_cast<long long>(n0 / Cfg::EPI_COLS) * rows + c.row();
            part_m[at] = m;
            part_s[at] = s;
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

    template <class Cfg, class Wait, class Rel>
    __device__ __forceinline__ bool run(const EpiCtx &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, uint32_t t_row, int col0, bool have,
                                        Wait wait, Rel release) const {
        const int n0 = w.n0 + col0;
        const bool in = c.row() < c.M;
        const int64_t y = in ? __ldg(target + c.row()) : -1;
        const bool counts = y >= 0 && y < V;
        const float l = counts ? lse[c.row()] : 0.0f;
        const float g = counts ? (dloss ? dloss[c.row()] : 1.0f) : 0.0f;
        const int64_t yc = y - v0 - n0;
        if (!wait()) return false;
#pragma unroll 1
        for (int cc = 0; cc < Cfg::EPI_COLS; cc += 64) {
            uint32_t p[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
                acc_cols32(t_row + col0 + cc + 32 * h, have, v);
                if (h == 1 && cc + 64 >= Cfg::EPI_COLS) release();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float x = exp2f((__uint_as_float(v[j]) - l) * kLog2e);
                    if (yc == cc + 32 * h + j) x -= 1.0f;
                    v[j] = __float_as_uint(counts ? x * g : 0.0f);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    p[16 * h + j] =
                        pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            }
            put_rows64(c, &maps.c[0], nullptr, 0, n0 + cc, p);
        }
        return true;
    }
};

// lse and loss of a row from its column blocks' (m, s).  A block takes 32 rows
// (a warp's loads are 128 consecutive bytes), eight warps every eighth column
// block of them; a running (m, s) each, joined through shared memory.
__device__ __forceinline__ void join_ms(float &m, float &s, float m2, float s2) {
    const float n = fmaxf(m, m2);
    const float ref = n == -CUDART_INF_F ? 0.0f : n;
    s = s * exp2f((m - ref) * kLog2e) + s2 * exp2f((m2 - ref) * kLog2e);
    m = n;
}

__global__ void __launch_bounds__(256)
    xent_join_kernel(const float *part_m, const float *part_s, long long rows, int blocks, int T,
                     long long V, const int64_t *target, const float *target_logit, float *loss,
                     float *lse) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float sm[8][32], ss[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int t = blockIdx.x * 32 + lane;
    float m = -CUDART_INF_F, s = 0.0f;
    if (t < T) {
#pragma unroll 4
        for (int b = w; b < blocks; b += 8)
            join_ms(m, s, part_m[b * rows + t], part_s[b * rows + t]);
    }
    sm[w][lane] = m;
    ss[w][lane] = s;
    __syncthreads();
    if (w == 0 && t < T) {
#pragma unroll
        for (int i = 1; i < 8; ++i) join_ms(m, s, sm[i][lane], ss[i][lane]);
        const float l = m + logf(s);
        const int64_t y = target[t];
        if (lse) lse[t] = l;
        if (loss) loss[t] = y >= 0 && y < V ? l - target_logit[t] : 0.0f;
    }
}

using XentPair = OpCfg<256, 3, 2, 2, false, true>;
using XentOne = OpCfg<128, 6, 1, 1, false, true>;

template <class Cfg, class Epi>
static pgemm_status launch_logits(const OpDevice &dev, int T, int cols, int D, const OpMat &X,
                                  const OpMat &W, long long v0, OpMaps &maps, const Epi &e,
                                  cudaStream_t s) {
    if (D > 0) {
        pgemm_status st = op_encode(&maps.a[0], OpElem::BF16, X.p, D, T, X.ld, 64, 128);
        if (st == PGEMM_OK)
            st = op_encode(&maps.b[0], OpElem::BF16, W.p + v0 * W.ld, D, cols, W.ld, 64,
                           Cfg::B_COLS);
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
    const int block_cols = pair ? XentPair::EPI_COLS : XentOne::EPI_COLS;
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
    const long long at_t = arena.add(rows * 4);
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

    {
        OpMaps maps{};
        EpiXentStats e{target, arena.at<float>(at_m), arena.at<float>(at_s), rows,
                       arena.at<float>(at_t)};
        st = pair ? launch_logits<XentPair>(dev, T, V, D, x, w, 0, maps, e, s)
                  : launch_logits<XentOne>(dev, T, V, D, x, w, 0, maps, e, s);
        if (st != PGEMM_OK) return st;
        st = launch_small(xent_join_kernel, dim3((T + 31) / 32), dim3(256), s,
                          static_cast<const float *>(e.part_m), static_cast<const float *>(e.part_s),
                          rows, blocks, T, static_cast<long long>(V), target,
                          static_cast<const float *>(e.target_logit), loss, lse_buf);
        if (st != PGEMM_OK) return st;
    }

    int x_done = 0;
    for (int i = 0; i < pieces; ++i) {
        const long long v0 = i * piece;
        const int cols = static_cast<int>(V - v0 < piece ? V - v0 : piece);
        uint16_t *P = arena.at<uint16_t>(at_p);
        OpMaps maps{};
        if ((st = op_encode(&maps.c[0], OpElem::BF16, P, cols, T, piece, 64, 32)) != PGEMM_OK)
            return st;
        EpiXentGrad e{target, lse_buf, dloss, v0, V};
        st = op_use_pair(dev, T, cols, 256, 128, 1)
                 ? launch_logits<XentPair>(dev, T, cols, D, x, w, v0, maps, e, s)
                 : launch_logits<XentOne>(dev, T, cols, D, x, w, v0, maps, e, s);
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
