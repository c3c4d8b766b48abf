// linear_bf16: Y = act(X W + b) + R, and its gradients dX = dZ W^T, dW = X^T dZ and
// db = colsum dZ with dZ = dY act'(Z).  Z is kept in fp32 (a bf16 Z would add an
// error of up to 2^-8 of its size to the derivative) or computed again; keeping costs
// 8 bytes an element of traffic, computing 2 K operations, even near K = 1000.
#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

// Epilogue of the recomputing backward pass: Z = acc + b stays in fp32 and
// dZ = dY * act'(Z) is rounded to bf16 once, as the operand of the gradient
// products.
struct EpiLinearGrad {
    const uint16_t *bias, *dy;
    long long dy_ld;
    uint16_t *dz;
    long long dz_ld;
    int act;

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        int col0, cols;
        epi_cols<Cfg>(w, e, col0, cols);
        const int nf = w.n0 + col0;
        const bool have = acc.have();
        RowsIn in{dy, dy_ld};
        if (Cfg::ROUND == 0) in.load(c, nf);  // travels while the products finish
        // 32 columns from nf + cc: v holds the accumulator's
        auto finish = [&](int cc, uint32_t *v) {
            const int n = nf + cc;
            uint32_t r[16], p[16];
            if (bias != nullptr) {
                float b[32];
                get_vec32(bias, c.N, n, b);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + b[j]);
            }
            in.take(c, r);
            if (cc + 32 < cols) in.load(c, n + 32);
            auto derive = [&](auto A) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float value;
                    const float lo =
                        bf16_lo(r[j]) *
                        act_value_grad<decltype(A)::value>(__uint_as_float(v[2 * j]), value);
                    const float hi =
                        bf16_hi(r[j]) *
                        act_value_grad<decltype(A)::value>(__uint_as_float(v[2 * j + 1]), value);
                    p[j] = pack_bf16(lo, hi);
                }
            };
            if constexpr (Cfg::ROUND > 0)
                derive(std::integral_constant<int, PGEMM_ACT_RELU>{});
            else
                with_act(act, derive);
            put_rows32(c, &maps.c[0], dz, dz_ld, n, p);
        };
        if constexpr (Cfg::ROUND > 0) {
            float f[Cfg::EPI_COLS];
            if (!acc_sum_unit<Cfg>(acc, col0, cols, f)) return false;
            in.load(c, nf);  // (the sums fill the registers until here)
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

template <class Cfg>
static pgemm_status launch_grad(const OpDevice &dev, int M, int N, int K, const OpMat &X,
                                const OpMat &W, const EpiLinearGrad &e, cudaStream_t s) {
    OpMaps maps{};
    pgemm_status st = PGEMM_OK;
    if (K > 0) {
        st = op_encode(&maps.a[0], X.p, K, M, X.ld, 128);
        if (st == PGEMM_OK) st = op_encode(&maps.b[0], W.p, N, K, W.ld, 64);
    }
    if (st == PGEMM_OK) st = op_encode_out(&maps.c[0], OpElem::BF16, e.dz, N, M, e.dz_ld);
    if (st != PGEMM_OK) return st;
    constexpr int TM = Cfg::BM * Cfg::CG;
    OpArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.m_tiles = op_blocks(M, TM);
    a.n_seg = a.n_tiles = op_blocks(N, Cfg::TILE_N);
    a.k_seg = a.k_tiles = op_blocks(K, Cfg::SBK);
    a.parts = 1;
    return op_launch<Cfg, EpiLinearGrad>(dev, maps, a, e, s);
}

static pgemm_status linear_forward(int M, int N, int K, const uint16_t *X, const uint16_t *W,
                                   const uint16_t *bias, int act, const uint16_t *residual,
                                   uint16_t *Y, float *preact, cudaStream_t s) {
    if (M < 0 || N < 0 || K < 0 || !op_act_known(act)) return PGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return PGEMM_OK;
    if (!Y || (K > 0 && (!X || !W))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(W) || !op_aligned16(bias) || !op_aligned16(residual) ||
        !op_aligned16(Y) || !op_aligned16(preact))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    // (what may decide a ReLU's derivative goes in rounds, op_sign_rounds)
    const bool tokens =
        M <= kTokensMax || (!op_sign_rounds(act, K) && op_tokens_fit(dev, M, N, K));
    OpProduct p;
    p.form = OpForm::NN;
    p.M = M;
    p.N = N;
    p.K = K;
    p.out[0] = Y;
    p.epi = OpEpilogue{bias, act, residual, preact};
    OpArena arena(dev, s);
    OpRelayout rl;
    if (K > 0) {
        rl.add(&p.A[0], X, M, K, arena);
        if (M <= kTokensMax && op_raw_us(dev, M, N, K, false, false) <=
                          op_relayout_us(K, N, K % 8 != 0))
            p.B[0] = OpMat{W, N};  // read where it is, whatever its pitch
        else
            rl.add(&p.B[0], W, K, N, arena);
    }
    if (!tokens) op_product_plan(dev, p, arena);
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    if (tokens) return op_tokens_linear(dev, M, N, K, p.A[0], p.B[0], p.epi, Y, s);
    if ((st = op_product(dev, p, arena, s)) != PGEMM_OK) return st;
    return op_product_join(dev, p, arena, s);
}

static pgemm_status linear_backward(int M, int N, int K, const uint16_t *X, const uint16_t *W,
                                    const uint16_t *bias, int act, const uint16_t *dY,
                                    const float *preact, uint16_t *dX, uint16_t *dW,
                                    uint16_t *dbias, cudaStream_t s) {
    if (M < 0 || N < 0 || K < 0 || !op_act_known(act)) return PGEMM_ERR_INVALID_VALUE;
    const bool want_x = dX && M > 0 && K > 0, want_w = dW && K > 0 && N > 0;
    const bool want_b = dbias && N > 0;
    if (!want_x && !want_w && !want_b) return PGEMM_OK;
    const bool some = M > 0 && N > 0;  // dY has elements
    const bool recompute = some && act != PGEMM_ACT_NONE && !preact;
    if (some && !dY) return PGEMM_ERR_INVALID_VALUE;
    if (some && K > 0 && ((!X && (want_w || recompute)) || (!W && (want_x || recompute))))
        return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(W) || !op_aligned16(bias) || !op_aligned16(dY) ||
        !op_aligned16(preact) || !op_aligned16(dX) || !op_aligned16(dW) || !op_aligned16(dbias))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    if (want_b && M == 0 &&
        cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 2, s) != cudaSuccess)
        return PGEMM_ERR_CUDA;

    OpArena arena(dev, s);
    OpRelayout rl;
    const bool x_tokens = want_x && op_tokens_fit(dev, M, K, N);
    const bool tokens = M <= kTokensMax || (recompute && !op_sign_rounds(act, K) &&
                                            op_tokens_fit(dev, M, N, K));
    OpMat x, w, dz;
    if (some && K > 0) {
        if (X && (want_w || recompute)) rl.add(&x, X, M, K, arena);
        // the products of a few rows can read it where it is
        const bool others = ((want_w || recompute) && K % 8 != 0) || act == PGEMM_ACT_NONE;
        const bool in_place = M <= kTokensMax && (!want_x || x_tokens) && (!recompute || tokens) &&
                              (want_x ? op_raw_us(dev, M, K, N, false, true) : 0.0) +
                                      (recompute ? op_raw_us(dev, M, N, K, false, false) : 0.0) <=
                                  op_relayout_us(K, N, others);
        if (in_place)
            w = OpMat{W, N};
        else if (want_x || recompute)  // (else W may be absent)
            rl.add(&w, W, K, N, arena);
    }
    const bool own_dz = some && act != PGEMM_ACT_NONE;  // dZ is not dY itself
    long long dz_at = 0;
    if (own_dz) {
        dz.ld = op_round_up(N, 64);
        dz_at = arena.add(dz.ld * M * 2);
    } else if (some && (want_x || want_w)) {  // (the column sums read dY itself)
        rl.add(&dz, dY, M, N, arena);
    }
    OpProduct px, pw;
    if (want_x && !x_tokens) {
        px.form = OpForm::NT;
        px.M = M;
        px.N = K;
        px.K = N;
        px.out[0] = dX;
        op_product_plan(dev, px, arena);
    }
    if (want_w) {
        pw.form = OpForm::TN;
        pw.M = K;
        pw.N = N;
        pw.K = M;
        pw.out[0] = dW;
        op_product_plan(dev, pw, arena);
    }
    OpActGrad g;
    const bool elementwise = own_dz && preact;
    if (some) {
        g.M = M;
        g.N = N;
        g.dbias = want_b ? dbias : nullptr;
        op_act_grad_plan(g, arena);
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;

    // dZ first: from the kept Z elementwise, with the column sums beside it, or
    // by the product that recomputes Z; then the products and column sums that
    // read it, which overlap one another; then what joins their parts.
    if (own_dz) {
        uint16_t *dz_buf = arena.at<uint16_t>(dz_at);
        dz.p = dz_buf;
        if (elementwise) {
            g.act = act;
            g.z = preact;
            g.dy = dY;
            g.dy_ld = N;
            g.dz = dz_buf;
            g.dz_ld = dz.ld;
            st = op_act_grad(dev, g, arena, false, s);
        } else if (tokens) {
            st = op_tokens_linear_grad(dev, M, N, K, x, w, bias, act, dY, dz_buf, dz.ld, s);
        } else {
            const EpiLinearGrad e{bias, dY, N, dz_buf, dz.ld, act};
            const bool pair = op_use_pair(dev, M, N, K, 256, 128);
            if (op_sign_rounds(act, K))
                st = pair ? launch_grad<OpCfg<256, 3, 2, 2, false, false, false, SignPair::value>>(
                                dev, M, N, K, x, w, e, s)
                          : launch_grad<OpCfg<128, 6, 1, 1, false, false, false, SignOne::value>>(
                                dev, M, N, K, x, w, e, s);
            else
                st = pair ? launch_grad<OpCfg<256, 3, 2, 2, false, false>>(dev, M, N, K, x, w, e, s)
                          : launch_grad<OpCfg<128, 6, 1, 1, false, false>>(dev, M, N, K, x, w, e, s);
        }
        if (st != PGEMM_OK) return st;
    }
    bool overlap = false;  // the first kernel that reads dZ waits for it
    if (want_x) {
        px.A[0] = dz;
        px.B[0] = w;
        st = x_tokens ? op_tokens_transposed(dev, M, K, N, px.A, px.B, 1, dX, s)
                      : op_product(dev, px, arena, s);
        if (st != PGEMM_OK) return st;
        overlap = true;
    }
    if (want_w) {
        pw.A[0] = x;
        pw.B[0] = dz;
        pw.overlap = overlap;
        if ((st = op_product(dev, pw, arena, s)) != PGEMM_OK) return st;
        overlap = true;
    }
    if (some && want_b && !elementwise) {
        g.dy = own_dz ? dz.p : dY;
        g.dy_ld = own_dz ? dz.ld : N;
        if ((st = op_act_grad(dev, g, arena, overlap, s)) != PGEMM_OK) return st;
        overlap = false;
    }
    if (some && (st = op_act_grad_join(dev, g, arena, overlap, s)) != PGEMM_OK) return st;
    if ((st = op_product_join(dev, px, arena, s)) != PGEMM_OK) return st;
    return op_product_join(dev, pw, arena, s);
}

}  // namespace pg

extern "C" {

pgemm_status linear_bf16(int M, int N, int K, const uint16_t *X, const uint16_t *W,
                         const uint16_t *bias, int act, const uint16_t *residual, uint16_t *Y,
                         float *preact, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::linear_forward(M, N, K, X, W, bias, act, residual, Y, preact, stream);
    });
}

pgemm_status linear_bf16_backward(int M, int N, int K, const uint16_t *X, const uint16_t *W,
                                  const uint16_t *bias, int act, const uint16_t *dY,
                                  const float *preact, uint16_t *dX, uint16_t *dW,
                                  uint16_t *dbias, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::linear_backward(M, N, K, X, W, bias, act, dY, preact, dX, dW, dbias, stream);
    });
}

}  // extern "C"
