// gated_bf16: H = act(X Wg) * (X Wu), and its gradients.
//
// Both projections run as one product: the left half of the accumulator is
// X Wg, the right half X Wu for the same columns, so X is read once and an
// epilogue thread holds both values of every element it writes: H costs one pass of
// the tensor core over X, and nothing goes to memory between the projections and
// the product.  Tensor-bound: 4096 x 16384 x 4096 624 us, one call after another
// (1.76 PFLOP/s, above the 1.69 that plain products sustain under the power cap).
#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

struct EpiGated {
    uint16_t *h;
    float *preact;  // [2][M][F]: X Wg, X Wu; or nullptr
    long long ld;   // F
    int act;
    int tma_h, tma_preact;

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        int col0, width;
        const bool mine = epi_cols_dual<Cfg>(w, e, col0, width);
        if (!mine) return acc.skip();
        const int n0 = w.n0 + col0;
        uint32_t g[2][32], u[2][32], p[32];
        if constexpr (Cfg::ROUND > 0) {
            float x[64], y[64];
            if (!acc_sum<64, 64>(acc, col0, x, width + col0, y)) return false;
#pragma unroll
            for (int j = 0; j < 64; ++j) {
                g[j / 32][j % 32] = __float_as_uint(x[j]);
                u[j / 32][j % 32] = __float_as_uint(y[j]);
            }
        } else {
            if (!acc.wait()) return false;
            const uint32_t t_row = acc.row() + col0;
            if (acc.have()) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    tmem_ld_32x32b_x32(t_row + 32 * k, g[k]);
                    tmem_ld_32x32b_x32(t_row + width + 32 * k, u[k]);
                }
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) g[0][j] = g[1][j] = u[0][j] = u[1][j] = 0u;
            }
            acc.release();
        }
        if (preact != nullptr) {
            const CUtensorMap *mg = tma_preact ? &maps.c[1] : nullptr;
            const CUtensorMap *mu = tma_preact ? &maps.c[2] : nullptr;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                put_words16(c, mg, preact, ld, c.m0, n0 + 16 * k, g[k / 2] + 16 * (k % 2));
                put_words16(c, mu, preact + ld * c.M, ld, c.m0, n0 + 16 * k,
                            u[k / 2] + 16 * (k % 2));
            }
        }
        auto combine = [&](auto A) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    p[16 * k + j] = pack_bf16(
                        act_value<decltype(A)::value>(__uint_as_float(g[k][2 * j])) *
                            __uint_as_float(u[k][2 * j]),
                        act_value<decltype(A)::value>(__uint_as_float(g[k][2 * j + 1])) *
                            __uint_as_float(u[k][2 * j + 1]));
        };
        if constexpr (Cfg::ROUND > 0)
            combine(std::integral_constant<int, PGEMM_ACT_RELU>{});
        else
            with_act(act, combine);
        if (tma_h) {
            put_rows32_batch<2>(c, &maps.c[0], n0, p);
        } else {
            put_rows32(c, nullptr, h, ld, n0, p);
            put_rows32(c, nullptr, h, ld, n0 + 32, p + 16);
        }
        return true;
    }
};

// Epilogue of the recomputing backward pass: dG = dH * U * act'(G),
// dU = dH * act(G) from fp32 G and U, each rounded to bf16 once as an operand
// of the gradient products.
struct EpiGatedGrad {
    const uint16_t *dh;
    long long ld;  // F
    uint16_t *dg, *du;
    long long dz_ld;
    int act;

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        int col0, width;
        const bool mine = epi_cols_dual<Cfg>(w, e, col0, width);
        if (!mine) return acc.skip();
        RowsIn in{dh, ld};
        if (Cfg::ROUND == 0) in.load(c, w.n0 + col0);  // travels while the products finish
        // 32 columns from w.n0 + col0 + 32 k
        auto finish = [&](int k, const uint32_t *g, const uint32_t *u) {
            const int n = w.n0 + col0 + 32 * k;
            uint32_t r[16], p[16], q[16];
            in.take(c, r);
            if (k == 0) in.load(c, n + 32);
            auto derive = [&](auto A) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float y0 = bf16_lo(r[j]), y1 = bf16_hi(r[j]);
                    float a0, a1;
                    const float d0 =
                        act_value_grad<decltype(A)::value>(__uint_as_float(g[2 * j]), a0);
                    const float d1 =
                        act_value_grad<decltype(A)::value>(__uint_as_float(g[2 * j + 1]), a1);
                    p[j] = pack_bf16(y0 * d0 * __uint_as_float(u[2 * j]),
                                     y1 * d1 * __uint_as_float(u[2 * j + 1]));
                    q[j] = pack_bf16(y0 * a0, y1 * a1);
                }
            };
            if constexpr (Cfg::ROUND > 0)
                derive(std::integral_constant<int, PGEMM_ACT_RELU>{});
            else
                with_act(act, derive);
            put_rows32(c, &maps.c[0], dg, dz_ld, n, p);
            put_rows32(c, &maps.c[1], du, dz_ld, n, q);
        };
        if constexpr (Cfg::ROUND > 0) {
            float x[64], y[64];
            if (!acc_sum<64, 64>(acc, col0, x, width + col0, y)) return false;
            in.load(c, w.n0 + col0);  // (the sums fill the registers until here)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t g[32], u[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    g[j] = __float_as_uint(x[32 * k + j]);
                    u[j] = __float_as_uint(y[32 * k + j]);
                }
                finish(k, g, u);
            }
            return true;
        }
        const bool have = acc.have();
        if (!acc.wait()) return false;
        const uint32_t t_row = acc.row() + col0;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            uint32_t g[32], u[32];
            acc_cols32(t_row + 32 * k, have, g);
            acc_cols32(t_row + width + 32 * k, have, u);
            if (k == 1) acc.release();
            finish(k, g, u);
        }
        return true;
    }
};

template <class Cfg, class Epi>
static pgemm_status launch_dual(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                                const OpMat &Wg, const OpMat &Wu, OpMaps &maps, const Epi &e,
                                cudaStream_t s) {
    if (K > 0) {
        pgemm_status st = op_encode(&maps.a[0], X.p, K, M, X.ld, 128);
        if (st == PGEMM_OK) st = op_encode(&maps.b[0], Wg.p, F, K, Wg.ld, 64);
        if (st == PGEMM_OK) st = op_encode(&maps.b[1], Wu.p, F, K, Wu.ld, 64);
        if (st != PGEMM_OK) return st;
    }
    constexpr int TM = Cfg::BM * Cfg::CG;
    OpArgs a{};
    a.M = M;
    a.N = F;
    a.K = K;
    a.m_tiles = op_blocks(M, TM);
    a.n_seg = a.n_tiles = op_blocks(F, Cfg::TILE_N);
    a.k_seg = a.k_tiles = op_blocks(K, Cfg::SBK);
    a.parts = 1;
    return op_launch<Cfg, Epi>(dev, maps, a, e, s);
}

using DualPair = OpCfg<256, 3, 2, 2, false, false, true>;
using DualOne = OpCfg<128, 6, 1, 1, false, false, true>;

using SignDualPair = OpCfg<256, 3, 2, 2, false, false, true, SignPair::value>;
using SignDualOne = OpCfg<128, 6, 1, 1, false, false, true, SignOne::value>;

// sign: the epilogue decides a ReLU's derivative, or keeps what will.
template <class Epi>
static pgemm_status launch_dual_size(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                                     const OpMat &Wg, const OpMat &Wu, OpMaps &maps, const Epi &e,
                                     bool sign, cudaStream_t s) {
    const bool pair = op_use_pair(dev, M, F, K, 128, 64);
    if (sign && op_sign_rounds(e.act, K))
        return pair ? launch_dual<SignDualPair>(dev, M, F, K, X, Wg, Wu, maps, e, s)
                    : launch_dual<SignDualOne>(dev, M, F, K, X, Wg, Wu, maps, e, s);
    return pair ? launch_dual<DualPair>(dev, M, F, K, X, Wg, Wu, maps, e, s)
                : launch_dual<DualOne>(dev, M, F, K, X, Wg, Wu, maps, e, s);
}

static pgemm_status gated_forward(int M, int F, int K, const uint16_t *X, const uint16_t *Wg,
                                  const uint16_t *Wu, int act, uint16_t *H, float *preact,
                                  cudaStream_t s) {
    if (M < 0 || F < 0 || K < 0 || !op_act_known(act)) return PGEMM_ERR_INVALID_VALUE;
    if (M == 0 || F == 0) return PGEMM_OK;
    if (!H || (K > 0 && (!X || !Wg || !Wu))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(Wg) || !op_aligned16(Wu) || !op_aligned16(H) ||
        !op_aligned16(preact))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    // (what may decide a ReLU's derivative goes in rounds, op_sign_rounds)
    const bool tokens =
        M <= kTokensMax || (!op_sign_rounds(act, K) && op_tokens_gated_fit(dev, M, F, K));
    OpArena arena(dev, s);
    OpRelayout rl;
    OpMat x, wg, wu;
    if (K > 0) {
        rl.add(&x, X, M, K, arena);
        if (M <= kTokensMax && op_raw_us(dev, M, F, K, true, false) <=
                          op_relayout_us(2ll * K, F, K % 8 != 0)) {
            wg = OpMat{Wg, F};  // read where they are, whatever their pitch
            wu = OpMat{Wu, F};
        } else {
            rl.add(&wg, Wg, K, F, arena);
            rl.add(&wu, Wu, K, F, arena);
        }
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    if (tokens) return op_tokens_gated(dev, M, F, K, x, wg, wu, act, H, preact, s);
    OpMaps maps{};
    EpiGated e{H, preact, F, act, F % 8 == 0, preact != nullptr && F % 4 == 0};
    if (e.tma_h) st = op_encode_out(&maps.c[0], OpElem::BF16, H, F, M, F);
    if (e.tma_preact) {
        if (st == PGEMM_OK) st = op_encode_out(&maps.c[1], OpElem::F32, preact, F, M, F);
        if (st == PGEMM_OK)
            st = op_encode_out(&maps.c[2], OpElem::F32, preact + static_cast<long long>(M) * F, F,
                               M, F);
    }
    if (st != PGEMM_OK) return st;
    return launch_dual_size(dev, M, F, K, x, wg, wu, maps, e, preact != nullptr, s);
}

static pgemm_status gated_backward(int M, int F, int K, const uint16_t *X, const uint16_t *Wg,
                                   const uint16_t *Wu, int act, const uint16_t *dH,
                                   const float *preact, uint16_t *dX, uint16_t *dWg,
                                   uint16_t *dWu, cudaStream_t s) {
    if (M < 0 || F < 0 || K < 0 || !op_act_known(act)) return PGEMM_ERR_INVALID_VALUE;
    if ((dWg == nullptr) != (dWu == nullptr)) return PGEMM_ERR_INVALID_VALUE;
    const bool want_x = dX && M > 0 && K > 0, want_w = dWg && K > 0 && F > 0;
    if (!want_x && !want_w) return PGEMM_OK;  // K > 0 from here on
    const bool some = M > 0 && F > 0;
    // what some kernel of this call reads; the rest may be absent
    const bool need_x = want_w || !preact, need_w = want_x || !preact;
    if (some && (!dH || (need_x && !X) || (need_w && (!Wg || !Wu))))
        return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(Wg) || !op_aligned16(Wu) || !op_aligned16(dH) ||
        !op_aligned16(preact) || !op_aligned16(dX) || !op_aligned16(dWg) || !op_aligned16(dWu))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    OpArena arena(dev, s);
    OpRelayout rl;
    const bool x_tokens = want_x && op_tokens_fit(dev, M, K, 2ll * F);
    const bool tokens = M <= kTokensMax || (!preact && !op_sign_rounds(act, K) &&
                                            op_tokens_gated_fit(dev, M, F, K));
    OpMat x, wg, wu, dg, du;
    long long dg_at = 0, du_at = 0;
    if (some) {
        if (need_x) rl.add(&x, X, M, K, arena);
        // the products of a few rows can read them where they are
        const bool in_place = M <= kTokensMax && (!want_x || x_tokens) && (preact || tokens) &&
                              (want_x ? op_raw_us(dev, M, K, 2ll * F, false, true) : 0.0) +
                                      (preact ? 0.0 : op_raw_us(dev, M, F, K, true, false)) <=
                                  op_relayout_us(2ll * K, F, K % 8 != 0);
        if (in_place) {
            wg = OpMat{Wg, F};
            wu = OpMat{Wu, F};
        } else if (need_w) {
            rl.add(&wg, Wg, K, F, arena);
            rl.add(&wu, Wu, K, F, arena);
        }
        dg.ld = du.ld = op_round_up(F, 64);
        dg_at = arena.add(dg.ld * M * 2);
        du_at = arena.add(du.ld * M * 2);
    }
    OpProduct px, pw;
    if (want_x && !x_tokens) {
        px.form = OpForm::NT;
        px.M = M;
        px.N = K;
        px.K = F;
        px.k_segments = 2;
        px.out[0] = dX;
        op_product_plan(dev, px, arena);
    }
    if (want_w) {
        pw.form = OpForm::TN;
        pw.M = K;
        pw.N = F;
        pw.K = M;
        pw.n_segments = 2;
        pw.out[0] = dWg;
        pw.out[1] = dWu;
        op_product_plan(dev, pw, arena);
    }
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    if ((st = rl.run(dev, arena, s)) != PGEMM_OK) return st;
    if (some) {
        uint16_t *dg_buf = arena.at<uint16_t>(dg_at), *du_buf = arena.at<uint16_t>(du_at);
        dg.p = dg_buf;
        du.p = du_buf;
        if (preact) {
            OpActGrad g;
            g.M = M;
            g.N = F;
            g.act = act;
            g.z = preact;
            g.u = preact + static_cast<long long>(M) * F;
            g.dy = dH;
            g.dy_ld = F;
            g.dz = dg_buf;
            g.du = du_buf;
            g.dz_ld = dg.ld;
            st = op_act_grad(dev, g, arena, false, s);
        } else if (tokens) {
            st = op_tokens_gated_grad(dev, M, F, K, x, wg, wu, act, dH, dg_buf, du_buf, dg.ld, s);
        } else {
            OpMaps maps{};
            EpiGatedGrad e{dH, F, dg_buf, du_buf, dg.ld, act};
            st = op_encode_out(&maps.c[0], OpElem::BF16, dg_buf, F, M, dg.ld);
            if (st == PGEMM_OK)
                st = op_encode_out(&maps.c[1], OpElem::BF16, du_buf, F, M, du.ld);
            if (st == PGEMM_OK)
                st = launch_dual_size(dev, M, F, K, x, wg, wu, maps, e, true, s);
        }
        if (st != PGEMM_OK) return st;
    }
    if (want_x) {
        px.A[0] = dg;
        px.A[1] = du;
        px.B[0] = wg;
        px.B[1] = wu;
        st = x_tokens ? op_tokens_transposed(dev, M, K, F, px.A, px.B, 2, dX, s)
                      : op_product(dev, px, arena, s);
        if (st != PGEMM_OK) return st;
    }
    if (want_w) {
        pw.A[0] = x;
        pw.B[0] = dg;
        pw.B[1] = du;
        pw.overlap = want_x;  // behind dX, which has waited for dG and dU
        if ((st = op_product(dev, pw, arena, s)) != PGEMM_OK) return st;
    }
    if ((st = op_product_join(dev, px, arena, s)) != PGEMM_OK) return st;
    return op_product_join(dev, pw, arena, s);
}

}  // namespace pg

extern "C" {

pgemm_status gated_bf16(int M, int F, int K, const uint16_t *X, const uint16_t *Wg,
                        const uint16_t *Wu, int act, uint16_t *H, float *preact,
                        pgemm_stream_t stream) {
    return pg::op_guard(
        [&] { return pg::gated_forward(M, F, K, X, Wg, Wu, act, H, preact, stream); });
}

pgemm_status gated_bf16_backward(int M, int F, int K, const uint16_t *X, const uint16_t *Wg,
                                 const uint16_t *Wu, int act, const uint16_t *dH,
                                 const float *preact, uint16_t *dX, uint16_t *dWg, uint16_t *dWu,
                                 pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::gated_backward(M, F, K, X, Wg, Wu, act, dH, preact, dX, dWg, dWu, stream);
    });
}

}  // extern "C"
