// Host-side services shared by the operators' dispatch (op_*.cu): the device
// set-up and scratch pool of the library, tensor maps, operand relayout and
// the generic product with its split-K join.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "pgemm.h"

namespace pg {

// The current device as the operators need it (api.cu sets it up once).
struct OpDevice {
    int sm_count = 0;
    KernelCtx ctx{};
    cudaMemPool_t pool = nullptr;
    void *state = nullptr;  // the library's record of the device
};

pgemm_status op_device(OpDevice *out);  // the current device, set up
// One-time set-up of a kernel (shared-memory attributes, schedule slots).
pgemm_status op_kernel_setup(const OpDevice &dev, const KernelInfo &k, int *slots);
// A 2-D tensor map of 16- or 32-bit elements: `inner` x `outer` with row pitch
// `ld` (elements).  op_encode: an operand, boxes of 64 columns x box_y rows with
// the 128-byte swizzle.  op_encode_out: an output, boxes of 64 bytes x 32 rows
// with the 64-byte swizzle of the epilogues' staging buffers.
pgemm_status op_encode(CUtensorMap *map, const void *base, long long inner, long long outer,
                       long long ld, int box_y);
enum class OpElem { BF16, F32 };
pgemm_status op_encode_out(CUtensorMap *map, OpElem type, const void *base, long long inner,
                           long long outer, long long ld);
cudaError_t launch_repack(const void *src0, long long sld0, void *dst0, long long dld0, int rows0,
                          int cols0, const void *src1, long long sld1, void *dst1, long long dld1,
                          int rows1, int cols1, int eb, int sm_count, cudaStream_t s);

inline long long op_round_up(long long v, long long m) { return (v + m - 1) / m * m; }
// ceil(v / m): v up to 2^31 - 1 would overflow in 32 bits
inline int op_blocks(long long v, long long m) { return static_cast<int>((v + m - 1) / m); }
inline bool op_act_known(int act) { return act >= PGEMM_ACT_NONE && act <= PGEMM_ACT_SILU; }
inline bool op_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Stream-ordered scratch of one call: sizes are added first, allocated in one
// piece from the library's pool, and given back on the stream when the call
// returns.
class OpArena {
  public:
    explicit OpArena(const OpDevice &d, cudaStream_t s) : dev_(d), stream_(s) {}
    OpArena(const OpArena &) = delete;
    OpArena &operator=(const OpArena &) = delete;
    ~OpArena() {
        if (base_) cudaFreeAsync(base_, stream_);
    }
    // bytes rounded up so that every part starts on a 1024-byte boundary
    long long add(long long bytes) {
        const long long at = total_;
        total_ += op_round_up(bytes > 0 ? bytes : 0, 1024);
        return at;
    }
    pgemm_status alloc() {
        if (total_ == 0) return PGEMM_OK;
        return cudaMallocFromPoolAsync(&base_, static_cast<size_t>(total_), dev_.pool, stream_) ==
                       cudaSuccess
                   ? PGEMM_OK
                   : PGEMM_ERR_CUDA;
    }
    template <class T>
    T *at(long long offset) const {
        return reinterpret_cast<T *>(static_cast<uint8_t *>(base_) + offset);
    }

  private:
    const OpDevice &dev_;
    cudaStream_t stream_;
    void *base_ = nullptr;
    long long total_ = 0;
};

// A bf16 matrix as a product reads it: rows x cols, pitch ld (elements), rows
// on 16-byte boundaries.
struct OpMat {
    const uint16_t *p = nullptr;
    long long ld = 0;
};

// Makes caller matrices (contiguous rows) readable by TMA: a matrix whose rows
// are not multiples of 16 bytes is copied to a 128-byte pitch.  plan() says
// where, run() launches the copies (two matrices a launch) and fills in `out`.
class OpRelayout {
  public:
    void add(OpMat *out, const uint16_t *src, long long rows, long long cols, OpArena &arena) {
        out->p = src;
        out->ld = cols;
        if (cols % 8 == 0 || rows == 0 || cols == 0) return;
        Job &j = jobs_[n_++];
        j = Job{out, src, rows, cols, op_round_up(cols, 64), 0};
        j.at = arena.add(j.rows * j.ld * 2);
    }
    pgemm_status run(const OpDevice &dev, OpArena &arena, cudaStream_t s);

  private:
    struct Job {
        OpMat *out;
        const uint16_t *src;
        long long rows, cols, ld, at;
    };
    Job jobs_[6];
    int n_ = 0;
};

// How the two operands of a product lie in memory (A is M x K, B is K x N).
enum class OpForm {
    NN,  // A rows of K, B rows of N
    NT,  // A rows of K, B stored N x K
    TN,  // A stored K x M, B rows of N
};

// The epilogue of a product with bf16 output (EpiOut, op_products.cu).
struct OpEpilogue {
    const uint16_t *bias = nullptr;      // N
    int act = PGEMM_ACT_NONE;
    const uint16_t *residual = nullptr;  // M x N, rows of N
    float *preact = nullptr;             // M x N fp32, rows of N: acc + bias
    const float *scale = nullptr;        // one value on the device that multiplies acc
};

// out[j] (bf16, rows of N) = epilogue(sum over K segments of A * B).
//   k_segments = 2: out[0] = A[0] B[0] + A[1] B[1] (both K columns each)
//   n_segments = 2: out[j] = A[0] B[j]
// Outputs are user matrices: any N; TMA stores where rows are 16-byte
// multiples.  Few tiles with a long K are split along K into parts whose fp32
// sums are joined in part order by a second kernel.
struct OpPlan {
    bool pair;
    int parts;
};
struct OpProduct {
    OpForm form = OpForm::NN;
    int M = 0, N = 0, K = 0;
    OpMat A[2], B[2];
    uint16_t *out[2] = {nullptr, nullptr};
    int k_segments = 1, n_segments = 1;
    OpEpilogue epi;
    // a caller's own area of fp32 parts instead (cross entropy sums the pieces
    // of its vocabulary there): the parts are written, nothing is joined
    float *parts_area = nullptr;
    // behind another kernel that this product does not depend on (op_begin)
    bool overlap = false;
    OpPlan plan{};           // op_product_plan's
    long long area_at = -1;  // the parts' place in the arena, if it is split
};
// In this order: choose the tiles and parts and reserve what the parts need in
// the call's arena; launch; join the parts, if any.
void op_product_plan(const OpDevice &dev, OpProduct &p, OpArena &arena);
pgemm_status op_product(const OpDevice &dev, const OpProduct &p, const OpArena &arena,
                        cudaStream_t s);
pgemm_status op_product_join(const OpDevice &dev, const OpProduct &p, const OpArena &arena,
                             cudaStream_t s);

// The same products of a few rows, bound by reading the weights, and of more rows whose
// tiles are too few for the GPU (op_tokens.cu).
constexpr int kTokensMax = 128;
// Whether a gradient product of M rows (N outputs, K reduction columns) goes that
// way.  A cluster shares a tile's K among eight CTAs at most, so few columns with a
// long K leave most SMs idle, where the tiled product takes up to 32 parts (a whole
// cross-entropy gradient, streaming against tiled dX: 4 tokens x 82768 x 592
// 117 against 95 us, 16 x 15640 x 520 35 against 39).
// With more rows: where that is quicker than the tiled product.
bool op_tokens_fit(const OpDevice &dev, int M, long long N, long long K);
bool op_tokens_gated_fit(const OpDevice &dev, int M, int F, int K);
// What weights whose rows TMA cannot read cost those products beyond others (N
// outputs, K reduction columns), and what copying a matrix to another pitch costs
// instead (`others`: in a launch that is needed anyway): us, estimates that choose
// between the two.
double op_raw_us(const OpDevice &dev, int M, long long N, long long K, bool dual,
                 bool transposed);
inline double op_relayout_us(long long rows, long long cols, bool others) {
    return (others ? 1.8 : 3.5) + static_cast<double>(rows) * static_cast<double>(cols) * 4 / 7.5e6;
}
pgemm_status op_tokens_linear(const OpDevice &dev, int M, int N, int K, const OpMat &X,
                              const OpMat &W, const OpEpilogue &e, uint16_t *Y, cudaStream_t s);
pgemm_status op_tokens_gated(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                             const OpMat &Wg, const OpMat &Wu, int act, uint16_t *H,
                             float *preact, cudaStream_t s);
// dZ = dY act'(X W + b); dG and dU of a gated block (rows of dz_ld elements).
pgemm_status op_tokens_linear_grad(const OpDevice &dev, int M, int N, int K, const OpMat &X,
                                   const OpMat &W, const uint16_t *bias, int act,
                                   const uint16_t *dy, uint16_t *dz, long long dz_ld,
                                   cudaStream_t s);
pgemm_status op_tokens_gated_grad(const OpDevice &dev, int M, int F, int K, const OpMat &X,
                                  const OpMat &Wg, const OpMat &Wu, int act, const uint16_t *dh,
                                  uint16_t *dg, uint16_t *du, long long dz_ld, cudaStream_t s);
// out (M x N) = the sum over segments of X[j] W[j]^T, X M x K, W N x K.
pgemm_status op_tokens_transposed(const OpDevice &dev, int M, int N, int K, const OpMat *X,
                                  const OpMat *W, int segments, uint16_t *out, cudaStream_t s);

// What a product takes by the estimate that chooses its tiles and parts, us; the same for
// a gated product (F columns of both).
double op_product_us(const OpDevice &dev, long long M, long long N, long long K);
double op_gated_us(const OpDevice &dev, long long M, long long F, long long K);
// Parts a product of these sizes would be split into (parts_area: M padded to
// 32 rows, N to 64 columns, one such matrix a part and segment).
int op_product_parts(const OpDevice &dev, int M, int N, int K, int segments);
long long op_parts_ld(int N);
long long op_parts_rows(int M);
// out = epilogue(sum of `parts` matrices), in order.
pgemm_status op_join_parts(const OpDevice &dev, const float *area, int parts, int segments, int M,
                           int N, uint16_t *const out[2], const OpEpilogue &epi,
                           cudaStream_t s);
// The first of `parts` such matrices <- their sum, in order.
pgemm_status op_fold_parts(const OpDevice &dev, float *area, int parts, int M, int N,
                           cudaStream_t s);

// The larger tile on a CTA pair (256 x pair_n outputs), or one CTA's (128 x
// one_n): whichever needs less time for an M x N x K product (op_products.cu).
bool op_use_pair(const OpDevice &dev, long long M, long long N, long long K, long long pair_n,
                 long long one_n);

// dZ = dY * act'(Z) from kept fp32 pre-activations, and column sums of dZ
// (act none and dz nullptr: of dY itself).  op_products.cu.
struct OpActGrad {
    int M = 0, N = 0, act = PGEMM_ACT_NONE;
    const float *z = nullptr;        // M x N, rows of N; nullptr only with act none
    const float *u = nullptr;        // gated: the value projection
    const uint16_t *dy = nullptr;    // M x N, rows of dy_ld
    long long dy_ld = 0;
    uint16_t *dz = nullptr;          // rows of dz_ld, or nullptr
    uint16_t *du = nullptr;          // gated
    long long dz_ld = 0;
    uint16_t *dbias = nullptr;       // N, or nullptr
    long long colsum_at = 0;         // op_act_grad_plan's
};
// Reserve the partial column sums; the elementwise pass; their sum into dbias.
void op_act_grad_plan(OpActGrad &g, OpArena &arena);
pgemm_status op_act_grad(const OpDevice &dev, const OpActGrad &g, const OpArena &arena,
                         bool overlap, cudaStream_t s);
pgemm_status op_act_grad_join(const OpDevice &dev, const OpActGrad &g, const OpArena &arena,
                              bool overlap, cudaStream_t s);

// A C entry point's body: no C++ exception leaves it.
template <class F>
pgemm_status op_guard(F &&f) {
    try {
        return f();
    } catch (...) {
        return PGEMM_ERR_CUDA;
    }
}

}  // namespace pg
