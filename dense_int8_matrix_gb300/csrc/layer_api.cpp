// C entry points of the bfloat16 layer's operators: argument checks, plans,
// dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "checks.h"
#include "context.h"
#include "internal.h"
#include "layer.h"

using namespace gemm;

namespace {

// Scratch from the library's pool for one call, returned on the same stream.
class Scratch {
  public:
    Scratch(cudaMemPool_t pool, cudaStream_t stream) : pool_(pool), stream_(stream) {}
    ~Scratch() {
        if (ptr_) cudaFreeAsync(ptr_, stream_);
    }
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    void* take(int64_t bytes) {   // once per call; nullptr if there is none
        if (cudaMallocFromPoolAsync(&ptr_, static_cast<size_t>(bytes), pool_, stream_) != cudaSuccess) ptr_ = nullptr;
        return ptr_;
    }

  private:
    cudaMemPool_t pool_;
    cudaStream_t stream_;
    void* ptr_ = nullptr;
};

bool act_ok(int32_t act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU; }

// ---- products ------------------------------------------------------------------
gemm_status check_linear_shape(int32_t form, int64_t m, int64_t k, int64_t n) {
    if (form < GEMM_FORM_NT || form > GEMM_FORM_TN) return GEMM_ERR_INVALID_ARG;
    return dim_ok(m) && dim_ok(k) && dim_ok(n) ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

// Estimated microseconds of a product on the small tiles: `tiles` of bm rows by
// 128 columns, `steps` K steps of 64, `split` CTAs to a tile; on the two-SM tiles
// in the function below.  The constants were fitted to the times of every
// configuration on 220 drawn products of all forms on GB300 (152 SMs): a step, what a round of
// CTAs costs besides, the epilogue (on small tiles 1.3 times as long for rows of D
// that are no whole vectors: `odd`; the two-SM tiles' takes no longer), and the join of a split.  Two CTAs share an SM below 64 rows and
// then take 2.5 times as long; clusters of four and eight cannot use every SM.
double small_time(double tiles, int64_t steps, int bm, int split, bool odd, int num_sms) {
    const double step = bm == 16 ? 0.24 : bm == 32 ? 0.26 : bm == 64 ? 0.25 : 0.36;
    const double epilogue = bm == 16 ? 0.13 : bm == 32 ? 0.47 : (bm == 64 ? 1.0 : 1.5) * (odd ? 1.3 : 1.0);
    const double part = bm < 64 ? (split == 8 ? 1.68 : split == 4 ? 1.86 : 2.0) : split == 8 ? 0.79 : split == 4 ? 0.84 : 1.0;
    const double ctas = tiles * split, room = std::max(1.0, std::floor(part * num_sms));
    const double share = bm < 64 && ctas > num_sms ? 2.5 : 1.0;
    return 2.5 + std::ceil(ctas / room) * ((bm < 64 ? 1.65 : 0.7) + step * share * static_cast<double>(ceil_div(steps, split)) + epilogue) +
           (split > 1 ? 0.75 + 2.4 * bm / 128 : 0.0);
}
// A tile's epilogue runs beside the next tile's products; a last round that
// fills at most half of the pairs runs as halves.
double pair_time(double tiles, int64_t steps, int num_sms) {
    const double pairs = std::max(1, num_sms / 2), epilogue = 4.3, k = static_cast<double>(steps);
    const double whole = 0.6 + 0.46 * k, half = 0.56 + 0.38 * k;
    const double rounds = std::floor(tiles / pairs), left = tiles - rounds * pairs;
    double t = 2.9 + (rounds > 0 ? whole + (rounds - 1) * std::max(whole, epilogue) : 0.0);
    if (left == 0) return t + epilogue;
    const double last = 2 * left > pairs ? whole : half;
    t += rounds > 0 ? std::max(last, epilogue) : last;
    return t + (2 * left > pairs ? epilogue : epilogue / 2);
}

// The tile and split of a product: the least estimate.  On 870 other products, with
// the kernels as they are, the choice takes 1.4 % longer than the best
// configuration of each (the worst by 33 %).  It sees the form and the sizes, not
// the activation.
void choose_linear(gemm_plan_linear* p) {
    const int64_t steps = ceil_div(p->k, 64);
    const bool odd = p->n % 8 != 0;
    p->path = GEMM_PATH_TENSOR;
    p->bm = p->bn = 256;
    p->split_k = 1;
    double best = pair_time(static_cast<double>(ceil_div(p->m, 256)) * static_cast<double>(ceil_div(p->n, 256)), steps, p->num_sms);
    for (int bm = p->form == GEMM_FORM_TN ? 64 : 16; bm <= 128; bm *= 2) {
        if ((bm < 128 && p->m > 8 * bm) || (bm > 16 && bm >= 4 * p->m)) continue;
        const double tiles = static_cast<double>(ceil_div(p->m, bm)) * static_cast<double>(ceil_div(p->n, 128));
        if (8 * tiles > INT32_MAX) continue;
        for (int s = 1; s <= 8 && s <= steps; s *= 2) {
            const double t = small_time(tiles, steps, bm, s, odd, p->num_sms);
            if (t >= best) continue;
            best = t;
            p->path = GEMM_PATH_SKINNY;
            p->bm = bm;
            p->bn = 128;
            p->split_k = s;
        }
    }
}

gemm_status make_linear_plan(int32_t form, int64_t m, int64_t k, int64_t n, int32_t num_sms, gemm_plan_linear* out) {
    if (!out || num_sms < 1) return GEMM_ERR_INVALID_ARG;
    const gemm_status st = check_linear_shape(form, m, k, n);
    if (st != GEMM_OK) return st;
    std::memset(out, 0, sizeof(*out));
    out->version = GEMM_PLAN_LINEAR_VERSION;
    out->num_sms = num_sms;
    out->form = form;
    out->m = m;
    out->k = k;
    out->n = n;
    choose_linear(out);
    return GEMM_OK;
}

bool linear_config_ok(const gemm_plan_linear* p) {
    if (p->path == GEMM_PATH_TENSOR) return p->bm == 256 && (p->bn == 128 || p->bn == 256) && p->split_k == 1;
    const int bm = p->bm, s = p->split_k;
    return p->path == GEMM_PATH_SKINNY && (bm == 64 || bm == 128 || (p->form != GEMM_FORM_TN && (bm == 16 || bm == 32))) &&
           p->bn == 128 && (s == 1 || s == 2 || s == 4 || s == 8);
}

// A matrix that TMA can read as it lies.
bool tma_rows(const void* p, int64_t ld) { return al(p, 16) && ld % 8 == 0; }

}  // namespace

extern "C" {

gemm_status gemm_bf16_linear_plan(int32_t form, int64_t m, int64_t k, int64_t n, gemm_plan_linear* out) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_linear_shape(form, m, k, n);
    if (st != GEMM_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != GEMM_OK) return st;
    return make_linear_plan(form, m, k, n, sms, out);
}

gemm_status gemm_bf16_linear_plan_for_sms(int32_t form, int64_t m, int64_t k, int64_t n, int32_t num_sms,
                                          gemm_plan_linear* out) {
    return make_linear_plan(form, m, k, n, num_sms, out);
}

gemm_status gemm_bf16_linear_run(const gemm_plan_linear* plan, const uint16_t* A, int64_t lda, const uint16_t* B,
                                 int64_t ldb, const float* bias, int32_t activation, uint16_t* Z, int64_t ldz,
                                 const void* residual, int64_t ldr, int32_t out_type, void* D, int64_t ldd,
                                 void* stream) {
    const gemm_plan_linear* p = plan;
    if (!p || p->version != GEMM_PLAN_LINEAR_VERSION) return GEMM_ERR_INVALID_ARG;
    if (check_linear_shape(p->form, p->m, p->k, p->n) != GEMM_OK || !linear_config_ok(p)) return GEMM_ERR_INVALID_ARG;
    if (!A || !B || !D) return GEMM_ERR_INVALID_ARG;
    const int32_t act = activation & ~GEMM_ACT_GRADIENT;
    const bool grad = (activation & GEMM_ACT_GRADIENT) != 0 && act != GEMM_ACT_NONE;
    if (!act_ok(act) || (grad && !Z)) return GEMM_ERR_INVALID_ARG;
    if (activation == (GEMM_ACT_NONE | GEMM_ACT_GRADIENT)) Z = nullptr;   // its derivative is 1: not read
    if (out_type != GEMM_OUT_BF16 && out_type != GEMM_OUT_F32) return GEMM_ERR_INVALID_ARG;
    const int64_t rows_a = p->form == GEMM_FORM_TN ? p->k : p->m, cols_a = p->form == GEMM_FORM_TN ? p->m : p->k;
    const int64_t rows_b = p->form == GEMM_FORM_NT ? p->n : p->k, cols_b = p->form == GEMM_FORM_NT ? p->k : p->n;
    if (!pitch_ok(lda, cols_a) || !pitch_ok(ldb, cols_b) || !pitch_ok(ldd, p->n) || (Z && !pitch_ok(ldz, p->n)) ||
        (residual && !pitch_ok(ldr, p->n)))
        return GEMM_ERR_INVALID_ARG;
    if (residual == D && ldr != ldd) return GEMM_ERR_INVALID_ARG;
    const uintptr_t es = out_type == GEMM_OUT_F32 ? 4 : 2;
    if (!al(A, 2) || !al(B, 2) || !al(Z, 2) || !al(D, es) || !al(residual, es) || !al(bias, 4)) return GEMM_ERR_MISALIGNED;
    const void* const z_out = grad ? nullptr : Z;
    if (!apart({D, z_out}, {A, B, bias}) || D == Z || (z_out && z_out == residual)) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    LinearLaunch L;
    L.A = A;
    L.B = B;
    L.bias = bias;
    L.R = residual;
    L.Z = Z;
    L.D = D;
    L.err = ctx.err_word;
    L.m = p->m;
    L.k = p->k;
    L.n = p->n;
    L.lda = lda;
    L.ldb = ldb;
    L.ldd = ldd;
    L.ldr = ldr;
    L.ldz = ldz;
    L.form = p->form;
    L.act = act;
    L.grad = grad;
    L.out_f32 = out_type == GEMM_OUT_F32;
    L.bm = p->bm;
    L.bn = p->bn;
    L.split_k = p->split_k;
    L.num_sms = ctx.num_sms;
    L.pairs = ctx.pairs;
    Scratch scratch(ctx.pool, s);
    const bool sampled = trace_begin_call();
    Repitch ra{A, lda, nullptr, (cols_a + 7) / 8 * 8, tma_rows(A, lda) ? 0 : rows_a, cols_a};
    Repitch rb{B, ldb, nullptr, (cols_b + 7) / 8 * 8, tma_rows(B, ldb) ? 0 : rows_b, cols_b};
    if (ra.rows || rb.rows) {   // one launch, and scratch, for both
        const int64_t in_a = (ra.rows * ra.pitch * 2 + 255) / 256 * 256;
        uint8_t* copy = static_cast<uint8_t*>(scratch.take(in_a + rb.rows * rb.pitch * 2));
        if (!copy) return GEMM_ERR_CUDA;
        ra.dst = copy;
        rb.dst = copy + in_a;
        void* unit = trace_unit_begin(GEMM_KERNEL_STAGE, s, sampled);
        const cudaError_t e = launch_repitch(ra, rb, ctx.num_sms, s);
        trace_unit_end(unit, s);
        if (e != cudaSuccess) return GEMM_ERR_CUDA;
        trace_launch(GEMM_KERNEL_STAGE);
        if (ra.rows) {
            L.A = ra.dst;
            L.lda = ra.pitch;
        }
        if (rb.rows) {
            L.B = rb.dst;
            L.ldb = rb.pitch;
        }
    }
    const int kind = p->path == GEMM_PATH_SKINNY ? GEMM_KERNEL_SKINNY : GEMM_KERNEL_TC;
    void* unit = trace_unit_begin(kind, s, sampled);
    const cudaError_t e = p->path == GEMM_PATH_SKINNY ? launch_linear_skinny(L, s) : launch_linear_tc2(L, s);
    trace_unit_end(unit, s);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    trace_launch(kind);
    return GEMM_OK;
}

gemm_status gemm_activation_backward(const uint16_t* dY, int64_t lddy, const uint16_t* Z, int64_t ldz,
                                     int32_t activation, int64_t rows, int64_t cols, uint16_t* dZ, int64_t lddz,
                                     float* dbias, void* stream) {
    if (!dY || (!dZ && !dbias) || !act_ok(activation) || (!Z && activation != GEMM_ACT_NONE)) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || !dim_ok(cols)) return GEMM_ERR_INVALID_ARG;
    if (activation == GEMM_ACT_NONE) Z = nullptr;   // not read
    if (!pitch_ok(lddy, cols) || (Z && !pitch_ok(ldz, cols)) || (dZ && !pitch_ok(lddz, cols))) return GEMM_ERR_INVALID_ARG;
    if ((dZ == dY && lddz != lddy) || (dZ && dZ == Z && lddz != ldz)) return GEMM_ERR_INVALID_ARG;
    if (!al(dY, 2) || !al(Z, 2) || !al(dZ, 2) || !al(dbias, 4)) return GEMM_ERR_MISALIGNED;
    if (!apart({dbias}, {dY, Z, dZ})) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    ActBwd a;
    a.dY = dY;
    a.Z = Z;
    a.dZ = dZ;
    a.dbias = dbias;
    a.partial = nullptr;
    a.rows = rows;
    a.cols = cols;
    a.lddy = lddy;
    a.ldz = ldz;
    a.lddz = lddz;
    a.act = activation;
    a.num_sms = ctx.num_sms;
    a.parts = act_bwd_parts(a);
    Scratch scratch(ctx.pool, s);
    const int clusters = act_bwd_clusters(a);
    const bool joined = dbias && clusters > 1;
    if (joined) {
        a.partial = static_cast<float*>(scratch.take(clusters * cols * 4));
        if (!a.partial) return GEMM_ERR_CUDA;
    }
    const gemm_status r = staged([&] { return launch_act_bwd(a, s); }, s);
    if (r == GEMM_OK && joined) trace_launch(GEMM_KERNEL_STAGE);   // the sums are joined by a second kernel
    return r;
}

gemm_status gemm_layer_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* W, const float* bias,
                            float eps, int32_t x_type, int32_t y_type, int64_t rows, int64_t d, void* H, int64_t ldh,
                            float* mean, float* rstd, void* Y, int64_t ldy, void* stream) {
    if (!X || !W || !Y || (R && !H)) return GEMM_ERR_INVALID_ARG;
    if (!real_type(x_type) || !real_type(y_type)) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || d < 1 || d > GEMM_NORM_MAX_D || !(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(ldx, d) || (R && !pitch_ok(ldr, d)) || (H && !pitch_ok(ldh, d)) || !pitch_ok(ldy, d))
        return GEMM_ERR_INVALID_ARG;
    // in place only over the same elements
    if (H && ((H == X && ldh != ldx) || (H == R && ldh != ldr))) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(x_type);
    if (!al(X, es) || !al(R, es) || !al(H, es) || !al(Y, elem_bytes(y_type)) || !al(W, 4) || !al(bias, 4) || !al(mean, 4) ||
        !al(rstd, 4))
        return GEMM_ERR_MISALIGNED;
    if (!apart({H, mean, rstd, Y}, {W, bias}) || !apart({mean, rstd, Y}, {X, R})) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    LayerNormFwd a;
    a.X = X;
    a.R = R;
    a.W = W;
    a.bias = bias;
    a.eps = eps;
    a.x_type = x_type;
    a.y_type = y_type;
    a.rows = rows;
    a.d = d;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.H = H;
    a.Y = Y;
    a.mean = mean;
    a.rstd = rstd;
    a.num_sms = ctx.num_sms;
    a.err = ctx.err_word;
    return staged([&] { return launch_layer_norm_fwd(a, s); }, s);
}

gemm_status gemm_layer_norm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const float* W,
                                     const float* mean, const float* rstd, const void* dR, int64_t lddr,
                                     int32_t x_type, int32_t y_type, int64_t rows, int64_t d, void* dX, int64_t lddx,
                                     float* dW, float* dbias, void* stream) {
    if (!dY || !H || !W || !mean || !rstd || !dX) return GEMM_ERR_INVALID_ARG;
    if (!real_type(x_type) || !real_type(y_type)) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || d < 1 || d > GEMM_NORM_MAX_D) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(lddy, d) || !pitch_ok(ldh, d) || (dR && !pitch_ok(lddr, d)) || !pitch_ok(lddx, d))
        return GEMM_ERR_INVALID_ARG;
    if ((dX == dR && lddx != lddr) || (dX == dY && (lddx != lddy || x_type != y_type))) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(x_type);
    if (!al(dY, elem_bytes(y_type)) || !al(H, es) || !al(dR, es) || !al(dX, es) || !al(W, 4) || !al(mean, 4) ||
        !al(rstd, 4) || !al(dW, 4) || !al(dbias, 4))
        return GEMM_ERR_MISALIGNED;
    if (!apart({dX, dW, dbias}, {H, W, mean, rstd}) || !apart({dW, dbias}, {dY, dR})) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    LayerNormBwd a;
    a.dY = dY;
    a.H = H;
    a.dR = dR;
    a.W = W;
    a.mean = mean;
    a.rstd = rstd;
    a.x_type = x_type;
    a.y_type = y_type;
    a.rows = rows;
    a.d = d;
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddr = lddr;
    a.lddx = lddx;
    a.dX = dX;
    a.dW = dW;
    a.dbias = dbias;
    a.partial = nullptr;
    a.num_sms = ctx.num_sms;
    a.err = ctx.err_word;
    a.parts = layer_norm_bwd_parts(a);
    Scratch scratch(ctx.pool, s);
    if ((dW || dbias) && a.parts > 1) {
        a.partial = static_cast<float*>(scratch.take(2 * static_cast<int64_t>(a.parts) * d * 4));
        if (!a.partial) return GEMM_ERR_CUDA;
    }
    int launches = 0;
    const gemm_status r = staged([&] { return launch_layer_norm_bwd(a, s, &launches); }, s);
    for (int i = 1; r == GEMM_OK && i < launches; ++i) trace_launch(GEMM_KERNEL_STAGE);
    return r;
}

gemm_status gemm_balance(const void* X, int64_t ldx, int32_t x_type, int64_t rows, int32_t experts,
                         const int32_t* index, int32_t top_k, float coef, int32_t* counts, int32_t* offsets,
                         int32_t* used, float* lse, float* probs, float* loss, void* stream) {
    if (!X || !index || !counts || !used || !lse || !probs || !loss || !real_type(x_type)) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || experts < 1 || experts > GEMM_BALANCE_MAX_EXPERTS || top_k < 1 || rows * top_k > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(ldx, experts)) return GEMM_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(index), static_cast<const void*>(counts), static_cast<const void*>(offsets),
                          static_cast<const void*>(used), static_cast<const void*>(lse), static_cast<const void*>(probs),
                          static_cast<const void*>(loss)})
        if (!al(p, 4)) return GEMM_ERR_MISALIGNED;
    if (!al(X, elem_bytes(x_type))) return GEMM_ERR_MISALIGNED;
    if (!apart({counts, offsets, used, lse, probs, loss}, {X, index})) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Balance a;
    a.X = X;
    a.x_type = x_type;
    a.rows = rows;
    a.ldx = ldx;
    a.experts = experts;
    a.top_k = top_k;
    a.index = index;
    a.coef = coef;
    a.counts = counts;
    a.offsets = offsets;
    a.used = used;
    a.lse = lse;
    a.probs = probs;
    a.loss = loss;
    a.num_sms = ctx.num_sms;
    a.parts = balance_parts(a);
    Scratch scratch(ctx.pool, s);
    a.partial_p = nullptr;
    a.partial_c = nullptr;
    if (a.parts > 1) {
        const int64_t sums = static_cast<int64_t>(a.parts) * experts;
        a.partial_p = static_cast<float*>(scratch.take(4 * (2 * sums + a.parts)));
        if (!a.partial_p) return GEMM_ERR_CUDA;
        a.partial_c = reinterpret_cast<int32_t*>(a.partial_p + sums);
    }
    int launches = 0;
    const gemm_status r = staged([&] { return launch_balance(a, s, &launches); }, s);
    for (int i = 1; r == GEMM_OK && i < launches; ++i) trace_launch(GEMM_KERNEL_STAGE);
    return r;
}

gemm_status gemm_balance_backward(const void* X, int64_t ldx, int32_t x_type, int64_t rows, int32_t experts,
                                  const float* lse, const int32_t* counts, const int32_t* used, float coef,
                                  const float* dloss, const void* dR, int64_t lddr, void* dX, int64_t lddx,
                                  void* stream) {
    if (!X || !lse || !counts || !used || !dloss || !dX || !real_type(x_type)) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || experts < 1 || experts > GEMM_BALANCE_MAX_EXPERTS) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(ldx, experts) || (dR && !pitch_ok(lddr, experts)) || !pitch_ok(lddx, experts)) return GEMM_ERR_INVALID_ARG;
    if (dX == dR && lddx != lddr) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(x_type);
    if (!al(X, es) || !al(dR, es) || !al(dX, es) || !al(lse, 4) || !al(counts, 4) || !al(used, 4) || !al(dloss, 4))
        return GEMM_ERR_MISALIGNED;
    if (!apart({dX}, {X, lse, counts, used, dloss})) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    BalanceBwd a;
    a.X = X;
    a.dR = dR;
    a.dX = dX;
    a.x_type = x_type;
    a.rows = rows;
    a.ldx = ldx;
    a.lddr = lddr;
    a.lddx = lddx;
    a.experts = experts;
    a.lse = lse;
    a.counts = counts;
    a.used = used;
    a.coef = coef;
    a.dloss = dloss;
    a.num_sms = ctx.num_sms;
    return staged([&] { return launch_balance_bwd(a, s); }, s);
}

}  // extern "C"
