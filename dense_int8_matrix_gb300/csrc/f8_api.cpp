// C entry points of the 8-bit operators: argument checks, plans, dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "checks.h"
#include "context.h"
#include "f8.h"
#include "internal.h"

using namespace gemm;

namespace {

gemm_status check_f8_shape(int32_t mode, int32_t groups, int64_t m, int64_t k, int64_t n, int32_t a_type,
                           int32_t b_type, int32_t b_scale) {
    if (mode < GEMM_GROUP_NONE || mode > GEMM_GROUP_K) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(m) || !dim_ok(k) || !dim_ok(n)) return GEMM_ERR_INVALID_ARG;
    if (groups < 1 || groups > GEMM_F8_MAX_GROUPS || (mode == GEMM_GROUP_NONE && groups != 1)) return GEMM_ERR_INVALID_ARG;
    if (mode == GEMM_GROUP_ROWS && groups * n > kMaxDim) return GEMM_ERR_INVALID_ARG;
    if (mode == GEMM_GROUP_K && (groups * m > kMaxDim || k % kF8Block != 0)) return GEMM_ERR_INVALID_ARG;
    for (int32_t t : {a_type, b_type})
        if (t != GEMM_F8_E4M3 && t != GEMM_F8_E5M2) return GEMM_ERR_INVALID_ARG;
    if (b_scale != GEMM_SCALE_ROWS && b_scale != GEMM_SCALE_BLOCKS) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// Estimated microseconds of a product of `tiles` tiles of bm rows by 128
// columns and `blocks` K blocks, split_k CTAs to a tile.  The constants were
// fitted to the times of every configuration on 238 drawn products on GB300
// (152 SMs): a block of a tile, what a round of CTAs costs besides, and the
// join of a split.  Two CTAs share an SM below 64 rows and then take 1.9 times
// as long; clusters of four and eight cannot use every SM (of eight: 15 fit, 300 x
// 16384 x 640 17 us; 16 do not, 128 x 8192 x 2048 23 us).
double skinny_time(double tiles, int64_t blocks, int bm, int split, int num_sms) {
    const double block = bm <= 32 ? 0.17 : bm == 64 ? 0.22 : 0.40;
    const double part = bm < 64 ? (split == 8 ? 256.0 : 304.0) / 152 : split == 8 ? 120.0 / 152 : split == 4 ? 128.0 / 152 : 1.0;
    const double ctas = tiles * split, room = std::max(1.0, std::floor(part * num_sms));
    const double rounds = std::ceil(ctas / room);
    const double share = bm < 64 && ctas > num_sms ? 1.9 : 1.0;
    return rounds * ((bm < 64 ? 3.0 : 3.4) + block * share * static_cast<double>(ceil_div(blocks, split))) +
           (split > 1 ? 1.0 + 2.5 * bm / 128 : 0.0);
}

// The same for two-SM tiles; fewer than fill half the pairs run as halves.
double pair_time(double tiles, int64_t blocks, int num_sms) {
    const double pairs = std::max(1, num_sms / 2);
    const double b = static_cast<double>(blocks);
    return 3.6 + (2 * tiles <= pairs ? 0.36 * b : std::ceil(tiles / pairs) * (3.4 + 0.47 * b));
}

// The tile and split of a product: the least estimate.  Rows are those of a
// group, on average.  On 139 other drawn products the choice took 3.4 % longer
// than the best configuration of each, against 6.7 % for tiles chosen by the
// number of rows and split as far as SMs were idle (100 x 8192 x 8192 21.7 us
// with 128 rows split in two, 19.9 with two tiles of 64; 128 x 8192 x 2048
// 23.1 split in eight, whose clusters do not fit at once, and 11.4).
void choose_config(gemm_plan_f8* p) {
    const int64_t kb = ceil_div(p->k, kF8Block);
    const bool by_rows = p->group_mode == GEMM_GROUP_ROWS, by_k = p->group_mode == GEMM_GROUP_K;
    const int64_t rows = by_rows ? ceil_div(p->m, p->groups) : p->m;
    const double groups = static_cast<double>(by_rows ? std::min<int64_t>(p->m, p->groups) : p->groups);
    const int64_t blocks = by_k ? ceil_div(kb, p->groups) : kb;   // of a tile
    p->path = GEMM_PATH_TENSOR;
    p->bm = p->bn = 256;
    p->split_k = 1;
    double best = rows <= 64 ? 1e300
                             : pair_time(groups * static_cast<double>(ceil_div(rows, 256) * ceil_div(p->n, 256)), blocks, p->num_sms);
    for (int bm = 16; bm <= 128; bm *= 2) {
        if (bm < 128 && (rows > 4 * bm || bm > 2 * std::max<int64_t>(rows, 16))) continue;
        if (bm == 128 && rows < 64) continue;
        const double tiles = groups * static_cast<double>(ceil_div(rows, bm)) * static_cast<double>(ceil_div(p->n, 128));
        for (int s = 1; s <= 8; s *= 2) {
            if (s > 1 && blocks / s < 2) break;
            const double t = skinny_time(tiles, blocks, bm, s, p->num_sms);
            if (t >= best) continue;
            best = t;
            p->path = GEMM_PATH_SKINNY;
            p->bm = bm;
            p->bn = 128;
            p->split_k = s;
        }
    }
}

gemm_status make_f8_plan(int32_t mode, int32_t groups, int64_t m, int64_t k, int64_t n, int32_t a_type, int32_t b_type,
                         int32_t b_scale, int32_t num_sms, gemm_plan_f8* out) {
    if (!out || num_sms < 1) return GEMM_ERR_INVALID_ARG;
    const gemm_status st = check_f8_shape(mode, groups, m, k, n, a_type, b_type, b_scale);
    if (st != GEMM_OK) return st;
    std::memset(out, 0, sizeof(*out));
    out->version = GEMM_PLAN_F8_VERSION;
    out->num_sms = num_sms;
    out->group_mode = mode;
    out->m = m;
    out->k = k;
    out->n = n;
    out->groups = groups;
    out->a_type = a_type;
    out->b_type = b_type;
    out->b_scale = b_scale;
    choose_config(out);
    return GEMM_OK;
}

// A compiled configuration: the two-SM tiles, or the skinny tiles and splits.
bool f8_config_ok(const gemm_plan_f8* p) {
    if (p->path == GEMM_PATH_TENSOR) return p->bm == 256 && (p->bn == 128 || p->bn == 256) && p->split_k == 1;
    const int bm = p->bm, s = p->split_k;
    return p->path == GEMM_PATH_SKINNY && (bm == 16 || bm == 32 || bm == 64 || bm == 128) && p->bn == 128 &&
           (s == 1 || s == 2 || s == 4 || s == 8);
}

gemm_status plan_here(int32_t mode, int32_t groups, int64_t m, int64_t k, int64_t n, int32_t a_type, int32_t b_type,
                      int32_t b_scale, gemm_plan_f8* out) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_f8_shape(mode, groups, m, k, n, a_type, b_type, b_scale);
    if (st != GEMM_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != GEMM_OK) return st;
    return make_f8_plan(mode, groups, m, k, n, a_type, b_type, b_scale, sms, out);
}

gemm_status run_f8(const gemm_plan_f8* p, const uint8_t* A, int64_t lda, const float* a_scale, const uint8_t* Bt,
                   int64_t ldb, const float* b_scale, const int32_t* offsets, int32_t out_type, void* D, int64_t ldd,
                   cudaStream_t stream) {
    if (!p || p->version != GEMM_PLAN_F8_VERSION) return GEMM_ERR_INVALID_ARG;
    const gemm_status st0 =
        check_f8_shape(p->group_mode, p->groups, p->m, p->k, p->n, p->a_type, p->b_type, p->b_scale);
    if (st0 != GEMM_OK) return st0;
    if (!f8_config_ok(p)) return GEMM_ERR_INVALID_ARG;
    if ((offsets != nullptr) != (p->group_mode != GEMM_GROUP_NONE)) return GEMM_ERR_INVALID_ARG;
    if (!A || !Bt || !a_scale || !b_scale || !D) return GEMM_ERR_INVALID_ARG;
    if (out_type != GEMM_OUT_BF16 && out_type != GEMM_OUT_F32) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(lda, p->k) || !pitch_ok(ldb, p->k) || !pitch_ok(ldd, p->n)) return GEMM_ERR_INVALID_ARG;
    if (!al(A, 16) || !al(Bt, 16) || lda % 16 || ldb % 16 || !al(a_scale, 4) || !al(b_scale, 4) ||
        !al(D, out_type == GEMM_OUT_F32 ? 4 : 2) || !al(offsets, 4))
        return GEMM_ERR_MISALIGNED;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    F8Launch L;
    L.A = A;
    L.Bt = Bt;
    L.a_scale = a_scale;
    L.b_scale = b_scale;
    L.offsets = offsets;
    L.D = D;
    L.err = ctx.err_word;
    L.m = p->m;
    L.k = p->k;
    L.n = p->n;
    L.lda = lda;
    L.ldb = ldb;
    L.ldd = ldd;
    L.rows_a = p->m;
    L.rows_b = p->group_mode == GEMM_GROUP_ROWS ? p->n * p->groups : p->n;
    L.groups = p->groups;
    L.group_mode = p->group_mode;
    L.a_type = p->a_type;
    L.b_type = p->b_type;
    L.b_scale_mode = p->b_scale;
    L.out_f32 = out_type == GEMM_OUT_F32;
    L.bm = p->bm;
    L.bn = p->bn;
    L.split_k = p->split_k;
    L.num_sms = ctx.num_sms;
    L.pairs = ctx.pairs;
    const int kind = p->path == GEMM_PATH_SKINNY ? GEMM_KERNEL_SKINNY : GEMM_KERNEL_TC;
    const bool sampled = trace_begin_call();
    void* unit = trace_unit_begin(kind, stream, sampled);
    const cudaError_t e = p->path == GEMM_PATH_SKINNY ? launch_f8_skinny(L, stream) : launch_f8_tc2(L, stream);
    trace_unit_end(unit, stream);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    trace_launch(kind);
    return GEMM_OK;
}

gemm_status check_quant(const void* X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx, int32_t f8_type,
                        const void* Q, int64_t ldq, int64_t qcols, const float* scale) {
    if (!X || !Q || !scale || !dim_ok(rows) || !dim_ok(cols)) return GEMM_ERR_INVALID_ARG;
    if (x_type != GEMM_DTYPE_BF16 && x_type != GEMM_DTYPE_F32) return GEMM_ERR_INVALID_ARG;
    if (f8_type != GEMM_F8_E4M3 && f8_type != GEMM_F8_E5M2) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(ldx, cols) || !pitch_ok(ldq, qcols)) return GEMM_ERR_INVALID_ARG;
    if (!al(X, elem_bytes(x_type)) || !al(scale, 4)) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

gemm_status run_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* W, float eps, int32_t x_type,
                     int64_t rows, int64_t d, void* H, int64_t ldh, float* rstd, void* Q, int64_t ldq, float* scale,
                     bool to_i8, cudaStream_t stream) {
    if (!X || !W || !Q || !scale || (R && !H)) return GEMM_ERR_INVALID_ARG;
    if (x_type != GEMM_DTYPE_BF16 && x_type != GEMM_DTYPE_F32) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || d < 1 || d > GEMM_NORM_MAX_D || !(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(ldx, d) || (R && !pitch_ok(ldr, d)) || (H && !pitch_ok(ldh, d)) || !pitch_ok(ldq, d))
        return GEMM_ERR_INVALID_ARG;
    // in place only over the same elements
    if (H && ((H == X && ldh != ldx) || (H == R && ldh != ldr))) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(x_type);
    if (!al(X, es) || !al(R, es) || !al(H, es) || !al(W, 4) || !al(rstd, 4) || !al(scale, 4)) return GEMM_ERR_MISALIGNED;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    NormFwd a;
    a.X = X;
    a.R = R;
    a.W = W;
    a.eps = eps;
    a.x_type = x_type;
    a.rows = rows;
    a.d = d;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldq = ldq;
    a.H = H;
    a.rstd = rstd;
    a.Q = Q;
    a.scale = scale;
    a.to_i8 = to_i8;
    a.num_sms = ctx.num_sms;
    return staged([&] { return launch_norm_fwd(a, stream); }, stream);
}

}  // namespace

extern "C" {

gemm_status gemm_f8_plan(int64_t m, int64_t k, int64_t n, int32_t a_type, int32_t b_type, int32_t b_scale,
                         gemm_plan_f8* out) {
    return plan_here(GEMM_GROUP_NONE, 1, m, k, n, a_type, b_type, b_scale, out);
}

gemm_status gemm_f8_grouped_plan(int32_t group_mode, int32_t groups, int64_t m, int64_t k, int64_t n, int32_t a_type,
                                 int32_t b_type, int32_t b_scale, gemm_plan_f8* out) {
    if (group_mode == GEMM_GROUP_NONE) return GEMM_ERR_INVALID_ARG;
    return plan_here(group_mode, groups, m, k, n, a_type, b_type, b_scale, out);
}

gemm_status gemm_f8_plan_for_sms(int32_t group_mode, int32_t groups, int64_t m, int64_t k, int64_t n, int32_t a_type,
                                 int32_t b_type, int32_t b_scale, int32_t num_sms, gemm_plan_f8* out) {
    return make_f8_plan(group_mode, groups, m, k, n, a_type, b_type, b_scale, num_sms, out);
}

gemm_status gemm_f8_run(const gemm_plan_f8* plan, const uint8_t* A, int64_t lda, const float* a_scale,
                        const uint8_t* Bt, int64_t ldb, const float* b_scale, int32_t out_type, void* D, int64_t ldd,
                        void* stream) {
    return run_f8(plan, A, lda, a_scale, Bt, ldb, b_scale, nullptr, out_type, D, ldd, static_cast<cudaStream_t>(stream));
}

gemm_status gemm_f8_grouped_run(const gemm_plan_f8* plan, const uint8_t* A, int64_t lda, const float* a_scale,
                                const uint8_t* Bt, int64_t ldb, const float* b_scale, const int32_t* offsets,
                                int32_t out_type, void* D, int64_t ldd, void* stream) {
    if (!offsets) return GEMM_ERR_INVALID_ARG;
    return run_f8(plan, A, lda, a_scale, Bt, ldb, b_scale, offsets, out_type, D, ldd, static_cast<cudaStream_t>(stream));
}

gemm_status gemm_f8_quantize(const void* X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx, int32_t f8_type,
                             int32_t scale_mode, uint8_t* Q, int64_t ldq, float* scale, void* stream) {
    gemm_status st = check_quant(X, x_type, rows, cols, ldx, f8_type, Q, ldq, cols, scale);
    if (st != GEMM_OK) return st;
    if (scale_mode != GEMM_SCALE_ROWS && scale_mode != GEMM_SCALE_BLOCKS) return GEMM_ERR_INVALID_ARG;
    DeviceContext ctx;
    st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    F8Quant q;
    q.X = X;
    q.x_type = x_type;
    q.rows = rows;
    q.cols = cols;
    q.ldx = ldx;
    q.f8_type = f8_type;
    q.offsets = nullptr;
    q.groups = 1;
    q.kp = 0;
    q.Q = Q;
    q.ldq = ldq;
    q.scale = scale;
    q.num_sms = ctx.num_sms;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return staged([&] { return scale_mode == GEMM_SCALE_ROWS ? launch_f8_quant_rows(q, s) : launch_f8_quant_blocks(q, s); }, s);
}

gemm_status gemm_f8_quantize_cols(const void* X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                  int32_t f8_type, const int32_t* offsets, int32_t groups, uint8_t* Q, int64_t ldq,
                                  float* scale, void* stream) {
    if (groups < 1 || groups > GEMM_F8_MAX_GROUPS || (!offsets && groups != 1)) return GEMM_ERR_INVALID_ARG;
    const int64_t kp = gemm_f8_padded_k(rows, groups);
    gemm_status st = check_quant(X, x_type, rows, cols, ldx, f8_type, Q, ldq, kp, scale);
    if (st != GEMM_OK) return st;
    if (!al(Q, 16) || ldq % 16 || !al(offsets, 4)) return GEMM_ERR_MISALIGNED;
    DeviceContext ctx;
    st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    F8Quant q;
    q.X = X;
    q.x_type = x_type;
    q.rows = rows;
    q.cols = cols;
    q.ldx = ldx;
    q.f8_type = f8_type;
    q.offsets = offsets;
    q.groups = groups;
    q.kp = kp;
    q.Q = Q;
    q.ldq = ldq;
    q.scale = scale;
    q.num_sms = ctx.num_sms;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return staged([&] { return launch_f8_quant_cols(q, s); }, s);
}

int64_t gemm_f8_padded_k(int64_t rows, int32_t groups) {
    if (rows < 1 || rows > kMaxDim || groups < 1) return 0;
    return (rows + (kF8Block - 1) * static_cast<int64_t>(groups)) / kF8Block * kF8Block;
}

gemm_status gemm_norm_f8(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* W, float eps,
                         int32_t x_type, int64_t rows, int64_t d, void* H, int64_t ldh, float* rstd, uint8_t* Q,
                         int64_t ldq, float* scale, void* stream) {
    return run_norm(X, ldx, R, ldr, W, eps, x_type, rows, d, H, ldh, rstd, Q, ldq, scale, false,
                    static_cast<cudaStream_t>(stream));
}

gemm_status gemm_norm_i8(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* W, float eps,
                         int32_t x_type, int64_t rows, int64_t d, void* H, int64_t ldh, float* rstd, int8_t* Q,
                         int64_t ldq, float* row_scale, void* stream) {
    return run_norm(X, ldx, R, ldr, W, eps, x_type, rows, d, H, ldh, rstd, Q, ldq, row_scale, true,
                    static_cast<cudaStream_t>(stream));
}

gemm_status gemm_norm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const float* W,
                               const float* rstd, const void* dR, int64_t lddr, int32_t x_type, int64_t rows, int64_t d,
                               void* dX, int64_t lddx, float* dW, void* stream) {
    if (!dY || !H || !W || !rstd || !dX) return GEMM_ERR_INVALID_ARG;
    if (x_type != GEMM_DTYPE_BF16 && x_type != GEMM_DTYPE_F32) return GEMM_ERR_INVALID_ARG;
    if (!dim_ok(rows) || d < 1 || d > GEMM_NORM_MAX_D) return GEMM_ERR_INVALID_ARG;
    if (!pitch_ok(lddy, d) || !pitch_ok(ldh, d) || (dR && !pitch_ok(lddr, d)) || !pitch_ok(lddx, d))
        return GEMM_ERR_INVALID_ARG;
    if (dX == dR && lddx != lddr) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(x_type);
    if (!al(dY, es) || !al(H, es) || !al(dR, es) || !al(dX, es) || !al(W, 4) || !al(rstd, 4) || !al(dW, 4))
        return GEMM_ERR_MISALIGNED;
    DeviceContext ctx;
    const gemm_status st = device_context(&ctx);
    if (st != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    NormBwd a;
    a.dY = dY;
    a.H = H;
    a.dR = dR;
    a.W = W;
    a.rstd = rstd;
    a.x_type = x_type;
    a.rows = rows;
    a.d = d;
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddr = lddr;
    a.lddx = lddx;
    a.dX = dX;
    a.dW = dW;
    a.partial = nullptr;
    a.num_sms = ctx.num_sms;
    a.err = ctx.err_word;
    a.grid = norm_bwd_grid(a);
    void* ws = nullptr;
    if (dW && a.grid > 1) {
        if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(a.grid) * static_cast<size_t>(d) * 4, ctx.pool, s) !=
            cudaSuccess)
            return GEMM_ERR_CUDA;
        a.partial = static_cast<float*>(ws);
    }
    const gemm_status r = staged([&] { return launch_norm_bwd(a, s); }, s);
    if (r == GEMM_OK && ws) trace_launch(GEMM_KERNEL_STAGE);   // dw's sums are added by a second kernel
    if (ws) cudaFreeAsync(ws, s);
    return r;
}

}  // extern "C"
