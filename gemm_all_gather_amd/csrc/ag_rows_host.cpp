// Host side of the operators that take whole rows: codes of 8 bits and back, the root-mean-square norm and its gradients.
// Validation, the number of workgroups, the workspace's layout and the launches.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ag.h"
#include "ag_matrix.h"
#include "ag_rows.h"
#include "ag_status.h"

namespace {

using namespace ag;

ag_status_t check_rows(int64_t M, int64_t K, int dtype, bool f32)
{
    if (M < 0 || K < 0) return fail(AG_ERR_INVALID_ARG, "M or K is negative");
    if (M >= kMaxDim || K > kMaxRow)
        return fail(AG_ERR_UNSUPPORTED, "M %lld, K %lld: M below 2^31, K up to 2^20", static_cast<long long>(M),
                    static_cast<long long>(K));
    if (dtype == AG_F32 && !f32) return fail(AG_ERR_UNSUPPORTED, "the norm takes AG_F16 or AG_BF16 rows");
    if (dtype != AG_F16 && dtype != AG_BF16 && dtype != AG_F32) return fail(AG_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return AG_OK;
}

int size_of(int dtype) { return dtype == AG_F32 ? 4 : 2; }

int64_t row_groups(int64_t M, const RowsShape& s) { return (M + s.per_group - 1) / s.per_group; }

// Workgroups of a pass over rows.  A row (or a workgroup's few short ones) each: workgroups that take rows in turn measured 5.2
// TB/s where these reach 5.7 (the norm of 16384 x 8192 bf16 with residual and codes, 182 and 165 us).
int rows_programs(int64_t M, const RowsShape& s) { return static_cast<int>(std::min(row_groups(M, s), kMaxRowsPrograms)); }

// A norm's 1024 threads have a CU to themselves, and nothing runs beside the end of one workgroup and the start of the next: they
// take rows in turn (4096 x 16384 bf16 104 us, a row each 113).
int norm_programs(int64_t M, const RowsShape& s, int cus) { return s.threads == 1024 ? static_cast<int>(std::min<int64_t>(M, cus)) : rows_programs(M, s); }

// ------------------------------------------------------------------ codes

struct Codes {
    Mat rows, q, scale;
};

ag_status_t plan_codes(const void* x, int64_t ldx, const int8_t* q, int64_t ldq, const float* scale, int64_t M, int64_t K,
                       int dtype, const char* name, Codes* c)
{
    ag_status_t s = check_rows(M, K, dtype, true);
    if (s != AG_OK) return s;
    c->rows = Mat{name, addr(x), M, K, ldx ? ldx : K, size_of(dtype)};
    c->q = Mat{"q", addr(q), M, K, ldq ? ldq : K, 1};
    c->scale = Mat{"scale", addr(scale), 1, M, M, 4};
    for (const Mat* m : {&c->rows, &c->q, &c->scale})
        if ((s = check_mat(*m, true)) != AG_OK) return s;
    return AG_OK;
}

// ------------------------------------------------------------------ the norm

constexpr double kLeastEps = 1e-60;      // a row of zeros has the finite rstd 1e30 then

struct Norm {
    Mat x, residual, weight, h, y, q, scale, rstd;
    RowsShape shape{};
    int programs = 0;
};

ag_status_t plan_norm(const ag_rms_norm_args_t* a, int cus, Norm* n)
{
    if (!a) return fail(AG_ERR_INVALID_ARG, "args is NULL");
    for (int32_t r : a->reserved)
        if (r != 0) return fail(AG_ERR_INVALID_ARG, "a reserved field is not 0");
    ag_status_t s = check_rows(a->M, a->K, a->dtype, false);
    if (s != AG_OK) return s;
    if (!(a->eps >= kLeastEps) || !std::isfinite(a->eps))
        return fail(AG_ERR_INVALID_ARG, "eps %g is not finite and %g or more", a->eps, kLeastEps);
    const int64_t M = a->M, K = a->K;
    n->x = Mat{"x", addr(a->x), M, K, a->ldx ? a->ldx : K, 2};
    n->residual = Mat{"residual", addr(a->residual), M, K, a->ldr ? a->ldr : K, 2};
    n->weight = Mat{"weight", addr(a->weight), 1, K, K, 2};
    n->h = Mat{"h", addr(a->h), M, K, a->ldh ? a->ldh : K, 2};
    n->y = Mat{"y", addr(a->y), M, K, a->ldy ? a->ldy : K, 2};
    n->q = Mat{"q", addr(a->q), M, K, a->ldq ? a->ldq : K, 1};
    n->scale = Mat{"scale", addr(a->scale), 1, M, M, 4};
    n->rstd = Mat{"rstd", addr(a->rstd), 1, M, M, 4};
    if ((s = check_mat(n->x, true)) != AG_OK) return s;
    for (const Mat* m : {&n->residual, &n->weight, &n->h, &n->y, &n->q, &n->scale, &n->rstd})
        if ((s = check_mat(*m, false)) != AG_OK) return s;
    if (M > 0 && K > 0 && (a->q == nullptr) != (a->scale == nullptr))
        return fail(AG_ERR_INVALID_ARG, "q and scale come together or not at all");
    if ((s = check_overlaps({n->x, n->residual, n->weight}, {n->y, n->q, n->scale, n->rstd})) != AG_OK) return s;
    if ((s = check_overlaps({n->weight, n->y, n->q, n->scale, n->rstd}, {n->h})) != AG_OK) return s;
    for (const Mat* m : {&n->x, &n->residual}) {
        const bool in_place = n->h.at == m->at && n->h.ld == m->ld;
        if (!in_place && share(n->h, *m)) return fail(AG_ERR_INVALID_ARG, "h overlaps %s without being it", m->name);
    }
    if (M == 0) return AG_OK;
    n->shape = rows_shape(K, true);
    n->programs = norm_programs(M, n->shape, cus);
    return AG_OK;
}

struct NormBackward {
    Mat dy, h, dh, weight, rstd, dx, dw;
    RowsShape shape{};
    int parts = 0;                  // rows of dw's sums: workgroups, or batches of rows in the two passes
    int64_t rows = 0;               // of a batch
    int64_t ldsums = 0;             // floats from one row of sums to the next
    int64_t means = 0;              // of rows, between the two passes
    bool sum = false;               // dw's sums are joined
    bool small = false;             // both gradients in one launch, without sums
    uint64_t sums_offset = 0, workspace = 0;
    int launches = 0;
};

ag_status_t plan_norm_backward(const ag_rms_norm_backward_args_t* a, int cus, NormBackward* n)
{
    if (!a) return fail(AG_ERR_INVALID_ARG, "args is NULL");
    for (int32_t r : a->reserved)
        if (r != 0) return fail(AG_ERR_INVALID_ARG, "a reserved field is not 0");
    ag_status_t s = check_rows(a->M, a->K, a->dtype, false);
    if (s != AG_OK) return s;
    if (a->dw_dtype != a->dtype && a->dw_dtype != AG_F32)
        return fail(AG_ERR_INVALID_ARG, "dw_dtype %d is neither the rows' dtype nor AG_F32", a->dw_dtype);
    if (a->accumulate != 0 && a->accumulate != 1) return fail(AG_ERR_INVALID_ARG, "accumulate %d is not 0 or 1", a->accumulate);
    const int64_t M = a->M, K = a->K;
    n->dy = Mat{"dy", addr(a->dy), M, K, a->lddy ? a->lddy : K, 2};
    n->h = Mat{"h", addr(a->h), M, K, a->ldh ? a->ldh : K, 2};
    n->dh = Mat{"dh", addr(a->dh), M, K, a->lddh ? a->lddh : K, 2};
    n->weight = Mat{"weight", addr(a->weight), 1, K, K, 2};
    n->rstd = Mat{"rstd", addr(a->rstd), 1, M, M, 4};
    n->dx = Mat{"dx", addr(a->dx), M, K, a->lddx ? a->lddx : K, 2};
    n->dw = Mat{"dw", addr(a->dw), 1, K, K, size_of(a->dw_dtype)};
    const bool any = !n->dx.empty() || !n->dw.empty();
    for (const Mat* m : {&n->dy, &n->h, &n->rstd})
        if ((s = check_mat(*m, any && K > 0)) != AG_OK) return s;
    for (const Mat* m : {&n->dh, &n->weight, &n->dx, &n->dw})
        if ((s = check_mat(*m, false)) != AG_OK) return s;
    if ((s = check_overlaps({n->dy, n->h, n->weight, n->rstd}, {n->dx, n->dw})) != AG_OK) return s;
    if (share(n->dw, n->dh)) return fail(AG_ERR_INVALID_ARG, "dw overlaps dh");
    const bool in_place = n->dx.at == n->dh.at && n->dx.ld == n->dh.ld;
    if (!in_place && share(n->dx, n->dh)) return fail(AG_ERR_INVALID_ARG, "dx overlaps dh without being it");
    if (!any) return AG_OK;
    n->sum = !n->dw.empty() && !(M == 0 && a->accumulate);
    n->launches = n->sum ? 1 : 0;
    if (M == 0) return AG_OK;
    n->shape = norm_backward_shape(K);
    n->ldsums = (K + 31) / 32 * 32;
    // Few rows: dw from dy and h again, beside dx, in one launch (80 x 520 fp16 8.6 us for 11.3, 512 x 4096 bf16 10.1 for 11.5; 1024
    // x 4096 19.4 for 16.0, as every column's sum goes down all rows in 32 lanes).
    if (n->sum && !n->dx.empty() && K <= 4096 && M <= 512) {
        n->small = true;
        n->parts = static_cast<int>(row_groups(M, n->shape));
        n->launches = 1;
        return AG_OK;
    }
    if (n->shape.vectors > 0) {
        // Rows in turn, 1024 threads of a CU: each workgroup leaves a row of sums.  Twice as many measured 211 us for 207
        // (16384 x 8192 bf16), at 1000 x 4100 19.7 for 15.0.
        const int64_t fill = static_cast<int64_t>(cus) * (1024 / (n->shape.threads * n->shape.per_group));
        n->parts = static_cast<int>(std::min(row_groups(M, n->shape), fill));
    } else {
        // about 2048 workgroups of 2048 columns, of at least 8 rows each
        const int64_t groups = (K + 2047) / 2048, parts = std::max<int64_t>(1, 8 * cus / groups);
        n->rows = std::max<int64_t>(8, (M + parts - 1) / parts);
        n->parts = static_cast<int>((M + n->rows - 1) / n->rows);
        if (!n->dx.empty()) n->means = M;
    }
    n->workspace = up256(static_cast<uint64_t>(n->means) * 4);
    n->sums_offset = n->workspace;
    if (n->sum) n->workspace += up256(static_cast<uint64_t>(n->parts) * n->ldsums * 4);
    n->launches = (n->shape.vectors == 0 && n->means > 0 ? 2 : 1) + (n->sum ? 1 : 0);
    return AG_OK;
}

}  // namespace

extern "C" {

ag_status_t ag_quantize_rows(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale, int64_t M, int64_t K,
                             ag_dtype_t dtype, void* stream)
{
    Codes c;
    ag_status_t s = plan_codes(x, ldx, q, ldq, scale, M, K, dtype, "x", &c);
    if (s != AG_OK) return s;
    if ((s = check_overlaps({c.rows}, {c.q, c.scale})) != AG_OK) return s;
    if (M == 0) return ok();
    RowsArgs a{};
    a.x = x;
    a.q = K > 0 ? q : nullptr;
    a.scale = scale;
    a.ldx = c.rows.ld;
    a.ldq = c.q.ld;
    a.M = M;
    a.K = static_cast<int32_t>(K);
    const hipError_t e = launch_rows(a, dtype, false, rows_programs(M, rows_shape(K, false)), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : fail_hip(e, "quantize rows");
}

ag_status_t ag_dequantize_rows(const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy, int64_t M,
                               int64_t K, ag_dtype_t dtype, void* stream)
{
    Codes c;
    ag_status_t s = plan_codes(y, ldy, q, ldq, scale, M, K, dtype, "y", &c);
    if (s != AG_OK) return s;
    if ((s = check_overlaps({c.q, c.scale}, {c.rows})) != AG_OK) return s;
    if (M == 0 || K == 0) return ok();
    const DequantizeArgs a{q, scale, y, c.q.ld, c.rows.ld, M, static_cast<int32_t>(K)};
    const hipError_t e = launch_dequantize(a, dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : fail_hip(e, "dequantize rows");
}

ag_status_t ag_plan_rms_norm(const ag_rms_norm_args_t* args, int num_cus, ag_rows_plan_t* plan)
{
    if (!plan) return fail(AG_ERR_INVALID_ARG, "plan is NULL");
    if (num_cus < 0) return fail(AG_ERR_INVALID_ARG, "num_cus %d < 0", num_cus);
    ag_status_t s;
    if (num_cus == 0 && (s = current_cus(&num_cus)) != AG_OK) return s;
    Norm n;
    if ((s = plan_norm(args, num_cus, &n)) != AG_OK) return s;
    ag_rows_plan_t p{};
    if (n.programs > 0) {
        p.threads_per_row = n.shape.threads;
        p.vectors_per_thread = n.shape.vectors;
        p.n_programs = n.programs;
        p.launches = 1;
        const uint64_t M = args->M, K = args->K;
        p.bytes_read = 2 * M * K * (args->residual ? 2 : 1) + (args->weight ? 2 * K : 0);
        p.bytes_written = M * K * ((args->h ? 2 : 0) + (args->y ? 2 : 0) + (args->q ? 1 : 0)) +
                          4 * M * ((args->scale ? 1 : 0) + (args->rstd ? 1 : 0));
    }
    *plan = p;
    return ok();
}

ag_status_t ag_rms_norm(const ag_rms_norm_args_t* args, void* stream)
{
    Norm n;
    // validation first (on any CU count), so that a bad argument is named even without a device
    ag_status_t s = plan_norm(args, 256, &n);
    if (s != AG_OK) return s;
    if (n.programs == 0) return ok();
    int cus = 0;
    if ((s = current_cus(&cus)) != AG_OK) return s;
    RowsArgs a{};
    a.x = args->x;
    a.residual = n.residual.empty() ? nullptr : args->residual;
    a.weight = args->weight;
    a.h = args->h;
    a.y = args->y;
    a.q = args->q;
    a.scale = args->scale;
    a.rstd = args->rstd;
    a.ldx = n.x.ld;
    a.ldr = n.residual.ld;
    a.ldh = n.h.ld;
    a.ldy = n.y.ld;
    a.ldq = n.q.ld;
    a.M = args->M;
    a.K = static_cast<int32_t>(args->K);
    a.eps = args->eps;
    const hipError_t e = launch_rows(a, args->dtype, true, norm_programs(args->M, n.shape, cus), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : fail_hip(e, "rms norm");
}

ag_status_t ag_plan_rms_norm_backward(const ag_rms_norm_backward_args_t* args, int num_cus, ag_rows_plan_t* plan)
{
    if (!plan) return fail(AG_ERR_INVALID_ARG, "plan is NULL");
    if (num_cus < 0) return fail(AG_ERR_INVALID_ARG, "num_cus %d < 0", num_cus);
    ag_status_t s;
    if (num_cus == 0 && (s = current_cus(&num_cus)) != AG_OK) return s;
    NormBackward n;
    if ((s = plan_norm_backward(args, num_cus, &n)) != AG_OK) return s;
    ag_rows_plan_t p{};
    p.launches = n.launches;
    if (p.launches > 0) {
        p.threads_per_row = n.shape.threads;
        p.vectors_per_thread = n.shape.vectors;
        p.n_programs = n.parts;
        p.workspace_bytes = n.workspace;
        const bool dx = !n.dx.empty(), dw = !n.dw.empty();
        const uint64_t M = args->M, K = args->K, d = dw ? n.dw.esize * K : 0;
        p.bytes_read = 2 * M * K * (dx && args->dh ? 3 : 2) + 4 * M + (args->weight ? 2 * K : 0) + (args->accumulate ? d : 0);
        p.bytes_written = (dx ? 2 * M * K : 0) + d;
    }
    *plan = p;
    return ok();
}

ag_status_t ag_rms_norm_backward(const ag_rms_norm_backward_args_t* args, void* workspace, size_t workspace_bytes, void* stream_)
{
    NormBackward n;
    ag_status_t s = plan_norm_backward(args, 256, &n);
    if (s != AG_OK) return s;
    if (n.launches == 0) return ok();
    int cus = 0;
    if ((s = current_cus(&cus)) != AG_OK) return s;
    if (cus != 256) {
        n = NormBackward{};
        if ((s = plan_norm_backward(args, cus, &n)) != AG_OK) return s;
    }
    s = check_workspace(workspace, workspace_bytes, n.workspace, {n.dy, n.h, n.dh, n.weight, n.rstd, n.dx, n.dw});
    if (s != AG_OK) return s;
    const hipStream_t stream = static_cast<hipStream_t>(stream_);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + n.sums_offset);
    const NormDwArgs d{sums, args->dw, n.ldsums, n.parts, static_cast<int32_t>(args->K), args->dw_dtype, args->accumulate};
    if (n.parts > 0) {
        NormBackwardArgs a{};
        a.dy = static_cast<const uint16_t*>(args->dy);
        a.h = static_cast<const uint16_t*>(args->h);
        a.dh = static_cast<const uint16_t*>(args->dh);
        a.weight = static_cast<const uint16_t*>(args->weight);
        a.rstd = args->rstd;
        a.dx = static_cast<uint16_t*>(args->dx);
        a.sums = n.sum && !n.small ? sums : nullptr;
        a.ldsums = n.ldsums;
        a.lddy = n.dy.ld;
        a.ldh = n.h.ld;
        a.lddh = n.dh.ld;
        a.lddx = n.dx.ld;
        a.M = args->M;
        a.K = static_cast<int32_t>(args->K);
        a.means = n.means > 0 ? static_cast<float*>(workspace) : nullptr;
        const int bf16 = args->dtype == AG_BF16;
        const hipError_t e = n.small ? launch_norm_backward_small(a, d, bf16, n.parts, stream)
                             : n.shape.vectors > 0 ? launch_norm_backward(a, bf16, n.parts, stream)
                                                 : launch_norm_backward_long(a, bf16, n.parts, static_cast<int>(n.rows), stream);
        if (e != hipSuccess) return fail_hip(e, "rms norm gradients");
    }
    if (n.sum && !n.small) {
        const hipError_t e = launch_norm_dw(d, stream);
        if (e != hipSuccess) return fail_hip(e, "rms norm weight gradient");
    }
    return ok();
}

}  // extern "C"
