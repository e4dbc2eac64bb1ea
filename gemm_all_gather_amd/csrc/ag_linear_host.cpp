// Host side of the linear layer and its gradients: validation, the choice of
// kernel, tile and split, the workspace's layout and the launches.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "ag.h"
#include "ag_linear.h"
#include "ag_status.h"

namespace {

using ag::fail;
using ag::fail_hip;
using ag::ok;

constexpr int64_t kMaxDim = int64_t{1} << 31;    // rows (M)
constexpr int64_t kMaxRow = int64_t{1} << 20;    // row length and stride: a tile's rows stay within 32-bit offsets

uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t{255}; }

// A matrix (or vector: rows = 1) in device memory.
struct Mat {
    const char* name;
    uint64_t at;
    int64_t rows, cols, ld;
    int esize;
    bool empty() const { return at == 0 || rows == 0 || cols == 0; }
    uint64_t extent() const { return (static_cast<uint64_t>(rows - 1) * ld + cols) * esize; }
};

// Whether two matrices share a byte.  Matrices of one row pitch whose columns lie side by side do not.
bool share(const Mat& a, const Mat& b)
{
    if (a.empty() || b.empty()) return false;
    if (a.at >= b.at + b.extent() || b.at >= a.at + a.extent()) return false;
    const uint64_t pitch = static_cast<uint64_t>(a.ld) * a.esize;
    if (a.rows > 1 && b.rows > 1 && pitch == static_cast<uint64_t>(b.ld) * b.esize) {
        const uint64_t d = (b.at >= a.at ? (b.at - a.at) : pitch - (a.at - b.at) % pitch) % pitch;
        const uint64_t ca = static_cast<uint64_t>(a.cols) * a.esize, cb = static_cast<uint64_t>(b.cols) * b.esize;
        if (d >= ca && d + cb <= pitch) return false;
    }
    return true;
}

ag_status_t check_mat(const Mat& m, bool needed)
{
    if (m.rows == 0 || m.cols == 0) return AG_OK;
    if (m.at == 0) return needed ? fail(AG_ERR_INVALID_ARG, "%s is NULL", m.name) : AG_OK;
    if (m.at % m.esize != 0) return fail(AG_ERR_INVALID_ARG, "%s is not aligned to its %d-byte elements", m.name, m.esize);
    if (m.ld < m.cols)
        return fail(AG_ERR_INVALID_ARG, "row stride %lld of %s is below its %lld columns", static_cast<long long>(m.ld),
                    m.name, static_cast<long long>(m.cols));
    if (m.rows > 1 && m.ld > kMaxRow)
        return fail(AG_ERR_UNSUPPORTED, "row stride %lld of %s is above %lld", static_cast<long long>(m.ld), m.name,
                    static_cast<long long>(kMaxRow));
    return AG_OK;
}

ag_status_t check_sizes(int64_t M, int64_t N, int64_t K, int dtype, int act)
{
    if (M < 0 || N < 0 || K < 0) return fail(AG_ERR_INVALID_ARG, "M, N or K is negative");
    if (M >= kMaxDim || N > kMaxRow || K > kMaxRow)
        return fail(AG_ERR_UNSUPPORTED, "M %lld, N %lld, K %lld: M below 2^31, N and K up to 2^20",
                    static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K));
    if (dtype == AG_F32) return fail(AG_ERR_UNSUPPORTED, "the linear layer takes AG_F16 or AG_BF16 operands");
    if (dtype != AG_F16 && dtype != AG_BF16) return fail(AG_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (act < AG_ACT_NONE || act > AG_ACT_SILU) return fail(AG_ERR_INVALID_ARG, "unknown activation %d", act);
    return AG_OK;
}

ag_status_t check_overlaps(std::initializer_list<Mat> ins, std::initializer_list<Mat> outs)
{
    for (const Mat* o = outs.begin(); o != outs.end(); ++o) {
        for (const Mat& i : ins)
            if (share(*o, i)) return fail(AG_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
        for (const Mat* q = outs.begin(); q != o; ++q)
            if (share(*o, *q)) return fail(AG_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
    }
    return AG_OK;
}

ag_status_t current_cus(int* cus)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return fail_hip(e, "hipDeviceGetAttribute(multiProcessorCount)");
    return AG_OK;
}

// One operand of a tiled product, and where its aligned copy goes when it needs one: LDS-direct loads
// take rows that start on 4 bytes.
struct Operand {
    uint64_t at;
    int64_t ld, rows, cols;      // as stored
    bool pack = false;
    uint64_t copy_offset = 0;
    int64_t copy_ld() const { return (cols + 7) / 8 * 8; }
    uint64_t copy_bytes() const { return up256(static_cast<uint64_t>(rows) * copy_ld() * 2); }
};

struct Product {
    bool on = false;
    bool stream = false;
    int form = ag::kFormNT, tile = ag::kLinearTile128;
    int64_t I = 0, J = 0, R = 0;
    int64_t tiles_i = 0, tiles_j = 0, stages = 0;
    int64_t full_tiles = 0, splits = 1, split_stages = 1, programs = 0;
    int64_t heavy = 0, common_rounds = 0;
    bool join = false;           // some tail tile is cut
    double us = 0;               // estimated
    uint64_t partial_bytes = 0;
    int launches() const { return !on ? 0 : join ? 2 : 1; }
};

// What a workgroup's 64-wide step measured in long products on all CUs (before a stage's loads lay over both its halves,
// which took 3% off the 256 x 256 ones).
struct Kind {
    double step_us[3], fixed_us;     // a 64-wide step by form (NT, NN, TN); a launch's start and epilogue
};
constexpr Kind kKinds[ag::kLinearTiles] = {{{1.42, 1.46, 1.48}, 6.0},     // 256 x 256
                                           {{0.53, 0.60, 0.75}, 4.0},     // 128 x 128
                                           {{1.02, 0.98, 1.00}, 5.0}};    // 256 x 128

// Whole tiles of one kind; us is a tile's time.
void whole_tiles(Product* p, int tile)
{
    int tm, tn, threads;
    ag::linear_tile_shape(tile, &tm, &tn, &threads);
    p->tile = tile;
    p->stages = std::max<int64_t>(1, (p->R + 63) / 64);
    p->tiles_i = (p->I + tm - 1) / tm;
    p->tiles_j = (p->J + tn - 1) / tn;
    p->full_tiles = p->programs = p->tiles_i * p->tiles_j;
    p->splits = 1;
    p->split_stages = p->stages;
    p->heavy = p->common_rounds = 0;
    p->join = false;
    p->partial_bytes = 0;
    p->us = p->stages * kKinds[tile].step_us[p->form] + kKinds[tile].fixed_us;
}

// Tile and cut with the shortest estimated time.  Whole rounds of tiles on all CUs go one to a workgroup; the
// rest (or that and the last round) either too, or its reductions are cut into parts.  A cut adds the partial
// tiles' traffic and a second launch.
ag_status_t choose(Product* p, int cus)
{
    constexpr double kBytesPerUs = 4e6, kJoinUs = 5.0;
    p->stages = std::max<int64_t>(1, (p->R + 63) / 64);
    double best = 0;
    bool found = false;
    for (int tile = 0; tile < ag::kLinearTiles; ++tile) {
        int tm, tn, threads;
        ag::linear_tile_shape(tile, &tm, &tn, &threads);
        const int64_t ti = (p->I + tm - 1) / tm, tj = (p->J + tn - 1) / tn;
        if (ti > 0x7fffffff || tj > 0x7fffffff || ti * tj > 0x7fffff00) continue;
        const int64_t tiles = ti * tj, rounds = tiles / cus;
        const double step_us = kKinds[tile].step_us[p->form];
        const double tile_us = p->stages * step_us + kKinds[tile].fixed_us;
        auto consider = [&](int64_t full, int64_t splits, int64_t run, double us) {
            if (found && us >= best) return;
            found = true;
            best = p->us = us;
            p->tile = tile;
            p->tiles_i = ti;
            p->tiles_j = tj;
            p->full_tiles = full;
            p->splits = splits;
            p->split_stages = run;
            p->join = splits > 1;
            p->programs = std::min<int64_t>(cus, std::max(full, (tiles - full) * splits));
            p->partial_bytes = splits > 1 ? up256(static_cast<uint64_t>(tiles - full) * splits * tm * tn * 4) : 0;
        };
        consider(tiles, 1, p->stages, static_cast<double>((tiles + cus - 1) / cus) * tile_us);
        for (int64_t keep = rounds; keep >= std::max<int64_t>(0, rounds - 1); --keep) {
            const int64_t tail = tiles - keep * cus;
            if (tail == 0) continue;
            for (int64_t s = 2; s <= std::min<int64_t>(32, p->stages / 2); ++s) {
                const int64_t run = (p->stages + s - 1) / s, splits = (p->stages + run - 1) / run;
                if (splits != s) continue;
                const double bytes = static_cast<double>(tail) * splits * tm * tn * 4;
                if (bytes > 512e6) break;
                const double parts = static_cast<double>((tail * splits + cus - 1) / cus);
                consider(keep * cus, splits, run,
                         keep * tile_us + parts * (run * step_us + kKinds[tile].fixed_us) + kJoinUs + 2 * bytes / kBytesPerUs);
            }
        }
    }
    return found ? AG_OK : fail(AG_ERR_UNSUPPORTED, "the product has more than 2^31 tiles");
}

// Two products in turn on n workgroups, whole 256 x 256 tiles: sets how the second's tiles are dealt out and
// returns the estimated time.  Of the first's tiles `heavy` workgroups have one more than the others, which
// therefore take more of the second's.
double in_turn(const Product& first, Product* second, int64_t n)
{
    const int64_t f = first.full_tiles, s = second->full_tiles, heavy = f % n;
    const double done = static_cast<double>(f / n) * first.us;
    if (heavy == 0) return done + static_cast<double>((s + n - 1) / n) * second->us;
    double best = 0;
    for (int64_t common = 0; common <= (s + n - 1) / n; ++common) {     // rounds that the heavy ones take part in
        const int64_t rest = std::max<int64_t>(0, s - common * n), more = (rest + n - heavy - 1) / (n - heavy);
        const double us = std::max(done + first.us + common * second->us, done + (common + more) * second->us);
        if (common == 0 || us < best) {
            best = us;
            second->heavy = heavy;
            second->common_rounds = common;
        }
    }
    return best;
}

void report(const Product& p, bool pack_a, bool pack_b, ag_product_plan_t* out)
{
    *out = ag_product_plan_t{};
    if (!p.on) return;
    if (p.stream) {
        out->variant = 1;
        out->tile_m = static_cast<int32_t>((p.I + 15) / 16 * 16);
        out->tile_n = 16;
        out->tile_k = 128;
        out->full_tiles = out->n_programs = static_cast<int32_t>((p.J + 15) / 16);
        out->splits = 1;
        return;
    }
    int threads;
    out->variant = 2;
    ag::linear_tile_shape(p.tile, &out->tile_m, &out->tile_n, &threads);
    out->tile_k = 64;
    out->full_tiles = static_cast<int32_t>(p.full_tiles);
    out->splits = static_cast<int32_t>(p.splits);
    out->n_programs = static_cast<int32_t>(p.programs);
    out->packed = (pack_a ? 1 : 0) | (pack_b ? 2 : 0);
}

// Places the copies and partial sums in the workspace after `used` bytes.
void place(Operand* o, uint64_t* used)
{
    o->pack = o->rows > 0 && o->cols > 0 && (o->at % 4 != 0 || (o->rows > 1 && o->ld % 2 != 0));
    if (!o->pack) return;
    o->copy_offset = *used;
    *used += o->copy_bytes();
}

ag_status_t pack(const Operand& o, void* workspace, hipStream_t stream, const uint16_t** at, int64_t* ld)
{
    if (!o.pack) {
        *at = reinterpret_cast<const uint16_t*>(o.at);
        // one row may have any stride: its tiles' other rows are never read
        *ld = o.rows > 1 ? o.ld : o.copy_ld();
        return AG_OK;
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + o.copy_offset);
    const hipError_t e = ag::launch_linear_pack(reinterpret_cast<const uint16_t*>(o.at), o.ld, dst, o.copy_ld(), o.rows,
                                                o.cols, stream);
    if (e != hipSuccess) return fail_hip(e, "linear operand copy");
    *at = dst;
    *ld = o.copy_ld();
    return AG_OK;
}

ag::LinearGemmArgs gemm_args(const Product& p, const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
                             const ag::LinearEpilogue& epi, float* partial)
{
    ag::LinearGemmArgs a{};
    a.A = A;
    a.B = B;
    a.lda = lda;
    a.ldb = ldb;
    a.I = p.I;
    a.J = p.J;
    a.R = p.R;
    a.tiles_i = static_cast<int32_t>(p.tiles_i);
    a.tiles_j = static_cast<int32_t>(p.tiles_j);
    a.stages = static_cast<int32_t>(p.stages);
    a.full_tiles = static_cast<int32_t>(p.full_tiles);
    a.splits = static_cast<int32_t>(p.splits);
    a.split_stages = static_cast<int32_t>(p.split_stages);
    a.heavy = static_cast<int32_t>(p.heavy);
    a.common_rounds = static_cast<int32_t>(p.common_rounds);
    a.partial = partial;
    a.epi = epi;
    return a;
}

ag_status_t run_product(const Product& p, const ag::LinearGemmArgs& a, int bf16, hipStream_t stream)
{
    hipError_t e = ag::launch_linear_gemm(a, bf16, p.form, p.tile, static_cast<int>(p.programs), stream);
    if (e != hipSuccess) return fail_hip(e, "linear product");
    if (p.join) {
        e = ag::launch_linear_join(a, bf16, p.form, p.tile, stream);
        if (e != hipSuccess) return fail_hip(e, "linear join");
    }
    return AG_OK;
}

ag_status_t check_workspace(const void* workspace, size_t have, uint64_t need, std::initializer_list<Mat> mats)
{
    if (need == 0) return AG_OK;
    if (workspace == nullptr || reinterpret_cast<uint64_t>(workspace) % 256 != 0)
        return fail(AG_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (have < need)
        return fail(AG_ERR_INVALID_ARG, "workspace of %zu bytes, %llu needed", have, static_cast<unsigned long long>(need));
    const Mat w{"workspace", reinterpret_cast<uint64_t>(workspace), 1, static_cast<int64_t>(need), static_cast<int64_t>(need), 1};
    for (const Mat& m : mats)
        if (share(w, m)) return fail(AG_ERR_INVALID_ARG, "the workspace overlaps %s", m.name);
    return AG_OK;
}

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

// ------------------------------------------------------------------ forward

struct Forward {
    Mat x, w, bias, residual, y, z;
    Product product;
    Operand ox, ow;
    uint64_t partial_offset = 0, workspace = 0;
    int launches = 0;
};

ag_status_t plan_forward(const ag_linear_args_t* a, int cus, Forward* f)
{
    if (!a) return fail(AG_ERR_INVALID_ARG, "args is NULL");
    for (int32_t r : a->reserved)
        if (r != 0) return fail(AG_ERR_INVALID_ARG, "a reserved field is not 0");
    ag_status_t s = check_sizes(a->M, a->N, a->K, a->dtype, a->act);
    if (s != AG_OK) return s;
    const int64_t M = a->M, N = a->N, K = a->K;
    f->x = Mat{"x", addr(a->x), M, K, a->ldx ? a->ldx : K, 2};
    f->w = Mat{"w", addr(a->w), N, K, a->ldw ? a->ldw : K, 2};
    f->bias = Mat{"bias", addr(a->bias), 1, N, N, 2};
    f->residual = Mat{"residual", addr(a->residual), M, N, a->ldr ? a->ldr : N, 2};
    f->y = Mat{"y", addr(a->y), M, N, a->ldy ? a->ldy : N, 2};
    f->z = Mat{"z", addr(a->z), M, N, a->ldz ? a->ldz : N, 2};
    const bool some = M > 0 && N > 0;
    for (const Mat* m : {&f->x, &f->w, &f->y})
        if ((s = check_mat(*m, some)) != AG_OK) return s;
    for (const Mat* m : {&f->bias, &f->residual, &f->z})
        if ((s = check_mat(*m, false)) != AG_OK) return s;
    if ((s = check_overlaps({f->x, f->w, f->bias}, {f->y, f->z})) != AG_OK) return s;
    if (share(f->z, f->residual)) return fail(AG_ERR_INVALID_ARG, "z overlaps residual");
    const bool in_place = f->y.at == f->residual.at && f->y.ld == f->residual.ld;
    if (!in_place && share(f->y, f->residual)) return fail(AG_ERR_INVALID_ARG, "y overlaps residual without being it");
    if (!some) return AG_OK;

    Product& p = f->product;
    p.on = true;
    p.form = ag::kFormNT;
    p.I = M;
    p.J = N;
    p.R = K;
    // Few rows of x: w is what there is to move, and is streamed.  Above 16 rows every workgroup reads that much more
    // of x, and from about 8M weights on tiles with cut reductions are faster: bf16, N x K 1024 x 1024, 32 rows 5.5
    // against 12.1 us; 3584 x 8192, 32 rows 26.2 against 20.3 (16 rows: 18.7 streamed).
    p.stream = M <= 16 || (M <= ag::kLinearStreamRows && N * K < (int64_t{1} << 23));
    if (!p.stream) {
        if ((s = choose(&p, cus)) != AG_OK) return s;
        f->ox = Operand{f->x.at, f->x.ld, M, K};
        f->ow = Operand{f->w.at, f->w.ld, N, K};
        place(&f->ox, &f->workspace);
        place(&f->ow, &f->workspace);
        f->partial_offset = f->workspace;
        f->workspace += p.partial_bytes;
    }
    f->launches = p.launches() + (f->ox.pack ? 1 : 0) + (f->ow.pack ? 1 : 0);
    return AG_OK;
}

// ------------------------------------------------------------------ backward

struct Backward {
    Mat dy, z, x, w, dx, dw, db;
    Product px, pw;
    Product rest;               // dw of dz's second term, before pw
    Operand ox, ow;
    bool slope = false, store_dz = false;
    bool together = false;      // dx, dw and db in one launch, side by side
    bool in_turn = false, dx_first = false;   // or one after the other
    bool db_alone = false;      // db in a launch of its own; else beside a product
    uint64_t dz_offset = 0, dz_rest_offset = 0, sums_offset = 0, partial_offset = 0, workspace = 0;
    int64_t parts = 0, lddz = 0, rows = 8;
    int launches = 0;
};

ag_status_t plan_backward(const ag_linear_backward_args_t* a, int cus, Backward* b)
{
    if (!a) return fail(AG_ERR_INVALID_ARG, "args is NULL");
    for (int32_t r : a->reserved)
        if (r != 0) return fail(AG_ERR_INVALID_ARG, "a reserved field is not 0");
    ag_status_t s = check_sizes(a->M, a->N, a->K, a->dtype, a->act);
    if (s != AG_OK) return s;
    if (a->dw_dtype != a->dtype && a->dw_dtype != AG_F32)
        return fail(AG_ERR_INVALID_ARG, "dw_dtype %d is neither the operands' dtype nor AG_F32", a->dw_dtype);
    if (a->accumulate != 0 && a->accumulate != 1) return fail(AG_ERR_INVALID_ARG, "accumulate %d is not 0 or 1", a->accumulate);
    const int64_t M = a->M, N = a->N, K = a->K;
    const int g = a->dw_dtype == AG_F32 ? 4 : 2;
    b->dy = Mat{"dy", addr(a->dy), M, N, a->lddy ? a->lddy : N, 2};
    b->z = Mat{"z", addr(a->z), M, N, a->ldz ? a->ldz : N, 2};
    b->x = Mat{"x", addr(a->x), M, K, a->ldx ? a->ldx : K, 2};
    b->w = Mat{"w", addr(a->w), N, K, a->ldw ? a->ldw : K, 2};
    b->dx = Mat{"dx", addr(a->dx), M, K, a->lddx ? a->lddx : K, 2};
    b->dw = Mat{"dw", addr(a->dw), N, K, a->lddw ? a->lddw : K, g};
    b->db = Mat{"db", addr(a->db), 1, N, N, g};
    const bool want_dx = !b->dx.empty(), want_dw = !b->dw.empty(), want_db = !b->db.empty();
    const bool any = want_dx || want_dw || want_db;
    if ((s = check_mat(b->dy, any)) != AG_OK) return s;
    if ((s = check_mat(b->z, any && a->act != AG_ACT_NONE)) != AG_OK) return s;
    if ((s = check_mat(b->x, want_dw)) != AG_OK) return s;
    if ((s = check_mat(b->w, want_dx)) != AG_OK) return s;
    for (const Mat* m : {&b->dx, &b->dw, &b->db})
        if ((s = check_mat(*m, false)) != AG_OK) return s;
    if ((s = check_overlaps({b->dy, b->z, b->x, b->w}, {b->dx, b->dw, b->db})) != AG_OK) return s;
    if (!any) return AG_OK;

    const bool act = a->act != AG_ACT_NONE;
    uint64_t used = 0;
    if (M > 0 && N > 0) {
        const bool aligned = b->dy.at % 4 == 0 && (M == 1 || b->dy.ld % 2 == 0);
        b->store_dz = (want_dx || want_dw) && (act || !aligned);
        b->slope = b->store_dz || want_db;
    }
    b->lddz = (N + 7) / 8 * 8;
    // about 1024 workgroups of 256 columns: enough for every CU, and few partial sums of a long column
    b->rows = std::max<int64_t>(8, std::min<int64_t>(256, (M * ((N + 255) / 256) / 1024 + 7) / 8 * 8));
    if (b->store_dz) {
        b->dz_offset = used;
        used += up256(static_cast<uint64_t>(M) * b->lddz * 2);
    }
    // A weight gradient in fp32 takes dz in two 16-bit terms and so two products: with one it would carry the error
    // of a 16-bit gradient (2-norm relative to dw's 1.7e-3 in bf16, 2.1e-4 in fp16; with two 2.5e-6 and 3.5e-7, as
    // far as fp32 sums go).  It costs a product: all gradients of 16384 x 3584 x 8192, bf16, 2245 to 2290 us against 1468
    // to 1490 of a bf16 dw, of 1024 rows 231 against 122.  dx and a 16-bit dw take one term: their own rounding is as
    // large (2.3e-3 in all against 1.7e-3), and two would double the time of both products.  relu's dz needs no rounding.
    const bool two_terms = b->store_dz && want_dw && act && a->act != AG_ACT_RELU && a->dw_dtype == AG_F32;
    if (two_terms) {
        b->dz_rest_offset = used;
        used += up256(static_cast<uint64_t>(M) * b->lddz * 2);
    }
    if (want_db) {
        b->parts = (M + b->rows - 1) / b->rows;
        b->sums_offset = used;
        used += up256(static_cast<uint64_t>(b->parts) * N * 4);
    }
    if (want_dx) {
        b->px = Product{};
        b->px.on = true;
        b->px.form = ag::kFormNN;
        b->px.I = M;
        b->px.J = K;
        b->px.R = N;
        if ((s = choose(&b->px, cus)) != AG_OK) return s;
        b->ow = Operand{b->w.at, b->w.ld, N, K};
        place(&b->ow, &used);
    }
    if (want_dw && !(M == 0 && a->accumulate)) {
        b->pw = Product{};
        b->pw.on = true;
        b->pw.form = ag::kFormTN;
        b->pw.I = N;
        b->pw.J = K;
        b->pw.R = M;
        if ((s = choose(&b->pw, cus)) != AG_OK) return s;
        b->ox = Operand{b->x.at, b->x.ld, M, K};
        place(&b->ox, &used);
        if (two_terms) b->rest = b->pw;
    }
    // Both products' 128 x 128 tiles on CUs of their own: one launch for what follows dz.
    if (b->px.on && b->pw.on) {
        Product x = b->px, w = b->pw;
        whole_tiles(&x, ag::kLinearTile128);
        whole_tiles(&w, ag::kLinearTile128);
        if (x.full_tiles + w.full_tiles <= cus &&
            std::max(x.us, w.us) < b->px.us + b->pw.us) {
            b->together = true;
            b->px = x;
            b->pw = w;
        }
    }
    // Otherwise both in turn, where that saves a good part of a round: 1000 x 4100 x 4100, dw added up in fp32, 179
    // us in launches of their own, 151 in turn (125 since a stage's loads lie over both its halves).  Long products are
    // held by power: idle CUs at a round's end let the others run faster, and 16384 x 3584 x 8192 measured 1505 in
    // turn against 1501.
    if (b->px.on && b->pw.on && !b->together) {
        Product x = b->px, w = b->pw;
        whole_tiles(&x, ag::kLinearTile256);
        whole_tiles(&w, ag::kLinearTile256);
        if (x.full_tiles <= 0x7fffff && w.full_tiles <= 0x7fffff) {
            const bool dx_first = x.us >= w.us;
            const double us = dx_first ? in_turn(x, &w, cus) : in_turn(w, &x, cus);
            const double apart = b->px.us + b->pw.us + (want_db ? 2.0 : 0.0) + 4.0 * (b->px.launches() + b->pw.launches() - 1);
            if (us < 0.87 * apart) {
                b->in_turn = true;
                b->dx_first = dx_first;
                x.programs = w.programs = cus;
                b->px = x;
                b->pw = w;
            }
        }
    }
    b->partial_offset = used;
    b->workspace = used + std::max({b->px.partial_bytes, b->pw.partial_bytes, b->rest.partial_bytes});
    b->db_alone = want_db && !b->px.on && !b->pw.on;
    b->launches = (b->slope ? 1 : 0) + (b->together || b->in_turn ? 1 : (b->db_alone ? 1 : 0) + b->px.launches() + b->pw.launches()) +
                  b->rest.launches() + (b->ow.pack ? 1 : 0) + (b->ox.pack ? 1 : 0);
    return AG_OK;
}

}  // namespace

extern "C" {

ag_status_t ag_plan_linear(const ag_linear_args_t* args, int num_cus, ag_linear_plan_t* plan)
{
    if (!plan) return fail(AG_ERR_INVALID_ARG, "plan is NULL");
    if (num_cus < 0) return fail(AG_ERR_INVALID_ARG, "num_cus %d < 0", num_cus);
    ag_status_t s;
    if (num_cus == 0 && (s = current_cus(&num_cus)) != AG_OK) return s;
    Forward f;
    if ((s = plan_forward(args, num_cus, &f)) != AG_OK) return s;
    ag_linear_plan_t p{};
    report(f.product, f.ox.pack, f.ow.pack, &p.product);
    const double M = static_cast<double>(args->M), N = static_cast<double>(args->N), K = static_cast<double>(args->K);
    p.workspace_bytes = f.workspace;
    if (f.product.on) {
        p.bytes_read = static_cast<uint64_t>(2 * (M * K + N * K + (args->bias ? N : 0) + (args->residual ? M * N : 0)));
        p.bytes_written = static_cast<uint64_t>(2 * M * N * (args->z ? 2 : 1));
        p.flops = 2 * M * N * K;
    }
    p.launches = f.launches;
    *plan = p;
    return ok();
}

ag_status_t ag_linear(const ag_linear_args_t* args, void* workspace, size_t workspace_bytes, void* stream_)
{
    int cus = 0;
    Forward f;
    // validation first (on any CU count), so that a bad argument is named even without a device
    ag_status_t s = plan_forward(args, 256, &f);
    if (s != AG_OK) return s;
    if (!f.product.on) return ok();
    if ((s = current_cus(&cus)) != AG_OK) return s;
    if (cus != 256) {
        f = Forward{};
        if ((s = plan_forward(args, cus, &f)) != AG_OK) return s;
    }
    s = check_workspace(workspace, workspace_bytes, f.workspace, {f.x, f.w, f.bias, f.residual, f.y, f.z});
    if (s != AG_OK) return s;
    const hipStream_t stream = static_cast<hipStream_t>(stream_);
    const int bf16 = args->dtype == AG_BF16;
    ag::LinearEpilogue e{};
    e.bias = static_cast<const uint16_t*>(args->bias);
    e.residual = static_cast<const uint16_t*>(args->residual);
    e.z = static_cast<uint16_t*>(args->z);
    e.out = args->y;
    e.ldr = f.residual.ld;
    e.ldz = f.z.ld;
    e.ldo = f.y.ld;
    e.act = args->act;
    if (f.product.stream) {
        ag::LinearStreamArgs a{static_cast<const uint16_t*>(args->x), static_cast<const uint16_t*>(args->w), f.x.ld, f.w.ld,
                               args->M, args->N, args->K, e};
        const hipError_t err = ag::launch_linear_stream(a, bf16, cus, stream);
        return err == hipSuccess ? ok() : fail_hip(err, "linear stream");
    }
    const uint16_t *A, *B;
    int64_t lda, ldb;
    if ((s = pack(f.ox, workspace, stream, &A, &lda)) != AG_OK) return s;
    if ((s = pack(f.ow, workspace, stream, &B, &ldb)) != AG_OK) return s;
    float* partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + f.partial_offset);
    s = run_product(f.product, gemm_args(f.product, A, lda, B, ldb, e, partial), bf16, stream);
    return s == AG_OK ? ok() : s;
}

ag_status_t ag_plan_linear_backward(const ag_linear_backward_args_t* args, int num_cus, ag_linear_plan_t* plan)
{
    if (!plan) return fail(AG_ERR_INVALID_ARG, "plan is NULL");
    if (num_cus < 0) return fail(AG_ERR_INVALID_ARG, "num_cus %d < 0", num_cus);
    ag_status_t s;
    if (num_cus == 0 && (s = current_cus(&num_cus)) != AG_OK) return s;
    Backward b;
    if ((s = plan_backward(args, num_cus, &b)) != AG_OK) return s;
    ag_linear_plan_t p{};
    report(b.px, false, b.ow.pack, &p.product);
    report(b.pw, false, b.ox.pack, &p.product_dw);
    const double M = static_cast<double>(args->M), N = static_cast<double>(args->N), K = static_cast<double>(args->K);
    const bool dx = !b.dx.empty(), dw = !b.dw.empty(), db = !b.db.empty();
    const int g = args->dw_dtype == AG_F32 ? 4 : 2;
    if (dx || dw || db) {
        const double grads = ((dw ? N * K : 0) + (db ? N : 0)) * g;
        p.bytes_read = static_cast<uint64_t>(2 * (M * N * (args->act != AG_ACT_NONE ? 2 : 1) + (dw ? M * K : 0) + (dx ? N * K : 0)) +
                                             (args->accumulate ? grads : 0));
        p.bytes_written = static_cast<uint64_t>(2 * (dx ? M * K : 0) + grads);
        p.flops = 2 * M * N * K * ((dx ? 1 : 0) + (dw ? 1 : 0));
    }
    p.workspace_bytes = b.workspace;
    p.launches = b.launches;
    *plan = p;
    return ok();
}

ag_status_t ag_linear_backward(const ag_linear_backward_args_t* args, void* workspace, size_t workspace_bytes, void* stream_)
{
    int cus = 0;
    Backward b;
    ag_status_t s = plan_backward(args, 256, &b);
    if (s != AG_OK) return s;
    if (b.launches == 0) return ok();
    if ((s = current_cus(&cus)) != AG_OK) return s;
    if (cus != 256) {
        b = Backward{};
        if ((s = plan_backward(args, cus, &b)) != AG_OK) return s;
    }
    s = check_workspace(workspace, workspace_bytes, b.workspace, {b.dy, b.z, b.x, b.w, b.dx, b.dw, b.db});
    if (s != AG_OK) return s;
    const hipStream_t stream = static_cast<hipStream_t>(stream_);
    const int bf16 = args->dtype == AG_BF16;
    char* ws = static_cast<char*>(workspace);
    float* sums = reinterpret_cast<float*>(ws + b.sums_offset);
    float* partial = reinterpret_cast<float*>(ws + b.partial_offset);
    const bool want_db = !b.db.empty();
    const uint16_t* dz = static_cast<const uint16_t*>(args->dy);
    int64_t lddz = args->M == 1 ? b.lddz : b.dy.ld;     // one row may have any stride
    if (b.slope) {
        ag::LinearSlopeArgs a{};
        a.dy = static_cast<const uint16_t*>(args->dy);
        a.z = args->act != AG_ACT_NONE ? static_cast<const uint16_t*>(args->z) : nullptr;
        a.dz = b.store_dz ? reinterpret_cast<uint16_t*>(ws + b.dz_offset) : nullptr;
        a.dz_rest = b.rest.on ? reinterpret_cast<uint16_t*>(ws + b.dz_rest_offset) : nullptr;
        a.sums = want_db ? sums : nullptr;
        a.lddy = b.dy.ld;
        a.ldz = b.z.ld;
        a.lddz = b.lddz;
        a.M = args->M;
        a.N = args->N;
        a.act = args->act;
        a.rows = static_cast<int32_t>(b.rows);
        const hipError_t e = ag::launch_linear_slope(a, bf16, stream);
        if (e != hipSuccess) return fail_hip(e, "linear slope");
        if (b.store_dz) {
            dz = a.dz;
            lddz = b.lddz;
        }
    }
    ag::LinearBiasGradArgs db{};
    if (want_db) {
        db.sums = sums;
        db.db = args->db;
        db.parts = b.parts;
        db.N = args->N;
        db.kind = args->dw_dtype == AG_F32 ? 2 : bf16;
        db.accumulate = args->accumulate;
    }
    ag::LinearGemmArgs dx{}, dw{};
    if (b.px.on) {
        const uint16_t* W;
        int64_t ldw;
        if ((s = pack(b.ow, workspace, stream, &W, &ldw)) != AG_OK) return s;
        ag::LinearEpilogue e{};
        e.out = args->dx;
        e.ldo = b.dx.ld;
        dx = gemm_args(b.px, dz, lddz, W, ldw, e, partial);
    }
    if (b.pw.on) {
        const uint16_t* X;
        int64_t ldx;
        if ((s = pack(b.ox, workspace, stream, &X, &ldx)) != AG_OK) return s;
        ag::LinearEpilogue e{};
        e.out = args->dw;
        e.ldo = b.dw.ld;
        e.out_f32 = args->dw_dtype == AG_F32;
        e.accumulate = args->accumulate;
        if (b.rest.on) {    // the small term first, on the earlier gradient if there is one; the other adds to it
            const uint16_t* dz_rest = reinterpret_cast<const uint16_t*>(ws + b.dz_rest_offset);
            if ((s = run_product(b.rest, gemm_args(b.rest, dz_rest, lddz, X, ldx, e, partial), bf16, stream)) != AG_OK) return s;
            e.accumulate = 1;
        }
        dw = gemm_args(b.pw, dz, lddz, X, ldx, e, partial);
    }
    if (b.together) {
        const hipError_t e = ag::launch_linear_grads(dx, dw, static_cast<int>(b.px.programs), static_cast<int>(b.pw.programs), db,
                                                     bf16, stream);
        return e == hipSuccess ? ok() : fail_hip(e, "linear gradients");
    }
    if (b.in_turn) {
        const hipError_t e = ag::launch_linear_grads_in_turn(dx, dw, b.dx_first, static_cast<int>(b.px.programs), db, bf16, stream);
        return e == hipSuccess ? ok() : fail_hip(e, "linear gradients");
    }
    if (b.db_alone) {
        const hipError_t e = ag::launch_linear_bias_grad(db, stream);
        if (e != hipSuccess) return fail_hip(e, "linear bias gradient");
    }
    (b.pw.on ? dw : dx).db = db;    // beside the product that comes last
    if (b.px.on && (s = run_product(b.px, dx, bf16, stream)) != AG_OK) return s;
    if (b.pw.on && (s = run_product(b.pw, dw, bf16, stream)) != AG_OK) return s;
    return ok();
}

}  // extern "C"
