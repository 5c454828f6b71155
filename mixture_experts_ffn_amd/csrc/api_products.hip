// api_products.hip — the C ABI of the experts' products on their own (grouped
// products and their gradients, products in 8-bit integers) and of the layer on
// int8 weights: validation, workspace layout, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "group_view.h"
#include "host.h"
#include "i8.h"
#include "kernels.h"
#include "moe_ffn.h"

using namespace moe::host;

namespace {

// Lays out consecutive arrays of a workspace.
struct Taker {
    size_t off = 0;
    size_t operator()(size_t bytes)
    {
        const size_t at = off;
        off = align_up(off + (bytes ? bytes : 1));
        return at;
    }
};

// What the grouped kernels walk, in a workspace (group.hip).
struct GroupLayout {
    size_t offsets, mtile_off, mtile_expert, tickets, order, alt_off, alt_expert;
    int64_t max_mtiles;
    void lay(Taker &take, int64_t M, int64_t E, int min_rows)
    {
        max_mtiles = moe::max_mtiles_bound(M, (int)E, min_rows);
        offsets = take(sizeof(int32_t) * (size_t)(E + 1));
        mtile_off = take(sizeof(int32_t) * (size_t)(E + 1));
        mtile_expert = take(sizeof(int32_t) * (size_t)max_mtiles);
        tickets = take(sizeof(int32_t) * 16);
        order = take(sizeof(int32_t) * (size_t)E);
        // second tables: 128-row tiles
        alt_off = take(sizeof(int32_t) * (size_t)(E + 1));
        alt_expert = take(sizeof(int32_t) * (size_t)moe::max_mtiles_bound(M, (int)E, 128));
    }
    moe::GroupSetup setup(void *ws, const void *given, int offsets_dtype, int64_t M, int64_t E, int BM) const
    {
        moe::GroupSetup g{};
        g.offsets = given;
        g.off64 = offsets_dtype == MOE_FFN_I64;
        g.M = M;
        g.E = (int)E;
        g.BM = BM;
        g.out_offsets = at<int32_t>(ws, offsets);
        g.mtile_off = at<int32_t>(ws, mtile_off);
        g.mtile_expert = at<int32_t>(ws, mtile_expert);
        g.tickets = at<int32_t>(ws, tickets);
        return g;
    }
};

constexpr int64_t kMaxRows = int64_t(1) << 30; // row and tile numbers stay within int32

// blocks: of columns, `width` (32 or 64) wide, of the kernel that has most
int check_groups(int64_t M, int64_t E, int offsets_dtype, int64_t blocks, int width)
{
    if (M < 0 || M > kMaxRows)
        return fail(MOE_FFN_ERR_SHAPE, "M must be in [0, 2^30] (got %lld)", (long long)M);
    if (E < 1 || E > 1024)
        return fail(MOE_FFN_ERR_SHAPE, "E must be in [1, 1024] (got %lld)", (long long)E);
    if (offsets_dtype != MOE_FFN_I32 && offsets_dtype != MOE_FFN_I64)
        return fail(MOE_FFN_ERR_DTYPE, "offsets_dtype must be I32 or I64 (got %d)", offsets_dtype);
    if (moe::max_mtiles_bound(M, (int)E, 32) * blocks >= (int64_t(1) << 31))
        return fail(MOE_FFN_ERR_SHAPE, "too many output tiles: M / 32 + E times columns / %d must be "
                                       "< 2^31", width);
    return MOE_FFN_OK;
}

// ---- grouped products -----------------------------------------------------------

int validate_grouped(const moe_ffn_grouped *g)
{
    if (!g)
        return fail(MOE_FFN_ERR_NULL, "product description is NULL");
    if (g->dtype != MOE_FFN_F32 && g->dtype != MOE_FFN_BF16)
        return fail(MOE_FFN_ERR_DTYPE, "dtype must be F32 or BF16 (got %d)", g->dtype);
    if (g->Kd < 8 || g->Kd % 8 || g->N < 8 || g->N % 8)
        return fail(MOE_FFN_ERR_SHAPE, "Kd and N must be positive multiples of 8 (got %lld, %lld)",
                    (long long)g->Kd, (long long)g->N);
    if (g->Kd >= (int64_t(1) << 31) / g->N)
        return fail(MOE_FFN_ERR_SHAPE, "Kd*N must be < 2^31");
    if (g->x_stride < g->Kd || g->x_stride % 8 || g->x_stride >= (int64_t(1) << 31))
        return fail(MOE_FFN_ERR_SHAPE, "x_stride must be a multiple of 8, Kd at least and < 2^31 (got %lld)",
                    (long long)g->x_stride);
    if (g->transposed != 0 && g->transposed != 1)
        return fail(MOE_FFN_ERR_SHAPE, "transposed must be 0 or 1 (got %d)", g->transposed);
    return check_groups(g->M, g->E, g->offsets_dtype, (std::max(g->Kd, g->N) + 63) / 64, 64);
}

// At most BM - 1 rows of padding a group.
int64_t tiles_of(int64_t M, int64_t E, int64_t BM) { return (M + std::min(M, E) * (BM - 1)) / BM; }

// gemm_rows.hip serves products of up to so many tiles of 32 x 256: it reads the weights
// once for each 32 rows of a group, but cuts a tile's columns and contraction finer,
// where the kernels of taller tiles leave most CUs without one.  Both sides in us with
// weights out of memory ([K, N]; [N, K] weights, those kernels in brackets): 1 row of 7168
// x 4096 30 (79); 24 (85), 128 rows 47 (134); 50 (110), 256 70 (132); 91 (107), 512 133 (131);
// 167 (106); 8 rows over 8 of 32 groups 88 (117); 108 (122); 4096 x 1536, 16 groups, 256 rows
// 51 (63); 62 (70), 512 rows 68 (65); 84 (67); 512 x 512 x 2048 over 4 groups 12.6 (19); 16 (17).
constexpr int64_t kFewTiles = 160;
// fp32, where the other kernel (gemm_f32.hip, in brackets) is bound by the length of its
// chain of steps: up to 16 mean rows a group, or 64 in all, and more than 1 MB of weights. 1
// row of 4096 x 4096 25 (67); 24 (68), 32 rows 36 (68); 45 (70), 8 rows over 8 of 32 groups of
// 2048 x 2816 41 (83); 31 (81), 400 of 512 x 4096 over 32 67 (100); 62 (121), but 300 of 2048 x
// 2048 over 8 74 (69); 78 (67), 1202 of 264 x 200 over 6 20 (9); 10 (8), 16 of 256 x 256 8.7 (6.2);
// 7.7 (6.3).
bool few_tiles(int dtype, int64_t M, int64_t E, int64_t K, int64_t N)
{
    if (dtype != MOE_FFN_F32)
        return tiles_of(M, E, 32) * ((N + 255) / 256) <= kFewTiles;
    return (M <= 16 * E || M <= 64) && std::min(M, E) * K * N > (1 << 18) &&
           K * N < (int64_t(1) << 30); // a group's weights below 4 GiB
}

// Whether calls of these sizes may read the set-up's tables, and so need a workspace.
bool needs_setup(const moe_ffn_grouped &g)
{
    return g.dtype != MOE_FFN_F32 || g.E > moe::kViewGroups;
}

struct GroupedLayout {
    GroupLayout groups{};
    size_t total;
};
GroupedLayout grouped_layout(const moe_ffn_grouped &g)
{
    GroupedLayout L;
    Taker take;
    if (needs_setup(g))
        L.groups.lay(take, g.M, g.E, few_tiles(g.dtype, g.M, g.E, g.Kd, g.N) || few_tiles(g.dtype, g.M, g.E, g.N, g.Kd) ? 16 : 64);
    L.total = take.off;
    return L;
}

// A product of rows and weights: out [M, N] = a [M, K] (rows lda apart) . W[e],
// W[e] of [K, N], or of [N, K] if nt.
struct RowsProduct {
    const void *a, *w;
    void *out;
    int64_t M, K, N, lda;
    bool nt;
};

// The kernels and the tile heights for a product: gemm_rows.hip for few tiles (above),
// with 16 or 32 rows (48 x 2048 x 2816 over 4 groups by 16 rows 16.2 us, by 32 22.8); else
// by the mean rows of a group: up to 64 tiles of 64 rows, up to 256 of 128, from there on
// by the model in kernels.h: for what the host knows, routed rows that split evenly, or,
// where a product is long beside a launch (a skewed routing decides 10 % of it), by the
// set-up kernel.
struct RowsPlan {
    int BM;          // rows of an M-tile; both: of the first tables
    bool few;        // gemm_rows.hip
    bool fast;       // gemm_mfma.hip serves the low tiles
    bool big, both;  // 256-row tiles; either, as the set-up decides
    moe::TileModel model;
    // the product forms the groups by itself
    bool alone(int64_t E) const { return few && E <= moe::kViewGroups; }
};
RowsPlan plan_rows(int dtype, const RowsProduct &p, int64_t E, int num_cus)
{
    RowsPlan r{64, false, false, false, false, {}};
    if (few_tiles(dtype, p.M, E, p.K, p.N)) {
        r.few = true;
        r.BM = p.M <= 16 * E ? 16 : 32;
        return r;
    }
    if (dtype == MOE_FFN_F32)
        return r; // moe::kF32Rows
    const double rows = (double)p.M / (double)E;
    r.fast = !p.nt && p.lda == p.K && moe::fast_gemm_supported(1, p.N, p.K);
    r.BM = rows <= 64 ? 64 : 128;
    if (rows > 256 && p.K % 32 == 0 && p.K >= 128 &&
        p.M * p.lda * 2 < (int64_t(1) << 32)) { // 32-bit row offsets
        r.model = {(float)((p.N + 255) / 256) / (float)num_cus, r.fast};
        r.both = E > 1 && (double)p.M * (double)p.N * (double)p.K > 6e10; // 100 us and more
        r.big = r.both || moe::tall_tiles(r.model, (float)p.M, (float)p.M / 256 + 0.5f * (float)E,
                                          (float)p.M / 128 + 0.5f * (float)E);
    }
    if (r.big)
        r.BM = 256;
    return r;
}

hipError_t run_rows(int dtype, const RowsProduct &p, const RowsPlan &plan, const moe::GroupSource &src,
                    const GroupLayout &G, void *ws, int num_cus, hipStream_t s)
{
    const int64_t E = src.E;
    const int32_t *offsets = at<int32_t>(ws, G.offsets), *mtile_off = at<int32_t>(ws, G.mtile_off),
                  *mtile_expert = at<int32_t>(ws, G.mtile_expert);
    if (plan.few) {
        moe::RowsArgs a{};
        a.A = p.a;
        a.W = p.w;
        a.C = p.out;
        a.src = src;
        if (E > moe::kViewGroups) {
            a.offsets = offsets;
            a.mtile_off = mtile_off;
            a.mtile_expert = mtile_expert;
        }
        a.E = (int)E;
        a.N = (int)p.N;
        a.K = (int)p.K;
        a.lda = p.lda;
        a.max_mtiles = tiles_of(p.M, E, plan.BM);
        a.once = moe::weights_once(p.M, E, plan.BM);
        return moe::launch_rows(dtype == MOE_FFN_BF16, p.nt, plan.BM, a, num_cus, s);
    }
    if (dtype == MOE_FFN_F32) {
        moe::F32Grouped a{};
        a.A = static_cast<const float *>(p.a);
        a.B = static_cast<const float *>(p.w);
        a.C = static_cast<float *>(p.out);
        a.src = src;
        if (E > moe::kViewGroups) {
            a.offsets = offsets;
            a.mtile_off = mtile_off;
            a.mtile_expert = mtile_expert;
        }
        a.E = (int)E;
        a.N = (int)p.N;
        a.K = (int)p.K;
        a.lda = p.lda;
        a.ldb = p.nt ? p.K : p.N;
        a.max_mtiles = (int)moe::max_mtiles_bound(p.M, (int)E, moe::kF32Rows);
        return moe::launch_f32_grouped(p.nt ? moe::F32_NT : moe::F32_NN, a, num_cus, s);
    }
    moe::FastFwdArgs f{};
    f.w2 = p.w;
    f.act = const_cast<void *>(p.a);
    f.o = p.out;
    f.offsets = offsets;
    f.mtile_off = mtile_off;
    f.mtile_expert = mtile_expert;
    f.tickets = at<int32_t>(ws, G.tickets);
    f.T = (int)p.M;
    f.H = (int)p.N;
    f.I = (int)p.K;
    f.E = (int)E;
    f.K = 1;
    f.drop_mt = -1;
    f.lda = (int)p.lda;
    if (plan.big) {
        const hipError_t err = moe::launch_grouped_big(p.nt, f, num_cus, s);
        if (err != hipSuccess || !plan.both)
            return err;
        mtile_off = f.mtile_off = at<int32_t>(ws, G.alt_off);
        mtile_expert = f.mtile_expert = at<int32_t>(ws, G.alt_expert);
    }
    const int BM = plan.big ? 128 : plan.BM;
    if (plan.fast) {
        f.max_mtiles = (int)moe::max_mtiles_bound(p.M, (int)E, BM);
        return moe::launch_fast_fwd(moe::FAST_G2, BM, f, num_cus, s);
    }
    moe::EngineArgs a{};
    a.A = static_cast<const moe::bf16_t *>(p.a);
    a.B = static_cast<const moe::bf16_t *>(p.w);
    a.C = static_cast<moe::bf16_t *>(p.out);
    a.offsets = offsets;
    a.mtile_off = mtile_off;
    a.mtile_expert = mtile_expert;
    a.topk = 1;
    a.E = (int)E;
    a.Er = (int)E;
    a.N = (int)p.N;
    a.Kd = (int)p.K;
    a.lda = (int)p.lda;
    a.ldb = (int)(p.nt ? p.K : p.N);
    a.ldc = (int)p.N;
    a.b_estride = p.K * p.N;
    return moe::launch_engine(p.nt ? moe::ENG_B4 : moe::ENG_F2, BM, a, num_cus, s);
}

// The set-up's side of a plan.
void set_plan(moe::GroupSetup &set, const RowsPlan &plan, const GroupLayout &G, void *ws)
{
    if (!plan.both)
        return;
    set.alt.mtile_off = at<int32_t>(ws, G.alt_off);
    set.alt.mtile_expert = at<int32_t>(ws, G.alt_expert);
    set.alt.model = plan.model;
}

} // namespace

extern "C" {

int moe_ffn_grouped_workspace_size(const moe_ffn_grouped *g, size_t *ws_bytes)
{
    clear_error();
    int rc = validate_grouped(g);
    if (rc)
        return rc;
    if (!ws_bytes)
        return fail(MOE_FFN_ERR_NULL, "ws_bytes is NULL");
    *ws_bytes = grouped_layout(*g).total;
    return MOE_FFN_OK;
}

int moe_ffn_grouped_mm(const moe_ffn_grouped *g, const void *x, const void *weight,
                       const void *offsets, void *y, void *ws, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc = validate_grouped(g);
    if (rc)
        return rc;
    if (g->M == 0)
        return MOE_FFN_OK;
    const GroupedLayout L = grouped_layout(*g);
    if ((rc = check_ptr(x, "x")) || (rc = check_ptr(weight, "weight")) ||
        (rc = check_ptr(offsets, "offsets", g->offsets_dtype == MOE_FFN_I64 ? 8 : 4)) ||
        (rc = check_ptr(y, "y")) || (L.total && (rc = check_ptr(ws, "ws"))))
        return rc;
    if (ws_bytes < L.total)
        return fail(MOE_FFN_ERR_WORKSPACE, "workspace too small: %zu < %zu", ws_bytes, L.total);
    int num_cus = 0;
    if ((rc = check_device(&num_cus)))
        return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const RowsProduct p{x, weight, y, g->M, g->Kd, g->N, g->x_stride, g->transposed == 1};
    const RowsPlan plan = plan_rows(g->dtype, p, g->E, num_cus);
    moe::GroupSetup set = L.groups.setup(ws, offsets, g->offsets_dtype, g->M, g->E, plan.BM);
    set_plan(set, plan, L.groups, ws);
    set.out = y;
    set.out_row = g->N * (int64_t)elem_size(g->dtype);
    const moe::GroupSource src{offsets, set.off64, g->M, set.E};
    if (needs_setup(*g) && !plan.alone(g->E))
        HIP_TRY(moe::launch_group_setup(set, s), "group set-up launch");
    HIP_TRY(run_rows(g->dtype, p, plan, src, L.groups, ws, num_cus, s), "grouped product launch");
    return MOE_FFN_OK;
}

int moe_ffn_grouped_mm_bwd(const moe_ffn_grouped *g, const void *dy, const void *x,
                           const void *weight, const void *offsets, void *dx, void *d_weight,
                           void *ws, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc = validate_grouped(g);
    if (rc)
        return rc;
    const GroupedLayout L = grouped_layout(*g);
    const size_t item = elem_size(g->dtype);
    if (d_weight && (rc = check_ptr(d_weight, "d_weight")))
        return rc;
    if (g->M > 0) {
        if ((rc = check_ptr(dy, "dy")) ||
            (rc = check_ptr(offsets, "offsets", g->offsets_dtype == MOE_FFN_I64 ? 8 : 4)) ||
            (L.total && (rc = check_ptr(ws, "ws"))) || (dx && ((rc = check_ptr(dx, "dx")) ||
                                                  (rc = check_ptr(weight, "weight")))) ||
            (d_weight && (rc = check_ptr(x, "x"))))
            return rc;
        if (ws_bytes < L.total)
            return fail(MOE_FFN_ERR_WORKSPACE, "workspace too small: %zu < %zu", ws_bytes, L.total);
    }
    int num_cus = 0;
    if ((rc = check_device(&num_cus)))
        return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->M == 0) {
        if (d_weight)
            HIP_TRY(moe::launch_zero_fill(d_weight, (size_t)(g->E * g->Kd * g->N) * item, s),
                    "zero launch");
        return MOE_FFN_OK;
    }
    if (!dx && !d_weight)
        return MOE_FFN_OK;
    // dx = dy . W^T: the weights are read along the other axis than the forward's
    const RowsProduct p{dy, weight, dx, g->M, g->N, g->Kd, g->N, g->transposed == 0};
    const RowsPlan plan = plan_rows(g->dtype, p, g->E, num_cus);
    moe::GroupSetup set = L.groups.setup(ws, offsets, g->offsets_dtype, g->M, g->E, plan.BM);
    set_plan(set, plan, L.groups, ws);
    set.out = dx;
    set.out_row = g->Kd * (int64_t)item;
    // the weight's gradient: a^T b with a's columns the weight's rows
    const int wm = (int)(g->transposed ? g->N : g->Kd), wn = (int)(g->transposed ? g->Kd : g->N);
    const void *a = g->transposed ? dy : x, *b = g->transposed ? x : dy;
    const int64_t lda = g->transposed ? g->N : g->x_stride, ldb = g->transposed ? g->x_stride : g->N;
    if (d_weight && g->dtype == MOE_FFN_BF16)
        set.order = at<int32_t>(ws, L.groups.order);
    const moe::GroupSource src{offsets, set.off64, g->M, set.E};
    if (needs_setup(*g) && (d_weight || !plan.alone(g->E)))
        HIP_TRY(moe::launch_group_setup(set, s), "group set-up launch");
    if (dx)
        HIP_TRY(run_rows(g->dtype, p, plan, src, L.groups, ws, num_cus, s), "input gradient launch");
    if (!d_weight)
        return MOE_FFN_OK;
    const int32_t *o = at<int32_t>(ws, L.groups.offsets);
    if (g->dtype == MOE_FFN_F32) {
        moe::F32Grouped w{};
        w.A = static_cast<const float *>(a);
        w.B = static_cast<const float *>(b);
        w.C = static_cast<float *>(d_weight);
        w.src = src;
        w.offsets = needs_setup(*g) ? o : nullptr;
        w.E = (int)g->E;
        w.M = wm;
        w.N = wn;
        w.lda = lda;
        w.ldb = ldb;
        HIP_TRY(moe::launch_f32_grouped(moe::F32_TN, w, num_cus, s), "weight gradient launch");
        return MOE_FFN_OK;
    }
    moe::EngineArgs w{};
    w.A = static_cast<const moe::bf16_t *>(a);
    w.B = static_cast<const moe::bf16_t *>(b);
    w.C = static_cast<moe::bf16_t *>(d_weight);
    w.offsets = o;
    w.topk = 1;
    w.E = (int)g->E;
    w.Er = (int)g->E;
    w.M = wm;
    w.N = wn;
    w.lda = (int)lda;
    w.ldb = (int)ldb;
    w.order = set.order;
    HIP_TRY(moe::launch_engine(moe::ENG_GW, 128, w, num_cus, s), "weight gradient launch");
    return MOE_FFN_OK;
}

} // extern "C"

// ---- int8 -------------------------------------------------------------------------

namespace {

constexpr int64_t kI8MaxK = 131072; // 128 * 127 * Kd < 2^31

struct I8WeightLayout {
    size_t scales, total; // codes start at 0
};
I8WeightLayout i8_weight_layout(int64_t E, int64_t Kd, int64_t N, int panels)
{
    const moe::I8Dims d(Kd, N / panels);
    const size_t tiles = (size_t)E * panels * d.NT;
    I8WeightLayout L;
    L.scales = align_up(tiles * d.KS * 1024);
    L.total = align_up(L.scales + tiles * 32 * sizeof(float));
    return L;
}

int validate_i8_weight(const moe_ffn_int8_weight *w, bool dtype_used = true)
{
    if (!w)
        return fail(MOE_FFN_ERR_NULL, "weight description is NULL");
    if (dtype_used && w->dtype != MOE_FFN_F32 && w->dtype != MOE_FFN_BF16)
        return fail(MOE_FFN_ERR_DTYPE, "dtype must be F32 or BF16 (got %d)", w->dtype);
    if (w->E < 1 || w->E > 1024)
        return fail(MOE_FFN_ERR_SHAPE, "E must be in [1, 1024] (got %lld)", (long long)w->E);
    if (w->panels != 1 && w->panels != 2)
        return fail(MOE_FFN_ERR_SHAPE, "panels must be 1 or 2 (got %d)", w->panels);
    if (w->Kd < 8 || w->Kd % 8 || w->Kd > kI8MaxK)
        return fail(MOE_FFN_ERR_SHAPE, "Kd must be a positive multiple of 8 and <= 131072 (got %lld)",
                    (long long)w->Kd);
    if (w->N < 8 || w->N % (8 * w->panels) || w->N >= (int64_t(1) << 31))
        return fail(MOE_FFN_ERR_SHAPE, "N must be a positive multiple of 8 * panels (got %lld)",
                    (long long)w->N);
    if (w->Kd * w->N >= (int64_t(1) << 31))
        return fail(MOE_FFN_ERR_SHAPE, "Kd*N must be < 2^31");
    return MOE_FFN_OK;
}

// The GEMM addresses a group's codes, 32 columns and 64 values at least, by 32 bits.
int check_i8_group(int64_t Kd, int64_t N, int panels)
{
    const moe::I8Dims d(Kd, N / panels);
    if ((int64_t)panels * d.NT * d.KS * 1024 >= (int64_t(1) << 32))
        return fail(MOE_FFN_ERR_SHAPE, "one matrix's packed weights must be below 4 GiB");
    return MOE_FFN_OK;
}

int check_packed(const moe_ffn_int8_weight *w, const void *packed, size_t packed_bytes)
{
    const int rc = check_ptr(packed, "packed");
    if (rc)
        return rc;
    const size_t need = i8_weight_layout(w->E, w->Kd, w->N, w->panels).total;
    if (packed_bytes < need)
        return fail(MOE_FFN_ERR_WORKSPACE, "packed buffer too small: %zu < %zu", packed_bytes, need);
    return MOE_FFN_OK;
}

int validate_i8_rows(int64_t M, int64_t Kd, int64_t stride, int dtype)
{
    if (dtype != MOE_FFN_F32 && dtype != MOE_FFN_BF16)
        return fail(MOE_FFN_ERR_DTYPE, "dtype must be F32 or BF16 (got %d)", dtype);
    if (M < 0 || M > kMaxRows)
        return fail(MOE_FFN_ERR_SHAPE, "M must be in [0, 2^30] (got %lld)", (long long)M);
    if (Kd < 8 || Kd % 8 || Kd > kI8MaxK)
        return fail(MOE_FFN_ERR_SHAPE, "Kd must be a positive multiple of 8 and <= 131072 (got %lld)",
                    (long long)Kd);
    if (stride < Kd || stride % 8)
        return fail(MOE_FFN_ERR_SHAPE, "x_stride must be a multiple of 8 and Kd at least (got %lld)",
                    (long long)stride);
    return MOE_FFN_OK;
}

// Rows of an M-tile, by the mean rows of a group and the number of 32 x 32 tiles (whole
// layers in us, both sides of each rule):
//  - up to 20 rows: 32, which pads least (64 tokens through 16 experts of 4096 x 1536,
//    top 4: 76 against 81 with 64);
//  - up to 1536 tiles: 32, where the waves share a tile's contraction (512 x 1024 x 512,
//    8 experts, top 2: 34 against 42 with 128);
//  - up to 48 rows, most groups fit 64 (512 x 2048 x 1408, 64 experts, top 6: 153 against
//    161; 128 x 7168 x 2048, 32, top 8: 267 and 301);
//  - up to 5000 tiles there are too few of 128 (2048 x 1024 x 512, 8 experts, top 2: 50
//    and 54);
//  - else 128 (256 x 4096 x 1536, 16 experts, top 4: 106 against 125 with 64; 768 x 2048 x
//    1408, 64, top 6: 176 and 197; 4096: 408 and 483).
int i8_tile_rows(int64_t M, int64_t E, int64_t widest)
{
    const double rows = (double)M / (double)E;
    const int64_t tiles = moe::max_mtiles_bound(M, (int)E, 32) * ((widest + 31) / 32);
    return rows <= 20 || tiles <= 1536 ? 32 : rows <= 48 || tiles <= 5000 ? 64 : 128;
}

struct I8ProductLayout {
    int BM;
    GroupLayout groups{}; // more groups than a wave's lanes
    size_t total;
};
I8ProductLayout i8_product_layout(const moe_ffn_int8_product &p)
{
    I8ProductLayout L;
    L.BM = i8_tile_rows(p.M, p.weight.E, p.weight.N);
    Taker take;
    if (p.weight.E > moe::kViewGroups)
        L.groups.lay(take, p.M, p.weight.E, L.BM);
    L.total = take.off;
    return L;
}

int validate_i8_product(const moe_ffn_int8_product *p)
{
    if (!p)
        return fail(MOE_FFN_ERR_NULL, "product description is NULL");
    int rc = validate_i8_weight(&p->weight, false);
    if (rc)
        return rc;
    if (p->out_dtype != MOE_FFN_F32 && p->out_dtype != MOE_FFN_BF16)
        return fail(MOE_FFN_ERR_DTYPE, "out_dtype must be F32 or BF16 (got %d)", p->out_dtype);
    if ((rc = check_i8_group(p->weight.Kd, p->weight.N, p->weight.panels)))
        return rc;
    const moe::I8Dims d(p->weight.Kd, p->weight.N / p->weight.panels);
    return check_groups(p->M, p->weight.E, p->offsets_dtype, (int64_t)p->weight.panels * d.NT, 32);
}

struct I8FwdLayout {
    moe::RoutePlan rp;
    int BM;
    int64_t max_mtiles;
    size_t status, hist, bad, counts, offsets, mtile_off, mtile_expert, sorted_slot, slot_pos;
    size_t x_codes, x_scales, act, act_codes, act_scales, o, total;
};

void i8_fwd_layout(const moe_ffn_problem &p, I8FwdLayout &L)
{
    const int64_t TK = p.T * p.K;
    const int E = (int)p.E;
    L.BM = i8_tile_rows(TK, E, std::max(p.H, p.I));
    L.rp = moe::make_route_plan(TK, E);
    L.max_mtiles = moe::max_mtiles_bound(TK, E, L.BM);
    Taker take;
    L.status = take(sizeof(int32_t));
    L.hist = take(sizeof(int32_t) * (size_t)E * (size_t)L.rp.NB);
    L.bad = take(sizeof(int32_t) * (size_t)L.rp.NB);
    L.counts = take(sizeof(int32_t) * (size_t)E);
    L.offsets = take(sizeof(int32_t) * (size_t)(E + 1));
    L.mtile_off = take(sizeof(int32_t) * (size_t)(E + 1));
    L.mtile_expert = take(sizeof(int32_t) * (size_t)L.max_mtiles);
    // padded like the bf16 forward's (routing fills whole blocks of it)
    L.sorted_slot = take(sizeof(int32_t) * ((size_t)TK + 256));
    L.slot_pos = take(sizeof(int32_t) * (size_t)TK);
    L.x_codes = take((size_t)p.T * moe::I8Dims(p.H, 8).row());
    L.x_scales = take(sizeof(float) * (size_t)p.T);
    L.act = take(sizeof(float) * (size_t)TK * (size_t)p.I);
    L.act_codes = take((size_t)TK * moe::I8Dims(p.I, 8).row());
    L.act_scales = take(sizeof(float) * (size_t)TK);
    L.o = take(sizeof(float) * (size_t)TK * (size_t)p.H);
    L.total = take.off;
}

int validate_i8_fwd(const moe_ffn_problem *p, uint32_t flags)
{
    int rc = validate_problem(p);
    if (rc)
        return rc;
    if (p->dtype != MOE_FFN_BF16)
        return fail(MOE_FFN_ERR_DTYPE, "the int8 forward supports BF16 only (got dtype %d)", p->dtype);
    if (p->Is != 0)
        return fail(MOE_FFN_ERR_SHAPE, "the int8 forward takes no shared expert (Is must be 0)");
    if (p->H > kI8MaxK || p->I > kI8MaxK)
        return fail(MOE_FFN_ERR_SHAPE, "H and I must be <= 131072");
    if (p->T * moe::I8Dims(p->H, 8).row() >= (int64_t(1) << 32))
        return fail(MOE_FFN_ERR_SHAPE, "T*H must be < 2^32 (4 GiB of token codes)");
    if (p->T >= (int64_t(1) << 24)) // a workgroup of 256 threads a token in the combine
        return fail(MOE_FFN_ERR_SHAPE, "T must be < 2^24 (got %lld)", (long long)p->T);
    if ((rc = check_i8_group(p->H, 2 * p->I, 2)) || (rc = check_i8_group(p->I, p->H, 1)))
        return rc;
    const int64_t blocks = std::max((p->H + 31) / 32, 2 * ((p->I + 31) / 32));
    if ((rc = check_groups(p->T * p->K, p->E, MOE_FFN_I32, blocks, 32)))
        return rc;
    if (flags & ~(MOE_FFN_CHECK_IDS | MOE_FFN_CHECK_STATUS))
        return fail(MOE_FFN_ERR_SHAPE, "flags: only CHECK_IDS and CHECK_STATUS apply (got 0x%x)", flags);
    return MOE_FFN_OK;
}

// An id out of range, once the stream has reached here.
int check_ids(const int32_t *status, int64_t E, hipStream_t s)
{
    int32_t st = 0;
    HIP_TRY(hipMemcpyAsync(&st, status, sizeof st, hipMemcpyDeviceToHost, s), "status copy");
    HIP_TRY(hipStreamSynchronize(s), "stream sync");
    if (st & moe::MOE_DEV_BAD_ID)
        return fail(MOE_FFN_ERR_EXPERT_ID, "topk_ids holds a value outside [0, %lld)", (long long)E);
    return MOE_FFN_OK;
}

} // namespace

extern "C" {

int moe_ffn_int8_weight_size(const moe_ffn_int8_weight *w, size_t *packed_bytes)
{
    clear_error();
    const int rc = validate_i8_weight(w);
    if (rc)
        return rc;
    if (!packed_bytes)
        return fail(MOE_FFN_ERR_NULL, "packed_bytes is NULL");
    *packed_bytes = i8_weight_layout(w->E, w->Kd, w->N, w->panels).total;
    return MOE_FFN_OK;
}

int moe_ffn_int8_quantize(const moe_ffn_int8_weight *w, const void *weight, void *packed,
                          size_t packed_bytes, void *stream)
{
    clear_error();
    int rc = validate_i8_weight(w);
    if (rc || (rc = check_ptr(weight, "weight")) || (rc = check_packed(w, packed, packed_bytes)) ||
        (rc = check_device()))
        return rc;
    const I8WeightLayout L = i8_weight_layout(w->E, w->Kd, w->N, w->panels);
    HIP_TRY(moe::launch_i8_quantize_weight(w->dtype, weight, packed, at<float>(packed, L.scales), w->E,
                                           w->Kd, w->N, w->panels, static_cast<hipStream_t>(stream)),
            "quantisation launch");
    return MOE_FFN_OK;
}

int moe_ffn_int8_pack(const moe_ffn_int8_weight *w, const void *codes, const float *scales,
                      void *packed, size_t packed_bytes, void *stream)
{
    clear_error();
    int rc = validate_i8_weight(w);
    if (rc || (rc = check_ptr(codes, "codes")) || (rc = check_ptr(scales, "scales", 4)) ||
        (rc = check_packed(w, packed, packed_bytes)) || (rc = check_device()))
        return rc;
    const I8WeightLayout L = i8_weight_layout(w->E, w->Kd, w->N, w->panels);
    HIP_TRY(moe::launch_i8_pack_weight(codes, scales, packed, at<float>(packed, L.scales), w->E, w->Kd,
                                       w->N, w->panels, static_cast<hipStream_t>(stream)),
            "packing launch");
    return MOE_FFN_OK;
}

int moe_ffn_int8_dequantize(const moe_ffn_int8_weight *w, const void *packed, size_t packed_bytes,
                            void *weight, void *stream)
{
    clear_error();
    int rc = validate_i8_weight(w);
    if (rc || (rc = check_ptr(weight, "weight")) || (rc = check_packed(w, packed, packed_bytes)) ||
        (rc = check_device()))
        return rc;
    const I8WeightLayout L = i8_weight_layout(w->E, w->Kd, w->N, w->panels);
    HIP_TRY(moe::launch_i8_dequantize_weight(w->dtype, packed,
                                             at<float>(const_cast<void *>(packed), L.scales), weight,
                                             w->E, w->Kd, w->N, w->panels,
                                             static_cast<hipStream_t>(stream)),
            "dequantisation launch");
    return MOE_FFN_OK;
}

int moe_ffn_int8_row_bytes(int64_t Kd, int64_t *row_bytes)
{
    clear_error();
    const int rc = validate_i8_rows(0, Kd, Kd, MOE_FFN_BF16);
    if (rc)
        return rc;
    if (!row_bytes)
        return fail(MOE_FFN_ERR_NULL, "row_bytes is NULL");
    *row_bytes = moe::I8Dims(Kd, 8).row();
    return MOE_FFN_OK;
}

int moe_ffn_int8_quantize_rows(const moe_ffn_int8_rows *r, const void *x, void *codes,
                               float *scales, void *stream)
{
    clear_error();
    if (!r)
        return fail(MOE_FFN_ERR_NULL, "rows description is NULL");
    int rc = validate_i8_rows(r->M, r->Kd, r->x_stride, r->dtype);
    if (rc || r->M == 0)
        return rc;
    if ((rc = check_ptr(x, "x")) || (rc = check_ptr(codes, "codes")) ||
        (rc = check_ptr(scales, "scales", 4)) || (rc = check_device()))
        return rc;
    HIP_TRY(moe::launch_i8_quantize_rows(r->dtype, x, r->x_stride, codes, scales, r->M, r->Kd,
                                         static_cast<hipStream_t>(stream)),
            "row quantisation launch");
    return MOE_FFN_OK;
}

int moe_ffn_int8_mm_workspace_size(const moe_ffn_int8_product *p, size_t *ws_bytes)
{
    clear_error();
    const int rc = validate_i8_product(p);
    if (rc)
        return rc;
    if (!ws_bytes)
        return fail(MOE_FFN_ERR_NULL, "ws_bytes is NULL");
    *ws_bytes = i8_product_layout(*p).total;
    return MOE_FFN_OK;
}

int moe_ffn_int8_mm(const moe_ffn_int8_product *p, const void *codes, const float *scales,
                    const void *packed, size_t packed_bytes, const void *offsets, void *y,
                    void *ws, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc = validate_i8_product(p);
    if (rc)
        return rc;
    if (!offsets && p->weight.E != 1)
        return fail(MOE_FFN_ERR_NULL, "offsets is NULL with E = %lld", (long long)p->weight.E);
    if (p->M == 0)
        return MOE_FFN_OK;
    const I8ProductLayout L = i8_product_layout(*p);
    if ((rc = check_ptr(codes, "codes")) || (rc = check_ptr(scales, "scales", 4)) ||
        (rc = check_packed(&p->weight, packed, packed_bytes)) ||
        (offsets && (rc = check_ptr(offsets, "offsets", p->offsets_dtype == MOE_FFN_I64 ? 8 : 4))) ||
        (rc = check_ptr(y, "y")) || (L.total && (rc = check_ptr(ws, "ws"))))
        return rc;
    if (ws_bytes < L.total)
        return fail(MOE_FFN_ERR_WORKSPACE, "workspace too small: %zu < %zu", ws_bytes, L.total);
    int num_cus = 0;
    if ((rc = check_device(&num_cus)))
        return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const moe_ffn_int8_weight &w = p->weight;
    const moe::I8Dims d(w.Kd, w.N / w.panels);
    moe::I8GemmArgs a{};
    a.src = {offsets, p->offsets_dtype == MOE_FFN_I64, p->M, (int)w.E};
    a.max_mtiles = (int)tiles_of(p->M, w.E, L.BM);
    if (w.E > moe::kViewGroups) {
        moe::GroupSetup set = L.groups.setup(ws, offsets, p->offsets_dtype, p->M, w.E, L.BM);
        set.out = y;
        set.out_row = w.N * (int64_t)elem_size(p->out_dtype);
        HIP_TRY(moe::launch_group_setup(set, s), "group set-up launch");
        a.offsets = set.out_offsets;
        a.mtile_off = set.mtile_off;
        a.mtile_expert = set.mtile_expert;
    }
    a.wcodes = static_cast<const uint8_t *>(packed);
    a.wscales = at<float>(const_cast<void *>(packed), i8_weight_layout(w.E, w.Kd, w.N, w.panels).scales);
    a.acodes = static_cast<const uint8_t *>(codes);
    a.ascales = scales;
    a.out = y;
    a.M = p->M;
    a.E = (int)w.E;
    a.topk = 1;
    a.out_bytes = (int)elem_size(p->out_dtype);
    a.N = (int)w.N;
    a.NT = d.NT;
    a.KS = d.KS;
    a.panels = w.panels;
    a.BM = L.BM;
    a.once = moe::weights_once(p->M, w.E, L.BM);
    // Past what the 256 MB last-level cache holds the output leaves it to the inputs, so
    // that weights that the last call left there are found (24576 x 1408 x 2048 over 64
    // groups: 80 us against 105)
    a.stream_out = p->M * (d.row() + w.N * (int64_t)elem_size(p->out_dtype)) + w.E * w.Kd * w.N >
                   ((int64_t)192 << 20);
    HIP_TRY(moe::launch_i8_gemm(p->out_dtype == MOE_FFN_BF16 ? moe::I8_BF16 : moe::I8_F32, a, num_cus, s),
            "int8 product launch");
    return MOE_FFN_OK;
}

int moe_ffn_int8_workspace_size(const moe_ffn_problem *p, uint32_t flags, size_t *ws_bytes)
{
    clear_error();
    const int rc = validate_i8_fwd(p, flags);
    if (rc)
        return rc;
    if (!ws_bytes)
        return fail(MOE_FFN_ERR_NULL, "ws_bytes is NULL");
    I8FwdLayout L;
    i8_fwd_layout(*p, L);
    *ws_bytes = L.total;
    return MOE_FFN_OK;
}

int moe_ffn_int8_fwd(const moe_ffn_problem *p, const void *x, const void *topk_ids,
                     const float *topk_weights, const void *up_packed, const void *down_packed,
                     void *y, void *ws, size_t ws_bytes, uint32_t flags, void *stream)
{
    clear_error();
    int rc = validate_i8_fwd(p, flags);
    if (rc)
        return rc;
    if (p->T == 0)
        return MOE_FFN_OK;
    I8FwdLayout L;
    i8_fwd_layout(*p, L);
    if ((rc = check_ptr(x, "x")) ||
        (rc = check_ptr(topk_ids, "topk_ids", p->ids_dtype == MOE_FFN_I64 ? 8 : 4)) ||
        (rc = check_ptr(topk_weights, "topk_weights", 4)) ||
        (rc = check_ptr(up_packed, "up_packed")) || (rc = check_ptr(down_packed, "down_packed")) ||
        (rc = check_ptr(y, "y")) || (rc = check_ptr(ws, "ws")))
        return rc;
    if (ws_bytes < L.total)
        return fail(MOE_FFN_ERR_WORKSPACE, "workspace too small: %zu < %zu", ws_bytes, L.total);
    int num_cus = 0;
    if ((rc = check_device(&num_cus)))
        return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t TK = p->T * p->K;
    const int E = (int)p->E;

    moe::RouteBufs rb{};
    rb.status = at<int32_t>(ws, L.status);
    rb.hist = at<int32_t>(ws, L.hist);
    rb.bad = at<int32_t>(ws, L.bad);
    rb.counts = at<int32_t>(ws, L.counts);
    rb.offsets = at<int32_t>(ws, L.offsets);
    rb.mtile_off = at<int32_t>(ws, L.mtile_off);
    rb.mtile_expert = at<int32_t>(ws, L.mtile_expert);
    rb.sorted_slot = at<int32_t>(ws, L.sorted_slot);
    rb.slot_pos = at<int32_t>(ws, L.slot_pos);
    rb.T = p->T;
    // the token rows by further blocks of the routing launch, which they keep in
    // registers, or by a launch of their own
    const moe::MxRows rows{x, at<void>(ws, L.x_codes), nullptr, at<void>(ws, L.x_scales), p->T,
                           (int)p->H, 0, (int)moe::I8Dims(p->H, 8).row(), 8};
    const bool ride = p->H <= moe::kRideMaxH;
    HIP_TRY(moe::launch_route(topk_ids, p->ids_dtype == MOE_FFN_I64, TK, E, L.BM, L.rp, rb, s,
                              ride ? &rows : nullptr),
            "route launch");
    if (!ride)
        HIP_TRY(moe::launch_i8_quantize_rows(MOE_FFN_BF16, x, p->H, rows.codes,
                                             static_cast<float *>(rows.scales), p->T, p->H, s),
                "token quantisation launch");
    if ((flags & MOE_FFN_CHECK_IDS) && (rc = check_ids(rb.status, E, s)))
        return rc;

    moe::I8GemmArgs g{};
    g.sorted_slot = rb.sorted_slot;
    g.offsets = rb.offsets;
    g.mtile_off = rb.mtile_off;
    g.mtile_expert = rb.mtile_expert;
    g.max_mtiles = (int)L.max_mtiles;
    g.E = E;
    g.BM = L.BM;
    g.once = moe::weights_once(TK, E, L.BM);

    moe::I8GemmArgs g1 = g;
    const moe::I8Dims up(p->H, p->I), down(p->I, p->H);
    g1.wcodes = static_cast<const uint8_t *>(up_packed);
    g1.wscales = at<float>(const_cast<void *>(up_packed), i8_weight_layout(E, p->H, 2 * p->I, 2).scales);
    g1.acodes = at<uint8_t>(ws, L.x_codes);
    g1.ascales = at<float>(ws, L.x_scales);
    g1.out = at<void>(ws, L.act);
    g1.M = p->T;
    g1.topk = (int)p->K;
    g1.N = (int)p->I;
    g1.NT = up.NT;
    g1.KS = up.KS;
    g1.panels = 2;
    g1.stream_out = TK * p->I * 4 > ((int64_t)192 << 20);
    HIP_TRY(moe::launch_i8_gemm(moe::I8_SWIGLU, g1, num_cus, s), "gemm1 launch");

    // rows of dropped slots, behind the last expert's, are quantised too and not read
    HIP_TRY(moe::launch_i8_quantize_rows(MOE_FFN_F32, g1.out, p->I, at<void>(ws, L.act_codes),
                                         at<float>(ws, L.act_scales), TK, p->I, s),
            "act quantisation launch");

    moe::I8GemmArgs g2 = g;
    g2.wcodes = static_cast<const uint8_t *>(down_packed);
    g2.wscales = at<float>(const_cast<void *>(down_packed), i8_weight_layout(E, p->I, p->H, 1).scales);
    g2.acodes = at<uint8_t>(ws, L.act_codes);
    g2.ascales = at<float>(ws, L.act_scales);
    g2.out = at<void>(ws, L.o);
    g2.M = TK;
    g2.topk = 1;
    g2.N = (int)p->H;
    g2.NT = down.NT;
    g2.KS = down.KS;
    g2.panels = 1;
    // o stays in fp32 up to the sum over a token's slots: rounded to bf16 first, y is off by
    // 0.0024 of its size where y's own rounding gives 0.0017, and by all of it where slots cancel
    g2.stream_out = TK * p->H * 4 > ((int64_t)192 << 20); // where the combine reads it past the cache
    HIP_TRY(moe::launch_i8_gemm(moe::I8_F32, g2, num_cus, s), "gemm2 launch");

    HIP_TRY(moe::launch_combine(MOE_FFN_F32, MOE_FFN_BF16, g2.out, rb.slot_pos, topk_weights, y, p->T,
                                (int)p->H, (int)p->K, rb.offsets, E, 0, s),
            "combine launch");
    if (flags & MOE_FFN_CHECK_STATUS)
        return check_ids(rb.status, E, s);
    return MOE_FFN_OK;
}

} // extern "C"
