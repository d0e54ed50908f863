// C ABI of the operators on grouped rows (declared in include/tgemm.h): the
// grouped products' planner and launcher, the routing tables, the weighted
// sum of a token's rows, and the gradient of the fused epilogue.  Host code only.
#include <hip/hip_runtime.h>

#include <new>

#include "capi_util.hpp"

using tg::capi_aligned;
using tg::capi_fail;
using tg::capi_ok;
using tg::capi_overlap;

struct gemm_group_plan {
    gemm_group_plan_info info;
    const tg::GroupVariant *v;
    gemm_plan *one;             // one group's product: its checks and its pre-shuffled image
    int elem, out, elem_bytes, out_bytes;
    bool inner;                 // the inner size is grouped (GEMM_LAYOUT_AT_BN)
    int tiles_m, tiles_n, group_m;
};

namespace {

constexpr int64_t kMaxRows = GEMM_GROUP_MAX_ROWS;
constexpr int64_t kRange = (int64_t)1 << 31;     // bytes one buffer resource of the kernels covers
constexpr int64_t kThreads = (int64_t)1 << 32;   // a launch has fewer
constexpr int64_t kStepRows = 64;                // K-rows of one step with a ragged inner size (bf16)

const tg::GroupVariant *find(const tg::GroupVariant *v, int n, int bm, int elem, int out, int layout)
{
    const bool pre = layout == GEMM_LAYOUT_BT_PRESHUFFLED, akm = layout == GEMM_LAYOUT_AT_BN;
    const bool bkn = akm || layout == GEMM_LAYOUT_BN;
    for (int i = 0; i < n; ++i)
        if (v[i].bm == bm && v[i].elem == elem && v[i].out == out && v[i].preshuffled == pre && v[i].bkn == bkn &&
            v[i].akm == akm)
            return &v[i];
    return nullptr;
}

const tg::GroupVariant *pick(int bm, int elem, int out, int layout)
{
    int n = 0;
    const tg::GroupVariant *v = bm == 256 ? tg::group_wide_variants(&n) : tg::group_tiled_variants(&n);
    return find(v, n, bm, elem, out, layout);
}

// Rows per tile from the mean rows per group, M being the rows there is room
// for.  Up to 24 rows (decode) the 32-row tiles stream the active experts'
// weights at the rate of a copy; larger tiles read the same weights with fewer
// workgroups in flight.  Measured on uneven groups (us for tiles of 32 / 64 /
// 128 / 256), bf16, 64 groups, N 2048, K 1024: mean 8: 44 / 43 / 47 / 52; mean
// 48: 60 / 55 / 61 / 66; mean 120: 106 / 85 / 81 / 83; 16 groups, N 2048, K 4096:
// mean 80: 74 / 59 / 70 / 94; mean 170: 121 / 100 / 76 / 103; mean 300 (64 / 128 /
// 256): 147 / 139 / 115; mean 1000: 392 / 319 / 291.
// One list serves all types and layouts; where it is not the best of the four
// (16 groups, N 2048, K 4096): e4m3 mean 400 (64 / 128 / 256) 77 / 61 / 67, mean 600
// 107 / 89 / 100; bf16 pre-shuffled mean 24 (32 / 64) 57 / 44.  The rule does not
// look at the number of workgroups: few groups with N below 1024, not
// measured, leave CUs idle, as the weight gradient's 256 x 256 tiles do where
// the groups' C are small.
int default_tile(int groups, int64_t M, int layout)
{
    if (layout == GEMM_LAYOUT_AT_BN)
        return 256;
    const int64_t mean = (M + groups - 1) / groups;
    return mean <= 24 ? 32 : (mean <= 96 ? 64 : (mean <= 192 ? 128 : 256));
}

}  // namespace

extern "C" {

gemm_group_plan *gemm_group_plan_create_opt(int groups, int64_t M, int64_t N, int64_t K, int dtype, int layout,
                                            int tile_rows)
{
    if (groups < 1 || groups > GEMM_GROUP_MAX) {
        capi_fail(GEMM_ERR_INVALID_ARG, "groups=%d outside 1..%d", groups, GEMM_GROUP_MAX);
        return nullptr;
    }
    if (tile_rows != 0 && tile_rows != 32 && tile_rows != 64 && tile_rows != 128 && tile_rows != 256) {
        capi_fail(GEMM_ERR_INVALID_ARG, "tile_rows=%d is none of 0, 32, 64, 128, 256", tile_rows);
        return nullptr;
    }
    if (dtype != GEMM_BF16_OUT_F32 && dtype != GEMM_BF16_OUT_BF16 && dtype != GEMM_E4M3_OUT_BF16) {
        if (dtype < GEMM_BF16_OUT_F32 || dtype > GEMM_W4A8_OUT_BF16)
            capi_fail(GEMM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
        else
            capi_fail(GEMM_ERR_UNSUPPORTED, "grouped products take bf16 and fp8 e4m3 operands");
        return nullptr;
    }
    if (layout < GEMM_LAYOUT_BT || layout > GEMM_LAYOUT_AT_BN) {
        capi_fail(GEMM_ERR_INVALID_ARG, "unknown layout %d", layout);
        return nullptr;
    }
    const bool inner = layout == GEMM_LAYOUT_AT_BN;
    const bool bf16 = dtype != GEMM_E4M3_OUT_BF16;
    if (layout == GEMM_LAYOUT_AT || (!bf16 && (inner || layout == GEMM_LAYOUT_BN))) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "no grouped product for this dtype and layout");
        return nullptr;
    }
    if (M < 0 || N < 0 || K < 0) {
        capi_fail(GEMM_ERR_INVALID_ARG, "negative size (M=%lld N=%lld K=%lld)", (long long)M, (long long)N,
                  (long long)K);
        return nullptr;
    }
    if ((inner ? K : M) > kMaxRows) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "more than 2^24 grouped rows");
        return nullptr;
    }
    if (inner && M * kStepRows * (int64_t)sizeof(uint16_t) >= kRange) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "M=%lld: 64 rows of A must stay below 2^31 bytes (32-bit offsets)", (long long)M);
        return nullptr;
    }
    // One group's product: gemm_plan_create's checks on the sizes.  The
    // ragged size has none of its own, so the smallest legal one stands for it.
    gemm_plan *one = inner ? gemm_plan_create(M, N, 32, dtype, layout) : gemm_plan_create(1, N, K, dtype, layout);
    if (!one)
        return nullptr;
    gemm_group_plan *p = new (std::nothrow) gemm_group_plan();
    if (!p) {
        gemm_plan_destroy(one);
        capi_fail(GEMM_ERR_INVALID_ARG, "out of host memory");
        return nullptr;
    }
    p->one = one;
    p->elem = bf16 ? tg::kBf16 : tg::kFp8;
    p->out = dtype == GEMM_BF16_OUT_F32 ? tg::kOutF32 : tg::kOutBf16;
    p->elem_bytes = bf16 ? 2 : 1;
    p->out_bytes = p->out == tg::kOutF32 ? 4 : 2;
    p->inner = inner;
    const int bm = tile_rows ? tile_rows : default_tile(groups, M, layout);
    p->v = pick(bm, p->elem, p->out, layout);
    if (!p->v) {
        gemm_group_plan_destroy(p);
        capi_fail(GEMM_ERR_UNSUPPORTED, "no grouped kernel with %d-row tiles for this dtype and layout", bm);
        return nullptr;
    }
    gemm_group_plan_info &I = p->info;
    I.M = M;
    I.N = N;
    I.K = K;
    I.groups = groups;
    I.dtype = dtype;
    I.layout = layout;
    I.tile_m = bm;
    I.tile_n = p->v->bn;
    I.threads = p->v->threads;
    I.lds_bytes = p->v->lds_bytes;
    p->tiles_n = (int)((N + p->v->bn - 1) / p->v->bn);
    int64_t tiles;
    if (inner) {
        p->tiles_m = (int)((M + bm - 1) / bm);
        tiles = (int64_t)p->tiles_m * groups;
    } else {
        // sum of ceil(rows / bm) over the groups, whatever the offsets
        const int64_t bound = (M + (int64_t)groups * (bm - 1)) / bm;
        tiles = bound < M ? bound : M;
        p->tiles_m = (int)tiles;
    }
    p->group_m = bm >= 256 ? 4 : 8;
    if (inner && p->group_m > p->tiles_m)
        p->group_m = p->tiles_m > 0 ? p->tiles_m : 1;
    if (tiles * p->tiles_n * p->v->threads >= kThreads) {
        gemm_group_plan_destroy(p);
        capi_fail(GEMM_ERR_UNSUPPORTED, "too many tiles (a launch has fewer than 2^32 threads)");
        return nullptr;
    }
    I.grid = (int32_t)(tiles * p->tiles_n);
    capi_ok();
    return p;
}

gemm_group_plan *gemm_group_plan_create(int groups, int64_t M, int64_t N, int64_t K, int dtype, int layout)
{
    return gemm_group_plan_create_opt(groups, M, N, K, dtype, layout, 0);
}

void gemm_group_plan_destroy(gemm_group_plan *plan)
{
    if (plan)
        gemm_plan_destroy(plan->one);
    delete plan;
}

int gemm_group_plan_query(const gemm_group_plan *plan, gemm_group_plan_info *info)
{
    if (!plan || !info)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan or info");
    *info = plan->info;
    return capi_ok();
}

size_t gemm_group_preshuffled_b_bytes(const gemm_group_plan *plan)
{
    return plan ? gemm_preshuffled_b_bytes(plan->one) * (size_t)plan->info.groups : 0;
}

int gemm_group_preshuffle_b(const gemm_group_plan *plan, const void *B, void *B_shuf, hipStream_t stream)
{
    if (!plan)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan");
    if (plan->inner || plan->info.layout == GEMM_LAYOUT_BN)
        return capi_fail(GEMM_ERR_INVALID_ARG, "the pre-shuffled image is made from B stored N x K");
    const size_t bytes = gemm_preshuffled_b_bytes(plan->one), all = gemm_group_preshuffled_b_bytes(plan);
    if (bytes == 0)
        return capi_ok();
    if (!B || !B_shuf)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL B or B_shuf");
    if (capi_overlap(B, all, B_shuf, all))
        return capi_fail(GEMM_ERR_INVALID_ARG, "B_shuf overlaps B");
    // The image's outermost mode is N / 16, so the matrices' images lie one
    // behind the other like those of one taller B.
    gemm_plan *tall = gemm_plan_create(1, plan->info.N * plan->info.groups, plan->info.K, plan->info.dtype,
                                       GEMM_LAYOUT_BT_PRESHUFFLED);
    if (tall) {
        const int rc = gemm_preshuffle_b(tall, B, B_shuf, stream);
        gemm_plan_destroy(tall);
        return rc;
    }
    for (int g = 0; g < plan->info.groups; ++g)          // taller than one plan may be
        if (int rc = gemm_preshuffle_b(plan->one, (const uint8_t *)B + g * bytes, (uint8_t *)B_shuf + g * bytes, stream))
            return rc;
    return capi_ok();
}

int gemm_group_run(const gemm_group_plan *plan, const void *A, const void *B, void *C, const int32_t *offsets,
                   const int32_t *row_index, int64_t a_rows, const gemm_epilogue_args *epi, void *preact,
                   hipStream_t stream)
{
    if (!plan)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan");
    const gemm_group_plan_info &I = plan->info;
    tg::TiledArgs a{};
    if (int rc = tg::capi_epilogue(epi, &a.epi))
        return rc;
    if (plan->inner && (row_index || preact))
        return capi_fail(GEMM_ERR_INVALID_ARG, "row_index and preact do not belong to GEMM_LAYOUT_AT_BN");
    if (plan->inner && (a.epi.bias || a.epi.sa_rows || a.epi.sb_cols))
        return capi_fail(GEMM_ERR_INVALID_ARG, "GEMM_LAYOUT_AT_BN takes scales of one value and no bias");
    if (row_index && (a_rows < 0 || a_rows > ((int64_t)1 << 30)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "a_rows=%lld outside 0..2^30", (long long)a_rows);
    if (row_index && a_rows * I.K * plan->elem_bytes >= kRange)
        return capi_fail(GEMM_ERR_UNSUPPORTED, "A behind row_index must stay below 2^31 bytes (32-bit offsets)");
    if (I.grid == 0)
        return capi_ok();
    const int64_t rows_a = plan->inner ? I.K : (row_index ? a_rows : I.M);
    const size_t abytes = (size_t)rows_a * (size_t)(plan->inner ? I.M : I.K) * plan->elem_bytes;
    const size_t bbytes = (size_t)I.N * (size_t)I.K * plan->elem_bytes * (plan->inner ? 1 : (size_t)I.groups);
    const size_t cbytes = (size_t)I.M * (size_t)I.N * plan->out_bytes * (plan->inner ? (size_t)I.groups : 1);
    if ((!A && abytes) || (!B && bbytes) || !C)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL A, B or C");
    if (!offsets || !capi_aligned(offsets, 4) || !capi_aligned(row_index, 4))
        return capi_fail(GEMM_ERR_INVALID_ARG, "offsets is NULL, or offsets or row_index is not 4-byte aligned");
    if (!capi_aligned(A, 16) || !capi_aligned(B, 16) || !capi_aligned(C, 16) || !capi_aligned(preact, 16))
        return capi_fail(GEMM_ERR_INVALID_ARG, "A, B, C and preact must be 16-byte aligned");
    const size_t obytes = ((size_t)I.groups + 1) * 4, xbytes = row_index ? (size_t)I.M * 4 : 0;
    if (capi_overlap(C, cbytes, A, abytes) || capi_overlap(C, cbytes, B, bbytes) ||
        capi_overlap(C, cbytes, offsets, obytes) || capi_overlap(C, cbytes, row_index, xbytes))
        return capi_fail(GEMM_ERR_INVALID_ARG, "C overlaps A, B, offsets or row_index");
    if (capi_overlap(preact, cbytes, A, abytes) || capi_overlap(preact, cbytes, B, bbytes) ||
        capi_overlap(preact, cbytes, C, cbytes) || capi_overlap(preact, cbytes, offsets, obytes) ||
        capi_overlap(preact, cbytes, row_index, xbytes))
        return capi_fail(GEMM_ERR_INVALID_ARG, "preact overlaps A, B, C, offsets or row_index");
    if (int rc = tg::capi_check_device())
        return rc;
    a.A = A;
    a.B = B;
    a.C = C;
    a.epi.pre = preact;
    a.M = (int32_t)I.M;
    a.N = (int32_t)I.N;
    a.K = (int32_t)I.K;
    const int64_t kbytes = plan->inner ? 0 : I.K * plan->elem_bytes;
    a.kbytes = a.kbytes_b = (int32_t)kbytes;
    a.k_tiles = (int32_t)((kbytes + tg::kTileKBytes - 1) / tg::kTileKBytes);
    a.tail_bytes = kbytes % tg::kTileKBytes ? (int32_t)(kbytes % tg::kTileKBytes) : tg::kTileKBytes;
    a.ldb_bytes = (int32_t)(I.N * plan->elem_bytes);
    a.lda_bytes = (int32_t)(I.M * plan->elem_bytes);
    a.grid = I.grid;
    a.tiles_m = plan->tiles_m;
    a.tiles_n = plan->tiles_n;
    a.group_m = plan->group_m;
    a.splits = 1;
    a.grp.offsets = offsets;
    a.grp.row_index = row_index;
    a.grp.groups = I.groups;
    a.grp.rows = (int32_t)(plan->inner ? I.K : I.M);
    a.grp.a_rows = (int32_t)(row_index ? a_rows : 0);
    a.grp.b_stride = I.N * I.K * plan->elem_bytes;
    const hipError_t e = plan->v->launch(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "grouped launch: %s", hipGetErrorString(e));
    return capi_ok();
}

// ---------------------------------------------------------------- routing tables

namespace {

// One block, and one launch, for up to kSortOne slots; above, blocks of 1024
// slots, one per thread, or more, so that there is at most one per CU (each
// block reads every block's counts).
constexpr int64_t kSortOne = 4096;
constexpr int64_t kSortBlocks = 256;
constexpr int64_t kSortStep = 1024;      // 16 waves x 64 slots

void sort_split(int64_t slots, int32_t *blocks, int32_t *block_slots)
{
    int64_t b = slots <= kSortOne ? 1 : (slots + kSortStep - 1) / kSortStep;
    b = b > kSortBlocks ? kSortBlocks : b;
    int64_t per = (slots + b - 1) / b;
    per = (per + kSortStep - 1) / kSortStep * kSortStep;
    per = per < kSortStep ? kSortStep : per;
    *block_slots = (int32_t)per;
    *blocks = (int32_t)(slots ? (slots + per - 1) / per : 1);
}

}  // namespace

size_t gemm_group_sort_workspace_bytes(int64_t slots, int groups)
{
    if (slots < 0 || slots > kMaxRows || groups < 1 || groups > GEMM_GROUP_MAX)
        return 0;
    int32_t blocks, per;
    sort_split(slots, &blocks, &per);
    return blocks > 1 ? (size_t)blocks * (size_t)groups * 4 : 0;
}

int gemm_group_sort(const int32_t *ids, int64_t slots, int topk, int groups, int32_t *offsets, int32_t *row_token,
                    int32_t *slot_row, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (groups < 1 || groups > GEMM_GROUP_MAX)
        return capi_fail(GEMM_ERR_INVALID_ARG, "groups=%d outside 1..%d", groups, GEMM_GROUP_MAX);
    if (slots < 0 || slots > kMaxRows)
        return capi_fail(GEMM_ERR_INVALID_ARG, "slots=%lld outside 0..2^24", (long long)slots);
    if (topk < 1 || slots % topk != 0)
        return capi_fail(GEMM_ERR_INVALID_ARG, "slots=%lld is not a multiple of topk=%d", (long long)slots, topk);
    if (!offsets || (slots && (!ids || !row_token || !slot_row)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL ids, offsets, row_token or slot_row");
    const void *all[] = {ids, offsets, row_token, slot_row, workspace};
    const size_t need = gemm_group_sort_workspace_bytes(slots, groups);
    const size_t n = (size_t)slots * 4;
    const size_t bytes[] = {n, ((size_t)groups + 1) * 4, n, n, need};
    for (const void *p : all)
        if (!capi_aligned(p, 4))
            return capi_fail(GEMM_ERR_INVALID_ARG, "ids, the tables and the workspace must be 4-byte aligned");
    if (need && (!workspace || workspace_bytes < need))
        return capi_fail(GEMM_ERR_INVALID_ARG, "the sort needs a workspace of %zu bytes", need);
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (capi_overlap(all[i], bytes[i], all[j], bytes[j]))
                return capi_fail(GEMM_ERR_INVALID_ARG, "ids, the tables and the workspace must not overlap");
    if (int rc = tg::capi_check_device())
        return rc;
    tg::SortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.row_token = row_token;
    a.slot_row = slot_row;
    a.counts = (int32_t *)workspace;
    a.slots = (int32_t)slots;
    a.topk = topk;
    a.groups = groups;
    sort_split(slots, &a.blocks, &a.block_slots);
    while ((1 << a.id_bits) < groups)
        ++a.id_bits;
    const hipError_t e = tg::launch_group_sort(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "sort launch: %s", hipGetErrorString(e));
    return capi_ok();
}

// ---------------------------------------------------------------- combine

namespace {

int check_combine(int64_t tokens, int topk, int64_t N, int type, int64_t src_rows)
{
    if (tokens < 0 || tokens > kMaxRows)
        return capi_fail(GEMM_ERR_INVALID_ARG, "tokens=%lld outside 0..2^24", (long long)tokens);
    if (topk < 1 || topk > 64)
        return capi_fail(GEMM_ERR_INVALID_ARG, "topk=%d outside 1..64", topk);
    if (N < 0 || N >= ((int64_t)1 << 21) || N % 16 != 0)
        return capi_fail(N < 0 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_UNSUPPORTED,
                         "N=%lld must be a multiple of 16 below 2^21", (long long)N);
    if (type != GEMM_TYPE_F32 && type != GEMM_TYPE_BF16)
        return capi_fail(GEMM_ERR_INVALID_ARG, "unknown type %d", type);
    if (src_rows < 0 || src_rows >= ((int64_t)1 << 31))
        return capi_fail(GEMM_ERR_INVALID_ARG, "src_rows=%lld outside 0..2^31 - 1", (long long)src_rows);
    return GEMM_OK;
}

int out_type(int type) { return type == GEMM_TYPE_F32 ? tg::kOutF32 : tg::kOutBf16; }
size_t type_bytes(int type) { return type == GEMM_TYPE_F32 ? 4 : 2; }

}  // namespace

int gemm_group_combine(int64_t tokens, int topk, int64_t N, int type, const void *src, int64_t src_rows,
                       const int32_t *slot_row, const float *weights, const void *residual, void *out,
                       hipStream_t stream)
{
    if (int rc = check_combine(tokens, topk, N, type, src_rows))
        return rc;
    if (tokens == 0 || N == 0)
        return capi_ok();
    if (!slot_row || !out || (!src && src_rows))
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL src, slot_row or out");
    if (!capi_aligned(src, 16) || !capi_aligned(residual, 16) || !capi_aligned(out, 16) ||
        !capi_aligned(slot_row, 4) || !capi_aligned(weights, 4))
        return capi_fail(GEMM_ERR_INVALID_ARG, "src, residual and out must be 16-byte aligned, slot_row and weights 4");
    const size_t obytes = (size_t)tokens * (size_t)N * type_bytes(type);
    const size_t sbytes = (size_t)src_rows * (size_t)N * type_bytes(type), tbytes = (size_t)tokens * topk * 4;
    if (capi_overlap(out, obytes, src, sbytes) || capi_overlap(out, obytes, slot_row, tbytes) ||
        capi_overlap(out, obytes, weights, tbytes) || (residual != out && capi_overlap(out, obytes, residual, obytes)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "out overlaps src, slot_row, weights or (other than in place) residual");
    if (int rc = tg::capi_check_device())
        return rc;
    tg::CombineArgs a{};
    a.src = src;
    a.residual = residual;
    a.out = out;
    a.slot_row = slot_row;
    a.weights = weights;
    a.tokens = tokens;
    a.N = N;
    a.topk = topk;
    a.src_rows = (int32_t)src_rows;
    a.type = out_type(type);
    const hipError_t e = tg::launch_group_combine(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "combine launch: %s", hipGetErrorString(e));
    return capi_ok();
}

int gemm_group_combine_grad(int64_t tokens, int topk, int64_t N, int type, const void *d_out, const void *src,
                            int64_t src_rows, const int32_t *slot_row, const float *weights, void *d_src,
                            float *d_weights, hipStream_t stream)
{
    if (int rc = check_combine(tokens, topk, N, type, src_rows))
        return rc;
    if (tokens == 0)
        return capi_ok();
    if (!slot_row || (!d_out && N) || (!d_src && src_rows && N) || (!src && d_weights && src_rows && N))
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL d_out, src, slot_row or d_src");
    if (!capi_aligned(src, 16) || !capi_aligned(d_out, 16) || !capi_aligned(d_src, 16) || !capi_aligned(slot_row, 4) ||
        !capi_aligned(weights, 4) || !capi_aligned(d_weights, 4))
        return capi_fail(GEMM_ERR_INVALID_ARG,
                         "d_out, src and d_src must be 16-byte aligned, slot_row and the weights 4");
    const size_t obytes = (size_t)tokens * (size_t)N * type_bytes(type);
    const size_t sbytes = (size_t)src_rows * (size_t)N * type_bytes(type), tbytes = (size_t)tokens * topk * 4;
    const struct {
        const void *p;
        size_t n;
    } in[] = {{d_out, obytes}, {src, sbytes}, {slot_row, tbytes}, {weights, tbytes}};
    for (const auto &x : in)
        if (capi_overlap(d_src, sbytes, x.p, x.n) || capi_overlap(d_weights, tbytes, x.p, x.n))
            return capi_fail(GEMM_ERR_INVALID_ARG, "d_src or d_weights overlaps an input");
    if (capi_overlap(d_src, sbytes, d_weights, tbytes))
        return capi_fail(GEMM_ERR_INVALID_ARG, "d_src overlaps d_weights");
    if (int rc = tg::capi_check_device())
        return rc;
    tg::CombineArgs a{};
    a.src = src;
    a.d_out = d_out;
    a.out = d_src;
    a.slot_row = slot_row;
    a.weights = weights;
    a.d_weights = d_weights;
    a.tokens = tokens;
    a.N = N;
    a.topk = topk;
    a.src_rows = (int32_t)src_rows;
    a.type = out_type(type);
    const hipError_t e = tg::launch_group_combine_grad(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "combine gradient launch: %s", hipGetErrorString(e));
    return capi_ok();
}

// ---------------------------------------------------------------- epilogue gradient

namespace {

// Rows per chunk: 64 where that alone gives the chip two workgroups per CU,
// else 16, so that few rows still spread over it.
int act_chunk(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 511) / 512) >= 512 ? 64 : 16; }

// An upper bound on the sum of ceil(rows / chunk) over the groups.
int64_t act_chunks(int64_t M, int64_t N, int groups)
{
    const int c = act_chunk(M, N);
    const int64_t bound = (M + (int64_t)groups * (c - 1)) / c;
    return bound < M ? bound : M;
}

}  // namespace

size_t gemm_act_grad_workspace_bytes(int64_t M, int64_t N, int groups)
{
    if (M < 0 || N < 0 || M > kMaxRows || N >= ((int64_t)1 << 21) || groups < 1 || groups > GEMM_GROUP_MAX)
        return 0;
    return (size_t)act_chunks(M, N, groups) * (size_t)N * 4;
}

int gemm_act_grad(int64_t M, int64_t N, int type, int epilogue, const void *d_c, const void *z, void *d_z,
                  float *d_bias, int groups, const int32_t *offsets, void *workspace, size_t workspace_bytes,
                  hipStream_t stream)
{
    if (groups < 1 || groups > GEMM_GROUP_MAX || (!offsets && groups != 1))
        return capi_fail(GEMM_ERR_INVALID_ARG, "groups=%d outside 1..%d, or several groups without offsets", groups,
                         GEMM_GROUP_MAX);
    if (M < 0 || N < 0)
        return capi_fail(GEMM_ERR_INVALID_ARG, "negative size (M=%lld N=%lld)", (long long)M, (long long)N);
    if (M > kMaxRows || N >= ((int64_t)1 << 21) || N % 16 != 0)
        return capi_fail(GEMM_ERR_UNSUPPORTED, "M=%lld must be at most 2^24, N=%lld a multiple of 16 below 2^21",
                         (long long)M, (long long)N);
    if (type != GEMM_TYPE_F32 && type != GEMM_TYPE_BF16)
        return capi_fail(GEMM_ERR_INVALID_ARG, "unknown type %d", type);
    if (epilogue < GEMM_EPI_NONE || epilogue > GEMM_EPI_BIAS_GELU)
        return capi_fail(GEMM_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
    if (N == 0 || (M == 0 && !d_bias))
        return capi_ok();
    static const int kAct[] = {tg::kActNone, tg::kActNone, tg::kActRelu, tg::kActSilu, tg::kActGelu};
    const int act = kAct[epilogue];
    if (M && (!d_c || !d_z || (!z && act != tg::kActNone)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL d_c, z or d_z");
    if (!capi_aligned(d_c, 16) || !capi_aligned(z, 16) || !capi_aligned(d_z, 16) || !capi_aligned(d_bias, 16) ||
        !capi_aligned(offsets, 4))
        return capi_fail(GEMM_ERR_INVALID_ARG, "d_c, z, d_z and d_bias must be 16-byte aligned, offsets 4");
    const size_t bytes = (size_t)M * (size_t)N * type_bytes(type);
    const size_t bbytes = (size_t)groups * (size_t)N * 4, gbytes = ((size_t)groups + 1) * 4;
    if ((d_z != d_c && capi_overlap(d_z, bytes, d_c, bytes)) || (d_z != z && capi_overlap(d_z, bytes, z, bytes)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "d_z must be d_c or z itself, or overlap neither");
    if (capi_overlap(d_z, bytes, offsets, gbytes) || capi_overlap(d_bias, bbytes, d_z, bytes) ||
        capi_overlap(d_bias, bbytes, d_c, bytes) || capi_overlap(d_bias, bbytes, z, bytes) ||
        capi_overlap(d_bias, bbytes, offsets, gbytes))
        return capi_fail(GEMM_ERR_INVALID_ARG, "d_bias or the offsets overlap another operand");
    const size_t need = d_bias ? gemm_act_grad_workspace_bytes(M, N, groups) : 0;
    if (need && (!workspace || workspace_bytes < need || !capi_aligned(workspace, 16)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "d_bias needs a 16-byte aligned workspace of %zu bytes", need);
    if (need && (capi_overlap(workspace, need, d_z, bytes) || capi_overlap(workspace, need, d_c, bytes) ||
                 capi_overlap(workspace, need, z, bytes) || capi_overlap(workspace, need, d_bias, bbytes) ||
                 capi_overlap(workspace, need, offsets, gbytes)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "the workspace overlaps another operand");
    if (int rc = tg::capi_check_device())
        return rc;
    tg::ActGradArgs a{};
    a.d_c = d_c;
    a.z = z;
    a.d_z = d_z;
    a.d_bias = d_bias;
    a.partial = d_bias ? (float *)workspace : nullptr;
    a.offsets = offsets;
    a.N = N;
    a.M = (int32_t)M;
    a.groups = groups;
    a.chunk = act_chunk(M, N);
    a.max_chunks = (int32_t)act_chunks(M, N, groups);
    a.act = act;
    a.type = out_type(type);
    const hipError_t e = tg::launch_act_grad(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "epilogue gradient launch: %s", hipGetErrorString(e));
    return capi_ok();
}

}  // extern "C"
