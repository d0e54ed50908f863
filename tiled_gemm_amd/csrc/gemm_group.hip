// Grouped products on 256 x 256 tiles: the schedule of gemm_dma.hip (both
// operands staged through LDS by the loads' own LDS writes, one barrier per
// 128-byte K step, fragments read PD groups ahead of their MFMAs) on ragged row
// groups, entered through group.hpp.
//
// What is different here:
//   * a wave's row blocks are interleaved with the other row of waves' (block
//     i of wave row wm holds rows 16 (2 i + wm) ..), so that a tile with at
//     most half its rows is half the MFMAs, half the A loads and half the A
//     reads for every wave (LIGHT: 4 row blocks per wave instead of 8).  The
//     light tiles of all groups come last, where they fill the last round of
//     workgroups.  A light tile is a body of its own: one loop over both
//     sizes spilled 50 to 120 registers.
//   * A's rows may come through row_index (a lane's load offset is then the
//     gathered row's; the loop does not change).
//   * the weight gradient's K-rows (A K x M, B K x N) are the ragged size, and
//     may lie past 2^32 bytes: the buffer resources move with the step.
//   * always the extended epilogue (the pre-activation may be saved).
#include "group.hpp"

namespace tg {

namespace {

constexpr int GM_BM = 256;
constexpr int GM_BN = 256;
constexpr int GM_A = GM_BM * kTileKBytes;      // 32 KiB of A per stage
constexpr int GM_B = GM_BN * kTileKBytes;
constexpr int GM_STAGE = GM_A + GM_B;
constexpr int GM_EB = 4;                        // row blocks per batch of the epilogue
constexpr int GM_EPI = 8 * epi_lds_floats<4, GM_EB>() * 4;
constexpr int GM_LDS = 2 * GM_STAGE > GM_EPI ? 2 * GM_STAGE : GM_EPI;     // 136 KiB
static_assert(GM_LDS <= 160 * 1024, "gfx950 LDS is 160 KiB per workgroup");
constexpr int GM_WGM = 2, GM_WGN = 4, GM_WAVES = 8, GM_THREADS = 512;
constexpr int GM_FN = GM_BN / GM_WGN / 16;     // 4 column blocks per wave
constexpr int GM_KN_ROWS = 64;                  // K-rows per step of a K x M or K x N operand (bf16)
constexpr int GM_KN_CPR = 512 / kChunkBytes;

}  // namespace

// One tile.  LIGHT: at most 128 rows.
template <int ELEM, int OUT, bool BPRE, int PD, bool BKN, bool AKM, bool LIGHT>
__device__ inline void group_tile(const TiledArgs &p, int tm, int tn, uint8_t *lds)
{
    constexpr bool F8 = ELEM == kFp8;
    static_assert(ELEM == kBf16 || (F8 && !BKN && !AKM), "bf16, or fp8 e4m3 with B N x K");
    static_assert(!BPRE || (!BKN && !AKM), "a pre-shuffled B is N x K");
    static_assert(!(AKM && LIGHT), "light tiles belong to ragged rows");
    constexpr int FM = LIGHT ? 4 : 8, FN = GM_FN;          // row and column blocks per wave
    constexpr int AR = FM / 2;                              // A loads per lane and step
    constexpr int BR = GM_B / (GM_THREADS * kChunkBytes);
    constexpr int NL = AR + BR;
    constexpr int NG = F8 ? FM : 2 * FM;                    // groups per step: half h = g / FM (bf16)
    static_assert(PD >= 1 && (F8 ? PD < FM : PD <= FM), "prefetch distance");

    const int w = wave_id();
    const int l = lane_id();
    const int q = l >> 4, r16 = l & 15;
    const int wm = w / GM_WGN, wn = w % GM_WGN;
    const int m0 = tm * GM_BM, n0 = tn * GM_BN;
    const int rows_a = min(p.M - m0, GM_BM);
    const int rows_b = min(p.N - n0, GM_BN);
    const uint32_t kb = (uint32_t)p.kbytes;
    const uint32_t lda = (uint32_t)p.lda_bytes, ldb = (uint32_t)p.ldb_bytes;
    const int nk = p.k_tiles;
    const uint32_t tail = (uint32_t)p.tail_bytes;
    auto row_of = [&](int i) { return (i * GM_WGM + wm) * 16 + r16; };

    // ---- load sources (see gemm_dma.hip).  The weight gradient's resources
    // are made per step instead.
    const bool gather = !AKM && p.grp.row_index;
    const auto rA = gather ? make_rsrc(p.A, (uint32_t)p.grp.a_rows * kb)
                           : make_rsrc((const uint8_t *)p.A + (AKM ? (size_t)0 : (size_t)m0 * kb),
                                       AKM ? 0u : (uint32_t)rows_a * kb);
    const auto rB = BKN ? make_rsrc((const uint8_t *)p.B + (size_t)n0 * 2, AKM ? 0u : rest_bytes((size_t)p.K * ldb, (size_t)n0 * 2))
                        : make_rsrc((const uint8_t *)p.B + (size_t)n0 * kb, (uint32_t)rows_b * kb);
    uint32_t voffA[AR], voffB[BR];
    uint32_t tailA = 0, tailB = 0;
#pragma unroll
    for (int r = 0; r < AR; ++r) {
        const int pc = (r * GM_WAVES + w) * 64 + l;
        if constexpr (AKM) {
            const int row = pc / GM_KN_CPR, c = (pc % GM_KN_CPR) ^ bkn_swz(row);
            voffA[r] = (uint32_t)row * lda + (uint32_t)c * kChunkBytes;
            tailA |= 1u << r;                               // rows past K are out of range
        } else {
            const int row = pc >> 3, c = swz_chunk(row, pc & 7);
            voffA[r] = gather ? group_a_off(p.grp, p.M, m0 + row, kb, (uint32_t)c * kChunkBytes)
                              : (uint32_t)row * kb + (uint32_t)c * kChunkBytes;
            tailA |= ((uint32_t)(c * kChunkBytes) < tail ? 1u : 0u) << r;
        }
    }
#pragma unroll
    for (int r = 0; r < BR; ++r) {
        const int u = r * GM_WAVES + w, pc = u * 64 + l;
        if constexpr (BKN) {
            const int row = pc / GM_KN_CPR, c = (pc % GM_KN_CPR) ^ bkn_swz(row);
            voffB[r] = (uint32_t)row * ldb + (uint32_t)c * kChunkBytes;
            tailB |= 1u << r;
        } else if constexpr (BPRE) {
            voffB[r] = (uint32_t)(u >> 1) * 16u * kb + (uint32_t)(u & 1) * 1024u + (uint32_t)l * 16u;
            tailB |= ((uint32_t)((u & 1) * 64) < tail ? 1u : 0u) << r;
        } else {
            const int row = pc >> 3, c = swz_chunk(row, pc & 7);
            voffB[r] = (uint32_t)row * kb + (uint32_t)c * kChunkBytes;
            tailB |= ((uint32_t)(c * kChunkBytes) < tail ? 1u : 0u) << r;
        }
    }
    const uint32_t kBStep = BKN ? (uint32_t)GM_KN_ROWS * ldb : (BPRE ? 2048u : (uint32_t)kTileKBytes);
    // Load idx (A's first) of step kt into stage S; past the last step, and the
    // missing half of a half-filled one, zeros.  MASK == false: step kt is
    // whole and in range.
    auto issue_one = [&](int kt, auto s_c, int idx, auto mask_c) {
        constexpr int S = decltype(s_c)::value;
        const bool a = idx < AR;
        const int r = a ? idx : idx - AR;
        uint8_t *dst = lds + S * GM_STAGE + (a ? 0 : GM_A) + (r * GM_WAVES + w) * 1024;
        if constexpr (AKM) {
            // The group's K-rows may pass 2^32 bytes: the resource moves with
            // the step (64-bit, scalar) and ends with the group, so that rows
            // past it read zeros.
            const uint32_t ld = a ? lda : ldb;
            const int64_t at = (int64_t)kt * GM_KN_ROWS * ld;
            const int64_t first = (int64_t)(a ? m0 : n0) * 2;
            const int64_t left = (int64_t)p.K * ld - first - at;
            const uint32_t bytes = (uint32_t)max((int64_t)0, min(left, (int64_t)0x7FFFFFFF));
            buf_load16_to_lds(make_rsrc((const uint8_t *)(a ? p.A : p.B) + first + at, bytes), dst,
                              a ? voffA[idx < AR ? idx : 0] : voffB[idx < AR ? 0 : idx - AR], 0);
            issue_fence();
            return;
        }
        uint32_t vo = a ? voffA[idx < AR ? idx : 0] : voffB[idx < AR ? 0 : idx - AR];
        if constexpr (decltype(mask_c)::value) {
            const bool part = (kt == nk - 1) && tail != (uint32_t)kTileKBytes;
            vo = keep_or_oob((kt < nk) & (!part | ((((a ? tailA : tailB) >> r) & 1u) != 0)), vo);
        }
        buf_load16_to_lds(a ? rA : rB, dst, vo, (uint32_t)kt * (a ? (uint32_t)kTileKBytes : kBStep));
        issue_fence();
    };

    // ---- fragments (see gemm_dma.hip for the lane orders)
    // K x M or K x N operand: two transpose reads, of K-rows k = 32 h + 8 q + 4 t
    // + r16 / 4 of the step, chunk c ^ bkn_swz(k) of the 512-byte row.  The swizzle
    // has the same value for every h and t, and flips bits 1 to 3 of the chunk,
    // so four offsets per operand serve all its blocks; the rest are constants.
    uint32_t trA[4], trB[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int s = bkn_swz(8 * q + (r16 >> 2)), b = (r16 & 3) >> 1;
        const uint32_t lane = (uint32_t)(4096 * q + 512 * (r16 >> 2) + 8 * (r16 & 1));
        trA[x] = lane + (uint32_t)(((4 * x + 2 * wm + b) ^ s) << 4);          // row block i: x = i % 4, + 256 (i / 4)
        trB[x] = lane + (uint32_t)(((8 * wn + 2 * x + b) ^ s) << 4) + GM_A;   // column block x of the wave
    }
    auto tr_frag = [&](const uint8_t *at, int h) -> u32x4 {
        const u32x2 t0 = lds_read_tr16(at + h * 16384), t1 = lds_read_tr16(at + h * 16384 + 2048);
        return u32x4{t0.x, t0.y, t1.x, t1.y};
    };
    auto a16 = [&](int s, int i, int h) -> u32x4 {
        const uint8_t *sA = lds + s * GM_STAGE;
        if constexpr (AKM)
            return tr_frag(sA + trA[i & 3] + (i >> 2) * 256, h);
        const int row = row_of(i);
        return lds_load16(sA + row * kTileKBytes + swz_chunk(row, h * 4 + q) * kChunkBytes);
    };
    auto b16 = [&](int s, int j, int h) -> u32x4 {
        if constexpr (BKN)
            return tr_frag(lds + s * GM_STAGE + trB[j], h);
        const uint8_t *sB = lds + s * GM_STAGE + GM_A;
        const int nb = wn * FN + j;
        if constexpr (BPRE)
            return lds_load16(sB + (nb * 2 + h) * 1024 + l * 16);
        const int row = nb * 16 + r16;
        return lds_load16(sB + row * kTileKBytes + swz_chunk(row, h * 4 + q) * kChunkBytes);
    };
    using FragT = typename std::conditional<F8, i32x8, u32x4>::type;
    // bf16: B fragments by half, the next step's half 0 taking the registers
    // of this step's.  fp8: one set; the last group of a step reloads fragment
    // j right after its last MFMA (two sets do not fit beside 128 accumulators).
    FragT fa[NG], fb[F8 ? 1 : 2][FN];
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto load_group = [&](int s, int t) {
        if constexpr (F8) {
            fa[t] = join32(a16(s, t, 0), a16(s, t, 1));
        } else {
            if (t % FM == 0) {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    fb[t / FM][j] = b16(s, j, t / FM);
            }
            fa[t] = a16(s, t % FM, t / FM);
        }
    };
    auto barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto step = [&](int kt, auto s_c, auto mask_c) {
        constexpr int S = decltype(s_c)::value;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g == NG - PD) {
                // Every read of stage S has been issued: wait for them and for
                // step kt + 1's loads, meet, then refill stage S with step kt + 2.
                __builtin_amdgcn_s_waitcnt(0);
                barrier();
            }
            if (g >= NG - PD) {
                const int go = g - (NG - PD);
#pragma unroll
                for (int idx = go * NL / PD; idx < (go + 1) * NL / PD; ++idx)
                    issue_one(kt + 2, s_c, idx, mask_c);
            }
            if (g + PD < NG)
                load_group(S, g + PD);
            else
                load_group(S ^ 1, g + PD - NG);
            const int i = g % FM, h = g / FM;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (F8) {
                    acc[i][j] = mfma_fp8x8(fb[0][j], fa[g], acc[i][j]);
                    if (g == NG - 1) {
                        __builtin_amdgcn_sched_barrier(0);
                        fb[0][j] = join32(b16(S ^ 1, j, 0), b16(S ^ 1, j, 1));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
                    acc[i][j] = mfma_bf16(fb[h][j], fa[g], acc[i][j]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    using s0 = std::integral_constant<int, 0>;
    using s1 = std::integral_constant<int, 1>;
    using masked = std::true_type;
    using whole = std::false_type;
#pragma unroll
    for (int idx = 0; idx < NL; ++idx)
        issue_one(0, s0{}, idx, masked{});
#pragma unroll
    for (int idx = 0; idx < NL; ++idx)
        issue_one(1, s1{}, idx, masked{});
    // Step 0 has landed; step 1 is waited for inside step 0.
    static_assert(NL < 16, "the low bits of vmcnt");
    __builtin_amdgcn_s_waitcnt(((kWaitVmcnt0 & ~0xC00F) | NL) & 0xC07F);
    barrier();
    if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fb[0][j] = join32(b16(0, j, 0), b16(0, j, 1));
    }
#pragma unroll
    for (int t = 0; t < PD; ++t)
        load_group(0, t);
    // Steps run in pairs, one per stage.
    const int nfull = tail == (uint32_t)kTileKBytes ? nk : nk - 1;
    int kt = 0;
    for (; kt + 1 < nfull - 2; kt += 2) {
        step(kt, s0{}, whole{});
        step(kt + 1, s1{}, whole{});
    }
    for (; kt < nk; kt += 2) {
        step(kt, s0{}, masked{});
        if (kt + 1 == nk)
            break;
        step(kt + 1, s1{}, masked{});
    }
    __builtin_amdgcn_s_waitcnt(0);

    // ---- epilogue
    const EpiView ev = AKM ? epi_view(p.epi, p.M, p.N) : group_epi_view(p.epi, p.grp, p.M, p.N);
    constexpr int OB = OUT == kOutF32 ? 4 : 2;
    const uint32_t ldc = (uint32_t)p.N * OB;
    const auto rC = make_rsrc((uint8_t *)p.C + (size_t)m0 * ldc, (uint32_t)rows_a * ldc);
    const EpiExt ex = epi_ext(p.epi, (size_t)m0 * ldc, (uint32_t)rows_a * ldc);
    // Every wave has read its last fragments (those past the last step among
    // them) before LDS is reused.
    barrier();
    epi_store_tile<OUT, GM_EB>(ev, ex, rC, reinterpret_cast<float *>(lds) + w * epi_lds_floats<FN, GM_EB>(), acc,
                               wm * 16, GM_WGM * 16, n0 + wn * FN * 16, p.N, ldc, [](f32x4 a) { return a; },
                               [&](int row) {
                                   return AKM ? epi_row_scale(ev, 0) : group_row_scale(ev, p.grp, p.M, m0 + row);
                               });
}

template <int ELEM, int OUT, bool BPRE, int PD, bool BKN, bool AKM>
__global__ __launch_bounds__(GM_THREADS, 1) void gemm_group_kernel(const TiledArgs p0)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[GM_LDS];
    TiledArgs p = p0;
    int tm, tn;
    if constexpr (AKM) {
        group_enter_inner<OUT>(p, GM_KN_ROWS, &tm, &tn);
        group_tile<ELEM, OUT, BPRE, PD, BKN, AKM, false>(p, tm, tn, lds);
    } else {
        if (!group_enter<OUT, true>(p, GM_BM, p.tiles_n, p.group_m, &tm, &tn))
            return;
        constexpr int PDL = ELEM == kFp8 ? (PD < 3 ? PD : 3) : (PD < 4 ? PD : 4);
        if (p.M - tm * GM_BM <= GM_BM / 2)
            group_tile<ELEM, OUT, BPRE, PDL, BKN, AKM, true>(p, tm, tn, lds);
        else
            group_tile<ELEM, OUT, BPRE, PD, BKN, AKM, false>(p, tm, tn, lds);
    }
}

template <int ELEM, int OUT, bool BPRE, int PD, bool BKN, bool AKM>
static hipError_t launch_group(const TiledArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_group_kernel<ELEM, OUT, BPRE, PD, BKN, AKM>), dim3(a.grid), dim3(GM_THREADS), 0, s, a);
    return hipGetLastError();
}
#define TG_GROUP(ELEM, OUT, BPRE, PD, BKN, AKM)                                          \
    GroupVariant{GM_BM, GM_BN, GM_THREADS, ELEM, OUT, BPRE, BKN, AKM, GM_LDS,             \
                 &launch_group<ELEM, OUT, BPRE, PD, BKN, AKM>}

static const GroupVariant kGroup[] = {
    // PD: the loads of a step are spread over its last PD groups and waited for
    // PD groups before the end of the next, so a small PD leaves them more time
    // and a large one the fragments.  Measured (16 groups of 2048 rows, us):
    // transposed A and B, 4 / 2 / 1: 779 / 635 / 589; B K x N, 5 / 4 / 2: 552 /
    // 533 / 520; fp8 pre-shuffled, 2 / 1: 333 / 317; bf16 N x K, 6 / 5 / 3: 446 /
    // 442 / 454.
    TG_GROUP(kBf16, kOutBf16, false, 5, false, false), TG_GROUP(kBf16, kOutF32, false, 4, false, false),
    TG_GROUP(kBf16, kOutBf16, true, 6, false, false),  TG_GROUP(kBf16, kOutF32, true, 4, false, false),
    TG_GROUP(kFp8, kOutBf16, false, 1, false, false),  TG_GROUP(kFp8, kOutBf16, true, 1, false, false),
    TG_GROUP(kBf16, kOutBf16, false, 2, true, false),  TG_GROUP(kBf16, kOutF32, false, 2, true, false),
    TG_GROUP(kBf16, kOutBf16, false, 1, true, true),   TG_GROUP(kBf16, kOutF32, false, 1, true, true),
};

const GroupVariant *group_wide_variants(int *count)
{
    *count = (int)(sizeof(kGroup) / sizeof(kGroup[0]));
    return kGroup;
}

}  // namespace tg
