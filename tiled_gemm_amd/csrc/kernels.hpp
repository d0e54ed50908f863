// Kernel argument blocks and launcher entry points shared by the HIP kernel
// translation units and the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "layout.hpp"

namespace tg {

// kMx8 / kMx4: MX block-scaled e4m3 / e2m1 operands, one E8M0 scale per 32
// elements along K.  kI8: int8 A and B; kW4A8: int8 A, packed int4 B.
enum Elem { kBf16 = 0, kFp8 = 1, kMx8 = 2, kMx4 = 3, kI8 = 4, kW4A8 = 5 };
enum Out { kOutF32 = 0, kOutBf16 = 1 };

// Epilogue operands (device pointers): C = act((acc * s_a) * s_b + bias), and
// in the extended epilogue (the variants' launch_ex) + res, with the
// pre-activation also written to pre.
enum EpiAct { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };
struct EpiArgs {
    const float *sa;        // nullptr (1), one value for every row, or one per row of C
    const float *sb;        // nullptr (1), one value for every column, or one per column
    const float *bias;      // nullptr (0) or one per column
    int32_t sa_rows;        // 0: sa[0] for every row; 1: sa[row]
    int32_t sb_cols;        // 0: sb[0] for every column; 1: sb[col]
    int32_t act;            // EpiAct
    const void *res;        // launch_ex: nullptr (0) or M x N of C's type, may be C itself
    void *pre;              // launch_ex: nullptr or M x N of C's type
};

// Ragged row groups (the grouped kernels only; see group.hpp).
struct GroupArgs {
    const int32_t *offsets;     // groups + 1 row offsets, device data
    const int32_t *row_index;   // nullptr, or the row of A behind every row of C
    int32_t groups;
    int32_t rows;               // rows the grouped operands have room for
    int32_t a_rows;             // rows of A behind row_index
    int64_t b_stride;           // bytes from one group's B to the next
};

struct TiledArgs {
    const void *A;
    const void *B;
    void *C;
    EpiArgs epi;
    int32_t M, N;
    int32_t kbytes;         // bytes of one row of A (K * elem_bytes)
    int32_t k_tiles;        // ceil(kbytes / 128)
    int32_t tail_bytes;     // valid bytes of the last K tile: 64 or 128
    int32_t grid, tiles_m, tiles_n, group_m;
    // MX operands only: the block-scale images of A and B (see
    // BscaleArgs) and their number of 4-slice groups along K.
    const uint8_t *sa_img;
    const uint8_t *sb_img;
    int32_t s_groups;
    int32_t kbytes_b;       // bytes of one row of B (kbytes, or kbytes / 2 for int4 B)
    int32_t K;              // elements along K
    int32_t ldb_bytes;      // B stored K x N: bytes of one row of B (N * elem_bytes)
    int32_t lda_bytes;      // A stored K x M: bytes of one row of A (M * elem_bytes)
    // Split K: with splits > 1 the launch has grid = tiles * splits
    // workgroups; workgroup g takes tile g % tiles and the split_steps K steps
    // starting at step (g / tiles) * split_steps (the last split: the rest),
    // and writes its fp32 partial tile to C + (g / tiles) * M * N * 4 bytes
    // with the identity epilogue.  splits == 1: the whole K, C as given.
    int32_t splits;
    int32_t split_steps;
    GroupArgs grp;
};

// Sum of the split-K partials and the epilogue: C[m][n] = cvt(epi(sum over
// s in order of W[s][m][n])), W holding `splits` fp32 M x N matrices.
struct SplitReduceArgs {
    const float *W;
    void *C;
    EpiArgs epi;
    int32_t M, N;
    int32_t splits;
    int32_t out;            // kOutF32 or kOutBf16
    bool ex;                // extended epilogue (epi.res, epi.pre)
};

// Block-scale image of an MX operand with R rows: the bytes
// (ceil(R / 64), G, 64, 4, 4) in row-major order -- row quad (64 rows), group
// of 4 MFMA K-slices (128 elements each), lane l, 16-row block b of the quad,
// slice s of the group -- holding the E8M0 scale of row 64 quad + 16 b + l % 16
// for the 32 elements of slice 4 g + s that lane l feeds the MFMA
// (elements 32 (l / 16) .. +31 of the slice); 127 (unit scale) past the rows
// or the blocks.  One 16-byte load per lane brings a wave the scales of 4 row
// blocks for 4 K-slices.
struct BscaleArgs {
    const uint8_t *src;     // R x (K / 32) E8M0 bytes, row-major
    uint8_t *dst;           // the image
    int32_t rows;           // R
    int32_t kblocks;        // K / 32
    int32_t groups;         // G = ceil(ceil(K / 128) / 4)
    int32_t quads;          // ceil(R / 64)
    // 0: the layout above.  1: the 32x32x64 MFMA's (MXFP4 tile kernel): word
    // w of lane l, byte b holds row 64 quad + 32 (w / 2) + l % 32, K block
    // 16 g + 2 (2 b + w % 2) + l / 32, so one 16-byte load per lane brings
    // both 32-row halves of a quad for the 8 64-element slices of a group.
    int32_t form;
};

struct SkinnyArgs {
    const void *A;
    const void *B;
    void *C;
    EpiArgs epi;
    int32_t M, N;
    int32_t kbytes;
    int32_t k_tiles;
    int32_t tail_bytes;
    int32_t kbytes_b;       // bytes of one row of B (kbytes, or kbytes / 2 for int4 B)
    // MX operands only: the block-scale images (see BscaleArgs) and their
    // number of 4-slice groups along K.
    const uint8_t *sa_img;
    const uint8_t *sb_img;
    int32_t s_groups;
};

struct PreshuffleArgs {
    const void *B;
    void *Bs;
    Layout src;             // B bytes through the 5 pre-shuffle coordinates
    Layout dst;             // the pre-shuffled image
    int32_t nblocks;        // N / 16
    int32_t kblocks;        // kbytes / 64
};

// Tiled-kernel variants compiled into the library.
struct TiledVariant {
    int bm, bn, wgm, wgn;   // output tile and wave grid (wgm x wgn waves)
    int elem, out;
    bool preshuffled;
    int lds_bytes;
    int lds_stages;         // K steps the LDS ring holds
    hipError_t (*launch)(const TiledArgs &, hipStream_t);
    bool bkn = false;       // B stored K x N
    bool akm = false;       // A stored K x M
    // The kernel with the extended epilogue (residual, saved pre-activation):
    // present for every variant a plan with the planner's own choice can get.
    hipError_t (*launch_ex)(const TiledArgs &, hipStream_t) = nullptr;
};

struct SkinnyVariant {
    int mblocks;            // 16-row blocks of M covered (M <= 16 * mblocks)
    int elem, out;
    int waves;              // waves per workgroup, each taking a slice of K
    int stages;             // LDS stages per wave
    int lds_bytes;
    hipError_t (*launch)(const SkinnyArgs &, int grid, hipStream_t);
    bool preshuffled = false;   // B is the pre-shuffled image (register-staged B)
    hipError_t (*launch_ex)(const SkinnyArgs &, int grid, hipStream_t) = nullptr;   // extended epilogue
};

// A grouped kernel (group.hpp): tiles of bm x bn.
struct GroupVariant {
    int bm, bn, threads;
    int elem, out;
    bool preshuffled, bkn, akm;
    int lds_bytes;
    hipError_t (*launch)(const TiledArgs &, hipStream_t);
};
const GroupVariant *group_wide_variants(int *count);
const GroupVariant *group_tiled_variants(int *count);

constexpr int kMaxGroups = 1024;

struct SortArgs {
    const int32_t *ids;
    int32_t *offsets, *row_token, *slot_row;
    int32_t *counts;            // blocks x groups (workspace); unused with one block
    int32_t slots, topk, groups;
    int32_t blocks, block_slots;    // slots per block, a multiple of 1024
    int32_t id_bits;            // bits that tell the ids 0 .. groups - 1 apart
};
hipError_t launch_group_sort(const SortArgs &, hipStream_t);

struct CombineArgs {
    const void *src;            // src_rows x N
    const void *residual;       // combine: nullptr or tokens x N
    const void *d_out;          // gradient: tokens x N
    void *out;                  // combine: tokens x N; gradient: d_src, src_rows x N
    const int32_t *slot_row;    // tokens x topk
    const float *weights;       // nullptr (1) or tokens x topk
    float *d_weights;           // gradient: nullptr or tokens x topk
    int64_t tokens, N;
    int32_t topk, src_rows;
    int32_t type;               // kOutF32 or kOutBf16
};
hipError_t launch_group_combine(const CombineArgs &, hipStream_t);
hipError_t launch_group_combine_grad(const CombineArgs &, hipStream_t);

struct ActGradArgs {
    const void *d_c, *z;
    void *d_z;
    float *d_bias;              // nullptr or groups x N
    float *partial;             // max_chunks x N (workspace); nullptr without d_bias
    const int32_t *offsets;     // nullptr: one group of M rows
    int64_t N;
    int32_t M, groups;
    int32_t chunk, max_chunks;  // rows per chunk; an upper bound on the chunks of all groups
    int32_t act, type;
};
hipError_t launch_act_grad(const ActGradArgs &, hipStream_t);

constexpr int kSkinnyTileN = 32;
constexpr int kTiledThreads = 256;

const TiledVariant *tiled_variants(int *count);
const TiledVariant *small_variants(int *count);  // extended epilogue only, small tiles
hipError_t launch_split_reduce(const SplitReduceArgs &a, hipStream_t s);
const TiledVariant *pipe_variants(int *count);
const TiledVariant *dma_variants(int *count);
const TiledVariant *mxw_variants(int *count);   // MX on the 32x32x64 scaled MFMA
const SkinnyVariant *skinny_variants(int *count);
hipError_t launch_preshuffle(const PreshuffleArgs &, hipStream_t);
hipError_t launch_bscale_image(const BscaleArgs &, hipStream_t);

// The library's static split-K workspace (gemm_run_ws_noalloc): its device
// address on the current device (looked up on the first call per device).
constexpr size_t kStaticWorkspaceBytes = size_t(64) << 20;
constexpr int kMaxDevices = 64;
hipError_t static_workspace(void **ptr);

}  // namespace tg
