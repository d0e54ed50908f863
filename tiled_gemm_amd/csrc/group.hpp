// Device-side mapping of workgroups to the tiles of ragged row groups.
//
// The groups' offsets are device data, so the host launches an upper bound on
// the number of tiles and every workgroup finds its own: the 64 lanes of a
// wave count the tiles of ceil(G / 64) groups each, one wave-wide prefix sum
// places them, and a ballot names the lane, then a short scalar walk the group.
// One load latency and six lane shifts, about a microsecond, and no table in
// memory that a second launch would have to write first.
#pragma once

#include "device.hpp"
#include "kernels.hpp"

namespace tg {

// Offsets are clamped to [0, rows] here, so no value in them can lead a
// kernel outside its buffers.
__device__ inline int group_lo(const int32_t *off, int g, int rows) { return min(max(off[g], 0), rows); }
__device__ inline int group_hi(const int32_t *off, int g, int rows, int lo) { return min(max(off[g + 1], lo), rows); }

struct GroupScan {
    int excl, incl;     // this lane's groups: tiles before them, tiles up to their end
    int per;            // groups per lane
    int total;          // tiles of all groups (the same in every lane)
};

// How many tiles a group of n rows has; tiles never cross a group.
struct TilesAll {                   // of `tile` rows, the last one ragged
    int tile;
    __device__ int operator()(int n) const { return (n + tile - 1) / tile; }
};
struct TilesHeavy {                 // those with more than half their rows
    int tile;
    __device__ int operator()(int n) const { return (n + tile / 2 - 1) / tile; }
};
struct TilesLight {                 // the last one, where it has at most half
    int tile;
    __device__ int operator()(int n) const { return TilesAll{tile}(n) - TilesHeavy{tile}(n); }
};

template <typename Count>
__device__ inline GroupScan group_scan_by(const int32_t *off, int groups, int rows, Count count)
{
    GroupScan s;
    const int l = (int)(threadIdx.x & 63);
    s.per = (groups + 63) >> 6;
    int n = 0;
    for (int i = 0; i < s.per; ++i) {
        const int g = l * s.per + i;
        if (g < groups) {
            const int lo = group_lo(off, g, rows);
            n += count(group_hi(off, g, rows, lo) - lo);
        }
    }
    int x = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        x += l >= d ? y : 0;
    }
    s.incl = x;
    s.excl = x - n;
    s.total = __builtin_amdgcn_readlane(x, 63);
    return s;
}

__device__ inline GroupScan group_scan(const int32_t *off, int groups, int rows, int tile)
{
    return group_scan_by(off, groups, rows, TilesAll{tile});
}

struct GroupTile {
    int g;              // group
    int lo, hi;         // its rows
    int first;          // tiles before the group
    int tiles;          // its tiles
};

// The group that holds tile t (0 <= t < s.total; the same t in every lane).
template <typename Count>
__device__ inline GroupTile group_find_by(const GroupScan &s, const int32_t *off, int groups, int rows, Count count,
                                          int t)
{
    GroupTile r;
    const unsigned long long m = __ballot(s.incl > t);
    const int lane = __builtin_amdgcn_readfirstlane(__builtin_ctzll(m));
    r.first = __builtin_amdgcn_readlane(s.excl, lane);
    r.g = lane * s.per;
    r.lo = group_lo(off, r.g, rows);
    r.hi = group_hi(off, r.g, rows, r.lo);
    r.tiles = count(r.hi - r.lo);
    for (int i = 1; i < s.per && t >= r.first + r.tiles; ++i) {
        r.first += r.tiles;
        ++r.g;
        r.lo = group_lo(off, r.g, rows);
        r.hi = group_hi(off, r.g, rows, r.lo);
        r.tiles = count(r.hi - r.lo);
    }
    r.g = __builtin_amdgcn_readfirstlane(r.g);
    r.lo = __builtin_amdgcn_readfirstlane(r.lo);
    r.hi = __builtin_amdgcn_readfirstlane(r.hi);
    r.first = __builtin_amdgcn_readfirstlane(r.first);
    r.tiles = __builtin_amdgcn_readfirstlane(r.tiles);
    return r;
}

__device__ inline GroupTile group_find(const GroupScan &s, const int32_t *off, int groups, int rows, int tile, int t)
{
    return group_find_by(s, off, groups, rows, TilesAll{tile}, t);
}

// Workgroup w of `total` renumbered so that each XCD (w % 8) gets a contiguous
// run: neighbours share A rows or B columns in that XCD's L2.
__device__ inline int xcd_run(int w, int total)
{
    const int xcd = w % kXcds, per = total / kXcds, rem = total % kXcds;
    return xcd * per + min(xcd, rem) + w / kXcds;
}

// Restricts a grouped kernel's arguments to the group of this workgroup's
// tile: A, C, M and the epilogue's vectors to the group's rows, B to the
// group's matrix.  *tm, *tn: the tile inside the group.  False: no tile left.
// LIGHT: the groups' last tiles with at most half their rows, which such a
// kernel finishes in about half the time, come after all others, so that
// they and not whole tiles fill the last round of workgroups.
template <int OUT, bool LIGHT>
__device__ inline bool group_enter(TiledArgs &p, int bm, int tiles_n, int group_m, int *tm, int *tn)
{
    const int32_t *off = p.grp.offsets;
    const int groups = p.grp.groups, rows = p.grp.rows;
    // The launch covers the rows there is room for.  What offsets[groups] alone
    // rules out leaves before the scan (a capacity of several times the rows
    // would otherwise pay a scan for every workgroup too many).
    const int64_t most = ((int64_t)group_lo(off, groups, rows) + (int64_t)groups * (bm - 1)) / bm * tiles_n;
    if ((int64_t)blockIdx.x >= most)
        return false;
    const GroupScan s = LIGHT ? group_scan_by(off, groups, rows, TilesHeavy{bm}) : group_scan(off, groups, rows, bm);
    // offsets that run backwards may count more tiles than 32 bits hold work for
    const int total = min((int64_t)s.total * tiles_n, (int64_t)gridDim.x);
    GroupTile g;
    if ((int)blockIdx.x < total) {
        const int v = xcd_run(blockIdx.x, total);
        g = LIGHT ? group_find_by(s, off, groups, rows, TilesHeavy{bm}, v / tiles_n)
                  : group_find(s, off, groups, rows, bm, v / tiles_n);
        const int r = v - g.first * tiles_n;
        const int width = group_m * tiles_n, band = r / width, first = band * group_m;
        const int high = min(g.tiles - first, group_m);
        const int in = r - band * width;
        *tm = first + in % high;
        *tn = in / high;
    } else {
        if constexpr (!LIGHT)
            return false;
        const GroupScan s2 = group_scan_by(off, groups, rows, TilesLight{bm});
        const int k = (int)blockIdx.x - total;
        if (k >= (int64_t)s2.total * tiles_n)
            return false;
        g = group_find_by(s2, off, groups, rows, TilesLight{bm}, k / tiles_n);
        *tm = TilesHeavy{bm}(g.hi - g.lo);
        *tn = k - g.first * tiles_n;
    }
    constexpr size_t OB = OUT == kOutF32 ? 4 : 2;
    const size_t c_off = (size_t)g.lo * (size_t)p.N * OB;
    if (p.grp.row_index) {
        p.grp.row_index += g.lo;
    } else {
        p.A = (const uint8_t *)p.A + (size_t)g.lo * (size_t)p.kbytes;
        if (p.epi.sa && p.epi.sa_rows)
            p.epi.sa += g.lo;
    }
    p.B = (const uint8_t *)p.B + (size_t)g.g * (size_t)p.grp.b_stride;
    p.C = (uint8_t *)p.C + c_off;
    if (p.epi.pre)
        p.epi.pre = (uint8_t *)p.epi.pre + c_off;
    if (p.epi.sb && p.epi.sb_cols)
        p.epi.sb += (size_t)g.g * (size_t)p.N;
    if (p.epi.bias)
        p.epi.bias += (size_t)g.g * (size_t)p.N;
    p.M = g.hi - g.lo;
    return true;
}

// The same for the weight gradient: group g's C, and A and B from its first
// row on, K being its rows.  Every group has tiles_m * tiles_n tiles.
template <int OUT>
__device__ inline void group_enter_inner(TiledArgs &p, int k_rows, int *tm, int *tn)
{
    const int tiles = p.tiles_m * p.tiles_n;
    // Groups in turn, each spread over all XCDs (their rows differ, so an XCD
    // that owned whole groups would finish early or late).
    const int g = (int)blockIdx.x / tiles, r = xcd_run((int)blockIdx.x - g * tiles, tiles);
    const int width = p.group_m * p.tiles_n, band = r / width, first = band * p.group_m;
    const int high = min(p.tiles_m - first, p.group_m);
    const int in = r - band * width;
    *tm = first + in % high;
    *tn = in / high;
    const int lo = group_lo(p.grp.offsets, g, p.grp.rows), hi = group_hi(p.grp.offsets, g, p.grp.rows, lo);
    p.A = (const uint8_t *)p.A + (size_t)lo * (size_t)p.lda_bytes;
    p.B = (const uint8_t *)p.B + (size_t)lo * (size_t)p.ldb_bytes;
    p.C = (uint8_t *)p.C + (size_t)g * (size_t)p.M * (size_t)p.N * (OUT == kOutF32 ? 4u : 2u);
    p.K = __builtin_amdgcn_readfirstlane(hi - lo);
    p.k_tiles = (p.K + k_rows - 1) / k_rows;
    p.tail_bytes = kTileKBytes;
}

// Byte offset in A of byte c of group row `row`: through row_index when there
// is one; past every buffer for rows past the group or an index outside A.
__device__ inline uint32_t group_a_off(const GroupArgs &g, int M, int row, uint32_t kb, uint32_t c)
{
    if (!g.row_index)
        return (uint32_t)row * kb + c;                 // past the group's rows: past the record count
    const int idx = row < M ? g.row_index[row] : -1;
    return (uint32_t)idx < (uint32_t)g.a_rows ? (uint32_t)idx * kb + c : kOobOffset;
}

// The epilogue's vectors, and s_a of one group row, through row_index as well
// (0 for a row of zeros, whose sums are 0 whatever the scale).
__device__ inline EpiView group_epi_view(const EpiArgs &e, const GroupArgs &g, int M, int N)
{
    EpiView v = epi_view(e, M, N);
    if (g.row_index && e.sa_rows)
        v.ra = make_rsrc(e.sa, (uint32_t)g.a_rows * 4u);
    return v;
}
__device__ inline float group_row_scale(const EpiView &v, const GroupArgs &g, int M, int row)
{
    if (!v.has_a || !g.row_index || v.sa_step == 0)
        return epi_row_scale(v, row);
    const int idx = row < M ? g.row_index[row] : -1;
    const uint32_t off = (uint32_t)idx < (uint32_t)g.a_rows ? (uint32_t)idx * 4u : kOobOffset;
    return as_f32(buf_load4(v.ra, off, 0));
}

}  // namespace tg
