// groups.hpp -- which product, and which tile of it, a workgroup of a grouped
// launch takes.  Included inside kernels.hpp's namespace by the operator
// library (MPGEMM_GROUPED).
//
// A grouped launch is `groups` products over consecutive rows: group g owns
// rows [offsets[g], offsets[g+1]).  The offsets live in device memory, so
// the host knows only the sum: it launches enough workgroups for any split of
// the rows (row_tiles in ops.hip) and those without a tile leave at once.
//
// Measured (us; BF16, 32 experts of 2048x2048): 32768 rows of equal shares 271
// (B column-major) and 282 (row-major), gradient by the weights 325, against 216
// at the rate of a large library product: FP32 tiles of 256 KiB are written at
// the end of each round of tiles.  With unequal shares 313, 330 and about
// 340: the compute units hold waves 83% (rows) and 93% (weights) of the time.
//
// Offsets are read as untrusted data: each range is clamped to [0, rows], so
// whatever they hold no workgroup leaves the operands.

struct GroupArgs {
    const int32_t *offsets;  // groups + 1 values; nullptr: one group of all rows
    int32_t groups;
    int32_t rows;            // rows of the grouped operands
    int64_t stride;          // elements from one group's B (or C, where K is grouped) to the next
};

struct GroupTile {
    int group, start, rows;  // the group and its rows
    int tm, tn;              // the tile within the group's product
};

__device__ __forceinline__ int clamp_row(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Workgroup id -> position in the tile order, undoing the round-robin
// dispatch over XCDs (as tile_coords does) for nb live workgroups.
__device__ __forceinline__ int xcd_order(int bid, int nb)
{
    const int xcd = bid % kNumXcd;
    const int local = bid / kNumXcd;
    const int per = nb / kNumXcd;
    const int rem = nb % kNumXcd;
    return (xcd < rem) ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
}

// The same with the tiles dealt to the XCDs in runs of 16: a group's tiles
// take as long as it has rows, so whole groups per XCD would leave the XCDs of
// the short ones idle.
__device__ __forceinline__ int dealt_order(int bid, int nb)
{
    constexpr int RUN = 16;
    if (bid >= nb / (RUN * kNumXcd) * (RUN * kNumXcd))
        return bid;
    const int xcd = bid % kNumXcd;
    const int local = bid / kNumXcd;
    return ((local / RUN) * kNumXcd + xcd) * RUN + local % RUN;
}

// Tile of this workgroup among all groups' ceil(rows/bm) x tiles_n tiles,
// groups one after the other.  Every wave works it out for itself (64 groups
// at a time, one per lane, a prefix sum over lanes), so no barrier and no
// LDS: one load of offsets and ~20 lane operations.
__device__ __forceinline__ bool find_row_tile(const GroupArgs &ga, int bm, int tiles_n, int group_m, GroupTile &out)
{
    const int lane = threadIdx.x & 63;
    const int bid = blockIdx.x;
    int g = 0, start = 0, rows = ga.rows, mt = (ga.rows + bm - 1) / bm, t;
    if (ga.offsets == nullptr) {
        const int nb = mt * tiles_n;
        if (bid >= nb)
            return false;
        t = xcd_order(bid, nb);
    } else {
        int s = 0, n = 0, tiles = 0, incl = 0;
        auto load = [&](int first) __attribute__((always_inline)) {
            const int i = first + lane;
            s = n = 0;
            if (i < ga.groups) {
                s = clamp_row(ga.offsets[i], 0, ga.rows);
                n = clamp_row(ga.offsets[i + 1], s, ga.rows) - s;
            }
            tiles = (n + bm - 1) / bm;
            incl = tiles;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(incl, d);
                if (lane >= d)
                    incl += v;
            }
        };
        int64_t total = 0;
        for (int first = 0; first < ga.groups; first += 64) {
            load(first);
            total += __builtin_amdgcn_readlane(incl, 63);
        }
        // (more than the grid only if the groups' ranges overlap)
        const int64_t live = total * tiles_n;
        const int nb = live < (int64_t)gridDim.x ? (int)live : (int)gridDim.x;
        if (bid >= nb)
            return false;
        t = xcd_order(bid, nb);
        int64_t before = 0;
        for (int first = 0; first < ga.groups; first += 64) {
            if (ga.groups > 64)
                load(first);
            const uint64_t past = __ballot((before + incl) * tiles_n > t);
            if (past != 0) {
                const int at = __builtin_ctzll(past);
                g = first + at;
                start = __builtin_amdgcn_readlane(s, at);
                rows = __builtin_amdgcn_readlane(n, at);
                mt = __builtin_amdgcn_readlane(tiles, at);
                before += __builtin_amdgcn_readlane(incl, at) - mt;
                break;
            }
            before += __builtin_amdgcn_readlane(incl, 63);
        }
        t -= (int)(before * tiles_n);
    }
    const int band = group_m * tiles_n;
    const int first_m = (t / band) * group_m;
    const int in_band = t % band;
    const int height = min(mt - first_m, group_m);
    out.group = g;
    out.start = start;
    out.rows = rows;
    out.tm = first_m + in_band % height;
    out.tn = in_band / height;
    return true;
}

// The group with the nth most rows (n from 0; the first of equals first), for
// up to 64 groups, one per lane.  Where a tile takes as long as its group has
// rows, the longest go first and the short ones fill the end.
__device__ __forceinline__ int nth_longest(const GroupArgs &ga, int n)
{
    const int lane = threadIdx.x & 63;
    int rows = -1;
    if (lane < ga.groups) {
        const int s = clamp_row(ga.offsets[lane], 0, ga.rows);
        rows = clamp_row(ga.offsets[lane + 1], s, ga.rows) - s;
    }
    int longer = 0;
    for (int i = 0; i < ga.groups; ++i) {
        const int other = __builtin_amdgcn_readlane(rows, i);
        longer += other > rows || (other == rows && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < ga.groups && longer == n));
}

// The 16-bit grouped products on the pipelined kernel.  A row-major: the
// groups split the rows of A and C, each with a B of its own.  A
// column-major: the groups split K (rows of the stored A and B), each with a
// C of its own.  alpha == 0 reads neither A nor B: K becomes 0.
template <int BM, int BN, bool SPLIT_K>
__device__ __forceinline__ bool locate_group(GemmArgs &args, const GroupArgs &ga, int &tm, int &tn)
{
    if (args.alpha == 0.0f)
        args.K = 0;
    if constexpr (!SPLIT_K) {
        GroupTile t;
        if (!find_row_tile(ga, BM, args.tiles_n, args.group_m, t))
            return false;
        args.A += (int64_t)t.start * args.lda;
        args.C += (int64_t)t.start * args.ldc;
        args.B += (int64_t)t.group * ga.stride;
        args.M = t.rows;
        tm = t.tm;
        tn = t.tn;
    } else {
        const int per = args.tiles_m * args.tiles_n;
        const int t = dealt_order(blockIdx.x, gridDim.x);
        const int place = t / per;
        int g = place;
        if (ga.groups <= 64)
            g = nth_longest(ga, place);
        const int start = clamp_row(ga.offsets[g], 0, ga.rows);
        const int rows = clamp_row(ga.offsets[g + 1], start, ga.rows) - start;
        args.A += (int64_t)start * args.lda;
        args.B += (int64_t)start * args.ldb;
        args.C += (int64_t)g * ga.stride;
        args.K = args.alpha == 0.0f ? 0 : rows;
        const int local = t - place * per;
        // (bands of 4 tile rows: 16 tiles in a row are a 4x4 block)
        const int band = 4 * args.tiles_n;
        const int first_m = (local / band) * 4;
        const int in_band = local % band;
        const int height = min(args.tiles_m - first_m, 4);
        tm = first_m + in_band % height;
        tn = in_band / height;
    }
    return true;
}
