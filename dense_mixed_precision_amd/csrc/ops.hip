// ops.hip -- host side of the operators beside the GEMM (include/mpgemm_ops.h):
// argument validation, the choice of kernel, launches.
#include "mpgemm_ops.h"
#include "mpgemm_ops_query.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

// The GEMM's device code, compiled here for grouped launches, in a namespace
// of its own: a program may link both libraries.
#define MPGEMM_GROUPED
#define mpg mpg_ops
#include "kernels.hpp"

namespace mpg {
#include "i8_kernels.hpp"
#include "narrow_rows.hpp"
#include "token_kernels.hpp"
}  // namespace mpg

#include "host_util.hpp"

namespace {

using mpg::GemmArgs;
using mpg::GroupArgs;
using mpg::I8Args;
using mpg::I8Cfg;
using mpg::kColMajor;
using mpg::kInBF16;
using mpg::kInF16;
using mpg::kRowMajor;
using mpg::PipeCfg;

// ---------------------------------------------------------------------------
// Products of 8-bit codes
// ---------------------------------------------------------------------------
using i8_launch = void (*)(const I8Args &, dim3, hipStream_t);

template <class Cfg, int OUT>
void launch_i8(const I8Args &a, dim3 grid, hipStream_t s)
{
    hipLaunchKernelGGL((mpg::i8_tile<Cfg, OUT>), grid, dim3(Cfg::NT), 0, s, a);
}

struct I8Entry {
    int bm, bn, bkb, stages, waves;
    i8_launch launch[3];  // by output type
};

template <class Cfg>
constexpr I8Entry i8_entry()
{
    return I8Entry{Cfg::BM, Cfg::BN, Cfg::BKB, Cfg::STAGES, Cfg::NW,
                   {&launch_i8<Cfg, mpg::kTF16>, &launch_i8<Cfg, mpg::kTBF16>, &launch_i8<Cfg, mpg::kTF32>}};
}

const I8Entry kI8Table[] = {
    i8_entry<I8Cfg<256, 256, 128, 2, 4, 2>>(),
    i8_entry<I8Cfg<128, 256, 128, 2, 4, 3>>(),
    i8_entry<I8Cfg<128, 128, 128, 2, 4, 3>>(),
    i8_entry<I8Cfg<128, 128, 128, 2, 4, 2>>(),  // 66 KiB of LDS: two workgroups per compute unit
    i8_entry<I8Cfg<64, 128, 128, 2, 4, 3>>(),
    i8_entry<I8Cfg<64, 64, 256, 2, 4, 3>>(),
    i8_entry<I8Cfg<16, 64, 256, 1, 4, 4>>(),
};
enum : int { kI8Big = 0, kI8Wide = 1, kI8Mid = 2, kI8Two = 3, kI8Half = 4, kI8Small = 5, kI8Few = 6 };

bool i8_fits(const I8Entry &e, int64_t lda, int64_t ldw, int64_t K)
{
    return span_fits(e.bm, lda, K, 1) && span_fits(e.bn, ldw, K, 1);
}

// The narrow kernel by the size of its grid: 4 waves with 8 loads in flight
// each where there are workgroups enough to fill the compute units several
// times over, else 8 waves with 4 (8-bit codes, 64 rows over 64 experts of
// 2048x2048, 8192 workgroups: 48.0 against 58.9 us; 16x4096x4096, 256
// workgroups: 6.7 against 6.4; 1x1024x16384, 64: 12.2 against 11.3).
constexpr int64_t kNarrowManyWgs = 1024;

int narrow_waves(int64_t grid) { return grid >= kNarrowManyWgs ? 4 : 8; }

template <int IN, int OUT>
void launch_narrow(const mpg::NarrowArgs &a, int64_t grid, hipStream_t s)
{
    if (narrow_waves(grid) == 4)
        hipLaunchKernelGGL((mpg::narrow_rows<IN, OUT, 8, 4>), dim3((unsigned)grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::narrow_rows<IN, OUT, 4, 8>), dim3((unsigned)grid), dim3(512), 0, s, a);
}

using narrow_launch = void (*)(const mpg::NarrowArgs &, int64_t, hipStream_t);

const narrow_launch kNarrowI8Launch[3] = {&launch_narrow<mpg::kNarrowI8, mpg::kTF16>,
                                          &launch_narrow<mpg::kNarrowI8, mpg::kTBF16>,
                                          &launch_narrow<mpg::kNarrowI8, mpg::kTF32>};

// 256x256 tiles where they take at most a third of the 128x128 tiles' rounds
// over the compute units (us; 16-bit, 32768 rows over 32 experts of 2048x2048:
// 271, 128x256 329, 128x128 443, gradient by the weights 332, 396, 498; 8-bit
// 4096^3 58, 73, 89).
bool big_tiles_win(int64_t t256, int64_t t128) { return 3 * cdiv(t256, kNumCu) <= cdiv(t128, kNumCu); }

// A round of 128x256 tiles takes 1.5 to 1.8 times as long as one of 128x128
// (16-bit, 8192 rows over 32 experts 91, 128x128 124; 8-bit 2048x4096x4096
// 36, 128x128 46, 256x256 48).  At short K it is the writing of C, where two
// 128x128 tiles a unit do better (K = 512, 6560 rows over 82 experts of 1379:
// 16-bit 31 against 39, 8-bit 27 against 30).
bool wide_tiles_win(int64_t twide, int64_t t128, int64_t K)
{
    return K > 512 && 8 * cdiv(twide, kNumCu) <= 5 * cdiv(t128, kNumCu);
}

// The narrow kernel's workgroups split K over their waves, which fills more of
// the chip than the tiles where C is small: up to this many of its 16x16 tiles
// (8 bits 67x46x7908 6.9 us against 15.5 with 16x64 tiles, 256x256x4096 6.5
// and 9.1, 24x4096x4096, 512 tiles, 9.9 and 12.1, 219x646x5295, 574, 40 and 19;
// 16 bits, 500 rows over 4 groups of 128x4096 10.2 and 17.5 with 32x64, 80 rows
// over 2 of 2048x1024, 768, 9.1 and 7.2).
constexpr int64_t kNarrowFewTiles = 512;

// Table entry of an 8-bit product, or -1 for the narrow kernel.  By sweeps of
// every entry (us, graph-replayed, M, N, K in order, one set of operands: what
// fits the memory-side cache is read from there; three sets in turn take
// 128x8192x8192 29 and 256x8192x8192 40), besides the rules above:
//   up to 16 rows a group: narrow (8x8192x8192 15.1, 16x64 tiles 15.8;
//     16x4096x4096 6.4 against 9.3), but 64x128 tiles for 5 rows and more
//     a group over at least 512 of them (512 rows over 64 experts of
//     2048x2048 50.2 against 60.9; 64 rows 48.0 narrow against 59);
//   128x128 from 192 tiles (512x8192x8192 49.0, 64x128 54.0; 2048^3 15.2
//     against 16.0; below, 256x8192x8192, 128 tiles, 40.0 against 32.9), with
//     two ring stages and two workgroups per compute unit where there are
//     more tiles than units, or at short K (16384 rows over 32 experts of
//     2048x2048 108 against 127 with three; 6560 over 82 of 59x1379 20 against
//     29; 2048^3 16.0 against 15.3);
//   64x128 from 129 tiles (1024x2048x2048 10.5, 64x64 14.5; 128x8192x8192,
//     128 tiles, 32.5 against 22.6);
//   64x64 from 128 tiles above 32 rows (128x8192x8192 22.6, 16x64 39.4;
//     512x2048x2048 8.2 against 13.9; 32x8192x8192 19.3 against 16.7);
//   else 16x64 (128x2048x2048, 64 tiles of 64x64: 6.1 against 7.1).
int select_i8(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw)
{
    const int64_t per = cdiv(M, groups);
    auto tiles = [&](int64_t bm, int64_t bn) { return likely_tiles(M, groups, bm, cdiv(N, bn)); };
    auto fits = [&](int id) { return i8_fits(kI8Table[id], lda, ldw, K); };
    if (tiles(16, 16) <= kNarrowFewTiles)
        return -1;
    if (per <= 16)
        return per > 4 && groups > 1 && tiles(64, 128) >= 512 && fits(kI8Half) ? kI8Half : -1;
    if (per > 128 && N > 128 && big_tiles_win(tiles(256, 256), tiles(128, 128)) && fits(kI8Big))
        return kI8Big;
    if (per > 64 && N > 128 && wide_tiles_win(tiles(128, 256), tiles(128, 128), K) && fits(kI8Wide))
        return kI8Wide;
    if (per > 64 && tiles(128, 128) >= 192 && fits(kI8Mid))
        return tiles(128, 128) > kNumCu || K <= 512 ? kI8Two : kI8Mid;
    if (tiles(64, 128) > 128 && fits(kI8Half))
        return kI8Half;
    if (per > 32 && tiles(64, 64) >= 128 && fits(kI8Small))
        return kI8Small;
    return fits(kI8Few) ? kI8Few : -1;
}

// ---------------------------------------------------------------------------
// Grouped 16-bit products
// ---------------------------------------------------------------------------
using grouped_launch = void (*)(const GemmArgs &, const GroupArgs &, dim3, hipStream_t);

// `launch` streams C past the caches; `launch_plain` does not (the same where
// an entry has one form only).  Lines that a row of C shares with the next
// cost up to half more time streamed where C is much of the work: 256-column
// tiles (us; 32768 rows over 32 experts of 2048x2049 326 plain, 376 streamed;
// 65536 over 8 of 256x1030 112 and 173; whole lines 278 and 287, 80 and 79) and
// 128x128 ones two to a compute unit (both gradients of 9 rows over 101
// experts of 1888x1381 314 and 545).
struct GroupedEntry {
    int bm, bn, bk, stages, waves;
    grouped_launch launch, launch_plain;
};

template <class Cfg, bool STREAM>
void launch_grouped(const GemmArgs &a, const GroupArgs &g, dim3 grid, hipStream_t s)
{
    hipLaunchKernelGGL((mpg::gemm_grouped_pipe<Cfg, STREAM>), grid, dim3(Cfg::NT), 0, s, a, g);
}

template <class Cfg, bool BOTH = false>
constexpr GroupedEntry grouped_entry()
{
    return GroupedEntry{Cfg::BM, Cfg::BN, Cfg::BK, Cfg::STAGES, Cfg::NT / 64, &launch_grouped<Cfg, true>,
                        &launch_grouped<Cfg, !BOTH>};
}

// The tiles of one form of the product.  Where the groups split the rows
// (A row-major): 256x256, 128x256, 128x128 with two ring stages (64 KiB of LDS:
// two workgroups per compute unit) or three, 64x128 and 32x64; where they split
// K (A column-major): 256x256, 128x256, 128x128 with two stages and 64x64.
enum : int { kGroupedBig = 0, kGroupedWide = 1, kGroupedTwo = 2, kGroupedMid = 3, kGroupedHalf = 4, kGroupedFew = 5,
             kWgradSmall = 3 };

template <int LB, int IN>
const GroupedEntry *rows_table()
{
    static constexpr GroupedEntry table[] = {
        grouped_entry<PipeCfg<256, 256, 64, 2, 4, 2, kRowMajor, LB, IN, 1, 16>, true>(),
        grouped_entry<PipeCfg<128, 256, 64, 2, 4, 3, kRowMajor, LB, IN, 1, 16>, true>(),
        grouped_entry<PipeCfg<128, 128, 64, 2, 4, 2, kRowMajor, LB, IN>, true>(),
        grouped_entry<PipeCfg<128, 128, 64, 2, 4, 3, kRowMajor, LB, IN>>(),
        grouped_entry<PipeCfg<64, 128, 64, 2, 4, 3, kRowMajor, LB, IN, 1, 16>>(),
        grouped_entry<PipeCfg<32, 64, 128, 2, 4, 3, kRowMajor, LB, IN, 1, 16>>(),
    };
    return table;
}

template <int IN>
const GroupedEntry *wgrad_table()
{
    static constexpr GroupedEntry table[] = {
        grouped_entry<PipeCfg<256, 256, 64, 2, 4, 2, kColMajor, kRowMajor, IN, 1, 16>, true>(),
        grouped_entry<PipeCfg<128, 256, 64, 2, 4, 3, kColMajor, kRowMajor, IN, 1, 16>, true>(),
        grouped_entry<PipeCfg<128, 128, 64, 2, 4, 2, kColMajor, kRowMajor, IN>, true>(),
        grouped_entry<PipeCfg<64, 64, 64, 2, 2, 2, kColMajor, kRowMajor, IN>>(),
    };
    return table;
}

const GroupedEntry *grouped_family(int la, int lb, int in)
{
    if (la == kColMajor)
        return in == kInBF16 ? wgrad_table<kInBF16>() : wgrad_table<kInF16>();
    if (lb == kColMajor)
        return in == kInBF16 ? rows_table<kColMajor, kInBF16>() : rows_table<kColMajor, kInF16>();
    return in == kInBF16 ? rows_table<kRowMajor, kInBF16>() : rows_table<kRowMajor, kInF16>();
}

// Do the rows of an FP32 C start on 128-byte lines?
bool whole_lines(const float *C, int64_t ldc) { return aligned(C, 128) && ldc % 32 == 0; }

bool grouped_fits(const GroupedEntry &e, int la, int lb, int64_t lda, int64_t ldb, int64_t ldc)
{
    return (la == kRowMajor ? span_fits(e.bm, lda, e.bk, 2) : span_fits(e.bk, lda, e.bm, 2)) &&
           (lb == kRowMajor ? span_fits(e.bk, ldb, e.bn, 2) : span_fits(e.bn, ldb, e.bk, 2)) &&
           span_fits(e.bm, ldc, e.bn, 4);
}

// Table entry of a grouped product whose rows the groups split, or -1 for the
// narrow kernel (column-major B).  By sweeps of every entry (us,
// graph-replayed; "per" rows a group, N = K = 2048, 32 or 64 experts where
// nothing else stands), besides the rules above:
//   up to 16 per and B column-major: narrow for at most 4 per (1 per over 64
//     experts 95, 32x64 106) or few tiles, else 32x64 (8 per over 64 experts
//     108 against 123);
//   128x128 above 64 per from 128 tiles (3000 rows, 13 experts of 617x800,
//     182 tiles: 12.1, 64x128 15.0), two workgroups per compute unit where
//     there are more tiles than units, or at short K (18000 rows, 13 experts
//     45 against 52 with three stages; 6560 over 82 of 59x1379 17.5 against
//     24; 4096 over 32 89 against 80);
//   64x128 from 192 tiles above 32 per (64 per: 67, 32x64 77; 54 against 78
//     with B row-major), or at any per with B row-major (32 per: 52 against
//     58; B column-major 65 against 58);
//   else 32x64 (300 rows, 13 experts of 617x800: 6.8, 64x128 9.0).
int select_grouped(const GroupedEntry *table, int lb, int64_t groups, int64_t R, int64_t N, int64_t K, int64_t lda,
                   int64_t ldb, int64_t ldc)
{
    const int64_t per = cdiv(R, groups);
    auto tiles = [&](int64_t bm, int64_t bn) { return likely_tiles(R, groups, bm, cdiv(N, bn)); };
    auto fits = [&](int id) { return grouped_fits(table[id], kRowMajor, lb, lda, ldb, ldc); };
    if (lb == kColMajor && (tiles(16, 16) <= kNarrowFewTiles || (per <= 16 && (per <= 4 || tiles(32, 64) < 512))))
        return -1;
    if (per > 64 && N > 128) {
        if (per > 128 && big_tiles_win(tiles(256, 256), tiles(128, 128)) && fits(kGroupedBig))
            return kGroupedBig;
        if (wide_tiles_win(tiles(128, 256), tiles(128, 128), K) && fits(kGroupedWide))
            return kGroupedWide;
    }
    if (per > 64 && tiles(128, 128) >= kNumCu / 2 && fits(kGroupedMid))
        return tiles(128, 128) > kNumCu || K <= 256 ? kGroupedTwo : kGroupedMid;
    if ((per > 32 || lb == kRowMajor) && tiles(64, 128) >= 192 && fits(kGroupedHalf))
        return kGroupedHalf;
    return kGroupedFew;
}

// Table entry of a gradient by the weights (M x N per group; the groups split
// K).  Up to 128 rows a group it is the writing of C: 128x128 with two
// workgroups per compute unit, one writing while the other multiplies (512
// rows over 64 experts of 2048x2048 164, 256x256 195; 4096 over 32 112 and
// 115; 32768 over 32 412 and 325).  Below 128 tiles of 128x128, 64x64.
int select_wgrad(const GroupedEntry *table, int64_t groups, int64_t R, int64_t M, int64_t N, int64_t lda, int64_t ldb,
                 int64_t ldc)
{
    auto tiles = [&](int64_t bm, int64_t bn) { return mul_sat(mul_sat(cdiv(M, bm), cdiv(N, bn)), groups); };
    auto fits = [&](int id) { return grouped_fits(table[id], kColMajor, kRowMajor, lda, ldb, ldc); };
    if (cdiv(R, groups) > 128) {
        if (M > 128 && N > 128 && big_tiles_win(tiles(256, 256), tiles(128, 128)) && fits(kGroupedBig))
            return kGroupedBig;
        if (N > 128 && wide_tiles_win(tiles(128, 256), tiles(128, 128), cdiv(R, groups)) && fits(kGroupedWide))
            return kGroupedWide;
    }
    return tiles(128, 128) >= kNumCu / 2 && fits(kGroupedTwo) ? kGroupedTwo : kWgradSmall;
}

// ---------------------------------------------------------------------------
// What a product of checked arguments launches; the queries report it
// ---------------------------------------------------------------------------
struct Choice {
    int error;               // or MPGEMM_OK
    int id;                  // table entry, or -1: the narrow kernel
    int64_t tiles_m, tiles_n, grid;
};

// `groups` 0: without offsets.
Choice choose_i8(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw)
{
    Choice c{};
    if (groups == 0)
        groups = 1;
    if (!span_fits(16, lda, K, 1) || !span_fits(16, ldw, K, 1)) {
        c.error = MPGEMM_ELD;
        return c;
    }
    c.id = select_i8(groups, M, N, K, lda, ldw);
    c.tiles_m = row_tiles(M, groups, c.id < 0 ? 16 : kI8Table[c.id].bm);
    c.tiles_n = cdiv(N, c.id < 0 ? 16 : kI8Table[c.id].bn);
    c.grid = mul_sat(c.tiles_m, c.tiles_n);
    c.error = c.grid > kMaxGrid ? MPGEMM_EDIM : MPGEMM_OK;
    return c;
}

Choice choose_grouped(const GroupedEntry *table, int lb, int64_t groups, int64_t R, int64_t N, int64_t K, int64_t lda,
                      int64_t ldb, int64_t ldc)
{
    Choice c{};
    c.id = select_grouped(table, lb, groups, R, N, K, lda, ldb, ldc);
    if (c.id < 0 && !(span_fits(16, lda, K, 2) && span_fits(16, ldb, K, 2)))
        c.id = kGroupedFew;
    if (c.id >= 0 && !grouped_fits(table[c.id], kRowMajor, lb, lda, ldb, ldc)) {
        c.error = MPGEMM_ELD;
        return c;
    }
    c.tiles_m = row_tiles(R, groups, c.id < 0 ? 16 : table[c.id].bm);
    c.tiles_n = cdiv(N, c.id < 0 ? 16 : table[c.id].bn);
    c.grid = mul_sat(c.tiles_m, c.tiles_n);
    c.error = c.grid > kMaxGrid ? MPGEMM_EDIM : MPGEMM_OK;
    return c;
}

// (tiles of one group's C)
Choice choose_wgrad(const GroupedEntry *table, int64_t groups, int64_t R, int64_t M, int64_t N, int64_t lda, int64_t ldb,
                    int64_t ldc)
{
    Choice c{};
    c.id = select_wgrad(table, groups, R, M, N, lda, ldb, ldc);
    if (!grouped_fits(table[c.id], kColMajor, kRowMajor, lda, ldb, ldc)) {
        c.error = MPGEMM_ELD;
        return c;
    }
    c.tiles_m = cdiv(M, table[c.id].bm);
    c.tiles_n = cdiv(N, table[c.id].bn);
    c.grid = mul_sat(mul_sat(c.tiles_m, c.tiles_n), groups);
    c.error = c.grid > kMaxGrid ? MPGEMM_EDIM : MPGEMM_OK;
    return c;
}

template <class Entry>
mpgemm_ops_kernel report_tile(const Entry &e, int bk, int64_t grid)
{
    return mpgemm_ops_kernel{0, e.bm, e.bn, bk, e.stages, e.waves, grid};
}

mpgemm_ops_kernel report_narrow(int64_t grid) { return mpgemm_ops_kernel{1, 16, 16, 0, 0, narrow_waves(grid), grid}; }

// Dimensions and leading dimensions of the products; no pointers.
int check_i8(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw)
{
    if (groups < 1 || groups > MPGEMM_MAX_GROUPS || M < 0 || N < 0 || K < 0 || M > kMax32 || N > kMax32 ||
        K > MPGEMM_I8_MAX_K)
        return MPGEMM_EDIM;
    return lda < at_least_one(K) || ldw < at_least_one(K) ? MPGEMM_ELD : MPGEMM_OK;
}

int check_grouped(int layout_b, int64_t groups, int64_t R, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc)
{
    if (layout_b != MPGEMM_ROW_MAJOR && layout_b != MPGEMM_COL_MAJOR)
        return MPGEMM_ELAYOUT;
    if (groups < 1 || groups > MPGEMM_MAX_GROUPS || R < 0 || N < 0 || K < 0 || R > kMax32 || N > kMax32 || K > kMax32)
        return MPGEMM_EDIM;
    return lda < at_least_one(K) || ldb < at_least_one(layout_b == MPGEMM_COL_MAJOR ? K : N) || ldc < at_least_one(N)
               ? MPGEMM_ELD
               : MPGEMM_OK;
}

int check_wgrad(int64_t groups, int64_t R, int64_t M, int64_t N, int64_t lda, int64_t ldb, int64_t ldc)
{
    if (groups < 1 || groups > MPGEMM_MAX_GROUPS || R < 0 || M < 0 || N < 0 || R > kMax32 || M > kMax32 || N > kMax32)
        return MPGEMM_EDIM;
    return lda < at_least_one(M) || ldb < at_least_one(N) || ldc < at_least_one(N) ? MPGEMM_ELD : MPGEMM_OK;
}

// ---------------------------------------------------------------------------
// Launches of the row kernels by type
// ---------------------------------------------------------------------------
// Rows in expert order are made token by token, through the inverse of the
// order in a workspace, from 64 MiB of rows: each token is then read once.  Two
// more launches (4 slots a token, 2048 BF16 values, us by rows and by tokens:
// gather 32 MiB 10.5 and 11.3, 64 MiB 20.3 and 19.5, 256 MiB 84.8 and 60.1;
// to codes 12.7 and 13.0, 20.6 and 17.1, 75.1 and 57.9).
constexpr int64_t kByTokensBytes = (int64_t)64 << 20;

int64_t inverse_bytes(int64_t T, int64_t R, int64_t top_k, int64_t row_bytes)
{
    const int64_t pairs = mul_sat(T, top_k);
    const bool fits = top_k >= 2 && top_k <= kMaxSlots && pairs <= 2 * R && pairs <= kMax32;
    return fits && mul_sat(R, row_bytes) >= kByTokensBytes ? 4 * pairs : 0;
}

void launch_fill(int32_t *v, int64_t count, hipStream_t s)
{
    const int64_t blocks = cdiv(count, 1024);
    hipLaunchKernelGGL(mpg::fill_absent, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s, v, count);
}

// `inverse`: the workspace for the way by tokens, or nullptr.
template <int XT>
void launch_quantize(mpg::QuantArgs a, int32_t *inverse, hipStream_t s)
{
    // 16 lanes per row that they hold in 2 vectors each; in 8 where there are
    // rows for every wave slot at four a wave; a wave where it holds the row
    // in 8 and there are rows for every slot; else one workgroup (BF16, us:
    // 131072 rows of 35 values 13.2 by 16 lanes with 2 vectors, 18.3 with 8,
    // 63.6 by 64; 65536 of 600 24.7 and 40.1, 2048 of 600 4.4 and 3.5).
    constexpr int64_t VN = XT == mpg::kTF32 ? 4 : 8;
    constexpr int64_t kWaveRow = 64 * 8 * VN;
    if (inverse) {
        launch_fill(inverse, (int64_t)a.T * a.top_k, s);
        hipLaunchKernelGGL((mpg::quantize_invert<XT>), row_grid(cdiv(a.R, 256)), dim3(256), 0, s, a, inverse);
        a.inverse = inverse;
        if (a.H <= kWaveRow)
            hipLaunchKernelGGL((mpg::quantize_rows<XT, 64, 8, true>), row_grid(cdiv(a.T, 4)), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((mpg::quantize_rows<XT, 256, 4, true>), row_grid(a.T), dim3(256), 0, s, a);
        return;
    }
    if (a.H <= 16 * 2 * VN)
        hipLaunchKernelGGL((mpg::quantize_rows<XT, 16, 2>), row_grid(cdiv(a.R, 16)), dim3(256), 0, s, a);
    else if (a.R >= 32 * kNumCu && a.H <= 16 * 8 * VN)
        hipLaunchKernelGGL((mpg::quantize_rows<XT, 16, 8>), row_grid(cdiv(a.R, 16)), dim3(256), 0, s, a);
    else if (a.R >= 8 * kNumCu && a.H <= kWaveRow)
        hipLaunchKernelGGL((mpg::quantize_rows<XT, 64, 8>), row_grid(cdiv(a.R, 4)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::quantize_rows<XT, 256, 4>), row_grid(a.R), dim3(256), 0, s, a);
}

// One vector a lane: 16 or 64 lanes per token where they hold its row (16384
// tokens of 8 slots and 35 FP32 values 7.0 us, by 256 threads 22.5).
template <int YT, int OT>
void launch_combine(const mpg::CombineArgs &a, hipStream_t s)
{
    constexpr int64_t VN = YT == mpg::kTF32 ? 4 : 8;
    const int64_t z = cdiv(a.H, 256 * VN);
    if (a.H <= 16 * VN)
        hipLaunchKernelGGL((mpg::combine_rows<YT, OT, 16>), row_grid(cdiv(a.T, 16)), dim3(256), 0, s, a);
    else if (a.H <= 64 * VN)
        hipLaunchKernelGGL((mpg::combine_rows<YT, OT, 64>), row_grid(cdiv(a.T, 4)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::combine_rows<YT, OT, 256>), row_grid(a.T, z < 65535 ? z : 65535), dim3(256), 0, s, a);
}

template <int YT>
void launch_combine(int o_type, const mpg::CombineArgs &a, hipStream_t s)
{
    if (o_type == MPGEMM_T_F16)
        launch_combine<YT, mpg::kTF16>(a, s);
    else if (o_type == MPGEMM_T_BF16)
        launch_combine<YT, mpg::kTBF16>(a, s);
    else
        launch_combine<YT, mpg::kTF32>(a, s);
}

// Rows of up to 256 values: 16 lanes per pair (78743 pairs of 119 values,
// BF16 and FP32: 15.3 us, with 64 lanes 28.9).
template <int DT, int YT, int GT>
void launch_combine_backward(const mpg::CombineBackArgs &a, hipStream_t s)
{
    const int64_t pairs = (int64_t)a.T * a.top_k;
    if (a.H <= 256)
        hipLaunchKernelGGL((mpg::combine_rows_backward<DT, YT, GT, 16>), row_grid(cdiv(pairs, 16)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::combine_rows_backward<DT, YT, GT, 64>), row_grid(cdiv(pairs, 4)), dim3(256), 0, s, a);
}

template <int DT, int YT>
void launch_combine_backward(int g_type, const mpg::CombineBackArgs &a, hipStream_t s)
{
    if (g_type == MPGEMM_T_F16)
        launch_combine_backward<DT, YT, mpg::kTF16>(a, s);
    else if (g_type == MPGEMM_T_BF16)
        launch_combine_backward<DT, YT, mpg::kTBF16>(a, s);
    else
        launch_combine_backward<DT, YT, mpg::kTF32>(a, s);
}

template <int DT>
void launch_combine_backward(int y_type, int g_type, const mpg::CombineBackArgs &a, hipStream_t s)
{
    if (y_type == MPGEMM_T_F16)
        launch_combine_backward<DT, mpg::kTF16>(g_type, a, s);
    else if (y_type == MPGEMM_T_BF16)
        launch_combine_backward<DT, mpg::kTBF16>(g_type, a, s);
    else
        launch_combine_backward<DT, mpg::kTF32>(g_type, a, s);
}

// Pairs one workgroup sorts alone.
constexpr int64_t kRouteOne = 4096;

struct RoutePlan {
    int64_t blocks, per_wave;
};

RoutePlan plan_route(int64_t pairs)
{
    if (pairs <= kRouteOne)
        return RoutePlan{1, cdiv(cdiv(pairs, mpg::kRouteWaves), 64) * 64};
    int64_t blocks = cdiv(pairs, 2048);
    if (blocks > 256)
        blocks = 256;
    const int64_t per_wave = cdiv(cdiv(pairs, blocks * mpg::kRouteWaves), 64) * 64;
    return RoutePlan{cdiv(pairs, per_wave * mpg::kRouteWaves), per_wave};
}

template <int WIDE>
void launch_route(const mpg::RouteArgs &a, int64_t blocks, hipStream_t s)
{
    const size_t one = (size_t)(a.E + 1) * 4;
    const size_t lds = one * (mpg::kRouteWaves + 1) + mpg::kRouteWaves * 4;
    if (blocks == 1) {
        hipLaunchKernelGGL(mpg::route_one<WIDE>, dim3(1), dim3(mpg::kRouteThreads), lds, s, a);
        return;
    }
    hipLaunchKernelGGL(mpg::route_hist<WIDE>, dim3((unsigned)blocks), dim3(mpg::kRouteThreads), one, s, a);
    hipLaunchKernelGGL(mpg::route_place_blocks<WIDE>, dim3((unsigned)blocks), dim3(mpg::kRouteThreads), lds, s, a);
}

}  // namespace

extern "C" {

int mpgemm_quantize_rows(int x_type, int64_t T, int64_t H, const void *X, int64_t ldx,
                         const int32_t *order, int64_t R, int64_t top_k,
                         int8_t *Q, int64_t ldq, float *scale,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!is_type(x_type))
        return MPGEMM_ETYPE;
    if (T < 0 || H < 0 || R < 0 || T > kMax32 || H > kMaxWidth || R > kMax32)
        return MPGEMM_EDIM;
    if (order ? (top_k < 1 || top_k > kMax32) : R != T)
        return MPGEMM_EDIM;
    if (ldx < at_least_one(H) || ldq < at_least_one(H))
        return MPGEMM_ELD;
    if (R == 0)
        return MPGEMM_OK;
    if (scale == nullptr || (H > 0 && (Q == nullptr || (T > 0 && X == nullptr))))
        return MPGEMM_ENULL;
    if (!aligned(X, size_of(x_type)) || !aligned(order, 4) || !aligned(scale, 4) || !aligned(workspace, 4))
        return MPGEMM_EALIGN;
    const mpg::QuantArgs a{X, Q, scale, order, nullptr, ldx, ldq, (int32_t)T, (int32_t)H, (int32_t)R, (int32_t)top_k};
    const int64_t need = order ? inverse_bytes(T, R, top_k, H * size_of(x_type)) : 0;
    int32_t *const inverse = need > 0 && workspace_bytes >= need ? static_cast<int32_t *>(workspace) : nullptr;
    forget_error();
    if (x_type == MPGEMM_T_F16)
        launch_quantize<mpg::kTF16>(a, inverse, stream_of(stream));
    else if (x_type == MPGEMM_T_BF16)
        launch_quantize<mpg::kTBF16>(a, inverse, stream_of(stream));
    else
        launch_quantize<mpg::kTF32>(a, inverse, stream_of(stream));
    return launched();
}

int mpgemm_i8_gemm(int out_type, int64_t groups, int64_t M, int64_t N, int64_t K,
                   const int8_t *A, int64_t lda, const int8_t *W, int64_t ldw, int64_t stride_w,
                   void *C, int64_t ldc, const float *scale_a, const float *scale_w,
                   const float *bias, const int32_t *offsets, void *stream)
{
    if (!is_type(out_type))
        return MPGEMM_ETYPE;
    if (const int error = check_i8(groups, M, N, K, lda, ldw))
        return error;
    if (ldc < at_least_one(N) || stride_w < 0)
        return MPGEMM_ELD;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    if (C == nullptr || scale_a == nullptr || scale_w == nullptr || (K > 0 && (A == nullptr || W == nullptr)) ||
        (groups > 1 && offsets == nullptr))
        return MPGEMM_ENULL;
    if (!aligned(C, size_of(out_type)) || !aligned(scale_a, 4) || !aligned(scale_w, 4) || !aligned(bias, 4) ||
        !aligned(offsets, 4))
        return MPGEMM_EALIGN;
    const GroupArgs group_args{offsets, (int32_t)groups, (int32_t)M, stride_w};
    const Choice c = choose_i8(offsets ? groups : 0, M, N, K, lda, ldw);
    if (c.error)
        return c.error;
    if (c.id < 0) {
        mpg::NarrowArgs a{};
        a.A = reinterpret_cast<const uint8_t *>(A);
        a.W = reinterpret_cast<const uint8_t *>(W);
        a.C = C;
        a.lda = lda;
        a.ldw = ldw;
        a.ldc = ldc;
        a.stride_w = stride_w;
        a.N = (int32_t)N;
        a.KB = (int32_t)K;
        a.tiles_n = (int32_t)c.tiles_n;
        a.groups = group_args;
        a.scale_a = scale_a;
        a.scale_w = scale_w;
        a.bias = bias;
        forget_error();
        kNarrowI8Launch[out_type](a, c.grid, stream_of(stream));
        return launched();
    }
    I8Args a{};
    a.A = A;
    a.W = W;
    a.C = C;
    a.scale_a = scale_a;
    a.scale_w = scale_w;
    a.bias = bias;
    a.lda = lda;
    a.ldw = ldw;
    a.ldc = ldc;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.tiles_n = (int32_t)c.tiles_n;
    a.group_m = 8;
    a.stream_c = aligned(C, 128) && ldc * size_of(out_type) % 128 == 0;
    a.groups = group_args;
    forget_error();
    kI8Table[c.id].launch[out_type](a, dim3((unsigned)c.grid), stream_of(stream));
    return launched();
}

int64_t mpgemm_route_workspace(int64_t pairs, int64_t experts)
{
    if (pairs < 0 || pairs > ((int64_t)1 << 30) || experts < 1 || experts > MPGEMM_MAX_GROUPS)
        return MPGEMM_EDIM;
    const RoutePlan p = plan_route(pairs);
    return p.blocks == 1 || pairs == 0 ? 0 : p.blocks * (experts + 1) * 4;
}

int mpgemm_route(int id_type, int64_t pairs, int64_t experts, const void *ids,
                 int32_t *order, int32_t *position, int32_t *offsets,
                 void *workspace, int64_t workspace_bytes, void *stream)
{
    if (id_type != MPGEMM_ID_I32 && id_type != MPGEMM_ID_I64)
        return MPGEMM_ETYPE;
    const int64_t need = mpgemm_route_workspace(pairs, experts);
    if (need < 0)
        return MPGEMM_EDIM;
    if (offsets == nullptr || (pairs > 0 && (ids == nullptr || order == nullptr || position == nullptr)))
        return MPGEMM_ENULL;
    if (!aligned(ids, id_type == MPGEMM_ID_I64 ? 8 : 4) || !aligned(order, 4) || !aligned(position, 4) ||
        !aligned(offsets, 4) || !aligned(workspace, 4))
        return MPGEMM_EALIGN;
    if (need > 0 && workspace == nullptr)
        return MPGEMM_ENULL;
    if (workspace_bytes < need)
        return MPGEMM_EWORKSPACE;
    forget_error();
    if (pairs == 0) {
        hipLaunchKernelGGL(mpg::route_none, dim3(1), dim3(mpg::kRouteThreads), 0, stream_of(stream), offsets,
                           (int)experts);
        return launched();
    }
    const RoutePlan p = plan_route(pairs);
    mpg::RouteArgs a{};
    a.ids = ids;
    a.order = order;
    a.position = position;
    a.offsets = offsets;
    a.hist = static_cast<int32_t *>(workspace);
    a.pairs = (int32_t)pairs;
    a.E = (int32_t)experts;
    a.bits = 32 - __builtin_clz((unsigned)experts);
    a.per_wave = (int32_t)p.per_wave;
    if (id_type == MPGEMM_ID_I64)
        launch_route<1>(a, p.blocks, stream_of(stream));
    else
        launch_route<0>(a, p.blocks, stream_of(stream));
    return launched();
}

int64_t mpgemm_rows_workspace(int type, int64_t T, int64_t H, int64_t R, int64_t top_k)
{
    if (!is_type(type))
        return MPGEMM_ETYPE;
    if (T < 0 || H < 0 || R < 0 || top_k < 1 || T > kMax32 || H > kMaxWidth || R > kMax32 || top_k > kMax32)
        return MPGEMM_EDIM;
    return inverse_bytes(T, R, top_k, H * size_of(type));
}

int mpgemm_gather_rows(int type, int64_t T, int64_t H, const void *X, int64_t ldx,
                       const int32_t *order, int64_t R, int64_t top_k,
                       void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!is_type(type))
        return MPGEMM_ETYPE;
    const int64_t es = size_of(type);
    if (T < 0 || H < 0 || R < 0 || T > kMax32 || H > kMaxWidth || R > kMax32 || top_k < 1 || top_k > kMax32)
        return MPGEMM_EDIM;
    if (ldx < at_least_one(H) || ldy < at_least_one(H) || ldx > INT64_MAX / 4 || ldy > INT64_MAX / 4)
        return MPGEMM_ELD;
    if (R == 0 || H == 0)
        return MPGEMM_OK;
    if (order == nullptr || Y == nullptr || (T > 0 && X == nullptr))
        return MPGEMM_ENULL;
    if (!aligned(X, es) || !aligned(Y, es) || !aligned(order, 4) || !aligned(workspace, 4))
        return MPGEMM_EALIGN;
    const mpg::GatherArgs a{static_cast<const uint8_t *>(X), static_cast<uint8_t *>(Y), order, ldx * es, ldy * es,
                            (int32_t)T, (int32_t)R, (int32_t)top_k, (int32_t)(H * es)};
    forget_error();
    const int64_t need = inverse_bytes(T, R, top_k, H * es);
    if (need > 0 && workspace != nullptr && workspace_bytes >= need) {
        int32_t *const inverse = static_cast<int32_t *>(workspace);
        launch_fill(inverse, T * top_k, stream_of(stream));
        hipLaunchKernelGGL(mpg::gather_invert, row_grid(cdiv(R, 256)), dim3(256), 0, stream_of(stream), a, inverse);
        hipLaunchKernelGGL(mpg::gather_tokens, row_grid(cdiv(T, 4)), dim3(256), 0, stream_of(stream), a, inverse);
    } else {
        // rows of up to 512 bytes by 16 lanes (131072 rows of 35 BF16 values 8.5
        // us, by 64 lanes 24.8)
        if (a.row_bytes <= 512)
            hipLaunchKernelGGL(mpg::gather_rows<16>, row_grid(cdiv(R, 16)), dim3(256), 0, stream_of(stream), a);
        else
            hipLaunchKernelGGL(mpg::gather_rows<64>, row_grid(cdiv(R, 4)), dim3(256), 0, stream_of(stream), a);
    }
    return launched();
}

int mpgemm_combine_rows(int y_type, int o_type, int64_t T, int64_t top_k, int64_t H, int64_t R,
                        const void *Y, int64_t ldy, const int32_t *position, const float *weights,
                        void *O, int64_t ldo, void *stream)
{
    if (!is_type(y_type) || !is_type(o_type))
        return MPGEMM_ETYPE;
    if (T < 0 || H < 0 || R < 0 || top_k < 0 || T > kMax32 || H > kMaxWidth || R > kMax32 || top_k > kMaxSlots)
        return MPGEMM_EDIM;
    if (ldy < at_least_one(H) || ldo < at_least_one(H))
        return MPGEMM_ELD;
    if (T == 0 || H == 0)
        return MPGEMM_OK;
    if (O == nullptr || (top_k > 0 && (position == nullptr || (R > 0 && Y == nullptr))))
        return MPGEMM_ENULL;
    if (!aligned(Y, size_of(y_type)) || !aligned(O, size_of(o_type)) || !aligned(position, 4) || !aligned(weights, 4))
        return MPGEMM_EALIGN;
    const mpg::CombineArgs a{Y, O, position, weights, ldy, ldo, (int32_t)T, (int32_t)H, (int32_t)R, (int32_t)top_k};
    forget_error();
    if (y_type == MPGEMM_T_F16)
        launch_combine<mpg::kTF16>(o_type, a, stream_of(stream));
    else if (y_type == MPGEMM_T_BF16)
        launch_combine<mpg::kTBF16>(o_type, a, stream_of(stream));
    else
        launch_combine<mpg::kTF32>(o_type, a, stream_of(stream));
    return launched();
}

int mpgemm_combine_rows_backward(int d_type, int y_type, int dy_type,
                                 int64_t T, int64_t top_k, int64_t H, int64_t R,
                                 const void *dO, int64_t ldo, const void *Y, int64_t ldy,
                                 const int32_t *position, const float *weights,
                                 void *dY, int64_t lddy, float *dweights, void *stream)
{
    if (!is_type(d_type) || !is_type(y_type) || !is_type(dy_type))
        return MPGEMM_ETYPE;
    if (T < 0 || H < 0 || R < 0 || top_k < 0 || T > kMax32 || H > kMaxWidth || R > kMax32 || top_k > kMax32 ||
        mul_sat(T, top_k) > kMax32)
        return MPGEMM_EDIM;
    if (ldo < at_least_one(H) || lddy < at_least_one(H) || (dweights && ldy < at_least_one(H)))
        return MPGEMM_ELD;
    if (T == 0 || top_k == 0)
        return MPGEMM_OK;
    if (position == nullptr || (H > 0 && (dO == nullptr || (R > 0 && (dY == nullptr || (dweights && Y == nullptr))))))
        return MPGEMM_ENULL;
    if (!aligned(dO, size_of(d_type)) || !aligned(dY, size_of(dy_type)) ||
        (dweights && !aligned(Y, size_of(y_type))) || !aligned(position, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return MPGEMM_EALIGN;
    const mpg::CombineBackArgs a{dO, Y, dY, dweights, position, weights, ldo, ldy, lddy,
                                 (int32_t)T, (int32_t)H, (int32_t)R, (int32_t)top_k};
    forget_error();
    if (d_type == MPGEMM_T_F16)
        launch_combine_backward<mpg::kTF16>(y_type, dy_type, a, stream_of(stream));
    else if (d_type == MPGEMM_T_BF16)
        launch_combine_backward<mpg::kTBF16>(y_type, dy_type, a, stream_of(stream));
    else
        launch_combine_backward<mpg::kTF32>(y_type, dy_type, a, stream_of(stream));
    return launched();
}

int mpgemm_grouped(int in_type, int layout_b, int64_t groups, int64_t R, int64_t N, int64_t K,
                   const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b,
                   float *C, int64_t ldc, float alpha, float beta,
                   const int32_t *offsets, void *stream)
{
    if (in_type != MPGEMM_IN_F16 && in_type != MPGEMM_IN_BF16)
        return MPGEMM_ETYPE;
    if (const int error = check_grouped(layout_b, groups, R, N, K, lda, ldb, ldc))
        return error;
    if (stride_b < 0)
        return MPGEMM_ELD;
    if (R == 0 || N == 0)
        return MPGEMM_OK;
    const bool reads = K > 0 && alpha != 0.0f;
    if (C == nullptr || offsets == nullptr || (reads && (A == nullptr || B == nullptr)))
        return MPGEMM_ENULL;
    if (!aligned(C, 4) || !aligned(offsets, 4) || (reads && (!aligned(A, 2) || !aligned(B, 2))))
        return MPGEMM_EALIGN;
    const GroupArgs group_args{offsets, (int32_t)groups, (int32_t)R, stride_b};
    const GroupedEntry *const table = grouped_family(kRowMajor, layout_b, in_type);
    const Choice c = choose_grouped(table, layout_b, groups, R, N, K, lda, ldb, ldc);
    if (c.error)
        return c.error;
    if (c.id < 0) {
        mpg::NarrowArgs a{};
        a.A = reinterpret_cast<const uint8_t *>(A);
        a.W = reinterpret_cast<const uint8_t *>(B);
        a.C = C;
        a.lda = 2 * lda;
        a.ldw = 2 * ldb;
        a.ldc = ldc;
        a.stride_w = 2 * stride_b;
        a.N = (int32_t)N;
        a.KB = (int32_t)(2 * K);
        a.tiles_n = (int32_t)c.tiles_n;
        a.groups = group_args;
        a.alpha = alpha;
        a.beta = beta;
        forget_error();
        if (in_type == MPGEMM_IN_BF16)
            launch_narrow<kInBF16, mpg::kTF32>(a, c.grid, stream_of(stream));
        else
            launch_narrow<kInF16, mpg::kTF32>(a, c.grid, stream_of(stream));
        return launched();
    }
    GemmArgs a{};
    a.A = A;
    a.B = B;
    a.C = C;
    a.M = R;
    a.N = N;
    a.K = K;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.alpha = alpha;
    a.beta = beta;
    a.tiles_n = (int32_t)c.tiles_n;
    a.group_m = 8;
    a.splits = 1;
    forget_error();
    const GroupedEntry &e = table[c.id];
    (whole_lines(C, ldc) ? e.launch : e.launch_plain)(a, group_args, dim3((unsigned)c.grid), stream_of(stream));
    return launched();
}

int mpgemm_grouped_wgrad(int in_type, int64_t groups, int64_t R, int64_t M, int64_t N,
                         const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                         float *C, int64_t ldc, int64_t stride_c, float alpha, float beta,
                         const int32_t *offsets, void *stream)
{
    if (in_type != MPGEMM_IN_F16 && in_type != MPGEMM_IN_BF16)
        return MPGEMM_ETYPE;
    if (const int error = check_wgrad(groups, R, M, N, lda, ldb, ldc))
        return error;
    if (stride_c < 0)
        return MPGEMM_ELD;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    // (one group's C may not run into the next one's)
    if (groups > 1 && stride_c < add_sat(mul_sat(M - 1, ldc), N))
        return MPGEMM_ELD;
    const bool reads = R > 0 && alpha != 0.0f;
    if (C == nullptr || offsets == nullptr || (reads && (A == nullptr || B == nullptr)))
        return MPGEMM_ENULL;
    if (!aligned(C, 4) || !aligned(offsets, 4) || (reads && (!aligned(A, 2) || !aligned(B, 2))))
        return MPGEMM_EALIGN;
    const GroupedEntry *const table = grouped_family(kColMajor, kRowMajor, in_type);
    const Choice c = choose_wgrad(table, groups, R, M, N, lda, ldb, ldc);
    if (c.error)
        return c.error;
    GemmArgs a{};
    a.A = A;
    a.B = B;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = R;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.alpha = alpha;
    a.beta = beta;
    a.tiles_m = (int32_t)c.tiles_m;
    a.tiles_n = (int32_t)c.tiles_n;
    a.group_m = 8;
    a.splits = 1;
    forget_error();
    const GroupedEntry &e = table[c.id];
    const bool lines = whole_lines(C, ldc) && stride_c % 32 == 0;
    (lines ? e.launch : e.launch_plain)(a, GroupArgs{offsets, (int32_t)groups, (int32_t)R, stride_c},
                                        dim3((unsigned)c.grid), stream_of(stream));
    return launched();
}

int mpgemm_i8_query(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw,
                    mpgemm_ops_kernel *out)
{
    if (const int error = check_i8(groups == 0 ? 1 : groups, M, N, K, lda, ldw))
        return error;
    if (out == nullptr)
        return MPGEMM_ENULL;
    *out = mpgemm_ops_kernel{};
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    const Choice c = choose_i8(groups, M, N, K, lda, ldw);
    if (c.error)
        return c.error;
    *out = c.id < 0 ? report_narrow(c.grid) : report_tile(kI8Table[c.id], kI8Table[c.id].bkb, c.grid);
    return MPGEMM_OK;
}

int mpgemm_grouped_query(int layout_b, int64_t groups, int64_t R, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                         int64_t ldc, mpgemm_ops_kernel *out)
{
    if (const int error = check_grouped(layout_b, groups, R, N, K, lda, ldb, ldc))
        return error;
    if (out == nullptr)
        return MPGEMM_ENULL;
    *out = mpgemm_ops_kernel{};
    if (R == 0 || N == 0)
        return MPGEMM_OK;
    // (the tiles are the same for both input types)
    const GroupedEntry *const table = grouped_family(kRowMajor, layout_b, kInF16);
    const Choice c = choose_grouped(table, layout_b, groups, R, N, K, lda, ldb, ldc);
    if (c.error)
        return c.error;
    *out = c.id < 0 ? report_narrow(c.grid) : report_tile(table[c.id], table[c.id].bk, c.grid);
    return MPGEMM_OK;
}

int mpgemm_grouped_wgrad_query(int64_t groups, int64_t R, int64_t M, int64_t N, int64_t lda, int64_t ldb, int64_t ldc,
                               mpgemm_ops_kernel *out)
{
    if (const int error = check_wgrad(groups, R, M, N, lda, ldb, ldc))
        return error;
    if (out == nullptr)
        return MPGEMM_ENULL;
    *out = mpgemm_ops_kernel{};
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    const GroupedEntry *const table = grouped_family(kColMajor, kRowMajor, kInF16);
    const Choice c = choose_wgrad(table, groups, R, M, N, lda, ldb, ldc);
    if (c.error)
        return c.error;
    *out = report_tile(table[c.id], table[c.id].bk, c.grid);
    return MPGEMM_OK;
}

}  // extern "C"
