// host_util.hpp -- sizes, limits and launches that the host sides of the
// operator libraries share (mpgemm_ops.h's types; each library has its own copy).
#ifndef MPGEMM_HOST_UTIL_HPP
#define MPGEMM_HOST_UTIL_HPP

#include "mpgemm_ops.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

constexpr int kNumCu = 256;
constexpr int64_t kMax32 = 0x7FFFFFFF;
constexpr int64_t kMaxWidth = (int64_t)1 << 28;  // values of a token's row: a row spans at most 1 GiB
// slots of a token: the kernels that walk them in runs of 4 or 8 count in 32 bits
constexpr int64_t kMaxSlots = (int64_t)1 << 30;
constexpr int64_t kMaxSpan = 0x7FFFFFF0;  // bytes a 32-bit buffer offset may reach

int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// Saturating product and sum of sizes >= 0: a saturated value fails every
// limit it is compared with.
int64_t mul_sat(int64_t a, int64_t b)
{
    if (a == 0 || b == 0)
        return 0;
    return a > INT64_MAX / b ? INT64_MAX : a * b;
}
int64_t add_sat(int64_t a, int64_t b) { return a > INT64_MAX - b ? INT64_MAX : a + b; }

bool aligned(const void *p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (uint64_t)(bytes - 1)) == 0; }

bool is_type(int t) { return t == MPGEMM_T_F16 || t == MPGEMM_T_BF16 || t == MPGEMM_T_F32; }
int64_t size_of(int t) { return t == MPGEMM_T_F32 ? 4 : 2; }

// A launch holds fewer than 2^32 threads in one dimension: at most this many
// workgroups of up to 512.
constexpr int64_t kMaxGrid = (int64_t)1 << 22;

// `blocks` workgroups (fewer than 2^31) over x and y; the last ones may have
// nothing to do.
dim3 row_grid(int64_t blocks, int64_t z = 1)
{
    if (blocks <= kMaxGrid)
        return dim3((unsigned)blocks, 1, (unsigned)z);
    return dim3((unsigned)kMaxGrid, (unsigned)cdiv(blocks, kMaxGrid), (unsigned)z);
}

hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

// An error left by an earlier, unrelated call must not be reported as ours.
void forget_error() { (void)hipGetLastError(); }
int launched() { return hipGetLastError() == hipSuccess ? MPGEMM_OK : MPGEMM_ELAUNCH; }

// Do `rows` stored rows of `width` elements, `ld` apart, fit 32-bit buffer
// offsets?
bool span_fits(int64_t rows, int64_t ld, int64_t width, int64_t bytes)
{
    return mul_sat(add_sat(mul_sat(rows, ld), width), bytes) < kMaxSpan;
}

// M tiles of at most `bm` rows that any split of `rows` rows into `groups`
// ranges can make.
int64_t row_tiles(int64_t rows, int64_t groups, int64_t bm)
{
    if (groups <= 1)
        return cdiv(rows, bm);
    const int64_t most = (rows + groups * (bm - 1)) / bm;
    return most < rows ? most : rows;
}

// Tiles that `rows` rows in `groups` groups are likely to make: half a tile
// more per group than the rows alone, one for each group at least.
int64_t likely_tiles(int64_t rows, int64_t groups, int64_t bm, int64_t tiles_n)
{
    const int64_t least = rows < groups ? rows : groups;
    const int64_t likely = groups <= 1 ? cdiv(rows, bm) : cdiv(rows, bm) + groups / 2;
    return mul_sat(likely > least ? likely : least, tiles_n);
}

}  // namespace

#endif  // MPGEMM_HOST_UTIL_HPP
