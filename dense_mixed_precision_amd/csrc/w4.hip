// w4.hip -- host side of the products with 4-bit weights (include/mpgemm_w4.h):
// argument validation, the choice of kernel, launches.
#include "mpgemm_w4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

// The GEMM's device code, for its matrix instructions, copies and groups, in a
// namespace of its own: a program may link the other libraries too.
#define MPGEMM_GROUPED
#define mpg mpg_w4
#include "kernels.hpp"

namespace mpg {
#include "copy4.hpp"
#include "elements.hpp"
#include "w4_kernels.hpp"
}  // namespace mpg

#include "host_util.hpp"

namespace {

using mpg::W4Args;

constexpr int64_t kMaxGroup = (int64_t)1 << 28;

bool is_scale_type(int t) { return t == MPGEMM_T_F16 || t == MPGEMM_T_BF16; }

// log2 of a group's size, or -1.
int group_shift(int64_t group)
{
    if (group < 32 || group > kMaxGroup || (group & (group - 1)) != 0)
        return -1;
    return __builtin_ctzll((uint64_t)group);
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
using w4_launch = void (*)(const W4Args &, dim3, hipStream_t);

template <int IN, int GS, int NA, int NF, int WAVES, int STAGES>
void launch_narrow(const W4Args &a, dim3 grid, hipStream_t s)
{
    hipLaunchKernelGGL((mpg::w4_narrow<IN, GS, NA, NF, WAVES, STAGES>), grid, dim3(64 * WAVES), 0, s, a);
}

template <class Cfg>
void launch_tile(const W4Args &a, dim3 grid, hipStream_t s)
{
    hipLaunchKernelGGL(mpg::w4_tile<Cfg>, grid, dim3(Cfg::NT), 0, s, a);
}

struct W4Entry {
    bool narrow;
    int bm, bn, bk, stages, waves;
    w4_launch launch[2][3];  // by input type, group size
};

template <int NA, int NF, int WAVES, int STAGES>
constexpr W4Entry narrow_entry()
{
    using mpg::kCoarse, mpg::kGroup32, mpg::kGroup64, mpg::kInBF16, mpg::kInF16;
    return W4Entry{true, 4 * NA, 16 * NF, 128, STAGES, WAVES,
                   {{&launch_narrow<kInF16, kCoarse, NA, NF, WAVES, STAGES>,
                     &launch_narrow<kInF16, kGroup64, NA, NF, WAVES, STAGES>,
                     &launch_narrow<kInF16, kGroup32, NA, NF, WAVES, STAGES>},
                    {&launch_narrow<kInBF16, kCoarse, NA, NF, WAVES, STAGES>,
                     &launch_narrow<kInBF16, kGroup64, NA, NF, WAVES, STAGES>,
                     &launch_narrow<kInBF16, kGroup32, NA, NF, WAVES, STAGES>}}};
}

template <int BM, int NF, int NW>
constexpr W4Entry tile_entry()
{
    using mpg::kCoarse, mpg::kGroup32, mpg::kGroup64, mpg::kInBF16, mpg::kInF16, mpg::W4Cfg;
    return W4Entry{false, BM, 16 * NF * NW, 128, 3, NW,
                   {{&launch_tile<W4Cfg<kInF16, kCoarse, BM, NF, NW>>, &launch_tile<W4Cfg<kInF16, kGroup64, BM, NF, NW>>,
                     &launch_tile<W4Cfg<kInF16, kGroup32, BM, NF, NW>>},
                    {&launch_tile<W4Cfg<kInBF16, kCoarse, BM, NF, NW>>,
                     &launch_tile<W4Cfg<kInBF16, kGroup64, BM, NF, NW>>,
                     &launch_tile<W4Cfg<kInBF16, kGroup32, BM, NF, NW>>}}};
}

// Narrow kernels by tokens x channels and waves, then tiles.
enum : int {
    kFew4 = 0, kFew16 = 1, kNarrow8 = 2, kNarrow8Four = 3, kNarrow16 = 4, kNarrow16Four = 5, kNarrow32 = 6,
    kNarrow64 = 7, kTile64 = 8, kTile64Wide = 9, kTile128 = 10
};
const W4Entry kTable[] = {
    narrow_entry<1, 1, 8, 3>(), narrow_entry<4, 1, 8, 2>(), narrow_entry<2, 2, 8, 2>(), narrow_entry<2, 2, 4, 2>(),
    narrow_entry<4, 2, 8, 2>(), narrow_entry<4, 2, 4, 2>(), narrow_entry<8, 2, 4, 2>(), narrow_entry<16, 2, 4, 2>(),
    tile_entry<64, 2, 4>(), tile_entry<64, 2, 8>(), tile_entry<128, 2, 8>(),
};

// Table entry of a product.  By sweeps of every entry (us, graph-replayed,
// three sets of operands in turn, M, N, K in order; groups of 128, BF16):
//   the narrow kernel with the smallest tile whose workgroups go around the
//     compute units once: 16x16 (16x1024x8192 8.0, 16x32 10.6; 64x1024x8192 8.6
//     against 11.2), for few tokens 4x16 (1x4096x4096 5.2, 8x32 6.3), then 8x32
//     (8x8192x8192 11.7, 16x32 12.4), 16x32 (128x1024x8192 11.5, 32x32 15.8),
//     32x32 (256x1024x8192 16.1, 64x32 23.3);
//   8 waves where each has 4 steps of K at least, else 4 (8x8192x8192 11.7
//     against 13.3; 8x8192x1024 4.6 against 4.4);
//   past one round, up to 16 rows a group: 4 waves, 8x32 up to 4 rows a group,
//     else 16x32 (64 rows over 64 experts of 2048x2048 25.3 and 29.4; 64 over 8 of
//     4096x4096 25.0 and 21.8; 8 waves 33 to 55);
//   128x256 tiles from 192 of them above 64 rows a group (1024x8192x8192 133,
//     64x256 174; 512x8192x8192, 128 of them, 116 against 88);
//   64x256 from 160 (512x8192x8192 88, 64x128 95; 256x8192x8192, 128 of them, 85
//     against 67);
//   64x128, two workgroups a compute unit, from 192 (256x8192x8192 67, 64x32 89;
//     128x8192x8192, 128 of them, 66 against 46);
//   else 64x32.
// The tiles take K in whole steps of 128 and K >= 128.
//
// Groups of 32 and 64 take the same entries, which a sweep of 1 to 1,024 rows by
// 8192x8192 and of 8 to 1,024 by 4096x4096 bears out within 4% (64x4096x4096 in
// groups of 32: 32x32 13.6, 64x32 20.6; 1024x8192x8192: 128x256 180, 64x256 238).
// Where another entry is faster, in groups of 128 and alike in finer ones:
//   a single matrix just past one round of its tile (us, taken and best):
//     1x8224x8192 16.9 (4x16 14.4), 8x8224x8192 18.8 (8x32 17.0), 20x8224x8192
//     44.3 (16x32 23.9, 32x32 32.6), 32x14336x8192 46.8 (16x32 32.6), 20x28672x8192
//     68.1 (16x32 58.6);
//   unequal groups of 17 to 64 rows on average: 1,200 rows over 32 experts of
//     2048x2048 54.6 (128x256 39.2, 64x128 46.9).
int select_w4(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda)
{
    const int64_t per = cdiv(M, groups);
    auto tiles = [&](int id) { return likely_tiles(M, groups, kTable[id].bm, cdiv(N, kTable[id].bn)); };
    const bool deep = K >= 8 * 4 * 128;
    if (tiles(kFew16) <= kNumCu)
        return per <= 4 ? kFew4 : kFew16;
    if (per <= 8 && tiles(kNarrow8) <= kNumCu)
        return deep ? kNarrow8 : kNarrow8Four;
    if (tiles(kNarrow16) <= kNumCu)
        return deep ? kNarrow16 : kNarrow16Four;
    if (per <= 16)
        return per <= 4 ? kNarrow8Four : kNarrow16Four;
    if (tiles(kNarrow32) <= kNumCu)
        return kNarrow32;
    if (K < 128)
        return kNarrow64;
    if (per > 64 && tiles(kTile128) >= 192 && span_fits(kTable[kTile128].bm, lda, K, 2))
        return kTile128;
    if (tiles(kTile64Wide) >= 160)
        return kTile64Wide;
    return tiles(kTile64) >= 192 ? kTile64 : kNarrow64;
}

struct Choice {
    int error;
    int id;
    int64_t tiles_n, grid;
};

int check_w4(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t group, int64_t lda, int64_t ldq, int64_t lds)
{
    if (groups < 1 || groups > MPGEMM_MAX_GROUPS || M < 0 || N < 0 || K < 0 || M > kMax32 || N > kMax32 ||
        K > kMaxWidth || group_shift(group) < 0)
        return MPGEMM_EDIM;
    const int64_t bytes = cdiv(K, 2), count = cdiv(K, group);
    if (lda < at_least_one(K) || ldq < at_least_one(bytes) || lds < at_least_one(count) || !span_fits(64, lda, K, 2) ||
        !span_fits(32, ldq, bytes, 1) || !span_fits(32, lds, count, 2))
        return MPGEMM_ELD;
    return MPGEMM_OK;
}

// `groups` 0: without offsets.
Choice choose_w4(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda)
{
    Choice c{};
    if (groups == 0)
        groups = 1;
    c.id = select_w4(groups, M, N, K, lda);
    c.tiles_n = cdiv(N, kTable[c.id].bn);
    c.grid = mul_sat(row_tiles(M, groups, kTable[c.id].bm), c.tiles_n);
    c.error = c.grid > kMaxGrid ? MPGEMM_EDIM : MPGEMM_OK;
    return c;
}

// ---------------------------------------------------------------------------
// Rows to codes and back
// ---------------------------------------------------------------------------
template <int WT>
void launch_pack(int s_type, const mpg::W4PackArgs &a, hipStream_t s)
{
    const dim3 grid = row_grid(cdiv((int64_t)a.N * a.parts, 4));
    if (s_type == MPGEMM_T_F16)
        hipLaunchKernelGGL((mpg::w4_pack<WT, mpg::kTF16>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::w4_pack<WT, mpg::kTBF16>), grid, dim3(256), 0, s, a);
}

template <int WT>
void launch_unpack(int s_type, const mpg::W4UnpackArgs &a, hipStream_t s)
{
    const dim3 grid = row_grid(cdiv((int64_t)a.N * a.parts, 4));
    if (s_type == MPGEMM_T_F16)
        hipLaunchKernelGGL((mpg::w4_unpack<mpg::kTF16, WT>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mpg::w4_unpack<mpg::kTBF16, WT>), grid, dim3(256), 0, s, a);
}

// What both directions ask of their arguments; `parts` waves a row, of `span`
// values each.
int check_pack(int w_type, int s_type, int64_t N, int64_t K, int64_t group, const void *W, int64_t ldw, const void *Q,
               int64_t ldq, const void *scale, int64_t lds, int64_t span, int64_t &parts)
{
    if (!is_type(w_type) || !is_scale_type(s_type))
        return MPGEMM_ETYPE;
    if (N < 0 || K < 0 || N > kMax32 || K > kMaxWidth || group_shift(group) < 0)
        return MPGEMM_EDIM;
    parts = cdiv(K, span);
    if (mul_sat(N, parts) > kMax32)
        return MPGEMM_EDIM;
    if (ldw < at_least_one(K) || ldq < at_least_one(cdiv(K, 2)) || lds < at_least_one(cdiv(K, group)))
        return MPGEMM_ELD;
    if (N == 0 || K == 0)
        return MPGEMM_OK;
    if (W == nullptr || Q == nullptr || scale == nullptr)
        return MPGEMM_ENULL;
    return !aligned(W, size_of(w_type)) || !aligned(scale, 2) ? MPGEMM_EALIGN : MPGEMM_OK;
}

}  // namespace

extern "C" {

int mpgemm_w4_quantize(int w_type, int s_type, int64_t N, int64_t K, int64_t group,
                       const void *W, int64_t ldw, uint8_t *Q, int64_t ldq,
                       void *scale, int64_t lds, void *stream)
{
    int64_t parts = 0;
    if (const int error = check_pack(w_type, s_type, N, K, group, W, ldw, Q, ldq, scale, lds,
                                     group > mpg::kPackSpan ? group : mpg::kPackSpan, parts))
        return error;
    if (N == 0 || K == 0)
        return MPGEMM_OK;
    const mpg::W4PackArgs a{W, Q, static_cast<uint16_t *>(scale), ldw, ldq, lds, (int32_t)N, (int32_t)K,
                            group_shift(group), (int32_t)parts};
    forget_error();
    if (w_type == MPGEMM_T_F16)
        launch_pack<mpg::kTF16>(s_type, a, stream_of(stream));
    else if (w_type == MPGEMM_T_BF16)
        launch_pack<mpg::kTBF16>(s_type, a, stream_of(stream));
    else
        launch_pack<mpg::kTF32>(s_type, a, stream_of(stream));
    return launched();
}

int mpgemm_w4_dequantize(int w_type, int s_type, int64_t N, int64_t K, int64_t group,
                         const uint8_t *Q, int64_t ldq, const void *scale, int64_t lds,
                         void *W, int64_t ldw, void *stream)
{
    int64_t parts = 0;
    if (const int error = check_pack(w_type, s_type, N, K, group, W, ldw, Q, ldq, scale, lds, 512, parts))
        return error;
    if (N == 0 || K == 0)
        return MPGEMM_OK;
    const mpg::W4UnpackArgs a{Q, static_cast<const uint16_t *>(scale), W, ldq, lds, ldw, (int32_t)N, (int32_t)K,
                              group_shift(group), (int32_t)parts};
    forget_error();
    if (w_type == MPGEMM_T_F16)
        launch_unpack<mpg::kTF16>(s_type, a, stream_of(stream));
    else if (w_type == MPGEMM_T_BF16)
        launch_unpack<mpg::kTBF16>(s_type, a, stream_of(stream));
    else
        launch_unpack<mpg::kTF32>(s_type, a, stream_of(stream));
    return launched();
}

int mpgemm_w4_gemm(int in_type, int out_type, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t group,
                   const uint16_t *A, int64_t lda, const uint8_t *Q, int64_t ldq, int64_t stride_q,
                   const void *scale, int64_t lds, int64_t stride_s, void *C, int64_t ldc,
                   const float *bias, const int32_t *offsets, void *stream)
{
    if ((in_type != MPGEMM_IN_F16 && in_type != MPGEMM_IN_BF16) || !is_type(out_type))
        return MPGEMM_ETYPE;
    if (const int error = check_w4(groups, M, N, K, group, lda, ldq, lds))
        return error;
    if (ldc < at_least_one(N) || stride_q < 0 || stride_s < 0)
        return MPGEMM_ELD;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    if (C == nullptr || (K > 0 && (A == nullptr || Q == nullptr || scale == nullptr)) ||
        (groups > 1 && offsets == nullptr))
        return MPGEMM_ENULL;
    if (!aligned(A, 2) || !aligned(scale, 2) || !aligned(C, size_of(out_type)) || !aligned(bias, 4) ||
        !aligned(offsets, 4))
        return MPGEMM_EALIGN;
    const Choice c = choose_w4(offsets ? groups : 0, M, N, K, lda);
    if (c.error)
        return c.error;
    W4Args a{};
    a.A = A;
    a.Q = Q;
    a.S = static_cast<const uint16_t *>(scale);
    a.C = C;
    a.bias = bias;
    a.lda = lda;
    a.ldq = ldq;
    a.lds = lds;
    a.ldc = ldc;
    a.stride_s = stride_s;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.shift = group_shift(group);
    a.out_type = out_type;
    a.tiles_n = (int32_t)c.tiles_n;
    a.group_m = 8;
    a.groups = mpg::GroupArgs{offsets, (int32_t)groups, (int32_t)M, stride_q};
    forget_error();
    const int gs = a.shift >= 7 ? mpg::kCoarse : a.shift == 6 ? mpg::kGroup64 : mpg::kGroup32;
    kTable[c.id].launch[in_type][gs](a, dim3((unsigned)c.grid), stream_of(stream));
    return launched();
}

int mpgemm_w4_query(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t group,
                    int64_t lda, int64_t ldq, int64_t lds, mpgemm_ops_kernel *out)
{
    if (const int error = check_w4(groups == 0 ? 1 : groups, M, N, K, group, lda, ldq, lds))
        return error;
    if (out == nullptr)
        return MPGEMM_ENULL;
    *out = mpgemm_ops_kernel{};
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    const Choice c = choose_w4(groups, M, N, K, lda);
    if (c.error)
        return c.error;
    const W4Entry &e = kTable[c.id];
    *out = mpgemm_ops_kernel{e.narrow, e.bm, e.bn, e.bk, e.stages, e.waves, c.grid};
    return MPGEMM_OK;
}

}  // extern "C"
