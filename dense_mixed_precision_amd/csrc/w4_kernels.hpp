// w4_kernels.hpp -- 4-bit weights with a scale per group of a row's values
// (gfx950): rows to codes and back, and products of 16-bit tokens with them.
// Included by w4.hip in kernels.hpp's namespace, after elements.hpp.
//
//     C[i][j] = sum_g S[j][g] * (sum_{k in g} A[i][k] * code[j][k]) (+ bias[j])
//
// A code (-8 .. 7) stands in its nibble as code + 8; value k of a row is the
// low nibble of byte k/2 where k is even, the high one where it is odd.
//
// The matrix instructions multiply the codes themselves, which 16-bit values
// hold exactly; each group's sum is FP32 and joins the running FP32 sum through
// one fused multiply-add with its scale.  So no weight is rounded, and the
// result is as near as the product of the weights in FP32.

struct W4Args {
    const uint16_t *A;
    const uint8_t *Q;
    const uint16_t *S;
    void *C;
    const float *bias;       // or nullptr
    int64_t lda, ldq, lds, ldc;   // elements (of Q: bytes)
    int64_t stride_s;        // elements from one group of rows' scales to the next
    int32_t N, K;
    int32_t shift;           // log2 of the values that share a scale
    int32_t out_type;        // kT*
    int32_t tiles_n;
    int32_t group_m;
    GroupArgs groups;        // (stride: bytes of Q)
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// Codes as 16-bit values times kCodeScale: bf16 ones come as sixteenths.
template <int IN>
constexpr float kCodeScale = IN == kInBF16 ? 16.0f : 1.0f;

// Eight codes of four bytes, in order.
//
// FP16: a pair of nibbles one byte apart is spread over the halves of a
// register; behind the leading bits of 1024 the low nibble q reads 1024 + q,
// behind those of 64 the high one (already shifted by 4) 64 + q.  One packed
// sum takes 1032 and 72 away, exactly.  12 instructions.
// BF16: the conversion of 4-bit integers (to sixteenths, in FP32) and the
// packing of two FP32 values, exactly.  14 instructions.
template <int IN>
__device__ __forceinline__ half8 codes8(uint32_t w)
{
    u32x4 out;
    if constexpr (IN == kInF16) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t x = __builtin_amdgcn_perm(0u, w, 0x0C000C00u | (uint32_t)(p << 16) | (uint32_t)p);
            x = (x & 0x00F0000Fu) | 0x54006400u;
            const half2v h = __builtin_bit_cast(half2v, x) + half2v{(_Float16)-1032.0f, (_Float16)-72.0f};
            out[p] = __builtin_bit_cast(uint32_t, h);
        }
    } else {
        w ^= 0x88888888u;
        uint32_t v = w >> 4;
        asm("" : "+v"(v));  // (so that the shifts below are byte selects)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x2 h;
            h[0] = (__bf16)__builtin_amdgcn_cvt_off_f32_i4((w >> (8 * p)) & 0xFFu);
            h[1] = (__bf16)__builtin_amdgcn_cvt_off_f32_i4((v >> (8 * p)) & 0xFFu);
            out[p] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return __builtin_bit_cast(half8, out);
}

template <int IN>
__device__ __forceinline__ float scale_value(uint32_t bits)
{
    if constexpr (IN == kInBF16)
        return __builtin_bit_cast(float, bits << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Groups of a row's values by the number that share a scale.  With 128 or more
// (COARSE) a lane's 32 consecutive codes go to four matrix instructions as they
// lie: instruction j takes values 32*kg + 8*j + 0..7 of a step of 128 from the
// lanes of part kg = lane / 16.  With fewer, an instruction's 32 values must lie
// in one group: the four registers of codes are transposed over the four parts,
// and instruction j takes 32*j + 8*kg + 0..7.
constexpr int kCoarse = 0, kGroup64 = 1, kGroup32 = 2;

template <int GS>
__device__ __forceinline__ u32x4 deal_codes(u32x4 w)
{
    if constexpr (GS != kCoarse) {
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        return u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
    }
    return w;
}

// Value (of a step of 128) that lane part kg's first slot of instruction j takes.
template <int GS>
__device__ __forceinline__ constexpr int slot_value(int j, int kg)
{
    return GS == kCoarse ? 32 * kg + 8 * j : 32 * j + 8 * kg;
}

// ---- 16 bytes of a row that may end inside them --------------------------------
// `left` bytes of the row remain at the place (of `len` in all, len >= 16): where
// it ends inside the 16, its last 16 bytes are loaded instead and shifted down,
// so that zeros stand behind it; behind the row zeros are read.
__device__ __forceinline__ uint32_t end_offset(uint32_t row, int at, int len)
{
    const int left = len - at;
    return row == kOOB || left <= 0 ? kOOB : row + (uint32_t)(left >= 16 ? at : len - 16);
}

__device__ __forceinline__ u32x4 end_shift(u32x4 v, int left)
{
    if (left <= 0 || left >= 16)
        return v;
    return __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, v) >> (8 * (16 - left)));
}

// The same of a row of fewer than 16 bytes, loaded ES bytes at a time.
template <int ES>
__device__ __forceinline__ u32x4 short_row(const __amdgpu_buffer_rsrc_t &rs, uint32_t row, int at, int len)
{
    unsigned __int128 v = 0;
    for (int e = 0; e < 16; e += ES) {
        const uint32_t off = row != kOOB && at + e < len ? row + at + e : kOOB;
        uint32_t x;
        if constexpr (ES == 1)
            x = __builtin_amdgcn_raw_buffer_load_b8(rs, off, 0, 0) & 0xFFu;
        else
            x = __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0) & 0xFFFFu;
        v |= (unsigned __int128)x << (8 * e);
    }
    return __builtin_bit_cast(u32x4, v);
}

// COUNT neighbouring values of a row of C, `left` of them within it.
template <int COUNT>
__device__ __forceinline__ void store_values(int type, void *C, int64_t at, int left, const float *v)
{
    if (type == kTF32)
        i8_store<kTF32, COUNT>((float *)C + at, 0, left, v);
    else if (type == kTF16)
        i8_store<kTF16, COUNT>((_Float16 *)C + at, 0, left, v);
    else
        i8_store<kTBF16, COUNT>((__bf16 *)C + at, 0, left, v);
}

// ---------------------------------------------------------------------------
// Few tokens: the weights straight from memory into operand registers
// ---------------------------------------------------------------------------
// A workgroup makes 16*MT tokens x 16*NF channels, its WAVES waves splitting K in
// steps of 128 values; a lane's 16 bytes of a weight row are 32 codes.  Tokens
// are the first operand, so a lane's accumulators are four tokens of one
// channel and one scale serves them; its NF channels are neighbours, stored
// together.  The waves' sums are added in LDS in wave order.
template <int IN, int GS, int MT, int NF, int WAVES, int DEPTH>
__global__ void __launch_bounds__(64 * WAVES)
w4_narrow(W4Args args)
{
    constexpr int NS = GS == kCoarse ? 1 : GS == kGroup64 ? 2 : 4;  // scales per step
    constexpr int PER = 4 / NS;                                     // instructions per scale
    __shared__ floatx4 part[WAVES][MT * NF][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupTile gt;
    if (!find_row_tile(args.groups, 16 * MT, args.tiles_n, args.group_m, gt))
        return;
    const int row0 = gt.start + gt.tm * 16 * MT;
    const int rows = min(gt.rows - gt.tm * 16 * MT, 16 * MT);
    const int n0 = gt.tn * 16 * NF;
    const int cols = args.N - n0;
    const int K = args.K, KB = (K + 1) / 2, KA = 2 * K;
    const int groups_k = (K + (1 << args.shift) - 1) >> args.shift;
    const int r = lane & 15, kg = lane >> 4;
    const __amdgpu_buffer_rsrc_t rsA = make_rsrc(args.A + (int64_t)row0 * args.lda);
    const __amdgpu_buffer_rsrc_t rsQ =
        make_rsrc(args.Q + (int64_t)gt.group * args.groups.stride + (int64_t)n0 * args.ldq);
    const __amdgpu_buffer_rsrc_t rsS = make_rsrc(args.S + (int64_t)gt.group * args.stride_s + (int64_t)n0 * args.lds);
    // 32-bit offsets of rows: the host checks that a tile's rows span less than 2 GiB
    uint32_t offA[MT], offQ[NF], offS[NF];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        offA[m] = 16 * m + r < rows ? (uint32_t)(2 * (16 * m + r) * (int)args.lda) : kOOB;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int c = NF * r + f;
        offQ[f] = c < cols ? (uint32_t)(c * (int)args.ldq) : kOOB;
        offS[f] = c < cols ? (uint32_t)(2 * c * (int)args.lds) : kOOB;
    }
    const int steps = (K + 127) / 128, full = K / 128;
    const int per = (steps + WAVES - 1) / WAVES;
    const int s0 = min(wave * per, steps), s1 = min(s0 + per, steps);

    u32x4 rq[DEPTH][NF], ra[DEPTH][MT][4];
    uint32_t rs[DEPTH][NF][NS];
    auto issue = [&](int d, int s) __attribute__((always_inline)) {
        if (s < full) {
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                rq[d][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsQ, offQ[f] + 16 * kg,
                                                                                           64 * s, 0));
                if constexpr (GS == kCoarse) {
                    rs[d][f][0] = __builtin_amdgcn_raw_buffer_load_b16(rsS, offS[f], 2 * (s >> (args.shift - 7)), 0);
                } else if constexpr (GS == kGroup64) {
                    const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(rsS, offS[f], 4 * s, 0);
                    rs[d][f][0] = x & 0xFFFFu;
                    rs[d][f][1] = x >> 16;
                } else {
                    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rsS, offS[f], 8 * s, 0));
                    rs[d][f][0] = x[0] & 0xFFFFu;
                    rs[d][f][1] = x[0] >> 16;
                    rs[d][f][2] = x[1] & 0xFFFFu;
                    rs[d][f][3] = x[1] >> 16;
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ra[d][m][j] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsA, offA[m] + 2 * slot_value<GS>(j, kg), 256 * s, 0));
            return;
        }
        // the step that K ends in
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int at = 64 * s + 16 * kg;
            if (KB >= 16)
                rq[d][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         rsQ, end_offset(offQ[f], at, KB), 0, 0));
            else
                rq[d][f] = short_row<1>(rsQ, offQ[f], at, KB);
#pragma unroll
            for (int g = 0; g < NS; ++g) {
                const int i = GS == kCoarse ? s >> (args.shift - 7) : NS * s + g;
                rs[d][f][g] = __builtin_amdgcn_raw_buffer_load_b16(
                    rsS, offS[f] != kOOB && i < groups_k ? offS[f] + 2 * i : kOOB, 0, 0);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 256 * s + 2 * slot_value<GS>(j, kg);
                if (KA >= 16)
                    ra[d][m][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                rsA, end_offset(offA[m], at, KA), 0, 0));
                else
                    ra[d][m][j] = short_row<2>(rsA, offA[m], at, KA);
            }
    };
    floatx4 acc[MT][NF];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](int d, int s) __attribute__((always_inline)) {
        if (s >= full) {
            if (KB >= 16)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    rq[d][f] = end_shift(rq[d][f], KB - (64 * s + 16 * kg));
            if (KA >= 16)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ra[d][m][j] = end_shift(ra[d][m][j], KA - (256 * s + 2 * slot_value<GS>(j, kg)));
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const u32x4 w = deal_codes<GS>(rq[d][f]);
            half8 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = codes8<IN>(w[j]);
#pragma unroll
            for (int g = 0; g < NS; ++g) {
                const float scale = scale_value<IN>(rs[d][f][g]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    floatx4 p = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = g * PER; j < (g + 1) * PER; ++j)
                        p = mfma16<IN>(__builtin_bit_cast(half8, ra[d][m][j]), b[j], p);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[m][f][v] = __builtin_fmaf(scale, p[v], acc[m][f][v]);
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (s0 + d < s1)
            issue(d, s0 + d);
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (s + d < s1) {
                multiply(d, s + d);
                if (s + d + DEPTH < s1)
                    issue(d, s + d + DEPTH);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            part[wave][m * NF + f][lane] = acc[m][f];
    __syncthreads();
    const int c = NF * r;
    const int left = cols - c;
    for (int m = wave; m < MT; m += WAVES) {
        floatx4 sum[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            sum[f] = part[0][m * NF + f][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                sum[f] += part[w][m * NF + f][lane];
        }
        if (left <= 0)
            continue;
        float bias[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            bias[f] = args.bias && f < left ? args.bias[(int64_t)gt.group * args.N + n0 + c + f] : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 16 * m + 4 * kg + v;
            if (row >= rows)
                continue;
            float out[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const float x = kCodeScale<IN> * sum[f][v];
                out[f] = args.bias ? x + bias[f] : x;
            }
            store_values<NF>(args.out_type, args.C, (int64_t)(row0 + row) * args.ldc + n0 + c, left, out);
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: token tiles through LDS
// ---------------------------------------------------------------------------
// A workgroup makes BM tokens x 16*NF*NW channels.  Its token tile (BM x 256
// values, K-contiguous) goes through two LDS buffers by direct copies; each
// wave has channels of its own, whose codes come straight into registers, two K
// tiles ahead, and are expanded once, one register of them beside each 16 tokens'
// matrix instructions.  Per step of 128 values and 16 tokens x 16 channels the
// group's sum is a chain of matrix instructions of its own, joined to the running
// sum by the scale.
// LDS: chunk c (16 bytes) of row r stands at c ^ (r % 16), so the 16 rows of
// an operand read touch all banks once.
template <int IN_, int GS_, int BM_, int NF_, int NW_>
struct W4Cfg {
    static constexpr int IN = IN_, GS = GS_, BM = BM_, NF = NF_, NW = NW_;
    static constexpr int BN = 16 * NF * NW, BK = 256, NT = 64 * NW;
    static constexpr int FM = BM / 16;
    static constexpr int ROW = 2 * BK;                  // bytes of a row of the tile
    static constexpr int BUF = BM * ROW;
    static constexpr int COPIES = BUF / 1024 / NW;      // per wave and tile
    static constexpr int NS = GS == kCoarse ? 1 : GS == kGroup64 ? 2 : 4;
    static constexpr int PER = 4 / NS;
    static constexpr int EXPAND = 4 * NF / FM;          // registers of codes per 16 tokens
    static_assert(COPIES >= 1 && BUF % (1024 * NW) == 0, "copies split evenly over waves");
    static_assert(EXPAND >= 1 && (4 * NF) % FM == 0, "codes are expanded evenly over the tokens");
    static_assert(2 * BUF <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT)
w4_tile(W4Args args)
{
    constexpr int IN = Cfg::IN, GS = Cfg::GS, BM = Cfg::BM, NF = Cfg::NF, NW = Cfg::NW, FM = Cfg::FM;
    constexpr int NS = Cfg::NS, PER = Cfg::PER;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * Cfg::BUF];
    lds_u8 *const lds = (lds_u8 *)smem;
    const uint32_t lds_base = (uint32_t)(uintptr_t)lds;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupTile gt;
    if (!find_row_tile(args.groups, BM, args.tiles_n, args.group_m, gt))
        return;
    const int row0 = gt.start + gt.tm * BM;
    const int rows = gt.rows - gt.tm * BM;               // > 0
    const int n0 = gt.tn * Cfg::BN + wave * 16 * NF;     // this wave's channels
    const int cols = args.N - n0;
    const int K = args.K, KB = (K + 1) / 2, KA = 2 * K;
    const int groups_k = (K + (1 << args.shift) - 1) >> args.shift;
    const int r = lane & 15, kg = lane >> 4;
    const uint16_t *const Ap = args.A + (int64_t)row0 * args.lda;
    const int num_k = (K + 255) / 256;

    // ---- token copies: copy q of this wave fills rows 2*(q*NW + wave), + 1
    const i32x4 rsA = make_rsrc4(Ap);
    uint32_t voff[Cfg::COPIES];
#pragma unroll
    for (int q = 0; q < Cfg::COPIES; ++q) {
        const int row = 2 * (q * NW + wave) + (lane >> 5);
        const int chunk = (lane & 31) ^ (row & 15);
        voff[q] = row < rows ? (uint32_t)(row * (int)args.lda * 2 + 16 * chunk) : kOOB;
    }
    auto copy_tokens = [&](int t) __attribute__((always_inline)) {
        const uint32_t region = lds_base + (t & 1) * Cfg::BUF;
        const int left = KA - 512 * t;                   // bytes of a row from this tile on
#pragma unroll
        for (int q = 0; q < Cfg::COPIES; ++q) {
            uint32_t off = voff[q];
            if (left < 512) {
                const int row = 2 * (q * NW + wave) + (lane >> 5);
                const int chunk = (lane & 31) ^ (row & 15);
                if (16 * chunk + 16 > left)
                    off = kOOB;
            }
            dma16(rsA, region + (q * NW + wave) * 1024, off, 512 * t);
        }
    };
    // The chunk that K ends inside, into the places where the copies wrote
    // zeros: one row per thread.
    auto fill_end = [&](int t) __attribute__((always_inline)) {
        const int left = KA - 512 * t;
        const int chunk = left / 16, bytes = left % 16;
        for (int row = threadIdx.x; row < BM && row < rows; row += Cfg::NT) {
            u32x4 v;
            const uint16_t *const a = Ap + (int64_t)row * args.lda;
            if (K >= 8) {
                v = end_shift(*(const u32x4_any *)(a + K - 8), bytes);
            } else {
                unsigned __int128 x = 0;
                for (int e = 0; e < K; ++e)
                    x |= (unsigned __int128)a[e] << (16 * e);
                v = __builtin_bit_cast(u32x4, x);
            }
            *(lds_u32x4 *)(lds + (t & 1) * Cfg::BUF + row * 512 + 16 * (chunk ^ (row & 15))) = v;
        }
    };

    // ---- codes and scales
    const bool works = cols > 0;
    const __amdgpu_buffer_rsrc_t rsQ =
        make_rsrc(args.Q + (int64_t)gt.group * args.groups.stride + (int64_t)(works ? n0 : 0) * args.ldq);
    const __amdgpu_buffer_rsrc_t rsS =
        make_rsrc(args.S + (int64_t)gt.group * args.stride_s + (int64_t)(works ? n0 : 0) * args.lds);
    uint32_t offQ[NF], offS[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int c = NF * r + f;
        offQ[f] = c < cols ? (uint32_t)(c * (int)args.ldq) : kOOB;
        offS[f] = c < cols ? (uint32_t)(2 * c * (int)args.lds) : kOOB;
    }
    u32x4 raw[2][2][NF];     // [tile % 2][step][channel]
    uint32_t scales[2][2][NF][NS];
    auto load_codes = [&](u32x4 (&to)[2][NF], int t) __attribute__((always_inline)) {
        const bool whole = 256 * t + 256 <= K;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int at = 128 * t + 64 * h + 16 * kg;
                if (whole)
                    to[h][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             rsQ, offQ[f] + 64 * h + 16 * kg, 128 * t, 0));
                else if (KB >= 16)
                    to[h][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             rsQ, end_offset(offQ[f], at, KB), 0, 0));
                else
                    to[h][f] = short_row<1>(rsQ, offQ[f], at, KB);
            }
    };
    // (only a row's end is shifted, and tiles behind K have none)
    auto end_codes = [&](u32x4 (&to)[2][NF], int t) __attribute__((always_inline)) {
        if (256 * t + 256 <= K || KB < 16)
            return;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                to[h][f] = end_shift(to[h][f], KB - (128 * t + 64 * h + 16 * kg));
    };
    auto load_scales = [&](uint32_t (&to)[2][NF][NS], int t) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int g = 0; g < NS; ++g) {
                    const int i = GS == kCoarse ? (2 * t + h) >> (args.shift - 7) : NS * (2 * t + h) + g;
                    to[h][f][g] = __builtin_amdgcn_raw_buffer_load_b16(
                        rsS, offS[f] != kOOB && i < groups_k ? offS[f] + 2 * i : kOOB, 0, 0);
                }
    };

    floatx4 acc[FM][NF];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[i][f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    half8 code[2][NF][4];    // [step % 2][channel][instruction]
    u32x4 dealt[NF];         // the next step's codes, before they are expanded
    auto expand = [&](int set, int n) __attribute__((always_inline)) {
        code[set][n / 4][n % 4] = codes8<IN>(dealt[n / 4][n % 4]);
    };

    if (num_k > 0) {
        copy_tokens(0);
        if (works) {
            load_codes(raw[0], 0);
            load_codes(raw[1], 1);
            load_scales(scales[0], 0);
            end_codes(raw[0], 0);
#pragma unroll
            for (int f = 0; f < NF; ++f)
                dealt[f] = deal_codes<GS>(raw[0][0][f]);
#pragma unroll
            for (int n = 0; n < 4 * NF; ++n)
                expand(0, n);
        }
    }
    // One K tile, P = t % 2 (so that registers are named at compile time).
    auto tile = [&](int t, auto parity) __attribute__((always_inline)) {
        constexpr int P = decltype(parity)::value;
        wait_vmcnt<0>();
        if (t == num_k - 1 && (KA & 15) != 0)
            fill_end(t);
        __syncthreads();
        if (t + 1 < num_k)
            copy_tokens(t + 1);
        if (!works)
            return;
        // what landed before the barrier is taken here, so that no wait for it
        // comes behind the loads below
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                asm volatile("" : "+v"(raw[0][h][f]), "+v"(raw[1][h][f]));
#pragma unroll
                for (int g = 0; g < NS; ++g)
                    asm volatile("" : "+v"(scales[P][h][f][g]));
            }
        end_codes(raw[P ^ 1], t + 1);
        const u32x4 *const second = raw[P][1];
        u32x4 later[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            later[f] = second[f];
        load_scales(scales[P ^ 1], t + 1);
        u32x4 fresh[2][NF];
        load_codes(fresh, t + 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float s[NF][NS];
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int g = 0; g < NS; ++g)
                    s[f][g] = scale_value<IN>(scales[P][h][f][g]);
#pragma unroll
            for (int f = 0; f < NF; ++f)
                dealt[f] = deal_codes<GS>(h == 0 ? later[f] : raw[P ^ 1][0][f]);
            half8 a[2][4];
            auto read = [&](int set, int i) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int chunk = (16 * h + slot_value<GS>(j, kg) / 8) ^ r;
                    a[set][j] = *(const __attribute__((address_space(3))) half8 *)(lds + P * Cfg::BUF +
                                                                                   (16 * i + r) * 512 + 16 * chunk);
                }
            };
            read(0, 0);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (i + 1 < FM)
                    read((i + 1) & 1, i + 1);
                floatx4 p[NF][NS];
#pragma unroll
                for (int g = 0; g < NS; ++g)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        p[f][g] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        p[f][j / PER] = mfma16<IN>(a[i & 1][j], code[h][f][j], p[f][j / PER]);
#pragma unroll
                for (int e = 0; e < Cfg::EXPAND; ++e)
                    expand(h ^ 1, i * Cfg::EXPAND + e);
#pragma unroll
                for (int g = 0; g < NS; ++g)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            acc[i][f][v] = __builtin_fmaf(s[f][g], p[f][g][v], acc[i][f][v]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                raw[P][h][f] = fresh[h][f];
    };
    for (int t = 0; t < num_k; t += 2) {
        tile(t, std::integral_constant<int, 0>{});
        if (t + 1 < num_k)
            tile(t + 1, std::integral_constant<int, 1>{});
    }
    if (!works)
        return;
    const int c = NF * r;
    const int left = cols - c;
    if (left <= 0)
        return;
    float bias[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
        bias[f] = args.bias && f < left ? args.bias[(int64_t)gt.group * args.N + n0 + c + f] : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 16 * i + 4 * kg + v;
            if (row >= rows)
                continue;
            float out[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const float x = kCodeScale<IN> * acc[i][f][v];
                out[f] = args.bias ? x + bias[f] : x;
            }
            store_values<NF>(args.out_type, args.C, (int64_t)(row0 + row) * args.ldc + n0 + c, left, out);
        }
}

// ---------------------------------------------------------------------------
// Rows to codes and back
// ---------------------------------------------------------------------------
struct W4PackArgs {
    const void *W;           // N x K
    uint8_t *Q;
    uint16_t *S;
    int64_t ldw, ldq, lds;
    int32_t N, K;
    int32_t shift;
    int32_t parts;           // waves per row
};

// A group's scale and codes.  With m the largest magnitude, s is m/7 rounded to
// FP32 and then to the scale's type; a value's code is the whole number of
// -8 .. 7 nearest to w/s, the even one in the middle, decided exactly: both are
// scaled by the power of two that brings s to [0.5, 1), q = rint(w * (1/s)) is
// off by one at most, and the remainder w - q*s (one fused multiply-add, exact
// near the middle of two codes: q*s has at most 15 bits, and what is left is a
// multiple of 2^-25 below 1) against s/2 says which way.  A group with an
// infinity or a NaN, or whose scale its type does not hold, has a NaN scale
// and codes 0.
template <int ST>
struct W4Scale {
    float s, half, inv;
    int ex;
    bool live;
    uint16_t bits;
    __device__ __forceinline__ explicit W4Scale(uint32_t top)
    {
        typedef typename ElemOf<ST>::type E;
        const float most = __builtin_bit_cast(float, top);
        E e = (E)(most / 7.0f);
        float v = (float)e;
        if (top >= 0x7F800000u || __builtin_bit_cast(uint32_t, v) >= 0x7F800000u) {
            e = (E)__builtin_nanf("");
            v = 0.0f;
        }
        bits = __builtin_bit_cast(uint16_t, e);
        live = v > 0.0f;
        ex = live ? __builtin_amdgcn_frexp_expf(v) : 0;
        s = live ? __builtin_amdgcn_ldexpf(v, -ex) : 1.0f;
        half = 0.5f * s;
        inv = 1.0f / s;
    }
    __device__ __forceinline__ uint32_t nibble(float w) const
    {
        const float x = __builtin_amdgcn_ldexpf(w, -ex);
        float q = __builtin_rintf(x * inv);
        const float rest = __builtin_fmaf(-q, s, x);
        const bool odd = ((int)q & 1) != 0;
        if (rest > half || (rest == half && odd))
            q += 1.0f;
        else if (rest < -half || (rest == -half && odd))
            q -= 1.0f;
        q = q < -8.0f ? -8.0f : q > 7.0f ? 7.0f : q;
        return live ? (uint32_t)((int)q + 8) : 8u;
    }
};

__device__ __forceinline__ uint32_t magnitude(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; }

// Eight values of a row from k on, zeros behind it.
template <class E>
__device__ __forceinline__ void load_values(const E *w, int64_t k, int64_t K, float (&v)[8])
{
    if (k + 8 <= K) {
        const Pack<E, 8> p = *(const Pack<E, 8> *)(w + k);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = (float)p.v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = k + e < K ? (float)w[k + e] : 0.0f;
    }
}

// A lane has 8 neighbouring values, a wave 512 of a row.  Groups of up to 512
// values are the lanes of one wave; of larger ones a wave has one, read twice.
template <int WT, int ST>
__global__ void __launch_bounds__(256)
w4_pack(W4PackArgs args)
{
    typedef typename ElemOf<WT>::type E;
    const int lane = threadIdx.x & 63;
    const uint32_t unit = (uint32_t)wg_number() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = unit / (uint32_t)args.parts;
    if (row >= args.N)
        return;
    const int64_t K = args.K, size = (int64_t)1 << args.shift;
    const int64_t span = size > 512 ? size : 512;
    const int64_t first = (unit - row * args.parts) * span, end = first + span < K ? first + span : K;
    const E *const w = (const E *)args.W + row * args.ldw;
    float v[8];
    uint32_t top = 0;
    for (int64_t k = first + 8 * lane; k < end; k += 512) {
        load_values(w, k, K, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, magnitude(v[e]));
    }
    const int lanes = args.shift >= 9 ? 64 : 1 << (args.shift - 3);
    for (int d = 1; d < lanes; d *= 2)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const W4Scale<ST> scale(top);
    const int64_t at = first + 8 * lane;
    if ((lane & (lanes - 1)) == 0 && at < end)
        args.S[row * args.lds + (at >> args.shift)] = scale.bits;
    uint8_t *const q = args.Q + row * args.ldq;
    for (int64_t k = at; k < end; k += 512) {
        if (size > 512)
            load_values(w, k, K, v);
        Pack<uint8_t, 4> o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o.v[e] = (uint8_t)(scale.nibble(v[2 * e]) | scale.nibble(v[2 * e + 1]) << 4);
        if (k + 8 <= K) {
            *(Pack<uint8_t, 4> *)(q + k / 2) = o;
        } else {
            // (a value behind the row is 0, so the spare nibble is 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + 2 * e < K)
                    q[k / 2 + e] = o.v[e];
        }
    }
}

struct W4UnpackArgs {
    const uint8_t *Q;
    const uint16_t *S;
    void *W;
    int64_t ldq, lds, ldw;
    int32_t N, K;
    int32_t shift;
    int32_t parts;           // waves per row, of 512 values each
};

template <int ST, int WT>
__global__ void __launch_bounds__(256)
w4_unpack(W4UnpackArgs args)
{
    typedef typename ElemOf<WT>::type E;
    const int lane = threadIdx.x & 63;
    const uint32_t unit = (uint32_t)wg_number() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = unit / (uint32_t)args.parts;
    if (row >= args.N)
        return;
    const int64_t K = args.K, k = (unit - row * args.parts) * 512 + 8 * lane;
    if (k >= K)
        return;
    const uint8_t *const q = args.Q + row * args.ldq + k / 2;
    const float s = scale_value<ST == kTBF16 ? kInBF16 : kInF16>(args.S[row * args.lds + (k >> args.shift)]);
    E *const w = (E *)args.W + row * args.ldw + k;
    if (k + 8 <= K) {
        const Pack<uint8_t, 4> b = *(const Pack<uint8_t, 4> *)q;
        Pack<E, 8> o;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o.v[e] = (E)((float)((int)(b.v[e / 2] >> (4 * (e & 1)) & 15) - 8) * s);
        *(Pack<E, 8> *)w = o;
    } else {
        for (int e = 0; k + e < K; ++e)
            w[e] = (E)((float)((int)(q[e / 2] >> (4 * (e & 1)) & 15) - 8) * s);
    }
}
