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
        uint32_t mask = 0x00F0000Fu;
        asm("" : "+v"(mask));  // (in a register, for one instruction of and and or)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t x = __builtin_amdgcn_perm(0u, w, 0x0C000C00u | (uint32_t)(p << 16) | (uint32_t)p);
            x = (x & mask) | 0x54006400u;
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

// Groups of a row's values by the number that share a scale: 128 or more, 64, 32.
constexpr int kCoarse = 0, kGroup64 = 1, kGroup32 = 2;

// A lane's 16 bytes are 32 consecutive codes of its row, part kg = lane / 16 of a
// step of 128.  A matrix instruction's 32 values shall lie in one group, and 8 of
// them in each part's tokens side by side: the four registers of codes are
// transposed over the four parts, and instruction j takes the values 32*j +
// 8*kg + 0..7.
__device__ __forceinline__ u32x4 deal_codes(u32x4 w)
{
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// Rows in LDS.  An operand read takes four turns, of lanes 0-3, 12-15, 20-27 and
// so on: rows 0-3 and 12-15 of one part with rows 4-11 of the next.  Chunk c of a
// row of tokens (16 of them) stands at c ^ (r % 16), and piece p of a row of codes
// (four of them) at p ^ -(r / 4): the 16 lanes of a turn then have 16 different
// places of 16 bytes in the banks' 256.  Kernels of 4 or 8 tokens, whose operand
// rows repeat, miss that for tokens: the two parts of a turn meet at 4 or 8 places,
// in other rows (conflict cycles of those that read LDS: 39% at 4x16, 34% and 25%
// at 8x32 with 8 and 4 waves; none with 16 tokens or more).
__device__ __forceinline__ int piece_place(int p, int r) { return p ^ (-(r >> 2) & 3); }

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
// Few tokens: each wave streams its part of K through LDS of its own
// ---------------------------------------------------------------------------
// A workgroup makes up to 4*NA tokens (MT operands of 16) x 16*NF channels, its
// WAVES waves splitting K in steps of 128 values.  Tokens are the matrix
// instruction's first operand, so a lane's accumulators are four tokens of one
// channel and one scale serves them; its NF channels are neighbours, stored
// together.  The waves' sums are added in LDS in wave order.
//
// An operand's lane l holds row l % 16, so loaded straight into registers every
// four neighbouring lanes would ask for four cache lines, one after the other
// (measured: 42 cycles an instruction, 15.4 us for 8x8192x8192 whatever is kept
// in flight).  So a step's rows go to LDS by direct copies whose neighbouring
// lanes copy neighbouring bytes, STAGES steps ahead, and are read from there:
//   codes   channels NF*r + f together, 64 bytes each
//   tokens  256 bytes a row
//   scales  the 4-byte words of each channel that hold the step's
// (in the places of piece_place).  A wave waits for its own copies only; there is
// no barrier before the sums.  Every step issues the same copies, those behind the
// wave's last from empty buffers, so that one count waits for all of them, and the
// loop has one copy of its body: the instructions of a launch come from memory
// once more, about 0.1 us for 128 bytes of them, which a call of few microseconds
// notices.
//
// Bound: for few tokens the codes' way from memory and the vector work, half of it
// their expansion (8x8192x8192 FP16 11.3-12.1 us, 2.9 TB/s of codes, vector units
// busy 48% of the time a compute unit holds waves; 64 BF16 rows over 64 experts of
// 2048x2048, of which they reach about 41, 25.5-27 us, 75%); for 32 to 64 the
// tokens, which every compute unit reads whole (64x8192x8192 24.6-25.6 us: 1 MiB of
// tokens and 128 KiB of codes a workgroup); for one small product the launch
// (1x4096x4096 5.2-6.0).  With 4 waves the compiler keeps the matrix instructions'
// sums in accumulation registers: a move a value before each joining (4 waves here
// and in w4_tile; none with 8).
template <int IN, int GS, int NA, int NF, int WAVES, int STAGES>
__global__ void __launch_bounds__(64 * WAVES)
w4_narrow(W4Args args)
{
    constexpr int MT = (NA + 3) / 4;                                // operands of 16 tokens
    constexpr int NS = GS == kCoarse ? 1 : GS == kGroup64 ? 2 : 4;  // scales per step
    constexpr int PER = 4 / NS;                                     // instructions per scale
    constexpr int CH = 16 * NF;                                     // channels
    constexpr int WORDS = NS / 2 + 1;                               // 4-byte words that NS scales may touch
    constexpr int COPY_S = (WORDS * CH + 63) / 64;
    constexpr int COPIES = NF + NA + COPY_S;
    constexpr int AT_A = 1024 * NF, AT_S = AT_A + 1024 * NA;
    constexpr int SLOT = AT_S + 256 * COPY_S;
    constexpr int RING = STAGES * SLOT > 1024 * MT * NF ? STAGES * SLOT : 1024 * MT * NF;
    static_assert(NA < 4 ? 4 % NA == 0 : NA % 4 == 0, "whole operands, or an even part of one");
    static_assert(COPIES * (STAGES - 1) < 64, "vmcnt is 6 bits");
    static_assert(WAVES * RING <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * RING];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lds_u8 *const lds = (lds_u8 *)smem + wave * RING;
    const uint32_t lds_base = (uint32_t)(uintptr_t)lds;
    GroupTile gt;
    if (!find_row_tile(args.groups, 4 * NA, args.tiles_n, args.group_m, gt))
        return;
    const int row0 = gt.start + gt.tm * 4 * NA;
    const int rows = min(gt.rows - gt.tm * 4 * NA, 4 * NA);
    const int n0 = gt.tn * CH;
    const int cols = args.N - n0;
    const int K = args.K, KB = (K + 1) / 2, KA = 2 * K;
    const int groups_k = (K + (1 << args.shift) - 1) >> args.shift;
    const int r = lane & 15, kg = lane >> 4;
    const uint16_t *const Ap = args.A + (int64_t)row0 * args.lda;
    const uint8_t *const Qp = args.Q + (int64_t)gt.group * args.groups.stride + (int64_t)n0 * args.ldq;
    const uint16_t *const Sp = args.S + (int64_t)gt.group * args.stride_s + (int64_t)n0 * args.lds;
    const int odd = (int)(reinterpret_cast<uintptr_t>(Sp) >> 1 & 1);  // Sp lies in the middle of a word
    const int steps = (K + 127) / 128, full = K / 128;
    const int per = (steps + WAVES - 1) / WAVES;
    const int s0 = min(wave * per, steps), s1 = min(s0 + per, steps);

    // ---- copies
    // 32-bit offsets of rows: the host checks that a tile's rows span less than 2 GiB
    const int rowQ = lane >> 2, pieceQ = piece_place(lane & 3, lane >> 2);
    const int rowA = lane >> 4;
    uint32_t offQ[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
        offQ[f] = NF * rowQ + f < cols ? (uint32_t)((NF * rowQ + f) * (int)args.ldq) : kOOB;
    i32x4 rsA = make_rsrc4(Ap), rsQ = make_rsrc4(Qp), rsS = make_rsrc4(Sp - odd);
    auto issue = [&](int s) __attribute__((always_inline)) {
        const uint32_t to = lds_base + (s - s0) % STAGES * SLOT;
        rsA[2] = rsQ[2] = rsS[2] = s < s1 ? kNumRecords : 0;
        const bool end = s == full;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint32_t off = offQ[f] + 16 * pieceQ;
            dma16(rsQ, to + 1024 * f, end ? end_offset(offQ[f], 64 * s + 16 * pieceQ, KB) : off, end ? 0 : 64 * s);
        }
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            const int row = 4 * q + rowA, chunk = (lane & 15) ^ (row & 15);
            const uint32_t off = row < rows ? (uint32_t)(2 * row * (int)args.lda) : kOOB;
            dma16(rsA, to + AT_A + 1024 * q, end ? end_offset(off, 256 * s + 16 * chunk, KA) : off + 16 * chunk,
                  end ? 0 : 256 * s);
        }
#pragma unroll
        for (int q = 0; q < COPY_S; ++q) {
            const int c = (64 * q + lane) % CH, word = (64 * q + lane) / CH;
            const int first = GS == kCoarse ? s >> (args.shift - 7) : NS * s;
            const int i = odd + c * (int)args.lds + first;   // in 16-bit values from the aligned base
            const bool ok = c < cols && word < WORDS && 2 * (i / 2 + word) < i + min(NS, groups_k - first);
            dma4(rsS, to + AT_S + 256 * q, ok ? (uint32_t)(4 * (i / 2 + word)) : kOOB);
        }
    };

    floatx4 acc[MT][NF];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const u32x4 (&rq)[NF], const u32x4 (&ra)[MT][4], const float (&scale)[NF][NS])
        __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const u32x4 w = deal_codes(rq[f]);
            half8 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = codes8<IN>(w[j]);
#pragma unroll
            for (int g = 0; g < NS; ++g)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    floatx4 p = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = g * PER; j < (g + 1) * PER; ++j)
                        p = mfma16<IN>(__builtin_bit_cast(half8, ra[m][j]), b[j], p);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[m][f][v] = __builtin_fmaf(scale[f][g], p[v], acc[m][f][v]);
                }
        }
    };
    u32x4 rq[NF], ra[MT][4];
    float scale[NF][NS];
    if (full > 0) {
        for (int d = 0; d < STAGES - 1; ++d)
            issue(s0 + d);
        for (int s = s0; s < s1; ++s) {
            // (what was read from the slot that is filled now has arrived)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(s + STAGES - 1);
            wait_vmcnt<COPIES * (STAGES - 1)>();
            const lds_u8 *const from = lds + (s - s0) % STAGES * SLOT;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int c = NF * r + f;
                rq[f] = *(const lds_u32x4 *)(from + 1024 * f + 64 * r + 16 * piece_place(kg, r));
                const int i = odd + c * (int)args.lds + (GS == kCoarse ? s >> (args.shift - 7) : 0);
#pragma unroll
                for (int g = 0; g < NS; ++g) {
                    const int at = (i & 1) + g;
                    const uint32_t x = *(const __attribute__((address_space(3))) uint16_t *)(
                        from + AT_S + 4 * ((at >> 1) * CH + c) + 2 * (at & 1));
                    scale[f][g] = scale_value<IN>(x);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (operand rows without a token repeat those of the others)
                    const int row = NA < 4 ? r % (4 * NA) : 16 * m + r;
                    ra[m][j] = *(const lds_u32x4 *)(from + AT_A + 256 * row +
                                                    16 * ((4 * j + kg) ^ (row & 15)));
                }
            if (s == full) {
                // K ends in this step
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    rq[f] = end_shift(rq[f], KB - (64 * s + 16 * kg));
                    if constexpr (NS > 1)
#pragma unroll
                        for (int g = 0; g < NS; ++g)
                            scale[f][g] = NS * s + g < groups_k ? scale[f][g] : 0.0f;
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ra[m][j] = end_shift(ra[m][j], KA - (256 * s + 2 * (32 * j + 8 * kg)));
            }
            multiply(rq, ra, scale);
        }
    } else if (s0 < s1) {
        // K < 128: the only step, by single values
        const __amdgpu_buffer_rsrc_t bA = make_rsrc(Ap), bQ = make_rsrc(Qp), bS = make_rsrc(Sp);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int c = NF * r + f;
            rq[f] = short_row<1>(bQ, c < cols ? (uint32_t)(c * (int)args.ldq) : kOOB, 16 * kg, KB);
#pragma unroll
            for (int g = 0; g < NS; ++g)
                scale[f][g] = scale_value<IN>(__builtin_amdgcn_raw_buffer_load_b16(
                    bS, c < cols && g < groups_k ? (uint32_t)(2 * (c * (int)args.lds + g)) : kOOB, 0, 0) & 0xFFFFu);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ra[m][j] = short_row<2>(bA, 16 * m + r < rows ? (uint32_t)(2 * (16 * m + r) * (int)args.lda) : kOOB,
                                        2 * (32 * j + 8 * kg), KA);
        multiply(rq, ra, scale);
    }
    wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    typedef __attribute__((address_space(3))) floatx4 lds_f32x4;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            *(lds_f32x4 *)(lds + 1024 * (m * NF + f) + 16 * lane) = acc[m][f];
    __syncthreads();
    const int c = NF * r;
    const int left = cols - c;
    for (int m = wave; m < MT; m += WAVES) {
        floatx4 sum[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            sum[f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int w = 0; w < WAVES; ++w)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                sum[f] += *(const lds_f32x4 *)((lds_u8 *)smem + w * RING + 1024 * (m * NF + f) + 16 * lane);
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
// Many tokens: token tiles shared by the waves
// ---------------------------------------------------------------------------
// A workgroup makes BM tokens x 16*NF*NW channels in steps of 128 values of K.
// All waves read the tokens of a step from LDS; each has channels of its own,
// whose codes it expands once, in registers, one step ahead and between the
// matrix instructions of the step before (an expansion into LDS would be read
// by no one else and cost the LDS as much again).  Per step and 16 x 16 outputs
// the sum of a group is a chain of matrix instructions of its own, joined to the
// running sum by the scale.
// Tokens, codes and scales come by direct copies, laid out as in w4_narrow, into
// three slots each.  Before its last 16 tokens' instructions, whose operands are
// in registers, a step publishes the next: it waits for that one's tokens and
// scales and the codes of the one behind it (a later batch stays in flight),
// passes the barrier, and goes on with the next step's first reads underway; that
// one issues the batch that takes the slots it freed, a few copies after each 16
// tokens.  The sums of 16 tokens join the running ones beside the next 16 tokens'
// instructions.
//
// Bound: the matrix cores at the board's power limit, with the vector work that
// goes beside them: 8192^3 BF16 1.06 ms, 1.04e15 operations/s (a 16-bit library
// product 0.83), matrix pipes busy 48% at 2.1 GHz, vector instructions issued in
// 58% of the cycles.  Timed with parts left out: without the joining of sums
// 0.99 ms, without the expansion of codes no less, copies, barriers and matrix
// instructions alone 0.78.  Copies issued all at once instead of a few after each
// 16 tokens cost 5%, registers spilt by sums that the compiler moves down a
// quarter (see join).
template <int IN_, int GS_, int BM_, int NF_, int NW_>
struct W4Cfg {
    static constexpr int IN = IN_, GS = GS_, BM = BM_, NF = NF_, NW = NW_;
    static constexpr int BN = 16 * NF * NW, BK = 128, STAGES = 3, NT = 64 * NW;
    static constexpr int FM = BM / 16;
    static constexpr int NS = GS == kCoarse ? 1 : GS == kGroup64 ? 2 : 4;  // scales per step
    static constexpr int PER = 4 / NS;                                     // instructions per scale
    static constexpr int CH = 16 * NF;                                     // channels of a wave
    static constexpr int WORDS = NS / 2 + 1;                               // 4-byte words that NS scales may touch
    static constexpr int COPY_A = BM / 4 / NW, COPY_S = (WORDS * CH + 63) / 64;
    static constexpr int COPIES = COPY_A + NF + COPY_S;                    // of a wave and step
    static constexpr int BUF_A = 256 * BM, BUF_Q = 1024 * NF, BUF_S = 256 * COPY_S;  // (Q and S: of a wave)
    static constexpr int AT_Q = STAGES * BUF_A, AT_S = AT_Q + STAGES * NW * BUF_Q;
    static constexpr int LDS_BYTES = AT_S + STAGES * NW * BUF_S;
    static constexpr int EXPAND = (4 * NF + FM - 1) / FM;                  // registers of codes per 16 tokens
    static_assert(BM % (4 * NW) == 0, "copies split evenly over waves");
    static_assert(COPIES * 2 < 64, "vmcnt is 6 bits");
    static_assert(LDS_BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT)
w4_tile(W4Args args)
{
    constexpr int IN = Cfg::IN, GS = Cfg::GS, BM = Cfg::BM, NF = Cfg::NF, NW = Cfg::NW, FM = Cfg::FM;
    constexpr int NS = Cfg::NS, PER = Cfg::PER, CH = Cfg::CH, STAGES = Cfg::STAGES;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES];
    lds_u8 *const lds = (lds_u8 *)smem;
    const uint32_t lds_base = (uint32_t)(uintptr_t)lds;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupTile gt;
    if (!find_row_tile(args.groups, BM, args.tiles_n, args.group_m, gt))
        return;
    const int row0 = gt.start + gt.tm * BM;
    const int rows = gt.rows - gt.tm * BM;               // > 0
    const int n0 = gt.tn * Cfg::BN + wave * CH;          // this wave's channels
    const int cols = args.N - n0;                        // (none: it only copies)
    const int K = args.K, KB = (K + 1) / 2, KA = 2 * K;
    const int groups_k = (K + (1 << args.shift) - 1) >> args.shift;
    const int r = lane & 15, kg = lane >> 4;
    const uint16_t *const Ap = args.A + (int64_t)row0 * args.lda;
    const int64_t first = cols > 0 ? n0 : 0;
    const uint8_t *const Qp = args.Q + (int64_t)gt.group * args.groups.stride + first * args.ldq;
    const uint16_t *const Sp = args.S + (int64_t)gt.group * args.stride_s + first * args.lds;
    const int odd = (int)(reinterpret_cast<uintptr_t>(Sp) >> 1 & 1);  // Sp lies in the middle of a word
    const int steps = (K + 127) / 128, full = K / 128;

    // ---- copies, as in w4_narrow
    const int pieceQ = piece_place(lane & 3, lane >> 2), rowA = lane >> 4;
    uint32_t offA[Cfg::COPY_A], offQ[NF];
#pragma unroll
    for (int q = 0; q < Cfg::COPY_A; ++q) {
        const int row = 4 * (q * NW + wave) + rowA;
        const int chunk = (lane & 15) ^ (row & 15);
        offA[q] = row < rows ? (uint32_t)(2 * row * (int)args.lda + 16 * chunk) : kOOB;
    }
    int firstS[Cfg::COPY_S];
    bool okS[Cfg::COPY_S];
#pragma unroll
    for (int q = 0; q < Cfg::COPY_S; ++q) {
        const int c = (64 * q + lane) % CH;
        firstS[q] = odd + c * (int)args.lds;
        okS[q] = c < cols && (64 * q + lane) / CH < Cfg::WORDS;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int c = NF * (lane >> 2) + f;
        offQ[f] = c < cols ? (uint32_t)(c * (int)args.ldq) : kOOB;
    }
    i32x4 rsA = make_rsrc4(Ap), rsQ = make_rsrc4(Qp), rsS = make_rsrc4(Sp - odd);
    // Copy q of batch s: tokens and scales of step s into slot `slot`, codes of
    // step s + 1 into the next.
    auto next_slot = [](int slot) __attribute__((always_inline)) { return slot + 1 == STAGES ? 0 : slot + 1; };
    auto copy_codes = [&](int s, int slot, int f) __attribute__((always_inline)) {
        rsQ[2] = s < steps ? kNumRecords : 0;
        const bool end = s == full;
        const uint32_t off = end ? end_offset(offQ[f], 64 * full + 16 * pieceQ, KB) : offQ[f] + 16 * pieceQ;
        dma16(rsQ, lds_base + Cfg::AT_Q + (slot * NW + wave) * Cfg::BUF_Q + 1024 * f, off, end ? 0 : 64 * s);
    };
    auto copy_one = [&](int s, int slot, int q) __attribute__((always_inline)) {
        if (q < Cfg::COPY_A) {
            rsA[2] = s < steps ? kNumRecords : 0;
            // (the chunk that K ends inside is filled by fill_end)
            const int chunk = (lane & 15) ^ ((4 * (q * NW + wave) + rowA) & 15);
            const int left = s == full ? KA - 256 * full : 256;
            dma16(rsA, lds_base + slot * Cfg::BUF_A + 1024 * (NW * q + wave), 16 * chunk + 16 > left ? kOOB : offA[q],
                  256 * s);
        } else if (q < Cfg::COPY_A + Cfg::COPY_S) {
            q -= Cfg::COPY_A;
            rsS[2] = s < steps ? kNumRecords : 0;
            const int word = (64 * q + lane) / CH;
            const int g = GS == kCoarse ? s >> (args.shift - 7) : NS * s;
            const int i = firstS[q] + g;                 // in 16-bit values from the aligned base
            const bool ok = (i & ~1) + 2 * word < i + min(NS, groups_k - g);
            dma4(rsS, lds_base + Cfg::AT_S + (slot * NW + wave) * Cfg::BUF_S + 256 * q,
                 okS[q] && ok ? (uint32_t)(2 * (i & ~1) + 4 * word) : kOOB);
        } else {
            copy_codes(s + 1, next_slot(slot), q - Cfg::COPY_A - Cfg::COPY_S);
        }
    };
    auto copy_batch = [&](int s, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < Cfg::COPIES; ++q)
            copy_one(s, slot, q);
    };
    // The chunk that K ends inside, into the places where this wave's own
    // copies wrote zeros.
    auto fill_end = [&](int slot) __attribute__((always_inline)) {
        const int left = KA - 256 * full, chunk = left / 16;
#pragma unroll
        for (int q = 0; q < Cfg::COPY_A; ++q) {
            const int row = 4 * (q * NW + wave) + rowA;
            if ((lane & 15) == 0 && row < rows) {
                const u32x4 v = *(const u32x4_any *)(Ap + (int64_t)row * args.lda + K - 8);
                *(lds_u32x4 *)(lds + slot * Cfg::BUF_A + 256 * row + 16 * (chunk ^ (row & 15))) = end_shift(v, left % 16);
            }
        }
    };

    floatx4 acc[FM][NF];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[i][f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    half8 code[2][NF][4];    // [step % 2][channel][instruction]
    u32x4 raw[NF];           // the next step's, before they are expanded
    auto read_codes = [&](int s, int slot) __attribute__((always_inline)) {
        const lds_u8 *const from = lds + Cfg::AT_Q + (slot * NW + wave) * Cfg::BUF_Q + 64 * r + 16 * piece_place(kg, r);
#pragma unroll
        for (int f = 0; f < NF; ++f)
            raw[f] = *(const lds_u32x4 *)(from + 1024 * f);
        if (s == full)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                raw[f] = end_shift(raw[f], KB - (64 * s + 16 * kg));
    };
    auto expand = [&](int set, int n) __attribute__((always_inline)) {
        if (n < 4 * NF) {
            if (n % 4 == 0)
                raw[n / 4] = deal_codes(raw[n / 4]);
            code[set][n / 4][n % 4] = codes8<IN>(raw[n / 4][n % 4]);
            // (here, and not where the next step uses them)
            asm volatile("" : "+v"(code[set][n / 4][n % 4]));
        }
    };
    half8 a[2][4];           // operands of 16 tokens, and of the next
    auto read_tokens = [&](int set, int slot, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a[set][j] = *(const __attribute__((address_space(3))) half8 *)(
                lds + slot * Cfg::BUF_A + 4096 * i + 256 * r + 16 * ((4 * j + kg) ^ r));
    };
    float scale[2][NF][NS];  // [step % 2]
    auto read_scales = [&](int set, int s, int slot) __attribute__((always_inline)) {
        const lds_u8 *const from = lds + Cfg::AT_S + (slot * NW + wave) * Cfg::BUF_S;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int c = NF * r + f;
            const int i = odd + c * (int)args.lds + (GS == kCoarse ? s >> (args.shift - 7) : 0);
#pragma unroll
            for (int g = 0; g < NS; ++g) {
                const int at = (i & 1) + g;
                scale[set][f][g] = scale_value<IN>(*(const __attribute__((address_space(3))) uint16_t *)(
                    from + 4 * ((at >> 1) * CH + c) + 2 * (at & 1)));
                if (NS > 1 && s == full)
                    scale[set][f][g] = NS * s + g < groups_k ? scale[set][f][g] : 0.0f;
            }
        }
    };
    constexpr bool LATER = NS == 1;   // sums join a step of 16 tokens later (fine groups have too many)
    floatx4 p[LATER ? 2 : 1][NF][NS];
    auto join = [&](int set, int sums, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < NS; ++g)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[i][f][v] = __builtin_fmaf(scale[set][f][g], p[sums][f][g][v], acc[i][f][v]);
        // (here, and not where the next sums join: those would wait in registers)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            asm volatile("" : "+v"(acc[i][f]));
    };
    const bool works = cols > 0;

    // Makes step s visible; LEFT later copies of this wave may be in flight.
    auto publish = [&](int s, int slot, auto later) __attribute__((always_inline)) {
        if (s == full && (KA & 15) != 0) {
            wait_vmcnt<0>();
            fill_end(slot);
        } else {
            wait_vmcnt<decltype(later)::value>();
        }
        __syncthreads();
    };
    if (steps > 0) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
            copy_codes(0, 0, f);
        copy_batch(0, 0);
        copy_batch(1, 1);
        wait_vmcnt<2 * Cfg::COPIES>();
        if (works) {
            read_codes(0, 0);
#pragma unroll
            for (int n = 0; n < 4 * NF; ++n)
                expand(0, n);
        }
        publish(0, 0, std::integral_constant<int, Cfg::COPIES>{});
        if (works) {
            read_tokens(0, 0, 0);
            read_codes(1, 1);
            read_scales(0, 0, 0);
        }
    }
    // One step, P = s % 2 (so that registers are named at compile time).
    int slot = 0;
    auto step = [&](int s, auto parity) __attribute__((always_inline)) {
        constexpr int P = decltype(parity)::value;
        const int after = next_slot(slot), third = next_slot(after);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const bool last = i + 1 == FM;
            if (last && s + 1 < steps) {
                publish(s + 1, after, std::integral_constant<int, Cfg::COPIES>{});
                read_tokens((i + 1) & 1, after, 0);
                read_scales(P ^ 1, s + 1, after);
            } else if (!last) {
                read_tokens((i + 1) & 1, slot, i + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int g = 0; g < NS; ++g)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    p[LATER ? i & 1 : 0][f][g] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    floatx4 &sum = p[LATER ? i & 1 : 0][f][j / PER];
                    sum = mfma16<IN>(a[i & 1][j], code[P][f][j], sum);
                }
            if constexpr (LATER) {
                if (i > 0)
                    join(P, (i - 1) & 1, i - 1);
                else if (s > 0)
                    join(P ^ 1, (FM - 1) & 1, FM - 1);
            } else {
                join(P, 0, i);
            }
#pragma unroll
            for (int e = 0; e < Cfg::EXPAND; ++e)
                expand(P ^ 1, i * Cfg::EXPAND + e);
            __builtin_amdgcn_sched_barrier(0);
            // a few copies at a time: all at once would hold up the wave
            constexpr int SLICE = (Cfg::COPIES + FM - 2) / (FM - 1);
            if (!last)
#pragma unroll
                for (int q = i * SLICE; q < (i + 1) * SLICE; ++q)
                    if (q < Cfg::COPIES)
                        copy_one(s + 2, third, q);
            __builtin_amdgcn_sched_barrier(0);
        }
        read_codes(s + 2, third);
        slot = after;
    };
    // A wave without channels only copies: the matrix cores are left to the
    // waves with work.
    if (!works) {
        for (int s = 0; s + 1 < steps; ++s) {
            slot = next_slot(slot);
            copy_batch(s + 2, next_slot(slot));
            publish(s + 1, slot, std::integral_constant<int, Cfg::COPIES>{});
        }
        wait_vmcnt<0>();
        return;
    }
    for (int s = 0; s < steps; s += 2) {
        step(s, std::integral_constant<int, 0>{});
        if (s + 1 < steps)
            step(s + 1, std::integral_constant<int, 1>{});
    }
    if (LATER && steps > 0) {
        if (steps % 2)
            join(0, (FM - 1) & 1, FM - 1);
        else
            join(1, (FM - 1) & 1, FM - 1);
    }
    wait_vmcnt<0>();  // (copies from empty buffers: none may land in another workgroup's LDS)
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
// -8 .. 7 nearest to w/s, the even one in the middle, decided exactly.  Both are
// first multiplied by the power of two that brings s to [0.5, 1) or near it
// (exact: s stays a normal number, and a w that would become too small for one
// has code 0 either way).  A group with an infinity or a NaN, or whose scale its
// type does not hold, has a NaN scale and codes 0.
//
// 16-bit w: with w = P*2^j and s = A*2^i, P and A of 11 bits, a quotient that is
// no middle of two codes differs from one by at least 2^-16 of itself, so FP32
// decides; a middle is an FP32 number itself, which t = w * (1/s) plus its exact
// remainder times 1/s gives, whatever the last digit of 1/s is.
// FP32 w: q = rint(w * (1/s)) is off by one at most, and the remainder w - q*s
// (one fused multiply-add, exact near a middle: q*s has at most 15 bits, and
// what is left is a multiple of 2^-25 of s) against s/2 says which way.
template <int WT, int ST>
struct W4Scale {
    float s, f, inv;
    uint16_t bits;
    __device__ __forceinline__ explicit W4Scale(uint32_t top)
    {
        typedef typename ElemOf<ST>::type E;
        const float most = __builtin_bit_cast(float, top);
        // m/7 rounded correctly: m * (1/7) plus its exact remainder times 1/7
        constexpr float seventh = 1.0f / 7.0f;
        float v = most * seventh;
        v = __builtin_fmaf(__builtin_fmaf(-7.0f, v, most), seventh, v);
        if (most < 0x1p-100f)
            v = most / 7.0f;  // (where that would round twice)
        E e = (E)v;
        v = (float)e;
        if (top >= 0x7F800000u || __builtin_bit_cast(uint32_t, v) >= 0x7F800000u) {
            e = (E)__builtin_nanf("");
            v = 0.0f;
        }
        bits = __builtin_bit_cast(uint16_t, e);
        int ex = __builtin_amdgcn_frexp_expf(v);
        ex = ex < -126 ? -126 : ex > 126 ? 126 : ex;
        // (without a scale every code is 0: by f = 0, for infinities see code)
        f = v > 0.0f ? __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23) : 0.0f;
        s = v > 0.0f ? v * f : 1.0f;
        inv = __builtin_amdgcn_rcpf(s);
    }
    // The code of a value, as a float.
    __device__ __forceinline__ float code(float w) const
    {
        const float x = w * f;
        float q;
        if constexpr (WT != kTF32) {
            const float t = x * inv;
            q = __builtin_rintf(__builtin_fmaf(__builtin_fmaf(-t, s, x), inv, t));
        } else {
            q = __builtin_rintf(x * inv);
            const float rest = __builtin_fmaf(-q, s, x), half = 0.5f * s;
            const bool odd = ((int)q & 1) != 0;
            if (rest > half || (rest == half && odd))
                q += 1.0f;
            else if (rest < -half || (rest == -half && odd))
                q -= 1.0f;
        }
        q = __builtin_amdgcn_fmed3f(q, -8.0f, 7.0f);
        return f == 0.0f ? 0.0f : q;
    }
    // Eight codes in four bytes: the pairs' bytes are whole FP32 numbers.
    __device__ __forceinline__ uint32_t pack(const float (&v)[8]) const
    {
        uint32_t o = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_fmaf(16.0f, code(v[2 * e + 1]), code(v[2 * e]) + 136.0f), e, o);
        return o;
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

// The largest of 2^n neighbouring lanes' numbers, lanes that start at a multiple
// of that: within 16 lanes by register moves.
__device__ __forceinline__ uint32_t most_of_lanes(uint32_t v, int lanes)
{
    auto with = [&](uint32_t other) __attribute__((always_inline)) { v = max(v, other); };
    if (lanes >= 2)
        with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1 /* quad_perm 1 0 3 2 */, 0xF, 0xF, true));
    if (lanes >= 4)
        with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E /* quad_perm 2 3 0 1 */, 0xF, 0xF, true));
    if (lanes >= 8)
        with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141 /* row_half_mirror */, 0xF, 0xF, true));
    if (lanes >= 16)
        with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140 /* row_mirror */, 0xF, 0xF, true));
    if (lanes >= 32)
        with((uint32_t)__shfl_xor((int)v, 16));
    if (lanes >= 64)
        with((uint32_t)__shfl_xor((int)v, 32));
    return v;
}

// A lane has 16 neighbouring values, a wave 1024 of a row.  Groups of up to 1024
// values are the lanes of one wave; of larger ones a wave has one, read twice.
// Bound: the vector units and HBM (8192x8192 BF16 in groups of 128 53 us, 3.2 TB/s;
// 87 with 8 values a lane, whose scales and remainders cost as much as the codes).
constexpr int kPackSpan = 1024;

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
    const int64_t span = size > kPackSpan ? size : kPackSpan;
    const int64_t first = (unit - row * args.parts) * span, end = first + span < K ? first + span : K;
    const E *const w = (const E *)args.W + row * args.ldw;
    float v[2][8];
    uint32_t top = 0;
    const int64_t at = first + 16 * lane;
    auto load = [&](int64_t k) __attribute__((always_inline)) {
        load_values(w, k, K, v[0]);
        load_values(w, k + 8, K, v[1]);
    };
    for (int64_t k = at; k < end; k += kPackSpan) {
        load(k);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            top = max(top, magnitude(v[e / 8][e % 8]));
    }
    const int lanes = args.shift >= 10 ? 64 : 1 << (args.shift - 4);
    top = most_of_lanes(top, lanes);
    const W4Scale<WT, ST> scale(top);
    if ((lane & (lanes - 1)) == 0 && at < end)
        args.S[row * args.lds + (at >> args.shift)] = scale.bits;
    uint8_t *const q = args.Q + row * args.ldq;
    for (int64_t k = at; k < end; k += kPackSpan) {
        if (size > kPackSpan)
            load(k);
        const u32x2 o = {scale.pack(v[0]), scale.pack(v[1])};
        if (k + 16 <= K) {
            *(Pack<uint8_t, 8> *)(q + k / 2) = __builtin_bit_cast(Pack<uint8_t, 8>, o);
        } else {
            // (a value behind the row is 0, so the spare nibble is 8)
            for (int e = 0; e < 8; ++e)
                if (k + 2 * e < K)
                    q[k / 2 + e] = (uint8_t)(o[e / 4] >> (8 * (e % 4)));
        }
    }
}

// A lane makes 8 values of four bytes.  Bound: the writing of the values (8192x8192
// to FP32 50 us, 6 TB/s).
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
