// i8_kernels.hpp -- products of 8-bit codes with scales per token and channel
// (gfx950).  Included by ops.hip after kernels.hpp, in its namespace.
//
//     C[i][j] = (float)(sum_k A[i][k] * W[j][k]) * scale_a[i] * scale_w[j] (+ bias[j])
//
// A: tokens x K codes, W: channels x K codes (both K-contiguous), the sum
// exact in 32-bit integers, rounded once to FP32 before the scales (see
// i8_value for theirs) and once more to the output type.  With groups, token rows
// [offsets[g], offsets[g+1]) use W[g], scale_w[g], bias[g].
//
// i8_tile<Cfg>: the schedule of the 16-bit pipelined kernel (an LDS ring of K
// tiles filled by direct-to-LDS copies, operands one k-step ahead of their
// matrix instructions) on v_mfma_i32_16x16x64_i8: a lane supplies 16
// K-consecutive codes, the same 16 bytes as 8 16-bit values, so tiles,
// swizzles and copies are those of a 16-bit product half as deep.  What
// differs:
//  * the weights are the instruction's first operand and the tokens its
//    second, so a lane's accumulators are neighbouring channels of one token:
//    one scale_a per lane and operand, and wide stores;
//  * pairs of weight operands take interleaved groups of 4 channels (operand
//    2p + h, row r holds channel 32p + 8*(r/4) + 4h + r%4), which gives a
//    lane 8 consecutive channels: 16-byte stores of 16-bit outputs;
//  * K % 16 needs no extra step: the vector that straddles K is filled
//    through registers with zeros behind K;
//  * scales and bias wait in LDS behind the ring, and C leaves in whole
//    128-byte lines.
// Bound: the matrix cores at the board's power limit for large products (8192^3
// to FP32 452-471 us, 2.3e15-2.4e15 operations/s, matrix pipes busy 60% of the time at
// 1.84 GHz, no LDS bank conflicts); between rounds of tiles the first copies
// and the stores show (8192x8192x2048 to BF16 133 us, of which about 40 are not
// products), and with experts of unequal sizes the last round is part empty
// (16384 rows over 32 experts of 2048x2048 98 us: compute units hold waves
// 72% of the time).
// Matrix-core layout (v_mfma_i32_16x16x64_i8): lane l supplies
// A[l%16][16*(l/16) + 0..15] and B[16*(l/16) + 0..15][l%16]; accumulator v
// of lane l holds D[4*(l/16) + v][l%16].

struct I8Args {
    const int8_t *A;
    const int8_t *W;
    void *C;
    const float *scale_a;
    const float *scale_w;
    const float *bias;       // or nullptr
    int64_t lda, ldw, ldc;   // elements
    int32_t N, K;
    int32_t tiles_n;
    int32_t group_m;
    int32_t stream_c;        // rows of C start on 128-byte lines: stores past the caches
    GroupArgs groups;
};

// Element types of tensors, as MPGEMM_T_* in the header.
constexpr int kTF16 = 0;
constexpr int kTBF16 = 1;
constexpr int kTF32 = 2;

template <int T>
struct ElemOf;
template <>
struct ElemOf<kTF16> {
    typedef _Float16 type;
};
template <>
struct ElemOf<kTBF16> {
    typedef __bf16 type;
};
template <>
struct ElemOf<kTF32> {
    typedef float type;
};

// 16 bytes at any address
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

// N elements at any element-aligned address (the vector memory of gfx9
// devices runs in unaligned mode under ROCm).
template <class E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Pack {
    E v[N];
};

// One K-contiguous operand tile of BX rows of BKB bytes in LDS; see OpTile.
// PAIR: read by paired operands (rows 0..3, 8..11, 16..19, 24..27 of 32, or
// those plus 4, in one 16-lane group); otherwise 16 consecutive rows.
template <int BX, int BKB, int NW, bool PAIR>
struct I8Tile {
    static constexpr int CH = BKB / 16;      // 16-byte chunks per row
    static constexpr int RPI = 64 / CH;      // rows per copy instruction
    static constexpr int PW = BX / RPI / NW; // copies per wave per tile
    static constexpr int BYTES = BX * BKB;
    static_assert(CH == 8 || CH == 16, "rows of 128 or 256 bytes");
    static_assert((BX / RPI) % NW == 0 && PW >= 1, "copies must split evenly over waves");
    // The 16 rows that one 16-lane group of a ds_read_b128 touches at one
    // chunk must fall on 256 distinct bytes of the 64 banks.  256-byte rows:
    // 16 different chunks; 128-byte rows: the row's lowest bit picks the half
    // of the banks, the other three bits that vary pick one of 8 chunks.
    __device__ static __forceinline__ int swz(int r)
    {
        if constexpr (PAIR) {
            const int hi = (r >> 3) & 3;     // bits 3, 4
            return CH == 16 ? (r & 3) | (hi << 2) : ((r >> 1) & 1) | (hi << 1);
        } else {
            return CH == 16 ? (r & 15) : ((r >> 1) & 7);
        }
    }
};

template <int BM_, int BN_, int BKB_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct I8Cfg {
    static constexpr int BM = BM_, BN = BN_, BKB = BKB_;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
    static constexpr int FM = WTM / 16, FN = WTN / 16;
    static constexpr int KS = BKB / 64;               // k-steps per tile
    static constexpr bool PAIR = FN % 2 == 0;
    using TA = I8Tile<BM, BKB, NW, false>;
    using TW = I8Tile<BN, BKB, NW, PAIR>;
    static constexpr int STAGE_BYTES = TA::BYTES + TW::BYTES;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    // behind the ring: scale_a of the tile's rows, scale_w and bias of its
    // columns, in units of 64 floats
    static constexpr int UA = (BM + 63) / 64, UW = (BN + 63) / 64;
    static constexpr int UNITS = UA + 2 * UW;
    static constexpr int LDS_BYTES = RING_BYTES + UNITS * 256;
    static constexpr int NCOPY = TA::PW + TW::PW;
    static constexpr int COPY_WINDOW = STAGES == 2 ? (NCOPY < KS * FM ? NCOPY : KS * FM) : KS * FM;
    static_assert(WTM % 16 == 0 && WTN % 16 == 0, "wave tiles are multiples of the instruction's");
    static_assert(KS >= 2, "a K tile holds two k-steps at least");
    static_assert(STAGES >= 2 && STAGES <= 8, "2..8 LDS stages");
    static_assert(NCOPY * (STAGES - 1) < 64, "vmcnt is 6 bits");
    static_assert(LDS_BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
};

typedef int32_t i32x4v __attribute__((ext_vector_type(4)));

// One value of the product: the exact sum and its product with scale_a each
// rounded to FP32, then the product with scale_w and the bias rounded once.
// The fma is written out: left to the compiler's contraction of products and
// sums, that rounding would be an option of the build.
__device__ __forceinline__ float i8_value(int32_t sum, float sa, float sw, float bias, bool has_bias)
{
    const float v = (float)sum * sa;
    return has_bias ? __builtin_fmaf(v, sw, bias) : v * sw;
}

// COUNT consecutive channels of one token, from column `col` (left = columns
// from it to the edge).
template <int OUT, int COUNT>
__device__ __forceinline__ void i8_store(typename ElemOf<OUT>::type *row, int col, int left, const float *v)
{
    typedef typename ElemOf<OUT>::type E;
    if (left >= COUNT) {
        Pack<E, COUNT> p;
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            p.v[e] = (E)v[e];
        *(Pack<E, COUNT> *)(row + col) = p;
    } else {
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            if (e < left)
                row[col + e] = (E)v[e];
    }
}

// Wait until at most `newer` whole tiles' copies (0 .. MOST) are in flight.
template <class Cfg, int MOST>
__device__ __forceinline__ void wait_tiles(int newer)
{
    if constexpr (MOST <= 0) {
        wait_vmcnt<0>();
    } else {
        if (newer >= MOST)
            wait_vmcnt<MOST * Cfg::NCOPY>();
        else
            wait_tiles<Cfg, MOST - 1>(newer);
    }
}

// One wave instruction: lane l copies 4 bytes from rsrc at voff into LDS at
// byte address lds_addr + 4*l (see dma16).
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds_addr, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"(lds_addr), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

template <class Cfg, int OUT>
__global__ void __launch_bounds__(Cfg::NT)
i8_tile(I8Args args)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BKB = Cfg::BKB, S = Cfg::STAGES;
    constexpr int FM = Cfg::FM, FN = Cfg::FN, KS = Cfg::KS, NCOPY = Cfg::NCOPY;
    using TA = typename Cfg::TA;
    using TW = typename Cfg::TW;
    typedef typename ElemOf<OUT>::type E;

    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES];
    lds_u8 *const lds = (lds_u8 *)smem;
    const uint32_t lds_base = (uint32_t)(uintptr_t)lds;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / Cfg::WAVES_N;
    const int wn = wave % Cfg::WAVES_N;

    GroupTile gt;
    if (!find_row_tile(args.groups, BM, args.tiles_n, args.group_m, gt))
        return;
    const int K = args.K;
    const int row0 = gt.start + gt.tm * BM;          // first token row of the tile
    const int rows_left = gt.rows - gt.tm * BM;      // > 0
    const int n0 = gt.tn * BN;
    const int cols_left = args.N - n0;               // > 0
    const int8_t *const Ap = args.A + (int64_t)row0 * args.lda;
    const int8_t *const Wp = args.W + (int64_t)gt.group * args.groups.stride + (int64_t)n0 * args.ldw;

    // ---- copies: slot q of this wave fills LDS rows RPI*j .. of its operand
    // (j = i*NW + wave) from a fixed place of the operand; the K tile moves
    // the scalar offset.  Rows outside the product, and in the last tile
    // chunks at or past K, read zeros.
    const i32x4 rsA = make_rsrc4(Ap), rsW = make_rsrc4(Wp);
    uint32_t voff[NCOPY];
#pragma unroll
    for (int q = 0; q < NCOPY; ++q) {
        const bool is_a = q < TA::PW;
        const int i = is_a ? q : q - TA::PW;
        const int j = i * Cfg::NW + wave;
        const int r = TA::RPI * j + lane / TA::CH;
        const int c = (lane % TA::CH) ^ (is_a ? TA::swz(r) : TW::swz(r));
        const bool ok = r < (is_a ? rows_left : cols_left);
        voff[q] = ok ? (uint32_t)(r * (int)(is_a ? args.lda : args.ldw) + 16 * c) : kOOB;
    }
    const int num_k = (K + BKB - 1) / BKB;
    const int klast = K - (num_k - 1) * BKB;         // bytes of the last tile
    // this lane's 16-byte chunk of slot q's rows (looked at in the last tile)
    auto chunk_of = [&](int q) __attribute__((always_inline)) {
        const bool is_a = q < TA::PW;
        const int i = is_a ? q : q - TA::PW;
        const int r = TA::RPI * (i * Cfg::NW + wave) + lane / TA::CH;
        return (lane % TA::CH) ^ (is_a ? TA::swz(r) : TW::swz(r));
    };
    uint32_t copy_region = 0, copy_soff = 0;
    int copy_tile = 0;
    auto begin_copies = [&](int t, int buf) __attribute__((always_inline)) {
        copy_region = lds_base + buf * Cfg::STAGE_BYTES;
        copy_soff = (uint32_t)t * BKB;
        copy_tile = t;
    };
    auto copy_one = [&](int q) __attribute__((always_inline)) {
        if (copy_tile >= num_k)
            return;
        const bool is_a = q < TA::PW;
        const int j = (is_a ? q : q - TA::PW) * Cfg::NW + wave;
        uint32_t off = voff[q];
        if (copy_tile == num_k - 1 && klast < BKB && 16 * chunk_of(q) + 16 > klast)
            off = kOOB;
        dma16(is_a ? rsA : rsW, copy_region + (is_a ? 0 : TA::BYTES) + j * 1024, off, copy_soff);
    };
    // The vectors of the last tile that straddle K, into the slots where the
    // copies wrote zeros: the row's last 16 bytes, shifted down so that zeros
    // stand behind K (a row of less than 16 bytes byte by byte).  Two rows'
    // loads at a time: the accumulators leave no registers for more.
    auto fill = [&](int buf) __attribute__((always_inline)) {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int c_at = klast / 16, nv = klast % 16;
        auto place = [&](int q, int &r, bool &here) __attribute__((always_inline)) {
            const bool is_a = q < TA::PW;
            const int j = (is_a ? q : q - TA::PW) * Cfg::NW + wave;
            r = TA::RPI * j + ln / TA::CH;
            const int c = (ln % TA::CH) ^ (is_a ? TA::swz(r) : TW::swz(r));
            here = c == c_at && r < (is_a ? rows_left : cols_left);
            return j;
        };
#pragma unroll
        for (int q0 = 0; q0 < NCOPY; q0 += 2) {
            u32x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int q = q0 + h;
                if (q >= NCOPY)
                    break;
                const bool is_a = q < TA::PW;
                int r;
                bool here;
                place(q, r, here);
                v[h] = u32x4{0, 0, 0, 0};
                if (here) {
                    const int8_t *const row = is_a ? Ap + (int64_t)r * args.lda : Wp + (int64_t)r * args.ldw;
                    if (K >= 16) {
                        v[h] = *(const u32x4_any *)(row + K - 16);
                    } else {
                        for (int e = 0; e < nv; ++e) {
                            const uint32_t b = (uint32_t)(uint8_t)row[e] << (8 * (e & 3));
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                v[h][w] |= e / 4 == w ? b : 0u;
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int q = q0 + h;
                if (q >= NCOPY)
                    break;
                const bool is_a = q < TA::PW;
                int r;
                bool here;
                const int j = place(q, r, here);
                if (here) {
                    u32x4 x = v[h];
                    if (K >= 16)
                        x = __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, x) >> (8 * (16 - nv)));
                    *(lds_u32x4 *)(lds + buf * Cfg::STAGE_BYTES + (is_a ? 0 : TA::BYTES) + j * 1024 + ln * 16) = x;
                }
            }
        }
    };

    // ---- operand reads
    const int a_row = wm * Cfg::WTM + (lane & 15);
    const int a_base = a_row * BKB, a_sw = TA::swz(a_row);
    const int w_row = wn * Cfg::WTN + (Cfg::PAIR ? 8 * ((lane & 15) >> 2) + (lane & 3) : (lane & 15));
    const int w_base = w_row * BKB, w_sw = TW::swz(w_row);
    i32x4v ra[FM], rw[2][FN];
    auto read_a = [&](int buf, int ks, int f) __attribute__((always_inline)) {
        ra[f] = *(const __attribute__((address_space(3))) i32x4v *)(lds + buf * Cfg::STAGE_BYTES + a_base +
                                                                    f * 16 * BKB + ((4 * ks + lane / 16) ^ a_sw) * 16);
    };
    auto read_w = [&](int buf, int ks, int set, int f) __attribute__((always_inline)) {
        const int drow = Cfg::PAIR ? 32 * (f / 2) + 4 * (f % 2) : 16 * f;
        rw[set][f] = *(const __attribute__((address_space(3))) i32x4v *)(lds + buf * Cfg::STAGE_BYTES + TA::BYTES +
                                                                         w_base + drow * BKB +
                                                                         ((4 * ks + lane / 16) ^ w_sw) * 16);
    };

    i32x4v acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = i32x4v{0};

    // Make tile t (in buffer buf) visible: its copies have landed (`newer`
    // whole tiles issued after it may still be in flight).
    auto publish = [&](int t, int buf, int newer) __attribute__((always_inline)) {
        if (t == num_k - 1 && (klast & 15) != 0) {
            wait_vmcnt<0>();
            fill(buf);
        } else {
            // (the counts are compile-time operands of the wait)
            wait_tiles<Cfg, S - 1>(newer);
        }
        __syncthreads();
    };
    auto copy_slice = [&](int p) __attribute__((always_inline)) {
        constexpr int CW = Cfg::COPY_WINDOW;
#pragma unroll
        for (int c = 0; c < NCOPY; ++c)
            if (c >= (p * NCOPY + CW - 1) / CW && c < ((p + 1) * NCOPY + CW - 1) / CW)
                copy_one(c);
    };

    // The scales and the bias go to LDS ahead of the ring, so that the epilogue
    // does not start with a trip to memory.
#pragma unroll
    for (int u0 = 0; u0 < Cfg::UNITS; u0 += Cfg::NW) {
        const int u = u0 + wave;
        if (u < Cfg::UNITS) {
            const bool is_a = u < Cfg::UA, is_w = u < Cfg::UA + Cfg::UW;
            const int at = 64 * (is_a ? u : is_w ? u - Cfg::UA : u - Cfg::UA - Cfg::UW) + lane;
            const float *const src = is_a ? args.scale_a + row0
                                          : (is_w ? args.scale_w : args.bias) + (int64_t)gt.group * args.N + n0;
            if (is_w || args.bias)
                dma4(make_rsrc4(src), lds_base + Cfg::RING_BYTES + 256 * u,
                     at < (is_a ? rows_left : cols_left) ? (uint32_t)(4 * at) : kOOB);
        }
    }
    if (num_k == 0) {
        wait_vmcnt<0>();
        __syncthreads();
    }
    if (num_k > 0) {
#pragma unroll
        for (int t = 0; t < S; ++t) {
            begin_copies(t, t);
#pragma unroll
            for (int c = 0; c < NCOPY; ++c)
                copy_one(c);
        }
        publish(0, 0, num_k - 1 < S - 1 ? num_k - 1 : S - 1);
#pragma unroll
        for (int f = 0; f < FM; ++f)
            read_a(0, 0, f);
#pragma unroll
        for (int f = 0; f < FN; ++f)
            read_w(0, 0, 0, f);
    }
    int buf = 0;
    // A wave whose part of the tile lies outside the product only copies: the
    // matrix cores are left to the waves with work.
    if (wm * Cfg::WTM >= rows_left || wn * Cfg::WTN >= cols_left) {
        for (int kt = 0; kt < num_k; ++kt) {
            const int nbuf = (buf + 1 == S) ? 0 : buf + 1;
            if (kt + 1 < num_k) {
                const int newer = num_k - 2 - kt;
                publish(kt + 1, nbuf, newer < S - 2 ? newer : S - 2);
            }
            begin_copies(kt + S, buf);
#pragma unroll
            for (int c = 0; c < NCOPY; ++c)
                copy_one(c);
            buf = nbuf;
        }
        return;
    }
    for (int kt = 0; kt < num_k; ++kt) {
        const int nbuf = (buf + 1 == S) ? 0 : buf + 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int set = ks & 1;
            const bool last = ks + 1 == KS;
            if (last && kt + 1 < num_k) {
                const int newer = num_k - 2 - kt;
                publish(kt + 1, nbuf, newer < S - 2 ? newer : S - 2);
            }
            if (last)
                begin_copies(kt + S, buf);
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if (!last)
                    read_w(buf, ks + 1, set ^ 1, f);
                else if (kt + 1 < num_k)
                    read_w(nbuf, 0, set ^ 1, f);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(rw[set][j], ra[i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (!last)
                    read_a(buf, ks + 1, i);
                else if (kt + 1 < num_k)
                    read_a(nbuf, 0, i);
                // the last k-step opens the window of tile kt+S; the others
                // continue that of tile kt+S-1, which the ring fill issued
                // whole when kt == 0
                if (last)
                    copy_slice(i);
                else if (kt > 0)
                    copy_slice(FM + ks * FM + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        buf = nbuf;
    }

    // ---- epilogue: lane l holds token l%16 of operand i and, per operand
    // pair, channels 32p + 8*(l/16) + 0..7 (unpaired: 16j + 4*(l/16) + 0..3)
    constexpr int COUNT = Cfg::PAIR ? 8 : 4;
    constexpr int NP = Cfg::PAIR ? FN / 2 : FN;
    const int lrow = wm * Cfg::WTM + (lane & 15);
    const int lcol = wn * Cfg::WTN + COUNT * (lane >> 4);
    const __attribute__((address_space(3))) float *const sc =
        (const __attribute__((address_space(3))) float *)(lds + Cfg::RING_BYTES);
    const bool has_bias = args.bias != nullptr;
    float sa[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        sa[i] = sc[lrow + 16 * i];
    // the values of this lane's COUNT channels of pair p, for operand i
    auto values = [&](int p, int i, const float (&sw)[COUNT], const float (&bv)[COUNT], float (&v)[COUNT])
        __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < COUNT; ++e) {
            const int32_t sum = acc[i][Cfg::PAIR ? 2 * p + e / 4 : p][e % 4];
            v[e] = i8_value(sum, sa[i], sw[e], bv[e], has_bias);
        }
    };
    auto scales = [&](int p, float (&sw)[COUNT], float (&bv)[COUNT]) __attribute__((always_inline)) {
        const int c = lcol + 4 * COUNT * p;
#pragma unroll
        for (int e = 0; e < COUNT; ++e) {
            sw[e] = sc[64 * Cfg::UA + c + e];
            bv[e] = has_bias ? sc[64 * (Cfg::UA + Cfg::UW) + c + e] : 0.0f;
        }
    };
    E *const out = (E *)args.C + (int64_t)row0 * args.ldc + n0;
    // Whole lines.  A store of 16 bytes a lane covers 64 bytes of each of 16
    // rows (16-bit values), or every other 16 bytes of 128 (FP32): partial
    // lines, which cost the L2 about a third more time.  Lanes r and r + 8 of
    // a group of 16 swap one of their two 16-byte pieces, so that one store
    // fills 128 bytes of rows 0..7 and the next those of rows 8..15.  Where
    // they are lines of C, they stream past the caches and leave those to the
    // operands (8192x8192x2048 to FP32 170 -> 152 us, to BF16 145 -> 133;
    // 2048^3 to FP32 17.3 -> 15.7).
    constexpr int NQ = OUT == kTF32 ? 1 : 2;  // pairs that make one line
    if constexpr (Cfg::PAIR && NP % NQ == 0) {
        if (wn * Cfg::WTN + Cfg::WTN <= cols_left) {
            const bool low = (lane & 8) == 0;
            const int srow = wm * Cfg::WTM + (lane & 7);
#pragma unroll
            for (int q = 0; q < NP; q += NQ) {
                float sw[NQ][COUNT], bv[NQ][COUNT];
#pragma unroll
                for (int h = 0; h < NQ; ++h)
                    scales(q + h, sw[h], bv[h]);
                // column of this lane's piece within the line
                const int c = OUT == kTF32 ? lcol + 32 * q + (low ? 0 : 4) : lcol + 32 * (low ? q : q + 1);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    u32x4 piece[2];
                    if constexpr (OUT == kTF32) {
                        float v[COUNT];
                        values(q, i, sw[0], bv[0], v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            piece[e / 4][e % 4] = __builtin_bit_cast(uint32_t, v[e]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[COUNT];
                            values(q + h, i, sw[h], bv[h], v);
                            Pack<E, 8> o;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o.v[e] = (E)v[e];
                            piece[h] = __builtin_bit_cast(u32x4, o);
                        }
                    }
                    u32x4 first, second;  // of rows 0..7 and 8..15
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t mine0 = piece[0][e], mine1 = piece[1][e];
                        const uint32_t theirs = __builtin_amdgcn_update_dpp(0, low ? mine1 : mine0, 0x128 /* row_ror:8 */,
                                                                            0xF, 0xF, true);
                        first[e] = low ? mine0 : theirs;
                        second[e] = low ? theirs : mine1;
                    }
                    auto store = [&](int row, const u32x4 &x) __attribute__((always_inline)) {
                        u32x4_any *const to = (u32x4_any *)(out + (int64_t)row * args.ldc + c);
                        if (row < rows_left) {
                            if (args.stream_c)
                                __builtin_nontemporal_store(x, to);
                            else
                                *to = x;
                        }
                    };
                    store(srow + 16 * i, first);
                    store(srow + 16 * i + 8, second);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = lcol + 4 * COUNT * p;
        const int left = cols_left - c;
        if (left <= 0)
            continue;
        float sw[COUNT], bv[COUNT];
        scales(p, sw, bv);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (lrow + 16 * i >= rows_left)
                continue;
            float v[COUNT];
            values(p, i, sw, bv, v);
            i8_store<OUT, COUNT>(out + (int64_t)(lrow + 16 * i) * args.ldc, c, left, v);
        }
    }
}
