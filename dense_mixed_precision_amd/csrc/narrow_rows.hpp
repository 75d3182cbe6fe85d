// narrow_rows.hpp -- products of few token rows with a weight matrix read once
// (gfx950).  Included by ops.hip in kernels.hpp's namespace, after
// i8_kernels.hpp.
//
// At most 16 token rows per tile make the product a stream over the weights
// (N x K, K-contiguous): 16 channels per workgroup, its waves splitting K,
// the weights straight from memory into operand registers with DEPTH loads in
// flight, the tokens beside them (a few rows, from the L2).  Nothing of a weight row is
// used twice, so an LDS ring would only add a copy and a barrier per K tile.
// The waves' partial tiles are summed in LDS in wave order.
//
// Bound: HBM.  8x8192x8192 codes 14.4 us, 4.65 TB/s; 64 BF16 rows over 64
// experts of 2048x2048, of which they reach about 41, 58 us, 5.9 TB/s (1 GiB
// copies at 5.2).
//
// The same bytes serve 8-bit codes (v_mfma_i32_16x16x64_i8, 16 codes per lane)
// and 16-bit values (v_mfma_f32_16x16x32_{f16,bf16}, 8 per lane); the weights
// are the first operand, so accumulator v of lane l is channel 4*(l/16) + v of
// token l%16.

constexpr int kNarrowI8 = 2;  // besides kInF16 and kInBF16

struct NarrowArgs {
    const uint8_t *A;        // tokens
    const uint8_t *W;        // N x K per group
    void *C;
    int64_t lda, ldw, ldc;   // bytes, bytes, elements
    int64_t stride_w;        // bytes
    int32_t N, KB;           // channels, bytes of a row
    int32_t tiles_n;
    GroupArgs groups;
    // 8-bit codes
    const float *scale_a, *scale_w, *bias;
    // 16-bit values
    float alpha, beta;
};

template <int IN>
struct NarrowAcc {
    typedef floatx4 type;
    static constexpr int ES = 2;
};
template <>
struct NarrowAcc<kNarrowI8> {
    typedef i32x4v type;
    static constexpr int ES = 1;
};

template <int IN, int OUT, int DEPTH, int WAVES>
__global__ void __launch_bounds__(64 * WAVES)
narrow_rows(NarrowArgs args)
{
    typedef typename NarrowAcc<IN>::type Acc;
    typedef typename ElemOf<OUT>::type E;
    constexpr int ES = NarrowAcc<IN>::ES;
    __shared__ Acc part[WAVES][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupTile gt;
    if (!find_row_tile(args.groups, 16, args.tiles_n, 1, gt))
        return;
    const int row0 = gt.start + gt.tm * 16;
    const int rows = min(gt.rows - gt.tm * 16, 16);
    const int n0 = gt.tn * 16;
    const int cols = args.N - n0;
    const int KB = (IN != kNarrowI8 && args.alpha == 0.0f) ? 0 : args.KB;
    const int r = lane & 15;          // token of the second operand, channel of the first
    const int kq = 16 * (lane >> 4);  // this lane's bytes within a 64-byte step
    const bool a_ok = r < rows;
    const uint8_t *const Ap = args.A + (int64_t)row0 * args.lda;
    const uint8_t *const Wp = args.W + (int64_t)gt.group * args.stride_w + (int64_t)n0 * args.ldw;
    const __amdgpu_buffer_rsrc_t rsA = make_rsrc(Ap), rsW = make_rsrc(Wp);
    // 32-bit offsets: the host checks that 16 rows span less than 2 GiB
    const uint32_t offA = (uint32_t)(r * (int)args.lda + kq);
    const uint32_t offW = r < cols ? (uint32_t)(r * (int)args.ldw + kq) : kOOB;

    // this wave's 64-byte steps of the whole vectors; the last KB % 16 bytes
    // are a step of their own
    const int whole = KB & ~15;
    const int steps = (whole + 63) / 64;
    const int per = (steps + WAVES - 1) / WAVES;
    const int s0 = min(wave * per, steps), s1 = min(s0 + per, steps);
    u32x4 ra[DEPTH], rw[DEPTH];
    auto issue = [&](int d, int s) __attribute__((always_inline)) {
        const bool k_ok = 64 * s + kq < whole;
        rw[d] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsW, k_ok ? offW : kOOB, 64 * s, 0));
        ra[d] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsA, (a_ok && k_ok) ? offA + 64 * s : kOOB,
                                                                                0, 0));
    };
    Acc acc = Acc{0};
    auto multiply = [&](const u32x4 &w, const u32x4 &a) __attribute__((always_inline)) {
        if constexpr (IN == kNarrowI8)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4v, w), __builtin_bit_cast(i32x4v, a),
                                                        acc, 0, 0, 0);
        else
            acc = mfma16<IN>(__builtin_bit_cast(half8, w), __builtin_bit_cast(half8, a), acc);
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (s0 + d < s1)
            issue(d, s0 + d);
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (s + d < s1) {
                multiply(rw[d], ra[d]);
                if (s + d + DEPTH < s1)
                    issue(d, s + d + DEPTH);
            }
        }
    }
    // the last KB % 16 bytes, in the first 16 lanes: element loads, zeros
    // behind the row
    if (wave == WAVES - 1 && whole < KB) {
        const int left = lane < 16 ? KB - whole : 0;
        auto tail = [&](const __amdgpu_buffer_rsrc_t &rs, uint32_t off) __attribute__((always_inline)) {
            uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 16 / ES; ++e) {
                const int at = ES * e;
                const uint32_t o = at < left && off != kOOB ? off + whole + at : kOOB;
                uint32_t x;
                if constexpr (ES == 1)
                    x = __builtin_amdgcn_raw_buffer_load_b8(rs, o, 0, 0) & 0xFFu;
                else
                    x = __builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0) & 0xFFFFu;
                v[at / 4] |= x << (8 * (at % 4));
            }
            return u32x4{v[0], v[1], v[2], v[3]};
        };
        multiply(tail(rsW, offW), tail(rsA, a_ok ? offA : kOOB));
    }

    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0)
        return;
    Acc sum = part[0][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        sum += part[w][lane];

    const int c = 4 * (lane >> 4);
    const int left = cols - c;
    if (!a_ok || left <= 0)
        return;
    E *const out = (E *)args.C + (int64_t)(row0 + r) * args.ldc + n0;
    float v[4];
    if constexpr (IN == kNarrowI8) {
        const int64_t at = (int64_t)gt.group * args.N + n0 + c;
        const float sa = args.scale_a[row0 + r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool ok = e < left;
            v[e] = i8_value(sum[e], sa, ok ? args.scale_w[at + e] : 0.0f, ok && args.bias ? args.bias[at + e] : 0.0f,
                            args.bias != nullptr);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = args.alpha * sum[e];
            if (args.beta != 0.0f && e < left)
                v[e] = __builtin_fmaf(args.beta, (float)out[c + e], v[e]);
        }
    }
    i8_store<OUT, 4>(out, c, left, v);
}
