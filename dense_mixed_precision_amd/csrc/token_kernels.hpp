// token_kernels.hpp -- rows of tokens: 8-bit codes with a scale per row, the
// order of (token, slot) pairs by expert, rows brought into that order and
// back, and the gradients (gfx950).  Included by ops.hip in kernels.hpp's
// namespace, after elements.hpp.
//
// All of these stream their operands once; they are bound by HBM, and at
// decoding sizes by the launch.  Index arrays are read as untrusted data:
// an index outside the operands counts as absent.

// Whole numbers of `count` values, all -1.
__global__ void __launch_bounds__(256)
fill_absent(int32_t *v, int64_t count)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
        v[i] = -1;
}

// The inverse of `order` (R values) over `pairs` pairs, filled with -1 before:
// inverse[order[p]] = p.  A pair that stands in `order` more than once keeps one
// row here; redo(pair, row) sees to each of the others.
template <class Redo>
__device__ __forceinline__ void invert_one(const int32_t *order, int32_t *inverse, int64_t p, int64_t pairs, Redo redo)
{
    const int pair = order[p];
    if (pair < 0 || pair >= pairs)
        return;
    const int old = atomicExch(&inverse[pair], (int)p);
    if (old >= 0)
        redo(pair, old);
}

// ---------------------------------------------------------------------------
// Rows to 8-bit codes
// ---------------------------------------------------------------------------
// One row x: m = max|x|, scale = m/127, code = the whole number nearest
// 127*x/m, the even one in the middle, decided exactly.  x and m are first
// scaled by the power of two that brings m to [1, 2) (exact).
//
// 16-bit x: p = 127*x is exact, and p/m rounded correctly to FP32 decides.  In
// whole numbers p = P*2^j, m = A*2^i with A < 2^11 and j <= i (or the same with
// j = i): a quotient that is no middle lies at least 2^(j-i)/(2A) > 2^(j-i-12)
// from one, and p/m < 2^(j-i+8) has an FP32 error below 2^(j-i-16); a middle
// is an FP32 number itself.  The quotient is p*inv plus its exact remainder
// times inv, which is correctly rounded as inv is.
//
// FP32 x: p + lo = 127*x in two floats, q = rint(p*inv) is off by one at most,
// and d = p - q*m (one fma, exact: |d| is about m/2 and a multiple of the
// operands' last places) plus lo against +-m/2 says which way.
template <int XT>
__device__ __forceinline__ int code_of(float x, float f, float f127, float m, float inv)
{
    if constexpr (XT != kTF32) {
        const float p = x * f127;
        const float t = p * inv;
        return (int)__builtin_rintf(__builtin_fmaf(__builtin_fmaf(-t, m, p), inv, t));
    } else {
        x *= f;
        const float p = 127.0f * x;
        const float lo = __builtin_fmaf(127.0f, x, -p);
        float q = __builtin_rintf(p * inv);
        const float d = __builtin_fmaf(-q, m, p);
        const float h = 0.5f * m;
        const float over = (d - h) + lo;    // > 0: above the middle of q and q + 1
        const float under = (d + h) + lo;   // < 0: below the middle of q - 1 and q
        const bool odd = ((int)q & 1) != 0;
        if (over > 0.0f || (over == 0.0f && odd))
            q += 1.0f;
        else if (under < 0.0f || (under == 0.0f && odd))
            q -= 1.0f;
        return (int)q;
    }
}

// A row's scale and codes, from its largest magnitude as bits (at or above
// 0x7F800000: the row holds an infinity or a NaN).
struct RowScale {
    float scale, f, f127, m, inv;
    bool finite;
    __device__ __forceinline__ explicit RowScale(uint32_t top)
    {
        const float most = __builtin_bit_cast(float, top);
        finite = top < 0x7F800000u;
        const bool live = finite && top != 0;
        scale = finite ? most / 127.0f : __builtin_nanf("");
        // the power of two that brings the maximum to [1, 2), as far as one
        // float holds it; a row of zeros has codes 0 by f = 0
        int ex = (int)(top >> 23) - 127;
        ex = ex < -100 ? -100 : ex > 126 ? 126 : ex;
        f = live ? __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23) : 0.0f;
        f127 = 127.0f * f;
        m = live ? most * f : 1.0f;
        inv = 1.0f / m;
    }
    template <int XT>
    __device__ __forceinline__ int code(float x) const
    {
        return finite ? code_of<XT>(x, f, f127, m, inv) : 0;
    }
};

struct QuantArgs {
    const void *X;
    int8_t *Q;
    float *scale;
    const int32_t *order;    // or nullptr: row i of X
    const int32_t *inverse;  // TOKENS: T x top_k, the rows of Q of each token's pairs
    int64_t ldx, ldq;
    int32_t T, H, R, top_k;
};

// Bound: HBM; 16384 FP16 rows of 4096 from 8192 tokens 36 us with the inverse
// (3.7 TB/s of the bytes it cannot do without), 16 BF16 rows 3.3 (launch).
// NT threads per row, 256 / NT rows per workgroup.  The first CACHE vectors
// of each thread stay in registers between the maximum and the codes; longer
// rows are read again.  With NT = 64 a row is one wave's: no barrier, and the
// 32 waves of a compute unit keep as many rows in flight; with NT = 16 a wave
// has four short ones.
// TOKENS: a row is a token's, read and coded once and written to each row of
// Q that one of its pairs has (see quantize_invert).
template <int XT, int NT, int CACHE, bool TOKENS = false>
__global__ void __launch_bounds__(256)
quantize_rows(QuantArgs args)
{
    typedef typename ElemOf<XT>::type E;
    constexpr int VN = VecOf<E>::N;
    typedef typename VecOf<E>::type V;
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x % NT;
    const int64_t row = wg_number() * (256 / NT) +
                        (NT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : (int)threadIdx.x / NT);
    if (row >= (TOKENS ? args.T : args.R))
        return;
    int64_t src = row;
    if (!TOKENS && args.order) {
        const int pair = args.order[row];
        src = pair < 0 ? -1 : pair / args.top_k;
        if (src < 0 || src >= args.T)
            return;  // no such row: what is there stays
    }
    const E *const x = (const E *)args.X + src * args.ldx;
    const int H = args.H;
    const int nv = H / VN;
    V keep[CACHE];
    uint32_t top = 0;  // |x| as bits: above every finite value for infinities and NaN
    auto see = [&](E e) __attribute__((always_inline)) {
        const float f = (float)e;
        const uint32_t b = __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
        top = b > top ? b : top;
    };
#pragma unroll
    for (int c = 0; c < CACHE; ++c) {
        const int i = c * NT + tid;
        if (i < nv)
            keep[c] = *(const V *)(x + (int64_t)i * VN);
    }
#pragma unroll
    for (int c = 0; c < CACHE; ++c)
        if (c * NT + tid < nv)
#pragma unroll
            for (int e = 0; e < VN; ++e)
                see(keep[c].v[e]);
    for (int i = CACHE * NT + tid; i < nv; i += NT) {
        const V v = *(const V *)(x + (int64_t)i * VN);
#pragma unroll
        for (int e = 0; e < VN; ++e)
            see(v.v[e]);
    }
    for (int i = nv * VN + tid; i < H; i += NT)
        see(x[i]);
#pragma unroll
    for (int d = (NT < 64 ? NT : 64) / 2; d > 0; d /= 2) {
        const uint32_t o = __shfl_xor((int)top, d);
        top = o > top ? o : top;
    }
    if constexpr (NT > 64) {
        if ((tid & 63) == 0)
            part[tid / 64] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 64; ++w)
            top = part[w] > top ? part[w] : top;
    }
    const RowScale r(top);
    auto code = [&](E e) __attribute__((always_inline)) { return r.code<XT>((float)e); };
    auto codes = [&](const V &v) __attribute__((always_inline)) {
        Pack<int8_t, VN> o;
#pragma unroll
        for (int e = 0; e < VN; ++e)
            o.v[e] = (int8_t)code(v.v[e]);
        return o;
    };
    // the rows of Q, up to 8 at a time
    constexpr int SLOTS = TOKENS ? 8 : 1;
    for (int s0 = 0; s0 < (TOKENS ? args.top_k : 1); s0 += SLOTS) {
        int to[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            to[s] = (int)row;
            if constexpr (TOKENS)
                to[s] = s0 + s < args.top_k ? args.inverse[row * args.top_k + s0 + s] : -1;
            if (to[s] >= 0 && tid == 0)
                args.scale[to[s]] = r.scale;
        }
        auto emit = [&](int i, const V &v) __attribute__((always_inline)) {
            const Pack<int8_t, VN> o = codes(v);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (to[s] >= 0)
                    *(Pack<int8_t, VN> *)(args.Q + to[s] * args.ldq + (int64_t)i * VN) = o;
        };
#pragma unroll
        for (int c = 0; c < CACHE; ++c)
            if (c * NT + tid < nv)
                emit(c * NT + tid, keep[c]);
        for (int i = CACHE * NT + tid; i < nv; i += NT)
            emit(i, *(const V *)(x + (int64_t)i * VN));
        for (int i = nv * VN + tid; i < H; i += NT) {
            const int8_t o = (int8_t)code(x[i]);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (to[s] >= 0)
                    args.Q[to[s] * args.ldq + i] = o;
        }
    }
}

// The inverse of the order for quantize_rows<.., TOKENS>.  A row of Q whose
// pair stands in `order` again is coded here, by one thread.
template <int XT>
__global__ void __launch_bounds__(256)
quantize_invert(QuantArgs args, int32_t *inverse)
{
    typedef typename ElemOf<XT>::type E;
    const int64_t p = wg_number() * 256 + threadIdx.x;
    if (p >= args.R)
        return;
    invert_one(args.order, inverse, p, (int64_t)args.T * args.top_k, [&](int pair, int old) {
        const E *const x = (const E *)args.X + (int64_t)(pair / args.top_k) * args.ldx;
        uint32_t top = 0;
        for (int i = 0; i < args.H; ++i) {
            const uint32_t b = __builtin_bit_cast(uint32_t, (float)x[i]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
        const RowScale r(top);
        args.scale[old] = r.scale;
        for (int i = 0; i < args.H; ++i)
            args.Q[old * args.ldq + i] = (int8_t)r.code<XT>((float)x[i]);
    });
}

// ---------------------------------------------------------------------------
// The order of pairs by expert
// ---------------------------------------------------------------------------
// A stable counting sort of `pairs` expert ids into experts 0 .. E-1; ids
// outside are class E, behind the last expert.  order[p] = pair at sorted
// position p (-1 behind the last expert), position[pair] = p (-1: no expert),
// offsets[e] = first position of expert e.
//
// One workgroup sorts up to 4096 pairs (256 pairs over 64 experts 3.2 us);
// more take two launches (131072 pairs over 128 experts 4.7 + 11.3 us: the
// first counts, and every workgroup of the second adds up the counts before it).
// Each wave owns consecutive pairs and a row of counters in LDS, so equal
// experts keep their order without atomics whose order matters: within 64
// pairs the lanes of one expert are found by ballots over the id's bits, and
// the counts before a lane are its rank.
struct RouteArgs {
    const void *ids;
    int32_t *order, *position, *offsets;
    int32_t *hist;      // [blocks][E + 1] counts (several blocks)
    int32_t pairs, E, bits;
    int32_t per_wave;   // pairs per wave, a multiple of 64
};

constexpr int kRouteWaves = 4;
constexpr int kRouteThreads = 64 * kRouteWaves;

template <int WIDE>
__device__ __forceinline__ int expert_of(const RouteArgs &a, int i)
{
    if constexpr (WIDE != 0) {
        const int64_t e = ((const int64_t *)a.ids)[i];
        return e >= 0 && e < a.E ? (int)e : a.E;
    } else {
        const int32_t e = ((const int32_t *)a.ids)[i];
        return e >= 0 && e < a.E ? e : a.E;
    }
}

// Up to kRouteRun pairs of a wave's at a time, their experts loaded together.
constexpr int kRouteRun = 8;

template <int WIDE>
__device__ __forceinline__ void load_experts(const RouteArgs &a, int i0, int last, int lane, int (&e)[kRouteRun])
{
#pragma unroll
    for (int r = 0; r < kRouteRun; ++r) {
        const int i = i0 + 64 * r + lane;
        e[r] = i < last ? expert_of<WIDE>(a, i) : -1;
    }
}

// Counts of one wave's pairs into its LDS row (zeroed here).
template <int WIDE>
__device__ __forceinline__ void route_count(const RouteArgs &a, int32_t *cnt, int first, int last, int lane)
{
    for (int e = lane; e <= a.E; e += 64)
        cnt[e] = 0;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    for (int i0 = first; i0 < last; i0 += 64 * kRouteRun) {
        int e[kRouteRun];
        load_experts<WIDE>(a, i0, last, lane, e);
#pragma unroll
        for (int r = 0; r < kRouteRun; ++r)
            if (e[r] >= 0)
                atomicAdd(&cnt[e[r]], 1);
    }
}

// Positions of one wave's pairs, from the counters at their first positions.
template <int WIDE>
__device__ __forceinline__ void route_place(const RouteArgs &a, int32_t *cnt, int first, int last, int lane)
{
    for (int i0 = first; i0 < last; i0 += 64 * kRouteRun) {
        int ex[kRouteRun];
        load_experts<WIDE>(a, i0, last, lane, ex);
#pragma unroll
        for (int r = 0; r < kRouteRun; ++r) {
            const int i = i0 + 64 * r + lane;
            const int e = ex[r];
            const bool ok = e >= 0;
            uint64_t same = __ballot(ok);
            if (same == 0)
                break;
            for (int b = 0; b < a.bits; ++b) {
                const uint64_t set = __ballot((e >> b) & 1);
                same &= ((e >> b) & 1) ? set : ~set;
            }
            const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
            int base = 0;
            if (ok && rank == 0)
                base = atomicAdd(&cnt[e], __builtin_popcountll(same));
            base = __shfl(base, ok ? __builtin_ctzll(same) : lane);
            if (ok) {
                const int p = base + rank;
                a.order[p] = e < a.E ? i : -1;
                a.position[i] = e < a.E ? p : -1;
            }
        }
    }
}

// Exclusive prefix sum over the E + 1 values of `v` in LDS, by one workgroup
// of kRouteThreads (each thread a run of consecutive values).
__device__ __forceinline__ void route_scan(int32_t *v, int count, int32_t *sums)
{
    const int t = threadIdx.x;
    const int per = (count + kRouteThreads - 1) / kRouteThreads;
    const int lo = t * per < count ? t * per : count;
    const int hi = lo + per < count ? lo + per : count;
    int total = 0;
    for (int i = lo; i < hi; ++i)
        total += v[i];
    int incl = total;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(incl, d);
        if ((t & 63) >= d)
            incl += o;
    }
    if ((t & 63) == 63)
        sums[t / 64] = incl;
    __syncthreads();
    int before = incl - total;
    for (int w = 0; w < t / 64; ++w)
        before += sums[w];
    for (int i = lo; i < hi; ++i) {
        const int x = v[i];
        v[i] = before;
        before += x;
    }
    __syncthreads();
}

extern __shared__ int32_t route_lds[];

// Few pairs: the whole sort by one workgroup.
template <int WIDE>
__global__ void __launch_bounds__(kRouteThreads)
route_one(RouteArgs a)
{
    int32_t *const cnt = route_lds;                          // [waves][E + 1]
    int32_t *const first = cnt + kRouteWaves * (a.E + 1);    // [E + 1]
    int32_t *const sums = first + a.E + 1;                   // [waves]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lo = min(wave * a.per_wave, a.pairs), hi = min(lo + a.per_wave, a.pairs);
    route_count<WIDE>(a, cnt + wave * (a.E + 1), lo, hi, lane);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) {
        int total = 0;
        for (int w = 0; w < kRouteWaves; ++w)
            total += cnt[w * (a.E + 1) + e];
        first[e] = total;
    }
    __syncthreads();
    route_scan(first, a.E + 1, sums);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) {
        int at = first[e];
        a.offsets[e] = at;
        for (int w = 0; w < kRouteWaves; ++w) {
            const int n = cnt[w * (a.E + 1) + e];
            cnt[w * (a.E + 1) + e] = at;
            at += n;
        }
    }
    __syncthreads();
    route_place<WIDE>(a, cnt + wave * (a.E + 1), lo, hi, lane);
}

// Many pairs, first launch: each workgroup's counts per expert.
template <int WIDE>
__global__ void __launch_bounds__(kRouteThreads)
route_hist(RouteArgs a)
{
    int32_t *const cnt = route_lds;  // [E + 1]
    const int lo = min((int64_t)blockIdx.x * kRouteWaves * a.per_wave, (int64_t)a.pairs);
    const int hi = min((int64_t)lo + kRouteWaves * a.per_wave, (int64_t)a.pairs);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads)
        cnt[e] = 0;
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += kRouteThreads)
        atomicAdd(&cnt[expert_of<WIDE>(a, i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads)
        a.hist[(int64_t)blockIdx.x * (a.E + 1) + e] = cnt[e];
}

// Second launch: every workgroup sums the counts of all and of those before
// it, and places its pairs.
template <int WIDE>
__global__ void __launch_bounds__(kRouteThreads)
route_place_blocks(RouteArgs a)
{
    int32_t *const cnt = route_lds;                          // [waves][E + 1]
    int32_t *const first = cnt + kRouteWaves * (a.E + 1);    // [E + 1]
    int32_t *const sums = first + a.E + 1;                   // [waves]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t begin = ((int64_t)blockIdx.x * kRouteWaves + wave) * a.per_wave;
    const int lo = (int)min(begin, (int64_t)a.pairs), hi = (int)min(begin + a.per_wave, (int64_t)a.pairs);
    route_count<WIDE>(a, cnt + wave * (a.E + 1), lo, hi, lane);
    int before[8];  // this thread's experts' counts in the blocks before (E + 1 <= 8 * threads)
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        const int e = s * kRouteThreads + threadIdx.x;
        before[s] = 0;
        if (e <= a.E) {
            int total = 0;
#pragma unroll 16
            for (int b = 0; b < (int)gridDim.x; ++b) {
                const int n = a.hist[(int64_t)b * (a.E + 1) + e];
                total += n;
                before[s] += b < (int)blockIdx.x ? n : 0;
            }
            first[e] = total;
        }
    }
    __syncthreads();
    route_scan(first, a.E + 1, sums);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        const int e = s * kRouteThreads + threadIdx.x;
        if (e <= a.E) {
            int at = first[e];
            if (blockIdx.x == 0)
                a.offsets[e] = at;
            at += before[s];
            for (int w = 0; w < kRouteWaves; ++w) {
                const int n = cnt[w * (a.E + 1) + e];
                cnt[w * (a.E + 1) + e] = at;
                at += n;
            }
        }
    }
    __syncthreads();
    route_place<WIDE>(a, cnt + wave * (a.E + 1), lo, hi, lane);
}

// No pairs: every expert starts at 0.
__global__ void __launch_bounds__(kRouteThreads)
route_none(int32_t *offsets, int E)
{
    for (int e = threadIdx.x; e <= E; e += kRouteThreads)
        offsets[e] = 0;
}

// ---------------------------------------------------------------------------
// Rows into expert order, and back
// ---------------------------------------------------------------------------
struct GatherArgs {
    const uint8_t *X;
    uint8_t *Y;
    const int32_t *order;
    int64_t ldx, ldy;        // bytes
    int32_t T, R, top_k;
    int32_t row_bytes;
};

// Y[p] = X[order[p] / top_k]: LANES lanes per row (64, or 16 for short rows).
template <int LANES>
__global__ void __launch_bounds__(256)
gather_rows(GatherArgs a)
{
    const int lane = threadIdx.x % LANES;
    const int sub = threadIdx.x / LANES;
    const int64_t p = wg_number() * (256 / LANES) + (LANES == 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
    if (p >= a.R)
        return;
    const int pair = a.order[p];
    const int t = pair < 0 ? -1 : pair / a.top_k;
    if (t < 0 || t >= a.T)
        return;
    const uint8_t *const x = a.X + (int64_t)t * a.ldx;
    uint8_t *const y = a.Y + p * a.ldy;
    const int nv = a.row_bytes / 16;
    // 4 vectors a lane at a time: the loads first, so that they are in flight
    // together
    for (int i0 = lane; i0 < nv; i0 += 4 * LANES) {
        u32x4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (i0 + LANES * c < nv)
                v[c] = *(const u32x4_any *)(x + (int64_t)(i0 + LANES * c) * 16);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (i0 + LANES * c < nv)
                *(u32x4_any *)(y + (int64_t)(i0 + LANES * c) * 16) = v[c];
    }
    for (int i = nv * 16 + lane; i < a.row_bytes; i += LANES)
        y[i] = x[i];
}

__global__ void __launch_bounds__(256)
gather_invert(GatherArgs a, int32_t *inverse)
{
    const int64_t p = wg_number() * 256 + threadIdx.x;
    if (p >= a.R)
        return;
    invert_one(a.order, inverse, p, (int64_t)a.T * a.top_k, [&](int pair, int old) {
        const uint8_t *const x = a.X + (int64_t)(pair / a.top_k) * a.ldx;
        uint8_t *const y = a.Y + (int64_t)old * a.ldy;
        for (int i = 0; i < a.row_bytes; ++i)
            y[i] = x[i];
    });
}

// Many rows: each token's row is read once and written to the rows of its
// pairs (131072 BF16 rows of 2048 from 16384 tokens 104 us, 5.8 TB/s; by rows
// 149).  By rows of Y (gather_rows) the reads of a token's row lie far apart
// and come from beyond the L2 top_k times.  The stores stream past the caches.
__global__ void __launch_bounds__(256)
gather_tokens(GatherArgs a, const int32_t *inverse)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = wg_number() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const uint8_t *const x = a.X + t * a.ldx;
    const int nv = a.row_bytes / 16;
    for (int i0 = lane; i0 < nv; i0 += 256) {
        u32x4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (i0 + 64 * c < nv)
                v[c] = *(const u32x4_any *)(x + (int64_t)(i0 + 64 * c) * 16);
        for (int s = 0; s < a.top_k; ++s) {
            const int p = inverse[t * a.top_k + s];
            if (p < 0)
                continue;
            uint8_t *const y = a.Y + p * a.ldy;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (i0 + 64 * c < nv)
                    __builtin_nontemporal_store(v[c], (u32x4_any *)(y + (int64_t)(i0 + 64 * c) * 16));
        }
    }
    for (int i = nv * 16 + lane; i < a.row_bytes; i += 64)
        for (int s = 0; s < a.top_k; ++s) {
            const int p = inverse[t * a.top_k + s];
            if (p >= 0)
                a.Y[p * a.ldy + i] = x[i];
        }
}

struct CombineArgs {
    const void *Y;           // R x H, the experts' rows
    void *O;                 // T x H
    const int32_t *position; // T x top_k
    const float *weights;    // T x top_k, or nullptr: ones
    int64_t ldy, ldo;
    int32_t T, H, R, top_k;
};

// O[t] = sum_s weights[t][s] * Y[position[t][s]], in FP32, slots ascending
// (HBM; 33 tokens of 8 slots and 2048 values 3.9 us, a launch and two trips to
// memory); one thread per 16 bytes of a row of Y, LANES threads per token (256
// and as many workgroups as the row needs, or 64 or 16 for short rows).  Four
// slots' rows are loaded before the first is used.
template <int YT, int OT, int LANES>
__global__ void __launch_bounds__(256)
combine_rows(CombineArgs a)
{
    typedef typename ElemOf<YT>::type EY;
    typedef typename ElemOf<OT>::type EO;
    constexpr int VN = VecOf<EY>::N;
    typedef typename VecOf<EY>::type V;
    const int lane = threadIdx.x % LANES;
    const int sub = threadIdx.x / LANES;
    const int64_t t = wg_number() * (256 / LANES) + (LANES == 16 ? sub : __builtin_amdgcn_readfirstlane(sub));
    if (t >= a.T)
        return;
    const int32_t *const at = a.position + t * a.top_k;
    for (int64_t c = (int64_t)VN * (blockIdx.z * LANES + lane); c < a.H; c += (int64_t)VN * LANES * gridDim.z) {
        const int left = (int)(a.H - c);
        float acc[VN];
#pragma unroll
        for (int e = 0; e < VN; ++e)
            acc[e] = 0.0f;
        for (int s0 = 0; s0 < a.top_k; s0 += 4) {
            V v[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = s0 + j < a.top_k ? at[s0 + j] : -1;
                w[j] = 0.0f;
#pragma unroll
                for (int e = 0; e < VN; ++e)
                    v[j].v[e] = (EY)0.0f;
                if (p >= 0 && p < a.R) {
                    w[j] = a.weights ? a.weights[t * a.top_k + s0 + j] : 1.0f;
                    const EY *const y = (const EY *)a.Y + (int64_t)p * a.ldy + c;
                    if (left >= VN) {
                        v[j] = *(const V *)y;
                    } else {
#pragma unroll
                        for (int e = 0; e < VN; ++e)
                            if (e < left)
                                v[j].v[e] = y[e];
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < VN; ++e)
                    acc[e] = __builtin_fmaf(w[j], (float)v[j].v[e], acc[e]);
        }
        i8_store<OT, VN>((EO *)a.O + t * a.ldo + c, 0, left, acc);
    }
}

struct CombineBackArgs {
    const void *dO;          // T x H
    const void *Y;           // R x H, or nullptr with dweights
    void *dY;                // R x H
    float *dweights;         // T x top_k, or nullptr
    const int32_t *position;
    const float *weights;
    int64_t ldo, ldy, lddy;
    int32_t T, H, R, top_k;
};

// Of each pair (t, s) with a position p: dY[p] = weights[t][s] * dO[t] and
// dweights[t][s] = <dO[t], Y[p]>, the products summed in FP32; a pair without
// one has dweights 0.  Bound: HBM (16384 tokens of 4 slots, an eighth without a
// position, 2048 values 156 us, 4.95 TB/s).  LANES lanes per pair (64, or 16 for short rows); the
// slots of a token are neighbours, so dO[t] comes from memory once.
template <int DT, int YT, int GT, int LANES>
__global__ void __launch_bounds__(256)
combine_rows_backward(CombineBackArgs a)
{
    typedef typename ElemOf<DT>::type ED;
    typedef typename ElemOf<YT>::type EY;
    typedef typename ElemOf<GT>::type EG;
    constexpr int VN = 8;
    const int lane = threadIdx.x % LANES;
    const int sub = threadIdx.x / LANES;
    const int64_t pair = wg_number() * (256 / LANES) + (LANES == 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
    if (pair >= (int64_t)a.T * a.top_k)
        return;
    const int p = a.position[pair];
    const bool there = p >= 0 && p < a.R;
    float dot = 0.0f;
    if (there) {
        const float w = a.weights ? a.weights[pair] : 1.0f;
        const ED *const d = (const ED *)a.dO + (pair / a.top_k) * a.ldo;
        const EY *const y = (const EY *)a.Y + (int64_t)p * a.ldy;
        EG *const g = (EG *)a.dY + (int64_t)p * a.lddy;
        const int nv = a.H / VN;
        for (int i = lane; i < nv; i += LANES) {
            const Pack<ED, VN> dv = *(const Pack<ED, VN> *)(d + (int64_t)i * VN);
            Pack<EG, VN> gv;
            if (a.dweights) {
                const Pack<EY, VN> yv = *(const Pack<EY, VN> *)(y + (int64_t)i * VN);
#pragma unroll
                for (int e = 0; e < VN; ++e)
                    dot = __builtin_fmaf((float)dv.v[e], (float)yv.v[e], dot);
            }
#pragma unroll
            for (int e = 0; e < VN; ++e)
                gv.v[e] = (EG)(w * (float)dv.v[e]);
            *(Pack<EG, VN> *)(g + (int64_t)i * VN) = gv;
        }
        for (int i = nv * VN + lane; i < a.H; i += LANES) {
            const float dv = (float)d[i];
            if (a.dweights)
                dot = __builtin_fmaf(dv, (float)y[i], dot);
            g[i] = (EG)(w * dv);
        }
    }
    if (a.dweights) {
        // (lanes of one pair are alike in `there`, and only they add)
#pragma unroll
        for (int s = LANES / 2; s > 0; s /= 2)
            dot += __shfl_xor(dot, s);
        if (lane == 0)
            a.dweights[pair] = dot;
    }
}
