// router_kernels.hpp -- the router in front of the experts (gfx950): the top_k
// experts of each token, their use and the loss that evens it, and the gradient
// by the logits.  Included by router.hip in namespace mpg, after elements.hpp.
//
// A token's row of E logits lies in the registers of 16 lanes (four tokens a
// wave; E up to 256, top_k up to 16) or of 64, V neighbouring values a lane.
// All of a row's sums and maxima are FP32 over lanes: four register moves by
// lane rotation, and two exchanges more where 64 lanes have it.

struct RouterArgs {
    const void *logits;
    int64_t ldl;
    int32_t T, E, top_k;
};

// ---- over the LPT lanes of a token ---------------------------------------------
template <int N>
__device__ __forceinline__ uint32_t rotated(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N /* row_ror:N */, 0xF, 0xF, true);
}

// op over the token's lanes, the same in each (op commutes; every lane adds
// up the same pairs).
template <int LPT, class Op>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, Op op)
{
    v = op(v, rotated<8>(v));
    v = op(v, rotated<4>(v));
    v = op(v, rotated<2>(v));
    v = op(v, rotated<1>(v));
    if constexpr (LPT == 64) {
        v = op(v, (uint32_t)__shfl_xor((int)v, 16));
        v = op(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}

template <int LPT>
__device__ __forceinline__ uint32_t most_of(uint32_t v)
{
    return over_lanes<LPT>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int LPT>
__device__ __forceinline__ float sum_of(float v)
{
    return __builtin_bit_cast(float, over_lanes<LPT>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}

// ---- logits --------------------------------------------------------------------
// Whole numbers in the order of the logits: 0 for -inf (no expert), above
// kInfKey for a NaN; -0 and 0 are equal.
constexpr uint32_t kInfKey = 0xFF800000u;

__device__ __forceinline__ uint32_t key_of(float x)
{
    x += 0.0f;
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u)
        return 0xFFFFFFFFu;
    return b == 0xFF800000u ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __builtin_bit_cast(float, key ^ ((key >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(x) for x <= 0, 0 below the normal numbers: 2^(x / ln 2) by the hardware's
// power of two, with what the rounding of x / ln 2 lost (and the rest of 1/ln 2)
// put back to first order, so that large -x cost no digits.
__device__ __forceinline__ float exp_of(float x)
{
    x = __builtin_fmaxf(x, -150.0f);
    constexpr float hi = 1.44269504088896340736f, lo = (float)(1.44269504088896340736 - (double)hi);
    const float t = x * hi;
    const float rest = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, 0.69314718055994530942f * rest, e);
}

// The V values of a row from `at` on, -inf behind its E.
template <class E, int V>
__device__ __forceinline__ void load_row(const E *row, int at, int count, float (&x)[V])
{
    if (at + V <= count) {
        const Pack<E, V> p = *(const Pack<E, V> *)(row + at);
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = (float)p.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = at + i < count ? (float)row[at + i] : -__builtin_inff();
    }
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A row's largest logit: NaN where the row holds one.
template <int LPT, int V>
__device__ __forceinline__ float top_of(const float (&x)[V])
{
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        m = larger(m, x[i]);
    return __builtin_bit_cast(float, over_lanes<LPT>(__builtin_bit_cast(uint32_t, m), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, larger(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}

// Has a row with this largest logit probabilities, and are they numbers?
__device__ __forceinline__ bool has_any(float top) { return top != -__builtin_inff(); }
__device__ __forceinline__ bool is_finite_row(float top) { return top < __builtin_inff(); }

// Probabilities of a row from its largest logit: zeros without any expert, NaN
// with a NaN or +inf.
template <int LPT, int V>
__device__ __forceinline__ void softmax(const float (&x)[V], float top, float (&p)[V])
{
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        p[i] = exp_of(x[i] - top);
        sum += p[i];
    }
    sum = sum_of<LPT>(sum);
    // (-inf minus -inf went to exp_of as a NaN and came back as 0)
    const float inv = !has_any(top) ? 0.0f : is_finite_row(top) ? 1.0f / sum : __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < V; ++i)
        p[i] *= inv;
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------
// top_k times: the largest key left over all lanes, the first lane that has it,
// and in that lane its first value; it is taken out.  Every lane learns the
// key, and lane s keeps slot s's; the lane that has the expert writes its id.
// Bound: the rounds' chains of lane moves and compares (16384x128 FP32, 8 slots, 6.7
// us, 1.4 TB/s; 64x64, 4 slots, 2.5: the launch).
template <int LT, int LPT, int V>
__global__ void __launch_bounds__(256)
select_experts(RouterArgs args, int normalize, int32_t *ids, float *weights)
{
    typedef typename ElemOf<LT>::type E;
    const int lane = threadIdx.x % LPT;
    const int base = (threadIdx.x & 63) - lane;       // the token's first lane in the wave
    const int64_t t = wg_number() * (256 / LPT) + threadIdx.x / LPT;
    // (lanes of tokens behind the last go along: the exchanges need the whole wave)
    const bool there = t < args.T;
    float x[V];
    load_row<E, V>((const E *)args.logits + (there ? t : 0) * args.ldl, lane * V, args.E, x);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        key[i] = key_of(x[i]);
    const int k = args.top_k;
    uint32_t first = 0, mine = 0;                     // keys of the first slot and of this lane's
    for (int s = 0; s < k; ++s) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            best = max(best, key[i]);
        const uint32_t top = most_of<LPT>(best);
        first = s == 0 ? top : first;
        mine = lane == s ? top : mine;
        const uint64_t holders = __ballot(best == top) >> base;
        const bool winner = (int)__builtin_ctzll(holders) == lane;
        int at = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            at = key[i] == top ? i : at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = winner && i == at ? 0u : key[i];
        if (winner && there)
            ids[t * k + s] = top == 0 ? -1 : lane * V + at;
    }
    const float m = logit_of(first);
    const float e = mine == 0 ? 0.0f : exp_of(logit_of(mine) - m);
    float sum;
    if (normalize) {
        sum = sum_of<LPT>(e);
    } else {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            sum += exp_of(x[i] - m);
        sum = sum_of<LPT>(sum);
    }
    if (there && lane < k)
        weights[t * k + lane] = mine == 0 ? 0.0f : first >= kInfKey ? __builtin_nanf("") : e / sum;
}

// ---------------------------------------------------------------------------
// Use of the experts
// ---------------------------------------------------------------------------
struct BalanceArgs {
    RouterArgs r;
    const void *ids;
    float coefficient;
    float *loss, *probs;
    int32_t *counts;
    // workspace: per block E sums of probabilities, E + 1 counts; then a word
    // that counts finished blocks of the second launch, and per such block its
    // share of sum counts * probs, of pairs and of tokens
    uint32_t *ws;
    int32_t blocks, per_block;     // of the first launch; tokens of each
};

// Experts one block of the second launch adds up.
constexpr int kBalanceExperts = 16;

// First launch: each block adds up the probabilities of its tokens, a lane
// always those of the same experts, and counts its pairs in LDS.  Bound: memory
// latency and the exponentials (32768x256 BF16 with 8 slots 9-10 us, 1.8 TB/s).
template <int LT, int LPT, int V, int WIDE>
__global__ void __launch_bounds__(256)
balance_tokens(BalanceArgs args)
{
    typedef typename ElemOf<LT>::type E;
    constexpr int TOKENS = 256 / LPT;                  // at a time
    extern __shared__ uint32_t balance_lds[];          // counts: E + 1; sums: 4 waves x LPT*V
    int32_t *const cnt = (int32_t *)balance_lds;
    float *const part = (float *)(balance_lds + args.r.E + 1);
    const int lane = threadIdx.x % LPT;
    const int n = args.r.E;
    for (int e = threadIdx.x; e <= n; e += 256)
        cnt[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        args.ws[(int64_t)args.blocks * (2 * n + 1)] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * args.per_block;
    const int64_t t1 = t0 + args.per_block < args.r.T ? t0 + args.per_block : args.r.T;
    const int64_t p1 = t1 * args.r.top_k;
    for (int64_t i = t0 * args.r.top_k + threadIdx.x; i < p1; i += 256) {
        int e;
        if constexpr (WIDE != 0) {
            const int64_t id = ((const int64_t *)args.ids)[i];
            e = id >= 0 && id < n ? (int)id : -1;
        } else {
            e = ((const int32_t *)args.ids)[i];
        }
        if (e >= 0 && e < n)
            atomicAdd(&cnt[e], 1);
    }
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum[i] = 0.0f;
    int tokens = 0;
    // (lanes of tokens behind the last read the block's first and add nothing)
    const E *const logits = (const E *)args.r.logits;
    float x[V], next[V];
    const int64_t mine = t0 + threadIdx.x / LPT;
    if (t0 < t1)
        load_row<E, V>(logits + (mine < t1 ? mine : t0) * args.r.ldl, lane * V, n, x);
    for (int64_t t = mine, first = t0; first < t1; t += TOKENS, first += TOKENS) {
        if (first + TOKENS < t1)
            load_row<E, V>(logits + (t + TOKENS < t1 ? t + TOKENS : t0) * args.r.ldl, lane * V, n, next);
        const float top = top_of<LPT, V>(x);
        float p[V];
        softmax<LPT, V>(x, top, p);
        if (t < t1) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum[i] += p[i];
            tokens += lane == 0 && has_any(top);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = next[i];
    }
    if (tokens != 0)
        atomicAdd(&cnt[n], tokens);
    // the wave's tokens, then the waves' in order
    if constexpr (LPT == 16) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sum[i] += __shfl_xor(sum[i], 16);
            sum[i] += __shfl_xor(sum[i], 32);
        }
    }
    if ((threadIdx.x & 63) < LPT)
#pragma unroll
        for (int i = 0; i < V; ++i)
            part[(threadIdx.x >> 6) * LPT * V + lane * V + i] = sum[i];
    __syncthreads();
    uint32_t *const out = args.ws + (int64_t)blockIdx.x * (2 * n + 1);
    for (int e = threadIdx.x; e <= n; e += 256) {
        if (e < n)
            out[e] = __builtin_bit_cast(uint32_t, part[e] + part[LPT * V + e] + part[2 * LPT * V + e] +
                                                      part[3 * LPT * V + e]);
        out[n + e] = (uint32_t)cnt[e];
    }
}

// Second launch: a block adds up its experts over the first launch's blocks (64
// threads each, in a fixed order), and the last block to finish the loss.  Bound:
// two trips to memory and the count of blocks (512 blocks' sums of 256 experts 6.5
// us; one block, 13 experts, 2.1).
__global__ void __launch_bounds__(1024)
balance_sum(BalanceArgs args)
{
    constexpr int SLICES = 1024 / kBalanceExperts;
    const int n = args.r.E, words = 2 * n + 1;
    // threads 0..15 of a row of 16 have expert `e`'s neighbours: loads of one
    // block's words side by side
    const int col = threadIdx.x % kBalanceExperts, slice = threadIdx.x / kBalanceExperts;
    const int e = blockIdx.x * kBalanceExperts + col;
    __shared__ float psum[16][kBalanceExperts];
    __shared__ int32_t csum[16][kBalanceExperts];
    float p = 0.0f;
    int32_t c = 0;
    if (e <= n) {
#pragma unroll 8
        for (int b = slice; b < args.blocks; b += SLICES) {
            const uint32_t *const w = args.ws + (int64_t)b * words;
            if (e < n)
                p += __builtin_bit_cast(float, w[e]);
            c += (int32_t)w[n + e];
        }
    }
    // a wave's four threads of an expert, then the waves in order
    p += __shfl_xor(p, 16);
    p += __shfl_xor(p, 32);
    c += __shfl_xor(c, 16);
    c += __shfl_xor(c, 32);
    if ((threadIdx.x & 63) < kBalanceExperts) {
        psum[threadIdx.x >> 6][col] = p;
        csum[threadIdx.x >> 6][col] = c;
    }
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    p = 0.0f;
    c = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        p += psum[w][col];
        c += csum[w][col];
    }
    const bool mine = threadIdx.x < kBalanceExperts;
    if (mine && e <= n)
        args.counts[e] = c;
    if (mine && e < n && args.probs)
        args.probs[e] = p;
    float a = mine && e < n ? (float)c * p : 0.0f;
    int32_t b = mine && e < n ? c : 0;
    int32_t tokens = mine && e == n ? c : 0;
    auto add_up = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            a += __shfl_xor(a, d);
            b += __shfl_xor(b, d);
            tokens += __shfl_xor(tokens, d);
        }
    };
    add_up();
    if (gridDim.x > 1) {
        uint32_t *const done = args.ws + (int64_t)args.blocks * words;
        uint32_t *const share = done + 1;              // per block: sum, pairs, tokens
        bool last = false;
        if (threadIdx.x == 0) {
            share[3 * blockIdx.x] = __builtin_bit_cast(uint32_t, a);
            share[3 * blockIdx.x + 1] = (uint32_t)b;
            share[3 * blockIdx.x + 2] = (uint32_t)tokens;
            __threadfence();
            last = atomicAdd(done, 1u) == gridDim.x - 1;
        }
        if (__ballot(last) == 0)
            return;
        __threadfence();
        a = 0.0f;
        b = 0;
        tokens = 0;
        for (unsigned i = threadIdx.x; i < gridDim.x; i += 64) {
            a += __builtin_bit_cast(float, __hip_atomic_load(&share[3 * i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            b += (int32_t)__hip_atomic_load(&share[3 * i + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            tokens += (int32_t)__hip_atomic_load(&share[3 * i + 2], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        add_up();
    }
    if (threadIdx.x == 0)
        *args.loss = b == 0 || tokens == 0 ? 0.0f
                                           : args.coefficient * (float)n * a / ((float)b * (float)tokens);
}

// ---------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------
struct RouterBackArgs {
    RouterArgs r;
    const void *ids;
    const float *dweights;       // or nullptr
    const int32_t *counts;       // or nullptr
    const float *dloss;          // or nullptr: 1
    float coefficient;
    int32_t normalize;
    void *dlogits;
    int64_t ldd;
};

// A token's slots are its first top_k lanes.  Their parts reach the lanes that
// have their experts through a row of LDS of the token's own (value i of lane l
// at i*LPT + l, so that a wave's accesses spread over the banks): put there, read
// by all, and cleared again.  Slots of one expert are added up first, in slot
// order, by the first of them, so nothing depends on the order of stores; they
// are found by what is left of their lane numbers in that row.  One wave's LDS
// operations happen in order; the fences keep the compiler to it.
// Bound: vector work and memory (32768x256 BF16 with 8 slots and the loss 13 us,
// 2.7 TB/s; 16384x128 FP32 normalised 5.3 us, 3.2 TB/s).
template <int LT, int DT, int LPT, int V, int WIDE>
__global__ void __launch_bounds__(256)
router_backward(RouterBackArgs args)
{
    typedef typename ElemOf<LT>::type E;
    typedef typename ElemOf<DT>::type D;
    constexpr int TOKENS = 256 / LPT;
    __shared__ float rows[TOKENS][LPT * V];
    const int lane = threadIdx.x % LPT;
    const int n = args.r.E, k = args.dweights ? args.r.top_k : 0;
    float *const row = rows[threadIdx.x / LPT];
    auto fence = []() __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    // the loss's pull on each of this lane's experts
    float pull[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        pull[i] = 0.0f;
    if (args.counts) {
        float mine = 0.0f, c[V];
        if (lane * V + V <= n) {
            const Pack<int32_t, V> w = *(const Pack<int32_t, V> *)(args.counts + lane * V);
#pragma unroll
            for (int i = 0; i < V; ++i)
                c[i] = (float)w.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                c[i] = lane * V + i < n ? (float)args.counts[lane * V + i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            mine += c[i];
        const float pairs = sum_of<LPT>(mine), tokens = (float)args.counts[n];
        const float g = (args.dloss ? *args.dloss : 1.0f) * args.coefficient * (float)n;
        const float unit = pairs > 0.0f && tokens > 0.0f ? g / (pairs * tokens) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            pull[i] = unit * c[i];
    }
    const bool by_prob = args.counts != nullptr || !args.normalize;
    if (k > 0)
#pragma unroll
        for (int i = 0; i < V; ++i)
            row[i * LPT + lane] = 0.0f;
    // (lanes of tokens behind the last go along with the block's first token)
    const int64_t stride = (int64_t)gridDim.x * TOKENS;
    float next[V], next_dw = 0.0f;
    int64_t next_id = -1;
    auto load = [&](int64_t first) __attribute__((always_inline)) {
        const int64_t t = first + threadIdx.x / LPT, src = t < args.r.T ? t : first;
        load_row<E, V>((const E *)args.r.logits + src * args.r.ldl, lane * V, n, next);
        if (lane < k) {
            const int64_t i = src * k + lane;
            if constexpr (WIDE != 0)
                next_id = ((const int64_t *)args.ids)[i];
            else
                next_id = ((const int32_t *)args.ids)[i];
            next_dw = args.dweights[i];
        }
    };
    const int64_t start = (int64_t)blockIdx.x * TOKENS;
    if (start < args.r.T)
        load(start);
    for (int64_t first = start; first < args.r.T; first += stride) {
        const int64_t t = first + threadIdx.x / LPT;
        const bool there = t < args.r.T;
        const int64_t src = there ? t : first;
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = next[i];
        const int id = next_id >= 0 && next_id < n ? (int)next_id : -1;
        const float dw = id >= 0 ? next_dw : 0.0f;
        if (first + stride < args.r.T)
            load(first + stride);
        const float top = top_of<LPT, V>(x);
        float z[V];              // the slots' parts
#pragma unroll
        for (int i = 0; i < V; ++i)
            z[i] = 0.0f;
        if (k > 0) {
            float part = dw;
            if (args.normalize) {
                const float l = id >= 0 ? (float)((const E *)args.r.logits)[src * args.r.ldl + id] : -__builtin_inff();
                const uint32_t key = key_of(l), best = most_of<LPT>(key);
                float w = key == 0 ? 0.0f : exp_of(l - logit_of(best));
                const float sum = sum_of<LPT>(w);
                w = key == 0 ? 0.0f : best >= kInfKey ? __builtin_nanf("") : w / sum;
                // (a pair of an expert at -inf has no part: its 0 would meet what dw holds)
                const float mean = sum_of<LPT>(key == 0 ? 0.0f : w * dw);
                part = key == 0 ? 0.0f : w * (dw - mean);
            }
            float *const place = row + id % V * LPT + id / V;
            float total = part;
            bool is_first = id >= 0;
            fence();
            if (id >= 0)
                *place = (float)lane;
            fence();
            if (__ballot(id >= 0 && *place != (float)lane) != 0) {
                // some token has an expert in several slots
                total = 0.0f;
                for (int s = 0; s < k; ++s) {
                    const int other = __shfl(id, s, LPT);
                    const float v = __shfl(part, s, LPT);
                    if (other == id) {
                        total += v;
                        is_first = is_first && s >= lane;
                    }
                }
            }
            fence();
            if (is_first)
                *place = total;
            fence();
#pragma unroll
            for (int i = 0; i < V; ++i)
                z[i] = row[i * LPT + lane];
            if (!args.normalize)
                // (nor has one here: 32768x256 BF16 with 8 slots 10.6 us, without this 10.4)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    z[i] = x[i] == -__builtin_inff() ? 0.0f : z[i];
            fence();
            if (id >= 0)
                *place = 0.0f;
        }
        float out[V];
        if (by_prob) {
            float p[V];
            softmax<LPT, V>(x, top, p);
            float u[V], mean = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[i] = args.normalize ? pull[i] : pull[i] + z[i];
                mean += p[i] * u[i];
            }
            mean = sum_of<LPT>(mean);
#pragma unroll
            for (int i = 0; i < V; ++i)
                out[i] = p[i] * (u[i] - mean) + (args.normalize ? z[i] : 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                out[i] = has_any(top) && !is_finite_row(top) ? __builtin_nanf("") : z[i];
        }
        if (!there)
            continue;
        D *const to = (D *)args.dlogits + t * args.ldd;
        if (lane * V + V <= n) {
            Pack<D, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i)
                o.v[i] = (D)out[i];
            *(Pack<D, V> *)(to + lane * V) = o;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < n)
                    to[lane * V + i] = (D)out[i];
        }
    }
}
