// elements.hpp -- element types and vectors of the operators' kernels, and the
// number of a workgroup.  Included in kernels.hpp's namespace, after it.
#ifndef MPGEMM_ELEMENTS_HPP
#define MPGEMM_ELEMENTS_HPP

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

// Rows are read and written in vectors of 16 bytes at any element alignment.
template <class E>
struct VecOf {
    static constexpr int N = 16 / sizeof(E);
    typedef Pack<E, N> type;
};

// Workgroup number of a launch over x and y (see row_grid): one dimension holds
// fewer than 2^32 threads.
__device__ __forceinline__ int64_t wg_number() { return blockIdx.x + (int64_t)blockIdx.y * gridDim.x; }

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

#endif  // MPGEMM_ELEMENTS_HPP
