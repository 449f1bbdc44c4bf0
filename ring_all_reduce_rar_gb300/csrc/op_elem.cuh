// op_elem.cuh -- element access and reductions shared by the model
// operators' kernels.  Values are widened to binary32 when read and rounded
// once when written.
#pragma once

#include <cuda_fp8.h>

#include "elem_ops.cuh"

namespace rar {

template <int DT>
__device__ __forceinline__ float widen(uint32_t bits) {
    if constexpr (DT == DT_F32) return __uint_as_float(bits);
    else if constexpr (DT == DT_BF16) return bf16_bits_to_float(bits & 0xFFFFu);
    else return f16_bits_to_float(bits & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ uint32_t narrow(float f) {
    if constexpr (DT == DT_F32) return __float_as_uint(f);
    else if constexpr (DT == DT_BF16) return float_to_bf16_bits(f);
    else return float_to_f16_bits(f);
}
template <int DT>
__device__ __forceinline__ float load_f(const void *base, long long i) {
    return widen<DT>(load_elem<DT>(static_cast<const char *>(base), i));
}
template <int DT>
__device__ __forceinline__ void store_f(void *base, long long i, float f) {
    store_elem<DT>(static_cast<char *>(base), i, narrow<DT>(f));
}

// Two and eight 16-bit values, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (DT == DT_BF16) {
        __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&r);
    } else {
        __half2 r = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&r);
    }
}
template <int DT>
__device__ __forceinline__ uint4 narrow8(const float *v) {
    return make_uint4(narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]), narrow2<DT>(v[6], v[7]));
}

// An index array of 32- or 64-bit signed integers.
__device__ __forceinline__ long long load_index(const void *base, int bytes, long long i) {
    return bytes == 8 ? __ldg(static_cast<const long long *>(base) + i) : (long long)__ldg(static_cast<const int *>(base) + i);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// The scale of a group whose largest magnitude is amax: the e4m3 range
// [-448, 448] spans the group; never 0, infinite or NaN.
__device__ __forceinline__ float scale_of(float amax) {
    constexpr float kInv = 1.0f / 448.0f;
    const float x = fminf(amax, 3.402823466e38f), q = x * kInv;
    // the quotient, rounded once (see CodeOf; one below 2^-126 is not used)
    return fmaxf(fmaf(fmaf(-q, 448.0f, x), kInv, q), 1.175494351e-38f);
}
// Codes of values divided by a scale.  The product with the reciprocal,
// corrected once by its remainder, is the correctly rounded quotient (Markstein
// 1990): the scale and its reciprocal are normal numbers, and where the
// remainder underflows the quotient is far below the smallest code (or the
// scale is 2^-126 and the product exact).  It is inf or NaN where the value is.
struct CodeOf {
    float scale, inv;
    __device__ __forceinline__ explicit CodeOf(float s) {
        scale = s;
        inv = __frcp_rn(s);
    }
    __device__ __forceinline__ float quotient(float v) const {
        const float q = v * inv, r = fmaf(-q, scale, v), c = fmaf(r, inv, q);
        return fabsf(q) <= 512.0f ? c : q;  // (the remainder of an infinity is NaN)
    }
    __device__ __forceinline__ uint8_t one(float v) const {
        return (uint8_t)__nv_cvt_float_to_fp8(quotient(v), __NV_SATFINITE, __NV_E4M3);
    }
    __device__ __forceinline__ uint32_t four(const float *v) const {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(quotient(v[0]), quotient(v[1])), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(quotient(v[2]), quotient(v[3])), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
};

// The codes of 4 or 8 values, in one store.
__device__ __forceinline__ void store_codes(uint8_t *to, const float (&v)[4], float scale) {
    *reinterpret_cast<uint32_t *>(to) = CodeOf(scale).four(v);
}
__device__ __forceinline__ void store_codes(uint8_t *to, const float (&v)[8], float scale) {
    const CodeOf c(scale);
    *reinterpret_cast<uint2 *>(to) = make_uint2(c.four(v), c.four(v + 4));
}

// A 16-byte vector of a row as it was read: VE elements, widened where they
// are used, so that a load in flight takes 4 registers.
template <int DT>
struct RowBits {
    static constexpr int VE = 16 / ElemInfo<DT>::bytes;
    uint32_t w[4];
    // (coherent: where a call works in place the row is written later, and the read-only path is
    // for what no thread writes while the kernel runs)
    __device__ __forceinline__ void load(const void *row, int vec, bool has) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (has) q = static_cast<const uint4 *>(row)[vec];
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (DT == DT_F32) return __uint_as_float(w[e]);
        else if constexpr (DT == DT_BF16) return __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        else return widen<DT>(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
    }
};
// s += the vector, element by element; two elements an instruction.
template <int DT>
__device__ __forceinline__ void add_vec(float (&s)[RowBits<DT>::VE], const RowBits<DT> &b) {
#pragma unroll
    for (int e = 0; e < RowBits<DT>::VE; e += 2)
        asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
            : "+f"(s[e]), "+f"(s[e + 1])
            : "f"(b.get(e)), "f"(b.get(e + 1)));
}
template <int DT>
__device__ __forceinline__ void store_vec(void *row, int vec, const float *f) {
    uint4 q;
    if constexpr (DT == DT_F32) q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else q = narrow8<DT>(f);
    static_cast<uint4 *>(row)[vec] = q;
}
// A row of `dim` elements in 16-byte vectors.  ODD: the row begins anywhere in
// one; its elements are [lo, lo + dim) from that vector's first, and the vectors
// at its ends are accessed by the elements that belong to the row.
template <int DT, bool ODD>
struct RowView {
    static constexpr int VE = RowBits<DT>::VE, EB = ElemInfo<DT>::bytes;
    int lo, hi;  // lo 0 and hi a multiple of VE unless ODD; hi 0: no row
    __device__ __forceinline__ bool has(int vec) const { return vec * VE < hi; }
    __device__ __forceinline__ bool has(int vec, int e) const { return !ODD ? has(vec) : vec * VE + e >= lo && vec * VE + e < hi; }
    __device__ __forceinline__ bool whole(int vec) const { return !ODD ? has(vec) : vec * VE >= lo && vec * VE + VE <= hi; }
    // the row's element that element e of a vector is
    __device__ __forceinline__ int column(int vec, int e) const { return vec * VE + e - lo; }
    __device__ __forceinline__ void load_elems(const char *row, int vec, RowBits<DT> &b) const {
        b.w[0] = b.w[1] = b.w[2] = b.w[3] = 0u;
#pragma unroll
        for (int e = 0; e < VE; e++)
            if (has(vec, e)) {
                const uint32_t x = load_elem<DT>(row, column(vec, e));
                if (VE == 4) b.w[e] = x;
                else b.w[e / 2] |= e % 2 ? x << 16 : x;
            }
    }
    __device__ __forceinline__ void load(const char *row, int vec, RowBits<DT> &b) const {
        if (!ODD || whole(vec)) b.load(row - lo * EB, vec, has(vec));
        else load_elems(row, vec, b);
    }
    // of one vector of columns (weight), which has no part in the row's alignment
    __device__ __forceinline__ void load_columns(const void *v, int vec, RowBits<DT> &b) const {
        if (!ODD) b.load(v, vec, has(vec));
        else load_elems(static_cast<const char *>(v), vec, b);
    }
    __device__ __forceinline__ void store(char *row, int vec, const float *f) const {
        if (whole(vec)) {
            store_vec<DT>(row - lo * EB, vec, f);
        } else if (ODD) {
#pragma unroll
            for (int e = 0; e < VE; e++)
                if (has(vec, e)) store_f<DT>(row, column(vec, e), f[e]);
        }
    }
};
// chunk_of with 32-bit divisions where the buffer allows them.
struct Chunks {
    long long base, extra;
    bool small;
    __device__ __forceinline__ Chunks(long long n, int p) : small(n < 0x7FFFFFFF) {
        if (small) base = (uint32_t)n / (uint32_t)p, extra = (uint32_t)n % (uint32_t)p;
        else base = n / p, extra = n % p;
    }
    __device__ __forceinline__ int of(long long i) const {
        if (!small) return chunk_of(i, base, extra);
        const uint32_t b = (uint32_t)base, x = (uint32_t)extra, big = x * (b + 1), k = (uint32_t)i;
        return (int)(k < big ? k / (b + 1) : x + (k - big) / b);
    }
};

// Calls f(IntC<dtype>{}) for a floating dtype.
template <typename F>
cudaError_t dispatch_float(int dtype, F &&f) {
    switch (dtype) {
    case DT_F32: return f(IntC<DT_F32>{});
    case DT_BF16: return f(IntC<DT_BF16>{});
    case DT_F16: return f(IntC<DT_F16>{});
    }
    return cudaErrorInvalidValue;
}

}  // namespace rar
