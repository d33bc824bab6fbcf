// Pieces shared by the layer kernels (group norm, gated activation, 8-bit
// checkpoints): eight channels of a row at a time, the activations and the
// 8-bit forms.
//
// A thread always works on eight channels of a row, an "oct".  Where every
// row and operand allows it (VEC), they are consecutive and move as 16-byte
// vectors (two for fp32, one 8-byte vector for 8-bit numbers).  Otherwise
// they lie `step` channels apart, so that the `step` neighbouring threads of
// a team read neighbouring elements, and each moves by itself with its
// channel checked against the row's end.  Either way a team covers the same
// 8 * step consecutive channels, so whatever is computed over a team (a
// checkpoint block's largest magnitude) does not depend on the path.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <cstdint>

#include "layers.h"

namespace tsx {
namespace dev {

// Where a thread's oct sits in a row: channels ch, ch + step, ..., those
// under `cols` exist.  VEC: step 1, and all eight exist or none.
struct OctAt {
    int ch;
    int step;
    int cols;
};

template <bool VEC>
__device__ __forceinline__ OctAt oct_at(int v, int team, int cols)
{
    OctAt o;
    o.cols = cols;
    if constexpr (VEC) {
        o.ch = v * 8;
        o.step = 1;
    } else {
        o.ch = (v & ~(team - 1)) * 8 + (v & (team - 1));   // a power of two
        o.step = team;
    }
    return o;
}

// Eight elements as they lie in memory.
template <int DT>
struct Oct {
    uint32_t w[DT == TSX_F32 ? 8 : 4];
};

template <int DT>
__device__ __forceinline__ void oct_zero(Oct<DT>& o)
{
#pragma unroll
    for (int i = 0; i < int(sizeof(o.w) / 4); ++i)
        o.w[i] = 0;
}

// Address of an oct's first element; rows are `pitch` elements apart.
template <int DT>
__device__ __forceinline__ const char* oct_ptr(const void* base, int64_t row, int64_t pitch, int ch)
{
    return static_cast<const char*>(base) + (row * pitch + ch) * elem_size(DT);
}
template <int DT>
__device__ __forceinline__ char* oct_ptr(void* base, int64_t row, int64_t pitch, int ch)
{
    return static_cast<char*>(base) + (row * pitch + ch) * elem_size(DT);
}

// An fp32 oct is 32 bytes, which move at once where they are aligned to that:
// in two halves every sector is asked for twice (tensors are only sure to be
// aligned to 16).
__device__ __forceinline__ bool whole_sector(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// The vector loads go past L1.  They are no read-only-cache loads, since an
// output may be one of the inputs; every thread loads what it overwrites
// before it stores.  The compiler keeps that order: vectors are loaded and
// stored by volatile assembly, single elements through pointers of one type.
template <int DT, bool VEC>
__device__ __forceinline__ Oct<DT> oct_load(const char* p, const OctAt& at)
{
    Oct<DT> o;
    if constexpr (VEC) {
        if constexpr (DT == TSX_F32) {
            if (whole_sector(p)) {
                asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(o.w[0]), "=r"(o.w[1]), "=r"(o.w[2]), "=r"(o.w[3]), "=r"(o.w[4]), "=r"(o.w[5]),
                               "=r"(o.w[6]), "=r"(o.w[7])
                             : "l"(p));
                return o;
            }
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(o.w[4]), "=r"(o.w[5]), "=r"(o.w[6]), "=r"(o.w[7])
                         : "l"(p + 16));
        }
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(o.w[0]), "=r"(o.w[1]), "=r"(o.w[2]), "=r"(o.w[3])
                     : "l"(p));
    } else if constexpr (DT == TSX_F32) {
        const uint32_t* e = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o.w[j] = at.ch + j * at.step < at.cols ? e[j * at.step] : 0u;
    } else {
        const unsigned short* e = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = at.ch + 2 * j * at.step < at.cols ? e[2 * j * at.step] : 0;
            const uint32_t hi = at.ch + (2 * j + 1) * at.step < at.cols ? e[(2 * j + 1) * at.step] : 0;
            o.w[j] = lo | hi << 16;
        }
    }
    return o;
}

// An oct's fp32 values as four pairs: arithmetic on them is two elements to an
// instruction (fma.rn.f32x2 and its kin), with the rounding of the scalar ones.
__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

// A sum that does not become one fma with the paired product before it, as the
// compiler makes of a paired sum.
__device__ __forceinline__ float2 add_alone(float2 a, float2 b)
{
    return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

template <int DT>
__device__ __forceinline__ void oct_floats(const Oct<DT>& o, float2 (&f)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == TSX_F32)
            f[j] = make_float2(__uint_as_float(o.w[2 * j]), __uint_as_float(o.w[2 * j + 1]));
        else if constexpr (DT == TSX_BF16)
            f[j] = make_float2(__uint_as_float(o.w[j] << 16), __uint_as_float(o.w[j] & 0xffff0000u));
        else
            f[j] = __half22float2(*reinterpret_cast<const __half2*>(&o.w[j]));
    }
}

// Rounded once, to nearest even, into the element type.
template <int DT>
__device__ __forceinline__ Oct<DT> oct_round(const float2 (&f)[4])
{
    Oct<DT> o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == TSX_F32) {
            o.w[2 * j] = __float_as_uint(f[j].x);
            o.w[2 * j + 1] = __float_as_uint(f[j].y);
        } else if constexpr (DT == TSX_BF16) {
            const __nv_bfloat162 v = __float22bfloat162_rn(f[j]);
            o.w[j] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __half2 v = __float22half2_rn(f[j]);
            o.w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    return o;
}

__device__ __forceinline__ void store16(char* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int DT, bool VEC>
__device__ __forceinline__ void oct_store(char* p, const OctAt& at, const Oct<DT>& o)
{
    if constexpr (VEC) {
        if constexpr (DT == TSX_F32) {
            if (whole_sector(p)) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o.w[0]), "r"(o.w[1]),
                             "r"(o.w[2]), "r"(o.w[3]), "r"(o.w[4]), "r"(o.w[5]), "r"(o.w[6]), "r"(o.w[7])
                             : "memory");
                return;
            }
            store16(p + 16, o.w[4], o.w[5], o.w[6], o.w[7]);
        }
        store16(p, o.w[0], o.w[1], o.w[2], o.w[3]);
    } else if constexpr (DT == TSX_F32) {
        uint32_t* e = reinterpret_cast<uint32_t*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at.ch + j * at.step < at.cols)
                e[j * at.step] = o.w[j];
    } else {
        unsigned short* e = reinterpret_cast<unsigned short*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at.ch + j * at.step < at.cols)
                e[j * at.step] = static_cast<unsigned short>(o.w[j / 2] >> (j % 2 * 16));
    }
}

// Eight values of a per-channel vector, fp32 (wide) or of the element type.
// packed: base and channels are aligned to 16 bytes.
template <int DT, bool VEC>
__device__ __forceinline__ void param_floats(const void* base, bool wide, bool packed, int ch0, const OctAt& at,
                                             float2 (&f)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = make_float2(0.f, 0.f);
    if (at.ch >= at.cols)
        return;
    if (VEC && packed) {
        if (wide || DT == TSX_F32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + ch0 + at.ch);
            const float4 u = __ldg(p), v = __ldg(p + 1);
            f[0] = make_float2(u.x, u.y);
            f[1] = make_float2(u.z, u.w);
            f[2] = make_float2(v.x, v.y);
            f[3] = make_float2(v.z, v.w);
        } else {
            oct_floats(oct_load<DT, true>(oct_ptr<DT>(base, 0, 0, ch0 + at.ch), at), f);
        }
        return;
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.f;
        if (at.ch + j * at.step < at.cols) {
            const int ch = ch0 + at.ch + j * at.step;
            if (wide || DT == TSX_F32)
                v[j] = __ldg(static_cast<const float*>(base) + ch);
            else if constexpr (DT == TSX_BF16)
                v[j] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[ch]);
            else if constexpr (DT == TSX_F16)
                v[j] = __half2float(static_cast<const __half*>(base)[ch]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = make_float2(v[2 * j], v[2 * j + 1]);
}

// ----------------------------------------------------------- activations

// sigmoid(z) = 1 / (1 + 2^t), t = -z log2(e), by the hardware's base-2
// exponential and reciprocal (ex2.approx, within 2 ulps, and rcp.approx, within
// 1): under 2^-21 together.  The roundings of t change 2^t, and so the sigmoid by
// a share 1 - sigmoid(z) of that: 2^-23 |z| for silu, 2^-21 of gelu's argument.
// For 16-bit elements that is far below the result's own rounding; for fp32 it is
// 2 to 4 ulps at ordinary z.  The division and the exponential with its range
// reduction would save them, at dozens of instructions an element where a whole
// kernel has 13 to 25.  Sigmoids under 2^-126 become 0, and with them silu under
// 2^-119 (z < -87.3) and its slope, and gelu's slope under 2^-118.
__device__ __forceinline__ float2 sigmoid_of(float2 t)
{
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(e, pair_of(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
}

constexpr float kLog2E = 1.44269504088896341f;

// The tanh form of gelu through the sigmoid: tanh(u) = 2 sigmoid(2 u) - 1, so
// gelu(z) = z sigmoid(2 k (z + 0.044715 z^3)), k = sqrt(2 / pi).  The argument
// is taken at |z| <= 24, where the sigmoid has long reached 0 or 1 in fp32:
// the cube of a large z stays finite, and 0 * infinity is never formed.
constexpr float kGelu2K = 1.5957691216057308f;
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float2 gelu_clamped(float2 z)
{
    return make_float2(fminf(fmaxf(z.x, -24.f), 24.f), fminf(fmaxf(z.y, -24.f), 24.f));
}

// f(A) with A the activation (the form of a checkpoint) as a constant.  A
// choice that every row makes anew cuts the code into blocks of one row, in
// which little hides the latency of the arithmetic: the kernels choose once for
// the few rows that they hold, and compute all of them, with zeros in place of
// those that do not exist.
template <int V>
struct Known {
    __device__ constexpr operator int() const { return V; }
};
template <class F>
__device__ __forceinline__ void by_act(int act, F f)
{
    if (act == TSX_ACT_SILU)
        f(Known<TSX_ACT_SILU>());
    else if (act == TSX_ACT_GELU)
        f(Known<TSX_ACT_GELU>());
    else
        f(Known<TSX_ACT_NONE>());
}
template <class F>
__device__ __forceinline__ void by_form(int form, F f)
{
    if (form == TSX_INT8)
        f(Known<TSX_INT8>());
    else
        f(Known<TSX_E4M3>());
}

// v = act(z) for an oct.
__device__ __forceinline__ void act_value(int act, const float2 (&z)[4], float2 (&v)[4])
{
    if (act == TSX_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __fmul2_rn(z[j], sigmoid_of(__fmul2_rn(z[j], pair_of(-kLog2E))));
    } else if (act == TSX_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = gelu_clamped(z[j]);
            const float2 u = __ffma2_rn(__fmul2_rn(t, t), pair_of(-kLog2E * kGelu2K * kGeluCube),
                                        pair_of(-kLog2E * kGelu2K));
            v[j] = __fmul2_rn(z[j], sigmoid_of(__fmul2_rn(t, u)));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = z[j];
    }
}

// act(z) and its derivative, from t = act_scale(act) * z.  For silu the factor
// is the exponential's -log2(e), which a caller with a product to spare folds
// into it: with p the sigmoid, act = -ln(2) t p and act' = p + act (1 - p).
__device__ __forceinline__ float act_scale(int act) { return act == TSX_ACT_SILU ? -kLog2E : 1.f; }
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ void act_slope(int act, const float2 (&t)[4], float2 (&slope)[4])
{
    const float2 one = pair_of(1.f), minus = pair_of(-1.f);
    if (act == TSX_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = sigmoid_of(t[j]);
            slope[j] = __ffma2_rn(__fmul2_rn(t[j], p), __ffma2_rn(p, pair_of(kLn2), pair_of(-kLn2)), p);
        }
    } else if (act == TSX_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c = gelu_clamped(t[j]), c2 = __fmul2_rn(c, c);
            const float2 u = __ffma2_rn(c2, pair_of(-kLog2E * kGelu2K * kGeluCube), pair_of(-kLog2E * kGelu2K));
            const float2 p = sigmoid_of(__fmul2_rn(c, u));
            const float2 inner = __ffma2_rn(c2, pair_of(3.f * kGelu2K * kGeluCube), pair_of(kGelu2K));
            const float2 rest = __fmul2_rn(__fmul2_rn(t[j], p), __ffma2_rn(p, minus, one));
            slope[j] = __ffma2_rn(rest, inner, p);   // 0, not 0 * infinity
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            slope[j] = one;
    }
}

__device__ __forceinline__ void act_both(int act, const float2 (&z)[4], float2 (&v)[4], float2 (&slope)[4])
{
    const float2 one = pair_of(1.f), minus = pair_of(-1.f);
    if (act == TSX_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = sigmoid_of(__fmul2_rn(z[j], pair_of(-kLog2E)));
            v[j] = __fmul2_rn(z[j], p);
            slope[j] = __ffma2_rn(v[j], __ffma2_rn(p, minus, one), p);   // p + v (1 - p)
        }
    } else if (act == TSX_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = gelu_clamped(z[j]), t2 = __fmul2_rn(t, t);
            const float2 u = __ffma2_rn(t2, pair_of(-kLog2E * kGelu2K * kGeluCube), pair_of(-kLog2E * kGelu2K));
            const float2 p = sigmoid_of(__fmul2_rn(t, u));
            const float2 inner = __ffma2_rn(t2, pair_of(3.f * kGelu2K * kGeluCube), pair_of(kGelu2K));
            v[j] = __fmul2_rn(z[j], p);
            slope[j] = __ffma2_rn(__fmul2_rn(v[j], __ffma2_rn(p, minus, one)), inner, p);   // 0, not 0 * infinity
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = z[j];
            slope[j] = one;
        }
    }
}

// ------------------------------------------------------------ 8-bit forms

// One scale of a block from the bits of its largest magnitude: amax / 127
// (int8) or amax / 448 (e4m3, its largest number), as a product with the
// rounded reciprocal; inv is the factor that takes values to the 8-bit
// numbers.  Under 2^-119 the block is held as zeros with scale 0 (the
// reciprocal of a smaller scale would overflow).  A block with an infinity or
// a NaN in it gets the scale NaN and so reads back as NaN throughout: a
// gradient check downstream sees it.
struct HeldScale {
    float scale, inv;
};
__device__ __forceinline__ HeldScale held_scale(uint32_t amax_bits, int form)
{
    HeldScale s;
    s.scale = __fmul_rn(__uint_as_float(amax_bits), form == TSX_INT8 ? 1.f / 127.f : 1.f / 448.f);
    s.inv = __frcp_rn(s.scale);
    if (amax_bits < 0x04000000u)   // 2^-119
        s.scale = s.inv = 0.f;
    if (amax_bits >= 0x7f800000u) {
        s.scale = __uint_as_float(0x7fc00000u);
        s.inv = 0.f;
    }
    return s;
}

// The largest magnitude of an oct, as the element type's bits: unsigned
// integers order magnitudes as floats do, with infinity above every number and
// NaN above infinity, which a float maximum would drop.  16-bit elements are
// compared two at a time.
template <int DT>
__device__ __forceinline__ uint32_t oct_amax_bits(const Oct<DT>& o)
{
    if constexpr (DT == TSX_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, o.w[j] & 0x7fffffffu);
        return m;
    } else {
        const uint32_t m = __vmaxu2(__vmaxu2(o.w[0] & 0x7fff7fffu, o.w[1] & 0x7fff7fffu),
                                    __vmaxu2(o.w[2] & 0x7fff7fffu, o.w[3] & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16);
    }
}
// Those bits as an fp32 magnitude.
template <int DT>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t m)
{
    if constexpr (DT == TSX_F32)
        return m;
    else if constexpr (DT == TSX_BF16)
        return m << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
}

// Eight 8-bit numbers as they lie in memory (channel j in byte j).
struct Held {
    uint32_t w[2];
};

// x * inv rounded to nearest even into the 8-bit form.  int8: adding 1.5 *
// 2^23 leaves the whole number in the sum's low byte (|x inv| <= 127 plus
// rounding, well inside); the product is rounded by itself first.
__device__ __forceinline__ Held held_round(const float2 (&f)[4], float inv, int form)
{
    Held h;
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = __fmul2_rn(f[j], pair_of(inv));
    if (form == TSX_INT8) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = add_alone(v[j], pair_of(12582912.f));   // the product is rounded by itself
#pragma unroll
        for (int k = 0; k < 2; ++k)
            h.w[k] = __byte_perm(
                __byte_perm(__float_as_uint(v[2 * k].x), __float_as_uint(v[2 * k].y), 0x0040),
                __byte_perm(__float_as_uint(v[2 * k + 1].x), __float_as_uint(v[2 * k + 1].y), 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(v[2 * k], __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(v[2 * k + 1], __NV_SATFINITE, __NV_E4M3);
            h.w[k] = lo | hi << 16;
        }
    }
    if (inv == 0.f)   // zeros; also where 0 * infinity or NaN stood
        h.w[0] = h.w[1] = 0;
    return h;
}

// The numbers q.  int8: the byte, offset by 128, becomes the low byte of 2^23 +
// b; subtracting 2^23 + 128 leaves the number exactly, without an integer
// conversion.
__device__ __forceinline__ void held_numbers(const Held& h, int form, float2 (&f)[4])
{
    if (form == TSX_INT8) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t u = h.w[k] ^ 0x80808080u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 b = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 | 2 * j)),
                                             __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541 | 2 * j)));
                f[2 * k + j] = __fadd2_rn(b, pair_of(-8388736.f));
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __half2_raw r =
                    __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h.w[k] >> (16 * j)), __NV_E4M3);
                f[2 * k + j] = __half22float2(__half2(r));
            }
    }
}

// The fp32 values q * scale.
__device__ __forceinline__ void held_floats(const Held& h, float scale, int form, float2 (&f)[4])
{
    held_numbers(h, form, f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = __fmul2_rn(f[j], pair_of(scale));
}

template <bool VEC>
__device__ __forceinline__ Held held_load(const uint8_t* p, const OctAt& at)
{
    Held h;
    if constexpr (VEC) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(h.w[0]), "=r"(h.w[1]) : "l"(p));
    } else {
        h.w[0] = h.w[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at.ch + j * at.step < at.cols)
                h.w[j / 4] |= static_cast<uint32_t>(p[j * at.step]) << (j % 4 * 8);
    }
    return h;
}

template <bool VEC>
__device__ __forceinline__ void held_store(uint8_t* p, const OctAt& at, const Held& h)
{
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = make_uint2(h.w[0], h.w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at.ch + j * at.step < at.cols)
                p[j * at.step] = static_cast<uint8_t>(h.w[j / 4] >> (j % 4 * 8));
    }
}

// Block of a channel; blocks are 32, 64 or 128 channels.
__device__ __forceinline__ int block_of(int ch, int block) { return ch >> (31 - __clz(block)); }

// Where a thread's checkpoint bytes and its team's scale go: first row, and
// from row to row of its walk.
struct HeldPtr {
    uint8_t* q;
    float* scale;
    int64_t q_step, scale_step;
    __device__ __forceinline__ HeldPtr() {}
    __device__ __forceinline__ HeldPtr(const HeldOut& out, int64_t row, int64_t rows_apart, int cols, int64_t blocks,
                                       int ch, int block)
        : q(static_cast<uint8_t*>(out.q) + row * cols + ch),
          scale(out.scale + row * blocks + block_of(ch, block)),
          q_step(rows_apart * cols),
          scale_step(rows_apart * blocks)
    {
    }
    __device__ __forceinline__ void advance(int rows)
    {
        q += rows * q_step;
        scale += rows * scale_step;
    }
};

// Where the octs of hold_rows go: `n` rows of one walk, or two of each of two.
struct HeldRows {
    HeldPtr out;
    int n;
    __device__ __forceinline__ bool has(int i) const { return i < n; }
    __device__ __forceinline__ uint8_t* q(int i) const { return out.q + i * out.q_step; }
    __device__ __forceinline__ float* scale(int i) const { return out.scale + i * out.scale_step; }
};
struct HeldPairs {
    HeldPtr first, second;
    int n;
    __device__ __forceinline__ bool has(int i) const { return (i & 1) < n; }
    __device__ __forceinline__ uint8_t* q(int i) const { return (i < 2 ? first.q : second.q) + (i & 1) * first.q_step; }
    __device__ __forceinline__ float* scale(int i) const
    {
        return (i < 2 ? first.scale : second.scale) + (i & 1) * first.scale_step;
    }
};

// Four octs of a thread to 8 bits, each with its team's scale, to where `out`
// says, which also says which of them exist (none: the thread only lends its
// lane).  All lanes of a warp come together, those of a team with the same
// octs; `live` threads hold channels.  The maxima of two rows of 16-bit elements share a
// shuffle, and where a team has as many lanes as there are rows, each lane
// works out one row's scale for all.
template <int DT, bool VEC, class Out>
__device__ __forceinline__ void hold_rows(const Oct<DT> (&o)[4], bool live, const OctAt& at, int team, int form,
                                          const Out& out)
{
    constexpr int N = 4;
    const int lane = static_cast<int>(threadIdx.x) & 31, base = lane & ~(team - 1);
    const bool block = at.ch - (lane - base) * (VEC ? kOct : 1) < at.cols;   // the team has a block at all
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        m[i] = live ? oct_amax_bits<DT>(o[i]) : 0u;
    if constexpr (DT == TSX_F32) {
        for (int d = 1; d < team; d <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    } else {
        uint32_t two[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            two[i] = m[2 * i] | m[2 * i + 1] << 16;
        for (int d = 1; d < team; d <<= 1)
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                two[i] = __vmaxu2(two[i], __shfl_xor_sync(0xffffffffu, two[i], d));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            m[2 * i] = two[i] & 0xffffu;
            m[2 * i + 1] = two[i] >> 16;
        }
    }
    float inv[N];
    if (team >= N) {
        const int mine = lane - base;   // the first N lanes of the team have a row each
        uint32_t own = m[0];
#pragma unroll
        for (int i = 1; i < N; ++i)
            own = mine == i ? m[i] : own;
        const HeldScale s = held_scale(magnitude_bits<DT>(own), form);
        if (block && mine < N && out.has(mine))
            *out.scale(mine) = s.scale;
#pragma unroll
        for (int i = 0; i < N; ++i)
            inv[i] = __shfl_sync(0xffffffffu, s.inv, base + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const HeldScale s = held_scale(magnitude_bits<DT>(m[i]), form);
            inv[i] = s.inv;
            if (block && lane == base && out.has(i))
                *out.scale(i) = s.scale;
        }
    }
    by_form(form, [&](auto known) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 f[4];
            oct_floats(o[i], f);
            const Held h = held_round(f, inv[i], known);
            if (live && out.has(i))
                held_store<VEC>(out.q(i), at, h);
        }
    });
}

}  // namespace dev
// Launch `Kernel` with clusters of `ranks` CTAs along x (1: none); `early`: it
// may start while the stream's last kernel still runs (it waits by itself).
// More than 48 KB of shared memory is asked for once on each device.  The result
// is this launch's own: the runtime's last error may be another call's.
template <auto Kernel, class... Args>
cudaError_t launch_grid(dim3 grid, int threads, size_t smem, int ranks, bool early, cudaStream_t st, Args... args)
{
    if (smem > 48 * 1024) {
        constexpr int kDevices = 64;
        static std::atomic<bool> allowed[kDevices];
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e == cudaSuccess && (device >= kDevices || !allowed[device].load())) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynSmem);
            if (e == cudaSuccess && device < kDevices)
                allowed[device].store(true);
        }
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2]{};
    if (ranks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = unsigned(ranks);
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (early) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace tsx
