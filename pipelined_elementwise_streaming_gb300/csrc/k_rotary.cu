// Rotary positions and norms of heads: forward, backward, and forward into a
// paged cache.
//
// A pair (a, b) of a head at position p becomes (a c - b s, b c + a s), c and s
// the amplitude times the cosine and sine of p f; with a norm the pair is x rstd
// weight, rstd = 1 / sqrt(mean(x^2) + eps).  Backward, for d the gradient turned
// back, dx = rstd d w - x rstd^3 sum(d w x) / dim and dw = sum(d x rstd).
//
// One pass over the tensors, bound by HBM.  A thread owns eight channels of a head
// and keeps them: two quads that hold four whole pairs, so that a rotation needs no
// other thread and a norm a few shuffles within the team of threads of a head.  It
// computes its four sines and cosines once for a token and uses them for the several
// heads that it goes over, the next of them on their way while it works on some.  A
// table of sines and cosines would be read instead: 4 bytes to a channel and token, as
// much as two 16-bit heads.  Angles are whole numbers: the position times the part of
// a turn that a position adds, modulo 2^64.  Sixteen channels to a thread, one batch of
// heads at a time, took 35 us where this takes 27 (see below), for want of warps: 112
// registers a thread in place of 58 to 73.
//
// Measured on GB300, GPU time of a call in a CUDA graph over tensors that take turns;
// in parentheses the time of the bytes at the 6791 GB/s of a copy.  bf16 [8192, 32 + 8
// heads, 128], all of it from one projection: rotary 27.0 us (24.7), with norms 29.6
// (24.7), the gradient through both 55.0 (37.1), its sums for the weights among them;
// fp32 [4096, 40, 128] with norms 29.3 (24.7), gradient 46.4 (37.1).  f16 [8191, 32,
// 96], 64 channels of a head turned, interleaved: 15.7 (14.8).  Both passes of fp32
// [4096, 24, 64] without norms: 15.4 (14.8).  Appending 6400 tokens of f16 [16 + 8 + 8,
// 64] in pages of 64: 9.1 (7.3).  What is left: instructions, at 61 % of the issue
// slots with norms forward and 50 % backward, where two CTAs fit an SM.

#include "attention.h"
#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kWarps = kRotaryThreads / 32;
constexpr int kStarts = 1024;   // sequences whose starts a CTA keeps in shared memory

// Sine and cosine of `turn` / 2^32 of a turn.
template <int DT>
__device__ __forceinline__ float2 cos_sin(uint32_t turn)
{
    float c, s;
    if constexpr (DT == TSX_F32) {
        // the nearest quarter turn apart, the rest within an eighth: a rest of 30
        // bits rounds to fp32 with 2^-26 of a radian at most
        const uint32_t quarter = (turn + (1u << 29)) >> 30;
        sincospif(static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) * 0x1p-31f, &s, &c);
        const float t = c;
        if (quarter & 1) {
            c = -s;
            s = t;
        }
        if (quarter & 2) {
            c = -c;
            s = -s;
        }
    } else {
        // the hardware's, within 2^-21 on -pi .. pi, and 2^-22 by the argument's rounding:
        // a 2^-8 part (fp16) or less of the half step of the result
        const float x = static_cast<float>(static_cast<int32_t>(turn)) * 1.46291807926715968e-9f;   // pi / 2^31
        c = __cosf(x);
        s = __sinf(x);
    }
    return make_float2(c, s);
}

__device__ __forceinline__ uint32_t turn_of(int64_t position, uint64_t turns)
{
    return static_cast<uint32_t>((static_cast<uint64_t>(position) * turns) >> 32);
}

__device__ __forceinline__ int64_t position_of(const RotaryArgs& a, int64_t token)
{
    return a.wide_positions ? static_cast<const int64_t*>(a.positions)[token]
                            : static_cast<const int32_t*>(a.positions)[token];
}

// Where a token of a batch stands: its position, and the slot that it gets.
struct TokenPlace {
    int64_t position;
    int64_t offset;   // elements from the cache's start
    bool live;        // it belongs to a sequence
    bool stored;      // and has a slot
};

// `starts`: the first min(seqs, kStarts) + 1 of them, in shared memory.
__device__ __forceinline__ TokenPlace token_place(const PagedArgs& p, const int32_t* starts, int64_t token,
                                                  int64_t slot_pitch)
{
    TokenPlace t{};
    const int32_t* s = p.seqs <= kStarts ? starts : p.starts;
    if (token < s[0] || token >= s[p.seqs])
        return t;
    int lo = 0, hi = p.seqs;   // s[lo] <= token < s[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s[mid] <= token)
            lo = mid;
        else
            hi = mid;
    }
    t.live = true;
    const int64_t most = min(static_cast<int64_t>(p.most_pages) * p.page_size, static_cast<int64_t>(kMostKeys));
    const int64_t length = min(static_cast<int64_t>(p.lengths[lo]), most);
    t.position = length - s[lo + 1] + token;
    if (t.position < 0)
        return t;
    if (t.position >= length)   // starts that fall
        return t;
    const int at = static_cast<int>(t.position), n = at / p.page_size;   // < most_pages
    const int64_t page = p.pages[lo * p.pages_pitch + n];
    t.stored = page >= 0 && page < p.cache_pages;
    t.offset = page * p.page_pitch + (at - n * p.page_size) * slot_pitch;
    return t;
}

__device__ __forceinline__ void load_starts(const PagedArgs& p, int32_t* starts)
{
    if (p.seqs <= kStarts)
        for (int i = threadIdx.x; i <= p.seqs; i += blockDim.x)
            starts[i] = p.starts[i];
    __syncthreads();
}

// A thread's eight channels: two quads of a head, and the first of the four pairs
// that they are.
struct Slot {
    int ch[2];
    bool has, turned;
    int pair;
};

template <bool INTER>
__device__ __forceinline__ Slot slot_of(int j, int dim, int rot)
{
    Slot s;
    s.pair = 4 * j;
    s.has = 8 * j < dim;
    s.turned = 8 * j < rot;
    if (INTER || !s.turned) {   // neighbours; what does not turn is laid out alike
        s.ch[0] = 8 * j;
        s.ch[1] = 8 * j + 4;
    } else {
        s.ch[0] = 4 * j;
        s.ch[1] = rot / 2 + 4 * j;
    }
    return s;
}

template <int DT>
__device__ __forceinline__ void slot_angles(const RotaryArgs& a, const Slot& s, int64_t position, float (&c)[4],
                                            float (&n)[4])
{
    // By generic loads: lanes ask for different words, which the constant cache answers
    // one after the other (8 tokens of 40 heads 2.05 us in place of 2.64).
    uint64_t turns[4];
    const uint64_t* from = a.turns + s.pair;
    asm volatile("ld.v2.b64 {%0, %1}, [%2];" : "=l"(turns[0]), "=l"(turns[1]) : "l"(from));
    asm volatile("ld.v2.b64 {%0, %1}, [%2];" : "=l"(turns[2]), "=l"(turns[3]) : "l"(from + 2));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = 1.f;
        n[i] = 0.f;
        if (s.turned) {
            const float2 v = cos_sin<DT>(turn_of(position, turns[i]));
            c[i] = v.x * a.amplitude;
            n[i] = v.y * a.amplitude;
        }
    }
}

// Four elements as they lie in memory, loaded and stored at once; in the order of
// oct_load and oct_store, so that an output may be an input.
template <int DT>
struct Quad {
    uint32_t w[DT == TSX_F32 ? 4 : 2];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < int(sizeof(w) / 4); ++i)
            w[i] = 0;
    }
    __device__ __forceinline__ void load(const char* p)
    {
        if constexpr (DT == TSX_F32)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "l"(p));
        else
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
    __device__ __forceinline__ void store(char* p) const
    {
        if constexpr (DT == TSX_F32)
            store16(p, w[0], w[1], w[2], w[3]);
        else
            asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
    }
    __device__ __forceinline__ void floats(float2 (&f)[2]) const
    {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (DT == TSX_F32)
                f[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
            else if constexpr (DT == TSX_BF16)
                f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
            else
                f[j] = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        }
    }
    // Rounded once, to nearest even, into the element type.
    __device__ __forceinline__ void round(const float2 (&f)[2])
    {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (DT == TSX_F32) {
                w[2 * j] = __float_as_uint(f[j].x);
                w[2 * j + 1] = __float_as_uint(f[j].y);
            } else if constexpr (DT == TSX_BF16) {
                const __nv_bfloat162 v = __float22bfloat162_rn(f[j]);
                w[j] = *reinterpret_cast<const uint32_t*>(&v);
            } else {
                const __half2 v = __float22half2_rn(f[j]);
                w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
    }
};

// The pairs of two quads turned by the angles, or (BACK) against them.
template <bool INTER, bool BACK>
__device__ __forceinline__ void turn(const float (&c)[4], const float (&n)[4], float2 (&u)[2], float2 (&v)[2])
{
    if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 t = make_float2(BACK ? u[j].y : -u[j].y, BACK ? -u[j].x : u[j].x);
            u[j] = __ffma2_rn(t, pair_of(n[j]), __fmul2_rn(u[j], pair_of(c[j])));
            const float2 w = make_float2(BACK ? v[j].y : -v[j].y, BACK ? -v[j].x : v[j].x);
            v[j] = __ffma2_rn(w, pair_of(n[2 + j]), __fmul2_rn(v[j], pair_of(c[2 + j])));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 cc = make_float2(c[2 * j], c[2 * j + 1]), nn = make_float2(n[2 * j], n[2 * j + 1]);
            const float2 mm = make_float2(-nn.x, -nn.y), p = u[j];
            u[j] = __ffma2_rn(v[j], BACK ? nn : mm, __fmul2_rn(p, cc));
            v[j] = __ffma2_rn(p, BACK ? mm : nn, __fmul2_rn(v[j], cc));
        }
    }
}

// Sum over the `team` neighbouring threads of a head; every thread of the warp takes part.
__device__ __forceinline__ float team_sum(float v, int team)
{
    for (int m = team / 2; m > 0; m >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
// The same of several sums at once, whose shuffles then do not wait for one another.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], int team)
{
    for (int m = team / 2; m > 0; m >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    }
}

__device__ __forceinline__ float dot(const float2 (&u)[2], const float2 (&v)[2], const float2 (&x)[2],
                                     const float2 (&y)[2])
{
    float2 q = __fmul2_rn(u[0], x[0]);
    q = __ffma2_rn(u[1], x[1], q);
    q = __ffma2_rn(v[0], y[0], q);
    q = __ffma2_rn(v[1], y[1], q);
    return q.x + q.y;
}

// A thread's quads of N heads, `step` bytes apart from `p` on, of which `left` exist;
// `second`: bytes from the first quad to the second.
template <int DT, int N>
struct Heads {
    Quad<DT> u[N], v[N];
    __device__ __forceinline__ void load(const char* p, int64_t step, int second, int left)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u[i].zero();
            v[i].zero();
            if (i < left) {
                u[i].load(p);
                v[i].load(p + second);
            }
            p += step;
        }
    }
};

__device__ __forceinline__ const RotaryRole& role_of(const RotaryArgs& a)
{
    const int b = blockIdx.x;
    return a.role[a.roles > 1 && b >= a.role[1].first ? (a.roles > 2 && b >= a.role[2].first ? 2 : 1) : 0];
}

template <int DT>
__device__ __forceinline__ void quad_weights(const RotaryArgs& a, const RotaryRole& r, int ch, float2 (&w)[2])
{
    if (a.wide_params || DT == TSX_F32) {
        const float* p = static_cast<const float*>(r.weight) + ch;
        if (r.packed_weight) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p));
            w[0] = make_float2(v.x, v.y);
            w[1] = make_float2(v.z, v.w);
        } else {
            w[0] = make_float2(__ldg(p), __ldg(p + 1));
            w[1] = make_float2(__ldg(p + 2), __ldg(p + 3));
        }
    } else {
        const unsigned short* p = static_cast<const unsigned short*>(r.weight) + ch;
        Quad<DT> q;
        q.w[0] = __ldg(p) | static_cast<uint32_t>(__ldg(p + 1)) << 16;
        q.w[1] = __ldg(p + 2) | static_cast<uint32_t>(__ldg(p + 3)) << 16;
        q.floats(w);
    }
}

template <int DT>
__device__ __forceinline__ void slot_weights(const RotaryArgs& a, const RotaryRole& r, const Slot& s, float2 (&wu)[2],
                                             float2 (&wv)[2])
{
    wu[0] = wu[1] = wv[0] = wv[1] = pair_of(1.f);
    if (r.weight && s.has) {
        quad_weights<DT>(a, r, s.ch[0], wu);
        quad_weights<DT>(a, r, s.ch[1], wv);
    }
}

// Forward.  The gradient of the rotation alone is the same with frequencies of the
// other sign.  A team has one token's heads, `parts` apart.
template <int DT, bool INTER, bool NORM, bool PAGED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    constexpr int N = rotary_batch(DT);
    __shared__ int32_t starts[PAGED ? kStarts + 1 : 1];
    const RotaryRole& r = role_of(a);
    if constexpr (PAGED)
        load_starts(a.paged, starts);
    const int teams = kRotaryThreads / a.team, lane = threadIdx.x & (a.team - 1);
    const uint32_t item = (blockIdx.x - r.first) * teams + threadIdx.x / a.team;   // tokens * heads < 2^31
    const uint32_t which = item / static_cast<uint32_t>(r.parts);
    const int64_t token = which;
    const int part = static_cast<int>(item - which * r.parts);
    const Slot s = slot_of<INTER>(lane, a.dim, a.rot);
    bool live = token < a.tokens;
    int64_t position = 0, base = token * r.out_pitch;
    if constexpr (PAGED) {
        if (live) {
            const TokenPlace t = token_place(a.paged, starts, token, r.out_pitch);
            live = t.live && (t.stored || !r.paged);
            position = t.position;
            if (r.paged)
                base = t.offset;
        }
    } else if (live) {
        position = position_of(a, token);
    }
    const int second = (s.ch[1] - s.ch[0]) * elem_size(DT);
    const char* in = r.x + (token * r.x_pitch + part * r.x_head + s.ch[0]) * elem_size(DT);
    char* out = r.out + (base + part * r.out_head + s.ch[0]) * elem_size(DT);
    const int64_t in_step = r.parts * r.x_head * elem_size(DT), out_step = r.parts * r.out_head * elem_size(DT);
    int left = live && s.has ? (r.heads - part + r.parts - 1) / r.parts : 0;
    Heads<DT, N> now, next;
    now.load(in, in_step, second, left);
    // while the first heads are on their way
    float c[4], n[4];
    float2 wu[2], wv[2];
    if (r.turn) {
        slot_angles<DT>(a, s, position, c, n);
        if constexpr (NORM)
            slot_weights<DT>(a, r, s, wu, wv);
    }
    for (int h0 = 0; h0 < r.heads; h0 += N * r.parts) {   // alike for all threads of the CTA
        in += N * in_step;
        next.load(in, in_step, second, left - N);
        float rstd[N];
        if (NORM && r.turn) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 p[2], q[2];
                now.u[i].floats(p);
                now.v[i].floats(q);
                rstd[i] = dot(p, q, p, q);
            }
            team_sums(rstd, a.team);
#pragma unroll
            for (int i = 0; i < N; ++i)
                rstd[i] = rsqrtf(rstd[i] * a.by_dim + a.eps);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (r.turn && (NORM || s.turned)) {   // the others keep their bits
                float2 p[2], q[2];
                now.u[i].floats(p);
                now.v[i].floats(q);
                if constexpr (NORM) {
                    const float2 f = pair_of(rstd[i]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        p[j] = __fmul2_rn(__fmul2_rn(p[j], f), wu[j]);
                        q[j] = __fmul2_rn(__fmul2_rn(q[j], f), wv[j]);
                    }
                }
                if (s.turned)
                    turn<INTER, false>(c, n, p, q);
                now.u[i].round(p);
                now.v[i].round(q);
            }
            if (i < left) {
                now.u[i].store(out);
                now.v[i].store(out + second);
            }
            out += out_step;
        }
        left -= N;
        now = next;
    }
}

// Sums of a CTA's warps [kWarps][dim] to its slice.
__device__ __forceinline__ void store_slice(const RotaryRole& r, int dim, const float* sums)
{
    __syncthreads();
    float* to = r.slices + static_cast<int64_t>(blockIdx.x - r.first) * dim;
    for (int ch = threadIdx.x; ch < dim; ch += blockDim.x) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += sums[w * kRotaryDim + ch];
        to[ch] = v;
    }
}

// Backward through norm and rotation.  CTAs stay for all their tokens, so that the
// weights' gradients come out as one slice to a CTA.
template <int DT, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads, backward_ctas(DT))
    rotary_norm_backward_kernel(const __grid_constant__ RotaryArgs a)
{
    constexpr int N = rotary_batch(DT) / 2;
    __shared__ float sums[kWarps * kRotaryDim];
    const RotaryRole& r = role_of(a);
    let_next_start();
    const uint32_t teams = kRotaryThreads / a.team;
    const int lane = threadIdx.x & (a.team - 1);
    const Slot s = slot_of<INTER>(lane, a.dim, a.rot);
    float2 wu[2], wv[2], su[2], sv[2];
    slot_weights<DT>(a, r, s, wu, wv);
    su[0] = su[1] = sv[0] = sv[1] = pair_of(0.f);
    const int second = (s.ch[1] - s.ch[0]) * elem_size(DT);
    const int64_t in_step = r.parts * r.x_head * elem_size(DT), saved_step = r.parts * r.saved_head * elem_size(DT),
                  out_step = r.parts * r.out_head * elem_size(DT);
    const uint32_t items = static_cast<uint32_t>(a.tokens) * r.parts;   // < 2^31
    for (uint32_t first = (blockIdx.x - r.first) * teams; first < items; first += r.ctas * teams) {
        const uint32_t item = first + threadIdx.x / a.team, which = item / static_cast<uint32_t>(r.parts);
        const int64_t token = which;
        const int part = static_cast<int>(item - which * r.parts);
        const bool live = item < items;
        const int64_t position = live ? position_of(a, token) : 0;
        const char* in = r.x + (token * r.x_pitch + part * r.x_head + s.ch[0]) * elem_size(DT);
        const char* saved = r.saved + (token * r.saved_pitch + part * r.saved_head + s.ch[0]) * elem_size(DT);
        char* out = r.out + (token * r.out_pitch + part * r.out_head + s.ch[0]) * elem_size(DT);
        int left = live && s.has ? (r.heads - part + r.parts - 1) / r.parts : 0;
        Heads<DT, N> d, x, next_d, next_x;
        d.load(in, in_step, second, left);
        x.load(saved, saved_step, second, left);
        float c[4], n[4];
        slot_angles<DT>(a, s, position, c, n);
        for (int h0 = 0; h0 < r.heads; h0 += N * r.parts) {   // alike for all threads of the CTA
            in += N * in_step;
            saved += N * saved_step;
            next_d.load(in, in_step, second, left - N);
            next_x.load(saved, saved_step, second, left - N);
            // sums over the head of x^2, and of d weight x: times rstd, that along xhat
            float sums2[2 * N];
            float2 p[N][2], q[N][2];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 xu[2], xv[2], pw[2], qw[2];
                d.u[i].floats(p[i]);
                d.v[i].floats(q[i]);
                x.u[i].floats(xu);
                x.v[i].floats(xv);
                if (s.turned)
                    turn<INTER, true>(c, n, p[i], q[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pw[j] = __fmul2_rn(p[i][j], wu[j]);
                    qw[j] = __fmul2_rn(q[i][j], wv[j]);
                }
                sums2[2 * i] = dot(xu, xv, xu, xv);
                sums2[2 * i + 1] = dot(pw, qw, xu, xv);
            }
            team_sums(sums2, a.team);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // 0 where there is no head: with an eps of 0 the root of its zeros is infinite, and its sums NaN
                const float rstd = i < left ? rsqrtf(sums2[2 * i] * a.by_dim + a.eps) : 0.f;
                const float2 f = pair_of(rstd), m = pair_of(-(sums2[2 * i + 1] * rstd) * a.by_dim);
                float2 xu[2], xv[2];
                x.u[i].floats(xu);
                x.v[i].floats(xv);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    xu[j] = __fmul2_rn(xu[j], f);
                    xv[j] = __fmul2_rn(xv[j], f);
                    su[j] = __ffma2_rn(p[i][j], xu[j], su[j]);
                    sv[j] = __ffma2_rn(q[i][j], xv[j], sv[j]);
                    xu[j] = __fmul2_rn(__ffma2_rn(xu[j], m, __fmul2_rn(p[i][j], wu[j])), f);
                    xv[j] = __fmul2_rn(__ffma2_rn(xv[j], m, __fmul2_rn(q[i][j], wv[j])), f);
                }
                if (i < left) {
                    d.u[i].round(xu);
                    d.v[i].round(xv);
                    d.u[i].store(out);
                    d.v[i].store(out + second);
                }
                out += out_step;
            }
            left -= N;
            d = next_d;
            x = next_x;
        }
    }
    if (!r.slices)
        return;
    for (int m = a.team; m < 32; m *= 2)   // over the teams of a warp
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            su[j].x += __shfl_xor_sync(0xffffffffu, su[j].x, m);
            su[j].y += __shfl_xor_sync(0xffffffffu, su[j].y, m);
            sv[j].x += __shfl_xor_sync(0xffffffffu, sv[j].x, m);
            sv[j].y += __shfl_xor_sync(0xffffffffu, sv[j].y, m);
        }
    if ((threadIdx.x & 31) < a.team && s.has) {
        float* to = sums + threadIdx.x / 32 * kRotaryDim;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            to[s.ch[0] + 2 * j] = su[j].x;
            to[s.ch[0] + 2 * j + 1] = su[j].y;
            to[s.ch[1] + 2 * j] = sv[j].x;
            to[s.ch[1] + 2 * j + 1] = sv[j].y;
        }
    }
    store_slice(r, a.dim, sums);
}

// ---------------------------------------------------- element by element
// Any layout: a warp to a head, a lane to every 32nd pair and to every 32nd of
// the channels that do not turn.

template <int DT>
struct Elem {
    using type = unsigned short;
};
template <>
struct Elem<TSX_F32> {
    using type = float;
};

template <int DT>
__device__ __forceinline__ float elem_load(const char* base, int64_t at)
{
    const typename Elem<DT>::type v = reinterpret_cast<const typename Elem<DT>::type*>(base)[at];
    if constexpr (DT == TSX_F32)
        return v;
    else if constexpr (DT == TSX_BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
        return __half2float(__ushort_as_half(v));
}

template <int DT>
__device__ __forceinline__ void elem_store(char* base, int64_t at, float f)
{
    typename Elem<DT>::type* p = reinterpret_cast<typename Elem<DT>::type*>(base) + at;
    if constexpr (DT == TSX_F32)
        *p = f;
    else if constexpr (DT == TSX_BF16)
        *p = __bfloat16_as_ushort(__float2bfloat16_rn(f));
    else
        *p = __half_as_ushort(__float2half_rn(f));
}

template <int DT>
__device__ __forceinline__ void elem_copy(char* to, const char* from, int64_t at)
{
    reinterpret_cast<typename Elem<DT>::type*>(to)[at] = reinterpret_cast<const typename Elem<DT>::type*>(from)[at];
}

template <int DT>
__device__ __forceinline__ float weight_of(const RotaryArgs& a, const RotaryRole& r, int ch)
{
    if (!r.weight)
        return 1.f;
    return a.wide_params ? static_cast<const float*>(r.weight)[ch]
                         : elem_load<DT>(static_cast<const char*>(r.weight), ch);
}

constexpr int kPairs = kRotaryDim / 64, kOthers = kRotaryDim / 32;   // of a lane at most

// BACK: the gradient through norm and rotation.
template <int DT, bool BACK>
__global__ void __launch_bounds__(kRotaryThreads) rotary_any_kernel(const __grid_constant__ RotaryArgs a)
{
    __shared__ int32_t starts[kStarts + 1];
    __shared__ float sums[BACK ? kWarps * kRotaryDim : 1];
    const RotaryRole& r = role_of(a);
    if constexpr (BACK)
        let_next_start();
    if (!a.positions)
        load_starts(a.paged, starts);
    const int lane = threadIdx.x & 31, rot = r.turn ? a.rot : 0, half = rot / 2;
    const bool norm = a.norm && r.turn;
    const int step = a.layout == TSX_ROPE_INTERLEAVED ? 2 : 1, far = a.layout == TSX_ROPE_INTERLEAVED ? 1 : half;
    float sa[kPairs], sb[kPairs], so[kOthers];   // sums for the weight's gradient
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
        sa[k] = sb[k] = 0.f;
#pragma unroll
    for (int k = 0; k < kOthers; ++k)
        so[k] = 0.f;
    const uint32_t items = static_cast<uint32_t>(a.tokens) * r.parts;   // < 2^31
    for (uint32_t item = (blockIdx.x - r.first) * kWarps + threadIdx.x / 32; item < items;
         item += r.ctas * kWarps) {   // alike for all threads of a warp
        const int64_t token = item / static_cast<uint32_t>(r.parts);
        int64_t position = 0, base = token * r.out_pitch;
        if (a.positions) {
            position = position_of(a, token);
        } else {
            const TokenPlace t = token_place(a.paged, starts, token, r.out_pitch);
            if (!t.live || (r.paged && !t.stored))
                continue;
            position = t.position;
            if (r.paged)
                base = t.offset;
        }
        float c[kPairs], n[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            c[k] = 1.f;
            n[k] = 0.f;
            if (lane + 32 * k < half) {
                const float2 v = cos_sin<DT>(turn_of(position, a.turns[lane + 32 * k]));
                c[k] = v.x * a.amplitude;
                n[k] = v.y * a.amplitude;
            }
        }
        for (int h = static_cast<int>(item - token * r.parts); h < r.heads; h += r.parts) {
            const char* in = r.x + (token * r.x_pitch + h * r.x_head) * elem_size(DT);
            const char* saved = r.saved + (token * r.saved_pitch + h * r.saved_head) * elem_size(DT);
            char* out = r.out + (base + h * r.out_head) * elem_size(DT);
            float u[kPairs], v[kPairs], o[kOthers], x[kPairs], y[kPairs], z[kOthers];
            float squares = 0.f, along = 0.f;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const int i = lane + 32 * k;
                u[k] = v[k] = x[k] = y[k] = 0.f;
                if (i < half) {
                    u[k] = elem_load<DT>(in, i * step);
                    v[k] = elem_load<DT>(in, i * step + far);
                    if constexpr (BACK) {
                        x[k] = elem_load<DT>(saved, i * step);
                        y[k] = elem_load<DT>(saved, i * step + far);
                    }
                }
                squares += BACK ? x[k] * x[k] + y[k] * y[k] : u[k] * u[k] + v[k] * v[k];
            }
#pragma unroll
            for (int k = 0; k < kOthers; ++k) {
                const int ch = rot + lane + 32 * k;
                o[k] = z[k] = 0.f;
                if (ch < a.dim) {
                    o[k] = elem_load<DT>(in, ch);
                    if constexpr (BACK)
                        z[k] = elem_load<DT>(saved, ch);
                }
                squares += BACK ? z[k] * z[k] : o[k] * o[k];
            }
            float rstd = 1.f;
            if (norm)
                rstd = rsqrtf(team_sum(squares, 32) / a.dim + a.eps);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const int i = lane + 32 * k;
                if (i >= half)
                    continue;
                const int c0 = i * step, c1 = i * step + far;
                if constexpr (BACK) {
                    const float p = u[k];
                    u[k] = p * c[k] + v[k] * n[k];
                    v[k] = v[k] * c[k] - p * n[k];
                    x[k] *= rstd;
                    y[k] *= rstd;
                    sa[k] += u[k] * x[k];
                    sb[k] += v[k] * y[k];
                    u[k] *= weight_of<DT>(a, r, c0);
                    v[k] *= weight_of<DT>(a, r, c1);
                    along += u[k] * x[k] + v[k] * y[k];
                } else {
                    if (norm) {
                        u[k] = u[k] * rstd * weight_of<DT>(a, r, c0);
                        v[k] = v[k] * rstd * weight_of<DT>(a, r, c1);
                    }
                    const float p = u[k];
                    u[k] = p * c[k] - v[k] * n[k];
                    v[k] = v[k] * c[k] + p * n[k];
                }
            }
#pragma unroll
            for (int k = 0; k < kOthers; ++k) {
                const int ch = rot + lane + 32 * k;
                if (ch >= a.dim)
                    continue;
                if constexpr (BACK) {
                    z[k] *= rstd;
                    so[k] += o[k] * z[k];
                    o[k] *= weight_of<DT>(a, r, ch);
                    along += o[k] * z[k];
                } else if (norm) {
                    o[k] = o[k] * rstd * weight_of<DT>(a, r, ch);
                }
            }
            if constexpr (BACK) {
                const float m = team_sum(along, 32) / a.dim;
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    u[k] = (u[k] - x[k] * m) * rstd;
                    v[k] = (v[k] - y[k] * m) * rstd;
                }
#pragma unroll
                for (int k = 0; k < kOthers; ++k)
                    o[k] = (o[k] - z[k] * m) * rstd;
            }
            __syncwarp();   // all lanes have loaded: the output may lie over an input
#pragma unroll
            for (int k = 0; k < kPairs; ++k)
                if (lane + 32 * k < half) {
                    elem_store<DT>(out, (lane + 32 * k) * step, u[k]);
                    elem_store<DT>(out, (lane + 32 * k) * step + far, v[k]);
                }
#pragma unroll
            for (int k = 0; k < kOthers; ++k)
                if (rot + lane + 32 * k < a.dim) {
                    if (BACK || norm)
                        elem_store<DT>(out, rot + lane + 32 * k, o[k]);
                    else   // as it is, to the bit
                        elem_copy<DT>(out, in, rot + lane + 32 * k);
                }
        }
    }
    if constexpr (BACK) {
        if (!r.slices)
            return;
        float* to = sums + threadIdx.x / 32 * kRotaryDim;
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            if (lane + 32 * k < half) {
                to[(lane + 32 * k) * step] = sa[k];
                to[(lane + 32 * k) * step + far] = sb[k];
            }
#pragma unroll
        for (int k = 0; k < kOthers; ++k)
            if (rot + lane + 32 * k < a.dim)
                to[rot + lane + 32 * k] = so[k];
        store_slice(r, a.dim, sums);
    }
}

// The weights' gradients from the CTAs' slices: 32 channels to a CTA, 32 threads
// to a channel, in an order that the number of slices fixes.
__global__ void __launch_bounds__(1024) rotary_weights_kernel(const __grid_constant__ RotaryArgs a, float* dq_weight,
                                                              float* dk_weight)
{
    __shared__ float part[32][33];
    const bool of_q = blockIdx.y == 0;
    float* to = of_q ? dq_weight : dk_weight;
    const float* slices = nullptr;
    int count = 0;
    for (int i = 0; i < a.roles; ++i)   // a role that has no heads is not there, and its gradient 0
        if ((a.role[i].which == 0) == of_q) {
            slices = a.role[i].slices;
            count = a.role[i].ctas;
        }
    wait_for_last();
    if (!to)
        return;
    const int ch = blockIdx.x * 32 + threadIdx.x % 32, row = threadIdx.x / 32;
    float v = 0.f;
    if (ch < a.dim && slices)
#pragma unroll 8
        for (int i = row; i < count; i += 32)
            v += slices[static_cast<int64_t>(i) * a.dim + ch];
    part[row][threadIdx.x % 32] = v;
    __syncthreads();
    v = part[threadIdx.x % 32][row];   // a warp to a channel
    v = team_sum(v, 32);
    if (threadIdx.x % 32 == 0 && blockIdx.x * 32 + row < a.dim)
        to[blockIdx.x * 32 + row] = v;
}

template <int DT, bool NORM, bool PAGED>
cudaError_t launch_vec(const RotaryArgs& a, int ctas, cudaStream_t st)
{
    if (a.layout == TSX_ROPE_INTERLEAVED)
        return launch_grid<rotary_kernel<DT, true, NORM, PAGED>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
    return launch_grid<rotary_kernel<DT, false, NORM, PAGED>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
}

template <int DT>
cudaError_t launch_forward(const RotaryArgs& a, bool vec, int ctas, cudaStream_t st)
{
    if (!vec)
        return launch_grid<rotary_any_kernel<DT, false>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
    if (a.positions)
        return a.norm ? launch_vec<DT, true, false>(a, ctas, st) : launch_vec<DT, false, false>(a, ctas, st);
    return a.norm ? launch_vec<DT, true, true>(a, ctas, st) : launch_vec<DT, false, true>(a, ctas, st);
}

template <int DT>
cudaError_t launch_backward(const RotaryArgs& a, bool vec, int ctas, cudaStream_t st)
{
    if (!vec)
        return launch_grid<rotary_any_kernel<DT, true>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
    if (a.layout == TSX_ROPE_INTERLEAVED)
        return launch_grid<rotary_norm_backward_kernel<DT, true>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
    return launch_grid<rotary_norm_backward_kernel<DT, false>>(dim3(unsigned(ctas)), kRotaryThreads, 0, 1, false, st, a);
}

}  // namespace

cudaError_t launch_rotary(int dtype, const RotaryArgs& a, bool vec, int ctas, cudaStream_t st)
{
    return dtype == TSX_F32    ? launch_forward<TSX_F32>(a, vec, ctas, st)
           : dtype == TSX_BF16 ? launch_forward<TSX_BF16>(a, vec, ctas, st)
                               : launch_forward<TSX_F16>(a, vec, ctas, st);
}

cudaError_t launch_rotary_norm_backward(int dtype, const RotaryArgs& a, bool vec, int ctas, cudaStream_t st)
{
    return dtype == TSX_F32    ? launch_backward<TSX_F32>(a, vec, ctas, st)
           : dtype == TSX_BF16 ? launch_backward<TSX_BF16>(a, vec, ctas, st)
                               : launch_backward<TSX_F16>(a, vec, ctas, st);
}

cudaError_t launch_rotary_weights(const RotaryArgs& a, float* dq_weight, float* dk_weight, cudaStream_t st)
{
    return launch_grid<rotary_weights_kernel>(dim3(unsigned((a.dim + 31) / 32), 2), 1024, 0, 1, true, st, a, dq_weight,
                                              dk_weight);
}

}  // namespace tsx
