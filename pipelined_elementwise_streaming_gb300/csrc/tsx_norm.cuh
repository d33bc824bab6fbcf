// Pieces shared by the group-norm kernels: where a thread works, sums over a
// CTA's threads by channel and by group, and what a thread keeps for its
// channels.
//
// For the M = l * (c / groups) elements of a sample's group:
//   forward   mean = sum x / M,  var = sum (x - mean)^2 / M,  rstd = 1 / sqrt(var + eps)
//             y = act(z),  z = (x - mean) rstd weight + bias
//   backward  dz = dy act'(z),  xhat = (x - mean) rstd
//             dbias = sum dz,  dweight = sum dz xhat  (over samples and rows)
//             dx = rstd (dz weight - S1 / M - xhat S2 / M)
//             S1 = sum dz weight,  S2 = sum dz weight xhat  (over the group)
//
// Variances are never taken as E[x^2] - mean^2, which loses every digit once
// the mean is large against the spread.  A thread takes the mean and the
// squared deviations of a few rows that it holds, and such (count, mean, M2)
// triples are combined pairwise:
//   mean = mean_a + (mean_b - mean_a) n_b / n,   n = n_a + n_b,
//   M2 = M2_a + M2_b + (mean_b - mean_a)^2 n_a n_b / n.
//
// A CTA adds in two steps, each in an order that its shape alone fixes: the
// row lanes of a channel (or oct) by halves, a tree of log2(lanes) steps
// through shared memory, then the channels of a group by a team of
// neighbouring threads with shuffles.
#pragma once

#include "tsx_oct.cuh"

namespace tsx {
namespace dev {

// A thread's place in its CTA: its channels (eight of a run) and its row
// lane.  Runs hold whole groups, or (pieces > 1) are part of one.
struct NormPlace {
    OctAt at;
    int p;        // row lane
    int ch0;      // the run's first channel
    int group0;   // the run's first group
    int groups;   // groups of the run
    int piece;    // which run of its group (0 unless a group is cut)
    bool live;    // the thread has channels
};

template <bool VEC>
__device__ __forceinline__ NormPlace norm_place(const NormArgs& a)
{
    const NormLayout& lay = a.lay;
    NormPlace s;
    s.p = static_cast<int>(threadIdx.x) / lay.V;
    const int v = static_cast<int>(threadIdx.x) - s.p * lay.V;
    int cols;
    if (lay.pieces == 1) {
        s.piece = 0;
        s.group0 = static_cast<int>(blockIdx.y) * lay.run_groups;
        s.groups = min(lay.run_groups, a.groups - s.group0);
        s.ch0 = s.group0 * a.per_group;
        cols = s.groups * a.per_group;
    } else {
        s.group0 = static_cast<int>(blockIdx.y) / lay.pieces;
        s.piece = static_cast<int>(blockIdx.y) - s.group0 * lay.pieces;
        s.groups = 1;
        s.ch0 = s.group0 * a.per_group + s.piece * lay.run_cols;
        cols = min(lay.run_cols, a.per_group - s.piece * lay.run_cols);
    }
    s.at = oct_at<VEC>(v, lay.team, cols);
    s.live = s.p < lay.P && s.at.ch < cols;
    return s;
}

// Columns of a run in the shared-memory sums: its octs (BY_OCT: eight
// consecutive channels always lie in one group) or its channels; and those of
// one group.
template <bool BY_OCT>
__device__ __forceinline__ int run_width(const NormPlace& s) { return BY_OCT ? s.at.cols / 8 : s.at.cols; }

__device__ __forceinline__ int group_cols(const NormArgs& a, const NormPlace& s)
{
    return a.lay.pieces == 1 ? a.per_group : s.at.cols;
}

// The group of a run's channel, counted within the run.
__device__ __forceinline__ int local_group(const NormArgs& a, int ch)
{
    return a.lay.pieces == 1 ? static_cast<int>(static_cast<unsigned>(ch) / static_cast<unsigned>(a.per_group)) : 0;
}

__device__ __forceinline__ int half_of(int lanes)   // the largest power of two below `lanes`
{
    int h = 1;
    while (2 * h < lanes)
        h *= 2;
    return h;
}

// N triples of a thread: `count` elements each, their mean and squared
// deviations.
template <int N>
struct Triples {
    float count, mean[N], m2[N];
    __device__ __forceinline__ void clear()
    {
        count = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            mean[k] = m2[k] = 0.f;
    }
    __device__ __forceinline__ void join(float n, const float (&mu)[N], const float (&dev)[N])
    {
        const float total = count + n;
        if (total == 0.f)
            return;
        const float w = n / total, cross = count * w;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float d = mu[k] - mean[k];
            mean[k] += d * w;
            m2[k] += dev[k] + d * d * cross;
        }
        count = total;
    }
    // The eight channels of `have` rows that the thread holds: their mean, then
    // their squared deviations from it.
    template <int ROWS>
    __device__ __forceinline__ void add_rows(const float (&f)[ROWS][8], int have)
    {
        float mu[N], dev[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            mu[k] = dev[k] = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (i < have) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mu[j % N] += f[i][j];
            }
        const float n = have * (8.f / N), each = 1.f / n;
#pragma unroll
        for (int k = 0; k < N; ++k)
            mu[k] *= each;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (i < have) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = f[i][j] - mu[j % N];
                    dev[j % N] += d * d;
                }
            }
        if (have)
            join(n, mu, dev);
    }
};

// The triples of the `lanes` row lanes that share a thread's channels, joined
// into lane `lane` 0's; slots: [P][width] pairs of shared memory.  All threads
// of the CTA call it.
template <int N>
__device__ __forceinline__ void join_lanes(const NormPlace& s, int lane, int lanes, float2* slots, float* counts,
                                           int width, Triples<N>& t)
{
    auto col = [&](int j) { return N == 1 ? s.at.ch / 8 : s.at.ch + j * s.at.step; };
    for (int half = half_of(lanes); lanes > 1 && half > 0; half >>= 1) {
        if (s.live && lane >= half && lane < 2 * half) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (N == 1 || s.at.ch + j * s.at.step < s.at.cols)
                    slots[s.p * width + col(j)] = make_float2(t.mean[j], t.m2[j]);
            counts[s.p] = t.count;   // the same from every thread of the lane
        }
        __syncthreads();
        if (s.live && lane < half && lane + half < lanes) {
            float mu[N], dev[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                mu[j] = dev[j] = 0.f;
                if (N == 1 || s.at.ch + j * s.at.step < s.at.cols) {
                    const float2 o = slots[(s.p + half) * width + col(j)];
                    mu[j] = o.x;
                    dev[j] = o.y;
                }
            }
            t.join(counts[s.p + half], mu, dev);
        }
    }
}

// The same for plain sums of pairs, channel by channel.
__device__ __forceinline__ void add_lanes(const NormPlace& s, int lane, int lanes, float2* slots, int width,
                                          float (&x)[8], float (&y)[8])
{
    for (int half = half_of(lanes); lanes > 1 && half > 0; half >>= 1) {
        if (s.live && lane >= half && lane < 2 * half) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s.at.ch + j * s.at.step < s.at.cols)
                    slots[s.p * width + s.at.ch + j * s.at.step] = make_float2(x[j], y[j]);
        }
        __syncthreads();
        if (s.live && lane < half && lane + half < lanes) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s.at.ch + j * s.at.step < s.at.cols) {
                    const float2 o = slots[(s.p + half) * width + s.at.ch + j * s.at.step];
                    x[j] += o.x;
                    y[j] += o.y;
                }
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int d = 1; d < lanes; d <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// f(item, lane, lanes, real) for `items` items of `entries` entries each, one
// team of threads (a power of two, at most 32) to an item; a team past the
// last item repeats it with `real` false.  Called by whole warps.
template <class F>
__device__ __forceinline__ void each_item(int items, int entries, F f)
{
    int lanes = 1;
    while (lanes < 32 && 2 * lanes <= entries)
        lanes *= 2;
    const int teams = static_cast<int>(blockDim.x) / lanes;
    const int me = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
    for (int i0 = 0; i0 < items; i0 += teams) {
        const int i = i0 + me;
        f(i < items ? i : items - 1, lane, lanes, i < items);
    }
}

// (mean, M2) of each of the `items` groups from `per` columns each, all of
// `count` elements: out[item].  columns: [item][per], as (mean, M2).
__device__ __forceinline__ void join_columns(const float2* columns, int items, int per, float count, float2* out)
{
    each_item(items, per, [&](int g, int lane, int lanes, bool real) {
        float sum = 0.f, dev = 0.f;
        for (int e = lane; e < per; e += lanes)
            sum += columns[g * per + e].x;
        const float mean = lanes_sum(sum, lanes) / per;
        for (int e = lane; e < per; e += lanes) {
            const float2 t = columns[g * per + e];
            const float d = t.x - mean;
            dev += t.y + count * d * d;
        }
        dev = lanes_sum(dev, lanes);
        if (real && lane == 0)
            out[g] = make_float2(mean, dev);
    });
}

__device__ __forceinline__ float rstd_of(float m2, float m, float eps) { return 1.f / sqrtf(m2 / m + eps); }

// One weight, as fp32.
template <int DT>
__device__ __forceinline__ float weight_at(const NormArgs& a, const void* weight, int ch)
{
    if (a.wide_params || DT == TSX_F32)
        return __ldg(static_cast<const float*>(weight) + ch);
    if constexpr (DT == TSX_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(weight)[ch]);
    else
        return __half2float(static_cast<const __half*>(weight)[ch]);
}

// (S1, S2) of each of the run's groups from its channels' sums of dz and dz
// xhat (columns: [run_cols]).
template <int DT>
__device__ __forceinline__ void weigh_columns(const NormArgs& a, const NormPlace& s, const void* weight,
                                              const float2* columns, float2* out)
{
    const int per = group_cols(a, s);
    each_item(s.groups, per, [&](int g, int lane, int lanes, bool real) {
        float s1 = 0.f, s2 = 0.f;
        for (int e = lane; e < per; e += lanes) {
            const int ch = g * per + e;
            const float w = weight_at<DT>(a, weight, s.ch0 + ch);
            s1 += w * columns[ch].x;
            s2 += w * columns[ch].y;
        }
        s1 = lanes_sum(s1, lanes);
        s2 = lanes_sum(s2, lanes);
        if (real && lane == 0)
            out[g] = make_float2(s1, s2);
    });
}

// What a thread keeps for its channels: mean and rstd of their groups, weight
// and bias.
template <bool BY_OCT>
struct Chan {
    float mean[BY_OCT ? 1 : 8], rstd[BY_OCT ? 1 : 8], w[8], b[8];
    __device__ __forceinline__ float mu(int j) const { return mean[BY_OCT ? 0 : j]; }
    __device__ __forceinline__ float rs(int j) const { return rstd[BY_OCT ? 0 : j]; }
    template <int DT, bool VEC>
    __device__ __forceinline__ void params(const NormArgs& a, const NormPlace& s, const void* weight,
                                           const void* bias)
    {
        param_floats<DT, VEC>(weight, a.wide_params, s.ch0, s.at, w);
        param_floats<DT, VEC>(bias, a.wide_params, s.ch0, s.at, b);
    }
    __device__ __forceinline__ void statistics(const NormArgs& a, const NormPlace& s, const float2* stats)
    {
#pragma unroll
        for (int j = 0; j < (BY_OCT ? 1 : 8); ++j) {
            const int ch = s.at.ch + j * s.at.step;
            const float2 t = stats[ch < s.at.cols ? local_group(a, ch) : 0];
            mean[j] = t.x;
            rstd[j] = t.y;
        }
    }
    template <int DT>
    __device__ __forceinline__ void apply(const NormArgs& a, const float (&x)[8], float (&y)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = act_value<DT>((x[j] - mu(j)) * rs(j) * w[j] + b[j], a.act);
    }
    // xhat and dz
    template <int DT>
    __device__ __forceinline__ void slopes(const NormArgs& a, const float (&dy)[8], const float (&x)[8],
                                           float (&hat)[8], float (&dz)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            hat[j] = (x[j] - mu(j)) * rs(j);
            float value, slope;
            act_both<DT>(hat[j] * w[j] + b[j], a.act, value, slope);
            dz[j] = dy[j] * slope;
        }
    }
};

// An oct to 8 bits, as the forward pass saves it.  By whole warps.
template <bool VEC>
__device__ __forceinline__ void hold(const NormArgs& a, const NormPlace& s, const float (&f)[8], bool live,
                                     int64_t row, const HeldOut& out)
{
    const uint32_t m = team_max(live ? oct_amax_bits(f) : 0u, a.lay.team);
    const HeldScale hs = held_scale(m, a.form);
    if (!live)
        return;
    held_store<VEC>(out.q, row * a.c + s.ch0, s.at, held_round(f, hs, a.form));
    const int ch = s.ch0 + s.at.ch;
    if (ch % a.block == 0)
        out.scale[row * a.blocks + ch / a.block] = hs.scale;
}

// What the backward pass loads of one row's oct.
template <int DT, bool VEC, bool HELD>
struct GradRow {
    Oct<DT> dy;
    Oct<DT> x;      // HELD: unused
    Held q;
    float scale[VEC ? 1 : 8];   // consecutive channels of an aligned oct share a block; others need not
    __device__ __forceinline__ void load(const NormArgs& a, const NormPlace& s, const void* pdy, const Saved& src,
                                         int64_t row)
    {
        dy = oct_load<DT, VEC>(pdy, row * a.y_pitch + s.ch0, s.at);
        if constexpr (HELD) {
            q = held_load<VEC>(src.q, row * a.c + s.ch0, s.at);
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 8); ++j) {
                const int ch = s.at.ch + j * s.at.step;
                scale[j] = ch < s.at.cols ? __ldg(src.scale + row * a.blocks + (s.ch0 + ch) / a.block) : 0.f;
            }
        } else {
            x = oct_load<DT, VEC>(src.x, row * a.x_pitch + s.ch0, s.at);
        }
    }
    __device__ __forceinline__ void floats(const NormArgs& a, float (&fd)[8], float (&fx)[8]) const
    {
        oct_floats(dy, fd);
        saved_floats(a, fx);
    }
    __device__ __forceinline__ void saved_floats(const NormArgs& a, float (&fx)[8]) const
    {
        if constexpr (!HELD) {
            oct_floats(x, fx);
        } else if constexpr (VEC) {
            held_floats(q, scale[0], a.form, fx);
        } else {
            held_floats(q, 1.f, a.form, fx);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                fx[j] *= scale[j];
        }
    }
};

}  // namespace dev

// f<DT, VEC, BY_OCT>(...) for the runtime type and layout.
#define TSX_BY_LAYOUT(dtype, lay, CALL)                                                        \
    do {                                                                                       \
        const int kind = (lay).oct_in_group ? 2 : (lay).vec ? 1 : 0;                           \
        if ((dtype) == TSX_F16) {                                                              \
            if (kind == 2) { CALL(TSX_F16, true, true); }                                      \
            else if (kind == 1) { CALL(TSX_F16, true, false); }                                \
            else { CALL(TSX_F16, false, false); }                                              \
        } else if ((dtype) == TSX_BF16) {                                                      \
            if (kind == 2) { CALL(TSX_BF16, true, true); }                                     \
            else if (kind == 1) { CALL(TSX_BF16, true, false); }                               \
            else { CALL(TSX_BF16, false, false); }                                             \
        } else {                                                                               \
            if (kind == 2) { CALL(TSX_F32, true, true); }                                      \
            else if (kind == 1) { CALL(TSX_F32, true, false); }                                \
            else { CALL(TSX_F32, false, false); }                                              \
        }                                                                                      \
    } while (0)

}  // namespace tsx
