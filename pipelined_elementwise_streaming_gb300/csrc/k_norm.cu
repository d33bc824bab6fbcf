// Group norm with an activation over channels-last tensors, and its gradient.
//
// For the M = l * (c / groups) elements of a sample's group:
//   forward   mean = sum x / M,  var = sum (x - mean)^2 / M,  rstd = 1 / sqrt(var + eps)
//             y = act(z),  z = (x - mean) rstd weight + bias
//   backward  dz = dy act'(z),  xhat = (x - mean) rstd
//             dbias = sum dz,  dweight = sum dz xhat  (over samples and rows)
//             dx = rstd (dz weight - S1 / M - xhat S2 / M)
//             S1 = sum dz weight,  S2 = sum dz weight xhat  (over the group)
// The streaming pair of kernels reads its operands twice: one kernel sums,
// the next applies.  HBM bounds both; the second read comes out of L2 where
// the tensor fits there.
//
// Variances are never taken as E[x^2] - mean^2, which loses every digit once
// the mean is large against the spread.  A thread takes the mean and the
// squared deviations of a few rows that it holds, and such (count, mean, M2)
// triples are combined pairwise: with m the joint mean,
//   M2 = M2_a + M2_b + n_a (mean_a - m)^2 + n_b (mean_b - m)^2.

#include "tsx_oct.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kRowsAtOnce = 4;

// A thread's place in its CTA's run of channels and range of rows.
struct NormPlace {
    OctAt at;
    int p;              // the thread's first row within the range
    int ch0;            // the run's first channel
    int group0;         // the run's first group
    int groups;         // groups of the run
    int piece;          // which run of its group (0 unless a group is cut)
    int64_t sample, split;
    int64_t row0;       // the range's first row, counted through all samples
    int64_t rows;       // rows of the range
    bool live;
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
    s.sample = static_cast<int64_t>(blockIdx.x) / lay.splits;
    s.split = static_cast<int64_t>(blockIdx.x) - s.sample * lay.splits;
    s.row0 = s.sample * a.l + s.split * lay.range;
    s.rows = min(lay.range, a.l - s.split * lay.range);
    return s;
}

// Rows of a range that the threads of row lane p take: p, p + P, ...
__device__ __forceinline__ int64_t rows_of_lane(int64_t rows, int p, int P)
{
    return rows > p ? (rows - p + P - 1) / P : 0;
}

// The group of a run's channel, counted within the run.
__device__ __forceinline__ int local_group(const NormArgs& a, int ch) { return a.lay.pieces == 1 ? ch / a.per_group : 0; }

// Sums over a CTA's threads, group by group.  Each thread has left a pair for
// its oct (BY_OCT: eight consecutive channels of one group) or for each of
// its channels in `slots`, [P][width] with width = octs or channels of the
// run; a group owns `per` neighbouring columns of it.  Teams of `lanes`
// threads add a group's entries, always in the same order.
__device__ __forceinline__ int lanes_for(int entries)
{
    int lanes = 1;
    while (lanes < 32 && 2 * lanes <= entries)
        lanes *= 2;
    return lanes;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int d = 1; d < lanes; d <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// f(group, lane, lanes) for every group of the run, by whole warps; a team
// past the last group repeats it, with `real` false.
template <class F>
__device__ __forceinline__ void each_group(int groups, int entries, F f)
{
    const int lanes = lanes_for(entries);
    const int teams = static_cast<int>(blockDim.x) / lanes;
    const int me = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
    for (int g0 = 0; g0 < groups; g0 += teams) {
        const int g = g0 + me;
        f(g < groups ? g : groups - 1, lane, lanes, g < groups);
    }
}

// Channels (as the run counts them) that a group owns in a piece.
__device__ __forceinline__ int group_cols(const NormArgs& a, const NormPlace& s)
{
    return a.lay.pieces == 1 ? a.per_group : s.at.cols;
}

// ------------------------------------------------------------- forward

// First kernel: (mean, M2) of every range, run and group.
template <int DT, bool VEC, bool BY_OCT>
__global__ void __launch_bounds__(kLayerThreads) norm_stats_kernel(NormArgs a, const void* x, float2* part)
{
    extern __shared__ float2 slots[];
    const NormPlace s = norm_place<VEC>(a);
    constexpr int N = BY_OCT ? 1 : 8;   // running triples of a thread
    const int P = a.lay.P;
    float mean[N], m2[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        mean[k] = m2[k] = 0.f;
    float count = 0.f;   // rows so far
    for (int64_t r0 = s.p; s.live && r0 < s.rows; r0 += int64_t(kRowsAtOnce) * P) {
        Oct<DT> o[kRowsAtOnce];
        int have = 0;
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (r0 + i * P < s.rows) {
                o[i] = oct_load<DT, VEC>(x, (s.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at);
                have = i + 1;
            }
        float f[kRowsAtOnce][8], sum[N], dev[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] = dev[k] = 0.f;
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (i < have) {
                oct_floats(o[i], f[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum[BY_OCT ? 0 : j] += f[i][j];
            }
        const float each = 1.f / (have * (BY_OCT ? 8.f : 1.f));
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] *= each;   // now the batch's mean
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (i < have) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = f[i][j] - sum[BY_OCT ? 0 : j];
                    dev[BY_OCT ? 0 : j] += d * d;
                }
            }
        // a batch mean that is off by a rounding shifts dev by its square only
        const float total = count + have;
        const float w = have / total, cross = count * w * (BY_OCT ? 8.f : 1.f);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float d = sum[k] - mean[k];
            mean[k] += d * w;
            m2[k] += dev[k] + d * d * cross;
        }
        count = total;
    }
    const int width = BY_OCT ? s.at.cols / 8 : s.at.cols;
    if (s.live) {
        if constexpr (BY_OCT) {
            slots[s.p * width + s.at.ch / 8] = make_float2(mean[0], m2[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s.at.ch + j * s.at.step < s.at.cols)
                    slots[s.p * width + s.at.ch + j * s.at.step] = make_float2(mean[j], m2[j]);
        }
    }
    __syncthreads();
    const int per = BY_OCT ? group_cols(a, s) / 8 : group_cols(a, s);
    const int entries = P * per;
    each_group(s.groups, entries, [&](int g, int lane, int lanes, bool real) {
        float sum = 0.f, dev = 0.f;
        for (int e = lane; e < entries; e += lanes) {
            const int p = e / per;
            const float n = static_cast<float>(rows_of_lane(s.rows, p, P));
            sum += n * slots[p * width + g * per + e - p * per].x;
        }
        const float mean_g = lanes_sum(sum, lanes) / (static_cast<float>(s.rows) * per);
        for (int e = lane; e < entries; e += lanes) {
            const int p = e / per;
            const float n = static_cast<float>(rows_of_lane(s.rows, p, P)) * (BY_OCT ? 8.f : 1.f);
            const float2 t = slots[p * width + g * per + e - p * per];
            const float d = t.x - mean_g;
            dev += t.y + n * d * d;
        }
        dev = lanes_sum(dev, lanes);
        if (real && lane == 0) {
            const int64_t at = (s.sample * a.lay.splits + s.split) * a.lay.pieces + s.piece;
            part[at * a.groups + s.group0 + g] = make_float2(mean_g, dev);
        }
    });
}

// The statistics of the run's groups from their parts, into `stats` [groups]
// as (mean, rstd).  Ends with the CTA synchronised.
__device__ __forceinline__ void join_stats(const NormArgs& a, const NormPlace& s, const float2* part, float2* stats)
{
    const int64_t count = a.lay.splits * a.lay.pieces;
    const float2* first = part + s.sample * count * a.groups + s.group0;
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    each_group(s.groups, count < 32 ? int(count) : 32, [&](int g, int lane, int lanes, bool real) {
        // elements of part k
        auto size = [&](int64_t k) {
            const int64_t split = k / a.lay.pieces;
            const int piece = static_cast<int>(k - split * a.lay.pieces);
            const int64_t rows = min(a.lay.range, a.l - split * a.lay.range);
            const int cols = a.lay.pieces == 1 ? a.per_group : min(a.lay.run_cols, a.per_group - piece * a.lay.run_cols);
            return static_cast<float>(rows) * static_cast<float>(cols);
        };
        float sum = 0.f, dev = 0.f;
        for (int64_t k = lane; k < count; k += lanes)
            sum += first[k * a.groups + g].x * (size(k) / m);
        const float mean = lanes_sum(sum, lanes);
        for (int64_t k = lane; k < count; k += lanes) {
            const float2 t = first[k * a.groups + g];
            const float d = t.x - mean;
            dev += t.y + size(k) * d * d;
        }
        dev = lanes_sum(dev, lanes);
        if (real && lane == 0)
            stats[g] = make_float2(mean, 1.f / sqrtf(dev / m + a.eps));
    });
    __syncthreads();
}

// What a thread keeps for its channels: mean and rstd of their groups, weight
// and bias.
template <bool BY_OCT>
struct Chan {
    float mean[BY_OCT ? 1 : 8], rstd[BY_OCT ? 1 : 8], w[8], b[8];
    __device__ __forceinline__ float mu(int j) const { return mean[BY_OCT ? 0 : j]; }
    __device__ __forceinline__ float rs(int j) const { return rstd[BY_OCT ? 0 : j]; }
};

template <int DT, bool VEC, bool BY_OCT>
__device__ __forceinline__ void chan_params(const NormArgs& a, const NormPlace& s, const void* weight,
                                            const void* bias, Chan<BY_OCT>& k)
{
    param_floats<DT, VEC>(weight, a.wide_params, s.ch0, s.at, k.w);
    param_floats<DT, VEC>(bias, a.wide_params, s.ch0, s.at, k.b);
}

template <bool BY_OCT>
__device__ __forceinline__ void chan_stats(const NormArgs& a, const NormPlace& s, const float2* stats,
                                           Chan<BY_OCT>& k)
{
#pragma unroll
    for (int j = 0; j < (BY_OCT ? 1 : 8); ++j) {
        const int ch = s.at.ch + j * s.at.step;
        const float2 t = stats[ch < s.at.cols ? local_group(a, ch) : 0];
        k.mean[j] = t.x;
        k.rstd[j] = t.y;
    }
}

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

// Second kernel: y, and with HOLD the checkpoint of x.
template <int DT, bool VEC, bool BY_OCT, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_apply_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held, const float2* part)
{
    extern __shared__ float2 stats[];
    const NormPlace s = norm_place<VEC>(a);
    Chan<BY_OCT> k;
    chan_params<DT, VEC, BY_OCT>(a, s, weight, bias, k);
    join_stats(a, s, part, stats);
    chan_stats<BY_OCT>(a, s, stats, k);
    if (s.split == 0 && s.piece == 0)
        for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
            mean[s.sample * a.groups + s.group0 + g] = stats[g].x;
            rstd[s.sample * a.groups + s.group0 + g] = stats[g].y;
        }
    const int P = a.lay.P;
    // whole warps walk together: the teams' shuffles need every lane
    for (int64_t base = 0; base < s.rows; base += int64_t(kRowsAtOnce) * P) {
        const int64_t r0 = base + s.p;
        Oct<DT> o[kRowsAtOnce];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (s.live && r0 + i * P < s.rows)
                o[i] = oct_load<DT, VEC>(x, (s.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at);
            else
                oct_zero(o[i]);
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int64_t row = s.row0 + r0 + i * P;
            const bool live = s.live && r0 + i * P < s.rows;
            float f[8], out[8];
            oct_floats(o[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                out[j] = act_value<DT>((f[j] - k.mu(j)) * k.rs(j) * k.w[j] + k.b[j], a.act);
            if (live)
                oct_store<DT, VEC>(y, row * a.y_pitch + s.ch0, s.at, oct_round<DT>(out));
            if constexpr (HOLD)
                hold<VEC>(a, s, f, live, row, held);
        }
    }
}

// ------------------------------------------------------------ backward

// What a thread loads of one row.
template <int DT, bool HELD>
struct GradRow {
    Oct<DT> dy;
    Oct<DT> x;      // HELD: unused
    Held q;
    float scale[HELD ? 8 : 1];
};

template <int DT, bool VEC, bool HELD>
__device__ __forceinline__ void grad_load(const NormArgs& a, const NormPlace& s, const void* dy, const Saved& x,
                                          int64_t row, GradRow<DT, HELD>& g)
{
    g.dy = oct_load<DT, VEC>(dy, row * a.y_pitch + s.ch0, s.at);
    if constexpr (HELD) {
        g.q = held_load<VEC>(x.q, row * a.c + s.ch0, s.at);
        // consecutive channels of an aligned oct share a block; others need not
#pragma unroll
        for (int j = 0; j < (VEC ? 1 : 8); ++j) {
            const int ch = s.at.ch + j * s.at.step;
            g.scale[j] = ch < s.at.cols ? __ldg(x.scale + row * a.blocks + (s.ch0 + ch) / a.block) : 0.f;
        }
    } else {
        g.x = oct_load<DT, VEC>(x.x, row * a.x_pitch + s.ch0, s.at);
    }
}

template <int DT, bool VEC, bool HELD>
__device__ __forceinline__ void grad_floats(const NormArgs& a, const GradRow<DT, HELD>& g, float (&dy)[8],
                                            float (&x)[8])
{
    oct_floats(g.dy, dy);
    if constexpr (!HELD) {
        oct_floats(g.x, x);
    } else if constexpr (VEC) {
        held_floats(g.q, g.scale[0], a.form, x);
    } else {
        held_floats(g.q, 1.f, a.form, x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] *= g.scale[j];
    }
}

__device__ __forceinline__ void load_stats(const NormArgs& a, const NormPlace& s, const float* mean, const float* rstd,
                                           float2* stats)
{
    for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
        const int64_t at = s.sample * a.groups + s.group0 + g;
        stats[g] = make_float2(mean[at], rstd[at]);
    }
    __syncthreads();
}

// First kernel: S1 and S2 of every range, run and group, and the range's sums
// for dweight and dbias.
template <int DT, bool VEC, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_sums_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, float2* part, float* chan)
{
    extern __shared__ float2 shared[];
    const NormPlace s = norm_place<VEC>(a);
    float2* stats = shared;                       // [run_groups]
    float2* slots = shared + a.lay.run_groups;    // [P][run_cols]
    Chan<BY_OCT> k;
    chan_params<DT, VEC, BY_OCT>(a, s, weight, bias, k);
    load_stats(a, s, mean, rstd, stats);
    chan_stats<BY_OCT>(a, s, stats, k);
    float sz[8], szx[8];   // sums of dz and dz xhat, channel by channel
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sz[j] = szx[j] = 0.f;
    const int P = a.lay.P;
    for (int64_t r0 = s.p; s.live && r0 < s.rows; r0 += 2 * P) {
        GradRow<DT, HELD> g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + i * P < s.rows)
                grad_load<DT, VEC, HELD>(a, s, dy, x, s.row0 + r0 + i * P, g[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + i * P < s.rows) {
                float fd[8], fx[8];
                grad_floats<DT, VEC, HELD>(a, g[i], fd, fx);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = (fx[j] - k.mu(j)) * k.rs(j);
                    float value, slope;
                    act_both<DT>(hat * k.w[j] + k.b[j], a.act, value, slope);
                    const float dz = fd[j] * slope;
                    sz[j] += dz;
                    szx[j] += dz * hat;
                }
            }
    }
    // channel by channel over the row lanes, then group by group
    const int width = s.at.cols;
    if (s.live)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s.at.ch + j * s.at.step < width)
                slots[s.p * width + s.at.ch + j * s.at.step] = make_float2(sz[j], szx[j]);
    __syncthreads();
    float* out = chan + (s.sample * a.lay.splits + s.split) * 2 * a.c + s.ch0;
    for (int ch = threadIdx.x; ch < width; ch += blockDim.x) {
        float2 t = slots[ch];
        for (int p = 1; p < P; ++p) {
            const float2 u = slots[p * width + ch];
            t.x += u.x;
            t.y += u.y;
        }
        slots[ch] = t;
        out[ch] = t.y;
        out[a.c + ch] = t.x;
    }
    __syncthreads();
    const int per = group_cols(a, s);
    each_group(s.groups, per, [&](int g, int lane, int lanes, bool real) {
        float s1 = 0.f, s2 = 0.f;
        for (int e = lane; e < per; e += lanes) {
            const int ch = g * per + e;
            const float2 t = slots[ch];
            float w;
            if (a.wide_params || DT == TSX_F32)
                w = __ldg(static_cast<const float*>(weight) + s.ch0 + ch);
            else if constexpr (DT == TSX_BF16)
                w = __bfloat162float(static_cast<const __nv_bfloat16*>(weight)[s.ch0 + ch]);
            else
                w = __half2float(static_cast<const __half*>(weight)[s.ch0 + ch]);
            s1 += w * t.x;
            s2 += w * t.y;
        }
        s1 = lanes_sum(s1, lanes);
        s2 = lanes_sum(s2, lanes);
        if (real && lane == 0) {
            const int64_t at = (s.sample * a.lay.splits + s.split) * a.lay.pieces + s.piece;
            part[at * a.groups + s.group0 + g] = make_float2(s1, s2);
        }
    });
}

// Second kernel: dx.
template <int DT, bool VEC, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, void* dx, const float2* part)
{
    extern __shared__ float2 shared[];
    const NormPlace s = norm_place<VEC>(a);
    float2* stats = shared;                      // [run_groups]
    float2* sums = shared + a.lay.run_groups;    // [run_groups]: S1 / M, S2 / M
    Chan<BY_OCT> k;
    chan_params<DT, VEC, BY_OCT>(a, s, weight, bias, k);
    const int64_t count = a.lay.splits * a.lay.pieces;
    const float2* first = part + s.sample * count * a.groups + s.group0;
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    each_group(s.groups, count < 32 ? int(count) : 32, [&](int g, int lane, int lanes, bool real) {
        float s1 = 0.f, s2 = 0.f;
        for (int64_t i = lane; i < count; i += lanes) {
            const float2 t = first[i * a.groups + g];
            s1 += t.x;
            s2 += t.y;
        }
        s1 = lanes_sum(s1, lanes);
        s2 = lanes_sum(s2, lanes);
        if (real && lane == 0)
            sums[g] = make_float2(s1 / m, s2 / m);
    });
    load_stats(a, s, mean, rstd, stats);   // synchronises
    chan_stats<BY_OCT>(a, s, stats, k);
    float s1[BY_OCT ? 1 : 8], s2[BY_OCT ? 1 : 8];
#pragma unroll
    for (int j = 0; j < (BY_OCT ? 1 : 8); ++j) {
        const int ch = s.at.ch + j * s.at.step;
        const float2 t = sums[ch < s.at.cols ? local_group(a, ch) : 0];
        s1[j] = t.x;
        s2[j] = t.y;
    }
    const int P = a.lay.P;
    for (int64_t r0 = s.p; s.live && r0 < s.rows; r0 += 2 * P) {
        GradRow<DT, HELD> g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + i * P < s.rows)
                grad_load<DT, VEC, HELD>(a, s, dy, x, s.row0 + r0 + i * P, g[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + i * P < s.rows) {
                float fd[8], fx[8], out[8];
                grad_floats<DT, VEC, HELD>(a, g[i], fd, fx);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = (fx[j] - k.mu(j)) * k.rs(j);
                    float value, slope;
                    act_both<DT>(hat * k.w[j] + k.b[j], a.act, value, slope);
                    out[j] = k.rs(j) * (fd[j] * slope * k.w[j] - s1[BY_OCT ? 0 : j] - hat * s2[BY_OCT ? 0 : j]);
                }
                oct_store<DT, VEC>(dx, (s.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at, oct_round<DT>(out));
            }
    }
}

// dweight and dbias: the sums of the [slices][2][c] partial sums, slice after
// slice within each of eight row lanes, then lane after lane.
constexpr int kParamCols = 32, kParamLanes = 8;
__global__ void __launch_bounds__(kParamCols* kParamLanes)
    norm_params_kernel(const float* chan, int64_t slices, int c, float* dweight, float* dbias)
{
    __shared__ float part[kParamLanes][kParamCols];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kParamCols + threadIdx.x;   // of 2 c
    float t = 0.f;
    if (col < 2 * static_cast<int64_t>(c)) {
#pragma unroll 8
        for (int64_t i = threadIdx.y; i < slices; i += kParamLanes)
            t += __ldg(chan + i * 2 * c + col);
    }
    part[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && col < 2 * static_cast<int64_t>(c)) {
        for (int i = 1; i < kParamLanes; ++i)
            t += part[i][threadIdx.x];
        if (col < c)
            dweight[col] = t;
        else
            dbias[col - c] = t;
    }
}

__global__ void norm_empty_kernel(float* mean, float* rstd, int64_t count, float eps)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        mean[i] = 0.f;
        rstd[i] = 1.f / sqrtf(eps);
    }
}

}  // namespace

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

cudaError_t launch_norm(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                        float* mean, float* rstd, HeldOut held, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const size_t slots = size_t(lay.P) * (lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols) * sizeof(float2);
    const size_t stats = size_t(lay.run_groups) * sizeof(float2);
#define CALL(DT, VEC, BY_OCT) \
    norm_stats_kernel<DT, VEC, BY_OCT><<<grid, lay.threads, slots, st>>>(a, x, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
#define CALL(DT, VEC, BY_OCT)                                                                                \
    if (held.q)                                                                                              \
        norm_apply_kernel<DT, VEC, BY_OCT, true>                                                             \
            <<<grid, lay.threads, stats, st>>>(a, x, weight, bias, y, mean, rstd, held, scratch.part);       \
    else                                                                                                     \
        norm_apply_kernel<DT, VEC, BY_OCT, false>                                                            \
            <<<grid, lay.threads, stats, st>>>(a, x, weight, bias, y, mean, rstd, held, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_norm_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                 const void* bias, const float* mean, const float* rstd, void* dx, float* dweight,
                                 float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const size_t sums = (size_t(lay.run_groups) + size_t(lay.P) * lay.run_cols) * sizeof(float2);
#define CALL(DT, VEC, BY_OCT)                                                                                    \
    if (x.q)                                                                                                     \
        norm_sums_kernel<DT, VEC, BY_OCT, true><<<grid, lay.threads, sums, st>>>(a, dy, x, weight, bias, mean,    \
                                                                                 rstd, scratch.part, scratch.chan); \
    else                                                                                                         \
        norm_sums_kernel<DT, VEC, BY_OCT, false><<<grid, lay.threads, sums, st>>>(a, dy, x, weight, bias, mean,   \
                                                                                  rstd, scratch.part, scratch.chan)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const size_t stats = 2 * size_t(lay.run_groups) * sizeof(float2);
#define CALL(DT, VEC, BY_OCT)                                                                               \
    if (x.q)                                                                                                \
        norm_grad_kernel<DT, VEC, BY_OCT, true>                                                             \
            <<<grid, lay.threads, stats, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.part);       \
    else                                                                                                    \
        norm_grad_kernel<DT, VEC, BY_OCT, false>                                                            \
            <<<grid, lay.threads, stats, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int64_t cols = 2 * int64_t(a.c);
    norm_params_kernel<<<unsigned((cols + kParamCols - 1) / kParamCols), dim3(kParamCols, kParamLanes), 0, st>>>(
        scratch.chan, a.n * lay.splits, a.c, dweight, dbias);
    return cudaGetLastError();
}

cudaError_t launch_norm_empty(float* mean, float* rstd, int64_t count, float eps, cudaStream_t st)
{
    const int64_t blocks = (count + 255) / 256;
    norm_empty_kernel<<<unsigned(blocks < 1024 ? blocks : 1024), 256, 0, st>>>(mean, rstd, count, eps);
    return cudaGetLastError();
}

}  // namespace tsx
