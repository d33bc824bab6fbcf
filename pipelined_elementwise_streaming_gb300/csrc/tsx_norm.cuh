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
// A CTA adds in an order that its shape alone fixes: threads leave what they
// have of their channels (or octs) in shared memory, and warps join a group's
// columns over all row lanes.
#pragma once

#include <type_traits>

#include "tsx_device.cuh"
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
    s.p = lane_of(threadIdx.x, lay.per_v);
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

// ------------------------------------------------------------- clusters

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The place that `p` has in this CTA, in the cluster's CTA `rank`.
__device__ __forceinline__ void cluster_put(const float2* p, int rank, float2 v)
{
    const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(there), "f"(v.x), "f"(v.y) : "memory");
}

// Programmatic launches: a kernel lets the next one of the stream start once
// all its CTAs have said so (or ended), and that one waits for it to end, its
// memory visible, before it uses what it wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Rows of the k-th range of `range` rows of a sample (0 past its end).
__device__ __forceinline__ int range_rows(const NormArgs& a, int64_t range, int64_t k)
{
    const int64_t left = a.l - k * range;
    return static_cast<int>(left < 0 ? 0 : left < range ? left : range);
}

// ------------------------------------------------- means and deviations

// What a thread has of its channels: `count` elements each, their mean and
// squared deviations.  BY_OCT: one triple for the eight channels together.
template <bool BY_OCT>
struct Triples {
    static constexpr int N = BY_OCT ? 1 : 4;
    using V = typename std::conditional<BY_OCT, float, float2>::type;
    float count;
    V mean[N], m2[N];
    static __device__ __forceinline__ V zero()
    {
        if constexpr (BY_OCT)
            return 0.f;
        else
            return make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ void clear()
    {
        count = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            mean[k] = m2[k] = zero();
    }
    __device__ __forceinline__ void join(float n, const V (&mu)[N], const V (&dev)[N])
    {
        const float total = count + n;
        if (total == 0.f)
            return;
        const float w = __fdividef(n, total), cross = count * w;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (BY_OCT) {
                const float d = mu[k] - mean[k];
                mean[k] += d * w;
                m2[k] += dev[k] + d * d * cross;
            } else {
                const float2 d = __ffma2_rn(mean[k], pair_of(-1.f), mu[k]);
                mean[k] = __ffma2_rn(d, pair_of(w), mean[k]);
                m2[k] = __ffma2_rn(__fmul2_rn(d, d), pair_of(cross), __fadd2_rn(m2[k], dev[k]));
            }
        }
        count = total;
    }
    // ROWS rows of the thread's channels, of which the first `have` count (all
    // are finite zeros beyond): their mean, then their squared deviations.
    template <int ROWS, bool ALL>
    __device__ __forceinline__ void add_rows(const float2 (&f)[ROWS][4], int have)
    {
        float2 sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum[j] = f[0][j];
#pragma unroll
            for (int i = 1; i < ROWS; ++i)
                sum[j] = __fadd2_rn(sum[j], f[i][j]);
        }
        const float n = (ALL ? ROWS : have) * (BY_OCT ? 8.f : 1.f), each = 1.f / n;
        float2 minus[4];   // minus the mean
        V mu[N], dev[N];
        if constexpr (BY_OCT) {
            const float2 t = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
            mu[0] = (t.x + t.y) * each;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                minus[j] = pair_of(-mu[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mu[j] = __fmul2_rn(sum[j], pair_of(each));
                minus[j] = __fmul2_rn(mu[j], pair_of(-1.f));
            }
        }
        float2 sq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sq[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (ALL || i < have) {
                    const float2 d = __fadd2_rn(f[i][j], minus[j]);
                    sq[j] = __ffma2_rn(d, d, sq[j]);
                }
        }
        if constexpr (BY_OCT) {
            const float2 t = __fadd2_rn(__fadd2_rn(sq[0], sq[1]), __fadd2_rn(sq[2], sq[3]));
            dev[0] = t.x + t.y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dev[j] = sq[j];
        }
        if (ALL || have)
            join(n, mu, dev);
    }
    // The first `have` of N rows' octs, four at a time.
    template <int DT, int ROWS>
    __device__ __forceinline__ void add_octs(const Oct<DT> (&o)[ROWS], int have)
    {
#pragma unroll
        for (int i0 = 0; i0 < ROWS; i0 += 4) {
            float2 f[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                oct_floats(o[i0 + i], f[i]);
            if (have >= i0 + 4)
                add_rows<4, true>(f, 4);
            else if (have > i0)
                add_rows<4, false>(f, have - i0);
        }
    }
    // To a row of shared-memory columns (octs or channels) as (mean, M2).
    __device__ __forceinline__ void leave(const OctAt& at, float2* row) const
    {
        if constexpr (BY_OCT) {
            row[at.ch / 8] = make_float2(mean[0], m2[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at.ch + 2 * j * at.step < at.cols)
                    row[at.ch + 2 * j * at.step] = make_float2(mean[j].x, m2[j].x);
                if (at.ch + (2 * j + 1) * at.step < at.cols)
                    row[at.ch + (2 * j + 1) * at.step] = make_float2(mean[j].y, m2[j].y);
            }
        }
    }
};

// Row of the shared-memory columns: odd, so that the row lanes of one column
// lie in different banks.
__host__ __device__ constexpr int slot_stride(int width) { return width | 1; }

__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int d = 1; d < lanes; d <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// (mean, M2) of each of `samples` x `groups` items from the columns that the
// row lanes left: slots[samples * lanes][slot_stride], which it overwrites;
// `per` neighbouring columns to a group, `scale` elements to a column and row,
// `rows` rows dealt to the lanes in turn.  In two steps: threads side by side
// join side by side columns, each over a share of the lanes, with all its
// loads on their way at once; then a team of threads to an item, up to a warp,
// joins its columns' shares.  One step, a team to an item over all lanes, took 3.9 us of the
// 18.8 of f16 [8, 4096, 320], a chain of 13 dependent rounds.  Called by all
// threads after a barrier; ends without one.
__device__ __forceinline__ void join_groups(const NormLayout& lay, float2* slots, int stride, int samples, int groups,
                                            int lanes, int per, int rows, float scale, float2* out)
{
    const int threads = static_cast<int>(blockDim.x), items = samples * groups, width = groups * per;
    const int all = samples * width, len = lay.share_lanes, shares = lay.shares;
    const int base = rows / lanes, more = rows - base * lanes;   // lane p has base + (p < more) rows
    const float less = base * scale, much = less + scale;
    if (len > 1) {
        for (int i = threadIdx.x; i < shares * all; i += threads) {
            const int share = shares == 1 ? 0 : i / all, col = i - share * all;
            const int q = samples == 1 ? 0 : col / width;
            const int p0 = share * len, p1 = min(p0 + len, lanes);
            float2* first = slots + q * lanes * stride + col - q * width;
            float sum = 0.f, dev = 0.f;
#pragma unroll 4
            for (int p = p0; p < p1; ++p)
                sum += (p < more ? much : less) * first[p * stride].x;
            const float n = ((p1 - p0) * base + max(min(more, p1) - p0, 0)) * scale;
            const float mean = n > 0.f ? __fdividef(sum, n) : 0.f;
#pragma unroll 4
            for (int p = p0; p < p1; ++p) {
                const float2 v = first[p * stride];
                const float d = v.x - mean;
                dev += v.y + (p < more ? much : less) * d * d;
            }
            first[p0 * stride] = make_float2(mean, dev);
        }
        __syncthreads();
    }
    int shift = 5;   // log2 of the team
    while (shift > 0 && (threads >> shift) < items)
        --shift;
    const int team = 1 << shift, teams = threads >> shift;
    const int me = static_cast<int>(threadIdx.x) >> shift, t = static_cast<int>(threadIdx.x) & (team - 1);
    int wide = 0;   // log2 of the team's threads side by side along a row
    while (wide < shift && (1 << wide) < per)
        ++wide;
    const int k0 = t & ((1 << wide) - 1), s0 = t >> wide, step = team >> wide;
    for (int i0 = 0; i0 < items; i0 += teams) {
        const int item = min(i0 + me, items - 1);   // spare teams repeat the last
        const int q = samples == 1 ? 0 : item / groups, g = item - q * groups;
        const float2* first = slots + q * lanes * stride + g * per;
        float n = 0.f, sum = 0.f, dev = 0.f;
        for (int share = s0; share < shares; share += step) {
            const int p0 = share * len, p1 = min(p0 + len, lanes);
            const float c = ((p1 - p0) * base + max(min(more, p1) - p0, 0)) * scale;
            for (int k = k0; k < per; k += 1 << wide) {
                n += c;
                sum += c * first[p0 * stride + k].x;
            }
        }
        for (int d = 1; d < team; d <<= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, d);
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
        const float mean = n > 0.f ? __fdividef(sum, n) : 0.f;
        for (int share = s0; share < shares; share += step) {
            const int p0 = share * len, p1 = min(p0 + len, lanes);
            const float c = ((p1 - p0) * base + max(min(more, p1) - p0, 0)) * scale;
            for (int k = k0; k < per; k += 1 << wide) {
                const float2 v = first[p0 * stride + k];
                const float d = v.x - mean;
                dev += v.y + c * d * d;
            }
        }
        dev = lanes_sum(dev, team);
        if (t == 0 && i0 + me < items)
            out[item] = make_float2(mean, dev);
    }
}

// (mean, M2) of the parts v[0], v[step], ... of the ranges of `range` rows that
// `rows` rows make, `per` elements to a row.
__device__ __forceinline__ float2 join_ranges(const float2* v, int step, int count, int rows, int range, float per)
{
    float n = 0.f, sum = 0.f, dev = 0.f;
    int left = rows;
#pragma unroll 4
    for (int r = 0; r < count; ++r) {
        const float c = static_cast<float>(min(left, range));
        n += c;
        sum += c * v[r * step].x;
        left = max(left - range, 0);
    }
    const float mean = n > 0.f ? __fdividef(sum, n) : 0.f;
    left = rows;
#pragma unroll 4
    for (int r = 0; r < count; ++r) {
        const float2 u = v[r * step];
        const float d = u.x - mean;
        dev += u.y + static_cast<float>(min(left, range)) * per * d * d;
        left = max(left - range, 0);
    }
    return make_float2(mean, dev);
}

// --------------------------------------------------------- sums of pairs

// A thread's sums of its eight channels, two each, to its row of columns.
__device__ __forceinline__ void leave_sums(const OctAt& at, const float2 (&x)[4], const float2 (&y)[4], float2* row)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (at.ch + 2 * j * at.step < at.cols)
            row[at.ch + 2 * j * at.step] = make_float2(x[j].x, y[j].x);
        if (at.ch + (2 * j + 1) * at.step < at.cols)
            row[at.ch + (2 * j + 1) * at.step] = make_float2(x[j].y, y[j].y);
    }
}

// columns[samples][width] = the sums over each sample's row lanes of
// slots[samples * lanes][slot_stride]: every column by several threads, each
// adding its share of the lanes, then share after share.  Called by all
// threads after a barrier; ends with one.  work: [threads].
__device__ __forceinline__ void sum_lanes(const float2* slots, int stride, int samples, int lanes, int width,
                                          float2* columns, float2* work)
{
    const int threads = static_cast<int>(blockDim.x), all = samples * width;
    int shares = threads / all;
    shares = shares < 1 ? 1 : shares > lanes ? lanes : shares;
    for (int i = threadIdx.x; i < shares * all; i += threads) {
        const int share = shares == 1 ? 0 : i / all, col = i - share * all;
        const int q = samples == 1 ? 0 : col / width;
        const float2* first = slots + q * lanes * stride + col - q * width;
        float2 t = make_float2(0.f, 0.f);
        for (int p = share; p < lanes; p += shares)
            t = __fadd2_rn(t, first[p * stride]);
        (shares == 1 ? columns : work)[i] = t;
    }
    __syncthreads();
    if (shares > 1) {
        for (int i = threadIdx.x; i < all; i += threads) {
            float2 t = work[i];
            for (int k = 1; k < shares; ++k)
                t = __fadd2_rn(t, work[k * all + i]);
            columns[i] = t;
        }
        __syncthreads();
    }
}

// f(item, lane, lanes, real) for `items` items of `entries` entries each, one
// team of threads (a power of two, at most 32) to an item; a team past the
// last item repeats it with `real` false.  Called by whole warps.
template <class F>
__device__ __forceinline__ void each_item(int items, int entries, F f)
{
    int lanes = 1, shift = 0;
    while (lanes < 32 && 2 * lanes <= entries) {
        lanes *= 2;
        ++shift;
    }
    const int teams = static_cast<int>(blockDim.x) >> shift;
    const int me = static_cast<int>(threadIdx.x) >> shift, lane = static_cast<int>(threadIdx.x) & (lanes - 1);
    for (int i0 = 0; i0 < items; i0 += teams) {
        const int i = i0 + me;
        f(i < items ? i : items - 1, lane, lanes, i < items);
    }
}

// rsqrtf is within two ulps and one instruction where 1 / sqrtf takes dozens;
// every thread of a token's group forms it.
__device__ __forceinline__ float rstd_of(float m2, float inv_m, float eps) { return rsqrtf(m2 * inv_m + eps); }

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

// (S1, S2), times act_scale, of each of samples x groups items from the
// channels' sums of dz and dz xhat: columns[samples][width],
// out[samples][groups].
template <int DT>
__device__ __forceinline__ void weigh_columns(const NormArgs& a, const NormPlace& s, int samples, int width,
                                              const void* weight, const float2* columns, float2* out)
{
    const int per = group_cols(a, s);
    each_item(samples * s.groups, per, [&](int i, int lane, int lanes, bool real) {
        const int q = samples == 1 ? 0 : i / s.groups, g = i - q * s.groups;
        float s1 = 0.f, s2 = 0.f;
        for (int e = lane; e < per; e += lanes) {
            const int ch = g * per + e;
            const float w = weight_at<DT>(a, weight, s.ch0 + ch) * act_scale(a.act);
            const float2 v = columns[q * width + ch];
            s1 += w * v.x;
            s2 += w * v.y;
        }
        s1 = lanes_sum(s1, lanes);
        s2 = lanes_sum(s2, lanes);
        if (real && lane == 0)
            out[i] = make_float2(s1, s2);
    });
}

// out[group] = the sums of a group's pairs, one to an oct and row lane:
// pairs[lanes][width], `per` neighbouring octs to a group.  By whole warps.
__device__ __forceinline__ void add_octs(const float2* pairs, int width, int lanes, int groups, int per, float2* out)
{
    each_item(groups, lanes * per, [&](int g, int lane, int team, bool real) {
        float2 t = make_float2(0.f, 0.f);
        for (int e = lane; e < lanes * per; e += team) {
            const int p = e / per;
            t = __fadd2_rn(t, pairs[p * width + g * per + e - p * per]);
        }
        t.x = lanes_sum(t.x, team);
        t.y = lanes_sum(t.y, team);
        if (real && lane == 0)
            out[g] = t;
    });
}

// A run's sums of dz and dz xhat, of(channel), into the CTA's slice for dbias
// and dweight.  more: added to what the slice has, by reductions, so that nobody
// waits for the old value (bf16 [8192, 4096] in one group 534 us, by loads and
// stores 595).  They are no race for an order: a slice is one CTA's, the same
// thread of it comes to a channel each time, and what a thread does to one
// address keeps its order.
template <class F>
__device__ __forceinline__ void add_slice(float* chan, int c, int ch0, int width, bool more, F of)
{
    float* out = chan + static_cast<int64_t>(blockIdx.x) * 2 * c + ch0;
    for (int ch = threadIdx.x; ch < width; ch += blockDim.x) {
        const float2 v = of(ch);
        if (more) {
            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(out + ch), "f"(v.y) : "memory");
            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(out + c + ch), "f"(v.x) : "memory");
        } else {
            out[ch] = v.y;
            out[c + ch] = v.x;
        }
    }
}

// A value for each of a thread's channels that is the same within a group, as
// pairs (BY_OCT: one for all).
template <bool BY_OCT>
struct Grouped {
    float2 v[BY_OCT ? 1 : 4];
    __device__ __forceinline__ float2 at(int j) const { return v[BY_OCT ? 0 : j]; }
};

// The two halves of the pairs table[group] for a thread's channels.
template <bool BY_OCT>
__device__ __forceinline__ void grouped(const NormArgs& a, const NormPlace& s, const float2* table,
                                        Grouped<BY_OCT>& first, Grouped<BY_OCT>& second)
{
    int g = s.at.ch < s.at.cols ? local_group(a, s.at.ch) : 0;
    if constexpr (BY_OCT) {
        const float2 t = table[g];
        first.v[0] = pair_of(t.x);
        second.v[0] = pair_of(t.y);
    } else {
        float2 t[8];
        if (s.at.step == 1 && a.lay.pieces == 1) {   // neighbours: the next group after the last of this one
            int left = (g + 1) * a.per_group - s.at.ch;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                t[j] = table[g];
                if (--left == 0) {
                    left = a.per_group;
                    if (g + 1 < s.groups)
                        ++g;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int ch = s.at.ch + j * s.at.step;
                t[j] = table[ch < s.at.cols ? local_group(a, ch) : 0];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            first.v[j] = make_float2(t[2 * j].x, t[2 * j + 1].x);
            second.v[j] = make_float2(t[2 * j].y, t[2 * j + 1].y);
        }
    }
}

// What a thread keeps for its channels forward: y = act((x - mean) scale +
// bias), scale = rstd weight.  One operation less, x scale + (bias - mean
// scale), would leave the rounding of mean scale, which is large where a group
// is constant and rstd as large as 1 / sqrt(eps).
template <bool BY_OCT>
struct Affine {
    Grouped<BY_OCT> minus;   // minus the mean
    float2 scale[4], bias[4];
    // before the statistics are there: weight and bias
    template <int DT, bool VEC>
    __device__ __forceinline__ void params(const NormArgs& a, const NormPlace& s, const void* weight,
                                           const void* bias_)
    {
        param_floats<DT, VEC>(weight, a.wide_params, a.packed_params, s.ch0, s.at, scale);
        param_floats<DT, VEC>(bias_, a.wide_params, a.packed_params, s.ch0, s.at, bias);
    }
    // stats: (mean, rstd) by group of the run
    __device__ __forceinline__ void statistics(const NormArgs& a, const NormPlace& s, const float2* stats)
    {
        Grouped<BY_OCT> rstd;
        grouped<BY_OCT>(a, s, stats, minus, rstd);
#pragma unroll
        for (int j = 0; j < (BY_OCT ? 1 : 4); ++j)
            minus.v[j] = __fmul2_rn(minus.v[j], pair_of(-1.f));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            scale[j] = __fmul2_rn(scale[j], rstd.at(j));
    }
    __device__ __forceinline__ void apply(int act, const float2 (&x)[4], float2 (&y)[4]) const
    {
        float2 z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            z[j] = __ffma2_rn(__fadd2_rn(x[j], minus.at(j)), scale[j], bias[j]);
        act_value(act, z, y);
    }
};

// A bias times act_scale.  One of the type's far end, which shuts a channel or
// holds it open, stays finite: the slope of silu forms t p, infinity times zero
// if not.
__device__ __forceinline__ float scaled_bias(float bias, float factor)
{
    constexpr float most = 3.402823466e38f;
    const float t = bias * factor;
    return fabsf(t) > most && fabsf(bias) <= most ? copysignf(most, t) : t;
}

// And backward: xhat = (x - mean) rstd; weight and bias times act_scale, so
// that act' comes from t = xhat w + b.
template <bool BY_OCT>
struct Chan {
    Grouped<BY_OCT> minus, rstd;
    float2 w[4], b[4];
    template <int DT, bool VEC>
    __device__ __forceinline__ void params(const NormArgs& a, const NormPlace& s, const void* weight,
                                           const void* bias)
    {
        param_floats<DT, VEC>(weight, a.wide_params, a.packed_params, s.ch0, s.at, w);
        param_floats<DT, VEC>(bias, a.wide_params, a.packed_params, s.ch0, s.at, b);
        const float f = act_scale(a.act);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = __fmul2_rn(w[j], pair_of(f));
            b[j] = make_float2(scaled_bias(b[j].x, f), scaled_bias(b[j].y, f));
        }
    }
    __device__ __forceinline__ void statistics(const NormArgs& a, const NormPlace& s, const float2* stats)
    {
        grouped<BY_OCT>(a, s, stats, minus, rstd);
#pragma unroll
        for (int j = 0; j < (BY_OCT ? 1 : 4); ++j)
            minus.v[j] = __fmul2_rn(minus.v[j], pair_of(-1.f));
    }
    __device__ __forceinline__ void statistics(float mean, float rs)   // BY_OCT
    {
        minus.v[0] = pair_of(-mean);
        rstd.v[0] = pair_of(rs);
    }
    // dz
    __device__ __forceinline__ void slopes(int act, const float2 (&dy)[4], const float2 (&xhat)[4],
                                           float2 (&dz)[4]) const
    {
        float2 t[4], slope[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            t[j] = __ffma2_rn(xhat[j], w[j], b[j]);
        act_slope(act, t, slope);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dz[j] = __fmul2_rn(dy[j], slope[j]);
    }
};

// dx = rstd (dz weight - S1 / M - xhat S2 / M).  S1 and S2 are sums of the very
// products dz w, act_scale and all, that dx starts from, and rstd is multiplied
// last: in a group of one element the difference then is zero, not what two
// roundings leave.
template <bool BY_OCT>
struct Gradient {
    Grouped<BY_OCT> s1, s2, rstd;   // -S1 / M and -S2 / M; rstd / act_scale
    // sums: (-S1 / M, -S2 / M) by group of the run
    __device__ __forceinline__ void set(const NormArgs& a, const NormPlace& s, const Chan<BY_OCT>& k,
                                        const float2* sums)
    {
        grouped<BY_OCT>(a, s, sums, s1, s2);
        scale(a, k);
    }
    __device__ __forceinline__ void set(const NormArgs& a, const Chan<BY_OCT>& k, float sum1, float sum2)   // BY_OCT
    {
        s1.v[0] = pair_of(sum1);
        s2.v[0] = pair_of(sum2);
        scale(a, k);
    }
    __device__ __forceinline__ void scale(const NormArgs& a, const Chan<BY_OCT>& k)
    {
        const float2 f = pair_of(1.f / act_scale(a.act));
#pragma unroll
        for (int j = 0; j < (BY_OCT ? 1 : 4); ++j)
            rstd.v[j] = __fmul2_rn(f, k.rstd.v[j]);
    }
    __device__ __forceinline__ void of(const Chan<BY_OCT>& k, const float2 (&dz)[4], const float2 (&xhat)[4],
                                       float2 (&dx)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dx[j] = __fmul2_rn(rstd.at(j),
                               __ffma2_rn(xhat[j], s2.at(j), add_alone(__fmul2_rn(dz[j], k.w[j]), s1.at(j))));
    }
};

// Where a thread reads or writes an operand: its first row, and the step from
// one of its rows to the next.
struct Walk {
    const char* p;
    int64_t step;
};
template <int DT>
__device__ __forceinline__ Walk walk(const void* base, int64_t row, int rows_apart, int64_t pitch, const NormPlace& s)
{
    return Walk{oct_ptr<DT>(base, row, pitch, s.ch0 + s.at.ch), rows_apart * pitch * elem_size(DT)};
}
struct WalkOut {
    char* p;
    int64_t step;
};
template <int DT>
__device__ __forceinline__ WalkOut walk_out(void* base, int64_t row, int rows_apart, int64_t pitch,
                                            const NormPlace& s)
{
    return WalkOut{oct_ptr<DT>(base, row, pitch, s.ch0 + s.at.ch), rows_apart * pitch * elem_size(DT)};
}

// The next N rows of a walk, of which the thread has `n` (>= N: no row is
// looked at twice).
template <int DT, bool VEC, int N>
__device__ __forceinline__ void load_rows(const Walk& w, const OctAt& at, int n, Oct<DT> (&o)[N])
{
    if (n >= N) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = oct_load<DT, VEC>(w.p + i * w.step, at);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n)
                o[i] = oct_load<DT, VEC>(w.p + i * w.step, at);
            else
                oct_zero(o[i]);
    }
}

// What the backward pass reads: dy, and x or its checkpoint.
template <int DT, bool VEC, bool HELD>
struct GradWalk {
    Walk dy, x;
    const uint8_t* q;
    const float* scale;
    int64_t q_step, scale_step;
    __device__ __forceinline__ GradWalk(const NormArgs& a, const NormPlace& s, const void* pdy, const Saved& src,
                                        int64_t row, int rows_apart)
    {
        dy = walk<DT>(pdy, row, rows_apart, a.y_pitch, s);
        if constexpr (HELD) {
            q = static_cast<const uint8_t*>(src.q) + row * a.c + s.ch0 + s.at.ch;
            q_step = static_cast<int64_t>(rows_apart) * a.c;
            scale = src.scale + row * a.blocks + (VEC ? block_of(s.ch0 + s.at.ch, a.block) : 0);
            scale_step = rows_apart * a.blocks;
        } else {
            x = walk<DT>(src.x, row, rows_apart, a.x_pitch, s);
        }
    }
    __device__ __forceinline__ void advance(int rows)
    {
        dy.p += rows * dy.step;
        if constexpr (HELD) {
            q += rows * q_step;
            scale += rows * scale_step;
        } else {
            x.p += rows * x.step;
        }
    }
};

// One row of them: the i-th of the walk's next ones.
template <int DT, bool VEC, bool HELD>
struct GradRow {
    Oct<DT> dy;
    Oct<DT> x;      // HELD: unused
    Held q;
    float scale[VEC ? 1 : 8];   // consecutive channels of an aligned oct share a block; others need not
    __device__ __forceinline__ void load(const NormArgs& a, const NormPlace& s, const GradWalk<DT, VEC, HELD>& w,
                                         int i)
    {
        dy = oct_load<DT, VEC>(w.dy.p + i * w.dy.step, s.at);
        if constexpr (HELD) {
            q = held_load<VEC>(w.q + i * w.q_step, s.at);
            load_scales(a, s, w, i);
        } else {
            x = oct_load<DT, VEC>(w.x.p + i * w.x.step, s.at);
        }
    }
    // A row that does not exist: its dz is 0.
    __device__ __forceinline__ void clear()
    {
        oct_zero(dy);
        if constexpr (HELD) {
            q.w[0] = q.w[1] = 0;
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 8); ++j)
                scale[j] = 0.f;
        } else {
            oct_zero(x);
        }
    }
    __device__ __forceinline__ void load_scales(const NormArgs& a, const NormPlace& s,
                                                const GradWalk<DT, VEC, HELD>& w, int i)
    {
        if constexpr (VEC) {
            scale[0] = __ldg(w.scale + i * w.scale_step);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int ch = s.at.ch + j * s.at.step;
                scale[j] = ch < s.at.cols ? __ldg(w.scale + i * w.scale_step + block_of(s.ch0 + ch, a.block)) : 0.f;
            }
        }
    }
    // xhat = (x - mean) rstd, of a checkpoint with x = q scale
    template <bool BY_OCT>
    __device__ __forceinline__ void hats(int form, const Chan<BY_OCT>& k, float2 (&hat)[4]) const
    {
        float2 f[4];
        if constexpr (!HELD)
            oct_floats(x, f);
        else
            held_numbers(q, form, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 d;
            if constexpr (!HELD)
                d = __fadd2_rn(f[j], k.minus.at(j));
            else if constexpr (VEC)
                d = __ffma2_rn(f[j], pair_of(scale[0]), k.minus.at(j));
            else
                d = __ffma2_rn(f[j], make_float2(scale[2 * j], scale[2 * j + 1]), k.minus.at(j));
            hat[j] = __fmul2_rn(d, k.rstd.at(j));
        }
    }
};

// An oct's 16-byte vectors on their way to shared memory, `step` apart there.
template <int DT>
__device__ __forceinline__ void oct_async(uint32_t dst, uint32_t step, const char* from)
{
    if constexpr (DT != TSX_F32) {
        cp_async(dst, from, 16, 16);
    } else {
        // Neighbouring threads' vectors are 32 bytes apart, so each of the two
        // copies takes half of every sector: through L1 the sectors come once.
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst + h * step), "l"(from + 16 * h)
                         : "memory");
    }
}

// Rows of x on their way: a queue in shared memory that each thread fills by
// cp.async for itself alone, so that no barrier guards it and the bytes in
// flight do not depend on registers.  Four rows to a batch; kBatches batches
// are on their way at any time.
template <int DT>
struct RowQueue {
    static constexpr int kBatch = 4, kBatches = 2, kRows = kBatch * kBatches;
    static constexpr uint32_t kVecs = elem_size(DT) / 2;   // 16-byte vectors of an oct
    static constexpr uint32_t kStep = kNormThreads * 16;
    static constexpr size_t kBytes = size_t(kRows) * kVecs * kStep;
    Walk w;
    uint32_t at;   // this thread's first slot
    int left;      // rows that are still to be asked for
    __device__ __forceinline__ RowQueue(const Walk& walk, char* shared, int rows)
        : w(walk), at(smem_addr(shared) + threadIdx.x * 16), left(rows)
    {
#pragma unroll
        for (int b = 0; b < kBatches; ++b)
            ask(b);
    }
    // The walk's next rows, into the slots of batch b.
    __device__ __forceinline__ void ask(int b)
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < left)
                oct_async<DT>(at + (b * kBatch + i) * kVecs * kStep, kStep, w.p + i * w.step);
        cp_async_commit();
        w.p += kBatch * w.step;
        left -= kBatch;
    }
    // The rows of batch b, the oldest, of which n exist; others are zeros.
    __device__ __forceinline__ void take(int b, int n, Oct<DT> (&o)[kBatch]) const
    {
        cp_async_wait(kBatches - 1);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < n) {
#pragma unroll
                for (uint32_t h = 0; h < kVecs; ++h)
                    lds16(at + ((b * kBatch + i) * kVecs + h) * kStep, o[i].w + 4 * h);
            } else {
                oct_zero(o[i]);
            }
    }
    static __device__ __forceinline__ void lds16(uint32_t at, uint32_t* w)
    {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at));
    }
};

// use(o, n) for a thread's rows, four octs o at a time, of which n exist,
// through the queue where they are vectors.  `loop` rows are gone through, of
// which the thread's row lane has `count` (n is below zero past them): lanes
// that meet in shuffles come with the same `loop`.  `live` threads have
// channels; the others' octs are zeros.  begin() runs once the first rows are
// on their way.
template <int DT, bool VEC, class Begin, class Use>
__device__ __forceinline__ void each_four(Walk w, const OctAt& at, char* queue, int loop, int count, bool live,
                                          Begin begin, Use use)
{
    if constexpr (VEC) {
        RowQueue<DT> q(w, queue, live ? count : 0);
        begin();
        for (int done = 0; done < loop; done += q.kRows)
#pragma unroll
            for (int b = 0; b < q.kBatches; ++b) {
                const int i = done + b * q.kBatch;
                if (i < loop) {
                    Oct<DT> o[4];
                    q.take(b, live ? count - i : 0, o);
                    use(o, count - i);
                    q.ask(b);
                }
            }
        cp_async_wait(0);
    } else {
        begin();
        for (int i = 0; i < loop; i += 4) {
            Oct<DT> o[4];
            load_rows<DT, VEC>(w, at, live ? count - i : 0, o);
            w.p += 4 * w.step;
            use(o, count - i);
        }
    }
}

// The backward pass's rows on their way, dy and x or its checkpoint, the same
// way.  The kernels hold dz's sums, weights and statistics in over 50 registers;
// with four rows in registers beside them, 57 KB an SM were on their way in
// bursts (sums of bf16 [4, 16384, 512] from int8: 34 us), with a queue of eight
// rows twice that without a pause (31 us, and 27 with the first rows asked for
// before the statistics).
constexpr int kQueueBatch = 2;   // rows to a cp.async group
template <int DT>
TSX_HD constexpr int queue_rows() { return DT == TSX_F32 ? 4 : 8; }
template <int DT, bool HELD>
TSX_HD constexpr int queue_row_bytes()   // of one thread
{
    return elem_size(DT) * 8 + (HELD ? 8 + 4 : elem_size(DT) * 8);
}

template <int DT, bool HELD>
struct GradQueue {
    static constexpr int kRows = queue_rows<DT>(), kBatches = kRows / kQueueBatch;
    static constexpr uint32_t kVecs = elem_size(DT) / 2;   // 16-byte vectors of an oct
    static constexpr uint32_t k16 = kNormThreads * 16, k8 = kNormThreads * 8, k4 = kNormThreads * 4;
    static constexpr size_t kBytes = size_t(kRows) * kNormThreads * queue_row_bytes<DT, HELD>();
    GradWalk<DT, true, HELD> w;
    uint32_t dy, x, scale;   // this thread's place in the queue's arrays
    int left;                // rows that are still to be asked for
    __device__ __forceinline__ GradQueue(const GradWalk<DT, true, HELD>& walk, char* shared, int rows)
        : w(walk), left(rows)
    {
        dy = smem_addr(shared) + threadIdx.x * 16;
        const uint32_t after = smem_addr(shared) + kRows * kVecs * k16;
        x = after + threadIdx.x * (HELD ? 8 : 16);
        scale = after + kRows * k8 + threadIdx.x * 4;
#pragma unroll
        for (int b = 0; b < kBatches; ++b)
            ask(b);
    }
    // The walk's next rows, into the slots of batch b.
    __device__ __forceinline__ void ask(int b)
    {
#pragma unroll
        for (int i = 0; i < kQueueBatch; ++i)
            if (i < left) {
                const uint32_t slot = b * kQueueBatch + i;
                oct_async<DT>(dy + slot * kVecs * k16, k16, w.dy.p + i * w.dy.step);
                if constexpr (HELD) {
                    cp_async(x + slot * k8, w.q + i * w.q_step, 8, 8);
                    cp_async(scale + slot * k4, w.scale + i * w.scale_step, 4, 4);
                } else {
                    oct_async<DT>(x + slot * kVecs * k16, k16, w.x.p + i * w.x.step);
                }
            }
        cp_async_commit();
        w.advance(kQueueBatch);
        left -= kQueueBatch;
    }
    // Row i of batch b.
    __device__ __forceinline__ void take(int b, int i, GradRow<DT, true, HELD>& g) const
    {
        const uint32_t slot = b * kQueueBatch + i;
#pragma unroll
        for (uint32_t h = 0; h < kVecs; ++h)
            lds16(dy + (slot * kVecs + h) * k16, g.dy.w + 4 * h);
        if constexpr (HELD) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(g.q.w[0]), "=r"(g.q.w[1]) : "r"(x + slot * k8));
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(g.scale[0]) : "r"(scale + slot * k4));
        } else {
#pragma unroll
            for (uint32_t h = 0; h < kVecs; ++h)
                lds16(x + (slot * kVecs + h) * k16, g.x.w + 4 * h);
        }
    }
    static __device__ __forceinline__ void lds16(uint32_t at, uint32_t* w)
    {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at));
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
