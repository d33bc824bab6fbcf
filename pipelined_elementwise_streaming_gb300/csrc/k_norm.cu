// Group norm over samples that are not held on chip: the streaming kernels,
// which read their operands twice.  The first kernel sums over ranges of rows
// (one CTA to a range of a run of channels), the second joins the ranges' sums
// and applies.
//
// One wave of CTAs, so that each pays once for its parameters and its sums.
// The second kernel is launched to start early: it asks for its first rows
// before it waits for the sums.  Samples cut into more than 160 ranges are cut
// for clusters of eight, which join their ranges' sums through rank 0's shared
// memory, so that the second kernel's CTAs have few parts to join each.
//
// Measured on GB300 (GPU time of a call in a CUDA graph over tensors that take
// turns, so that nothing is left in L2; HBM's own time at 6786 GB/s for what the
// kernels read and write in parentheses):
//   bf16 [1, 262144, 128], 32 groups, silu: 40.3 us (29.7)
//   bf16 [4, 16384, 512], 32 groups, silu, int8 checkpoint: 101.2 us (75.1) for
//   both passes; its kernels launched alone, cold: statistics 16.1 (9.9), apply
//   and checkpoint 36.9 (25.0), gradient's sums 28.2 (15.1), dx 33.1 (25.0)
// About 6 us of each kernel are its start, its first rows' latency and its sums;
// the rest runs at 85 to 100 % of HBM's rate, but for the checkpoint's and the
// gradient's arithmetic (13 to 18 instructions an element), which holds those
// kernels at 75 to 85 %.
// Samples of few rows, one to a CTA, are far from that: what a CTA does once
// outweighs its row.  Tokens of 4096 channels in one group, bf16 [8192, 1, 4096]:
// 642 us forward (29.7; HBM's time for reading once 19.8), 536 backward (49.5).

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kPartsAtOnce = 16;   // parts that a thread of the gradient's second kernel loads at once

// CTAs to an SM that the registers are cut for.
template <int DT>
TSX_HD constexpr int forward_ctas() { return DT == TSX_F32 ? 2 : 3; }
constexpr int kBackwardCtas = 2;

__device__ __forceinline__ char* next_16(float2* p)
{
    return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p) + 15) & ~static_cast<uintptr_t>(15));
}

// A range of rows: `at` counts them sample by sample.  The
// `ranks` CTAs of a cluster take neighbouring ranges and join their sums.
struct Range {
    int64_t sample, split;
    int64_t row0;   // first row, counted through all samples
    int rows;       // rows of the range
    int rank;
    int mine;       // rows of the thread's lane: p, p + P, ...
};

__device__ __forceinline__ Range range_of(const NormArgs& a, const NormPlace& s, unsigned at)
{
    Range r;
    const unsigned splits = static_cast<unsigned>(a.lay.splits);
    r.sample = at / splits;
    r.split = at % splits;
    r.rank = static_cast<int>(static_cast<unsigned>(r.split) % static_cast<unsigned>(a.lay.ranks));
    r.row0 = r.sample * a.l + r.split * a.lay.range;
    r.rows = range_rows(a, a.lay.range, r.split);
    r.mine = s.p < a.lay.P && s.p < r.rows ? (r.rows - s.p + a.lay.P - 1) / a.lay.P : 0;
    return r;
}

// The parts of a sample: one to each cluster and piece.
__device__ __forceinline__ int parts_of(const NormArgs& a) { return static_cast<int>(a.lay.splits) / a.lay.ranks * a.lay.pieces; }

__device__ __forceinline__ float2* part_of(const NormArgs& a, const NormPlace& s, const Range& r, float2* part)
{
    return part + (r.sample * parts_of(a) + r.split / a.lay.ranks * a.lay.pieces + s.piece) * a.groups + s.group0;
}

// ------------------------------------------------------------- forward

// First kernel: (mean, M2) of every cluster's range, run and group.
template <int DT, bool VEC, bool BY_OCT>
__global__ void __launch_bounds__(kNormThreads, forward_ctas<DT>()) norm_stats_kernel(NormArgs a, const void* x, float2* part)
{
    extern __shared__ float4 shared4[];
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a, s, blockIdx.x);
    const int P = a.lay.P, width = run_width<BY_OCT>(s), stride = slot_stride(width);
    float2* sums = reinterpret_cast<float2*>(shared4);   // [run_groups]
    float2* ranks = sums + a.lay.run_groups;             // clusters: [ranks][run_groups]
    float2* slots = ranks + (a.lay.ranks > 1 ? a.lay.ranks * a.lay.run_groups : 0);   // [P][stride]
    let_next_start();
    if (a.lay.ranks > 1)
        cluster_arrive();   // waited for before anything is put into another CTA
    Triples<BY_OCT> t;
    t.clear();
    each_four<DT, VEC>(walk<DT>(x, r.row0 + s.p, P, a.x_pitch, s), s.at, next_16(slots + P * stride), r.mine, r.mine, s.live,
                       [] {}, [&](const Oct<DT>(&o)[4], int n) {
                           if (s.live)
                               t.add_octs(o, n);
                       });
    if (s.live)
        t.leave(s.at, slots + s.p * stride);
    __syncthreads();
    float2* out = part_of(a, s, r, part);
    join_groups(a.lay, slots, stride, 1, s.groups, P, group_cols(a, s) / (BY_OCT ? 8 : 1), r.rows, BY_OCT ? 8.f : 1.f,
                a.lay.ranks > 1 ? sums : out);
    if (a.lay.ranks > 1) {
        __syncthreads();
        cluster_wait();
        for (int g = threadIdx.x; g < s.groups; g += blockDim.x)
            cluster_put(ranks + r.rank * s.groups + g, 0, sums[g]);
        cluster_arrive();
        cluster_wait();
        if (r.rank == 0)
            for (int g = threadIdx.x; g < s.groups; g += blockDim.x)
                out[g] = join_ranges(ranks + g, s.groups, a.lay.ranks,
                                     static_cast<int>(max(a.l - r.split * a.lay.range, int64_t(0))),
                                     static_cast<int>(a.lay.range), static_cast<float>(group_cols(a, s)));
    }
}

// The statistics of the run's groups from their parts, into `stats` [groups]
// as (mean, rstd).  Neighbouring threads read neighbouring groups.  Ends with
// the CTA synchronised.
__device__ __forceinline__ void join_parts(const NormArgs& a, const NormPlace& s, int64_t sample, const float2* part,
                                           float2* stats, float4* work)
{
    const int count = parts_of(a);
    const float2* first = part + sample * count * a.groups + s.group0;
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    const int threads = static_cast<int>(blockDim.x);
    // `lanes` threads to a group, each joins every lanes-th part
    const int lanes = s.groups < threads ? threads / s.groups : 1;
    const int64_t range = a.lay.range * a.lay.ranks;
    const int full = static_cast<int>(a.l / range);   // ranges before the one that may be short
    const float rows = static_cast<float>(range), rest = static_cast<float>(a.l - full * range);
    for (int i = threadIdx.x; i < lanes * s.groups; i += threads) {
        const int lane = i / s.groups, g = i - lane * s.groups;
        Triples<true> t;
        t.clear();
#pragma unroll 4
        for (int k = lane; k < count; k += lanes) {
            const float2 v = first[static_cast<int64_t>(k) * a.groups + g];
            int split = k, cols = a.per_group;
            if (a.lay.pieces > 1) {
                split = k / a.lay.pieces;
                cols = min(a.lay.run_cols, a.per_group - (k - split * a.lay.pieces) * a.lay.run_cols);
            }
            const float mu[1] = {v.x}, dev[1] = {v.y};
            t.join((split < full ? rows : split == full ? rest : 0.f) * static_cast<float>(cols), mu, dev);
        }
        work[i] = make_float4(t.count, t.mean[0], t.m2[0], 0.f);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < s.groups; g += threads) {
        Triples<true> t;
        t.clear();
        for (int k = 0; k < lanes; ++k) {
            const float4 v = work[k * s.groups + g];
            const float mu[1] = {v.y}, dev[1] = {v.z};
            t.join(v.x, mu, dev);
        }
        stats[g] = make_float2(t.mean[0], rstd_of(t.m2[0], 1.f / m, a.eps));
    }
    __syncthreads();
}

// Second kernel: y, and with HOLD the checkpoint of x.
template <int DT, bool VEC, bool BY_OCT, bool HOLD>
__global__ void __launch_bounds__(kNormThreads, forward_ctas<DT>())
    norm_apply_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held, const float2* part)
{
    extern __shared__ float4 work[];   // [threads or groups], then [run_groups] statistics
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a, s, blockIdx.x);
    const int P = a.lay.P;
    Affine<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    float2* stats = reinterpret_cast<float2*>(work + max(static_cast<int>(blockDim.x), a.lay.run_groups));
    WalkOut out = walk_out<DT>(y, r.row0 + s.p, P, a.y_pitch, s);
    HeldPtr to;
    if constexpr (HOLD)
        to = HeldPtr(held, r.row0 + s.p, P, a.c, a.blocks, s.ch0 + s.at.ch, a.block);
    auto begin = [&] {
        wait_for_last();
        join_parts(a, s, r.sample, part, stats, work);
        k.statistics(a, s, stats);
        if (r.split == 0 && s.piece == 0)
            for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
                mean[r.sample * a.groups + s.group0 + g] = stats[g].x;
                rstd[r.sample * a.groups + s.group0 + g] = stats[g].y;
            }
    };
    // every lane of a warp comes to the checkpoint's shuffles
    const int loop = HOLD ? (r.rows + P - 1) / P : r.mine;
    each_four<DT, VEC>(walk<DT>(x, r.row0 + s.p, P, a.x_pitch, s), s.at, next_16(stats + a.lay.run_groups), loop,
                       r.mine, s.live, begin, [&](const Oct<DT>(&o)[4], int n) {
                           by_act(a.act, [&](auto act) {
#pragma unroll
                               for (int i = 0; i < 4; ++i) {
                                   float2 f[4], v[4];
                                   oct_floats(o[i], f);
                                   k.apply(act, f, v);
                                   if (s.live && i < n)
                                       oct_store<DT, VEC>(out.p + i * out.step, s.at, oct_round<DT>(v));
                               }
                           });
                           out.p += 4 * out.step;
                           if constexpr (HOLD) {
                               hold_rows<DT, VEC>(o, s.live, s.at, a.lay.team, a.form, HeldRows{to, n});
                               to.advance(4);
                           }
                       });
}

// ------------------------------------------------------------ backward

__device__ __forceinline__ void load_stats(const NormArgs& a, const NormPlace& s, int64_t sample, const float* mean,
                                           const float* rstd, float2* stats)
{
    for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
        const int64_t at = sample * a.groups + s.group0 + g;
        stats[g] = make_float2(mean[at], rstd[at]);
    }
    __syncthreads();
}

// use(g, n) for a thread's `rows` rows, two of them, g, at a time, of which n
// exist, through the queue where they are vectors; begin() runs once the first
// are on their way.  The loop over the queue's batches stays a loop: unrolled,
// with a choice of the activation in each batch, the kernels are so long that
// fetching them shows (a step of bf16 [4, 16384, 512] over an int8 checkpoint,
// whose kernels follow one another, 108.4 us against 100.7).
template <int DT, bool VEC, bool HELD, class Begin, class Use>
__device__ __forceinline__ void each_two(const NormArgs& a, const NormPlace& s, GradWalk<DT, VEC, HELD> w,
                                         char* queue, int rows, Begin begin, Use use)
{
    if constexpr (VEC) {
        GradQueue<DT, HELD> q(w, queue, rows);
        begin();
        for (int left = rows; left > 0; left -= q.kRows)
#pragma unroll 1
            for (int b = 0; b < q.kBatches; ++b) {
                cp_async_wait(q.kBatches - 1);
                const int n = left - b * kQueueBatch;
                if (n > 0) {
                    GradRow<DT, true, HELD> g[kQueueBatch];
#pragma unroll
                    for (int i = 0; i < kQueueBatch; ++i)
                        if (i < n)
                            q.take(b, i, g[i]);
                        else
                            g[i].clear();
                    use(g, n);
                }
                q.ask(b);
            }
        cp_async_wait(0);
    } else {
        begin();
        for (int left = rows; left > 0; left -= kQueueBatch) {
            GradRow<DT, VEC, HELD> g[kQueueBatch];
#pragma unroll
            for (int i = 0; i < kQueueBatch; ++i)
                if (i < left)
                    g[i].load(a, s, w, i);
                else
                    g[i].clear();
            w.advance(kQueueBatch);
            use(g, left);
        }
    }
}

// First kernel: S1 and S2 (times act_scale) of every cluster's range, run and
// group, and the CTA's sums for dweight and dbias.  MANY: samples are not cut,
// and each CTA takes every gridDim.x-th of them, so that dweight and dbias have
// no more slices than there are CTAs.
template <int DT, bool VEC, bool BY_OCT, bool HELD, bool MANY>
__global__ void __launch_bounds__(kNormThreads, kBackwardCtas)
    norm_sums_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, float2* part, float* chan)
{
    extern __shared__ __align__(16) float2 shared[];
    const NormPlace s = norm_place<VEC>(a);
    const int P = a.lay.P, width = s.at.cols, stride = slot_stride(width);
    float2* stats = shared;                         // [run_groups]: (mean, rstd), then (S1, S2)
    float2* ranks = stats + a.lay.run_groups;       // clusters: [ranks][run_groups]
    float2* work = ranks + (a.lay.ranks > 1 ? a.lay.ranks * a.lay.run_groups : 0);   // [threads]
    float2* columns = work + kNormThreads;          // [run_cols]
    float2* slots = columns + a.lay.run_cols;       // [P][stride]
    char* queue = next_16(slots + P * stride);
    let_next_start();
    if (a.lay.ranks > 1)
        cluster_arrive();
    Chan<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    unsigned at = blockIdx.x;
    do {
        const Range r = range_of(a, s, at);
        auto begin = [&] {
            load_stats(a, s, r.sample, mean, rstd, stats);
            k.statistics(a, s, stats);
        };
        float2 sz[4], szx[4];   // sums of dz and dz xhat, channel by channel
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sz[j] = szx[j] = make_float2(0.f, 0.f);
        const GradWalk<DT, VEC, HELD> w(a, s, dy, x, r.row0 + s.p, P);
        each_two<DT, VEC, HELD>(a, s, w, queue, s.live ? r.mine : 0, begin,
                                [&](const GradRow<DT, VEC, HELD>(&g)[kQueueBatch], int) {
            by_act(a.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < kQueueBatch; ++i) {
                    float2 fd[4], hat[4], dz[4];
                    oct_floats(g[i].dy, fd);
                    g[i].hats(a.form, k, hat);
                    k.slopes(act, fd, hat, dz);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sz[j] = __fadd2_rn(sz[j], dz[j]);
                        szx[j] = __ffma2_rn(dz[j], hat[j], szx[j]);
                    }
                }
            });
        });
        if (s.live)
            leave_sums(s.at, sz, szx, slots + s.p * stride);
        float2* sums = part_of(a, s, r, part);
        float2* mine = a.lay.ranks > 1 ? stats : sums;
        if constexpr (BY_OCT) {
            // S1 and S2 from the threads' weighted sums, beside the channels' sums
            float2 t1 = make_float2(0.f, 0.f), t2 = t1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t1 = __ffma2_rn(sz[j], k.w[j], t1);
                t2 = __ffma2_rn(szx[j], k.w[j], t2);
            }
            if (s.live)
                work[s.p * (width / 8) + s.at.ch / 8] = make_float2(t1.x + t1.y, t2.x + t2.y);
            __syncthreads();
            add_octs(work, width / 8, P, s.groups, group_cols(a, s) / 8, mine);
            __syncthreads();
            sum_lanes(slots, stride, 1, P, width, columns, work);
        } else {
            __syncthreads();
            sum_lanes(slots, stride, 1, P, width, columns, work);
            weigh_columns<DT>(a, s, 1, width, weight, columns, mine);
        }
        add_slice(chan, a.c, s.ch0, width, MANY && at != blockIdx.x, [&](int ch) { return columns[ch]; });
        if (a.lay.ranks > 1) {
            __syncthreads();
            cluster_wait();
            for (int i = threadIdx.x; i < s.groups; i += blockDim.x)
                cluster_put(ranks + r.rank * s.groups + i, 0, stats[i]);
            cluster_arrive();
            cluster_wait();
            if (r.rank == 0)
                for (int i = threadIdx.x; i < s.groups; i += blockDim.x) {
                    float2 t = ranks[i];
                    for (int n = 1; n < a.lay.ranks; ++n)
                        t = __fadd2_rn(t, ranks[n * s.groups + i]);
                    sums[i] = t;
                }
        }
        at += gridDim.x;
    } while (MANY && at < static_cast<unsigned>(a.n));
}

// Columns to a CTA of the sums over slices: 32, or 8 where 32 would leave few
// CTAs (the gradient of bf16 [2000, 64, 256]: 16 CTAs 75.0 us, 64 CTAs 71.8;
// [1000, 33, 512] 44.4, 42.8; but [4, 1024, 1280] 15.7 in 80 CTAs, 15.9 in 320,
// tokens [4000, 2048] 14.6 in 128, 16.2 in 512).
constexpr int kParamCols = 32, kParamFew = 8, kParamCtas = 64;

// dweight and dbias: the sums of the [slices][2][c] partial sums.  A CTA takes
// COLS of the 2 c columns, a warp 32 / COLS slices at a time; then a warp's
// lanes and last the warps are added in their order.  work: [warps][COLS].
template <int COLS>
__device__ __forceinline__ void add_params(const float* chan, int64_t slices, int c, int64_t block, float* dweight,
                                           float* dbias, float* work)
{
    const int lane = static_cast<int>(threadIdx.x) % 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int warps = static_cast<int>(blockDim.x) / 32, own = static_cast<int>(threadIdx.x) / COLS;
    const int64_t col = block * COLS + lane % COLS;   // of 2 c
    const bool real = col < 2 * static_cast<int64_t>(c);
    float t = 0.f;
    if (real) {
#pragma unroll 8
        for (int64_t i = own; i < slices; i += blockDim.x / COLS)
            t += chan[i * 2 * c + col];
    }
    for (int d = COLS; d < 32; d <<= 1)
        t += __shfl_xor_sync(0xffffffffu, t, d);
    if (lane < COLS)
        work[warp * COLS + lane] = t;
    __syncthreads();
    if (warp == 0) {
        t = 0.f;
        for (int i = lane / COLS; i < warps; i += 32 / COLS)
            t += work[i * COLS + lane % COLS];
        for (int d = COLS; d < 32; d <<= 1)
            t += __shfl_xor_sync(0xffffffffu, t, d);
        if (real && lane < COLS) {
            if (col < c)
                dweight[col] = t;
            else
                dbias[col - c] = t;
        }
    }
}

// Second kernel: dx; the CTAs past the ranges', if any, add up dweight and dbias.
template <int DT, bool VEC, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kNormThreads, kBackwardCtas)
    norm_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, void* dx, float* dweight, float* dbias, const float2* part, const float* chan)
{
    extern __shared__ __align__(16) float2 shared[];
    const int64_t ranges = a.n * a.lay.splits;
    if (blockIdx.x >= ranges) {
        wait_for_last();
        add_params<kParamCols>(chan, a.lay.slices, a.c, (blockIdx.x - ranges) * gridDim.y + blockIdx.y, dweight, dbias,
                   reinterpret_cast<float*>(shared));
        return;
    }
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a, s, blockIdx.x);
    const int P = a.lay.P;
    float2* stats = shared;                      // [run_groups]
    float2* sums = stats + a.lay.run_groups;     // [run_groups]: -S1 / M, -S2 / M
    float2* work = sums + a.lay.run_groups;      // [threads or groups]
    const int threads = static_cast<int>(blockDim.x);
    Chan<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    const GradWalk<DT, VEC, HELD> w(a, s, dy, x, r.row0 + s.p, P);
    char* queue = next_16(work + max(threads, a.lay.run_groups));
    Gradient<BY_OCT> to;
    WalkOut out = walk_out<DT>(dx, r.row0 + s.p, P, a.x_pitch, s);
    auto begin = [&] {
        wait_for_last();
        const int count = parts_of(a);
        const float2* first = part + r.sample * count * a.groups + s.group0;
        const float m = -static_cast<float>(a.l) * static_cast<float>(a.per_group);
        const int lanes = s.groups < threads ? threads / s.groups : 1;
        for (int i = threadIdx.x; i < lanes * s.groups; i += threads) {
            const int lane = i / s.groups, group = i - lane * s.groups;
            float2 t = make_float2(0.f, 0.f);
            for (int n = lane; n < count; n += kPartsAtOnce * lanes) {
                float2 v[kPartsAtOnce];
#pragma unroll
                for (int j = 0; j < kPartsAtOnce; ++j)
                    v[j] = n + j * lanes < count ? first[static_cast<int64_t>(n + j * lanes) * a.groups + group]
                                                 : make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kPartsAtOnce; ++j)
                    t = __fadd2_rn(t, v[j]);
            }
            work[i] = t;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < s.groups; i += threads) {
            float2 t = work[i];
            for (int n = 1; n < lanes; ++n)
                t = __fadd2_rn(t, work[n * s.groups + i]);
            sums[i] = make_float2(t.x / m, t.y / m);
        }
        load_stats(a, s, r.sample, mean, rstd, stats);   // synchronises
        k.statistics(a, s, stats);
        to.set(a, s, k, sums);
    };
    each_two<DT, VEC, HELD>(a, s, w, queue, s.live ? r.mine : 0, begin,
                            [&](const GradRow<DT, VEC, HELD>(&g)[kQueueBatch], int n) {
        by_act(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < kQueueBatch; ++i) {
                float2 fd[4], hat[4], dz[4], v[4];
                oct_floats(g[i].dy, fd);
                g[i].hats(a.form, k, hat);
                k.slopes(act, fd, hat, dz);
                to.of(k, dz, hat, v);
                if (i < n)
                    oct_store<DT, VEC>(out.p + i * out.step, s.at, oct_round<DT>(v));
            }
        });
        out.p += kQueueBatch * out.step;
    });
}

template <int COLS>
__global__ void __launch_bounds__(1024)
    norm_params_kernel(const float* chan, int64_t slices, int c, float* dweight, float* dbias)
{
    __shared__ float work[32 * COLS];
    wait_for_last();
    add_params<COLS>(chan, slices, c, blockIdx.x, dweight, dbias, work);
}

__global__ void norm_empty_kernel(float* mean, float* rstd, int64_t count, float eps)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        mean[i] = 0.f;
        rstd[i] = 1.f / sqrtf(eps);
    }
}

// Shared memory of the queues, from the next multiple of 16 on.
size_t queue_bytes(int dtype, const NormLayout& lay, bool held)
{
    if (!lay.vec)
        return 0;
    const int row = dtype == TSX_F32 ? (held ? queue_row_bytes<TSX_F32, true>() : queue_row_bytes<TSX_F32, false>())
                                     : (held ? queue_row_bytes<TSX_BF16, true>() : queue_row_bytes<TSX_BF16, false>());
    const int rows = dtype == TSX_F32 ? queue_rows<TSX_F32>() : queue_rows<TSX_BF16>();
    return 16 + size_t(kNormThreads) * rows * row;
}

size_t row_queue_bytes(int dtype, const NormLayout& lay)
{
    if (!lay.vec)
        return 0;
    return 16 + (dtype == TSX_F32 ? RowQueue<TSX_F32>::kBytes : RowQueue<TSX_BF16>::kBytes);
}

// Pairs that the first kernels keep for their groups, and in clusters for
// every rank's.
size_t rank_sums(const NormLayout& lay) { return size_t(lay.run_groups) * (lay.ranks > 1 ? lay.ranks + 1 : 1); }

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                        float* mean, float* rstd, HeldOut held, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const int width = lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols;
    const size_t slots =
        (rank_sums(lay) + size_t(lay.P) * slot_stride(width)) * sizeof(float2) + row_queue_bytes(dtype, lay);
    const int items = lay.threads > lay.run_groups ? lay.threads : lay.run_groups;
    const size_t stats = items * sizeof(float4) + lay.run_groups * sizeof(float2) + row_queue_bytes(dtype, lay);
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC, BY_OCT) \
    e = launch_grid<norm_stats_kernel<DT, VEC, BY_OCT>>(grid, lay.threads, slots, lay.ranks, false, st, a, x, \
                    scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    if (e != cudaSuccess)
        return e;
#define CALL(DT, VEC, BY_OCT)                                                                                       \
    e = held.q ? launch_grid<norm_apply_kernel<DT, VEC, BY_OCT, true>>(grid, lay.threads, stats, 1, true, st, a, x, \
                             weight, bias, y, mean, rstd, held, scratch.part)                                       \
               : launch_grid<norm_apply_kernel<DT, VEC, BY_OCT, false>>(grid, lay.threads, stats, 1, true, st, a, x, \
                             weight, bias, y, mean, rstd, held, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    return e;
}

cudaError_t launch_norm_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                 const void* bias, const float* mean, const float* rstd, void* dx, float* dweight,
                                 float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 first(unsigned(lay.slices), unsigned(lay.runs)), grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const size_t sums = (rank_sums(lay) + kNormThreads + lay.run_cols +
                         size_t(lay.P) * slot_stride(lay.run_cols)) * sizeof(float2) + queue_bytes(dtype, lay, x.q);
    cudaError_t e = cudaSuccess;
    const bool many = lay.slices < a.n * lay.splits;
#define KERNEL(DT, VEC, BY_OCT, HELD, MANY)                                                                       \
    launch_grid<norm_sums_kernel<DT, VEC, BY_OCT, HELD, MANY>>(first, lay.threads, sums, lay.ranks, false, st, a, \
                                                               dy, x, weight, bias, mean, rstd, scratch.part,     \
                                                               scratch.chan)
#define CALL(DT, VEC, BY_OCT)                                                                                     \
    e = x.q ? (many ? KERNEL(DT, VEC, BY_OCT, true, true) : KERNEL(DT, VEC, BY_OCT, true, false))                 \
            : (many ? KERNEL(DT, VEC, BY_OCT, false, true) : KERNEL(DT, VEC, BY_OCT, false, false))
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
#undef KERNEL
    if (e != cudaSuccess)
        return e;
    const int items = lay.threads > lay.run_groups ? lay.threads : lay.run_groups;
    const size_t stats = (2 * size_t(lay.run_groups) + items) * sizeof(float2) + queue_bytes(dtype, lay, x.q);
    // An output may be an input: dweight or dbias in the place of weight or bias
    // is written once no CTA reads those any more, by a kernel of its own, of as
    // many threads so that it adds in the same order.
    const bool apart = dweight == weight || dweight == bias || dbias == weight || dbias == bias;
    const int64_t param_ctas = (2 * int64_t(a.c) + kParamCols - 1) / kParamCols;
    const dim3 all(unsigned(grid.x + (apart ? 0 : (param_ctas + lay.runs - 1) / lay.runs)), grid.y);
#define CALL(DT, VEC, BY_OCT)                                                                                     \
    e = x.q ? launch_grid<norm_grad_kernel<DT, VEC, BY_OCT, true>>(all, lay.threads, stats, 1, true, st, a, dy, x,  \
                          weight, bias, mean, rstd, dx, dweight, dbias, scratch.part, scratch.chan)               \
            : launch_grid<norm_grad_kernel<DT, VEC, BY_OCT, false>>(all, lay.threads, stats, 1, true, st, a, dy, x, \
                          weight, bias, mean, rstd, dx, dweight, dbias, scratch.part, scratch.chan)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    if (e != cudaSuccess || !apart)
        return e;
    return launch_grid<norm_params_kernel<kParamCols>>(dim3(unsigned(param_ctas)), lay.threads, 0, 1, true, st,
                                                       scratch.chan, lay.slices, a.c, dweight, dbias);
}

cudaError_t launch_norm_params(const NormArgs& a, int64_t slices, const float* chan, float* dweight, float* dbias,
                               cudaStream_t st)
{
    const int64_t cols = 2 * int64_t(a.c);
    if (cols >= kParamCols * kParamCtas)
        return launch_grid<norm_params_kernel<kParamCols>>(dim3(unsigned((cols + kParamCols - 1) / kParamCols)), 1024, 0,
                                                           1, true, st, chan, slices, a.c, dweight, dbias);
    return launch_grid<norm_params_kernel<kParamFew>>(dim3(unsigned((cols + kParamFew - 1) / kParamFew)), 1024, 0, 1,
                                                      true, st, chan, slices, a.c, dweight, dbias);
}

cudaError_t launch_norm_empty(float* mean, float* rstd, int64_t count, float eps, cudaStream_t st)
{
    const int64_t blocks = (count + 255) / 256;
    return launch_grid<norm_empty_kernel>(dim3(unsigned(blocks < 1024 ? blocks : 1024)), 256, 0, 1, false, st, mean, rstd,
                                          count, eps);
}

}  // namespace tsx
