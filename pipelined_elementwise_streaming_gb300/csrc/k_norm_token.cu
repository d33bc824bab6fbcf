// Group norm of tokens (l = 1) whose groups are a power of two of octs, at
// most a warp's 32: every group lies in neighbouring lanes of one warp, so its
// sums are a few shuffles, a row is read once, and no barrier stands between
// its load and its store.  A CTA walks a contiguous share of the rows, so that
// weight and bias (and the sums for their gradients) stay in registers; rows
// on their way wait in a queue in shared memory that each thread fills for
// itself.  As many CTAs as the SMs hold at once: three each, two where the
// gradient or a checkpoint takes the registers.
//
// HBM bounds the larger calls, the launch the smallest.  Measured on GB300, GPU
// time of a call in a CUDA graph over tensors that take turns, so that nothing is
// left in L2, HBM's own time at 6786 GB/s in parentheses: bf16 [8192, 4096] in 32
// groups 22.8 us (19.8), with an int8 checkpoint 33.6 (24.9), its gradient 41.8
// (29.7; from registers in place of the queue 12 us more); fp32 [4096, 4096] 22.0
// (19.8); bf16 [16, 4096] 3.1.

#include <algorithm>

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

// Sums over each group's lanes, all rows at once: the shuffles of one row hide
// the latency of another's.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], int lanes)
{
    for (int d = 1; d < lanes; d <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
}

__device__ __forceinline__ float oct_sum(const float2 (&f)[4])
{
    const float2 t = __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
    return t.x + t.y;
}

template <int DT, bool HOLD>
__global__ void __launch_bounds__(kTokenThreads, HOLD ? 2 : 3)
    norm_token_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held)
{
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;   // threads to a group
    const float inv_m = 1.f / static_cast<float>(a.per_group);   // a power of two
    Affine<true> k;
    k.params<DT, true>(a, s, weight, bias);
    const int group = s.group0 + local_group(a, s.at.ch);
    const bool first = s.at.ch % a.per_group == 0;
    const int P = a.lay.P;
    const int step_s = P * a.groups;
    // the CTA's rows: P side by side from a contiguous share of all rows
    const int64_t share = a.lay.range, first_row = static_cast<int64_t>(blockIdx.x) * share;
    const int rows = static_cast<int>(min(share, a.n - first_row));
    const int mine = s.p < P && s.p < rows ? (rows - s.p + P - 1) / P : 0;
    const int64_t row0 = first_row + s.p;
    const WalkOut to = walk_out<DT>(y, row0, P, a.y_pitch, s);
    char* out = to.p;
    float* pm = mean + row0 * a.groups + group;
    float* pr = rstd + row0 * a.groups + group;
    HeldPtr hp;
    if constexpr (HOLD)
        hp = HeldPtr(held, row0, P, a.c, a.blocks, s.ch0 + s.at.ch, a.block);
    auto use = [&](const Oct<DT>(&o)[4], int n) {
        float mu[4], dev[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f[4];
            oct_floats(o[i], f);
            mu[i] = oct_sum(f);
        }
        team_sums(mu, lanes);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f[4], sq = make_float2(0.f, 0.f);
            oct_floats(o[i], f);
            mu[i] *= inv_m;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = __fadd2_rn(f[j], pair_of(-mu[i]));
                sq = __ffma2_rn(d, d, sq);
            }
            dev[i] = sq.x + sq.y;
        }
        team_sums(dev, lanes);
        by_act(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float rs = rstd_of(dev[i], inv_m, a.eps);
                float2 f[4], v[4];
                oct_floats(o[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 hat = __fmul2_rn(__fadd2_rn(f[j], pair_of(-mu[i])), pair_of(rs));
                    f[j] = __ffma2_rn(hat, k.scale[j], k.bias[j]);   // weight and bias as they came
                }
                act_value(act, f, v);
                if (s.live && i < n) {
                    oct_store<DT, true>(out + i * to.step, s.at, oct_round<DT>(v));
                    if (first) {
                        pm[i * step_s] = mu[i];
                        pr[i * step_s] = rs;
                    }
                }
            }
        });
        out += 4 * to.step;
        pm += 4 * step_s;
        pr += 4 * step_s;
        if constexpr (HOLD) {
            hold_rows<DT, true>(o, s.live, s.at, a.lay.team, a.form, HeldRows{hp, n});
            hp.advance(4);
        }
    };
    // every lane of a warp comes to the shuffles
    extern __shared__ float4 queue[];
    each_four<DT, true>(walk<DT>(x, row0, P, a.x_pitch, s), s.at, reinterpret_cast<char*>(queue), (rows + P - 1) / P,
                        mine, s.live, [] {}, use);
}

template <int DT, bool HELD>
__global__ void __launch_bounds__(kTokenThreads, 2)
    norm_token_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                           const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float4 shared4[];   // the queue, then the sums for dweight and dbias
    constexpr int N = kQueueBatch;
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;
    const float minus_m = -1.f / static_cast<float>(a.per_group);
    const int group = s.group0 + local_group(a, s.at.ch);
    const int P = a.lay.P, step_s = P * a.groups;
    const int64_t share = a.lay.range, first_row = static_cast<int64_t>(blockIdx.x) * share, row0 = first_row + s.p;
    const int rows = static_cast<int>(min(share, a.n - first_row));
    const int mine = s.live && s.p < rows ? (rows - s.p + P - 1) / P : 0;
    let_next_start();
    GradQueue<DT, HELD> queue(GradWalk<DT, true, HELD>(a, s, dy, x, row0, P), reinterpret_cast<char*>(shared4), mine);
    // statistics of the next rows: they come a batch ahead, as two loads in
    // 16 lanes of a group are not worth a queue
    const float* pm = mean + row0 * a.groups + group;
    const float* pr = rstd + row0 * a.groups + group;
    float next_mu[N], next_rs[N];
    auto ask_stats = [&](int left) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            next_mu[i] = i < left ? __ldg(pm + i * step_s) : 0.f;
            next_rs[i] = i < left ? __ldg(pr + i * step_s) : 0.f;
        }
        pm += N * step_s;
        pr += N * step_s;
    };
    ask_stats(mine);
    Chan<true> k;
    k.params<DT, true>(a, s, weight, bias);
    WalkOut to = walk_out<DT>(dx, row0, P, a.x_pitch, s);
    float2 sz[4], szx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sz[j] = szx[j] = make_float2(0.f, 0.f);
    const int loop = (rows + P - 1) / P;   // every lane of a warp comes to the shuffles
    for (int done = 0; done < loop; done += queue.kRows)
#pragma unroll 1
        for (int b = 0; b < queue.kBatches && done + b * N < loop; ++b) {
            const int n = mine - done - b * N;
            float mu[N], rs[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                mu[i] = next_mu[i];
                rs[i] = next_rs[i];
            }
            ask_stats(n - N);
            cp_async_wait(queue.kBatches - 1);
            GradRow<DT, true, HELD> g[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n)
                    queue.take(b, i, g[i]);
                else
                    g[i].clear();
            by_act(a.act, [&](auto act) {
                float2 hat[N][4], dz[N][4];
                float s1[N], s2[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float2 fd[4], t1 = make_float2(0.f, 0.f), t2 = t1;
                    oct_floats(g[i].dy, fd);
                    k.statistics(mu[i], rs[i]);
                    g[i].hats(a.form, k, hat[i]);
                    k.slopes(act, fd, hat[i], dz[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 dzx = __fmul2_rn(dz[i][j], hat[i][j]);
                        sz[j] = __fadd2_rn(sz[j], dz[i][j]);
                        szx[j] = __fadd2_rn(szx[j], dzx);
                        t1 = __ffma2_rn(dz[i][j], k.w[j], t1);
                        t2 = __ffma2_rn(dzx, k.w[j], t2);
                    }
                    s1[i] = t1.x + t1.y;
                    s2[i] = t2.x + t2.y;
                }
                team_sums(s1, lanes);
                team_sums(s2, lanes);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    Gradient<true> grad;
                    float2 out[4];
                    k.statistics(mu[i], rs[i]);
                    grad.set(a, k, s1[i] * minus_m, s2[i] * minus_m);
                    grad.of(k, dz[i], hat[i], out);
                    if (i < n)
                        oct_store<DT, true>(to.p + i * to.step, s.at, oct_round<DT>(out));
                }
            });
            queue.ask(b);
            to.p += N * to.step;
        }
    cp_async_wait(0);
    __syncthreads();
    const int width = s.at.cols, slot = slot_stride(width);
    float2* work = reinterpret_cast<float2*>(shared4);   // [threads]
    float2* columns = work + kTokenThreads;              // [run_cols]
    float2* slots = columns + a.lay.run_cols;            // [P][stride]
    if (s.live)
        leave_sums(s.at, sz, szx, slots + s.p * slot);
    __syncthreads();
    sum_lanes(slots, slot, 1, P, width, columns, work);
    add_slice(chan, a.c, s.ch0, width, false, [&](int ch) { return columns[ch]; });
}

}  // namespace

cudaError_t launch_norm_token(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias,
                              void* y, float* mean, float* rstd, HeldOut held, cudaStream_t st)
{
    const dim3 grid(unsigned(a.lay.splits), unsigned(a.lay.runs));
    cudaError_t e = cudaSuccess;
#define CALL(DT)                                                                                                     \
    e = held.q ? launch_grid<norm_token_kernel<DT, true>>(grid, a.lay.threads, RowQueue<DT>::kBytes, 1, false, st,   \
                                                          a, x, weight, bias, y, mean, rstd, held)                   \
               : launch_grid<norm_token_kernel<DT, false>>(grid, a.lay.threads, RowQueue<DT>::kBytes, 1, false, st,  \
                                                           a, x, weight, bias, y, mean, rstd, held)
    if (dtype == TSX_F16) { CALL(TSX_F16); }
    else if (dtype == TSX_BF16) { CALL(TSX_BF16); }
    else { CALL(TSX_F32); }
#undef CALL
    return e;
}

cudaError_t launch_norm_token_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                       const void* bias, const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, NormScratch scratch, cudaStream_t st)
{
    const dim3 grid(unsigned(a.lay.splits), unsigned(a.lay.runs));
    const size_t slots =
        (kTokenThreads + a.lay.run_cols + size_t(a.lay.P) * slot_stride(a.lay.run_cols)) * sizeof(float2);
    cudaError_t e = cudaSuccess;
#define CALL(DT)                                                                                                 \
    e = x.q ? launch_grid<norm_token_grad_kernel<DT, true>>(grid, a.lay.threads,                                 \
                                                            std::max(slots, GradQueue<DT, true>::kBytes), 1,     \
                                                            false, st, a, dy, x, weight, bias, mean, rstd, dx,   \
                                                            scratch.chan)                                        \
            : launch_grid<norm_token_grad_kernel<DT, false>>(grid, a.lay.threads,                                \
                                                             std::max(slots, GradQueue<DT, false>::kBytes), 1,   \
                                                             false, st, a, dy, x, weight, bias, mean, rstd, dx,  \
                                                             scratch.chan)
    if (dtype == TSX_F16) { CALL(TSX_F16); }
    else if (dtype == TSX_BF16) { CALL(TSX_BF16); }
    else { CALL(TSX_F32); }
#undef CALL
    if (e != cudaSuccess)
        return e;
    return launch_norm_params(a, a.lay.slices, scratch.chan, dweight, dbias, st);
}

}  // namespace tsx
