// Internal declarations of the layer operators (include/tsx_layers.h): how
// their rows are laid over threads, and their kernels' arguments.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tsx_internal.h"
#include "tsx_layers.h"

namespace tsx {

// t / V for a thread t, as t * per >> 20 with per = (2^20 + e) / V, 0 <= e < V:
// the product is t / V * 2^20 and less than 2^20 / V more while t e < 2^20,
// which t, V < 2^10 are.  The kernels' CTAs live for a few rows, so that the
// tens of instructions of a division count.
constexpr uint32_t lane_factor(int V) { return ((1u << 20) + uint32_t(V) - 1) / uint32_t(V); }
TSX_HD constexpr int lane_of(int t, uint32_t per) { return int((uint32_t(t) * per) >> 20); }

// How [rows, cols] is laid over CTAs and threads.  A row is cut into `chunks`
// runs of chunk_cols channels (grid.y); a CTA holds P rows of one run at a
// time, V threads to a row, each with eight channels (csrc/tsx_oct.cuh).
struct RowLayout {
    int64_t rows;
    int cols;
    int chunk_cols;   // channels of a run: a multiple of 8, of the block where there are checkpoints
    int chunks;
    int V;            // threads to a row: ceil(chunk_cols / 8) rounded up to whole teams
    uint32_t per_v;   // lane_factor(V)
    int P;            // rows side by side
    int team;         // neighbouring threads that share a checkpoint block (1, 2, ..., 16)
    int threads;      // P * V rounded up to whole warps
    bool vec;         // 16-byte vectors (else element by element)
};

constexpr int kOct = 8;                // channels to a thread
constexpr int kLayerThreads = 256;     // most threads of an elementwise layer kernel's CTA
constexpr int kNormThreads = 256;      // of a group-norm kernel's
constexpr int kTokenThreads = 256;

// The layout of rows cut for CTAs of about `want` threads; block: channels
// to a scale, 0 without checkpoints.
RowLayout row_layout(int64_t rows, int64_t cols, int block, bool vec, int want);

// A tensor as the kernels take it: `q` and `scale` in place of `x` for a
// checkpoint ([rows, cols] bytes and [rows, ceil(cols / block)] floats).
struct Saved {
    const void* x;
    const void* q;
    const float* scale;
};
struct HeldOut {
    void* q;
    float* scale;
};

struct PackArgs {
    RowLayout lay;
    int64_t pitch;
    int form, block;
    int64_t blocks;   // scales to a row
};
cudaError_t launch_pack(int dtype, const PackArgs& a, const void* x, HeldOut held, cudaStream_t st);
cudaError_t launch_unpack(int dtype, const PackArgs& a, const void* q, const float* scale, void* x, cudaStream_t st);

struct GatedArgs {
    RowLayout lay;
    int64_t in_pitch, out_pitch;
    int act, form, block;
    int64_t blocks;
};
cudaError_t launch_gated(int dtype, const GatedArgs& a, const void* gate, const void* up, void* h, HeldOut held_gate,
                         HeldOut held_up, cudaStream_t st);
cudaError_t launch_gated_backward(int dtype, const GatedArgs& a, const void* dh, Saved gate, Saved up, void* dgate,
                                  void* dup, void* h, cudaStream_t st);

// Group norm.  The channels are cut into runs that hold whole groups (or, for
// groups wider than a CTA's row, into `pieces` runs a group), the l rows of a
// sample into `splits` ranges; a CTA takes one range of one run.
struct NormLayout {
    bool vec;
    bool oct_in_group;   // vec, and eight consecutive channels never straddle two groups
    int team;            // as in RowLayout
    int run_groups;      // groups to a run
    int run_cols;        // channels of a run
    int runs;
    int pieces;          // runs to a group (1 unless a group is wider than a CTA's row)
    int V, P, threads;
    uint32_t per_v;      // lane_factor(V)
    int64_t splits;      // row ranges of a sample; token kernels: CTAs that share the rows of a run
    int64_t range;       // rows to a range, or to a rank
    int64_t slices;      // backward: CTAs that share a run's samples; each adds up its own for dweight and dbias
    // kernels that hold samples on chip: CTAs of a cluster that share a
    // sample, samples side by side in a CTA, row lanes of each (P = samples * lanes)
    int ranks, samples, lanes;
    int lane_rows;       // rows to a lane at most
    int shares, share_lanes;   // forward: shares of the row lanes that are joined first, and lanes to a share
    int kind;            // NormKind
};
// How a call runs: streaming kernels that read their operands twice (any
// layout), samples held on chip, tokens whose groups lie within a warp.
enum NormKind { kNormStream = 0, kNormHeld = 1, kNormToken = 2 };

struct NormArgs {
    NormLayout lay;
    int64_t n, l;
    int c, groups, per_group;
    int64_t x_pitch, y_pitch;
    float eps;
    int act, form, block;
    int64_t blocks;      // scales to a row of a checkpoint
    int wide_params;     // weight and bias are fp32 (else of the element type)
    int packed_params;   // and both aligned to 16 bytes
};

// Scratch of one call (see tsx_group_norm_workspace):
//   part   streaming: [n][splits * pieces][groups] pairs: (mean, sum of squared deviations)
//          forward, the two sums of the gradient backward
//   chan   [slices][2][c] backward: sums for dweight and dbias, one slice to each of a run's
//          CTAs; at most 16 MB, or one slice
struct NormScratch {
    float2* part;
    float* chan;
};

cudaError_t launch_norm(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                        float* mean, float* rstd, HeldOut held, NormScratch scratch, cudaStream_t st);
cudaError_t launch_norm_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                 const void* bias, const float* mean, const float* rstd, void* dx, float* dweight,
                                 float* dbias, NormScratch scratch, cudaStream_t st);
// Shared memory of a CTA of the kernels that hold samples on chip.
size_t held_bytes(const NormLayout& lay, int es, bool backward, bool held);
cudaError_t launch_norm_held(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, HeldOut held, cudaStream_t st);
cudaError_t launch_norm_held_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                      const void* bias, const float* mean, const float* rstd, void* dx,
                                      float* dweight, float* dbias, NormScratch scratch, cudaStream_t st);
cudaError_t launch_norm_token(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias,
                              void* y, float* mean, float* rstd, HeldOut held, cudaStream_t st);
cudaError_t launch_norm_token_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                       const void* bias, const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, NormScratch scratch, cudaStream_t st);
// dweight and dbias from [slices][2][c] partial sums.
cudaError_t launch_norm_params(const NormArgs& a, int64_t slices, const float* chan, float* dweight, float* dbias,
                               cudaStream_t st);
// Statistics of groups without elements: mean 0, rstd 1 / sqrt(eps).
cudaError_t launch_norm_empty(float* mean, float* rstd, int64_t count, float eps, cudaStream_t st);

}  // namespace tsx
