// Internal declarations of the operators around attention
// (include/tsx_attention.h): their kernels' arguments.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tsx_attention.h"
#include "tsx_internal.h"

namespace tsx {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryDim = 256;   // channels of a head at most

// One of the tensors that a rotary call goes over: its CTAs, `first` .. first +
// ctas - 1, work on the heads of tokens, `parts` teams of threads to a token.
struct RotaryRole {
    const char* x;       // forward: what is normed and turned; backward: the gradient
    const char* saved;   // backward: the forward call's input
    char* out;
    int64_t x_pitch, x_head, saved_pitch, saved_head, out_pitch, out_head;
    const void* weight;   // NULL: ones
    float* slices;        // backward: [ctas][dim] sums for the weight's gradient, or NULL
    int heads, parts, first, ctas;
    int which;            // 0 queries, 1 keys, 2 values
    int turn;             // 0: neither normed nor turned
    int paged;            // out is a cache, out_pitch its slots' pitch
    int packed_weight;    // the weight is aligned to 16 bytes
};

// Keys of a sequence at most, so that positions and what is added to them fit 32 bits.
constexpr int kMostKeys = 0x7fffffff - (1 << 20);

// Where the tokens of a batch lie (see tsx_batch and tsx_cache).
struct PagedArgs {
    const int32_t *starts, *lengths, *pages;
    int64_t pages_pitch, cache_pages, page_pitch;
    int seqs, most_pages, page_size;
    int page_shift;   // log2 of a page size that is a power of two, else -1
};

struct RotaryArgs {
    RotaryRole role[3];
    int roles;
    int64_t tokens;
    const void* positions;   // NULL: the batch's
    int wide_positions;      // of 8 bytes
    int dim, rot, layout, norm, wide_params;
    int team;                // threads to a head: a power of two
    float eps, amplitude, by_dim;   // by_dim: 1 / dim
    PagedArgs paged;
    alignas(16) uint64_t turns[TSX_ROPE_PAIRS];
};

// Heads that a thread of the vector kernels has on their way while it works on as
// many, forward; backward half as many, of two tensors.
TSX_HD constexpr int rotary_batch(int dtype) { return dtype == TSX_F32 ? 2 : 4; }
// CTAs of the gradient through a norm that an SM holds: bf16 [8192, 32 + 8, 128] 60.6
// us in three with one head under way, 56.2 in two with two; fp32 the other way round,
// 46.7 and 54.1.
TSX_HD constexpr int backward_ctas(int dtype) { return dtype == TSX_F32 ? 3 : 2; }

cudaError_t launch_rotary(int dtype, const RotaryArgs& a, bool vec, int ctas, cudaStream_t st);
cudaError_t launch_rotary_norm_backward(int dtype, const RotaryArgs& a, bool vec, int ctas, cudaStream_t st);
// dq_weight and dk_weight from the roles' slices.
cudaError_t launch_rotary_weights(const RotaryArgs& a, float* dq_weight, float* dk_weight, cudaStream_t st);

namespace dev {
struct Tail;
}

// Attention over a paged cache (csrc/tsx_attend.cuh).
struct AttendArgs {
    PagedArgs paged;
    const char *k, *v, *q;
    char* out;
    float* lse;
    int64_t slot_pitch, head_pitch, q_pitch, q_head, out_pitch, out_head, tokens;
    int heads, group, dim;   // heads of the cache, queries to each
    float scale_log2;        // scale / ln 2
    int negated;             // many rows: scores of -q, and scale_log2 above 0
    int ctas;
    // scratch: for each CTA two slots of [rows][padded dim] sums and [rows] (maximum, sum of weights), and its Tail
    float* parts;
    float2* stats;
    dev::Tail* tails;
    float4* folded;   // and for each of its threads with sums a row of those and one more
};
// Threads of a CTA that hold sums, and how many fours of them each.
TSX_HD constexpr int fold_threads(bool many) { return many ? 256 : 128; }
TSX_HD constexpr int fold_fours(bool many, int padded) { return many ? padded / 4 : padded / 8; }
// Few rows to a head, any dim: tiles of 8 or of 16 `rows`.
int attend_few_ctas(int dim);
// Many rows to a head, dim up to 128: one CTA to an SM.
int attend_many_rows();
// maps: of keys and values in boxes of 64 channels and min(page, 128) slots, or NULL.
cudaError_t launch_attend_many(int dtype, const AttendArgs& a, const CUtensorMap* maps, cudaStream_t st);
cudaError_t launch_attend_few(int dtype, const AttendArgs& a, int rows, cudaStream_t st);

}  // namespace tsx
