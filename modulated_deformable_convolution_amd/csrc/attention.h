// attention.h -- arguments and launchers of the attention operators: rotary
// positions, norms of queries and keys, attention over packed sequences.
#pragma once

#include <hip/hip_runtime_api.h>
#include <hip/hip_vector_types.h>

#include <cstddef>
#include <cstdint>

#include "mdcn.h"

namespace mdcn {

constexpr int kMaxRotaryDim = 256;
constexpr int kMaxRotaryAxes = 8;
constexpr int kMaxAttendDim = 128;

// [tokens][heads][dim] in device memory, dim contiguous; strides in elements.
struct Heads {
    const void *data;
    int64_t token_stride, head_stride;
};

// The angle of pair i at position p is turns[i] * p, in units of 2^-64 turns, modulo
// a turn.  Passed to the kernels by value (1.2 KB of kernel arguments), so a handle
// holds no device memory.
struct RotaryTable {
    uint64_t turns[kMaxRotaryDim / 2];
    uint8_t axis[kMaxRotaryDim / 2];
};

struct RotaryArgs {
    Heads q, k;            // rotate, norm_rotate: inputs; backward: the forward's inputs
    Heads gq, gk;          // norm_rotate's backward: gradients of its outputs
    Heads oq, ok;          // outputs (backward: gradients of the inputs)
    const void *q_gain, *k_gain;
    float *partial;        // backward: [blocks][2][dim] sums of the gains' gradients
    const int32_t *positions;
    int64_t axis_stride, tokens;
    int32_t q_heads, k_heads, dim, pairs;
    int32_t adjacent, inverse;
    float eps;
    RotaryTable table;
};

enum class RotaryKind { Rotate, NormRotate, NormRotateBackward };

// Blocks of the backward, one row of `partial` each.
int rotary_backward_blocks(int64_t tokens);
// How a call is laid out: values of a vector, lanes of a head, rounds of heads that a wave
// takes and waves that share a token's.
struct RotaryShape {
    int width, lanes, rounds, waves;
};
RotaryShape rotary_shape(RotaryKind kind, mdcn_dtype dtype, const RotaryArgs &a);
hipError_t launch_rotary(RotaryKind kind, mdcn_dtype dtype, const RotaryArgs &a, hipStream_t s);
// Sums partial's rows into the two gain gradients.
hipError_t launch_gain_sum(mdcn_dtype dtype, const RotaryArgs &a, void *dq_gain, void *dk_gain,
                           hipStream_t s);

struct AttendArgs {
    Heads q, k, v, out;    // out: output of the forward, input of the backward
    Heads go, dq, dk, dv;  // backward
    float *lse;            // [q_heads][q_tokens]
    // backward: [q_heads][q_tokens], {lse * log2(e) (fp16: 15 less), sum of go * out}
    float2 *stats;
    // backward in fp16, at every 32nd row of a sequence: the largest of 32 rows
    float2 *row_tops;      // [q_heads][q_tokens], {|go|, |sum of go * out|}
    float *key_tops;       // [k_heads][k_tokens], |v|
    const int32_t *cu_q, *cu_k, *used_k;
    int32_t batch, q_tokens, k_tokens;
    int32_t q_heads, k_heads, dim, causal;
    float scale;
    int32_t workers;       // split kernel: workgroups, and its unit is 32 << unit_shift keys
    int32_t unit_shift;
    int32_t splits;        // backward: workgroups that share a tile of keys
    int32_t fill;          // forward: kFillOut, kFillLse
    int32_t fill_from;     // first of the workgroups that fill (see outside_rows)
    int32_t tops_from;     // backward in fp16: first of the workgroups that take key_tops
    float *partial;        // sums that several workgroups leave for one result
};

// Whether tokens that belong to no sequence get zeros in out and -infinity in lse.
constexpr int kFillOut = 1, kFillLse = 2;

// Waves that share the keys of 32 queries in attend, and of dq in the backward: 1 in
// workgroups of 128 queries, 2 or 4 in workgroups of 64.
int attend_key_waves(mdcn_dtype dtype, const AttendArgs &a);
hipError_t launch_attend(mdcn_dtype dtype, const AttendArgs &a, hipStream_t s);
// Whether the kernel that splits keys over the chip is the faster one for a
// batch of these sizes.
bool attend_prefers_split(mdcn_dtype dtype, const AttendArgs &a);
// Workgroups of the split kernel and the bytes of `partial` they need.
int attend_split_workers(mdcn_dtype dtype, int dim);
size_t attend_split_bytes(mdcn_dtype dtype, int dim);
int attend_split_unit_shift(const AttendArgs &a);
hipError_t launch_attend_split(mdcn_dtype dtype, AttendArgs a, hipStream_t s);
// Workgroups that share the queries of a tile of keys; more than one need
// splits * 2 * k_tokens * k_heads * dim floats of `partial`.
int attend_backward_splits(const AttendArgs &a);
hipError_t launch_attend_backward(mdcn_dtype dtype, const AttendArgs &a, hipStream_t s);

}  // namespace mdcn
