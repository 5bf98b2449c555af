// Launch parameters and launchers of the operators around the scan, shared by their host entry
// points (so_api.cu) and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "selective_scan_ops.h"

namespace so {

// ---------------------------------------------------------------- gated linear recurrence

struct RecParams {
    const void* x;         // [batch, L, D] io
    const void* gate;      // [batch, L, D] io
    const float* bias;     // [D] or null
    const float* init;     // [batch, D] or null
    const void* out_in;    // backward: the forward call's output
    const void* dout;      // backward
    const float* dlast;    // backward: [batch, D] or null
    void* out;             // forward: [batch, L, D]; backward: dx
    void* dgate;           // backward
    float* last;           // forward: last state or null; backward: dinitial or null
    float* dbias_part;     // backward: [batch * S * cluster, D] partial sums of ds, or null
    float* dbias;          // backward: [D] or null
    int64_t batch, L, D;
    float4* seg_maps;      // [columns, S, 32] maps of the segments of a split column (S > 1)
    int32_t cluster;       // CTAs that walk one column of 64 channels together
    int32_t S, seg_len;    // segments of a column, their steps (whole rounds of the cluster)
    int32_t aggregate;     // set by the launcher
    int32_t form, complement, reverse;
    unsigned int* status;  // the device error word, or'ed by waits that gave up
};

constexpr int kRecMostCluster = 8;

cudaError_t launch_recurrence(const RecParams& p, int io_dtype, bool backward, cudaStream_t st);

// Steps of a CTA's tile.
int recurrence_tile(int io_dtype, bool backward);

// ---------------------------------------------------------------- gradient of the scan

struct BwdParams {
    const void *u, *delta, *B, *C, *z, *dout;
    const float *A, *Dskip, *bias, *init, *dlast;
    ss_scan_grads g;
    float* ckpt;      // states at the start of every slice, from the segment start (thread order)
    float* cum;       // [K*batch, slices, D] Delta summed from the segment start (SPLIT)
    float* seg_h;     // [K*batch, S, cells] end state of a segment scanned from zero
    float* seg_p;     // the same shape: product of Abar over the segment
    float* seg_g;     // the same shape: gradient that a zero-ended segment hands to the one before
    float* dbc;       // [K*batch, channel tiles, L, 2, states padded] partial sums of dB and dC
    float* dpar;      // [K*batch*S, D, states padded + 2] partial sums of dA, dDskip, ddelta_bias
    float* du_part;   // [K, batch, L, D] (several directions share u)
    float* dz_part;   // [K, batch, L, D] (several directions with a gate)
    int64_t batch, L, D, seg_len;
    int32_t N, K, S;
    int32_t dirs[SS_MAX_DIRS];
    int32_t H, W;
    int32_t softplus, u_per_dir, params_per_dir;
};

constexpr int kBwdTile = 4;       // steps of a slice: one checkpoint each
constexpr int kBwdCells = 1024;   // (channel, state) cells of a CTA, states padded to 8 or 16

// One translation unit per io type and number of groups of 4 states (2: N up to 8, 4: up to 16).
cudaError_t launch_scan_bwd_f32_2(const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_f32_4(const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_bf16_2(const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_bf16_4(const BwdParams& p, cudaStream_t st);

// ---------------------------------------------------------------- single-token step

struct StepParams {
    const void *u, *delta, *B, *C, *z;
    const float *A, *Dskip, *bias, *conv_w, *conv_b;
    float* state;
    const int32_t* slots;
    void* conv_state;
    void* out;
    int64_t batch, D, num_slots;
    int32_t N, softplus, conv_width;
    int32_t rows;  // rows of a CTA, set by the launcher
};

cudaError_t launch_step(const StepParams& p, int io_dtype, cudaStream_t st);

// ---------------------------------------------------------------- parked states

struct StateParams {
    const float* state_in;  // store
    float* state_out;       // load
    uint8_t* codes;
    float* scales;
    const int32_t* src;     // slots of the source pool, or null
    const int32_t* dst;     // slots of the destination pool, or null
    int64_t src_slots, dst_slots;
    int64_t rows, D;
    int32_t N, bits;
};

cudaError_t launch_state(const StateParams& p, bool load, cudaStream_t st);

}  // namespace so
