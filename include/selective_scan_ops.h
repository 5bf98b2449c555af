/*
 * selective_scan_ops.h -- C ABI of the operators around the selective scan: its gradient, the
 * gated linear recurrence with its gradient, the single-token step, and the parking of recurrent
 * states in 8 or 4 bits.  They live in the same library as selective_scan_fwd and follow the
 * conventions stated at the top of selective_scan.h: dense row-major DEVICE pointers owned by the
 * caller, no allocation, no synchronisation, work enqueued on `stream` (of the current device,
 * SS_ERR_DEVICE otherwise), arguments validated before anything is launched, base pointers of io
 * tensors and workspaces 16-byte aligned and dim * sizeof(io element) a multiple of 16.  Inputs
 * must not overlap outputs or the workspace.  A workspace belongs to one call until that call's
 * work is done; its contents on entry do not matter.  Results do not depend on the order in which
 * blocks run: no floating-point atomics.
 *
 * Every call can be captured into a CUDA graph, after a first call of its kind on the device (which
 * loads the kernels and looks up the device error word); while a stream is captured its device is
 * not checked.  gated_recurrence_fwd and gated_recurrence_bwd wait inside a kernel for the other
 * blocks of a cluster; like every wait of the library these are bounded (2 s) and a wait that gives up is
 * reported by selective_scan_device_status.
 */
#ifndef SELECTIVE_SCAN_OPS_H
#define SELECTIVE_SCAN_OPS_H

#include "selective_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ gated linear recurrence
 *
 *   s_t = gate_t + gate_bias            (SS_GATE_SIGMOID; gate_bias may be NULL for zero)
 *   a_t = sigmoid(s_t)                  SS_GATE_SIGMOID
 *   a_t = exp(gate_t)                   SS_GATE_EXP: the gate is the logarithm of the decay
 *                                       (normally <= 0; gate_bias must be NULL)
 *   h_t = a_t * h_{t-1} + c_t * x_t     c_t = 1 - a_t with `complement`, 1 without
 *   out_t = h_t
 *
 * elementwise per channel, along t = 0..L-1 (SS_DIR_FWD) or t = L-1..0 (SS_DIR_REV).  The state
 * is held in fp32; out is rounded to the io type once.  Both a and 1 - a are relatively accurate (2^-21
 * and |s_t| 2^-22; the sigmoid down to 2^-100), so that a memory of thousands of steps keeps its length
 * and a gate that closes leaves a h_{t-1} and nothing else.  An infinite state stays: no decay is below 2^-149, that of
 * a gate of -inf included.
 */
typedef enum { SS_GATE_SIGMOID = 0, SS_GATE_EXP = 1 } ss_gate_form;

typedef struct {
    int32_t form;       /* ss_gate_form                                                       */
    int32_t complement; /* nonzero: c_t = 1 - a_t                                             */
    int32_t dir;        /* SS_DIR_FWD or SS_DIR_REV                                           */
    int32_t reserved;   /* must be 0                                                          */
} ss_recurrence_opts;

/* Bytes of workspace of the two calls below (0: none needed).  `shape->dstate` must be 1; `backward` selects
 * the call.  Host-only. */
ss_status gated_recurrence_workspace_size(const ss_shape* shape, const ss_recurrence_opts* opts,
                                          int32_t backward, size_t* bytes);

/*   x, gate        [batch, L, D] io        gate_bias      [D] fp32 or NULL
 *   initial_state  [batch, D] fp32 or NULL (zero)
 *   out            [batch, L, D] io        last_state     [batch, D] fp32 or NULL: the state
 *                                                         after the last step visited        */
ss_status gated_recurrence_fwd(const ss_shape* shape, const ss_recurrence_opts* opts,
                               const void* x, const void* gate, const float* gate_bias,
                               const float* initial_state, void* out, float* last_state,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of a scalar loss through gated_recurrence_fwd.
 *
 *   G_t   = dout_t + a_{t+1} G_{t+1}         (dlast_state added at the last step visited)
 *   dx    = c_t G_t
 *   ds    = G_t (h_{t-1} - [complement] x_t) a_t (1 - a_t)     SS_GATE_SIGMOID
 *   dgate = G_t (h_{t-1} - [complement] x_t) a_t               SS_GATE_EXP
 *
 *   out            the forward call's output (the states, as rounded to the io type)
 *   dout           [batch, L, D] io        dlast_state    [batch, D] fp32 or NULL (zero)
 *   dx, dgate      [batch, L, D] io        dgate_bias     [D] fp32 or NULL (SS_GATE_SIGMOID)
 *   dinitial_state [batch, D] fp32 or NULL
 */
ss_status gated_recurrence_bwd(const ss_shape* shape, const ss_recurrence_opts* opts,
                               const void* x, const void* gate, const float* gate_bias,
                               const float* initial_state, const void* out, const void* dout,
                               const float* dlast_state, void* dx, void* dgate,
                               float* dgate_bias, float* dinitial_state, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ gradient of the scan
 *
 * Gradients of a scalar loss through selective_scan_fwd, for the same shape, direction map and
 * inputs.  The states are recomputed from checkpoints that the call writes to its workspace; the
 * forward call keeps nothing.  With h, Abar, Delta of direction k at step t and p = map_k(t):
 *
 *   dy    = dout_p silu(z_p)                      g_t = C_t dy + Abar_{t+1} g_{t+1}
 *   dC_t  = sum_d dy h_t                          dB_t = sum_d g_t Delta_t u_p
 *   du_p += Dskip dy + Delta_t sum_n g_t B_t      (summed over the directions that read u)
 *   dDelta_t = u_p sum_n g_t B_t + sum_n g_t A Abar_t h_{t-1}
 *   ddelta_t = dDelta_t sigmoid(delta_t + bias)   (softplus; dDelta_t without)
 *   dA    = sum_{b,t} g_t Delta_t Abar_t h_{t-1}  dDskip = sum_{b,t} dy u_p
 *   dz_p  = dout_p silu'(z_p) sum_k y_k           ddelta_bias = sum_{b,t} ddelta_t
 *
 * The state and every sum are fp32.  Gradients have the shapes and types of what they belong to.
 * The workspace is large: one state in four, 4 bytes x K x batch x L / 4 x D x N (N padded to 8 or 16),
 * and the partial sums of dB and dC over 1024 / N channels; 507 MB for 8 x 2048 x 1536 x 16, 12.8 GB
 * for 1 x 131072 x 5120 x 16.
 */
typedef struct {
    void* du;              /* [batch, L, D] io ([K, batch, L, D] with SS_FLAG_U_PER_DIRECTION)  */
    void* ddelta;          /* [K, batch, L, D] io                                               */
    float* dA;             /* [D, N] fp32 ([K, D, N] with SS_FLAG_PARAMS_PER_DIRECTION)         */
    void* dB;              /* [K, batch, L, N] io                                               */
    void* dC;              /* [K, batch, L, N] io                                               */
    float* dDskip;         /* [D] or [K, D] fp32, or NULL (may be asked for only with Dskip)    */
    void* dz;              /* [batch, L, D] io: required with z, NULL without                   */
    float* ddelta_bias;    /* [D] or [K, D] fp32, or NULL (may be asked for only with the bias) */
    float* dinitial_state; /* [K, batch, D, N] fp32, or NULL                                    */
} ss_scan_grads;

/* opts may give `segments`, `initial_state` and the flags SS_FLAG_GENERIC_A (no effect: the
 * gradient always takes the general A), SS_FLAG_U_PER_DIRECTION and SS_FLAG_PARAMS_PER_DIRECTION.
 * The exact ZOH, int8 Delta, the fused convolution, the timing events and the test hook are
 * refused with SS_ERR_UNSUPPORTED. */
ss_status selective_scan_bwd_workspace_size(const ss_shape* shape, const ss_direction_map* dmap,
                                            const ss_launch_opts* opts, size_t* bytes);

/*   dout         [batch, L, D] io
 *   dlast_state  [K, batch, D, N] fp32: the gradient of last_state, or NULL (zero)
 *   grads        every one of du, ddelta, dA, dB, dC is required                             */
ss_status selective_scan_bwd(const ss_shape* shape, const void* u, const void* delta,
                             const float* A, const void* B, const void* C, const float* Dskip,
                             const void* z, const float* delta_bias, int32_t softplus,
                             const ss_direction_map* dmap, const void* dout,
                             const float* dlast_state, const ss_scan_grads* grads,
                             void* workspace, size_t workspace_bytes, void* stream,
                             const ss_launch_opts* opts);

/* ------------------------------------------------------------------ single-token step
 *
 * One step of the forward scan for each of `batch` rows, on states that stay in a pool: row r
 * works on state[slots[r]], which is updated in place.  The arithmetic of selective_scan_fwd with
 * one forward direction: u (after the optional causal convolution and SiLU), Delta, the
 * recurrence, the readout with the D skip, the silu(z) gate.
 *
 *   shape        batch rows, seqlen must be 1, dim, dstate, io type; num_slots >= 1
 *   u, delta, z  [batch, D] io (z may be NULL)       B, C   [batch, N] io
 *   A, Dskip, delta_bias as in selective_scan_fwd
 *   state        [num_slots, D, N] fp32, 16-byte aligned, in place
 *   slots        [batch] int32 device array, or NULL for slot r = row r.  A row whose slot is
 *                outside [0, num_slots) is padding: its out row and every state stay as they
 *                were.  Of several rows that name one slot, the lowest takes it and the others
 *                are padding.  Every row looks through the entries before its own, so the look-ups
 *                grow with the square of the rows (nothing beside the states for some thousand of
 *                them); with a list, batch is at most 2^20 (SS_ERR_SHAPE)
 *   conv_weight  [D, conv_width] fp32 (conv_width 1..SS_MAX_CONV_WIDTH) or NULL; conv_bias [D]
 *                fp32 or NULL; tap conv_width-1 multiplies this token's u
 *   conv_state   [num_slots, conv_width-1, D] io: the inputs before this token, oldest first, in
 *                place (shifted by one); required with conv_width >= 2
 *   out          [batch, D] io
 */
ss_status selective_scan_step(const ss_shape* shape, int64_t num_slots, const void* u,
                              const void* delta, const float* A, const void* B, const void* C,
                              const float* Dskip, const void* z, const float* delta_bias,
                              int32_t softplus, float* state, const int32_t* slots,
                              const float* conv_weight, const float* conv_bias,
                              int32_t conv_width, void* conv_state, void* out, void* stream);

/* ------------------------------------------------------------------ parked states
 *
 * States of sequences that do not run (a prefix that will be continued, a preempted sequence) in
 * 8 or 4 bits: per (slot, channel) one fp32 scale and N codes,
 *
 *   amax = max_n |h_n|;  code_n = round(h_n * q / amax), ties to even;  scale = amax / q
 *   h_n is read back as code_n * scale                   q = 127 (8 bits), 7 (4 bits)
 *
 * An all-zero channel has scale 0 and codes 0.  A channel that holds an infinity or a NaN has
 * scale NaN and codes 0, and reads back as NaN in every state.
 *
 *   codes   [cache_slots, D, N] int8 (8 bits) or [cache_slots, D, (N+1)/2] bytes (4 bits: two's
 *           complement nibbles, the even state in the low half, 0 behind an odd N)
 *   scales  [cache_slots, D] fp32
 *   state   [state_slots, D, N] fp32, 16-byte aligned
 *   src_slots, dst_slots  [rows] int32 device arrays, or NULL for slot r = row r; rows with a
 *           slot outside its pool are skipped, and of several rows with one destination the
 *           lowest is taken; with a list of destinations rows is at most 2^20 (SS_ERR_SHAPE), as in
 *           the step
 */
ss_status selective_state_store(int64_t rows, int64_t dim, int64_t dstate, int32_t bits,
                                const float* state, int64_t state_slots,
                                const int32_t* src_slots, void* codes, float* scales,
                                int64_t cache_slots, const int32_t* dst_slots, void* stream);

ss_status selective_state_load(int64_t rows, int64_t dim, int64_t dstate, int32_t bits,
                               const void* codes, const float* scales, int64_t cache_slots,
                               const int32_t* src_slots, float* state, int64_t state_slots,
                               const int32_t* dst_slots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELECTIVE_SCAN_OPS_H */
