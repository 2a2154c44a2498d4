/*
 * kda.h - C ABI of the MI355X (gfx950) Kimi Delta Attention core.
 *
 * The operation is the gated delta rule with a bounded per-channel decay:
 *
 *   g_t  = g_min * sigmoid(exp(A_log[h]) * z_t)      per Dk channel
 *   S_t  = (I - beta_t k_t k_t^T) Diag(exp(g_t)) S_{t-1} + beta_t k_t v_t^T
 *   o_t  = S_t^T q_t
 *
 * with q, k L2-normalised and beta = sigmoid(beta_raw).  Decay is applied before
 * the delta erase and the readout uses the updated state ("Implémenter KDA",
 * 'La forme récurrente de référence' and its pitfalls).  The gate is the bounded
 * one of "线性注意力交互式演示" §1.2 Eq. 8 and "Implémenter KDA" 'La décroissance
 * bornée'.  The three switches mirror the in-kernel switches of "KDAAttention
 * 层", 'chunk_kda 内部做了什么'.
 *
 * Conventions for every entry point:
 *  - Tensor pointers are DEVICE pointers to contiguous row-major buffers, 16-byte
 *    aligned.  Layouts: q, k, z [B,T,H,Dk]; v [B,T,H,Dv]; beta_raw [B,T,H];
 *    A_log [H] fp32; states [B,H,Dk,Dv] fp32; transitions [B,H,Dk,Dk] fp32.
 *    Decode tensors drop the T axis.  q, k, v, z, beta_raw and o share `dt`.
 *  - The caller owns every buffer, including the workspace.  The library never
 *    allocates, frees or synchronises; work is enqueued on `stream` (0 = null
 *    stream) and is asynchronous.
 *  - Arguments are validated on the host before anything is enqueued, so a
 *    rejected call writes nothing and makes no HIP call.  A failed launch
 *    returns KDA_ERR_HIP.  There is no global mutable state: concurrent calls
 *    are safe as long as they do not share output buffers or workspace.
 *  - Supported sizes: Dk, Dv in {16, 32, 64, 128}; chunk in {16, 32, 64}; any
 *    T >= 0 (a ragged tail chunk is padded with identity transitions).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,      /* a required pointer is NULL                         */
    KDA_ERR_SHAPE = 2,     /* unsupported or negative size, or bad chunk         */
    KDA_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned                   */
    KDA_ERR_DTYPE = 4,     /* unknown dtype or unknown switch bits               */
    KDA_ERR_GATE = 5,      /* g_min not finite or not negative (bounded gate)  */
    KDA_ERR_WORKSPACE = 6, /* workspace NULL, misaligned or too small           */
    KDA_ERR_HIP = 7,       /* a kernel launch failed                             */
    KDA_ERR_SCRATCH = 8,   /* kda_chunk_fwd_noalloc: sizes beyond its scratch   */
    KDA_ERR_SCALE = 9      /* a scale is not finite (for softmax: or below 2^-64) */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* Switch bits ("KDAAttention 层", 'three in_kernel switches'; all on by default).
 * With a bit clear the caller supplies the activated value in the same slot:
 * the already-normalised q/k, beta itself in place of beta_raw, or the
 * log-decay g (which must lie in [g_min, 0]) in place of the gate logit z.
 *
 * KDA_GATE_SOFTPLUS (only together with KDA_GATE_IN_KERNEL, KDA_ERR_DTYPE
 * otherwise) replaces the bounded gate by the unbounded KDA v1 gate
 * g = -exp(A_log[h]) * softplus(z) ("Implémenter KDA" 'La décroissance
 * bornée', the form the bounded gate replaces; "线性注意力交互式演示" Tab 3).
 * g_min is then not used.  The chunked form stays exact for any decay: a
 * 16-token block whose decay leaves the range of the factored products is
 * evaluated element by element in log space. */
enum {
    KDA_QK_L2NORM = 1u,
    KDA_BETA_SIGMOID = 2u,
    KDA_GATE_IN_KERNEL = 4u,
    KDA_FLAGS_DEFAULT = 7u,
    KDA_GATE_SOFTPLUS = 8u
};

/* Largest token tile whose factored inverse retention exp(-g_min * n) stays
 * below dtype_max / 2^10: floor(ln(dtype_max / 2^10) / -g_min)
 * ("KDA 模块交互式演示" §1.4 safe_chunk_size; Tab 9).  Returns 16 for g_min = -5
 * with either dtype, 8 for g_min = -10, and -1 for a non-finite or
 * non-negative g_min or an unknown dtype.  Host only; no HIP call.
 * kda_chunk_fwd factors the decay of 16-token tiles; when this returns less
 * than 16 for the call's bounded gate it evaluates every tile whose decay
 * leaves the factored range element by element (the path the unbounded v1
 * gate takes), so any finite negative g_min is accepted. */
int kda_safe_chunk_size(float g_min, kda_dtype dt);

/* Bytes of device workspace kda_chunk_fwd needs for these sizes (0 for invalid
 * sizes).  The workspace holds the per-chunk intermediates of the chunkwise
 * form and the state carried between slices; it must be 256-byte aligned.
 * Host only. */
size_t kda_chunk_fwd_workspace(int B, int T, int H, int Dk, int Dv, int chunk,
                               kda_dtype dt);

/* Chunkwise KDA forward ("KDA 模块交互式演示" §1.5 Eqs. 3-4 with the UT transform;
 * "Implémenter KDA" 'La forme par blocs').  Intra-chunk work is parallel,
 * the state is carried serially from chunk to chunk in fp32.
 *   S0     nullable: initial state [B,H,Dk,Dv] fp32; NULL means zero.
 *   o      [B,T,H,Dv], dtype dt (required when T > 0).
 *   S_out  nullable: final state [B,H,Dk,Dv] fp32; may alias S0 exactly.
 *   M_out  nullable: segment transition M = M_T ... M_1 [B,H,Dk,Dk] fp32 of the
 *          whole call ("Implémenter KDA" Test 2), for segment composition.
 *   P_out  nullable: correction rows [B,T,H,Dk], dtype dt, with
 *          o_t(S0) = o_t(0) + P_t S0 ("KDA 模块交互式演示" §1.6; the recurrence is
 *          affine in S0).  Requesting M_out or P_out doubles the state width.
 *   chunk  0 selects 64.
 * Returns KDA_OK or the first validation error. */
kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const void* z,
                         const void* beta_raw, const float* A_log, const float* S0,
                         void* o, float* S_out, float* M_out, void* P_out,
                         int B, int T, int H, int Dk, int Dv, int chunk,
                         float g_min, unsigned flags, kda_dtype dt,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Number of kernels one kda_chunk_fwd call launches for these sizes (0 for
 * invalid sizes).  The intra-chunk and inter-chunk kernels alternate over
 * slices of the sequence (one slice unless the per-chunk intermediates of
 * the whole sequence exceed 1 GiB); the workspace holds one slice.  Host only. */
int kda_chunk_fwd_kernel_count(int B, int T, int H, int Dk, int Dv, int chunk, kda_dtype dt);

/* Same computation and validation as kda_chunk_fwd, for measurement: events[0]
 * is recorded on `stream` before the first kernel and events[k + 1] after
 * kernel k (kernels alternate intra-chunk, inter-chunk), so the caller can time
 * each kernel with hipEventElapsedTime.  n_events must be at least
 * kda_chunk_fwd_kernel_count(...) + 1; KDA_ERR_NULL otherwise or if an event
 * is NULL. */
kda_status kda_chunk_fwd_timed(const void* q, const void* k, const void* v, const void* z,
                               const void* beta_raw, const float* A_log, const float* S0,
                               void* o, float* S_out, float* M_out, void* P_out,
                               int B, int T, int H, int Dk, int Dv, int chunk,
                               float g_min, unsigned flags, kda_dtype dt,
                               void* workspace, size_t workspace_bytes, hipStream_t stream,
                               hipEvent_t* events, int n_events);

/* kda_chunk_fwd with the layer's input-side short convolution fused into it
 * ("KDA 模块交互式演示" §1.1 ShortConv and §1.7 完整层; "Implémenter KDA"
 * 'La paramétrisation'): q, k and v are the raw inputs of the convolution and
 * the core runs on
 *   x'[b,t,c] = SiLU(bias[c] + sum_{j=0..3} w[c,j] * x[b, t-3+j, c])
 * for each of q, k, v, with the values rounded to dt as if stored (so the
 * call equals kda_short_conv of each followed by kda_chunk_fwd, bit for bit).
 * The L2 norm of q', k' and every other switch act as in kda_chunk_fwd.
 *   conv_w      [H*Dk + H*Dk + H*Dv, 4] fp32 device: the taps of the q
 *               channels (head-major, [H][Dk]), then of the k channels, then
 *               of the v channels; tap 3 multiplies the current token.
 *   conv_b      [H*Dk + H*Dk + H*Dv] fp32 device (same channel order) or NULL.
 *   conv_state  [B, 3, H*Dk + H*Dk + H*Dv] dtype dt device or NULL (zeros):
 *               the three raw inputs before t = 0, oldest first (the window
 *               kda_short_conv hands on).  The window after the call is the
 *               last three raw inputs of (conv_state, x); the call does not
 *               write it.
 * Everything else as in kda_chunk_fwd without M_out and P_out (the same
 * workspace).  KDA_ERR_NULL without conv_w, KDA_ERR_ALIGN when conv_w,
 * conv_b or conv_state is not 16-byte aligned. */
kda_status kda_chunk_fwd_conv(const void* q, const void* k, const void* v, const void* z,
                              const void* beta_raw, const float* A_log, const float* S0,
                              const float* conv_w, const float* conv_b, const void* conv_state,
                              void* o, float* S_out, int B, int T, int H, int Dk, int Dv, int chunk,
                              float g_min, unsigned flags, kda_dtype dt,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The layer body without its projections ("KDA 模块交互式演示" §1.7
 * KimiDeltaAttention 完整层; "Implémenter KDA" 'La paramétrisation' and 'La
 * porte de sortie de rang plein'): the optional input-side convolution of
 * kda_chunk_fwd_conv, the chunkwise core of kda_chunk_fwd, and the output side
 * applied to each row of the core's output o before it is stored:
 *   y[b,t,h,c] = sigmoid(gate[b,t,h,c]) * o[b,t,h,c] * gate_weight[c]
 *                / sqrt(mean_c' o[b,t,h,c']^2 + 1e-6)
 * with o rounded to dt first (as kda_output_gate reads a stored o), so the
 * call equals kda_chunk_fwd(_conv) followed by kda_output_gate up to the
 * summation order of the norm.  o itself is never written to memory.
 *   conv_w, conv_b, conv_state  as in kda_chunk_fwd_conv; conv_w NULL: no
 *               convolution (q, k, v go to the core as given).
 *   gate        [B,T,H,Dv] dtype dt device (required when T > 0).
 *   gate_weight [Dv] fp32 device or NULL (ones), shared by the heads.
 *   y           [B,T,H,Dv] dtype dt device; it may overlap no input, S_out or
 *               the workspace (KDA_ERR_SHAPE).
 *   workspace   kda_layer_fwd_workspace bytes, 256-byte aligned: the chunk
 *               call's workspace plus an exchange area of 8 x chunk
 *               floats per chunk-head.
 * The workgroups that share a head's Dv channels exchange per-token partial
 * sums of squares through the workspace; when the device cannot hold all of
 * them at once the call runs the core into y and the output side over y in
 * place instead (same results).  The exchange counts on the device holding
 * the call's whole grid: calls of this entry point running at the same time
 * on one device (different streams) can share out its capacity so that
 * neither grid is whole, and their waits then run out after about a second
 * and write NaN rows; issue them in order on one stream.  Everything else as
 * kda_chunk_fwd without M_out and P_out. */
size_t kda_layer_fwd_workspace(int B, int T, int H, int Dk, int Dv, int chunk, kda_dtype dt);
kda_status kda_layer_fwd(const void* q, const void* k, const void* v, const void* z,
                         const void* beta_raw, const float* A_log, const float* S0,
                         const float* conv_w, const float* conv_b, const void* conv_state,
                         const void* gate, const float* gate_weight,
                         void* y, float* S_out, int B, int T, int H, int Dk, int Dv, int chunk,
                         float g_min, unsigned flags, kda_dtype dt,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

/* kda_chunk_fwd for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, computation, validation and results as kda_chunk_fwd
 * without the workspace.  The per-chunk blocks and the state carried between
 * slices of the sequence live in a built-in device buffer of 64 MiB that every
 * GPU the library runs on holds until the process ends; the sequence is cut
 * into as many slices as that buffer requires.  The call allocates nothing
 * and calls no allocating routine; its first call on a device looks up that
 * device's buffer address.
 *   Limit: B * H * (blk + Dk * (Dk + Dv) * 4) <= 64 MiB, with blk the bytes
 *   of one chunk block (28 160 for bf16, Dk = 128, chunk 32; 59 904 at chunk
 *   64; 55 808 for fp32 at chunk 32), rounded as in kda_chunk_fwd_workspace;
 *   e.g. B * H <= 421 at Dk = Dv = 128, chunk 32, bf16.  Larger sizes return
 *   KDA_ERR_SCRATCH and enqueue nothing.
 *   Every call on a GPU uses that GPU's one buffer: calls that can overlap in
 *   time on one GPU (different streams, or host threads sharing a stream
 *   without ordering) race and give wrong results.  Calls issued in order on
 *   one stream are safe; nothing in the buffer needs to start at zero. */
kda_status kda_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const void* z,
                                 const void* beta_raw, const float* A_log, const float* S0,
                                 void* o, float* S_out, float* M_out, void* P_out,
                                 int B, int T, int H, int Dk, int Dv, int chunk,
                                 float g_min, unsigned flags, kda_dtype dt, hipStream_t stream);

/* One decode step per (b,h), state updated IN PLACE ("KDA 模块交互式演示" §1.7
 * kda_step; "Implémenter KDA" reference step): decay, erase along k, write,
 * then read the updated state.  q, k, z [B,H,Dk]; v [B,H,Dv]; beta_raw [B,H];
 * S [B,H,Dk,Dv] fp32 in/out; o [B,H,Dv] dtype dt. */
kda_status kda_step(const void* q, const void* k, const void* v, const void* z,
                    const void* beta_raw, const float* A_log, float* S, void* o,
                    int B, int H, int Dk, int Dv, float g_min, unsigned flags,
                    kda_dtype dt, hipStream_t stream);

/* Grouped value heads and the per-dimension gate bias ("KDAAttention 层"
 * 完整数据流 and its parameter table: q, k [B,T,H,K]; v [B,T,HV,V]; g
 * [B,T,HV,K]; beta [B,T,HV]; A_log [HV]; dt_bias [HV,K]).  HV is a positive
 * multiple of H; value head hv reads q/k head hv / (HV / H).  Every other
 * argument is as in kda_chunk_fwd with H replaced by HV (z, beta_raw, A_log,
 * S0, o, S_out, M_out, P_out and the workspace, sized by
 * kda_chunk_fwd_workspace(B, T, HV, ...)).  dt_bias: [HV, Dk] fp32 device,
 * 16-byte aligned, added to z before the bounded gate, or NULL; it needs
 * KDA_GATE_IN_KERNEL (KDA_ERR_DTYPE otherwise).  KDA_ERR_SHAPE when HV is
 * not a positive multiple of H.  H == HV with dt_bias NULL is kda_chunk_fwd. */
kda_status kda_chunk_fwd_grouped(const void* q, const void* k, const void* v, const void* z,
                                 const void* beta_raw, const float* A_log, const float* dt_bias,
                                 const float* S0, void* o, float* S_out, float* M_out, void* P_out,
                                 int B, int T, int H, int HV, int Dk, int Dv, int chunk,
                                 float g_min, unsigned flags, kda_dtype dt,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The decode step of kda_chunk_fwd_grouped: q, k [B,H,Dk]; v [B,HV,Dv]; z
 * [B,HV,Dk]; beta_raw [B,HV]; A_log [HV]; dt_bias [HV,Dk] or NULL; S
 * [B,HV,Dk,Dv] fp32 updated in place; o [B,HV,Dv]. */
kda_status kda_step_grouped(const void* q, const void* k, const void* v, const void* z,
                            const void* beta_raw, const float* A_log, const float* dt_bias,
                            float* S, void* o, int B, int H, int HV, int Dk, int Dv,
                            float g_min, unsigned flags, kda_dtype dt, hipStream_t stream);

/* Segment prefix scan ("KDA 模块交互式演示" §1.6 KCP; "Implémenter KDA" Test 3
 * and 'La loi de composition associative'): for s = 0..n_seg-1,
 *   S_prefix[s] = M[s] S_prev + S_tilde[s],  S_prev = (s ? S_prefix[s-1] : S_in).
 *   M [n_seg,B,H,Dk,Dk], S_tilde and S_prefix [n_seg,B,H,Dk,Dv], all fp32;
 *   S_in nullable [B,H,Dk,Dv] (NULL = zero).  S_prefix must not overlap the
 *   inputs (KDA_ERR_SHAPE). */
kda_status kda_segment_compose(int n_seg, const float* M, const float* S_tilde,
                               const float* S_in, float* S_prefix,
                               int B, int H, int Dk, int Dv, hipStream_t stream);

/* Output correction of segments run from a zero state (the affine split of
 * "Implémenter KDA" Test 2 applied to outputs): for every segment s and token t,
 *   o[s,b,t,h,:] += P[s,b,t,h,:] S_prev[s,b,h]   with
 *   S_prev[s] = (s ? S_prefix[s-1] : S_in)   (S_in NULL: segment 0 untouched).
 * P and o are segment-major [n_seg,B,T_seg,H,Dk] / [n_seg,B,T_seg,H,Dv] in dt
 * (a B = 1 sequence cut into equal segments already has this layout);
 * S_prefix [n_seg,B,H,Dk,Dv] fp32 as written by kda_segment_compose. */
kda_status kda_segment_fixup(int n_seg, const void* P, const float* S_in,
                             const float* S_prefix, void* o, int B, int T_seg,
                             int H, int Dk, int Dv, kda_dtype dt, hipStream_t stream);

/* The layer's input side for one of q, k, v ("KDA 模块交互式演示" §1.1
 * ShortConv and §1.7 完整层; "Implémenter KDA" 'La paramétrisation'): a causal
 * depthwise convolution of kernel 4 over the token axis, then SiLU when silu
 * is non-zero:
 *   y[b,t,c] = act(bias[c] + sum_{j=0..3} w[c,j] * x[b, t-3+j, c]).
 * Tap 3 multiplies the current token, so w[c] = (0,0,0,1) with no bias is the
 * identity the pages initialise to.
 *   x, y       [B,T,C] device, dtype dt, token-major (C = heads * head dim,
 *              the q/k/v layout above), C a multiple of 8; y must not
 *              overlap x.
 *   w          [C,4] fp32 device; bias [C] fp32 device or NULL (zero).
 *   state_in   [B,3,C] dtype dt device, the three inputs before t = 0, oldest
 *              first (a previous call's state_out), or NULL (zeros: the
 *              sequence starts here).
 *   state_out  [B,3,C] dtype dt device or NULL: receives the last three
 *              inputs of (state_in, x), the window the next call or the next
 *              decode token continues from.  It must not overlap x or y, and
 *              may be state_in itself (updated in place) only when T <= 32;
 *              otherwise it must not overlap state_in.
 * T = 0 copies state_in (or zeros) to state_out.  Errors: KDA_ERR_DTYPE,
 * KDA_ERR_SHAPE (negative size, C % 8, a forbidden overlap), KDA_ERR_NULL /
 * KDA_ERR_ALIGN (x, y, w, states: present and 16-byte aligned as required),
 * KDA_ERR_HIP.  Nothing is enqueued when an argument is rejected. */
kda_status kda_short_conv(const void* x, const float* w, const float* bias,
                          const void* state_in, void* state_out, void* y,
                          int B, int T, int C, int silu, kda_dtype dt, hipStream_t stream);

/* The layer's output side before its projection ("KDA 模块交互式演示" §1.7
 * 完整层; "Implémenter KDA" 'La porte de sortie de rang plein', kda_output):
 * per (b,t,h), over the head's Dv channels,
 *   y = sigmoid(gate) * o / sqrt(mean(o^2) + 1e-6) * weight[c].
 *   o, gate, y  [B,T,H,Dv] device, dtype dt; y may be o or gate itself (in
 *               place) but must not otherwise overlap them.
 *   weight      [Dv] fp32 device, shared by the heads, or NULL (ones).
 * Dv in {16,32,64,128}.  Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE (sizes, a
 * forbidden overlap), KDA_ERR_NULL / KDA_ERR_ALIGN (o, gate, y present and
 * 16-byte aligned), KDA_ERR_HIP.  Nothing is enqueued when an argument is
 * rejected. */
kda_status kda_output_gate(const void* o, const void* gate, const float* weight, void* y,
                           int B, int T, int H, int Dv, kda_dtype dt, hipStream_t stream);

/* Backward of kda_chunk_fwd (training).  The pages give the forward only; this
 * is its derivative, for a loss L with dL/do = dout and dL/dS_T = dS_T:
 *   dq, dk, dz [B,T,H,Dk] and dv [B,T,H,Dv], dbeta_raw [B,T,H]: device, dtype
 *              dt, the gradients with respect to the raw inputs through the
 *              switched activations (with a switch off, with respect to the
 *              activated quantity the caller passed in that slot);
 *   dA_log     [H] fp32 device: written (summed over batch and tokens; zero
 *              with the gate switch off);
 *   dS0        [B,H,Dk,Dv] fp32 device or NULL: the gradient with respect to
 *              the initial state.
 * Inputs as for kda_chunk_fwd (HV = H, no gate bias; every switch bit,
 * KDA_GATE_SOFTPLUS included); dout [B,T,H,Dv] dtype dt; dS_T [B,H,Dk,Dv]
 * fp32 or NULL (zero).  The arithmetic is fp32 in 32-token chunks, every decay
 * factor in one exponent (exact for any log-decay).  The workspace
 * (kda_chunk_bwd_workspace bytes, 256-byte aligned) holds the per-chunk
 * operators, the state at each chunk start and the state adjoint at each
 * chunk end.  Outputs may overlap neither an input, another output nor the
 * workspace (KDA_ERR_SHAPE).  Errors otherwise as kda_chunk_fwd. */
size_t kda_chunk_bwd_workspace(int B, int T, int H, int Dk, int Dv);
kda_status kda_chunk_bwd(const void* q, const void* k, const void* v, const void* z,
                         const void* beta_raw, const float* A_log, const float* S0,
                         const void* dout, const float* dS_T,
                         void* dq, void* dk, void* dv, void* dz, void* dbeta_raw,
                         float* dA_log, float* dS0,
                         int B, int T, int H, int Dk, int Dv, float g_min, unsigned flags,
                         kda_dtype dt, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/* Backward of kda_chunk_fwd_grouped: q, k [B,T,H,Dk] read by HV = G H value
 * heads (value head hv reads q/k head hv / G), v, z, beta_raw, A_log, S0 and
 * dout per value head, dt_bias [HV,Dk] fp32 or NULL (added to the gate logit;
 * needs KDA_GATE_IN_KERNEL).  dq, dk [B,T,H,Dk] are the sums over the value
 * heads that read each q/k head; ddt_bias [HV,Dk] fp32 (required with a bias,
 * ignored without) is the logit gradient summed over batch and tokens; the
 * other outputs as kda_chunk_bwd, per value head.  Workspace:
 * kda_chunk_bwd_grouped_workspace(B, T, H, HV, Dk, Dv, dt_bias != NULL)
 * bytes (0 for invalid sizes).  Errors as kda_chunk_fwd_grouped. */
size_t kda_chunk_bwd_grouped_workspace(int B, int T, int H, int HV, int Dk, int Dv, int with_bias);
kda_status kda_chunk_bwd_grouped(const void* q, const void* k, const void* v, const void* z,
                                 const void* beta_raw, const float* A_log, const float* dt_bias,
                                 const float* S0, const void* dout, const float* dS_T,
                                 void* dq, void* dk, void* dv, void* dz, void* dbeta_raw,
                                 float* dA_log, float* ddt_bias, float* dS0,
                                 int B, int T, int H, int HV, int Dk, int Dv, float g_min, unsigned flags,
                                 kda_dtype dt, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* ------------------------------------------------------------------------
 * Softmax attention: the other token mixer of a KDA stack ("KDA 模块交互式演示"
 * §1.8: every fourth layer attends over all keys), with the position encoding
 * in front of it and the 8-bit cache it decodes from.  Layouts as above:
 * q [B,Tq,H,D]; k, v [B,Tk,HK,D]; query head h reads key/value head h / G with
 * G = H / HK (H a positive multiple of HK); D in {16, 32, 64, 128}.
 *
 * Row strides: ld* is the distance between consecutive tokens of a tensor in
 * elements (0 selects heads * D, a contiguous tensor; otherwise at least that
 * and a multiple of 16 bytes; at most 2^23 elements for k and v of kda_attn_fwd
 * and for q, k and v of kda_attn_bwd); sequences are T * ld apart and heads D
 * apart, so q, k and v may be the parts of one packed projection [B,T,H+2HK,D],
 * or, with T = 1, of the last token of a longer one.
 *
 * Lengths: device arrays of B ints, read when the kernels run; values outside
 * the tensor's range are clamped to it (cache_len: only negative ones, to 0).
 * Nothing at or past a sequence's length is read, whatever it holds.
 *
 * Sizes (KDA_ERR_SHAPE past them): Tk, max_pages * page and the rows G * Tq of
 * a key/value head up to 2^29; B * HK * (G * Tq / 32 + 1) and B * HK *
 * (Tk / 32 + 1) below 2^24; in the backward the 16-byte pieces of o, 200 tokens
 * a sequence on top, below 2^32; B * T * D of a rotation below 2^32; pages that
 * an append may touch, B * HK * (T / page + 2), below 2^24. */

/* Inverse frequencies of the rotary position encoding for `rot` channels
 * (positive, even, at most 128):
 * inv_freq[i] = base^(-2i/rot), i < rot / 2, host memory, in radians per
 * position, scaled for contexts `factor` times the `trained` length:
 *   KDA_ROTARY_NONE    unscaled (factor, trained and beta_* unused);
 *   KDA_ROTARY_LINEAR  every frequency divided by factor;
 *   KDA_ROTARY_NTK     base * factor^(rot / (rot - 2)) in place of base (rot = 2: base);
 *   KDA_ROTARY_YARN    by parts: frequencies that turn more than beta_fast
 *                      times within the trained length are kept, those below
 *                      beta_slow turns are divided by factor, those between
 *                      are blended linearly in i; *scale = 0.1 ln(factor) + 1.
 * *scale (nullable) receives the scale of the rotated values, 1 otherwise.
 * KDA_ERR_NULL without inv_freq; KDA_ERR_SHAPE for rot, kind or trained < 1
 * (by parts); KDA_ERR_SCALE unless base > 1, factor >= 1, beta_fast >
 * beta_slow > 0, all finite.  Host only; no HIP call. */
enum { KDA_ROTARY_NONE = 0, KDA_ROTARY_LINEAR = 1, KDA_ROTARY_NTK = 2, KDA_ROTARY_YARN = 3 };
kda_status kda_rotary_freqs(double* inv_freq, float* scale, int rot, double base, int kind, double factor,
                            int trained, double beta_fast, double beta_slow);

/* Rotary position encoding of q and k in one pass: with a = scale cos(p w_i),
 * b = scale sin(p w_i) for token position p,
 *   (x_j, x_j') -> (a x_j - b x_j', b x_j + a x_j')  over the pairs of the
 * first `rot` channels of each head; channels rot .. D-1 are copied.
 *   mode       KDA_ROTARY_INTERLEAVED: pair i is channels (2i, 2i+1);
 *              otherwise (i, i + rot/2).  KDA_ROTARY_INVERSE: b -> -b, the
 *              transposed map, so the same call is the gradient.
 *   q, q_out   [B,T,H,D] with strides ldq, ldqo; k, k_out [B,T,HK,D] with ldk,
 *              ldko, or NULL (HK then ignored).  q_out may be q itself with the
 *              same stride (in place), k_out likewise; outputs may not
 *              otherwise overlap an input or each other (KDA_ERR_SHAPE).
 *   positions  [B,T] int device, or NULL: 0 .. T-1 in every sequence.
 *   inv_freq   [rot/2] double device (kda_rotary_freqs).  Angles are formed in
 *              64 bits and reduced to a turn, so far positions keep their
 *              precision.
 *   rot        even, 2 .. D.
 * Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE, KDA_ERR_SCALE (scale not finite),
 * KDA_ERR_NULL, KDA_ERR_ALIGN, KDA_ERR_HIP. */
enum { KDA_ROTARY_INTERLEAVED = 1u, KDA_ROTARY_INVERSE = 2u };
kda_status kda_rotary(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                      const double* inv_freq, int B, int T, int H, int HK, int D, int rot,
                      int ldq, int ldk, int ldqo, int ldko, float scale, unsigned mode, kda_dtype dt,
                      hipStream_t stream);

/* Softmax attention forward.  Query i of sequence b stands at key position
 * p = i + kv_len[b] - q_len[b] (the last query at the last key) and sees the
 * keys j < kv_len[b] with j <= p if `causal`, and j > p - window if window > 0:
 *   o_i = sum_j P_ij v_j,  P_ij = exp(scale q_i.k_j - lse_i),
 *   lse_i = ln sum_j exp(scale q_i.k_j)   over the visible j.
 * A query that sees no key, and queries i >= q_len[b], get o = 0 and
 * lse = -infinity.
 *   q_len, kv_len  [B] int device or NULL (Tq, Tk).
 *   o    [B,Tq,H,D] contiguous, dtype dt;  lse [B,H,Tq] fp32 or NULL.
 *   scale  at least 2^-64, and finite times log2 e (KDA_ERR_SCALE otherwise).
 *   workspace  kda_attn_fwd_workspace bytes, 256-byte aligned: partial results
 *        of calls with few query rows, whose key axis is split over several
 *        workgroups (0 bytes, and NULL accepted, for the others).
 * Statistics and sums are fp32; bf16 probabilities are rounded to bf16 before
 * their product with v.  A masked key inside the lengths has no effect as long
 * as its k and v are finite; a NaN or infinity in v at such a key may reach
 * rows of the same tile.  o may overlap no input, lse or the workspace.
 * Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE, KDA_ERR_SCALE, KDA_ERR_NULL,
 * KDA_ERR_ALIGN, KDA_ERR_WORKSPACE, KDA_ERR_HIP. */
size_t kda_attn_fwd_workspace(int B, int Tq, int Tk, int H, int HK, int D, kda_dtype dt);
kda_status kda_attn_fwd(const void* q, const void* k, const void* v, const int* q_len, const int* kv_len,
                        void* o, float* lse, int B, int Tq, int Tk, int H, int HK, int D,
                        int ldq, int ldk, int ldv, float scale, int causal, int window, kda_dtype dt,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Backward of kda_attn_fwd for a loss with dL/do = dout, from the forward's
 * inputs and its o and lse (the probabilities are recomputed):
 *   dv_j = sum_i P_ij dout_i,   dS_ij = P_ij (dout_i.v_j - dout_i.o_i),
 *   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,
 * dk and dv summed over the G query heads of each key/value head.  Sums are
 * fp32; in bf16 P and dS are rounded to bf16 before their products.  No
 * atomics: results do not vary from run to run.  With causal = 0 and window = 0
 * k and v may be a part of the keys that o and lse were formed with: dk and dv
 * are then that part's, and dq its share of the sum.  With a causal mask or a
 * window (of any length) they are all of them; dout_i.o_i is then formed from
 * P and v instead of o for rows that see at most 32 keys (axes of 32 keys,
 * windows of 16; in bf16 the first 32 queries under a causal mask), where the
 * rounding of o would show in the gradients.
 *   o, dout, dq [B,Tq,H,D], dk, dv [B,Tk,HK,D]: contiguous, dtype dt.  Rows
 *   past the lengths, and rows that see or are seen by nothing, get 0; o, lse
 *   and dout are not read past q_len.  What is not finite inside the lengths, or
 *   has a product past fp32's range there, may reach the gradients of rows and
 *   keys of the same tile too.
 *   workspace  kda_attn_bwd_workspace bytes, 256-byte aligned.
 * Outputs may overlap neither an input, another output nor the workspace
 * (KDA_ERR_SHAPE).  Errors otherwise as kda_attn_fwd. */
size_t kda_attn_bwd_workspace(int B, int Tq, int Tk, int H, int HK, int D, kda_dtype dt);
kda_status kda_attn_bwd(const void* q, const void* k, const void* v, const int* q_len, const int* kv_len,
                        const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                        int B, int Tq, int Tk, int H, int HK, int D, int ldq, int ldk, int ldv,
                        float scale, int causal, int window, kda_dtype dt,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The 8-bit key/value cache.  Pages of `page` tokens (16, 32, 64 or 128), one
 * scale for each page and key/value head; a stored code c (e4m3: 1 sign, 4
 * exponent, 3 mantissa bits, largest 448) stands for c * scale:
 *   k_cache [n_pages,HK,page,D] bytes, v_cache [n_pages,HK,D,page] bytes (a
 *   page of v is stored transposed, as the attention's products read it),
 *   k_scale, v_scale [n_pages,HK] fp32;
 *   block_table [B,max_pages] int: page number of each `page` tokens of a
 *   sequence; an entry outside 0 .. n_pages-1 names no page.
 *
 * kda_cache_append writes new_len[b] tokens (NULL: T) of k, v [B,T,HK,D] (dtype
 * dt, strides ldk, ldv) behind the cache_len[b] tokens sequence b already has.
 * The scale of a page is the smallest power of two with max|x| <= 448 scale
 * over the finite values written (at least 2^-100), never below the scale of
 * tokens already in the page; where it grows, those tokens' codes are moved to
 * it.  Values are divided by the scale and rounded to nearest even; infinities
 * become +-448, NaN stays NaN.  Tokens whose page is missing (no entry, or past
 * max_pages) are dropped; pages without new tokens, and bytes past the last
 * token, are left as they were.  Among the pages that one call writes none may
 * be named twice (shared pages are for reading).
 * Sizes as above, n_pages * HK <= 2^30; no buffer may overlap another.
 * Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE, KDA_ERR_NULL, KDA_ERR_ALIGN, KDA_ERR_HIP. */
kda_status kda_cache_append(const void* k, const void* v, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, const int* block_table,
                            const int* cache_len, const int* new_len, int n_pages, int max_pages,
                            int B, int T, int HK, int D, int page, int ldk, int ldv, kda_dtype dt,
                            hipStream_t stream);

/* Attention of the new_len[b] (NULL: Tq) newest tokens over that cache, after
 * their append (the decode step for Tq = 1; drafted tokens or a prompt's chunk
 * for more): query i stands at position p = cache_len[b] + i and sees the cached
 * tokens j <= p, and j > p - window if window > 0, also where cache_len[b] lies
 * past the max_pages * page tokens of the table.  Tokens whose page is missing
 * are not seen.  Queries past new_len, and those that see nothing, get o = 0.
 * A NaN code of v at a cached token that a query does not see may reach it from
 * the same 64 tokens.
 *   q [B,Tq,H,D] (stride ldq), o [B,Tq,H,D] contiguous, dtype dt.
 *   workspace  kda_attn_step_workspace(B, Tq, H, HK, D, max_pages * page)
 *        bytes, 256-byte aligned: partial results where the cache is split
 *        over several workgroups.
 * fp32 queries and probabilities enter the products as three bf16 parts (24
 * bits), bf16 ones as they are (probabilities rounded to bf16).
 * Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE, KDA_ERR_SCALE, KDA_ERR_NULL,
 * KDA_ERR_ALIGN, KDA_ERR_WORKSPACE, KDA_ERR_HIP. */
size_t kda_attn_step_workspace(int B, int Tq, int H, int HK, int D, int max_len);
kda_status kda_attn_step(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, const int* block_table, const int* cache_len,
                         const int* new_len, void* o, int n_pages, int max_pages, int B, int Tq,
                         int H, int HK, int D, int page, int ldq, float scale, int window, kda_dtype dt,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * One prompt continued several times (beams, parallel samples): sequences share the
 * pages of what they have in common, attend over it once, and are reordered as a
 * selection says.
 *
 * Pages.  refs [n_pages] int: how many table entries name a page, summed over every
 * table (and other holder) of the cache; 0 is a free page.  A table entry outside
 * 0 .. n_pages-1 names none; tables [B,max_pages], lengths and pages as for
 * kda_cache_append.  The calls below keep refs in step with the tables that they
 * are given.  One set of tables serves the caches of all layers: bookkeeping is one
 * call, and its list of copies (src, dst: page numbers, -1 in entries without one) is
 * given to kda_cache_copy for each layer.  Which page is taken, and who keeps a shared
 * one, follows the order of (sequence, page), so results do not vary from run to run.
 * Sizes: B * max_pages below 2^30, n_pages up to 2^30; page in {16, 32, 64, 128}. */

/* Sequences that follow their parents: R requests of K_in sequences become R of K_out.
 * Row c of request r gets the pages that hold tokens of row parent[r][c] (an index
 * within the request; one outside 0 .. K_in-1 makes an empty row), -1 behind them,
 * and its length.  The references of all of its entries are counted; those of the
 * old rows are dropped unless `keep` (the prompt stays beside its samples).  Tokens
 * are not copied: kda_cache_reserve gives every sequence a page of its own to write to.
 *   table [R*K_in,max_pages], cache_len [R*K_in], parent [R,K_out] int;
 *   table_out [R*K_out,max_pages], len_out [R*K_out] int; refs [n_pages], updated.
 * K_in, K_out up to 1024.  Outputs may overlap no other buffer (KDA_ERR_SHAPE).
 * Errors: KDA_ERR_SHAPE, KDA_ERR_NULL, KDA_ERR_ALIGN, KDA_ERR_HIP. */
kda_status kda_cache_fork(const int* table, const int* cache_len, const int* parent, int* table_out,
                          int* len_out, int* refs, int R, int K_in, int K_out, int max_pages,
                          int n_pages, int page, int keep, hipStream_t stream);

/* Room for new_len[b] (NULL: T) tokens behind the cache_len[b] of each sequence,
 * before their kda_cache_append.  Of the pages that these tokens touch,
 *   - one that is missing becomes the lowest free page (a page whose older tokens are
 *     missing stays missing: appends drop its tokens);
 *   - one that others hold too (refs > 1) is left to them for the lowest free page, into
 *     which it has to be copied if it holds older tokens; where nobody outside the
 *     call's sequences holds it, the last of them keeps it.
 * A page that has a number and one reference is left as it is, so reserving again, or for
 * more tokens, is safe.  Entries for which no page is free become -1 (a shared page is
 * given up: this sequence's tokens in it are then missing).
 *   table [B,max_pages], refs [n_pages]: updated;  cache_len, new_len [B] int;
 *   src, dst [B] int: the page to copy for each sequence and where to;
 *   info [2] int: entries that got no page, and free pages left.
 * B times the pages that T tokens may touch, ceil((T - 1) / page) + 1, is below 2^30.
 * Errors as kda_cache_fork. */
kda_status kda_cache_reserve(int* table, int* refs, const int* cache_len, const int* new_len,
                             int* src, int* dst, int* info, int B, int T, int max_pages, int n_pages,
                             int page, hipStream_t stream);

/* Gives back the pages of each sequence that hold none of its tokens
 * keep_from[b] .. keep_to[b]-1 (NULL: 0): all of them without either (the sequence
 * ends), those behind accepted tokens (drafted ones are dropped), those that a
 * window has passed.  Their entries become -1; cache_len is the caller's.
 *   table [B,max_pages], refs [n_pages]: updated;  keep_from, keep_to [B] int.
 * Errors as kda_cache_fork. */
kda_status kda_cache_free(int* table, int* refs, const int* keep_from, const int* keep_to,
                          int B, int max_pages, int n_pages, int page, hipStream_t stream);

/* Moves the pages in use to the front of the cache, U of them: the i-th used page from
 * U on goes to the i-th free page below U (both in ascending order), the others stay.
 *   table [B,max_pages], refs [n_pages] -> table_out, refs_out (which may be table and
 *   refs themselves);  remap [n_pages] int: a page's new number, -1 for a free one, for
 *   tables that other holders have;  src, dst [n_pages / 2] int: the copies, -1 behind
 *   the last;  info [2] int: their number (the `count` of kda_cache_copy), and U.
 * Entries that name a free page become -1.  Errors as kda_cache_fork. */
kda_status kda_cache_compact(const int* table, const int* refs, int* table_out, int* refs_out,
                             int* remap, int* src, int* dst, int* info, int B, int max_pages,
                             int n_pages, hipStream_t stream);

/* Copies pages, codes and scales: page src[i] of one cache becomes page dst[i] of another
 * (or of the same: all four pointers equal) for i < n, and i < count[0] if count is not
 * NULL; entries that name no page are passed over.  No page may be written twice by a
 * call, nor read by the call that writes it.
 *   caches as for kda_cache_append, of n_src and n_dst pages;  src, dst [n], count [1] int.
 * HK * page * D below 2^31.  Different caches may not overlap (KDA_ERR_SHAPE).  Errors as
 * kda_cache_fork. */
kda_status kda_cache_copy(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                          void* k_to, void* v_to, float* k_scale_to, float* v_scale_to,
                          const int* src, const int* dst, const int* count, int n, int n_src, int n_dst,
                          int HK, int D, int page, hipStream_t stream);

/* kda_attn_step for groups of sequences that have a common prefix, which is read once a
 * group instead of once a sequence: group g is the sequences group_first[g] ..
 * group_first[g+1]-1, whose first prefix_len[g] tokens are the same.  Their whole pages
 * are read through the row of the group's first sequence; the page in which a prefix
 * ends, of which every sequence has a copy (whose codes move as its scale grows), and
 * what follows through each sequence's own.  The result is that of kda_attn_step up to
 * the order of its sums and, in bf16, the rounding of probabilities: where groups have
 * more than 32 rows they may be relative to a maximum that lies a factor 2 below the row's,
 * and are then divided by the sum of the rounded ones.  Everything else as there; a
 * sequence of no group has no prefix, one whose length is below the prefix sees no
 * further than its length.
 * The group's first row is read for all of it: its pages have to stay as long as any
 * sequence of the group sees them.  Where kda_cache_free gives them back (that sequence
 * has ended, or its window has passed them) they are missing for the whole group, without an
 * error: let the group begin with another sequence then, or leave the row until all have ended.
 * How the work is divided (row tiles, parts) follows max_pages * page and B / n_groups, since
 * lengths are on the device: 64 samples on 4096 tokens take 25 us with a table of 4608 tokens, 33
 * with one of 32768.
 *   group_first [n_groups+1] int, not descending (values outside 0 .. B are clamped);
 *   prefix_len [n_groups] int (clamped to the table).
 *   workspace  kda_attn_shared_workspace(B, Tq, H, HK, D, n_groups, max_pages * page)
 *        bytes, 256-byte aligned: partial results of prefixes and of own keys.
 * Sizes as there, and n_groups up to 2^16, B * Tq * (H / HK) up to 2^29, B * Tq * H * D below 2^34;
 * below 2^23 workgroups (about 16 rows each, for groups and sequences, times the parts that fill the card).
 * Errors as kda_attn_step. */
size_t kda_attn_shared_workspace(int B, int Tq, int H, int HK, int D, int n_groups, int max_len);
kda_status kda_attn_shared(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* block_table, const int* cache_len,
                           const int* new_len, const int* group_first, const int* prefix_len, void* o,
                           int n_groups, int n_pages, int max_pages, int B, int Tq, int H, int HK, int D,
                           int page, int ldq, float scale, int window, kda_dtype dt,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* States that follow their parents: row c of request r of `out` becomes row
 * parent[r][c] (an index within the request) of request r of `state`, zeros if that is
 * outside 0 .. K_in-1.  For the states [B,H,Dk,Dv] of kda_step and the windows
 * [B,3,C] of kda_short_conv; any row of bytes.
 *   state [R*K_in] rows, out [R*K_out] rows of row_bytes bytes (a multiple of 16), parent
 *   [R,K_out] int.  out may be state itself where K_in = K_out <= 64: rows whose parent
 *   they are themselves are then not touched.  No other overlap (KDA_ERR_SHAPE).
 * Sizes: R * K up to 2^24, and below 2^24 pieces of 2 KB (in place, all rows of a request
 * together) or 16 KB of a row.
 * Errors: KDA_ERR_SHAPE, KDA_ERR_NULL, KDA_ERR_ALIGN (row_bytes too), KDA_ERR_HIP. */
kda_status kda_state_reorder(const void* state, void* out, const int* parent, int R, int K_in, int K_out,
                             size_t row_bytes, hipStream_t stream);

/* Beam search's selection: over the K beams of a request and the V tokens,
 *   s(b,w) = scores[b] + x_bw - ln sum_w' exp(x_bw'),
 * the M largest, largest first, equal ones in the order of (b, w).
 *   logits   [R,K,V] dtype dt, rows ld elements apart (0: V); any ld >= V.
 *            Within a beam the order is that of the logits.
 *   scores   [R,K] fp32, or NULL (zeros).  A beam whose score is not finite has no
 *            continuation (the unused beams of a first step: -infinity).
 *   done     [R,K] bytes or NULL: a finished beam (not 0) has one continuation, `end`
 *            (a token, 0 .. V-1), with its score unchanged, whatever its logits are.
 *   scores_out [R,M] fp32, parent, token [R,M] int.  Where fewer than M continuations
 *            have a score above -infinity the rest is -infinity, -1, -1.
 * Logits of -infinity are no continuations, nor is one whose score fp32 rounds to
 * -infinity; a beam with a NaN or +infinity has none.  Continuations are compared in 64
 * bits and their scores rounded once.  lse is good to about 1e-7 (exponentials are fp32,
 * sums of more than 32 of them 64 bits); at worst, where many logits of one value make up a
 * row's sum beside larger ones, it is off by 2e-6 (V up to 2^20; 3e-6 up to 2^30).
 * K, M up to 64, V up to 2^30, R * K below 2^18.
 *   workspace  kda_beam_select_workspace bytes, 256-byte aligned.
 * Outputs may overlap no other buffer.  Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE,
 * KDA_ERR_NULL, KDA_ERR_ALIGN, KDA_ERR_WORKSPACE, KDA_ERR_HIP. */
size_t kda_beam_select_workspace(int R, int K, int V, int M, kda_dtype dt);
kda_status kda_beam_select(const void* logits, const float* scores, const unsigned char* done,
                           float* scores_out, int* parent, int* token, int R, int K, int V, int M,
                           int ld, int end, kda_dtype dt, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* Static description of a status code (never NULL). */
const char* kda_status_string(kda_status s);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
