/*
 * flashsample.h -- C ABI of libflashsample: exact categorical sampling fused
 * into the LM-head matmul, for AMD Instinct MI355X (gfx950).
 *
 * The operation ("FlashSampling: Fast and Memory-Efficient Exact Sampling";
 * wiki summary page, sections "Key claims" and "Method"; arXiv abstract):
 * for each batch row b the library draws one token id from
 * softmax(z_b / T_b), z_b = W h_b, by the Gumbel-Max trick -- the argmax over
 * v of  s[b][v] = z[b][v] / T_b + g[b][v]  with g standard Gumbel noise.  The
 * logits are formed tile by tile on chip, scaled, perturbed and reduced to
 * one (max, argmax) pair per row and per vocabulary tile; a small reduction
 * over tiles returns the id.  The B x V logits never reach device memory.
 *
 * Noise field.  The pages leave the generator open; here it is
 * Philox-4x32-10 (Salmon et al., SC'11).  For batch row b and GLOBAL
 * vocabulary id gv = vocab_offset + v:
 *   x = word (gv mod 4) of Philox4x32_10(counter = {gv / 4, b, step_lo,
 *       step_hi}, key = {seed_lo, seed_hi})
 *   u = (x + 1/2) * 2^-32                   (all 32 bits; 0 < u < 1)
 *   g = -log(-log u)
 * Equal logits therefore tie for the largest score only when two ids draw
 * the same word (about V * 2^-33 of draws).
 * Keying on the global id makes the field independent of tiling and of
 * vocabulary sharding, so per-shard results merge to the unsharded result
 * (wiki summary, "Method", tensor-parallel paragraph).
 *
 * Scores.  s = z * fp32(1/T_b) + g, with z accumulated in fp32 from bf16
 * products.  A row whose temperature is not a positive number (0, -0,
 * negative, NaN) is greedy: s = z (no scaling, no noise).  Ties go to the
 * smaller global id.
 *
 * Conventions for every entry point:
 *   - h is bf16 [B][D] row-major, W is bf16 [V][D] row-major (the layout of
 *     an nn.Linear weight); both device pointers, 16-byte aligned; D % 8 == 0.
 *   - temperature, out_ids, out_maxval, partials: device pointers, 4-byte
 *     aligned.  workspace: device pointer, 256-byte aligned.
 *   - stream is a hipStream_t (NULL = the default stream).  Calls are
 *     asynchronous and ordered on that stream; the caller keeps every buffer
 *     alive until the stream has reached the work.
 *   - Ownership: the caller owns all memory.  The library allocates nothing
 *     on the sampling path (the one device array it holds, for
 *     fs_sample_packed_noalloc, is static) and keeps no pointer after
 *     returning; between calls it holds only a forced-configuration switch
 *     (fs_force_config), per-device caches of device facts and launch sizes,
 *     and the profiling recorder (fs_profile_enable).
 *   - Errors: the return code is the only channel.  Arguments are checked on
 *     the host before any HIP call; a rejected call launches nothing and
 *     writes nothing.  FS_ERR_HIP carries the runtime's message in
 *     fs_last_error() (thread-local).  An error that an earlier failed HIP
 *     call left pending in the calling thread is discarded before a call's
 *     first launch, so it is not reported again.  Device-resident values are
 *     not inspected: NaN or infinite entries in h or W give undefined ids.
 *   - B == 0 is a no-op that returns FS_OK (pointers may then be NULL).
 *     The samplers take at most 1048560 (16 * 65535) batch rows per call and
 *     the unfused baseline at most 65535 (the launch grids' row limit);
 *     larger B is FS_ERR_UNSUPPORTED.
 *   - Reentrant: concurrent calls are safe if they use distinct workspaces.
 *   - Failure testing: with FS_FAULT_INJECT=launch in the environment, every
 *     entry point that would launch device work returns FS_ERR_HIP once its
 *     arguments have passed the checks, and launches nothing;
 *     fs_last_error() then names the injection.
 */
#ifndef FLASHSAMPLE_H
#define FLASHSAMPLE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FS_API __attribute__((visibility("default")))

typedef enum {
  FS_OK = 0,
  FS_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size or range */
  FS_ERR_UNSUPPORTED = 2, /* valid request this build cannot run */
  FS_ERR_WORKSPACE = 3,   /* workspace_bytes below the required size */
  FS_ERR_HIP = 4          /* a HIP runtime call or launch failed */
} fs_status;

/* Bytes of workspace fs_sample / fs_sample_partial need for (B, D, V).
 * Returns 0 when the sizes are invalid (see fs_sample). */
FS_API size_t fs_workspace_bytes(int32_t B, int32_t D, int32_t V);

/* Bytes of workspace fs_sample_unfused needs: the materialised fp32 logits
 * and probabilities (2 * B * V * 4 bytes) plus per-row statistics. */
FS_API size_t fs_unfused_workspace_bytes(int32_t B, int32_t D, int32_t V);

/* Sample one token id per batch row (wiki summary, "Method": per-tile
 * maximisers over vocabulary tiles, then the partition argmax).
 *   h            bf16 [B][D]
 *   W            bf16 [V][D]; row v has global id vocab_offset + v
 *   B, D, V      B >= 0; D >= 8, D % 8 == 0; V >= 1
 *   vocab_offset >= 0 and vocab_offset + V <= 2^31 - 1
 *   temperature  fp32 [B]; !(T > 0) selects greedy for that row
 *   seed, step   64-bit noise key and step counter (fresh per decode step)
 *   out_ids      int32 [B]: sampled GLOBAL id per row
 *   out_maxval   fp32 [B]: the winning perturbed score s
 *   workspace    >= fs_workspace_bytes(B, D, V) bytes; contents on entry
 *                are ignored (scratch for per-tile partials)             */
FS_API fs_status fs_sample(const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                    int32_t vocab_offset, const float* temperature, uint64_t seed,
                    uint64_t step, int32_t* out_ids, float* out_maxval,
                    void* workspace, size_t workspace_bytes, void* stream);

/* Fragment-order weights.  The sampler reads W one MFMA operand fragment at
 * a time (16 vocabulary rows x 32 k, 16 bytes per lane); from row-major W
 * each such read takes 64 bytes from each of 16 rows 8 KB apart, which costs
 * HBM page locality.  fs_pack_weights copies W once (at model load) into the
 * fragment order the kernels consume: the vocabulary rows in groups of 16
 * starting at row -(vocab_offset mod 4), each group stored k-step by k-step
 * as 64 pieces of 16 bytes (element ((g * D/32 + s) * 64 + l) * 8 + j holds
 * W[16 g + (l mod 16) - (vocab_offset mod 4)][32 s + 8 (l / 16) + j], zero
 * outside [0, V)).
 *   W            bf16 [V][D], device, 16-byte aligned; D % 32 == 0
 *   vocab_offset the offset the packed weights will be sampled at (only its
 *                value mod 4 shapes the layout)
 *   W_packed     device, 16-byte aligned, >= fs_packed_weights_bytes(V, D,
 *                vocab_offset) bytes (0 for invalid arguments); caller-owned
 * fs_sample_packed takes fs_sample's arguments with W_packed in place of W
 * (packed for the same V, D and vocab_offset mod 4).  Its kernels read the
 * same operand fragments as fs_sample's: run in one configuration
 * (fs_force_config) the two return the same ids and scores bit for bit; the
 * automatic choices may differ (fs_selected_config_packed), and then so may
 * the scores' last bits, within the parity bound of fs_sample.  It runs the
 * persistent, DMA-staged and LDS-staged kernels; a shape whose configuration
 * has no fragment-order kernel (the K-split and streaming loops chosen for
 * small batches at unusual D) returns FS_ERR_UNSUPPORTED.  D % 32 != 0 is
 * FS_ERR_INVALID_ARG. */
FS_API size_t fs_packed_weights_bytes(int32_t V, int32_t D, int32_t vocab_offset);
FS_API fs_status fs_pack_weights(const void* W, int32_t V, int32_t D, int32_t vocab_offset,
                                 void* W_packed, size_t packed_bytes, void* stream);
FS_API fs_status fs_sample_packed(const void* h, const void* W_packed, int32_t B, int32_t D,
                                  int32_t V, int32_t vocab_offset, const float* temperature,
                                  uint64_t seed, uint64_t step, int32_t* out_ids,
                                  float* out_maxval, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* fs_sample_packed without a workspace argument, for callers that cannot
 * allocate device memory around the call (code being captured into a graph,
 * tight serving loops, harnesses that forbid allocation).  The tile partials
 * go to an 8 MiB array the library holds in each device's memory until the
 * process ends; the call allocates nothing.  Its kernels and results are
 * fs_sample_packed's.  Every call on one device shares that array, so calls
 * that overlap on one device (concurrent streams, or several host threads)
 * race and must be serialised by the caller.  A shape whose partials exceed
 * the array (2 * 4 * B * ceil((V + 3) / rows) bytes, rows the chosen
 * configuration's vocabulary rows per block: 16 for the small-batch
 * kernels, 256 or more for the batch-tiled ones) returns FS_ERR_WORKSPACE
 * and launches nothing; other errors as fs_sample_packed. */
FS_API fs_status fs_sample_packed_noalloc(const void* h, const void* W_packed, int32_t B,
                                          int32_t D, int32_t V, int32_t vocab_offset,
                                          const float* temperature, uint64_t seed, uint64_t step,
                                          int32_t* out_ids, float* out_maxval, void* stream);

/* One vocabulary shard's contribution for the grouped / tensor-parallel flow
 * (wiki summary, "Method": each rank reduces its own shard to a per-row
 * (local max, local argmax) pair, and only those pairs are exchanged).
 * Same inputs and semantics as fs_sample over rows [vocab_offset,
 * vocab_offset + V) of the global vocabulary; writes partial_val[b] and
 * partial_idx[b] (GLOBAL ids), i.e. slot p of a P x B partial buffer when
 * the caller passes base + p * B. */
FS_API fs_status fs_sample_partial(const void* h, const void* W, int32_t B, int32_t D,
                            int32_t V, int32_t vocab_offset, const float* temperature,
                            uint64_t seed, uint64_t step, float* partial_val,
                            int32_t* partial_idx, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Cross-part argmax (wiki summary, "Method": the final cross-rank argmax).
 *   partial_val  fp32 [P][B], partial_idx int32 [P][B] (part-major)
 *   P >= 1, B >= 0
 * Per row: the largest value wins; on equal values the smaller id wins.
 * Bit-exact: the result depends only on the set of pairs, not their order. */
FS_API fs_status fs_merge(const float* partial_val, const int32_t* partial_idx, int32_t P,
                   int32_t B, int32_t* out_ids, float* out_maxval, void* stream);

/* Grouped (hierarchical) sampler, one vocabulary group per call (arXiv
 * abstract page and wiki summary, "Key claims": grouped variants for online
 * and tensor-parallel settings are exact by hierarchical factorisation of
 * the categorical distribution; wiki summary, "Method", last paragraph: the
 * online, chunked setting).  As fs_sample_partial, plus
 *   partial_lse  fp32 [B], device: per row the log-sum-exp of the group's
 *                scaled logits, log sum_v exp(z_v * (1/T)); for greedy rows
 *                (T not > 0) the group's largest logit.
 * partial_val / partial_idx are bit-identical to fs_sample_partial's on the
 * same inputs.  Same workspace (fs_workspace_bytes) and errors. */
FS_API fs_status fs_sample_partial_lse(const void* h, const void* W, int32_t B, int32_t D,
                                int32_t V, int32_t vocab_offset, const float* temperature,
                                uint64_t seed, uint64_t step, float* partial_val,
                                int32_t* partial_idx, float* partial_lse, void* workspace,
                                size_t workspace_bytes, void* stream);

/* The same on fragment-order weights (fs_pack_weights, for this group's rows
 * at this vocab_offset mod 4): W_packed in place of W, D % 32 == 0. */
FS_API fs_status fs_sample_partial_lse_packed(const void* h, const void* W_packed, int32_t B,
                                              int32_t D, int32_t V, int32_t vocab_offset,
                                              const float* temperature, uint64_t seed,
                                              uint64_t step, float* partial_val,
                                              int32_t* partial_idx, float* partial_lse,
                                              void* workspace, size_t workspace_bytes,
                                              void* stream);

/* The grouped sampler's per-group partials for G groups in one launch.  The
 * vocabulary W[0 .. V) is split at the HOST array cuts (0 = cuts[0] <
 * cuts[1] < ... < cuts[G] = V, 1 <= G <= 64); slot g of the outputs (element
 * g * B + b of partial_val / partial_idx / partial_lse, [G][B] part-major as
 * fs_merge_lse reads them) holds what fs_sample_partial_lse would return over
 * W rows [cuts[g], cuts[g+1]) at vocab_offset + cuts[g]: the group's
 * Gumbel-max (value, global id) and its log-sum-exp.  One fused launch covers
 * every group (each group's vocabulary rows are tiled from its own first row,
 * so no tile mixes two groups) and one merge launch fills the slots, instead
 * of G launches each over a slice too short to fill the device.  In one
 * configuration (fs_force_config) the slots' values and ids equal the
 * separate calls bit for bit, and so do the log-sum-exps on the batch-tiled
 * configurations; the persistent ones (small batches) add a group's
 * log-sum-exp partials in another order, equal within rounding.
 *   workspace   >= fs_groups_workspace_bytes(B, D, V, G) bytes (0 for invalid
 *               arguments); contents on entry ignored
 * Errors as fs_sample_partial_lse; a cuts array that does not partition
 * [0, V) or G outside [1, 64] is FS_ERR_INVALID_ARG.  The _packed form reads
 * fragment-order W (fs_pack_weights at the same vocab_offset mod 4) and needs
 * every group start cuts[g] (0 < g < G) to be a multiple of 16. */
FS_API size_t fs_groups_workspace_bytes(int32_t B, int32_t D, int32_t V, int32_t n_groups);
FS_API fs_status fs_sample_groups_lse(const void* h, const void* W, int32_t B, int32_t D,
                                      int32_t V, int32_t vocab_offset, const float* temperature,
                                      uint64_t seed, uint64_t step, const int32_t* cuts,
                                      int32_t n_groups, float* partial_val, int32_t* partial_idx,
                                      float* partial_lse, void* workspace,
                                      size_t workspace_bytes, void* stream);
FS_API fs_status fs_sample_groups_lse_packed(const void* h, const void* W_packed, int32_t B,
                                             int32_t D, int32_t V, int32_t vocab_offset,
                                             const float* temperature, uint64_t seed,
                                             uint64_t step, const int32_t* cuts, int32_t n_groups,
                                             float* partial_val, int32_t* partial_idx,
                                             float* partial_lse, void* workspace,
                                             size_t workspace_bytes, void* stream);

/* Grouped merge: the categorical distribution factorises as
 * P(i) = P(G) P(i | G) with P(G) proportional to exp(LSE_G), and each
 * group's partial already holds a sample of P(i | G).
 *   partial_val, partial_idx, partial_lse  [P][B] (part-major), from
 *                fs_sample_partial_lse, group p in slot p
 *   temperature  fp32 [B], device (greedy rows as in fs_sample)
 *   seed, step   key of the group draws: gamma_p is the Gumbel value of
 *                Philox-4x32-10 word 0 at counter (2^31 | p, row, step low,
 *                step high) under key (seed low, seed high), a counter the
 *                token noise never uses
 * Per row b the group p* = argmax_p (lse_p + gamma_p) (greedy rows:
 * argmax_p lse_p), ties to the smaller p; out_ids[b] / out_maxval[b] are
 * that group's partial, out_lse[b] the row's total log-sum-exp over the
 * groups (greedy rows: the largest lse_p).  All pointers device, 4-byte
 * aligned; P >= 1, B >= 0. */
FS_API fs_status fs_merge_lse(const float* partial_val, const int32_t* partial_idx,
                       const float* partial_lse, int32_t P, int32_t B,
                       const float* temperature, uint64_t seed, uint64_t step,
                       int32_t* out_ids, float* out_maxval, float* out_lse, void* stream);

/* Online (chunked) sampler with early finalisation (wiki summary, "Method",
 * last paragraph: in the online setting the sampler streams over pieces of
 * the vocabulary and may finalise before it has seen them all).  The
 * vocabulary is processed in the chunks W[cuts[c] .. cuts[c+1]), c = 0 ..
 * n_chunks - 1, in order; the running (max, argmax) over the chunks seen so
 * far is the Gumbel-max over them.  The pages state no stopping rule; the one
 * used here follows from Cauchy-Schwarz: row b is final after chunk c once
 * its running best exceeds
 *     (|h_b| * later_norm[c] * fp32(1/T_b) + g_max) * (1 + 2^-8)
 * (greedy rows: |h_b| * later_norm[c] * (1 + 2^-8)), where later_norm[c] is
 * the largest row norm of W over the chunks after c and g_max =
 * -log(-log(1 - 2^-33)) the largest Gumbel value of the noise field.  No later
 * score can overtake such a row, so the ids and scores are those of
 * fs_sample over the whole of W; only the work changes.  Once every row is
 * final the remaining chunks' kernels return without reading their W rows.
 *
 * fs_online_bounds computes later_norm once per weight matrix and chunking:
 *   W            bf16 [V][D], device, 16-byte aligned, D % 8 == 0
 *   cuts         HOST int32 [n_chunks + 1]: 0 = cuts[0] < cuts[1] < ... <
 *                cuts[n_chunks] = V; 1 <= n_chunks <= 65536
 *   later_norm   fp64 [n_chunks], device, 8-byte aligned: later_norm[c] =
 *                max over rows v >= cuts[c+1] of |W_v| (fp64 sums), and
 *                later_norm[n_chunks - 1] = 0
 *   workspace    >= fs_online_bounds_workspace_bytes(V, n_chunks) bytes
 *
 * fs_sample_online takes fs_sample's arguments plus
 *   cuts, n_chunks  as above (HOST array), relative to W row 0: chunk c holds
 *                global ids vocab_offset + cuts[c] .. vocab_offset + cuts[c+1] - 1
 *   later_norm   from fs_online_bounds for the same W and cuts (device)
 *   out_chunks   int32 [B], device: chunks folded into row b's result (the
 *                chunk after which it became final, else n_chunks)
 *   workspace    >= fs_online_workspace_bytes(B, D, V, n_chunks) bytes
 * out_ids / out_maxval as fs_sample.  D <= 32768 (FS_ERR_UNSUPPORTED beyond:
 * the margin 1 + 2^-8 covers the device's fp32 rounding of logits up to that
 * length).  Other errors as fs_sample; a cuts array that does not partition
 * [0, V) is FS_ERR_INVALID_ARG.  Both workspace-size functions return 0 for
 * invalid arguments. */
FS_API size_t fs_online_bounds_workspace_bytes(int32_t V, int32_t n_chunks);
FS_API size_t fs_online_workspace_bytes(int32_t B, int32_t D, int32_t V, int32_t n_chunks);
FS_API fs_status fs_online_bounds(const void* W, int32_t V, int32_t D, const int32_t* cuts,
                                  int32_t n_chunks, double* later_norm, void* workspace,
                                  size_t workspace_bytes, void* stream);
FS_API fs_status fs_sample_online(const void* h, const void* W, int32_t B, int32_t D,
                                  int32_t V, int32_t vocab_offset, const float* temperature,
                                  uint64_t seed, uint64_t step, const int32_t* cuts,
                                  int32_t n_chunks, const double* later_norm, int32_t* out_ids,
                                  float* out_maxval, int32_t* out_chunks, void* workspace,
                                  size_t workspace_bytes, void* stream);
/* The same on fragment-order weights (fs_pack_weights at the same
 * vocab_offset mod 4): W_packed in place of W, every chunk start cuts[c]
 * (0 < c < n_chunks) a multiple of 16, D % 32 == 0 (FS_ERR_INVALID_ARG
 * otherwise).  later_norm comes from fs_online_bounds on the row-major W or
 * from fs_online_bounds_packed on W_packed (same values up to fp64 summation
 * order).  Results as fs_sample_packed over the whole W. */
FS_API fs_status fs_online_bounds_packed(const void* W_packed, int32_t V, int32_t D,
                                         int32_t vocab_offset, const int32_t* cuts,
                                         int32_t n_chunks, double* later_norm, void* workspace,
                                         size_t workspace_bytes, void* stream);
FS_API fs_status fs_sample_online_packed(const void* h, const void* W_packed, int32_t B,
                                         int32_t D, int32_t V, int32_t vocab_offset,
                                         const float* temperature, uint64_t seed, uint64_t step,
                                         const int32_t* cuts, int32_t n_chunks,
                                         const double* later_norm, int32_t* out_ids,
                                         float* out_maxval, int32_t* out_chunks,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* The standard unfused decode step the method replaces (wiki summary,
 * "Method", first paragraph): (1) matmul writing fp32 logits [B][V] to
 * device memory, (2) softmax of z / T writing probabilities, (3)+(4)
 * Gumbel perturbation of log-probabilities and argmax.  Same arguments,
 * noise field and outputs as fs_sample (out_maxval is reported on the
 * s = z / T + g scale by adding back each row's log-normaliser); workspace
 * >= fs_unfused_workspace_bytes(B, D, V).  A baseline for measurement. */
FS_API fs_status fs_sample_unfused(const void* h, const void* W, int32_t B, int32_t D,
                            int32_t V, int32_t vocab_offset, const float* temperature,
                            uint64_t seed, uint64_t step, int32_t* out_ids,
                            float* out_maxval, void* workspace, size_t workspace_bytes,
                            void* stream);

/* ---- the LM head in 8-bit floating point ----
 *
 * Weights and hidden states as e4m3 values (no infinities, largest 448) with a
 * scale for each block of 128 columns -- and of 128 rows, for W --, products in
 * 8 bits, sums in fp32: half the bytes of a decode step, and up to twice the rate
 * of a batch's bf16 logits and log-probabilities.  A scale is the power of two 2^e with the least e >= -110 for which
 * no finite entry of its block exceeds 448 * 2^e (e = 0 for a block of zeros),
 * stored as the byte e + 127 (e8m0); values are rounded to nearest even; entries
 * that are not finite become NaN.  The last block of a row or of the vocabulary
 * may be short.
 *   z[b][v] = sum over blocks k of  2^(eh[b][k] + eW[v / 128][k]) *
 *             sum_{d in k} qh[b][d] qW[v][d]
 * h is given in bf16 and quantised by the call.  Samples, logits in fp32, the
 * tokens' own logits, and all logits of log-probabilities of up to 64 rows or with V
 * up to 8192 are sums in fp32 of exact products.  bf16 logits of more than 32 rows (16
 * with D above 5120) and the other log-probabilities' log-sum-exp take the 8-bit matrix
 * instructions, which cut a product 13 bits below the largest of eight neighbouring
 * ones, towards zero: a logit is off by 1.5e-5 of the logits' spread, and by 1e-5 of
 * itself where its products share a sign (h along the row of W); never by more than
 * 7 * 2^-12 of the sum, over the eights, of their largest product.  With one entry or few
 * that carry a row's log-sum-exp (at low temperatures) that is its error, divided by T;
 * many average it out (1777 tokens on 151936 entries: 4e-7 of the log-probabilities'
 * norm at T = 1; 6e-7 to 9e-7 on 8193 to 20000 with temperatures from 0.3).
 *   D            a multiple of 64 up to 16384; V up to 2^31 - 513; B up to 2^22
 *                (FS_ERR_UNSUPPORTED beyond, and where a launch would hold 2^32
 *                threads)
 *   W_packed     the values in fragment order (below), 16-byte aligned
 *   W_scale      bytes [ceil(V / 128)][ceil(D / 128)], device: 17 to 247
 *   workspace    >= fs_fp8_workspace_bytes(B, D, V) bytes (0 for invalid sizes);
 *                contents on entry ignored
 * NaN or infinite entries of h or W give NaN in the logits that they enter (for
 * the sampler undefined ids); finite ones of 1.9375 * 2^127 or more round to 2^128 and
 * may be infinite in the products.  All calls are asynchronous on `stream`, allocate
 * nothing, give equal bits for equal calls and may be captured into graphs; calls
 * that overlap need distinct workspaces and outputs.  Outputs and workspaces
 * overlap neither one another nor an input. */

/* Quantises W (bf16 [V][D], 16-byte aligned).
 *   packed       zero: out_q is e4m3 [V][D] row-major (D % 8 == 0); nonzero: in the
 *                fragment order that the products read (D % 64 == 0), rows in
 *                groups of 16 and 64 columns at a time: byte
 *                ((g * D/64 + s) * 64 + l) * 16 + j holds
 *                W[16 g + l mod 16][64 s + 16 (l / 16) + j], zero past row V
 *   out_q        16-byte aligned, q_bytes >= fs_fp8_weights_bytes(V, D, packed)
 *                (0 for invalid sizes)
 *   out_scale    bytes [ceil(V / 128)][ceil(D / 128)]
 * fs_pack_weights_fp8 takes row-major values (a checkpoint's, with scales of the
 * above kind) into fragment order. */
FS_API size_t fs_fp8_weights_bytes(int32_t V, int32_t D, int32_t packed);
FS_API fs_status fs_quantize_weights_fp8(const void* W, int32_t V, int32_t D, int32_t packed,
                                         void* out_q, size_t q_bytes, void* out_scale,
                                         void* stream);
FS_API fs_status fs_pack_weights_fp8(const void* q, int32_t V, int32_t D, void* out_packed,
                                     size_t packed_bytes, void* stream);

FS_API size_t fs_fp8_workspace_bytes(int32_t B, int32_t D, int32_t V);

/* The logits: out_logits [B] rows of V, row_pitch elements apart (>= V; what lies
 * between rows is left as it is), bf16 (rounded once) or with out_fp32 nonzero
 * fp32.  Rows may start at any element. */
FS_API fs_status fs_logits_fp8(const void* h, const void* W_packed, const void* W_scale, int32_t B,
                               int32_t D, int32_t V, int32_t out_fp32, void* out_logits,
                               int64_t row_pitch, void* workspace, size_t workspace_bytes,
                               void* stream);

/* fs_token_logprobs on the 8-bit head: same arguments and outputs otherwise. */
FS_API fs_status fs_token_logprobs_fp8(const void* h, const void* W_packed, const void* W_scale,
                                       int32_t B, int32_t D, int32_t V, int32_t vocab_offset,
                                       const float* temperature, const int32_t* token_ids,
                                       float* out_logprob, float* out_lse, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* fs_sample on the 8-bit head: same noise field and outputs; vocab_offset a
 * multiple of 4.  Its (score, id) pairs of shards merge with fs_merge. */
FS_API fs_status fs_sample_fp8(const void* h, const void* W_packed, const void* W_scale, int32_t B,
                               int32_t D, int32_t V, int32_t vocab_offset,
                               const float* temperature, uint64_t seed, uint64_t step,
                               int32_t* out_ids, float* out_maxval, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ---- training on sampled tokens ----
 *
 * What a user does with the tokens that the samplers above return: score them
 * under a model (fs_token_logprobs), turn the scores into a loss and its
 * gradient (fs_policy_loss, fs_preference_loss), take that gradient back
 * through the LM head (fs_token_logprobs_backward) and clip gradients by
 * their global norm (fs_clip_grad_norm).  All calls are asynchronous on
 * `stream`, allocate nothing, add in a fixed order (equal calls give equal
 * bits) and may be captured into graphs; calls that overlap need distinct
 * workspaces and outputs.  Outputs and workspaces overlap neither one another
 * nor an input, except where a call says so.
 */

/* Log-probabilities of given tokens under softmax(z_b / T_b), z_b = W h_b, with
 * no logits in memory.
 *   h, W, B, D, V, vocab_offset  as fs_sample (D up to 2^20, B up to 2^24,
 *                V up to 2^31 - 513, FS_ERR_UNSUPPORTED beyond, and where a
 *                launch would hold 2^32 threads: never for V up to 2^31 - 4096
 *                and B * V up to 2^37); the _packed form reads W in
 *                fragment order (fs_pack_weights, D % 32 == 0)
 *   temperature  fp32 [B], device, or NULL (all 1).  As in the samplers the
 *                logits are scaled by fp32(1/T), and a row whose temperature
 *                is not a positive number is scored unscaled (below 2^-128
 *                fp32(1/T) is infinite: NaN)
 *   token_ids    int32 [B], device: GLOBAL ids; negative: the row has none
 *   out_logprob  fp32 [B]: log p(token); 0 for rows without a token; -inf for
 *                a token outside [vocab_offset, vocab_offset + V)
 *   out_lse      fp32 [B]: log sum_v exp(z_v / T) over these V rows
 *   workspace    >= fs_token_logprobs_workspace_bytes(B, D, V) bytes (0 for
 *                invalid sizes); contents on entry ignored
 * On a vocabulary shard logprob + lse is the token's scaled logit on the rank
 * that holds it and -inf elsewhere, and the log-sum-exp of the ranks' lse is
 * the whole vocabulary's.  NaN entries of h or W give NaN in their rows, and so
 * do scaled logits of +inf; one of -inf has probability 0 (all of them: NaN). */
FS_API size_t fs_token_logprobs_workspace_bytes(int32_t B, int32_t D, int32_t V);
FS_API fs_status fs_token_logprobs(const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                                   int32_t vocab_offset, const float* temperature,
                                   const int32_t* token_ids, float* out_logprob, float* out_lse,
                                   void* workspace, size_t workspace_bytes, void* stream);
FS_API fs_status fs_token_logprobs_packed(const void* h, const void* W_packed, int32_t B, int32_t D,
                                          int32_t V, int32_t vocab_offset, const float* temperature,
                                          const int32_t* token_ids, float* out_logprob,
                                          float* out_lse, void* workspace, size_t workspace_bytes,
                                          void* stream);

/* Gradients through fs_token_logprobs: with g = grad_logprob, p = exp(z / T -
 * lse) and [.] 1 or 0,
 *   dz_v = g / T ([v = token] (1 - exp(logprob)) - [v != token] p_v)
 *   grad_h = dz W,  grad_W = dz^T h
 * Rows without a token (negative id) have no gradient: their grad_h is 0 and
 * their h, logprob, lse and grad_logprob are not used (they may be NaN).
 *   h, W, B, D, V, vocab_offset, temperature, token_ids  as in the forward
 *                call (row-major W; B up to 2^22, B * D up to 2^38, with
 *                grad_W V below 2^30: FS_ERR_UNSUPPORTED beyond)
 *   logprob, lse fp32 [B]: the forward call's outputs; on a vocabulary shard
 *                the whole vocabulary's (logprob is read only for the tokens
 *                of this shard): grad_h is then this shard's share, to be
 *                summed over the ranks, and grad_W its own rows
 *   grad_h       bf16 [B][D], grad_W bf16 [V][D]; either may be NULL (not
 *                wanted).  dz is rounded to bf16 between the products
 *                (but for the tokens' own, which stay fp32), sums are fp32,
 *                results are rounded once
 *   workspace    >= fs_token_logprobs_backward_workspace_bytes(B, D, V) bytes
 *                (0 for invalid sizes).  It holds dz for a slice of the
 *                vocabulary at a time (up to 1 GiB, or 512 bytes per row if
 *                that is more), partial sums of grad_h in
 *                fp32 (up to 512 MiB, or one [B][D] if that is more) and six
 *                bytes per element of h; contents on entry ignored
 * B == 0 sets grad_W to 0. */
FS_API size_t fs_token_logprobs_backward_workspace_bytes(int32_t B, int32_t D, int32_t V);
FS_API fs_status fs_token_logprobs_backward(const void* h, const void* W, int32_t B, int32_t D,
                                            int32_t V, int32_t vocab_offset,
                                            const float* temperature, const int32_t* token_ids,
                                            const float* logprob, const float* lse,
                                            const float* grad_logprob, void* grad_h, void* grad_W,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream);

/* Softmax cross entropy of the LM head with its gradients, with no logits in
 * memory.  With z_b = W h_b, lse = log sum_v exp z_v, p = exp(z - lse), y the
 * target, s = label_smoothing and l = z_loss, a row's loss is
 *   (1 - s) (lse - z_y) + s (lse - mean_v z_v) + l lse^2
 * and u = grad_scale (mean: over the number of rows that have a target)
 *   dz_v = u ((1 + 2 l lse) p_v - s / V - [v = y] (1 - s))
 *   grad_h = dz W,  grad_W = dz^T h
 * Rows without a target (negative, as -100) have loss and gradient 0 and count
 * in no mean; their h is not used (it may be NaN).  A target of V or more has
 * probability 0: its row's loss is +inf (unless s is 1, where no target counts), and
 * the gradient that of the other entries.
 *   h, W         bf16 [B][D] and [V][D], D % 8 == 0: sizes as
 *                fs_token_logprobs_backward takes them; the whole vocabulary
 *   targets      int32 [B], device
 *   label_smoothing in [0, 1], z_loss >= 0, grad_scale: finite
 *   mean         nonzero: the loss is the mean over the rows that have a target
 *                (0 without any), zero: their sum
 *   out_stats    fp32 [3]: the loss; the mean of lse - z_y (its exp is the
 *                perplexity); the mean of lse^2
 *   out_losses   fp32 [B]: every row's loss
 *   grad_h, grad_W  bf16 [B][D], [V][D], the gradient of grad_scale * loss;
 *                either or both may be NULL (not wanted).  dz is rounded to bf16
 *                between the products (but for the targets' own, which stay
 *                fp32), sums are fp32, results are rounded once
 *   workspace    >= fs_cross_entropy_workspace_bytes(B, D, V, grads) bytes (0 for
 *                invalid sizes), grads nonzero where a gradient is wanted.  It
 *                holds two bytes per row and vocabulary entry, up to 4 GiB (a
 *                larger batch, and one of more than 512 rows with D <= 256, takes a
 *                slice of the vocabulary at a time and makes the logits twice); what
 *                fs_token_logprobs_backward holds beside dz; V x D in fp32 for each
 *                of the parts that many rows on a small head are taken in; without
 *                gradients a copy of h alone; and 12 bytes per row and
 *                16 to 128 vocabulary entries (the more rows, the more entries;
 *                without gradients up to 16 KiB for each of 32 rows); contents on
 *                entry ignored
 * Logits of -inf have probability 0 (grad_W is 0 in their rows; grad_h, a product
 * with W, takes 0 times its infinite entries: NaN); NaN or +inf among a row's give
 * NaN.  B == 0 sets the stats and grad_W to 0. */
FS_API size_t fs_cross_entropy_workspace_bytes(int32_t B, int32_t D, int32_t V, int32_t grads);
FS_API fs_status fs_cross_entropy(const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                                  const int32_t* targets, double label_smoothing, double z_loss,
                                  int32_t mean, double grad_scale, float* out_stats,
                                  float* out_losses, void* grad_h, void* grad_W, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Losses over a packed batch: sequence s holds tokens [cu_seqlens[s],
 * cu_seqlens[s+1]) of the flat token arrays (int32 [n_sequences + 1], device,
 * non-decreasing; offsets outside [0, n_tokens] are clamped to it).  Sequences
 * may be empty; n_tokens up to 2^31 - 1.  mask is uint8 [n_tokens], device, or NULL: a token counts
 * where it is nonzero.  Tokens that do not count get gradient 0 and their
 * other entries are not used (they may be NaN).  Entries of out_grad before
 * the first and behind the last sequence are set to 0 with zero_outside, else
 * left as they were.  Sums are held in fp64.
 * Up to 2^20 sequences (FS_ERR_UNSUPPORTED beyond).
 *   workspace  >= fs_loss_workspace_bytes(n_sequences, n_tokens) bytes (for
 *              the preference loss n_sequences = 2 * n_pairs); small batches
 *              need 0 bytes, and then it may be NULL (0 for invalid sizes
 *              too); contents on entry ignored */
FS_API size_t fs_loss_workspace_bytes(int32_t n_sequences, int32_t n_tokens);

typedef enum { FS_KL_K1 = 1, FS_KL_K2 = 2, FS_KL_K3 = 3 } fs_kl_kind;
typedef enum { FS_TOKEN_MEAN = 0, FS_SEQUENCE_MEAN = 1 } fs_loss_reduction;

/* Clipped policy loss with a KL penalty, and its gradient.  Per token, with
 * r = exp(logprob - old_logprob), q = ref_logprob - logprob and advantage A:
 *   surrogate  -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A); with
 *              dual_clip = c > 1 and A < 0 no larger than -c A (0: off)
 *   kl         K1: -q;  K2: q^2 / 2;  K3: exp(q) - q - 1  (0 without a
 *              reference)
 *   loss       surrogate + kl_coef * kl (kl_coef 0: the surrogate alone, and
 *              the mean kl is still reported)
 * averaged over the tokens that count (FS_TOKEN_MEAN) or, per sequence and
 * then over the sequences that have such tokens (FS_SEQUENCE_MEAN).  Without
 * any token that counts everything is 0.  A token has a surrogate gradient
 * where r A attains the minimum and, with dual_clip, r is not above c.
 *   logprob, old_logprob  fp32 [n_tokens];  ref_logprob fp32 [n_tokens] or NULL
 *   advantages  fp32 [n_tokens] if advantage_per_token, else [n_sequences]
 *   clip_low in [0, 1); clip_high >= 0; kl_coef, grad_scale finite
 *   out_stats   fp32 [4]: loss, mean surrogate, mean kl, share of the tokens
 *               that count whose surrogate is clipped
 *   out_grad    fp32 [n_tokens]: grad_scale * d loss / d logprob */
FS_API fs_status fs_policy_loss(const float* logprob, const float* old_logprob,
                                const float* ref_logprob, const float* advantages,
                                const uint8_t* mask, const int32_t* cu_seqlens,
                                int32_t n_sequences, int32_t n_tokens,
                                int32_t advantage_per_token, double clip_low, double clip_high,
                                double dual_clip, double kl_coef, fs_kl_kind kl_kind,
                                fs_loss_reduction reduction, double grad_scale,
                                int32_t zero_outside, float* out_stats, float* out_grad,
                                void* workspace, size_t workspace_bytes, void* stream);

typedef enum {
  FS_PREFERENCE_SIGMOID = 0,
  FS_PREFERENCE_HINGE = 1,
  FS_PREFERENCE_IPO = 2
} fs_preference_kind;

/* Preference loss of paired answers, and its gradient.  Sequences 0 ..
 * n_pairs - 1 are the chosen answers, n_pairs .. 2 n_pairs - 1 the rejected
 * ones (cu_seqlens int32 [2 n_pairs + 1]).  With S the sum over an answer's
 * tokens that count (length_normalised: the mean) of logprob - ref_logprob
 * (logprob alone without a reference), D = S_chosen - S_rejected and
 * x = beta D - margin, a pair's loss is
 *   SIGMOID  -(1 - e) log sigmoid(x) - e log sigmoid(-x), e = label_smoothing
 *            in [0, 0.5]
 *   HINGE    max(0, 1 - x)
 *   IPO      (D - 1 / (2 beta))^2      (margin must be 0)
 * averaged over the pairs both of whose answers have a token that counts; the
 * other pairs have no loss and gradient 0.
 *   beta        positive and finite
 *   out_stats   fp32 [3]: loss, share of those pairs with D > 0, mean beta D
 *   out_rewards fp32 [2 n_pairs]: beta S of every answer (0 for empty ones)
 *   out_grad    fp32 [n_tokens]: grad_scale * d loss / d logprob */
FS_API fs_status fs_preference_loss(const float* logprob, const float* ref_logprob,
                                    const uint8_t* mask, const int32_t* cu_seqlens,
                                    int32_t n_pairs, int32_t n_tokens, fs_preference_kind kind,
                                    double beta, double margin, double label_smoothing,
                                    int32_t length_normalised, double grad_scale,
                                    int32_t zero_outside, float* out_stats, float* out_rewards,
                                    float* out_grad, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* Clipping by the global norm: norm = sqrt(sum over all tensors of x^2), and
 * every element times min(1, max_norm / (norm + 1e-6)).  A norm that is not
 * finite scales nothing (out_norm tells it).
 *   grads, out  HOST arrays of n device pointers; out[i] receives tensor i
 *               and may equal grads[i]; out == NULL: in place.  Otherwise
 *               tensors must not overlap one another.
 *   numel       HOST int64 [n], each >= 0;  dtypes HOST fs_dtype [n]
 *   (pointers aligned to their type; 16-byte aligned ones are read faster)
 *   max_norm    >= 0, or infinity: the norm alone
 *   out_norm    fp32 [1], device: the norm before clipping, summed in fp64
 *   workspace   >= fs_clip_grad_norm_workspace_bytes(numel, n) bytes (0 for
 *               invalid sizes)
 * 0 <= n <= 65536.  The host arrays may be reused once the call returns. */
typedef enum { FS_BF16 = 0, FS_FP16 = 1, FS_FP32 = 2 } fs_dtype;
FS_API size_t fs_clip_grad_norm_workspace_bytes(const int64_t* numel, int32_t n);
FS_API fs_status fs_clip_grad_norm(const void* const* grads, void* const* out,
                                   const int64_t* numel, const fs_dtype* dtypes, int32_t n,
                                   float max_norm, float* out_norm, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Diagnostics: the device noise field, from the same device functions the
 * samplers use.  Writes, for gv = gv0 .. gv0 + n - 1 of one (seed, step,
 * row), the raw Philox word (out_bits, may be NULL) and the Gumbel value g
 * (out_gumbel, may be NULL).  n >= 0; gv0 + n <= 2^32. */
FS_API fs_status fs_debug_noise(uint64_t seed, uint64_t step, uint32_t row, uint32_t gv0,
                         int64_t n, uint32_t* out_bits, float* out_gumbel,
                         void* stream);

/* Diagnostics: g = -log(-log u(x)) for n given words (device arrays). */
FS_API fs_status fs_debug_gumbel(const uint32_t* bits, int64_t n, float* out_gumbel,
                          void* stream);

/* Diagnostics: the compute-unit count and the peak shader clock (kHz) the
 * HIP runtime reports for `device`, from which a caller derives the dense
 * MFMA peak it measures against.  Either output may be NULL. */
FS_API fs_status fs_device_info(int32_t device, int32_t* compute_units, int32_t* clock_khz);

/* Kernel configurations of the fused sampler.  fs_force_config(id) pins
 * every later fs_sample call in the process to configuration id (0 ..
 * fs_num_configs() - 1); id = -1 restores the automatic choice.  Results do
 * not depend on the configuration.  Not synchronised with concurrent calls. */
FS_API int32_t fs_num_configs(void);
FS_API const char* fs_config_name(int32_t id);
FS_API fs_status fs_force_config(int32_t id);
/* Configuration fs_sample would use for batch size B (after forcing), the
 * one fs_sample_packed would use, and the one fs_sample_groups_lse (packed
 * != 0: fs_sample_groups_lse_packed) would use over a V-row vocabulary (the
 * same choice as fs_sample's, or fs_sample_packed's).  -1 for an invalid
 * shape. */
FS_API int32_t fs_selected_config(int32_t B, int32_t D, int32_t V);
FS_API int32_t fs_selected_config_packed(int32_t B, int32_t D, int32_t V);
FS_API int32_t fs_selected_config_groups(int32_t B, int32_t D, int32_t V, int32_t packed);

/* Profiling of the fused kernel.  fs_profile_enable(capacity) creates
 * 2 * capacity HIP events (outside any sampling call); while enabled, each of
 * the next `capacity` fs_sample / fs_sample_partial / fs_sample_partial_lse
 * calls (and their _packed forms) records one event before and one after its
 * fused-kernel launch, on the caller's stream (the online sampler's chunk
 * launches are not recorded).
 * fs_profile_read waits for the recorded events, returns the number of timed
 * launches and the sum, minimum and maximum of their durations in
 * milliseconds (any output may be NULL), and re-arms the recorder.
 * fs_profile_enable(0) destroys the events.  Not for concurrent callers. */
FS_API fs_status fs_profile_enable(int32_t capacity);
FS_API fs_status fs_profile_read(int32_t* launches, double* total_ms, double* min_ms,
                                 double* max_ms);

FS_API const char* fs_status_string(fs_status s);
FS_API const char* fs_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FLASHSAMPLE_H */
