// Host-side launchers of the library's kernels (internal).
#pragma once

#include <mutex>

#include "chunk_common.cuh"

namespace sala {

// Kernels of the library, for the timing instrumentation (names in api.cu).
enum KernelId {
    kKSegTable = 0,
    kKPrefillFused,
    kKRecurrentStep,
    kKRecurrentStepIndexed,
    kKOutputNormGate,
    kKQkPrologue,
    kKGdnStep,
    kKGdnFwd,
    kKGdnNewv,
    kKPrefillPair,
    kKVerifyDrafts,
    kKDraftStep,
    kKPoolPlan,
    kKPoolCopy,
    kKKvAppend,
    kKPagedPlan,
    kKPagedAttention,
    kKPagedCombine,
    kKPagedWeights,
    kKKvSelect,
    kKKvMove,
    kKTokenLogprobs,
    kKernelCount
};

// While timing is enabled, brackets one launch with events on `stream` (no-op otherwise).
class LaunchTimer {
  public:
    LaunchTimer(KernelId id, cudaStream_t stream);
    ~LaunchTimer();
    LaunchTimer(const LaunchTimer &) = delete;
    LaunchTimer &operator=(const LaunchTimer &) = delete;

  private:
    KernelId id_;
    cudaStream_t stream_;
    cudaEvent_t start_ = nullptr;
};

// Device address of the library's status word on the current device.
cudaError_t device_status_address(int **out);

cudaError_t launch_recurrent_step(const void *q, const void *k, const void *v, const float *g,
                                  float scale, float *S, void *o, int64_t units,
                                  cudaStream_t stream);

// The q/k prologue in kernel-argument form (qw null: none). inv_freq[i] = float(theta^(-i/64)),
// computed on the host in double precision and rounded once.
struct QkPrologue {
    const uint16_t *qw = nullptr, *kw = nullptr;   // bf16 [128] RMSNorm weights
    const int64_t *pos = nullptr;                  // decode: [N] positions
    float eps = 0.f;
    float inv_freq[64] = {};
};
QkPrologue make_qk_prologue(const sala_qk_prologue *p, const int64_t *positions);

// The same step on states in a pool [P, H, 128, 128] (fp32, or bf16 if `bf16`) addressed by
// idx[N] (negative: padding row, o = 0; >= P: SALA_ERR_BAD_INDEX recorded in `status`), with
// the q/k prologue fused if pro.qw is set.
cudaError_t launch_recurrent_step_indexed(const void *q, const void *k, const void *v,
                                          const float *g, float scale, void *pool, bool bf16,
                                          const int32_t *idx, int64_t P, void *o, int64_t N,
                                          int H, const QkPrologue &pro, int *status,
                                          cudaStream_t stream);

// The q/k prologue in place on a prefill's q and k ([T_total, H, 128] rows; positions from
// the segment table's sequence bounds plus start_pos).
cudaError_t launch_qk_prologue(void *q, void *k, const QkPrologue &pro, const SegTable &t,
                               const int64_t *start_pos, int64_t T_total, int H, int *status,
                               cudaStream_t stream);

// Segment table from cu_seqlens (or B equal rows); also zeroes the work ticket and the
// hand-off flags of the fused prefill, and writes hT (= h0, or zeros) of empty sequences.
cudaError_t launch_seg_table(const SegTable &t, int64_t T_total, uint32_t *ticket,
                             uint32_t *flags, int64_t nflags, int H, const float *h0, float *hT,
                             int *status, cudaStream_t st);

// The fused tensor-core prefill (prefill_fused.cu): one persistent launch of `grid` CTAs
// (the final state of empty sequences is written by the segment-table kernel). `incl` holds [max_units, 128, 128] fp32 hand-off
// states, `flags` [max_units] words, `ticket` one word; `epoch` is nonzero and differs from
// the previous call's. `status` receives SALA_ERR_TIMEOUT if a bounded wait gives up.
cudaError_t setup_fused_kernel();

// The same prefill at two CTAs per SM (prefill_pair.cu): one unit in flight per CTA, half of
// an SM's shared and tensor memory each; `grid` up to twice the SM count. Same arguments.
cudaError_t launch_prefill_pair(const ChunkArgs &a, const SegTable &t, int64_t T_total,
                                int64_t max_units, const float *h0, float *hT, float *incl,
                                uint32_t *flags, uint32_t *ticket, uint32_t epoch, int grid,
                                int *status, cudaStream_t st);
cudaError_t setup_pair_kernel();
cudaError_t launch_prefill_fused(const ChunkArgs &a, const SegTable &t, int64_t T_total,
                                 int64_t max_units, const float *h0, float *hT, float *incl,
                                 uint32_t *flags, uint32_t *ticket, uint32_t epoch, int grid,
                                 int *status, cudaStream_t st);

// out[t] = RMSNorm(o[t]) * w * sigmoid(z[t]) over the H * 128 features of each of T tokens
// (bf16 in and out, fp32 arithmetic); out may be o.
cudaError_t launch_output_norm_gate(const void *o, const void *z, const void *w, float eps,
                                    void *out, int64_t T, int H, cudaStream_t stream);

// One gated-delta-rule step on [units] dense fp32 states (one CTA per (sequence, head)).
cudaError_t launch_gdn_step(const void *q, const void *k, const void *v, const float *g,
                            const float *beta, float scale, float *S, void *o, int64_t units,
                            cudaStream_t stream);

// The gated delta rule over whole sequences (recurrent form), one CTA per (sequence, head);
// sequence bounds from t.cu (or rows of t.T_row tokens); h0 / hT may be null.
cudaError_t launch_gdn_fwd(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, float scale, const float *h0, const SegTable &t,
                           int64_t T_total, void *o, float *hT, int H, cudaStream_t stream);

// Failure-path test settings of the fused prefill (sala_gla_debug_prefill_knobs): the limit
// of the wait for a predecessor's state (0: the default 2 s) and a unit whose flag is withheld
// (-1: none).
void prefill_fault_knobs(uint64_t *wait_ns, int64_t *withhold);

// The gated delta rule's chunked form: new_v = U - W S of every token (bf16 [T_total, H, 128]
// into nv) for sala_gla_gdn_chunk_fwd, one CTA per (sequence, head); sequence bounds from t.cu
// (or rows of t.T_row tokens), kept inside the tensors.
cudaError_t setup_gdn_chunk_kernel();
cudaError_t launch_gdn_newv(const void *k, const void *v, const float *g, const float *beta,
                            const float *h0, const SegTable &t, int64_t T_total, void *nv, int H,
                            int *status, cudaStream_t st);

// Drafted tokens against the target's probabilities (fp32, or bf16 if `bf16`): rows of V
// probabilities, `p_stride` / `q_stride` elements apart; q and num_drafts may be null.
cudaError_t launch_verify_drafts(const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                                 bool bf16, const int32_t *x, const int32_t *num_drafts,
                                 const float *u, const float *s, int32_t *tokens,
                                 int32_t *accepted, int64_t N, int K, int64_t V, int sm_count,
                                 const int *fits, int *status, cudaStream_t stream);
// fits[i]: clusters that run at once with at most i + 1 CTAs on an SM.
constexpr int kVerifyFits = 6;
cudaError_t setup_verify_drafts_kernel(int *fits);

// Decode step over T drafted tokens on pooled states, after committing accepted[n] + 1 of the
// T_pend tokens of the step before (T or T_pend may be 0).
cudaError_t launch_draft_step(const void *q, const void *k, const void *v, const float *g,
                              const int32_t *num_tokens, const void *pend_k, const void *pend_v,
                              const float *pend_g, const int32_t *accepted, float scale, void *pool,
                              bool bf16, const int32_t *slots, int64_t P, void *o, int64_t N,
                              int64_t T, int64_t T_pend, int H, int sm_count, int *status,
                              cudaStream_t stream);

cudaError_t setup_draft_step_kernel();

// States of a pool [L, P, H, 128, 128]: n pairs of slots copied (source < 0: zeros, destination
// < 0: skipped), n requests forked into the lowest free slots, n slots freed, the used slots
// moved to the front.
cudaError_t launch_state_pool_copy(const void *src_pool, bool src_bf16, int64_t src_P, void *dst_pool,
                                   bool dst_bf16, int64_t dst_P, const int32_t *src,
                                   const int32_t *dst, int64_t n, int64_t L, int H, int *status,
                                   cudaStream_t st);
cudaError_t launch_state_pool_fork(void *pool, bool bf16, int64_t L, int64_t P, int H, int32_t *used,
                                   const int32_t *parents, int32_t *children, int64_t n, int *status,
                                   cudaStream_t st);
cudaError_t launch_state_pool_free(int32_t *used, int64_t P, const int32_t *slots, int64_t n, int *status,
                                   cudaStream_t st);
cudaError_t launch_state_pool_compact(void *pool, bool bf16, int64_t L, int64_t P, int H, int32_t *used,
                                      int32_t *mapping, int32_t *live, cudaStream_t st);

// A paged cache and a step's new tokens (see sala_kv_cache); kernels take it by value.
struct KvArgs {
    uint8_t *k, *v;                    // [P, H, S, 128] pages, bf16 or e4m3
    const float *k_scale, *v_scale;    // [H] or null
    float *weights;                    // [P, H, S] or null
    const int32_t *table, *lens;       // [N, W], [N]
    const int64_t *cu;                 // [N + 1] token offsets, or null: T_row tokens each
    int64_t P, W, N, T, T_row;         // T: tokens in all
    int S, log_S, H;                   // S = 1 << log_S places to a page, H key/value heads
    bool e4m3;
    int *status;
};

// Keys and values of new tokens (strides in elements between tokens) into the pages.
cudaError_t launch_kv_append(const KvArgs &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             cudaStream_t st);

// Attention of the new tokens; G query heads on each key/value head. `lse` may be null. `ws`: scratch of
// paged_attention_scratch bytes.
size_t paged_attention_scratch(const KvArgs &c, int G, bool accumulate, int sm_count);
cudaError_t setup_paged_attention_kernel();
cudaError_t launch_paged_attention(const KvArgs &c, const void *q, int64_t q_stride, float scale, void *o, float *lse,
                                   bool accumulate, int G, void *ws, int sm_count, cudaStream_t st);

// Eviction: `kept` [N, H, budget] gets the former places (then -1), the kept tokens move.
cudaError_t launch_kv_evict(const KvArgs &c, int64_t budget, int64_t sinks, int64_t recent, int32_t *new_lens,
                            int32_t *kept, int sm_count, cudaStream_t st);

// Log probabilities of tokens [N, M], entropy and the K largest logits of rows of V (fp32, or bf16 if `bf16`).
// `ws`: scratch of token_logprobs_scratch bytes, for rows cut into token_logprobs_parts.
int token_logprobs_parts(int64_t N, int64_t V, bool bf16, int K, int sm_count);
size_t token_logprobs_scratch(int64_t N, int parts, int K);
cudaError_t launch_token_logprobs(const void *x, int64_t stride, bool bf16, const int32_t *tokens, float *logprobs,
                                  float *entropy, int32_t *top_tokens, float *top_logprobs, int64_t N, int64_t V,
                                  int M, int K, void *ws, int parts, int sm_count, int *status, cudaStream_t st);

// Nonzero tag of one prefill call for the hand-off flags (differs from the previous call's).
uint32_t next_prefill_epoch();

// Tokens per segment of the fused prefill for T_total tokens and H heads on sm_count SMs.
int64_t choose_segment_tokens(int64_t T_total, int64_t H, int sm_count);

}  // namespace sala
