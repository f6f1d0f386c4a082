// Internal interface of the serving operators: the paged 8-bit key/value
// cache (append, gather, attention) and sampling.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>

namespace q4 {

constexpr int kKvBlock = 16;        // tokens that share a scale
constexpr int kKvMaxSeqs = 2048;    // sequences of one call

// A cache: codes int8 [pages][heads][page][dim], scales fp32 [pages][heads][page / 16].
struct KvView {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int pages, heads, dim, page;   // page: tokens, a power of two in [16, 256]
  int page_log2;
};

// The batch: sequence b holds kv_len[b] tokens, the last cu[b + 1] - cu[b] of
// them new; new tokens are packed in sequence order, T rows in all.
struct KvBatch {
  const int32_t* table;      // [B][table_stride] page of each run of `page` tokens
  long long table_stride;
  const int32_t* kv_len;     // [B]
  const int32_t* cu;         // [B + 1]
  int B, T;
};

struct KvAppendParams {
  KvView c;
  KvBatch b;
  void* q_out;               // [T][Hq][dim], or null (no queries)
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;   // elements between rows of tokens
  int Hq;
  int in_bf16, out_bf16;
  const float* cos;          // [rope_rows][rope_dim / 2], or null (no rotation)
  const float* sin;
  int rope_rows, rope_dim, rope_pairs;
  const int32_t* positions;  // [T] rows of the tables, or null: the tokens' slots
  const float* q_norm;       // [dim] or null
  const float* k_norm;
  float eps;
  unsigned* err;
};
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t st);

struct KvGatherParams {
  KvView c;
  const int32_t* table;
  long long table_stride;
  const int32_t* first;      // [B] first token read of each sequence
  const int32_t* cu;         // [B + 1] output rows of each sequence
  int B, T;
  void* k_out;               // [T][heads][dim]
  void* v_out;
  int out_bf16;
  unsigned* err;
};
cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t st);

struct KvAttnCall {
  KvView c;
  KvBatch b;
  void* out;                 // [T][Hq][dim]
  const void* q;
  long long q_stride;
  int Hq;
  int q_bf16, out_bf16;
  float scale;
  int causal;
  long long window;          // keys seen by a query, itself included; 0: all
  long long sinks;           // first tokens that stay visible whatever the window
  const int32_t* tree;       // [T][tree_words] bits: new tokens of its sequence that each one sees, or null
  int tree_words;
  float* lse;                // [T][Hq] log of each row's sum of exponentials, or null
  unsigned* err;
};
// Whether a call has sinks, a tree or sums to give: kernels have forms of their own for it.
inline bool kv_attn_more(const KvAttnCall& a) { return (a.sinks > 0 && a.window > 0) || a.tree || a.lse; }
// Workspace bytes, the first kv_attn_header_bytes() of them zero before the
// first use and left zero.
size_t kv_attn_header_bytes();
size_t kv_attn_split_bytes(int dim, int sms);
// Sequences with at most max_rows query rows (new tokens x query heads of a kv
// head), and zeros for rows of no sequence.  max_q: new tokens of a sequence at most.
cudaError_t launch_kv_attn_split(const KvAttnCall& a, int max_q, int max_rows, void* ws, int sms,
                                 cudaStream_t st);
// On the tensor cores, split over the cached tokens: sequences with at most max_rows query rows, and zeros for rows of
// no sequence; bf16 q and out.  Workspace as for the split form, of kv_draft_bytes.
size_t kv_draft_bytes(int dim, int sms);
cudaError_t launch_kv_draft(const KvAttnCall& a, int max_rows, void* ws, int sms, cudaStream_t st);
// Sequences with more than split_rows query rows (0: all, and zeros for rows of no
// sequence); bf16 q and out.  rows: rows of fp16 keys and values the workspace holds (kv_prompt_rows).
long long kv_prompt_rows(int B, long long max_kv, long long total_kv);
size_t kv_prompt_bytes(const KvView& c, int B, long long rows);
cudaError_t launch_kv_prompt(const KvAttnCall& a, int split_rows, long long rows, void* ws,
                             cudaStream_t st);

// Attention weights of cached tokens.
struct KvWeighCall {
  KvView c;
  KvBatch b;
  float* weight;             // [pages][heads][page]
  const void* q;
  long long q_stride;
  int Hq, q_bf16;
  const float* lse;          // [T][Hq]
  const int32_t* held;       // [B] tokens that have a weight already, or null (those before the new ones)
  float scale;
  int causal;
  long long window, sinks;
  unsigned* err;
};
// max_q: new tokens of a sequence at most, as far as the caller knows.
cudaError_t launch_kv_weigh(const KvWeighCall& a, long long max_q, int sms, cudaStream_t st);
// On the tensor cores, bf16 queries: sequences with more than split_rows query rows of a head (0: all of them).
cudaError_t launch_kv_weigh_prompt(const KvWeighCall& a, int split_rows, int sms, cudaStream_t st);
int kv_weigh_prompt_group();

// The tokens of a sequence and head that a budget leaves.
struct KvSelectParams {
  KvView c;
  const int32_t* table;
  long long table_stride;
  const int32_t* kv_len;
  const int32_t* budget;
  const float* weight;
  int32_t* kept;             // [B][heads][width]
  long long width;
  int32_t* count;            // [B]
  int B;
  long long sinks, recent;
  unsigned* err;
};
cudaError_t launch_kv_select(const KvSelectParams& p, long long max_kv, int sms, cudaStream_t st);

// Moves tokens to consecutive places.
struct KvCompactParams {
  KvView c;
  float* weight;             // or null
  const int32_t* table;
  long long table_stride;
  const int32_t* to_table;   // or null: within `table`
  long long to_stride;
  const int32_t* kv_len;
  const int32_t* first;      // or null
  const int32_t* kept;       // [B][kept_heads][width]
  int kept_heads;
  long long width;
  const int32_t* count;
  int B;
  unsigned* err;
};
cudaError_t launch_kv_compact(const KvCompactParams& p, cudaStream_t st);

// Penalties, biases and masks of rows of logits.
struct AdjustParams {
  void* out;
  const void* logits;
  long long out_stride, stride;   // elements between rows
  int out_bf16, bf16, T, V;
  const int32_t* request;    // [T] or null
  long long requests;
  const int32_t* history;    // [requests][history_width] or null
  int history_width;
  const int32_t* history_len;   // [T]
  const int32_t* prompt_len;    // [T] or null
  const float* repetition;   // each [T] or null
  const float* frequency;
  const float* presence;
  const int32_t* bias_index;    // [requests][bias_width] or null
  const float* bias;
  int bias_width;
  const int32_t* mask;       // [masks][ceil(V / 32)] or null
  long long masks;
  const int32_t* mask_row;   // [T] or null
  unsigned* err;
};
cudaError_t launch_adjust(const AdjustParams& p, int sms, cudaStream_t st);

struct SampleParams {
  int32_t* tokens;
  float* probs;              // or null
  const void* logits;
  long long stride;          // elements between rows
  int bf16, T, V;
  const float* u;
  const float* temperature;  // each [T] or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
};
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st);
// Longest row launch_sample takes.
int sample_max_vocab();

// Rows of the table of entry points that need the device: SM count and status
// word of the current device (a Q4_* status).
int device_info(int* sms, unsigned** status);
// Scratch of `st` for the attention calls without a workspace, its header
// zeroed when it is allocated; eager calls only (nullptr while the stream is
// captured or when it cannot be allocated).  A larger one replaces it once the
// stream has drained, so the caller enqueues its kernels before it lets go of
// `hold`: another host thread's call on the stream may need a larger one.
void* kv_stream_scratch(cudaStream_t st, size_t bytes, std::unique_lock<std::mutex>& hold);

}  // namespace q4
