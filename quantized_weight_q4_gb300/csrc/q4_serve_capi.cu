// C ABI of the serving operators (include/q4.h): the paged 8-bit cache,
// attention over it, and sampling.  Argument checks and workspaces.
#include <cstdint>

#include <cuda_runtime.h>

#include "q4.h"
#include "q4_kv.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(int dtype) { return dtype == Q4_F32 || dtype == Q4_BF16; }
int64_t size_of(int dtype) { return dtype == Q4_F32 ? 4 : 2; }
int status_of(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

constexpr int64_t kMaxTokens = 1 << 24;

int check_cache(const q4_kv_cache* c, q4::KvView* v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->pages <= 0 || c->heads <= 0 || c->dim <= 0 ||
      c->page_tokens <= 0)
    return Q4_ERR_ARG;
  if ((c->dim != 64 && c->dim != 128) || c->page_tokens < 16 || c->page_tokens > 256 ||
      (c->page_tokens & (c->page_tokens - 1)) || c->heads > 1024 || c->pages > (1LL << 30) ||
      c->pages * c->heads * (c->page_tokens / 16) > 0x7fffffffLL)
    return Q4_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return Q4_ERR_ALIGN;
  *v = {c->k, c->v, c->k_scale, c->v_scale, static_cast<int>(c->pages), static_cast<int>(c->heads),
        static_cast<int>(c->dim), static_cast<int>(c->page_tokens), 4};
  while ((1 << v->page_log2) < v->page) ++v->page_log2;
  return Q4_OK;
}

int check_batch(const int32_t* table, int64_t table_stride, const int32_t* len, const int32_t* cu, int64_t B,
                int64_t T) {
  if (!table || !len || !cu || table_stride <= 0 || B <= 0 || T <= 0) return Q4_ERR_ARG;
  if (B > q4::kKvMaxSeqs || T > kMaxTokens || table_stride > (1LL << 27)) return Q4_ERR_SHAPE;
  if (!aligned(table, 4) || !aligned(len, 4) || !aligned(cu, 4)) return Q4_ERR_ALIGN;
  return Q4_OK;
}

// Rows of `heads` heads, `stride` elements apart: every head starts at a multiple of 16 bytes.
int check_rows(const void* p, int64_t stride, int64_t heads, int64_t dim, int dtype) {
  if (!p) return Q4_ERR_ARG;
  if (stride < heads * dim || stride > (1LL << 40)) return Q4_ERR_ARG;
  if (!aligned(p, 16) || stride * size_of(dtype) % 16) return Q4_ERR_ALIGN;
  return Q4_OK;
}

}  // namespace

extern "C" {

int q4_kv_append(const q4_kv_cache* cache, void* q_out, int q_out_dtype, const void* q, int64_t q_stride,
                 const void* k, int64_t k_stride, const void* v, int64_t v_stride, int dtype, int64_t Hq,
                 const q4_rope* rope, const float* q_norm, const float* k_norm, float eps,
                 const int32_t* page_table, int64_t table_stride, const int32_t* kv_len, const int32_t* cu_q,
                 int64_t B, int64_t T, void* stream) {
  q4::KvAppendParams p = {};
  int rc = check_cache(cache, &p.c);
  if (rc == Q4_OK) rc = check_batch(page_table, table_stride, kv_len, cu_q, B, T);
  if (rc != Q4_OK) return rc;
  if (!known(dtype) || (q && !known(q_out_dtype))) return Q4_ERR_DTYPE;
  if (!q != !q_out || (q && Hq <= 0) || (q_norm && !q) || !(eps >= 0.f)) return Q4_ERR_ARG;
  if (q && Hq > 4096) return Q4_ERR_SHAPE;
  rc = check_rows(k, k_stride, cache->heads, cache->dim, dtype);
  if (rc == Q4_OK) rc = check_rows(v, v_stride, cache->heads, cache->dim, dtype);
  if (rc == Q4_OK && q) rc = check_rows(q, q_stride, Hq, cache->dim, dtype);
  if (rc != Q4_OK) return rc;
  if (!aligned(q_out, 16) || !aligned(q_norm, 4) || !aligned(k_norm, 4)) return Q4_ERR_ALIGN;
  if (rope) {
    if (!rope->cos || !rope->sin || rope->rows <= 0 || rope->dim <= 0 || rope->dim > cache->dim ||
        (rope->style != Q4_ROPE_HALVES && rope->style != Q4_ROPE_PAIRS))
      return Q4_ERR_ARG;
    if (rope->dim % 8 || rope->rows > (1LL << 30)) return Q4_ERR_SHAPE;
    if (!aligned(rope->cos, 16) || !aligned(rope->sin, 16)) return Q4_ERR_ALIGN;
    p.cos = rope->cos;
    p.sin = rope->sin;
    p.rope_rows = static_cast<int>(rope->rows);
    p.rope_dim = static_cast<int>(rope->dim);
    p.rope_pairs = rope->style == Q4_ROPE_PAIRS;
  }
  int sms = 0;
  rc = q4::device_info(&sms, &p.err);
  if (rc != Q4_OK) return rc;
  p.b = {page_table, table_stride, kv_len, cu_q, static_cast<int>(B), static_cast<int>(T)};
  p.q_out = q_out;
  p.q = q, p.k = k, p.v = v;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.Hq = static_cast<int>(q ? Hq : 0);
  p.in_bf16 = dtype == Q4_BF16;
  p.out_bf16 = q_out_dtype == Q4_BF16;
  p.q_norm = q_norm, p.k_norm = k_norm, p.eps = eps;
  return status_of(q4::launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

int q4_kv_gather(void* k_out, void* v_out, int dtype, const q4_kv_cache* cache, const int32_t* page_table,
                 int64_t table_stride, const int32_t* first, const int32_t* cu, int64_t B, int64_t T, void* stream) {
  q4::KvGatherParams p = {};
  int rc = check_cache(cache, &p.c);
  if (rc == Q4_OK) rc = check_batch(page_table, table_stride, first, cu, B, T);
  if (rc != Q4_OK) return rc;
  if (!k_out || !v_out) return Q4_ERR_ARG;
  if (!known(dtype)) return Q4_ERR_DTYPE;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return Q4_ERR_ALIGN;
  int sms = 0;
  rc = q4::device_info(&sms, &p.err);
  if (rc != Q4_OK) return rc;
  p.table = page_table, p.table_stride = table_stride;
  p.first = first, p.cu = cu;
  p.B = static_cast<int>(B), p.T = static_cast<int>(T);
  p.k_out = k_out, p.v_out = v_out;
  p.out_bf16 = dtype == Q4_BF16;
  return status_of(q4::launch_kv_gather(p, static_cast<cudaStream_t>(stream)));
}

namespace {

// Query rows (new tokens x query heads that share a kv head) up to which a
// sequence takes the split form, for B sequences of up to max_kv tokens.  The
// split form streams the codes once for every 16 rows, 1650 blocks of 16 tokens
// a microsecond (heads of 64: 2800) with 30 blocks' time to start each; the
// prompt form first writes the codes as fp16 and then takes 1.55 us for each
// 128 tokens and 256 rows, on one SM however long they are, with 8 us to start
// and end.
// Measured with 8 kv heads of 128 (split / prompt form, us): one sequence of
// 16,000 tokens, 128 rows 59 / 212, 512 rows 187 / 220; 16 sequences of 8,000,
// 64 rows 183 / 265, 128 rows 323 / 266; 16 of 500, 64 rows 25 / 42, 128 rows
// 54 / 44; 64 of 300, 64 rows 73 / 97, 128 rows 131 / 102; 64 of 1,000, 64 rows
// 133 / 174, 128 rows 245 / 194; 64 of 4,000, 64 rows 366 / 533, 96 rows
// 537 / 535.  Heads of 64: 16 of 500, 64 rows 17 / 32; 16 of 8,000, 64 rows
// 111 / 191, 128 rows 194 / 191; 64 of 300, 96 rows 63 / 68; 64 of 4,000, 64
// rows 207 / 372, 128 rows 396 / 374.
constexpr int kRowTile = 16, kMostSplitRows = 1024;
constexpr double kStartBlocks = 30;
double split_rate(int dim) { return dim == 128 ? 1650 : 2800; }
// of one block of a head: writing its codes as fp16, and reading them again
double expand_us(int dim) { return 16.0 * dim * 6 / 5.5e6; }
double read_us(int dim) { return 16.0 * dim * 4 / 6e6; }

int split_rows_of(const q4::KvView& c, int64_t B, int64_t max_kv, int sms) {
  const double heads = static_cast<double>(B) * c.heads, blocks = static_cast<double>((max_kv + 15) / 16);
  const double expand = heads * blocks * expand_us(c.dim), read = heads * blocks * read_us(c.dim);
  int rows = kRowTile;
  for (int r = 2 * kRowTile; r <= kMostSplitRows; r += kRowTile) {
    const double split = 10 + heads * (r / kRowTile) * (blocks + kStartBlocks) / split_rate(c.dim);
    const double ctas = heads * ((r + 255) / 256);
    const double walk = static_cast<double>(static_cast<int64_t>((ctas + sms - 1) / sms)) * (((max_kv + 127) / 128) * 1.55 + 8);
    if (split > 10 + expand + (walk > read ? walk : read)) break;
    rows = r;
  }
  return rows;
}

// Tokens of a sequence above which sequences of up to `rows` query rows take
// the split form in every batch: by the costs above the prompt form takes at
// least expand_us + read_us for a block, so that it can be the faster one only
// while starting the split form's tiles weighs more than what each block saves.
int64_t most_prompt_tokens(int dim, int64_t rows) {
  if (rows > kMostSplitRows) return INT64_MAX;
  const double tiles = static_cast<double>((rows + kRowTile - 1) / kRowTile), block = tiles / split_rate(dim);
  const double saved = expand_us(dim) + read_us(dim) - block;
  return saved > 1e-9 ? 16 * (static_cast<int64_t>(kStartBlocks * block / saved) + 1) : INT64_MAX;
}

struct AttnPlan {
  bool prompt;          // the call may have sequences for the prompt form
  int split_rows;       // query rows up to which a sequence takes the split form
  long long rows;       // fp16 rows of the prompt form
  size_t split_bytes, total;
};

// sized: with room for the prompt form wherever a call of these bounds, or of smaller ones, takes it
AttnPlan attn_plan(const q4::KvView& c, int64_t Hq, int64_t B, int64_t T, int64_t max_q, int64_t max_kv,
                   int64_t total_kv, bool bf16, bool sized, int sms) {
  AttnPlan p = {};
  const int64_t most_rows = (max_q < T ? max_q : T) * (Hq / c.heads);
  p.split_rows = sized ? kRowTile : split_rows_of(c, B, max_kv, sms);
  p.prompt = bf16 && most_rows > p.split_rows;
  p.split_bytes = (q4::kv_attn_split_bytes(c.dim, sms) + 255) / 256 * 256;
  p.total = p.split_bytes;
  if (p.prompt) {
    const int64_t longest = sized ? most_prompt_tokens(c.dim, most_rows) : max_kv;
    p.rows = q4::kv_prompt_rows(static_cast<int>(B), longest < max_kv ? longest : max_kv, total_kv);
    p.total += q4::kv_prompt_bytes(c, static_cast<int>(B), p.rows);
  }
  return p;
}

}  // namespace

size_t q4_kv_attention_workspace_size(const q4_kv_cache* cache, int64_t Hq, int64_t B, int64_t T, int64_t max_q,
                                      int64_t max_kv, int64_t total_kv) {
  q4::KvView v;
  if (check_cache(cache, &v) != Q4_OK || Hq <= 0 || Hq % v.heads || B <= 0 || B > q4::kKvMaxSeqs || T <= 0 ||
      max_q <= 0 || max_kv <= 0 || max_kv > (1LL << 30) || total_kv < 0)
    return 0;
  int sms = 0;
  unsigned* status = nullptr;
  if (q4::device_info(&sms, &status) != Q4_OK) return 0;
  return attn_plan(v, Hq, B, T, max_q, max_kv, total_kv, true, true, sms).total;
}

int q4_kv_attention(void* out, int out_dtype, const void* q, int q_dtype, int64_t q_stride, int64_t Hq,
                    const q4_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                    const int32_t* kv_len, const int32_t* cu_q, int64_t B, int64_t T, int64_t max_q, int64_t max_kv,
                    int64_t total_kv, float scale, int causal, int64_t window, void* workspace,
                    size_t workspace_bytes, void* stream) {
  q4::KvAttnCall a = {};
  int rc = check_cache(cache, &a.c);
  if (rc == Q4_OK) rc = check_batch(page_table, table_stride, kv_len, cu_q, B, T);
  if (rc != Q4_OK) return rc;
  if (!out || Hq <= 0 || max_q <= 0 || max_kv <= 0 || total_kv < 0 || window < 0 || (causal != 0 && causal != 1) ||
      (window > 0 && !causal))
    return Q4_ERR_ARG;
  if (!known(q_dtype) || !known(out_dtype)) return Q4_ERR_DTYPE;
  if (Hq % cache->heads || Hq > 4096 || max_kv > (1LL << 30)) return Q4_ERR_SHAPE;
  rc = check_rows(q, q_stride, Hq, cache->dim, q_dtype);
  if (rc != Q4_OK) return rc;
  if (!aligned(out, 16) || !aligned(workspace, 16)) return Q4_ERR_ALIGN;
  int sms = 0;
  rc = q4::device_info(&sms, &a.err);
  if (rc != Q4_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const AttnPlan plan = attn_plan(a.c, Hq, B, T, max_q, max_kv, total_kv,
                                  q_dtype == Q4_BF16 && out_dtype == Q4_BF16, false, sms);
  if (plan.rows > 0x7fffffffLL) return Q4_ERR_SHAPE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  std::unique_lock<std::mutex> hold;
  if (ws) {
    if (workspace_bytes < plan.total) return Q4_ERR_WORKSPACE;
  } else {
    ws = static_cast<uint8_t*>(q4::kv_stream_scratch(st, plan.total, hold));
    if (!ws) return Q4_ERR_WORKSPACE;
  }
  a.b = {page_table, table_stride, kv_len, cu_q, static_cast<int>(B), static_cast<int>(T)};
  a.out = out, a.q = q, a.q_stride = q_stride, a.Hq = static_cast<int>(Hq);
  a.q_bf16 = q_dtype == Q4_BF16, a.out_bf16 = out_dtype == Q4_BF16;
  a.scale = scale, a.causal = causal, a.window = window;
  const int most = static_cast<int>(max_q < T ? max_q : T);
  if (!plan.prompt) return status_of(q4::launch_kv_attn_split(a, most, 0x7fffffff, ws, sms, st));
  // one sequence: no second form beside the prompt's
  const int split_rows = B == 1 ? 0 : plan.split_rows;
  cudaError_t e = cudaSuccess;
  if (B > 1) e = q4::launch_kv_attn_split(a, most, split_rows, ws, sms, st);
  if (e == cudaSuccess) e = q4::launch_kv_prompt(a, split_rows, plan.rows, ws + plan.split_bytes, st);
  return status_of(e);
}

int q4_sample(int32_t* tokens, float* probs, const void* logits, int logits_dtype, int64_t stride, int64_t T,
              int64_t V, const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
              const float* min_p, void* stream) {
  if (!tokens || !logits || !u || T <= 0 || V <= 0 || stride < V) return Q4_ERR_ARG;
  if (!known(logits_dtype)) return Q4_ERR_DTYPE;
  if (V > q4::sample_max_vocab() || T > (1 << 20) || stride > (1LL << 40)) return Q4_ERR_SHAPE;
  if (!aligned(logits, size_of(logits_dtype)) || !aligned(tokens, 4) || !aligned(probs, 4) || !aligned(u, 4) ||
      !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4))
    return Q4_ERR_ALIGN;
  q4::SampleParams p = {};
  p.tokens = tokens, p.probs = probs;
  p.logits = logits, p.stride = stride, p.bf16 = logits_dtype == Q4_BF16;
  p.T = static_cast<int>(T), p.V = static_cast<int>(V);
  p.u = u, p.temperature = temperature, p.top_k = top_k, p.top_p = top_p, p.min_p = min_p;
  return status_of(q4::launch_sample(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
