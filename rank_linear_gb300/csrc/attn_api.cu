// attn_api.cu -- the entry points of include/lora_attention.h: argument
// checks, workspace layout and launches.
#include <cmath>

#include "attn.h"
#include "host.h"
#include "lora_attention.h"

namespace lora {
namespace {

constexpr int64_t kMaxLen = int64_t(1) << 24;

int64_t tiles_of(int64_t n) { return (n + 127) / 128; }

lora_status_t check_shape(const lora_attention_t *p) {
  if (p == nullptr) return fail(LORA_ERR_INVALID_ARG, "shape is NULL");
  if (p->batch < 0 || p->q_len < 0 || p->k_len < 0)
    return fail(LORA_ERR_INVALID_ARG, "batch, q_len or k_len is negative");
  if (p->q_heads < 1 || p->k_heads < 1 || p->q_heads % p->k_heads != 0)
    return fail(LORA_ERR_INVALID_ARG, "%d query heads over %d key heads", p->q_heads, p->k_heads);
  if (p->dim < 1) return fail(LORA_ERR_INVALID_ARG, "dim = %d", p->dim);
  if ((p->causal | 1) != 1) return fail(LORA_ERR_INVALID_ARG, "causal = %d is not 0 or 1", p->causal);
  if (!(p->scale > 0.f) || !std::isfinite(p->scale))
    return fail(LORA_ERR_INVALID_ARG, "scale must be finite and above 0");
  if (!(p->softcap >= 0.f) || !std::isfinite(p->softcap))
    return fail(LORA_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  if ((p->q_docs == nullptr) != (p->k_docs == nullptr))
    return fail(LORA_ERR_INVALID_ARG, "q_docs and k_docs are given together or not at all");
  if (p->prefix != nullptr && !p->causal)
    return fail(LORA_ERR_INVALID_ARG, "a prefix needs causal = 1");
  for (const void *x : {static_cast<const void *>(p->slopes), static_cast<const void *>(p->q_docs),
                        static_cast<const void *>(p->k_docs), static_cast<const void *>(p->prefix)})
    if (reinterpret_cast<uintptr_t>(x) % 4 != 0)
      return fail(LORA_ERR_INVALID_ARG, "slopes, documents or prefix is not 4-byte aligned");
  if (p->dim % 8 != 0 || p->dim > 128)
    return fail(LORA_ERR_UNSUPPORTED, "dim = %d: a multiple of 8 up to 128 is needed", p->dim);
  if (p->q_len >= kMaxLen || p->k_len >= kMaxLen)
    return fail(LORA_ERR_UNSUPPORTED, "q_len or k_len is 2^24 or more");
  if (p->batch > 65535 || p->q_heads > 65535 ||
      p->batch * p->q_heads * (p->q_len + p->k_len + 1) > (int64_t(1) << 33))
    return fail(LORA_ERR_UNSUPPORTED, "too many heads or rows for one launch");
  // Tiles of all heads are numbered in 32 bits, with room for the blocks' next
  // numbers past the end; a launch of the one-token form has at most a block
  // more for every 64 positions of a head, which is less than 2^27 (above).
  const int64_t longest = p->q_len > p->k_len ? p->q_len : p->k_len;
  if (p->batch * p->q_heads * (longest > 0 ? tiles_of(longest) : 1) > (int64_t(1) << 30))
    return fail(LORA_ERR_UNSUPPORTED, "more than 2^30 tiles of 128 tokens over all heads");
  return LORA_OK;
}

// A tensor of the op: its pointer, and the strides of the dimensions that have
// more than one entry (16-byte rows).  Only what is read with plain loads may
// be broadcast (stride 0): a tensor map's strides are not below its rows, and
// an output's entries have a place each.
enum Use { kLoaded, kMapped, kWritten };
lora_status_t check_tensor(const char *name, const void *p, const int64_t (&s)[3], int64_t batch,
                           int64_t len, int64_t heads, Use use) {
  const int64_t n[3] = {batch, len, heads};
  LORA_TRY(check_ptr(p, name, batch * len == 0));
  for (int i = 0; i < 3; ++i) {
    if (n[i] > 1 && (s[i] < 0 || s[i] % 8 != 0))
      return fail(LORA_ERR_UNSUPPORTED,
                  "%s: stride %lld is not a non-negative multiple of 8 elements", name,
                  (long long)s[i]);
    if (n[i] > 1 && s[i] == 0 && use != kLoaded)
      return fail(LORA_ERR_UNSUPPORTED, "%s is broadcast (stride 0): a tensor of its own is needed",
                  name);
  }
  return LORA_OK;
}

AttnArgs make_args(const lora_attention_t *p, const DevInfo &di) {
  AttnArgs a;
  a.B = static_cast<int>(p->batch);
  a.Sq = static_cast<int>(p->q_len);
  a.Sk = static_cast<int>(p->k_len);
  a.Hq = p->q_heads;
  a.Hk = p->k_heads;
  a.D = p->dim;
  a.group = p->q_heads / p->k_heads;
  a.causal = p->causal;
  a.scale = p->scale;
  a.cap = p->softcap;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = p->q[i];
    a.sk[i] = p->k[i];
    a.sv[i] = p->v[i];
    a.so[i] = p->o[i];
    a.sdo[i] = p->d_o[i];
    a.sdq[i] = p->dq[i];
    a.sdk[i] = p->dk[i];
    a.sdv[i] = p->dv[i];
  }
  a.slopes = p->slopes;
  a.q_docs = p->q_docs;
  a.k_docs = p->k_docs;
  a.qds = p->q_docs_stride;
  a.kds = p->k_docs_stride;
  a.prefix = p->prefix;
  a.dev_status = di.status;
  return a;
}

// Map of a [batch][token][head][dim] tensor (see AttnMaps).  An empty tensor
// gets a map over another's first row, which no copy reads.
lora_status_t tensor_map(CUtensorMap *tm, const void *p, const int64_t (&s)[3], const AttnArgs &a,
                         int len, int heads, const char *what) {
  auto fn = encode_fn();
  if (!fn) return fail(LORA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const uint64_t n[3] = {uint64_t(len), uint64_t(heads), uint64_t(a.B)};
  const int64_t by[3] = {s[1], s[2], s[0]};
  cuuint64_t dims[4] = {uint64_t(a.D), 1, 1, 1};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = n[i] > 0 ? n[i] : 1;
    strides[i] = n[i] > 1 ? uint64_t(by[i]) * 2 : uint64_t(a.D) * 2;
  }
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(LORA_ERR_CUDA, "tensor map for %s (strides %lld, %lld, %lld) failed: CUresult %d",
                what, (long long)s[0], (long long)s[1], (long long)s[2], static_cast<int>(r));
  return LORA_OK;
}

// Map of q with 2^shift heads of a token side by side: boxes of 64 elements x
// those heads x as many tokens as make 128 rows.
lora_status_t grouped_map(CUtensorMap *tm, const void *p, const int64_t (&s)[3], const AttnArgs &a,
                          int shift) {
  auto fn = encode_fn();
  if (!fn) return fail(LORA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int heads = 1 << shift;
  cuuint64_t dims[5] = {uint64_t(a.D), uint64_t(heads), uint64_t(a.Sq), uint64_t(a.Hq / heads),
                        uint64_t(a.B)};
  const int64_t by[4] = {s[2], s[1], s[2] * heads, s[0]};
  cuuint64_t strides[4];
  for (int i = 0; i < 4; ++i) strides[i] = uint64_t(dims[i + 1] > 1 ? by[i] : a.D) * 2;
  cuuint32_t box[5] = {64, uint32_t(heads), uint32_t(128 / heads), 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(p), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(LORA_ERR_CUDA, "tensor map for groups of q (strides %lld, %lld, %lld) failed: CUresult %d",
                (long long)s[0], (long long)s[1], (long long)s[2], static_cast<int>(r));
  return LORA_OK;
}

// Workspace: [document ranges of the query tiles, of the key tiles][item
// counters][order of the key tiles][statistics of the query rows, two]; the
// forward's [maxima and sums][outputs] of the parts of items it cuts.
struct Plan {
  size_t q_ranges = 0, k_ranges = 0, counter = 0, order = 0, sub = 0, neg_delta = 0, bytes = 0;
  AttnFwdPlan fwd;
  size_t stat = 0, part = 0;
};
Plan make_plan(const lora_attention_t *p, bool backward) {
  Plan w;
  size_t off = 0;
  if (p->q_docs != nullptr) {
    w.q_ranges = off;
    off += rup(size_t(p->batch) * tiles_of(p->q_len) * 16, 256);
    w.k_ranges = off;
    off += rup(size_t(p->batch) * tiles_of(p->k_len) * 16, 256);
    w.counter = off;
    off += 256;
    w.order = off;
    if (backward) off += rup(size_t(p->batch) * tiles_of(p->k_len) * 4, 256);
  }
  if (backward) {
    const size_t rows = size_t(p->batch) * p->q_heads * tiles_of(p->q_len) * 128;
    w.sub = off;
    off += rup(rows * 4, 256);
    w.neg_delta = off;
    off += rup(rows * 4, 256);
  } else {
    w.fwd = attn_fwd_plan(p->batch, p->q_heads, p->q_heads / p->k_heads, p->q_len, p->k_len, p->dim, p->causal != 0,
                          p->prefix != nullptr, p->q_docs != nullptr);
    w.stat = off;
    off += rup(attn_fwd_stat_bytes(w.fwd), 256);
    w.part = off;
    off += rup(attn_fwd_part_bytes(w.fwd, p->dim), 256);
  }
  w.bytes = off;
  return w;
}

// Workspace of the one-token form: [maximum and sum][output] of the chunks.
struct TokenSpace {
  AttnTokenPlan plan;
  size_t part = 0, bytes = 0;
};
TokenSpace make_token_space(const lora_attention_t *p) {
  TokenSpace w;
  w.plan = attn_token_plan(p->batch, p->k_heads, p->q_heads / p->k_heads, p->k_len);
  if (w.plan.splits > 1) {
    const size_t rows = size_t(p->batch) * p->q_heads * w.plan.splits;
    w.part = rup(rows * 8, 256);
    w.bytes = w.part + rows * (p->dim <= 64 ? 64 : 128) * 4;
  }
  return w;
}

lora_status_t make_ranges(AttnArgs &a, const Plan &w, void *ws, bool backward, cudaStream_t st) {
  if (a.q_docs == nullptr) return LORA_OK;
  a.q_ranges = reinterpret_cast<const int4 *>(at(ws, w.q_ranges));
  a.k_ranges = reinterpret_cast<const int4 *>(at(ws, w.k_ranges));
  a.counter = reinterpret_cast<unsigned *>(at(ws, w.counter));
  LORA_TRY(run(LORA_K_ATTN_PREP, st, "document ranges", [&] { return launch_attn_ranges(a, st); }));
  if (!backward || a.Sk == 0) return LORA_OK;
  a.order = reinterpret_cast<const int *>(at(ws, w.order));
  return run(LORA_K_ATTN_PREP, st, "key tiles by work", [&] { return launch_attn_order(a, st); });
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_attention_workspace_bytes(const lora_attention_t *shape, int backward) {
  clear_error();
  if (check_shape(shape) != LORA_OK) return 0;
  return make_plan(shape, backward != 0).bytes;
}

lora_status_t lora_attention_fwd(const lora_attention_t *shape, const void *q, const void *k,
                                 const void *v, void *o, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(shape));
  const bool no_q = shape->batch == 0 || shape->q_len == 0;
  const bool no_k = shape->batch == 0 || shape->k_len == 0;
  LORA_TRY(check_tensor("q", q, shape->q, shape->batch, shape->q_len, shape->q_heads, kMapped));
  LORA_TRY(check_tensor("k", k, shape->k, shape->batch, shape->k_len, shape->k_heads, kMapped));
  LORA_TRY(check_tensor("v", v, shape->v, shape->batch, shape->k_len, shape->k_heads, kMapped));
  LORA_TRY(check_tensor("o", o, shape->o, shape->batch, shape->q_len, shape->q_heads, kWritten));
  if (reinterpret_cast<uintptr_t>(lse) % 4 != 0)
    return fail(LORA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  const Plan w = make_plan(shape, false);
  LORA_TRY(check_ws(workspace, workspace_bytes, w.bytes));
  if (no_q) return LORA_OK;
  DevInfo di;
  LORA_TRY(device_info(di));
  AttnArgs a = make_args(shape, di);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnMaps m;
  LORA_TRY(w.fwd.special() ? grouped_map(&m.q, q, shape->q, a, w.fwd.shift)
                           : tensor_map(&m.q, q, shape->q, a, a.Sq, a.Hq, "q"));
  LORA_TRY(tensor_map(&m.k, no_k ? q : k, shape->k, a, a.Sk, a.Hk, "k"));
  LORA_TRY(tensor_map(&m.v, no_k ? q : v, shape->v, a, a.Sk, a.Hk, "v"));
  LORA_TRY(make_ranges(a, w, workspace, false, st));
  const bool cut = w.fwd.tail > 0;
  void *stat = cut ? at(workspace, w.stat) : nullptr, *part = cut ? at(workspace, w.part) : nullptr;
  LORA_TRY(run(LORA_K_ATTN_FWD, st, "attention forward",
               [&] { return launch_attn_fwd(a, m, w.fwd, stat, part, di.sms, st); }));
  if (!cut) return LORA_OK;
  return run(LORA_K_ATTN_FWD, st, "join of the attention forward",
             [&] { return launch_attn_fwd_join(a, w.fwd, stat, part, st); });
}

lora_status_t lora_attention_bwd(const lora_attention_t *shape, const void *d_o, const void *q,
                                 const void *k, const void *v, const void *o, const float *lse,
                                 void *dq, void *dk, void *dv, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(shape));
  const bool no_q = shape->batch == 0 || shape->q_len == 0;
  const bool no_k = shape->batch == 0 || shape->k_len == 0;
  LORA_TRY(check_tensor("do", d_o, shape->d_o, shape->batch, shape->q_len, shape->q_heads, kMapped));
  LORA_TRY(check_tensor("q", q, shape->q, shape->batch, shape->q_len, shape->q_heads, kMapped));
  LORA_TRY(check_tensor("k", k, shape->k, shape->batch, shape->k_len, shape->k_heads, kMapped));
  LORA_TRY(check_tensor("v", v, shape->v, shape->batch, shape->k_len, shape->k_heads, kMapped));
  LORA_TRY(check_tensor("o", o, shape->o, shape->batch, shape->q_len, shape->q_heads, kLoaded));
  LORA_TRY(check_tensor("dq", dq, shape->dq, shape->batch, shape->q_len, shape->q_heads, kWritten));
  LORA_TRY(check_tensor("dk", dk, shape->dk, shape->batch, shape->k_len, shape->k_heads, kWritten));
  LORA_TRY(check_tensor("dv", dv, shape->dv, shape->batch, shape->k_len, shape->k_heads, kWritten));
  if ((lse == nullptr && !no_q) || reinterpret_cast<uintptr_t>(lse) % 4 != 0)
    return fail(LORA_ERR_INVALID_ARG, "lse is NULL or not 4-byte aligned");
  const Plan w = make_plan(shape, true);
  LORA_TRY(check_ws(workspace, workspace_bytes, w.bytes));
  if (no_q && no_k) return LORA_OK;
  DevInfo di;
  LORA_TRY(device_info(di));
  AttnArgs a = make_args(shape, di);
  a.q = q;
  a.k = k;
  a.v = v;
  a.d_o = d_o;
  a.o = const_cast<void *>(o);
  a.lse = const_cast<float *>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.sub = reinterpret_cast<float *>(at(workspace, w.sub));
  a.neg_delta = reinterpret_cast<float *>(at(workspace, w.neg_delta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnBwdMaps m;
  LORA_TRY(tensor_map(&m.q, no_q ? k : q, shape->q, a, a.Sq, a.Hq, "q"));
  LORA_TRY(tensor_map(&m.d_o, no_q ? k : d_o, shape->d_o, a, a.Sq, a.Hq, "do"));
  LORA_TRY(tensor_map(&m.k, no_k ? q : k, shape->k, a, a.Sk, a.Hk, "k"));
  LORA_TRY(tensor_map(&m.v, no_k ? q : v, shape->v, a, a.Sk, a.Hk, "v"));
  LORA_TRY(make_ranges(a, w, workspace, true, st));
  if (!no_q)
    LORA_TRY(run(LORA_K_ATTN_PREP, st, "statistics of the rows",
                 [&] { return launch_attn_stats(a, st); }));
  if (!no_q)
    LORA_TRY(run(LORA_K_ATTN_DQ, st, "attention dq", [&] { return launch_attn_dq(a, m, di.sms, st); }));
  if (!no_k)
    LORA_TRY(run(LORA_K_ATTN_DKV, st, "attention dk and dv",
                 [&] { return launch_attn_dkv(a, m, di.sms, st); }));
  return LORA_OK;
}

size_t lora_attention_token_workspace_bytes(const lora_attention_t *shape) {
  clear_error();
  if (check_shape(shape) != LORA_OK) return 0;
  return make_token_space(shape).bytes;
}

lora_status_t lora_attention_token(const lora_attention_t *shape, const void *q, const void *k,
                                   const void *v, const int32_t *lengths, void *o,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(shape));
  if (shape->q_len != 1 || shape->causal || shape->q_docs != nullptr || shape->prefix != nullptr)
    return fail(LORA_ERR_INVALID_ARG, "one token: q_len = 1 and no causal, documents or prefix");
  const bool empty = shape->batch == 0;
  LORA_TRY(check_tensor("q", q, shape->q, shape->batch, shape->q_len, shape->q_heads, kLoaded));
  LORA_TRY(check_tensor("k", k, shape->k, shape->batch, shape->k_len, shape->k_heads, kLoaded));
  LORA_TRY(check_tensor("v", v, shape->v, shape->batch, shape->k_len, shape->k_heads, kLoaded));
  LORA_TRY(check_tensor("o", o, shape->o, shape->batch, shape->q_len, shape->q_heads, kWritten));
  if ((lengths == nullptr && !empty) || reinterpret_cast<uintptr_t>(lengths) % 4 != 0)
    return fail(LORA_ERR_INVALID_ARG, "lengths is NULL or not 4-byte aligned");
  const TokenSpace w = make_token_space(shape);
  LORA_TRY(check_ws(workspace, workspace_bytes, w.bytes));
  if (empty) return LORA_OK;
  DevInfo di;
  LORA_TRY(device_info(di));
  AttnArgs a = make_args(shape, di);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lengths = lengths;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *part = w.bytes > 0 ? at(workspace, w.part) : nullptr;
  LORA_TRY(run(LORA_K_ATTN_TOKEN, st, "attention of one token",
               [&] { return launch_attn_token(a, w.plan, workspace, part, st); }));
  if (w.plan.splits == 1) return LORA_OK;
  return run(LORA_K_ATTN_TOKEN, st, "join of one token's attention",
             [&] { return launch_attn_token_join(a, w.plan, workspace, part, st); });
}

}  // extern "C"
