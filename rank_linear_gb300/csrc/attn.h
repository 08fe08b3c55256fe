// attn.h -- arguments and launchers of the attention kernels.
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "internal.h"

namespace lora {

struct AttnArgs {
  int B = 0, Sq = 0, Sk = 0, Hq = 0, Hk = 0, D = 0, group = 1, causal = 0;
  float scale = 1.f, cap = 0.f;
  int64_t sq[3] = {}, sk[3] = {}, sv[3] = {}, so[3] = {};
  int64_t sdo[3] = {}, sdq[3] = {}, sdk[3] = {}, sdv[3] = {};
  const void *q = nullptr, *k = nullptr, *v = nullptr, *d_o = nullptr;
  void *o = nullptr, *dq = nullptr, *dk = nullptr, *dv = nullptr;
  float *lse = nullptr;
  // backward, [batch][q_heads][q_len rounded up to a tile]: -lse in log2 units
  // (-inf where nothing is seen, and past the end), and -do . o
  float *sub = nullptr, *neg_delta = nullptr;
  const float *slopes = nullptr;
  const int *q_docs = nullptr, *k_docs = nullptr, *prefix = nullptr, *lengths = nullptr;
  int64_t qds = 0, kds = 0;
  // documents of every 128-token tile ([batch][tiles] DocRange), with q_docs
  const int4 *q_ranges = nullptr, *k_ranges = nullptr;
  // with documents: counters (kAttnCounters, zeroed with the ranges) that the
  // persistent blocks take their items from
  unsigned *counter = nullptr;
  // with documents, backward: the key tiles ([batch][tiles] numbers) in the
  // order of falling work
  const int *order = nullptr;
  unsigned *dev_status = nullptr;
};
constexpr int kAttnCounters = 1;

// A [batch][token][head][dim] bf16 tensor's map: boxes of 64 elements x 128
// tokens of one head, 128-byte swizzle, zeros outside.
struct AttnMaps {
  CUtensorMap q, k, v;
};
struct AttnBwdMaps {
  CUtensorMap q, k, v, d_o;
};

// Forward: how the items (kQueries queries of a head) are shared out.  The first
// `rounds` rounds of whole items, one to a block, are handed out to and fro;
// what is left of the items, fewer than there are blocks, is cut along the
// keys: `tail` items in equal shares for `workers` blocks, each share part of
// one item or of two.  An item has up to `segments` parts, joined by a second
// launch.  tail = 0: nothing is cut.  shift > 0: an item's rows are 2^shift
// heads of a group, side by side for one query after the other (the map of q
// is then one of five dimensions).
struct AttnFwdPlan {
  int rounds = INT_MAX, tail = 0, workers = 0, segments = 0, shift = 0;
  bool special() const { return tail > 0 || shift > 0; }
};
constexpr int kAttnQueries = 256;
// The parts' maxima and sums (float2 [tail][segments][kAttnQueries]), and their
// outputs ([tail][segments][dim rounded up to 64 / 4][kAttnQueries] float4).
size_t attn_fwd_stat_bytes(const AttnFwdPlan &t);
size_t attn_fwd_part_bytes(const AttnFwdPlan &t, int D);
AttnFwdPlan attn_fwd_plan(int64_t B, int64_t Hq, int group, int64_t Sq, int64_t Sk, int D,
                          bool causal, bool prefix, bool docs);

// Ranges of the documents (and counters zeroed); then the order, if asked for.
cudaError_t launch_attn_ranges(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_order(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_fwd(const AttnArgs &a, const AttnMaps &m, const AttnFwdPlan &t, void *stat,
                            void *part, int sms, cudaStream_t s);
cudaError_t launch_attn_fwd_join(const AttnArgs &a, const AttnFwdPlan &t, const void *stat,
                                 const void *part, cudaStream_t s);
cudaError_t launch_attn_stats(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_dq(const AttnArgs &a, const AttnBwdMaps &m, int sms, cudaStream_t s);
cudaError_t launch_attn_dkv(const AttnArgs &a, const AttnBwdMaps &m, int sms, cudaStream_t s);

// One token: the cache's length in `splits` chunks of `chunk` keys, the heads
// of a group in head_chunks blocks; partial results of [batch][q_heads][splits]
// (maximum and sum: float2; output: dim rounded up to 64 floats), joined by the
// second launch where splits > 1.
struct AttnTokenPlan {
  int chunk = 64, splits = 1, head_chunks = 1;
};
AttnTokenPlan attn_token_plan(int64_t B, int64_t Hk, int group, int64_t Sk);
cudaError_t launch_attn_token(const AttnArgs &a, const AttnTokenPlan &t, void *stat, void *part,
                              cudaStream_t s);
cudaError_t launch_attn_token_join(const AttnArgs &a, const AttnTokenPlan &t, void *stat,
                                   void *part, cudaStream_t s);

}  // namespace lora
