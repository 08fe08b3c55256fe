// loss.cu -- softmax cross entropy of a frozen head with the gradient of the
// hidden states (include/lora_loss.h; ch05 "Acceleration principles: Triton
// kernels and fused LoRA", §5.7): the C entry points and what stands around the
// two products of loss_gemm.cu.
//
//   k_loss_index    the tokens that count, in order, and the weights' sum
//   k_loss_gather   a strip of them: X's rows side by side, the target's logit
//   (first product) sums of exponentials relative to the target's
//   k_loss_rows     losses, each row's factor, the target's element of E
//   (second product), k_loss_join of its ranges; k_loss_mean or the join: the loss
//
// With every exponential relative to the target's own, a row's sum without the
// target is S = 1 / p_t - 1, the loss log1p(S) and the target's element of
// p - [v = t] is -S / (1 + S): no difference of near numbers, whether the target
// is nearly certain or hopeless.  The reference is the target's score in fp32
// arithmetic, known beforehand; the target's own exponential is that of its score in the
// product, as all others': the tensor cores cut off a little of a score at each 16
// products (5e-6 of it at a dim of 4096), which a difference of two scores hardly shows
// (with 1 for it, losses at scores of 30 were 1e-4 off).
#include <algorithm>
#include <climits>
#include <cmath>

#include "host.h"
#include "loss.cuh"
#include "lora_loss.h"
#include "ptx.cuh"

namespace lora {
namespace {

struct Tokens {
  const void *targets;
  int bits64;
  const float *weights;
  int64_t rows;
  __device__ __forceinline__ int64_t target(int64_t n) const {
    return bits64 ? static_cast<const int64_t *>(targets)[n]
                  : static_cast<int64_t>(static_cast<const int32_t *>(targets)[n]);
  }
};

// A sum as an unevaluated pair of fp32 (Knuth's exact sum of two numbers; fp64 is
// slow here: the mean of 2048 tokens took 9 us).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fadd_rn(s, -a.hi);
  const float err = __fadd_rn(__fadd_rn(a.hi, -__fadd_rn(s, -t)), __fadd_rn(b.hi, -t));
  const float lo = __fadd_rn(__fadd_rn(a.lo, b.lo), err);
  const float hi = __fadd_rn(s, lo);
  // (where the sum is not finite the error is not a number)
  return isfinite(hi) ? Pair{hi, __fadd_rn(lo, -__fadd_rn(hi, -s))} : Pair{s, 0.f};
}
// a b, with its rounding error.
__device__ __forceinline__ Pair times(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, isfinite(p) ? __fmaf_rn(a, b, -p) : 0.f};
}
// Over the block (of whole warps, 32 at most), the same in every thread, in a fixed
// order.
__device__ __forceinline__ Pair block_sum(Pair v, Pair *slot) {
  auto warp_sum = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      v = plus(v, Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  };
  warp_sum();
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const bool there = (threadIdx.x & 31) < blockDim.x >> 5;
  v = there ? slot[threadIdx.x & 31] : Pair{0.f, 0.f};
  warp_sum();
  return v;
}

// One block: eight tokens a thread at a time, their places by a scan.
__global__ void __launch_bounds__(1024) k_loss_index(Tokens tk, int mean, LossHead *head,
                                                     int *__restrict__ live,
                                                     float *__restrict__ losses) {
  __shared__ int counts[32];
  __shared__ Pair slot[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int done = 0;
  Pair sum = {0.f, 0.f};
  for (int64_t base = 0; base < tk.rows; base += 8192) {
    const int64_t n0 = base + threadIdx.x * 8;
    unsigned mask = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t n = n0 + j;
      if (n >= tk.rows) break;
      if (tk.target(n) >= 0) {
        mask |= 1u << j;
        if (tk.weights != nullptr) sum = plus(sum, Pair{tk.weights[n], 0.f});
      } else {
        losses[n] = 0.f;
      }
    }
    const int mine = __popc(mask);
    int before = mine;  // inclusive scan of the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    if (lane == 31) counts[warp] = before;
    __syncthreads();
    int c = counts[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += u;
    }
    const int all = __shfl_sync(0xffffffffu, c, 31);
    const int warps_before = __shfl_sync(0xffffffffu, c, warp > 0 ? warp - 1 : 0);
    int at = done + before - mine + (warp > 0 ? warps_before : 0);
    for (int j = 0; j < 8; ++j)
      if (mask >> j & 1u) live[at++] = static_cast<int>(n0 + j);
    done += all;
    __syncthreads();  // counts is free again
  }
  float divisor = 1.f;
  if (mean) {
    divisor = tk.weights != nullptr ? block_sum(sum, slot).hi : static_cast<float>(done);
    if (divisor == 0.f) divisor = 1.f;
  }
  if (threadIdx.x == 0) {
    head->live = done;
    head->divisor = divisor;
  }
}

struct Strip {
  const LossHead *head;
  const int *live;  // this strip's first
  int first, rows;  // place of the strip among the tokens that count; its room
  float *ref, *slope;
  float *scale;  // from the first product to k_loss_rows: the target's u
  int *target;
};

// Few tokens (1024 at most): each block of the gather finds the token of its place
// by itself, which saves the index's launch; the first writes what k_loss_index
// would have.  The token with rank `rank` among those that count (-1: there is none).
constexpr int kFewTokens = 1024;
__device__ __forceinline__ int64_t own_index(const Tokens &tk, int mean, int rank, LossHead *head,
                                             int *__restrict__ live, float *__restrict__ losses) {
  __shared__ int counts[8];
  __shared__ int found;
  __shared__ Pair slot[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first = blockIdx.x == 0;
  if (threadIdx.x == 0) found = -1;
  unsigned mask = 0;
  Pair sum = {0.f, 0.f};
  const int n0 = threadIdx.x * (kFewTokens / 256);
#pragma unroll
  for (int j = 0; j < kFewTokens / 256; ++j) {
    const int n = n0 + j;
    if (n >= tk.rows) continue;
    if (tk.target(n) >= 0) {
      mask |= 1u << j;
      if (first && mean && tk.weights != nullptr) sum = plus(sum, Pair{tk.weights[n], 0.f});
    } else if (first) {
      losses[n] = 0.f;
    }
  }
  const int mine = __popc(mask);
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += u;
  }
  if (lane == 31) counts[warp] = before;
  __syncthreads();
  int at = before - mine, all = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k < warp) at += counts[k];
    all += counts[k];
  }
#pragma unroll
  for (int j = 0; j < kFewTokens / 256; ++j)
    if (mask >> j & 1u) {
      if (at == rank) found = n0 + j;
      if (first) live[at] = n0 + j;
      ++at;
    }
  if (first) {
    float divisor = 1.f;
    if (mean) {
      divisor = tk.weights != nullptr ? block_sum(sum, slot).hi : static_cast<float>(all);
      if (divisor == 0.f) divisor = 1.f;
    }
    if (threadIdx.x == 0) {
      head->live = all;
      head->divisor = divisor;
    }
  }
  __syncthreads();
  return found;
}

// W warps a token of the strip: X's row copied beside the others, z = c(x . W_t) in fp32; and a line of
// zeros for each token that does not count among those at the strip's places.
template <int W, bool OWN>
__global__ void __launch_bounds__(256) k_loss_gather(Tokens tk, int mean, LossHead *head, int *all_live,
                                                     float *losses, Strip st,
                                                     const __nv_bfloat16 *__restrict__ w, int64_t ldw,
                                                     int64_t vocab, const __nv_bfloat16 *x,
                                                     int64_t ldx, __nv_bfloat16 *__restrict__ xs,
                                                     __nv_bfloat16 *dx, int64_t lddx, int dim,
                                                     float cap) {
  __shared__ float sums[8];
  griddep_wait();
  griddep_launch_dependents();
  constexpr int T = 32 * W;  // threads of a token
  const int lane = threadIdx.x % T;
  const int i = blockIdx.x * (8 / W) + threadIdx.x / T;
  const int64_t n0 = int64_t(st.first) + i;  // a token by its own number
  if (dx != nullptr && n0 < tk.rows && tk.target(n0) < 0) {
    uint4 *o = reinterpret_cast<uint4 *>(dx + n0 * lddx);
    for (int c = lane; c < dim / 8; c += T) o[c] = make_uint4(0u, 0u, 0u, 0u);
  }
  int64_t n;
  if constexpr (OWN) {
    static_assert(W == 8, "a block a token");
    n = own_index(tk, mean, st.first + i, head, all_live, losses);
    if (n < 0) return;
  } else {
    if (i >= st.rows || n0 >= st.head->live) return;  // the same in a token's threads
    n = st.live[i];
  }
  const int64_t t = tk.target(n);
  const bool known = t < vocab;
  const uint4 *xr = reinterpret_cast<const uint4 *>(x + n * ldx);
  const uint4 *wr = reinterpret_cast<const uint4 *>(w + (known ? t : 0) * ldw);
  uint4 *out = reinterpret_cast<uint4 *>(xs + int64_t(i) * dim);
  float s = 0.f;
#pragma unroll 4
  for (int c = lane; c < dim / 8; c += T) {
    const uint4 a = xr[c], b = wr[c];
    out[c] = a;
    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s = fmaf(__uint_as_float(p[j] << 16), __uint_as_float(q[j] << 16), s);
      s = fmaf(__uint_as_float(p[j] & 0xffff0000u), __uint_as_float(q[j] & 0xffff0000u), s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (W > 1) {
    static_assert(W == 1 || W == 8, "the block is one token's");
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += sums[k];
  }
  if (lane == 0) {
    float slope = 1.f;
    if (cap > 0.f) s = loss_cap(s, cap, 1.f / cap, slope);
    // (a target beyond the vocabulary makes its row NaN)
    st.ref[i] = known ? s * 1.4426950408889634f : NAN;
    st.slope[i] = slope;
    st.scale[i] = 0.f;  // (of a target beyond the vocabulary)
    st.target[i] = known ? static_cast<int>(t) : -1;
  }
}

// Eight tokens a block (32 left most SMs without one): a thread adds every 128th
// partial sum of one of them, eight on their way at once, then a warp joins a
// token's 128.
constexpr int kRowTokens = 8;
__global__ void __launch_bounds__(1024) k_loss_rows(Tokens tk, Strip st,
                                                    const LossPart *__restrict__ parts, int pieces,
                                                    __nv_bfloat16 *e, int64_t lde, int vocab,
                                                    float *__restrict__ losses) {
  constexpr int PER = 1024 / kRowTokens;
  __shared__ float sums[kRowTokens][PER + 1], ups[kRowTokens][PER + 1];
  __shared__ float far[kRowTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = blockIdx.x * kRowTokens;
  const int rows = min(st.rows, st.head->live - st.first);
  if (i0 >= rows) return;
  {
    float s = 0.f, m = 0.f;
    const int token = threadIdx.x % kRowTokens, from = threadIdx.x / kRowTokens;
    const LossPart *p = parts + i0 + token;
    constexpr int AHEAD = 8;
    for (int k = from; k < pieces; k += PER * AHEAD) {
      LossPart u[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        u[j] = k + PER * j < pieces ? p[int64_t(k + PER * j) * st.rows] : LossPart{0.f, 0.f};
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (u[j].up != m) {  // hardly ever: both are 0
          const float top = fmaxf(u[j].up, m);
          s *= exp2f(m - top);
          u[j].sum *= exp2f(u[j].up - top);
          m = top;
        }
        s += u[j].sum;
      }
    }
    sums[token][from] = s;
    ups[token][from] = m;
  }
  __syncthreads();
  const int i = i0 + warp;  // of the first warps: their token
  float s = 0.f, top = 0.f, u = 0.f;
  if (warp < kRowTokens) {
    // (where scores are so large that the target's two differ by more, a bound on it keeps
    // all finite)
    if (i < rows) u = st.scale[i];
    u = u < -60.f ? -60.f : u > 60.f ? 60.f : u;
#pragma unroll
    for (int k = 0; k < PER / 32; ++k) top = fmaxf(top, ups[warp][lane + 32 * k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int k = 0; k < PER / 32; ++k) {
      const float m = ups[warp][lane + 32 * k];
      s += m == top ? sums[warp][lane + 32 * k] : sums[warp][lane + 32 * k] * exp2f(m - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  const float own = exp2f(u - top), all = s + own;  // the target's, and with it
  if (lane == 0 && warp < kRowTokens) {
    far[warp] = i < rows ? top : 0.f;
    if (i < rows) {
      const int n = st.live[i];
      losses[n] = top == 0.f ? log1pf(s / own) : fmaf(top - u, 0.69314718055994531f, logf(all));
      if (e != nullptr) {
        const float g = (tk.weights != nullptr ? tk.weights[n] : 1.f) / st.head->divisor;
        st.scale[i] = g / all;
      }
    }
  }
  if (e == nullptr) return;
  __syncthreads();
  // Rows with an exponential beyond 2^64: the pieces that were kept on another
  // scale than the row's largest are brought to it (none, for all but rows whose
  // target is hopeless).
  for (int r = 0; r < kRowTokens; ++r) {
    if (far[r] == 0.f) continue;
    __nv_bfloat16 *row = e + int64_t(i0 + r) * lde;
    for (int c = threadIdx.x; c < vocab; c += 1024) {
      const float up = parts[int64_t(c / kLossPiece) * st.rows + i0 + r].up;
      if (up != far[r]) row[c] = __float2bfloat16_rn(__bfloat162float(row[c]) * exp2f(up - far[r]));
    }
  }
  __syncthreads();
  if (lane == 0 && warp < kRowTokens && i < rows && st.target[i] >= 0)
    e[int64_t(i) * lde + st.target[i]] = __float2bfloat16_rn(-s * st.slope[i]);
}

// loss = sum of w_n loss_n / divisor over the tokens that count, by one block.
__device__ __forceinline__ void mean_loss(const Tokens &tk, const LossHead *head,
                                          const int *__restrict__ live,
                                          const float *__restrict__ losses, float *__restrict__ loss,
                                          Pair *slot) {
  const int n = head->live;
  const float divisor = head->divisor;
  Pair s = {0.f, 0.f};
#pragma unroll 4
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int t = live[k];
    s = plus(s, times(losses[t], tk.weights != nullptr ? tk.weights[t] : 1.f));
  }
  s = block_sum(s, slot);
  if (threadIdx.x == 0) loss[0] = s.hi / divisor;
}
__global__ void __launch_bounds__(1024) k_loss_mean(Tokens tk, const LossHead *head,
                                                    const int *__restrict__ live,
                                                    const float *__restrict__ losses,
                                                    float *__restrict__ loss) {
  __shared__ Pair slot[32];
  griddep_wait();
  griddep_launch_dependents();
  mean_loss(tk, head, live, losses, loss, slot);
}

// Ranges of the second product -> dX: a block takes 32 rows and 32 columns of a cut
// tile, a thread four of them over all ranges (in their order, eight loads of each
// four on their way), and writes whole 64-byte pieces.  (64 columns a block left most
// SMs idle where there are few tiles and many ranges: 20 us for 31 ranges of 2
// tiles.)  The last block takes the mean loss, when the last strip's is there.
constexpr int JOIN_COLS = 32, JOIN_ROWS = 32, JOIN_HALF = kLossTileM / 2;  // rows of a CTA's half of a tile
__global__ void __launch_bounds__(256) k_loss_join(const __grid_constant__ LossGemm g, int pairs,
                                                   Tokens tk, const int *__restrict__ live,
                                                   const float *__restrict__ losses,
                                                   float *__restrict__ loss) {
  __shared__ float sums[JOIN_COLS][JOIN_ROWS + 1];
  __shared__ Pair mean_slot[8];
  griddep_wait();
  griddep_launch_dependents();
  const int joiners = gridDim.x - 1;
  if (static_cast<int>(blockIdx.x) == joiners) {
    if (loss != nullptr) mean_loss(tk, g.head, live, losses, loss, mean_slot);  // after the last strip
    return;
  }
  const int M = max(0, min(g.strip, g.head->live - g.first));
  const int m_pairs = (M + kLossTileM - 1) / kLossTileM, n_tiles = (g.n + kLossTileN - 1) / kLossTileN;
  const int kb = (g.k + kLossBlockK - 1) / kLossBlockK;
  const LossShare share = loss_share(m_pairs * n_tiles, pairs, kb);
  constexpr int PER_TILE = (kLossTileM / JOIN_ROWS) * (kLossTileN / JOIN_COLS);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int u = blockIdx.x; u < share.rest * PER_TILE; u += joiners) {
    const int tile = share.whole + u / PER_TILE;
    int slot = 0;
    const int ranges = loss_ranges(share, tile, slot);
    if (ranges < 2) return;  // none is cut
    const int part = u % PER_TILE, c0 = part % (kLossTileN / JOIN_COLS) * JOIN_COLS;
    const int r0 = part / (kLossTileN / JOIN_COLS) * JOIN_ROWS;  // of the tile's 256
    int mp, nb;
    loss_tile(tile, m_pairs, n_tiles, g.group, mp, nb);
    const int row0 = mp * kLossTileM + r0, col0 = nb * kLossTileN + c0;
    if (row0 >= M || col0 >= g.n) continue;  // the same in the whole block
    const float *in = g.slots + size_t(slot) * kLossSlotFloats + size_t(r0 / JOIN_HALF) * (JOIN_HALF * kLossTileN) +
                      size_t(c0) * JOIN_HALF + r0 % JOIN_HALF + lane;
    float s[JOIN_COLS / 8];
#pragma unroll
    for (int j = 0; j < JOIN_COLS / 8; ++j) s[j] = 0.f;
#pragma unroll 8
    for (int k = 0; k < ranges; ++k)
#pragma unroll
      for (int j = 0; j < JOIN_COLS / 8; ++j) s[j] += in[k * kLossSlotFloats + (j * 8 + w) * JOIN_HALF];
    const float f = row0 + lane < M ? g.scale[row0 + lane] : 0.f;
    __syncthreads();  // the last unit's sums are out
#pragma unroll
    for (int j = 0; j < JOIN_COLS / 8; ++j) sums[j * 8 + w][lane] = s[j] * f;
    __syncthreads();
    // eight threads a row, four columns each
    const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
    if (row0 + r < M && col0 + c < g.n)  // n is a multiple of 8
      *reinterpret_cast<uint2 *>(g.out + int64_t(g.place[row0 + r]) * g.ldo + col0 + c) =
          make_uint2(loss_pack(sums[c][r], sums[c + 1][r]), loss_pack(sums[c + 2][r], sums[c + 3][r]));
  }
}

__global__ void __launch_bounds__(256) k_loss_scale(const __nv_bfloat16 *dx, int64_t ldi,
                                                    const float *__restrict__ factor,
                                                    __nv_bfloat16 *out, int64_t ldo, int64_t rows,
                                                    int dim) {
  griddep_wait();
  griddep_launch_dependents();
  const float f = factor[0];
  const int64_t per = dim / 8, total = rows * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per, c = i - r * per;
    const uint4 v = reinterpret_cast<const uint4 *>(dx + r * ldi)[c];
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(u[j] << 16) * f,
                                                     __uint_as_float(u[j] & 0xffff0000u) * f);
      u[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint4 *>(out + r * ldo)[c] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ---------------------------------------------------------------- workspace
// A strip's exponentials (without dX its rows of X and sums) take at most kStripBytes, and
// all of it kStripMost; of 256 tokens at least.  (The second cuts heads of fewer than some four
// words a hidden element: 60000 x 4096 x 4096 into two, 2.79 ms where 2.74 in one of 1.1 GB.)
constexpr int64_t kStripBytes = int64_t(512) << 20, kStripMost = int64_t(640) << 20;

struct Plan {
  int strip = 0, pieces = 0, slots = 0;
  int64_t lde = 0;
  size_t head = 0, live = 0, xs = 0, ref = 0, slope = 0, scale = 0, target = 0, parts = 0, e = 0,
         ranges = 0, bytes = 0;
};
Plan make_plan(const lora_loss_t &sh, bool with_dx) {
  Plan p;
  p.lde = rup(sh.vocab, 8);
  p.pieces = static_cast<int>((sh.vocab + kLossTileN - 1) / kLossTileN * (kLossTileN / kLossPiece));
  const int64_t row = int64_t(p.pieces) * sizeof(LossPart) + sh.dim * 2 + 16;
  int64_t strip = with_dx ? std::min(kStripBytes / (p.lde * 2), kStripMost / (p.lde * 2 + row)) : kStripBytes / row;
  strip = strip / kLossTileM * kLossTileM;
  strip = strip < kLossTileM ? kLossTileM : strip > 65536 ? 65536 : strip;
  const int64_t all = rup(sh.rows > 0 ? sh.rows : 1, kLossTileM);
  p.strip = static_cast<int>(all < strip ? all : strip);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  p.head = take(sizeof(LossHead));
  p.live = take(size_t(sh.rows) * 4);
  p.xs = take(size_t(p.strip) * sh.dim * 2);
  p.ref = take(size_t(p.strip) * 4);
  p.slope = take(size_t(p.strip) * 4);
  p.scale = take(size_t(p.strip) * 4);
  p.target = take(size_t(p.strip) * 4);
  p.parts = take(size_t(p.pieces) * p.strip * sizeof(LossPart));
  if (with_dx) {
    p.e = take(size_t(p.strip) * p.lde * 2);
    const int64_t tiles = int64_t(p.strip / kLossTileM) * ((sh.dim + kLossTileN - 1) / kLossTileN);
    const int64_t ranges = (sh.vocab + 63) / 64 / 16;  // of a tile, at most (two where one is cut)
    const int64_t most = tiles * (ranges > 2 ? ranges : 2);
    p.slots = static_cast<int>(most < kLossSlots ? most : kLossSlots);
    p.ranges = take(size_t(p.slots) * kLossSlotFloats * sizeof(float));
  }
  p.bytes = at;
  return p;
}

lora_status_t check_shape(const lora_loss_t *sh) {
  if (sh == nullptr) return fail(LORA_ERR_INVALID_ARG, "shape is NULL");
  if (sh->rows < 0 || sh->vocab < 1 || sh->dim < 1)
    return fail(LORA_ERR_INVALID_ARG, "rows = %lld, vocab = %lld, dim = %d", (long long)sh->rows,
                (long long)sh->vocab, sh->dim);
  if (sh->rows > INT_MAX - 65536 || sh->vocab > INT_MAX - 511)
    return fail(LORA_ERR_UNSUPPORTED, "over 2^31 - 65537 rows, or a vocabulary over 2^31 - 512");
  if (sh->dim % 8 != 0 || sh->dim > 65536)
    return fail(LORA_ERR_UNSUPPORTED, "dim = %d is not a multiple of 8, at most 65536", sh->dim);
  if (sh->target_bits != 32 && sh->target_bits != 64)
    return fail(LORA_ERR_INVALID_ARG, "target_bits = %d is not 32 or 64", sh->target_bits);
  if ((sh->mean | 1) != 1) return fail(LORA_ERR_INVALID_ARG, "mean is 0 or 1");
  // (beyond these its inverse leaves fp32's normal numbers)
  if (sh->softcap != 0.f && !(sh->softcap >= 0x1p-100f && sh->softcap <= 0x1p100f))
    return fail(LORA_ERR_INVALID_ARG, "softcap = %g is not 0 or within 2^-100 .. 2^100", sh->softcap);
  return LORA_OK;
}
lora_status_t check_rows(const void *p, int64_t stride, int64_t rows, const lora_loss_t *sh,
                         const char *name) {
  LORA_TRY(check_ptr(p, name));
  if (rows > 1 && (stride < sh->dim || stride % 8 != 0))
    return fail(LORA_ERR_INVALID_ARG, "%s's row stride %lld is not a multiple of 8, at least dim", name,
                (long long)stride);
  return LORA_OK;
}
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A 2-D bf16 map with the 128-byte swizzle; what lies outside reads as zero.
lora_status_t map2d(CUtensorMap *tm, const void *ptr, int64_t inner, int64_t outer, int64_t pitch,
                    uint32_t box_inner, uint32_t box_outer, const char *what) {
  auto fn = encode_fn();
  if (!fn) return fail(LORA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
  cuuint32_t box[2] = {box_inner, box_outer}, es[2] = {1, 1};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims,
                        strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(LORA_ERR_CUDA, "tensor map for %s failed: CUresult %d", what, static_cast<int>(r));
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_loss_workspace_bytes(const lora_loss_t *sh, int with_dx) {
  clear_error();
  if (check_shape(sh) != LORA_OK) return 0;
  return make_plan(*sh, with_dx != 0).bytes;
}

lora_status_t lora_loss(const lora_loss_t *sh, const void *X, const void *W, const void *targets,
                        const float *weights, float *loss, float *losses, void *dX,
                        void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh));
  if (loss == nullptr || !aligned(loss, 4))
    return fail(LORA_ERR_INVALID_ARG, "loss is NULL or not aligned");
  if (sh->rows > 0) {
    LORA_TRY(check_rows(X, sh->x, sh->rows, sh, "X"));
    LORA_TRY(check_rows(W, sh->w, sh->vocab, sh, "W"));
    if (dX != nullptr) {
      LORA_TRY(check_rows(dX, sh->dx, sh->rows, sh, "dX"));
      if (dX == W || (dX == X && sh->rows > 1 && sh->dx != sh->x))
        return fail(LORA_ERR_INVALID_ARG, "dX is W, or X with another stride");
    }
    if (targets == nullptr || losses == nullptr)
      return fail(LORA_ERR_INVALID_ARG, "targets or losses is NULL");
    if (!aligned(targets, sh->target_bits / 8) || !aligned(losses, 4) || !aligned(weights, 4))
      return fail(LORA_ERR_INVALID_ARG, "targets, losses or weights is not aligned to its type");
    if (losses == weights) return fail(LORA_ERR_INVALID_ARG, "losses and weights are the same tensor");
  }
  const bool grad = dX != nullptr && sh->rows > 0;
  const Plan p = make_plan(*sh, grad);
  LORA_TRY(check_ws(workspace, workspace_bytes, p.bytes));
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Tokens tk = {targets, sh->target_bits == 64, weights, sh->rows};
  auto *head = reinterpret_cast<LossHead *>(at(workspace, p.head));
  int *live = reinterpret_cast<int *>(at(workspace, p.live));
  const bool own_index = sh->rows > 0 && sh->rows <= kFewTokens;
  if (!own_index)
    LORA_TRY(run(LORA_K_LOSS_PREP, st, "loss index", [&] {
      return launch_pdl(k_loss_index, dim3(1), dim3(1024), 0, st, tk, int(sh->mean), head, live, losses);
    }));
  const auto *x = static_cast<const __nv_bfloat16 *>(X), *w = static_cast<const __nv_bfloat16 *>(W);
  auto *xs = reinterpret_cast<__nv_bfloat16 *>(at(workspace, p.xs));
  auto *parts = reinterpret_cast<LossPart *>(at(workspace, p.parts));
  auto *e = grad ? reinterpret_cast<__nv_bfloat16 *>(at(workspace, p.e)) : nullptr;
  const int64_t ldx = sh->rows > 1 ? sh->x : sh->dim, ldw = sh->vocab > 1 ? sh->w : sh->dim;
  const int64_t lddx = sh->rows > 1 ? sh->dx : sh->dim;
  const int pairs = sh->rows > 0 ? loss_pairs(di.sms) : 0;
  for (int64_t first = 0; first < sh->rows; first += p.strip) {
    Strip s = {};
    s.head = head;
    s.live = live + first;
    s.first = static_cast<int>(first);
    s.rows = p.strip;
    s.ref = reinterpret_cast<float *>(at(workspace, p.ref));
    s.slope = reinterpret_cast<float *>(at(workspace, p.slope));
    s.scale = reinterpret_cast<float *>(at(workspace, p.scale));
    s.target = reinterpret_cast<int *>(at(workspace, p.target));
    LORA_TRY(run(LORA_K_LOSS_PREP, st, "loss gather", [&] {
      const int64_t here = sh->rows - first < p.strip ? sh->rows - first : p.strip;
      // (a warp a token: 16 us for 2048 of 4096 elements, 6 for 150 of 1000; a block: 10, 3)
      const bool wide = sh->dim >= 1024 || own_index;
      auto k = own_index ? k_loss_gather<8, true> : wide ? k_loss_gather<8, false> : k_loss_gather<1, false>;
      return launch_pdl(k, dim3(static_cast<unsigned>(wide ? here : (here + 7) / 8)), dim3(256), 0, st, tk,
                        int(sh->mean), head, live, losses, s, w, ldw, sh->vocab, x, ldx, xs, static_cast<__nv_bfloat16 *>(dX), lddx,
                        int(sh->dim), sh->softcap);
    }));
    LossGemm g;
    LORA_TRY(map2d(&g.a, xs, sh->dim, p.strip, sh->dim, 64, 128, "X"));
    LORA_TRY(map2d(&g.b, W, sh->dim, sh->vocab, ldw, 64, 128, "W"));
    if (grad)
      LORA_TRY(map2d(&g.e, e, sh->vocab, p.strip, p.lde, 64, 32, "exponentials"));
    else
      g.e = g.a;  // (not used)
    g.head = head;
    g.first = static_cast<int>(first);
    g.strip = p.strip;
    g.n = static_cast<int>(sh->vocab);
    g.k = sh->dim;
    g.group = 16;
    g.cap = sh->softcap;
    g.ref = s.ref;
    g.target = s.target;
    g.parts = parts;
    g.own = s.scale;
    g.dev_status = di.status;
    LORA_TRY(run(LORA_K_LOSS_LOGITS, st, "loss logits",
                 [&] { return launch_loss_gemm(grad ? 1 : 0, g, pairs, st); }));
    LORA_TRY(run(LORA_K_LOSS_ROWS, st, "loss rows", [&] {
      const int64_t here = sh->rows - first < p.strip ? sh->rows - first : p.strip;
      return launch_pdl(k_loss_rows, dim3(static_cast<unsigned>((here + kRowTokens - 1) / kRowTokens)), dim3(1024), 0, st, tk, s, parts, p.pieces, e,
                        p.lde, int(sh->vocab), losses);
    }));
    if (!grad) continue;
    LORA_TRY(map2d(&g.a, e, sh->vocab, p.strip, p.lde, 64, 128, "exponentials"));
    LORA_TRY(map2d(&g.b, W, sh->dim, sh->vocab, ldw, 64, 64, "W"));
    g.n = sh->dim;
    g.k = static_cast<int>(sh->vocab);
    g.scale = s.scale;
    g.place = s.live;
    g.out = static_cast<__nv_bfloat16 *>(dX);
    g.ldo = lddx;
    g.slots = reinterpret_cast<float *>(at(workspace, p.ranges));
    LORA_TRY(run(LORA_K_LOSS_GRAD, st, "loss gradient", [&] { return launch_loss_gemm(2, g, pairs, st); }));
    float *last = first + p.strip >= sh->rows ? loss : nullptr;
    LORA_TRY(run(LORA_K_LOSS_GRAD, st, "loss gradient join", [&] {
      return launch_pdl(k_loss_join, dim3(static_cast<unsigned>(di.sms * 8 + 1)), dim3(256), 0, st, g, pairs,
                        tk, live, losses, last);
    }));
  }
  if (grad) return LORA_OK;
  return run(LORA_K_LOSS_ROWS, st, "loss mean", [&] {
    return launch_pdl(k_loss_mean, dim3(1), dim3(1024), 0, st, tk, head, live, losses, loss);
  });
}

lora_status_t lora_loss_scale(const lora_loss_t *sh, const void *dX, const float *factor, void *out,
                              void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh));
  if (sh->rows == 0) return LORA_OK;
  LORA_TRY(check_rows(dX, sh->dx, sh->rows, sh, "dX"));
  LORA_TRY(check_rows(out, sh->x, sh->rows, sh, "out"));
  if (dX == out && sh->rows > 1 && sh->dx != sh->x)
    return fail(LORA_ERR_INVALID_ARG, "out is dX with another stride");
  if (factor == nullptr || !aligned(factor, 4))
    return fail(LORA_ERR_INVALID_ARG, "factor is NULL or not aligned");
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t want = (sh->rows * (sh->dim / 8) + 255) / 256, most = int64_t(di.sms) * 8;
  return run(LORA_K_LOSS_ROWS, st, "loss scale", [&] {
    return launch_pdl(k_loss_scale, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0,
                      st, static_cast<const __nv_bfloat16 *>(dX), sh->dx, factor,
                      static_cast<__nv_bfloat16 *>(out), sh->x, sh->rows, int(sh->dim));
  });
}

}  // extern "C"
