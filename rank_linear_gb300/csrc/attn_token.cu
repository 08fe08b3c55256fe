// attn_token.cu -- attention of one new token over a cache (include/lora_attention.h).
//
// Bound by HBM: the live part of K and V is read once for every eight query
// heads of a group, from global memory straight into the registers that
// mma.sync takes (no shared memory, no barrier in the loop).  What makes
// this work is that a dot product does not care about the order of its terms:
// the 16 bytes of a key that a lane loads are taken to be the elements that
// the MMA's layout wants there, and the query is laid out to match.
//
//   S^T[16 keys][8 heads] = K Q^T   a lane loads keys lane/4 and lane/4 + 8,
//     elements 32 c + 8 (lane % 4) + 0..7: the words of K steps 2c and 2c + 1.
//   O^T[dims][8 heads] += V^T P^T   a lane loads keys 2 (lane % 4) + {0, 1, 8, 9},
//     elements 64 e + 8 (lane / 4) + 0..7; word j of two keys, byte-permuted
//     into pairs of keys, is rows 2j and 2j + 1 of its eight.
//
// The keys of the next step are asked for before the present one's softmax, its
// values at the start of the step: with 3 blocks an SM (168 registers, a
// few words spilled) that keeps HBM busy.  (Measured and not kept: 4 blocks of 128
// registers 118 us for the ragged batch where 3 take 95; L2 prefetches 1 to 6
// steps ahead, values a step ahead in registers, all slower.)  131071 positions
// of one sequence, 8 key heads of 128: 83 us (6.5 TB/s, 0.95 of a copy); 32
// ragged ones up to 8192 long 97 us (6.1 TB/s).  That is with a cache that the
// longest sequence fills: chunks are cut from its capacity, so that in one much
// larger than its contents few blocks have work.
//
// P is transposed between the two by movmatrix.  The running maximum is
// followed only when some score exceeds it by 2^8 (a vote instead of
// shuffles); sums in fp32.  P is taken as the sum of two bf16 numbers, 16 bits
// of it, two MMAs: o is then off by its own rounding alone (0.0017 of its norm
// where P in one bf16 made it 0.0023), for 1.5 % of the time.
//
// The cache's length is cut into `splits` chunks; a second kernel joins their
// partial results in order.
#include "attn.cuh"
#include "host.h"

namespace lora {
namespace {

constexpr int kWarps = 4, kHeads = 8, kKeys = 16;  // keys of a warp's step
constexpr float kRescaleAt = 8.f;

struct Params {
  AttnArgs a;
  float2 *stat;  // [B][Hq][splits]: maximum (log2 units) and sum
  float *part;   // [B][Hq][splits][dim rounded up to 64], relative to that maximum
  int chunk, splits, head_chunks;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 load_if(bool there, const __nv_bfloat16 *p) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

template <int NB, bool CAP, bool BIAS>  // NB blocks of 64 elements of a head
__global__ void __launch_bounds__(32 * kWarps, 3) k_attn_token(const Params p) {
  const AttnArgs &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int quad = lane / 4, part = lane % 4;
  griddep_wait();
  griddep_launch_dependents();
  // neighbouring blocks take the key heads of the same keys, which lie side by
  // side in a [positions][heads] cache
  int id = blockIdx.x;
  const int g = id % a.Hk;
  id /= a.Hk;
  const int hc = id % p.head_chunks;
  id /= p.head_chunks;
  const int split = id % p.splits, b = id / p.splits;
  const int len = min(max(a.lengths[b], 0), a.Sk);
  const int from = split * p.chunk, to = min(from + p.chunk, len);
  const int h0 = g * a.group + hc * kHeads;               // the block's first head
  const int heads = min(kHeads, a.group - hc * kHeads);   // and how many
  if (from >= to && !(p.splits == 1)) return;

  // this lane's heads in S^T and O^T are h0 + 2 part and the next
  ScoreConst sc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) sc[i] = score_const(a, min(h0 + 2 * part + i, a.Hq - 1));

  // Q: head quad, elements 32 c + 8 part + 0..7
  uint4 q[2 * NB];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) {
    const int e = 32 * c + 8 * part;
    q[c] = load_if(quad < heads && e < a.D, static_cast<const __nv_bfloat16 *>(a.q) +
                                                b * a.sq[0] + (h0 + quad) * a.sq[2] + e);
  }
  const __nv_bfloat16 *kp =
      static_cast<const __nv_bfloat16 *>(a.k) + b * a.sk[0] + g * a.sk[2] + 8 * part;
  const __nv_bfloat16 *vp =
      static_cast<const __nv_bfloat16 *>(a.v) + b * a.sv[0] + g * a.sv[2] + 8 * quad;

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[4 * NB][4];
#pragma unroll
  for (int j = 0; j < 4 * NB; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  uint4 kw[2][2 * NB], vw[4][NB];
  auto load_k = [&](int key0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int key = key0 + quad + 8 * r;
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c)
        kw[r][c] = load_if(key < to && 32 * c + 8 * part < a.D, kp + key * a.sk[1] + 32 * c);
    }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = key0 + 2 * part + (r & 1) + (r >> 1) * 8;
#pragma unroll
      for (int e = 0; e < NB; ++e)
        vw[r][e] = load_if(key < to && 64 * e + 8 * quad < a.D, vp + key * a.sv[1] + 64 * e);
    }
  };

  constexpr int kStep = kWarps * kKeys;
  int key0 = from + warp * kKeys;
  if (key0 < to) load_k(key0);
  for (; key0 < to; key0 += kStep) {
    load_v(key0);
    float s[4] = {0.f, 0.f, 0.f, 0.f};  // keys quad, quad + 8 x heads 2 part, 2 part + 1
#pragma unroll
    for (int c = 0; c < 2 * NB; ++c) {
      const uint32_t lo[4] = {kw[0][c].x, kw[1][c].x, kw[0][c].y, kw[1][c].y};
      const uint32_t hi[4] = {kw[0][c].z, kw[1][c].z, kw[0][c].w, kw[1][c].w};
      mma_16816(s, lo, q[c].x, q[c].y);
      mma_16816(s, hi, q[c].z, q[c].w);
    }
    if (key0 + kStep < to) load_k(key0 + kStep);
    const bool small = !CAP || all_small<4>(sc[0], s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + quad + 8 * (i >> 1);
      const ScoreConst &c = sc[i & 1];
      if constexpr (CAP) {  // the polynomial of one score: its coefficients take no registers
        if (small) {
          const float x = s[i] * c.x_by, u = x * x;
          float p = tanh_poly(5);
#pragma unroll
          for (int j = 4; j >= 0; --j) p = fmaf(p, u, tanh_poly(j));
          s[i] = x * c.cap2 * p;
        } else {
          const float2 near = cap_near(c, make_float2(s[i], s[i]));
          s[i] = cap_any(c, s[i], cap_r(c, s[i]), near.x);
        }
      } else {
        s[i] *= c.scale2;
      }
      if constexpr (BIAS) s[i] = fmaf(-c.slope2, static_cast<float>(len - 1 - key), s[i]);
      if (key >= to) s[i] = -INFINITY;
    }
    float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
    if (__any_sync(~0u, top[0] > m[0] + kRescaleAt || top[1] > m[1] + kRescaleAt)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], x));
        const float m1 = fmaxf(m[i], top[i]);
        const float by = m[i] == -INFINITY ? 0.f : ex2(m[i] - m1);
        m[i] = m1;
        l[i] *= by;
#pragma unroll
        for (int j = 0; j < 4 * NB; ++j) {
          o[j][i] *= by;
          o[j][i + 2] *= by;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = ex2(s[i] - (m[i & 1] == -INFINITY ? 0.f : m[i & 1]));
      l[i & 1] += s[i];
    }
    // P as a sum of two bf16: the tensor core has time for both
    const uint32_t h0 = pack_bf16(s[0], s[1]), h1 = pack_bf16(s[2], s[3]);
    const uint32_t p0 = transpose_8x8(h0), p1 = transpose_8x8(h1);
    auto rest = [](uint32_t h, float x, float y) {
      return pack_bf16(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
    };
    const uint32_t r0 = transpose_8x8(rest(h0, s[0], s[1]));
    const uint32_t r1 = transpose_8x8(rest(h1, s[2], s[3]));
#pragma unroll
    for (int e = 0; e < NB; ++e) {
      const uint32_t w[4][4] = {{vw[0][e].x, vw[0][e].y, vw[0][e].z, vw[0][e].w},
                                {vw[1][e].x, vw[1][e].y, vw[1][e].z, vw[1][e].w},
                                {vw[2][e].x, vw[2][e].y, vw[2][e].z, vw[2][e].w},
                                {vw[3][e].x, vw[3][e].y, vw[3][e].z, vw[3][e].w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x[4] = {__byte_perm(w[0][j], w[1][j], 0x5410),
                               __byte_perm(w[0][j], w[1][j], 0x7632),
                               __byte_perm(w[2][j], w[3][j], 0x5410),
                               __byte_perm(w[2][j], w[3][j], 0x7632)};
        mma_16816(o[4 * e + j], x, p0, p1);
        mma_16816(o[4 * e + j], x, r0, r1);
      }
    }
  }

  // ---- the warps' results join in shared memory, in the order of the warps
  __shared__ float sm[kWarps][kHeads], sl[kWarps][kHeads];
  __shared__ float so[kWarps][kHeads][64 * NB + 4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int x = 4; x < 32; x *= 2) l[i] += __shfl_xor_sync(~0u, l[i], x);
    if (quad == 0) {
      sm[warp][2 * part + i] = m[i];
      sl[warp][2 * part + i] = l[i];
    }
  }
#pragma unroll
  for (int e = 0; e < NB; ++e)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float *to_row = &so[warp][2 * part + i][64 * e + 8 * quad];
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        *reinterpret_cast<float4 *>(to_row + 2 * j) =
            make_float4(o[4 * e + j][i], o[4 * e + j][i + 2], o[4 * e + j + 1][i],
                        o[4 * e + j + 1][i + 2]);
    }
  __syncthreads();
  for (int x = threadIdx.x; x < heads * 16 * NB; x += 32 * kWarps) {
    const int head = x / (16 * NB), e = x % (16 * NB) * 4;
    float top = sm[0][head];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w][head]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float by = sm[w][head] == -INFINITY ? 0.f : ex2(sm[w][head] - top);
      const float4 v = *reinterpret_cast<const float4 *>(&so[w][head][e]);
      sum = fmaf(by, sl[w][head], sum);
      acc.x = fmaf(by, v.x, acc.x);
      acc.y = fmaf(by, v.y, acc.y);
      acc.z = fmaf(by, v.z, acc.z);
      acc.w = fmaf(by, v.w, acc.w);
    }
    const int64_t row = static_cast<int64_t>(b) * a.Hq + h0 + head;
    if (p.splits == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (e < a.D)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + b * a.so[0] +
                                   (h0 + head) * a.so[2] + e) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    } else {
      if (e == 0) p.stat[row * p.splits + split] = make_float2(top, sum);
      *reinterpret_cast<float4 *>(p.part + (row * p.splits + split) * (64 * NB) + e) = acc;
    }
  }
}

// Joins the chunks of one head per block: a thread takes 4 elements of every
// lanes-th chunk, and the lanes' sums meet in shared memory in their order.
template <int NB>
struct Join {
  static constexpr int kCols = 16 * NB, kLanes = 512 / kCols;
};
template <int NB>
__global__ void __launch_bounds__(512) k_attn_token_join(const Params p) {
  constexpr int kCols = Join<NB>::kCols, kLanes = Join<NB>::kLanes;
  const AttnArgs &a = p.a;
  __shared__ float4 acc_s[kLanes][kCols];
  __shared__ float sum_s[kLanes], top_s[kLanes];
  const int y = threadIdx.x / kCols, x = threadIdx.x % kCols;
  const int h = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  griddep_wait();
  griddep_launch_dependents();
  const int len = min(max(a.lengths[b], 0), a.Sk);
  const int n = (len + p.chunk - 1) / p.chunk;
  const int64_t row = (static_cast<int64_t>(b) * a.Hq + h) * p.splits;
  // each lane relative to its own maximum
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 4;
  for (int i0 = y; i0 < n; i0 += U * kLanes) {
    float2 st[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kLanes;
      st[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        st[u] = __ldcg(&p.stat[row + i]);
        v[u] = __ldcg(reinterpret_cast<const float4 *>(p.part + (row + i) * (4 * kCols)) + x);
      }
    }
    float t1 = top;
#pragma unroll
    for (int u = 0; u < U; ++u) t1 = fmaxf(t1, st[u].x);
    const float keep = top == -INFINITY ? 0.f : ex2(top - t1);
    top = t1;
    sum *= keep;
    acc.x *= keep;
    acc.y *= keep;
    acc.z *= keep;
    acc.w *= keep;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float by = st[u].x == -INFINITY ? 0.f : ex2(st[u].x - top);
      sum = fmaf(by, st[u].y, sum);
      acc.x = fmaf(by, v[u].x, acc.x);
      acc.y = fmaf(by, v[u].y, acc.y);
      acc.z = fmaf(by, v[u].z, acc.z);
      acc.w = fmaf(by, v[u].w, acc.w);
    }
  }
  acc_s[y][x] = acc;
  if (x == 0) {
    sum_s[y] = sum;
    top_s[y] = top;
  }
  __syncthreads();
  if (y != 0 || 4 * x >= a.D) return;
#pragma unroll
  for (int i = 1; i < kLanes; ++i) top = fmaxf(top, top_s[i]);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const float by = top_s[i] == -INFINITY ? 0.f : ex2(top_s[i] - top);
    const float4 v = acc_s[i][x];
    sum = fmaf(by, sum_s[i], sum);
    acc.x = fmaf(by, v.x, acc.x);
    acc.y = fmaf(by, v.y, acc.y);
    acc.z = fmaf(by, v.z, acc.z);
    acc.w = fmaf(by, v.w, acc.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + b * a.so[0] + h * a.so[2] + 4 * x) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

template <int NB>
cudaError_t launch(const Params &p, cudaStream_t s) {
  const AttnArgs &a = p.a;
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  auto *kernel = cap ? (bias ? k_attn_token<NB, true, true> : k_attn_token<NB, true, false>)
                     : (bias ? k_attn_token<NB, false, true> : k_attn_token<NB, false, false>);
  const int64_t grid = int64_t(a.B) * a.Hk * p.head_chunks * p.splits;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), 0, s, p);
}

}  // namespace

// Chunks of the cache's length.  A GB300's 152 SMs hold 3 blocks each: enough
// chunks for two rounds of them, of 256 keys at the least where one round is
// full with those, else of 64 (a step of the block).  Measured, rounds 1 / 2 /
// 4 / 8: 80 / 83 / 87 / 95 us for one sequence of 131071 positions, 152 / 95 /
// 102 / 99 us for 32 ragged ones (the shortest a tenth of 8192), which leave
// blocks of one round without work.
AttnTokenPlan attn_token_plan(int64_t B, int64_t Hk, int group, int64_t Sk) {
  AttnTokenPlan t;
  t.head_chunks = (group + kHeads - 1) / kHeads;
  const int64_t rows = B * Hk * t.head_chunks, places = 152 * 3;
  auto chunk_of = [&](int64_t blocks) {
    const int64_t splits = rows > 0 && blocks > rows ? blocks / rows : 1;
    return (Sk + splits * 64 - 1) / (splits * 64) * 64;
  };
  int64_t chunk = chunk_of(2 * places);
  if (chunk < 256) chunk = chunk_of(places) < 256 ? chunk_of(places) : 256;
  t.chunk = static_cast<int>(chunk < 64 ? 64 : chunk);
  t.splits = static_cast<int>(Sk > 0 ? (Sk + t.chunk - 1) / t.chunk : 1);
  return t;
}

cudaError_t launch_attn_token(const AttnArgs &a, const AttnTokenPlan &t, void *stat, void *part,
                              cudaStream_t s) {
  const Params p{a, static_cast<float2 *>(stat), static_cast<float *>(part), t.chunk, t.splits,
                 t.head_chunks};
  return a.D <= 64 ? launch<1>(p, s) : launch<2>(p, s);
}
cudaError_t launch_attn_token_join(const AttnArgs &a, const AttnTokenPlan &t, void *stat,
                                   void *part, cudaStream_t s) {
  const Params p{a, static_cast<float2 *>(stat), static_cast<float *>(part), t.chunk, t.splits,
                 t.head_chunks};
  const dim3 grid(static_cast<unsigned>(int64_t(a.B) * a.Hq));
  return a.D <= 64 ? launch_pdl(k_attn_token_join<1>, grid, dim3(512), 0, s, p)
                   : launch_pdl(k_attn_token_join<2>, grid, dim3(512), 0, s, p);
}

}  // namespace lora
