// Attention over keys of another length with a relative position bias
// (oases_attn.h): what its kernels share.
#pragma once

#include "common.cuh"
#include "oases_attn.h"

namespace oases {
namespace xattn {

struct Strides {
  int64_t b, s, h;  // elements between sequences, tokens, heads
};

constexpr int MAX_BUCKETS = 128;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

// Of one sign's n + 1 buckets, the smallest distance of each but the first.
struct Borders {
  int n;
  int at[MAX_BUCKETS];
  // the bucket of distance x
  __host__ __device__ int bucket(int x) const {
    int lo = 0, hi = n;  // the number of borders at or below x
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (at[mid] <= x) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  }
};

// The bias by distance, written to the workspace by bias_tables(): for every head the
// values at n = -(R + PAD) .. R + PAD, where R is the distance from which the bucket no
// longer changes; the PAD places beyond repeat the ends, so that a tile that holds some
// |n| < R reads every one of its distances without clamping.
constexpr int BIAS_PAD = 320;
struct Bias {
  const float* value = nullptr;  // [heads][pitch], in units of log2(e) for the tensor-core kernels
  const int2* range = nullptr;   // [buckets]: the distances n of each bucket (first, last)
  const uint8_t* index = nullptr;  // the bucket of n = -R .. R
  int pitch = 0, R = 0, buckets = 0;
  int left = 0, right = 0;       // buckets of n <= -R and of n >= R
  __device__ __forceinline__ const float* at(int h, int n) const {  // |n| <= R + PAD
    return value + (int64_t)h * pitch + (R + BIAS_PAD) + n;
  }
  __device__ __forceinline__ float clamped(int h, int n) const { return *at(h, max(-R, min(R, n))); }
};

// Element-wise warps of the dk, dv kernel (bf16): each writes a partial row of the
// bias's gradient.
constexpr int DKV_WARPS = 16;

// A query whose lse lies below -2^20 gives no gradient: none of its keys counts (lse =
// -infinity), or all of its scores lie where fp32 no longer tells weights apart.  Nor does
// one whose lse lies above 2^24, where the roundings of s and of lse, in base 2 some 2.7
// together, make anything of e^(s - lse), infinity too.  (A NaN stays one.)
__device__ __forceinline__ bool beyond_weights(float lse) { return lse < -1048576.f || lse > 16777216.f; }

struct Args {
  const void *q, *k, *v;
  Strides sq, sk, sv, so, sdo, sdq, sdk, sdv;
  void* o;           // forward: output; backward: the forward's
  float* lse;        // [batch][heads][q_len]
  const void* d_o;
  void *dq, *dk, *dv;
  float* delta;      // workspace: fp32 [batch][heads][q_len]; bf16 -delta, and -lse in base 2,
  float* neg_lse2;   // [batch][heads][q_pitch]
  int q_pitch;       // q_len, rounded up to whole tiles
  const int *kv_lens, *q_start;
  int q_start0;
  int B, Sq, Sk, H, G, share, D, causal;
  DType t;
  float scale;
  Bias bias;
  float* bias_part;  // partial gradients of the bias [heads][bias_rows][buckets], null: not wanted
  int64_t bias_rows;
  float *piece_dq, *piece_dkv;  // sums of pieces of items or shares (backward), workspace
  int splits;        // forward: shares of the keys, joined by join_splits()
  float* part_o;     // [splits][batch][q_len][heads][D], normalised
  float* part_lse;   // [splits][batch][heads][q_len]

  // the first query's position of sequence b, and how many keys any of its queries sees: a
  // causal call over a cache leaves what stands behind its last query alone (0 times a NaN
  // there would be one)
  __device__ __forceinline__ int start(int b) const {
    return q_start ? max(-(1 << 28), min(1 << 28, q_start[b])) : q_start0;
  }
  __device__ __forceinline__ int len(int b) const {
    const int n = kv_lens ? max(0, min(Sk, kv_lens[b])) : Sk;
    return causal ? max(0, min(n, start(b) + Sq)) : n;
  }
  __device__ __forceinline__ int64_t stat(int b, int h, int i) const {
    return ((int64_t)b * H + h) * Sq + i;
  }
};

// Backward, bf16: items in whole rounds of the SMs, then `rest` items of `pieces` each.
struct Pieces {
  int whole, rest, pieces;
};
struct BwdCut {
  Pieces dq, dkv;
};
// fp32: rows of a tile, and the shares of the other side's blocks of the backward.
struct F32Cut {
  int q_rows, kv_rows, q_shares, kv_shares;
};

}  // namespace xattn

// forward of a few rows a key head, any type
bool xattn_few_takes(const xattn::Args& a);
int xattn_few_splits(const xattn::Args& a);
cudaError_t xattn_few(const xattn::Args& a, const void* table, const xattn::Borders& border,
                      bool bidirectional, cudaStream_t st);
// bf16, tensor cores
cudaError_t xattn_fwd_tc(const xattn::Args& a, cudaStream_t st);
size_t xattn_dq_piece_bytes(int D);
bool xattn_bwd_cut(const xattn::Args& a, xattn::BwdCut* cut);  // false: too many items
cudaError_t xattn_bwd_tc(const xattn::Args& a, cudaStream_t st);
// fp32 (CUDA cores)
xattn::F32Cut xattn_f32_cut(const xattn::Args& a);
cudaError_t xattn_fwd_f32(const xattn::Args& a, cudaStream_t st);
cudaError_t xattn_bwd_f32(const xattn::Args& a, cudaStream_t st);

}  // namespace oases
