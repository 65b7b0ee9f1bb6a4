// Attention over keys of another length with a relative position bias
// (oases_attn.h): entry points, workspace, the bias by distance and its gradient.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <numeric>

#include "xattn.cuh"

namespace oases {
void api_begin();
oases_status api_end(cudaError_t e);

namespace {
using namespace xattn;

// ---- buckets --------------------------------------------------------------------
// A product a^na b^nb of two distances' powers: little end first, in as many words as it
// takes for a, b <= 65537 (17 bits each) and na + nb <= 64.  (No memory of the heap's: the
// entry points that come here throw nothing.)
struct Big {
  static constexpr int WORDS = 17 * 64 / 32;
  uint32_t d[WORDS] = {1};
  int n = 1;
  Big(uint32_t a, int na, uint32_t b, int nb) {
    for (int i = 0; i < na; ++i) times(a);
    for (int i = 0; i < nb; ++i) times(b);
  }
  void times(uint32_t m) {
    uint64_t c = 0;
    for (int i = 0; i < n; ++i) {
      c += (uint64_t)d[i] * m;
      d[i] = (uint32_t)c;
      c >>= 32;
    }
    if (c) d[n++] = (uint32_t)c;
  }
  bool operator<(const Big& o) const {
    if (n != o.n) return n < o.n;
    for (int i = n; i-- > 0;)
      if (d[i] != o.d[i]) return d[i] < o.d[i];
    return false;
  }
};

// Bucket E + u begins at the smallest whole number at or above x = E (max_distance / E)^(u / L).
// In doubles x comes from at most 63 products of one root, both off by some 2^-53 each: by
// less than 210 x 2^-53 x 65536 < 2e-9 in all.  Where no whole number is so near (1e-6 here),
// that decides; else whole arithmetic does, a^L against E^(L - u) max_distance^u with the
// exponents divided by what they have in common (where x is a whole number they are small).
// The check of a descriptor of 128 causal buckets takes 0.8 us on the host, one without a bias
// 0.6 (70 with every border decided by the powers in full).
Borders borders(int N, int max_distance) {
  Borders r;
  const int E = N / 2, L = N - E;
  r.n = N - 1;
  for (int t = 1; t <= E && t < N; ++t) r.at[t - 1] = t;
  const double root = pow((double)max_distance / E, 1.0 / L);
  double x = E;
  for (int u = 1; u < L; ++u) {
    x *= root;
    const double near = nearbyint(x);
    int a = (int)ceil(x);
    if (fabs(x - near) < 1e-6) {
      const int g = std::gcd(L, u);
      a = (int)near;
      if (Big(a, L / g, 1, 0) < Big(E, (L - u) / g, max_distance, u / g)) ++a;
    }
    r.at[E + u - 1] = a;
  }
  return r;
}

struct Shape {
  Args a = {};
  bool grad_f32 = false, accumulate = false;
  bool bidirectional = false;
  int per_sign = 0, R = 0;  // buckets of one sign; the distance from which the bucket stays
  Borders border = {};
};

bool strides_ok(const oases_strides& s, int64_t esize, int batch, int tokens, int heads, Strides* out) {
  const int64_t v[3] = {s.batch, s.token, s.head};
  const int n[3] = {batch, tokens, heads};
  const bool empty = batch == 0 || tokens == 0 || heads == 0;
  int64_t w[3];
  for (int i = 0; i < 3; ++i) {
    // not read: any that the tensor maps accept
    w[i] = n[i] > 1 && !empty ? v[i] : 16;
    if (w[i] <= 0 || w[i] > (1ll << 36) || w[i] * esize % 16 != 0) return false;
  }
  *out = {w[0], w[1], w[2]};
  return true;
}

oases_status shape(const oases_attn_desc* d, bool backward, Shape* s) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->batch < 0 || d->q_len < 0 || d->k_len < 0 || d->heads <= 0 || d->kv_heads <= 0 ||
      d->heads % d->kv_heads != 0 || d->head_dim <= 0 || d->q_start < 0)
    return OASES_ERR_INVALID_ARG;
  if (((d->causal | d->accumulate) & ~1) || !(d->scale > 0.f) || !(d->scale < INFINITY))
    return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  int N = 0;
  if (d->buckets != 0) {
    if (d->bidirectional & ~1) return OASES_ERR_INVALID_ARG;
    N = d->bidirectional ? d->buckets / 2 : d->buckets;
    if (N < 2 || (d->bidirectional && d->buckets % 2) || d->max_distance <= N / 2)
      return OASES_ERR_INVALID_ARG;
    if (d->buckets > MAX_BUCKETS || d->max_distance > 65536) return OASES_ERR_UNSUPPORTED;
  }
  if (d->head_dim % 8 != 0 || d->head_dim > 128) return OASES_ERR_UNSUPPORTED;
  constexpr int MOST = 1 << 24;
  if (std::max({d->q_len, d->k_len, d->q_start, d->heads}) > MOST || (int64_t)d->batch * d->heads > MOST)
    return OASES_ERR_UNSUPPORTED;
  Args& a = s->a;
  a.t = static_cast<DType>(d->dtype);
  const int64_t e = (int64_t)dtype_size(a.t);
  const int B = d->batch, Sq = d->q_len, Sk = d->k_len, H = d->heads, G = d->kv_heads;
  if (!strides_ok(d->q, e, B, Sq, H, &a.sq) || !strides_ok(d->k, e, B, Sk, G, &a.sk) ||
      !strides_ok(d->v, e, B, Sk, G, &a.sv) || !strides_ok(d->o, e, B, Sq, H, &a.so))
    return OASES_ERR_INVALID_ARG;
  if (backward && (!strides_ok(d->d_o, e, B, Sq, H, &a.sdo) || !strides_ok(d->dq, e, B, Sq, H, &a.sdq) ||
                   !strides_ok(d->dk, e, B, Sk, G, &a.sdk) || !strides_ok(d->dv, e, B, Sk, G, &a.sdv)))
    return OASES_ERR_INVALID_ARG;
  a.B = B, a.Sq = Sq, a.Sk = Sk, a.H = H, a.G = G, a.share = H / G, a.D = d->head_dim;
  a.causal = d->causal;
  a.q_start0 = d->q_start;
  a.scale = d->scale;
  a.splits = 1;
  a.q_pitch = (Sq + 127) / 128 * 128;
  s->grad_f32 = d->grad_dtype == OASES_F32;
  s->accumulate = d->accumulate != 0;
  if (N) {
    s->bidirectional = d->bidirectional != 0;
    s->per_sign = N;
    s->border = borders(N, d->max_distance);
    s->R = s->border.at[N - 2];
    a.bias.buckets = d->buckets;
    a.bias.R = s->R;
    a.bias.pitch = (2 * (s->R + BIAS_PAD) + 1 + 3) / 4 * 4;
    a.bias.left = N - 1;
    a.bias.right = s->bidirectional ? d->buckets - 1 : 0;
  }
  return OASES_OK;
}

// ---- the bias by distance ---------------------------------------------------------
// value[h][n + R + PAD] = factor * table[bucket(n)][h], and the run of distances of
// each bucket, and the bucket of each n.  A finite value stays finite behind the factor.
// (The heads along the grid's first dimension: the second ends at 65535.)
template <typename T>
__global__ void __launch_bounds__(256)
xattn_bias_kernel(const T* table, float* value, int2* range, uint8_t* index, const __grid_constant__ Borders border,
                  int heads, int pitch, int R, int buckets, int bidirectional, float factor) {
  pdl_wait();
  pdl_trigger();
  const int N = border.n + 1;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < buckets) {
    constexpr int FAR = 1 << 30;
    const int u = threadIdx.x % N;
    const int first = u == 0 ? 0 : border.at[u - 1], last = u + 1 < N ? border.at[u] - 1 : FAR;
    int2 r;
    if (bidirectional && threadIdx.x >= N)
      r = make_int2(max(first, 1), last);
    else
      r = make_int2(-last, !bidirectional && u == 0 ? FAR : -first);
    range[threadIdx.x] = r;
  }
  const int h = blockIdx.x, i = blockIdx.y * blockDim.x + threadIdx.x;
  if (i >= pitch) return;
  const int n = i - (R + BIAS_PAD);
  const int x = bidirectional ? abs(n) : max(-n, 0);
  const int bucket = border.bucket(x) + (bidirectional && n > 0 ? N : 0);
  if (h == 0 && abs(n) <= R) index[n + R] = (uint8_t)bucket;
  const float v = ld_elem(table, (int64_t)bucket * heads + h);
  float w = v * factor;
  if (fabsf(v) < INFINITY) w = fminf(fmaxf(w, -3.402823466e38f), 3.402823466e38f);
  value[(int64_t)h * pitch + i] = w;
}

// dbias[u][h] = the sum of the head's `rows` partial rows, in a fixed order.
__global__ void __launch_bounds__(1024)
xattn_bias_grad_kernel(const float* part, int64_t rows, int heads, int buckets, void* out, DType t,
                       int accumulate) {
  __shared__ float red[1024];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x;
  const int lanes = 1024 / buckets;  // rows at a time
  const int u = threadIdx.x % buckets, r0 = threadIdx.x / buckets;
  float v = 0.f;
  if (r0 < lanes)
#pragma unroll 8
    for (int64_t r = r0; r < rows; r += lanes) v += part[(h * rows + r) * buckets + u];
  red[threadIdx.x] = v;
  __syncthreads();
  if (r0 != 0) return;
  v = 0.f;
  for (int r = 0; r < lanes; ++r) v += red[r * buckets + u];
  const int64_t at = (int64_t)u * heads + h;
  if (accumulate) v += static_cast<const float*>(out)[at];
  store_any(out, t, at, v);
}

// ---- shares of the keys ---------------------------------------------------------------
// Where the forward has fewer items than the GPU has places for them, the keys are
// shared out, `least` blocks to a share at least.
int shares(int64_t items, int places, int blocks, int least) {
  if (items >= places || blocks < 2 * least) return 1;
  return (int)std::min<int64_t>(places / items, blocks / least);
}

// o = sum 2^.. of the shares' o, lse of all: a warp per query and head.
template <typename T>
__global__ void __launch_bounds__(256)
xattn_join_kernel(const __grid_constant__ Args a, int64_t rows) {
  pdl_wait();
  pdl_trigger();
  const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;  // (batch, query, head)
  if (r >= rows) return;
  const int lane = threadIdx.x % 32, h = (int)(r % a.H);
  const int64_t bq = r / a.H, b = bq / a.Sq;
  const int qi = (int)(bq - b * a.Sq);
  const int64_t at = a.stat((int)b, h, qi), step = (int64_t)a.B * a.H * a.Sq;
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_lse[s * step + at]);
  float sum = 0.f, v[4] = {};
  for (int s = 0; s < a.splits; ++s) {
    const float l = a.part_lse[s * step + at];
    if (l == -INFINITY) continue;  // a share without keys
    const float w = expf(l - top);
    sum += w;
    if (4 * lane < a.D) {
      const float4 x = *reinterpret_cast<const float4*>(a.part_o + (s * rows + r) * a.D + 4 * lane);
      v[0] = fmaf(w, x.x, v[0]), v[1] = fmaf(w, x.y, v[1]), v[2] = fmaf(w, x.z, v[2]), v[3] = fmaf(w, x.w, v[3]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* o = static_cast<T*>(a.o) + b * a.so.b + qi * a.so.s + h * a.so.h;
  if (4 * lane < a.D)
#pragma unroll
    for (int c = 0; c < 4; ++c) st_elem(o, 4 * lane + c, v[c] * inv);
  if (lane == 0) a.lse[at] = top + logf(sum);
}
cudaError_t join_splits(const Args& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.Sq * a.H;
  const dim3 grid((unsigned)((rows + 7) / 8));
  return a.t == DType::F32 ? launch_pdl(xattn_join_kernel<float>, grid, dim3(256), 0, st, a, rows)
                           : launch_pdl(xattn_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a, rows);
}

// ---- workspace ---------------------------------------------------------------------
struct Layout {
  size_t value = 0, range = 0, index = 0, delta = 0, part = 0, part_o = 0, part_lse = 0, total = 0;
  size_t neg_lse2 = 0, piece_dq = 0, piece_dkv = 0;
  int splits = 1;
  int64_t rows = 0;  // partial rows of the bias gradient, for each head
};
Layout layout(const Shape& s, bool backward) {
  Layout l;
  auto take = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += align256(bytes);
  };
  const Args& a = s.a;
  if (a.B == 0 || a.Sq == 0 || a.Sk == 0) return l;
  if (a.bias.buckets && (backward || !xattn_few_takes(a))) {
    take(&l.value, (size_t)a.H * a.bias.pitch * 4);
    take(&l.range, (size_t)a.bias.buckets * 8);
    take(&l.index, (size_t)2 * s.R + 1);
  }
  if (!backward) {
    const int sms = sm_count();
    if (xattn_few_takes(a))
      l.splits = xattn_few_splits(a);
    else if (a.t == DType::BF16)
      l.splits = shares((int64_t)a.B * a.H * ((a.Sq + 255) / 256), sms, (a.Sk + 127) / 128, 4);
    else
      l.splits = xattn_f32_cut(a).q_shares;
    if (l.splits > 1) {
      take(&l.part_o, (size_t)l.splits * a.B * a.Sq * a.H * a.D * 4);
      take(&l.part_lse, (size_t)l.splits * a.B * a.Sq * a.H * 4);
    }
  } else {
    take(&l.delta, (size_t)a.B * a.H * a.q_pitch * 4);
    if (a.t == DType::BF16) take(&l.neg_lse2, (size_t)a.B * a.H * a.q_pitch * 4);
    BwdCut cut;
    if (a.t == DType::F32) {
      const F32Cut c = xattn_f32_cut(a);
      if (c.q_shares > 1) take(&l.piece_dq, (size_t)c.q_shares * a.B * a.Sq * a.H * a.D * 4);
      if (c.kv_shares > 1) take(&l.piece_dkv, (size_t)c.kv_shares * 2 * a.B * a.Sk * a.G * a.D * 4);
      l.rows = (int64_t)a.B * ((a.Sq + c.q_rows - 1) / c.q_rows) * c.q_shares;
    } else if (xattn_bwd_cut(a, &cut)) {  // (else the call itself refuses)
      if (cut.dq.pieces > 1) take(&l.piece_dq, (size_t)cut.dq.rest * cut.dq.pieces * xattn_dq_piece_bytes(a.D));
      if (cut.dkv.pieces > 1) take(&l.piece_dkv, (size_t)cut.dkv.rest * cut.dkv.pieces * 2 * 128 * a.D * 4);
      const int64_t tiles = (int64_t)a.B * ((a.Sk + 127) / 128);  // as kv_item() counts them
      l.rows = (tiles + (tiles - cut.dkv.whole / a.G) * (cut.dkv.pieces - 1)) * DKV_WARPS;
    }
    if (a.bias.buckets) {
      take(&l.part, (size_t)l.rows * a.H * a.bias.buckets * 4);
    }
  }
  return l;
}

cudaError_t bias_tables(const Shape& s, const void* table, char* ws, const Layout& l, Bias* out,
                        float factor, cudaStream_t st) {
  const Bias& b = s.a.bias;
  *out = b;
  float* value = reinterpret_cast<float*>(ws + l.value);
  int2* range = reinterpret_cast<int2*>(ws + l.range);
  out->value = value;
  out->range = range;
  uint8_t* index = reinterpret_cast<uint8_t*>(ws + l.index);
  out->index = index;
  const dim3 grid(s.a.H, (b.pitch + 255) / 256);
  if (s.a.t == DType::F32)
    return launch_pdl(xattn_bias_kernel<float>, grid, dim3(256), 0, st, (const float*)table, value, range, index,
                      s.border, s.a.H, b.pitch, s.R, b.buckets, (int)s.bidirectional, factor);
  return launch_pdl(xattn_bias_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                    (const __nv_bfloat16*)table, value, range, index, s.border, s.a.H, b.pitch, s.R,
                    b.buckets, (int)s.bidirectional, factor);
}

// lse = -infinity of every query, where there are no keys at all
__global__ void xattn_fill_kernel(float* p, int64_t n, float v) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = v;
}

// A [tokens, heads, D] tensor of every sequence set to 0, 16 bytes at a time.
__global__ void xattn_zero_kernel(char* p, Strides s, int esize, int tokens, int heads, int chunks, int64_t n) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    int64_t r = i;
    const int64_t c = r % chunks;
    r /= chunks;
    const int64_t h = r % heads;
    r /= heads;
    const int64_t t = r % tokens, b = r / tokens;
    *reinterpret_cast<uint4*>(p + (b * s.b + t * s.s + h * s.h) * esize + c * 16) = make_uint4(0, 0, 0, 0);
  }
}
cudaError_t zero(void* p, const Strides& s, const Args& a, int tokens, int heads, cudaStream_t st) {
  const int e = (int)dtype_size(a.t), chunks = a.D * e / 16;
  const int64_t n = (int64_t)a.B * tokens * heads * chunks;
  if (n == 0) return cudaSuccess;
  return launch_pdl(xattn_zero_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, st,
                    static_cast<char*>(p), s, e, tokens, heads, chunks, n);
}

cudaError_t forward(Shape& s, const void* bias, char* ws, cudaStream_t st) {
  Args& a = s.a;
  if (a.Sk == 0) {
    const int64_t n = (int64_t)a.B * a.H * a.Sq;
    OASES_TRY(zero(a.o, a.so, a, a.Sq, a.H, st));
    return launch_pdl(xattn_fill_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, st,
                      a.lse, n, -INFINITY);
  }
  const Layout l = layout(s, false);
  const bool few = xattn_few_takes(a);
  if (a.bias.buckets && !few)
    OASES_TRY(bias_tables(s, bias, ws, l, &a.bias, a.t == DType::BF16 ? LOG2E : 1.f, st));
  a.splits = l.splits;
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + l.part_lse);
  OASES_TRY(few ? xattn_few(a, bias, s.border, s.bidirectional, st)
                : a.t == DType::BF16 ? xattn_fwd_tc(a, st) : xattn_fwd_f32(a, st));
  return a.splits > 1 ? join_splits(a, st) : cudaSuccess;
}

cudaError_t backward(Shape& s, const void* bias, void* dbias, char* ws, cudaStream_t st) {
  Args& a = s.a;
  const DType gt = s.grad_f32 ? DType::F32 : a.t;
  if (a.B == 0 || a.Sq == 0 || a.Sk == 0) {  // sums over nothing
    OASES_TRY(zero(a.dq, a.sdq, a, a.Sq, a.H, st));
    OASES_TRY(zero(a.dk, a.sdk, a, a.Sk, a.G, st));
    OASES_TRY(zero(a.dv, a.sdv, a, a.Sk, a.G, st));
    if (!dbias || s.accumulate) return cudaSuccess;
    return cudaMemsetAsync(dbias, 0, (size_t)a.bias.buckets * a.H * dtype_size(gt), st);
  }
  const Layout l = layout(s, true);
  if (a.bias.buckets) OASES_TRY(bias_tables(s, bias, ws, l, &a.bias, a.t == DType::BF16 ? LOG2E : 1.f, st));
  a.delta = reinterpret_cast<float*>(ws + l.delta);
  a.neg_lse2 = reinterpret_cast<float*>(ws + l.neg_lse2);
  a.bias_rows = l.rows;
  a.piece_dq = reinterpret_cast<float*>(ws + l.piece_dq);
  a.piece_dkv = reinterpret_cast<float*>(ws + l.piece_dkv);
  a.bias_part = dbias ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  OASES_TRY(a.t == DType::BF16 ? xattn_bwd_tc(a, st) : xattn_bwd_f32(a, st));
  if (!dbias) return cudaSuccess;
  return launch_pdl(xattn_bias_grad_kernel, dim3(a.H), dim3(1024), 0, st, (const float*)a.bias_part,
                    l.rows, a.H, a.bias.buckets, dbias, gt, (int)s.accumulate);
}

}  // namespace
}  // namespace oases

extern "C" size_t oases_attn_workspace_bytes(const oases_attn_desc* desc, int backward) {
  oases::Shape s;
  if (oases::shape(desc, backward != 0, &s) != OASES_OK) return 0;
  return oases::layout(s, backward != 0).total;
}

extern "C" oases_status oases_attn_fwd(const oases_attn_desc* desc, const void* q, const void* k,
                                       const void* v, const int32_t* kv_lens,
                                       const int32_t* q_start, const void* bias, void* o,
                                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  using namespace oases;
  api_begin();
  Shape s;
  const oases_status c = shape(desc, false, &s);
  if (c != OASES_OK) return c;
  if (misaligned({q, k, v, o, workspace}, 16) || misaligned({lse, kv_lens, q_start}, 4) ||
      misaligned({bias}, dtype_size(s.a.t)))
    return OASES_ERR_INVALID_ARG;
  if (s.a.B == 0 || s.a.Sq == 0) return OASES_OK;
  if (!q || !o || !lse || (s.a.Sk && (!k || !v)) || (s.a.bias.buckets && !bias) ||
      (!s.a.bias.buckets && bias))
    return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, false).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  s.a.q = q, s.a.k = k, s.a.v = v, s.a.o = o, s.a.lse = lse;
  s.a.kv_lens = kv_lens, s.a.q_start = q_start;
  return api_end(forward(s, bias, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
}

extern "C" oases_status oases_attn_bwd(const oases_attn_desc* desc, const void* q, const void* k,
                                       const void* v, const int32_t* kv_lens,
                                       const int32_t* q_start, const void* bias, const void* o,
                                       const float* lse, const void* d_o, void* dq, void* dk,
                                       void* dv, void* dbias, void* workspace, size_t ws_bytes,
                                       void* stream) {
  using namespace oases;
  api_begin();
  Shape s;
  const oases_status c = shape(desc, true, &s);
  if (c != OASES_OK) return c;
  const size_t ge = s.grad_f32 ? 4 : dtype_size(s.a.t);
  if (misaligned({q, k, v, o, d_o, dq, dk, dv, workspace}, 16) ||
      misaligned({lse, kv_lens, q_start}, 4) || misaligned({bias}, dtype_size(s.a.t)) ||
      misaligned({dbias}, ge))
    return OASES_ERR_INVALID_ARG;
  const bool rows = s.a.B > 0 && s.a.Sq > 0, keys = s.a.B > 0 && s.a.Sk > 0;
  if ((rows && (!q || !o || !lse || !d_o || !dq)) || (keys && (!k || !v || !dk || !dv)))
    return OASES_ERR_INVALID_ARG;
  if (rows && keys && !bias != !s.a.bias.buckets) return OASES_ERR_INVALID_ARG;
  if (dbias && !s.a.bias.buckets) return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, true).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  s.a.q = q, s.a.k = k, s.a.v = v, s.a.o = const_cast<void*>(o), s.a.lse = const_cast<float*>(lse);
  s.a.kv_lens = kv_lens, s.a.q_start = q_start;
  s.a.d_o = d_o, s.a.dq = dq, s.a.dk = dk, s.a.dv = dv;
  return api_end(backward(s, bias, dbias, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
}
