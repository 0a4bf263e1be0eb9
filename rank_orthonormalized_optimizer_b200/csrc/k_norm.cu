// The norms around a block, fused with the block's gate and residual scale, and their
// gradients.
//
//   h = x + s gate * z,  z = post_gain * y rms(y)  (post norm)  or  z = y
//   u = pre_gain * h rms(h),   rms(v) = 1 / sqrt(mean(v^2) + eps)
//
// y is the block's output, x the residual stream, u the next block's input; u can be
// kept in 8 bits in the same pass (rows.cuh), from the fp32 u: one rounding.  Backward,
// with hn = h rms(h), yn = y rms(y), w = pre_gain du, c = s gate post_gain:
//
//   g  = dh + rms(h) (w - hn mean(w hn));          dx = g
//   dy = rms(y) (c g - yn mean(c g yn))            (s gate g without the post norm)
//   dpre_gain = sum_t du hn;  S = sum_t g yn (y without the post norm)
//   dpost_gain = s gate S;    dgate = s post_gain S     (one column sum gives both)
//
// Both passes are bound by HBM: every row is read once, held in registers between the row
// sums, and written once.  The forward pass takes a row per CTA (four rows, a warp each,
// up to 1024 features); the gains then come from L1, which the rows are loaded past.  The
// backward pass walks rows with a fixed grid and keeps each thread's column sums in
// registers; a second kernel adds the CTAs' partial sums in a fixed order, so results
// repeat bit for bit.  All sums are fp32; only the stored rows are rounded.
#include "operator.h"
#include "rows.cuh"

namespace dion {
namespace {

constexpr int64_t kMaxFeatures = 16384;  // a row stays in the registers of one CTA
constexpr int kWarpRows = 4;             // rows of a CTA in the warp-per-row form
constexpr int kParts = 296;              // backward: CTAs, and partial column sums, at most

struct NormP {
  const void *x, *y;
  void *h, *u;
  const float *pre, *post, *gate;
  uint8_t *q, *scale;
  int64_t ldx, ldy, ldh, ldu, ldq, tokens;
  int features;
  int post_norm;
  float eps, s, inv_d;
};

struct NormGradP {
  const void *h, *y, *du, *dh;
  void *dx, *dy;
  const float *pre, *post, *gate;
  float* parts;  // [grid][2][features]
  int64_t ldh, ldy, lddu, lddh, lddx, lddy, tokens;
  int features;
  int post_norm;
  float eps, s, inv_d;
};

// Sum of N values over the NT threads that share a row (a warp, or the whole CTA).
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (NT == 32) return;
  constexpr int W = NT / 32;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  __syncthreads();  // the last sum's readers are done
  if (l == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[w * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[k * N + i];
}

// Column of element e of this thread's row elements: groups of 8 where rows are 16-byte
// aligned (AL), single elements otherwise (32 lanes then hold 32 neighbouring columns).
template <int NT, bool AL>
__device__ __forceinline__ int column(int tid, int e) {
  return AL ? ((e / 8) * NT + tid) * 8 + (e % 8) : e * NT + tid;
}

template <typename T, int NT, int VPT, bool AL>
__device__ __forceinline__ void load_row(const T* p, int tid, int d, float* v) {
  if (AL) {
    Raw8<T> raw[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * NT + tid) * 8;
      raw[k] = c < d ? load_raw(p + c) : zero_raw<T>();
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) unpack(raw[k], v + 8 * k);
  } else {
#pragma unroll
    for (int e = 0; e < 8 * VPT; ++e) {
      const int c = e * NT + tid;
      v[e] = c < d ? to_float(p[c]) : 0.f;
    }
  }
}

template <typename T, int NT, int VPT, bool AL>
__device__ __forceinline__ void store_row(T* p, int tid, int d, const float* v) {
  if (AL) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * NT + tid) * 8;
      if (c < d) store8(p + c, v + 8 * k);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8 * VPT; ++e) {
      const int c = e * NT + tid;
      if (c < d) p[c] = from_float<T>(v[e]);
    }
  }
}

// Eight gains from column c (1 where there is no array).
template <bool AL>
__device__ __forceinline__ void gains8(const float* g, int c, int d, float* v) {
  if (g && c + 7 < d) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(g + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(g + c + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.f;
  }
}
template <int NT, bool AL>
__device__ __forceinline__ void gains(const float* g, int tid, int k, int d, float* v) {
  if (AL) {
    gains8<AL>(g, (k * NT + tid) * 8, d, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<NT, AL>(tid, 8 * k + j);
      v[j] = g && c < d ? __ldg(g + c) : 1.f;
    }
  }
}

template <typename T, int NT, int VPT, bool AL>
__global__ void __launch_bounds__(NT == 32 ? 32 * kWarpRows : NT) k_norm(const NormP p) {
  constexpr int E = 8 * VPT;
  __shared__ float red[NT == 32 ? 1 : NT / 32];
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = NT == 32 ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.tokens) return;  // a whole warp, in the form without block barriers only
  const int d = p.features;
  float h[E];
  load_row<T, NT, VPT, AL>(static_cast<const T*>(p.x) + row * p.ldx, tid, d, h);
  if (p.y) {
    float y[E];
    load_row<T, NT, VPT, AL>(static_cast<const T*>(p.y) + row * p.ldy, tid, d, y);
    float f = p.s;
    if (p.post_norm) {
      float ss[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) ss[0] = fmaf(y[e], y[e], ss[0]);
      row_sum<NT, 1>(ss, red);
      f *= rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float a[8], b[8];
      gains<NT, AL>(p.post, tid, k, d, a);
      gains<NT, AL>(p.gate, tid, k, d, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[8 * k + j] = fmaf(a[j] * b[j], y[8 * k + j] * f, h[8 * k + j]);
    }
    if (p.h) store_row<T, NT, VPT, AL>(static_cast<T*>(p.h) + row * p.ldh, tid, d, h);
  }
  if (!p.u) return;
  float ss[1] = {0.f};
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (column<NT, AL>(tid, e) < d) ss[0] = fmaf(h[e], h[e], ss[0]);
  row_sum<NT, 1>(ss, red);
  const float r = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float a[8];
    gains<NT, AL>(p.pre, tid, k, d, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[8 * k + j] = a[j] * (h[8 * k + j] * r);
  }
  store_row<T, NT, VPT, AL>(static_cast<T*>(p.u) + row * p.ldu, tid, d, h);
  if (!p.q) return;
  uint8_t* q = p.q + row * p.ldq;
  uint8_t* scale = p.scale + row * (p.ldq / 32);
  if (AL) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * NT + tid) * 8;
      if (c >= d)  // the row's end inside the vector, and the padding of its last block
#pragma unroll
        for (int j = 0; j < 8; ++j) h[8 * k + j] = 0.f;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, abs_bits(h[8 * k + j]));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (c >= p.ldq) continue;
      const int e = act_exponent(top);
      const float f = act_unscale(e);
      const bool fine = top < kInfBits;
      uint2 o = make_uint2(0, 0);
      const float* v = h + 8 * k;
      if (fine) {
        o.x = e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16;
        o.y = e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16;
      }
      *reinterpret_cast<uint2*>(q + c) = o;
      if ((tid & 3) == 0) scale[c / 32] = fine ? e + 127 : 255;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = column<NT, AL>(tid, e);
      const float v = c < d ? h[e] : 0.f;
      const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(v));
      if (c >= p.ldq) continue;
      const int x = act_exponent(top);
      const bool fine = top < kInfBits;
      q[c] = fine ? (uint8_t)e4m3x2(v * act_unscale(x), 0.f) : 0;
      if ((tid & 31) == 0) scale[c / 32] = fine ? x + 127 : 255;
    }
  }
}

template <typename T, int NT, int VPT, bool AL>
__global__ void __launch_bounds__(NT == 32 ? 32 * kWarpRows : NT) k_norm_grad(const NormGradP p) {
  constexpr int E = 8 * VPT;
  constexpr int RPC = NT == 32 ? kWarpRows : 1;
  __shared__ float red[NT == 32 ? 1 : 3 * NT / 32];
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int sub = NT == 32 ? threadIdx.x >> 5 : 0;
  const int d = p.features;
  float apre[E], apost[E];
#pragma unroll
  for (int e = 0; e < E; ++e) apre[e] = apost[e] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * RPC + sub; row < p.tokens; row += (int64_t)gridDim.x * RPC) {
    float h[E], g[E], w[E], y[E];  // w: du; g: dh, then the gradient of h
    float sum[3] = {0.f, 0.f, 0.f};
    if (p.dh) {
      load_row<T, NT, VPT, AL>(static_cast<const T*>(p.dh) + row * p.lddh, tid, d, g);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = 0.f;
    }
    if (p.du) {
      load_row<T, NT, VPT, AL>(static_cast<const T*>(p.h) + row * p.ldh, tid, d, h);
      load_row<T, NT, VPT, AL>(static_cast<const T*>(p.du) + row * p.lddu, tid, d, w);
    }
    if (p.y) load_row<T, NT, VPT, AL>(static_cast<const T*>(p.y) + row * p.ldy, tid, d, y);
    if (p.du) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float a[8];
        gains<NT, AL>(p.pre, tid, k, d, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * k + j;
          sum[0] = fmaf(h[e], h[e], sum[0]);
          sum[1] = fmaf(a[j] * w[e], h[e], sum[1]);
        }
      }
    }
    if (p.y && p.post_norm)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[2] = fmaf(y[e], y[e], sum[2]);
    row_sum<NT, 3>(sum, red);
    if (p.du) {
      const float r = rsqrtf(fmaf(sum[0], p.inv_d, p.eps));
      const float m1 = sum[1] * r * p.inv_d;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float a[8];
        gains<NT, AL>(p.pre, tid, k, d, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * k + j;
          const float hn = h[e] * r;
          apre[e] = fmaf(w[e], hn, apre[e]);
          g[e] = fmaf(r, fmaf(-hn, m1, a[j] * w[e]), g[e]);
        }
      }
    }
    if (p.dx) store_row<T, NT, VPT, AL>(static_cast<T*>(p.dx) + row * p.lddx, tid, d, g);
    if (!p.y) continue;
    const float ry = p.post_norm ? rsqrtf(fmaf(sum[2], p.inv_d, p.eps)) : 1.f;
    float dot[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float a[8], b[8];
      gains<NT, AL>(p.post, tid, k, d, a);
      gains<NT, AL>(p.gate, tid, k, d, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = 8 * k + j;
        y[e] *= ry;
        apost[e] = fmaf(g[e], y[e], apost[e]);
        g[e] *= p.s * a[j] * b[j];
        dot[0] = fmaf(g[e], y[e], dot[0]);
      }
    }
    if (p.post_norm) {
      row_sum<NT, 1>(dot, red);
      const float m2 = dot[0] * p.inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = ry * fmaf(-y[e], m2, g[e]);
    }
    if (p.dy) store_row<T, NT, VPT, AL>(static_cast<T*>(p.dy) + row * p.lddy, tid, d, g);
  }
  // this CTA's column sums; in the warp-per-row form the warps add theirs in order
  float* part = p.parts + (int64_t)blockIdx.x * 2 * d;
  for (int turn = 0; turn < RPC; ++turn) {
    if (sub == turn) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = column<NT, AL>(tid, e);
        if (c < d) {
          part[c] = (turn ? part[c] : 0.f) + apre[e];
          part[d + c] = (turn ? part[d + c] : 0.f) + apost[e];
        }
      }
    }
    if (RPC > 1) __syncthreads();
  }
}

struct GainP {
  const float* parts;
  int nparts, features;
  const float *post, *gate;
  float *dpre, *dpost, *dgate;
  float s;
  int accumulate;
};

// Adds the CTAs' partial sums of 32 columns: eight warps take every eighth part, and the
// eight sums are added in order.
__global__ void __launch_bounds__(256) k_norm_gains(const GainP p) {
  __shared__ float sh[2][8][32];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + l;
  float a = 0.f, b = 0.f;
  if (c < p.features) {
    for (int k = w; k < p.nparts; k += 8) {
      const float* part = p.parts + (int64_t)k * 2 * p.features + c;
      a += part[0];
      b += part[p.features];
    }
  }
  sh[0][w][l] = a;
  sh[1][w][l] = b;
  __syncthreads();
  if (w != 0 || c >= p.features) return;
  a = b = 0.f;
  for (int k = 0; k < 8; ++k) {
    a += sh[0][k][l];
    b += sh[1][k][l];
  }
  const float gate = p.gate ? p.gate[c] : 1.f, post = p.post ? p.post[c] : 1.f;
  if (p.dpre) p.dpre[c] = (p.accumulate ? p.dpre[c] : 0.f) + a;
  if (p.dpost) p.dpost[c] = (p.accumulate ? p.dpost[c] : 0.f) + p.s * gate * b;
  if (p.dgate) p.dgate[c] = (p.accumulate ? p.dgate[c] : 0.f) + p.s * post * b;
}

// Threads of a row and 8-element vectors of a thread, by the features: a warp up to 1024,
// then the smallest CTA that holds the row in two vectors a thread, four at the widest.
template <typename F>
void by_width(int64_t d, F f) {
  if (d <= 256) f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  else if (d <= 512) f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  else if (d <= 1024) f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
  else if (d <= 2048) f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  else if (d <= 4096) f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  else if (d <= 8192) f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
}

template <typename T>
void launch_norm(const NormP& p, bool al, cudaStream_t s) {
  by_width(p.features, [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    const unsigned grid = (unsigned)(NT == 32 ? (p.tokens + kWarpRows - 1) / kWarpRows : p.tokens);
    const unsigned threads = NT == 32 ? 32 * kWarpRows : NT;
    if (al) k_norm<T, NT, VPT, true><<<grid, threads, 0, s>>>(p);
    else k_norm<T, NT, VPT, false><<<grid, threads, 0, s>>>(p);
  });
}

template <typename T>
void launch_grad(const NormGradP& p, bool al, unsigned grid, cudaStream_t s) {
  by_width(p.features, [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    const unsigned threads = NT == 32 ? 32 * kWarpRows : NT;
    if (al) k_norm_grad<T, NT, VPT, true><<<grid, threads, 0, s>>>(p);
    else k_norm_grad<T, NT, VPT, false><<<grid, threads, 0, s>>>(p);
  });
}

unsigned grad_grid(int64_t tokens, int64_t features) {
  const int64_t rows = features <= 1024 ? (tokens + kWarpRows - 1) / kWarpRows : tokens;
  return (unsigned)(rows < kParts ? rows : kParts);
}

dion_status check_norm(int64_t tokens, int64_t features, int32_t dtype, float eps, float s) {
  if (!valid_dtype(dtype)) return set_error(DION_ERR_INVALID_ARG, "dtype %d is not a dion_dtype", dtype);
  const dion_status st = check_tokens(tokens);
  if (st != DION_OK) return st;
  if (features < 1 || features > kMaxFeatures)
    return set_error(DION_ERR_UNSUPPORTED_SHAPE, "features %lld outside [1, %lld]",
                     (long long)features, (long long)kMaxFeatures);
  if (!(eps > 0.f) || !std::isfinite(eps))
    return set_error(DION_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!std::isfinite(s)) return set_error(DION_ERR_INVALID_ARG, "residual_scale is not finite");
  return DION_OK;
}

dion_status check_gain(const char* name, const void* g) {
  if (g && !aligned_to(g, 4))
    return set_error(DION_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
  return DION_OK;
}

#define DION_TRY(call)                                 \
  do {                                                 \
    const dion_status st_ = (call);                    \
    if (st_ != DION_OK) return st_;                    \
  } while (0)

dion_status norm_impl(const dion_norm* a, void* stream) {
  if (!a) return set_error(DION_ERR_INVALID_ARG, "args is NULL");
  DION_TRY(check_norm(a->tokens, a->features, a->dtype, a->eps, a->residual_scale));
  const int64_t es = dtype_bytes(a->dtype);
  // an empty array's pointer may be NULL, so which rows are given says nothing without tokens
  if (a->tokens > 0) {
    if (!a->y && (a->h || a->post_gain || a->gate || a->post_norm))
      return set_error(DION_ERR_INVALID_ARG, "h, post_norm, post_gain and gate need y");
    if (a->post_gain && !a->post_norm)
      return set_error(DION_ERR_INVALID_ARG, "post_gain needs post_norm");
    if (!a->u && (!a->y || a->pre_gain || a->kept))
      return set_error(DION_ERR_INVALID_ARG, a->y ? "pre_gain and kept need u" : "neither y nor u: nothing to do");
    if (a->y && !a->h && !a->u) return set_error(DION_ERR_INVALID_ARG, "neither h nor u: nothing to write");
  }
  DION_TRY(check_gain("pre_gain", a->pre_gain));
  DION_TRY(check_gain("post_gain", a->post_gain));
  DION_TRY(check_gain("gate", a->gate));
  if (a->kept) {
    DION_TRY(check_kept(*a->kept));
    if (a->kept->tokens != a->tokens || a->kept->features != a->features)
      return set_error(DION_ERR_INVALID_ARG, "kept has another shape than the rows");
  }
  bool al = a->features % 8 == 0;
  struct { const char* name; const void* p; int64_t ld; bool need; } rows[] = {
      {"x", a->x, a->ldx, true}, {"y", a->y, a->ldy, a->y != nullptr},
      {"h", a->h, a->ldh, a->h != nullptr}, {"u", a->u, a->ldu, a->u != nullptr}};
  for (const auto& r : rows) {
    if (!r.need || a->tokens == 0) continue;
    DION_TRY(check_rows(r.name, r.p, r.ld, a->features, es));
    al = al && rows_aligned16(r.p, r.ld, es);
  }
  for (const float* g : {a->pre_gain, a->post_gain, a->gate}) al = al && (!g || aligned_to(g, 16));
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  if (a->tokens == 0) return DION_OK;
  NormP p{};
  p.x = a->x; p.y = a->y; p.h = a->h; p.u = a->u;
  p.pre = a->pre_gain; p.post = a->post_gain; p.gate = a->gate;
  if (a->kept) { p.q = a->kept->q; p.scale = a->kept->scale; }
  p.ldx = a->ldx; p.ldy = a->ldy; p.ldh = a->ldh; p.ldu = a->ldu;
  p.ldq = kept_ld(a->features);
  p.tokens = a->tokens; p.features = (int)a->features; p.post_norm = a->post_norm != 0;
  p.eps = a->eps; p.s = a->residual_scale; p.inv_d = (float)(1.0 / (double)a->features);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a->dtype) {
    case DION_BF16: launch_norm<__nv_bfloat16>(p, al, s); break;
    case DION_FP16: launch_norm<__half>(p, al, s); break;
    default: launch_norm<float>(p, al, s);
  }
  return launch_status("k_norm");
}

dion_status norm_grad_impl(const dion_norm_grad* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return set_error(DION_ERR_INVALID_ARG, "args is NULL");
  DION_TRY(check_norm(a->tokens, a->features, a->dtype, a->eps, a->residual_scale));
  const int64_t es = dtype_bytes(a->dtype);
  if (a->tokens > 0) {  // as above
    if (!a->y && (a->dy || a->post_norm || a->post_gain || a->gate || a->dpost_gain || a->dgate))
      return set_error(DION_ERR_INVALID_ARG,
                       "dy, post_norm, post_gain, gate, dpost_gain and dgate need y");
    if ((a->post_gain || a->dpost_gain) && !a->post_norm)
      return set_error(DION_ERR_INVALID_ARG, "post_gain and dpost_gain need post_norm");
    if (!a->du && (a->pre_gain || a->dpre_gain))
      return set_error(DION_ERR_INVALID_ARG, "pre_gain and dpre_gain need du");
    if (!a->du && !a->dh) return set_error(DION_ERR_INVALID_ARG, "neither du nor dh is given");
    if (!a->dx && !a->dy && !a->dpre_gain && !a->dpost_gain && !a->dgate)
      return set_error(DION_ERR_INVALID_ARG, "no gradient is asked for");
  }
  for (const auto& g : {a->pre_gain, a->post_gain, a->gate}) DION_TRY(check_gain("a gain", g));
  for (const auto& g : {a->dpre_gain, a->dpost_gain, a->dgate}) DION_TRY(check_gain("a gain's gradient", g));
  bool al = a->features % 8 == 0;
  struct { const char* name; const void* p; int64_t ld; bool need; } rows[] = {
      {"h", a->h, a->ldh, a->du != nullptr}, {"y", a->y, a->ldy, a->y != nullptr},
      {"du", a->du, a->lddu, a->du != nullptr}, {"dh", a->dh, a->lddh, a->dh != nullptr},
      {"dx", a->dx, a->lddx, a->dx != nullptr}, {"dy", a->dy, a->lddy, a->dy != nullptr}};
  for (const auto& r : rows) {
    if (!r.need || a->tokens == 0) continue;
    DION_TRY(check_rows(r.name, r.p, r.ld, a->features, es));
    al = al && rows_aligned16(r.p, r.ld, es);
  }
  for (const float* g : {a->pre_gain, a->post_gain, a->gate}) al = al && (!g || aligned_to(g, 16));
  const size_t need = dion_norm_backward_workspace(a->tokens, a->features);
  if (need && !ws) return set_error(DION_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return set_error(DION_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  if (!aligned_to(ws, 16)) return set_error(DION_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = grad_grid(a->tokens, a->features);
  if (grid > 0) {
    NormGradP p{};
    p.h = a->h; p.y = a->y; p.du = a->du; p.dh = a->dh; p.dx = a->dx; p.dy = a->dy;
    p.pre = a->pre_gain; p.post = a->post_gain; p.gate = a->gate;
    p.parts = static_cast<float*>(ws);
    p.ldh = a->ldh; p.ldy = a->ldy; p.lddu = a->lddu; p.lddh = a->lddh; p.lddx = a->lddx; p.lddy = a->lddy;
    p.tokens = a->tokens; p.features = (int)a->features; p.post_norm = a->post_norm != 0;
    p.eps = a->eps; p.s = a->residual_scale; p.inv_d = (float)(1.0 / (double)a->features);
    switch (a->dtype) {
      case DION_BF16: launch_grad<__nv_bfloat16>(p, al, grid, s); break;
      case DION_FP16: launch_grad<__half>(p, al, grid, s); break;
      default: launch_grad<float>(p, al, grid, s);
    }
    DION_TRY(launch_status("k_norm_grad"));
  }
  if (!a->dpre_gain && !a->dpost_gain && !a->dgate) return DION_OK;
  // no rows: the sums are zero (added to nothing, or written as zeros)
  const GainP gp{static_cast<const float*>(ws), (int)grid, (int)a->features, a->post_gain, a->gate,
                 a->dpre_gain, a->dpost_gain, a->dgate, a->residual_scale, a->accumulate != 0};
  k_norm_gains<<<(unsigned)((a->features + 31) / 32), 256, 0, s>>>(gp);
  return launch_status("k_norm_gains");
}

}  // namespace
}  // namespace dion

extern "C" {

dion_status dion_norm_forward(const dion_norm* args, void* stream) {
  return dion::norm_impl(args, stream);
}

size_t dion_norm_backward_workspace(int64_t tokens, int64_t features) {
  if (tokens < 1 || tokens > dion::kMaxTokens || features < 1 || features > dion::kMaxFeatures) return 0;
  return (size_t)dion::grad_grid(tokens, features) * 2 * (size_t)features * sizeof(float);
}

dion_status dion_norm_backward(const dion_norm_grad* args, void* d_workspace, size_t workspace_bytes,
                               void* stream) {
  return dion::norm_grad_impl(args, d_workspace, workspace_bytes, stream);
}

}  // extern "C"
