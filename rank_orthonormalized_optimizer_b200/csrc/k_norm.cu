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
// Both passes are bound by HBM: every row is read once and written once, and lives in the
// registers or the shared memory of the threads that own its columns in between.  A batch is
// streamed: a fixed grid walks the rows, each thread fetching its own columns of the rows to
// come into a ring of shared memory (cp.async; no thread reads another's slots, so the ring
// needs no barrier) while it works on the current one, with its gains in registers.  Rows that
// do not start on 16 bytes come as they lie and are read element by element (8192 x 4095 bf16
// backward 152 us, 789 loaded directly).  Where no ring fits (fp32 backward, more than 8192
// features) rows are loaded directly, a row per CTA, four rows a CTA up to 512 features.
// 16384 x 4096 bf16: forward 87 us, kept in 8 bits as well 97 to 108, backward 129 to 136 in short
// runs and 148 repeated, which is 5.4 to 6.2 TB/s of the 6.56 that a copy reaches.  A row's barriers
// cost most where a CTA has its SM for itself, so the backward pass adds a row's last sum and the
// next row's first ones in one (8192 x 8192 142 us, with a sum for each and two barriers a sum 187;
// 16384 x 4096 129 and 143; short runs).  The backward pass keeps each thread's column
// sums over its rows; a second kernel adds the CTAs' sums in a fixed order, so results repeat
// bit for bit.  All sums are fp32; only the stored rows are rounded.
#include "operator.h"
#include "rows.cuh"

#include <algorithm>
#include <type_traits>

namespace dion {
namespace {

constexpr int64_t kMaxFeatures = 16384;  // a row stays in the registers of one CTA
constexpr int kWarpRows = 4;             // rows of a CTA in the warp-per-row form
constexpr int kSms = 148;                // grids (and so workspace sizes) do not depend on the device
constexpr int kSmemMost = 226 * 1024;    // of the rings of one SM's CTAs

// Threads of a CTA, and CTAs of a streaming grid on an SM (512 threads of 128 registers).
constexpr int cta_threads(int nt) { return nt == 32 ? 32 * kWarpRows : nt; }
constexpr int ctas_per_sm(int nt) { return cta_threads(nt) > 512 ? 1 : 512 / cta_threads(nt); }
// The backward stream's: from two warps on those that make up 384 threads, each with longer rings
// and fewer parts (16384 x 1024 bf16 41.7 us, with 512 threads 42.9; x 2048 71 and 74).
constexpr int grad_ctas_per_sm(int nt) {
  const int most = ctas_per_sm(nt), want = (384 + nt - 1) / nt;
  return nt == 32 || most < want ? most : want;
}

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
  float* parts;  // [grid][2][part_ld(features)]
  int64_t ldh, ldy, lddu, lddh, lddx, lddy, tokens;
  int features;
  int post_norm;
  float eps, s, inv_d;
};

// 1 / sqrt(v) to about half an ulp: one Newton step on the approximation, with v r in two parts.
// An error here is a row's, and moves values of the 8-bit form across ties: with rsqrtf alone (off
// by up to two ulps) it was 1.5 times as far from the 64-bit result as the plain fp32 form, with
// the step 0.91 times (mean of six draws of 8192 x 4096, some 40 values each; v r in one part
// 0.97).  __frsqrt_rn does as well and cost 5 us of 100 (16384 x 4096, kept), the step nothing.
// An infinite v gives 0.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v), p = v * r, low = fmaf(v, r, -p);
  return v < INFINITY ? fmaf(0.5f * r, fmaf(-low, r, fmaf(-p, r, 1.f)), r) : r;
}

// Sums of N values over the NT threads that share a row (a warp, or the whole CTA).  The warps'
// sums go through one half of red; the next call takes the other, whose readers were all done
// before this call's barrier, so one barrier a call is enough.
template <int NT> constexpr int red_floats() { return NT == 32 ? 1 : 2 * 4 * (NT / 32); }
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& half) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (NT == 32) return;
  constexpr int W = NT / 32, LD = N == 1 ? 1 : 4;
  half ^= 1;
  float* sums = red + half * 4 * W;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sums[(threadIdx.x >> 5) * LD + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float a[LD];
    if constexpr (LD == 4)
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(sums + 4 * k);
    else
      a[0] = sums[k];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += a[i];
  }
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

// Eight values of a row's 8-bit form, from column c; four neighbouring lanes hold a block, and
// every lane of the warp calls.
__device__ __forceinline__ void keep8(uint8_t* q, uint8_t* scale, int c, int ldq, const float* v) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[j]));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (c >= ldq) return;
  const int e = act_exponent(top);
  const float f = act_unscale(e);
  const bool fine = top < kInfBits;
  uint2 o = make_uint2(0, 0);
  if (fine) {
    o.x = e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16;
    o.y = e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16;
  }
  *reinterpret_cast<uint2*>(q + c) = o;
  if ((c & 31) == 0) scale[c / 32] = fine ? e + 127 : 255;
}

// The 8-bit form of a row's u, whose elements are in v: zeros past the row's end.
template <int NT, int VPT, bool AL>
__device__ __forceinline__ void keep_row(const NormP& p, int64_t row, int tid, const float* v) {
  const int ldq = (int)p.ldq;
  uint8_t* q = p.q + row * ldq;
  uint8_t* scale = p.scale + row * (ldq / 32);
  if (AL) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) keep8(q, scale, (k * NT + tid) * 8, ldq, v + 8 * k);
  } else {
#pragma unroll
    for (int e = 0; e < 8 * VPT; ++e) {  // a warp holds 32 neighbouring columns
      const int c = column<NT, AL>(tid, e);
      const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(v[e]));
      if (c >= ldq) continue;
      const int x = act_exponent(top);
      const bool fine = top < kInfBits;
      q[c] = fine ? (uint8_t)e4m3x2(v[e] * act_unscale(x), 0.f) : 0;
      if ((tid & 31) == 0) scale[c / 32] = fine ? x + 127 : 255;
    }
  }
}

template <typename T, int NT, int VPT, bool AL>
__global__ void __launch_bounds__(cta_threads(NT)) k_norm(const NormP p) {
  constexpr int E = 8 * VPT;
  __shared__ __align__(16) float red[red_floats<NT>()];
  int half = 0;
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
      row_sum<NT, 1>(ss, red, half);
      f *= inv_sqrt(fmaf(ss[0], p.inv_d, p.eps));
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
  row_sum<NT, 1>(ss, red, half);
  const float r = inv_sqrt(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float a[8];
    gains<NT, AL>(p.pre, tid, k, d, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[8 * k + j] = a[j] * (h[8 * k + j] * r);
  }
  store_row<T, NT, VPT, AL>(static_cast<T*>(p.u) + row * p.ldu, tid, d, h);
  if (!p.q) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (column<NT, AL>(tid, e) >= d) h[e] = 0.f;
  keep_row<NT, VPT, AL>(p, row, tid, h);
}

// ---- the ring: this thread's 8-element pieces of A arrays of a row, STAGES rows
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <typename T, int NT, int VPT, int A, bool AL> struct Ring;
template <typename T, int NT, int VPT, int A>
struct Ring<T, NT, VPT, A, true> {
  static constexpr int kPiece = 8 * sizeof(T);
  static constexpr int kThreads = cta_threads(NT);
  static constexpr int kStage = A * VPT * kPiece * kThreads;
  uint32_t base;  // of this thread's slots: 16-byte slots of neighbouring threads lie together
  __device__ __forceinline__ explicit Ring(void* smem) {
    base = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * 16;
  }
  __device__ __forceinline__ uint32_t slot(int stage, int array, int k, int half) const {
    return base + stage * kStage + ((array * VPT + k) * (kPiece / 16) + half) * 16 * kThreads;
  }
  __device__ __forceinline__ void fetch(int stage, int array, const void* p, int64_t ld, int64_t r,
                                        int64_t, int tid, int d) const {
    const T* row = static_cast<const T*>(p) + r * ld;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * NT + tid) * 8;
      if (c < d)
#pragma unroll
        for (int i = 0; i < kPiece / 16; ++i) copy16(slot(stage, array, k, i), row + c + i * (16 / sizeof(T)));
    }
  }
  __device__ __forceinline__ void arrived() const {}
  __device__ __forceinline__ uint4 read16(uint32_t a) const {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
  }
  // piece k as 8 floats, zeros past the row's end
  __device__ __forceinline__ void read(int stage, int array, const void*, int64_t, int64_t, int k, int tid,
                                       int d, float* v) const {
    Raw8<T> raw = zero_raw<T>();
    if ((k * NT + tid) * 8 < d) {
      raw.a = read16(slot(stage, array, k, 0));
      if constexpr (kPiece == 32) raw.b = read16(slot(stage, array, k, 1));
    }
    unpack(raw, v);
  }
};
// Rows that do not start on 16 bytes: the row's 16-byte aligned neighbourhood, as it lies in
// memory, fetched by all of the row's threads and read back an element at a time (column
// (8 k + j) NT + tid, so that a warp's accesses are consecutive).  Here threads do read each
// other's slots: arrived() waits for all of them.  The elements around the row come along with
// its first and last 16 bytes and are not used; where those 16 bytes stick out of the whole array
// (its first and last row) the row's elements are copied one by one.
template <typename T, int NT, int VPT, int A>
struct Ring<T, NT, VPT, A, false> {
  static constexpr int kRow = NT * VPT * 8 * (int)sizeof(T) + 16;
  static constexpr int kStage = A * kRow * (cta_threads(NT) / NT);
  uint32_t base;
  __device__ __forceinline__ explicit Ring(void* smem) {
    base = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
           (NT == 32 ? (threadIdx.x >> 5) * A * kRow : 0);
  }
  __device__ __forceinline__ uint32_t row_slot(int stage, int array) const {
    return base + stage * kStage + array * kRow;
  }
  __device__ __forceinline__ void fetch(int stage, int array, const void* p, int64_t ld, int64_t r,
                                        int64_t tokens, int tid, int d) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + ((tokens - 1) * ld + d) * sizeof(T);
    const uintptr_t row = lo + r * ld * sizeof(T), from = row & ~(uintptr_t)15;
    const int n = (int)((row - from + d * sizeof(T) + 15) / 16);
    const uint32_t to = row_slot(stage, array);
    for (int i = tid; i < n; i += NT) {
      const uintptr_t at = from + 16 * i;
      if (at >= lo && at + 16 <= hi) {
        copy16(to + 16 * i, reinterpret_cast<const void*>(at));
      } else {
#pragma unroll
        for (int j = 0; j < 16 / (int)sizeof(T); ++j) {
          const uintptr_t e = at + j * sizeof(T);
          if (e < lo || e >= hi) continue;
          if constexpr (sizeof(T) == 2)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 16 * i + 2 * j),
                         "h"(*reinterpret_cast<const uint16_t*>(e)) : "memory");
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 16 * i + 4 * j),
                         "r"(*reinterpret_cast<const uint32_t*>(e)) : "memory");
        }
      }
    }
  }
  __device__ __forceinline__ void arrived() const {
    if (NT == 32) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ void read(int stage, int array, const void* p, int64_t ld, int64_t r, int k,
                                       int tid, int d, float* v) const {
    const uint32_t at = row_slot(stage, array) +
                        (uint32_t)((reinterpret_cast<uintptr_t>(p) + r * ld * sizeof(T)) & 15);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (8 * k + j) * NT + tid;
      v[j] = 0.f;
      if (c >= d) continue;
      if constexpr (sizeof(T) == 2) {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at + c * 2) : "memory");
        v[j] = to_float(*reinterpret_cast<const T*>(&w));
      } else {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(at + c * 4) : "memory");
      }
    }
  }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// u (and its 8-bit form) of one row from h, whose elements are in v; the thread's pre-gains in w.
template <typename T, int NT, int VPT, bool AL>
__device__ __forceinline__ void finish_row(const NormP& p, int64_t row, int tid, float* v, const float* w,
                                           float r) {
  const int d = p.features;
#pragma unroll
  for (int e = 0; e < 8 * VPT; ++e) v[e] = column<NT, AL>(tid, e) < d ? w[e] * (v[e] * r) : 0.f;
  store_row<T, NT, VPT, AL>(static_cast<T*>(p.u) + row * p.ldu, tid, d, v);
  if (p.q) keep_row<NT, VPT, AL>(p, row, tid, v);
}

template <typename T, int NT, int VPT, bool AL, int STAGES>
__global__ void __launch_bounds__(cta_threads(NT), ctas_per_sm(NT)) k_norm_stream(const NormP p) {
  constexpr int E = 8 * VPT, RPC = NT == 32 ? kWarpRows : 1;
  extern __shared__ uint4 ring_smem[];
  __shared__ __align__(16) float red[red_floats<NT>()];
  int half = 0;
  const Ring<T, NT, VPT, 2, AL> ring(ring_smem);
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int d = p.features;
  const int64_t step = (int64_t)gridDim.x * RPC;
  const int64_t first = (int64_t)blockIdx.x * RPC + (NT == 32 ? threadIdx.x >> 5 : 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.tokens) {
      ring.fetch(stage, 0, p.x, p.ldx, row, p.tokens, tid, d);
      if (p.y) ring.fetch(stage, 1, p.y, p.ldy, row, p.tokens, tid, d);
    }
    ring_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(first + i * step, i);
  float w[E], c[E];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float a[8], b[8];
    gains<NT, AL>(p.pre, tid, k, d, w + 8 * k);
    gains<NT, AL>(p.post, tid, k, d, a);
    gains<NT, AL>(p.gate, tid, k, d, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) c[8 * k + j] = a[j] * b[j];
  }
  int stage = 0;
  for (int64_t row = first; row < p.tokens; row += step) {
    ring_wait<STAGES - 2>();
    ring.arrived();
    float h[E];
#pragma unroll
    for (int k = 0; k < VPT; ++k) ring.read(stage, 0, p.x, p.ldx, row, k, tid, d, h + 8 * k);
    float ss[1] = {0.f};
    if (p.y) {
      float y[E];
#pragma unroll
      for (int k = 0; k < VPT; ++k) ring.read(stage, 1, p.y, p.ldy, row, k, tid, d, y + 8 * k);
      float f = p.s;
      if (p.post_norm) {
#pragma unroll
        for (int e = 0; e < E; ++e) ss[0] = fmaf(y[e], y[e], ss[0]);
        row_sum<NT, 1>(ss, red, half);
        f *= inv_sqrt(fmaf(ss[0], p.inv_d, p.eps));
        ss[0] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = fmaf(c[e], y[e] * f, h[e]);
      if (p.h) store_row<T, NT, VPT, AL>(static_cast<T*>(p.h) + row * p.ldh, tid, d, h);
    }
    // the slots read in the last round take the next row
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    if (++stage == STAGES) stage = 0;
    if (!p.u) continue;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (column<NT, AL>(tid, e) < d) ss[0] = fmaf(h[e], h[e], ss[0]);
    row_sum<NT, 1>(ss, red, half);
    finish_row<T, NT, VPT, AL>(p, row, tid, h, w, inv_sqrt(fmaf(ss[0], p.inv_d, p.eps)));
  }
  ring_wait<0>();
}

// This CTA's column sums; where a CTA holds several rows its warps add theirs in order.  The
// parts' rows are padded to whole vectors.
__host__ __device__ constexpr int64_t part_ld(int64_t d) { return (d + 7) / 8 * 8; }
template <int NT, int VPT, bool AL>
__device__ __forceinline__ void write_parts(const NormGradP& p, int tid, float* apre, float* apost) {
  constexpr int E = 8 * VPT, RPC = NT == 32 ? kWarpRows : 1;
  __shared__ float sum[NT == 32 ? 2 * E * 32 : 1];
  const int d = p.features;
  float* part = p.parts + blockIdx.x * 2 * part_ld(d);
  if (NT == 32) {
    for (int turn = 0; turn < RPC; ++turn) {
      if ((threadIdx.x >> 5) == turn)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          apre[e] += turn ? sum[e * 32 + tid] : 0.f;
          apost[e] += turn ? sum[(E + e) * 32 + tid] : 0.f;
          sum[e * 32 + tid] = apre[e];
          sum[(E + e) * 32 + tid] = apost[e];
        }
      __syncthreads();
    }
    if ((threadIdx.x >> 5) != RPC - 1) return;
  }
  if (AL) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * NT + tid) * 8;
      if (c < d) {
        store8(part + c, apre + 8 * k);
        store8(part + part_ld(d) + c, apost + 8 * k);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = column<NT, AL>(tid, e);
      if (c < d) {
        part[c] = apre[e];
        part[part_ld(d) + c] = apost[e];
      }
    }
  }
}

template <typename T, int NT, int VPT, bool AL, int STAGES>
__global__ void __launch_bounds__(cta_threads(NT), grad_ctas_per_sm(NT)) k_norm_grad_stream(const NormGradP p) {
  constexpr int E = 8 * VPT, RPC = NT == 32 ? kWarpRows : 1;
  extern __shared__ uint4 ring_smem[];
  __shared__ __align__(16) float red[red_floats<NT>()];
  int half = 0;
  grid_trigger();  // a grid of one round, whose CTAs fill the SMs
  enum { H, DU, DH, Y };
  const Ring<T, NT, VPT, 4, AL> ring(ring_smem);
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int d = p.features;
  const int64_t step = (int64_t)gridDim.x * RPC;
  const int64_t first = (int64_t)blockIdx.x * RPC + (NT == 32 ? threadIdx.x >> 5 : 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.tokens) {
      if (p.du) {
        ring.fetch(stage, H, p.h, p.ldh, row, p.tokens, tid, d);
        ring.fetch(stage, DU, p.du, p.lddu, row, p.tokens, tid, d);
      }
      if (p.dh) ring.fetch(stage, DH, p.dh, p.lddh, row, p.tokens, tid, d);
      if (p.y) ring.fetch(stage, Y, p.y, p.ldy, row, p.tokens, tid, d);
    }
    ring_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(first + i * step, i);
  float w[E], c[E], apre[E], apost[E];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float a[8], b[8];
    gains<NT, AL>(p.pre, tid, k, d, w + 8 * k);
    gains<NT, AL>(p.post, tid, k, d, a);
    gains<NT, AL>(p.gate, tid, k, d, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) c[8 * k + j] = p.s * a[j] * b[j];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) apre[e] = apost[e] = 0.f;
  // the row's sums for both norms, this thread's share
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  auto statistics = [&](int64_t row, int stage) {
    sum[0] = sum[1] = sum[2] = 0.f;
    if (p.du)
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float h[8], u[8];
        ring.read(stage, H, p.h, p.ldh, row, k, tid, d, h);
        ring.read(stage, DU, p.du, p.lddu, row, k, tid, d, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[0] = fmaf(h[j], h[j], sum[0]);
          sum[1] = fmaf(w[8 * k + j] * u[j], h[j], sum[1]);
        }
      }
    if (p.y && p.post_norm)
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float y[8];
        ring.read(stage, Y, p.y, p.ldy, row, k, tid, d, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[2] = fmaf(y[j], y[j], sum[2]);
      }
  };
  ring_wait<STAGES - 2>();
  ring.arrived();
  if (first < p.tokens) statistics(first, 0);
  row_sum<NT, 4>(sum, red, half);
  int stage = 0;
  for (int64_t row = first; row < p.tokens; row += step) {
    if (!AL) ring.arrived();  // all have read the last row
    // the slots read in the last round take the next row
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    float g[E];
    const float r = inv_sqrt(fmaf(sum[0], p.inv_d, p.eps));
    const float m1 = sum[1] * r * p.inv_d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float h[8], u[8];
      if (p.dh) {
        ring.read(stage, DH, p.dh, p.lddh, row, k, tid, d, g + 8 * k);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[8 * k + j] = 0.f;
      }
      if (p.du) {
        ring.read(stage, H, p.h, p.ldh, row, k, tid, d, h);
        ring.read(stage, DU, p.du, p.lddu, row, k, tid, d, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * k + j;
          const float hn = h[j] * r;
          apre[e] = fmaf(u[j], hn, apre[e]);
          g[e] = fmaf(r, fmaf(-hn, m1, w[e] * u[j]), g[e]);
        }
      }
    }
    if (p.dx) store_row<T, NT, VPT, AL>(static_cast<T*>(p.dx) + row * p.lddx, tid, d, g);
    const float ry = p.post_norm ? inv_sqrt(fmaf(sum[2], p.inv_d, p.eps)) : 1.f;
    sum[3] = 0.f;
    if (p.y)
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float y[8];
        ring.read(stage, Y, p.y, p.ldy, row, k, tid, d, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * k + j;
          const float yn = y[j] * ry;
          apost[e] = fmaf(g[e], yn, apost[e]);
          g[e] *= c[e];
          sum[3] = fmaf(g[e], yn, sum[3]);
        }
      }
    // this row's last sum and the next row's first ones share a barrier
    const int next = stage + 1 == STAGES ? 0 : stage + 1;
    ring_wait<STAGES - 2>();
    ring.arrived();
    if (row + step < p.tokens) statistics(row + step, next);
    row_sum<NT, 4>(sum, red, half);
    if (p.dy) {
      if (p.post_norm) {
        const float m2 = sum[3] * p.inv_d;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float y[8];
          ring.read(stage, Y, p.y, p.ldy, row, k, tid, d, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[8 * k + j] = ry * fmaf(-y[j] * ry, m2, g[8 * k + j]);
        }
      }
      store_row<T, NT, VPT, AL>(static_cast<T*>(p.dy) + row * p.lddy, tid, d, g);
    }
    stage = next;
  }
  ring_wait<0>();
  write_parts<NT, VPT, AL>(p, tid, apre, apost);
}

// The form without a ring.  Rows of more than two pieces a thread keep the column sums in
// shared memory (registers would spill), each thread its own columns'.
template <typename T, int NT, int VPT, bool AL>
__global__ void __launch_bounds__(cta_threads(NT)) k_norm_grad(const NormGradP p) {
  constexpr int E = 8 * VPT;
  constexpr int RPC = NT == 32 ? kWarpRows : 1;
  constexpr bool WIDE = VPT > 2;
  extern __shared__ float wide[];  // [2][E][NT]
  __shared__ __align__(16) float red[red_floats<NT>()];
  int half = 0;
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int sub = NT == 32 ? threadIdx.x >> 5 : 0;
  const int d = p.features;
  float apre[WIDE ? 1 : E], apost[WIDE ? 1 : E];
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) wide[e * NT + tid] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) apre[WIDE ? 0 : e] = apost[WIDE ? 0 : e] = 0.f;
  }
  auto add_pre = [&](int e, float a, float b) {
    if (WIDE) wide[e * NT + tid] = fmaf(a, b, wide[e * NT + tid]);
    else apre[WIDE ? 0 : e] = fmaf(a, b, apre[WIDE ? 0 : e]);
  };
  auto add_post = [&](int e, float a, float b) {
    if (WIDE) wide[(E + e) * NT + tid] = fmaf(a, b, wide[(E + e) * NT + tid]);
    else apost[WIDE ? 0 : e] = fmaf(a, b, apost[WIDE ? 0 : e]);
  };
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
    row_sum<NT, 3>(sum, red, half);
    if (p.du) {
      const float r = inv_sqrt(fmaf(sum[0], p.inv_d, p.eps));
      const float m1 = sum[1] * r * p.inv_d;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float a[8];
        gains<NT, AL>(p.pre, tid, k, d, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * k + j;
          const float hn = h[e] * r;
          add_pre(e, w[e], hn);
          g[e] = fmaf(r, fmaf(-hn, m1, a[j] * w[e]), g[e]);
        }
      }
    }
    if (p.dx) store_row<T, NT, VPT, AL>(static_cast<T*>(p.dx) + row * p.lddx, tid, d, g);
    if (!p.y) continue;
    const float ry = p.post_norm ? inv_sqrt(fmaf(sum[2], p.inv_d, p.eps)) : 1.f;
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
        add_post(e, g[e], y[e]);
        g[e] *= p.s * a[j] * b[j];
        dot[0] = fmaf(g[e], y[e], dot[0]);
      }
    }
    if (p.post_norm) {
      row_sum<NT, 1>(dot, red, half);
      const float m2 = dot[0] * p.inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = ry * fmaf(-y[e], m2, g[e]);
    }
    if (p.dy) store_row<T, NT, VPT, AL>(static_cast<T*>(p.dy) + row * p.lddy, tid, d, g);
  }
  if (WIDE) {
    float* part = p.parts + blockIdx.x * 2 * part_ld(d);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = column<NT, AL>(tid, e);
      if (c < d) {
        part[c] = wide[e * NT + tid];
        part[part_ld(d) + c] = wide[(E + e) * NT + tid];
      }
    }
  } else {
    write_parts<NT, WIDE ? 2 : VPT, AL>(p, tid, apre, apost);
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

// Adds the CTAs' partial sums of COLS columns: the threads that share a column take turns over
// the parts, and their sums are added in a fixed tree.  32 columns a CTA read whole lines; below
// 4096 features 8 (a sector) leave more CTAs (16384 x 1024: 7 us, with 32 columns 10 us).
constexpr int kGainThreads = 1024;
template <int COLS>
__global__ void __launch_bounds__(kGainThreads) k_norm_gains(const GainP p) {
  __shared__ float sh[2][kGainThreads / 32][COLS];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int c = blockIdx.x * COLS + l % COLS;
  float a = 0.f, b = 0.f;
  grid_wait();
  if (c < p.features) {
#pragma unroll 4
    for (int k = threadIdx.x / COLS; k < p.nparts; k += kGainThreads / COLS) {
      const float* part = p.parts + k * 2 * part_ld(p.features) + c;
      a += part[0];
      b += part[part_ld(p.features)];
    }
  }
#pragma unroll
  for (int o = COLS; o < 32; o <<= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (l < COLS) {
    sh[0][w][l] = a;
    sh[1][w][l] = b;
  }
  __syncthreads();
  if (threadIdx.x >= COLS || c >= p.features) return;
  a = b = 0.f;
#pragma unroll
  for (int k = 0; k < kGainThreads / 32; ++k) {
    a += sh[0][k][l];
    b += sh[1][k][l];
  }
  const float gate = p.gate ? p.gate[c] : 1.f, post = p.post ? p.post[c] : 1.f;
  if (p.dpre) p.dpre[c] = (p.accumulate ? p.dpre[c] : 0.f) + a;
  if (p.dpost) p.dpost[c] = (p.accumulate ? p.dpost[c] : 0.f) + p.s * gate * b;
  if (p.dgate) p.dgate[c] = (p.accumulate ? p.dgate[c] : 0.f) + p.s * post * b;
}

// Threads of a row and 8-element pieces of a thread, by the features: a warp up to 512, then
// the smallest CTA that holds the row in two pieces a thread, four at the widest.  (8192 x 5120
// bf16: 71 and 112 us forward and backward with 320 threads, 78 and 134 with 512.)
template <typename F>
void by_width(int64_t d, F f) {
  if (d <= 256) f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  else if (d <= 512) f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  else if (d <= 1024) f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  else if (d <= 1536) f(std::integral_constant<int, 96>(), std::integral_constant<int, 2>());
  else if (d <= 2048) f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  else if (d <= 2560) f(std::integral_constant<int, 160>(), std::integral_constant<int, 2>());
  else if (d <= 4096) f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  else if (d <= 5120) f(std::integral_constant<int, 320>(), std::integral_constant<int, 2>());
  else if (d <= 6144) f(std::integral_constant<int, 384>(), std::integral_constant<int, 2>());
  else if (d <= 8192) f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
}

// CTAs that take all rows when each takes its share once, and a streaming grid's.
int64_t row_ctas(int64_t tokens, int nt) { return nt == 32 ? (tokens + kWarpRows - 1) / kWarpRows : tokens; }
int64_t stream_ctas(int nt) { return (int64_t)kSms * ctas_per_sm(nt); }

cudaError_t allow_smem(const void* kernel, int bytes) {
  return bytes <= 32 * 1024 ? cudaSuccess  // with the static part well inside the default limit
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Rows of the rings, none where they do not fit (the direct form).  Backward, two rows are in work
// and one or two on their way; forward one is in work, and more than two on their way gain nothing.
// fp32 forward on aligned rows takes the direct form, too: a piece is two 16-byte copies there, half
// a sector each, and the stream of 8192 x 4096 ran at 133 us against 85 us.
template <typename T, int NT, int VPT, int A, bool AL>
constexpr int ring_stages() {
  constexpr int stage = Ring<T, NT, VPT, A, AL>::kStage * (A == 4 ? grad_ctas_per_sm(NT) : ctas_per_sm(NT));
  if (VPT > 2 || (A == 2 && AL && sizeof(T) == 4)) return 0;
  constexpr int least = A == 4 ? 3 : 2, most = A == 4 ? 4 : 3, fit = kSmemMost / stage;
  return fit < least ? 0 : fit < most ? fit : most;
}

template <typename K, typename P>
cudaError_t launch_with(K* kernel, unsigned grid, int threads, int bytes, const P& p, cudaStream_t s) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), bytes);
  if (e == cudaSuccess) kernel<<<grid, threads, bytes, s>>>(p);
  return e;
}

template <typename T, int NT, int VPT, bool AL>
cudaError_t launch_norm(const NormP& p, cudaStream_t s) {
  constexpr int stages = ring_stages<T, NT, VPT, 2, AL>();
  const int64_t rows = row_ctas(p.tokens, NT);
  if constexpr (stages > 0)
    return launch_with(k_norm_stream<T, NT, VPT, AL, stages>, (unsigned)std::min(rows, stream_ctas(NT)),
                       cta_threads(NT), stages * Ring<T, NT, VPT, 2, AL>::kStage, p, s);
  else
    return launch_with(k_norm<T, NT, VPT, AL>, (unsigned)rows, cta_threads(NT), 0, p, s);
}

template <typename T, int NT, int VPT, bool AL>
cudaError_t launch_grad(const NormGradP& p, unsigned& grid, cudaStream_t s) {
  constexpr int stages = ring_stages<T, NT, VPT, 4, AL>();
  if constexpr (stages > 0) {
    grid = std::min(grid, (unsigned)(kSms * grad_ctas_per_sm(NT)));
    return launch_with(k_norm_grad_stream<T, NT, VPT, AL, stages>, grid, cta_threads(NT),
                       stages * Ring<T, NT, VPT, 4, AL>::kStage, p, s);
  } else
    return launch_with(k_norm_grad<T, NT, VPT, AL>, grid, cta_threads(NT),
                       VPT > 2 ? 2 * 8 * VPT * NT * 4 : 0, p, s);
}

template <typename T>
cudaError_t launch_norm(const NormP& p, bool al, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  by_width(p.features, [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    e = al ? launch_norm<T, NT, VPT, true>(p, s) : launch_norm<T, NT, VPT, false>(p, s);
  });
  return e;
}

template <typename T>
cudaError_t launch_grad(const NormGradP& p, bool al, unsigned& grid, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  by_width(p.features, [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    e = al ? launch_grad<T, NT, VPT, true>(p, grid, s) : launch_grad<T, NT, VPT, false>(p, grid, s);
  });
  return e;
}

unsigned grad_grid(int64_t tokens, int64_t features) {
  int64_t grid = 0;
  by_width(features, [&](auto nt, auto) {
    constexpr int NT = decltype(nt)::value;
    // every CTA adds a row of partial sums: one CTA an SM up to eight rows for each of these, and
    // from there on the streaming grid at once (just above, its CTAs have a row or two each)
    const int64_t rows = row_ctas(tokens, NT);
    grid = std::min(rows, rows < 8 * kSms ? (int64_t)kSms : stream_ctas(NT));
  });
  return (unsigned)grid;
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
    al = al && rows_vector(r.p, r.ld, es);
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
  cudaError_t e = cudaSuccess;
  switch (a->dtype) {
    case DION_BF16: e = launch_norm<__nv_bfloat16>(p, al, s); break;
    case DION_FP16: e = launch_norm<__half>(p, al, s); break;
    default: e = launch_norm<float>(p, al, s);
  }
  if (e != cudaSuccess) return set_error(DION_ERR_CUDA, "k_norm: %s", cudaGetErrorString(e));
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
    al = al && rows_vector(r.p, r.ld, es);
  }
  for (const float* g : {a->pre_gain, a->post_gain, a->gate}) al = al && (!g || aligned_to(g, 16));
  const size_t need = dion_norm_backward_workspace(a->tokens, a->features);
  if (need && !ws) return set_error(DION_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return set_error(DION_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  if (!aligned_to(ws, 32)) return set_error(DION_ERR_MISALIGNED, "workspace is not 32-byte aligned");
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned grid = grad_grid(a->tokens, a->features);  // the parts that the workspace holds, at most
  if (grid > 0) {
    NormGradP p{};
    p.h = a->h; p.y = a->y; p.du = a->du; p.dh = a->dh; p.dx = a->dx; p.dy = a->dy;
    p.pre = a->pre_gain; p.post = a->post_gain; p.gate = a->gate;
    p.parts = static_cast<float*>(ws);
    p.ldh = a->ldh; p.ldy = a->ldy; p.lddu = a->lddu; p.lddh = a->lddh; p.lddx = a->lddx; p.lddy = a->lddy;
    p.tokens = a->tokens; p.features = (int)a->features; p.post_norm = a->post_norm != 0;
    p.eps = a->eps; p.s = a->residual_scale; p.inv_d = (float)(1.0 / (double)a->features);
    cudaError_t e = cudaSuccess;
    switch (a->dtype) {
      case DION_BF16: e = launch_grad<__nv_bfloat16>(p, al, grid, s); break;
      case DION_FP16: e = launch_grad<__half>(p, al, grid, s); break;
      default: e = launch_grad<float>(p, al, grid, s);
    }
    if (e != cudaSuccess) return set_error(DION_ERR_CUDA, "k_norm_grad: %s", cudaGetErrorString(e));
    DION_TRY(launch_status("k_norm_grad"));
  }
  if (!a->dpre_gain && !a->dpost_gain && !a->dgate) return DION_OK;
  // no rows: the sums are zero (added to nothing, or written as zeros)
  const GainP gp{static_cast<const float*>(ws), (int)grid, (int)a->features, a->post_gain, a->gate,
                 a->dpre_gain, a->dpost_gain, a->dgate, a->residual_scale, a->accumulate != 0};
  const int cols = a->features >= 4096 ? 32 : 8;
  return launch_status("k_norm_gains",
                       launch_after(cols == 32 ? k_norm_gains<32> : k_norm_gains<8>,
                                    dim3((unsigned)((a->features + cols - 1) / cols)), kGainThreads, 0, s, gp));
}

}  // namespace
}  // namespace dion

extern "C" {

dion_status dion_norm_forward(const dion_norm* args, void* stream) {
  return dion::norm_impl(args, stream);
}

size_t dion_norm_backward_workspace(int64_t tokens, int64_t features) {
  if (tokens < 1 || tokens > dion::kMaxTokens || features < 1 || features > dion::kMaxFeatures) return 0;
  return (size_t)dion::grad_grid(tokens, features) * 2 * (size_t)dion::part_ld(features) * sizeof(float);
}

dion_status dion_norm_backward(const dion_norm_grad* args, void* d_workspace, size_t workspace_bytes,
                               void* stream) {
  return dion::norm_grad_impl(args, d_workspace, workspace_bytes, stream);
}

}  // extern "C"
