// Activations kept in 8 bits between the forward and the backward pass, and read back.
//
// A block of 32 features of a token becomes 32 e4m3 bytes and one exponent byte (the rule
// stands in rows.cuh): 33 bytes where bf16 takes 64.  Both directions are one pass over
// HBM with no reuse, 3.03 bytes per bf16 element; what bounds them is the copy bandwidth.
// Rows that start on 16 bytes move 8 elements a thread (four neighbouring lanes share a
// block, so its maximum takes two shuffles), kUnroll of them in flight; other rows go one
// element a lane, a warp to a block.
#include "operator.h"
#include "rows.cuh"

#include <algorithm>

namespace dion {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

struct ActP {
  const void* x;   // save: source; load: destination (cast)
  int64_t ldx;
  uint8_t* q;
  uint8_t* scale;
  int64_t tokens, features, ld;  // ld = features rounded up to 32
};

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_act_save(const ActP p) {
  const I per_row = (I)(p.ld / 8), total = (I)(p.tokens * per_row);
  const T* x = static_cast<const T*>(p.x);
  const I stride = (I)gridDim.x * kThreads;
  // whole groups of four lanes share a block: the loop runs to a multiple of 32
  const I end = (total + 31) / 32 * 32;
  for (I i0 = (I)blockIdx.x * kThreads + threadIdx.x; i0 < end; i0 += stride * kUnroll) {
    Raw8<T> raw[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride, r = i / per_row;
      row[u] = r;
      col[u] = (int)(i - r * per_row) * 8;
      raw[u] = (i < total && col[u] < p.features) ? load_raw(x + row[u] * p.ldx + col[u]) : zero_raw<T>();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride;
      float v[8];
      unpack(raw[u], v);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[j]));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = act_exponent(top);
      const float f = act_unscale(e);
      const bool fine = top < kInfBits;
      if (i < total) {
        uint2 o = make_uint2(0, 0);
        if (fine) {
          o.x = e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16;
          o.y = e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16;
        }
        *reinterpret_cast<uint2*>(p.q + row[u] * p.ld + col[u]) = o;
        if ((i & 3) == 0) p.scale[row[u] * (p.ld / 32) + col[u] / 32] = fine ? e + 127 : 255;
      }
    }
  }
}

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_act_save_any(const ActP p) {
  const I per_row = (I)(p.ld / 32), total = (I)(p.tokens * per_row);
  const T* x = static_cast<const T*>(p.x);
  const int lane = threadIdx.x & 31;
  for (I b = ((I)blockIdx.x * kThreads + threadIdx.x) / 32; b < total; b += (I)gridDim.x * kThreads / 32) {
    const I r = b / per_row;
    const int64_t row = r, col = (int64_t)(b - r * per_row) * 32 + lane;
    const float v = col < p.features ? to_float(x[row * p.ldx + col]) : 0.f;
    const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(v));
    const int e = act_exponent(top);
    const bool fine = top < kInfBits;
    p.q[row * p.ld + col] = fine ? (uint8_t)e4m3x2(v * act_unscale(e), 0.f) : 0;
    if (lane == 0) p.scale[b] = fine ? e + 127 : 255;
  }
}

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_act_load(const ActP p) {
  const I per_row = (I)(p.ld / 8), total = (I)(p.tokens * per_row);
  T* x = static_cast<T*>(const_cast<void*>(p.x));
  const I stride = (I)gridDim.x * kThreads;
  for (I i0 = (I)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += stride * kUnroll) {
    uint2 raw[kUnroll];
    uint32_t E[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride, r = i / per_row;
      row[u] = r;
      col[u] = (int)(i - r * per_row) * 8;
      if (i < total && col[u] < p.features) {
        raw[u] = *reinterpret_cast<const uint2*>(p.q + row[u] * p.ld + col[u]);
        E[u] = p.scale[row[u] * (p.ld / 32) + col[u] / 32];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride;
      if (i >= total || col[u] >= p.features) continue;
      const float f = act_scale(E[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = e4m3x2_float(((j < 2 ? raw[u].x : raw[u].y) >> (16 * (j & 1))) & 0xffffu);
        v[2 * j] = t.x * f;
        v[2 * j + 1] = t.y * f;
      }
      store8(x + row[u] * p.ldx + col[u], v);
    }
  }
}

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_act_load_any(const ActP p) {
  const I per_row = (I)(p.ld / 32), total = (I)(p.tokens * per_row);
  T* x = static_cast<T*>(const_cast<void*>(p.x));
  const int lane = threadIdx.x & 31;
  for (I b = ((I)blockIdx.x * kThreads + threadIdx.x) / 32; b < total; b += (I)gridDim.x * kThreads / 32) {
    const I r = b / per_row;
    const int64_t row = r, col = (int64_t)(b - r * per_row) * 32 + lane;
    if (col < p.features)
      x[row * p.ldx + col] =
          from_float<T>(e4m3x2_float(p.q[row * p.ld + col]).x * act_scale(p.scale[b]));
  }
}

template <typename T, typename I>
void launch_as(const ActP& p, bool save, bool vec, unsigned grid, cudaStream_t s) {
  if (save) {
    if (vec) k_act_save<T, I><<<grid, kThreads, 0, s>>>(p);
    else k_act_save_any<T, I><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (vec) k_act_load<T, I><<<grid, kThreads, 0, s>>>(p);
    else k_act_load_any<T, I><<<grid, kThreads, 0, s>>>(p);
  }
}

template <typename T>
dion_status launch(const ActP& p, bool save, int sms, cudaStream_t s) {
  // the vector form takes whole 8-element groups of 16-byte aligned rows
  const bool vec = rows_aligned16(p.x, p.ldx, sizeof(T)) && p.features % 8 == 0;
  const int64_t items = vec ? p.tokens * (p.ld / 8) : p.tokens * p.ld;  // a thread's each
  const int64_t cap = (int64_t)sms * (vec ? 8 : 32);
  const int64_t per_cta = vec ? kThreads * kUnroll : kThreads;
  const unsigned grid = (unsigned)std::min((items + per_cta - 1) / per_cta, cap);
  // indexes in 32 bits where all of them fit (a loop's last step overshoots by its stride):
  // the division by the row length is what costs
  if (items + cap * kThreads * kUnroll < (int64_t(1) << 31)) launch_as<T, uint32_t>(p, save, vec, grid, s);
  else launch_as<T, int64_t>(p, save, vec, grid, s);
  return launch_status(save ? "k_act_save" : "k_act_load");
}

dion_status act_impl(const void* x, int64_t ldx, int32_t dtype, const dion_act_kept* kept, bool save,
                     void* stream) {
  if (!kept) return set_error(DION_ERR_INVALID_ARG, "kept is NULL");
  if (!valid_dtype(dtype)) return set_error(DION_ERR_INVALID_ARG, "dtype %d is not a dion_dtype", dtype);
  dion_status st = check_kept(*kept);
  if (st != DION_OK) return st;
  if (kept->tokens > 0 &&
      (st = check_rows("x", x, ldx, kept->features, dtype_bytes(dtype))) != DION_OK)
    return st;
  int sms = 0;
  if ((st = check_sm100(&sms)) != DION_OK) return st;
  if (kept->tokens == 0) return DION_OK;
  const ActP p{x, ldx, kept->q, kept->scale, kept->tokens, kept->features, kept_ld(kept->features)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DION_BF16: return launch<__nv_bfloat16>(p, save, sms, s);
    case DION_FP16: return launch<__half>(p, save, sms, s);
    default: return launch<float>(p, save, sms, s);
  }
}

}  // namespace
}  // namespace dion

extern "C" {

dion_status dion_act_save(const void* x, int64_t ldx, int32_t dtype, const dion_act_kept* kept,
                          void* stream) {
  return dion::act_impl(x, ldx, dtype, kept, true, stream);
}

dion_status dion_act_load(const dion_act_kept* kept, void* x, int64_t ldx, int32_t dtype,
                          void* stream) {
  return dion::act_impl(x, ldx, dtype, kept, false, stream);
}

}  // extern "C"
