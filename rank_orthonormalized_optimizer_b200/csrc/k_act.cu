// Activations kept in 8 bits between the forward and the backward pass, and read back.
//
// A block of 32 features of a token becomes 32 e4m3 bytes and one exponent byte (the rule
// stands in rows.cuh): 33 bytes where bf16 takes 64.  Both directions are one pass over
// HBM with no reuse, 3.03 bytes per bf16 element; what bounds them is the copy bandwidth.
// A thread moves 32 bytes of a row (16 elements of the 2-byte types, so two neighbouring lanes
// share a block and its maximum takes a shuffle), 16 where the rows only start on 16 bytes,
// kUnroll pieces in flight.  Rows without alignment are read 8 single elements a thread (their
// 8-bit rows are aligned all the same) and written one element a lane, a warp to a block.
#include "operator.h"
#include "rows.cuh"

#include <algorithm>

namespace dion {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kBlocks = 8;  // blocks of a warp in flight, in the load without vectors

struct ActP {
  const void* x;   // save: source; load: destination (cast)
  int64_t ldx;
  uint8_t* q;
  uint8_t* scale;
  int64_t tokens, features, ld;  // ld = features rounded up to 32
};

// 8 H elements of a row at once, or one by one (H = 0: rows without alignment; their lines stay
// in L1 between the accesses), n of them inside the row.
template <typename T, int H>
__device__ __forceinline__ void load_pieces(const T* p, int n, Raw8<T>* raw) {
  if constexpr (H == 2) {
    ld_stream32(p, raw[0].a, raw[1].a);
  } else if constexpr (H == 1) {
    raw[0] = load_raw(p);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __ldg(reinterpret_cast<const unsigned short*>(p) + j) : 0u;
    raw[0].a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + j) : 0u;
    raw[0].a = make_uint4(w[0], w[1], w[2], w[3]);
    raw[0].b = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T, typename I, int VEC>
__global__ void __launch_bounds__(kThreads) k_act_save(const ActP p, const RowDiv<I> row_of) {
  constexpr int H = VEC == 2 ? 2 : 1, N = 8 * H;
  const I per_row = (I)(p.ld / N), total = (I)(p.tokens * per_row);
  const T* x = static_cast<const T*>(p.x);
  const I stride = (I)gridDim.x * kThreads;
  // whole groups of lanes share a block: the loop runs to a multiple of 32
  const I end = (total + 31) / 32 * 32;
  for (I i0 = (I)blockIdx.x * kThreads + threadIdx.x; i0 < end; i0 += stride * kUnroll) {
    Raw8<T> raw[kUnroll][H];
    int64_t row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride, r = row_of(i);
      row[u] = r;
      col[u] = (int)(i - r * per_row) * N;
      if (i < total && col[u] < p.features) load_pieces<T, VEC>(x + row[u] * p.ldx + col[u], (int)min((int64_t)8, p.features - col[u]), raw[u]);
      else
#pragma unroll
        for (int h = 0; h < H; ++h) raw[u][h] = zero_raw<T>();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride;
      uint32_t top = abs_bits8(raw[u][0]);
      if (H == 2) top = max(top, abs_bits8(raw[u][H - 1]));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      if (H == 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = act_exponent(top);
      const float f = act_unscale(e);
      const bool fine = top < kInfBits;
      uint32_t o[2 * H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float v[8];
        unpack(raw[u][h], v);
        o[2 * h] = fine ? e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16 : 0u;
        o[2 * h + 1] = fine ? e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16 : 0u;
      }
      if (i < total) {
        uint8_t* q = p.q + row[u] * p.ld + col[u];
        if constexpr (H == 2) st_vec(q, make_uint4(o[0], o[1], o[2], o[3]));
        else *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
        if (i % (4 / H) == 0) p.scale[row[u] * (p.ld / 32) + col[u] / 32] = fine ? e + 127 : 255;
      }
    }
  }
}

template <typename T, typename I, int H>
__global__ void __launch_bounds__(kThreads) k_act_load(const ActP p, const RowDiv<I> row_of) {
  constexpr int N = 8 * H;
  const I per_row = (I)(p.ld / N), total = (I)(p.tokens * per_row);
  T* x = static_cast<T*>(const_cast<void*>(p.x));
  const I stride = (I)gridDim.x * kThreads;
  for (I i0 = (I)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += stride * kUnroll) {
    uint32_t raw[kUnroll][2 * H];
    uint32_t E[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride, r = row_of(i);
      row[u] = r;
      col[u] = (int)(i - r * per_row) * N;
      if (i < total && col[u] < p.features) {
        const uint8_t* q = p.q + row[u] * p.ld + col[u];
        if constexpr (H == 2) {
          const uint4 v = ld_stream(q);
          raw[u][0] = v.x; raw[u][1] = v.y; raw[u][2 * H - 2] = v.z; raw[u][2 * H - 1] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(q);
          raw[u][0] = v.x; raw[u][1] = v.y;
        }
        E[u] = p.scale[row[u] * (p.ld / 32) + col[u] / 32];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const I i = i0 + u * stride;
      if (i >= total || col[u] >= p.features) continue;
      const float f = act_scale(E[u]);
      float v[N];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 t = e4m3x2_float((raw[u][j / 2] >> (16 * (j & 1))) & 0xffffu);
        v[2 * j] = t.x * f;
        v[2 * j + 1] = t.y * f;
      }
      T* to = x + row[u] * p.ldx + col[u];
      if constexpr (H == 2) st_vec32(to, pack8(v, T()), pack8(v + 8, T()));
      else store8(to, v);
    }
  }
}

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_act_load_any(const ActP p, const RowDiv<I> row_of) {
  const I per_row = (I)(p.ld / 32), total = (I)(p.tokens * per_row);
  T* x = static_cast<T*>(const_cast<void*>(p.x));
  const int lane = threadIdx.x & 31;
  const I stride = (I)gridDim.x * (kThreads / 32);
  for (I b0 = (I)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; b0 < total; b0 += stride * kBlocks) {
    uint32_t q[kBlocks], E[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const I b = b0 + u * stride;
      q[u] = b < total ? p.q[(int64_t)b * 32 + lane] : 0;
      E[u] = b < total ? p.scale[b] : 0;
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const I b = b0 + u * stride, r = row_of(b);
      const int64_t col = (int64_t)(b - r * per_row) * 32 + lane;
      if (b < total && col < p.features)
        x[(int64_t)r * p.ldx + col] = from_float<T>(e4m3x2_float(q[u]).x * act_scale(E[u]));
    }
  }
}

template <typename T, typename I, int H>
void launch_as(const ActP& p, bool save, unsigned grid, cudaStream_t s) {
  if (save) k_act_save<T, I, H><<<grid, kThreads, 0, s>>>(p, RowDiv<I>(p.ld / (H == 2 ? 16 : 8)));
  else if constexpr (H > 0) k_act_load<T, I, H><<<grid, kThreads, 0, s>>>(p, RowDiv<I>(p.ld / (8 * H)));
  else k_act_load_any<T, I><<<grid, kThreads, 0, s>>>(p, RowDiv<I>(p.ld / 32));
}

// H pieces of 8 elements to a thread; 0: the forms for rows without alignment.
template <typename T, int H>
void launch(const ActP& p, bool save, int sms, cudaStream_t s) {
  const bool by_warp = !save && H == 0;
  const int64_t items = p.tokens * (by_warp ? p.ld / 32 : p.ld / (H == 2 ? 16 : 8));
  const int64_t cap = (int64_t)sms * 8;
  const int64_t per_cta = by_warp ? kThreads / 32 : kThreads * kUnroll;
  const unsigned grid = (unsigned)std::min((items + per_cta - 1) / per_cta, cap);
  // indexes in 32 bits where all of them fit (a loop's last step overshoots by its stride):
  // the division by the row length is what costs
  if (items + cap * kThreads * kBlocks < (int64_t(1) << 31)) launch_as<T, uint32_t, H>(p, save, grid, s);
  else launch_as<T, int64_t, H>(p, save, grid, s);
}

template <typename T>
dion_status launch(const ActP& p, bool save, int sms, cudaStream_t s) {
  const bool vec = p.features % 8 == 0 && rows_vector(p.x, p.ldx, sizeof(T));
  const bool wide = vec && sizeof(T) == 2 && p.features % 16 == 0 && p.ldx % 16 == 0 && aligned_to(p.x, 32);
  if constexpr (sizeof(T) == 2) {
    if (wide) launch<T, 2>(p, save, sms, s);
    else if (vec) launch<T, 1>(p, save, sms, s);
    else launch<T, 0>(p, save, sms, s);
  } else {
    if (vec) launch<T, 1>(p, save, sms, s);
    else launch<T, 0>(p, save, sms, s);
  }
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
