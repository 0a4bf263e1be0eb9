// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   out[t] = s table[id[t]]            dtable[v] = s sum over t with id[t] = v of dout[t]
//
// An id outside [0, vocab) stands for no token (padding): its row of out is zero and it
// adds to no row of dtable.  Both are bound by HBM: the lookup reads and writes each row
// once; the gradient reads every row of dout once and writes the whole fp32 table, most of
// which is zeros (2^15 rows of 4096 take 0.54 GB).
//
// The gradient sorts the positions by id (a stable radix sort, so equal ids keep their
// order), and the sorted list is cut into segments of kSeg positions.  A CTA adds up the
// rows of each run of equal ids in its segment; a run inside one segment is written to the
// table at once, the pieces of a longer one go to the workspace and a second kernel adds
// them in order.  No floating-point atomics: results repeat bit for bit.
#include "operator.h"
#include "rows.cuh"

namespace dion {
namespace {

constexpr int kThreads = 256;
constexpr int kSeg = 32;             // sorted positions per segment
constexpr int kCols = 8 * kThreads;  // columns of a CTA in the sum over a segment
constexpr int kDigit = 8;            // bits per pass of the sort
constexpr int kBins = 1 << kDigit;
constexpr int kKeys = 16;                   // keys per thread of a sort tile
constexpr int kTile = kThreads * kKeys;     // keys per CTA
constexpr int kJoinWarps = 8;

// ---------------------------------------------------------------- lookup
struct LookupP {
  const void* table;
  const void* ids;
  void* out;
  int64_t ldt, ldo, tokens, vocab, features;
  int id64;
  float scale;
};

__device__ __forceinline__ int64_t load_id(const void* ids, int id64, int64_t t) {
  return id64 ? __ldg(static_cast<const long long*>(ids) + t) : __ldg(static_cast<const int*>(ids) + t);
}

// One item: VEC consecutive elements of an output row.
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_lookup(const LookupP p) {
  constexpr int U = 4;
  const int64_t per_row = p.features / VEC, total = p.tokens * per_row;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const TI* table = static_cast<const TI*>(p.table);
  TO* out = static_cast<TO*>(p.out);
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += stride * U) {
    int64_t row[U], id[U];
    int64_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * stride;
      row[u] = i / per_row;
      col[u] = (i - row[u] * per_row) * VEC;
      id[u] = i < total ? load_id(p.ids, p.id64, row[u]) : -1;
    }
    if (VEC == 8) {
      Raw8<TI> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = id[u] >= 0 && id[u] < p.vocab ? load_raw(table + id[u] * p.ldt + col[u]) : zero_raw<TI>();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * stride >= total) continue;
        float v[8];
        unpack(raw[u], v);
        const float f = id[u] >= 0 && id[u] < p.vocab ? p.scale : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
        store8(out + row[u] * p.ldo + col[u], v);
      }
    } else {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = id[u] >= 0 && id[u] < p.vocab ? p.scale * to_float(table[id[u] * p.ldt + col[u]]) : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * stride < total) out[row[u] * p.ldo + col[u]] = from_float<TO>(v[u]);
    }
  }
}

template <typename TI, typename TO>
void launch_lookup(const LookupP& p, bool vec, int sms, cudaStream_t s) {
  const int64_t items = p.tokens * (vec ? p.features / 8 : p.features);
  const int64_t want = (items + kThreads - 1) / kThreads, cap = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(want < cap ? want : cap);
  if (vec) k_embed_lookup<TI, TO, 8><<<grid, kThreads, 0, s>>>(p);
  else k_embed_lookup<TI, TO, 1><<<grid, kThreads, 0, s>>>(p);
}

// ---------------------------------------------------------------- sort
struct SortP {
  const void* ids;  // first pass: keys come from the ids
  int id64;
  const uint32_t *key_in, *val_in;
  uint32_t *key_out, *val_out;
  uint32_t* hist;  // [kBins][tiles]: counts, then the exclusive sums over (bin, tile)
  int64_t tokens, vocab;
  int tiles, shift, first;
};

__device__ __forceinline__ uint32_t sort_key(const SortP& p, int64_t i) {
  if (!p.first) return p.key_in[i];
  const int64_t id = load_id(p.ids, p.id64, i);
  return id >= 0 && id < p.vocab ? (uint32_t)id : (uint32_t)p.vocab;  // no token: sorted last
}

__global__ void __launch_bounds__(kThreads) k_sort_count(const SortP p) {
  __shared__ uint32_t bins[kBins];
  bins[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll 4
  for (int k = 0; k < kKeys; ++k) {
    const int64_t i = base + k * kThreads + threadIdx.x;
    if (i < p.tokens) atomicAdd(&bins[(sort_key(p, i) >> p.shift) & (kBins - 1)], 1u);
  }
  __syncthreads();
  p.hist[(int64_t)threadIdx.x * p.tiles + blockIdx.x] = bins[threadIdx.x];
}

// Exclusive sums over n counts in place, one CTA.
__global__ void __launch_bounds__(1024) k_sort_scan(uint32_t* hist, int64_t n) {
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t carry;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (threadIdx.x == 0) carry = 0;
  for (int64_t base = 0; base < n; base += 1024) {
    const int64_t i = base + threadIdx.x;
    const uint32_t v = i < n ? hist[i] : 0;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (l >= o) x += y;
    }
    if (l == 31) warp_sum[w] = x;
    __syncthreads();
    if (w == 0) {
      uint32_t t = warp_sum[l];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
        if (l >= o) t += y;
      }
      warp_sum[l] = t;
    }
    __syncthreads();
    const uint32_t before = carry + (w ? warp_sum[w - 1] : 0u) + x - v;
    if (i < n) hist[i] = before;
    __syncthreads();
    if (threadIdx.x == 0) carry += warp_sum[31];
    __syncthreads();
  }
}

// Stable scatter of one tile: a warp owns 32 * kKeys consecutive keys and ranks 32 at a
// time by the lanes that hold the same digit.
__global__ void __launch_bounds__(kThreads) k_sort_scatter(const SortP p) {
  constexpr int W = kThreads / 32;
  __shared__ uint32_t bins[W][kBins];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  for (int i = l; i < kBins; i += 32) bins[w][i] = 0;
  __syncwarp();
  const int64_t base = (int64_t)blockIdx.x * kTile + (int64_t)w * 32 * kKeys;
  uint32_t key[kKeys], val[kKeys], pos[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int64_t i = base + k * 32 + l;
    const bool in = i < p.tokens;
    key[k] = in ? sort_key(p, i) : 0;
    val[k] = in ? (p.first ? (uint32_t)i : p.val_in[i]) : 0;
  }
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const bool in = base + k * 32 + l < p.tokens;
    const uint32_t dig = in ? (key[k] >> p.shift) & (kBins - 1) : kBins;  // absent keys: apart
    const uint32_t same = __match_any_sync(0xffffffffu, dig);
    uint32_t before = 0;
    if (in) before = bins[w][dig];
    __syncwarp();
    const uint32_t rank = __popc(same & ((1u << l) - 1));
    if (in && rank == 0) bins[w][dig] = before + __popc(same);
    __syncwarp();
    pos[k] = before + rank;
  }
  __syncthreads();
  // this digit's start for each warp: the tile's start plus the earlier warps' counts
  {
    uint32_t at = p.hist[(int64_t)threadIdx.x * p.tiles + blockIdx.x];
    for (int i = 0; i < W; ++i) {
      const uint32_t n = bins[i][threadIdx.x];
      bins[i][threadIdx.x] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    if (base + k * 32 + l >= p.tokens) continue;
    const uint32_t to = bins[w][(key[k] >> p.shift) & (kBins - 1)] + pos[k];
    p.key_out[to] = key[k];
    p.val_out[to] = val[k];
  }
}

// ---------------------------------------------------------------- gradient
struct GradP {
  const uint32_t *key, *val;  // sorted ids and their positions
  const void* dout;
  float* dtable;
  float* parts;  // [segments][2][features]: a run's piece that began earlier / goes on later
  int64_t ldo, ldt, tokens, vocab, features;
  float scale;
  int accumulate;
};

__global__ void __launch_bounds__(kThreads) k_embed_zero(float* dtable, int64_t ldt, int64_t vocab,
                                                         int64_t features, int vec) {
  const int64_t step = vec ? 4 : 1;
  const int64_t per_row = features / step, total = vocab * per_row;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per_row;
    float* p = dtable + row * ldt + (i - row * per_row) * step;
    if (vec) *reinterpret_cast<float4*>(p) = make_float4(0.f, 0.f, 0.f, 0.f);
    else *p = 0.f;
  }
}

template <bool AL>
__device__ __forceinline__ int64_t grad_col(int e) {
  return (int64_t)blockIdx.y * kCols + (AL ? threadIdx.x * 8 + e : e * kThreads + threadIdx.x);
}

template <bool AL>
__device__ __forceinline__ void grad_store(float* p, int64_t features, const float* v, float scale,
                                           bool add) {
  if (AL) {
    const int64_t c = grad_col<AL>(0);
    if (c >= features) return;
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[e] * scale;
    if (add) {
      const float4 a = *reinterpret_cast<const float4*>(p + c), b = *reinterpret_cast<const float4*>(p + c + 4);
      o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
      o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
    }
    store8(p + c, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = grad_col<AL>(e);
      if (c < features) p[c] = v[e] * scale + (add ? p[c] : 0.f);
    }
  }
}

template <typename T, bool AL>
__global__ void __launch_bounds__(kThreads) k_embed_sum(const GradP p) {
  __shared__ uint32_t key[kSeg + 2], val[kSeg];  // key[0], key[n + 1]: the neighbours
  const int64_t s0 = (int64_t)blockIdx.x * kSeg;
  const int n = (int)min((int64_t)kSeg, p.tokens - s0);
  const uint32_t none = 0xffffffffu;
  for (int i = threadIdx.x; i < n + 2; i += kThreads) {
    const int64_t at = s0 + i - 1;
    key[i] = at >= 0 && at < p.tokens ? p.key[at] : none;
    if (i >= 1 && i <= n) val[i - 1] = p.val[at];
  }
  __syncthreads();
  constexpr int U = 4;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool began = key[0] == key[1];  // the current run began in an earlier segment
  const T* dout = static_cast<const T*>(p.dout);
  const int64_t c0 = grad_col<AL>(0);
  for (int i0 = 0; i0 < n; i0 += U) {
    if (key[i0 + 1] >= p.vocab) break;  // padding, sorted last
    float v[U][8];
    if (AL) {
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = i0 + u < n && key[i0 + u + 1] < p.vocab && c0 < p.features
                     ? load_raw(dout + val[i0 + u] * p.ldo + c0) : zero_raw<T>();
#pragma unroll
      for (int u = 0; u < U; ++u) unpack(raw[u], v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t c = grad_col<AL>(e);
          v[u][e] = i0 + u < n && key[i0 + u + 1] < p.vocab && c < p.features
                        ? to_float(dout[val[i0 + u] * p.ldo + c]) : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= n || key[i + 1] >= p.vocab) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
      const bool last = i == n - 1;
      const bool goes_on = key[i + 2] == key[i + 1];
      if (goes_on && !last) continue;
      float* parts = p.parts + (int64_t)blockIdx.x * 2 * p.features;
      if (began) grad_store<AL>(parts, p.features, acc, 1.f, false);
      else if (goes_on) grad_store<AL>(parts + p.features, p.features, acc, 1.f, false);
      else grad_store<AL>(p.dtable + (int64_t)key[i + 1] * p.ldt, p.features, acc, p.scale, p.accumulate);
      began = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    }
  }
}

// Joins the pieces of the runs that cross segments: the segment where such a run starts
// adds its pieces, each warp every kJoinWarps-th, and then the warps' sums, in order.
__global__ void __launch_bounds__(32 * kJoinWarps) k_embed_join(const GradP p) {
  __shared__ float sh[kJoinWarps][32];
  const int64_t seg = blockIdx.x;
  const int64_t end = min(p.tokens, (seg + 1) * kSeg);
  if (end >= p.tokens) return;
  const uint32_t k = p.key[end - 1];
  if (k >= p.vocab || p.key[end] != k) return;                      // no run goes on
  const int64_t s0 = seg * kSeg;
  if (s0 > 0 && p.key[s0] == k && p.key[s0 - 1] == k) return;       // it began earlier
  int64_t lo = end, hi = p.tokens;                                   // first position past the run
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.key[mid] == k) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / kSeg;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  for (int64_t c0 = (int64_t)blockIdx.y * 32; c0 < p.features; c0 += (int64_t)gridDim.y * 32) {
    const int64_t c = c0 + l;
    float a = 0.f;
    if (c < p.features) {
      if (w == 0) a = p.parts[(2 * seg + 1) * p.features + c];
#pragma unroll 4
      for (int64_t s = seg + 1 + w; s <= last; s += kJoinWarps) a += p.parts[2 * s * p.features + c];
    }
    sh[w][l] = a;
    __syncthreads();
    if (w == 0 && c < p.features) {
      a = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) a += sh[i][l];
      float* to = p.dtable + (int64_t)k * p.ldt + c;
      *to = a * p.scale + (p.accumulate ? *to : 0.f);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host
struct GradLayout {
  int64_t tiles, segs;
  size_t key[2], val[2], hist, parts, bytes;
};

GradLayout grad_layout(int64_t tokens, int64_t features) {
  GradLayout g{};
  g.tiles = (tokens + kTile - 1) / kTile;
  g.segs = (tokens + kSeg - 1) / kSeg;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    g.key[i] = take((size_t)tokens * 4);
    g.val[i] = take((size_t)tokens * 4);
  }
  g.hist = take((size_t)g.tiles * kBins * 4);
  g.parts = take((size_t)g.segs * 2 * (size_t)features * 4);
  g.bytes = at;
  return g;
}

constexpr int64_t kMaxVocab = (int64_t(1) << 31) - 2;
constexpr int64_t kMaxWidth = 1 << 24;

dion_status check_embed(int64_t tokens, int64_t vocab, int64_t features, const void* ids,
                        int32_t id_bytes, float scale) {
  const dion_status st = check_tokens(tokens);
  if (st != DION_OK) return st;
  if (vocab < 1 || vocab > kMaxVocab)
    return set_error(DION_ERR_INVALID_ARG, "vocab %lld outside [1, 2^31 - 2]", (long long)vocab);
  if (features < 1 || features > kMaxWidth)
    return set_error(DION_ERR_UNSUPPORTED_SHAPE, "features %lld outside [1, 2^24]", (long long)features);
  if (id_bytes != 4 && id_bytes != 8)
    return set_error(DION_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
  if (tokens > 0 && !ids) return set_error(DION_ERR_INVALID_ARG, "ids is NULL");
  if (!aligned_to(ids, (size_t)id_bytes))
    return set_error(DION_ERR_MISALIGNED, "ids are not aligned to their %d bytes", id_bytes);
  if (!std::isfinite(scale)) return set_error(DION_ERR_INVALID_ARG, "scale is not finite");
  return DION_OK;
}

#define DION_TRY(call)              \
  do {                              \
    const dion_status st_ = (call); \
    if (st_ != DION_OK) return st_; \
  } while (0)

dion_status lookup_impl(const dion_embed* a, void* stream) {
  if (!a) return set_error(DION_ERR_INVALID_ARG, "args is NULL");
  DION_TRY(check_embed(a->tokens, a->vocab, a->features, a->ids, a->id_bytes, a->scale));
  if (!valid_dtype(a->table_dtype) || !valid_dtype(a->out_dtype))
    return set_error(DION_ERR_INVALID_ARG, "table_dtype or out_dtype is not a dion_dtype");
  const int64_t ti = dtype_bytes(a->table_dtype), to = dtype_bytes(a->out_dtype);
  if (a->tokens > 0) {
    DION_TRY(check_rows("table", a->table, a->ldt, a->features, ti));
    DION_TRY(check_rows("out", a->out, a->ldo, a->features, to));
  }
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  if (a->tokens == 0) return DION_OK;
  const LookupP p{a->table, a->ids, a->out, a->ldt, a->ldo, a->tokens, a->vocab, a->features,
                  a->id_bytes == 8, a->scale};
  const bool vec = a->features % 8 == 0 && rows_aligned16(a->table, a->ldt, ti) &&
                   rows_aligned16(a->out, a->ldo, to);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto from = [&](auto in) {
    using TI = decltype(in);
    switch (a->out_dtype) {
      case DION_BF16: launch_lookup<TI, __nv_bfloat16>(p, vec, sms, s); break;
      case DION_FP16: launch_lookup<TI, __half>(p, vec, sms, s); break;
      default: launch_lookup<TI, float>(p, vec, sms, s);
    }
  };
  switch (a->table_dtype) {
    case DION_BF16: from(__nv_bfloat16()); break;
    case DION_FP16: from(__half()); break;
    default: from(float());
  }
  return launch_status("k_embed_lookup");
}

template <typename T>
void launch_sum(const GradP& p, bool al, dim3 grid, cudaStream_t s) {
  if (al) k_embed_sum<T, true><<<grid, kThreads, 0, s>>>(p);
  else k_embed_sum<T, false><<<grid, kThreads, 0, s>>>(p);
}

dion_status embed_grad_impl(const dion_embed_grad* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return set_error(DION_ERR_INVALID_ARG, "args is NULL");
  DION_TRY(check_embed(a->tokens, a->vocab, a->features, a->ids, a->id_bytes, a->scale));
  if (!valid_dtype(a->dtype)) return set_error(DION_ERR_INVALID_ARG, "dtype %d is not a dion_dtype", a->dtype);
  const int64_t es = dtype_bytes(a->dtype);
  if (a->tokens > 0) DION_TRY(check_rows("dout", a->dout, a->ldo, a->features, es));
  DION_TRY(check_rows("dtable", a->dtable, a->ldt, a->features, 4));
  const GradLayout g = grad_layout(a->tokens, a->features);
  if (a->tokens > 0) {
    if (!ws) return set_error(DION_ERR_INVALID_ARG, "workspace is NULL");
    if (ws_bytes < g.bytes)
      return set_error(DION_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, g.bytes);
    if (!aligned_to(ws, 16)) return set_error(DION_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  }
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool vec_table = a->features % 4 == 0 && rows_aligned16(a->dtable, a->ldt, 4);
  if (!a->accumulate) {
    k_embed_zero<<<(unsigned)(sms * 8), kThreads, 0, s>>>(a->dtable, a->ldt, a->vocab, a->features, vec_table);
    DION_TRY(launch_status("k_embed_zero"));
  }
  if (a->tokens == 0) return DION_OK;
  char* base = static_cast<char*>(ws);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(base + g.key[0]), reinterpret_cast<uint32_t*>(base + g.key[1])};
  uint32_t* val[2] = {reinterpret_cast<uint32_t*>(base + g.val[0]), reinterpret_cast<uint32_t*>(base + g.val[1])};
  SortP sp{};
  sp.ids = a->ids;
  sp.id64 = a->id_bytes == 8;
  sp.hist = reinterpret_cast<uint32_t*>(base + g.hist);
  sp.tokens = a->tokens;
  sp.vocab = a->vocab;
  sp.tiles = (int)g.tiles;
  int bits = 0;  // of the largest key, vocab (the padding's)
  while (bits < 32 && (a->vocab >> bits) != 0) ++bits;
  int at = 0;
  for (int shift = 0; shift < bits; shift += kDigit, at ^= 1) {
    sp.first = shift == 0;
    sp.shift = shift;
    sp.key_in = key[at ^ 1];
    sp.val_in = val[at ^ 1];
    sp.key_out = key[at];
    sp.val_out = val[at];
    k_sort_count<<<(unsigned)g.tiles, kThreads, 0, s>>>(sp);
    k_sort_scan<<<1, 1024, 0, s>>>(sp.hist, (int64_t)kBins * g.tiles);
    k_sort_scatter<<<(unsigned)g.tiles, kThreads, 0, s>>>(sp);
    DION_TRY(launch_status("the sort of the tokens"));
  }
  GradP p{};
  p.key = key[at ^ 1];
  p.val = val[at ^ 1];
  p.dout = a->dout;
  p.dtable = a->dtable;
  p.parts = reinterpret_cast<float*>(base + g.parts);
  p.ldo = a->ldo; p.ldt = a->ldt;
  p.tokens = a->tokens; p.vocab = a->vocab; p.features = a->features;
  p.scale = a->scale;
  p.accumulate = a->accumulate != 0;
  const bool al = a->features % 8 == 0 && vec_table && rows_aligned16(a->dout, a->ldo, es);
  const dim3 grid((unsigned)g.segs, (unsigned)((a->features + kCols - 1) / kCols));
  switch (a->dtype) {
    case DION_BF16: launch_sum<__nv_bfloat16>(p, al, grid, s); break;
    case DION_FP16: launch_sum<__half>(p, al, grid, s); break;
    default: launch_sum<float>(p, al, grid, s);
  }
  DION_TRY(launch_status("k_embed_sum"));
  if (g.segs > 1) {
    const int64_t cols = (a->features + 31) / 32;
    k_embed_join<<<dim3((unsigned)g.segs, (unsigned)(cols < 128 ? cols : 128)), 32 * kJoinWarps, 0, s>>>(p);
    DION_TRY(launch_status("k_embed_join"));
  }
  return DION_OK;
}

}  // namespace
}  // namespace dion

extern "C" {

dion_status dion_embed_lookup(const dion_embed* args, void* stream) {
  return dion::lookup_impl(args, stream);
}

size_t dion_embed_backward_workspace(int64_t tokens, int64_t features) {
  if (tokens < 1 || tokens > dion::kMaxTokens || features < 1 || features > dion::kMaxWidth) return 0;
  return dion::grad_layout(tokens, features).bytes;
}

dion_status dion_embed_backward(const dion_embed_grad* args, void* d_workspace,
                                size_t workspace_bytes, void* stream) {
  return dion::embed_grad_impl(args, d_workspace, workspace_bytes, stream);
}

}  // extern "C"
