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
// order; one cluster does it for a batch of up to kClusterMost positions), and the
// sorted list is cut into segments of kSeg positions.  A CTA adds up the rows of each run of
// equal ids in its segment; a run inside one segment is written to the table at once, the
// pieces of a longer one go to the workspace and a last kernel adds them in order.  Beside
// the segments' CTAs others write the zeros of the rows that no token met, so that every row
// of the table is written once.  No floating-point atomics: results repeat bit for bit.
#include "operator.h"
#include "rows.cuh"

#include <algorithm>
#include <type_traits>

namespace dion {
namespace {

constexpr int kThreads = 256;
constexpr int kSeg = 32;             // sorted positions per segment
constexpr int kDigit = 8;            // bits per pass of the sort
constexpr int kBins = 1 << kDigit;
constexpr int kKeys = 8;                    // keys per thread of a sort tile
constexpr int kTile = kThreads * kKeys;     // keys per CTA
constexpr int kZeroRows = 1024;             // rows of a CTA that writes zeros, at most
constexpr int kJoinGroups = 4;              // threads that share a column in the join

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

// N elements at once; the pointer is aligned to them (fp32: to 16 bytes at most).
template <typename T, int N> struct alignas(sizeof(T) * N) Few { T v[N]; };
template <typename T, int N>
__device__ __forceinline__ void load_few(const T* p, float* v) {
  const Few<T, N> f = *reinterpret_cast<const Few<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_float(f.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_few(T* p, const float* v) {
  Few<T, N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.v[i] = from_float<T>(v[i]);
  *reinterpret_cast<Few<T, N>*>(p) = f;
}

// One item: VEC consecutive elements of an output row.
constexpr int kLookups = 4;  // items of a thread in flight (of single elements twice as many)
template <typename TI, typename TO, int VEC, typename I>
__global__ void __launch_bounds__(kThreads) k_embed_lookup(const LookupP p, const RowDiv<I> row_of) {
  constexpr int U = VEC < 4 ? 2 * kLookups : kLookups;
  const I per_row = (I)(p.features / VEC), total = (I)(p.tokens * per_row);
  const I stride = (I)gridDim.x * kThreads;
  const TI* table = static_cast<const TI*>(p.table);
  TO* out = static_cast<TO*>(p.out);
  for (I i0 = (I)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += stride * U) {
    int64_t row[U], id[U];
    int64_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const I i = i0 + u * stride, r = row_of(i);
      row[u] = r;
      col[u] = (int64_t)(i - r * per_row) * VEC;
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
      float v[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = id[u] >= 0 && id[u] < p.vocab;
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[u][j] = 0.f;
        if (in) load_few<TI, VEC>(table + id[u] * p.ldt + col[u], v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * stride >= total) continue;
        const float f = id[u] >= 0 && id[u] < p.vocab ? p.scale : 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[u][j] *= f;
        store_few<TO, VEC>(out + row[u] * p.ldo + col[u], v[u]);
      }
    }
  }
}

template <typename TI, typename TO, int VEC>
void launch_lookup(const LookupP& p, int sms, cudaStream_t s) {
  const int64_t per_row = p.features / VEC, items = p.tokens * per_row;
  const int64_t want = (items + kThreads - 1) / kThreads, cap = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(want < cap ? want : cap);
  // as the 8-bit form's: 32-bit indexes where they fit
  if (items + cap * kThreads * 2 * kLookups < (int64_t(1) << 31))
    k_embed_lookup<TI, TO, VEC, uint32_t><<<grid, kThreads, 0, s>>>(p, RowDiv<uint32_t>(per_row));
  else
    k_embed_lookup<TI, TO, VEC, int64_t><<<grid, kThreads, 0, s>>>(p, RowDiv<int64_t>(per_row));
}

// vec: elements that every row of both arrays can move at once.
template <typename TI, typename TO>
void launch_lookup(const LookupP& p, int vec, int sms, cudaStream_t s) {
  switch (vec) {
    case 8: launch_lookup<TI, TO, 8>(p, sms, s); break;
    case 4: launch_lookup<TI, TO, 4>(p, sms, s); break;
    case 2: launch_lookup<TI, TO, 2>(p, sms, s); break;
    default: launch_lookup<TI, TO, 1>(p, sms, s);
  }
}

// ---------------------------------------------------------------- sort
struct SortP {
  const void* ids;  // first pass: keys come from the ids
  int id64;
  const uint32_t *key_in, *val_in;
  uint32_t *key_out, *val_out;
  uint32_t* hist;  // [kBins][tiles]: counts, then the exclusive sums over (bin, tile)
  uint32_t* nspans;  // set to zero by the sort
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
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.nspans = 0;
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

// Exclusive sums over n counts in place (n a multiple of 8), one CTA, eight counts a thread.
__global__ void __launch_bounds__(1024) k_sort_scan(uint32_t* hist, int64_t n) {
  __shared__ uint32_t warp_sum[32];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  uint32_t carry = 0;
  for (int64_t base = 0; base < n; base += 8 * 1024) {
    const int64_t i = base + threadIdx.x * 8;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (i < n) {
      a = *reinterpret_cast<const uint4*>(hist + i);
      b = *reinterpret_cast<const uint4*>(hist + i + 4);
    }
    const uint32_t v = a.x + a.y + a.z + a.w + b.x + b.y + b.z + b.w;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (l >= o) x += y;
    }
    if (l == 31) warp_sum[w] = x;
    __syncthreads();
    uint32_t t = warp_sum[l];  // every warp sums the warps' totals for itself
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
      if (l >= o) t += y;
    }
    uint32_t at = carry + x - v + (w ? __shfl_sync(0xffffffffu, t, w - 1) : 0u);
    carry += __shfl_sync(0xffffffffu, t, 31);
    if (i < n) {
      uint32_t c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t own = c[k];
        c[k] = at;
        at += own;
      }
      *reinterpret_cast<uint4*>(hist + i) = make_uint4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<uint4*>(hist + i + 4) = make_uint4(c[4], c[5], c[6], c[7]);
    }
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

// The whole sort in one cluster, for batches whose key and position fit one word (position in
// the low bits).  CTA c holds words [c share, (c + 1) share), a warp 32 rounds of them; a pass
// ranks each word among its warp's (32 at a time, by the lanes that hold the same digit), sums
// the counts per digit over the warps and, through distributed shared memory, over the CTAs,
// and sends each word to its place in whichever CTA holds it.  Ranking is what takes the time
// (a __match_any_sync every 70 cycles or so on an SM), hence the eight SMs: in one CTA the sort
// of 16384 positions took 40 us, with per-thread counters in place of the match 50 us.
constexpr int kClusterCtas = 8, kClusterThreads = 512, kClusterKeys = 8;
constexpr int64_t kClusterMost = (int64_t)kClusterCtas * kClusterThreads * kClusterKeys;

__device__ __forceinline__ void sort_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cta_address(const void* p, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(cta));
  return r;
}

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads, 1)
    k_sort_cluster(const SortP p, int passes, int pos_bits, int rounds) {
  constexpr int W = kClusterThreads / 32;
  __shared__ uint32_t words[2][kClusterThreads * kClusterKeys];
  __shared__ uint16_t bins[W][kBins];  // places stay below 2^16
  __shared__ uint32_t total[kBins];   // of this CTA, per digit
  __shared__ uint32_t sums[kBins / 32];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const uint32_t cta = blockIdx.x;    // one cluster: the rank
  grid_trigger();
  const uint32_t share = (uint32_t)rounds * kClusterThreads;
  const int first = w * 32 * rounds + l;
  if (cta == 0 && threadIdx.x == 0) *p.nspans = 0;
#pragma unroll
  for (int k = 0; k < kClusterKeys; ++k) {
    if (k >= rounds) break;
    const int64_t i = (int64_t)cta * share + first + k * 32;
    // words past the end stay behind all others: all ones, and last among equals
    words[0][first + k * 32] = i < p.tokens ? sort_key(p, i) << pos_bits | (uint32_t)i : 0xffffffffu;
  }
  __syncwarp();
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pos_bits + pass * kDigit;
    for (int i = l; i < kBins; i += 32) bins[w][i] = 0;
    __syncwarp();
    uint32_t word[kClusterKeys], pos[kClusterKeys];
#pragma unroll
    for (int k = 0; k < kClusterKeys; ++k) {
      if (k >= rounds) break;
      word[k] = words[pass & 1][first + k * 32];
      const uint32_t dig = word[k] >> shift & (kBins - 1);
      const uint32_t same = __match_any_sync(0xffffffffu, dig);
      const uint32_t rank = __popc(same & ((1u << l) - 1));
      const uint32_t before = bins[w][dig];
      __syncwarp();
      if (rank == 0) bins[w][dig] = (uint16_t)(before + __popc(same));
      __syncwarp();
      pos[k] = before + rank;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t at = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t c = bins[i][threadIdx.x];
        bins[i][threadIdx.x] = (uint16_t)at;
        at += c;
      }
      total[threadIdx.x] = at;
    }
    sort_cluster_sync();
    uint32_t all = 0, before = 0, scan = 0;  // of this digit: over the CTAs, in the earlier ones
    if (threadIdx.x < kBins) {
#pragma unroll
      for (uint32_t c = 0; c < kClusterCtas; ++c) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cta_address(&total[threadIdx.x], c)));
        all += v;
        before += c < cta ? v : 0;
      }
      scan = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (l >= o) scan += y;
      }
      if (l == 31) sums[w] = scan;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t at = before + scan - all;
      for (int i = 0; i < w; ++i) at += sums[i];
#pragma unroll
      for (int i = 0; i < W; ++i) bins[i][threadIdx.x] = (uint16_t)(bins[i][threadIdx.x] + at);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kClusterKeys; ++k) {
      if (k >= rounds) break;
      const uint32_t to = bins[w][word[k] >> shift & (kBins - 1)] + pos[k], owner = to / share;
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cta_address(&words[(pass & 1) ^ 1][to - owner * share], owner)),
                   "r"(word[k])
                   : "memory");
    }
    sort_cluster_sync();  // every word has arrived, and no CTA is read or written after the last
  }
#pragma unroll
  for (int k = 0; k < kClusterKeys; ++k) {
    if (k >= rounds) break;
    const int64_t i = (int64_t)cta * share + first + k * 32;
    if (i < p.tokens) {
      const uint32_t word = words[passes & 1][first + k * 32];
      p.key_out[i] = word >> pos_bits;
      p.val_out[i] = word & ((1u << pos_bits) - 1);
    }
  }
}

// ---------------------------------------------------------------- gradient
struct GradP {
  const uint32_t *key, *val;  // sorted ids and their positions
  const void* dout;
  float* dtable;
  float* parts;     // [segments][2][features]: a run's piece that began earlier / goes on later
  uint32_t* spans;  // segments in which a run starts that goes on past their end
  uint32_t* nspans;
  int64_t ldo, ldt, tokens, vocab, features;
  int64_t sum_ctas;  // CTAs that add up segments; those after them write zeros
  int col_ctas;      // CTAs that share a segment's columns
  int zero_rows;
  float scale;
  int accumulate;
};

// Column e of this thread's eight, in the group of 8 NT columns that starts at c0.
template <int NT, bool AL>
__device__ __forceinline__ int64_t grad_col(int64_t c0, int e) {
  return c0 + (AL ? threadIdx.x * 8 + e : e * NT + threadIdx.x);
}

template <int NT, bool AL>
__device__ __forceinline__ void grad_store(float* p, int64_t c0, int64_t features, const float* v,
                                           float scale, bool add) {
  if (AL) {
    const int64_t c = grad_col<NT, AL>(c0, 0);
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
      const int64_t c = grad_col<NT, AL>(c0, e);
      if (c < features) p[c] = v[e] * scale + (add ? p[c] : 0.f);
    }
  }
}

// First sorted position whose key is >= k.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t n, uint32_t k) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (key[mid] < k) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Zeros of the rows [first, first + zero_rows) that no token met.
template <int NT>
__device__ __forceinline__ void write_zeros(const GradP& p, int64_t first) {
  __shared__ uint8_t met[kZeroRows];
  __shared__ int64_t range[2];
  const int rows = (int)min((int64_t)p.zero_rows, p.vocab - first);
  for (int i = threadIdx.x; i < rows; i += NT) met[i] = 0;
  if (threadIdx.x < 2) range[threadIdx.x] = lower_bound(p.key, p.tokens, (uint32_t)(first + (threadIdx.x ? rows : 0)));
  __syncthreads();
  for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += NT) met[p.key[i] - first] = 1;
  __syncthreads();
  // a row at a time, by a warp or by the whole CTA: single elements up to a 16-byte boundary,
  // vectors, and single elements to the end
  const int group = p.features >= 4 * NT ? NT : 32, l = threadIdx.x % group;
  for (int r = threadIdx.x / group; r < rows; r += NT / group) {
    if (met[r]) continue;
    float* row = p.dtable + (first + r) * p.ldt;
    const int64_t head = min(p.features, (int64_t)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 4);
    const int64_t body = (p.features - head) / 4;
    float4* to = reinterpret_cast<float4*>(row + head);
    if (l < head) row[l] = 0.f;
    for (int64_t c = l; c < body; c += group) to[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t tail = head + body * 4 + l;
    if (tail < p.features) row[tail] = 0.f;
  }
}

// Rows that do not start on 16 bytes: their 16-byte aligned neighbourhoods as they lie in memory,
// kGroup rows at a time into one of two buffers (cp.async), read back element by element.  The
// elements around a row come along and are not used; 16 bytes that stick out of the whole array
// (its first and last row) are copied one element at a time.
template <typename T, int NT>
struct RowStage {
  static constexpr int kRow = NT * 8 * (int)sizeof(T) + 16;
  static constexpr int kGroup = sizeof(T) == 4 ? 4 : 8;
  static constexpr int kBytes = 2 * kGroup * kRow;
  uint32_t base;
  uintptr_t lo, hi;  // the array
  __device__ __forceinline__ RowStage(void* smem, const GradP& p) {
    base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    lo = reinterpret_cast<uintptr_t>(p.dout);
    hi = lo + ((p.tokens - 1) * p.ldo + p.features) * sizeof(T);
  }
  __device__ __forceinline__ uintptr_t address(const GradP& p, uint32_t pos, int64_t col0) const {
    return lo + (pos * p.ldo + col0) * sizeof(T);
  }
  // the columns [col0, col0 + cols) of positions val[0 .. rows)
  __device__ __forceinline__ void fetch(const GradP& p, int buffer, const uint32_t* val, int rows,
                                        int64_t col0, int cols) const {
    constexpr int kPieces = kRow / 16;
    for (int i = threadIdx.x; i < rows * kPieces; i += NT) {
      const int r = i / kPieces, piece = i % kPieces;
      const uintptr_t row = address(p, val[r], col0), at = (row & ~(uintptr_t)15) + 16 * piece;
      if (at >= row + cols * sizeof(T)) continue;
      const uint32_t to = base + (buffer * kGroup + r) * kRow + 16 * piece;
      if (at >= lo && at + 16 <= hi) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(at) : "memory");
      } else {
        for (int j = 0; j < 16 / (int)sizeof(T); ++j) {
          const uintptr_t e = at + j * sizeof(T);
          if (e < lo || e >= hi) continue;
          if constexpr (sizeof(T) == 2)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 2 * j), "h"(*reinterpret_cast<const uint16_t*>(e)) : "memory");
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 4 * j), "r"(*reinterpret_cast<const uint32_t*>(e)) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ float read(const GradP& p, int buffer, int r, uint32_t pos, int64_t col0, int c) const {
    const uint32_t at = base + (buffer * kGroup + r) * kRow + (uint32_t)(address(p, pos, col0) & 15) + c * (int)sizeof(T);
    if constexpr (sizeof(T) == 2) {
      uint16_t w;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at) : "memory");
      return to_float(*reinterpret_cast<const T*>(&w));
    } else {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
      return v;
    }
  }
};

template <typename T, int NT, bool AL>
__global__ void __launch_bounds__(NT) k_embed_sum(const GradP p) {
  grid_wait();
  if (blockIdx.x >= p.sum_ctas) {
    write_zeros<NT>(p, (blockIdx.x - p.sum_ctas) * p.zero_rows);
    return;
  }
  __shared__ uint32_t key[kSeg + 2], val[kSeg];  // key[0], key[n + 1]: the neighbours
  __shared__ int met;                            // positions before the padding, which is sorted last
  extern __shared__ uint4 stage_smem[];
  const int64_t seg = blockIdx.x / p.col_ctas;
  const int64_t col0 = (blockIdx.x - seg * p.col_ctas) * (8 * NT);
  const int64_t s0 = seg * kSeg;
  const int in = (int)min((int64_t)kSeg, p.tokens - s0);
  if (threadIdx.x == 0) met = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < in + 2; i += NT) {
    const int64_t at = s0 + i - 1;
    key[i] = at >= 0 && at < p.tokens ? p.key[at] : 0xffffffffu;
    if (i >= 1 && i <= in) {
      val[i - 1] = p.val[at];
      if (key[i] < p.vocab) atomicAdd(&met, 1);
    }
  }
  __syncthreads();
  const int n = met;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool began = key[0] == key[1];  // the current run began in an earlier segment
  // adds position i's elements; writes the sum where its run ends, or the segment
  auto add = [&](int i, const float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += v[e];
    const bool goes_on = key[i + 2] == key[i + 1];
    if (goes_on && i != in - 1) return;
    float* parts = p.parts + seg * 2 * p.features;
    if (began) {
      grad_store<NT, AL>(parts, col0, p.features, acc, 1.f, false);
    } else if (goes_on) {
      grad_store<NT, AL>(parts + p.features, col0, p.features, acc, 1.f, false);
      if (threadIdx.x == 0 && col0 == 0) p.spans[atomicAdd(p.nspans, 1u)] = (uint32_t)seg;
    } else {
      grad_store<NT, AL>(p.dtable + (int64_t)key[i + 1] * p.ldt, col0, p.features, acc, p.scale, p.accumulate);
    }
    began = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  };
  if constexpr (AL) {
    constexpr int U = 8;  // rows in flight
    const T* dout = static_cast<const T*>(p.dout);
    const int64_t c0 = grad_col<NT, AL>(col0, 0);
    for (int i0 = 0; i0 < n; i0 += U) {
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = i0 + u < n && c0 < p.features ? load_raw(dout + val[i0 + u] * p.ldo + c0) : zero_raw<T>();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u >= n) break;
        float v[8];
        unpack(raw[u], v);
        add(i0 + u, v);
      }
    }
  } else {
    using Stage = RowStage<T, NT>;
    const Stage stage(stage_smem, p);
    const int cols = (int)min((int64_t)(8 * NT), p.features - col0);
    stage.fetch(p, 0, val, min(n, Stage::kGroup), col0, cols);
    for (int g = 0, i0 = 0; i0 < n; ++g, i0 += Stage::kGroup) {
      const int next = i0 + Stage::kGroup;
      stage.fetch(p, (g + 1) & 1, val + min(next, kSeg), max(0, min(n - next, Stage::kGroup)), col0, cols);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      for (int u = 0; u < Stage::kGroup && i0 + u < n; ++u) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = e * NT + threadIdx.x;
          v[e] = c < cols ? stage.read(p, g & 1, u, val[i0 + u], col0, c) : 0.f;
        }
        add(i0 + u, v);
      }
      __syncthreads();  // the buffer is free again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
}

// Joins the pieces of the runs that cross segments.  The list's order varies from run to run,
// a row's sum does not: kJoinGroups threads a column take every kJoinGroups-th piece each, and
// their sums are added in order.  V4: four columns a thread.
constexpr int kJoinCols = 128;  // threads over the columns
template <bool V4>
__global__ void __launch_bounds__(kJoinCols * kJoinGroups) k_embed_join(const GradP p) {
  constexpr int V = V4 ? 4 : 1;
  __shared__ float sh[kJoinGroups][kJoinCols * V];
  const int64_t blocks = (p.features + kJoinCols * V - 1) / (kJoinCols * V);
  grid_wait();
  const int64_t items = *p.nspans * blocks;
  const int g = threadIdx.x / kJoinCols, l = threadIdx.x % kJoinCols, lane = threadIdx.x & 31;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t seg = p.spans[item / blocks];
    const uint32_t k = p.key[(seg + 1) * kSeg];  // inside the list: the run goes on there
    // the run's last segment: the next 32 segments' first keys, then 32 probes at a time
    const int64_t segs = (p.tokens + kSeg - 1) / kSeg;
    auto of_run = [&](int64_t s) { return s < segs && p.key[s * kSeg] == k; };
    int64_t last = seg + 1 + __popc(__ballot_sync(0xffffffffu, of_run(seg + 2 + lane)));
    if (last == seg + 33) {
      int64_t hi = segs;  // past hi it is not the run
      while (hi - last > 1) {
        const int64_t step = (hi - last + 32) / 33;
        const int64_t at = last + step * (lane + 1);
        const int n = __popc(__ballot_sync(0xffffffffu, at < hi && of_run(at)));
        hi = min(hi, last + step * (n + 1));
        last += step * n;
      }
    }
    const int64_t c = ((item % blocks) * kJoinCols + l) * V;
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.f;
    auto add = [&](const float* from) {
      if (V4) {
        const float4 v = *reinterpret_cast<const float4*>(from);
        a[0] += v.x; a[V4 ? 1 : 0] += v.y; a[V4 ? 2 : 0] += v.z; a[V4 ? 3 : 0] += v.w;
      } else {
        a[0] += *from;
      }
    };
    if (c < p.features) {
      if (g == 0) add(p.parts + (2 * seg + 1) * p.features + c);
#pragma unroll 8
      for (int64_t s = seg + 1 + g; s <= last; s += kJoinGroups) add(p.parts + 2 * s * p.features + c);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sh[g][l * V + i] = a[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinCols * V; i += kJoinCols * kJoinGroups) {
      const int64_t col = (item % blocks) * (kJoinCols * V) + i;
      if (col >= p.features) continue;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kJoinGroups; ++j) sum += sh[j][i];
      float* to = p.dtable + (int64_t)k * p.ldt + col;
      *to = sum * p.scale + (p.accumulate ? *to : 0.f);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) k_embed_zero(float* dtable, int64_t ldt, int64_t vocab,
                                                         int64_t features) {
  const int64_t total = vocab * features;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / features;
    dtable[row * ldt + i - row * features] = 0.f;
  }
}

// ---------------------------------------------------------------- host
struct GradLayout {
  int64_t tiles, segs;
  size_t key[2], val[2], hist, spans, parts, bytes;
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
  g.spans = take((size_t)(g.segs + 1) * 4);  // the count first
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
  int vec = 8;
  while (vec > 1 && !(a->features % vec == 0 && a->ldt % vec == 0 && a->ldo % vec == 0 &&
                      aligned_to(a->table, vec * ti) && aligned_to(a->out, vec * to)))
    vec /= 2;
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

// Threads of a segment's CTA: a warp's worth of 8 columns each up to 256 columns, at most 256.
template <typename T>
cudaError_t launch_sum(GradP p, bool al, int64_t segs, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    p.col_ctas = (int)((p.features + 8 * NT - 1) / (8 * NT));
    p.sum_ctas = segs * p.col_ctas;
    // zeros: 512 bytes a thread, enough to pay for finding the CTA's rows in the list (the table
    // of 32768 x 4096: 132 us, with 256 bytes 146)
    p.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(kZeroRows, NT * 512 / (4 * p.features)));
    const int64_t grid = p.sum_ctas + (p.accumulate ? 0 : (p.vocab + p.zero_rows - 1) / p.zero_rows);
    const int bytes = al ? 0 : RowStage<T, NT>::kBytes;
    if (bytes > 0)
      e = cudaFuncSetAttribute(k_embed_sum<T, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
      e = launch_after(al ? k_embed_sum<T, NT, true> : k_embed_sum<T, NT, false>, dim3((unsigned)grid), NT, bytes, s, p);
  };
  if (p.features <= 256) go(std::integral_constant<int, 32>());
  else if (p.features <= 512) go(std::integral_constant<int, 64>());
  else if (p.features <= 1024) go(std::integral_constant<int, 128>());
  else go(std::integral_constant<int, 256>());
  return e;
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
    if (!aligned_to(ws, 32)) return set_error(DION_ERR_MISALIGNED, "workspace is not 32-byte aligned");
  }
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a->tokens == 0) {
    if (a->accumulate) return DION_OK;
    k_embed_zero<<<(unsigned)(sms * 8), kThreads, 0, s>>>(a->dtable, a->ldt, a->vocab, a->features);
    return launch_status("k_embed_zero");
  }
  char* base = static_cast<char*>(ws);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(base + g.key[0]), reinterpret_cast<uint32_t*>(base + g.key[1])};
  uint32_t* val[2] = {reinterpret_cast<uint32_t*>(base + g.val[0]), reinterpret_cast<uint32_t*>(base + g.val[1])};
  SortP sp{};
  sp.ids = a->ids;
  sp.id64 = a->id_bytes == 8;
  sp.hist = reinterpret_cast<uint32_t*>(base + g.hist);
  sp.nspans = reinterpret_cast<uint32_t*>(base + g.spans);
  sp.tokens = a->tokens;
  sp.vocab = a->vocab;
  sp.tiles = (int)g.tiles;
  int bits = 0;  // of the largest key, vocab (the padding's)
  while (bits < 32 && (a->vocab >> bits) != 0) ++bits;
  const int passes = (bits + kDigit - 1) / kDigit;
  int at = 0;
  int pos_bits = 1;
  while ((a->tokens - 1) >> pos_bits) ++pos_bits;
  if (a->tokens <= kClusterMost && bits + pos_bits <= 32) {
    sp.first = 1;
    sp.key_out = key[0];
    sp.val_out = val[0];
    const int per_round = kClusterCtas * kClusterThreads;
    k_sort_cluster<<<kClusterCtas, kClusterThreads, 0, s>>>(sp, passes, pos_bits,
                                                            (int)((a->tokens + per_round - 1) / per_round));
    DION_TRY(launch_status("k_sort_cluster"));
  } else {
    for (int pass = 0; pass < passes; ++pass, at ^= 1) {
      sp.first = pass == 0;
      sp.shift = pass * kDigit;
      sp.key_in = key[at ^ 1];
      sp.val_in = val[at ^ 1];
      sp.key_out = key[at];
      sp.val_out = val[at];
      k_sort_count<<<(unsigned)g.tiles, kThreads, 0, s>>>(sp);
      k_sort_scan<<<1, 1024, 0, s>>>(sp.hist, (int64_t)kBins * g.tiles);
      k_sort_scatter<<<(unsigned)g.tiles, kThreads, 0, s>>>(sp);
      DION_TRY(launch_status("the sort of the tokens"));
    }
    at ^= 1;
  }
  GradP p{};
  p.key = key[at];
  p.val = val[at];
  p.dout = a->dout;
  p.dtable = a->dtable;
  p.parts = reinterpret_cast<float*>(base + g.parts);
  p.nspans = sp.nspans;
  p.spans = sp.nspans + 1;
  p.ldo = a->ldo; p.ldt = a->ldt;
  p.tokens = a->tokens; p.vocab = a->vocab; p.features = a->features;
  p.scale = a->scale;
  p.accumulate = a->accumulate != 0;
  const bool al = a->features % 8 == 0 && rows_vector(a->dtable, a->ldt, 4) && rows_vector(a->dout, a->ldo, es);
  DION_TRY(launch_status("k_embed_sum", a->dtype == DION_BF16   ? launch_sum<__nv_bfloat16>(p, al, g.segs, s)
                                        : a->dtype == DION_FP16 ? launch_sum<__half>(p, al, g.segs, s)
                                                                : launch_sum<float>(p, al, g.segs, s)));
  if (g.segs > 1) {
    // the list is on the device: a grid that fills the SMs, whose CTAs leave at once without work
    const bool v4 = a->features % 4 == 0;  // the pieces in the workspace then start on 16 bytes
    DION_TRY(launch_status("k_embed_join", launch_after(v4 ? k_embed_join<true> : k_embed_join<false>,
                                                        dim3((unsigned)(sms * 4)), kJoinCols * kJoinGroups, 0, s, p)));
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
