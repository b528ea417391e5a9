// experts.cu -- the rows around products grouped by expert: a router's choice
// of experts and its gradient, the (token, choice) pairs sorted by expert, the
// tokens' rows to their places and back with weights, and the gradients.
//
// Everything here is bound by memory, by latency or, the router, by
// instructions; nothing waits on the host, and every sum has a fixed order.
// Measured: route 16384 x 256, top 8 8.5 us (2.0 TB/s), its gradient 7.1, sort of
// 131072 pairs over 256 experts 6.9, dispatch of 16384 x 4096 fp8 rows four times
// 57 (6.0 TB/s), combine of 8 x 8001 x 4096 in bf16 101 (6.5 TB/s), combine's
// gradient with the router's, 4 x 8192 x 2048, 54 (5.6 TB/s).
#include <cfloat>

#include "ops.cuh"
#include "groups.cuh"

namespace g12 {
namespace {

constexpr int kMaxTop = 32;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Order-preserving integer of a logit; 0 for those never chosen (masked by
// -infinity, NaN).  -0 counts as 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t u = __float_as_uint(l + 0.0f);
  if (!(l > -INFINITY)) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// ------------------------------------------------------------------ router
struct RouteArgs {
  int64_t rows, ld;
  int experts, top, type, normalize;
  const void* logits;
  int32_t* expert;
  float* weight;
};

// A lane's logits of a row (lane l holds l, l + 32, ...).
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, int type, int64_t at, int experts, float (&l)[V]) {
  const int lane = threadIdx.x & 31;
  if (type == GEMM_OUT_F32) {
    const float* from = static_cast<const float*>(logits) + at;
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = v * 32 + lane < experts ? from[v * 32 + lane] : -INFINITY;
  } else {
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(logits) + at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      l[v] = v * 32 + lane < experts ? __bfloat162float(from[v * 32 + lane]) : -INFINITY;
  }
}

// One warp per row, its logits in registers.
template <int V>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ uint2 lists[V >= 2 ? kWarps : 1][V >= 2 ? 32 : 1];  // candidates
  uint2* const list = lists[V >= 2 ? threadIdx.x >> 5 : 0];
  const uint32_t lane = threadIdx.x & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[V];
    load_logits(a.logits, a.type, row * a.ld, a.experts, l);
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) most = fmaxf(most, l[v]);  // passes over NaN
    uint32_t largest = logit_key(most);
    const uint32_t first = __reduce_max_sync(0xffffffffu, largest);
    const float m = first == 0u ? 0.0f : key_value(first);
    // Lane j's choice: which of the `top` it is (place), its index and its value.
    int mine = -1, place = lane;
    float value = -INFINITY;
    uint32_t candidates = 33;
    if constexpr (V >= 2) {
      // The `top`-th largest of the lanes' own largest is a bound from below on
      // the `top` largest of all.  What reaches it -- hardly more than `top` --
      // goes to one lane each, in the order of the indexes, and counts how many
      // come before it: half the instructions of a search for each choice
      // (16384 rows of 256, 8 choices: 15.4 us that way).
      uint32_t best = first;
      for (int j = 1; j < a.top && best != 0u; ++j) {
        if (largest == best) largest = 0u;
        best = __reduce_max_sync(0xffffffffu, largest);
      }
      // fewer than `top` lanes: all that are not masked
      const float bound = best == 0u ? -FLT_MAX : key_value(best);
      candidates = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = l[v] >= bound;
        const uint32_t with = __ballot_sync(0xffffffffu, in);
        const uint32_t at = candidates + __popc(with & ((1u << lane) - 1u));
        if (in && at < 32u) list[at] = make_uint2(__float_as_uint(l[v]), v * 32 + lane);
        candidates += __popc(with);
      }
      if (candidates <= 32u) {
        __syncwarp();
        const uint2 c = list[lane];
        const uint32_t k = lane < candidates ? logit_key(__uint_as_float(c.x)) : 0u;
        place = 0;
        for (uint32_t i = 0; i < candidates; ++i) {
          const uint32_t other = __shfl_sync(0xffffffffu, k, i);
          place += other > k || (other == k && i < lane) ? 1 : 0;
        }
        if (lane < candidates && place < a.top) {
          mine = static_cast<int>(c.y);
          value = __uint_as_float(c.x);
        } else if (lane >= candidates) {
          place = lane;  // choices that cannot be made
        }
        __syncwarp();
      }
    }
    if (candidates > 32u) {
      uint32_t key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = logit_key(l[v]);
      for (int j = 0; j < a.top; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) best = max(best, key[v]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0u) break;
        int at = V * 32;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] == best) at = v * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (at == v * 32 + lane) key[v] = 0u;
        if (lane == j) {
          mine = at;
          value = key_value(best);
        }
      }
    }
    const float e = mine < 0 ? 0.0f : expf(value - m);
    float sum = e;
    if (!a.normalize) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += expf(l[v] - m);
    }
    sum = warp_sum(sum);
    if (place < a.top) {
      a.expert[row * a.top + place] = mine;
      a.weight[row * a.top + place] = mine < 0 ? 0.0f : e / sum;
    }
  }
}

struct RouteGradArgs {
  int64_t rows, ld, ldd;
  int experts, top, type, dtype, normalize;
  const void* logits;
  const int32_t* expert;
  const float* dweight;
  void* dlogits;
};

template <int V>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(const __grid_constant__ RouteGradArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    int e = -1;
    float dw = 0.0f, chosen = -INFINITY;
    if (lane < a.top) {
      e = a.expert[row * a.top + lane];
      if (e < 0 || e >= a.experts) e = -1;
    }
    if (e >= 0) {
      dw = a.dweight[row * a.top + lane];
      chosen = load1(a.logits, a.type, row * a.ld + e);
    }
    // the shares of the chosen ones: of themselves alone no other logit is read
    float l[V], most = chosen;
    if (!a.normalize) {
      load_logits(a.logits, a.type, row * a.ld, a.experts, l);
#pragma unroll
      for (int v = 0; v < V; ++v) most = fmaxf(most, l[v]);
    }
    const uint32_t largest = __reduce_max_sync(0xffffffffu, logit_key(most));
    const float m = largest == 0u ? 0.0f : key_value(largest);
    chosen = e >= 0 ? expf(chosen - m) : 0.0f;
    float sum = chosen;
    if (!a.normalize) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        l[v] = expf(l[v] - m);
        sum += l[v];
      }
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float dot = warp_sum(dw * (chosen * inv));
    // this lane's logits: their share's gradient, less the dot
    float g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = a.normalize ? 0.0f : -dot * (l[v] * inv);
    const float mine = (a.normalize ? dw - dot : dw) * (chosen * inv);
    // the choices among them, hardly ever more than two, in their order
    uint32_t todo = 0u;
    for (int j = 0; j < a.top; ++j) {
      const int ej = __shfl_sync(0xffffffffu, e, j);
      if (ej >= 0 && (ej & 31) == lane) todo |= 1u << j;
    }
    while (__any_sync(0xffffffffu, todo != 0u)) {
      const int j = todo != 0u ? __ffs(todo) - 1 : 0;
      const int ej = __shfl_sync(0xffffffffu, e, j);
      const float gj = __shfl_sync(0xffffffffu, mine, j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (todo != 0u && ej == v * 32 + lane) g[v] += gj;
      todo &= todo - 1u;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * 32 + lane;
      if (i < a.experts) store1(a.dlogits, a.dtype, row * a.ldd + i, g[v]);
    }
  }
}

// -------------------------------------------------------------------- sort
// A stable counting sort.  The pairs are cut into one contiguous chunk per CTA
// and that into one contiguous part per warp; a pair's place is its expert's
// first row, plus the expert's pairs in earlier chunks, in the chunk's earlier
// parts, in the part's earlier rounds of 32, and in lower lanes.  Pairs
// without an expert count as one more expert behind the last.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 8;  // rounds whose ids are loaded together, at most

struct SortArgs {
  int64_t n;
  int experts;
  int bits;        // of experts + 1, which stands for lanes without a pair
  int64_t chunk;   // pairs per CTA, a multiple of 32 * kSortWarps
  const int32_t* expert;
  int32_t* slot;
  int32_t* offsets;
  int32_t* source;
  int32_t* counts;  // [CTA][experts + 1]; nullptr: one CTA
};

// Lanes of the warp with this lane's key (below 2^bits; all lanes call it).  By
// a vote per bit: the instruction that compares all lanes takes some 300 cycles
// where their keys differ (131072 pairs over 256 experts: 14.3 us against 8.0).
__device__ __forceinline__ uint32_t same_key(int key, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint32_t v = __ballot_sync(0xffffffffu, one);
    same &= one ? v : ~v;
  }
  return same;
}

__device__ __forceinline__ int sort_key(const SortArgs& a, int64_t i) {
  const int e = a.expert[i];
  return e < 0 || e >= a.experts ? a.experts : e;
}

// Counts of each chunk.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ uint4 dyn_smem[];
  int* cnt = reinterpret_cast<int*>(dyn_smem);
  const int buckets = a.experts + 1;
  for (int g = threadIdx.x; g < buckets; g += kSortThreads) cnt[g] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
  for (int64_t base = lo; base < hi; base += kSortThreads * kSortAhead) {
    int key[kSortAhead];
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
      const int64_t i = base + u * kSortThreads + threadIdx.x;
      key[u] = i < hi ? sort_key(a, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u)
      if (key[u] >= 0) atomicAdd(&cnt[key[u]], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < buckets; g += kSortThreads)
    a.counts[static_cast<int64_t>(blockIdx.x) * buckets + g] = cnt[g];
}

// Shared memory: first[experts + 1], then counts [warp][experts + 1].  AHEAD:
// rounds taken together, so that a whole part needs no branch between them.
template <int AHEAD>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ uint4 dyn_smem[];
  __shared__ int warp_total[kSortWarps];
  __shared__ int carry;
  const int buckets = a.experts + 1;
  int* first = reinterpret_cast<int*>(dyn_smem);
  int* cnt = first + buckets;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* mine = cnt + warp * buckets;
  for (int g = threadIdx.x; g < kSortWarps * buckets; g += kSortThreads) cnt[g] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t part = a.chunk / kSortWarps;
  const int64_t lo = blockIdx.x * a.chunk + warp * part, hi = min(lo + part, a.n);
  const uint32_t below = (1u << lane) - 1u;

  // A part of one batch of rounds keeps its keys, and each pair's place within
  // the part, for the second half; a longer one goes through its pairs again.
  int key[AHEAD], rank[AHEAD];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t i = base + u * 32 + lane;
      key[u] = i < hi ? sort_key(a, i) : buckets;
    }
  };
  // Places of a batch from `mine`, which moves on.  A whole batch runs without
  // branches between its rounds.
  auto count = [&](int64_t base) {
    const bool whole = base + 32 * AHEAD <= hi;
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (!whole && base + u * 32 >= hi) break;
      const uint32_t same = same_key(key[u], a.bits);
      const bool in = key[u] < buckets;
      rank[u] = in ? mine[key[u]] + __popc(same & below) : 0;
      __syncwarp();
      if (in && (same & below) == 0u) mine[key[u]] += __popc(same);
      __syncwarp();
    }
  };
  // What other chunks have of bucket g: in all, and before this one.
  auto others = [&](int g, int& total, int& before) {
    total = before = 0;
    if (g >= buckets || a.counts == nullptr) return;
    const int chunks = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
#pragma unroll 16
    for (int b = 0; b < chunks; ++b) {
      const int c = __ldcg(a.counts + static_cast<int64_t>(b) * buckets + g);
      if (b < me) before += c;
      total += c;
    }
  };
  const bool once = part <= 32 * AHEAD;
  int total, before;
  others(static_cast<int>(threadIdx.x), total, before);
  for (int64_t base = lo; base < hi; base += 32 * AHEAD) {
    load(base);
    count(base);
  }
  __syncthreads();
  // Over the warps, and (several CTAs) over the chunks: what comes before.
  // Then the experts' first rows, 512 at a time.
  for (int g0 = 0; g0 < buckets; g0 += kSortThreads) {
    const int g = g0 + static_cast<int>(threadIdx.x);
    if (g0 > 0) others(g, total, before);
    if (g < buckets) {
      int run = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * buckets + g];
        cnt[w * buckets + g] = run;
        run += c;
      }
      if (a.counts == nullptr) total = run;
    }
    int sum = total;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, s);
      if (lane >= s) sum += v;
    }
    if (lane == 31) warp_total[warp] = sum;
    __syncthreads();
    int start = carry + sum - total;
    for (int w = 0; w < warp; ++w) start += warp_total[w];
    if (g < buckets) {
      first[g] = start + before;
      if (blockIdx.x == 0) a.offsets[g] = start;
    }
    __syncthreads();
    if (threadIdx.x == kSortThreads - 1) carry = start + total;
    __syncthreads();
  }

  for (int64_t base = lo; base < hi; base += 32 * AHEAD) {
    if (!once) {
      load(base);
      count(base);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t i = base + u * 32 + lane;
      if (i >= hi) continue;
      // (`once`: the part's first place was not in `mine` yet)
      const int at = first[key[u]] + rank[u] + (once ? mine[key[u]] : 0);
      const bool real = key[u] < a.experts;
      a.slot[i] = real ? at : -1;
      if (a.source != nullptr) a.source[at] = real ? static_cast<int32_t>(i) : -1;
    }
  }
}

// ----------------------------------------------------------------- dispatch
struct DispatchArgs {
  int64_t rows, n;
  int top;
  const uint8_t* x;
  int64_t x_pitch;    // bytes
  uint8_t* a;
  int64_t a_pitch;
  int64_t pieces;     // of a row: units of the copy's width
  int tpr;            // threads per row
  int64_t row_ctas;   // CTAs that copy rows; the others copy scales
  int64_t kb;
  const float* xs;
  int64_t ld_xs;
  float* as;
  int64_t ld_as;
  const int32_t* slot;
};

// T: what a thread moves at a time, AHEAD of them on their way together.  Each
// row is read once and written `top` times.
template <typename T, int AHEAD>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ DispatchArgs p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x >= p.row_ctas) {  // scales: consecutive threads on consecutive rows
    if (blockIdx.y > 0) return;
    const int64_t total = p.kb * p.rows;
    const int64_t step = (static_cast<int64_t>(gridDim.x) - p.row_ctas) * kThreads;
    for (int64_t i = (blockIdx.x - p.row_ctas) * kThreads + threadIdx.x; i < total; i += step) {
      const int64_t b = i / p.rows, r = i - b * p.rows;
      const float s = p.xs[b * p.ld_xs + r];
      for (int j = 0; j < p.top; ++j) {
        const int64_t at = p.slot[r * p.top + j];
        if (at >= 0 && at < p.n) p.as[b * p.ld_as + at] = s;
      }
    }
    return;
  }
  const int per_cta = kThreads / p.tpr;
  const int t = threadIdx.x % p.tpr;
  for (int64_t row = blockIdx.x * per_cta + threadIdx.x / p.tpr; row < p.rows;
       row += p.row_ctas * per_cta) {
    const T* from = reinterpret_cast<const T*>(p.x + row * p.x_pitch);
    const int32_t* slot = p.slot + row * p.top;
    const int64_t wide = static_cast<int64_t>(p.tpr) * AHEAD;
    for (int64_t c = blockIdx.y * wide + t; c < p.pieces; c += gridDim.y * wide) {
      T v[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (c + u * p.tpr < p.pieces) v[u] = __ldcs(from + c + u * p.tpr);
      for (int j = 0; j < p.top; ++j) {
        const int64_t at = slot[j];
        if (at < 0 || at >= p.n) continue;
        T* to = reinterpret_cast<T*>(p.a + at * p.a_pitch);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (c + u * p.tpr < p.pieces) to[c + u * p.tpr] = v[u];
      }
    }
  }
}

// ------------------------------------------------------------------ combine
struct CombineArgs {
  int64_t rows, n;
  int dim, top, tpr;
  const void* a;
  int64_t lda;
  int a_type;
  const int32_t* slot;
  const float* weight;    // nullptr: 1
  const void* residual;   // nullptr: none
  int64_t ldr;
  int r_type;
  void* out;
  int64_t ldo;
  int o_type;
};

template <bool VEC>
__device__ __forceinline__ int chunk_col(int chunk) {
  return VEC ? chunk * 8 : (chunk >> 4) * kFp8Block + (chunk & 15);
}

// A thread makes eight elements of a row, adding the choices in their order;
// the rows of AHEAD choices are on their way at a time.
template <bool VEC, int TA, int AHEAD>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineArgs p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int per_cta = kThreads / p.tpr;
  const int t = threadIdx.x % p.tpr;
  const int chunks = VEC ? p.dim / 8 : (p.dim + kFp8Block - 1) / kFp8Block * 16;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + threadIdx.x / p.tpr;
  if (row >= p.rows) return;
  for (int chunk = blockIdx.y * p.tpr + t; chunk < chunks; chunk += gridDim.y * p.tpr) {
    const int c = chunk_col<VEC>(chunk);
    if (c >= p.dim) continue;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (p.residual != nullptr)
      widen8<VEC, kAnyType>(load8<VEC, kAnyType>(p.residual, p.r_type, row * p.ldr, c, p.dim, true),
                            p.r_type, sum);
    for (int j0 = 0; j0 < p.top; j0 += AHEAD) {
      Raw8<TA> raw[AHEAD];
      float w[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int j = j0 + u;
        const int64_t at = j < p.top ? p.slot[row * p.top + j] : -1;
        const bool in = at >= 0 && at < p.n;
        raw[u] = load8<VEC, TA>(p.a, p.a_type, at * p.lda, c, p.dim, in);
        w[u] = !in ? 0.0f : (p.weight == nullptr ? 1.0f : p.weight[row * p.top + j]);
        // a pair without a row adds nothing, whatever its weight
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        float v[8];
        widen8<VEC, TA>(raw[u], p.a_type, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[u], v[i], sum[i]);
      }
    }
    store8<VEC>(p.out, p.o_type, row * p.ldo, c, p.dim, sum);
  }
}

struct CombineGradArgs {
  int64_t rows, n;
  int dim, top, tpr;  // tpr: 32 or kThreads
  const void* dout;
  int64_t lddo;
  int do_type;
  const void* a;
  int64_t lda;
  int a_type;
  const int32_t* slot;
  const float* weight;
  void* da;           // or nullptr
  int64_t ldda;
  int da_type;
  float* dweight;     // or nullptr
};

// One warp or one CTA per row: the row of dout is read once for CHOICES
// choices, whose products with it are summed over the row at the end.
template <bool VEC, int TD, int TA, int CHOICES>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const __grid_constant__ CombineGradArgs p) {
  __shared__ float red[kWarps][CHOICES];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = kThreads / p.tpr;
  const int t = threadIdx.x % p.tpr;
  const int chunks = VEC ? p.dim / 8 : (p.dim + kFp8Block - 1) / kFp8Block * 16;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + threadIdx.x / p.tpr; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * per_cta) {
    // (one at a time: those of a row may be in CTAs of their own)
    const int first = CHOICES == 1 ? static_cast<int>(blockIdx.y) : 0;
    const int step = CHOICES == 1 ? static_cast<int>(gridDim.y) : CHOICES;
    for (int j0 = first; j0 < p.top; j0 += step) {
      int64_t at[CHOICES];
      float w[CHOICES], dot[CHOICES];
#pragma unroll
      for (int u = 0; u < CHOICES; ++u) {
        const int j = j0 + u;
        at[u] = j < p.top ? p.slot[row * p.top + j] : -1;
        if (at[u] >= p.n) at[u] = -1;
        w[u] = at[u] >= 0 ? p.weight[row * p.top + j] : 0.0f;
        dot[u] = 0.0f;
      }
      for (int chunk = t; chunk < chunks; chunk += p.tpr) {
        const int c = chunk_col<VEC>(chunk);
        if (c >= p.dim) continue;
        Raw8<TA> raw[CHOICES];
        const Raw8<TD> rd = load8<VEC, TD>(p.dout, p.do_type, row * p.lddo, c, p.dim, true);
        if (p.dweight != nullptr) {
#pragma unroll
          for (int u = 0; u < CHOICES; ++u)
            raw[u] = load8<VEC, TA>(p.a, p.a_type, at[u] * p.lda, c, p.dim, at[u] >= 0);
        }
        float d[8];
        widen8<VEC, TD>(rd, p.do_type, d);
#pragma unroll
        for (int u = 0; u < CHOICES; ++u) {
          if (at[u] < 0) continue;
          float v[8];
          if (p.dweight != nullptr) {
            widen8<VEC, TA>(raw[u], p.a_type, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[u] = fmaf(d[i], v[i], dot[u]);
          }
          if (p.da != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[u] * d[i];
            store8<VEC>(p.da, p.da_type, at[u] * p.ldda, c, p.dim, v);
          }
        }
      }
      if (p.dweight == nullptr) continue;
#pragma unroll
      for (int u = 0; u < CHOICES; ++u) dot[u] = warp_sum(dot[u]);
      if (p.tpr == 32) {
#pragma unroll
        for (int u = 0; u < CHOICES; ++u)
          if (lane == u && j0 + u < p.top) p.dweight[row * p.top + j0 + u] = dot[u];
        continue;
      }
      __syncthreads();  // the previous sums have been read
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < CHOICES; ++u) red[warp][u] = dot[u];
      }
      __syncthreads();
      if (threadIdx.x < CHOICES && j0 + static_cast<int>(threadIdx.x) < p.top) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += red[i][threadIdx.x];
        p.dweight[row * p.top + j0 + threadIdx.x] = s;
      }
    }
  }
}

// -------------------------------------------------------------- host pieces
bool ids_ok(const void* p, int bytes = 4) { return p != nullptr && !ops_misaligned(p, bytes); }

// A row-major array of fp32 or bf16; vec is cleared where its rows cannot be
// moved in 16-byte pieces.
bool rows_ok(const void* p, int type, int64_t ld, int64_t rows, int64_t dim, bool& vec) {
  const int bytes = float_type_bytes(type);
  if (p == nullptr || bytes == 0 || ld < dim || ld > kOpsMaxDim || ops_misaligned(p, bytes)) return false;
  if (ops_misaligned(p, 16) || (rows > 1 && ld % (16 / bytes) != 0)) vec = false;
  return true;
}

gemm_status_t check_route(int64_t rows, int64_t G, int64_t top, const void* logits, int64_t ld, int type) {
  const int bytes = float_type_bytes(type);
  if (rows < 0 || G < 0 || top < 0 || top > G || bytes == 0 || rows > kOpsMaxDim || G > kOpsMaxDim ||
      rows * top > kOpsMaxDim)
    return GEMM_ERR_INVALID_VALUE;
  if (rows > 0 && G > 0 &&
      (logits == nullptr || ld < G || ld > kOpsMaxDim || ops_misaligned(logits, bytes)))
    return GEMM_ERR_INVALID_VALUE;
  if (G > kMaxGroups || top > kMaxTop) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

template <template <int> class Launch, typename A>
cudaError_t by_experts(int experts, const A& a, int64_t rows, int num_sms, cudaStream_t s) {
  const int64_t ctas = (rows + kWarps - 1) / kWarps, fit = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(ctas < fit ? ctas : fit));
  if (experts <= 32) return Launch<1>::go(grid, a, s);
  if (experts <= 64) return Launch<2>::go(grid, a, s);
  if (experts <= 128) return Launch<4>::go(grid, a, s);
  if (experts <= 256) return Launch<8>::go(grid, a, s);
  if (experts <= 512) return Launch<16>::go(grid, a, s);
  return Launch<32>::go(grid, a, s);
}

template <int V>
struct LaunchRoute {
  static cudaError_t go(dim3 grid, const RouteArgs& a, cudaStream_t s) {
    return ops_launch<route_kernel<V>>(grid, kThreads, 0, 1, s, a);
  }
};
template <int V>
struct LaunchRouteGrad {
  static cudaError_t go(dim3 grid, const RouteGradArgs& a, cudaStream_t s) {
    return ops_launch<route_grad_kernel<V>>(grid, kThreads, 0, 1, s, a);
  }
};

// Pairs of a launch with one CTA, and pairs per CTA of one with several (as
// many CTAs as kSortMostCtas).  Every CTA's walk over the chunks' counts is what
// large sorts take: 131072 pairs over 128 experts 6.7 us (64 chunks), 262144 11.8
// (128), 524288 15.8 and 1048576 16.2 (256 both).  Chunks of 1024 and 4096 instead: 131072 pairs
// over 256 experts 9.8 and 8.0 us against 6.7, 32768 over 64 5.2 and 8.3
// against 5.2.
constexpr int64_t kSortSingle = 4096;
constexpr int64_t kSortChunk = 2048;
constexpr int64_t kSortMostCtas = 256;

template <typename T>
cudaError_t launch_dispatch(DispatchArgs& p, int64_t row_bytes, int num_sms, cudaStream_t s) {
  p.pieces = row_bytes / static_cast<int64_t>(sizeof(T));
  // Few pieces: one a thread, rows cut into several CTAs (16 x 4096 bf16, eight
  // choices each 2.1 us, 3.5 with four a thread).
  const bool few = p.rows * p.pieces <= static_cast<int64_t>(num_sms) * kThreads;
  const int ahead = few ? 1 : 4;
  p.tpr = 32;
  while (p.tpr < kThreads && p.pieces > static_cast<int64_t>(p.tpr) * ahead) p.tpr *= 2;
  const int64_t per_cta = kThreads / p.tpr;
  const int64_t want = (p.rows + per_cta - 1) / per_cta, fit = static_cast<int64_t>(num_sms) * 64;
  p.row_ctas = want < fit ? want : fit;
  int64_t scale_ctas = 0;
  if (p.as != nullptr) {
    scale_ctas = (p.kb * p.rows + kThreads - 1) / kThreads;
    if (scale_ctas > fit) scale_ctas = fit;
  }
  const unsigned ctas = static_cast<unsigned>(p.row_ctas + scale_ctas);
  if (few)
    return ops_launch<dispatch_kernel<T, 1>>(dim3(ctas, static_cast<unsigned>((p.pieces + p.tpr - 1) / p.tpr)),
                                             kThreads, 0, 1, s, p);
  return ops_launch<dispatch_kernel<T, 4>>(dim3(ctas), kThreads, 0, 1, s, p);
}

template <bool VEC, int TA>
cudaError_t launch_combine(CombineArgs& p, cudaStream_t s) {
  const int64_t chunks = VEC ? p.dim / 8 : (p.dim + kFp8Block - 1) / kFp8Block * 16;
  p.tpr = 8;
  while (p.tpr < kThreads && chunks > p.tpr) p.tpr *= 2;
  const int64_t per_cta = kThreads / p.tpr, across = (chunks + p.tpr - 1) / p.tpr;
  const dim3 grid(static_cast<unsigned>((p.rows + per_cta - 1) / per_cta),
                  static_cast<unsigned>(across < 65535 ? across : 65535));
  // As many choices ahead as there are, or as the registers hold (8192 rows of
  // 4096 in bf16 with a residual, always 8 ahead: 73 us for one choice, 76 for
  // two, 67 for four without one; here 41, 47 and 52).
  if constexpr (VEC) {
    if (p.top == 1) return ops_launch<combine_kernel<VEC, TA, 1>>(grid, kThreads, 0, 1, s, p);
    if (p.top == 2) return ops_launch<combine_kernel<VEC, TA, 2>>(grid, kThreads, 0, 1, s, p);
    if (TA == GEMM_OUT_BF16 && p.top > 4)
      return ops_launch<combine_kernel<VEC, TA, 8>>(grid, kThreads, 0, 1, s, p);
  }
  return ops_launch<combine_kernel<VEC, TA, 4>>(grid, kThreads, 0, 1, s, p);
}

template <bool VEC, int TD, int TA>
cudaError_t launch_combine_grad(CombineGradArgs& p, int num_sms, cudaStream_t s) {
  const int64_t chunks = VEC ? p.dim / 8 : (p.dim + kFp8Block - 1) / kFp8Block * 16;
  // A warp a row up to 1024 elements, and to 2048 if there are enough rows (a CTA
  // and a warp a row: 1024 x 2048 bf16, eight choices 10.8 and 18.8 us, 2048 x 1024,
  // four 8.5 and 5.5).
  const bool warp = chunks <= 128 || (chunks <= 256 && p.rows > static_cast<int64_t>(num_sms) * 2 * kWarps);
  p.tpr = warp ? 32 : kThreads;
  const int64_t per_cta = kThreads / p.tpr;
  const int64_t want = (p.rows + per_cta - 1) / per_cta, fit = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(want < fit ? want : fit));
  if constexpr (VEC) {
    // Few rows: every choice for itself (16 x 4096 bf16, eight choices 2.5 us, 4.8
    // four at a time).
    const bool few = p.top > 4 && p.rows * p.top <= static_cast<int64_t>(num_sms) * 4 * per_cta;
    if (few || p.top == 1)
      return ops_launch<combine_grad_kernel<VEC, TD, TA, 1>>(
          dim3(grid.x, static_cast<unsigned>(few ? p.top : 1)), kThreads, 0, 1, s, p);
    if (p.top == 2) return ops_launch<combine_grad_kernel<VEC, TD, TA, 2>>(grid, kThreads, 0, 1, s, p);
  }
  return ops_launch<combine_grad_kernel<VEC, TD, TA, 4>>(grid, kThreads, 0, 1, s, p);
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" {

gemm_status_t gemm_expert_route(int64_t rows, int64_t G, int64_t top, const void* logits, int64_t ld,
                                int logits_type, int normalize, int32_t* expert, float* weight,
                                void* stream) {
  gemm_status_t st = check_route(rows, G, top, logits, ld, logits_type);
  if (st != GEMM_OK) return st;
  if (rows == 0 || top == 0) return GEMM_OK;
  if (!ids_ok(expert) || !ids_ok(weight)) return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  uint32_t* err = nullptr;
  st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  const RouteArgs a{rows, ld, static_cast<int>(G), static_cast<int>(top), logits_type, normalize != 0,
                    logits, expert, weight};
  return abi_from_cuda(by_experts<LaunchRoute>(a.experts, a, rows, sms, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_expert_route_backward(int64_t rows, int64_t G, int64_t top, const void* logits,
                                         int64_t ld, int logits_type, int normalize,
                                         const int32_t* expert, const float* dweight, void* dlogits,
                                         int64_t ldd, int dlogits_type, void* stream) {
  gemm_status_t st = check_route(rows, G, top, logits, ld, logits_type);
  if (st != GEMM_OK) return st;
  const int bytes = float_type_bytes(dlogits_type);
  if (bytes == 0) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || G == 0) return GEMM_OK;
  if (dlogits == nullptr || ldd < G || ldd > kOpsMaxDim || ops_misaligned(dlogits, bytes) ||
      (top > 0 && (!ids_ok(expert) || !ids_ok(dweight))))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  uint32_t* err = nullptr;
  st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  const RouteGradArgs a{rows, ld, ldd, static_cast<int>(G), static_cast<int>(top), logits_type,
                        dlogits_type, normalize != 0, logits, expert, dweight, dlogits};
  return abi_from_cuda(
      by_experts<LaunchRouteGrad>(a.experts, a, rows, sms, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_expert_sort(int64_t n, int64_t G, const int32_t* expert, int32_t* slot,
                               int32_t* offsets, int32_t* source, void* stream) {
  if (n < 0 || G < 0 || n > kOpsMaxDim || !ids_ok(offsets)) return GEMM_ERR_INVALID_VALUE;
  if (n > 0 && (!ids_ok(expert) || !ids_ok(slot))) return GEMM_ERR_INVALID_VALUE;
  if (source != nullptr && ops_misaligned(source, 4)) return GEMM_ERR_INVALID_VALUE;
  if (G > kMaxGroups) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  SortArgs a{};
  a.n = n;
  a.experts = static_cast<int>(G);
  a.expert = expert;
  a.slot = slot;
  a.offsets = offsets;
  a.source = source;
  const size_t buckets = static_cast<size_t>(G) + 1;
  const size_t smem = sizeof(int) * buckets * (1 + kSortWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::unique_lock<std::mutex> lock;
  int64_t ctas = 1;
  if (n > kSortSingle) {
    ctas = (n + kSortChunk - 1) / kSortChunk;
    if (ctas > kSortMostCtas) ctas = kSortMostCtas;
    float* ws = nullptr;
    st = abi_scratch(s, ctas * static_cast<int64_t>(buckets), lock, &ws);
    if (st != GEMM_OK) return st;
    a.counts = reinterpret_cast<int32_t*>(ws);
  }
  while ((1 << a.bits) < a.experts + 2) ++a.bits;
  const int64_t unit = 32 * kSortWarps;
  a.chunk = ((n + ctas - 1) / ctas + unit - 1) / unit * unit;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (ctas > 1) {
    const cudaError_t e = ops_launch<sort_count_kernel>(grid, kSortThreads, sizeof(int) * buckets, 1, s, a);
    if (e != cudaSuccess) return abi_from_cuda(e);
  }
  if (a.chunk <= 4 * unit)
    return abi_from_cuda(ops_launch<sort_place_kernel<4>>(grid, kSortThreads, smem, 1, s, a));
  return abi_from_cuda(ops_launch<sort_place_kernel<kSortAhead>>(grid, kSortThreads, smem, 1, s, a));
}

gemm_status_t gemm_expert_dispatch(int64_t rows, int64_t top, int64_t n, int64_t dim, int elem_bytes,
                                   const void* x, int64_t ldx, const int32_t* slot, void* a, int64_t lda,
                                   const float* x_scales, int64_t ld_xs, float* a_scales, int64_t ld_as,
                                   void* stream) {
  if (rows < 0 || top < 0 || n < 0 || dim < 0 || rows > kOpsMaxDim || n > kOpsMaxDim ||
      dim > kOpsMaxDim || top > kOpsMaxDim || rows * top > kOpsMaxDim ||
      (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4))
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || top == 0 || n == 0 || dim == 0) return GEMM_OK;
  if ((x_scales == nullptr) != (a_scales == nullptr) || x == nullptr || a == nullptr || !ids_ok(slot) ||
      ldx < dim || lda < dim || ldx > kOpsMaxDim || lda > kOpsMaxDim || ops_misaligned(x, elem_bytes) ||
      ops_misaligned(a, elem_bytes))
    return GEMM_ERR_INVALID_VALUE;
  const bool one = x_scales != nullptr && ld_xs == 0 && ld_as == 0;  // scale for each row
  if (x_scales != nullptr && (ops_misaligned(x_scales, 4) || ops_misaligned(a_scales, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if (x_scales != nullptr && !one &&
      (ld_xs < rows || ld_as < n || ld_xs > kOpsMaxDim || ld_as > kOpsMaxDim))
    return GEMM_ERR_INVALID_VALUE;
  if (top > kMaxTop) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  DispatchArgs p{};
  p.rows = rows;
  p.n = n;
  p.top = static_cast<int>(top);
  p.x = static_cast<const uint8_t*>(x);
  p.x_pitch = ldx * elem_bytes;
  p.a = static_cast<uint8_t*>(a);
  p.a_pitch = lda * elem_bytes;
  p.kb = one ? 1 : (dim + kFp8Block - 1) / kFp8Block;
  p.xs = x_scales;
  p.ld_xs = ld_xs;
  p.as = a_scales;
  p.ld_as = ld_as;
  p.slot = slot;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t bytes = dim * elem_bytes;
  // the widest unit that every row's start and length allow
  const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(a) |
                       static_cast<uint64_t>(p.x_pitch) | static_cast<uint64_t>(p.a_pitch) |
                       static_cast<uint64_t>(bytes);
  if (all % 16 == 0) return abi_from_cuda(launch_dispatch<uint4>(p, bytes, sms, s));
  if (all % 4 == 0) return abi_from_cuda(launch_dispatch<unsigned int>(p, bytes, sms, s));
  if (all % 2 == 0) return abi_from_cuda(launch_dispatch<unsigned short>(p, bytes, sms, s));
  return abi_from_cuda(launch_dispatch<unsigned char>(p, bytes, sms, s));
}

gemm_status_t gemm_expert_combine(int64_t rows, int64_t top, int64_t n, int64_t dim, const void* a,
                                  int64_t lda, int a_type, const int32_t* slot, const float* weight,
                                  const void* residual, int64_t ldr, int residual_type, void* out,
                                  int64_t ldo, int out_type, void* stream) {
  if (rows < 0 || top < 0 || n < 0 || dim < 0 || rows > kOpsMaxDim || n > kOpsMaxDim ||
      dim > (int64_t{1} << 30) || top > kOpsMaxDim || rows * top > kOpsMaxDim ||
      float_type_bytes(a_type) == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || dim == 0) return GEMM_OK;
  bool vec = dim % 8 == 0;
  if (!rows_ok(out, out_type, ldo, rows, dim, vec)) return GEMM_ERR_INVALID_VALUE;
  if (residual != nullptr && !rows_ok(residual, residual_type, ldr, rows, dim, vec))
    return GEMM_ERR_INVALID_VALUE;
  if (top > 0 && (!ids_ok(slot) || (weight != nullptr && ops_misaligned(weight, 4))))
    return GEMM_ERR_INVALID_VALUE;
  if (top > 0 && n > 0 && !rows_ok(a, a_type, lda, n, dim, vec)) return GEMM_ERR_INVALID_VALUE;
  if (top > kMaxTop) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  CombineArgs p{rows, n, static_cast<int>(dim), n > 0 ? static_cast<int>(top) : 0, 0, a, lda, a_type,
                slot, weight, residual, ldr, residual_type, out, ldo, out_type};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!vec) return abi_from_cuda(launch_combine<false, kAnyType>(p, s));
  return abi_from_cuda(a_type == GEMM_OUT_BF16 ? launch_combine<true, GEMM_OUT_BF16>(p, s)
                                               : launch_combine<true, GEMM_OUT_F32>(p, s));
}

gemm_status_t gemm_expert_combine_backward(int64_t rows, int64_t top, int64_t n, int64_t dim,
                                           const void* dout, int64_t lddo, int dout_type, const void* a,
                                           int64_t lda, int a_type, const int32_t* slot,
                                           const float* weight, void* da, int64_t ldda, int da_type,
                                           float* dweight, void* stream) {
  if (rows < 0 || top < 0 || n < 0 || dim < 0 || rows > kOpsMaxDim || n > kOpsMaxDim ||
      dim > (int64_t{1} << 30) || top > kOpsMaxDim || rows * top > kOpsMaxDim ||
      float_type_bytes(dout_type) == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || top == 0 || (da == nullptr && dweight == nullptr)) return GEMM_OK;
  bool vec = dim % 8 == 0;
  if (!ids_ok(slot) || !ids_ok(weight) || (dweight != nullptr && ops_misaligned(dweight, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if (dim > 0 && !rows_ok(dout, dout_type, lddo, rows, dim, vec)) return GEMM_ERR_INVALID_VALUE;
  // (`a` is read for dweight only)
  if (dim > 0 && n > 0 && dweight != nullptr && !rows_ok(a, a_type, lda, n, dim, vec))
    return GEMM_ERR_INVALID_VALUE;
  if (dim > 0 && n > 0 && da != nullptr && !rows_ok(da, da_type, ldda, n, dim, vec))
    return GEMM_ERR_INVALID_VALUE;
  if (top > kMaxTop) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  CombineGradArgs p{rows, n, static_cast<int>(dim), static_cast<int>(top), 0, dout, lddo, dout_type,
                    a, lda, a_type, slot, weight, da, ldda, da_type, dweight};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  constexpr int B = GEMM_OUT_BF16, F = GEMM_OUT_F32;
  if (!vec) return abi_from_cuda(launch_combine_grad<false, kAnyType, kAnyType>(p, sms, s));
  const bool ab = dweight == nullptr ? dout_type == B : a_type == B;
  if (dout_type == B)
    return abi_from_cuda(ab ? launch_combine_grad<true, B, B>(p, sms, s)
                            : launch_combine_grad<true, B, F>(p, sms, s));
  return abi_from_cuda(ab ? launch_combine_grad<true, F, B>(p, sms, s)
                          : launch_combine_grad<true, F, F>(p, sms, s));
}

}  // extern "C"
