// Log probabilities of given tokens, with entropy and top alternatives, and
// their gradient with respect to the logits.
//
// With m the row's largest logit, a row is reduced to
//   S = sum 2^y,  T = sum y 2^y,  y = (x - m) log2 e,
// so that ln p_v = x_v - m - ln S and the entropy is ln S - ln 2 T/S. One pass
// over the row: the sums are taken with the shift of a logit c near the
// largest so far (a warp's first tile sets it, and it is raised only where
// logits exceed it by more than kSlack), and moved to m at the end. Lanes each
// raising their own c in every tile cost 9.4 instructions an element against
// 7.8 so, and 228 us against 167 for 4,096 rows of 129,280 bf16.
//
// What bounds it: reading the rows. 4,096 x 129,280 bf16 takes 167 us, 6.3
// TB/s (97% of the copy rate), and 197 us where the card's power cap holds the
// SM clock at 1.67 GHz: bf16 rows need 70% of the exponential unit's rate at
// full clock. 592 x 151,936 fp32: 56 us, 6.4 TB/s. Few rows are bound by
// latency: 5.2 us for one row of 151,936 by a cluster of 8 CTAs, of which 3.0
// remain with no tile to read; 20 alternatives add 5 us.
#include <algorithm>

#include "elements.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr long long kMaxStride = 1ll << 32;
// exponents below this give 2^y = 0; the clamp keeps y 2^y from being -inf * 0
constexpr float kMinExp = -16384.f;

struct ScoreArgs {
  const void* logits;
  long long n_rows, stride;
  const int64_t* row_start;
  const int32_t* tokens;
  int C, V, top_k;
  float* logprob;
  float* entropy;
  float* stats;
  int32_t* top_tokens;
  float* top_logprobs;
  unsigned* err;
  int items;
  int parts;   // CTAs of a cluster, each with an equal part of the row
  int gather;  // the items left out come last in the grid
  int group;   // rows of 32 vectors of a segment (alternatives): 1, or a multiple of kAhead
  int room;    // candidates that shared memory holds
};

struct GradArgs {
  const void* logits;
  long long stride, gstride;
  const int32_t* tokens;
  const float* stats;
  const float* entropy;
  const float* g_logprob;
  const float* g_entropy;
  int V;
  void* dlogits;
  unsigned* err;
  int pieces;  // CTAs of a row
};

// 2^y, relative error below 2^-22; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// The j-th pair of a 16-byte vector's elements, and the vector's length.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kLen = 4;
  static constexpr unsigned kNegInf = 0xff800000u;
  __device__ __forceinline__ static F2 pair(const uint4& v, int j) {
    return j == 0 ? f2(__uint_as_float(v.x), __uint_as_float(v.y)) : f2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static uint4 pack(const F2 (&d)[2]) {
    return make_uint4(__float_as_uint(f2_lo(d[0])), __float_as_uint(f2_hi(d[0])), __float_as_uint(f2_lo(d[1])),
                      __float_as_uint(f2_hi(d[1])));
  }
  // the elements, none below -1e38 (near terms: y stays finite, 2^y is 0)
  __device__ __forceinline__ static uint4 floor(const uint4& v) {
    return make_uint4(__float_as_uint(fmax_nan(__uint_as_float(v.x), -1e38f)),
                      __float_as_uint(fmax_nan(__uint_as_float(v.y), -1e38f)),
                      __float_as_uint(fmax_nan(__uint_as_float(v.z), -1e38f)),
                      __float_as_uint(fmax_nan(__uint_as_float(v.w), -1e38f)));
  }
  __device__ __forceinline__ static float largest(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int kLen = 8;
  static constexpr unsigned kNegInf = 0xff80ff80u;
  __device__ __forceinline__ static F2 pair(const uint4& v, int j) {
    const unsigned u = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
    return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  __device__ __forceinline__ static uint4 pack(const F2 (&d)[4]) {
    return make_uint4(pack_bf16(f2_lo(d[0]), f2_hi(d[0])), pack_bf16(f2_lo(d[1]), f2_hi(d[1])),
                      pack_bf16(f2_lo(d[2]), f2_hi(d[2])), pack_bf16(f2_lo(d[3]), f2_hi(d[3])));
  }
  __device__ __forceinline__ static unsigned max2(unsigned a, unsigned b) {   // NaN gives way
    unsigned d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ static uint4 floor(const uint4& v) {
    constexpr unsigned kLow = 0xfe96fe96u;   // -1e38
    uint4 d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d.x) : "r"(v.x), "r"(kLow));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d.y) : "r"(v.y), "r"(kLow));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d.z) : "r"(v.z), "r"(kLow));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d.w) : "r"(v.w), "r"(kLow));
    return d;
  }
  __device__ __forceinline__ static float largest(const uint4& v) {
    const unsigned m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};

// A row as 16-byte vectors: `head` elements in front of the first aligned one,
// nvec vectors, `tail` elements behind.
template <typename T>
struct Row {
  const T* x;
  int head, nvec, tail;
  __device__ __forceinline__ Row(const T* p, int V) : x(p) {
    constexpr int E = Vec<T>::kLen;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    head = min(V, (E - off) % E);
    nvec = (V - head) / E;
    tail = V - head - nvec * E;
  }
  __device__ __forceinline__ const uint4* vecs() const { return reinterpret_cast<const uint4*>(x + head); }
};

// --------------------------------------------------------------- scores

constexpr int kAhead = 4;                 // vectors of a lane in flight
constexpr int kTile = 32 * kAhead;        // vectors of a tile: one warp, one step
constexpr int kMaxWarps = 8;
// Items up to which the items left out come last in the grid: every CTA then
// reads all tokens first (576 items 32.3 -> 29.9 us, 2,176 65.4 -> 62.0; 4,352
// 122.3 -> 123.6, 8,704 190 -> 227).
constexpr int kGather = 2560;
constexpr int kMaxParts = 8;              // CTAs of a row (the portable cluster size)
constexpr int kMaxSegs = 256;             // segments of a CTA's part
constexpr float kSlack = 4.f;             // how far logits may exceed the sums' c before it is raised
constexpr int kRoom = 2048;               // candidates beside the top_k that are kept

// Sum and tilted sum of some elements of a row with the shift of a logit c
// near their largest: S = sum 2^y, T = sum y 2^y, y = x log2 e - shift2(c);
// c = -inf: no finite element, S and T are 0 (or NaN).
struct Sums {
  float c;
  double S, T;
};

// Up to kNear the terms take one fused step, y = fl(x log2 e - h) with
// h = fl(c log2 e): h is the same number in every term, so its rounding (at
// most 2^-7 there) cancels, and the sum's shift is h. Beyond, the difference
// x - c is taken first.
constexpr float kNear = 65536.f;
__device__ __forceinline__ bool is_near(float c) { return fabsf(c) < kNear; }
__device__ __forceinline__ double shift2(float c) {
  return is_near(c) ? static_cast<double>(c * kLog2e) : static_cast<double>(c) * kLog2e;
}

// Moves the sums to a larger c.
__device__ __forceinline__ void raise(Sums& s, float to) {
  if (!(to > s.c)) return;
  if (s.c != -INFINITY) {
    const float d = static_cast<float>(shift2(to) - shift2(s.c));
    const double f = ex2(-d);
    s.T = f > 0.0 ? (s.T - d * s.S) * f : s.S * 0.0;
    s.S *= f;
  }
  s.c = to;
}

// The sums of eight lanes, 0 to 7, in all of them.
__device__ __forceinline__ Sums join8(Sums s) {
  float c = s.c;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
  raise(s, c);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
    s.T += __shfl_xor_sync(0xffffffffu, s.T, o);
  }
  return s;
}

// Adds the kCount vectors v to a lane's sums; up to 64 terms are added in fp32.
template <typename T, int kCount>
__device__ __forceinline__ void add_terms(const uint4 (&v)[kCount], Sums& sums) {
  const bool near = is_near(sums.c);
  const float h = sums.c * kLog2e, shift = sums.c == -INFINITY ? 0.f : sums.c;
  F2 s = f2(0.f, 0.f), t = f2(0.f, 0.f);
  if (near) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const uint4 c = Vec<T>::floor(v[k]);
#pragma unroll
      for (int j = 0; j < Vec<T>::kLen / 2; ++j) {
        const F2 y = fma2(Vec<T>::pair(c, j), f2(kLog2e, kLog2e), f2(-h, -h));
        const F2 e = f2(ex2(f2_lo(y)), ex2(f2_hi(y)));
        s = add2(s, e);
        t = fma2(e, y, t);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kCount; ++k)
#pragma unroll
      for (int j = 0; j < Vec<T>::kLen / 2; ++j) {
        const F2 x = Vec<T>::pair(v[k], j);
        const F2 y = f2(fmax_nan((f2_lo(x) - shift) * kLog2e, kMinExp), fmax_nan((f2_hi(x) - shift) * kLog2e, kMinExp));
        const F2 e = f2(ex2(f2_lo(y)), ex2(f2_hi(y)));
        s = add2(s, e);
        t = fma2(e, y, t);
      }
  }
  sums.S += static_cast<double>(f2_lo(s) + f2_hi(s));
  sums.T += static_cast<double>(f2_lo(t) + f2_hi(t));
}

// The alternatives' order as one number: the logit's order (-0 as 0), then the
// lowest token. No alternative is 0. NaN and -inf are no candidates.
__device__ __forceinline__ unsigned order_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ unsigned long long rank_key(float x, int v) {
  return (static_cast<unsigned long long>(order_of(x)) << 32) | (0xffffffffu - static_cast<unsigned>(v));
}
__device__ __forceinline__ float order_value(unsigned o) {
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ int key_token(unsigned long long k) {
  return static_cast<int>(0xffffffffu - static_cast<unsigned>(k));
}

// Descending order over a warp's lanes: a bitonic sort, and the 32 largest of
// two sorted sets (the larger of one's i-th and the other's 31-i-th is a
// bitonic sequence of them).
__device__ __forceinline__ unsigned long long exchange(unsigned long long key, int distance, bool larger) {
  const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, distance);
  return (key > other) == larger ? key : other;
}
__device__ __forceinline__ unsigned long long clean32(unsigned long long key, int lane) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) key = exchange(key, d, (lane & d) == 0);
  return key;
}
__device__ __forceinline__ unsigned long long sort32(unsigned long long key, int lane) {
#pragma unroll
  for (int size = 2; size < 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d > 0; d >>= 1) key = exchange(key, d, ((lane & size) == 0) == ((lane & d) == 0));
  return clean32(key, lane);
}
__device__ __forceinline__ unsigned long long merge32(unsigned long long a, unsigned long long b, int lane) {
  b = __shfl_sync(0xffffffffu, b, 31 - lane);
  return clean32(a > b ? a : b, lane);
}

// The 32 largest of n keys in order (0 behind the n-th) to warp 0's lanes and
// to `out`: each warp sorts its share of the keys by 32, then the warps' best
// are merged in pairs. All warps of the CTA call; `out` is ready when they
// return. Keys are different, or 0.
template <typename Key>
__device__ __forceinline__ void take_largest(int n, Key key, unsigned long long (*s_best)[32],
                                             unsigned long long* out) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5;
  const int busy = min(W, (n + 31) / 32);
  unsigned long long best = 0ull;
  for (int i = w * 32; i < n; i += W * 32) {
    const unsigned long long more = sort32(i + lane < n ? key(i + lane) : 0ull, lane);
    best = i == w * 32 ? more : merge32(best, more, lane);
  }
  if (w != 0 && w < busy) s_best[w][lane] = best;
  for (int step = 1; step < busy; step *= 2) {
    __syncthreads();
    if (w % (2 * step) == 0 && w + step < busy) {
      best = merge32(best, s_best[w + step][lane], lane);
      if (w != 0) s_best[w][lane] = best;
    }
  }
  if (w == 0) out[lane] = best;
  __syncthreads();
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Writes the first CTA's copy of a shared 64-bit word.
__device__ __forceinline__ void write_first(const void* p, unsigned long long v) {
  unsigned a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
               : "=r"(a)
               : "r"(static_cast<unsigned>(__cvta_generic_to_shared(p))));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// The item that comes `index`-th when the items left out (token -1) come last:
// otherwise a batch's short requests leave some SMs with four rows to read
// and others with none. Each CTA counts all tokens by itself; the order is by
// the thread that looks at an item, the same in every CTA.
__device__ int gathered_item(const int32_t* tokens, int items, int index, int* s_before, int* s_item) {
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, nt = blockDim.x;
  int used = 0, seen = 0;
  for (int i = tid; i < items; i += nt) {
    used += __ldg(tokens + i) != -1;
    ++seen;
  }
  int inc = used;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_before[w] = inc;
  __syncthreads();
  int before = inc - used, total = 0;
  for (int j = 0; j < (nt >> 5); ++j) {
    if (j < w) before += s_before[j];
    total += s_before[j];
  }
  // items of the threads in front: items / nt each, and one more of the first
  const int skipped_before = tid * (items / nt) + min(tid, items % nt) - before;
  const bool out = index >= total;
  int rank = out ? index - total - skipped_before : index - before;
  if (rank >= 0 && rank < (out ? seen - used : used))
    for (int i = tid; i < items; i += nt)
      if ((__ldg(tokens + i) != -1) != out && rank-- == 0) *s_item = i;
  __syncthreads();
  return *s_item;
}

// One cluster of `parts` CTAs an item, each with an equal part of the row's
// tiles. Alternatives: the top_k elements lie in the top_k segments with the
// largest maxima (equal ones: the first), because each segment in front of
// another holds an element in front of all of the other's. The pass over the
// row notes the segments' maxima only; the chosen segments are read again for
// the elements that reach the last one's maximum.
//
// A warp steps through tiles of 128 vectors, the next one in flight; 8 warps
// and 64 registers let four CTAs share an SM (8 warps against 16, and 4 vectors
// a lane against 8 without the next tile in flight: 171 against 198 us for the
// bf16 rows above; two tiles in flight and three CTAs measured no faster).
template <typename T, bool kTop>
__global__ void __launch_bounds__(kMaxWarps * 32, 4) logprobs_kernel(ScoreArgs a) {
  constexpr int E = Vec<T>::kLen;
  extern __shared__ unsigned long long s_keys[];        // [room]
  __shared__ unsigned s_seg[kTop ? kMaxSegs : 1];
  __shared__ unsigned long long s_best[kTop ? kMaxWarps : 1][32], s_top[32];
  __shared__ int s_count;
  __shared__ Sums s_sums[kMaxWarps];
  __shared__ float s_m[kMaxWarps];
  __shared__ double s_lse[3];
  // in the first CTA of a cluster: every CTA's largest logit, sums and alternatives
  __shared__ unsigned long long s_peer[kMaxParts][3], s_peer_top[kTop ? kMaxParts : 1][32];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, nt = blockDim.x, W = nt >> 5;
  const int parts = a.parts, part = parts > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int V = a.V, k = a.top_k;
  __shared__ int s_before[kMaxWarps + 1], s_item;
  int item = blockIdx.x / parts;
  if (a.gather) item = gathered_item(a.tokens, a.items, item, s_before, &s_item);
  const int b = item / a.C;
  const int tok = a.tokens[item];
  bool skip = tok == -1;
  const long long row = a.row_start != nullptr ? a.row_start[b] + (item - b * a.C) : static_cast<long long>(item);
  if (!skip && (tok < 0 || tok >= V || row < 0 || row >= a.n_rows)) {
    if (tid == 0 && part == 0) record_bad_item(a.err, item);
    skip = true;
  }
  if (skip) {                       // the same for every CTA of the cluster
    if (part != 0) return;
    if (tid == 0) {
      a.logprob[item] = 0.f;
      if (a.entropy != nullptr) a.entropy[item] = 0.f;
      if (a.stats != nullptr) reinterpret_cast<float2*>(a.stats)[item] = make_float2(0.f, 0.f);
    }
    for (int i = tid; kTop && i < k; i += nt) {
      a.top_tokens[static_cast<long long>(item) * k + i] = -1;
      a.top_logprobs[static_cast<long long>(item) * k + i] = -INFINITY;
    }
    return;
  }
  if (parts > 1) cluster_arrive();  // the first CTA's shared memory is written only once it runs
  const Row<T> r(static_cast<const T*>(a.logits) + row * a.stride, V);
  const uint4* vecs = r.vecs();
  const float xt = part == 0 && tid == 0 ? to_float(r.x[tok]) : 0.f;
  const int tiles = (r.nvec + kTile - 1) / kTile;
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * part / parts);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (part + 1) / parts);
  const int segs = ((t1 - t0) * kAhead + a.group - 1) / a.group;
  if (kTop && a.group > kAhead) {
    for (int i = tid; i < segs; i += nt) s_seg[i] = 0u;
    __syncthreads();
  }

  float m = -INFINITY;                     // the lane's largest logit
  Sums sums{-INFINITY, 0.0, 0.0};          // c is the warp's: the largest logit when it was set
  auto load = [&](uint4 (&v)[kAhead], int t) {
    const int i0 = t * kTile + lane;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const unsigned ni = Vec<T>::kNegInf;
      v[u] = i0 + u * 32 < r.nvec ? __ldg(vecs + i0 + u * 32) : make_uint4(ni, ni, ni, ni);
    }
  };
  uint4 next[kAhead];
  if (t0 + w < t1) load(next, t0 + w);
  for (int t = t0 + w; t < t1; t += W) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = next[u];
    if (t + W < t1) load(next, t + W);
    float most = -INFINITY;
    if (kTop && a.group == 1) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float here = Vec<T>::largest(v[u]);
        const unsigned o = __reduce_max_sync(0xffffffffu, order_of(fmaxf(here, -INFINITY)));
        if (lane == 0) s_seg[(t - t0) * kAhead + u] = o;
        most = fmaxf(most, here);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) most = fmaxf(most, Vec<T>::largest(v[u]));
      if (kTop) {
        const unsigned o = __reduce_max_sync(0xffffffffu, order_of(most));
        if (lane == 0) {
          if (a.group == kAhead)
            s_seg[t - t0] = o;
          else
            atomicMax(&s_seg[(t - t0) * kAhead / a.group], o);
        }
      }
    }
    m = fmaxf(m, most);
    if (__any_sync(0xffffffffu, most > sums.c + kSlack))      // rare behind the first tile
      raise(sums, order_value(__reduce_max_sync(0xffffffffu, order_of(most))));
    add_terms<T>(v, sums);
  }
  // the ends outside the vectors: at most kLen - 1 elements each
  const int ends = (part == 0 ? r.head : 0) + (part == parts - 1 ? r.tail : 0);
  int end_at = -1;
  float end_x = -INFINITY;
  if (w == 0 && ends > 0) {
    if (lane < ends) {
      end_at = part == 0 && lane < r.head ? lane : V - ends + lane;
      end_x = to_float(r.x[end_at]);
    }
    m = fmaxf(m, end_x);
    raise(sums, order_value(__reduce_max_sync(0xffffffffu, order_of(m))));
    if (lane < ends) {
      const float c = sums.c == -INFINITY ? 0.f : sums.c;
      const float y = fmax_nan(is_near(c) ? fmaf(end_x, kLog2e, -(c * kLog2e)) : (end_x - c) * kLog2e, kMinExp);
      const float e = ex2(y);
      sums.S += e;
      sums.T += static_cast<double>(e * y);
    }
  }
  m = order_value(__reduce_max_sync(0xffffffffu, order_of(m)));
  sums.S = warp_sum(sums.S);
  sums.T = warp_sum(sums.T);
  if (lane == 0) {
    s_m[w] = m;
    s_sums[w] = sums;
  }
  if (tid == 0) s_count = 0;
  __syncthreads();
  Sums all{-INFINITY, 0.0, 0.0};
  if (w == 0) {
    m = -INFINITY;
    if (lane < W) {
      all = s_sums[lane];
      m = s_m[lane];
    }
    all = join8(all);
    m = order_value(__reduce_max_sync(0xffffffffu, order_of(m)));
  }

  if (kTop) {
    // the segments to read again: below the k-th largest maximum is nothing to
    // find; -inf is never a candidate
    take_largest(segs, [&](int i) { return (static_cast<unsigned long long>(s_seg[i]) << 32) | (0xffffffffu - i); },
                 s_best, s_top);
    const int chosen = min(k, segs);
    const float tau = segs >= k ? order_value(static_cast<unsigned>(s_top[k - 1] >> 32)) : -INFINITY;
    const int units = chosen * a.group;                // rows of 32 vectors
    auto vec_of = [&](int unit) {                      // the lane's vector, -1: none
      const int at = t0 * kAhead + key_token(s_top[unit / a.group]) * a.group + unit % a.group;
      const int i = at * 32 + lane;
      return at < t1 * kAhead && i < r.nvec ? i : -1;
    };
    auto offer = [&](float x, int v, unsigned long long above) {
      if (!(x >= tau) || x == -INFINITY) return;
      const unsigned long long key = rank_key(x, v);
      if (key <= above) return;
      const int at = atomicAdd(&s_count, 1);
      if (at < a.room) s_keys[at] = key;
    };
    auto offer_vec = [&](int i, const uint4& v, unsigned long long above) {
      if (i < 0 || !(Vec<T>::largest(v) >= tau)) return;
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const F2 p = Vec<T>::pair(v, j);
        offer(f2_lo(p), r.head + i * E + 2 * j, above);
        offer(f2_hi(p), r.head + i * E + 2 * j + 1, above);
      }
    };
    if (end_at >= 0) offer(end_x, end_at, 0ull);
    for (int u0 = w; u0 < units; u0 += 4 * W) {
      int i[4];
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        i[q] = u0 + q * W < units ? vec_of(u0 + q * W) : -1;
        if (i[q] >= 0) v[q] = __ldg(vecs + i[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) offer_vec(i[q], v[q], 0ull);
    }
    __syncthreads();
    const int found = s_count;
    if (found <= a.room) {
      take_largest(found, [&](int i) { return s_keys[i]; }, s_best, s_top);
    } else {
      // more candidates than room (many equal or sorted logits): as many units
      // at a time as fit beside the best so far, which raise the bar
      __shared__ unsigned long long s_so_far[32];
      const int step = (a.room - 32) / (32 * E);       // room is at least 32 + 32 E
      int have = 0;
      unsigned long long bar = 0ull;
      for (int u0 = 0; u0 < units; u0 += step) {
        __syncthreads();
        if (tid == 0) s_count = have;
        if (tid < have) s_keys[tid] = s_so_far[tid];
        __syncthreads();
        if (u0 == 0 && end_at >= 0) offer(end_x, end_at, 0ull);
        for (int u = u0 + w; u < min(units, u0 + step); u += W) {
          const int i = vec_of(u);
          if (i >= 0) offer_vec(i, __ldg(vecs + i), bar);
        }
        __syncthreads();
        const int n = s_count;
        take_largest(n, [&](int i) { return s_keys[i]; }, s_best, s_so_far);
        have = min(n, k);
        if (n >= k) bar = s_so_far[k - 1];
      }
      __syncthreads();
      if (tid < 32) s_top[tid] = tid < have ? s_so_far[tid] : 0ull;
      __syncthreads();
    }
  }

  if (parts > 1) {
    cluster_wait();
    if (w == 0) {
      if (lane == 0) {
        write_first(&s_peer[part][0],
                    (static_cast<unsigned long long>(__float_as_uint(m)) << 32) | __float_as_uint(all.c));
        write_first(&s_peer[part][1], __double_as_longlong(all.S));
        write_first(&s_peer[part][2], __double_as_longlong(all.T));
      }
      if (kTop) write_first(&s_peer_top[part][lane], lane < k ? s_top[lane] : 0ull);
    }
    cluster_arrive();
    cluster_wait();
    if (part != 0) return;
    if (w == 0) {
      m = -INFINITY;
      all = Sums{-INFINITY, 0.0, 0.0};
      if (lane < parts) {
        const unsigned long long mc = s_peer[lane][0];
        m = __uint_as_float(static_cast<unsigned>(mc >> 32));
        all = Sums{__uint_as_float(static_cast<unsigned>(mc)), __longlong_as_double(s_peer[lane][1]),
                   __longlong_as_double(s_peer[lane][2])};
      }
      all = join8(all);
      m = order_value(__reduce_max_sync(0xffffffffu, order_of(m)));
    }
    if (kTop)     // sorted lists: merged in pairs
      for (int n = parts / 2; n > 0; n /= 2) {
        for (int p = w; p < n; p += W) {
          const unsigned long long best = merge32(s_peer_top[p][lane], s_peer_top[p + n][lane], lane);
          (n == 1 ? s_top : s_peer_top[p])[lane] = best;
        }
        __syncthreads();
      }
  }
  const bool bad = !(all.S < 1e300);   // a NaN or +inf in the row
  if (tid == 0) {
    // ln sum e^(x - m), from the sum's own shift
    const double top = m == -INFINITY ? 0.0 : static_cast<double>(m);
    const double off = m == -INFINITY ? 0.0 : shift2(all.c) - top * kLog2e;
    const double lnSum = log(all.S), lnS = lnSum + off * kLn2;
    float lp = xt == -INFINITY ? xt : static_cast<float>(static_cast<double>(xt) - top - lnS);
    float H = all.S > 0.0 ? static_cast<float>(lnSum - kLn2 * (all.T / all.S)) : 0.f;
    if (bad) lp = H = NAN;
    a.logprob[item] = lp;
    if (a.entropy != nullptr) a.entropy[item] = H;
    if (a.stats != nullptr)
      reinterpret_cast<float2*>(a.stats)[item] =
          bad ? make_float2(NAN, NAN) : make_float2(m, static_cast<float>(all.S * exp2(off)));
    s_lse[0] = top;
    s_lse[1] = lnS;
    s_lse[2] = bad ? 1.0 : 0.0;
  }
  if (kTop && w == 0) {
    __syncwarp();
    const double top = s_lse[0], lnS = s_lse[1];
    const bool nan = s_lse[2] != 0.0;
    if (lane < k) {
      const unsigned long long key = s_top[lane];
      const long long o = static_cast<long long>(item) * k + lane;
      a.top_tokens[o] = key != 0ull ? key_token(key) : -1;
      a.top_logprobs[o] = nan ? NAN
                          : key == 0ull ? -INFINITY
                                        : static_cast<float>(order_value(static_cast<unsigned>(key >> 32)) - top - lnS);
    }
  }
}

// ------------------------------------------------------------- gradient

constexpr int kGradThreads = 256;
constexpr int kGradAhead = 4;

// dlogits_v = p_v (c0 + c1 y_v) + g [v = t]: with y = (x - m) log2 e,
// p = 2^y / s and ln p = y ln 2 - ln s, the bracket is
// -g - g_H (ln p + H). Elementwise once the row's sums are known, so the row
// is cut into pieces of kGradThreads * kGradAhead vectors, a CTA each, with
// all of a thread's loads in flight before the row's scalars are read. Bound
// by memory: 512 rows of 151,936 fp32 take 93 us, 6.7 TB/s read and written
// (102% of the copy rate), 3,000 of 50,257 bf16 100 us, 6.0 TB/s.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(GradArgs a) {
  constexpr int E = Vec<T>::kLen;
  const int row = blockIdx.x / a.pieces, piece = blockIdx.x - row * a.pieces, tid = threadIdx.x, V = a.V;
  const Row<T> r(static_cast<const T*>(a.logits) + row * a.stride, V);
  T* d = static_cast<T*>(a.dlogits) + row * a.gstride;
  const uint4* vecs = r.vecs();
  uint4* dvecs = reinterpret_cast<uint4*>(d + r.head);
  const int i0 = piece * kGradThreads * kGradAhead + tid;
  uint4 v[kGradAhead];
  if (kVec) {
#pragma unroll
    for (int u = 0; u < kGradAhead; ++u)
      if (i0 + u * kGradThreads < r.nvec) v[u] = __ldcs(vecs + i0 + u * kGradThreads);
  }
  const int tok = a.tokens[row];
  const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
  const float g = a.g_logprob[row];
  if (tid == 0 && piece == 0 && (tok < -1 || tok >= V))
    record_bad_item(a.err, row);
  const bool none = tok < 0 || tok >= V || st.x == -INFINITY;
  const float f = 1.f / st.y, lf = -logf(st.y);
  float c0 = -g, c1 = 0.f;
  if (a.g_entropy != nullptr) {
    const float gh = a.g_entropy[row];
    c0 -= gh * (lf + a.entropy[row]);
    c1 = -gh * static_cast<float>(kLn2);
  }
  const float m = st.x;
  auto one = [&](float x, int v) {
    const float y = fmax_nan((x - m) * kLog2e, kMinExp);
    float dv = ex2(y) * f * fmaf(c1, y, c0);
    if (v == tok && x != -INFINITY) dv += g;
    return none ? 0.f : dv;
  };
  if constexpr (!kVec) {     // rows and gradients aligned differently: element by element
    constexpr int kPer = kGradAhead * E;
    const int e0 = piece * kGradThreads * kPer + tid;
#pragma unroll 4
    for (int u = 0; u < kPer; ++u) {
      const int e = e0 + u * kGradThreads;
      if (e < V) store(d + e, one(to_float(r.x[e]), e));
    }
  } else {
#pragma unroll
    for (int u = 0; u < kGradAhead; ++u) {
      const int i = i0 + u * kGradThreads;
      if (i < r.nvec) {
        F2 q[E / 2];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const F2 x = Vec<T>::pair(v[u], j);
          const int e = r.head + i * E + 2 * j;
          q[j] = f2(one(f2_lo(x), e), one(f2_hi(x), e + 1));
        }
        __stcs(dvecs + i, Vec<T>::pack(q));
      }
    }
    if (piece == a.pieces - 1 && tid < r.head + r.tail) {
      const int e = tid < r.head ? tid : V - r.tail + tid - r.head;
      store(d + e, one(to_float(r.x[e]), e));
    }
  }
}


template <typename T>
cudaError_t launch_logprobs(ScoreArgs a, int items, cudaStream_t s) {
  constexpr int E = Vec<T>::kLen;
  const int tiles = std::max(1, (a.V / E + kTile - 1) / kTile);
  // rows to read, as far as can be told here: a round's emitted tokens fill
  // about half of its items or less. Where nearly all drafts are accepted there
  // are up to twice as many, and a row may get more CTAs than is best for them
  // (the 366 rows below)
  const long long rows = a.C > 1 ? (items + 1) / 2 : items;
  // few rows: a row is shared by the CTAs of a cluster, while that leaves each
  // eight tiles or more. Two CTAs up to four an SM; four and eight, whose
  // placing leaves SMs unevenly filled, up to two an SM (rows of 151,936 fp32:
  // 74 by 2 CTAs 17.6 us, by 4 13.0, by 8 15.9; 148 by 1 28.5, by 2 19.9, by
  // 4 25.1; 296 by 1 34.5, by 2 30.8; 366 by 1 38.9, by 2 45.5)
  int parts = 1;
  while (parts < kMaxParts && rows * 2 * parts <= (parts == 1 ? 4 * kSms : 2 * kSms) && tiles / (2 * parts) >= 8)
    parts *= 2;
  const int most = (tiles + parts - 1) / parts;
  a.items = items;
  a.parts = parts;
  a.gather = a.C > 1 && items > kSms / 2 && items <= kGather;
  // segments of one row of 32 vectors while shared memory holds so many, else
  // of whole tiles: fewer maxima to note (one a tile), more to read again
  a.group = most * kAhead <= kMaxSegs ? 1 : (most + kMaxSegs - 1) / kMaxSegs * kAhead;
  // many short rows: twice as many CTAs of four warps (4,000 rows of 32,000
  // bf16 with 5 alternatives 78.8 -> 69.3 us, 1,000 of 5,000 fp32 7.8 -> 5.8;
  // 366 of 151,936 fp32 39.5 -> 56)
  const int warps = std::min(most, rows > 4 * kSms && most <= 64 ? kMaxWarps / 2 : kMaxWarps);
  a.room = 32 + std::max(32 * E, std::min(kRoom, most * kTile * E));
  const bool top = a.top_k > 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items) * parts);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = top ? a.room * sizeof(unsigned long long) : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, top ? logprobs_kernel<T, true> : logprobs_kernel<T, false>, a);
}

template <typename T>
cudaError_t launch_grad(GradArgs a, int N, cudaStream_t s) {
  constexpr int E = Vec<T>::kLen;
  const int per = kGradThreads * kGradAhead * E;
  a.pieces = (a.V + per - 1) / per;
  if (static_cast<long long>(N) * a.pieces > 0x7fffffffll) return cudaErrorInvalidValue;
  // vectors if every row's gradient has the row's own alignment
  const bool vec = (a.stride - a.gstride) % E == 0;
  (vec ? logprobs_grad_kernel<T, true> : logprobs_grad_kernel<T, false>)<<<N * a.pieces, kGradThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_logprobs(const void* logits, dspark_dtype dtype, int64_t n_rows, int64_t row_stride,
                              const int64_t* row_start, const int32_t* tokens, int B, int C, int V, int top_k,
                              float* logprob, float* entropy, float* stats, int32_t* top_tokens,
                              float* top_logprobs, void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (!is_element_type(dtype)) return DSPARK_ERR_INVALID_ARG;
  if (B < 0 || C < 0 || static_cast<long long>(B) * C > kMaxItems || V < 1 || V > kMaxV) return DSPARK_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > kMaxStride || row_stride < V || row_stride > kMaxStride) return DSPARK_ERR_INVALID_ARG;
  if (n_rows > (1ll << 60) / row_stride) return DSPARK_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > DSPARK_MAX_TOP_K) return DSPARK_ERR_INVALID_ARG;
  if (B == 0 || C == 0) return DSPARK_OK;
  if (!is_given(logits) || !is_given(tokens) || !is_given(logprob) || !is_given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (!is_aligned16(row_start) || !is_aligned16(entropy) || !is_aligned16(stats)) return DSPARK_ERR_INVALID_ARG;
  if (top_k > 0 && (!is_given(top_tokens) || !is_given(top_logprobs))) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  ScoreArgs a{logits, n_rows, row_stride, row_start, tokens, C, V, top_k, logprob, entropy, stats, top_tokens,
              top_logprobs, reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset), 0, 1, 0, 1, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DSPARK_F32 ? launch_logprobs<float>(a, B * C, s) : launch_logprobs<uint16_t>(a, B * C, s);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status dspark_logprobs_grad(const void* logits, dspark_dtype dtype, int64_t row_stride,
                                   const int32_t* tokens, const float* stats, const float* entropy,
                                   const float* g_logprob, const float* g_entropy, int N, int V, void* dlogits,
                                   int64_t grad_stride, void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (!is_element_type(dtype)) return DSPARK_ERR_INVALID_ARG;
  if (N < 0 || N > kMaxItems || V < 1 || V > kMaxV) return DSPARK_ERR_INVALID_ARG;
  if (row_stride < V || row_stride > kMaxStride || grad_stride < V || grad_stride > kMaxStride)
    return DSPARK_ERR_INVALID_ARG;
  if (N == 0) return DSPARK_OK;
  if (!is_given(logits) || !is_given(tokens) || !is_given(stats) || !is_given(g_logprob) || !is_given(dlogits) || !is_given(workspace))
    return DSPARK_ERR_INVALID_ARG;
  if (g_entropy != nullptr && (!is_given(g_entropy) || !is_given(entropy))) return DSPARK_ERR_INVALID_ARG;
  if (dlogits == logits && row_stride != grad_stride) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  GradArgs a{logits, row_stride, grad_stride, tokens, stats, entropy, g_logprob, g_entropy, V, dlogits,
             reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset), 1};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DSPARK_F32 ? launch_grad<float>(a, N, s) : launch_grad<uint16_t>(a, N, s);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
