// Embedding lookup with scaling, and its gradient with respect to the table
// by sorted tokens. Both move rows and compute next to nothing: what bounds
// them is memory, and for few items the latency of the loads that wait for one
// another (token, row; sorted order, row, parts).
#include <algorithm>

#include "elements.cuh"

namespace dspark {
namespace {

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- lookup

struct EmbedArgs {
  const void* table;
  const int32_t* tokens;
  int n, V, r;
  float scale;
  void* out;
  unsigned* err;
};

constexpr int kThreads = 256;

// Neighbouring columns of a thread: eight if both sides are bf16 (16 bytes),
// else four, so that a warp's store instruction covers whole 32-byte sectors
// (eight fp32 columns a thread are two half-sector stores: 78 -> 53 us for
// 16,384 rows of 4,096, bf16 to fp32).
template <typename TI, typename TO>
constexpr int kCols = sizeof(TI) + sizeof(TO) == 4 ? 8 : 4;

template <int N>
__device__ __forceinline__ void load_cols(const float* p, float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p + j));
    v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
  }
}
template <int N>
__device__ __forceinline__ void load_cols(const uint16_t* p, float (&v)[N]) {
  unsigned w[N / 2];
  if constexpr (N == 8) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  }
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
// kStream: marked as not needed again soon.
template <bool kStream, typename V>
__device__ __forceinline__ void put(V* p, const V& v) {
  if constexpr (kStream)
    __stcs(p, v);
  else
    *p = v;
}
template <int N, bool kStream = false>
__device__ __forceinline__ void save_cols(float* p, const float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4)
    put<kStream>(reinterpret_cast<float4*>(p + j), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
}
template <int N, bool kStream = false>
__device__ __forceinline__ void save_cols(uint16_t* p, const float (&v)[N]) {
  if constexpr (N == 8)
    put<kStream>(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                         pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
  else
    put<kStream>(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
}

// blockDim.x threads a row (kCols columns each, or single ones where r is no
// multiple of kCols), blockDim.y * kRows rows a CTA, kRows of them in flight a
// thread. 16,384 rows of 4,096, bf16 to fp32: 55 us, 6.0 TB/s with each table
// row read once (92% of the copy rate); 64 rows of 256: 1.4 us. Single columns
// are loads and stores of 2 or 4 bytes, bound by their number: 16,384 distinct
// rows, bf16 to fp32, of 4,096 columns 67 us and of 4,095 110, of 1,000 20 and
// of 1,001 32 (bf16 to bf16 14 and 30, fp32 to fp32 24 and 35).
template <typename TI, typename TO, bool kVec, int kRows>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a) {
  constexpr int N = kVec ? kCols<TI, TO> : 1;
  const int i0 = blockIdx.x * blockDim.y * kRows + threadIdx.y;
  int t[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int i = i0 + u * blockDim.y;
    t[u] = i < a.n ? __ldg(a.tokens + i) : -1;
    if (t[u] < -1 || t[u] >= a.V) {
      if (threadIdx.x == 0) record_bad_item(a.err, i);
      t[u] = -1;
    }
  }
  const TI* table = static_cast<const TI*>(a.table);
  TO* out = static_cast<TO*>(a.out);
  for (int c = threadIdx.x * N; c < a.r; c += blockDim.x * N) {
    float v[kRows][N];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (t[u] >= 0) {
        const TI* p = table + static_cast<long long>(t[u]) * a.r + c;
        if constexpr (kVec)
          load_cols<N>(p, v[u]);
        else
          v[u][0] = to_float(__ldg(p));
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[u][j] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u * blockDim.y;
      if (i >= a.n) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) v[u][j] = t[u] >= 0 ? v[u][j] * a.scale : 0.f;
      TO* q = out + static_cast<long long>(i) * a.r + c;
      if constexpr (kVec)
        save_cols<N, true>(q, v[u]);
      else
        store(q, v[u][0]);
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t s) {
  const bool vec = a.r % kCols<TI, TO> == 0;
  const int units = vec ? a.r / kCols<TI, TO> : a.r;
  int x = 8;
  while (x < units && x < kThreads) x *= 2;
  const dim3 block(x, kThreads / x);
  // two rows a thread once that fills the GPU (60,000 rows of 256, bf16 to
  // fp32: one 20.9 us, two 16.3, four 18.2, eight 18.8)
  const int rows = static_cast<long long>(a.n) >= 8ll * kSms * block.y ? 2 : 1;
  const int grid = ceil_div(a.n, static_cast<int>(block.y) * rows);
  auto kernel = vec ? (rows == 2 ? embed_kernel<TI, TO, true, 2> : embed_kernel<TI, TO, true, 1>)
                    : (rows == 2 ? embed_kernel<TI, TO, false, 2> : embed_kernel<TI, TO, false, 1>);
  kernel<<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

// -------------------------------------------------------------- gradient
//
// dtable[v] = scale * sum of dout's rows whose token is v. Three kernels, each started
// while the one before it runs out:
//
// sort_kernel: CTA g owns table rows [g R, (g+1) R). It reads all n tokens,
//   counts those below its rows (its offset in the sorted order, so the CTAs
//   need not talk to each other) and counting-sorts its own, stably: each
//   warp takes a contiguous piece of the tokens, keeps its matches in order,
//   counts them per row, and places them after the earlier warps'. It then
//   zeroes its rows that no token points at.
// sum_kernel: the sorted items in windows of equal length, one a warp. A short
//   run of equal tokens is summed by the warp in whose window it starts. A
//   longer one is summed by all whose windows it touches, so that a frequent
//   token does not hold up one warp or CTA: a CTA joins its warps' parts in
//   shared memory, and those of a run that goes on go to scratch.
// join_kernel: adds the CTAs' parts of each such run in order.
//
// Few items: direct_kernel, one CTA an item and up to 8 slabs, no sorting; without accumulate it
// runs beside zero_kernel and waits for it before it writes.
//
// Measured: 512 rows of 256 fp32 added to a gradient 3.7 us (direct), written
// whole into 151,936 rows 26.6 (zeroing alone 24); 10,007 of 200 bf16 into
// 50,257 fp32 rows 16.9 (sort beside zeroing 10, sums 8.5, joins 4, starts
// overlapped); 65,536 of 1,024 bf16 into 129,280 86 (45, 33, 6). An owner that
// summed its own rows as well took twice as long: one CTA an SM has too few
// loads in flight. Joining through counters in the sums' kernel cost as much
// as the third kernel, since a release waits for the SM's stores. Zeroing what
// is left beside the sums, and two slabs a warp, gained nothing for the last of
// these, where memory is busy anyway and the sums issue 73% of the slots they
// have at four CTAs an SM; smaller ones were not tried.

struct GradArgs {
  const void* dout;
  const int32_t* tokens;
  int n, V, r;
  float scale;
  int accumulate;
  void* dtable;
  unsigned* err;
  int R, slabs, pieces;   // table rows of an owner; slabs of a row; pieces (a CTA's windows) of the sorted items
  int direct;             // slabs of a CTA of the direct path
  int keep;               // matches that a warp of the sort keeps in shared memory; more are found again
  int* n_sorted;          // items with a token
  int4* sorted;           // [n] item, token, and the run [begin, end) it is in
  float* parts;           // [pieces][2][slabs][32 lanes]: of the long run that comes in, of the one that leaves
};

constexpr int kSortWarps = 16, kSortThreads = kSortWarps * 32;
constexpr int kMaxR = 2048;     // rows of an owner (11 bits beside 20 of an item's place in a warp's piece)
constexpr int kWindow = 16;     // sorted items of a warp
constexpr int kShort = 16;      // a run up to this length belongs to one warp (kWindow + kShort <= 32)
constexpr int kAhead = 6;       // rows of a warp in flight
constexpr int kSumWarps = 8, kSumThreads = kSumWarps * 32, kPiece = kSumWarps * kWindow;
constexpr int kDirectItems = 4096, kDirectAlways = 512, kDirectWork = 6144;   // items; items; items times slabs
constexpr int kDirectWarps = 8, kDirectThreads = kDirectWarps * 32;

template <typename TO>
__device__ __forceinline__ void zero_row(TO* d, int r, int lane) {
  const int bytes = r * static_cast<int>(sizeof(TO));
  if (bytes % 16 == 0) {
    for (int k = lane; k < bytes / 16; k += 32) reinterpret_cast<uint4*>(d)[k] = make_uint4(0, 0, 0, 0);
  } else {
    for (int k = lane; k < r; k += 32) store(d + k, 0.f);
  }
}

// 16 warps sort. With accumulate off 16 more zero the rows meanwhile, blindly
// until the counts are known (what they zero of rows with tokens sum_kernel
// writes over), then only those without a token; the sorting warps join them.
template <typename TO>
__global__ void __launch_bounds__(2 * kSortThreads, 1) sort_kernel(GradArgs a) {
  extern __shared__ unsigned smem[];
  constexpr int W = kSortWarps, nt = kSortThreads;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, R = a.R, n = a.n;
  unsigned* hist = smem;                                   // [W][R] counts, then places
  unsigned* total = hist + W * R;                          // [R] tokens of a row
  unsigned* begin = total + R;                             // [R] and where they start in the sorted order
  unsigned* mine = begin + R + w * a.keep;                 // [W][keep]
  __shared__ unsigned s_below, s_red[W];
  __shared__ int s_rows;
  __shared__ volatile int s_counted;
  const int v0 = blockIdx.x * R, rows = min(R, a.V - v0);
  auto fill = [&]() {          // by whole warps, four rows at a time
    TO* d = static_cast<TO*>(a.dtable) + static_cast<long long>(v0) * a.r;
    while (true) {
      int k = 0;
      if (lane == 0) k = atomicAdd(&s_rows, 4);
      k = __shfl_sync(0xffffffffu, k, 0);
      if (k >= rows) return;
      const bool counted = s_counted != 0;
      __threadfence_block();
      for (int j = k; j < min(rows, k + 4); ++j)
        if (!counted || total[j] == 0u) zero_row(d + static_cast<long long>(j) * a.r, a.r, lane);
    }
  };
  if (tid == 0) {
    s_rows = 0;
    s_counted = 0;
    s_below = 0;
  }
  __syncthreads();
  if (w >= W) {
    fill();
    return;
  }
  using Sorters = NamedSync<1, kSortThreads>;
  const unsigned lt = (1u << lane) - 1u;
  for (int k = tid; k < (W + 1) * R; k += nt) hist[k] = 0;      // and total
  Sorters::sync();

  // each warp's matches, in order: four neighbouring tokens a lane
  const int len = ceil_div(ceil_div(n, W), 128) * 128;
  const int lo = min(n, w * len), hi = min(n, lo + len);
  unsigned* count = hist + w * R;
  int found = 0;
  unsigned below = 0;
  for (int i0 = lo; i0 < hi; i0 += 128 * kAhead) {
    int4 q[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * 128 + lane * 4;
      if (i + 4 <= hi) {
        q[u] = __ldg(reinterpret_cast<const int4*>(a.tokens + i));
      } else {
        q[u].x = i < hi ? __ldg(a.tokens + i) : -1;
        q[u].y = i + 1 < hi ? __ldg(a.tokens + i + 1) : -1;
        q[u].z = i + 2 < hi ? __ldg(a.tokens + i + 2) : -1;
        q[u].w = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * 128 + lane * 4;
      const int t[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      bool hit[4];
      bool any = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {           // -1 and bad ids are in no range
        below += static_cast<unsigned>(t[c]) < static_cast<unsigned>(v0);
        hit[c] = static_cast<unsigned>(t[c] - v0) < static_cast<unsigned>(rows);
        any |= hit[c];
      }
      if (blockIdx.x == 0)
        for (int c = 0; c < 4; ++c)
          if (t[c] < -1 || t[c] >= a.V) record_bad_item(a.err, i + c);
      if (__ballot_sync(0xffffffffu, any) == 0u) continue;
      int at = found;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const unsigned mask = __ballot_sync(0xffffffffu, hit[c]);
        at += __popc(mask & lt);
        found += __popc(mask);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!hit[c]) continue;
        const unsigned off = static_cast<unsigned>(t[c] - v0);
        atomicAdd(count + off, 1u);
        atomicAdd(total + off, 1u);
        if (at < a.keep) mine[at] = (static_cast<unsigned>(i + c - lo) << 11) | off;
        ++at;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0 && below != 0u) atomicAdd(&s_below, below);
  Sorters::sync();
  if (tid == 0) {                    // behind the barrier: every total is there
    __threadfence_block();
    s_counted = 1;
  }

  // places: rows in order, within a row the warps in order
  const int per = ceil_div(rows, nt), r0 = min(rows, tid * per), r1 = min(rows, r0 + per);
  unsigned sum = 0;
  for (int k = r0; k < r1; ++k) sum += total[k];
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_red[w] = inc;
  Sorters::sync();
  unsigned place = s_below + inc - sum;
  for (int j = 0; j < w; ++j) place += s_red[j];
  for (int k = r0; k < r1; ++k) {
    begin[k] = place;
    if (total[k] == 0u) continue;          // most rows
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const unsigned x = hist[j * R + k];
      hist[j * R + k] = place;
      place += x;
    }
  }
  if (blockIdx.x == gridDim.x - 1 && tid == nt - 1) *a.n_sorted = static_cast<int>(place);
  Sorters::sync();

  auto put = [&](bool hit, unsigned off, int item) {   // by the whole warp
    const unsigned peers = __match_any_sync(0xffffffffu, hit ? off : 0xffffffffu);
    if (hit) {
      const int first = static_cast<int>(begin[off]);
      a.sorted[count[off] + __popc(peers & lt)] =
          make_int4(item, v0 + static_cast<int>(off), first, first + static_cast<int>(total[off]));
    }
    __syncwarp();
    if (hit && (peers & lt) == 0u) count[off] += __popc(peers);
    __syncwarp();
  };
  if (found <= a.keep) {
    for (int k0 = 0; k0 < found; k0 += 32) {
      const bool hit = k0 + lane < found;
      const unsigned e = hit ? mine[k0 + lane] : 0u;
      put(hit, e & 2047u, lo + static_cast<int>(e >> 11));
    }
  } else {
    for (int i0 = lo; i0 < hi; i0 += 32 * kAhead) {
      int t[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * 32 + lane;
        t[u] = i < hi ? __ldg(a.tokens + i) : -1;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool hit = t[u] >= v0 && t[u] < v0 + rows;
        if (__any_sync(0xffffffffu, hit)) put(hit, static_cast<unsigned>(t[u] - v0), i0 + u * 32 + lane);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!a.accumulate) fill();
}

// A lane's columns of a row of TI, 16 bytes: neighbours (kVec: the rows are
// aligned to that), or 32 apart. A slab is a warp's columns.
template <typename TI>
constexpr int kLane = 16 / static_cast<int>(sizeof(TI));
template <typename TI>
constexpr int kSlab = 32 * kLane<TI>;

template <typename TI, bool kVec>
__device__ __forceinline__ uint4 load_lane(const TI* p, int lane, int cols) {
  constexpr int E = kLane<TI>;
  uint4 v = make_uint4(0, 0, 0, 0);
  if constexpr (kVec) {
    if (lane * E < cols) v = __ldcs(reinterpret_cast<const uint4*>(p) + lane);
  } else {
    unsigned x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      x[j] = 0u;
      if (lane + 32 * j < cols) {
        if constexpr (E == 4)
          x[j] = __float_as_uint(p[lane + 32 * j]);
        else
          x[j] = p[lane + 32 * j];
      }
    }
    if constexpr (E == 4)
      v = make_uint4(x[0], x[1], x[2], x[3]);
    else
      v = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
  }
  return v;
}

template <int E>
__device__ __forceinline__ void add_lane(float (&s)[E], const uint4& v) {
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (E == 4) {
      s[j] += __uint_as_float(w[j]);
    } else {
      s[2 * j] += __uint_as_float(w[j] << 16);
      s[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// A warp's columns of a row to shared memory, without waiting: where the rows
// are aligned each lane copies its own columns and later reads those; else the
// row's 16-byte blocks are copied, from the one that holds the first column
// on, and a lane reads columns 32 apart, the first `skew` bytes into the place.
template <typename T, bool kVec, int E>
struct Place {
  static constexpr int kBytes = 32 * E * static_cast<int>(sizeof(T));
  static constexpr int kSize = kVec ? kBytes : kBytes + 16;
  __device__ __forceinline__ static void fetch(char* to, const T* p, int lane, int cols) {
    unsigned at = static_cast<unsigned>(__cvta_generic_to_shared(to));
    if constexpr (kVec) {
      constexpr int kMine = E * static_cast<int>(sizeof(T)), kStep = kMine < 16 ? kMine : 16;
      if (lane * E < cols) {
#pragma unroll
        for (int j = 0; j < kMine; j += kStep)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at + lane * kMine + j),
                       "l"(reinterpret_cast<const char*>(p) + lane * kMine + j), "n"(kStep)
                       : "memory");
      }
    } else {
      const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
      const int bytes = skew + min(cols, 32 * E) * static_cast<int>(sizeof(T));
      const char* from = reinterpret_cast<const char*>(p) - skew;
      for (int j = lane * 16; j < bytes; j += 512)      // the last block up to the row's end only
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(at + j), "l"(from + j),
                     "r"(min(16, bytes - j))
                     : "memory");
    }
  }
  // Adds the lane's columns, once its copies (kVec) or the warp's are there.
  __device__ __forceinline__ static void add(float (&s)[E], const char* place, const T* p, int lane) {
    if constexpr (kVec) {
      const T* v = reinterpret_cast<const T*>(place) + lane * E;
      if constexpr (sizeof(T) * E == 16) {
        add_lane(s, *reinterpret_cast<const uint4*>(v));
      } else if constexpr (sizeof(T) == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(v);
        s[0] += __uint_as_float(x.x << 16), s[1] += __uint_as_float(x.x & 0xffff0000u);
        s[2] += __uint_as_float(x.y << 16), s[3] += __uint_as_float(x.y & 0xffff0000u);
      } else {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const float4 x = reinterpret_cast<const float4*>(v)[j / 4];
          s[j] += x.x, s[j + 1] += x.y, s[j + 2] += x.z, s[j + 3] += x.w;
        }
      }
    } else {
      const T* v = reinterpret_cast<const T*>(place + (reinterpret_cast<uintptr_t>(p) & 15u)) + lane;
#pragma unroll
      for (int j = 0; j < E; ++j) s[j] += to_float(v[32 * j]);     // columns behind the row: not saved
    }
  }
};

template <int E>
__device__ __forceinline__ void clear(float (&s)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) s[j] = 0.f;
}

template <typename TO, bool kVec, int E>
__device__ __forceinline__ void save_lane(TO* d, int lane, int cols, const float (&v)[E]) {
  if constexpr (kVec) {
    if (lane * E < cols) save_cols<E>(d + lane * E, v);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (lane + 32 * j < cols) store(d + lane + 32 * j, v[j]);
  }
}

// dtable[token, a lane's columns from col on] (+)= scale * s
template <typename TO, bool kVec, int E>
__device__ __forceinline__ void finish(const GradArgs& a, int token, int col, int lane, const float (&s)[E]) {
  TO* d = static_cast<TO*>(a.dtable) + static_cast<long long>(token) * a.r + col;
  const int cols = a.r - col;
  float v[E];
#pragma unroll
  for (int j = 0; j < E; ++j) v[j] = s[j] * a.scale;
  if (a.accumulate) {
    if constexpr (kVec) {
      if (lane * E < cols) Place<TO, true, E>::add(v, reinterpret_cast<const char*>(d), d, lane);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (lane + 32 * j < cols) v[j] += to_float(d[lane + 32 * j]);
    }
  }
  save_lane<TO, kVec, E>(d, lane, cols, v);
}

template <typename TI, typename TO, bool kVec, bool kAdd>
struct SumShared {
  static constexpr int E = kLane<TI>;
  alignas(16) char rows[kSumWarps][kAhead][Place<TI, kVec, E>::kSize];
  alignas(16) char old[kAdd ? kSumWarps : 1][kAdd ? kAhead : 1][Place<TO, kVec, E>::kSize];
  float part[kSumWarps][2][E][32];
  int4 run[kSumWarps][2];   // token, begin, end of each long run's part; token -1: none
  int4 list[kSumWarps][32];
};

// A lane's place in the scratch for piece g's part of a long run: the run that
// comes in (k = 0), or starts there and leaves (1).
template <int E>
__device__ __forceinline__ float4* part_of(const GradArgs& a, int g, int k, int slab, int lane) {
  return reinterpret_cast<float4*>(a.parts) + (((2ll * g + k) * a.slabs + slab) * 32 + lane) * (E / 4);
}

// A window a warp, on one slab; the long runs' parts are joined in the CTA.
template <typename TI, typename TO, bool kVec, bool kAdd>
__global__ void __launch_bounds__(kSumThreads, kAdd ? 2 : 5) sum_kernel(GradArgs a) {
  constexpr int E = kLane<TI>;
  extern __shared__ __align__(16) unsigned char sum_smem[];
  SumShared<TI, TO, kVec, kAdd>& sh = *reinterpret_cast<SumShared<TI, TO, kVec, kAdd>*>(sum_smem);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = blockIdx.x / a.slabs, slab = blockIdx.x - piece * a.slabs;
  const int p0 = piece * kPiece, lo = p0 + w * kWindow, pos = lo + lane;
  const int col = slab * kSlab<TI>, cols = a.r - col;
  if (lane < 2) sh.run[w][lane].x = -1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // what lies behind the last sorted item is read but not used
  int4 it = make_int4(0, 0, 0, 0);
  if (pos < a.n) it = __ldcg(a.sorted + pos);
  const int N = __ldcg(a.n_sorted), hi = min(N, lo + kWindow);
  if (p0 >= N) return;
  // the warp's items, moved together: lane j then holds the j-th
  unsigned ends, shorts;
  int items;
  {
    const bool is_short = it.w - it.z <= kShort;
    const bool mine = pos < N && (is_short ? it.z >= lo && it.z < hi : pos < hi);
    const bool is_end = pos == it.w - 1 || (!is_short && pos == hi - 1);
    const unsigned mask = __ballot_sync(0xffffffffu, mine);
    items = __popc(mask);
    if (mine)
      sh.list[w][__popc(mask & ((1u << lane) - 1u))] =
          make_int4(it.x | (is_end ? 1 << 30 : 0) | (is_short ? 1 << 29 : 0), it.y, it.z, it.w);
    __syncwarp();
    it = sh.list[w][lane];      // behind the last item: not used
    ends = __ballot_sync(0xffffffffu, lane < items && (it.x >> 30 & 1) != 0);
    shorts = __ballot_sync(0xffffffffu, (it.x >> 29 & 1) != 0);
    it.x &= (1 << 29) - 1;
  }
  const TI* dout = static_cast<const TI*>(a.dout) + col;
  TO* dtable = static_cast<TO*>(a.dtable) + col;
  float sum[E];
  clear(sum);
  // rows go through a ring of kAhead places; each lane reads what it copied
  auto fetch = [&](int j, int u) {
    if (j < items) {
      const int item = __shfl_sync(0xffffffffu, it.x, j);
      Place<TI, kVec, E>::fetch(sh.rows[w][u], dout + static_cast<long long>(item) * a.r, lane, cols);
      if (kAdd && ((ends & shorts) >> j & 1u) != 0u) {     // what the run's sum is added to
        const int token = __shfl_sync(0xffffffffu, it.y, j);
        Place<TO, kVec, E>::fetch(sh.old[kAdd ? w : 0][kAdd ? u : 0], dtable + static_cast<long long>(token) * a.r,
                                  lane, cols);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(u, u);
  auto take = [&](int j, int u) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    if (!kVec) __syncwarp();      // the other lanes' copies
    Place<TI, kVec, E>::add(sum, sh.rows[w][u],
                            kVec ? dout : dout + static_cast<long long>(__shfl_sync(0xffffffffu, it.x, j)) * a.r, lane);
    if ((ends >> j & 1u) != 0u) {
      const int token = __shfl_sync(0xffffffffu, it.y, j);
      if ((shorts >> j & 1u) != 0u) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] *= a.scale;
        TO* d = dtable + static_cast<long long>(token) * a.r;
        if constexpr (kAdd) Place<TO, kVec, E>::add(sum, sh.old[w][u], d, lane);
        save_lane<TO, kVec, E>(d, lane, cols, sum);
      } else {
        // a long run's part: it came in, or starts here (and leaves: it is longer than a window)
        const int begin = __shfl_sync(0xffffffffu, it.z, j), end = __shfl_sync(0xffffffffu, it.w, j);
        const int k = begin < lo ? 0 : 1;
        if (lane == 0) sh.run[w][k] = make_int4(token, begin, end, 0);
#pragma unroll
        for (int e = 0; e < E; ++e) sh.part[w][k][e][lane] = sum[e];
      }
      clear(sum);
    }
    if (!kVec) __syncwarp();      // the place is read
    fetch(j + kAhead, u);
  };
  // unrolled over the ring, so that its places are constants (88 -> 86 us for
  // the 65,536 rows above)
#pragma unroll 1
  for (int j0 = 0; j0 < items; j0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u < items) take(j0 + u, u);
  }
  if (!__syncthreads_or((ends & ~shorts) != 0u)) return;
  // The first part of a run here is one that starts in a window, or comes into
  // the piece: the warp of that window adds the parts behind it.
  for (int k = w == 0 ? 0 : 1; k < 2; ++k) {
    const int4 run = sh.run[w][k];
    if (run.x < 0) continue;
    const int stop = min((run.z - 1 - p0) / kWindow, kSumWarps - 1);   // the last window it touches
    clear(sum);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = sh.part[w][k][e][lane];
    for (int i = w + 1; i <= stop; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += sh.part[i][0][e][lane];
    if (run.y >= p0 && run.z <= p0 + kPiece) {
      finish<TO, kVec>(a, run.x, col, lane, sum);
    } else {
      float4* part = part_of<E>(a, piece, run.y < p0 ? 0 : 1, slab, lane);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) part[e] = make_float4(sum[4 * e], sum[4 * e + 1], sum[4 * e + 2], sum[4 * e + 3]);
    }
  }
}

// Adds parts [lo, hi) of the run whose parts start at piece `first`.
template <int E>
__device__ __forceinline__ void add_parts(const GradArgs& a, int first, int lo, int hi, int slab, int lane,
                                          float (&sum)[E]) {
  constexpr int kParts = 64 / E;
  for (int g = lo; g < hi; g += kParts) {
    float4 x[kParts][E / 4];
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int j = 0; j < E / 4; ++j)
        x[u][j] = g + u < hi ? __ldcg(part_of<E>(a, first + g + u, g + u == 0 ? 1 : 0, slab, lane) + j)
                             : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        sum[4 * j] += x[u][j].x;
        sum[4 * j + 1] += x[u][j].y;
        sum[4 * j + 2] += x[u][j].z;
        sum[4 * j + 3] += x[u][j].w;
      }
  }
}

// The runs that leave a piece, a warp a piece and slab: the run that holds the
// piece's last item, if it starts in the piece and goes on. One of up to
// kAlone parts is the warp's, more are shared by all warps of the CTA.
constexpr int kJoinWarps = 8;
template <typename TI, typename TO, bool kVec>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(GradArgs a) {
  constexpr int E = kLane<TI>, kAlone = 64 / E;
  __shared__ float s_part[kJoinWarps][E][32];
  __shared__ int2 s_run[kJoinWarps];     // token, parts (more than kAlone, or 0)
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x / a.slabs, slab = blockIdx.x - block * a.slabs, col = slab * kSlab<TI>;
  const int piece = block * kJoinWarps + w, last = (piece + 1) * kPiece - 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int4 it = make_int4(0, 0, 0, 0);
  if (last < a.n) it = __ldcg(a.sorted + last);
  const int N = __ldcg(a.n_sorted);
  const bool leaves = last < N && it.w - it.z > kShort && it.z >= piece * kPiece && it.w > last + 1;
  const int parts = leaves ? (it.w - 1) / kPiece - piece + 1 : 0;
  float sum[E];
  if (parts > 0 && parts <= kAlone) {
    clear(sum);
    add_parts<E>(a, piece, 0, parts, slab, lane, sum);
    finish<TO, kVec>(a, it.y, col, lane, sum);
  }
  if (lane == 0) s_run[w] = make_int2(it.y, parts > kAlone ? parts : 0);
  if (!__syncthreads_or(parts > kAlone)) return;
  for (int j = 0; j < kJoinWarps; ++j) {
    const int2 run = s_run[j];
    if (run.y == 0) continue;
    const int per = ceil_div(run.y, kJoinWarps), p0 = min(run.y, w * per), p1 = min(run.y, p0 + per);
    clear(sum);
    add_parts<E>(a, block * kJoinWarps + j, p0, p1, slab, lane, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) s_part[w][e][lane] = sum[e];
    __syncthreads();
    if (w == 0) {
      for (int g = 1; g < kJoinWarps; ++g)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] += s_part[g][e][lane];
      finish<TO, kVec>(a, run.x, col, lane, sum);
    }
    __syncthreads();
  }
}

// One CTA an item and up to kDirectWarps slabs; the CTA of a token's first
// item sums all of that token's items. Its warps share the slabs and, where
// there are fewer slabs than warps, the items in equal parts.
constexpr int kZeroThreads = 512;
__global__ void __launch_bounds__(kZeroThreads) zero_kernel(uint4* d, long long vecs, uint16_t* rest, int halves) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long step = static_cast<long long>(gridDim.x) * kZeroThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kZeroThreads + threadIdx.x; i < vecs; i += step)
    d[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && threadIdx.x < halves) rest[threadIdx.x] = 0;
}

// kItems: n at most. 512 rows of 256 fp32: 3.7 us, three dependent loads
// (tokens, rows, and the gradient's rows) and the launch.
template <typename TI, typename TO, bool kVec, int kItems>
__global__ void __launch_bounds__(kDirectThreads) direct_kernel(GradArgs a) {
  constexpr int kLoads = kItems / kDirectThreads, kWords = kItems / 32 / 32, E = kLane<TI>;
  __shared__ unsigned s_hits[kItems / 32];
  __shared__ short s_items[kItems];
  __shared__ float s_sum[kDirectWarps][E][32];
  const int i = blockIdx.x, tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  // zero_kernel is done; every CTA waits, so that the grid ends after it
  auto zeroed = [&]() {
    if (!a.accumulate) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  int mine[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int j = u * kDirectThreads + tid;
    mine[u] = j < a.n ? __ldg(a.tokens + j) : -1;
  }
  const int t = __ldg(a.tokens + i);
  if (t < 0 || t >= a.V) {
    if (t != -1 && tid == 0 && blockIdx.y == 0) record_bad_item(a.err, i);
    zeroed();
    return;
  }
  bool before = false;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    before |= mine[u] == t && u * kDirectThreads + tid < i;
    const unsigned mask = __ballot_sync(0xffffffffu, mine[u] == t);
    if (lane == 0) s_hits[u * kDirectWarps + w] = mask;
  }
  if (__syncthreads_or(before)) {
    zeroed();
    return;
  }
  // the token's items in order: kWords neighbouring words of hits a lane
  unsigned word[kWords];
  int mine_count = 0;
#pragma unroll
  for (int u = 0; u < kWords; ++u) {
    word[u] = s_hits[lane * kWords + u];
    mine_count += __popc(word[u]);
  }
  int at = mine_count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += x;
  }
  const int total = __shfl_sync(0xffffffffu, at, 31);
  at -= mine_count;
  if (w == 0)
#pragma unroll
    for (int u = 0; u < kWords; ++u)
      for (unsigned m = word[u]; m != 0u; m &= m - 1)
        s_items[at++] = static_cast<short>((lane * kWords + u) * 32 + __ffs(m) - 1);
  __syncthreads();
  const int slab0 = static_cast<int>(blockIdx.y) * a.direct, here = min(a.direct, a.slabs - slab0);
  const int groups = kDirectWarps / here;
  const int group = w / here, col = (slab0 + w % here) * kSlab<TI>;
  float sum[E];
  clear(sum);
  if (group < groups) {
    const int per = ceil_div(total, groups), lo = min(total, group * per), hi = min(total, lo + per);
    const TI* dout = static_cast<const TI*>(a.dout) + col;
    for (int j = lo; j < hi; j += kAhead) {
      uint4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        x[u] = j + u < hi ? load_lane<TI, kVec>(dout + static_cast<long long>(s_items[j + u]) * a.r, lane, a.r - col)
                          : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add_lane(sum, x[u]);
    }
    if (group > 0)
#pragma unroll
      for (int j = 0; j < E; ++j) s_sum[w][j][lane] = sum[j];
  }
  __syncthreads();
  zeroed();
  if (w >= here) return;
  for (int g = 1; g < groups; ++g)
#pragma unroll
    for (int j = 0; j < E; ++j) sum[j] += s_sum[g * here + w][j][lane];
  finish<TO, kVec>(a, t, col, lane, sum);
}

// Sizes of the sorted path for (n, V, r) and rows of dout of `lane_cols`
// columns a lane, and its scratch.
struct GradPlan {
  int R, owners, keep, slabs, pieces;
  size_t smem, off_n, off_sorted, off_parts, bytes;
};
constexpr int kSortSmem = 224 << 10;    // what an owner's words of any plan fit in
GradPlan grad_plan(int n, int V, int r, int lane_cols) {
  constexpr int kSmemWords = kSortSmem / 4;
  GradPlan p{};
  p.R = std::min(kMaxR, ceil_div(V, kSms));     // one owner an SM, more for very large V
  p.owners = ceil_div(V, p.R);
  p.keep = std::min((kSmemWords - 256 - (kSortWarps + 2) * p.R) / kSortWarps, std::max(32, ceil_div(n, kSortWarps)));
  p.slabs = ceil_div(r, 32 * lane_cols);
  p.pieces = std::max(1, ceil_div(n, kPiece));
  p.smem = (static_cast<size_t>(kSortWarps + 2) * p.R + static_cast<size_t>(kSortWarps) * p.keep) * sizeof(unsigned);
  p.off_n = kScratchOffset;
  p.off_sorted = p.off_n + 256;
  p.off_parts = align_up(p.off_sorted + static_cast<size_t>(n) * sizeof(int4), 256);
  p.bytes = align_up(p.off_parts + static_cast<size_t>(p.pieces) * 2 * p.slabs * 32 * lane_cols * sizeof(float), 256);
  return p;
}

bool embed_sizes_ok(int n, int V, int r) {
  return n >= 0 && n <= kMaxItems && V >= 1 && V <= kMaxV && r >= 1 && r <= DSPARK_MAX_EMBED_R;
}

template <typename TI, typename TO, bool kVec>
cudaError_t launch_grad(GradArgs a, char* ws, cudaStream_t s) {
  const GradPlan p = grad_plan(a.n, a.V, a.r, kLane<TI>);
  a.slabs = p.slabs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.accumulate ? 0 : 1;
  // Each CTA of the direct path reads all tokens, and its 8 warps share a
  // frequent token's items only as far as the slabs leave warps for it
  // (accumulating rows of fp32, direct against sorted: 1,500 x 256 7.1 us
  // against 11.9, 3,000 x 256 11.7 against 12.4, 750 x 1,024 8.3 against 11.5,
  // 4,000 x 64 13.5 against 13.2, 4,000 x 256 14.2 against 12.9, 2,379 x 1,024
  // 23.4 against 12.6).
  if (a.n <= kDirectAlways ||
      (a.n <= kDirectItems && static_cast<long long>(a.n) * a.slabs <= kDirectWork)) {
    if (!a.accumulate) {
      const long long bytes = static_cast<long long>(a.V) * a.r * static_cast<long long>(sizeof(TO));
      char* d = static_cast<char*>(a.dtable);
      const long long vecs = bytes / 16;
      const long long blocks = (vecs + kZeroThreads - 1) / kZeroThreads;
      const int grid = static_cast<int>(std::max(1ll, std::min<long long>(2 * kSms, blocks)));
      zero_kernel<<<grid, kZeroThreads, 0, s>>>(reinterpret_cast<uint4*>(d), vecs,
                                                reinterpret_cast<uint16_t*>(d + vecs * 16),
                                                static_cast<int>(bytes - vecs * 16) / 2);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (a.n == 0) return cudaSuccess;
    // Fewer slabs a CTA leave more of its warps for a frequent token's items,
    // but more CTAs read the tokens (8, 4 and 2 a CTA: 600 x 384 6.4 us, 6.5,
    // 5.3; 1,200 x 512 9.2, 9.2, 9.8; 600 x 1,024 10.7, 7.9, 8.1; 512 x 2,048
    // 10.4, 9.1, 11.3; 300 x 8,192 12.2, 14.6, 22.1).
    a.direct = a.slabs <= 4 && a.n <= 1024 ? 2 : a.slabs <= 16 ? 4 : kDirectWarps;
    cfg.gridDim = dim3(a.n, ceil_div(a.slabs, a.direct));
    cfg.blockDim = dim3(kDirectThreads);
    return cudaLaunchKernelEx(&cfg, a.n <= 1024 ? direct_kernel<TI, TO, kVec, 1024> : direct_kernel<TI, TO, kVec, 4096>,
                              a);
  }
  a.R = p.R;
  a.keep = p.keep;
  a.pieces = p.pieces;
  a.n_sorted = reinterpret_cast<int*>(ws + p.off_n);
  a.sorted = reinterpret_cast<int4*>(ws + p.off_sorted);
  a.parts = reinterpret_cast<float*>(ws + p.off_parts);
  // The limit is the function's, on the device, for all host threads: one that
  // went by this call's sizes could be lowered by another thread before the
  // launch below.
  cudaError_t e = cudaFuncSetAttribute(sort_kernel<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
  if (e != cudaSuccess) return e;
  sort_kernel<TO><<<p.owners, (a.accumulate ? 1 : 2) * kSortThreads, p.smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(p.pieces * p.slabs);
  cfg.blockDim = dim3(kSumThreads);
  cfg.numAttrs = 1;
  auto sum = a.accumulate ? sum_kernel<TI, TO, kVec, true> : sum_kernel<TI, TO, kVec, false>;
  cfg.dynamicSmemBytes = a.accumulate ? sizeof(SumShared<TI, TO, kVec, true>) : sizeof(SumShared<TI, TO, kVec, false>);
  e = cudaFuncSetAttribute(sum, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, sum, a);
  if (e != cudaSuccess) return e;
  static_assert(kDirectAlways >= kPiece, "the sorted path has more than one piece");
  cfg.gridDim = dim3(ceil_div(p.pieces, kJoinWarps) * p.slabs);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<TI, TO, kVec>, a);
}

template <typename TI, typename TO>
cudaError_t launch_grad(const GradArgs& a, char* ws, cudaStream_t s) {
  return a.r % kLane<TI> == 0 ? launch_grad<TI, TO, true>(a, ws, s) : launch_grad<TI, TO, false>(a, ws, s);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_embed(const void* table, dspark_dtype table_dtype, const int32_t* tokens, int n, int V, int r,
                           float scale, void* out, dspark_dtype out_dtype, void* workspace, size_t ws_bytes,
                           dspark_stream_t stream) {
  if (!is_element_type(table_dtype) || !is_element_type(out_dtype) || !embed_sizes_ok(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  if (n == 0) return DSPARK_OK;
  if (!is_given(table) || !is_given(tokens) || !is_given(out) || !is_given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  const EmbedArgs a{table, tokens, n, V, r, scale, out,
                    reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32_out = out_dtype == DSPARK_F32;
  const cudaError_t e =
      table_dtype == DSPARK_F32
          ? (f32_out ? launch_embed<float, float>(a, s) : launch_embed<float, uint16_t>(a, s))
          : (f32_out ? launch_embed<uint16_t, float>(a, s) : launch_embed<uint16_t, uint16_t>(a, s));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

size_t dspark_embed_grad_workspace_bytes(int n, int V, int r) {
  return embed_sizes_ok(n, V, r) ? std::max(grad_plan(n, V, r, 4).bytes, grad_plan(n, V, r, 8).bytes) : 0;
}

dspark_status dspark_embed_grad(const void* dout, dspark_dtype dout_dtype, const int32_t* tokens, int n, int V, int r,
                                float scale, int accumulate, void* dtable, dspark_dtype dtable_dtype,
                                void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (!is_element_type(dout_dtype) || !is_element_type(dtable_dtype) || !embed_sizes_ok(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DSPARK_ERR_INVALID_ARG;
  if (!is_given(dtable) || !is_given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (n > 0 && (!is_given(dout) || !is_given(tokens))) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < dspark_embed_grad_workspace_bytes(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  GradArgs a{};
  a.dout = dout;
  a.tokens = tokens;
  a.n = n;
  a.V = V;
  a.r = r;
  a.scale = scale;
  a.accumulate = accumulate;
  a.dtable = dtable;
  char* ws = static_cast<char*>(workspace);
  a.err = reinterpret_cast<unsigned*>(ws + kErrOffset);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dout_dtype == DSPARK_F32
          ? (dtable_dtype == DSPARK_F32 ? launch_grad<float, float>(a, ws, s) : launch_grad<float, uint16_t>(a, ws, s))
          : (dtable_dtype == DSPARK_F32 ? launch_grad<uint16_t, float>(a, ws, s)
                                        : launch_grad<uint16_t, uint16_t>(a, ws, s));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
