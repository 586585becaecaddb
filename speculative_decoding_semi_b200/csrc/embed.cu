// Embedding lookup with scaling, and its gradient with respect to the table
// by sorted tokens.
#include <algorithm>

#include "common.cuh"

namespace dspark {
namespace {

constexpr int kMaxItems = 1 << 24;
constexpr int kMaxSms = 148;   // owners of table rows, one CTA each (more only for very large V)

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }

// Two fp32 values as a pair of bf16, rounded to nearest even.
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  unsigned r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.f)); }

__device__ __forceinline__ void record_bad_token(unsigned* err, int item) {
  set_error(err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(item));
}

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
template <int N>
__device__ __forceinline__ void save_cols(float* p, const float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4)
    *reinterpret_cast<float4*>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
}
template <int N>
__device__ __forceinline__ void save_cols(uint16_t* p, const float (&v)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// blockDim.x threads a row (kCols columns each, or single ones where r is no
// multiple of kCols), blockDim.y * kRows rows a CTA, kRows of them in flight a
// thread.
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
      if (threadIdx.x == 0) record_bad_token(a.err, i);
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
        save_cols<N>(q, v[u]);
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
  // four rows a thread once that fills the GPU
  const int rows = static_cast<long long>(a.n) >= 8ll * kMaxSms * block.y ? 4 : 1;
  const int grid = ceil_div(a.n, static_cast<int>(block.y) * rows);
  auto kernel = vec ? (rows == 4 ? embed_kernel<TI, TO, true, 4> : embed_kernel<TI, TO, true, 1>)
                    : (rows == 4 ? embed_kernel<TI, TO, false, 4> : embed_kernel<TI, TO, false, 1>);
  kernel<<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

// -------------------------------------------------------------- gradient
//
// dtable[v] = scale * sum of dout's rows whose token is v. Two kernels:
//
// sort_kernel: CTA g owns table rows [g R, (g+1) R). It reads all n tokens,
//   counts those below its rows (its offset in the sorted order, so the CTAs
//   need not talk to each other) and counting-sorts its own, stably: each of
//   16 warps takes a contiguous piece of the tokens, keeps its matches in
//   order, counts them per row, and places them after the earlier warps'.
//   It then zeroes its rows that no token points at.
// sum_kernel: the sorted items in equal pieces, whatever the lengths of the
//   runs of equal tokens, so that a frequent token is summed by many CTAs. A
//   run inside a piece is written at once; the parts of a run that crosses
//   pieces go to scratch, and the CTA that delivers the last part (a counter)
//   adds them in order. Which CTA that is does not change the order.
//
// Few items with accumulate: direct_kernel, one CTA an item, no sorting.

struct GradArgs {
  const void* dout;
  const int32_t* tokens;
  int n, V, r;
  float scale;
  int accumulate;
  void* dtable;
  unsigned* err;
  int R, slabs, pieces;   // table rows of an owner; 128-column slabs; pieces of the sorted items
  int* n_sorted;          // items with a token
  unsigned* arrived;      // [pieces][slabs] parts of the run that starts in a piece and leaves it
  int4* sorted;           // [n] item, token, and the run [begin, end) it is in
  float* parts;           // [pieces][2][slabs * 128]: of the run that comes in, of the run that leaves
};

constexpr int kSortWarps = 16, kSortThreads = kSortWarps * 32;
constexpr int kMaxR = 2048;     // rows of an owner (11 bits beside 20 of an item's place in a warp's piece)
constexpr int kKeep = 512;      // matches that a warp keeps in shared memory; more are found again
constexpr int kSumWarps = 8, kSumThreads = kSumWarps * 32;
constexpr int kSlab = 128;      // columns of a warp's quad: four a lane
constexpr int kDirectItems = 1024;
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

template <typename TO>
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(GradArgs a) {
  extern __shared__ unsigned smem[];
  unsigned* hist = smem;                                   // [16][R] counts, then places
  unsigned* total = hist + kSortWarps * a.R;               // [R] tokens of a row
  unsigned* kept = total + a.R;                            // [16][kKeep]
  __shared__ unsigned s_below, s_red[kSortWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, R = a.R, n = a.n;
  const int v0 = blockIdx.x * R, rows = min(R, a.V - v0);
  const unsigned lt = (1u << lane) - 1u;
  for (int k = tid; k < kSortWarps * R; k += kSortThreads) hist[k] = 0;
  if (tid == 0) s_below = 0;
  for (int k = blockIdx.x * kSortThreads + tid; k < a.pieces * a.slabs; k += gridDim.x * kSortThreads) a.arrived[k] = 0;
  __syncthreads();

  // each warp's matches, in order: four neighbouring tokens a lane
  const int len = ceil_div(ceil_div(n, kSortWarps), 128) * 128;
  const int lo = min(n, w * len), hi = min(n, lo + len);
  unsigned* mine = kept + w * kKeep;
  unsigned* count = hist + w * R;
  int found = 0;
  unsigned below = 0;
  constexpr int kAhead = 8;
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
      bool any = false, bad = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        bad |= t[c] < -1 || t[c] >= a.V;
        below += t[c] >= 0 && t[c] < v0;
        hit[c] = t[c] >= v0 && t[c] < v0 + rows;
        any |= hit[c];
      }
      if (bad && blockIdx.x == 0)
        for (int c = 0; c < 4; ++c)
          if (t[c] < -1 || t[c] >= a.V) record_bad_token(a.err, i + c);
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
        if (at < kKeep) mine[at] = (static_cast<unsigned>(i + c - lo) << 11) | off;
        ++at;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0 && below != 0u) atomicAdd(&s_below, below);
  __syncthreads();

  // places: rows in order, within a row the warps in order
  const int per = ceil_div(rows, kSortThreads), r0 = min(rows, tid * per), r1 = min(rows, r0 + per);
  unsigned sum = 0;
  for (int k = r0; k < r1; ++k) {
    unsigned c = 0;
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) {
      const unsigned x = hist[j * R + k];
      hist[j * R + k] = c;
      c += x;
    }
    total[k] = c;
    sum += c;
  }
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_red[w] = inc;
  __syncthreads();
  unsigned place = s_below + inc - sum;
  for (int j = 0; j < w; ++j) place += s_red[j];
  for (int k = r0; k < r1; ++k) {
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) hist[j * R + k] += place;
    place += total[k];
  }
  if (blockIdx.x == gridDim.x - 1 && tid == kSortThreads - 1) *a.n_sorted = static_cast<int>(place);
  __syncthreads();

  auto put = [&](bool hit, unsigned off, int item) {   // by the whole warp
    const unsigned peers = __match_any_sync(0xffffffffu, hit ? off : 0xffffffffu);
    if (hit) {
      const int at = static_cast<int>(count[off]) + __popc(peers & lt);
      // the run: warp 0's first place to the last warp's end
      a.sorted[at] = make_int4(item, v0 + static_cast<int>(off), 0, 0);
    }
    __syncwarp();
    if (hit && (peers & lt) == 0u) count[off] += __popc(peers);
    __syncwarp();
  };
  if (found <= kKeep) {
    for (int k0 = 0; k0 < found; k0 += 32) {
      const bool hit = k0 + lane < found;
      const unsigned e = hit ? mine[k0 + lane] : 0u;
      put(hit, e & 2047u, lo + static_cast<int>(e >> 11));
    }
  } else {
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane, t = i < hi ? __ldg(a.tokens + i) : -1;
      const unsigned off = static_cast<unsigned>(t - v0);
      const bool hit = t >= 0 && off < static_cast<unsigned>(rows);
      if (__any_sync(0xffffffffu, hit)) put(hit, off, i);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  // after the placement the last warp's place is each run's end
  const unsigned* ends = hist + (kSortWarps - 1) * R;
  for (int k = w; k < rows; k += kSortWarps) {
    const int c = static_cast<int>(total[k]), end = static_cast<int>(ends[k]);
    for (int j = lane; j < c; j += 32) {
      int4* s = a.sorted + (end - c + j);
      reinterpret_cast<int2*>(s)[1] = make_int2(end - c, end);
    }
    if (c == 0 && !a.accumulate) zero_row(static_cast<TO*>(a.dtable) + static_cast<long long>(v0 + k) * a.r, a.r, lane);
  }
}

// Four columns of a row: neighbours (r a multiple of 4), or 32 apart. A slab
// of a warp is kQuads times 128 columns.
template <typename T, bool kVec>
__device__ __forceinline__ float4 load_quad(const T* p, int lane, int cols) {
  float4 v = make_float4(0, 0, 0, 0);
  if constexpr (!kVec) {
    if (lane < cols) v.x = to_float(p[lane]);
    if (lane + 32 < cols) v.y = to_float(p[lane + 32]);
    if (lane + 64 < cols) v.z = to_float(p[lane + 64]);
    if (lane + 96 < cols) v.w = to_float(p[lane + 96]);
  } else if (lane * 4 < cols) {
    if constexpr (sizeof(T) == 4) {
      v = __ldcs(reinterpret_cast<const float4*>(p) + lane);
    } else {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p) + lane);
      v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                      __uint_as_float(u.y & 0xffff0000u));
    }
  }
  return v;
}
template <typename T, bool kVec>
__device__ __forceinline__ void save_quad(T* p, int lane, int cols, float4 v) {
  if constexpr (!kVec) {
    if (lane < cols) store(p + lane, v.x);
    if (lane + 32 < cols) store(p + lane + 32, v.y);
    if (lane + 64 < cols) store(p + lane + 64, v.z);
    if (lane + 96 < cols) store(p + lane + 96, v.w);
  } else if (lane * 4 < cols) {
    if constexpr (sizeof(T) == 4)
      reinterpret_cast<float4*>(p)[lane] = v;
    else
      reinterpret_cast<uint2*>(p)[lane] = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

__device__ __forceinline__ float4 plus(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// dtable[token, quad] (+)= scale * sum; `col` the quad's first column
template <typename TO, bool kVec>
__device__ __forceinline__ void finish(const GradArgs& a, int token, int col, int lane, float4 s) {
  TO* d = static_cast<TO*>(a.dtable) + static_cast<long long>(token) * a.r + col;
  s = make_float4(s.x * a.scale, s.y * a.scale, s.z * a.scale, s.w * a.scale);
  if (a.accumulate) s = plus(s, load_quad<TO, kVec>(d, lane, a.r - col));
  save_quad<TO, kVec>(d, lane, a.r - col, s);
}

// A piece is kSumWarps * P sorted items, P a warp, on one slab.
template <typename TI, typename TO, bool kVec, int kQuads, int P>
__global__ void __launch_bounds__(kSumThreads, 4) sum_kernel(GradArgs a) {
  constexpr int kPiece = kSumWarps * P;
  constexpr int kRowsAhead = 8 / kQuads;
  __shared__ float4 s_part[kSumWarps][2][kQuads][32];
  __shared__ int4 s_run[kSumWarps][2];   // token, begin, end of each part; token -1: none
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = blockIdx.x / a.slabs, slab = blockIdx.x - piece * a.slabs;
  const int p0 = piece * kPiece, lo = p0 + w * P, col0 = slab * kQuads * kSlab;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // what lies behind the last sorted item is read but not used
  int4 it = make_int4(0, -1, 0, 0);
  if (lane < P && lo + lane < a.n) it = __ldcg(a.sorted + lo + lane);
  const int N = __ldcg(a.n_sorted);
  if (p0 >= N) return;
  const int hi = min(N, lo + P);
  const TI* dout = static_cast<const TI*>(a.dout) + col0;
  if (lane < 2) s_run[w][lane].x = -1;
  const unsigned ends = __ballot_sync(0xffffffffu, lo + lane < hi && (lo + lane == it.w - 1 || lo + lane == hi - 1));
  float4 sum[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) sum[q] = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int j0 = 0; lo + j0 < hi && j0 < P; j0 += kRowsAhead) {
    float4 x[kRowsAhead][kQuads];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int item = __shfl_sync(0xffffffffu, it.x, j0 + u);
#pragma unroll
      for (int q = 0; q < kQuads; ++q)
        x[u][q] = lo + j0 + u < hi ? load_quad<TI, kVec>(dout + static_cast<long long>(item) * a.r + q * kSlab, lane,
                                                         a.r - col0 - q * kSlab)
                                   : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
#pragma unroll
      for (int q = 0; q < kQuads; ++q) sum[q] = plus(sum[q], x[u][q]);
      if ((ends >> (j0 + u)) & 1u) {      // the run, or this warp's part of it, ends here
        const int token = __shfl_sync(0xffffffffu, it.y, j0 + u);
        const int begin = __shfl_sync(0xffffffffu, it.z, j0 + u), end = __shfl_sync(0xffffffffu, it.w, j0 + u);
        const int k = begin < lo ? 0 : 1;       // came in, or leaves
        const bool whole = begin >= lo && end <= hi;
        if (!whole && lane == 0) s_run[w][k] = make_int4(token, begin, end, 0);
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          if (whole)
            finish<TO, kVec>(a, token, col0 + q * kSlab, lane, sum[q]);
          else
            s_part[w][k][q][lane] = sum[q];
          sum[q] = make_float4(0, 0, 0, 0);
        }
      }
    }
  }
  __syncthreads();
  if (w != 0) return;
  // the warps' parts in order: equal tokens are one run
  const int piece_end = min(N, p0 + kPiece);
  int token = -1, begin = 0, end = 0;
#pragma unroll
  for (int q = 0; q < kQuads; ++q) sum[q] = make_float4(0, 0, 0, 0);
  const long long row = static_cast<long long>(a.slabs) * kQuads * kSlab / 4;
  auto flush = [&]() {
    if (token < 0) return;
    if (begin < p0 || end > piece_end) {
      float4* parts = reinterpret_cast<float4*>(a.parts + col0) + lane;
#pragma unroll
      for (int q = 0; q < kQuads; ++q)
        __stcg(parts + (2ll * piece + (begin < p0 ? 0 : 1)) * row + q * kSlab / 4, sum[q]);
      const int first = begin / kPiece, last = (end - 1) / kPiece;
      __threadfence();
      __syncwarp();
      unsigned before = 0;
      if (lane == 0) before = atom_add_acq_rel_gpu(a.arrived + static_cast<long long>(first) * a.slabs + slab, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != static_cast<unsigned>(last - first)) return;
      __threadfence();
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const float4* from = parts + q * kSlab / 4;
        sum[q] = __ldcg(from + (2ll * first + 1) * row);
        int g = first + 1;
        for (; g + 8 <= last + 1; g += 8) {
          float4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = __ldcg(from + 2ll * (g + u) * row);
#pragma unroll
          for (int u = 0; u < 8; ++u) sum[q] = plus(sum[q], x[u]);
        }
        for (; g <= last; ++g) sum[q] = plus(sum[q], __ldcg(from + 2ll * g * row));
      }
    }
#pragma unroll
    for (int q = 0; q < kQuads; ++q) finish<TO, kVec>(a, token, col0 + q * kSlab, lane, sum[q]);
  };
  for (int j = 0; j < kSumWarps * 2; ++j) {
    const int4 run = s_run[j >> 1][j & 1];
    if (run.x < 0) continue;
    if (run.x != token) {
      flush();
      token = run.x;
      begin = run.y;
      end = run.z;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) sum[q] = make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < kQuads; ++q) sum[q] = plus(sum[q], s_part[j >> 1][j & 1][q][lane]);
  }
  flush();
}

// One CTA an item and up to kDirectWarps slabs; the CTA of a token's first
// item sums all of that token's items. Its warps share the slabs and, where
// there are fewer slabs than warps, the items in equal parts.
template <typename TI, typename TO, bool kVec>
__global__ void __launch_bounds__(kDirectThreads) direct_kernel(GradArgs a) {
  constexpr int kLoads = kDirectItems / kDirectThreads;
  __shared__ unsigned s_hits[kDirectItems / 32];
  __shared__ short s_items[kDirectItems];
  __shared__ float4 s_sum[kDirectWarps][32];
  const int i = blockIdx.x, tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  int mine[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int j = u * kDirectThreads + tid;
    mine[u] = j < a.n ? __ldg(a.tokens + j) : -1;
  }
  const int t = __ldg(a.tokens + i);
  if (t < 0 || t >= a.V) {
    if (t != -1 && tid == 0 && blockIdx.y == 0) record_bad_token(a.err, i);
    return;
  }
  bool before = false;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    before |= mine[u] == t && u * kDirectThreads + tid < i;
    const unsigned mask = __ballot_sync(0xffffffffu, mine[u] == t);
    if (lane == 0) s_hits[u * kDirectWarps + w] = mask;
  }
  if (__syncthreads_or(before)) return;
  // the token's items in order
  const unsigned word = s_hits[lane];
  int at = __popc(word);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += x;
  }
  const int total = __shfl_sync(0xffffffffu, at, 31);
  at -= __popc(word);
  if (w == 0)
    for (unsigned m = word; m != 0u; m &= m - 1) s_items[at++] = static_cast<short>(lane * 32 + __ffs(m) - 1);
  __syncthreads();
  const int here = min(kDirectWarps, a.slabs - static_cast<int>(blockIdx.y) * kDirectWarps);   // slabs of this CTA
  const int groups = kDirectWarps / here;
  const int group = w / here, col = (static_cast<int>(blockIdx.y) * kDirectWarps + w % here) * kSlab;
  if (group < groups) {
    const int per = ceil_div(total, groups), lo = min(total, group * per), hi = min(total, lo + per);
    const TI* dout = static_cast<const TI*>(a.dout) + col;
    float4 sum = make_float4(0, 0, 0, 0);
    constexpr int kRowsAhead = 8;
    for (int j = lo; j < hi; j += kRowsAhead) {
      float4 x[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        x[u] = j + u < hi ? load_quad<TI, kVec>(dout + static_cast<long long>(s_items[j + u]) * a.r, lane, a.r - col)
                          : make_float4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) sum = plus(sum, x[u]);
    }
    s_sum[w][lane] = sum;
  }
  __syncthreads();
  if (w >= here) return;
  float4 sum = s_sum[w][lane];
  for (int g = 1; g < groups; ++g) sum = plus(sum, s_sum[g * here + w][lane]);
  finish<TO, kVec>(a, t, col, lane, sum);
}

// Sizes of the two-kernel path for (n, V, r) with slabs of `quads` quads, and
// its scratch.
struct GradPlan {
  int R, owners, slabs, P, pieces;
  size_t smem, off_n, off_arrived, off_sorted, off_parts, bytes;
};
GradPlan grad_plan(int n, int V, int r, int quads) {
  GradPlan p{};
  p.R = std::min(kMaxR, ceil_div(V, kMaxSms));
  p.owners = ceil_div(V, p.R);
  p.slabs = ceil_div(r, quads * kSlab);
  // 32 items a warp where that still makes four CTAs an SM, else 8
  p.P = static_cast<long long>(n) * p.slabs >= 4ll * kMaxSms * kSumWarps * 32 ? 32 : 8;
  p.pieces = std::max(1, ceil_div(n, kSumWarps * p.P));
  p.smem = static_cast<size_t>(kSortWarps * p.R + p.R + kSortWarps * kKeep) * sizeof(unsigned);
  p.off_n = kScratchOffset;
  p.off_arrived = p.off_n + 256;
  p.off_sorted = align_up(p.off_arrived + static_cast<size_t>(p.pieces) * p.slabs * sizeof(unsigned), 256);
  p.off_parts = align_up(p.off_sorted + static_cast<size_t>(n) * sizeof(int4), 256);
  p.bytes = align_up(p.off_parts + static_cast<size_t>(p.pieces) * 2 * p.slabs * quads * kSlab * sizeof(float), 256);
  return p;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p != nullptr && aligned16(p); }
bool dtype_ok(dspark_dtype t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool embed_sizes_ok(int n, int V, int r) {
  return n >= 0 && n <= kMaxItems && V >= 1 && V <= kMaxV && r >= 1 && r <= DSPARK_MAX_EMBED_R;
}

template <typename TI, typename TO, bool kVec, int kQuads>
cudaError_t launch_sorted(GradArgs a, char* ws, cudaStream_t s) {
  const GradPlan p = grad_plan(a.n, a.V, a.r, kQuads);
  a.R = p.R;
  a.slabs = p.slabs;
  a.pieces = p.pieces;
  a.n_sorted = reinterpret_cast<int*>(ws + p.off_n);
  a.arrived = reinterpret_cast<unsigned*>(ws + p.off_arrived);
  a.sorted = reinterpret_cast<int4*>(ws + p.off_sorted);
  a.parts = reinterpret_cast<float*>(ws + p.off_parts);
  cudaError_t e = cudaFuncSetAttribute(sort_kernel<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(p.smem));
  if (e != cudaSuccess) return e;
  sort_kernel<TO><<<p.owners, kSortThreads, p.smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.n == 0) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.pieces * p.slabs);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, p.P == 32 ? sum_kernel<TI, TO, kVec, kQuads, 32> : sum_kernel<TI, TO, kVec, kQuads, 8>, a);
}

template <typename TI, typename TO, bool kVec>
cudaError_t launch_grad(GradArgs a, char* ws, cudaStream_t s) {
  if (a.accumulate && a.n <= kDirectItems) {
    if (a.n == 0) return cudaSuccess;
    a.slabs = ceil_div(a.r, kSlab);
    direct_kernel<TI, TO, kVec><<<dim3(a.n, ceil_div(a.slabs, kDirectWarps)), kDirectThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  // two quads a lane keep as many bytes in flight for bf16 as one for fp32
  if constexpr (sizeof(TI) == 2)
    if (a.r > kSlab) return launch_sorted<TI, TO, kVec, 2>(a, ws, s);
  return launch_sorted<TI, TO, kVec, 1>(a, ws, s);
}

template <typename TI, typename TO>
cudaError_t launch_grad(const GradArgs& a, char* ws, cudaStream_t s) {
  return a.r % 4 == 0 ? launch_grad<TI, TO, true>(a, ws, s) : launch_grad<TI, TO, false>(a, ws, s);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_embed(const void* table, dspark_dtype table_dtype, const int32_t* tokens, int n, int V, int r,
                           float scale, void* out, dspark_dtype out_dtype, void* workspace, size_t ws_bytes,
                           dspark_stream_t stream) {
  if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype) || !embed_sizes_ok(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  if (n == 0) return DSPARK_OK;
  if (!given(table) || !given(tokens) || !given(out) || !given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  const EmbedArgs a{table, tokens, n, V, r, scale, out,
                    reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = table_dtype == DSPARK_F32
                            ? (out_dtype == DSPARK_F32 ? launch_embed<float, float>(a, s) : launch_embed<float, uint16_t>(a, s))
                            : (out_dtype == DSPARK_F32 ? launch_embed<uint16_t, float>(a, s)
                                                       : launch_embed<uint16_t, uint16_t>(a, s));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

size_t dspark_embed_grad_workspace_bytes(int n, int V, int r) {
  return embed_sizes_ok(n, V, r) ? std::max(grad_plan(n, V, r, 1).bytes, grad_plan(n, V, r, 2).bytes) : 0;
}

dspark_status dspark_embed_grad(const void* dout, dspark_dtype dout_dtype, const int32_t* tokens, int n, int V, int r,
                                float scale, int accumulate, void* dtable, dspark_dtype dtable_dtype,
                                void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (!dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype) || !embed_sizes_ok(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DSPARK_ERR_INVALID_ARG;
  if (!given(dtable) || !given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (n > 0 && (!given(dout) || !given(tokens))) return DSPARK_ERR_INVALID_ARG;
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
