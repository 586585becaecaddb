// Log probabilities of given tokens, with entropy and top alternatives, and
// their gradient with respect to the logits.
//
// With m the row's largest logit, a row is reduced to
//   S = sum 2^y,  T = sum y 2^y,  y = (x - m) log2 e,
// so that ln p_v = x_v - m - ln S and the entropy is ln S - ln 2 T/S. The
// difference x - m is taken before the product, so that masks of the type's
// lowest value, and rows with nothing else, stay within range.
#include <algorithm>

#include "common.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr int kMaxItems = 1 << 24;
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
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) {
  asm volatile("{ .reg .b16 h; cvt.rn.bf16.f32 h, %1; st.global.b16 [%0], h; }" ::"l"(p), "f"(v) : "memory");
}

// Order of the alternatives as one number: the logit's order (NaN as -inf, -0
// as 0), then the lowest token.
__device__ __forceinline__ unsigned long long rank_key(float x, int v) {
  x = fmaxf(x, -INFINITY) + 0.f;
  const unsigned b = __float_as_uint(x);
  const unsigned o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<unsigned long long>(o) << 32) | (0xffffffffu - static_cast<unsigned>(v));
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const unsigned o = static_cast<unsigned>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ int key_token(unsigned long long k) {
  return static_cast<int>(0xffffffffu - static_cast<unsigned>(k));
}

constexpr int kThreads = 256;

// One CTA a row, one pass for the sums and one for each alternative.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(ScoreArgs a) {
  __shared__ double redd[33];
  __shared__ float redf[33];
  __shared__ unsigned long long s_best;
  const int item = blockIdx.x, tid = threadIdx.x, V = a.V;
  const int b = item / a.C, c = item - b * a.C;
  const int tok = a.tokens[item];
  bool skip = tok == -1;
  const long long row = a.row_start != nullptr ? a.row_start[b] + c : static_cast<long long>(item);
  if (!skip && (tok < 0 || tok >= V || row < 0 || row >= a.n_rows)) {
    if (tid == 0) set_error(a.err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(item));
    skip = true;
  }
  if (skip) {
    if (tid == 0) {
      a.logprob[item] = 0.f;
      if (a.entropy != nullptr) a.entropy[item] = 0.f;
      if (a.stats != nullptr) a.stats[2ll * item] = a.stats[2ll * item + 1] = 0.f;
    }
    for (int i = tid; i < a.top_k; i += kThreads) {
      a.top_tokens[static_cast<long long>(item) * a.top_k + i] = -1;
      a.top_logprobs[static_cast<long long>(item) * a.top_k + i] = -INFINITY;
    }
    return;
  }
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  float m = -INFINITY;
  for (int v = tid; v < V; v += kThreads) m = fmaxf(m, to_float(x[v]));
  m = block_max<kThreads>(m, redf);
  const float shift = m == -INFINITY ? 0.f : m;
  double S = 0.0, Tsum = 0.0;
  for (int v = tid; v < V; v += kThreads) {
    const float y = fmax_nan((to_float(x[v]) - shift) * kLog2e, kMinExp);
    const float e = exp2f(y);
    S += e;
    Tsum += static_cast<double>(e * y);
  }
  S = block_sum<kThreads>(S, redd);
  Tsum = block_sum<kThreads>(Tsum, redd);
  const double lnS = log(S);
  const bool bad = !(S < 1e300);  // a NaN or +inf in the row
  if (tid == 0) {
    const float xt = to_float(x[tok]);
    float lp = xt == -INFINITY ? xt : static_cast<float>(static_cast<double>(xt) - shift - lnS);
    float H = S > 0.0 ? static_cast<float>(lnS - kLn2 * (Tsum / S)) : 0.f;
    if (bad) lp = H = NAN;
    a.logprob[item] = lp;
    if (a.entropy != nullptr) a.entropy[item] = H;
    if (a.stats != nullptr) {
      a.stats[2ll * item] = bad ? NAN : m;
      a.stats[2ll * item + 1] = bad ? NAN : static_cast<float>(S);
    }
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < a.top_k; ++i) {
    if (tid == 0) s_best = 0ull;
    __syncthreads();
    unsigned long long best = 0ull;
    for (int v = tid; v < V; v += kThreads) {
      const unsigned long long k = rank_key(to_float(x[v]), v);
      if (k < last && k > best) best = k;
    }
    atomicMax(&s_best, best);
    __syncthreads();
    last = s_best;
    __syncthreads();
    if (tid == 0) {
      const long long o = static_cast<long long>(item) * a.top_k + i;
      const float xv = last == 0ull ? -INFINITY : key_value(last);
      a.top_tokens[o] = xv == -INFINITY ? -1 : key_token(last);
      a.top_logprobs[o] = bad ? NAN
                          : xv == -INFINITY
                              ? xv
                              : static_cast<float>(static_cast<double>(xv) - shift - lnS);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(GradArgs a) {
  const int row = blockIdx.x, tid = threadIdx.x, V = a.V;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  T* d = static_cast<T*>(a.dlogits) + row * a.gstride;
  const int tok = a.tokens[row];
  const float m = a.stats[2ll * row], s = a.stats[2ll * row + 1];
  if (tid == 0 && (tok < -1 || tok >= V))
    set_error(a.err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(row));
  if (tok < 0 || tok >= V || m == -INFINITY) {
    for (int v = tid; v < V; v += kThreads) store(d + v, 0.f);
    return;
  }
  // p = 2^y f, ln p = y ln 2 + lf
  const float f = 1.f / s;
  const float lf = static_cast<float>(-log(static_cast<double>(s)));
  const float g = a.g_logprob[row];
  const float gh = a.g_entropy != nullptr ? a.g_entropy[row] : 0.f;
  const float c0 = -g - (a.g_entropy != nullptr ? gh * (lf + a.entropy[row]) : 0.f);
  const float c1 = -gh * static_cast<float>(kLn2);
  for (int v = tid; v < V; v += kThreads) {
    const float xv = to_float(x[v]);
    const float y = fmax_nan((xv - m) * kLog2e, kMinExp);
    const float p = exp2f(y) * f;
    float dv = p * fmaf(c1, y, c0);
    if (v == tok && xv != -INFINITY) dv += g;
    store(d + v, dv);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p != nullptr && aligned16(p); }

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_logprobs(const void* logits, dspark_dtype dtype, int64_t n_rows, int64_t row_stride,
                              const int64_t* row_start, const int32_t* tokens, int B, int C, int V, int top_k,
                              float* logprob, float* entropy, float* stats, int32_t* top_tokens,
                              float* top_logprobs, void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (B < 0 || C < 0 || static_cast<long long>(B) * C > kMaxItems || V < 1 || V > kMaxV) return DSPARK_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > kMaxStride || row_stride < V || row_stride > kMaxStride) return DSPARK_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > DSPARK_MAX_TOP_K) return DSPARK_ERR_INVALID_ARG;
  if (B == 0 || C == 0) return DSPARK_OK;
  if (!given(logits) || !given(tokens) || !given(logprob) || !given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(row_start) || !aligned16(entropy) || !aligned16(stats)) return DSPARK_ERR_INVALID_ARG;
  if (top_k > 0 && (!given(top_tokens) || !given(top_logprobs))) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  const ScoreArgs a{logits, n_rows, row_stride, row_start, tokens, C, V, top_k, logprob, entropy, stats, top_tokens,
                    top_logprobs, reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == DSPARK_F32)
    logprobs_kernel<float><<<B * C, kThreads, 0, s>>>(a);
  else
    logprobs_kernel<uint16_t><<<B * C, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status dspark_logprobs_grad(const void* logits, dspark_dtype dtype, int64_t row_stride,
                                   const int32_t* tokens, const float* stats, const float* entropy,
                                   const float* g_logprob, const float* g_entropy, int N, int V, void* dlogits,
                                   int64_t grad_stride, void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (N < 0 || N > kMaxItems || V < 1 || V > kMaxV) return DSPARK_ERR_INVALID_ARG;
  if (row_stride < V || row_stride > kMaxStride || grad_stride < V || grad_stride > kMaxStride)
    return DSPARK_ERR_INVALID_ARG;
  if (N == 0) return DSPARK_OK;
  if (!given(logits) || !given(tokens) || !given(stats) || !given(g_logprob) || !given(dlogits) || !given(workspace))
    return DSPARK_ERR_INVALID_ARG;
  if (g_entropy != nullptr && (!given(g_entropy) || !given(entropy))) return DSPARK_ERR_INVALID_ARG;
  if (dlogits == logits && row_stride != grad_stride) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < kScratchOffset) return DSPARK_ERR_INVALID_ARG;
  const GradArgs a{logits, row_stride, grad_stride, tokens, stats, entropy, g_logprob, g_entropy, V, dlogits,
                   reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == DSPARK_F32)
    logprobs_grad_kernel<float><<<N, kThreads, 0, s>>>(a);
  else
    logprobs_grad_kernel<uint16_t><<<N, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
