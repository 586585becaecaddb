// Embedding lookup with scaling, and its gradient with respect to the table.
#include <algorithm>

#include "common.cuh"

namespace dspark {
namespace {

constexpr int kMaxItems = 1 << 24;
constexpr int kThreads = 256;

struct EmbedArgs {
  const void* table;
  const int32_t* tokens;
  int n, V, r;
  float scale;
  void* out;
  unsigned* err;
};

struct EmbedGradArgs {
  const void* dout;
  const int32_t* tokens;
  int n, V, r;
  float scale;
  int accumulate;
  void* dtable;
  unsigned* err;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) {
  asm volatile("{ .reg .b16 h; cvt.rn.bf16.f32 h, %1; st.global.b16 [%0], h; }" ::"l"(p), "f"(v) : "memory");
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a) {
  const int i = blockIdx.x;
  const int t = a.tokens[i];
  TO* out = static_cast<TO*>(a.out) + static_cast<long long>(i) * a.r;
  const bool ok = t >= 0 && t < a.V;
  if (!ok && t != -1 && threadIdx.x == 0)
    set_error(a.err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(i));
  const TI* row = static_cast<const TI*>(a.table) + static_cast<long long>(ok ? t : 0) * a.r;
  for (int k = threadIdx.x; k < a.r; k += kThreads) store(out + k, ok ? to_float(row[k]) * a.scale : 0.f);
}

template <typename TO>
__global__ void __launch_bounds__(kThreads) zero_kernel(EmbedGradArgs a) {
  TO* d = static_cast<TO*>(a.dtable) + static_cast<long long>(blockIdx.x) * a.r;
  for (int k = threadIdx.x; k < a.r; k += kThreads) store(d + k, 0.f);
}

// One CTA an item; the CTA of a token's first item sums all of that token's
// items in order.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) embed_grad_kernel(EmbedGradArgs a) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int t = a.tokens[i];
  if (t < 0 || t >= a.V) {
    if (t != -1 && tid == 0) set_error(a.err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(i));
    return;
  }
  int before = 0;
  for (int j = tid; j < i; j += kThreads) before |= a.tokens[j] == t;
  if (__syncthreads_or(before)) return;
  TO* d = static_cast<TO*>(a.dtable) + static_cast<long long>(t) * a.r;
  for (int k0 = 0; k0 < a.r; k0 += kThreads) {
    const int k = k0 + tid;
    float s = 0.f;
    for (int j = i; j < a.n; ++j)
      if (a.tokens[j] == t && k < a.r) s += to_float(static_cast<const TI*>(a.dout)[static_cast<long long>(j) * a.r + k]);
    if (k < a.r) store(d + k, a.accumulate ? fmaf(s, a.scale, to_float(d[k])) : s * a.scale);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p != nullptr && aligned16(p); }
bool dtype_ok(dspark_dtype t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool embed_sizes_ok(int n, int V, int r) {
  return n >= 0 && n <= kMaxItems && V >= 1 && V <= kMaxV && r >= 1 && r <= DSPARK_MAX_EMBED_R;
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
  auto kernel = table_dtype == DSPARK_F32
                    ? (out_dtype == DSPARK_F32 ? embed_kernel<float, float> : embed_kernel<float, uint16_t>)
                    : (out_dtype == DSPARK_F32 ? embed_kernel<uint16_t, float> : embed_kernel<uint16_t, uint16_t>);
  kernel<<<n, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

size_t dspark_embed_grad_workspace_bytes(int n, int V, int r) {
  if (!embed_sizes_ok(n, V, r)) return 0;
  return kScratchOffset;
}

dspark_status dspark_embed_grad(const void* dout, dspark_dtype dout_dtype, const int32_t* tokens, int n, int V, int r,
                                float scale, int accumulate, void* dtable, dspark_dtype dtable_dtype,
                                void* workspace, size_t ws_bytes, dspark_stream_t stream) {
  if (!dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype) || !embed_sizes_ok(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DSPARK_ERR_INVALID_ARG;
  if (!given(dtable) || !given(workspace)) return DSPARK_ERR_INVALID_ARG;
  if (n > 0 && (!given(dout) || !given(tokens))) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < dspark_embed_grad_workspace_bytes(n, V, r)) return DSPARK_ERR_INVALID_ARG;
  const EmbedGradArgs a{dout, tokens, n, V, r, scale, accumulate, dtable,
                        reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kErrOffset)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!accumulate) (dtable_dtype == DSPARK_F32 ? zero_kernel<float> : zero_kernel<uint16_t>)<<<V, kThreads, 0, s>>>(a);
  if (n > 0) {
    auto kernel =
        dout_dtype == DSPARK_F32
            ? (dtable_dtype == DSPARK_F32 ? embed_grad_kernel<float, float> : embed_grad_kernel<float, uint16_t>)
            : (dtable_dtype == DSPARK_F32 ? embed_grad_kernel<uint16_t, float> : embed_grad_kernel<uint16_t, uint16_t>);
    kernel<<<n, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
