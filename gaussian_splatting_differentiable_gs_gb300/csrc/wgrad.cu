// wgrad.cu -- gs_act8_wgrad: the weight gradient dw = dy^T x8 of a linear
// layer from the 8-bit checkpoint of its input.
#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kTile = 64, kStep = 16;

template <typename T, typename TO>
__global__ void __launch_bounds__(256) wgrad_kernel(int64_t tokens, int rows, int C, const T* dy,
                                                    int64_t dys, const int8_t* q, int64_t qs,
                                                    const uint8_t* e, int64_t es, TO* dw,
                                                    int64_t dws, int accumulate) {
  __shared__ float a[kStep][kTile + 1], b[kStep][kTile + 1];
  const int n0 = blockIdx.x * kTile, k0 = blockIdx.y * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < tokens; t0 += kStep) {
    for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
      const int s = i / kTile, c = i % kTile;
      const int64_t t = t0 + s;
      a[s][c] = t < tokens && n0 + c < rows ? to_f32(dy[t * dys + n0 + c]) : 0.f;
      b[s][c] = t < tokens && k0 + c < C
                    ? (float)q[t * qs + k0 + c] * act8_step(e[t * es + (k0 + c) / GS_ACT8_GROUP])
                    : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += a[s][ty + 16 * i] * b[s][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + ty + 16 * i, c = k0 + tx + 16 * j;
      if (n < rows && c < C) {
        TO* p = dw + n * dws + c;
        *p = from_f32<TO>(acc[i][j] + (accumulate ? to_f32(*p) : 0.f));
      }
    }
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_act8_wgrad_workspace_bytes(int64_t tokens, int32_t rows, int32_t channels,
                                                int32_t dtype) {
  if (tokens < 0 || rows < 1 || channels < 1 || !dtype_ok(dtype)) return 0;
  return 256;
}

extern "C" gs_status gs_act8_wgrad(int64_t tokens, int32_t rows, int32_t channels, int32_t dtype,
                                   const void* dy, int64_t dy_stride, const int8_t* q,
                                   int64_t q_stride, const uint8_t* e, int64_t e_stride, void* dw,
                                   int64_t dw_stride, int32_t out_dtype, int32_t accumulate,
                                   void* workspace, size_t ws_bytes, void* stream) {
  if (tokens < 0 || tokens >= ((int64_t)1 << 31) || rows < 1 || channels < 1 || !dtype_ok(dtype) ||
      (out_dtype != GS_F32 && out_dtype != GS_BF16) || !dw ||
      !aligned_to(dw, dtype_size(out_dtype)) || !workspace || !aligned16(workspace) ||
      ws_bytes < gs_act8_wgrad_workspace_bytes(tokens, rows, channels, dtype))
    return GS_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !q || !e || !aligned_to(dy, dtype_size(dtype)) || !aligned16(q) ||
                     q_stride % 16))
    return GS_ERR_INVALID_ARG;
  const dim3 grid((unsigned)div_up(rows, kTile), (unsigned)div_up(channels, kTile));
  cudaStream_t st = (cudaStream_t)stream;
#define GS_WGRAD(T, TO)                                                                        \
  wgrad_kernel<T, TO><<<grid, 256, 0, st>>>(tokens, rows, channels, (const T*)dy, dy_stride, q, \
                                            q_stride, e, e_stride, (TO*)dw, dw_stride,          \
                                            accumulate)
#define GS_WGRAD_OUT(T) \
  do { if (out_dtype == GS_F32) GS_WGRAD(T, float); else GS_WGRAD(T, __nv_bfloat16); } while (0)
  if (dtype == GS_BF16) GS_WGRAD_OUT(__nv_bfloat16);
  else if (dtype == GS_F16) GS_WGRAD_OUT(__half);
  else GS_WGRAD_OUT(float);
#undef GS_WGRAD_OUT
#undef GS_WGRAD
  GS_CHECK_LAUNCH();
  return GS_OK;
}
