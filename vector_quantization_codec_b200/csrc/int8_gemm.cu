// int8_gemm.cu -- product of 8-bit integers with a scale per token and per
// output channel:
//   Y[t][i] = T(float(sum_j xq[t][j] wq[i][j]) * (x_scale_t * w_scale_i)).
// The sum is an exact 32-bit integer (|sum| <= 128 * 128 * 32768 = 2^29), so no
// order of summation changes a result.
#include "common.cuh"
#include "launch.cuh"

namespace qamw {
namespace {

constexpr int kSimpleTile = 64;

struct Int8GemmArgs {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int ntok, d_out, d_in;
};

__device__ __forceinline__ void put(float* y, int64_t at, float v) { y[at] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, int64_t at, float v) {
  y[at] = __float2bfloat16_rn(v);
}

template <typename T>
__global__ void __launch_bounds__(256) k_int8_gemm(const Int8GemmArgs a) {
  __shared__ int xs[kSimpleTile][17], ws[kSimpleTile][17];
  const int64_t i0 = (int64_t)blockIdx.x * kSimpleTile;
  const int t0 = blockIdx.y * kSimpleTile;
  const int ti = threadIdx.x & 15, tt = threadIdx.x >> 4;
  int acc[4][4] = {};
  pdl_wait();
  pdl_trigger();
  for (int k0 = 0; k0 < a.d_in; k0 += 64) {
    for (int e = threadIdx.x; e < kSimpleTile * 16; e += 256) {
      const int r = e >> 4, k = e & 15;
      xs[r][k] = t0 + r < a.ntok
                     ? *reinterpret_cast<const int*>(a.x + (int64_t)(t0 + r) * a.d_in + k0 + 4 * k)
                     : 0;
      ws[r][k] = i0 + r < a.d_out
                     ? *reinterpret_cast<const int*>(a.w + (i0 + r) * a.d_in + k0 + 4 * k)
                     : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          acc[r][s] = __dp4a(xs[tt + 16 * r][k], ws[ti + 16 * s][k], acc[r][s]);
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int t = t0 + tt + 16 * r;
      const int64_t i = i0 + ti + 16 * s;
      if (t < a.ntok && i < a.d_out)
        put(reinterpret_cast<T*>(a.y), (int64_t)t * a.d_out + i,
            __fmul_rn((float)acc[r][s], __fmul_rn(a.xs[t], a.ws[i])));
    }
}

}  // namespace

cudaError_t launch_int8_gemm(const int8_t* d_x, const float* d_x_scale, int ntok, const int8_t* d_w,
                             const float* d_w_scale, int d_out, int d_in, void* d_y, int dtype,
                             int32_t* d_status, cudaStream_t stream) {
  (void)d_status;
  Int8GemmArgs a = {d_x, d_x_scale, d_w, d_w_scale, d_y, ntok, d_out, d_in};
  const dim3 grid((unsigned)((d_out + kSimpleTile - 1) / kSimpleTile),
                  (unsigned)((ntok + kSimpleTile - 1) / kSimpleTile));
  return dtype == QAMW_DTYPE_F32
             ? launch_pdl(k_int8_gemm<float>, grid, dim3(256), 0, stream, a)
             : launch_pdl(k_int8_gemm<__nv_bfloat16>, grid, dim3(256), 0, stream, a);
}

}  // namespace qamw
