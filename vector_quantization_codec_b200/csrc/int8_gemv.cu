// int8_gemv.cu -- the 8-bit product for a few tokens (decoding): every weight
// byte is read once and takes part in a handful of four-way integer dot
// products, so the call is bound by the weights' way from HBM and, for small
// matrices, by latency.  The sums are the exact integers of int8_gemm.cu.
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace qamw {
namespace {

constexpr int kGemvWarps = 8;

struct Int8GemvArgs {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int ntok, d_out, d_in;
  int per_row;  // warps that share a row: 1, 2, 4 or 8
};

__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// The tokens sit in shared memory; a warp takes ROWS rows of W at a time (or,
// where there are fewer rows than warps to fill the machine with, its share of
// the rows' 512-byte pieces, the shares added up through shared memory), 16
// bytes a lane, 4 KB of W in flight.  Each 16 bytes of a token that come out of
// shared memory serve ROWS rows: with two tokens and more that is what keeps the
// shared memory from being the bound.
template <int NTOK, int ROWS, typename T>
__global__ void __launch_bounds__(kGemvWarps * 32, 4) k_int8_gemv(const Int8GemvArgs a) {
  constexpr int kAhead = 8 / ROWS;
  // [NTOK][d_in / 16], and room for the reads past the end (which meet zeros of W)
  extern __shared__ __align__(16) uint4 xv[];
  __shared__ int part[2][kGemvWarps][ROWS][NTOK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nv = a.d_in / 16, G = a.per_row, g = warp % G, mine = warp / G;
  const int rows_cta = kGemvWarps / G * ROWS;
  const int64_t step = (int64_t)gridDim.x * rows_cta;
  T* y = reinterpret_cast<T*>(a.y);
  // While the kernel ahead finishes: the first rows on their way into L2, whatever they
  // hold by then; the loads that count come after the wait.  Back to back, 1 token:
  // 4096 -> 4096 4.6 us without, 3.8 with, 4096 -> 11008 8.9 and 7.5; behind a norm of
  // the token 6.3 and 5.6 for the two.
  {
    const int64_t r = (int64_t)blockIdx.x * rows_cta + mine * ROWS;
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int v = (j * G + g) * 32 + lane;
        if ((lane & 7) == 0 && v < nv && r + k < a.d_out)  // a line a lane
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w + ((r + k) * nv + v) * 16));
      }
  }
  pdl_wait();
  pdl_trigger();
  uint4 w[ROWS][kAhead];
  const auto load = [&](int64_t r, int v0) {  // zeros past the ends
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const uint4* row = reinterpret_cast<const uint4*>(a.w) + (r + k) * nv;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int v = v0 + j * 32 * G;
        w[k][j] = v < nv && r + k < a.d_out ? __ldcs(row + v) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  int64_t r = (int64_t)blockIdx.x * rows_cta + mine * ROWS;  // this warp's first row
  load(r, g * 32 + lane);                                    // in flight while the tokens come in
  for (int v = threadIdx.x; v < NTOK * nv; v += kGemvWarps * 32)
    xv[v] = v < a.ntok * nv ? reinterpret_cast<const uint4*>(a.x)[v] : make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * rows_cta; r0 < a.d_out; r0 += step, r += step) {
    int acc[ROWS][NTOK];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int t = 0; t < NTOK; ++t) acc[k][t] = 0;
    for (int v0 = g * 32 + lane; v0 - lane < nv;) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
#pragma unroll
        for (int t = 0; t < NTOK; ++t) {
          const uint4 x = xv[t * nv + v0 + j * 32 * G];
#pragma unroll
          for (int k = 0; k < ROWS; ++k) acc[k][t] = dot16(w[k][j], x, acc[k][t]);
        }
      }
      v0 += kAhead * 32 * G;
      if (v0 - lane < nv) load(r, v0);
    }
    // the next rows' first pieces, ahead of these rows' reduction
    load(r + step, g * 32 + lane);
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int t = 0; t < NTOK; ++t) acc[k][t] = __reduce_add_sync(0xffffffffu, acc[k][t]);
    if (G > 1) {
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
#pragma unroll
          for (int t = 0; t < NTOK; ++t) part[parity][warp][k][t] = acc[k][t];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
#pragma unroll
        for (int t = 0; t < NTOK; ++t) {
          acc[k][t] = 0;
          for (int h = 0; h < G; ++h) acc[k][t] += part[parity][mine * G + h][k][t];
        }
      parity ^= 1;
    }
    if (g == 0 && lane == 0) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (r + k < a.d_out) {
          const float wi = a.ws[r + k];
#pragma unroll
          for (int t = 0; t < NTOK; ++t)
            if (t < a.ntok)
              put(y + (int64_t)t * a.d_out + r + k,
                  __fmul_rn((float)acc[k][t], __fmul_rn(a.xs[t], wi)));
        }
    }
  }
}

template <int NTOK, int ROWS, typename T>
cudaError_t run_gemv(Int8GemvArgs a, cudaStream_t stream) {
  auto fn = &k_int8_gemv<NTOK, ROWS, T>;
  const void* p = reinterpret_cast<const void*>(fn);
  a.per_row = 1;
  while (a.per_row < kGemvWarps && (int64_t)a.d_out * a.per_row < 24 * ROWS * sm_count() &&
         a.per_row * 2 * 512 <= a.d_in)
    a.per_row *= 2;
  const size_t smem = (size_t)NTOK * a.d_in + (size_t)(8 / ROWS) * 512 * a.per_row;
  cudaError_t err = allow_smem(p, smem + 1024);
  if (err != cudaSuccess) return err;
  const int rows_cta = kGemvWarps / a.per_row * ROWS;
  const int grid = persistent_grid(p, kGemvWarps * 32, smem, ((int64_t)a.d_out + rows_cta - 1) / rows_cta);
  return launch_pdl(fn, dim3(grid), dim3(kGemvWarps * 32), smem, stream, a);
}

template <typename T>
cudaError_t run_gemv_any(const Int8GemvArgs& a, cudaStream_t stream) {
  if (a.ntok == 1) return run_gemv<1, 1, T>(a, stream);
  if (a.ntok == 2) return run_gemv<2, 1, T>(a, stream);
  return run_gemv<4, 2, T>(a, stream);
}

}  // namespace

cudaError_t launch_int8_gemv(const int8_t* d_x, const float* d_x_scale, int ntok, const int8_t* d_w,
                             const float* d_w_scale, int d_out, int d_in, void* d_y, int dtype,
                             cudaStream_t stream) {
  const Int8GemvArgs a = {d_x, d_x_scale, d_w, d_w_scale, d_y, ntok, d_out, d_in, 1};
  return dtype == QAMW_DTYPE_F32 ? run_gemv_any<float>(a, stream)
                                 : run_gemv_any<__nv_bfloat16>(a, stream);
}

}  // namespace qamw
