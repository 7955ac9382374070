// int8_gemv.cu -- the 8-bit product for a few tokens (decoding): every weight
// byte is read once and takes part in a handful of products, so the call is bound
// by the weights' way from HBM and, for small matrices, by latency.  The sums are
// the exact integers of int8_gemm.cu.  Measured (B200, back to back over weights
// larger than L2): 1 token 4096 -> 32001 18.8 us (7.0 TB/s), 4096 -> 11008 7.5 us
// (6.0 TB/s), 4096 -> 4096 3.8 us; 5 tokens 4096 -> 32001 22.0 us (6.0 TB/s).
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace qamw {
namespace {

constexpr int kGemvWarps = 8;
constexpr size_t kGemvStatic = 9 * 1024;  // bound on the kernels' static shared memory

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

// One or two tokens.  They sit in shared memory; a warp takes a row of W at a
// time (or, where there are fewer rows than warps to fill the machine with, its
// share of the row's 512-byte pieces, the shares added up through shared memory),
// 16 bytes a lane, 4 KB of W in flight.
constexpr int kAhead = 8;
template <int NTOK, typename T>
__global__ void __launch_bounds__(kGemvWarps * 32, 4) k_int8_gemv(const Int8GemvArgs a) {
  // [NTOK][d_in / 16], the last token's row up to a whole step (reads past the end
  // meet zeros of W)
  extern __shared__ __align__(16) uint4 xv[];
  __shared__ int part[2][kGemvWarps][NTOK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nv = a.d_in / 16, G = a.per_row, g = warp % G, mine = warp / G;
  const int rows_cta = kGemvWarps / G;
  const int64_t step = (int64_t)gridDim.x * rows_cta;
  T* y = reinterpret_cast<T*>(a.y);
  // While the kernel ahead finishes: the first rows on their way into L2, whatever they
  // hold by then; the loads that count come after the wait.  Back to back, 1 token:
  // 4096 -> 4096 4.6 us without, 3.8 with, 4096 -> 11008 8.9 and 7.5; behind a norm of
  // the token 6.3 and 5.6 for the two.
  {
    const int64_t r = (int64_t)blockIdx.x * rows_cta + mine;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int v = (j * G + g) * 32 + lane;
      if ((lane & 7) == 0 && v < nv && r < a.d_out)  // a line a lane
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w + (r * nv + v) * 16));
    }
  }
  pdl_wait();
  pdl_trigger();
  uint4 w[kAhead];
  const auto load = [&](int64_t r, int v0) {  // zeros past the ends
    const uint4* row = reinterpret_cast<const uint4*>(a.w) + r * nv;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int v = v0 + j * 32 * G;
      w[j] = v < nv && r < a.d_out ? __ldcs(row + v) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t r = (int64_t)blockIdx.x * rows_cta + mine;  // this warp's first row
  load(r, g * 32 + lane);                             // in flight while the tokens come in
  for (int v = threadIdx.x; v < NTOK * nv; v += kGemvWarps * 32)
    xv[v] = reinterpret_cast<const uint4*>(a.x)[v];
  __syncthreads();
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * rows_cta; r0 < a.d_out; r0 += step, r += step) {
    int acc[NTOK];
#pragma unroll
    for (int t = 0; t < NTOK; ++t) acc[t] = 0;
    for (int v0 = g * 32 + lane; v0 - lane < nv;) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int t = 0; t < NTOK; ++t) acc[t] = dot16(w[j], xv[t * nv + v0 + j * 32 * G], acc[t]);
      v0 += kAhead * 32 * G;
      if (v0 - lane < nv) load(r, v0);
    }
    // the next row's first pieces, ahead of this row's reduction
    load(r + step, g * 32 + lane);
#pragma unroll
    for (int t = 0; t < NTOK; ++t) acc[t] = __reduce_add_sync(0xffffffffu, acc[t]);
    if (G > 1) {
      if (lane == 0) {
#pragma unroll
        for (int t = 0; t < NTOK; ++t) part[parity][warp][t] = acc[t];
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NTOK; ++t) {
        acc[t] = 0;
        for (int h = 0; h < G; ++h) acc[t] += part[parity][mine * G + h][t];
      }
      parity ^= 1;
    }
    if (g == 0 && lane == 0 && r < a.d_out) {
      const float wi = a.ws[r];
#pragma unroll
      for (int t = 0; t < NTOK; ++t)
        put(y + (int64_t)t * a.d_out + r, __fmul_rn((float)acc[t], __fmul_rn(a.xs[t], wi)));
    }
  }
}

template <int NTOK, typename T>
cudaError_t run_gemv(Int8GemvArgs a, cudaStream_t stream) {
  auto fn = &k_int8_gemv<NTOK, T>;
  const void* p = reinterpret_cast<const void*>(fn);
  a.per_row = 1;
  while (a.per_row < kGemvWarps && (int64_t)a.d_out * a.per_row < 24 * sm_count() &&
         a.per_row * 2 * 512 <= a.d_in)
    a.per_row *= 2;
  // the last token's reads end with its last whole step of kAhead pieces per warp
  const size_t step = (size_t)kAhead * 512 * a.per_row;
  const size_t smem = (size_t)(NTOK - 1) * a.d_in + (a.d_in + step - 1) / step * step;
  cudaError_t err = allow_smem(p, smem + kGemvStatic);
  if (err != cudaSuccess) return err;
  const int rows_cta = kGemvWarps / a.per_row;
  const int grid = persistent_grid(p, kGemvWarps * 32, smem, ((int64_t)a.d_out + rows_cta - 1) / rows_cta);
  return launch_pdl(fn, dim3(grid), dim3(kGemvWarps * 32), smem, stream, a);
}

// ------------------------------------------------------------ up to eight tokens

// mma m16n8k32 of 8-bit integers: D += A B, A 16 rows of W, B eight tokens.
__device__ __forceinline__ void mma_m16n8k32(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp takes 16 rows of W and its share of their 256-byte pieces.  Lane l
// loads 16 bytes of rows l / 4 and l / 4 + 8 at column 64 k + 16 (l % 4): four
// words each, which two MMAs take as their A fragments; the same 16 columns of
// token l / 4 are the B fragments (the order of the columns within a product
// does not matter as long as both sides share it).  So W goes straight from
// global memory into fragments, and the tokens (rows past the last one zero) come
// out of shared memory, 16 bytes a lane; the warps' sums meet in shared memory.
// The legacy MMA is far from its bound here: one per 512 bytes of W.  Eight
// pieces in flight with two CTAs per SM, or 64 registers and four CTAs, were
// slower (4 tokens 4096 -> 11008: 13.7, 13.0 us against 10.4).
constexpr int kPieces = 4;  // 64-byte pieces of 16 rows in flight per warp: 4 KB
struct Int8MmaArgs {
  Int8GemvArgs g;
  int pitch;  // bytes between tokens in shared memory: 64 mod 128, so that the lanes
              // of two tokens never meet in a bank
};

template <typename T>
__global__ void __launch_bounds__(kGemvWarps * 32, 3) k_int8_gemv_mma(const Int8MmaArgs b) {
  const Int8GemvArgs& a = b.g;
  extern __shared__ __align__(16) unsigned char xb[];  // [8][pitch], and 256 G bytes
  __shared__ int part[2][kGemvWarps][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.per_row, g = warp % G, mine = warp / G;
  const int gid = lane >> 2, tig = lane & 3;
  const int groups_cta = kGemvWarps / G;
  const int64_t groups = ((int64_t)a.d_out + 15) / 16, step = (int64_t)gridDim.x * groups_cta;
  T* y = reinterpret_cast<T*>(a.y);
  const auto address = [&](int64_t grp, int h, int k) {  // row gid + 8 h of the group, column k
    return a.w + (grp * 16 + gid + 8 * h) * a.d_in + k + 16 * tig;
  };
  int64_t grp = (int64_t)blockIdx.x * groups_cta + mine;
  // while the kernel ahead finishes: the first pieces on their way into L2
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < kPieces; j += 2)
      if (tig == 0 && grp * 16 + gid + 8 * h < a.d_out && (g * kPieces + j) * 64 < a.d_in)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(address(grp, h, (g * kPieces + j) * 64)));
  pdl_wait();
  pdl_trigger();
  uint4 w[kPieces][2];
  const auto load = [&](int64_t grp, int k0) {  // zeros past the ends
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[j][h] = k0 + 64 * j < a.d_in && grp * 16 + gid + 8 * h < a.d_out
                      ? __ldcs(reinterpret_cast<const uint4*>(address(grp, h, k0 + 64 * j)))
                      : make_uint4(0u, 0u, 0u, 0u);
  };
  load(grp, g * kPieces * 64);
  const int nv = a.d_in / 16;
  for (int v = threadIdx.x; v < 8 * nv; v += kGemvWarps * 32) {
    const int t = v / nv, c = v - t * nv;
    *reinterpret_cast<uint4*>(xb + t * b.pitch + 16 * c) =
        t < a.ntok ? reinterpret_cast<const uint4*>(a.x)[v] : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  int parity = 0;
  for (int64_t g0 = (int64_t)blockIdx.x * groups_cta; g0 < groups; g0 += step, grp += step) {
    int acc[4] = {};
    for (int k0 = g * kPieces * 64; k0 < a.d_in;) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(xb + gid * b.pitch + k0 + 64 * j + 16 * tig);
        mma_m16n8k32(acc, w[j][0].x, w[j][1].x, w[j][0].y, w[j][1].y, x.x, x.y);
        mma_m16n8k32(acc, w[j][0].z, w[j][1].z, w[j][0].w, w[j][1].w, x.z, x.w);
      }
      k0 += G * kPieces * 64;
      if (k0 < a.d_in) load(grp, k0);
    }
    // the next rows' first pieces, ahead of these rows' sums
    load(grp + step, g * kPieces * 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) part[parity][warp][e][lane] = acc[e];
    __syncthreads();
    // value (e, l) of a group: row l / 4 + 8 (e / 2), token 2 (l % 4) + e % 2
    for (int i = threadIdx.x; i < groups_cta * 128; i += kGemvWarps * 32) {
      const int l = i & 31, e = (i >> 5) & 3, q = i >> 7;
      const int64_t row = (g0 + q) * 16 + (l >> 2) + 8 * (e >> 1);
      const int t = 2 * (l & 3) + (e & 1);
      if (row < a.d_out && t < a.ntok) {
        int sum = 0;
        for (int h = 0; h < G; ++h) sum += part[parity][q * G + h][e][l];
        put(y + (int64_t)t * a.d_out + row, __fmul_rn((float)sum, __fmul_rn(a.xs[t], a.ws[row])));
      }
    }
    parity ^= 1;
  }
}

template <typename T>
cudaError_t run_gemv_mma(const Int8GemvArgs& a, cudaStream_t stream) {
  auto fn = &k_int8_gemv_mma<T>;
  const void* p = reinterpret_cast<const void*>(fn);
  Int8MmaArgs b = {a, a.d_in + (a.d_in % 128 == 0 ? 64 : 0)};
  b.g.per_row = 1;
  while (b.g.per_row < kGemvWarps && b.g.per_row * 2 * kPieces * 64 <= a.d_in) b.g.per_row *= 2;
  const size_t smem = (size_t)8 * b.pitch + 64 * kPieces * b.g.per_row;
  cudaError_t err = allow_smem(p, smem + kGemvStatic);
  if (err != cudaSuccess) return err;
  const int groups_cta = kGemvWarps / b.g.per_row;
  const int64_t groups = ((int64_t)a.d_out + 15) / 16;
  const int grid = persistent_grid(p, kGemvWarps * 32, smem, (groups + groups_cta - 1) / groups_cta);
  return launch_pdl(fn, dim3(grid), dim3(kGemvWarps * 32), smem, stream, b);
}

template <typename T>
cudaError_t run_any(const Int8GemvArgs& a, bool mma, cudaStream_t stream) {
  if (mma) return run_gemv_mma<T>(a, stream);
  return a.ntok == 1 ? run_gemv<1, T>(a, stream) : run_gemv<2, T>(a, stream);
}

}  // namespace

cudaError_t launch_int8_gemv(const int8_t* d_x, const float* d_x_scale, int ntok, const int8_t* d_w,
                             const float* d_w_scale, int d_out, int d_in, void* d_y, int dtype,
                             bool mma, cudaStream_t stream) {
  const Int8GemvArgs a = {d_x, d_x_scale, d_w, d_w_scale, d_y, ntok, d_out, d_in, 1};
  return dtype == QAMW_DTYPE_F32 ? run_any<float>(a, mma, stream) : run_any<__nv_bfloat16>(a, mma, stream);
}

}  // namespace qamw
