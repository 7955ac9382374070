// int8_rows.cu -- rows to 8-bit integers with one fp32 scale per row: the
// encoders of W8A8 weights and tokens, and the RMS norm (with the residual's
// addition) whose output is in 8 bits.
//
// Row x of d columns, per-column factor c_j (s_j for weights, 1 / s_j for
// tokens, g_j / s_j for the norm; s absent = 1), T = the type of x:
//   h_j   = T(x_j + res_j)             (norm with residual, written back)
//   v_j   = h_j c_j
//   a     = max_j |v_j|
//   q_j   = rint(v_j (127 / a))        (ties to even; 0 for a < 2^-100)
//   scale = a / 127, times 1 / sqrt(mean h^2 + eps) for the norm.
// The norm's 1 / rms is common to the row, so it cancels out of q: one pass and
// one reduction give the maximum and the sum of squares together, and q depends
// on no order of summation (the maximum is exact, every other step that decides
// q is a single fp32 rounding).  |v_j (127 / a)| <= 127 (1 + 2^-22), so q stays
// in [-127, 127].
//
// Every element is read once and kept in registers between the reduction and
// the rounding.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "launch.cuh"

namespace qamw {
namespace {

constexpr float kInt8Max = 127.f;
constexpr float kRowTiny = 7.888609052210118e-31f;  // 2^-100: 127 / a stays finite above it
constexpr uint32_t kInfBits = 0x7f800000u;

struct Int8RowsArgs {
  const void* x;
  const void* res;   // norm with residual
  const void* gain;  // norm
  const __half* s;   // nullable
  void* sum;         // norm with residual: h
  int8_t* q;
  float* scale;
  int32_t* status;
  int64_t rows;
  int d;
  float eps;
  int divide;  // tokens and norm: c = (g or 1) / s, weights: c = s
};

// Eight consecutive values, as loaded: bf16 in 16 bytes, fp32 in 32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p, int64_t vec) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + vec);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  }
  __device__ __forceinline__ void load_kept(const void* p, int64_t vec) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + vec);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void add(const Raw8& o) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__fadd_rn(get(2 * e), o.get(2 * e)),
                         __fadd_rn(get(2 * e + 1), o.get(2 * e + 1)));
  }
  __device__ __forceinline__ void store(void* p, int64_t vec) const {
    reinterpret_cast<uint4*>(p)[vec] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ __forceinline__ void set(float4 a, float4 b) {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void load(const void* p, int64_t vec) {
    const float4* s = reinterpret_cast<const float4*>(p) + 2 * vec;
    set(__ldcs(s), __ldcs(s + 1));
  }
  __device__ __forceinline__ void load_kept(const void* p, int64_t vec) {
    const float4* s = reinterpret_cast<const float4*>(p) + 2 * vec;
    set(__ldg(s), __ldg(s + 1));
  }
  __device__ __forceinline__ float get(int i) const { return f[i]; }
  __device__ __forceinline__ void add(const Raw8& o) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __fadd_rn(f[e], o.f[e]);
  }
  __device__ __forceinline__ void store(void* p, int64_t vec) const {
    float4* s = reinterpret_cast<float4*>(p) + 2 * vec;
    s[0] = make_float4(f[0], f[1], f[2], f[3]);
    s[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
  }
};

// The column factors of eight columns.
template <typename T, bool NORM>
__device__ __forceinline__ void factors(const Int8RowsArgs& a, int vec, float (&c)[8]) {
  if constexpr (NORM) {
    Raw8<T> g;
    g.load_kept(a.gain, vec);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = g.get(e);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f;
  }
  if (a.s != nullptr) {
    float s[8];
    load_halves<8>(a.s + 8 * vec, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = a.divide ? __fdiv_rn(c[e], s[e]) : s[e];
  }
}

// Sum and maximum over the threads of a row (a warp, or the whole CTA).
struct RowRed {
  float sum;
  uint32_t top;
};
template <bool NORM>
__device__ __forceinline__ RowRed reduce_row(RowRed r, bool by_warp, RowRed* slots) {
  if constexpr (NORM) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
  }
  r.top = __reduce_max_sync(0xffffffffu, r.top);
  if (by_warp) return r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  if (lane == 0) slots[warp] = r;
  __syncthreads();
  RowRed o;
  o.sum = 0.f;
  o.top = 0u;
  if (lane < nwarps) o = slots[lane];
  if constexpr (NORM) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) o.sum += __shfl_xor_sync(0xffffffffu, o.sum, k);
  }
  o.top = __reduce_max_sync(0xffffffffu, o.top);
  return o;
}

// Rows of c in shared memory: eight columns as two float4, 16 bytes apart by
// half the row, so that a warp's 16-byte loads are consecutive.
__device__ __forceinline__ void put_factors(float4* tab, int nvec, int v, const float (&c)[8]) {
  tab[v] = make_float4(c[0], c[1], c[2], c[3]);
  tab[nvec + v] = make_float4(c[4], c[5], c[6], c[7]);
}
__device__ __forceinline__ void get_factors(const float4* tab, int nvec, int v, float (&c)[8]) {
  const float4 a = tab[v], b = tab[nvec + v];
  c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
  c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
}

// Four rounded values as the bytes of a word.  x + 1.5 2^23 rounds x to a whole
// number (ties to even) whose low byte is the low byte of the sum's pattern: an
// addition in place of a conversion, which has a quarter of its rate.
__device__ __forceinline__ uint32_t pack_rounded(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.f;
  const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, kMagic)),
                                  __float_as_uint(__fadd_rn(b, kMagic)), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, kMagic)),
                                  __float_as_uint(__fadd_rn(d, kMagic)), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// How a row is shared out (MODE) and where its thread keeps c_j:
//   kWarpRow  a warp per row, eight rows a CTA (d <= 1024); c in registers;
//   kWideRow  a CTA per row, one vector of eight columns a thread; c in
//             registers: the shortest chain for a few rows;
//   kDeepRow  a CTA per row, VEC vectors a thread; c in shared memory, so that
//             the registers allow about a thousand threads per SM, each with
//             VEC loads per input in flight.
enum { kWarpRow, kWideRow, kDeepRow };

template <typename T, int MODE, int VEC, bool NORM, bool RES>
__global__ void __launch_bounds__(MODE == kWarpRow ? 256 : 1024, 1)
    k_int8_rows(const Int8RowsArgs a) {
  __shared__ RowRed slots[2][32];
  extern __shared__ __align__(16) float4 c_tab[];
  constexpr bool kByWarp = MODE == kWarpRow;
  const int n = kByWarp ? 32 : blockDim.x;
  const int t = kByWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int nvec = a.d / 8;
  const int64_t groups = kByWarp ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  const int64_t first =
      kByWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  float c[MODE == kDeepRow ? 1 : VEC][8];
  if constexpr (MODE == kDeepRow) {
    for (int v = t; v < nvec; v += n) {  // each thread reads back what it wrote
      factors<T, NORM>(a, v, c[0]);
      put_factors(c_tab, nvec, v, c[0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) factors<T, NORM>(a, t + i * n, c[i]);
  }
  int flags = 0, parity = 0;
  for (int64_t row = first; row < a.rows; row += groups) {
    const int64_t base = row * nvec;
    Raw8<T> h[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int v = t + i * n;
      h[i].zero();
      if (v < nvec) h[i].load(a.x, base + v);
    }
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = t + i * n;
        if (v < nvec) {
          Raw8<T> r;
          r.load(a.res, base + v);
          h[i].add(r);
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = t + i * n;
        if (v < nvec) h[i].store(a.sum, base + v);
      }
    }
    RowRed r;
    r.sum = 0.f;
    r.top = 0u;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) {
        if constexpr (MODE == kDeepRow) get_factors(c_tab, nvec, t + i * n, c[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = h[i].get(e);
          if constexpr (NORM) r.sum = fmaf(f, f, r.sum);
          r.top = max(r.top, __float_as_uint(fabsf(__fmul_rn(f, c[MODE == kDeepRow ? 0 : i][e]))));
        }
      }
    r = reduce_row<NORM>(r, kByWarp, slots[parity]);
    parity ^= 1;
    const float top = __uint_as_float(r.top);
    const bool finite = r.top < kInfBits, some = finite && top >= kRowTiny;
    const float inv = some ? __fdiv_rn(kInt8Max, top) : 0.f;
    float scale = some ? __fdiv_rn(top, kInt8Max) : 0.f;
    if constexpr (NORM) {
      if (some && r.sum > FLT_MAX) {
        // the squares overflow (|h| beyond about 2^56): again with h 2^-70, whose
        // squares fit; what underflows there is far below the row's largest
        RowRed w;
        w.sum = 0.f;
        w.top = 0u;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float f = h[i].get(e) * 8.470329472543003e-22f;
            w.sum = fmaf(f, f, w.sum);
          }
        w = reduce_row<NORM>(w, kByWarp, slots[parity]);
        parity ^= 1;
        scale = scale * 8.470329472543003e-22f * (1.f / sqrtf(w.sum / (float)a.d));
      } else {
        scale *= 1.f / sqrtf(r.sum / (float)a.d + a.eps);
      }
    }
    if (t == 0) {
      a.scale[row] = finite ? scale : __uint_as_float(0x7fc00000u);
      if (!finite) flags |= QAMW_STATUS_NONFINITE;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int v = t + i * n;
      if (v < nvec) {
        if constexpr (MODE == kDeepRow) get_factors(c_tab, nvec, v, c[0]);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          f[e] = __fmul_rn(__fmul_rn(h[i].get(e), c[MODE == kDeepRow ? 0 : i][e]), inv);
        uint2 w = make_uint2(pack_rounded(f[0], f[1], f[2], f[3]), pack_rounded(f[4], f[5], f[6], f[7]));
        if (!some) w = make_uint2(0u, 0u);
        reinterpret_cast<uint2*>(a.q)[base + v] = w;
      }
    }
  }
  raise_flag(a.status, flags);
}

template <typename T, int MODE, int VEC, bool NORM, bool RES>
cudaError_t run_rows(const Int8RowsArgs& a, int threads, cudaStream_t stream) {
  auto fn = &k_int8_rows<T, MODE, VEC, NORM, RES>;
  const size_t smem = MODE == kDeepRow ? (size_t)a.d * sizeof(float) : 0;
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(fn), smem);
  if (err != cudaSuccess) return err;
  const int64_t per = MODE == kWarpRow ? threads / 32 : 1;
  const int grid =
      persistent_grid(reinterpret_cast<const void*>(fn), threads, smem, (a.rows + per - 1) / per);
  return launch_pdl(fn, dim3(grid), dim3(threads), smem, stream, a);
}

template <typename T, bool NORM, bool RES>
cudaError_t run_rows_any(const Int8RowsArgs& a, cudaStream_t stream) {
  const int nvec = a.d / 8;
  if (a.d <= 1024) {
    const int threads = (int)std::min<int64_t>(8, a.rows) * 32;
    switch ((nvec + 31) / 32) {
      case 1: return run_rows<T, kWarpRow, 1, NORM, RES>(a, threads, stream);
      case 2: return run_rows<T, kWarpRow, 2, NORM, RES>(a, threads, stream);
      default: return run_rows<T, kWarpRow, 4, NORM, RES>(a, threads, stream);
    }
  }
  if (a.rows <= 2 * sm_count() && nvec <= 1024)
    return run_rows<T, kWideRow, 1, NORM, RES>(a, (nvec + 31) / 32 * 32, stream);
  return run_rows<T, kDeepRow, 4, NORM, RES>(a, ((nvec + 3) / 4 + 31) / 32 * 32, stream);
}

}  // namespace

cudaError_t launch_int8_encode(const void* d_x, int dtype, int64_t rows, int d,
                               const uint16_t* d_chan_scale, bool divide, int8_t* d_q,
                               float* d_scale, int32_t* d_status, cudaStream_t stream) {
  Int8RowsArgs a = {};
  a.x = d_x;
  a.s = reinterpret_cast<const __half*>(d_chan_scale);
  a.q = d_q;
  a.scale = d_scale;
  a.status = d_status;
  a.rows = rows;
  a.d = d;
  a.divide = divide ? 1 : 0;
  return dtype == QAMW_DTYPE_F32 ? run_rows_any<float, false, false>(a, stream)
                                 : run_rows_any<__nv_bfloat16, false, false>(a, stream);
}

cudaError_t launch_rmsnorm_int8(const void* d_x, const void* d_residual, int dtype,
                                const void* d_gain, float eps, int64_t rows, int d,
                                const uint16_t* d_chan_scale, void* d_sum, int8_t* d_q,
                                float* d_scale, int32_t* d_status, cudaStream_t stream) {
  Int8RowsArgs a = {};
  a.x = d_x;
  a.res = d_residual;
  a.gain = d_gain;
  a.s = reinterpret_cast<const __half*>(d_chan_scale);
  a.sum = d_sum;
  a.q = d_q;
  a.scale = d_scale;
  a.status = d_status;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.divide = 1;
  if (dtype == QAMW_DTYPE_F32)
    return d_residual ? run_rows_any<float, true, true>(a, stream)
                      : run_rows_any<float, true, false>(a, stream);
  return d_residual ? run_rows_any<__nv_bfloat16, true, true>(a, stream)
                    : run_rows_any<__nv_bfloat16, true, false>(a, stream);
}

}  // namespace qamw
