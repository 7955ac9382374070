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
// Every element is read once and kept on chip between the reduction and the
// rounding, so large batches are bound by HBM (measured, B200: norm with residual
// 8192 x 5120 bf16 46.3 us, 6.35 TB/s, 99% of a copy's rate; fp32 96 us, 5.7 TB/s;
// fp32 weights 4096 x 11008 35.5 us, 6.34 TB/s; bf16 tokens 4001 x 13824 26.7 us,
// 6.20 TB/s), narrow bf16 rows without a residual by instructions (norm 8192 x 5120
// 26.9 us, 4.7 TB/s, weights 4096 x 4096 9.8 us, 5.1 TB/s: about 190 per warp and row
// of 16 elements a lane), and a few rows by the chain of launch, load, reduction and
// store (1 x 4096 2.5 us).  Rows too long for the ring below (kDeepRow) have no
// loads in flight between the reduction and the next row: 2000 x 28672 tokens bf16
// 43 us, 4.0 TB/s, fp32 59 us, 4.9 TB/s, norm with residual bf16 91 us, 4.4 TB/s.
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
  unsigned tries;  // polls of a worker's wait for a row (k_int8_ring)
  float eps;
  float one;   // 1 (see pack_rounded)
  int divide;  // tokens and norm: c = (g or 1) / s, weights: c = s
  int stages;  // rows of the ring (k_int8_ring)
};
// A launch with more than 96 bytes of arguments took 0.35 us longer to issue (3.3, not 2.9).
static_assert(sizeof(Int8RowsArgs) <= 96, "arguments of a launch");

// Bound on the row kernels' static shared memory.
constexpr size_t kStaticRoom = 1024;

// Eight consecutive values, as loaded: bf16 in 16 bytes, fp32 in 32.  LoadOnce
// is for global data that the call reads once.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void set(uint4 u) { w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w; }
  __device__ __forceinline__ void load_once(const void* p, int64_t vec) {
    set(__ldcs(reinterpret_cast<const uint4*>(p) + vec));
  }
  __device__ __forceinline__ void load(const void* p, int64_t vec) {
    set(reinterpret_cast<const uint4*>(p)[vec]);
  }
  __device__ __forceinline__ float2 get(int i) const {  // values 2 i, 2 i + 1
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void add(const Raw8& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = add2(get(i), o.get(i));
      w[i] = pack_bf16x2(f.x, f.y);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t vec) const {
    reinterpret_cast<uint4*>(p)[vec] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw8<float> {
  float2 f[4];
  __device__ __forceinline__ void set(float4 a, float4 b) {
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void load_once(const void* p, int64_t vec) {
    const float4* s = reinterpret_cast<const float4*>(p) + 2 * vec;
    set(__ldcs(s), __ldcs(s + 1));
  }
  __device__ __forceinline__ void load(const void* p, int64_t vec) {
    const float4* s = reinterpret_cast<const float4*>(p) + 2 * vec;
    set(s[0], s[1]);
  }
  __device__ __forceinline__ float2 get(int i) const { return f[i]; }
  __device__ __forceinline__ void add(const Raw8& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = add2(f[i], o.f[i]);
  }
  __device__ __forceinline__ void store(void* p, int64_t vec) const {
    float4* s = reinterpret_cast<float4*>(p) + 2 * vec;
    s[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    s[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};

// The factors c_j of eight columns.
template <typename T, bool NORM>
__device__ __forceinline__ void factors(const Int8RowsArgs& a, int vec, float2 (&c)[4]) {
  if constexpr (NORM) {
    Raw8<T> g;
    g.load(a.gain, vec);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = g.get(i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = make_float2(1.f, 1.f);
  }
  if (a.s != nullptr) {
    // from L2: an ordinary load here (as good by the rule in common.cuh) was scheduled
    // worse, 27.5 us at tokens 4001 x 13824 bf16 against 26.7
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(a.s) + vec);
    const __half2* h = reinterpret_cast<const __half2*>(&u);
    float s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      s[2 * i] = f.x;
      s[2 * i + 1] = f.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = a.divide ? make_float2(__fdiv_rn(c[i].x, s[2 * i]), __fdiv_rn(c[i].y, s[2 * i + 1]))
                      : make_float2(s[2 * i], s[2 * i + 1]);
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The gain and the channel scales of eight columns on their way into L2.
template <typename T, bool NORM>
__device__ __forceinline__ void prefetch_factors(const Int8RowsArgs& a, int vec) {
  if constexpr (NORM) prefetch_l2(static_cast<const char*>(a.gain) + (size_t)vec * 8 * sizeof(T));
  if (a.s != nullptr) prefetch_l2(a.s + 8 * vec);
}

// max(|a|, |b|, |c|), NaN if one of them is: one instruction for two elements.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A thread's part of a row's statistics: sum of squares (two partial sums) and
// the largest |v|, NaN when one of the thread's values is.
struct RowStat {
  float2 sum;
  float top;
};

// v = h c of eight columns into the statistics.
template <bool NORM, typename T>
__device__ __forceinline__ void take(RowStat& r, const Raw8<T>& h, const float2 (&c)[4],
                                     float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = h.get(i);
    if constexpr (NORM) r.sum = fma2(f, f, r.sum);
    v[i] = mul2(f, c[i]);
    r.top = max3_abs(r.top, v[i].x, v[i].y);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Scratch of a row's reduction over a CTA (two of them, used in turn: the next
// row's writes then need no barrier of their own).
struct RowSlots {
  uint32_t top[32];
  float sum[32];
};

// The row's largest |v| (bits; NaN and Inf are the largest of all) to every
// thread, its sum of squares to the first warp of the row alone: only the scale
// depends on it.
template <bool NORM>
__device__ __forceinline__ uint32_t reduce_row(RowStat r, bool by_warp, RowSlots& slots, float& sum) {
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(r.top));
  if constexpr (NORM) sum = warp_sum(r.sum.x + r.sum.y);
  if (by_warp) return top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  if (lane == 0) {
    slots.top[warp] = top;
    if constexpr (NORM) slots.sum[warp] = sum;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, lane < nwarps ? slots.top[lane] : 0u);
  if constexpr (NORM)
    if (warp == 0) sum = warp_sum(lane < nwarps ? slots.sum[lane] : 0.f);
  return top;
}

// What the rounding of a row needs: 127 / a, or that the row gives q = 0 (below
// 2^-100, or not finite).
struct RowOut {
  float inv;
  bool some;
};
__device__ __forceinline__ RowOut row_out(uint32_t top) {
  RowOut o;
  o.some = top < kInfBits && __uint_as_float(top) >= kRowTiny;
  o.inv = o.some ? __fdiv_rn(kInt8Max, __uint_as_float(top)) : 0.f;
  return o;
}

// The row's scale, by its first warp.  Squares that overflow (|h| beyond about
// 2^56) are summed again with h 2^-80 from memory, by the warp alone: h is x, or
// the sum that the row's threads have written ahead of the reduction's barrier.
// 2^15 squares of 2^(128 - 80) stay below 2^111, and a sum that overflowed is
// above 2^-32 then; scale and factor are joined in 64 bits, since scale 2^-80 and
// 1 / rms alone may both leave the normal range.
constexpr float kDown = 8.271806125530277e-25f;  // 2^-80
template <typename T, bool NORM>
__device__ __forceinline__ void put_scale(const Int8RowsArgs& a, int64_t row, uint32_t top, bool some,
                                          float sum, int lane, int& flags) {
  float scale = some ? __fdiv_rn(__uint_as_float(top), kInt8Max) : 0.f;
  if constexpr (NORM) {
    if (some && !(sum <= FLT_MAX)) {
      const int nvec = a.d / 8;
      const void* h = a.sum != nullptr ? a.sum : a.x;
      float2 w = make_float2(0.f, 0.f);
      for (int v = lane; v < nvec; v += 32) {
        Raw8<T> r;
        r.load(h, row * nvec + v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = mul2(r.get(i), make_float2(kDown, kDown));
          w = fma2(f, f, w);
        }
      }
      scale = (float)((double)scale * kDown / sqrt((double)warp_sum(w.x + w.y) / a.d));
    } else {
      scale *= 1.f / sqrtf(sum / (float)a.d + a.eps);
    }
  }
  const bool finite = top < kInfBits;
  if (lane == 0) {
    a.scale[row] = finite ? scale : __uint_as_float(0x7fc00000u);
    if (!finite) flags |= QAMW_STATUS_NONFINITE;
  }
}

// Four products v inv rounded to the bytes of a word.  x + 1.5 2^23 rounds x to a
// whole number (ties to even) whose low byte is the low byte of the sum's
// pattern: an addition in place of a conversion, which has a quarter of its
// rate.  The product has to be rounded first; a packed addition behind it gets
// fused with it, so the addition is fma(x, one, 1.5 2^23) with a `one` that the
// compiler does not know.
__device__ __forceinline__ uint32_t pack_rounded(float2 a, float2 b, float2 inv, float2 one) {
  const float2 magic = make_float2(12582912.f, 12582912.f);
  a = fma2(mul2(a, inv), one, magic);
  b = fma2(mul2(b, inv), one, magic);
  const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// Eight values v_j into the row's q at vector `at`.
__device__ __forceinline__ void put_q(const Int8RowsArgs& a, int64_t at, const float2 (&v)[4],
                                      const RowOut& o) {
  const float2 inv = make_float2(o.inv, o.inv), one = make_float2(a.one, a.one);
  reinterpret_cast<uint2*>(a.q)[at] =
      make_uint2(pack_rounded(v[0], v[1], inv, one), pack_rounded(v[2], v[3], inv, one));
}

// How a row is shared out (MODE) and where its thread keeps c_j:
//   kWarpRow  a warp per row, eight rows a CTA (d <= 512); c in registers;
//   kWideRow  a CTA per row, one vector of eight columns a thread; c in
//             registers: the shortest chain for a few rows;
//   kDeepRow  a CTA per row, four vectors a thread; c in shared memory (as two
//             arrays of float4, so that a warp's loads are consecutive): rows
//             too long for the ring below.
enum { kWarpRow, kWideRow, kDeepRow };

template <typename T, int MODE, int VEC, bool NORM, bool RES>
__global__ void __launch_bounds__(MODE == kWarpRow ? 256 : 1024, 1)
    k_int8_rows(const Int8RowsArgs a) {
  __shared__ RowSlots slots[2];
  extern __shared__ __align__(16) float4 c_tab[];
  constexpr bool kByWarp = MODE == kWarpRow, kTable = MODE == kDeepRow;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = kByWarp ? 32 : blockDim.x;
  const int t = kByWarp ? lane : threadIdx.x;
  const int nvec = a.d / 8;
  const int64_t groups = kByWarp ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  const int64_t first = kByWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  float2 c[kTable ? 1 : VEC][4];
  if constexpr (kTable) {
    for (int v = t; v < nvec; v += n) {  // each thread reads back what it wrote
      factors<T, NORM>(a, v, c[0]);
      c_tab[v] = make_float4(c[0][0].x, c[0][0].y, c[0][1].x, c[0][1].y);
      c_tab[nvec + v] = make_float4(c[0][2].x, c[0][2].y, c[0][3].x, c[0][3].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) factors<T, NORM>(a, t + i * n, c[i]);
  }
  const auto from_table = [&](int v) {
    const float4 p = c_tab[v], q = c_tab[nvec + v];
    c[0][0] = make_float2(p.x, p.y), c[0][1] = make_float2(p.z, p.w);
    c[0][2] = make_float2(q.x, q.y), c[0][3] = make_float2(q.z, q.w);
  };
  int flags = 0, parity = 0;
  for (int64_t row = first; row < a.rows; row += groups) {
    const int64_t base = row * nvec;
    Raw8<T> h[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) h[i].load_once(a.x, base + t + i * n);
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = t + i * n;
        if (v < nvec) {
          Raw8<T> r;
          r.load_once(a.res, base + v);
          h[i].add(r);
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (t + i * n < nvec) h[i].store(a.sum, base + t + i * n);
    }
    RowStat r;
    r.sum = make_float2(0.f, 0.f);
    r.top = 0.f;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) {
        if constexpr (kTable) from_table(t + i * n);
        take<NORM>(r, h[i], c[kTable ? 0 : i], v);
      }
    float sum = 0.f;
    const uint32_t top = reduce_row<NORM>(r, kByWarp, slots[parity], sum);
    parity ^= 1;
    const RowOut o = row_out(top);
    if (kByWarp || warp == 0) {
      __syncwarp();  // by_warp: the lanes' sums are written before one of them reads
      put_scale<T, NORM>(a, row, top, o.some, sum, lane, flags);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t + i * n < nvec) {
        if constexpr (kTable) from_table(t + i * n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(h[i].get(e), c[kTable ? 0 : i][e]);
        if (o.some)
          put_q(a, base + t + i * n, v, o);
        else
          reinterpret_cast<uint2*>(a.q)[base + t + i * n] = make_uint2(0u, 0u);
      }
  }
  raise_flag(a.status, flags);
}

template <typename T, int MODE, int VEC, bool NORM, bool RES>
cudaError_t run_rows(const Int8RowsArgs& a, int threads, cudaStream_t stream) {
  auto fn = &k_int8_rows<T, MODE, VEC, NORM, RES>;
  const size_t smem = MODE == kDeepRow ? (size_t)a.d * sizeof(float) : 0;
  // the opt-in is for static and dynamic together above 48 KB: asked for with room
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(fn), smem + kStaticRoom);
  if (err != cudaSuccess) return err;
  const int64_t per = MODE == kWarpRow ? threads / 32 : 1;
  const int grid =
      persistent_grid(reinterpret_cast<const void*>(fn), threads, smem, (a.rows + per - 1) / per);
  return launch_pdl(fn, dim3(grid), dim3(threads), smem, stream, a);
}

// Many rows: a CTA per row again, its inputs brought into a ring of `stages`
// rows in shared memory by bulk copies, so that about 100 KB per SM are in
// flight whatever the rows' threads are waiting for.  Two vectors a thread; c
// and, between the reduction and the rounding, v in registers.  The reduction's
// barrier also says that every thread has read the row, so the stage is refilled
// right behind it.  The last warp has no vectors: it issues the copies and forms
// the scales (a chain of divisions and a root, some 300 cycles) while the others
// go on to the next row.
//
// A worker whose wait for a row gives up reads nothing of it, sets the row's flag and
// puts kGaveUp, above every value's bits, in the place of its largest |v|.  Behind the
// row's barrier the helper sees the flag before it refills a stage, and the reduction
// tells the workers: all leave the loop together, before a code or scale of the row is
// written, and the helper lets its copies in flight land.
constexpr int kRingVec = 2;
constexpr int kRingMax = 8;
constexpr uint32_t kGaveUp = 0xffffffffu;
// Threads of a CTA at most; fewer with fp32 and a residual (d <= 13312 then),
// which needs more than 64 registers.
template <typename T, bool RES>
constexpr int ring_threads() {
  return RES && sizeof(T) == 4 ? 864 : 1024;
}

template <typename T, bool NORM, bool RES>
__global__ void __launch_bounds__(ring_threads<T, RES>(), 1)
    k_int8_ring(const Int8RowsArgs a) {
  __shared__ RowSlots slots[2];
  __shared__ uint64_t full[kRingMax];
  __shared__ volatile int gave_up[2];  // by row parity, as the slots
  extern __shared__ __align__(128) unsigned char ring[];
  const int n = blockDim.x - 32, t = threadIdx.x, nvec = a.d / 8;
  const int lane = t & 31, warp = t >> 5, nwarps = n >> 5, stages = a.stages;
  const uint32_t row_bytes = (uint32_t)a.d * sizeof(T), stage = row_bytes * (RES ? 2 : 1);
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    gave_up[0] = gave_up[1] = 0;
  }
  __syncthreads();
  // While the kernel ahead finishes, this CTA's first rows and its factors on their
  // way into L2, whatever they hold by then; what counts is read after the wait.
  // (8192 x 5120 bf16 with residual, back to back: 48.1 us without, 46.3 with.)
  if (warp == nwarps) {
    for (int j = lane; j < stages; j += 32) {
      const int64_t row = blockIdx.x + (int64_t)j * gridDim.x;
      if (row < a.rows) {
        bulk_prefetch_l2(static_cast<const unsigned char*>(a.x) + row * row_bytes, row_bytes);
        if constexpr (RES)
          bulk_prefetch_l2(static_cast<const unsigned char*>(a.res) + row * row_bytes, row_bytes);
      }
    }
  } else {
    for (int v = t; v < nvec; v += n) prefetch_factors<T, NORM>(a, v);
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  int flags = 0, parity = 0, s = 0;
  if (warp == nwarps) {
    const auto fetch = [&](int64_t row, int s) {
      if (row >= a.rows) return;
      unsigned char* dst = ring + (size_t)s * stage;
      mbar_expect_tx(&full[s], stage);
      bulk_g2s(dst, static_cast<const unsigned char*>(a.x) + row * row_bytes, row_bytes, &full[s]);
      if constexpr (RES)
        bulk_g2s(dst + row_bytes, static_cast<const unsigned char*>(a.res) + row * row_bytes,
                 row_bytes, &full[s]);
    };
    if (lane == 0) {
      fence_proxy_async_global();  // x and the residual may come from the kernel ahead
      for (int j = 0; j < stages; ++j) fetch(blockIdx.x + (int64_t)j * gridDim.x, j);
    }
    for (int64_t row = blockIdx.x, j = 0; row < a.rows; row += gridDim.x, ++j) {
      __syncthreads();
      if (gave_up[parity]) {  // this CTA's rows j .. j + stages - 1 are in flight
        const int64_t mine = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;
        for (int64_t i = j; i < min(mine, j + stages); ++i)
          mbar_wait_bounded(&full[i % stages], (uint32_t)(i / stages) & 1u);
        break;
      }
      if (lane == 0) fetch(row + (int64_t)stages * gridDim.x, s);
      const RowSlots& r = slots[parity];
      const uint32_t top = __reduce_max_sync(0xffffffffu, lane < nwarps ? r.top[lane] : 0u);
      const float sum = NORM ? warp_sum(lane < nwarps ? r.sum[lane] : 0.f) : 0.f;
      put_scale<T, NORM>(a, row, top, row_out(top).some, sum, lane, flags);
      parity ^= 1;
      if (++s == stages) s = 0;
    }
  } else {
    float2 c[kRingVec][4];
#pragma unroll
    for (int i = 0; i < kRingVec; ++i)
      if (t + i * n < nvec) factors<T, NORM>(a, t + i * n, c[i]);
    uint32_t u = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
      const int64_t base = row * nvec;
      const unsigned char* src = ring + (size_t)s * stage;
      float2 v[kRingVec][4];
      RowStat r;
      r.sum = make_float2(0.f, 0.f);
      r.top = __uint_as_float(kGaveUp);
      if (mbar_wait_bounded(&full[s], u & 1u, a.tries)) {
        r.top = 0.f;
#pragma unroll
        for (int i = 0; i < kRingVec; ++i) {
          const int at = t + i * n;
          if (at < nvec) {
            Raw8<T> h;
            h.load(src, at);
            if constexpr (RES) {
              Raw8<T> o;
              o.load(src + row_bytes, at);
              h.add(o);
              h.store(a.sum, base + at);
            }
            take<NORM>(r, h, c[i], v[i]);
          }
        }
      } else {
        gave_up[parity] = 1;
      }
      RowSlots& slot = slots[parity];
      uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(r.top));
      float sum = 0.f;
      if constexpr (NORM) sum = warp_sum(r.sum.x + r.sum.y);
      if (lane == 0) {
        slot.top[warp] = top;
        if constexpr (NORM) slot.sum[warp] = sum;
      }
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, lane < nwarps ? slot.top[lane] : 0u);
      parity ^= 1;
      const RowOut o = row_out(top);
      if (o.some) {
#pragma unroll
        for (int i = 0; i < kRingVec; ++i)
          if (t + i * n < nvec) put_q(a, base + t + i * n, v[i], o);
      } else if (top == kGaveUp) {
        flags |= QAMW_STATUS_TIMEOUT;
        break;
      } else {
#pragma unroll
        for (int i = 0; i < kRingVec; ++i)
          if (t + i * n < nvec) reinterpret_cast<uint2*>(a.q)[base + t + i * n] = make_uint2(0u, 0u);
      }
      if (++s == stages) {
        s = 0;
        ++u;
      }
    }
  }
  raise_flag(a.status, flags);
}

// Shared memory of an SM that the rings of its CTAs (about 1024 threads together)
// take: 104 KB in flight were as fast as it got (208 KB: 8192 x 5120 bf16 with
// residual 53.5 us against 48.9), but a ring has two rows at least.
constexpr size_t kRingBytes = 104 * 1024, kRingMost = 208 * 1024;

template <typename T, bool NORM, bool RES>
cudaError_t run_ring(const Int8RowsArgs& a, int threads, size_t smem, cudaStream_t stream) {
  auto fn = &k_int8_ring<T, NORM, RES>;
  // the opt-in is for static and dynamic together above 48 KB: asked for with room
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(fn), smem + kStaticRoom);
  if (err != cudaSuccess) return err;
  const int grid = persistent_grid(reinterpret_cast<const void*>(fn), threads, smem, a.rows);
  return launch_pdl(fn, dim3(grid), dim3(threads), smem, stream, a);
}

template <typename T, bool NORM, bool RES>
cudaError_t run_rows_any(Int8RowsArgs a, cudaStream_t stream) {
  const int nvec = a.d / 8;
  if (a.d <= 512) {
    const int threads = (int)std::min<int64_t>(8, a.rows) * 32;
    return nvec <= 32 ? run_rows<T, kWarpRow, 1, NORM, RES>(a, threads, stream)
                      : run_rows<T, kWarpRow, 2, NORM, RES>(a, threads, stream);
  }
  if (a.rows <= 2 * sm_count() && nvec <= 1024)
    return run_rows<T, kWideRow, 1, NORM, RES>(a, (nvec + 31) / 32 * 32, stream);
  const size_t stage = (size_t)a.d * sizeof(T) * (RES ? 2 : 1);
  const int threads = ((nvec + kRingVec - 1) / kRingVec + 31) / 32 * 32 + 32;
  if (threads <= ring_threads<T, RES>() && 2 * stage <= kRingMost) {
    const size_t per = kRingBytes / std::max(1, 1024 / threads);
    a.stages = (int)std::min<size_t>(kRingMax, std::max<size_t>(2, per / stage));
    return run_ring<T, NORM, RES>(a, threads, a.stages * stage, stream);
  }
  return run_rows<T, kDeepRow, 4, NORM, RES>(a, ((nvec + 3) / 4 + 31) / 32 * 32, stream);
}

}  // namespace

cudaError_t launch_int8_encode(const void* d_x, int dtype, int64_t rows, int d,
                               const uint16_t* d_chan_scale, bool divide, int8_t* d_q,
                               float* d_scale, int32_t* d_status, cudaStream_t stream) {
  Int8RowsArgs a = {};
  a.tries = kSpinLimit;
  a.one = 1.f;
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
                                float* d_scale, int32_t* d_status, cudaStream_t stream,
                                unsigned tries) {
  Int8RowsArgs a = {};
  a.tries = tries;
  a.one = 1.f;
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
