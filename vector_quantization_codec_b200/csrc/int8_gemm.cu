// int8_gemm.cu -- product of 8-bit integers with a scale per token and per
// output channel, on the fifth-generation tensor cores (tcgen05.mma kind::i8,
// exact 32-bit accumulators in tensor memory):
//   Y[t][i] = T(float(sum_j xq[t][j] wq[i][j]) * (x_scale_t * w_scale_i)).
// The sum is an exact integer (|sum| <= 128 * 128 * 32768 = 2^29), so no tile,
// split or order of summation changes a result.
//
// The weights' rows are M of the MMA (lane of tensor memory = output channel)
// and the tokens are N (column): N follows the token count in steps of 16 or
// 32, and the 32 lanes of an epilogue warp store 32 consecutive outputs of a
// token whatever d_out is.
//
// Measured (B200, back to back over weights larger than L2): 8192 tokens 4096 ->
// 11008 227 us, 3.3 Pop/s, twice the bf16 rate of a library product (at the power
// cap of a long loop 261 us, 2.8); 2048 tokens 62 us with the tensor pipe active
// 82% of the time; 777 tokens 5120 -> 13824 44.1 us (2.5 Pop/s); 100 tokens 11008
// -> 4096 14.3 us, where the weights' way from HBM takes 7 and the cluster's
// partial sums 2.5; 16 tokens 4096 -> 11008 11.3 us (4.1 TB/s).  Outputs that leave
// by direct stores: 8192 tokens 4096 -> 11008 in fp32 289 us, bf16 4096 -> 11009
// 283; 777 tokens 5120 -> 13824 in fp32 47.8, bf16 -> 13825 46.5.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace qamw {
namespace {

constexpr int kRowsM = 128;           // output channels per CTA
constexpr int kChunk = 128;           // bytes of a row per stage: one swizzled line
constexpr uint32_t kTileA = kRowsM * kChunk;
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;          // warps 0-7: two per tensor-memory lane quarter
constexpr int kMmaWarp = 8;           // owner of the tensor memory; one thread issues the MMAs
constexpr int kCopyWarp = 9;          // one thread issues the copies
constexpr int kStoreWarp = 10;         // one thread issues the stores of staged outputs
constexpr int kThreads = 11 * 32;

// Batches up to this size write their outputs directly: too few to fill a block.
constexpr int kFewTokens = 16;
constexpr int kBlockTok = 64;  // tokens per staged block of outputs (of 128 channels, bf16)
constexpr uint32_t kBlock = kBlockTok * kRowsM * 2;
constexpr int kBlocks = 2;
// Shared memory, all of it dynamic so that its start is aligned for the swizzle:
// stages and (at the end of the same room) the staged blocks; then barriers,
// token scales and the tensor-memory address.
constexpr uint32_t kSmem = 224u * 1024u;
struct Int8Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], accfull[2], accempty[2], fin;
  float xs[2][2][128];  // [tile parity][half of the epilogue warps]
  uint32_t tmem_slot;
};
constexpr size_t kSmemAll = kSmem + sizeof(Int8Shared);
static_assert(kSmemAll <= 227 * 1024, "shared memory of an SM");
constexpr int kMaxSplits = 8;             // CTAs of a cluster

struct Int8GemmArgs {
  const float* xs;
  const float* ws;
  void* y;
  int32_t* status;
  int64_t tiles;   // (row tile, token tile) pairs, token tiles fastest
  int ntok, d_out;
  int chunks;      // of 128 bytes along d_in
  int tail;        // 32-byte steps of the last chunk (2 or 4)
  int nt;          // tokens per tile
  int tok_tiles;
  int stages;
  int boxes;       // chunks per stage
  int staged;      // bf16 outputs leave by tensor stores (map_y)
  int splits;      // CTAs (a cluster) that share a tile's chunks; 1: persistent over tiles
  // Polls of the waits of the copying thread and of the epilogue warps, kSpinLimit or 0
  // (for the check of giving up; the MMA thread, whose waits are the ones that cost time,
  // then runs into its limit).  Nothing between: the CTAs of a pair that gave up at
  // different steps rely on the second that the limit takes for the copies of the one
  // that went on to land.
  unsigned tries;
};

__device__ __forceinline__ void put(float* y, int64_t at, float v) { y[at] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, int64_t at, float v) {
  y[at] = __float2bfloat16_rn(v);
}

// True in one lane of a converged warp.  The compiler knows that one thread
// runs what this guards and keeps its operands in uniform registers; behind
// `lane == 0` four MMAs took 367 cycles to issue, more than they ran.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}

// Address of this CTA's shared address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int4 lds_cluster(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// Box of `map` at (column x, row y) into this CTA's shared memory; completion on
// the barrier at `bar` (CG 2: a shared::cluster address, the leader's barrier).
template <int CG>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// Block of shared memory to (column x, row y) of `map`, clipped at its edges.
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// Instruction descriptor of kind::i8: signed A and B (1 at bits 7-9 and 10-12),
// 32-bit integer accumulator (2 at bits 4-5), both K-major, N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` (CG 2: on the barrier at that offset of the cluster's CTAs in
// the mask `ctas`) once every MMA issued so far is done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t ctas) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)ctas)
        : "memory");
  else
    tc_commit(bar);
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
}

// 16 lanes x 16 columns of tensor memory as matrix fragments: v[4 j], v[4 j + 1]
// are columns 8 j + 2 (l % 4), + 1 of lane l / 4 (l: thread of the warp), and
// v[4 j + 2], v[4 j + 3] those of lane l / 4 + 8.  The caller waits.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, int (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr));
}

// Four 8 x 8 blocks of 16-bit values, transposed: thread t gives the address of
// row t % 8 (a column of the fragment) of block t / 8.
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// 16 consecutive 32-bit columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, int (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// One 128-byte chunk of a CTA's rows and tokens.
__host__ __device__ inline uint32_t box_bytes(int cg, int nt) {
  return kTileA + (uint32_t)(nt / cg) * kChunk;
}

// Columns of tensor memory: two accumulators, a power of two from 32.
__host__ __device__ inline uint32_t tmem_cols(int nt) {
  uint32_t c = 32;
  while (c < 2u * nt) c *= 2;
  return c;
}

// Sum of the `splits` partial tiles [token][128 channels] of a cluster: CTA
// `split` adds up and writes tokens split, split + splits, ..., of its 128
// channels, a warp one token at a time (its k-th is split + splits (warp + 8 k)),
// a lane four channels i, i + 1, ...; 16 loads in flight.  The CTAs with the same
// channels have the cluster ranks r0, r0 + CG, ...; w and xs are the scales of
// the lane's channels and of the warp's tokens, loaded long before.
template <int CG, typename T>
__device__ __forceinline__ void add_partials(const Int8GemmArgs& a, int64_t i, int t0, int split,
                                             uint32_t r0, uint32_t part, int warp, int lane,
                                             const float (&w)[4], const float* xs) {
  constexpr int kAhead = 4, kRanks = 4;
  T* y = reinterpret_cast<T*>(a.y);
  const bool fours = (a.d_out & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7u) == 0;
  const int nt = min(a.nt, a.ntok - t0), c0 = split + a.splits * warp, stride = a.splits * kEpiWarps;
  for (int k0 = 0; c0 + k0 * stride < nt; k0 += kAhead) {
    int sum[kAhead][4] = {};
    for (int rb = 0; rb < a.splits; rb += kRanks) {
      int4 v[kAhead][kRanks];
#pragma unroll
      for (int r = 0; r < kRanks; ++r) {
        const uint32_t from = cluster_addr(part + 16u * lane, r0 + (uint32_t)(CG * min(rb + r, a.splits - 1)));
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int c = c0 + (k0 + j) * stride;
          v[j][r] = rb + r < a.splits && c < nt ? lds_cluster(from + 4u * kRowsM * (uint32_t)c)
                                                : make_int4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
          sum[j][0] += v[j][r].x;
          sum[j][1] += v[j][r].y;
          sum[j][2] += v[j][r].z;
          sum[j][3] += v[j][r].w;
        }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + (k0 + j) * stride;
      if (c >= nt) break;
      T* out = y + (int64_t)(t0 + c) * a.d_out + i;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __fmul_rn((float)sum[j][e], __fmul_rn(xs[k0 + j], w[e]));
      if (std::is_same<T, __nv_bfloat16>::value && fours) {
        if (i < a.d_out)
          *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < a.d_out) put(out, e, f[e]);
      }
    }
  }
}

// CG = 2: a pair of CTAs works on a tile of 256 output channels (128 in each
// CTA's tensor memory) and nt tokens, each CTA staging its own 128 rows of W and
// half of the tokens; the even CTA (leader) issues the MMAs of both.
// CG = 1: a tile of 128 channels per CTA.
// With splits > 1 a cluster of that many CTAs or pairs shares the chunks of one
// tile and adds its integer partial sums through distributed shared memory; else
// the CTAs or pairs are persistent over tiles.
// Roles meet at mbarriers only: copies fill a ring of stages (full / empty), the
// MMAs fill one of two accumulators (accfull / accempty), the epilogue warps
// read the other out.
template <int CG, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    k_int8_gemm(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_y, const Int8GemmArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw;
  Int8Shared& sh = *reinterpret_cast<Int8Shared*>(smem + kSmem);
  uint64_t *full = sh.full, *empty = sh.empty, *accfull = sh.accfull, *accempty = sh.accempty;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t crank = CG == 2 || a.splits > 1 ? cluster_rank() : 0u;
  // place in the pair, split of the tile's chunks, the pair's leader and mask
  const uint32_t rank = CG == 2 ? (crank & 1u) : 0u;
  const int split = (int)(crank / CG);
  const uint32_t leader = crank - rank, pair = 3u << leader;
  const int S = a.stages;
  const uint32_t box = box_bytes(CG, a.nt), stage = box * a.boxes, cols = tmem_cols(a.nt);
  // tiles of this CTA (pair, cluster): first, first + step, ...
  const int per = CG * a.splits;
  const int64_t first = blockIdx.x / per, step = gridDim.x / per;
  const int c_lo = (int)((int64_t)split * a.chunks / a.splits);
  const int c_hi = (int)((int64_t)(split + 1) * a.chunks / a.splits);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], kEpiWarps * CG);
    }
    mbar_init(&sh.fin, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc<CG>(&sh.tmem_slot, cols);
  tc_fence_before();
  if (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_slot;
  // every operand and scale may come from the kernel ahead
  pdl_wait();
  pdl_trigger();
  int flags = 0;
  int64_t split_i = 0;
  int split_t0 = 0;
  float split_w[4] = {};

  if (warp == kCopyWarp) {
    if (elect_one()) {
      fence_proxy_async_global();  // both operands may come from the kernel ahead
      int s = 0;
      uint32_t u = 0;
      bool ok = true;
      for (int64_t tile = first; tile < a.tiles && ok; tile += step) {
        const int64_t m = tile / a.tok_tiles;
        const int row = (int)(m * (kRowsM * CG)) + (CG == 2 ? (int)rank * kRowsM : 0);
        const int tok = (int)(tile - m * a.tok_tiles) * a.nt + (CG == 2 ? (int)rank * (a.nt / 2) : 0);
        for (int c = c_lo; c < c_hi; c += a.boxes) {
          const int nb = min(a.boxes, c_hi - c);
          if (u > 0 && !mbar_wait_bounded(&empty[s], (u - 1) & 1u, a.tries)) {
            ok = false;
            break;
          }
          if (CG == 1 || rank == 0) mbar_expect_tx(&full[s], box * CG * nb);
          const uint32_t bar = CG == 2 ? cluster_addr(smem_u32(&full[s]), leader) : smem_u32(&full[s]);
          uint32_t dst = smem_u32(smem) + (uint32_t)s * stage;
          for (int j = 0; j < nb; ++j, dst += box) {
            copy_box<CG>(dst, &map_w, (c + j) * kChunk, row, bar);
            copy_box<CG>(dst + kTileA, &map_x, (c + j) * kChunk, tok, bar);
          }
          if (++s == S) {
            s = 0;
            ++u;
          }
        }
      }
      // nothing in flight at exit: the last use of each stage (in round u, or u - 1 from
      // stage s on) has been consumed, which also means that a pair's arrivals on these
      // barriers have landed
      const int used = u > 0 ? S : s;
      for (int k = 0; k < used && ok; ++k)
        ok = mbar_wait_bounded(&empty[k], (k < s ? u : u - 1) & 1u, a.tries);
      if (!ok) {  // given up: the copies at least have to land (a pair's leader waits for both)
        flags |= QAMW_STATUS_TIMEOUT;
        if (CG == 1 || rank == 0)
          for (int k = 0; k < used; ++k)
            if (!mbar_wait_bounded(&full[k], (k < s ? u : u - 1) & 1u)) break;
      }
    }
  } else if (warp == kMmaWarp) {
    if ((CG == 1 || rank == 0) && elect_one()) {
      const uint32_t idesc = idesc_i8(kRowsM * CG, a.nt);
      int s = 0, n = 0;
      uint32_t u = 0;
      bool ok = true;
      for (int64_t tile = first; tile < a.tiles && ok; tile += step, ++n) {
        const int b = n & 1;
        if (n >= 2 && !mbar_wait_bounded(&accempty[b], (uint32_t)((n >> 1) - 1) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * a.nt);
        for (int c = c_lo; c < c_hi; c += a.boxes) {
          const int nb = min(a.boxes, c_hi - c);
          if (!mbar_wait_bounded(&full[s], u & 1u)) {
            ok = false;
            break;
          }
          uint32_t sa = smem_u32(smem) + (uint32_t)s * stage;
          for (int j = 0; j < nb; ++j, sa += box) {
            const uint64_t da = smem_desc_sw128(sa), db = smem_desc_sw128(sa + kTileA);
            const int steps = c + j == a.chunks - 1 ? a.tail : kChunk / 32;
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k)  // 32 bytes of a row per MMA
              if (k < steps)
                mma_i8<CG>(d, da + 2u * k, db + 2u * k, idesc, (c + j > c_lo || k > 0) ? 1u : 0u);
          }
          commit<CG>(&empty[s], pair);
          if (++s == S) {
            s = 0;
            ++u;
          }
        }
        if (ok) commit<CG>(&accfull[b], pair);
      }
      if (!ok) flags |= QAMW_STATUS_TIMEOUT;
      // every MMA is done before the tensor memory and the stages are given up
      commit<CG>(&sh.fin, 1u << leader);
      if (!mbar_wait_bounded(&sh.fin, 0)) flags |= QAMW_STATUS_TIMEOUT;
    }
  } else if (warp == kStoreWarp) {
    if (a.staged) {
      const bool one = elect_one();
      const uint32_t blocks = smem_u32(smem) + kSmem - kBlocks * kBlock;
      int block = 0;
      for (int64_t tile = first; tile < a.tiles; tile += step) {
        const int64_t m = tile / a.tok_tiles;
        const int i0 = (int)(m * (kRowsM * CG)) + (int)rank * kRowsM;
        const int t0 = (int)(tile - m * a.tok_tiles) * a.nt;
        const int nt = min(a.nt, a.ntok - t0);
        for (int c = 0; c < nt; c += kBlockTok) {
          // the block that comes next is free once its stores have read it: the epilogue
          // warps write it behind this barrier
          if (one) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps + 32) : "memory");
          if (one) {
            const uint32_t buf = blocks + block * kBlock;
            // 64 channels x 32 tokens a store: a tile may end in the middle of a block
            for (int k = 0; k < 2; ++k)
              for (int h = 0; h < 2; ++h)
                if (i0 + 64 * k < a.d_out && c + 32 * h < nt)
                  store_box(&map_y, i0 + 64 * k, t0 + c + 32 * h, buf + k * (kBlock / 2) + h * (kBlock / 4));
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          block ^= 1;
        }
      }
      if (one) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else if (a.splits == 1) {
    T* y = reinterpret_cast<T*>(a.y);
    // warp w: lanes (channels) 32 (w % 4) .. + 31, columns 32 k + 16 (w / 4) .. + 15
    const int q4 = warp & 3, half = warp >> 2;
    const uint32_t blocks = smem_u32(smem) + kSmem - kBlocks * kBlock;
    int n = 0, block = 0;
    bool alive = true;
    for (int64_t tile = first; tile < a.tiles; tile += step, ++n) {
      const int b = n & 1;
      const int64_t m = tile / a.tok_tiles;
      const int64_t i0 = m * (kRowsM * CG) + (CG == 2 ? (int64_t)rank * kRowsM : 0);
      const int64_t i = i0 + 32 * q4 + lane;
      const int t0 = (int)(tile - m * a.tok_tiles) * a.nt;
      const int nt = min(a.nt, a.ntok - t0);
      const bool mine = i < a.d_out;
      const float wi = !a.staged && mine ? a.ws[i] : 0.f;
      float wg[4];  // staged: channels lane / 4 + 8 g of the warp's 32
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t k = i0 + 32 * q4 + (lane >> 2) + 8 * g;
        wg[g] = a.staged && k < a.d_out ? a.ws[k] : 0.f;
      }
      // the scales of the warp's tokens, all loads in flight together: entry k is token
      // 32 (k / 16) + 16 half + k % 16 of the tile
      float x4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = 64 * k + 32 * (lane >> 4) + 16 * half + (lane & 15);
        x4[k] = c < nt ? a.xs[t0 + c] : 0.f;
      }
      // one lane polls: 32 pollers a warp would slow the other roles' waits.  A
      // wait that gives up is not repeated; the warps still meet at the barriers.
      const bool ok =
          !alive || lane != 0 || mbar_wait_bounded(&accfull[b], (uint32_t)(n >> 1) & 1u, a.tries);
      if (__any_sync(0xffffffffu, !ok)) {
        flags |= QAMW_STATUS_TIMEOUT;
        alive = false;
      }
      // (the four warps of a half write the same; a warp that gets here has seen the
      // others done with the tile before the last, whose scales these replace)
      float* xs = sh.xs[b][half];
#pragma unroll
      for (int k = 0; k < 4; ++k) xs[lane + 32 * k] = x4[k];
      __syncwarp();
      tc_fence_after();
      if (a.staged) {
        // 64 tokens x 128 channels of all eight warps go through shared memory and
        // leave by tensor stores.  (Direct 2-byte stores, or shuffles to wider ones,
        // kept the load-store unit busy for 4300 cycles a tile of 256 tokens.)
        for (int c = 0; c < nt; c += kBlockTok) {
          const uint32_t buf = blocks + block * kBlock;
          block ^= 1;
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) {
            const int cw = c + 32 * sb + 16 * half;
            if (cw < nt) {
              int v[2][8];
              tmem_ld_frag(tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(b * a.nt + cw), v[0]);
              tmem_ld_frag(tmem + ((uint32_t)(32 * q4 + 16) << 16) + (uint32_t)(b * a.nt + cw), v[1]);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 x2 =
                    *reinterpret_cast<const float2*>(xs + c / 2 + 16 * sb + 8 * j + 2 * (lane & 3));
                uint32_t w[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const int lo = v[g >> 1][4 * j + 2 * (g & 1)], hi = v[g >> 1][4 * j + 2 * (g & 1) + 1];
                  const float2 f = mul2(make_float2((float)lo, (float)hi), mul2(x2, make_float2(wg[g], wg[g])));
                  w[g] = pack_bf16x2(f.x, f.y);
                }
                // block g of eight channels = 16-byte unit 4 (q4 % 2) + g of the 64
                // channels q4 / 2; swizzled as the tensor store expects
                const int tok = 32 * sb + 16 * half + 8 * j + (lane & 7), unit = 4 * (q4 & 1) + (lane >> 3);
                stmatrix4_t(buf + (uint32_t)((q4 >> 1) * (kBlock / 2) + tok * 128 + ((unit ^ (tok & 7)) << 4)), w);
              }
            }
          }
          fence_proxy_async_smem();
          asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps + 32) : "memory");
        }
      } else {
        const int64_t pitch = a.d_out;
        for (int c = 16 * half; c < nt; c += 32) {
          int v[16];
          tmem_ld16(tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(b * a.nt + c), v);
          T* out = y + (t0 + c) * pitch + i;
          const float* xc = xs + c / 32 * 16;
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = __fmul_rn((float)v[e], __fmul_rn(xc[e], wi));
          if (mine) {
            if (c + 16 <= nt) {
#pragma unroll
              for (int e = 0; e < 16; ++e) put(out, e * pitch, f[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c + e < nt) put(out, e * pitch, f[e]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(cluster_addr(smem_u32(&accempty[b]), leader));
        else
          mbar_arrive(&accempty[b]);
      }
    }
  } else {
    // the scales that add_partials will need, while the products come in
    const int64_t m = first / a.tok_tiles;
    split_i = m * (kRowsM * CG) + (int64_t)rank * kRowsM + 4 * lane;
    split_t0 = (int)(first - m * a.tok_tiles) * a.nt;
#pragma unroll
    for (int e = 0; e < 4; ++e) split_w[e] = split_i + e < a.d_out ? a.ws[split_i + e] : 0.f;
    {
      const int t = split_t0 + split + a.splits * (warp + kEpiWarps * lane);
      (&sh.xs[0][0][0])[32 * warp + lane] = t < a.ntok ? a.xs[t] : 0.f;
    }
    // the CTA's partial sums into its own shared memory (the stages are free:
    // every MMA that reads them is done), [token][channel]
    int* part = reinterpret_cast<int*>(smem);
    const bool ok = lane != 0 || mbar_wait_bounded(&accfull[0], 0, a.tries);
    if (__any_sync(0xffffffffu, !ok)) flags |= QAMW_STATUS_TIMEOUT;
    tc_fence_after();
    for (int c = 16 * (warp >> 2); c < a.nt; c += 32) {
      int v[16];
      tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) part[(c + e) * kRowsM + (tid & (kRowsM - 1))] = v[e];
    }
  }
  tc_fence_before();
  if (a.splits > 1) {
    __syncwarp();
    cluster_sync();
    if (warp < kEpiWarps)
      add_partials<CG, T>(a, split_i, split_t0, split, rank, smem_u32(smem), warp, lane, split_w,
                          &sh.xs[0][0][0] + 32 * warp);
  }
  __syncwarp();
  if (CG == 2 || a.splits > 1)
    cluster_sync();  // no CTA leaves while another reads its memory or signals its barriers
  else
    __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free<CG>(tmem, cols);
  }
  raise_flag(a.status, flags);
}

// bf16 [rows][d_out] for tensor stores of 64 channels (one swizzled line) x 32 tokens.
bool encode_out_map(CUtensorMap* map, void* p, int64_t rows, int d_out) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d_out, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d_out * 2};
  const cuuint32_t boxes[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 8-bit matrix [rows][d_in] for boxes of 128 bytes x `box` rows, swizzled.
bool encode_map(CUtensorMap* map, const int8_t* p, int64_t rows, int d_in, int box) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d_in, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d_in};
  const cuuint32_t boxes[2] = {kChunk, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, boxes,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Int8Plan {
  int cg, nt, splits, boxes, stages;
  bool staged;
};

// Clusters of `per` CTAs of k_int8_gemm that the current device holds at once.  A
// cluster's CTAs share a GPC, whose SMs are rarely a multiple of four or eight: a
// B200 of 148 SMs holds 45, 33, 22 and 15 of three, four, six and eight CTAs.  (By
// SMs / 8 = 18 the estimate below took 16 clusters of eight for one wave: 16 tokens
// 4096 -> 2048 took 9.6 us in two, and takes 5.7 with six CTAs a cluster.)
int clusters_at_once(int per) {
  static std::atomic<int> cached[64][kMaxSplits + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return std::max(1, sm_count() / per);
  int n = cached[dev][per].load(std::memory_order_relaxed);
  if (n > 0) return n;
  // registers, shared memory and threads of a CTA are alike in all four instances
  auto fn = &k_int8_gemm<1, float>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)per);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAll;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)per;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (per == 1 || allow_smem(reinterpret_cast<const void*>(fn), kSmemAll) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1)
    n = std::max(1, sm_count() / per);
  cached[dev][per].store(n, std::memory_order_relaxed);
  return n;
}

// Estimated time (ns) of a plan, fitted to 360 measured (shape, plan) pairs when 32
// tokens were staged a barrier.  Over 28 shapes from 9 x 4096 -> 4096 to 8192 x 4096
// -> 11008, with 716 plans measured on the kernel as it is, the plan that it picks is
// within 6% of the fastest (mean 1%), but for 16 x 4096 -> 2048 (10%: six CTAs a
// cluster, not four).  A chunk of a CTA
// costs the longest of its MMAs, its way through shared memory (128 channels and nt /
// cg tokens) and a floor; the last tile's epilogue is not hidden, earlier ones are
// unless the depth is short; sharing a tile's chunks among CTAs costs two cluster
// barriers and the reading of the partial sums.
int64_t plan_ns(int ntok, int d_out, int chunks, int cg, int nt, int splits, int at_once) {
  const int64_t tiles =
      (int64_t)((d_out + kRowsM * cg - 1) / (kRowsM * cg)) * ((ntok + nt - 1) / nt);
  const int64_t waves = (tiles + at_once - 1) / at_once;
  const int chunk = std::max(std::max(118 * nt / 100, 98 * (kRowsM + nt / cg) / 100), 225);
  const int main = (chunks + splits - 1) / splits * chunk, epilogue = 10 * nt;
  int64_t t = waves * (std::max(main, epilogue) + 1900) + epilogue;
  if (splits > 1) t += waves * 2150 + (waves - 1) * epilogue + 7 * nt;
  return t;
}

// bf16_rows: bf16 outputs whose rows are multiples of 16 bytes.
Int8Plan plan_int8(int ntok, int d_out, int d_in, bool bf16_rows) {
  Int8Plan p = {};
  const int chunks = (d_in + kChunk - 1) / kChunk;
  int64_t best = INT64_MAX;
  int at_once[kMaxSplits + 1];
  for (int per = 1; per <= kMaxSplits; ++per) at_once[per] = clusters_at_once(per);
  for (int cg = 1; cg <= 2; ++cg) {
    // tokens in steps of 16 per CTA; single CTAs only where a pair's tile would be
    // wider than the batch needs
    const int unit = 16 * cg, most = cg == 1 ? 128 : 256;
    if (cg == 1 && ntok > 512) continue;
    for (int nt = unit; nt <= most && nt < ntok + unit; nt += unit)
      for (int splits = 1; splits * cg <= kMaxSplits; ++splits) {
        if (splits > 1 && 2 * splits > chunks) break;
        if (splits * cg == 5 || splits * cg == 7) continue;  // leave SMs of a GPC unused
        const int64_t t = plan_ns(ntok, d_out, chunks, cg, nt, splits, at_once[cg * splits]);
        if (t < best) {
          best = t;
          p.cg = cg;
          p.nt = nt;
          p.splits = splits;
        }
      }
  }
  // the wait for a stage and its commit cost the MMA thread about 240 cycles:
  // several chunks per stage, as long as three stages fit
  p.staged = bf16_rows && p.splits == 1 && ntok > kFewTokens && (p.nt % 32 == 0 || ntok <= p.nt);
  const uint32_t ring = kSmem - (p.staged ? kBlocks * kBlock : 0);
  p.boxes = 4;
  while (p.boxes > 1 && ring / (box_bytes(p.cg, p.nt) * p.boxes) < 3) --p.boxes;
  p.stages = (int)std::min<uint32_t>(kMaxStages, ring / (box_bytes(p.cg, p.nt) * p.boxes));
  return p;
}

// A few tokens: the weights' rows straight from global memory, by dot products (a
// warp a row, 32 rows of an SM at once) or by the warp-level MMA (a CTA 16 rows, 48
// of an SM at once), or else the tensor-core kernel of this file.  Measured, us,
// dot / MMA / tensor core (back to back over weights larger than L2 where they are):
//   1 token   4096 -> 4096   3.8 / 6.1 / 7.3     4096 -> 32001 19.3 / 21.6 / 23.0
//   2 tokens  4096 -> 4096   4.8 / 6.2 / 7.4     4096 -> 32001 21.1 / 21.9 / 23.1
// Rows shorter than a warp's 4 KB leave loads empty, which shows where a warp takes
// several rows:
//   1 token   1024 -> 6000   3.4 / 3.9 / 4.2     1024 -> 13824  5.7 / 4.4 / 6.2
//   1 token    256 -> 4096   2.7 / 3.3 / 3.1      256 -> 32001 10.4 / 4.9 / 5.1
//   2 tokens  2048 -> 4096   3.7 / 4.2 / 5.4     2048 -> 13824  7.5 / 6.6 / 8.4
// and so do rows that are a little longer, with two tokens:
//   2 tokens  5120 -> 4096   6.5 / 7.4 / 8.3     5120 -> 13824 14.9 / 13.6 / 14.4
//   2 tokens  5632 -> 11008 13.7 / 14.5 / 14.1   5376 -> 11008 13.9 / 13.5 / 14.0
// Two long tokens leave no room for four CTAs of the dot products on an SM:
//   2 tokens 20480 -> 4096  15.7 / - / 16.9     32768 -> 4096  38.0 / - / 25.7
//   2 tokens 32768 -> 2048  20.1 / - / 22.3     32768 -> 13824 83.2 / - / 85.2
// The MMA takes too many steps per 16 rows where d_in is large, and a round of rows
// that fills few SMs costs as much as a full one:
//   5 tokens  4096 -> 8192   -   / 9.2 / 9.4     5120 -> 8192   -   / 12.1 / 10.7
//   5 tokens  5120 -> 11008  -  / 13.2 / 13.3    5632 -> 11008  -   / 14.7 / 14.2
//   5 tokens  5632 -> 2048   -   / 6.3 / 6.9     8192 -> 1024   -   / 7.4 / 6.1
enum class FewTokens { kNone, kDot, kMma };

FewTokens few_token_kernel(int ntok, int d_out, int d_in) {
  if (ntok > 8 || d_in < 256) return FewTokens::kNone;
  const int64_t sms = sm_count(), groups = ((int64_t)d_out + 15) / 16, at_once = 3 * sms;
  // one round of 16 rows per CTA, or a last round that is not almost empty
  const bool full = groups <= at_once || 4 * groups >= 3 * ((groups + at_once - 1) / at_once * at_once);
  const bool mma_fits = d_in >= 512 && (d_in <= 4096 || (d_in <= 5376 && full) ||
                                        (d_in <= 6144 && d_out <= 24 * sms));
  const FewTokens mma = mma_fits ? FewTokens::kMma : FewTokens::kNone;
  if (ntok > 2) return mma;
  if (d_in <= 1024 * ntok && d_out > 48 * sms) return mma;
  if (ntok == 2 && d_in > 4096 && d_in <= 5376 && d_out > 32 * sms && full) return mma;
  if (ntok == 2 && d_in > 26000 && d_out > 24 * sms) return FewTokens::kNone;
  return FewTokens::kDot;
}

template <int CG, typename T>
cudaError_t run_gemm(const Int8Plan& p, const CUtensorMap& mw, const CUtensorMap& mx,
                     const CUtensorMap& my, const Int8GemmArgs& a, cudaStream_t stream) {
  auto fn = &k_int8_gemm<CG, T>;
  // all of the ring, whatever the stages need of it: one CTA that owns tensor
  // memory per SM, so that an allocation never waits for a CTA that could be
  // waiting for it
  constexpr size_t smem = kSmemAll;
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(fn), smem);
  if (err != cudaSuccess) return err;
  const int per = CG * p.splits;
  const int64_t most = p.splits > 1 ? a.tiles : std::max(1, sm_count() / per);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.tiles, most) * per));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)per;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, mw, mx, my, a);
}

}  // namespace

cudaError_t launch_int8_gemm(const int8_t* d_x, const float* d_x_scale, int ntok, const int8_t* d_w,
                             const float* d_w_scale, int d_out, int d_in, void* d_y, int dtype,
                             int32_t* d_status, cudaStream_t stream, unsigned tries) {
  const FewTokens few = few_token_kernel(ntok, d_out, d_in);
  if (few != FewTokens::kNone)
    return launch_int8_gemv(d_x, d_x_scale, ntok, d_w, d_w_scale, d_out, d_in, d_y, dtype,
                            few == FewTokens::kMma, stream);
  const Int8Plan p = plan_int8(ntok, d_out, d_in,
                               dtype == QAMW_DTYPE_BF16 && d_out % 8 == 0 &&
                                   (reinterpret_cast<uintptr_t>(d_y) & 15u) == 0);
  CUtensorMap mw, mx, my = {};
  if (!encode_map(&mw, d_w, d_out, d_in, kRowsM) || !encode_map(&mx, d_x, ntok, d_in, p.nt / p.cg))
    return cudaErrorInvalidValue;
  Int8GemmArgs a = {};
  a.xs = d_x_scale;
  a.ws = d_w_scale;
  a.y = d_y;
  a.status = d_status;
  a.ntok = ntok;
  a.d_out = d_out;
  a.chunks = (d_in + kChunk - 1) / kChunk;
  a.tail = (d_in - (a.chunks - 1) * kChunk) / 32;
  a.nt = p.nt;
  a.tok_tiles = (ntok + p.nt - 1) / p.nt;
  a.tiles = (int64_t)((d_out + kRowsM * p.cg - 1) / (kRowsM * p.cg)) * a.tok_tiles;
  a.stages = p.stages;
  a.boxes = p.boxes;
  a.splits = p.splits;
  a.tries = tries;
  a.staged = p.staged;
  if (a.staged && !encode_out_map(&my, d_y, ntok, d_out)) return cudaErrorInvalidValue;
  if (dtype == QAMW_DTYPE_F32)
    return p.cg == 2 ? run_gemm<2, float>(p, mw, mx, my, a, stream)
                     : run_gemm<1, float>(p, mw, mx, my, a, stream);
  return p.cg == 2 ? run_gemm<2, __nv_bfloat16>(p, mw, mx, my, a, stream)
                   : run_gemm<1, __nv_bfloat16>(p, mw, mx, my, a, stream);
}

}  // namespace qamw
