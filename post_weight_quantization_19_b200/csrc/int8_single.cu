// gptq_int8_linear and gptq_int8_gated, weights as the rows of the tensor-core product: up to
// 64 tokens, and up to 256 (gated: 128) where k is split.
//
//   y[t, i] = xs[t] ws[i] sum_j x[t, j] w[i, j] + bias[i]
//   gated:  y = act(the gate's) * (the up projection's)
//
// One CTA per tile of 128 rows of W and all N <= 256 tokens; a gated tile has the 128
// rows of both layers, each with its sums in its own columns of tensor memory, so that a
// thread ends up with both projections of a row and writes their product alone.
// TMA brings slabs of 128 columns of W and x to 128-byte-swizzled shared memory, one
// thread issues the MMAs (kind::i8, 32 columns each), four warps write the results.
// The sums are exact: |sum| <= 65536 * 2^14 = 2^30.
//
// Few tokens are bound by reading W once, so the shape serves the copies: rings of about
// 100 KB, two CTAs to an SM (and the next kernel's beside the last one's), and the first
// loads leave before the CTA has met.  Where tiles are few, the k range is split over a
// cluster: each CTA of it owns 128 / ctas_k rows of the tile and the others push their sums
// of those rows into its shared memory (st.async, counted on its mbarrier), so the sums
// cross once and nobody asks for them.  Integers: their order changes nothing.
#include "int8_linear.h"
#include "launch_after.h"

namespace gptq {
namespace {

constexpr int ROWS = 128;                 // rows of W per tile (UMMA M)
constexpr int SLAB = 128;                 // columns per stage
constexpr int TOKENS = 256;               // most tokens (UMMA N), of both layers' sums together
constexpr int STAGES = 12;                // at most
// Waits of a CTA that may run out one behind the other before it sends its sums: the loader's for
// a free stage and for the last load of each, the MMAs' for an accumulator, a stage and their end.
constexpr int SETTLE = STAGES + 4;
constexpr int SINGLE_THREADS = 32 * 6;
constexpr size_t SINGLE_SMEM = 208 * 1024;
constexpr size_t SHARED_SM = 102 * 1024;  // where two CTAs share an SM
// Tensor memory is taken CTA by CTA, without a limit on the wait, and the CTAs of a cluster then
// wait for each other.  So CTAs of several streams' kernels that meet on one SM must never ask
// for more than its 512 columns together: two clusters could each hold what the other waits
// for.  Shared memory keeps them apart, 228 KB to an SM.  At least LEAST_SMEM each, 57 KB with
// what is static: three at most, of 128 columns or fewer.  With more, up to 256, at least
// WIDE_SMEM: two of them leave no room for a third.  (Kernels that take all columns leave none
// for any of these: 185 KB or more, or the packed layer's 768 threads of 72 registers or more.)
constexpr size_t SM_SMEM = 228 * 1024, CTA_RESERVED = 1024;
constexpr size_t LEAST_SMEM = 48 * 1024, WIDE_SMEM = 78 * 1024;

struct SingleArgs {
  Int8Args p;
  int N;              // tokens, rounded up to a multiple of 16
  int rows;           // of W per tile, a multiple of 8
  int deep;           // slabs per stage
  int tiles;
  int ctas_k;         // CTAs of a cluster, along k
  int stages;
  uint32_t columns;   // of tensor memory: two accumulators, with k split one
  int slots;          // split k: where the CTAs' sums meet, an offset in shared memory; 0: in the ring
  int *status;
};

struct SingleShared {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain, sums;
  uint32_t tmem_base;
  int abort;
  alignas(16) uint16_t stage[4][16 * 32];   // results on their way out, per warp: [token][row]
  alignas(16) float xs[4][TOKENS];          // scales of a tile's tokens, per warp
};

constexpr size_t smem_held(size_t bytes) { return bytes + 1024 + sizeof(SingleShared) + CTA_RESERVED; }
static_assert(4 * smem_held(LEAST_SMEM) > SM_SMEM, "more CTAs to an SM than columns of tensor memory");
static_assert(2 * smem_held(WIDE_SMEM) + smem_held(LEAST_SMEM) > SM_SMEM, "more columns asked for than there are");

__device__ __forceinline__ void single_timeout(int *status, SingleShared &sh) {
  atomicCAS(status, 0, (int)GPTQ_ERR_TIMEOUT);
  *(volatile int *)&sh.abort = 1;
}

// Four integers into the shared memory of a CTA of the cluster, counted on its mbarrier.
__device__ __forceinline__ void push4(uint32_t addr, uint32_t bar, int a, int b, int c, int d) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.s32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
               : "memory");
}

// A row's parameters.
struct Row {
  float scale[2], bias[2];
};
template <bool GATED>
__device__ __forceinline__ Row row_of(const Int8Args &p, int64_t row) {
  Row r{};
#pragma unroll
  for (int k = 0; k < (GATED ? 2 : 1); ++k) {
    if (row >= p.r) continue;
    r.scale[k] = __ldcg(p.w_scales[k] + row);
    if (p.bias[k]) r.bias[k] = load_typed(p.bias[k], p.ytype, row);
  }
  return r;
}

// Results of one row and two tokens from their sums.
template <bool GATED, int ACT, typename Y>
__device__ __forceinline__ F2 results(int a0, int a1, int b0, int b1, float x0, float x1, const Row &r) {
  const F2 v{scaled_sum(a0, x0, r.scale[0], r.bias[0]), scaled_sum(a1, x1, r.scale[0], r.bias[0])};
  if constexpr (!GATED) return v;
  return gated_pair<ACT, Y>(
      v, F2{scaled_sum(b0, x0, r.scale[1], r.bias[1]), scaled_sum(b1, x1, r.scale[1], r.bias[1])});
}

// 16 tokens of an accumulator's 32 rows to y, `live` of the rows in the tile; a lane is a
// row.  16-bit results go through shared memory and out 16 bytes, eight rows of a token,
// per lane, where y's rows allow it.
template <typename Y>
__device__ __forceinline__ void write_tokens(const float (&v)[16], int count, int t0, int64_t row0, int live,
                                             const Int8Args &p, uint16_t *stage, int lane) {
  Y *y = static_cast<Y *>(p.y);
  bool wide = false;
  if constexpr (sizeof(Y) == 2) wide = p.r % 8 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
  if (wide) {
    if constexpr (sizeof(Y) == 2) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) reinterpret_cast<Y *>(stage)[i * 32 + lane] = to_result<Y>(v[i]);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = h * 8 + (lane >> 2);
        const uint4 o = reinterpret_cast<const uint4 *>(stage)[h * 32 + lane];
        if (tok < count && (lane & 3) * 8 < live)   // live: a multiple of 8
          *reinterpret_cast<uint4 *>(y + (int64_t)(t0 + tok) * p.r + row0 + (lane & 3) * 8) = o;
      }
    }
  } else if (lane < live) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < count) y[(int64_t)(t0 + i) * p.r + row0 + lane] = to_result<Y>(v[i]);
  }
}

template <bool GATED, int ACT, typename Y>
__global__ void __launch_bounds__(SINGLE_THREADS, 1)
    int8_single_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmU, const SingleArgs a) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ SingleShared sh;
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  constexpr int LAYERS = GATED ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = a.N, w_bytes = a.rows * SLAB, x_at = a.deep * LAYERS * w_bytes;
  const int stage_bytes = x_at + a.deep * N * SLAB;
  const int crank = blockIdx.x % a.ctas_k, ctas = gridDim.x / a.ctas_k, cta = blockIdx.x / a.ctas_k;
  const int tiles = a.tiles;
  const int steps = (a.p.d + SLAB * a.deep - 1) / (SLAB * a.deep);
  const int k0 = (int)((int64_t)steps * crank / a.ctas_k);
  const int k1 = (int)((int64_t)steps * (crank + 1) / a.ctas_k);
  const uint32_t acc_columns = LAYERS * N;

  const int n = (int)a.p.n, fours = (n + 3) / 4;   // tokens, in fours
  const int owned = a.rows / a.ctas_k;   // rows
  // (what a load takes is kept ready: one thread issues them all, and divisions in its loop
  // cost 800 clocks a step, more than the step's data)
  auto load = [&](int m0, int k, uint32_t dst, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, stage_bytes);
    // columns from multiples of 128 bytes (past d, r and n: zeros)
    int col = k * (a.deep * SLAB);
    uint32_t x = dst + x_at;
    for (int j = 0; j < a.deep; ++j, col += SLAB, x += N * SLAB) {
      load_2d(dst, &tmW, col, m0, bar);
      dst += w_bytes;
      if constexpr (GATED) {
        load_2d(dst, &tmU, col, m0, bar);
        dst += w_bytes;
      }
      load_2d(x, &tmX, col, 0, bar);
    }
  };
  const uint32_t ring = smem_u32(smem);
  int ahead = 0;   // thread 0: slabs of the first tile asked for at the start

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], 4);
    }
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.sums, 1);
    sh.abort = 0;
    fence_mbar_init();
    if (a.ctas_k > 1) mbar_arrive_expect_tx(&sh.sums, (a.ctas_k - 1) * LAYERS * fours * owned * 16);
    for (int k = k0; k < k1 && k < k0 + a.stages; ++k)   // (into L2, whoever wrote them)
      for (int j = 0; j < a.deep; ++j) {
        prefetch_2d(&tmW, (k * a.deep + j) * SLAB, cta * a.rows);
        if constexpr (GATED) prefetch_2d(&tmU, (k * a.deep + j) * SLAB, cta * a.rows);
      }
    pdl_wait();
    for (; ahead < a.stages && k0 + ahead < k1; ++ahead)
      load(cta * a.rows, k0 + ahead, ring + ahead * stage_bytes, &sh.full[ahead]);
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem_base, a.columns);
    tmem_relinquish();
  }
  __syncwarp();
  if (a.ctas_k > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // barriers are there
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  // Tensor memory is there before the next kernel may start, so that its CTAs cannot take it
  // from one that they wait for.  (Products of the solve, which take it later, leave no CTA
  // of this kernel room beside them.  Taken behind the wait: one token x
  // 4096 x 4096 8.0 us, not 7.3.)
  pdl_wait_then_release();

  if (warp == 0) {
    // ---------------------------------------------------------------- W and x by TMA
    if (lane == 0) {
      int stage = ahead == a.stages ? 0 : ahead;
      uint32_t phase = ahead == a.stages ? 1 : 0;
      bool ok = true, full = phase != 0;   // full: every stage has been asked for
      for (int t = cta; t < tiles && ok; t += ctas) {
        for (int k = t == cta ? k0 + ahead : k0; k < k1; ++k) {
          ok = wait_or_abort(&sh.empty[stage], phase ^ 1, &sh.abort);
          if (!ok) {
            single_timeout(a.status, sh);
            break;
          }
          load(t * a.rows, k, ring + stage * stage_bytes, &sh.full[stage]);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
            full = true;
          }
        }
      }
      // the last load of every stage has landed: stages before `stage` in this phase, the
      // others in the one before
      for (int s = 0; s < a.stages; ++s)
        if (full || s < stage) (void)mbar_wait_bounded(&sh.full[s], s < stage ? phase : phase ^ 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- the MMAs
    const uint32_t idesc = instr_desc_i8(ROWS, N);
    const uint64_t first = smem_desc(smem_u32(smem), 16, 1024, 2);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int stage = 0;
    uint32_t phase = 0, buf = 0, cphase = 0;
    bool ok = true;
    for (int t = cta; t < tiles && ok; t += ctas) {
      ok = mbar_wait_bounded(&sh.acc_empty[buf], ((cphase >> buf) & 1u) ^ 1u);
      for (int k = k0; k < k1; ++k) {
        ok = ok && mbar_wait_bounded(&sh.full[stage], phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane()) {
          // (a tile of fewer rows multiplies what lies behind them too, for results that
          // nobody reads)
          const uint32_t d0 = tm + buf * acc_columns;
          uint64_t w = first + (uint64_t)(stage * stage_bytes >> 4), x = w + (x_at >> 4);
          for (int j = 0; j < a.deep; ++j, w += LAYERS * w_bytes >> 4, x += N * SLAB >> 4)
#pragma unroll
            for (int q = 0; q < SLAB / 32; ++q) {
              umma_i8_ss(d0, w + q * 2, x + q * 2, idesc, k > k0 || j > 0 || q > 0);
              if constexpr (GATED)
                umma_i8_ss(d0 + N, w + (w_bytes >> 4) + q * 2, x + q * 2, idesc, k > k0 || j > 0 || q > 0);
            }
          umma_commit(&sh.empty[stage]);
          if (k == k1 - 1) umma_commit(&sh.acc_full[buf]);
        }
        __syncwarp();
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      cphase ^= 1u << buf;
      buf ^= 1;
    }
    if (!ok && lane == 0) single_timeout(a.status, sh);
    __syncwarp();
    if (elect_lane()) {
      umma_commit(&sh.drain);
      (void)mbar_wait_bounded(&sh.drain, 0);
    }
    __syncwarp();
  } else if (a.ctas_k == 1) {
    // ---------------------------------------------------------------- results
    const int quarter = warp & 3;
    uint32_t buf = 0, cphase = 0;
    bool ok = true;
    for (int t = cta; t < tiles && ok; t += ctas) {
      const int64_t row0 = (int64_t)t * a.rows + quarter * 32;
      const int64_t left = min((int64_t)a.rows - quarter * 32, a.p.r - row0);
      const int live = left < 0 ? 0 : left < 32 ? (int)left : 32;
      const Row par = row_of<GATED>(a.p, row0 + lane);
      __syncwarp();
      for (int c = lane; c < N; c += 32) sh.xs[quarter][c] = c < n ? __ldcg(a.p.x_scales + c) : 0.f;
      __syncwarp();
      if (gives_up(a.p, warp, lane, t, ctas, tiles)) ok = false;
      ok = ok && mbar_wait_bounded(&sh.acc_full[buf], (cphase >> buf) & 1u);
      ok = __all_sync(0xffffffffu, ok);   // (one lane's wait may run out alone)
      if (!ok && lane == 0) single_timeout(a.status, sh);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + buf * acc_columns;
      for (int c0 = 0; c0 < n && live > 0; c0 += 16) {
        float s0[16], s1[16];   // sums' bits
        tmem_ld_32x32b_x16(base + c0, s0);
        if constexpr (GATED) tmem_ld_32x32b_x16(base + N + c0, s1);
        tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const F2 f = results<GATED, ACT, Y>(
              __float_as_int(s0[i]), __float_as_int(s0[i + 1]), GATED ? __float_as_int(s1[i]) : 0,
              GATED ? __float_as_int(s1[i + 1]) : 0, sh.xs[quarter][c0 + i], sh.xs[quarter][c0 + i + 1], par);
          v[i] = f.x;
          v[i + 1] = f.y;
        }
        write_tokens<Y>(v, n - c0, c0, row0, live, a.p, sh.stage[quarter], lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
      cphase ^= 1u << buf;
      buf ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (a.ctas_k > 1) {
    // One tile per cluster, its sums in this CTA's tensor memory.  Each row's go to the CTA
    // that owns it: [source][layer][four tokens][row].
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (a.slots == 0) cluster_sync();   // every ring is free
    int4 *slots = reinterpret_cast<int4 *>(smem + a.slots);
    const int per_source = LAYERS * fours * owned;
    if (warp >= 2) {
      tc_fence_after();
      const int quarter = warp & 3, lrow = quarter * 32 + lane;
      const int owner = lrow / owned, mine = lrow % owned;
      const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t there = cluster_addr(slots + (size_t)crank * per_source + mine, owner);
      const uint32_t bar = cluster_addr(&sh.sums, owner);
      for (int c0 = 0; c0 < fours * 4; c0 += 16) {
#pragma unroll
        for (int l = 0; l < LAYERS; ++l) {
          float v[16];   // sums' bits
          tmem_ld_32x32b_x16(base + l * N + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const int four = c0 / 4 + i / 4;
            if (four >= fours) continue;
            const int at = (l * fours + four) * owned;
            const int4 s = make_int4(__float_as_int(v[i]), __float_as_int(v[i + 1]), __float_as_int(v[i + 2]),
                                     __float_as_int(v[i + 3]));
            if (owner == crank)
              slots[(size_t)crank * per_source + mine + at] = s;
            else
              push4(there + at * 16, bar, s.x, s.y, s.z, s.w);
          }
        }
      }
    }
    // what the results need, while the sums arrive: a thread keeps to one row
    const int64_t row = (int64_t)cta * a.rows + crank * owned + threadIdx.x % owned;   // SINGLE_THREADS % owned == 0
    const Row par = row_of<GATED>(a.p, row);
    float *xs = sh.xs[0];
    for (int c = threadIdx.x; c < fours * 4; c += SINGLE_THREADS)
      xs[c] = c < n ? __ldcg(a.p.x_scales + c) : 0.f;
    // (a CTA that gave up pushed its sums all the same, whatever they are)
    if ((a.p.give_up == GPTQ_GIVE_UP_SUMS && crank == 0) || !mbar_wait_bounded(&sh.sums, 0)) single_timeout(a.status, sh);
    __syncthreads();
    if (!*(volatile int *)&sh.abort) {
      Y *y = static_cast<Y *>(a.p.y) + row;
      for (int i = threadIdx.x; i < fours * owned && row < a.p.r; i += SINGLE_THREADS) {
        const int tok = i / owned * 4;
        const float4 scale = *reinterpret_cast<const float4 *>(xs + tok);
        int4 s[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= a.ctas_k) break;
#pragma unroll
          for (int l = 0; l < LAYERS; ++l) {
            const int4 v = slots[(size_t)k * per_source + l * fours * owned + i];
            s[l].x += v.x, s[l].y += v.y, s[l].z += v.z, s[l].w += v.w;
          }
        }
        const F2 lo = results<GATED, ACT, Y>(s[0].x, s[0].y, s[1].x, s[1].y, scale.x, scale.y, par);
        const F2 hi = results<GATED, ACT, Y>(s[0].z, s[0].w, s[1].z, s[1].w, scale.z, scale.w, par);
        const float f[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (tok + q < n) y[(int64_t)(tok + q) * a.p.r] = to_result<Y>(f[q]);
      }
    }
    // No CTA's memory goes while sums may be on their way to it: one that gave up stays until
    // they have landed.  Every CTA sends its own, after SETTLE waits that ran out at most.
    // (A cluster barrier in every launch's way out cost 0.1 to 0.5 us.)
    if (*(volatile int *)&sh.abort)
      for (int i = 0; i < SETTLE && !mbar_wait_bounded(&sh.sums, 0); ++i) {
      }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, a.columns);
  }
}

template <bool GATED, int ACT, typename Y>
int launch_typed(const SingleArgs &a, const CUtensorMap &tx, const CUtensorMap &tw, const CUtensorMap &tu,
                 unsigned ctas, size_t bytes, cudaStream_t st) {
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(int8_single_kernel<GATED, ACT, Y>, SINGLE_SMEM + 1024, attr)) return rc;
  return launch_after(int8_single_kernel<GATED, ACT, Y>, ctas, SINGLE_THREADS, bytes + 1024, (unsigned)a.ctas_k, st, tx, tw, tu, a);
}

template <bool GATED, int ACT, typename... A>
int launch_act(const SingleArgs &a, A &&...rest) {
  switch (a.p.ytype) {
    case GPTQ_F16: return launch_typed<GATED, ACT, __half>(a, rest...);
    case GPTQ_BF16: return launch_typed<GATED, ACT, __nv_bfloat16>(a, rest...);
    default: return launch_typed<GATED, ACT, float>(a, rest...);
  }
}

}  // namespace

namespace {

// Rows of W per tile, CTAs along k, and whether two CTAs share an SM, for up to 64 tokens,
// which are bound by the copies of W: all SMs copying, with as few steps as it takes to
// meet.  Measured (us; tiles of 128 rows split over 2, 4, 8 CTAs, and unsplit tiles that make
// 148 or 296; the split ones take 0.2 to 0.3 less since there is one tile of tokens alone):
//   1 token, 4096 x 4096     8.7, 7.7, 7.2   7.9, 10.4   (32 tiles)
//   24 tokens, 4096 x 11008  15.9, 12.5, 11.6   15.8, 21.5
//   16 tokens, 8192 x 8192   15.1, 14.4, 17.6   16.6, 15.9   (64 tiles)
//   1 token, 11008 x 4096    14.1, 17.5, 20.1   11.7, 10.9   (86 tiles)
//   1 token, 12288 x 49152   97.7, 102.8, 99.3   100.1, 91.9
//   64 tokens, 11008 x 4096  24.0, 26.4, 26.0   12.4, 14.1
//   gated, 24 tokens, 4096 x 4096  13.1, 10.4, 12.2
//   gated, 16 tokens, 5120 x 5120  15.4, 15.5, 19.5   15.4, 19.7   (40 tiles)
//   gated, 1 token, 11008 x 4096   22.9, 25.9, 28.5   16.6, 16.8
//   16 tokens, 512 x 512     4.0, 3.9, 3.9   3.3, 3.3   (2.7 with stages no deeper than d)
// Gated tiles have twice the bytes, so that one CTA fills an SM's share.

// Clusters of c CTAs that run at once, one or two CTAs to an SM: the SMs of a cluster lie in
// one part of the chip, whose last few stay empty, so fewer than the SMs would hold; one more
// is a second round.  Measured: 15 of 8, 33 with two to an SM, 33 of 4 (10 tokens,
// 4224 x 8192 9.2 us as 33 x 8 CTAs, 4352 x 8192 15.1 as 34 x 8; gated, 10 tokens, 2048 x 8192
// 17.0 as 16 x 8, 12.1 as 16 x 4).
int clusters_at_once(int c, int per_sm, int sms) {
  if (c == 8) return sms * (per_sm == 2 ? 33 : 15) / 148;
  if (c == 4) return sms * 33 / 148 * per_sm;
  return sms / 2 * per_sm;
}

struct Shape {
  int rows, ctas_k;
  bool shared;
};
Shape shape_for(int64_t r, int slabs, int N, bool gated, int sms) {
  const int64_t tiles = (r + ROWS - 1) / ROWS;
  if (slabs >= 8)
    for (int c = 8; c >= (gated ? 2 : 4); c /= 2) {
      if (slabs < 2 * c) continue;
      if (tiles <= clusters_at_once(c, 1, sms)) return Shape{ROWS, c, false};
      if (!gated && tiles <= clusters_at_once(c, 2, sms)) return Shape{ROWS, c, true};
    }
  const int64_t parts = gated || N > 48 ? sms : 2 * sms;
  const int64_t rows = (r + 8 * parts - 1) / (8 * parts) * 8;
  const bool shared = !gated && N <= 48 && (r + rows - 1) / rows > sms;
  return Shape{rows < ROWS ? (int)rows : ROWS, 1, shared};
}

}  // namespace

int int8_split(const Int8Args &p, int sms) {   // the widest split that finds room, or 1
  const int64_t tiles = (p.r + ROWS - 1) / ROWS;
  const int slabs = (p.d + SLAB - 1) / SLAB, layers = p.gated ? 2 : 1;
  for (int c = 8; c >= 2; c /= 2)
    if (tiles <= clusters_at_once(c, 1, sms) && slabs >= 2 * c && p.n <= TOKENS / layers) return c;
  return 1;
}

namespace {

// What a launch takes but its tensor maps and the status word.
int single_plan(const Int8Args &p, int sms, SingleArgs &a, unsigned &ctas, size_t &bytes) {
  const int layers = p.gated ? 2 : 1, slabs = (p.d + SLAB - 1) / SLAB;
  const int split = p.n > FEW_TOKENS ? int8_split(p, sms) : 0;
  if (split == 1) return GPTQ_ERR_INVALID_ARG;   // (more than 64 tokens: only with k split)
  a.p = p;
  a.N = (int)((p.n + 15) / 16 * 16);
  const Shape shape = split ? Shape{ROWS, split, false} : shape_for(p.r, slabs, a.N, p.gated, sms);
  a.rows = shape.rows;
  a.ctas_k = shape.ctas_k;
  const int64_t tiles = (p.r + a.rows - 1) / a.rows;
  if (tiles > INT32_MAX / 8) return GPTQ_ERR_INVALID_ARG;
  a.tiles = (int)tiles;
  // stages of 16 KB of W, at least four of them
  const size_t room = shape.shared ? SHARED_SM : SINGLE_SMEM, slab = (size_t)(layers * a.rows + a.N) * SLAB;
  a.deep = ROWS / a.rows;
  while (a.deep > 1 && a.deep * slab * 4 > room) --a.deep;
  const int steps = (slabs + a.deep - 1) / a.deep;
  a.deep = (slabs + steps - 1) / steps;   // slabs past d would be loaded and multiplied as zeros
  const size_t stage = slab * a.deep;
  // a tile of fewer rows reads up to 128 rows of the last stage
  const size_t pad = (size_t)(ROWS - a.rows) * SLAB;
  // split k: the sums of the rows that a CTA owns meet beside the ring, or in it
  const size_t meet = a.ctas_k > 1 ? (size_t)layers * a.N * a.rows * 4 : 0;
  const size_t apart = a.N * layers <= 32 ? meet : 0;
  const size_t fit = (room - apart - pad) / stage;
  if (fit < 2 || meet > SINGLE_SMEM) return GPTQ_ERR_INVALID_ARG;   // (never: 64 KB a stage at most)
  a.stages = fit > STAGES ? STAGES : (int)fit;
  const int64_t work = a.ctas_k > 1 ? (steps + a.ctas_k - 1) / a.ctas_k : (tiles + sms - 1) / sms * steps;
  if (a.stages > work) a.stages = (int)work;   // no more than there are steps
  bytes = a.stages * stage;
  a.slots = apart ? (int)bytes : 0;
  bytes += apart;
  if (bytes < meet) bytes = meet;
  bytes += pad;
  a.columns = 32;
  while (a.columns < (uint32_t)((a.ctas_k > 1 ? 1 : 2) * layers * a.N)) a.columns *= 2;
  const size_t least = a.columns > 128 ? WIDE_SMEM : LEAST_SMEM;
  if (bytes < least) bytes = least;
  const int64_t most = shape.shared ? 2 * sms : sms;
  ctas = (unsigned)(a.ctas_k > 1 ? tiles * a.ctas_k : (tiles < most ? tiles : most));
  return GPTQ_OK;
}

}  // namespace

int int8_single_plan(const Int8Args &p, int sms, Int8Plan &plan) {
  SingleArgs a{};
  unsigned ctas;
  size_t bytes;
  if (const int rc = single_plan(p, sms, a, ctas, bytes)) return rc;
  plan = Int8Plan{false, (int)ctas, a.ctas_k, a.N, a.rows, a.stages, (int)a.columns, bytes + 1024 + sizeof(SingleShared)};
  return GPTQ_OK;
}

int launch_int8_single(const Int8Args &p, cudaStream_t st) {
  SingleArgs a{};
  unsigned ctas;
  size_t bytes;
  if (const int rc = single_plan(p, num_sms(), a, ctas, bytes)) return rc;
  a.status = device_status_word();
  if (!a.status) return GPTQ_ERR_CUDA;
  CUtensorMap tx, tw, tu;
  if (const int rc = int8_map(&tx, p.x, p.n, p.d, a.N)) return rc;
  if (const int rc = int8_map(&tw, p.w[0], p.r, p.d, a.rows)) return rc;
  tu = tw;
  if (p.gated)
    if (const int rc = int8_map(&tu, p.w[1], p.r, p.d, a.rows)) return rc;
  if (!p.gated) return launch_act<false, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, bytes, st);
  switch (p.activation) {
    case GPTQ_ACT_NONE: return launch_act<true, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, bytes, st);
    case GPTQ_ACT_RELU: return launch_act<true, GPTQ_ACT_RELU>(a, tx, tw, tu, ctas, bytes, st);
    case GPTQ_ACT_SILU: return launch_act<true, GPTQ_ACT_SILU>(a, tx, tw, tu, ctas, bytes, st);
    default: return launch_act<true, GPTQ_ACT_GELU>(a, tx, tw, tu, ctas, bytes, st);
  }
}

}  // namespace gptq
