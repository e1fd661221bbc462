// gptq_int8_linear and gptq_int8_gated, weights as the rows of the tensor-core product:
// any number of tokens, and the kernel for up to a few hundred of them.
//
//   y[t, i] = xs[t] ws[i] sum_j x[t, j] w[i, j] + bias[i]
//   gated:  y = act(the gate's) * (the up projection's)
//
// One CTA per tile of 128 rows of W and N <= 256 tokens; a gated tile has the 128
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
constexpr int TOKENS = 256;               // most tokens per tile (UMMA N)
constexpr int STAGES = 8;                 // at most
constexpr int SINGLE_THREADS = 32 * 6;
constexpr size_t SINGLE_SMEM = 208 * 1024;
constexpr size_t SHARED_SM = 108 * 1024;  // where two CTAs share an SM

struct SingleArgs {
  Int8Args p;
  int N;              // tokens per tile, a multiple of 16
  int nM, nN;         // tiles
  int ctas_k;         // CTAs of a cluster, along k
  int stages;
  uint32_t columns;   // of tensor memory
  int buffers;        // accumulators, 1 or 2
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
};

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

template <bool GATED, int ACT>
__device__ __forceinline__ float result(int s0, int s1, float xs, const Row &r) {
  const float v = scaled_sum(s0, xs, r.scale[0], r.bias[0]);
  if constexpr (!GATED) return v;
  return activate<ACT>(v) * scaled_sum(s1, xs, r.scale[1], r.bias[1]);
}

// 16 tokens of an accumulator's 32 rows to y; a lane is a row.  16-bit results go
// through shared memory and out 16 bytes, eight rows of a token, per lane, where y's
// rows allow it.
template <typename Y>
__device__ __forceinline__ void write_tokens(const float (&v)[16], int count, int64_t t0, int64_t row,
                                             const Int8Args &p, uint16_t *stage, int lane) {
  Y *y = static_cast<Y *>(p.y);
  bool wide = false;
  if constexpr (sizeof(Y) == 2)
    wide = p.r % 8 == 0 && row - lane + 32 <= p.r && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
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
        if (tok < count)
          *reinterpret_cast<uint4 *>(y + (t0 + tok) * p.r + (row - lane) + (lane & 3) * 8) = o;
      }
    }
  } else if (row < p.r) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < count) y[(t0 + i) * p.r + row] = to_result<Y>(v[i]);
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
  constexpr int W_BYTES = LAYERS * ROWS * SLAB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = a.N, stage_bytes = W_BYTES + N * SLAB;
  const int crank = blockIdx.x % a.ctas_k, ctas = gridDim.x / a.ctas_k, cta = blockIdx.x / a.ctas_k;
  const int tiles = a.nM * a.nN;
  const int slabs = (a.p.d + SLAB - 1) / SLAB;
  const int k0 = (int)((int64_t)slabs * crank / a.ctas_k);
  const int k1 = (int)((int64_t)slabs * (crank + 1) / a.ctas_k);
  const uint32_t acc_columns = LAYERS * N;

  // the tokens of a split tile that exist, in fours
  const int fours = a.ctas_k > 1 ? (int)((min((int64_t)N, a.p.n - (int64_t)(cta / a.nM) * N) + 3) / 4) : 0;
  const int owned = ROWS / a.ctas_k;   // rows
  auto load = [&](int t, int k, int stage) {
    mbar_arrive_expect_tx(&sh.full[stage], stage_bytes);
    uint8_t *dst = smem + (size_t)stage * stage_bytes;
    // columns from multiples of 128 bytes (past d, r and n: zeros)
    tma_load_2d(dst, &tmW, k * SLAB, t % a.nM * ROWS, &sh.full[stage]);
    if constexpr (GATED) tma_load_2d(dst + ROWS * SLAB, &tmU, k * SLAB, t % a.nM * ROWS, &sh.full[stage]);
    tma_load_2d(dst + W_BYTES, &tmX, k * SLAB, t / a.nM * N, &sh.full[stage]);
  };
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
    for (int k = k0; k < k1 && k < k0 + a.stages; ++k) {   // (into L2, whoever wrote them)
      prefetch_2d(&tmW, k * SLAB, cta % a.nM * ROWS);
      if constexpr (GATED) prefetch_2d(&tmU, k * SLAB, cta % a.nM * ROWS);
    }
    pdl_wait_then_release();
    for (; ahead < a.stages && k0 + ahead < k1; ++ahead) load(cta, k0 + ahead, ahead);
  } else {
    if (warp == 1) {
      tmem_alloc(&sh.tmem_base, a.columns);
      tmem_relinquish();
    }
    pdl_wait_then_release();
  }
  __syncwarp();
  if (a.ctas_k > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // barriers are there
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- W and x by TMA
    if (lane == 0) {
      int stage = ahead == a.stages ? 0 : ahead;
      uint32_t phase = ahead == a.stages ? 1 : 0, issued = (1u << ahead) - 1u, issued_par = 0;
      bool ok = true;
      for (int t = cta; t < tiles && ok; t += ctas) {
        for (int k = t == cta ? k0 + ahead : k0; k < k1; ++k) {
          ok = !*(volatile int *)&sh.abort && mbar_wait_bounded(&sh.empty[stage], phase ^ 1);
          if (!ok) {
            single_timeout(a.status, sh);
            break;
          }
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          load(t, k, stage);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) (void)mbar_wait_bounded(&sh.full[s], (issued_par >> s) & 1u);
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
          const uint64_t w = first + (uint64_t)(stage * stage_bytes >> 4), x = w + (W_BYTES >> 4);
          const uint32_t d0 = tm + buf * acc_columns;
#pragma unroll
          for (int q = 0; q < SLAB / 32; ++q) {
            umma_i8_ss(d0, w + q * 2, x + q * 2, idesc, k > k0 || q > 0);
            if constexpr (GATED)
              umma_i8_ss(d0 + N, w + (ROWS * SLAB >> 4) + q * 2, x + q * 2, idesc, k > k0 || q > 0);
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
      if (a.buffers == 2) buf ^= 1;
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
    const int quarter = warp & 3, lrow = quarter * 32 + lane;
    uint32_t buf = 0, cphase = 0;
    bool ok = true;
    for (int t = cta; t < tiles && ok; t += ctas) {
      const int64_t row = (int64_t)(t % a.nM) * ROWS + lrow, t0 = (int64_t)(t / a.nM) * N;
      const int count = (int)(a.p.n - t0 < N ? a.p.n - t0 : N);
      const Row par = row_of<GATED>(a.p, row);
      ok = mbar_wait_bounded(&sh.acc_full[buf], (cphase >> buf) & 1u);
      if (!ok && lane == 0) single_timeout(a.status, sh);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + buf * acc_columns;
      for (int c0 = 0; c0 < count; c0 += 16) {
        float s0[16], s1[16];   // sums' bits
        tmem_ld_32x32b_x16(base + c0, s0);
        if constexpr (GATED) tmem_ld_32x32b_x16(base + N + c0, s1);
        tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float xs = c0 + i < count ? __ldcg(a.p.x_scales + t0 + c0 + i) : 0.f;
          v[i] = result<GATED, ACT>(__float_as_int(s0[i]), GATED ? __float_as_int(s1[i]) : 0, xs, par);
        }
        write_tokens<Y>(v, count - c0, t0 + c0, row, a.p, sh.stage[quarter], lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
      cphase ^= 1u << buf;
      if (a.buffers == 2) buf ^= 1;
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
    // (a CTA that gave up pushed its sums all the same, whatever they are)
    if (!mbar_wait_bounded(&sh.sums, 0)) single_timeout(a.status, sh);
    __syncthreads();
    if (!*(volatile int *)&sh.abort) {
      const int64_t m0 = (int64_t)(cta % a.nM) * ROWS + crank * owned, t0 = (int64_t)(cta / a.nM) * N;
      Y *y = static_cast<Y *>(a.p.y);
      for (int i = threadIdx.x; i < fours * owned; i += SINGLE_THREADS) {
        const int64_t row = m0 + i % owned, tok = t0 + i / owned * 4;
        if (row >= a.p.r) continue;
        const Row par = row_of<GATED>(a.p, row);
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
        const int s0[4] = {s[0].x, s[0].y, s[0].z, s[0].w}, s1[4] = {s[1].x, s[1].y, s[1].z, s[1].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (tok + q < a.p.n)
            y[(tok + q) * a.p.r + row] =
                to_result<Y>(result<GATED, ACT>(s0[q], s1[q], __ldcg(a.p.x_scales + tok + q), par));
      }
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

int launch_int8_single(const Int8Args &p, cudaStream_t st) {
  SingleArgs a{};
  a.p = p;
  const int sms = num_sms(), layers = p.gated ? 2 : 1;
  const int slabs = (p.d + SLAB - 1) / SLAB;
  const int64_t nM = (p.r + ROWS - 1) / ROWS;
  // tokens in equal parts
  const int64_t parts = (p.n + TOKENS - 1) / TOKENS;
  a.N = (int)((p.n + parts * 16 - 1) / (parts * 16) * 16);
  const int64_t nN = (p.n + a.N - 1) / a.N;
  if (nM * nN > INT32_MAX / 8) return GPTQ_ERR_INVALID_ARG;
  a.nM = (int)nM;
  a.nN = (int)nN;
  const int64_t tiles = nM * nN;
  const bool shared = a.N <= 64;
  a.ctas_k = 1;
  for (int c = 2; c <= 8; c *= 2)
    if (tiles * c <= sms && slabs >= 2 * c) a.ctas_k = c;
  const size_t stage = (size_t)(layers * ROWS + a.N) * SLAB;
  const size_t meet = (size_t)layers * a.N * ROWS * 4;   // split k: the sums of the rows that a CTA owns
  if (meet > SINGLE_SMEM / stage * stage) a.ctas_k = 1;
  const size_t apart = a.ctas_k > 1 && a.N <= 32 ? meet : 0;
  const size_t fit = ((shared ? SHARED_SM : SINGLE_SMEM) - apart) / stage;
  a.stages = fit > STAGES ? STAGES : (int)fit;
  size_t bytes = a.stages * stage;
  a.slots = apart ? (int)bytes : 0;
  bytes += apart;
  if (a.ctas_k > 1 && bytes < meet) bytes = meet;
  a.buffers = a.ctas_k == 1 && 2 * layers * a.N <= (shared ? 256 : 512) ? 2 : 1;
  a.columns = 32;
  while (a.columns < (uint32_t)(a.buffers * layers * a.N)) a.columns *= 2;
  a.status = device_status_word();
  if (!a.status) return GPTQ_ERR_CUDA;
  CUtensorMap tx, tw, tu;
  if (const int rc = int8_map(&tx, p.x, p.n, p.d, a.N)) return rc;
  if (const int rc = int8_map(&tw, p.w[0], p.r, p.d, ROWS)) return rc;
  tu = tw;
  if (p.gated)
    if (const int rc = int8_map(&tu, p.w[1], p.r, p.d, ROWS)) return rc;
  const int64_t most = shared ? 2 * sms : sms;
  const unsigned ctas = (unsigned)(a.ctas_k > 1 ? tiles * a.ctas_k : (tiles < most ? tiles : most));
  if (!p.gated) return launch_act<false, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, bytes, st);
  switch (p.activation) {
    case GPTQ_ACT_NONE: return launch_act<true, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, bytes, st);
    case GPTQ_ACT_RELU: return launch_act<true, GPTQ_ACT_RELU>(a, tx, tw, tu, ctas, bytes, st);
    case GPTQ_ACT_SILU: return launch_act<true, GPTQ_ACT_SILU>(a, tx, tw, tu, ctas, bytes, st);
    default: return launch_act<true, GPTQ_ACT_GELU>(a, tx, tw, tu, ctas, bytes, st);
  }
}

}  // namespace gptq
