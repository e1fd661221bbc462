// gptq_int8_linear and gptq_int8_gated for many tokens: pairs of CTAs, tokens as the rows
// of the tensor-core product.
//
// A pair takes a tile of 256 tokens and N <= 256 rows of W with one MMA of both tensor
// cores (cta_group::2, M = 256): each CTA loads its own 128 tokens of x and half of W's
// rows, so a 128-column slab of a 256 x 256 tile costs each CTA 32 KB in the 512 clocks
// that its MMAs take, where a single CTA's tile of 128 x 256 loads 48 KB.  In a gated
// block one CTA loads N / 2 rows of the gate and the other the same rows of the up
// projection: the sums of both lie in the two halves of a token's columns of tensor
// memory, and the thread that owns the token writes their product alone.
// Two accumulators of 256 columns: eight warps of each CTA write one out, a thread a
// token, while the other fills.
#include "int8_linear.h"
#include "launch_after.h"

namespace gptq {
namespace {

constexpr int TOKENS = 128;               // per CTA of a pair
constexpr int SLAB = 128;                 // columns per stage
constexpr int ROWS = 256;                 // most rows of W per tile (UMMA N)
constexpr int STAGES = 10;                // at most
constexpr int X_BYTES = TOKENS * SLAB;
constexpr int OUT_WARPS = 8;
constexpr int PAIR_THREADS = 32 * (2 + OUT_WARPS);
constexpr size_t PAIR_SMEM = (size_t)6 * (X_BYTES + ROWS / 2 * SLAB);

struct PairArgs {
  Int8Args p;
  int N;              // rows of W per tile, of both layers together; a multiple of 32
  int nT, nR;         // tiles along the tokens and along the rows
  int stages;
  int *status;
};

struct PairShared {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) float scale[2][ROWS], bias[2][ROWS];   // of a tile's columns, by accumulator
  uint32_t stage[OUT_WARPS][32 * 17];                // results of 32 tokens on their way out, per warp
};

__device__ __forceinline__ void pair_timeout(int *status, PairShared &sh) {
  atomicCAS(status, 0, (int)GPTQ_ERR_TIMEOUT);
  *(volatile int *)&sh.abort = 1;
}

__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 16 results of one token to its row of y, all of them in y, whose rows are multiples of
// `align` bytes, 16 or 32.
template <typename Y>
__device__ __forceinline__ void write16(Y *y, const float (&v)[16], int align) {
  constexpr int WORDS = 16 * sizeof(Y) / 4;
  uint32_t o[WORDS];
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    if constexpr (sizeof(Y) == 2)
      o[i] = to_pair<Y>(v[2 * i], v[2 * i + 1]);
    else
      o[i] = __float_as_uint(v[i]);
  }
  if (align >= 32) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8) {
      const uint32_t w[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
      store32(reinterpret_cast<uint32_t *>(y) + i, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4)
      reinterpret_cast<uint4 *>(y)[i / 4] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
  }
}

// Results that a thread cannot write by vectors, y's rows not being multiples of 16 bytes or
// ending: through shared memory, [token][column], so that a store writes 64 bytes of a row
// and not a column of 32 rows.  393 tokens x 13021x736 12 us, one column at a time 67.
template <typename Y>
constexpr int STAGED = 64 / (int)sizeof(Y);   // columns
template <typename Y>
constexpr int STAGE_PITCH = STAGED<Y> + 1;
template <typename Y>
__device__ __forceinline__ void write_staged(Y *y, const Y *stage, int64_t r, int tokens, int columns, int lane) {
  __syncwarp();
  constexpr int EACH = 32 / STAGED<Y>;   // tokens per store
  const int c = lane % STAGED<Y>, t0 = lane / STAGED<Y>;
  const Y *src = stage + t0 * STAGE_PITCH<Y> + c;
  Y *dst = y + t0 * r + c;
  if (c < columns)
#pragma unroll 8
    for (int t = t0; t < tokens; t += EACH, src += EACH * STAGE_PITCH<Y>, dst += EACH * r) *dst = *src;
  __syncwarp();
}

template <bool GATED, int ACT, typename Y>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmU, const PairArgs a) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ PairShared sh;
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int half = a.N / 2, stage_bytes = X_BYTES + half * SLAB;
  const int per_tile = GATED ? half : a.N;          // rows of y's columns per tile
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int tiles = a.nT * a.nR;
  const int slabs = (a.p.d + SLAB - 1) / SLAB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], 2 * OUT_WARPS);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    if constexpr (GATED) prefetch_tmap(&tmU);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();   // both CTAs' barriers before either signals the other
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  pdl_wait_then_release();

  if (warp == 0) {
    // ---------------------------------------------------------------- x and W by TMA
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, full = false;   // full: every stage has been asked for
      const CUtensorMap *tm = GATED && rank ? &tmU : &tmW;
      const uint32_t ring = smem_u32(smem), bars = cluster_addr(&sh.full[0], 0);   // the issuing CTA's
      for (int t = pair; t < tiles && ok; t += pairs) {
        const int t0 = t % a.nT * (2 * TOKENS) + rank * TOKENS, r0 = t / a.nT * per_tile;
        const int row = GATED ? r0 : r0 + rank * half;
        for (int k = 0; k < slabs; ++k) {
          ok = wait_or_abort(&sh.empty[stage], phase ^ 1, &sh.abort);
          if (!ok) {
            pair_timeout(a.status, sh);
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[stage], 2 * stage_bytes);
          const uint32_t dst = ring + stage * stage_bytes, bar = bars + stage * 8;
          // columns from multiples of 128 bytes (past d, r and n: zeros)
          load_2d_pair(dst, &tmX, k * SLAB, t0, bar);
          load_2d_pair(dst + X_BYTES, tm, k * SLAB, row, bar);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
            full = true;
          }
        }
      }
      // the last load of every stage has landed (counted on the first CTA's barriers): stages
      // before `stage` in this phase, the others in the one before
      if (rank == 0)
        for (int s = 0; s < a.stages; ++s)
          if (full || s < stage) (void)mbar_wait_bounded(&sh.full[s], s < stage ? phase : phase ^ 1);
      // a second CTA whose loads the other may not have waited for: time to land
      if (rank == 1 && !ok)
        for (const unsigned long long t0 = global_ns(); global_ns() - t0 < 1000000;) {
        }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- the MMAs
    const uint32_t idesc = instr_desc_i8(2 * TOKENS, a.N);
    const uint64_t first = smem_desc(smem_u32(smem), 16, 1024, 2);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int stage = 0;
    uint32_t phase = 0, buf = 0, cphase = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      ok = mbar_wait_bounded(&sh.acc_empty[buf], ((cphase >> buf) & 1u) ^ 1u);
      for (int k = 0; k < slabs; ++k) {
        ok = ok && mbar_wait_bounded(&sh.full[stage], phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane()) {
          const uint64_t x = first + (uint64_t)(stage * stage_bytes >> 4), w = x + (X_BYTES >> 4);
#pragma unroll
          for (int q = 0; q < SLAB / 32; ++q)
            umma_i8_pair(tm + buf * ROWS, x + q * 2, w + q * 2, idesc, k > 0 || q > 0);
          umma_commit_both(&sh.empty[stage]);
          if (k == slabs - 1) umma_commit_both(&sh.acc_full[buf]);
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
    if (!ok && lane == 0) pair_timeout(a.status, sh);
    __syncwarp();
    if (elect_lane()) {
      umma_commit_pair_local(&sh.drain);
      (void)mbar_wait_bounded(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- results
    const int quarter = warp & 3, side = (warp - 2) >> 2;
    const int c_begin = side * (per_tile / 2 / 16 * 16), c_end = side ? per_tile : per_tile / 2 / 16 * 16;
    const int64_t pitch = a.p.r * (int64_t)sizeof(Y);
    // the largest power of two, up to 32, that all rows of y and 16 columns are multiples of
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.p.y) | (uintptr_t)pitch;
    const int align = base % 32 == 0 ? 32 : base % 16 == 0 ? 16 : 1;
    uint32_t buf = 0, cphase = 0;
    bool ok = true;
    // (a warp that gave up still walks the tiles: the others wait for it at their barrier)
    for (int t = pair; t < tiles; t += pairs) {
      const int64_t tok = (int64_t)(t % a.nT) * (2 * TOKENS) + rank * TOKENS + quarter * 32 + lane;
      const int64_t r0 = (int64_t)(t / a.nT) * per_tile;
      // the columns' scales and biases, while the accumulator fills
      for (int c = (warp - 2) * 32 + lane; c < a.N; c += 32 * OUT_WARPS) {
        const bool second = GATED && c >= half;
        const float *scales = second ? a.p.w_scales[1] : a.p.w_scales[0];
        const void *bias = second ? a.p.bias[1] : a.p.bias[0];
        const int64_t row = r0 + (second ? c - half : c);
        const bool live = row < a.p.r;
        sh.scale[buf][c] = live ? __ldcg(scales + row) : 0.f;
        sh.bias[buf][c] = live && bias ? load_typed(bias, a.p.ytype, row) : 0.f;
      }
      const float xs = tok < a.p.n ? __ldcg(a.p.x_scales + tok) : 0.f;
      // (the other accumulator's parameters are still being read by slower warps, this one's
      // were read before the barrier of the tile between)
      asm volatile("bar.sync 1, %0;" ::"n"(32 * OUT_WARPS) : "memory");
      if (gives_up(a.p, warp, lane, t, pairs, tiles)) ok = false;
      ok = ok && mbar_wait_bounded(&sh.acc_full[buf], (cphase >> buf) & 1u);
      ok = __all_sync(0xffffffffu, ok);   // (one lane's wait may run out alone)
      if (!ok && lane == 0) pair_timeout(a.status, sh);
      if (ok) {
        tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + buf * ROWS;
        Y *y = static_cast<Y *>(a.p.y) + tok * a.p.r + r0;
        // (the same for the whole warp)
        const bool vectors = align >= 16 && r0 + per_tile <= a.p.r;
        const int64_t tokens = a.p.n - (tok - lane);
        Y *stage = reinterpret_cast<Y *>(sh.stage[warp - 2]);
        for (int c = c_begin; c < c_end; c += 16) {
          float s0[16], s1[16], v[16];   // sums' bits
          tmem_ld_32x32b_x16(acc + c, s0);
          if constexpr (GATED) tmem_ld_32x32b_x16(acc + half + c, s1);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = scaled_sum(__float_as_int(s0[i]), xs, sh.scale[buf][c + i], sh.bias[buf][c + i]);
          if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const int at = half + c + i;
              const F2 r = gated_pair<ACT, Y>(
                  F2{v[i], v[i + 1]},
                  F2{scaled_sum(__float_as_int(s1[i]), xs, sh.scale[buf][at], sh.bias[buf][at]),
                     scaled_sum(__float_as_int(s1[i + 1]), xs, sh.scale[buf][at + 1], sh.bias[buf][at + 1])});
              v[i] = r.x;
              v[i + 1] = r.y;
            }
          }
          if (vectors) {
            if (tok < a.p.n) write16<Y>(y + c, v, align);
          } else {
            const int at = (c - c_begin) % STAGED<Y>;
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[lane * STAGE_PITCH<Y> + at + i] = to_result<Y>(v[i]);
            if (at + 16 == STAGED<Y> || c + 16 >= c_end) {
              const int64_t left = a.p.r - r0 - (c - at);
              write_staged<Y>(y - lane * a.p.r + c - at, stage, a.p.r, (int)(tokens < 32 ? tokens : 32),
                              (int)(left < at + 16 ? left : at + 16), lane);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(&sh.acc_empty[buf], 0));
      }
      cphase ^= 1u << buf;
      buf ^= 1;
    }
  }

  __syncthreads();
  tc_fence_before();
  __syncwarp();
  cluster_sync();   // neither CTA's memory goes while the other may touch it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool GATED, int ACT, typename Y>
int launch_typed(const PairArgs &a, const CUtensorMap &tx, const CUtensorMap &tw, const CUtensorMap &tu,
                 unsigned ctas, cudaStream_t st) {
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(int8_pair_kernel<GATED, ACT, Y>, PAIR_SMEM + 1024, attr)) return rc;
  return launch_after(int8_pair_kernel<GATED, ACT, Y>, ctas, PAIR_THREADS, PAIR_SMEM + 1024, 2, st, tx, tw, tu, a);
}

template <bool GATED, int ACT, typename... A>
int launch_act(const PairArgs &a, A &&...rest) {
  switch (a.p.ytype) {
    case GPTQ_F16: return launch_typed<GATED, ACT, __half>(a, rest...);
    case GPTQ_BF16: return launch_typed<GATED, ACT, __nv_bfloat16>(a, rest...);
    default: return launch_typed<GATED, ACT, float>(a, rest...);
  }
}

}  // namespace

// Rows of W per tile, and what it takes (us).  A slab of a tile takes its MMAs, 0.32 us for
// 256 rows, but below 100 rows the copy of x bounds it.  Measured (us, N = 64, 128, 160, 256):
// 128 tokens, 4096 x 4096 10.2, 10.3, 10.9, 14.1; 64 tokens, 11008 x 4096 22.5, 16.9, 12.0,
// 14.6; 1000 tokens, 11008 x 4096 69, 39, 35.1, 34.3; 4096 tokens, 4096 x 11008 244, 135, 125,
// 115; gated, 333 tokens, 11008 x 4096 68, 39, 35.2, 34.7 (224: 33.9).
static double pair_rows(const Int8Args &p, int pairs, int *rows) {
  const int64_t nT = (p.n + 2 * TOKENS - 1) / (2 * TOKENS), slabs = (p.d + SLAB - 1) / SLAB;
  double best = 1e30;
  for (int N = ROWS; N >= 64; N -= 32) {
    const int64_t per_tile = p.gated ? N / 2 : N, tiles = nT * ((p.r + per_tile - 1) / per_tile);
    const double slab = 0.115 + 0.0008 * N;
    const double us = (double)((tiles + pairs - 1) / pairs * slabs) * (slab < 0.195 ? 0.195 : slab) + 4.2 + 0.004 * N;
    if (us < best) best = us, *rows = N;
  }
  return best;
}

bool int8_pairs_faster(const Int8Args &p, int sms) {
  const int split = int8_split(p, sms);
  if (split == 1) return true;
  // single CTAs that split k: 100 GB/s a CTA, and their sums' way (128 tokens, 4096 x 11008
  // 16.4 us, pairs 20.4; 256 tokens 21.5, 21.0; 128 tokens, 4096 x 4096 11.5, 10.2; 223
  // tokens, 645 x 27424 20.0 over 8 CTAs, 29.1 over 4)
  const int64_t slabs = (p.d + SLAB - 1) / SLAB, layers = p.gated ? 2 : 1;
  const double bytes = (double)((slabs + split - 1) / split) * (double)((layers * 128 + p.n) * SLAB);
  int rows;
  return pair_rows(p, sms / 2, &rows) <= 7.0 + 0.0156 * layers * p.n + bytes * 1e-5;
}

static int pair_plan(const Int8Args &p, int sms, PairArgs &a, unsigned &ctas) {
  a.p = p;
  const int pairs = sms / 2;
  (void)pair_rows(p, pairs, &a.N);
  const int per_tile = p.gated ? a.N / 2 : a.N;
  a.stages = (int)(PAIR_SMEM / (X_BYTES + a.N / 2 * SLAB));
  if (a.stages > STAGES) a.stages = STAGES;
  const int64_t nT = (p.n + 2 * TOKENS - 1) / (2 * TOKENS), nR = (p.r + per_tile - 1) / per_tile;
  if (nT * nR > INT32_MAX / 8) return GPTQ_ERR_INVALID_ARG;
  a.nT = (int)nT;
  a.nR = (int)nR;
  ctas = 2 * (unsigned)(nT * nR < pairs ? nT * nR : pairs);
  return GPTQ_OK;
}

int int8_pair_plan(const Int8Args &p, int sms, Int8Plan &plan) {
  PairArgs a{};
  unsigned ctas;
  if (const int rc = pair_plan(p, sms, a, ctas)) return rc;
  plan = Int8Plan{true, (int)ctas, 2, 2 * TOKENS, p.gated ? a.N / 2 : a.N, a.stages, 512,
                  PAIR_SMEM + 1024 + sizeof(PairShared)};
  return GPTQ_OK;
}

int launch_int8_pair(const Int8Args &p, cudaStream_t st) {
  PairArgs a{};
  unsigned ctas;
  if (const int rc = pair_plan(p, num_sms(), a, ctas)) return rc;
  a.status = device_status_word();
  if (!a.status) return GPTQ_ERR_CUDA;
  CUtensorMap tx, tw, tu;
  if (const int rc = int8_map(&tx, p.x, p.n, p.d, TOKENS)) return rc;
  if (const int rc = int8_map(&tw, p.w[0], p.r, p.d, a.N / 2)) return rc;
  tu = tw;
  if (p.gated)
    if (const int rc = int8_map(&tu, p.w[1], p.r, p.d, a.N / 2)) return rc;
  if (!p.gated) return launch_act<false, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, st);
  switch (p.activation) {
    case GPTQ_ACT_NONE: return launch_act<true, GPTQ_ACT_NONE>(a, tx, tw, tu, ctas, st);
    case GPTQ_ACT_RELU: return launch_act<true, GPTQ_ACT_RELU>(a, tx, tw, tu, ctas, st);
    case GPTQ_ACT_SILU: return launch_act<true, GPTQ_ACT_SILU>(a, tx, tw, tu, ctas, st);
    default: return launch_act<true, GPTQ_ACT_GELU>(a, tx, tw, tu, ctas, st);
  }
}

}  // namespace gptq
