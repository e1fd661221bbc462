// gptq_regroup: the columns of a packed act-order layer sorted by group.
//
// Source: "一文读懂GPTQ" §三 -- desc_act quantises the columns in another
// order than theirs, so the columns of one group lie scattered over the row
// (g_idx).  With perm the stable order of the columns by g_idx, column j of
// the result is column perm[j], and position j belongs to group j / group.
//
// Two kernels.  The order: one warp per group reads g_idx 128 entries at a time
// and places the columns of its group by ballot, in order; a slot that stays
// empty (a group with too few columns) is marked -1, so perm holds a -1 if and
// only if some group has another number of columns than `group`.
//
// The rows, r*d*bits/8 bytes in and out: a CTA takes eight rows (four of 8-bit
// codes) and transposes them so that one shared-memory word holds a column's
// codes of all its rows, a nibble (byte) each.  Moving a column is then one
// random 4-byte read for eight codes instead of eight byte reads; reading codes
// one by one took 490 us where this takes about 10 (8192 x 8192, 3 bits).
// Codes of 2 and 3 bits travel as nibbles.  Rows too long for that (d > 49152)
// go through bytes in shared memory, one row at a time.
#include "gptq_internal.h"
#include "pack_bits.cuh"
#include "unpack_bits.cuh"

namespace gptq {
namespace {

constexpr int ORDER_WARPS = 8;
constexpr int ROW_THREADS = 256;

__global__ void __launch_bounds__(32 * ORDER_WARPS)
    group_order_kernel(const int32_t *__restrict__ g_idx, int d, int group, int G,
                       int32_t *__restrict__ perm) {
  extern __shared__ __align__(16) uint16_t groups[];   // g_idx, 0xFFFF for entries outside [0, G)
  for (int c = threadIdx.x; c < d; c += 32 * ORDER_WARPS) {
    const int v = __ldg(g_idx + c);
    groups[c] = v >= 0 && v < G ? (uint16_t)v : (uint16_t)0xFFFFu;   // G <= 2048
  }
  __syncthreads();
  const int g = blockIdx.x * ORDER_WARPS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (g >= G) return;
  int32_t *slots = perm + (int64_t)g * group;
  int found = 0;
#pragma unroll 2
  for (int c0 = 0; c0 < d; c0 += 128) {   // d % 32 == 0
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c0 + 32 * k < d ? groups[c0 + 32 * k + lane] : 0xFFFF;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool mine = v[k] == g;
      const uint32_t hit = __ballot_sync(0xffffffffu, mine);
      const int at = found + __popc(hit & ((1u << lane) - 1u));
      if (mine && at < group) slots[at] = c0 + 32 * k + lane;
      found += __popc(hit);
    }
  }
  for (int at = found + lane; at < group; at += 32) slots[at] = -1;
}

// perm[0] < 0 if any entry is: what the host reads.
__device__ void report_order(int32_t *perm, int d) {
  int bad = 0;
  for (int j = threadIdx.x; j < d; j += blockDim.x) bad |= perm[j] < 0;
  if (__syncthreads_or(bad) && threadIdx.x == 0) perm[0] = -1;
}

// ---- eight codes of a row as the nibbles of a word, low first

__device__ __forceinline__ uint32_t nibbles_of_3(uint32_t v) {   // 24 bits
  v = (v & 0x00000FFFu) | ((v << 4) & 0x0FFF0000u);
  v = (v & 0x003F003Fu) | ((v << 2) & 0x3F003F00u);
  return (v & 0x07070707u) | ((v << 1) & 0x70707070u);
}
__device__ __forceinline__ uint32_t threes_of_nibbles(uint32_t v) {
  v = (v & 0x07070707u) | ((v >> 1) & 0x38383838u);
  v = (v & 0x003F003Fu) | ((v >> 2) & 0x0FC00FC0u);
  return (v & 0x00000FFFu) | ((v >> 4) & 0x00FFF000u);
}
__device__ __forceinline__ uint32_t nibbles_of_2(uint32_t v) {   // 16 bits
  v = (v | (v << 8)) & 0x00FF00FFu;
  v = (v | (v << 4)) & 0x0F0F0F0Fu;
  return (v | (v << 2)) & 0x33333333u;
}
__device__ __forceinline__ uint32_t twos_of_nibbles(uint32_t v) {
  v = (v | (v >> 2)) & 0x0F0F0F0Fu;
  v = (v | (v >> 4)) & 0x00FF00FFu;
  return (v | (v >> 8)) & 0x0000FFFFu;
}

// Words of BITS-bit codes <-> words of nibbles (8-bit codes: bytes), one unit
// of a row.
template <int BITS>
struct Unit {
  static constexpr int COLS = BITS == 8 ? 4 : BITS == 4 ? 8 : BITS == 2 ? 16 : 32;
  static constexpr int ROWS = BITS == 8 ? 4 : 8;       // rows in a column's word
  static constexpr int IN = COLS * BITS / 32;          // packed words
  static constexpr int OUT = COLS / ROWS;              // words of nibbles or bytes
  static __device__ __forceinline__ void widen(const uint32_t (&w)[IN], uint32_t (&o)[OUT]) {
    if constexpr (BITS == 8 || BITS == 4) o[0] = w[0];
    if constexpr (BITS == 2) o[0] = nibbles_of_2(w[0] & 0xFFFFu), o[1] = nibbles_of_2(w[0] >> 16);
    if constexpr (BITS == 3) {
      o[0] = nibbles_of_3(w[0] & 0xFFFFFFu);
      o[1] = nibbles_of_3(__funnelshift_r(w[0], w[1], 24) & 0xFFFFFFu);
      o[2] = nibbles_of_3(__funnelshift_r(w[1], w[2], 16) & 0xFFFFFFu);
      o[3] = nibbles_of_3(w[2] >> 8);
    }
  }
  static __device__ __forceinline__ void narrow(const uint32_t (&o)[OUT], uint32_t (&w)[IN]) {
    if constexpr (BITS == 8 || BITS == 4) w[0] = o[0];
    if constexpr (BITS == 2) w[0] = twos_of_nibbles(o[0]) | twos_of_nibbles(o[1]) << 16;
    if constexpr (BITS == 3) {
      const uint32_t a = threes_of_nibbles(o[0]), b = threes_of_nibbles(o[1]);
      const uint32_t c = threes_of_nibbles(o[2]), e = threes_of_nibbles(o[3]);
      w[0] = a | b << 24;
      w[1] = b >> 8 | c << 16;
      w[2] = c >> 16 | e << 8;
    }
  }
};

// a[i] element j <-> a[j] element i: 8 x 8 nibbles, or 4 x 4 bytes.
template <int R>
__device__ __forceinline__ void transpose(uint32_t (&a)[R]) {
#pragma unroll
  for (int s = R / 2; s >= (R == 8 ? 2 : 1); s /= 2) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i & s) continue;
      const uint32_t x = a[i], y = a[i + s];
      const bool halves = s == R / 2;
      a[i] = __byte_perm(x, y, halves ? 0x5410 : 0x6240);
      a[i + s] = __byte_perm(x, y, halves ? 0x7632 : 0x7351);
    }
  }
  if constexpr (R == 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint32_t x = a[i], y = a[i + 1];
      a[i] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
      a[i + 1] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
    }
  }
}

// Word of column c: 16-byte chunks exchanged within 128 bytes, so that threads
// that write 32 columns apart use different banks.
__device__ __forceinline__ int place(int c) { return c ^ ((c >> 5 & 7) << 2); }

// STAGED: the order in shared memory too (2 bytes per column, as places), read
// from global memory once in whole lines.
template <int BITS, bool STAGED>
__global__ void __launch_bounds__(ROW_THREADS)
    regroup_rows_kernel(const uint32_t *__restrict__ qweight, int32_t *perm, int64_t r, int d,
                        uint32_t *__restrict__ out) {
  using U = Unit<BITS>;
  extern __shared__ __align__(16) uint32_t columns[];   // [d]: a column's codes of the CTA's rows
  if (blockIdx.x == gridDim.x - 1) {
    report_order(perm, d);
    return;
  }
  const int64_t wpr = (int64_t)(d / 32) * BITS;
  const int units = d / U::COLS;
  const int64_t row0 = (int64_t)blockIdx.x * U::ROWS;
  const int rows = (int)min((int64_t)U::ROWS, r - row0);
  uint16_t *order = reinterpret_cast<uint16_t *>(columns + d);
  if constexpr (STAGED) {
    for (int j = threadIdx.x; j < d; j += ROW_THREADS) {
      const int from = *(volatile const int32_t *)(perm + j);
      order[j] = (uint16_t)place(from < 0 ? 0 : from);
    }
  }
  for (int u = threadIdx.x; u < units; u += ROW_THREADS) {
    uint32_t n[U::ROWS][U::OUT];
#pragma unroll
    for (int i = 0; i < U::ROWS; ++i) {
      uint32_t w[U::IN];
#pragma unroll
      for (int k = 0; k < U::IN; ++k)
        w[k] = i < rows ? __ldg(qweight + (row0 + i) * wpr + (int64_t)u * U::IN + k) : 0u;
      U::widen(w, n[i]);
    }
#pragma unroll
    for (int k = 0; k < U::OUT; ++k) {
      uint32_t a[U::ROWS];
#pragma unroll
      for (int i = 0; i < U::ROWS; ++i) a[i] = n[i][k];
      transpose<U::ROWS>(a);
#pragma unroll
      for (int i = 0; i < U::ROWS; i += 4)
        *reinterpret_cast<uint4 *>(columns + place(u * U::COLS + k * U::ROWS + i)) =
            make_uint4(a[i], a[i + 1], a[i + 2], a[i + 3]);
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < units; u += ROW_THREADS) {
    uint32_t n[U::ROWS][U::OUT];
#pragma unroll
    for (int k = 0; k < U::OUT; ++k) {
      uint32_t a[U::ROWS];
#pragma unroll
      for (int i = 0; i < U::ROWS; ++i) {
        const int j = u * U::COLS + k * U::ROWS + i;
        if constexpr (STAGED) {
          a[i] = columns[order[j]];
        } else {
          const int from = *(volatile const int32_t *)(perm + j);
          a[i] = columns[place(from < 0 ? 0 : from)];
        }
      }
      transpose<U::ROWS>(a);
#pragma unroll
      for (int i = 0; i < U::ROWS; ++i) n[i][k] = a[i];
    }
#pragma unroll
    for (int i = 0; i < U::ROWS; ++i) {
      uint32_t w[U::IN];
      U::narrow(n[i], w);
      if (i < rows)
#pragma unroll
        for (int k = 0; k < U::IN; ++k) out[(row0 + i) * wpr + (int64_t)u * U::IN + k] = w[k];
    }
  }
}

template <int BITS>
__global__ void __launch_bounds__(ROW_THREADS)
    regroup_kernel(const uint32_t *__restrict__ qweight, int32_t *perm, int64_t r, int d,
                   uint32_t *__restrict__ out) {
  extern __shared__ __align__(16) uint8_t row_codes[];   // [d]
  const int nchunk = d / 32;
  if (blockIdx.x == gridDim.x - 1) {
    report_order(perm, d);
    return;
  }
  for (int64_t row = blockIdx.x; row < r; row += gridDim.x - 1) {
    const uint32_t *src = qweight + row * nchunk * BITS;
    uint32_t *dst = out + row * nchunk * BITS;
    __syncthreads();   // the previous row's gathers are done
    for (int k = threadIdx.x; k < nchunk; k += ROW_THREADS) {
      uint32_t w[BITS];
#pragma unroll
      for (int t = 0; t < BITS; ++t) w[t] = __ldg(src + (int64_t)k * BITS + t);
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        b[i] = code_at<BITS>(w, 4 * i) | code_at<BITS>(w, 4 * i + 1) << 8 |
               code_at<BITS>(w, 4 * i + 2) << 16 | code_at<BITS>(w, 4 * i + 3) << 24;
      uint4 *p = reinterpret_cast<uint4 *>(row_codes + (size_t)k * 32);
      p[0] = make_uint4(b[0], b[1], b[2], b[3]);
      p[1] = make_uint4(b[4], b[5], b[6], b[7]);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < nchunk; k += ROW_THREADS) {
      uint32_t c[32], w[BITS];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int from = *(volatile const int32_t *)(perm + k * 32 + j);
        c[j] = row_codes[from < 0 ? 0 : from];
      }
      pack32<BITS>(c, w);
#pragma unroll
      for (int t = 0; t < BITS; ++t) dst[(int64_t)k * BITS + t] = w[t];
    }
  }
}

// Columns whose words fit shared memory, and with their order.
constexpr int LONGEST = 49152, LONGEST_STAGED = 32768;

template <int BITS, bool STAGED>
int launch_rows(const uint32_t *q, int32_t *perm, int64_t r, int d, uint32_t *out, cudaStream_t st) {
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(regroup_rows_kernel<BITS, STAGED>, 192 * 1024, attr)) return rc;
  const int64_t ctas = (r + Unit<BITS>::ROWS - 1) / Unit<BITS>::ROWS;
  regroup_rows_kernel<BITS, STAGED>
      <<<(unsigned)ctas + 1, ROW_THREADS, (size_t)d * (STAGED ? 6 : 4), st>>>(q, perm, r, d, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int BITS>
int launch_regroup(const uint32_t *q, int32_t *perm, int64_t r, int d, uint32_t *out,
                   cudaStream_t st) {
  // one more CTA than the rows need: it reports the order
  if (d > LONGEST) {
    static std::atomic<bool> attr[64] = {};
    if (const int rc = ensure_smem_attr(regroup_kernel<BITS>, 65536, attr)) return rc;
    const int64_t cap = (int64_t)num_sms() * 8;
    regroup_kernel<BITS><<<(unsigned)(r < cap ? r : cap) + 1, ROW_THREADS, (size_t)d, st>>>(
        q, perm, r, d, out);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  return d <= LONGEST_STAGED ? launch_rows<BITS, true>(q, perm, r, d, out, st)
                             : launch_rows<BITS, false>(q, perm, r, d, out, st);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_regroup(const int32_t *qweight, const int32_t *g_idx, int64_t r, int64_t d,
                            int bits, int group, int32_t *out, int32_t *perm,
                            gptq_stream_t stream) {
  if (r < 0 || r > (int64_t)INT32_MAX) return GPTQ_ERR_INVALID_ARG;
  if (d <= 0 || d % 32 != 0 || d > 65536) return GPTQ_ERR_INVALID_ARG;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return GPTQ_ERR_INVALID_ARG;
  if (group < 32 || group % 32 != 0 || d % group != 0) return GPTQ_ERR_INVALID_ARG;
  if (!g_idx || !perm || (r > 0 && (!qweight || !out))) return GPTQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(qweight) % 4 || reinterpret_cast<uintptr_t>(g_idx) % 4 ||
      reinterpret_cast<uintptr_t>(out) % 4 || reinterpret_cast<uintptr_t>(perm) % 4)
    return GPTQ_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int G = (int)(d / group);
  static std::atomic<bool> attr[64] = {};
  if (const int arc = ensure_smem_attr(group_order_kernel, 2 * 65536, attr)) return arc;
  group_order_kernel<<<(G + ORDER_WARPS - 1) / ORDER_WARPS, 32 * ORDER_WARPS, (size_t)d * 2, st>>>(
      g_idx, (int)d, group, G, perm);
  GPTQ_LAUNCH_CHECK();
  const uint32_t *q = reinterpret_cast<const uint32_t *>(qweight);
  uint32_t *o = reinterpret_cast<uint32_t *>(out);
  int rc;
  switch (bits) {
    case 2: rc = launch_regroup<2>(q, perm, r, (int)d, o, st); break;
    case 3: rc = launch_regroup<3>(q, perm, r, (int)d, o, st); break;
    case 4: rc = launch_regroup<4>(q, perm, r, (int)d, o, st); break;
    default: rc = launch_regroup<8>(q, perm, r, (int)d, o, st); break;
  }
  if (rc != GPTQ_OK) return rc;
  int32_t first = 0;
  GPTQ_CUDA_TRY(cudaMemcpyAsync(&first, perm, sizeof(first), cudaMemcpyDeviceToHost, st));
  GPTQ_CUDA_TRY(cudaStreamSynchronize(st));
  return first < 0 ? GPTQ_ERR_INVALID_ARG : GPTQ_OK;
}
