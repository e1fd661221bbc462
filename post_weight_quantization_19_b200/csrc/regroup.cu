// gptq_regroup: the columns of a packed act-order layer sorted by group.
//
// Source: "一文读懂GPTQ" §三 -- desc_act quantises the columns in another
// order than theirs, so the columns of one group lie scattered over the row
// (g_idx).  With perm the stable order of the columns by g_idx, column j of
// the result is column perm[j], and position j belongs to group j / group.
//
// Two kernels.  The order, one CTA: each of its 32 warps takes a run of columns
// and counts its groups (match_any gives a column's rank among the 32 that a
// warp reads at once), the counts are summed over the warps, and a second pass
// places the columns.  Whether every group has `group` columns is reported in a
// word of mapped host memory as soon as the counts are there; the host waits for
// that alone, while the columns are placed and the rows move.  If one has not,
// perm becomes the identity.
//
// The rows, r*d*bits/8 bytes in and out: a CTA takes eight rows (four of 8-bit
// codes) and transposes them so that one shared-memory word holds a column's
// codes of all its rows, a nibble (byte) each.  Moving a column is then one
// random 4-byte read for eight codes instead of eight byte reads; reading codes
// one by one took 490 us where this takes 28 (8192 x 8192, 3 bits: bound by the 5.7
// instructions a code costs; 17 us for 11008 x 4096, 4 bits).
// Codes of 2 and 3 bits travel as nibbles.  Rows too long for that (d > 49152)
// go through bytes in shared memory, one row at a time.
#include <mutex>

#include "gptq_internal.h"
#include "overlap.h"
#include "pack_bits.cuh"
#include "unpack_bits.cuh"

namespace gptq {
namespace {

constexpr int ORDER_WARPS = 32;
constexpr int ROW_THREADS = 256;
enum { PENDING = 0, ACCEPTED, REFUSED };   // the order, in a call's word of host memory

__global__ void __launch_bounds__(32 * ORDER_WARPS)
    group_order_kernel(const int32_t *__restrict__ g_idx, int d, int group, int G,
                       int32_t *__restrict__ perm, volatile int *report) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the rows: see below
  extern __shared__ __align__(16) uint16_t counts[];   // [ORDER_WARPS][G]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t *mine = counts + warp * G;
  const int chunks = d / 32;                            // d % 32 == 0
  const int c0 = chunks * warp / ORDER_WARPS, c1 = chunks * (warp + 1) / ORDER_WARPS;
  for (int i = threadIdx.x; i < ORDER_WARPS * G; i += 32 * ORDER_WARPS) counts[i] = 0;
  __syncthreads();
  int bad = 0;
#pragma unroll 4
  for (int c = c0; c < c1; ++c) {
    const int g = __ldg(g_idx + c * 32 + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, g);
    if (g < 0 || g >= G)
      bad = 1;
    else if ((same & ((1u << lane) - 1u)) == 0)         // the first of its group
      mine[g] += (uint16_t)__popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += 32 * ORDER_WARPS) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < ORDER_WARPS; ++w) {
      const int v = counts[w * G + g];
      counts[w * G + g] = (uint16_t)sum;                // of the warps before
      sum += v;
    }
    bad |= sum != group;
  }
  if (__syncthreads_or(bad)) {
    for (int j = threadIdx.x; j < d; j += 32 * ORDER_WARPS) perm[j] = j;
    if (threadIdx.x == 0) *report = REFUSED;
    return;
  }
  if (threadIdx.x == 0) *report = ACCEPTED;
#pragma unroll 4
  for (int c = c0; c < c1; ++c) {
    const int g = __ldg(g_idx + c * 32 + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, g);
    const int before = __popc(same & ((1u << lane) - 1u));
    const int base = mine[g];
    __syncwarp();
    if (before == 0) mine[g] = (uint16_t)(base + __popc(same));
    __syncwarp();
    perm[g * group + base + before] = c * 32 + lane;
  }
}

// ---- eight codes of a row as the nibbles of a word, low first

// (v where the mask is set, w elsewhere: one instruction)
__device__ __forceinline__ uint32_t choose(uint32_t mask, uint32_t v, uint32_t w) {
  return (v & mask) | (w & ~mask);
}
__device__ __forceinline__ uint32_t nibbles_of_3(uint32_t v) {   // 24 bits; above them anything
  v = choose(0x0000FFFFu, v, v << 4);   // 12 bits in each half, 6 in each byte, 3 in each nibble,
  v = choose(0x00FF00FFu, v, v << 2);   // with others' bits between them until the end
  v = choose(0x0F0F0F0Fu, v, v << 1);
  return v & 0x77777777u;
}
__device__ __forceinline__ uint32_t threes_of_nibbles(uint32_t v) {
  v -= (v & 0x70707070u) >> 1;          // lo + 16 hi -> lo + 8 hi, and so on
  v -= (v & 0x3F003F00u) / 4 * 3;
  return v - (v & 0x0FFF0000u) / 16 * 15;
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
      o[0] = nibbles_of_3(w[0]);
      o[1] = nibbles_of_3(__funnelshift_r(w[0], w[1], 24));
      o[2] = nibbles_of_3(__funnelshift_r(w[1], w[2], 16));
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
// from global memory once in whole lines.  perm is still being written when this
// kernel starts: it is read with ordinary loads, behind the wait.
template <int BITS, bool STAGED>
__global__ void __launch_bounds__(ROW_THREADS)
    regroup_rows_kernel(const uint32_t *__restrict__ qweight, const int32_t *perm, int64_t r, int d,
                        uint32_t *__restrict__ out) {
  using U = Unit<BITS>;
  extern __shared__ __align__(16) uint32_t columns[];   // [d]: a column's codes of the CTA's rows
  const int pitch = d / 32 * BITS;   // words per row
  const int units = d / U::COLS;
  uint16_t *order = reinterpret_cast<uint16_t *>(columns + d);
  const int64_t groups = (r + U::ROWS - 1) / U::ROWS;
  for (int64_t block = blockIdx.x; block < groups; block += gridDim.x) {
    const int rows = (int)min((int64_t)U::ROWS, r - block * U::ROWS);
    const uint32_t *src = qweight + block * U::ROWS * pitch;
    uint32_t *dst = out + block * U::ROWS * pitch;
    for (int u = threadIdx.x; u < units; u += ROW_THREADS) {
      uint32_t n[U::ROWS][U::OUT];
#pragma unroll
      for (int i = 0; i < U::ROWS; ++i) {
        uint32_t w[U::IN];
#pragma unroll
        for (int k = 0; k < U::IN; ++k)
          w[k] = i < rows ? __ldg(src + i * pitch + u * U::IN + k) : 0u;
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
    if (block == blockIdx.x) {
      // launched beside the order's kernel: nothing was written, nothing of it read
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if constexpr (STAGED) {
        constexpr int EACH = 16;   // loads in flight
        for (int j0 = threadIdx.x; j0 < d; j0 += EACH * ROW_THREADS) {
          int from[EACH];
#pragma unroll
          for (int i = 0; i < EACH; ++i) from[i] = j0 + i * ROW_THREADS < d ? perm[j0 + i * ROW_THREADS] : 0;
#pragma unroll
          for (int i = 0; i < EACH; ++i)
            if (j0 + i * ROW_THREADS < d) order[j0 + i * ROW_THREADS] = (uint16_t)place(from[i]);
        }
      }
    }
    __syncthreads();
    for (int u = threadIdx.x; u < units; u += ROW_THREADS) {
      uint32_t n[U::ROWS][U::OUT];
#pragma unroll
      for (int k = 0; k < U::OUT; ++k) {
        uint32_t a[U::ROWS];
        const int j = u * U::COLS + k * U::ROWS;
        if constexpr (STAGED) {
#pragma unroll
          for (int i = 0; i < U::ROWS; i += 4) {
            const uint2 o = *reinterpret_cast<const uint2 *>(order + j + i);
            a[i] = columns[o.x & 0xFFFFu];
            a[i + 1] = columns[o.x >> 16];
            a[i + 2] = columns[o.y & 0xFFFFu];
            a[i + 3] = columns[o.y >> 16];
          }
        } else {
#pragma unroll
          for (int i = 0; i < U::ROWS; ++i) a[i] = columns[place(perm[j + i])];
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
          for (int k = 0; k < U::IN; ++k) dst[i * pitch + u * U::IN + k] = w[k];
      }
    }
    __syncthreads();   // columns is free for the next rows
  }
}

template <int BITS>
__global__ void __launch_bounds__(ROW_THREADS)
    regroup_kernel(const uint32_t *__restrict__ qweight, const int32_t *perm, int64_t r, int d,
                   uint32_t *__restrict__ out) {
  extern __shared__ __align__(16) uint8_t row_codes[];   // [d]
  asm volatile("griddepcontrol.wait;" ::: "memory");     // perm
  const int nchunk = d / 32;
  for (int64_t row = blockIdx.x; row < r; row += gridDim.x) {
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
        c[j] = row_codes[perm[k * 32 + j]];
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
  // as many CTAs as fit at once, each keeping the order for all its rows
  const size_t smem = (size_t)d * (STAGED ? 6 : 4);
  int per_sm = (int)((200u << 10) / (smem + 1024));
  per_sm = per_sm < 1 ? 1 : (per_sm > 8 ? 8 : per_sm);
  const int64_t most = (r + Unit<BITS>::ROWS - 1) / Unit<BITS>::ROWS, fit = (int64_t)num_sms() * per_sm;
  const dim3 grid((unsigned)(most < fit ? most : fit));
  GPTQ_LAUNCH_PDL((regroup_rows_kernel<BITS, STAGED>), grid, dim3(ROW_THREADS), smem, st, q, perm, r, d, out);
  return GPTQ_OK;
}

template <int BITS>
int launch_regroup(const uint32_t *q, int32_t *perm, int64_t r, int d, uint32_t *out,
                   cudaStream_t st) {
  if (r == 0) return GPTQ_OK;
  if (d > LONGEST) {
    static std::atomic<bool> attr[64] = {};
    if (const int rc = ensure_smem_attr(regroup_kernel<BITS>, 65536, attr)) return rc;
    const int64_t cap = (int64_t)num_sms() * 8;
    const dim3 grid((unsigned)(r < cap ? r : cap));
    GPTQ_LAUNCH_PDL((regroup_kernel<BITS>), grid, dim3(ROW_THREADS), (size_t)d, st, q, perm, r, d, out);
    return GPTQ_OK;
  }
  return d <= LONGEST_STAGED ? launch_rows<BITS, true>(q, perm, r, d, out, st)
                             : launch_rows<BITS, false>(q, perm, r, d, out, st);
}

// Words of mapped host memory that calls report in: one per call in flight, kept for
// later calls in a list through the words themselves.  (A copy of one word to the
// host's stack cost more than the kernels.)
struct Word {
  int value;
  Word *next;
};
std::mutex g_words_mutex;
Word *g_words = nullptr;

int take_word(Word **word) {
  {
    std::lock_guard<std::mutex> lock(g_words_mutex);
    if (g_words) {
      *word = g_words;
      g_words = g_words->next;
      return GPTQ_OK;
    }
  }
  // (allowed while another stream is being captured, whose capture it would end otherwise)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  GPTQ_CUDA_TRY(cudaThreadExchangeStreamCaptureMode(&mode));
  void *p = nullptr;
  const cudaError_t e = cudaHostAlloc(&p, 64, cudaHostAllocMapped | cudaHostAllocPortable);
  (void)cudaThreadExchangeStreamCaptureMode(&mode);
  GPTQ_CUDA_TRY(e);
  *word = static_cast<Word *>(p);
  return GPTQ_OK;
}

void give_word(Word *word) {
  std::lock_guard<std::mutex> lock(g_words_mutex);
  word->next = g_words;
  g_words = word;
}

int enqueue_regroup(const uint32_t *q, const int32_t *g_idx, int64_t r, int d, int bits, int group,
                    uint32_t *out, int32_t *perm, int *report, cudaStream_t st) {
  const int G = d / group;
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(group_order_kernel, ORDER_WARPS * 2048 * 2, attr)) return rc;
  group_order_kernel<<<1, 32 * ORDER_WARPS, (size_t)ORDER_WARPS * G * 2, st>>>(g_idx, d, group, G,
                                                                             perm, report);
  GPTQ_LAUNCH_CHECK();
  switch (bits) {
    case 2: return launch_regroup<2>(q, perm, r, d, out, st);
    case 3: return launch_regroup<3>(q, perm, r, d, out, st);
    case 4: return launch_regroup<4>(q, perm, r, d, out, st);
    default: return launch_regroup<8>(q, perm, r, d, out, st);
  }
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
  // (the order is written while g_idx is still read)
  const Span in[] = {{qweight, (size_t)r * (d / 32) * bits * 4}, {g_idx, (size_t)d * 4}};
  const Span out_codes = {out, in[0].bytes}, out_perm = {perm, (size_t)d * 4};
  if (overlap(out_codes, out_perm)) return GPTQ_ERR_INVALID_ARG;
  for (const Span &s : in)
    if (overlap(out_codes, s) || overlap(out_perm, s)) return GPTQ_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  GPTQ_CUDA_TRY(cudaStreamIsCapturing(st, &capture));
  if (capture != cudaStreamCaptureStatusNone) return GPTQ_ERR_INVALID_ARG;   // it waits for its result
  Word *word = nullptr;
  if (const int rc = take_word(&word)) return rc;
  volatile int *seen = &word->value;
  *seen = PENDING;
  int rc = enqueue_regroup(reinterpret_cast<const uint32_t *>(qweight), g_idx, r, (int)d, bits, group,
                           reinterpret_cast<uint32_t *>(out), perm, &word->value, st);
  // (before the order's kernel has run the word is pending; a launch that failed
  // or a fault on the device ends the wait through the stream's state)
  for (unsigned spins = 1; *seen == PENDING; ++spins) {
    if (spins % 1024) continue;
    const cudaError_t e = cudaStreamQuery(st);
    if (e == cudaErrorNotReady) continue;
    if (e != cudaSuccess) {   // the word may still be written: not given back
      set_last_error(__FILE__, __LINE__, "cudaStreamQuery", e);
      return GPTQ_ERR_CUDA;
    }
    if (*seen == PENDING) break;   // all that was enqueued is done: its launch failed
  }
  if (rc == GPTQ_OK && *seen != ACCEPTED) rc = *seen == REFUSED ? GPTQ_ERR_INVALID_ARG : GPTQ_ERR_CUDA;
  give_word(word);
  return rc;
}
