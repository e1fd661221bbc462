// gptq_regroup: the columns of a packed act-order layer sorted by group.
//
// Source: "一文读懂GPTQ" §三 -- desc_act quantises the columns in another
// order than theirs, so the columns of one group lie scattered over the row
// (g_idx).  With perm the stable order of the columns by g_idx, column j of
// the result is column perm[j], and position j belongs to group j / group.
//
// Two kernels.  The order: one warp per group reads g_idx 32 entries at a time
// and places the columns of its group by ballot, in order; a slot that stays
// empty (a group with too few columns) is marked -1, so perm holds a -1 if and
// only if some group has another number of columns than `group`.  The rows:
// r*d*bits/8 bytes in and out; a row is unpacked to bytes in shared memory,
// and each thread gathers 32 of them and packs them.
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
  const int g = blockIdx.x * ORDER_WARPS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (g >= G) return;
  int32_t *slots = perm + (int64_t)g * group;
  int found = 0;
  for (int c0 = 0; c0 < d; c0 += 32) {   // d % 32 == 0
    const bool mine = __ldg(g_idx + c0 + lane) == g;
    const uint32_t hit = __ballot_sync(0xffffffffu, mine);
    const int at = found + __popc(hit & ((1u << lane) - 1u));
    if (mine && at < group) slots[at] = c0 + lane;
    found += __popc(hit);
  }
  for (int at = found + lane; at < group; at += 32) slots[at] = -1;
}

template <int BITS>
__global__ void __launch_bounds__(ROW_THREADS)
    regroup_kernel(const uint32_t *__restrict__ qweight, int32_t *perm, int64_t r, int d,
                   uint32_t *__restrict__ out) {
  extern __shared__ __align__(16) uint8_t row_codes[];   // [d]
  const int nchunk = d / 32;
  // block 0 tells the host: perm[0] < 0 if any entry is
  if (blockIdx.x == 0) {
    int bad = 0;
    for (int j = threadIdx.x; j < d; j += ROW_THREADS) bad |= perm[j] < 0;
    if (__syncthreads_or(bad) && threadIdx.x == 0) perm[0] = -1;
  }
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
        const int from = *(volatile const int32_t *)(perm + k * 32 + j);
        c[j] = row_codes[from < 0 ? 0 : from];
      }
      pack32<BITS>(c, w);
#pragma unroll
      for (int t = 0; t < BITS; ++t) dst[(int64_t)k * BITS + t] = w[t];
    }
  }
}

template <int BITS>
int launch_regroup(const uint32_t *q, int32_t *perm, int64_t r, int d, uint32_t *out,
                   cudaStream_t st) {
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(regroup_kernel<BITS>, 65536, attr)) return rc;
  const int64_t cap = (int64_t)num_sms() * 8;
  const int64_t grid = r < 1 ? 1 : (r < cap ? r : cap);
  regroup_kernel<BITS><<<(unsigned)grid, ROW_THREADS, (size_t)d, st>>>(q, perm, r, d, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
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
  group_order_kernel<<<(G + ORDER_WARPS - 1) / ORDER_WARPS, 32 * ORDER_WARPS, 0, st>>>(
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
