// gptq_packed_linear: y = x W^^T + bias straight from a packed layer, for any
// number of tokens.
//
// Sources: the GPTQ reading card ("GPTQ: Accurate Post-Training Quantization
// for Generative Pre-trained Transformers", 计算设置) -- the quantised layers
// run from their packed weights at inference; "一文读懂GPTQ" §三 -- codes in
// int32 arrays, group_size, desc_act.
//
//   y[t, i] = xs[t] sum_j s[i, j/g] (q[i, j] - z[i, j/g]) x[t, p(j)] + bias[i]
//
// A few tokens' product is bound by reading and unpacking the weights
// (packed_few.cuh); more tokens', by conversion and then by the tensor cores
// (packed_many.cu).  This file checks the arguments, brings x into the
// layer's column order and, for many tokens, 8-bit codes into fp16.
#include <type_traits>

#include "overlap.h"
#include "packed_linear.h"

namespace gptq {
namespace {

// Which product: few tokens at once are bound by the weights' bytes and codes, and
// warp-level products, which need no start-up, are faster: always up to 8
// tokens, with 8-bit x up to 16, and with 16-bit x for layers of up to 2^25 codes.
// Measured (warp-level, tcgen05; us): 16 tokens, 4 bits, fp16, 4096 x 4096 12.8,
// 12.6; 9 tokens 8.9, 12.2; 8192 x 8192, 8 tokens 25.7, 25.1, 16 tokens 35.8,
// 25.1; 16 tokens of 8-bit x, 11008 x 4096 16.2, 25.2.
// fp32 results take the tensor core two or three parts of every weight: the warp-level
// products, 16 tokens at a time, up to 32 tokens, of 8-bit x up to 64.  Measured: 4096 x
// 11008, 32 tokens fp16 44.0, 41.4, bf16 45.2, 62.7, 64 tokens 79.4, 43.1 and 80.6, 65.3;
// 11008 x 4096, 64 tokens of 8-bit x 45.6, 59.3, 128 tokens 88.4, 63.6.
bool few_tokens(int64_t n, int64_t r, int64_t d, int xtype, int ytype) {
  if (ytype == GPTQ_F32) return n <= (xtype == GPTQ_I8 ? 64 : 32);
  return n <= 8 || (n <= 16 && (xtype == GPTQ_I8 || r * d <= (1 << 25)));
}

// x in the layer's column order: out[t, j] = x[t, perm[j]], entries outside
// [0, d) clamped; WIDEN: 8-bit codes as fp16 (exact), the operand of the
// tensor-core product, in that order if perm is given.  A thread takes eight
// columns of one token; the columns are spread over the grid so that a few
// tokens fill the GPU.  Up to 8 bytes per element, from L2 for few tokens.
constexpr int GATHER_THREADS = 128;

template <typename T, bool WIDEN>
__global__ void __launch_bounds__(GATHER_THREADS)
    gather_columns_kernel(const T *__restrict__ x, const int32_t *__restrict__ perm, int d,
                          void *__restrict__ out) {
  // (the product starts beside this kernel and waits for it before it reads x)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using O = typename std::conditional<WIDEN, uint16_t, T>::type;
  const int j0 = (blockIdx.y * GATHER_THREADS + threadIdx.x) * 8;
  if (j0 >= d) return;   // d % 8 == 0
  const T *row = x + (int64_t)blockIdx.x * d;
  alignas(16) T v[8];
  if (perm) {
    int c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __ldg(perm + j0 + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldg(row + min(max(c[i], 0), d - 1));
  } else {
    *reinterpret_cast<uint2 *>(v) = __ldg(reinterpret_cast<const uint2 *>(row + j0));   // WIDEN only
  }
  alignas(16) O o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (WIDEN)
      o[i] = __half_as_ushort(__short2half_rn((short)(signed char)v[i]));
    else
      o[i] = v[i];
  }
  O *dst = static_cast<O *>(out) + (int64_t)blockIdx.x * d + j0;
  if constexpr (sizeof(O) == 2)
    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(o);
  else
    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(o);
}

bool valid_packed(int64_t n, int64_t r, int64_t d, int bits, int group, int xtype) {
  if (n < 0 || n > (int64_t)INT32_MAX || r < 0 || r > (int64_t)INT32_MAX) return false;
  if (d <= 0 || d % 32 != 0 || d > 65536) return false;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return false;
  if (group != -1 && (group < 32 || group % 32 != 0 || d % group != 0)) return false;
  return xtype == GPTQ_F16 || xtype == GPTQ_BF16 || xtype == GPTQ_I8;
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_packed_linear_workspace_bytes(int64_t n, int64_t r, int64_t d, int bits,
                                                     int group, int xtype, int permuted) {
  if (!valid_packed(n, r, d, bits, group, xtype) || n == 0 || r == 0) return 0;
  // (fp32 results may do with less)
  const bool widen = xtype == GPTQ_I8 && !few_tokens(n, r, d, xtype, GPTQ_F16);
  if (!permuted && !widen) return 0;
  return align_up((size_t)n * d * (xtype == GPTQ_I8 && !widen ? 1 : 2), 256);
}

extern "C" int gptq_packed_linear(const void *x, int xtype, const float *x_scales, int64_t n,
                                  const int32_t *qweight, const float *scales,
                                  const int32_t *zeros, const int32_t *perm, int64_t r, int64_t d,
                                  int bits, int group, const void *bias, void *y, int ytype,
                                  void *workspace, size_t workspace_bytes, gptq_stream_t stream) {
  if (!valid_packed(n, r, d, bits, group, xtype)) return GPTQ_ERR_INVALID_ARG;
  if (ytype != GPTQ_F32 && (xtype == GPTQ_I8 ? ytype != GPTQ_F16 && ytype != GPTQ_BF16 : ytype != xtype))
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0 || r == 0) return GPTQ_OK;
  if (!x || !qweight || !scales || !zeros || !y) return GPTQ_ERR_INVALID_ARG;
  if ((xtype == GPTQ_I8) != (x_scales != nullptr)) return GPTQ_ERR_INVALID_ARG;
  const size_t ysize = ytype == GPTQ_F32 ? 4 : 2;
  if (misaligned(x, 16) || misaligned(qweight, 4) || misaligned(scales, 4) ||
      misaligned(zeros, 4) || misaligned(perm, 4) || misaligned(x_scales, 4) ||
      misaligned(bias, ysize) || misaligned(y, ysize) || misaligned(workspace, 256))
    return GPTQ_ERR_INVALID_ARG;
  const size_t need = gptq_packed_linear_workspace_bytes(n, r, d, bits, group, xtype, perm != nullptr);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GPTQ_ERR_NO_MEMORY;
  const int64_t G = group < 0 ? 1 : d / group;
  const size_t params = (size_t)r * G * 4;
  const Span out = {y, (size_t)n * r * ysize}, scratch = {workspace, need};
  if (overlap(out, scratch)) return GPTQ_ERR_INVALID_ARG;
  for (const Span &s : {Span{x, (size_t)n * d * (xtype == GPTQ_I8 ? 1 : 2)}, Span{x_scales, (size_t)n * 4},
                        Span{qweight, (size_t)r * (d / 32) * bits * 4}, Span{scales, params},
                        Span{zeros, params}, Span{perm, (size_t)d * 4}, Span{bias, (size_t)r * ysize}})
    if (overlap(out, s) || overlap(scratch, s)) return GPTQ_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const bool few = few_tokens(n, r, d, xtype, ytype), widen = xtype == GPTQ_I8 && !few;
  if (widen || perm) {
    const dim3 grid((unsigned)n, (unsigned)((d / 8 + GATHER_THREADS - 1) / GATHER_THREADS));
    if (widen)
      gather_columns_kernel<uint8_t, true><<<grid, GATHER_THREADS, 0, st>>>(
          static_cast<const uint8_t *>(x), perm, (int)d, workspace);
    else if (xtype == GPTQ_I8)
      gather_columns_kernel<uint8_t, false><<<grid, GATHER_THREADS, 0, st>>>(
          static_cast<const uint8_t *>(x), perm, (int)d, workspace);
    else
      gather_columns_kernel<uint16_t, false><<<grid, GATHER_THREADS, 0, st>>>(
          static_cast<const uint16_t *>(x), perm, (int)d, workspace);
    GPTQ_LAUNCH_CHECK();
    x = workspace;
    if (widen) xtype = GPTQ_F16;
  }
  const PackedArgs a{x, x_scales, reinterpret_cast<const uint32_t *>(qweight), scales, zeros,
                     bias, y, n, r, (int)d, bits, group, (int)G, xtype, ytype,
                     widen || perm ? 1 : 0};
  if (!few) return ytype == GPTQ_F32 ? launch_packed_many_f32(a, st) : launch_packed_many(a, st);
  return xtype == GPTQ_F16    ? launch_packed_few_f16(a, st)
         : xtype == GPTQ_BF16 ? launch_packed_few_bf16(a, st)
                              : launch_packed_few_i8(a, st);
}
