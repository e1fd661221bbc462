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
// One warp per row and four tokens: lane l takes the 32-code chunks l, l + 32,
// ..., whose codes belong to one group each.  fp32 sums.
#include "packed_linear.h"
#include "unpack_bits.cuh"

namespace gptq {
namespace {

constexpr int FEW_TOKENS = 16;   // up to here the weights' bytes bound the product

// x in the layer's column order: out[t, j] = x[t, perm[j]], entries outside
// [0, d) clamped.  One CTA per token (8 n d or 6 n d bytes, from L2 for few).
template <typename T>
__global__ void __launch_bounds__(256) gather_columns_kernel(const T *__restrict__ x,
                                                             const int32_t *__restrict__ perm, int d,
                                                             T *__restrict__ out) {
  const int64_t row = (int64_t)blockIdx.x * d;
  for (int j = threadIdx.x; j < d; j += blockDim.x)
    out[row + j] = x[row + min(max(__ldg(perm + j), 0), d - 1)];
}

constexpr int SIMPLE_WARPS = 8;
constexpr int SIMPLE_TOKENS = 4;

__device__ __forceinline__ float load_x(const void *p, int type, int64_t i) {
  if (type == GPTQ_I8) return (float)reinterpret_cast<const int8_t *>(p)[i];
  return load_as_float(p, type, i);
}

template <int BITS>
__global__ void __launch_bounds__(32 * SIMPLE_WARPS) packed_linear_simple_kernel(PackedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * SIMPLE_WARPS + (threadIdx.x >> 5);
  if (row >= a.r) return;
  const int nchunk = a.d / 32;
  const uint32_t *qrow = a.qweight + row * nchunk * BITS;
  for (int64_t t0 = (int64_t)blockIdx.y * SIMPLE_TOKENS; t0 < a.n;
       t0 += (int64_t)gridDim.y * SIMPLE_TOKENS) {
    float acc[SIMPLE_TOKENS] = {};
    for (int k = lane; k < nchunk; k += 32) {
      uint32_t w[BITS];
#pragma unroll
      for (int i = 0; i < BITS; ++i) w[i] = __ldg(qrow + (int64_t)k * BITS + i);
      const int gi = a.group > 0 ? k * 32 / a.group : 0;
      const float s = __ldg(a.scales + row * a.G + gi);
      const int z = min(max(__ldg(a.zeros + row * a.G + gi), 0), (1 << BITS) - 1);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float wv = s * (float)((int)code_at<BITS>(w, j) - z);
        const int c = k * 32 + j;
#pragma unroll
        for (int t = 0; t < SIMPLE_TOKENS; ++t)
          if (t0 + t < a.n) acc[t] = fmaf(wv, load_x(a.x, a.xtype, (t0 + t) * a.d + c), acc[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < SIMPLE_TOKENS; ++t) {
      float v = acc[t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0 && t0 + t < a.n) {
        if (a.x_scales) v *= a.x_scales[t0 + t];
        if (a.bias) v += load_as_float(a.bias, a.ytype, row);
        store_float(a.y, a.ytype, (t0 + t) * a.r + row, v);
      }
    }
  }
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
  return permuted ? align_up((size_t)n * d * (xtype == GPTQ_I8 ? 1 : 2), 256) : 0;
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
  cudaStream_t st = (cudaStream_t)stream;
  if (perm) {
    if (xtype == GPTQ_I8)
      gather_columns_kernel<<<(unsigned)n, 256, 0, st>>>(static_cast<const uint8_t *>(x), perm, (int)d,
                                                         static_cast<uint8_t *>(workspace));
    else
      gather_columns_kernel<<<(unsigned)n, 256, 0, st>>>(static_cast<const uint16_t *>(x), perm, (int)d,
                                                         static_cast<uint16_t *>(workspace));
    GPTQ_LAUNCH_CHECK();
    x = workspace;
  }
  const PackedArgs a{x, x_scales, reinterpret_cast<const uint32_t *>(qweight), scales, zeros,
                     bias, y, n, r, (int)d, bits, group, group < 0 ? 1 : (int)(d / group), xtype, ytype};
  if (n <= FEW_TOKENS) return launch_packed_few(a, st);
  const int64_t tb = (n + SIMPLE_TOKENS - 1) / SIMPLE_TOKENS;
  const dim3 grid((unsigned)((r + SIMPLE_WARPS - 1) / SIMPLE_WARPS), (unsigned)(tb < 4096 ? tb : 4096));
  switch (bits) {
    case 2: packed_linear_simple_kernel<2><<<grid, 32 * SIMPLE_WARPS, 0, st>>>(a); break;
    case 3: packed_linear_simple_kernel<3><<<grid, 32 * SIMPLE_WARPS, 0, st>>>(a); break;
    case 4: packed_linear_simple_kernel<4><<<grid, 32 * SIMPLE_WARPS, 0, st>>>(a); break;
    default: packed_linear_simple_kernel<8><<<grid, 32 * SIMPLE_WARPS, 0, st>>>(a); break;
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}
