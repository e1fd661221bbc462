// gptq_int8_weights: a packed layer with one scale per row as 8-bit integers.
//
// Sources: "一文读懂GPTQ" §三 -- codes in int32 words; "LLM 量化技术" §1.2 -- the value
// of a code is s (q - z), so with one group per row w = q - z are integers with
// the row's scale s.
//
// Codes of 2, 3 and 4 bits give |w| <= 15.  8-bit codes fit where the zero point is
// the symmetric quantiser's 128; elsewhere a w may not, and its row's scale becomes NaN.
//
// r d (bits/8 + 1) bytes, read and written once.  A thread turns 32 codes (BITS words)
// into 32 bytes; the threads of a row stand side by side, several rows to a CTA.
#include "launch_after.h"
#include "overlap.h"
#include "unpack_bits.cuh"

namespace gptq {
namespace {

constexpr int THREADS = 256;

// Codes 4k .. 4k + 3 of a chunk as bytes.
template <int BITS>
__device__ __forceinline__ uint32_t four_codes(const uint32_t (&w)[BITS], int k) {
  if constexpr (BITS == 8) return w[k];
  if constexpr (BITS == 4) {
    const uint32_t v = w[k >> 1] >> ((k & 1) * 16), lo = v & 0x0F0Fu, hi = (v >> 4) & 0x0F0Fu;
    return __byte_perm(lo, hi, 0x5140);
  }
  return code_at<BITS>(w, 4 * k) | code_at<BITS>(w, 4 * k + 1) << 8 | code_at<BITS>(w, 4 * k + 2) << 16 |
         code_at<BITS>(w, 4 * k + 3) << 24;
}

// A chunk's words, four at a time where they are aligned (wide).
template <int BITS>
__device__ __forceinline__ void read_chunk(const uint32_t *src, bool wide, uint32_t (&q)[BITS]) {
  if (BITS >= 4 && wide) {
#pragma unroll
    for (int i = 0; i + 4 <= BITS; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src + i);
      q[i] = v.x, q[i + 1] = v.y, q[i + 2] = v.z, q[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) q[i] = src[i];
  }
}

template <int BITS>
__global__ void __launch_bounds__(THREADS)
    int8_weights_kernel(const uint32_t *qweight, const float *scales, const int32_t *zeros, int64_t r, int chunks,
                        int per_row, bool wide, bool whole, int8_t *w, float *w_scales) {
  __shared__ int outside[THREADS / 32];   // per row of the CTA
  const int rows = THREADS / per_row, mine = threadIdx.x / per_row, at = threadIdx.x % per_row;
  const int64_t row = (int64_t)blockIdx.x * rows + mine;
  if (at == 0) outside[mine] = 0;
  pdl_wait_then_release();
  __syncthreads();
  if (row < r) {
    const int z = min(max(__ldcg(zeros + row), 0), (1 << BITS) - 1);
    const uint32_t zzzz = (uint32_t)z * 0x01010101u;
    bool lost = false;
    // (several chunks are read before any is written: the compiler may not move reads over writes)
    constexpr int AT_ONCE = BITS == 8 ? 2 : 4;
    for (int c0 = at; c0 < chunks; c0 += AT_ONCE * per_row) {
      uint32_t q[AT_ONCE][BITS];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        if (c0 + j * per_row < chunks) read_chunk<BITS>(qweight + (row * chunks + c0 + j * per_row) * BITS, wide, q[j]);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const int c = c0 + j * per_row;
        if (c >= chunks) break;
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t v = four_codes<BITS>(q[j], k);
          if constexpr (BITS < 8) {
            o[k] = ((v | 0x80808080u) - zzzz) ^ 0x80808080u;   // per byte: no borrow leaves it
          } else if (z == 128) {
            o[k] = v ^ 0x80808080u;
          } else {
            o[k] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = (int)((v >> (8 * i)) & 0xFFu) - z;
              lost |= e < -128 || e > 127;
              o[k] |= ((uint32_t)min(max(e, -128), 127) & 0xFFu) << (8 * i);
            }
          }
        }
        int8_t *dst = w + (row * chunks + c) * 32;
        if (whole) {   // a sector in one store
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]), "r"(o[1]),
                       "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        } else {
          reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
    if (lost) outside[mine] = 1;
  }
  __syncthreads();
  if (row < r && at == 0) w_scales[row] = outside[mine] ? __uint_as_float(0x7FC00000u) : __ldcg(scales + row);
}

template <int BITS>
int launch_weights(const uint32_t *q, const float *s, const int32_t *z, int64_t r, int chunks, int8_t *w,
                   float *ws, cudaStream_t st) {
  // threads per row: four chunks each at most, where a CTA has as many
  int per_row = 32;
  while (per_row < THREADS && per_row * 4 < chunks) per_row *= 2;
  const int rows = THREADS / per_row;
  return launch_after(int8_weights_kernel<BITS>, (unsigned)((r + rows - 1) / rows), THREADS, 0, 1, st, q, s, z, r,
                      chunks, per_row, reinterpret_cast<uintptr_t>(q) % 16 == 0, reinterpret_cast<uintptr_t>(w) % 32 == 0,
                      w, ws);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_int8_weights(const int32_t *qweight, const float *scales, const int32_t *zeros, int64_t r,
                                 int64_t d, int bits, int8_t *w, float *w_scales, gptq_stream_t stream) {
  if (r < 0 || r > (int64_t)INT32_MAX) return GPTQ_ERR_INVALID_ARG;
  if (d <= 0 || d % 32 != 0 || d > 65536) return GPTQ_ERR_INVALID_ARG;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return GPTQ_ERR_INVALID_ARG;
  if (r == 0) return GPTQ_OK;
  if (!qweight || !scales || !zeros || !w || !w_scales) return GPTQ_ERR_INVALID_ARG;
  for (const void *p : {(const void *)qweight, (const void *)scales, (const void *)zeros, (const void *)w_scales})
    if (reinterpret_cast<uintptr_t>(p) % 4) return GPTQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(w) % 16) return GPTQ_ERR_INVALID_ARG;
  const Span out = {w, (size_t)r * d}, out_scales = {w_scales, (size_t)r * 4};
  if (overlap(out, out_scales)) return GPTQ_ERR_INVALID_ARG;
  for (const Span &s : {Span{qweight, (size_t)r * (d / 32) * bits * 4}, Span{scales, (size_t)r * 4},
                        Span{zeros, (size_t)r * 4}})
    if (overlap(out, s) || overlap(out_scales, s)) return GPTQ_ERR_INVALID_ARG;
  const uint32_t *q = reinterpret_cast<const uint32_t *>(qweight);
  const int chunks = (int)(d / 32);
  cudaStream_t st = (cudaStream_t)stream;
  switch (bits) {
    case 2: return launch_weights<2>(q, scales, zeros, r, chunks, w, w_scales, st);
    case 3: return launch_weights<3>(q, scales, zeros, r, chunks, w, w_scales, st);
    case 4: return launch_weights<4>(q, scales, zeros, r, chunks, w, w_scales, st);
    default: return launch_weights<8>(q, scales, zeros, r, chunks, w, w_scales, st);
  }
}
