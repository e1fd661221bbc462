// gptq_int8_linear and gptq_int8_gated: products in 8-bit integers with a scale per
// token and per row of the weights.
//
// Sources: "LLM 量化技术" §1.2 -- the symmetric quantiser, x = s q on both sides, so that
// a product of two quantised numbers is the integers' product times both scales; the
// GPTQ reading card, 计算设置 -- the quantised layers run at inference.
//
// This file checks the arguments and chooses the kernel.
#include <initializer_list>
#include <mutex>

#include "int8_linear.h"
#include "overlap.h"

namespace gptq {

namespace {
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

bool valid_sizes(int64_t n, int64_t r, int64_t d) {
  // (the last tile's coordinates, too, are 32-bit)
  constexpr int64_t MOST = (int64_t)INT32_MAX - 512;
  return n >= 0 && n <= MOST && r >= 0 && r <= MOST && d > 0 && d % 32 == 0 && d <= 65536;
}

// up to 64 tokens W's bytes are the bound; more, its products or x's bytes
bool by_pairs(const Int8Args &a, int sms) { return a.n > FEW_TOKENS && int8_pairs_faster(a, sms); }

// Checks and launches; layers: 1, or 2 of a gated block.
int int8_product(const Int8Args &a, int layers, int64_t d, cudaStream_t st) {
  if (!valid_sizes(a.n, a.r, d)) return GPTQ_ERR_INVALID_ARG;
  if (a.ytype != GPTQ_F16 && a.ytype != GPTQ_BF16 && a.ytype != GPTQ_F32) return GPTQ_ERR_INVALID_ARG;
  if (a.n == 0 || a.r == 0) return GPTQ_OK;
  const size_t ysize = a.ytype == GPTQ_F32 ? 4 : 2;
  if (!a.x || !a.x_scales || !a.y || misaligned(a.x, 16) || misaligned(a.x_scales, 4) || misaligned(a.y, ysize))
    return GPTQ_ERR_INVALID_ARG;
  const Span out = {a.y, (size_t)a.n * a.r * ysize};
  if (overlap(out, Span{a.x, (size_t)a.n * d}) || overlap(out, Span{a.x_scales, (size_t)a.n * 4}))
    return GPTQ_ERR_INVALID_ARG;
  for (int k = 0; k < layers; ++k) {
    if (!a.w[k] || !a.w_scales[k] || misaligned(a.w[k], 16) || misaligned(a.w_scales[k], 4) ||
        misaligned(a.bias[k], ysize))
      return GPTQ_ERR_INVALID_ARG;
    for (const Span &s : {Span{a.w[k], (size_t)a.r * d}, Span{a.w_scales[k], (size_t)a.r * 4},
                          Span{a.bias[k], (size_t)a.r * ysize}})
      if (overlap(out, s)) return GPTQ_ERR_INVALID_ARG;
  }
  return by_pairs(a, num_sms()) ? launch_int8_pair(a, st) : launch_int8_single(a, st);
}

}  // namespace

int int8_map(CUtensorMap *map, const int8_t *p, int64_t rows, int d, int box_rows) {
  const EncodeTiledFn enc = encode_fn();
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t pitch[1] = {(cuuint64_t)d};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  if (!enc || enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(p), dims, pitch, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    set_last_error_msg(__FILE__, __LINE__, "cuTensorMapEncodeTiled rejected a matrix of 8-bit integers");
    return GPTQ_ERR_CUDA;
  }
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_int8_linear(const int8_t *x, const float *x_scales, int64_t n, const int8_t *w,
                                const float *w_scales, int64_t r, int64_t d, const void *bias, void *y,
                                int ytype, gptq_stream_t stream) {
  const Int8Args a{x, x_scales, {w, nullptr}, {w_scales, nullptr}, {bias, nullptr}, y, n, r, (int)d, ytype,
                   GPTQ_ACT_NONE, false};
  return int8_product(a, 1, d, (cudaStream_t)stream);
}

extern "C" int gptq_int8_gated(const int8_t *x, const float *x_scales, int64_t n, const int8_t *gate,
                               const float *gate_scales, const int8_t *up, const float *up_scales, int64_t r,
                               int64_t d, const void *gate_bias, const void *up_bias, int activation, void *y,
                               int ytype, gptq_stream_t stream) {
  if (activation < GPTQ_ACT_NONE || activation > GPTQ_ACT_GELU) return GPTQ_ERR_INVALID_ARG;
  const Int8Args a{x, x_scales, {gate, up}, {gate_scales, up_scales}, {gate_bias, up_bias}, y, n, r, (int)d,
                   ytype, activation, true};
  return int8_product(a, 2, d, (cudaStream_t)stream);
}

extern "C" int gptq_selftest_int8_timeout(const int8_t *x, const float *x_scales, int64_t n, const int8_t *w,
                                          const float *w_scales, int64_t r, int64_t d, int what, float *y,
                                          gptq_stream_t stream) {
  if (what < GPTQ_GIVE_UP_WARP || what > GPTQ_GIVE_UP_THREAD) return GPTQ_ERR_INVALID_ARG;
  Int8Args a{x, x_scales, {w, nullptr}, {w_scales, nullptr}, {nullptr, nullptr}, y, n, r, (int)d, GPTQ_F32,
             GPTQ_ACT_NONE, false};
  a.give_up = what;
  return int8_product(a, 1, d, (cudaStream_t)stream);
}

extern "C" int gptq_int8_plan(int64_t n, int64_t r, int64_t d, int gated, int sms, int64_t *plan) {
  if (!valid_sizes(n, r, d) || n == 0 || r == 0 || sms < 2 || sms > 4096 || !plan) return GPTQ_ERR_INVALID_ARG;
  Int8Args a{};
  a.n = n;
  a.r = r;
  a.d = (int)d;
  a.gated = gated != 0;
  Int8Plan p;
  if (const int rc = by_pairs(a, sms) ? int8_pair_plan(a, sms, p) : int8_single_plan(a, sms, p)) return rc;
  const int64_t v[] = {p.pairs, p.ctas, p.cluster, p.tokens, p.rows, p.stages, p.columns, (int64_t)p.smem};
  for (int i = 0; i < 8; ++i) plan[i] = v[i];
  return GPTQ_OK;
}
