// MXFP4 quantization and read-back, and the token operands of the MXFP4
// products.
//
// Per block of 32 consecutive elements of a row, a = max |v|:
//   scale byte = max(exponent field of a - top, 0), i.e. 2^max(floor(log2 a) -
//   top, -127), top = 2 (E2M1) or 8 (E4M3); codes = v / scale rounded to
//   nearest even, saturating. Dividing by a power of two is exact in fp32, so
//   each element is rounded once.
// Every kernel here is bound by its bytes. A thread takes 8 consecutive
// elements, four neighbouring lanes a block (its maximum by two shuffles), so
// that a warp reads and writes whole lines.
#include "common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace moe {

namespace {

constexpr int kTop4 = 2, kTop8 = 8;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Elements c .. c + 7 of a row (zeros from `cols` on); vec: 16-byte loads are
// aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int64_t c, int64_t cols, bool vec,
                                      float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + c);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(b[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float(row[c + i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t cols, bool vec,
                                      float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    const float4 a = *reinterpret_cast<const float4*>(row + c);
    const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? row[c + i] : 0.0f;
  }
}

// Bits of the largest magnitude of the block that four lanes hold 8 elements
// of each. Unsigned bit patterns order magnitudes with infinities and NaNs on
// top, which a float maximum would drop.
__device__ __forceinline__ uint32_t block_amax_bits(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// The four scale bytes of a 128-element tile of a row, from the 16 lanes that
// hold it (valid in the first of them).
__device__ __forceinline__ uint32_t gather_scale_word(uint32_t byte, int lane) {
  uint32_t w = byte << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  return w | __shfl_xor_sync(0xffffffffu, w, 8);
}

__device__ __forceinline__ uint32_t encode8_e2m1(const float (&v)[8], float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= e2m1_pair(mx_scaled(v[2 * i], inv), mx_scaled(v[2 * i + 1], inv)) << (8 * i);
  return w;
}
__device__ __forceinline__ uint2 encode8_e4m3(const float (&v)[8], float inv) {
  return make_uint2(mx_encode4(mx_scaled(v[0], inv), mx_scaled(v[1], inv), mx_scaled(v[2], inv),
                               mx_scaled(v[3], inv)),
                    mx_encode4(mx_scaled(v[4], inv), mx_scaled(v[5], inv), mx_scaled(v[6], inv),
                               mx_scaled(v[7], inv)));
}

// src [rows][cols] with row stride ld -> codes and tiled scales. PAIRED: row R
// of the result comes from two matrices (gate, up) of groups of I rows, whose
// rows alternate in runs of 64.
template <typename TIn, bool PAIRED>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(
    const TIn* __restrict__ src, const TIn* __restrict__ src2, int64_t rows, int64_t cols,
    int64_t ld, int64_t I, bool vec, uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  pdl_entry();
  const int lane = threadIdx.x & 31;
  const int64_t kt = mxfp4_k_tiles(cols);
  const int64_t per_row = kt * 16;
  const int64_t n = (rows + 127) / 128 * 128 * per_row;  // a multiple of 32
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row;
    const int64_t c8 = i - r * per_row;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < rows) {
      const TIn* row;
      if constexpr (PAIRED) {
        const int64_t e = r / (2 * I), w = r - e * 2 * I;
        row = (((w >> 6) & 1) ? src2 : src) + (e * I + (w >> 7) * 64 + (w & 63)) * ld;
      } else {
        row = src + r * ld;
      }
      load8(row, c8 * 8, cols, vec, v);
    }
    const uint32_t byte = mx_scale_byte(block_amax_bits(v), kTop4);
    const uint32_t word = gather_scale_word(byte, lane);
    if (r < rows)
      *reinterpret_cast<uint32_t*>(q + r * (kt * 64) + c8 * 4) = encode8_e2m1(v, mx_inv_scale(byte));
    if ((lane & 15) == 0)
      *reinterpret_cast<uint32_t*>(scales + ((r >> 7) * kt + (c8 >> 4)) * 512 +
                                   mxfp4_scale_word((uint32_t)(r & 127))) = word;
  }
}

template <typename TOut>
__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ scales,
                                                               int64_t rows, int64_t cols,
                                                               TOut* __restrict__ out, int64_t ld,
                                                               bool vec) {
  pdl_entry();
  const int64_t kt = mxfp4_k_tiles(cols);
  const int64_t per_row = (cols + 7) / 8;
  const int64_t n = rows * per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row;
    const int64_t c8 = i - r * per_row, c = c8 * 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q + r * (kt * 64) + c8 * 4);
    const uint32_t byte = scales[((r >> 7) * kt + (c8 >> 4)) * 512 +
                                 mxfp4_scale_word((uint32_t)(r & 127)) + ((c8 >> 2) & 3)];
    const float s = mx_scale_or_nan(byte);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = e2m1_values(w >> (8 * j));
      v[2 * j] = f.x * s;  // exact: two significant bits, exponents of bf16 and fp32
      v[2 * j + 1] = f.y * s;
    }
    TOut* dst = out + r * ld + c;
    if constexpr (sizeof(TOut) == 2) {
      if (vec && c + 8 <= cols) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) dst[j] = __float2bfloat16_rn(v[j]);
      }
    } else {
      if (vec && c + 8 <= cols) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) dst[j] = v[j];
      }
    }
  }
}

// Token rows x [T][K] (bf16, row stride ld) -> the GEMM's token operand: E4M3
// codes (128 kt bytes per row) or E2M1 codes (64 kt bytes), zeros past K, and
// the scales of each token tile (kt x RA tiles of 512 bytes per token tile,
// the 128-row halves of a k tile together).
//
// ROUTED: token t's row is written at the positions slot_pos[t k + r] of its k
// slots, in the scale tile of that expert (rows of an expert are cut into
// tiles by token_tile_rows), and once in token order for a shared expert
// (shared_q). Otherwise at row t. One thread = 8 elements of one token; the
// element work is done once for all k copies.
template <bool ROUTED, bool E2M1>
__global__ void __launch_bounds__(256) quantize_tokens_kernel(MxTokenArgs a) {
  pdl_entry();
  const int lane = threadIdx.x & 31;
  const int kt = (int)mxfp4_k_tiles(a.K);
  const int per_row = kt * 16;
  const int64_t n = ((int64_t)a.T * per_row + 31) / 32 * 32;
  const int code_row = (E2M1 ? 64 : 128) * kt;
  const int P = a.T * a.k;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int t = (int)(i / per_row);
    const int c8 = (int)(i - (int64_t)t * per_row);
    const bool live = t < a.T;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live)
      load8(reinterpret_cast<const __nv_bfloat16*>(a.x) + (int64_t)t * a.ld, (int64_t)c8 * 8, a.K,
            a.vec != 0, v);
    const uint32_t byte = mx_scale_byte(block_amax_bits(v), E2M1 ? kTop4 : kTop8);
    const uint32_t word = gather_scale_word(byte, lane);
    const float inv = mx_inv_scale(byte);
    uint2 codes;
    if constexpr (E2M1)
      codes = make_uint2(encode8_e2m1(v, inv), 0);
    else
      codes = encode8_e4m3(v, inv);
    if (!live) continue;
    auto put = [&](uint8_t* q, uint8_t* s, int64_t row, int64_t tile, int j) {
      if constexpr (E2M1)
        *reinterpret_cast<uint32_t*>(q + row * code_row + c8 * 4) = codes.x;
      else
        *reinterpret_cast<uint2*>(q + row * code_row + c8 * 8) = codes;
      if ((c8 & 15) == 0)
        *reinterpret_cast<uint32_t*>(s + ((tile * kt + (c8 >> 4)) * a.tiling.row_atoms + (j >> 7)) * 512 +
                                     mxfp4_scale_word((uint32_t)(j & 127))) = word;
    };
    if constexpr (ROUTED) {
      for (int r = 0; r < a.k; ++r) {
        const int64_t slot = (int64_t)t * a.k + r;
        const int p = a.slot_pos[slot], e = a.topk_ids[slot];
        if ((unsigned)p >= (unsigned)P || (unsigned)e >= (unsigned)a.E) {
          if (c8 == 0) set_status(a.status, MOE_ERR_DEVICE_CHECK);
          continue;
        }
        const int first = a.offsets[e], m = a.offsets[e + 1] - first;
        const int local = p - first;
        if (local < 0 || local >= m) {
          if (c8 == 0) set_status(a.status, MOE_ERR_DEVICE_CHECK);
          continue;
        }
        const int tn = token_tile_rows(m, a.tiling.rows, a.tiling.unit);
        const int mt = local / tn;
        put(a.q, a.s, p, group_scale_tile(first, e, a.tiling.rows) + mt, local - mt * tn);
      }
    }
    if (!ROUTED || a.shared_q) {
      const int tn = token_tile_rows(a.T, a.tiling.rows, a.tiling.unit);
      const int mt = t / tn;
      put(ROUTED ? a.shared_q : a.q, ROUTED ? a.shared_s : a.s, t, mt, t - mt * tn);
    }
  }
}

unsigned grid_for(int64_t n, int num_sms) {
  int64_t blocks = (n + 255) / 256;
  const int64_t cap = 32 * (int64_t)num_sms;
  if (blocks > cap) blocks = cap;
  return (unsigned)(blocks < 1 ? 1 : blocks);
}

bool vec_ok(const void* p, int64_t ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * es % 16 == 0;
}

}  // namespace

cudaError_t launch_quantize_mxfp4(int dtype, const void* src, const void* src2, int64_t rows,
                                  int64_t cols, int64_t ld, int64_t I, uint8_t* q, uint8_t* scales,
                                  int num_sms, cudaStream_t st) {
  const unsigned g = grid_for((rows + 127) / 128 * 128 * mxfp4_k_tiles(cols) * 16, num_sms);
  auto run = [&](auto kernel, auto tag) {
    using T = decltype(tag);
    const bool vec = vec_ok(src, ld, sizeof(T)) && (!src2 || vec_ok(src2, ld, sizeof(T)));
    return launch_chained(kernel, dim3(g), dim3(256), 0, st, 1, (const T*)src, (const T*)src2,
                          rows, cols, ld, I, vec, q, scales);
  };
  if (dtype == MOE_DTYPE_BF16)
    return src2 ? run(quantize_mxfp4_kernel<__nv_bfloat16, true>, __nv_bfloat16())
                : run(quantize_mxfp4_kernel<__nv_bfloat16, false>, __nv_bfloat16());
  return src2 ? run(quantize_mxfp4_kernel<float, true>, float())
              : run(quantize_mxfp4_kernel<float, false>, float());
}

cudaError_t launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* scales, int64_t rows,
                                    int64_t cols, int dtype, void* out, int64_t ld, int num_sms,
                                    cudaStream_t st) {
  const unsigned g = grid_for(rows * ((cols + 7) / 8), num_sms);
  if (dtype == MOE_DTYPE_BF16)
    return launch_chained(dequantize_mxfp4_kernel<__nv_bfloat16>, dim3(g), dim3(256), 0, st, 1, q,
                          scales, rows, cols, (__nv_bfloat16*)out, ld, vec_ok(out, ld, 2));
  return launch_chained(dequantize_mxfp4_kernel<float>, dim3(g), dim3(256), 0, st, 1, q, scales,
                        rows, cols, (float*)out, ld, vec_ok(out, ld, 4));
}

cudaError_t launch_quantize_tokens(const MxTokenArgs& args, bool routed, bool e2m1, int num_sms,
                                   cudaStream_t st) {
  MxTokenArgs a = args;
  if (a.T == 0) return cudaSuccess;
  a.vec = vec_ok(a.x, a.ld, 2) ? 1 : 0;
  const unsigned g = grid_for((int64_t)a.T * mxfp4_k_tiles(a.K) * 16, num_sms);
  auto fn = routed ? quantize_tokens_kernel<true, false>
                   : (e2m1 ? quantize_tokens_kernel<false, true>
                           : quantize_tokens_kernel<false, false>);
  return launch_chained(fn, dim3(g), dim3(256), 0, st, 1, a);
}

}  // namespace moe
