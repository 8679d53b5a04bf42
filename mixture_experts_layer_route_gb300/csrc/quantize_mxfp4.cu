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

// Blocks are (x: groups of 8 elements of a row, y: rows), so that no thread
// divides; a thread walks down its column with kRowsAhead rows' loads in flight.
constexpr int kRowsAhead = 4;

// src [rows][cols] with row stride ld -> codes and tiled scales. PAIRED: row R
// of the result comes from two matrices (gate, up) of groups of I rows, whose
// rows alternate in runs of 64.
template <typename TIn, bool PAIRED>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(
    const TIn* __restrict__ src, const TIn* __restrict__ src2, int64_t rows, int64_t cols,
    int64_t ld, int64_t I, bool vec, uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  pdl_entry();
  const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
  const int64_t kt = mxfp4_k_tiles(cols);
  const int64_t c8 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;  // a warp's 32 are in or
  const bool in = c8 < kt * 16;                                       // out by halves of 16
  const int64_t padded = (rows + 127) / 128 * 128;  // rows of the scale tiles
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  auto row_of = [&](int64_t r) {
    if constexpr (PAIRED) {
      const int64_t e = r / (2 * I), w = r - e * 2 * I;
      return (((w >> 6) & 1) ? src2 : src) + (e * I + (w >> 7) * 64 + (w & 63)) * ld;
    } else {
      return src + r * ld;
    }
  };
  // The loop's trip count is the same for all rows of a warp: the bound below
  // counts whole blocks of rows.
  const int64_t r0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
  for (int64_t rb = (int64_t)blockIdx.y * blockDim.y; rb < padded; rb += kRowsAhead * step) {
    float v[kRowsAhead][8];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const int64_t r = r0 + (rb - (int64_t)blockIdx.y * blockDim.y) + j * step;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (in && r < rows) load8(row_of(r), c8 * 8, cols, vec, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const int64_t r = r0 + (rb - (int64_t)blockIdx.y * blockDim.y) + j * step;
      const uint32_t byte = mx_scale_byte(block_amax_bits(v[j]), kTop4);
      const uint32_t word = gather_scale_word(byte, lane);
      if (in && r < rows)
        *reinterpret_cast<uint32_t*>(q + r * (kt * 64) + c8 * 4) =
            encode8_e2m1(v[j], mx_inv_scale(byte));
      if (in && r < padded && (lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(scales + ((r >> 7) * kt + (c8 >> 4)) * 512 +
                                     mxfp4_scale_word((uint32_t)(r & 127))) = word;
    }
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
  const int64_t c8 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, c = c8 * 8;
  if (c >= cols) return;
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  for (int64_t r0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r0 < rows;
       r0 += kRowsAhead * step) {
    uint32_t w[kRowsAhead], byte[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const int64_t r = r0 + j * step;
      if (r >= rows) continue;
      w[j] = *reinterpret_cast<const uint32_t*>(q + r * (kt * 64) + c8 * 4);
      byte[j] = scales[((r >> 7) * kt + (c8 >> 4)) * 512 + mxfp4_scale_word((uint32_t)(r & 127)) +
                       ((c8 >> 2) & 3)];
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const int64_t r = r0 + j * step;
      if (r >= rows) continue;
      const float s = mx_scale_or_nan(byte[j]);
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e2m1_values(w[j] >> (8 * i));
        v[2 * i] = f.x * s;  // exact: two significant bits, exponents of bf16 and fp32
        v[2 * i + 1] = f.y * s;
      }
      TOut* dst = out + r * ld + c;
      if (vec && c + 8 <= cols) {
        if constexpr (sizeof(TOut) == 2) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < cols) {
            if constexpr (sizeof(TOut) == 2)
              dst[i] = __float2bfloat16_rn(v[i]);
            else
              dst[i] = v[i];
          }
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
// (shared_q). Otherwise at row t. A block takes 2048 elements of one token (8 a
// thread); its first threads look the k destinations up once for all of it (a
// look-up per thread took four times as long as the copies), and the element
// work is done once for all k copies.
template <bool ROUTED, bool E2M1>
__global__ void __launch_bounds__(256) quantize_tokens_kernel(MxTokenArgs a) {
  pdl_entry();
  struct Dest {
    int64_t row, tile;  // row < 0: none
    int j;              // row inside the token tile
  };
  __shared__ Dest dest[ROUTED ? 33 : 1];
  const int lane = threadIdx.x & 31;
  const int kt = (int)mxfp4_k_tiles(a.K);
  const int per_row = kt * 16;
  const int chunks = (per_row + 255) / 256;
  const int t = (int)(blockIdx.x / (unsigned)chunks);
  const int c8 = (int)(blockIdx.x - (unsigned)t * chunks) * 256 + (int)threadIdx.x;
  const int code_row = (E2M1 ? 64 : 128) * kt;
  if constexpr (ROUTED) {
    if ((int)threadIdx.x < a.k) {
      const int64_t slot = (int64_t)t * a.k + threadIdx.x;
      const int p = a.slot_pos[slot], e = a.topk_ids[slot];
      Dest d = {-1, 0, 0};
      if ((unsigned)e < (unsigned)a.E && (unsigned)p < (unsigned)(a.T * a.k)) {
        const int first = a.offsets[e], m = a.offsets[e + 1] - first;
        const int local = p - first;
        if (local >= 0 && local < m) {
          const int tn = token_tile_rows(m, a.tiling.rows, a.tiling.unit);
          const int mt = local / tn;
          d = {p, group_scale_tile(first, e, a.tiling.rows) + mt, local - mt * tn};
        }
      }
      if (d.row < 0) set_status(a.status, MOE_ERR_DEVICE_CHECK);
      dest[threadIdx.x] = d;
    }
  }
  if (threadIdx.x == 32) {  // the row in token order
    const int tn = token_tile_rows(a.T, a.tiling.rows, a.tiling.unit);
    const int mt = t / tn;
    dest[ROUTED ? 32 : 0] = {t, mt, t - mt * tn};
  }
  const bool in = c8 < per_row;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (in)
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
  __syncthreads();
  if (!in) return;
  auto put = [&](uint8_t* q, uint8_t* s, const Dest& d) {
    if (d.row < 0) return;
    if constexpr (E2M1)
      *reinterpret_cast<uint32_t*>(q + d.row * code_row + c8 * 4) = codes.x;
    else
      *reinterpret_cast<uint2*>(q + d.row * code_row + c8 * 8) = codes;
    if ((c8 & 15) == 0)
      *reinterpret_cast<uint32_t*>(
          s + ((d.tile * kt + (c8 >> 4)) * a.tiling.row_atoms + (d.j >> 7)) * 512 +
          mxfp4_scale_word((uint32_t)(d.j & 127))) = word;
  };
  if constexpr (ROUTED) {
    for (int r = 0; r < a.k; ++r) put(a.q, a.s, dest[r]);
    if (a.shared_q) put(a.shared_q, a.shared_s, dest[32]);
  } else {
    put(a.q, a.s, dest[0]);
  }
}

// Blocks of 256 threads over (8-element groups of a row, rows): as wide as the
// row up to 256 groups, enough rows in flight to fill the GPU eight blocks deep.
struct RowGrid {
  dim3 grid, block;
};
RowGrid row_grid(int64_t groups, int64_t rows, int num_sms) {
  unsigned bx = 16;
  while (bx < 256 && bx < groups) bx *= 2;
  const unsigned by = 256 / bx;
  const int64_t gx = (groups + bx - 1) / bx;
  int64_t gy = (rows + by - 1) / by;
  int64_t cap = (8 * (int64_t)num_sms + gx - 1) / gx;
  if (gy > cap) gy = cap;
  return {dim3((unsigned)gx, (unsigned)gy), dim3(bx, by)};
}

bool vec_ok(const void* p, int64_t ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * es % 16 == 0;
}

}  // namespace

cudaError_t launch_quantize_mxfp4(int dtype, const void* src, const void* src2, int64_t rows,
                                  int64_t cols, int64_t ld, int64_t I, uint8_t* q, uint8_t* scales,
                                  int num_sms, cudaStream_t st) {
  const RowGrid g = row_grid(mxfp4_k_tiles(cols) * 16, (rows + 127) / 128 * 128, num_sms);
  auto run = [&](auto kernel, auto tag) {
    using T = decltype(tag);
    const bool vec = vec_ok(src, ld, sizeof(T)) && (!src2 || vec_ok(src2, ld, sizeof(T)));
    return launch_chained(kernel, g.grid, g.block, 0, st, 1, (const T*)src, (const T*)src2,
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
  const RowGrid g = row_grid((cols + 7) / 8, rows, num_sms);
  if (dtype == MOE_DTYPE_BF16)
    return launch_chained(dequantize_mxfp4_kernel<__nv_bfloat16>, g.grid, g.block, 0, st, 1, q,
                          scales, rows, cols, (__nv_bfloat16*)out, ld, vec_ok(out, ld, 2));
  return launch_chained(dequantize_mxfp4_kernel<float>, g.grid, g.block, 0, st, 1, q, scales,
                        rows, cols, (float*)out, ld, vec_ok(out, ld, 4));
}

cudaError_t launch_quantize_tokens(const MxTokenArgs& args, bool routed, bool e2m1,
                                   cudaStream_t st) {
  MxTokenArgs a = args;
  if (a.T == 0) return cudaSuccess;
  a.vec = vec_ok(a.x, a.ld, 2) ? 1 : 0;
  const int64_t blocks = (int64_t)a.T * ((mxfp4_k_tiles(a.K) * 16 + 255) / 256);
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
  auto fn = routed ? quantize_tokens_kernel<true, false>
                   : (e2m1 ? quantize_tokens_kernel<false, true>
                           : quantize_tokens_kernel<false, false>);
  return launch_chained(fn, dim3((unsigned)blocks), dim3(256), 0, st, 1, a);
}

}  // namespace moe
