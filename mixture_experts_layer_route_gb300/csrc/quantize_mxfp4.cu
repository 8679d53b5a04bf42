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

// Eight consecutive elements of a row as loaded, and what a block needs of them.
template <typename T>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  // n elements of a row that 16-byte loads may not take, zeros after them.
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < n ? (uint32_t)h[2 * i] : 0u) |
             (2 * i + 1 < n ? (uint32_t)h[2 * i + 1] << 16 : 0u);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // fp32 bits of the largest magnitude of the block that four lanes hold (two
  // 16-bit maxima per instruction).
  __device__ __forceinline__ uint32_t block_amax_bits() const {
    const uint32_t k = 0x7FFF7FFFu;
    uint32_t m = __vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void scaled(float inv, float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16) * inv;
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
    }
  }
};

template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_some(const float* p, int n) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  // Unsigned bit patterns order magnitudes with infinities and NaNs on top,
  // which a float maximum would drop.
  __device__ __forceinline__ uint32_t block_amax_bits() const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  }
  __device__ __forceinline__ void scaled(float inv, float (&v)[8]) const {
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i] * inv;
  }
};

// Codes of eight scaled elements; a NaN block (scale byte 255) has zeros.
template <typename T>
__device__ __forceinline__ uint32_t encode8_e2m1(const Raw8<T>& r, uint32_t byte) {
  float v[8];
  r.scaled(mx_inv_scale(byte), v);
  uint32_t w = e2m1_pair(v[0], v[1]) | e2m1_pair(v[2], v[3]) << 8 | e2m1_pair(v[4], v[5]) << 16 |
               e2m1_pair(v[6], v[7]) << 24;
  return byte == 255u ? 0u : w;
}
template <typename T>
__device__ __forceinline__ uint2 encode8_e4m3(const Raw8<T>& r, uint32_t byte) {
  float v[8];
  r.scaled(mx_inv_scale(byte), v);
  const uint2 w = make_uint2(mx_encode4(v[0], v[1], v[2], v[3]), mx_encode4(v[4], v[5], v[6], v[7]));
  return byte == 255u ? make_uint2(0, 0) : w;
}

// Blocks are (x: groups of 8 elements of a row, y: rows), so that no thread
// divides; a thread walks down its column with a few rows' loads in flight.
// src [rows][cols] with row stride ld -> codes and tiled scales. PAIRED: row R
// of the result comes from two matrices (gate, up) of groups of I rows, whose
// rows alternate in runs of 64. VEC: rows are 16-byte aligned and whole groups.
template <typename TIn, bool PAIRED, bool VEC>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(
    const TIn* __restrict__ src, const TIn* __restrict__ src2, int64_t rows, int64_t cols,
    int64_t ld, int64_t I, uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  constexpr int AHEAD = sizeof(TIn) == 2 ? 4 : 2;
  pdl_entry();
  const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
  const int64_t kt = mxfp4_k_tiles(cols);
  const int64_t c8 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;  // a warp's 32 are in or
  const bool in = c8 < kt * 16;                                       // out by halves of 16
  const int left = (int)min((int64_t)8, cols - c8 * 8);               // elements of this group
  const int64_t padded = (rows + 127) / 128 * 128;  // rows of the scale tiles
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  auto group_of = [&](int64_t r) {
    const TIn* p;
    if constexpr (PAIRED) {
      const int64_t e = r / (2 * I), w = r - e * 2 * I;
      p = (((w >> 6) & 1) ? src2 : src) + (e * I + (w >> 7) * 64 + (w & 63)) * ld;
    } else {
      p = src + r * ld;
    }
    return p + c8 * 8;
  };
  // The trip count is the same for all rows of a warp: it counts blocks of rows.
  int64_t r0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
  for (int64_t rb = (int64_t)blockIdx.y * blockDim.y; rb < padded;
       rb += AHEAD * step, r0 += AHEAD * step) {
    Raw8<TIn> v[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int64_t r = r0 + j * step;
      v[j].zero();
      if (in && r < rows && left > 0) {
        if constexpr (VEC)
          v[j].load(group_of(r));
        else
          v[j].load_some(group_of(r), left);
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int64_t r = r0 + j * step;
      const uint32_t byte = mx_scale_byte(v[j].block_amax_bits(), kTop4);
      if (!in) continue;
      if (r < rows)
        *reinterpret_cast<uint32_t*>(q + r * (kt * 64) + c8 * 4) = encode8_e2m1(v[j], byte);
      if (r < padded && (lane & 3) == 0)
        scales[((r >> 7) * kt + (c8 >> 4)) * 512 + mxfp4_scale_word((uint32_t)(r & 127)) +
               ((c8 >> 2) & 3)] = (uint8_t)byte;
    }
  }
}

// VEC: rows of out are 16-byte aligned and whole groups of 8.
template <typename TOut, bool VEC>
__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ scales,
                                                               int64_t rows, int64_t cols,
                                                               TOut* __restrict__ out,
                                                               int64_t ld) {
  constexpr int AHEAD = 4;
  pdl_entry();
  const int64_t kt = mxfp4_k_tiles(cols);
  const int64_t c8 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, c = c8 * 8;
  if (c >= cols) return;
  const int left = (int)min((int64_t)8, cols - c);
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  for (int64_t r0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r0 < rows;
       r0 += AHEAD * step) {
    uint32_t w[AHEAD], byte[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int64_t r = r0 + j * step;
      w[j] = byte[j] = 0;
      if (r >= rows) continue;
      w[j] = *reinterpret_cast<const uint32_t*>(q + r * (kt * 64) + c8 * 4);
      byte[j] = scales[((r >> 7) * kt + (c8 >> 4)) * 512 + mxfp4_scale_word((uint32_t)(r & 127)) +
                       ((c8 >> 2) & 3)];
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
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
      if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) {
            if constexpr (sizeof(TOut) == 2)
              dst[i] = __float2bfloat16_rn(v[i]);
            else
              dst[i] = v[i];
          }
      } else if constexpr (sizeof(TOut) == 2) {
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
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n_zero;
         i += (int64_t)gridDim.x * 256)
      a.zero[i] = 0;
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
  if (!ROUTED && a.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;
  if (threadIdx.x == 32) {  // the row in token order
    const int tn = token_tile_rows(a.T, a.tiling.rows, a.tiling.unit);
    const int mt = t / tn;
    dest[ROUTED ? 32 : 0] = {t, mt, t - mt * tn};
  }
  const bool in = c8 < per_row;
  Raw8<__nv_bfloat16> v;
  v.zero();
  const int left = min(8, a.K - c8 * 8);  // elements of this group
  if (in && left > 0) {
    const __nv_bfloat16* p =
        reinterpret_cast<const __nv_bfloat16*>(a.x) + (int64_t)t * a.ld + c8 * 8;
    if (a.vec && left == 8)
      v.load(p);
    else
      v.load_some(p, left);
  }
  const uint32_t byte = mx_scale_byte(v.block_amax_bits(), E2M1 ? kTop4 : kTop8);
  uint32_t word = byte << (8 * ((lane >> 2) & 3));  // the k tile's four scale bytes
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
  uint2 codes;
  if constexpr (E2M1)
    codes = make_uint2(encode8_e2m1(v, byte), 0);
  else
    codes = encode8_e4m3(v, byte);
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

// y[t][c] = sum_r topk_w[t][r] slot[slot_pos[t][r]][c], in rank order, then the
// shared expert's slot. A block takes 2048 features of one token (8 a thread),
// looks its positions and weights up once, and has four slots' loads in flight
// a thread. A position out of range is reported and its slot left out.
template <typename TOut>
__global__ void __launch_bounds__(256) combine_slots_kernel(
    const int16_t* __restrict__ q, const uint8_t* __restrict__ s,
    const int32_t* __restrict__ slot_pos, const float* __restrict__ topk_w, int T, int k, int H,
    int shared, TOut* __restrict__ y, int* status) {
  pdl_entry();
  __shared__ int pos[33];
  __shared__ float weight[33];
  const int P = T * k;
  const int chunks = (H / 8 + 255) / 256;
  const int t = (int)(blockIdx.x / (unsigned)chunks);
  const int c8 = (int)(blockIdx.x - (unsigned)t * chunks) * 256 + (int)threadIdx.x;
  const int KP = k + shared;
  if ((int)threadIdx.x < KP) {
    int p = P + t;
    float w = 1.0f;
    if ((int)threadIdx.x < k) {
      p = slot_pos[(int64_t)t * k + threadIdx.x];
      w = topk_w[(int64_t)t * k + threadIdx.x];
      if ((unsigned)p >= (unsigned)P) {
        set_status(status, MOE_ERR_DEVICE_CHECK);
        p = -1;
      }
    }
    pos[threadIdx.x] = p;
    weight[threadIdx.x] = w;
  }
  __syncthreads();
  if (c8 >= H / 8) return;
  const uint4* src = reinterpret_cast<const uint4*>(q) + c8;
  const uint8_t* sc = s + (c8 >> 2);
  float a[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j0 = 0; j0 < KP; j0 += 4) {
    uint4 u[4];
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = j0 + j < KP ? pos[j0 + j] : -1;
      u[j] = p >= 0 ? __ldcs(src + (int64_t)p * (H / 8)) : make_uint4(0, 0, 0, 0);
      b[j] = p >= 0 ? sc[(int64_t)p * (H / 32)] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j0 + j >= KP) continue;
      const float x = mx_scale_or_nan(b[j]) * weight[j0 + j];
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = slot_codes(w[i]);
        a[2 * i] = __fmaf_rn(v.x, x, a[2 * i]);
        a[2 * i + 1] = __fmaf_rn(v.y, x, a[2 * i + 1]);
      }
    }
  }
  const int64_t at = (int64_t)t * (H / 8) + c8;
  if constexpr (sizeof(TOut) == 2) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    reinterpret_cast<uint4*>(y)[at] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    reinterpret_cast<float4*>(y)[2 * at] = make_float4(a[0], a[1], a[2], a[3]);
    reinterpret_cast<float4*>(y)[2 * at + 1] = make_float4(a[4], a[5], a[6], a[7]);
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
  auto run = [&](auto tag) {
    using T = decltype(tag);
    const bool vec = cols % 8 == 0 && vec_ok(src, ld, sizeof(T)) &&
                     (!src2 || vec_ok(src2, ld, sizeof(T)));
    auto fn = src2 ? (vec ? quantize_mxfp4_kernel<T, true, true>
                          : quantize_mxfp4_kernel<T, true, false>)
                   : (vec ? quantize_mxfp4_kernel<T, false, true>
                          : quantize_mxfp4_kernel<T, false, false>);
    return launch_chained(fn, g.grid, g.block, 0, st, 1, (const T*)src, (const T*)src2, rows, cols,
                          ld, I, q, scales);
  };
  return dtype == MOE_DTYPE_BF16 ? run(__nv_bfloat16()) : run(float());
}

cudaError_t launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* scales, int64_t rows,
                                    int64_t cols, int dtype, void* out, int64_t ld, int num_sms,
                                    cudaStream_t st) {
  const RowGrid g = row_grid((cols + 7) / 8, rows, num_sms);
  auto run = [&](auto tag) {
    using T = decltype(tag);
    const bool vec = cols % 8 == 0 && vec_ok(out, ld, sizeof(T));
    auto fn = vec ? dequantize_mxfp4_kernel<T, true> : dequantize_mxfp4_kernel<T, false>;
    return launch_chained(fn, g.grid, g.block, 0, st, 1, q, scales, rows, cols, (T*)out, ld);
  };
  return dtype == MOE_DTYPE_BF16 ? run(__nv_bfloat16()) : run(float());
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

cudaError_t launch_mx4_combine(const Mx4Slots& s, const int32_t* slot_pos, const float* topk_w,
                               int T, int k, int H, bool shared, bool out_f32, void* y,
                               int* status, cudaStream_t st) {
  const int64_t blocks = (int64_t)T * ((H / 8 + 255) / 256);
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
  const dim3 g((unsigned)blocks), b(256);
  if (out_f32)
    return launch_chained(combine_slots_kernel<float>, g, b, 0, st, 1, (const int16_t*)s.q,
                          (const uint8_t*)s.s, slot_pos, topk_w, T, k, H, shared ? 1 : 0,
                          (float*)y, status);
  return launch_chained(combine_slots_kernel<__nv_bfloat16>, g, b, 0, st, 1, (const int16_t*)s.q,
                        (const uint8_t*)s.s, slot_pos, topk_w, T, k, H, shared ? 1 : 0,
                        (__nv_bfloat16*)y, status);
}

}  // namespace moe
