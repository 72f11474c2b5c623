// Quantisers of MXFP4 vectors and of 4-bit main-KV rows, and their inverses (formats in mx4.cuh;
// [SW] shareware.cn/news/167317 §六.1, §十三.4).
//
// All four stream memory: a value is read once and its code written once.  A lane takes eight
// neighbouring values (16 or 32 bytes a load), so four lanes hold a block: its largest magnitude
// is two shuffles (compared as integers: the order of non-negative floats, and an infinity or a
// NaN stays the largest), and a warp's loads and code stores are contiguous.
// (Sixteen values a lane halve the shuffles, but the loads were no longer contiguous: slower.)
// Measured, quantised and back: 262144 x 64 bf16, 85 MB in 15.0 us, 5.65 TB/s, 0.86 of the copy rate;
// 262144 main-KV rows from bf16, 361 MB in 75 us, 4.8 TB/s, 0.73 (issue active 68 % of the cycles);
// a few rows: the latency of two launches, 2.1 us.
#include "launch.cuh"
#include "mx4.cuh"

namespace cskv {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;                          // 256-value pieces of a warp in flight
constexpr int kMxWarpValues = 256 * kMxUnroll;        // values a warp takes
constexpr int kMxCtaValues = kMxWarpValues * (kMxThreads / 32);

// Largest magnitude (as bits; an infinity or a NaN stays the largest) of the four lanes that hold a
// block.
__device__ __forceinline__ uint32_t block_amax(const float (&x)[8]) {
  float a = fabsf(x[0]), b = fabsf(x[4]);
#pragma unroll
  for (int i = 1; i < 4; ++i) a = amax_nan(a, x[i]), b = amax_nan(b, x[4 + i]);
  uint32_t m = __float_as_uint(amax_nan(a, b));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// x * 2^(127 - e) for the conversion.
__device__ __forceinline__ void scale_down(float (&x)[8], uint32_t e) {
  const float inv = mx_inv_scale(e);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv;
}

// Eight decoded values of a lane, stored: bf16 pairs straight from the codes, fp32 by value.
__device__ __forceinline__ void store_e2m1x8(__nv_bfloat16* to, uint32_t w, uint32_t e) {
  *reinterpret_cast<uint4*>(to) = e2m1x8_bf16(w, scale_bf16x2(e));
}
__device__ __forceinline__ void store_e2m1x8(float* to, uint32_t w, uint32_t e) {
  const float s = mx_scale(e);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = e2m1_value(w >> (4 * i)) * s;
  Vec8<float>::store(to, f);
}
__device__ __forceinline__ void store_e4m3x8(__nv_bfloat16* to, uint32_t w0, uint32_t w1, uint32_t e) {
  *reinterpret_cast<uint4*>(to) = e4m3x8_bf16(w0, w1, scale_bf16x2(e));
}
__device__ __forceinline__ void store_e4m3x8(float* to, uint32_t w0, uint32_t w1, uint32_t e) {
  const float s = mx_scale(e);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = e4m3_value((i < 4 ? w0 : w1) >> (8 * (i & 3))) * s;
  Vec8<float>::store(to, f);
}

template <typename T>
__global__ void __launch_bounds__(kMxThreads) mxfp4_quantize_kernel(const T* __restrict__ x, int64_t blocks,
                                                                    uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  // first block of this warp; a lane's piece u is block b0 + 8u + lane/4, values 8 (lane % 4) ..
  const int64_t b0 = ((int64_t)blockIdx.x * kMxCtaValues + (threadIdx.x >> 5) * kMxWarpValues) / kMxBlock;
  const T* from = x + b0 * kMxBlock + 8 * lane;
  uint8_t* to = codes + b0 * (kMxBlock / 2) + 4 * lane;
  const int left = (int)min((int64_t)(8 * kMxUnroll), blocks - b0) - (lane >> 2);  // blocks from this lane's first on
  float f[kMxUnroll][8];
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u) {
    if (left > 8 * u)
      Vec8<T>::load(from + 256 * u, f[u]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) f[u][i] = 0.f;
  }
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u) {
    const uint32_t e = mx_scale_code(block_amax(f[u]), kE2m1Emax);
    scale_down(f[u], e);
    if ((lane & 3) == u) mine = e;
    if (left > 8 * u) *reinterpret_cast<uint32_t*>(to + 128 * u) = e == 0xFFu ? 0u : e2m1x8(f[u]);
  }
  // lane l keeps the scale of piece l % 4, block l / 4: a warp's 32 scale bytes in one store
  const int64_t b = b0 + 8 * (lane & 3) + (lane >> 2);
  if (b < blocks) scales[b] = (uint8_t)mine;
}

template <typename T>
__global__ void __launch_bounds__(kMxThreads) mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales,
                                                                      int64_t blocks, T* __restrict__ out) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t b0 = ((int64_t)blockIdx.x * kMxCtaValues + (threadIdx.x >> 5) * kMxWarpValues) / kMxBlock;
  const uint8_t *from = codes + b0 * (kMxBlock / 2) + 4 * lane, *sc = scales + b0 + (lane >> 2);
  T* to = out + b0 * kMxBlock + 8 * lane;
  const int left = (int)min((int64_t)(8 * kMxUnroll), blocks - b0) - (lane >> 2);  // blocks from this lane's first on
  uint32_t w[kMxUnroll], e[kMxUnroll];
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u) {
    w[u] = left > 8 * u ? __ldg(reinterpret_cast<const uint32_t*>(from + 128 * u)) : 0u;
    e[u] = left > 8 * u ? __ldg(sc + 8 * u) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u)
    if (left > 8 * u) store_e2m1x8(to + 256 * u, w[u], e[u]);
}

// ---------------------------------------------------------------- 4-bit main-KV rows
// A warp takes four rows as four groups of 32 lanes with eight values each: three groups are the
// rows' 96 E2M1 pieces, one their 32 E4M3 pieces, so no lane waits for the other format's code
// (with a row a warp both codes ran for every row, and the kernels were bound by issue: 41 and 44 us
// for 262144 rows).
constexpr int kKv4Warps = 8;
constexpr int kKv4Rows = 4;

// Piece of a lane in group j: the row among the warp's four, and where its eight values, its codes
// and its block's scale sit in a row.
struct Kv4Piece {
  int row, value, code, scale;
};
__device__ __forceinline__ Kv4Piece kv4_piece(int j, int lane) {
  Kv4Piece p;
  if (j < 3) {
    const int i = lane + 32 * j, part = i % 24;  // K dims 0..63: 8 pieces, V: 16
    p.row = i / 24;
    p.value = 8 * part + (part < 8 ? 0 : 64);
    p.code = part < 8 ? 4 * part : kKv4V + 4 * (part - 8);
  } else {
    p.row = lane >> 3;
    p.value = 64 + 8 * (lane & 7);
    p.code = kKv4Rope + 8 * (lane & 7);
  }
  p.scale = kKv4Scales + (p.value >> 5);
  return p;
}

template <typename T>
__global__ void __launch_bounds__(32 * kKv4Warps) kv_quantize_fp4_kernel(const T* __restrict__ rows, int64_t n,
                                                                        const int64_t* __restrict__ dst, int64_t cap,
                                                                        uint8_t* __restrict__ out, int* st) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows;
  if (r0 >= n) return;
  const int here = (int)min((int64_t)kKv4Rows, n - r0);  // rows of this warp
  const T* from = rows + (size_t)r0 * kRow;
  float x[4][8];
  int64_t to[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Kv4Piece q = kv4_piece(j, lane);
    // past the end: the warp's first row again, not stored
    const int row = q.row < here ? q.row : 0;
    to[j] = dst ? __ldg(dst + r0 + row) : r0 + row;
    Vec8<T>::load(from + (row * kRow + q.value), x[j]);
    if (q.row >= here) to[j] = -1;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Kv4Piece q = kv4_piece(j, lane);
    const uint32_t e = mx_scale_code(block_amax(x[j]), j == 3 ? kE4m3Emax : kE2m1Emax);
    scale_down(x[j], e);
    if (to[j] < 0) continue;
    if (to[j] >= cap) {
      if (q.value == 64) flag(st, CSKV_DEV_BAD_INDEX);  // once a row
      continue;
    }
    uint8_t* o = out + (size_t)to[j] * kKv4RowBytes;
    if (j == 3) {
      const uint2 w = e4m3x8(x[j]);
      *reinterpret_cast<uint2*>(o + q.code) = e == 0xFFu ? make_uint2(0u, 0u) : w;
    } else {
      *reinterpret_cast<uint32_t*>(o + q.code) = e == 0xFFu ? 0u : e2m1x8(x[j]);
    }
    // a block's first lane stores its scale, its second one zero byte of the row's end
    if ((lane & 3) < 2) o[q.scale + ((lane & 1) ? 8 : 0)] = (lane & 1) ? 0 : (uint8_t)e;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kKv4Warps) kv_dequantize_fp4_kernel(const uint8_t* __restrict__ cache,
                                                                          const int64_t* __restrict__ src,
                                                                          int64_t cap, int64_t n,
                                                                          T* __restrict__ out, int* st) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows;
  if (r0 >= n) return;
  const int here = (int)min((int64_t)kKv4Rows, n - r0);  // rows of this warp
  // all groups' loads go out before the first is decoded
  uint2 w[4];
  uint32_t e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Kv4Piece q = kv4_piece(j, lane);
    int64_t i = q.row >= here ? -1 : src ? __ldg(src + r0 + q.row) : r0 + q.row;
    if (i >= cap) {
      if (q.value == 64) flag(st, CSKV_DEV_BAD_INDEX);  // once a row
      i = -1;
    }
    const uint8_t* row = cache + (size_t)(i < 0 ? 0 : i) * kKv4RowBytes;
    if (j == 3)
      w[j] = i < 0 ? make_uint2(0u, 0u) : __ldg(reinterpret_cast<const uint2*>(row + q.code));
    else
      w[j] = make_uint2(i < 0 ? 0u : __ldg(reinterpret_cast<const uint32_t*>(row + q.code)), 0u);
    e[j] = i < 0 ? 127u : __ldg(row + q.scale);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Kv4Piece q = kv4_piece(j, lane);
    if (q.row >= here) continue;
    T* to = out + (size_t)r0 * kRow + (q.row * kRow + q.value);
    if (j == 3)
      store_e4m3x8(to, w[j].x, w[j].y, e[j]);
    else
      store_e2m1x8(to, w[j].x, e[j]);
  }
}

// ---------------------------------------------------------------- launchers
template <typename... KArgs, typename... Args>
static cudaError_t launch_1d(void (*kern)(KArgs...), int64_t ctas, int threads, cudaStream_t stream, Args... args) {
  cudaError_t e = ensure_smem(kern, 0);
  if (e == cudaSuccess) e = launch_dependent(kern, dim3((unsigned)ctas), dim3(threads), 0, stream, args...);
  note_launch();
  return e;
}

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t blocks, uint8_t* codes, uint8_t* scales,
                                  cudaStream_t stream) {
  const int64_t ctas = (blocks * kMxBlock + kMxCtaValues - 1) / kMxCtaValues;
  return dtype == CSKV_F32
             ? launch_1d(mxfp4_quantize_kernel<float>, ctas, kMxThreads, stream, (const float*)x, blocks, codes, scales)
             : launch_1d(mxfp4_quantize_kernel<__nv_bfloat16>, ctas, kMxThreads, stream, (const __nv_bfloat16*)x,
                         blocks, codes, scales);
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks, int dtype, void* out,
                                    cudaStream_t stream) {
  const int64_t ctas = (blocks * kMxBlock + kMxCtaValues - 1) / kMxCtaValues;
  return dtype == CSKV_F32
             ? launch_1d(mxfp4_dequantize_kernel<float>, ctas, kMxThreads, stream, codes, scales, blocks, (float*)out)
             : launch_1d(mxfp4_dequantize_kernel<__nv_bfloat16>, ctas, kMxThreads, stream, codes, scales, blocks,
                         (__nv_bfloat16*)out);
}

cudaError_t launch_kv_quantize_fp4(const void* rows, int dtype, int64_t n, const int64_t* dst, int64_t cap,
                                   uint8_t* out, int* st, cudaStream_t stream) {
  const int64_t ctas = (n + kKv4Warps * kKv4Rows - 1) / (kKv4Warps * kKv4Rows);
  return dtype == CSKV_F32 ? launch_1d(kv_quantize_fp4_kernel<float>, ctas, 32 * kKv4Warps, stream, (const float*)rows,
                                       n, dst, cap, out, st)
                           : launch_1d(kv_quantize_fp4_kernel<__nv_bfloat16>, ctas, 32 * kKv4Warps, stream,
                                       (const __nv_bfloat16*)rows, n, dst, cap, out, st);
}

cudaError_t launch_kv_dequantize_fp4(const uint8_t* cache, const int64_t* src, int64_t cap, int64_t n, int dtype,
                                     void* out, int* st, cudaStream_t stream) {
  const int64_t ctas = (n + kKv4Warps * kKv4Rows - 1) / (kKv4Warps * kKv4Rows);
  return dtype == CSKV_F32 ? launch_1d(kv_dequantize_fp4_kernel<float>, ctas, 32 * kKv4Warps, stream, cache, src, cap,
                                       n, (float*)out, st)
                           : launch_1d(kv_dequantize_fp4_kernel<__nv_bfloat16>, ctas, 32 * kKv4Warps, stream, cache,
                                       src, cap, n, (__nv_bfloat16*)out, st);
}

}  // namespace cskv
