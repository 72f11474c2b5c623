// Quantisers of MXFP4 vectors and of 4-bit main-KV rows, and their inverses (formats in mx4.cuh;
// [SW] shareware.cn/news/167317 §六.1, §十三.4).
//
// All four stream memory: a value is read once and its code written once.  A lane takes eight
// neighbouring values (16 or 32 bytes a load), so four lanes hold a block: its largest magnitude
// is two shuffles (compared as integers: the order of non-negative floats, and an infinity or a
// NaN stays the largest), and a warp's loads and code stores are contiguous.
// (Sixteen values a lane halve the shuffles, but the loads were no longer contiguous: slower.)
// Measured, quantised and back: 262144 x 64 bf16, 85 MB in 15.2 us, 5.6 TB/s, 0.86 of the copy rate;
// 262144 main-KV rows from bf16, 180 MB in 34.5 us, 5.2 TB/s, 0.80, and back in 30 us, 6.0 TB/s, 0.92;
// a few rows: the latency of two launches, 2.4 us.
#include <algorithm>

#include "launch.cuh"
#include "mx4.cuh"

namespace cskv {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;                          // 256-value pieces of a warp in flight
constexpr int kMxWarpValues = 256 * kMxUnroll;        // values a warp takes
static_assert(kMxCtaValues == kMxWarpValues * (kMxThreads / 32));

// Eight neighbouring values as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
};

// Largest magnitude of the block that four lanes hold, as the bits of an fp32 value (an infinity or a NaN
// stays the largest).  bf16: in pairs.
__device__ __forceinline__ uint32_t amax_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t block_amax(const Raw8<__nv_bfloat16>& x) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = amax_nan_bf16x2(amax_nan_bf16x2(x.w.x & kAbs, x.w.y & kAbs), amax_nan_bf16x2(x.w.z & kAbs, x.w.w & kAbs));
  m = amax_nan_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = amax_nan_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t block_amax(const Raw8<float>& x) {
  const float a = amax_nan(amax_nan(amax_nan(fabsf(x.a.x), x.a.y), x.a.z), x.a.w);
  const float b = amax_nan(amax_nan(amax_nan(fabsf(x.b.x), x.b.y), x.b.z), x.b.w);
  uint32_t m = __float_as_uint(amax_nan(a, b));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// x * 2^(127 - e) for the conversion.
__device__ __forceinline__ void mul_pair(float a, float b, uint64_t s, float& x, float& y) {
  uint64_t d;
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tmul.rn.f32x2 %0, t, %3;\n\t}" : "=l"(d) : "f"(a), "f"(b), "l"(s));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t twice(float s) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(s));
  return d;
}
__device__ __forceinline__ void scaled_down(const Raw8<__nv_bfloat16>& r, uint32_t e, float (&x)[8]) {
  const uint64_t s = twice(mx_inv_scale(e));
  const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    mul_pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u), s, x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void scaled_down(const Raw8<float>& r, uint32_t e, float (&x)[8]) {
  const uint64_t s = twice(mx_inv_scale(e));
  mul_pair(r.a.x, r.a.y, s, x[0], x[1]), mul_pair(r.a.z, r.a.w, s, x[2], x[3]);
  mul_pair(r.b.x, r.b.y, s, x[4], x[5]), mul_pair(r.b.z, r.b.w, s, x[6], x[7]);
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
  Raw8<T> r[kMxUnroll] = {};
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u)
    if (left > 8 * u) r[u].load(from + 256 * u);
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < kMxUnroll; ++u) {
    const uint32_t e = mx_scale_code(block_amax(r[u]), kE2m1Emax);
    float f[8];
    scaled_down(r[u], e, f);
    if ((lane & 3) == u) mine = e;
    if (left > 8 * u) *reinterpret_cast<uint32_t*>(to + 128 * u) = e == 0xFFu ? 0u : e2m1x8(f);
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
// for 262144 rows; 37 and 37 with four rows a warp and no loop, whose address arithmetic was half of
// the instructions).
constexpr int kKv4Warps = 8;
constexpr int kKv4Rows = 4;
constexpr int64_t kKv4MostCtas = 16 * 148;  // a warp works out its pieces' places once, then strides over the rows

// Piece of a lane in group j: the row among the warp's four, and where its eight values, its codes
// and its block's scale sit (from the first row's values, and from its bytes).
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

// LIST: rows go to the cache rows of a list (elsewhere: to their own numbers).  A warp puts its four
// rows together in shared memory and stores them in 16-byte pieces, whole sectors of neighbouring rows
// (4-byte codes and single scale bytes, stored from the lanes that hold them, took 37 us for 262144 rows, this 34).
template <typename T, bool LIST>
__global__ void __launch_bounds__(32 * kKv4Warps) kv_quantize_fp4_kernel(const T* __restrict__ rows, int64_t n,
                                                                        const int64_t* __restrict__ dst, int64_t cap,
                                                                        uint8_t* __restrict__ out, int* st) {
  __shared__ uint4 made[kKv4Warps][kKv4Rows * kKv4RowBytes / 16];
  pdl_wait();
  const int lane = threadIdx.x & 31;
  uint4* mine = made[threadIdx.x >> 5];
  uint8_t* bytes = reinterpret_cast<uint8_t*>(mine);
  constexpr int kPieces = kKv4RowBytes / 16;  // 16-byte pieces of a row
  Kv4Piece q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = kv4_piece(j, lane);
  if (lane < kKv4Rows) *reinterpret_cast<uint2*>(bytes + lane * kKv4RowBytes + kKv4Scales + 8) = make_uint2(0u, 0u);
  const int64_t step = (int64_t)gridDim.x * kKv4Warps * kKv4Rows;
  int64_t r0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows;
  Raw8<T> x[4];
  auto load = [&](int64_t at, int j) {
    // past the end: the warp's first row again, not stored
    const int row = at + q[j].row < n ? q[j].row : 0;
    x[j].load(rows + (size_t)at * kRow + (row * kRow + q[j].value));
  };
  if (r0 < n)
#pragma unroll
    for (int j = 0; j < 4; ++j) load(r0, j);
  for (; r0 < n; r0 += step) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e = mx_scale_code(block_amax(x[j]), j == 3 ? kE4m3Emax : kE2m1Emax);
      float y[8];
      scaled_down(x[j], e, y);
      if (r0 + step < n) load(r0 + step, j);  // the next rows' values, behind this group's
      uint8_t* o = bytes + q[j].row * kKv4RowBytes;
      if (j == 3) {
        const uint2 w = e4m3x8(y);
        *reinterpret_cast<uint2*>(o + q[j].code) = e == 0xFFu ? make_uint2(0u, 0u) : w;
      } else {
        *reinterpret_cast<uint32_t*>(o + q[j].code) = e == 0xFFu ? 0u : e2m1x8(y);
      }
      if ((lane & 3) == 0) o[q[j].scale] = (uint8_t)e;
    }
    __syncwarp();
    const int pieces = (int)min((int64_t)kKv4Rows, n - r0) * kPieces;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      if (i >= pieces) continue;
      if (LIST) {
        const int row = i / kPieces;
        const int64_t to = __ldg(dst + r0 + row);
        if (to >= cap && i == row * kPieces) flag(st, CSKV_DEV_BAD_INDEX);
        if (to >= 0 && to < cap) reinterpret_cast<uint4*>(out + (size_t)to * kKv4RowBytes)[i - row * kPieces] = mine[i];
      } else {
        reinterpret_cast<uint4*>(out + (size_t)r0 * kKv4RowBytes)[i] = mine[i];
      }
    }
    __syncwarp();
  }
}

template <typename T, bool LIST>
__global__ void __launch_bounds__(32 * kKv4Warps) kv_dequantize_fp4_kernel(const uint8_t* __restrict__ cache,
                                                                          const int64_t* __restrict__ src,
                                                                          int64_t cap, int64_t n,
                                                                          T* __restrict__ out, int* st) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  Kv4Piece q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = kv4_piece(j, lane);
  const int64_t step = (int64_t)gridDim.x * kKv4Warps * kKv4Rows;
  for (int64_t r0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows; r0 < n; r0 += step) {
    const int here = (int)min((int64_t)kKv4Rows, n - r0);  // rows of this warp
    const uint8_t* base = cache + (LIST ? 0 : (size_t)r0 * kKv4RowBytes);
    // all groups' loads go out before the first is decoded
    uint2 w[4];
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = make_uint2(0u, 0u), e[j] = 127u;
      if (q[j].row >= here) continue;
      const uint8_t* row = base + q[j].row * kKv4RowBytes;
      if (LIST) {
        const int64_t i = __ldg(src + r0 + q[j].row);
        if (i >= cap && q[j].value == 64) flag(st, CSKV_DEV_BAD_INDEX);  // once a row
        if (i < 0 || i >= cap) continue;
        row = base + (size_t)i * kKv4RowBytes;
      }
      if (j == 3)
        w[j] = __ldg(reinterpret_cast<const uint2*>(row + q[j].code));
      else
        w[j].x = __ldg(reinterpret_cast<const uint32_t*>(row + q[j].code));
      e[j] = __ldg(row + q[j].scale);
    }
    T* to = out + (size_t)r0 * kRow;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (q[j].row >= here) continue;
      T* at = to + (q[j].row * kRow + q[j].value);
      if (j == 3)
        store_e4m3x8(at, w[j].x, w[j].y, e[j]);
      else
        store_e2m1x8(at, w[j].x, e[j]);
    }
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

static int64_t kv4_ctas(int64_t n) {
  return std::min(kKv4MostCtas, (n + kKv4Warps * kKv4Rows - 1) / (kKv4Warps * kKv4Rows));
}

template <typename T>
static cudaError_t launch_kv4_quantize_as(const void* rows, int64_t n, const int64_t* dst, int64_t cap, uint8_t* out,
                                          int* st, cudaStream_t stream) {
  return launch_1d(dst ? kv_quantize_fp4_kernel<T, true> : kv_quantize_fp4_kernel<T, false>, kv4_ctas(n),
                   32 * kKv4Warps, stream, (const T*)rows, n, dst, cap, out, st);
}

cudaError_t launch_kv_quantize_fp4(const void* rows, int dtype, int64_t n, const int64_t* dst, int64_t cap,
                                   uint8_t* out, int* st, cudaStream_t stream) {
  return dtype == CSKV_F32 ? launch_kv4_quantize_as<float>(rows, n, dst, cap, out, st, stream)
                           : launch_kv4_quantize_as<__nv_bfloat16>(rows, n, dst, cap, out, st, stream);
}

template <typename T>
static cudaError_t launch_kv4_dequantize_as(const uint8_t* cache, const int64_t* src, int64_t cap, int64_t n,
                                            void* out, int* st, cudaStream_t stream) {
  return launch_1d(src ? kv_dequantize_fp4_kernel<T, true> : kv_dequantize_fp4_kernel<T, false>, kv4_ctas(n),
                   32 * kKv4Warps, stream, cache, src, cap, n, (T*)out, st);
}

cudaError_t launch_kv_dequantize_fp4(const uint8_t* cache, const int64_t* src, int64_t cap, int64_t n, int dtype,
                                     void* out, int* st, cudaStream_t stream) {
  return dtype == CSKV_F32 ? launch_kv4_dequantize_as<float>(cache, src, cap, n, out, st, stream)
                           : launch_kv4_dequantize_as<__nv_bfloat16>(cache, src, cap, n, out, st, stream);
}

}  // namespace cskv
