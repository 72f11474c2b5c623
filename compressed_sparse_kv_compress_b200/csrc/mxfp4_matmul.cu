// Product of MXFP4 matrices: out[m, n] = sum_k a[m, k] b[n, k], on tcgen05 kind::mxf4.
//
// [TR] trdm.cn/news/516303 §4.2 (the indexer projects its queries and keys in low precision),
// [SW] shareware.cn/news/167317 §六.1 (FP4 suffices for ranking): rows of E2M1 codes with one E8M0
// scale per 32 values (mx4.cuh), exact products, fp32 accumulation.
//
// Large products are bound by the tensor pipe (and by shared memory, which feeds it 128 bytes a
// cycle: a 128 x 192 tile needs 106), a few rows by the bytes of b.  A persistent CTA an SM, with
// roles: one thread loads code tiles by TMA (128-byte swizzle, 256 codes deep, zeros past the edges),
// four warps load the rows' scales and lay them out as the tensor core wants them, one thread
// copies scales to tensor memory and issues the products, four warps write out the tile before
// last (two accumulators).  The 128-row operand is a, or, for a few rows of a, b: the tile is then
// as narrow as those rows.
#include <cuda.h>

#include "launch.cuh"
#include "roles.cuh"

namespace cskv {

constexpr int kMmThreads = 320;          // warp 0 TMA, 1 products, 2-5 scales, 6-9 output
constexpr int kMmScaleWarps = 4;
constexpr int kMmDeep = 256;             // codes of a stage: 128 bytes a row
constexpr uint32_t kMmTileP = 128 * 128;  // bytes of the 128-row operand's tile
constexpr int kMmSfStep = 32;            // TMEM columns of one stage's scales

struct MmParams {
  CUtensorMap p_map, q_map;  // codes of the 128-row operand P and of the other, Q
  const uint8_t *p_scale, *q_scale;
  int64_t p_rows, q_rows, k32;  // k32: scale bytes of a row
  int64_t ld;                   // N
  int p_tiles, q_tiles, steps;
  int p_is_a;                   // out[p, q] (P rows are a's), else out[q, p]
  int wide;                     // scale rows are whole 4-byte words
  void* out;
  int* st;
};

template <int NQ>
struct MmShape {
  static constexpr int qc = (NQ + 127) / 128;               // 128-row scale chunks of Q
  static constexpr uint32_t codes = kMmTileP + NQ * 128u;   // a stage's code bytes
  static constexpr uint32_t scales = 1024u * (1 + qc);      // two K chunks each
  static constexpr uint32_t stage = (codes + scales + 1023u) / 1024u * 1024u;
  static constexpr int stages = (int)(196608u / stage) < 8 ? (int)(196608u / stage) : 8;
  static constexpr size_t smem = (size_t)stage * stages + 1024;
  static constexpr int acc_cols = NQ < 32 ? 32 : NQ;        // TMEM columns of an accumulator
  static constexpr int sf_col = 2 * acc_cols;
  static constexpr int cols = sf_col + 2 * kMmSfStep <= 128 ? 128 : sf_col + 2 * kMmSfStep <= 256 ? 256 : 512;
  static_assert(sf_col + 2 * kMmSfStep <= 512 && 8 * (1 + qc) <= kMmSfStep, "tensor memory");
};

struct MmShared {
  uint64_t full[8], sf_full[8], empty[8], acc_full[2], acc_empty[2], bail;
  uint32_t tmem;
  int abort;
};

// Scale bytes 8 step .. 8 step + 7 of a row, zeros past its end or for a row that is not there.
__device__ __forceinline__ uint2 mm_scales(const uint8_t* scale, int64_t row, int64_t rows, int64_t k32, int step,
                                           int wide) {
  uint32_t w[2] = {0u, 0u};
  if (row < rows) {
    const uint8_t* s = scale + row * k32 + 8 * (int64_t)step;
    const int left = (int)min((int64_t)8, k32 - 8 * (int64_t)step);
    if (wide) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
      if (left > 4) w[1] = __ldg(reinterpret_cast<const uint32_t*>(s) + 1);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 2] |= (uint32_t)__ldg(s + i) << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int NQ, typename T>
__global__ void __launch_bounds__(kMmThreads, 1) mxfp4_matmul_kernel(const __grid_constant__ MmParams p) {
  using Sh = MmShape<NQ>;
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t* buf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  __shared__ MmShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tiles = (int64_t)p.p_tiles * p.q_tiles;

  if (warp == 1) {
    tmem_alloc(&sh.tmem, Sh::cols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < Sh::stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.sf_full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 4);
    }
    mbar_init(&sh.bail, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();

  // tile -> (P tile, Q tile): neighbouring CTAs share a Q tile
  if (warp == 0) {
    // ---------------------------------------------------------------- codes
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int pt = (int)(tile % p.p_tiles), qt = (int)(tile / p.p_tiles);
        for (int k = 0; k < p.steps && ok; ++k, ++g) {
          const uint32_t s = g % Sh::stages;
          if (g >= Sh::stages) ok = role_wait(&sh.empty[s], g / Sh::stages - 1, &sh.abort, p.st);
          if (!ok) break;
          uint8_t* dst = buf + s * Sh::stage;
          mbar_arrive_expect_tx(&sh.full[s], Sh::codes);
          tma_load_2d(dst, &p.p_map, k * 128, pt * 128, &sh.full[s]);
          tma_load_2d(dst + kMmTileP, &p.q_map, k * 128, qt * NQ, &sh.full[s]);
        }
      }
      // the last loads have landed before this CTA's memory is released
      for (uint32_t i = 0; i < Sh::stages && i < g; ++i)
        mbar_wait_bounded(&sh.full[(g - 1 - i) % Sh::stages], ((g - 1 - i) / Sh::stages) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t base = smem_u32(buf);
      uint32_t g = 0, n = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++n) {
        if (n >= 2) ok = role_wait(&sh.acc_empty[n & 1], n / 2 - 1, &sh.abort, p.st);
        tc_fence_after();
        for (int k = 0; k < p.steps && ok; ++k, ++g) {
          const uint32_t s = g % Sh::stages, at = base + s * Sh::stage, sf = at + Sh::codes;
          ok = role_wait(&sh.full[s], g / Sh::stages, &sh.abort, p.st) &&
               role_wait(&sh.sf_full[s], g / Sh::stages, &sh.abort, p.st);
          if (!ok) break;
          tc_fence_after();
          // scales: chunk c of P (K chunk c), then of Q (K chunk c, 128 rows each)
          const uint32_t col = tmem + Sh::sf_col + (g & 1) * kMmSfStep;
#pragma unroll
          for (int c = 0; c < 2 * (1 + Sh::qc); ++c)
            tc_cp_scales(col + 4 * c, smem_desc_noswz(sf + 512 * c, 16, 128));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mxf4(tmem + (n & 1) * Sh::acc_cols, smem_desc_sw128(at + 32 * kk, 16, 1024),
                        smem_desc_sw128(at + kMmTileP + 32 * kk, 16, 1024), idesc_mxf4(128, NQ, 2 * (kk & 1)),
                        col + 4 * (kk >> 1), col + 8 + 4 * Sh::qc * (kk >> 1), k > 0 || kk > 0);
          tc_commit(&sh.empty[s]);
        }
        if (ok) tc_commit(&sh.acc_full[n & 1]);
      }
      if (!ok) {  // gave up: nothing of this CTA may still be in flight when its memory is released
        tc_commit(&sh.bail);
        mbar_wait_bounded(&sh.bail, 0);
      }
    }
    __syncwarp();
  } else if (warp < 2 + kMmScaleWarps) {
    // ---------------------------------------------------------------- scales
    // Warp w takes every fourth step.  A row's eight bytes are two words, one for each 512-byte
    // chunk of 128 rows x 4 K scales: row r at 16 (r % 32) + 4 (r / 32).
    constexpr int kRows = (128 + NQ + 31) / 32;
    uint32_t g = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
      const int64_t p0 = (tile % p.p_tiles) * 128, q0 = (tile / p.p_tiles) * NQ;
      for (int k = 0; k < p.steps && ok; ++k, ++g) {
        if ((int)(g % kMmScaleWarps) != warp - 2) continue;
        uint2 w[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = lane + 32 * i;
          w[i] = r < 128      ? mm_scales(p.p_scale, p0 + r, p.p_rows, p.k32, k, p.wide)
                 : r < 128 + NQ ? mm_scales(p.q_scale, q0 + r - 128, p.q_rows, p.k32, k, p.wide)
                                : make_uint2(0u, 0u);
        }
        const uint32_t s = g % Sh::stages;
        if (g >= Sh::stages) ok = role_wait_warp(&sh.empty[s], g / Sh::stages - 1, &sh.abort, p.st);
        if (!ok) break;
        uint8_t* sf = buf + s * Sh::stage + Sh::codes;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = lane + 32 * i;
          const int q = r - 128;
          uint8_t* to = r < 128 ? sf + 16 * (r & 31) + 4 * (r >> 5)
                                : sf + 1024 + 512 * (q >> 7) + 16 * (q & 31) + 4 * ((q & 127) >> 5);
          if (r < 128 + NQ) {
            *reinterpret_cast<uint32_t*>(to) = w[i].x;
            *reinterpret_cast<uint32_t*>(to + (r < 128 ? 512 : 512 * Sh::qc)) = w[i].y;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sf_full[s]);
      }
    }
  } else {
    // ---------------------------------------------------------------- output
    const int quad = warp & 3;  // the TMEM lanes this warp may read
    const int64_t row_in = quad * 32 + lane;
    constexpr int kStep = NQ < 32 ? 16 : 32;
    const bool vec = (p.ld * sizeof(T)) % 16 == 0;  // rows of out start on 16-byte boundaries
    T* out = reinterpret_cast<T*>(p.out);
    uint32_t n = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++n) {
      const int64_t pr = (tile % p.p_tiles) * 128 + row_in, q0 = (tile / p.p_tiles) * NQ;
      ok = role_wait_warp(&sh.acc_full[n & 1], n / 2, &sh.abort, p.st);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (n & 1) * Sh::acc_cols + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < NQ; c += kStep) {
        uint32_t v[32];
        __syncwarp();
        if constexpr (kStep == 16) {
          uint32_t x[16];
          tmem_ld16(acc + c, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = x[i];
        } else {
          tmem_ld32(acc + c, v);
        }
        tmem_ld_wait();
        const int64_t q = q0 + c;
        if (pr >= p.p_rows || q >= p.q_rows) continue;
        if (!p.p_is_a) {  // out[q, p]: neighbouring lanes on neighbouring columns
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (q + i < p.q_rows) {
              if constexpr (sizeof(T) == 2)
                out[(q + i) * p.ld + pr] = __float2bfloat16_rn(__uint_as_float(v[i]));
              else
                out[(q + i) * p.ld + pr] = __uint_as_float(v[i]);
            }
        } else if (vec && q + kStep <= p.q_rows) {
          T* dst = out + pr * p.ld + q;
#pragma unroll
          for (int i = 0; i < kStep; i += 8) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[i + j]);
            Vec8<T>::store(dst + i, f);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (q + i < p.q_rows) {
              if constexpr (sizeof(T) == 2)
                out[pr * p.ld + q + i] = __float2bfloat16_rn(__uint_as_float(v[i]));
              else
                out[pr * p.ld + q + i] = __uint_as_float(v[i]);
            }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[n & 1]);
    }
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::cols);
  }
}

// ---------------------------------------------------------------- host side
using MmEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once); null if it has none.
static MmEncode mm_encoder() {
  static const MmEncode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<MmEncode>(f);
  }();
  return fn;
}

// Map of a code matrix [rows, K/2 bytes]: boxes of box_rows x 128 bytes in the 128-byte swizzle,
// zeros past the edges.
static bool mm_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box_rows) {
  const MmEncode enc = mm_encoder();
  if (!enc) return false;
  const cuuint64_t dim[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows}, stride[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows}, step[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dim, stride, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NQ, typename T>
static cudaError_t mm_launch_as(const MmParams& p, int sms, cudaStream_t stream) {
  auto kern = mxfp4_matmul_kernel<NQ, T>;
  cudaError_t e = ensure_smem(kern, MmShape<NQ>::smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.p_tiles * p.q_tiles;
  e = launch_dependent(kern, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kMmThreads), MmShape<NQ>::smem, stream, p);
  note_launch();
  return e;
}

template <int NQ>
static cudaError_t mm_launch(MmParams& p, const uint8_t* q_codes, int64_t K, int out_dt, int sms, cudaStream_t stream) {
  p.q_tiles = (int)((p.q_rows + NQ - 1) / NQ);
  if (!mm_map(&p.q_map, q_codes, p.q_rows, K, NQ)) return cudaErrorNotSupported;
  return out_dt == CSKV_F32 ? mm_launch_as<NQ, float>(p, sms, stream) : mm_launch_as<NQ, __nv_bfloat16>(p, sms, stream);
}

cudaError_t launch_mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scale, const uint8_t* b_codes,
                                const uint8_t* b_scale, int64_t M, int64_t N, int64_t K, int out_dt, void* out,
                                int sms, int* st, cudaStream_t stream) {
  MmParams p = {};
  // up to 64 rows of a: b is the 128-row operand and the tile as narrow as a
  p.p_is_a = M > 64;
  const uint8_t *pc = p.p_is_a ? a_codes : b_codes, *qc = p.p_is_a ? b_codes : a_codes;
  p.p_scale = p.p_is_a ? a_scale : b_scale;
  p.q_scale = p.p_is_a ? b_scale : a_scale;
  p.p_rows = p.p_is_a ? M : N;
  p.q_rows = p.p_is_a ? N : M;
  p.k32 = K / 32;
  p.ld = N;
  p.steps = (int)((K + kMmDeep - 1) / kMmDeep);
  p.wide = p.k32 % 4 == 0 && (((uintptr_t)a_scale | (uintptr_t)b_scale) & 3u) == 0;
  p.out = out;
  p.st = st;
  p.p_tiles = (int)((p.p_rows + 127) / 128);
  if (!mm_map(&p.p_map, pc, p.p_rows, K, 128)) return cudaErrorNotSupported;
  if (!p.p_is_a)
    return M <= 16 ? mm_launch<16>(p, qc, K, out_dt, sms, stream)
           : M <= 32 ? mm_launch<32>(p, qc, K, out_dt, sms, stream)
                     : mm_launch<64>(p, qc, K, out_dt, sms, stream);
  // the width whose waves of tiles take the fewest column steps (a tile costs its columns and a
  // fixed part, about 32 columns' worth)
  int best = 192;
  int64_t cost = INT64_MAX;
  for (int nq : {192, 128, 64}) {
    const int64_t tiles = (int64_t)p.p_tiles * ((p.q_rows + nq - 1) / nq);
    const int64_t c = (tiles + sms - 1) / sms * (nq + 32);
    if (c < cost) cost = c, best = nq;
  }
  return best == 192 ? mm_launch<192>(p, qc, K, out_dt, sms, stream)
         : best == 128 ? mm_launch<128>(p, qc, K, out_dt, sms, stream)
                       : mm_launch<64>(p, qc, K, out_dt, sms, stream);
}

}  // namespace cskv
