// Product of MXFP4 matrices: out[m, n] = sum_k a[m, k] b[n, k], on tcgen05 kind::mxf4.
//
// [TR] trdm.cn/news/516303 §4.2 (the indexer projects its queries and keys in low precision),
// [SW] shareware.cn/news/167317 §六.1 (FP4 suffices for ranking): rows of E2M1 codes with one E8M0
// scale per 32 values (mx4.cuh), exact products, fp32 accumulation.
//
// A persistent CTA an SM, with roles: one thread loads code tiles by TMA (128-byte swizzle, 256 codes
// deep, zeros past the edges), four warps load the rows' scales and lay them out as the tensor core
// wants them, one warp copies scales to tensor memory and issues the products, four warps write
// out a tile while the next one's products run (two accumulators).  The 128-row operand P is a,
// or, for a few rows of a, b: the tile is then as narrow as those rows, and few tiles are split over
// the inner length inside a thread-block cluster, since one step is a chain of latencies.
//
// What bounds it: a step (256 deep) of a 128 x 192 tile is four products of about 95 cycles, but its
// 41 KB take 640 at the 64 bytes a cycle that an SM reads from L2, and 640 at shared memory's 128,
// where they are written and read once each; the issuing warp takes about 650 a step.  The tensor pipe
// is active for 44 % of the cycles.  Steps that count here: scales copied a step before their products
// (4096^3: 50.5 -> 46.4 us), one wait and one commit a step (41.0), a row's scales loaded one
// sector, four steps, at a time (38.2).
// Measured (device time): 4096^3, bf16 out: 40 us, 3.4 PFLOP/s, with the codes in L2 (38 to 40.6 from
// GPU to GPU), 45 us, 3.0 PFLOP/s, with codes that are not; 4096 x 512 x 4096: 11.7 us; one row x 4096 x
// 4096: 6.1 us, 1.5 TB/s of codes; 67 x 1000 x 2080: 10.8 us.
#include <cuda.h>

#include "launch.cuh"
#include "roles.cuh"

namespace cskv {

constexpr int kMmThreads = 320;          // warp 0 TMA, 1 products, 2-5 scales, 6-9 output
constexpr int kMmScaleWarps = 4, kMmOutWarp = 2 + kMmScaleWarps;
constexpr int kMmDeep = 256;             // codes of a stage: 128 bytes a row
constexpr uint32_t kMmTileP = 128 * 128;  // bytes of P's 128 rows of codes
constexpr uint32_t kMmOutPad = 144;      // bytes of a staged output row: 128 and a skew of four banks
constexpr int kMmMaxSplit = 8;           // CTAs of a cluster that share a tile's inner length

struct MmParams {
  CUtensorMap p_map, q_map;  // codes of the 128-row operand P and of the other, Q
  const uint8_t *p_scale, *q_scale;
  int64_t p_rows, q_rows, k32;  // k32: scale bytes of a row
  int64_t ld;                   // N
  int p_tiles, q_tiles, steps;
  int split;                    // CTAs that share a tile (the size of the cluster)
  int p_is_a;                   // out[p, q] (P rows are a's), else out[q, p]
  int wide;                     // alignment of every row's scales: 32, 16, 8, 4 or 1 bytes
  void* out;
  int* st;
};

// Tiles of 128 rows of P by NQ of Q.
template <int NQ>
struct MmShape {
  static constexpr int qc = (NQ + 127) / 128;                // 128-row scale chunks of Q
  static constexpr uint32_t codes = kMmTileP + NQ * 128u;    // a stage's code bytes
  static constexpr uint32_t scales = 1024u * (1 + qc);       // a step's scales: two K chunks each
  static constexpr int stages = (int)(163840u / codes) < 8 ? (int)(163840u / codes) : 8;
  static constexpr uint32_t off_scales = codes * stages, off_out = off_scales + scales * stages;
  static constexpr size_t smem = off_out + 4 * 32 * kMmOutPad + 1024;
  static constexpr int acc_cols = NQ < 32 ? 32 : NQ;         // TMEM columns of an accumulator
  // a step's scales in TMEM: when those of step g + 1 are copied, step g's codes are there, so the
  // products of step g - stages, the last ones that read the same columns, are complete
  static constexpr int sf_col = 2 * acc_cols, sf_step = 8 * (1 + qc), sf_bufs = stages + 1;
  static constexpr int used = sf_col + sf_bufs * sf_step;
  static constexpr int cols = used <= 128 ? 128 : used <= 256 ? 256 : 512;
  static_assert(used <= 512, "tensor memory");
  static_assert(off_scales >= 128u * NQ * 4u, "a split tile's partial fits the ring");
};

struct MmShared {
  uint64_t full[8], empty[8], first, acc_full[2], acc_empty[2], bail;
  uint32_t tmem;
  int abort;
};

// Scale bytes of steps k .. end - 1 of a row, which lie in one aligned group of four steps (32 bytes,
// one sector), at their places in the group.  Zeros past the row's end or for a row that is not there.
// `wide`: the alignment of all rows, the widest load of which serves (the lanes' rows are all in
// different sectors, so a load costs 32 lookups; 4096^3 by 32 / 16 / 8 / 4 / 1 bytes: 38 / 40 / 43 / 53 /
// 90 us; by single bytes 171).
__device__ __forceinline__ void mm_scales(const uint8_t* scale, int64_t row, int64_t rows, int64_t k32, int k, int end,
                                          int wide, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0u;
  if (row >= rows) return;
  const int64_t at = 8 * (int64_t)(k & ~3);
  const uint8_t* s = scale + row * k32 + at;
  const int from = 8 * (k & 3), to = (int)min(8 * (int64_t)end, k32) - (int)at;
  if (wide == 32) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(s));
  } else if (wide == 16) {
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      if (4 * i + 16 > from && 4 * i < to) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(s + 4 * i));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
  } else if (wide == 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      if (4 * i >= from && 4 * i < to) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(s + 4 * i));
        w[i] = v.x, w[i + 1] = v.y;
      }
  } else if (wide == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (4 * i >= from && 4 * i < to) w[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  } else {
    // rows that begin anywhere: the aligned words around them (by bytes where such a word reaches out
    // of the matrix), shifted into place; what follows the row is cut off
    const int a = (int)(reinterpret_cast<uintptr_t>(s) & 3);
    const uint8_t* last = scale + rows * k32;
    uint32_t v[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      const uint8_t* at4 = s - a + 4 * i;
      v[i] = 0u;
      if (4 * i + 4 <= a + from || 4 * i >= a + to) continue;
      if (at4 >= scale && at4 + 4 <= last)
        v[i] = __ldg(reinterpret_cast<const uint32_t*>(at4));
      else
        for (int j = 0; j < 4; ++j)
          if (at4 + j >= scale && at4 + j < last) v[i] |= (uint32_t)__ldg(at4 + j) << (8 * j);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = __funnelshift_r(v[i], v[i + 1], 8 * a);
      if (4 * i + 4 > to) w[i] &= 4 * i < to ? (1u << (8 * (to & 3))) - 1u : 0u;
    }
  }
}

// Columns q .. q + STEP - 1 of row `pr` of a tile.
template <int STEP, typename T>
__device__ __forceinline__ void mm_store(const MmParams& p, int64_t pr, int64_t q, const float (&v)[STEP]) {
  if (pr >= p.p_rows || q >= p.q_rows) return;
  T* out = reinterpret_cast<T*>(p.out);
  auto one = [](float x) {
    if constexpr (sizeof(T) == 2)
      return __float2bfloat16_rn(x);
    else
      return x;
  };
  const bool whole = q + STEP <= p.q_rows;
  if (!p.p_is_a) {  // out[q, p]: neighbouring lanes on neighbouring columns
#pragma unroll
    for (int i = 0; i < STEP; ++i)
      if (whole || q + i < p.q_rows) out[(q + i) * p.ld + pr] = one(v[i]);
    return;
  }
  T* dst = out + pr * p.ld + q;
#pragma unroll
  for (int i = 0; i < STEP; ++i)
    if (whole || q + i < p.q_rows) dst[i] = one(v[i]);
}

template <int NQ, typename T>
__global__ void __launch_bounds__(kMmThreads, 1) mxfp4_matmul_kernel(const __grid_constant__ MmParams p) {
  using Sh = MmShape<NQ>;
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t* buf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  __shared__ MmShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tiles = (int64_t)p.p_tiles * p.q_tiles;
  // this CTA's part of its tiles' inner length (its rank in a one-dimensional cluster)
  const int split = p.split, rank = (int)(blockIdx.x % (unsigned)split);
  const int64_t tile0 = blockIdx.x / split, stride = gridDim.x / split;
  const int k0 = (int)((int64_t)p.steps * rank / split), k1 = (int)((int64_t)p.steps * (rank + 1) / split);

  if (warp == 1) {
    tmem_alloc(&sh.tmem, Sh::cols);
    tmem_relinquish();
  }
  if (tid == 32 * kMmOutWarp) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.p_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.q_map) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < Sh::stages; ++i) {
      mbar_init(&sh.full[i], 1 + kMmScaleWarps);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.first, kMmScaleWarps);
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
      for (int64_t tile = tile0; tile < tiles && ok; tile += stride) {
        const int pt = (int)(tile % p.p_tiles), qt = (int)(tile / p.p_tiles);
        for (int k = k0; k < k1 && ok; ++k, ++g) {
          const uint32_t s = g % Sh::stages;
          if (g >= Sh::stages) ok = role_wait(&sh.empty[s], g / Sh::stages - 1, &sh.abort, p.st);
          if (!ok) break;
          uint8_t* dst = buf + s * Sh::codes;
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
    // A step's descriptors differ by their address field alone (16-byte units).
    const uint32_t base = smem_u32(buf);
    const uint64_t d_codes = smem_desc_sw128(base, 16, 1024), d_scales = smem_desc_noswz(base + Sh::off_scales, 16, 128);
    uint32_t n = 0, s = 0, sp = 0;  // tiles; stage and phase of a step
    uint32_t ss = 0, sb = 0, pb = 0;  // scales' stage; TMEM buffer of the copies, of the products
    // A wait that gave up does not end the loops: what decides them has to be uniform for the compiler,
    // or every operand is moved to a uniform register at each use (which took longer than the
    // products).  The products then run on what is there, and the call is flagged.
    // Scales of a step -> tensor memory, 512 bytes a chunk of 128 rows and 4 K scales: P's two K chunks,
    // then Q's rows by K chunk.
    auto copy_scales = [&]() {
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 2 * (1 + Sh::qc); ++i)
          tc_cp_scales(tmem + Sh::sf_col + sb * Sh::sf_step + 4 * i, d_scales + ss * (Sh::scales >> 4) + 32 * i);
      }
      if (++ss == Sh::stages) ss = 0;
      if (++sb == Sh::sf_bufs) sb = 0;
    };
    if (tile0 < tiles) {
      role_wait(&sh.first, 0, &sh.abort, p.st);
      __syncwarp();
      tc_fence_after();
      copy_scales();
      __syncwarp();
    }
    for (int64_t tile = tile0; tile < tiles; tile += stride, ++n) {
      const uint32_t ab = n & 1;
      if (n >= 2) role_wait(&sh.acc_empty[ab], n / 2 - 1, &sh.abort, p.st);
      for (int k = k0; k < k1; ++k) {
        role_wait(&sh.full[s], sp, &sh.abort, p.st);
        __syncwarp();
        tc_fence_after();
        // a step's scales go out before the products of the step before it, which need not wait for
        // them then
        if (k + 1 < k1 || tile + stride < tiles) copy_scales();
        const uint32_t col = tmem + Sh::sf_col + pb * Sh::sf_step;
        const uint64_t d = d_codes + s * (Sh::codes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mxf4(tmem + ab * Sh::acc_cols, d + 2 * kk, d + (kMmTileP >> 4) + 2 * kk,
                        idesc_mxf4(128, NQ, 2 * (kk & 1)), col + 4 * (kk >> 1), col + 8 + 4 * Sh::qc * (kk >> 1),
                        k > k0 || kk > 0);
          tc_commit(&sh.empty[s]);  // and the scales of the next step are copied
          if (k + 1 == k1) tc_commit(&sh.acc_full[ab]);
        }
        __syncwarp();
        if (++s == Sh::stages) s = 0, sp ^= 1;
        if (++pb == Sh::sf_bufs) pb = 0;
      }
    }
    if (elect_one()) {  // nothing of this CTA may still be in flight when its memory is released
      tc_commit(&sh.bail);
      mbar_wait_bounded(&sh.bail, 0);
    }
    __syncwarp();
  } else if (warp < kMmOutWarp) {
    // ---------------------------------------------------------------- scales
    // Warp w takes every fourth group of 32 rows, four steps at a time (a row's 32 bytes, the next
    // four on their way).  A step's eight bytes are two words, one for each 512-byte chunk of
    // 128 rows x 4 K scales: row r at 16 (r % 32) + 4 (r / 32).  A step's scales are counted with the
    // codes of the step before it, which is when they are copied on, so that a step of the products
    // has one wait and one commit.
    constexpr int kGroups = 4 + (NQ + 31) / 32, kMine = (kGroups + kMmScaleWarps - 1) / kMmScaleWarps;
    const int w0 = warp - 2;
    uint32_t cur[kMine][8], nxt[kMine][8];
    auto load = [&](int64_t tile, int k, uint32_t (&w)[kMine][8]) {
      const int64_t p0 = (tile % p.p_tiles) * 128, q0 = (tile / p.p_tiles) * NQ;
      const int end = min((k & ~3) + 4, k1);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = 32 * (w0 + kMmScaleWarps * i) + lane;
        if (i == 0)  // P's four groups
          mm_scales(p.p_scale, p0 + r, p.p_rows, p.k32, k, end, p.wide, w[i]);
        else
          mm_scales(p.q_scale, r < 128 + NQ ? q0 + r - 128 : p.q_rows, p.q_rows, p.k32, k, end, p.wide, w[i]);
      }
    };
    // step g - 1 - stages is complete: its stage of `full` may be counted for step g - 1, and step
    // g - stages' scales, copied before its products, have left their place (step 0's before step 0's)
    auto room = [&](uint32_t at) {
      if (at < (uint32_t)Sh::stages) return true;
      const uint32_t h = at == (uint32_t)Sh::stages ? 0 : at - 1 - Sh::stages;
      return role_wait_warp(&sh.empty[h % Sh::stages], h / Sh::stages, &sh.abort, p.st);
    };
    uint32_t g = 0;
    bool ok = true;
    int64_t tile = tile0;
    int k = k0;
    if (tile < tiles) load(tile, k, cur);
    while (tile < tiles && ok) {
      const int base = k & ~3, end = min(base + 4, k1);
      const int64_t next_tile = end < k1 ? tile : tile + stride;
      const int next_k = end < k1 ? end : k0;
      if (next_tile < tiles) load(next_tile, next_k, nxt);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (base + j < k || base + j >= end || !ok) continue;
        if (!(ok = room(g))) continue;
        uint8_t* sf = buf + Sh::off_scales + g % Sh::stages * Sh::scales + 16 * lane;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int q = 32 * (w0 + kMmScaleWarps * (i - 1));  // Q's rows of this group
          uint8_t* to = i == 0 ? sf + 4 * w0 : sf + 1024 + 512 * (q >> 7) + 4 * ((q & 127) >> 5);
          if (i == 0 || q + lane < NQ) {
            *reinterpret_cast<uint32_t*>(to) = cur[i][2 * j];
            *reinterpret_cast<uint32_t*>(to + (i == 0 ? 512 : 512 * Sh::qc)) = cur[i][2 * j + 1];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(g ? &sh.full[(g - 1) % Sh::stages] : &sh.first);
        ++g;
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) cur[i][j] = nxt[i][j];
      tile = next_tile;
      k = next_k;
    }
    // the last step has no successor
    if (ok && g && room(g) && lane == 0) mbar_arrive(&sh.full[(g - 1) % Sh::stages]);
  } else {
    // ---------------------------------------------------------------- output
    // A split tile's partial goes to shared memory instead ([column][row]; the ring is done with).
    const int quad = warp & 3;  // the TMEM lanes this warp may read
    const int row_in = quad * 32 + lane;
    constexpr int kStep = NQ < 32 ? 16 : 32;
    uint8_t* cross = buf + Sh::off_out + (warp - kMmOutWarp) * 32 * kMmOutPad;
    const bool wide_out = p.p_is_a && (p.ld * sizeof(T)) % 16 == 0;  // every 8th column is a 16-byte place
    uint32_t n = 0;
    bool ok = true;
    for (int64_t tile = tile0; tile < tiles && ok; tile += stride, ++n) {
      const int64_t pr = (tile % p.p_tiles) * 128 + row_in, q0 = (tile / p.p_tiles) * NQ;
      const uint32_t ab = n & 1;
      ok = role_wait_warp(&sh.acc_full[ab], n / 2, &sh.abort, p.st);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + ab * Sh::acc_cols + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < NQ; c += kStep) {
        uint32_t v[kStep];
        __syncwarp();
        if constexpr (kStep == 16)
          tmem_ld16(acc + c, v);
        else
          tmem_ld32(acc + c, v);
        tmem_ld_wait();
        float f[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) f[i] = __uint_as_float(v[i]);
        if (split == 1 && kStep == 32 && p.p_is_a) {
          // out[p, q]: the warp's 32 x 32 values cross in shared memory, so that lanes store whole
          // stretches of a row (64 or 128 bytes) instead of single values of 32 rows: 16 bytes a lane, or
          // one value where rows are not whole 16-byte words or the columns end (1498 x 1069 x 64 by
          // single values of 32 rows 26 us, this 7.9)
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = f[(i + j) % kStep];
            Vec8<T>::store(reinterpret_cast<T*>(cross + lane * kMmOutPad) + i, x);
          }
          __syncwarp();
          if (wide_out && q0 + c + 32 <= p.q_rows) {
            constexpr int kLanes = 2 * sizeof(T);  // lanes of a row: 16 bytes each
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
              const int r = i * (32 / kLanes) + lane / kLanes, at = lane % kLanes;
              const uint4 w = *reinterpret_cast<const uint4*>(cross + r * kMmOutPad + 16 * at);
              if (pr - lane + r < p.p_rows)
                *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + (pr - lane + r) * p.ld + q0 + c + at * (16 / sizeof(T))) = w;
            }
          } else if (q0 + c + lane < p.q_rows) {
            const int rows = (int)min((int64_t)32, p.p_rows - (pr - lane));
            T* to = reinterpret_cast<T*>(p.out) + (pr - lane) * p.ld + q0 + c + lane;
#pragma unroll 4
            for (int r = 0; r < rows; ++r, to += p.ld) *to = reinterpret_cast<const T*>(cross + r * kMmOutPad)[lane];
          }
          __syncwarp();
        } else if (split == 1) {
          mm_store<kStep, T>(p, pr, q0 + c, f);
        } else {
#pragma unroll
          for (int i = 0; i < kStep; ++i) reinterpret_cast<float*>(buf)[(c + i) * 128 + row_in] = f[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[ab]);
    }
  }
  if (split > 1) {
    // ---------------------------------------------------------------- a split tile's sum
    // Each CTA adds up its share of the columns over the cluster, in rank order.
    __syncwarp();
    cluster_sync();
    if (warp >= kMmOutWarp && warp < kMmOutWarp + 4) {
      const int row_in = (warp - kMmOutWarp) * 32 + lane;
      const int64_t pr = (tile0 % p.p_tiles) * 128 + row_in, q0 = (tile0 / p.p_tiles) * NQ;
      const int c0 = NQ * rank / split, c1 = NQ * (rank + 1) / split;
      for (int c = c0; c < c1; c += 2) {  // NQ / split is 2 at least
        float f[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < kMmMaxSplit; ++r)
          if (r < split) {
            f[0] += ld_cluster_f32(smem_u32(buf) + (c * 128 + row_in) * 4, r);
            f[1] += ld_cluster_f32(smem_u32(buf) + ((c + 1) * 128 + row_in) * 4, r);
          }
        mm_store<2, T>(p, pr, q0 + c, f);
      }
    }
    cluster_sync();  // the others may still read this CTA's partial
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : tiles < sms ? tiles : sms));
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = MmShape<NQ>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  note_launch();
  return e;
}

template <int NQ>
static cudaError_t mm_launch(MmParams& p, const uint8_t* p_codes, const uint8_t* q_codes, int64_t K, int out_dt,
                             int sms, cudaStream_t stream) {
  p.p_tiles = (int)((p.p_rows + 127) / 128);
  p.q_tiles = (int)((p.q_rows + NQ - 1) / NQ);
  // few tiles: their inner length is split over a cluster, two steps a CTA at least
  p.split = 1;
  if (NQ <= 64)
    while (p.split < kMmMaxSplit && (int64_t)p.p_tiles * p.q_tiles * p.split * 2 <= sms && p.steps >= 4 * p.split)
      p.split *= 2;
  if (!mm_map(&p.p_map, p_codes, p.p_rows, K, 128) || !mm_map(&p.q_map, q_codes, p.q_rows, K, NQ))
    return cudaErrorNotSupported;
  return out_dt == CSKV_F32 ? mm_launch_as<NQ, float>(p, sms, stream)
                            : mm_launch_as<NQ, __nv_bfloat16>(p, sms, stream);
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
  const uintptr_t places = (uintptr_t)a_scale | (uintptr_t)b_scale | (uintptr_t)p.k32;
  p.wide = places % 32 == 0 ? 32 : places % 16 == 0 ? 16 : places % 8 == 0 ? 8 : places % 4 == 0 ? 4 : 1;
  p.out = out;
  p.st = st;
  if (!p.p_is_a)
    return M <= 16 ? mm_launch<16>(p, pc, qc, K, out_dt, sms, stream)
           : M <= 32 ? mm_launch<32>(p, pc, qc, K, out_dt, sms, stream)
                     : mm_launch<64>(p, pc, qc, K, out_dt, sms, stream);
  // the width whose waves of tiles take the least time (a tile costs its columns and a fixed part,
  // about 64 columns' worth)
  int best = 192;
  int64_t least = INT64_MAX;
  for (int nq : {192, 128, 64}) {
    const int64_t tiles = (int64_t)((p.p_rows + 127) / 128) * ((p.q_rows + nq - 1) / nq);
    const int64_t cost = (tiles + sms - 1) / sms * (nq + 64);
    if (cost < least) least = cost, best = nq;
  }
  return best == 192   ? mm_launch<192>(p, pc, qc, K, out_dt, sms, stream)
         : best == 128 ? mm_launch<128>(p, pc, qc, K, out_dt, sms, stream)
                       : mm_launch<64>(p, pc, qc, K, out_dt, sms, stream);
}

}  // namespace cskv
