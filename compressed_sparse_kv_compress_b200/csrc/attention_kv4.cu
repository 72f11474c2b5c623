// Hybrid attention over a compressed cache in 4-bit rows (mx4.cuh), bf16 queries, on tcgen05.
//
// [SW] = shareware.cn/news/167317: §十三.4 (the main KV in few bits, position-sensitive dims
// higher), §十一 (MQA: the heads share one KV), §十二 (sink).  [TR] = trdm.cn/news/516303, §3.1
// (online softmax).
//
// Formula, per query and head: o = softmax(scale q K^T with the sink) V over the query's row list
// (attn_rows.cuh).  Decoded rows are exact in bf16, so the products are those of exact rows
// with fp32 accumulation.  P is rounded to bf16 for P V, the type that the tensor core takes beside bf16
// V (its sum is kept in fp32): at most 2^-8 of a weight, independently from row to row, which makes the
// relative error of bf16 outputs against 64 bits 0.0022 where their own rounding alone makes 0.0017.
//
// What bounds it: a chunk of 128 rows is 2 x 128^3 MMA operations a head tile (1024 cycles of an
// SM's tensor pipe), 128 exponentials a head (8 cycles at 16 a cycle: 512 for 64 heads, 1024 for 128)
// and 32K decoded values (about 4 ALU operations a pair, 1024 cycles at 64 a cycle), against 22.5 KB of
// rows, so one persistent CTA an SM works on all of it at once with specialised warps.  For many
// queries a chunk takes about 3650 cycles (4096 queries x 64 heads x 1152 rows: 462 us), more than any of
// these: the roles' own chains, waits and a query's end are what is left.  For a few queries it is
// a latency chain, so a query's rows are split over the SMs (one query of 128 heads: 1152 rows on nine
// SMs 14.2 us, 8320 rows on 33 17.2 us, the merge among them).
//   warp 19     resolves row lists into a table of row addresses, up to four chunks ahead
//   warps 16-17 copy the stored rows to shared memory, up to two chunks ahead
//   warps 8-15  decode them to bf16 in the 128-byte-swizzle layout, four for K, four for V (with up to
//               64 heads, warps 2, 3 and 6-11: see there)
//   warp 18     one thread issues S = Q K^T and O (+)= P V; Q and P are A operands in tensor
//               memory, so only K and V are read from shared memory
//   warps 0-7   softmax: TMEM lane h is head h; S -> P in place, O rescaled when the running
//               maximum grows by more than 2^8 (any reference serves the online softmax), output
// Two K and three V buffers (32 KB each) and two S / P buffers pipeline the chunks, across queries
// too.  The roles' loops are kept short: unrolled ones missed the instruction cache.
// Measured (device time): 4096 queries of 64 heads over 1152 rows 462 us (155 GFLOP, 335 TFLOP/s; the
// softmax warps wait for 13 % of the time, the others longer: a warp's own chain of instructions); one
// query of 128 heads over 1152 rows 13.9 us, over 8320 rows 17.0 us; 64 ragged queries 22.2 us.
#include "attn_rows.cuh"
#include "mx4.cuh"
#include "roles.cuh"

namespace cskv {

constexpr int k4Chunk = 128;                            // rows of a chunk
constexpr int k4SoftWarps = 8, k4GatherWarps = 8;       // four for K, four for V, 32 rows each
constexpr int k4Copy = k4SoftWarps + k4GatherWarps, k4CopyWarps = 2, k4Mma = k4Copy + 2, k4Resolve = k4Copy + 3;
constexpr int k4Threads = 32 * 20;
constexpr int k4Table = 4;                              // chunks the row table (and their notes) hold
constexpr int k4KStages = 2, k4VStages = 3, k4RawStages = 2;
constexpr uint32_t k4Region = 128 * 128;                // 128 rows x 128 bytes: one swizzled region
constexpr uint32_t k4Half = 2 * k4Region;               // a chunk's K (or V): dims 0-63, 64-127
constexpr uint32_t k4OffV = k4KStages * k4Half, k4OffRaw = k4OffV + k4VStages * k4Half;
constexpr uint32_t k4Raw = k4Chunk * kKv4RowBytes;      // a chunk's rows as stored
constexpr size_t k4Smem = k4OffRaw + k4RawStages * k4Raw + 1024;
constexpr uint32_t k4ColO = 256, k4ColQ = 384;          // TMEM: S/P buffers at 0 and 128, O, Q
constexpr float k4Grow = 8.f;                           // log2: growth of the maximum that rescales

struct K4Chunk {
  int nc;            // MMA rows: the chunk's rows rounded up to 16 (0: none)
  int last;          // last chunk of its (query, split)
  uint32_t mask[4];  // bit r: row r is attended
  uint32_t raw[4];   // bit r: row r is a bf16 window row
};

struct K4Shared {
  uint64_t tab_full[k4Table], tab_empty[k4Table], k_full[k4KStages], k_empty[k4KStages], v_full[k4VStages];
  uint64_t raw_full[k4RawStages], raw_empty[k4RawStages];
  // o_done: a phase a chunk, whose P V is complete; o_last: a phase a (query, split), whose last P V is.
  // Waits are by parity, so a role may wait for a phase only when it knows the one before to be
  // complete.  S of a chunk is issued ahead of the P V of the chunk before, so a chunk's softmax knows
  // of the P V two chunks back: enough to wait for the one before its own, not for its own.
  uint64_t v_empty[k4VStages], s_full[2], p_full[2], max_full[4], sum_full[4], o_done, o_last, q_full, bail;
  uint32_t tmem;
  int abort;
  K4Chunk tab_meta[k4Table], meta[k4Table];
  // [chunk parity][column half][head], [parity of the (query, split)][half][head]: the two warps of a
  // group meet once a chunk with rows, and once a (query, split), so one of them may be a chunk or a
  // (query, split) ahead of the other's reads
  float half_max[2][2][128], half_sum[2][2][128];
  uint64_t row[k4Table][k4Chunk];               // address of each row; 0: skipped
};

__device__ __forceinline__ bool k4_wait(K4Shared& sh, uint64_t* bar, uint32_t phase, int* st) {
  return role_wait(bar, phase, &sh.abort, st);
}
__device__ __forceinline__ bool k4_wait_warp(K4Shared& sh, uint64_t* bar, uint32_t phase, int* st) {
  return role_wait_warp(bar, phase, &sh.abort, st);
}

// Byte offset of 16-byte piece c (0..15 of 128 bf16 dims) of row r in a K or V buffer.
__device__ __forceinline__ uint32_t k4_off(int r, int c) {
  return (uint32_t)(c >> 3) * k4Region + (uint32_t)r * 128 + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}
// Shared memory by 32-bit addresses (generic ones cost twice the arithmetic).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 bytes, or zeros with bytes = 0.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One E2M1 block: 16 bytes of codes at `src`, its scale code at `scale` -> four 16-byte pieces at
// `to`, whose places differ by xor.
__device__ __forceinline__ void put_e2m1_block(uint32_t src, uint32_t scale, uint32_t to) {
  const uint4 c = lds128(src);
  const uint32_t s = scale_bf16x2(lds_u8(scale));
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int v = 0; v < 4; ++v) sts128(to ^ (16u * v), e2m1x8_bf16(w[v], s));
}
// Sixteen E4M3 codes -> two pieces.
__device__ __forceinline__ void put_e4m3_half(uint32_t src, uint32_t scale, uint32_t to) {
  const uint4 c = lds128(src);
  const uint32_t s = scale_bf16x2(lds_u8(scale));
  sts128(to, e4m3x8_bf16(c.x, c.y, s));
  sts128(to ^ 16u, e4m3x8_bf16(c.z, c.w, s));
}

__global__ void __launch_bounds__(k4Threads, 1) attn_kv4_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t* buf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  __shared__ K4Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.max_splits, H = p.H;
  const int64_t items = (int64_t)p.T * S;

  const int quads = (H + 31) / 32, soft = 2 * quads;  // TMEM lane groups with heads, softmax warps at work
  // This warp's number among the decoding warps (0-3 K, 4-7 V).  A warp's scheduler is its number mod 4,
  // and the softmax warps have to be on their TMEM lanes' schedulers: with up to 64 heads those are two,
  // and three of four decoding warps go to the other two (4096 queries: 508 -> 479 us; all of them
  // there 534).
  int dec = warp < k4Copy ? warp - k4SoftWarps : -1;
  if (quads <= 2) dec = warp == 8 || warp == 9 ? warp - 2 : (warp & 2) && warp < 12 ? (warp >> 2) * 2 + (warp & 1) : -1;

  // ---- set-up that reads no input overlaps the previous kernel (dependent launch)
  if (warp == k4Mma) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < k4Table; ++i) {
      mbar_init(&sh.tab_full[i], 1);
      mbar_init(&sh.tab_empty[i], k4GatherWarps + k4CopyWarps);
    }
    for (int i = 0; i < k4RawStages; ++i) {
      mbar_init(&sh.raw_full[i], 32 * k4CopyWarps);
      mbar_init(&sh.raw_empty[i], k4GatherWarps);
    }
    for (int i = 0; i < k4KStages; ++i) {
      mbar_init(&sh.k_full[i], k4GatherWarps / 2);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < k4VStages; ++i) {
      mbar_init(&sh.v_full[i], k4GatherWarps / 2);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 2);
      mbar_init(&sh.p_full[i], soft);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.max_full[i], 2);
      mbar_init(&sh.sum_full[i], 2);
    }
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.o_last, 1);
    mbar_init(&sh.q_full, soft);
    mbar_init(&sh.bail, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();

  if (warp >= k4SoftWarps + k4GatherWarps) {
    if (warp == k4Resolve) {
      // ---------------------------------------------------------------- row lists
      uint32_t g = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const int t = (int)(item / S), split = (int)(item % S);
        const QueryRows q = query_rows(p, t);
        if (q.s < 0 && split == 0 && lane == 0) flag(p.st, CSKV_DEV_BAD_INDEX);
        const int64_t r0 = (int64_t)split * p.rows_per_split;
        const int64_t r1 = q.s < 0 ? r0 : max(r0, min(q.n_rows, r0 + p.rows_per_split));
        if (q.s >= 0 && split == S - 1 && lane == 0 && q.n_rows > r0 + p.rows_per_split) flag(p.st, CSKV_DEV_CAPACITY);
        const int chunks = max(1, (int)((r1 - r0 + k4Chunk - 1) / k4Chunk));
        // the selected entries of a chunk load one chunk ahead
        int32_t e[4];
        const bool csa = p.mode == CSKV_CSA;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t r = r0 + 32 * j + lane;
          e[j] = csa && r < r1 && r < q.n_cmp ? __ldg(p.idx + (size_t)t * p.k + r) : -2;
        }
        for (int c = 0; c < chunks && ok; ++c, ++g) {
          const int64_t a = r0 + (int64_t)c * k4Chunk;
          const int rows = (int)min((int64_t)k4Chunk, r1 - a);
          const int slot = g % k4Table;
          if (g >= k4Table) ok = k4_wait_warp(sh, &sh.tab_empty[slot], g / k4Table - 1, p.st);
          if (!ok) break;
          int32_t en[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t rn = a + k4Chunk + 32 * j + lane;
            en[j] = csa && rn < r1 && rn < q.n_cmp ? __ldg(p.idx + (size_t)t * p.k + rn) : -2;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 32 * j + lane;
            int64_t off = -1;
            bool is_raw = false;
            if (r < rows) off = resolve_row(p, q, t, a + r, &is_raw, e[j] < -1 ? (int64_t)-2 : (int64_t)e[j]);
            uint64_t at = 0;
            if (off >= 0)
              at = is_raw ? reinterpret_cast<uint64_t>(reinterpret_cast<const __nv_bfloat16*>(p.kv_raw) + off)
                          : reinterpret_cast<uint64_t>(p.kv_cmp) + (uint64_t)off / kRow * kKv4RowBytes;
            sh.row[slot][r] = at;
            const uint32_t m = __ballot_sync(0xffffffffu, off >= 0), mr = __ballot_sync(0xffffffffu, off >= 0 && is_raw);
            if (lane == 0) sh.tab_meta[slot].mask[j] = m, sh.tab_meta[slot].raw[j] = mr;
            e[j] = en[j];
          }
          if (lane == 0) {
            sh.tab_meta[slot].nc = max(0, (rows + 15) & ~15);
            sh.tab_meta[slot].last = c == chunks - 1;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.tab_full[slot]);
        }
      }
    } else if (warp < k4Mma) {
      // -------------------------------------------------------------- stored rows -> shared memory
      // As they are, 11 pieces of 16 bytes a row, neighbouring lanes on neighbouring pieces (a bulk
      // copy a row took 75 cycles each).  Skipped and window rows: zeros, which decode as zeros.
      const int first = (warp - k4Copy) * (k4Chunk / k4CopyWarps);
      uint32_t g = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; item < items && ok; ++g) {
        const uint32_t slot = g % k4Table, sr = g % k4RawStages;
        ok = k4_wait_warp(sh, &sh.tab_full[slot], g / k4Table, p.st) &&
             (g < k4RawStages || k4_wait_warp(sh, &sh.raw_empty[sr], g / k4RawStages - 1, p.st));
        if (!ok) break;
        const K4Chunk& m = sh.tab_meta[slot];
        if (m.last) item += gridDim.x;
        const uint32_t dst = smem_u32(buf) + k4OffRaw + sr * k4Raw + first * kKv4RowBytes;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          if (first + 32 * w >= m.nc) continue;
          const uint32_t have = m.mask[(first >> 5) + w] & ~m.raw[(first >> 5) + w];
          // 32 rows: 352 pieces, 11 a lane; the addresses first, so that the copies follow one another
          const uint8_t* at[11];
#pragma unroll
          for (int i = 0; i < 11; ++i) {
            const int x = lane + 32 * i, r = x / 11;
            at[i] = (have >> r) & 1u
                        ? reinterpret_cast<const uint8_t*>(sh.row[slot][first + 32 * w + r]) + 16 * (x - 11 * r)
                        : nullptr;
          }
#pragma unroll
          for (int i = 0; i < 11; ++i)
            cp16(dst + (w * 32 * 11 + lane + 32 * i) * 16, at[i] ? (const void*)at[i] : p.kv_cmp, at[i] ? 16u : 0u);
        }
        cp_async_arrive(&sh.raw_full[sr]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.tab_empty[slot]);
      }
      cp_async_wait_all();
    } else if (warp == k4Mma) {
      // -------------------------------------------------------------- MMA issue
      // Descriptors differ by their address field alone (16-byte units).
      const uint32_t kv = smem_u32(buf);
      const uint64_t d_k = smem_desc_sw128(kv, 16, 1024), d_v = smem_desc_sw128(kv + k4OffV, k4Region, 1024);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, false, true);
      uint32_t g = 0, n = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t c) {
        const uint32_t st = c % k4KStages;
        if (!k4_wait_warp(sh, &sh.k_full[st], c / k4KStages, p.st)) return false;
        tc_fence_after();
        const int nc = sh.meta[c % k4Table].nc;
        const uint32_t idesc = idesc_bf16_f32(128, nc, false, false), tS = tmem + (c & 1) * 128;
        const uint64_t d = d_k + st * (k4Half >> 4);
        if (elect_one()) {
          if (nc) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_f16_ta(tS, tmem + k4ColQ + kk * 8, d + (kk >> 2) * (k4Region >> 4) + (kk & 3) * 2, idesc, kk > 0);
          }
          tc_commit(&sh.k_empty[st]);
          tc_commit(&sh.s_full[c & 1]);
          mbar_arrive(&sh.s_full[c & 1]);  // passes the chunk's notes on to the softmax warps
        }
        __syncwarp();
        return true;
      };
      for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x, ++n) {
        ok = k4_wait_warp(sh, &sh.q_full, n, p.st);
        tc_fence_after();
        ok = ok && issue_s(g);
        bool first = true;
        for (bool more = true; more && ok; ++g) {
          const uint32_t st = g % k4VStages;
          const int nc = sh.meta[g % k4Table].nc;
          more = !sh.meta[g % k4Table].last;
          // the next chunk's S goes first if its K is there before this chunk's P
          bool ahead = false;
          if (more) {
            for (int i = 0; i < (1 << 22) && !ahead && !__all_sync(0xffffffffu, mbar_test(&sh.p_full[g & 1], (g >> 1) & 1u)); ++i) {
              if (__all_sync(0xffffffffu, mbar_try_wait(&sh.k_full[(g + 1) % k4KStages], ((g + 1) / k4KStages) & 1u))) {
                ahead = true;
                ok = issue_s(g + 1);
              }
            }
          }
          ok = ok && k4_wait_warp(sh, &sh.v_full[st], g / k4VStages, p.st) &&
               k4_wait_warp(sh, &sh.p_full[g & 1], g >> 1, p.st);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tP = tmem + (g & 1) * 128;
          const uint64_t d = d_v + st * (k4Half >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (kk * 16 < nc)
                tc_mma_f16_ta(tmem + k4ColO, tP + (kk >> 2) * 64 + (kk & 3) * 8, d + kk * 128, idesc_o, !first || kk > 0);
            tc_commit(&sh.v_empty[st]);
            tc_commit(&sh.o_done);
            if (!more) tc_commit(&sh.o_last);
          }
          __syncwarp();
          if (nc) first = false;
          if (more && !ahead) ok = issue_s(g + 1);
        }
      }
      if (!ok && elect_one()) {  // gave up: nothing of this CTA may still be in flight when its memory is released
        tc_commit(&sh.bail);
        mbar_wait_bounded(&sh.bail, 0);
      }
      __syncwarp();
    }
  } else if (dec >= 0) {
    // ---------------------------------------------------------------- rows -> bf16 in shared memory
    // Warps 0-3 of the eight decode K, the others V, 32 rows each, a few rows at a time through
    // short loops.  E2M1: sixteen rows' K blocks (lane l: row l % 16, block l / 16) or eight rows'
    // V blocks (row l % 8, block l / 8); E4M3: eight rows' sixteen codes (row l % 8, piece l / 8).
    // Eight neighbouring lanes hold the same piece of eight rows: their swizzled stores meet all
    // banks once, and so do their loads of rows 176 bytes apart.
    const int gw = dec & 3, l8 = lane & 7, l16 = lane & 15, pv = lane >> 3, pk = lane >> 4;
    const bool is_v = dec >= 4;
    const int row0 = gw * 32;
    // a lane's E2M1 block of each step of e2m1_rows rows: one code for K and V, two blocks a turn, since
    // the instruction cache is what counts (one code each 474 us, four blocks a turn 575)
    const int e2m1_rows = is_v ? 8 : 16, lr = is_v ? l8 : l16;
    const uint32_t e2m1_code = lr * kKv4RowBytes + (is_v ? kKv4V + 16 * pv : 16 * pk);
    const uint32_t e2m1_scale = lr * kKv4RowBytes + kKv4Scales + (is_v ? 4 + pv : pk);
    const uint32_t e2m1_to = k4_off(row0 + lr, 4 * (is_v ? pv : pk));
    const uint32_t base = smem_u32(buf), raw_base = base + k4OffRaw + row0 * kKv4RowBytes;
    uint32_t g = 0;
    bool ok = true;
    for (int64_t item = blockIdx.x; item < items && ok; ++g) {
      const uint32_t slot = g % k4Table, sr = g % k4RawStages, sk = g % k4KStages, sv = g % k4VStages;
      ok = k4_wait_warp(sh, &sh.tab_full[slot], g / k4Table, p.st) &&
           k4_wait_warp(sh, &sh.raw_full[sr], g / k4RawStages, p.st) &&
           (is_v ? (g < k4VStages || k4_wait_warp(sh, &sh.v_empty[sv], g / k4VStages - 1, p.st))
                 : (g < k4KStages || k4_wait_warp(sh, &sh.k_empty[sk], g / k4KStages - 1, p.st)));
      if (!ok) break;
      const K4Chunk& m = sh.tab_meta[slot];
      if (m.last) item += gridDim.x;
      const uint32_t raw = m.raw[gw];  // window rows among this warp's 32
      const uint32_t src = raw_base + sr * k4Raw;
      const uint32_t dst = base + (is_v ? k4OffV + sv * k4Half : sk * k4Half);
      if (row0 < m.nc) {
        if (raw != 0xFFFFFFFFu) {
          uint32_t code = src + e2m1_code, scale = src + e2m1_scale, put = dst + e2m1_to;
#pragma unroll 1
          for (int j = 0; j < 32; j += 2 * e2m1_rows) {  // two blocks a turn
            put_e2m1_block(code, scale, put);
            put_e2m1_block(code + e2m1_rows * kKv4RowBytes, scale + e2m1_rows * kKv4RowBytes, put + e2m1_rows * 128);
            code += 2 * e2m1_rows * kKv4RowBytes, scale += 2 * e2m1_rows * kKv4RowBytes, put += 2 * e2m1_rows * 128;
          }
          if (!is_v) {
            uint32_t at = src + l8 * kKv4RowBytes, to = dst + k4_off(row0 + l8, 8 + 2 * pv);
#pragma unroll 1
            for (int j = 0; j < 4; ++j, at += 8 * kKv4RowBytes, to += 8 * 128)
              put_e4m3_half(at + kKv4Rope + 16 * pv, at + kKv4Scales + 2 + (pv >> 1), to);
          }
        }
        if (raw) {
          // window rows: a half warp copies half a row (16 bytes a lane) straight to its place, over
          // the zeros decoded for it
          __syncwarp();
#pragma unroll 1
          for (int r = pk; r < 32; r += 2)
            if ((raw >> r) & 1u)
              cp16(dst + k4_off(row0 + r, l16),
                   reinterpret_cast<const uint8_t*>(sh.row[slot][row0 + r]) + (is_v ? 256 : 0) + 16 * l16, 16u);
          cp_async_wait_all();
        }
      }
      if (dec == 0 && lane == 0) sh.meta[slot] = m;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(is_v ? &sh.v_full[sv] : &sh.k_full[sk]);
        mbar_arrive(&sh.raw_empty[sr]);
        mbar_arrive(&sh.tab_empty[slot]);
      }
    }
  } else if (warp < k4SoftWarps) {
    // ---------------------------------------------------------------- softmax and output
    // warps w and w + 4 share the TMEM lanes of heads 32w .. 32w + 31: each takes half of a
    // chunk's columns, of Q's and of O's dims, and they exchange row maxima and sums
    const int quad = warp & 3, half = warp >> 2, h = quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float sl2 = p.scale_log2;
    const float sk = (p.sink && h < H) ? __ldg(p.sink + h) * kLog2e : -INFINITY;
    auto put_q = [&](int64_t item) {
      {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                          ((size_t)(item / S) * H + h) * kHeadDim + 64 * half);
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 w = h < H ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
          v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
        }
        tmem_st32(tmem + k4ColQ + lane_base + 32 * half, v);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    };
    uint32_t g = 0, n = 0;
    bool ok = true;
    if (quad < quads && blockIdx.x < items) put_q(blockIdx.x);
    for (int64_t item = quad < quads ? blockIdx.x : items; item < items && ok; item += gridDim.x, ++n) {
      float m = -INFINITY, l = 0.f;
      bool filled = false;  // O holds something
      for (bool more = true; more; ++g) {
        const uint32_t st = g % k4Table, sp = g & 1;
        ok = k4_wait_warp(sh, &sh.s_full[sp], g >> 1, p.st);
        if (!ok) break;
        tc_fence_after();
        const int nc = sh.meta[st].nc;
        more = !sh.meta[st].last;
        const uint32_t tS = tmem + sp * 128 + 64 * half + lane_base;
        if (nc) {
          // this half's 64 columns, 16 at a time; those past nc hold old values, and their mask bits
          // are clear
          const uint32_t vm0 = sh.meta[st].mask[2 * half], vm1 = sh.meta[st].mask[2 * half + 1];
          const bool whole = (vm0 & vm1) == 0xFFFFFFFFu;
          auto columns = [&](int c, uint32_t (&v)[16]) {
            tmem_ld16(tS + c, v);
            tmem_ld_wait();
            if (!whole) {
              const uint32_t b = (c < 32 ? vm0 : vm1) >> (c & 31);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!((b >> i) & 1u)) v[i] = 0xFF800000u;  // -inf
            }
          };
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t v[16];
            columns(c, v);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              mx4[(i >> 1) & 3] = fmaxf(mx4[(i >> 1) & 3], fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
          }
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          sh.half_max[sp][half][h] = mx;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.max_full[quad]);
          ok = k4_wait_warp(sh, &sh.max_full[quad], g, p.st);
          if (!ok) break;
          mx = fmaxf(mx, sh.half_max[sp][half ^ 1][h]) * sl2;
          const float m_new = mx > m + k4Grow || m == -INFINITY ? fmaxf(mx, m) : m;
          const float alpha = m_new == -INFINITY || m_new == m ? 1.f : fast_exp2(m - m_new);
          const float nm = m_new == -INFINITY ? 0.f : -m_new;
          // P = 2^(s scale - m) as bf16, over this half's columns that have been read
          const uint64_t sl2x2 = pack2(sl2, sl2), nmx2 = pack2(nm, nm);
          uint64_t l2[2] = {0ull, 0ull};
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t v[16], w[8];
            columns(c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sl2x2, nmx2), e0, e1);
              e0 = fast_exp2(e0), e1 = fast_exp2(e1);
              l2[i & 1] = add2(l2[i & 1], pack2(e0, e1));
              const __nv_bfloat162 e = __floats2bfloat162_rn(e0, e1);
              w[i] = *reinterpret_cast<const uint32_t*>(&e);
            }
            tmem_st8(tS + (c >> 1), w);
          }
          // O of the earlier chunks is rescaled once its last product is complete (tensor-memory
          // accesses are warp-wide, so a warp rescales when one of its rows needs it)
          if (filled && __any_sync(0xffffffffu, alpha != 1.f)) {
            ok = k4_wait_warp(sh, &sh.o_done, g - 1, p.st);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tO = tmem + k4ColO + lane_base + 64 * half;
#pragma unroll 1
            for (int cc = 0; cc < 64; cc += 16) {
              uint32_t o[16];
              tmem_ld16(tO + cc, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + cc, o);
            }
          }
          tmem_st_wait();
          float la, lb;
          unpack2(add2(l2[0], l2[1]), la, lb);
          l = l * alpha + (la + lb);
          m = m_new;
        } else if (lane == 0) {
          mbar_arrive(&sh.max_full[quad]);
        }
        filled = filled || nc > 0;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[sp]);
      }
      if (!ok) break;
      // every S of this query is complete: the next query's Q may take its place
      if (item + gridDim.x < items) put_q(item + gridDim.x);
      sh.half_sum[n & 1][half][h] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sum_full[quad]);
      ok = k4_wait_warp(sh, &sh.sum_full[quad], n, p.st) && k4_wait_warp(sh, &sh.o_last, n, p.st);
      if (!ok) break;
      tc_fence_after();
      l += sh.half_sum[n & 1][half ^ 1][h];
      // maxima pass over NaN, sums do not: logits that are all NaN (or NaN and masked) leave l = NaN under
      // m = -inf, which below and in the merge stands for no rows; any finite reference keeps them
      if (l != l && m == -INFINITY) m = 0.f;
      const int t = (int)(item / S), split = (int)(item % S);
      const uint32_t tO = tmem + k4ColO + lane_base + 64 * half;
      if (S == 1) {
        const float M = fmaxf(m, sk);
        float f = 0.f, L = 0.f;
        if (M != -INFINITY) {
          f = m == -INFINITY ? 0.f : exp2f(m - M);
          L = l * f + (p.sink ? exp2f(sk - M) : 0.f);
        }
        const float inv = L > 0.f || L != L ? f / L : 0.f;
        const size_t row = ((size_t)t * H + h) * kHeadDim + 64 * half;
#pragma unroll 1
        for (int cc = 0; cc < 64; cc += 16) {
          uint32_t v[16];
          __syncwarp();
          if (filled) {
            tmem_ld16(tO + cc, v);
            tmem_ld_wait();
          }
          if (h < H) {
            // a row without attended columns has no O of its own
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
              float o[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = filled && inv != 0.f ? __uint_as_float(v[i + j]) * inv : 0.f;
              if (p.out_bf16)
                Vec8<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(p.out) + row + cc + i, o);
              else
                Vec8<float>::store(p.out + row + cc + i, o);
            }
          }
        }
        if (half == 0 && h < H && p.lse)
          p.lse[(size_t)t * H + h] = L > 0.f || L != L ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
      } else {
        // partial for the merge kernel: [query][split][head][dim], (m, l) [query][split][head] (m =
        // -inf: no rows, and no partial)
        const size_t sb = ((size_t)t * S + split) * H + h;
        float* dst = p.part_acc + sb * kHeadDim + 64 * half;
        if (filled) {
#pragma unroll 1
          for (int cc = 0; cc < 64; cc += 16) {
            uint32_t v[16];
            __syncwarp();
            tmem_ld16(tO + cc, v);
            tmem_ld_wait();
            if (h < H) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(dst + cc + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        }
        if (half == 0 && h < H) reinterpret_cast<float2*>(p.part_ml)[sb] = make_float2(m, l);
      }
      tc_fence_before();
    }
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == k4Mma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merges the splits of a query ([TR] §3.1), the sink once ([SW] §十二): M = max(max_s m_s, sink),
// L = sum_s 2^(m_s - M) l_s + 2^(sink - M), o = sum_s 2^(m_s - M) acc_s / L.  A CTA a head, its two to
// eight warps a share of the splits each, a lane four dims.  Bound by latency: eight splits' loads
// of a warp go out together.
constexpr int k4MergeWarps = 8;

__global__ void __launch_bounds__(32 * k4MergeWarps) attn_kv4_merge_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float4 part[k4MergeWarps][32];
  __shared__ float part_l[k4MergeWarps];
  const int t = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.H, S = p.max_splits, warps = blockDim.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const size_t sb = (size_t)t * S * H + h;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + sb;
  const float4* acc = reinterpret_cast<const float4*>(p.part_acc + sb * kHeadDim) + lane;
  const float sk = p.sink ? __ldg(p.sink + h) * kLog2e : -INFINITY;
  float M = sk;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, __ldcg(ml + (size_t)s * H).x);
  M = warp_max(M);
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = warp; s < S; s += warps) {
    const float2 x = __ldcg(ml + (size_t)s * H);
    const float4 a = __ldcg(acc + (size_t)s * H * (kHeadDim / 4));
    if (x.x != -INFINITY) {
      const float f = exp2f(x.x - M);
      L = fmaf(x.y, f, L);
      o.x = fmaf(a.x, f, o.x), o.y = fmaf(a.y, f, o.y), o.z = fmaf(a.z, f, o.z), o.w = fmaf(a.w, f, o.w);
    }
  }
  part[warp][lane] = o;
  if (lane == 0) part_l[warp] = L;
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < warps; ++w) {
    const float4 a = part[w][lane];
    o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
    L += part_l[w];
  }
  if (p.sink && M != -INFINITY) L += exp2f(sk - M);
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  const size_t dst = ((size_t)t * H + h) * kHeadDim + 4 * lane;
  if (p.out_bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + dst) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(p.out + dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
  if (lane == 0 && p.lse) p.lse[(size_t)t * H + h] = L > 0.f || L != L ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
}

// Splits of a query: whole chunks, as many as fill the SMs once, but no more than pay: a chunk takes
// about 1.5 us, a split more about 0.05 us of the merge.
void attn_kv4_plan(int T, int64_t rows_max, int sms, int* R, int* S) {
  const int64_t chunks = rows_max > 0 ? (rows_max + k4Chunk - 1) / k4Chunk : 1;
  const int64_t can = T < sms ? sms / T : 1, one = (chunks + can - 1) / can;
  int64_t per = one;  // chunks of a split
  auto cost = [&](int64_t n) { return 30 * n + (chunks + n - 1) / n; };
  while (per < 2 * one && per < chunks && cost(per + 1) < cost(per)) ++per;
  *R = (int)(per * k4Chunk);
  *S = (int)((chunks + per - 1) / per);
}

cudaError_t launch_attn_kv4(const AttnParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = ensure_smem(attn_kv4_kernel, k4Smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.T * p.max_splits;
  e = launch_dependent(attn_kv4_kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(k4Threads), k4Smem, stream, p);
  note_launch();
  if (e != cudaSuccess || p.max_splits == 1) return e;
  e = ensure_smem(attn_kv4_merge_kernel, 0);
  if (e != cudaSuccess) return e;
  const int warps = p.max_splits <= 2 ? 2 : p.max_splits <= 16 ? 4 : k4MergeWarps;
  e = launch_dependent(attn_kv4_merge_kernel, dim3(p.H, p.T), dim3(32 * warps), 0, stream, p);
  note_launch();
  return e;
}

}  // namespace cskv
