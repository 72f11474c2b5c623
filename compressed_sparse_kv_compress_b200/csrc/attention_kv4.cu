// Hybrid attention over a compressed cache in 4-bit rows (mx4.cuh), bf16 queries, on tcgen05.
//
// [SW] = shareware.cn/news/167317: §十三.4 (the main KV in few bits, position-sensitive dims
// higher), §十一 (MQA: the heads share one KV), §十二 (sink).  [TR] = trdm.cn/news/516303, §3.1
// (online softmax).
//
// Formula, per query and head: o = softmax(scale q K^T with the sink) V over the query's row list
// (attn_rows.cuh).  Decoded rows are exact in bf16, so the products are those of exact rows
// with fp32 accumulation; P is rounded to bf16 for P V (its sum is kept in fp32).
//
// What bounds it: a chunk of 128 rows is 2 x 128^3 MMA operations a head tile (1024 cycles of an
// SM's tensor pipe), 128 x 128 exponentials (1024 cycles at 16 a cycle) and 32K decoded values
// (about 4 ALU operations a pair, 1024 cycles at 64 a cycle), against 22.5 KB of rows: for many
// queries it is bound by arithmetic on all three pipes, so one persistent CTA an SM keeps them
// busy at once with specialised warps; for a few queries it is a latency chain, so a query's rows
// are split over the SMs.
//   warp 13     resolves row lists into a table of row addresses, up to four chunks ahead
//   warps 4-11  load rows (16 bytes of codes a lane, the next chunk's loads in flight while this
//               one is decoded), decode to bf16 and store them in the 128-byte-swizzle layout
//   warp 12     one thread issues S = Q K^T and O (+)= P V; Q and P are A operands in tensor
//               memory, so only K and V are read from shared memory
//   warps 0-3   softmax: TMEM lane h is head h; S -> P in place, O rescaled when the running
//               maximum grows by more than 2^8 (any reference serves the online softmax), output
// Two chunk buffers (64 KB each) and two S / P buffers pipeline the chunks, across queries too.
#include "attn_rows.cuh"
#include "mx4.cuh"
#include "sm100.cuh"

namespace cskv {

constexpr int k4Chunk = 128;                            // rows of a chunk
constexpr int k4GatherWarps = 8, k4GatherThreads = 32 * k4GatherWarps;
constexpr int k4Mma = 4 + k4GatherWarps, k4Resolve = k4Mma + 1;
constexpr int k4Threads = 32 * (k4Resolve + 1);
constexpr int k4Table = 4;                              // chunks the row table holds
constexpr uint32_t k4Region = 128 * 128;                // 128 rows x 128 bytes: one swizzled region
constexpr uint32_t k4Stage = 4 * k4Region;              // K dims 0-63, 64-127, V dims 0-63, 64-127
constexpr size_t k4Smem = 2 * (size_t)k4Stage + 1024;
constexpr uint32_t k4ColO = 256, k4ColQ = 384;          // TMEM: S/P buffers at 0 and 128, O, Q
constexpr float k4Grow = 8.f;                           // log2: growth of the maximum that rescales

struct K4Chunk {
  int nc;            // MMA rows: the chunk's rows rounded up to 16 (0: none)
  int last;          // last chunk of its (query, split)
  int raw;           // holds raw window rows
  uint32_t mask[4];  // bit r: row r is attended
};

struct K4Shared {
  uint64_t tab_full[k4Table], tab_empty[k4Table], kv_full[2], kv_empty[2], s_full[2], p_full[2], o_done, q_full, bail;
  uint32_t tmem;
  int abort;
  K4Chunk tab_meta[k4Table], meta[2];
  uint64_t row[k4Table][k4Chunk];  // row address; 0 skipped; bit 0: a raw bf16 row
};

// Waits for phase `phase` of a barrier.  Bounded: one role that gives up makes every role of the
// CTA leave its loop.
__device__ __forceinline__ bool k4_wait(K4Shared& sh, uint64_t* bar, uint32_t phase, int* st) {
  for (int i = 0; i < (1 << 22); ++i) {
    if (mbar_try_wait(bar, phase & 1u)) return true;
    if (*(volatile int*)&sh.abort) return false;
  }
  *(volatile int*)&sh.abort = 1;
  flag(st, CSKV_DEV_TIMEOUT);
  return false;
}
// The same for a whole warp, whose lanes agree on the answer.
__device__ __forceinline__ bool k4_wait_warp(K4Shared& sh, uint64_t* bar, uint32_t phase, int* st) {
  return __all_sync(0xffffffffu, k4_wait(sh, bar, phase, st));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 2^(e - 127) twice, as bf16 (2^-127 is a subnormal; 0xFF is NaN).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t e) {
  const uint32_t b = e == 0xFFu ? 0x7FC0u : e == 0 ? 0x0040u : e << 7;
  return b * 0x00010001u;
}
// Four E2M1 codes (16 bits of w) -> two words of bf16 pairs: the high and low byte of each
// magnitude come from 8-byte tables by byte permute; a selector nibble's top bit (the sign) turns
// the selected 0x80 into 0xFF, whose low bit moves to the sign place.
__device__ __forceinline__ void e2m1x4_bf16(uint32_t w, uint32_t wm, uint32_t s, uint32_t& o0, uint32_t& o1) {
  const uint32_t hi = prmt(0x3F3F3F00u, 0x40404040u, wm), lo = prmt(0xC0800000u, 0xC0804000u, wm);
  const uint32_t sg = prmt(0x80808080u, 0x80808080u, w);
  const uint32_t hs = hi | ((sg << 7) & 0x80808080u);
  o0 = mul_bf16x2(prmt(lo, hs, 0x5140u), s);
  o1 = mul_bf16x2(prmt(lo, hs, 0x7362u), s);
}
__device__ __forceinline__ uint4 e2m1x8_bf16(uint32_t w, uint32_t s) {
  uint4 o;
  const uint32_t wm = w & 0x77777777u;
  e2m1x4_bf16(w, wm, s, o.x, o.y);
  e2m1x4_bf16(w >> 16, wm >> 16, s, o.z, o.w);
  return o;
}
// Two E4M3 codes in the high bytes of h's halves -> bf16: exponent and mantissa moved into place
// (value * 2^-120), then two exact products (one would overflow the factor for large scales).
__device__ __forceinline__ uint32_t e4m3x2_bf16(uint32_t h, uint32_t s) {
  const uint32_t b = ((h >> 4) & 0x07F007F0u) | (h & 0x80008000u);
  return mul_bf16x2(mul_bf16x2(b, 0x7B807B80u), s);
}
__device__ __forceinline__ uint4 e4m3x8_bf16(uint32_t w0, uint32_t w1, uint32_t s) {
  return make_uint4(e4m3x2_bf16(prmt(w0, 0u, 0x1404u), s), e4m3x2_bf16(prmt(w0, 0u, 0x3424u), s),
                    e4m3x2_bf16(prmt(w1, 0u, 0x1404u), s), e4m3x2_bf16(prmt(w1, 0u, 0x3424u), s));
}

// Byte offset of 16-byte piece c (0..31 of the 512-byte bf16 row) of row r in a chunk buffer.
__device__ __forceinline__ uint32_t k4_off(int r, int c) {
  return (uint32_t)(c >> 3) * k4Region + (uint32_t)r * 128 + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}

// One thread's share of a chunk's codes: three E2M1 blocks and one E4M3 block.
struct K4Codes {
  uint4 c4[3], c8[2];
  uint32_t e[4];  // scale codes; bit 8: the row is skipped, bit 9: not a 4-bit row of this chunk
};

__global__ void __launch_bounds__(k4Threads, 1) attn_kv4_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t* buf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  __shared__ K4Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.max_splits, H = p.H;
  const int64_t items = (int64_t)p.T * S;

  // ---- set-up that reads no input overlaps the previous kernel (dependent launch)
  if (warp == k4Mma) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < k4Table; ++i) {
      mbar_init(&sh.tab_full[i], 1);
      mbar_init(&sh.tab_empty[i], k4GatherWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kv_full[i], k4GatherWarps);
      mbar_init(&sh.kv_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
    }
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.q_full, 4);
    mbar_init(&sh.bail, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();

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
      int64_t e[4];
      const bool csa = p.mode == CSKV_CSA;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + 32 * j + lane;
        e[j] = csa && r < r1 && r < q.n_cmp ? (int64_t)__ldg(p.idx + (size_t)t * p.k + r) : -2;
      }
      for (int c = 0; c < chunks && ok; ++c, ++g) {
        const int64_t a = r0 + (int64_t)c * k4Chunk;
        const int rows = (int)min((int64_t)k4Chunk, r1 - a);
        const int slot = g % k4Table;
        if (g >= k4Table) ok = k4_wait_warp(sh, &sh.tab_empty[slot], g / k4Table - 1, p.st);
        if (!ok) break;
        uint32_t raw_any = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 32 * j + lane;
          int64_t off = -1;
          bool is_raw = false;
          if (r < rows) off = resolve_row(p, q, t, a + r, &is_raw, e[j] < -1 ? (int64_t)-2 : e[j]);
          uint64_t at = 0;
          if (off >= 0)
            at = is_raw ? reinterpret_cast<uint64_t>(reinterpret_cast<const __nv_bfloat16*>(p.kv_raw) + off) | 1u
                        : reinterpret_cast<uint64_t>(p.kv_cmp) + (uint64_t)(off / kRow) * kKv4RowBytes;
          sh.row[slot][r] = at;
          const uint32_t m = __ballot_sync(0xffffffffu, off >= 0);
          raw_any |= __ballot_sync(0xffffffffu, off >= 0 && is_raw);
          if (lane == 0) sh.tab_meta[slot].mask[j] = m;
          const int64_t rn = a + k4Chunk + r;
          e[j] = csa && rn < r1 && rn < q.n_cmp ? (int64_t)__ldg(p.idx + (size_t)t * p.k + rn) : -2;
        }
        if (lane == 0) {
          sh.tab_meta[slot].nc = max(0, (rows + 15) & ~15);
          sh.tab_meta[slot].last = c == chunks - 1;
          sh.tab_meta[slot].raw = raw_any != 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.tab_full[slot]);
      }
    }
  } else if (warp >= 4 && warp < k4Mma) {
    // ---------------------------------------------------------------- rows -> bf16 in shared memory
    const int gt = tid - 128, gw = warp - 4;
    // E2M1 blocks i = gt + 256 j of the chunk's 768: row i / 6, block i % 6 (K blocks 0, 1, V
    // blocks 4..7); the E4M3 block: row gt / 2, block 2 + gt % 2
    const int r8 = gt >> 1, b8 = 2 + (gt & 1);
    auto load = [&](uint32_t g, K4Codes& k) {
      const int slot = g % k4Table;
      const int nc = sh.tab_meta[slot].nc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = gt + k4GatherThreads * j;
        const int r = j < 3 ? i / 6 : r8;
        const int b6 = i % 6, b = j < 3 ? (b6 < 2 ? b6 : b6 + 2) : b8;
        const uint64_t at = r < nc ? sh.row[slot][r] : 1;
        const uint8_t* row = reinterpret_cast<const uint8_t*>(at);
        k.e[j] = at == 0 ? 0x100u : (at & 1) ? 0x200u : 0u;
        if (k.e[j] == 0) {
          k.e[j] = __ldg(row + kKv4Scales + b);
          if (j < 3) {
            k.c4[j] = __ldg(reinterpret_cast<const uint4*>(row + (b < 2 ? 16 * b : kKv4V + 16 * (b - 4))));
          } else {
            k.c8[0] = __ldg(reinterpret_cast<const uint4*>(row + kKv4Rope + 32 * (b - 2)));
            k.c8[1] = __ldg(reinterpret_cast<const uint4*>(row + kKv4Rope + 32 * (b - 2)) + 1);
          }
        }
      }
    };
    uint32_t g = 0;
    bool ok = true;
    int64_t item = blockIdx.x;
    K4Codes cur, nxt;
    if (item < items) {
      ok = k4_wait_warp(sh, &sh.tab_full[0], 0, p.st);
      if (ok) load(0, cur);
    }
    while (item < items && ok) {
      const int slot = g % k4Table, st = g & 1;
      const K4Chunk meta = sh.tab_meta[slot];
      if (meta.last) item += gridDim.x;
      if (item < items) {  // there is a next chunk: its loads go out before this one is decoded
        ok = k4_wait_warp(sh, &sh.tab_full[(g + 1) % k4Table], (g + 1) / k4Table, p.st);
        if (!ok) break;
        load(g + 1, nxt);
      }
      if (g >= 2) ok = k4_wait_warp(sh, &sh.kv_empty[st], (g >> 1) - 1, p.st);
      if (!ok) break;
      uint8_t* dst = buf + st * k4Stage;
      if (meta.raw) {
        // window rows: a warp copies whole 512-byte rows, a lane 16 bytes
        for (int r = gw; r < meta.nc; r += k4GatherWarps) {
          const uint64_t at = sh.row[slot][r];
          if (at & 1) cp_async16(dst + k4_off(r, lane), reinterpret_cast<const uint8_t*>(at - 1) + 16 * lane, 16u);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (cur.e[j] & 0x200u) continue;
        const int i = gt + k4GatherThreads * j;
        const int r = j < 3 ? i / 6 : r8;
        const int b6 = i % 6, b = j < 3 ? (b6 < 2 ? b6 : b6 + 2) : b8;
        const bool skip = cur.e[j] & 0x100u;
        const uint32_t s = scale_bf16x2(cur.e[j] & 0xFFu);
        // the four pieces of a block in an order that differs between the lanes of a row, so that
        // a quarter warp's stores meet different banks
        const int rot = j < 3 ? b6 >> 1 : 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint4 o = make_uint4(0u, 0u, 0u, 0u);
          int pc;
          if (j < 3) {
            pc = (v + rot) & 3;
            const uint4 c = cur.c4[j];
            const uint32_t w = pc == 0 ? c.x : pc == 1 ? c.y : pc == 2 ? c.z : c.w;
            if (!skip) o = e2m1x8_bf16(w, s);
          } else {
            pc = v;
            const uint4 c = cur.c8[v >> 1];
            if (!skip) o = (v & 1) ? e4m3x8_bf16(c.z, c.w, s) : e4m3x8_bf16(c.x, c.y, s);
          }
          *reinterpret_cast<uint4*>(dst + k4_off(r, 4 * b + pc)) = o;
        }
      }
      if (gt == 0) sh.meta[st] = meta;
      if (meta.raw) cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.tab_empty[slot]);
        mbar_arrive(&sh.kv_full[st]);
      }
      cur = nxt;
      ++g;
    }
  } else if (warp == k4Mma) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t kv = smem_u32(buf);
      uint32_t g = 0, n = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t c) {
        const int st = c & 1;
        if (!k4_wait(sh, &sh.kv_full[st], c >> 1, p.st)) return false;
        tc_fence_after();
        const int nc = sh.meta[st].nc;
        if (nc) {
          const uint32_t idesc = idesc_bf16_f32(128, nc, false, false);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_f16_ta(tmem + st * 128, tmem + k4ColQ + kk * 8,
                          smem_desc_sw128(kv + st * k4Stage + (uint32_t)(kk >> 2) * k4Region + (uint32_t)(kk & 3) * 32,
                                          16, 1024),
                          idesc, kk > 0);
        }
        tc_commit(&sh.s_full[st]);
        return true;
      };
      for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x, ++n) {
        ok = k4_wait(sh, &sh.q_full, n, p.st);
        tc_fence_after();
        ok = ok && issue_s(g);
        bool first = true;
        for (bool more = true; more && ok; ++g) {
          const int st = g & 1;
          const int nc = sh.meta[st].nc;
          more = !sh.meta[st].last;
          if (more) ok = issue_s(g + 1);
          ok = ok && k4_wait(sh, &sh.p_full[st], g >> 1, p.st);
          if (!ok) break;
          tc_fence_after();
          const uint32_t idesc = idesc_bf16_f32(128, 128, false, true);
          for (int kk = 0; kk < nc / 16; ++kk)
            tc_mma_f16_ta(tmem + k4ColO, tmem + st * 128 + kk * 8,
                          smem_desc_sw128(kv + st * k4Stage + 2 * k4Region + (uint32_t)kk * 2048, k4Region, 1024),
                          idesc, !first || kk > 0);
          if (nc) first = false;
          tc_commit(&sh.kv_empty[st]);
          tc_commit(&sh.o_done);
        }
      }
      if (!ok) {  // gave up: nothing of this CTA may still be in flight when its memory is released
        tc_commit(&sh.bail);
        mbar_wait_bounded(&sh.bail, 0);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int h = tid;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const bool active = warp * 32 < H;  // a warp without heads only keeps the barriers in step
    const float sl2 = p.scale_log2;
    const float sk = (p.sink && h < H) ? __ldg(p.sink + h) * kLog2e : -INFINITY;
    auto put_q = [&](int64_t item) {
      if (active) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                          ((size_t)(item / S) * H + h) * kHeadDim);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = h < H ? __ldg(src + 8 * half + i) : make_uint4(0u, 0u, 0u, 0u);
            v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
          }
          tmem_st32(tmem + k4ColQ + lane_base + 32 * half, v);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    };
    uint32_t g = 0;
    bool ok = true;
    if (blockIdx.x < items) put_q(blockIdx.x);
    for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x) {
      float m = -INFINITY, l = 0.f;
      bool filled = false;  // O holds something
      for (bool more = true; more; ++g) {
        const int st = g & 1;
        ok = k4_wait_warp(sh, &sh.kv_full[st], g >> 1, p.st) &&  // the chunk's description
             k4_wait_warp(sh, &sh.s_full[st], g >> 1, p.st);
        if (!ok) break;
        tc_fence_after();
        const int nc = sh.meta[st].nc;
        more = !sh.meta[st].last;
        const uint32_t tS = tmem + st * 128 + lane_base;
        if (active && nc) {
          // pass 1: the row maximum over attended columns (columns past nc hold old values; their
          // mask bits are clear)
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          for (int cc = 0; cc < nc; cc += 32) {
            const uint32_t vm = sh.meta[st].mask[cc >> 5];
            uint32_t v[32];
            tmem_ld32(tS + cc, v);
            tmem_ld_wait();
            if (vm == 0xFFFFFFFFu) {
#pragma unroll
              for (int i = 0; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(v[i]));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                mx4[i & 3] = fmaxf(mx4[i & 3], ((vm >> i) & 1u) ? __uint_as_float(v[i]) : -INFINITY);
            }
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          const float m_new = mx > m + k4Grow || m == -INFINITY ? fmaxf(mx, m) : m;
          const float alpha = m_new == -INFINITY || m_new == m ? 1.f : fast_exp2(m - m_new);
          const float nm = m_new == -INFINITY ? 0.f : -m_new;
          // pass 2: P = 2^(s scale - m) as bf16 over the columns already read
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
          for (int cc = 0; cc < nc; cc += 32) {
            const uint32_t vm = sh.meta[st].mask[cc >> 5];
            uint32_t v[32], w[16];
            tmem_ld32(tS + cc, v);
            tmem_ld_wait();
            float e[32];
            if (vm == 0xFFFFFFFFu) {
#pragma unroll
              for (int i = 0; i < 32; ++i) e[i] = fast_exp2(fmaf(__uint_as_float(v[i]), sl2, nm));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                e[i] = ((vm >> i) & 1u) ? fast_exp2(fmaf(__uint_as_float(v[i]), sl2, nm)) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) l4[i & 3] += e[i];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(e[2 * i], e[2 * i + 1]);
              w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            tmem_st16(tS + (cc >> 1), w);
          }
          // O of the earlier chunks is rescaled once its last product is complete (tensor-memory
          // accesses are warp-wide, so a warp rescales when one of its rows needs it)
          if (filled && __any_sync(0xffffffffu, alpha != 1.f)) {
            ok = k4_wait_warp(sh, &sh.o_done, g - 1, p.st);
            if (!ok) break;
            tc_fence_after();
            for (int cc = 0; cc < 128; cc += 32) {
              uint32_t v[32];
              tmem_ld32(tmem + k4ColO + lane_base + cc, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(tmem + k4ColO + lane_base + cc, v);
            }
          }
          tmem_st_wait();
          l = l * alpha + ((l4[0] + l4[1]) + (l4[2] + l4[3]));
          m = m_new;
        }
        filled = filled || nc > 0;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[st]);
      }
      if (!ok) break;
      // every S of this query is complete: the next query's Q may take its place
      if (item + gridDim.x < items) put_q(item + gridDim.x);
      ok = k4_wait_warp(sh, &sh.o_done, g - 1, p.st);
      if (!ok) break;
      tc_fence_after();
      const int t = (int)(item / S), split = (int)(item % S);
      if (active && S == 1) {
        const float M = fmaxf(m, sk);
        float f = 0.f, L = 0.f;
        if (M != -INFINITY) {
          f = m == -INFINITY ? 0.f : exp2f(m - M);
          L = l * f + (p.sink ? exp2f(sk - M) : 0.f);
        }
        const float inv = L > 0.f || L != L ? f / L : 0.f;
        const size_t row = ((size_t)t * H + h) * kHeadDim;
        for (int cc = 0; cc < 128; cc += 32) {
          uint32_t v[32];
          __syncwarp();
          if (filled) {
            tmem_ld32(tmem + k4ColO + lane_base + cc, v);
            tmem_ld_wait();
          }
          if (h < H) {
            // a row without attended columns has no O of its own
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
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
        if (h < H && p.lse) p.lse[(size_t)t * H + h] = L > 0.f || L != L ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
      } else if (active && filled) {
        // partial for attn_combine_kernel, dimension-major ([split][j][h])
        const size_t sb = (size_t)t * S + split;
        float* dst = p.part_acc + sb * kHeadDim * H + h;
        for (int cc = 0; cc < 128; cc += 32) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld32(tmem + k4ColO + lane_base + cc, v);
          tmem_ld_wait();
          if (h < H) {
#pragma unroll
            for (int i = 0; i < 32; ++i) dst[(size_t)(cc + i) * H] = __uint_as_float(v[i]);
          }
        }
        if (h < H) {
          p.part_ml[sb * 2 * H + h] = m;
          p.part_ml[(sb * 2 + 1) * H + h] = l;
        }
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

// Splits of a query: whole chunks, as many as fill the SMs once; `most` bounds them by the
// workspace.
void attn_kv4_plan(int T, int64_t rows_max, int most, int sms, int* R, int* S) {
  const int64_t chunks = (rows_max + k4Chunk - 1) / k4Chunk;
  int64_t s = T < sms ? sms / T : 1;
  s = s < most ? s : most;
  s = s < chunks ? s : chunks;
  if (s < 1) s = 1;
  const int64_t per = (chunks + s - 1) / s;
  *R = (int)(per * k4Chunk);
  *S = (int)(chunks ? (chunks + per - 1) / per : 1);
  if (*R < k4Chunk) *R = k4Chunk;
}

cudaError_t launch_attn_kv4(const AttnParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = ensure_smem(attn_kv4_kernel, k4Smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.T * p.max_splits;
  e = launch_dependent(attn_kv4_kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(k4Threads), k4Smem, stream, p);
  note_launch();
  if (e != cudaSuccess || p.max_splits == 1) return e;
  return launch_attn_combine(p, stream);
}

}  // namespace cskv
