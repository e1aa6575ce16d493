// fa_cache_decode.cuh -- attention of few query rows over the 8-bit cache.
//
// The rows of a K/V head share every key and value that is read; a thread
// block takes all of them, up to 16 * kMT.
//
// Mathematics.  S = Q K^T and O += P V on the tensor cores (m16n8k16, f16 in,
// fp32 out), with an online softmax in base 2.  Nothing is lost on the way to
// f16: stored values of both kinds are f16 numbers, and a bf16 query row is
// scaled by a power of two so that its largest entry lies in [2^9, 2^10) (an
// entry 2^-34 below that is lost at most).  Over the 16 tokens of a step the
// scales ks, vs are constant, and row i's weights are kept as
//
//   P'_ij = 2^(s_ij + log2 vs_j - r_i),   O = sum_j P'_ij v8_j / l_i,   l_i = sum_j P'_ij / vs_j
//
// with r_i 2^11 below the running maximum of s + log2 vs (fa_cache_line.cuh):
// v_scale costs an addition in the exponent.  P' is rounded to f16: by 2^-11
// (the output has 2^-8 or 2^-11) down to weights 2^-25 of the row's largest, by
// 2^-36 of the largest below, "largest" in units of value, weight * v_scale.
// So a first token that holds nearly all of a row's weight, with a value near 0,
// leaves the others' sum right, and an outlier's large v_scale hides other
// blocks only past that range.  The sums are not rounded to f16.  1 / l, 1 / vs,
// exponentials, logarithms and the softcap's quotient are the special function
// unit's, 2^-22 off: a two-thousandth of what f16 weights are.
//
// Work.  A producer warp brings tiles of 32 tokens into a ring, with their
// scales (two, one for K and one for V, where few wide tiles must keep the
// memory busy); the other warps take turns at the tiles, and each keeps a
// running maximum, sum and output of its own in registers, so that no barrier
// stands between two tiles.  The ring is filled by TMA where a tile's part of a
// cache block is 4 KB and more, else by cp.async (fa_cache_attn_launch.cuh).
// Tiles are shared out evenly over the machine (fa_cache_line.cuh).
//
// Layout.  Neither product cares about the order of its summed index, nor
// about the order of the columns it produces: lane (g, t) takes the bytes
// 32t .. 32t+31 of key g (QK) and 16 bytes of one value row (PV) as they lie
// in memory, so that all shared-memory reads are 16 bytes wide and, with the
// 128-byte swizzle, free of conflicts; the matching permutation is applied to
// Q once, and undone by where O is written.
//
// Bound: memory; 2 * D bytes a token and K/V head, read once.  32 sequences of
// up to 8192 tokens, H 32/8, D 128, e4m3: 66.7 us, 5.4 TB/s; one of 131072: 52.7
// us, 5.1 TB/s; its start, the join and the second launch among them.  Tried and
// slower: loads straight to registers (79.9 us on the first), a cp.async queue a
// lane (83.7 us), one block of 10 + 2 warps an SM (102 us).
#pragma once

#include "fa_cache_line.cuh"
#include "fa_cache_tree.cuh"

namespace fa {

// kTree_: the rows are the drafts of a tree (fa_cache_tree.cuh).
template <int kKind_, bool kF16_, int kD_, int kMT_, bool kTma_, bool kTree_ = false>
struct DecCfg {
  static constexpr bool kTree = kTree_;
  static constexpr int kLead = 0;
  static constexpr bool kTma = kTma_;
  static constexpr int kKind = kKind_;
  static constexpr bool kF16 = kF16_;  // type of q and o
  static constexpr int kD = kD_, kMT = kMT_;
  static constexpr int kTile = 32;  // tokens
  static constexpr int kLift = 11;  // of the weights (a reference that moves costs little here)
  // As many consumer warps as the outputs that each holds (kMT * D / 2 registers
  // a lane) leave room for, and two producers an SM: one block of 8 warps with
  // 255 registers, or two of 6 with 168.
  static constexpr bool kWide = kMT * kD > 128;
  static constexpr int kWarps = kWide ? 6 : 5, kProducers = kWide ? 2 : 1, kCtas = kWide ? 1 : 2;
  static constexpr int kThreads = 32 * (kWarps + kProducers);
  static constexpr int kCols = kD >= 128 ? kD / 128 : 1;    // 128-byte column blocks of a row
  static constexpr int kRowBytes = kD >= 128 ? 128 : 64;    // of one column block
  static constexpr int kTileBytes = kTile * kD;             // K; V alike
  static constexpr int kStageBytes = 2 * kTileBytes;
  // The ring: a whole number of stages for each warp.  Tile k takes stage k %
  // kStages and warp k % kWarps, so that a stage's tiles all belong to one
  // warp: copies land in any order, and a warp that waited for one tile of a
  // stage cannot mistake its phase for the next one's.
  static constexpr int kStages = kWide ? 196608 / kStageBytes / 6 * 6 : kD == 64 ? 20 : 10;
  static constexpr int kMinTiles = 2 * kWarps;  // of one block
  static constexpr int kRows = 16 * kMT;
  static constexpr int kKSteps = kD / 16, kNTiles = kD / 8;
  static constexpr int kQBytes = kRows * kD * 2;
  static constexpr int kRingBytes = kStages * kStageBytes;
  // The warps join their outputs 8 rows at a time in memory of its own, so that
  // the ring goes on to the next segment meanwhile; wide ones, all rows at once,
  // in the ring's.
  static constexpr int kJoinRows = kWide ? kRows : 8;
  static constexpr int kJoinBytes = kWarps * kJoinRows * kD * 4;
  static_assert((!kWide || kJoinBytes <= kRingBytes) && kStages % kWarps == 0 && kStages > kWarps && kStages <= 32,
                "ring size");
  static_assert(kMT * kD <= 256, "32 rows of 256 columns do not fit the registers");
  static constexpr int kOffJoin = kWide ? 0 : kRingBytes;
  static constexpr int kOffQ = kRingBytes + (kWide ? 0 : kJoinBytes), kOffMl = kOffQ + kQBytes, kOffMeta = kOffMl + kWarps * kRows * 8;
  static constexpr int kOffBar = kOffMeta + 64 * 32, kOffRs = kOffBar + kStages * 16;
  static constexpr int kOffTmp = kOffRs + kRows * 4;
  static constexpr int kSmem = 1024 + kOffTmp + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

// What a consumer needs beside a tile's bytes, for its two halves of 16
// tokens: ks; log2 vs and 1 / vs, less the weights' lift (0 and 0 where values
// do not count: a zero scale; 1 / vs is -1 where nothing is stored).
struct DecMeta {
  float ks[2], lv[2], rv[2];
  int blk[2];  // for the producer itself
};

// ------------------------------------------------------------------ tensor-core pieces

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes from the cache to shared memory; zeros if not `there`.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Address of 16-byte unit `u` of row `r` in a swizzled column block.
template <class C>
__device__ __forceinline__ uint32_t dec_unit(uint32_t base, int r, int u) {
  if constexpr (C::kRowBytes == 128) return base + r * 128 + ((u ^ (r & 7)) << 4);
  return base + r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

// The 32-bit words of key `r` that lane t multiplies: word kk holds the two
// element pairs of its k-step kk.
template <class C>
__device__ __forceinline__ void dec_key_words(uint32_t tile, int r, int t, uint32_t (&w)[C::kKSteps]) {
  if constexpr (C::kD == 64) {
    const uint4 v = lds128(dec_unit<C>(tile, r, t));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
#pragma unroll
    for (int c = 0; c < C::kCols; ++c) {
      const uint32_t base = tile + c * C::kTile * 128;
      const uint4 v0 = lds128(dec_unit<C>(base, r, 2 * t)), v1 = lds128(dec_unit<C>(base, r, 2 * t + 1));
      w[8 * c + 0] = v0.x, w[8 * c + 1] = v0.y, w[8 * c + 2] = v0.z, w[8 * c + 3] = v0.w;
      w[8 * c + 4] = v1.x, w[8 * c + 5] = v1.y, w[8 * c + 6] = v1.z, w[8 * c + 7] = v1.w;
    }
  }
}

// The 32-bit word, in the A operand [k-step, lane, 4] of 16 query rows, of
// row r's elements d and d + 1 (d even).
template <int kD>
__device__ __forceinline__ int dec_q_word(int r, int d) {
  const int t = kD == 64 ? d / 16 : (d & 127) / 32;
  const int kk = kD == 64 ? (d & 15) / 4 : 8 * (d / 128) + (d & 31) / 4;
  return (kk * 32 + (r & 7) * 4 + t) * 4 + ((d & 3) / 2) * 2 + (r >> 3);
}

// Output columns.  Value n of PV's column tile i is column dec_col(i, n).
template <class C>
__device__ __forceinline__ int dec_col(int i, int n) {
  if constexpr (C::kD == 64) return 8 * n + i;
  return 128 * (i >> 4) + 16 * n + (i & 15);
}

// ------------------------------------------------------------------ the kernel

// Where the warps leave column d (a multiple of 4) of their row `r` to be joined.
template <class C>
__device__ __forceinline__ float* dec_join_at(float* base, int r, int d) {
  return base + r * C::kD + (d & ~31) + ((((d >> 2) & 7) + 2 * (d >> 5) + r) & 7) * 4;
}

// A bounded wait by one thread; false once it ran out (or another did).  The
// bound is looked at before the hardware may suspend the thread: a bound of a
// cycle expires wherever there is something to wait for.
__device__ __forceinline__ bool dec_wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, const CacheAttnParams& a) {
  if (mbar_test(bar, parity)) return true;
  const long long begin = clock64_now();
  do {
    if (*abort) return false;
    if (clock64_now() - begin > a.timeout_cycles) {
      atomicOr(a.c.status, kStatusTimeout);
      *abort = 1;
      return false;
    }
  } while (!mbar_try_wait(bar, parity));
  return true;
}
// A bounded wait by a whole warp; false once it ran out (or another did).
__device__ __forceinline__ bool dec_wait(uint64_t* bar, uint32_t parity, volatile int* abort, const CacheAttnParams& a) {
  bool ok = mbar_test(bar, parity);
  if (!ok) {
    const long long begin = clock64_now();
    while (!*abort && clock64_now() - begin <= a.timeout_cycles && !(ok = mbar_try_wait(bar, parity))) {
    }
  }
  if (__all_sync(0xFFFFFFFFu, ok)) return true;
  if ((threadIdx.x & 31) == 0) {
    if (!*abort) atomicOr(a.c.status, kStatusTimeout);
    *abort = 1;
  }
  return false;
}

// The way out of a producer that has issued tiles 0 .. issued - 1: its copies
// land before the block ends (a bounded wait; older tiles than the ring holds
// have been consumed).
template <class C>
__device__ __forceinline__ void dec_drain(uint64_t* s_full, int issued) {
  if constexpr (C::kTma) {
    const long long begin = clock64_now();
    for (int k = max(0, issued - C::kStages); k < issued; ++k)
      while (!mbar_try_wait(s_full + k % C::kStages, (uint32_t)(k / C::kStages) & 1u) &&
             clock64_now() - begin < kDecDrainCycles) {
      }
  } else {
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ DecParams p) {
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  constexpr int kW = C::kWarps, kS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_q = smem + C::kOffQ;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kOffMl);        // [warp][row]: reference, sum
  DecMeta* s_meta = reinterpret_cast<DecMeta*>(smem + C::kOffMeta);  // [tile % 64]
  uint64_t* s_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* s_empty = s_full + kS;
  float* s_rs = reinterpret_cast<float*>(smem + C::kOffRs);  // [row]: 2^-(scaling of the query row)
  volatile int* s_abort = reinterpret_cast<int*>(smem + C::kOffTmp);
  volatile int* s_issued = s_abort + 1;  // [producer], where there are two
  float* s_join = reinterpret_cast<float*>(smem + C::kOffJoin);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(s_full + s, C::kProducers * (C::kTma ? 1 : 33));
      mbar_init(s_empty + s, 1);
    }
    fence_barrier_init();
    *s_abort = 0;
    if constexpr (C::kTma) {
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
  }

  // The join kernel may take its place on the machine as soon as there is room.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // This block's part of the line, and where it begins.
  DecPlace at;
  if (!dec_find<C>(p, blockIdx.x, at)) return;
  const int t0 = at.part * (int)blockIdx.x, t1 = (int)min((long long)at.total, (long long)t0 + at.part);
  __syncthreads();  // the barriers are ready
  const int sub = min(c.page, C::kTile), sub_log2 = min(c.page_log2, 5);  // a block's part of a tile
  const int subs = C::kTile >> sub_log2;                                  // parts a tile: 1 or 2
  int tile0 = 0;  // tiles of this block's earlier pieces: tile k of all uses stage k % kS

#pragma unroll 1
  for (int pos = t0; pos < t1;) {
    const int b = at.b, h = at.h;
    const DecSeq seq = at.seq;
    // the first tile of a sequence tells about its length
    if (tid == 0 && h == 0 && pos == at.seg0) (void)checked_len(c, a.lens[b]);
    const int tiles = dec_tiles<C>(p, seq, 0);
    const int2 span = dec_group_span<C>(p, seq, 0);
    const int first_tile = span.x / C::kTile + pos - at.seg0;
    const int n_tiles = min(t1, at.seg0 + tiles) - pos;
    const bool whole = n_tiles == tiles;

    if (warp >= kW) {
      // ---------------------------------------------------------- producer
      const bool keys = C::kProducers == 1 || warp == kW, values = C::kProducers == 1 || warp > kW;
      // Parts of 32 tiles' (or 16) blocks at a time: lane l looks up part l's
      // block, one batch ahead, and writes its scales where the consumers of
      // tile k find them (entry k % 64: the ring is shorter than a batch, so
      // that nobody reads the batch before the last any more).
      const int shift = subs - 1, per_batch = 32 >> shift, sub_at = lane & shift;
      int stage = tile0 % kS;
      uint32_t phase = (uint32_t)(tile0 / kS) & 1u;
      int issued = 0, next_blk = -1;
      bool ok = true;
      auto look_up = [&](int k0) {
        const int k = k0 + (lane >> shift), tok = (first_tile + k) * C::kTile + sub_at * sub;
        return k < n_tiles && tok < span.y && tok + sub > span.x
                   ? checked_block(c, c.table, c.table_stride, b, tok >> c.page_log2)
                   : -1;
      };
      next_blk = look_up(0);
      int y = (first_tile * C::kTile) & (c.page - 1);  // 0 where blocks are no longer than a tile
#pragma unroll 1
      for (int k0 = 0; k0 < n_tiles && ok; k0 += per_batch) {
        const int blk = next_blk;
        float ks = 0.0f, vs = 0.0f;
        if (blk >= 0) {
          if (keys) ks = __ldg(c.k_scale + (long long)blk * c.H + h);
          if (values) vs = __ldg(c.v_scale + (long long)blk * c.H + h);
        }
        next_blk = look_up(k0 + per_batch);
        if (k0 + (lane >> shift) < n_tiles) {
          DecMeta* meta = s_meta + ((tile0 + k0 + (lane >> shift)) & 63);
          const bool counts = vs >= 1.17549435e-38f;
          const float lv = counts ? lg2(vs) : 0.0f, rv = blk < 0 ? -1.0f : counts ? rcp_approx(vs) * dec_unlift(C::kLift) : 0.0f;
          if (keys) meta->ks[sub_at] = ks;
          if (values) meta->lv[sub_at] = lv, meta->rv[sub_at] = rv;
          if (subs == 1) {
            if (keys) meta->ks[1] = ks;
            if (values) meta->lv[1] = lv, meta->rv[1] = rv;
          }
          meta->blk[values ? 0 : 1] = blk;  // (two producers: one each)
        }
        __syncwarp();
        const int n = min(per_batch, n_tiles - k0);
        if constexpr (C::kTma) {
          // One thread, four tiles at a time: look-ups and first tries of the
          // four go together (this loop is what a tile costs the block at least).
          if (lane == 0) {
#pragma unroll 1
            for (int i = 0; i < n && ok; i += 4) {
              int from[4], at_stage[4];
              uint32_t par[4];
              bool ready[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                from[u] = s_meta[(tile0 + issued + u) & 63].blk[values ? 0 : 1];
                at_stage[u] = stage + u < kS ? stage + u : stage + u - kS;
                par[u] = stage + u < kS ? phase : phase ^ 1u;
                ready[u] = tile0 + issued + u < kS || (i + u < n && mbar_try_wait(s_empty + at_stage[u], par[u] ^ 1u));
              }
              const int m = min(4, n - i);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                if (u < m && ok) {
                  ok = ready[u] || dec_wait_one(s_empty + at_stage[u], par[u] ^ 1u, s_abort, a);
                  if (ok) {
                    uint64_t* bar = s_full + at_stage[u];
                    uint8_t* dst = smem + at_stage[u] * C::kStageBytes;
                    if (from[u] < 0) {
                      mbar_arrive(bar);
                    } else {
                      mbar_arrive_expect_tx(bar, (uint32_t)(C::kStageBytes / C::kProducers));
#pragma unroll
                      for (int col = 0; col < C::kCols; ++col) {
                        uint8_t* d = dst + col * C::kTile * C::kRowBytes;
                        if (keys) tma_load_4d(d, &tk, bar, col * 128, y, h, from[u]);
                        if (values) tma_load_4d(d + C::kTileBytes, &tv, bar, col * 128, y, h, from[u]);
                      }
                    }
                    ++issued;
                    y = (y + C::kTile) & (c.page - 1);
                  }
                }
              }
              stage += m;
              if (stage >= kS) stage -= kS, phase ^= 1u;
            }
          }
          issued = __shfl_sync(0xFFFFFFFFu, issued, 0);
          stage = __shfl_sync(0xFFFFFFFFu, stage, 0);
          phase = __shfl_sync(0xFFFFFFFFu, phase, 0);
          y = __shfl_sync(0xFFFFFFFFu, y, 0);
          ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
        } else {
          // 16-byte units, in the swizzle that a tensor map would give them; the
          // warp copies kRowsAtOnce rows at a time.
          constexpr int kUnits = C::kRowBytes / 16, kRowsAtOnce = 32 / kUnits;
          const int unit = lane % kUnits, r_lane = lane / kUnits;
#pragma unroll 1
          for (int i = 0; i < n; ++i, ++issued) {
            const int b0 = __shfl_sync(0xFFFFFFFFu, blk, i << shift);
            const int b1 = subs == 2 ? __shfl_sync(0xFFFFFFFFu, blk, 2 * i + 1) : b0;
            // a half's first row of this lane
            const uint8_t *k_from[2], *v_from[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const long long at_blk = max(half ? b1 : b0, 0), row = ((y + 16 * half) & (c.page - 1)) + r_lane;
              k_from[half] = c.k + at_blk * c.ks[0] + h * c.ks[1] + row * c.ks[2] + unit * 16;
              v_from[half] = c.v + at_blk * c.vs[0] + h * c.vs[1] + row * c.vs[2] + unit * 16;
            }
            if (tile0 + issued >= kS && !dec_wait(s_empty + stage, phase ^ 1u, s_abort, a)) {
              ok = false;
              break;
            }
            const uint32_t to = smem_u32(smem + stage * C::kStageBytes);
#pragma unroll
            for (int r0 = 0; r0 < C::kTile; r0 += kRowsAtOnce) {
              const bool there = (r0 < 16 ? b0 : b1) >= 0;
#pragma unroll
              for (int col = 0; col < C::kCols; ++col) {
                const uint32_t d = dec_unit<C>(to + col * C::kTile * C::kRowBytes, r0 + r_lane, unit);
                if (keys) copy16(d, k_from[r0 / 16] + (r0 & 15) * c.ks[2] + col * 128, there);
                if (values) copy16(d + C::kTileBytes, v_from[r0 / 16] + (r0 & 15) * c.vs[2] + col * 128, there);
              }
            }
            uint64_t* bar = s_full + stage;
            copy_arrive(bar);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);  // the scales
            y = (y + C::kTile) & (c.page - 1);
            if (++stage == kS) stage = 0, phase ^= 1u;
          }
        }
      }
      // After an expired wait the block ends here.  Of two producers, one may
      // have stopped at an earlier tile: it arrives for the tiles that only the
      // other issued (no more than a ring's length), so that both see those land.
      int end = tile0 + issued;
      if (C::kProducers == 2 && lane == 0) s_issued[warp - kW] = end;
      if (C::kWide ? __syncthreads_or(!ok) : !ok) {
        if constexpr (C::kProducers == 2 && C::kTma) {
          const int other = s_issued[kW + 1 - warp];
          if (lane == 0)
            for (int k = end; k < other; ++k) mbar_arrive(s_full + k % kS);
          end = max(end, other);
        }
        dec_drain<C>(s_full, end);
        return;
      }
    } else {
      // ---------------------------------------------------------- consumers
      // The query rows, scaled to f16 and laid out as the tensor core's operand:
      // all of this warp's on their way at once.
      constexpr int kE = C::kD / 32, kMine = (C::kRows + kW - 1) / kW;  // elements a lane; rows a warp
      uint32_t qw[kMine][kE / 2];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int row = warp + i * kW, qi = row / a.group, head = h * a.group + row % a.group;
        const bool in = row < p.rows && qi < seq.nq;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + b * a.qs[0] +
                                                              head * a.qs[1] + qi * a.qs[2]) + lane * (kE / 2);
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) qw[i][e] = in ? __ldg(q + e) : 0u;
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = warp + i * kW;
        if (r >= C::kRows) break;
        float f[kE], up = 1.0f, down = 1.0f;
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) {
          f[2 * e] = half_bits_to_f32<C::kF16>(qw[i][e]);
          f[2 * e + 1] = half_bits_to_f32<C::kF16>(qw[i][e] >> 16);
        }
        if (!C::kF16 && r < p.rows) {
          float top = 0.0f;
#pragma unroll
          for (int e = 0; e < kE; ++e) top = fmaxf(top, fabsf(f[e]));
          top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));  // (the order of bits, for floats >= 0)
          dec_row_scale(top, up, down);
        }
        if (lane == 0) s_rs[r] = down;
#pragma unroll
        for (int e = 0; e < kE; e += 2)
          reinterpret_cast<uint32_t*>(s_q)[(r >> 4) * C::kKSteps * 128 + dec_q_word<C::kD>(r & 15, lane * kE + e)] =
              pack_f16x2(f[e] * up, f[e + 1] * up);
      }
      named_bar_sync(1, 32 * kW);

      float o[C::kMT][C::kNTiles][4];
      float m[C::kMT][2], l[C::kMT][2], rs[C::kMT][2];  // m: the reference
      int hi_row[C::kMT][2], lo_row[C::kMT][2];  // the tokens that this lane's two rows see
      int lo_all = 0, hi_all = 0x7fffffff;       // ... that every row of the warp sees
      uint32_t drafts[C::kTree ? C::kMT : 1][2];  // of a tree: the drafts that they see, beside those tokens
      const int base = seq.len - seq.nq;
      uint32_t line = 0;  // of lane i: node i and the nodes above it
      const TreeOf tree = tree_of(a, b);
      if constexpr (C::kTree) line = tree_lines(lane < seq.nq ? tree_parent(tree, lane) : -1);
#pragma unroll
      for (int mt = 0; mt < C::kMT; ++mt) {
#pragma unroll
        for (int i = 0; i < C::kNTiles; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          m[mt][x] = -INFINITY;
          l[mt][x] = 0.0f;
          const int row = mt * 16 + g + 8 * x;
          rs[mt][x] = s_rs[row];
          const int i = row / a.group;
          const bool real = row < p.rows && i < seq.nq;
          int2 v = make_int2(0, 0x7fffffff);
          if constexpr (C::kTree) {
            drafts[mt][x] = __shfl_sync(0xFFFFFFFFu, line, i & 31);
            if (real) v = make_int2(tree_window(tree, base, drafts[mt][x]), base);
            else drafts[mt][x] = 0u;
          } else if (real) {
            v = dec_span(a, seq, i, i);
          }
          // a row of the tile that is no query row may see anything: nothing of it is written
          lo_row[mt][x] = v.x;
          hi_row[mt][x] = row < p.rows && !real ? 0 : v.y;
          lo_all = max(lo_all, lo_row[mt][x]);
          hi_all = min(hi_all, hi_row[mt][x]);
        }
      }
      lo_all = __reduce_max_sync(0xFFFFFFFFu, lo_all);
      hi_all = __reduce_min_sync(0xFFFFFFFFu, hi_all);
      // Scores stay raw where one positive factor a row and block brings them
      // to base 2; a softcap, or a scale that is not positive, is applied first.
      const bool raw = a.cap_out == 0.0f && a.scale_log2 > 0.0f;

      const int k_first = (warp + kW - tile0 % kW) % kW;  // this warp's first tile of the piece
      int stage = (tile0 + k_first) % kS;
      uint32_t phase = (uint32_t)((tile0 + k_first) / kS) & 1u;
      bool dead = false;
      for (int k = k_first; k < n_tiles; k += kW) {
        if (!dec_wait(s_full + stage, phase, s_abort, a)) {
          dead = true;
          break;
        }
        const uint32_t tile_k = smem_u32(smem + stage * C::kStageBytes), tile_v = tile_k + C::kTileBytes;
        const int tok0 = (first_tile + k) * C::kTile;
        const DecMeta* meta_at = s_meta + ((tile0 + k) & 63);
        const float4 meta = *reinterpret_cast<const float4*>(meta_at);  // ks, ks, log2 vs, log2 vs
        const float2 rv = *reinterpret_cast<const float2*>(meta_at->rv);
        const bool full = rv.x >= 0.0f && rv.y >= 0.0f && lo_all <= tok0 && tok0 + C::kTile <= hi_all;

        // S = Q K^T: 4 column tiles of 8 tokens
        float sc[C::kMT][4][4];
#pragma unroll
        for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[mt][j][0] = sc[mt][j][1] = sc[mt][j][2] = sc[mt][j][3] = 0.0f;
#pragma unroll
        for (int jj = 0; jj < 4; jj += 2) {
          uint32_t w0[C::kKSteps], w1[C::kKSteps];
          dec_key_words<C>(tile_k, jj * 8 + g, t, w0);
          dec_key_words<C>(tile_k, jj * 8 + 8 + g, t, w1);
#pragma unroll
          for (int kk = 0; kk < C::kKSteps; ++kk) {
            uint32_t x0, x1, y0, y1;
            to_f16x4<C::kKind>(w0[kk], x0, x1);
            to_f16x4<C::kKind>(w1[kk], y0, y1);
#pragma unroll
            for (int mt = 0; mt < C::kMT; ++mt) {
              const uint4 q = lds128(smem_u32(s_q) + (uint32_t)(((mt * C::kKSteps + kk) * 32 + lane) * 16));
              const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
              mma_f16(sc[mt][jj], qa, x0, x1);
              mma_f16(sc[mt][jj + 1], qa, y0, y1);
            }
          }
        }

        // Masks, and the running maximum of s + log2 vs in base 2.
        float fa[C::kMT][2][2];  // [row][half]: score to base 2
        float mx[C::kMT][2];
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < C::kMT; ++mt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // (not 0, so that a hidden score stays -inf; stored values times a zero scale are as good as 0)
            fa[mt][x][0] = fmaxf(meta.x * rs[mt][x] * a.scale_log2, 1e-37f);
            fa[mt][x][1] = fmaxf(meta.y * rs[mt][x] * a.scale_log2, 1e-37f);
          }
          if (!raw) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float v = sc[mt][j][e] * (j < 2 ? meta.x : meta.y) * rs[mt][e >> 1];
                // cap * tanh(x) = cap * (1 - 2 / (2^(2 x log2 e) + 1))
                sc[mt][j][e] = a.cap_out > 0.0f
                                   ? fmaf(-2.0f * a.cap_out, rcp_approx(ex2(v * a.cap_in * 2.8853900817779268f) + 1.0f), a.cap_out)
                                   : v * a.scale_log2;
              }
            fa[mt][0][0] = fa[mt][0][1] = fa[mt][1][0] = fa[mt][1][1] = 1.0f;
          }
          if (!full) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = tok0 + j * 8 + 2 * t + (e & 1), x = e >> 1;
                bool hidden = tok < lo_row[mt][x] || tok >= hi_row[mt][x];
                if constexpr (C::kTree) hidden = hidden && !tree_bit(drafts[mt][x], tok - base);
                if (hidden || (j < 2 ? rv.x : rv.y) < 0.0f) sc[mt][j][e] = -INFINITY;
              }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float va = fmaxf(fmax3(sc[mt][0][2 * x], sc[mt][0][2 * x + 1], sc[mt][1][2 * x]), sc[mt][1][2 * x + 1]);
            const float vb = fmaxf(fmax3(sc[mt][2][2 * x], sc[mt][2][2 * x + 1], sc[mt][3][2 * x]), sc[mt][3][2 * x + 1]);
            float v = fmaxf(fmaf(va, fa[mt][x][0], meta.z), fmaf(vb, fa[mt][x][1], meta.w));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
            mx[mt][x] = v;
            grow = grow || dec_grown(v, m[mt][x]);
          }
        }
        if (p.scores) {  // for cache_finish_kernel: 8 neighbouring tokens of a row a quad
          float* out = p.scores + (((long long)b * c.H + h) * ((c.M * (c.page >> 4) + 1) / 2) + (tok0 >> 5)) * p.rows * 32 + 2 * t;
#pragma unroll
          for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = mt * 16 + g + 8 * x;
              if (r < p.rows) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  __stcg(reinterpret_cast<float2*>(out + r * 32 + 8 * j),
                         make_float2(sc[mt][j][2 * x] * fa[mt][x][j >> 1], sc[mt][j][2 * x + 1] * fa[mt][x][j >> 1]));
              }
            }
        }
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
          for (int mt = 0; mt < C::kMT; ++mt) {
            float al[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float m2 = fmaxf(m[mt][x], dec_reference<C>(mx[mt][x]));
              al[x] = m2 == -INFINITY ? 1.0f : ex2(m[mt][x] - m2);
              l[mt][x] *= al[x];
              m[mt][x] = m2;
            }
#pragma unroll
            for (int i = 0; i < C::kNTiles; ++i) {
              fmul2(o[mt][i][0], o[mt][i][1], o[mt][i][0], o[mt][i][1], al[0], al[0]);
              fmul2(o[mt][i][2], o[mt][i][3], o[mt][i][2], o[mt][i][3], al[1], al[1]);
            }
          }
        }
        // Half by half (16 tokens, inside one cache block): P' and its sum.
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pa[C::kMT][4];  // P' as the A operand
          const float lv = half ? meta.w : meta.z, rv_half = half ? rv.y : rv.x, by = rv_half > 0.0f ? rv_half : dec_unlift(C::kLift);
#pragma unroll
          for (int mt = 0; mt < C::kMT; ++mt) {
            const float m0 = lv - (m[mt][0] == -INFINITY ? 0.0f : m[mt][0]);
            const float m1 = lv - (m[mt][1] == -INFINITY ? 0.0f : m[mt][1]);
            const float f0 = fa[mt][0][half], f1 = fa[mt][1][half];
            float pv[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const float* x = sc[mt][2 * half + jj];
              ffma2(pv[jj][0], pv[jj][1], x[0], x[1], f0, f0, m0, m0);
              ffma2(pv[jj][2], pv[jj][3], x[2], x[3], f1, f1, m1, m1);
#pragma unroll
              for (int e = 0; e < 4; ++e) pv[jj][e] = ex2(pv[jj][e]);
            }
            l[mt][0] = fmaf((pv[0][0] + pv[0][1]) + (pv[1][0] + pv[1][1]), by, l[mt][0]);
            l[mt][1] = fmaf((pv[0][2] + pv[0][3]) + (pv[1][2] + pv[1][3]), by, l[mt][1]);
            pa[mt][0] = pack_f16x2(pv[0][0], pv[0][1]);
            pa[mt][1] = pack_f16x2(pv[0][2], pv[0][3]);
            pa[mt][2] = pack_f16x2(pv[1][0], pv[1][1]);
            pa[mt][3] = pack_f16x2(pv[1][2], pv[1][3]);
            if (rv_half == 0.0f) pa[mt][0] = pa[mt][1] = pa[mt][2] = pa[mt][3] = 0u;
          }
          // O += P V over these 16 tokens: lane t takes tokens 2t, 2t+1, 2t+8, 2t+9
          const int row = half * 16 + 2 * t;
          constexpr int kWords = C::kD == 64 ? 2 : 4;
#pragma unroll
          for (int col = 0; col < C::kCols; ++col) {
            const uint32_t base = tile_v + col * C::kTile * C::kRowBytes;
            uint32_t v[4][kWords];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = row + (e & 1) + 8 * (e >> 1);
              if constexpr (C::kD == 64) {
                const uint2 x = lds64(dec_unit<C>(base, r, g >> 1) + (g & 1) * 8);
                v[e][0] = x.x, v[e][1] = x.y;
              } else {
                const uint4 x = lds128(dec_unit<C>(base, r, g));
                v[e][0] = x.x, v[e][1] = x.y, v[e][2] = x.z, v[e][3] = x.w;
              }
            }
            if (!full) {  // bytes that no row may see could be NaN
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = tok0 + row + (e & 1) + 8 * (e >> 1);
                if (tok < span.x || tok >= span.y || rv_half < 0.0f) {
#pragma unroll
                  for (int w = 0; w < kWords; ++w) v[e][w] = 0u;
                }
              }
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                uint32_t a0, a1, b0, b1;
                to_f16x4<C::kKind>(__byte_perm(v[0][w], v[1][w], hh ? 0x7362 : 0x5140), a0, a1);
                to_f16x4<C::kKind>(__byte_perm(v[2][w], v[3][w], hh ? 0x7362 : 0x5140), b0, b1);
#pragma unroll
                for (int mt = 0; mt < C::kMT; ++mt) {
                  mma_f16(o[mt][4 * kWords * col + 4 * w + 2 * hh], pa[mt], a0, b0);
                  mma_f16(o[mt][4 * kWords * col + 4 * w + 2 * hh + 1], pa[mt], a1, b1);
                }
              }
            }
          }
        }
        __syncwarp();  // every lane has read the stage: it may be filled again
        if (lane == 0) mbar_arrive(s_empty + stage);
        stage += kW;
        if (stage >= kS) stage -= kS, phase ^= 1u;
      }

      // Join the warps: O at the block's common reference.
#pragma unroll
      for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 1);
          l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 2);
          if (t == 0) s_ml[warp * C::kRows + mt * 16 + g + 8 * x] = make_float2(m[mt][x], l[mt][x]);
        }
      // The maxima are there (and every warp is done with the ring).
      if (C::kWide ? __syncthreads_or(dead) : named_bar_or(1, 32 * kW, dead)) return;
      const int slot = 2 * blockIdx.x + (pos > at.seg0 ? 0 : 1);
#pragma unroll
      for (int pass = 0; pass < C::kRows / C::kJoinRows; ++pass) {
        if (pass * C::kJoinRows >= p.rows) break;
        if (pass > 0) named_bar_sync(1, 32 * kW);  // the rows before have been read
#pragma unroll
        for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!C::kWide && 2 * mt + x != pass) continue;
            const int r = mt * 16 + g + 8 * x;
            float top = -INFINITY;
            for (int w = 0; w < kW; ++w) top = fmaxf(top, s_ml[w * C::kRows + r].x);
            const float f = m[mt][x] == -INFINITY ? 0.0f : ex2(m[mt][x] - top);
            if (t == 0) s_ml[warp * C::kRows + r].y = l[mt][x] * f;
            // four columns at a time, units rotated so that no two lanes meet in a bank
#pragma unroll
            for (int q = 0; q < C::kNTiles / 2; ++q) {  // 2 * D / 8 values a row: columns of n = 2t, then 2t + 1
              const int i = (q * 4) % C::kNTiles, e = 2 * x + (q * 4) / C::kNTiles;
              const int d = dec_col<C>(i, 2 * t + (e & 1));
              *reinterpret_cast<float4*>(dec_join_at<C>(s_join, warp * C::kJoinRows + r - pass * C::kJoinRows, d)) =
                  make_float4(o[mt][i][e] * f, o[mt][i + 1][e] * f, o[mt][i + 2][e] * f, o[mt][i + 3][e] * f);
            }
          }
        named_bar_sync(1, 32 * kW);
#pragma unroll 1
        for (int v = tid; v < min(p.rows - pass * C::kJoinRows, C::kJoinRows) * (C::kD / 4); v += 32 * kW) {
          const int rj = v / (C::kD / 4), r = pass * C::kJoinRows + rj, d = (v % (C::kD / 4)) * 4;
          float top = -INFINITY, sum = 0.0f;
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const float2 ml = s_ml[w * C::kRows + r];
            const float4 y = *reinterpret_cast<const float4*>(dec_join_at<C>(s_join, w * C::kJoinRows + rj, d));
            top = fmaxf(top, ml.x);
            sum += ml.y;
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
          }
          if (whole) {
            dec_write<C>(a, b, h, r, d, x, top, sum);
          } else {
            *reinterpret_cast<float4*>(p.part_o + ((long long)slot * C::kRows + r) * C::kD + d) = x;
            if (d == 0) p.part_ml[(long long)slot * C::kRows + r] = make_float2(top, sum);
          }
        }
      }
      if constexpr (C::kWide)
        fence_proxy_async_smem();  // what was written into the ring's memory goes before the next copies into it
      else
        named_bar_sync(1, 32 * kW);  // the maxima and the query rows are free again
    }
    if constexpr (C::kWide) __syncthreads();  // the ring's memory and the maxima are free again
    tile0 += n_tiles;
    pos += n_tiles;
    dec_next(p, at, tiles);
  }
  // Consumers whose wait expired have left without looking at the last copies.
  // (Wide heads' producers leave with the consumers, above.)
  if (!C::kWide && warp >= kW) dec_drain<C>(s_full, tile0);
}

}  // namespace fa
