// fa_cache_prompt.cuh -- attention of many query rows over the 8-bit cache.
//
// The same operation as fa_cache_decode.cuh, for rows enough to fill the
// tensor core's 128-row tiles (a piece of a prompt, or many drafts): tcgen05
// MMAs with accumulators in tensor memory, two row tiles a thread block taking
// turns at the tensor core (one where D = 256).
//
// Mathematics.  All products in f16 with fp32 accumulation: a stored value is
// an f16 number, a bf16 query row is scaled by a power of two.  With k_scale
// and v_scale constant over groups of 16 or 64 tokens (ks, vs), row i's weights are kept as
//
//   P'_ij = 2^(s_ij + log2 vs_j - r_i),   O = sum_j P'_ij v8_j / l_i,   l_i = sum_j P'_ij / vs_j
//
// with r_i 2^7 below the running maximum of s + log2 vs (fa_cache_line.cuh):
// one FMA and one exponential a score, and the scales cost an operation per
// group.  P' is rounded to f16, by 2^-11 down to 2^-21 of the row's largest
// (weight * v_scale) and by 2^-32 of the largest below (fa_cache_decode.cuh);
// the sums are not.
//
// Roles.  Warps 0 and 1 issue MMAs, one per row tile; the converter warps load
// stored bytes straight from global memory into registers, half a block of 128
// keys ahead, widen them to f16 and write them in the tensor core's
// 128-byte-swizzled layout; one softmax warpgroup per row tile owns a row a
// thread, loads and scales its query rows itself, and writes its output.
//
// Order.  A row tile's scores go to two buffers in turn (64 keys each where two
// tiles share the tensor memory), and the next buffer's scores are issued
// before this one's P V, so that they are ready when the softmax is done with
// this one.  (With one buffer of 128 keys a tile, the tiles taking turns, each
// block's scores, softmax and P V ran one after the other: 908 us against 865 on
// the workload below.)  The softmax weighs a row against the maximum so far while
// it finds the new one, and does it again where that has grown by more than 2^7.
//
// Bound: the softmax warps' chains of dependent instructions, two warps a
// scheduler, then the tensor cores (58% busy) and shared memory (the widened
// tiles are written once for 256 rows).  2 x 2048 rows at the end of 16384
// tokens, H 32/8, D 128, e4m3: 795 us, 1297 TFLOP/s.  Leaving out, in a copy,
// the exponentials, the maximum or half the MMAs gained 10%, 6% and 4%.
#pragma once

#include "fa_cache_line.cuh"

namespace fa {

// kGroup_: tokens that surely share a cache block, and so a scale: 16, or 64
// where blocks have 64 tokens and more (a quarter of the operations by group.
// 1024 rows, 8192 tokens in blocks of 64, H 32/8: D 64 115.0 us with 64 and 121.2
// with 16, D 128 144.8 and 157.7, D 256 350 and 381).
// kRaw_: no softcap and a positive scale, so that a score's FMA scales it too
// (with one, and 16: 198, 238 and 418 us).
template <int kKind_, bool kF16_, int kD_, int kGroup_, bool kRaw_>
struct PromptCfg {
  static constexpr bool kRaw = kRaw_;  // scores need no more than a positive factor
  static constexpr int kGroup = kGroup_, kGroups = 128 / kGroup;  // groups a block of keys
  static constexpr int kKind = kKind_;
  static constexpr bool kF16 = kF16_;
  static constexpr int kD = kD_;
  static constexpr int kTiles = kD <= 128 ? 2 : 1;   // 128-row tiles a block
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kTile = 128;                  // keys a block of the line
  static constexpr int kMinTiles = 4;
  // Of the weights: half of what f16 has room for, since a row whose maximum
  // leaves the other half does its softmax twice (prompt piece: 802 us with 7,
  // 815 with 10, 821 with 11).
  static constexpr int kLift = 7;
  static constexpr int kStages = kD == 64 ? 3 : kD == 128 ? 2 : 1;  // of K; of V alike
  static constexpr int kIssuers = kTiles;
  // Keys a score buffer; a row tile has two, so that the next scores are being
  // computed while a softmax runs.
  static constexpr int kKeys = kTiles == 2 ? 64 : 128, kParts = 128 / kKeys;
  static constexpr int kConvWarps = kTiles == 2 ? 4 : 8;
  static constexpr int kThreads = 128 + 32 * kConvWarps + 128 * kTiles;  // 512
  static constexpr int kQBytes = 128 * kD * 2;       // one row tile
  static constexpr int kKvBytes = 128 * kD * 2;
  static constexpr int kOffK = kTiles * kQBytes, kOffV = kOffK + kStages * kKvBytes;
  static constexpr int kOffMeta = kOffV + kStages * kKvBytes, kOffCtl = kOffMeta + 4 * kGroups * 16;
  static constexpr int kSmem = 1024 + kOffCtl + 512;
  static constexpr int kColO = 256;                  // S: two buffers of kKeys columns a tile; P over S
  // Registers: 512 threads x 128 at launch; the softmax warps, which hold a
  // row of scores each, take the others'.
  static constexpr int kRegsCtrl = kTiles == 2 ? 56 : 64, kRegsConv = 104, kRegsSoft = kTiles == 2 ? 176 : 232;
  static_assert(kRegsCtrl < 128 && kRegsConv < 128 && kRegsSoft > 128, "which warps give, which take");
  static_assert(128 * kRegsCtrl + 32 * kConvWarps * kRegsConv + 128 * kTiles * kRegsSoft <= 512 * 128,
                "register split exceeds the launch allocation");
  static_assert(kThreads == 512 && kSmem <= 232448, "thread block shape");
};

struct PromptCtl {
  uint64_t q_full[2];              // 4 softmax warps: query tile written
  uint64_t k_full[3], k_empty[3];  // converters / MMAs (one arrival an issuer)
  uint64_t v_full[3], v_empty[3];
  uint64_t s_full[2][2];           // [tile][buffer]: S computed
  uint64_t p_ready[2];             // softmax wrote P (and rescaled O)
  uint64_t o_ready[2];             // each PV done
  uint64_t drain[2];
  int n[2][2];                     // [tile][piece & 1]: blocks of a piece (0: no more), beside q_full
  uint32_t tmem;
  int abort;
};

// kStrict: the bound is looked at before the hardware may suspend the thread
// at all, as in dec_wait_one (everywhere, that made the prompt piece 0.7% slower);
// else before it may do so twice.
template <bool kStrict = false>
__device__ __forceinline__ bool prompt_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            const CacheAttnParams& a) {
  if (kStrict ? mbar_test(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long begin = clock64_now();
  do {
    if (*abort) return false;
    if (clock64_now() - begin > a.timeout_cycles) {
      *abort = 1;
      atomicOr(a.c.status, kStatusTimeout);
      return false;
    }
  } while (!mbar_try_wait(bar, parity));
  return true;
}
template <bool kStrict = false>
__device__ __forceinline__ bool prompt_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                 const CacheAttnParams& a) {
  return __all_sync(0xFFFFFFFFu, prompt_wait<kStrict>(bar, parity, abort, a));
}

// 16 stored bytes -> 16 f16.
template <int kKind>
__device__ __forceinline__ void widen16(const uint4& w, uint4& lo, uint4& hi) {
  to_f16x4<kKind>(w.x, lo.x, lo.y);
  to_f16x4<kKind>(w.y, lo.z, lo.w);
  to_f16x4<kKind>(w.z, hi.x, hi.y);
  to_f16x4<kKind>(w.w, hi.z, hi.w);
}

// A row's scores to base 2 where one positive factor cannot do it.
template <class C>
__device__ __forceinline__ void prompt_scale(uint32_t (&x)[C::kKeys], const CacheAttnParams& a, const float4* meta, float rs) {
#pragma unroll
  for (int g = 0; g < C::kKeys / C::kGroup; ++g) {
    const float ks = meta[g].x * rs, ci = ks * a.cap_in * 2.8853900817779268f;
#pragma unroll
    for (int k = C::kGroup * g; k < C::kGroup * (g + 1); ++k) {
      const float v = __uint_as_float(x[k]);
      // cap * tanh(y) = cap * (1 - 2 / (2^(2 y log2 e) + 1))
      x[k] = __float_as_uint(a.cap_out > 0.0f ? fmaf(-2.0f * a.cap_out, rcp_approx(ex2(v * ci) + 1.0f), a.cap_out)
                                              : v * (ks * a.scale_log2));
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) cache_prompt_kernel(const __grid_constant__ DecParams p) {
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float4* s_meta = reinterpret_cast<float4*>(smem + C::kOffMeta);  // [block % 4][group]: ks, log2 vs, 1 / vs less the lift, there
  PromptCtl* ctl = reinterpret_cast<PromptCtl*>(smem + C::kOffCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecPlace at;
  if (!dec_find<C>(p, blockIdx.x, at)) return;  // the whole block: nothing is set up yet
  const int t0 = at.part * (int)blockIdx.x, t1 = (int)min((long long)at.total, (long long)t0 + at.part);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 4);
      mbar_init(&ctl->s_full[i][0], 1);
      mbar_init(&ctl->s_full[i][1], 1);
      mbar_init(&ctl->p_ready[i], 4);
      mbar_init(&ctl->o_ready[i], 1);
      mbar_init(&ctl->drain[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl->k_full[i], C::kConvWarps);
      mbar_init(&ctl->v_full[i], C::kConvWarps);
      mbar_init(&ctl->k_empty[i], C::kIssuers);
      mbar_init(&ctl->v_empty[i], C::kIssuers);
    }
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  volatile int* abort = &ctl->abort;

  if (warp < 4) {
    // ============================================================ control
    regs_dec<C::kRegsCtrl>();
    if (warp < C::kIssuers) {
      const int t = warp;  // row tile
      constexpr uint32_t idS = make_idesc_fmt(kFmtF16, 128, C::kKeys, false, false);
      constexpr uint32_t idPV = make_idesc_fmt(kFmtF16, 128, C::kD, false, true);
      const uint64_t dQ = make_sdesc_sw128(smem_u32(smem + t * C::kQBytes), 16, 1024);
      const uint64_t dK = make_sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV = make_sdesc_sw128(smem_u32(smem + C::kOffV), 128 * 128, 1024);
      const uint32_t lead = elect_lead();
      auto wait = [&](uint64_t* bar, uint32_t parity) { return prompt_warp_wait(bar, parity, abort, a); };
      // Scores (part of the block in `stage`) into buffer `buf`.
      auto issue_S = [&](int buf, int stage, int part) {
        const uint64_t k0 = dK + ((stage * C::kKvBytes + part * (C::kKeys * 128)) >> 4);
        const uint32_t dst = tmem + t * 128 + buf * C::kKeys;
#pragma unroll
        for (int kk = 0; kk < C::kD / 16; ++kk) {
          const uint32_t off = (kk / 4) * ((128 * 128) >> 4) + (kk % 4) * 2;
          mma_f16_ss_by(lead, dst, dQ + off, k0 + off, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit_by(lead, &ctl->s_full[t][buf]);
        if (part == C::kParts - 1) mma_commit_by(lead, &ctl->k_empty[stage]);
      };
      auto issue_PV = [&](int buf, int stage, int part, bool first) {
        const uint64_t v0 = dV + ((stage * C::kKvBytes + part * (C::kKeys * 128)) >> 4);
        const uint32_t src = tmem + t * 128 + buf * C::kKeys, dst = tmem + C::kColO + t * C::kD;
#pragma unroll
        for (int kk = 0; kk < C::kKeys / 16; ++kk)
          mma_f16_ts_by(lead, dst, src + kk * 8, v0 + ((kk * 16 * 128) >> 4), idPV, first && kk == 0 ? 0u : 1u);
        mma_commit_by(lead, &ctl->o_ready[t]);
        if (part == C::kParts - 1) mma_commit_by(lead, &ctl->v_empty[stage]);
      };
      int nth = 0, stage = 0;  // score buffers filled, and the block's stage
      uint32_t par = 0;        // parity of the stage's use
      bool ok = true;
#pragma unroll 1
      for (int pieces = 0; ok; ++pieces) {
        ok = prompt_warp_wait<true>(&ctl->q_full[t], pieces & 1, abort, a);  // (query rows take a while to come)
        if (!ok) break;
        const int n = ctl->n[t][pieces & 1];
        if (n == 0) break;
        ok = wait(&ctl->k_full[stage], par);
        if (!ok) break;
        tc_fence_after();
        issue_S(nth & 1, stage, 0);
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int next = stage + 1 == C::kStages ? 0 : stage + 1;
          const uint32_t next_par = par ^ (next == 0 ? 1u : 0u);
#pragma unroll
          for (int part = 0; part < C::kParts; ++part) {
            // the next scores go before this PV
            if (part + 1 < C::kParts) {
              issue_S((nth + 1) & 1, stage, part + 1);
            } else if (j + 1 < n) {
              ok = wait(&ctl->k_full[next], next_par);
              if (!ok) break;
              tc_fence_after();
              issue_S((nth + 1) & 1, next, 0);
            }
            ok = (part > 0 || wait(&ctl->v_full[stage], par)) && wait(&ctl->p_ready[t], (uint32_t)nth & 1u);
            if (!ok) break;
            tc_fence_after();
            issue_PV(nth & 1, stage, part, j == 0 && part == 0);
            ++nth;
          }
          stage = next;
          par = next_par;
        }
      }
      // Every MMA issued here has completed before the block lets go of its
      // memory (after an expired wait too; bounded).
      mma_commit_by(lead, &ctl->drain[t]);
      if (lead) {
        const long long begin = clock64_now();
        while (!mbar_try_wait(&ctl->drain[t], 0) && clock64_now() - begin < kDecDrainCycles) {
        }
      }
      __syncwarp();
    }
  } else if (warp < 4 + C::kConvWarps) {
    // ============================================================ converters
    regs_dec<C::kRegsConv>();
    const int cw = warp - 4;
    constexpr int kUnits = C::kD / 16;                  // 16-byte units a key
    constexpr int kPer = 128 * kUnits / (32 * C::kConvWarps);  // units a thread and tile: 4 (D = 64) or 8
    // Lane bits 0-1: unit, 2: key, then units, then keys: eight neighbours
    // write eight different 16-byte columns of the swizzled rows.
    constexpr int kHigh = kUnits / 4;                   // 1, 2 or 4
    const int unit = (lane & 3) + 4 * ((lane >> 3) % kHigh);
    const int key_in = ((lane >> 2) & 1) + 2 * ((lane >> 3) / kHigh);  // of the warp's keys
    constexpr int kKeysWarp = 32 / kUnits;              // keys a warp takes at once: 8, 4, 2
    constexpr int kKeysStep = kKeysWarp * C::kConvWarps;  // 32 (D = 64) or 16
    const int key0 = cw * kKeysWarp + key_in;
    const uint32_t col = (uint32_t)(unit / 4) * (128 * 128);
    int nth = 0, stage = 0;  // blocks done; the next one's stage, and the parity of its use
    uint32_t par = 0;
    bool ok = true;
#pragma unroll 1
    for (int pos = t0; pos < t1 && ok;) {
      if (cw == 0 && lane == 0 && at.h == 0 && at.rg == 0 && pos == at.seg0) (void)checked_len(c, a.lens[at.b]);
      const int tiles = dec_tiles<C>(p, at.seq, at.rg), n = min(t1, at.seg0 + tiles) - pos;
      const int2 span = dec_group_span<C>(p, at.seq, at.rg);
      const int first = span.x / 128 + pos - at.seg0;
      const int b = at.b, h = at.h;
      // A batch of blocks at a time, and one batch ahead: lane kGroups * q + g
      // looks up group g of the batch's block q (its cache block), then the
      // scales.
      constexpr int kG = C::kGroups, kBatch = 32 / kG;
      int blk = -1, next_blk;
      float4 mine;           // the group's scales, as the softmax reads them
      uint32_t there, none;  // bit by lane: a block is there; its values' scale is 0
      auto look_up = [&](int j0) {
        const int j = j0 + lane / kG, tok = (first + j) * 128 + C::kGroup * (lane % kG);
        return j < n && tok < span.y && tok + C::kGroup > span.x
                   ? checked_block(c, c.table, c.table_stride, b, tok >> c.page_log2)
                   : -1;
      };
      next_blk = look_up(0);
      auto turn_over = [&](int j0) {  // the batch of blocks j0 .. becomes the one in the lanes
        blk = next_blk;
        float ks = 0.0f, vs = 0.0f;
        if (blk >= 0) {
          ks = __ldg(c.k_scale + (long long)blk * c.H + h);
          vs = __ldg(c.v_scale + (long long)blk * c.H + h);
        }
        // (values of a zero scale are stored zeros for all that counts: they are
        // cleared below, and count with the scale 1)
        const bool zero = !(vs >= 1.17549435e-38f);
        mine = make_float4(ks, zero ? 0.0f : lg2(vs), dec_unlift(C::kLift) * (zero ? 1.0f : 1.0f / vs), blk >= 0 ? 1.0f : 0.0f);
        there = __ballot_sync(0xFFFFFFFFu, blk >= 0);
        none = __ballot_sync(0xFFFFFFFFu, zero);
        next_blk = look_up(j0 + kBatch);
      };
      auto of_block = [&](uint32_t bits, int j) { return (bits >> (kG * (j % kBatch))) & ((1u << kG) - 1u); };
      // One set of registers, always on its way: as soon as K_j is widened and
      // stored, the registers take V_j, and then K_{j+1}, so that every load has
      // half a block's time to arrive.
      uint4 x[kPer];
      auto load = [&](int j, const uint8_t* pool, const long long* st) {
        const long long step = kKeysStep * st[2];
        const int tok0 = (first + j) * 128;
        if (C::kGroup == 64 && of_block(there, j) == (1u << kG) - 1u && tok0 >= span.x && tok0 + 128 <= span.y) {
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const uint8_t* from = pool + __shfl_sync(0xFFFFFFFFu, blk, (j % kBatch) * kG + g) * st[0] +
                                  (key0 + ((g * C::kGroup) & (c.page - 1))) * st[2];
#pragma unroll
            for (int i = g * (kPer / kG); i < (g + 1) * (kPer / kG); ++i, from += step)
              x[i] = __ldg(reinterpret_cast<const uint4*>(from));
          }
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int key = key0 + i * kKeysStep, tok = tok0 + key;
            const int at_blk = __shfl_sync(0xFFFFFFFFu, blk, (j % kBatch) * kG + key / C::kGroup);
            x[i] = make_uint4(0, 0, 0, 0);  // where nobody sees them or nothing is stored
            if (at_blk >= 0 && tok >= span.x && tok < span.y)
              x[i] = __ldg(reinterpret_cast<const uint4*>(pool + at_blk * st[0] + (key & (c.page - 1)) * st[2]));
          }
        }
      };
      auto store = [&](int i, uint8_t* tile) {
        const int key = key0 + i * kKeysStep;
        uint4 lo, hi;
        widen16<C::kKind>(x[i], lo, hi);
        uint8_t* row = tile + col + key * 128;
        const int u = (unit % 4) * 2;
        *reinterpret_cast<uint4*>(row + ((u ^ (key & 7)) << 4)) = lo;
        *reinterpret_cast<uint4*>(row + (((u + 1) ^ (key & 7)) << 4)) = hi;
      };
      const uint8_t* const k_pool = c.k + h * c.ks[1] + unit * 16;
      const uint8_t* const v_pool = c.v + h * c.vs[1] + unit * 16;
      turn_over(0);
      load(0, k_pool, c.ks);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (nth >= C::kStages && !(ok = prompt_warp_wait(&ctl->k_empty[stage], par ^ 1u, abort, a))) break;
        if (cw == 0 && lane / kG == j % kBatch) s_meta[(nth & 3) * kG + lane % kG] = mine;
        const uint32_t zero = of_block(none, j);
        uint8_t* tile = smem + C::kOffK + stage * C::kKvBytes;
#pragma unroll
        for (int i = 0; i < kPer; ++i) store(i, tile);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->k_full[stage]);
        load(j, v_pool, c.vs);
        if (j % kBatch == kBatch - 1) turn_over(j + 1);
        if (nth >= C::kStages && !(ok = prompt_warp_wait(&ctl->v_empty[stage], par ^ 1u, abort, a))) break;
        tile = smem + C::kOffV + stage * C::kKvBytes;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if ((zero >> ((key0 + i * kKeysStep) / C::kGroup)) & 1u) x[i] = make_uint4(0, 0, 0, 0);
          store(i, tile);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->v_full[stage]);
        if (j + 1 < n) load(j + 1, k_pool, c.ks);
        ++nth;
        if (++stage == C::kStages) stage = 0, par ^= 1u;
      }
      pos += n;
      dec_next(p, at, tiles);
    }
  } else {
    // ============================================================ softmax
    regs_inc<C::kRegsSoft>();
    const int t = C::kTiles == 2 ? (warp - 8) >> 2 : 0;
    const int tl = tid - (512 - 128 * C::kTiles) - 128 * t;  // row of the tile = TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::kColO + t * C::kD;
    uint8_t* q_tile = smem + t * C::kQBytes;
    constexpr int kGroups = C::kKeys / C::kGroup;  // groups a score buffer
    int nth = 0, pieces = 0;  // score buffers and pieces before this one
    bool ok = true;
#pragma unroll 1
    for (int pos = t0; pos < t1 && ok; ++pieces) {
      const int tiles = dec_tiles<C>(p, at.seq, at.rg), n = min(t1, at.seg0 + tiles) - pos;
      const int2 span = dec_group_span<C>(p, at.seq, at.rg);
      const int first = span.x / 128 + pos - at.seg0;
      const bool whole = n == tiles, head_cut = pos > at.seg0;
      const int row = at.rg * C::kRows + t * 128 + tl, i = row / a.group, head = at.h * a.group + row % a.group;
      const bool real = row < p.rows;
      const int2 see = real ? dec_span(a, at.seq, i, i) : make_int2(0, 0);
      // The warp's query rows, kLanes lanes a row, all loads under way at once:
      // the row's largest entry, then its f16 form.  (S of the piece before is
      // done: the tile may be written.)
      float rs = 1.0f;
      {
        constexpr int kLanes = C::kD / 8, kAtOnce = 32 / kLanes;  // rows a load
        const uint16_t* mine = see.x < see.y
                                   ? static_cast<const uint16_t*>(a.q) + at.b * a.qs[0] + head * a.qs[1] + i * a.qs[2]
                                   : nullptr;
        uint4 w[kLanes];
#pragma unroll
        for (int u = 0; u < kLanes; ++u) {
          const uint16_t* q = reinterpret_cast<const uint16_t*>(
              __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), u * kAtOnce + lane / kLanes));
          w[u] = make_uint4(0, 0, 0, 0);
          if (q) w[u] = __ldg(reinterpret_cast<const uint4*>(q) + lane % kLanes);
        }
#pragma unroll
        for (int u = 0; u < kLanes; ++u) {
          if constexpr (!C::kF16) {
            uint32_t* x = &w[u].x;
            float top = 0.0f, up, down;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmax3(top, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
#pragma unroll
            for (int o = 1; o < kLanes; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            dec_row_scale(top, up, down);
            const float got = __shfl_sync(0xFFFFFFFFu, down, (lane % kAtOnce) * kLanes);
            if (lane / kAtOnce == u) rs = got;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack_f16x2(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
          }
          const int r = (warp & 3) * 32 + u * kAtOnce + lane / kLanes, c16 = lane % kLanes;
          *reinterpret_cast<uint4*>(q_tile + (c16 / 8) * (128 * 128) + r * 128 + (((c16 % 8) ^ (r & 7)) << 4)) = w[u];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if ((warp & 3) == 0) ctl->n[t][pieces & 1] = n;
        mbar_arrive(&ctl->q_full[t]);
      }

      const float f_row = rs * a.scale_log2;
      float m = -INFINITY, l = 0.0f;  // m: the reference
#pragma unroll 1
      for (int j = 0; j < n * C::kParts; ++j, ++nth) {
        const int buf = nth & 1;
        ok = prompt_warp_wait(&ctl->s_full[t][buf], (uint32_t)(nth >> 1) & 1u, abort, a);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_addr + t * 128 + buf * C::kKeys;
        const float4* meta = s_meta + ((nth / C::kParts) & 3) * C::kGroups + (nth % C::kParts) * kGroups;
        const int key0 = first * 128 + j * C::kKeys, lo = see.x - key0, hi = see.y - key0;
        uint32_t x[C::kKeys];  // the row's scores (fp32 bits)
#pragma unroll
        for (int cc = 0; cc < C::kKeys / 32; ++cc)
          tmem_ld32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
        tmem_wait_ld();
        reg_fence(x);
        if constexpr (!C::kRaw) prompt_scale<C>(x, a, meta, rs);
        if (lo > 0 || hi < C::kKeys) {
#pragma unroll
          for (int k = 0; k < C::kKeys; ++k)
            if (k < lo || k >= hi) x[k] = 0xFF800000u;
        }
        // Group by group: a raw score times f plus y is the score's weight in
        // base 2 (s + log2 vs); y = -inf where nothing is stored.
        float f[kGroups], y[kGroups], inv_vs[kGroups], mx;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float4 q = meta[g];
          f[g] = C::kRaw ? fmaxf(q.x * f_row, 1e-37f) : 1.0f;  // (not 0: a hidden score stays -inf)
          y[g] = q.w == 0.0f ? -INFINITY : q.y;
          inv_vs[g] = q.z;
        }
        // The weights against the maximum so far, and the new maximum beside
        // them: neither waits for the other.  Where a row's maximum has grown
        // too far for that, once more against the new one.
        float corr = 1.0f, part;
        bool moved = false;
#pragma unroll 1
        while (true) {
          const float base = m == -INFINITY ? 0.0f : m;
          mx = -INFINITY, part = 0.0f;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float off = y[g] - base;
            float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c0 = 0; c0 < C::kGroup; c0 += 16) {
              uint32_t pk[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int k = C::kGroup * g + c0 + 2 * e;
                float x0 = __uint_as_float(x[k]), x1 = __uint_as_float(x[k + 1]);
                v[e & 3] = fmax3(v[e & 3], x0, x1);
                ffma2(x0, x1, x0, x1, f[g], f[g], off, off);
                x0 = ex2(x0), x1 = ex2(x1);
                fadd2(sum[(e & 1) * 2], sum[(e & 1) * 2 + 1], x0, x1);
                pk[e] = pack_f16x2(x0, x1);
              }
              tmem_st8(tS + (C::kGroup * g + c0) / 2, pk);
            }
            mx = fmaxf(mx, fmaf(fmax3(fmaxf(v[0], v[1]), v[2], v[3]), f[g], y[g]));
            part = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), inv_vs[g], part);
          }
          const bool resc = dec_grown(mx, m);  // (not twice: from its own reference a maximum is no further than the lift)
          if (!__any_sync(0xFFFFFFFFu, resc)) break;
          moved = true;
          if (resc) {
            const float r = dec_reference<C>(mx);
            corr = ex2(m - r);  // 0 when m = -inf
            m = r;
          }
        }
        l = fmaf(l, corr, part);
        if (j > 0) {  // the PV before has landed (each phase is consumed, in order)
          ok = prompt_warp_wait(&ctl->o_ready[t], (uint32_t)(nth - 1) & 1u, abort, a);
          if (!ok) break;
        }
        if (j > 0 && moved) {
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < C::kD / 32; ++cc) {
            uint32_t rr[32];
            tmem_ld32(tO + cc * 32, rr);
            tmem_wait_ld();
            reg_fence(rr);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float o0, o1;
              fmul2(o0, o1, __uint_as_float(rr[e]), __uint_as_float(rr[e + 1]), corr, corr);
              rr[e] = __float_as_uint(o0);
              rr[e + 1] = __float_as_uint(o1);
            }
            tmem_st32(tO + cc * 32, rr);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_ready[t]);
      }
      if (!ok) break;
      ok = prompt_warp_wait(&ctl->o_ready[t], (uint32_t)(nth - 1) & 1u, abort, a);
      if (!ok) break;
      tc_fence_after();
      const bool none = l == 0.0f;  // sees nothing (another row's NaN value may be in its O; a NaN row stays one)
      const float inv = dec_unlift(C::kLift) / l;
      const long long slot = (long long)(2 * blockIdx.x + (head_cut ? 0 : 1)) * C::kRows + t * 128 + tl;
      uint8_t* dst = static_cast<uint8_t*>(a.o) + (at.b * a.os[0] + head * a.os[1] + i * a.os[2]) * 2;
#pragma unroll 1
      for (int cc = 0; cc < C::kD / 32; ++cc) {
        uint32_t rr[32];
        tmem_ld32(tO + cc * 32, rr);
        tmem_wait_ld();
        reg_fence(rr);
        if (real && whole) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float o0 = __uint_as_float(rr[8 * u + 2 * e]) * inv, o1 = __uint_as_float(rr[8 * u + 2 * e + 1]) * inv;
              y[e] = none ? 0u : C::kF16 ? pack_f16x2(o0, o1) : pack_bf16x2(o0, o1);
            }
            *reinterpret_cast<uint4*>(dst + cc * 64 + u * 16) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else if (real) {
          uint4* part = reinterpret_cast<uint4*>(p.part_o + slot * C::kD + cc * 32);
#pragma unroll
          for (int u = 0; u < 8; ++u) part[u] = make_uint4(rr[4 * u], rr[4 * u + 1], rr[4 * u + 2], rr[4 * u + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      if (real) {
        if (whole)
          a.lse[((long long)at.b * a.Hq + head) * a.n + i] = none ? -INFINITY : ((m + C::kLift) + lg2(l)) * kDecLn2;
        else
          p.part_ml[slot] = make_float2(m, l);
      }
      pos += n;
      dec_next(p, at, tiles);
    }
    if (ok && lane == 0) {
      if ((warp & 3) == 0) ctl->n[t][pieces & 1] = 0;
      mbar_arrive(&ctl->q_full[t]);
    }
    tmem_wait_st();  // (behind an expired wait, weights may be on their way to memory that is given back below)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
