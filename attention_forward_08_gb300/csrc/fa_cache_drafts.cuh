// fa_cache_drafts.cuh -- attention of a tree of drafts over the 8-bit cache,
// for more rows (drafts times the heads of a group) than the decode kernel's
// registers hold.
//
// The same operation and mathematics as fa_cache_prompt.cuh: rows are the tensor
// core's rows, P'_ij = 2^(s_ij + log2 vs_j - r_i) in f16, r_i 2^7 below the running
// maximum.  What differs is where the time goes: a piece of a prompt has many
// row groups that find a head's keys in L2; here one row group, or two, reads
// them from HBM, once.
//
// Loads.  One warp looks up blocks and scales, up to 16 blocks of 128 keys
// ahead; one keeps 48 KB of stored bytes on their way, by TMA into a ring of
// their own (in registers of the converter warps the compiler waits for the last
// of several loads where the first is needed); the converter warps widen what
// has landed.
//
// Streams.  Up to 128 rows (kSplit) are one row tile, and the two softmax
// warpgroups take the blocks of keys in turn, each with its own maximum, sum
// and output in tensor memory, which are joined at a piece's end: as many
// blocks are in work at a time as with two row tiles.  Up to 256 rows are two
// tiles as in the prompt kernel.  D = 256 has room for one stream, and for 64 rows
// (half of a tile; its other half computes what lies behind, which nobody reads).
//
// Bound: memory, 2 * D bytes a token and K/V head; then the converters and the
// softmax warps' chains.
#pragma once

#include "fa_cache_decode.cuh"
#include "fa_cache_prompt.cuh"
#include "fa_cache_tree.cuh"

namespace fa {

template <int kKind_, bool kF16_, int kD_, int kGroup_, bool kRaw_, bool kSplit_>
struct DraftCfg {
  static constexpr bool kTree = true;
  static constexpr bool kRaw = kRaw_;      // scores need no more than a positive factor
  static constexpr bool kSplit = kSplit_;  // two streams of keys for one row tile
  static constexpr int kGroup = kGroup_;   // tokens that surely share a cache block: 16, or 64
  static constexpr int kKind = kKind_;
  static constexpr bool kF16 = kF16_;
  static constexpr int kD = kD_;
  static_assert(kD <= 128 || !kSplit, "no room for two outputs");
  static constexpr int kTiles = kD <= 128 && !kSplit ? 2 : 1;  // 128-row tiles
  static constexpr int kSoft = kD <= 128 ? 2 : 1;              // softmax warpgroups, issuers
  static constexpr int kRows = kD == 256 ? 64 : 128 * kTiles;
  static constexpr int kQRows = kD == 256 ? 64 : 128;          // of a tile in shared memory
  static constexpr int kTile = 128;  // keys a block of the line
  static constexpr int kMinTiles = 4;
  static constexpr int kLift = 7;
  // Stages of the widened K and V, and the ring of stored bytes: pieces of 128
  // keys (D = 256: 64).
  static constexpr int kStagesK = kD == 64 ? 4 : kD == 128 ? 2 : 1, kStagesV = kD == 128 && !kSplit ? 1 : kStagesK;
  static constexpr int kPieceKeys = kD == 256 ? 64 : 128, kPieceBytes = kPieceKeys * kD, kPieces = 128 / kPieceKeys;
  static constexpr int kRing = 49152 / kPieceBytes;
  static constexpr int kKeys = kD <= 128 ? 64 : 128, kParts = 128 / kKeys;  // keys a score buffer
  static constexpr int kConvWarps = 8;
  static constexpr int kThreads = 128 + 32 * kConvWarps + 128 * kSoft;
  // Registers: at launch 640 threads x 96 or 512 x 128.
  static constexpr int kRegsLaunch = kThreads == 640 ? 96 : 128;
  static constexpr int kRegsCtrl = kD <= 128 ? 48 : 56, kRegsConv = kD <= 128 ? 64 : 72, kRegsSoft = kD <= 128 ? 152 : 240;
  static_assert(kRegsCtrl < kRegsLaunch && kRegsConv < kRegsLaunch && kRegsSoft > kRegsLaunch, "which warps give, which take");
  static_assert(128 * kRegsCtrl + 32 * kConvWarps * kRegsConv + 128 * kSoft * kRegsSoft <= kThreads * kRegsLaunch,
                "register split exceeds the launch allocation");
  static constexpr int kUnits = kD / 16;                            // 16-byte units a key
  static constexpr int kSet = kPieceKeys * kUnits / (32 * kConvWarps);  // a converter's units of a piece: 2 or 4
  static constexpr int kQBytes = kQRows * kD * 2, kKvBytes = 128 * kD * 2;
  static constexpr int kOffK = kTiles * kQBytes, kOffV = kOffK + kStagesK * kKvBytes;
  static constexpr int kOffRing = kOffV + kStagesV * kKvBytes, kOffInfo = kOffRing + 49152;
  static constexpr int kColO = 256;  // S: two buffers of kKeys columns a stream; P over S
};

constexpr int kDraftAhead = 16;   // blocks of keys that are looked up ahead, in batches of 4
constexpr int kDraftWords = 8;    // of a row's drafts that are kept (more are looked for again and again)

template <class C>
struct DraftInfo {
  float4 meta[kDraftAhead][8];          // by 16 keys: ks, log2 vs, 1 / vs less the lift, there
  int2 from[kDraftAhead][8];            // cache block (-1: none), head
  int range[kDraftAhead][8];            // keys that are stored and seen: lo | hi << 8; values that count: lo << 16 | hi << 24
  int tok[kDraftAhead];                 // a block's first token
  uint32_t all[kDraftAhead];            // 1: all keys are stored and seen; 2: all values count
  uint32_t line[kDraftWords][128 * C::kSoft];  // the drafts that a softmax thread's row sees
  float2 ml[2][128];                    // (streams) references and sums
  uint64_t q_full[2];                   // 4 softmax warps: query tile written
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2][2];                // [stream][buffer]: S computed
  uint64_t p_ready[2];                  // softmax wrote P (and rescaled O)
  uint64_t o_ready[2];                  // each PV done
  uint64_t info_full[4], info_empty[4], ring_full[6], ring_empty[6], drain[2];
  int n[2][2];                          // [stream][piece & 1]: blocks of a piece (0: no more), beside q_full
  uint32_t tmem;
  int abort;
};

template <class C>
constexpr int kDraftSmem = 1024 + C::kOffInfo + (int)sizeof(DraftInfo<C>);

// A row's scores to base 2 where one positive factor cannot do it.
template <class C>
__device__ __forceinline__ void draft_scale(uint32_t (&x)[C::kKeys], const CacheAttnParams& a, const float4* meta, float rs) {
#pragma unroll
  for (int g = 0; g < C::kKeys / C::kGroup; ++g) {
    const float ks = meta[g * (C::kGroup / 16)].x * rs, ci = ks * a.cap_in * 2.8853900817779268f;
#pragma unroll
    for (int k = C::kGroup * g; k < C::kGroup * (g + 1); ++k) {
      const float v = __uint_as_float(x[k]);
      // cap * tanh(y) = cap * (1 - 2 / (2^(2 y log2 e) + 1))
      x[k] = __float_as_uint(a.cap_out > 0.0f ? fmaf(-2.0f * a.cap_out, rcp_approx(ex2(v * ci) + 1.0f), a.cap_out)
                                              : v * (ks * a.scale_log2));
    }
  }
}

// Of 32 keys, those that row i sees: the ones from lo to hi - 1, where the drafts
// begin, and its drafts.
template <class C>
__device__ __forceinline__ uint32_t draft_seen(const CacheAttnParams& a, int b, int i, const uint32_t* line, int lo, int hi) {
  const int from = min(max(lo, 0), 32), to = min(max(hi, 0), 32);
  uint32_t seen = from < to ? (0xFFFFFFFFu >> (32 - (to - from))) << from : 0u;
  if (hi < 32) seen |= a.n <= 32 * kDraftWords ? tree_read_line<128 * C::kSoft>(line, a.n, -hi) : tree_walk(a, b, i, -hi);
  return seen;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) cache_drafts_kernel(
    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ DecParams p) {
  static_assert(kDraftSmem<C> <= 232448, "shared memory");
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  DraftInfo<C>* info = reinterpret_cast<DraftInfo<C>*>(smem + C::kOffInfo);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecPlace at;
  if (!dec_find<C>(p, blockIdx.x, at)) return;  // the whole block: nothing is set up yet
  const int t0 = at.part * (int)blockIdx.x, t1 = (int)min((long long)at.total, (long long)t0 + at.part);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&info->q_full[i], 4);
      mbar_init(&info->s_full[i][0], 1);
      mbar_init(&info->s_full[i][1], 1);
      mbar_init(&info->p_ready[i], 4);
      mbar_init(&info->o_ready[i], 1);
      mbar_init(&info->drain[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&info->k_full[i], C::kConvWarps);
      mbar_init(&info->v_full[i], C::kConvWarps);
      mbar_init(&info->k_empty[i], C::kTiles);
      mbar_init(&info->v_empty[i], C::kTiles);
      mbar_init(&info->info_full[i], 1);
      mbar_init(&info->info_empty[i], C::kSoft);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&info->ring_full[i], 1);
      mbar_init(&info->ring_empty[i], C::kConvWarps);
    }
    info->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    tmem_alloc(&info->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = info->tmem;
  volatile int* abort = &info->abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return prompt_warp_wait(bar, parity, abort, a); };
  // Block nb of this thread block's has stages nb % kStagesK and nb % kStagesV;
  // stream t takes every block, or those with nb % 2 == t.
  constexpr int kStep = C::kSplit ? 2 : 1;

  if (warp < 4) {
    // ============================================================ control
    regs_dec<C::kRegsCtrl>();
    if (warp < C::kSoft) {
      // ---------------------------------------------------------- MMAs
      const int t = warp;
      constexpr uint32_t idS = make_idesc_fmt(kFmtF16, 128, C::kKeys, false, false);
      constexpr uint32_t idPV = make_idesc_fmt(kFmtF16, 128, C::kD, false, true);
      const uint64_t dQ = make_sdesc_sw128(smem_u32(smem + (C::kSplit ? 0 : t * C::kQBytes)), 16, 1024);
      const uint64_t dK = make_sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV = make_sdesc_sw128(smem_u32(smem + C::kOffV), 128 * 128, 1024);
      const uint32_t lead = elect_lead();
      auto issue_S = [&](int buf, int stage, int part) {
        const uint64_t k0 = dK + ((stage * C::kKvBytes + part * (C::kKeys * 128)) >> 4);
        const uint32_t dst = tmem + t * 128 + buf * C::kKeys;
#pragma unroll
        for (int kk = 0; kk < C::kD / 16; ++kk) {
          mma_f16_ss_by(lead, dst, dQ + (kk / 4) * ((C::kQRows * 128) >> 4) + (kk % 4) * 2,
                        k0 + (kk / 4) * ((128 * 128) >> 4) + (kk % 4) * 2, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit_by(lead, &info->s_full[t][buf]);
        if (part == C::kParts - 1) mma_commit_by(lead, &info->k_empty[stage]);
      };
      auto issue_PV = [&](int buf, int stage, int part, bool first) {
        const uint64_t v0 = dV + ((stage * C::kKvBytes + part * (C::kKeys * 128)) >> 4);
        const uint32_t src = tmem + t * 128 + buf * C::kKeys, dst = tmem + C::kColO + t * C::kD;
#pragma unroll
        for (int kk = 0; kk < C::kKeys / 16; ++kk)
          mma_f16_ts_by(lead, dst, src + kk * 8, v0 + ((kk * 16 * 128) >> 4), idPV, first && kk == 0 ? 0u : 1u);
        mma_commit_by(lead, &info->o_ready[t]);
        if (part == C::kParts - 1) mma_commit_by(lead, &info->v_empty[stage]);
      };
      auto stage_of = [](int nb) { return nb & (C::kStagesK - 1); };
      auto par_of = [](int nb) { return (uint32_t)(nb / C::kStagesK) & 1u; };
      int nth = 0, before = 0;  // this stream's score buffers; all blocks of earlier pieces
      bool ok = true;
#pragma unroll 1
      for (int pieces = 0; ok; ++pieces) {
        uint64_t* const q_full = &info->q_full[C::kSplit ? 0 : t];
        ok = prompt_warp_wait<true>(q_full, pieces & 1, abort, a);  // (query rows take a while to come)
        if (!ok) break;
        const int n = info->n[C::kSplit ? 0 : t][pieces & 1];
        if (n == 0) break;
        const int begin = C::kSplit && (before & 1) != t ? before + 1 : before, end = before + n;
        before = end;
        if (begin >= end) continue;
        ok = wait(&info->k_full[stage_of(begin)], par_of(begin));
        if (!ok) break;
        tc_fence_after();
        issue_S(nth & 1, stage_of(begin), 0);
#pragma unroll 1
        for (int nb = begin; nb < end && ok; nb += kStep) {
          const int stage = stage_of(nb), next = nb + kStep, stage_v = nb & (C::kStagesV - 1);
#pragma unroll
          for (int part = 0; part < C::kParts; ++part) {
            // the next scores go before this PV
            if (part + 1 < C::kParts) {
              issue_S((nth + 1) & 1, stage, part + 1);
            } else if (next < end) {
              ok = wait(&info->k_full[stage_of(next)], par_of(next));
              if (!ok) break;
              tc_fence_after();
              issue_S((nth + 1) & 1, stage_of(next), 0);
            }
            ok = (part > 0 || wait(&info->v_full[stage_v], (uint32_t)(nb / C::kStagesV) & 1u)) && wait(&info->p_ready[t], (uint32_t)nth & 1u);
            if (!ok) break;
            tc_fence_after();
            issue_PV(nth & 1, stage_v, part, nb == begin && part == 0);
            ++nth;
          }
          if (!ok) break;
          if ((nb & 3) == (C::kSplit ? 2 + t : 3)) mma_commit_by(lead, &info->info_empty[(nb >> 2) & 3]);
        }
      }
      // Every MMA issued here has completed before the block lets go of its
      // memory (after an expired wait too; bounded).
      mma_commit_by(lead, &info->drain[t]);
      if (lead) {
        const long long begin = clock64_now();
        while (!mbar_try_wait(&info->drain[t], 0) && clock64_now() - begin < kDecDrainCycles) {
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------- blocks and scales
      // Four blocks of keys at a time, a lane 16 keys.
      int pos = t0, left = 0, tok = 0;  // of the piece: blocks left, the next one's first token
      int2 span = make_int2(0, 0);
      bool ok = true;
#pragma unroll 1
      for (int nb = 0; nb < t1 - t0 && ok; nb += 4) {
        int b = 0, h = 0, mine = 0, lo = 0, hi = 0;  // this lane's keys: the first, and those that are seen
        bool any = false;                            // are some of its kGroup keys seen?
#pragma unroll 1
        for (int q = 0; q < min(4, t1 - t0 - nb); ++q) {
          if (left == 0) {
            if (pos > t0) dec_next(p, at, dec_tiles<C>(p, at.seq, at.rg));
            if (lane == 0 && at.h == 0 && at.rg == 0 && pos == at.seg0) (void)checked_len(c, a.lens[at.b]);
            span = dec_group_span<C>(p, at.seq, at.rg);
            left = min(t1, at.seg0 + dec_tiles<C>(p, at.seq, at.rg)) - pos;
            tok = (span.x / 128 + pos - at.seg0) * 128;
          }
          if ((lane >> 3) == q) {
            b = at.b, h = at.h;
            mine = tok + 16 * (lane & 7);
            lo = max(span.x - mine, 0), hi = max(min(span.y - mine, 16), 0);
            const int of = mine & ~(C::kGroup - 1);
            any = of < span.y && of + C::kGroup > span.x;
          }
          tok += 128;
          --left, ++pos;
        }
        const int slot = (nb + (lane >> 3)) & (kDraftAhead - 1), g = lane & 7, batch = nb >> 2;
        const int blk = any ? checked_block(c, c.table, c.table_stride, b, mine >> c.page_log2) : -1;
        float ks = 0.0f, vs = 0.0f;
        if (blk >= 0) {
          ks = __ldg(c.k_scale + (long long)blk * c.H + h);
          vs = __ldg(c.v_scale + (long long)blk * c.H + h);
        }
        if (batch >= 4) ok = wait(&info->info_empty[batch & 3], (uint32_t)((batch >> 2) - 1) & 1u);
        if (!ok) break;
        // (values of a zero scale are zeros, and count with the scale 1)
        const bool zero = !(vs >= 1.17549435e-38f);
        info->meta[slot][g] = make_float4(ks, zero ? 0.0f : lg2(vs), dec_unlift(C::kLift) * (zero ? 1.0f : 1.0f / vs), blk >= 0 ? 1.0f : 0.0f);
        info->from[slot][g] = make_int2(blk, h);
        if (g == 0) info->tok[slot] = mine;
        const int keys = blk >= 0 && lo < hi ? lo | (hi << 8) : 0;
        info->range[slot][g] = keys | (zero ? 0 : keys << 16);
        const uint32_t k_all = __ballot_sync(0xFFFFFFFFu, keys == 16 << 8), v_all = __ballot_sync(0xFFFFFFFFu, keys == 16 << 8 && !zero);
        const int shift = lane & 24;
        if (g == 0) info->all[slot] = (((k_all >> shift) & 255u) == 255u ? 1u : 0u) | (((v_all >> shift) & 255u) == 255u ? 2u : 0u);
        __syncwarp();
        if (lane == 0) mbar_arrive(&info->info_full[batch & 3]);
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------- stored bytes
      // A lane a 16-key group; one of those that share a box of the tensor map
      // copies it (its block, if any of them has one).
      constexpr int kGroupsHere = C::kPieceKeys / 16;
      const int rows = min(c.page, C::kPieceKeys), share = rows / 16;
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int nb = 0; nb < t1 - t0 && ok; ++nb) {
        if ((nb & 3) == 0) ok = wait(&info->info_full[(nb >> 2) & 3], (uint32_t)(nb >> 4) & 1u);
        if (!ok) break;
        const int at_info = nb & (kDraftAhead - 1), tok = info->tok[at_info];
#pragma unroll 1
        for (int i = 0; i < 2 * C::kPieces; ++i) {
          const bool is_v = i >= C::kPieces;
          const int g0 = (is_v ? i - C::kPieces : i) * kGroupsHere, g = g0 + lane % kGroupsHere;
          const int2 from = info->from[at_info][g];
          int blk = lane < kGroupsHere ? from.x : -1;
#pragma unroll
          for (int o = 1; o < kGroupsHere; o <<= 1) {
            const int other = __shfl_xor_sync(0xFFFFFFFFu, blk, o);
            if (o < share) blk = max(blk, other);
          }
          const bool box = lane < kGroupsHere && (lane & (share - 1)) == 0 && blk >= 0;
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, box));
          if (issued >= C::kRing) ok = wait(&info->ring_empty[slot], phase ^ 1u);
          if (!ok) break;
          uint64_t* const bar = &info->ring_full[slot];
          if (lane == 0) {
            if (boxes > 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * rows * C::kD));
            else mbar_arrive(bar);
          }
          __syncwarp();
          if (box)
            tma_load_4d(smem + C::kOffRing + slot * C::kPieceBytes + lane * 16 * C::kD, is_v ? &tv : &tk, bar, 0,
                        (tok + 16 * g) & (c.page - 1), from.y, blk);
          __syncwarp();
          ++issued;
          if (++slot == C::kRing) slot = 0, phase ^= 1u;
        }
      }
      // Copies land before the block ends (also where nobody looked at them; bounded).
      const long long begin = clock64_now();
      for (int k = max(0, issued - C::kRing); k < issued; ++k)
        while (!mbar_try_wait(&info->ring_full[k % C::kRing], (uint32_t)(k / C::kRing) & 1u) &&
               clock64_now() - begin < kDecDrainCycles) {
        }
    }
  } else if (warp < 4 + C::kConvWarps) {
    // ============================================================ converters
    regs_dec<C::kRegsConv>();
    const int cw = warp - 4;
    // Lane bits 0-1: unit, 2: key, then units, then keys: eight neighbours
    // write eight different 16-byte columns of the swizzled rows.
    constexpr int kHigh = C::kUnits / 4;
    constexpr int kKeysWarp = 32 / C::kUnits, kKeysStep = kKeysWarp * C::kConvWarps;  // 64, 32, 16
    const int unit = (lane & 3) + 4 * ((lane >> 3) % kHigh);
    const int key0 = cw * kKeysWarp + ((lane >> 2) & 1) + 2 * ((lane >> 3) / kHigh);
    const int g0 = key0 >> 4, r = key0 & 15;  // its keys of a piece are key r of groups g0, g0 + kKeysStep / 16, ..
    uint8_t* const to = smem + C::kOffK + (uint32_t)(unit / 4) * (128 * 128) + key0 * 128;
    const uint32_t lo16 = (((unit % 4) * 2) ^ (key0 & 7)) << 4, hi16 = (((unit % 4) * 2 + 1) ^ (key0 & 7)) << 4;
    const uint32_t from = smem_u32(smem + C::kOffRing) + key0 * C::kD + unit * 16;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int nb = 0; nb < t1 - t0 && ok; ++nb) {
      const int at_info = nb & (kDraftAhead - 1);
#pragma unroll
      for (int i = 0; i < 2 * C::kPieces; ++i) {
        const bool is_v = i >= C::kPieces;
        const int piece = is_v ? i - C::kPieces : i;
        ok = wait(&info->ring_full[slot], phase);
        if (!ok) break;
        uint4 x[C::kSet];
#pragma unroll
        for (int u = 0; u < C::kSet; ++u) x[u] = lds128(from + slot * C::kPieceBytes + u * (kKeysStep * C::kD));
        if (!(info->all[at_info] & (is_v ? 2u : 1u))) {  // where nobody sees them or nothing is stored: zeros
          const int* range = info->range[at_info] + piece * (C::kPieceKeys / 16) + g0;
#pragma unroll
          for (int u = 0; u < C::kSet; ++u) {
            const int keys = range[u * (kKeysStep / 16)] >> (is_v ? 16 : 0);
            if (!(r >= (keys & 255) && r < ((keys >> 8) & 255))) x[u] = make_uint4(0, 0, 0, 0);
          }
        }
        constexpr int kStages[2] = {C::kStagesK, C::kStagesV};
        const int stages = kStages[is_v], stage = nb & (stages - 1);
        if (piece == 0 && nb >= stages) {
          ok = wait(is_v ? &info->v_empty[stage] : &info->k_empty[stage], (uint32_t)(nb / stages + 1) & 1u);
          if (!ok) break;
        }
        uint8_t* const row = to + (is_v ? C::kOffV - C::kOffK : 0) + stage * C::kKvBytes + piece * (C::kPieceKeys * 128);
#pragma unroll
        for (int u = 0; u < C::kSet; ++u) {  // (a step of kKeysStep keys leaves the swizzle as it is)
          uint4 lo, hi;
          widen16<C::kKind>(x[u], lo, hi);
          *reinterpret_cast<uint4*>(row + u * (kKeysStep * 128) + lo16) = lo;
          *reinterpret_cast<uint4*>(row + u * (kKeysStep * 128) + hi16) = hi;
        }
        if (piece == C::kPieces - 1) fence_proxy_async_smem();
        __syncwarp();
        // (The slot is free once what was read has been used: given back right behind
        // the loads, it was filled again before a warp that waited for its stage
        // had its bytes.)
        if (lane == 0) {
          if (piece == C::kPieces - 1) mbar_arrive(is_v ? &info->v_full[stage] : &info->k_full[stage]);
          mbar_arrive(&info->ring_empty[slot]);
        }
        if (++slot == C::kRing) slot = 0, phase ^= 1u;
      }
    }
  } else {
    // ============================================================ softmax
    regs_inc<C::kRegsSoft>();
    const int t = (warp - 4 - C::kConvWarps) >> 2;
    const int tl = tid - (C::kThreads - 128 * C::kSoft) - 128 * t;  // row of the tile = TMEM lane
    const int row_tile = C::kSplit ? 0 : t;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::kColO + t * C::kD;
    uint8_t* q_tile = smem + row_tile * C::kQBytes;
    constexpr int kGroups = C::kKeys / C::kGroup;  // groups a score buffer
    int nth = 0, before = 0, pieces = 0;  // the stream's score buffers, all blocks, and pieces before this one
    bool ok = true;
#pragma unroll 1
    for (int pos = t0; pos < t1; ++pieces) {
      const int tiles = dec_tiles<C>(p, at.seq, at.rg), n = min(t1, at.seg0 + tiles) - pos;
      const int2 span = dec_group_span<C>(p, at.seq, at.rg);
      const int first = span.x / 128 + pos - at.seg0;
      const bool whole = n == tiles, head_cut = pos > at.seg0;
      const int row = at.rg * C::kRows + row_tile * 128 + tl, i = row / a.group, head = at.h * a.group + row % a.group;
      const bool real = tl < C::kQRows && row < p.rows;
      const int base = at.seq.len - at.seq.nq;  // the first draft's slot
      const bool some = real && i < at.seq.nq && base + i >= 0;
      // Does any row of this warp's count?  (Rows are those of whole tiles.)
      const bool work = __any_sync(0xFFFFFFFFu, real);
      // The warp's query rows, kLanes lanes a row, all loads under way at once:
      // the row's largest entry, then its f16 form.  (S of the piece before is
      // done: the tile may be written.  Both streams load, the first writes.)
      float rs = 1.0f;
      {
        constexpr int kLanes = C::kD / 8, kAtOnce = 32 / kLanes;  // rows a load
        const uint16_t* mine = some ? static_cast<const uint16_t*>(a.q) + at.b * a.qs[0] + head * a.qs[1] + i * a.qs[2]
                                    : nullptr;
        constexpr int kPass = kLanes < 16 ? kLanes : 16;
#pragma unroll
        for (int u0 = 0; u0 < kLanes; u0 += kPass) {
          uint4 w[kPass];
#pragma unroll
          for (int u = 0; u < kPass; ++u) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(
                __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), (u0 + u) * kAtOnce + lane / kLanes));
            w[u] = make_uint4(0, 0, 0, 0);
            if (q) w[u] = __ldg(reinterpret_cast<const uint4*>(q) + lane % kLanes);
          }
#pragma unroll
          for (int u = 0; u < kPass; ++u) {
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
              if (lane / kAtOnce == u0 + u) rs = got;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = pack_f16x2(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
            }
            const int r = (warp & 3) * 32 + (u0 + u) * kAtOnce + lane / kLanes, c16 = lane % kLanes;
            if (r < C::kQRows && (!C::kSplit || t == 0))
              *reinterpret_cast<uint4*>(q_tile + (c16 / 8) * (C::kQRows * 128) + r * 128 + (((c16 % 8) ^ (r & 7)) << 4)) = w[u];
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && (!C::kSplit || t == 0)) {
        if ((warp & 3) == 0) info->n[t][pieces & 1] = n;
        mbar_arrive(&info->q_full[t]);
      }
      int lo_row = 0;  // the first token before the drafts that the row sees
      if (some && a.window > 0) lo_row = tree_first(a, base, tree_depth(a, at.b, i));
      uint32_t* const line = &info->line[0][t * 128 + tl];
      if (some && a.n <= 32 * kDraftWords && (first + n) * 128 > base) tree_write_line<128 * C::kSoft>(a, at.b, i, line);
      __syncwarp();

      const float f_row = rs * a.scale_log2;
      float m = -INFINITY, l = 0.0f;  // m: the reference
      int done = 0;                   // score buffers of this piece
#pragma unroll 1
      for (int nb = C::kSplit && (before & 1) != t ? before + 1 : before; nb < before + n && ok; nb += kStep) {
#pragma unroll 1
        for (int part_at = 0; part_at < C::kParts; ++part_at, ++nth, ++done) {
          const int buf = nth & 1;
          ok = wait(&info->s_full[t][buf], (uint32_t)(nth >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tS = tmem + lane_addr + t * 128 + buf * C::kKeys;
          const float4* meta = info->meta[nb & (kDraftAhead - 1)] + part_at * (C::kKeys / 16);
          const int key0 = (first + nb - before) * 128 + part_at * C::kKeys, lo = lo_row - key0, hi = base - key0;
          float corr = 1.0f;
          bool moved = false;
          if (work) {
            uint32_t x[C::kKeys];  // the row's scores (fp32 bits)
#pragma unroll
            for (int cc = 0; cc < C::kKeys / 32; ++cc)
              tmem_ld32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
            tmem_wait_ld();
            reg_fence(x);
            if constexpr (!C::kRaw) draft_scale<C>(x, a, meta, rs);
            if (lo > 0 || hi < C::kKeys) {
              uint32_t seen[C::kKeys / 32] = {};
              if (some) {
#pragma unroll
                for (int w = 0; w < C::kKeys / 32; ++w) seen[w] = draft_seen<C>(a, at.b, i, line, lo - 32 * w, hi - 32 * w);
              }
#pragma unroll
              for (int k = 0; k < C::kKeys; ++k)
                if (!((seen[k / 32] >> (k & 31)) & 1u)) x[k] = 0xFF800000u;
            }
            // Group by group: a raw score times f plus y is the score's weight in
            // base 2 (s + log2 vs); y = -inf where nothing is stored.
            float f[kGroups], y[kGroups], inv_vs[kGroups], mx, part;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const float4 q = meta[g * (C::kGroup / 16)];
              f[g] = C::kRaw ? fmaxf(q.x * f_row, 1e-37f) : 1.0f;  // (not 0: a hidden score stays -inf)
              y[g] = q.w == 0.0f ? -INFINITY : q.y;
              inv_vs[g] = q.z;
            }
            // The weights against the maximum so far, and the new maximum beside
            // them: neither waits for the other.  Where a row's maximum has grown
            // too far for that, once more against the new one.
#pragma unroll 1
            while (true) {
              const float from = m == -INFINITY ? 0.0f : m;
              mx = -INFINITY, part = 0.0f;
#pragma unroll
              for (int g = 0; g < kGroups; ++g) {
                const float off = y[g] - from;
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
          }
          if (done > 0) {  // the PV before has landed (each phase is consumed, in order)
            ok = wait(&info->o_ready[t], (uint32_t)(nth - 1) & 1u);
            if (!ok) break;
          }
          if (done > 0 && moved) {
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
          if (lane == 0) mbar_arrive(&info->p_ready[t]);
        }
      }
      if (ok && done > 0) ok = wait(&info->o_ready[t], (uint32_t)(nth - 1) & 1u);
      // (a NaN row stays one; one that is none, or that sees nothing, has no sum)
      if (!some) l = 0.0f;
      const long long slot = (long long)(2 * blockIdx.x + (head_cut ? 0 : 1)) * C::kRows + row_tile * 128 + tl;
      uint8_t* dst = static_cast<uint8_t*>(a.o) + (at.b * a.os[0] + head * a.os[1] + i * a.os[2]) * 2;
      float f0 = 1.0f, f1 = 0.0f;  // of this stream's output, and the other's
      bool mine = true, other = false;
      if constexpr (C::kSplit) {
        info->ml[t][tl] = make_float2(m, l);
        tc_fence_before();
        if (named_bar_or(3, 256, !ok)) {
          ok = false;
          break;
        }
        const float2 ml = info->ml[t ^ 1][tl];
        mine = done > 0, other = n > 1 || !mine;
        const float top = fmaxf(m, ml.x), z = top == -INFINITY ? 0.0f : top;
        f0 = ex2(m - z), f1 = ex2(ml.x - z);
        l = t == 0 ? fmaf(l, f0, ml.y * f1) : fmaf(ml.y, f1, l * f0);  // (alike in both)
        m = top;
      } else if (!ok) {
        break;
      }
      tc_fence_after();
      const bool none = l == 0.0f;  // sees nothing (another row's NaN value may be in its O)
      const float inv = whole ? dec_unlift(C::kLift) / l : 1.0f;
      f0 *= inv, f1 *= inv;
      // (of two streams' outputs each warpgroup writes half of the columns)
      constexpr int kCols = C::kSplit ? C::kD / 2 : C::kD;
      const uint32_t tOther = tmem + lane_addr + C::kColO + (t ^ 1) * C::kD;
      const int d0 = C::kSplit ? t * kCols : 0;
      if (work) {
#pragma unroll 1
        for (int d = d0; d < d0 + kCols; d += 32) {
          uint32_t rr[32], ro[C::kSplit ? 32 : 1] = {};
          if (mine) tmem_ld32(tO + d, rr);
          if constexpr (C::kSplit) {
            if (other) tmem_ld32(tOther + d, ro);
          }
          tmem_wait_ld();
          reg_fence(rr);
          reg_fence(ro);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float o = mine ? __uint_as_float(rr[e]) * f0 : 0.0f;
            if constexpr (C::kSplit) {
              if (other) o = fmaf(__uint_as_float(ro[e]), f1, o);
            }
            rr[e] = none ? 0u : __float_as_uint(o);
          }
          if (real && whole) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float o0 = __uint_as_float(rr[8 * u + 2 * e]), o1 = __uint_as_float(rr[8 * u + 2 * e + 1]);
                y[e] = C::kF16 ? pack_f16x2(o0, o1) : pack_bf16x2(o0, o1);
              }
              *reinterpret_cast<uint4*>(dst + d * 2 + u * 16) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (real) {
            uint4* part = reinterpret_cast<uint4*>(p.part_o + slot * C::kD + d);
#pragma unroll
            for (int u = 0; u < 8; ++u) part[u] = make_uint4(rr[4 * u], rr[4 * u + 1], rr[4 * u + 2], rr[4 * u + 3]);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      if (real && (!C::kSplit || t == 0)) {
        if (whole)
          a.lse[((long long)at.b * a.Hq + head) * a.n + i] = none ? -INFINITY : ((m + C::kLift) + lg2(l)) * kDecLn2;
        else
          p.part_ml[slot] = make_float2(none ? -INFINITY : m, l);
      }
      if constexpr (C::kSplit) named_bar_sync(3, 256);  // both outputs have been read
      before += n;
      pos += n;
      dec_next(p, at, tiles);
    }
    if (ok && lane == 0 && (!C::kSplit || t == 0)) {
      if ((warp & 3) == 0) info->n[t][pieces & 1] = 0;
      mbar_arrive(&info->q_full[t]);
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
