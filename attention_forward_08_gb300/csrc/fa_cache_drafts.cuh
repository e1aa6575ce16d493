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
// ahead.  Four converter warps take K and four V, so that neither waits for the
// other's place, and each works alone: a lane copies 16 bytes a time into a place
// of its own (cp.async; three pieces of 2 KB a warp, 48 KB in all), widens them and
// writes them where the tensor core reads.  No barrier stands between the copy
// and the use.  (Loads to registers: the compiler waits for the last of several
// where the first is needed.  TMA into common rings: the barriers of a piece cost as
// much as its conversion, 94 us for 16 sequences of up to 8192 tokens with pieces of
// 8 KB, 132 with 4.)
//
// Streams.  Up to 128 rows (kSplit) are one row tile, and of every block of keys
// each of the two softmax warpgroups takes one half, with its own maximum, sum
// and output in tensor memory, which are joined at a piece's end: as many keys
// are in work at a time as with two row tiles.  Up to 64 rows (32) are in the
// tile twice (four times), and a copy weighs every second (fourth) run of keys,
// with a maximum, sum and output of its own: the tensor cores compute the whole
// tile anyhow, and a softmax thread has half (a quarter) of the work.
// D = 256 has room for one stream, and for 64 rows (half of a tile; its other half
// computes what lies behind, which nobody reads).  More rows are several row
// groups, whose second finds the keys in L2.
//
// Bound: memory, 2 * D bytes a token and K/V head; now the converters' and the
// softmax warps' chains (2300 cycles a block of 128 keys of D 128; issue slots half
// busy) and what is done once a piece (20000 cycles).  8 heads of 128, e4m3: 64 rows
// of 16 sequences of up to 8192 tokens 70 us, 2.6 TB/s (the prompt kernel on causal
// rows: 122); 104 rows at 131071 tokens 99 us, 2.7 TB/s (164); 240 rows of 8 x up to
// 6000 tokens 67 us (77).  Tried and slower, on the first and the second when they
// took 76 and 105: the stored bytes by bulk copies, a barrier a piece (85 us); the
// query rows by way of all softmax warps' registers (75, 118).
#pragma once

#include <type_traits>

#include "fa_cache_decode.cuh"
#include "fa_cache_prompt.cuh"
#include "fa_cache_tree.cuh"

namespace fa {

// kDup_: copies of the rows in the row tile, each with its share of the keys.
template <int kD_, int kGroup_, bool kRaw_, int kDup_>
struct DraftCfg {
  static constexpr bool kTree = true;
  static constexpr int kDup = kDup_;
  static constexpr bool kRaw = kRaw_;      // scores need no more than a positive factor
  static constexpr int kGroup = kGroup_;   // tokens that surely share a cache block: 16, or 64
  static constexpr int kD = kD_;
  static constexpr bool kSplit = kD <= 128;  // two streams of keys
  static_assert(kSplit ? kGroup == 16 : kDup == 1, "copies of rows are joined as streams are");
  static constexpr int kSoft = kSplit ? 2 : 1;             // softmax warpgroups, issuers
  static constexpr int kRows = kD == 256 ? 64 : 128;       // of a row group
  static constexpr int kTile = 128;  // keys a block of the line
  static constexpr int kMinTiles = 4;
  // What a piece costs before and behind its keys, in blocks of keys: parts of the line
  // that begin more segments get fewer keys.  (64 rows of 16 sequences of up to 8192
  // tokens, D 128: 76 us with 0, 70.4 with 6, 69.7 with 8, 74 with 12; 240 rows: 76, 67.5,
  // 67.3, 72; D 256: 66, 65.2 with 3, 65.0 with 5, 71 with 8; D 64, 104 rows at 131071
  // tokens: 92.7 with 0, 87.6 with 5, 86.7 with 10, 86.4 with 15, and 33 rows of 16
  // sequences of up to 8192: 57.8, 53.4, 55.4, 58.3.)
  static constexpr int kLead = kD == 64 ? 10 : kD == 128 ? 8 : 5;
  static constexpr int kLift = 7;
  static constexpr int kKeys = 64;   // keys a score buffer: a unit
  // Widened K and V: stages of 16 KB (D = 256: 32).  Stored bytes: three pieces of
  // 2 KB a converter warp.
  static constexpr int kStageKeys = kD == 64 ? 128 : 64, kStageBytes = kStageKeys * kD * 2;
  static constexpr int kStages = kD == 256 ? 2 : 4;  // of K; of V alike
  static constexpr int kPieceKeys = 2048 / kD, kPieceBytes = 2048, kRing = 3;
  static constexpr int kPieces = kStageKeys / kPieceKeys;  // a stage: 4, 4, 8
  static constexpr int kStageUnits = kStageKeys / kKeys;
  // Issuers that are done with a stage, one after the other.
  static constexpr int kReaders = kSplit ? kStageUnits : 1;
  static constexpr int kConvWarps = 8;  // half of them for K, half for V
  static constexpr int kThreads = 128 + 32 * kConvWarps + 128 * kSoft;
  // Registers: at launch 640 threads x 96 or 512 x 128.
  static constexpr int kRegsLaunch = kThreads == 640 ? 96 : 128;
  static constexpr int kRegsCtrl = kD <= 128 ? 48 : 56, kRegsConv = kD <= 128 ? 64 : 72, kRegsSoft = kD <= 128 ? 152 : 240;
  static_assert(kRegsCtrl < kRegsLaunch && kRegsConv < kRegsLaunch && kRegsSoft > kRegsLaunch, "which warps give, which take");
  static_assert(128 * kRegsCtrl + 32 * kConvWarps * kRegsConv + 128 * kSoft * kRegsSoft <= kThreads * kRegsLaunch,
                "register split exceeds the launch allocation");
  static constexpr int kVecs = kD / 16;                              // 16-byte vectors a key
  static constexpr int kSet = kPieceBytes / 16 / 32;  // a lane's of a piece: 4
  static constexpr int kQBytes = kRows * kD * 2;
  // Columns of an output that are written at a time; the copies' for both streams
  // over the query rows, as far as those go.
  static constexpr int kChunk = kDup > 1 ? 32 : 16, kHand = (128 - 128 / kDup) * 128;
  static constexpr int kOffK = kQBytes, kOffV = kOffK + kStages * kStageBytes;
  static constexpr int kOffRing = kOffV + kStages * kStageBytes;
  static constexpr int kOffHand1 = 2 * kHand <= kQBytes ? kHand : kOffRing + kConvWarps * kRing * kPieceBytes;
  static constexpr int kOffInfo = kOffRing + kConvWarps * kRing * kPieceBytes + (kOffHand1 > kHand ? kHand : 0);
  static_assert(kHand <= kQBytes, "room for the copies' outputs");
  static constexpr int kColO = 256;  // S: two buffers of kKeys columns a stream; P over S
};

template <class C, bool kF16_>
struct DraftJoin : C {
  static constexpr bool kF16 = kF16_;
};

constexpr int kDraftAhead = 16;   // blocks of keys that are looked up ahead, in batches of 4
constexpr int kDraftWords = 8;    // of a row's drafts that are kept (more are looked for again and again)

template <class C>
struct DraftInfo {
  float4 meta[kDraftAhead][8];          // by 16 keys: ks, log2 vs, 1 / vs less the lift, there
  long long from[2][kDraftAhead][8];    // K, V: bytes from the pool's begin to the first of 16 keys
  int range[kDraftAhead][8];            // keys that are stored and seen: lo | hi << 8; values that count: lo << 16 | hi << 24
  uint32_t line[kDraftWords][128 * C::kSoft];  // the drafts that a softmax thread's row sees
  float2 ml[2][128];                    // (streams) references and sums
  float rs[128];                        // (streams) a row's factor back
  uint64_t q_full;                      // 4 softmax warps: query tile written
  uint64_t full[2][4], empty[2][4];     // [K, V][stage]
  uint64_t s_full[2][2];                // [stream][buffer]: S computed
  uint64_t p_ready[2][2];               // softmax wrote P (and rescaled O); a warp may be a unit ahead of another
  uint64_t o_ready[2][2];               // PV done, by buffer: nobody is two phases of one behind
  uint64_t info_full[4], info_empty[4], drain[2];
  int n[2];                             // [piece & 1]: blocks of a piece (0: no more), beside q_full
  int blocks;                           // of keys, of all pieces
  uint32_t tmem;
  int abort;
};

template <class C>
constexpr int kDraftSmem = 1024 + C::kOffInfo + (int)sizeof(DraftInfo<C>);

// A row's scores to base 2 where one positive factor cannot do it.
template <class C>
__device__ __forceinline__ void draft_scale(uint32_t (&x)[C::kKeys / C::kDup], const CacheAttnParams& a, const float4* meta, float rs) {
#pragma unroll
  for (int g = 0; g < C::kKeys / C::kDup / C::kGroup; ++g) {
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
// begin, and its drafts: bits of `line` where there are up to 32, else of `lines`.
template <class C>
__device__ __forceinline__ uint32_t draft_seen(const TreeOf& tree, int i, uint32_t line, const uint32_t* lines, int lo, int hi) {
  const int from = min(max(lo, 0), 32), to = min(max(hi, 0), 32);
  uint32_t seen = from < to ? (0xFFFFFFFFu >> (32 - (to - from))) << from : 0u;
  if (hi < 32) {
    if (tree.n <= 32)
      seen |= hi >= 0 ? line << hi : hi > -32 ? line >> -hi : 0u;
    else
      seen |= tree.n <= 32 * kDraftWords ? tree_read_line<128 * C::kSoft>(lines, tree.n, -hi) : tree_walk(tree, i, -hi);
  }
  return seen;
}

// Of a segment of `tiles` places on the line, the blocks of keys before this part
// of the line, t0 .. t1 - 1, and in it (none or less: it ends before the first).
template <class C>
__device__ __forceinline__ int draft_first(const DecPlace& seg, int t0) { return max(t0 - seg.seg0 - C::kLead, 0); }
template <class C>
__device__ __forceinline__ int draft_blocks(const DecPlace& seg, int tiles, int t0, int t1) {
  return min(t1 - seg.seg0, tiles) - C::kLead - draft_first<C>(seg, t0);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) cache_drafts_kernel(const __grid_constant__ DecParams p) {
  static_assert(kDraftSmem<C> <= 232448, "shared memory");
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  DraftInfo<C>* info = reinterpret_cast<DraftInfo<C>*>(smem + C::kOffInfo);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecPlace at;
  if (!dec_find<C>(p, blockIdx.x, at)) {  // the whole block: nothing is set up yet
    if (tid == 0) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int t0 = at.part * (int)blockIdx.x, t1 = (int)min((long long)at.total, (long long)t0 + at.part);
  if (tid == 0) {
    p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
    mbar_init(&info->q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&info->s_full[i][0], 1);
      mbar_init(&info->s_full[i][1], 1);
      mbar_init(&info->p_ready[i][0], 4);
      mbar_init(&info->p_ready[i][1], 4);
      mbar_init(&info->o_ready[i][0], 1);
      mbar_init(&info->o_ready[i][1], 1);
      mbar_init(&info->drain[i], 1);
    }
    for (int kv = 0; kv < 2; ++kv) {
      for (int i = 0; i < 4; ++i) {
        mbar_init(&info->full[kv][i], C::kPieces);
        mbar_init(&info->empty[kv][i], C::kReaders);
      }
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&info->info_full[i], 1);
      mbar_init(&info->info_empty[i], C::kSoft);
    }
    info->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&info->tmem, 512);
    tmem_relinquish();
  } else if (warp == 3) {  // the blocks of keys in this part of the line
    DecPlace seg = at;
    int blocks = 0;
#pragma unroll 1
    while (true) {
      const int tiles = dec_tiles<C>(p, seg.seq, seg.rg);
      blocks += max(draft_blocks<C>(seg, tiles, t0, t1), 0);
      if (t1 <= seg.seg0 + tiles) break;
      dec_next(p, seg, tiles);
    }
    info->blocks = blocks;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = info->tmem;
  volatile int* abort = &info->abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return prompt_warp_wait(bar, parity, abort, a); };
  // Units: halves of this thread block's blocks of keys.  Stream t takes unit t of
  // every block, or all.
  constexpr int kUnitStep = C::kSplit ? 2 : 1;

  if (warp < 4) {
    // ============================================================ control
    regs_dec<C::kRegsCtrl>();
    if (warp < C::kSoft) {
      // ---------------------------------------------------------- MMAs
      const int t = warp;
      constexpr uint32_t idS = make_idesc_fmt(kFmtF16, 128, C::kKeys, false, false);
      constexpr uint32_t idPV = make_idesc_fmt(kFmtF16, 128, C::kD, false, true);
      const uint64_t dQ = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dK = make_sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV = make_sdesc_sw128(smem_u32(smem + C::kOffV), C::kStageKeys * 128, 1024);
      const uint32_t lead = elect_lead();
      // Unit u's bytes in its stage; and is it the last unit that this stream takes of it?
      auto at_stage = [](int u, int stages) {
        return (uint32_t)((u / C::kStageUnits) & (stages - 1)) * C::kStageBytes + (u % C::kStageUnits) * (C::kKeys * 128);
      };
      constexpr int kLast = C::kStageUnits - 1;
      auto leaves = [&](int u) { return C::kSplit || u % C::kStageUnits == kLast; };
      auto issue_S = [&](int buf, int u) {
        const uint64_t k0 = dK + (at_stage(u, C::kStages) >> 4);
        const uint32_t dst = tmem + t * 128 + buf * C::kKeys;
#pragma unroll
        for (int kk = 0; kk < C::kD / 16; ++kk)
          mma_f16_ss_by(lead, dst, dQ + (kk / 4) * ((C::kRows * 128) >> 4) + (kk % 4) * 2,
                        k0 + (kk / 4) * ((C::kStageKeys * 128) >> 4) + (kk % 4) * 2, idS, kk > 0 ? 1u : 0u);
        mma_commit_by(lead, &info->s_full[t][buf]);
        if (leaves(u)) mma_commit_by(lead, &info->empty[0][(u / C::kStageUnits) & (C::kStages - 1)]);
      };
      auto issue_PV = [&](int buf, int u, bool first) {
        const uint64_t v0 = dV + (at_stage(u, C::kStages) >> 4);
        const uint32_t src = tmem + t * 128 + buf * C::kKeys, dst = tmem + C::kColO + t * C::kD;
#pragma unroll
        for (int kk = 0; kk < C::kKeys / 16; ++kk)
          mma_f16_ts_by(lead, dst, src + kk * 8, v0 + ((kk * 16 * 128) >> 4), idPV, first && kk == 0 ? 0u : 1u);
        mma_commit_by(lead, &info->o_ready[t][buf]);
        if (leaves(u)) mma_commit_by(lead, &info->empty[1][(u / C::kStageUnits) & (C::kStages - 1)]);
      };
      auto full = [&](int kv, int stages, int u) {
        const int nth = u / C::kStageUnits;
        return wait(&info->full[kv][nth & (stages - 1)], (uint32_t)(nth / stages) & 1u);
      };
      int nth = 0, before = 0;  // this stream's units; all blocks of earlier pieces
      bool ok = true;
#pragma unroll 1
      for (int pieces = 0; ok; ++pieces) {
        ok = prompt_warp_wait<true>(&info->q_full, pieces & 1, abort, a);  // (query rows take a while to come)
        if (!ok) break;
        const int n = info->n[pieces & 1];
        if (n == 0) break;
        const int begin = 2 * before + (C::kSplit ? t : 0), end = 2 * (before + n);
        before += n;
        ok = full(0, C::kStages, begin);
        if (!ok) break;
        tc_fence_after();
        issue_S(nth & 1, begin);
#pragma unroll 1
        for (int u = begin; u < end; u += kUnitStep, ++nth) {
          if (u + kUnitStep < end) {  // the next scores go before this PV
            ok = full(0, C::kStages, u + kUnitStep);
            if (!ok) break;
            tc_fence_after();
            issue_S((nth + 1) & 1, u + kUnitStep);
          }
          ok = full(1, C::kStages, u) && wait(&info->p_ready[t][nth & 1], (uint32_t)(nth >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          issue_PV(nth & 1, u, u == begin);
          // (the last unit that this stream takes of four blocks that were looked up together)
          if ((u & 7) == (C::kSplit ? 6 + t : 7)) mma_commit_by(lead, &info->info_empty[(u >> 3) & 3]);
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
      const int blocks = info->blocks;
      int left = 0, tok = 0;  // of the piece: blocks left, the next one's first token
      bool begun = false;
      int2 span = make_int2(0, 0);
      bool ok = true;
#pragma unroll 1
      for (int nb = 0; nb < blocks && ok; nb += 4) {
        int b = 0, h = 0, mine = 0, lo = 0, hi = 0;  // this lane's keys: the first, and those that are seen
        bool any = false;                            // are some of its kGroup keys seen?
#pragma unroll 1
        for (int q = 0; q < min(4, blocks - nb); ++q) {
          if (left == 0) {
            if (begun) dec_next(p, at, dec_tiles<C>(p, at.seq, at.rg));
            begun = true;
            const int first = draft_first<C>(at, t0);
            if (lane == 0 && at.h == 0 && at.rg == 0 && first == 0) (void)checked_len(c, a.lens[at.b]);
            span = dec_group_span<C>(p, at.seq, at.rg);
            left = draft_blocks<C>(at, dec_tiles<C>(p, at.seq, at.rg), t0, t1);
            tok = (span.x / 128 + first) * 128;
          }
          if ((lane >> 3) == q) {
            b = at.b, h = at.h;
            mine = tok + 16 * (lane & 7);
            lo = max(span.x - mine, 0), hi = max(min(span.y - mine, 16), 0);
            const int of = mine & ~(C::kGroup - 1);
            any = of < span.y && of + C::kGroup > span.x;
          }
          tok += 128;
          --left;
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
        const long long row = mine & (c.page - 1);
        info->from[0][slot][g] = blk >= 0 ? blk * c.ks[0] + h * c.ks[1] + row * c.ks[2] : 0;
        info->from[1][slot][g] = blk >= 0 ? blk * c.vs[0] + h * c.vs[1] + row * c.vs[2] : 0;
        const int keys = blk >= 0 && lo < hi ? lo | (hi << 8) : 0;
        info->range[slot][g] = keys | (zero ? 0 : keys << 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(&info->info_full[batch & 3]);
      }
    }
  } else if (warp < 4 + C::kConvWarps) {
    // ============================================================ converters
    regs_dec<C::kRegsConv>();
    constexpr int kTeam = C::kConvWarps / 2;  // of K, of V: piece k is warp k % kTeam's
    const int kv = (warp - 4) / kTeam, cw = (warp - 4) % kTeam;
    // Lane bits 0-1: vector, 2: key, then vectors, then keys: eight neighbours
    // write eight different 16-byte columns of the swizzled rows.
    constexpr int kHigh = C::kVecs / 4;
    constexpr int kKeysWarp = 32 / C::kVecs;  // keys at once: 8, 4, 2
    static_assert(kKeysWarp * C::kSet == C::kPieceKeys, "a piece is a set");
    const int vec = (lane & 3) + 4 * ((lane >> 3) % kHigh);
    const int key0 = ((lane >> 2) & 1) + 2 * ((lane >> 3) / kHigh);
    uint8_t* const to = smem + (kv ? C::kOffV : C::kOffK) + (uint32_t)(vec / 4) * (C::kStageKeys * 128) + key0 * 128;
    const uint32_t lo16 = (((vec % 4) * 2) ^ key0) << 4, hi16 = (((vec % 4) * 2 + 1) ^ key0) << 4;
    const uint32_t mine = smem_u32(smem + C::kOffRing + (warp - 4) * C::kRing * C::kPieceBytes) + lane * 16;
    const long long stride = kv ? c.vs[2] : c.ks[2];
    const uint8_t* const pool = (kv ? c.v : c.k) + vec * 16 + key0 * stride;
    const int pieces = 128 / C::kPieceKeys * info->blocks;
    const bool e4m3 = p.kind == kKindE4m3;
    int known = 0;  // blocks that are looked up
    bool ok = true;
    auto copy = [&](int k, int slot) {  // of piece k, as one group
      const int nb = k * C::kPieceKeys / 128, at = nb & (kDraftAhead - 1);
      if (k < pieces && nb >= known) {
        ok = wait(&info->info_full[(nb >> 2) & 3], (uint32_t)(nb >> 4) & 1u);
        known += 4;
      }
      if (k < pieces && ok) {
        // (a piece's keys lie in one 16-key group, or two; what is known about them is read before the first copy)
        constexpr int kGroupsHere = C::kPieceKeys > 16 ? C::kPieceKeys / 16 : 1;
        const int first = (k * C::kPieceKeys) % 128;
        long long off[kGroupsHere];
        int keys[kGroupsHere];
#pragma unroll
        for (int g = 0; g < kGroupsHere; ++g) {
          off[g] = info->from[kv][at][first / 16 + g];
          keys[g] = info->range[at][first / 16 + g] >> (16 * kv);
        }
#pragma unroll
        for (int g = 0; g < kGroupsHere; ++g) {
          constexpr int kOfGroup = C::kSet / kGroupsHere;
          const uint8_t* from = pool + off[g] + first % 16 * stride;
          const int lo = keys[g] & 255, hi = (keys[g] >> 8) & 255;
#pragma unroll
          for (int u = 0; u < kOfGroup; ++u, from += kKeysWarp * stride) {
            const int r = first % 16 + key0 + u * kKeysWarp;
            // (zeros where nobody sees them or nothing is stored)
            copy16(mine + slot * C::kPieceBytes + (g * kOfGroup + u) * 512, from, r >= lo && r < hi);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(cw, 0);
    copy(cw + kTeam, 1);
    int slot = 0;
#pragma unroll 1
    for (int k = cw; k < pieces && ok; k += kTeam) {
      const int nth = k / C::kPieces, part = k % C::kPieces, stage = nth & (C::kStages - 1);
      // (asked early, so that the answer is there when it is needed)
      const bool room = nth < C::kStages || mbar_test(&info->empty[kv][stage], (uint32_t)(nth / C::kStages + 1) & 1u);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      uint4 x[C::kSet];
#pragma unroll
      for (int u = 0; u < C::kSet; ++u) x[u] = lds128(mine + slot * C::kPieceBytes + u * 512);
      copy(k + 2 * kTeam, slot + 2 >= C::kRing ? slot + 2 - C::kRing : slot + 2);
      if (!__all_sync(0xFFFFFFFFu, room)) ok = ok && wait(&info->empty[kv][stage], (uint32_t)(nth / C::kStages + 1) & 1u);
      if (!ok) break;
      uint8_t* const row = to + stage * C::kStageBytes + part * (C::kPieceKeys * 128);
      auto widen = [&](auto kind) {
#pragma unroll
        for (int u = 0; u < C::kSet; ++u) {
          uint4 lo, hi;
          widen16<decltype(kind)::value>(x[u], lo, hi);
          const uint32_t turn = (u * (kKeysWarp << 4)) & 0x70u;  // (the swizzle goes by the key's low three bits)
          *reinterpret_cast<uint4*>(row + u * (kKeysWarp * 128) + (lo16 ^ turn)) = lo;
          *reinterpret_cast<uint4*>(row + u * (kKeysWarp * 128) + (hi16 ^ turn)) = hi;
        }
      };
      if (e4m3) widen(std::integral_constant<int, kKindE4m3>());
      else widen(std::integral_constant<int, kKindInt8>());
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&info->full[kv][stage]);
      if (++slot == C::kRing) slot = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (after an expired wait copies may be on their way)
  } else {
    // ============================================================ softmax
    regs_inc<C::kRegsSoft>();
    const int t = (warp - 4 - C::kConvWarps) >> 2;
    const int tl = tid - (C::kThreads - 128 * C::kSoft) - 128 * t;  // row of the tile = TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::kColO + t * C::kD;  // the stream's output
    constexpr int kMine = C::kKeys / C::kDup, kGroups = kMine / C::kGroup;  // keys of a score buffer a thread weighs; groups
    constexpr int kCopy = 128 / C::kDup;                                    // rows of a copy
    const int copy = C::kDup > 1 ? tl / kCopy : 0;                          // (a warp's)
    int nth = 0, before = 0, pieces = 0;  // the stream's units, all blocks, and pieces before this one
    bool ok = true;
    // The product of a unit's weights has landed.
    auto landed = [&](int unit) { return wait(&info->o_ready[t][unit & 1], (uint32_t)(unit >> 1) & 1u); };
#pragma unroll 1
    for (int pos = t0; pos < t1; ++pieces) {
      const int tiles = dec_tiles<C>(p, at.seq, at.rg), n = draft_blocks<C>(at, tiles, t0, t1), from_block = draft_first<C>(at, t0);
      if (n <= 0) break;
      const int2 span = dec_group_span<C>(p, at.seq, at.rg);
      const int first = span.x / 128 + from_block;
      const bool whole = n == tiles - C::kLead, head_cut = from_block > 0;
      const int row = C::kDup > 1 ? tl & (kCopy - 1) : at.rg * C::kRows + tl, i = row / a.group, head = at.h * a.group + row % a.group;
      const bool real = tl < C::kRows && row < p.rows;
      const int base = at.seq.len - at.seq.nq;  // the first draft's slot
      const bool some = real && i < at.seq.nq && base + i >= 0;
      // Does any row of this warp's count?  (With copies, all warps go on together.)
      const bool work = C::kDup > 1 || __any_sync(0xFFFFFFFFu, real);
      // Up to 32 nodes' parents are on their way with the rows, a lane a node.
      const TreeOf tree = tree_of(a, at.b);
      int up = -1;
      if (tree.n <= 32 && lane < at.seq.nq) up = tree_parent(tree, lane);
      // The warp's query rows, kLanes lanes a row, straight to their place in the
      // tile; then, a thread a row, their f16 form.  (S of the piece before is done: the
      // tile may be written.  With two streams, the first does it.  The loops are
      // rolled: what runs once a piece costs the fetching of its instructions.)
      float rs = 1.0f;
      if (!C::kSplit || t == 0) {
        constexpr int kLanes = C::kD / 8, kAtOnce = 32 / kLanes;  // rows a copy
        const long long from = some ? (at.b * a.qs[0] + head * a.qs[1] + i * a.qs[2]) * 2 : -1;
        const int r0 = (warp & 3) * 32, c16 = lane % kLanes;
        if (r0 < C::kRows) {
          uint8_t* const col = smem + (c16 / 8) * (C::kRows * 128);
#pragma unroll 2
          for (int r = lane / kLanes; r < 32; r += kAtOnce) {
            const long long off = __shfl_sync(0xFFFFFFFFu, from, r);
            copy16(smem_u32(col + (r0 + r) * 128 + (((c16 % 8) ^ (r & 7)) << 4)),
                   static_cast<const uint8_t*>(a.q) + max(off, 0LL) + c16 * 16, off >= 0);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          if (!p.f16) {
            uint8_t* const mine = smem + tl * 128;
            float top = 0.0f, up;
#pragma unroll 4
            for (int c = 0; c < kLanes; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(mine + (c / 8) * (C::kRows * 128) + (((c % 8) ^ (tl & 7)) << 4));
              const uint32_t* x = &w.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top = fmax3(top, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
            }
            dec_row_scale(top, up, rs);
#pragma unroll 4
            for (int c = 0; c < kLanes; ++c) {
              uint4* const at16 = reinterpret_cast<uint4*>(mine + (c / 8) * (C::kRows * 128) + (((c % 8) ^ (tl & 7)) << 4));
              uint4 w = *at16;
              uint32_t* x = &w.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = pack_f16x2(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
              *at16 = w;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if ((warp & 3) == 0) info->n[pieces & 1] = n;
          mbar_arrive(&info->q_full);
        }
        if constexpr (C::kSplit) info->rs[tl] = rs;
      }
      if constexpr (C::kSplit) {
        __syncwarp();  // (here and below: bar.sync and tcgen05's .aligned forms take whole warps)
        named_bar_sync(3, 256);
        rs = info->rs[tl];
      }
      // What the row sees: tokens from lo_row on before the drafts, and its line.
      int lo_row = 0;
      uint32_t line = 0u;
      uint32_t* const lines = &info->line[0][t * 128 + tl];
      if (tree.n <= 32) {
        line = __shfl_sync(0xFFFFFFFFu, tree_lines(up), i & 31);
        if (some) lo_row = tree_window(tree, base, line);
      } else if (some) {
        if (tree.window > 0) lo_row = tree_first(tree, base, tree_depth(tree, i));
        if (tree.n <= 32 * kDraftWords && (first + n) * 128 > base) tree_write_line<128 * C::kSoft>(tree, i, lines);
      }
      __syncwarp();

      const float f_row = rs * a.scale_log2;
      float m = -INFINITY, l = 0.0f;  // m: the reference
      bool fresh = true;              // no unit of this piece yet
#pragma unroll 1
      for (int u = 2 * before + (C::kSplit ? t : 0); u < 2 * (before + n); u += kUnitStep, ++nth, fresh = false) {
        const int buf = nth & 1, nb = u >> 1, part_at = u & 1;
        ok = wait(&info->s_full[t][buf], (uint32_t)(nth >> 1) & 1u);
        if (!ok) break;
        if (nth > 1 && !(ok = landed(nth - 2))) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_addr + t * 128 + buf * C::kKeys;
        const float4* meta = info->meta[nb & (kDraftAhead - 1)] + (part_at * C::kKeys + copy * kMine) / 16;
        const int key0 = (first + nb - before) * 128 + part_at * C::kKeys + copy * kMine, lo = lo_row - key0, hi = base - key0;
        float corr = 1.0f;
        bool moved = false;
        if (work) {
          uint32_t x[kMine];  // the row's scores (fp32 bits)
          if constexpr (kMine == 16) {
            tmem_ld16(tS + copy * kMine, x);
          } else {
#pragma unroll
            for (int cc = 0; cc < kMine / 32; ++cc)
              tmem_ld32(tS + copy * kMine + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
          }
          tmem_wait_ld();
          reg_fence(x);
          if constexpr (!C::kRaw) draft_scale<C>(x, a, meta, rs);
          if (lo > 0 || hi < kMine) {
            uint32_t seen[(kMine + 31) / 32] = {};
            if (some) {
#pragma unroll
              for (int w = 0; w < (kMine + 31) / 32; ++w) seen[w] = draft_seen<C>(tree, i, line, lines, lo - 32 * w, hi - 32 * w);
            }
#pragma unroll
            for (int k = 0; k < kMine; ++k)
              if (!((seen[k / 32] >> (k & 31)) & 1u)) x[k] = 0xFF800000u;
          }
          __syncwarp();
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
                tmem_st8(tS + (copy * kMine + C::kGroup * g + c0) / 2, pk);
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
            __syncwarp();
          }
          l = fmaf(l, corr, part);
          if constexpr (C::kDup > 1) {  // the other copies' keys weigh nothing here
            const uint32_t none[8] = {};
#pragma unroll
            for (int q = 1; q < C::kDup; ++q)
#pragma unroll
              for (int c0 = 0; c0 < kMine / 2; c0 += 8) tmem_st8(tS + ((copy + q) % C::kDup) * (kMine / 2) + c0, none);
          }
        }
        // (The product that read this buffer's weights has landed: its scores were
        // issued behind that.  Outputs that are to be rescaled have one more to come.)
        if (!fresh && moved) {
          if (!(ok = landed(nth - 1))) break;
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
        if (lane == 0) mbar_arrive(&info->p_ready[t][buf]);
      }
      if (ok) ok = landed(nth - 1);
      // (a NaN row stays one; one that is none, or that sees nothing, has no sum)
      if (!some) l = 0.0f;
      const long long slot = (long long)(2 * blockIdx.x + (head_cut ? 0 : 1)) * C::kRows + (C::kDup > 1 ? row : tl);
      uint8_t* dst = static_cast<uint8_t*>(a.o) + (at.b * a.os[0] + head * a.os[1] + i * a.os[2]) * 2;
      float f0 = 1.0f, f1 = 0.0f;  // of the two streams' outputs
      if constexpr (C::kSplit) {
        info->ml[t][tl] = make_float2(m, l);
        tc_fence_before();
        if (named_bar_or(3, 256, !ok)) {
          ok = false;
          break;
        }
        // The row's sum over its copies and streams, always in the same order.
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int q = 0; q < C::kDup; ++q)
          top = fmax3(top, info->ml[0][q * kCopy + (tl & (kCopy - 1))].x, info->ml[1][q * kCopy + (tl & (kCopy - 1))].x);
        const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int q = 0; q < C::kDup; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 ml = info->ml[u][q * kCopy + (tl & (kCopy - 1))];
            sum = fmaf(ml.y, ex2(ml.x - z), sum);
          }
        f0 = ex2(info->ml[0][tl].x - z), f1 = ex2(info->ml[1][tl].x - z);
        m = top, l = sum;
      } else if (!ok) {
        break;
      }
      tc_fence_after();
      const bool none = l == 0.0f;  // sees nothing (another row's NaN value may be in its O)
      const float inv = whole ? dec_unlift(C::kLift) / l : 1.0f;
      f0 *= inv, f1 *= inv;
      // Of two streams' outputs each warpgroup writes half of the columns; copies
      // but the first hand theirs over where the query rows have been.
      constexpr int kCols = C::kSplit ? C::kD / 2 : C::kD;
      const uint32_t tO0 = C::kSplit ? tmem + lane_addr + C::kColO : tO, tO1 = tO0 + C::kD;
      const int d0 = C::kSplit ? t * kCols : 0;
      uint8_t* const hand = smem + t * C::kOffHand1;
      if (work) {
#pragma unroll 1
        for (int d = d0; d < d0 + kCols; d += C::kChunk) {
          constexpr int kN = C::kChunk;
          uint32_t rr[kN], ro[C::kSplit ? kN : 1] = {};
          if constexpr (kN == 16) tmem_ld16(tO0 + d, rr);
          else tmem_ld32(tO0 + d, rr);
          if constexpr (C::kSplit && kN == 16) tmem_ld16(tO1 + d, ro);
          else if constexpr (C::kSplit) tmem_ld32(tO1 + d, ro);
          tmem_wait_ld();
          reg_fence(rr);
          reg_fence(ro);
          float o[kN];
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            o[e] = __uint_as_float(rr[e]) * f0;
            if constexpr (C::kSplit) o[e] = fmaf(__uint_as_float(ro[e]), f1, o[e]);
          }
          if constexpr (C::kDup > 1) {
            if (copy > 0) {
#pragma unroll
              for (int u = 0; u < kN / 4; ++u)
                *reinterpret_cast<float4*>(hand + (tl - kCopy) * 128 + ((u ^ (tl & 7)) << 4)) =
                    make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
            named_bar_sync(1 + t, 128);
            if (copy == 0) {
#pragma unroll
              for (int q = 0; q < C::kDup - 1; ++q)
#pragma unroll
                for (int u = 0; u < kN / 4; ++u) {
                  const float4 y = *reinterpret_cast<const float4*>(hand + (q * kCopy + tl) * 128 + ((u ^ (tl & 7)) << 4));
                  o[4 * u] += y.x, o[4 * u + 1] += y.y, o[4 * u + 2] += y.z, o[4 * u + 3] += y.w;
                }
            }
            named_bar_sync(1 + t, 128);
          }
          if (real && copy == 0) {
#pragma unroll
            for (int e = 0; e < kN; ++e) o[e] = none ? 0.0f : o[e];
            if (whole) {
#pragma unroll
              for (int u = 0; u < kN / 8; ++u) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  y[e] = p.f16 ? pack_f16x2(o[8 * u + 2 * e], o[8 * u + 2 * e + 1]) : pack_bf16x2(o[8 * u + 2 * e], o[8 * u + 2 * e + 1]);
                *reinterpret_cast<uint4*>(dst + d * 2 + u * 16) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
              float4* part = reinterpret_cast<float4*>(p.part_o + slot * C::kD + d);
#pragma unroll
              for (int u = 0; u < kN / 4; ++u) part[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      if (real && copy == 0 && (!C::kSplit || t == 0)) {
        if (whole)
          a.lse[((long long)at.b * a.Hq + head) * a.n + i] = none ? -INFINITY : ((m + C::kLift) + lg2(l)) * kDecLn2;
        else
          p.part_ml[slot] = make_float2(none ? -INFINITY : m, l);
        // (a segment that begins here and goes on in blocks up to the last one named)
        if (tl == 0 && !whole && !head_cut)
          p.cuts[blockIdx.x] = make_int4(at.b, at.h, at.rg, (at.seg0 + tiles - 1) / at.part);
      }
      __syncwarp();
      if constexpr (C::kSplit) named_bar_sync(3, 256);  // both outputs have been read
      before += n;
      pos = at.seg0 + tiles;
      dec_next(p, at, tiles);
    }
    if (ok && lane == 0 && (!C::kSplit || t == 0)) {
      if ((warp & 3) == 0) info->n[pieces & 1] = 0;
      mbar_arrive(&info->q_full);
    }
    __syncwarp();
    tmem_wait_st();  // (behind an expired wait, weights may be on their way to memory that is given back below)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a cut segment, four columns a thread.  The block that began
// it has left where it is and how far it goes: to find that again, as
// cache_join_kernel does, took these grids 11 us and more, since none of their blocks
// fits beside the attention's.
template <class C, bool kF16>
__global__ void __launch_bounds__(kJoinThreads) cache_drafts_join_kernel(const __grid_constant__ DecParams p) {
  const CacheAttnParams& a = p.a;
  constexpr int kAtOnce = kJoinThreads / (C::kD / 4);  // rows
  const int c0 = blockIdx.y, r = blockIdx.x * kAtOnce + threadIdx.x / (C::kD / 4), d = threadIdx.x % (C::kD / 4) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
  const int4 cut = __ldcg(p.cuts + c0);
  const int row = cut.z * C::kRows + r;
  if (cut.x < 0 || r >= C::kRows || row >= p.rows) return;
  float top = -INFINITY, sum = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = c0; i <= cut.w; ++i) {
    const long long slot = (long long)(2 * i + (i == c0)) * C::kRows + r;
    const float2 ml = __ldcg(p.part_ml + slot);
    const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot * C::kD + d));
    const float m2 = fmaxf(top, ml.x), z = m2 == -INFINITY ? 0.0f : m2;
    const float f = ex2(top - z), g = ex2(ml.x - z);
    top = m2;
    sum = fmaf(sum, f, ml.y * g);
    x.x = fmaf(x.x, f, y.x * g), x.y = fmaf(x.y, f, y.y * g), x.z = fmaf(x.z, f, y.z * g), x.w = fmaf(x.w, f, y.w * g);
  }
  dec_write<DraftJoin<C, kF16>>(a, cut.x, cut.y, row, d, x, top, sum);
}

}  // namespace fa
