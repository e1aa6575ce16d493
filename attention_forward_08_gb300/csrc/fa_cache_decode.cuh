// fa_cache_decode.cuh -- attention of few query rows over the 8-bit cache.
//
// Rows.  The R = n * group rows of a K/V head (row r: query row r / group,
// head r % group of the group) share every key and value that is read; a
// thread block takes up to 16 * kMT of them (a "row group").
//
// Mathematics.  S = Q K^T and O += P V on the tensor cores (m16n8k16, f16 in,
// fp32 out), with an online softmax in base 2.  Nothing is lost on the way to
// f16: stored values of both kinds are f16 numbers, and a bf16 query row is
// scaled by a power of two so that its largest entry lies in [2^9, 2^10) (an
// entry 2^-34 below that is lost at most).  A block's k_scale multiplies its
// scores in fp32.  Its v_scale never touches a value: O is accumulated in the
// units of the current block and multiplied by the ratio of the two scales
// when a block with another one follows, together with the softmax's own
// rescaling.  P is rounded to f16 (2^-11; the output has 2^-8 or 2^-11), its
// sum is not.
//
// Work.  Every warp runs on its own: it takes tiles of 32 tokens, TMA brings
// them into the warp's own ring, and running maximum, sum and output stay in
// the warp's registers, so that no barrier stands between two tiles.  The
// tiles of all (sequence, head, row group) segments form one line that is cut
// into equal parts, one for each thread block, wherever the cuts fall:
// sequences of any lengths load the machine evenly, and nothing is planned on
// the host.  A block that holds a whole segment writes the output; the parts
// of a cut segment go to the workspace and a second, small kernel joins them.
//
// Layout.  Neither product cares about the order of its summed index, nor
// about the order of the columns it produces: lane (g, t) takes the bytes
// 32t .. 32t+31 of key g (QK) and 16 bytes of one value row (PV) as they lie
// in memory, so that all shared-memory reads are 16 bytes wide and, with the
// 128-byte swizzle, free of conflicts; the matching permutation is applied to
// Q once, and undone by where O is written.
//
// Bound: memory; 2 * D bytes a token and K/V head, read once per row group.
#pragma once

#include <cuda.h>

#include "fa_cache_ops.cuh"
#include "fa_ptx.cuh"

namespace fa {

constexpr float kDecLn2 = 0.6931471805599453f;
constexpr float kDecLazy = 8.0f;  // the running maximum moves when it grows by more than 2^8: p stays below 2^8 in f16
constexpr long long kDecDrainCycles = 1LL << 33;

template <int kKind_, bool kF16_, int kD_, int kMT_>
struct DecCfg {
  static constexpr int kKind = kKind_;
  static constexpr bool kF16 = kF16_;  // type of q and o
  static constexpr int kD = kD_, kMT = kMT_;
  static constexpr int kTile = 32;  // tokens
  static constexpr int kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kCtas = kD == 256 ? 1 : 2;           // per SM
  static constexpr int kCols = kD >= 128 ? kD / 128 : 1;    // 128-byte column blocks of a row
  static constexpr int kRowBytes = kD >= 128 ? 128 : 64;    // of one column block
  static constexpr int kTileBytes = kTile * kD;             // K; V alike
  static constexpr int kStages = kD == 64 ? 4 : 3;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRows = 16 * kMT;
  static constexpr int kKSteps = kD / 16, kNTiles = kD / 8;
  static constexpr int kQBytes = kRows * kD * 2;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // The warps join through the ring's memory: kWarps x (rows x D fp32), then maxima and sums.
  static constexpr int kJoinBytes = kWarps * kRows * kD * 4;
  static constexpr int kBulk = kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes;
  static_assert(kD != 256 || kMT == 1, "32 rows of 256 columns do not fit the registers");
  static constexpr int kSmem = 1024 + kBulk + kQBytes + kWarps * kRows * 8 + kRows * 4 + kWarps * kStages * 8 + 128;
};

struct DecParams {
  CacheAttnParams a;
  int rows, row_groups;   // rows of a K/V head; groups of kRows
  int max_ctas;
  float* part_o;          // [2 * max_ctas, kRows, D]
  float2* part_ml;        // [2 * max_ctas, kRows]: maximum, sum
};

// ------------------------------------------------------------------ the line of tiles

struct DecSeq {
  int len, nq;
};
__device__ __forceinline__ DecSeq dec_seq(const CacheAttnParams& a, int b) {
  DecSeq s;
  const long long most = (long long)a.c.M * a.c.page;
  const int len = a.lens[b];
  s.len = len < 0 ? 0 : (int)min((long long)len, most);
  s.nq = a.n_q ? min(max(a.n_q[b], 0), a.n) : a.n;
  return s;
}

// Tokens that rows r0 .. r1-1 of a K/V head see: [lo, hi), empty as {0, 0}.
__device__ __forceinline__ int2 dec_span(const CacheAttnParams& a, const DecSeq& s, int r0, int r1) {
  const int i0 = r0 / a.group, i1 = min((r1 - 1) / a.group, s.nq - 1);
  if (i0 > i1) return make_int2(0, 0);
  const int p0 = s.len - s.nq + i0, p1 = s.len - s.nq + i1;
  const int hi = a.causal ? min(s.len, p1 + 1) : s.len;
  const int lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// Tiles of one segment: at least one, so that empty rows are written too.
template <class C>
__device__ __forceinline__ int dec_tiles(const DecParams& p, const DecSeq& s, int rg) {
  const int2 v = dec_span(p.a, s, rg * C::kRows, min(p.rows, (rg + 1) * C::kRows));
  return max(1, (v.y + C::kTile - 1) / C::kTile - v.x / C::kTile);
}
template <class C>
__device__ __forceinline__ long long dec_seq_tiles(const DecParams& p, int b) {  // all heads
  const DecSeq s = dec_seq(p.a, b);
  long long n = 0;
  for (int rg = 0; rg < p.row_groups; ++rg) n += dec_tiles<C>(p, s, rg);
  return n * p.a.c.H;
}

// Sum over the block of one value a thread; `tmp` holds one value a warp.
__device__ __forceinline__ long long block_sum(long long v, long long* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  long long s = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += tmp[w];
  __syncthreads();
  return s;
}

// Tiles before sequence `b` (all of them: b = B), by the whole block.
template <class C>
__device__ __forceinline__ long long dec_tiles_before(const DecParams& p, int b, long long* tmp) {
  long long n = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) n += dec_seq_tiles<C>(p, i);
  return block_sum(n, tmp);
}

// Thread blocks that share the line: all, or fewer when some would get less
// than two tiles a warp.
template <class C>
__device__ __forceinline__ int dec_ctas(const DecParams& p, long long total) {
  const long long want = (total + 2 * C::kWarps - 1) / (2 * C::kWarps);
  return (int)min((long long)p.max_ctas, max(1LL, want));
}
__device__ __forceinline__ long long dec_start(long long total, int ctas, int c) { return total * c / ctas; }

// ------------------------------------------------------------------ tensor-core pieces

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four stored bytes -> two f16x2 (bytes 0, 1 and bytes 2, 3), exact.  int8: a
// byte u = x + 128 in the low mantissa bits of 1024 is the number 1024 + u.
template <int kKind>
__device__ __forceinline__ void to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kKind == kKindE4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off), hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&ha);
    hi = *reinterpret_cast<uint32_t*>(&hb);
  }
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

// Output columns.  Value n of PV's column tile i is column dec_col(i, n).
template <class C>
__device__ __forceinline__ int dec_col(int i, int n) {
  if constexpr (C::kD == 64) return 8 * n + i;
  return 128 * (i >> 4) + 16 * n + (i & 15);
}

// ------------------------------------------------------------------ the kernel

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ DecParams p) {
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_q = smem + C::kBulk;
  float2* s_ml = reinterpret_cast<float2*>(s_q + C::kQBytes);             // [warp][row]
  float* s_rs = reinterpret_cast<float*>(s_ml + C::kWarps * C::kRows);    // [row]: 2^-(scaling of the query row)
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_rs + C::kRows);         // [warp][stage]
  long long* s_tmp = reinterpret_cast<long long*>(s_bar + C::kWarps * C::kStages);  // [4 warps], then the search
  float* s_join = reinterpret_cast<float*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
  uint64_t* bars = s_bar + warp * C::kStages;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + s, 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  uint32_t phases = 0;  // parity of each stage's next wait

  // This block's part of the line, and where it begins.
  const long long total = dec_tiles_before<C>(p, a.B, s_tmp);
  const int ctas = dec_ctas<C>(p, total);
  if ((int)blockIdx.x >= ctas) return;
  const long long t0 = dec_start(total, ctas, blockIdx.x), t1 = dec_start(total, ctas, blockIdx.x + 1);
  int b = 0;
  long long before = 0;  // tiles before sequence b
  for (int base = 0;; base += C::kThreads) {  // chunks of sequences, then inside the chunk
    const int i = base + tid;
    long long mine = i < a.B ? dec_seq_tiles<C>(p, i) : 0, upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) s_tmp[warp] = upto;
    if (tid == 0) s_tmp[4] = -1;
    __syncthreads();
    long long off = before, all = before;
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) off += s_tmp[w];
      all += s_tmp[w];
    }
    upto += off;
    if (mine > 0 && upto - mine <= t0 && t0 < upto) {
      s_tmp[4] = i;
      s_tmp[5] = upto - mine;
    }
    __syncthreads();
    const long long hit = s_tmp[4];
    if (hit >= 0) {
      b = (int)hit;
      before = s_tmp[5];
      break;
    }
    before = all;
    __syncthreads();
    if (base + C::kThreads >= a.B) return;  // not reached: t0 < total
  }

  const int sub = min(c.page, C::kTile), subs = C::kTile / sub, sub_log2 = min(c.page_log2, 5);
  DecSeq seq = dec_seq(a, b);
  if (blockIdx.x == 0 || before >= t0) {  // one block per sequence tells about lengths
    if (tid == 0) (void)checked_len(c, a.lens[b]);
  }
  long long seg0 = before;  // first tile of the current segment
  int h = 0, rg = 0;
  {  // advance to the segment of t0
    long long per_head = 0;
    for (int r = 0; r < p.row_groups; ++r) per_head += dec_tiles<C>(p, seq, r);
    h = (int)((t0 - seg0) / per_head);
    seg0 += h * per_head;
    while (seg0 + dec_tiles<C>(p, seq, rg) <= t0) seg0 += dec_tiles<C>(p, seq, rg++);
  }

  for (long long at = t0; at < t1;) {
    const int r0 = rg * C::kRows, r1 = min(p.rows, r0 + C::kRows);
    const int tiles = dec_tiles<C>(p, seq, rg);
    const int2 span = dec_span(a, seq, r0, r1);
    const int first_tile = span.x / C::kTile + (int)(at - seg0);
    const int n_tiles = (int)(min(t1, seg0 + tiles) - at);
    const bool whole = n_tiles == tiles;

    // This warp's tiles: first_tile + warp, + kWarps, ...  Lane l looks up the
    // sub-blocks (a block's part of a tile) of the tiles to come, 32 / subs
    // tiles at a time, and their scales.
    const int mine = n_tiles > warp ? (n_tiles - warp + C::kWarps - 1) / C::kWarps : 0;
    const int per_batch = 32 / subs;
    int look_blk = -1;
    float look_ks = 0.0f, look_vs = 0.0f;
    auto look_up = [&](int k0) {  // tiles k0 .. of this warp
      const int k = k0 + (lane >> (subs - 1));
      const int tok = (first_tile + warp + k * C::kWarps) * C::kTile + (lane & (subs - 1)) * sub;
      look_blk = -1;
      look_ks = look_vs = 0.0f;
      if (k < mine && tok < span.y && tok + sub > span.x) {
        look_blk = checked_block(c, c.table, c.table_stride, b, tok >> c.page_log2);
        if (look_blk >= 0) {
          look_ks = __ldg(c.k_scale + (long long)look_blk * c.H + h);
          look_vs = __ldg(c.v_scale + (long long)look_blk * c.H + h);
        }
      }
    };
    // Sub-block `u` of this warp's tile k: its block (-1: none), by shuffle.
    auto issue = [&](int k, int blk0, int blk1) {  // lane 0 only
      const int s = k % C::kStages;
      uint8_t* dst = ring + s * C::kStageBytes;
      const int boxes = (blk0 >= 0) + (subs == 2 && blk1 >= 0);
      if (boxes == 0) {
        mbar_arrive(bars + s);
        return;
      }
      mbar_arrive_expect_tx(bars + s, (uint32_t)(boxes * sub * C::kD * 2));
      const int row = ((first_tile + warp + k * C::kWarps) * C::kTile) & (c.page - 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int blk = u ? blk1 : blk0;
        if (u < subs && blk >= 0) {
          const int y = sub < C::kTile ? 0 : row;  // blocks shorter than a tile start inside it
#pragma unroll
          for (int col = 0; col < C::kCols; ++col) {
            uint8_t* d = dst + col * C::kTile * C::kRowBytes + u * sub * C::kRowBytes;
            tma_load_4d(d, &tk, bars + s, col * 128, y, h, blk);
            tma_load_4d(d + C::kTileBytes, &tv, bars + s, col * 128, y, h, blk);
          }
        }
      }
    };
    int looked = 0;  // the batch in the lanes begins at this tile
    look_up(0);
    int issued = 0;
    // The scales of tiles that were looked up in an earlier batch than the one
    // in the lanes: tiles are consumed in order, at most kStages behind.
    float ring_ks[C::kStages][2], ring_vs[C::kStages][2];
    int ring_ok[C::kStages];
    auto advance = [&]() {  // issue the next tile, by the whole warp
      if (issued - looked >= per_batch) {
        looked = issued;
        look_up(issued);
      }
      const int from = (issued - looked) * subs;
      const int b0 = __shfl_sync(0xFFFFFFFFu, look_blk, from);
      const int b1 = __shfl_sync(0xFFFFFFFFu, look_blk, from + subs - 1);
      const float k0 = __shfl_sync(0xFFFFFFFFu, look_ks, from), k1 = __shfl_sync(0xFFFFFFFFu, look_ks, from + subs - 1);
      const float v0 = __shfl_sync(0xFFFFFFFFu, look_vs, from), v1 = __shfl_sync(0xFFFFFFFFu, look_vs, from + subs - 1);
      if (lane == 0) issue(issued, b0, b1);
      // a ring kept in registers: the newest entry is last
#pragma unroll
      for (int s = 0; s + 1 < C::kStages; ++s) {
        ring_ks[s][0] = ring_ks[s + 1][0], ring_ks[s][1] = ring_ks[s + 1][1];
        ring_vs[s][0] = ring_vs[s + 1][0], ring_vs[s][1] = ring_vs[s + 1][1];
        ring_ok[s] = ring_ok[s + 1];
      }
      ring_ks[C::kStages - 1][0] = k0, ring_ks[C::kStages - 1][1] = k1;
      ring_vs[C::kStages - 1][0] = v0, ring_vs[C::kStages - 1][1] = v1;
      ring_ok[C::kStages - 1] = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
      ++issued;
    };
    auto advance_none = [&]() {  // past the last tile: the register ring moves on
#pragma unroll
      for (int s = 0; s + 1 < C::kStages; ++s) {
        ring_ks[s][0] = ring_ks[s + 1][0], ring_ks[s][1] = ring_ks[s + 1][1];
        ring_vs[s][0] = ring_vs[s + 1][0], ring_vs[s][1] = ring_vs[s + 1][1];
        ring_ok[s] = ring_ok[s + 1];
      }
    };
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
      if (s < mine)
        advance();
      else
        advance_none();
    }

    // The query rows, scaled to f16 and laid out as the tensor core's operand.
    for (int r = warp; r < C::kRows; r += C::kWarps) {
      constexpr int kE = C::kD / 32;  // elements a lane
      float f[kE];
      const int row = r0 + r, i = row / a.group, head = h * a.group + row % a.group;
      const bool in = row < r1 && i < seq.nq;
      float top = 0.0f;
      if (in) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + b * a.qs[0] + head * a.qs[1] + i * a.qs[2] + lane * kE;
#pragma unroll
        for (int e = 0; e < kE; ++e) f[e] = half_bits_to_f32<C::kF16>(q[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) f[e] = 0.0f;
      }
      float up = 1.0f;
      if constexpr (!C::kF16) {
#pragma unroll
        for (int e = 0; e < kE; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // 2^(9 - exponent), kept inside the normal numbers
        const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -110), 127);
        up = __uint_as_float((uint32_t)(9 - ex + 127) << 23);
        if (lane == 0) s_rs[r] = __uint_as_float((uint32_t)(ex - 9 + 127) << 23);
      } else if (lane == 0) {
        s_rs[r] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const int d = lane * kE + e;
        const int tt = C::kD == 64 ? d / 16 : (d & 127) / 32;
        const int kk = C::kD == 64 ? (d & 15) / 4 : 8 * (d / 128) + (d & 31) / 4;
        const int reg = ((d & 3) / 2) * 2 + ((r & 15) >> 3);
        const uint32_t at2 = (uint32_t)((((r >> 4) * C::kKSteps + kk) * 32 + (r & 7) * 4 + tt) * 16 + reg * 4);
        *reinterpret_cast<uint32_t*>(s_q + at2) = pack_f16x2(f[e] * up, f[e + 1] * up);
      }
    }
    __syncthreads();

    float o[C::kMT][C::kNTiles][4];
    float m[C::kMT][2], l[C::kMT][2], rs[C::kMT][2];
    int hi_row[C::kMT][2], lo_row[C::kMT][2];  // the tokens that this lane's two rows see
    float vs_unit = 1.0f;                      // O is in units of this scale
#pragma unroll
    for (int mt = 0; mt < C::kMT; ++mt) {
#pragma unroll
      for (int i = 0; i < C::kNTiles; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[mt][x] = -INFINITY;
        l[mt][x] = 0.0f;
        const int r = mt * 16 + g + 8 * x, row = r0 + r;
        rs[mt][x] = s_rs[r];
        const int2 v = row < r1 ? dec_span(a, seq, row, row + 1) : make_int2(0, 0);
        lo_row[mt][x] = v.x;
        hi_row[mt][x] = v.y;
      }
    }

    int k = 0;
    bool dead = false;
    for (; k < mine; ++k) {
      const int s = k % C::kStages;
      {
        const uint32_t par = (phases >> s) & 1u;
        bool ok = mbar_try_wait(bars + s, par);
        const long long begin = clock64_now();
        while (!ok) {
          ok = mbar_try_wait(bars + s, par);
          if (!ok && clock64_now() - begin > a.timeout_cycles) break;
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          dead = true;
          if (lane == 0) atomicOr(c.status, kStatusTimeout);
          break;
        }
        phases ^= 1u << s;
      }
      const uint32_t tile_k = smem_u32(ring + s * C::kStageBytes), tile_v = tile_k + C::kTileBytes;
      const int tok0 = (first_tile + warp + k * C::kWarps) * C::kTile;
      const float ks0 = ring_ks[0][0], ks1 = ring_ks[0][1], vs0 = ring_vs[0][0], vs1 = ring_vs[0][1];
      const int ok_blk = ring_ok[0];
      // Whole: every row of the warp sees every token, and every block is there.
      bool full = ok_blk == 3;
#pragma unroll
      for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) full = full && lo_row[mt][x] <= tok0 && tok0 + C::kTile <= hi_row[mt][x];
      full = __all_sync(0xFFFFFFFFu, full);

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

      // Scores in base 2; masks; the running maximum.
      uint32_t pa[C::kMT][2][4];  // P as the A operand of the two k-steps of PV
      float grow = 0.0f;          // rescaling wanted by some row
      float mx[C::kMT][2];
#pragma unroll
      for (int mt = 0; mt < C::kMT; ++mt) {
        const float f00 = ks0 * rs[mt][0], f01 = ks0 * rs[mt][1], f10 = ks1 * rs[mt][0], f11 = ks1 * rs[mt][1];
        if (a.cap_out > 0.0f) {  // cap * tanh(x) = cap * (1 - 2 / (2^(2 x log2 e) + 1))
          const float ci = a.cap_in * 2.8853900817779268f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f = (j < 2 ? (e < 2 ? f00 : f01) : (e < 2 ? f10 : f11)) * ci;
              sc[mt][j][e] = fmaf(-2.0f * a.cap_out, rcp_approx(ex2(sc[mt][j][e] * f) + 1.0f), a.cap_out);
            }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[mt][j][e] *= (j < 2 ? (e < 2 ? f00 : f01) : (e < 2 ? f10 : f11)) * a.scale_log2;
        }
        if (!full) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = tok0 + j * 8 + 2 * t + (e & 1), x = e >> 1;
              if (tok < lo_row[mt][x] || tok >= hi_row[mt][x] || !(ok_blk & (j < 2 ? 1 : 2)))
                sc[mt][j][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(fmaxf(sc[mt][0][2 * x], sc[mt][0][2 * x + 1]), fmaxf(sc[mt][1][2 * x], sc[mt][1][2 * x + 1]));
          v = fmaxf(v, fmaxf(fmaxf(sc[mt][2][2 * x], sc[mt][2][2 * x + 1]),
                             fmaxf(sc[mt][3][2 * x], sc[mt][3][2 * x + 1])));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
          mx[mt][x] = v;
          if (v > m[mt][x] + kDecLazy) grow = 1.0f;
        }
      }
      const bool move = __any_sync(0xFFFFFFFFu, grow > 0.0f);
      // Two halves of 16 tokens, each inside one block: O in that block's units.
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float vs = half ? vs1 : vs0;
        const float unit = vs > 0.0f ? vs : vs_unit;  // a zero scale: stored values are zeros, or do not matter
        const bool first = half == 0 && move;
        if (first || unit != vs_unit) {
          // (finite, so that an output of 0 stays 0)
          const float by_unit = unit != vs_unit ? fminf(__fdividef(vs_unit, unit), 1e38f) : 1.0f;
#pragma unroll
          for (int mt = 0; mt < C::kMT; ++mt) {
            float al[2] = {by_unit, by_unit};
            if (first) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float m2 = fmaxf(m[mt][x], mx[mt][x]);
                const float f = m2 == -INFINITY ? 1.0f : ex2(m[mt][x] - m2);
                l[mt][x] *= f;
                al[x] *= f;
                m[mt][x] = m2;
              }
            }
#pragma unroll
            for (int i = 0; i < C::kNTiles; ++i) {
              o[mt][i][0] *= al[0], o[mt][i][1] *= al[0];
              o[mt][i][2] *= al[1], o[mt][i][3] *= al[1];
            }
          }
          vs_unit = unit;
        }
#pragma unroll
        for (int mt = 0; mt < C::kMT; ++mt) {
          const float m0 = m[mt][0] == -INFINITY ? 0.0f : m[mt][0], m1 = m[mt][1] == -INFINITY ? 0.0f : m[mt][1];
          float pv[2][4];
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[jj][e] = ex2(sc[mt][2 * half + jj][e] - (e < 2 ? m0 : m1));
              l[mt][e >> 1] += pv[jj][e];
            }
          }
          const float z = vs > 0.0f ? 1.0f : 0.0f;
          pa[mt][half][0] = pack_f16x2(pv[0][0] * z, pv[0][1] * z);
          pa[mt][half][1] = pack_f16x2(pv[0][2] * z, pv[0][3] * z);
          pa[mt][half][2] = pack_f16x2(pv[1][0] * z, pv[1][1] * z);
          pa[mt][half][3] = pack_f16x2(pv[1][2] * z, pv[1][3] * z);
        }
        // O += P V over these 16 tokens: lane t takes tokens 2t, 2t+1, 2t+8, 2t+9
        const int row = half * 16 + 2 * t;
        uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
        if (!full) {  // bytes that no row may see could be NaN
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = tok0 + row + (e & 1) + 8 * (e >> 1);
            if (tok < span.x || tok >= span.y || !(ok_blk & (half ? 2 : 1))) keep[e] = 0u;
          }
        }
        if constexpr (C::kD == 64) {
          uint2 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = row + (e & 1) + 8 * (e >> 1);
            v[e] = lds64(dec_unit<C>(tile_v, r, g >> 1) + (g & 1) * 8);
            v[e].x &= keep[e], v[e].y &= keep[e];
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t x0 = w ? v[0].y : v[0].x, x1 = w ? v[1].y : v[1].x, x2 = w ? v[2].y : v[2].x,
                           x3 = w ? v[3].y : v[3].x;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t a0, a1, b0, b1;
              to_f16x4<C::kKind>(__byte_perm(x0, x1, hh ? 0x7362 : 0x5140), a0, a1);
              to_f16x4<C::kKind>(__byte_perm(x2, x3, hh ? 0x7362 : 0x5140), b0, b1);
#pragma unroll
              for (int mt = 0; mt < C::kMT; ++mt) {
                mma_f16(o[mt][4 * w + 2 * hh], pa[mt][half], a0, b0);
                mma_f16(o[mt][4 * w + 2 * hh + 1], pa[mt][half], a1, b1);
              }
            }
          }
        } else {
#pragma unroll
          for (int col = 0; col < C::kCols; ++col) {
            const uint32_t base = tile_v + col * C::kTile * 128;
            uint32_t v[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 x = lds128(dec_unit<C>(base, row + (e & 1) + 8 * (e >> 1), g));
              v[e][0] = x.x & keep[e], v[e][1] = x.y & keep[e], v[e][2] = x.z & keep[e], v[e][3] = x.w & keep[e];
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                uint32_t a0, a1, b0, b1;
                to_f16x4<C::kKind>(__byte_perm(v[0][w], v[1][w], hh ? 0x7362 : 0x5140), a0, a1);
                to_f16x4<C::kKind>(__byte_perm(v[2][w], v[3][w], hh ? 0x7362 : 0x5140), b0, b1);
#pragma unroll
                for (int mt = 0; mt < C::kMT; ++mt) {
                  mma_f16(o[mt][16 * col + 4 * w + 2 * hh], pa[mt][half], a0, b0);
                  mma_f16(o[mt][16 * col + 4 * w + 2 * hh + 1], pa[mt][half], a1, b1);
                }
              }
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage: it may be filled again
      if (issued < mine)
        advance();
      else
        advance_none();
    }
    // Join the warps: O in units of 1, at the block's common maximum.
#pragma unroll
    for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 2);
        if (t == 0) s_ml[warp * C::kRows + mt * 16 + g + 8 * x] = make_float2(m[mt][x], l[mt][x]);
      }
    // Every warp is done with its ring, and the maxima are there.  After an
    // expired wait the block ends, once its copies in flight have landed (a
    // bounded wait again).
    if (__syncthreads_or(dead)) {
      for (; k < issued; ++k) {
        const int s = k % C::kStages;
        const long long begin = clock64_now();
        while (!mbar_try_wait(bars + s, (phases >> s) & 1u) && clock64_now() - begin < kDecDrainCycles) {
        }
        phases ^= 1u << s;
      }
      return;
    }
#pragma unroll
    for (int mt = 0; mt < C::kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + g + 8 * x;
        float top = -INFINITY;
        for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, s_ml[w * C::kRows + r].x);
        const float f = m[mt][x] == -INFINITY ? 0.0f : ex2(m[mt][x] - top) * vs_unit;
        float* dst = s_join + (long long)(warp * C::kRows + r) * C::kD;
#pragma unroll
        for (int i = 0; i < C::kNTiles; ++i) {
          dst[dec_col<C>(i, 2 * t)] = o[mt][i][2 * x] * f;
          dst[dec_col<C>(i, 2 * t + 1)] = o[mt][i][2 * x + 1] * f;
        }
      }
    __syncthreads();
    const bool head_cut = at > seg0;
    const int slot = 2 * blockIdx.x + (head_cut ? 0 : 1);
    for (int v = tid; v < C::kRows * (C::kD / 8); v += C::kThreads) {
      const int r = v / (C::kD / 8), d = (v % (C::kD / 8)) * 8;
      if (r0 + r >= r1) break;
      float top = -INFINITY, sum = 0.0f, x[8] = {};
      for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, s_ml[w * C::kRows + r].x);
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 ml = s_ml[w * C::kRows + r];
        if (ml.x > -INFINITY) sum += ml.y * ex2(ml.x - top);
        const float4* q = reinterpret_cast<const float4*>(s_join + (long long)(w * C::kRows + r) * C::kD + d);
        const float4 y0 = q[0], y1 = q[1];
        x[0] += y0.x, x[1] += y0.y, x[2] += y0.z, x[3] += y0.w;
        x[4] += y1.x, x[5] += y1.y, x[6] += y1.z, x[7] += y1.w;
      }
      if (whole) {
        const int row = r0 + r, i = row / a.group, head = h * a.group + row % a.group;
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        uint4 y;
        uint32_t* u = &y.x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[e] = C::kF16 ? pack_f16x2(x[2 * e] * inv, x[2 * e + 1] * inv) : pack_bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + b * a.os[0] + head * a.os[1] + i * a.os[2] + d) = y;
        if (d == 0)
          a.lse[((long long)b * a.Hq + head) * a.n + i] = sum > 0.0f ? (top + log2f(sum)) * kDecLn2 : -INFINITY;
      } else {
        float4* q = reinterpret_cast<float4*>(p.part_o + ((long long)slot * C::kRows + r) * C::kD + d);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (d == 0) p.part_ml[(long long)slot * C::kRows + r] = make_float2(top, sum);
      }
    }
    fence_proxy_async_smem();  // what was written into the ring's memory goes before the next copies into it
    __syncthreads();           // the ring's memory and the maxima are free again
    at = min(t1, seg0 + tiles);
    seg0 += tiles;
    if (++rg == p.row_groups) {
      rg = 0;
      if (++h == c.H) {
        h = 0;
        if (++b < a.B) {
          seq = dec_seq(a, b);
          if (tid == 0) (void)checked_len(c, a.lens[b]);
        }
      }
    }
  }
}

// Joins the parts of segments that lie in more than one thread block.  One
// block per (head, sequence); rows of all row groups.
template <class C>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ DecParams p) {
  const CacheAttnParams& a = p.a;
  __shared__ long long tmp[4];
  const int rg = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const long long before = dec_tiles_before<C>(p, b, tmp), total = dec_tiles_before<C>(p, a.B, tmp);
  const DecSeq seq = dec_seq(a, b);
  long long per_head = 0, u0 = 0;
  for (int r = 0; r < p.row_groups; ++r) {
    const int n = dec_tiles<C>(p, seq, r);
    if (r < rg) u0 += n;
    per_head += n;
  }
  u0 += before + h * per_head;
  const long long u1 = u0 + dec_tiles<C>(p, seq, rg);
  const int ctas = dec_ctas<C>(p, total);
  auto owner = [&](long long u) {
    int c = (int)min((long long)ctas - 1, u * ctas / total);
    while (c > 0 && dec_start(total, ctas, c) > u) --c;
    while (c + 1 < ctas && dec_start(total, ctas, c + 1) <= u) ++c;
    return c;
  };
  const int c0 = owner(u0), c1 = owner(u1 - 1);
  if (c0 == c1) return;
  const int r0 = rg * C::kRows, r1 = min(p.rows, r0 + C::kRows);
  for (int v = tid; v < C::kRows * (C::kD / 8); v += 128) {
    const int r = v / (C::kD / 8), d = (v % (C::kD / 8)) * 8;
    if (r0 + r >= r1) break;
    float top = -INFINITY, sum = 0.0f, x[8] = {};
    for (int c = c0; c <= c1; ++c) top = fmaxf(top, p.part_ml[(long long)(2 * c + (c == c0)) * C::kRows + r].x);
    for (int c = c0; c <= c1; ++c) {
      const long long slot = (long long)(2 * c + (c == c0)) * C::kRows + r;
      const float2 ml = p.part_ml[slot];
      if (ml.x == -INFINITY) continue;
      const float f = ex2(ml.x - top);
      sum = fmaf(ml.y, f, sum);
      const float4* q = reinterpret_cast<const float4*>(p.part_o + slot * C::kD + d);
      const float4 y0 = q[0], y1 = q[1];
      x[0] = fmaf(y0.x, f, x[0]), x[1] = fmaf(y0.y, f, x[1]), x[2] = fmaf(y0.z, f, x[2]), x[3] = fmaf(y0.w, f, x[3]);
      x[4] = fmaf(y1.x, f, x[4]), x[5] = fmaf(y1.y, f, x[5]), x[6] = fmaf(y1.z, f, x[6]), x[7] = fmaf(y1.w, f, x[7]);
    }
    const int row = r0 + r, i = row / a.group, head = h * a.group + row % a.group;
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    uint4 y;
    uint32_t* u = &y.x;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = C::kF16 ? pack_f16x2(x[2 * e] * inv, x[2 * e + 1] * inv) : pack_bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + b * a.os[0] + head * a.os[1] + i * a.os[2] + d) = y;
    if (d == 0) a.lse[((long long)b * a.Hq + head) * a.n + i] = sum > 0.0f ? (top + log2f(sum)) * kDecLn2 : -INFINITY;
  }
}

}  // namespace fa
