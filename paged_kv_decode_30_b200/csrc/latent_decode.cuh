// Latent decode attention in the absorbed form on the 5th-generation tensor
// cores: q = [q_c | q_r] of every head against the latent rows [c | r] of a
// sequence's pages, values c.
//
// A latent row is key and value at once and serves all heads, so the packed
// query rows (q_len x heads, NT of them per CTA) share every byte read. Per
// tile of 128 tokens, tokens are the M dimension of both products:
//   S^T [128 tokens, NT] = C Q_c^T + R Q_r^T   (K: R + 64 elements)
//   O^T [R dims, NT]    += C^T P^T             (K: 128 tokens; R / 128 blocks)
// The tile C enters both from the same shared memory: K-major for S^T and
// MN-major for O^T. O^T stays in TMEM over a sequence; NT is bounded by TMEM
// (512 columns) and by shared memory (Q and one to two tiles).
//
// Bounds: a tile brings 128 x (2R + 2 rope) bytes (FP8: R + 2 rope) for 2 x
// 128 x NT x (2R + rope) operations. At R = 512 and 64 rows or fewer HBM is
// the bound; with more rows several CTAs take the same tiles (row tiles), the
// later ones from L2, and the matrix products and the shared memory they are
// fed from become the bound.
//
// Schedule: the tiles of all sequences form one line, with a gap for what a change
// of sequence takes, cut into equal ranges for `teams` teams; the CTAs of a team
// take the same range for one row tile each, at the same time, so that HBM sees
// each tile once. A sequence that lies in one range is finished by its CTA; one
// that is cut leaves partial results that a second kernel joins. The ranges follow from kv_lens by a scan
// that every CTA makes for itself: no counters, no atomics, one order of sums.
//
// FP8 rows are e4m3 codes with a power-of-two scale 2^e a row. Codes go to the
// matrix instructions as they are (kind::f8f6f4); a bf16 query row times a
// power of two is the exact sum of two e4m3 terms [hi; 16 lo]; the rotated
// parts are bf16 products into columns of their own. With x_j the score
// (log2 units) the weight is w_j = 2^(x_j + e_j - m), m a reference that follows
// x + e, split in two e4m3 terms as well; the normaliser adds w_j 2^-e_j.
//
// Two e4m3 terms hold a weight to 2^-8 of itself or to 2^-14, whichever is coarser.
// A long flat tail below a peak can consist of weights under that step (131 k tokens
// that share a fifth of the probability, the rest on one: all of them became zero,
// a fifth of the output), so m follows the scores down as well as up. Per row a
// credit counts how many tiles' worth of such errors, 128 x 2^-14 = 2^-7 each, the
// weights have paid for: a tile whose largest weight is w adds w / 4 and takes one away
// (2^14 w, if all its weights are below the step). Before it is used up m moves to the
// tile at hand. What the step rounds off is then at most 2^-7 / 4 = 2^-9 of a row's sum
// of weights, whatever its length, and a row moves only where its weights stay low.
// (Normally distributed scores, 2.5 in log2 units, rows of different scales: a group of
// eight rows moves in 20% of 40 tiles instead of 12% with a running maximum, in 11% of
// 400 instead of 2%; 2 in log2 units: 5% of 40 instead of 2%.) Such scores take 56.8 us
// instead of 51.9 for two sequences of 110 k tokens, 64 heads, and 61.4 instead of 57.2
// for 72 of up to 6000 tokens, 48 rows; with w / 2 instead of w / 4, 55.2 and 60.8; with
// HEAD 4 instead of 5, 58.4 and 62.9; with the largest weights known to a factor of 4
// only, as bits that take one reduction instead of eight, 57.3 and 61.9.
//
// Roles (warps): 0 TMA producer, 1 S^T issuer, 2 O^T issuer, 3 schedule,
// 4.. softmax (groups of four warps, a thread = a token of S^T = an element of
// each O^T block, with 8 query rows, 16 where 8 would take too many warps).
// Every wait is bounded.
#pragma once

#include "pda_device.cuh"
#include "split_tma.cuh"  // MMA issue, instruction descriptors, TMA loads, e4m3 splits
#include "tcgen05.cuh"

namespace pda {

struct LatentArgs {
  const uint16_t* q;  // bf16 [B, M, R + rope_dim], M = q_len * H
  const uint8_t* latent_pages;
  const uint16_t* rope_pages;
  const uint8_t* scales;
  const int32_t* page_table;
  const int32_t* kv_lens;
  uint16_t* out;  // bf16 [B, M, R]
  float* lse;     // [B, M] or null
  int* err;
  float* o_part;    // [teams * row_tiles * 2][NT][R]
  float* lse_part;  // [teams * row_tiles * 2][NT]
  int2* cut;        // [teams]: (sequence, last team) of the cut sequence that starts in the team
  int B, Lq, H, M, rope_dim, page_size, log2_page, max_pages, num_pages, causal_offset, window;
  int teams, row_tiles, item_cost;
  float scale_log2;
};

constexpr int kTile = 128;

// Keys [lo, hi) that query row i of a sequence of L keys sees.
__device__ __forceinline__ void latent_visible(const LatentArgs& a, int L, int i, int& lo, int& hi) {
  long long pos = (long long)L - 1;
  if (a.causal_offset >= 0) pos = (long long)a.causal_offset + i;
  else if (a.causal_offset == -2) pos = (long long)L - a.Lq + i;
  const long long h = a.causal_offset != -1 ? pos + 1 : (long long)L;
  const long long l = a.window > 0 ? pos - a.window + 1 : 0;
  hi = (int)(h < 0 ? 0 : (h > L ? L : h));
  lo = (int)(l < 0 ? 0 : (l > L ? L : l));
}

// A length from kv_lens, held to what the page table covers.
__device__ __forceinline__ int latent_len(const LatentArgs& a, int kv_len) {
  return min(max(kv_len, 0), a.max_pages << a.log2_page);
}

// First tile and number of tiles that any query row of the sequence sees.
__device__ __forceinline__ void latent_tiles(const LatentArgs& a, int L, int& first, int& n) {
  int lo, hi, x;
  latent_visible(a, L, 0, lo, x);
  latent_visible(a, L, a.Lq - 1, x, hi);
  first = lo / kTile;
  n = hi > lo ? (hi + kTile - 1) / kTile - first : 0;
}

// A sequence's share of the line: its tiles, and one unit if it has none, so
// that some CTA writes its rows.
__device__ __forceinline__ int latent_weight(const LatentArgs& a, int kv_len) {
  int first, n;
  latent_tiles(a, latent_len(a, kv_len), first, n);
  return max(n, 1);
}

struct LatentItem {
  int b;              // < 0: no more items
  int L, first, n;    // kv length, first tile, tiles
  int part;           // slot of the partial results, -1: the sequence is finished here
  int lo_u, hi_u;     // keys that some row of the row tile sees
  int lo_x, hi_x;     // keys that all rows of it see
  int pad[3];
};

// The sequences' shares of the line, as a warp holds them. Up to 128 sequences
// the schedule warp has them to itself, four consecutive ones a lane; more: every
// warp adds up one chunk, and the schedule warp looks into the chunks it needs.
struct LatentShares {
  static constexpr int K = 4;
  bool few;
  int chunk, sum;          // sequences a warp; this lane's sum
  int lens[K], wts[K];
};

template <int WARPS>
__device__ __forceinline__ void latent_load_shares(const LatentArgs& a, LatentShares& sh, int warp, int lane,
                                                   bool schedules) {
  sh.few = a.B <= 32 * LatentShares::K;
  sh.chunk = (a.B + WARPS - 1) / WARPS;
  sh.sum = 0;  // (the host refuses calls of 2^31 tiles or more)
#pragma unroll
  for (int k = 0; k < LatentShares::K; ++k) sh.lens[k] = sh.wts[k] = 0;
  auto share_of = [&](int L) {
    if (blockIdx.x == 0 && (L < 0 || L > (a.max_pages << a.log2_page))) record_error_at(a.err, kErrBadPage);
    return latent_weight(a, L);
  };
  if (!sh.few) {
    for (int b = warp * sh.chunk + lane; b < min(a.B, (warp + 1) * sh.chunk); b += 32)
      sh.sum += share_of(__ldg(a.kv_lens + b));
  } else if (schedules) {
#pragma unroll
    for (int k = 0; k < LatentShares::K; ++k)
      if (lane * LatentShares::K + k < a.B) sh.lens[k] = __ldg(a.kv_lens + lane * LatentShares::K + k);
#pragma unroll
    for (int k = 0; k < LatentShares::K; ++k) {
      if (lane * LatentShares::K + k < a.B) sh.wts[k] = share_of(sh.lens[k]);
      sh.sum += sh.wts[k];
    }
  }
}

// Walks the line (the whole schedule warp, after the block's barrier; sums: the
// warps' chunk sums): its length, team `team`'s range [s, e) of it (a line shorter
// than the number of teams leaves the last ones idle, so that no range is empty),
// and publish(b, kv_len, t0, t1, whole, goes_on) for every sequence that overlaps
// the range: its tiles [t0, t1), whether they are all, whether it goes on behind
// the range. Stops once ok is false. Returns the cut sequence that starts in the
// range (-1: none) and the team of its last tile.
template <int WARPS, typename F>
__device__ __forceinline__ int2 latent_schedule(const LatentArgs& a, const LatentShares& sh, const int* sums,
                                                int team, int lane, const bool& ok, F publish) {
  constexpr unsigned FULL = 0xFFFFFFFFu;
  constexpr int K = LatentShares::K;
  const int own_sum = sh.few ? sh.sum : lane < WARPS ? sums[lane] : 0;
  int upto = own_sum;  // up to and with this lane's sequences, or chunk `lane`
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += y;
  }
  // A sequence after a range's first costs what item_cost tiles cost (less where a
  // range is short): the line has gaps of that length between the sequences.
  const int tiles = __shfl_sync(FULL, upto, 31);
  const int gap = min(a.item_cost, max(tiles / a.teams - 1, 0)), total = tiles + gap * (a.B - 1);
  // the first `more` teams take share + 1 units, the rest share
  const int teams = min(a.teams, total), share = total / teams, more = total - share * teams;
  const int s = team < teams ? share * team + min(team, more) : total;
  const int e = team < teams ? s + share + (team < more ? 1 : 0) : 0;
  int cut_b = -1, cut_last = 0;  // the cut sequence that starts here and the unit of its last tile
  auto found = [&](int b, int len, int begin, int w) {
    const int t0 = max(s, begin) - begin, t1 = min(e, begin + w) - begin;
    const bool whole = t0 == 0 && t1 == w;
    if (t0 == 0 && !whole) {
      cut_b = b;
      cut_last = begin + w - 1;
    }
    publish(b, len, t0, t1, whole, begin + w > e);
  };
  if (sh.few) {
    int begin[K], hits = 0;
    begin[0] = upto - own_sum + gap * lane * K;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k > 0) begin[k] = begin[k - 1] + sh.wts[k - 1] + gap;
      if (sh.wts[k] > 0 && begin[k] < e && begin[k] + sh.wts[k] > s && s < e) hits |= 1 << k;
    }
    unsigned lanes = __ballot_sync(FULL, hits != 0);
    while (lanes && ok) {
      const int src = __ffs(lanes) - 1, mask = __shfl_sync(FULL, hits, src);
      lanes &= lanes - 1;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok && (mask >> k & 1))
          found(src * K + k, __shfl_sync(FULL, sh.lens[k], src), __shfl_sync(FULL, begin[k], src),
                __shfl_sync(FULL, sh.wts[k], src));
    }
  } else {
    // the chunk that holds unit s, then on to the range's end
    const int end = upto + gap * (min(a.B, (lane + 1) * sh.chunk) - 1);
    int w = __ffs(__ballot_sync(FULL, s < e && end > s)) - 1;
    int at = __shfl_sync(FULL, upto - own_sum, max(w, 0));  // tiles before the sequences looked at next
    for (; w >= 0 && w < WARPS && ok && at + gap * (w * sh.chunk) < e; ++w) {
      const int b1 = min(a.B, (w + 1) * sh.chunk);
      for (int b0 = w * sh.chunk; b0 < b1 && ok && at + gap * b0 < e; b0 += 32) {
        const int len = b0 + lane < b1 ? __ldg(a.kv_lens + b0 + lane) : 0;
        const int wt = b0 + lane < b1 ? latent_weight(a, len) : 0;
        int inc = wt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULL, inc, o);
          if (lane >= o) inc += y;
        }
        const int begin = at + inc - wt + gap * (b0 + lane);
        unsigned hit = __ballot_sync(FULL, wt > 0 && begin < e && begin + wt > s);
        while (hit && ok) {
          const int src = __ffs(hit) - 1;
          hit &= hit - 1;
          found(b0 + src, __shfl_sync(FULL, len, src), __shfl_sync(FULL, begin, src), __shfl_sync(FULL, wt, src));
        }
        at += __shfl_sync(FULL, inc, 31);
      }
    }
  }
  if (ok) publish(-1, 0, 0, 0, false, false);
  const int wide = (share + 1) * more;
  return make_int2(cut_b, cut_last < wide ? cut_last / (share + 1) : more + (cut_last - wide) / share);
}

// Item d: tiles [t0, t1) of sequence b for the row tile of query rows i0 .. i1;
// slot: where its partial results go if they are not all (a team's range holds at
// most one cut piece that ends in it, its first, and one that goes on, its last).
__device__ __forceinline__ void latent_fill(const LatentArgs& a, LatentItem& d, int b, int kv_len, int t0, int t1,
                                            bool whole, int slot, int i0, int i1) {
  const int L = latent_len(a, kv_len);
  int first, n;
  latent_tiles(a, L, first, n);
  d.b = b;
  d.L = L;
  d.first = first + t0;
  d.n = n == 0 ? 0 : t1 - t0;
  d.part = whole ? -1 : slot;
  latent_visible(a, L, i0, d.lo_u, d.hi_x);
  latent_visible(a, L, i1, d.lo_x, d.hi_u);
}

template <int R_, bool FP8_, int NT_>
struct LatentCfg {
  static constexpr int R = R_, NT = NT_, NB = R / 128;
  static constexpr bool FP8 = FP8_;
  static constexpr int HALF = kTile * 128;              // a 128-byte column of a tile
  // A tile lies in shared memory as [8-token group][128-byte column][8 tokens]
  // [128 bytes], the order in which one TMA box writes a run of tokens. It comes
  // in units of two 128-byte columns of 128 tokens with barriers of their own, so
  // that S^T starts on what is there, and the ring need not hold whole tiles. (FP8
  // in whole rows of 64 tokens, two tiles of two such units: 62.0 us instead of 59.3 for two
  // sequences of 110 k tokens, 64 heads.)
  static constexpr int COLS_U = 2;                      // 128-byte columns of a unit
  static constexpr int GS = COLS_U * 1024;              // bytes of an 8-token group
  static constexpr int UPT = FP8 ? NB / 2 : NB;         // units of a tile
  static constexpr int BPU = NB / UPT;                  // 128-element blocks of a unit
  static constexpr int BLK = kTile / 8 * GS;
  static constexpr int N1 = FP8 ? 2 * NT : NT;          // S^T columns of the latent product
  static constexpr int N2 = FP8 ? 2 * NT : NT;          // O^T columns of a block
  static constexpr int SN = FP8 ? 3 * NT : NT;          // S^T columns (FP8: rotated part apart)
  // Q operand, K-major: FP8 per block [hi; lo] rows of 128 codes, bf16 per 64
  // elements NT rows; then the rotated part, NT rows of 64 bf16.
  static constexpr int Q_BLK = FP8 ? N1 * 128 : 2 * NT * 128;
  static constexpr int Q_ROPE = NB * Q_BLK;
  static constexpr int Q_BYTES = Q_ROPE + NT * 128;
  static constexpr int P_ROW = 2 * NT;                  // bytes of a token's weights
  static constexpr int P_BYTES = kTile * P_ROW;
  static constexpr uint32_t P_SWIZZLE = P_ROW == 128 ? kSw128 : P_ROW == 64 ? kSw64 : kSw32;
  // Shared memory is Q, weights, the rotated parts' slots and as many units of
  // latents as fit. The widest bf16 case has room for one tile only
  // if the weights take the place of the rotated parts, which the S^T product
  // has read by then.
  static constexpr bool OVERLAY = !FP8 && NT == 64 && R == 512;
  static constexpr int P_BUFS = (OVERLAY || (NT == 32 && R == 512)) ? 1 : 2;
  static constexpr int R_SLOTS = FP8 && !(NT == 32 && R == 512) ? 2 : 1;
  static constexpr int ROPE_SLOT = HALF;
  static constexpr int STATE = 20 * NT * 4 + 1024 + (FP8 ? 8 * NT * 4 : 0);
  static constexpr int FREE = 227 * 1024 - 1024 - STATE - Q_BYTES - (OVERLAY ? 0 : P_BUFS * P_BYTES) -
                              R_SLOTS * ROPE_SLOT;
  static constexpr int SLOTS = FREE / BLK < 3 * UPT ? FREE / BLK : 3 * UPT;
  static constexpr int OFF_BLK = 0;
  static constexpr int OFF_ROPE = OFF_BLK + SLOTS * BLK;
  static constexpr int OFF_Q = OFF_ROPE + R_SLOTS * ROPE_SLOT;
  static constexpr int OFF_P = OVERLAY ? OFF_ROPE : OFF_Q + Q_BYTES;
  static constexpr int OFF_STATE = OVERLAY ? OFF_Q + Q_BYTES : OFF_P + P_BUFS * P_BYTES;
  static constexpr int OFF_M = OFF_STATE;               // running maximum per row, negated
  static constexpr int OFF_ALPHA = OFF_M + NT * 4;
  static constexpr int OFF_WMAX = OFF_ALPHA + NT * 4;   // [4][NT]
  static constexpr int OFF_LRED = OFF_WMAX + 4 * NT * 4;   // [2][4][NT]: sums of weights, of rounded ones
  static constexpr int OFF_INV = OFF_LRED + 8 * NT * 4;
  static constexpr int OFF_CS = OFF_INV + NT * 4;       // score scale per row (FP8)
  static constexpr int OFF_RANGE = OFF_CS + NT * 4;     // int2 visible keys per row
  static constexpr int OFF_TOP = OFF_RANGE + NT * 8;    // FP8: [2][4][NT] largest weights of a tile
  static constexpr int OFF_CREDIT = OFF_TOP + (FP8 ? 8 * NT * 4 : 0);  // FP8: [NT] credit, [NT] greatest m
  static constexpr int OFF_ITEM = OFF_CREDIT + (FP8 ? 2 * NT * 4 : 0);
  static constexpr int ITEMS = 4;
  static constexpr int OFF_BAR = OFF_ITEM + ITEMS * (int)sizeof(LatentItem);
  static constexpr int BARS = 2 * SLOTS + 2 * R_SLOTS + 2 + 2 + 2 + 3 + 2 + 2 * ITEMS;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;   // TMEM address, abort flag, counts of loads, scan sums
  static constexpr int SMEM = OFF_MISC + 32 + 32 * 4;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int RH = NT == 64 ? 16 : 8;          // query rows per softmax thread
  static constexpr int GROUPS = NT / RH;
  static constexpr int SOFT = 4;                        // first softmax warp
  static constexpr int WARPS = SOFT + 4 * GROUPS;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int SOFT_THREADS = 128 * GROUPS;
  static constexpr int COL_O = 0, COL_S = NB * N2;
  static constexpr int COLS = COL_S + 2 * SN;
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512 && SLOTS >= UPT && SMEM_ALLOC <= 227 * 1024, "capacity");
  static_assert(BLK % 1024 == 0 && Q_BLK % 1024 == 0 && Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0, "alignment");
  // A row's weights start at 2^HEAD for its largest score so far (exactly, so that a
  // peak is not rounded: with m in whole numbers it was off by up to 2^-8), and m moves
  // once one would pass 2^TOP (e4m3 holds 448 = 2^8.8). FP8: m moves down as well, by no
  // more than DOWN below its greatest value: what rounds off there is 2^-50 of the
  // largest weight a tile, and sums of 2^31 tokens, 2^30 the largest 2^-e, stay below
  // 2^127.
  static constexpr float HEAD = FP8 ? 5.f : 0.f, TOP = FP8 ? 8.75f : 8.f, DOWN = 40.f;
  // What a change of sequence takes, in tiles (queries, sums and stores; bf16 tiles
  // are twice as long, and go on being loaded meanwhile). Us at 0 / 1 / 2 / 3 / 4 / 6 for
  // 60 to 300 sequences of 0 to 1500 .. 6000 tokens, a head a packed row:
  //   bf16, R 512, 32 rows 71.7 / 69.7 / 71.9 / 74.3 / 75.8 / 80.2
  //                64      68.0 / 65.1 / 66.9 / 69.6 / 72.5 / 75.9
  //                128     65.3 / 59.9 / 60.9 / 61.5 / 61.2 / 61.6
  //         R 256, 16      63.3 / 62.3 / 62.4 / 63.4 / 64.0 / 65.7
  //                32      65.7 / 64.6 / 64.6 / 65.5 / 66.7 / 67.9
  //                64      64.6 / 59.4 / 57.5 / 58.0 / 58.9 / 60.3
  //   FP8,  R 512, 16      66.8 / 63.4 / 60.4 / 59.3 / 60.3 / 62.7
  //                32      70.0 / 62.6 / 59.2 / 57.0 / 57.7 / 61.1
  //                48      73.8 / 70.3 / 65.9 / 62.4 / 62.0 / 65.0
  //                128     84.4 / 77.9 / 74.1 / 72.6 / 72.4 / 73.9
  //         R 256, 16      64.7 / 62.2 / 58.5 / 57.4 / 56.2 / 57.2
  //                32      72.8 / 68.2 / 67.1 / 63.6 / 63.0 / 64.7
  static constexpr int ITEM_COST = !FP8 ? 1 : NT == 16 ? 3 : 4;
};

__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Loads `box` tokens from token group `group` on, of every token the 128-byte
// columns from `col` on (make_tokens_map).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int col, int group,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(col), "r"(group), "r"(smem_addr(bar))
      : "memory");
}

// 128-byte-swizzled address of 16-byte piece c of row n in a block of rows.
__device__ __forceinline__ uint32_t sw128(int n, int c) {
  return (n >> 3) * 1024 + (n & 7) * 128 + ((c ^ (n & 7)) << 4);
}

// Sums of N values over a warp's lanes: every step hands half of the values to
// the partner, so lane l ends with the sum of value l / (32 / N) in v[0].
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < h; ++k) {
      const float send = up ? v[k] : v[k + h], keep = up ? v[k + h] : v[k];
      v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
}

// N (8 or 16) consecutive fp32 TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float (&v)[N]) {
  if constexpr (N == 16) tmem_ld16(taddr, v);
  else tmem_ld8(taddr, v);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const float (&v)[N]) {
  if constexpr (N == 16) tmem_st16(taddr, v);
  else tmem_st8(taddr, v);
}

template <int R, bool FP8, int NT>
__global__ void __launch_bounds__(LatentCfg<R, FP8, NT>::THREADS, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap map_c,
                         const __grid_constant__ CUtensorMap map_r,
                         const __grid_constant__ CUtensorMap map_q, const LatentArgs a) {
  using C = LatentCfg<R, FP8, NT>;
  constexpr unsigned FULL = 0xFFFFFFFFu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int team = blockIdx.x / a.row_tiles, rt = blockIdx.x % a.row_tiles;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [SLOTS] latents landed
  uint64_t* empty = full + C::SLOTS;         // [SLOTS] its O^T products done
  uint64_t* rfull = empty + C::SLOTS;        // [R_SLOTS] rotated parts landed
  uint64_t* rempty = rfull + C::R_SLOTS;     // [R_SLOTS] and read (overlay: and the weights too)
  uint64_t* s_full = rempty + C::R_SLOTS;    // [2] S^T in TMEM
  uint64_t* p_ready = s_full + 2;            // [2] S^T read, weights in shared memory
  uint64_t* o_full = p_ready + 2;            // [2] O^T of the tile added
  uint64_t* q_full = o_full + 2;             // Q of the item in shared memory
  uint64_t* q_free = q_full + 1;             // S^T products of the item done
  uint64_t* o_free = q_free + 1;             // O^T of the item read back
  uint64_t* drain = o_free + 1;              // [2] after giving up: an issuer's products done
  uint64_t* item_full = drain + 2;           // [ITEMS]
  uint64_t* item_free = item_full + C::ITEMS;  // [ITEMS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* loads = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // units, rotated parts, Qs asked for
  int* sums = reinterpret_cast<int*>(smem + C::OFF_MISC + 32);  // [WARPS]
  LatentItem* items = reinterpret_cast<LatentItem*>(smem + C::OFF_ITEM);

  LatentShares shares;  // (the loads go out first)
  latent_load_shares<C::WARPS>(a, shares, warp, lane, warp == 3);
  if (tid < C::BARS) {
    uint64_t* bar = full + tid;
    const uint32_t count = bar >= p_ready && bar < o_full                 ? C::SOFT_THREADS
                           : bar == o_free || (FP8 && bar == q_full)      ? C::SOFT_THREADS
                           : bar >= item_full && bar < item_free          ? 32
                           : bar >= item_free ? C::GROUPS + 3  // softmax groups, producer, both MMA issuers
                                              : 1;
    mbar_init(bar, count);
    fence_mbar_init();
  }
  if (tid == 0) *abort_flag = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!shares.few) {
    const int sum = __reduce_add_sync(FULL, shares.sum);
    if (lane == 0) sums[warp] = sum;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // the merge may be set up beside us; it waits for our end

  if (warp == 3) {
    // ======================= schedule (whole warp) =============================
    const int i0 = rt * NT / a.H, i1 = (min(a.M, rt * NT + NT) - 1) / a.H;  // query rows of the row tile
    int j = 0, qloads = 0;
    bool ok = true;
    auto publish = [&](int b, int kv_len, int t0, int t1, bool whole, bool goes_on) {  // uniform over the warp
      if (j >= C::ITEMS)
        ok = __all_sync(FULL, wait_or_abort(&item_free[j % C::ITEMS], ((j / C::ITEMS) - 1) & 1, abort_flag, a.err));
      if (!ok) return;
      LatentItem& d = items[j % C::ITEMS];
      if (lane == 0) {
        if (b >= 0) latent_fill(a, d, b, kv_len, t0, t1, whole, (team * a.row_tiles + rt) * 2 + goes_on, i0, i1);
        else d.b = -1;
      }
      __syncwarp();
      mbar_arrive(&item_full[j % C::ITEMS]);
      if (!FP8 && b >= 0) {  // Q rows by TMA, once the item before has been multiplied
        if (j >= 1) ok = __all_sync(FULL, wait_or_abort(q_free, (j - 1) & 1, abort_flag, a.err));
        qloads += ok;
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(q_full, C::Q_BYTES);
#pragma unroll 1
          for (int c = 0; c <= R / 64; ++c)
            tma_load_2d(sbase + C::OFF_Q + c * (NT * 128), &map_q, c * 64, b * a.M + rt * NT, q_full);
        }
        __syncwarp();
      }
      ++j;
    };
    const int2 cut = latent_schedule<C::WARPS>(a, shares, sums, team, lane, ok, publish);
    if (!ok) *abort_flag = 1;
    if (lane == 0) loads[2] = qloads;
    if (rt == 0 && lane == 0) a.cut[team] = cut;
    __syncwarp();
  } else if (warp == 0) {
    // ======================= TMA producer (whole warp) =========================
    // Unit u of tile t (counted over all items) goes to slot (t * UPT + u) % SLOTS.
    // Lane g copies page segment g of the tile's tokens.
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_c) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_r) : "memory");
    }
    const int seg_rows = min(a.page_size, kTile), log2_seg = min(a.log2_page, 7);
    int g = 0, blk = 0, ropes = 0;
    bool ok = true;
    for (int j = 0; ok; ++j) {
      ok = __all_sync(FULL, wait_or_abort(&item_full[j % C::ITEMS], (j / C::ITEMS) & 1, abort_flag, a.err));
      if (!ok) break;
      const LatentItem d = items[j % C::ITEMS];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_free[j % C::ITEMS]);
      if (d.b < 0) break;
      const int32_t* pt = a.page_table + (long long)d.b * a.max_pages;
      // segments of tile t that hold tokens, counted from the tile's first token
      auto segments = [&](int t) { return min(kTile, d.L - t * kTile + seg_rows - 1) >> log2_seg; };
      auto page_of = [&](int t) -> int {  // the page of this lane's segment of tile t
        if (t >= d.first + d.n || lane >= segments(t)) return 0;
        return __ldg(pt + ((t * kTile + lane * seg_rows) >> a.log2_page));
      };
      // The rotated parts go first (their slot is free as soon as S^T is): they are
      // multiplied while the latents are on their way. (Overlay: their slot holds
      // the weights until O^T is done.)
      auto load_rope = [&](int nseg, int row) {
        const int rs = g % C::R_SLOTS;
        if (g >= C::R_SLOTS)
          ok = __all_sync(FULL, wait_or_abort(&rempty[rs], ((g / C::R_SLOTS) - 1) & 1, abort_flag, a.err));
        if (!ok) return false;
        if (lane == 0) mbar_arrive_expect_tx(&rfull[rs], (uint32_t)(nseg * seg_rows) * 128u);
        __syncwarp();
        if (lane < nseg)
          tma_load_2d(sbase + C::OFF_ROPE + rs * C::ROPE_SLOT + lane * seg_rows * 128, &map_r, 0, row, &rfull[rs]);
        ++ropes;
        return true;
      };
      int pid = page_of(d.first), pid_next = page_of(d.first + 1);
      for (int t = d.first; ok && t < d.first + d.n; ++t, ++g) {
        const int nseg = segments(t);
        // A team of several CTAs: the next tile's segments into L2, by one of them:
        // the copies, issued when shared memory is free, then find them there (74
        // sequences of 8192 tokens, 128 heads: 235 -> 216 us). A CTA by itself is
        // bound by HBM, and slower with it (148 sequences, 64 heads: 255 -> 268 us).
        if (a.row_tiles > 1 && t + 1 < d.first + d.n && lane < segments(t + 1) && (unsigned)pid_next < (unsigned)a.num_pages &&
            (t % a.row_tiles) == rt) {
          const long long next = (long long)pid_next * a.page_size + (((t + 1) * kTile + lane * seg_rows) & (a.page_size - 1));
          l2_prefetch(a.latent_pages + next * (FP8 ? R : 2 * R), seg_rows * (FP8 ? R : 2 * R));
          l2_prefetch(a.rope_pages + next * a.rope_dim, seg_rows * a.rope_dim * 2);
        }
        if ((unsigned)pid >= (unsigned)a.num_pages) {
          record_error_at(a.err, kErrBadPage);
          pid = 0;
        }
        const int row = pid * a.page_size + ((t * kTile + lane * seg_rows) & (a.page_size - 1));
        pid = pid_next;
        pid_next = page_of(t + 2);
        if (!C::OVERLAY && !load_rope(nseg, row)) break;
#pragma unroll 1
        for (int k = 0; k < C::UPT; ++k, ++blk) {
          const int sl = blk % C::SLOTS;
          if (blk >= C::SLOTS) {
            ok = __all_sync(FULL, wait_or_abort(&empty[sl], ((blk / C::SLOTS) - 1) & 1, abort_flag, a.err));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[sl], (uint32_t)((nseg * seg_rows) >> 3) * C::GS);
          __syncwarp();
          if (lane < nseg)
            tma_load_4d(sbase + C::OFF_BLK + sl * C::BLK + ((lane * seg_rows) >> 3) * C::GS, &map_c, 2 * k, row >> 3,
                        &full[sl]);
        }
        if (!ok) break;
        if (C::OVERLAY && !load_rope(nseg, row)) break;
      }
    }
    if (!ok) *abort_flag = 1;
    if (lane == 0) {
      loads[0] = blk;
      loads[1] = ropes;
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ======================= MMA issuers: S^T (warp 1), O^T (warp 2) ===========
    // The whole warp follows the loop and one elected lane issues: the
    // operands then stay in uniform registers, and an MMA costs what the
    // tensor core and its shared-memory reads take (measured: 48 cycles at 64
    // columns, 40 at 32; from a single-lane branch 58 to 73). Descriptors of
    // one operand differ by constants in their address field.
    const bool leader = elect_one();
    bool ok = true;
    int g = 0, blk = 0;
    auto agreed = [&](bool v) { return __all_sync(FULL, v); };
    for (int j = 0; ok; ++j) {
      ok = agreed(wait_or_abort(&item_full[j % C::ITEMS], (j / C::ITEMS) & 1, abort_flag, a.err));
      if (!ok) break;
      const int n = items[j % C::ITEMS].n, b = items[j % C::ITEMS].b;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_free[j % C::ITEMS]);
      if (b < 0) break;
      if (warp == 1) {
        ok = agreed(wait_or_abort(q_full, j & 1, abort_flag, a.err));
        for (int t = 0; ok && t < n; ++t, ++g) {
          const int bb = g & 1;
          if (g >= 2) ok = agreed(wait_or_abort(&p_ready[bb], ((g - 2) >> 1) & 1, abort_flag, a.err));
          const uint32_t dt = tmem + C::COL_S + bb * C::SN;
          const uint64_t q0 = umma_desc(sbase + C::OFF_Q, 16, 1024, kSw128);
          // bf16: into the columns of the latents' product, whichever comes first
          auto rope_product = [&]() {
            const int rs = g % C::R_SLOTS;
            ok = ok && agreed(wait_or_abort(&rfull[rs], (g / C::R_SLOTS) & 1, abort_flag, a.err));
            if (!ok) return false;
            tmem_fence_after();
            if (leader) {
              constexpr uint32_t idesc = umma_idesc_bf16(128, NT, false, false);
              const uint64_t ra = umma_desc(sbase + C::OFF_ROPE + rs * C::ROPE_SLOT, 16, 1024, kSw128);
              const uint64_t qb = q0 + (C::Q_ROPE >> 4);
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_f16(FP8 ? dt + C::N1 : dt, ra + 2 * s, qb + 2 * s, idesc, C::OVERLAY || s > 0);
              if constexpr (!C::OVERLAY) umma_commit(&rempty[rs]);
            }
            __syncwarp();
            return true;
          };
          if (!C::OVERLAY && !rope_product()) break;
#pragma unroll 1
          for (int k = 0; ok && k < C::UPT; ++k, ++blk) {
            const int sl = blk % C::SLOTS;
            ok = agreed(wait_or_abort(&full[sl], (blk / C::SLOTS) & 1, abort_flag, a.err));
            if (!ok) break;
            tmem_fence_after();
            const uint64_t ca = umma_desc(sbase + C::OFF_BLK + sl * C::BLK, 16, C::GS, kSw128);
            const uint64_t qb = q0 + ((k * C::BPU * C::Q_BLK) >> 4);
            if (leader) {  // eight steps of 32 bytes a token
              constexpr uint32_t idesc = FP8 ? umma_idesc_e4m3(128, C::N1) : umma_idesc_bf16(128, NT, false, false);
#pragma unroll
              for (int s = 0; s < 8; ++s) {
                const uint64_t cs = ca + (((s >> 2) * 1024 + (s & 3) * 32) >> 4);
                const uint64_t qs = qb + (((s >> 2) * (FP8 ? C::Q_BLK : NT * 128) + (s & 3) * 32) >> 4);
                if constexpr (FP8) umma_f8(dt, cs, qs, idesc, k > 0 || s > 0);
                else umma_f16(dt, cs, qs, idesc, !C::OVERLAY || k > 0 || s > 0);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (C::OVERLAY && !rope_product()) break;
          if (leader) umma_commit(&s_full[bb]);
          __syncwarp();
        }
        if (ok && leader) umma_commit(q_free);
      } else {
        if (j >= 1) ok = agreed(wait_or_abort(o_free, (j - 1) & 1, abort_flag, a.err));
        for (int t = 0; ok && t < n; ++t, ++g) {
          const int bb = g & 1;
          ok = agreed(wait_or_abort(&p_ready[bb], (g >> 1) & 1, abort_flag, a.err));
          if (!ok) break;
          tmem_fence_after();
          constexpr uint32_t SBO = 8 * C::P_ROW;
          const uint64_t pd = umma_desc(sbase + C::OFF_P + (g % C::P_BUFS) * C::P_BYTES, C::P_BYTES, SBO, C::P_SWIZZLE);
#pragma unroll 1
          for (int k = 0; k < C::UPT; ++k, ++blk) {
            const int sl = blk % C::SLOTS;
            const uint64_t ca = umma_desc(sbase + C::OFF_BLK + sl * C::BLK, 1024, C::GS, kSw128);
            const uint32_t dt = tmem + C::COL_O + k * C::BPU * C::N2;
            if (leader) {
              if constexpr (FP8) {  // two blocks, 32 tokens a step
                constexpr uint32_t idesc = umma_idesc_e4m3_mn(128, C::N2);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  umma_f8(dt + (s >> 2) * C::N2, ca + (((s & 3) * 4 * C::GS + (s >> 2) * 1024) >> 4),
                          pd + (((s & 3) * 4 * SBO) >> 4), idesc, t > 0 || (s & 3) > 0);
              } else {  // one block, 16 tokens a step
                constexpr uint32_t idesc = umma_idesc_bf16(128, C::N2, true, true);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  umma_f16(dt, ca + ((s * 2 * C::GS) >> 4), pd + ((s * 2 * SBO) >> 4), idesc, t > 0 || s > 0);
              }
              umma_commit(&empty[sl]);
            }
            __syncwarp();
          }
          if (leader) {
            if constexpr (C::OVERLAY) umma_commit(&rempty[g % C::R_SLOTS]);
            umma_commit(&o_full[bb]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
  } else {
    // ======================= softmax ===========================================
    // A group of four warps owns RH query rows; thread i is token i of the tile
    // in S^T and element i of each block in O^T.
    constexpr int GT = 128, RH = C::RH;
    constexpr float kLn2 = 0.69314718055994531f, kUnset = -1e30f;
    const int q4 = warp & 3, grp = (warp - C::SOFT) >> 2, gbar = 2 + grp, r0 = RH * grp;
    const int i = 32 * q4 + lane;
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    float* sm_nm = reinterpret_cast<float*>(smem + C::OFF_M);
    float* sm_alpha = reinterpret_cast<float*>(smem + C::OFF_ALPHA);
    float* wmax = reinterpret_cast<float*>(smem + C::OFF_WMAX);
    float* lred = reinterpret_cast<float*>(smem + C::OFF_LRED);
    float* sm_inv = reinterpret_cast<float*>(smem + C::OFF_INV);
    float* sm_cs = reinterpret_cast<float*>(smem + C::OFF_CS);
    float* sm_top = reinterpret_cast<float*>(smem + C::OFF_TOP);
    float* sm_credit = reinterpret_cast<float*>(smem + C::OFF_CREDIT);
    int2* sm_range = reinterpret_cast<int2*>(smem + C::OFF_RANGE);
    const uint32_t s_tm = tmem + lane_off + C::COL_S + (FP8 ? 2 * r0 : r0);
    const uint32_t o_tm = tmem + lane_off + C::COL_O + (FP8 ? 2 * r0 : r0);
    const int R0 = rt * NT + r0, rows = min(RH, a.M - R0);  // this group's packed rows
    int g = 0;
    bool ok = true;
    for (int j = 0; ok; ++j) {
      const bool got = wait_or_abort(&item_full[j % C::ITEMS], (j / C::ITEMS) & 1, abort_flag, a.err);
      if (!named_bar_and(gbar, GT, got)) {
        ok = false;
        break;
      }
      const LatentItem& d = items[j % C::ITEMS];
      if (d.b < 0) break;
      const int first = d.first, n = d.n, L = d.L, b = d.b;
      if constexpr (FP8) {
        // The item's Q operand. 2^e2 puts a row's max |q_c| in [128, 256); then
        // q_c * 2^e2 = hi + lo / 16 in e4m3, exact for every element within
        // 2^13 of the row's largest (others to 2^-21 of it). A warp has RH / 4
        // rows; all their loads go out first.
        uint8_t* qs = smem + C::OFF_Q;
        constexpr int E = R / 32, W = RH / 4;  // elements of a row per lane, rows
        uint4 raw[W][E / 8], rope[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int row = R0 + q4 + 4 * w;
          const uint16_t* src = a.q + ((long long)b * a.M + row) * (R + a.rope_dim);
#pragma unroll
          for (int k = 0; k < E / 8; ++k)
            raw[w][k] = row < a.M ? __ldg(reinterpret_cast<const uint4*>(src + lane * E) + k) : make_uint4(0, 0, 0, 0);
          rope[w] = row < a.M && lane * 8 < a.rope_dim ? __ldg(reinterpret_cast<const uint4*>(src + R) + lane)
                                                       : make_uint4(0, 0, 0, 0);
        }
        if (j >= 1 && !wait_or_abort(q_free, (j - 1) & 1, abort_flag, a.err)) *abort_flag = 1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int rr = q4 + 4 * w, nrow = r0 + rr;
          float f[E];
#pragma unroll
          for (int k = 0; k < E / 8; ++k) bf16x8_to_f32(raw[w][k], *reinterpret_cast<float(*)[8]>(f + 8 * k));
          float mx = 0.f;
#pragma unroll
          for (int k = 0; k < E; ++k) mx = fmaxf(mx, fabsf(f[k]));
          mx = redux_max(mx);
          // 2^e2 from the exponent field of mx (0 for a row of zeros; within 2^+-120)
          const int e2 = mx > 0.f ? min(max(134 - (int)(__float_as_uint(mx) >> 23), -120), 120) : 0;
          const float up = __int_as_float((127 + e2) << 23);
          // (an infinite element, which e4m3 does not have, makes the row's scores NaN)
          if (lane == 0)
            sm_cs[nrow] = mx < INFINITY ? a.scale_log2 * __int_as_float((127 - e2) << 23) : __int_as_float(0x7FC00000);
          uint32_t hw[E / 4], lw[E / 4];
#pragma unroll
          for (int x = 0; x < E / 4; ++x) {  // (bf16's 8 bits times 2^e2 fit f16, in which the split works)
            const uint32_t s01 = e4m3_split2(f[4 * x] * up, f[4 * x + 1] * up);
            const uint32_t s23 = e4m3_split2(f[4 * x + 2] * up, f[4 * x + 3] * up);
            hw[x] = __byte_perm(s01, s23, 0x5410);
            lw[x] = __byte_perm(s01, s23, 0x7632);
          }
          const int rh = 2 * r0 + rr, rl = rh + RH, el = lane * E;
          uint8_t* blk_base = qs + (el >> 7) * C::Q_BLK;
          const int c = (el & 127) >> 4;
          if constexpr (E == 16) {
            *reinterpret_cast<uint4*>(blk_base + sw128(rh, c)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(blk_base + sw128(rl, c)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
          } else {
            *reinterpret_cast<uint2*>(blk_base + sw128(rh, c) + (el & 8)) = make_uint2(hw[0], hw[1]);
            *reinterpret_cast<uint2*>(blk_base + sw128(rl, c) + (el & 8)) = make_uint2(lw[0], lw[1]);
          }
          if (lane < 8) *reinterpret_cast<uint4*>(qs + C::Q_ROPE + sw128(nrow, lane)) = rope[w];
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      if (i < RH) {
        int lo = 0, hi = 0;
        if (R0 + i < a.M) latent_visible(a, L, (R0 + i) / a.H, lo, hi);
        sm_range[r0 + i] = make_int2(lo, hi);
        sm_nm[r0 + i] = -kUnset;
        if constexpr (FP8) {
          sm_credit[r0 + i] = 2.f;  // (until the row's first key)
          sm_credit[NT + r0 + i] = kUnset;
        }
      }
      named_bar(gbar, GT);
      // FP8: this token's scale exponent, looked up a tile ahead
      const int32_t* pt = a.page_table + (long long)b * a.max_pages;
      auto scale_of = [&](int t) -> int {
        const int jt = t * kTile + i;
        if (!FP8 || t >= first + n || jt >= L) return 127;
        const int page = __ldg(pt + (jt >> a.log2_page));
        if ((unsigned)page >= (unsigned)a.num_pages) return 127;
        return __ldg(a.scales + (long long)page * a.page_size + (jt & (a.page_size - 1)));
      };
      int sc_next = scale_of(first);
      bool low = false;  // FP8, threads i < rows: row i's credit runs out
      float l_sum[RH], l_rnd[RH];  // this token's part of the row sums: of the weights, of the rounded ones
#pragma unroll
      for (int r = 0; r < RH; ++r) l_sum[r] = l_rnd[r] = 0.f;
      for (int t = first; t < first + n; ++t, ++g) {
        const int bb = g & 1;
        const float e_tok = FP8 ? (float)(min(max(sc_next, 97), 157) - 127) : 0.f;
        sc_next = scale_of(t + 1);
        bool good = __all_sync(FULL, wait_or_abort(&s_full[bb], (g >> 1) & 1, abort_flag, a.err));
        // Raw scores; FP8: hi + lo / 16 of the latent parts, and the rotated parts.
        float sc[RH], se[FP8 ? RH : 1];
        if (good) {
          tmem_fence_after();
          const uint32_t ta = s_tm + bb * C::SN;
          if constexpr (FP8) {
            float hl[2 * RH];
            tmem_ldn(ta, hl);
            tmem_ldn(tmem + lane_off + C::COL_S + bb * C::SN + C::N1 + r0, se);
#pragma unroll
            for (int r = 0; r < RH; r += 2)
              f2_unpack(f2_fma(f2_pack(hl[RH + r], hl[RH + r + 1]), f2_pack(0.0625f, 0.0625f), f2_pack(hl[r], hl[r + 1])),
                        sc[r], sc[r + 1]);
          } else {
            tmem_ldn(ta, sc);
          }
        } else {
#pragma unroll
          for (int r = 0; r < RH; ++r) sc[r] = -INFINITY;
          if constexpr (FP8)
#pragma unroll
            for (int r = 0; r < RH; ++r) se[r] = 0.f;
        }
        const int t0 = t * kTile, jt = t0 + i;
        const bool clean = t0 >= d.lo_x && t0 + kTile <= d.hi_x;
        if (!clean) {
          // A token that no row sees may hold NaN: its latents become zeros
          // before they meet its zero weights. The groups share the blocks.
          if (good && (jt < d.lo_u || jt >= d.hi_u)) {
            for (int k = grp; k < C::NB; k += C::GROUPS) {
              const int u = g * C::UPT + k / C::BPU;
              uint8_t* row = smem + C::OFF_BLK + (u % C::SLOTS) * C::BLK + (i >> 3) * C::GS + (i & 7) * 128 +
                             k % C::BPU * 1024;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const int cc = (c + i) & 7;
                *reinterpret_cast<uint4*>(row + cc * 16) = make_uint4(0, 0, 0, 0);
                if constexpr (!FP8) *reinterpret_cast<uint4*>(row + 1024 + cc * 16) = make_uint4(0, 0, 0, 0);
              }
            }
          }
        }
        // Scores in log2 units less the rows' running maxima (or as they are),
        // FP8 with the token's exponent added; -inf where the row does not see
        // the token. Two rows an instruction.
        const f32x2 scale2 = f2_pack(a.scale_log2, a.scale_log2);
        auto relative = [&](bool less_max, float (&x)[RH]) {
#pragma unroll
          for (int r = 0; r < RH; r += 2) {
            const f32x2 base = less_max ? *reinterpret_cast<const f32x2*>(sm_nm + r0 + r) : f2_pack(0.f, 0.f);
            f32x2 v;
            if constexpr (FP8) {
              const float up = __int_as_float((int)(e_tok + 127.f) << 23);
              v = f2_fma(f2_pack(se[r], se[r + 1]), scale2, f2_add(base, f2_pack(e_tok, e_tok)));
              v = f2_fma(f2_pack(sc[r], sc[r + 1]),
                         f2_mul(*reinterpret_cast<const f32x2*>(sm_cs + r0 + r), f2_pack(up, up)), v);
            } else {
              v = f2_fma(f2_pack(sc[r], sc[r + 1]), scale2, base);
            }
            f2_unpack(v, x[r], x[r + 1]);
          }
          if (!clean) {
#pragma unroll
            for (int r = 0; r < RH; ++r) {
              const int2 v = sm_range[r0 + r];
              if (!(jt >= v.x && jt < v.y)) x[r] = -INFINITY;
            }
          }
        };
        float x[RH];
        relative(true, x);
        // The running maximum moves only when a score passes it by so much that
        // a weight would pass 2^TOP; most tiles skip the exchange.
        float top = x[0];
#pragma unroll
        for (int r = 1; r < RH; ++r) top = fmaxf(top, x[r]);
        const bool moves = named_bar_or(gbar, GT, !good || top > C::TOP || low);
        // FP8: a row's credit with the tile before, whose largest weights all warps have
        // left by then. It is looked at a tile later still, so that two tiles have to be left.
        auto credit_of = [&]() {
          const float* wt = sm_top + ((g - 1) & 1) * 4 * NT + r0 + i;
          const float wm = fmaxf(fmaxf(wt[0], wt[NT]), fmaxf(wt[2 * NT], wt[3 * NT]));
          return sm_credit[r0 + i] + (t > first ? wm * 0.25f - fminf(1.f, wm * 16384.f) : 0.f);
        };
        if (moves) {
          if (!named_bar_and(gbar, GT, good)) {
            ok = false;
            break;
          }
          relative(false, x);
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            const float wm = redux_max(x[r]);
            if (lane == r) wmax[q4 * NT + r0 + r] = wm;
          }
          named_bar(gbar, GT);
          if (i < RH) {
            const int rr = r0 + i;
            const float most = fmaxf(fmaxf(wmax[rr], wmax[NT + rr]), fmaxf(wmax[2 * NT + rr], wmax[3 * NT + rr]));
            const float m_old = -sm_nm[rr];
            if constexpr (FP8) {
              float m_new = most - C::HEAD;  // (-inf: no key of this tile is seen)
              float credit = credit_of();
              if (m_new > m_old) {
                low = false;  // (the tile pays for itself and seven more)
              } else if (low && most != -INFINITY) {
                const float least = sm_credit[NT + rr] - C::DOWN;
                if (m_new <= least) credit = 1e9f;  // the end of the way down: no more to pay
                m_new = fminf(fmaxf(m_new, least), m_old);
                low = false;
              } else {
                m_new = m_old;
                low = i < rows && credit < 2.f;
              }
              const float al = fast_exp2(m_old - m_new);
              sm_alpha[rr] = al;
              sm_credit[rr] = credit * al;
              sm_credit[NT + rr] = fmaxf(sm_credit[NT + rr], m_new);
              sm_nm[rr] = -m_new;
            } else {
              const float m_new = fmaxf(m_old, most - C::HEAD);
              sm_alpha[rr] = fast_exp2(m_old - m_new);
              sm_nm[rr] = -m_new;
            }
          }
          named_bar(gbar, GT);
          float al[RH];
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            al[r] = sm_alpha[r0 + r];
            l_sum[r] *= al[r];
            l_rnd[r] *= al[r];
          }
          if (t > first) {  // what the item's earlier tiles added moves along
            good = __all_sync(FULL, wait_or_abort(&o_full[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, a.err));
            if (good) {
              tmem_fence_after();
#pragma unroll 1
              for (int k = 0; k < C::NB; ++k) {  // (FP8: both terms' columns, 2 RH of them)
                float o[FP8 ? 2 * RH : RH];
                tmem_ldn(o_tm + k * C::N2, o);
#pragma unroll
                for (int r = 0; r < (FP8 ? 2 * RH : RH); ++r) o[r] *= al[r % RH];
                tmem_stn(o_tm + k * C::N2, o);
              }
              tmem_fence_before();
            } else {
              *abort_flag = 1;
            }
          }
          relative(true, x);
        }
#pragma unroll
        for (int r = 0; r < RH; ++r) x[r] = fast_exp2(x[r]);
        uint32_t w[RH / 2];  // FP8: first terms, then second terms; bf16: pairs
        if constexpr (FP8) {
#pragma unroll
          for (int r = 0; r < RH; r += 4) {
            const uint32_t s01 = e4m3_split2(x[r], x[r + 1]), s23 = e4m3_split2(x[r + 2], x[r + 3]);
            w[r / 4] = __byte_perm(s01, s23, 0x5410);
            w[RH / 4 + r / 4] = __byte_perm(s01, s23, 0x7632);
          }
        } else {
#pragma unroll
          for (int r = 0; r < RH; r += 2) w[r / 2] = pack_bf16x2(x[r], x[r + 1]);  // (the type of the other operand)
        }
        // The buffer's last reader: the O^T products P_BUFS tiles ago. (Overlay:
        // the rotated parts of this tile were loaded after those, and read.)
        if (!C::OVERLAY && g >= C::P_BUFS) {
          const int u = g - C::P_BUFS;
          if (!wait_or_abort(&o_full[u & 1], (u >> 1) & 1, abort_flag, a.err)) *abort_flag = 1;
        }
        uint8_t* sp = smem + C::OFF_P + (g % C::P_BUFS) * C::P_BYTES + i * C::P_ROW;
        const int z = C::P_ROW == 128 ? i & 7 : C::P_ROW == 64 ? (i >> 1) & 3 : (i >> 2) & 1;
#pragma unroll
        for (int c = 0; c < RH / 8; ++c)
          *reinterpret_cast<uint4*>(sp + (((RH / 8 * grp + c) ^ z) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        tmem_fence_before();
        mbar_arrive(&p_ready[bb]);
        // the sums, beside the products
        const float down = FP8 ? __int_as_float((int)(127.f - e_tok) << 23) : 1.f;
#pragma unroll
        for (int r = 0; r < RH; r += 2) {
          const f32x2 old = f2_pack(l_sum[r], l_sum[r + 1]), v = f2_pack(x[r], x[r + 1]);
          f2_unpack(FP8 ? f2_fma(v, f2_pack(down, down), old) : f2_add(v, old), l_sum[r], l_sum[r + 1]);
          if constexpr (!FP8)
            f2_unpack(f2_add(bf16x2_to_f2(w[r / 2]), f2_pack(l_rnd[r], l_rnd[r + 1])), l_rnd[r], l_rnd[r + 1]);
        }
        if constexpr (FP8) {  // the rows' largest weights of this tile
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            const float wm = redux_max(x[r]);
            if (lane == r) sm_top[((g & 1) * 4 + q4) * NT + r0 + r] = wm;
          }
          if (!moves && i < rows) {
            const float credit = credit_of();
            sm_credit[r0 + i] = credit;
            low = credit < 2.f;
          }
        }
      }
      if (!ok) break;
      // ---- the item's end: normalise O^T and store it, or the partial results.
      // Sums over the 128 tokens in one order, over the warp's lanes, each lane
      // ending with one row's sum, then over the four warps; beside the last
      // tile's products.
      lane_sums(l_sum, lane);
      if constexpr (!FP8) lane_sums(l_rnd, lane);
      if (lane % (32 / RH) == 0) {
        lred[q4 * NT + r0 + lane / (32 / RH)] = l_sum[0];
        if constexpr (!FP8) lred[(4 + q4) * NT + r0 + lane / (32 / RH)] = l_rnd[0];
      }
      named_bar(gbar, GT);
      const int part = d.part;
      if (i < RH) {
        const int rr = r0 + i;
        const float l = lred[rr] + lred[NT + rr] + lred[2 * NT + rr] + lred[3 * NT + rr];
        const float ln = FP8 ? l : lred[4 * NT + rr] + lred[5 * NT + rr] + lred[6 * NT + rr] + lred[7 * NT + rr];
        if (i < rows) {
          // (0 without keys; NaN of a score that is NaN or +inf passes on)
          const float lse = l == 0.f ? -INFINITY : (log2f(l) - sm_nm[rr]) * kLn2;
          if (part >= 0) a.lse_part[(long long)part * NT + rr] = lse;
          else if (a.lse) a.lse[(long long)b * a.M + R0 + i] = lse;
        }
        sm_inv[rr] = ln == 0.f ? 0.f : 1.f / ln;
      }
      named_bar(gbar, GT);
      float inv[RH];
#pragma unroll
      for (int r = 0; r < RH; ++r) inv[r] = sm_inv[r0 + r];
      float* po = a.o_part + ((long long)part * NT + r0) * R + i;
      uint16_t* oo = a.out + ((long long)b * a.M + R0) * R + i;
      bool good = true;
#pragma unroll (NT == 64 ? 1 : 2)
      for (int k = 0; k < C::NB; ++k, po += 128, oo += 128) {
        float o[RH];
#pragma unroll
        for (int r = 0; r < RH; ++r) o[r] = 0.f;
        if (n > 0) {  // the last tile's products of block k are done
          const int blk = (g - 1) * C::UPT + k / C::BPU;
          good = good && wait_or_abort(&empty[blk % C::SLOTS], (blk / C::SLOTS) & 1, abort_flag, a.err);
          if (!__all_sync(FULL, good)) break;
          tmem_fence_after();
          if constexpr (FP8) {
            float hl[2 * RH];
            tmem_ldn(o_tm + k * C::N2, hl);
#pragma unroll
            for (int r = 0; r < RH; ++r) o[r] = fmaf(hl[RH + r], 0.0625f, hl[r]);
          } else {
            tmem_ldn(o_tm + k * C::N2, o);
          }
#pragma unroll
          for (int r = 0; r < RH; ++r) o[r] = inv[r] == 0.f ? 0.f : o[r] * inv[r];
        }
        if (part >= 0) {
#pragma unroll
          for (int r = 0; r < RH; ++r)
            if (r < rows) po[r * R] = o[r];
        } else {
#pragma unroll
          for (int r = 0; r < RH; ++r)
            if (r < rows) oo[r * R] = __bfloat16_as_ushort(__float2bfloat16_rn(o[r]));
        }
      }
      tmem_fence_before();
      mbar_arrive(o_free);
      if (!named_bar_and(gbar, GT, good)) {  // the group no longer reads the item and its row state
        ok = false;
        break;
      }
      if (i == 0) mbar_arrive(&item_free[j % C::ITEMS]);
    }
    if (!ok) *abort_flag = 1;
  }

  tmem_fence_before();
  __syncthreads();
  if (*abort_flag) {  // some role gave up: what was issued finishes before its memory goes away
    constexpr long long lim = kWaitTimeoutCycles / 16;
    if (warp == 0 && lane == 0) {  // copies: the last ones into each slot
      for (int n = max(0, loads[0] - C::SLOTS); n < loads[0]; ++n)
        mbar_wait(&full[n % C::SLOTS], (n / C::SLOTS) & 1, a.err, lim);
      for (int n = max(0, loads[1] - C::R_SLOTS); n < loads[1]; ++n)
        mbar_wait(&rfull[n % C::R_SLOTS], (n / C::R_SLOTS) & 1, a.err, lim);
      if (!FP8 && loads[2] > 0) mbar_wait(q_full, (loads[2] - 1) & 1, a.err, lim);
    } else if (warp == 1 || warp == 2) {  // products: by the lane that issued them
      if (elect_one()) {
        umma_commit(&drain[warp - 1]);
        mbar_wait(&drain[warp - 1], 0, a.err, lim);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                 : "memory");
  }
}

// Joins the partial results of the sequences that lie in several teams' ranges:
// lse = ln sum_k exp(lse_k), out = sum_k exp(lse_k - lse) o_k; a part whose lse is NaN
// makes the row NaN. Of a sequence of
// few parts (most cuts leave two or three) a warp takes a row; of one of many
// parts a block takes a row, WARPS / V warps with every so manyth part each.
// Bound by latency: the list of cuts, then a row's lse and parts, loaded together;
// and by the instructions themselves, which no SM has at hand when the main kernel
// ends. A variant for 2, 3 and 4 parts each, loads of eight parts unrolled and the
// exact exp2f took 3.4 us more (2 sequences of 110 k tokens, 64 heads: 54.8 us
// instead of 51.4), more variants for 5 to 8 parts another 1.5 to 3.
constexpr int kMergeFew = 4, kMergeTeams = 256, kMergeThreads = 512;

template <int R>
__global__ void __launch_bounds__(kMergeThreads, 2) latent_merge_kernel(const LatentArgs a, int log2_nt) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
  constexpr unsigned FULL = 0xFFFFFFFFu;
  constexpr int WARPS = kMergeThreads / 32, V = R / 128, GROUPS = WARPS / V;
  __shared__ float4 part_o[GROUPS - 1][V][32];
  __shared__ int3 cuts[kMergeTeams];  // (team, parts, sequence): those of few parts from the front, the rest from the back
  __shared__ int2 warp_n[kMergeTeams / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_primary();
  int n_few = 0, n_many = 0;
  {
    const int2 c = tid < a.teams ? a.cut[tid] : make_int2(-1, 0);
    // (a schedule that gave up may have left anything)
    const int parts = c.x >= 0 && c.x < a.B && c.y > tid && c.y < a.teams ? c.y - tid + 1 : 0;
    const bool few = parts > 0 && parts <= kMergeFew, many = parts > kMergeFew;
    const unsigned f = __ballot_sync(FULL, few), m = __ballot_sync(FULL, many);
    if (lane == 0 && warp < kMergeTeams / 32) warp_n[warp] = make_int2(__popc(f), __popc(m));
    __syncthreads();
    int f0 = 0, m0 = 0;
#pragma unroll
    for (int w = 0; w < kMergeTeams / 32; ++w) {
      const int2 n = warp_n[w];
      if (w < warp) {
        f0 += n.x;
        m0 += n.y;
      }
      n_few += n.x;
      n_many += n.y;
    }
    const unsigned below = (1u << lane) - 1;
    if (few) cuts[f0 + __popc(f & below)] = make_int3(tid, parts, c.x);
    if (many) cuts[kMergeTeams - 1 - m0 - __popc(m & below)] = make_int3(tid, parts, c.x);
    __syncthreads();
  }
  // slot of part k: the piece goes on behind the team's range but in the last
  auto slot_of = [&](const int3& c, int row, int k) {
    return ((long long)(((c.x + k) * a.row_tiles + (row >> log2_nt)) * 2 + (k + 1 < c.y ? 1 : 0)) << log2_nt) +
           (row & ((1 << log2_nt) - 1));
  };
  // sum_k exp(lse_k - m) and the largest lse_k (0 if all are -inf), m; l0: this lane's
  auto row_lse = [&](const int3& c, int row, float l0, float& m) {
    m = l0;
#pragma unroll 1
    for (int k = lane + 32; k < c.y; k += 32) m = fmaxf(m, a.lse_part[slot_of(c, row, k)]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    if (m == -INFINITY) m = 0.f;
    float sum = fast_exp2((l0 - m) * kLog2e);
#pragma unroll 1
    for (int k = lane + 32; k < c.y; k += 32) sum += fast_exp2((a.lse_part[slot_of(c, row, k)] - m) * kLog2e);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    return sum;
  };
  auto store = [&](long long o, int col, const float4& v) {
    *reinterpret_cast<uint2*>(a.out + o * R + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  };

  // A row of up to kMergeFew parts: all its loads go out together, in two halves
  // of the columns for the registers.
  auto few_row = [&](const int3& c, int row) {
    constexpr int P = kMergeFew, X = V / 2;
    float l[P], m = -INFINITY;
    const float4* src[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const long long s = slot_of(c, row, min(k, c.y - 1));
      l[k] = k < c.y ? a.lse_part[s] : -INFINITY;
      src[k] = reinterpret_cast<const float4*>(a.o_part + s * R) + lane;
    }
    const long long o = (long long)c.z * a.M + row;
#pragma unroll
    for (int x0 = 0; x0 < V; x0 += X) {
      float4 q[X][P];
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int k = 0; k < P; ++k) q[x][k] = k < 2 || k < c.y ? src[k][32 * (x0 + x)] : make_float4(0.f, 0.f, 0.f, 0.f);
      if (x0 == 0) {  // the parts' weights, and the row's lse
#pragma unroll
        for (int k = 0; k < P; ++k) m = fmaxf(m, l[k]);
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < P; ++k) sum += l[k] = fast_exp2((l[k] - base) * kLog2e);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < P; ++k) l[k] *= inv;
        if (lane == 0 && a.lse) a.lse[o] = sum == 0.f ? -INFINITY : base + log2f(sum) * kLn2;
      }
#pragma unroll
      for (int x = 0; x < X; ++x) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          acc.x = fmaf(l[k], q[x][k].x, acc.x);
          acc.y = fmaf(l[k], q[x][k].y, acc.y);
          acc.z = fmaf(l[k], q[x][k].z, acc.z);
          acc.w = fmaf(l[k], q[x][k].w, acc.w);
        }
        store(o, (lane + 32 * (x0 + x)) * 4, acc);
      }
    }
  };
  for (int u = blockIdx.x * WARPS + warp; u < n_few * a.M; u += gridDim.x * WARPS) {
    const int ci = u / a.M, row = u - ci * a.M;
    const int3 c = cuts[ci];
    few_row(c, row);
  }

  for (int u = blockIdx.x; u < n_many * a.M; u += gridDim.x) {
    const int ci = u / a.M, row = u - ci * a.M;
    const int3 c = cuts[kMergeTeams - 1 - ci];
    const int x = warp % V, grp = warp / V;
    const float l0 = lane < c.y ? a.lse_part[slot_of(c, row, lane)] : -INFINITY;
    float m;
    const float sum = row_lse(c, row, l0, m);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sum != 0.f) {
      const float inv = 1.f / sum;
#pragma unroll 2
      for (int k = grp; k < c.y; k += GROUPS) {
        const long long s = slot_of(c, row, k);
        const float w = fast_exp2((a.lse_part[s] - m) * kLog2e) * inv;  // 0 for a part without keys
        const float4 q = *(reinterpret_cast<const float4*>(a.o_part + s * R) + lane + 32 * x);
        acc.x = fmaf(w, q.x, acc.x);
        acc.y = fmaf(w, q.y, acc.y);
        acc.z = fmaf(w, q.z, acc.z);
        acc.w = fmaf(w, q.w, acc.w);
      }
    }
    if (grp > 0) part_o[grp - 1][x][lane] = acc;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int k = 0; k < GROUPS - 1; ++k) {
        const float4 q = part_o[k][x][lane];
        acc.x += q.x;
        acc.y += q.y;
        acc.z += q.z;
        acc.w += q.w;
      }
      const long long o = (long long)c.z * a.M + row;
      store(o, (lane + 32 * x) * 4, acc);
      if (x == 0 && lane == 0 && a.lse) a.lse[o] = sum == 0.f ? -INFINITY : m + log2f(sum) * kLn2;
    }
    __syncthreads();
  }
}

}  // namespace pda
