// Attention over an expanded latent cache on the 5th-generation tensor cores:
// ragged query rows against keys [k_nope(head) | k_rope(shared)] and values of
// each head, with causal and window masks.
//
// A CTA takes 256 query rows of one sequence and head as two tiles A and B of
// 128 (the M dimension) and walks the keys 128 at a time:
//   S = Q K^T   [128, 128 keys]   K: 128 + 64 elements, both from shared memory
//   O += P V    [128, 128 dims]   K: 128 keys, P from TMEM, V from shared memory
// S (2 x 128 columns) and O (2 x 128) fill TMEM; the weights P, bf16, take the
// first 64 columns of their S. (bf16 because V is: the operands of a product have one
// type. A second term for what bf16 leaves of a weight would make 28 products of a
// step's 20; without it an output is 1.2 to 1.4 times as far off as one rounding.) The
// two tiles run half a step apart: while the softmax warps of one tile work, the
// tensor core has the other tile's products,
//   P_A V(t), Q_A K(t + 1), P_B V(t), Q_B K(t + 1), ...
// The products of a CTA execute in the order in which they are issued, so Q_A
// K(t + 1) overwrites the weights that P_A V(t) has read.
//
// Bounds: a step of both tiles is 2 x (12 x 68 + 8 x 64) = 2656 tensor cycles
// (an M = N = 128 product of 16 takes 64, 68 with both operands from shared
// memory), and 2 x 128 x 128 exponentials, 2048 cycles of the special function
// units: the tensor core is the bound, closely followed by the exponentials.
//
// Shared memory: Q 96 KB, two stages of K (48 KB each) and one V (32 KB, freed
// and filled in halves of 64 keys). No room for a second V.
//
// Roles (warps): 0 TMA producer, 1 and 2 MMA issuers of tiles A and B (which
// also zero the V rows that no query row sees: they may hold NaN, which a zero
// weight does not cancel), 3 idle; 4-7 softmax of tile A, 8-11 of tile B, a
// thread a query row. Every wait is bounded.
#pragma once

#include "pda_device.cuh"
#include "split_tma.cuh"  // instruction descriptors
#include "tcgen05.cuh"

namespace pda {

struct PrefillArgs {
  const int32_t* q_offsets;
  const int32_t* kv_offsets;
  uint16_t* out;  // bf16 [total_q, H, 128]
  float* lse;     // [total_q, H] or null
  int* err;
  int B, H, total_q, total_kv, max_q, tiles, units, causal_offset, window;
  bool by_rows;  // how units are numbered
  float scale_log2;
};

struct PrefillCfg {
  static constexpr int D = 128, QT = 128, KT = 128;
  static constexpr int CHUNK = 128 * 128;            // 128 rows of 64 bf16
  static constexpr int OFF_Q = 0;                    // 2 tiles x 3 chunks
  static constexpr int OFF_K = OFF_Q + 6 * CHUNK;    // 2 stages x 3 chunks
  static constexpr int OFF_V = OFF_K + 6 * CHUNK;    // 2 chunks
  static constexpr int OFF_BAR = OFF_V + 2 * CHUNK;
  // q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2][2], o_full[2], turn[2], drain[2]
  static constexpr int BARS = 22;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 384;
  static constexpr int COL_S = 0, COL_O = 256;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

// Keys [lo, hi) that query row i of a sequence of nq rows and nk keys sees.
__device__ __forceinline__ void prefill_visible(const PrefillArgs& a, int nq, int nk, int i, int& lo, int& hi) {
  long long pos = (long long)nk - 1;
  if (a.causal_offset >= 0) pos = (long long)a.causal_offset + i;
  else if (a.causal_offset == -2) pos = (long long)nk - nq + i;
  const long long h = a.causal_offset != -1 ? pos + 1 : (long long)nk;
  const long long l = a.window > 0 ? pos - a.window + 1 : 0;
  hi = (int)(h < 0 ? 0 : (h > nk ? nk : h));
  lo = (int)(l < 0 ? 0 : (l > nk ? nk : l));
}

// Units of the grid are 256 query rows of a sequence. Either every sequence has `tiles`
// units, the last tiles first; or (by_rows) sequence b has the units from q_offsets[b] /
// 256 + b on, the last units first: that leaves it enough for its rows wherever they
// begin, and all of them fit total_q / 256 + B however the rows are shared out.
__device__ __forceinline__ int prefill_begin(const PrefillArgs& a, int b) { return (__ldg(a.q_offsets + b) >> 8) + b; }

// Sequence (-1: none) and tile of unit u, for a whole warp.
__device__ __forceinline__ void prefill_unit(const PrefillArgs& a, int u, int lane, int& b, int& tile) {
  if (!a.by_rows) {
    b = u % a.B;
    tile = a.tiles - 1 - u / a.B;
    return;
  }
  // the sequences that begin at u or before: 32 at a time, closer and closer
  u = a.units - 1 - u;
  int base = 0, span = a.B;
  for (;;) {
    const int step = (span + 31) / 32, at = base + lane * step;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, lane * step < span && prefill_begin(a, min(at, a.B - 1)) <= u));
    b = base + (k - 1) * step;
    if (step == 1 || k == 0) break;
    base = b;
    span = min(step, a.B - base);
  }
  tile = b >= 0 ? u - prefill_begin(a, b) : 0;
}

// Whether a sequence's rows and keys lie within the tensors.
__device__ __forceinline__ bool prefill_fits(const PrefillArgs& a, int qb, int nq, int kb, int nk) {
  return qb >= 0 && nq >= 0 && nq <= a.total_q - qb && kb >= 0 && nk >= 0 && nk <= a.total_kv - kb;
}

// Records offsets of sequence b that do not fit (units found by rows may pass it over).
__device__ __forceinline__ void prefill_check(const PrefillArgs& a, int b) {
  const int qb = __ldg(a.q_offsets + b), kb = __ldg(a.kv_offsets + b);
  if (!prefill_fits(a, qb, __ldg(a.q_offsets + b + 1) - qb, kb, __ldg(a.kv_offsets + b + 1) - kb))
    record_error_at(a.err, kErrBadPage);
}

// D += A B with A (bf16, K-major) in TMEM.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// 32 consecutive TMEM columns of this thread's lane; the caller waits
// (tmem_wait_ld) before it uses them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's TMEM loads; the registers pass through so that no use moves above it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Weights 2^(s * scale - m) of 64 scores, as bf16 pairs, and their sum added to
// `sum`. (With a quarter of the exponentials as polynomials on the FMA pipe a
// step took a tenth fewer cycles, and the long case the same time: in a loop of it the
// GPU runs at its power limit, 990 W, at 1.64 GHz instead of 1.9: 8192 rows, 16 heads
// take 323 us there and 287 after a pause. Dividing by the sum of the rounded weights
// instead: three instructions more a pair, 342 us instead of 329, and no smaller error.)
__device__ __forceinline__ void weights64(const uint32_t* s, f32x2 scale2, f32x2 minus_m2, f32x2 (&sum)[2],
                                          uint32_t* p) {
#pragma unroll
  for (int k = 0; k < 64; k += 2) {
    const f32x2 x = f2_fma(f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale2, minus_m2);
    float u, v;
    f2_unpack(x, u, v);
    u = fast_exp2(u);
    v = fast_exp2(v);
    sum[(k >> 1) & 1] = f2_add(sum[(k >> 1) & 1], f2_pack(u, v));
    p[k >> 1] = pack_bf16x2(u, v);
  }
}

__global__ void __launch_bounds__(PrefillCfg::THREADS, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv,
                          const __grid_constant__ CUtensorMap map_r, const PrefillArgs a) {
  using C = PrefillCfg;
  constexpr unsigned FULL = 0xFFFFFFFFu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Heads vary fastest, so that the CTAs of one time read few sequences' keys.
  // The CTAs start in the order of their index; the longest work comes first,
  // so that the SMs finish close together. One sequence's tiles are in that
  // order from the last one down (a causal mask gives it the most keys). Of
  // several sequences every CTA ranks all units, (sequence, tile) pairs, by their
  // key tiles, a unit a thread; more units than threads keep their order.
  const int h = blockIdx.x % a.H, y = blockIdx.x / a.H;
  if (a.by_rows && h == 0 && tid == 0 && y < a.B) prefill_check(a, y);
  int b, tile;
  if (a.B > 1 && a.units <= C::THREADS) {  // (so there are no more sequences than threads)
    int* cost = reinterpret_cast<int*>(smem);
    int* mine = cost + C::THREADS;  // sequence, tile
    int pb = -1, pt = 0, nq = 0, nk = 0, c = -1;  // (-1: behind the last unit, or of no sequence)
    if (!a.by_rows) {
      if (tid < a.units) {
        pb = tid % a.B;
        pt = a.tiles - 1 - tid / a.B;
        nq = __ldg(a.q_offsets + pb + 1) - __ldg(a.q_offsets + pb);
        nk = __ldg(a.kv_offsets + pb + 1) - __ldg(a.kv_offsets + pb);
      }
    } else {
      int3* seq = reinterpret_cast<int3*>(mine + 4);  // first unit, rows, keys
      if (tid < a.B)
        seq[tid] = make_int3(prefill_begin(a, tid), __ldg(a.q_offsets + tid + 1) - __ldg(a.q_offsets + tid),
                             __ldg(a.kv_offsets + tid + 1) - __ldg(a.kv_offsets + tid));
      __syncthreads();
      if (tid < a.units) {
        const int u = a.units - 1 - tid;
        int x = 0, e = a.B;
        while (x < e) {
          const int mid = (x + e) >> 1;
          if (seq[mid].x <= u) x = mid + 1;
          else e = mid;
        }
        pb = x - 1;
        if (pb >= 0) {
          pt = u - seq[pb].x;
          nq = seq[pb].y;
          nk = seq[pb].z;
        }
      }
    }
    if (pb >= 0) {
      const int first = pt * 2 * C::QT, last = min(min(nq, a.max_q), first + 2 * C::QT) - 1;
      c = 0;
      if (last >= first) {
        int lo, hi, z;
        prefill_visible(a, nq, nk, first, lo, z);
        prefill_visible(a, nq, nk, last, z, hi);
        c = 1 + max(hi - lo, 0);
      }
    }
    cost[tid] = c;
    __syncthreads();
    int rank = 0;
    for (int k = 0; k < a.units; k += 4) {  // (entries behind the last unit are -1)
      const int4 o = *reinterpret_cast<const int4*>(cost + k);
      rank += (o.x > c || (o.x == c && k < tid)) + (o.y > c || (o.y == c && k + 1 < tid)) +
              (o.z > c || (o.z == c && k + 2 < tid)) + (o.w > c || (o.w == c && k + 3 < tid));
    }
    if (tid < a.units && rank == y) {
      mine[0] = pb;
      mine[1] = pt;
    }
    __syncthreads();
    b = mine[0];
    tile = mine[1];
    fence_proxy_async_smem();  // (Q lands where the costs lay)
    __syncthreads();
  } else {
    prefill_unit(a, y, lane, b, tile);
  }
  if (b < 0 || tile < 0) return;  // (offsets that decrease may give a tile in front of their sequence)
  const int qb = __ldg(a.q_offsets + b), nq_all = __ldg(a.q_offsets + b + 1) - qb;
  const int kb = __ldg(a.kv_offsets + b), nk = __ldg(a.kv_offsets + b + 1) - kb;
  if (!prefill_fits(a, qb, nq_all, kb, nk)) {
    if (threadIdx.x == 0) record_error_at(a.err, kErrBadPage);
    return;
  }
  const int row0 = tile * 2 * C::QT, rows = min(min(nq_all, a.max_q) - row0, 2 * C::QT);
  if (rows <= 0) return;

  const uint32_t sbase = smem_addr(smem);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [tile]
  uint64_t* k_full = q_full + 2;   // [stage]
  uint64_t* k_empty = k_full + 2;  // [stage]
  uint64_t* v_full = k_empty + 2;  // [half]
  uint64_t* v_empty = v_full + 2;  // [half]
  uint64_t* s_full = v_empty + 2;  // [tile] S in TMEM, and the products before it done
  uint64_t* p_full = s_full + 2;   // [tile][half] weights of 64 keys in TMEM
  uint64_t* o_full = p_full + 4;   // [tile] all products done
  uint64_t* turn = o_full + 2;     // [tile] its products of a step may be issued
  uint64_t* drain = turn + 2;      // [tile] after giving up: all its products done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* loads = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // K tiles, V halves asked for

  // Key tiles [t0, t1) of either query tile, and keys [lo, hi) that any row sees.
  int t0[2], t1[2], lo_u = 0, hi_u = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = row0 + x * C::QT, last = row0 + min(rows, (x + 1) * C::QT) - 1;
    t0[x] = t1[x] = 0;
    if (last >= first) {
      int lo, hi, z;
      prefill_visible(a, nq_all, nk, first, lo, z);
      prefill_visible(a, nq_all, nk, last, z, hi);
      if (hi > lo) {
        t0[x] = lo / C::KT;
        t1[x] = (hi + C::KT - 1) / C::KT;
        if (hi_u == 0) lo_u = lo;
        hi_u = max(hi_u, hi);
      }
    }
  }
  const bool has_a = t1[0] > t0[0], has_b = t1[1] > t0[1];
  const int tb = has_a && has_b ? min(t0[0], t0[1]) : has_a ? t0[0] : t0[1];
  const int te = has_a && has_b ? max(t1[0], t1[1]) : has_a ? t1[0] : t1[1];
  auto active = [&](int x, int t) { return t >= t0[x] && t < t1[x]; };
  // keys of tile t that no row sees must not meet the product as NaN
  auto ragged = [&](int t) { return t * C::KT < lo_u || (t + 1) * C::KT > hi_u; };

  if (tid < C::BARS) {
    uint64_t* bar = q_full + tid;
    const bool both = (bar >= k_empty && bar < v_full) || (bar >= v_empty && bar < s_full);  // both MMA warps
    mbar_init(bar, bar >= p_full && bar < o_full ? 128 : both ? 2 : 1);
    fence_mbar_init();
  }
  if (tid == 0) *abort_flag = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Registers: 384 x 168 at launch; the softmax warps hold a row of 128 scores.
  // 4 x 32 x 72 + 8 x 32 x 208 = 62464 of 64512.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ======================= TMA producer (one lane) =========================
      if (lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_kv) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_r) : "memory");
        bool ok = true;
        auto load_q = [&](int x) {
          mbar_arrive_expect_tx(&q_full[x], 3 * C::CHUNK);
          for (int c = 0; c < 3; ++c)
            tma_load_3d(sbase + C::OFF_Q + (3 * x + c) * C::CHUNK, &map_q, 64 * c, h, qb + row0 + x * C::QT, &q_full[x]);
        };
        auto load_k = [&](int t) {
          const int n = t - tb, st = n & 1;
          if (n >= 2) ok = ok && wait_or_abort(&k_empty[st], ((n >> 1) - 1) & 1, abort_flag, a.err);
          if (!ok) return;
          const uint32_t dst = sbase + C::OFF_K + st * 3 * C::CHUNK;
          mbar_arrive_expect_tx(&k_full[st], 3 * C::CHUNK);
          for (int x = 0; x < 4; ++x)  // (64-element column, 64 keys)
            tma_load_3d(dst + (x >> 1) * C::CHUNK + (x & 1) * (C::CHUNK / 2), &map_kv, (x >> 1) * 64, h,
                        kb + t * C::KT + (x & 1) * 64, &k_full[st]);
          tma_load_2d(dst + 2 * C::CHUNK, &map_r, 0, kb + t * C::KT, &k_full[st]);
        };
        if (has_a) load_q(0);
        if (te > tb) load_k(tb);
        if (has_b) load_q(1);
        int kloads = te > tb, vloads = 0;
        for (int t = tb; ok && t < te; ++t) {
          if (t + 1 < te) load_k(t + 1);
          if (ok && t + 1 < te) ++kloads;
          for (int half = 0; ok && half < 2; ++half) {
            const int n = t - tb;
            if (n >= 1) ok = wait_or_abort(&v_empty[half], (n - 1) & 1, abort_flag, a.err);
            if (!ok) break;
            const uint32_t dst = sbase + C::OFF_V + half * (C::CHUNK / 2);
            mbar_arrive_expect_tx(&v_full[half], C::CHUNK);
            tma_load_3d(dst, &map_kv, C::D, h, kb + t * C::KT + half * 64, &v_full[half]);
            tma_load_3d(dst + C::CHUNK, &map_kv, C::D + 64, h, kb + t * C::KT + half * 64, &v_full[half]);
            ++vloads;
          }
        }
        if (!ok) *abort_flag = 1;
        loads[0] = kloads;
        loads[1] = vloads;
      }
      __syncwarp();
    } else if (warp < 3) {
      // ======================= MMA issuers: tile A (warp 1), tile B (warp 2) =====
      // A warp's issue runs only a few products ahead of the tensor core, so what
      // it spends on barriers would leave the core idle: with a warp a tile, one
      // looks at its barriers while the other's products run. Both follow every
      // key tile, so that no barrier gets two phases ahead of either.
      const int x = warp - 1;
      const bool leader = elect_one();
      bool ok = true;
      auto agreed = [&](bool v) { return __all_sync(FULL, v); };
      auto scores = [&](int t) {  // S_x = Q_x K(t)^T, K(t) has landed
        const int st = (t - tb) & 1;
        if (!active(x, t)) {
          if (lane == 0) mbar_arrive(&k_empty[st]);
          __syncwarp();
          return;
        }
        if (t == t0[x]) {
          ok = agreed(wait_or_abort(&q_full[x], 0, abort_flag, a.err));
          if (!ok) return;
        }
        tmem_fence_after();
        if (leader) {
          constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
          const uint64_t qd = umma_desc(sbase + C::OFF_Q + x * 3 * C::CHUNK, 16, 1024, kSw128);
          const uint64_t kd = umma_desc(sbase + C::OFF_K + st * 3 * C::CHUNK, 16, 1024, kSw128);
#pragma unroll
          for (int s = 0; s < 12; ++s) {
            const int off = ((s >> 2) * C::CHUNK + (s & 3) * 32) >> 4;
            umma_f16(tmem + C::COL_S + x * 128, qd + off, kd + off, idesc, s > 0);
          }
          umma_commit(&s_full[x]);
          umma_commit(&k_empty[st]);
        }
        __syncwarp();
      };
      auto key_tile = [&](int t) {
        return agreed(wait_or_abort(&k_full[(t - tb) & 1], ((t - tb) >> 1) & 1, abort_flag, a.err));
      };
      // The tiles' products alternate step by step. Left alone the two drift into
      // step, both with their softmax and then both with their products.
      auto my_turn = [&](int n) {
        return x == 0 && n == 0 ? true : agreed(wait_or_abort(&turn[x], (n - (x == 0 ? 1 : 0)) & 1, abort_flag, a.err));
      };
      if (te > tb) {
        ok = key_tile(tb);
        if (ok) scores(tb);
      }
      for (int t = tb; ok && t < te; ++t) {
        const int n = t - tb;
        ok = (t + 1 == te || key_tile(t + 1)) &&
             agreed(wait_or_abort(&v_full[0], n & 1, abort_flag, a.err) &&
                    wait_or_abort(&v_full[1], n & 1, abort_flag, a.err));
        if (!ok) break;
        if (ragged(t)) {  // V rows that no query row sees become zeros; both warps write the same
          for (int r = lane; r < C::KT; r += 32) {
            const int key = t * C::KT + r;
            if (key >= lo_u && key < hi_u) continue;
            uint8_t* row = smem + C::OFF_V + r * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int cc = (c + r) & 7;
              *reinterpret_cast<uint4*>(row + cc * 16) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(row + C::CHUNK + cc * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (active(x, t)) {  // O_x += P_x V(t), as the halves of P_x come
          const uint64_t vd = umma_desc(sbase + C::OFF_V, C::CHUNK, 1024, kSw128);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && agreed(wait_or_abort(&p_full[2 * x + half], (t - t0[x]) & 1, abort_flag, a.err));
            if (half == 0 && ok) ok = my_turn(n);
            if (!ok) break;
            tmem_fence_after();
            if (leader) {
              constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, true);
#pragma unroll
              for (int s = 4 * half; s < 4 * half + 4; ++s)
                umma_f16_ts(tmem + C::COL_O + x * 128, tmem + C::COL_S + x * 128 + 8 * s, vd + ((s * 2048) >> 4),
                            idesc, t > t0[x] || s > 0);
              umma_commit(&v_empty[half]);
              if (half == 1 && t + 1 == t1[x]) umma_commit(&o_full[x]);
            }
            __syncwarp();
          }
          if (!ok) break;
        } else {
          ok = my_turn(n);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive(&v_empty[0]);
            mbar_arrive(&v_empty[1]);
          }
          __syncwarp();
        }
        if (t + 1 < te) scores(t + 1);
        if (lane == 0) mbar_arrive(&turn[1 - x]);
        __syncwarp();
      }
      if (!ok) *abort_flag = 1;
      __syncwarp();
    }
  } else {
    // ======================= softmax: a thread a query row ======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr float kLn2 = 0.69314718055994531f, kUnset = -1e30f;
    const int x = (warp - 4) >> 2, q4 = warp & 3, r = 32 * q4 + lane;
    const int i = row0 + x * C::QT + r;
    const bool live = x * C::QT + r < rows;
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    const uint32_t s_tm = tmem + lane_off + C::COL_S + x * 128, o_tm = tmem + lane_off + C::COL_O + x * 128;
    int lo = 0, hi = 0;
    if (live) prefill_visible(a, nq_all, nk, i, lo, hi);
    float m = kUnset, l = 0.f;
    bool ok = true;
    for (int t = t0[x]; t < t1[x]; ++t) {
      ok = __all_sync(FULL, wait_or_abort(&s_full[x], (t - t0[x]) & 1, abort_flag, a.err));
      if (!ok) break;
      tmem_fence_after();
      // Loads of 32 scores run beside the maximum of the 32 before.
      uint32_t s[128];
      const int j0 = t * C::KT;
      const bool masked = __any_sync(FULL, lo > j0 || hi < j0 + C::KT);
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      tmem_ld32_async(s_tm, s);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tmem_wait_ld32(s + 32 * c);
        if (c < 3) tmem_ld32_async(s_tm + 32 * (c + 1), s + 32 * (c + 1));
        if (masked) {
#pragma unroll
          for (int k = 32 * c; k < 32 * c + 32; ++k)
            if (j0 + k < lo || j0 + k >= hi) s[k] = 0xFF800000u;  // -inf
        }
#pragma unroll
        for (int k = 32 * c; k < 32 * c + 32; k += 2)
          mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
      }
      const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.scale_log2;
      // The running maximum moves only when a weight would pass 2^8; the warp
      // then moves what its rows have added up so far.
      if (__any_sync(FULL, top - m > 8.f)) {
        const float m_new = fmaxf(m, top), al = fast_exp2(m - m_new);
        m = m_new;
        l *= al;
        if (t > t0[x]) {  // O is idle: S of this tile was ready after all products before it
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32_async(o_tm + 32 * c, o);
            tmem_wait_ld32(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
            tmem_st32(o_tm + 32 * c, o);
          }
        }
      }
      // The weights go to the tensor core in halves: it multiplies the first 64
      // keys' while the second 64 keys' are computed.
      const f32x2 sc2 = f2_pack(a.scale_log2, a.scale_log2), nm2 = f2_pack(-m, -m);
      f32x2 sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[32];
        weights64(s + 64 * half, sc2, nm2, sum2, p);
        tmem_st32(s_tm + 32 * half, p);
        tmem_wait_st();
        tmem_fence_before();
        mbar_arrive(&p_full[2 * x + half]);
      }
      float u, v;
      f2_unpack(f2_add(sum2[0], sum2[1]), u, v);
      l += u + v;
    }
    if (!ok) *abort_flag = 1;
    // ---- normalise and store --------------------------------------------------
    const bool any = t1[x] > t0[x];
    if (ok && any) ok = wait_or_abort(&o_full[x], 0, abort_flag, a.err);
    ok = __all_sync(FULL, ok);
    if (ok) {
      tmem_fence_after();
      // (the sum is 0 without keys; NaN of a score that is NaN or +inf passes on)
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long row = (long long)(qb + i) * a.H + h;
#pragma unroll 2
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (any) {
          tmem_ld32_async(o_tm + 32 * c, o);
          tmem_wait_ld32(o);
        }
        if (live) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k] = inv == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * C::D + 32 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      }
      if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      *abort_flag = 1;
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (*abort_flag) {  // some role gave up: what was issued finishes before its memory goes away
    constexpr long long lim = kWaitTimeoutCycles / 16;
    if (warp == 0 && lane == 0) {  // copies: the last of each kind into each place
      if (has_a) mbar_wait(&q_full[0], 0, a.err, lim);
      if (has_b) mbar_wait(&q_full[1], 0, a.err, lim);
      for (int n = max(0, loads[0] - 2); n < loads[0]; ++n) mbar_wait(&k_full[n & 1], (n >> 1) & 1, a.err, lim);
      for (int n = max(0, loads[1] - 2); n < loads[1]; ++n) mbar_wait(&v_full[n & 1], (n >> 1) & 1, a.err, lim);
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace pda
