// qsa_dense_decode: softmax attention of one token over every token its
// sequence holds in the paged cache, split over the cache's length and joined;
// on request the attention weight that each micro-block received is added into
// a running total (the total qsa_evict selects by).
//
//   z_t = scale q . k_t,  lse = log sum_t exp(z_t),  o = sum_t exp(z_t - lse) v_t
//   mass_out[s][b] = decay mass_in[s][b] + sum_{q of s} sum_h sum_{t in b} exp(z_t - lse)
//
// What bounds it: the K/V bytes, each read once (2 x 256 elements per token and
// KV head).  At 16 Q heads per KV head that is 16 flop per BF16 byte, far below
// the card's balance, so the matrix work runs on mma.sync with the 16 rows the
// group fills; a tcgen05 tile would have 128 rows, K and V rows interleaved in
// its operand, and an instruction floor that alone exceeds the copy time.
//
// Split.  A tile is 16 tokens of one (query, KV head): 4 micro-blocks, one contiguous
// run of the page (16 KiB BF16, 8 KiB e4m3).  The tiles of all pairs,
// query-major, form one list that the CTAs (one per SM) share evenly, so ragged
// lengths leave no SM idle; the lengths are read on the device (no host copy of
// q_pos).  A pair inside one CTA is written to out / lse at once; of the others
// a CTA holds at most two pieces (its first and its last), so the partials need
// 2 CTAs x 16 rows of workspace whatever the batch, and a second small kernel
// joins them and adds up the weights.
//
// CTA = consumer warps + 1 copy warp, one CTA per SM.  A consumer warp takes whole
// tiles (S = Q K^T, a running maximum and sum, O += P V over all 256 dims) with no
// exchange until the pair's piece ends; its 16 x 256 accumulator takes 128
// registers.  BF16: 6 consumers, 255 registers each (8 warps or fewer), and 12
// tiles in flight.  e4m3: half the bytes a token, so the arithmetic counts: 8
// consumers with 224 registers, which the copy warp's group gives up, and 24
// tiles.  The copy warp resolves 32 tiles' pages at once, one batch ahead, a lane
// each moves a tile, and it brings the Q rows of the next pairs.
//
// Measured on one B200 (time of the call, share of the 6.54 TB/s copy rate; a range is
// from a card at rest to one that has been busy):
//   BF16, 32 x 131,072 tokens, 24/2 heads     1,181-1,246 us   105-111%
//   BF16, 8 x 32,768 tokens, 16/2 heads          85-87 us      94-97%
//   e4m3, 64 x 16K-262K tokens, 12/1 heads      495-525 us     80-85%; power-capped, ALU 38%,
//                                                              tensor 32% of active cycles
//   BF16, 16 x 9K-16K tokens, 24/2, with totals   73-75 us     82-84%
//   BF16, 1 x 4,096 tokens, 16/2                  9.5 us       of it 7 main kernel, 3 join
//   BF16, 200 x 1-700 tokens, 3/1                 15 us
// What did not pay for e4m3: 6 or 7 consumers (512, 526 us then), 32-token tiles
// (no change), one tile's products beside the last one's values (508 against 494),
// e4m3 matrix instructions (25 to 38 cycles against 8 for FP16 ones of half the depth).
#include "qsa_common.cuh"
#include "tensor_map.cuh"

namespace {

using namespace qsa;

constexpr int kTile = 16;                        // tokens of one matrix product
constexpr int kTileRuns = kTile / kRatio;        // 4 micro-blocks
constexpr int kTilesPerPage = kPage / kTile;
constexpr int kPieceCost = 8;                    // what a pair costs a CTA beside its tiles, in tiles
// Places a CTA takes at least, so that one short sequence is not cut into pieces whose
// join costs more than they save (1 x 4,096 tokens, 16/2 heads: 10.1 us with 4, 10.2 with
// 6, 11.3 with 8); with more pairs than that a CTA may hold one pair alone (167 queries
// of 1 to 4 tokens, 12/1 heads, e4m3: 10.3 us, 15.4 without this).
constexpr int kMinPlaces = 4;
constexpr int kMaxCtas = 256;                    // partial slots reserved: 2 per CTA
constexpr int kQStride = kHeadDim * 2 + 16;      // Q rows 528 B apart: conflict-free 16-byte fragment reads
constexpr int kSlice = 32;                       // dims of O that the warps join at once
constexpr int kSlices = kHeadDim / kSlice;
constexpr int kSliceBytes = 16 * kSlice * 4;     // of one warp
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kTab = 48;  // queries whose length a CTA keeps in shared memory
// Q rows of the next pairs: 32 rows' room, as many groups of G rows as fit (6 at most);
// row 31 stays zero for the rows beyond G
constexpr int kQRows = 32, kMaxQ = 6;
constexpr int kBarConsumers = 1;
// The running maximum a warp subtracts may lag the true one by this much (base
// 2), so that O is seldom rescaled: exp2 stays below 2^8, harmless in fp32 sums
// and in the BF16 weights, whose precision is relative.
constexpr float kLag = 8.f;
// e4m3 V takes FP16 weights, whose precision is relative from 2^-14 up only.  What is
// subtracted lies 7 below the running maximum there, so the largest weights are between
// 2^7 and 2^15 and a tile may hold weights down to 2^-21 of theirs; one with a smaller
// weight takes the wide form (see as_operand).
constexpr float kLeastF16 = 0x1p-14f;

// BF16: runs lie in shared memory as in the cache (128-byte swizzled rows), a
// plain bulk copy each tile.  e4m3: the cache's rows are plain; a tensor-map copy
// swizzles them on the way, as [row][2 halves of 128 B].
template <bool F8>
struct Lay {
  static constexpr int kWarps = F8 ? 8 : 6;  // consumer warps
  static constexpr int kConsumerThreads = kWarps * 32;
  static constexpr int kThreads = kConsumerThreads + (F8 ? 128 : 32);  // + the copy warp (e4m3: in a warpgroup)
  // e4m3: 384 threads are launched with 168 registers; the consumers' two warpgroups
  // take 224, the copy warp's keeps 56: 256 x 224 + 128 x 56 = 384 x 168
  static constexpr int kRegs = 168, kConsumerRegs = 224, kCopyRegs = 56;
  static_assert(256 * kConsumerRegs + 128 * kCopyRegs <= 384 * kRegs, "more registers than were launched");
  static constexpr int kRunBytes = 2 * kRatio * kHeadDim * (F8 ? 1 : 2);
  static constexpr int kStageBytes = kTileRuns * kRunBytes;
  static constexpr int kStages = F8 ? 24 : 12;
  static constexpr float kBias = F8 ? 7.f : 0.f;  // weights are relative to 2^(maximum - kBias): see kLeastF16
  // Tile T and tile T + kStages, which reuses its stage, belong to one warp: it has
  // seen the stage's last phase end before it waits for the next.  A parity wait
  // cannot tell a phase from the one two before, so another warp could run ahead.
  static_assert(kStages % kWarps == 0, "a stage has one consumer");
  static constexpr int kOffQ = kStages * kStageBytes;           // the pieces' Q rows
  static constexpr int kOffML = kOffQ + kQRows * kQStride;      // [warp][16 rows] (m, l)
  static constexpr int kOffScale = kOffML + kWarps * 16 * 8;    // e4m3: logit scale of each row
  static constexpr int kOffHeld = kOffScale + kMaxQ * 16 * 4;   // each warp's held stage
  static constexpr int kOffValid = kOffHeld + 8 * 4;          // tokens in each stage
  static constexpr int kOffPlan = (kOffValid + kStages * 4 + 15) & ~15;
  static constexpr int kOffTab = kOffPlan + 16 * 8;             // (len, seq) of queries q0 ..
  static constexpr int kOffBar = kOffTab + kTab * 8;            // full, empty, Q full, Q empty
  static constexpr int kOffAbort = kOffBar + 2 * (kStages + kMaxQ) * 8;
  static constexpr int kSmem = kOffAbort + 16;
  static constexpr int kIssue = F8 ? 8 : 3;  // copy-warp lanes that wait and issue together, a tile each
  static_assert(kSmem <= 232448, "shared memory budget");
  static constexpr int kRounds = F8 ? 2 : 1;  // the join puts O into a held stage in so many parts
  static_assert(kSlices * kSliceBytes <= kRounds * kStageBytes, "a part of a warp's O fits the stage it holds");
};

struct DenseArgs {
  const uint8_t* kv;
  const int32_t* bt;
  int32_t num_pages, max_seqs, mpps, hkv;
  const __nv_bfloat16* q;
  int32_t nq, hq, G;
  const int32_t* q_seq;
  const int32_t* q_pos;
  float scale_log2;
  int2* span;       // [nq][hkv] first and last CTA that hold tiles of the pair; last < first: none
  float* part_lse;  // [2 CTAs][G], base 2
  float* part_o;    // [2 CTAs][G][256], normalised
  __nv_bfloat16* out;
  float* lse;
  float* bsum;  // [nq][hq][max tiles][4] sums of exp2(z - bmax) per micro-block, or null
  float* bmax;  // [nq][hq][max tiles]
  int32_t ctas;
  int32_t q_bufs;  // groups of Q rows held at once
  int32_t* st;
  CUtensorMap tm;  // e4m3: kv_pages as rows of 128 bytes, boxes of one tile
};

// Tokens query q attends to; 0 for a padding row (q_seq < 0), an empty context
// (q_pos == -1) and, flagged, for a sequence or position out of range.
__device__ __forceinline__ int query_len(const DenseArgs& a, int q, bool report) {
  const int seq = a.q_seq[q], p = a.q_pos[q];
  if (seq < 0 || p == -1) return 0;
  if (seq >= a.max_seqs) {
    if (report) flag(a.st, QSA_DEV_BAD_SEQ);
    return 0;
  }
  if (p < 0 || (int64_t)p >= (int64_t)a.mpps * kPage) {
    if (report) flag(a.st, QSA_DEV_BAD_POS);
    return 0;
  }
  return p + 1;
}

__device__ __forceinline__ int tiles_of(int len) {
  return (len + kTile - 1) / kTile;
}

// The list that the CTAs share out: every pair takes kPieceCost places (what
// joining its warps costs beside a tile), then one per tile.
struct Shares {
  int n, base, rem;  // CTAs; the first `rem` take base + 1 places, the others base
};
__device__ __forceinline__ Shares make_shares(int total, int pairs, int ctas) {
  Shares s;
  s.n = min(ctas, max(pairs, (total + kMinPlaces - 1) / kMinPlaces));
  s.base = total / s.n;
  s.rem = total - s.base * s.n;
  return s;
}
__device__ __forceinline__ int share_begin(const Shares& s, int c) { return c * s.base + min(c, s.rem); }
__device__ __forceinline__ int share_of(const Shares& s, int x) {  // the CTA that holds place x
  const int cut = s.rem * (s.base + 1);
  return x < cut ? x / (s.base + 1) : s.rem + (x - cut) / s.base;
}

__device__ __forceinline__ int cost_of(int tiles) {  // a pair of one tile joins nothing
  return tiles > 1 ? kPieceCost : 1;
}
__device__ __forceinline__ int places_of(int len) {
  return len ? tiles_of(len) + cost_of(tiles_of(len)) : 0;
}

// A CTA's position in the list: a piece of pair (q, g).
struct Walk {
  int q, g;
  int len, seq;  // of the query
  int t0, t1;    // tiles of the pair in this CTA
  int begin;     // the pair's first place
  int q_tab;     // the query of tab[0]
  const int2* tab;
};

__device__ __forceinline__ bool set_span(Walk& w, int x0, int x1) {
  const int nt = tiles_of(w.len), lo = w.begin + cost_of(nt);
  w.t0 = max(0, x0 - lo);
  w.t1 = min(nt, x1 - lo);
  return w.t1 > 0;
}

// Step to the next pair with tiles in the share; false when there is none.
__device__ __forceinline__ bool next_piece(const DenseArgs& a, Walk& w, int x1) {
  const int begin = w.begin + places_of(w.len);
  if (begin >= x1) return false;
  w.begin = begin;
  if (w.g + 1 < a.hkv) {
    ++w.g;
  } else {
    do {
      ++w.q;
      const int k = w.q - w.q_tab;
      const int2 e = k < kTab ? w.tab[k] : make_int2(query_len(a, w.q, false), a.q_seq[w.q]);
      w.len = e.x;
      w.seq = e.y;
    } while (w.len == 0);
    w.g = 0;
  }
  return set_span(w, 0, x1);
}

// Bounded wait; false (and the abort flag) when the limit passed.
__device__ __forceinline__ bool wait_bar(const DenseArgs& a, uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 255u) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        flag(a.st, QSA_DEV_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// ------------------------------------------------------------------ copy warp

// 2-D tensor-map copy into this CTA's shared memory, completing on an mbarrier.
__device__ __forceinline__ void tma2d(uint32_t sdst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                      uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3}], [%4], %5;" ::"r"(sdst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}

template <bool F8>
__device__ void copy_warp(const DenseArgs& a, uint8_t* smem, Walk w, int x1) {
  using LY = Lay<F8>;
  const int lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem);
  const uint32_t full = smem_u32(smem + LY::kOffBar), empty = full + LY::kStages * 8;
  int* valid = reinterpret_cast<int*>(smem + LY::kOffValid);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LY::kOffAbort);
  const uint64_t policy = l2_policy_evict_first(), policy_q = l2_policy_evict_normal();
  uint32_t T = 0, n_issued = 0;  // tiles taken up, tiles whose copies were issued
  uint32_t piece = 0, qi = 0, lap = 0;  // pieces whose Q rows were issued; the next one's place and its round
  const uint32_t q_full = empty + LY::kStages * 8, q_empty = q_full + kMaxQ * 8;
  auto lookup = [&](const Walk& at, int t) {
    int page = -1;
    if (t < at.t1) page = __ldg(a.bt + (int64_t)at.seq * a.mpps + t / kTilesPerPage);
    return page;
  };
  int page = lookup(w, w.t0 + lane);
  bool more = true, stop = false;
  while (more && !stop) {
    {  // Q rows of the group, 512 bytes each
      if (lap > 0 && !wait_bar(a, q_empty + qi * 8, (lap - 1) & 1u, abort_flag)) stop = true;
      if (__any_sync(0xffffffffu, stop)) {
        stop = true;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(q_full + qi * 8, a.G * kHeadDim * 2);
      __syncwarp();
      if (lane < a.G)
        bulk_g2s(smem_u32(smem + LY::kOffQ) + (qi * a.G + lane) * kQStride,
                 a.q + ((size_t)w.q * a.hq + (size_t)w.g * a.G + lane) * kHeadDim, kHeadDim * 2, q_full + qi * 8,
                 policy_q);
      ++piece;
      if (++qi == (uint32_t)a.q_bufs) {
        qi = 0;
        ++lap;
      }
    }
    // lane = tile: pages of 32 tiles at a time, the next batch's (of this pair or the
    // next one) requested before this batch's copies
    Walk after = w;
    more = next_piece(a, after, x1);
    const int page_after = more ? lookup(after, after.t0 + lane) : -1;
    for (int tb = w.t0; tb < w.t1 && !stop; tb += 32) {
      const int page_next = lookup(w, tb + 32 + lane);
      const int n = min(32, w.t1 - tb), t = tb + lane;
      const bool bad = page < 0 || page >= a.num_pages;
      if (lane < n && bad) flag(a.st, QSA_DEV_BAD_PAGE);
      const int tok = min(kTile, w.len - t * kTile);
      const int runs = (tok + kRatio - 1) / kRatio;  // whole micro-blocks that hold a token
      const uint8_t* src = a.kv + (((size_t)page * a.hkv + w.g) * kBlocksPerPage +
                                   (size_t)(t % kTilesPerPage) * kTileRuns) * LY::kRunBytes;
      const uint32_t mine = T + lane;
      const int stage = (int)(mine % LY::kStages);
      const uint32_t bar = full + stage * 8, dst = ring + stage * LY::kStageBytes;
      for (int i0 = 0; i0 < n; i0 += LY::kIssue) {
        const bool on = lane >= i0 && lane < min(n, i0 + LY::kIssue);
        bool ok = true;
        if (on && mine >= LY::kStages)
          ok = wait_bar(a, empty + stage * 8, (mine / LY::kStages - 1) & 1u, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {  // the tiles before these have been issued, these have not
          n_issued = T + i0;
          stop = true;
          break;
        }
        if (on) {
          valid[stage] = bad ? 0 : tok;
          if (bad) {
            mbar_arrive(bar);
          } else {
            if constexpr (F8) {  // the whole tile: what lies behind the end is the page's own
              mbar_arrive_expect_tx(bar, LY::kStageBytes);
              tma2d(dst, &a.tm, 0,
                    ((page * a.hkv + w.g) * kBlocksPerPage + t % kTilesPerPage * kTileRuns) * 2 * kRatio * 2, bar,
                    policy);
            } else {
              mbar_arrive_expect_tx(bar, runs * LY::kRunBytes);
              bulk_g2s(dst, src, runs * LY::kRunBytes, bar, policy);
            }
          }
        }
      }
      if (!stop) n_issued = T + n;
      T += n;
      page = page_next;
    }
    w = after;
    page = page_after;
  }
  // never leave the CTA with copies in flight: each lane waits for one stage's last copy
  const uint32_t left = min(n_issued, (uint32_t)LY::kStages), left_q = min(piece, (uint32_t)a.q_bufs);
  uint32_t bar = 0, parity = 0;
  if (lane < (int)left) {
    const uint32_t t = n_issued - 1 - lane;
    bar = full + (t % LY::kStages) * 8;
    parity = (t / LY::kStages) & 1u;
  } else if (lane >= 24 && lane - 24 < (int)left_q) {
    const uint32_t t = piece - 1 - (lane - 24);
    bar = q_full + (t % a.q_bufs) * 8;
    parity = (t / a.q_bufs) & 1u;
  }
  static_assert(LY::kStages <= 24 && kMaxQ <= 8, "a lane per copy that may be in flight");
  if (bar) {
    const uint64_t s0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
      if (global_timer_ns() - s0 > kWaitLimitNs) break;
  }
  __syncwarp();
}

// ------------------------------------------------------------------ consumers

// 2^x, denormal results flushed: below 2^-126 a weight adds nothing to a sum that holds one of 2^-8 or more
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two FP16 values that are e4m3 values, as BF16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
}

// Which token of the tile a lane's logits and V rows belong to: columns n = 2tq + e of
// S's n-tile j (lane tq of each quad holds e = 0, 1) are micro-block 2j + e, row tq ^ e
// (BF16) or tq ^ 2e (e4m3).  K's columns n, n + 1 are then read from rows whose swizzles
// send the same chunks to different halves of the banks, and V's four quad lanes from
// four different rows: both fragments come in conflict-free 16-byte reads.
__device__ __forceinline__ int tile_run(int j, int e) { return 2 * j + e; }
template <bool F8>
__device__ __forceinline__ int tile_row(int tq, int e) {
  return F8 ? tq ^ (2 * e) : tq ^ e;
}

template <bool F8>
__device__ void consumers(const DenseArgs& a, uint8_t* smem, Walk w, const Shares& sh, int x1) {
  using LY = Lay<F8>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring = smem_u32(smem);
  const uint32_t full = smem_u32(smem + LY::kOffBar), empty = full + LY::kStages * 8;
  const uint32_t q_full = empty + LY::kStages * 8, q_empty = q_full + kMaxQ * 8;
  const volatile int* valid = reinterpret_cast<const volatile int*>(smem + LY::kOffValid);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LY::kOffAbort);
  int* held_s = reinterpret_cast<int*>(smem + LY::kOffHeld);
  float2* ml = reinterpret_cast<float2*>(smem + LY::kOffML);
  float* scales = reinterpret_cast<float*>(smem + LY::kOffScale);
  constexpr int kWarps = LY::kWarps, kConsumerThreads = LY::kConsumerThreads;
  const int G = a.G;
  const int64_t max_tiles = (int64_t)a.mpps * kTilesPerPage;

  // K: column n = gq of n-tile j, V: this lane's tokens (j, e)
  const int ke = gq & 1, kr = tile_row<F8>(gq >> 1, ke);
  uint32_t k_off[2], v_off[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    k_off[j] = tile_run(j, ke) * LY::kRunBytes + kr * (F8 ? 256 : 128);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = tile_row<F8>(tq, e);
      // BF16: V row 4 + r of the run, chunk (gq >> 1) + 4 (gq & 1) of each 64-dim atom;
      // e4m3: 128-byte rows 8 + 2r + half of the run, 16-dim chunk gq
      v_off[j][e] = tile_run(j, e) * LY::kRunBytes +
                    (F8 ? 1024 + r * 256 + ((gq ^ (2 * r)) << 4)
                        : (4 + r) * 128 + ((((gq >> 1) + 4 * (gq & 1)) ^ (4 + r)) << 4));
    }
  }

  uint32_t T_base = 0;
  uint32_t qi = 0, lap = 0;  // place and round of the piece's Q rows
  for (;;) {
    const int n_tiles = w.t1 - w.t0;
    // ---- Q rows of the group (for the rows beyond it, the one that stays zero)
    const uint32_t q_at = smem_u32(smem + LY::kOffQ), qb = q_at + qi * G * kQStride;
    const uint32_t q_row0 = gq < G ? qb + gq * kQStride : q_at + (kQRows - 1) * kQStride;
    const uint32_t q_row1 = gq + 8 < G ? qb + (gq + 8) * kQStride : q_at + (kQRows - 1) * kQStride;
    if (!*abort_flag) wait_bar(a, q_full + qi * 8, lap & 1u, abort_flag);
    __syncwarp();
    const int rank = (int)((warp + kWarps - T_base % kWarps) % kWarps);  // this warp's first tile of the piece
    const bool lone = n_tiles == 1;  // one warp has the piece; the others only let its Q rows go
    if (lone && rank != 0) {
      if (lane == 0) mbar_arrive(q_empty + qi * 8);
      if (++qi == (uint32_t)a.q_bufs) {
        qi = 0;
        ++lap;
      }
      ++T_base;
      if (!next_piece(a, w, x1)) break;
      continue;
    }
    float sc0 = a.scale_log2, sc1 = a.scale_log2;
    if constexpr (F8) {
      float* row_scale = scales + qi * 16;
      // FP16 operands: each row is scaled by a power of two that puts its largest element
      // into [2^13, 2^14), and its logit scale takes the factor back.  An element is off by
      // at most 2^-38 of the row's largest (half of FP16's smallest step), and exact from
      // 2^-30 of it up, where FP16's steps of 2^-24 hold BF16's 8 bits
      for (int row = lone ? 0 : warp; row < G; row += lone ? 1 : kWarps) {
        const uint4 v = lds128(qb + row * kQStride + lane * 16);
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t mx = 0;  // largest magnitude, as ordered bits
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = max(mx, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
        mx = __reduce_max_sync(0xffffffffu, mx);
        const int ex = (int)(mx >> 7);  // biased exponent
        // -114 for the largest floats; 126 keeps 2^-up a normal number for the smallest
        const int up = ex == 255 ? 0 : min(126, 127 + 13 - ex);
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 h = __floats2half2_rn(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xffff0000u) * f);
          x[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        sts128(qb + row * kQStride + lane * 16, make_uint4(x[0], x[1], x[2], x[3]));
        if (lane == 0) row_scale[row] = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
      }
      fence_proxy_async();  // these writes come before the copy of the piece after next
      if (lone)
        __syncwarp();
      else
        named_bar_sync(kBarConsumers, kConsumerThreads);
      if (gq < G) sc0 = row_scale[gq];
      if (gq + 8 < G) sc1 = row_scale[gq + 8];
    }

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[32][4];
#pragma unroll
    for (int nt = 0; nt < 32; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;

    int held = -1;
    // the tile of this warp's step ti has landed: its stage; -1 when the wait was given up
    auto landed = [&](int ti) {
      const uint32_t T = T_base + ti;
      const int stage = (int)(T % LY::kStages);
      const bool got = !*abort_flag && wait_bar(a, full + stage * 8, (T / LY::kStages) & 1u, abort_flag);
      __syncwarp();
      return __all_sync(0xffffffffu, got) ? stage : -1;
    };
    // ---- S = Q K^T of the tile at kb: two n-tiles of 8 tokens
    auto products = [&](uint32_t kb, float(&s)[2][4]) {
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if constexpr (F8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 64 dims: lane tq holds dims 64i + 16tq .. + 15
          const uint32_t qo = (4 * i + tq) * 32;
          const uint4 qa0 = lds128(q_row0 + qo), qa1 = lds128(q_row0 + qo + 16);
          const uint4 qc0 = lds128(q_row1 + qo), qc1 = lds128(q_row1 + qo + 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 kk =
                lds128(kb + k_off[j] + (i >> 1) * 128 + (((4 * (i & 1) + tq) ^ (2 * kr + (i >> 1))) << 4));
            const uint4 k0 = e4m3x8_to_f16x8(make_uint2(kk.x, kk.y)), k1 = e4m3x8_to_f16x8(make_uint2(kk.z, kk.w));
            mma_f16_16816(s[j], qa0.x, qc0.x, qa0.y, qc0.y, k0.x, k0.y);
            mma_f16_16816(s[j], qa0.z, qc0.z, qa0.w, qc0.w, k0.z, k0.w);
            mma_f16_16816(s[j], qa1.x, qc1.x, qa1.y, qc1.y, k1.x, k1.y);
            mma_f16_16816(s[j], qa1.z, qc1.z, qa1.w, qc1.w, k1.z, k1.w);
          }
        }
      } else {
        float s2[2][4];  // a second accumulator each: half the chain of dependent products
#pragma unroll
        for (int j = 0; j < 2; ++j) s2[j][0] = s2[j][1] = s2[j][2] = s2[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 32 dims of atom i / 2: lane tq holds chunk 2tq + i % 2
          const int ch = 2 * tq + (i & 1);
          const uint4 qa = lds128(q_row0 + (8 * (i >> 1) + ch) * 16);
          const uint4 qc = lds128(q_row1 + (8 * (i >> 1) + ch) * 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 kk = lds128(kb + k_off[j] + (i >> 1) * 1024 + ((ch ^ kr) << 4));
            mma_bf16_16816(s[j], qa.x, qc.x, qa.y, qc.y, kk.x, kk.y);
            mma_bf16_16816(s2[j], qa.z, qc.z, qa.w, qc.w, kk.z, kk.w);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[j][c] += s2[j][c];
      }
    };
    // ---- S to weights: mask, running maximum and sum (base 2; the scale is positive, so the
    // largest product is the largest logit).  The result: whether the tile is wide, that is,
    // e4m3 V and a weight below FP16's normal numbers (see as_operand).
    auto weigh = [&](int ti, int nv, float(&p)[2][4]) {
      auto seen = [&](int j, int e) { return tile_run(j, e) * kRatio + tile_row<F8>(tq, e) < nv; };
      if (nv != kTile) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!seen(j, e)) p[j][e] = p[j][2 + e] = -INFINITY;
      }
      float r0 = fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[1][0], p[1][1]));
      float r1 = fmaxf(fmaxf(p[0][2], p[0][3]), fmaxf(p[1][2], p[1][3]));
      r0 = fmaxf(r0, __shfl_xor_sync(0xffffffffu, r0, 1));
      r1 = fmaxf(r1, __shfl_xor_sync(0xffffffffu, r1, 1));
      r0 = fmaxf(r0, __shfl_xor_sync(0xffffffffu, r0, 2)) * sc0;
      r1 = fmaxf(r1, __shfl_xor_sync(0xffffffffu, r1, 2)) * sc1;
      // -inf + kLag = -inf: the first logit always moves it
      const bool up0 = r0 > m0 + (kLag + LY::kBias), up1 = r1 > m1 + (kLag + LY::kBias);
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float n0 = up0 ? r0 - LY::kBias : m0, n1 = up1 ? r1 - LY::kBias : m1;
        const float al0 = up0 ? exp2_fast(m0 - n0) : 1.f, al1 = up1 ? exp2_fast(m1 - n1) : 1.f;
        m0 = n0;
        m1 = n1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int nt = 0; nt < 32; ++nt) {
          o[nt][0] *= al0;
          o[nt][1] *= al0;
          o[nt][2] *= al1;
          o[nt][3] *= al1;
        }
      }
      // rows that have seen no token yet keep every weight at 0
      const float sub0 = m0 == -INFINITY ? 0.f : -m0, sub1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[j][0] = exp2_fast(fmaf(p[j][0], sc0, sub0));
        p[j][1] = exp2_fast(fmaf(p[j][1], sc0, sub0));
        p[j][2] = exp2_fast(fmaf(p[j][2], sc1, sub1));
        p[j][3] = exp2_fast(fmaf(p[j][3], sc1, sub1));
      }
      auto least4 = [&](int j) { return fminf(fminf(p[j][0], p[j][1]), fminf(p[j][2], p[j][3])); };
      float least = fminf(least4(0), least4(1));  // of the lane's weights
      if (nv != kTile) {  // also where a scale has underflowed to 0
        least = 1.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (seen(j, e))
              least = fminf(least, fminf(p[j][e], p[j][2 + e]));
            else
              p[j][e] = p[j][2 + e] = 0.f;
      }
      const bool wide = F8 && __any_sync(0xffffffffu, least < kLeastF16);
      l0 += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
      l1 += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
      // weight of each micro-block: sums over its 4 tokens, one per quad lane (run 2j + e
      // over the quad: halve the runs a lane carries twice)
      if (a.bsum) {
        const bool hi = tq & 2, odd = tq & 1;
        const float a0 = (hi ? p[1][0] : p[0][0]) + __shfl_xor_sync(0xffffffffu, hi ? p[0][0] : p[1][0], 2);
        const float a1 = (hi ? p[1][1] : p[0][1]) + __shfl_xor_sync(0xffffffffu, hi ? p[0][1] : p[1][1], 2);
        const float c0 = (hi ? p[1][2] : p[0][2]) + __shfl_xor_sync(0xffffffffu, hi ? p[0][2] : p[1][2], 2);
        const float c1 = (hi ? p[1][3] : p[0][3]) + __shfl_xor_sync(0xffffffffu, hi ? p[0][3] : p[1][3], 2);
        const float b0 = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
        const float b1 = (odd ? c1 : c0) + __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 1);
        const int64_t base = ((int64_t)w.q * a.hq + (int64_t)w.g * G) * max_tiles + w.t0 + ti;
        if (gq < G) {
          const int64_t at = base + gq * max_tiles;
          a.bsum[at * 4 + tq] = b0;
          if (tq == 0) a.bmax[at] = m0;
        }
        if (gq + 8 < G) {
          const int64_t at = base + (gq + 8) * max_tiles;
          a.bsum[at * 4 + tq] = b1;
          if (tq == 0) a.bmax[at] = m1;
        }
      }
      return wide;
    };
    // ---- weights to the operand of P V.  BF16 V: a BF16 hi + lo pair (about 17 significant
    // bits; 8 alone would show in short contexts).  e4m3 V: FP16, 11 bits against the cache's
    // 4, while all of the tile's weights are normal numbers (an FP16 hi + lo pair took 7%
    // more time on long batches).  A wide tile takes the BF16 pair, whose exponents are
    // fp32's, and V widened to BF16: below a key that outweighs all others and whose value
    // is near 0, the output is made of weights that FP16 would round coarsely, or drop while
    // l counts them.  The test and the second form cost 4% where no tile is wide (64 x
    // 16K-131K tokens, 12/1 heads: 391 -> 409 us) and 24% more where all are (507).
    auto as_operand = [&](const float(&p)[2][4], bool wide, uint32_t(&pa)[4], uint32_t(&pl)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = p[k >> 1][2 * (k & 1)], y = p[k >> 1][2 * (k & 1) + 1];
        if (F8 && !wide) {
          const __half2 h = __floats2half2_rn(x, y);
          pa[k] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          split_bf16(x, y, pa[k], pl[k]);
        }
      }
    };
    // ---- O += P V of the tile at kb
    auto add_values = [&](uint32_t kb, int nv, const uint32_t(&pa)[4], const uint32_t(&pl)[4]) {
      constexpr int kParts = F8 ? 2 : 4;  // e4m3: 128 dims per 16-byte read of the 8 column groups; BF16: 64
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        uint32_t x[2][2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 v = lds128(kb + (F8 ? v_off[j][e] ^ (c * (128 + 16)) : v_off[j][e] + c * 1024));
            if (nv != kTile && tile_run(j, e) * kRatio + tile_row<F8>(tq, e) >= nv)
              v = make_uint4(0, 0, 0, 0);  // rows behind the end may hold anything
            x[j][e][0] = v.x;
            x[j][e][1] = v.y;
            x[j][e][2] = v.z;
            x[j][e][3] = v.w;
          }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (F8) {  // 4 dims: the two tokens' bytes are paired, then widened
            const uint2 t0 = e4m3x4_to_f16x4(__byte_perm(x[0][0][r], x[0][1][r], 0x5140));
            const uint2 t1 = e4m3x4_to_f16x4(__byte_perm(x[0][0][r], x[0][1][r], 0x7362));
            const uint2 u0 = e4m3x4_to_f16x4(__byte_perm(x[1][0][r], x[1][1][r], 0x5140));
            const uint2 u1 = e4m3x4_to_f16x4(__byte_perm(x[1][0][r], x[1][1][r], 0x7362));
            mma_f16_16816(o[c * 16 + 4 * r + 0], pa[0], pa[1], pa[2], pa[3], t0.x, u0.x);
            mma_f16_16816(o[c * 16 + 4 * r + 1], pa[0], pa[1], pa[2], pa[3], t0.y, u0.y);
            mma_f16_16816(o[c * 16 + 4 * r + 2], pa[0], pa[1], pa[2], pa[3], t1.x, u1.x);
            mma_f16_16816(o[c * 16 + 4 * r + 3], pa[0], pa[1], pa[2], pa[3], t1.y, u1.y);
          } else {
            const uint32_t lo0 = __byte_perm(x[0][0][r], x[0][1][r], 0x5410);
            const uint32_t hi0 = __byte_perm(x[0][0][r], x[0][1][r], 0x7632);
            const uint32_t lo1 = __byte_perm(x[1][0][r], x[1][1][r], 0x5410);
            const uint32_t hi1 = __byte_perm(x[1][0][r], x[1][1][r], 0x7632);
            mma_bf16_16816(o[c * 8 + 2 * r], pa[0], pa[1], pa[2], pa[3], lo0, lo1);
            mma_bf16_16816(o[c * 8 + 2 * r + 1], pa[0], pa[1], pa[2], pa[3], hi0, hi1);
            mma_bf16_16816(o[c * 8 + 2 * r], pl[0], pl[1], pl[2], pl[3], lo0, lo1);
            mma_bf16_16816(o[c * 8 + 2 * r + 1], pl[0], pl[1], pl[2], pl[3], hi0, hi1);
          }
        }
      }
    };
    // the same of an e4m3 tile with wide weights: V as BF16
    auto add_values_wide = [&](uint32_t kb, int nv, const uint32_t(&pa)[4], const uint32_t(&pl)[4]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // 8 of a chunk's 16 dims
        const int part = c >> 1, r0 = 2 * (c & 1);
        uint32_t x[2][2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t at = kb + (v_off[j][e] ^ (part * (128 + 16))) + r0 * 4;
            const bool off = nv != kTile && tile_run(j, e) * kRatio + tile_row<F8>(tq, e) >= nv;
            const uint2 v = lds64(at);
            x[j][e][0] = off ? 0 : v.x;
            x[j][e][1] = off ? 0 : v.y;
          }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint2 t = e4m3x4_to_f16x4(__byte_perm(x[0][0][r], x[0][1][r], k ? 0x7362 : 0x5140));
            const uint2 u = e4m3x4_to_f16x4(__byte_perm(x[1][0][r], x[1][1][r], k ? 0x7362 : 0x5140));
            float(&o0)[4] = o[part * 16 + 4 * (r0 + r) + 2 * k], (&o1)[4] = o[part * 16 + 4 * (r0 + r) + 2 * k + 1];
            const uint32_t b0 = f16x2_to_bf16x2(t.x), b1 = f16x2_to_bf16x2(u.x);
            mma_bf16_16816(o0, pa[0], pa[1], pa[2], pa[3], b0, b1);
            mma_bf16_16816(o0, pl[0], pl[1], pl[2], pl[3], b0, b1);
            const uint32_t b2 = f16x2_to_bf16x2(t.y), b3 = f16x2_to_bf16x2(u.y);
            mma_bf16_16816(o1, pa[0], pa[1], pa[2], pa[3], b2, b3);
            mma_bf16_16816(o1, pl[0], pl[1], pl[2], pl[3], b2, b3);
          }
      }
    };
    for (int ti = rank; ti < n_tiles; ti += kWarps) {
      const int stage = landed(ti);
      if (stage < 0) break;
      const int nv = valid[stage];
      const uint32_t kb = ring + stage * LY::kStageBytes;
      float s[2][4];
      uint32_t pa[4], pl[4];
      products(kb, s);
      if (weigh(ti, nv, s)) {
        as_operand(s, true, pa, pl);
        add_values_wide(kb, nv, pa, pl);
      } else {
        as_operand(s, false, pa, pl);
        add_values(kb, nv, pa, pl);
      }
      held = stage;
      if (ti + kWarps < n_tiles) {  // the last stage is kept for the join
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + stage * 8);
      }
    }
    T_base += n_tiles;
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty + qi * 8);
    if (++qi == (uint32_t)a.q_bufs) {
      qi = 0;
      ++lap;
    }

    // ---- join the warps' (m, l, O)
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // whole pair here: straight to out; else to the partial slot of the pair that this
    // CTA took over (0) or leaves unfinished (1)
    const int nt_pair = tiles_of(w.len);
    const bool direct = w.t0 == 0 && w.t1 == nt_pair;
    const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
    const size_t out_row = direct ? (size_t)w.q * a.hq + (size_t)w.g * G : (size_t)slot * G;
    auto put_lse = [&](float lse_0, float lse_1) {  // by one warp; base 2
      float* at = (direct ? a.lse : a.part_lse) + out_row;
      const float f = direct ? 0.69314718055994530942f : 1.f;
      if (tq == 0) {
        if (gq < G) at[gq] = lse_0 * f;
        if (gq + 8 < G) at[gq + 8] = lse_1 * f;
      }
      if (w.t0 == 0 && lane == 0)
        a.span[w.q * a.hkv + w.g] =
            make_int2(blockIdx.x, direct ? blockIdx.x
                                         : share_of(sh, w.begin + cost_of(nt_pair) + nt_pair - 1));
    };
    // the columns and n-tiles of dim slice sl (see the join below)
    auto e_of = [](int sl) { return F8 ? (sl >> 1) & 1 : sl & 1; };
    auto i0_of = [](int sl) { return F8 ? 16 * (sl >> 2) + 8 * (sl & 1) : 8 * (sl >> 1); };
    if (lone) {  // nothing to join
      if (held >= 0 && lane == 0) mbar_arrive(empty + held * 8);
      const float f0 = l0 > 0.f ? 1.f / l0 : l0, f1 = l1 > 0.f ? 1.f / l1 : l1;  // 0: no token; NaN stays NaN
      put_lse(m0 + log2f(l0), m1 + log2f(l1));
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) {
        const int e = e_of(sl), i0 = i0_of(sl);
        const int dim = F8 ? 128 * (sl >> 2) + 32 * tq + 16 * e + 8 * (sl & 1) : kSlice * sl + 8 * tq;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          if (gq + 8 * hr >= G) continue;
          const float f = hr ? f1 : f0;
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = o[i0 + k][2 * hr + e] * f;
          const size_t at = (out_row + gq + 8 * hr) * kHeadDim + dim;
          if (direct) {  // out is 8-byte aligned
            *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            *reinterpret_cast<uint2*>(a.out + at + 4) = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
          } else {
            *reinterpret_cast<float4*>(a.part_o + at) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(a.part_o + at + 4) = make_float4(y[4], y[5], y[6], y[7]);
          }
        }
      }
      if (!next_piece(a, w, x1)) break;
      continue;
    }
    if (lane == 0) held_s[rank] = held;
    if (tq == 0) {
      ml[rank * 16 + gq] = make_float2(m0, l0);
      ml[rank * 16 + gq + 8] = make_float2(m1, l1);
    }
    named_bar_sync(kBarConsumers, kConsumerThreads);
    const int nw = min(kWarps, n_tiles);  // warps that had a tile: ranks 0 .. nw - 1
    float fac[2], M[2], L[2];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float2 e[kWarps];
#pragma unroll
      for (int v = 0; v < kWarps; ++v) e[v] = ml[v * 16 + gq + 8 * hr];
      M[hr] = -INFINITY;
      L[hr] = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) M[hr] = fmaxf(M[hr], e[v].x);
      const float sub = M[hr] == -INFINITY ? 0.f : M[hr];
#pragma unroll
      for (int v = 0; v < kWarps; ++v) L[hr] += e[v].y * exp2_fast(e[v].x - sub);
      // L = 0: no token; a NaN stays one.  The quotient is within 2 ulp: one of the fp32
      // roundings of a row's factor, next to the BF16 rounding of out
      fac[hr] = L[hr] > 0.f ? __fdividef(exp2_fast((hr ? m1 : m0) - sub), L[hr]) : L[hr];
    }
    // O: every warp puts its own into the stage it holds, and a thread adds up float4s of
    // them: 8 slices of 16 rows x 32 dims, 16-byte chunks swizzled by the row.
    // BF16: n-tile 8 (sl >> 1) + i holds, in column 2tq + e, dim 64 (sl >> 1) + 32e + 8tq + i:
    //       slice sl takes e = sl & 1.
    // e4m3: n-tile 16c + i, column 2tq + e, dim 128c + 32tq + 16e + i: slice sl takes
    //       c = sl >> 2, e = (sl >> 1) & 1 and i = 8 (sl & 1) .. + 7.
    constexpr int kPart = kSlices / LY::kRounds;  // slices of a round
#pragma unroll
    for (int rd = 0; rd < LY::kRounds; ++rd) {
      if (rd) named_bar_sync(kBarConsumers, kConsumerThreads);  // the last part has been read
      if (held >= 0) {
        uint8_t* at = smem + held * LY::kStageBytes + gq * (kSlice * 4);
#pragma unroll
        for (int ls = 0; ls < kPart; ++ls) {
          const int sl = rd * kPart + ls, e = e_of(sl), i0 = i0_of(sl);
#pragma unroll
          for (int hr = 0; hr < 2; ++hr)
            if (8 * hr < G) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float4*>(at + ls * kSliceBytes + 8 * hr * (kSlice * 4) + (((2 * tq + k) ^ gq) << 4)) =
                    make_float4(o[i0 + 4 * k][2 * hr + e] * fac[hr], o[i0 + 4 * k + 1][2 * hr + e] * fac[hr],
                                o[i0 + 4 * k + 2][2 * hr + e] * fac[hr], o[i0 + 4 * k + 3][2 * hr + e] * fac[hr]);
            }
        }
      }
      named_bar_sync(kBarConsumers, kConsumerThreads);
      uint32_t from[kWarps];
#pragma unroll
      for (int v = 0; v < kWarps; ++v) from[v] = ring + max(held_s[v], 0) * LY::kStageBytes;
#pragma unroll 2
      for (int i = tid; i < G * kPart * 8; i += kConsumerThreads) {
        const int row = i / (kPart * 8), ls = i / 8 % kPart, sl = rd * kPart + ls, chunk = i & 7;
        const int off = ls * kSliceBytes + row * (kSlice * 4) + ((chunk ^ (row & 7)) << 4);
        uint4 y[kWarps];
#pragma unroll
        for (int v = 0; v < kWarps; ++v) y[v] = v < nw ? lds128(from[v] + off) : make_uint4(0, 0, 0, 0);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          acc.x += __uint_as_float(y[v].x);
          acc.y += __uint_as_float(y[v].y);
          acc.z += __uint_as_float(y[v].z);
          acc.w += __uint_as_float(y[v].w);
        }
        const int dim = F8 ? 128 * (sl >> 2) + 32 * (chunk >> 1) + 16 * ((sl >> 1) & 1) + 8 * (sl & 1) + 4 * (chunk & 1)
                           : kSlice * sl + 4 * chunk;
        const size_t at = (out_row + row) * kHeadDim + dim;
        if (direct)
          *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
        else
          *reinterpret_cast<float4*>(a.part_o + at) = acc;
      }
    }
    if (warp == kWarps - 1) put_lse(M[0] + log2f(L[0]), M[1] + log2f(L[1]));  // -inf when L = 0
    if (!next_piece(a, w, x1)) break;
    // every stage has been read: hand the held ones back to the copies, which come after
    // these ordinary writes
    fence_proxy_async();
    named_bar_sync(kBarConsumers, kConsumerThreads);
    if (held >= 0 && lane == 0) mbar_arrive(empty + held * 8);
  }
}

template <bool F8>
__global__ void __launch_bounds__(Lay<F8>::kThreads, 1) dense_decode_kernel(const __grid_constant__ DenseArgs a) {
  using LY = Lay<F8>;
  constexpr int kThreads = LY::kThreads, kWarps = LY::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  int* plan = reinterpret_cast<int*>(smem + LY::kOffPlan);  // [0], [1] the first query and its place, [4..] warp sums
  int2* tab = reinterpret_cast<int2*>(smem + LY::kOffTab);
  if (tid == 0) {
    const uint32_t bars = smem_u32(smem + LY::kOffBar);
    for (int i = 0; i < 2 * LY::kStages + kMaxQ; ++i) mbar_init(bars + i * 8, 1);
    for (int i = 0; i < kMaxQ; ++i) mbar_init(bars + (2 * LY::kStages + kMaxQ + i) * 8, LY::kWarps);
    fence_mbar_init();
    *reinterpret_cast<volatile int*>(smem + LY::kOffAbort) = 0;
  }
  // the zero row (a group of 16 needs none, and fills all 32)
  if (a.G < 16 && warp == 1)
    sts128(smem_u32(smem + LY::kOffQ) + (kQRows - 1) * kQStride + lane * 16, make_uint4(0, 0, 0, 0));
  pdl_wait_previous();
  // ---- the share of this CTA.  A thread per query, kThreads of them a round; with
  // one round (the usual batch) the lengths are loaded once and kept.
  const bool one_round = a.nq <= kThreads;
  const bool whole_tab = a.nq <= kTab;
  int total = 0, first = 0, len = 0, filled = 0;  // filled: queries that see tokens
  auto scan_round = [&](int base, bool report) {  // places before query base + tid; total moves on
    const int q = base + tid;
    len = q < a.nq ? query_len(a, q, report) : 0;
    const int n = places_of(len) * a.hkv;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) plan[4 + warp] = inc;
    if (whole_tab && q < a.nq) tab[q] = make_int2(len, a.q_seq[q]);
    filled += __syncthreads_count(len > 0);
    first = total + inc - n;
#pragma unroll
    for (int v = 0; v < kThreads / 32; ++v) {
      const int x = plan[4 + v];
      if (v < warp) first += x;
      total += x;
    }
    if (!one_round) __syncthreads();
  };
  for (int b = 0; b < a.nq; b += kThreads) {
    scan_round(b, blockIdx.x == 0);
    if (blockIdx.x == 0 && b + tid < a.nq && len == 0)
      for (int g = 0; g < a.hkv; ++g) a.span[(b + tid) * a.hkv + g] = make_int2(0, -1);
  }
  if (total == 0) return;
  const Shares sh = make_shares(total, filled * a.hkv, a.ctas);
  if ((int)blockIdx.x >= sh.n) return;
  const int x0 = share_begin(sh, blockIdx.x), x1 = share_begin(sh, blockIdx.x + 1);
  auto find_first = [&](int base) {  // the query that holds place x0
    if (len > 0 && first <= x0 && x0 < first + places_of(len) * a.hkv) {
      plan[0] = base + tid;
      plan[1] = first;
    }
  };
  if (one_round) {
    find_first(0);
  } else {
    total = 0;
    for (int b = 0; b < a.nq; b += kThreads) {
      scan_round(b, false);
      find_first(b);
    }
  }
  __syncthreads();
  Walk w;
  w.q = plan[0];
  w.begin = plan[1];
  w.tab = tab;
  w.q_tab = whole_tab ? 0 : w.q;
  if (!whole_tab) {
    if (tid < kTab && w.q + tid < a.nq) tab[tid] = make_int2(query_len(a, w.q + tid, false), a.q_seq[w.q + tid]);
    __syncthreads();
  }
  w.len = tab[w.q - w.q_tab].x;
  w.seq = tab[w.q - w.q_tab].y;
  w.g = (x0 - w.begin) / places_of(w.len);
  w.begin += w.g * places_of(w.len);
  if (!set_span(w, x0, x1)) return;  // the share ends before the pair's first tile
  if constexpr (F8) {  // by whole warpgroups, and by every one that is left
    if (warp < kWarps)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LY::kConsumerRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LY::kCopyRegs));
    if (warp > kWarps) return;
  }
  if (warp < kWarps)
    consumers<F8>(a, smem, w, sh, x1);
  else
    copy_warp<F8>(a, smem, w, x1);
}

// ------------------------------------------------------------------ join + weights

constexpr int kJoinThreads = 256;
constexpr int kFewPieces = 8;  // pieces of a head that 64 threads join alone

struct JoinArgs {
  DenseArgs d;
  const float* mass_in;
  float* mass_out;
  int64_t mass_ld;
  float decay;
  int32_t mass_blocks;  // CTAs per query for the weights
  int32_t n_mass;       // all of them, the first of the grid
  int32_t parts;        // CTAs per pair for the join
  int32_t slice_bits;   // the dims of a head of many pieces are shared by 1, 2 or 4 blocks
};

// The partial slot of CTA c's piece of a pair that spans several CTAs.
__device__ __forceinline__ int slot_of(const int2& span, int c) { return 2 * c + (c == span.x ? 1 : 0); }

// Base-2 lse of (q, h), by 8 neighbouring lanes: the joined pieces' or, for a
// pair that one CTA held, the one already in lse.
__device__ __forceinline__ float joined_lse2(const DenseArgs& a, int q, int h) {
  const int sub = threadIdx.x & 7;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int2 p = a.span[q * a.hkv + h / a.G];
  if (p.y < p.x) return -INFINITY;
  if (p.x == p.y) return a.lse[(size_t)q * a.hq + h] * 1.44269504088896340736f;
  const int row = h % a.G;
  float M = -INFINITY;
  for (int c = p.x + sub; c <= p.y; c += 8) M = fmaxf(M, a.part_lse[(size_t)slot_of(p, c) * a.G + row]);
#pragma unroll
  for (int d = 4; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, d));
  if (M == -INFINITY) return -INFINITY;
  float L = 0.f;
  for (int c = p.x + sub; c <= p.y; c += 8) L += exp2f(a.part_lse[(size_t)slot_of(p, c) * a.G + row] - M);
#pragma unroll
  for (int d = 4; d; d >>= 1) L += __shfl_xor_sync(lanes, L, d);
  return M + log2f(L);
}

// The first blocks add up weights, which takes longest: 64 tiles (256 micro-blocks) of one
// query's sequence each, the heads spread over 4 groups of 64 threads.  The others join:
// `parts` of them a (query, KV head) pair.
// The join's time is the latency of two dependent loads (span; pieces' lse and rows
// together), so it asks for all rows at once and waits as seldom as it can: up to 8
// pieces a head, 64 threads join one with no exchange (the call on 125 pairs of 12 heads, 2
// pieces each: 24.4 us with a block a head, 22.7 so); more pieces are spread over the block,
// and few heads over 2 or 4 blocks each, by their dims (the call on 2 sequences of 2K and
// 44K tokens, 12/1 heads: 22.0 us unsplit, 18.6 so).  Sums run in a fixed order.
__global__ void __launch_bounds__(kJoinThreads) dense_join_kernel(const __grid_constant__ JoinArgs ja) {
  const DenseArgs& a = ja.d;
  pdl_launch_dependents();
  pdl_wait_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float4 acc_s[kJoinThreads];
  __shared__ float lse_s[kMaxCtas];  // pieces' lse, then their weights (kMaxCtas <= kJoinThreads: one each)
  __shared__ float red_s[2][kJoinThreads / 32];
  static_assert(kMaxCtas <= kJoinThreads, "a thread per piece");
  if ((int)blockIdx.x >= ja.n_mass) {
    const int pair = (blockIdx.x - ja.n_mass) / ja.parts, part = (blockIdx.x - ja.n_mass) % ja.parts;
    const int2 p = a.span[pair];
    if (p.x == p.y) return;  // written by its CTA
    const int n = max(0, p.y - p.x + 1);
    const float4* rows = reinterpret_cast<const float4*>(a.part_o);
    // of a head: weights relative to 2^M, their sum, the rows they weigh
    auto put = [&](int row, int c4, float M, float L, float4 r) {
      const size_t qh = (size_t)pair * a.G + row;
      const float inv = L == 0.f ? 0.f : 1.f / L;  // 0: no token; a NaN stays one
      reinterpret_cast<uint2*>(a.out + qh * kHeadDim)[c4] =
          make_uint2(pack_bf16(r.x * inv, r.y * inv), pack_bf16(r.z * inv, r.w * inv));
      if (c4 == 0) a.lse[qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    };
    auto weight = [](float v, float M) { return v == -INFINITY ? 0.f : exp2f(v - M); };  // 0: an empty piece
    if (n <= kFewPieces) {  // 64 threads a head, nothing shared
      const int c4 = tid & 63;
      for (int row = (tid >> 6) * ja.parts + part; row < a.G; row += ja.parts * 4) {
        float4 x[kFewPieces];
        float v[kFewPieces];
#pragma unroll
        for (int k = 0; k < kFewPieces; ++k) {
          v[k] = -INFINITY;
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < n) {
            const size_t at = (size_t)slot_of(p, p.x + k) * a.G + row;
            v[k] = a.part_lse[at];
            x[k] = rows[at * (kHeadDim / 4) + c4];
          }
        }
        float M = v[0], L = 0.f;
#pragma unroll
        for (int k = 1; k < kFewPieces; ++k) M = fmaxf(M, v[k]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kFewPieces; ++k) {
          const float f = weight(v[k], M);
          L += f;
          acc.x += f * x[k].x;
          acc.y += f * x[k].y;
          acc.z += f * x[k].z;
          acc.w += f * x[k].w;
        }
        put(row, c4, M, L, acc);
      }
      return;
    }
    // many pieces: the block takes a slice of a head's dims, groups of threads share the pieces
    const int bits = ja.slice_bits, cols = 64 >> bits, groups = 4 << bits;
    const int grp = tid >> (6 - bits), col = tid & (cols - 1);
    for (int item = part; item < a.G << bits; item += ja.parts) {
      const int row = item >> bits, c4 = (item & ((1 << bits) - 1)) * cols + col;
      __syncthreads();  // the last item's use of the shared arrays has ended
      // rows: requested before their weights are known
      const float4* base = rows + (size_t)row * (kHeadDim / 4) + c4;
      const size_t step = (size_t)a.G * (kHeadDim / 4);
      constexpr int kAhead = 4;
      float4 x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (grp + groups * k < n) x[k] = base[slot_of(p, p.x + grp + groups * k) * step];
      const float v = tid < n ? a.part_lse[(size_t)slot_of(p, p.x + tid) * a.G + row] : -INFINITY;
      float M = v;
#pragma unroll
      for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      if (lane == 0) red_s[0][warp] = M;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kJoinThreads / 32; ++k) M = fmaxf(M, red_s[0][k]);
      float e = weight(v, M);
      if (tid < n) lse_s[tid] = e;
#pragma unroll
      for (int d = 16; d; d >>= 1) e += __shfl_xor_sync(0xffffffffu, e, d);
      if (lane == 0) red_s[1][warp] = e;
      __syncthreads();
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < kJoinThreads / 32; ++k) L += red_s[1][k];
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = grp; i0 < n; i0 += groups * kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + groups * k;
          if (i >= n) break;
          const float f = lse_s[i];
          acc.x += f * x[k].x;
          acc.y += f * x[k].y;
          acc.z += f * x[k].z;
          acc.w += f * x[k].w;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + groups * (kAhead + k);
          if (i < n) x[k] = base[slot_of(p, p.x + i) * step];
        }
      }
      acc_s[tid] = acc;
      __syncthreads();
      if (grp == 0) {
#pragma unroll 4
        for (int k = 1; k < groups; ++k) {
          const float4 y = acc_s[k * cols + col];
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
        }
        put(row, c4, M, L, acc);
      }
    }
    return;
  }
  // ---- weights.  The longest query of a sequence (the first of several) adds up all of
  // the sequence's queries in order, so the total does not depend on which block runs
  // first.  Its blocks take every mass_blocks-th 64 tiles.
  constexpr int kHeads = 8, kRound = 4 * kHeads;  // heads of a group and of the block at once
  const int q0 = blockIdx.x / ja.mass_blocks, grp = tid >> 6;
  float4(*sum_s)[64] = reinterpret_cast<float4(*)[64]>(&acc_s[0]);
  const int seq = a.q_seq[q0], longest = query_len(a, q0, false);
  const int64_t max_tiles = (int64_t)a.mpps * kTilesPerPage;
  __shared__ unsigned same_s[kJoinThreads / 32];  // queries of this sequence, 256 at a time
  for (int t0 = (int)(blockIdx.x % ja.mass_blocks) * 64; t0 < tiles_of(longest); t0 += ja.mass_blocks * 64) {
    const int tile = t0 + (tid & 63);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const int blocks = (longest + kRatio - 1) / kRatio;
    const int64_t row = (int64_t)seq * ja.mass_ld;
    float old[4] = {};  // requested before anything else is waited for
    if (grp == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (tile * kTileRuns + k < blocks) old[k] = ja.mass_in[row + tile * kTileRuns + k];
    }
    for (int qb = 0; qb < a.nq; qb += kJoinThreads) {
      const int qt = qb + tid;
      const unsigned same = __ballot_sync(0xffffffffu, qt < a.nq && a.q_seq[qt] == seq && query_len(a, qt, false) > 0);
      __syncthreads();
      if (lane == 0) same_s[warp] = same;
      __syncthreads();
      for (int v = 0; v < kJoinThreads / 32; ++v)
        for (unsigned bits = same_s[v]; bits; bits &= bits - 1) {
          const int q = qb + v * 32 + __ffs(bits) - 1;
          const int len = query_len(a, q, false);
          if (len > longest || (len == longest && q < q0)) return;  // the same in every thread
          const bool on = tile < (len + kTile - 1) / kTile;
          for (int h0 = 0; h0 < a.hq; h0 += kRound) {
            float bm[kHeads];
            float4 b[kHeads];
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {  // head h0 + 4k + grp, requested before its lse is known
              const int h = h0 + 4 * k + grp;
              bm[k] = -INFINITY;
              b[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (on && h < a.hq) {
                const int64_t at = ((int64_t)q * a.hq + h) * max_tiles + tile;
                bm[k] = a.bmax[at];
                b[k] = reinterpret_cast<const float4*>(a.bsum)[at];
              }
            }
            const int hl = h0 + (tid >> 3);
            const float v2 = hl < a.hq ? joined_lse2(a, q, hl) : -INFINITY;
            __syncthreads();
            if ((tid & 7) == 0) lse_s[tid >> 3] = v2;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
              const float l2 = lse_s[4 * k + grp];
              const float f = l2 == -INFINITY || bm[k] == -INFINITY ? 0.f : exp2f(bm[k] - l2);  // 0: no token seen
              sum.x += f * b[k].x;
              sum.y += f * b[k].y;
              sum.z += f * b[k].z;
              sum.w += f * b[k].w;
            }
          }
        }
    }
    sum_s[grp][tid & 63] = sum;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        const float4 y = sum_s[k][tid];
        sum.x += y.x;
        sum.y += y.y;
        sum.z += y.z;
        sum.w += y.w;
      }
      const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = tile * kTileRuns + k;
        if (b < blocks) ja.mass_out[row + b] = ja.decay * old[k] + v[k];
      }
    }
    __syncthreads();  // sum_s is used again
  }
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

struct WorkspaceMap {
  int64_t span, part_lse, part_o, bsum, bmax, total;
};

WorkspaceMap workspace_map(const qsa_cache_t& c, int32_t nq, int32_t hq, bool with_mass) {
  const int64_t G = hq / c.num_kv_heads;
  WorkspaceMap m;
  m.span = 0;
  m.part_lse = align256((int64_t)nq * c.num_kv_heads * 8);
  m.part_o = m.part_lse + align256(2 * kMaxCtas * G * 4);
  m.bsum = m.part_o + align256(2 * kMaxCtas * G * kHeadDim * 4);
  const int64_t tiles = with_mass ? (int64_t)nq * hq * c.max_pages_per_seq * kTilesPerPage : 0;
  m.bmax = m.bsum + align256(tiles * 16);
  m.total = m.bmax + align256(tiles * 4);
  return m;
}

int check_shape(const qsa_cache_t* cache, int32_t nq, int32_t hq) {
  if (!cache || nq < 0 || hq < 1) return QSA_ERR_INVALID_ARG;
  const qsa_cache_t& c = *cache;
  if (c.num_pages < 1 || c.max_seqs < 1 || c.max_pages_per_seq < 1 || c.num_kv_heads < 1) return QSA_ERR_INVALID_ARG;
  if (hq % c.num_kv_heads != 0) return QSA_ERR_INVALID_ARG;
  if (hq / c.num_kv_heads > QSA_MAX_GROUP) return QSA_ERR_UNSUPPORTED;
  if (c.max_pages_per_seq > 0x7fffffff / kPage) return QSA_ERR_UNSUPPORTED;  // positions are int32
  if (((int64_t)c.max_pages_per_seq * kTilesPerPage + 8) * c.num_kv_heads > 0x7fffffff / (nq > 0 ? nq : 1))
    return QSA_ERR_UNSUPPORTED;  // places are int32
  return QSA_OK;
}

template <bool F8>
int launch_dense(const DenseArgs& a, cudaStream_t s) {
  // the attribute belongs to the device's copy of the kernel
  if (cudaFuncSetAttribute(dense_decode_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<F8>::kSmem) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  if constexpr (F8) {  // a kernel built with fewer registers would wait for its share forever
    static const bool enough = [] {
      cudaFuncAttributes f;
      const bool ok = cudaFuncGetAttributes(&f, dense_decode_kernel<F8>) == cudaSuccess;
      if (!ok) (void)cudaGetLastError();
      return ok && f.numRegs >= Lay<F8>::kRegs;
    }();
    if (!enough) return QSA_ERR_CUDA;
  }
  return qsa_host::launch(dense_decode_kernel<F8>, dim3((unsigned)a.ctas), dim3(Lay<F8>::kThreads), (size_t)Lay<F8>::kSmem, s,
                          a);
}

}  // namespace

extern "C" int64_t qsa_dense_decode_workspace_bytes(const qsa_cache_t* cache, int32_t nq, int32_t hq,
                                                    int32_t with_mass) {
  const int rc = check_shape(cache, nq, hq);
  if (rc != QSA_OK) return rc;
  return workspace_map(*cache, nq, hq, with_mass != 0).total;
}

extern "C" int qsa_dense_decode(const qsa_cache_t* cache, const void* q, int32_t nq, int32_t hq, const int32_t* q_seq,
                                const int32_t* q_pos, float scale, void* out, float* lse, const float* mass_in,
                                float* mass_out, int64_t mass_ld, float decay, void* workspace,
                                int64_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_shape(cache, nq, hq);
  if (rc != QSA_OK) return rc;
  const qsa_cache_t& c = *cache;
  if (!(scale > 0.f) || (mass_in == nullptr) != (mass_out == nullptr)) return QSA_ERR_INVALID_ARG;
  if (c.kv_dtype != QSA_KV_BF16 && c.kv_dtype != QSA_KV_FP8_E4M3) return QSA_ERR_UNSUPPORTED;
  if (nq == 0) return QSA_OK;
  if (!c.kv_pages || !c.block_table || !q || !q_seq || !q_pos || !out || !lse || !workspace) return QSA_ERR_INVALID_ARG;
  auto misaligned = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (misaligned(c.kv_pages, 16) || misaligned(q, 16) || misaligned(out, 8) || misaligned(workspace, 256))
    return QSA_ERR_INVALID_ARG;
  const bool mass = mass_in != nullptr;
  if (mass && mass_ld < (int64_t)c.max_pages_per_seq * kBlocksPerPage) return QSA_ERR_INVALID_ARG;
  const WorkspaceMap m = workspace_map(c, nq, hq, mass);
  if (workspace_bytes < m.total) return QSA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DenseArgs a;
  a.kv = static_cast<const uint8_t*>(c.kv_pages);
  a.bt = c.block_table;
  a.num_pages = c.num_pages;
  a.max_seqs = c.max_seqs;
  a.mpps = c.max_pages_per_seq;
  a.hkv = c.num_kv_heads;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.nq = nq;
  a.hq = hq;
  a.G = hq / c.num_kv_heads;
  a.q_seq = q_seq;
  a.q_pos = q_pos;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.span = reinterpret_cast<int2*>(ws + m.span);
  a.part_lse = reinterpret_cast<float*>(ws + m.part_lse);
  a.part_o = reinterpret_cast<float*>(ws + m.part_o);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.bsum = mass ? reinterpret_cast<float*>(ws + m.bsum) : nullptr;
  a.bmax = mass ? reinterpret_cast<float*>(ws + m.bmax) : nullptr;
  a.ctas = sms < kMaxCtas ? sms : kMaxCtas;
  a.q_bufs = a.G == 16 ? 2 : (kQRows - 1) / a.G < kMaxQ ? (kQRows - 1) / a.G : kMaxQ;
  a.st = dev_status;
  if (c.kv_dtype == QSA_KV_FP8_E4M3) {
    const int64_t rows = (int64_t)c.num_pages * c.num_kv_heads * kBlocksPerPage * (2 * kRatio * kHeadDim / 128);
    if (rows > 0x7fffffff) return QSA_ERR_UNSUPPORTED;  // tensor-map coordinates are int32
    const auto enc = qsa_host::tensor_map_encoder();
    const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
    const cuuint32_t box[2] = {128, (cuuint32_t)(Lay<true>::kStageBytes / 128)}, es[2] = {1, 1};
    if (!enc || enc(&a.tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.kv_pages, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QSA_ERR_CUDA;
  }
  JoinArgs j;
  j.d = a;
  j.mass_in = mass_in;
  j.mass_out = mass_out;
  j.mass_ld = mass_ld;
  j.decay = decay;
  const int64_t tiles = (int64_t)c.max_pages_per_seq * kTilesPerPage;
  // 64 tiles a block while that makes no more than about 8 blocks per SM; the lengths may
  // be far below the table's capacity, and a block that finds nothing costs about 1 us
  const int64_t most = (tiles + 63) / 64, fit = (8 * (int64_t)a.ctas + nq - 1) / nq;
  j.mass_blocks = (int32_t)(most < fit ? most : fit);
  // About 4 CTAs per SM, as many as are resident at once (8: 125 queries with totals 26.1
  // us instead of 25.0); the dims split only while that leaves 2 per SM (8 x 32,768 tokens,
  // 128 heads: 85.0 us split in two, 86.0 in four)
  const int64_t pairs = (int64_t)nq * c.num_kv_heads, want = (4 * a.ctas + pairs - 1) / pairs;
  j.slice_bits = pairs * a.G * 4 <= 2 * a.ctas ? 2 : pairs * a.G * 2 <= 2 * a.ctas ? 1 : 0;
  const int64_t items = (int64_t)a.G << j.slice_bits;
  j.parts = (int32_t)(want < items ? want : items);
  const int64_t n_mass = mass ? (int64_t)nq * j.mass_blocks : 0, grid = n_mass + pairs * j.parts;
  if (grid > 0x7fffffff) return QSA_ERR_UNSUPPORTED;
  j.n_mass = (int32_t)n_mass;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int r = c.kv_dtype == QSA_KV_FP8_E4M3 ? launch_dense<true>(a, s) : launch_dense<false>(a, s);
  if (r != QSA_OK) return r;
  // Launched early, the blocks would pile up on the first SMs to come free: a grid of at
  // most one or two per SM asks for shared memory that keeps it to so many (1 x 4,096
  // tokens: 10.1 -> 9.5 us; 3 of 6K to 16K: 16.9 -> 16.1)
  const size_t spread = grid <= a.ctas ? 110 * 1024 : grid <= 2 * a.ctas ? 70 * 1024 : 0;
  if (spread && cudaFuncSetAttribute(dense_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 110 * 1024) !=
                    cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  return qsa_host::launch(dense_join_kernel, dim3((unsigned)grid), dim3(kJoinThreads), spread, s, j);
}
