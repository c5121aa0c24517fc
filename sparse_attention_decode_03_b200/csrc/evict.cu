// qsa_evict: cut sequences of the cache group down to a budget of micro-blocks,
// by the attention weight each block has accumulated (qsa_dense_decode's mass).
//
// Kept of a sequence with nb > budget complete blocks: its first `sink` blocks,
// its last `recent`, and of those between the budget - sink - recent with the
// largest mass (ties: lower index; a NaN mass ranks below every number).  The
// kept blocks close ranks in their order, the open block follows them, and the
// mass row follows its blocks.  A micro-block is the unit because it is what
// the side cache describes: its K/V run of every KV head and its kc row move
// together.
//
// evict_select_kernel, a CTA per sequence or a cluster of up to 8: radix select of the
// cut (11 + 11 + 10 bits of the order-preserving key) over masses held in shared
// memory, histograms summed over the cluster's shared memory, then one ordered pass
// that writes the kept indices, the number kept before every unit, and the moved mass
// row.  Bound by the latency of its passes: 6 us for 4K tokens; a call that cuts one
// sequence of 262,144 tokens to 1,024 blocks took 168 us with one CTA, 53 with a cluster.
//
// evict_move_kernel: units of 8 destination blocks and one KV head (8 runs, 32 KiB
// BF16) are claimed by warps, one CTA per SM, each warp with a buffer of its own in
// shared memory: 6 of them BF16, 12 e4m3, as many as fit; lane b moves block b with bulk
// copies.  What bounds it is the traffic: each kept run is read once and written once.
// Small calls use units half that size.  Units of a page (3 buffers an SM) left the SMs idle at the end: 86 us instead of 81 at
// 48 x 4.3K-4.9K tokens; of 4 blocks, 82, and 195 instead of 192 at 8 x 33K-50K.
// The move is in place (or into other pages), so a unit's place may be written only when
// the blocks it held have been read.  Kept blocks move towards lower indices
// only; hence unit c's old blocks go to units <= c, and a warp that has read its
// own blocks has only to wait until the one or two lower units that took
// blocks out of unit c's place have been read as well.  Units are claimed by ticket,
// lower ones first, and read before they wait, so the lowest unit at work
// never waits and every wait ends.
//
// Measured on one B200 (time of the call, share of the 6.54 TB/s copy rate; BF16 into
// other pages, each pass among others; then the same with a cold L2, into other pages and
// in place):
//   8 x 33K-50K tokens to 8,192 blocks, 2 heads      192 us   88%; cold 197, in place 199
//   48 x 4.3K-4.9K tokens to 1,024 blocks, 1 head     81 us   81%; 10 us of it selection;
//                                                             cold 84, in place 92
//   1 x 4,163 tokens to 1,024 blocks, 2 heads         12 us   of it 6 selection, 5 moves;
//                                                             cold 18, in place 20
// e4m3, into other pages: 110, 52 and 11 us (floors 87, 35 and 1.4).
#include "qsa_common.cuh"

namespace {

using namespace qsa;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins0 = 2048, kBins1 = 2048, kBins2 = 1024;  // 11 + 11 + 10 bits of a key
constexpr int kFew = 256;  // keys that are ranked by comparing each with all
// Destination blocks that a warp moves at a time, many or few; ranks are kept for the smaller
constexpr int kUnitBlocks = 8, kSmallUnit = 4;
constexpr int kRanksPerPage = kBlocksPerPage / kSmallUnit;
constexpr int kMaxCluster = 8;
constexpr int kOnePerSm = 116 * 1024;
constexpr int kMaxRoom = 48 * 1024;  // masses the selection keeps in shared memory: 192 KiB, 196,608 tokens
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

struct EvictArgs {
  qsa_cache_t c;
  const int32_t* dst_table;  // where kept blocks go (block_table itself: in place)
  const int32_t* seq_ids;
  const int32_t* seq_len;
  int32_t n;
  const float* mass_in;
  float* mass_out;
  int64_t mass_ld;
  int32_t budget, sink, recent;
  int32_t* keep;
  int32_t* keep_count;
  int32_t* new_len;
  // workspace
  int32_t* ticket;
  int32_t* read_done;  // [n][hkv][units]
  int32_t* rank;       // [n][table_ranks + 2] kept blocks before each kSmallUnit, then the entry's
                       // old length (0: refused), so that new_len may be seq_len itself
  float* mass_tmp;     // [n][budget + 1]
  int32_t units;       // destination units a sequence can fill
  int32_t table_ranks; // ranks of a sequence's row of the table
  int32_t* st;
};

__device__ __forceinline__ uint32_t mass_key(float f) { return f != f ? 0u : float_key(f); }

// Sequence of entry i, or -1: padding (negative id), out of range or listed
// before (both flagged).  Called by a whole block; the same in every thread.
__device__ __forceinline__ int entry_seq(const EvictArgs& a, int i, bool report) {
  const int seq = a.seq_ids[i];
  if (seq < 0) return -1;
  bool bad = seq >= a.c.max_seqs;
  for (int j = threadIdx.x; j < i; j += blockDim.x) bad |= a.seq_ids[j] == seq;
  bad = __syncthreads_or(bad);
  if (bad && report && threadIdx.x == 0) flag(a.st, QSA_DEV_BAD_SEQ);
  return bad ? -1 : seq;
}

// All threads of the cluster's CTAs; orders shared and global memory among them.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The shared-memory word at `p` of CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t remote_addr(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_remote(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote(void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_remote(void* p, int rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote_addr(p, rank)), "r"(v) : "memory");
  return old;
}

// kCluster: an entry is shared by a cluster of `cluster` CTAs, else one CTA takes it.
template <bool kCluster>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(EvictArgs a, int cluster, int room) {
  const int ctas = kCluster ? cluster : 1;
  extern __shared__ float mass_s[];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int i = blockIdx.x / ctas, part = blockIdx.x % ctas;  // entry, and CTA of its cluster
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gtid = part * kSelThreads + tid, gthreads = ctas * kSelThreads;
  __shared__ uint32_t hist[kBins0 + kBins1 + kBins2];
  __shared__ int warp_sum[2][kSelWarps];
  __shared__ uint32_t s_prefix, s_need, s_in_bin, s_few, total_s[2], slice_s[kMaxCluster];
  auto sync_all = [&] {
    if constexpr (!kCluster) {
      __syncthreads();
    } else {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  };
  const int hkv = a.c.num_kv_heads;
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  for (int k = gtid; k < hkv * a.units; k += gthreads) a.read_done[(int64_t)i * hkv * a.units + k] = 0;
  int32_t* keep = a.keep + (int64_t)i * a.budget;
  int seq = entry_seq(a, i, part == 0);
  const int len = a.seq_len[i];
  if (seq >= 0 && (len < 0 || (int64_t)len > (int64_t)a.c.max_pages_per_seq * kPage)) {
    if (gtid == 0) flag(a.st, QSA_DEV_BAD_POS);
    seq = -1;
  }
  int32_t* rank = a.rank + (int64_t)i * (a.table_ranks + 2);
  if (gtid == 0) rank[a.table_ranks + 1] = seq < 0 ? 0 : len;
  if (seq < 0) {  // nothing of this entry moves; the whole cluster leaves before its first barrier
    for (int k = gtid; k < a.budget; k += gthreads) keep[k] = -1;
    if (gtid == 0) {
      a.keep_count[i] = 0;
      a.new_len[i] = len;
    }
    return;
  }
  const int nb = len / kRatio, tail = len % kRatio;
  const float* mass = a.mass_in + (int64_t)seq * a.mass_ld;
  const bool cut = nb > a.budget;
  const int lo = cut ? a.sink : nb, hi = cut ? nb - a.recent : nb;  // blocks that compete
  const int want = cut ? a.budget - a.sink - a.recent : 0;
  const int count = cut ? a.budget : nb, left = count + (tail ? 1 : 0), blocks = nb + (tail ? 1 : 0);
  // Each CTA owns a run of blocks, each of its warps a run of those, a lane every 32nd.
  // The masses of a CTA's first `room` blocks stay in shared memory, later ones are
  // read again.
  const int steps = (nb + gthreads - 1) / gthreads;
  const int c0 = part * steps * kSelThreads, c1 = min(nb, c0 + steps * kSelThreads);
  const int b0 = c0 + warp * steps * 32 + lane;
  const bool held = steps * kSelThreads <= room;  // the same in every CTA
#pragma unroll 4
  for (int b = c0 + tid; b < min(c1, c0 + room); b += kSelThreads) mass_s[b - c0] = mass[b];
  const float m_open = tail && gtid == 0 ? mass[nb] : 0.f;
  auto each = [&](auto f) {  // every block of this lane: f(block, mass)
#pragma unroll 2
    for (int k = 0; k < steps; ++k) {
      const int b = b0 + 32 * k;
      f(b, b < nb ? (b - c0 < room ? mass_s[b - c0] : mass[b]) : 0.f);
    }
  };
  for (int k = tid; k < kBins0 + kBins1 + kBins2; k += kSelThreads) hist[k] = 0;
  if (tid == 0) s_few = 0;
  sync_all();  // also: every CTA of the cluster runs before its shared memory is touched
  // ---- the cut: the want-th largest key of [lo, hi), and how many equal to it are kept.
  // Every CTA of a cluster works it out for itself from the sum of all histograms.
  uint32_t T = 0xffffffffu;
  int need = 0;
  if (want > 0) {
    uint32_t prefix = 0;
    int rest = want;
    uint32_t* h = hist;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? kBins2 : kBins0;
      const uint32_t mask = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
      each([&](int b, float x) {
        const uint32_t key = mass_key(x);
        if (b >= lo && b < hi && (key & mask) == prefix) atomicAdd(&h[(key >> sh) & (bins - 1)], 1u);
      });
      sync_all();
      // counts from the top: CTA c of the cluster sums slice c of the bins, its thread t
      // bin t of them (2t and 2t + 1 of 2,048 in one CTA), warp w the t of its lanes
      const int slice = bins / ctas, per = slice > kSelThreads ? 2 : 1;
      const int top = bins - 1 - part * slice - tid * per;
      uint32_t first = 0, second = 0;
      if constexpr (!kCluster) {
        first = h[top];
        second = per == 2 ? h[top - 1] : 0u;
      } else if (tid < slice) {
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < ctas) first += ld_remote(&h[top], c);
      }
      const uint32_t own = first + second;
      const uint32_t sum = __reduce_add_sync(0xffffffffu, own);
      if (lane == 0) warp_sum[0][warp] = (int)sum;
      __syncthreads();
      uint32_t before_warp = __reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)warp_sum[0][lane] : 0u);
      if constexpr (kCluster) {  // the slices above
        const uint32_t total = __reduce_add_sync(0xffffffffu, (uint32_t)warp_sum[0][lane]);
        if (tid < ctas) st_remote(&slice_s[part], tid, total);
        sync_all();
        before_warp += __reduce_add_sync(0xffffffffu, lane < part ? slice_s[lane] : 0u);
      }
      if (before_warp < (uint32_t)rest && before_warp + sum >= (uint32_t)rest) {  // the cut is in this warp's bins
        uint32_t inc = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
          if (lane >= d) inc += y;
        }
        const uint32_t before = before_warp + inc - own;
        if (before < (uint32_t)rest && before + own >= (uint32_t)rest) {
          const bool low = before + first < (uint32_t)rest;
          const uint32_t to = prefix | ((uint32_t)(top - low) << sh), nd = (uint32_t)rest - before - (low ? first : 0u);
          const uint32_t in = low ? second : first;
          if constexpr (!kCluster) {
            s_prefix = to;
            s_need = nd;
            s_in_bin = in;
          } else {
            for (int c = 0; c < ctas; ++c) {
              st_remote(&s_prefix, c, to);
              st_remote(&s_need, c, nd);
              st_remote(&s_in_bin, c, in);
            }
          }
        }
      }
      sync_all();
      prefix = s_prefix;
      rest = (int)s_need;
      h += bins;
      const int n = (int)s_in_bin;
      if (pass < 2 && n <= kFew) {  // few keys left: listed in the first CTA (h is free now), each
                                    // counts those above it
        each([&](int b, float x) {
          const uint32_t key = mass_key(x);
          if (b >= lo && b < hi && (key & ~0u << sh) == prefix) {
            if constexpr (!kCluster)
              h[atomicAdd(&s_few, 1u)] = key;
            else
              st_remote(&h[add_remote(&s_few, 0, 1u)], 0, key);
          }
        });
        sync_all();
        if (kCluster && part > 0) {
          if (tid < n) h[tid] = ld_remote(&h[tid], 0);
          __syncthreads();
        }
        if (tid < n) {
          const uint32_t key = h[tid];
          int above = 0, equal = 0;
#pragma unroll 4
          for (int k = 0; k < n; ++k) {
            above += h[k] > key;
            equal += h[k] == key;
          }
          if (above < rest && above + equal >= rest) {  // the same in every thread with this key
            s_prefix = key;
            s_need = (uint32_t)(rest - above);
          }
        }
        __syncthreads();
        prefix = s_prefix;
        rest = (int)s_need;
        break;
      }
    }
    T = prefix;
    need = rest;
  }
  // ---- blocks kept for certain, and ties, before each warp's run
  auto classify = [&](int b, float x, bool& g, bool& e) {
    const uint32_t key = mass_key(x);
    const bool competes = b >= lo && b < hi;
    g = b < nb && (!competes || (want > 0 && key > T));
    e = b < nb && competes && want > 0 && key == T;
  };
  int gt = 0, eq = 0;
  each([&](int b, float x) {
    bool g, e;
    classify(b, x, g, e);
    gt += g;
    eq += e;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_sum[0][warp] = gt;
    warp_sum[1][warp] = eq;
  }
  __syncthreads();
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[0][lane] : 0);
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[1][lane] : 0);
  if constexpr (kCluster) {
    if (warp == kSelWarps - 1 && lane == 0) {
      total_s[0] = (uint32_t)(gt0 + gt);
      total_s[1] = (uint32_t)(eq0 + eq);
    }
    sync_all();  // every held mass of the row has been read: it may be overwritten
    gt0 += __reduce_add_sync(0xffffffffu, lane < part ? (int)ld_remote(&total_s[0], lane) : 0);
    eq0 += __reduce_add_sync(0xffffffffu, lane < part ? (int)ld_remote(&total_s[1], lane) : 0);
    __syncwarp();
    cluster_arrive();  // done with the other CTAs' shared memory; waited for before leaving
  }
  // ---- in order: kept indices, blocks kept before each place, and the moved masses
  // (rows too long to be held pass through the workspace)
  float* out = a.mass_out + (int64_t)seq * a.mass_ld;
  float* tmp = held ? out : a.mass_tmp + (int64_t)i * (a.budget + 1);
  each([&](int b, float x) {
    bool g, e;
    classify(b, x, g, e);
    const unsigned gm = __ballot_sync(0xffffffffu, g), em = __ballot_sync(0xffffffffu, e);
    const unsigned below = (1u << lane) - 1u;
    const int eb = eq0 + __popc(em & below);
    const int at = gt0 + __popc(gm & below) + min(eb, need);
    if (b < nb) {
      if (b % kSmallUnit == 0) rank[b / kSmallUnit] = at;
      if (g || (e && eb < need)) {
        keep[at] = b;
        tmp[at] = x;
      }
    }
    gt0 += __popc(gm);
    eq0 += __popc(em);
  });
  for (int k = count + gtid; k < a.budget; k += gthreads) keep[k] = -1;
  for (int k = (nb + kSmallUnit - 1) / kSmallUnit + gtid; k <= a.table_ranks; k += gthreads) rank[k] = count;
  if (gtid == 0) {
    if (tail) tmp[count] = m_open;
    a.keep_count[i] = count;
    a.new_len[i] = count * kRatio + tail;
  }
  if constexpr (kCluster) {
    __syncwarp();
    cluster_wait();
  }
  if (!held) {
    sync_all();  // the whole row has been read
    for (int b = gtid; b < left; b += gthreads) out[b] = tmp[b];
  }
  for (int b = left + gtid; b < blocks; b += gthreads) out[b] = 0.f;
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void st_release(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// 1-D bulk async copy shared -> global; addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// A unit of the move, as lane b of a warp sees it: the unit's block b.
struct Unit {
  int unit, g;           // kUnit destination blocks of the sequence, KV head
  int32_t* done;         // read flags of the sequence and head
  int src, dst;          // physical page * 16 + slot; src -1: nothing to move
  int p0, p1;            // lower units that take blocks out of this one (none: p1 < p0); only a page
                         // of the sequence's own, written in place, still holds them
  bool any, in_place;    // the unit receives blocks; its page is the sequence's own
};

// kRunBytes: 4096 (BF16) or 2048 (e4m3); kUnit blocks of a unit; kWorkers warps, each with a buffer of one unit;
// kInPlace: dst_table is block_table.
template <int kRunBytes, int kUnit, int kWorkers>
struct MoveLay {
  static constexpr int kKcBytes = kIdxDim * 2;
  static constexpr int kBuf = kUnit * (kRunBytes + kKcBytes);
  static constexpr int kSmem = kWorkers * kBuf + kWorkers * 8;
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int kRunBytes, int kUnit, int kWorkers, bool kInPlace>
__global__ void __launch_bounds__(kWorkers * 32) evict_move_kernel(EvictArgs a, int units) {
  using LY = MoveLay<kRunBytes, kUnit, kWorkers>;
  constexpr int kRanks = kUnit / kSmallUnit, kUnitsPerPage = kBlocksPerPage / kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t buf = smem_u32(smem) + warp * LY::kBuf, bar = smem_u32(smem) + kWorkers * LY::kBuf + warp * 8;
  pdl_launch_dependents();
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait_previous();
  const int hkv = a.c.num_kv_heads;
  uint8_t* kv = static_cast<uint8_t*>(a.c.kv_pages);
  uint8_t* kc = static_cast<uint8_t*>(a.c.kc_pages);
  auto claim = [&]() {
    int t = 0;
    if (lane == 0) t = atomicAdd(a.ticket, 1);
    return __shfl_sync(0xffffffffu, t, 0);
  };
  // blocks that an entry has moved, from those it keeps and its old length
  auto total_of = [&](int count, int len) {
    if (kInPlace && count == len / kRatio) return 0;  // nothing was cut
    return count + (len % kRatio ? 1 : 0);
  };
  auto old_len = [&](int i) { return a.rank[(int64_t)i * (a.table_ranks + 2) + a.table_ranks + 1]; };
  // In place: head fastest, then entry, then unit, since a unit waits for lower ones of its
  // own sequence, which then were claimed a round of all entries ago at least (48 x
  // 4.3K-4.9K tokens, cold: 90 us, unit before entry 111).  Into other pages nothing waits,
  // and sequences in turn are read faster (8 x 33K-50K tokens: 191.7 us, in place's order 195).
  auto look_up = [&](int t) {
    Unit u;
    const int i = kInPlace ? t / hkv % a.n : t / (hkv * a.units);
    u.g = t % hkv;
    u.unit = kInPlace ? t / hkv / a.n : t / hkv % a.units;
    const int32_t* rank = a.rank + (int64_t)i * (a.table_ranks + 2);
    u.done = a.read_done + ((int64_t)i * hkv + u.g) * a.units;
    u.src = -1;
    u.dst = 0;
    const int k = u.unit * kUnit + lane;
    // independent loads first; keep may hold nothing meaningful at k, then it is not used
    const int count = a.keep_count[i], len = old_len(i), seq = a.seq_ids[i];
    const int k0 = rank[u.unit * kRanks], k1 = rank[(u.unit + 1) * kRanks];
    const int64_t row = (int64_t)max(0, min(seq, a.c.max_seqs - 1)) * a.c.max_pages_per_seq;
    const int dp = a.dst_table[row + u.unit / kUnitsPerPage], own = a.c.block_table[row + u.unit / kUnitsPerPage];
    const int kept = lane < kUnit && k < a.budget ? a.keep[(int64_t)i * a.budget + k] : 0;
    const int total = total_of(count, len);
    u.in_place = dp == own;
    u.any = u.unit * kUnit < total;
    if (!u.any && !kInPlace) {  // the entry's other units hold nothing either
      if (lane == 0) atomicMax(a.ticket, (i + 1) * hkv * a.units);
    } else if (!u.any) {  // on to the next unit in order that receives blocks
      constexpr int kLook = 4;  // x 32 entries, this unit's and then the next one's
      unsigned has[kLook];
#pragma unroll
      for (int k = 0; k < kLook; ++k) {
        const int e = i + 1 + k * 32 + lane, j = e % a.n;
        has[k] = __ballot_sync(0xffffffffu, total_of(a.keep_count[j], old_len(j)) > (u.unit + e / a.n) * kUnit);
      }
      int skip = kLook * 32;
#pragma unroll
      for (int k = kLook - 1; k >= 0; --k)
        if (has[k]) skip = k * 32 + __ffs(has[k]) - 1;
      const bool over = skip == kLook * 32 && a.n <= kLook * 32;  // no entry has blocks in later units
      if (lane == 0) atomicMax(a.ticket, over ? units : (u.unit * a.n + i + 1 + skip) * hkv);
    }
    u.p0 = k0 / kUnit;
    u.p1 = k1 > k0 && dp == own ? min(u.unit - 1, (k1 - 1) / kUnit) : -1;
    if (lane < kUnit && k < total) {
      const int b = k < count ? kept : len / kRatio;
      const int sp = a.c.block_table[row + b / kBlocksPerPage];
      if (sp < 0 || sp >= a.c.num_pages || dp < 0 || dp >= a.c.num_pages) {
        flag(a.st, QSA_DEV_BAD_PAGE);
      } else {
        u.src = sp * kBlocksPerPage + b % kBlocksPerPage;
        u.dst = dp * kBlocksPerPage + k % kBlocksPerPage;
        if (u.src == u.dst) u.src = -1;  // stays where it is
      }
    }
    return u;
  };
  auto run_at = [&](int unit, int g) {  // page * 16 + slot -> the run of head g
    return kv + (((int64_t)(unit / kBlocksPerPage) * hkv + g) * kBlocksPerPage + unit % kBlocksPerPage) * kRunBytes;
  };
  const uint64_t policy = l2_policy_evict_first();
  const uint32_t my_run = buf + lane * kRunBytes, my_kc = buf + kUnit * kRunBytes + lane * LY::kKcBytes;
  uint32_t parity = 0;
  bool sound = true;
  int t = claim();
  Unit u;
  if (t < units) u = look_up(t);
  while (t < units) {
    const bool moves = u.src >= 0, with_kc = kc && u.g == 0;
    const unsigned movers = __ballot_sync(0xffffffffu, moves);
    // ---- read
    if (movers) {
      const int bytes = (kv ? kRunBytes : 0) + (with_kc ? LY::kKcBytes : 0);
      bulk_wait_read();  // the last unit's blocks have left the buffer
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes * __popc(movers));
      __syncwarp();
      if (moves) {
        if (kv) bulk_g2s(my_run, run_at(u.src, u.g), kRunBytes, bar, policy);
        if (with_kc) bulk_g2s(my_kc, kc + (int64_t)u.src * LY::kKcBytes, LY::kKcBytes, bar, policy);
      }
    }
    // ---- the next unit's tables meanwhile (a claimed unit reads before it waits for anything)
    const Unit now = u;
    const int t_next = claim();
    if (t_next < units) u = look_up(t_next);
    // ---- the lower units that take blocks out of this one: usually read by now (at most
    // kUnit kept blocks came from here, so they went to two units)
    const int dep = now.p0 + lane;
    const bool has_dep = movers && dep <= now.p1;
    bool clear = !has_dep || ld_acquire(now.done + dep);
    if (movers) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimitNs))) {
        // the blocks have not arrived: their flag stays down, so nobody overwrites them, and nothing
        // is stored; one more bounded wait, so as not to leave with copies into this buffer in flight
        if (lane == 0) flag(a.st, QSA_DEV_TIMEOUT);
        mbar_wait_bounded(bar, parity, kWaitLimitNs);
        break;
      }
      parity ^= 1u;
    }
    const bool wait = !__all_sync(0xffffffffu, clear);
    const bool early = now.in_place || !movers;  // its neighbours wait; else the flag keeps out of the stores' way
    if (early && now.any && lane == 0) st_release(now.done + now.unit, 1);
    if (movers) {
      if (wait && !clear) {
        const uint64_t t0 = global_timer_ns();
        while (!ld_acquire(now.done + dep))
          if (global_timer_ns() - t0 > kWaitLimitNs) {
            sound = false;
            break;
          }
      }
      sound = __all_sync(0xffffffffu, sound);
      if (!sound) {  // a lower unit has not read what lies there; the buffer's copies have arrived
        if (lane == 0) flag(a.st, QSA_DEV_TIMEOUT);
        break;
      }
      __syncwarp();
      fence_proxy_async_all();  // the flags were read as ordinary memory, the stores are asynchronous
      // ---- write
      if (moves) {
        if (kv) bulk_s2g(run_at(now.dst, now.g), my_run, kRunBytes);
        if (with_kc) bulk_s2g(kc + (int64_t)now.dst * LY::kKcBytes, my_kc, LY::kKcBytes);
      }
      bulk_commit();
      if (!early && lane == 0) st_release(now.done + now.unit, 1);
    }
    t = t_next;
  }
  bulk_wait_read();  // the buffer outlives the stores' reads; the grid's end completes their writes
}

struct WorkspaceMap {
  int64_t ticket, read_done, rank, mass_tmp, total;
};

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// destination units that a sequence can fill
int32_t units_of(const qsa_cache_t& c, int32_t budget, int32_t unit) {
  const int32_t u = (budget + unit) / unit, most = c.max_pages_per_seq * (kBlocksPerPage / unit);  // and the open block
  return u < most ? u : most;
}

WorkspaceMap workspace_map(const qsa_cache_t& c, int32_t n, int32_t budget) {
  WorkspaceMap m;
  m.ticket = 0;
  m.read_done = 256;
  m.rank = m.read_done + align256((int64_t)n * c.num_kv_heads * units_of(c, budget, kSmallUnit) * 4);
  m.mass_tmp = m.rank + align256((int64_t)n * ((int64_t)c.max_pages_per_seq * kRanksPerPage + 2) * 4);
  m.total = m.mass_tmp + align256((int64_t)n * ((int64_t)budget + 1) * 4);
  return m;
}

int check_evict(const qsa_cache_t* cache, int32_t n, int32_t budget) {
  if (!cache || n < 0 || budget < 1) return QSA_ERR_INVALID_ARG;
  const qsa_cache_t& c = *cache;
  if (c.num_pages < 1 || c.max_seqs < 1 || c.max_pages_per_seq < 1 || c.num_kv_heads < 1) return QSA_ERR_INVALID_ARG;
  if (c.max_pages_per_seq > 0x7fffffff / kPage || c.num_pages > 0x7fffffff / kBlocksPerPage)
    return QSA_ERR_UNSUPPORTED;  // positions and page * 16 + slot are int32
  if (budget > 1 << 30) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

template <bool kCluster>
int launch_select(const EvictArgs& a, int ctas, int room, size_t smem, cudaStream_t s) {
  if (cudaFuncSetAttribute(evict_select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRoom * 4) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n * ctas));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel<kCluster>, a, ctas, room) != cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  return QSA_OK;
}

template <int kRunBytes, int kUnit, int kWorkers>
int launch_move(const EvictArgs& a, int units, int sms, cudaStream_t s) {
  // never two CTAs on an SM: launched early, those of a small call would pile up (one
  // sequence of 4,163 tokens: 13.5 us so, 11.8 with one each)
  constexpr int need = MoveLay<kRunBytes, kUnit, kWorkers>::kSmem, smem = need > kOnePerSm ? need : kOnePerSm;
  const auto kernel = a.dst_table == a.c.block_table ? evict_move_kernel<kRunBytes, kUnit, kWorkers, true>
                                                     : evict_move_kernel<kRunBytes, kUnit, kWorkers, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  const int grid = units < sms ? units : sms;  // at least a unit per CTA: few units spread over the SMs
  return qsa_host::launch(kernel, dim3((unsigned)grid), dim3(kWorkers * 32),
                          (size_t)smem, s, a, units);
}

}  // namespace

extern "C" int64_t qsa_evict_workspace_bytes(const qsa_cache_t* cache, int32_t n, int32_t budget) {
  const int rc = check_evict(cache, n, budget);
  if (rc != QSA_OK) return rc;
  return workspace_map(*cache, n, budget).total;
}

extern "C" int qsa_evict(const qsa_cache_t* cache, const int32_t* dst_table, const int32_t* seq_ids,
                         const int32_t* seq_len, int32_t n, const float* mass_in, float* mass_out, int64_t mass_ld,
                         int32_t budget, int32_t sink, int32_t recent, int32_t* keep, int32_t* keep_count,
                         int32_t* new_len, void* workspace, int64_t workspace_bytes, int32_t* dev_status,
                         void* stream) {
  const int rc = check_evict(cache, n, budget);
  if (rc != QSA_OK) return rc;
  const qsa_cache_t& c = *cache;
  if (sink < 0 || recent < 0 || (int64_t)sink + recent > budget) return QSA_ERR_INVALID_ARG;
  if (c.kv_dtype != QSA_KV_BF16 && c.kv_dtype != QSA_KV_FP8_E4M3) return QSA_ERR_UNSUPPORTED;
  if (n == 0) return QSA_OK;
  if ((!c.kv_pages && !c.kc_pages) || !c.block_table || !seq_ids || !seq_len || !mass_in || !mass_out || !keep ||
      !keep_count || !new_len || !workspace)
    return QSA_ERR_INVALID_ARG;
  auto misaligned = [](const void* p, uintptr_t k) { return (reinterpret_cast<uintptr_t>(p) & (k - 1)) != 0; };
  if (misaligned(c.kv_pages, 16) || misaligned(c.kc_pages, 16) || misaligned(workspace, 256))
    return QSA_ERR_INVALID_ARG;
  if (mass_ld < (int64_t)c.max_pages_per_seq * kBlocksPerPage) return QSA_ERR_INVALID_ARG;
  const WorkspaceMap m = workspace_map(c, n, budget);
  if (workspace_bytes < m.total) return QSA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  EvictArgs a;
  a.c = c;
  a.dst_table = dst_table ? dst_table : c.block_table;
  a.seq_ids = seq_ids;
  a.seq_len = seq_len;
  a.n = n;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.mass_ld = mass_ld;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.keep = keep;
  a.keep_count = keep_count;
  a.new_len = new_len;
  a.ticket = reinterpret_cast<int32_t*>(ws + m.ticket);
  a.read_done = reinterpret_cast<int32_t*>(ws + m.read_done);
  a.rank = reinterpret_cast<int32_t*>(ws + m.rank);
  a.mass_tmp = reinterpret_cast<float*>(ws + m.mass_tmp);
  a.table_ranks = c.max_pages_per_seq * kRanksPerPage;
  a.st = dev_status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  // Buffers per SM: 6 units of 8 blocks (BF16) or 12 keep the memory busy.  A call of at
  // most two such units per SM ends sooner with 4 of half the size: they spread more
  // evenly, and the first stores start earlier (one sequence of 4,163 tokens, two
  // CTAs an SM allowed, in a graph: 11.4 us, 12.7 with 2 of full size, 12.9 with 3 of half)
  a.units = units_of(c, budget, kUnitBlocks);
  const bool few = (int64_t)n * c.num_kv_heads * a.units <= 2 * sms;
  if (few) a.units = units_of(c, budget, kSmallUnit);
  const int64_t units = (int64_t)n * c.num_kv_heads * a.units;
  if (units > 0x3fffffff) return QSA_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // CTAs per entry: a cluster when its row may be long, as many as keep the call on
  // about the card's SMs (the call on one row of 65,500 blocks: 54 us with 8, 168 with 1;
  // on 8 of 10K blocks: 191, 198; on one of 1,040 blocks 14, 16)
  const int64_t blocks = (int64_t)c.max_pages_per_seq * kBlocksPerPage;
  int ctas = 1;
  while (blocks > 4096 && ctas < kMaxCluster && (int64_t)n * ctas * 2 <= 128) ctas *= 2;
  const int64_t own = (blocks + (int64_t)ctas * kSelThreads - 1) / ((int64_t)ctas * kSelThreads) * kSelThreads;
  const int room = own < kMaxRoom ? (int)own : kMaxRoom;
  if ((int64_t)n * ctas > 0x7fffffff) return QSA_ERR_UNSUPPORTED;
  // More than half an SM's shared memory: one CTA per SM.  Launched early, behind a
  // kernel that fills the GPU, the CTAs would otherwise pile up on the first SMs to
  // come free (8 rows of 10K blocks, selection alone: 38 us instead of 24).
  const size_t smem = (size_t)(room * 4 > kOnePerSm ? room * 4 : kOnePerSm);
  const int r = ctas > 1 ? launch_select<true>(a, ctas, room, smem, s) : launch_select<false>(a, 1, room, smem, s);
  if (r != QSA_OK) return r;
  if (c.kv_dtype == QSA_KV_FP8_E4M3)
    return few ? launch_move<2048, kSmallUnit, 4>(a, (int)units, sms, s)
               : launch_move<2048, kUnitBlocks, 12>(a, (int)units, sms, s);
  return few ? launch_move<4096, kSmallUnit, 4>(a, (int)units, sms, s)
             : launch_move<4096, kUnitBlocks, 6>(a, (int)units, sms, s);
}
