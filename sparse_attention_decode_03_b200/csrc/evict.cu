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
// evict_select_kernel, one CTA per sequence: radix select of the cut (11 + 11 +
// 10 bits of the order-preserving key), then one ordered pass that writes the
// kept indices, the number kept before every page, and the moved mass row.
//
// evict_move_kernel, one CTA per (sequence, destination page, KV head).  What
// bounds it is the traffic: each kept run is read once and written once.  The
// move is in place (or into other pages), so a page may be written only when
// the blocks it held have been read.  Kept blocks move towards lower indices
// only; hence page c's old blocks go to pages <= c, and a CTA that has read its
// own 16 blocks into registers has only to wait until the one or two lower
// pages that took blocks out of page c have been read as well.  CTAs take their
// work by ticket, lower pages first, and read before they wait, so every wait
// is for a CTA that is running and reads without waiting.
#include "qsa_common.cuh"

namespace {

using namespace qsa;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
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
  int32_t* read_done;  // [n][hkv][pages of the budget]
  int32_t* rank;       // [n][max_pages_per_seq + 2] kept blocks before each page, then the entry's
                       // old length (0: refused), so that new_len may be seq_len itself
  float* mass_tmp;     // [n][budget + 1]
  int32_t pages;       // destination pages a sequence can fill
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  pdl_launch_dependents();
  pdl_wait_previous();
  const int i = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ uint32_t hist[kBins];
  __shared__ int warp_sum[2][kSelWarps];
  __shared__ uint32_t s_prefix, s_need;
  const int hkv = a.c.num_kv_heads;
  if (i == 0 && tid == 0) *a.ticket = 0;
  for (int k = tid; k < hkv * a.pages; k += kSelThreads) a.read_done[(int64_t)i * hkv * a.pages + k] = 0;
  int32_t* keep = a.keep + (int64_t)i * a.budget;
  int seq = entry_seq(a, i, true);
  const int len = a.seq_len[i];
  if (seq >= 0 && (len < 0 || (int64_t)len > (int64_t)a.c.max_pages_per_seq * kPage)) {
    if (tid == 0) flag(a.st, QSA_DEV_BAD_POS);
    seq = -1;
  }
  int32_t* rank = a.rank + (int64_t)i * (a.c.max_pages_per_seq + 2);
  if (tid == 0) rank[a.c.max_pages_per_seq + 1] = seq < 0 ? 0 : len;
  if (seq < 0) {  // nothing of this entry moves
    for (int k = tid; k < a.budget; k += kSelThreads) keep[k] = -1;
    if (tid == 0) {
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
  // ---- the cut: the want-th largest key of [lo, hi), and how many equal to it are kept
  uint32_t T = 0xffffffffu;
  int need = 0;
  if (want > 0) {
    uint32_t prefix = 0;
    int left = want;
    const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = shifts[pass], bins = 1 << widths[pass];
      for (int k = tid; k < bins; k += kSelThreads) hist[k] = 0;
      __syncthreads();
      const uint32_t mask = pass == 0 ? 0u : ~0u << (sh + widths[pass]);
      for (int b = lo + tid; b < hi; b += kSelThreads) {
        const uint32_t key = mass_key(mass[b]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> sh) & (bins - 1)], 1u);
      }
      __syncthreads();
      // suffix counts: thread t owns bins 2t, 2t + 1 counted from the top
      const int per = bins / kSelThreads;  // 2 or 1
      uint32_t own = 0;
      for (int k = 0; k < per; ++k) own += hist[bins - 1 - (tid * per + k)];
      uint32_t inc = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      if (lane == 31) warp_sum[0][warp] = (int)inc;
      __syncthreads();
      uint32_t before = inc - own;
      for (int w = 0; w < warp; ++w) before += (uint32_t)warp_sum[0][w];
      if (before < (uint32_t)left && before + own >= (uint32_t)left) {
        uint32_t acc = before;
        for (int k = 0; k < per; ++k) {
          const int bin = bins - 1 - (tid * per + k);
          if (acc + hist[bin] >= (uint32_t)left) {
            s_prefix = prefix | ((uint32_t)bin << sh);
            s_need = (uint32_t)left - acc;
            break;
          }
          acc += hist[bin];
        }
      }
      __syncthreads();
      prefix = s_prefix;
      left = (int)s_need;
      __syncthreads();
    }
    T = prefix;
    need = left;
  }
  // ---- kept blocks in order: each warp owns a run of whole pages' worth of blocks
  const int per_warp = ((nb + kSelWarps * 32 - 1) / (kSelWarps * 32)) * 32;
  const int b0 = warp * per_warp, b1 = min(nb, b0 + per_warp);
  int gt = 0, eq = 0;  // blocks kept for certain, and ties
  for (int b = b0 + lane; b - lane < b1; b += 32) {
    bool g = false, e = false;
    if (b < b1) {
      if (b < lo || b >= hi) {
        g = true;
      } else if (want > 0) {
        const uint32_t key = mass_key(mass[b]);
        g = key > T;
        e = key == T;
      }
    }
    gt += __popc(__ballot_sync(0xffffffffu, g));
    eq += __popc(__ballot_sync(0xffffffffu, e));
  }
  if (lane == 0) {
    warp_sum[0][warp] = gt;
    warp_sum[1][warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int w = 0; w < warp; ++w) {
    gt0 += warp_sum[0][w];
    eq0 += warp_sum[1][w];
  }
  const int count = cut ? a.budget : nb;
  float* tmp = a.mass_tmp + (int64_t)i * (a.budget + 1);
  for (int b = b0 + lane; b - lane < b1; b += 32) {
    bool g = false, e = false;
    float m = 0.f;
    if (b < b1) {
      m = mass[b];
      if (b < lo || b >= hi) {
        g = true;
      } else if (want > 0) {
        const uint32_t key = mass_key(m);
        g = key > T;
        e = key == T;
      }
    }
    const unsigned gm = __ballot_sync(0xffffffffu, g), em = __ballot_sync(0xffffffffu, e);
    const unsigned below = (1u << lane) - 1u;
    const int eb = eq0 + __popc(em & below);
    const int at = gt0 + __popc(gm & below) + min(eb, need);
    if (b < b1) {
      if (b % kBlocksPerPage == 0) rank[b / kBlocksPerPage] = at;
      if (g || (e && eb < need)) {
        keep[at] = b;
        tmp[at] = m;
      }
    }
    gt0 += __popc(gm);
    eq0 += __popc(em);
  }
  for (int k = count + tid; k < a.budget; k += kSelThreads) keep[k] = -1;
  for (int P = (nb + kBlocksPerPage - 1) / kBlocksPerPage + tid; P <= a.c.max_pages_per_seq; P += kSelThreads)
    rank[P] = count;
  if (tid == 0) {
    if (tail) tmp[count] = mass[nb];
    a.keep_count[i] = count;
    a.new_len[i] = count * kRatio + tail;
  }
  __syncthreads();  // the whole row has been read: it may be overwritten
  const int blocks = nb + (tail ? 1 : 0), left = count + (tail ? 1 : 0);
  float* out = a.mass_out + (int64_t)seq * a.mass_ld;
  for (int b = tid; b < blocks; b += kSelThreads) out[b] = b < left ? tmp[b] : 0.f;
}

// 16-byte load that other CTAs' stores of this launch must not be cached against.
__device__ __forceinline__ uint4 ld_l2(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void st_release(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Runs of kRunBytes: 4096 (BF16) or 2048 (e4m3).
template <int kRunBytes>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
  constexpr int kRunThreads = kRunBytes / 16;              // threads that carry one run
  constexpr int kRunsAtOnce = kMoveThreads / kRunThreads;  // 1 or 2
  constexpr int kRounds = kBlocksPerPage / kRunsAtOnce;
  pdl_launch_dependents();
  pdl_wait_previous();
  const int tid = threadIdx.x;
  __shared__ int s_ticket, s_ok;
  __shared__ int s_src[kBlocksPerPage], s_dst;  // source page * 16 + slot (-1: none) of each block, destination page
  if (tid == 0) s_ticket = atomicAdd(a.ticket, 1);
  __syncthreads();
  const int hkv = a.c.num_kv_heads;
  const int g = s_ticket % hkv, page = (s_ticket / hkv) % a.pages, i = s_ticket / (hkv * a.pages);
  const int32_t* rank = a.rank + (int64_t)i * (a.c.max_pages_per_seq + 2);
  const int count = a.keep_count[i], len = rank[a.c.max_pages_per_seq + 1], seq = a.seq_ids[i];
  const int tail = len % kRatio, first = page * kBlocksPerPage;
  const int total = count + (tail ? 1 : 0);
  if (first >= total) return;
  const int nblk = min(kBlocksPerPage, total - first);
  const int64_t row = (int64_t)seq * a.c.max_pages_per_seq;
  if (tid < kBlocksPerPage) {
    int src = -1;
    if (tid < nblk) {
      const int b = first + tid < count ? a.keep[(int64_t)i * a.budget + first + tid] : len / kRatio;
      const int sp = a.c.block_table[row + b / kBlocksPerPage];
      if (sp < 0 || sp >= a.c.num_pages)
        flag(a.st, QSA_DEV_BAD_PAGE);
      else
        src = b % kBlocksPerPage + kBlocksPerPage * sp;
    }
    s_src[tid] = src;
  }
  if (tid == 32) {
    int dp = a.dst_table[row + page];
    if (dp < 0 || dp >= a.c.num_pages) {
      flag(a.st, QSA_DEV_BAD_PAGE);
      dp = -1;
    }
    s_dst = dp;
  }
  __syncthreads();
  const int dp = s_dst;
  // ---- read
  uint8_t* kv = static_cast<uint8_t*>(a.c.kv_pages);
  const int sub = tid / kRunThreads, off = (tid % kRunThreads) * 16;
  auto run_at = [&](int64_t unit) {  // page * 16 + slot -> the run of head g
    return ((unit / kBlocksPerPage * hkv + g) * kBlocksPerPage + unit % kBlocksPerPage) * kRunBytes + off;
  };
  uint4 x[kRounds], kc = make_uint4(0, 0, 0, 0);
  uint32_t landed = 0;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    x[r] = make_uint4(0, 0, 0, 0);
    const int src = s_src[r * kRunsAtOnce + sub];
    if (kv && src >= 0 && src != dp * kBlocksPerPage + r * kRunsAtOnce + sub) x[r] = ld_l2(kv + run_at(src));
  }
  uint8_t* kcp = static_cast<uint8_t*>(a.c.kc_pages);
  const int kblk = tid >> 4;
  const bool with_kc = kcp && g == 0 && s_src[kblk] >= 0 && s_src[kblk] != dp * kBlocksPerPage + kblk;
  if (with_kc) kc = ld_l2(kcp + (int64_t)s_src[kblk] * 256 + (tid & 15) * 16);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) landed |= x[r].x;
  __syncthreads_or((landed | kc.x) != 0);  // takes the loaded values: every thread's reads have landed before the flag
  int32_t* done = a.read_done + ((int64_t)i * hkv + g) * a.pages;
  if (tid == 0) {
    __threadfence();
    st_release(done + page, 1);
    // ---- wait for the lower pages that took blocks out of this one
    const int k0 = rank[page], k1 = rank[page + 1];
    int ok = 1;
    if (k1 > k0) {
      const int p1 = min(page - 1, (k1 - 1) / kBlocksPerPage);
      for (int p = k0 / kBlocksPerPage; p <= p1 && ok; ++p) {
        const uint64_t t0 = global_timer_ns();
        while (!ld_acquire(done + p)) {
          if (global_timer_ns() - t0 > kWaitLimitNs) {
            flag(a.st, QSA_DEV_TIMEOUT);
            ok = 0;
            break;
          }
        }
      }
    }
    __threadfence();
    s_ok = ok;
  }
  __syncthreads();
  if (!s_ok || dp < 0) return;
  // ---- write
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int b = r * kRunsAtOnce + sub, src = s_src[b];
    if (kv && src >= 0 && src != dp * kBlocksPerPage + b)
      *reinterpret_cast<uint4*>(kv + run_at((int64_t)dp * kBlocksPerPage + b)) = x[r];
  }
  if (with_kc)
    *reinterpret_cast<uint4*>(kcp + ((int64_t)dp * kBlocksPerPage + kblk) * 256 + (tid & 15) * 16) = kc;
}

struct WorkspaceMap {
  int64_t ticket, read_done, rank, mass_tmp, total;
};

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

int32_t pages_of_budget(int32_t budget) { return (int32_t)(((int64_t)budget + 1 + kBlocksPerPage - 1) / kBlocksPerPage); }

WorkspaceMap workspace_map(const qsa_cache_t& c, int32_t n, int32_t budget) {
  WorkspaceMap m;
  m.ticket = 0;
  m.read_done = 256;
  m.rank = m.read_done + align256((int64_t)n * c.num_kv_heads * pages_of_budget(budget) * 4);
  m.mass_tmp = m.rank + align256((int64_t)n * ((int64_t)c.max_pages_per_seq + 2) * 4);
  m.total = m.mass_tmp + align256((int64_t)n * ((int64_t)budget + 1) * 4);
  return m;
}

int check_evict(const qsa_cache_t* cache, int32_t n, int32_t budget) {
  if (!cache || n < 0 || budget < 1) return QSA_ERR_INVALID_ARG;
  const qsa_cache_t& c = *cache;
  if (c.num_pages < 1 || c.max_seqs < 1 || c.max_pages_per_seq < 1 || c.num_kv_heads < 1) return QSA_ERR_INVALID_ARG;
  if (c.max_pages_per_seq > 0x7fffffff / kPage || c.num_pages > 0x7fffffff / kBlocksPerPage)
    return QSA_ERR_UNSUPPORTED;  // positions and page * 16 + slot are int32
  if ((int64_t)budget > (int64_t)c.max_pages_per_seq * kBlocksPerPage) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
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
  a.pages = pages_of_budget(budget);
  if (a.pages > c.max_pages_per_seq) a.pages = c.max_pages_per_seq;
  a.st = dev_status;
  const int64_t grid = (int64_t)n * c.num_kv_heads * a.pages;
  if (grid > 0x7fffffff) return QSA_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int r = qsa_host::launch(evict_select_kernel, dim3((unsigned)n), dim3(kSelThreads), 0, s, a);
  if (r != QSA_OK) return r;
  return c.kv_dtype == QSA_KV_FP8_E4M3
             ? qsa_host::launch(evict_move_kernel<2048>, dim3((unsigned)grid), dim3(kMoveThreads), 0, s, a)
             : qsa_host::launch(evict_move_kernel<4096>, dim3((unsigned)grid), dim3(kMoveThreads), 0, s, a);
}
