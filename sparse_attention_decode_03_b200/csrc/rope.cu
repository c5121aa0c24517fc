// qsa_rope: rotary positions with one to three axes (time, height, width),
// applied to up to four tensors of the same tokens in one launch: the main
// queries and keys, and the indexer's, before qsa_append_kv and the attention.
//
// Pair i of a head (dims i and i + R/2, or 2i and 2i + 1) turns by the angle
// pos[axis(i)] * freq(i):
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin   (fp32, one rounding to BF16)
// Dims R and above are copied.  The angle is reduced to one turn in 64 bits: a
// position of a quarter-million tokens times a frequency near 1 has lost about
// 2^-7 rad in fp32.  sin and cos of the reduced turn are taken in fp32.
//
// What bounds it: the bytes of the rows for a prompt chunk, latency for a decode
// step.  A CTA takes up to 4 tokens and a share of their rows, 16 bytes per lane.
// The chunks that turn (R / 8 of a row) and those that are only copied go to
// different warps: with R = 64 of 256 dims a warp turns 4 rows at once instead of
// one with three quarters of its lanes idle, which took 139 instructions a row
// and 55 us for 8,192 tokens of 24 + 2 heads and an indexer's (now 45 us, 5.7 TB/s).  A half-split pair's partner chunk comes by
// shuffle.  The chunks of all its tokens are requested together, before the angles
// are computed: each CTA computes its tokens' R/2 sines and cosines once, for all
// heads.  Few tokens spread their rows over more CTAs instead.
#include "qsa_common.cuh"

namespace {

using namespace qsa;

constexpr int kWarps = 8;      // of a CTA; kWideWarps for long calls
constexpr int kWideWarps = 16;
constexpr int kTokens = 4;  // tokens of a CTA at most; a warp requests its chunks of all of them together
constexpr int kMaxPairs = QSA_ROPE_MAX_PAIRS;

// What turns a tensor's rows into warp-sized pieces: first the chunks that turn,
// rows_per rows to a warp, then the copied ones, 32 to a warp (none in place).
struct Cut {
  int turn_chunks, copy_chunks, rows_per, turns, copies;
};
Cut cut_of(const qsa_rope_tensor_t& t, int rot_dim) {
  Cut c;
  c.turn_chunks = rot_dim / 8;
  c.copy_chunks = (t.head_dim - rot_dim) / 8;
  c.rows_per = 32 / c.turn_chunks;
  c.turns = (t.heads + c.rows_per - 1) / c.rows_per;
  c.copies = t.in == t.out ? 0 : (t.heads * c.copy_chunks + 31) / 32;
  return c;
}

struct RopeArgs {
  qsa_rope_plan_t plan;
  qsa_rope_tensor_t t[QSA_ROPE_MAX_TENSORS];
  Cut cut[QSA_ROPE_MAX_TENSORS];
  int32_t num_tensors;
  int32_t items;  // warp-sized pieces of one token's rows
  const int32_t* pos;
  int64_t pos_stride;
  int32_t n;
  int32_t tokens;  // of a CTA
};

// 16-byte load that leaves L1 alone.  Not the read-only path: out may be in.
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// A piece, as one lane sees it.
struct Piece {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_stride, out_stride;
  int chunk;  // the lane's 8 dims of its row
  bool turns, live;
};

__device__ __forceinline__ Piece find_piece(const RopeArgs& a, int item, int lane) {
  int ti = 0;
  while (item >= a.cut[ti].turns + a.cut[ti].copies) {
    item -= a.cut[ti].turns + a.cut[ti].copies;
    ++ti;
  }
  const Cut& c = a.cut[ti];
  const qsa_rope_tensor_t& x = a.t[ti];
  Piece p;
  p.turns = item < c.turns;
  int head;
  if (p.turns) {
    head = item * c.rows_per + lane / c.turn_chunks;
    p.chunk = lane % c.turn_chunks;
    p.live = head < x.heads && lane / c.turn_chunks < c.rows_per;
  } else {
    const int k = (item - c.turns) * 32 + lane;
    head = k / c.copy_chunks;
    p.chunk = c.turn_chunks + k % c.copy_chunks;
    p.live = head < x.heads;
  }
  const int64_t at = (int64_t)head * x.head_dim + p.chunk * 8;
  p.in = static_cast<const __nv_bfloat16*>(x.in) + at;
  p.out = static_cast<__nv_bfloat16*>(x.out) + at;
  p.in_stride = x.in_stride;
  p.out_stride = x.out_stride;
  return p;
}

template <bool kAdjacent, int kW>
__global__ void __launch_bounds__(kW * 32) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 cs[kTokens][kMaxPairs];  // cos, sin
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.plan.rot_dim / 2;
  const int64_t tok0 = (int64_t)blockIdx.x * a.tokens;
  const int ntok = (int)min((int64_t)a.tokens, a.n - tok0);
  const int step = gridDim.y * kW;
  pdl_wait_previous();
  bool angles = false;
  for (int item = blockIdx.y * kW + warp; item < a.items || !angles; item += step) {
    const bool has = item < a.items;
    Piece p = {};
    if (has) p = find_piece(a, item, lane);
    uint4 v[kTokens];
    const __nv_bfloat16* src = p.in + tok0 * p.in_stride;
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (p.live && u < ntok) v[u] = ld_row(src + u * p.in_stride);
    }
    if (!angles) {  // every warp once, with its first rows on their way
      for (int k = tid; k < ntok * half; k += kW * 32) {
        const int i = k % half, t = k / half;
        double turn = (double)a.pos[a.plan.axis[i] * a.pos_stride + tok0 + t] * a.plan.freq[i] *
                      0.15915494309189533577;  // 1 / 2 pi
        turn -= rint(turn);
        float s, c;
        sincospif(2.f * (float)turn, &s, &c);
        cs[t][i] = make_float2(c, s);
      }
      __syncthreads();
      angles = true;
    }
    if (!has) continue;
    if (p.turns) {
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        if (u >= ntok) break;
        const float2* k2 = cs[u];
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t r[4];
        if constexpr (kAdjacent) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 k = k2[p.chunk * 4 + e];
            const float x0 = __uint_as_float(w[e] << 16), x1 = __uint_as_float(w[e] & 0xffff0000u);
            r[e] = pack_bf16(x0 * k.x - x1 * k.y, x1 * k.x + x0 * k.y);
          }
        } else {
          const int hc = a.plan.rot_dim / 16;  // chunks of a half
          const bool low = p.chunk < hc;
          const int from = lane + (low ? hc : -hc);
          const float2* k8 = k2 + (low ? p.chunk : p.chunk - hc) * 8;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t o = __shfl_sync(0xffffffffu, w[e], from & 31);
            const float4 k = *reinterpret_cast<const float4*>(k8 + 2 * e);
            const float s0 = low ? -k.y : k.y, s1 = low ? -k.w : k.w;
            r[e] = pack_bf16(__uint_as_float(w[e] << 16) * k.x + __uint_as_float(o << 16) * s0,
                             __uint_as_float(w[e] & 0xffff0000u) * k.z + __uint_as_float(o & 0xffff0000u) * s1);
          }
        }
        v[u] = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
    __nv_bfloat16* dst = p.out + tok0 * p.out_stride;
#pragma unroll
    for (int u = 0; u < kTokens; ++u)
      if (p.live && u < ntok) *reinterpret_cast<uint4*>(dst + u * p.out_stride) = v[u];
  }
}

// n rows of `row` elements, `stride` apart.
struct Rows {
  uintptr_t at;
  int64_t stride, row;
};

// Whether two sets of n rows share an element.  Rows of one stride may
// interleave (column slices of one buffer); of different strides, sets whose
// byte ranges cross count as overlapping.
bool rows_overlap(const Rows& x, const Rows& y, int32_t n) {
  const uintptr_t xe = x.at + 2 * (uintptr_t)((n - 1) * x.stride + x.row);
  const uintptr_t ye = y.at + 2 * (uintptr_t)((n - 1) * y.stride + y.row);
  if (xe <= y.at || ye <= x.at) return false;
  if (n == 1 || x.stride != y.stride) return true;
  const int64_t s = 2 * x.stride, d = (int64_t)(y.at - x.at);
  const int64_t r = ((d % s) + s) % s;  // y's column offset from x's rows, in bytes
  return r < 2 * x.row || r + 2 * y.row > s;
}

}  // namespace

extern "C" int qsa_rope(const qsa_rope_plan_t* plan, const qsa_rope_tensor_t* tensors, int32_t num_tensors,
                        const int32_t* pos, int64_t pos_stride, int32_t n, void* stream) {
  if (!plan || !tensors || num_tensors < 1 || num_tensors > QSA_ROPE_MAX_TENSORS || n < 0) return QSA_ERR_INVALID_ARG;
  if (plan->rot_dim < 16 || plan->rot_dim % 16 || plan->rot_dim > 2 * QSA_ROPE_MAX_PAIRS) return QSA_ERR_INVALID_ARG;
  if (plan->num_axes < 1 || plan->num_axes > QSA_ROPE_MAX_AXES) return QSA_ERR_INVALID_ARG;
  for (int i = 0; i < plan->rot_dim / 2; ++i)
    if (plan->axis[i] >= plan->num_axes || !(plan->freq[i] - plan->freq[i] == 0.0)) return QSA_ERR_INVALID_ARG;
  if (n == 0) return QSA_OK;
  if (!pos || (plan->num_axes > 1 && pos_stride < n)) return QSA_ERR_INVALID_ARG;
  RopeArgs a;
  a.plan = *plan;
  a.num_tensors = num_tensors;
  a.items = 0;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.n = n;
  for (int k = 0; k < num_tensors; ++k) {
    const qsa_rope_tensor_t& t = tensors[k];
    if (!t.in || !t.out || t.heads < 1) return QSA_ERR_INVALID_ARG;
    if (t.head_dim < plan->rot_dim || t.head_dim % 16 || t.head_dim > QSA_HEAD_DIM) return QSA_ERR_INVALID_ARG;
    const int64_t row = (int64_t)t.heads * t.head_dim;
    if (row > (1 << 24)) return QSA_ERR_UNSUPPORTED;
    if (n > 1 && (t.in_stride < row || t.out_stride < row)) return QSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(t.in) & 15u) || (reinterpret_cast<uintptr_t>(t.out) & 15u) ||
        (n > 1 && ((t.in_stride & 7) || (t.out_stride & 7))))
      return QSA_ERR_INVALID_ARG;
    a.t[k] = t;
    a.cut[k] = cut_of(t, plan->rot_dim);
    a.items += a.cut[k].turns + a.cut[k].copies;
  }
  // an output may be its own input; any other overlap would read rotated rows
  for (int j = 0; j < num_tensors; ++j) {
    const int64_t row = (int64_t)tensors[j].heads * tensors[j].head_dim;
    const Rows o{reinterpret_cast<uintptr_t>(tensors[j].out), tensors[j].out_stride, row};
    for (int k = 0; k < num_tensors; ++k) {
      const int64_t row_k = (int64_t)tensors[k].heads * tensors[k].head_dim;
      const Rows ik{reinterpret_cast<uintptr_t>(tensors[k].in), tensors[k].in_stride, row_k};
      const Rows ok{reinterpret_cast<uintptr_t>(tensors[k].out), tensors[k].out_stride, row_k};
      const bool in_place = j == k && ik.at == o.at && (n == 1 || ik.stride == o.stride);
      if (!in_place && rows_overlap(o, ik, n)) return QSA_ERR_INVALID_ARG;
      if (j < k && rows_overlap(o, ok, n)) return QSA_ERR_INVALID_ARG;
    }
  }
  // 4 tokens a CTA when that still fills the GPU (148 SMs x 5 CTAs), else fewer; then rows
  // spread over grid.y until there are about as many CTAs, a piece per warp at least
  // (8,192 tokens: 4 of them 45 us, 2: 56, 8: 47; 57 tokens: 2.5 us, unspread 3.8)
  constexpr int kFill = 1024;
  a.tokens = n >= 4 * kFill ? 4 : n >= 2 * kFill ? 2 : 1;
  const int64_t gx = ((int64_t)n + a.tokens - 1) / a.tokens;
  // 16 warps a CTA where a token has work for them (8,192 tokens of 24 + 2 heads and an
  // indexer's: 45.1 us, with 8 warps 48.0, with 24 51.4; one token: 2.45 us, with 8 2.28).
  // Streaming stores gain 0.9 us more, but the rows are read again by the next kernels.
  const bool wide = a.tokens == kTokens && a.items > kWarps;
  const int warps = wide ? kWideWarps : kWarps;
  const int rounds = (a.items + warps - 1) / warps;
  int gy = (int)(kFill / gx);
  gy = gy < 1 ? 1 : gy > rounds ? rounds : gy;
  const dim3 grid((unsigned)gx, (unsigned)gy), block((unsigned)warps * 32);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (wide)
    return plan->adjacent ? qsa_host::launch(rope_kernel<true, kWideWarps>, grid, block, 0, s, a)
                          : qsa_host::launch(rope_kernel<false, kWideWarps>, grid, block, 0, s, a);
  return plan->adjacent ? qsa_host::launch(rope_kernel<true, kWarps>, grid, block, 0, s, a)
                        : qsa_host::launch(rope_kernel<false, kWarps>, grid, block, 0, s, a);
}
