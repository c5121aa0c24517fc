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
// step.  A CTA takes up to 8 tokens and a share of their rows, a warp each row
// (two of up to 128 dims), 16 bytes per lane; a half-split pair's partner chunk
// comes by shuffle.  The rows of 4 tokens are requested together, before the
// angles are computed: each CTA computes its tokens' R/2 sines and cosines once,
// for all heads.  Few tokens spread their rows over more CTAs instead.
#include "qsa_common.cuh"

namespace {

using namespace qsa;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;  // tokens of a CTA at most
constexpr int kAhead = 4;   // tokens whose rows a warp requests together
constexpr int kMaxPairs = QSA_ROPE_MAX_PAIRS;

struct RopeArgs {
  qsa_rope_plan_t plan;
  qsa_rope_tensor_t t[QSA_ROPE_MAX_TENSORS];
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

// A warp-sized piece of a token's rows: 256-dim rows take a warp, rows of up to
// 128 dims half of one.
struct Piece {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_stride, out_stride;
  int chunk;  // the lane's 8 dims of its row
  bool live;
};

__device__ __forceinline__ Piece find_piece(const RopeArgs& a, int item, int lane) {
  int ti = 0, rows_per;
  for (;; ++ti) {
    rows_per = a.t[ti].head_dim <= 128 ? 2 : 1;
    const int cnt = (a.t[ti].heads + rows_per - 1) / rows_per;
    if (item < cnt) break;
    item -= cnt;
  }
  const qsa_rope_tensor_t& x = a.t[ti];
  const int lanes = 32 / rows_per;
  Piece p;
  p.chunk = lane % lanes;
  const int head = item * rows_per + lane / lanes;
  // in place, the dims that do not turn stay where they are
  p.live = head < x.heads && p.chunk * 8 < x.head_dim && !(x.in == x.out && p.chunk * 8 >= a.plan.rot_dim);
  const int64_t at = (int64_t)head * x.head_dim + p.chunk * 8;
  p.in = static_cast<const __nv_bfloat16*>(x.in) + at;
  p.out = static_cast<__nv_bfloat16*>(x.out) + at;
  p.in_stride = x.in_stride;
  p.out_stride = x.out_stride;
  return p;
}

template <bool kAdjacent>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[kTokens][kMaxPairs];  // cos, sin
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.plan.rot_dim / 2, rot_chunks = a.plan.rot_dim / 8;
  const int64_t tok0 = (int64_t)blockIdx.x * a.tokens;
  const int ntok = (int)min((int64_t)a.tokens, a.n - tok0);
  const int step = gridDim.y * kWarps;
  pdl_wait_previous();
  bool angles = false;
  for (int item = blockIdx.y * kWarps + warp; item < a.items || !angles; item += step) {
    const bool has = item < a.items;
    Piece p;
    if (has) p = find_piece(a, item, lane);
    for (int t0 = 0; t0 < ntok; t0 += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        if (has && t0 + u < ntok && p.live)
          v[u] = ld_row(p.in + (tok0 + t0 + u) * p.in_stride);
      }
      if (!angles) {  // every warp once, with its first rows on their way
        for (int k = tid; k < ntok * half; k += kThreads) {
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
      if (!has) break;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (t0 + u >= ntok) break;
        const float2* k2 = cs[t0 + u];
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t r[4];
        if constexpr (kAdjacent) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[e] = w[e];
            if (p.chunk < rot_chunks) {
              const float2 k = k2[p.chunk * 4 + e];
              const float x0 = __uint_as_float(w[e] << 16), x1 = __uint_as_float(w[e] & 0xffff0000u);
              r[e] = pack_bf16(x0 * k.x - x1 * k.y, x1 * k.x + x0 * k.y);
            }
          }
        } else {
          const int hc = rot_chunks / 2;  // chunks of a half
          const bool low = p.chunk < hc;
          const int from = lane + (low ? hc : -hc);
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, w[e], from & 31);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[e] = w[e];
            if (p.chunk < rot_chunks) {
              const float4 k = *reinterpret_cast<const float4*>(k2 + (low ? p.chunk : p.chunk - hc) * 8 + 2 * e);
              const float s0 = low ? -k.y : k.y, s1 = low ? -k.w : k.w;
              r[e] = pack_bf16(__uint_as_float(w[e] << 16) * k.x + __uint_as_float(o[e] << 16) * s0,
                               __uint_as_float(w[e] & 0xffff0000u) * k.z + __uint_as_float(o[e] & 0xffff0000u) * s1);
            }
          }
        }
        if (p.live)
          *reinterpret_cast<uint4*>(p.out + (tok0 + t0 + u) * p.out_stride) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
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
    a.items += t.head_dim <= 128 ? (t.heads + 1) / 2 : t.heads;
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
  // 8 tokens a CTA when that still fills the GPU (148 SMs x 8 CTAs), else fewer; then
  // rows spread over grid.y until there are about as many CTAs, a row per warp at least
  constexpr int kFill = 1024;
  a.tokens = n >= 8 * kFill ? 8 : n >= 4 * kFill ? 4 : n >= 2 * kFill ? 2 : 1;
  const int64_t gx = ((int64_t)n + a.tokens - 1) / a.tokens;
  const int rounds = (a.items + kWarps - 1) / kWarps;
  int gy = (int)(kFill / gx);
  gy = gy < 1 ? 1 : gy > rounds ? rounds : gy;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return plan->adjacent ? qsa_host::launch(rope_kernel<true>, grid, dim3(kThreads), 0, s, a)
                        : qsa_host::launch(rope_kernel<false>, grid, dim3(kThreads), 0, s, a);
}
