// New keys and values into a paged cache, keys (and queries) rotated on the
// way:  y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin  over channel pairs,
// fp32 from the table's cos and sin, rounded once to the element type.
//
// Bound by HBM: every input row is read once and every output row written
// once, and the table row of a token is shared by all of its heads.  A warp
// takes one token: it finds the token's sequence (32-way search of the
// offsets), its cache slot and its table row once, keeps its lanes' cos and
// sin in registers and walks the token's K, V and Q head rows with 16-byte
// loads and stores.  A lane owns the two 16-byte chunks that hold its
// rotation pairs, so that q_out may be q.  When tokens are few (a generation
// step) a token's rows are split over several warps (grid.y), since a lone
// warp per token is bound by the latency of its loads.
// 24,622 tokens of 24/8 heads, d = 128, with q and dense rotated keys: 98 us, 5.7
// TB/s (4 to 16 warps a CTA, 2 to 8 rows in flight and streaming hints: 98 to
// 105); 32 tokens: 2.9 us.
#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr int kWarps = 8;  // per CTA

// the last sequence with cu[b] <= t (0 when there is none), by the whole warp
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int n_seqs, int64_t t,
                                             int lane) {
  int lo = 0, n = n_seqs;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const bool below = at < lo + n && int64_t(__ldg(cu + at)) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    if (m == 0u) return lo;  // t lies in front of the first offset
    const int top = 31 - __clz(m);
    const int end = lo + n;
    lo += top * step;
    n = min(step, end - lo);
  }
  return lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps)
    kv_append_kernel(SeqGeo g, PagedCache c, const AppendIO io) {
  constexpr int kSlots = D / 16;           // 32-byte slots of a head row
  constexpr int kRowsPerPass = 32 / kSlots;  // head rows a warp moves at once
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= io.n_tokens) return;

  const int b = find_sequence(io.cu, io.n_seqs, t, lane);
  const int64_t c0 = __ldg(io.cu + b), c1 = __ldg(io.cu + b + 1);
  if (t < c0 || t >= c1) {
    // a row no sequence owns; offsets that leave the tensor or descend in
    // front of it are the caller's mistake
    if (lane == 0 && (c1 > io.n_tokens || c1 < c0)) report_invalid(io.status);
    return;
  }
  const int64_t pos = int64_t(__ldg(io.lens + b)) - (c1 - c0) + (t - c0);
  const int64_t pi = pos >= 0 ? pos / c.page_size : 0;
  const int64_t row = io.rope ? (io.rope_rows ? int64_t(__ldg(io.rope_rows + t)) : pos) : 0;
  bool bad = pos < 0 || pi >= c.table_width || c1 > io.n_tokens || c0 < 0 ||
             (io.rope && (row < 0 || row >= io.rope_n));
  int page = 0;
  if (!bad) {
    page = __ldg(c.table + int64_t(b) * c.table_stride + pi);
    bad = page < 0 || page >= c.n_pages;
  }
  if (bad) {
    if (lane == 0) report_invalid(io.status);
    return;
  }
  const int64_t slot = int64_t(page) * c.sp + (pos - pi * c.page_size) * c.st;

  // this lane's chunks: channels ca.. and cb.. (8 each); rotated pairs when
  // its 16 channels lie within rot
  const int j = lane % kSlots, sub = lane / kSlots;
  const bool turn = io.rope && 16 * j < io.rot;
  const bool halves = turn && !io.interleaved;
  const int ca = halves ? 8 * j : 16 * j;
  const int cb = halves ? (io.rot >> 1) + 8 * j : 16 * j + 8;
  float cs[8], sn[8];
  if (turn) {
    const float4* src = reinterpret_cast<const float4*>(io.rope + row * io.rot + 8 * j);
    const float4* ssrc = reinterpret_cast<const float4*>(io.rope + row * io.rot + (io.rot >> 1) + 8 * j);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(src + i), y = __ldg(ssrc + i);
      cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
      sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
    }
  }

  const int n_rows = 2 * g.kv_heads + (io.q.p ? g.heads : 0);
  const int stride = kRowsPerPass * gridDim.y;
#pragma unroll 4
  for (int r = blockIdx.y * kRowsPerPass + sub; r < n_rows; r += stride) {
    const bool is_k = r < g.kv_heads, is_v = !is_k && r < 2 * g.kv_heads;
    const int h = is_k ? r : (is_v ? r - g.kv_heads : r - 2 * g.kv_heads);
    const Rows& in = is_k ? io.k : (is_v ? io.v : io.q);
    const T* src = static_cast<const T*>(in.p) + t * in.sn + int64_t(h) * in.sh;
    uint4 a = *reinterpret_cast<const uint4*>(src + ca);
    uint4 z = *reinterpret_cast<const uint4*>(src + cb);
    if (turn && is_v) {
      // V is copied: the chunks' channels need no order
    } else if (turn) {
      uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
      uint32_t* pz = reinterpret_cast<uint32_t*>(&z);
      if (halves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x1 = unpack2<T>(pa[i]), x2 = unpack2<T>(pz[i]);
          pa[i] = pack2<T>(x1.x * cs[2 * i] - x2.x * sn[2 * i],
                           x1.y * cs[2 * i + 1] - x2.y * sn[2 * i + 1]);
          pz[i] = pack2<T>(x2.x * cs[2 * i] + x1.x * sn[2 * i],
                           x2.y * cs[2 * i + 1] + x1.y * sn[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<T>(pa[i]), y = unpack2<T>(pz[i]);
          pa[i] = pack2<T>(x.x * cs[i] - x.y * sn[i], x.y * cs[i] + x.x * sn[i]);
          pz[i] = pack2<T>(y.x * cs[4 + i] - y.y * sn[4 + i], y.y * cs[4 + i] + y.x * sn[4 + i]);
        }
      }
    }
    T* dst;
    if (is_k) {
      dst = static_cast<T*>(c.k) + slot + int64_t(h) * c.sh;
      if (io.k_out.p) {
        T* ko = static_cast<T*>(io.k_out.p) + t * io.k_out.sn + int64_t(h) * io.k_out.sh;
        *reinterpret_cast<uint4*>(ko + ca) = a;
        *reinterpret_cast<uint4*>(ko + cb) = z;
      }
    } else if (is_v) {
      dst = static_cast<T*>(c.v) + slot + int64_t(h) * c.sh;
    } else {
      dst = static_cast<T*>(io.q_out.p) + t * io.q_out.sn + int64_t(h) * io.q_out.sh;
    }
    *reinterpret_cast<uint4*>(dst + ca) = a;
    *reinterpret_cast<uint4*>(dst + cb) = z;
  }
}

template <typename T, int D>
cudaError_t launch_t(const SeqGeo& g, const PagedCache& c, const AppendIO& io, cudaStream_t st) {
  const int n_rows = 2 * g.kv_heads + (io.q.p ? g.heads : 0);
  const int per_pass = 32 / (D / 16);
  const int64_t passes = (n_rows + per_pass - 1) / per_pass;
  // about 16 warps on each of the 148 SMs when there are few tokens
  int64_t split = 148 * 16 / io.n_tokens;
  split = split < 1 ? 1 : (split > passes ? passes : split);
  const dim3 grid(unsigned((io.n_tokens + kWarps - 1) / kWarps), unsigned(split));
  kv_append_kernel<T, D><<<grid, 32 * kWarps, 0, st>>>(g, c, io);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const SeqGeo& g, const PagedCache& c, const AppendIO& io,
                             cudaStream_t st) {
  if (g.d == 128)
    return g.fp16 ? launch_t<__half, 128>(g, c, io, st) : launch_t<__nv_bfloat16, 128>(g, c, io, st);
  return g.fp16 ? launch_t<__half, 64>(g, c, io, st) : launch_t<__nv_bfloat16, 64>(g, c, io, st);
}

}  // namespace bsa
