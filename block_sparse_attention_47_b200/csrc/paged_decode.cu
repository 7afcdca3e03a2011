// Attention of one new token per sequence over a paged key-value cache:
//     o = softmax(scale q K^T) V   over the cached keys of the sequence.
//
// Bound by HBM: K and V are read once, 2 * len * kv_heads * d * 2 bytes.
//
// Split.  A head group is up to 16 query heads that share a kv head.  The work
// of a batch is the list of its 32-key units, ordered by (sequence, set of
// one, two or four head groups, position).  The CTAs, one per SM, take equal
// consecutive shares of that list whatever the lengths, so one long sequence
// uses the whole GPU and a ragged batch leaves no SM idle.  A share that
// covers a (sequence, set) whole writes its output; the others leave (max,
// sum, O) in the workspace, two slots per CTA and head group, and a second
// kernel joins them in position order, a CTA per border of two shares (one per
// sequence and head group cost the square of the batch, as each looks at all
// lengths: 65,536 sequences of 40 keys 15.1 ms).  Where no
// sequence can be longer than 512 keys and the (sequence, head group) pairs
// fit the SMs, each takes a CTA whole and there is nothing to join.
//
// In a CTA the four warps take the same unit of the set's head groups, whose
// rows lie side by side in token-major pages: with 16-token pages this reads
// 6.03 TB/s where four warps on four units of one head group read 5.74 (with
// 64-token pages 6.44 against 6.40).  Sets of fewer than four leave several
// warps to a head group, on successive units.  Each warp has its own ring of
// 16-byte asynchronous copies (K and V rows, zero-filled behind the length, so
// whatever a page's tail holds is never read), and runs ahead over unit and
// sequence borders.  Scores and P V go through m16n8k16 matrix instructions
// with the head group as M: K and V are read from shared memory once for all
// heads of the group, which plain FMAs could not keep up with for more than
// a few heads; the wide (tcgen05) form would need 128 rows.
#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr int kDecWarps = 4;
constexpr int kUnit = 32;       // keys
constexpr int kMaxCtas = 160;   // workspace slots are sized for this many
constexpr int kHeadTile = 16;   // query heads of one kv head per CTA pass
// up to here one CTA a (sequence, head group): 4 units a warp cost less than
// the second kernel (300 keys, 2 kv heads: 5.4 to 6.1 against 7.9 us)
constexpr int kWholeKeys = 512;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct DecCfg {
  static constexpr int ROW = D * 2;
  static constexpr int HALF = kUnit * ROW;  // K (or V) rows of a unit
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int OPAD = D + 8;        // floats per merged row: rows 8 banks apart
  static constexpr int OFF_O = kDecWarps * STAGES * STAGE;
  static constexpr int OFF_ML = OFF_O + kDecWarps * kHeadTile * OPAD * 4;
  static constexpr int OFF_SCAN = OFF_ML + kDecWarps * kHeadTile * 2 * 4;
  static constexpr int SMEM = OFF_SCAN + 96;
  static constexpr int SLOT = kHeadTile * (D + 2);  // floats of a workspace slot: O, m, l
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// ---- the list of units ---------------------------------------------------------
struct Shape {
  int n_seqs, hgroups, max_len;  // hgroups: head groups per sequence
  int hw, sets;                  // head groups of a set; sets per sequence
  const int32_t* lens;
  __device__ __forceinline__ int len(int b) const {
    const int n = __ldg(lens + b);
    return n < 0 ? 0 : (n > max_len ? max_len : n);
  }
  __device__ __forceinline__ int units(int b) const { return (len(b) + kUnit - 1) / kUnit; }
};

// Exclusive scan over the block of each thread's `v`; the total in `total`.
// `scratch`: one int64 per warp and one more.
template <int kThreads>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int64_t base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += scratch[w];
    total += scratch[w];
  }
  return base + x - v;
}

// CTAs that take part: at least two units a warp
__device__ __forceinline__ int64_t active_ctas(int64_t total, int64_t n, int hw) {
  const int64_t least = 2 * kDecWarps / hw;
  const int64_t a = (total + least - 1) / least;
  return a < 1 ? 1 : (a < n ? a : n);
}

// A CTA's share [s, e) of the `total` units, and where s lies: unit `rem` of
// the pair (b, set).  All threads of the block; `scratch`: one int64
// per warp and two more.  Lengths out of range are reported where `status` is given.
struct Share {
  int64_t s, e, total, rem;
  int b, set;
};
template <int kThreads>
__device__ __forceinline__ Share find_share(const Shape& sh, int64_t cta, int64_t n_ctas,
                                            int64_t* scratch, int32_t* status) {
  Share f{};
  const int per = (sh.n_seqs + kThreads - 1) / kThreads;
  const int b_lo = min(sh.n_seqs, int(threadIdx.x) * per), b_hi = min(sh.n_seqs, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += int64_t(sh.units(b)) * sh.sets;
    if (status) {
      const int n = __ldg(sh.lens + b);
      if (n < 0 || n > sh.max_len) report_invalid(status);
    }
  }
  const int64_t before = block_scan<kThreads>(mine, scratch, f.total);
  const int64_t active = active_ctas(f.total, n_ctas, sh.hw);
  f.s = cta < active ? f.total * cta / active : f.total;
  f.e = cta < active ? f.total * (cta + 1) / active : f.total;
  if (f.s >= f.e) return f;
  int* where = reinterpret_cast<int*>(scratch + kThreads / 32);  // b, then units before it
  if (before <= f.s && f.s < before + mine) {
    int64_t at = before;
    int b = b_lo;
    for (;; ++b) {
      const int64_t u = int64_t(sh.units(b)) * sh.sets;
      if (f.s < at + u) break;
      at += u;
    }
    where[0] = b;
    *reinterpret_cast<int64_t*>(where + 2) = at;
  }
  __syncthreads();
  f.b = where[0];
  f.rem = f.s - *reinterpret_cast<int64_t*>(where + 2);
  const int n = sh.units(f.b);
  f.set = int(f.rem / n);
  f.rem -= int64_t(f.set) * n;
  return f;
}

// a (sequence, head group) without a key: its output is 0
template <typename T, int D>
__device__ __forceinline__ void zero_output(const SeqGeo& g, const DecodeIO& io, int b, int hg) {
  const int hsub = (g.group + kHeadTile - 1) / kHeadTile;
  const int kvh = hg / hsub, row0 = (hg - kvh * hsub) * kHeadTile;
  const int rows = min(kHeadTile, g.group - row0);
  T* out = static_cast<T*>(io.o.p) + int64_t(b) * io.o.sn +
           (int64_t(kvh) * g.group + row0) * io.o.sh;
  for (int i = threadIdx.x; i < rows * (D / 8); i += blockDim.x) {
    const int r = i / (D / 8);
    *reinterpret_cast<uint4*>(out + r * io.o.sh + (i - r * (D / 8)) * 8) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kDecWarps, 1)
    paged_decode_kernel(SeqGeo g, PagedCache c, const DecodeIO io, Shape sh, bool whole) {
  using C = DecCfg<D>;
  constexpr int kThreads = 32 * kDecWarps;
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  constexpr float kShift = std::is_same<T, __half>::value ? 12.f : 0.f;
  extern __shared__ __align__(128) unsigned char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sO = reinterpret_cast<float*>(sm + C::OFF_O);
  float* sML = reinterpret_cast<float*>(sm + C::OFF_ML);
  int64_t* scratch = reinterpret_cast<int64_t*>(sm + C::OFF_SCAN);  // [kDecWarps] + where
  const uint32_t ring = smem_u32(sm) + warp * C::STAGES * C::STAGE;
  cudaTriggerProgrammaticLaunchCompletion();

  // ---- this CTA's share [s, e) of the units, and where s lies
  const int hw = sh.hw, pw = kDecWarps / hw;  // head groups; warps on one
  const int hl = warp % hw, pl = warp / hw;
  int b0, hg0;  // sequence and set
  int64_t s, e, rem0;
  const int64_t cta = blockIdx.x;
  if (whole) {
    b0 = int(blockIdx.x) / sh.sets;
    hg0 = int(blockIdx.x) - b0 * sh.sets;
    const int n = __ldg(sh.lens + b0);
    if (threadIdx.x == 0 && (n < 0 || n > sh.max_len)) report_invalid(io.status);
    s = 0;
    e = sh.units(b0);
    rem0 = 0;
    if (e == 0) {
      for (int i = 0; i < hw; ++i) zero_output<T, D>(g, io, b0, hg0 * hw + i);
      return;
    }
  } else {
    const Share f = find_share<kThreads>(sh, cta, gridDim.x, scratch,
                                         blockIdx.x == 0 ? io.status : nullptr);
    s = f.s, e = f.e;
    if (s >= e) return;
    b0 = f.b, hg0 = f.set;
    rem0 = f.rem;
  }

  // ---- the copies: this warp's units s + pl, s + pl + pw, .. of the list
  struct {
    int64_t idx;
    int b, hg, unit, n_units, len;
  } p{};
  auto settle = [&] {  // unit may lie behind its (sequence, head group): move on
    while (p.unit >= p.n_units) {
      p.unit -= p.n_units;
      if (++p.hg == sh.sets) {
        p.hg = 0;
        do {
          ++p.b;
        } while (p.b < sh.n_seqs && sh.units(p.b) == 0);
        if (p.b >= sh.n_seqs) break;
        p.len = sh.len(p.b);
        p.n_units = (p.len + kUnit - 1) / kUnit;
      }
    }
  };
  p.idx = s + pl;
  p.b = b0;
  p.len = sh.len(b0);
  p.n_units = (p.len + kUnit - 1) / kUnit;
  p.hg = hg0;
  p.unit = int(rem0) + pl;
  if (p.idx < e) settle();
  // the page of this lane's key in the next unit, fetched one unit ahead
  int page = 0, tok = 0;
  bool live = false;
  auto look_up = [&] {
    const int key = p.unit * kUnit + lane;
    live = key < p.len;
    const int pi = key / c.page_size;
    tok = key - pi * c.page_size;
    page = live ? __ldg(c.table + int64_t(p.b) * c.table_stride + pi) : 0;
  };
  if (p.idx < e) look_up();
  const int hsub = (g.group + kHeadTile - 1) / kHeadTile;  // head groups per kv head
  int put = 0;
  auto produce = [&] {
    if (p.idx < e) {
      if (live && (page < 0 || page >= c.n_pages)) {
        report_invalid(io.status);
        live = false;
      }
      const int64_t off = live ? int64_t(page) * c.sp + int64_t(tok) * c.st : -1;
      const int64_t head = int64_t((p.hg * hw + hl) / hsub) * c.sh;
      const uint32_t dst0 = ring + put * C::STAGE;
      const int ch = lane % CH;
#pragma unroll
      for (int it = 0; it < CH; ++it) {
        const int row = it * (32 / CH) + lane / CH;
        const int64_t o = __shfl_sync(0xffffffffu, off, row);
        const int64_t src = (o < 0 ? 0 : o + head) + ch * 8;
        const uint32_t dst = dst0 + row * C::ROW + ((ch ^ (row & 7)) << 4);
        cp_async16(dst, static_cast<const T*>(c.k) + src, o >= 0);
        cp_async16(dst + C::HALF, static_cast<const T*>(c.v) + src, o >= 0);
      }
      p.idx += pw;
      p.unit += pw;
      if (p.idx < e) {
        settle();
        look_up();
      }
    }
    cp_async_commit();
    put = put + 1 == C::STAGES ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) produce();

  // ---- the shares of one (sequence, head group) after the other
  const float sl2 = g.scale * kLog2e;
  int get = 0;
  int64_t idx = s, widx = s + pl;
  int b = b0, len = sh.len(b0), n_units = (len + kUnit - 1) / kUnit;
  int hg = hg0, unit0 = int(rem0);
  while (idx < e) {
    const int64_t pe = min(e, idx + (n_units - unit0));
    const int hgi = hg * hw + hl, kvh = hgi / hsub, row0 = (hgi - kvh * hsub) * kHeadTile;
    const int rows = min(kHeadTile, g.group - row0);
    const int64_t head0 = int64_t(kvh) * g.group + row0;
    // Q as the A operand: rows lane/4 and +8, zero behind the group
    uint32_t qa[D / 16][4];
    {
      const int r = lane >> 2, cc = 2 * (lane & 3);
      const T* q = static_cast<const T*>(io.q.p) + int64_t(b) * io.q.sn;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const bool on = r + 8 * hf < rows;
        const T* qr = q + (head0 + (on ? r + 8 * hf : 0)) * io.q.sh + cc;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][hf] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk) : 0u;
          qa[kk][2 + hf] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk + 8) : 0u;
        }
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    for (; widx < pe; widx += pw) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      produce();  // into the stage read in the previous turn
      const uint32_t sk = ring + get * C::STAGE, sv = sk + C::HALF;
      get = get + 1 == C::STAGES ? 0 : get + 1;
      float sc[kUnit / 8][4];
#pragma unroll
      for (int nt = 0; nt < kUnit / 8; ++nt) {
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const int row = nt * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 2) {
          uint32_t kb[4];
          ldsm_x4(kb, sk + row * C::ROW + (((2 * kk + (lane >> 3)) ^ (row & 7)) << 4));
          mma16816<T>(sc[nt], qa[kk], kb[0], kb[1]);
          mma16816<T>(sc[nt], qa[kk + 1], kb[2], kb[3]);
        }
      }
      const int key0 = (unit0 + int(widx - idx)) * kUnit + 2 * (lane & 3);
      if (key0 - 2 * (lane & 3) + kUnit > len) {
#pragma unroll
        for (int nt = 0; nt < kUnit / 8; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + nt * 8 + (i & 1) >= len) sc[nt][i] = -INFINITY;
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < kUnit / 8; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], sc[nt][i]);
      float base[2];
      bool grew = false;
      float alpha[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
        const float mn = fmaxf(m[hf], mx[hf] * sl2);
        base[hf] = mn == -INFINITY ? 0.f : mn;
        alpha[hf] = ex2_approx(m[hf] - base[hf]);
        grew |= mn > m[hf];
        m[hf] = mn;
      }
      uint32_t pa[kUnit / 16][4];
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < kUnit / 8; ++nt) {
        float pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pr[i] = ex2_approx(fmaf(sc[nt][i], sl2, kShift - base[i >> 1]));
          sum[i >> 1] += pr[i];
        }
        pa[nt >> 1][2 * (nt & 1)] = pack2<T>(pr[0], pr[1]);
        pa[nt >> 1][2 * (nt & 1) + 1] = pack2<T>(pr[2], pr[3]);
      }
      l[0] = l[0] * alpha[0] + sum[0];
      l[1] = l[1] * alpha[1] + sum[1];
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          acc[i][0] *= alpha[0];
          acc[i][1] *= alpha[0];
          acc[i][2] *= alpha[1];
          acc[i][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int kt = 0; kt < kUnit / 16; ++kt) {
        const int row = kt * 16 + (lane & 15);
#pragma unroll
        for (int dc = 0; dc < CH; dc += 2) {
          uint32_t vb[4];
          ldsm_x4_t(vb, sv + row * C::ROW + (((dc + (lane >> 4)) ^ (row & 7)) << 4));
          mma16816<T>(acc[dc], pa[kt], vb[0], vb[1]);
          mma16816<T>(acc[dc + 1], pa[kt], vb[2], vb[3]);
        }
      }
    }

    // ---- the parts of this share: pw warps each have one of a head group's
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      const int r = (lane >> 2) + 8 * hf;
      if ((lane & 3) == 0) {
        sML[(warp * kHeadTile + r) * 2] = m[hf];
        sML[(warp * kHeadTile + r) * 2 + 1] = l[hf];
      }
      float* row = sO + (warp * kHeadTile + r) * C::OPAD + 2 * (lane & 3);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(row + 8 * i) = make_float2(acc[i][2 * hf], acc[i][2 * hf + 1]);
    }
    if (pw > 1)
      __syncthreads();
    else
      __syncwarp();
    const bool entire = unit0 == 0 && pe - idx == n_units;
    // slot 0: a share that began in an earlier CTA; slot 1: one that goes on in the next
    float* slot = static_cast<float*>(io.workspace) +
                  ((cta * 2 + (unit0 == 0 ? 1 : 0)) * hw + hl) * C::SLOT;
    // this warp's turn: every pw-th 16 bytes of its head group's rows
    for (int i = pl * 32 + lane; i < rows * (D / 4); i += pw * 32) {
      const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
      float mm = -INFINITY;
      for (int w = hl; w < kDecWarps; w += hw) mm = fmaxf(mm, sML[(w * kHeadTile + r) * 2]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = hl; w < kDecWarps; w += hw) {
        const float f = ex2_approx(sML[(w * kHeadTile + r) * 2] - ref);
        ll = fmaf(sML[(w * kHeadTile + r) * 2 + 1], f, ll);
        const float4 x = *reinterpret_cast<const float4*>(sO + (w * kHeadTile + r) * C::OPAD + col);
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
      }
      if (entire) {
        const float inv = 1.f / ll;
        T* dst = static_cast<T*>(io.o.p) + int64_t(b) * io.o.sn + (head0 + r) * io.o.sh + col;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
      } else {
        *reinterpret_cast<float4*>(slot + r * D + col) = o;
        if (col == 0) {
          slot[kHeadTile * D + r] = mm;
          slot[kHeadTile * D + kHeadTile + r] = ll;
        }
      }
    }
    if (pw > 1)
      __syncthreads();
    else
      __syncwarp();
    // the next (sequence, set)
    idx = pe;
    unit0 = 0;
    if (idx < e && ++hg == sh.sets) {
      hg = 0;
      do {
        ++b;
      } while (sh.units(b) == 0);
      len = sh.len(b);
      n_units = (len + kUnit - 1) / kUnit;
    }
  }
  cp_async_wait<0>();
}

// The parts of each (sequence, head group) that several CTAs shared, in
// position order: a CTA per border of two shares and head group of a set.
// Sequences without a key get their zeros here.
template <typename T, int D>
__global__ void __launch_bounds__(128)
    paged_decode_join_kernel(SeqGeo g, const DecodeIO io, Shape sh, int n_ctas) {
  using C = DecCfg<D>;
  constexpr int kThreads = 128;
  __shared__ int64_t scratch[kThreads / 32 + 2];
  __shared__ float sml[2][kMaxCtas][kHeadTile];
  const int lane = threadIdx.x & 31;
  for (int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) & ~31; at < sh.n_seqs;
       at += int64_t(gridDim.x) * kThreads) {
    uint32_t none = __ballot_sync(0xffffffffu, at + lane < sh.n_seqs && sh.len(int(at) + lane) == 0);
    for (; none; none &= none - 1) {
      T* out = static_cast<T*>(io.o.p) + (at + __ffs(none) - 1) * io.o.sn;
      for (int i = lane; i < g.heads * (D / 8); i += 32) {
        const int h = i / (D / 8);
        *reinterpret_cast<uint4*>(out + h * io.o.sh + (i - h * (D / 8)) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  const int c = blockIdx.x / sh.hw, hl = blockIdx.x - c * sh.hw;
  const Share f = find_share<kThreads>(sh, c, n_ctas, scratch, nullptr);
  cudaGridDependencySynchronize();
  if (f.s >= f.e || f.rem == 0) return;  // no share, or one that begins with a pair
  const int b = f.b, hg = f.set * sh.hw + hl;
  const int hsub = (g.group + kHeadTile - 1) / kHeadTile;
  const int kvh = hg / hsub, row0 = (hg - kvh * hsub) * kHeadTile;
  const int rows = min(kHeadTile, g.group - row0);
  T* out = static_cast<T*>(io.o.p) + int64_t(b) * io.o.sn +
           (int64_t(kvh) * g.group + row0) * io.o.sh;
  const int64_t total = f.total, active = active_ctas(total, n_ctas, sh.hw);
  const int64_t s0 = f.s - f.rem, s1 = s0 + sh.units(b);
  // the CTA whose share holds unit i
  const int c0 = int(((s0 + 1) * active + total - 1) / total) - 1;
  const int c1 = int((s1 * active + total - 1) / total) - 1;
  if (c != c0 + 1) return;  // an earlier border lies in it, too
  const int parts = c1 - c0 + 1;
  const float* ws = static_cast<const float*>(io.workspace);
  auto slot = [&](int i) {
    return ws + (((c0 + i) * 2 + (i == 0 ? 1 : 0)) * sh.hw + hl) * int64_t(C::SLOT);
  };
  for (int i = threadIdx.x; i < parts * rows; i += kThreads) {
    const int p = i / rows, r = i - p * rows;
    sml[0][p][r] = slot(p)[kHeadTile * D + r];
    sml[1][p][r] = slot(p)[kHeadTile * D + kHeadTile + r];
  }
  __syncthreads();
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float mm = -INFINITY, ll = 0.f;
    for (int p = 0; p < parts; ++p) mm = fmaxf(mm, sml[0][p][r]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    for (int p = 0; p < parts; ++p) {
      const float f = ex2_approx(sml[0][p][r] - ref);
      sml[0][p][r] = f;
      ll = fmaf(sml[1][p][r], f, ll);
    }
    const float inv = 1.f / ll;
    for (int p = 0; p < parts; ++p) sml[0][p][r] *= inv;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const float f = sml[0][p][r];
      const float4 x = __ldcg(reinterpret_cast<const float4*>(slot(p) + r * D + col));
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
    *reinterpret_cast<uint2*>(out + r * io.o.sh + col) = make_uint2(pack2<T>(o.x, o.y), pack2<T>(o.z, o.w));
  }
}

template <typename T, int D>
cudaError_t launch_t(const SeqGeo& g, const PagedCache& c, const DecodeIO& io, cudaStream_t st) {
  using C = DecCfg<D>;
  const int sms = device_sms();
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  Shape sh;
  sh.n_seqs = io.n_seqs;
  sh.hgroups = g.kv_heads * ((g.group + kHeadTile - 1) / kHeadTile);
  const int64_t reach = int64_t(c.table_width) * c.page_size;
  // keys are counted in 32 bits, the last unit's end included
  sh.max_len = int(reach < (int64_t(1) << 31) - 64 ? reach : (int64_t(1) << 31) - 64);
  sh.lens = io.lens;
  auto kern = paged_decode_kernel<T, D>;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = allow_smem(kern, C::SMEM, seen);
  if (e != cudaSuccess) return e;
  const int64_t pairs = int64_t(io.n_seqs) * sh.hgroups;
  const bool whole = pairs <= ctas && sh.max_len <= kWholeKeys;
  sh.hw = whole ? 1 : (sh.hgroups % 4 == 0 ? 4 : (sh.hgroups % 2 == 0 ? 2 : 1));
  sh.sets = sh.hgroups / sh.hw;
  kern<<<whole ? unsigned(pairs) : unsigned(ctas), 32 * kDecWarps, C::SMEM, st>>>(g, c, io, sh,
                                                                                  whole);
  e = cudaGetLastError();
  if (e != cudaSuccess || whole) return e;
  // the join's launch overlaps the first kernel; it waits for its results itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas) * unsigned(sh.hw));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_join_kernel<T, D>, g, io, sh, ctas);
}

}  // namespace

size_t decode_workspace_bytes(const SeqGeo& g) {
  return sizeof(float) * 2 * kMaxCtas * kDecWarps * (g.d == 128 ? DecCfg<128>::SLOT : DecCfg<64>::SLOT);
}

cudaError_t launch_paged_decode(const SeqGeo& g, const PagedCache& c, const DecodeIO& io,
                                cudaStream_t st) {
  if (g.d == 128)
    return g.fp16 ? launch_t<__half, 128>(g, c, io, st) : launch_t<__nv_bfloat16, 128>(g, c, io, st);
  return g.fp16 ? launch_t<__half, 64>(g, c, io, st) : launch_t<__nv_bfloat16, 64>(g, c, io, st);
}

}  // namespace bsa
