// Attention over packed sequences on sm_100a, causal or full, grouped heads:
//     o_i = sum_j p_ij v_j,  p_i = softmax_j(scale q_i . k_j),  j < lim_i,
// lim_i = min(Lk, i + 1 + Lk - Lq) in causal order (the last query sees every
// key), Lk otherwise; a row that sees nothing gives 0.
//
// Bound by the tensor cores: 4 d flops per (query head, seen pair).
//
// A CTA takes two 128-row query tiles that walk the same K and V: the same
// rows of two heads of one kv head when the group is even (both tiles then
// have the same causal extent), else two successive tiles of one head.  Per
// 128-key step and tile: S = Q K^T (A = Q in shared memory), softmax by one
// warpgroup (a thread owns a row: one pass with a running maximum and sum),
// P over S's columns in tensor memory, O += P V (A = P in tensor memory).
// While one tile's scores are in its warpgroup the tensor pipe works on the
// other tile.  One thread issues all products, per tile in the order PV_i,
// S_(i+1): the pipe runs them in that order, so S_(i+1) may overwrite P_i's
// columns, and once S_(i+1) is signalled PV_i has finished and O may be
// rescaled.  O is rescaled only when the maximum has grown by more than 2^8.
//
// K and V come through one ring of 128-row TMA boxes of the packed tensors.
// The box of a sequence's last tile runs into its neighbour's rows (or into
// whatever lies behind the last sequence): such K columns are masked by a
// select, and those V rows are zeroed in shared memory before the product,
// since 0 times a NaN would reach the output.
//
// Few tiles and many keys (the next part of a long text): a cluster of CTAs
// shares a tile's key steps; each leaves its maxima, sums and unnormalised O
// in its own shared memory, and the cluster joins them from there in rank
// order, so no workspace is needed and results do not vary.
//
// Tensor memory (512 columns): S_u/P_u at 128 u, O_u at 256 + 128 u.
// Every wait is bounded (2 s) and reports BSA_ERR_TIMEOUT.
#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMinShare = 4;  // key steps a CTA of a cluster takes at least
#ifndef KSPLIT
#define KSPLIT 300
#endif
constexpr int kSplitCtas = KSPLIT;

template <int D>
struct FwdCfg {
  // warps 0-3 / 4-7: softmax of tile 0 / 1; 8: finds the tile, copies;
  // 9: products; 10: the V tail
  static constexpr int kThreads = 384;
  static constexpr int KB = D / 64;               // 64-column boxes
  static constexpr int BOX = 128 * 128;           // one box of 128 rows
  static constexpr int TILE = KB * BOX;           // 128 rows
  static constexpr int RING = D == 128 ? 5 : 8;   // K and V tiles
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_BAR = OFF_KV + RING * TILE;
  // full[RING] empty[RING] q s[2] p[2] o[2] fix_go fixed drain
  static constexpr int N_BARS = 2 * RING + 10;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;
  static constexpr uint32_t TMEM_COLS = 512, COL_O = 256;
  // a cluster's join: fp32 O [256][D], then (max, sum) [256]; over Q and the ring
  static constexpr int OFF_ML = 256 * D * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(OFF_ML + 256 * 8 <= OFF_BAR, "the join lies below the barriers");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

template <typename T, int D, bool HEADS, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, SeqGeo g, const PackedIO io) {
  using C = FwdCfg<D>;
  constexpr int RING = C::RING;
  constexpr float kShift = std::is_same<T, __half>::value ? 6.f : 0.f;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (base - raw);
  const uint32_t full = base + C::OFF_BAR, empty = full + 8 * RING, bar_q = empty + 8 * RING;
  const uint32_t bar_s = bar_q + 8, bar_p = bar_s + 16, bar_o = bar_p + 16;
  const uint32_t fix_go = bar_o + 16, fixed = fix_go + 8, drain = fixed + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  int* found = reinterpret_cast<int*>(sm + C::OFF_MISC + 8);  // any, q start, Lq, k start, Lk, tile
  auto slot = [&](int i) { return base + C::OFF_KV + uint32_t(i % RING) * C::TILE; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_hp = HEADS ? g.heads >> 1 : g.heads;
  const int rank = SPLIT ? int(cluster_rank()) : 0, ranks = SPLIT ? int(cluster_size()) : 1;
  const uint32_t unit = SPLIT ? blockIdx.x / uint32_t(ranks) : blockIdx.x;
  const int hp = int(unit % uint32_t(n_hp));
  const int head0 = HEADS ? 2 * hp : hp, kvh = head0 / g.group;

  // the walk of a tile: rows, and key steps of this CTA
  struct {
    bool any;
    int q0, Lq, k0, Lk, first;
    int kb, n0, n1, n;  // first key tile, steps of the two tiles, their maximum
  } w;
  auto plan = [&] {
    w.first *= HEADS ? 128 : 256;  // first row of tile 0
    auto steps = [&](int r) {      // key tiles that a tile's last row sees
      if (!w.any || r >= w.Lq) return 0;
      const int last = min(r + 128, w.Lq) - 1;
      const int lim = g.causal ? min(w.Lk, max(0, last + 1 + w.Lk - w.Lq)) : w.Lk;
      return (lim + 127) >> 7;
    };
    w.n0 = steps(w.first);
    w.n1 = HEADS ? w.n0 : steps(w.first + 128);
    w.n = max(w.n0, w.n1);
    w.kb = 0;
    if (SPLIT) {
      const int share = max(kMinShare, (w.n + ranks - 1) / ranks);
      w.kb = min(w.n, rank * share);
      const int end = min(w.n, w.kb + share);
      w.n0 = max(0, min(w.n0, end) - w.kb);
      w.n1 = max(0, min(w.n1, end) - w.kb);
      w.n = max(w.n0, w.n1);
    }
  };
  auto load_tile = [&](int i) {  // K (even) and V (odd) tiles in walk order
    const uint32_t bar = full + 8 * (i % RING);
    mbar_arrive_expect_tx(bar, C::TILE);
    tma_load_rows(slot(i), (i & 1) ? &mv : &mk, bar, w.k0 + (w.kb + (i >> 1)) * 128, kvh);
  };

  int loaded = 0;
  if (warp == 8) {
    const Tile t =
        find_tile<kWalkQ>(io.cu_q, io.total_q, io.cu_k, io.total_k, io.n_seqs, g.causal,
                          HEADS ? 128 : 256, unit / uint32_t(n_hp), lane, io.status);
    w.any = t.any;
    w.q0 = t.a.start, w.Lq = t.a.len, w.k0 = t.b.start, w.Lk = t.b.len, w.first = t.tile;
    if (lane == 0) {
      found[0] = t.any, found[1] = w.q0, found[2] = w.Lq, found[3] = w.k0, found[4] = w.Lk;
      found[5] = t.tile;
    }
    plan();
    named_bar_sync(1, 64);  // the barriers are set up
    // the copies that the first scores need start before the rest of the set-up
    if (lane == 0 && w.n > 0) {
      load_tile(0);
      loaded = 1;
      mbar_arrive_expect_tx(bar_q, ((w.n0 > 0) + (w.n1 > 0)) * C::TILE);
      for (int u = 0; u < 2; ++u)
        if ((u ? w.n1 : w.n0) > 0)
          tma_load_rows(base + C::OFF_Q + u * C::TILE, &mq, bar_q,
                        w.q0 + w.first + (HEADS ? 0 : 128 * u), head0 + (HEADS ? u : 0));
    }
    __syncwarp();
  } else if (warp == 10) {
    if (lane == 0) {
      for (int s = 0; s < RING; ++s) {
        mbar_init(full + 8 * s, 1);
        mbar_init(empty + 8 * s, 1);
      }
      mbar_init(bar_q, 1);
      for (int u = 0; u < 2; ++u) {
        mbar_init(bar_s + 8 * u, 1);
        mbar_init(bar_p + 8 * u, 4);
        mbar_init(bar_o + 8 * u, 1);
      }
      mbar_init(fix_go, 1);
      mbar_init(fixed, 1);
      mbar_init(drain, 1);
      *abort_flag = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    named_bar_sync(1, 64);
  } else if (warp == 11 && lane == 0) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  } else if (warp == 9) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (warp != 8) {
    w.any = found[0] != 0;
    w.q0 = found[1], w.Lq = found[2], w.k0 = found[3], w.Lk = found[4], w.first = found[5];
    plan();
  }
  const int n0 = w.n0, n1 = w.n1, n = w.n, kb = w.kb, Lk = w.Lk, Lq = w.Lq;
  const bool has_tail = n > 0 && (kb + n) * 128 > Lk;  // the walk ends in a partial key tile

  // what a softmax thread ends with: its row and the row's statistics
  const int u = (warp >> 2) & 1, quad = warp & 3;
  const int r = w.first + (HEADS ? 0 : 128 * u) + quad * 32 + lane;  // row within the sequence
  const bool exists = warp < 8 && w.any && r < Lq;
  const int nu = u ? n1 : n0;
  const uint32_t lane_base = uint32_t(quad * 32) << 16;
  const uint32_t tO = tmem + C::COL_O + 128u * u + lane_base;
  float m = -INFINITY, l = 0.f;
  bool ok = true;

  // The softmax threads hold a row of 128 scores and take the other warps'
  // registers: 256 * 216 + 128 * 72 = 384 * 168, those of the launch.
  if (warp == 8) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (lane == 0 && n > 0) {
      int i = loaded;
      for (; i < 2 * n; ++i) {
        if (i >= RING && !mbar_wait(empty + 8 * (i % RING), ((i / RING) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        load_tile(i);
      }
      if (!ok) report_timeout(abort_flag, io.status);
      // on an abort the newest copy into each slot (and Q) may still be landing
      if (!ok || *abort_flag) {
        mbar_wait(bar_q, 0, nullptr, 200000000ull);
        for (int j = i > RING ? i - RING : 0; j < i; ++j)
          mbar_wait(full + 8 * (j % RING), (j / RING) & 1, nullptr, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f32<T>(128, 128, false);
      constexpr uint32_t id_o = idesc_f32<T>(128, D, true);
      auto wait_full = [&](int i) {
        return mbar_wait(full + 8 * (i % RING), (i / RING) & 1, abort_flag);
      };
      auto scores = [&](int t, int i) {  // S_t = Q_t K_i^T
        const uint32_t sq = base + C::OFF_Q + t * C::TILE, sk = slot(2 * i);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + 128u * t, sdesc_sw128(sq + off, 16, 1024),
                    sdesc_sw128(sk + off, 16, 1024), id_s, kk > 0);
        }
        tc_commit(bar_s + 8 * t);
      };
      ok = mbar_wait(bar_q, 0, abort_flag) && wait_full(0);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
          if ((t ? n1 : n0) > 0) scores(t, 0);
        tc_commit(empty);
      }
      // test hook: with `stall` set no PV is issued and the softmax's wait runs out
      for (int i = 0; ok && i < n && !io.stall; ++i) {
        const int vi = 2 * i + 1, ki = 2 * i + 2;
        ok = wait_full(vi) && (i + 1 >= n || wait_full(ki));
        if (ok && has_tail && i == n - 1) {
          mbar_arrive(fix_go);  // the tail rows of V are zeroed by warp 10
          ok = mbar_wait(fixed, 0, abort_flag);
        }
        for (int t = 0; ok && t < 2; ++t) {
          const int nt = t ? n1 : n0;
          if (i >= nt) continue;
          ok = mbar_wait(bar_p + 8 * t, i & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = slot(vi);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + C::COL_O + 128u * t, tmem + 128u * t + 8u * kk,
                      sdesc_sw128(sv + kk * 2048, C::BOX, 1024), id_o, (i > 0 || kk > 0) ? 1u : 0u);
          if (i + 1 < nt)
            scores(t, i + 1);
          else
            tc_commit(bar_o + 8 * t);
        }
        if (!ok) break;
        tc_commit(empty + 8 * (vi % RING));
        if (i + 1 < n) tc_commit(empty + 8 * (ki % RING));
      }
      if (!ok) report_timeout(abort_flag, io.status);
      // every MMA this thread issued has completed once the drain barrier flips
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ V tail
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (has_tail) {
      // asked for at the walk's end: the limit grows with its length
      if (__all_sync(0xffffffffu, mbar_wait(fix_go, 0, abort_flag,
                                            2000000000ull + uint64_t(n) * 10000ull))) {
        const uint32_t sv = slot(2 * n - 1);
        for (int bx = 0; bx < C::KB; ++bx)
          for (int o = (Lk & 127) * 128 + lane * 16; o < C::BOX; o += 512)
            st_shared_v4(sv + bx * C::BOX + o, make_uint4(0u, 0u, 0u, 0u));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed);
      } else if (lane == 0) {
        report_timeout(abort_flag, io.status);
      }
    }
  } else if (warp == 11) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  } else {
    // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int lim = !exists ? 0 : (g.causal ? min(Lk, max(0, r + 1 + Lk - Lq)) : Lk);
    const uint32_t tS = tmem + 128u * u + lane_base;
    const float sl2 = g.scale * kLog2e;
    for (int i = 0; i < nu; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_s + 8 * u, i & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
      BSA_TMEM_LD128(tS, s);
      const int seen = lim - 128 * (kb + i);
      if (!__all_sync(0xffffffffu, !exists || seen >= 128)) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= seen) s[c] = 0xFF800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 2)
        mx[(c >> 1) & 3] = max3f(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      const float mxs = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
      float factor = 1.f;
      bool rescale = false;
      if (mxs > m + 8.f) {
        if (m != -INFINITY) {
          factor = ex2_approx(m - mxs);
          rescale = true;
        }
        m = mxs;
      }
      // the previous PV finished before this step's S did
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          BSA_TMEM_LD32(tO + 32u * ch, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor);
          BSA_TMEM_ST32(tO + 32u * ch, o);
        }
      }
      // P <= 2^8; fp16 shifts it up by 2^6 so that fewer small ones vanish.
      // One warp per scheduler takes 21.6 cycles a column pair here against
      // 16 of the exponential unit alone; moving a share of the exponentials
      // to the FMA pipe, or P to the products in parts, measured slower.
      const float off = (m == -INFINITY ? 0.f : -m) + kShift;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 128; c += 2) {
        float x0, x1;
        fma_f32x2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl2, sl2, off, off);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        const int a = (c >> 1) & 1;
        add_f32x2(sum[2 * a], sum[2 * a + 1], sum[2 * a], sum[2 * a + 1], p0, p1);
        s[c >> 1] = pack2<T>(p0, p1);
      }
      BSA_TMEM_ST64(tS, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p + 8 * u);
      l = l * factor + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
    if (ok && nu > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar_o + 8 * u, 0, abort_flag));
    if (!ok) {
      if (lane == 0) report_timeout(abort_flag, io.status);
    } else if (!SPLIT) {
      // -------------------------------------------------------- epilogue
      tc_fence_after();
      const int head = head0 + (HEADS ? u : 0);
      // a NaN sum stays one; a row that saw nothing gives 0
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (exists && io.lse)
        io.lse[int64_t(head) * io.total_q + w.q0 + r] = l == 0.f ? -INFINITY : m - kShift + log2f(l);
      // over the tile's own Q, which its products have read
      const uint32_t stage = base + C::OFF_Q + u * C::TILE + quad * 32 * (2 * D);
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        if (nu > 0) {  // else no product was issued
          BSA_TMEM_LD32(tO + 32u * ch, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            v[x] = pack2<T>(__uint_as_float(o[8 * j + 2 * x]) * inv,
                            __uint_as_float(o[8 * j + 2 * x + 1]) * inv);
          stage_chunk<D>(stage, lane, 4 * ch + j, make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
      const int row0 = r - lane;  // the warp's first row
      if (w.any)
        write_rows<T, D>(stage, static_cast<T*>(io.o.p) + int64_t(w.q0 + row0) * io.o.sn +
                                    int64_t(head) * io.o.sh,
                         io.o.sn, min(32, Lq - row0), lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (SPLIT) {
    // ------------------------------------------------------------ the join
    // each CTA's rows: (max, sum) and O, chunks of 4 floats swizzled by the row
    if (warp < 8) {
      const int row = 128 * u + quad * 32 + lane;
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(base + C::OFF_ML + row * 8), "f"(m),
                   "f"(l)
                   : "memory");
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        if (nu > 0) {
          BSA_TMEM_LD32(tO + 32u * ch, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(base + row * (D * 4) + (((8 * ch + j) ^ (row & 7)) << 4),
                       make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
      }
    }
    cluster_sync();
    // rank c writes rows c, c + ranks, ..: 16-byte output chunks, D / 8 a row
    if (w.any && !*abort_flag) {
      constexpr int CH = D / 8;
      for (int i = threadIdx.x; i < (256 / ranks) * CH; i += C::kThreads) {
        const int row = (i / CH) * ranks + rank, ch = i % CH;
        const int t = row >> 7, rr = w.first + (HEADS ? 0 : 128 * t) + (row & 127);
        if (rr >= Lq) continue;
        float mm = -INFINITY, ll = 0.f;
        for (int c = 0; c < ranks; ++c)
          mm = fmaxf(mm, ld_cluster_f2(peer_smem(base + C::OFF_ML + row * 8, c)).x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < ranks; ++c) {
          const float2 ml = ld_cluster_f2(peer_smem(base + C::OFF_ML + row * 8, c));
          if (ml.y == 0.f) continue;  // it saw nothing
          const float f = ex2_approx(ml.x - ref);
          ll = fmaf(ml.y, f, ll);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float4 v = ld_cluster_f4(
                peer_smem(base + row * (D * 4) + (((2 * ch + x) ^ (row & 7)) << 4), c));
            o[4 * x] = fmaf(v.x, f, o[4 * x]);
            o[4 * x + 1] = fmaf(v.y, f, o[4 * x + 1]);
            o[4 * x + 2] = fmaf(v.z, f, o[4 * x + 2]);
            o[4 * x + 3] = fmaf(v.w, f, o[4 * x + 3]);
          }
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int head = head0 + (HEADS ? t : 0);
        if (io.lse && ch == 0)
          io.lse[int64_t(head) * io.total_q + w.q0 + rr] =
              ll == 0.f ? -INFINITY : mm - kShift + log2f(ll);
        uint4 v = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                             pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
        *reinterpret_cast<uint4*>(static_cast<T*>(io.o.p) + int64_t(w.q0 + rr) * io.o.sn +
                                  int64_t(head) * io.o.sh + ch * 8) = v;
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its rows are read
  }
  if (warp == 9) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <typename T, int D, bool HEADS, bool SPLIT>
cudaError_t launch_t(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io, int64_t units,
                     int ranks, cudaStream_t st) {
  using C = FwdCfg<D>;
  auto kern = packed_fwd_kernel<T, D, HEADS, SPLIT>;
  // the register split waits for ever unless the launch brings 168 a thread
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs != 168) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = allow_smem(kern, C::SMEM, seen);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(units * ranks));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(ranks);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], g, io);
}

template <typename T, int D>
cudaError_t launch_d(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                     cudaStream_t st) {
  const bool heads = g.group % 2 == 0;
  // no more tiles than this whatever the lengths; the ones too many return
  const int64_t rows = heads ? 128 : 256;
  const int64_t tiles = io.total_q / rows + (io.n_seqs < io.total_q ? io.n_seqs : io.total_q);
  const int64_t units = tiles * (heads ? g.heads / 2 : g.heads);
  // a tile per CTA fills less than half of the 148 SMs and some sequence may
  // have keys enough for two shares: split the keys
  int ranks = 1;
  if (units <= 74 && io.total_k > 2 * kMinShare * 128) {
    ranks = 8;
    while (ranks > 2 && units * ranks > kSplitCtas) ranks /= 2;
  }
  if (ranks > 1)
    return heads ? launch_t<T, D, true, true>(g, maps, io, units, ranks, st)
                 : launch_t<T, D, false, true>(g, maps, io, units, ranks, st);
  return heads ? launch_t<T, D, true, false>(g, maps, io, units, 1, st)
               : launch_t<T, D, false, false>(g, maps, io, units, 1, st);
}

}  // namespace

cudaError_t launch_packed_fwd(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                              cudaStream_t st) {
  if (g.d == 128)
    return g.fp16 ? launch_d<__half, 128>(g, maps, io, st) : launch_d<__nv_bfloat16, 128>(g, maps, io, st);
  return g.fp16 ? launch_d<__half, 64>(g, maps, io, st) : launch_d<__nv_bfloat16, 64>(g, maps, io, st);
}

}  // namespace bsa
