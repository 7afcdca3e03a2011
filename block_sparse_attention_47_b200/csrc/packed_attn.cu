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
// K and V come as 128-row TMA boxes of the packed tensors, in a ring of
// stages of two tiles: V_i beside K_(i+1), which the same turn of the products
// takes, so a turn waits for and releases one stage (each such step costs the
// issuing thread some 150 cycles, during which the pipe runs dry).
// The box of a sequence's last tile runs into its neighbour's rows (or into
// whatever lies behind the last sequence): such K columns are masked by a
// select, and those V rows are zeroed in shared memory before the product,
// since 0 times a NaN would reach the output.
//
// The grid is one CTA per SM; a CTA takes every G-th tile of the list, longest
// walks first and back and forth, so that shares come out alike.  The steps of
// a CTA's entries form one sequence: the stage of an entry's last V holds the
// next one's first K, and the turn that issues a tile's last PV issues its next
// entry's first scores behind it, while the other tile is still at its softmax
// (that entry has been found and its Q loaded by then).  A warpgroup
// writes its rows under those products.  8,064 and 5,003 queries to 512 and 77
// keys, 24 heads, d = 128: 77 us, 91 with an entry's scores issued once both
// tiles of the previous one had finished.
//
// Few tiles and many keys (the next part of a long text): a cluster of CTAs
// shares a tile's key steps; each leaves its maxima, sums and unnormalised O
// in its own shared memory, and the cluster joins them from there in rank
// order, so no workspace is needed and results do not vary.
//
// Tensor memory (512 columns): S_u/P_u at 128 u, O_u at 256 + 128 u.
// Every wait is bounded and reports BSA_ERR_TIMEOUT: 2 s, 20 s where it may last
// as long as another tile's walk.
#include <cmath>

#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMinShare = 2;  // key steps a CTA of a cluster takes at least

template <int D>
struct FwdCfg {
  // warps 0-3 / 4-7: softmax of tile 0 / 1; 8: copies; 9: products; 10: the V
  // tails; 11: finds the entries
  static constexpr int kThreads = 384;
  static constexpr int KB = D / 64;               // 64-column boxes
  static constexpr int BOX = 128 * 128;           // one box of 128 rows
  static constexpr int TILE = KB * BOX;           // 128 rows
  static constexpr int RING = D == 128 ? 2 : 4;   // stages: V_(j-1), then K_j
  static constexpr int STAGE = 32 * 128;          // a warp's 32 rows of 64 output channels
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_STAGE = OFF_KV + RING * 2 * TILE;
  static constexpr int OFF_BAR = OFF_STAGE + 8 * STAGE;
  static constexpr int INFO = 4;                  // entries that may be published at a time
  // full[RING] empty[RING] q[2] q_free[2] info[INFO] info_free[INFO] s[2] p[2]
  // o[2] fix_go fixed drain
  static constexpr int N_BARS = 2 * RING + 2 * INFO + 13;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;  // tmem, abort, then info[INFO][8]
  static constexpr int SMEM = OFF_MISC + 16 + 32 * INFO + 1024;
  static constexpr uint32_t TMEM_COLS = 512, COL_O = 256;
  // a cluster's join: fp32 O [256][D], then (max, sum) [256]; over Q and the ring
  static constexpr int OFF_ML = 256 * D * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(OFF_ML + 256 * 8 <= OFF_BAR, "the join lies below the barriers");
};

// One entry of the tile list for this CTA: the sequence's rows and keys, the
// first row of tile 0, this CTA's key steps.
struct Plan {
  bool any;
  int q0, Lq, k0, Lk, first, hp;
  int kb, n0, n1, n;  // first key tile, steps of the two tiles, their maximum
  int off0, off1;     // where their rows start, from `first` on
};

template <typename T, int D, bool HEADS, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, SeqGeo g, const PackedIO io,
                      int n_units) {
  using C = FwdCfg<D>;
  constexpr int RING = C::RING;
  constexpr float kShift = std::is_same<T, __half>::value ? 6.f : 0.f;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (base - raw);
  const uint32_t full = base + C::OFF_BAR, empty = full + 8 * RING, bar_q = empty + 8 * RING;
  const uint32_t q_free = bar_q + 16, bar_info = q_free + 16;
  const uint32_t info_free = bar_info + 8 * C::INFO;
  const uint32_t bar_s = info_free + 8 * C::INFO, bar_p = bar_s + 16, bar_o = bar_p + 16;
  const uint32_t fix_go = bar_o + 16, fixed = fix_go + 8, drain = fixed + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  volatile int* info = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 16);  // [INFO][8]
  auto slot = [&](int j) { return base + C::OFF_KV + uint32_t(j % RING) * (2 * C::TILE); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_hp = HEADS ? g.heads >> 1 : g.heads;
  const int rank = SPLIT ? int(cluster_rank()) : 0, ranks = SPLIT ? int(cluster_size()) : 1;
  const int cta = int(blockIdx.x) / ranks, ctas = int(gridDim.x) / ranks;
  // this CTA's it-th entry of the list, back and forth over the CTAs
  auto unit_of = [&](int it) { return it * ctas + ((it & 1) ? ctas - 1 - cta : cta); };

  // (by value throughout: nothing of a role may live in local memory)
  // Two tiles of one head change places in every other entry, so that a run of
  // sequences of up to 128 queries, one tile each, serves both warpgroups
  // (4,096 of 64 tokens, 8 heads: 820 us, 1,026 on one warpgroup).
  auto plan = [&](Plan w, int it) {
    w.off0 = !HEADS && (it & 1) ? 128 : 0;
    w.off1 = HEADS ? 0 : 128 - w.off0;
    auto steps = [&](int r) {  // key tiles that a tile's last row sees
      if (r >= w.Lq) return 0;
      const int last = min(r + 128, w.Lq) - 1;
      const int lim = g.causal ? min(w.Lk, max(0, last + 1 + w.Lk - w.Lq)) : w.Lk;
      return (lim + 127) >> 7;
    };
    w.n0 = steps(w.first + w.off0);
    w.n1 = HEADS ? w.n0 : steps(w.first + w.off1);
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
    return w;
  };
  // The entry `it` as published by the finder; false at the list's end or
  // on an abort.  All lanes of the calling warp, or one thread alone (mask).
  // A wait may last as long as another tile's walk.
  constexpr uint64_t kLong = 20000000000ull;
  auto take = [&](int it, bool whole_warp) {
    const uint32_t b = uint32_t(it % C::INFO);
    Plan w{};
    bool got = mbar_wait(bar_info + 8 * b, (it / C::INFO) & 1, abort_flag, kLong);
    if (whole_warp) got = __all_sync(0xffffffffu, got);
    if (!got) {  // some role has given up, or does now
      report_timeout(abort_flag, io.status);
      return w;
    }
    const volatile int* e = info + 8 * b;
    w.any = e[0] != 0;
    w.q0 = e[1], w.Lq = e[2], w.k0 = e[3], w.Lk = e[4], w.first = e[5], w.hp = e[6];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(info_free + 8 * b);
    return w.any ? plan(w, it) : w;
  };

  if (warp == 10) {
    if (lane == 0) {
      for (int s = 0; s < RING; ++s) {
        mbar_init(full + 8 * s, 1);
        mbar_init(empty + 8 * s, 1);
      }
      for (int b = 0; b < C::INFO; ++b) {
        mbar_init(bar_info + 8 * b, 1);
        mbar_init(info_free + 8 * b, 11);  // every warp but the finder
      }
      for (int u = 0; u < 2; ++u) {
        mbar_init(bar_q + 8 * u, 1);
        mbar_init(q_free + 8 * u, 1);
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
  } else if (warp == 9) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  } else if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&mq);
    if (io.total_k > 0) {  // else there are no maps
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
  }
  // the first entry is found during the set-up
  Tile next{};
  int at = 0;  // its place in this CTA's share of the list
  auto find = [&] {
    for (; unit_of(at) < n_units; ++at) {
      const Tile t = find_tile<kWalkQ>(io.cu_q, io.total_q, io.cu_k, io.total_k, io.n_seqs,
                                       g.causal, HEADS ? 128 : 256, unit_of(at) / n_hp, lane,
                                       io.status);
      // only many sequences leave empty places in front of others
      if (SPLIT || t.any || io.n_seqs <= kListed) return t;
    }
    return Tile{};
  };
  if (warp == 11) next = find();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  bool ok = true;

  // a softmax thread's row of the entry, and the row's statistics
  const int u = (warp >> 2) & 1, quad = warp & 3;
  const uint32_t lane_base = uint32_t(quad * 32) << 16;
  const uint32_t tO = tmem + C::COL_O + 128u * u + lane_base;
  int nu = 0;
  float m = -INFINITY, l = 0.f;

  // The softmax threads hold a row of 128 scores and take the other warps'
  // registers: 256 * 200 + 128 * 104 = 384 * 168, those of the launch.
  if (warp == 8) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    int x = 0, nq0 = 0, nq1 = 0;  // stages and Q tiles so far (lane 0)
    auto kv_head = [&](const Plan& w) { return (HEADS ? 2 * w.hp : w.hp) / g.group; };
    // the next stage: V rows from vrow and K rows from krow on (none for < 0)
    auto load_stage = [&](int vrow, int vhead, int krow, int khead) {
      if (x >= RING && !mbar_wait(empty + 8 * (x % RING), ((x / RING) - 1) & 1, abort_flag))
        return false;
      const uint32_t bar = full + 8 * (x % RING);
      mbar_arrive_expect_tx(bar, ((vrow >= 0) + (krow >= 0)) * C::TILE);
      if (vrow >= 0) tma_load_rows(slot(x), &mv, bar, vrow, vhead);
      if (krow >= 0) tma_load_rows(slot(x) + C::TILE, &mk, bar, krow, khead);
      ++x;
      return true;
    };
    // a tile's Q once the previous entry's last scores have read theirs
    auto load_q = [&](const Plan& w, int t, int n, int& nq) {
      if (n == 0) return true;
      if (nq > 0 && !mbar_wait(q_free + 8 * t, (nq - 1) & 1, abort_flag, kLong)) return false;
      ++nq;
      mbar_arrive_expect_tx(bar_q + 8 * t, C::TILE);
      tma_load_rows(base + C::OFF_Q + t * C::TILE, &mq, bar_q + 8 * t,
                    w.q0 + w.first + (t ? w.off1 : w.off0), (HEADS ? 2 * w.hp + t : w.hp));
      return true;
    };
    Plan w = take(0, true);
    bool joined = false;  // K_0 came beside the previous entry's last V
    for (int it = 1; ok && w.any; ++it) {
      const bool walks = w.n > 0;
      const int head = kv_head(w);
      int row = w.k0 + w.kb * 128;  // K of the next step
      if (walks && lane == 0) {
        if (!joined) ok = load_stage(-1, 0, row, head);
        ok = ok && load_q(w, 0, w.n0, nq0) && load_q(w, 1, w.n1, nq1);
        for (int j = 1; ok && j < w.n; ++j) {
          row += 128;
          ok = load_stage(row - 128, head, row, head);
        }
      }
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      if (!ok) break;
      w = Plan{};
      if (!SPLIT) w = take(it, true);
      joined = walks && w.any && w.n > 0;
      if (walks && lane == 0)
        ok = load_stage(row, head, joined ? w.k0 + w.kb * 128 : -1, kv_head(w));
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
    }
    if (lane == 0) {
      if (!ok) report_timeout(abort_flag, io.status);
      // on an abort copies may still be landing: the newest into Q and each slot
      if (!ok || *abort_flag) {
        if (nq0 > 0) mbar_wait(bar_q, (nq0 - 1) & 1, nullptr, 200000000ull);
        if (nq1 > 0) mbar_wait(bar_q + 8, (nq1 - 1) & 1, nullptr, 200000000ull);
        for (int i = x > RING ? x - RING : 0; i < x; ++i)
          mbar_wait(full + 8 * (i % RING), (i / RING) & 1, nullptr, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f32<T>(128, 128, false);
      constexpr uint32_t id_o = idesc_f32<T>(128, D, true);
      int c = 0, nq0 = 0, nq1 = 0, tails = 0;  // c: the stage of an entry's K_0
      int done0 = 0, done1 = 0;  // steps of each tile so far
      auto wait_full = [&](int x) {
        return mbar_wait(full + 8 * (x % RING), (x / RING) & 1, abort_flag);
      };
      auto scores = [&](int t, int x) {  // S_t = Q_t K^T, K in stage x
        const uint32_t sq = base + C::OFF_Q + t * C::TILE, sk = slot(x) + C::TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + 128u * t, sdesc_sw128(sq + off, 16, 1024),
                    sdesc_sw128(sk + off, 16, 1024), id_s, kk > 0);
        }
        tc_commit(bar_s + 8 * t);
      };
      auto first_scores = [&](int t, int n, int& nq, int x) {  // of an entry
        if (n == 0) return true;
        if (!mbar_wait(bar_q + 8 * t, nq++ & 1, abort_flag)) return false;
        tc_fence_after();
        scores(t, x);
        if (n == 1) tc_commit(q_free + 8 * t);
        return true;
      };
      Plan w = take(0, false);
      bool joined = false;  // the first scores were issued with the previous entry's last step
      for (int it = 1; w.any;) {
        if (w.n == 0) {
          if (SPLIT) break;
          w = take(it++, false);
          continue;
        }
        const int n = w.n;
        const bool has_tail = (w.kb + n) * 128 > w.Lk;  // the walk ends in a partial key tile
        if (!joined) {
          ok = wait_full(c) && first_scores(0, w.n0, nq0, c) && first_scores(1, w.n1, nq1, c);
          if (!ok) break;
          tc_commit(empty + 8 * (c % RING));
        }
        // test hook: with `stall` set no PV is issued and the softmax's wait runs out
        if (io.stall) break;
        Plan nx{};
        for (int i = 0; i < n; ++i) {
          const bool last = i == n - 1;
          if (last && !SPLIT) nx = take(it++, false);
          joined = last && nx.any && nx.n > 0;
          ok = wait_full(c + i + 1);
          if (ok && has_tail && last) {
            mbar_arrive(fix_go);  // the tail rows of V are zeroed by warp 10
            ok = mbar_wait(fixed, tails & 1, abort_flag);
            ++tails;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? w.n1 : w.n0;
            if (ok && i < nt) {
              ok = mbar_wait(bar_p + 8 * t, (t ? done1 : done0)++ & 1, abort_flag);
              if (!ok) continue;
              tc_fence_after();
              const uint32_t sv = slot(c + i + 1);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_ts(tmem + C::COL_O + 128u * t, tmem + 128u * t + 8u * kk,
                          sdesc_sw128(sv + kk * 2048, C::BOX, 1024), id_o,
                          (i > 0 || kk > 0) ? 1u : 0u);
              if (i + 1 < nt) {
                scores(t, c + i + 1);
                if (i + 2 == nt) tc_commit(q_free + 8 * t);
              } else {
                tc_commit(bar_o + 8 * t);
              }
            }
            if (ok && joined) ok = first_scores(t, t ? nx.n1 : nx.n0, t ? nq1 : nq0, c + n);
          }
          if (!ok) break;
          tc_commit(empty + 8 * ((c + i + 1) % RING));
        }
        if (!ok) break;
        c += joined ? n : n + 1;
        w = nx;
      }
      if (!ok) report_timeout(abort_flag, io.status);
      // every MMA this thread issued has completed once the drain barrier flips
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ----------------------------------------------------------- V tails
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    int c = 0, tails = 0;
    Plan w = take(0, true);
    for (int it = 1; w.any; ++it) {
      Plan nx{};
      if (!SPLIT) nx = take(it, true);
      if (w.n > 0 && (w.kb + w.n) * 128 > w.Lk) {
        ok = __all_sync(0xffffffffu, mbar_wait(fix_go, tails & 1, abort_flag, kLong));
        if (!ok) break;
        ++tails;
        const uint32_t sv = slot(c + w.n);
        for (int bx = 0; bx < C::KB; ++bx)
          for (int o = (w.Lk & 127) * 128 + lane * 16; o < C::BOX; o += 512)
            st_shared_v4(sv + bx * C::BOX + o, make_uint4(0u, 0u, 0u, 0u));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed);
      }
      if (w.n > 0) c += nx.any && nx.n > 0 ? w.n : w.n + 1;
      w = nx;
    }
    if (!ok && lane == 0) report_timeout(abort_flag, io.status);
  } else if (warp == 11) {
    // ----------------------------------------------------------- entries
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    for (int it = 0;; ++it) {
      const uint32_t b = uint32_t(it % C::INFO);
      if (it >= C::INFO) {
        ok = __all_sync(0xffffffffu, mbar_wait(info_free + 8 * b, (it / C::INFO - 1) & 1,
                                               abort_flag, kLong));
        if (!ok) break;
      }
      if (lane == 0) {
        volatile int* e = info + 8 * b;
        e[0] = next.any, e[1] = next.a.start, e[2] = next.a.len, e[3] = next.b.start;
        e[4] = next.b.len, e[5] = next.tile * (HEADS ? 128 : 256), e[6] = unit_of(at) % n_hp;
        mbar_arrive(bar_info + 8 * b);
      }
      __syncwarp();
      if (SPLIT || !next.any) break;
      ++at;
      next = find();
    }
    if (!ok && lane == 0) report_timeout(abort_flag, io.status);
  } else {
    // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const uint32_t tS = tmem + 128u * u + lane_base;
    const float sl2 = g.scale * kLog2e;
    int done = 0, tiles = 0;  // steps and tiles with a walk so far
    for (int it = 0; !SPLIT || it < 1; ++it) {
      const Plan w = take(it, true);
      if (!w.any) break;
      nu = u ? w.n1 : w.n0;
      const int r = w.first + (u ? w.off1 : w.off0) + quad * 32 + lane;  // row within the sequence
      const bool exists = r < w.Lq;
      const int lim = !exists ? 0 : (g.causal ? min(w.Lk, max(0, r + 1 + w.Lk - w.Lq)) : w.Lk);
      m = -INFINITY;
      l = 0.f;
      for (int i = 0; i < nu; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s + 8 * u, (done + i) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        BSA_TMEM_LD128(tS, s);
        const int seen = lim - 128 * (w.kb + i);
        if (!__all_sync(0xffffffffu, !exists || seen >= 128)) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            if (x >= seen) s[x] = 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 128; x += 2)
          mx[(x >> 1) & 3] =
              max3f(mx[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
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
        for (int x = 0; x < 128; x += 2) {
          float x0, x1;
          fma_f32x2(x0, x1, __uint_as_float(s[x]), __uint_as_float(s[x + 1]), sl2, sl2, off, off);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const int a = (x >> 1) & 1;
          add_f32x2(sum[2 * a], sum[2 * a + 1], sum[2 * a], sum[2 * a + 1], p0, p1);
          s[x >> 1] = pack2<T>(p0, p1);
        }
        BSA_TMEM_ST64(tS, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 8 * u);
        l = l * factor + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
      }
      done += nu;
      if (ok && nu > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_o + 8 * u, tiles & 1, abort_flag));
        ++tiles;
      }
      if (!ok) break;
      tc_fence_after();
      if constexpr (!SPLIT) {
        // ------------------------------------------------------ epilogue
        const int head = HEADS ? 2 * w.hp + u : w.hp;
        // a NaN sum stays one; a row that saw nothing gives 0
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (exists && io.lse)
          io.lse[int64_t(head) * io.total_q + w.q0 + r] =
              l == 0.f ? -INFINITY : m - kShift + log2f(l);
        const uint32_t stage = base + C::OFF_STAGE + warp * C::STAGE;
        const int row0 = r - lane;  // the warp's first row
        T* dst = static_cast<T*>(io.o.p) + int64_t(w.q0 + row0) * io.o.sn + int64_t(head) * io.o.sh;
#pragma unroll 1
        for (int half = 0; half < D / 64; ++half) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t o[32];
            if (nu > 0) {  // else no product was issued
              BSA_TMEM_LD32(tO + 64u * half + 32u * ch, o);
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
              stage_chunk<64>(stage, lane, 4 * ch + j, make_uint4(v[0], v[1], v[2], v[3]));
            }
          }
          write_rows<T, 64>(stage, dst + 64 * half, io.o.sn, min(32, w.Lq - row0), lane);
        }
        // O has been read: the next entry's first PV may overwrite it once
        // this warp has handed in its P
        tc_fence_before();
      }
    }
    if (!ok && lane == 0) report_timeout(abort_flag, io.status);
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
    const bool live = info[0] != 0 && !*abort_flag;
    const int q0 = info[1], Lq = info[2], first = info[5], hp = info[6];
    if (live) {
      constexpr int CH = D / 8;
      for (int i = threadIdx.x; i < (256 / ranks) * CH; i += C::kThreads) {
        const int row = (i / CH) * ranks + rank, ch = i % CH;
        const int t = row >> 7, rr = first + (HEADS ? 0 : 128 * t) + (row & 127);
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
        const int head = HEADS ? 2 * hp + t : hp;
        if (io.lse && ch == 0)
          io.lse[int64_t(head) * io.total_q + q0 + rr] =
              ll == 0.f ? -INFINITY : mm - kShift + log2f(ll);
        uint4 v = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                             pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
        *reinterpret_cast<uint4*>(static_cast<T*>(io.o.p) + int64_t(q0 + rr) * io.o.sn +
                                  int64_t(head) * io.o.sh + ch * 8) = v;
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its rows are read
  }
  if (warp == 9) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <typename T, int D, bool HEADS, bool SPLIT>
cudaError_t launch_t(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io, int units,
                     int ranks, cudaStream_t st) {
  using C = FwdCfg<D>;
  auto kern = packed_fwd_kernel<T, D, HEADS, SPLIT>;
  // The register split waits for ever unless the launch brings 168 a thread:
  // the build checks that, and so does the first launch (an error of the query
  // itself is the call's and not kept).
  static std::atomic<bool> fits{false};
  cudaError_t e;
  if (!fits.load(std::memory_order_acquire)) {
    cudaFuncAttributes a{};
    e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    if (a.numRegs != 168) return cudaErrorInvalidConfiguration;
    fits.store(true, std::memory_order_release);
  }
  static std::atomic<uint64_t> seen{0};
  e = allow_smem(kern, C::SMEM, seen);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const int sms = device_sms();
  cfg.gridDim = dim3(unsigned(SPLIT ? units * ranks : (units < sms ? units : sms)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(ranks);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], g, io, units);
}

// CTAs that share a tile's keys, where a CTA per tile leaves half of the SMs
// idle.  Only the sums of the lengths are known here: a walk is taken to have
// total_k / 128 / n^0.6 key steps, between those of n equal sequences and the
// longest of unequal ones.  us with 1 | 2 | 4 | 8 CTAs a tile (bf16):
//   1 x 1,000 of 8/2 heads, 4 tiles:              20 |  14 |  11 |  11
//   384 x 5,000 of 8/2 heads, 12 tiles:           79 |  49 |  33 |  31
//   512 x 5,000 of 16 heads, 32 tiles:            80 |  50 |  37 |  83
//   600 x 1,200 of 16/8 heads, 40 tiles:          24 |  19 |  30 |  44
//   512 x 8,000 of 32/8 heads, 64 tiles:         111 |  63 |  75 | 128
//   8 x (250 x 250) of 4/2 heads:                 11 |  18 |  19 |  47
//   30 x (1 x 128) of 8/2 heads:                  10 |  20 |  36 |  72
//   16 x (1 x 4,000) of 8/2 heads:                60 |  35 |  43 |  71
//   256, 511, 64 x 5,000, 511, 2,113 of 16/2:     73 |  43 |  39 |  65
// So one wave of CTAs, and clusters of eight, of which few find room at a time,
// on half of the SMs.  Long walks of several sequences may take two waves of
// fours, and eights three quarters of the SMs: from 30 steps on 0.63 to 0.74
// of the time by twos where lengths differ, 1.16 to 1.22 where they are equal.
// Over 5,330 batches of 1 to 32 sequences, equal or log-uniform up to 20,000
// keys, this takes 1.09 times the best of the four sizes on average, 1.21 with
// the batch's keys in place of a walk's, 1.51 without clusters.
int split_ranks(const PackedIO& io, int64_t rows, int slots) {
  const int sms = device_sms();
  // the sequences' last tiles are half full on average
  const int64_t units = ((io.total_q + rows - 1) / rows + io.n_seqs / 2) * slots;
  if (2 * units > sms) return 1;
  const bool one = io.n_seqs == 1;
  const double steps = double(io.total_k) / 128 / (one ? 1. : std::pow(double(io.n_seqs), 0.6));
  if (8 * units <= sms / 2 ? steps >= 8 : 8 * units <= sms * 3 / 4 && steps >= (one ? 15 : 25))
    return 8;
  if (4 * units <= sms / 2 ? steps >= 3
                           : 4 * units <= (!one && steps >= 30 ? 2 * sms : sms) && steps >= 5)
    return 4;
  return steps >= 6 ? 2 : 1;
}

template <typename T, int D>
cudaError_t launch_d(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                     cudaStream_t st) {
  const bool heads = g.group % 2 == 0;
  const int64_t rows = heads ? 128 : 256;
  const int64_t tiles = tile_places(io.total_q, io.n_seqs, int(rows));
  const int units = int(tiles * (heads ? g.heads / 2 : g.heads));
  const int ranks = split_ranks(io, rows, heads ? g.heads / 2 : g.heads);
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
