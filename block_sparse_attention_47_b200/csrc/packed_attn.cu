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
// other tile, so neither waits for the other when a step's exponentials take
// as long as its products.  One thread issues all products of a tile in the
// order PV_i, S_(i+1): the pipe runs them in that order, so S_(i+1) may
// overwrite P_i's columns, and once S_(i+1) is signalled PV_i has finished
// and O may be rescaled.  O is rescaled only when the maximum has grown by
// more than 2^8.  A quarter of the exponentials runs on the FMA pipe.
//
// K and V come through one ring of 128-row TMA boxes of the packed tensors.
// The box of a sequence's last tile runs into its neighbour's rows (or into
// whatever lies behind the last sequence): such K columns are masked by a
// select, and those V rows are zeroed in shared memory before the product,
// since 0 times a NaN would reach the output.
//
// Tensor memory (512 columns): S_u/P_u at 128 u, O_u at 256 + 128 u.
// Every wait is bounded (2 s) and reports BSA_ERR_TIMEOUT.
#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct FwdCfg {
  // warps 0-3 / 4-7: softmax of tile 0 / 1; 8: copies; 9: products;
  // 10: the V tail; 11: finds the tile
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
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <typename T, int D, bool HEADS>
__global__ void __launch_bounds__(384, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, SeqGeo g, const PackedIO io) {
  using C = FwdCfg<D>;
  constexpr int RING = C::RING;
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
  const int hp = int(blockIdx.x % uint32_t(n_hp));

  if (warp == 11) {
    int b = 0, t = 0;
    const bool any = find_tile(io.cu_q, io.n_seqs, io.total_q, HEADS ? 128 : 256,
                               blockIdx.x / uint32_t(n_hp), lane, io.status, b, t);
    if (lane == 0) {
      found[0] = any;
      if (any) {
        const Span q = span_of(io.cu_q, b, io.total_q, io.status);
        const Span k = span_of(io.cu_k, b, io.total_k, io.status);
        found[1] = q.start;
        found[2] = q.len;
        found[3] = k.start;
        found[4] = k.len;
        found[5] = t;
      }
    }
  } else if (warp == 9) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  } else if (threadIdx.x == 0) {
    for (int s = 0; s < RING; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(bar_q, 1);
    for (int u = 0; u < 2; ++u) {
      mbar_init(bar_s + 8 * u, 1);
      mbar_init(bar_p + 8 * u, 128);
      mbar_init(bar_o + 8 * u, 1);
    }
    mbar_init(fix_go, 1);
    mbar_init(fixed, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool any = found[0] != 0;
  const int q0 = found[1], Lq = found[2], k0 = found[3], Lk = found[4];
  const int first = found[5] * (HEADS ? 128 : 256);  // first row of tile 0
  const int head0 = HEADS ? 2 * hp : hp;
  const int kvh = head0 / g.group;
  // steps of tile u: key tiles that its last row sees
  auto row_of = [&](int u) { return HEADS ? first : first + 128 * u; };
  auto steps_of = [&](int u) {
    const int r = row_of(u);
    if (!any || r >= Lq) return 0;
    const int last = min(r + 128, Lq) - 1;
    const int lim = g.causal ? min(Lk, max(0, last + 1 + Lk - Lq)) : Lk;
    return (lim + 127) >> 7;
  };
  const int n0 = steps_of(0), n1 = steps_of(1), n = max(n0, n1);
  const bool has_tail = n > 0 && n * 128 > Lk;  // the walk ends in a partial key tile

  if (warp == 8) {
    // ------------------------------------------------------------ copies
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
      const int tiles = (n0 > 0) + (n1 > 0);
      mbar_arrive_expect_tx(bar_q, tiles * C::TILE);
      for (int u = 0; u < 2; ++u)
        if ((u ? n1 : n0) > 0)
          for (int bx = 0; bx < C::KB; ++bx)
            tma_load_3d(base + C::OFF_Q + u * C::TILE + bx * C::BOX, &mq, bar_q, 64 * bx,
                        head0 + (HEADS ? u : 0), q0 + row_of(u));
      bool ok = true;
      int i = 0;
      for (; i < 2 * n; ++i) {
        if (i >= RING && !mbar_wait(empty + 8 * (i % RING), ((i / RING) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t bar = full + 8 * (i % RING);
        mbar_arrive_expect_tx(bar, C::TILE);
        for (int bx = 0; bx < C::KB; ++bx)
          tma_load_3d(slot(i) + bx * C::BOX, (i & 1) ? &mv : &mk, bar, 64 * bx, kvh,
                      k0 + (i >> 1) * 128);
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
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f32<T>(128, 128, false);
      constexpr uint32_t id_o = idesc_f32<T>(128, D, true);
      auto scores = [&](int u, int i) {  // S_u = Q_u K_i^T
        const uint32_t sq = base + C::OFF_Q + u * C::TILE, sk = slot(2 * i);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + 128u * u, sdesc_sw128(sq + off, 16, 1024),
                    sdesc_sw128(sk + off, 16, 1024), id_s, kk > 0);
        }
        tc_commit(bar_s + 8 * u);
      };
      bool ok = mbar_wait(bar_q, 0, abort_flag) && mbar_wait(full, 0, abort_flag);
      if (ok) {
        tc_fence_after();
        for (int u = 0; u < 2; ++u)
          if ((u ? n1 : n0) > 0) scores(u, 0);
        tc_commit(empty);
      }
      // test hook: with `stall` set no PV is issued and the softmax's wait runs out
      for (int i = 0; ok && i < n && !io.stall; ++i) {
        const int vi = 2 * i + 1, ki = 2 * i + 2;
        ok = mbar_wait(full + 8 * (vi % RING), (vi / RING) & 1, abort_flag) &&
             (i + 1 >= n || mbar_wait(full + 8 * (ki % RING), (ki / RING) & 1, abort_flag));
        if (ok && has_tail && i == n - 1) {
          mbar_arrive(fix_go);  // the tail rows of V are zeroed by warp 10
          ok = mbar_wait(fixed, 0, abort_flag);
        }
        for (int u = 0; ok && u < 2; ++u) {
          const int nu = u ? n1 : n0;
          if (i >= nu) continue;
          ok = mbar_wait(bar_p + 8 * u, i & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = slot(vi);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + C::COL_O + 128u * u, tmem + 128u * u + 8u * kk,
                      sdesc_sw128(sv + kk * 2048, C::BOX, 1024), id_o, (i > 0 || kk > 0) ? 1u : 0u);
          if (i + 1 < nu)
            scores(u, i + 1);
          else
            tc_commit(bar_o + 8 * u);
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
    if (has_tail) {
      // asked for at the walk's end: the limit grows with its length
      const bool ok = __all_sync(
          0xffffffffu, mbar_wait(fix_go, 0, abort_flag, 2000000000ull + uint64_t(n) * 10000ull));
      if (ok) {
        const uint32_t sv = slot(2 * n - 1);
        const int r0 = Lk - (n - 1) * 128;
        for (int bx = 0; bx < C::KB; ++bx)
          for (int o = r0 * 128 + lane * 16; o < C::BOX; o += 512)
            st_shared_v4(sv + bx * C::BOX + o, make_uint4(0u, 0u, 0u, 0u));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed);
      } else if (lane == 0) {
        report_timeout(abort_flag, io.status);
      }
    }
  } else if (warp < 8) {
    // ----------------------------------------------------------- softmax
    constexpr float kShift = std::is_same<T, __half>::value ? 6.f : 0.f;
    const int u = warp >> 2, quad = warp & 3;
    const int r = row_of(u) + quad * 32 + lane;  // row within the sequence
    const bool exists = any && r < Lq;
    const int lim = !exists ? 0 : (g.causal ? min(Lk, max(0, r + 1 + Lk - Lq)) : Lk);
    const int nu = u ? n1 : n0;
    const uint32_t lane_base = uint32_t(quad * 32) << 16;
    const uint32_t tS = tmem + 128u * u + lane_base, tO = tmem + C::COL_O + 128u * u + lane_base;
    const float sl2 = g.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < nu; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_s + 8 * u, i & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
      BSA_TMEM_LD128(tS, s);
      const int seen = lim - 128 * i;
      const bool whole = __all_sync(0xffffffffu, !exists || seen >= 128);
      if (!whole) {
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
      // P <= 2^8; fp16 shifts it up by 2^6 so that fewer small ones vanish
      const float off = (m == -INFINITY ? 0.f : -m) + kShift;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      if (whole) {
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          float x0, x1, p0, p1;
          fma_f32x2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl2, sl2, off, off);
          if (((c >> 1) & 3) == 3) {
            exp2_fma_x2(p0, p1, x0, x1);
          } else {
            p0 = ex2_approx(x0);
            p1 = ex2_approx(x1);
          }
          const int a = (c >> 1) & 1;
          add_f32x2(sum[2 * a], sum[2 * a + 1], sum[2 * a], sum[2 * a + 1], p0, p1);
          s[c >> 1] = pack2<T>(p0, p1);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(s[c]), sl2, off));
          const float p1 = ex2_approx(fmaf(__uint_as_float(s[c + 1]), sl2, off));
          sum[(c >> 1) & 3] += p0 + p1;
          s[c >> 1] = pack2<T>(p0, p1);
        }
      }
      l = l * factor + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
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
      BSA_TMEM_ST64(tS, s);
      tc_fence_before();
      mbar_arrive(bar_p + 8 * u);
    }
    // ---------------------------------------------------------- epilogue
    if (ok && nu > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar_o + 8 * u, 0, abort_flag));
    if (!ok) {
      if (lane == 0) report_timeout(abort_flag, io.status);
    } else {
      tc_fence_after();
      const int head = head0 + (HEADS ? u : 0);
      // a NaN sum stays one; a row that saw nothing gives 0
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* orow = static_cast<T*>(io.o.p) + int64_t(q0 + r) * io.o.sn + int64_t(head) * io.o.sh;
      if (exists && io.lse)
        io.lse[int64_t(head) * io.total_q + q0 + r] = l == 0.f ? -INFINITY : m - kShift + log2f(l);
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        if (nu > 0) {  // else no product was issued
          BSA_TMEM_LD32(tO + 32u * ch, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (exists) {
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * ch);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = pack2<T>(__uint_as_float(o[8 * j + 2 * x]) * inv,
                              __uint_as_float(o[8 * j + 2 * x + 1]) * inv);
            dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <typename T, int D, bool HEADS>
cudaError_t launch_t(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                     cudaStream_t st) {
  using C = FwdCfg<D>;
  auto kern = packed_fwd_kernel<T, D, HEADS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // no more tiles than this whatever the lengths; the ones too many return
  const int64_t rows = HEADS ? 128 : 256;
  const int64_t tiles = io.total_q / rows + (io.n_seqs < io.total_q ? io.n_seqs : io.total_q);
  const int64_t ctas = tiles * (HEADS ? g.heads / 2 : g.heads);
  kern<<<unsigned(ctas), C::kThreads, C::SMEM, st>>>(maps[0], maps[1], maps[2], g, io);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                     cudaStream_t st) {
  const bool heads = g.group % 2 == 0;
  if (g.d == 128)
    return heads ? launch_t<T, 128, true>(g, maps, io, st) : launch_t<T, 128, false>(g, maps, io, st);
  return heads ? launch_t<T, 64, true>(g, maps, io, st) : launch_t<T, 64, false>(g, maps, io, st);
}

}  // namespace

cudaError_t launch_packed_fwd(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                              cudaStream_t st) {
  return g.fp16 ? launch_d<__half>(g, maps, io, st) : launch_d<__nv_bfloat16>(g, maps, io, st);
}

}  // namespace bsa
