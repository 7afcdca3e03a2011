// Backward of the packed-sequence attention on sm_100a.  With P recomputed
// from the forward's row statistics, P = exp2(s scale log2(e) - lse2), and
// D = rowsum(dO * O):
//     dP = dO V^T,  dS = P * (dP - D),
//     dQ = scale dS K,  dK = scale sum_h dS_h^T Q_h,  dV = sum_h P_h^T dO_h,
// the sums over the query heads h of a kv head.
//
// Bound by the tensor cores: 10 d flops per (query head, seen pair), 14 with
// the scores and dP formed in both kernels, 18 where dQ forms them twice (see
// D below).  Two kernels rather than one with
// atomic dQ sums, so that gradients do not vary from run to run:
//   dQ     CTA = 128 query rows of a head, walking the key tiles they see.
//   dK/dV  CTA = 128 keys of a kv head, walking the query tiles that see them
//          of every head of the group, so shared heads are summed in the
//          accumulators.  Where there are few such tiles a cluster of CTAs
//          shares a tile's steps and adds its sums up in rank order.
// Per step the two score-like products are one N=128 burst each, two row
// groups of 128 threads take 64 of the 128 columns each, and the results
// return to tensor memory as A operands of the accumulations.  In dK/dV two
// 128-column regions change roles from step to step: S^T in one, dP^T in the
// other; P^T and dS^T go over S^T, so the next S^T can follow into dP^T's
// region as soon as the groups have read it, under their remaining work.  A
// batch of 4,096, 2,048, 1,111 and 300 tokens, 24/8 heads, d = 128: dK/dV 261 us
// (3,340 cycles a step, 2,048 of them products), dQ 223 us (2,200 a step, 1,536
// of them products).
//
// Preparation: lse2 and D are written per 128-row tile of a sequence (rows
// behind its end get lse2 = +inf, D = 0, so that P = 0 there), sequence b at
// row 128 (cu[b] / 128 + b), which keeps tiles apart and 512-byte aligned for
// bulk copies.
//
// D.  rowsum(dO * O) from the 16-bit O is off by half a step of O, and where a
// row sees few keys dP - D nearly cancels: dQ and dK came out up to four times
// less exact than their rounding.  dQ therefore takes query tiles of up to
// kExactSteps key steps twice: a first sweep sums D = sum_j P_ij dP_ij in
// fp32 (no accumulation), and the corrected D also serves dK/dV.  Longer rows
// average that error out and keep rowsum(dO * O).
//
// Tiles that run into a neighbour's rows: as the B operand of an accumulation
// (K in dQ; Q and dO in dK/dV) their foreign rows are zeroed in shared
// memory, since 0 times a NaN would reach the sums; as rows of the CTA's own
// tile they only reach results that are not stored.
//
// fp16.  P and dS enter the accumulations as 16-bit values.  P <= 1 is scaled
// by 2^13.  dS is scaled by the power of two that puts its largest possible
// value, 2 max_i |dO_i| max_j |V_j| (2-norms over the sequence's rows of a kv
// head), at 2^15, so that it does not overflow, and loses bits only below
// 2^-29 of that value, whatever the scale of the loss and of the sequences
// beside it.  bf16 needs neither.
#include "seq_internal.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 13.f;
// 128-key steps up to which D is summed from P and dP.  Relative errors of dQ
// over that of rounding an exact result, bf16, at 5, 128, 1,500 and 4,000
// causal tokens: none 2.41, 1.71, 1.59, 1.55; 8 steps 1.33, 1.41, 1.45, 1.47;
// all 1.33, 1.41, 1.44, 1.43.  Forward and backward of 7,555 tokens x 24
// heads: 633, 660 and 769 us.
constexpr int kExactSteps = 8;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// rows of the padded statistics, and where sequence b's begin
__host__ __device__ inline int64_t stat_rows(int64_t total_q, int64_t n_seqs) {
  return 128 * (total_q / 128 + n_seqs + 1);
}
__device__ __forceinline__ int64_t stat_start(int cu, int b) {
  return 128 * (int64_t(cu >> 7) + b);
}

// 128-key steps of a query tile whose last row is `last`
__device__ __forceinline__ int key_steps(bool causal, int last, int lq, int lk) {
  return ((causal ? min(lk, max(0, last + 1 + lk - lq)) : lk) + 127) >> 7;
}

// fp16: where a sequence's largest squared norms stand, of dO rows and, behind
// them, of V rows: kv_heads each
__device__ __forceinline__ int64_t norms_at(int seq, int kvh, int kv_heads) {
  return 2 * int64_t(seq) * kv_heads + kvh;
}

// the power of two of dS for one sequence and kv head (fp16)
__device__ __forceinline__ float ds_factor(const float* __restrict__ norms, int seq, int kvh,
                                           int kv_heads) {
  const float* at = norms + norms_at(seq, kvh, kv_heads);
  const float bound = 2.f * sqrtf(__ldcg(at)) * sqrtf(__ldcg(at + kv_heads));
  if (!(bound > 0.f) || isinf(bound)) return 1.f;
  return exp2f(fminf(fmaxf(floorf(15.f - log2f(bound)), -60.f), 60.f));
}

// zero the rows from r0 on of a 128-row tile of KB boxes (a whole warp)
__device__ __forceinline__ void zero_rows(uint32_t tile, int boxes, int r0, int lane) {
  for (int bx = 0; bx < boxes; ++bx)
    for (int o = r0 * 128 + lane * 16; o < 128 * 128; o += 512)
      st_shared_v4(tile + bx * 128 * 128 + o, make_uint4(0u, 0u, 0u, 0u));
}

// 64 columns of an accumulator, scaled, to 64 channels of a warp's 32 rows;
// `stage`: 4 KB of the warp's own.  live = false writes zeros.
template <typename T>
__device__ __forceinline__ void write_channels(uint32_t stage, uint32_t tcol, T* dst,
                                               int64_t stride, int n_rows, float f, bool live,
                                               int lane) {
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t a[32];
    BSA_TMEM_LD32(tcol + 32u * ch, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = live ? pack2<T>(__uint_as_float(a[8 * i + 2 * x]) * f,
                               __uint_as_float(a[8 * i + 2 * x + 1]) * f)
                    : 0u;
      stage_chunk<64>(stage, lane, 4 * ch + i, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  write_rows<T, 64>(stage, dst, stride, n_rows, lane);
}

// ============================================================================
// D = rowsum(dO * O), the statistics' layout, and the norms for fp16
// ============================================================================
template <typename T, int D>
__global__ void __launch_bounds__(256) bwd_prepare_kernel(SeqGeo g, const PackedBwdIO io,
                                                          int tiles) {
  cudaTriggerProgrammaticLaunchCompletion();  // dQ may set itself up
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int TPR = D / 8;  // threads per row, 16 bytes each
  __shared__ int where[6];    // any, sequence, tile, first row, length, length of the others
  __shared__ float top[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // fp16: the blocks behind the tiles' look at V, a key tile and kv head each
  const bool of_v = kHalf && int(blockIdx.x) >= tiles;
  int64_t tile = blockIdx.x;
  int head = blockIdx.y;
  if (of_v) {
    const int64_t i = (tile - tiles) * gridDim.y + blockIdx.y;
    tile = i / g.kv_heads;
    head = int(i - tile * g.kv_heads);
  }
  if (warp == 0) {
    const Tile f = find_tile<kWalkQ>(of_v ? io.cu_k : io.cu_q, of_v ? io.total_k : io.total_q,
                                     of_v ? io.cu_q : io.cu_k, of_v ? io.total_q : io.total_k,
                                     io.n_seqs, g.causal, 128, tile, lane, io.status);
    if (lane == 0)
      where[0] = f.any, where[1] = f.seq, where[2] = f.tile, where[3] = f.a.start,
      where[4] = f.a.len, where[5] = f.b.len;
  }
  __syncthreads();
  if (!where[0]) return;
  const int b = where[1], t = where[2];
  const Span q{where[3], where[4]};  // of V: the keys
  // D of tiles of few key steps comes from dQ: there O and (but for its norms
  // in fp16) dO need not be read
  const bool summed =
      !kHalf &&
      key_steps(g.causal, min(t * 128 + 128, q.len) - 1, q.len, where[5]) <= kExactSteps;
  const Rows z_rows = of_v ? io.v : io.dout;
  const int64_t stats = stat_rows(io.total_q, io.n_seqs);
  const int64_t out0 = int64_t(head) * stats + stat_start(q.start, b) + int64_t(t) * 128;
  float most = 0.f;
#pragma unroll 4
  for (int r = threadIdx.x / TPR; r < 128; r += 256 / TPR) {
    const int row = t * 128 + r;
    float acc = 0.f, sq = 0.f;
    if (row < q.len && !summed) {
      const int64_t at = q.start + row;
      const int c = (threadIdx.x % TPR) * 8;
      uint4 a = make_uint4(0u, 0u, 0u, 0u);
      if (!of_v)
        a = *reinterpret_cast<const uint4*>(static_cast<const T*>(io.o.p) + at * io.o.sn +
                                            int64_t(head) * io.o.sh + c);
      const uint4 z = *reinterpret_cast<const uint4*>(static_cast<const T*>(z_rows.p) +
                                                      at * z_rows.sn + int64_t(head) * z_rows.sh + c);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = unpack2<T>(av[i]), y = unpack2<T>(zv[i]);
        acc = fmaf(x.x, y.x, acc);
        acc = fmaf(x.y, y.y, acc);
        sq = fmaf(y.x, y.x, sq);
        sq = fmaf(y.y, y.y, sq);
      }
    }
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {
      acc += __shfl_xor_sync(0xffffffffu, acc, o);
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
    }
    most = fmaxf(most, sq);
    if (threadIdx.x % TPR == 0 && !of_v) {
      float lse = INFINITY;
      if (row < q.len) {
        lse = __ldg(io.lse + int64_t(head) * io.total_q + q.start + row);
        if (lse == -INFINITY) lse = INFINITY;  // the row saw nothing: P = 0
      }
      io.stat_lse[out0 + r] = lse;
      io.stat_delta[out0 + r] = row < q.len ? acc : 0.f;
    }
  }
  if constexpr (kHalf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) top[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 8; ++w) most = fmaxf(most, top[w]);
      // non-negative floats order as their bits; a maximum has no order of arrival
      float* to = io.norms + (of_v ? norms_at(b, head, g.kv_heads) + g.kv_heads
                                   : norms_at(b, head / g.group, g.kv_heads));
      atomicMax(reinterpret_cast<int*>(to), __float_as_int(most));
    }
  }
}

// ============================================================================
// dQ: CTA = 128 query rows of a head
// ============================================================================
template <int D>
struct DqCfg {
  // warps 0-3 / 4-7: row groups 0 / 1 (64 key columns of a step each);
  // 8: S/dP issuer; 9: finds the tile, copies; 10: accumulations; 11: the K tail
  static constexpr int kThreads = 384;
  static constexpr int KB = D / 64;
  static constexpr int NK = 3, NV = 2;       // K / V ring slots
  static constexpr int BOX = 128 * 128;
  static constexpr int TILE = KB * BOX;      // 128 rows
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_BAR = OFF_V + NV * TILE;
  // kfull[NK] kempty[NK] vfull[NV] vempty[NV] sd_ready read x_ready
  // x_free own q do fix_go fixed sums done drain[2] s_ready[2] s_read[2]
  static constexpr int N_BARS = 2 * NK + 2 * NV + 17;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int OFF_SUM = OFF_MISC + 64;  // float [group][128]: D of the two halves
  static constexpr int SMEM = OFF_SUM + 1024 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  // dO (A of dP) at 0, S at 64 (group w's half at 64 + 64 w), dP at 192, dS
  // at 320 (32 packed columns per group), dQ at 384
  static constexpr uint32_t COL_DO = 0, COL_S = 64, COL_DP = 192, COL_DS = 320, COL_ACC = 384;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <typename T, int D>
__global__ void __launch_bounds__(384, 1)
    packed_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv,
                     const __grid_constant__ CUtensorMap mdo, SeqGeo g, const PackedBwdIO io) {
  using C = DqCfg<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int NK = C::NK, NV = C::NV;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (base - raw);
  const uint32_t sQ = base + C::OFF_Q;
  const uint32_t kfull = base + C::OFF_BAR, kempty = kfull + 8 * NK;
  const uint32_t vfull = kempty + 8 * NK, vempty = vfull + 8 * NV;
  const uint32_t sd_ready = vempty + 8 * NV, read = sd_ready + 8, x_ready = read + 8;
  const uint32_t x_free = x_ready + 8, own = x_free + 8, bar_q = own + 8;
  const uint32_t bar_do = bar_q + 8, fix_go = bar_do + 8, fixed = fix_go + 8, sums = fixed + 8;
  const uint32_t done = sums + 8, drain = done + 8, s_ready = drain + 16, s_read = s_ready + 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  int* found = reinterpret_cast<int*>(sm + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = int(blockIdx.x % uint32_t(g.heads)), kvh = head / g.group;
  cudaTriggerProgrammaticLaunchCompletion();  // see the launch of dK/dV
  auto kslot = [&](int p) { return base + C::OFF_K + (p % NK) * C::TILE; };
  auto vslot = [&](int p) { return base + C::OFF_V + (p % NV) * C::TILE; };

  int q0 = 0, Lq = 0, k0 = 0, Lk = 0, first = 0, seq = 0, np = 0;
  bool any = false;
  auto plan = [&] {  // np: key tiles that the tile's last row sees
    np = any ? key_steps(g.causal, min(first + 128, Lq) - 1, Lq, Lk) : 0;
  };
  if (warp == 10) {
    if (lane == 0) {
      for (int s = 0; s < NK; ++s) {
        mbar_init(kfull + 8 * s, 1);
        mbar_init(kempty + 8 * s, 1);
      }
      for (int s = 0; s < NV; ++s) {
        mbar_init(vfull + 8 * s, 1);
        mbar_init(vempty + 8 * s, 1);
      }
      mbar_init(sd_ready, 1);
      mbar_init(read, 8);
      mbar_init(x_ready, 8);
      mbar_init(x_free, 1);
      mbar_init(own, 4);
      mbar_init(bar_q, 1);
      mbar_init(bar_do, 1);
      mbar_init(fix_go, 1);
      mbar_init(fixed, 1);
      mbar_init(sums, 8);
      mbar_init(done, 2);
      mbar_init(drain, 1);
      mbar_init(drain + 8, 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_ready + 8 * b, 1);
        mbar_init(s_read + 8 * b, 8);
      }
      *abort_flag = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    named_bar_sync(1, 64);
  } else if (warp == 8) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  } else if (warp == 11 && lane == 0 && io.total_q > 0 && io.total_k > 0) {  // else no maps
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mdo);
  } else if (warp == 9) {
    const Tile t = find_tile<kWalkQ>(io.cu_q, io.total_q, io.cu_k, io.total_k, io.n_seqs, g.causal,
                                     128, blockIdx.x / uint32_t(g.heads), lane, io.status);
    any = t.any, q0 = t.a.start, Lq = t.a.len, k0 = t.b.start, Lk = t.b.len;
    first = t.tile * 128, seq = t.seq;
    if (lane == 0) {
      found[0] = any, found[1] = q0, found[2] = Lq, found[3] = k0, found[4] = Lk;
      found[5] = first, found[6] = seq;
    }
    plan();
    named_bar_sync(1, 64);  // the barriers are set up
    // the first copies start before the rest of the set-up; dO passes through
    // the third K slot on its way to tensor memory
    if (lane == 0 && np > 0) {
      mbar_arrive_expect_tx(bar_do, C::TILE);
      tma_load_rows(kslot(2), &mdo, bar_do, q0 + first, head);
      mbar_arrive_expect_tx(bar_q, C::TILE);
      tma_load_rows(sQ, &mq, bar_q, q0 + first, head);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (warp != 9) {
    any = found[0] != 0;
    q0 = found[1], Lq = found[2], k0 = found[3], Lk = found[4], first = found[5], seq = found[6];
    plan();
  }
  const bool has_tail = np > 0 && np * 128 > Lk;
  // steps: a first sweep for D, then the one that accumulates (a single step
  // stays in tensor memory for the second)
  const bool exact = np > 0 && np <= kExactSteps;
  const int lead = exact && np > 1 ? np : 0, nt = lead + np;

  if (warp == 9) {
    // ---- the copies: K and V tiles into their rings
    if (lane == 0 && np > 0) {
      bool ok = true;
      int kl = 0, vl = 0;  // tiles whose K / V copies have been issued
      for (int p = 0; p < nt; ++p) {
        const int row = k0 + (p < lead ? p : p - lead) * 128;
        // (the third K slot is free once dO has been taken out of it)
        if ((p >= NK && !mbar_wait(kempty + 8 * (p % NK), ((p - NK) / NK) & 1, abort_flag)) ||
            (p == 2 && !mbar_wait(own, 0, abort_flag))) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(kfull + 8 * (p % NK), C::TILE);
        tma_load_rows(kslot(p), &mk, kfull + 8 * (p % NK), row, kvh);
        kl = p + 1;
        if (p >= NV && !mbar_wait(vempty + 8 * (p % NV), ((p - NV) / NV) & 1, abort_flag)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(vfull + 8 * (p % NV), C::TILE);
        tma_load_rows(vslot(p), &mv, vfull + 8 * (p % NV), row, kvh);
        vl = p + 1;
      }
      if (!ok) report_timeout(abort_flag, io.status);
      if (!ok || *abort_flag) {
        // the newest copies may still be landing
        mbar_wait(bar_q, 0, nullptr, 200000000ull);
        mbar_wait(bar_do, 0, nullptr, 200000000ull);
        for (int p = kl > NK ? kl - NK : 0; p < kl; ++p)
          mbar_wait(kfull + 8 * (p % NK), (p / NK) & 1, nullptr, 200000000ull);
        for (int p = vl > NV ? vl - NV : 0; p < vl; ++p)
          mbar_wait(vfull + 8 * (p % NV), (p / NV) & 1, nullptr, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---- the last tile's foreign K rows, once it has landed
    if (has_tail) {
      if (__all_sync(0xffffffffu, mbar_wait(fix_go, 0, abort_flag,
                                            2000000000ull + uint64_t(nt) * 10000ull))) {
        zero_rows(kslot(nt - 1), C::KB, Lk - (np - 1) * 128, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed);
      } else if (lane == 0) {
        report_timeout(abort_flag, io.status);
      }
    }
  } else if (warp == 8) {
    // ---- S and dP of each step, once its tiles are in and both groups have
    // read the previous step's
    if (lane == 0 && np > 0) {
      constexpr uint32_t idesc_s = idesc_f32<T>(128, 128, false);
      bool ok = mbar_wait(own, 0, abort_flag) && mbar_wait(bar_q, 0, abort_flag);
      // the first sweep's S alternate between their columns and the idle sum's,
      // so that P is formed under the next products (2,500 cycles a step with
      // S and dP handed over together)
      for (int p = 0; ok && p < lead; ++p) {
        ok = mbar_wait(kfull + 8 * (p % NK), (p / NK) & 1, abort_flag) &&
             (p < 2 || mbar_wait(s_read + 8 * (p & 1), ((p >> 1) - 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + (p & 1 ? C::COL_ACC : C::COL_S), sdesc_sw128(sQ + off, 16, 1024),
                    sdesc_sw128(kslot(p) + off, 16, 1024), idesc_s, kk > 0);
        }
        tc_commit(s_ready + 8 * (p & 1));
        tc_commit(kempty + 8 * (p % NK));  // no accumulation reads it
        ok = mbar_wait(vfull + 8 * (p % NV), (p / NV) & 1, abort_flag) &&
             (p == 0 || mbar_wait(read, (p - 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ts(tmem + C::COL_DP, tmem + C::COL_DO + 8u * kk,
                    sdesc_sw128(vslot(p) + (kk / 4) * C::BOX + (kk % 4) * 32, 16, 1024), idesc_s,
                    kk > 0);
        tc_commit(sd_ready);
        tc_commit(vempty + 8 * (p % NV));
      }
      for (int p = lead; ok && p < nt; ++p) {
        if (!mbar_wait(kfull + 8 * (p % NK), (p / NK) & 1, abort_flag) ||
            !mbar_wait(vfull + 8 * (p % NV), (p / NV) & 1, abort_flag) ||
            (p > 0 && !mbar_wait(read, (p - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (has_tail && p == nt - 1) {
          mbar_arrive(fix_go);
          if (!mbar_wait(fixed, 0, abort_flag)) {
            ok = false;
            break;
          }
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + C::COL_S, sdesc_sw128(sQ + off, 16, 1024),
                    sdesc_sw128(kslot(p) + off, 16, 1024), idesc_s, kk > 0);
          tc_mma_ts(tmem + C::COL_DP, tmem + C::COL_DO + 8u * kk,
                    sdesc_sw128(vslot(p) + off, 16, 1024), idesc_s, kk > 0);
        }
        tc_commit(sd_ready);
        tc_commit(vempty + 8 * (p % NV));
      }
      if (!ok) report_timeout(abort_flag, io.status);
      tc_commit(done);
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---- dQ += dS K once both groups' dS is in; B = K, N-major
    if (lane == 0 && np > 0) {
      constexpr uint32_t idesc_acc = idesc_f32<T>(128, D, true);
      bool ok = true;
      // test hook: with `stall` set no accumulation is issued (the timeout path)
      for (int p = lead; ok && p < nt && !io.stall; ++p) {
        ok = mbar_wait(x_ready, (p - lead) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts(tmem + C::COL_ACC, tmem + C::COL_DS + 8u * kk,
                    sdesc_sw128(kslot(p) + kk * 2048, C::BOX, 1024), idesc_acc,
                    (p > lead || kk > 0) ? 1u : 0u);
        tc_commit(x_free);
        tc_commit(kempty + 8 * (p % NK));
      }
      if (!ok) report_timeout(abort_flag, io.status);
      tc_commit(done);
      tc_commit(drain + 8);
      mbar_wait(drain + 8, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else {
    // ---- row groups: group grp takes key columns 64 grp .. of every step;
    // thread r of a group owns query row r = TMEM lane r
    const int grp = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane, r = first + row;
    const uint32_t lane_base = uint32_t(quad * 32) << 16;
    const bool exists = any && r < Lq;
    const int lim = !exists ? 0 : (g.causal ? min(Lk, max(0, r + 1 + Lk - Lq)) : Lk);
    bool ok = true;
    if (grp == 1 && np > 0) {
      // dO rows into tensor memory: the A operand of dP (rows behind the end
      // are foreign and only reach rows that are not stored)
      ok = __all_sync(0xffffffffu, mbar_wait(bar_do, 0, abort_flag));
      uint32_t rw[D / 2];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float4 x = ld_shared_f4(kslot(2) + (i >> 3) * C::BOX + row * 128 +
                                      (((i & 7) ^ (row & 7)) << 4));
        rw[4 * i] = __float_as_uint(x.x);
        rw[4 * i + 1] = __float_as_uint(x.y);
        rw[4 * i + 2] = __float_as_uint(x.z);
        rw[4 * i + 3] = __float_as_uint(x.w);
      }
      if constexpr (D == 128) {
        BSA_TMEM_ST64(tmem + C::COL_DO + lane_base, rw);
      } else {
        BSA_TMEM_ST32(tmem + C::COL_DO + lane_base, rw);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(own);
    }
    float lse2 = INFINITY, dlt = 0.f, fac = 1.f;
    cudaGridDependencySynchronize();  // the preparation has finished
    if (exists && np > 0) {
      const int64_t at = int64_t(head) * stat_rows(io.total_q, io.n_seqs) + stat_start(q0, seq) + r;
      lse2 = __ldcg(io.stat_lse + at);
      dlt = __ldcg(io.stat_delta + at);
      if constexpr (kHalf) fac = ds_factor(io.norms, seq, kvh, g.kv_heads);
    }
    const float sl2 = g.scale * kLog2e;
    const uint32_t tS = tmem + C::COL_S + 64u * grp + lane_base;
    const uint32_t tDP = tmem + C::COL_DP + 64u * grp + lane_base;
    const uint32_t tDS = tmem + C::COL_DS + 32u * grp + lane_base;
    if (exact) {
      // ---- D = sum_j P_ij dP_ij over this group's columns, then both groups'
      float part = 0.f;
      for (int p = 0; ok && p < np; ++p) {
        // (a single step's S and dP come together and are read again)
        ok = __all_sync(0xffffffffu, lead ? mbar_wait(s_ready + 8 * (p & 1), (p >> 1) & 1, abort_flag)
                                          : mbar_wait(sd_ready, 0, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int seen = lim - 128 * p - 64 * grp;
        uint32_t sv[64];
        BSA_TMEM_LD64((p & 1 ? tmem + C::COL_ACC + 64u * grp + lane_base : tS), sv);
        if (lead) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_read + 8 * (p & 1));
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float x0, x1;
          fma_f32x2(x0, x1, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), sl2, sl2, -lse2,
                    -lse2);
          sv[c] = __float_as_uint(ex2_approx(x0));
          sv[c + 1] = __float_as_uint(ex2_approx(x1));
        }
        if (lead) ok = __all_sync(0xffffffffu, mbar_wait(sd_ready, p & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[64];
        BSA_TMEM_LD64(tDP, dp);
        if (lead) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(read);
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          // masked columns may hold anything
          const float x = fmaf(__uint_as_float(sv[c]), __uint_as_float(dp[c]), acc[c & 3]);
          acc[c & 3] = c < seen ? x : acc[c & 3];
        }
        part += (acc[0] + acc[1]) + (acc[2] + acc[3]);
      }
      volatile float* buf = reinterpret_cast<volatile float*>(sm + C::OFF_SUM);
      buf[128 * grp + row] = part;
      __syncwarp();
      if (lane == 0) mbar_arrive(sums);
      ok = ok && __all_sync(0xffffffffu, mbar_wait(sums, 0, abort_flag));
      dlt = buf[row] + buf[128 + row];
      if (ok && grp == 0 && exists)
        io.stat_delta[int64_t(head) * stat_rows(io.total_q, io.n_seqs) + stat_start(q0, seq) + r] =
            dlt;
    }
    const float dlt_f = dlt * fac;
    for (int p = 0; ok && p < np; ++p) {
      ok = __all_sync(0xffffffffu, mbar_wait(sd_ready, (lead + p) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[64], dp[64];
      BSA_TMEM_LD64(tS, sv);
      BSA_TMEM_LD64(tDP, dp);
      // S and dP read: the issuer may start the next step's
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(read);
      const int seen = lim - 128 * p - 64 * grp;
      uint32_t pk[32];
      if (__all_sync(0xffffffffu, !exists || seen >= 64)) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float x0, x1, t0, t1, d0, d1;
          fma_f32x2(x0, x1, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), sl2, sl2, -lse2,
                    -lse2);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          if constexpr (kHalf)
            fma_f32x2(t0, t1, __uint_as_float(dp[c]), __uint_as_float(dp[c + 1]), fac, fac, -dlt_f,
                      -dlt_f);
          else
            add_f32x2(t0, t1, __uint_as_float(dp[c]), __uint_as_float(dp[c + 1]), -dlt, -dlt);
          fma_f32x2(d0, d1, p0, p1, t0, t1, 0.f, 0.f);
          pk[c / 2] = pack2<T>(d0, d1);
        }
      } else {
        // masked scores and dP may be anything: both are selected away
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(sv[c]), sl2, -lse2));
          const float p1 = ex2_approx(fmaf(__uint_as_float(sv[c + 1]), sl2, -lse2));
          const float t0 = fmaf(__uint_as_float(dp[c]), fac, -dlt_f);
          const float t1 = fmaf(__uint_as_float(dp[c + 1]), fac, -dlt_f);
          pk[c / 2] = pack2<T>(c < seen ? p0 * t0 : 0.f, c + 1 < seen ? p1 * t1 : 0.f);
        }
      }
      // the group's columns are free once the previous accumulation has read them
      if (p > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(x_free, (p - 1) & 1, abort_flag));
        if (!ok) break;
      }
      tc_fence_after();
      BSA_TMEM_ST32(tDS, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_ready);
    }
    if (ok && np > 0) ok = __all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag));
    if (!ok) {
      if (lane == 0) report_timeout(abort_flag, io.status);
    } else {
      // group grp writes channels 64 grp ..; no step: the gradient is 0
      tc_fence_after();
      if (any && 64 * grp < D) {
        const int row0 = first + quad * 32;  // the warp's first row
        write_channels<T>(sQ + warp * 4096, tmem + C::COL_ACC + 64u * grp + lane_base,
                          static_cast<T*>(io.dq.p) + int64_t(q0 + row0) * io.dq.sn +
                              int64_t(head) * io.dq.sh + 64 * grp,
                          io.dq.sn, min(32, Lq - row0), g.scale / fac, np > 0, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ============================================================================
// dK, dV: CTA = 128 keys of a kv head
// ============================================================================
template <int D>
struct DkdvCfg {
  // warps 0-3 / 4-7: row groups 0 / 1 (64 query columns of a step each);
  // 8: S^T/dP^T issuer; 9: finds the tile, copies; 10: accumulations; 11: the
  // Q/dO tails
  static constexpr int kThreads = 384;
  static constexpr int KB = D / 64;
  static constexpr int NR = 2;                 // Q/dO ring slots
  static constexpr int BOX = 128 * 128;
  static constexpr int TILE = KB * BOX;
  static constexpr int OFF_K = 0, OFF_V = TILE;
  static constexpr int OFF_STG = 2 * TILE;     // [slot][Q | dO]
  static constexpr int OFF_VEC = OFF_STG + NR * 2 * TILE;  // [slot][lse2 128 | D 128] fp32
  static constexpr int OFF_BAR = OFF_VEC + NR * 1024;
  // full[NR] s_ready dp_ready dp_read st_issued p_ready[2] ds_ready x_free own
  // fix_go fixed done drain[2].  p_ready has a barrier per region: P^T of step
  // p+1 may be in before the thread of the sums has looked for step p's.
  static constexpr int N_BARS = NR + 14;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  // step p: S^T at 128 (p & 1) (group w's half at + 64 w; P^T over its first
  // 32 columns, dS^T over its last), dP^T in the other region; dV at 256, dK
  // at 256 + D
  static constexpr uint32_t COL_DV = 256, COL_DK = 256 + D;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(2 * 128 * D * 4 <= OFF_VEC, "the join lies over the tiles");
};

// SPLIT: a cluster shares a tile's steps; each CTA's sums stay in its own
// shared memory and the cluster adds them from there in rank order.
template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
    packed_dkdv_kernel(const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mdo, SeqGeo g, const PackedBwdIO io) {
  using C = DkdvCfg<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int NR = C::NR;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (base - raw);
  const uint32_t sK = base + C::OFF_K, sV = base + C::OFF_V;
  const uint32_t full = base + C::OFF_BAR, s_ready = full + 8 * NR, dp_ready = s_ready + 8;
  const uint32_t dp_read = dp_ready + 8, st_issued = dp_read + 8;
  const uint32_t p_ready = st_issued + 8, ds_ready = p_ready + 16;
  const uint32_t x_free = ds_ready + 8, own = x_free + 8;
  const uint32_t fix_go = own + 8, fixed = fix_go + 8, done = fixed + 8, drain = done + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  int* found = reinterpret_cast<int*>(sm + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = SPLIT ? int(cluster_rank()) : 0, ranks = SPLIT ? int(cluster_size()) : 1;
  const uint32_t unit = blockIdx.x / uint32_t(ranks);
  const int kvh = int(unit % uint32_t(g.kv_heads));
  auto qslot = [&](int p) { return base + C::OFF_STG + (p % NR) * 2 * C::TILE; };
  auto doslot = [&](int p) { return qslot(p) + C::TILE; };
  auto vecslot = [&](int p) { return base + C::OFF_VEC + (p % NR) * 1024; };

  int q0 = 0, Lq = 0, k0 = 0, Lk = 0, first = 0, seq = 0;
  // query tiles qt0 .. qt0+per-1 of each of the group's heads, head after head
  int qt0 = 0, per = 1, np = 0;
  int skip = 0;  // steps of the tile that lower ranks take; np are this CTA's
  bool any = false;
  auto plan = [&] {
    if (any && Lq > 0) {
      if (g.causal) qt0 = max(0, first + Lq - Lk) >> 7;
      per = ((Lq + 127) >> 7) - qt0;
      np = per * g.group;
      if (SPLIT) {
        const int share = (np + ranks - 1) / ranks;
        skip = min(np, rank * share);
        np = min(np, skip + share) - skip;
      }
    }
  };
  // Q and dO tiles of step p with their rows' lse2 and D
  const int64_t stats = stat_rows(io.total_q, io.n_seqs);
  int lh = kvh * g.group, lt = 0, loaded = 0;  // head, query tile and step of the next load
  auto load = [&] {
    const int p = loaded++;
    const uint32_t bar = full + 8 * (p % NR);
    mbar_arrive_expect_tx(bar, 2 * C::TILE + 1024);
    tma_load_rows(qslot(p), &mq, bar, q0 + lt * 128, lh);
    tma_load_rows(doslot(p), &mdo, bar, q0 + lt * 128, lh);
    const int64_t at = lh * stats + stat_start(q0, seq) + lt * 128;
    bulk_load(vecslot(p), io.stat_lse + at, 512, bar);
    bulk_load(vecslot(p) + 512, io.stat_delta + at, 512, bar);
    if (++lt == qt0 + per) {
      lt = qt0;
      ++lh;
    }
  };
  if (warp == 10) {
    if (lane == 0) {
      for (int s = 0; s < NR; ++s) mbar_init(full + 8 * s, 1);
      mbar_init(s_ready, 1);
      mbar_init(dp_ready, 1);
      mbar_init(dp_read, 8);
      mbar_init(st_issued, 1);
      mbar_init(p_ready, 8);
      mbar_init(p_ready + 8, 8);
      mbar_init(ds_ready, 8);
      mbar_init(x_free, 1);
      mbar_init(own, 1);
      mbar_init(fix_go, 1);
      mbar_init(fixed, 1);
      mbar_init(done, 2);
      mbar_init(drain, 1);
      mbar_init(drain + 8, 1);
      *abort_flag = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    named_bar_sync(1, 64);
  } else if (warp == 8) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  } else if (warp == 11 && lane == 0 && io.total_q > 0 && io.total_k > 0) {  // else no maps
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mdo);
  } else if (warp == 9) {
    const Tile t = find_tile<kWalkK>(io.cu_k, io.total_k, io.cu_q, io.total_q, io.n_seqs, g.causal,
                                     128, unit / uint32_t(g.kv_heads), lane, io.status);
    any = t.any, q0 = t.b.start, Lq = t.b.len, k0 = t.a.start, Lk = t.a.len;
    first = t.tile * 128, seq = t.seq;
    if (lane == 0) {
      found[0] = any, found[1] = q0, found[2] = Lq, found[3] = k0, found[4] = Lk;
      found[5] = first, found[6] = seq;
    }
    plan();
    lh += skip / per;
    lt = qt0 + skip % per;
    named_bar_sync(1, 64);  // the barriers are set up
    // the first copies start before the rest of the set-up
    if (lane == 0 && np > 0) {
      mbar_arrive_expect_tx(own, 2 * C::TILE);
      tma_load_rows(sK, &mk, own, k0 + first, kvh);
      tma_load_rows(sV, &mv, own, k0 + first, kvh);
      // dQ writes the row statistics that come with the queries
      cudaGridDependencySynchronize();
      load();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (warp != 9) {
    any = found[0] != 0;
    q0 = found[1], Lq = found[2], k0 = found[3], Lk = found[4], first = found[5], seq = found[6];
    plan();
  }
  const bool has_tail = np > 0 && (Lq & 127) != 0;  // a head's last tile is partial

  if (warp == 9) {
    // ---- the copies: step p into the slot of step p - 2 once its
    // accumulations have finished
    if (lane == 0 && np > 0) {
      bool ok = true;
      while (ok && loaded < np) {
        if (loaded >= NR) ok = mbar_wait(x_free, (loaded - NR) & 1, abort_flag);
        if (ok) load();
      }
      if (!ok) report_timeout(abort_flag, io.status);
      if (!ok || *abort_flag) {
        // the newest copies may still be landing
        mbar_wait(own, 0, nullptr, 200000000ull);
        for (int p = loaded > NR ? loaded - NR : 0; p < loaded; ++p)
          mbar_wait(full + 8 * (p % NR), (p / NR) & 1, nullptr, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---- the foreign rows of the heads' last Q and dO tiles
    if (has_tail) {
      int tails = 0;
      for (int p = per - 1 - skip % per; p < np; p += per) {
        if (!__all_sync(0xffffffffu, mbar_wait(fix_go, tails++ & 1, abort_flag,
                                               2000000000ull + uint64_t(np) * 10000ull))) {
          if (lane == 0) report_timeout(abort_flag, io.status);
          break;
        }
        zero_rows(qslot(p), C::KB, Lq & 127, lane);
        zero_rows(doslot(p), C::KB, Lq & 127, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed);
      }
    }
  } else if (warp == 8) {
    // ---- S^T and dP^T of each step
    if (lane == 0 && np > 0) {
      constexpr uint32_t idesc_s = idesc_f32<T>(128, 128, false);
      int in_head = skip % per, tails = 0;
      bool ok = mbar_wait(own, 0, abort_flag);
      for (int p = 0; ok && p < np; ++p) {
        const uint32_t cS = 128u * (p & 1), cDP = 128u - cS;
        ok = mbar_wait(full + 8 * (p % NR), (p / NR) & 1, abort_flag);
        if (!ok) break;
        if (++in_head == per) {
          in_head = 0;
          if (has_tail) {
            mbar_arrive(fix_go);
            ok = mbar_wait(fixed, tails & 1, abort_flag);
            if (!ok) break;
            ++tails;
          }
        }
        // S^T once the groups have read dP^T of step p-1 from its region
        if (p > 0) ok = mbar_wait(dp_read, (p - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + cS, sdesc_sw128(sK + off, 16, 1024),
                    sdesc_sw128(qslot(p) + off, 16, 1024), idesc_s, kk > 0);
        }
        // before s_ready: whoever has P^T of this step then finds its phase over
        mbar_arrive(st_issued);
        tc_commit(s_ready);
        // dP^T once the accumulations of step p-1 have read P^T and dS^T from its region
        if (p > 0) ok = mbar_wait(x_free, (p - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BOX + (kk % 4) * 32;
          tc_mma_ss(tmem + cDP, sdesc_sw128(sV + off, 16, 1024),
                    sdesc_sw128(doslot(p) + off, 16, 1024), idesc_s, kk > 0);
        }
        tc_commit(dp_ready);
      }
      if (!ok) report_timeout(abort_flag, io.status);
      tc_commit(done);
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---- dV += P^T dO once both groups' P^T is in, then dK += dS^T Q; B read
    // N-major.  (All products by one thread, which needs no wait between dK and
    // the next dP^T, took 270 us where two threads take 260.)
    if (lane == 0 && np > 0) {
      constexpr uint32_t idesc_acc = idesc_f32<T>(128, D, true);
      bool ok = true;
      // test hook: with `stall` set no accumulation is issued (the timeout path)
      for (int p = 0; ok && p < np && !io.stall; ++p) {
        const uint32_t cS = 128u * (p & 1);
        auto sums = [&](uint32_t acc, uint32_t col, uint32_t rows) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + acc, tmem + col + 64u * (kk >> 2) + 8u * (kk & 3),
                      sdesc_sw128(rows + kk * 2048, C::BOX, 1024), idesc_acc,
                      (p > 0 || kk > 0) ? 1u : 0u);
        };
        ok = mbar_wait(p_ready + 8 * (p & 1), (p >> 1) & 1, abort_flag);
        if (!ok) break;
        sums(C::COL_DV, cS, doslot(p));
        // dK is queued behind the next S^T, which the groups wait for first; so
        // x_free of step p comes only after load p + 1, and the copies cannot
        // be overtaken at x_free
        ok = (p + 1 == np || mbar_wait(st_issued, (p + 1) & 1, abort_flag)) &&
             mbar_wait(ds_ready, p & 1, abort_flag);
        if (!ok) break;
        sums(C::COL_DK, cS + 32u, qslot(p));
        tc_commit(x_free);
      }
      if (!ok) report_timeout(abort_flag, io.status);
      tc_commit(done);
      tc_commit(drain + 8);
      mbar_wait(drain + 8, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else {
    // ---- row groups: key row r of the tile = TMEM lane r
    const int grp = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane, kr = first + row;
    const uint32_t lane_base = uint32_t(quad * 32) << 16;
    const bool exists = any && kr < Lk;
    const float sl2 = g.scale * kLog2e;
    if (kHalf) cudaGridDependencySynchronize();  // the norms
    const float fac = kHalf && np > 0 ? ds_factor(io.norms, seq, kvh, g.kv_heads) : 1.f;
    const float fac_p = kHalf ? fac * exp2f(-kPShift) : 1.f;
    const float shift = kHalf ? kPShift : 0.f;
    bool ok = true;
    int qt = qt0 + skip % per;
    for (int p = 0; p < np; ++p) {
      const uint32_t tS = tmem + 128u * (p & 1) + 64u * grp + lane_base;
      const uint32_t tDP = tmem + 128u * ((p & 1) ^ 1) + 64u * grp + lane_base;
      ok = __all_sync(0xffffffffu, mbar_wait(s_ready, p & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      // query columns from `from` on see this key (rows behind Lq have P = 0)
      const int from = g.causal ? kr + Lq - Lk - 128 * qt - 64 * grp : 0;
      if (++qt == qt0 + per) qt = qt0;
      const bool dense = __all_sync(0xffffffffu, !exists || from <= 0);
      uint32_t sv[64], dp[64];
      BSA_TMEM_LD64(tS, sv);
      const float* lse = reinterpret_cast<const float*>(sm + C::OFF_VEC + (p % NR) * 1024) + 64 * grp;
      const float* dlt = lse + 128;
      // P^T over S^T first, so that dV starts while dS^T is computed; the
      // probabilities stay in sv.  32 query columns at a time.
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        uint32_t pk[16];
        float4 l4[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) l4[i] = reinterpret_cast<const float4*>(lse)[8 * h2 + i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = 32 * h2 + 4 * i;
          float x0, x1, x2, x3;
          fma_f32x2(x0, x1, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), sl2, sl2,
                    shift - l4[i].x, shift - l4[i].y);
          fma_f32x2(x2, x3, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]), sl2, sl2,
                    shift - l4[i].z, shift - l4[i].w);
          float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
          if (!dense) {
            p0 = c >= from ? p0 : 0.f;
            p1 = c + 1 >= from ? p1 : 0.f;
            p2 = c + 2 >= from ? p2 : 0.f;
            p3 = c + 3 >= from ? p3 : 0.f;
          }
          sv[c] = __float_as_uint(p0);
          sv[c + 1] = __float_as_uint(p1);
          sv[c + 2] = __float_as_uint(p2);
          sv[c + 3] = __float_as_uint(p3);
          pk[2 * i] = pack2<T>(p0, p1);
          pk[2 * i + 1] = pack2<T>(p2, p3);
        }
        BSA_TMEM_ST16(tS + 16u * h2, pk);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready + 8 * (p & 1));
      // dS^T = P^T * (dP^T - D) beside P^T, 32 columns at a time
      ok = __all_sync(0xffffffffu, mbar_wait(dp_ready, p & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        BSA_TMEM_LD32(tDP + 32u * h2, (dp + 32 * h2));
        if (h2 == 1) {
          // dP^T read: the next S^T may go over it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_read);
        }
        uint32_t pk[16];
#pragma unroll
        for (int c4 = 8 * h2; c4 < 8 * h2 + 8; ++c4) {
          const float4 t4 = reinterpret_cast<const float4*>(dlt)[c4];
          const float dv[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            const int c = 4 * c4 + u;
            float t0, t1, d0, d1;
            add_f32x2(t0, t1, __uint_as_float(dp[c]), __uint_as_float(dp[c + 1]), -dv[u],
                      -dv[u + 1]);
            if constexpr (kHalf) fma_f32x2(t0, t1, t0, t1, fac_p, fac_p, 0.f, 0.f);
            fma_f32x2(d0, d1, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), t0, t1, 0.f,
                      0.f);
            pk[(c - 32 * h2) / 2] = pack2<T>(d0, d1);
          }
        }
        BSA_TMEM_ST16(tS + 32u + 16u * h2, pk);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    if (ok && np > 0) ok = __all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag));
    if (!ok) {
      if (lane == 0) report_timeout(abort_flag, io.status);
    } else if (!SPLIT) {
      // group 0 writes dV, group 1 dK; keys no query saw have zero gradients
      tc_fence_after();
      const Rows& out = grp ? io.dk : io.dv;
      const float f = grp ? g.scale / fac : (kHalf ? exp2f(-kPShift) : 1.f);
      if (any) {
        const int row0 = first + quad * 32;  // the warp's first row
        T* dst = static_cast<T*>(out.p) + int64_t(k0 + row0) * out.sn + int64_t(kvh) * out.sh;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c)
          write_channels<T>(sK + warp * 4096,
                            tmem + (grp ? C::COL_DK : C::COL_DV) + 64u * c + lane_base,
                            dst + 64 * c, out.sn, min(32, Lk - row0), f, np > 0, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (SPLIT) {
    // ---- the join: fp32 dV then dK of this CTA's steps, 128 rows each, 16-byte
    // chunks swizzled by the row, over the tiles
    if (warp < 8) {
      const int grp = warp >> 2, row = (warp & 3) * 32 + lane;
      const uint32_t mine = base + grp * (128 * D * 4) + row * (D * 4);
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t a[32];
        BSA_TMEM_LD32(tmem + (grp ? C::COL_DK : C::COL_DV) + 32u * ch +
                          (uint32_t((warp & 3) * 32) << 16), a);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(mine + (((8 * ch + j) ^ (row & 7)) << 4),
                       np > 0 ? make_uint4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3])
                              : make_uint4(0u, 0u, 0u, 0u));
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync();
    if (any && !*abort_flag) {
      // rank c writes rows c, c + ranks, .. of both: 16-byte output chunks
      constexpr int CH = D / 8;
      const float fac = kHalf ? ds_factor(io.norms, seq, kvh, g.kv_heads) : 1.f;
      for (int i = threadIdx.x; i < 2 * (128 / ranks) * CH; i += C::kThreads) {
        const int ch = i % CH, rr = (i / CH) * ranks + rank, grp = rr >> 7, row = rr & 127;
        if (first + row >= Lk) continue;
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < ranks; ++c) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float4 v = ld_cluster_f4(peer_smem(base + grp * (128 * D * 4) + row * (D * 4) +
                                                         (((2 * ch + x) ^ (row & 7)) << 4), c));
            o[4 * x] += v.x, o[4 * x + 1] += v.y, o[4 * x + 2] += v.z, o[4 * x + 3] += v.w;
          }
        }
        const float f = grp ? g.scale / fac : (kHalf ? exp2f(-kPShift) : 1.f);
        const Rows& out = grp ? io.dk : io.dv;
        *reinterpret_cast<uint4*>(static_cast<T*>(out.p) + int64_t(k0 + first + row) * out.sn +
                                  int64_t(kvh) * out.sh + ch * 8) =
            make_uint4(pack2<T>(o[0] * f, o[1] * f), pack2<T>(o[2] * f, o[3] * f),
                       pack2<T>(o[4] * f, o[5] * f), pack2<T>(o[6] * f, o[7] * f));
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are read
  }
  if (warp == 8) tmem_dealloc(tmem, C::TMEM_COLS);
  cudaGridDependencySynchronize();  // whatever a tile did: dQ has finished, too
}

// CTAs that share a key tile: a tile takes one step per query tile and head of
// its group, and few kv heads leave SMs idle beside long chains of steps.  us of
// the whole backward with 1 | 2 | 4 | 8 CTAs a tile (16 or 32 heads, bf16):
//   1,024 queries, 1 kv head:   507 | 276 | 163 | 109
//   512 queries, 8 kv heads:     54 |  43 |  39 |  76
//   1,024 queries, 8 kv heads:   99 |  74 |  78 | 141
//   2,048 queries, 4 kv heads:  313 | 199 | 160 | 227
//   900 queries, 16 kv heads:    49 |  58 |  94 | 195
// One wave pays from three steps a CTA, two waves from ten; few clusters of
// eight find room at a time.
int split_ranks(const SeqGeo& g, const PackedBwdIO& io) {
  // the sequences' last tiles are half full on average
  const int64_t units = (io.total_k / 128 + io.n_seqs / 2) * g.kv_heads;
  const int64_t steps = (io.total_q + 127) / 128 * g.group;
  if (units * 8 <= 148 && steps >= 64) return 8;
  for (int r = 4; r > 1; r /= 2)
    if (units * r <= 148 ? steps >= 3 * r : (units * r <= 300 && steps >= 10 * r)) return r;
  return 1;
}

// A launch that may set itself up on the SMs that the kernel before it leaves
// idle; it waits for that kernel before it reads the row statistics.
template <typename K, typename... A>
cudaError_t launch_after(K kern, unsigned ctas, int ranks, int threads, int smem, bool early,
                         cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  int n = 0;
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (ranks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(ranks);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// the norms of every sequence and kv head, dO's and V's
size_t norm_count(const SeqGeo& g, int64_t n_seqs) {
  return 2 * size_t(g.kv_heads) * size_t(g.fp16 && n_seqs > 1 ? n_seqs : 1);
}

template <typename T, int D>
cudaError_t launch_t(const SeqGeo& g, const CUtensorMap* maps, const PackedBwdIO& io,
                     cudaStream_t st) {
  auto tiles = [&](int64_t rows) { return tile_places(rows, io.n_seqs, 128); };
  cudaError_t e;
  if (io.total_q > 0) {
    const int64_t n_tiles = tiles(io.total_q);
    int64_t v_blocks = 0;
    if (std::is_same<T, __half>::value) {
      e = cudaMemsetAsync(io.norms, 0, sizeof(float) * norm_count(g, io.n_seqs), st);
      if (e != cudaSuccess) return e;
      if (io.total_k > 0) v_blocks = (tiles(io.total_k) * g.kv_heads + g.heads - 1) / g.heads;
    }
    bwd_prepare_kernel<T, D>
        <<<dim3(unsigned(n_tiles + v_blocks), g.heads), 256, 0, st>>>(g, io, int(n_tiles));
    auto dq = packed_dq_kernel<T, D>;
    static std::atomic<uint64_t> seen{0};
    e = allow_smem(dq, DqCfg<D>::SMEM, seen);
    if (e != cudaSuccess) return e;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_after(dq, unsigned(n_tiles * g.heads), 1, DqCfg<D>::kThreads, DqCfg<D>::SMEM, true,
                     st, maps[0], maps[1], maps[2], maps[3], g, io);
    if (e != cudaSuccess) return e;
  }
  if (io.total_k > 0) {
    const int ranks = split_ranks(g, io);
    const int64_t units = tiles(io.total_k) * g.kv_heads;
    auto go = [&](auto dkdv, std::atomic<uint64_t>& seen) {
      const cudaError_t r = allow_smem(dkdv, DkdvCfg<D>::SMEM, seen);
      if (r != cudaSuccess) return r;
      return launch_after(dkdv, unsigned(units * ranks), ranks, DkdvCfg<D>::kThreads,
                          DkdvCfg<D>::SMEM, io.total_q > 0, st, maps[0], maps[1], maps[2], maps[3],
                          g, io);
    };
    static std::atomic<uint64_t> seen[2];
    e = ranks > 1 ? go(packed_dkdv_kernel<T, D, true>, seen[1])
                  : go(packed_dkdv_kernel<T, D, false>, seen[0]);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t packed_bwd_workspace_bytes(const SeqGeo& g, int64_t total_q, int64_t n_seqs) {
  // statistics (lse2 and D per head and padded row) and the norms
  return sizeof(float) * (2 * size_t(g.heads) * stat_rows(total_q, n_seqs) + norm_count(g, n_seqs));
}

void packed_bwd_workspace_split(const SeqGeo& g, PackedBwdIO* io, void* workspace) {
  const size_t n = size_t(g.heads) * stat_rows(io->total_q, io->n_seqs);
  io->stat_lse = static_cast<float*>(workspace);
  io->stat_delta = io->stat_lse + n;
  io->norms = io->stat_delta + n;
}

cudaError_t launch_packed_bwd(const SeqGeo& g, const CUtensorMap* maps, const PackedBwdIO& io,
                              cudaStream_t st) {
  if (g.d == 128)
    return g.fp16 ? launch_t<__half, 128>(g, maps, io, st) : launch_t<__nv_bfloat16, 128>(g, maps, io, st);
  return g.fp16 ? launch_t<__half, 64>(g, maps, io, st) : launch_t<__nv_bfloat16, 64>(g, maps, io, st);
}

}  // namespace bsa
