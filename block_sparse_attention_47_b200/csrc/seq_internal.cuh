// Internal definitions shared by the token-sequence translation units
// (packed attention, paged cache): problem geometry, the paged cache, the
// element types, and the host-side checks of bsa_api.cu they use.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "../../include/bsa_seq.h"
#include "bsa_internal.cuh"

namespace bsa {

// ---- host side, defined in bsa_api.cu --------------------------------------
void clear_error();
bsa_status cuda_error(cudaError_t e, const char* what);
bsa_status require_device();                 // the current device is sm_100
bsa_status resolve_status(int32_t** status);  // the caller's word or the library's
int device_sms();                            // of the current device
bool stall_enabled();                        // bsa_debug_stall_pv of this thread
void range_push(const char* name);
void range_pop();
// a [rows, heads, d] 16-bit tensor as a 4-D map whose box is box_rows rows of
// one head, 64 columns after the other ([column box][row][64] in shared memory)
bsa_status make_rows_map(CUtensorMap* m, const void* ptr, int64_t rows, int heads, int d,
                         int64_t stride_n, int64_t stride_h, int box_rows, bool fp16);

// Opt a kernel in to its shared memory, once per device.
template <typename K>
inline cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (seen.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_release);
  return e;
}

struct SeqGeo {
  int heads, kv_heads, group, d;
  bool fp16;
  bool causal;
  float scale;
};

struct Rows {  // a strided [rows, heads, d] tensor
  void* p;
  int64_t sn, sh;
};

struct PagedCache {
  void *k, *v;
  int64_t sp, st, sh;  // page, token, head strides (elements)
  int n_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  int table_width;
};

// ---- launchers ---------------------------------------------------------------
struct AppendIO {
  Rows k, v, q, q_out, k_out;  // q.p / k_out.p may be null
  const int32_t* cu;
  const int32_t* lens;
  const float* rope;
  const int32_t* rope_rows;
  int rope_n, rot, interleaved;
  int n_seqs;
  int64_t n_tokens;
  int32_t* status;
};
cudaError_t launch_kv_append(const SeqGeo& g, const PagedCache& c, const AppendIO& io,
                             cudaStream_t st);

size_t decode_workspace_bytes(const SeqGeo& g);
struct DecodeIO {
  Rows q, o;
  const int32_t* lens;
  int n_seqs;
  void* workspace;
  int32_t* status;
};
// Pointers of one packed forward; maps: Q, K, V (128-row boxes; K and V are
// not read when total_k is 0).
struct PackedIO {
  const int32_t *cu_q, *cu_k;
  int n_seqs;
  int64_t total_q, total_k;
  Rows o;
  float* lse;  // [heads, total_q], exp2 domain, or null
  int32_t* status;
  int stall;   // test hook: no PV is issued
};
cudaError_t launch_packed_fwd(const SeqGeo& g, const CUtensorMap* maps, const PackedIO& io,
                              cudaStream_t st);

// Pointers of one packed backward; maps: Q, K, V, dO (128-row boxes).
struct PackedBwdIO {
  const int32_t *cu_q, *cu_k;
  int n_seqs;
  int64_t total_q, total_k;
  Rows o, dout, v, dq, dk, dv;
  const float* lse;    // [heads, total_q] from the forward
  // workspace: statistics per head and padded row, the largest squared norms
  // of dO and V rows per sequence and kv head (fp16)
  float *stat_lse, *stat_delta, *norms;
  int32_t* status;
  int stall;
};
size_t packed_bwd_workspace_bytes(const SeqGeo& g, int64_t total_q, int64_t n_seqs);
void packed_bwd_workspace_split(const SeqGeo& g, PackedBwdIO* io, void* workspace);
cudaError_t launch_packed_bwd(const SeqGeo& g, const CUtensorMap* maps, const PackedBwdIO& io,
                              cudaStream_t st);

cudaError_t launch_paged_decode(const SeqGeo& g, const PagedCache& c, const DecodeIO& io,
                                cudaStream_t st);

#if defined(__CUDACC__)
// ---- device helpers ------------------------------------------------------------
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<__half2*>(&u));
}

__device__ __forceinline__ void report_invalid(int32_t* status) {
  atomicCAS(status, 0, int32_t(BSA_ERR_INVALID_ARG));
}

// Instruction descriptor of kind::f16 with fp16 or bf16 A and B, fp32 D.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool b_mn_major) {
  return idesc_bf16_f32(M, N, b_mn_major) &
         (std::is_same<T, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);
}

#define BSA_TMEM_ST16(taddr, r)                                                               \
  asm volatile(                                                                               \
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "                                        \
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"                         \
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),                                          \
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), \
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),       \
      "r"(r[15])                                                                              \
      : "memory")

// 128 columns of this thread's tensor-memory lane
#define BSA_TMEM_LD128(taddr, r)  \
  asm volatile(  \
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"  \
      "tcgen05.wait::ld.sync.aligned;"  \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])  \
      : "r"(taddr)  \
      : "memory")

// one box of such a map: `row` and the next rows of `head`
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int row, int head) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(0), "r"(head)
      : "memory");
}

// ---- clusters that share one tile ------------------------------------------------
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

// ---- packed sequences ------------------------------------------------------------
// One sequence of a packed call; offsets that descend or leave the tensor are
// reported and read as an empty sequence.
struct Span {
  int start, len;
};
__device__ __forceinline__ Span checked_span(int a, int z, int64_t total, int32_t* status) {
  if (a < 0 || z < a || z > total) {
    report_invalid(status);
    return {0, 0};
  }
  return {a, z - a};
}

// A tile of a packed call: the rows of sequence `seq` in the tiled tensor (a)
// and in the other one (b).
struct Tile {
  bool any;
  int seq, tile;
  Span a, b;
};

// How long the walks of a sequence's tiles are.  kWalkQ: tiles of `rows`
// queries (a) over 128-key steps of b, the last tile's the longest; kWalkK:
// tiles of 128 keys (a) over the 128-query steps of b that see them, the
// first tile's the longest.
enum { kWalkQ, kWalkK };

// tiles whose walk is longer than thr steps (they are the longest-walk end)
template <int WALK>
__device__ __forceinline__ int tiles_beyond(const Span& a, const Span& b, bool causal, int rows,
                                            int thr) {
  const int n = (a.len + rows - 1) / rows;
  if (thr < 0) return n;
  if (WALK == kWalkQ) {
    if (b.len <= 128 * thr) return 0;
    if (!causal) return n;
    const int need = 128 * thr - (b.len - a.len);  // rows up to here see no more than thr steps
    return n - (need < 0 ? 0 : need / rows);
  }
  const int left = (b.len + 127) / 128 - thr;
  if (left <= 0) return 0;
  if (!causal) return n;
  const int reach = 128 * left - (b.len - a.len);
  return reach <= 0 ? 0 : min(n, (reach + 127) / 128);
}

// The list of all sequences' tiles of `rows` rows has this many places.
constexpr int kListed = 32;
__host__ __device__ __forceinline__ int64_t tile_places(int64_t total, int64_t n_seqs, int rows) {
  return total / rows + (n_seqs <= kListed && total < n_seqs ? total : n_seqs);
}

// Of more than kListed sequences: sequence b's tiles start at place
// cu[b] / rows + b, which leaves room for every tile whatever the lengths and
// up to n_seqs places empty, so a place's sequence is searched for, 32 ways a
// turn, instead of counted up to (16,384 sequences of 20 tokens, 8 heads:
// forward 88 ms by counting).  The place also checks the offsets of the
// sequence of its own number, so that bad ones are reported wherever the
// search went.
template <int WALK>
__device__ __forceinline__ Tile search_tile(const int32_t* __restrict__ cu_a, int64_t total_a,
                                            const int32_t* __restrict__ cu_b, int64_t total_b,
                                            int n_seqs, int rows, int64_t target, int lane,
                                            int32_t* status) {
  Tile t{};
  if (target < n_seqs && lane == 0) {
    checked_span(__ldg(cu_a + target), __ldg(cu_a + target + 1), total_a, status);
    checked_span(__ldg(cu_b + target), __ldg(cu_b + target + 1), total_b, status);
  }
  __syncwarp();
  auto place = [&](int s) { return max(__ldg(cu_a + s), 0) / rows + int64_t(s); };
  int lo = 0, n = n_seqs;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, at < lo + n && place(at) <= target);
    if (m == 0u) return t;  // in front of the first sequence
    const int top = 31 - __clz(m), end = lo + n;
    lo += top * step;
    n = min(step, end - lo);
  }
  t.seq = lo;
  t.a = checked_span(__ldg(cu_a + lo), __ldg(cu_a + lo + 1), total_a, status);
  t.b = checked_span(__ldg(cu_b + lo), __ldg(cu_b + lo + 1), total_b, status);
  const int64_t i = target - place(lo), tiles = (int64_t(t.a.len) + rows - 1) / rows;
  t.any = i >= 0 && i < tiles;
  if (t.any) t.tile = int(WALK == kWalkQ ? tiles - 1 - i : i);
  return t;
}

// The tile `target` of the list, by a whole warp; any = false where there is
// none (behind the list's end, or an empty place of many sequences).  Up to
// kListed sequences: without empty places, and long walks first, so that the
// grid does not end on them, in four classes (walks beyond 1/2, 1/4 and 1/8
// of the longest, the others).
template <int WALK>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ cu_a, int64_t total_a,
                                          const int32_t* __restrict__ cu_b, int64_t total_b,
                                          int n_seqs, bool causal, int rows, int64_t target,
                                          int lane, int32_t* status) {
  if (n_seqs > kListed)
    return search_tile<WALK>(cu_a, total_a, cu_b, total_b, n_seqs, rows, target, lane, status);
  Tile t{};
  Span a{0, 0}, b{0, 0};
  if (lane < n_seqs) {
    a = checked_span(__ldg(cu_a + lane), __ldg(cu_a + lane + 1), total_a, status);
    b = checked_span(__ldg(cu_b + lane), __ldg(cu_b + lane + 1), total_b, status);
  }
  const int n_all = (a.len + rows - 1) / rows;
  const int longest =
      __reduce_max_sync(0xffffffffu, a.len > 0 ? (b.len + 127) / 128 : 0);
  // this sequence's tiles of each class and of those before it, and the scans
  // of all four over the sequences side by side
  int upto[4], incl[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    upto[c] = c == 3 ? n_all : tiles_beyond<WALK>(a, b, causal, rows, longest >> (c + 1));
    incl[c] = upto[c] - (c ? upto[c - 1] : 0);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int v = __shfl_up_sync(0xffffffffu, incl[c], o);
      if (lane >= o) incl[c] += v;
    }
  }
  int64_t before = 0;
  int in = 0, up = 0;  // the scans of the class that holds the place
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int total = __shfl_sync(0xffffffffu, incl[c], 31);
    if (!t.any) {
      t.any = before + total > target;
      in = incl[c], up = upto[c];
      if (!t.any) before += total;
    }
  }
  if (!t.any) return t;
  const int l = __ffs(__ballot_sync(0xffffffffu, before + in > target)) - 1;
  // its place among the sequence's tiles, longest walk first
  const int p = __shfl_sync(0xffffffffu, int(target - before) - in + up, l);
  const int n_l = __shfl_sync(0xffffffffu, n_all, l);
  t.seq = l;
  t.tile = WALK == kWalkQ ? n_l - 1 - p : p;
  t.a = {__shfl_sync(0xffffffffu, a.start, l), __shfl_sync(0xffffffffu, a.len, l)};
  t.b = {__shfl_sync(0xffffffffu, b.start, l), __shfl_sync(0xffffffffu, b.len, l)};
  return t;
}

// Rows of a 16-bit tile through shared memory, so that a warp writes whole
// rows: a thread stages its own row (16-byte chunks swizzled by the row), and
// the warp then writes 16 bytes a lane, 512 consecutive ones at d = 128.
// `stage`: this warp's 32 rows of D * 2 bytes.
template <int D>
__device__ __forceinline__ void stage_chunk(uint32_t stage, int row, int chunk, uint4 v) {
  st_shared_v4(stage + row * (2 * D) + ((chunk ^ (row & 7)) << 4), v);
}
template <typename T, int D>
__device__ __forceinline__ void write_rows(uint32_t stage, T* dst, int64_t stride, int n_rows,
                                           int lane) {
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  __syncwarp();
#pragma unroll
  for (int it = 0; it < CH; ++it) {
    const int row = it * (32 / CH) + lane / CH, ch = lane % CH;
    const float4 v = ld_shared_f4(stage + row * (2 * D) + ((ch ^ (row & 7)) << 4));
    if (row < n_rows)
      *reinterpret_cast<float4*>(dst + int64_t(row) * stride + ch * 8) = v;
  }
  __syncwarp();
}

__device__ __forceinline__ void report_timeout(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  atomicCAS(status, 0, int32_t(BSA_ERR_TIMEOUT));
}
#endif

}  // namespace bsa
