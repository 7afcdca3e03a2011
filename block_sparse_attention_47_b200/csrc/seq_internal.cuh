// Internal definitions shared by the token-sequence translation units
// (packed attention, paged cache): problem geometry, the paged cache, the
// element types, and the host-side checks of bsa_api.cu they use.
#pragma once

#include <cuda_fp16.h>

#include "../../include/bsa_seq.h"
#include "bsa_internal.cuh"

namespace bsa {

// ---- host side, defined in bsa_api.cu --------------------------------------
void clear_error();
bsa_status cuda_error(cudaError_t e, const char* what);
bsa_status require_device();                 // the current device is sm_100
bsa_status resolve_status(int32_t** status);  // the caller's word or the library's
bool stall_enabled();                        // bsa_debug_stall_pv of this thread
void range_push(const char* name);
void range_pop();
// a [rows, heads, d] 16-bit tensor as a 3-D map, box 64 columns x 1 head x box_rows
bsa_status make_rows_map(CUtensorMap* m, const void* ptr, int64_t rows, int heads, int d,
                         int64_t stride_n, int64_t stride_h, int box_rows, bool fp16);

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
#endif

}  // namespace bsa
