// quant_cache.cu -- a paged KV cache in 8 bits: new tokens quantised as they
// are written into their pages, the block-mean summary kept current, and
// tokens read back.
//
// Format.  A row (one token's key or value of one KV head) is d codes e4m3
// (4 exponent, 3 fraction bits) and one exponent byte e; a value is
// code * 2^(e - 127).  e is the least exponent that brings the row's largest
// magnitude within 448, the largest e4m3 value: with amax = 1.f * 2^E (biased
// E), e = E - 8 + (1.f > 1.75), kept within [10, 246].  A power of two makes
// the division exact, so a code is one rounding (to nearest, ties to even;
// at most 2^-4 of the value) away from its input, and the value it stands for
// is exact in bf16.  A scale with a fraction could use the top binade better,
// but codes that are floating point themselves lose nothing to it.
// Infinities and NaN become the NaN code and do not enter amax: e4m3 has no
// infinity, and a saturated value would hide a broken row.
//
// Layout.  Codes [P][Hkv][64][d] and exponents [P][Hkv][64], pages of 64
// tokens as in the bf16 paged cache, so a head's page is one run of memory.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace bsa {
namespace qcache {

constexpr int kThreads = 256;

// Exponent byte of a row whose largest finite magnitude is m.
__device__ __forceinline__ uint32_t exponent_byte(float m) {
  const uint32_t u = __float_as_uint(m);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 10), 246));
}
__device__ __forceinline__ float two_to(uint32_t e) { return __uint_as_float(e << 23); }

// Eight codes -> eight values.
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&v)[8]) {
  const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(ws[i >> 1] >> ((i & 1) * 16));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// One CTA per (sequence, KV head, touched block): the block's new tokens are
// quantised row by row (GS lanes a row, eight channels a lane; keys and values
// alternate), and if the append completes the block its mean key is summed
// from the codes, tokens ascending, fp32, one division -- from shared memory,
// which also takes the tokens that lay in the block before.  One launch, no
// block waits for another.
template <int GS>
__global__ void __launch_bounds__(kThreads) append_kernel(const QuantCacheArgs p) {
  griddep_wait();
  extern __shared__ uint4 smem_q[];
  uint8_t* codes = reinterpret_cast<uint8_t*>(smem_q);       // [64][d]
  uint8_t* exps = codes + 64 * p.d;                            // [64]
  const int j = blockIdx.x % p.touched;
  const int bg = blockIdx.x / p.touched;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  const int64_t L = p.seq_lens[b];
  const int64_t n = p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
  if (n == 0) return;
  if (L < 0) {
    if (threadIdx.x == 0) atomicOr(p.status, BSA_DEV_BAD_INDEX);
    return;
  }
  const int64_t blk = (L >> 6) + j;
  const int64_t first = max(L, blk * 64), end = min(L + n, blk * 64 + 64);   // positions written here
  if (first >= end) return;
  const int page = blk < p.table_stride ? p.table[static_cast<int64_t>(b) * p.table_stride + blk] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.status, BSA_DEV_BAD_INDEX);
    return;
  }
  const int64_t page_row = (static_cast<int64_t>(page) * p.Hkv + g) * 64;
  const bool complete = p.pooled != nullptr && L + n >= blk * 64 + 64;
  const int o0 = static_cast<int>(first & 63), rows = static_cast<int>(end - first);
  const int64_t src0 = static_cast<int64_t>(bg) * p.T + (first - L);
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS;
  const bool on = 8 * l < p.d;
  // the lanes of this row's group: the groups of a warp may leave the loop at different rows
  const uint32_t group_mask = (GS == 32 ? 0xffffffffu : ((1u << (GS & 31)) - 1u)) << (threadIdx.x % 32 / GS * GS);
  for (int r0 = grp; r0 < 2 * rows; r0 += kThreads / GS * 4) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * (kThreads / GS);
      x[u] = make_uint4(0, 0, 0, 0);
      if (r < 2 * rows && on)
        x[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(r & 1 ? p.v_new : p.k_new) +
                                                    (src0 + (r >> 1)) * p.d + 8 * l));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * (kThreads / GS);
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float v[8], m = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
#pragma unroll
      for (int o = GS / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(group_mask, m, o));
      const uint32_t e = exponent_byte(m);
      const float inv = two_to(254u - e);
      uint32_t code[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE,
                                                __NV_E4M3);
        if (!(fabsf(v[2 * i]) < INFINITY)) two = (two & 0xFF00u) | 0x7Fu;
        if (!(fabsf(v[2 * i + 1]) < INFINITY)) two = (two & 0x00FFu) | 0x7F00u;
        code[i >> 1] |= two << ((i & 1) * 16);
      }
      if (r < 2 * rows && on) {
        const int o = o0 + (r >> 1);
        uint8_t* pool = r & 1 ? p.v_pool : p.k_pool;
        *reinterpret_cast<uint2*>(pool + (page_row + o) * p.d + 8 * l) = make_uint2(code[0], code[1]);
        if (l == 0) (r & 1 ? p.v_exp : p.k_exp)[page_row + o] = static_cast<uint8_t>(e);
        if (complete && !(r & 1)) {
          *reinterpret_cast<uint2*>(codes + o * p.d + 8 * l) = make_uint2(code[0], code[1]);
          if (l == 0) exps[o] = static_cast<uint8_t>(e);
        }
      }
    }
  }
  if (!complete) return;
  // the tokens that lay in this block before (positions [0, o0) of it)
  for (int t = threadIdx.x; t < o0 * (p.d / 8); t += kThreads)
    reinterpret_cast<uint2*>(codes)[t] = reinterpret_cast<const uint2*>(p.k_pool + page_row * p.d)[t];
  for (int t = threadIdx.x; t < o0; t += kThreads) exps[t] = p.k_exp[page_row + t];
  __syncthreads();
  for (int ch = threadIdx.x; ch < p.d; ch += kThreads) {
    float sum = 0.0f;
#pragma unroll 16
    for (int t = 0; t < 64; ++t) {
      const __half h = __half(__nv_cvt_fp8_to_halfraw(codes[t * p.d + ch], __NV_E4M3));
      sum = __fadd_rn(sum, __fmul_rn(__half2float(h), two_to(exps[t])));
    }
    p.pooled[(static_cast<int64_t>(bg) * p.table_stride + blk) * p.d + ch] = __fdiv_rn(sum, 64.0f);
  }
}

// Tokens starts[b] + t of every sequence and head, t < T and below the
// sequence's length, as bf16 (exact) or fp32 rows; other output rows are left
// as they were.  One thread per eight channels.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const QuantCacheArgs p) {
  griddep_wait();
  const int pieces = p.d / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.total) return;
  const int piece = static_cast<int>(i % pieces);
  const int64_t row = i / pieces;                 // (b * Hkv + g) * T + t
  const int t = static_cast<int>(row % p.T);
  const int64_t bg = row / p.T;
  const int b = static_cast<int>(bg / p.Hkv), g = static_cast<int>(bg - static_cast<int64_t>(b) * p.Hkv);
  const int64_t pos = (p.starts ? p.starts[b] : 0) + static_cast<int64_t>(t);
  if (pos >= p.seq_lens[b]) return;
  const int64_t blk = pos >> 6;
  const int page = (pos >= 0 && blk < p.table_stride) ? __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + blk) : -1;
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, BSA_DEV_BAD_INDEX);
    return;
  }
  const int64_t src = (static_cast<int64_t>(page) * p.Hkv + g) * 64 + (pos & 63);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* out = static_cast<T*>(kv ? p.v_out : p.k_out);
    if (out == nullptr) continue;
    float v[8];
    decode8(__ldg(reinterpret_cast<const uint2*>((kv ? p.v_pool : p.k_pool) + src * p.d + 8 * piece)),
            two_to((kv ? p.v_exp : p.k_exp)[src]), v);
    T* dst = out + row * p.d + 8 * piece;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

}  // namespace qcache

cudaError_t launch_quant_append(QuantCacheArgs a, cudaStream_t st) {
  // an append of T tokens touches at most this many blocks of a sequence
  a.touched = (a.T + 62) / 64 + 1;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hkv * a.touched);
  const size_t smem = 64 * static_cast<size_t>(a.d) + 64;
  auto kernel = a.d <= 64 ? qcache::append_kernel<8> : (a.d <= 128 ? qcache::append_kernel<16> : qcache::append_kernel<32>);
  return launch_dependent(kernel, dim3(grid), dim3(qcache::kThreads), smem, st, a);
}

cudaError_t launch_quant_read(QuantCacheArgs a, bool bf16, cudaStream_t st) {
  a.total = static_cast<int64_t>(a.B) * a.Hkv * a.T * (a.d / 8);
  const unsigned grid = static_cast<unsigned>((a.total + qcache::kThreads - 1) / qcache::kThreads);
  return launch_dependent(bf16 ? qcache::read_kernel<__nv_bfloat16> : qcache::read_kernel<float>, dim3(grid),
                          dim3(qcache::kThreads), 0, st, a);
}

}  // namespace bsa
