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

constexpr int kThreads = 256;          // reads
constexpr int kAppendThreads = 128;

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

// Largest magnitude of two or three values; NaN if one is NaN.
__device__ __forceinline__ float amax2(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
template <int GS>
__device__ __forceinline__ float group_amax(float m) {
#pragma unroll
  for (int o = GS / 2; o; o >>= 1) m = amax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The codes of a lane's 8 W bf16 values and the row's exponent byte; called by
// whole warps.  Rows with infinities or NaN take branches of their own: their
// selects would cost every row a third of its instructions.
template <int GS, int W>
__device__ __forceinline__ void quantise_row(const uint4 (&x)[W], uint32_t (&code)[2 * W], uint32_t& e) {
  float v[8 * W];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  float m = amax2(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < 8 * W; i += 2) m = amax3(m, v[i], v[i + 1]);
  m = group_amax<GS>(m);
  const bool broken = !(m < INFINITY);      // the same for the whole row
  const bool any_broken = __any_sync(0xffffffffu, broken);
  if (any_broken) {
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * W; ++i) f = fmaxf(f, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
    f = group_amax<GS>(f);
    if (broken) m = f;
  }
  e = exponent_byte(m);
  const uint64_t inv = f2_pack(two_to(254u - e), two_to(254u - e));
#pragma unroll
  for (int k = 0; k < 2 * W; ++k) {
    uint32_t two[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 t;
      f2_unpack(f2_mul(f2_pack(v[4 * k + 2 * i], v[4 * k + 2 * i + 1]), inv), t.x, t.y);
      two[i] = __nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
    }
    code[k] = two[0] | (two[1] << 16);
  }
  if (any_broken) {      // a conversion saturates infinities
#pragma unroll
    for (int i = 0; i < 8 * W; ++i)
      if (!(fabsf(v[i]) < INFINITY)) code[i >> 2] = (code[i >> 2] & ~(0xFFu << (8 * (i & 3)))) | 0x7Fu << (8 * (i & 3));
  }
}
template <int W>
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint32_t (&code)[2 * W]) {
  if constexpr (W == 2)
    *reinterpret_cast<uint4*>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
}

// One CTA per (sequence, KV head, touched block): the block's new tokens are
// quantised row by row (GS lanes a row, 8 W channels a lane, the next token's key
// and value on their way meanwhile), and if the append completes the block its mean key is summed
// from the codes, tokens ascending, fp32, one division -- from shared memory,
// which also takes the tokens that lay in the block before.  One launch, no
// block waits for another.
template <int GS, int W>
__global__ void __launch_bounds__(kAppendThreads, W == 2 ? 8 : 10) append_kernel(const QuantCacheArgs p) {
  griddep_wait();
  extern __shared__ uint4 smem_q[];
  uint8_t* codes = reinterpret_cast<uint8_t*>(smem_q);          // [64][d]
  __shared__ __align__(4) uint8_t exps[2][64];
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
  const bool complete = p.pooled != nullptr && L + n >= blk * 64 + 64;
  const int o0 = static_cast<int>(first & 63), rows = static_cast<int>(end - first);
  const int64_t src0 = static_cast<int64_t>(bg) * p.T + (first - L);
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS, c0 = 8 * W * l;
  const bool on = c0 < p.d;
  constexpr int kGroups = kAppendThreads / GS;
  const __nv_bfloat16* src[2] = {static_cast<const __nv_bfloat16*>(p.k_new) + src0 * p.d + c0,
                                 static_cast<const __nv_bfloat16*>(p.v_new) + src0 * p.d + c0};
  uint4 x[2][W], nx[2][W];
  auto load = [&](uint4 (&y)[2][W], int t) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int k = 0; k < W; ++k)
        y[kv][k] = t < rows && on ? __ldg(reinterpret_cast<const uint4*>(src[kv] + t * p.d + 8 * k))
                                  : make_uint4(0, 0, 0, 0);
  };
  load(x, grp);       // the first rows are on their way while the page is looked up
  const int page = blk < p.table_stride ? p.table[static_cast<int64_t>(b) * p.table_stride + blk] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.status, BSA_DEV_BAD_INDEX);
    return;
  }
  const int64_t page_row = (static_cast<int64_t>(page) * p.Hkv + g) * 64;
  uint8_t* dst[2] = {p.k_pool + (page_row + o0) * p.d + c0, p.v_pool + (page_row + o0) * p.d + c0};
  for (int t0 = 0; t0 < rows; t0 += kGroups) {       // whole warps: rows past the last are zeros, and not stored
    const int t = t0 + grp;
    load(nx, t + kGroups);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t e, code[2 * W];
      quantise_row<GS, W>(x[kv], code, e);
      if (!on || t >= rows) continue;
      store_codes<W>(dst[kv] + t * p.d, code);
      if (l == 0) exps[kv][o0 + t] = static_cast<uint8_t>(e);
      if (kv == 0 && complete) store_codes<W>(codes + (o0 + t) * p.d + c0, code);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int k = 0; k < W; ++k) x[kv][k] = nx[kv][k];
  }
  if (complete) {   // the tokens that lay in this block before (positions [0, o0) of it)
    for (int t = threadIdx.x; t < o0 * (p.d / 8); t += kAppendThreads)
      reinterpret_cast<uint2*>(codes)[t] = reinterpret_cast<const uint2*>(p.k_pool + page_row * p.d)[t];
    for (int t = threadIdx.x; t < o0; t += kAppendThreads) exps[0][t] = p.k_exp[page_row + t];
  }
  __syncthreads();
  {   // the new rows' exponents, together
    static_assert(kAppendThreads == 128, "a thread writes one of the block's 2 x 64 exponents");
    const int kv = threadIdx.x >> 6, o = threadIdx.x & 63;
    if (o >= o0 && o < o0 + rows) (kv ? p.v_exp : p.k_exp)[page_row + o] = exps[kv][o];
  }
  if (!complete) return;
  // four channels a thread: a product is exact, so the fused form rounds each sum once, as the pooling does
  for (int ch = 4 * threadIdx.x; ch < p.d; ch += 4 * kAppendThreads) {
    uint64_t s01 = 0, s23 = 0;
#pragma unroll 4
    for (int t0 = 0; t0 < 64; t0 += 4) {
      const uint32_t es = *reinterpret_cast<const uint32_t*>(&exps[0][t0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t four = *reinterpret_cast<const uint32_t*>(codes + (t0 + i) * p.d + ch);
        const float scale = __uint_as_float((i < 3 ? es << (23 - 8 * i) : es >> 1) & 0x7F800000u);
        const uint64_t sc = f2_pack(scale, scale);
        const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(four & 0xFFFFu, __NV_E4M3)));
        const float2 c = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(four >> 16, __NV_E4M3)));
        s01 = f2_fma(f2_pack(a.x, a.y), sc, s01);
        s23 = f2_fma(f2_pack(c.x, c.y), sc, s23);
      }
    }
    float4 v;
    f2_unpack(s01, v.x, v.y);
    f2_unpack(s23, v.z, v.w);
    *reinterpret_cast<float4*>(p.pooled + (static_cast<int64_t>(bg) * p.table_stride + blk) * p.d + ch) =
        make_float4(__fdiv_rn(v.x, 64.0f), __fdiv_rn(v.y, 64.0f), __fdiv_rn(v.z, 64.0f), __fdiv_rn(v.w, 64.0f));
  }
}

// Tokens starts[b] + t of every sequence and head, t < T and below the
// sequence's length, as bf16 (exact) or fp32 rows; other output rows are left
// as they were.  One CTA per 64 output rows of a (sequence, head); GS lanes a
// row, eight channels a lane, its keys and values of two rows in flight (a read of
// 16K-token contexts: 50.3 us; four rows 61.6, 16 channels a lane 57.6 us -- the
// registers cost more occupancy than they bring loads).
template <typename T, int GS>
__global__ void __launch_bounds__(kThreads) read_kernel(const QuantCacheArgs p) {
  griddep_wait();
  constexpr int kGroups = kThreads / GS, kFlight = 2;
  const int tile = blockIdx.x % p.touched;
  const int bg = blockIdx.x / p.touched;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  const int64_t start = p.starts ? p.starts[b] : 0;
  const int t_end = static_cast<int>(
      min(min(static_cast<int64_t>(p.T), p.seq_lens[b] - start), static_cast<int64_t>(tile) * 64 + 64));
  const int c0 = 8 * (threadIdx.x % GS), grp = threadIdx.x / GS;
  if (c0 >= p.d) return;
  for (int t0 = tile * 64 + grp; t0 < t_end; t0 += kGroups * kFlight) {
    uint2 code[2][kFlight];
    uint32_t e[2][kFlight];
    bool ok[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int t = t0 + u * kGroups;
      const int64_t pos = start + t, blk = pos >> 6;
      int page = -1;
      ok[u] = false;
      if (t < t_end) {
        if (pos >= 0 && blk < p.table_stride) page = __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + blk);
        ok[u] = page >= 0 && page < p.num_pages;
        if (!ok[u]) atomicOr(p.status, BSA_DEV_BAD_INDEX);
      }
      const int64_t src = (static_cast<int64_t>(page) * p.Hkv + g) * 64 + (pos & 63);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!ok[u] || (kv ? p.v_out : p.k_out) == nullptr) continue;
        code[kv][u] = __ldg(reinterpret_cast<const uint2*>((kv ? p.v_pool : p.k_pool) + src * p.d + c0));
        e[kv][u] = __ldg((kv ? p.v_exp : p.k_exp) + src);
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        T* out = static_cast<T*>(kv ? p.v_out : p.k_out);
        if (!ok[u] || out == nullptr) continue;
        T* dst = out + (static_cast<int64_t>(bg) * p.T + t0 + u * kGroups) * p.d + c0;
        float v[8];
        decode8(code[kv][u], two_to(e[kv][u]), v);
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
          reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_read(const QuantCacheArgs& a, unsigned grid, cudaStream_t st) {
  auto kernel = a.d <= 64 ? read_kernel<T, 8> : (a.d <= 128 ? read_kernel<T, 16> : read_kernel<T, 32>);
  return launch_dependent(kernel, dim3(grid), dim3(kThreads), 0, st, a);
}

}  // namespace qcache

cudaError_t launch_quant_append(QuantCacheArgs a, cudaStream_t st) {
  // an append of T tokens touches at most this many blocks of a sequence
  a.touched = static_cast<int>((a.T + 62ll) / 64 + 1);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hkv * a.touched);
  const size_t smem = 64 * static_cast<size_t>(a.d);
  // 16 channels a lane where the width allows it: half of the shuffles and exponents a channel (append of 8K prompts,
  // d = 128: 33.5 us against 37.3 with 8 channels a lane)
  auto kernel = qcache::append_kernel<32, 1>;
  if (a.d % 16 == 0)
    kernel = a.d <= 64 ? qcache::append_kernel<4, 2> : (a.d <= 128 ? qcache::append_kernel<8, 2> : qcache::append_kernel<16, 2>);
  else if (a.d <= 128)
    kernel = a.d <= 64 ? qcache::append_kernel<8, 1> : qcache::append_kernel<16, 1>;
  return launch_dependent(kernel, dim3(grid), dim3(qcache::kAppendThreads), smem, st, a);
}

cudaError_t launch_quant_read(QuantCacheArgs a, bool bf16, cudaStream_t st) {
  a.touched = static_cast<int>((a.T + 63ll) / 64);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hkv * a.touched);
  return bf16 ? qcache::launch_read<__nv_bfloat16>(a, grid, st) : qcache::launch_read<float>(a, grid, st);
}

}  // namespace bsa
